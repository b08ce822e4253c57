"""Shared attention's launches wait for one another, but not while they hold
tensor memory that the other may need."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_logit_filter_gb300", "csrc")


def test_tensor_memory_is_free_before_a_launch_waits_for_another():
    """A CTA that waits for the launch before it must not hold columns which a CTA of that launch may still ask for:
    tcgen05.alloc has no time limit."""
    with open(os.path.join(CSRC, "attention_tc.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    waits = [m.start() for m in re.finditer(r"griddepcontrol\.wait", text)]
    frees = [m.start() for m in re.finditer(r"tcgen05\.dealloc", text)]
    assert len(waits) == 1 and len(frees) == 1 and frees[0] < waits[0]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(8, 128), (1, 128), (2, 256)])
def test_beside_another_call_that_uses_tensor_memory(T, D):
    """Two streams: shared attention (a CTA of 256 rows takes all columns, as do heads of 256), and plain attention."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as tk
    g = torch.Generator().manual_seed(T + D)
    B, Hq, Hkv, P, L = 40, 8, 2, 16, 900
    M = -(-(L + 60 + T) // P)
    pool = B * M
    table = torch.randperm(pool, generator=g).view(B, M).int()
    table[:, :800 // P] = table[:1, :800 // P]
    table = torch.cat([table, torch.full((B, 2500), -1, dtype=torch.int32)], 1).cuda()    # (planned as if it were long)
    k, v = (torch.randn(pool, P, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in (0, 1))
    q = torch.randn(B, T, Hq, D, generator=g).to(torch.bfloat16).cuda()
    context = (L + torch.randint(0, 60, (B,), generator=g)).int().cuda()
    shared = torch.tensor([800], dtype=torch.int32).cuda()
    one = lambda: tk.shared_attention(q, k, v, context, table, shared, max_context=40000, max_shared=39000, want_lse=True)  # noqa: E731
    two = lambda: tk.tree_attention(q, k, v, context, pages=table, max_context=L + 60, want_lse=True)  # noqa: E731
    want = one()
    assert tk.last_launch_count() == 3
    plain = two()
    sides = [torch.cuda.Stream() for _ in (0, 1, 2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(sides[0]):
            a = one()
        with torch.cuda.stream(sides[1]):
            b = two()
        with torch.cuda.stream(sides[2]):
            c = one()
    torch.cuda.synchronize()
    tk.device_status()
    for got, ref in ((a, want), (b, plain), (c, want)):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
