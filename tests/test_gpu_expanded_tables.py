"""One row of a block table, expanded, serves all requests of an attention call."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_shared import tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 6])
def test_one_row_for_all_requests(tk, B):  # noqa: F811
    g = torch.Generator().manual_seed(B)
    k, v = (torch.randn(24, 16, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in (0, 1))
    q = torch.randn(B, 3, 4, 64, generator=g).to(torch.bfloat16).cuda()
    context = (300 + torch.arange(B)).int().cuda()
    row = torch.randperm(24, generator=g)[:22].int().cuda()
    one = row.expand(B, 22)
    full = one.clone(memory_format=torch.contiguous_format)
    assert B == 1 or one.stride(0) == 0
    assert torch.equal(tk.tree_attention(q, k, v, context, pages=one), tk.tree_attention(q, k, v, context, pages=full))
    shared = torch.tensor([300], dtype=torch.int32).cuda()
    assert torch.equal(tk.shared_attention(q, k, v, context, one, shared), tk.shared_attention(q, k, v, context, full, shared))
