"""How shared_attention splits its work where what a group shares is longer or
shorter than the bound that the call was planned by."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_shared import tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["own", "e4m3"])
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("shared,max_shared", [((11968, 6400, 0), 11968), ((11968, 64, 0), 3000)])
def test_no_part_takes_all_the_rest(tk, cache, T, shared, max_shared):  # noqa: F811
    """Keys of zeros: a part's log-sum, which the workspace holds behind the parts' rows, says how many tokens it took."""
    size, Hq, Hkv, D, P, L = 8, 4, 1, 128, 64, 16384
    G = len(shared)
    B, rows = G * size, G * size * T * Hq
    M = L // P + 1
    table = torch.arange(M, dtype=torch.int32).expand(B, M).contiguous().cuda()
    type_ = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    k, v = (torch.zeros(M, P, Hkv, D, device="cuda").to(type_) for _ in (0, 1))
    kw = {} if cache == "own" else {n: torch.full((M, P, Hkv), 127, dtype=torch.uint8, device="cuda") for n in ("k_exp", "v_exp")}
    q = torch.ones(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    context = torch.full((B,), L, dtype=torch.int32, device="cuda")
    bounds = dict(max_context=L, max_shared=max_shared)
    need = tk.shared_attention_workspace_size(q, k, table, G, **bounds)
    parts = need // (rows * (D + 1) * 4)
    assert need == parts * rows * (D + 1) * 4
    space = torch.zeros(need, dtype=torch.uint8, device="cuda")
    tk.shared_attention(q, k, v, context, table, torch.tensor(shared, dtype=torch.int32, device="cuda"), workspace=space, **kw, **bounds)
    assert tk.last_launch_count() == 3
    tk.device_status()
    lse = space.view(torch.float32)[parts * rows * D:].view(parts, B, T, Hq).cpu().double()
    took = torch.exp(lse).round().long()[:, :, 0, 0]      # [parts, B], of each request's first node, which sees itself too
    front = int((took[:, -1] > 0).int().argmax())         # the shared tokens' parts come first; the last group has none
    assert front >= 2 and parts - front >= 2
    for b in range(0, B, size):
        for some, total in ((took[:front, b], shared[b // size]), (took[front:, b], L + 1 - shared[b // size])):
            assert int(some.sum()) == total
            assert int(some.max()) == int(some[0]), (b, some.tolist())
