"""Tensors expanded over a dimension (a stride of zero) are read like any others."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_verify import check, make, tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["ratio", "certain", "greedy"])
@pytest.mark.parametrize("V", [5, 1003])
@pytest.mark.parametrize("requests", [4, 1])
def test_verify_of_one_row_for_all_nodes(tk, mode, V, requests):  # noqa: F811
    """Of each request, and of all of them."""
    d, device = make(4, 5, V, "bf16", mode, True, seed=31 + V), {}
    for name in ("target", "draft"):
        if d[name] is not None:
            device[name] = d[name][:requests, :1].cuda().expand(4, 5, V)
            assert device[name].stride(1) == 0
            d[name] = device[name].cpu().contiguous()
    check(tk, d, device=device)
