"""A caller's workspace has to have its bytes in one piece: an expanded or
strided tensor counts more elements than there is memory behind them."""
import pytest

torch = pytest.importorskip("torch")


def bad(device):
    yield torch.empty(1, dtype=torch.uint8, device=device).expand(1 << 24)
    yield torch.empty((1, 1 << 12), dtype=torch.uint8, device=device).expand(1 << 12, 1 << 12)
    yield torch.empty(1 << 25, dtype=torch.uint8, device=device)[::2]
    yield torch.empty((1 << 12, 1 << 13), dtype=torch.uint8, device=device)[:, :1 << 12]


def test_only_whole_tensors():
    from top_logit_filter_gb300 import _workspace
    cpu = torch.device("cpu")
    for w in bad(cpu):
        assert w.numel() >= 1 << 24
        with pytest.raises(ValueError, match="contiguous uint8"):
            _workspace(w, 1 << 24, cpu)
    for w in (torch.empty(99, dtype=torch.uint8), torch.empty(400, dtype=torch.float32), 5):
        with pytest.raises(ValueError, match="contiguous uint8"):
            _workspace(w, 100, cpu)
    whole = torch.empty(100, dtype=torch.uint8)
    assert _workspace(whole, 100, cpu) is whole and _workspace(whole.view(10, 10), 100, cpu).numel() == 100
    assert _workspace(None, 0, cpu).numel() == 1


@pytest.mark.gpu
def test_every_call_refuses():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as tk
    x = torch.randn(4, 1000, device="cuda")
    q = torch.randn(1, 1, 4, 64, device="cuda").half()
    cache = torch.randn(1, 9000, 1, 64, device="cuda").half()
    context = torch.tensor([8000], dtype=torch.int32, device="cuda")
    for w in bad("cuda"):
        for call in (lambda: tk.sort(x, workspace=w), lambda: tk.sample_v2(x, workspace=w),
                     lambda: tk.beam_select(x, torch.zeros(2, 2, device="cuda"), 4, workspace=w),
                     lambda: tk.tree_attention(q, cache, cache, context, workspace=w)):
            with pytest.raises(ValueError, match="contiguous uint8"):
                call()
