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


def test_sizes_are_offered():
    import top_logit_filter_gb300 as tk
    from top_logit_filter_gb300 import build
    build.build()
    assert tk.beam_select_workspace_size(2, 4, 1000, torch.float16, 8) > 0
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    q = torch.empty(1, 1, 8, 64, dtype=bf)
    for kind in (bf, e4):
        long = torch.empty(600, 16, 2, 64, dtype=torch.uint8 if kind is e4 else kind)
        long = long.view(kind) if kind is e4 else long
        table = torch.empty(1, 600, dtype=torch.int32)
        need = tk.tree_attention_workspace_size(q, long, table)
        # parts of [1, 1, 8] rows of 64 values and a log-sum each
        assert need > 0 and need % (8 * 65 * 4) == 0
        assert tk.tree_attention_workspace_size(q, long, table, max_context=10) == 0
    assert tk.tree_attention_workspace_size(q, torch.empty(1, 32, 2, 64, dtype=bf)) == 0


@pytest.mark.gpu
def test_sizes_are_enough():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as tk
    q = torch.randn(1, 2, 8, 64, device="cuda").half()
    cache = torch.randn(1, 9000, 2, 64, device="cuda").half()
    context = torch.tensor([8000], dtype=torch.int32, device="cuda")
    need = tk.tree_attention_workspace_size(q, cache)
    given = tk.tree_attention(q, cache, cache, context, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(given, tk.tree_attention(q, cache, cache, context))
    with pytest.raises(ValueError, match="workspace"):
        tk.tree_attention(q, cache, cache, context, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    x, s = torch.randn(4, 1000, device="cuda"), torch.zeros(2, 2, device="cuda")
    work = torch.empty(tk.beam_select_workspace_size(2, 2, 1000, x.dtype, 5), dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(tk.beam_select(x, s, 5, workspace=work), tk.beam_select(x, s, 5)))
