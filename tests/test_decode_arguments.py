"""More of what the decoding calls refuse and accept, without a GPU: what
passes every check ends at the missing device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from test_decode_host import BF16, FAKE, INVALID, LAUNCH, MB, _cache, _state, lib  # noqa: E402,F401

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


@needs_no_gpu
@pytest.mark.parametrize("page_size,max_pages,ok", [(1, 2 ** 31 - 1, False), (16, 2 ** 27 - 1, False), (2 ** 31 - 1, 1, False),
                                                    (64, (2 ** 31 - 1024) // 64, True), (1, 2 ** 31 - 1024, True)])
def test_tree_attention_capacity(lib, page_size, max_pages, ok):
    """The kernel counts tokens in 32 bits and looks up to a few tiles past the last: a capacity within 1023 of 2^31
    would wrap, and read past the block table."""
    from top_logit_filter_gb300 import _lib
    a = _lib.TreeAttentionArgs(q=FAKE, out=FAKE + MB, k=_cache(dt=BF16, exp=None, tok=64, head=64, page=64),
                               v=_cache(data=FAKE + (1 << 40), dt=BF16, exp=None, tok=64, head=64, page=64),
                               table=FAKE + (1 << 44), context=FAKE + 3 * MB, workspace=FAKE + (1 << 42),
                               workspace_bytes=1 << 40, B=1, T=1, Hq=1, Hkv=1, D=64, pages=8, page_size=page_size,
                               max_pages=max_pages, ld_table=max_pages, max_context=64, q_batch_stride=64, q_token_stride=64,
                               q_head_stride=64, out_batch_stride=64, out_token_stride=64, out_head_stride=64, dtype=BF16, scale=0.125)
    st, why = lib.topkp_tree_attention(ctypes.byref(a), None), lib.topkp_last_error_string().decode()
    assert (st == LAUNCH and "device" in why) if ok else (st == INVALID and "page" in why), (st, why)
