"""The calls for several continuations of one prompt without a GPU: each
refuses bad arguments with the library's status codes before it touches the
device; what passes every check ends at the missing device."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")
from test_decode_host import BF16, E4M3, F16, F32, FAKE, INVALID, LAUNCH, MB, NULLPTR, ROOT, _cache, lib  # noqa: E402,F401

GB = 1 << 30
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


def test_structures_are_those_of_the_header(tmp_path):
    import shutil
    import subprocess
    from top_logit_filter_gb300 import _lib
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "topkp_decode.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu", '
                   'sizeof(topkp_draft_verify_args), sizeof(topkp_pages), sizeof(topkp_cache_fork_args), offsetof(topkp_draft_verify_args, eps), '
                   'offsetof(topkp_cache_fork_args, grow_all), (size_t)TOPKP_MAX_ROWS); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(_lib.DraftVerifyArgs), ctypes.sizeof(_lib.Pages), ctypes.sizeof(_lib.CacheForkArgs),
                   _lib.DraftVerifyArgs.eps.offset, _lib.CacheForkArgs.grow_all.offset, _lib.TOPKP_MAX_ROWS]


@needs_no_gpu
def test_draft_verify(lib):  # noqa: F811
    from top_logit_filter_gb300 import _lib

    def call(**kw):
        a = dict(target=FAKE, draft=FAKE + 16 * MB, tokens=FAKE + 32 * MB, parent=FAKE + 33 * MB, nodes=FAKE + 34 * MB, uniform=FAKE + 35 * MB,
                 race=FAKE + 36 * MB, count=FAKE + 48 * MB, path=FAKE + 49 * MB, token=FAKE + 50 * MB, logprob=FAKE + 51 * MB, B=3, T=4,
                 V=1000, target_batch_stride=4000, target_node_stride=1000, draft_batch_stride=4000, draft_node_stride=1000, ld_race=1000,
                 dtype=BF16, eps=1e-10)
        a.update(kw)
        return lib.topkp_draft_verify(ctypes.byref(_lib.DraftVerifyArgs(**a)), None)
    assert lib.topkp_draft_verify(None, None) == NULLPTR
    assert call() == LAUNCH
    for ok in (dict(draft=None), dict(draft=None, uniform=None, race=None), dict(parent=None, nodes=None, logprob=None), dict(T=64, target_batch_stride=64000),
               dict(target_batch_stride=0), dict(T=1, target_node_stride=0), dict(B=1, ld_race=0), dict(dtype=F32), dict(dtype=F16, target=FAKE + 2)):
        assert call(**ok) == LAUNCH, ok
    for bad in (dict(dtype=E4M3), dict(dtype=7), dict(B=-1), dict(B=1 << 28), dict(V=0), dict(V=(1 << 23) + 1), dict(T=0), dict(T=65), dict(uniform=None),
                dict(race=None), dict(uniform=None, race=None), dict(eps=-1.0), dict(eps=float("nan")), dict(target_node_stride=999),
                dict(target_batch_stride=-1), dict(draft_node_stride=999), dict(draft_batch_stride=-1), dict(ld_race=999), dict(target=FAKE + 1),
                dict(draft=FAKE + 16 * MB + 1), dict(tokens=FAKE + 32 * MB + 2), dict(parent=FAKE + 33 * MB + 1), dict(race=FAKE + 36 * MB + 2),
                dict(count=FAKE + 48 * MB + 2), dict(logprob=FAKE + 51 * MB + 1), dict(count=FAKE + 2000), dict(path=FAKE + 16 * MB), dict(token=FAKE + 36 * MB),
                dict(logprob=FAKE + 35 * MB), dict(path=FAKE + 48 * MB), dict(token=FAKE + 49 * MB + 4)):
        assert call(**bad) == INVALID, bad
        assert b"draft_verify" in lib.topkp_last_error_string()
    for bad in (dict(target=None), dict(tokens=None), dict(count=None), dict(path=None), dict(token=None)):
        assert call(**bad) == NULLPTR, bad
    assert call(B=0) == 0 and call(B=0, target=None, tokens=None) == 0 and lib.topkp_last_launch_count() == 0


def _pages(lib, data=FAKE, page=4096, block=4096, blocks=1, entry=256):  # noqa: F811
    from top_logit_filter_gb300 import _lib
    return _lib.Pages(data, page, block, blocks, entry)


@needs_no_gpu
def test_cache_fork(lib):  # noqa: F811
    from top_logit_filter_gb300 import _lib

    def call(*states, count=None, **kw):
        arr = (_lib.Pages * max(len(states), 1))(*states)
        a = dict(states=ctypes.addressof(arr), table=FAKE + GB, lengths=FAKE + GB + MB, source=FAKE + GB + 2 * MB, grow=FAKE + GB + 3 * MB,
                 refs=FAKE + GB + 4 * MB, table_out=FAKE + GB + 5 * MB, refs_out=FAKE + GB + 6 * MB, missing=FAKE + GB + 7 * MB,
                 workspace=FAKE + GB + 8 * MB, workspace_bytes=1 << 20, count=len(states) if count is None else count, R=3, N=5, max_pages=7,
                 ld_table=7, ld_out=9, pages=100, page_size=16, grow_all=0)
        a.update(kw)
        return lib.topkp_cache_fork(ctypes.byref(_lib.CacheForkArgs(**a)), None)
    one = _pages(lib)
    assert lib.topkp_cache_fork(None, None) == NULLPTR
    assert call(one) == LAUNCH and call() == LAUNCH
    for ok in (dict(grow=None, grow_all=3), dict(N=0, source=None, table_out=None), dict(R=0, table=None, lengths=None), dict(refs_out=FAKE + GB + 4 * MB),
               dict(R=8192, N=8192, max_pages=8)):
        ok = dict(ok)
        if ok.get("R") == 8192:
            ok.update(ld_table=8, table_out=FAKE + 2 * GB, workspace=FAKE + 3 * GB)
            ok["source"], ok["lengths"], ok["grow"] = FAKE + GB + 2 * MB, FAKE + GB + MB, None
        assert call(one, **ok) == LAUNCH, (ok, lib.topkp_last_error_string())
    for bad in (dict(count=-1), dict(R=-1), dict(N=-1), dict(R=8193), dict(N=8193), dict(pages=0), dict(pages=1 << 31), dict(page_size=0),
                dict(max_pages=0), dict(ld_table=6), dict(ld_out=6), dict(grow_all=-1), dict(max_pages=1 << 29, ld_table=1 << 29, ld_out=1 << 29),
                dict(page_size=1 << 30), dict(table=FAKE + GB + 2), dict(missing=FAKE + GB + 7 * MB + 1), dict(workspace=None), dict(workspace_bytes=100),
                dict(workspace=FAKE + GB + 8 * MB + 4), dict(table_out=FAKE + GB), dict(table_out=FAKE + GB + 8), dict(refs_out=FAKE + GB + 4 * MB + 4),
                dict(missing=FAKE + GB + 4 * MB), dict(missing=FAKE + GB + 6 * MB + 8), dict(refs_out=FAKE + GB + MB), dict(workspace=FAKE + GB + 6 * MB)):
        assert call(one, **bad) == INVALID, bad
    for bad in (dict(states=None), dict(table=None), dict(lengths=None), dict(source=None), dict(refs=None), dict(table_out=None), dict(refs_out=None),
                dict(missing=None)):
        assert call(one, **bad) == NULLPTR, bad
    for state in (_pages(lib, entry=-1), _pages(lib, blocks=-1), _pages(lib, page=-4096), _pages(lib, block=-1, blocks=2), _pages(lib, page=4095),
                  _pages(lib, blocks=2, block=4095, page=1 << 20), _pages(lib, blocks=2, page=8191), _pages(lib, data=FAKE + GB - 64),
                  _pages(lib, entry=1 << 40, page=1 << 50)):
        assert call(state) == INVALID, (state.data, state.page_stride)
    assert call(_pages(lib, data=None)) == NULLPTR
    # nothing to move: no address is looked at
    assert call(_pages(lib, data=None, blocks=0)) == LAUNCH and call(_pages(lib, data=None, entry=0)) == LAUNCH
    # states between each other's pages, and over each other
    pair = [_pages(lib, data=FAKE + i * 4096, page=8192) for i in (0, 1)]
    assert call(*pair) == LAUNCH and call(*pair, pair[0]) == INVALID
    assert call(_pages(lib), _pages(lib, data=FAKE + 100 * 4096 - 1)) == INVALID
    assert call(*[_pages(lib, data=FAKE + i * 409600) for i in range(300)]) == LAUNCH
    assert b"share a byte" not in lib.topkp_last_error_string()
    assert lib.topkp_cache_fork_workspace_size(8193, 10) == 0 and lib.topkp_cache_fork_workspace_size(4, 0) == 0
    assert lib.topkp_cache_fork_workspace_size(5, 100) == 3 * 512 + 256


@needs_no_gpu
def test_cache_compact(lib):  # noqa: F811
    from top_logit_filter_gb300 import _lib

    def call(*states, count=None, B=3, W=5, table=FAKE + GB, ld=7, M=7, pages=100, P=16, start=FAKE + GB + MB, keep=FAKE + GB + 2 * MB,
             kept=FAKE + GB + 3 * MB):
        arr = (_lib.Pages * max(len(states), 1))(*states)
        return lib.topkp_cache_compact(arr, len(states) if count is None else count, B, W, table, ld, M, pages, P, start, keep, kept, None)
    one = _pages(lib)
    assert call(one) == LAUNCH and call(one, table=None, M=1, pages=3) == LAUNCH
    assert call() == 0 and call(one, B=0) == 0 and call(one, W=0) == 0
    for bad in (dict(count=-1), dict(B=-1), dict(B=65536), dict(W=65), dict(W=-1), dict(ld=6), dict(M=0), dict(pages=0), dict(P=0), dict(table=None),
                dict(table=None, M=1, pages=4), dict(start=FAKE + GB + MB + 2), dict(table=FAKE + GB + 1), dict(keep=FAKE + GB + 2 * MB + 1),
                dict(start=FAKE + 64), dict(keep=FAKE + 4096 * 99)):
        assert call(one, **bad) == INVALID, bad
    for bad in (dict(start=None), dict(keep=None), dict(kept=None)):
        assert call(one, **bad) == NULLPTR, bad
    assert call(one, one) == INVALID and call(_pages(lib, data=None)) == NULLPTR


@needs_no_gpu
def test_shared_attention(lib):  # noqa: F811
    from top_logit_filter_gb300 import _lib

    def args(**kw):
        a = dict(q=FAKE, out=FAKE + MB, lse=None, k=_cache(dt=BF16, exp=None), v=_cache(data=FAKE + 48 * MB, dt=BF16, exp=None),
                 table=FAKE + 2 * MB, context=FAKE + 3 * MB, nodes=None, tree=None, workspace=FAKE + GB, workspace_bytes=1 << 33, B=6, T=4, Hq=8,
                 Hkv=4, D=64, pages=8, page_size=16, max_pages=4, ld_table=4, max_context=64, q_batch_stride=2048, q_token_stride=512,
                 q_head_stride=64, out_batch_stride=2048, out_token_stride=512, out_head_stride=64, dtype=BF16, scale=0.125)
        a.update(kw)
        return _lib.TreeAttentionArgs(**a)

    def call(shared=FAKE + 5 * MB, groups=2, most=64, **kw):
        return lib.topkp_shared_attention(ctypes.byref(args(**kw)), shared, groups, most, None)
    assert lib.topkp_shared_attention(None, FAKE, 1, 0, None) == NULLPTR
    assert call() == LAUNCH and call(groups=6) == LAUNCH and call(groups=1, most=-5) == LAUNCH
    assert call(groups=0) == INVALID and call(groups=4) == INVALID and call(groups=-2) == INVALID
    assert call(shared=None) == NULLPTR and call(table=None, pages=6, max_pages=1) == NULLPTR
    assert call(shared=FAKE + 5 * MB + 2) == INVALID
    assert call(shared=FAKE + MB) == INVALID                 # the output over it
    assert call(D=60) == INVALID and call(tree=FAKE + 4 * MB, T=65) == INVALID and call(q=None) == NULLPTR
    assert call(B=0) == 0 and call(T=0) == 0
    long = dict(B=60, max_context=60000, max_pages=4096, ld_table=4096, page_size=16)
    a = args(**long)
    need = lib.topkp_shared_attention_workspace_size(ctypes.byref(a), 2, 59000)
    # parts of the shared tokens and of the own: rows of 64 values and a log-sum each
    assert need > 0 and need % (60 * 4 * 8 * 65 * 4) == 0 and need // (60 * 4 * 8 * 65 * 4) >= 2
    assert call(most=59000, workspace_bytes=need - 1, **long) == INVALID and call(most=59000, workspace=None, **long) == INVALID
    assert call(most=59000, workspace_bytes=need, **long) == LAUNCH
    # one request a group, nothing shared, or too little to be worth it: each by itself
    alone = lib.topkp_tree_attention_workspace_size(ctypes.byref(a))
    assert lib.topkp_shared_attention_workspace_size(ctypes.byref(a), 60, 59000) == alone
    assert lib.topkp_shared_attention_workspace_size(ctypes.byref(a), 2, 63) == alone
    assert lib.topkp_shared_attention_workspace_size(ctypes.byref(a), 7, 59000) == 0
    assert lib.topkp_shared_attention_workspace_size(None, 1, 1) == 0
    # rows of a group are counted in 32 bits
    assert call(groups=1, B=2048, T=65535 * 4, Hkv=4, Hq=8, q_batch_stride=1 << 30, out_batch_stride=1 << 30, out=FAKE + (1 << 45),
                workspace=FAKE + (1 << 50), workspace_bytes=1 << 49) == INVALID


def test_python_faces_refuse():
    import top_logit_filter_gb300 as tk
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        tk.draft_verify(torch.zeros(1, 2, 8), i32(1, 2))
    with pytest.raises(ValueError):
        tk.cache_fork([torch.zeros(4, 2, 8)], i32(1, 2), i32(1), i32(1), i32(4))
    with pytest.raises(ValueError):
        tk.cache_compact([torch.zeros(4, 2, 8)], i32(1), i32(1, 2), i32(1))
    with pytest.raises(ValueError):
        tk.shared_attention(torch.zeros(1, 1, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), i32(1), i32(1, 1), i32(1))


def test_states_of_one_shape_lie_alike():
    """The descriptors of a list of tensors, whatever precedes a tensor in it (no device needed)."""
    import struct
    from top_logit_filter_gb300 import decode
    decode._ready()
    a, b = torch.zeros(6, 4, 2, 8), torch.zeros(6, 4, 2, 8)
    both = torch.zeros(6, 2, 4, 3, 5, dtype=torch.uint8)
    some = [a, b, both[:, 0], both[:, 1], torch.zeros(6, 4, 2, 8, dtype=torch.float16), a, torch.zeros(6, 4, dtype=torch.uint8), torch.zeros(6, 4, 2, 8)[..., :8]]
    many, packed, pages, page_size = decode._page_states(some, 1, torch.device("cpu"))
    assert (pages, page_size) == (6, 4) and len(many) == 8
    for i, t in enumerate(some):
        row, blk, blocks, _, size = decode._layout(t, 1, "t")
        assert struct.unpack_from("=Q4q", packed, 40 * i) == (t.data_ptr(), row, blk, blocks, size)
    for bad in ([a, torch.zeros(6, 5, 2, 8)], [a, torch.zeros(5, 4, 2, 8)], [torch.zeros(6)], [a[..., :4]], [a, 3]):
        with pytest.raises(ValueError):
            decode._page_states(bad, 1, torch.device("cpu"))
    _, packed, pages, page_size = decode._page_states(torch.zeros(6, 3, 4, 8), 2, torch.device("cpu"))
    assert (pages, page_size) == (6, 4) and struct.unpack("=Q4q", packed)[1:] == (384, 128, 3, 32)
