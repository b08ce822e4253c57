"""The decoding calls without a GPU: include/topkp_decode.h's entry points
are exported, and each refuses bad arguments with the library's status codes
before it touches the device."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, F16, BF16, E4M3 = 0, 1, 2, 3
NULLPTR, INVALID, LAUNCH = 161001, 161002, 561000
FAKE = 1 << 20
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from top_logit_filter_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_exports_match_the_header(lib):
    from top_logit_filter_gb300 import _lib
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "topkp_decode.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(topkp_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(_lib.DECODE_EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


def test_header_is_c(tmp_path):
    """include/topkp_decode.h compiles as C99, and its structures are those of the binding."""
    import shutil
    import subprocess
    from top_logit_filter_gb300 import _lib
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "topkp_decode.h"\nint main(void) { printf("%zu %zu %zu", sizeof(topkp_state), '
                   'sizeof(topkp_cache), sizeof(topkp_tree_attention_args)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(t) for t in (_lib.State, _lib.Cache, _lib.TreeAttentionArgs)]


def test_beam_select_refusals(lib):
    def call(x=FAKE, B=2, K=3, V=8, ld=8, dt=BF16, sc=FAKE + MB, fin=None, pad=0, n=4, o=(2, 3, 4), ws=5, wn=1 << 16):
        outs = [None if i is None else FAKE + i * MB for i in o]
        return lib.topkp_beam_select(x, B, K, V, ld, dt, sc, fin, pad, n, *outs, FAKE + ws * MB if isinstance(ws, int) else ws, wn, None)
    assert call(dt=3) == INVALID
    assert call(B=-1) == INVALID
    assert call(V=0) == INVALID and call(V=(1 << 23) + 1, ld=1 << 24) == INVALID
    assert call(K=0) == INVALID and call(K=65) == INVALID
    assert call(n=0) == INVALID and call(n=129) == INVALID
    assert call(pad=8) == INVALID and call(pad=-1) == INVALID
    assert call(x=None) == NULLPTR and call(sc=None) == NULLPTR
    assert call(o=(2, None, 4)) == NULLPTR and call(ws=None) == NULLPTR
    assert call(ld=7) == INVALID
    assert call(x=FAKE + 1) == INVALID and call(sc=FAKE + MB + 2) == INVALID
    assert call(wn=16) == INVALID
    assert b"workspace" in lib.topkp_last_error_string()
    assert call(o=(0, 3, 4)) == INVALID              # an output over the logits
    assert call(o=(2, 2, 4)) == INVALID              # two outputs in one place
    assert call(fin=FAKE + 5 * MB) == INVALID        # finished inside the workspace
    assert call(B=0) == 0 and call(B=0, x=None) == 0
    assert lib.topkp_beam_select_workspace_size(0, 3, 8, BF16, 4) == 0
    assert lib.topkp_beam_select_workspace_size(2, 3, 8, BF16, 4) > 0


def _state(lib, src=FAKE, dst=FAKE, row=1024, drow=None, blk=1024, dblk=None, blocks=1, entries=8, size=128):
    from top_logit_filter_gb300 import _lib
    return _lib.State(src, dst, row, row if drow is None else drow, blk, blk if dblk is None else dblk, blocks, entries, size)


def test_beam_reorder_refusals(lib):
    from top_logit_filter_gb300 import _lib

    def call(*states, B=2, K=2, parent=FAKE + 8 * MB, lengths=None, count=None):
        arr = (_lib.State * max(len(states), 1))(*states)
        return lib.topkp_beam_reorder(arr, len(states) if count is None else count, B, K, parent, lengths, None)
    ok = _state(lib)
    assert call(ok, K=0) == INVALID and call(ok, K=65) == INVALID
    assert call(ok, B=-1) == INVALID and call(count=-1) == INVALID
    assert call(ok, parent=None) == NULLPTR
    assert call(ok, parent=FAKE + 8 * MB + 2) == INVALID
    assert call(_state(lib, src=None)) == NULLPTR
    assert call(_state(lib, entries=-1)) == INVALID
    assert call(_state(lib, row=512)) == INVALID                       # rows overlap
    assert call(_state(lib, blocks=2, blk=512, row=4096)) == INVALID   # blocks overlap
    assert call(_state(lib, drow=2048)) == INVALID                     # in place with two layouts
    assert call(_state(lib, dst=FAKE + 512)) == INVALID                # partly over its source
    assert call(ok, _state(lib, src=FAKE + 64 * MB, dst=FAKE)) == INVALID   # written over another state
    assert call(ok, parent=FAKE + 1024) == INVALID                     # a state over parent
    assert call(ok, B=0) == 0 and call() == 0
    assert call(_state(lib, entries=0)) in (0, LAUNCH)


def _cache(data=FAKE + 16 * MB, exp=FAKE + 32 * MB, dt=E4M3, page=4096, tok=256, head=64, eps=64, ets=4, ehs=1):
    from top_logit_filter_gb300 import _lib
    return _lib.Cache(data, exp, dt, page, tok, head, eps, ets, ehs)


def test_cache_refusals(lib):
    def write(k=FAKE, v=FAKE + MB, N=5, H=4, D=64, ts=256, hs=64, dt=BF16, slots=FAKE + 2 * MB, kc=None, vc=0, pages=8, P=16):
        kc = _cache() if kc is None else kc
        vc = _cache(data=FAKE + 48 * MB, exp=FAKE + 64 * MB) if vc == 0 else vc
        return lib.topkp_cache_write(k, v, N, H, D, ts, hs, ts, hs, dt, slots, ctypes.byref(kc),
                                     ctypes.byref(vc) if vc is not None else None, pages, P, None)

    def read(k=FAKE, v=FAKE + MB, N=5, H=4, D=64, dt=BF16, slots=FAKE + 2 * MB, kc=None, vc=0, pages=8, P=16):
        kc = _cache() if kc is None else kc
        vc = _cache(data=FAKE + 48 * MB, exp=FAKE + 64 * MB) if vc == 0 else vc
        return lib.topkp_cache_read(slots, N, H, D, ctypes.byref(kc), ctypes.byref(vc) if vc is not None else None,
                                    pages, P, dt, k, v, None)
    for call in (write, read):
        assert call(dt=7) == INVALID
        assert call(N=-1) == INVALID and call(D=0) == INVALID and call(D=257) == INVALID
        assert call(pages=0) == INVALID and call(P=0) == INVALID
        assert call(k=None) == NULLPTR and call(slots=None) == NULLPTR
        assert call(v=None) == NULLPTR and call(vc=None) == NULLPTR    # v and v_cache go together
        assert call(kc=_cache(data=None)) == NULLPTR
        assert call(kc=_cache(exp=None)) == NULLPTR
        assert call(kc=_cache(dt=BF16)) == INVALID                     # exponents of a bf16 cache
        assert call(kc=_cache(dt=F16, exp=None)) == INVALID            # neither the rows' type nor e4m3
        assert call(kc=_cache(tok=32)) == INVALID and call(kc=_cache(page=-1)) == INVALID
        assert call(kc=_cache(dt=BF16, exp=None, tok=256), vc=_cache(data=FAKE + 48 * MB, exp=FAKE + 64 * MB)) == INVALID
        assert call(slots=FAKE + 2 * MB + 4) == INVALID
        assert call(k=FAKE + 16 * MB + 128) == INVALID                 # rows inside a cache
        assert call(N=0) == 0 and call(N=0, k=None) == 0
    assert read(v=FAKE + 64) == INVALID                                # outputs overlap
    assert read(slots=FAKE + 8) == INVALID


def test_tree_attention_refusals(lib):
    from top_logit_filter_gb300 import _lib

    def args(**kw):
        a = dict(q=FAKE, out=FAKE + MB, lse=None, k=_cache(dt=BF16, exp=None), v=_cache(data=FAKE + 48 * MB, dt=BF16, exp=None),
                 table=FAKE + 2 * MB, context=FAKE + 3 * MB, nodes=None, tree=FAKE + 4 * MB, workspace=FAKE + 128 * MB,
                 workspace_bytes=1 << 30, B=2, T=4, Hq=8, Hkv=4, D=64, pages=8, page_size=16, max_pages=4, ld_table=4,
                 max_context=64, q_batch_stride=2048, q_token_stride=512, q_head_stride=64, out_batch_stride=2048,
                 out_token_stride=512, out_head_stride=64, dtype=BF16, scale=0.125)
        a.update(kw)
        return _lib.TreeAttentionArgs(**a)

    def call(**kw):
        a = args(**kw)
        return lib.topkp_tree_attention(ctypes.byref(a), None)
    assert lib.topkp_tree_attention(None, None) == NULLPTR
    assert call(dtype=F32) == INVALID
    assert call(Hq=6) == INVALID and call(Hkv=0) == INVALID
    assert call(D=60) == INVALID and call(D=264) == INVALID and call(D=0) == INVALID
    assert call(T=65) == INVALID                                        # masks of more than 64 nodes
    assert call(pages=0) == INVALID and call(page_size=0) == INVALID and call(ld_table=3) == INVALID
    assert call(table=None) == INVALID                                  # no table, yet pages
    assert call(q=None) == NULLPTR and call(out=None) == NULLPTR and call(context=None) == NULLPTR
    assert call(k=_cache(data=None, dt=BF16, exp=None)) == NULLPTR
    assert call(k=_cache()) == INVALID                                  # e4m3 keys, bf16 values
    assert call(k=_cache(dt=F16, exp=None)) == INVALID
    assert call(k=_cache(dt=BF16, exp=None, tok=260)) == INVALID        # a stride that is no multiple of 8
    assert call(k=_cache(data=FAKE + 16 * MB + 2, dt=BF16, exp=None)) == INVALID
    assert call(q_head_stride=68) == INVALID and call(q=FAKE + 8) == INVALID
    assert call(out_head_stride=8) == INVALID
    assert call(tree=FAKE + 4 * MB + 4) == INVALID
    assert call(out=FAKE) == INVALID                                    # out over q
    assert call(lse=FAKE + MB) == INVALID                               # lse over out
    assert call(B=0) == 0 and call(T=0) == 0
    a = args(B=1, max_context=60000, max_pages=4096, ld_table=4096, pages=8192)
    need = lib.topkp_tree_attention_workspace_size(ctypes.byref(a))
    assert need > 0
    assert call(B=1, max_context=60000, max_pages=4096, ld_table=4096, pages=8192, workspace_bytes=need - 1) == INVALID
    assert call(B=1, max_context=60000, max_pages=4096, ld_table=4096, pages=8192, workspace=None) == INVALID


def test_tree_attention_refuses_wide_exponent_strides(lib):
    from top_logit_filter_gb300 import _lib

    def call(eps=64, ets=4, pages=8, page_size=16):
        k, v = _cache(eps=eps, ets=ets), _cache(data=FAKE + 48 * MB, exp=FAKE + 64 * MB)
        a = _lib.TreeAttentionArgs(q=FAKE, out=FAKE + MB, k=k, v=v, table=FAKE + 2 * MB, context=FAKE + 3 * MB, workspace=None,
                                   workspace_bytes=0, B=2, T=0, Hq=8, Hkv=4, D=64, pages=pages, page_size=page_size, max_pages=4,
                                   ld_table=4, max_context=64, q_batch_stride=2048, q_token_stride=512, q_head_stride=64,
                                   out_batch_stride=2048, out_token_stride=512, out_head_stride=64, dtype=BF16, scale=0.125)
        assert lib.topkp_tree_attention(ctypes.byref(a), None) == 0     # nothing to do
        a.T = 4
        st = lib.topkp_tree_attention(ctypes.byref(a), None)
        return st, lib.topkp_last_error_string().decode()
    for kw in (dict(eps=1 << 32), dict(ets=1 << 32)):
        st, why = call(**kw)
        assert st == INVALID and "32 bits" in why, (kw, why)
    st, why = call(eps=1 << 32, pages=1)                                # a stride that nothing is multiplied with
    assert "32 bits" not in why


def test_no_device_fails_loudly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    from top_logit_filter_gb300 import _lib
    assert lib.topkp_beam_select(FAKE, 2, 3, 8, 8, BF16, FAKE + MB, None, 0, 4, FAKE + 2 * MB, FAKE + 3 * MB, FAKE + 4 * MB,
                                 FAKE + 5 * MB, 1 << 16, None) == LAUNCH
    arr = (_lib.State * 1)(_state(lib))
    assert lib.topkp_beam_reorder(arr, 1, 2, 2, FAKE + 8 * MB, None, None) == LAUNCH


def test_python_faces_refuse():
    import top_logit_filter_gb300 as tk
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        tk.beam_select(cpu, torch.zeros(2, 2), 4)
    with pytest.raises(ValueError):
        tk.beam_reorder([cpu], torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        tk.cache_write(torch.zeros(2, 2, 8), torch.zeros(2, 2, 8), torch.zeros(2, dtype=torch.int64), cpu, cpu)
    with pytest.raises(ValueError):
        tk.cache_read(torch.zeros(2, dtype=torch.int64), cpu, cpu)
    with pytest.raises(ValueError):
        tk.tree_attention(torch.zeros(1, 1, 2, 8), cpu, cpu, torch.zeros(1, dtype=torch.int32))


def test_state_layouts():
    """Strides of rows and blocks as the reordering reads them off a tensor (no device needed)."""
    from top_logit_filter_gb300.decode import _layout
    t = torch.zeros(6, 10, 4, 8, dtype=torch.bfloat16)
    assert _layout(t, 1, "s") == (640, 640, 1, 10, 64)
    assert _layout(t, 2, "s") == (640, 64, 10, 4, 16)          # ten blocks of four entries
    assert _layout(t[:, :, :2], 2, "s") == (640, 64, 10, 2, 16)
    assert _layout(t[:, :7], 1, "s") == (640, 448, 1, 7, 64)
    assert _layout(torch.zeros(6, dtype=torch.int32), 1, "s") == (4, 4, 1, 1, 4)
    with pytest.raises(ValueError):
        _layout(t[..., :4], 1, "s")
    with pytest.raises(ValueError):
        _layout(t.transpose(1, 2), 1, "s")
