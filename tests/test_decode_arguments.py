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


def _reorder(lib, states, B, K, parent=1 << 45):
    from top_logit_filter_gb300 import _lib
    arr = (_lib.State * max(len(states), 1))(*states)
    st = lib.topkp_beam_reorder(arr, len(states), B, K, parent, None, None)
    assert st in (LAUNCH, INVALID), lib.topkp_last_error_string()
    return st == LAUNCH


def _view(t, base=FAKE, time_dim=1, out=None):
    from top_logit_filter_gb300 import _lib
    from top_logit_filter_gb300.decode import _layout
    row, blk, blocks, entries, size = _layout(t, time_dim, "t")
    at = base + t.storage_offset() * t.element_size()
    if out is None:
        return _lib.State(at, at, row, row, blk, blk, blocks, entries, size)
    drow, dblk = _layout(out, time_dim, "out")[:2]
    return _lib.State(at, base + out.storage_offset() * out.element_size(), row, drow, blk, dblk, blocks, entries, size)


@needs_no_gpu
def test_reorder_takes_interleaved_views(lib):
    """Views of one tensor that share no byte are states of one call, in place and from one to the other."""
    c = torch.zeros(8, 2, 5, 3, 16, dtype=torch.bfloat16)                    # keys and values side by side
    assert _reorder(lib, [_view(c[:, 0]), _view(c[:, 1])], 2, 4)
    assert _reorder(lib, [_view(c[:, 0], out=c[:, 1])], 2, 4)
    assert not _reorder(lib, [_view(c[:, 0]), _view(c[:, 1]), _view(c[:, 0])], 2, 4)
    assert not _reorder(lib, [_view(c), _view(c[:, 1])], 2, 4)
    assert not _reorder(lib, [_view(c[:, 0, 1:4]), _view(c[:, 0, 3:])], 2, 4)
    layers = torch.zeros(8, 40, 2, 7, 24, dtype=torch.uint8)                 # rows outermost: every layer of a row together
    each = [_view(layers[:, i, j]) for i in range(40) for j in (0, 1)]
    assert _reorder(lib, each, 2, 4) and _reorder(lib, each[::-1], 4, 2)
    assert not _reorder(lib, each + [_view(layers[:, 39, 1, 3:4])], 2, 4)
    heads = torch.zeros(6, 3, 2, 9, 8, dtype=torch.float32)                  # [rows, heads, (keys, values), time, dim]
    assert _reorder(lib, [_view(heads[:, :, 0], time_dim=2), _view(heads[:, :, 1], time_dim=2)], 2, 3)
    assert not _reorder(lib, [_view(heads[:, :, 0], time_dim=2), _view(heads[:, 1:, 0], time_dim=2)], 2, 3)
    # one after another, and a view that wraps past the end of the other's rows
    flat = torch.zeros(4096, dtype=torch.uint8)
    assert _reorder(lib, [_view(flat[i * 256:][:256].view(4, 64)) for i in range(9)], 1, 4)
    a, b = flat.as_strided((4, 20), (100, 1), 90), flat.as_strided((4, 60), (100, 1), 110)
    assert _reorder(lib, [_view(a), _view(b)], 1, 4)
    assert not _reorder(lib, [_view(a), _view(flat.as_strided((4, 60), (100, 1), 109))], 1, 4)


@needs_no_gpu
def test_reorder_overlap_against_bytes(lib):
    """Random layouts in a small space against a map of their bytes: what shares one is refused, and with equal
    strides nothing else is."""
    import random
    rng = random.Random(5)
    from top_logit_filter_gb300 import _lib
    seen = [0, 0]
    for trial in range(4000):
        K, B = rng.randint(1, 4), rng.randint(1, 3)
        R = B * K
        row = rng.randint(8, 60)
        alike = rng.random() < 0.7
        block = rng.randint(1, row)
        states, spots = [], []
        for i in range(rng.choice((2, 2, 3, 5, 40))):
            if not alike:
                row, block = rng.randint(8, 60), rng.randint(1, 20)
            blocks = rng.randint(1, 3) if alike and block * 3 <= row else 1
            most = min(row - (blocks - 1) * block, block) if blocks > 1 else row
            size = rng.randint(1, max(1, min(most, 6)))
            at, to = rng.randint(0, 400), rng.randint(0, 400)
            if rng.random() < 0.6:
                to = at
            states.append(_lib.State(FAKE + at, FAKE + to, row, row, block, block, blocks, 1, size))

            def where(base):
                return {base + r * row + k * block + x for r in range(R) for k in range(blocks) for x in range(size)}
            spots.append((where(to), where(at) if to != at else set(), blocks, block))
        clash = any(spots[i][0] & spots[j][1] for i in range(len(spots)) for j in range(len(spots)))
        clash = clash or any(spots[i][0] & spots[j][0] for i in range(len(spots)) for j in range(i))
        got = _reorder(lib, states, B, K)
        if clash:
            assert not got, trial
        elif alike and len({s[2] > 1 for s in spots}) == 1:
            assert got, trial
        seen[got] += 1
    assert min(seen) > 300, seen


@needs_no_gpu
def test_reorder_of_many_states(lib):
    """The check does not go over all pairs: ten times the states cost about ten times as long."""
    import time

    def cost(n):
        states = [_view(torch.empty(8, 64, 128, dtype=torch.uint8), base=FAKE + i * MB) for i in range(n)]
        from top_logit_filter_gb300 import _lib
        arr, best = (_lib.State * n)(*states), 1e9
        for _ in range(5):
            t0 = time.perf_counter()
            for _ in range(20):
                lib.topkp_beam_reorder(arr, n, 2, 4, 1 << 45, None, None)
            best = min(best, time.perf_counter() - t0)
        return best
    small = cost(320)
    assert cost(3200) < 40 * small
