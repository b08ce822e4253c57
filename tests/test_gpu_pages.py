"""cache_fork and cache_compact on the GPU against lists."""
import math

import pytest

torch = pytest.importorskip("torch")
import continuation_oracle as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as m
    return m


def bytes_of(g, *shape):
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)


def states_of(g, pool, P):
    """Pages of several layouts: entries of 32, 12 and 3 bytes, heads before tokens, keys and values in one tensor."""
    both = bytes_of(g, pool, 2, P, 2, 16)
    return [(bytes_of(g, pool, P, 2, 16), 1), (bytes_of(g, pool, P, 3), 1), (bytes_of(g, pool, P, 12), 1),
            (bytes_of(g, pool, 3, P, 16), 2), (bytes_of(g, pool, 5, P, 7), 2), (both[:, 0], 1), (both[:, 1], 1)]


def make(g, groups, beams, P, longest, pool, outside=0.2, partly=True):
    """A table whose groups share their prompts' whole pages, and references by others."""
    free = torch.randperm(pool, generator=g).tolist()
    M = -(-longest // P) + 3
    table, lengths = [], []
    for _ in range(groups):
        prompt = int(torch.randint(0, longest + 1, (1,), generator=g))
        shared = [free.pop() for _ in range(prompt // P)]
        for _ in range(beams):
            n = min(longest, prompt + int(torch.randint(0, 2 * P + 1, (1,), generator=g)))
            row = shared + [free.pop() for _ in range(-(-n // P) - len(shared) + int(torch.randint(0, 2, (1,), generator=g)))]
            table.append((row + [-1] * M)[:M])
            lengths.append(n)
    refs = [0] * pool
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    for p in range(pool):
        if float(torch.rand(1, generator=g)) < outside and (refs[p] == 0 or partly):
            refs[p] += 1
    return table, lengths, refs


def check_fork(tk, g, table, lengths, source, refs, grow, P, tensors, in_place=False, M=None):
    M = len(table[0]) if table else M
    pool = len(refs)
    i32 = lambda x, shape=None: (torch.tensor(x, dtype=torch.int32) if shape is None else torch.tensor(x, dtype=torch.int32).view(shape)).cuda()  # noqa: E731
    growths = grow if isinstance(grow, list) else [grow] * len(source)
    if table:
        new, counts, missing, copies = R.fork(table, lengths, source, refs, growths, P)
    else:
        new, counts, missing, copies = R.fork([[-1] * M], [0], [-1 for _ in source], refs, growths, P)
    want = [t.clone() for t, _ in tensors]
    for t, (_, dim) in zip(want, tensors):
        v = t.movedim(dim, 1)
        for a, b, live in copies:
            v[b, :live] = v[a, :live]
    dev = [t.cuda() for t, _ in tensors]
    r = i32(refs)
    for dim in sorted({d for _, d in tensors}):
        some = [t for t, (_, d) in zip(dev, tensors) if d == dim]
        args = (i32(table, (len(table), M)), i32(lengths), i32(source), r)
        kw = dict(grow=i32(grow) if isinstance(grow, list) else grow, time_dim=dim)
        if in_place and dim == max(d for _, d in tensors):
            kw["refs_out"] = r
        got_table, got_refs, got_missing = tk.cache_fork(some, *args, **kw)
        assert got_table.tolist() == new
        assert got_refs.tolist() == counts and int(got_missing) == missing
    for t, w in zip(dev, want):
        t = t.cpu()
        if not torch.equal(t, w):
            p = next(p for p in range(pool) if not torch.equal(t[p], w[p]))
            raise AssertionError((p, [c for c in copies if p in c[:2]]))
    return new, counts, missing


@pytest.mark.parametrize("groups,beams,P,longest,pool", [(1, 1, 16, 40, 30), (3, 4, 4, 50, 400), (7, 1, 5, 33, 300), (20, 8, 3, 20, 3000),
                                                         (2, 2, 64, 700, 200), (5, 3, 1, 9, 400), (300, 4, 2, 7, 9001)])
def test_fork(tk, groups, beams, P, longest, pool):
    g = torch.Generator().manual_seed(pool)
    for trial, partly in enumerate((False, True)):
        table, lengths, refs = make(g, groups, beams, P, longest, pool, partly=partly)
        n = groups * beams
        tensors = states_of(g, pool, P) if pool < 1000 else [(bytes_of(g, pool, P, 4), 1)]
        # beams follow their parents
        source = [b * beams + int(torch.randint(0, beams, (1,), generator=g)) for b in range(groups) for _ in range(beams)]
        check_fork(tk, g, table, lengths, source, refs, 1, P, tensors)
        # some end, some are forked, some begin; each grows differently
        source = torch.randint(-2, n + 2, (n + 5,), generator=g).tolist()
        grow = torch.randint(-1, 3 * P, (n + 5,), generator=g).tolist()
        check_fork(tk, g, table, lengths, source, refs, grow, P, tensors, in_place=True)


def test_fork_identity_everything_and_nothing(tk):
    g = torch.Generator().manual_seed(2)
    table, lengths, refs = make(g, 6, 3, 8, 60, 200, partly=False)
    tensors = states_of(g, 200, 8)
    same, counts, _ = check_fork(tk, g, table, lengths, list(range(18)), refs, 0, 8, tensors)
    for row, old, n in zip(same, table, lengths):      # pages past the live ones are given up
        assert row[:-(-n // 8)] == old[:-(-n // 8)] and set(row[-(-n // 8):]) == {-1}
    _, counts, _ = check_fork(tk, g, table, lengths, [], refs, 0, 8, tensors)
    assert counts == [r - sum(p == row[i] for row in table for i in range(len(row))) for p, r in enumerate(refs)]
    check_fork(tk, g, table, lengths, [4] * 40, refs, 9, 8, tensors)
    # no old row at all: requests begin
    check_fork(tk, g, [], [], [-1, 0, 5], [0] * 20 + [1] * 180, [0, 17, 40], 8, tensors, M=6)


@pytest.mark.parametrize("pool,holes", [(70001, 0.5), (40003, 0.999), (32768, 0.0), (8191, 1.0)])
def test_fork_large_pools(tk, pool, holes):
    """Free pages ranked over several rounds of the pool, few of them and many."""
    g = torch.Generator().manual_seed(pool)
    refs = (torch.rand(pool, generator=g) < holes).int()
    refs[torch.randint(0, pool, (600,), generator=g)] = 0        # some are free in any case
    where = torch.nonzero(refs == 0)[:, 0]
    where = where[torch.randperm(where.numel(), generator=g)][:90].tolist()
    table = [where[i * 6:i * 6 + 6] + [-1] * 3 for i in range(15)]
    for p in where:
        refs[p] += 1
    lengths = torch.randint(0, 13, (15,), generator=g).tolist()
    source = torch.randint(-1, 15, (40,), generator=g).tolist()
    check_fork(tk, g, table, lengths, source, refs.tolist(), torch.randint(0, 12, (40,), generator=g).tolist(), 2,
               [(bytes_of(g, pool, 2, 4), 1)])


def test_fork_the_most_rows(tk):
    """8192 rows on either side: shared memory at its largest."""
    g = torch.Generator().manual_seed(6)
    R, pool = 8192, 60000
    order = torch.randperm(pool, generator=g)
    table = torch.stack([order[:R], order[R:2 * R], torch.full((R,), -1)], 1)
    lengths = torch.randint(0, 9, (R,), generator=g)
    refs = torch.zeros(pool, dtype=torch.int64)
    refs[order[:2 * R]] = 1
    source = torch.randint(0, R, (R,), generator=g)
    check_fork(tk, g, table.tolist(), lengths.tolist(), source.tolist(), refs.tolist(), 3, 4, [(bytes_of(g, pool, 4, 3), 1)])


def test_fork_short_of_pages(tk):
    g = torch.Generator().manual_seed(3)
    for in_place in (False, True):
        table, lengths, refs = make(g, 4, 2, 4, 30, 90)
        refs = [max(r, 1) for r in refs]
        free = [p for p in range(90) if not any(p in row for row in table)][:5]
        for p in free:
            refs[p] = 0
        tensors = states_of(g, 90, 4)
        new, counts, missing = check_fork(tk, g, table, lengths, list(range(8)) + [0, 1, 2], refs, 9, 4, tensors, in_place=in_place)
        assert missing > 0 and counts == refs and all(set(row) == {-1} for row in new)


def test_fork_partial_pages_that_others_hold(tk):
    g = torch.Generator().manual_seed(4)
    P, pool = 8, 40
    tensors = states_of(g, pool, P)
    # two rows of different lengths over the same pages: one holds page 7 whole, the other in part
    table = [[5, 7, 9, -1, -1], [5, 7, -1, -1, -1], [5, 7, -1, -1, -1]]
    refs = [0] * pool
    refs[5], refs[7], refs[9] = 3, 3, 1
    check_fork(tk, g, table, [20, 12, 12], [0, 1, 2, 1], refs, 1, P, tensors)
    check_fork(tk, g, table, [20, 12, 12], [2, 1], refs, 1, P, tensors)      # the first of them keeps it once row 0 is gone
    refs[7] = 4                                                              # a prefix kept for later
    check_fork(tk, g, table, [20, 12, 12], [2, 1], refs, 1, P, tensors)
    # entries that hold nothing, in the whole pages and as the last one; lengths out of range; a table that is full
    table = [[5, -1, 9, 3, 11], [40, 99, 12, -7, -1], [13, 14, 15, 16, 17]]
    refs = [0] * pool
    for p in (5, 9, 3, 11, 12, 13, 14, 15, 16, 17):
        refs[p] = 1
    check_fork(tk, g, table, [30, 20, 999], [0, 0, 1, 1, 2, 2], refs, 30, P, tensors)
    check_fork(tk, g, table, [30, 28, -3], [1, 0, 2, 1], refs, [0, 2 ** 31 - 1, 5, 1], P, tensors)


def test_fork_many_states_stream_and_graph(tk):
    g = torch.Generator().manual_seed(5)
    table, lengths, refs = make(g, 3, 2, 4, 30, 120, partly=False)
    check_fork(tk, g, table, lengths, [0, 0, 1, 3, 3, 5], refs, 2, 4, [(bytes_of(g, 120, 4, 4), 1) for _ in range(131)])
    assert tk.last_launch_count() == 3
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    t, ln, src, rf = i32(table), i32(lengths), i32([0, 0, 1, 3, 3, 5]), i32(refs)
    x = bytes_of(g, 120, 4, 16).cuda()
    y = x.clone()
    want = tk.cache_fork(x, t, ln, src, rf, grow=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tk.cache_fork(y, t, ln, src, rf, grow=3)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tk.cache_fork(x, t, ln, src, rf, grow=3)
    src.copy_(i32([5, 4, 3, 2, 1, 0]))
    z = x.clone()
    graph.replay()
    torch.cuda.synchronize()
    want = tk.cache_fork(z, t, ln, src, rf, grow=3)
    assert all(torch.equal(a, b) for a, b in zip(want, out)) and torch.equal(x, z)
    # a strided table, and where the new one goes
    wide = torch.full((6, t.shape[1] + 3), 77, dtype=torch.int32, device="cuda")
    old = torch.full_like(wide, 5)
    old[:, :t.shape[1]] = t
    tk.cache_fork(z, old[:, :t.shape[1]], ln, src, rf, grow=3, out=wide[:, :t.shape[1]])
    assert torch.equal(wide[:, :t.shape[1]], out[0]) and (wide[:, t.shape[1]:] == 77).all()


def test_fork_of_far_pages(tk):
    """Pages whose byte offsets pass 2^32."""
    stride = (1 << 31) + 48
    buf = torch.empty(2 * stride + 4 * 32, dtype=torch.uint8, device="cuda")
    x = buf.as_strided((3, 4, 32), (stride, 32, 1))
    x.copy_(torch.arange(3 * 4 * 32, device="cuda").view(3, 4, 32) % 251)
    t = torch.tensor([[0, -1]], dtype=torch.int32).cuda()
    refs = torch.tensor([1, 1, 0], dtype=torch.int32).cuda()
    new, _, _ = tk.cache_fork(x, t, torch.tensor([3], dtype=torch.int32).cuda(), torch.tensor([0, 0], dtype=torch.int32).cuda(), refs)
    assert new.tolist() == [[0, -1], [2, -1]] and torch.equal(x[2, :3], x[0, :3]) and not torch.equal(x[2, 3], x[0, 3])
    tk.cache_compact(x, torch.tensor([2], dtype=torch.int32).cuda(), torch.tensor([[0, 5]], dtype=torch.int32).cuda(),
                     torch.tensor([2], dtype=torch.int32).cuda(), pages=torch.tensor([[1, 2]], dtype=torch.int32).cuda())
    assert torch.equal(x[1, 3], x[2, 3])


# ----------------------------------------------------------------- compaction
@pytest.mark.parametrize("B,W,P,M", [(1, 2, 4, 5), (3, 64, 16, 9), (9, 33, 5, 20), (70, 8, 64, 2), (2, 64, 1, 90)])
def test_compact(tk, B, W, P, M):
    g = torch.Generator().manual_seed(B + W)
    pool = B * M + 2
    for paged in (True, False):
        if paged:
            table = torch.randperm(pool, generator=g)[:B * M].view(B, M).int()
            if B > 2:
                table[1, M // 2], table[2, 0] = -1, pool
            tensors = states_of(g, pool, P)
        else:
            table, tensors = None, states_of(g, B, P * M)
        start = torch.randint(-2, P * M, (B,), generator=g).int()
        kept = torch.randint(-1, W + 3, (B,), generator=g).int()
        keep = torch.stack([torch.randperm(3 * W, generator=g)[:W].sort().values for _ in range(B)]).int()
        if B > 2:
            keep[0] = torch.arange(W)                 # nothing moves
            keep[2] = torch.randint(-5, 2 * W, (W,), generator=g).int()   # in no order, some twice
        dev = [t.cuda() for t, _ in tensors]
        for dim in (1, 2):
            some = [t for t, (_, d) in zip(dev, tensors) if d == dim]
            got = tk.cache_compact(some, start.cuda(), keep.cuda(), kept.cuda(), pages=None if table is None else table.cuda(), time_dim=dim)
            assert got is some and tk.last_launch_count() == 1
        for i, (t, dim) in enumerate(tensors):
            want, = R.compact([t], start.tolist(), keep.tolist(), kept.tolist(), None if table is None else table.tolist(), dim)
            assert torch.equal(dev[i].cpu(), want), (i, paged)


def test_compact_many_states_and_graph(tk):
    g = torch.Generator().manual_seed(7)
    many = [bytes_of(g, 4, 20, 8).cuda() for _ in range(140)]
    ref = [t.cpu() for t in many]
    start, kept = torch.tensor([3, 0, 5, 2], dtype=torch.int32).cuda(), torch.tensor([3, 2, 1, 4], dtype=torch.int32).cuda()
    keep = torch.tensor([[0, 4, 5, 9]] * 4, dtype=torch.int32).cuda()
    tk.cache_compact(many, start, keep, kept)
    assert tk.last_launch_count() == 2
    want = R.compact(ref, start.tolist(), keep.tolist(), kept.tolist(), None)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(many, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tk.cache_compact(many, start, keep, kept)
    kept.fill_(4)
    graph.replay()
    torch.cuda.synchronize()
    want = R.compact(want, start.tolist(), keep.tolist(), [4] * 4, None)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(many, want))


def test_refusals(tk):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(6, 4, 8, device="cuda")
    ok = dict(states=x, pages=i32(2, 3), lengths=i32(2), source=i32(2), refs=torch.ones(6, dtype=torch.int32, device="cuda"))
    tk.cache_fork(**ok)
    for bad, kind in ((dict(states=[]), ValueError), (dict(states=x[0, 0]), ValueError), (dict(states=x.cpu()), ValueError),
                      (dict(states=[x, torch.zeros(6, 5, 8, device="cuda")]), ValueError), (dict(refs=i32(5)), ValueError),
                      (dict(states=x.transpose(1, 2)), ValueError), (dict(lengths=i32(3)), ValueError), (dict(source=i32(2).long()), TypeError),
                      (dict(pages=i32(2, 3).float()), TypeError), (dict(pages=i32(2, 0)), tk.TopKPError), (dict(grow=-1), tk.TopKPError),
                      (dict(grow=i32(3)), ValueError), (dict(out=i32(2, 2)), ValueError), (dict(refs_out=i32(12)[::2]), ValueError),
                      (dict(states=[x, x]), tk.TopKPError), (dict(states=[x, x[:, :, 4:]]), (tk.TopKPError, ValueError)),
                      (dict(source=i32(8193)), tk.TopKPError), (dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), ValueError),
                      (dict(out=ok["pages"]), tk.TopKPError), (dict(lengths=ok["refs"][:2], refs_out=ok["refs"]), tk.TopKPError)):
        with pytest.raises(kind):
            tk.cache_fork(**{**ok, **bad})
    assert tk.cache_fork_workspace_size(4, 1000) >= 3 * 4000 and tk.cache_fork_workspace_size(8193, 10) == 0
    ok = dict(states=x, start=i32(6), keep=i32(6, 4), kept=i32(6))
    assert tk.cache_compact(**ok) is x
    for bad, kind in ((dict(keep=i32(6, 65)), tk.TopKPError), (dict(start=i32(5)), ValueError), (dict(keep=i32(5, 4), start=i32(5), kept=i32(5)), ValueError),
                      (dict(pages=i32(5, 2)), ValueError), (dict(states=[x, x]), tk.TopKPError), (dict(keep=i32(6, 4).long()), TypeError),
                      (dict(states=x.view(6, 4, 8)[..., ::2]), ValueError)):
        with pytest.raises(kind):
            tk.cache_compact(**{**ok, **bad})
    assert tk.cache_compact([], i32(6), i32(6, 4), i32(6)) == []
    assert math.isfinite(float(x.sum()))
