"""shared_attention on the GPU against 64-bit attention of each request."""
import math

import pytest

torch = pytest.importorskip("torch")
import decode_oracle as R  # noqa: E402
from test_gpu_decode import T_, make_tree  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as m
    return m


def build_case(dtype, cache, shared, size, own, T, Hkv, D, P, seed, nodes=None, spread=0.0):
    """Caches that hold NaN wherever no live token is; own: [B] tokens of each request behind the shared ones."""
    g = torch.Generator().manual_seed(seed)
    B = len(shared) * size
    contexts = [shared[b // size] + own[b] for b in range(B)]
    per = -(-(max(contexts) + T) // P)
    quant = cache == "e4m3"
    pool = B * per + 3
    order = torch.randperm(pool, generator=g)
    table = order[:B * per].view(B, per).clone().int()
    for b in range(B):           # whole shared pages are the group's first request's
        first = b // size * size
        table[b, :shared[b // size] // P] = table[first, :shared[b // size] // P]
    full = [torch.full((pool, P, Hkv, D), math.nan) for _ in (0, 1)]
    exps = [torch.full((pool, P, Hkv), 255) for _ in (0, 1)]
    for i in (0, 1):
        front = {}
        for b in range(B):
            n = T if nodes is None else nodes[b]
            ln = contexts[b] + n
            x = torch.randn(ln, Hkv, D, generator=g) * (1.0, 1.5)[i]
            x = x * torch.exp(spread * torch.randn(ln, Hkv, 1, generator=g))
            s = shared[b // size]
            x[:s] = front.setdefault(b // size, x[:s].clone())[:s]
            t = torch.arange(ln)
            page, at = table[b].long()[t // P], t % P
            if quant:
                q, e = R.quantise(x)
                full[i][page, at] = q.float()
                exps[i][page, at] = e.long()
            else:
                full[i][page, at] = x
    return g, B, contexts, table, [x.to(R.E4M3 if quant else T_[dtype]) for x in full], exps


def attend(tk, dtype, cache, shared, size, own, T, Hq, Hkv, D, P, tree=None, nodes=None, seed=0, say=None, scale=None, launches=None,
           max_context=None, max_shared=None, qview=False, spread=0.0, capacity=0):
    """capacity: of the table, beyond the live tokens; with it bounds may be given that make the call plan for much longer ones."""
    g, B, contexts, table, store, exps = build_case(dtype, cache, shared, size, own, T, Hkv, D, P, seed, nodes, spread)
    if capacity > table.shape[1] * P:
        table = torch.cat([table, torch.full((B, -(-capacity // P) - table.shape[1]), -1, dtype=torch.int32)], 1)
    quant = cache == "e4m3"
    q = (1.2 * torch.randn(B, T, Hq, D, generator=g)).to(T_[dtype])
    bits, words = (None, None) if tree is None else tree
    scale = D ** -0.5 if scale is None else scale
    kw = dict(tree=None if words is None else words.cuda(), nodes=None if nodes is None else torch.tensor(nodes, dtype=torch.int32).cuda(),
              want_lse=True, scale=scale, max_context=max_context, max_shared=max_shared)
    if quant:
        kw.update(k_exp=exps[0].to(torch.uint8).cuda(), v_exp=exps[1].to(torch.uint8).cuda())
    qd = q.cuda()
    if qview:      # nodes apart within a wider tensor, requests farther apart than their nodes
        qd = torch.full((B, T + 2, Hq + 1, D), math.nan, dtype=q.dtype, device="cuda")[:, 1:T + 1, :Hq]
        qd.copy_(q)
    out, lse = tk.shared_attention(qd, *(x.cuda() for x in store), torch.tensor(contexts, dtype=torch.int32).cuda(), table.cuda(),
                                   torch.tensor(shared if say is None else say, dtype=torch.int32).cuda(), **kw)
    if launches is not None:
        assert tk.last_launch_count() == launches
    torch.cuda.synchronize()
    tk.device_status()
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(B):
        n = T if nodes is None else nodes[b]
        ln = contexts[b] + n
        t = torch.arange(ln)
        page, at = table[b].long()[t // P], t % P
        k, v = (x.float()[page, at].double() for x in store)
        if quant:
            k, v = (torch.ldexp(x, e[page, at][..., None] - 127) for x, e in zip((k, v), exps))
        sees = (torch.tril(torch.ones(T, T, dtype=torch.bool)) if bits is None else bits[b])[:, :n]
        o, l, absv, big, off = R.attention(q[b].double(), k, v, contexts[b], n, sees, scale)
        vmax = float(v.abs().max()) if v.numel() else 0.0
        tol, ltol = R.attention_bounds(T_[dtype], o, l, absv, big, ln, D, vmax, off if quant else 0)
        bad = ~((out[b] - o).abs() <= tol)
        assert not bad.any(), (b, contexts[b], bad.nonzero()[0].tolist(), float((out[b] - o).abs().max()))
        assert torch.equal(torch.isinf(lse[b]), torch.isinf(l)), (b, contexts[b])
        fin = torch.isfinite(l)
        assert ((lse[b] - l).abs()[fin] <= ltol[fin]).all(), (b, float((lse[b] - l).abs()[fin].max()))


@pytest.mark.parametrize("dtype,cache", [("bf16", "own"), ("f16", "own"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("size,T,Hq,Hkv,D,P", [(40, 1, 4, 1, 128, 16), (64, 1, 16, 2, 64, 64), (33, 3, 2, 1, 96, 48), (100, 1, 1, 1, 256, 8),
                                               (24, 9, 8, 1, 128, 128), (60, 5, 8, 1, 128, 32)])
def test_one_prefix(tk, dtype, cache, size, T, Hq, Hkv, D, P):
    g = torch.Generator().manual_seed(size)
    own = torch.randint(0, 90, (size,), generator=g).tolist()
    attend(tk, dtype, cache, [1500], size, own, T, Hq, Hkv, D, P, seed=1, max_context=1600, max_shared=1500)
    # planned as if they were far longer: the grouped kernels, in several parts each
    for bound in (40000, 120000):
        attend(tk, dtype, cache, [1500], size, own, T, Hq, Hkv, D, P, seed=1, max_context=bound, max_shared=bound - 500, capacity=bound, launches=3)
    if T > 1:
        attend(tk, dtype, cache, [1111], size, own, T, Hq, Hkv, D, P, tree=make_tree(size, T, 2), seed=2, max_context=60000, max_shared=59000,
               qview=True, capacity=60000, launches=3)


@pytest.mark.parametrize("cache", ["own", "e4m3"])
def test_ragged_groups_and_requests(tk, cache):
    size = 30
    own = [0, 1, 63, 64, 65, 130] * 5
    nodes = [3, 0, 1, 2, 3, 3] * 5
    for D in (64, 128):
        # shared lengths around a tile's, and none; requests without nodes
        attend(tk, "bf16", cache, [0, 63, 64, 65, 1000, 129], size, own * 6, 3, 4, 2, D, 16, nodes=nodes * 6, seed=3, max_shared=39000,
               capacity=40000, launches=3)
    # a request that has no node and a short context of its own does not shorten the prefix of the others, nor read past it
    attend(tk, "bf16", cache, [900], size, own, 3, 4, 2, 128, 16, nodes=nodes, seed=4, launches=3, max_context=40000, max_shared=39000,
           capacity=40000)


@pytest.mark.parametrize("cache", ["own", "e4m3"])
def test_a_group_whose_first_requests_are_padding(tk, cache):
    """Requests without nodes hold no pages and no context: the prefix is read through the first that has any."""
    size, T, P = 20, 2, 16
    own = [9 * i % 70 for i in range(2 * size)]
    nodes = ([0, 0, 1] + [2] * (size - 3)) + [0] * size      # and a group of nothing but padding
    g, B, contexts, table, store, exps = build_case("bf16", cache, [640, 500], size, own, T, 1, 128, P, 3, nodes)
    table = torch.cat([table, torch.full((B, 4000), -1, dtype=torch.int32)], 1)
    for b in range(B):
        if nodes[b] == 0:
            table[b] = -1 if b % 2 else 2 ** 31 - 1
            contexts[b] = 0 if b % 2 else 10 ** 9
    q = torch.randn(B, T, 8, 128, generator=g).to(torch.bfloat16)
    kw = {} if cache == "own" else dict(k_exp=exps[0].to(torch.uint8).cuda(), v_exp=exps[1].to(torch.uint8).cuda())
    args = [q.cuda(), *(x.cuda() for x in store), torch.tensor(contexts, dtype=torch.int32).cuda(), table.cuda()]
    shared = torch.tensor([640, 500], dtype=torch.int32).cuda()
    kw.update(nodes=torch.tensor(nodes, dtype=torch.int32).cuda(), want_lse=True)
    out, lse = tk.shared_attention(*args, shared, **kw)
    assert tk.last_launch_count() == 3
    want, wlse = tk.tree_attention(*args[:4], pages=args[4], max_context=800, **kw)
    tk.device_status()
    on = torch.tensor([i < nodes[b] for b in range(B) for i in range(T)]).view(B, T)
    assert (out[~on] == 0).all() and (lse[~on] == -math.inf).all()
    # both are within the same bounds of 64 bits (tested above and beside tree_attention): values of about 1 over 600 tokens
    assert ((out.float() - want.float()).abs()[on] <= 2 * 2.0 ** -8 * (want.float().abs()[on] + 1.5)).all()
    assert ((lse - wlse).abs()[on] <= 1e-3).all()


def test_any_bound_of_what_is_shared(tk):
    own = [5 * i % 97 for i in range(48)]
    for say in ([700], [640], [639], [1], [0], [-5], [704 - 1]):
        attend(tk, "bf16", "own", [700], 48, own, 1, 4, 1, 128, 16, say=say, seed=5, max_context=60000, max_shared=59000,
               capacity=60000, launches=3)
    # too much is cut to the shortest context (equal contents up to there)
    attend(tk, "bf16", "own", [704], 48, [0] + own[1:], 1, 4, 1, 128, 64, say=[704], seed=6, max_context=60000, max_shared=59000,
           capacity=60000, launches=3)
    attend(tk, "bf16", "own", [704], 48, [0] * 48, 1, 4, 1, 128, 64, say=[10 ** 9], seed=6, max_context=60000, max_shared=59000,
           capacity=60000, launches=3)
    # wrong bounds plan badly and change nothing
    attend(tk, "bf16", "own", [2000], 48, own, 1, 4, 1, 128, 16, seed=7, max_context=128, max_shared=128)
    attend(tk, "bf16", "own", [300], 48, own, 1, 4, 1, 128, 16, seed=8)


def test_extremes(tk):
    own = [7 * i % 50 for i in range(40)]
    kw = dict(seed=9, max_context=60000, max_shared=59000, capacity=60000, launches=3)
    attend(tk, "bf16", "own", [1000], 40, own, 1, 8, 2, 128, 16, scale=8.0, **kw)
    attend(tk, "f16", "e4m3", [1000], 40, own, 2, 8, 2, 128, 16, spread=1.0, **kw)
    attend(tk, "bf16", "own", [1000], 40, own, 1, 8, 2, 128, 16, scale=0.0, **kw)
    attend(tk, "bf16", "own", [1000], 40, own, 1, 8, 2, 128, 16, scale=-0.05, **kw)


def test_few_requests_go_by_themselves(tk):
    attend(tk, "bf16", "own", [100, 90, 80], 1, [3, 4, 5], 2, 4, 2, 64, 16, seed=1, launches=1)
    attend(tk, "bf16", "own", [60, 50], 2, [3, 4, 5, 0], 2, 4, 2, 64, 16, seed=1, max_shared=60, launches=1)


def test_workspace_streams_and_graph(tk):
    g, B, contexts, table, store, _ = build_case("bf16", "own", [800, 1000], 20, [3 * i for i in range(40)], 1, 2, 128, 16, 11)
    q = torch.randn(B, 1, 8, 128, generator=g).to(torch.bfloat16).cuda()
    k, v = (x.cuda() for x in store)
    ctx, table = torch.tensor(contexts, dtype=torch.int32).cuda(), table.cuda()
    shared = torch.tensor([800, 1000], dtype=torch.int32).cuda()
    table = torch.cat([table, torch.full((B, 3000), -1, dtype=torch.int32, device="cuda")], 1)    # (room that nobody uses yet)
    kw = dict(max_context=40000, max_shared=39000, want_lse=True)
    need = tk.shared_attention_workspace_size(q, k, table, 2, max_context=40000, max_shared=39000)
    want = tk.shared_attention(q, k, v, ctx, table, shared, **kw)
    assert tk.last_launch_count() == 3 and need > 0
    got = tk.shared_attention(q, k, v, ctx, table, shared, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(ValueError, match="workspace"):
        tk.shared_attention(q, k, v, ctx, table, shared, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"), **kw)
    sides = [torch.cuda.Stream() for _ in (0, 1)]
    q2 = (2 * q.float()).to(q.dtype)
    other = tk.shared_attention(q2, k, v, ctx, table, shared, **kw)
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(sides[0]):
            a = tk.shared_attention(q, k, v, ctx, table, shared, **kw)
        with torch.cuda.stream(sides[1]):
            b = tk.shared_attention(q2, k, v, ctx, table, shared, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, a)) and all(torch.equal(x, y) for x, y in zip(other, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tk.shared_attention(q, k, v, ctx, table, shared, **kw)
    shared.copy_(torch.tensor([10, 700], dtype=torch.int32))
    q.copy_(q2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    again = tk.shared_attention(q2, k, v, ctx, table, shared, **kw)
    assert all(torch.equal(x, y) for x, y in zip(out, again))
    tk.device_status()


def test_refusals(tk):
    bf = torch.bfloat16
    q, k = torch.zeros(4, 1, 4, 64, dtype=bf, device="cuda"), torch.zeros(8, 16, 2, 64, dtype=bf, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ok = dict(q=q, k_cache=k, v_cache=k, context=i32(4), pages=i32(4, 2), shared=i32(2))
    tk.shared_attention(**ok)
    for bad, kind in ((dict(shared=i32(3)), ValueError), (dict(shared=i32(0)), ValueError), (dict(shared=i32(2).long()), TypeError),
                      (dict(pages=None), ValueError), (dict(pages=i32(3, 2)), ValueError), (dict(q=q.float()), TypeError),
                      (dict(q=q[..., :60]), (ValueError, tk.TopKPError)), (dict(k_cache=k[..., :32]), ValueError),
                      (dict(context=i32(3)), ValueError), (dict(shared=i32(2).cpu()), ValueError)):
        with pytest.raises(kind):
            tk.shared_attention(**{**ok, **bad})
