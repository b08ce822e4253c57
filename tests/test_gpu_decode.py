"""The decoding calls on the GPU against plain 64-bit references: beam
selection, reordering, the quantised cache and the attention over it."""
import math

import pytest

torch = pytest.importorskip("torch")
import decode_oracle as R  # noqa: E402

pytestmark = pytest.mark.gpu

T_ = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


@pytest.fixture(scope="module")
def tk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as m
    return m


# ------------------------------------------------------------ beam selection
def check_beam(tk, x, scores, n, finished=None, pad=0):
    """x, scores on the CPU; x may be a strided view of a wider tensor."""
    B, K = scores.shape
    V = x.shape[1]
    base = torch.full((x.shape[0], x.stride(0) if x.shape[0] > 1 else V), 7.0, dtype=x.dtype).cuda()
    xd = base[:, :V]
    xd.copy_(x)
    got = tk.beam_select(xd, scores.cuda(), n, finished=None if finished is None else finished.cuda(), pad_token=pad)
    score, parent, token = (t.cpu() for t in got)
    cand = R.beam_candidates(x, scores, finished, pad)
    # candidates of two beams nearer than 2 * 1e-6 may change places: compare by value there
    value, index = torch.sort(cand, dim=1, descending=True, stable=True)
    for b in range(B):
        for j in range(n):
            want = float(value[b, j]) if j < K * V else -INF
            if want == -INF:
                assert score[b, j] == -INF and token[b, j] == -1 and parent[b, j] == j % K, (b, j)
                continue
            tol = 1e-6 + abs(want) * 2.0 ** -24
            assert abs(float(score[b, j]) - want) <= tol, (b, j, float(score[b, j]), want)
            flat = int(parent[b, j]) * V + int(token[b, j])
            if flat != int(index[b, j]):
                other = int(parent[b, j]) != int(index[b, j]) // V
                assert other and abs(float(cand[b, flat]) - want) <= 2e-6, (b, j, flat, int(index[b, j]))
        live = [(int(p), int(t)) for p, t in zip(parent[b], token[b]) if int(t) >= 0]
        assert len(set(live)) == len(live)
        # a beam's own candidates come in the order of its logits, equal ones by index
        for k in range(K):
            if finished is not None and finished[b, k]:
                continue
            mine = [t for p, t in live if p == k]
            keys = [(-float(x[b * K + k, t]), t) for t in mine]
            assert keys == sorted(keys), (b, k)


def rows(R_, V, dtype, seed, ld=None, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R_, ld or V, generator=g) * spread).to(T_[dtype])
    return x[:, :V]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,K,V,n,ld", [(1, 1, 1, 1, None), (2, 3, 5, 8, None), (3, 4, 1000, 8, 1003), (2, 2, 4099, 5, 4101),
                                        (2, 5, 32000, 11, None), (1, 64, 700, 128, 701), (300, 2, 1024, 4, None),
                                        (1, 2, 151936, 64, None)])
def test_beam_select(tk, dtype, B, K, V, n, ld):
    g = torch.Generator().manual_seed(V + n)
    scores = -torch.rand(B, K, generator=g) * 3
    fin = (torch.rand(B, K, generator=g) < 0.2).to(torch.uint8)
    check_beam(tk, rows(B * K, V, dtype, V, ld), scores, n)
    check_beam(tk, rows(B * K, V, dtype, V + 1, ld), scores, n, fin, pad=min(2, V - 1))


def test_beam_select_unaligned_base(tk):
    for off in (1, 3, 5):
        wide = rows(4, 2000, "bf16", off).cuda()
        x = wide[:, off:off + 1501]
        s = torch.zeros(2, 2)
        a = tk.beam_select(x, s.cuda(), 6)
        b = tk.beam_select(x.contiguous(), s.cuda(), 6)
        # the alignment changes how a row's sum is grouped, not which elements are listed
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
        assert ((a[0] - b[0]).abs() <= 2e-6 + a[0].abs() * 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_select_ties_and_masks(tk, dtype):
    lowest = torch.finfo(T_[dtype]).min
    # equal logits everywhere: the lists overflow, and the order is by index
    check_beam(tk, torch.zeros(4, 40000, dtype=T_[dtype]), torch.tensor([[0.0, 0.0], [-1.0, 0.0]]), 70)
    # few distinct values, long runs of ties
    check_beam(tk, rows(4, 33000, dtype, 3).round(), torch.tensor([[0.0, -0.25], [-1.0, -0.5]]), 64)
    # what a filter leaves: -inf everywhere but some; a row without any; dead and first-step beams
    x = rows(6, 9000, dtype, 5).clone()
    x[x < 5.5] = -INF
    x[1] = -INF
    x[4, 1:] = -INF
    check_beam(tk, x, torch.tensor([[0.0, -1.0], [-INF, -2.0], [-0.5, -INF]]), 12)
    # the type's lowest value as a mask, in part of a row and in all of it
    x = rows(4, 9000, dtype, 6).clone()
    x[0, 10:] = lowest
    x[1] = lowest
    x[2, ::2] = -INF
    x[3] = -INF
    x[3, 77] = lowest
    check_beam(tk, x, torch.tensor([[0.0, -1.0], [-3.0, -2.0]]), 30)
    # rising and falling rows: every later chunk outbids the bound, or none does
    ramp = torch.arange(150000.0) / 1000.0
    check_beam(tk, torch.stack([ramp, ramp.flip(0)]).to(T_[dtype]).repeat(200, 1), torch.zeros(200, 2), 20)
    # one token far above a flat row: the sum of many small terms behind a large one
    x = torch.zeros(512, 140001, dtype=T_[dtype])
    x[:, 70001] = 11.0
    check_beam(tk, x, torch.zeros(256, 2), 2)
    # signed zeros are equal
    x = torch.zeros(2, 600, dtype=T_[dtype])
    x[:, ::2] = -0.0
    check_beam(tk, x, torch.zeros(1, 2), 9)


def test_beam_select_stream_and_graph(tk):
    x, s = rows(8, 5000, "bf16", 9).cuda(), torch.zeros(2, 4).cuda()
    want = tk.beam_select(x, s, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tk.beam_select(x, s, 8)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert tk.last_launch_count() == 2
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = tk.beam_select(x, s, 8)
    x.copy_(rows(8, 5000, "bf16", 10))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, tk.beam_select(x, s, 8)))


# ----------------------------------------------------------------- reordering
def ref_reorder(src, dst, parent, lengths, time_dim):
    B, K = parent.shape
    new = dst.clone()
    for b in range(B):
        for j in range(K):
            p = int(parent[b, j])
            if not 0 <= p < K:
                continue
            r, f = b * K + j, b * K + p
            if src.dim() == 1:
                new[r] = src[f] if lengths is None or lengths[b, p] > 0 else new[r]
                continue
            n = src.shape[time_dim] if lengths is None else min(max(int(lengths[b, p]), 0), src.shape[time_dim])
            new[r].narrow(time_dim - 1, 0, n).copy_(src[f].narrow(time_dim - 1, 0, n))
    return new


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 7, 8, 16, 31, 32, 64])
def test_reorder(tk, K, in_place):
    g = torch.Generator().manual_seed(K)
    B = 3
    shapes = [((B * K, 33, 2, 8), torch.bfloat16, 1), ((B * K, 2, 21, 3), torch.float32, 2), ((B * K, 19), torch.uint8, 1),
              ((B * K,), torch.int64, 1), ((B * K, 5, 7, 2), torch.float16, 1)]
    parent = torch.randint(0, K, (B, K), generator=g, dtype=torch.int32)
    parent[0, 0] = 0
    lengths = torch.randint(0, 40, (B, K), generator=g, dtype=torch.int32)
    for shape, dt, td in shapes:
        for ln in (None, lengths):
            src = torch.randint(0, 100, shape, generator=g).to(dt)
            dst = src if in_place else torch.randint(0, 100, shape, generator=g).to(dt)
            want = ref_reorder(src, dst, parent, ln, td)
            sd = src.cuda()
            dd = None if in_place else dst.cuda()
            got = tk.beam_reorder(sd, parent.cuda(), lengths=None if ln is None else ln.cuda(), time_dim=td, out=dd)
            assert got.data_ptr() == (sd if in_place else dd).data_ptr()
            assert torch.equal(got.cpu(), want), (shape, dt, ln is not None)
            if not in_place:
                assert torch.equal(sd.cpu(), src)


def test_reorder_many_states_and_strides(tk):
    g = torch.Generator().manual_seed(1)
    B, K = 2, 4
    parent = torch.tensor([[1, 1, 0, 3], [2, -1, 9, 0]], dtype=torch.int32)   # two entries outside: left alone
    states = [torch.randn(B * K, 6, 5, generator=g) for _ in range(70)]
    got = tk.beam_reorder([s.cuda() for s in states], parent.cuda())
    assert tk.last_launch_count() == 3
    for s, o in zip(states, got):
        assert torch.equal(o.cpu(), ref_reorder(s, s, parent, None, 1))
    # rows of a wider buffer; what lies between them stays
    wide = torch.randn(B * K, 9, 16, generator=g).cuda()
    before = wide.clone().cpu()
    tk.beam_reorder(wide[:, 2:5], parent.cuda())
    want = before.clone()
    want[:, 2:5] = ref_reorder(before[:, 2:5], before[:, 2:5], parent, None, 1)
    assert torch.equal(wide.cpu(), want)
    assert tk.beam_reorder([], parent.cuda()) == []
    tk.beam_reorder(torch.zeros(0, 4).cuda(), torch.zeros((0, 4), dtype=torch.int32).cuda())


def test_reorder_past_32_bits(tk):
    """Rows whose byte offsets pass 2^32."""
    K, T = 3, 1 << 23
    x = torch.zeros(K, T, 256, dtype=torch.uint8, device="cuda")
    x[:, ::4097] = (torch.arange(K, device="cuda") + 1).to(torch.uint8)[:, None, None]
    x[:, -1] = (torch.arange(K, device="cuda") + 11).to(torch.uint8)[:, None]
    tk.beam_reorder(x, torch.tensor([[2, 1, 0]], dtype=torch.int32, device="cuda"))
    assert x[0, 0, 0] == 3 and x[2, 4097, 5] == 1 and x[0, -1, -1] == 13 and x[2, -1, 0] == 11 and x[1, -1, 3] == 12


# ---------------------------------------------------------------------- cache
def awkward(N, H, D, dtype, seed):
    """Rows with zeros, outliers, borders of the scale, tiny values, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, H, D, generator=g)
    x *= torch.exp(2 * torch.randn(N, H, 1, generator=g))
    if N > 12:
        x[0] = 0
        x[1] = -0.0
        x[2, :, 0] = 448.0
        x[2, :, 1:] *= 1e-3
        x[3] = 448.0 * 0.5
        x[4, :, -1] = 449.0 if dtype == "f32" else 452.0
        x[5] *= 1e-7
        x[6, :, 0] = INF
        x[7, :, -1] = -INF
        x[8, :, 0] = math.nan
        x[9] = torch.finfo(T_[dtype]).max
        x[10] = torch.finfo(T_[dtype]).tiny
        x[11, :, 0] = INF
        x[11, :, 1:] = 0
    return x.to(T_[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,H,D,P", [(1, 1, 64, 16), (37, 3, 80, 8), (130, 2, 128, 48), (50, 1, 256, 64), (40, 5, 7, 3),
                                     (33, 2, 1, 1), (29, 2, 250, 16)])
def test_cache_round_trip(tk, dtype, N, H, D, P):
    g = torch.Generator().manual_seed(N)
    pages = -(-N // P) + 2
    slots = torch.randperm(pages * P, generator=g)[:N]
    if N > 20:
        slots[15], slots[16] = -1, pages * P          # both skipped
    k, v = awkward(N, H, D, dtype, N), awkward(N, H, D, dtype, N + 1)
    keep = (slots >= 0) & (slots < pages * P)
    # quantised
    kc, vc = (torch.zeros(pages, P, H, D, dtype=R.E4M3, device="cuda") for _ in (0, 1))
    ke, ve = (torch.full((pages, P, H), 9, dtype=torch.uint8, device="cuda") for _ in (0, 1))
    tk.cache_write(k.cuda(), v.cuda(), slots.cuda(), kc, vc, k_exp=ke, v_exp=ve)
    for x, c, e in ((k, kc, ke), (v, vc, ve)):
        q, byte = R.quantise(x)
        want = torch.zeros(pages * P, H, D, dtype=torch.float64)
        want[slots[keep]] = q[keep]
        wexp = torch.full((pages * P, H), 9)
        wexp[slots[keep]] = byte[keep].long()
        assert torch.equal(e.cpu().view(-1, H).long(), wexp)
        got = c.cpu().view(torch.uint8).view(R.E4M3).float().double().view(-1, H, D)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(nan=0), want.nan_to_num(nan=0))
    for out in ("f32", "f16", "bf16"):
        rk, rv = tk.cache_read(slots.cuda(), kc, vc, k_exp=ke, v_exp=ve, dtype=T_[out])
        for x, r in ((k, rk), (v, rv)):
            q, byte = R.quantise(x)
            # scaled exactly, rounded once
            want = torch.ldexp(q, byte[..., None] - 127)
            want[~keep] = 0
            want = want.to(torch.float32).to(T_[out]) if out != "f32" else want.to(torch.float32)
            assert torch.equal(r.cpu().nan_to_num(nan=0, posinf=1e30 if out != "f16" else 6e4, neginf=-1e30 if out != "f16" else -6e4),
                               want.nan_to_num(nan=0, posinf=1e30 if out != "f16" else 6e4, neginf=-1e30 if out != "f16" else -6e4)), out
            assert torch.equal(torch.isnan(r.cpu()), torch.isnan(want))
    # in the rows' own type: bits kept
    kc, vc = (torch.zeros(pages, P, H, D, dtype=T_[dtype], device="cuda") for _ in (0, 1))
    tk.cache_write(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
    rk, rv = tk.cache_read(slots.cuda(), kc, vc)
    for x, r in ((k, rk), (v, rv)):
        want = x.clone()
        want[~keep] = 0
        ints = torch.int32 if dtype == "f32" else torch.int16
        assert torch.equal(r.cpu().view(ints), want.view(ints))


def test_cache_strides_and_keys_alone(tk):
    g = torch.Generator().manual_seed(2)
    N, H, D, P, pages = 20, 3, 64, 4, 6
    qkv = torch.randn(N, 5 * H, D, generator=g).to(torch.bfloat16).cuda()
    k, v = qkv[:, :H], qkv[:, 2 * H:3 * H]              # rows inside a fused projection
    both = torch.zeros(pages, 2, H, P, D, dtype=torch.bfloat16, device="cuda")
    kc, vc = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)   # heads before tokens, keys and values interleaved
    slots = torch.randperm(pages * P, generator=g)[:N].cuda()
    tk.cache_write(k, v, slots, kc, vc)
    rk, rv = tk.cache_read(slots, kc, vc)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    kc2 = torch.zeros(pages, P, H, D, dtype=R.E4M3, device="cuda")
    ke2 = torch.zeros(pages, P, H, dtype=torch.uint8, device="cuda")
    tk.cache_write(k, None, slots, kc2, None, k_exp=ke2)
    r, none = tk.cache_read(slots, kc2, None, k_exp=ke2, dtype=torch.float32)
    assert none is None
    q, byte = R.quantise(k.cpu())
    assert torch.equal(r.cpu().double(), torch.ldexp(q, byte[..., None] - 127))
    # the strides of one head of many: an unaligned dense row
    odd = torch.randn(N, H, D + 1, generator=g).to(torch.bfloat16).cuda()[..., 1:]
    tk.cache_write(odd, odd, slots, kc, vc)
    rk, rv = tk.cache_read(slots, kc, vc)
    assert torch.equal(rk, odd) and torch.equal(rv, odd)


# ------------------------------------------------------------------ attention
def make_tree(B, T, seed, empty=False):
    g = torch.Generator().manual_seed(seed)
    bits = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            if i:
                bits[b, i] = bits[b, int(torch.randint(0, i, (1,), generator=g))]
            bits[b, i, i] = True
    if empty:
        bits[:, T // 2] = False
    words = torch.zeros(B, T, dtype=torch.int64)
    for j in range(T):
        words |= bits[:, :, j].long() << j if j < 63 else torch.where(bits[:, :, j], torch.tensor(-2 ** 63), torch.tensor(0))
    return bits, words


def attend(tk, dtype, cache, T, Hq, Hkv, D, P, contexts, tree=None, nodes=None, seed=0, capacity=None, scale=None,
           max_context=None, gap=False, extra=2, vfill=math.nan, spread=0.0, kv=(1.0, 1.5), qsize=1.2):
    """Builds a cache that holds NaN wherever no live token is, runs the call, checks every element."""
    g = torch.Generator().manual_seed(seed)
    B = len(contexts)
    cap = max(contexts) + T if capacity is None else capacity
    paged = P > 0
    per = -(-cap // P) if paged else 1
    pool, psz = (B * per + extra, P) if paged else (B, cap)
    table = torch.randperm(pool, generator=g)[:B * per].view(B, per).int() if paged else None
    quant = cache == "e4m3"
    kind = R.E4M3 if quant else T_[dtype]
    full = [torch.full((pool, psz, Hkv, D), vfill) for _ in (0, 1)]
    exps = [torch.full((pool, psz, Hkv), 255) for _ in (0, 1)]
    lens = []
    for b in range(B):
        n = T if nodes is None else int(nodes[b])
        ln = min(contexts[b] + n, per * psz)
        lens.append(ln)
        t = torch.arange(ln)
        page, at = (table[b].long()[t // P], t % P) if paged else (torch.full((ln,), b), t)
        for i in (0, 1):
            x = torch.randn(ln, Hkv, D, generator=g) * kv[i]
            x = x * torch.exp(spread * torch.randn(ln, Hkv, 1, generator=g))
            if quant:
                q, e = R.quantise(x)
                full[i][page, at] = q.float()
                exps[i][page, at] = e.long()
            else:
                full[i][page, at] = x
    store = [x.to(kind) for x in full]
    q = torch.randn(B, T, Hq, D, generator=g) * qsize
    q = (q * torch.exp(2 * spread * torch.randn(B, T, Hq, D, generator=g))).to(T_[dtype])
    bits, words = (None, None) if tree is None else tree
    scale = D ** -0.5 if scale is None else scale
    dev = [x.cuda() for x in store]
    if gap:  # a cache inside wider strides
        wide = [torch.full((pool, psz, Hkv + 1, D + 8), math.nan, dtype=torch.float32).to(kind).cuda() for _ in dev]
        for w, x in zip(wide, dev):
            w.view(torch.uint8)[:, :, :Hkv, :D * (1 if quant else 2)] = x.view(torch.uint8)
        dev = [w[:, :, :Hkv, :D] for w in wide]
    kw = dict(pages=None if table is None else table.cuda(), tree=None if words is None else words.cuda(),
              nodes=None if nodes is None else torch.tensor(nodes, dtype=torch.int32).cuda(), want_lse=True, scale=scale,
              max_context=max_context)
    if quant:
        kw.update(k_exp=exps[0].to(torch.uint8).cuda(), v_exp=exps[1].to(torch.uint8).cuda())
    qd = q.cuda()
    out, lse = tk.tree_attention(qd, *dev, torch.tensor(contexts, dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    tk.device_status()
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(B):
        n = T if nodes is None else int(nodes[b])
        ctx = min(contexts[b], per * psz)
        t = torch.arange(lens[b])
        page, at = (table[b].long()[t // P], t % P) if paged else (torch.full((lens[b],), b), t)
        k, v = (x.float()[page, at].double() for x in store)
        if quant:
            k, v = (torch.ldexp(x, e[page, at][..., None] - 127) for x, e in zip((k, v), exps))
        sees = (torch.tril(torch.ones(T, T, dtype=torch.bool)) if bits is None else bits[b])[:, :n]
        o, l, absv, big, off = R.attention(q[b].double(), k, v, ctx, n, sees, scale)
        vmax = float(v.abs().max()) if v.numel() else 0.0
        tol, ltol = R.attention_bounds(T_[dtype], o, l, absv, big, lens[b], D, vmax, off if quant else 0)
        bad = ~((out[b] - o).abs() <= tol)
        assert not bad.any(), (b, contexts[b], bad.nonzero()[0].tolist(), float((out[b] - o).abs().max()))
        assert torch.equal(torch.isinf(lse[b]), torch.isinf(l)), (b, contexts[b])
        fin = torch.isfinite(l)
        assert ((lse[b] - l).abs()[fin] <= ltol[fin]).all(), (b, float((lse[b] - l).abs()[fin].max()))


@pytest.mark.parametrize("dtype,cache", [("bf16", "own"), ("f16", "own"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("T,Hq,Hkv,D,P", [(1, 4, 4, 64, 16), (1, 8, 1, 128, 0), (1, 6, 2, 96, 48), (5, 7, 1, 64, 16),
                                          (16, 8, 2, 128, 64), (27, 9, 3, 80, 8), (64, 4, 1, 128, 128), (64, 16, 1, 128, 32),
                                          (3, 4, 2, 256, 16), (40, 4, 1, 256, 0), (2, 2, 1, 8, 1), (8, 32, 2, 64, 5)])
def test_attention(tk, dtype, cache, T, Hq, Hkv, D, P):
    contexts = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 130, 300]
    attend(tk, dtype, cache, T, Hq, Hkv, D, P, contexts, seed=T)
    attend(tk, dtype, cache, T, Hq, Hkv, D, P, contexts[::2], tree=make_tree(6, T, T), seed=T + 1)


@pytest.mark.parametrize("cache", ["own", "e4m3"])
@pytest.mark.parametrize("T,G,D,P", [(1, 4, 128, 16), (16, 4, 128, 64), (64, 8, 64, 0), (33, 5, 128, 24)])
def test_attention_long_and_split(tk, cache, T, G, D, P):
    attend(tk, "bf16", cache, T, G, 1, D, P, [5000, 2999, 1, 0], tree=make_tree(4, T, 3), seed=7)
    attend(tk, "bf16", cache, T, G, 1, D, P, [9001], seed=8)
    attend(tk, "bf16", cache, T, G, 1, D, P, [700, 2100], seed=9, max_context=64)   # the bound is wrong: results are not


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,D,P", [(31, 1, 128, 16), (8, 4, 128, 64), (32, 1, 64, 8), (16, 2, 256, 32), (11, 3, 96, 16),
                                     (33, 1, 128, 64), (1, 32, 72, 0), (1, 1, 256, 24), (4, 8, 128, 5)])
def test_attention_few_rows_quantised(tk, dtype, T, G, D, P):
    """Around 32 rows, where four warps begin to share a row's tokens: tiles' quarters that see nothing, one part and many."""
    contexts = [0, 1, 7, 15, 16, 17, 31, 48, 49, 63, 64, 65, 200]
    attend(tk, dtype, "e4m3", T, 2 * G, 2, D, P, contexts, seed=T + G)
    attend(tk, dtype, "e4m3", T, G, 1, D, P, [0, 3, 50, 64, 130], tree=make_tree(5, T, T), nodes=[T, 0, 1, T, T], seed=T)
    attend(tk, dtype, "e4m3", T, G, 1, D, P, [3000, 17], spread=1.0, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (20, 4, 64), (64, 4, 128), (8, 2, 256)])
def test_attention_quantised_sizes(tk, dtype, T, G, D):
    """Rows of very different scales, and all-large or all-small keys, values and queries."""
    attend(tk, dtype, "e4m3", T, G, 1, D, 16, [300, 70], spread=1.0, seed=1)
    attend(tk, dtype, "e4m3", T, G, 1, D, 16, [300, 70], kv=(30.0, 800.0), qsize=0.02, seed=2)
    attend(tk, dtype, "e4m3", T, G, 1, D, 16, [300, 70], kv=(2e-3, 0.01), qsize=200.0, seed=3)
    if dtype == "bf16":   # scales beyond 2^7, and far below fp16's range
        attend(tk, dtype, "e4m3", T, G, 1, D, 16, [300, 70], kv=(1e6, 1e7), qsize=1e-6, seed=4)
        attend(tk, dtype, "e4m3", T, G, 1, D, 16, [300, 70], kv=(1e-9, 1e-12), qsize=1e8, seed=5)


def test_attention_nan_goes_where_it_is_seen(tk):
    """A value or key that is NaN spoils the rows that see it (e4m3's NaN code too)."""
    g = torch.Generator().manual_seed(1)
    for cache in ("bf16", "e4m3"):
        B, T, Hq, D = 2, 3, 4, 128
        k, v = (torch.randn(B, 40, 1, D, generator=g) for _ in (0, 1))
        k[0, 5, 0, 7] = math.nan
        v[1, 6, 0, 9] = math.nan
        q = torch.randn(B, T, Hq, D, generator=g).to(torch.bfloat16).cuda()
        ctx = torch.tensor([30, 30], dtype=torch.int32).cuda()
        kw = {}
        if cache == "e4m3":
            kc, vc = (torch.zeros(B, 40, 1, D, dtype=torch.uint8, device="cuda").view(R.E4M3) for _ in (0, 1))
            ke, ve = (torch.zeros(B, 40, 1, dtype=torch.uint8, device="cuda") for _ in (0, 1))
            tk.cache_write(k.reshape(-1, 1, D).to(torch.bfloat16).cuda(), v.reshape(-1, 1, D).to(torch.bfloat16).cuda(),
                           torch.arange(B * 40, device="cuda"), kc, vc, k_exp=ke, v_exp=ve)
            kw = dict(k_exp=ke, v_exp=ve)
        else:
            kc, vc = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
        out = tk.tree_attention(q, kc, vc, ctx, **kw).cpu()
        assert torch.isnan(out[0]).all()
        assert torch.isnan(out[1, :, :, 9]).all() and torch.isfinite(out[1, :, :, :9]).all() and torch.isfinite(out[1, :, :, 10:]).all()


@pytest.mark.parametrize("T", [4, 33])
def test_attention_empty_rows_and_ragged_trees(tk, T):
    # a node that sees nothing, requests with fewer nodes, no context at all
    attend(tk, "bf16", "own", T, 4, 2, 64, 16, [0, 40, 0, 7], tree=make_tree(4, T, 5, empty=True), seed=1)
    attend(tk, "bf16", "own", T, 4, 2, 64, 16, [0, 40, 9, 7], tree=make_tree(4, T, 6), nodes=[T, 1, 0, 2], seed=2)
    attend(tk, "bf16", "e4m3", T, 4, 2, 128, 16, [0, 40, 9, 130], nodes=[0, 1, 2, 3], seed=3)


def test_attention_capacity_and_strides(tk):
    # contexts at and past the capacity; nodes beyond it are seen by none
    attend(tk, "bf16", "own", 4, 4, 2, 64, 16, [30, 64, 64, 10], capacity=64, seed=1)
    attend(tk, "bf16", "own", 20, 8, 2, 128, 0, [30, 64, 60, 10], capacity=64, seed=2)
    attend(tk, "bf16", "own", 5, 4, 2, 64, 16, [33, 70], gap=True, seed=3)
    attend(tk, "f16", "e4m3", 30, 8, 2, 128, 16, [33, 170], gap=True, seed=4)
    # extreme products: one token takes all
    attend(tk, "bf16", "own", 3, 4, 2, 64, 16, [33, 170], scale=8.0, seed=5)
    attend(tk, "bf16", "own", 33, 4, 1, 64, 16, [33, 170], scale=8.0, seed=6)
    attend(tk, "bf16", "own", 33, 4, 1, 64, 16, [33, 170], scale=0.0, seed=6)


def test_attention_views_and_workspace(tk):
    g = torch.Generator().manual_seed(4)
    B, T, Hq, Hkv, D, P = 2, 12, 8, 2, 128, 16
    qkv = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    q = qkv[:, :, :Hq]
    kc, vc = (torch.randn(16, P, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in (0, 1))
    table = torch.randperm(16, generator=g).view(B, 8).int().cuda()
    ctx = torch.tensor([100, 51], dtype=torch.int32).cuda()
    a = tk.tree_attention(q, kc, vc, ctx, pages=table)
    b = tk.tree_attention(q.contiguous(), kc, vc, ctx, pages=table)
    assert torch.equal(a, b)
    out = torch.full((B, T, Hq, 2 * D), 5.0, dtype=torch.bfloat16, device="cuda")
    tk.tree_attention(q, kc, vc, ctx, pages=table, out=out[..., :D])
    assert torch.equal(out[..., :D], a) and (out[..., D:] == 5).all()
    # heads before tokens
    kt, vt = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    assert torch.equal(tk.tree_attention(q, kt, vt, ctx, pages=table), a)
    # a page outside the pool reads as zeros
    bad = table.clone()
    bad[0, 3], bad[1, 0] = -1, 16
    zk, zv = torch.cat([kc, torch.zeros_like(kc[:1])]), torch.cat([vc, torch.zeros_like(vc[:1])])
    zt = table.clone()
    zt[0, 3], zt[1, 0] = 16, 16
    assert torch.equal(tk.tree_attention(q, kc, vc, ctx, pages=bad), tk.tree_attention(q, zk, zv, ctx, pages=zt))
    # another stream, twice the same bits, and a graph over changing contexts
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = tk.tree_attention(q, kc, vc, ctx, pages=table)
    side.synchronize()
    assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = tk.tree_attention(q, kc, vc, ctx, pages=table, max_context=116)
    ctx.copy_(torch.tensor([3, 116], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d, tk.tree_attention(q, kc, vc, ctx, pages=table, max_context=116))


@pytest.mark.parametrize("T", [1, 32])
def test_attention_past_32_bits(tk, T):
    """Pages whose element offsets pass 2^32: the same rows read near and far."""
    g = torch.Generator().manual_seed(6)
    Hkv, D, P, pages = 1, 128, 16, 4
    stride = (1 << 32) // 3 + 8 - ((1 << 32) // 3) % 8       # elements between pages; page 3 starts past 2^32
    buf = [torch.empty(3 * stride + P * D, dtype=torch.uint8, device="cuda").view(R.E4M3) for _ in (0, 1)]
    far = [b.as_strided((pages, P, Hkv, D), (stride, D, D, 1)) for b in buf]
    exps = [torch.empty(pages, P, Hkv, dtype=torch.uint8, device="cuda") for _ in (0, 1)]
    k, v = (torch.randn(pages * P, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in (0, 1))
    tk.cache_write(k, v, torch.arange(pages * P, device="cuda"), *far, k_exp=exps[0], v_exp=exps[1])
    near = [torch.empty(pages, P, Hkv, D, dtype=torch.uint8, device="cuda").view(R.E4M3) for _ in (0, 1)]
    nexp = [torch.empty_like(e) for e in exps]
    tk.cache_write(k, v, torch.arange(pages * P, device="cuda"), *near, k_exp=nexp[0], v_exp=nexp[1])
    q = torch.randn(1, T, 4, D, generator=g).to(torch.bfloat16).cuda()
    ctx = torch.tensor([pages * P - T], dtype=torch.int32).cuda()
    table = torch.tensor([[3, 1, 0, 2]], dtype=torch.int32).cuda()
    a = tk.tree_attention(q, *far, ctx, pages=table, k_exp=exps[0], v_exp=exps[1])
    b = tk.tree_attention(q, *near, ctx, pages=table, k_exp=nexp[0], v_exp=nexp[1])
    assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    rk, _ = tk.cache_read(torch.arange(pages * P, device="cuda"), *far, k_exp=exps[0], v_exp=exps[1])
    nk, _ = tk.cache_read(torch.arange(pages * P, device="cuda"), *near, k_exp=nexp[0], v_exp=nexp[1])
    assert torch.equal(rk, nk)
