"""draft_verify on the GPU against a 64-bit walk down each request's tree."""
import math

import pytest

torch = pytest.importorskip("torch")
import continuation_oracle as R  # noqa: E402

pytestmark = pytest.mark.gpu

T_ = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf
# documented: a decision may differ where its sides lie within this of one another
NEAR = 1e-6


@pytest.fixture(scope="module")
def tk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    import top_logit_filter_gb300 as m
    return m


def make(B, T, V, dtype, mode, tree, seed, noise=0.5, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    target = torch.randn(B, T, V, generator=g) * spread
    lead = torch.randint(0, V, (B, T, 3), generator=g)
    target.scatter_add_(2, lead, 6 + torch.randn(B, T, 3, generator=g))
    draft = target + noise * torch.randn(B, T, V, generator=g)
    target, draft = target.to(T_[dtype]), draft.to(T_[dtype])
    parent = torch.zeros(B, T, dtype=torch.int32)
    for t in range(1, T):
        parent[:, t] = torch.randint(0, t, (B,), generator=g) if tree else t - 1
    race = torch.empty(B, T, V).exponential_(generator=g)
    tokens = torch.zeros(B, T, dtype=torch.int32)
    for t in range(T):
        row = draft[torch.arange(B), parent[:, t].long()].float()
        tokens[:, t] = (row - torch.log(race[:, t])).argmax(1).int()
    uniform = torch.rand(B, T, generator=g)
    race = torch.empty(B, V).exponential_(generator=g)
    return dict(target=target, draft=draft if mode == "ratio" else None, tokens=tokens, parent=parent if tree else None,
                uniform=uniform if mode != "greedy" else None, race=race if mode != "greedy" else None)


def check(tk, d, nodes=None, eps=1e-10, device=None, most_near=None):
    """Runs the call and compares every request whose decisions are not within NEAR; returns the accepted lengths."""
    device = device or {}
    args = {k: device.get(k, None if d[k] is None else d[k].cuda()) for k in d}
    nd = None if nodes is None else torch.tensor(nodes, dtype=torch.int32).cuda()
    target = args.pop("target")
    tokens = args.pop("tokens")
    got = tk.draft_verify(target, tokens, nodes=nd, eps=eps, want_logprob=True, **args)
    assert tk.last_launch_count() == 1
    count, path, token, logprob = (t.cpu() for t in got)
    B, T, V = d["target"].shape
    near = 0
    for b in range(B):
        n = T if nodes is None else min(max(nodes[b], 0), T)
        want, drawn, logs, margin = R.verify(d["target"][b], None if d["draft"] is None else d["draft"][b], d["tokens"][b].tolist(),
                                             None if d["parent"] is None else d["parent"][b].tolist(), n,
                                             None if d["uniform"] is None else d["uniform"][b], None if d["race"] is None else d["race"][b],
                                             eps, d["uniform"] is None)
        if margin <= NEAR:
            near += 1
            continue
        where = (b, want, drawn, margin, path[b].tolist(), int(token[b]))
        assert int(count[b]) == len(want), where
        assert path[b].tolist() == want + [-1] * (T - len(want)), where
        assert int(token[b]) == drawn, where
        # x - max is one fp32 rounding of at most 2^-24 |x - max|, the sum is within 1e-6; the result is rounded once
        for j in range(T):
            ref = logs[j] if j < len(logs) else 0.0
            assert abs(float(logprob[b, j]) - ref) <= 2e-6 + 2.0 ** -23 * abs(ref), (b, j, float(logprob[b, j]), ref)
    assert near <= (max(1, B // 50) if most_near is None else most_near), near
    return count


@pytest.mark.parametrize("mode", ["ratio", "certain", "greedy"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,V,tree", [(1, 1, 1, False), (2, 3, 5, True), (1, 5, 1000, False), (3, 4, 1003, False), (5, 64, 777, True),
                                        (8, 9, 32000, False), (9, 16, 4099, True), (320, 3, 1024, False), (1, 6, 151936, False),
                                        (40, 33, 2048, True), (160, 2, 8193, False)])
def test_verify(tk, dtype, mode, B, T, V, tree):
    check(tk, make(B, T, V, dtype, mode, tree, seed=B + T + V))


@pytest.mark.parametrize("mode", ["ratio", "certain"])
def test_flat_and_sharp_distributions(tk, mode):
    for spread, noise in ((0.1, 0.05), (0.5, 3.0), (12.0, 1.0), (40.0, 8.0)):
        check(tk, make(20, 12, 3001, "f32", mode, True, seed=3, spread=spread, noise=noise))
        check(tk, make(20, 12, 3008, "bf16", mode, True, seed=4, spread=spread, noise=noise))


@pytest.mark.parametrize("mode", ["ratio", "certain", "greedy"])
def test_ragged_requests(tk, mode):
    d = make(12, 7, 1500, "bf16", mode, True, seed=6)
    count = check(tk, d, nodes=[7, 0, 1, 2, -3, 9, 4, 5, 6, 7, 0, 1])
    assert count[1] == 0 and count[4] == 0 and count[10] == 0 and count[2] == 1
    d = make(6, 7, 1500, "f16", mode, False, seed=7)
    check(tk, d, nodes=[7, 0, 1, 2, 3, 4])


@pytest.mark.parametrize("mode", ["ratio", "certain", "greedy"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks_and_strange_tokens(tk, mode, dtype):
    lowest = torch.finfo(T_[dtype]).min
    d = make(14, 6, 900, dtype, mode, True, seed=8)
    x = d["target"]
    x[0] = torch.where(x[0] >= 4, x[0], -INF)     # what a filter left
    x[1, 0] = -INF                                # no token at all
    x[2, :, 1:] = -INF                            # one token
    x[3] = torch.where(x[3] >= 4, x[3], lowest)   # masks of the type's lowest value, in part and throughout
    x[4] = lowest
    x[5] = -INF
    x[5, :, 77] = lowest
    x[6] = 0.0                                    # equal logits
    d["tokens"][7] = torch.tensor([0, -1, 900, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32)
    d["tokens"][8] = 17                           # the same token again and again
    d["parent"][8] = 0
    d["parent"][9] = torch.tensor([0, 5, -1, 3, 2 ** 31 - 1, 2], dtype=torch.int32)   # parents that come later, or never
    if d["draft"] is not None:
        q = d["draft"]
        q[0] = torch.where(q[0] >= 4, q[0], -INF)
        q[10] = -INF                              # a draft that cannot have drawn anything
        q[11] = x[11]                             # the draft is the target
        q[12] = lowest
        d["uniform"][13] = 0.0
    elif mode == "certain":
        d["uniform"][13] = 0.0
        d["race"][12, ::2] = 0.0
    check(tk, d)
    if mode == "certain":                         # eps 0 and zeros: infinite candidates, the first of them
        d["race"][12, :300] = 0.0
        count, path, token = tk.draft_verify(x.cuda(), d["tokens"].cuda(), uniform=d["uniform"].cuda(), race=d["race"].cuda(),
                                             parent=d["parent"].cuda(), eps=0.0)
        assert int(token[12]) < 300


def test_what_is_left_is_nothing(tk):
    """Certain children that take every token the filter left: the draw is from the whole again."""
    x = torch.full((1, 4, 64), -INF)
    x[0, 0, 10], x[0, 0, 20] = 1.0, 1.5
    tokens = torch.tensor([[0, 10, 20, 10]], dtype=torch.int32)
    parent = torch.zeros(1, 4, dtype=torch.int32)
    one = torch.ones(1, 4) * 2.0                  # never below a probability
    for race in (torch.ones(1, 64), torch.ones(1, 64).index_fill(1, torch.tensor([20]), 100.0)):
        count, path, token = tk.draft_verify(x.cuda(), tokens.cuda(), uniform=one.cuda(), race=race.cuda(), parent=parent.cuda())
        assert int(count) == 1 and int(token) == (20 if race[0, 20] == 1 else 10)


def test_rows_off_the_path_are_not_read(tk):
    d = make(30, 12, 1111, "f32", "ratio", True, seed=9)
    count = check(tk, d)
    assert int(count.max()) > 2
    _, path, _ = tk.draft_verify(*(d[k].cuda() for k in ("target", "tokens", "uniform", "race", "draft", "parent")))
    path = path.cpu()
    e = {k: None if v is None else v.clone() for k, v in d.items()}
    dev = {}
    for name in ("target", "draft"):
        y = d[name].clone()
        for b in range(30):
            on = set(path[b].tolist())
            for t in range(12):
                if t not in on:
                    y[b, t] = math.nan
        dev[name] = y.cuda()
    check(tk, e, device=dev)


def test_layouts(tk):
    d = make(6, 5, 1001, "bf16", "ratio", False, seed=10)
    base = tk.draft_verify(*(d[k].cuda() for k in ("target", "tokens", "uniform", "race", "draft")), want_logprob=True)
    wide = torch.full((6, 7, 1100), 9.0, dtype=torch.bfloat16, device="cuda")
    for off in (0, 1, 4, 7, 8):
        dev = {}
        for i, k in enumerate(("target", "draft")):
            w = wide.clone()
            w[:, 1:6, off + 3 * i:off + 3 * i + 1001] = d[k].cuda()
            dev[k] = w[:, 1:6, off + 3 * i:off + 3 * i + 1001]
        r = torch.full((6, 1200), 1e-20, device="cuda")
        r[:, off:off + 1001] = d["race"].cuda()
        dev["race"] = r[:, off:off + 1001]
        check(tk, d, device=dev)
    # the vocabulary is not the innermost dimension, and a batch that is expanded
    got = tk.draft_verify(d["target"].cuda().transpose(1, 2).contiguous().transpose(1, 2), d["tokens"].cuda(), d["uniform"].cuda(),
                          d["race"].cuda().t().contiguous().t(), d["draft"].cuda(), want_logprob=True)
    assert all(torch.equal(a, b) for a, b in zip(base, got))
    e = {k: None if v is None else v[:1].expand(6, *v.shape[1:]) for k, v in d.items()}
    check(tk, e)


def test_far_rows_and_a_long_vocabulary(tk):
    """Rows whose element offsets pass 2^32, and the largest vocabulary."""
    d = make(3, 3, 5000, "bf16", "ratio", False, seed=21)
    far = torch.empty(2 ** 32 + 60000, dtype=torch.bfloat16, device="cuda")
    dev = {}
    for i, k in enumerate(("target", "draft")):
        x = far.as_strided((3, 3, 5000), (2 ** 31 + 8 * i, 5000, 1), 17000 * i)     # (the second lies in the gaps of the first)
        x.copy_(d[k].cuda())
        dev[k] = x
    check(tk, d, device=dev)
    del far, dev
    V = 1 << 23
    for dtype, mode in (("f32", "ratio"), ("bf16", "certain")):
        check(tk, make(1, 2, V, dtype, mode, False, seed=22), most_near=0)


def test_other_stream_graph_and_two_at_once(tk):
    d = {k: None if v is None else v.cuda() for k, v in make(10, 8, 20000, "bf16", "ratio", True, seed=11).items()}
    f = {k: None if v is None else v.cuda() for k, v in make(10, 8, 20000, "bf16", "ratio", True, seed=12).items()}

    def run(x):
        return tk.draft_verify(x["target"], x["tokens"], x["uniform"], x["race"], x["draft"], x["parent"], want_logprob=True)
    want, other = run(d), run(f)
    sides = [torch.cuda.Stream() for _ in (0, 1)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(sides[0]):
            a = run(d)
        with torch.cuda.stream(sides[1]):
            b = run(f)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, want)) and all(torch.equal(x, y) for x, y in zip(b, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(d)
    for k in d:
        d[k].copy_(f[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, other))


@pytest.mark.parametrize("mode", ["ratio", "certain"])
def test_tokens_are_distributed_as_the_targets(tk, mode):
    """The first two emitted tokens of 60000 requests with the same rows, drafts drawn anew each time."""
    g = torch.Generator(device="cuda").manual_seed(13)
    B, T, V = 60000, 6, 6
    # node 0 has children 1, 2, 3; node 1 has 4, node 2 has 5.  The second token's row depends on the node: make it the first token's
    rows = torch.randn(V + 1, V, generator=g, device="cuda") * 1.2
    drafts = rows + torch.randn(V + 1, V, generator=g, device="cuda")
    parent = torch.tensor([0, 0, 0, 0, 1, 2], dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    tokens = torch.zeros(B, T, dtype=torch.int64, device="cuda")

    def draw(which):  # a token of each request from the draft's rows
        if mode == "certain":
            return (drafts[which]).topk(3, 1).indices.gather(1, torch.randint(0, 3, (B, 1), generator=g, device="cuda"))[:, 0]
        return torch.multinomial(torch.softmax(drafts[which], 1), 1, generator=g)[:, 0]
    root = torch.full((B,), V, device="cuda")
    for t in (1, 2, 3):
        tokens[:, t] = draw(root)
    for t in (4, 5):
        tokens[:, t] = draw(tokens[:, t - 3])
    which = torch.cat([root[:, None], tokens[:, 1:]], 1)
    target, draft = rows[which], drafts[which]
    uniform = torch.rand(B, T, generator=g, device="cuda")
    race = torch.empty(B, V, device="cuda").exponential_(generator=g)
    count, path, token = tk.draft_verify(target, tokens.int(), uniform, race, draft if mode == "ratio" else None, parent)
    first = torch.where(count > 1, tokens.gather(1, path[:, 1:2].long().clamp(min=0))[:, 0], token.long())
    p = torch.softmax(rows[V].double(), 0)
    seen = torch.bincount(first, minlength=V).double() / B
    # six standard deviations of a share of 60000
    assert ((seen - p).abs() <= 6 * torch.sqrt(p * (1 - p) / B)).all(), (seen, p)
    for t in range(V):
        mine = (count > 1) & (first == t)
        n = int(mine.sum())
        if n < 500:
            continue
        second = torch.where(count[mine] > 2, tokens[mine].gather(1, path[mine][:, 2:3].long().clamp(min=0))[:, 0], token[mine].long())
        p = torch.softmax(rows[t].double(), 0)
        seen = torch.bincount(second, minlength=V).double() / n
        assert ((seen - p).abs() <= 6 * torch.sqrt(p * (1 - p) / n)).all(), (t, seen, p)


def test_refusals(tk):
    d = {k: None if v is None else v.cuda() for k, v in make(2, 3, 50, "f32", "ratio", True, seed=1).items()}
    ok = lambda **kw: tk.draft_verify(**{**d, **kw})  # noqa: E731
    ok()
    for bad, kind in ((dict(target=d["target"].cpu()), ValueError), (dict(target=d["target"].double()), TypeError),
                      (dict(tokens=d["tokens"].long()), TypeError), (dict(tokens=d["tokens"][:, :2]), ValueError),
                      (dict(race=None), ValueError), (dict(uniform=None), ValueError), (dict(uniform=None, race=None), ValueError),
                      (dict(race=d["race"][:, :9]), ValueError), (dict(draft=d["draft"][:, :2]), ValueError),
                      (dict(draft=d["draft"].half()), TypeError), (dict(parent=d["parent"].float()), TypeError),
                      (dict(eps=-1.0), tk.TopKPError), (dict(eps=math.nan), tk.TopKPError),
                      (dict(nodes=torch.zeros(3, dtype=torch.int32).cuda()), ValueError)):
        with pytest.raises(kind):
            ok(**bad)
    with pytest.raises(tk.TopKPError):
        tk.draft_verify(torch.zeros(1, 65, 8, device="cuda"), torch.zeros(1, 65, dtype=torch.int32, device="cuda"))
    empty = tk.draft_verify(torch.zeros(0, 3, 8, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda"))
    assert [tuple(t.shape) for t in empty] == [(0,), (0, 3), (0,)]
