"""Cases, plain forms and exact values of what several continuations of one
prompt need: the verification of drafted tokens, the forking of their block
tables and pages, the compaction of a drafted tree's accepted tokens, and the
attention of a batch whose requests share a prefix.

``run`` computes an operator in elementary torch operations, or, where
``own`` is true, through ``top_logit_filter_gb300``.  Sizes: the
vocabularies are those of the filter's workloads; heads, lengths and page
sizes are generic.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
VOCABS = (1024, 32000, 128256, 151936, 152064)
EPS = 1e-10


def listed():
    return [
        # one request, a drafted chain of four: latency
        dict(name="verify one request", op="verify", B=1, T=5, V=32000, dtype="f16", mode="ratio", tree=False),
        # a serving batch at the filter's headline vocabulary
        dict(name="verify chains of 64", op="verify", B=64, T=6, V=128256, dtype="bf16", mode="ratio", tree=False),
        # full-precision logits, the longest chains: the most bytes
        dict(name="verify wide fp32", op="verify", B=128, T=8, V=152064, dtype="f32", mode="ratio", tree=False),
        # drafted trees whose children were drawn one by one: residuals of residuals
        dict(name="verify trees", op="verify", B=32, T=64, V=151936, dtype="bf16", mode="ratio", tree=True),
        # one prompt goes on as eight samples; the pool is busy with others
        dict(name="fork one prompt", op="fork", B=1, K=1, N=8, L=4001, own=0, page=16, H=8, D=128, count=8, dtype="bf16"),
        # a step of beam search over pages: shared prompts, partial pages follow their beams
        dict(name="fork beams", op="fork", B=32, K=8, N=8, L=4096, own=512, page=64, H=8, D=128, count=8, dtype="e4m3"),
        # prompts of a batch go on as sixteen samples each: the most pages copied
        dict(name="fork prompts", op="fork", B=64, K=1, N=16, L=2000, own=0, page=64, H=8, D=128, count=8, dtype="bf16"),
        # a tree's accepted path, one request of many layers
        dict(name="compact one request", op="compact", B=1, T=32, L=1001, page=16, H=8, D=128, count=32, dtype="f16"),
        # the paths of a batch
        dict(name="compact batch", op="compact", B=64, T=64, L=2000, page=64, H=8, D=128, count=16, dtype="bf16"),
        # eight samples of one prompt
        dict(name="samples of one prompt", op="attention", groups=1, size=8, T=1, Hq=32, Hkv=8, D=128, prefix=4000, own=300,
             page=16, dtype="f16", cache="f16", chain=True),
        # beams of eight over long prompts in a quantised cache, eight queries to a head
        dict(name="beams over long prompts", op="attention", groups=16, size=8, T=1, Hq=64, Hkv=8, D=128, prefix=32000, own=500,
             page=64, dtype="bf16", cache="e4m3", chain=True),
        # a batch under one long document, drafted trees of 16: the most arithmetic
        dict(name="trees under one document", op="attention", groups=1, size=32, T=16, Hq=32, Hkv=8, D=128, prefix=65500, own=2000,
             page=64, dtype="bf16", cache="bf16", chain=False),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("verify", "verify", "verify", "fork", "compact", "attention", "attention", "attention"))
    if op == "verify":
        tree = rng.random() < 0.4
        T = rng.choice((2, 4, 8, 16, 31, 64)) if tree else rng.choice((1, 2, 3, 4, 6, 8, 9))
        V = rng.choice(VOCABS + (_between(rng, 1000, 152064),))
        dtype = rng.choice(("f32", "f16", "bf16"))
        B = _between(rng, 1, max(1, min(128, 32 * 64 * 151936 * 2 // (T * V * _SIZE[dtype]))))
        return dict(op=op, B=B, T=T, V=V, dtype=dtype, mode=rng.choice(("ratio", "ratio", "certain", "greedy")), tree=tree)
    H, D = rng.choice((1, 2, 8, 16)), rng.choice((64, 80, 128))
    page, dtype, count = rng.choice((8, 16, 48, 64, 128)), rng.choice(("f16", "bf16", "e4m3")), rng.choice((1, 2, 8, 16))
    if op == "fork":
        K, N = rng.choice(((1, 4), (1, 16), (1, 3), (4, 4), (8, 8), (4, 2)))
        L, more = _between(rng, 1, 8192), 0 if K == 1 else rng.choice((5, 60, 500))
        B = _between(rng, 1, max(1, min(64, (1 << 31) // (count * H * D * _SIZE[dtype] * (L + (K + N) * (more + 3 * page))))))
        return dict(op=op, B=B, K=K, N=N, L=L, own=more, page=page, H=H, D=D, count=count, dtype=dtype)
    if op == "compact":
        T, L = rng.choice((2, 5, 16, 27, 64)), _between(rng, 1, 4096)
        B = _between(rng, 1, max(1, min(64, (1 << 31) // (count * H * D * _SIZE[dtype] * (L + 2 * T + page)))))
        return dict(op=op, B=B, T=T, L=L, page=page, H=H, D=D, count=count, dtype=dtype)
    Hkv, G, D = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 7, 8)), rng.choice((64, 96, 128, 128, 256))
    T = rng.choice((1, 1, 1, 4, 9, 16, 32))
    groups, size = rng.choice((1, 1, 2, 5, 16)), rng.choice((1, 2, 4, 8, 13, 32, 64))
    prefix, more = _between(rng, 1, 60000), _between(rng, 1, 2000)
    rows = 32 * 16 * 32 * 65500
    while groups * size * T * Hkv * G * (prefix + more) * D > rows * 128 or groups * (prefix + size * (more + T)) * Hkv * D > 1 << 29:
        groups, size, prefix = max(1, groups // 2), max(1, size // 2), max(1, prefix // 2)
    dtype = rng.choice(("f16", "bf16"))
    return dict(op=op, groups=groups, size=size, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, prefix=prefix, own=more, page=page, dtype=dtype,
                cache="e4m3" if rng.random() < 0.4 else dtype, chain=T == 1 or rng.random() < 0.3)


# ------------------------------------------------------------------- inputs
def _exponent(x):
    """The smallest e with every |x| of a last dimension <= 448 * 2^e (448 = 0.875 * 2^9), no less than -126."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875).int()).clamp(min=-126)
    return torch.where(amax > 0, e, torch.full_like(e, -126))


def _quantised(x):
    """A cache's values and exponents as a write leaves them (x: a float32 tensor, changed)."""
    e = _exponent(x)
    return x.mul_(torch.exp2(-e.float())[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _tree(B, T, draw01):
    """Parents of B random trees of T nodes: each node hangs on an earlier one."""
    up = (draw01((B, T)) * torch.arange(T, device="cuda")).long()
    up[:, :1] = 0
    return up


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, c = "cuda", dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def uniform(shape):
        return torch.rand(shape, generator=g, device=dev)

    def whole(lo, hi, shape, dtype=torch.int32):
        return torch.randint(lo, hi + 1, shape, generator=g, device=dev, dtype=dtype)

    def race(*shape):
        return torch.empty(shape, device=dev).exponential_(generator=g)

    if c["op"] == "verify":
        B, T, V = c["B"], c["T"], c["V"]
        x = normal(B * T, V).mul_(2.0)
        # a few likely tokens a row, and one that leads, as a trained model gives them
        x.scatter_add_(1, whole(0, V - 1, (B * T, 12), torch.int64), 4 + 2 * normal(B * T, 12))
        x.scatter_add_(1, whole(0, V - 1, (B * T, 1), torch.int64), 10 + 2 * normal(B * T, 1))
        parent = _tree(B, T, uniform) if c["tree"] else None
        above = parent if parent is not None else (torch.arange(T, device=dev) - 1).clamp(min=0).expand(B, T)
        # the draft model agrees with the target's four times out of five
        draft = normal(B * T, V).mul_(0.5).add_(x).to(_T[c["dtype"]])
        target = x.to(_T[c["dtype"]]).view(B, T, V)
        del x
        tokens = torch.empty((B, T), dtype=torch.int64, device=dev)
        for t in range(T):  # a node's token is a draw from the draft's row of its parent
            row = draft.view(B, T, V)[torch.arange(B, device=dev), above[:, t]].float()
            tokens[:, t] = (row - torch.log(race(B, V))).argmax(1)
        state = dict(c=c, target=target, draft=draft.view(B, T, V) if c["mode"] == "ratio" else None, tokens=tokens.int(),
                     parent=None if parent is None else parent.int(), uniform=None, race=None)
        if c["mode"] != "greedy":
            state["uniform"], state["race"] = uniform((B, T)), race(B, V)
        return state
    if c["op"] == "fork":
        B, K, N, P = c["B"], c["K"], c["N"], c["page"]
        R = B * K
        prompt = whole(max(1, c["L"] // 2), c["L"], (B, 1))
        prompt[0] = c["L"]
        more = whole(c["own"] // 2, c["own"], (B, 1))
        lengths = (prompt + more).expand(B, K).reshape(-1)
        M, per = -(-(c["L"] + c["own"]) // P) + 2, -(-c["own"] // P) + 2  # pages of a row, and of it alone
        pool = B * M + R * per + B * N * 2 + 50
        order = torch.randperm(pool, generator=g, device=dev)
        # the prompt's whole pages are one for all beams of a request
        i = torch.arange(M, device=dev)[None]
        shared = (prompt // P if K > 1 else (lengths.view(B, K) + P - 1) // P).expand(B, K).reshape(-1, 1)
        held = (lengths[:, None] + P - 1) // P
        b = torch.arange(R, device=dev)[:, None] // K
        mine = B * M + torch.arange(R, device=dev)[:, None] * per + (i - shared).clamp(0, per - 1)
        at = torch.where(i < shared, b * M + i, mine)
        table = torch.where(i < held, order[at], -1).int()
        refs = torch.bincount(table[table >= 0].long(), minlength=pool).int()
        # other requests hold a part of the rest
        busy = (torch.arange(pool, device=dev) < B * M // 2) & (refs == 0)
        refs = torch.where(busy & (uniform((pool,)) < 0.3), 1, refs).int()
        source = (torch.arange(B, device=dev)[:, None] * K + whole(0, K - 1, (B, N))).int().view(-1)
        states = [normal(pool, P, c["H"], c["D"], dtype=torch.bfloat16).to(_T[c["dtype"]]) for _ in range(c["count"])]
        return dict(c=c, table=table, lengths=lengths.int().contiguous(), source=source, refs=refs, states=states)
    if c["op"] == "compact":
        B, T, P = c["B"], c["T"], c["page"]
        M = -(-(c["L"] + T) // P)
        pool = B * M + 3
        table = torch.randperm(pool, generator=g, device=dev)[: B * M].to(torch.int32).view(B, M)
        start = whole(c["L"] // 2, c["L"], (B,))
        # a path down a tree of T nodes numbered level by level: its nodes lie behind the place they go to
        count = whole(1, max(1, min(T // 2, 12)), (B,))
        score = uniform((B, T))
        score[:, 0] = -1.0
        j = torch.arange(T, device=dev)[None]
        far = torch.where((j > 0) & (j <= count[:, None]), 2.0, score)  # so that compacting twice is compacting once
        picked = torch.where(j < count[:, None], far.argsort(1), T).sort(1).values
        keep = torch.where(j < count[:, None], picked, 0).int()
        states = [normal(pool, P, c["H"], c["D"], dtype=torch.bfloat16).to(_T[c["dtype"]]) for _ in range(c["count"])]
        return dict(c=c, table=table, start=start, keep=keep.contiguous(), count=count, states=states)
    groups, S, T, Hq, Hkv, D, P = (c[n] for n in ("groups", "size", "T", "Hq", "Hkv", "D", "page"))
    B, quant = groups * S, c["cache"] == "e4m3"
    shared = whole(c["prefix"] // 2, c["prefix"], (groups,))
    shared[0] = c["prefix"]
    shared = shared // P * P  # what the requests share are whole pages
    context = shared.repeat_interleave(S) + whole(c["own"] // 2, c["own"], (B,))
    front, back = c["prefix"] // P, -(-(c["own"] + T) // P) + 1
    pool = groups * front + B * back
    order = torch.randperm(pool, generator=g, device=dev)
    i = torch.arange(front + back, device=dev)[None]
    first = (shared // P).repeat_interleave(S)[:, None]
    b = torch.arange(B, device=dev)[:, None]
    table = order[torch.where(i < first, b // S * front + i, groups * front + b * back + (i - first).clamp(0, back - 1))].to(torch.int32)
    both = []
    for _ in (0, 1):
        x = normal(pool, P, Hkv, D, dtype=torch.bfloat16 if pool * P * Hkv * D > 1 << 28 else torch.float32)
        both.append(_quantised(x.float()) if quant else (x.to(_T[c["cache"]]), None))
    tree = None
    if not c["chain"]:
        up = _tree(B, T, uniform)
        tree = torch.zeros((B, T), dtype=torch.int64, device=dev)
        for t in range(T):
            tree[:, t] = (1 << t) | (tree.gather(1, up[:, t : t + 1])[:, 0] if t else 0)
    return dict(c=c, q=(1.5 * normal(B, T, Hq, D)).to(_T[c["dtype"]]), caches=[x for x, _ in both], exps=[e for _, e in both],
                table=table, context=context.int(), shared=shared.int(), tree=tree, most=(c["prefix"] + c["own"], c["prefix"]))


# -------------------------------------------------------------- plain forms
def _softmax(x):
    """Probabilities in 64 bits, and the row's log-sum; zeros where nothing is finite."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0), m + torch.log(total)


def _plain_verify(s):
    # in 64 bits: a token is accepted or not by the sides of an inequality
    c = s["c"]
    B, T, V = c["B"], c["T"], c["V"]
    rows, ids = torch.arange(B, device="cuda"), torch.arange(V, device="cuda")
    cur = torch.zeros(B, dtype=torch.int64, device="cuda")
    depth = torch.zeros_like(cur)
    path = torch.full((B, T), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    logprob = torch.zeros((B, T), dtype=torch.float64, device="cuda")
    greedy, certain = c["mode"] == "greedy", c["mode"] != "ratio"
    tried = torch.zeros((B, V), dtype=torch.bool, device="cuda")
    less = torch.zeros((B, 1), dtype=torch.float64, device="cuda")
    weight = torch.ones_like(less)

    def left(less):
        """The node's distribution, what the tried children left of it, the draft's, and log-probabilities."""
        x = s["target"][rows, cur]
        p, lse = _softmax(x)
        if greedy:
            top = torch.where(x == x.amax(1, keepdim=True), ids, V).amin(1, keepdim=True)
            return None, (ids == top).double(), None, x.double() - lse
        if certain:
            return p, torch.where(tried, 0.0, p), None, x.double() - lse
        q = _softmax(s["draft"][rows, cur])[0]
        return p, (p - less * q).clamp(min=0), q, x.double() - lse

    for i in range(1, T):
        child = (s["parent"][:, i] == cur) if s["parent"] is not None else (cur == i - 1)
        x = s["tokens"][:, i : i + 1].long()
        p, r, q, logp = left(less)
        if greedy:
            accept = child & (r.gather(1, x)[:, 0] > 0)
        else:
            bound = s["uniform"][:, i : i + 1].double() * weight * (1.0 if certain else q.gather(1, x))
            accept = child & (bound < r.gather(1, x))[:, 0]
        reject = (child & ~accept)[:, None]
        if certain:
            tried |= reject & (ids == x)
            weight = torch.where(reject, torch.where(tried, 0.0, p).sum(1, keepdim=True) if not greedy else weight, weight)
        else:
            less = torch.where(reject, less + weight, less)
            weight = torch.where(reject, (p - less * q).clamp(min=0).sum(1, keepdim=True), weight)
        logprob[rows, depth] = torch.where(accept, logp.gather(1, x)[:, 0], logprob[rows, depth])
        depth += accept
        cur = torch.where(accept, i, cur)
        path[rows, depth] = cur
        tried &= ~accept[:, None]
        less, weight = torch.where(accept[:, None], 0.0, less), torch.where(accept[:, None], 1.0, weight)
    p, r, _, logp = left(less)
    if not greedy:
        r = torch.where(r.amax(1, keepdim=True) > 0, r, p) / (s["race"].double() + EPS)
    token = torch.where(r == r.amax(1, keepdim=True), ids, V).amin(1)
    logprob[rows, depth] = logp.gather(1, token[:, None])[:, 0]
    return (depth + 1).int(), path.int(), token.int(), logprob.float()


def _plain_fork(s):
    c, table, refs = s["c"], s["table"], s["refs"]
    P, M, pool = c["page"], table.shape[1], refs.shape[0]
    i, row = torch.arange(M, device="cuda")[None], torch.arange(s["source"].shape[0], device="cuda")
    hold = refs - torch.bincount(torch.where(table >= 0, table, pool).view(-1).long(), minlength=pool + 1)[:pool]
    length = s["lengths"][s["source"].long()].long()
    old = table[s["source"].long()].long()
    full = (length // P)[:, None]
    hold = hold + torch.bincount(torch.where(i < full, old, pool).view(-1), minlength=pool + 1)[:pool]
    # the last page, if it is partly filled: one of its holders keeps it if nobody else has it
    part = length % P > 0
    last = torch.where(part, old.gather(1, full.clamp(max=M - 1))[:, 0], pool)
    first = torch.full((pool + 1,), 1 << 30, dtype=torch.int64, device="cuda").scatter_reduce(0, last, row, "amin")
    keeps = part & (first[last] == row) & (torch.cat([hold, hold[:1]])[last] == 0)
    hold = hold + torch.bincount(torch.where(keeps, last, pool), minlength=pool + 1)[:pool]
    copies = part & ~keeps
    used = full[:, 0] + part
    need = ((length + 1 + P - 1) // P).clamp(max=M)
    demand = copies + (need - used).clamp(min=0)
    base = torch.cumsum(demand, 0) - demand
    free = torch.sort((hold != 0).int(), stable=True).indices  # the free pages first
    total, many = demand.sum(), (hold == 0).sum()
    fresh = free[(base[:, None] + (i - full - (keeps[:, None] & part[:, None]).int()).clamp(min=0)).clamp(max=pool - 1)]
    new = torch.where(i < full, old, torch.where(keeps[:, None] & (i == full), last[:, None], torch.where(i < need[:, None], fresh, -1)))
    given = torch.zeros(pool, dtype=torch.int64, device="cuda").scatter(0, free, (torch.arange(pool, device="cuda") < total).long())
    missing = (total - many).clamp(min=0)
    new = torch.where(missing > 0, -1, new).int()
    out = torch.where(missing > 0, refs, hold + given).int()
    which = copies & (missing == 0)
    src, dst = last[which], new.long().gather(1, full.clamp(max=M - 1))[:, 0][which]
    live = (torch.arange(P, device="cuda")[None] < (length % P)[which][:, None])[:, :, None, None]
    as_bytes = [x.view(torch.uint8) for x in s["states"]]
    [x.index_copy_(0, dst, torch.where(live, x[src], x[dst])) for x in as_bytes]
    return [new, out, missing.int().view(1), *s["states"]]


def _plain_compact(s):
    c = s["c"]
    P, T = c["page"], c["T"]
    j = torch.arange(T, device="cuda")[None]
    move = (j < s["count"][:, None]) & (s["keep"] > j)
    b = torch.arange(c["B"], device="cuda")[:, None].expand(-1, T)[move]
    frm, to = (s["start"][:, None] + s["keep"])[move].long(), (s["start"][:, None] + j)[move].long()
    src, dst = (s["table"][b, t // P].long() * P + t % P for t in (frm, to))
    flat = [x.view(torch.uint8).flatten(0, 1) for x in s["states"]]
    [x.index_copy_(0, dst, x[src]) for x in flat]
    return list(s["states"])


def _values(cache, exp):
    """A cache's values in 32 bits."""
    x = cache.float()
    return x if exp is None else x * torch.exp2(exp.float() - 127)[..., None]


def _plain_attention(s):
    c = s["c"]
    groups, S, T, Hq, Hkv, D, P = (c[n] for n in ("groups", "size", "T", "Hq", "Hkv", "D", "page"))
    B, G, L, own_len = groups * S, Hq // Hkv, c["prefix"] // P * P, c["own"] + T

    def rows(side, page, at):  # tokens of [rows, tokens] as [rows, Hkv, tokens, D] in 32 bits
        cache, exp = s["caches"][side], s["exps"][side]
        x = cache.view(torch.uint8 if exp is not None else cache.dtype)[page, at].view(cache.dtype)
        return _values(x, None if exp is None else exp[page, at]).transpose(1, 2)

    q = s["q"].float().view(groups, S * T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(groups, Hkv, S * T * G, D) * D ** -0.5
    t = torch.arange(max(L, 1), device="cuda")
    page = s["table"].view(groups, S, -1)[:, 0].long()[:, t // P]
    a = torch.matmul(q, rows(0, page, (t % P).expand_as(page)).transpose(2, 3))  # [groups, Hkv, S T G, L]
    a.masked_fill_((t[None] >= s["shared"][:, None])[:, None, None, :], float("-inf"))
    # each request's own tokens, the drafted ones among them
    mine = s["shared"].long().repeat_interleave(S)[:, None] + torch.arange(own_len, device="cuda")[None]
    own_page = s["table"].long().gather(1, mine // P)
    qr = q.view(groups, Hkv, S, T * G, D).transpose(1, 2).reshape(B, Hkv, T * G, D)
    o = torch.matmul(qr, rows(0, own_page, mine % P).transpose(2, 3)).view(B, Hkv, T, G, own_len)
    node = mine - s["context"][:, None].long()
    i = torch.arange(T, device="cuda")[None, :, None]
    drafted = node[:, None] <= i if s["tree"] is None else (s["tree"][:, :, None] >> node.clamp(0, 63)[:, None]) & 1 > 0
    sees = (node[:, None] < 0) | (drafted & (node < T)[:, None])
    o.masked_fill_(~sees[:, None, :, None, :], float("-inf"))
    o = o.view(B, Hkv, T * G, own_len)

    def by_group(x):  # [B, Hkv, T G, ...] as [groups, Hkv, S T G, ...]
        return x.reshape(groups, S, Hkv, T * G, -1).transpose(1, 2).reshape(groups, Hkv, S * T * G, -1)

    def by_request(x):
        return x.reshape(groups, Hkv, S, T * G, -1).transpose(1, 2).reshape(B, Hkv, T * G, -1)

    m = torch.maximum(by_request(a.amax(-1, keepdim=True)), o.amax(-1, keepdim=True))
    a.sub_(by_group(m)).exp_()
    o.sub_(m).exp_()
    total = by_request(a.sum(-1, keepdim=True)) + o.sum(-1, keepdim=True)
    out = by_request(torch.matmul(a, rows(1, page, (t % P).expand_as(page)))) + torch.matmul(o, rows(1, own_page, mine % P))
    out = (out / total).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = (m + torch.log(total)).view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return out.to(s["q"].dtype), lse


def _own(s):
    import top_logit_filter_gb300 as tk

    op = s["c"]["op"]
    if op == "verify":
        return tk.draft_verify(s["target"], s["tokens"], uniform=s["uniform"], race=s["race"], draft=s["draft"], parent=s["parent"],
                               eps=EPS, want_logprob=True)
    if op == "fork":
        table, refs, missing = tk.cache_fork(s["states"], s["table"], s["lengths"], s["source"], s["refs"], grow=1)
        return [table, refs, missing, *s["states"]]
    if op == "compact":
        return tk.cache_compact(s["states"], s["start"], s["keep"], s["count"], pages=s["table"])
    return tk.shared_attention(s["q"], *s["caches"], s["context"], s["table"], s["shared"], tree=s["tree"], k_exp=s["exps"][0],
                               v_exp=s["exps"][1], max_context=s["most"][0], max_shared=s["most"][1], want_lse=True)


def run(state):
    if own:
        return _own(state)
    return {"verify": _plain_verify, "fork": _plain_fork, "compact": _plain_compact, "attention": _plain_attention}[state["c"]["op"]](state)


def work(case):
    c, op = case, case["op"]
    if op == "verify":
        # the rows of the accepted path: four drafted tokens of five are accepted where the draft's probabilities
        # are known, half of them otherwise; a tree is about as deep as its logarithm
        on = 0.8 if c["mode"] == "ratio" else 0.5
        depth = min(c["T"], 1 + 2 * math.log(c["T"])) if c["tree"] else c["T"]
        rows = (1 - on ** depth) / (1 - on)
        drafted = rows * (depth - 1) / depth if c["mode"] == "ratio" else 0.0
        each = c["V"] * _SIZE[c["dtype"]]
        return {"bytes": int(c["B"] * (rows * each + drafted * each + (0 if c["mode"] == "greedy" else 4 * c["V"]) + 12 * c["T"])),
                "flops": int(4 * c["B"] * c["V"] * (rows + drafted))}
    if op == "fork":
        B, K, N, P = c["B"], c["K"], c["N"], c["page"]
        M, per = -(-(c["L"] + c["own"]) // P) + 2, -(-c["own"] // P) + 2
        pool = B * M + B * K * per + B * N * 2 + 50
        kept = K * (1 - (1 - 1 / K) ** N)  # rows that go on, each of which keeps its partial page
        entry = c["H"] * c["D"] * _SIZE[c["dtype"]] * c["count"]
        copied = B * (N - kept) * P / 2 * entry * (1 - 1 / P)
        read = B * min(kept, N - kept) * P / 2 * entry * (1 - 1 / P)
        return {"bytes": int(copied + read + 4 * (B * (K + N) * M + 2 * pool)), "flops": 0}
    if op == "compact":
        kept = max(1, min(c["T"] // 2, 12)) / 2
        return {"bytes": int(2 * c["B"] * kept * c["H"] * c["D"] * _SIZE[c["dtype"]] * c["count"] + 4 * c["B"] * c["T"]), "flops": 0}
    B = c["groups"] * c["size"]
    mean = c["prefix"] if c["groups"] == 1 else 0.75 * c["prefix"]
    mine = 0.75 * c["own"] + c["T"]
    one = 2 * c["Hkv"] * (c["D"] * _SIZE[c["cache"]] + (1 if c["cache"] == "e4m3" else 0))
    q = B * c["T"] * c["Hq"]
    return {"bytes": int((c["groups"] * mean + B * mine) * one + 2 * q * c["D"] * _SIZE[c["dtype"]] + 4 * q),
            "flops": int(4 * q * c["D"] * (mean + mine))}


# -------------------------------------------------------------- exact values
def _exact_verify(s):
    """One request at a time, down its tree, in logarithms."""
    c = s["c"]
    B, T = c["B"], c["T"]
    count, path = torch.zeros(B, dtype=torch.int32), torch.full((B, T), -1, dtype=torch.int32)
    token, logprob = torch.zeros(B, dtype=torch.int32), torch.zeros((B, T), dtype=torch.float64)
    parent = None if s["parent"] is None else s["parent"].tolist()
    tokens = s["tokens"].tolist()
    u = None if s["uniform"] is None else s["uniform"].double().tolist()
    for b in range(B):
        node, steps = 0, [0]
        while True:
            logp = torch.log_softmax(s["target"][b, node].double(), 0)
            kids = [i for i in range(node + 1, T) if (parent[b][i] if parent else i - 1) == node]
            chosen = None
            if c["mode"] == "greedy":
                x = s["target"][b, node]
                best = int(torch.nonzero(x == x.max())[0])
                chosen = next((i for i in kids if tokens[b][i] == best), None)
                drawn = best
            else:
                p = torch.exp(logp)
                q = torch.exp(torch.log_softmax(s["draft"][b, node].double(), 0)) if c["mode"] == "ratio" else None
                now = p
                for i in kids:
                    t = tokens[b][i]
                    if u[b][i] * (float(q[t]) if q is not None else 1.0) < float(now[t]):
                        chosen = i
                        break
                    if q is None:
                        now = now.clone()
                        now[t] = 0
                    else:
                        now = torch.relu(now - q)
                    now = now / now.sum()
                drawn = int(torch.argmax(torch.log(now) - torch.log(s["race"][b].double() + EPS))) if chosen is None else None
            if chosen is None:
                logprob[b, len(steps) - 1] = logp[drawn]
                token[b] = drawn
                break
            logprob[b, len(steps) - 1] = logp[tokens[b][chosen]]
            node = chosen
            steps.append(node)
        count[b] = len(steps)
        path[b, : len(steps)] = torch.tensor(steps)
    return tuple(t.cuda() for t in (count, path, token, logprob))


def _exact_fork(s):
    """Row by row, with lists; the states in 64 bits."""
    P, M = s["c"]["page"], s["table"].shape[1]
    table, lengths, source, refs = (s[n].tolist() for n in ("table", "lengths", "source", "refs"))
    left = list(refs)
    for row in table:
        for page in row:
            if page >= 0:
                left[page] -= 1
    rows, claims = [], {}
    for n, r in enumerate(source):
        full = table[r][: lengths[r] // P]
        for page in full:
            left[page] += 1
        rows.append(full)
        if lengths[r] % P:
            claims.setdefault(table[r][len(full)], []).append(n)
    copies = {}
    for page, who in claims.items():
        keeper = who[0] if left[page] == 0 else None
        for n in who:
            if n == keeper:
                rows[n] = rows[n] + [page]
            else:
                copies[n] = page
        left[page] += keeper is not None
    free = iter([page for page, many in enumerate(left) if many == 0] + [None] * (1 << 20))
    pairs = []
    for n, r in enumerate(source):
        if n in copies:
            page = next(free)
            pairs.append((copies[n], page, lengths[r] % P))
            rows[n] = rows[n] + [page]
        while len(rows[n]) < min(M, -(-(lengths[r] + 1) // P)):
            rows[n] = rows[n] + [next(free)]
    lacking = sum(page is None for row in rows for page in row)
    if lacking:
        return [torch.full((len(rows), M), -1, dtype=torch.int32, device="cuda"), s["refs"].clone(),
                torch.tensor([lacking], dtype=torch.int32, device="cuda"), *[x.double() for x in s["states"]]]
    counts = list(refs)
    for old in table:
        for page in old:
            if page >= 0:
                counts[page] -= 1
    for row in rows:
        for page in row:
            counts[page] += 1
    made = torch.tensor([row + [-1] * (M - len(row)) for row in rows], dtype=torch.int32, device="cuda")
    states = []
    for x in s["states"]:
        y = x.double()
        for src, dst, live in pairs:
            y[dst, :live] = x[src, :live].double()
        states.append(y)
    return [made, torch.tensor(counts, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), *states]


def exact(case, seed):
    c, op = case, case["op"]
    if op == "attention" and 4.0 * c["groups"] * c["size"] * c["T"] * c["Hq"] * c["D"] * (c["prefix"] + c["own"]) > 1e12:
        return None
    s = prepare(case, seed)
    if op == "verify":
        return _exact_verify(s)
    if op == "fork":
        return _exact_fork(s)
    if op == "compact":
        P, made = c["page"], []
        table, start, keep, count = (s[n].tolist() for n in ("table", "start", "keep", "count"))
        for x in s["states"]:
            y = x.double()
            for b in range(c["B"]):
                for j in range(count[b]):
                    frm, to = start[b] + keep[b][j], start[b] + j
                    if frm > to:
                        y[table[b][to // P], to % P] = x[table[b][frm // P], frm % P].double()
            made.append(y)
        return made
    S, T, Hq, Hkv, D, P = (c[n] for n in ("size", "T", "Hq", "Hkv", "D", "page"))
    B = c["groups"] * S
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, Hq), dtype=torch.float64, device="cuda")
    for b in range(B):
        ctx = int(s["context"][b])
        at = torch.arange(ctx + T, device="cuda")
        page, off = s["table"][b].long()[at // P], at % P
        k, v = (cache.view(torch.uint8)[page, off].view(cache.dtype).double() if cache.dtype == torch.float8_e4m3fn else cache[page, off].double()
                for cache in s["caches"])
        if s["exps"][0] is not None:
            k, v = (torch.ldexp(x, e[page, off].int()[..., None] - 127) for x, e in zip((k, v), s["exps"]))
        sees = torch.ones((T, ctx + T), dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            sees[:, ctx:] = torch.tril(sees[:, ctx:])
        else:
            sees[:, ctx:] = torch.tensor([[w >> j & 1 for j in range(T)] for w in s["tree"][b].tolist()], device="cuda") > 0
        for h in range(Hq):
            a = s["q"][b, :, h].double() @ k[:, h // (Hq // Hkv)].T / math.sqrt(D)
            a = torch.where(sees, a, float("-inf"))
            lse[b, :, h] = torch.logsumexp(a, 1)
            out[b, :, h] = torch.softmax(a, 1) @ v[:, h // (Hq // Hkv)]
    return out, lse
