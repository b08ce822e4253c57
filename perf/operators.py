"""Cases, plain forms and exact values of the decoding operators: the beam
search selection, the reordering of its states, the cache that is quantised
as it is written, and the attention of drafted trees over that cache.

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


def listed():
    return [
        # one request, four beams: a step whose cost is latency
        dict(name="beam one request", op="beam", B=1, K=4, V=32000, n=8, dtype="f16", first=False, filtered=False),
        # a serving batch at the filter's headline vocabulary
        dict(name="beam batch of 64", op="beam", B=64, K=4, V=128256, n=8, dtype="bf16", first=False, filtered=False),
        # wide beams on fp32 logits, some beams finished: the largest selection
        dict(name="beam wide fp32", op="beam", B=32, K=32, V=151936, n=64, dtype="f32", first=False, filtered=False),
        # the states of a small batch follow its beams (a cache of [rows, time, heads, dim], a second buffer)
        dict(name="reorder small", op="reorder", B=2, K=4, T=640, H=8, D=128, count=8, dtype="bf16", in_place=False),
        # a large batch's caches, ragged, in place: only the rows that changed move
        dict(name="reorder large in place", op="reorder", B=32, K=8, T=1536, H=8, D=128, count=4, dtype="bf16", in_place=True),
        # one decode step of a batch writes its keys and values quantised
        dict(name="write decode step", op="write", N=64, H=8, D=128, page=64, dtype="bf16", cache="e4m3"),
        # a long prompt's keys and values
        dict(name="write prompts", op="write", N=65501, H=8, D=128, page=64, dtype="bf16", cache="e4m3"),
        # a shared prefix read back for another use
        dict(name="read prefix", op="read", N=32749, H=8, D=128, page=16, dtype="bf16", cache="e4m3"),
        # one request, a drafted tree of 16 over a short contiguous cache
        dict(name="tree one request", op="attention", B=1, T=16, Hq=32, Hkv=8, D=128, L=1001, page=0, dtype="f16", cache="f16", chain=False),
        # single tokens of a ragged batch over a paged cache
        dict(name="single tokens paged", op="attention", B=64, T=1, Hq=32, Hkv=8, D=128, L=8192, page=16, dtype="bf16", cache="bf16", chain=True),
        # trees of 64 with eight queries to a head over a quantised cache: the most arithmetic
        dict(name="trees of 64 quantised", op="attention", B=16, T=64, Hq=64, Hkv=8, D=128, L=16000, page=64, dtype="bf16", cache="e4m3", chain=False),
        # a drafted chain on two very long requests
        dict(name="long requests", op="attention", B=2, T=5, Hq=32, Hkv=8, D=128, L=131000, page=64, dtype="bf16", cache="bf16", chain=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("beam", "beam", "reorder", "write", "read", "attention", "attention", "attention"))
    if op == "beam":
        K = rng.choice((1, 2, 3, 4, 5, 8, 16, 32))
        V = rng.choice(VOCABS + (_between(rng, 1000, 152064),))
        B = _between(rng, 1, max(1, min(128, 32 * 32 * 151936 // (K * V) // 2)))
        return dict(op=op, B=B, K=K, V=V, n=rng.choice((K, 2 * K, 2 * K, 2 * K + 1)), dtype=rng.choice(("f32", "f16", "bf16")),
                    first=rng.random() < 0.2, filtered=rng.random() < 0.3)
    if op == "reorder":
        K, H, D = rng.choice((2, 3, 4, 8, 16)), rng.choice((1, 2, 8, 16)), rng.choice((64, 80, 128))
        T, count = _between(rng, 16, 4096), rng.choice((1, 2, 4, 16))
        B = _between(rng, 1, max(1, min(64, 32 * 8 * 1536 * 8 * 128 * 4 // (K * H * D * T * count) // 2)))
        return dict(op=op, B=B, K=K, T=T, H=H, D=D, count=count, dtype=rng.choice(("f16", "bf16", "e4m3")),
                    in_place=rng.random() < 0.5)
    if op in ("write", "read"):
        H, D = rng.choice((1, 2, 4, 8, 16)), rng.choice((64, 80, 128, 256))
        N = _between(rng, 1, min(65501, 65501 * 8 * 128 // (H * D)))
        dtype = rng.choice(("f32", "f16", "bf16")) if op == "write" else rng.choice(("f16", "bf16"))
        return dict(op=op, N=N, H=H, D=D, page=rng.choice((8, 16, 48, 64, 128)), dtype=dtype,
                    cache="e4m3" if rng.random() < 0.75 or dtype == "f32" else dtype)
    Hkv, G, D = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 7, 8, 16)), rng.choice((64, 64, 96, 128, 128, 128, 256))
    T = rng.choice((1, 1, 2, 5, 8, 16, 27, 32, 64))
    L = _between(rng, 1, 60000)
    most = 64 * 8 * 8192 * 128 // 2
    B = _between(rng, 1, max(1, min(64, most // (Hkv * L * D), 16 * 8 * 512 * 16000 * 128 // (Hkv * L * D * G * T) // 2)))
    dtype = rng.choice(("f16", "bf16"))
    return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, L=L, page=rng.choice((0, 16, 16, 48, 64, 128)), dtype=dtype,
                cache="e4m3" if rng.random() < 0.4 else dtype, chain=T == 1 or rng.random() < 0.3)


# ------------------------------------------------------------------- inputs
def _pool(c):
    """Pages of the pool, tokens of a page and pages of a request."""
    if not c["page"]:
        return c["B"], c["L"] + c["T"], 1
    each = -(-(c["L"] + c["T"]) // c["page"])
    return c["B"] * each, c["page"], each


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, c = "cuda", dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def whole(lo, hi, shape, dtype=torch.int32):
        return torch.randint(lo, hi + 1, shape, generator=g, device=dev, dtype=dtype)

    if c["op"] == "beam":
        R = c["B"] * c["K"]
        x = normal(R, c["V"]).mul_(2.0)
        # a few likely tokens a row, as a trained model gives them
        x.scatter_add_(1, torch.randint(0, c["V"], (R, 12), generator=g, device=dev), 4 + 2 * normal(R, 12))
        x = x.to(_T[c["dtype"]])
        if c["filtered"]:  # what the filter left: 50 tokens a row
            x = torch.where(x >= torch.topk(x.float(), 50, 1).values[:, -1:].to(x.dtype), x, float("-inf"))
        scores = -normal(c["B"], c["K"]).abs() * 2 - 8
        finished = torch.zeros((c["B"], c["K"]), dtype=torch.uint8, device=dev)
        if c["first"]:  # the first step: one live beam
            scores = torch.cat([torch.zeros_like(scores[:, :1]), torch.full_like(scores[:, 1:], float("-inf"))], 1)
        elif c["K"] > 1:
            finished[:, -1] = (torch.rand(c["B"], generator=g, device=dev) < 0.25).to(torch.uint8)
        return dict(c=c, logits=x, scores=scores.contiguous(), finished=finished)
    if c["op"] == "reorder":
        R = c["B"] * c["K"]
        kind = _T[c["dtype"]]
        many = [normal(R, c["T"], c["H"], c["D"], dtype=torch.bfloat16).to(kind) for _ in range(c["count"])]
        parent = whole(0, c["K"] - 1, (c["B"], c["K"]))
        if c["in_place"]:  # a beam that goes on keeps its row: applying the map twice is applying it once
            used = torch.zeros_like(parent).scatter_(1, parent.long(), 1).bool()
            parent = torch.where(used, torch.arange(c["K"], device=dev, dtype=torch.int32)[None], parent)
        # the beams of a request have one length
        lengths = whole(max(1, c["T"] // 2), c["T"], (c["B"], 1)).expand(c["B"], c["K"]).contiguous()
        out = None if c["in_place"] else [torch.zeros_like(s) for s in many]
        return dict(c=c, states=many, parent=parent, lengths=lengths, out=out)
    if c["op"] in ("write", "read"):
        N, H, D, P = c["N"], c["H"], c["D"], c["page"]
        pool = -(-N // P) + 3
        slots = torch.randperm(pool * P, generator=g, device=dev)[:N] if N < 1024 else None
        if slots is None:  # a prompt fills whole pages in a random order
            order = torch.randperm(pool, generator=g, device=dev)[: -(-N // P)]
            slots = (order[:, None] * P + torch.arange(P, device=dev)[None]).reshape(-1)[:N].contiguous()
        if N >= 50:  # padding of a batch
            slots[whole(0, N - 1, (N // 50,), torch.int64)] = -1
        kind, quant = _T[c["cache"]], c["cache"] == "e4m3"
        state = dict(c=c, slots=slots)
        channel = torch.exp(0.5 * normal(2, H, D))  # some channels are larger than others
        if c["op"] == "write":
            state["k"], state["v"] = ((normal(N, H, D) * channel[i]).to(_T[c["dtype"]]) for i in (0, 1))
            state["caches"] = [torch.zeros((pool, P, H, D), dtype=kind, device=dev) for _ in (0, 1)]
            state["exps"] = [torch.zeros((pool, P, H), dtype=torch.uint8, device=dev) for _ in (0, 1)] if quant else [None, None]
        else:
            made = [normal(pool, P, H, D) * channel[i] for i in (0, 1)]
            both = [_quantised(x) for x in made] if quant else [(x.to(kind), None) for x in made]
            state["caches"], state["exps"] = [x for x, _ in both], [e for _, e in both]
        return state
    B, T, Hq, Hkv, D, L = (c[n] for n in ("B", "T", "Hq", "Hkv", "D", "L"))
    pool, P, each = _pool(c)
    quant = c["cache"] == "e4m3"
    both = []
    for _ in (0, 1):
        x = normal(pool, P, Hkv, D, dtype=torch.bfloat16 if pool * P * Hkv * D > 1 << 28 else torch.float32)
        both.append(_quantised(x.float()) if quant else (x.to(_T[c["cache"]]), None))
    table = torch.randperm(pool, generator=g, device=dev).to(torch.int32).reshape(B, each) if c["page"] else None
    context = whole(L // 2, L, (B,))
    context[0] = L
    tree = None
    if not c["chain"]:
        tree = torch.zeros((B, T), dtype=torch.int64, device=dev)
        up = (torch.rand((B, T), generator=g, device=dev) * torch.arange(T, device=dev)).long()
        for i in range(T):
            tree[:, i] = (1 << i) | (tree.gather(1, up[:, i : i + 1])[:, 0] if i else 0)
    return dict(c=c, q=(1.5 * normal(B, T, Hq, D)).to(_T[c["dtype"]]), caches=[x for x, _ in both], exps=[e for _, e in both],
                table=table, context=context, tree=tree, longest=L)


# -------------------------------------------------------------- plain forms
def _plain_beam(s):
    c = s["c"]
    B, K, V, n = c["B"], c["K"], c["V"], c["n"]
    # in 64 bits: candidates of two beams may differ in their last bits only
    x = s["logits"].double().view(B, K, V)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    score = s["scores"].double()[..., None]
    cand = torch.where(torch.isinf(x), x, score + (x - lse))
    over = torch.where(torch.arange(V, device=x.device) == PAD, score, float("-inf"))
    cand = torch.where(s["finished"].bool()[..., None], over, cand).view(B, K * V)
    value, index = torch.sort(cand, dim=1, descending=True, stable=True)
    value, index = value[:, :n], index[:, :n]
    none = torch.isinf(value)
    slot = torch.arange(n, device=x.device) % K
    parent = torch.where(none, slot, index // V).int()
    token = torch.where(none, -1, index % V).int()
    return value.float(), parent, token


PAD = 2


def _plain_reorder(s):
    c = s["c"]
    base = torch.arange(c["B"], device="cuda")[:, None] * c["K"]
    rows = (base + s["parent"]).view(-1)
    live = (torch.arange(c["T"], device="cuda")[None] < s["lengths"].view(-1)[rows][:, None])[:, :, None, None]
    to = s["states"] if s["out"] is None else s["out"]
    as_bytes = [(x.view(torch.uint8), t.view(torch.uint8)) for x, t in zip(s["states"], to)]
    [t.copy_(torch.where(live, x[rows], t)) for x, t in as_bytes]
    return list(to)


def _plain_write(s):
    c = s["c"]
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    for_one = [_write_one(x[keep], at, cache, exp) for x, cache, exp in zip((s["k"], s["v"]), s["caches"], s["exps"])]
    return [t for pair in for_one for t in pair]


def _write_one(x, at, cache, exp):
    flat = cache.view(-1, *cache.shape[2:])
    if exp is None:
        flat[at] = x
        return (cache,)
    x = x.float()
    e = _exponent(x)
    q = (x * torch.exp2(-e.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    flat.view(torch.uint8)[at] = q.view(torch.uint8)
    exp.view(-1, exp.shape[2])[at] = (e + 127).to(torch.uint8)
    return cache, exp


def _values(cache, exp):
    """A cache's values in 32 bits."""
    x = cache.float()
    return x if exp is None else x * torch.exp2(exp.float() - 127)[..., None]


def _plain_read(s):
    c = s["c"]
    at, skip = s["slots"].clamp(min=0), (s["slots"] < 0)[:, None, None]

    def one(cache, exp):
        x = cache.view(torch.uint8 if exp is not None else cache.dtype).flatten(0, 1)[at]
        x = x.view(cache.dtype)
        x = _values(x, None if exp is None else exp.flatten(0, 1)[at])
        return torch.where(skip, 0.0, x).to(_T[c["dtype"]])

    return one(s["caches"][0], s["exps"][0]), one(s["caches"][1], s["exps"][1])


def _seen(s, length):
    """[B, T, length]: whether node i sees the cache's token t."""
    c = s["c"]
    B, T = c["B"], c["T"]
    t = torch.arange(length, device="cuda")
    node = t[None, :] - s["context"][:, None].long()  # which node a token is
    i = torch.arange(T, device="cuda")[None, :, None]
    if s["tree"] is None:
        drafted = node[:, None, :] <= i
    else:
        drafted = (s["tree"][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1 > 0
    return (node[:, None, :] < 0) | (drafted & (node < T)[:, None, :])


def _plain_attention(s):
    c = s["c"]
    B, T, Hq, Hkv, D = (c[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    G, length = Hq // Hkv, s["longest"] + T

    def rows(cache, exp):  # [B, Hkv, length, D] in 32 bits
        if s["table"] is not None:
            cache = cache.view(torch.uint8 if exp is not None else cache.dtype)[s["table"].long()].flatten(1, 2).view(cache.dtype)
            exp = None if exp is None else exp[s["table"].long()].flatten(1, 2)
        return _values(cache[:, :length], None if exp is None else exp[:, :length]).transpose(1, 2)

    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    a = torch.matmul(q, rows(s["caches"][0], s["exps"][0]).transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, T, G, length)
    a.masked_fill_(~_seen(s, length)[:, None, :, None, :], float("-inf"))
    m = a.amax(-1, keepdim=True)
    a.sub_(m).exp_()
    total = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(B, Hkv, T * G, length), rows(s["caches"][1], s["exps"][1])).view(B, Hkv, T, G, D) / total
    lse = (m + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(B, T, Hq)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(s["q"].dtype), lse


def _own(s):
    import top_logit_filter_gb300 as tk

    op = s["c"]["op"]
    if op == "beam":
        return tk.beam_select(s["logits"], s["scores"], s["c"]["n"], finished=s["finished"], pad_token=PAD)
    if op == "reorder":
        return tk.beam_reorder(s["states"], s["parent"], lengths=s["lengths"], out=s["out"])
    if op == "write":
        tk.cache_write(s["k"], s["v"], s["slots"], *s["caches"], k_exp=s["exps"][0], v_exp=s["exps"][1])
        return [t for pair in zip(s["caches"], s["exps"]) for t in pair if t is not None]
    if op == "read":
        return tk.cache_read(s["slots"], *s["caches"], k_exp=s["exps"][0], v_exp=s["exps"][1], dtype=_T[s["c"]["dtype"]])
    return tk.tree_attention(s["q"], *s["caches"], s["context"], pages=s["table"], tree=s["tree"], k_exp=s["exps"][0],
                             v_exp=s["exps"][1], max_context=s["longest"], want_lse=True)


def run(state):
    if own:
        return _own(state)
    return {"beam": _plain_beam, "reorder": _plain_reorder, "write": _plain_write, "read": _plain_read,
            "attention": _plain_attention}[state["c"]["op"]](state)


def work(case):
    c, op = case, case["op"]
    if op == "beam":
        R, N = c["B"] * c["K"], c["B"] * c["n"]
        # a maximum, an exponential and a sum for each element
        return {"bytes": R * c["V"] * _SIZE[c["dtype"]] + R * 5 + N * 12, "flops": 4 * R * c["V"]}
    if op == "reorder":
        # parents drawn with replacement: K * (1 - (1 - 1/K)^K) of a request's rows go on
        K = c["K"]
        on = K * (1 - (1 - 1 / K) ** K)
        row = 0.75 * c["T"] * c["H"] * c["D"] * _SIZE[c["dtype"]] * c["count"]
        # in place the rows that go on stay, and those with a second child are read (about a quarter of K)
        moved = (K - on) + K * (1 - (1 - 1 / K) ** K - (1 - 1 / K) ** (K - 1)) if c["in_place"] else on + K
        return {"bytes": int(c["B"] * row * moved), "flops": 0}
    if op in ("write", "read"):
        one = c["N"] * c["H"] * c["D"]
        exps = 2 * c["N"] * c["H"] if c["cache"] == "e4m3" else 0
        return {"bytes": 2 * one * (_SIZE[c["dtype"]] + _SIZE[c["cache"]]) + exps + 8 * c["N"], "flops": 4 * one if exps else 0}
    tokens = c["B"] * (0.75 * c["L"] + c["T"])
    q = c["B"] * c["T"] * c["Hq"]
    cache = 2 * tokens * c["Hkv"] * (c["D"] * _SIZE[c["cache"]] + (1 if c["cache"] == "e4m3" else 0))
    return {"bytes": int(cache + 2 * q * c["D"] * _SIZE[c["dtype"]] + 4 * q), "flops": int(4 * tokens * c["T"] * c["Hq"] * c["D"])}


# -------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "beam":
        # each beam's own best first, then the best of those
        B, K, V, n = c["B"], c["K"], c["V"], c["n"]
        best = []
        for b in range(B):
            rows = []
            for k in range(K):
                base = s["scores"][b, k].double()
                if s["finished"][b, k]:
                    rows.append(base[None])
                else:
                    x = s["logits"][b * K + k].double()
                    rows.append(base + torch.topk(x, min(n, V)).values - torch.logsumexp(x, 0))
            every = torch.cat(rows + [torch.full((n,), float("-inf"), dtype=torch.float64, device="cuda")])
            best.append(torch.sort(every, descending=True).values[:n])
        return torch.stack(best), None, None
    if op == "reorder":
        to = s["states"] if s["out"] is None else s["out"]
        parent, lengths = s["parent"].cpu(), s["lengths"].cpu()
        made = []
        for x, t in zip(s["states"], to):
            x, t = x.double(), t.double()
            new = t.clone()
            for b in range(c["B"]):
                for j in range(c["K"]):
                    p = int(parent[b, j])
                    w = int(lengths[b, p])
                    new[b * c["K"] + j, :w] = x[b * c["K"] + p, :w]
            made.append(new)
        return made
    if op in ("write", "read"):
        slots = s["slots"]
        keep = torch.nonzero(slots >= 0)[:, 0]
        page, at = slots[keep] // c["page"], slots[keep] % c["page"]
        made = []
        if op == "read":
            for cache, exp in zip(s["caches"], s["exps"]):
                got = torch.zeros((c["N"], c["H"], c["D"]), dtype=torch.float64, device="cuda")
                x = cache.double()[page, at]
                got[keep] = x if exp is None else torch.ldexp(x, exp[page, at].int()[..., None] - 127)
                made.append(got)
            return tuple(made)
        for x, cache, exp in zip((s["k"], s["v"]), s["caches"], s["exps"]):
            x = x.double()[keep]
            to = cache.double()
            if exp is None:
                to[page, at] = x
                made.append(to)
                continue
            top = x.abs().amax(-1, keepdim=True)
            part, e = torch.frexp(torch.where(top > 0, top / 448, 1e-30))
            e = (e - (part == 0.5).int()).double()
            y = x / torch.exp2(e)
            # to four significant bits, and no finer than 2^-9
            step = torch.exp2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].double() - 4)
            to[page, at] = torch.round(y / step) * step
            made += [to, None]
        return made
    B, T, Hq, Hkv, D = (c[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    if 4.0 * B * T * Hq * D * (c["L"] + T) > 1e12:
        return None
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, Hq), dtype=torch.float64, device="cuda")
    for b in range(B):
        ctx = int(s["context"][b])
        at = torch.arange(ctx + T, device="cuda")
        page, off = (at * 0 + b, at) if s["table"] is None else (s["table"][b].long()[at // c["page"]], at % c["page"])
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
            a = s["q"][b, :, h].double() @ k[:, h // G].T / math.sqrt(D)
            a = torch.where(sees, a, float("-inf"))
            lse[b, :, h] = torch.logsumexp(a, 1)
            out[b, :, h] = torch.softmax(a, 1) @ v[:, h // G]
    return out, lse
