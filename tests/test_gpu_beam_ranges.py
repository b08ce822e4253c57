"""Beam selection over the whole range of scores and logits: any finite size,
logits a step apart, wide beams with finished ones among them."""
import math

import pytest

torch = pytest.importorskip("torch")
np = pytest.importorskip("numpy")
from test_gpu_decode import T_, rows, tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu
INF = math.inf


# ------------------------------------------------------------ beam selection
def candidates(x, scores, finished, pad):
    """[B, K, V] float64 candidates from the formula, with no bound on scores or logits; -inf where there is none."""
    B, K = scores.shape
    x = x.double().view(B, K, -1)
    m = x.amax(-1, keepdim=True)
    none = torch.isinf(m)
    m = torch.where(none, torch.zeros_like(m), m)
    d = x - m
    total = torch.exp(d).sum(-1, keepdim=True)
    total = torch.where(none, torch.ones_like(total), total)
    s = scores.double()[..., None]
    cand = torch.where(torch.isinf(x) | torch.isinf(s), torch.full_like(x, -INF), s + (d - torch.log(total)))
    if finished is not None:
        only = torch.where(torch.arange(x.shape[2]) == pad, s, torch.full_like(s, -INF))
        cand = torch.where(finished.bool()[..., None], only, cand)
    return cand


def check(tk, x, scores, n, finished=None, pad=0):
    """Against 64 bits: descending candidates, one beam's in the order of its logits (the lower index of equal ones),
    those of two beams in either order where they differ by less than the sums' documented 1e-6 and 64 bits' own steps."""
    B, K = scores.shape
    V = x.shape[1]
    got = tk.beam_select(x.cuda(), scores.cuda(), n, finished=None if finished is None else finished.cuda(), pad_token=pad)
    score, parent, token = (t.cpu() for t in got)
    cand = candidates(x, scores, finished, pad)
    logit = x.double().view(B, K, V)
    for b in range(B):
        c, lg = cand[b].reshape(-1).numpy(), logit[b].reshape(-1).numpy()
        at = np.flatnonzero(c > -INF)
        if at.size > 4 * n + 64:  # only what may come out
            at = at[c[at] >= np.partition(c[at], -n)[-n]]
        # the last key counts first; within a beam by its logits whatever 64 bits make of the sums
        at = at[np.lexsort((at, -lg[at], at // V, -c[at]))]
        for j in range(n):
            if j >= at.size:
                assert score[b, j] == -INF and token[b, j] == -1 and parent[b, j] == j % K, (b, j)
                continue
            want, flat = float(c[at[j]]), int(parent[b, j]) * V + int(token[b, j])
            step = 2e-6 + abs(want) * 2.0 ** -50
            tol = step / 2 + abs(want) * 2.0 ** -24
            assert abs(float(score[b, j]) - want) <= tol, (b, j, float(score[b, j]), want)
            if flat != at[j]:
                assert int(parent[b, j]) != at[j] // V and abs(float(c[flat]) - want) <= step, (b, j, flat, int(at[j]), want)
        live = [(int(p), int(t)) for p, t in zip(parent[b], token[b]) if int(t) >= 0]
        assert len(set(live)) == len(live)
        for k in range(K):
            mine = [t for p, t in live if p == k]
            keys = [(-float(logit[b, k, t]), t) for t in mine]
            assert (finished is not None and finished[b, k]) or keys == sorted(keys), (b, k)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dead", [-1e7, -8388607.0, -8388609.0, -1e9, -3e38, 1e7, 1e9])
def test_beam_scores_of_any_size(tk, dtype, dead):
    """Marks of dead beams, over logits that are all negative, all positive and both."""
    for off in (-30.0, 30.0, 0.0):
        x = (rows(8, 5000, dtype, 3).float() + off).to(T_[dtype])
        s = torch.tensor([[0.0, dead, dead, dead], [-3.5, dead, -1.25, dead]])
        check(tk, x, s, 8)
        fin = torch.tensor([[0, 1, 0, 0], [1, 0, 0, 1]], dtype=torch.uint8)
        check(tk, x, s, 8, fin, pad=7)
        # fewer live candidates than are asked for: dead beams' follow in their order
        few = x.clone()
        few[0, 3:] = -INF
        few[4:, 2:] = -INF
        check(tk, few, s, 12, fin, pad=7)
    # every beam far
    check(tk, rows(8, 5000, dtype, 4), torch.full((2, 4), dead), 8)


def test_beam_scores_of_the_lowest_value(tk):
    low = torch.finfo(torch.float32).min
    check(tk, rows(6, 3000, "f32", 5) - 9, torch.tensor([[-2.0, low, low], [low, low, low]]), 70)
    check(tk, rows(6, 3000, "f32", 6), torch.tensor([[low, low, low], [low, 0.0, low]]), 9,
          torch.tensor([[1, 0, 1], [0, 1, 1]], dtype=torch.uint8))


@pytest.mark.parametrize("V,R_", [(3001, 4), (40001, 4), (33003, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_logits_of_any_size(tk, dtype, V, R_):
    """Logits beyond 6e4, as a temperature of 1e-4 makes them."""
    s = -torch.rand(R_ // 2, 2, generator=torch.Generator().manual_seed(V)) * 5
    t = T_[dtype]
    base = rows(R_, V, "f32", V)
    check(tk, (base * 1e4).to(t), s, 9)                # far on both sides
    check(tk, (base * 1e4 - 3e5).to(t), s, 9)          # all far below
    check(tk, (base * 1e4 + 3e5).to(t), s, 9)          # all far above
    check(tk, (base * 1e34).to(t), s, 9)
    x = base.to(t)
    x[0, V // 2] = 1e30                                # one far above a plain row
    x[1, ::3] = torch.finfo(t).min                     # masks
    x[1, 1] = -INF
    x[2] = torch.finfo(t).min
    x[2, V - 1] = -70000.0
    x[3] = -70000.0
    x[3, V // 3] = -65000.0
    check(tk, x, s, 9)
    # rows that cross the bounds between ordinary and far logits, rising and falling, steps of a few units
    ramp = torch.linspace(-30.0, 30.0, V)
    for mid in (-60000.0, -59900.0, 59900.0, 60000.0):
        x = torch.stack([mid + ramp, (mid + ramp).flip(0)]).repeat(R_ // 2, 1)
        check(tk, x.to(t), s, 9)
    wide = torch.linspace(-2e5, 2e5, V)
    check(tk, torch.stack([wide, wide.flip(0)]).repeat(R_ // 2, 1).to(t), s, 9)


def test_beam_logits_of_fp16_ends(tk):
    x = (rows(4, 5000, "f32", 8) * 2e4).clamp(-65504, 65504).to(torch.float16)
    check(tk, x, torch.zeros(2, 2), 9)
    check(tk, -x.abs(), torch.zeros(2, 2), 9)
    x = torch.full((2, 5000), -65504.0, dtype=torch.float16)
    x[0, 4321] = 3.0
    check(tk, x, torch.tensor([[0.0, -1.0]]), 9)


def test_beam_order_of_near_logits(tk):
    """Logits a step of fp32 apart, far finer than a candidate's 64-bit sum with its score and normaliser."""
    V = 4000
    g = torch.Generator().manual_seed(9)
    steps = torch.randperm(V, generator=g)
    one = torch.tensor([1e-7]).view(torch.int32)
    x = (one + steps.int()).view(torch.float32)[None]
    check(tk, torch.cat([x, x.flip(1)]), torch.zeros(1, 2), 64)
    check(tk, torch.cat([x * 1e-20, -x]), torch.tensor([[-300.0, -300.0]]), 64)
    # equal ones by index, signed zeros are equal
    z = torch.zeros(2, V)
    z[0, ::2] = -0.0
    z[1, 5::7] = 1e-30
    check(tk, z, torch.tensor([[0.0, -1.0]]), 30)


@pytest.mark.parametrize("dtype,K,V,B", [("f32", 16, 151936, 2), ("f32", 32, 151936, 1), ("f16", 12, 131072, 3),
                                         ("bf16", 4, 33001, 64), ("f32", 9, 152064, 1)])
def test_beam_many_wide_beams(tk, dtype, K, V, B):
    """Random logits with finished beams where a thread reads four pieces at once and a warp four vectors."""
    g = torch.Generator().manual_seed(K)
    scores = -torch.rand(B, K, generator=g) * 4
    fin = (torch.rand(B, K, generator=g) < 0.3).to(torch.uint8)
    scores[0, 1] = -1e9
    check(tk, rows(B * K, V, dtype, V), scores, 64, fin, pad=V - 1)
    check(tk, rows(B * K, V, dtype, V + 1), scores, K)


@pytest.mark.parametrize("dtype,K,V,n", [("f32", 32, 151936, 64), ("bf16", 16, 152064, 128), ("f16", 64, 32000, 100)])
def test_beam_few_live_among_many(tk, dtype, K, V, n):
    """One or two live beams hold all the best: the groups of units bound them badly, and thousands of units pass."""
    x = rows(K, V, dtype, n)
    for dead in (-INF, -1e9, -3e38, -40.0):
        s = torch.full((1, K), dead)
        s[0, K // 2] = -1.0
        check(tk, x, s, n)
        s[0, K - 1] = -1.5
        fin = torch.zeros(1, K, dtype=torch.uint8)
        fin[0, ::5] = 1
        check(tk, x, s, n, fin, pad=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_thousands_of_equal_units(tk, dtype):
    """More equal maxima than are listed at once, equal to the last bit or nearly so, over beams of equal and other scores."""
    K, V = 12, 151936
    s = torch.tensor([[0.0, -1.0, 0.0, -1e9, 0.0, -0.5, -INF, 0.0, -2.0, 0.0, 0.0, 0.0]])
    z = torch.zeros(K, V, dtype=T_[dtype])
    check(tk, z, s, 128)
    z[:, ::2] = -0.0
    z[7, 77777] = -1.0
    check(tk, z, s, 70, torch.tensor([[0, 0, 1, 0, 0, 0, 0, 1, 0, 0, 0, 1]], dtype=torch.uint8), pad=9)
    few = rows(K, V, dtype, 5).clamp(-2, 2).round()     # the largest value in every unit
    check(tk, few, s, 128)
    near = torch.full((K, V), 2.0).view(torch.int32) + torch.randint(0, 3, (K, V), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    check(tk, near.view(torch.float32).to(T_[dtype]), s, 64)


def test_beam_signed_zeros(tk):
    """Nothing but zeros of either sign, where bounds and sums are exactly zero too."""
    g = torch.Generator().manual_seed(2)
    for K, V, n in ((32, 1, 32), (32, 2, 50), (5, 1, 9), (3, 700, 20)):
        sign = torch.where(torch.rand(K, V, generator=g) < 0.5, 0.0, -0.0)
        fin = (torch.rand(1, K, generator=g) < 0.3).to(torch.uint8)
        for zero in (0.0, -0.0):
            check(tk, sign, torch.full((1, K), zero), n)
            check(tk, sign, torch.full((1, K), zero), n, fin)
            check(tk, torch.full((K, V), -0.0, dtype=torch.bfloat16), torch.full((1, K), zero), n, fin)
