"""draft_verify with certain drafts where a rejected token held nearly all of
the row: the decision on the next child, against 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
from test_gpu_verify import T_, check, make, tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# How far a decision's sides are put from one another, relative to p.  The kernel's may be off by: an exponential 2^-22 and
# two roundings of 2^-24 each, about 4e-7, on either side; the row's sum, of batches of 16 terms, 30 roundings of 2^-24 at
# the most where they all go one way, 2e-6, and about 2e-7 as they come; what is left of it at the most twice that.
APART = 5e-6
LAST = 1.0 - 2.0 ** -24   # the largest number of [0, 1): rejects all but 2^-24


def sharp(dtype, V, masses, share, side, seed, repeat=False):
    """One request: the root's children take masses[0] of the row, masses[1] of the rest and so on, and are all rejected
    but the last, which has `share` of what is left then and whose number lies APART from its probability.  With `repeat`
    each rejected token is tried twice."""
    g = torch.Generator().manual_seed(seed)
    K = len(masses) + 1
    x = torch.log_softmax(torch.randn(V, generator=g).double(), 0)
    at = torch.randperm(V, generator=g)[:K]
    left = 1.0
    for i, m in enumerate(masses):
        x[at[i]] = math.log(left * m)
        left *= 1 - m
    rest = torch.ones(V, dtype=torch.bool)
    rest[at] = False
    x[at[-1]] = math.log(left * share)
    x[rest] += math.log(left * (1 - share)) - torch.logsumexp(x[rest], 0)
    x = x.float().to(T_[dtype])
    p = torch.softmax(x.double(), 0)
    first = [t for t in at[:-1].tolist() for _ in range(2 if repeat else 1)]
    kids = first + [int(at[-1])]
    # the probability of the last child among what is left, in 64 bits of the rounded logits
    taken = torch.zeros(V, dtype=torch.bool)
    taken[at[:-1]] = True
    border = float(p[at[-1]] / p[~taken].sum())
    uniform = [0.5] + [LAST] * len(first) + [border * (1 + side * APART)]
    return x, kids, uniform


def batch(dtype, V, cases):
    T = 1 + max(len(k) for _, k, _ in cases)
    B = len(cases)
    d = make(B, T, V, dtype, "certain", True, seed=V)
    d["parent"][:] = 0
    for b, (x, kids, uniform) in enumerate(cases):
        d["target"][b, 0] = x
        d["tokens"][b, 1:] = -1                    # (no token: never accepted, changes nothing)
        d["tokens"][b, 1:1 + len(kids)] = torch.tensor(kids, dtype=torch.int32)
        d["uniform"][b, :len(uniform)] = torch.tensor(uniform)
    return d


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [777, 32000, 32003, 128256])
def test_a_rejected_token_that_held_nearly_all(tk, dtype, V):  # noqa: F811
    cases, want = [], []
    for i, mass in enumerate((0.3, 0.49, 0.6, 0.9, 0.994, 1 - 5e-4, 1 - 1.1e-4, 1 - 1.5e-5)):
        for share in (0.9, 0.3, 0.01):
            for side in (-1, 1):
                cases.append(sharp(dtype, V, [mass], share, side, i))
                want.append(2 if side < 0 else 1)
    count = check(tk, batch(dtype, V, cases), most_near=0)
    assert count.tolist() == want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1000, 32000])
def test_one_after_another(tk, dtype, V):  # noqa: F811
    """Several rejected tokens, each most of what the ones before it left; some tried again."""
    cases, want = [], []
    for i, masses in enumerate(([0.9, 0.9], [0.5, 0.6, 0.7, 0.8], [0.99, 0.99], [0.9] * 4, [0.2] * 8, [0.97, 0.1, 0.95], [0.3, 0.999])):
        for side in (-1, 1):
            for repeat in (False, True):
                cases.append(sharp(dtype, V, masses, 0.4, side, 10 + i, repeat))
                want.append(2 if side < 0 else 1)
    count = check(tk, batch(dtype, V, cases), most_near=0)
    assert count.tolist() == want


def test_one_request_and_many(tk):  # noqa: F811
    """Clusters of sixteen CTAs to one."""
    for copies in (1, 3, 20, 80, 330):
        cases = [sharp("bf16", 32000, [0.998, 0.9], 0.5, side, 5) for side in (-1, 1)]
        d = batch("bf16", 32000, (cases * copies)[:copies])
        assert check(tk, d, most_near=0).tolist() == [2 if i % 2 == 0 else 1 for i in range(copies)]


@pytest.mark.parametrize("drafted", [False, True])
def test_what_fp32_does_not_hold_counts_as_zero(tk, drafted):  # noqa: F811
    """A token 2^-127 times as probable as the largest: neither accepted nor drawn, where 2^-125 is."""
    for power, kept in ((-125, True), (-127, False)):
        x = torch.full((1, 2, 300), -math.inf)
        x[:, :, 7], x[:, :, 9] = 0.0, power * math.log(2.0)
        kw = dict(draft=x.cuda()) if drafted else {}
        race = torch.ones(1, 300)
        race[0, 7] = 2.0 ** 64                     # (and 9 has a race so short that it would win by a factor of two)
        race[0, 9] = 2.0 ** (64 + power - 1)
        tokens = torch.tensor([[0, 9]], dtype=torch.int32)
        count, path, token = tk.draft_verify(x.cuda(), tokens.cuda(), uniform=torch.zeros(1, 2).cuda(), race=race.cuda(), eps=0.0, **kw)
        assert int(count) == (2 if kept else 1) and int(token) == (9 if kept else 7), (power, int(count), int(token))
