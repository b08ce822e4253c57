"""Plain 64-bit references of the decoding calls (include/topkp_decode.h), on
the CPU, written from the formulas in that header's comments."""
import math

import torch

E4M3 = torch.float8_e4m3fn
# half a step relative to the value
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def beam_candidates(logits, scores, finished, pad):
    """[B, K * V] float64 candidate scores; -inf where there is none."""
    B, K = scores.shape
    x = logits.double().reshape(B, K, -1)
    V = x.shape[2]
    xc = torch.where(torch.isinf(x), x, x.clamp(-60000, 60000))
    m = xc.amax(-1, keepdim=True)
    dead = torch.isinf(m)
    m = torch.where(dead, torch.zeros_like(m), m)
    total = torch.exp(xc - m).sum(-1, keepdim=True)
    total = torch.where(dead, torch.ones_like(total), total)
    s = scores.double()[..., None]
    cand = torch.where(torch.isinf(x) | torch.isinf(s), torch.full_like(x, -math.inf), s - torch.log(total) + (xc - m))
    if finished is not None:
        only = torch.where(torch.arange(V) == pad, s, torch.full_like(s, -math.inf))
        cand = torch.where(finished.bool()[..., None], only, cand)
    return cand.reshape(B, K * V)


def quantise(x):
    """e4m3 values (as float64) and exponent bytes of rows x [..., D]."""
    x = x.double()
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    amax = fin.amax(-1)
    m, e = torch.frexp(amax)                       # amax = m * 2^e, 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e.clamp(min=-126), torch.full_like(e, -126))
    y = torch.ldexp(x, -e[..., None]).clamp(-448, 448)
    _, ye = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(y), ye - 4)   # 4 significant bits, no finer than 2^-9
    return torch.round(y / step) * step, e + 127


def attention(q, k, v, ctx, n, sees, scale):
    """One request.  q [T, Hq, D], k, v [len, Hkv, D] float64 (tokens 0 .. ctx + n), sees [T, n] bool.
    Returns out, lse, weight sums of |v|, a bound of the products' magnitude, and how far a product may be off where
    Q is a sum of e4m3 terms: each element by half of e4m3's smallest step, 2^-10, with the row's largest at 224 or more."""
    T, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    absv = torch.zeros(T, Hq, D, dtype=torch.float64)
    big = torch.zeros(T, Hq, dtype=torch.float64)
    off = torch.zeros(T, Hq, dtype=torch.float64)
    for i in range(T):
        vis = torch.zeros(L, dtype=torch.bool)
        if i < n:
            vis[:ctx] = True
            vis[ctx:] = sees[i][: L - ctx]
        if not vis.any():
            continue
        for h in range(Hq):
            kk, vv = k[vis, h // G], v[vis, h // G]
            s = kk @ q[i, h] * scale
            m = s.max()
            p = torch.exp(s - m)
            t = p.sum()
            out[i, h] = p @ vv / t
            absv[i, h] = p @ vv.abs() / t
            lse[i, h] = m + torch.log(t)
            big[i, h] = (kk.abs() @ q[i, h].abs()).max() * scale
            off[i, h] = kk.abs().sum(1).max() * q[i, h].abs().max() * scale * 2.0 ** -17
    return out, lse, absv, big, off


def attention_bounds(dtype, out, lse, absv, big, L, D, vmax, off=0):
    """How far a result may be: the output's own rounding, the probabilities'
    (relative to the type, with fp16's absolute 2^-25 below its normal
    range), the products' fp32 sums, and the exponentials' and sums' fp32."""
    u, e32 = HALF[dtype], 2.0 ** -24
    ds = (D + 8) * e32 * big + off                # a product of D terms in fp32, scaled
    rel = 2 * ds + (L + 64) * e32 + 2.0 ** -21
    tol = u * out.abs() + absv * (u * (1 + u) + rel[..., None]) + 1e-30
    if dtype == torch.float16:
        tol = tol + L * 2.0 ** -25 * vmax + 2.0 ** -25
    return tol, ds + (L + 64) * e32 + 2.0 ** -21 + 4 * e32 * lse.abs().nan_to_num(posinf=0, neginf=0)
