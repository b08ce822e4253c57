"""The attention and the cache beyond the usual: far tails of fp16
probabilities, chains of more than 64 nodes, and the kernels that only many
tokens reach."""
import math

import pytest

torch = pytest.importorskip("torch")
import decode_oracle as R  # noqa: E402
from test_gpu_decode import T_, attend, awkward, ref_reorder, tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("T,D", [(1, 128), (16, 128), (40, 64), (80, 128), (3, 256)])
def test_attention_fp16_far_tail(tk, cache, T, D):
    """A few tokens at 1 and 2^18 of them 18 below, which together weigh a thousandth: all in one part of the work."""
    L, G, u = 1 << 18, 2, 2.0 ** -11
    kind = R.E4M3 if cache == "e4m3" else torch.float16
    k = torch.zeros(1, L + T, 1, D)
    v = torch.full((1, L + T, 1, D), 8.0)
    k[..., 0] = -18.0
    peaks = [0, 16, 32, 48]     # one for each quarter of the first tile
    k[:, peaks, :, 0] = 0.0
    v[:, peaks] = 1.0
    q = torch.zeros(1, T, G, D, dtype=torch.float16)
    q[..., 0] = 1.0
    kw = {}
    if cache == "e4m3":
        one = torch.full((1, L + T, 1), 127, dtype=torch.uint8).cuda()
        kw = dict(k_exp=one, v_exp=one.clone())
    out, lse = tk.tree_attention(q.cuda(), k.to(kind).cuda(), v.to(kind).cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                                 scale=1.0, max_context=1, want_lse=True, **kw)
    tk.device_status()
    for i in range(T):
        tail = (L - 4 + i + 1) * math.exp(-18.0)
        want = (4 + 8 * tail) / (4 + tail)
        # the sums of 64 tokens at a time and of all tiles; each tail probability is off by half of fp16's smallest
        # step, 2^-25, at 2^7 times its size or less often
        e = (L / 64 + 64) * 2.0 ** -24 + 2.0 ** -21
        tol = want * (u + e + L / 16 * 2.0 ** -24) + 8 * (L + T) * 2.0 ** -32
        assert (out[0, i].double().cpu() - want).abs().max() <= tol, (i, float(out[0, i, 0, 0]), want)
        assert (lse[0, i].double().cpu() - math.log(4 + tail)).abs().max() <= e


@pytest.mark.parametrize("dtype,cache", [("bf16", "own"), ("f16", "own"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("T,Hq,Hkv,D,P", [(65, 4, 2, 64, 16), (129, 3, 1, 128, 0), (500, 2, 1, 128, 48), (300, 1, 1, 256, 64)])
def test_attention_long_chains(tk, dtype, cache, T, Hq, Hkv, D, P):
    """Chains of more than 64 nodes, whole and ragged, over no context and some."""
    attend(tk, dtype, cache, T, Hq, Hkv, D, P, [0, 1, 70], seed=T)
    attend(tk, dtype, cache, T, Hq, Hkv, D, P, [0, 40, 333], nodes=[T, T // 2, 64], seed=T + 1)


# ---------------------------------------------------------------------- cache
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,H,D,P", [(5003, 8, 128, 48), (20011, 3, 80, 64), (40013, 1, 128, 16)])
def test_cache_of_many_tokens(tk, dtype, N, H, D, P):
    """As many rows as make a thread take four tokens."""
    g = torch.Generator().manual_seed(N)
    pages = -(-N // P) + 3
    slots = torch.randperm(pages * P, generator=g)[:N]
    slots[::31] = -1
    slots[5::97] = pages * P + 4
    keep = (slots >= 0) & (slots < pages * P)
    k, v = awkward(N, H, D, dtype, N), awkward(N, H, D, dtype, N + 1)
    ints = torch.int32 if dtype == "f32" else torch.int16
    kc, vc = (torch.zeros(pages, P, H, D, dtype=T_[dtype], device="cuda") for _ in (0, 1))
    tk.cache_write(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
    for x, c, r in zip((k, v), (kc, vc), tk.cache_read(slots.cuda(), kc, vc)):
        want = torch.zeros(pages * P, H, D, dtype=T_[dtype])
        want[slots[keep]] = x[keep]
        assert torch.equal(c.cpu().view(-1, H, D).view(ints), want.view(ints))
        back = x.clone()
        back[~keep] = 0
        assert torch.equal(r.cpu().view(ints), back.view(ints))
    kc, vc = (torch.zeros(pages, P, H, D, dtype=torch.uint8, device="cuda").view(R.E4M3) for _ in (0, 1))
    ke, ve = (torch.full((pages, P, H), 9, dtype=torch.uint8, device="cuda") for _ in (0, 1))
    tk.cache_write(k.cuda(), v.cuda(), slots.cuda(), kc, vc, k_exp=ke, v_exp=ve)
    read = {o: tk.cache_read(slots.cuda(), kc, vc, k_exp=ke, v_exp=ve, dtype=T_[o]) for o in ("f32", "f16", "bf16")}
    for i, (x, c, e) in enumerate(((k, kc, ke), (v, vc, ve))):
        q, byte = R.quantise(x)
        want, wexp = torch.zeros(pages * P, H, D, dtype=torch.float64), torch.full((pages * P, H), 9)
        want[slots[keep]], wexp[slots[keep]] = q[keep], byte[keep].long()
        assert torch.equal(e.cpu().view(-1, H).long(), wexp)
        got = c.cpu().view(torch.uint8).view(R.E4M3).float().double().view(-1, H, D)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(nan=0), want.nan_to_num(nan=0))
        value = torch.ldexp(q, byte[..., None] - 127)
        value[~keep] = 0
        for o, pair in read.items():
            w, r = value.float().to(T_[o]), pair[i].cpu()
            assert torch.equal(torch.isnan(r), torch.isnan(w))
            assert torch.equal(r.masked_fill(torch.isnan(r), 0), w.masked_fill(torch.isnan(w), 0)), o


# ----------------------------------------------------------------- reordering
@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 8), (torch.float32, 3), (torch.uint8, 5)])
def test_reorder_interleaved_views(tk, dtype, dim):
    """Keys and values of every layer in one tensor, rows outermost: all of them states of one call."""
    g = torch.Generator().manual_seed(dim)
    B, K = 3, 4
    c = torch.randint(0, 100, (B * K, 20, 2, 9, 2, dim), generator=g).to(dtype)
    parent = torch.randint(0, K, (B, K), generator=g, dtype=torch.int32)
    lengths = torch.randint(0, 12, (B, K), generator=g, dtype=torch.int32)
    for ln in (None, lengths):
        want = torch.stack([torch.stack([ref_reorder(c[:, i, j], c[:, i, j], parent, ln, 1) for j in (0, 1)], 1) for i in range(20)], 1)
        dev = c.cuda()
        tk.beam_reorder([dev[:, i, j] for i in range(20) for j in (0, 1)], parent.cuda(), lengths=None if ln is None else ln.cuda())
        assert torch.equal(dev.cpu(), want)
    # heads before time, and from one half into the other
    h = torch.randint(0, 100, (B * K, 3, 2, 9, dim), generator=g).to(dtype)
    want = torch.stack([ref_reorder(h[:, :, j], h[:, :, j], parent, None, 2) for j in (0, 1)], 2)
    dev = h.cuda()
    tk.beam_reorder([dev[:, :, j] for j in (0, 1)], parent.cuda(), time_dim=2)
    assert torch.equal(dev.cpu(), want)
    dev = c.cuda()
    tk.beam_reorder(dev[:, :, 0], parent.cuda(), out=dev[:, :, 1], time_dim=2)
    want = c.clone()
    want[:, :, 1] = ref_reorder(c[:, :, 0], c[:, :, 1], parent, None, 2)
    assert torch.equal(dev.cpu(), want)


@pytest.mark.parametrize("dtype,last,step,top", [("f16", 63456.0, 63488.0, 65536.0),
                                                 ("bf16", 1.9296875 * 2.0 ** 127, 1.9375 * 2.0 ** 127, math.inf),
                                                 ("f32", (1.9375 - 2.0 ** -23) * 2.0 ** 127, 1.9375 * 2.0 ** 127, math.inf)])
@pytest.mark.parametrize("D,P", [(64, 16), (7, 3)])
def test_cache_at_the_end_of_a_type(tk, dtype, last, step, top, D, P):
    """The rounding to e4m3 takes a type's largest magnitudes past its range; below them it does not."""
    t = T_[dtype]
    x = torch.ones(4, 1, D, dtype=t)
    x[0, 0, 1], x[1, 0, 2], x[2, 0, 3], x[3, 0, 0] = last, step, -step, torch.finfo(t).max
    c = torch.zeros(2, P, 1, D, dtype=torch.uint8, device="cuda").view(R.E4M3)
    e = torch.zeros(2, P, 1, dtype=torch.uint8, device="cuda")
    at = torch.arange(4, device="cuda")
    tk.cache_write(x.cuda(), None, at, c, None, k_exp=e)
    own, f32 = (tk.cache_read(at, c, None, k_exp=e, dtype=o)[0][:, 0].float().cpu() for o in (t, torch.float32))
    assert own[0, 1] == f32[0, 1] == (61440.0 if dtype == "f16" else 1.875 * 2.0 ** 127)
    assert own[1, 2] == math.inf and own[2, 3] == -math.inf and own[3, 0] == math.inf
    assert f32[1, 2] == top and f32[2, 3] == -top and f32[3, 0] == top
