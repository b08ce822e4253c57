"""The calls for several continuations of one prompt run together: samples of
one prompt over shared pages, with drafted trees, against the same model run in
64 bits without caches, and against the calls one request at a time."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
from test_gpu_decode_example import ex, plain_logits  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("above,page_size,P", [((0, 0, 0, 1, 1, 2, 3), 16, 40), ((0, 0, 1, 2, 3), 5, 33), ((0,), 16, 17), ((0, 0, 0, 0, 0, 0), 64, 130)])
def test_samples_are_scored_as_the_model_scores_them(ex, above, page_size, P):  # noqa: F811
    """Every emitted token's log-probability is that of its own sample's whole text: pages, forks, compactions and the shared
    prefix have followed it."""
    model = ex.ToyModel(seed=7)
    g = torch.Generator(device="cuda").manual_seed(P)
    prompt = torch.randint(0, model.vocab, (P,), generator=g, device="cuda")
    out, logps = ex.sample_drafted(model, prompt, samples=6, rounds=7, page_size=page_size, above=above, seed=P)
    longer = 0
    for tokens, logp in zip(out, logps):
        assert len(tokens) == len(logp) and len(tokens) >= 7
        longer += len(tokens) > 7
        text = torch.cat([prompt, torch.tensor(tokens, device="cuda")])[None]
        want = torch.log_softmax(plain_logits(model, text)[0, P - 1:-1], -1).gather(1, text[0, P:, None])[:, 0]
        # bf16 activations: logits of about 4 with 2^-8 a rounding through two layers
        assert (torch.tensor(logp, device="cuda").double() - want).abs().max() <= 4 * 8 * 2.0 ** -8
    assert len({tuple(t) for t in out}) == 6
    if len(above) > 1:
        assert longer > 0    # some drafted token was accepted


def test_a_pool_that_runs_dry_says_so(ex):  # noqa: F811
    model = ex.ToyModel(seed=8)
    prompt = torch.randint(0, model.vocab, (20,), device="cuda")
    caches = ex.PagedCaches(model, pool=3, page_size=8, max_pages=9)
    caches.fork(torch.full((1,), -1, dtype=torch.int32, device="cuda"), 19)
    assert int(caches.missing) == 0 and (caches.refs == 1).all()
    model.forward(prompt[None, :-1], caches.attend())
    caches.lengths += 19
    before = [t.clone() for t in caches.states]
    caches.fork(torch.zeros(4, dtype=torch.int32, device="cuda"), 6)
    # three copies of the last page, and a page more for each of the four: 19 + 6 tokens
    assert int(caches.missing) == 7 and (caches.refs == 1).all() and (caches.pages == -1).all()
    assert all(torch.equal(a, b) for a, b in zip(before, caches.states))


def test_a_round_in_a_graph(ex):  # noqa: F811
    """Verification, compaction, forking and attention captured together, replayed over changing inputs: as the same calls made one by one."""
    import top_logit_filter_gb300 as tk
    g = torch.Generator(device="cuda").manual_seed(3)
    N, T, V, P, M, pool, H, D = 24, 5, 3000, 16, 12, 400, 2, 64
    parent = torch.tensor([0, 0, 0, 1, 2], dtype=torch.int32, device="cuda").expand(N, T).contiguous()
    masks = torch.tensor([1, 3, 5, 11, 21], device="cuda").expand(N, T).contiguous()

    def fresh():
        target = torch.randn((N, T, V), generator=g, device="cuda") * 2
        target[:, :, :3] += 7
        draft = target + 0.5 * torch.randn((N, T, V), generator=g, device="cuda")
        tokens = torch.randint(0, 3, (N, T), generator=g, device="cuda", dtype=torch.int32)
        lengths = 70 + torch.randint(0, 60, (N,), generator=g, device="cuda", dtype=torch.int32)
        table = torch.full((N, M), -1, dtype=torch.int32, device="cuda")
        order = torch.randperm(pool, generator=g, device="cuda").int()
        table[:, :4] = order[:4]                         # four pages for all
        need = (lengths + T + P - 1) // P
        mine = order[4 + torch.arange(N, device="cuda")[:, None] * 8 + torch.arange(8, device="cuda")[None]]
        table[:, 4:] = torch.where(torch.arange(4, M, device="cuda")[None] < need[:, None], mine, -1)
        refs = torch.bincount(table[table >= 0].long(), minlength=pool).int()
        k, v = (torch.randn((pool, P, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in (0, 1))
        q = torch.randn((N, T, 8, D), generator=g, device="cuda").to(torch.bfloat16)
        return dict(target=target, draft=draft, tokens=tokens, lengths=lengths, table=table, refs=refs, k=k, v=v, q=q,
                    uniform=torch.rand((N, T), generator=g, device="cuda"), race=torch.empty((N, V), device="cuda").exponential_(generator=g),
                    source=torch.randint(0, N, (N,), generator=g, device="cuda", dtype=torch.int32))

    shared = torch.tensor([64], dtype=torch.int32, device="cuda")

    def step(s):
        a = tk.shared_attention(s["q"], s["k"], s["v"], s["lengths"], s["table"], shared, tree=masks, max_context=100000, max_shared=90000)
        count, path, token, logp = tk.draft_verify(s["target"], s["tokens"], s["uniform"], s["race"], draft=s["draft"], parent=parent, want_logprob=True)
        tk.cache_compact([s["k"], s["v"]], s["lengths"], path, count, pages=s["table"])
        table, refs, missing = tk.cache_fork([s["k"], s["v"]], s["table"], s["lengths"] + count, s["source"], s["refs"], grow=T)
        return a, count, path, token, logp, table, refs, missing

    s = fresh()
    step({k: v.clone() for k, v in s.items()})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step({k: v.clone() for k, v in s.items()})
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    for _ in range(3):
        new = fresh()
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        want = step(new)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(s["k"], new["k"]) and torch.equal(s["v"], new["v"])
        assert int(want[-1]) == 0
    tk.device_status()


def test_example_runs(ex, capsys):  # noqa: F811
    ex.main()
    assert "samples of one prompt" in capsys.readouterr().out
