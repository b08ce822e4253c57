"""examples/decode_hypotheses.py: beams and a drafted tree, end to end,
against the same model run in 64 bits without caches."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_logit_filter_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_hypotheses as m
    return m


def plain_logits(model, tokens):
    """[R, T, vocab] of full causal attention in 64 bits."""
    x = model.embed[tokens].double()
    R, T = tokens.shape
    G = model.Hq // model.Hkv

    def norm(y):
        return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    for i in range(model.layers):
        y = norm(x)
        q = (y @ model.wq[i].double()).view(R, T, model.Hq, model.D)
        k, v = (y @ model.wkv[i].double()).view(R, T, 2, model.Hkv, model.D).unbind(2)
        k, v = (t.repeat_interleave(G, 2) for t in (k, v))
        s = torch.einsum("rthd,rshd->rhts", q, k) / math.sqrt(model.D)
        s = s.masked_fill(~torch.tril(torch.ones(T, T, dtype=torch.bool, device=s.device)), -math.inf)
        x = x + torch.einsum("rhts,rshd->rthd", torch.softmax(s, -1), v).reshape(R, T, -1) @ model.wo[i].double()
    return norm(x) @ model.head.double()


@pytest.mark.parametrize("quantised", [False, True])
def test_beams_score_what_the_model_scores(ex, quantised):
    model = ex.ToyModel(seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    prompts = torch.randint(0, model.vocab, (3, 17), generator=g, device="cuda")
    B, beams, steps = 3, 4, 6
    tokens, scores = ex.beam_search(model, prompts, beams=beams, steps=steps, quantised=quantised)
    assert (scores[:, :-1] >= scores[:, 1:]).all()
    # every hypothesis scored again as a whole: its cache must have followed it
    rows = torch.cat([prompts.repeat_interleave(beams, 0), tokens.view(B * beams, steps)], 1)
    logp = torch.log_softmax(plain_logits(model, rows), -1)[:, prompts.shape[1] - 1:-1]
    want = logp.gather(2, rows[:, prompts.shape[1]:, None])[..., 0].sum(1).view(B, beams)
    # bf16 activations: logits of about 4 with 2^-8 a rounding through two layers; e4m3 keys and values 2^-4 each
    tol = steps * 4 * (8 * 2.0 ** -8 + (2 * 2.0 ** -4 if quantised else 0))
    assert (scores.double() - want).abs().max() <= tol
    assert len({tuple(t) for t in tokens[0].tolist()}) == beams


def test_tree_accepts_what_one_token_at_a_time_gives(ex):
    model = ex.ToyModel(seed=4)
    g = torch.Generator(device="cuda").manual_seed(6)
    prompt = torch.randint(0, model.vocab, (1, 30), generator=g, device="cuda")
    # the model's own next two tokens, one at a time over a cache of the same kind
    caches = ex.Caches(model, 1, 64, False)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    logits = model.forward(prompt, caches.attend(zero))[:, -1]
    first = int(logits.argmax())
    second = int(model.forward(torch.tensor([[first]], device="cuda"), caches.attend(zero + 30))[0, 0].argmax())
    # drafted: a wrong branch first, then the right one
    above = [0, 0, 0, 1, 2, 2]
    nodes = [int(prompt[0, -1]), (first + 1) % model.vocab, first, 5, (second + 1) % model.vocab, second]
    masks = [1]
    for i in range(1, 6):
        masks.append(masks[above[i]] | 1 << i)
    caches = ex.Caches(model, 1, 64, False)
    model.forward(prompt[:, :-1], caches.attend(zero))
    path, _ = ex.verify_tree(model, caches, zero + 29, torch.tensor([nodes], device="cuda"),
                             torch.tensor([masks], device="cuda"), above)
    assert path == [0, 2, 5]


def test_example_runs(ex, capsys):
    ex.main()
    assert "accepted nodes" in capsys.readouterr().out
