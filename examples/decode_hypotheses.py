"""Decoding with several hypotheses at once, end to end, on a toy attention
model with random weights.

    python examples/decode_hypotheses.py

``beam_search``: every step writes the beams' new keys and values into caches
(quantised to e4m3 as they are written, if asked for), attends one token a
beam over them, selects the best continuations over beams and vocabulary, and
lets the caches follow the selected beams in place.

``verify_tree``: a tree of drafted tokens goes through the model in one pass
over the same kind of cache; the filter and the sample pick a token after
every node, and the longest drafted path that agrees with them is accepted.

``sample_drafted``: one prompt goes on as several samples over a paged cache.
Its pages are shared, attention reads the prompt once for all samples, and each
round a drafted tree of every sample is verified against the target's
probabilities, its accepted tokens move up behind the context, and pages grow
or return to the pool, all without a word from the host.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_logit_filter_gb300 as tk  # noqa: E402


class ToyModel:
    """Attention layers with a residual and an RMS norm; no positions."""

    def __init__(self, vocab=1024, layers=2, Hq=8, Hkv=2, D=64, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.vocab, self.layers, self.Hq, self.Hkv, self.D = vocab, layers, Hq, Hkv, D
        d = Hq * D

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) / math.sqrt(shape[0])).to(torch.bfloat16)

        self.embed = torch.randn(vocab, d, generator=g, device=device).to(torch.bfloat16)
        self.wq = [weight(d, d) for _ in range(layers)]
        self.wkv = [weight(d, 2 * Hkv * D) for _ in range(layers)]
        self.wo = [weight(d, d) for _ in range(layers)]
        self.head = weight(d, vocab) * 4

    def norm(self, x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def forward(self, tokens, attend):
        """tokens [R, T]; attend(layer, q, k, v) -> like q.  Returns logits [R, T, vocab]."""
        x = self.embed[tokens]
        R, T = tokens.shape
        for i in range(self.layers):
            y = self.norm(x)
            q = (y @ self.wq[i]).view(R, T, self.Hq, self.D)
            k, v = (y @ self.wkv[i]).view(R, T, 2, self.Hkv, self.D).unbind(2)
            x = x + attend(i, q, k, v).reshape(R, T, -1) @ self.wo[i]
        return self.norm(x) @ self.head


class Caches:
    """A cache a layer, [rows, capacity, heads, dim], of bf16 or e4m3."""

    def __init__(self, model, rows, capacity, quantised, device="cuda"):
        kind = torch.float8_e4m3fn if quantised else torch.bfloat16
        shape = (rows, capacity, model.Hkv, model.D)
        self.kv = [[torch.zeros(shape, dtype=torch.uint8 if quantised else kind, device=device).view(kind) for _ in (0, 1)]
                   for _ in range(model.layers)]
        self.exp = [[torch.zeros(shape[:3], dtype=torch.uint8, device=device) if quantised else None for _ in (0, 1)]
                    for _ in range(model.layers)]
        self.capacity = capacity
        self.first = torch.arange(rows, device=device)[:, None] * capacity

    def attend(self, lengths, tree=None):
        """For ToyModel.forward: new tokens stand at lengths[r] and on."""
        def run(layer, q, k, v):
            R, T = q.shape[:2]
            slots = (self.first + lengths[:, None] + torch.arange(T, device=q.device)).view(-1)
            (kc, vc), (ke, ve) = self.kv[layer], self.exp[layer]
            tk.cache_write(k.reshape(R * T, *k.shape[2:]), v.reshape(R * T, *v.shape[2:]), slots, kc, vc, k_exp=ke, v_exp=ve)
            return tk.tree_attention(q, kc, vc, lengths.int(), tree=tree, k_exp=ke, v_exp=ve)
        return run

    def reorder(self, parent, lengths):
        states = [t for pair in self.kv + self.exp for t in pair if t is not None]
        tk.beam_reorder(states, parent, lengths=lengths)


def beam_search(model, prompts, beams=4, steps=8, end=None, quantised=True):
    """prompts [B, P].  Returns tokens [B, beams, steps] and scores [B, beams], best first."""
    B, P = prompts.shape
    dev = prompts.device
    caches = Caches(model, B * beams, P + steps, quantised)
    rows = prompts.repeat_interleave(beams, 0)
    lengths = torch.zeros(B * beams, dtype=torch.int64, device=dev)
    logits = model.forward(rows, caches.attend(lengths))[:, -1].contiguous()
    lengths += P
    # one live beam: all hold the prompt
    scores = torch.full((B, beams), -math.inf, device=dev)
    scores[:, 0] = 0.0
    finished = torch.zeros((B, beams), dtype=torch.bool, device=dev)
    history = torch.zeros((B, beams, 0), dtype=torch.int64, device=dev)
    for step in range(steps):
        scores, parent, token = tk.beam_select(logits, scores, beams, finished=finished, pad_token=0 if end is None else end)
        at = parent.long()
        history = torch.cat([history.gather(1, at[..., None].expand(-1, -1, step)), token.long()[..., None]], 2)
        finished = finished.gather(1, at) | (token == (-2 if end is None else end))
        if step + 1 < steps:
            caches.reorder(parent, lengths.view(B, beams).int())
            logits = model.forward(token.long().clamp(min=0).view(-1, 1), caches.attend(lengths))[:, 0].contiguous()
            lengths += 1
    return history, scores


def verify_tree(model, caches, lengths, tokens, tree, above, k=50):
    """One request's drafted tree: tokens [1, T] (node 0 the last accepted
    token), tree [1, T] its masks, above [T] each node's parent.  Returns the
    accepted nodes, the first included, and the token to go on with."""
    logits = model.forward(tokens, caches.attend(lengths, tree))[0].contiguous()
    T = tokens.shape[1]
    top = torch.full((T,), k, dtype=torch.int32, device=tokens.device)
    chosen, _ = tk.apply_sample(logits, k=top, want_out=False)   # the filter's best token after each node
    chosen, tokens = chosen.tolist(), tokens[0].tolist()
    path = [0]
    while True:
        child = [i for i in range(T) if above[i] == path[-1] and i and tokens[i] == chosen[path[-1]]]
        if not child:
            return path, chosen[path[-1]]
        path.append(child[0])


class PagedCaches:
    """Pages of keys and values a layer, a block table and the pages' holders."""

    def __init__(self, model, pool, page_size, max_pages, device="cuda"):
        shape = (pool, page_size, model.Hkv, model.D)
        self.kv = [[torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in (0, 1)] for _ in range(model.layers)]
        self.states = [t for pair in self.kv for t in pair]
        self.page_size = page_size
        self.pages = torch.full((0, max_pages), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(0, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pool, dtype=torch.int32, device=device)

    def fork(self, source, grow):
        """Row n goes on from row source[n] (-1: it begins), with room for ``grow`` more tokens."""
        self.pages, _, self.missing = tk.cache_fork(self.states, self.pages, self.lengths, source, self.refs, grow=grow, refs_out=self.refs)
        old = torch.cat([self.lengths, torch.zeros(1, dtype=torch.int32, device=source.device)])
        self.lengths = old[source.long()]  # (-1 is the last, a zero)

    def attend(self, tree=None, shared=None, longest=None, prefix=None):
        """For ToyModel.forward: new tokens stand at lengths[r] and on."""
        def run(layer, q, k, v):
            R, T = q.shape[:2]
            at = self.lengths[:, None].long() + torch.arange(T, device=q.device)
            page = self.pages.long().gather(1, at // self.page_size)
            slots = torch.where(page >= 0, page * self.page_size + at % self.page_size, -1).view(-1)
            kc, vc = self.kv[layer]
            tk.cache_write(k.reshape(R * T, *k.shape[2:]), v.reshape(R * T, *v.shape[2:]), slots, kc, vc)
            if shared is None:
                return tk.tree_attention(q, kc, vc, self.lengths, pages=self.pages, tree=tree)
            return tk.shared_attention(q, kc, vc, self.lengths, self.pages, shared, tree=tree, max_context=longest, max_shared=prefix)
        return run


def sample_drafted(model, prompt, samples=8, rounds=6, page_size=16, above=(0, 0, 0, 1, 1, 2, 3), seed=0):
    """prompt [P], P > 1.  Draws ``samples`` continuations of it; ``above`` is each drafted node's parent.
    Returns each sample's tokens, and the log-probability the target gave them when they were accepted or drawn."""
    dev = prompt.device
    g = torch.Generator(device=dev).manual_seed(seed)
    T, P, N = len(above), prompt.numel(), samples
    parent = torch.tensor(above, dtype=torch.int32, device=dev).expand(N, T).contiguous()
    masks = [1]
    for i in range(1, T):
        masks.append(masks[above[i]] | 1 << i)
    tree = torch.tensor(masks, device=dev).expand(N, T).contiguous()
    longest = P + rounds * T
    caches = PagedCaches(model, pool=(N + 1) * (-(-longest // page_size) + 1), page_size=page_size, max_pages=-(-longest // page_size) + 1)
    # the prompt but its last token, once; then a row for each sample
    caches.fork(torch.full((1,), -1, dtype=torch.int32, device=dev), P - 1)
    model.forward(prompt[None, :-1], caches.attend())
    caches.lengths += P - 1
    shared = caches.lengths.clone()
    caches.fork(torch.zeros(N, dtype=torch.int32, device=dev), T)
    stay = torch.arange(N, dtype=torch.int32, device=dev)
    last = prompt[-1].expand(N).clone()
    out, logps = [[] for _ in range(N)], [[] for _ in range(N)]

    def race(*shape):
        return torch.empty(shape, device=dev).exponential_(generator=g)

    for _ in range(rounds):
        # a cheap draft: what the embedding alone says comes next, a token of each node's parent's distribution
        tokens = last[:, None].expand(N, T).clone()
        draft = torch.empty((N, T, model.vocab), device=dev, dtype=torch.bfloat16)
        for i in range(T):
            if i:
                tokens[:, i] = (draft[:, above[i]].float() - torch.log(race(N, model.vocab))).argmax(1)
            draft[:, i] = model.norm(model.embed[tokens[:, i]]) @ model.head
        target = model.forward(tokens, caches.attend(tree, shared, longest, P - 1))
        count, path, token, logp = tk.draft_verify(target, tokens.int(), torch.rand((N, T), generator=g, device=dev), race(N, model.vocab),
                                                   draft=draft, parent=parent, want_logprob=True)
        tk.cache_compact(caches.states, caches.lengths, path, count, pages=caches.pages)
        caches.lengths = caches.lengths + count
        caches.fork(stay, T)     # pages past the accepted tokens return, new ones come
        last = token.long()
        # (the host only looks on)
        for n, (c, p, t, l) in enumerate(zip(count.tolist(), path.tolist(), token.tolist(), logp.tolist())):
            out[n] += [int(tokens[n, i]) for i in p[1:c]] + [t]
            logps[n] += l[:c]
    assert int(caches.missing) == 0
    return out, logps


def main():
    model = ToyModel()
    prompts = torch.randint(0, model.vocab, (2, 12), device="cuda")
    for quantised in (False, True):
        tokens, scores = beam_search(model, prompts, quantised=quantised)
        print("e4m3 cache" if quantised else "bf16 cache", "best beam", tokens[0, 0].tolist(), "score %.3f" % float(scores[0, 0]))
    # a tree of seven nodes after the prompt's last token: two children each
    caches = Caches(model, 1, 64, True)
    start = torch.zeros(1, dtype=torch.int64, device="cuda")
    model.forward(prompts[:1, :-1], caches.attend(start))
    above = [0, 0, 0, 1, 1, 2, 2]
    masks = [1]
    for i in range(1, 7):
        masks.append(masks[above[i]] | 1 << i)
    nodes = torch.cat([prompts[:1, -1:], torch.randint(0, model.vocab, (1, 6), device="cuda")], 1)
    path, token = verify_tree(model, caches, start + prompts.shape[1] - 1, nodes, torch.tensor([masks], device="cuda"), above)
    print("accepted nodes", path, "next token", token)
    out, _ = sample_drafted(model, prompts[0])
    print("samples of one prompt:", [len(t) for t in out], "tokens, the first", out[0])
    tk.device_status()


if __name__ == "__main__":
    main()
