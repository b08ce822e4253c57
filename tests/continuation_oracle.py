"""Plain references of the calls for several continuations of one prompt
(include/topkp_decode.h): 64-bit values or lists, on the CPU, written from
the comments of that header."""
import math

import torch


def _softmax(x):
    x = x.double()
    m = float(x.max())
    if m == -math.inf:
        return torch.zeros_like(x), None
    e = torch.exp(x - m)
    # log-probabilities by way of x - m: beside a maximum of 1e38 the sum's logarithm would be lost
    return e / e.sum(), (x - m) - math.log(float(e.sum()))


def verify(target, draft, tokens, parent, n, uniform, race, eps, greedy=False):
    """One request: target, draft [T, V] or None, lists of tokens, parents (or None) and numbers.
    Returns (path, token, log-probabilities, margin): the least distance of a decision's two sides, relative to p or
    to the larger candidate."""
    V = target.shape[1]
    if n == 0:
        return [], -1, [], math.inf
    node, path, logprob, margin = 0, [0], [], math.inf
    while True:
        p, logp = _softmax(target[node])
        kids = [i for i in range(node + 1, n) if (parent[i] if parent is not None else i - 1) == node]
        now, chosen, weight = p, None, 1.0            # what is left of p, normalised; its sum before that
        if greedy:
            x = target[node].double()
            drawn = int(torch.nonzero(x == x.max())[0]) if float(x.max()) > -math.inf else -1
            chosen = next((i for i in kids if tokens[i] == drawn and drawn >= 0), None)
        else:
            q = _softmax(draft[node])[0] if draft is not None else None
            for i in kids:
                t = tokens[i]
                if not 0 <= t < V:
                    continue
                left, right = float(uniform[i]) * (float(q[t]) if q is not None else 1.0), float(now[t])
                if p[t] > 0:
                    # before the division by the sum the sides carry errors relative to p and to their own size
                    margin = min(margin, abs(left - right) * weight / max(left * weight, float(p[t])))
                if left < right:
                    chosen = i
                    break
                if q is None:
                    now = now.clone()
                    now[t] = 0
                else:
                    now = torch.relu(now - q)
                s = float(now.sum())
                now, weight = (now / s if s > 0 else now), weight * s
            if chosen is None:
                if not (now > 0).any():
                    now = p
                key = now / (race.double() + eps)
                best = torch.sort(key, descending=True, stable=True)
                drawn = int(best.indices[0]) if float(best.values[0]) > 0 else -1
                if V > 1 and drawn >= 0:
                    a, b = float(best.values[0]), float(best.values[1])
                    # p - a q carries an error relative to p
                    scale = 1.0 if q is None or weight == 0 else max(1.0, float(p[drawn] / (now[drawn] * weight)))
                    margin = min(margin, (a - b) / a / scale if math.isfinite(a) else math.inf)
        if chosen is None:
            logprob.append(float(logp[drawn]) if drawn >= 0 else 0.0)
            return path, drawn, logprob, margin
        logprob.append(float(logp[tokens[chosen]]))
        node = chosen
        path.append(node)


def fork(table, lengths, source, refs, grow, page_size):
    """Lists in, lists out: (new table, new refs, missing, copies as (from, to, tokens))."""
    pool, M, P = len(refs), len(table[0]) if table else 0, page_size

    def good(p):
        return p if 0 <= p < pool else -1
    hold = list(refs)
    for row in table:
        for p in row:
            if good(p) >= 0:
                hold[p] -= 1
    rows, claims, needs = [], {}, []
    for n, s in enumerate(source):
        length = min(max(lengths[s], 0), M * P) if 0 <= s < len(table) else 0
        full = [good(p) for p in table[s][: length // P]] if length else []
        for p in full:
            if p >= 0:
                hold[p] += 1
        part = length % P
        last = good(table[s][len(full)]) if part else -1
        if last >= 0:
            claims.setdefault(last, []).append(n)
        rows.append((full, part, last))
        needs.append(min(M, -(-(length + max(grow[n], 0)) // P)))
    keeper = {p: who[0] for p, who in claims.items() if hold[p] == 0}
    for p in keeper:
        hold[p] += 1
    free = [p for p in range(pool) if hold[p] == 0]
    new, copies, used = [], [], 0
    for n, (full, part, last) in enumerate(rows):
        row = list(full)
        if part:
            if last < 0 or keeper.get(last) == n:
                row.append(last)
            else:
                row.append(("fresh", used))
                copies.append((last, used, part))
                used += 1
        while len(row) < needs[n]:
            row.append(("fresh", used))
            used += 1
        new.append(row + [-1] * (M - len(row)))
    if used > len(free):
        return [[-1] * M for _ in source], list(refs), used - len(free), []
    for k in range(used):
        hold[free[k]] = 1
    new = [[free[p[1]] if isinstance(p, tuple) else p for p in row] for row in new]
    return new, hold, 0, [(a, free[k], t) for a, k, t in copies]


def compact(states, start, keep, kept, table, time_dim=1):
    """Copies of the states [pages, ...] with the kept tokens moved."""
    made = []
    for x in states:
        old, new = x.movedim(time_dim, 1), x.clone()
        to = new.movedim(time_dim, 1)
        P = old.shape[1]
        for b in range(len(start)):
            row = [b] if table is None else table[b]

            def place(t):
                if t < 0 or t >= len(row) * P or not 0 <= row[t // P] < x.shape[0]:
                    return None
                return row[t // P], t % P
            for j in range(min(max(kept[b], 0), len(keep[b]))):
                k = keep[b][j]
                if k <= j or start[b] < 0:
                    continue
                f, t = place(start[b] + k), place(start[b] + j)
                if f is not None and t is not None:
                    to[t] = old[f]
        made.append(new)
    return made
