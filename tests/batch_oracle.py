"""Plain 64-bit forms of what differs from row to row in a batch (experts, adapters, sampling), on the CPU, from their
definitions.  Test infrastructure only."""
import math

import torch

U32 = 2.0**-24
HALF_STEP = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


def route(logits, k, score, bias, groups, top_groups, group_best, renorm, scale):
    """(weights float64 [tokens, k], ids [tokens, k]), one token at a time."""
    weights, ids = [], []
    for row in logits.double().tolist():
        n = len(row)
        x = [-math.inf if math.isnan(v) else v for v in row]
        if score == "softmax":
            m = max(x)
            e = [0.0 if v == -math.inf else 1.0 if v == m else math.exp(v - m) for v in x]
            s = [v / sum(e) if sum(e) > 0 else 0.0 for v in e]
        else:
            s = [0.0 if v == -math.inf else 1 / (1 + math.exp(-v)) if v > -700 else math.exp(v) for v in x]
        b = bias.double().tolist() if bias is not None else [0.0] * n
        c = [-math.inf if v == -math.inf or math.isnan(a + o) else a + o for a, o, v in zip(s, b, x)]
        size = n // groups
        # without a bias and without sums the logits themselves are compared: fp64 scores may no longer tell them apart
        by = c if bias is not None or (groups > 1 and group_best == 2) else x
        worth = [sum(sorted(by[g * size : (g + 1) * size])[-group_best:]) for g in range(groups)]
        worth = [-math.inf if math.isnan(w) else w for w in worth]
        kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        among = [e for g in kept for e in range(g * size, (g + 1) * size) if c[e] > -math.inf and by[e] > -math.inf]
        chosen = sorted(among, key=lambda e: (-by[e], e))[:k]
        total = sum(s[e] for e in chosen)
        w = [(s[e] / total if total > 0 else 0.0) if renorm else s[e] for e in chosen]
        weights.append([scale * v for v in w] + [0.0] * (k - len(chosen)))
        ids.append(chosen + [-1] * (k - len(chosen)))
    return torch.tensor(weights, dtype=torch.float64).view(-1, k), torch.tensor(ids, dtype=torch.int32).view(-1, k)


def lists(ids, n):
    flat = [i if 0 <= i < n else n for i in ids.flatten().tolist()]
    order = sorted(range(len(flat)), key=lambda p: flat[p])
    return torch.tensor(order, dtype=torch.int32), torch.tensor([sum(i < e for i in flat) for e in range(n + 1)], dtype=torch.int32)


def adapter(y, x, a, b, index, ranks, scale):
    """(out, size): the result and the sum of its terms' sizes."""
    out, size = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    for t, i in enumerate(index.tolist()):
        if not 0 <= i < a.shape[0]:
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        s = 1.0 if scale is None else float(scale[i])
        w, v = a[i, :r].double(), b[i, :, :r].double()
        out[t] += s * (v @ (w @ x[t].double()))
        size[t] = abs(s) * (v.abs() @ (w.abs() @ x[t].double().abs()))
    return out, size


def adapter_bound(out, size, cols, rank, dtype):
    """Three terms of a factor leave 2^-27 of it, and the products left out 2^-25: below one u = 2^-24 of each term.  fp32 sums
    of 3 (or 5) products per column and of the parts are off by one u each, relative to the sum of the terms' sizes;
    roundings are independent, add in squares, and sixteen times that is never reached.  Then the sum with y and the
    output's own rounding."""
    n = 16 * math.sqrt(5 * cols + 64) + 16 * math.sqrt(5 * rank + 64) + 4
    return min(n, 5 * (cols + rank) + 132) * U32 * size + (HALF_STEP[dtype] + U32) * out.abs() * 1.01 + 1e-37


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability) of one row (float64 [vocab])."""
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x.double())
    m = float(x.max())
    if m == -math.inf:
        return -1, -math.inf
    greedy = not temperature > 0
    z = torch.where(x == m, torch.zeros_like(x), (x - m) / (1.0 if greedy else temperature))
    e = torch.where((x > -math.inf) & ~z.isnan(), torch.exp(z), torch.zeros_like(x))
    logp = torch.log(e / e.sum())
    first = int((x == m).nonzero()[0, 0])
    if greedy:
        return first, float(logp[first])
    order = torch.sort(-x, stable=True).indices
    order = order[x[order] > -math.inf]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        w = e[order]
        n = int((w.cumsum(0) < max(top_p, 0.0) * w.sum()).sum()) + 1
        order = order[:n]
    if min_p > 0:
        order = order[e[order] >= min(min_p, 1.0)]
    order = torch.sort(order).values
    c = e[order].cumsum(0)
    if u >= 1:
        at = int((e[order] > 2.0**-44).nonzero()[-1, 0])
    else:
        at = min(int((c <= (u if u > 0 else 0.0) * c[-1]).sum()), len(order) - 1)
    token = int(order[at])
    return token, float(logp[token])
