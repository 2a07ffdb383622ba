"""Plain 64-bit forms of the operators between a block's projections, on the CPU, from their definitions: one token,
one head and one key at a time where that is what the definition says.  Test infrastructure only."""
import math

import torch

HALF_STEP = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
U32 = 2.0**-24


def rope_rows(x, positions, freq, layout, rope_scale=1.0, norm=None, eps=0.0):
    """x [tokens, heads, dim] -> normed and rotated rows (float64), and for each value the size of what it is summed from."""
    y = x.double().clone()
    if norm is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * norm.double()
    out, size = y.clone(), y.abs()
    rot = 0 if freq is None else 2 * freq.numel()
    for i in range(rot // 2):
        lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        a = positions.double() * freq[i]
        c, s = (a.cos() * rope_scale)[:, None], (a.sin() * rope_scale)[:, None]
        out[..., lo] = y[..., lo] * c - y[..., hi] * s
        out[..., hi] = y[..., hi] * c + y[..., lo] * s
        size[..., lo] = size[..., hi] = (y[..., lo].abs() + y[..., hi].abs()) * abs(rope_scale)
    return out, size


def attention(q, k_cache, v_cache, table, kv_len, cu, scale, window):
    """(out, lse, spread, logit size): spread = the probabilities' mean of |v|, logit size = max over keys of scale sum |q||k|."""
    tokens, heads, dim = q.shape
    _, kvh, page, _ = k_cache.shape
    group = heads // kvh
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    spread, size = torch.zeros_like(out), torch.zeros(tokens, heads, dtype=torch.float64)
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            pos = kv_len[b] - n + i
            low = max(0, pos - window + 1) if window else 0
            keys = list(range(low, pos + 1))
            if not keys:
                continue
            pages, at = table[b, [j // page for j in keys]].long(), torch.tensor([j % page for j in keys])
            for h in range(heads):
                k, v = k_cache[pages, h // group, at].double(), v_cache[pages, h // group, :, at].double()
                x = q[cu[b] + i, h].double()
                s = k @ x * scale
                p = torch.softmax(s, 0)
                t = cu[b] + i
                out[t, h], lse[t, h] = p @ v, torch.logsumexp(s, 0)
                spread[t, h], size[t, h] = p @ v.abs(), (k.abs() @ x.abs()).max() * abs(scale)
    return out, lse, spread, size


def attention_bound(out, spread, size, dim, keys, out_dtype, cache_dtype):
    """What rounding can do: a logit of `dim` exact products summed in fp32 is off by (dim + 4) u of its terms' sum, a
    probability by that much relatively, twice (numerator and sum); sums over keys by (keys + 16) u; probabilities in
    the cache's type by its half step where the output has that type; the output by its own."""
    logit = (dim + 4) * U32 * size[..., None]
    p = 0.0 if out_dtype == torch.float32 else HALF_STEP[cache_dtype]
    return spread * (2 * logit + (keys + 16) * U32 + p) * 1.01 + HALF_STEP[out_dtype] * out.abs() + 1e-30


def gdn(q, k, v, g, beta, state, cu, scale, l2norm, eps):
    """(out, states, column norm): the recurrence, and the largest norm that a column of a state or a value had."""
    hv, group = v.shape[1], v.shape[1] // q.shape[1]
    q, k, v, g, beta = q.double(), k.double(), v.double(), g.double(), beta.double()
    if l2norm:
        q = q / (q.square().sum(-1, keepdim=True) + eps).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + eps).sqrt()
    out, states = torch.zeros_like(v), state.double().clone()
    big = max(float(states.norm(dim=2).max()) if states.numel() else 0.0, float(v.abs().max()) if v.numel() else 0.0)
    for b in range(len(cu) - 1):
        for h in range(hv):
            s = states[b, h].clone()
            for t in range(cu[b], cu[b + 1]):
                kk, qq = k[t, h // group], q[t, h // group]
                s = s * g[t, h].exp()
                s = s + torch.outer(kk, beta[t, h] * (v[t, h] - s.T @ kk))
                out[t, h] = scale * (s.T @ qq)
                big = max(big, float(s.norm(dim=0).max()))
            states[b, h] = s
    return out, states, big


def gdn_bound(length, dk, big):
    """Absolute error of a state value.  Keys of norm one and decays of at most one never let an error grow, so the
    roundings add up: (length + 1) tokens of dk + 16 each, every one at most u of a column's norm.  Roundings are
    independent: they add in squares, and sixteen times that is never reached (nor is the plain sum)."""
    n = (length + 1) * (dk + 16)
    return min(n, 16 * math.sqrt(n)) * U32 * big
