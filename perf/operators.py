"""Measured cases of the operators between a block's projections: rotary append, paged attention, gated delta rule.

`listed()` and `draw()` give cases as plain dicts; `prepare()` makes a case's inputs from a seed; `run()` does one
pass, in plain torch where `own` is false and through the package where it is true; `exact()` evaluates the
definition in 64 bits, sequence by sequence and token by token; `work()` counts the bytes and operations that a pass
cannot do without.

Head layouts follow the projections of this repository's decode step (a 7168-row qkv product and a 6144-column output
product): 24 query and 2 key heads of 256, or 48 and 4 of 128.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
CHUNK = 64


# ---- cases ---------------------------------------------------------------------------------------------------------

def _append(name, tokens, heads, kv_heads, dim, rot, layout, norm, dtype, cache, page, start):
    c = {"op": "append", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
         "layout": layout, "norm": norm, "dtype": dtype, "cache": cache, "page": page, "start": start}
    return dict(c, name=name) if name else c


def _attn(name, seqs, new, keys, ragged, heads, kv_heads, dim, page, cache, out, window):
    c = {"op": "attn", "seqs": seqs, "new": new, "keys": keys, "ragged": ragged, "heads": heads, "kv_heads": kv_heads,
         "dim": dim, "page": page, "cache": cache, "out": out, "window": window}
    return dict(c, name=name) if name else c


def _gdn(name, seqs, length, ragged, k_heads, v_heads, dk, dv, dtype):
    c = {"op": "gdn", "seqs": seqs, "len": length, "ragged": ragged, "k_heads": k_heads, "v_heads": v_heads,
         "dk": dk, "dv": dv, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one stream, one token: the fp32 row of the fused qkv product, far into a long context
        _append("append_token", 1, 24, 2, 256, 64, "half", True, "f32", "bf16", 64, 100_003),
        # one token for each of 64 streams, whole head rotated, no norm
        _append("append_batch", 64, 48, 4, 128, 128, "interleaved", False, "bf16", "bf16", 64, 7_000),
        # a long prompt's chunk
        _append("append_prompt", 4_099, 24, 2, 256, 64, "half", True, "f32", "bf16", 64, 16_384),
        # one stream, one token, a short context: latency
        _attn("attn_token", 1, 1, 1_000, False, 24, 2, 256, 64, "bf16", "f32", 0),
        # a serving batch of single tokens with ragged contexts
        _attn("attn_batch", 32, 1, 8_192, True, 48, 4, 128, 64, "bf16", "bf16", 0),
        # one stream far into a long document
        _attn("attn_long", 1, 1, 131_075, False, 24, 2, 256, 64, "bf16", "f32", 0),
        # a prompt's chunk over what came before it
        _attn("attn_chunk", 1, 2_048, 8_100, False, 48, 4, 128, 64, "bf16", "bf16", 0),
        # several prompts of different lengths, sliding window
        _attn("attn_ragged", 6, 500, 3_001, True, 24, 2, 256, 16, "f16", "f32", 1_024),
        # one stream, one token
        _gdn("gdn_token", 1, 1, False, 16, 48, 128, 128, "f32"),
        # a serving batch of single tokens
        _gdn("gdn_batch", 64, 1, False, 16, 48, 128, 128, "bf16"),
        # a long prompt
        _gdn("gdn_prompt", 1, 4_096, False, 16, 48, 128, 128, "bf16"),
        # several prompts of different lengths
        _gdn("gdn_ragged", 5, 701, True, 16, 48, 128, 128, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attn", "attn", "gdn", "gdn"))
    if op == "append":
        dim = rng.choice((64, 128, 256))
        kv = rng.choice((1, 2, 4, 8))
        return _append(None, _log(rng, 1, 4_099), kv * rng.choice((1, 3, 6, 12)), kv, dim, rng.choice((dim, dim // 2, dim // 4)),
                       rng.choice(("half", "interleaved")), rng.random() < 0.5, rng.choice(("f32", "bf16", "f16")),
                       rng.choice(("bf16", "f16")), rng.choice((16, 64, 128)), _log(rng, 1, 1_000_000))
    if op == "attn":
        dim = rng.choice((64, 128, 256))
        kv = rng.choice((1, 2, 4))
        heads = kv * rng.choice((1, 4, 6, 12))
        if rng.random() < 0.5:  # single tokens
            seqs, new, keys = _log(rng, 1, 48), 1, _log(rng, 1, 16_000)
        else:
            seqs, new = _log(rng, 1, 8), _log(rng, 2, 512)
            keys = new + _log(rng, 1, 4_000)
        cache = rng.choice(("bf16", "f16"))
        return _attn(None, seqs, new, keys, rng.random() < 0.7, heads, kv, dim, rng.choice((16, 32, 64, 128)), cache,
                     rng.choice(("f32", cache)), rng.choice((0, 0, 0, _log(rng, 16, 2_000))))
    k_heads = rng.choice((2, 4, 8, 16))
    if rng.random() < 0.4:
        seqs, length = _log(rng, 1, 64), 1
    else:
        seqs, length = _log(rng, 1, 6), _log(rng, 2, 1_500)
    return _gdn(None, seqs, length, rng.random() < 0.7, k_heads, k_heads * rng.choice((1, 2, 3)), rng.choice((64, 128)),
                rng.choice((64, 128)), rng.choice(("f32", "bf16", "f16")))


def _lens(c):
    """Lengths of the sequences: (new tokens, keys in all) for attention, tokens for the delta rule."""
    n = c["seqs"]
    if c["op"] == "attn":
        if not c["ragged"]:
            return [c["new"]] * n, [c["keys"]] * n
        new = [max(1, c["new"] - (i * 7919) % max(1, c["new"])) for i in range(n)]
        return new, [max(a, c["keys"] - (i * 104_729) % max(1, (3 * c["keys"]) // 4)) for i, a in enumerate(new)]
    if not c["ragged"]:
        return [c["len"]] * n
    return [max(1, c["len"] - (i * 7919) % c["len"]) for i in range(n)]


def _lows(c, new, keys):
    """First key that any of a sequence's new tokens sees."""
    return [max(0, k - a - c["window"] + 1) if c["window"] else 0 for a, k in zip(new, keys)]


def work(case):
    c = case
    if c["op"] == "append":
        n = c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * (e + 2) + c["tokens"] * 12, "flops": n * 6}
    if c["op"] == "attn":
        new, keys = _lens(c)
        rows = sum(k - lo for k, lo in zip(keys, _lows(c, new, keys)))
        pairs = 0
        for a, k in zip(new, keys):
            w = c["window"] or k
            first = k - a + 1  # keys that the first new token could see
            full = max(0, min(a, k - max(first, w) + 1)) if k >= w else 0  # tokens that see a whole window
            rest = a - full
            pairs += full * w + rest * first + rest * (rest - 1) // 2
        n = sum(new) * c["heads"] * c["dim"]
        return {"bytes": rows * c["kv_heads"] * c["dim"] * 4 + n * (2 + (4 if c["out"] == "f32" else 2)),
                "flops": 4 * c["dim"] * c["heads"] * pairs}
    t = sum(_lens(c))
    e = 4 if c["dtype"] == "f32" else 2
    s = c["v_heads"] * c["dk"] * c["dv"]
    return {"bytes": t * (2 * c["k_heads"] * c["dk"] + 2 * c["v_heads"] * c["dv"]) * e + t * c["v_heads"] * 8 + 2 * c["seqs"] * s * 4,
            "flops": 7 * t * s}


# ---- inputs --------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev = torch.device("cuda")

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    c = case
    if c["op"] == "append":
        t, hq, hk, d, page = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = normal(t, (hq + 2 * hk) * d, dtype=DT[c["dtype"]])  # as a fused projection leaves it
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], 1))
        pages = -(-t // page) + 2
        order = torch.randperm(pages, generator=gen, device=dev)
        at = torch.arange(t, device=dev) + 3  # the first page has tokens already
        slots = order[at // page] * page + at % page
        freq = 10_000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        return {"case": c, "q": q, "k": k, "v": v, "positions": (at + c["start"]).to(torch.int32), "slots": slots, "freq": freq,
                "q_norm": normal(d, std=0.2) + 1 if c["norm"] else None, "k_norm": normal(d, std=0.2) + 1 if c["norm"] else None,
                "k_cache": normal(pages, hk, page, d, dtype=DT[c["cache"]]), "v_cache": normal(pages, hk, d, page, dtype=DT[c["cache"]]),
                "out": torch.empty(t, hq, d, dtype=DT[c["cache"]], device=dev)}
    if c["op"] == "attn":
        new, keys = _lens(c)
        hq, hk, d, page, dt = c["heads"], c["kv_heads"], c["dim"], c["page"], DT[c["cache"]]
        width = -(-max(keys) // page)
        used = [-(-k // page) for k in keys]
        pages = sum(used) + 1
        order = torch.randperm(pages, generator=gen, device=dev)
        first = ints([sum(used[:i]) for i in range(len(used))])
        col = torch.arange(width, device=dev)
        # a sequence's row of the table ends with entries that nothing reads
        at = torch.where(col[None] < ints(used)[:, None], first[:, None] + col[None], torch.zeros_like(first)[:, None])
        return {"case": c, "q": normal(sum(new), hq, d, dtype=dt), "k_cache": normal(pages, hk, page, d, dtype=dt),
                "v_cache": normal(pages, hk, d, page, dtype=dt), "table": order[at].to(torch.int32), "kv_len": ints(keys),
                "cu": ints([sum(new[:i]) for i in range(len(new) + 1)]), "new_max": max(new), "key_max": max(keys),
                "out": torch.empty(sum(new), hq, d, dtype=DT[c["out"]], device=dev)}
    n = _lens(c)
    t, b, hk, hv, dk, dv, dt = sum(n), len(n), c["k_heads"], c["v_heads"], c["dk"], c["dv"], DT[c["dtype"]]
    qkv = normal(t, 2 * hk * dk + hv * dv, dtype=dt)
    q, k, v = qkv.split([hk * dk, hk * dk, hv * dv], 1)
    return {"case": c, "q": q.unflatten(1, (-1, dk)), "k": k.unflatten(1, (-1, dk)), "v": v.unflatten(1, (-1, dv)),
            "g": -torch.exp(normal(t, hv, std=1.5) - 2.5), "beta": torch.sigmoid(normal(t, hv, std=1.5)),
            "state": normal(b, hv, dk, dv, std=0.3), "new_state": torch.empty(b, hv, dk, dv, device=dev),
            "cu": ints([sum(n[:i]) for i in range(b + 1)]), "max": max(n), "out": torch.empty(t, hv, dv, dtype=dt, device=dev)}


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(state):
    return {"append": _run_append, "attn": _run_attn, "gdn": _run_gdn}[state["case"]["op"]](state)


def _rotate(x, cos, sin, rot, layout):
    """Rotate the first `rot` values of each head: x [tokens, heads, dim], cos and sin [tokens, 1, rot / 2]."""
    y, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2 :]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = y[..., 0::2], y[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _run_append(s):
    c = s["case"]
    if own:
        import bit_quantized_matvec_amd as tq

        tq.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freq"], s["k_cache"], s["v_cache"],
                       q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, layout=c["layout"], out=s["out"])
        return s["out"], s["k_cache"], s["v_cache"]
    a = s["positions"].double()[:, None] * s["freq"]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    q, k = s["q"].float(), s["k"].float()
    if s["q_norm"] is not None:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_norm"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_norm"]
    q, k = _rotate(q, cos, sin, c["rot"], c["layout"]), _rotate(k, cos, sin, c["rot"], c["layout"])
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_cache"][page, :, at] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, :, :, at] = s["v"].to(s["v_cache"].dtype)
    return q.to(s["out"].dtype), s["k_cache"], s["v_cache"]


def _run_attn(s):
    c = s["case"]
    if own:
        import bit_quantized_matvec_amd as tq

        if "ws" not in s:  # kept by the program from its first pass on
            s["ws"] = tq.attn_workspace(s["q"].shape[0], c["seqs"], c["heads"], c["kv_heads"], c["dim"], device=s["q"].device)
        tq.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], s["cu"], max_len=s["new_max"],
                      window=c["window"], out=s["out"], ws=s["ws"])
        return s["out"]
    b, hk, d, n, m = c["seqs"], c["kv_heads"], c["dim"], s["new_max"], s["key_max"]
    group = c["heads"] // hk
    table = s["table"].long()
    k = s["k_cache"][table].transpose(1, 2).flatten(2, 3)[:, :, :m].float()  # [b, hk, m, d]
    v = s["v_cache"][table].permute(0, 2, 1, 4, 3).flatten(2, 3)[:, :, :m].float()
    cu, keys = s["cu"].long(), s["kv_len"].long()
    new = cu[1:] - cu[:-1]
    i, j = torch.arange(n, device=table.device), torch.arange(m, device=table.device)
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [b, hk, n * group, d]
    pos = (keys - new)[:, None, None] + i[None, :, None]
    seen = (j <= pos) & (j < keys[:, None, None])
    if c["window"]:
        seen &= j > pos - c["window"]
    v = v * (j < keys[:, None])[:, None, :, None]
    x = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (n, group)) * d**-0.5
    x = x.masked_fill(~seen[:, None, :, None], -torch.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul((p / p.sum(-1, keepdim=True)).flatten(2, 3), v)  # [b, hk, n * group, d]
    o = o.unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[i[None] < new[:, None]].to(s["out"].dtype)


def _run_gdn(s):
    c = s["case"]
    if own:
        import bit_quantized_matvec_amd as tq

        if "ws" not in s:
            s["ws"] = tq.gdn_workspace(s["q"].shape[0], c["seqs"], c["v_heads"], c["dk"], c["dv"], max_len=s["max"], device=s["q"].device)
        tq.gdn(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["cu"], max_len=s["max"], l2norm=True, eps=EPS,
               out=s["out"], state_out=s["new_state"], ws=s["ws"])
        return s["out"], s["new_state"]
    size = min(CHUNK, s["max"])
    count = -(-s["max"] // size)
    cu = s["cu"].long()
    i = torch.arange(count * size, device=cu.device)
    real = i < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)

    def lay(x):  # [tokens, heads, ...] -> [seqs, heads, chunks, size, ...]; what is past a sequence's end is zero
        y = x[rows] * real.view(*real.shape, *[1] * (x.dim() - 1))
        return y.transpose(1, 2).unflatten(2, (count, size))

    q, k, v = lay(s["q"].float()), lay(s["k"].float()), lay(s["v"].float())
    g, beta = lay(s["g"].double()), lay(s["beta"]).unsqueeze(-1)
    group = c["v_heads"] // c["k_heads"]
    q = (q * torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS) * c["dk"] ** -0.5).repeat_interleave(group, 1)
    k = (k * torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS)).repeat_interleave(group, 1)
    g = g.cumsum(-1)
    far = torch.exp(g).float().unsqueeze(-1)
    near = torch.exp((g.unsqueeze(-1) - g.unsqueeze(-2)).tril()).float().tril()
    last = torch.exp(g[..., -1:] - g).float().unsqueeze(-1)
    u, w = beta * v, beta * far * k
    if size > 1:
        a = (beta * torch.matmul(k, k.transpose(-1, -2)) * near).tril(-1)
        # (I + a)^-1: inverses of the diagonal blocks of 1, 2, 4, ... rows, each pair of them joined by what lies between
        at = torch.arange(size, device=cu.device)
        inv = torch.eye(size, device=cu.device).expand_as(a)
        for step in range((size - 1).bit_length()):
            row, col = at[:, None] >> step, at >> step
            between = a * ((row == col + 1) & (row % 2 == 1))
            inv = inv - torch.matmul(torch.matmul(inv, between), inv)
        u, w = torch.matmul(inv, u), torch.matmul(inv, w)
    inner = torch.matmul(q, k.transpose(-1, -2)) * near
    q, k = far * q, (last * k).transpose(-1, -2)
    state, o = s["state"], []
    for n in range(count):
        x = u[:, :, n] - torch.matmul(w[:, :, n], state)
        o.append(torch.matmul(q[:, :, n], state) + torch.matmul(inner[:, :, n], x))
        state = far[:, :, n, -1:] * state + torch.matmul(k[:, :, n], x)
    o = torch.cat(o, 2).transpose(1, 2)
    return o[real].to(s["out"].dtype), state


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "gdn": _exact_gdn}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    lo = list(range(half)) if c["layout"] == "half" else list(range(0, rot, 2))
    hi = [x + half for x in lo] if c["layout"] == "half" else [x + 1 for x in lo]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["positions"].double()[:, None, None] * s["freq"])  # rotations as complex numbers

    def one(x, w):
        y = x.double().clone()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / c["dim"] + EPS) * w.double()
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    k, v = s["k_cache"].double(), s["v_cache"].double()
    flat_k = k.transpose(1, 2).flatten(0, 1)  # [slots, heads, dim], a copy
    flat_v = v.permute(0, 3, 1, 2).flatten(0, 1)
    flat_k[s["slots"]] = one(s["k"], s["k_norm"])
    flat_v[s["slots"]] = s["v"].double()
    k = flat_k.unflatten(0, (-1, c["page"])).transpose(1, 2)
    v = flat_v.unflatten(0, (-1, c["page"])).permute(0, 2, 3, 1)
    return one(s["q"], s["q_norm"]), k, v


def _exact_attn(s):
    c = s["case"]
    new, keys = _lens(c)
    group, at, out = c["heads"] // c["kv_heads"], 0, []
    for b, (n, m) in enumerate(zip(new, keys)):
        pages = s["table"][b, : -(-m // c["page"])].long()
        k = s["k_cache"][pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :m]
        v = s["v_cache"][pages].double().permute(1, 0, 3, 2).flatten(1, 2)[:, :m]
        pos = torch.arange(m - n, m, device=k.device)[:, None]
        key = torch.arange(m, device=k.device)[None]
        hide = key > pos
        if c["window"]:
            hide |= key <= pos - c["window"]
        heads = []
        for h in range(c["heads"]):
            x = s["q"][at : at + n, h].double() @ k[h // group].T / math.sqrt(c["dim"])
            x[hide] = -math.inf
            heads.append(torch.softmax(x, -1) @ v[h // group])
        out.append(torch.stack(heads, 1))
        at += n
    return torch.cat(out)


def _exact_gdn(s):
    c = s["case"]
    group, at, outs, states = c["v_heads"] // c["k_heads"], 0, [], []
    for b, n in enumerate(_lens(c)):
        q, k, v = (s[x][at : at + n].double() for x in "qkv")
        q = (q / (q.square().sum(-1, keepdim=True) + EPS).sqrt() / math.sqrt(c["dk"])).repeat_interleave(group, 1)
        k = (k / (k.square().sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(group, 1)
        decay, beta = s["g"][at : at + n].double().exp(), s["beta"][at : at + n].double()
        m, rows = s["state"][b].double(), []
        for t in range(n):
            m = m * decay[t][:, None, None]
            d = beta[t][:, None] * (v[t] - (m * k[t][:, :, None]).sum(1))
            m = m + k[t][:, :, None] * d[:, None]
            rows.append((m * q[t][:, :, None]).sum(1))
        outs.append(torch.stack(rows))
        states.append(m)
        at += n
    return torch.cat(outs), torch.stack(states)
