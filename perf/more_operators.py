"""Measured cases of what differs from row to row in a batch that shares its weights: each token's experts (the routing and the
ternary products), each request's low-rank adapter beside a shared projection, each request's sampling.

`listed()` and `draw()` give cases as plain dicts; `prepare()` makes a case's inputs from a seed; `run()` does one
pass, in plain torch where `own` is false and through the package where it is true; `exact()` evaluates the
definition in 64 bits, expert by expert, adapter by adapter and row by row; `work()` counts the bytes and operations that a
pass cannot do without.

Widths follow the matrices of this repository's decode step (5120, 6144, 7168 and 17408).
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases ---------------------------------------------------------------------------------------------------------

def _route(name, tokens, experts, k, score, bias, groups, top_groups, dtype):
    c = {"op": "route", "tokens": tokens, "experts": experts, "k": k, "score": score, "bias": bias, "groups": groups,
         "top_groups": top_groups, "dtype": dtype}
    return dict(c, name=name) if name else c


def _experts(name, tokens, experts, k, rows, cols, share):
    c = {"op": "experts", "tokens": tokens, "experts": experts, "k": k, "rows": rows, "cols": cols, "share": share}
    return dict(c, name=name) if name else c


def _adapt(name, tokens, adapters, rank, cols, rows, runs, x, w, y):
    c = {"op": "adapt", "tokens": tokens, "adapters": adapters, "rank": rank, "cols": cols, "rows": rows, "runs": runs,
         "x": x, "w": w, "y": y}
    return dict(c, name=name) if name else c


def _sample(name, rows, vocab, dtype, filters):
    c = {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "filters": filters}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one stream's token: softmax over 64 experts
        _route("route_token", 1, 64, 8, "softmax", False, 1, 1, "f32"),
        # a prompt's chunk: sigmoid scores, a bias for balance, 4 of 8 groups
        _route("route_prompt", 4_099, 256, 8, "sigmoid", True, 8, 4, "bf16"),
        # one stream's token: gate and up of its 8 experts
        _experts("experts_token", 1, 64, 8, 2_048, 5_120, True),
        # a serving batch of single tokens: down of every token's experts, each with activations of its own
        _experts("experts_batch", 48, 64, 8, 5_120, 1_024, False),
        # a prompt's chunk
        _experts("experts_prompt", 2_048, 32, 4, 2_048, 5_120, True),
        # one stream's token beside the fused qkv product
        _adapt("adapt_token", 1, 4, 16, 5_120, 7_168, False, "f32", "bf16", "f32"),
        # a serving batch of single tokens beside the gate product, ranks of 8 to 32
        _adapt("adapt_batch", 64, 24, 32, 5_120, 17_408, False, "f32", "bf16", "f32"),
        # several prompts' chunks, an adapter each
        _adapt("adapt_prompt", 4_099, 5, 64, 5_120, 7_168, True, "bf16", "bf16", "f32"),
        # a shorter one into an odd width, all in 16 bits
        _adapt("adapt_ragged", 701, 3, 16, 6_144, 5_003, True, "f16", "f16", "f16"),
        # one stream's next token
        _sample("sample_token", 1, 131_072, "f32", "kpm"),
        # a serving batch whose requests set what they like, greedy ones among them
        _sample("sample_batch", 64, 131_072, "f32", "mixed"),
        # a large batch over a large odd vocabulary, top-p alone
        _sample("sample_large", 256, 200_003, "bf16", "p"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "adapt", "adapt", "sample", "sample"))
    if op == "route":
        experts = rng.choice((8, 16, 60, 64, 96, 128, 160, 256))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0 and experts // g >= 2])
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, top * (experts // groups)))
        return _route(None, _log(rng, 1, 4_099), experts, k, rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, groups, top,
                      rng.choice(("f32", "bf16", "f16")))
    if op == "experts":
        experts = rng.choice((4, 8, 16, 31, 64))
        share = rng.random() < 0.5
        rows, cols = rng.choice((_log(rng, 64, 2_048), rng.choice((512, 1_024, 2_048)))), 256 * _log(rng, 1, 20)
        return _experts(None, _log(rng, 1, 1_024), experts, rng.randint(1, min(8, experts)), rows, cols, share)
    if op == "adapt":
        x = rng.choice(("f32", "f32", "bf16", "f16"))
        w = rng.choice(("bf16", "f16")) if x == "f32" else x
        tokens = _log(rng, 1, 96) if rng.random() < 0.5 else _log(rng, 97, 4_099)
        rows, cols = rng.choice((_log(rng, 64, 7_168), rng.choice((1_024, 5_120, 7_168)))), 8 * _log(rng, 32, 896)
        return _adapt(None, tokens, _log(rng, 1, 24), 8 * rng.randint(1, 8), cols, rows, tokens > 96, x, w, rng.choice(("f32", x)))
    vocab = rng.choice((_log(rng, 1_000, 200_003), 32_768, 131_072))
    return _sample(None, min(_log(rng, 1, 256), 25_000_000 // vocab), vocab, rng.choice(("f32", "bf16", "f16")),
                   rng.choice(("kpm", "mixed", "p", "k", "m", "none")))


def _ranks(c):
    """The smallest and the largest rank of a case's adapters."""
    return 8 * max(1, c["rank"] // 32), 8 * max(1, c["rank"] // 8)


def work(case):
    c = case
    if c["op"] == "route":
        n = c["tokens"] * c["experts"]
        return {"bytes": n * BYTES[c["dtype"]] + c["tokens"] * c["k"] * 12 + 4 * (c["experts"] + 1) + 4 * c["experts"] * c["bias"], "flops": 4 * n}
    if c["op"] == "experts":
        pairs = c["tokens"] * c["k"]
        touched = c["experts"] * (1 - (1 - c["k"] / c["experts"]) ** c["tokens"])  # expected, of even choices
        ins = c["tokens"] if c["share"] else pairs
        return {"bytes": int(touched * c["rows"] * c["cols"] * 34 / 128) + ins * (c["cols"] + c["cols"] // 64) + pairs * (8 + 4 * c["rows"]),
                "flops": 2 * pairs * c["rows"] * c["cols"]}
    if c["op"] == "adapt":
        t, n, r = c["tokens"], c["adapters"], sum(_ranks(c)) / 2  # expected, of even choices
        touched = n * (1 - (1 - 1 / n) ** t)
        return {"bytes": int(t * c["cols"] * BYTES[c["x"]] + 2 * t * c["rows"] * BYTES[c["y"]] + touched * r * (c["cols"] + c["rows"]) * 2 + 4 * t),
                "flops": int(2 * t * r * (c["cols"] + c["rows"]))}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * BYTES[c["dtype"]] + c["rows"] * 28, "flops": 10 * n}


# ---- inputs --------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev = torch.device("cuda")
    c = case

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    def ints(hi, *shape, lo=0):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    if c["op"] == "route":
        bias = uniform(c["experts"], lo=-0.05, hi=0.05) if c["bias"] else None
        return {"case": c, "logits": normal(c["tokens"], c["experts"], std=1.5).to(DT[c["dtype"]]), "bias": bias}
    if c["op"] == "experts":
        n, t, k, rows, cols = c["experts"], c["tokens"], c["k"], c["rows"], c["cols"]
        codes = torch.zeros(n, rows, cols // 128, 32, dtype=torch.uint8, device=dev)
        for s in range(4):  # codes 0, 1, 2 in each 2-bit field
            codes |= torch.randint(0, 3, codes.shape, generator=gen, device=dev, dtype=torch.uint8) << (2 * s)
        scale = uniform(n, rows, cols // 128, 1, lo=0.01, hi=0.05).half().view(torch.uint8)
        weights = torch.cat([scale, codes], -1).flatten(1)  # [experts, canonical bytes]
        ids = (normal(t, n) + normal(n, std=0.5)).topk(k, 1).indices.to(torch.int32)  # some experts are liked better
        x = normal(t if c["share"] else t * k, cols // 256, 256)
        d = x.abs().amax(-1) / 127
        q = torch.round(x / d[..., None]).to(torch.int8).flatten(1)
        flat = ids.flatten().long()
        order = torch.sort(flat, stable=True).indices.to(torch.int32)
        count = torch.bincount(flat, minlength=n)
        offsets = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
        return {"case": c, "weights": weights, "ids": ids, "order": order, "offsets": offsets, "most": int(count.max()), "q": q, "d": d,
                "out": torch.empty(t * k, rows, device=dev)}
    if c["op"] == "adapt":
        n, t, r = c["adapters"], c["tokens"], c["rank"]
        if c["runs"]:  # each request's tokens lie together
            index = torch.sort(ints(n, t)).values
        else:  # single tokens of many requests; some have no adapter
            index = ints(n, t, lo=-1) if t > 1 else ints(n, t)
        return {"case": c, "index": index, "x": normal(t, c["cols"], dtype=DT[c["x"]]), "y": normal(t, c["rows"], std=3.0, dtype=DT[c["y"]]),
                "a": normal(n, r, c["cols"], std=c["cols"] ** -0.5, dtype=DT[c["w"]]), "b": normal(n, c["rows"], r, std=r**-0.5, dtype=DT[c["w"]]),
                "ranks": ints(_ranks(c)[1] // 8 + 1, n, lo=_ranks(c)[0] // 8) * 8, "scale": uniform(n, lo=0.5, hi=2.0),
                "out": torch.empty(t, c["rows"], dtype=DT[c["y"]], device=dev)}
    rows, vocab, f = c["rows"], c["vocab"], c["filters"]
    logits = normal(rows, vocab, std=2.0)
    liked = torch.randint(0, vocab, (rows, 24), generator=gen, device=dev)
    logits.scatter_add_(1, liked, uniform(rows, 24, hi=12.0))
    pick = lambda values: torch.tensor(values, device=dev)[torch.randint(0, len(values), (rows,), generator=gen, device=dev)]  # noqa: E731
    s = {"case": c, "logits": logits.to(DT[c["dtype"]]), "u": torch.rand(rows, generator=gen, device=dev), "temperature": uniform(rows, lo=0.6, hi=1.3),
         "top_k": None, "top_p": None, "min_p": None, "out": torch.empty(rows, dtype=torch.int32, device=dev), "logprob": torch.empty(rows, device=dev)}
    if f == "mixed":
        s["temperature"] = s["temperature"] * pick([0.0, 1.0, 1.0, 1.0, 1.0])  # zero: greedy
        s["top_k"] = pick([0, 0, 20, 50, 400]).to(torch.int32)
        s["top_p"], s["min_p"] = pick([1.0, 0.95, 0.9, 0.7]), pick([0.0, 0.0, 0.02, 0.1])
    if f in ("k", "kpm"):
        s["top_k"] = ints(100, rows, lo=20)
    if f in ("p", "kpm"):
        s["top_p"] = uniform(rows, lo=0.7, hi=0.99)
    if f in ("m", "kpm"):
        s["min_p"] = uniform(rows, lo=0.01, hi=0.1)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(state):
    return {"route": _run_route, "experts": _run_experts, "adapt": _run_adapt, "sample": _run_sample}[state["case"]["op"]](state)


def _run_route(s):
    c = s["case"]
    if own:
        import bit_quantized_matvec_amd as tq

        if "out" not in s:  # kept by the program from its first pass on
            t, k, dev = c["tokens"], c["k"], s["logits"].device
            s["out"] = (torch.empty(t, k, device=dev), torch.empty(t, k, dtype=torch.int32, device=dev))
            s["lists"] = (torch.empty(t * k, dtype=torch.int32, device=dev), torch.empty(c["experts"] + 1, dtype=torch.int32, device=dev))
        weights, experts = tq.route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                                    group_best=2 if c["bias"] else 1, renorm=True, scale=2.5, out=s["out"])
        order, offsets = tq.expert_lists(experts, c["experts"], out=s["lists"])
        return weights, experts, order, offsets
    x = s["logits"].double()  # scores that are nearly equal decide
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.exp(x - x.amax(-1, keepdim=True))
    if c["score"] == "softmax":
        p = p / p.sum(-1, keepdim=True)
    choice = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        best = choice.unflatten(1, (c["groups"], -1)).sort(-1, descending=True).values[..., : 2 if c["bias"] else 1].sum(-1)
        rank = torch.sort(best, dim=-1, descending=True, stable=True).indices.argsort(-1)
        choice = choice.masked_fill((rank >= c["top_groups"]).repeat_interleave(c["experts"] // c["groups"], 1), -torch.inf)
    experts = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    weights = p.gather(1, experts)
    weights = (weights / weights.sum(-1, keepdim=True) * 2.5).float()
    flat = experts.flatten()
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    ids = torch.arange(c["experts"], device=flat.device)
    offsets = torch.cat([flat.new_zeros(1), (flat == ids[:, None]).sum(1).cumsum(0)]).to(torch.int32)
    return weights, experts.to(torch.int32), order, offsets


def _run_experts(s):
    c = s["case"]
    n, rows, cols, pairs = c["experts"], c["rows"], c["cols"], c["tokens"] * c["k"]
    if own:
        import bit_quantized_matvec_amd as tq

        if "w" not in s:  # laid out when the program loads them
            s["w"] = torch.stack([tq.repack(w, "pq2_0", rows, cols) for w in s["weights"]])
        return tq.gemm_experts("pq2_0", s["w"], rows, cols, s["q"], s["d"], s["order"], s["offsets"], out=s["out"])
    if "w" not in s:  # decoded when the program loads them
        blocks = s["weights"].view(n, rows, cols // 128, 34)
        codes = blocks[..., 2:, None] >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=blocks.device) & 3
        s["w"] = ((codes.flatten(-2).float() - 1) * blocks[..., :2].contiguous().view(torch.float16).float()).flatten(-2)
    x = (s["q"].view(-1, cols // 256, 256).float() * s["d"][..., None]).flatten(1)
    if c["share"]:
        x = x.repeat_interleave(c["k"], 0)
    ids = s["ids"].flatten().long()
    if pairs <= n:  # few: a copy of each pair's own matrix
        return torch.matmul(s["w"][ids], x[:, :, None])[..., 0]
    order, offsets = s["order"].long(), s["offsets"].long()
    sorted_ids = ids[order]
    at = torch.arange(pairs, device=x.device) - offsets[sorted_ids]
    padded = x.new_zeros(n, s["most"], cols)
    padded[sorted_ids, at] = x[order]
    y = torch.matmul(padded, s["w"].transpose(1, 2))
    out = torch.empty_like(s["out"])
    out[order] = y[sorted_ids, at]
    return out


def _run_adapt(s):
    c = s["case"]
    if own:
        import bit_quantized_matvec_amd as tq

        if "ws" not in s:
            s["ws"] = tq.adapter_workspace(c["tokens"], c["adapters"], c["rank"], c["cols"], device=s["x"].device)
        return tq.adapter_add(s["y"], s["x"], s["a"], s["b"], s["index"], ranks=s["ranks"], scale=s["scale"], out=s["out"], ws=s["ws"])
    n, r = c["adapters"], c["rank"]
    x, a, b, index = s["x"].float(), s["a"].float(), s["b"].float(), s["index"].long()
    used = (torch.arange(r, device=x.device) < s["ranks"][:, None]) * s["scale"][:, None]  # [adapters, rank]
    if c["tokens"] < n:  # few: each token's own matrices
        some = (index >= 0)[:, None] * used[index.clamp(min=0)]
        at = index.clamp(min=0)
        h = torch.matmul(a[at], x[:, :, None]) * some[:, :, None]
        add = torch.matmul(b[at], h)[..., 0]
    else:  # every token with every adapter, and all but its own masked
        h = torch.matmul(x, a.flatten(0, 1).t()).unflatten(1, (n, r))
        h = h * (index[:, None] == torch.arange(n, device=x.device))[:, :, None] * used
        add = torch.matmul(h.flatten(1), b.transpose(1, 2).flatten(0, 1))
    return (s["y"].float() + add).to(s["out"].dtype)


def _run_sample(s):
    c = s["case"]
    if own:
        import bit_quantized_matvec_amd as tq

        if "ws" not in s:
            s["ws"] = tq.sample_workspace(c["rows"], c["vocab"], device=s["logits"].device)
        tq.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], out=s["out"],
                  logprob=s["logprob"], ws=s["ws"])
        return s["out"], s["logprob"]
    x = s["logits"].double()  # sums over the vocabulary, and values next to a border
    t = s["temperature"].double()[:, None]
    m, best = x.amax(-1, keepdim=True), x.argmax(-1)
    e = torch.exp((x - m) / torch.where(t > 0, t, torch.ones_like(t)))
    total = e.sum(-1)
    y, order = torch.sort(x, dim=-1, descending=True, stable=True)  # equal ones: the lowest index first
    se = e.gather(1, order)
    rank = torch.arange(c["vocab"], device=x.device)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        se = se * ((rank < k) | (k == 0))
    keep = se > 0
    if s["top_p"] is not None:
        before = se.cumsum(-1)
        p = s["top_p"].double()[:, None]
        keep &= (before - se < p * before[:, -1:]) | (p >= 1)
    if s["min_p"] is not None:
        keep &= se >= s["min_p"].double()[:, None]
    w = torch.zeros_like(e).scatter(1, order, se * keep).cumsum(-1)
    token = (w > s["u"].double()[:, None] * w[:, -1:]).to(torch.int8).argmax(-1)
    token = torch.where(t[:, 0] > 0, token, best)
    logprob = torch.log(e.gather(1, token[:, None])[:, 0] / total)
    return token.to(torch.int32), logprob.float()


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "adapt": _exact_adapt, "sample": _exact_sample}[case["op"]](s)


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu()
    p = torch.softmax(x, -1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-x))
    bias = torch.zeros(c["experts"], dtype=torch.float64) if s["bias"] is None else s["bias"].double().cpu()
    size, weights, experts = c["experts"] // c["groups"], [], []
    for row in p.tolist():
        choice = [a + b for a, b in zip(row, bias.tolist())]
        best = [sum(sorted(choice[g * size : (g + 1) * size])[-2 if c["bias"] else -1 :]) for g in range(c["groups"])]
        kept = sorted(range(c["groups"]), key=lambda g: (-best[g], g))[: c["top_groups"]]
        among = [e for g in sorted(kept) for e in range(g * size, (g + 1) * size)]
        chosen = sorted(among, key=lambda e: (-choice[e], e))[: c["k"]]
        total = sum(row[e] for e in chosen)
        weights.append([2.5 * row[e] / total for e in chosen])
        experts.append(chosen)
    flat = [e for row in experts for e in row]
    order = sorted(range(len(flat)), key=lambda i: flat[i])
    count = [0] * (c["experts"] + 1)
    for e in flat:
        count[e + 1] += 1
    offsets = torch.tensor(count).cumsum(0)
    return torch.tensor(weights, dtype=torch.float64), torch.tensor(experts), torch.tensor(order), offsets


def _exact_experts(s):
    c = s["case"]
    dev, g = s["q"].device, c["cols"] // 128
    fields = torch.tensor([[(b >> 2 * i & 3) - 1 for i in range(4)] for b in range(256)], dtype=torch.float64, device=dev)
    x = s["q"].double() * s["d"].double().repeat_interleave(256, 1)
    out = torch.zeros(c["tokens"] * c["k"], c["rows"], dtype=torch.float64, device=dev)
    ids = s["ids"].flatten()
    for e in range(c["experts"]):
        pairs = (ids == e).nonzero()[:, 0]
        if not len(pairs):
            continue
        blocks = s["weights"][e].view(c["rows"] * g, 34)
        w = fields[blocks[:, 2:].long()].flatten(1) * blocks[:, :2].contiguous().view(torch.float16).double()
        out[pairs] = x[pairs // c["k"] if c["share"] else pairs] @ w.view(c["rows"], c["cols"]).T
    return out


def _exact_adapt(s):
    c = s["case"]
    out = s["y"].double().clone()
    for i, (rank, scale) in enumerate(zip(s["ranks"].tolist(), s["scale"].tolist())):
        t = (s["index"] == i).nonzero()[:, 0]
        out[t] += scale * (s["x"][t].double() @ s["a"][i, :rank].double().T @ s["b"][i, :, :rank].double().T)
    return out


def _exact_sample(s):
    c = s["case"]
    tokens, logprobs = [], []
    at = lambda name, i, off: off if s[name] is None else float(s[name][i])  # noqa: E731
    for i in range(c["rows"]):
        x = s["logits"][i].double()
        t = float(s["temperature"][i])
        logp = torch.log_softmax(x / t if t > 0 else x, -1)
        if t > 0:
            order = torch.sort(-x, stable=True).indices
            k, p, low = int(at("top_k", i, 0)), at("top_p", i, 1.0), at("min_p", i, 0.0)
            order = order[: k or c["vocab"]]
            w = torch.exp(logp[order] - logp.max())
            if p < 1:
                n = int((w.cumsum(0) < p * w.sum()).sum()) + 1
                order, w = order[:n], w[:n]
            order = torch.sort(order[w >= low]).values
            w = torch.exp(logp[order] - logp.max()).cumsum(0)
            token = int(order[min(int((w <= float(s["u"][i]) * w[-1]).sum()), len(order) - 1)])
        else:
            token = int((x == x.max()).nonzero()[0, 0])
        tokens.append(token)
        logprobs.append(float(logp[token]))
    return torch.tensor(tokens), torch.tensor(logprobs, dtype=torch.float64)
