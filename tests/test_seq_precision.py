"""How many bits the operators between a block's projections keep, on inputs whose errors are few and known: what the general
bounds of the other tests leave room for (a term of a split operand left out, 2^-17 of a value) does not fit here.

The limits are on the root of the mean square, over thousands of values, of the errors in units of 2^-24 of values of size one.
A value goes through some twenty roundings of at most one unit each, evenly spread (0.58 of it in the mean square), half of them
at half the size: 2 to 3 units.  Each term left out of a split costs more than twice the limit; the tests without the GPU plant
those in a plain emulation."""
import math

import pytest
import torch

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0**-24
ATTN_LIMIT, GDN_LIMIT = 6.0, 8.0


def units(got, want):
    """Root of the mean square, and largest, in units of 2^-24."""
    off = (got.double().cpu() - want) / U
    return float(off.square().mean().sqrt()), float(off.abs().max())


def terms(x, n, dtype=BF):
    """x (float32) as the sum of n terms of a 16-bit type."""
    total = torch.zeros_like(x)
    for _ in range(n):
        total = total + (x - total).to(dtype).float()
    return total


# ---- attention: two keys per token, scores that are exact -------------------------------------------------------------

def attn_case(tokens, hq, hk, dim, ct, seed=0, tiny=False):
    """Queries that are unit vectors, keys whose scores are numbers of the type, and a window of two: each output is a mean of
    two values with weights e^a and e^b.  `tiny`: V, and the K that scores come from, below fp16's normal range."""
    g = torch.Generator()
    g.manual_seed(seed + dim)
    page, keys = 16, tokens + 10
    pages = -(-keys // page)
    table = torch.randperm(pages, generator=g)
    q = torch.zeros(tokens, hq, dim, dtype=ct)
    q[..., 3] = 1
    kc = torch.randn(pages, hk, page, dim, generator=g).to(ct)
    vc = (1 + torch.rand(pages, hk, dim, page, generator=g)).to(ct)
    kc[..., 3] = (2 * torch.rand(pages, hk, page, generator=g) - 1).to(ct)
    if tiny:
        q, vc = q * 2**14, (torch.ceil(vc.float() * 128) * 2.0**-24).to(ct)
        kc[..., 3] = (torch.round(kc[..., 3].float() * 1024) * 2.0**-24).to(ct)
        assert float(vc.max()) < 2.0**-14 and float(kc[..., 3].abs().max()) <= 2.0**-14
    a = float(q[0, 0, 3]) * kc[table, ..., 3].double().transpose(1, 2).flatten(0, 1)[:keys]      # [keys, hk]
    v = vc[table].double().permute(0, 3, 1, 2).flatten(0, 1)[:keys]           # [keys, hk, dim]
    return q, kc, vc, table, keys, a, v


def attn_want(a, v, tokens, group, weight=torch.exp):
    x, y = a[-tokens - 1 : -1], a[-tokens:]
    top = torch.maximum(x, y)
    p, r = weight(x - top).unsqueeze(-1), weight(y - top).unsqueeze(-1)
    # (the sum of the weights is taken before they are split)
    e, f = torch.exp(x - top).unsqueeze(-1), torch.exp(y - top).unsqueeze(-1)
    return ((p * v[-tokens - 1 : -1] + r * v[-tokens:]) / (e + f)).repeat_interleave(group, 1)


@pytest.mark.parametrize("ct,left", [(BF, 2), (HF, 1)])
def test_attention_limit_sees_a_term_left_out(ct, left):
    _, _, _, _, _, a, v = attn_case(200, 8, 8, 64, ct)
    want = attn_want(a, v, 200, 1)
    cut = attn_want(a, v, 200, 1, lambda x: terms(torch.exp(x).float(), left, ct).double())
    kept = attn_want(a, v, 200, 1, lambda x: terms(torch.exp(x).float(), left + 1, ct).double())
    assert units(cut, want)[0] > 2 * ATTN_LIMIT and units(kept, want)[0] < ATTN_LIMIT / 2


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hk,rows", [(150, 32, 32, 128), (120, 1, 1, 16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ct,tiny", [(BF, False), (HF, False), (HF, True)])
def test_attention_keeps_the_weights_bits(tokens, hq, hk, rows, dim, ct, tiny):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_matvec_amd as tq

    assert tq.lib().tq_paged_attn_tile_rows(tokens, 1, tokens, hq, hk, dim) == rows
    q, kc, vc, table, keys, a, v = attn_case(tokens, hq, hk, dim, ct, tiny=tiny)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.int()[None].cuda(), ints([keys]), ints([0, tokens]), scale=1.0, window=2, max_len=tokens,
                        out_dtype=F32, ws=tq.attn_workspace(tokens, 1, hq, hk, dim))
    want = attn_want(a, v, tokens, hq // hk)
    rms, worst = units(got / want.cuda(), torch.ones_like(want))
    print(f"rms {rms:.2f}, worst {worst:.1f}")
    assert rms < ATTN_LIMIT and worst < 8 * ATTN_LIMIT


# ---- delta rule: keys along the axes, two tokens of a chunk to each ----------------------------------------------------

def gdn_case(n, kh, vh, dk, dv, it, seed=0):
    """Token t's key and query lie along axis (t / 2) mod dk, gates are one: a row of the state meets two tokens of a chunk and
    no other row."""
    g = torch.Generator()
    g.manual_seed(seed + dk + n)

    def some(*shape, low=0.5):  # magnitudes between low and one, either sign
        return (low + (1 - low) * torch.rand(*shape, generator=g)) * (1 - 2 * torch.randint(0, 2, shape, generator=g))

    axis = torch.arange(n) // 2 % dk
    q, k = torch.zeros(n, kh, dk), torch.zeros(n, kh, dk)
    for h in range(kh):
        q[torch.arange(n), h, axis], k[torch.arange(n), h, axis] = some(n, low=0.75), some(n, low=0.75)
    v, beta = some(n, vh, dv), some(n, vh, low=0.75).abs()
    return q.to(it), k.to(it), v.to(it), torch.zeros(n, vh), beta, some(1, vh, dk, dv), axis


def gdn_want(q, k, v, beta, state, axis, chunk=64, **left):
    """Outputs and states, row by row and chunk by chunk.  `left`: the terms that an operand is cut to, computed in float32;
    without it, float64."""
    f = F32 if left else torch.float64
    cut = lambda x, name: terms(x, left[name]) if name in left and left[name] else x  # noqa: E731
    n, vh, dv = v.shape
    group = vh // k.shape[1]
    alpha = q.to(f)[torch.arange(n), :, axis].repeat_interleave(group, 1)[..., None]   # [n, vh, 1]
    kappa = k.to(f)[torch.arange(n), :, axis].repeat_interleave(group, 1)[..., None]
    v, b, s, out = v.to(f), beta.to(f)[..., None], state[0].to(f).clone(), torch.zeros(n, vh, dv, dtype=f)
    qc, kc = cut(alpha, "Q"), cut(kappa, "K")
    for t in range(0, n, 2):
        assert t % chunk % 2 == 0
        pair, row = range(t, min(t + 2, n)), s[:, axis[t]]
        low = cut(row, "S")
        r = [b[i] * v[i] - b[i] * (kc[i] * low) for i in pair]
        x = [cut(r[0], "R")]
        if len(r) == 2:
            x.append(cut(r[1], "R") - cut(b[t + 1] * (kc[t] * kc[t + 1]), "T") * x[0])
        for i in pair:
            out[i] = qc[i] * low
            for j in range(t, i + 1):
                out[i] += cut(qc[i] * kc[j], "P") * cut(x[j - t], "X")
        for i in pair:
            row = row + kc[i] * cut(x[i - t], "Z")
        s[:, axis[t]] = row
    return out, s


def test_gdn_emulation_is_the_recurrence():
    import seq_oracle as so

    q, k, v, g, beta, state, axis = gdn_case(200, 1, 2, 64, 32, F32)
    want, states, _ = so.gdn(q, k, v, g, beta, state, [0, 200], 1.0, False, 0.0)
    out, after = gdn_want(q, k, v, beta, state, axis)
    assert float((out - want).abs().max()) < 1e-12 and float((after - states[0]).abs().max()) < 1e-12


@pytest.mark.parametrize("name", ["none", "S", "R", "T", "X", "P", "Z", "Q", "K"])
def test_gdn_limit_sees_a_term_left_out(name):
    q, k, v, _, beta, state, axis = gdn_case(300, 1, 2, 64, 32, F32)
    out, after = gdn_want(q, k, v, beta, state, axis)
    got, states = gdn_want(q, k, v, beta, state, axis, **{name: 2})
    worst = max(units(got, out)[0], units(states, after)[0])
    print(f"{name}: {worst:.2f}")
    assert worst < GDN_LIMIT / 2 if name == "none" else worst > 1.5 * GDN_LIMIT


@pytest.mark.gpu
@pytest.mark.parametrize("n,kh,vh,dk,dv", [(300, 1, 2, 64, 32), (700, 2, 2, 128, 64), (64, 1, 1, 128, 128), (2100, 16, 48, 64, 32)])
@pytest.mark.parametrize("it", [F32, BF, HF])
@pytest.mark.parametrize("chunks", [True, False])
def test_gdn_keeps_fp32s_bits(n, kh, vh, dk, dv, it, chunks):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_matvec_amd as tq

    q, k, v, g, beta, state, axis = gdn_case(n, kh, vh, dk, dv, it)
    out, after = gdn_want(q, k, v, beta, state, axis)
    c = lambda x: x.cuda()  # noqa: E731
    gs = state.cuda()
    got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale=1.0, max_len=n, out_dtype=F32,
                 ws=tq.gdn_workspace(n, 1, vh, dk, dv, max_len=n) if chunks else None)
    for have, want, what in ((got, out, "out"), (gs[0], after, "state")):
        rms, worst = units(have, want)
        print(f"{what}: rms {rms:.2f}, worst {worst:.1f}")
        assert rms < GDN_LIMIT and worst < 16 * GDN_LIMIT, what
