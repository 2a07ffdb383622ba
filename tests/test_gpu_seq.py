"""GPU parity of the operators between a block's projections with their 64-bit definitions (seq_oracle.py)."""
import math

import pytest
import torch

import seq_oracle as so

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_matvec_amd as m

    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def near(got, want, bound, what):
    got = got.double().cpu()
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {float((off / bound)[bad].max()):.3g} times it"


# ---- rope_append ---------------------------------------------------------------------------------------------------

ROPE = [
    # tokens, heads, kv_heads, dim, rot, layout, page, in, cache, norm, start, order
    (1, 24, 2, 256, 64, "half", 64, F32, BF, True, 100_003, "run"),
    (1, 1, 1, 64, 0, "half", 16, BF, BF, False, 0, "run"),
    (2, 3, 1, 64, 16, "interleaved", 16, HF, HF, True, 5, "run"),
    (7, 48, 4, 128, 128, "half", 32, BF, HF, False, 1_048_000, "run"),
    (130, 6, 2, 128, 96, "half", 64, F32, HF, True, 3, "run"),
    (130, 6, 2, 256, 256, "interleaved", 64, BF, BF, True, 40, "shuffled"),
    (257, 4, 4, 64, 32, "interleaved", 256, F32, BF, False, 0, "run"),
    (300, 12, 1, 256, 48, "half", 128, HF, BF, True, 9, "holes"),
    (2100, 2, 1, 64, 64, "half", 16, BF, BF, False, 77, "run"),
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("fused", [True, False])
def test_rope_append(tq, case, fused):
    tokens, hq, hk, d, rot, layout, page, it, ct, norm, start, order = case
    r = gen(tokens + d)
    if fused:
        qkv = torch.randn(tokens, (hq + 2 * hk) * d, generator=r).to(it)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], 1))
        dq, dk, dv = (x.unflatten(1, (-1, d)) for x in qkv.cuda().split([hq * d, hk * d, hk * d], 1))
    else:  # heads outside tokens
        q, k, v = (torch.randn(n, tokens, d, generator=r).to(it).transpose(0, 1) for n in (hq, hk, hk))
        dq, dk, dv = (x.transpose(0, 1).cuda().transpose(0, 1) for x in (q, k, v))
    pages = -(-(tokens + 5) // page) + 1
    table = torch.randperm(pages, generator=r)
    at = torch.arange(tokens) + 5
    slots = table[at // page] * page + at % page
    if order == "shuffled":
        slots = slots[torch.randperm(tokens, generator=r)]
    if order == "holes":
        slots[torch.rand(tokens, generator=r) < 0.2] = -1
    positions = (torch.arange(tokens) + start).int()
    freq, rope_scale = tq.rope_frequencies(rot, 1e6, scaling="yarn", factor=4, original=32768) if rot else (None, 1.0)
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=r)) if norm else (None, None)
    kc, vc = torch.randn(pages, hk, page, d, generator=r).to(ct), torch.randn(pages, hk, d, page, generator=r).to(ct)
    gk, gv = kc.cuda(), vc.cuda()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda = lambda x: None if x is None else x.cuda()  # noqa: E731
    got = tq.rope_append(dq, dk, dv, positions.cuda() if rot else None, slots.cuda(), cuda(freq), gk, gv, q_norm=cuda(wq), k_norm=cuda(wk),
                         layout=layout, rope_scale=rope_scale, bad_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0 and got.dtype == ct and got.is_contiguous()
    # fp32: a norm over d values, two products and a sum, an angle of at most half a turn rounded to fp32
    u = so.U32 * (d / 8 + 24 + math.pi * 4)

    def bound(want, size):
        return so.HALF_STEP[ct] * want.abs() + u * size + (2.0**-25 if ct == HF else 0)  # fp16 steps below its normal range

    want, size = so.rope_rows(q, positions, freq, layout, rope_scale, wq, 1e-6)
    near(got, want, bound(want, size), "q")
    want, size = so.rope_rows(k, positions, freq, layout, rope_scale, wk, 1e-6)
    live = slots >= 0
    page_of, place = slots[live] // page, slots[live] % page
    near(gk.cpu()[page_of, :, place], want[live], bound(want, size)[live], "k")
    assert torch.equal(gv.cpu()[page_of, :, :, place], v.to(ct)[live])
    # nothing else was touched
    kc[page_of, :, place] = gk.cpu()[page_of, :, place]
    vc[page_of, :, :, place] = gv.cpu()[page_of, :, :, place]
    assert torch.equal(kc, gk.cpu()) and torch.equal(vc, gv.cpu())


def test_rope_append_slots_out_of_range(tq):
    tokens, d, page, pages = 20, 64, 16, 2
    r = gen(1)
    q, k, v = (torch.randn(tokens, n, d, generator=r).cuda() for n in (2, 1, 1))
    kc, vc = tq.kv_cache(pages, 1, page, d)
    slots = torch.arange(tokens) + 16  # 16 .. 35: the last four are past the cache
    slots[0] = 2**40
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tq.rope_append(q, k, v, None, slots.cuda(), None, kc, vc, bad_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 1
    assert torch.equal(out, q.bfloat16())
    assert torch.equal(kc[1, 0, 1:16], k[1:16, 0].bfloat16()) and torch.equal(vc[1, 0, :, 1:16].t(), v[1:16, 0].bfloat16())
    assert not bool(kc[0].any()) and not bool(kc[1, :, 0].any()) and not bool(vc[0].any()) and not bool(vc[1, :, :, 0].any())


# ---- paged_attn ----------------------------------------------------------------------------------------------------

def attn_inputs(new, keys, hq, hk, d, page, ct, seed=0, spare=2):
    r = gen(seed + sum(keys) + d)
    used = [-(-k // page) for k in keys]
    width = max(used + [1]) + 1
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=r)
    table = torch.full((len(keys), width), -7, dtype=torch.int32)  # what nothing may read
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at : at + u].int()
        at += u
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    q = torch.randn(cu[-1], hq, d, generator=r).to(ct)
    kc, vc = torch.randn(pages, hk, page, d, generator=r).to(ct), torch.randn(pages, hk, d, page, generator=r).to(ct)
    return q, kc, vc, table, cu


def attn_check(tq, new, keys, hq, hk, d, page, ct, ot, window=0, scale=None, ws=True, lse=True, poison=True, strided=False, cu_given=True, seed=0):
    q, kc, vc, table, cu = attn_inputs(new, keys, hq, hk, d, page, ct, seed)
    if poison:  # NaN and infinities in every place that no token sees
        seen = torch.zeros(kc.shape[0], page, dtype=torch.bool)
        for b, k in enumerate(keys):
            lo = max(0, k - new[b] - window + 1) if window else 0
            for j in range(lo, k):
                seen[table[b, j // page], j % page] = True
        kc[~seen.unsqueeze(1).expand(-1, hk, -1)] = math.nan
        vc.transpose(2, 3)[~seen.unsqueeze(1).expand(-1, hk, -1)] = math.inf
        if window:  # pages before every window may be gone
            for b, k in enumerate(keys):
                table[b, : max(0, k - new[b] - window + 1) // page] = -1
    scale = d**-0.5 if scale is None else scale
    gq = q.cuda()
    if strided:
        wide = torch.zeros(q.shape[0], hq + 1, 2 * d, dtype=ct, device="cuda")
        wide[:, :hq, :d] = gq
        gq = wide[:, :hq, :d]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    flag, w = ints([0]), None
    gl = torch.full((cu[-1], hq), 7.0, device="cuda") if lse else None
    if ws:
        w = tq.attn_workspace(cu[-1], len(keys), hq, hk, d)
    args = (gq, kc.cuda(), vc.cuda(), table.cuda(), ints(keys), ints(cu) if cu_given else None)
    kw = dict(scale=scale, window=window, max_len=max(new + [0]), out_dtype=ot, lse=gl, ws=w, bad_flag=flag)
    got = tq.paged_attn(*args, **kw)
    torch.cuda.synchronize()
    assert int(flag) == 0
    want, wl, spread, size = so.attention(q, kc, vc, table, keys, cu, scale, window)
    near(got, want, so.attention_bound(want, spread, size, d, max(keys + [1]), ot, ct), "out")
    if lse:
        empty = torch.isinf(wl)
        assert torch.equal(torch.isinf(gl.cpu()), empty) and bool((gl.cpu()[empty] < 0).all())
        near(gl.cpu()[~empty], wl[~empty], ((d + 4) * size + max(keys + [1]) + 16 + wl.abs())[~empty] * so.U32, "lse")
    # again on the same workspace, and without one
    assert torch.equal(tq.paged_attn(*args, **kw), got)
    if ws:
        plain = tq.paged_attn(*args, **{**kw, "ws": None})
        near(plain, want, so.attention_bound(want, spread, size, d, max(keys + [1]), ot, ct), "out without a workspace")


TOKEN = [
    # keys of the sequences (one token each), heads, kv heads, dim, page, cache, out, window
    ([1], 1, 1, 64, 16, BF, BF, 0),
    ([2, 1, 31], 12, 1, 128, 16, BF, F32, 0),
    ([32, 33, 63, 64, 65], 6, 2, 128, 32, HF, HF, 0),
    ([1000], 24, 2, 256, 64, BF, F32, 0),
    ([700, 5, 128, 129, 257, 1], 8, 4, 64, 64, HF, F32, 0),
    ([515, 90, 17], 4, 4, 256, 16, BF, BF, 100),
    ([300, 1111], 34, 2, 128, 256, BF, BF, 0),
    ([2500], 16, 1, 64, 128, BF, F32, 0),
    ([600, 40], 5, 1, 128, 16, HF, F32, 1),
]


@pytest.mark.parametrize("case", TOKEN, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_paged_attn_one_token(tq, case):
    keys, hq, hk, d, page, ct, ot, window = case
    attn_check(tq, [1] * len(keys), keys, hq, hk, d, page, ct, ot, window)
    attn_check(tq, [1] * len(keys), keys, hq, hk, d, page, ct, ot, window, strided=True, cu_given=False, lse=False, poison=False, seed=1)


CHUNK = [
    # new, keys, heads, kv heads, dim, page, cache, out, window
    ([2], [2], 2, 1, 64, 16, BF, BF, 0),
    ([5], [40], 12, 1, 128, 16, BF, F32, 0),
    ([17, 1, 0, 3], [17, 70, 30, 3], 6, 2, 128, 64, HF, F32, 0),
    ([64], [64], 4, 1, 256, 64, BF, BF, 0),
    ([65, 33], [200, 33], 4, 2, 256, 32, BF, F32, 0),
    ([130, 7], [131, 300], 6, 1, 64, 16, HF, HF, 0),
    ([100], [333], 3, 3, 128, 128, BF, BF, 0),
    ([90, 50], [190, 400], 4, 1, 128, 16, BF, BF, 33),
    ([70, 1], [70, 1], 6, 2, 256, 16, HF, F32, 16),
    ([9, 4], [4, 0], 2, 1, 64, 16, BF, F32, 0),          # tokens before the first key see nothing
    ([70, 60], [40, 100], 4, 1, 64, 16, BF, F32, 2**31 - 1),  # the widest window there is
    ([150], [150], 24, 2, 256, 64, BF, F32, 0),
    ([210, 40], [260, 41], 12, 1, 128, 64, BF, F32, 64),
    ([2, 2], [2300, 2100], 768, 64, 64, 64, BF, BF, 0),  # many key heads: few rows each, still split
]


@pytest.mark.parametrize("case", CHUNK, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_paged_attn_chunk(tq, case):
    new, keys, hq, hk, d, page, ct, ot, window = case
    attn_check(tq, new, keys, hq, hk, d, page, ct, ot, window)


def test_paged_attn_large_logits(tq):
    attn_check(tq, [3], [200], 4, 2, 128, 16, BF, F32, scale=3.0)
    attn_check(tq, [80], [300], 4, 2, 128, 16, HF, HF, scale=-2.0)


@pytest.mark.parametrize("ct,bad", [(BF, math.inf), (HF, -math.inf), (BF, math.nan)])
@pytest.mark.parametrize("new,keys", [(1, 40), (40, 90), (150, 200)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_paged_attn_a_late_key_stays_unseen(tq, ct, bad, new, keys, dim):
    """A non-finite value of a key reaches the tokens that see it and no other."""
    hq, hk, page = 4, 2, 16
    q, kc, vc, table, cu = attn_inputs([new], [keys], hq, hk, dim, page, ct)
    late = keys - max(1, new // 3)  # tokens before it do not see it
    vc[table[0, late // page], :, 5, late % page] = bad
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints([keys]), ints(cu), out_dtype=F32, max_len=new).cpu()
    first = late - (keys - new)  # the token at the late key
    clean = vc.clone()
    clean[table[0, late // page], :, 5, late % page] = 0
    want, _, spread, size = so.attention(q, kc, clean, table, [keys], cu, dim**-0.5, 0)
    bound = so.attention_bound(want, spread, size, dim, keys, F32, ct)
    near(got[:first], want[:first], bound[:first], "tokens before it")
    rest = [x for x in range(dim) if x != 5]
    near(got[first:][..., rest], want[first:][..., rest], bound[first:][..., rest], "other columns")
    hit = got[first:][..., 5]
    assert bool(torch.isnan(hit).all() if math.isnan(bad) else (hit == bad).all())


def test_paged_attn_bad_tables(tq):
    """Pages and lengths out of range: flagged, not read, and the keys behind them count as unseen."""
    hq, hk, d, page = 4, 2, 128, 16
    for new, keys in (([1, 1], [100, 64]), ([40, 70], [100, 64 + 32])):
        q, kc, vc, table, cu = attn_inputs(new, keys, hq, hk, d, page, BF)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        for entry in (kc.shape[0], -1, 2**30, -(2**31)):
            t = table.clone()
            t[0, 0] = entry
            flag = ints([0])
            got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), t.cuda(), ints(keys), ints(cu), out_dtype=F32, bad_flag=flag, max_len=max(new))
            torch.cuda.synchronize()
            assert int(flag) == 1
            # sequence 0 without its first page: the same as one that is 16 keys shorter
            short = table.clone()
            short[0, :-1] = table[0, 1:]
            want, _, spread, size = so.attention(q, kc, vc, short, [keys[0] - page, keys[1]], cu, d**-0.5, 0)
            near(got, want, so.attention_bound(want, spread, size, d, 128, F32, BF), "out")
        flag = ints([0])
        tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.clamp(min=0).cuda(), ints([2**31 - 1, keys[1]]), ints(cu), bad_flag=flag, max_len=max(new))
        tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.clamp(min=0).cuda(), ints([-5, keys[1]]), ints([-3, 1 << 30, 2]), max_len=max(new))
        torch.cuda.synchronize()
        assert int(flag) == 1


# ---- gdn -----------------------------------------------------------------------------------------------------------

def gdn_inputs(n, kh, vh, dk, dv, it, seed=0, states=None):
    r = gen(seed + sum(n) + dk + dv)
    t, b = sum(n), len(n)
    q, k, v = (torch.randn(t, h, x, generator=r).to(it) for h, x in ((kh, dk), (kh, dk), (vh, dv)))
    g, beta = -torch.exp(torch.randn(t, vh, generator=r) * 1.5 - 2.5), torch.sigmoid(torch.randn(t, vh, generator=r) * 1.5)
    state = torch.randn(states or b, vh, dk, dv, generator=r) * 0.3
    return q, k, v, g, beta, state, [sum(n[:i]) for i in range(b + 1)]


def gdn_check(tq, n, kh, vh, dk, dv, it, ot, g=None, beta=None, l2norm=True, same_key=False, strided=False, ws=True, hint=True, cu_given=True, seed=0):
    q, k, v, gg, bb, state, cu = gdn_inputs(n, kh, vh, dk, dv, it, seed)
    g, beta = gg if g is None else g(gg), bb if beta is None else beta(bb)
    if same_key:
        k = k[:1].expand_as(k).contiguous()
    if not l2norm:  # keys of norm one already, near enough
        k = (k.double() / k.double().norm(dim=-1, keepdim=True)).to(it)
        q = (q.double() / q.double().norm(dim=-1, keepdim=True)).to(it)
    if strided:
        qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).cuda()
        gq, gk, gv = (x.unflatten(1, (-1, w)) for x, w in zip(qkv.split([kh * dk, kh * dk, vh * dv], 1), (dk, dk, dv)))
    else:
        gq, gk, gv = q.cuda(), k.cuda(), v.cuda()
    gc = torch.tensor(cu, dtype=torch.int32, device="cuda") if cu_given else None
    hint = max(n + [0]) if hint else 0
    w = tq.gdn_workspace(sum(n), len(n), vh, dk, dv, max_len=hint) if ws else None
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    gs, after = state.cuda(), torch.full(state.shape, 9.0, device="cuda")
    args = (gq, gk, gv, g.cuda(), beta.cuda())
    kw = dict(l2norm=l2norm, out_dtype=ot, ws=w, max_len=hint, bad_flag=flag)
    got = tq.gdn(*args, gs, gc, state_out=after, **kw)
    torch.cuda.synchronize()
    assert int(flag) == 0 and torch.equal(gs.cpu(), state)
    want, states, big = so.gdn(q, k, v, g, beta, state, cu, dk**-0.5, l2norm, 1e-6)
    bound = so.gdn_bound(max(n + [0]), dk, big)
    near(after, states, torch.full_like(states, bound), "state")
    near(got, want, so.HALF_STEP[ot] * want.abs() + bound * dk**-0.5 + (2.0**-25 if ot == HF else 0), "out")
    # in place, twice the same
    again = tq.gdn(*args, gs, gc, **kw)
    assert torch.equal(again, got) and torch.equal(gs, after)


GDN = [
    # lengths, key heads, value heads, dk, dv, in, out
    ([1], 1, 1, 64, 32, F32, F32),
    ([1, 1, 1], 2, 6, 128, 128, BF, BF),
    ([2, 0, 5], 1, 2, 128, 64, HF, F32),
    ([9], 2, 2, 64, 256, BF, F32),
    ([16, 3], 1, 3, 128, 96, F32, F32),
    ([63], 1, 1, 128, 128, F32, F32),
    ([64], 1, 2, 64, 64, HF, HF),
    ([65, 1, 0, 64], 1, 2, 128, 128, BF, F32),
    ([200, 31], 2, 2, 128, 32, F32, F32),
    ([129, 128, 127], 1, 1, 64, 160, BF, BF),
    ([333], 1, 3, 128, 128, HF, F32),
]


@pytest.mark.parametrize("case", GDN, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("ws", [True, False])
def test_gdn(tq, case, ws):
    gdn_check(tq, *case, ws=ws)
    gdn_check(tq, *case, ws=ws, strided=True, hint=False, l2norm=False, seed=1)


def test_gdn_one_token_without_offsets(tq):
    gdn_check(tq, [1] * 5, 2, 4, 128, 64, F32, F32, cu_given=False)


@pytest.mark.parametrize("n", [[1, 3], [150, 70]])
def test_gdn_extreme_gates(tq, n):
    def resets(g):  # states cleared now and then, decays of nothing in between
        g = g.clone()
        g[::7] = -math.inf
        g[1::5] = 0.0
        return g

    gdn_check(tq, n, 1, 2, 128, 64, F32, F32, g=resets)
    gdn_check(tq, n, 1, 2, 128, 64, F32, F32, g=lambda g: g * 40 - 50)
    gdn_check(tq, n, 1, 2, 64, 64, F32, F32, g=torch.zeros_like, beta=torch.ones_like)
    gdn_check(tq, n, 1, 2, 128, 64, F32, F32, beta=torch.zeros_like)


@pytest.mark.parametrize("n", [[5], [190]])
def test_gdn_the_same_key_again(tq, n):
    """Every key alike and every write whole: the strongest coupling of a chunk's tokens."""
    gdn_check(tq, n, 1, 1, 128, 64, F32, F32, g=torch.zeros_like, beta=torch.ones_like, same_key=True)
    gdn_check(tq, n, 1, 1, 64, 32, BF, F32, same_key=True)


@pytest.mark.parametrize("n", [[1, 1, 1], [70, 3, 100]])
def test_gdn_slots(tq, n):
    q, k, v, g, beta, state, cu = gdn_inputs(n, 1, 2, 64, 64, F32, states=6)
    c = lambda x: x.cuda()  # noqa: E731
    gc = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ws = tq.gdn_workspace(sum(n), len(n), 2, 64, 64, max_len=max(n))
    order = [4, -1, 2]
    first = torch.stack([state[4], torch.zeros_like(state[0]), state[2]])
    want, states, big = so.gdn(q, k, v, g, beta, first, cu, 0.125, True, 1e-6)
    bound = so.gdn_bound(max(n), 64, big)
    for third, bad in ((2, 0), (6, 1), (2**31 - 1, 1)):
        if bad:  # out of range: starts from zeros, stores nothing
            first[2] = 0
            want, states, big = so.gdn(q, k, v, g, beta, first, cu, 0.125, True, 1e-6)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        gs = state.cuda()
        got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, gc, slots=torch.tensor(order[:2] + [third], dtype=torch.int32, device="cuda"), l2norm=True,
                     ws=ws, max_len=max(n), bad_flag=flag)
        torch.cuda.synchronize()
        assert int(flag) == bad
        near(got, want, so.HALF_STEP[F32] * want.abs() + bound * 0.125, "out")
        near(gs[4], states[0], torch.full_like(states[0], bound), "state 4")
        if not bad:
            near(gs[2], states[2], torch.full_like(states[2], bound), "state 2")
        kept = [0, 1, 3, 5] + ([2] if bad else [])
        assert torch.equal(gs[kept].cpu(), state[kept])


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-4, 3, 900, 9], [0, 0, 0, 0], [7, 200, -200, 8]])
def test_gdn_bad_offsets_stay_in_bounds(tq, cu):
    """Offsets that are no offsets: flagged; what they reach is computed, nothing outside the tensors is touched."""
    q, k, v, g, beta, state, _ = gdn_inputs([9], 1, 2, 64, 64, F32, states=3)
    c = lambda x: x.cuda()  # noqa: E731
    for ws in (None, tq.gdn_workspace(9, 3, 2, 64, 64, max_len=64)):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        gs = state.cuda()
        tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, torch.tensor(cu, dtype=torch.int32, device="cuda"), l2norm=True, ws=ws, max_len=64 if ws is not None else 0,
               bad_flag=flag)
        torch.cuda.synchronize()
        assert int(flag) == (0 if cu == [0, 0, 0, 0] else 1)
        if cu == [0, 0, 0, 0]:
            assert torch.equal(gs.cpu(), state)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["v", "k", "q", "beta", "g"])
def test_gdn_a_late_token_stays_late(tq, bad, where):
    """What is not finite at token 100 reaches no token before it, no other head and, through v, no other column."""
    n, late, vh, dk, dv = 170, 100, 2, 128, 64
    q, k, v, g, beta, state, cu = gdn_inputs([n], vh, vh, dk, dv, BF)
    bad_at = {"v": v, "k": k, "q": q}
    if where in bad_at:
        bad_at[where][late, 0, 5] = bad
    else:
        {"beta": beta, "g": g}[where][late, 0] = abs(bad)
    c = lambda x: x.cuda()  # noqa: E731
    gs = state.cuda()
    got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, torch.tensor(cu, dtype=torch.int32, device="cuda"), l2norm=True, out_dtype=F32, max_len=n,
                 ws=tq.gdn_workspace(n, 1, vh, dk, dv, max_len=n)).cpu()
    ok = {"v": v, "k": k, "q": q, "beta": beta, "g": g}
    clean = {x: torch.nan_to_num(y, 0.0, 0.0, 0.0) for x, y in ok.items()}
    want, states, big = so.gdn(clean["q"], clean["k"], clean["v"], clean["g"], clean["beta"], state, cu, dk**-0.5, True, 1e-6)
    bound = so.gdn_bound(n, dk, big) * dk**-0.5
    limit = so.HALF_STEP[F32] * want.abs() + bound
    near(got[:late], want[:late], limit[:late], "tokens before it")
    near(got[:, 1], want[:, 1], limit[:, 1], "the other head")
    near(gs[0, 1], states[0, 1], torch.full_like(states[0, 1], so.gdn_bound(n, dk, big)), "the other head's state")
    if where == "v":
        rest = [x for x in range(dv) if x != 5]
        near(got[:, 0][:, rest], want[:, 0][:, rest], limit[:, 0][:, rest], "other columns")
    assert not bool(torch.isfinite(got[late, 0]).all())
    if where == "q":  # only its own token
        near(got[late + 1 :], want[late + 1 :], limit[late + 1 :], "tokens after it")
        near(gs, states, torch.full_like(states, so.gdn_bound(n, dk, big)), "state")


@pytest.mark.parametrize("hint", ["right", "none", "short"])
@pytest.mark.parametrize("slots", [False, True])
def test_gdn_in_several_launches(tq, hint, slots):
    """More chunks than the workspace holds: states go from launch to launch, also those of sequences without a slot."""
    n, heads, dk, dv = [1500, 700, 0, 40, 5, 130], 64, 128, 32
    q, k, v, g, beta, state, cu = gdn_inputs(n, heads, heads, dk, dv, F32)
    max_len = {"right": max(n), "none": 0, "short": 64}[hint]
    c = lambda x: x.cuda()  # noqa: E731
    ws = tq.gdn_workspace(sum(n), len(n), heads, dk, dv, max_len=max_len)
    assert ws.numel() == 256 << 20
    order = [0, -1, 2, 3, -1, 5] if slots else None
    gs, after = state.cuda(), torch.full(state.shape, 9.0, device="cuda")
    got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, torch.tensor(cu, dtype=torch.int32, device="cuda"), l2norm=True, ws=ws, max_len=max_len, state_out=after,
                 slots=torch.tensor(order, dtype=torch.int32, device="cuda") if slots else None)
    torch.cuda.synchronize()
    some = [0, 17, 63]
    start = state.clone()
    if slots:
        start[1] = start[4] = 0
    want, states, big = so.gdn(q[:, some], k[:, some], v[:, some], g[:, some], beta[:, some], start[:, some], cu, dk**-0.5, True, 1e-6)
    bound = so.gdn_bound(max(n), dk, big)
    near(got[:, some], want, so.HALF_STEP[F32] * want.abs() + bound * dk**-0.5, "out")
    stored = [0, 2, 3, 5] if slots else [0, 1, 2, 3, 4, 5]
    near(after[stored][:, some], states[stored], torch.full_like(states[stored], bound), "state")
    if slots:
        assert bool((after[[1, 4]] == 9.0).all())


@pytest.mark.parametrize("it,ot", [(F32, F32), (BF, BF), (HF, F32)])
def test_gdn_many_chunks_of_shared_heads(tq, it, ot):
    """Enough chunks that a workgroup prepares all value heads of a key head; one of them has a token that is not finite."""
    n, kh, vh, dk, dv, late = [1900, 300], 16, 48, 64, 32, 1000
    q, k, v, g, beta, state, cu = gdn_inputs(n, kh, vh, dk, dv, it)
    beta[late, 1] = math.nan
    c = lambda x: x.cuda()  # noqa: E731
    gs = state.cuda()
    got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, torch.tensor(cu, dtype=torch.int32, device="cuda"), l2norm=True, out_dtype=ot, max_len=max(n),
                 ws=tq.gdn_workspace(sum(n), 2, vh, dk, dv, max_len=max(n))).cpu()
    for key in (0, 7, 15):
        heads = slice(3 * key, 3 * key + 3)
        want, states, big = so.gdn(q[:, key : key + 1], k[:, key : key + 1], v[:, heads], g[:, heads], torch.nan_to_num(beta[:, heads]), state[:, heads], cu,
                                   dk**-0.5, True, 1e-6)
        bound = so.gdn_bound(max(n), dk, big)
        limit = so.HALF_STEP[ot] * want.abs() + bound * dk**-0.5
        have, after = got[:, heads].double(), gs[:, heads].cpu().double()
        if key == 0:  # head 1 of the first sequence, from the late token on
            assert not bool(torch.isfinite(have[late : n[0], 1]).any()) and not bool(torch.isfinite(after[0, 1]).any())
            have[late : n[0], 1], after[0, 1] = want[late : n[0], 1], states[0, 1]
        near(have, want, limit, f"out of key head {key}")
        near(after, states, torch.full_like(states, bound), f"states of key head {key}")


@pytest.mark.parametrize("cu", [[0, 150, 90, 200], [-64, 90, 900, 200], [70, 200, -200, 130], [200, 0, 200, 0]])
def test_gdn_chunks_with_bad_offsets_stay_in_bounds(tq, cu):
    q, k, v, g, beta, state, _ = gdn_inputs([200], 1, 2, 64, 64, F32, states=3)
    c = lambda x: x.cuda()  # noqa: E731
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = tq.gdn_workspace(200, 3, 2, 64, 64, max_len=200)
    tq.gdn(c(q), c(k), c(v), c(g), c(beta), state.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"), l2norm=True, ws=ws, max_len=200, bad_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 1


# ---- streams and graphs --------------------------------------------------------------------------------------------

def block(tq, s):
    q = tq.rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["freq"], s["kc"], s["vc"], out=s["qo"])
    tq.paged_attn(q, s["kc"], s["vc"], s["table"], s["len"], s["cu"], max_len=s["n"], out=s["o"], ws=s["ws"])
    tq.gdn(s["gq"], s["gk"], s["gv"], s["g"], s["beta"], s["state"], s["cu"], l2norm=True, max_len=s["n"], out=s["go"], state_out=s["after"], ws=s["gws"])


def block_state(tq, n, seed):
    r = gen(seed)
    page, d, keys = 16, 128, 500
    c = lambda *shape, dtype=F32: torch.randn(*shape, generator=r).to(dtype).cuda()  # noqa: E731
    i = lambda x, dtype=torch.int32: torch.tensor(x, dtype=dtype, device="cuda")  # noqa: E731
    table = torch.randperm(40, generator=r)
    pos = torch.arange(keys - n, keys)
    s = {"q": c(n, 4, d), "k": c(n, 2, d), "v": c(n, 2, d), "pos": pos.int().cuda(), "slots": (table[pos // page] * page + pos % page).cuda(),
         "freq": tq.rope_frequencies(d, device="cuda")[0], "kc": c(40, 2, page, d, dtype=BF), "vc": c(40, 2, d, page, dtype=BF), "qo": c(n, 4, d, dtype=BF),
         "table": table.int()[None].cuda(), "len": i([keys]), "cu": i([0, n]), "n": n, "o": c(n, 4, d), "ws": tq.attn_workspace(n, 1, 4, 2, d),
         "gq": c(n, 2, d), "gk": c(n, 2, d), "gv": c(n, 4, d), "g": -c(n, 4).abs(), "beta": c(n, 4).sigmoid(), "state": c(1, 4, d, d), "go": c(n, 4, d),
         "after": c(1, 4, d, d), "gws": tq.gdn_workspace(n, 1, 4, d, d, max_len=n)}
    return s


NAMES = ("qo", "kc", "vc", "o", "go", "after")


@pytest.mark.parametrize("n", [1, 20, 150])
def test_graph_replays_equal_eager(tq, n):
    s = block_state(tq, n, n)
    block(tq, s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in NAMES}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(tq, s)
    for _ in range(4):
        for k in ("qo", "o", "go", "after"):
            s[k].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[k], want[k]) for k in NAMES)
        other = block_state(tq, n, n + 1)
        block(tq, other)  # eager work of other tensors in between
        torch.cuda.synchronize()


@pytest.mark.parametrize("n", [1, 150])
def test_runs_on_the_current_stream(tq, n):
    s = block_state(tq, n, 50 + n)
    block(tq, s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in NAMES}
    side = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    q, s["q"] = s["q"], torch.zeros_like(s["q"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            x = torch.mm(x, x).clamp(-1, 1)
        s["q"].copy_(q)  # arrives late, on this stream alone
        block(tq, s)
    side.synchronize()
    assert all(torch.equal(s[k], want[k]) for k in NAMES)


# ---- the two ways into a call ---------------------------------------------------------------------------------------

def test_output_given_or_made(tq):
    """A call with `out` is checked in C++, one without in Python: the same results."""
    s = block_state(tq, 20, 7)
    block(tq, s)
    want = {k: s[k].clone() for k in NAMES}
    q = tq.rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["freq"], s["kc"], s["vc"])
    o = tq.paged_attn(q, s["kc"], s["vc"], s["table"], s["len"], s["cu"], max_len=20, out_dtype=F32, ws=s["ws"])
    go = tq.gdn(s["gq"], s["gk"], s["gv"], s["g"], s["beta"], s["state"], s["cu"], l2norm=True, max_len=20, state_out=s["after"], ws=s["gws"])
    torch.cuda.synchronize()
    for name, got in (("qo", q), ("o", o), ("go", go), ("kc", s["kc"]), ("vc", s["vc"]), ("after", s["after"])):
        assert torch.equal(got, want[name]), name


@pytest.mark.parametrize("over,error", [
    (dict(q="double"), ValueError), (dict(k="bfloat16"), ValueError), (dict(k="cpu"), ValueError), (dict(pos="long"), ValueError),
    (dict(slots="int"), ValueError), (dict(slots=None), ValueError), (dict(freq="float"), ValueError), (dict(kc="float"), ValueError),
    (dict(vc="cpu"), ValueError), (dict(qo="float"), ValueError), (dict(q="shifted"), RuntimeError), (dict(eps=-1.0), RuntimeError),
    (dict(layout="pairs"), ValueError), (dict(v="narrow"), RuntimeError),
])
def test_rope_append_refuses_with_output_given(tq, over, error):
    s = {**block_state(tq, 5, 3), "eps": 1e-6, "layout": "half"}
    for name, how in over.items():
        if how == "shifted":  # rows that do not start at 16 bytes
            s[name] = torch.zeros(s[name].numel() + 8, device="cuda")[1 : 1 + s[name].numel()].view(s[name].shape)
        elif how == "narrow":
            s[name] = s[name][..., :64].contiguous()
        elif isinstance(how, str) and name != "layout":
            s[name] = getattr(s[name], how)()
        else:
            s[name] = how
    before = [s[x].clone() for x in ("qo", "kc", "vc")]
    with pytest.raises(error):
        tq.rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["freq"], s["kc"], s["vc"], eps=s["eps"], layout=s["layout"], out=s["qo"])
    torch.cuda.synchronize()
    assert all(torch.equal(x, s[y]) for x, y in zip(before, ("qo", "kc", "vc")))


@pytest.mark.parametrize("over,error", [
    (dict(qo="half"), RuntimeError), (dict(table="long"), ValueError), (dict(table="cpu"), ValueError), (dict(len="long"), ValueError),
    (dict(cu="long"), ValueError), (dict(o="half"), RuntimeError), (dict(ws="float"), ValueError), (dict(window=-1), RuntimeError),
    (dict(scale=math.inf), RuntimeError), (dict(n=-1), RuntimeError), (dict(vc="cpu"), ValueError),
])
def test_paged_attn_refuses_with_output_given(tq, over, error):
    s = {**block_state(tq, 5, 3), "window": 0, "scale": None}
    for name, how in over.items():
        s[name] = getattr(s[name], how)() if isinstance(how, str) else how
    before = s["o"].clone()
    with pytest.raises(error):
        tq.paged_attn(s["qo"], s["kc"], s["vc"], s["table"], s["len"], s["cu"], scale=s["scale"], window=s["window"], max_len=s["n"], out=s["o"], ws=s["ws"])
    torch.cuda.synchronize()
    assert torch.equal(before, s["o"])


@pytest.mark.parametrize("over,error", [
    (dict(gq="double"), ValueError), (dict(gk="half"), ValueError), (dict(g="cpu"), ValueError), (dict(beta="double"), ValueError),
    (dict(state="half"), ValueError), (dict(cu="long"), ValueError), (dict(go="half"), RuntimeError), (dict(n=-1), RuntimeError),
    (dict(scale=math.nan), RuntimeError), (dict(gws="float"), ValueError), (dict(after="cpu"), ValueError),
])
def test_gdn_refuses_with_output_given(tq, over, error):
    s = {**block_state(tq, 150, 3), "scale": None}
    for name, how in over.items():
        s[name] = getattr(s[name], how)() if isinstance(how, str) else how
    before = s["go"].clone()
    with pytest.raises(error):
        tq.gdn(s["gq"], s["gk"], s["gv"], s["g"], s["beta"], s["state"], s["cu"], scale=s["scale"], l2norm=True, max_len=s["n"], out=s["go"],
               state_out=s["after"], ws=s["gws"])
    torch.cuda.synchronize()
    assert torch.equal(before, s["go"])


# ---- long caches -----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("new,keys,hq,hk,d,page,ct,ot,window", [
    (1, 70_001, 6, 1, 256, 64, BF, F32, 0),     # joined in two levels
    (1, 33_000, 16, 2, 128, 16, HF, HF, 0),
    (1, 33_000, 17, 1, 64, 16, HF, F32, 30_000),
    (33, 20_000, 4, 1, 128, 64, BF, BF, 0),     # two tiles of 128 rows, split
    (70, 9_000, 2, 1, 256, 32, HF, F32, 5_000),
    (300, 5_000, 8, 4, 64, 128, BF, F32, 0),
])
def test_paged_attn_long(tq, new, keys, hq, hk, d, page, ct, ot, window):
    """Against float64 on the GPU: whole matrices, from the definition."""
    g = torch.Generator(device="cuda")
    g.manual_seed(keys)
    pages = -(-keys // page)
    table = torch.randperm(pages, generator=g, device="cuda")
    q = torch.randn(new, hq, d, generator=g, device="cuda").to(ct)
    kc, vc = torch.randn(pages, hk, page, d, generator=g, device="cuda").to(ct), torch.randn(pages, hk, d, page, generator=g, device="cuda").to(ct)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lse = torch.empty(new, hq, device="cuda")
    got = tq.paged_attn(q, kc, vc, table.int()[None], ints([keys]), ints([0, new]), window=window, max_len=new, out_dtype=ot, lse=lse,
                        ws=tq.attn_workspace(new, 1, hq, hk, d))
    pos = torch.arange(keys - new, keys, device="cuda")[:, None]
    key = torch.arange(keys, device="cuda")[None]
    hide = (key > pos) | ((key <= pos - window) if window else False)
    for h in range(hq):
        k = kc[table, h // (hq // hk)].flatten(0, 1)[:keys].double()
        v = vc[table, h // (hq // hk)].transpose(1, 2).flatten(0, 1)[:keys].double()
        x = q[:, h].double()
        s = (x @ k.t() * d**-0.5).masked_fill(hide, -math.inf)
        size = (x.abs() @ k.abs().t() * d**-0.5).masked_fill(hide, 0).amax(-1)
        p = torch.softmax(s, -1)
        want, spread = p @ v, p @ v.abs()
        near(got[:, h], want.cpu(), so.attention_bound(want.cpu(), spread.cpu(), size.cpu(), d, keys, ot, ct), f"head {h}")
        wl = torch.logsumexp(s, -1).cpu()
        near(lse[:, h], wl, ((d + 4) * size.cpu() + keys + 16 + wl.abs()) * so.U32, f"lse {h}")
