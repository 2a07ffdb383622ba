"""The operators between a block's projections where offsets pass 32 bits: large caches, many states, many tokens."""
import math

import pytest
import torch

import seq_oracle as so
from test_gpu_seq import BF, F32, gen, near, tq  # noqa: F401  (tq: the fixture)

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_pages_far_into_a_cache(tq):
    """K and V of 5.2 GB each: what is appended to pages spread over them is found there, by both attention kernels."""
    pages, hk, page, d = 40_000, 8, 64, 128
    kc, vc = tq.kv_cache(pages, hk, page, d)
    assert kc.numel() > 2**31
    r = gen(3)
    n = 300
    table = torch.tensor([pages - 1, 0, pages // 2, 16_384, 32_767])
    at = torch.arange(n)
    slots = table[at // page] * page + at % page
    q, k, v = (torch.randn(n, h, d, generator=r) for h in (32, hk, hk))
    freq, _ = tq.rope_frequencies(64, 1e4)
    qo = tq.rope_append(q.cuda(), k.cuda(), v.cuda(), at.int().cuda(), slots.cuda(), freq.cuda(), kc, vc)
    small_k, small_v = kc[table.cuda()].cpu(), vc[table.cuda()].cpu()
    want, size = so.rope_rows(k, at, freq, "half")
    have = small_k.transpose(1, 2).flatten(0, 1)[:n]
    near(have, want, so.HALF_STEP[BF] * want.abs() + so.U32 * 64 * size, "k")
    assert torch.equal(small_v.permute(0, 3, 1, 2).flatten(0, 1)[:n], v.bfloat16())
    assert int(torch.count_nonzero(kc)) == int(torch.count_nonzero(small_k)) and int(torch.count_nonzero(vc)) == int(torch.count_nonzero(small_v))
    local = torch.arange(len(table)).int()[None]
    for new, rows in ((40, 128), (1, 16)):
        assert tq.lib().tq_paged_attn_tile_rows(new, 1, new, 32, hk, d) == rows
        got = tq.paged_attn(qo[n - new :], kc, vc, table.int()[None].cuda(), ints([n]), ints([0, new]), max_len=new, out_dtype=F32,
                            ws=tq.attn_workspace(new, 1, 32, hk, d))
        ref, _, spread, size = so.attention(qo[n - new :].cpu(), small_k, small_v, local, [n], [0, new], d**-0.5, 0)
        near(got, ref, so.attention_bound(ref, spread, size, d, n, F32, BF), f"{new} tokens")


def test_many_tokens(tq):
    """Queries and outputs of more than 2^31 values: the last tokens are rotated, and attended, as by themselves."""
    n, hq, hk, d, page, last = 190_000, 48, 2, 256, 128, 20
    q = torch.zeros(n, hq, d, dtype=BF, device="cuda")
    assert q.numel() > 2**31
    r = gen(4)
    tail = torch.randn(last, hq, d, generator=r).to(BF)
    q[-last:] = tail.cuda()
    pages = -(-n // page)
    kc, vc = tq.kv_cache(pages, hk, page, d)
    k, v = (torch.randn(n, hk, d, device="cuda").to(BF) for _ in range(2))
    at = torch.arange(n, device="cuda")
    freq, _ = tq.rope_frequencies(d, 1e4, device="cuda")
    qo = tq.rope_append(q, k, v, at.int(), at, freq, kc, vc)
    want, size = so.rope_rows(tail, at[-last:].cpu(), freq.cpu(), "half")
    near(qo[-last:], want, so.HALF_STEP[BF] * want.abs() + so.U32 * 80 * size, "q")
    del q
    window = 50
    got = tq.paged_attn(qo, kc, vc, torch.arange(pages, device="cuda").int()[None], ints([n]), ints([0, n]), window=window, max_len=n)
    near_pages = torch.arange(pages - 2, pages)
    sk, sv = kc[near_pages.cuda()].cpu(), vc[near_pages.cuda()].cpu()
    base = (pages - 2) * page  # keys before it are out of every window here
    ref, _, spread, size = so.attention(qo[-last:].cpu(), sk, sv, torch.tensor([[0, 1]]).int(), [n - base], [0, last], d**-0.5, window)
    near(got[-last:], ref, so.attention_bound(ref, spread, size, d, window, BF, BF), "out")
    assert bool(torch.isfinite(got[:: n // 50]).all())


@pytest.mark.parametrize("length", [1, 90])
def test_states_far_into_a_pool(tq, length):
    """9 GB of states: the sequences' slots are read and written, the others stay."""
    states, kh, vh, dk, dv = 2_800, 16, 48, 128, 128
    pool = torch.zeros(states, vh, dk, dv, device="cuda")
    assert pool.numel() > 2**31
    r = gen(5 + length)
    slots = [states - 1, 3, 1_500]
    start = torch.randn(3, vh, dk, dv, generator=r) * 0.3
    pool[slots] = start.cuda()
    n = [length] * 3
    cu = [sum(n[:i]) for i in range(4)]
    q, k, v = (torch.randn(3 * length, h, w, generator=r) for h, w in ((kh, dk), (kh, dk), (vh, dv)))
    g, beta = -torch.rand(3 * length, vh, generator=r), torch.rand(3 * length, vh, generator=r)
    c = lambda x: x.cuda()  # noqa: E731
    got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), pool, ints(cu), slots=ints(slots), l2norm=True, max_len=length,
                 ws=tq.gdn_workspace(3 * length, 3, vh, dk, dv, max_len=length)).cpu()
    pick = [0, 2, 47]
    keys = [h // 3 for h in pick]
    want, after, big = so.gdn(q[:, keys], k[:, keys], v[:, pick], g[:, pick], beta[:, pick], start[:, pick], cu, dk**-0.5, True, 1e-6)
    bound = so.gdn_bound(length, dk, big)
    near(got[:, pick], want, so.HALF_STEP[F32] * want.abs() + bound * dk**-0.5, "out")
    near(pool[slots][:, pick], after, torch.full_like(after, bound), "states")
    pool[slots] = 0
    assert int(torch.count_nonzero(pool)) == 0


def test_a_long_sequence_of_many_values(tq):
    """Values and outputs of more than 2^31: behind a cleared state the last tokens give what they give by themselves."""
    n, kh, vh, dk, dv, last = 360_000, 16, 48, 128, 128, 100
    r = gen(7)
    v, out = (torch.zeros(n, vh, dv, dtype=BF, device="cuda") for _ in range(2))
    assert v.numel() > 2**31
    q, k = (torch.randn(n, kh, dk, device="cuda").to(BF) for _ in range(2))
    g, beta = torch.full((n, vh), -0.1, device="cuda"), torch.full((n, vh), 0.5, device="cuda")
    g[-last] = -math.inf
    tail = torch.randn(last, vh, dv, generator=r).to(BF)
    v[-last:] = tail.cuda()
    state = torch.randn(1, vh, dk, dv, device="cuda")
    tq.gdn(q, k, v, g, beta, state, ints([0, n]), l2norm=True, max_len=n, out=out, ws=tq.gdn_workspace(n, 1, vh, dk, dv, max_len=n))
    pick = [0, 25, 47]
    keys = [h // 3 for h in pick]
    want, after, big = so.gdn(q[-last:, keys].cpu(), k[-last:, keys].cpu(), tail[:, pick], g[-last:, pick].cpu(), beta[-last:, pick].cpu(),
                              torch.zeros(1, 3, dk, dv), [0, last], dk**-0.5, True, 1e-6)
    bound = so.gdn_bound(last, dk, big)
    # The 16-bit output takes the state, P and X in two terms: 2^-17 of a column's norm for S^T q, and twice that of up to ten
    # products for P X (a decay of 0.1 per token); all times dk^-1/2: less than 3 x 2^-17.
    near(out[-last:, pick], want, so.HALF_STEP[BF] * want.abs() + bound * dk**-0.5 + 3 * 2.0**-17 * big, "out")
    near(state[:, pick], after, torch.full_like(after, bound), "state")
