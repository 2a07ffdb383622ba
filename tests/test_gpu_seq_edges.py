"""Where the operators between a block's projections meet the ends of their ranges: lengths beyond the block table, and
finite inputs whose products are not."""
import math

import pytest
import torch

import seq_oracle as so
from test_gpu_seq import BF, F32, HF, attn_inputs, gdn_inputs, near, tq  # noqa: F401  (tq: the fixture)

pytestmark = pytest.mark.gpu


# ---- lengths beyond the table ----------------------------------------------------------------------------------------

def seen_attention(q, kc, vc, table, kv_len, cu, keys, window):
    """Each token over the keys that it sees: position and window from kv_len, keys from `keys` on are nobody's."""
    tokens, heads, d = q.shape
    page, group = kc.shape[2], heads // kc.shape[1]
    out, spread = torch.zeros(tokens, heads, d, dtype=torch.float64), torch.zeros(tokens, heads, d, dtype=torch.float64)
    lse, size = torch.full((tokens, heads), -math.inf, dtype=torch.float64), torch.zeros(tokens, heads, dtype=torch.float64)
    for b, m in enumerate(kv_len):
        for t in range(cu[b], cu[b + 1]):
            pos = m - cu[b + 1] + t
            low, end = max(0, pos - window + 1) if window else 0, min(pos + 1, keys)
            at = torch.arange(low, max(low, end))
            if not at.numel():
                continue
            pages = table[b, at // page].long()
            for h in range(heads):
                k, v = kc[pages, h // group, at % page].double(), vc[pages, h // group, :, at % page].double()
                x = q[t, h].double()
                s = k @ x * d**-0.5
                p = torch.softmax(s, 0)
                out[t, h], spread[t, h], lse[t, h] = p @ v, p @ v.abs(), torch.logsumexp(s, 0)
                size[t, h] = (k.abs() @ x.abs()).max() * d**-0.5
    return out, lse, spread, size


@pytest.mark.parametrize("new,hq,hk,dim,ct,ot", [
    ([1, 1], 4, 2, 128, BF, F32), ([1, 3], 2, 1, 256, HF, HF), ([17, 9], 2, 1, 64, BF, BF),          # 16 rows per workgroup
    ([40, 33], 16, 16, 64, BF, F32), ([40, 33], 32, 16, 128, HF, HF), ([40, 33], 16, 8, 256, BF, F32),  # 128
])
@pytest.mark.parametrize("page,width", [(16, 7), (64, 2)])
@pytest.mark.parametrize("over,window", [(50, 0), (5, 70), (50, 112), (50, 128), (50, 40), (2**31, 2**31 - 1), (2**31, 2**31 - 60), (2**31, 0)])
def test_paged_attn_lengths_beyond_the_table(tq, new, hq, hk, dim, ct, ot, page, width, over, window):
    """Flagged; the tokens keep their positions, and see of the table's keys what those positions and the window leave."""
    keys = page * width
    kv_len = [min(keys + over, 2**31 - 1), keys + 3]
    q, kc, vc, table, cu = attn_inputs(new, [keys] * 2, hq, hk, dim, page, ct)
    table = table[:, :width].contiguous()
    want, wl, spread, size = seen_attention(q, kc, vc, table, kv_len, cu, keys, window)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for ws in (tq.attn_workspace(cu[-1], 2, hq, hk, dim), None):
        flag, lse = ints([0]), torch.full((cu[-1], hq), 7.0, device="cuda")
        got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints(kv_len), ints(cu), window=window, max_len=max(new), out_dtype=ot, lse=lse,
                            ws=ws, bad_flag=flag)
        torch.cuda.synchronize()
        assert int(flag) == 1
        near(got, want, so.attention_bound(want, spread, size, dim, keys, ot, ct), "out")
        empty = torch.isinf(wl)
        assert torch.equal(torch.isinf(lse.cpu()), empty) and bool((lse.cpu()[empty] < 0).all())
        near(lse.cpu()[~empty], wl[~empty], ((dim + 4) * size + keys + 16 + wl.abs())[~empty] * so.U32, "lse")


# ---- finite inputs, products that are not -----------------------------------------------------------------------------

def gdn_run(tq, q, k, v, g, beta, state, cu, l2norm, eps=1e-6):
    c = lambda x: x.cuda()  # noqa: E731
    n = max(b - a for a, b in zip(cu, cu[1:]))
    gs = state.cuda()
    got = tq.gdn(c(q), c(k), c(v), c(g), c(beta), gs, torch.tensor(cu, dtype=torch.int32, device="cuda"), l2norm=l2norm, eps=eps, out_dtype=F32, max_len=n,
                 ws=tq.gdn_workspace(v.shape[0], len(cu) - 1, v.shape[1], k.shape[2], v.shape[2], max_len=n))
    torch.cuda.synchronize()
    return got.cpu(), gs.cpu()


@pytest.mark.parametrize("late", [0, 37, 64, 100, 169])
@pytest.mark.parametrize("what,beta_late", [(3e38, 1.5), (3.4e38, 1.0), (-3.4028234e38, 2.0), (-3.4e38, 1.0)])
def test_gdn_a_late_overflow_stays_late(tq, late, what, beta_late):
    """A write beyond fp32's range, or so near its end that its first bf16 term is infinite, reaches no token before its own,
    no other head and no other column."""
    n, vh, dk, dv = 170, 2, 128, 64
    q, k, v, g, beta, state, cu = gdn_inputs([n], vh, vh, dk, dv, F32)
    clean = v.clone()
    v[late, 0, 5], beta[late, 0] = what, beta_late
    clean[late, 0, 5] = 0
    got, after = gdn_run(tq, q, k, v, g, beta, state, cu, True)
    want, states, big = so.gdn(q, k, clean, g, beta, state, cu, dk**-0.5, True, 1e-6)
    bound = so.gdn_bound(n, dk, big)
    limit = so.HALF_STEP[F32] * want.abs() + bound * dk**-0.5
    rest = [x for x in range(dv) if x != 5]
    near(got[:late], want[:late], limit[:late], "tokens before it")
    near(got[:, 1], want[:, 1], limit[:, 1], "the other head")
    near(got[:, 0][:, rest], want[:, 0][:, rest], limit[:, 0][:, rest], "other columns")
    near(after[0, 0][:, rest], states[0, 0][:, rest], torch.full((dk, dv - 1), bound), "other columns' states")
    near(after[0, 1], states[0, 1], torch.full((dk, dv), bound), "the other head's state")


def test_gdn_large_writes_of_short_keys(tq):
    """Keys much shorter than their norm's eps: what a token writes fits fp32, what it writes over the key's norm does not."""
    n, late, dk, dv = 130, 90, 128, 64
    q, k, v, g, beta, state, cu = gdn_inputs([n], 1, 1, dk, dv, F32)
    g[:] = 0
    k[late] *= 1e-5
    v[late, 0, 5] = 1e37
    beta[late] = 1.0
    got, after = gdn_run(tq, q, k, v, g, beta, state, cu, True)
    want, states, big = so.gdn(q, k, v, g, beta, state, cu, dk**-0.5, True, 1e-6)
    assert bool(torch.isfinite(states).all()) and big < 1e38
    bound = so.gdn_bound(n, dk, big)
    near(got[late:], want[late:], so.HALF_STEP[F32] * want[late:].abs() + bound * dk**-0.5, "out")
    near(after, states, torch.full_like(states, bound), "state")
    v[late, 0, 5] = 0
    small, _, big = so.gdn(q, k, v, g, beta, state, cu, dk**-0.5, True, 1e-6)
    near(got[:late], small[:late], so.HALF_STEP[F32] * small[:late].abs() + so.gdn_bound(n, dk, big) * dk**-0.5, "tokens before it")


@pytest.mark.parametrize("late", [20, 63, 100])
def test_gdn_a_large_state_row_is_met_late(tq, late):
    """A row of the state near fp32's end that only a late token's key reaches, and overflows."""
    n, dk, dv = 120, 64, 32
    q, k, v, g, beta, state, cu = gdn_inputs([n], 1, 1, dk, dv, F32)
    k[..., 0] = q[..., 0] = 0
    k, q = (x / x.norm(dim=-1, keepdim=True) for x in (k, q))
    clean = state.clone()
    clean[..., 0, :] = 0
    state[..., 0, :] = 3e38
    g[:] = 0
    k[late] = 0
    k[late, 0, 0] = 1.0
    v[late], beta[late] = -3e38, 1.0
    got, _ = gdn_run(tq, q, k, v, g, beta, state, cu, False)
    want, _, big = so.gdn(q[:late], k[:late], v[:late], g[:late], beta[:late], clean, [0, late], dk**-0.5, False, 1e-6)
    near(got[:late], want, so.HALF_STEP[F32] * want.abs() + so.gdn_bound(n, dk, big) * dk**-0.5, "tokens before it")


@pytest.mark.parametrize("it", [F32, BF])
def test_gdn_columns_that_are_lost_leave_the_others(tq, it):
    """A column whose state is not finite: all its outputs are not from there on, and the others go on as ever, a later
    overflow's column, too, up to its own token."""
    n, vh, dk, dv = 700, 2, 128, 64
    q, k, v, g, beta, state, cu = gdn_inputs([n], vh, vh, dk, dv, it)
    clean, start = v.clone(), state.clone()
    state[0, 0, 3, 7] = math.inf                 # from the first token on
    v[70, 0, 5] = math.nan                       # from token 70 on
    v[300, 0, 40], beta[300, 0] = 3e38, 1.75     # from token 300 on: the write overflows
    v[555, 0, 41] = -math.inf
    clean[300, 0, 40] = 0
    got, after = gdn_run(tq, q, k, v, g, beta, state, cu, True)
    want, states, big = so.gdn(q, k, clean, g, beta, start, cu, dk**-0.5, True, 1e-6)
    bound = so.gdn_bound(n, dk, big)
    limit = so.HALF_STEP[F32] * want.abs() + bound * dk**-0.5
    near(got[:, 1], want[:, 1], limit[:, 1], "the other head")
    near(after[0, 1], states[0, 1], torch.full((dk, dv), bound), "the other head's state")
    for col in range(dv):
        first = {7: 0, 5: 70, 40: 300, 41: 555}.get(col, n)
        near(got[:first, 0, col], want[:first, 0, col], limit[:first, 0, col], f"column {col}")
        assert not bool(torch.isfinite(got[first:, 0, col]).any()), col
        if first == n:
            near(after[0, 0, :, col], states[0, 0, :, col], torch.full((dk,), bound), f"state of column {col}")
        else:
            assert not bool(torch.isfinite(after[0, 0, :, col]).any()), col


@pytest.mark.parametrize("power", [-30, -61])
def test_gdn_keys_of_next_to_no_length(tq, power):
    """With eps = 0 a key's norm is one however short the key is."""
    n, dk, dv = 150, 128, 64
    q, k, v, g, beta, state, cu = gdn_inputs([n], 1, 1, dk, dv, F32)
    k = k / k.norm(dim=-1, keepdim=True)
    k[70:80] *= 2.0**power
    got, after = gdn_run(tq, q, k, v, g, beta, state, cu, True, eps=0.0)
    want, states, big = so.gdn(q, k, v, g, beta, state, cu, dk**-0.5, True, 0.0)
    bound = so.gdn_bound(n, dk, big)
    near(got, want, so.HALF_STEP[F32] * want.abs() + bound * dk**-0.5, "out")
    near(after, states, torch.full_like(states, bound), "state")
