"""Where the operators between a block's projections meet the ends of their ranges: lengths beyond the block table."""
import math

import pytest
import torch

import seq_oracle as so
from test_gpu_seq import BF, F32, HF, attn_inputs, near, tq  # noqa: F401  (tq: the fixture)

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
