"""paged_attn in the kernel of 128 query rows per workgroup: every type, width and page size of it, each case checked to be
one that this kernel serves; twins in the kernel of 16 rows where the two could differ."""
import math

import pytest
import torch

import seq_oracle as so
from test_gpu_seq import BF, F32, HF, attn_check, attn_inputs, near, tq  # noqa: F401  (tq: the fixture)
from test_gpu_seq import test_paged_attn_long as long_check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fp16_steps(monkeypatch):
    """The oracle's bound, with the half step of an fp16 output below fp16's normal range (2^-25 whatever the value), which a
    weight of nearly one on a V of 3e-6 meets."""
    bound = so.attention_bound
    monkeypatch.setattr(so, "attention_bound", lambda *a: bound(*a) + (2.0**-25 if a[5] == HF else 0.0))


def serves(tq, new, hq, hk, d, rows, max_len=None):
    assert tq.lib().tq_paged_attn_tile_rows(sum(new), len(new), max(new) if max_len is None else max_len, hq, hk, d) == rows


CASES = [
    # new, keys, heads, kv heads, dim, page, cache, out, window
    ([40, 33], [140, 300], 16, 16, 64, 16, HF, HF, 0),
    ([130, 7, 0, 1], [131, 300, 20, 1], 24, 8, 64, 32, HF, F32, 0),
    ([90, 50], [190, 400], 32, 8, 64, 16, BF, BF, 33),
    ([70, 60], [40, 100], 32, 8, 64, 64, BF, F32, 2**31 - 1),  # tokens before the first key see nothing; the widest window
    ([18] * 9, [70, 18, 19, 64, 63, 65, 128, 129, 500], 8, 8, 64, 256, BF, BF, 0),
    ([100], [333], 48, 4, 128, 64, BF, BF, 0),
    ([45, 20, 0], [45, 333, 9], 24, 8, 128, 16, HF, HF, 0),
    ([64, 64], [64, 500], 16, 16, 128, 32, BF, BF, 100),
    ([50], [700], 34, 17, 128, 256, HF, F32, 0),
    ([31, 129], [200, 129], 12, 12, 128, 16, BF, F32, 1),
    ([64], [64], 24, 2, 256, 64, BF, BF, 0),
    ([65, 33], [200, 33], 24, 2, 256, 16, HF, HF, 0),
    ([70, 1], [170, 71], 24, 2, 256, 32, HF, F32, 16),
    ([90], [1200], 12, 4, 256, 128, BF, BF, 500),
    ([30, 20, 40], [10, 40, 0], 24, 4, 256, 16, BF, F32, 0),   # nothing seen: by the first of a sequence, by all of one
    ([129], [129], 4, 4, 256, 16, HF, HF, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c).replace(" ", ""))
def test_paged_attn_many_rows(tq, case):
    new, keys, hq, hk, d, page, ct, ot, window = case
    serves(tq, new, hq, hk, d, 128)
    attn_check(tq, new, keys, hq, hk, d, page, ct, ot, window)
    attn_check(tq, new, keys, hq, hk, d, page, ct, ot, window, strided=True, lse=False, poison=False, seed=1)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ct,ot", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_paged_attn_many_rows_scales(tq, d, ct, ot):
    new, hq, hk = [40], 32, 32
    serves(tq, new, hq, hk, d, 128)
    for scale in (-2.0, 0.0, 3.0, -1e-30):
        attn_check(tq, new, [150], hq, hk, d, 16, ct, ot, scale=scale, window=0 if scale else 70)


@pytest.mark.parametrize("ct,bad", [(BF, math.inf), (HF, -math.inf), (BF, math.nan), (HF, math.inf)])
@pytest.mark.parametrize("new,hq,hk,rows", [(40, 32, 16, 128), (60, 2, 1, 16)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_paged_attn_a_late_value_stays_late(tq, ct, bad, new, hq, hk, rows, page, dim):
    """A value of a key that is not finite reaches the tokens that see it and no other, in its columns."""
    keys = 200
    serves(tq, [new], hq, hk, dim, rows)
    q, kc, vc, table, cu = attn_inputs([new], [keys], hq, hk, dim, page, ct)
    late, cols = keys - new // 3, [5, dim - 3]
    vc[table[0, late // page], :, cols, late % page] = bad
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    first = late - (keys - new)
    clean = vc.clone()
    clean[table[0, late // page], :, cols, late % page] = 0
    want, _, spread, size = so.attention(q, kc, clean, table, [keys], cu, dim**-0.5, 0)
    rest = [x for x in range(dim) if x not in cols]
    for ot in (F32, ct):
        got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints([keys]), ints(cu), out_dtype=ot, max_len=new,
                            ws=tq.attn_workspace(new, 1, hq, hk, dim)).cpu()
        bound = so.attention_bound(want, spread, size, dim, keys, ot, ct)
        near(got[:first], want[:first], bound[:first], "tokens before it")
        near(got[first:][..., rest], want[first:][..., rest], bound[first:][..., rest], "other columns")
        hit = got[first:][..., cols]
        assert bool(torch.isnan(hit).all() if math.isnan(bad) else (hit == bad).all())


@pytest.mark.parametrize("new,hq,hk,rows", [(40, 32, 16, 128), (60, 2, 1, 16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ct", [BF, HF])
def test_paged_attn_a_seen_value_counts_whatever_its_score(tq, new, hq, hk, rows, dim, ct):
    """A key with a score of minus infinity is seen all the same: an infinite value there is not passed over."""
    keys, page, late = 100, 16, 70
    serves(tq, [new], hq, hk, dim, rows)
    q, kc, vc, table, cu = attn_inputs([new], [keys], hq, hk, dim, page, ct)
    q[..., 0] = 1.0
    kc[table[0, late // page], :, late % page, 0] = -math.inf
    vc[table[0, late // page], :, 5, late % page] = math.inf
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints([keys]), ints(cu), out_dtype=F32, max_len=new).cpu()
    first = late - (keys - new)
    assert not bool(torch.isfinite(got[first:, :, 5]).any())
    kc[table[0, late // page], :, late % page, 0] = -60000.0  # a weight of nothing
    vc[table[0, late // page], :, 5, late % page] = 0
    want, _, spread, _ = so.attention(q, kc, vc, table, [keys], cu, dim**-0.5, 0)
    kc[table[0, late // page], :, late % page, 0] = 0
    size = so.attention(q, kc, vc, table, [keys], cu, dim**-0.5, 0)[3]  # of the scores that have weight
    bound = so.attention_bound(want, spread, size, dim, keys, F32, ct)
    rest = [x for x in range(dim) if x != 5]
    near(got[:first], want[:first], bound[:first], "tokens before it")
    near(got[first:][..., rest], want[first:][..., rest], bound[first:][..., rest], "other columns")


@pytest.mark.parametrize("hq,hk,d,page,ct,ot", [(16, 16, 64, 16, HF, F32), (32, 16, 128, 16, BF, BF), (16, 16, 128, 64, HF, HF), (24, 8, 256, 16, BF, F32),
                                                (8, 8, 256, 64, HF, HF)])
def test_paged_attn_many_rows_bad_tables(tq, hq, hk, d, page, ct, ot):
    """Pages out of range: flagged, not read, and the keys behind them count as unseen."""
    new, keys = [40, 70], [3 * page + 41, 70 + page]
    serves(tq, new, hq, hk, d, 128)
    q, kc, vc, table, cu = attn_inputs(new, keys, hq, hk, d, page, ct)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    short = table.clone()  # sequence 0 without its second page: the same as one that is a page shorter
    short[0, 1:-1] = table[0, 2:]
    want, _, spread, size = so.attention(q, kc, vc, short, [keys[0] - page, keys[1]], cu, d**-0.5, 0)
    # (its last 40 keys, which causality tells apart, lie behind that page)
    for entry in (kc.shape[0], -1, 2**30, -(2**31)):
        t = table.clone()
        t[0, 1] = entry
        flag = ints([0])
        got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), t.cuda(), ints(keys), ints(cu), out_dtype=ot, bad_flag=flag, max_len=max(new),
                            ws=tq.attn_workspace(cu[-1], 2, hq, hk, d))
        torch.cuda.synchronize()
        assert int(flag) == 1
        near(got, want, so.attention_bound(want, spread, size, d, max(keys), ot, ct), "out")


@pytest.mark.parametrize("cu", [[0, 60, 20, 110], [-30, 40, 900, 110], [50, 200, -200, 80], [110, 0, 110, 0]])
@pytest.mark.parametrize("d", [64, 256])
def test_paged_attn_many_rows_bad_offsets_stay_in_bounds(tq, cu, d):
    """Offsets that are no offsets: flagged, and nothing outside the tensors is touched."""
    hq = hk = 16
    q, kc, vc, table, _ = attn_inputs([40, 30, 40], [140, 100, 90], hq, hk, d, 16, BF)
    serves(tq, [40, 30, 40], hq, hk, d, 128)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    flag, room = ints([0]), torch.full((112, hq, d), 3.0, device="cuda")
    tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.clamp(min=0).cuda(), ints([140, 100, 90]), ints(cu), max_len=40, out=room[1:111], bad_flag=flag,
                  ws=tq.attn_workspace(110, 3, hq, hk, d))
    torch.cuda.synchronize()
    assert int(flag) == 1
    assert bool((room[[0, 111]] == 3.0).all())


@pytest.mark.parametrize("hint", [0, 1, 40, 10**9])
def test_paged_attn_hints_limit_nothing(tq, hint):
    """max_len chooses between kernels; whatever it says, every token is served."""
    new, keys, hq, hk, d = [40, 1, 33], [140, 70, 300], 32, 16, 128
    serves(tq, new, hq, hk, d, 16 if hint == 1 else 128, max_len=hint)
    q, kc, vc, table, cu = attn_inputs(new, keys, hq, hk, d, 16, BF)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = tq.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints(keys), ints(cu), max_len=hint, out_dtype=F32,
                        ws=tq.attn_workspace(cu[-1], 3, hq, hk, d))
    want, _, spread, size = so.attention(q, kc, vc, table, keys, cu, d**-0.5, 0)
    near(got, want, so.attention_bound(want, spread, size, d, max(keys), F32, BF), "out")


LONG = [
    # new, keys, heads, kv heads, dim, page, cache, out, window
    (17, 20_000, 64, 8, 128, 64, BF, BF, 0),       # 32 parts: joined in two levels
    (17, 9_000, 24, 8, 256, 16, HF, F32, 0),
    (64, 6_000, 16, 16, 64, 32, HF, HF, 5_000),
    (33, 20_000, 32, 4, 128, 16, HF, F32, 0),
    (64, 7_000, 12, 2, 256, 64, BF, BF, 6_000),
    (17, 40_000, 64, 8, 64, 128, BF, F32, 0),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_paged_attn_many_rows_long(tq, case):
    """Keys split over workgroups, parts joined; against float64 on the GPU."""
    new, keys, hq, hk, d, page, ct, ot, window = case
    serves(tq, [new], hq, hk, d, 128)
    long_check(tq, new, keys, hq, hk, d, page, ct, ot, window)


@pytest.mark.parametrize("hq,hk,d,ct,ot,rows", [(64, 8, 128, BF, BF, 128), (24, 8, 256, HF, F32, 128), (32, 32, 64, BF, F32, 128), (24, 2, 256, BF, F32, 16)])
def test_paged_attn_graph_replays_and_streams(tq, hq, hk, d, ct, ot, rows):
    """Split keys, captured: every replay equals the eager call, on the capture's workspace; so does a call on another stream."""
    new, keys, page = [17], [4000], 16
    serves(tq, new, hq, hk, d, rows)
    q, kc, vc, table, cu = (x.cuda() if isinstance(x, torch.Tensor) else x for x in attn_inputs(new, keys, hq, hk, d, page, ct))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, offsets, ws = ints(keys), ints(cu), tq.attn_workspace(17, 1, hq, hk, d)
    out, lse = torch.empty(17, hq, d, dtype=ot, device="cuda"), torch.empty(17, hq, device="cuda")

    def call():
        tq.paged_attn(q, kc, vc, table, lens, offsets, max_len=17, out=out, lse=lse, ws=ws)

    call()
    torch.cuda.synchronize()
    want, want_lse = out.clone(), lse.clone()
    assert bool(torch.isfinite(want).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(4):
        out.fill_(3), lse.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        tq.paged_attn(q.flip(0).contiguous(), kc, vc, table, lens, offsets, max_len=17, out_dtype=ot, ws=tq.attn_workspace(17, 1, hq, hk, d))
        torch.cuda.synchronize()
    side, x, late = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda"), q.clone()
    q.zero_()
    out.fill_(3)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            x = torch.mm(x, x).clamp(-1, 1)
        q.copy_(late)  # arrives late, on this stream alone
        call()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
