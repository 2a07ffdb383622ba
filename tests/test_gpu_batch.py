"""GPU parity of what differs from row to row in a batch (experts, adapters, sampling) with their 64-bit definitions
(batch_oracle.py)."""
import math

import numpy as np
import pytest
import torch

import batch_oracle as bo
import tq_inputs as TI

pytestmark = pytest.mark.gpu

F32, BF, HF, I32 = torch.float32, torch.bfloat16, torch.float16, torch.int32


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


# ---- route ---------------------------------------------------------------------------------------------------------

ROUTE = [
    # tokens, experts, k, score, bias, groups, top_groups, group_best, renorm, type
    (1, 64, 8, "softmax", False, 1, 1, 1, True, F32),
    (1, 1, 1, "softmax", False, 1, 1, 1, False, BF),
    (5, 2, 2, "sigmoid", True, 1, 1, 1, True, HF),
    (7, 60, 4, "softmax", False, 1, 1, 1, False, BF),
    (33, 65, 6, "sigmoid", True, 1, 1, 1, True, F32),
    (130, 256, 8, "sigmoid", True, 8, 4, 2, True, BF),
    (130, 256, 8, "softmax", False, 8, 3, 1, True, F32),
    (64, 128, 32, "softmax", False, 4, 2, 2, False, HF),
    (9, 513, 9, "softmax", True, 27, 5, 2, True, F32),
    (3, 1024, 32, "sigmoid", True, 64, 7, 1, True, F32),
    (3, 1000, 17, "sigmoid", False, 1, 1, 1, True, BF),
    (2, 64, 1, "softmax", True, 64, 1, 1, True, F32),
]


@pytest.mark.parametrize("case", ROUTE, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("holes", [False, True])
def test_route(tq, case, holes):
    tokens, n, k, score, biased, groups, top, best, renorm, dt = case
    r = gen(tokens * 1000 + n)
    x = (torch.randn(tokens, n, generator=r) * 1.5).to(dt)  # 16-bit logits tie often
    bias = torch.rand(n, generator=r) * 0.2 - 0.1 if biased else None
    if holes:
        x[torch.rand(tokens, n, generator=r) < 0.5] = -math.inf
        x[torch.rand(tokens, n, generator=r) < 0.1] = math.nan
        x[0] = -math.inf
        x[-1] = torch.where(torch.rand(n, generator=r) < 0.3, x.new_full((n,), 0.0), -x.new_zeros(n))  # +0 and -0 are equal
        if tokens > 2:
            x[1, 0] = x[1, n // 2] = math.inf
        if biased:
            bias[n // 3] = -math.inf
    want_w, want_i = bo.route(x, k, score, bias, groups, top, best, renorm, 2.5)
    wide = torch.full((tokens, n + 3), math.nan, dtype=dt)
    wide[:, 1 : n + 1] = x
    for logits in (x.cuda(), wide.cuda()[:, 1 : n + 1]):
        w, i = tq.route(logits, k, score=score, bias=None if bias is None else bias.cuda(), groups=groups, top_groups=top, group_best=best, renorm=renorm, scale=2.5)
        assert torch.equal(i.cpu(), want_i)
        near(w, want_w, want_w.abs() * 2.0**-24 * 1.001 + 1e-45, "weights")  # fp64, rounded once


def test_route_ties_take_the_lowest_expert(tq):
    for n, k in ((64, 8), (200, 16), (1024, 32)):
        for x in (torch.zeros(1, n), -torch.zeros(1, n), torch.full((1, n), 3.25)):
            _, i = tq.route(x.cuda(), k)
            assert i.cpu().tolist() == [list(range(k))]
            _, i = tq.route(x.cuda(), k, score="sigmoid", bias=torch.zeros(n).cuda(), groups=4, top_groups=2, group_best=2)
            assert i.cpu().tolist() == [list(range(k))]
    x = torch.zeros(1, 256)
    x[0, [70, 6, 134, 255]] = 1.0  # lanes 6, 6, 6 and 63
    _, i = tq.route(x.cuda(), 5)
    assert i.cpu().tolist() == [[6, 70, 134, 255, 0]]


def test_route_scores_nearer_than_fp32_resolves(tq):
    """Biased scores whose difference fp32 loses: the bias takes the scores near 2^13."""
    x = torch.zeros(1, 64)
    x[0, :8] = torch.arange(8) * 1e-5
    w, i = tq.route(x.cuda(), 8, score="sigmoid", bias=torch.full((64,), 8192.0).cuda())
    assert i.cpu().tolist() == [[7, 6, 5, 4, 3, 2, 1, 0]]


# ---- lists ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("shape,n", [((0,), 3), ((1,), 1), ((1, 8), 64), ((5, 3), 2), ((700, 8), 256), ((65, 1), 1), ((9000,), 5), ((4099, 8), 16)])
def test_expert_lists(tq, shape, n):
    ids = torch.randint(-2, n + 2, shape, generator=gen(n), dtype=I32)
    want = bo.lists(ids, n)
    got = tq.expert_lists(ids.cuda(), n)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_expert_lists_extreme_ids(tq):
    ids = torch.tensor([2**31 - 1, -(2**31), 0, 65535, 65536, 1, 0], dtype=I32)
    order, offsets = tq.expert_lists(ids.cuda(), 65536)
    assert order.tolist() == [2, 6, 5, 3, 0, 1, 4]
    assert offsets[0] == 0 and offsets[1] == 2 and offsets[2] == 3 and offsets[65535] == 3 and offsets[65536] == 4


# ---- experts' products ---------------------------------------------------------------------------------------------

def experts_of(tq, seed, n, rows, cols):
    g = np.random.default_rng(seed)
    return torch.stack([tq.repack(torch.from_numpy(TI.pq2_matrix(g, rows, cols).reshape(-1)).cuda(), "pq2_0", rows, cols) for _ in range(n)])


EXPERTS = [
    # tokens, experts, k, rows, cols, own activations
    (1, 1, 1, 1, 256, False),
    (1, 8, 3, 65, 512, False),
    (2, 5, 5, 200, 768, True),
    (17, 4, 2, 64, 1280, False),
    (17, 3, 1, 130, 2304, True),
    (40, 2, 2, 96, 512, False),
    (90, 3, 3, 333, 256, False),
    (130, 2, 1, 1000, 1024, True),
    (300, 7, 4, 80, 512, False),
    (64, 64, 8, 48, 1024, False),
    (1, 64, 8, 2048, 5120, False),
    (100, 2, 1, 520, 5120, False),     # many pairs of one expert: 32 pairs and 256 rows at a time, four runs of five superchunks
    (70, 2, 1, 1030, 2304, True),      # runs of 3, 3 and 3, an odd last block
    (60, 1, 1, 3000, 1280, False),     # of 2, 2 and 1
    (20, 30, 3, 2600, 1536, False),    # few pairs each of many rows: several groups of row blocks per workgroup
    (12, 60, 6, 1500, 512, True),
]


@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("holes", [False, True])
def test_gemm_experts_equals_gemv(tq, case, holes):
    tokens, n, k, rows, cols, own = case
    r = gen(tokens + rows)
    w = experts_of(tq, tokens, n, rows, cols)
    ids = (torch.randn(tokens, n, generator=r) + torch.randn(n, generator=r)).topk(k, 1).indices.int()
    if holes:
        ids[torch.rand(ids.shape, generator=r) < 0.4] = -1
    x = torch.randn(tokens * k if own else tokens, cols, generator=r).cuda()
    q, d, bs = tq.quantize_q8k(x)
    pairs = tokens * k
    buf = torch.full((pairs + 2, rows), 7.0, device="cuda")
    flag = torch.zeros(1, dtype=I32, device="cuda")
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n), out=buf[1 : pairs + 1], bad_flag=flag)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all()) and flag.item() == 0
    flat = ids.flatten().tolist()
    for p in range(0, pairs, max(1, pairs // 40)):
        i = p if own else p // k
        want = torch.zeros(rows, device="cuda") if flat[p] < 0 else tq.gemv("pq2_0", w[flat[p]], rows, cols, q[i], d[i])
        assert torch.equal(y[p], want), f"pair {p}"
    again = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n))
    assert torch.equal(again, y)


def test_gemm_experts_against_the_oracle(tq, orc):
    rows, cols, n = 70, 512, 3
    g = np.random.default_rng(5)
    mats = [TI.pq2_matrix(g, rows, cols) for _ in range(n)]
    w = torch.stack([tq.repack(torch.from_numpy(m.reshape(-1)).cuda(), "pq2_0", rows, cols) for m in mats])
    x = torch.from_numpy(TI.activations(g, 9, cols))
    q, d, _ = tq.quantize_q8k(x.cuda())
    ids = torch.tensor([0, 2, 2, 1, 0, 0, 2, 1, 0], dtype=I32)
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n)).cpu().numpy().astype(np.float64)
    qo, do, _ = orc.quantize_q8k(x.numpy())
    for p, e in enumerate(ids.tolist()):
        want, size = orc.matmul("pq2_0", mats[e], qo[p : p + 1], do[p : p + 1], with_mag=True)
        bound = np.where(want[0] != 0, 1e-5 * np.abs(want[0]), 1e-5 * size[0])
        assert (np.abs(y[p] - want[0]) <= bound).all()


def test_gemm_experts_one_expert_for_all(tq):
    """As a prompt product: every pair with one expert of many."""
    w = experts_of(tq, 3, 6, 144, 1536)
    q, d, bs = tq.quantize_q8k(torch.randn(200, 1536, generator=gen(1)).cuda())
    for e in (0, 3, 5):
        ids = torch.full((200,), e, dtype=I32, device="cuda")
        y = tq.gemm_experts("pq2_0", w, 144, 1536, q, d, *tq.expert_lists(ids, 6))
        assert torch.equal(y, tq.gemm("pq2_0", w[e], 144, 1536, q, d, bs))


def test_gemm_experts_bad_lists(tq):
    """Numbers outside the pairs and offsets that leave the list are skipped and flagged; good pairs are right."""
    rows, cols, n = 64, 256, 2
    w = experts_of(tq, 4, n, rows, cols)
    q, d, _ = tq.quantize_q8k(torch.randn(4, cols, generator=gen(2)).cuda())

    def run(order, offsets):
        flag = torch.zeros(1, dtype=I32, device="cuda")
        out = torch.full((4, rows), 7.0, device="cuda")
        tq.gemm_experts("pq2_0", w, rows, cols, q, d, torch.tensor(order, dtype=I32).cuda(), torch.tensor(offsets, dtype=I32).cuda(), out=out, bad_flag=flag)
        return out, flag.item()

    y, flag = run([0, 99, -5, 3], [0, 2, 4])
    assert flag == 1 and torch.equal(y[0], tq.gemv("pq2_0", w[0], rows, cols, q[0], d[0])) and torch.equal(y[3], tq.gemv("pq2_0", w[1], rows, cols, q[3], d[3]))
    assert bool((y[1:3] == 7).all())
    for offsets in ([0, 1000, 4], [-7, 2, 4], [3, 1, 9], [2**31 - 1, -(2**31), 0]):
        assert run([0, 1, 2, 3], offsets)[1] == 1 or offsets == [3, 1, 4]


# ---- adapters ------------------------------------------------------------------------------------------------------

ADAPT = [
    # tokens, adapters, rank, cols, rows, x, weights, y
    (1, 1, 8, 8, 1, F32, BF, F32),
    (1, 4, 16, 5120, 300, F32, BF, F32),
    (3, 2, 24, 520, 77, BF, BF, BF),
    (17, 3, 16, 256, 260, HF, HF, HF),
    (40, 50, 32, 768, 129, F32, HF, F32),
    (64, 5, 64, 1000, 256, F32, BF, BF),
    (130, 2, 40, 512, 515, HF, HF, F32),
    (33, 3, 128, 264, 96, F32, BF, HF),
    (20, 2, 256, 2048, 64, BF, BF, F32),
    (1100, 3, 48, 136, 131, BF, BF, BF),
    (1030, 40, 80, 64, 70, F32, HF, F32),
    (300, 4, 72, 640, 192, F32, HF, HF),
]


@pytest.mark.parametrize("case", ADAPT, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("layout", ["plain", "views", "in place"])
def test_adapter_add(tq, case, layout):
    tokens, n, rank, cols, rows, xt, wt, yt = case
    r = gen(tokens + rows)
    x, y = torch.randn(tokens, cols, generator=r).to(xt), torch.randn(tokens, rows, generator=r).to(yt)
    a, b = (torch.randn(n, rank, cols, generator=r) * cols**-0.5).to(wt), (torch.randn(n, rows, rank, generator=r) * rank**-0.5).to(wt)
    index = torch.randint(-1, n, (tokens,), generator=r, dtype=I32)
    ranks = torch.randint(0, rank + 1, (n,), generator=r, dtype=I32) if layout != "plain" else None
    scale = torch.randn(n, generator=r) if layout != "in place" else None
    if ranks is not None:  # what lies behind an adapter's rank is not used
        if n > 1:
            ranks[0], ranks[1] = rank, rank // 2 + 1
        for i in range(n):
            a[i, ranks[i] :] = math.nan
            b[i, :, ranks[i] :] = math.inf
    want, size = bo.adapter(y, x, a, b, index, ranks, scale)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx, dy = x.cuda(), y.cuda()
    out = None
    if layout == "views":  # rows of wider tensors, every second row of the output, at odd places
        dx = torch.full((tokens, cols + 16), math.nan, dtype=xt, device="cuda")[:, 8 : cols + 8].copy_(x)
        dy = torch.full((tokens, rows + 3), math.nan, dtype=yt, device="cuda")[:, 1 : rows + 1].copy_(y)
        buf = torch.full((tokens, 2, rows + 1), 7.0, dtype=yt, device="cuda")
        out = buf[:, 0, 1:]
    flag = torch.zeros(1, dtype=I32, device="cuda")
    got = tq.adapter_add(dy, dx, a.cuda(), b.cuda(), index.cuda(), ranks=cuda(ranks), scale=cuda(scale), out=out, bad_flag=flag)
    near(got, want, bo.adapter_bound(want, size, cols, rank, yt), layout)
    assert flag.item() == 0
    if layout == "views":
        assert bool((buf[:, 1] == 7).all()) and bool((buf[:, 0, 0] == 7).all())
    elif layout == "plain":
        assert got is dy


def test_adapter_add_keeps_the_bits_of_fp32(tq):
    """Adapters that pick columns: every bit of x arrives, and tokens without an adapter keep theirs."""
    cols, rows = 64, 64
    x = (torch.randint(2**23, 2**24, (20, cols), generator=gen(3)).float() * 2.0**-23) * torch.where(torch.rand(20, cols, generator=gen(4)) < 0.5, -1.0, 1.0)
    a, b = torch.zeros(2, 64, cols), torch.zeros(2, rows, 64)
    perm = torch.randperm(64, generator=gen(5))
    a[0, torch.arange(64), perm] = 1.0
    b[0, torch.arange(64), torch.arange(64)] = 1.0
    a[1], b[1] = a[0] * (1 + 2.0**-7), b[0]
    index = torch.arange(20, dtype=I32) % 3 - 1
    for wt, one in ((BF, 1 + 2.0**-7), (HF, 1 + 2.0**-10)):
        a[1] = a[0] * one
        y = torch.zeros(20, rows)
        y[0] = -0.0
        got = tq.adapter_add(y.cuda(), x.cuda(), a.to(wt).cuda(), b.to(wt).cuda(), index.cuda(), out=torch.empty(20, rows, device="cuda")).cpu()
        assert torch.equal(got[index == 0], x[index == 0][:, perm])
        want = x[index == 1][:, perm].double() * one
        assert bool(((got[index == 1].double() - want).abs() <= 4 * 2.0**-24 * want.abs()).all())  # its 32 or more bits in fp32 sums: four roundings
        assert torch.equal(got[index == -1], y[index == -1]) and bool(torch.signbit(got[0]).all())


def test_adapter_add_not_finite_stays_with_its_token(tq):
    r = gen(6)
    x, y = torch.randn(20, 128, generator=r), torch.randn(20, 70, generator=r)
    a, b = torch.randn(1, 8, 128, generator=r).to(BF).cuda(), torch.randn(1, 70, 8, generator=r).to(BF).cuda()
    index = torch.zeros(20, dtype=I32, device="cuda")
    good = tq.adapter_add(y.cuda(), x.cuda(), a, b, index, out=torch.empty(20, 70, device="cuda"))
    x[3, 5], x[7, 100], x[11, 0] = math.nan, math.inf, 3e38
    got = tq.adapter_add(y.cuda(), x.cuda(), a, b, index, out=torch.empty(20, 70, device="cuda"))
    ok = torch.ones(20, dtype=torch.bool)
    ok[[3, 7, 11]] = False
    assert torch.equal(got[ok.cuda()], good[ok.cuda()])
    assert not bool(got[3].isfinite().any()) and not bool(got[7].isfinite().any())


def test_adapter_add_index_outside(tq):
    y = torch.randn(4, 16, generator=gen(7)).cuda()
    x = torch.randn(4, 8, generator=gen(8)).cuda()
    a, b = torch.ones(2, 8, 8, dtype=BF, device="cuda"), torch.ones(2, 16, 8, dtype=BF, device="cuda")
    flag = torch.zeros(1, dtype=I32, device="cuda")
    index = torch.tensor([0, 2, -1, 2**31 - 1], dtype=I32, device="cuda")
    got = tq.adapter_add(y, x, a, b, index, out=torch.empty_like(y), bad_flag=flag)
    assert flag.item() == 1 and torch.equal(got[1:], y[1:]) and not torch.equal(got[0], y[0])
    flag.zero_()
    tq.adapter_add(y, x, a, b, index.clamp(max=1), bad_flag=flag)
    assert flag.item() == 0


# ---- sampling ------------------------------------------------------------------------------------------------------

def sample_all(tq, x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    rows = x.shape[0]
    logprob = torch.empty(rows, device="cuda")
    got = tq.sample(x.cuda(), u.cuda(), temperature=cuda(temperature), top_k=cuda(top_k), top_p=cuda(top_p), min_p=cuda(min_p), logprob=logprob)
    at = lambda t, i, off: off if t is None else float(t[i])  # noqa: E731
    want = [bo.sample(x[i].double(), float(u[i]), at(temperature, i, 1.0), int(at(top_k, i, 0)), at(top_p, i, 1.0), at(min_p, i, 0.0)) for i in range(rows)]
    assert got.cpu().tolist() == [w[0] for w in want]
    lp = torch.tensor([w[1] for w in want], dtype=torch.float64)
    assert bool((lp.isinf() == logprob.cpu().isinf()).all())
    fine = lp.isfinite()
    # one rounding; the weights' own are 2^-44 of the largest each
    near(logprob.cpu()[fine], lp[fine], lp[fine].abs() * 2.0**-24 * 1.01 + x.shape[1] * 2.0**-44, "logprob")
    return got


def logits_of(rows, vocab, dt, seed, std=2.0):
    r = gen(seed)
    x = torch.randn(rows, vocab, generator=r) * std
    x.scatter_add_(1, torch.randint(0, vocab, (rows, 5), generator=r), torch.rand(rows, 5, generator=r) * 10)
    return x.to(dt)


@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 1000, 1024, 1025, 4099, 20_000, 65_537, 150_001])
@pytest.mark.parametrize("dt", [F32, BF, HF])
def test_sample(tq, vocab, dt):
    rows = 16
    r = gen(vocab)
    x, u = logits_of(rows, vocab, dt, vocab + 1), torch.rand(rows, generator=r)
    pick = lambda values: torch.tensor(values)[torch.randint(0, len(values), (rows,), generator=r)]  # noqa: E731
    t = pick([0.0, 0.5, 1.0, 1.3, 5.0])
    k, p, m = pick([0, 1, 2, 40, 1000, vocab, vocab + 5]).int(), pick([1.0, 0.999, 0.9, 0.5, 0.01]), pick([0.0, 0.001, 0.1, 1.0])
    sample_all(tq, x, u)
    sample_all(tq, x, u, t)
    sample_all(tq, x, u, t, top_k=k)
    sample_all(tq, x, u, None, top_p=p)
    sample_all(tq, x, u, t, min_p=m)
    sample_all(tq, x, u, t, k, p, m)
    wide = torch.full((rows, vocab + 7), math.nan, dtype=dt)
    wide[:, 3 : vocab + 3] = x
    got = tq.sample(wide.cuda()[:, 3 : vocab + 3], u.cuda(), temperature=t.cuda(), top_k=k.cuda(), top_p=p.cuda(), min_p=m.cuda())
    assert torch.equal(got, tq.sample(x.cuda(), u.cuda(), temperature=t.cuda(), top_k=k.cuda(), top_p=p.cuda(), min_p=m.cuda()))


@pytest.mark.parametrize("vocab", [10, 3000, 70_000])
def test_sample_equal_logits(tq, vocab):
    """Everything ties: the first ones by index stay, and are drawn evenly."""
    rows = 12
    x = torch.full((rows, vocab), -3.5)
    x[1::2] = 0.0
    x[1::4, ::2] = -0.0  # equal to +0
    u = torch.linspace(0, 1 - 2.0**-24, rows)
    k = torch.tensor([1, 2, 3, 7] * 3, dtype=I32)
    sample_all(tq, x, u, top_k=k)
    p = torch.tensor([0.5, 0.25, 0.3, 0.99] * 3)
    sample_all(tq, x, u, top_p=p)
    sample_all(tq, x, u, torch.full((rows,), 1e30), k * 3, p, torch.full((rows,), 1.0))
    few = x.bfloat16()
    few[:, vocab // 2 :] -= 1  # two values
    sample_all(tq, few, u, top_p=p)
    sample_all(tq, few, u, top_k=k + vocab // 2)


def test_sample_masks_and_infinities(tq):
    x = logits_of(10, 5000, F32, 3)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, :-1] = -math.inf
    x[4, ::2] = -math.inf
    x[5, 7], x[5, 4321] = math.inf, math.inf
    x[6, 100:] = math.nan
    x[7] = -3.4e38
    x[7, 9] = 3.4e38
    x[8] = torch.randn(5000, generator=gen(9)) * 1e-30
    u = torch.full((10,), 0.6)
    k = torch.tensor([0, 5, 5, 5, 3000, 5, 500, 3, 2000, 7], dtype=I32)
    p = torch.full((10,), 0.8)
    for t in (None, torch.zeros(10), torch.full((10,), 1e-30), torch.full((10,), 1e30)):
        sample_all(tq, x, u, t)
        sample_all(tq, x, u, t, top_k=k)
        sample_all(tq, x, u, t, top_p=p)
        sample_all(tq, x, u, t, k, p, torch.full((10,), 0.3))


def test_sample_parameters_out_of_range(tq):
    x = logits_of(8, 2000, F32, 5)
    u = torch.tensor([-1.0, 0.0, 1.0, 2.0, math.nan, math.inf, 0.5, 0.5])
    clean = torch.tensor([0.0, 0.0, 1.0, 1.0, 0.0, 1.0, 0.5, 0.5])
    one = lambda v: torch.full((8,), v)  # noqa: E731
    for arg, want in ((dict(), dict()), (dict(top_k=one(-4).int()), dict()), (dict(top_p=one(math.nan)), dict()), (dict(top_p=one(7.0)), dict()),
                      (dict(top_p=one(-1.0)), dict(top_k=one(1).int())), (dict(min_p=one(math.nan)), dict()), (dict(min_p=one(-2.0)), dict()),
                      (dict(min_p=one(9.0)), dict(min_p=one(1.0))), (dict(temperature=one(-1.0)), dict(temperature=one(0.0))),
                      (dict(temperature=one(math.nan)), dict(temperature=one(0.0)))):
        got = tq.sample(x.cuda(), u.cuda(), **{a: v.cuda() for a, v in arg.items()})
        assert torch.equal(got, sample_all(tq, x, clean, **want)), arg


def test_sample_shares(tq):
    """Even random numbers give every token its share."""
    x = torch.log(torch.tensor([1.0, 2.0, 3.0, 4.0, 6.0])).repeat(1600, 1)
    u = (torch.arange(1600) + 0.5) / 1600
    got = torch.bincount(tq.sample(x.cuda(), u.cuda()).cpu(), minlength=5)
    assert got.tolist() == [100, 200, 300, 400, 600]
