"""The operators of a mixed batch at the ends of their ranges: temperatures without measure, random numbers at the borders, scales and
inputs next to infinity, lists that decrease, and workspaces of exactly a larger call's size."""
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


def rows_match(tq, x, u, **params):
    got = tq.sample(x.cuda(), u.cuda(), **{k: v.cuda() for k, v in params.items()}).cpu()
    off = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    want = [bo.sample(x[i].double(), float(u[i]), *(params[k][i].item() if k in params else v for k, v in off.items())) for i in range(x.shape[0])]
    assert got.tolist() == [w[0] for w in want]


# ---- temperatures without an end -----------------------------------------------------------------------------------

@pytest.mark.parametrize("vocab", [40, 3000, 5 * 4096, 70_000])
@pytest.mark.parametrize("dt", [F32, BF, HF])
def test_sample_at_infinite_temperature(tq, vocab, dt):
    """All finite logits weigh the same, and nothing beside one of +inf, which lies in one slice, in several or in none."""
    r = gen(vocab)
    rows = 8
    x = torch.randn(rows, vocab, generator=r) * 4
    x[1, vocab // 2] = math.inf
    x[2, :: vocab // 4] = math.inf
    x[3, 0] = x[3, -1] = math.inf
    x[4] = math.inf
    x[5, : vocab // 2] = -math.inf
    x[6, ::3] = torch.finfo(dt).max
    x[6, 1::3] = torch.finfo(dt).min
    x[7, 5:] = math.nan
    x = x.to(dt)
    u = torch.rand(rows, generator=r)
    t = torch.full((rows,), math.inf)
    k = torch.full((rows,), 3, dtype=I32)
    many = torch.full((rows,), vocab // 2, dtype=I32)
    p, m = torch.full((rows,), 0.7), torch.tensor([1.0, 0.5] * (rows // 2))
    for params in (dict(), dict(top_k=k), dict(top_k=many), dict(top_p=p), dict(min_p=m), dict(top_k=many, top_p=p, min_p=m)):
        rows_match(tq, x, u, temperature=t, **params)
    # in one launch with others
    mixed = torch.tensor([math.inf, 1.0, 0.0, math.inf, 1e30, 1e-30, math.inf, 0.5])
    rows_match(tq, x, u, temperature=mixed, top_k=k, top_p=p, min_p=m)


# ---- min_p where bins do not measure z -----------------------------------------------------------------------------

@pytest.mark.parametrize("vocab", [300, 3000, 20_000])
@pytest.mark.parametrize("t", [1e-30, 6e-30, 7e-30, 1e-32, 1e-36])
def test_sample_min_p_at_small_temperatures(tq, t, vocab):
    """Twenty tokens that pass min_p, and all others below it with a weight that would move the draw."""
    r = gen(vocab)
    rows = 48
    z = -1.4 - 3.5 * torch.rand(rows, vocab, generator=r)
    some = torch.rand(rows, vocab, generator=r).argsort(1)[:, :20]
    z.scatter_(1, some, -1.1 * torch.rand(rows, 20, generator=r))
    z.scatter_(1, some[:, :1], 0.0)
    x = (z.double() * t).float()
    u = (torch.arange(rows) + 0.5) / rows
    params = dict(temperature=torch.full((rows,), t), min_p=torch.full((rows,), 0.3))
    rows_match(tq, x, u, **params)
    rows_match(tq, x, u, **params, top_p=torch.full((rows,), 0.99))
    rows_match(tq, x, u, **params, top_k=torch.full((rows,), 30, dtype=I32))


@pytest.mark.parametrize("bins", [3, 48, 200, 500])
def test_sample_min_p_at_far_negative_logits(tq, bins):
    """The largest logit lies `bins` eighths of z above where bins end, at -2^23 eighths."""
    r = gen(bins)
    rows, vocab, t = 48, 3000, 1e-4
    best = -(2.0**23 - bins) / 8 * t
    low = min(bins / 8 + 1, 8.0)
    z = -low - 0.2 - 2 * torch.rand(rows, vocab, generator=r)
    some = torch.rand(rows, vocab, generator=r).argsort(1)[:, :20]
    z.scatter_(1, some, -(low - 0.2) * torch.rand(rows, 20, generator=r))
    z.scatter_(1, some[:, :1], 0.0)
    x = (best + z.double() * t).float()  # (z in steps of 0.08)
    u = (torch.arange(rows) + 0.5) / rows
    rows_match(tq, x, u, temperature=torch.full((rows,), t), min_p=torch.full((rows,), math.exp(-low)))


# ---- what weighs nothing is not drawn ------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("low", [-30.0, -31.0, -31.75, -33.0])
def test_sample_slices_that_weigh_nothing(tq, low, dt):
    """The first and the last slices hold one token `low` below the largest and nothing else.  Tokens below 2^-44 of the largest
    (z = -30.5) weigh nothing, wherever the row is cut."""
    vocab = 5 * 4096
    x = torch.full((vocab,), -200.0)
    x[[10, 4096 + 20, 3 * 4096 + 30, vocab - 5]] = low
    x[2 * 4096 + torch.arange(3) * 1000] = torch.tensor([-1.0, 0.0, -2.0])
    u = torch.tensor([0.0, -1.0, math.nan, -math.inf, 1.0, 2.0, math.inf])
    first, last = (10, vocab - 5) if low > -30.5 else (2 * 4096, 2 * 4096 + 2000)
    want = torch.tensor([first] * 4 + [last] * 3, dtype=I32)
    n = len(u)
    full = lambda v, t=F32: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    for params in (dict(), dict(temperature=full(1.0)), dict(top_k=full(7, I32)), dict(top_k=full(6000, I32)), dict(min_p=full(1e-30))):
        logprob = torch.empty(n, device="cuda")
        got = tq.sample(x.to(dt).repeat(n, 1).cuda(), u.cuda(), logprob=logprob, **params).cpu()
        assert torch.equal(got, want), params
        assert bool(logprob.isfinite().all())
    cold = (x * 0.25).to(dt).repeat(n, 1).cuda()
    assert torch.equal(tq.sample(cold, u.cuda(), temperature=full(0.25)).cpu(), want)


# ---- adapters next to infinity -------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [3, 200, 2048])
@pytest.mark.parametrize("wt", [BF, HF])
def test_adapter_add_of_the_largest_floats(tq, tokens, wt):
    """fp32 values above bf16's largest are finite, in x and in A x."""
    big = torch.finfo(F32).max
    assert big > torch.finfo(BF).max
    r = gen(tokens)
    x, a, b = torch.randn(tokens, 64, generator=r), torch.zeros(2, 8, 64), torch.randn(2, 40, 8, generator=r) * 2.0**-10
    x[:, 3], x[:, 17] = big, -big * (1 - torch.rand(tokens, generator=r) * 2.0**-9)
    a[0, 0, 3], a[0, 1, 17], a[0, 2, 5] = 1.0, -1.0, 1.0
    a[1, 0, 3], a[1, 5, 17] = 2.0**-14, 1.5 * 2.0**-12
    a, b = a.to(wt), b.to(wt)
    index = torch.arange(tokens, dtype=I32) % 3 - 1
    y = torch.randn(tokens, 40, generator=r)
    got = tq.adapter_add(y.cuda(), x.cuda(), a.cuda(), b.cuda(), index.cuda()).double().cpu()
    want, size = bo.adapter(y, x, a, b, index, None, None)
    assert bool(want.isfinite().all()) and float(want.abs().max()) < big
    assert bool(((got - want).abs() <= bo.adapter_bound(want, size, 64, 8, F32)).all())


# ---- experts: scales that are not finite ---------------------------------------------------------------------------

@pytest.mark.parametrize("cols", [256, 768, 1280, 1536, 2304])
@pytest.mark.parametrize("tokens,k,n", [(90, 1, 2), (50, 1, 1), (9, 2, 4), (60, 2, 3)])
def test_gemm_experts_scales_that_are_not_finite(tq, tokens, k, n, cols):
    """A block's scale of infinity or NaN gives what the product gives."""
    g = np.random.default_rng(cols + tokens)
    rows = 70
    w = torch.stack([tq.repack(torch.from_numpy(TI.pq2_matrix(g, rows, cols).reshape(-1)).cuda(), "pq2_0", rows, cols) for _ in range(n)])
    q, d, _ = tq.quantize_q8k(torch.randn(tokens, cols, generator=gen(tokens)).cuda())
    for t in range(0, tokens, 3):
        d[t, (t // 3) % (cols // 256)] = (math.inf, -math.inf, math.nan)[t // 3 % 3]
    d[0, -1] = math.inf
    ids = torch.stack([torch.randperm(n, generator=gen(t))[:k] for t in range(tokens)]).int()
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n)).view(tokens, k, rows)
    for t in range(tokens):
        for j in range(k):
            want = tq.gemv("pq2_0", w[ids[t, j]], rows, cols, q[t], d[t])
            assert torch.equal(y[t, j].nan_to_num(7.0, 1e30, -1e30), want.nan_to_num(7.0, 1e30, -1e30)), (t, j)
    assert bool(y[0].isinf().any())


# ---- experts: lists that decrease ----------------------------------------------------------------------------------

@pytest.mark.parametrize("pairs,n,offsets", [(4, 2, [0, 3, 1]), (4, 2, [3, 1, 4]), (4, 2, [0, 5, 4]), (4, 2, [-1, 2, 4]), (4, 2, [0, 2, 5]), (100, 2, [0, 90, 20]),
                                             (100, 1, [60, 40]), (100, 1, [0, 101])])
def test_gemm_experts_flags_lists(tq, pairs, n, offsets):
    """Few pairs and many pairs per expert; the same call with a good list raises nothing."""
    rows, cols = 64, 256
    w = torch.stack([tq.repack(torch.from_numpy(TI.pq2_matrix(np.random.default_rng(i), rows, cols).reshape(-1)).cuda(), "pq2_0", rows, cols) for i in range(n)])
    q, d, _ = tq.quantize_q8k(torch.randn(pairs, cols, generator=gen(pairs)).cuda())
    ints = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    order = torch.arange(pairs, dtype=I32, device="cuda")
    guard = torch.full((pairs + 2, rows), 7.0, device="cuda")
    for lists, want in ((offsets, 1), (sorted(min(max(o, 0), pairs) for o in offsets), 0), ([0] * (n + 1), 0), ([pairs] * (n + 1), 0)):
        flag = ints([0])
        tq.gemm_experts("pq2_0", w, rows, cols, q, d, order, ints(lists), out=guard[1:-1], bad_flag=flag)
        assert flag.item() == want, lists
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())


@pytest.mark.parametrize("pairs", [5, 4000])
@pytest.mark.parametrize("at", [1, 77, 350, 699, 700])
def test_gemm_experts_flags_a_hidden_decrease(tq, pairs, at):
    """One offset of 701 is off, wherever the search for a slot looks."""
    n, rows, cols = 700, 64, 256
    w = torch.zeros(n, tq.repacked_bytes("pq2_0", rows, cols), dtype=torch.uint8, device="cuda")
    q, d, _ = tq.quantize_q8k(torch.randn(pairs, cols, generator=gen(at)).cuda())
    good = bo.lists(torch.randint(0, n, (pairs,), generator=gen(pairs + at), dtype=I32), n)
    for value, want in ((None, 0), (-1, 1), (pairs + 1, 1), (0, 1)):
        order, offsets = good[0].cuda(), good[1].clone()
        if value is not None:
            offsets[at] = value
            offsets[at - 1] = max(1, int(offsets[at - 1]))  # (so that 0 is a decrease)
        flag = torch.zeros(1, dtype=I32, device="cuda")
        tq.gemm_experts("pq2_0", w, rows, cols, q, d, order, offsets.cuda(), bad_flag=flag)
        assert flag.item() == want, value


# ---- workspaces of a larger call's size ----------------------------------------------------------------------------

@pytest.mark.parametrize("most,n,rank,cols", [(7000, 5, 64, 5120), (1500, 24, 32, 5120), (1696, 4, 64, 5120), (64, 9, 256, 2048)])
def test_adapter_workspace_serves_smaller_batches(tq, most, n, rank, cols):
    r = gen(most)
    need = tq.adapter_workspace_bytes(most, n, rank, cols)
    guard = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    ws = guard[:need]
    a, b = torch.randn(n, rank, cols, generator=r).to(BF).cuda(), torch.randn(n, 24, rank, generator=r).to(BF).cuda()
    x, y = torch.randn(most, cols, generator=r).to(BF).cuda(), torch.randn(most, 24, generator=r).cuda()
    index = torch.randint(-1, n, (most,), generator=r, dtype=I32).cuda()
    for tokens in sorted({1, 17, 64, 65, 1375, 1695, 2047, 2048, 6000, most}):
        if tokens > most:
            continue
        for adapters in (n, 1):
            i = index[:tokens].clamp(max=adapters - 1)
            args = (y[:tokens], x[:tokens], a[:adapters], b[:adapters], i)
            got = tq.adapter_add(*args, out=torch.empty_like(y[:tokens]), ws=ws)
            assert torch.equal(got, tq.adapter_add(*args, out=torch.empty_like(y[:tokens]))), tokens
    assert bool((guard[need:] == 171).all())


@pytest.mark.parametrize("most", [270_000, 540_000])
def test_sample_workspace_serves_smaller_vocabularies(tq, most):
    r = gen(most)
    need = tq.sample_workspace_bytes(3, most)
    guard = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    x, u, p = torch.randn(3, most, generator=r).cuda(), torch.rand(3, generator=r).cuda(), torch.full((3,), 0.9, device="cuda")
    for vocab in (1, 5000, 260_000, 266_233, 266_234, 530_000, most):
        if vocab <= most:
            got = tq.sample(x[:, :vocab], u, top_p=p, out=torch.empty(3, dtype=I32, device="cuda"), ws=guard[:need])
            assert torch.equal(got, tq.sample(x[:, :vocab], u, top_p=p)), vocab
    assert bool((guard[need:] == 171).all())


# ---- routing: the type's lowest values -----------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF, HF])
def test_route_of_the_lowest_logits(tq, dt):
    """Logits of a mask that is the type's lowest value are logits: the lowest experts share a softmax equally.  Sigmoids of them are
    0 in fp64 (fp32, bf16), and so are the weights."""
    low = torch.finfo(dt).min
    x = torch.full((2, 70), low, dtype=dt)
    x[1, 40] = 3.0
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(70)):
            for renorm in (False, True):
                want = bo.route(x, 4, score, bias, 1, 1, 1, renorm, 1.0)
                w, i = tq.route(x.cuda(), 4, score=score, bias=None if bias is None else bias.cuda(), renorm=renorm)
                assert torch.equal(i.cpu(), want[1]) and i.cpu().tolist() == [[0, 1, 2, 3], [40, 0, 1, 2]]
                assert bool(((w.cpu().double() - want[0]).abs() <= want[0] * 2.0**-24 * 1.001).all()) and bool(w.isfinite().all())
