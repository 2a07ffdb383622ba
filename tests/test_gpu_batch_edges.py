"""The operators of a mixed batch as they are used and at their ends: together, in graphs, on other streams, with used
workspaces, at the sizes where their kernels change, and where offsets pass 32 bits."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import batch_oracle as bo
import tq_inputs as TI

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def example():
    spec = importlib.util.spec_from_file_location("mixed_batch", os.path.join(ROOT, "examples", "mixed_batch.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_operators_together(tq):
    """A step of 70 requests at once and one by one: each value of a product may move by a step of the quantization."""
    (h, tokens, logprob), (h1, tokens1, logprob1) = example().run(70)
    assert float((h - h1).norm() / h1.norm()) < 4 / 127
    assert bool((tokens >= 0).all()) and bool((tokens < 4000).all()) and bool((logprob <= 0).all()) and bool(logprob.isfinite().all())
    assert int((tokens != tokens1).sum()) <= 35  # (those that move next to a border)


def test_one_graph_of_all(tq):
    """Routing, lists, experts, an adapter and sampling captured together; each replay on new inputs equals the eager calls."""
    m = example()
    model, n = m.Model(3), 20
    static = list(m.requests(n, 3))
    ws = {"a": tq.adapter_workspace(n, m.ADAPTERS, m.RANK, m.HIDDEN), "s": tq.sample_workspace(n, m.VOCAB)}
    out = {"y": torch.empty(n, m.HIDDEN, device="cuda"), "route": (torch.empty(n, 2, device="cuda"), torch.empty(n, 2, dtype=I32, device="cuda")),
           "lists": (torch.empty(2 * n, dtype=I32, device="cuda"), torch.empty(m.EXPERTS + 1, dtype=I32, device="cuda")),
           "up": torch.empty(2 * n, 2 * m.INNER, device="cuda"), "tokens": torch.empty(n, dtype=I32, device="cuda"), "logprob": torch.empty(n, device="cuda")}
    logits = torch.randn(n, m.VOCAB, generator=gen(1)).cuda()

    def step():
        x, adapter, u, t, k, p, mp = static
        tq.adapter_add(x, x, model.a, model.b, adapter, ranks=model.ranks, scale=model.scale, out=out["y"], ws=ws["a"])
        tq.route(out["y"][:, : m.EXPERTS], 2, bias=model.bias, out=out["route"])
        tq.expert_lists(out["route"][1], m.EXPERTS, out=out["lists"])
        q, d, _ = tq.quantize_q8k(out["y"])
        tq.gemm_experts("pq2_0", model.up, 2 * m.INNER, m.HIDDEN, q, d, *out["lists"], out=out["up"])
        tq.sample(logits, u, temperature=t, top_k=k, top_p=p, min_p=mp, out=out["tokens"], logprob=out["logprob"], ws=ws["s"])
        return [out["y"], *out["route"], *out["lists"], out["up"], out["tokens"], out["logprob"]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        for to, new in zip(static, m.requests(n, 10 + seed)):
            to.copy_(new)
        logits.copy_(torch.randn(n, m.VOCAB, generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out["y"], *out["route"], *out["lists"], out["up"], out["tokens"], out["logprob"])]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_other_streams(tq):
    """Two streams at once, each with workspaces of its own, and a wait before the results are used."""
    r = gen(2)
    x, u = torch.randn(8, 30_000, generator=r).cuda(), torch.rand(8, generator=r).cuda()
    p = torch.full((8,), 0.9, device="cuda")
    y, z = torch.randn(100, 300, generator=r).cuda(), torch.randn(100, 512, generator=r).cuda()
    a, b = torch.randn(3, 16, 512, generator=r).to(BF).cuda(), torch.randn(3, 300, 16, generator=r).to(BF).cuda()
    index = torch.randint(-1, 3, (100,), generator=r, dtype=I32).cuda()
    want = tq.sample(x, u, top_p=p), tq.adapter_add(y, z, a, b, index, out=torch.empty_like(y))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        ws = tq.sample_workspace(8, 30_000), tq.adapter_workspace(100, 3, 16, 512)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            out = torch.empty(8, dtype=I32, device="cuda"), torch.empty_like(y)
            for _ in range(20):
                tq.sample(x, u, top_p=p, out=out[0], ws=ws[0])
                tq.adapter_add(y, z, a, b, index, out=out[1], ws=ws[1])
            got.append((out, ws))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for out, _ in got:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_used_workspaces(tq):
    """Workspaces need no clearing, and a larger one serves smaller calls and other shapes."""
    r = gen(4)
    ws = torch.full((max(tq.sample_workspace_bytes(40, 200_000), tq.adapter_workspace_bytes(2100, 7, 64, 1024)),), 255, dtype=torch.uint8, device="cuda")
    for rows, vocab in ((40, 200_000), (3, 500), (40, 200_000), (1, 70_000), (17, 9_000)):
        x, u, k = torch.randn(rows, vocab, generator=r).cuda(), torch.rand(rows, generator=r).cuda(), torch.full((rows,), 30, dtype=I32, device="cuda")
        p = torch.full((rows,), 0.8, device="cuda")
        args = dict(top_k=k, top_p=p, out=torch.empty(rows, dtype=I32, device="cuda"))
        first = tq.sample(x, u, **args, ws=ws).clone()
        assert torch.equal(first, tq.sample(x, u, top_k=k, top_p=p)) and torch.equal(first, tq.sample(x, u, **args, ws=ws))
    for tokens in (2100, 2, 64, 65, 2047, 2048):
        y, x = torch.randn(tokens, 90, generator=r).cuda(), torch.randn(tokens, 1024, generator=r).cuda()
        a, b = torch.randn(7, 64, 1024, generator=r).to(HF).cuda(), torch.randn(7, 90, 64, generator=r).to(HF).cuda()
        index = torch.randint(-1, 7, (tokens,), generator=r, dtype=I32).cuda()
        out = [tq.adapter_add(y, x, a, b, index, out=torch.empty_like(y), ws=w) for w in (ws, ws, None)]
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
        ws.fill_(255)


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 63, 64, 65, 129, 1025, 2047, 2048, 2049])
@pytest.mark.parametrize("n", [1, 70])
def test_adapter_add_where_kernels_change(tq, tokens, n):
    r = gen(tokens + n)
    x, y = torch.randn(tokens, 72, generator=r), torch.randn(tokens, 33, generator=r)
    a, b = torch.randn(n, 24, 72, generator=r).to(BF), torch.randn(n, 33, 24, generator=r).to(BF)
    index = torch.randint(-1, n, (tokens,), generator=r, dtype=I32)
    index[: tokens // 2] = n - 1  # an adapter with many
    ranks = torch.randint(0, 25, (n,), generator=r, dtype=I32)
    ranks[-1] = 24
    got = tq.adapter_add(y.cuda(), x.cuda(), a.cuda(), b.cuda(), index.cuda(), ranks=ranks.cuda()).double().cpu()
    want, size = bo.adapter(y, x, a, b, index, ranks, None)
    assert bool(((got - want).abs() <= bo.adapter_bound(want, size, 72, 24, F32)).all())


def test_adapter_add_of_many_adapters(tq):
    r = gen(11)
    n, tokens = 3000, 200
    x, y = torch.randn(tokens, 64, generator=r), torch.randn(tokens, 40, generator=r)
    a, b = torch.randn(n, 8, 64, generator=r).to(BF), torch.randn(n, 40, 8, generator=r).to(BF)
    index = torch.randint(0, n, (tokens,), generator=r, dtype=I32)
    got = tq.adapter_add(y.cuda(), x.cuda(), a.cuda(), b.cuda(), index.cuda()).double().cpu()
    want, size = bo.adapter(y, x, a, b, index, None, None)
    assert bool(((got - want).abs() <= bo.adapter_bound(want, size, 64, 8, F32)).all())


def test_gemm_experts_of_many_experts(tq):
    g = np.random.default_rng(6)
    n, rows, cols = 700, 64, 256
    one = tq.repack(torch.from_numpy(TI.pq2_matrix(g, n * rows, cols).reshape(-1)).cuda(), "pq2_0", n * rows, cols)
    w = one.view(n, -1)  # 64 rows are one tile: the stacked matrices are one matrix
    q, d, bs = tq.quantize_q8k(torch.randn(5, cols, generator=gen(6)).cuda())
    whole = tq.gemm("pq2_0", one, n * rows, cols, q, d, bs).view(5, n, rows)
    ids = torch.randint(0, n, (5, 6), generator=gen(7), dtype=I32)
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n)).view(5, 6, rows)
    for t in range(5):
        assert torch.equal(y[t], whole[t, ids[t].long().cuda()])


@pytest.mark.parametrize("rows,cols", [(1, 256), (17, 1280), (64, 1024), (100, 2304), (257, 512), (300, 5120), (700, 1024)])
@pytest.mark.parametrize("tokens,k,n", [(40, 1, 1), (41, 1, 1), (81, 1, 2), (60, 2, 3), (61, 2, 3), (200, 3, 3), (48, 8, 64)])
def test_gemm_experts_where_kernels_change(tq, rows, cols, tokens, k, n):
    """Every pair, bit for bit, at the sides of the rules that choose a kernel."""
    g = np.random.default_rng(rows + cols + tokens)
    w = torch.stack([tq.repack(torch.from_numpy(TI.pq2_matrix(g, rows, cols).reshape(-1)).cuda(), "pq2_0", rows, cols) for _ in range(n)])
    q, d, bs = tq.quantize_q8k(torch.randn(tokens, cols, generator=gen(tokens)).cuda())
    ids = torch.stack([torch.randperm(n, generator=gen(t))[:k] for t in range(tokens)]).int()
    ids[torch.rand(tokens, k, generator=gen(1)) < 0.02] = -1
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n)).view(tokens, k, rows)
    whole = torch.stack([tq.gemm("pq2_0", w[e], rows, cols, q, d, bs) for e in range(n)] + [torch.zeros(tokens, rows, device="cuda")])
    at = torch.where(ids < 0, n, ids).long().cuda()
    assert torch.equal(y, whole[at, torch.arange(tokens, device="cuda")[:, None]])


def rows_match(tq, x, u, **params):
    got = tq.sample(x.cuda(), u.cuda(), **{k: v.cuda() for k, v in params.items()}).cpu()
    off = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    want = [bo.sample(x[i].double(), float(u[i]), *(params[k][i].item() if k in params else v for k, v in off.items())) for i in range(x.shape[0])]
    assert got.tolist() == [w[0] for w in want]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("vocab", [30_000, 150_003])
def test_sample_flat_rows(tq, dt, vocab):
    """More tokens next to the cuts than the lists hold: the whole row is searched."""
    r = gen(vocab)
    rows = 6
    x = (torch.randn(rows, vocab, generator=r) * 1e-3 + 2).to(dt)
    u = torch.rand(rows, generator=r)
    k, p = torch.tensor([1, 5_000, 20_000, 29_999, 0, 777], dtype=I32), torch.tensor([0.5, 0.1, 0.99, 0.7, 0.3, 1.0])
    m = torch.tensor([0.0, 0.999, 0.5, 0.9985, 1.0, 0.9999])
    rows_match(tq, x, u, top_k=k)
    rows_match(tq, x, u, top_p=p)
    rows_match(tq, x, u, top_k=k, top_p=p)
    rows_match(tq, x, u, min_p=m, top_p=p)
    rows_match(tq, x, u, temperature=torch.full((rows,), 50.0), top_k=k, top_p=p, min_p=m)


def test_sample_large_logits(tq):
    """Logits over temperature beyond what the bins tell apart."""
    r = gen(21)
    x, u = torch.randn(6, 4000, generator=r) * torch.tensor([1e3, 1e5, 1e7, 1e20, 1e-20, 1e37])[:, None], torch.rand(6, generator=r)
    k, p, m = torch.full((6,), 50, dtype=I32), torch.full((6,), 0.9), torch.full((6,), 0.01)
    for t in (1.0, 1e-4, 1e5, 1e8):
        temperature = torch.full((6,), t)
        rows_match(tq, x, u, temperature=temperature)
        rows_match(tq, x, u, temperature=temperature, top_k=k, top_p=p)
        rows_match(tq, x, u, temperature=temperature, top_p=p, min_p=m)


@pytest.mark.parametrize("rows,vocab", [(1500, 300), (3, 262_137), (3, 262_144), (2, 500_001), (2, 2**20), (2, 2**20 - 1)])
def test_sample_sizes(tq, rows, vocab):
    r = gen(rows + vocab)
    wide = (torch.randn(rows, vocab + 7, generator=r) * 2).bfloat16()
    u, p, k = torch.rand(rows, generator=r), torch.full((rows,), 0.7), torch.full((rows,), 100, dtype=I32)
    for off in (0, 7):
        x = wide[:, off : off + vocab]
        for params in (dict(top_p=p), dict(top_k=k), dict()):
            if rows > 100 and off:
                continue
            got = tq.sample(wide.cuda()[:, off : off + vocab], u.cuda(), **{n: v.cuda() for n, v in params.items()}).cpu()
            for i in range(0, rows, max(1, rows // 50)):
                want = bo.sample(x[i].double(), float(u[i]), 1.0, int(k[i]) if "top_k" in params else 0, float(p[i]) if "top_p" in params else 1.0, 0.0)
                assert int(got[i]) == want[0], (i, off, params)


# ---- offsets beyond 32 bits ----------------------------------------------------------------------------------------

def test_far_rows(tq):
    """Rows of logits, x, y and out that lie more than 2^31 values apart."""
    far = 2**31 + 16
    buf = torch.empty(far + 4096, dtype=BF, device="cuda")
    x = buf.as_strided((2, 3000), (far, 1))
    x.copy_(torch.randn(2, 3000, generator=gen(31)).to(BF))
    u, k = torch.tensor([0.3, 0.8]).cuda(), torch.tensor([40, 40], dtype=I32).cuda()
    assert torch.equal(tq.sample(x, u, top_k=k), tq.sample(x.contiguous(), u, top_k=k))
    w, i = tq.route(x[:, :64], 6)
    w1, i1 = tq.route(x[:, :64].contiguous(), 6)
    assert torch.equal(w, w1) and torch.equal(i, i1)
    a, b = torch.randn(1, 8, 1024, generator=gen(32)).to(BF).cuda(), torch.randn(1, 500, 8, generator=gen(33)).to(BF).cuda()
    index = torch.zeros(2, dtype=I32, device="cuda")
    y = torch.randn(2, 500, generator=gen(34)).to(BF).cuda()
    want = tq.adapter_add(y, x[:, :1024].contiguous(), a, b, index, out=torch.empty_like(y))
    out = buf.as_strided((2, 500), (far, 1), 2000)
    assert torch.equal(tq.adapter_add(y, x[:, :1024], a, b, index, out=out), want)
    z = buf.as_strided((2, 500), (far, 1), 1200)
    z.copy_(y)
    assert torch.equal(tq.adapter_add(z, x[:, :1024], a, b, index), want)


def test_experts_outputs_beyond_32_bits(tq):
    g = np.random.default_rng(8)
    rows, cols, n, pairs = 33_000, 256, 2, 66_000  # 2.2e9 outputs
    w = torch.stack([tq.repack(torch.from_numpy(TI.pq2_matrix(g, rows, cols).reshape(-1)).cuda(), "pq2_0", rows, cols) for _ in range(n)])
    q, d, _ = tq.quantize_q8k(torch.randn(pairs // 4, cols, generator=gen(9)).cuda())
    ids = torch.randint(-1, n, (pairs,), generator=gen(10), dtype=I32)
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, *tq.expert_lists(ids.cuda(), n))
    for p in (0, 1, 4095, 50_000, 65_075, 65_076, 65_077, 65_998, 65_999):
        e = int(ids[p])
        want = torch.zeros(rows, device="cuda") if e < 0 else tq.gemv("pq2_0", w[e], rows, cols, q[p // 4], d[p // 4])
        assert torch.equal(y[p], want), p


def test_adapter_weights_beyond_32_bits(tq):
    """A and B of 2.1e9 values: the last adapters' lie behind 2^31."""
    n, rank, cols, rows = 4100, 256, 2048, 2048
    a, b = torch.zeros(n, rank, cols, dtype=BF, device="cuda"), torch.zeros(n, rows, rank, dtype=BF, device="cuda")
    r = gen(12)
    x, y = torch.randn(3, cols, generator=r), torch.randn(3, rows, generator=r)
    index = torch.tensor([n - 1, 0, n - 2], dtype=I32)
    few_a, few_b = (torch.randn(3, rank, cols, generator=r) * cols**-0.5).to(BF), (torch.randn(3, rows, rank, generator=r) * rank**-0.5).to(BF)
    for i, at in enumerate(index.tolist()):
        a[at], b[at] = few_a[i].cuda(), few_b[i].cuda()
    got = tq.adapter_add(y.cuda(), x.cuda(), a, b, index.cuda()).double().cpu()
    want, size = bo.adapter(y, x, few_a, few_b, torch.arange(3), None, None)
    assert bool(((got - want).abs() <= bo.adapter_bound(want, size, cols, rank, F32)).all())


def test_results_do_not_depend_on_timing(tq):
    r = gen(41)
    x, u = torch.randn(30, 90_000, generator=r).bfloat16().cuda(), torch.rand(30, generator=r).cuda()
    p = torch.full((30,), 0.95, device="cuda")
    logprob = [torch.empty(30, device="cuda") for _ in range(8)]
    tokens = [tq.sample(x, u, top_p=p, logprob=l) for l in logprob]
    assert all(torch.equal(t, tokens[0]) for t in tokens) and all(torch.equal(l, logprob[0]) for l in logprob)
    ids = torch.randint(0, 50, (5000, 4), generator=r, dtype=I32).cuda()
    lists = [tq.expert_lists(ids, 50) for _ in range(8)]
    assert all(torch.equal(o, lists[0][0]) for o, _ in lists)
    assert math.isfinite(float(logprob[0].sum()))
