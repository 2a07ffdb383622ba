"""What the operators of a mixed batch (experts, adapters, sampling) refuse.  No kernel is launched: every call fails
validation, or has nothing to do."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def tq():
    import bit_quantized_matvec_amd as m

    return m


class FakeGpu(torch.Tensor):
    """Host memory that claims to be on the GPU: reaches the checks behind the first one."""

    @property
    def is_cuda(self):
        return True


def fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(FakeGpu)


I32, BF, HF = torch.int32, torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def no_stream(tq, monkeypatch):
    import sys

    for m in ("seq", "batch"):
        monkeypatch.setattr(sys.modules[f"bit_quantized_matvec_amd.{m}"], "_stream", lambda index: None)


def refuses(error, f, args, over, status=None):
    with pytest.raises(error) as e:
        f(**{**args, **over})
    if status is not None:
        assert e.value.status == status


ROUTE = dict(logits=fake(3, 16), k=4)


@pytest.mark.parametrize("over", [dict(logits=torch.zeros(3, 16)), dict(logits=fake(16)), dict(logits=fake(3, 16, dtype=torch.float64)), dict(logits=fake(16, 3).t()),
                                  dict(score="tanh"), dict(bias=fake(15)), dict(bias=fake(16, dtype=BF)), dict(out=(fake(3, 4), fake(3, 4))),
                                  dict(out=(fake(3, 5), fake(3, 4, dtype=I32))), dict(scale="1"), dict(groups=2**40), dict(top_groups=1.5)])
def test_route_refuses_tensors(tq, over):
    refuses(ValueError, tq.route, dict(ROUTE, out=(fake(3, 4), fake(3, 4, dtype=I32))), over)


@pytest.mark.parametrize("over,status", [(dict(k=0), -2), (dict(k=33), -2), (dict(k=17), -2), (dict(k=2.0), -2), (dict(logits=fake(3, 1025)), -2), (dict(groups=3), -2),
                                         (dict(groups=0), -2), (dict(groups=4, top_groups=5), -2), (dict(groups=4, top_groups=0), -2),
                                         (dict(groups=8, top_groups=1), -2), (dict(groups=4, top_groups=2, group_best=3), -2),
                                         (dict(groups=16, top_groups=8, group_best=2), -2), (dict(scale=math.inf), -2)])
def test_route_refuses_shapes(tq, over, status):
    k = over.get("k", 4)
    out = (fake(3, k), fake(3, k, dtype=I32)) if isinstance(k, int) else None
    refuses(tq.TQError, tq.route, dict(ROUTE, out=out), over, status)


@pytest.mark.parametrize("over,error", [(dict(experts=torch.zeros(3, dtype=I32)), ValueError), (dict(experts=fake(3)), ValueError),
                                        (dict(experts=fake(3, 2, dtype=I32).t()), ValueError), (dict(n=0), RuntimeError), (dict(n=65537), RuntimeError),
                                        (dict(out=(fake(3, dtype=I32), fake(4, dtype=I32))), ValueError)])
def test_expert_lists_refuses(tq, over, error):
    refuses(error, tq.expert_lists, dict(experts=fake(3, dtype=I32), n=4), over)


def experts_args(tq, rows=64, cols=512, n=3, pairs=6, inputs=2):
    return dict(fmt="pq2_0", w=fake(n, tq.repacked_bytes("pq2_0", rows, cols), dtype=torch.uint8), rows=rows, cols=cols, q=fake(inputs, cols, dtype=torch.int8),
                d=fake(inputs, cols // 256), order=fake(pairs, dtype=I32), offsets=fake(n + 1, dtype=I32), out=fake(pairs, rows))


@pytest.mark.parametrize("over", [dict(w=torch.zeros(3, 10, dtype=torch.uint8)), dict(w=fake(10, dtype=torch.uint8)), dict(q=fake(2, 512)),
                                  dict(q=fake(2, 256, dtype=torch.int8)), dict(q=fake(1024, dtype=torch.int8)), dict(d=fake(2, 1)), dict(order=fake(6)),
                                  dict(order=fake(3, 2, dtype=I32)), dict(offsets=fake(3, dtype=I32)), dict(out=fake(6, 63)), dict(bad_flag=fake(1)), dict(out=fake(5, 64))])
def test_gemm_experts_refuses_tensors(tq, over):
    refuses(ValueError, tq.gemm_experts, experts_args(tq), over)


def test_gemm_experts_refuses_shapes(tq):
    f, a = tq.gemm_experts, experts_args(tq)
    refuses(tq.TQError, f, a, dict(rows=65), -2)                          # other matrices than w's
    refuses(tq.TQError, f, a, dict(cols=500), -2)
    refuses(tq.TQError, f, experts_args(tq, pairs=5), {}, -2)             # 5 pairs of 2 inputs
    refuses(tq.TQError, f, experts_args(tq, inputs=0), {}, -2)
    w = fake(3, tq.repacked_bytes("ptq1_0", 64, 512), dtype=torch.uint8)
    refuses(tq.TQError, f, a, dict(fmt="ptq1_0", w=w), -5)
    refuses(tq.TQError, f, a, dict(fmt=7), -2)
    refuses(ValueError, f, a, dict(fmt="pq3"))


ADAPT = dict(y=fake(3, 10), x=fake(3, 16), a=fake(2, 8, 16, dtype=BF), b=fake(2, 10, 8, dtype=BF), index=fake(3, dtype=I32), ws=fake(1 << 16, dtype=torch.uint8))


@pytest.mark.parametrize("over", [dict(y=torch.zeros(3, 10)), dict(y=fake(10)), dict(y=fake(10, 3).t()), dict(x=fake(3, 8)), dict(x=fake(2, 16)),
                                  dict(x=fake(3, 16, dtype=torch.float64)), dict(a=fake(2, 8, 16)), dict(a=fake(2, 128, dtype=BF)), dict(b=fake(2, 10, 8, dtype=HF)),
                                  dict(b=fake(2, 8, 10, dtype=BF)), dict(index=fake(3, dtype=torch.int64)), dict(index=fake(4, dtype=I32)),
                                  dict(ranks=fake(3, dtype=I32)), dict(scale=fake(2, dtype=BF)), dict(out=fake(3, 11)), dict(out=fake(3, 10, dtype=BF)),
                                  dict(out=fake(1, 10).expand(3, 10)), dict(ws=fake(4, dtype=torch.uint8)), dict(bad_flag=fake(2, dtype=I32))])
def test_adapter_add_refuses_tensors(tq, over):
    refuses(ValueError, tq.adapter_add, ADAPT, over)


@pytest.mark.parametrize("over,status", [
    (dict(x=fake(3, 16, dtype=HF)), -4),                                              # neither fp32 nor the weights' type
    (dict(a=fake(2, 12, 16, dtype=BF), b=fake(2, 10, 12, dtype=BF)), -2),
    (dict(a=fake(2, 264, 16, dtype=BF), b=fake(2, 10, 264, dtype=BF)), -2),
    (dict(x=fake(3, 12), a=fake(2, 8, 12, dtype=BF)), -2),
    (dict(a=fake(0, 8, 16, dtype=BF), b=fake(0, 10, 8, dtype=BF)), -2),
    (dict(x=fake(3, 17)[:, :16]), -3),                                                # rows not on 16 bytes
    (dict(x=fake(49)[1:].view(3, 16)), -3),
    (dict(y=fake(3, 12)[:, 1:11], out=fake(3, 10)), 0),                               # y's rows need no alignment
])
def test_adapter_add_refuses_shapes(tq, over, status):
    if status == 0:  # the check passes: with no tokens nothing is launched
        tq.adapter_add(**{**ADAPT, "y": fake(0, 12)[:, 1:11], "x": fake(0, 16), "index": fake(0, dtype=I32), "out": fake(0, 10)})
        return
    refuses(tq.TQError, tq.adapter_add, ADAPT, over, status)


@pytest.mark.parametrize("stride", [1, 9])
def test_adapter_add_refuses_rows_that_overlap(tq, stride):
    y = fake(40).as_strided((3, 10), (stride, 1))
    refuses(tq.TQError, tq.adapter_add, ADAPT, dict(out=y), -2)
    refuses(tq.TQError, tq.adapter_add, ADAPT, dict(y=y, out=None), -2)


def test_adapter_add_in_place_needs_one_stride(tq):
    y = fake(3, 20)
    refuses(tq.TQError, tq.adapter_add, ADAPT, dict(y=y[:, :10], out=y.view(6, 10)[:3]), -2)


SAMPLE = dict(logits=fake(3, 50), u=fake(3), out=fake(3, dtype=I32), ws=fake(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("over", [dict(logits=torch.zeros(3, 50)), dict(logits=fake(50)), dict(logits=fake(50, 3).t()), dict(logits=fake(3, 50, dtype=I32)),
                                  dict(u=fake(4)), dict(u=None), dict(u=fake(3, dtype=torch.float64)), dict(temperature=fake(3, dtype=BF)), dict(temperature=1.0),
                                  dict(top_k=fake(3)), dict(top_p=fake(1)), dict(min_p=fake(3, 1)), dict(out=fake(3)), dict(logprob=fake(4)),
                                  dict(ws=fake(1, dtype=torch.uint8))])
def test_sample_refuses_tensors(tq, over):
    refuses(ValueError, tq.sample, SAMPLE, over)


@pytest.mark.parametrize("vocab", [0, 2**20 + 1])
def test_sample_refuses_shapes(tq, vocab):
    refuses(tq.TQError, tq.sample, SAMPLE, dict(logits=fake(3, vocab, dtype=BF)), -2)


def test_nothing_to_do(tq):
    w, i = tq.route(fake(0, 16), 4, out=(fake(0, 4), fake(0, 4, dtype=I32)))
    assert w.shape == (0, 4)
    assert tq.gemm_experts(**experts_args(tq, pairs=0, inputs=0)).shape == (0, 64)
    assert tq.sample(fake(0, 50), fake(0), out=fake(0, dtype=I32), ws=fake(1 << 16, dtype=torch.uint8)).shape == (0,)


def test_workspaces(tq):
    assert tq.adapter_workspace_bytes(64, 24, 32, 5120) > 0 and tq.sample_workspace_bytes(64, 131072) > 0
    for args in ((-1, 24, 32, 5120), (64, 0, 32, 5120), (64, 24, 12, 5120), (64, 24, 32, 100), (2**21, 24, 32, 5120)):
        assert tq.adapter_workspace_bytes(*args) == 0
    for args in ((-1, 100), (1, 0), (1, 2**21), (2**17, 100)):
        assert tq.sample_workspace_bytes(*args) == 0
    # larger calls need no less
    for t in (1, 16, 17, 200, 5000):
        assert tq.adapter_workspace_bytes(t, 24, 32, 5120) >= 4 * t * 33


def test_abi_null_and_alignment(tq):
    L, P = tq.lib(), ctypes.c_void_p
    good, odd = 0x100000, 0x100002
    for f in (L.tq_route, L.tq_gemm_experts, L.tq_adapter_add, L.tq_sample):
        assert f(None, None) == tq.ERR_NULL
    assert L.tq_expert_lists(P(good), 4, 2, P(good), None, None) == tq.ERR_NULL
    assert L.tq_expert_lists(None, 4, 2, P(good), P(good), None) == tq.ERR_NULL
    assert L.tq_expert_lists(P(odd), 4, 2, P(good), P(good), None) == tq.ERR_ALIGN
    assert L.tq_expert_lists(P(good), -1, 2, P(good), P(good), None) == tq.ERR_SHAPE
    assert L.tq_expert_lists(P(good), 2**26, 2, P(good), P(good), None) == tq.ERR_SHAPE
    b = tq.batch
    route = lambda **o: b._ROUTE.pack(*{**dict(l=good, b=0, w=good, i=good, s=16, t=3, n=16, k=4, g=1, tg=1, gb=1, sc=0, r=1, ty=0, f=1.0), **o}.values())  # noqa: E731
    assert L.tq_route(route(l=0), None) == tq.ERR_NULL and L.tq_route(route(i=0), None) == tq.ERR_NULL
    assert L.tq_route(route(l=odd), None) == tq.ERR_ALIGN and L.tq_route(route(ty=9), None) == tq.ERR_FORMAT and L.tq_route(route(s=2**41), None) == tq.ERR_SHAPE
    ex = lambda **o: b._EXPERTS.pack(*{**dict(w=good, q=good, d=good, o=good, f=good, y=good, b=0, r=64, c=256, p=4, i=2, e=3, fmt=1), **o}.values())  # noqa: E731
    assert L.tq_gemm_experts(ex(q=0), None) == tq.ERR_NULL and L.tq_gemm_experts(ex(q=odd), None) == tq.ERR_ALIGN
    assert L.tq_gemm_experts(ex(fmt=5), None) == tq.ERR_FORMAT and L.tq_gemm_experts(ex(e=0), None) == tq.ERR_SHAPE
    ad = lambda **o: b._ADAPTER.pack(*{**dict(x=good, y=good, a=good, b=good, o=good + 4096, i=good, r=0, s=0, w=good, f=0, xs=16, ys=10, os=10, t=3, c=16, rows=10,  # noqa: E731
                                              wb=1 << 20, n=2, rank=8, xt=0, wt=1, yt=0), **o}.values())
    assert L.tq_adapter_add(ad(w=0), None) == tq.ERR_NULL and L.tq_adapter_add(ad(a=odd), None) == tq.ERR_ALIGN
    assert L.tq_adapter_add(ad(wb=16), None) == tq.ERR_SHAPE and L.tq_adapter_add(ad(wt=0), None) == tq.ERR_FORMAT
    sa = lambda **o: b._SAMPLE.pack(*{**dict(l=good, u=good, t=0, k=0, p=0, m=0, o=good, g=0, w=good, s=50, r=3, v=50, wb=1 << 30, ty=0), **o}.values())  # noqa: E731
    assert L.tq_sample(sa(w=0), None) == tq.ERR_NULL and L.tq_sample(sa(w=good + 8), None) == tq.ERR_ALIGN and L.tq_sample(sa(wb=0), None) == tq.ERR_SHAPE
    assert L.tq_sample(sa(ty=3), None) == tq.ERR_FORMAT and tq.lib().tq_last_hip_error() == 0
