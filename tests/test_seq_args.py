"""What the operators between a block's projections refuse, and their host-side helpers.  No kernel is launched: every
call fails validation, or has nothing to do."""
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


@pytest.fixture(autouse=True)
def no_stream(tq, monkeypatch):
    monkeypatch.setattr(tq.seq, "_stream", lambda index: None)


T, HQ, HK, D, PAGE, PAGES = 3, 4, 2, 64, 16, 5


def rope_args(**over):
    a = dict(q=fake(T, HQ, D), k=fake(T, HK, D), v=fake(T, HK, D), positions=fake(T, dtype=torch.int32), slots=fake(T, dtype=torch.int64),
             inv_freq=fake(D // 2, dtype=torch.float64), k_cache=fake(PAGES, HK, PAGE, D, dtype=torch.bfloat16),
             v_cache=fake(PAGES, HK, D, PAGE, dtype=torch.bfloat16))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(T, HQ, D)),                                    # host memory
    dict(q=fake(T, HQ * D)),                                          # no head dimension
    dict(q=fake(T, HQ, D, dtype=torch.float64)),
    dict(k=fake(T, HK, D, dtype=torch.bfloat16)),                     # another type than q's
    dict(k=fake(T, HK, D).transpose(1, 2).contiguous().transpose(1, 2)),  # last dimension not contiguous
    dict(positions=fake(T, dtype=torch.int64)),
    dict(positions=fake(T + 1, dtype=torch.int32)),
    dict(slots=fake(T, dtype=torch.int32)),
    dict(slots=None),
    dict(inv_freq=fake(D // 2)),
    dict(k_cache=fake(PAGES, HK, PAGE, D)),                           # fp32 cache
    dict(v_cache=fake(PAGES, HK, PAGE, D, dtype=torch.bfloat16)),     # V not transposed
    dict(q_norm=fake(D + 1)),
    dict(k_norm=fake(D, dtype=torch.bfloat16)),
    dict(layout="pairs"),
    dict(out=fake(T, HQ, D)),                                         # not the cache's type
    dict(bad_flag=fake(2, dtype=torch.int32)),
])
def test_rope_append_refuses_tensors(tq, over):
    with pytest.raises(ValueError):
        tq.rope_append(**rope_args(**over))


@pytest.mark.parametrize("over,status", [
    (dict(k=fake(T + 1, HK, D)), -2),
    (dict(v=fake(T, HK + 1, D)), -2),
    (dict(q=fake(T, 3, D)), -2),                                      # 3 query heads on 2 key heads
    (dict(q=fake(T, HQ, 128)), -2),
    (dict(inv_freq=fake(4, dtype=torch.float64)), -2),                # 8 values: not a multiple of 16
    (dict(inv_freq=fake(D, dtype=torch.float64)), -2),                # more than the head
    (dict(eps=-1.0), -2),
    (dict(eps=math.nan), -2),
    (dict(rope_scale=math.inf), -2),
    (dict(positions=None), -1),
    (dict(k_cache=fake(PAGES, HK, 24, D, dtype=torch.bfloat16), v_cache=fake(PAGES, HK, D, 24, dtype=torch.bfloat16)), -2),
    (dict(q=fake(T, HQ, D + 1)[..., :D]), -3),                        # rows not on 16 bytes
    (dict(q=fake(T * HQ * D + 1)[1:].view(T, HQ, D)), -3),
])
def test_rope_append_refuses_shapes(tq, over, status):
    with pytest.raises(tq.TQError) as e:
        tq.rope_append(**rope_args(**over))
    assert e.value.status == status


def attn_args(**over):
    a = dict(q=fake(T, HQ, D, dtype=torch.float16), k_cache=fake(PAGES, HK, PAGE, D, dtype=torch.float16),
             v_cache=fake(PAGES, HK, D, PAGE, dtype=torch.float16), block_table=fake(2, 3, dtype=torch.int32), kv_len=fake(2, dtype=torch.int32),
             cu=fake(3, dtype=torch.int32))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(T, HQ, D, dtype=torch.float16)),
    dict(block_table=fake(2, 3, dtype=torch.int64)),
    dict(block_table=fake(6, dtype=torch.int32)),
    dict(block_table=fake(3, 2, dtype=torch.int32).t()),
    dict(kv_len=fake(3, dtype=torch.int32)),
    dict(cu=fake(2, dtype=torch.int32)),
    dict(out=fake(T, HQ, D + 1, dtype=torch.float16)),
    dict(out=fake(T, HQ, D), out_dtype=torch.float16),
    dict(out_dtype=torch.float64),
    dict(lse=fake(T, HQ + 1)),
    dict(ws=fake(64)),
])
def test_paged_attn_refuses_tensors(tq, over):
    with pytest.raises(ValueError):
        tq.paged_attn(**attn_args(**over))


@pytest.mark.parametrize("over,status", [
    (dict(q=fake(T, HQ, D, dtype=torch.bfloat16)), -2),               # not the cache's type
    (dict(q=fake(T, HQ, 128, dtype=torch.float16)), -2),
    (dict(q=fake(T, 3, D, dtype=torch.float16)), -2),
    (dict(cu=None), -2),                                              # 3 tokens, 2 sequences
    (dict(window=-1), -2),
    (dict(max_len=-1), -2),
    (dict(scale=math.nan), -2),
    (dict(out_dtype=torch.bfloat16), -4),                             # neither the cache's type nor fp32
    (dict(q=fake(T, HQ, D + 4, dtype=torch.float16)[..., :D]), -3),
    (dict(block_table=fake(0, 3, dtype=torch.int32), kv_len=fake(0, dtype=torch.int32), cu=fake(1, dtype=torch.int32)), -2),
])
def test_paged_attn_refuses_shapes(tq, over, status):
    with pytest.raises(tq.TQError) as e:
        tq.paged_attn(**attn_args(**over))
    assert e.value.status == status


KH, VH, DK, DV = 2, 4, 64, 32


def gdn_args(**over):
    a = dict(q=fake(T, KH, DK), k=fake(T, KH, DK), v=fake(T, VH, DV), g=fake(T, VH), beta=fake(T, VH), state=fake(2, VH, DK, DV),
             cu=fake(3, dtype=torch.int32))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(T, KH, DK)),
    dict(k=fake(T, KH, DK, dtype=torch.float16)),
    dict(v=fake(T, VH * DV)),
    dict(g=fake(T, KH)),
    dict(beta=fake(T, VH, dtype=torch.bfloat16)),
    dict(state=fake(2, VH, DK, DV, dtype=torch.bfloat16)),
    dict(state=fake(2, VH, DV, DK)),
    dict(state_out=fake(3, VH, DK, DV)),
    dict(cu=fake(3, dtype=torch.int64)),
    dict(cu=fake(0, dtype=torch.int32)),
    dict(slots=fake(3, dtype=torch.int32)),
    dict(out=fake(T, VH, DV + 1)),
    dict(out_dtype=torch.float64),
])
def test_gdn_refuses_tensors(tq, over):
    with pytest.raises(ValueError):
        tq.gdn(**gdn_args(**over))


@pytest.mark.parametrize("over,status", [
    (dict(k=fake(T, KH, 128)), -2),
    (dict(q=fake(T, 3, DK), k=fake(T, 3, DK)), -2),                   # 4 value heads on 3 key heads
    (dict(q=fake(T, KH, 96), k=fake(T, KH, 96), state=fake(2, VH, 96, DV)), -2),
    (dict(v=fake(T, VH, 48), state=fake(2, VH, DK, 48)), -2),
    (dict(cu=None), -2),                                              # 3 tokens, 2 states
    (dict(cu=fake(4, dtype=torch.int32)), -2),                        # 3 sequences, 2 states, no slots
    (dict(cu=fake(1, dtype=torch.int32)), -2),                        # tokens without a sequence
    (dict(state=fake(0, VH, DK, DV), slots=fake(2, dtype=torch.int32)), -2),
    (dict(state=fake(VH, DK, DV)), -2),
    (dict(scale=math.inf), -2),
    (dict(eps=-1e-6), -2),
    (dict(max_len=-5), -2),
    (dict(out_dtype=torch.float16), -4),
    (dict(v=fake(T, VH, DV + 2)[..., :DV]), -3),
])
def test_gdn_refuses_shapes(tq, over, status):
    with pytest.raises(tq.TQError) as e:
        tq.gdn(**gdn_args(**over))
    assert e.value.status == status


def test_nothing_to_do_launches_nothing(tq):
    assert tq.rope_append(**rope_args(q=fake(0, HQ, D), k=fake(0, HK, D), v=fake(0, HK, D), positions=fake(0, dtype=torch.int32),
                                      slots=fake(0, dtype=torch.int64), out=fake(0, HQ, D, dtype=torch.bfloat16))).shape == (0, HQ, D)
    assert tq.paged_attn(**attn_args(q=fake(0, HQ, D, dtype=torch.float16), out=fake(0, HQ, D, dtype=torch.float16))).shape == (0, HQ, D)
    assert tq.gdn(**gdn_args(q=fake(0, KH, DK), k=fake(0, KH, DK), v=fake(0, VH, DV), g=fake(0, VH), beta=fake(0, VH), cu=fake(1, dtype=torch.int32),
                             out=fake(0, VH, DV))).shape == (0, VH, DV)


def test_struct_sizes_and_null_arguments(tq):
    s = tq.seq
    assert (s._ROPE.size, s._ATTN.size, s._GDN.size) == (200, 184, 224)  # asserted against the header where the library is built
    L = tq.lib()
    for f in (L.tq_rope_append, L.tq_paged_attn, L.tq_gdn):
        assert f(None, ctypes.c_void_p(0)) == tq.ERR_NULL
    # a struct of zeros has sizes that nothing takes
    for f, n in ((L.tq_rope_append, 200), (L.tq_paged_attn, 184), (L.tq_gdn, 224)):
        assert f(bytes(n), ctypes.c_void_p(0)) in (tq.ERR_SHAPE, tq.ERR_FORMAT)


def test_workspace_sizes(tq):
    assert tq.attn_workspace_bytes(1, 1, 24, 5, 128) == 0    # 24 heads on 5
    assert tq.attn_workspace_bytes(1, 1, 24, 2, 100) == 0
    assert tq.gdn_workspace_bytes(64, 1, 8, 96, 128) == 0
    assert tq.gdn_workspace_bytes(-1, 1, 8, 128, 128) == 0


def test_rope_frequencies(tq):
    f, s = tq.rope_frequencies(64, 1e4)
    assert f.dtype == torch.float64 and f.shape == (32,) and s == 1.0
    assert f[0] == 1.0 and f[16].item() == pytest.approx(1e-2, rel=1e-14)
    lin, _ = tq.rope_frequencies(64, 1e4, scaling="linear", factor=4)
    assert torch.allclose(lin, f / 4, rtol=1e-15)
    ntk, _ = tq.rope_frequencies(64, 1e4, scaling="ntk", factor=4)
    assert ntk[0] == 1.0 and ntk[-1].item() == pytest.approx(f[-1].item() / 4, rel=1e-12)
    yarn, scale = tq.rope_frequencies(64, 1e4, scaling="yarn", factor=4, original=4096)
    assert scale == pytest.approx(0.1 * math.log(4) + 1)
    assert yarn[0] == f[0] and yarn[-1].item() == pytest.approx(f[-1].item() / 4, rel=1e-12)
    assert bool(((yarn <= f * (1 + 1e-15)) & (yarn >= f / 4 * (1 - 1e-15))).all())
    bands, _ = tq.rope_frequencies(64, 1e4, scaling="bands", factor=8, original=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(bands[turns >= 4], f[turns >= 4]) and torch.allclose(bands[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    for kw in (dict(rot=3), dict(rot=64, base=1.0), dict(rot=64, scaling="yarn", factor=2), dict(rot=64, scaling="other"), dict(rot=64, factor=0)):
        with pytest.raises(ValueError):
            tq.rope_frequencies(**kw)
