"""Which kernel a call of the operators between a block's projections takes, by its sizes.  No kernel is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def rows():
    import bit_quantized_matvec_amd as m

    return m.lib().tq_paged_attn_tile_rows


def test_paged_attn_rows_of_a_workgroup(rows):
    # one token each: 16, however many
    assert rows(1, 1, 1, 24, 2, 256) == rows(64, 64, 1, 48, 4, 128) == rows(4096, 4096, 0, 1024, 64, 64) == 16
    # a prompt that fills the card: 128
    assert rows(2048, 1, 2048, 48, 4, 128) == rows(500, 1, 0, 24, 2, 256) == rows(60, 2, 40, 32, 16, 64) == 128
    # few 16-row tiles: 16.  An eighth of the places (two workgroups per compute unit, one at 256 columns) decides
    assert rows(32, 1, 32, 16, 16, 64) == 16 and rows(48, 1, 48, 16, 16, 64) == 128       # 3, 4 tiles x 16 key heads
    assert rows(48, 1, 48, 7, 7, 256) == 16 and rows(48, 1, 48, 8, 8, 256) == 128         # 4 tiles x 7, 8
    # the longest sequence has 16 rows: 16
    assert rows(900, 100, 16, 64, 64, 64) == 16 and rows(900, 100, 17, 64, 64, 64) == 128
    assert rows(0, 0, 0, 24, 2, 256) == 16


@pytest.mark.parametrize("args", [(-1, 1, 1, 24, 2, 256), (1, -1, 1, 24, 2, 256), (1, 1, -1, 24, 2, 256), (1, 1, 1, 24, 5, 256), (1, 1, 1, 24, 2, 96),
                                  (1, 0, 1, 24, 2, 256), (1 << 21, 1, 1, 24, 2, 256)])
def test_paged_attn_rows_of_refused_sizes(rows, args):
    assert rows(*args) == 0


class OnSecondDevice(torch.Tensor):
    """Host memory that claims to be on a second GPU."""

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", 1)


def test_calls_run_on_the_tensors_device(monkeypatch):
    """The tensors' device is made current around a call (none has anything to do here), and its stream is taken."""
    import bit_quantized_matvec_amd as tq

    current, calls = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(tq.seq, "_current_device", lambda: current[0])
    monkeypatch.setattr(tq.seq, "_stream", lambda index: calls.append((index, current[0])))

    def t(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnSecondDevice)

    i32, bf = torch.int32, torch.bfloat16
    kc, vc = t(2, 1, 16, 64, dtype=bf), t(2, 1, 64, 16, dtype=bf)
    tq.rope_append(t(0, 1, 64), t(0, 1, 64), t(0, 1, 64), None, t(0, dtype=torch.int64), None, kc, vc, out=t(0, 1, 64, dtype=bf))
    tq.paged_attn(t(0, 1, 64, dtype=bf), kc, vc, t(1, 2, dtype=i32), t(1, dtype=i32), t(2, dtype=i32), out=t(0, 1, 64, dtype=bf))
    tq.gdn(t(0, 1, 64), t(0, 1, 64), t(0, 1, 32), t(0, 1), t(0, 1), t(1, 1, 64, 32), t(1, dtype=i32), out=t(0, 1, 32))
    assert calls == [(1, 1)] * 3 and current == [0]


@pytest.mark.parametrize("call,over", [
    ("rope", dict(inv_freq=[1.0] * 32)), ("rope", dict(eps="small")), ("rope", dict(rope_scale=None)),
    ("attn", dict(window=2**31)), ("attn", dict(window=1.5)), ("attn", dict(max_len=None)), ("attn", dict(max_len=2**63)), ("attn", dict(scale="1")),
    ("gdn", dict(max_len=2**64)), ("gdn", dict(eps=None)),
])
def test_arguments_that_no_field_holds(call, over):
    import bit_quantized_matvec_amd as tq

    def t(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnSecondDevice)

    i32, bf = torch.int32, torch.bfloat16
    kc, vc = t(2, 1, 16, 64, dtype=bf), t(2, 1, 64, 16, dtype=bf)
    if call == "rope":
        f, a = tq.rope_append, dict(q=t(0, 1, 64), k=t(0, 1, 64), v=t(0, 1, 64), positions=t(0, dtype=i32), slots=t(0, dtype=torch.int64),
                                    inv_freq=t(32, dtype=torch.float64), k_cache=kc, v_cache=vc, out=t(0, 1, 64, dtype=bf))
    elif call == "attn":
        f, a = tq.paged_attn, dict(q=t(0, 1, 64, dtype=bf), k_cache=kc, v_cache=vc, block_table=t(1, 2, dtype=i32), kv_len=t(1, dtype=i32),
                                   cu=t(2, dtype=i32), out=t(0, 1, 64, dtype=bf))
    else:
        f, a = tq.gdn, dict(q=t(0, 1, 64), k=t(0, 1, 64), v=t(0, 1, 32), g=t(0, 1), beta=t(0, 1), state=t(1, 1, 64, 32), cu=t(1, dtype=i32), out=t(0, 1, 32))
    with pytest.raises(ValueError):
        f(**{**a, **over})
