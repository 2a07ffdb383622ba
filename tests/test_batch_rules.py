"""The operators of a mixed batch on the CPU: which device and stream a call takes, and arguments that no field holds.  No
kernel is launched."""
import sys

import pytest
import torch

I32, BF = torch.int32, torch.bfloat16


class OnSecondDevice(torch.Tensor):
    """Host memory that claims to be on a second GPU."""

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", 1)


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnSecondDevice)


def calls(tq):
    u8 = torch.uint8
    w = t(2, tq.repacked_bytes("pq2_0", 64, 256), dtype=u8)
    return [lambda **o: tq.route(t(0, 8), **{**dict(k=2, out=(t(0, 2), t(0, 2, dtype=I32))), **o}),
            lambda **o: tq.gemm_experts("pq2_0", w, 64, 256, t(0, 256, dtype=torch.int8), t(0, 1), t(0, dtype=I32), t(3, dtype=I32), out=t(0, 64)),
            lambda **o: tq.adapter_add(t(0, 5), t(0, 8), t(1, 8, 8, dtype=BF), t(1, 5, 8, dtype=BF), t(0, dtype=I32), ws=t(4096, dtype=u8)),
            lambda **o: tq.sample(t(0, 9), t(0), out=t(0, dtype=I32), ws=t(1 << 20, dtype=u8))]


def test_calls_run_on_the_tensors_device(monkeypatch):
    """The tensors' device is made current around a call (none has anything to do here), and its stream is taken."""
    import bit_quantized_matvec_amd as tq

    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    for m in ("seq", "batch"):
        module = sys.modules[f"bit_quantized_matvec_amd.{m}"]
        monkeypatch.setattr(module, "_current_device", lambda: current[0])
        monkeypatch.setattr(module, "_stream", lambda index: seen.append((index, current[0])))
    for call in calls(tq):
        call()
    assert seen == [(1, 1)] * 4 and current == [0]


@pytest.mark.parametrize("over", [dict(groups=2**31), dict(scale="2"), dict(top_groups=None), dict(group_best=1.5)])
def test_arguments_that_no_field_holds(over):
    import bit_quantized_matvec_amd as tq

    with pytest.raises(ValueError):
        calls(tq)[0](**over)


def test_without_the_module(monkeypatch):
    """The checks in Python serve every call where the C++ ones are not there."""
    import bit_quantized_matvec_amd as tq

    monkeypatch.setattr(tq.batch, "_binding", None)
    for call in (lambda: tq.route(torch.zeros(1, 4), 2), lambda: tq.expert_lists(torch.zeros(2, dtype=I32), 2), lambda: tq.sample(torch.zeros(1, 4), torch.zeros(1)),
                 lambda: tq.adapter_add(torch.zeros(1, 4), torch.zeros(1, 8), torch.zeros(1, 8, 8, dtype=BF), torch.zeros(1, 4, 8, dtype=BF), torch.zeros(1, dtype=I32)),
                 lambda: tq.gemm_experts("pq2_0", torch.zeros(1, 4, dtype=torch.uint8), 64, 256, None, None, None, None)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
