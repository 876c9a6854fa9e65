"""Calls on tensors of a device that is not the current one are refused (stand-in device numbers, no GPU is touched)."""
import pytest

import lora_co_serving_gb300 as lm


class OnDevice:
    """What the check reads of a tensor."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.fixture
def current(monkeypatch):
    import torch
    return lambda d: monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: d, raising=False)


def test_current_device(current):
    current(0)
    lm._one_device(OnDevice(0), None, OnDevice(0))
    current(1)
    lm._one_device(OnDevice(1), OnDevice(1), None)


@pytest.mark.parametrize("now,devices", [(0, (1, 1)), (1, (0, 0, None)), (0, (1,)), (0, (0, 1)), (1, (0, 1)), (0, (-1, 0)),
                                         (0, (0, -1)), (0, (-1,))])
def test_other_devices_are_refused(current, now, devices):
    current(now)
    with pytest.raises(ValueError, match="one CUDA device"):
        lm._one_device(*(d if d is None else OnDevice(d) for d in devices))


def test_a_call_is_refused_before_anything_is_launched(current, monkeypatch):
    """Every entry of the operators goes through the check: none reaches the library with another device's tensors."""
    import torch
    current(0)
    lm.build()

    class NoCalls:
        def __getattr__(self, name):
            if name in ("lora_fp8_workspace_size", "lora_checkpoint_rows", "lora_last_error"):    # host functions
                return getattr(real, name)
            raise AssertionError(name + " was called")

    real = lm.library()
    monkeypatch.setattr(lm, "library", lambda: NoCalls())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)       # as if all lay on cuda:1
    e = torch.float8_e4m3fn
    x, w, ws = torch.zeros(4, 64), torch.zeros(32, 64, dtype=torch.uint8).view(e), torch.zeros(1, 1)
    labels, ref = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    ck = torch.zeros(4, 128, dtype=torch.uint8).view(e), torch.zeros(4, 2)
    for call in (lambda: lm.fp8_quantize(x), lambda: lm.fp8_quantize_weight(x), lambda: lm.fp8_linear(x, w, ws),
                 lambda: lm.swiglu_forward(x), lambda: lm.swiglu_backward(ck, x), lambda: lm.token_logprob(x, labels),
                 lambda: lm.preference_forward(x, labels, ref, []),
                 lambda: lm.preference_backward(x, labels, ref, torch.zeros(0), [])):
        with pytest.raises(ValueError, match="the current one"):
            call()
