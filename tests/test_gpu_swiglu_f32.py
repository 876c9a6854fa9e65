"""The MLP activation in float32 and at the ends of the exponential's range, against float64.

Tolerances, in units of 2^-24 of the result.  sig(g) of a negative g is e^g / (1 + e^g): an exponential (2 units in the
last place, 4 here), a sum (1, and half of the exponential's), a quotient (1) and a product (1), 9 at the most; a product
with the gate and one with up: 11, taken as 12.  The gradient of gate has 1 + g (1 - sig), which passes zero: relative to
its terms, 1 - sig 9, two products and a sum 12; with dh, sig, u and their products 24.
"""
import numpy as np
import pytest

import step_oracle as so

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    import lora_co_serving_gb300 as lm
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lm.build()
    lm.library()


def down(t):
    return t.detach().double().cpu().numpy()


def gates(spread, R, I):
    """Gates of a spread, up to where e^|g| still is a normal number."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(int(spread))
    x = torch.randn(R, I, device="cuda", generator=g) * spread
    return x.clamp(-86.0, 86.0), torch.randn(R, I, device="cuda", generator=g)


@pytest.mark.parametrize("spread", [0.1, 1.5, 4.0, 15.0, 40.0])
@pytest.mark.parametrize("I", [8, 136, 2176])
def test_forward(I, spread):
    import torch
    import lora_co_serving_gb300 as lm
    g, u = gates(spread, 67, I)
    h = lm.swiglu_forward(torch.cat([g, u], 1))
    torch.cuda.synchronize()
    ref = down(g) * so.sigmoid(down(g)) * down(u)
    assert (np.abs(down(h) - ref) <= 12 * UNIT * np.abs(ref) + 1e-37).all()


@pytest.mark.parametrize("spread", [0.1, 1.5, 4.0, 15.0, 40.0])
@pytest.mark.parametrize("I", [8, 136, 2176])
def test_backward(I, spread):
    import torch
    import lora_co_serving_gb300 as lm
    g, u = gates(spread, 67, I)
    _, saved = lm.swiglu_forward(torch.cat([g, u], 1), [(0, 67, 0, 1)], checkpoint=True)
    dh = torch.randn(67, I, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    d = lm.swiglu_backward(saved, dh)
    torch.cuda.synchronize()
    nb = so.blocks(I)
    gv, uv = (down(saved[0].float())[:, i * I:(i + 1) * I] * so.spread_rows(down(saved[1])[:, i * nb:(i + 1) * nb], I)
              for i in range(2))
    ref = so.swiglu_grad(gv, uv, down(dh))
    size = np.abs(down(dh) * uv) * so.sigmoid(gv) * (1 + np.abs(gv) * so.sigmoid(-gv))
    assert (np.abs(down(d)[:, :I] - ref[:, :I]) <= 24 * UNIT * size + 1e-37).all()
    assert (np.abs(down(d)[:, I:] - ref[:, I:]) <= 12 * UNIT * np.abs(ref[:, I:]) + 1e-37).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_negative_gates_meet_large_values(dtype):
    """Below -87.3 the sigmoid of a gate is a tiny number, not zero: it shows beside a large up, and in the gradients.
    (Below -100 it is below float32's smallest numbers at 24 bits; here every product is a normal number.)"""
    import torch
    import lora_co_serving_gb300 as lm
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    I = 128
    g = torch.linspace(-89.0, -85.0, I, device="cuda").expand(3, I).to(dt)
    u = torch.full((3, I), 1e30, device="cuda").to(dt)
    h = lm.swiglu_forward(torch.cat([g, u], 1))
    torch.cuda.synchronize()
    ref = down(g) * so.sigmoid(down(g)) * down(u)
    # e^-89 is 2^-128.4: four of float32's 24 bits are gone below its smallest normal number, 2^-126
    rel = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -19
    assert (np.abs(down(h) - ref) <= rel * np.abs(ref)).all()
