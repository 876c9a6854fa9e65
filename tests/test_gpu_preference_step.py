"""The operators around the layer run together: a preference fine-tuning step of a co-served block."""
import importlib.util
import os

import numpy as np
import pytest

import step_oracle as so

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    import lora_co_serving_gb300 as lm
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lm.build()
    lm.library()
    spec = importlib.util.spec_from_file_location("preference_finetune",
                                                  os.path.join(ROOT, "examples", "preference_finetune.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_loss_starts_at_log_2_and_falls(example):
    """The policy starts as the reference: every margin is zero.  The adapters of the decode rows are not trained:
    their logits stay as they are, bit for bit."""
    import torch
    losses, rewards, first, last = example.run(steps=8)
    assert abs(losses[0] - np.log(2.0)) < 1e-5
    assert (np.diff(losses) < 0).all() and losses[-1] < 0.5 * losses[0]
    assert (rewards[:, 0] > rewards[:, 1]).all()
    assert torch.equal(first, last)


def test_gradient_of_a_block_against_float64(example):
    """dB of the trained adapter against the chain rule in float64 on the same 8-bit values, every quantization on the
    way (activations, gradients, checkpoint) repeated.

    Tolerance: what differs is float32 against float64 sums and 16-bit roundings (2^-9 each) before the products; a
    value near a rounding boundary of e4m3 may fall to the other side of it, a step of 2^-4 to 2^-3 of itself, for about
    one value in 2^-9 / 2^-4 = 1/32 of them and in each of the five quantized operands: a random error of
    2^-3.5 * sqrt(1/32) * sqrt(5) = 3.5 % of the gradient's norm at the most."""
    import torch
    import lora_co_serving_gb300 as lm
    b = example.Block(256, 384, 512, np.array([16, 8, 32, 64], np.int32), seed=5)
    tokens, labels, pairs, segs, n = example.batch(3, 512, seed=9)
    x, saved, logits = b.forward(tokens, segs)
    f = lm.preference_forward(logits[:n], labels, torch.zeros(n, device="cuda"), pairs, 0.3)
    d = lm.preference_backward(logits[:n], labels, f.lse, f.coef, pairs)
    dA, dB = b.backward(x, saved, d, segs, slice(0, n))
    torch.cuda.synchronize()

    def down(t):
        return t.detach().float().cpu().numpy().astype(np.float64)

    def value(w):
        c = down(w[0])
        return c * so.spread_weight(down(w[1]), *c.shape)

    def q(v):
        c, s = so.quantize(v)
        return c * so.spread_rows(s, v.shape[1])

    dl = so.dlogits(down(logits[:n]), labels.cpu().numpy(), down(f.lse), down(f.coef), pairs, np.full(3, 1 / 3))
    dout = q(dl) @ value(b.head)
    dh = q(dout) @ value(b.down)
    ck = [down(saved[0])[:, i * 384:(i + 1) * 384] * so.spread_rows(down(saved[1])[:, i * 3:(i + 1) * 3], 384)
          for i in range(2)]
    dz = dout + q(so.swiglu_grad(ck[0], ck[1], dh)) @ value(b.gate_up)
    r = 16
    xa = down(x[:n]) @ down(b.pool.A[:r * 256]).reshape(r, 256).T
    want = 2.0 * xa.T @ dz
    got = down(dB[:r * 256]).reshape(r, 256)
    assert np.linalg.norm(got - want) <= 0.035 * np.linalg.norm(want)
    assert not down(dA[:r * 256]).any()          # B is zero: A has no gradient yet
