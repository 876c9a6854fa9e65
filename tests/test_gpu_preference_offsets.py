"""The preference gradient of rows whose logits lie far from zero, against the softmax of the logits in float64.

Tolerances.  A probability is e^(x - c) over a sum: |x - c| < 32 where it is not negligible, rounded and multiplied by
log2(e) (2^-19 each at 32), an exponential of a few units in the last place, and below a log-sum-exp of 256 half a unit of
that, 2^-17: 2^-16 of itself.  16-bit outputs add 2^-8.  At the label 1 - p cancels: 2^-16 of the row's factor.  A row's
gradient sums to zero within the sum of its entries' bounds, twice the factor times them.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


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


def rows(V, dtype, shift):
    """Logits of eight rows; the type's rounding of the shifted ones is part of the input."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(8, V, device="cuda", generator=g) * 3.0
    low = torch.finfo(dtype).min
    x[:4] += torch.tensor(shift, device="cuda")[:, None]
    x[4], x[5] = low, -1e9
    x[6] = shift[0]
    x[6, ::3] = float("-inf")
    x[7, V // 2:] = -1e9                          # an ordinary row, half of it masked
    return x.to(dtype)


@pytest.mark.parametrize("shift", [(0.0, 100.0, 255.0, 300.0), (-1e4, 1e4, -1e6, 1e6), (3e7, -3e9, 1e15, -1e30)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 1000, 4001, 9001, 50257])
def test_gradient_of_shifted_rows(V, dtype, shift):
    import torch
    import lora_co_serving_gb300 as lm
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x = rows(V, dt, shift)
    labels = torch.tensor([1, V - 1, 3, 2, 0, V // 2, 1, 1], device="cuda")
    pairs = [(0, 2, 2, 2), (4, 2, 6, 2)]
    f = lm.preference_forward(x, labels, torch.zeros(8, device="cuda"), pairs, 0.3)
    # factors near one whatever the loss's margin is
    coef = torch.tensor([[0.7, -0.7], [-0.9, 0.9]], device="cuda")
    dloss = torch.ones(2, device="cuda")
    d = lm.preference_backward(x, labels, f.lse, coef, pairs, dloss=dloss)
    y = x.clone()
    e = lm.preference_backward(y, labels, f.lse, coef, pairs, dloss=dloss, dlogits=y)
    wide = torch.full((8, V + 5), 9.0, dtype=dt, device="cuda")       # rows on another phase: element by element
    h = lm.preference_backward(x, labels, f.lse, coef, pairs, dloss=dloss, dlogits=wide[:, 1:V + 1])
    torch.cuda.synchronize()
    assert torch.equal(d, e) and torch.equal(d, h)
    assert (wide[:, 0] == 9.0).all() and (wide[:, V + 1:] == 9.0).all()
    xd, at = down(x), labels.cpu().numpy()
    p = np.exp(xd - xd.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    k = np.repeat([0.7, -0.7, -0.9, 0.9], 2).astype(np.float32).astype(np.float64)[:, None]
    want = -k * p
    want[np.arange(8), at] += k[:, 0]
    rel = 2.0 ** -16 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    tol = rel * np.abs(want) + 1e-37
    tol[np.arange(8), at] += 2.0 ** -16 * np.abs(k[:, 0])
    got = down(d)
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol, axis=1)
    assert (np.abs(got.sum(1)) <= 2 * rel * np.abs(k[:, 0]) + 2.0 ** -16 * np.abs(k[:, 0])).all()


def test_a_given_log_sum_exp_is_kept():
    """A log-sum-exp that is not the row's own (a vocabulary in parts, each with the whole one's) is taken as it is."""
    import torch
    import lora_co_serving_gb300 as lm
    V = 2000
    x = torch.randn(2, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) + 1000.0
    whole = torch.logsumexp(x.double(), 1).float()
    labels, pairs = torch.tensor([5, 700], device="cuda"), [(0, 1, 1, 1)]
    coef, dloss = torch.tensor([[1.0, -1.0]], device="cuda"), torch.ones(1, device="cuda")
    part = x[:, :1000].contiguous()
    d = lm.preference_backward(part, labels, whole, coef, pairs, dloss=dloss)
    torch.cuda.synchronize()
    want = -np.array([[1.0], [-1.0]]) * np.exp(down(part) - down(whole)[:, None])
    want[[0, 1], [5, 700]] += [1.0, -1.0]
    assert (np.abs(down(d) - want) <= 2.0 ** -16 * np.abs(want) + 2.0 ** -16 * (np.abs(want) > 0.5)).all()


def test_log_sum_exp_has_no_mean_error():
    """A sequence's sum of log ratios adds up thousands of log probabilities: their mean error counts, not a row's own.

    The fast exponential lies low by 4e-8 on average, which the kernel takes out; what is left is within half of that
    over vocabularies and spreads (4096 rows of 3e-7 each leave 5e-9 to chance, the mean of nine 2e-9)."""
    import torch
    import lora_co_serving_gb300 as lm
    T, off = 4096, []
    for V in (500, 4000, 32000):
        for sd in (1.0, 2.0, 3.0):
            x = torch.randn(T, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(V + int(sd))) * sd
            _, lse = lm.token_logprob(x, torch.zeros(T, dtype=torch.int64, device="cuda"))
            ref = torch.cat([torch.logsumexp(c.double(), 1) for c in x.split(256)])
            off.append(float((lse.double() - ref).mean()))
    assert abs(np.mean(off)) <= 2e-8 and max(map(abs, off)) <= 4e-8, off
