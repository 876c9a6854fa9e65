"""The preference loss and its gradient against float64, and the gradient against differences of the loss.

Tolerances.  A row's log-sum-exp has its exponents rounded once (x log2 e - n, |.| < 64: 2^-19 absolute at worst for a
term, half a unit of float32 there) and an exponential of a few units in the last place; it is itself a float32 number
of size up to 32, so 2^-18 absolute; a log probability twice that.  A sequence's sum of n such: n times.  Gradients:
p = e^(x - lse) is within 2^-17 of itself plus lse's error, 2^-16; 16-bit outputs add their rounding, 2^-8.
"""
import numpy as np
import pytest

import step_oracle as so

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    import lora_co_serving_gb300 as lm
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lm.build()
    lm.library()


def up(a, dtype="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(
        {"bf16": torch.bfloat16, "f32": torch.float32}[dtype])


def lab(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int64)).cuda()


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def case(seed, T, V, dtype, masked=0.3):
    rng = np.random.default_rng(seed)
    x = up(3.0 * rng.standard_normal((T, V)), dtype)
    labels = rng.integers(0, V, T)
    labels[rng.random(T) < masked] = -rng.integers(1, 200)
    ref = rng.standard_normal(T) * 0.5 - 3.0
    return x, labels, ref.astype(np.float32).astype(np.float64)


PAIRS = {
    "two rows": (2, [(0, 1, 1, 1)]),
    "ragged": (23, [(0, 3, 3, 9), (13, 1, 14, 2), (20, 3, 16, 4)]),
    "gaps, empty ones": (40, [(5, 10, 20, 0), (0, 0, 0, 0), (30, 4, 15, 5)]),
    "none": (6, []),
    "many": (300, [(4 * i, 2, 4 * i + 2, 1) for i in range(75)]),
}
SIZES = [(1, "f32"), (2, "bf16"), (7, "bf16"), (33, "f32"), (501, "bf16"), (504, "bf16"), (4099, "f32"),
         (32001, "bf16"), (50257, "f32")]


@pytest.mark.parametrize("table", sorted(PAIRS))
@pytest.mark.parametrize("V,dtype", SIZES)
def test_forward_and_backward(V, dtype, table):
    import torch
    import lora_co_serving_gb300 as lm
    T, pairs = PAIRS[table]
    x, labels, ref = case(V + T, T, V, dtype)
    beta, eps = 0.2, 0.1
    f = lm.preference_forward(x, lab(labels), up(ref), pairs, beta, eps)
    dl = np.random.default_rng(3).standard_normal(len(pairs)).astype(np.float32)
    d = lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs, dloss=up(dl))
    torch.cuda.synchronize()
    xd = down(x)
    loss, rewards, logp, lse, coef = so.preference(xd, labels, ref, pairs, beta, eps)
    unit = 2.0 ** -18
    assert (np.abs(down(f.lse) - lse) <= unit).all()
    assert (np.abs(down(f.logp) - logp) <= 2 * unit).all()
    assert not down(f.lse)[labels < 0].any() and not down(f.logp)[labels < 0].any()
    n = np.array([[cn, rn] for _, cn, _, rn in pairs]).reshape(-1, 2)
    tol = beta * 2 * unit * n + 2.0 ** -23 * np.abs(rewards)
    assert (np.abs(down(f.rewards) - rewards) <= tol).all()
    m_tol = tol.sum(1)
    assert (np.abs(down(f.loss) - loss) <= m_tol + 2.0 ** -22 * np.abs(loss)).all()
    assert (np.abs(down(f.coef) - coef) <= beta * m_tol[:, None] + 2.0 ** -22 * np.abs(coef)).all()
    want = so.dlogits(xd, labels, down(f.lse), down(f.coef), pairs, dl.astype(np.float64))
    k = np.zeros(T)
    for i, (c0, cn, r0, rn) in enumerate(pairs):
        k[c0:c0 + cn] = k[r0:r0 + rn] = np.abs(down(f.coef)[i, 0] * dl[i])
    tol = (2.0 ** -8 if dtype == "bf16" else 0.0) * np.abs(want) + 2.0 ** -16 * np.abs(want) + 1e-37
    tol[np.arange(T), np.maximum(labels, 0)] += 2.0 ** -16 * k            # 1 - p cancels at the label
    assert (np.abs(down(d) - want) <= tol).all()
    inside = np.zeros(T, bool)
    for c0, cn, r0, rn in pairs:
        inside[c0:c0 + cn] = inside[r0:r0 + rn] = True
    assert not down(d)[~inside | (labels < 0)].any()


def test_mean_is_the_default_and_in_place():
    import torch
    import lora_co_serving_gb300 as lm
    T, pairs = PAIRS["ragged"]
    for V, dtype in ((504, "bf16"), (501, "bf16"), (33, "f32")):
        x, labels, ref = case(1, T, V, dtype)
        f = lm.preference_forward(x, lab(labels), up(ref), pairs)
        d = lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs)
        e = lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs, dloss=up([1 / 3] * 3))
        y = x.clone()
        g = lm.preference_backward(y, lab(labels), f.lse, f.coef, pairs, dlogits=y)
        torch.cuda.synchronize()
        assert torch.equal(d, e) and torch.equal(d, g) and g.data_ptr() == y.data_ptr()


def test_gradient_is_the_differences():
    """Differences of the float64 loss over every logit of a small batch, chained through a weighted sum of losses."""
    import torch
    import lora_co_serving_gb300 as lm
    T, V, pairs = 9, 11, [(0, 2, 2, 3), (7, 2, 5, 2)]
    x, labels, ref = case(6, T, V, "f32", masked=0.2)
    w = np.array([0.7, -1.3])
    f = lm.preference_forward(x, lab(labels), up(ref), pairs, 0.5, 0.05)
    got = down(lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs, dloss=up(w)))
    torch.cuda.synchronize()
    xd, h = down(x), 1e-5
    num = np.zeros_like(xd)
    for t in range(T):
        for v in range(V):
            s = []
            for sign in (1, -1):
                z = xd.copy()
                z[t, v] += sign * h
                s.append((so.preference(z, labels, ref, pairs, 0.5, 0.05)[0] * w.astype(np.float32)).sum())
            num[t, v] = (s[0] - s[1]) / (2 * h)
    # float32 gradients of size below 1 (2^-16, above) and differences good to h^2 + 1e-15 / h
    assert np.abs(got - num).max() <= 2.0 ** -16 + 1e-8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_and_bad_logits(dtype):
    """-infinity is a probability of zero; a row without a finite logit, a NaN, +infinity or a label past the end
    gives NaN for its pair and no other; a label of probability zero gives an infinite loss with finite gradients."""
    import torch
    import lora_co_serving_gb300 as lm
    V = 300
    pairs = [(2 * i, 1, 2 * i + 1, 1) for i in range(7)]
    x, labels, ref = case(2, 14, V, dtype, masked=0.0)
    labels[:] = 5
    x[:, 5] = 1.0
    x[0, :200] = float("-inf")
    x[0, 5], labels[0] = 1.0, 250
    x[2] = float("-inf")
    x[4, 77] = float("nan")
    x[6, 299] = float("inf")
    labels[8] = V
    x[10, 5] = float("-inf")                       # the chosen token of pair 5 has probability zero
    x[13, 5] = float("-inf")                       # the rejected one of pair 6
    f = lm.preference_forward(x, lab(labels), up(ref), pairs, 0.1, 0.0)
    d = lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs)
    torch.cuda.synchronize()
    keep = np.where(labels < V, labels, 0)
    with np.errstate(all="ignore"):
        loss, rewards, logp, lse, coef = so.preference(down(x), keep, ref, pairs, 0.1, 0.0)
    got = down(f.loss)
    assert np.isnan(got[1:5]).all()
    assert np.isfinite(got[0]) and abs(got[0] - loss[0]) < 1e-5
    assert np.isposinf(got[5]) and got[6] == 0.0
    assert down(f.coef)[5, 0] == np.float32(-0.1) and down(f.coef)[6, 0] == 0.0
    g = down(d)
    assert np.isnan(g[2:10:2]).all()
    for t in (0, 1, 10, 11, 12, 13):
        assert np.isfinite(g[t]).all()
    assert not g[0, :5].any()                      # masked entries get exactly nothing
    assert g[10, 5] < 0 and not g[12:14].any()
    lp, z = lm.token_logprob(x, lab(labels))
    torch.cuda.synchronize()
    assert np.isneginf(down(lp)[10]) and np.isnan(down(lp)[[2, 4, 6, 8]]).all() and np.isfinite(down(z)[8])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows(dtype):
    """Rows a step apart that shifts them off 16 bytes, differently in the logits and in their gradient."""
    import torch
    import lora_co_serving_gb300 as lm
    T, pairs = PAIRS["ragged"]
    for V in (1, 5, 203, 1031):
        x, labels, ref = case(V, T, V, dtype)
        wide = torch.full((T, V + 3), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, 2:2 + V] = x
        out = torch.full((T, V + 6), 9.0, dtype=x.dtype, device="cuda")
        f = lm.preference_forward(x, lab(labels), up(ref), pairs)
        h = lm.preference_forward(wide[:, 2:2 + V], lab(labels), up(ref), pairs)
        d = lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs)
        e = lm.preference_backward(wide[:, 2:2 + V], lab(labels), f.lse, f.coef, pairs, dlogits=out[:, 3:3 + V])
        torch.cuda.synchronize()
        # the order of a row's sum follows its alignment: equal within the float32 bounds above
        assert (np.abs(down(f.lse) - down(h.lse)) <= 2.0 ** -18).all()
        assert torch.equal(d, e)
        assert (out[:, :3] == 9.0).all() and (out[:, 3 + V:] == 9.0).all()


def test_repeats_bit_for_bit_on_a_stream_and_in_a_graph():
    import torch
    import lora_co_serving_gb300 as lm
    T, pairs = PAIRS["many"]
    x, labels, ref = case(4, T, 5003, "bf16")
    labels, ref = lab(labels), up(ref)
    f = lm.preference_forward(x, labels, ref, pairs)
    d = lm.preference_backward(x, labels, f.lse, f.coef, pairs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = lm.preference_forward(x, labels, ref, pairs, stream=side)
    e = lm.preference_backward(x, labels, g.lse, g.coef, pairs, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(f, g)) and torch.equal(d, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = lm.preference_forward(x, labels, ref, pairs)
        k = lm.preference_backward(x, labels, h.lse, h.coef, pairs)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(f, h)) and torch.equal(d, k)


def test_large_logits_and_certain_rows():
    """Logits of thousands, and a row that is certain of its label: the loss keeps its digits."""
    import torch
    import lora_co_serving_gb300 as lm
    x = np.zeros((4, 1000), np.float32)
    x[0] = 5000.0 + np.arange(1000)
    x[1, 3] = 60.0
    x[2] = -7000.0
    x[3, 9] = -1e4
    labels = np.array([999, 3, 17, 8])
    f = lm.token_logprob(up(x), lab(labels))
    torch.cuda.synchronize()
    lse = so.log_softmax_parts(x.astype(np.float64))
    want = x[np.arange(4), labels].astype(np.float64) - lse
    assert (np.abs(down(f[1]) - lse) <= 2.0 ** -23 * np.abs(lse) + 2.0 ** -18).all()
    assert (np.abs(down(f[0]) - want) <= 2.0 ** -22 * np.abs(lse) + 2.0 ** -17).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 1000, 9001])
def test_rows_masked_with_a_finite_value(V, dtype):
    """A mask of the type's lowest value (or -1e9) over most of a row leaves the rest as it is; over the whole row every
    entry is as likely as any other, and the gradient stays finite."""
    import torch
    import lora_co_serving_gb300 as lm
    low = float(torch.finfo({"bf16": torch.bfloat16, "f32": torch.float32}[dtype]).min)
    x = up(np.random.default_rng(V).standard_normal((8, V)), dtype)
    plain = x.clone()
    keep = 3
    x[0, keep:], plain[0, keep:] = low, float("-inf")
    x[1, keep:], plain[1, keep:] = -1e9, float("-inf")
    x[2] = low
    x[3] = -1e9
    x[4], x[4, 1] = low, low / 2
    x[5] = 3e38
    labels = np.array([1, 2, 0, V - 1, 1, 2, 0, 1])
    lp, lse = lm.token_logprob(x, lab(labels))
    same = lm.token_logprob(plain, lab(labels))
    f = lm.preference_forward(x, lab(labels), up(np.zeros(8)), [(0, 4, 4, 4)])
    d = lm.preference_backward(x, lab(labels), f.lse, f.coef, [(0, 4, 4, 4)])
    torch.cuda.synchronize()
    for t in (0, 1, 6, 7):
        assert lp[t] == same[0][t] and lse[t] == same[1][t]
    # far rows: logarithms of sums of exact exponentials (0 or 1), a few units in the last place; at -1e9 the row's
    # exponent n is a number near 2^30.4, n log(2) is cut at 2^-24 of n (log(2) - its high part) = 2^11: 2^-12
    assert np.abs(down(lp)[[2, 3, 5]] + np.log(V)).max() <= 2.0 ** -11
    assert abs(down(lp)[4]) <= 2.0 ** -20
    assert np.isfinite(down(f.loss)).all() and np.isfinite(down(d)).all()


def test_offsets_past_32_bits():
    import torch
    import lora_co_serving_gb300 as lm
    T, V = 17003, 128256
    x = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 2048):
        x[t:t + 2048].normal_(generator=torch.Generator(device="cuda").manual_seed(t))
    pairs = [(0, 8000, 8000, T - 8000)]
    rng = np.random.default_rng(0)
    labels = np.where(rng.random(T) < 0.01, rng.integers(0, V, T), -1)
    rows = [0, 16743, 16744, T - 1]
    labels[rows] = [3, V - 1, 70000, 12]
    ref = np.zeros(T)
    f = lm.preference_forward(x, lab(labels), up(ref), pairs)
    d = lm.preference_backward(x, lab(labels), f.lse, f.coef, pairs, dlogits=x.clone())
    torch.cuda.synchronize()
    for t in rows:
        v = down(x[t:t + 1])
        z = so.log_softmax_parts(v)[0]
        assert abs(down(f.lse)[t] - z) <= 2.0 ** -18
        k = down(f.coef)[0, 0 if t < 8000 else 1]
        want = -k * np.exp(v[0] - down(f.lse)[t])
        want[labels[t]] += k
        assert (np.abs(down(d[t]) - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -16 * abs(k) * (want == want.max())
                + 1e-37).all()
