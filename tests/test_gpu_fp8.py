"""The 8-bit block format, its products and the MLP activation's checkpoint against their definitions in float64.

Tolerances.  Codes and scales are exact: a scale is a power of two, a code one rounding.  An output of 16 bits is a
float32 value rounded once: 2^-9 of itself, taken as 2^-8.  A float32 sum of n products is within n 2^-24 of the sum of
their magnitudes; matrix units may cut (rather than round) partial sums at a few bits more than 24, so the sums here
get (128 + blocks) 2^-22 of the sum of magnitudes.  The activation's float32 values come from an exponential and a
quotient, each a few units in the last place: 2^-17 covers e^-g for |g| <= 30 (its argument is rounded once, to
30 * 2^-24, before the power is taken).
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


def up(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(
        {"bf16": torch.bfloat16, "f32": torch.float32}[dtype])


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes_of(q):
    """float64 code values -> float8 tensor (exact)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(q, np.float32)).cuda().to(torch.float8_e4m3fn)


def same(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=True)


def draw(rng, T, K, spread=3.0):
    """Rows of very different magnitude, blocks of zeros, and values at the edges of the format."""
    x = rng.standard_normal((T, K)) * np.exp(spread * rng.standard_normal((T, 1)))
    x[rng.random((T, K)) < 0.05] = 0.0
    if T > 2 and K > 128:
        x[1, :128] = 0.0
        x[2, :128] = 448.0 * rng.choice([1.0, -0.5, 2.0 ** -9, 17.0 / 448, 2.0 ** -12], 128)
    return x


# ------------------------------------------------------------------------------------------------------- quantizers
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K", [(1, 16), (3, 32), (7, 144), (5, 2064), (130, 4096), (1, 28672), (33, 2176)])
def test_quantize_is_exact(T, K, dtype):
    import torch
    import lora_co_serving_gb300 as lm
    x = up(draw(np.random.default_rng(T * 7 + K), T, K), dtype)
    codes, scales = lm.fp8_quantize(x)
    torch.cuda.synchronize()
    q, s = so.quantize(down(x))
    assert same(down(scales), s)
    assert same(down(codes), q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_extremes(dtype):
    import torch
    import lora_co_serving_gb300 as lm
    x = np.zeros((10, 144), np.float32)
    x[1] = 1e-38
    x[2, 5] = 3.3e38
    x[3] = 2.0 ** -100
    x[4] = 1.75
    x[5] = 1.7578125                       # just above 1.75: the next power of two
    x[6, 130] = np.inf
    x[7, 3] = np.nan
    x[8, 0], x[8, 1] = -np.inf, 1.0
    x[9] = -448.0
    t = up(x, dtype)
    codes, scales = lm.fp8_quantize(t)
    torch.cuda.synchronize()
    q, s = so.quantize(down(t))
    assert same(down(scales), s)
    bad = np.isnan(so.spread_rows(s, 144))
    assert bad.sum() == 16 + 128 + 128
    assert same(down(codes)[~bad], q[~bad])
    assert np.isnan(down(codes) * so.spread_rows(down(scales), 144))[bad].all()


def test_quantize_strided():
    import torch
    import lora_co_serving_gb300 as lm
    big = up(draw(np.random.default_rng(2), 9, 400), "bf16")
    x = big[::2, 16:16 + 272]
    out = torch.full((5, 288), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    codes, scales = lm.fp8_quantize(x, codes=out[:, :272])
    torch.cuda.synchronize()
    q, s = so.quantize(down(x))
    assert same(down(codes), q) and same(down(scales), s)
    assert (out[:, 272:].view(torch.uint8) == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (130, 144), (520, 1040)])
def test_quantize_weight_is_exact(N, K, dtype):
    import torch
    import lora_co_serving_gb300 as lm
    w = up(draw(np.random.default_rng(N + K), N, K, 1.0), dtype)
    codes, scales = lm.fp8_quantize_weight(w)
    torch.cuda.synchronize()
    q, s = so.quantize_weight(down(w))
    assert same(down(scales), s) and same(down(codes), q)
    # the transposed weight's blocks are the transposed blocks
    if N % 16 == 0:
        ct, st = lm.fp8_quantize_weight(w.t().contiguous())
        torch.cuda.synchronize()
        assert same(down(ct), q.T) and same(down(st), s.T)


# ---------------------------------------------------------------------------------------------------------- products
def product(seed, T, K, N, dtype, x_spread=1.0):
    rng = np.random.default_rng(seed)
    x = draw(rng, T, K, x_spread)
    wq, wsc = so.quantize_weight(rng.standard_normal((N, K)) / np.sqrt(K))
    wsc = (wsc * rng.uniform(0.4, 2.3, wsc.shape)).astype(np.float32)       # scales need not be powers of two
    if dtype == "fp8":
        xq, xs = so.quantize(x)
        xs = (xs * rng.uniform(0.4, 2.3, xs.shape)).astype(np.float32)
        args = (codes_of(xq), codes_of(wq), up(wsc, "f32")), dict(x_scales=up(xs, "f32"))
    else:
        t = up(x, dtype)
        xq, xs = so.quantize(down(t))
        args = (t, codes_of(wq), up(wsc, "f32")), {}
    return args, xq, xs.astype(np.float64), wq, wsc.astype(np.float64)


def expect(xq, xs, wq, wsc):
    (T, K), N = xq.shape, wq.shape[0]
    xv, wv = xq * so.spread_rows(xs, K), wq * so.spread_weight(wsc, N, K)
    ref = xv @ wv.T
    tol = 2.0 ** -8 * np.abs(ref) + (128 + so.blocks(K)) * 2.0 ** -22 * (np.abs(xv) @ np.abs(wv).T) + 1e-37
    return ref, tol


SHAPES = [(1, 16, 8), (1, 4096, 512), (2, 128, 128), (3, 144, 264), (7, 272, 136), (8, 1040, 520), (15, 384, 1000),
          (16, 2048, 256), (17, 512, 392), (31, 128, 2048), (32, 1296, 128), (33, 640, 640), (63, 256, 72),
          (64, 4096, 256), (65, 1552, 344), (100, 896, 256), (127, 144, 1032), (128, 1024, 384), (129, 528, 512),
          (200, 2048, 520), (255, 640, 256), (256, 512, 776), (257, 1168, 264), (300, 128, 1288), (511, 384, 512),
          (513, 272, 904), (1000, 2304, 256), (2049, 144, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear(T, K, N, dtype):
    import torch
    import lora_co_serving_gb300 as lm
    (args, kw), *vals = product(T + K + N, T, K, N, dtype)
    y = lm.fp8_linear(*args, check_status=True, **kw)
    assert y.dtype == torch.bfloat16 and y.shape == (T, N)
    ref, tol = expect(*vals)
    assert (np.abs(down(y) - ref) <= tol).all(), np.max(np.abs(down(y) - ref) / tol)


# tiles of one CTA and of two, of 128 outputs and of 256, in one round and in several, whole and cut along K, with an
# even and an odd number of blocks
@pytest.mark.parametrize("T,K,N", [(300, 1552, 136), (2100, 144, 2056), (777, 5136, 2712), (70, 1552, 136),
                                   (300, 144, 12296), (2100, 144, 4104), (300, 5136, 2056), (777, 2064, 6152),
                                   (300, 8208, 2056), (777, 4112, 6152), (129, 1552, 136), (129, 1680, 136),
                                   (385, 144, 12296), (300, 2704, 2704), (900, 4112, 2712), (129, 144, 12296),
                                   (777, 144, 9224), (385, 2704, 12296), (129, 8208, 6152), (385, 4112, 12296)])
def test_linear_tile_shapes(T, K, N):
    import torch
    import lora_co_serving_gb300 as lm
    (args, kw), *vals = product(T + K + N, T, K, N, "fp8")
    y = lm.fp8_linear(*args, check_status=True, **kw)
    ref, tol = expect(*vals)
    assert (np.abs(down(y) - ref) <= tol).all(), np.max(np.abs(down(y) - ref) / tol)
    assert torch.equal(y, lm.fp8_linear(*args, **kw))


@pytest.mark.parametrize("T", [1, 5, 40, 130, 300])
def test_linear_strides_and_edges(T):
    """Rows of x and y lie apart; nothing beyond y's columns is written; another stream; repeated calls agree."""
    import torch
    import lora_co_serving_gb300 as lm
    K, N = 656, 392
    (args, _), *vals = product(T, T, K, N, "bf16")
    wide = torch.full((T, K + 48), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + K] = args[0]
    out = torch.full((T + 1, N + 24), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lm.fp8_workspace_size(T, K, N), dtype=torch.uint8, device="cuda").fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = lm.fp8_linear(wide[:, 16:16 + K], *args[1:], y=out[:T, 8:8 + N], workspace=ws, stream=side)
    side.synchronize()
    ref, tol = expect(*vals)
    assert (np.abs(down(y) - ref) <= tol).all()
    guard = out.clone()
    guard[:T, 8:8 + N] = -7.0
    assert (guard == -7.0).all()
    for _ in range(3):
        again = lm.fp8_linear(args[0], *args[1:])
        assert torch.equal(again, y)


@pytest.mark.parametrize("T", [3, 48, 140])
def test_linear_rows_are_independent(T):
    """A NaN or infinity in one row of x stays in that row; a row's result depends on no other row."""
    import torch
    import lora_co_serving_gb300 as lm
    K, N = 400, 264
    (args, _), *_ = product(9 + T, T, K, N, "bf16")
    base = lm.fp8_linear(*args)
    x = args[0].clone()
    x[1, 7], x[2, 399] = float("nan"), float("inf")
    y = lm.fp8_linear(x, *args[1:])
    torch.cuda.synchronize()
    assert torch.isnan(y[1:3].float()).all()
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[keep], base[keep])


def test_linear_extreme_scales():
    """Products whose scales lie near the ends of float32's range do not overflow on the way."""
    import torch
    import lora_co_serving_gb300 as lm
    T, K, N = 20, 256, 128
    (args, _), xq, xs, wq, wsc = product(5, T, K, N, "fp8")
    for big, small in ((2.0 ** 90, 2.0 ** -92), (2.0 ** -90, 2.0 ** 85)):
        y = lm.fp8_linear(codes_of(xq), codes_of(wq), up(wsc * small, "f32"), x_scales=up(xs * big, "f32"))
        torch.cuda.synchronize()
        ref, tol = expect(xq, xs * big, wq, wsc * small)
        assert (np.abs(down(y) - ref) <= tol).all()


def test_linear_empty_and_graph():
    import torch
    import lora_co_serving_gb300 as lm
    K, N = 512, 256
    (args, _), *vals = product(77, 24, K, N, "bf16")
    assert lm.fp8_linear(args[0][:0], *args[1:]).shape == (0, N)
    x = args[0].clone()
    y = torch.zeros(24, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lm.fp8_workspace_size(24, K, N), dtype=torch.uint8, device="cuda")
    lm.fp8_linear(x, *args[1:], y=y, workspace=ws)
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.fp8_linear(x, *args[1:], y=y, workspace=ws)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    x.mul_(2.0)                               # scales follow the new contents: exactly twice the result
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, 2 * want)


def test_linear_offsets_past_32_bits():
    """An output of more than 2^31 elements (4.6 GB): rows on both sides of the boundary."""
    import torch
    import lora_co_serving_gb300 as lm
    T, K, N = 70001, 128, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    w, wsc = lm.fp8_quantize_weight(torch.randn(N, K, device="cuda", generator=g))
    y = lm.fp8_linear(x, w, wsc, check_status=True)
    pick = [0, 1, 65535, 65536, 65537, T - 2, T - 1]
    xq, xs = so.quantize(down(x[pick]))
    ref, tol = expect(xq, xs, down(w), down(wsc))
    assert (np.abs(down(y[pick]) - ref) <= tol).all()


# ------------------------------------------------------------------------------------------------------------ swiglu
TABLES = [
    [],
    [(0, 1, 0, 1)],
    [(0, 7, 3, 0)],
    [(0, 5, -1, 0), (5, 1, 0, 1), (6, 0, 0, 1), (6, 12, 2, 1), (18, 3, 4, 0)],
    [(40, 31, 0, 1), (0, 40, 1, 0), (71, 2, -1, 0)],
    [(i, 1, 0, i % 2) for i in range(96)],
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fp8_out", [False, True])
@pytest.mark.parametrize("I", [8, 128, 136, 2056, 2176])
@pytest.mark.parametrize("table", range(len(TABLES)))
def test_swiglu_forward(table, I, fp8_out, dtype):
    import torch
    import lora_co_serving_gb300 as lm
    if fp8_out and I % 16:
        I += 8
    segs = TABLES[table]
    T = sum(s[1] for s in segs)
    rng = np.random.default_rng(table * 100 + I)
    gu = up(rng.standard_normal((T, 2 * I)) * 4.0, dtype)
    h, (ck, cs) = lm.swiglu_forward(gu, segs, checkpoint=True, fp8_out=fp8_out)
    plain = lm.swiglu_forward(gu, fp8_out=fp8_out)
    torch.cuda.synchronize()
    x = down(gu)
    ref = so.swiglu(x)
    if fp8_out:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(h, plain))
        q, s = so.quantize(ref)
        # a value within 2^-17 of a rounding boundary (or a block whose largest is, of a power of two) may go either way
        same_scale = down(h[1]) == s
        assert same_scale.mean() > 0.99 or same_scale.size < 100 and same_scale.mean() > 0.9 or T == 0
        err = np.abs(down(h[0]) * so.spread_rows(down(h[1]), I) - ref)
        assert (err <= 2.0 ** -4 * np.abs(ref) * 1.001 + 2.0 ** -10 * 2 * so.spread_rows(s, I)).all()
        exact = (down(h[0]) == q) & so.spread_rows(same_scale.astype(float), I).astype(bool)
        assert exact.mean() > 0.98 if exact.size > 1000 else True
    else:
        assert torch.equal(h, plain)
        tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -17) * np.abs(ref) + 1e-37
        assert (np.abs(down(h) - ref) <= tol).all()
    rows = np.concatenate([np.arange(a, a + n) for a, n, _, tr in sorted(segs) if tr] or [np.zeros(0, int)])
    assert ck.shape == (len(rows), 2 * I)
    for half in range(2):
        q, s = so.quantize(x[rows.astype(int), half * I:(half + 1) * I])
        nb = so.blocks(I)
        assert same(down(cs)[:, half * nb:(half + 1) * nb], s)
        assert same(down(ck)[:, half * I:(half + 1) * I], q)


def test_swiglu_forward_extremes():
    """Large gates saturate without overflowing; a NaN stays where it is (its block, in the checkpoint)."""
    import torch
    import lora_co_serving_gb300 as lm
    I = 256
    gu = np.ones((4, 2 * I), np.float32)
    gu[0, :I] = np.linspace(-3e4, 3e4, I)
    gu[1, 3] = np.nan
    gu[2, I + 200] = np.inf
    t = up(gu, "f32")
    h, (ck, cs) = lm.swiglu_forward(t, [(0, 4, 0, 1)], checkpoint=True)
    torch.cuda.synchronize()
    ref = so.swiglu(gu.astype(np.float64))
    got = down(h)
    fine = np.isfinite(ref)
    assert same(np.isfinite(got), fine)
    assert (np.abs(got - ref)[fine] <= 2.0 ** -17 * np.abs(ref)[fine] + 1e-30).all()
    assert np.isnan(down(cs)[1, 0]) and np.isfinite(down(cs)[1, 1:]).all()
    assert np.isnan(down(cs)[2, 3]) and np.isfinite(down(cs)[2, :3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,I", [(1, 8), (3, 136), (17, 2056), (130, 128), (64, 2176)])
def test_swiglu_backward(R, I, dtype):
    import torch
    import lora_co_serving_gb300 as lm
    rng = np.random.default_rng(R + I)
    (gq, gs), (uq, us) = so.quantize(4.0 * rng.standard_normal((R, I))), so.quantize(draw(rng, R, I, 1.0))
    dh = up(rng.standard_normal((R, I)) * 1e-3, dtype)
    saved = (codes_of(np.concatenate([gq, uq], 1)), up(np.concatenate([gs, us], 1), "f32"))
    got = lm.swiglu_backward(saved, dh)
    torch.cuda.synchronize()
    ref = so.swiglu_grad(gq * so.spread_rows(gs, I), uq * so.spread_rows(us, I), down(dh))
    g = gq * so.spread_rows(gs, I)
    # 1 + g (1 - sig) cancels where it passes zero (g = -1.28): error relative to its terms there
    size = np.concatenate([np.abs(down(dh) * uq * so.spread_rows(us, I)) * so.sigmoid(g) * (1 + np.abs(g)),
                           np.abs(ref[:, I:])], 1)
    tol = (2.0 ** -8 if dtype == "bf16" else 0.0) * np.abs(ref) + 2.0 ** -17 * size + 1e-37
    assert (np.abs(down(got) - ref) <= tol).all()
    if I % 128 == 0:
        q, s = lm.swiglu_backward(saved, dh, fp8_out=True)
        torch.cuda.synchronize()
        v = down(q) * so.spread_rows(down(s), 2 * I)
        assert (np.abs(v - ref) <= 2.0 ** -4 * 1.001 * np.abs(ref) + 2.0 ** -9 * so.spread_rows(down(s), 2 * I)).all()
        big = np.abs(ref.reshape(R, -1, 128)).max(2)
        assert (448 * down(s) >= big * (1 - 1e-4)).all() and (224 * down(s) < big * (1 + 1e-4) + 2.0 ** -100).all()


def test_swiglu_gradient_is_the_differences():
    """(h(g + d) - h(g - d)) / 2d of the definition at the checkpoint's values, against the kernel's gradient."""
    import torch
    import lora_co_serving_gb300 as lm
    R, I = 6, 128
    rng = np.random.default_rng(4)
    gu = up(rng.standard_normal((R, 2 * I)) * 2.0, "f32")
    _, saved = lm.swiglu_forward(gu, [(0, R, 0, 1)], checkpoint=True)
    dh = up(rng.standard_normal((R, I)), "f32")
    got = down(lm.swiglu_backward(saved, dh))
    torch.cuda.synchronize()
    v = np.concatenate([down(saved[0])[:, :I] * so.spread_rows(down(saved[1])[:, :1], I),
                        down(saved[0])[:, I:] * so.spread_rows(down(saved[1])[:, 1:], I)], 1)
    d = 1e-5
    num = np.empty_like(got)
    for half in range(2):
        step = np.zeros_like(v)
        step[:, half * I:(half + 1) * I] = d
        num[:, half * I:(half + 1) * I] = down(dh) * (so.swiglu(v + step) - so.swiglu(v - step)) / (2 * d)
    # differences of second order: d^2 times a third derivative below 4 (of order 1 values), and 1e-16 / d of rounding
    assert (np.abs(got - num) <= 2.0 ** -16 * (np.abs(num) + np.abs(v) * np.abs(np.tile(down(dh), 2))) + 1e-7).all()


def test_swiglu_strides_and_in_step():
    """Rows apart in every argument; the checkpoint feeds the backward on another stream."""
    import torch
    import lora_co_serving_gb300 as lm
    T, I = 37, 264
    rng = np.random.default_rng(8)
    wide = up(rng.standard_normal((T, 2 * I + 16)), "bf16")
    gu = wide[:, 8:8 + 2 * I]
    segs = [(0, 10, 0, 0), (10, 21, 1, 1), (31, 6, -1, 0)]
    out = torch.full((T, I + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    h, saved = lm.swiglu_forward(gu, segs, checkpoint=True, h=out[:, :I])
    ref = lm.swiglu_forward(gu.contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dh = torch.full((21, I + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    dh[:, :I] = ref[10:31]
    side.wait_stream(torch.cuda.current_stream())
    buf = torch.full((21, 2 * I + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    d = lm.swiglu_backward(saved, dh[:, :I], dgu=buf[:, :2 * I], stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(h, ref) and (out[:, I:] == 3.0).all() and (buf[:, 2 * I:] == 5.0).all()
    assert torch.equal(d, lm.swiglu_backward(saved, ref[10:31].contiguous()))


def test_swiglu_offsets_past_32_bits():
    """gate|up of more than 2^31 elements, the checkpoint of its last rows."""
    import torch
    import lora_co_serving_gb300 as lm
    T, I = 41003, 28672
    gu = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 4096):
        gu[t:t + 4096].normal_(generator=torch.Generator(device="cuda").manual_seed(t))
    segs = [(0, 5, 0, 1), (5, T - 45, 1, 0), (T - 40, 40, 0, 1)]
    h, saved = lm.swiglu_forward(gu, segs, checkpoint=True)
    torch.cuda.synchronize()
    for t in (0, 37449, 37450, T - 1):
        ref = so.swiglu(down(gu[t:t + 1]))
        assert (np.abs(down(h[t:t + 1]) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-37).all()
    q, s = so.quantize(down(gu[T - 1:, :I]))
    assert same(down(saved[0][44:, :I]), q) and same(down(saved[1][44:, :224]), s)
