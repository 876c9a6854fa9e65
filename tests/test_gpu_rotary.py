"""Rotary positions with norms, forward and backward, and the paged cache's rows, against float64 on the CPU.

Tolerances, in half steps u = 2^-24 of float32, before the one rounding to the output's type:
  norm      a sum of at most 256 squares (16 in a lane, then 4 shuffles: 21 roundings, halved by the root), the reciprocal
            root (2 units, 4 u), two products: 18 u of the value
  angle     a whole number of 2^-32 turns of at most an eighth: 1.5e-9 + half a step of pi / 4, 1 u; sine and cosine 2 units
            (4 u): 5 u; three roundings in a c - b s.  Together 26 u (|a| + |b|).  REACH = 32.
  gradient  the same for g; then w g, its sum with x r (21), and f (w g - x r mean): 64 u of f (|w g| + |x r| mean |w g x r|)
  weights   a term g x r is 50 u off; a lane adds at most 40 of them in the cases here, then come the 8 x 8 lanes and warps
            of a CTA, and 10 + 32 of the CTAs: at most 110 u, of a sum that has as many.  Together 160 u of the magnitudes.
"""
import pytest
import torch

import lora_co_serving_gb300 as lm
from attention_oracle import (E4, EPS, U, angles, frequencies, from_pairs, half_step, normed, pairs, quantized, reach, turned)

pytestmark = pytest.mark.gpu
REACH, GRAD, WGRAD = 32 * U, 64 * U, 160 * U


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(g, T, cols, dtype, pad=0, spread=1.0):
    """T rows of cols, in a wider matrix where pad > 0 (whose other columns are NaN); its float64 values."""
    x = (torch.randn(T, cols, generator=g) * torch.exp(spread * torch.randn(T, 1, generator=g))).to(dtype)
    wide = torch.full((T, cols + pad), float("nan"), dtype=dtype)
    wide[:, :cols] = x
    return wide.cuda()[:, :cols], x.double()


class Case:
    def __init__(self, T, hq, hk, D, dtype, rot=None, interleaved=False, norm="both", pad=0, base=10000.0, seed=0):
        g = gen(seed + T)
        self.T, self.hq, self.hk, self.D, self.dtype, self.interleaved = T, hq, hk, D, dtype, interleaved
        self.rot = D if rot is None else rot
        self.x, x = rows(g, T, (hq + hk) * D, dtype, pad)
        self.x64 = x.reshape(T, hq + hk, D)
        self.positions = torch.randint(0, 2 ** 20, (T,), generator=g)
        if T > 2:
            self.positions[1], self.positions[2] = 0, 2 ** 31 + 12345
        self.freqs = frequencies(self.rot, base)
        self.turns = lm.rotary_turns(self.rot, base) if self.rot else None
        self.angle = angles(self.positions, self.freqs)
        w = [(1.0 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)]
        self.wq, self.wk = w[0] if norm in ("both", "q") else None, w[1] if norm in ("both", "k") else None
        self.w64 = [None if t is None else t.double() for t in (self.wq, self.wk)]
        self.args = (self.positions.cuda() if self.rot else None, self.turns, hq, hk)
        self.kw = dict(q_weight=None if self.wq is None else self.wq.cuda(), interleaved=interleaved,
                       k_weight=None if self.wk is None else self.wk.cuda())

    def parts(self, x):
        return x[:, :self.hq], x[:, self.hq:]

    def result(self):
        """(queries and keys [T, heads, D], what their errors are relative to)."""
        n = torch.cat([normed(x, w) for x, w in zip(self.parts(self.x64), self.w64)], 1)
        if not self.rot:
            return n, n.abs()
        return turned(n, self.angle, self.rot, self.interleaved), reach(n, self.rot, self.interleaved)

    def gradient(self, dout):
        """(dx, its magnitudes, [dwq, dwk], their magnitudes)."""
        g = dout.reshape(self.T, -1, self.D)
        big = g.abs()
        if self.rot:
            g, big = turned(g, -self.angle, self.rot, self.interleaved), reach(g, self.rot, self.interleaved)
        dx, mag, dw, wmag = [], [], [], []
        for x, gi, bi, w in zip(self.parts(self.x64), self.parts(g), self.parts(big), self.w64):
            if w is None:
                dx.append(gi), mag.append(bi), dw.append(None), wmag.append(None)
                continue
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            n = x * r
            dx.append(r * (w * gi - n * (w * gi * n).mean(-1, keepdim=True)))
            mag.append(r * (w.abs() * bi + n.abs() * (w.abs() * bi * n.abs()).mean(-1, keepdim=True)))
            dw.append((gi * n).sum((0, 1)))
            wmag.append((bi * n.abs()).sum((0, 1)))
        return torch.cat(dx, 1).reshape(self.T, -1), torch.cat(mag, 1).reshape(self.T, -1), dw, wmag


def close(got, ref, tol):
    got = got.cpu().double().reshape(ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%d of %d off, worst %.3g times the tolerance" % (
        bad.sum(), bad.numel(), ((got - ref).abs() / tol.clamp(min=1e-300)).max())


BF, F32 = torch.bfloat16, torch.float32
CASES = [
    dict(T=1, hq=32, hk=8, D=128, dtype=BF),
    dict(T=5, hq=4, hk=2, D=64, dtype=F32, pad=64),
    dict(T=33, hq=3, hk=1, D=256, dtype=BF, rot=64, pad=8),
    dict(T=17, hq=1, hk=1, D=16, dtype=F32),
    dict(T=40, hq=2, hk=1, D=80, dtype=BF, norm="q"),
    dict(T=9, hq=14, hk=2, D=64, dtype=F32, rot=32, interleaved=True, norm="none"),
    dict(T=21, hq=5, hk=5, D=96, dtype=F32, interleaved=True, base=500000.0),
    dict(T=300, hq=28, hk=4, D=128, dtype=BF, pad=512),
    dict(T=260, hq=16, hk=2, D=128, dtype=F32, norm="k"),
    dict(T=64, hq=2, hk=2, D=48, dtype=BF, rot=0),
    dict(T=700, hq=8, hk=8, D=32, dtype=BF, rot=16),
]


def ids(c):
    return "-".join(str(v).replace("torch.", "") for v in c.values())


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_forward(c):
    k = Case(**c)
    y, mag = k.result()
    before = k.x.clone()
    out = lm.rotary_forward(k.x, *k.args, **k.kw)
    close(out, y.reshape(k.T, -1), (half_step(k.dtype) * y.abs() + REACH * mag).reshape(k.T, -1))
    assert torch.equal(k.x, before)
    again = lm.rotary_forward(k.x, *k.args, **k.kw, out=k.x)       # in place, in its wider rows
    assert again.data_ptr() == k.x.data_ptr() and torch.equal(out, k.x)


# rows and heads enough that a warp takes several rows, and chunks of several steps
MANY = [dict(T=3000, hq=12, hk=4, D=128, dtype=F32), dict(T=2500, hq=30, hk=3, D=64, dtype=BF), dict(T=1500, hq=6, hk=6, D=256, dtype=F32),
        dict(T=2600, hq=9, hk=2, D=80, dtype=F32, interleaved=True, pad=16), dict(T=1700, hq=72, hk=1, D=96, dtype=BF, rot=32)]


@pytest.mark.parametrize("c", MANY, ids=ids)
def test_forward_of_many_rows(c):
    test_forward(c)


@pytest.mark.parametrize("c", MANY, ids=ids)
def test_backward_of_many_rows(c):
    test_backward(c)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_backward(c):
    k = Case(**c)
    dout, d64 = rows(gen(7), k.T, (k.hq + k.hk) * k.D, k.dtype, c.get("pad", 0), 0.5)
    dx, mag, dw, wmag = k.gradient(d64)
    norm = k.wq is not None or k.wk is not None
    got, gq, gk = lm.rotary_backward(k.x if norm else None, *k.args, dout, **k.kw, weight_grads=True)
    close(got, dx, half_step(k.dtype) * dx.abs() + GRAD * mag)
    for g, ref, m in ((gq, dw[0], wmag[0]), (gk, dw[1], wmag[1])):
        assert (g is None) == (ref is None)
        if g is not None:
            close(g, ref, WGRAD * m)
    alone = lm.rotary_backward(k.x if norm else None, *k.args, dout, **k.kw)
    assert torch.equal(alone, got)
    _, gq2, gk2 = lm.rotary_backward(k.x if norm else None, *k.args, dout, **k.kw, weight_grads=True)
    assert all(a is None or torch.equal(a, b) for a, b in ((gq, gq2), (gk, gk2)))
    lm.rotary_backward(k.x if norm else None, *k.args, dout, **k.kw, dx=dout)
    assert torch.equal(dout, got)


def test_gradient_against_differences():
    """Derivative of sum(out * dout) along a direction: central differences of the float64 form, which the forward is held to."""
    k = Case(T=6, hq=3, hk=2, D=32, dtype=F32, rot=16, seed=3)
    dout, d64 = rows(gen(8), 6, 160, F32)
    dx, dwq, dwk = lm.rotary_backward(k.x, *k.args, dout, **k.kw, weight_grads=True)
    g = gen(9)
    d = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (k.x64, k.w64[0], k.w64[1])]

    def f(h):
        x = k.x64 + h * d[0]
        n = torch.cat([normed(x[:, :3], k.w64[0] + h * d[1]), normed(x[:, 3:], k.w64[1] + h * d[2])], 1)
        return (turned(n, k.angle, 16, False).reshape(6, -1) * d64).sum()

    h = 1e-5
    slope = (f(h) - f(-h)) / (2 * h)
    got = sum((a.cpu().double().reshape(b.shape) * b).sum() for a, b in ((dx, d[0]), (dwq, d[1]), (dwk, d[2])))
    mag = sum((a.cpu().double().reshape(b.shape) * b).abs().sum() for a, b in ((dx, d[0]), (dwq, d[1]), (dwk, d[2])))
    # h^2 third derivatives: 1e-10 of the terms; float64's cancellation 1e-16 / 1e-5; WGRAD of the terms
    assert abs(got - slope) <= (1e-8 + WGRAD) * mag


def test_positions_wrap_exactly():
    """Far and negative positions: a row turned by p and a row turned by -p are each other's inverse."""
    x = torch.randn(4, 2 * 64, generator=gen(1)).cuda()
    p = torch.tensor([2 ** 40 + 3, -5, 2 ** 62, -(2 ** 50)]).cuda()
    turns = lm.rotary_turns(64, 10000.0)
    there = lm.rotary_forward(x, p, turns, 1, 1)
    back = lm.rotary_forward(there, -p, turns, 1, 1)
    mag = reach(x.cpu().double().reshape(4, 2, 64), 64, False)
    far = from_pairs(*(2 * m for m in pairs(mag, 64, False)), mag[..., 64:], False)
    close(back, x.cpu().double().reshape(4, 2, 64), 2 * REACH * far)


def test_rows_of_extreme_length():
    """Squares past float32's range: zeros; an infinite or NaN element: its own row and head; zeros stay zeros; rows whose
    squares vanish are as long as eps says."""
    turns, w = lm.rotary_turns(64), torch.ones(64, device="cuda")
    x = torch.randn(6, 3 * 64, generator=gen(1)).cuda()
    x[0, :64], x[1, 70], x[2, 130], x[3, :64], x[4, 64:128] = 1e30, float("inf"), float("nan"), 0.0, 1e-30
    p = torch.arange(6).cuda()
    out = lm.rotary_forward(x, p, turns, 2, 1, q_weight=w, k_weight=w).reshape(6, 3, 64)
    assert (out[0, 0] == 0).all() and (out[3, 0] == 0).all() and out[4, 1].abs().max() < 1e-25 and out[4, 1].abs().max() > 0
    hit = torch.zeros(6, 3, dtype=torch.bool)
    hit[1, 1] = hit[2, 2] = True
    assert torch.equal(out.isfinite().all(-1).cpu(), ~hit) and out[2, 2].isnan().all() and out[1, 1].isnan().sum() == 2
    cache = lm.kv_cache(1, 1, 8, 64, torch.float8_e4m3fn)
    lm.rotary_forward(x, p, turns, 2, 1, q_weight=w, k_weight=w, v=x[:, :64], cache=cache, slots=p)
    k, v = lm.cache_read(cache, p, dtype=F32)
    assert k[2].isnan().all() and k[[0, 1, 3, 4, 5]].isfinite().all() and v.isfinite().all()


def test_no_rows():
    turns = lm.rotary_turns(64)
    e = torch.empty(0, 128, dtype=BF, device="cuda")
    p = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    assert lm.rotary_forward(e, p, turns, 1, 1).shape == (0, 128)
    dx, dq, dk = lm.rotary_backward(e, p, turns, 1, 1, e, q_weight=w, weight_grads=True)
    assert dx.shape == (0, 128) and dk is None and (dq == 0).all()
    c = lm.kv_cache(2, 1, 4, 64)
    lm.cache_write(e[:, :64], e[:, :64], c, p)
    assert lm.cache_read(c, p)[0].shape == (0, 64)


# ------------------------------------------------------------------------------------------------------ paged cache
def make_cache(n_pages, heads, page, D, e4m3, layout):
    """A cache whose every byte is marked (0x55), in one of three layouts."""
    dt = torch.float8_e4m3fn if e4m3 else BF
    n = 1 if e4m3 else 2
    if layout == "rows first":
        k, v = (torch.full((n_pages, page, heads, D * n), 0x55, dtype=torch.uint8, device="cuda").view(dt).transpose(1, 2)
                for _ in range(2))
    elif layout == "one buffer":
        both = torch.full((n_pages, 2, heads, page, D * n), 0x55, dtype=torch.uint8, device="cuda").view(dt)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.full((n_pages, heads, page, D * n), 0x55, dtype=torch.uint8, device="cuda").view(dt) for _ in range(2))
    if not e4m3:
        return lm.KVCache(k, v)
    z = torch.full((2, n_pages, page, heads), -7.0, device="cuda")
    return lm.KVCache(k, v, z[0].transpose(1, 2), z[1].transpose(1, 2))


def raw(t):
    return t.contiguous().view(torch.uint8).reshape(*t.shape[:3], -1)


CACHES = [(16, "heads first", 128, 8), (1, "rows first", 64, 3), (13, "one buffer", 80, 5), (64, "rows first", 256, 2),
          (24, "heads first", 16, 1)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["x bf16", "x f32"])
@pytest.mark.parametrize("page,layout,D,heads", CACHES)
def test_cache_rows(page, layout, D, heads, dtype, e4m3):
    T, n_pages = 45, -(-60 // page)
    g = gen(page + D)
    cache = make_cache(n_pages, heads, page, D, e4m3, layout)
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    outside = [0, T - 1, 20]
    for i, s in zip(outside, (-1, n_pages * page, 2 ** 40)):
        slots[i] = s
    k, k64 = rows(g, T, heads * D, dtype, 16)
    v, v64 = rows(g, T, heads * D, dtype, 32, 3.0)
    k[5, :D], k64[5, :D] = 0.0, 0.0
    before = [raw(t).clone() for t in cache[:2]]
    lm.cache_write(k, v, cache, slots.cuda())
    got = lm.cache_read(cache, slots.cuda(), dtype=F32)
    inside = torch.ones(T, dtype=torch.bool)
    inside[outside] = False
    for x64, y in ((k64, got[0]), (v64, got[1])):
        x = x64.reshape(T, heads, D)
        ref = quantized(x)[0] if e4m3 else x.to(BF).double()
        y = y.cpu().double().reshape(T, heads, D)
        assert torch.equal(y[inside], ref[inside])        # one rounding of the input, exactly
        assert (y[outside] == 0).all()
    half = lm.cache_read(cache, slots.cuda())             # both kinds of value are bf16 numbers
    assert all(torch.equal(a.float(), b) for a, b in zip(half, got))
    # rows that no slot named are as they were
    named = torch.zeros(n_pages * page, dtype=torch.bool)
    named[slots[inside]] = True
    for t, b in zip(cache[:2], before):
        same = (raw(t) == b).all(-1).permute(0, 2, 1).reshape(n_pages * page, heads)
        assert same[~named.cuda()].all() and not same[named.cuda()].all(1).any()
    if e4m3:
        for z in cache[2:]:
            kept = (z == -7.0).permute(0, 2, 1).reshape(n_pages * page, heads)
            assert torch.equal(kept, ~named.cuda()[:, None].expand(-1, heads))


def test_cache_reads_repeat_and_special_rows():
    cache = make_cache(4, 2, 8, 64, True, "heads first")
    x = torch.randn(3, 128, generator=gen(2))
    x[0, 5], x[1, 70], x[2, :64] = float("inf"), float("nan"), 0.0
    lm.cache_write(x.cuda(), x.cuda(), cache, torch.tensor([3, 9, 31]).cuda())
    k, v = lm.cache_read(cache, torch.tensor([31, 3, 3, 9, 31]).cuda(), dtype=F32)
    assert torch.equal(k.isnan(), v.isnan())
    n = k.cpu().isnan().reshape(5, 2, 64)
    assert n[1, 0].all() and n[2, 0].all() and n[3, 1].all() and n.sum() == 3 * 64     # a row and head, nothing else
    assert (k[0, :64] == 0).all() and torch.equal(k[0], k[4])
    assert (cache.k_scales[3, 0, 7] == 2.0 ** -108).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("c", [CASES[0], CASES[3], CASES[4], CASES[5], CASES[7]], ids=ids)
def test_forward_into_a_cache(c, e4m3):
    k = Case(**c)
    y, mag = k.result()
    D, n = k.D, k.hq * k.D
    cache = make_cache(6, k.hk, 64, D, e4m3, "rows first")
    slots = torch.randperm(6 * 64, generator=gen(4))[:k.T]
    if k.T > 4:
        slots[4] = -1
    v, v64 = rows(gen(5), k.T, k.hk * D, k.dtype, 64)
    q = lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots.cuda())
    plain = lm.rotary_forward(k.x, *k.args, **k.kw)
    assert q.shape == (k.T, n) and torch.equal(q, plain[:, :n])
    gk, gv = (t.cpu().double().reshape(k.T, k.hk, D) for t in lm.cache_read(cache, slots.cuda(), dtype=F32))
    inside = slots >= 0
    ky, km = y[:, k.hq:], mag[:, k.hq:]
    if e4m3:
        # half a step of a normal number, half of 2^-9 scales below; the scale may be twice the oracle's at a border
        s = quantized(ky)[1][..., None]
        tol = E4 * ky.abs() + 2.0 ** -9 * s + REACH * km
        ref = quantized(v64.reshape(k.T, k.hk, D))[0]
    else:
        tol = half_step(BF) * ky.abs() + REACH * km
        ref = v64.reshape(k.T, k.hk, D).to(BF).double()
    close(gk[inside], ky[inside], tol[inside])
    assert torch.equal(gv[inside], ref[inside]) and (gk[~inside] == 0).all() and (gv[~inside] == 0).all()
    both = lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots.cuda(), keep_keys=True)
    assert torch.equal(both, plain)
    lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots.cuda(), out=k.x[:, :n])
    assert torch.equal(k.x[:, :n], plain[:, :n])


def test_other_stream_and_graph():
    """On a stream that is not current, and captured into a graph whose inputs then change."""
    k = Case(T=50, hq=8, hk=2, D=128, dtype=BF)
    cache = make_cache(3, 2, 32, 128, True, "heads first")
    v, _ = rows(gen(6), 50, 256, BF)
    slots = torch.arange(50).cuda()
    ref = lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots)
    kept = [raw(t).clone() for t in cache[:2]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and all(torch.equal(raw(t), b) for t, b in zip(cache[:2], kept))
    x = k.x.clone()
    dout = torch.randn(50, 1280, generator=gen(10)).to(BF).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lm.rotary_forward(x, *k.args, **k.kw)
        dx, dq, dk = lm.rotary_backward(x, *k.args, dout, **k.kw, weight_grads=True)
        lm.cache_write(out[:, 1024:], v, cache, slots)
        got = lm.cache_read(cache, slots)
    for scale in (1.0, 3.0):
        x.copy_(k.x * scale)
        for _ in range(2):
            graph.replay()
        full = lm.rotary_forward(x, *k.args, **k.kw)
        assert torch.equal(out, full)
        ref = lm.rotary_backward(x, *k.args, dout, **k.kw, weight_grads=True)
        assert all(torch.equal(a, b) for a, b in zip((dx, dq, dk), ref))
        mine = make_cache(3, 2, 32, 128, True, "heads first")
        lm.cache_write(full[:, 1024:], v, mine, slots)
        assert all(torch.equal(a, b) for a, b in zip(got, lm.cache_read(mine, slots)))
