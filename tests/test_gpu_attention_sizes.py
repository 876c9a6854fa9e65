"""Sizes of the attention side that other kernels, or other branches of them, take: heads that fill their lanes in part, rows
enough that a lane or a warp takes several, sequences whose parts are joined in two stages.  Tolerances: those of
test_gpu_decode.py and test_gpu_rotary.py, whose sums these sizes do not exceed."""
import pytest
import torch

import lora_co_serving_gb300 as lm
import test_gpu_decode as decode
import test_gpu_rotary as rotary
from attention_oracle import E4, half_step, quantized
from test_gpu_rotary import BF, F32, REACH, close, gen, ids, make_cache, raw, rows

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["heads first", "rows first"])
@pytest.mark.parametrize("hq,hkv,D", [(6, 2, 144), (24, 2, 144), (5, 5, 208), (33, 3, 208), (8, 1, 240), (37, 1, 240), (4, 2, 112),
                                      (22, 2, 48), (16, 1, 176)])
def test_decode_heads_that_fill_their_warps_in_part(hq, hkv, D, layout, e4m3):
    c = decode.Case([37, 1, 130, 0, 64, 16, 300], hq, hkv, D, page=24, layout=layout, e4m3=e4m3)
    c.check(*c.run())


# one sequence's tiles over 19 CTAs and more: heads of one warp and of two, 8 and 16 query heads at a time, groups in parts
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lengths,hq,hkv,D,window,softcap", [
    ([20000], 10, 2, 256, 0, 0.0), ([9000, 200], 10, 2, 256, 4096, 50.0), ([12000], 24, 2, 256, 0, 0.0), ([9000], 24, 2, 240, 7001, 30.0),
    ([7000, 40], 6, 2, 144, 0, 0.0), ([8000], 48, 3, 128, 0, 0.0), ([6000, 0, 5000], 33, 1, 96, 0, 0.0), ([9000], 71, 1, 64, 0, 20.0),
    ([500], 10, 2, 256, 0, 0.0), ([900, 3], 24, 2, 128, 0, 0.0)])
def test_decode_sequences_in_many_parts(lengths, hq, hkv, D, window, softcap, e4m3):
    c = decode.Case(lengths, hq, hkv, D, page=64, e4m3=e4m3)
    first = c.run(window=window, softcap=softcap)
    c.check(*first, window=window, softcap=softcap)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run(window=window, softcap=softcap)))


# ------------------------------------------------------------------------------------------------------ cache rows
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["x bf16", "x f32"])
@pytest.mark.parametrize("T,page,layout,D,heads", [
    (45, 16, "heads first", 144, 3), (45, 13, "one buffer", 208, 5), (45, 24, "rows first", 240, 2), (45, 1, "rows first", 112, 1),
    (6001, 64, "heads first", 128, 8), (6003, 16, "rows first", 64, 3), (4999, 24, "one buffer", 144, 3),
    (5002, 13, "rows first", 240, 5), (6002, 128, "heads first", 256, 2), (9001, 1, "rows first", 16, 1), (6001, 64, "one buffer", 80, 4)])
def test_cache_rows(T, page, layout, D, heads, dtype, e4m3):
    """Rows written and read back are rounded once; from some 1200 rows of 8 heads on a lane takes four of them."""
    n_pages = -(-T // page) + 2
    g = gen(T + D)
    cache = make_cache(n_pages, heads, page, D, e4m3, layout)
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    outside = torch.tensor([0, 3, T // 2, T - 1])
    slots[outside] = torch.tensor([-1, n_pages * page, 2 ** 40, -2 ** 62])
    k, k64 = rows(g, T, heads * D, dtype, 16)
    v, v64 = rows(g, T, heads * D, dtype, 32, 3.0)
    before = [raw(t).clone() for t in cache[:2]]
    lm.cache_write(k, v, cache, slots.cuda())
    inside = torch.ones(T, dtype=torch.bool)
    inside[outside] = False
    for t in (F32, BF):                                  # both kinds of value are bf16 numbers
        for x64, y in zip((k64, v64), lm.cache_read(cache, slots.cuda(), dtype=t)):
            x = x64.reshape(T, heads, D)
            ref = quantized(x)[0] if e4m3 else x.to(BF).double()
            y = y.cpu().double().reshape(T, heads, D)
            assert torch.equal(y[inside], ref[inside]) and (y[outside] == 0).all()
    named = torch.zeros(n_pages * page, dtype=torch.bool)
    named[slots[inside]] = True
    for t, b in zip(cache[:2], before):                  # rows that no slot named are as they were
        same = (raw(t) == b).all(-1).permute(0, 2, 1).reshape(n_pages * page, heads)
        assert same[~named.cuda()].all() and not same[named.cuda()].all(1).any()
    if e4m3:
        for z in cache[2:]:
            kept = (z == -7.0).permute(0, 2, 1).reshape(n_pages * page, heads)
            assert torch.equal(kept, ~named.cuda()[:, None].expand(-1, heads))


# ------------------------------------------------------------------------------------------------------ rotary positions
PART = [dict(T=33, hq=3, hk=1, D=144, dtype=BF), dict(T=21, hq=2, hk=3, D=144, dtype=F32, interleaved=True, pad=16),
        dict(T=40, hq=5, hk=2, D=208, dtype=BF, rot=64, pad=8), dict(T=17, hq=4, hk=2, D=208, dtype=F32, rot=208),
        dict(T=30, hq=7, hk=1, D=240, dtype=BF, interleaved=True, norm="k"), dict(T=12, hq=2, hk=2, D=240, dtype=F32, rot=128, norm="none"),
        dict(T=25, hq=3, hk=3, D=112, dtype=BF, rot=96, interleaved=True), dict(T=19, hq=2, hk=1, D=176, dtype=F32, rot=16, norm="q"),
        dict(T=1500, hq=9, hk=3, D=144, dtype=BF, interleaved=True), dict(T=1400, hq=5, hk=2, D=240, dtype=F32, rot=64),
        dict(T=1300, hq=12, hk=4, D=208, dtype=BF)]


@pytest.mark.parametrize("c", PART, ids=ids)
def test_rotary_forward(c):
    rotary.test_forward(c)


@pytest.mark.parametrize("c", PART, ids=ids)
def test_rotary_backward(c):
    rotary.test_backward(c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("c", rotary.MANY + PART[:3] + PART[4:5] + PART[8:], ids=ids)
def test_rotary_into_a_cache(c, e4m3):
    """Several rows a warp and chunks of several steps, with a cache: every row's own slot, position, keys and values."""
    k = rotary.Case(**c)
    T, D, n = k.T, k.D, k.hq * k.D
    y, mag = k.result()
    n_pages = -(-T // 64) + 2
    cache = make_cache(n_pages, k.hk, 64, D, e4m3, "rows first")
    slots = torch.randperm(n_pages * 64, generator=gen(4))[:T]
    slots[torch.tensor([0, 4, T // 2, T - 1])] = torch.tensor([-1, n_pages * 64, -5, 2 ** 50])
    inside = (slots >= 0) & (slots < n_pages * 64)
    v, v64 = rows(gen(5), T, k.hk * D, k.dtype, 64)
    plain = lm.rotary_forward(k.x, *k.args, **k.kw)
    before = [raw(t).clone() for t in cache[:2]]
    q = lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots.cuda())
    assert q.shape == (T, n) and torch.equal(q, plain[:, :n])
    gk, gv = (t.cpu().double().reshape(T, k.hk, D) for t in lm.cache_read(cache, slots.cuda(), dtype=F32))
    ky, km = y[:, k.hq:], mag[:, k.hq:]
    if e4m3:        # half a step of a normal number, half of 2^-9 scales below; the scale may be twice the oracle's at a border
        tol = E4 * ky.abs() + 2.0 ** -9 * quantized(ky)[1][..., None] + REACH * km
        ref = quantized(v64.reshape(T, k.hk, D))[0]
    else:
        tol = half_step(BF) * ky.abs() + REACH * km
        ref = v64.reshape(T, k.hk, D).to(BF).double()
    close(gk[inside], ky[inside], tol[inside])
    assert torch.equal(gv[inside], ref[inside]) and (gk[~inside] == 0).all() and (gv[~inside] == 0).all()
    named = torch.zeros(n_pages * 64, dtype=torch.bool)
    named[slots[inside]] = True
    for t, b in zip(cache[:2], before):
        same = (raw(t) == b).all(-1).permute(0, 2, 1).reshape(n_pages * 64, k.hk)
        assert same[~named.cuda()].all()
    kept = [raw(t).clone() for t in cache[:2]]
    both = lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots.cuda(), keep_keys=True)
    assert torch.equal(both, plain) and all(torch.equal(raw(t), b) for t, b in zip(cache[:2], kept))
    lm.rotary_forward(k.x, *k.args, **k.kw, v=v, cache=cache, slots=slots.cuda(), out=k.x[:, :n])
    assert torch.equal(k.x[:, :n], plain[:, :n]) and all(torch.equal(raw(t), b) for t, b in zip(cache[:2], kept))
