"""What the attention side of a step refuses, and the index arithmetic that its kernels rest on (no GPU is touched)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import lora_co_serving_gb300 as lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # a device address that nothing reads


@pytest.fixture(scope="module")
def lib():
    lm.build()
    return lm.library()


def cache(k=FAKE, v=FAKE, ks=0, vs=0, strides=(4096, 1024, 64), scales=(64, 16, 1), pages=8, heads=4, rows=16, D=64, dt=0):
    return lm._CACHE_STRUCT.pack(k, v, ks, vs, *strides, *scales, pages, heads, rows, D, dt)


def e4m3(**kw):
    return cache(**{**dict(ks=FAKE, vs=FAKE, dt=1), **kw})


def rotary(turns=FAKE, qw=0, kw=0, hq=8, hk=4, D=64, rot=64, inter=0, eps=1e-6):
    return lm._ROTARY_STRUCT.pack(turns, qw, kw, hq, hk, D, rot, inter, eps)


def error(lib, rc):
    return rc, lib.lora_last_error().decode()


def forward(lib, T=4, dt=0, r=None, x=FAKE, ld_x=768, pos=FAKE, out=2 * FAKE, ld_out=768, v=None, ld_v=0, c=None,
            slots=None, keep=0):
    return error(lib, lib.lora_rotary_forward(T, dt, rotary() if r is None else r, x, ld_x, pos, out, ld_out, v, ld_v, c,
                                              slots, keep, None))


@pytest.mark.parametrize("kw,code,text", [
    (dict(dt=2), "LORA_ERR_DTYPE", "dtype"),
    (dict(T=-1), "LORA_ERR_INVALID_ARG", "T must be"),
    (dict(T=2 ** 31 - 1), "LORA_ERR_LIMIT", "rows"),
    (dict(r=rotary(hq=0)), "LORA_ERR_INVALID_ARG", "head"),
    (dict(r=rotary(hk=0)), "LORA_ERR_INVALID_ARG", "head"),
    (dict(r=rotary(hq=1000, hk=20)), "LORA_ERR_LIMIT", "heads"),
    (dict(r=rotary(D=72)), "LORA_ERR_LIMIT", "multiple of 16"),
    (dict(r=rotary(D=272)), "LORA_ERR_LIMIT", "256"),
    (dict(r=rotary(D=0, rot=0)), "LORA_ERR_LIMIT", "multiple of 16"),
    (dict(r=rotary(rot=8)), "LORA_ERR_LIMIT", "turned part"),
    (dict(r=rotary(rot=80)), "LORA_ERR_LIMIT", "turned part"),
    (dict(r=rotary(turns=0)), "LORA_ERR_INVALID_ARG", "turns is NULL"),
    (dict(r=rotary(turns=FAKE + 4)), "LORA_ERR_ALIGNMENT", "turns"),
    (dict(r=rotary(qw=FAKE + 2)), "LORA_ERR_ALIGNMENT", "weights"),
    (dict(r=rotary(qw=FAKE, eps=-1.0)), "LORA_ERR_INVALID_ARG", "eps"),
    (dict(r=rotary(kw=FAKE, eps=math.nan)), "LORA_ERR_INVALID_ARG", "eps"),
    (dict(x=None), "LORA_ERR_INVALID_ARG", "x is NULL"),
    (dict(out=None), "LORA_ERR_INVALID_ARG", "out is NULL"),
    (dict(ld_x=760), "LORA_ERR_INVALID_ARG", "rows of x overlap"),
    (dict(ld_x=772), "LORA_ERR_ALIGNMENT", "x must be"),
    (dict(x=FAKE + 8), "LORA_ERR_ALIGNMENT", "x must be"),
    (dict(ld_out=512), "LORA_ERR_INVALID_ARG", "rows of out overlap"),
    (dict(out=FAKE, ld_out=776), "LORA_ERR_INVALID_ARG", "in place"),
    (dict(pos=None), "LORA_ERR_INVALID_ARG", "positions is NULL"),
    (dict(pos=FAKE + 4), "LORA_ERR_ALIGNMENT", "positions"),
    (dict(c=cache(), v=FAKE, ld_v=256), "LORA_ERR_INVALID_ARG", "slots is NULL"),
    (dict(c=cache(), v=FAKE, ld_v=256, slots=FAKE + 4), "LORA_ERR_ALIGNMENT", "slots"),
    (dict(c=cache(), slots=FAKE), "LORA_ERR_INVALID_ARG", "v is NULL"),
    (dict(c=cache(), v=FAKE, ld_v=248, slots=FAKE), "LORA_ERR_INVALID_ARG", "rows of v overlap"),
    (dict(c=cache(heads=2), v=FAKE, ld_v=256, slots=FAKE), "LORA_ERR_INVALID_ARG", "heads"),
    (dict(c=cache(D=32), v=FAKE, ld_v=256, slots=FAKE), "LORA_ERR_INVALID_ARG", "heads"),
])
def test_rotary_forward_refusals(lib, kw, code, text):
    rc, msg = forward(lib, **kw)
    assert lm.ERRORS[rc] == code and text in msg


@pytest.mark.parametrize("kw,code,text", [
    (dict(c=None), "LORA_ERR_INVALID_ARG", "cache is NULL"),
    (dict(c=cache(dt=2)), "LORA_ERR_DTYPE", "element type"),
    (dict(c=cache(pages=-1)), "LORA_ERR_INVALID_ARG", "pages"),
    (dict(c=cache(rows=0)), "LORA_ERR_INVALID_ARG", "pages"),
    (dict(c=cache(heads=0)), "LORA_ERR_INVALID_ARG", "head"),
    (dict(c=cache(heads=1025)), "LORA_ERR_LIMIT", "1024"),
    (dict(c=cache(D=24)), "LORA_ERR_LIMIT", "multiple of 16"),
    (dict(c=cache(D=512)), "LORA_ERR_LIMIT", "256"),
    (dict(c=cache(k=0)), "LORA_ERR_INVALID_ARG", "NULL"),
    (dict(c=cache(v=0)), "LORA_ERR_INVALID_ARG", "NULL"),
    (dict(c=e4m3(ks=0)), "LORA_ERR_INVALID_ARG", "NULL"),
    (dict(c=e4m3(vs=0)), "LORA_ERR_INVALID_ARG", "NULL"),
    (dict(c=e4m3(vs=FAKE + 2)), "LORA_ERR_ALIGNMENT", "scales"),
    (dict(c=cache(k=FAKE + 8)), "LORA_ERR_ALIGNMENT", "cache"),
    (dict(c=cache(strides=(4096, 1024, 68))), "LORA_ERR_ALIGNMENT", "strides"),
    (dict(c=e4m3(strides=(4096, 1024, 72))), "LORA_ERR_ALIGNMENT", "strides"),
    (dict(c=cache(strides=(-4096, 1024, 64))), "LORA_ERR_INVALID_ARG", "negative"),
    (dict(c=e4m3(scales=(64, -16, 1))), "LORA_ERR_INVALID_ARG", "negative"),
    (dict(T=-1), "LORA_ERR_INVALID_ARG", "T must"),
    (dict(T=2 ** 31 - 1), "LORA_ERR_LIMIT", "rows"),
    (dict(dt=7), "LORA_ERR_DTYPE", "dtype"),
    (dict(k=None), "LORA_ERR_INVALID_ARG", "k is NULL"),
    (dict(v=None), "LORA_ERR_INVALID_ARG", "v is NULL"),
    (dict(ld_v=248), "LORA_ERR_INVALID_ARG", "rows of v overlap"),
    (dict(k=FAKE + 4), "LORA_ERR_ALIGNMENT", "k must be"),
    (dict(slots=None), "LORA_ERR_INVALID_ARG", "slots is NULL"),
])
def test_cache_refusals(lib, kw, code, text):
    a = {**dict(T=4, dt=0, k=FAKE, ld_k=256, v=FAKE, ld_v=256, c=cache(), slots=FAKE), **kw}
    rc, msg = error(lib, lib.lora_cache_write(a["T"], a["dt"], a["k"], a["ld_k"], a["v"], a["ld_v"], a["c"], a["slots"], None))
    assert lm.ERRORS[rc] == code and text in msg
    rc, msg = error(lib, lib.lora_cache_read(a["T"], a["dt"], a["c"], a["slots"], a["k"], a["ld_k"], a["v"], a["ld_v"], None))
    assert lm.ERRORS[rc] == code and text in msg


@pytest.mark.parametrize("kw,code,text", [
    (dict(dout=None), "LORA_ERR_INVALID_ARG", "dout is NULL"),
    (dict(dx=None), "LORA_ERR_INVALID_ARG", "dx is NULL"),
    (dict(x=None, r=rotary(qw=FAKE)), "LORA_ERR_INVALID_ARG", "x is NULL"),
    (dict(ld_dx=760), "LORA_ERR_INVALID_ARG", "rows of dx overlap"),
    (dict(dx=FAKE, ld_dx=776), "LORA_ERR_INVALID_ARG", "in place"),
    (dict(dq=FAKE), "LORA_ERR_INVALID_ARG", "not given"),
    (dict(r=rotary(qw=FAKE), dk=FAKE), "LORA_ERR_INVALID_ARG", "not given"),
    (dict(r=rotary(qw=FAKE), dq=FAKE), "LORA_ERR_WORKSPACE", "workspace"),
    (dict(r=rotary(qw=FAKE), dq=FAKE, ws=FAKE, n=1024), "LORA_ERR_WORKSPACE", "workspace"),
    (dict(r=rotary(qw=FAKE), dq=FAKE, ws=FAKE + 4, n=1 << 30), "LORA_ERR_WORKSPACE", "workspace"),
    (dict(T=0, r=rotary(qw=FAKE), dq=FAKE), "LORA_ERR_WORKSPACE", "workspace"),
    (dict(pos=None), "LORA_ERR_INVALID_ARG", "positions is NULL"),
])
def test_rotary_backward_refusals(lib, kw, code, text):
    a = {**dict(T=4, r=rotary(), x=FAKE, pos=FAKE, dout=FAKE, dx=2 * FAKE, ld_dx=768, dq=None, dk=None, ws=None, n=0), **kw}
    rc, msg = error(lib, lib.lora_rotary_backward(a["T"], 0, a["r"], a["x"], 768, a["pos"], a["dout"], 768, a["dx"], a["ld_dx"],
                                                  a["dq"], a["dk"], a["ws"], a["n"], None))
    assert lm.ERRORS[rc] == code and text in msg


@pytest.mark.parametrize("kw,code,text", [
    (dict(c=cache(dt=2)), "LORA_ERR_DTYPE", "element type"),
    (dict(heads=6), "LORA_ERR_INVALID_ARG", "multiple of the cache's heads"),
    (dict(heads=0), "LORA_ERR_INVALID_ARG", "multiple of the cache's heads"),
    (dict(heads=1028), "LORA_ERR_LIMIT", "1024"),
    (dict(B=-1), "LORA_ERR_INVALID_ARG", "B and window"),
    (dict(window=-1), "LORA_ERR_INVALID_ARG", "B and window"),
    (dict(scale=math.inf), "LORA_ERR_INVALID_ARG", "scale"),
    (dict(scale=math.nan), "LORA_ERR_INVALID_ARG", "scale"),
    (dict(softcap=-1.0), "LORA_ERR_INVALID_ARG", "softcap"),
    (dict(softcap=math.inf), "LORA_ERR_INVALID_ARG", "softcap"),
    (dict(q=None), "LORA_ERR_INVALID_ARG", "q is NULL"),
    (dict(q=FAKE + 2), "LORA_ERR_ALIGNMENT", "q must be"),
    (dict(out=None), "LORA_ERR_INVALID_ARG", "out is NULL"),
    (dict(ld_out=504), "LORA_ERR_INVALID_ARG", "rows of out overlap"),
    (dict(table=None), "LORA_ERR_INVALID_ARG", "table or lengths"),
    (dict(lengths=None), "LORA_ERR_INVALID_ARG", "table or lengths"),
    (dict(width=0), "LORA_ERR_INVALID_ARG", "rows of table"),
    (dict(ld_table=3), "LORA_ERR_INVALID_ARG", "rows of table"),
    (dict(lengths=FAKE + 2), "LORA_ERR_ALIGNMENT", "4-byte"),
    (dict(lse=FAKE + 2), "LORA_ERR_ALIGNMENT", "4-byte"),
])
def test_decode_refusals(lib, kw, code, text):
    a = {**dict(B=2, heads=8, q=FAKE, ld_q=512, c=cache(), table=FAKE, ld_table=4, width=4, lengths=FAKE, window=0, scale=0.1,
                softcap=0.0, out=2 * FAKE, ld_out=512, lse=None, ws=None, n=0), **kw}
    rc, msg = error(lib, lib.lora_decode_attention(a["B"], a["heads"], a["q"], a["ld_q"], a["c"], a["table"], a["ld_table"],
                                                   a["width"], a["lengths"], a["window"], a["scale"], a["softcap"], a["out"],
                                                   a["ld_out"], a["lse"], a["ws"], a["n"], None))
    assert lm.ERRORS[rc] == code and text in msg


def test_calls_without_rows_are_valid(lib):
    assert forward(lib, T=0, x=None, out=None, pos=None)[0] == 0
    assert lib.lora_cache_write(0, 0, None, 0, None, 0, cache(), None, None) == 0
    assert lib.lora_cache_read(0, 0, cache(pages=0, k=0, v=0), None, None, 0, None, 0, None) == 0
    assert lib.lora_rotary_backward(0, 0, rotary(), None, 0, None, None, 0, None, 0, None, None, None, 0, None) == 0
    assert lib.lora_decode_attention(0, 8, None, 0, cache(), None, 0, 0, None, 0, 0.1, 0.0, None, 0, None, None, 0, None) == 0


def test_workspace_sizes(lib):
    assert lib.lora_rotary_workspace_size(16, rotary()) >= 2 * 64 * 4
    assert lib.lora_rotary_workspace_size(16, rotary(D=24)) == 0 and "multiple of 16" in lib.lora_last_error().decode()
    assert lib.lora_decode_workspace_size(6, cache()) == 0 and "multiple" in lib.lora_last_error().decode()


class TestBinding:
    """What the Python side refuses before the library is called."""

    bf = torch.bfloat16

    def pool(self, dtype=None, heads=2, D=32, **kw):
        return lm.kv_cache(4, heads, 8, D, dtype, device="cpu")

    def refused(self, text, fn, *a, error=ValueError, **kw):
        with pytest.raises(error, match=text):
            fn(*a, **kw)

    def test_caches(self):
        c = self.pool()
        slots = torch.zeros(3, dtype=torch.int64)
        rows = torch.zeros(3, 64, dtype=self.bf)
        f8 = self.pool(torch.float8_e4m3fn)
        for bad, text in ((lm.KVCache(c.k[0], c.v[0]), "four dimensions"), (lm.KVCache(c.k, c.v[:2]), "one shape"),
                          (lm.KVCache(c.k, c.v.transpose(1, 2).contiguous().transpose(1, 2)), "one shape"),
                          (lm.KVCache(c.k, f8.v), "one shape"), (lm.KVCache(c.k[..., ::2], c.v[..., ::2]), "unit stride"),
                          (lm.KVCache(c.k, c.v, f8.k_scales, f8.v_scales), "no scales"), (lm.KVCache(f8.k, f8.v), "needs"),
                          (lm.KVCache(f8.k, f8.v, f8.k_scales[:2], f8.v_scales), "scales must be")):
            self.refused(text, lm.cache_write, rows, rows, bad, slots)
            self.refused(text, lm.cache_read, bad, slots)
        self.refused("bfloat16 or float8", lm.cache_read, lm.KVCache(c.k.float(), c.v.float()), slots, error=TypeError)
        self.refused("float32", lm.cache_read, lm.KVCache(f8.k, f8.v, f8.k_scales.double(), f8.v_scales.double()), slots,
                     error=TypeError)
        self.refused("bfloat16 or float8", lm.kv_cache, 1, 1, 1, 16, torch.float16, "cpu", error=TypeError)
        self.refused("k must be", lm.cache_write, rows[:, :32], rows, c, slots)
        self.refused("v must be", lm.cache_write, rows, rows.float(), c, slots, error=TypeError)
        self.refused("slots must be", lm.cache_write, rows, rows, c, slots.int(), error=TypeError)
        self.refused("slots must be", lm.cache_write, rows, rows, c, slots[:2])
        self.refused("one CUDA device", lm.cache_write, rows, rows, c, slots)
        self.refused("one CUDA device", lm.cache_read, c, slots)
        self.refused("unsupported dtype", lm.cache_read, c, slots, torch.float16, error=TypeError)

    def test_rotary(self):
        x, pos, turns = torch.zeros(3, 128, dtype=self.bf), torch.zeros(3, dtype=torch.int64), lm.rotary_turns(32, device="cpu")
        w, c, slots = torch.ones(32, dtype=self.bf), self.pool(), torch.zeros(3, dtype=torch.int64)
        v = torch.zeros(3, 64, dtype=self.bf)
        f, b = lm.rotary_forward, lm.rotary_backward
        self.refused("do not hold", f, x, pos, turns, 2, 1)
        self.refused("do not hold", f, x, pos, turns, 0, 2)
        self.refused("positions must", f, x, pos[:2], turns, 2, 2)
        self.refused("positions must", f, x, pos.int(), turns, 2, 2, error=TypeError)
        self.refused("need positions", f, x, None, turns, 2, 2)
        self.refused("turns must", f, x, pos, turns.double(), 2, 2, error=TypeError)
        self.refused("q_weight must", f, x, pos, turns, 2, 2, q_weight=w.float(), error=TypeError)
        self.refused("k_weight must", f, x, pos, turns, 2, 2, k_weight=w[:16])
        self.refused("needs v and slots", f, x, pos, turns, 2, 2, cache=c, slots=slots)
        self.refused("need a cache", f, x, pos, turns, 2, 2, v=v)
        self.refused("heads", f, torch.zeros(3, 96, dtype=self.bf), pos, turns, 2, 1, cache=c, v=v[:, :32], slots=slots)
        self.refused("out must", f, x, pos, turns, 2, 2, cache=c, v=v, slots=slots, out=x)
        self.refused("one CUDA device", f, x, pos, turns, 2, 2)
        self.refused("needs its input", b, None, pos, turns, 2, 2, x, q_weight=w)
        self.refused("one CUDA device", b, None, pos, turns, 2, 2, x)
        self.refused("multiple of 16", lm.rotary_turns, 24)
        self.refused("frequencies needed", lm.rotary_turns, 32, frequencies=[1.0])

    def test_decode(self):
        c, q = self.pool(), torch.zeros(2, 128, dtype=self.bf)
        table, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
        d = lm.decode_attention
        self.refused("do not hold", d, q[:, :96], c, table, n)
        self.refused("do not hold", d, q[:, :16], c, table, n)
        self.refused("q must be", d, q.float(), c, table, n, error=TypeError)
        self.refused("page_table must", d, q, c, table.long(), n, error=TypeError)
        self.refused("row for each", d, q, c, table[:1], n)
        self.refused("lengths must", d, q, c, table, n.long(), error=TypeError)
        self.refused("lengths must", d, q, c, table, n[:1])
        self.refused("out must", d, q, c, table, n, out=q[:1])
        self.refused("one CUDA device", d, q, c, table, n)


def test_other_devices_are_refused(monkeypatch):
    """As if every tensor lay on a device that is not the current one: no call reaches the library."""
    class NoCalls:
        def __getattr__(self, name):
            if name in ("lora_rotary_workspace_size", "lora_last_error"):          # host functions
                return getattr(real, name)
            raise AssertionError(name + " was called")

    lm.build()
    real = lm.library()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    monkeypatch.setattr(lm, "_stream_ptr", lambda stream: 0)
    monkeypatch.setattr(lm, "library", lambda: NoCalls())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    bf = torch.bfloat16
    x, pos, w = torch.zeros(3, 128, dtype=bf), torch.zeros(3, dtype=torch.int64), torch.ones(32, dtype=bf)
    turns, c = lm.rotary_turns(32, device="cpu"), lm.kv_cache(4, 2, 8, 32, device="cpu")
    n = torch.ones(3, dtype=torch.int32)
    for call in (lambda: lm.rotary_forward(x, pos, turns, 2, 2), lambda: lm.rotary_backward(None, pos, turns, 2, 2, x),
                 lambda: lm.rotary_backward(x, pos, turns, 2, 2, x, q_weight=w, weight_grads=True),
                 lambda: lm.cache_write(x[:, :64], x[:, :64], c, pos), lambda: lm.cache_read(c, pos),
                 lambda: lm.decode_attention(x, c, torch.zeros(3, 2, dtype=torch.int32), n)):
        with pytest.raises(ValueError, match="the current one"):
            call()


def test_turns_are_the_frequencies():
    """Whole-number turns against the angles of float64 products, where those are good: positions below 2^20."""
    from attention_oracle import angles, frequencies
    for rot, base in ((32, 10000.0), (128, 500000.0)):
        freqs = frequencies(rot, base)
        got = lm.rotary_turns(rot, base, device="cpu")
        assert got.dtype is torch.int64 and got.shape == (rot // 2,)
        assert [int(t) % 2 ** 64 for t in got] == [round(f / (2 * math.pi) * 2 ** 64) for f in freqs]
        p = torch.tensor([0, 1, 7, 4095, 1 << 19])
        a = angles(p, freqs)
        direct = p.double()[:, None] * torch.tensor(freqs, dtype=torch.float64)
        # a product is half a step of float64 off, 2^19 2^-53
        assert (torch.exp(1j * a) - torch.exp(1j * direct)).abs().max() < 2.0 ** -33


def test_index_arithmetic(tmp_path):
    """The kernel's division by the page size, its lines of tiles and the owners of their pieces, over many sizes."""
    src, exe = tmp_path / "t.cpp", str(tmp_path / "t")
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include "decode_split.h"
using namespace lora;
#define CHECK(x) do { if (!(x)) { printf("failed: %s\n", #x); return 1; } } while (0)
int main() {
    uint64_t r = 88172645463325252ull;
    auto rnd = [&](uint64_t n) { r ^= r << 13; r ^= r >> 7; r ^= r << 17; return r % n; };
    for (int i = 0; i < 3000; ++i) {
        const uint32_t d = i < 300 ? i + 1 : 1 + (uint32_t)rnd(i % 3 ? 5000 : 0x7FFFFFFF);
        const PageDivision p = page_division(d);
        for (int j = 0; j < 300; ++j) {
            uint32_t n = (uint32_t)rnd(0x80000000ull);
            if (j < 8) n = (uint32_t)j;
            else if (j < 100) { const uint64_t m = rnd(0x80000000ull / d) * d; n = (uint32_t)(j % 2 ? m : m ? m - 1 : 0); }
            else if (j == 100) n = 0x7FFFFFFF;
            CHECK(p.page_of(n) == n / d);
        }
    }
    for (int i = 0; i < 4000; ++i) {
        const int64_t W = 1 + (int64_t)rnd(i % 2 ? 2000 : 1ull << 33), C = 1 + (int64_t)rnd(608);
        const Line line{W, C < W ? C : W};
        CHECK(line.first_tile(0) == 0 && line.first_tile(line.ctas) == W);
        for (int j = 0; j < 50; ++j) {
            const int64_t p = j == 0 ? 0 : j == 1 ? W - 1 : (int64_t)rnd(W), c = line.owner(p);
            CHECK(c >= 0 && c < line.ctas && line.first_tile(c) <= p && p < line.first_tile(c + 1));
        }
        for (int64_t c = 0; c < line.ctas; ++c) CHECK(line.first_tile(c) < line.first_tile(c + 1));
    }
    // the rows of a sequence: inside its table's row, one at least where it is too short
    for (int i = 0; i < 200000; ++i) {
        const int32_t n = i % 5 ? (int32_t)rnd(100000) : (int32_t)rnd(1ull << 32), w = i % 3 ? 0 : (int32_t)rnd(1ull << 31);
        const int32_t width = 1 + (int32_t)rnd(i % 2 ? 100 : 2000000), page = 1 + (int32_t)rnd(i % 4 ? 200 : 100000);
        const Range g(n, w, width, page);
        const int64_t most = (int64_t)width * page;
        CHECK(g.start >= 0 && g.end <= most && g.poisoned == (n > most));
        CHECK(n > 0 ? g.start < g.end : g.start >= g.end);
        if (n > 0 && !g.poisoned) CHECK(g.end == n && g.start == (w > 0 && w < n ? n - w : 0));
        CHECK(g.tiles(64) == (g.end > g.start ? ((int64_t)g.end - g.start + 63) / 64 : 0));
    }
    return 0;
}
''')
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "lora_co_serving_gb300", "csrc"), str(src), "-o", exe],
                   check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
