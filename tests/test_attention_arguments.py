"""Arguments of the attention side's calls that would give a wrong answer without an error (no GPU is touched)."""
import math
import subprocess
from fractions import Fraction

import pytest
import torch

import lora_co_serving_gb300 as lm
from lora_co_serving_gb300 import _build
from test_attention_refusals import FAKE, cache, e4m3, error, lib, rotary  # noqa: F401  (lib: a fixture)


def decode(lib, B=2, heads=8, q=FAKE, ld_q=512, c=None, width=4, window=0, scale=0.1, softcap=0.0, out=2 * FAKE, ld_out=512):
    """A call that is refused for its workspace at the latest."""
    return error(lib, lib.lora_decode_attention(B, heads, q, ld_q, cache() if c is None else c, FAKE, width, width, FAKE, window,
                                                scale, softcap, out, ld_out, None, None, 0, None))


@pytest.mark.parametrize("c", [cache(), e4m3()], ids=["bf16", "e4m3"])
def test_decode_in_place_has_one_row_distance(lib, c):
    rc, msg = decode(lib, c=c, out=FAKE, ld_out=520)
    assert lm.ERRORS[rc] == "LORA_ERR_INVALID_ARG" and "in place, ld_out must be ld_q" in msg
    for kw in (dict(out=FAKE), dict(out=FAKE, ld_out=520, B=1), dict(ld_out=520)):
        rc, msg = decode(lib, c=c, **kw)
        assert "in place" not in msg


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32, -2 ** 32 + 5, 2 ** 63])
def test_window_is_not_cut_to_32_bits(monkeypatch, window):
    """No call with such a window reaches the library, where 2^32 + 5 would be 5."""
    bf, i32 = torch.bfloat16, torch.int32
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(lm, "_stream_ptr", lambda stream: 0)

    class Calls:
        def __getattr__(self, name):
            raise AssertionError(name + " was called")

    monkeypatch.setattr(lm, "library", lambda: Calls())
    q, c = torch.zeros(2, 128, dtype=bf), lm.kv_cache(4, 2, 8, 32, device="cpu")
    with pytest.raises(ValueError, match="window"):
        lm.decode_attention(q, c, torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), window=window,
                            workspace=torch.zeros(8, dtype=torch.uint8))


@pytest.mark.parametrize("shape", [(2 ** 32 + 8, 32), (2 ** 31, 32), (8, 2 ** 32 + 32)])
def test_sizes_are_not_cut_to_32_bits(monkeypatch, shape):
    """Rows and columns cross the ABI as C ints: 2^32 + 8 rows would be 8."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        lm._matrix(x, "x")
    if shape[1] == 32:
        slots = torch.empty(shape[0], dtype=torch.int64, device="meta")
        c = lm.kv_cache(4, 1, 8, 32, device="meta")
        monkeypatch.setattr(lm, "library", lambda: None)
        for call in (lambda: lm.cache_write(x, x, c, slots), lambda: lm.cache_read(c, slots),
                     lambda: lm.rotary_forward(x, slots, None, 1, 1), lambda: lm.fp8_quantize(x)):
            with pytest.raises(ValueError, match="2\\^31"):
                call()


@pytest.mark.parametrize("scale,softcap", [(0.1, 3e38), (0.1, 2.0 ** -140), (1e10, 1e-30), (3e38, 0.0), (-3e38, 0.0),
                                           (3e38, 0.5)])
def test_score_factors_stay_finite(lib, scale, softcap):
    """The kernel forms scale log2(e), or scale / cap and cap log2(e), in float32: where one is infinite, scores of zero would
    be NaN."""
    rc, msg = decode(lib, scale=scale, softcap=softcap)
    assert lm.ERRORS[rc] == "LORA_ERR_INVALID_ARG" and "softcap" in msg


@pytest.mark.parametrize("scale,softcap", [(2e38, 0.0), (0.0, 1e-40), (1.0, 2e38), (2e38, 2e38), (1e-45, 1e-45), (-1.0, 30.0)])
def test_other_score_factors_are_taken(lib, scale, softcap):
    rc, msg = decode(lib, scale=scale, softcap=softcap)
    assert "softcap" not in msg


def test_more_sequences_than_the_limit(lib):
    for B in (2 ** 31 - 1, 2 ** 31 - 1024):
        rc, msg = decode(lib, B=B)
        assert lm.ERRORS[rc] == "LORA_ERR_LIMIT" and "2^31 - 1025" in msg
    assert lm.ERRORS[decode(lib, B=2 ** 31 - 1025)[0]] != "LORA_ERR_LIMIT"


def test_shares_of_sequences(tmp_path):
    """The sequences that a thread counts the tiles of: all of them once, in order, for any number that is accepted."""
    src, exe = tmp_path / "t.cpp", str(tmp_path / "t")
    src.write_text(r'''
#include <cstdio>
#include <initializer_list>
#include "decode_split.h"
using namespace lora;
int main() {
    for (int32_t B : {1, 2, 127, 128, 129, 1000, 2500, 1 << 24, (1 << 30) + 7, 2147483647 - 1024}) {
        int32_t at = 0;
        for (int32_t i = 0; i < 128; ++i) {
            const Share s(B, i, 128);
            if (s.first < 0 || s.last < s.first || s.last > B || (s.first < s.last && s.first != at)) return printf("%d %d\n", B, i), 1;
            if (s.first < s.last) at = s.last;
        }
        if (at != B) return printf("%d\n", B), 1;
    }
    return 0;
}
''')
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", _build.CSRC, str(src), "-o",
                    exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("rot,base,frequencies", [(128, 10000.0, None), (256, 500000.0, None), (64, 1e6, None), (16, 2.0, None),
                                                  (16, 0.0, [1.0, math.pi, 3.0, 1e-5, 1e-15, 0.25, -0.75, 100.0])])
def test_turns_against_many_digits(rot, base, frequencies):
    """A float64 quotient f / 2 pi: its rounding is half a step, 2^-53, and float64's 2 pi is 2^-54 off: 2^-52 of the turns, then
    half a unit.  (Not the nearest whole number: for a frequency of 1 it is 181 units off, of 2.9e18.)"""
    given = [base ** (-2.0 * i / rot) for i in range(rot // 2)] if frequencies is None else frequencies
    got = lm.rotary_turns(rot, base, frequencies, device="cpu")
    for f, t in zip(given, got.tolist()):
        exact = Fraction(f) * 2 ** 63 / PI
        off = (t - exact + 2 ** 63) % 2 ** 64 - 2 ** 63          # whole turns count for nothing
        assert abs(off) <= abs(exact) / 2 ** 52 + Fraction(1, 2)
    one = lm.rotary_turns(16, 1.0, device="cpu").tolist()[0]
    assert 180 < abs(one - 2 ** 63 / PI) < 182


def test_weight_gradients_are_aligned(lib):
    """A store of a float32 to an address that is no multiple of 4 would fault on the device."""
    for dq, dk in ((FAKE + 2, None), (None, FAKE + 1), (FAKE, FAKE + 2)):
        for T in (0, 4):
            rc, msg = error(lib, lib.lora_rotary_backward(T, 0, rotary(qw=FAKE, kw=FAKE), FAKE, 768, FAKE, FAKE, 768, 2 * FAKE, 768,
                                                          dq, dk, FAKE, 1 << 30, None))
            assert lm.ERRORS[rc] == "LORA_ERR_ALIGNMENT" and "gradients" in msg


def test_workspaces_are_whole_bytes(monkeypatch):
    """A workspace is as long as its bytes say: a view whose elements lie on one another, or apart, is none."""
    i32, bf = torch.int32, torch.bfloat16
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(lm, "_stream_ptr", lambda stream: 0)

    class Calls:
        def __getattr__(self, name):
            raise AssertionError(name + " was called")

    monkeypatch.setattr(lm, "library", lambda: Calls())
    q, c = torch.zeros(2, 128, dtype=bf), lm.kv_cache(4, 2, 8, 32, device="cpu")
    w, p, turns = torch.ones(32, dtype=bf), torch.zeros(2, dtype=torch.int64), lm.rotary_turns(32, device="cpu")
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(64, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            lm.decode_attention(q, c, torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), workspace=ws)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            lm.rotary_backward(q, p, turns, 2, 2, q, q_weight=w, weight_grads=True, workspace=ws)
