"""What the operators around the layer refuse, on the host, before anything is launched (no GPU is touched)."""
import numpy as np
import pytest

import lora_co_serving_gb300 as lm

P, Q, R, S = 0x10000000, 0x20000000, 0x30000000, 0x40000000     # aligned addresses that nothing dereferences
WS = 0x50000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    lm.build()
    return lm.library()


def err(lib):
    return lib.lora_last_error().decode()


def seg(rows):
    a = lm.segments(rows)
    return a, a.ctypes.data, a.shape[0]


def test_quantize(lib):
    f = lib.lora_fp8_quantize
    assert f(0, 64, 0, None, 64, None, 64, None, None) == 0          # no rows: nothing to do
    assert f(4, 64, 7, P, 64, Q, 64, R, None) == -7
    assert f(-1, 64, 0, P, 64, Q, 64, R, None) == -1
    assert f(4, 0, 0, P, 64, Q, 64, R, None) == -1
    assert f(4, 56, 0, P, 64, Q, 64, R, None) == -5                  # K not a multiple of 16
    assert f(4, 64, 0, None, 64, Q, 64, R, None) == -1
    assert f(4, 64, 0, P, 56, Q, 64, R, None) == -1                  # rows overlap
    assert "overlap" in err(lib)
    assert f(4, 64, 0, P + 8, 64, Q, 64, R, None) == -5
    assert f(4, 64, 0, P, 68, Q, 64, R, None) == -5                  # rows 136 bytes apart
    assert f(4, 64, 1, P, 68, Q, 72, R, None) == -5                  # codes 72 bytes apart
    assert f(4, 64, 0, P, 64, Q, 64, None, None) == -1
    assert f(4, (1 << 22) + 16, 0, P, BIG, Q, BIG, R, None) == -10
    g = lib.lora_fp8_quantize_weight
    assert g(0, 64, 0, P, 64, Q, R, None) == -1
    assert g(8, 72, 0, P, 72, Q, R, None) == -5                      # K not a multiple of 16
    assert g(8, 64, 3, P, 64, Q, R, None) == -7
    assert g(8, 64, 0, P, 64, None, R, None) == -1


def test_linear(lib):
    def f(T=4, K=64, N=32, dt=0, x=P, ldx=64, xs=None, w=Q, ws=R, y=S, ldy=32, work=WS, n=1 << 30):
        return lib.lora_fp8_linear(T, K, N, dt, x, ldx, xs, w, ws, y, ldy, work, n, None)
    assert f(T=0, x=None, y=None, work=None) == 0
    assert f(dt=5) == -7
    assert f(dt=5, xs=R, work=None) == -6                            # 8-bit x: the element type is not looked at
    assert f(T=-1) == -1 and f(K=0) == -1 and f(N=-8) == -1
    assert f(K=56, ldx=56) == -5 and f(N=28) == -5
    assert f(x=P + 2) == -5 and f(w=Q + 8) == -5 and f(y=S + 8) == -5
    assert f(ldx=60) == -1 and f(ldy=24) == -1
    assert f(ldx=68) == -5 and f(ldy=36) == -5
    assert f(xs=R, ldx=72) == -5                                     # codes' rows 72 bytes apart
    assert f(ws=R + 2) == -5 and f(xs=R + 1) == -5
    assert f(T=2 ** 31 - 1) == -10 and f(K=(1 << 22) + 16, ldx=BIG) == -10
    assert f(x=None) == -1 and f(w=None) == -1 and f(ws=None) == -1 and f(y=None) == -1
    assert f(work=None) == -6 and f(work=WS + 64) == -6 and f(n=255) == -6
    assert "too small" in err(lib)
    need = lib.lora_fp8_workspace_size(40, 64, 32, 0)
    assert need >= 256 + 40 * 64 and f(T=40, n=need - 1) == -6       # x is quantized into the workspace
    assert 256 <= lib.lora_fp8_workspace_size(40, 64, 32, 1) <= need
    assert lib.lora_fp8_workspace_size(0, 64, 32, 0) >= 256
    assert lib.lora_fp8_workspace_size(4, 60, 32, 0) == 0 and lib.lora_fp8_workspace_size(-1, 64, 32, 0) == 0


def test_swiglu(lib):
    ok, a, n = seg([(0, 3, 0, 0), (3, 5, 1, 1)])

    def f(T=8, I=64, dt=0, gu=P, ld=128, segs=a, n_segs=n, h=Q, ldh=64, hs=None, ck=R, cs=S):
        return lib.lora_swiglu_forward(T, I, dt, gu, ld, segs, n_segs, h, ldh, hs, ck, cs, None)
    assert f(T=0, segs=None, n_segs=0, gu=None, ck=None) == 0
    assert f(dt=2) == -7 and f(T=-1) == -1 and f(I=0) == -1
    assert f(I=60, ld=120) == -5 and f(I=1 << 23, ld=BIG) == -10
    assert f(gu=None) == -1 and f(h=None) == -1 and f(cs=None) == -1
    assert f(ld=120) == -1 and f(ldh=56) == -1
    assert f(gu=P + 8) == -5 and f(ld=132) == -5 and f(ldh=68) == -5 and f(ck=R + 8) == -5
    assert f(hs=S, ldh=72) == -5                                     # 8-bit h: rows 72 bytes apart
    for rows, code in (([(0, 3, 0, 0)], -2), ([(0, 3, 0, 0), (2, 6, 1, 1)], -2), ([(0, 3, 0, 0), (4, 4, 1, 1)], -2),
                       ([(0, 9, 0, 0)], -2), ([(0, -1, 0, 0), (0, 8, 0, 0)], -2)):
        keep, b, m = seg(rows)
        assert f(segs=b, n_segs=m) == code, rows
        assert lib.lora_checkpoint_rows(8, b, m) == code
    assert f(segs=None, n_segs=2) == -1 and f(n_segs=-1) == -1
    keep, b, m = seg([(i, 1, 0, 1) for i in range(49)])
    assert f(T=49, segs=b, n_segs=m) == -10
    assert lib.lora_checkpoint_rows(8, a, n) == 5
    keep, b, m = seg([(3, 5, 1, 1), (8, 0, 0, 1), (0, 3, 0, 1)])     # any order, empty segments
    assert lib.lora_checkpoint_rows(8, b, m) == 8

    def g(R_=8, I=64, dt=0, ck=P, cs=S, dh=Q, ldh=64, d=R, ldd=128, ds=None):
        return lib.lora_swiglu_backward(R_, I, dt, ck, cs, dh, ldh, d, ldd, ds, None)
    assert g(R_=0, ck=None, dh=None) == 0
    assert g(dt=9) == -7 and g(R_=-1) == -1 and g(I=-8) == -1 and g(I=12) == -5
    assert g(ck=None) == -1 and g(cs=None) == -1 and g(dh=None) == -1 and g(d=None) == -1
    assert g(ldh=32) == -1 and g(ldd=64) == -1 and g(dh=Q + 4) == -5 and g(ldd=132) == -5
    assert g(ds=S) == -5                                             # 8-bit gradient of a width that blocks straddle


def pairs(rows):
    a = np.ascontiguousarray(np.asarray(rows, np.int32).reshape(-1, 4))
    return a, a.ctypes.data, a.shape[0]


def test_preference(lib):
    ok, a, n = pairs([(0, 3, 3, 2), (5, 0, 5, 3)])

    def f(T=8, V=10, dt=0, x=P, ld=10, lab=Q, ref=R, p=a, np_=n, beta=0.1, eps=0.0, out=S):
        return lib.lora_preference_forward(T, V, dt, x, ld, lab, ref, p, np_, beta, eps, out, out, out, out, out, None)
    assert f(T=0, x=None, lab=None, ref=None, p=None, np_=0) == 0
    assert f(dt=4) == -7 and f(T=-1) == -1 and f(V=0) == -1 and f(ld=9) == -1
    assert f(x=None) == -1 and f(lab=None) == -1 and f(ref=None) == -1 and f(out=None) == -1
    assert f(x=P + 1) == -5 and f(dt=1, x=P + 2) == -5
    for beta, eps in ((0.0, 0.0), (-1.0, 0.0), (float("nan"), 0.0), (float("inf"), 0.0), (0.1, 0.5), (0.1, -0.1),
                      (0.1, float("nan"))):
        assert f(beta=beta, eps=eps) == -1, (beta, eps)
    for rows in ([(0, 3, 2, 2)], [(0, 9, 0, 0)], [(-1, 2, 3, 1)], [(0, -1, 3, 1)], [(0, 2, 2, 3), (4, 1, 6, 1)],
                 [(0, 1, 2 ** 31 - 1, 2 ** 31 - 1)]):
        keep, b, m = pairs(rows)
        assert f(p=b, np_=m) == -2, rows
    assert f(p=None) == -1 and f(np_=-1) == -1
    keep, b, m = pairs([(2 * i, 1, 2 * i + 1, 1) for i in range(257)])
    assert f(T=600, p=b, np_=m) == -10

    def g(T=8, V=10, dt=0, x=P, ld=10, lab=Q, lse=R, coef=R, p=a, np_=n, dl=None, d=S, ldd=10):
        return lib.lora_preference_backward(T, V, dt, x, ld, lab, lse, coef, p, np_, dl, d, ldd, None)
    assert g(T=0, x=None, p=None, np_=0) == 0
    assert g(lse=None) == -1 and g(coef=None) == -1 and g(d=None) == -1 and g(ldd=9) == -1
    assert g(d=S + 1) == -5 and g(d=P, ldd=12) == -1                 # in place with another row distance
    h = lib.lora_token_logprob
    assert h(0, 10, 0, None, 10, None, None, None, None) == 0
    assert h(8, 10, 0, P, 10, Q, None, R, None) == -1 and h(8, 10, 3, P, 10, Q, R, R, None) == -7


def test_binding_checks_shapes():
    import torch
    e = torch.float8_e4m3fn
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.uint8).view(e)
    ws = torch.zeros(1, 1)
    with pytest.raises(ValueError, match=r"w must be \[32, 48\]"):
        lm.fp8_linear(x[:, :48], w, ws)
    with pytest.raises(ValueError, match="w_scales"):
        lm.fp8_linear(x, w, torch.zeros(2, 1))
    with pytest.raises(TypeError, match="w must be"):
        lm.fp8_linear(x, x, ws)
    with pytest.raises(TypeError, match="unsupported dtype"):
        lm.fp8_linear(x.half(), w, ws)
    with pytest.raises(TypeError, match="x must be"):
        lm.fp8_linear(x, w, ws, x_scales=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="unit column stride"):
        lm.fp8_quantize(torch.zeros(64, 4).t())
    with pytest.raises(ValueError, match="even number"):
        lm.swiglu_forward(torch.zeros(4, 65))
    with pytest.raises(ValueError, match="segment table"):
        lm.swiglu_forward(torch.zeros(4, 64), checkpoint=True)
    with pytest.raises(ValueError, match="checkpoint's codes"):
        lm.swiglu_backward((w, ws), torch.zeros(32, 64))
    with pytest.raises(TypeError, match="labels"):
        lm.token_logprob(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="ref_logp"):
        lm.preference_forward(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(3), [(0, 2, 2, 2)])
    with pytest.raises(ValueError, match="coef"):
        lm.preference_backward(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(4),
                               [(0, 2, 2, 2)])
    for call in (lambda: lm.fp8_linear(x, w, ws), lambda: lm.fp8_quantize(x), lambda: lm.swiglu_forward(x),
                 lambda: lm.fp8_quantize_weight(x),
                 lambda: lm.token_logprob(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)),
                 lambda: lm.preference_forward(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4), [])):
        with pytest.raises(ValueError, match="one CUDA device"):     # host memory never reaches a kernel
            call()
    with pytest.raises(lm.LoraError, match="segments"):
        lm.checkpoint_rows(4, [(0, 3, 0, 1)])
    assert lm.checkpoint_rows(4, [(0, 4, 0, 1)]) == 4
