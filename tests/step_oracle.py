"""Plain float64 forms of the operators around the layer (8-bit blocks, MLP activation, preference loss)."""
import numpy as np

BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def scale_of(amax):
    """Smallest power of two s with amax <= 448 s (amax at least 2^-100); NaN where amax is not finite."""
    a = np.maximum(np.asarray(amax, np.float64), 2.0 ** -100)
    ok = np.isfinite(a)
    m, e = np.frexp(np.where(ok, a, 1.0))
    return np.where(ok, np.ldexp(1.0, e - 9 + (m > 0.875)), np.nan)


def e4m3(v):
    """v rounded to the nearest e4m3 number, ties to even (|v| <= 448)."""
    v = np.asarray(v, np.float64)
    e = np.maximum(np.frexp(v)[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.rint(v / step) * step


def quantize(x):
    """x [T, K] -> (code values, scales [T, blocks])."""
    x = np.asarray(x, np.float64)
    q = np.empty_like(x)
    s = np.empty((x.shape[0], blocks(x.shape[1])))
    for b in range(s.shape[1]):
        c = slice(BLOCK * b, BLOCK * (b + 1))
        s[:, b] = scale_of(np.abs(x[:, c]).max(1))
        with np.errstate(invalid="ignore"):
            q[:, c] = e4m3(x[:, c] / s[:, b:b + 1])
    return q, s


def quantize_weight(w):
    w = np.asarray(w, np.float64)
    q = np.empty_like(w)
    s = np.empty((blocks(w.shape[0]), blocks(w.shape[1])))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            c = np.s_[BLOCK * i:BLOCK * (i + 1), BLOCK * j:BLOCK * (j + 1)]
            s[i, j] = scale_of(np.abs(w[c]).max())
            q[c] = e4m3(w[c] / s[i, j])
    return q, s


def spread_rows(s, K):
    return np.repeat(s, BLOCK, 1)[:, :K]


def spread_weight(s, N, K):
    return np.repeat(np.repeat(s, BLOCK, 0), BLOCK, 1)[:N, :K]


def sigmoid(g):
    return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(gu):
    I = gu.shape[1] // 2
    return gu[:, :I] * sigmoid(gu[:, :I]) * gu[:, I:]


def swiglu_grad(g, u, dh):
    s = sigmoid(g)
    return np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], 1)


def log_softmax_parts(x):
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        return (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]


def preference(x, labels, ref, pairs, beta, eps):
    """(loss [P], rewards [P, 2], logp [T], lse [T], coef [P, 2])."""
    T = x.shape[0]
    counted = labels >= 0
    lse = np.where(counted, log_softmax_parts(x), 0.0)
    at = x[np.arange(T), np.maximum(labels, 0)]
    logp = np.where(counted, at - lse, 0.0)
    d = np.zeros((len(pairs), 2))
    for i, (c0, cn, r0, rn) in enumerate(pairs):
        for j, (a, n) in enumerate(((c0, cn), (r0, rn))):
            k = counted[a:a + n]
            d[i, j] = beta * (logp[a:a + n][k] - ref[a:a + n][k]).sum()
    m = d[:, 0] - d[:, 1]
    soft = np.log1p(np.exp(-np.abs(m)))
    loss = (1 - eps) * (np.maximum(-m, 0) + soft) + eps * (np.maximum(m, 0) + soft)
    k = beta * (eps * sigmoid(m) - (1 - eps) * sigmoid(-m))
    return loss, d, logp, lse, np.stack([k, -k], 1)


def dlogits(x, labels, lse, coef, pairs, dloss):
    out = np.zeros_like(x)
    for i, (c0, cn, r0, rn) in enumerate(pairs):
        for j, (a, n) in enumerate(((c0, cn), (r0, rn))):
            for t in range(a, a + n):
                if labels[t] >= 0:
                    k = coef[i, j] * dloss[i]
                    out[t] = -k * np.exp(x[t] - lse[t])
                    out[t, labels[t]] += k
    return out
