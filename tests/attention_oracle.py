"""Float64 forms of the attention side of a step (include/lora_attention.h), and cases shared by its tests.  CPU tensors."""
import math

import torch

EPS = 1e-6
U = 2.0 ** -24              # half a step of float32, relative
BF = 2.0 ** -8              # of bf16
E4 = 2.0 ** -4              # of e4m3


def half_step(dtype):
    return BF if dtype is torch.bfloat16 else U


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def angles(positions, freqs):
    """Angles [T, R / 2] of whole-number positions in float64, the turns taken off in whole numbers."""
    turns = [round(f / (2.0 * math.pi) * 2.0 ** 64) for f in freqs]
    return torch.tensor([[2.0 * math.pi * (((p * t + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64) for t in turns]
                         for p in positions.tolist()], dtype=torch.float64).reshape(len(positions), len(freqs))


def pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def from_pairs(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def turned(x, angle, rot, interleaved):
    """x [T, H, D] turned by angle [T, rot / 2]."""
    a, b = pairs(x, rot, interleaved)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    return from_pairs(a * c - b * s, b * c + a * s, x[..., rot:], interleaved)


def reach(x, rot, interleaved):
    """|a| + |b| of each element's pair: what an error of the rotation is relative to."""
    a, b = (t.abs() for t in pairs(x, rot, interleaved))
    return from_pairs(a + b, a + b, x[..., rot:].abs(), interleaved)


def normed(x, w, eps=EPS):
    """x [T, H, D] normalised, w [H, D] or None."""
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def quantized(x):
    """(values that 8 bits hold for rows x [..., D], scales): the nearest e4m3 numbers in units of the row's scale."""
    a = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    s = torch.exp2(torch.ceil(torch.log2(a / 448.0)))
    s = torch.where(a > 448.0 * s, 2.0 * s, s)
    s = torch.where(a <= 224.0 * s, 0.5 * s, s)
    v = x / s
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step * s, s[..., 0]


def attention(q, k, v, scale, softcap=0.0):
    """q [n, D] over k, v [L, D]: (out [n, D], lse [n], probabilities [n, L], scores [n, L]); NaN-free for L = 0."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=q.dtype), None, None
    s = q @ k.t() * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    p = torch.softmax(s, -1)
    return p @ v, torch.logsumexp(s, -1), p, s
