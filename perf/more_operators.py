"""Measured cases of the attention side of a co-served decoder's step, between the fused q|k|v projection and the output
projection:

  rotary    each query and key head normalised (root mean square) and turned by its position, in one pass; with a cache
            the keys and values go into it in the same pass.  Its backward for the fine-tuning rows
  cache     key and value rows written into a paged cache, in 16 bits or in 8 (e4m3, one scale for each head's row: the
            smallest power of two that brings the row within e4m3's largest number), and read back
  decode    attention of one new token of each sequence over the paged cache

Where `own` is false, run() computes a pass in elementary torch operations in 32 bits (angles in 64); where it is true,
it makes the calls of this framework.  exact() gives the same outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0           # largest e4m3 value
AMAX_FLOOR = 2.0 ** -100   # a row's largest magnitude is taken as at least this, so that no scale is zero
EPS = 1e-6
DEVICE = "cuda"


# ----------------------------------------------------------------------------------------------------------- cases
def _rotary(mode, T, hq, hkv, D, **kw):
    c = dict(op="rotary", mode=mode, T=T, hq=hq, hkv=hkv, D=D, rot=D, interleaved=False, norm=True,
             dtype="bf16", theta=500000.0, page=64, cache="none", wgrad=False)
    return {**c, **kw}


def _cache(mode, T, hkv, D, **kw):
    return {**dict(op="cache", mode=mode, T=T, hkv=hkv, D=D, page=64, cache="fp8", dtype="bf16"), **kw}


def _decode(B, longest, hq, hkv, D, **kw):
    c = dict(op="decode", B=B, longest=longest, hq=hq, hkv=hkv, D=D, page=64, cache="bf16", window=0,
             softcap=0.0)
    return {**c, **kw}


def listed():
    return [
        # one decode token of an 8B-sized layer: launch latency
        {"name": "rotary decode 1", **_rotary("forward", 1, 32, 8, 128)},
        # a decode batch whose keys and values go into an 8-bit cache, and its new rows read back
        {"name": "rotary decode 320 cached", **_rotary("cached", 320, 32, 8, 128, cache="fp8")},
        # the whole co-serving batch of a 70B-sized layer
        {"name": "rotary co-serving 8192", **_rotary("forward", 8192, 64, 8, 128)},
        # the gradient of 2048 fine-tuning rows, norm weights among them
        {"name": "rotary backward 2048", **_rotary("backward", 2048, 32, 8, 128, wgrad=True)},
        # a ragged fine-tuning batch in float32, half of each small head turned, neighbours paired
        {"name": "rotary backward 777 f32",
         **_rotary("backward", 777, 14, 2, 64, rot=32, interleaved=True, norm=False, dtype="f32", theta=10000.0)},
        # a prefill's keys and values written in 8 bits and read back
        {"name": "cache write 4096", **_cache("write", 4096, 8, 128)},
        # a cached prefix of 32k tokens read back for the next piece of a prefill
        {"name": "cache read 32768", **_cache("read", 32768, 8, 128)},
        # one short sequence: latency
        {"name": "decode 1 x 700", **_decode(1, 700, 32, 8, 128)},
        # a decode batch of ragged lengths of an 8B-sized layer
        {"name": "decode 64 x 8192", **_decode(64, 8192, 32, 8, 128)},
        # one long sequence over an 8-bit cache, 70B-sized layer: split over the length
        {"name": "decode 1 x 131072 fp8", **_decode(1, 131072, 64, 8, 128, cache="fp8")},
        # a large decode batch of short sequences over an 8-bit cache
        {"name": "decode 256 x 2048 fp8", **_decode(256, 2048, 64, 8, 128, cache="fp8")},
        # wide heads in odd groups, pages that end anywhere, a window and capped scores
        {"name": "decode 5 x 20000 window", **_decode(5, 20000, 10, 2, 256, page=24, window=4096, softcap=50.0)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (64, 8), (40, 8), (28, 4), (14, 2), (16, 16), (12, 4), (8, 1), (48, 3), (71, 1), (10, 2)]


def draw(rng):
    op = rng.choice(["rotary", "cache", "decode"])
    hq, hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128, 128, 256, 96, 80])
    page = rng.choice([16, 64, 64, 128, 24, 13, 1])
    cache = rng.choice(["bf16", "fp8"])
    if op == "rotary":
        T = _log_int(rng, 1, 8192)
        while T * (hq + 2 * hkv) * D > 4096 * 72 * 128:
            T = T * 2 // 3
        mode = rng.choice(["forward", "cached", "backward"])
        return _rotary(mode, T, hq, hkv, D, rot=rng.choice([D, D, 32]), interleaved=rng.random() < 0.3,
                       norm=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]),
                       theta=rng.choice([10000.0, 500000.0]), page=page, cache=cache if mode == "cached" else "none",
                       wgrad=rng.random() < 0.5)
    if op == "cache":
        T = _log_int(rng, 1, 32768)
        while T * hkv * D > 16384 * 8 * 128:
            T = T * 2 // 3
        return _cache(rng.choice(["write", "read"]), T, hkv, D, page=page, cache=cache,
                      dtype=rng.choice(["bf16", "bf16", "f32"]))
    B, longest = _log_int(rng, 1, 256), _log_int(rng, 1, 131072)
    while B * longest * hkv * D > 65536 * 8 * 128:
        B, longest = max(1, B * 2 // 3), max(1, longest * 3 // 4)
    return _decode(B, longest, hq, hkv, D, page=page, cache=cache,
                   window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0]))


# ---------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) & 0x7FFFFFFF)


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEVICE).normal_(0.0, std, generator=g)


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _quantize(x):
    """x [..., D] in 32 bits -> e4m3 codes [..., D], float32 scales [...]."""
    m, e = torch.frexp(x.abs().amax(dim=-1).clamp(min=AMAX_FLOOR))    # a = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int())
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def _lengths(c):
    """Cached tokens of each sequence, the new one among them: from one token to the longest."""
    r = random.Random(c["B"] * 1000003 + c["longest"])
    return [c["longest"]] + [r.randint(max(1, c["longest"] // 16), c["longest"]) for _ in range(c["B"] - 1)]


def _pool(g, c, n_pages, filled):
    """A paged cache as a user's program keeps it: keys and values [pages, heads, page, D], with scales in 8 bits."""
    shape, s = (n_pages, c["hkv"], c["page"], c["D"]), {}
    for x in ("k", "v"):
        if c["cache"] == "bf16":
            s[x] = torch.zeros(shape, dtype=torch.bfloat16, device=DEVICE)
            s[x + "_scales"] = None
        else:
            s[x] = torch.zeros(shape, dtype=torch.uint8, device=DEVICE).view(torch.float8_e4m3fn)
            s[x + "_scales"] = torch.ones(shape[:3], dtype=torch.float32, device=DEVICE)
        step = max(1, (1 << 24) // (shape[1] * shape[2] * shape[3]))
        for p0 in range(0, n_pages if filled else 0, step):
            p1 = min(n_pages, p0 + step)
            rows = _normal(g, (p1 - p0,) + shape[1:])
            if c["cache"] == "bf16":
                s[x][p0:p1] = rows
            else:
                q, z = _quantize(rows)
                s[x].view(torch.uint8)[p0:p1], s[x + "_scales"][p0:p1] = q.view(torch.uint8), z
    return s


def _slots(g, c, T):
    """Places of T rows in the cache: consecutive within a page, the pages in any order, a few more pages than needed."""
    n = -(-T // c["page"]) + 3
    order = torch.randperm(n, device=DEVICE, generator=g)
    t = torch.arange(T, device=DEVICE)
    return order[t // c["page"]] * c["page"] + t % c["page"], n


def _inverse_frequencies(c):
    return [c["theta"] ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]


def _turns(freqs):
    """The frequencies as turns a position in units of 2^-64, as a user's program keeps them."""
    t = [int(round(f / (2.0 * math.pi) * 2.0 ** 64)) for f in freqs]
    return torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in t], dtype=torch.int64, device=DEVICE)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        T, D, H = c["T"], c["D"], c["hq"] + c["hkv"]
        x = _normal(g, (T, H + c["hkv"], D)) * torch.exp(_normal(g, (H + c["hkv"], 1), 0.5))
        loud = torch.rand(D, device=DEVICE, generator=g) < 0.03
        s["qkv"] = (x * torch.where(loud, 6.0, 1.0)).to(_dtype(c)).reshape(T, -1)
        # sequences at any depth of their context
        s["positions"] = torch.randint(0, 131072, (T,), device=DEVICE, generator=g)
        freqs = _inverse_frequencies(c)
        s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device=DEVICE)
        s["turns"] = _turns(freqs)
        w = [(1.0 + _normal(g, (D,), 0.2)).to(_dtype(c)) for _ in range(2)]
        s["wq"], s["wk"] = w if c["norm"] else (None, None)
        if c["mode"] == "backward":
            s["dout"] = (_normal(g, (T, H * D)) * torch.exp(_normal(g, (T, 1)) - 9.0)).to(_dtype(c))
        if c["mode"] == "cached":
            s["slots"], n = _slots(g, c, T)
            s.update(_pool(g, c, n, False))
        return s
    if c["op"] == "cache":
        s["slots"], n = _slots(g, c, c["T"])
        s.update(_pool(g, c, n, c["mode"] == "read"))
        if c["mode"] == "write":
            loud = torch.exp(_normal(g, (c["hkv"] * c["D"],), 0.7))
            s["kv"] = torch.cat([_normal(g, (c["T"], c["hkv"] * c["D"])) * loud for _ in range(2)], 1).to(_dtype(c))
        return s
    lengths = _lengths(c)
    used = [-(-n // c["page"]) for n in lengths]
    s.update(_pool(g, c, sum(used) + 2, True))
    order = torch.randperm(sum(used), device=DEVICE, generator=g).int()
    table = torch.zeros((c["B"], max(used)), dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEVICE)
    s["q"] = _normal(g, (c["B"], c["hq"] * c["D"]), 2.0).bfloat16()
    return s


# -------------------------------------------------------------------------------------------------- the plain forms
def _split_pairs(c, x):
    """The rotated part of x [..., D] as its pairs' first and second members, and the rest."""
    r = x[..., :c["rot"]]
    if c["interleaved"]:
        return r[..., 0::2], r[..., 1::2], x[..., c["rot"]:]
    return r[..., :c["rot"] // 2], r[..., c["rot"] // 2:], x[..., c["rot"]:]


def _join_pairs(c, a, b, rest):
    r = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _angles(s):
    a = s["positions"].double()[:, None] * s["freqs"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _weights(s, dtype):
    """The norm weights of every head [heads, D]."""
    c = s["case"]
    return torch.cat([s["wq"].to(dtype).expand(c["hq"], -1), s["wk"].to(dtype).expand(c["hkv"], -1)])


def _turned_plain(s):
    """Queries and keys [T, heads, D] normalised and turned, in 32 bits."""
    c = s["case"]
    x = s["qkv"].float().reshape(c["T"], -1, c["D"])[:, :c["hq"] + c["hkv"]]
    if c["norm"]:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * _weights(s, torch.float32)
    cos, sin = _angles(s)
    a, b, rest = _split_pairs(c, x)
    return _join_pairs(c, a * cos - b * sin, b * cos + a * sin, rest)


def _write_plain(s, k, v):
    """Rows k and v [T, heads, D], in 32 bits, into the cache."""
    page, at = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
    if s["case"]["cache"] == "bf16":
        s["k"][page, :, at], s["v"][page, :, at] = k.bfloat16(), v.bfloat16()
        return
    (qk, zk), (qv, zv) = _quantize(k), _quantize(v)
    s["k"].view(torch.uint8)[page, :, at], s["v"].view(torch.uint8)[page, :, at] = qk.view(torch.uint8), qv.view(torch.uint8)
    s["k_scales"][page, :, at], s["v_scales"][page, :, at] = zk, zv


def _read_plain(s):
    """The rows of the slots [T, heads D] in 16 bits."""
    page, at, out = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"], {}
    for x in ("k", "v"):
        if s["case"]["cache"] == "bf16":
            rows = s[x][page, :, at]
        else:
            codes = s[x].view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn)
            rows = (codes.float() * s[x + "_scales"][page, :, at][..., None]).bfloat16()
        out[x] = rows.reshape(rows.shape[0], -1)
    return out


def _rotary_plain(s):
    c = s["case"]
    T, D, hq, hkv = c["T"], c["D"], c["hq"], c["hkv"]
    if c["mode"] != "backward":
        y = _turned_plain(s)
        if c["mode"] == "forward":
            return {"out": y.to(_dtype(c)).reshape(T, -1)}
        v = s["qkv"].float().reshape(T, -1, D)[:, hq + hkv:]
        _write_plain(s, y[:, hq:], v)
        return {"q": y[:, :hq].to(_dtype(c)).reshape(T, -1), **_read_plain(s)}
    cos, sin = _angles(s)
    a, b, rest = _split_pairs(c, s["dout"].float().reshape(T, hq + hkv, D))
    g = _join_pairs(c, a * cos + b * sin, b * cos - a * sin, rest)
    if not c["norm"]:
        return {"dx": g.to(_dtype(c)).reshape(T, -1)}
    x = s["qkv"].float().reshape(T, -1, D)[:, :hq + hkv]
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, wg = x * r, g * _weights(s, torch.float32)
    out = {"dx": (r * (wg - n * (wg * n).mean(-1, keepdim=True))).to(_dtype(c)).reshape(T, -1)}
    if c["wgrad"]:
        dw = (g * n).sum(0)
        out["dwq"], out["dwk"] = dw[:hq].sum(0), dw[hq:].sum(0)
    return out


def _cache_plain(s):
    c = s["case"]
    if c["mode"] == "write":
        kv = s["kv"].float().reshape(c["T"], 2, c["hkv"], c["D"])
        _write_plain(s, kv[:, 0], kv[:, 1])
    return _read_plain(s)


def _decode_plain(s):
    c = s["case"]
    B, D, hkv = c["B"], c["D"], c["hkv"]
    n, L = c["hq"] // hkv, c["longest"]
    t = torch.arange(L, device=DEVICE)
    page, at = s["table"].long()[:, t // c["page"]], (t % c["page"]).expand(B, L)

    def rows(x):
        if c["cache"] == "bf16":
            return s[x][page, :, at].float()
        codes = s[x].view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn)
        return codes.float() * s[x + "_scales"][page, :, at][..., None]

    k = rows("k").permute(0, 2, 3, 1)
    z = (s["q"].float().reshape(B, hkv, n, D) @ k) * D ** -0.5
    del k
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    end = s["lengths"].long()[:, None]
    seen = (t < end) & ((t >= end - c["window"]) if c["window"] else (t >= 0))
    z = torch.where(seen[:, None, None], z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    del z
    l = p.sum(-1, keepdim=True)
    o = (p @ rows("v").permute(0, 2, 1, 3)) / l
    return {"out": o.bfloat16().reshape(B, -1), "lse": (m + torch.log(l)).reshape(B, -1)}


# ------------------------------------------------------------------------------------------- this framework's calls
def _handle(s):
    return s["k"], s["v"], s["k_scales"], s["v_scales"]


def _rotary_own(s):
    import lora_co_serving_gb300 as lm
    c = s["case"]
    n = (c["hq"] + c["hkv"]) * c["D"]
    args = s["positions"], s["turns"], c["hq"], c["hkv"]
    kw = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=c["interleaved"])
    x = s["qkv"][:, :n]
    if c["mode"] == "forward":
        return {"out": lm.rotary_forward(x, *args, **kw)}
    if c["mode"] == "cached":
        q = lm.rotary_forward(x, *args, **kw, v=s["qkv"][:, n:], cache=_handle(s), slots=s["slots"])
        k, v = lm.cache_read(_handle(s), s["slots"])
        return {"q": q, "k": k, "v": v}
    if c["norm"] and c["wgrad"]:
        dx, dwq, dwk = lm.rotary_backward(x, *args, s["dout"], **kw, weight_grads=True)
        return {"dx": dx, "dwq": dwq, "dwk": dwk}
    return {"dx": lm.rotary_backward(x if c["norm"] else None, *args, s["dout"], **kw)}


def _cache_own(s):
    import lora_co_serving_gb300 as lm
    c = s["case"]
    n = c["hkv"] * c["D"]
    if c["mode"] == "write":
        lm.cache_write(s["kv"][:, :n], s["kv"][:, n:], _handle(s), s["slots"])
    k, v = lm.cache_read(_handle(s), s["slots"])
    return {"k": k, "v": v}


def _decode_own(s):
    import lora_co_serving_gb300 as lm
    c = s["case"]
    out, lse = lm.decode_attention(s["q"], _handle(s), s["table"], s["lengths"], window=c["window"],
                                   softcap=c["softcap"], want_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _rotary_own, "cache": _cache_own, "decode": _decode_own}[op](state)
    return {"rotary": _rotary_plain, "cache": _cache_plain, "decode": _decode_plain}[op](state)


# ------------------------------------------------------------------------------------------------------------ work
def _row_bytes(c):
    """Bytes of one head's row in the cache."""
    return 2 * c["D"] if c["cache"] == "bf16" else c["D"] + 4


def work(case):
    c = case
    if c["op"] == "decode":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
        io = c["B"] * c["hq"] * (4 * c["D"] + 4)
        return {"bytes": seen * c["hkv"] * 2 * _row_bytes(c) + io, "flops": 4 * seen * c["hq"] * c["D"]}
    T, D, hkv = c["T"], c["D"], c["hkv"]
    e = 2 if c["dtype"] == "bf16" else 4
    held, read = 2 * T * hkv * _row_bytes(c), 4 * T * hkv * D
    if c["op"] == "cache":
        write = 2 * T * hkv * D * e + held if c["mode"] == "write" else 0
        return {"bytes": write + held + read + 8 * T, "flops": 2 * T * hkv * D * (3 if c["mode"] == "write" else 1)}
    qk = T * (c["hq"] + hkv) * D
    if c["mode"] == "forward":
        return {"bytes": 2 * qk * e + 8 * T, "flops": 8 * qk}
    if c["mode"] == "cached":
        return {"bytes": e * (qk + T * hkv * D + T * c["hq"] * D) + 2 * held + read + 16 * T, "flops": 10 * qk}
    return {"bytes": (3 if c["norm"] else 2) * qk * e + 8 * T, "flops": (16 if c["norm"] else 3) * qk}


# -------------------------------------------------------------------------------------- the definitions in 64 bits
def _value64(x):
    """The value that 8 bits hold for each entry of x [..., D]: the nearest e4m3 number in units of its row's scale."""
    a = x.abs().amax(-1, keepdim=True).clamp(min=AMAX_FLOOR)
    s = torch.exp2(torch.floor(torch.log2(a)) - 9.0)
    s = torch.where(a > E4M3_MAX * s, 2.0 * s, s)            # twice at most: a < 2^(floor + 1) < 4 * 448 s
    s = torch.where(a > E4M3_MAX * s, 2.0 * s, s)
    v = x / s
    # e4m3: 3 mantissa bits, exponents from -6; numbers below 2^-6 are multiples of 2^-9
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step * s


def _complex64(c, x):
    """The rotated part of x [..., D] as complex numbers."""
    if c["interleaved"]:
        return torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:-1], -1, 2).contiguous())
    h = c["rot"] // 2
    return torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous())


def _turn64(s, x, sign):
    """x [T, heads, D] turned by sign times its positions' angles."""
    c = s["case"]
    angle = sign * s["positions"].double()[:, None, None] * s["freqs"]
    z = _complex64(c, x) * torch.polar(torch.ones_like(angle), angle)
    part = torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([part, x[..., c["rot"]:]], -1)


def _held64(c, x):
    return _value64(x) if c["cache"] == "fp8" else x


def _rows64(s, x, pages, offsets):
    r = s[x].float()[pages, :, offsets].double() if s[x].dtype is torch.bfloat16 else \
        s[x].view(torch.uint8)[pages, :, offsets].view(torch.float8_e4m3fn).float().double()
    return r if s[x + "_scales"] is None else r * s[x + "_scales"][pages, :, offsets].double()[..., None]


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    D = c["D"]
    if c["op"] == "rotary":
        T, hq, H = c["T"], c["hq"], c["hq"] + c["hkv"]
        qkv = s["qkv"].double().reshape(T, -1, D)
        x = qkv[:, :H]
        rms = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
        w = _weights(s, torch.float64) if c["norm"] else None
        if c["mode"] != "backward":
            y = _turn64(s, x / rms * w if c["norm"] else x, 1.0)
            if c["mode"] == "forward":
                return {"out": y.reshape(T, -1)}
            return {"q": y[:, :hq].reshape(T, -1), "k": _held64(c, y[:, hq:]).reshape(T, -1),
                    "v": _held64(c, qkv[:, H:]).reshape(T, -1)}
        g = _turn64(s, s["dout"].double().reshape(T, H, D), -1.0)
        if not c["norm"]:
            return {"dx": g.reshape(T, -1)}
        along = (g * w * x).sum(-1, keepdim=True)
        out = {"dx": (g * w / rms - x * along / (D * rms ** 3)).reshape(T, -1)}
        if c["wgrad"]:
            out["dwq"], out["dwk"] = (t.sum((0, 1)) for t in (g * x / rms).split([hq, H - hq], 1))
        return out
    if c["op"] == "cache":
        if c["mode"] == "write":
            kv = s["kv"].double().reshape(c["T"], 2, c["hkv"], D)
            return {"k": _held64(c, kv[:, 0]).reshape(c["T"], -1), "v": _held64(c, kv[:, 1]).reshape(c["T"], -1)}
        pages, offsets = s["slots"] // c["page"], s["slots"] % c["page"]
        return {x: _rows64(s, x, pages, offsets).reshape(c["T"], -1) for x in ("k", "v")}
    n = c["hq"] // c["hkv"]
    out = torch.empty((c["B"], c["hkv"], n, D), dtype=torch.float64, device=DEVICE)
    lse = torch.empty((c["B"], c["hkv"], n), dtype=torch.float64, device=DEVICE)
    for b, length in enumerate(_lengths(c)):
        t = torch.arange(max(0, length - c["window"]) if c["window"] else 0, length, device=DEVICE)
        pages, offsets = s["table"][b].long()[t // c["page"]], t % c["page"]
        k, v = (_rows64(s, x, pages, offsets).transpose(0, 1) for x in ("k", "v"))
        z = torch.einsum("hnd,htd->hnt", s["q"][b].double().reshape(c["hkv"], n, D), k) / math.sqrt(D)
        if c["softcap"]:
            z = c["softcap"] * torch.tanh(z / c["softcap"])
        lse[b] = torch.logsumexp(z, -1)
        out[b] = torch.softmax(z, -1) @ v
    return {"out": out.reshape(c["B"], -1), "lse": lse.reshape(c["B"], -1)}
