"""Measured cases of the operators around the LoRA layer in a fine-tuning step of a co-served decoder:

  linear      a frozen projection (an MLP's, a head's: no adapter) as a product of 8-bit floating point (e4m3) numbers
              with a float32 scale for each block of 128: activations per row and 128 columns, weights per 128 x 128.
              An activation's scale is the smallest power of two that brings its block within e4m3's largest number
  swiglu      the MLP's activation h = silu(gate) * up, which keeps an 8-bit checkpoint of gate|up for the fine-tuning
              rows of the batch, and its backward from that checkpoint
  preference  the paired log-ratio loss of a policy against a reference over a batch of (chosen, rejected) sequences,
              and the gradient of the logits

Where `own` is false, run() computes a pass in elementary torch operations in 32 bits; where it is true, it makes the
calls of this framework.  exact() gives the same outputs in 64 bits from the definitions.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128          # columns (and weight rows) that share a scale
E4M3_MAX = 448.0     # largest e4m3 value
AMAX_FLOOR = 2.0 ** -100   # a block's largest magnitude is taken as at least this, so that no scale is zero
DEVICE = "cuda"


# ----------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode token through an attention-sized projection: launch and memory latency
        dict(name="linear decode 1", op="linear", T=1, K=4096, N=4096, x="bf16", grad=False),
        # a decode batch of 256 tokens through the fused gate|up projection of an 8B-sized layer: weight bandwidth
        dict(name="linear decode 256 gate-up", op="linear", T=256, K=4096, N=28672, x="bf16", grad=False),
        # a ragged prefill through the down projection, its input already in 8 bits from the activation
        dict(name="linear prefill 1111 down", op="linear", T=1111, K=14336, N=4096, x="fp8", grad=False),
        # the input gradient of 2048 fine-tuning rows through a 70B-sized frozen MLP projection
        dict(name="linear dX 2048", op="linear", T=2048, K=28672, N=8192, x="bf16", grad=True),
        # the whole co-serving batch of 8192 tokens through a 70B-sized MLP projection: compute
        dict(name="linear co-serving 8192", op="linear", T=8192, K=8192, N=28672, x="bf16", grad=False),
        # the activation of a small decode batch, no fine-tuning rows: latency
        dict(name="swiglu decode 33", op="swiglu", mode="forward", T=33, I=14336, train=0, n_seg=0, dtype="bf16"),
        # the co-serving batch's activation with its 2048 fine-tuning rows checkpointed, and their backward
        dict(name="swiglu step 8192", op="swiglu", mode="step", T=8192, I=14336, train=2048, n_seg=2, dtype="bf16"),
        # the backward of ragged fine-tuning segments at the 70B width
        dict(name="swiglu backward 1999", op="swiglu", mode="backward", T=1999, I=28672, train=1999, n_seg=5,
             dtype="bf16"),
        # the loss alone of two short pairs (an evaluation step): latency
        dict(name="preference loss 60", op="preference", mode="forward", pairs=2, T=60, V=32000, dtype="bf16"),
        # a usual step: 8 pairs, 4096 tokens, a 32k vocabulary
        dict(name="preference step 4096", op="preference", mode="step", pairs=8, T=4096, V=32000, dtype="bf16"),
        # the gradient in float32 over a vocabulary of odd size
        dict(name="preference grad f32", op="preference", mode="backward", pairs=3, T=1501, V=50257, dtype="f32"),
        # a large step: 16 pairs, 4096 tokens, a 128k vocabulary; the logits do not fit the L2
        dict(name="preference step 128k", op="preference", mode="step", pairs=16, T=4096, V=128256, dtype="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["linear", "swiglu", "preference"])
    if op == "linear":
        while True:
            c = dict(op=op, T=_log_int(rng, 1, 8192), K=_log_int(rng, 256, 28672, 16), N=_log_int(rng, 256, 28672, 8),
                     x=rng.choice(["bf16", "fp8"]), grad=rng.random() < 0.3)
            if c["T"] * c["K"] * c["N"] <= 8192 * 8192 * 28672 and c["K"] * c["N"] <= 8192 * 28672:
                return c
    if op == "swiglu":
        c = dict(op=op, mode=rng.choice(["forward", "step", "backward"]), T=_log_int(rng, 1, 8192),
                 I=_log_int(rng, 256, 28672, 8), dtype=rng.choice(["bf16", "bf16", "f32"]))
        while c["T"] * c["I"] > 4096 * 14336:
            c["T"], c["I"] = max(1, c["T"] * 2 // 3), max(256, c["I"] * 3 // 32 * 8)
        c["train"] = c["T"] if c["mode"] == "backward" else max(1, int(c["T"] * rng.choice([0.1, 0.25, 0.6])))
        c["n_seg"] = min(c["train"], rng.randint(1, 12))
        return c
    c = dict(op=op, mode=rng.choice(["forward", "step", "backward"]), pairs=_log_int(rng, 1, 32),
             V=_log_int(rng, 500, 152000), dtype=rng.choice(["bf16", "bf16", "f32"]))
    c["T"] = max(2 * c["pairs"], _log_int(rng, 16, 8192))
    while c["T"] * c["V"] > 1024 * 128256 and c["T"] > 2 * c["pairs"]:
        c["T"] = max(2 * c["pairs"], c["T"] // 2 + 1)
    return c


# ---------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) & 0x7FFFFFFF)


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEVICE).normal_(0.0, std, generator=g)


def _blocks(x, fill=0.0):
    """x [T, K] as [T, ceil(K / 128), 128], the last block filled up."""
    T, K = x.shape
    n = -(-K // BLOCK)
    if n * BLOCK != K:
        x = torch.nn.functional.pad(x, (0, n * BLOCK - K), value=fill)
    return x.reshape(T, n, BLOCK)


def _quantize(x):
    """x [T, K] in 32 bits -> e4m3 codes [T, K], float32 scales [T, ceil(K / 128)]."""
    T, K = x.shape
    b = _blocks(x)
    m, e = torch.frexp(b.abs().amax(dim=2).clamp(min=AMAX_FLOOR))    # a = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int())
    q = (b / s[:, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(T, -1)[:, :K].contiguous(), s.contiguous()


def _spread(s, K):
    """Scales [R, ceil(K / 128)] spread to the K columns."""
    return s.repeat_interleave(BLOCK, dim=1)[:, :K]


def _weight(g, N, K):
    """A frozen weight [N, K] in 8 bits, as a user's program keeps it: e4m3 codes and a scale per 128 x 128 block."""
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    codes = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=DEVICE)
    scales = torch.empty((nb, kb), dtype=torch.float32, device=DEVICE)
    rows = 16 * BLOCK                            # whole blocks of rows at a time
    for n0 in range(0, N, rows):
        w = _normal(g, (min(rows, N - n0), K), K ** -0.5)
        R = -(-w.shape[0] // BLOCK)
        p = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, R * BLOCK - w.shape[0]))
        p = p.reshape(R, BLOCK, kb, BLOCK)
        a = p.abs().amax(dim=(1, 3)).clamp(min=AMAX_FLOOR)
        q = (p * (E4M3_MAX / a)[:, None, :, None]).to(torch.float8_e4m3fn).reshape(R * BLOCK, kb * BLOCK)
        codes[n0:n0 + w.shape[0]] = q[:w.shape[0], :K]
        scales[n0 // BLOCK:n0 // BLOCK + R] = a / E4M3_MAX
    return codes, scales


def _activations(g, T, K, grad):
    """Activations with a few channels of large magnitude, or gradients whose rows differ in magnitude."""
    x = _normal(g, (T, K))
    if grad:
        return x * torch.exp(_normal(g, (T, 1)) - 9.0)
    loud = torch.rand(K, device=DEVICE, generator=g) < 0.004
    return x * torch.where(loud, 12.0, 1.0)


def _segments(c):
    """The batch's segment table: fine-tuning segments (adapter 0) among prefill and decode rows."""
    T, train, n = c["T"], c["train"], c["n_seg"]
    segs, t, left = [], 0, T - train
    for i in range(n):
        gap = left // (n + 1 - i)
        if gap:
            segs.append((t, gap, 1, 0))
            t, left = t + gap, left - gap
        ln = train // n + (1 if i < train % n else 0)
        segs.append((t, ln, 0, 1))
        t += ln
    if left:
        segs.append((t, left, -1, 0))
    return np.asarray(segs, np.int32).reshape(-1, 4)


def _train_rows(segs):
    rows = [np.arange(s, s + n) for s, n, _, tr in segs.tolist() if tr]
    return np.concatenate(rows) if rows else np.zeros(0, np.int64)


def _pairs(c):
    """Rows of the batch's sequences: [pairs, 4] = chosen start and length, rejected start and length, adding up to T."""
    r = random.Random(c["T"] * 1000003 + c["pairs"])
    n = 2 * c["pairs"]
    cuts = sorted(r.sample(range(1, c["T"]), n - 1)) if c["T"] > n else list(range(1, n))
    edge = [0] + cuts + [c["T"]]
    return np.asarray([[edge[2 * p], edge[2 * p + 1] - edge[2 * p], edge[2 * p + 1], edge[2 * p + 2] - edge[2 * p + 1]]
                       for p in range(c["pairs"])], np.int32)


def _sequence_of(pairs, T):
    """Sequence of each row: 2 p for the chosen one of pair p, 2 p + 1 for the rejected one."""
    s = np.zeros(T, np.int64)
    for p, (c0, cn, r0, rn) in enumerate(pairs.tolist()):
        s[c0:c0 + cn], s[r0:r0 + rn] = 2 * p, 2 * p + 1
    return s


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "linear":
        s["w"], s["ws"] = _weight(g, c["N"], c["K"])
        x = _activations(g, c["T"], c["K"], c["grad"])
        if c["x"] == "fp8":
            s["x"], s["xs"] = _quantize(x)
        else:
            s["x"], s["xs"] = x.to(torch.bfloat16), None
        return s
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    if c["op"] == "swiglu":
        s["segs"] = _segments(c)
        rows = _train_rows(s["segs"])
        s["rows"] = torch.from_numpy(rows).to(DEVICE)
        if c["mode"] != "forward":
            s["dh"] = _activations(g, len(rows), c["I"], True).to(dtype)
        gu = _normal(g, (c["T"], 2 * c["I"]), 1.5).to(dtype)
        if c["mode"] == "backward":              # the checkpoint is in hand: gate and up, in row blocks of 128 each
            halves = [_quantize(h.float()) for h in (gu[:, :c["I"]], gu[:, c["I"]:])]
            s["codes"] = torch.cat([h[0].view(torch.uint8) for h in halves], 1).view(torch.float8_e4m3fn)
            s["scales"] = torch.cat([h[1] for h in halves], 1)
        else:
            s["gu"] = gu
        return s
    T, V = c["T"], c["V"]
    s["pairs"] = _pairs(c)
    s["seq"] = torch.from_numpy(_sequence_of(s["pairs"], T)).to(DEVICE)
    labels = torch.randint(0, V, (T,), device=DEVICE, generator=g)
    x = torch.empty((T, V), dtype=dtype, device=DEVICE)
    for t0 in range(0, T, 1024):                 # logits of a trained model: the label's token stands out
        n = min(1024, T - t0)
        x[t0:t0 + n] = _normal(g, (n, V), 2.0)
    x[torch.arange(T, device=DEVICE), labels] += (torch.rand(T, device=DEVICE, generator=g) * 14.0).to(dtype)
    s["x"] = x
    # prompt tokens carry no label: the first part of each sequence
    first = torch.from_numpy(np.repeat(s["pairs"].reshape(-1, 2)[:, 0], s["pairs"].reshape(-1, 2)[:, 1])).to(DEVICE)
    size = torch.from_numpy(np.repeat(s["pairs"].reshape(-1, 2)[:, 1], s["pairs"].reshape(-1, 2)[:, 1])).to(DEVICE)
    prompt = torch.arange(T, device=DEVICE) - first < (size * 0.3).long()
    s["labels"] = torch.where(prompt, torch.full_like(labels, -1), labels)
    lse = torch.empty(T, device=DEVICE)
    for t0 in range(0, T, 1024):
        lse[t0:t0 + 1024] = torch.logsumexp(x[t0:t0 + 1024].float(), 1)
    lp = x.gather(1, labels[:, None])[:, 0].float() - lse
    s["ref"] = torch.where(prompt, torch.zeros_like(lp), lp + _normal(g, (T,), 0.3))
    s["beta"], s["smooth"] = 0.1, 0.05
    s["dloss"] = torch.full((c["pairs"],), 1.0 / c["pairs"], device=DEVICE)
    if c["mode"] == "backward":                  # what the loss's forward leaves for its backward
        s["lse"] = torch.where(prompt, torch.zeros_like(lse), lse)
        s["coef"] = (torch.rand(2 * c["pairs"], device=DEVICE, generator=g) - 0.5) * 2.0 * s["beta"]
    return s


# -------------------------------------------------------------------------------------------------- the plain forms
def _linear_plain(s):
    c = s["case"]
    q, xs = (s["x"], s["xs"]) if s["xs"] is not None else _quantize(s["x"].float())
    x = q.float() * _spread(xs, c["K"])
    w = s["w"].float() * _spread(s["ws"], c["K"]).repeat_interleave(BLOCK, dim=0)[:c["N"]]
    return (x @ w.t()).to(torch.bfloat16)


def _swiglu_plain(s):
    c, out = s["case"], {}
    I = c["I"]
    if c["mode"] != "backward":
        g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
        out["h"] = (g / (1.0 + torch.exp(-g)) * u).to(s["gu"].dtype)
    if c["mode"] == "forward":
        return out
    if c["mode"] == "step":
        g, u = (q.float() * _spread(z, I) for q, z in (_quantize(v[s["rows"]]) for v in (g, u)))
    else:
        n = -(-I // BLOCK)
        g = s["codes"][:, :I].float() * _spread(s["scales"][:, :n], I)
        u = s["codes"][:, I:].float() * _spread(s["scales"][:, n:], I)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    out["dgu"] = torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1).to(s["dh"].dtype)
    return out


def _preference_plain(s):
    c, out = s["case"], {}
    counted = s["labels"] >= 0
    at = s["labels"].clamp(min=0)[:, None]
    x = s["x"].float()
    if c["mode"] == "backward":
        lse, coef = s["lse"], s["coef"]
    else:
        m = x.amax(1)
        lse = m + torch.log(torch.exp(x - m[:, None]).sum(1))
        logp = torch.where(counted, x.gather(1, at)[:, 0] - lse, torch.zeros_like(lse))
        d = torch.zeros(2 * c["pairs"], device=x.device)
        d.index_add_(0, s["seq"], torch.where(counted, logp - s["ref"], torch.zeros_like(logp)))
        d = (s["beta"] * d).reshape(-1, 2)
        m = d[:, 0] - d[:, 1]
        soft = torch.log1p(torch.exp(-m.abs()))  # -log sigmoid(m) = max(-m, 0) + soft
        out["loss"] = (1.0 - s["smooth"]) * (torch.clamp(-m, min=0) + soft) + s["smooth"] * (torch.clamp(m, min=0) + soft)
        out["rewards"], out["logp"] = d, logp
        sig = 1.0 / (1.0 + torch.exp(-m))
        k = s["beta"] * (s["smooth"] * sig - (1.0 - s["smooth"]) * (1.0 - sig))
        coef = torch.stack([k, -k], 1).reshape(-1)
    if c["mode"] == "forward":
        return out
    k = torch.where(counted, coef[s["seq"]] * s["dloss"][s["seq"] // 2], torch.zeros_like(lse))
    p = torch.exp(x - lse[:, None])
    p = torch.where(counted[:, None], p, torch.zeros_like(p))
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    out["dlogits"] = (p * -k[:, None]).to(s["x"].dtype)
    return out


# ------------------------------------------------------------------------------------------- this framework's calls
def _linear_own(s):
    import lora_co_serving_gb300 as lm
    return lm.fp8_linear(s["x"], s["w"], s["ws"], x_scales=s["xs"])


def _swiglu_own(s):
    import lora_co_serving_gb300 as lm
    mode, out = s["case"]["mode"], {}
    if mode == "forward":
        out["h"] = lm.swiglu_forward(s["gu"])
        return out
    if mode == "step":
        out["h"], saved = lm.swiglu_forward(s["gu"], s["segs"], checkpoint=True)
    else:
        saved = (s["codes"], s["scales"])
    out["dgu"] = lm.swiglu_backward(saved, s["dh"])
    return out


def _preference_own(s):
    import lora_co_serving_gb300 as lm
    mode, out = s["case"]["mode"], {}
    if mode == "backward":
        lse, coef = s["lse"], s["coef"]
    else:
        f = lm.preference_forward(s["x"], s["labels"], s["ref"], s["pairs"], s["beta"], s["smooth"])
        out["loss"], out["rewards"], out["logp"], lse, coef = f.loss, f.rewards, f.logp, f.lse, f.coef
    if mode != "forward":
        out["dlogits"] = lm.preference_backward(s["x"], s["labels"], lse, coef, s["pairs"], dloss=s["dloss"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _linear_own, "swiglu": _swiglu_own, "preference": _preference_own}[op](state)
    return {"linear": _linear_plain, "swiglu": _swiglu_plain, "preference": _preference_plain}[op](state)


# ------------------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        nk, nn = -(-K // BLOCK), -(-N // BLOCK)
        x = 2 * T * K if c["x"] == "bf16" else T * K + 4 * T * nk
        return {"bytes": x + N * K + 4 * nn * nk + 2 * T * N, "flops": 2 * T * K * N}
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "swiglu":
        T, I, R = c["T"], c["I"], c["train"]
        kept = R * (2 * I + 8 * -(-I // BLOCK))          # the checkpoint: codes and scales
        fwd = 3 * T * I * e
        bwd = 3 * R * I * e
        return {"forward": {"bytes": fwd, "flops": 6 * T * I},
                "step": {"bytes": fwd + 2 * kept + bwd, "flops": 6 * T * I + 20 * R * I},
                "backward": {"bytes": kept + bwd, "flops": 16 * R * I}}[c["mode"]]
    T, V = c["T"], c["V"]
    counted = sum(int(n) - int(n * 0.3) for n in _pairs(c).reshape(-1, 2)[:, 1])
    read = counted * V * e + 20 * T
    return {"bytes": read + (0 if c["mode"] == "forward" else T * V * e),
            "flops": counted * V * {"forward": 4, "step": 8, "backward": 4}[c["mode"]]}


# -------------------------------------------------------------------------------------- the definitions in 64 bits
def _value64(x):
    """The value that 8 bits hold for each entry of x [T, K]: the nearest e4m3 number in units of its block's scale."""
    out = torch.empty_like(x)
    for k0 in range(0, x.shape[1], BLOCK):
        b = x[:, k0:k0 + BLOCK]
        a = b.abs().max(dim=1, keepdim=True).values.clamp(min=AMAX_FLOOR)
        s = torch.exp2(torch.floor(torch.log2(a)) - 9.0)
        s = torch.where(a > E4M3_MAX * s, 2.0 * s, s)        # twice at most: a < 2^(floor + 1) < 4 * 448 s
        s = torch.where(a > E4M3_MAX * s, 2.0 * s, s)
        v = b / s
        # e4m3: 3 mantissa bits, exponents from -6; numbers below 2^-6 are multiples of 2^-9
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
        out[:, k0:k0 + BLOCK] = torch.round(v / step) * step * s
    return out


def _scaled64(codes, scales):
    v = codes.float().double()
    for b in range(scales.shape[1]):
        v[:, BLOCK * b:BLOCK * (b + 1)] *= scales[:, b:b + 1].double()
    return v


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "linear":
        x = _scaled64(s["x"], s["xs"]) if c["x"] == "fp8" else _value64(s["x"].double())
        y = torch.empty((c["T"], c["N"]), dtype=torch.float64, device=DEVICE)
        for j in range(-(-c["N"] // BLOCK)):
            n0, n1 = j * BLOCK, min(c["N"], (j + 1) * BLOCK)
            w = _scaled64(s["w"][n0:n1].contiguous(), s["ws"][j:j + 1].expand(n1 - n0, -1))
            y[:, n0:n1] = x @ w.t()
        return y
    if c["op"] == "swiglu":
        I, out = c["I"], {}
        if c["mode"] != "backward":
            gu = s["gu"].double()
            out["h"] = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        if c["mode"] == "forward":
            return out
        if c["mode"] == "step":
            g, u = _value64(gu[s["rows"], :I]), _value64(gu[s["rows"], I:])
        else:
            n = -(-I // BLOCK)
            g, u = _scaled64(s["codes"][:, :I].contiguous(), s["scales"][:, :n]), \
                _scaled64(s["codes"][:, I:].contiguous(), s["scales"][:, n:])
        dh, sig = s["dh"].double(), torch.sigmoid(g)
        out["dgu"] = torch.cat([dh * u * (sig + g * sig * (1.0 - sig)), dh * g * sig], 1)
        return out
    T, V, P = c["T"], c["V"], c["pairs"]
    out, rows = {}, torch.nonzero(s["labels"] >= 0)[:, 0]
    if c["mode"] == "backward":
        lse, coef = s["lse"].double(), s["coef"].double()
    else:
        lse, logp = torch.zeros(T, dtype=torch.float64, device=DEVICE), torch.zeros(T, dtype=torch.float64,
                                                                                    device=DEVICE)
        for r in rows.split(512):
            x = s["x"][r].double()
            lse[r] = torch.logsumexp(x, 1)
            logp[r] = x.gather(1, s["labels"][r][:, None])[:, 0] - lse[r]
        gain = torch.stack([s["beta"] * (logp - s["ref"].double())[s["labels"].ge(0) & s["seq"].eq(q)].sum()
                            for q in range(2 * P)]).reshape(P, 2)
        m = gain[:, 0] - gain[:, 1]
        e = s["smooth"]
        out["loss"] = -(1.0 - e) * torch.nn.functional.logsigmoid(m) - e * torch.nn.functional.logsigmoid(-m)
        out["rewards"], out["logp"] = gain, logp
        k = s["beta"] * (e * torch.sigmoid(m) - (1.0 - e) * torch.sigmoid(-m))
        coef = torch.stack([k, -k], 1).reshape(-1)
    if c["mode"] == "forward":
        return out
    d = torch.zeros((T, V), dtype=torch.float64, device=DEVICE)
    for r in rows.split(512):
        k = (coef[s["seq"][r]] * s["dloss"].double()[s["seq"][r] // 2])[:, None]
        g = -k * torch.exp(s["x"][r].double() - lse[r][:, None])
        g.scatter_add_(1, s["labels"][r][:, None], k)
        d[r] = g
    out["dlogits"] = d
    return out
