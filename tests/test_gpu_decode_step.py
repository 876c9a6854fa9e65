"""The attention side's operators together, as a step of mixed decode, prefill and fine-tuning rows uses them.

Tolerances: the parts' own (test_gpu_rotary.py, test_gpu_decode.py), applied to the float64 forms of the values that the
step really used: what the projection gave, and what the cache held."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import lora_co_serving_gb300 as lm
from attention_oracle import BF, E4, U, angles, attention, frequencies, normed, quantized, reach, turned

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_mixed_step(e4m3):
    """One batch of 5 decode rows, a prefill of 40 rows and 30 fine-tuning rows through q|k|v, rotation, cache, attention
    and, for the fine-tuning rows, back to the projection's gradients."""
    hidden, hq, hk, D, page = 256, 8, 4, 64, 16
    q, kv = hq * D, hk * D
    N, n = q + 2 * kv, q + kv
    g = torch.Generator().manual_seed(3)
    ranks = np.array([8, 16], np.int32)
    A = (torch.rand(24 * hidden * 3, generator=g) - 0.5).mul_(2 * hidden ** -0.5).bfloat16().cuda()
    B = (0.1 * torch.randn(24 * N, generator=g)).bfloat16().cuda()
    pool = lm.Pool(A, B, np.array([0, 8 * hidden * 3]), np.array([0, 8 * N]), ranks, np.full(2, 2.0))
    W = (torch.randn(N, hidden, generator=g) * hidden ** -0.5).bfloat16().cuda()
    bounds = [0, q, n, N]
    segs = [(i, 1, i % 3 - 1, 0) for i in range(5)] + [(5, 40, 0, 0), (45, 30, 1, 1)]
    x = torch.randn(75, hidden, generator=g).bfloat16().cuda()
    qkv, xa = lm.sliced_forward(x, W, pool, bounds, segs, save_xa=True)

    # contexts of the decode rows: rows already cached
    past = [33, 0, 16, 100, 7]
    cache = lm.kv_cache(32, hk, page, D, torch.float8_e4m3fn if e4m3 else bf16)
    order = torch.randperm(32, generator=g)
    table = torch.zeros((6, 7), dtype=torch.int32)
    at = 0
    for b, L in enumerate(past + [39]):
        k = -(-(L + 1) // page)
        table[b, :k] = order[at:at + k].int()
        at += k

    def slot(b, t):
        return int(table[b, t // page]) * page + t % page

    old = [(b, t) for b in range(5) for t in range(past[b])]
    rows = torch.randn(2, len(old), kv, generator=g).bfloat16()
    lm.cache_write(rows[0].cuda(), rows[1].cuda(), cache, torch.tensor([slot(b, t) for b, t in old]).cuda())
    positions = torch.tensor(past + list(range(40)) + list(range(30)))
    slots = torch.tensor([slot(b, past[b]) for b in range(5)] + [slot(5, t) for t in range(40)] + [-1] * 30)
    turns = lm.rotary_turns(D)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16() for _ in range(2)]
    args = (positions.cuda(), turns, hq, hk)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda())
    qk = lm.rotary_forward(qkv[:, :n], *args, **kw, v=qkv[:, n:], cache=cache, slots=slots.cuda(), keep_keys=True)

    # queries and keys of every row
    y = qkv.cpu().double().reshape(75, -1, D)
    heads = torch.cat([normed(y[:, :hq], w[0].double()), normed(y[:, hq:hq + hk], w[1].double())], 1)
    angle = angles(positions, frequencies(D))
    ref, mag = turned(heads, angle, D, False), reach(heads, D, False)
    err = (qk.cpu().double().reshape(75, -1, D) - ref).abs()
    assert (err <= BF * ref.abs() + 32 * U * mag).all()

    # the cache holds the decode and prefill rows, rounded once
    got = [t.cpu().double().reshape(75, hk, D) for t in lm.cache_read(cache, slots.cuda(), dtype=torch.float32)]
    kept = ref[:45, hq:]
    tol = (E4 * kept.abs() + 2.0 ** -9 * quantized(kept)[1][..., None] if e4m3 else BF * kept.abs()) + 32 * U * mag[:45, hq:]
    assert ((got[0][:45] - kept).abs() <= tol).all() and (got[0][45:] == 0).all()
    v = y[:45, hq + hk:]
    assert torch.equal(got[1][:45], quantized(v)[0] if e4m3 else v)

    # decode rows, and the prefill's last row, over what the cache holds
    lengths = torch.tensor([L + 1 for L in past] + [40], dtype=torch.int32)
    queries = torch.cat([qk[:5, :q], qk[44:45, :q]])
    out, lse = lm.decode_attention(queries, cache, table.cuda(), lengths.cuda(), want_lse=True)
    for b, L in enumerate(lengths.tolist()):
        s = torch.tensor([slot(b, t) for t in range(L)]).cuda()
        k64, v64 = (t.cpu().double().reshape(L, hk, D) for t in lm.cache_read(cache, s, dtype=torch.float32))
        for h in range(hk):
            r = queries[b].cpu().double().reshape(hk, hq // hk, D)[h]
            o, z, p, sc = attention(r, k64[:, h], v64[:, h], D ** -0.5)
            most = (r.abs() @ k64[:, h].abs().t()).amax() * D ** -0.5
            delta = D * 2.0 ** -23 * most + 2.0 ** -20 * sc.abs().amax()
            tol = (2 * (delta + 2.0 ** -21) + 2.0 ** -11 + (L + 64) * 2.0 ** -23) * (p @ v64[:, h].abs()) + BF * o.abs()
            assert ((out[b].cpu().double().reshape(hk, hq // hk, D)[h] - o).abs() <= tol).all()

    # the fine-tuning rows' gradient, in the projection's own buffer, on to the adapters
    train = slice(45, 75)
    dqkv = torch.zeros(75, N, dtype=bf16, device="cuda")
    dqkv[train] = (0.01 * torch.randn(30, N, generator=g)).bfloat16().cuda()
    d64 = dqkv[train, :n].cpu().double().reshape(30, hq + hk, D)
    lm.rotary_backward(qkv[train, :n], positions[train].cuda(), turns, hq, hk, dqkv[train, :n], **kw, dx=dqkv[train, :n])
    leaf = y[train, :hq + hk].clone().requires_grad_()
    again = torch.cat([normed(leaf[:, :hq], w[0].double()), normed(leaf[:, hq:], w[1].double())], 1)
    turned(again, angle[train], D, False).backward(d64)
    err = (dqkv[train, :n].cpu().double().reshape(30, hq + hk, D) - leaf.grad).abs()
    big = reach(d64, D, False)
    r = torch.rsqrt(y[train, :hq + hk].square().mean(-1, keepdim=True))
    size = 1.0 + y[train, :hq + hk].abs() * r
    tol = BF * leaf.grad.abs() + 64 * U * r * 2.0 * size * (big + (big * size).mean(-1, keepdim=True))   # weights below 2
    assert (err <= tol).all()
    dX, dA, dB = lm.sliced_backward(x, W, pool, bounds, segs, dqkv, xa_saved=xa)
    assert dA.isfinite().all() and dB.isfinite().all() and dB[8 * N:].abs().sum() > 0 and (dB[:8 * N] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decode_loop(e4m3):
    """The example runs, gives the same tokens from a graph as without one, and its cache holds whole sequences."""
    import decode_loop
    eager = decode_loop.run(20, e4m3=e4m3, capture=False)
    graph = decode_loop.run(20, e4m3=e4m3)
    for a, b in zip(eager[:2] + eager[3:], graph[:2] + graph[3:]):
        assert torch.equal(a, b)
    tokens, logits, cache, table, lengths = graph
    assert logits.isfinite().all() and tokens.shape == (5, 20)
    for b, n in enumerate(lengths.tolist()):
        t = torch.arange(n, device="cuda")
        slots = table[b].long()[t // 16] * 16 + t % 16
        for got, want in zip(lm.cache_read(cache, slots), lm.cache_read(eager[2], slots)):
            assert torch.equal(got, want) and (got.abs().sum(1) > 0).all()
    assert math.isfinite(float(logits.float().abs().max()))
