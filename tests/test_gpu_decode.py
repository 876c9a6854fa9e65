"""Attention of one new token over the paged cache, against float64 on the CPU.

Tolerances, with S the largest scale sum_d |q_d k_d| of a row and u = 2^-24:
  score       D products added in float32 by the tensor core, which may truncate: D 2^-23 S; the scale, the change to powers
              of two and, where scores are capped, the tangent (2 units) and two more: 8 u of |score| + 4 u of the cap.
              Capping does not enlarge an error.  delta = D 2^-23 S + 2^-20 (|score| + cap)
  weight      e^s: delta and the exponential's 2 units: delta + 2^-21, and the same for the sum it is divided by
  product     a probability in bf16 and its rest in bf16: half a step of half a step, 2^-16 of it; 8-bit caches: in fp16,
              half a step, 2^-11; L terms and their joins added in float32: (L + 64) 2^-23
  out         (2 (delta + 2^-21) + 2^-16 or 2^-11 + (L + 64) 2^-23) sum_j p_j |v_j|, then half a step of bf16
  lse         delta + 2^-21 + (L + 64) 2^-23, and 2^-22 of itself
"""
import math

import pytest
import torch

import lora_co_serving_gb300 as lm
from attention_oracle import BF, attention, quantized

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Case:
    """Sequences of given lengths over pages in any order; every row and table entry that is not theirs is poison."""

    def __init__(self, lengths, hq, hkv, D, page=16, e4m3=False, layout="heads first", spread=0.5, seed=0, extra=2, q_std=2.0):
        g = gen(seed + sum(lengths) + D)
        self.lengths, self.hq, self.hkv, self.D, self.page, self.e4m3 = lengths, hq, hkv, D, page, e4m3
        B = len(lengths)
        used = [-(-max(n, 0) // page) for n in lengths]
        self.n_pages = sum(used) + extra
        order = torch.randperm(self.n_pages, generator=g).int()
        width = max(used + [1]) + 1
        self.table = torch.full((B, width + 3), 2 ** 30, dtype=torch.int32)     # entries that nobody may follow
        self.k64, self.v64 = [], []
        kv = torch.full((2, self.n_pages, hkv, page, D), float("nan"), dtype=torch.float64)
        at = 0
        for b, n in enumerate(lengths):
            mine = order[at:at + used[b]]
            at += used[b]
            self.table[b, :used[b]] = mine
            n = max(n, 0)
            x = torch.randn(2, n, hkv, D, generator=g, dtype=torch.float64) * \
                torch.exp(spread * torch.randn(2, n, hkv, 1, generator=g, dtype=torch.float64))
            x = x.to(bf16).double()
            t = torch.arange(n)
            kv[:, mine.long()[t // page], :, t % page] = x.permute(1, 0, 2, 3)
        self.q = (q_std * torch.randn(B, hq * D, generator=g)).to(bf16)
        nan_rows = kv.isnan()
        if e4m3:
            values, scales = quantized(torch.nan_to_num(kv))
            scales = torch.where(nan_rows[..., 0], math.nan, scales)
            codes = torch.where(nan_rows, math.nan, values / scales[..., None]).float().to(torch.float8_e4m3fn)
            z = [s.float().cuda() for s in scales]
            kv = values
        else:
            codes, z = kv.to(bf16), [None, None]
        t = [c.cuda() for c in codes]
        if layout == "rows first":
            t = [c.view(torch.uint8).transpose(1, 2).contiguous().view(c.dtype).transpose(1, 2) for c in
                 (x.contiguous() for x in t)]
            z = [s if s is None else s.transpose(1, 2).contiguous().transpose(1, 2) for s in z]
        self.cache = lm.KVCache(*t, *z)
        self.kv = kv
        self.width = width
        self.dev = self.q.cuda(), self.table.cuda()[:, :width], torch.tensor(lengths, dtype=torch.int32).cuda()

    def run(self, **kw):
        q, table, n = self.dev
        return lm.decode_attention(q, self.cache, table, n, want_lse=True, **kw)

    def check(self, out, lse, window=0, scale=None, softcap=0.0, only=None):
        D, n = self.D, self.hq // self.hkv
        scale = D ** -0.5 if scale is None else scale
        out, lse = out.cpu().double().reshape(-1, self.hkv, n, D), lse.cpu().double().reshape(-1, self.hkv, n)
        sq, sr = 0.0, 0.0
        for b, L in enumerate(self.lengths):
            if only is not None and b not in only:
                continue
            L = max(L, 0)
            t = torch.arange(max(0, L - window) if window else 0, L)
            pages = self.table[b].long()[t // self.page]
            for h in range(self.hkv):
                k, v = (self.kv[i, pages, h, t % self.page] for i in range(2))
                q = self.q[b].double().reshape(self.hkv, n, D)[h]
                o, z, p, s = attention(q, k, v, scale, softcap)
                if L == 0:
                    assert (out[b, h] == 0).all() and (lse[b, h] == -math.inf).all()
                    continue
                most = (q.abs() @ k.abs().t()).amax() * abs(scale)
                delta = D * 2.0 ** -23 * most + 2.0 ** -20 * (s.abs().amax() + softcap)
                join = (len(t) + 64) * 2.0 ** -23
                weight = 2.0 ** (-11 if self.e4m3 else -16)
                tol = (2 * (delta + 2.0 ** -21) + weight + join) * (p @ v.abs()) + BF * o.abs()
                err = (out[b, h] - o).abs()
                assert (err <= tol).all(), "sequence %d head %d: %.3g times the tolerance" % (b, h, (err / tol).max())
                zerr = (lse[b, h] - z).abs()
                assert (zerr <= delta + 2.0 ** -21 + join + 2.0 ** -22 * z.abs()).all(), (b, h, zerr.max())
                sq, sr = sq + float((out[b, h] - o).square().sum()), sr + float(o.square().sum())
        # all outputs together: errors of one rounding each, evenly spread over half a step at the most (BF / sqrt 3)
        if sr:
            assert math.sqrt(sq / sr) <= BF / math.sqrt(3.0) + 2.0 ** -12


HEADS = [(8, 8, 64), (32, 8, 128), (28, 4, 128), (24, 2, 128), (10, 2, 256), (71, 1, 64), (9, 3, 80), (33, 1, 96), (16, 1, 16),
         (48, 3, 256), (8, 1, 32)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,D", HEADS)
def test_heads(hq, hkv, D, e4m3):
    c = Case([37, 1, 130, 0, 64, 16], hq, hkv, D, e4m3=e4m3)
    c.check(*c.run())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page,layout", [(1, "heads first"), (3, "rows first"), (13, "heads first"), (16, "rows first"),
                                         (24, "rows first"), (128, "heads first"), (1000, "rows first")])
def test_pages(page, layout, e4m3):
    c = Case([1, 2, 15, 16, 17, 63, 64, 65, 300, 129], 8, 2, 128, page=page, layout=layout, e4m3=e4m3)
    c.check(*c.run())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lengths", [[3000], [1], [0], [0, 0, 0], [2500, 1, 0, 700, 64], [5] * 70, list(range(200)),
                                     [0] * 140 + [900] + [0] * 200 + [33],
                                     [i % 9 for i in range(2500)]], ids=lambda v: "%d of %d" % (len(v), max(v)))
def test_lengths(lengths, e4m3):
    c = Case(lengths, 8, 2, 64, e4m3=e4m3)
    c.check(*c.run())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 5000, 2 ** 31 - 1])
def test_window(window, e4m3):
    c = Case([200, 100, 99, 101, 1, 0, 777], 6, 2, 128, page=24, e4m3=e4m3)
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("scale,softcap", [(None, 30.0), (0.25, 0.0), (-0.5, 0.0), (1.0, 5.0), (0.0, 0.0)])
def test_scores(scale, softcap, e4m3):
    """Scores far apart (a scale of 1/4), equal ones (0), capped ones."""
    c = Case([150, 20, 64], 20, 2, 128, e4m3=e4m3)
    c.check(*c.run(scale=scale, softcap=softcap), scale=scale, softcap=softcap)


def test_value_scales_far_apart():
    """Value rows whose scales differ by 2^60, the large ones unlikely: numerators have a maximum of their own."""
    c = Case([90, 300], 8, 2, 128, e4m3=True, seed=5)
    big = torch.arange(c.n_pages * c.page).reshape(c.n_pages, 1, c.page) % 7 == 3
    f = torch.where(big, 2.0 ** 40, 2.0 ** -20).expand(c.n_pages, 2, c.page).double()
    c.cache.v_scales.mul_(f.cuda().float())
    c.kv[1] *= f[..., None]
    c.check(*c.run())


def test_large_queries_and_small():
    for std in (2.0 ** 100, 2.0 ** -100, 0.0):
        for e4m3 in (False, True):
            c = Case([40, 70], 8, 2, 64, e4m3=e4m3, q_std=std)
            s = 1.0 / std if std else 1.0
            c.check(*c.run(scale=s * 0.1), scale=s * 0.1)


def test_poison_stays_outside():
    """A page outside the cache or a table that is too short: NaN for that sequence; infinite and NaN rows: only where read."""
    for e4m3 in (False, True):
        c = Case([100, 50, 200, 30, 64], 8, 2, 128, e4m3=e4m3)
        q, table, n = c.dev
        table = table.clone()
        table[0, 3], table[2, 12] = c.n_pages, -1
        n = n.clone()
        n[3] = table.shape[1] * c.page + 1          # its row of the table is read to its end: pages that nobody has
        out, lse = lm.decode_attention(q, c.cache, table, n, want_lse=True)
        assert out[[0, 2, 3]].isnan().all() and lse[[0, 2, 3]].isnan().all()
        c.check(out, lse, only=(1, 4))
        n[3] = 2 ** 31 - 1
        n[1] = -5
        out, lse = lm.decode_attention(q, c.cache, table, n, want_lse=True)
        assert out[3].isnan().all() and (out[1] == 0).all() and (lse[1] == -math.inf).all()
        c.check(out, lse, only=(4,))
        table[0, 3], n[0] = c.table[0, 3].cuda(), 100
        c.cache.v[c.table[4, 1], 1, 5, 3] = float("inf") if not e4m3 else float("nan")   # e4m3 has no infinity
        out, _ = lm.decode_attention(q, c.cache, table, n, want_lse=True)
        hit = out[4].reshape(8, 128)[4:]
        assert not hit[:, 3].isfinite().any() and out[4, :4 * 128].isfinite().all()
        if not e4m3:
            assert hit[:, :3].isfinite().all() and hit[:, 4:].isfinite().all()
        assert not out[0].isnan().any()


def test_one_long_sequence():
    """Split over every CTA, with pages used again and again (a table may name a page twice)."""
    for e4m3 in (False, True):
        c = Case([4096], 8, 2, 128, page=64, e4m3=e4m3)
        c.lengths = [64 * 64 * 8]
        c.table = c.table[:, :64].repeat(1, 8)
        out, lse = lm.decode_attention(c.dev[0], c.cache, c.table.cuda(), torch.tensor(c.lengths, dtype=torch.int32).cuda(),
                                       want_lse=True)
        c.check(out, lse)


def test_rows_and_strides():
    """Queries and outputs as columns of wider rows; what lies beside them stays."""
    c = Case([33, 80, 7], 8, 2, 64)
    q, table, n = c.dev
    wide = torch.full((3, 1024), 7.0, dtype=bf16, device="cuda")
    wide[:, 128:128 + 512] = q
    out = torch.full((4, 640), 3.0, dtype=bf16, device="cuda")
    ref, lse = c.run()
    got = lm.decode_attention(wide[:, 128:640], c.cache, table, n, out=out[:3, 64:576])
    assert torch.equal(got, ref) and (out[3] == 3).all() and (out[:, :64] == 3).all() and (out[:, 576:] == 3).all()
    lm.decode_attention(wide[:, 128:640], c.cache, table, n, out=wide[:, 128:640])          # in the queries' place
    assert torch.equal(wide[:, 128:640], ref) and (wide[:, 640:] == 7).all()


def test_repeated_calls_and_streams():
    c = Case([2000, 64, 0, 1500, 3], 32, 8, 128, e4m3=True)
    first = c.run()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run()))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [c.run(stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(first, r))
    ws = torch.zeros(lm.decode_workspace_size(32, c.cache), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run(workspace=ws)))
    assert (ws[:lm.DECODE_COUNTER_BYTES] == 0).all()
    small = torch.zeros(lm.decode_workspace_size(32, c.cache) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(lm.LoraError, match="workspace"):
        c.run(workspace=small)


def test_graphs():
    """Two captured graphs and calls between their replays; lengths, pages and queries change under a graph."""
    c = Case([300, 0, 17, 900], 16, 2, 128)
    q, table, n = (t.clone() for t in c.dev)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lm.decode_attention(q, c.cache, table, n, want_lse=True))
        graphs.append(g)
    for lengths in ([300, 0, 17, 900], [1, 0, 16, 65], [0, 0, 0, 0], [257, 0, 3, 899]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        eager = lm.decode_attention(q, c.cache, table, n, want_lse=True)
        for g in graphs:
            g.replay()
        graphs[0].replay()
        again = lm.decode_attention(q, c.cache, table, n, want_lse=True)
        for o in outs + [again]:
            assert all(torch.equal(a, b) for a, b in zip(eager, o))
        c.lengths = lengths
        c.check(*eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(eager, o))


def test_a_cache_without_pages():
    """Sequences that claim rows of a cache that has none get NaN, those without rows zeros; nothing is read."""
    for dtype in (bf16, torch.float8_e4m3fn):
        cache = lm.kv_cache(0, 2, 16, 64, dtype)
        q = torch.ones(3, 256, dtype=bf16, device="cuda")
        n = torch.tensor([0, 5, 300], dtype=torch.int32).cuda()
        out, lse = lm.decode_attention(q, cache, torch.zeros(3, 20, dtype=torch.int32).cuda(), n, want_lse=True)
        assert (out[0] == 0).all() and out[1:].isnan().all() and lse[1:].isnan().all()
        slots = torch.tensor([0, -1, 7]).cuda()
        assert (lm.cache_read(cache, slots)[0] == 0).all()
        lm.cache_write(q[:, :128], q[:, :128], cache, slots)
