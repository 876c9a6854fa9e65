"""Decode attention called as its documentation allows and as few programs do; against float64, or bit by bit against the same
call in its usual form.  Tolerances: test_gpu_decode.py's."""
import threading

import pytest
import torch

import lora_co_serving_gb300 as lm
from attention_oracle import attention
from test_gpu_decode import Case

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16

# sequences that several CTAs share: joined in one stage; in two; a group of 71 heads, taken in five parts
SPLIT = [([600, 3, 900, 0, 2000], 8, 2, 128), ([20000], 8, 2, 128), ([9000, 1], 71, 1, 64), ([12000], 10, 2, 256),
         ([5000, 800], 32, 2, 128)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lengths,hq,hkv,D", SPLIT)
def test_in_place_over_several_ctas(lengths, hq, hkv, D, e4m3):
    """The result in the queries' own rows, where other CTAs still read the queries of the same and of other heads."""
    c = Case(lengths, hq, hkv, D, page=64, e4m3=e4m3)
    q, table, n = c.dev
    ref, lse = c.run()
    c.check(ref, lse)
    wide = torch.full((len(lengths), hq * D + 64), 5.0, dtype=bf16, device="cuda")
    for _ in range(3):
        wide[:, :hq * D] = q
        got, z = lm.decode_attention(wide[:, :hq * D], c.cache, table, n, want_lse=True, out=wide[:, :hq * D])
        assert torch.equal(got, ref) and torch.equal(z, lse) and (wide[:, hq * D:] == 5).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 64), (16, 1, 128), (20, 2, 256), (71, 1, 64)])
def test_probabilities_lose_none_of_the_outputs_digits(hq, hkv, D, e4m3):
    """Few tokens and small scores, where the sums' bound is far below what one number of 11 bits would cost a probability:
    outputs are the nearest bf16 numbers but for that bound.

    A probability is two numbers of 16 bits: bf16 leaves half a step of half a step, 2^-16 of it, fp16 2^-22.  The products
    and their sums as in test_gpu_decode.py; half a step of the output is taken at the output's own power of two."""
    lengths = [2 + i % 7 for i in range(48)]
    c = Case(lengths, hq, hkv, D, e4m3=e4m3, q_std=0.05, seed=11)
    out, lse = c.run()
    c.check(out, lse)
    n = hq // hkv
    out = out.cpu().double().reshape(-1, hkv, n, D)
    for b, L in enumerate(lengths):
        t = torch.arange(L)
        pages = c.table[b].long()[t // c.page]
        for h in range(hkv):
            k, v = (c.kv[i, pages, h, t % c.page] for i in range(2))
            q = c.q[b].double().reshape(hkv, n, D)[h]
            o, _, p, s = attention(q, k, v, D ** -0.5)
            most = (q.abs() @ k.abs().t()).amax() * D ** -0.5
            delta = D * 2.0 ** -23 * most + 2.0 ** -20 * s.abs().amax()
            bound = (2 * (delta + 2.0 ** -21) + 2.0 ** (-22 if e4m3 else -16) + (L + 64) * 2.0 ** -23) * (p @ v.abs())
            half = torch.exp2(torch.floor(torch.log2(o.abs() + bound)) - 8.0)
            err = (out[b, h] - o).abs()
            assert (err <= half + bound).all(), "sequence %d head %d: %.3g of the bound" % (b, h, ((err - half) / bound).max())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("power", [84, -84])
def test_large_and_small_values(power, e4m3):
    """Value rows near 2^84 (elements below 2^88) and 2^-84.  In 16 bits a power of two changes no digit of the result; in 8 it
    goes into the exponent that a numerator is formed from."""
    c = Case([700, 1, 33], 8, 2, 64, e4m3=e4m3, spread=0.2)
    assert c.kv[1].nan_to_num().abs().max() < 16
    ref, lse = c.run()
    if e4m3:
        c.cache.v_scales.mul_(2.0 ** power)
    else:
        c.cache.v.copy_((c.cache.v.double() * 2.0 ** power).to(bf16))
    c.kv[1] *= 2.0 ** power
    out, again = c.run()
    c.check(out, again)
    if not e4m3:
        assert torch.equal(out.double(), ref.double() * 2.0 ** power) and torch.equal(again, lse)


def test_threads_of_their_own():
    """A thread that decodes few rows beside one with a long batch and its gradient, each on its own stream: what they give
    alone, call after call."""
    g = torch.Generator().manual_seed(5)
    turns, w = lm.rotary_turns(64), torch.ones(64, device="cuda", dtype=bf16)
    c = Case([300, 0, 900, 17, 64, 5, 1200], 8, 2, 64, page=64, e4m3=True)
    q, table, n = c.dev

    def serve(x, p):
        y = lm.rotary_forward(x, p, turns, 8, 2, q_weight=w, k_weight=w)
        return (y, *lm.rotary_backward(x, p, turns, 8, 2, y, q_weight=w, k_weight=w, weight_grads=True),
                *lm.decode_attention(q, c.cache, table, n, want_lse=True))

    batches = [(torch.randn(T, 640, generator=g).to(bf16).cuda(), torch.arange(T).cuda()) for T in (5000, 7, 3000, 6)]
    alone = [serve(*b) for b in batches]
    torch.cuda.synchronize()
    errors = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(150):
                    got = serve(*batches[i])
                    if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                        errors.append("batch %d differs" % i)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:3]
