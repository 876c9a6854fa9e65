"""Decoding with one adapter a sequence: tokens of one decoder block, generated from a paged key-value cache.

The block is small and its weights are random; its parts and their order are a served model's:

  q|k|v       LoRA projection of the whole batch, a segment for each sequence      lm.sliced_forward
  attention   queries and keys normalised and turned by their positions, keys and
              values into the cache (16 or 8 bits), then the new token's attention lm.rotary_forward, lm.decode_attention
  output      LoRA projection, MLP and head with frozen 8-bit weights              lm.forward, lm.fp8_linear,
                                                                                   lm.swiglu_forward

A prompt is fed token by token.  A step's positions, slots and lengths are tensors on the device, so the step is captured
into a CUDA graph once and replayed for every token; a sequence that has come to its end drops out with a length of zero.

    python examples/decode_loop.py [tokens]
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import lora_co_serving_gb300 as lm  # noqa: E402


class Block:
    def __init__(self, hidden, heads, kv_heads, head_dim, inner, vocab, ranks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(n, k):
            return torch.randn(n, k, device="cuda", generator=g) * k ** -0.5

        def pool(out, slices):
            """Factors of every adapter: A [slices * r, hidden in], B [r, out]."""
            k = hidden if slices > 1 else heads * head_dim
            a_off = np.concatenate([[0], np.cumsum(ranks)[:-1]]).astype(np.int64) * k * slices
            b_off = np.concatenate([[0], np.cumsum(ranks)[:-1]]).astype(np.int64) * out
            n = int(np.sum(ranks))
            A = (torch.rand(n * k * slices, device="cuda", generator=g) - 0.5).mul_(2 * k ** -0.5).bfloat16()
            B = torch.randn(n * out, device="cuda", generator=g).mul_(0.1).bfloat16()
            return lm.Pool(A, B, a_off, b_off, ranks, np.full(len(ranks), 2.0))

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        q, kv = heads * head_dim, kv_heads * head_dim
        self.bounds = [0, q, q + kv, q + 2 * kv]
        self.qkv = normal(q + 2 * kv, hidden).bfloat16()
        self.out = normal(hidden, q).bfloat16()
        self.qkv_pool, self.out_pool = pool(q + 2 * kv, 3), pool(hidden, 1)
        self.gate_up = lm.fp8_quantize_weight(normal(2 * inner, hidden))
        self.down = lm.fp8_quantize_weight(normal(hidden, inner))
        self.head = lm.fp8_quantize_weight(normal(vocab, hidden))
        self.embedding = torch.randn(vocab, hidden, device="cuda", generator=g).bfloat16()
        self.q_norm, self.k_norm = (1.0 + 0.1 * torch.randn(2, head_dim, device="cuda", generator=g)).bfloat16()
        self.turns = lm.rotary_turns(head_dim)

    def step(self, tokens, segs, positions, slots, cache, table, lengths):
        """Logits of the next token of each sequence; the new rows are added to the cache."""
        x = self.embedding[tokens]
        qkv = lm.sliced_forward(x, self.qkv, self.qkv_pool, self.bounds, segs)
        n = self.bounds[2]
        q = lm.rotary_forward(qkv[:, :n], positions, self.turns, self.heads, self.kv_heads, q_weight=self.q_norm,
                              k_weight=self.k_norm, v=qkv[:, n:], cache=cache, slots=slots)
        attended = lm.decode_attention(q, cache, table, lengths)
        x = x + lm.forward(attended, self.out, self.out_pool, segs)
        h, h_scales = lm.swiglu_forward(lm.fp8_linear(x, *self.gate_up), fp8_out=True)
        x = x + lm.fp8_linear(h, *self.down, x_scales=h_scales)
        return lm.fp8_linear(x, *self.head)


def run(n_tokens=24, n_seqs=5, page=16, e4m3=False, capture=True, hidden=256, heads=8, kv_heads=4, head_dim=64, inner=512,
        vocab=512):
    """(tokens [n_seqs, n_tokens], logits of the last step, the cache, its page table, lengths) on the host or device."""
    ranks = np.array([8, 16, 32], np.int32)
    block = Block(hidden, heads, kv_heads, head_dim, inner, vocab, ranks)
    rng = np.random.default_rng(1)
    prompt = torch.from_numpy(rng.integers(0, vocab, (n_seqs, 6))).cuda()
    segs = [(i, 1, i % 4 - 1, 0) for i in range(n_seqs)]                      # adapter -1: the base model
    stop = torch.from_numpy(rng.integers(n_tokens // 2, n_tokens + 1, n_seqs)).cuda()
    stop[0] = n_tokens
    pages = -(-n_tokens // page)
    cache = lm.kv_cache(n_seqs * pages + 1, kv_heads, page, head_dim, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    table = torch.from_numpy(rng.permutation(n_seqs * pages).astype(np.int32).reshape(n_seqs, pages)).cuda()
    token = prompt[:, 0].clone()
    at = torch.zeros(n_seqs, dtype=torch.int64, device="cuda")                # position of each sequence's new token

    def step():
        alive = at < stop
        slots = torch.where(alive, table.gather(1, (at // page).clamp(max=pages - 1)[:, None])[:, 0].long() * page + at % page,
                            -1)
        lengths = torch.where(alive, at + 1, 0).int()
        return block.step(token, segs, at, slots, cache, table, lengths)

    graph = None
    if capture:
        for _ in range(2):
            step()                               # what is made on first use; the graph's first replay writes the rows again
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logits = step()
    tokens = [token.clone()]
    for t in range(n_tokens):
        if graph is None:
            logits = step()
        else:
            graph.replay()
        last = logits.clone()
        token.copy_(prompt[:, t + 1] if t + 1 < prompt.shape[1] else logits.argmax(1))
        at += 1
        tokens.append(token.clone())
    lengths = torch.minimum(at, stop)
    return torch.stack(tokens[:-1], 1), last, cache, table, lengths


if __name__ == "__main__":
    lm.build()
    tokens, _, _, _, lengths = run(int(sys.argv[1]) if len(sys.argv) > 1 else 24)
    for i, (row, n) in enumerate(zip(tokens.tolist(), lengths.tolist())):
        print("sequence %d, adapter %d:" % (i, i % 4 - 1), row[:n])
