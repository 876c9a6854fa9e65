"""A preference fine-tuning step of one co-served decoder block, from the mixed batch to the updated adapter.

The block is small and its weights are random; its parts and their order are a served model's:

  forward     x -> x + LoRA projection (adapters, one mixed batch)            lm.forward
                -> + MLP with frozen 8-bit weights: gate|up, activation, down  lm.fp8_linear, lm.swiglu_forward
                -> logits of a frozen 8-bit head                               lm.fp8_linear
  loss        the policy is the fine-tuning segments (adapter 0); the reference is the base model: the same tokens
              once more in the same batch as segments without an adapter      lm.token_logprob, lm.preference_forward
  backward    logits -> head -> MLP (from the activation's 8-bit checkpoint) -> LoRA gradients -> AdamW
                                  lm.preference_backward, lm.fp8_linear, lm.swiglu_backward, lm.backward, lm.adamw_step

Decode tokens of other adapters ride along in every forward, as in serving.

    python examples/preference_finetune.py [steps]
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
    """Frozen weights of the block (8 bits, with the transposed ones that the backward multiplies by) and its pool."""

    def __init__(self, hidden, inner, vocab, ranks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(n, k):
            return torch.randn(n, k, device="cuda", generator=g) * k ** -0.5

        self.W = normal(hidden, hidden).bfloat16()
        self.gate_up = lm.fp8_quantize_weight(normal(2 * inner, hidden))
        self.down = lm.fp8_quantize_weight(normal(hidden, inner))
        self.head = lm.fp8_quantize_weight(normal(vocab, hidden))
        self.gate_up_t, self.down_t, self.head_t = (self.transposed(w) for w in (self.gate_up, self.down, self.head))
        self.embedding = torch.randn(vocab, hidden, device="cuda", generator=g).bfloat16()
        off = np.concatenate([[0], np.cumsum(ranks)[:-1]]).astype(np.int64) * hidden
        n = int(np.sum(ranks)) * hidden
        A = (torch.rand(n, device="cuda", generator=g) - 0.5).mul_(2 * hidden ** -0.5).bfloat16()
        B = torch.randn(n, device="cuda", generator=g).mul_(0.02).bfloat16()
        B[:int(ranks[0]) * hidden] = 0            # the adapter to be trained starts as the base model
        self.hidden, self.pool = hidden, lm.Pool(A, B, off, off, ranks, np.full(len(ranks), 2.0))

    @staticmethod
    def transposed(w):
        """A weight's codes and scales for the product with its transpose: the blocks are the transposed blocks."""
        codes, scales = w
        return codes.view(torch.uint8).t().contiguous().view(codes.dtype), scales.t().contiguous()

    def forward(self, tokens, segs):
        x = self.embedding[tokens]
        z = x + lm.forward(x, self.W, self.pool, segs)
        gu = lm.fp8_linear(z, *self.gate_up)
        (h, h_scales), saved = lm.swiglu_forward(gu, segs, checkpoint=True, fp8_out=True)
        out = z + lm.fp8_linear(h, *self.down, x_scales=h_scales)
        return x, saved, lm.fp8_linear(out, *self.head)

    def backward(self, x, saved, dlogits, segs, rows):
        """LoRA gradients (pool-shaped) from the logits' gradient of the fine-tuning rows."""
        dout = lm.fp8_linear(dlogits, *self.head_t)
        dh = lm.fp8_linear(dout, *self.down_t)
        dgu, scales = lm.swiglu_backward(saved, dh, fp8_out=True)
        dY = torch.zeros((x.shape[0], self.hidden), dtype=x.dtype, device=x.device)
        dY[rows] = dout + lm.fp8_linear(dgu, *self.gate_up_t, x_scales=scales)
        _, dA, dB = lm.backward(x, self.W, self.pool, segs, dY, want_dx=False, recompute=True)
        return dA, dB


def batch(n_pairs, vocab, seed=1):
    """Tokens, labels and tables: policy rows, the same rows as the base model's, then decode tokens."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(20, 90, (n_pairs, 2))
    pairs, t, prompt = [], 0, []
    for c, r in lens.tolist():
        pairs.append((t, c, t + c, r))
        t += c + r
    tokens = rng.integers(0, vocab, t)
    labels = rng.integers(0, vocab, t)
    for c0, cn, r0, rn in pairs:                 # both answers of a pair follow one prompt, which is not scored
        tokens[r0:r0 + 8] = tokens[c0:c0 + 8]
        prompt += list(range(c0, c0 + 8)) + list(range(r0, r0 + 8))
    labels[prompt] = -1
    segs = [(0, t, 0, 1), (t, t, -1, 0)]
    decode = rng.integers(0, vocab, 40)
    segs += [(2 * t + i, 1, 1 + i % 3, 0) for i in range(40)]
    to = torch.from_numpy
    return (to(np.concatenate([tokens, tokens, decode])).cuda(), to(labels).cuda(), np.asarray(pairs, np.int32),
            np.asarray(segs, np.int32), t)


def run(steps=8, hidden=512, inner=1408, vocab=2048, n_pairs=6, beta=0.5, lr=2e-3):
    """The mean loss of each step, the rewards of the last one, and the decode rows' logits of the first and last."""
    block = Block(hidden, inner, vocab, np.array([16, 8, 32, 64], np.int32))
    tokens, labels, pairs, segs, n = batch(n_pairs, vocab)
    A, B = block.pool.A, block.pool.B
    master = [A.float(), B.float()]
    moments = [torch.zeros_like(m) for m in master for _ in range(2)]
    losses, decode = [], []
    for step in range(steps):
        x, saved, logits = block.forward(tokens, segs)
        policy, base = logits[:n], logits[n:2 * n]
        ref, _ = lm.token_logprob(base, labels)
        f = lm.preference_forward(policy, labels, ref, pairs, beta)
        dlogits = lm.preference_backward(policy, labels, f.lse, f.coef, pairs, dlogits=policy)   # in their place
        dA, dB = block.backward(x, saved, dlogits, segs, slice(0, n))
        lm.adamw_step(block.pool, hidden, hidden, dA, dB, moments[0], moments[1], moments[2], moments[3], [0],
                      step=step + 1, lr=lr, A_master=master[0], B_master=master[1])
        losses.append(f.loss.mean())
        decode.append(logits[2 * n:])
    return torch.stack(losses).cpu().numpy(), f.rewards.cpu().numpy(), decode[0], decode[-1]


if __name__ == "__main__":
    lm.build()
    losses, rewards, _, _ = run(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
    for i, loss in enumerate(losses):
        print("step %d: loss %.4f" % (i, loss))
    print("reward margins after the last step but one:", np.round(rewards[:, 0] - rewards[:, 1], 2))
