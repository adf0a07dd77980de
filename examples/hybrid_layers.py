"""A small stack of Falcon and softmax-attention layers, served: prompts of
different lengths in one packed call, then one token per sequence and step.

    python examples/hybrid_layers.py

Falcon layers keep a fixed-size state per sequence (packed chunk forward, then
recurrent steps); softmax-attention layers keep keys and values in a paged cache
held in 8 bits (norm and rotary positions, prompt attention, append, decode
attention).  The run compares every stepped token with a prompt call over the
whole sequences.  Weights are random; projections are plain matrix products.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_delta_rule_gb300 as F  # noqa: E402

WIDTH, D, HEADS, KV_HEADS, PAGE = 256, 64, 4, 2, 16
PROLOGUE = F.FALCON_PROLOGUE_L2NORM_QK | F.FALCON_PROLOGUE_GATE_LOGITS


def _weight(g, rows, cols):
    return (torch.randn((rows, cols), generator=g) * rows ** -0.5).bfloat16().cuda()


class FalconLayer:
    def __init__(self, g):
        self.w_in, self.w_out = _weight(g, WIDTH, 3 * HEADS * D + 2 * HEADS), _weight(g, HEADS * D, WIDTH)

    def _inputs(self, x):
        q, k, v, beta, lam = torch.split(x @ self.w_in, [HEADS * D] * 3 + [HEADS] * 2, dim=1)
        rows = [t.reshape(-1, HEADS, D).contiguous() for t in (q, k, v)]
        return rows + [beta.float().contiguous(), (lam.float() - 3.0).contiguous()]

    def _params(self, B, T):
        return F.Params(B=B, T=T, H=HEADS, dk=D, dv=D, variant=F.FALCON_1, prologue=PROLOGUE)

    def prompt(self, x, cu, longest):
        p = self._params(cu.numel() - 1, longest)
        o, self.carry = F.chunk_forward_varlen(p, cu, *self._inputs(x))
        return o.reshape(x.shape[0], -1) @ self.w_out

    def step(self, x):
        B = x.shape[0]
        q, k, v, beta, lam = (t.unsqueeze(1) for t in self._inputs(x))
        o = torch.empty_like(v)
        F.falcon_recurrent_step(self._params(B, 1), q, k, v, beta, lam, self.carry, o)
        return o.reshape(B, -1) @ self.w_out


class AttentionLayer:
    """Keys and values of every sequence live in pages of one cache; pages are dealt out in advance here."""

    def __init__(self, g, max_len, sequences):
        self.w_in = _weight(g, WIDTH, (HEADS + 2 * KV_HEADS) * D)
        self.w_out = _weight(g, HEADS * D, WIDTH)
        self.w_q, self.w_k = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        self.max_len, cols = max_len, -(-max_len // PAGE)
        freq, mscale = F.rope_frequencies(D, scaling="yarn", factor=4.0, original_len=64)
        self.table = F.rope_table(freq, max_len, mscale)
        order = torch.randperm(sequences * cols, generator=g).int().cuda()
        self.pages = order.reshape(sequences, cols)
        self.cache = F.empty_kv_cache(sequences * cols, KV_HEADS, PAGE, D)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def _inputs(self, x):
        """Slices of one projection: the operators take them as they are."""
        y = (x @ self.w_in).reshape(x.shape[0], HEADS + 2 * KV_HEADS, D)
        return torch.split(y, [HEADS, KV_HEADS, KV_HEADS], dim=1)

    def prompt(self, x, cu, longest):
        q, k, v = self._inputs(x)
        n = cu.diff()
        pos = torch.arange(x.shape[0], device="cuda") - torch.repeat_interleave(cu[:-1].long(), n)
        q, k = F.qk_norm_rope(q, k, pos, self.table, self.w_q, self.w_k)
        o = F.attn_prompt(q, k, v, cu, max_q=longest)
        F.kv_append(self.cache, k, v, cu, self.lens, self.pages, longest)
        self.lens += n.int()
        return o.reshape(x.shape[0], -1) @ self.w_out

    def step(self, x):
        q, k, v = self._inputs(x)
        q, _ = F.qk_norm_rope(q, None, self.lens.long(), self.table, self.w_q)
        cu = torch.arange(x.shape[0] + 1, dtype=torch.int32, device="cuda")
        F.kv_append(self.cache, k, v, cu, self.lens, self.pages, 1, self.table, self.w_k, norm=True)
        self.lens += 1
        o = F.attn_decode(q, self.cache, self.pages, self.lens, self.max_len)
        return o.reshape(x.shape[0], -1) @ self.w_out


class Stack:
    def __init__(self, seed, max_len, sequences):
        g = torch.Generator().manual_seed(seed)
        self.layers = [FalconLayer(g), AttentionLayer(g, max_len, sequences), FalconLayer(g),
                       AttentionLayer(g, max_len, sequences)]

    @staticmethod
    def _norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def prompt(self, x, cu, longest):
        for layer in self.layers:
            x = x + layer.prompt(self._norm(x), cu, longest)
        return x

    def step(self, x):
        for layer in self.layers:
            x = x + layer.step(self._norm(x))
        return x


def main(lengths=(70, 1, 33), steps=20, seed=0) -> float:
    """Relative error of the stepped tokens against one prompt call over everything."""
    total = [n + steps for n in lengths]
    g = torch.Generator().manual_seed(seed + 1)
    tokens = [torch.randn((n, WIDTH), generator=g).bfloat16().cuda() for n in total]
    cu = lambda ns: torch.tensor([0] + list(torch.tensor(ns).cumsum(0)), dtype=torch.int32).cuda()  # noqa: E731
    want = torch.split(Stack(seed, max(total), len(lengths)).prompt(torch.cat(tokens), cu(total), max(total)), total)
    stack = Stack(seed, max(total), len(lengths))
    first = stack.prompt(torch.cat([t[:n] for t, n in zip(tokens, lengths)]), cu(lengths), max(lengths))
    got = [[x] for x in torch.split(first, list(lengths))]
    for i in range(steps):
        y = stack.step(torch.stack([t[n + i] for t, n in zip(tokens, lengths)]))
        for b in range(len(lengths)):
            got[b].append(y[b:b + 1])
    a, b = torch.cat([torch.cat(x) for x in got]).float(), torch.cat(want).float()
    return ((a - b).square().mean() / b.square().mean()).sqrt().item()


if __name__ == "__main__":
    print(f"{len(Stack(0, 8, 1).layers)} layers, prompts of 70, 1 and 33 tokens, 20 steps: "
          f"relative error against one prompt call {main():.4f}")
