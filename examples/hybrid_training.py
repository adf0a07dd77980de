"""Training steps of a small stack of Falcon and softmax-attention layers.

    python examples/hybrid_training.py

The library's operators come with their gradients as calls of their own; here
they are tied into torch's differentiation by two small functions: the chunked
Falcon forward with its backward, and the softmax-attention layer's norm, rotary
positions and attention with theirs, whose gradients of q, k and v land in one fused
gradient of the projection.  Weights and data are random; everything around the
operators is plain torch.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_delta_rule_gb300 as F  # noqa: E402

WIDTH, D, HEADS, KV_HEADS = 128, 64, 4, 2


class FalconChunks(torch.autograd.Function):
    @staticmethod
    def forward(ctx, p, q, k, v, beta, lam):
        ctx.p = p
        ctx.save_for_backward(q, k, v, beta, lam)
        return F.chunk_forward(p, q, k, v, beta, lam, want_carry=False)[0]

    @staticmethod
    def backward(ctx, dO):
        g = F.backward(ctx.p, *ctx.saved_tensors, dO.contiguous())
        return None, g["dq"], g["dk"], g["dv"], g["dbeta"], g["dlam"]


class SoftmaxAttention(torch.autograd.Function):
    """From a fused projection x [tokens, HEADS + 2 KV_HEADS, D] and the norm weights to o [tokens, HEADS, D]."""

    COUNTS = [HEADS, KV_HEADS, KV_HEADS]

    @staticmethod
    def forward(ctx, x, w_q, w_k, positions, table, cu, longest):
        q, k, v = torch.split(x, SoftmaxAttention.COUNTS, 1)
        q, k = F.qk_norm_rope(q, k, positions, table, w_q, w_k)
        o, lse = F.attn_prompt(q, k, v, cu, max_q=longest, want_lse=True)
        ctx.longest = longest
        ctx.save_for_backward(x, w_q, w_k, positions, table, cu, q, k, o, lse)
        return o

    @staticmethod
    def backward(ctx, dO):
        x, w_q, w_k, positions, table, cu, qr, kr, o, lse = ctx.saved_tensors
        q, k, v = torch.split(x, SoftmaxAttention.COUNTS, 1)
        dx = torch.zeros_like(x)
        dq, dk, dv = torch.split(dx, SoftmaxAttention.COUNTS, 1)
        g = F.attn_prompt_backward(qr, kr, v, o, lse, dO.contiguous(), cu, max_q=ctx.longest, out={"dv": dv})
        h = F.qk_norm_rope_backward(q, k, g["dq"], g["dk"], positions, table, w_q, w_k, out={"dq": dq, "dk": dk})
        return dx, h["dw_q"], h["dw_k"], None, None, None, None


class Stack(torch.nn.Module):
    def __init__(self, seed: int, max_len: int, dtype):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        weight = lambda r, c: torch.nn.Parameter((torch.randn((r, c), generator=g) * r ** -0.5).to(dtype).cuda())  # noqa: E731
        self.falcon_in, self.falcon_out = weight(WIDTH, 3 * HEADS * D + 2 * HEADS), weight(HEADS * D, WIDTH)
        self.attn_in, self.attn_out = weight(WIDTH, (HEADS + 2 * KV_HEADS) * D), weight(HEADS * D, WIDTH)
        self.w_q, self.w_k = (torch.nn.Parameter(torch.ones(D, device="cuda")) for _ in range(2))
        self.table = F.rope_table(F.rope_frequencies(D)[0], max_len)
        self.dtype = F.FALCON_BF16 if dtype == torch.bfloat16 else F.FALCON_F32

    @staticmethod
    def _norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def forward(self, x):
        """x [B, T, WIDTH] -> [B, T, WIDTH]"""
        B, T, _ = x.shape
        q, k, v, beta, lam = torch.split(self._norm(x) @ self.falcon_in, [HEADS * D] * 3 + [HEADS] * 2, dim=2)
        rows = lambda t: t.reshape(B, T, HEADS, D)  # noqa: E731
        unit = lambda t: torch.nn.functional.normalize(rows(t).float(), dim=-1).to(t.dtype)  # noqa: E731
        p = F.Params(B=B, T=T, H=HEADS, dk=D, dv=D, dtype=self.dtype)
        o = FalconChunks.apply(p, unit(q), unit(k), rows(v).contiguous(), torch.sigmoid(beta.float()),
                               torch.sigmoid(lam.float() - 3.0))
        x = x + o.reshape(B, T, -1) @ self.falcon_out
        y = (self._norm(x) @ self.attn_in).reshape(B * T, HEADS + 2 * KV_HEADS, D)
        cu = torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
        pos = torch.arange(T, device="cuda").repeat(B)
        o = SoftmaxAttention.apply(y, self.w_q, self.w_k, pos, self.table, cu, T)
        return x + o.reshape(B, T, -1) @ self.attn_out


def loss_of(stack, x, target):
    return (stack(x).float() - target.float()).square().mean()


def main(B=3, T=100, steps=5, dtype=torch.bfloat16, seed=0) -> list[float]:
    """The loss before each step."""
    g = torch.Generator().manual_seed(seed + 1)
    x, target = (torch.randn((B, T, WIDTH), generator=g).to(dtype).cuda() for _ in range(2))
    stack = Stack(seed, T, dtype)
    opt = torch.optim.SGD(stack.parameters(), lr=0.5)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = loss_of(stack, x, target)
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    print("loss:", ", ".join(f"{v:.4f}" for v in main()))
