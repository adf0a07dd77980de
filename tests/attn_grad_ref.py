"""Dense fp64 reference of the softmax-attention gradient for the tests, with
the sums of absolute values that bound a kernel's rounding errors."""

from __future__ import annotations

import math

import torch


def attention_grad(q, k, v, cu_q, cu_k, scale, d_o, dlse=None, max_q=None):
    """Whole softmax matrices, a sequence and head at a time, of q, d_o [n, Hq, d], k, v [m, Hkv, d] (any dtype and
    device), cu_q and cu_k lists.

    Returns o, lse, the gradients {dq, dk, dv} and for each of them the sum A of the absolute values of what an
    element is a sum of: with W = P (|dO| |V|^T + sum_j P (|dO| |V|^T)), a bound of |dS| and of what D contributes,
      A_dv = P^T |dO|,  A_dk = scale W^T |Q|,  A_dq = scale W |K|.
    An error of relative size e in every P, dP and D is an error of at most e A in the gradients."""
    q, k, v, d_o = (x.double() for x in (q, k, v, d_o))
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    o, lse = torch.zeros_like(q), torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    g = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    A = {name: torch.zeros_like(x) for name, x in g.items()}
    for a, b, i, j in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        lq, lk = b - a, j - i
        rows = lq if max_q is None else min(lq, max_q)
        if rows == 0 or lk == 0:
            continue
        seen = torch.ones((lq, lk), dtype=torch.bool, device=q.device).tril(lk - lq)[:rows]
        r = slice(a, a + rows)
        for h in range(Hq):
            c = h // (Hq // Hkv)
            Q, K, V, G = q[r, h], k[i:j, c], v[i:j, c], d_o[r, h]
            s = (scale * (Q @ K.T)).masked_fill(~seen, -math.inf)
            lse[r, h] = torch.logsumexp(s, 1)
            some = seen.any(1, keepdim=True)
            P = torch.where(some, torch.exp(s - torch.where(some, lse[r, h, None], 0.0)), 0.0)
            o[r, h] = P @ V
            dP = G @ V.T
            e = 0.0 if dlse is None else dlse[r, h, None].double()
            dS = P * (dP - (P * dP).sum(1, keepdim=True) + e)
            g["dv"][i:j, c] += P.T @ G
            g["dq"][r, h] = scale * (dS @ K)
            g["dk"][i:j, c] += scale * (dS.T @ Q)
            aP = G.abs() @ V.abs().T
            W = P * (aP + (P * aP).sum(1, keepdim=True) + (0.0 if dlse is None else e.abs()))
            A["dv"][i:j, c] += P.T @ G.abs()
            A["dq"][r, h] = scale * (W @ K.abs())
            A["dk"][i:j, c] += scale * (W.T @ Q.abs())
    return o, lse, g, A
