"""Gradients of the softmax-attention operators on the GPU against fp64.

Tolerances follow from the number formats, u = half a step: 2^-8 for bf16.  A is
the sum of the absolute values of what an element of a gradient is the sum of
(tests/attn_grad_ref.py).  bf16: the weights P are rounded once (u), dS once (u),
o, which D is formed from, was rounded by the forward (u), the result is
rounded once (u of itself): at most 3 u A + u |x|.  fp32: operands, P and dS keep 22 bits (down to 2^-40 of
their row's largest); scores and dP are sums of up to 128 products, each off by up to 2^-22 of the sum of absolute values; the
scores' enter P through the exponential, times the largest sum of absolute values
of a score, S: at most 2^-22 (2 S + 8) A for all of it, and 2^-21 A for the
gradients' own sums over a tile and 2^-24 a tile after that.  Over a whole tensor roundings do
not line up: the norm of the error is below u (bf16; u / sqrt(3) each, less where
many terms add up) or 1e-5 (fp32) times 2 of the norm.
"""

from __future__ import annotations

import math
import time

import numpy as np
import pytest
import torch

from attn_grad_ref import attention_grad
from oracle import softmax_attention as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def F():
    import chunked_delta_rule_gb300 as F
    return F


def _np(x):
    return x.detach().cpu().double().numpy()


def _cu(lens):
    return [0] + list(np.cumsum(lens))


def _dev(cu):
    return torch.tensor([int(x) for x in cu], dtype=torch.int32, device="cuda")


def _rand(shape, dtype, seed, unit=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if unit:  # as the norm leaves the rows
        x = x / x.square().mean(-1, keepdim=True).sqrt()
    return x.to(DT[dtype]).cuda()


def _inputs(lq, lk, Hq, Hkv, d, dtype, seed=0, behind=0):
    n, m = sum(lq) + behind, sum(lk) + behind
    return (_rand((n, Hq, d), dtype, seed, True), _rand((m, Hkv, d), dtype, seed + 1, True),
            _rand((m, Hkv, d), dtype, seed + 2), _rand((n, Hq, d), dtype, seed + 3))


def _check(got, want, A, dtype, S):
    for name in want:
        x, y = got[name].double(), want[name]
        if dtype == "bf16":
            tol = 3 * U * A[name] + U * y.abs() + 1e-30
        else:
            tol = (2.0 ** -22 * (2 * S + 8) + 2.0 ** -20) * A[name] + 1e-30
        assert torch.isfinite(x).all(), name
        worst = ((x - y).abs() / tol).max().item() if x.numel() else 0.0
        assert worst <= 1.0, (name, worst)
        if x.numel() >= 4096 and y.norm() > 0.05 * A[name].norm():
            assert (x - y).norm() <= 2 * (U if dtype == "bf16" else 1e-5) * y.norm(), name


def _forward(F, q, k, v, cu_q, cu_k, max_q, scale=0.0):
    return F.attn_prompt(q, k, v, cu_q, cu_k, max_q, scale, want_lse=True)


def _S(q, k, scale):
    """Bound of the sum of absolute values of a score."""
    return scale * q.double().norm(dim=-1).max().item() * k.double().norm(dim=-1).max().item() if k.numel() and q.numel() else 0.0


SHAPES = [
    # lq, lk, Hq, Hkv, d
    ([1], [1], 1, 1, 16), ([2], [2], 2, 1, 32), ([1, 1, 1], [5, 130, 1], 4, 2, 64), ([17], [17], 3, 3, 128),
    ([63, 64, 65], [63, 64, 65], 4, 2, 64), ([127, 128, 129, 1], [127, 128, 129, 1], 2, 2, 128),
    ([300], [300], 8, 1, 32), ([130, 7], [400, 260], 6, 2, 64), ([200, 3], [40, 1], 4, 4, 64),
    ([0, 33, 0], [5, 33, 0], 2, 1, 64), ([20, 40], [0, 40], 2, 2, 128), ([257, 385], [257, 513], 4, 1, 128),
    ([5, 300, 90], [5, 300, 90], 12, 4, 16), ([511], [640], 2, 2, 64), ([900, 1, 340], [900, 70, 340], 3, 1, 64),
    ([140] * 5, [140] * 5, 2, 1, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,d", SHAPES)
def test_gradients(F, dtype, lq, lk, Hq, Hkv, d):
    q, k, v, dO = _inputs(lq, lk, Hq, Hkv, d, dtype, sum(lq) + d)
    dlse = _rand(q.shape[:2], "f32", 9) if sum(lq) % 2 else None
    cu_q, cu_k = _cu(lq), _cu(lk)
    o, lse = _forward(F, q, k, v, _dev(cu_q), _dev(cu_k), max(lq))
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu_q), _dev(cu_k), max(lq), dlse=dlse)
    _, _, want, A = attention_grad(q, k, v, cu_q, cu_k, d ** -0.5, dO, dlse)
    _check(got, want, A, dtype, _S(q, k, d ** -0.5))


@pytest.mark.parametrize("dtype,lq,lk,Hq,Hkv,d", [
    ("bf16", [2048, 1000], [2048, 1000], 2, 1, 64), ("bf16", [1500], [1500], 4, 2, 128),
    ("bf16", [1100], [1700], 2, 2, 32), ("bf16", [3000], [3000], 2, 1, 16), ("f32", [1500, 3], [1500, 3], 2, 1, 64),
    ("f32", [1025], [1030], 2, 2, 128), ("bf16", [128] * 40, [128] * 40, 2, 2, 64), ("bf16", [4, 2100], [800, 2100], 2, 2, 128),
])
def test_gradients_of_long_sequences(F, dtype, lq, lk, Hq, Hkv, d):
    q, k, v, dO = _inputs(lq, lk, Hq, Hkv, d, dtype, 77)
    cu_q, cu_k = _cu(lq), _cu(lk)
    o, lse = _forward(F, q, k, v, _dev(cu_q), _dev(cu_k), max(lq))
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu_q), _dev(cu_k), max(lq))
    _, _, want, A = attention_grad(q, k, v, cu_q, cu_k, d ** -0.5, dO)
    _check(got, want, A, dtype, _S(q, k, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,size", [(0.5, 4.0), (1e-3, 1.0)])
def test_large_and_small_scores(F, dtype, scale, size):
    """Scores of some hundreds (weights all but one-hot) and scores near zero (weights all but equal)."""
    q, k, v, dO = _inputs([200], [200], 2, 2, 64, dtype, 5)
    q, k = q * size, k * size
    cu = _cu([200])
    o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), 200, scale)
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), None, 200, scale)
    # fp32: the forward's log sum is itself off by 2^-24 of its size
    _, _, want, A = attention_grad(q, k, v, cu, cu, scale, dO)
    _check(got, want, A, dtype, _S(q, k, scale))


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("bf16", 64, 2, 1), ("bf16", 128, 2, 2), ("bf16", 16, 16, 1), ("bf16", 128, 16, 1),
                                            ("f32", 64, 2, 1)])
@pytest.mark.parametrize("power", [-126, -113, -101, -100, -99, -60, 100])
def test_scales_at_the_ends_of_the_range(F, dtype, d, Hq, Hkv, power):
    """Scales down to fp32's smallest normal number, with queries and keys whose scores are of ordinary size all the same:
    rows past the end of a sequence (the next one's) have no weight at any scale."""
    scale = 2.0 ** power
    lens = [1, 3, 2, 40]
    q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, 21)
    q, k = q * 2.0 ** (-power // 2 - 2), k * 2.0 ** (-power - -power // 2 - 3)
    cu = _cu(lens)
    o, lse, want, A = attention_grad(q, k, v, cu, cu, scale, dO)
    got = F.attn_prompt_backward(q, k, v, o.to(q.dtype), lse.float(), dO, _dev(cu), None, 40, scale)
    # the sizes of dq and dk back to those of ordinary scores
    for name, f in (("dq", 2.0 ** (-power // 2 - 2)), ("dk", 2.0 ** (-power - -power // 2 - 3))):
        got[name], want[name], A[name] = got[name].double() * f, want[name] * f, A[name] * f
    _check(got, want, A, dtype, _S(q, k, scale))


def test_bits_do_not_change(F):
    """The same call twice, on another stream, and its halves alone."""
    for dtype, d in (("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)):
        lens = [700, 333, 128]
        q, k, v, dO = _inputs(lens, lens, 8, 2, d, dtype, 3)
        cu = _dev(_cu(lens))
        o, lse = _forward(F, q, k, v, cu, cu, 700)
        a = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=700)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=700, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        c = F.attn_prompt_backward(q, k, v, o, lse, dO, cu)  # the loose bound of all tokens
        p = F.AttnParams(B=3, Hq=8, Hkv=2, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=700,
                         tokens=sum(lens), k_tokens=sum(lens))
        ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
        half = {n: torch.empty_like(x) for n, x in a.items()}
        F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, {"dq": half["dq"]}, ws)
        F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, {n: half[n] for n in ("dk", "dv")}, ws)
        for n in a:
            for other in (b, c, half):
                assert torch.equal(a[n], other[n]), (dtype, d, n)


def test_slices_of_fused_projections_and_gaps(F):
    """q, k, v slices of one projection, dq, dk, dv slices of one gradient; o and dO with gaps; nothing else written."""
    lens, Hq, Hkv, d = [150, 40, 260], 6, 2, 64
    n = sum(lens)
    for dtype in ("bf16", "f32"):
        x = _rand((n, Hq + 2 * Hkv, d), dtype, 1)
        q, k, v = torch.split(x, [Hq, Hkv, Hkv], 1)
        cu = _cu(lens)
        o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), 260)
        wide = torch.full((n, Hq + 3, d), 7.0, dtype=DT[dtype], device="cuda")
        wide[:, 1:1 + Hq] = o
        dwide = _rand((n, Hq + 1, d), dtype, 2)
        dO = dwide[:, 1:]
        grad = torch.full((n + 4, Hq + 2 * Hkv + 1, d), 5.0, dtype=DT[dtype], device="cuda")
        out = dict(zip(("dq", "dk", "dv"), torch.split(grad[2:-2, :-1], [Hq, Hkv, Hkv], 1)))
        got = F.attn_prompt_backward(q, k, v, wide[:, 1:1 + Hq], lse, dO, _dev(cu), max_q=260, out=out)
        assert got["dq"].data_ptr() == out["dq"].data_ptr()
        _, _, want, A = attention_grad(q, k, v, cu, cu, d ** -0.5, dO)
        _check(got, want, A, dtype, _S(q, k, d ** -0.5))
        assert (grad[:2] == 5).all() and (grad[-2:] == 5).all() and (grad[:, -1] == 5).all()


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,d", [
    ("bf16", [200, 77], 4, 2, 64), ("bf16", [200, 77], 4, 2, 128), ("bf16", [70], 2, 1, 16),
    ("f32", [200, 77], 4, 2, 64), ("f32", [130], 2, 2, 128), ("f32", [700], 8, 1, 32),
])
def test_odd_addresses(F, dtype, lens, Hq, Hkv, d):
    """Rows off the 16-byte boundaries, each operand in turn, agree with the aligned call's tolerances."""
    q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, 8)
    cu = _cu(lens)
    o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), max(lens))
    _, _, want, A = attention_grad(q, k, v, cu, cu, d ** -0.5, dO)

    def odd(x):
        buf = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        y = buf[1:].view(x.shape)
        return y.copy_(x)

    for which in range(6):
        args = [odd(x) if which == i else x for i, x in enumerate((q, k, v, o))]
        g = odd(dO) if which == 4 else dO
        out = {n: odd(torch.zeros_like(x)) for n, x in (("dq", q), ("dk", k), ("dv", v))} if which == 5 else None
        got = F.attn_prompt_backward(*args, lse, g, _dev(cu), max_q=max(lens), out=out)
        _check(got, want, A, dtype, _S(q, k, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_and_past_max_q(F, dtype):
    lens, d = [130, 260], 64
    q, k, v, dO = _inputs(lens, lens, 4, 2, d, dtype, 4, behind=9)
    for x in (q, k, v, dO):
        x[-9:] = math.nan
    cu = _cu(lens)
    o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), 260)
    o[-9:], lse[-9:] = math.nan, math.nan
    out = {n: torch.full_like(x, 3.0) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=260, out=out)
    _, _, want, A = attention_grad(q[:-9], k[:-9], v[:-9], cu, cu, d ** -0.5, dO[:-9])
    assert all((x[-9:] == 3).all() for x in got.values())
    _check({n: x[:-9] for n, x in got.items()}, want, A, dtype, _S(q[:-9], k[:-9], d ** -0.5))
    fresh = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=260)
    assert all(not x[-9:].any() for x in fresh.values())

    # rows past max_q of their sequence: untouched, and without influence
    out = {n: torch.full_like(x, 3.0) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    dO2 = dO.clone()
    dO2[100:130] = math.nan
    o2 = o.clone()
    o2[100:130] = math.nan
    got = F.attn_prompt_backward(q, k, v, o2, lse, dO2, _dev(cu), max_q=100, out=out)
    cut = torch.cat([torch.arange(100), 130 + torch.arange(100)])
    rest = torch.tensor(sorted(set(range(390)) - set(cut.tolist())))
    assert (got["dq"][rest.cuda()] == 3).all()
    dO3 = torch.nan_to_num(dO2)
    _, _, want, A = attention_grad(q[:-9], k[:-9], v[:-9], cu, cu, d ** -0.5, dO3[:-9], max_q=100)
    got = {n: x[:-9] for n, x in got.items()}
    got["dq"], want["dq"], A["dq"] = (x[cut.cuda()] for x in (got["dq"], want["dq"], A["dq"]))
    _check(got, want, A, dtype, _S(q[:-9], k[:-9], d ** -0.5))


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,d", [("bf16", [2000] * 8, 12, 12, 64), ("bf16", [4000], 16, 4, 128), ("bf16", [70] * 90, 8, 2, 128),
                                                 ("bf16", [2999], 8, 1, 32), ("f32", [1999], 8, 2, 128)])
def test_rows_past_a_sequence_cost_no_time(F, dtype, lens, Hq, Hkv, d):
    """Queries and their gradients that are not finite behind the last sequence, as memory that was never written may hold
    them, and in front of each: the same bits in dk and dv, and not some hundred times as long, as with zeros there."""
    n = sum(lens) + 9
    cu = _dev([5 + x for x in _cu(lens)])
    q, k, v, dO = _inputs([n], [n], Hq, Hkv, d, dtype, 3)
    p = F.AttnParams(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=max(lens),
                     tokens=n, k_tokens=n)
    ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
    o, lse = _forward(F, q, k, v, cu, cu, max(lens))
    times, results = [], []
    for value in (0.0, math.nan):
        for x in (q, dO):
            x[:5], x[-4:] = value, value
        out = {m: torch.zeros_like(x) for m, x in (("dk", k), ("dv", v))}
        ms = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, out, ws)
            b.record()
            b.synchronize()
            ms.append(a.elapsed_time(b))
        assert F.falcon_workspace_status(ws) == F.FALCON_OK
        times.append(min(ms))
        results.append(out)
    assert all(torch.equal(results[0][m], results[1][m]) for m in results[0])
    assert times[1] < 4 * times[0] + 0.05, times


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,d", [("bf16", [2000] * 8, 12, 12, 64), ("bf16", [4000], 16, 4, 128), ("bf16", [70] * 90, 8, 2, 128),
                                                 ("bf16", [2999], 8, 1, 32), ("bf16", [1, 3, 129, 65, 64, 128, 200] * 5, 4, 2, 64),
                                                 ("bf16", [1, 3, 129, 65, 64, 128, 200] * 5, 4, 2, 128), ("f32", [1999], 8, 2, 128)])
def test_keys_past_a_sequence_cost_no_time(F, dtype, lens, Hq, Hkv, d):
    """The same of dq, with all operands not finite around the sequences; and of the three together."""
    n = sum(lens) + 9
    cu = _dev([5 + x for x in _cu(lens)])
    x = q, k, v, dO = _inputs([n], [n], Hq, Hkv, d, dtype, 3)
    p = F.AttnParams(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=max(lens),
                     tokens=n, k_tokens=n)
    ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
    o, lse = _forward(F, q, k, v, cu, cu, max(lens))
    for names in (("dq",), ("dq", "dk", "dv")):
        times, results = [], []
        for value in (0.0, math.nan):
            for t in x:
                t[:5], t[-4:] = value, value
            out = {m: torch.zeros_like(t) for m, t in (("dq", q), ("dk", k), ("dv", v)) if m in names}
            ms = []
            for _ in range(5):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, out, ws)
                b.record()
                b.synchronize()
                ms.append(a.elapsed_time(b))
            assert F.falcon_workspace_status(ws) == F.FALCON_OK
            times.append(min(ms))
            results.append(out)
        assert all(torch.equal(results[0][m], results[1][m]) for m in names)
        assert times[1] < 4 * times[0] + 0.05, times


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("bf16", 64, 2, 1), ("bf16", 128, 2, 1), ("bf16", 32, 2, 1), ("f32", 64, 2, 1),
                                              ("f32", 128, 2, 1), ("f32", 16, 16, 1), ("f32", 128, 16, 1),
                                              ("bf16", 64, 16, 1), ("bf16", 128, 16, 1)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_infinities_and_nan_reach_only_what_sees_them(F, dtype, d, Hq, Hkv, value):
    """A key's row at 60 of 150 is not finite: queries before it see none of it.  A query's gradient at 100 is not finite:
    keys after it are not touched by it.  And the next sequence's first rows are not finite."""
    lens = [150, 40]
    cu = _cu(lens)
    for what in ("k", "v", "dO", "q", "next"):
        q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, 6)
        x = dict(q=q, k=k, v=v, dO=dO)
        if what == "next":
            for t in x.values():
                t[150:153] = value
        else:
            x[what][100 if what in ("dO", "q") else 60, 0, 3] = value
        o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), 150)
        got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=150)
        with np.errstate(all="ignore"):
            want = O.prompt_grad(_np(q), _np(k), _np(v), cu, cu, d ** -0.5, _np(dO))
        clean = [t.clone() for t in (q, k, v, dO)]
        for t in clean:
            torch.nan_to_num_(t, 0.0, 0.0, 0.0)
        _, _, _, A = attention_grad(*clean[:3], cu, cu, d ** -0.5, clean[3])
        first = 150 if what == "next" else 390
        for name, w in zip(("dq", "dk", "dv"), want):
            w = torch.from_numpy(w).cuda()
            fine = torch.isfinite(w)
            y = got[name].double()
            # where the definition is finite, so is the result, and right; a row that reads the value is not checked further
            tol = 3 * U * A[name] + U * w.abs() if dtype == "bf16" else 2e-5 * A[name]
            ok = ~fine | ((y - w).abs() <= tol + 1e-30)
            assert ok[:first].all(), (what, name, (~ok).nonzero()[:4].tolist())
            if what == "k":
                assert fine[:60].all() == (name == "dq"), name


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("bf16", 64, 2, 1), ("bf16", 128, 2, 1), ("bf16", 32, 16, 1), ("bf16", 128, 16, 1),
                                            ("f32", 64, 2, 1), ("f32", 128, 16, 1)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_infinities_and_nan_reach_all_that_sees_them(F, dtype, d, Hq, Hkv, value):
    """Where the definition's gradient is not finite, neither is the result."""
    lens = [150, 40]
    cu = _cu(lens)
    for what in ("k", "v", "dO", "q", "dlse"):
        q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, 6)
        dlse = _rand(q.shape[:2], "f32", 9)
        x = dict(q=q, k=k, v=v, dO=dO)
        if what == "dlse":
            dlse[100, 1] = value
        else:
            x[what][100 if what in ("dO", "q") else 60, 0, 3] = value
        o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), 150)
        got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=150, dlse=dlse)
        with np.errstate(all="ignore"):
            want = O.prompt_grad(_np(q), _np(k), _np(v), cu, cu, d ** -0.5, _np(dO), _np(dlse))
        for name, w in zip(("dq", "dk", "dv"), want):
            fine = torch.isfinite(torch.from_numpy(w).cuda())
            lost = ~fine & torch.isfinite(got[name])
            assert not lost.any(), (what, name, lost.nonzero()[:4].tolist(), int(lost.sum()), int((~fine).sum()))
            extra = fine & ~torch.isfinite(got[name])
            assert not extra.any(), (what, name, extra.nonzero()[:4].tolist(), int(extra.sum()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,d", [
    ([1500], [1500], 8, 1, 64), ([900], [1700], 16, 1, 128), ([700, 20, 333], [700, 20, 333], 12, 1, 32),
    ([1100], [600], 8, 1, 128), ([300], [5], 16, 1, 64),
])
def test_keys_shared_by_several_ctas(F, dtype, lq, lk, Hq, Hkv, d):
    """One key head: the queries of a block of keys are dealt out over a cluster, some of whose CTAs may have none."""
    q, k, v, dO = _inputs(lq, lk, Hq, Hkv, d, dtype, 31)
    cu_q, cu_k = _cu(lq), _cu(lk)
    o, lse = _forward(F, q, k, v, _dev(cu_q), _dev(cu_k), max(lq))
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu_q), _dev(cu_k), max(lq))
    _, _, want, A = attention_grad(q, k, v, cu_q, cu_k, d ** -0.5, dO)
    _check(got, want, A, dtype, _S(q, k, d ** -0.5))
    again = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu_q), _dev(cu_k), max(lq))
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [([1500] + [16] * 40, 8, 1, 64), ([7] * 30 + [1200, 1], 8, 2, 128), ([16] * 50 + [2100], 16, 2, 32)])
def test_one_long_sequence_beside_short_ones(F, dtype, lens, Hq, Hkv, d):
    q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, 41)
    cu = _cu(lens)
    o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), max(lens))
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=max(lens))
    _, _, want, A = attention_grad(q, k, v, cu, cu, d ** -0.5, dO)
    _check(got, want, A, dtype, _S(q, k, d ** -0.5))
    again = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=max(lens))
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_sizes(F, dtype, d):
    """Rows of dO and of v scaled by powers of two between 2^-30 and 2^30, some rows of dO zero with a gradient of their log
    sum: an error stays relative to what a sum is formed of.  (fp32's 2^-40 of a row's largest, times the largest of 64
    terms, is below 2^-22 of A but for elements 2^-12 below their row's largest, which have 2^-20.)"""
    lens = [260, 77]
    q, k, v, dO = _inputs(lens, lens, 4, 2, d, dtype, 12)
    g = torch.Generator().manual_seed(5)
    for x in (v, dO):
        x *= torch.exp2(torch.randint(-30, 31, (x.shape[0], 1, 1), generator=g).float()).cuda().to(x.dtype)
    dO[5::7] = 0
    dlse = _rand(q.shape[:2], "f32", 9)
    cu = _cu(lens)
    o, lse = _forward(F, q, k, v, _dev(cu), _dev(cu), 260)
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu), max_q=260, dlse=dlse)
    _, _, want, A = attention_grad(q, k, v, cu, cu, d ** -0.5, dO, dlse)
    S = _S(q, k, d ** -0.5)
    for n in want:
        tol = 3 * U * A[n] + U * want[n].abs() if dtype == "bf16" else (2.0 ** -22 * (2 * S + 8) + 2.0 ** -19) * A[n]
        worst = ((got[n].double() - want[n]).abs() / (tol + 1e-30)).max().item()
        assert worst <= 1.0, (n, worst)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up", [110, -110])
def test_rows_at_the_ends_of_fp32(F, d, up):
    """Queries of 2^110 against keys of 2^-110 and the other way round; scores of -60 and 60 from rows that are each other's
    negative or the same.  Such a score's products have one sign, and the tensor cores cut their sum off eight times (16 dims
    at a time, high halves; the other parts are below 2^-10 of it): 2^-23 S each, 2^-20 S of a weight on top of the
    tolerance of the other tests, whose products cancel.  The small operand's gradient lies at 2^-110 and below: dS times
    that row's factor (2^-15 of its largest element, or more) is off by 2^-150 where it is not a normal number, times 2^15
    for each of 90 terms, together below fp32's smallest normal number, 2^-126."""
    lens = [1, 1, 90, 2]
    q, k, v, dO = _inputs(lens, lens, 2, 2, d, "f32", 14)
    k[:2] = -q[:2]
    k[-2:] = q[-2:]
    scale = 60.0 / d
    q, k = q * 2.0 ** up, k * 2.0 ** -up
    cu = _cu(lens)
    o, lse, want, A = attention_grad(q, k, v, cu, cu, scale, dO)
    got = F.attn_prompt_backward(q, k, v, o.float(), lse.float(), dO, _dev(cu), None, 90, scale)
    S = _S(q, k, scale)
    for name, f in (("dq", 2.0 ** up), ("dk", 2.0 ** -up), ("dv", 1.0)):
        tol = (2.0 ** -22 * (2 * S + 8) + 2.0 ** -20 * S + 2.0 ** -20) * (A[name] * f) + 2.0 ** -126 * f
        worst = ((got[name].double() - want[name]).abs() * f / tol).max().item()
        assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
def test_calls_behind_one_another_over_one_workspace(F, dtype, d):
    """Calls of different sizes queued without a wait between them: the kernels of a call overlap, those of two do not."""
    calls, most = [], 0
    for lens, Hq, Hkv in (([900], 8, 1), ([33, 150], 4, 4), ([512, 300], 6, 2), ([1], 2, 2)):
        n = sum(lens)
        q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, n)
        cu = _dev(_cu(lens))
        o, lse = _forward(F, q, k, v, cu, cu, max(lens))
        p = F.AttnParams(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32,
                         max_q=max(lens), tokens=n, k_tokens=n)
        most = max(most, F.falcon_attn_prompt_backward_workspace_size(p))
        want = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=max(lens))
        calls.append((p, (q, k, v, cu, cu, o, lse, dO, None), want, {m: torch.zeros_like(x) for m, x in want.items()}))
    ws = F.alloc_workspace(most)
    torch.cuda.synchronize()
    for _ in range(6):
        for p, args, _, out in calls:
            F.falcon_attn_prompt_backward(p, *args, out, ws)
            ws.fill_(0xFF)  # what the next call does not write itself is of no use to it
    for _, _, want, out in calls:
        assert all(torch.equal(out[m], want[m]) for m in want)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (16, 1)])
def test_a_wait_that_runs_out_is_reported(F, dtype, d, Hq, Hkv):
    """The copies of the first kernel never begin: the call ends with a timeout, and the next one is right."""
    lens = [700]
    q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, 2)
    cu = _dev(_cu(lens))
    o, lse = _forward(F, q, k, v, cu, cu, 700)
    p = F.AttnParams(B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=700,
                     tokens=700, k_tokens=700)
    ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
    out = {m: torch.full_like(x, 3.0) for m, x in (("dq", q), ("dk", k), ("dv", v))}
    run = lambda: F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, out, ws)  # noqa: E731
    try:
        F.falcon_test_hooks(wait_limit_ns=2_000_000, stall=True)
        run()
        assert F.falcon_workspace_status(ws) == F.FALCON_ERR_TIMEOUT
    finally:
        F.falcon_test_hooks(0, False)
    assert (out["dk"] == 3).all() and (out["dv"] == 3).all()
    run()
    assert F.falcon_workspace_status(ws) == F.FALCON_OK
    want = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=700)
    assert all(torch.equal(out[m], want[m]) for m in want)


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("lens", [[700], [2000] * 12])
def test_a_wait_of_dq_alone_that_runs_out_is_reported(F, dtype, d, lens):
    """The copies of dQ's kernel never begin: reported after the limit, however many keys the call has; the next call is right."""
    n = sum(lens)
    q, k, v, dO = _inputs(lens, lens, 4, 2, d, dtype, 2)
    cu = _dev(_cu(lens))
    o, lse = _forward(F, q, k, v, cu, cu, lens[0])
    want = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=lens[0])["dq"]
    p = F.AttnParams(B=len(lens), Hq=4, Hkv=2, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=lens[0],
                     tokens=n, k_tokens=n)
    ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
    out = {"dq": torch.full_like(q, 3.0)}
    run = lambda: F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, out, ws)  # noqa: E731
    torch.cuda.synchronize()
    try:
        F.falcon_test_hooks(wait_limit_ns=2_000_000, stall=True)
        begin = time.perf_counter()
        run()
        assert F.falcon_workspace_status(ws) == F.FALCON_ERR_TIMEOUT
        took = time.perf_counter() - begin
    finally:
        F.falcon_test_hooks(0, False)
    # a CTA waits for the limit in at most five places after one another; at most 12 x 16 x 4 CTAs in 152 places
    assert took < 0.25, took
    assert (out["dq"] == 3).all()
    run()
    assert F.falcon_workspace_status(ws) == F.FALCON_OK
    assert torch.equal(out["dq"], want)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 32), ("f32", 128)])
def test_many_short_sequences(F, dtype, d):
    """Several blocks a CTA, most of them a few rows, some sequences empty, some with keys alone; rows before the first one."""
    g = torch.Generator().manual_seed(d)
    lq = torch.randint(0, 10, (260,), generator=g).tolist()
    lk = [n if i % 3 else max(0, n + i % 7 - 3) for i, n in enumerate(lq)]
    lq[7], lk[7] = 300, 410
    cu_q, cu_k = ([5 + x for x in _cu(n)] for n in (lq, lk))
    n, m, Hq, Hkv = cu_q[-1], cu_k[-1], 8, 4
    q, k, v, dO = (_rand((rows, H, d), dtype, seed, seed < 3) for seed, rows, H in
                   ((1, n, Hq), (2, m, Hkv), (3, m, Hkv), (4, n, Hq)))
    o, lse = _forward(F, q, k, v, _dev(cu_q), _dev(cu_k), max(lq))
    out = {name: torch.full_like(x, 3.0) for name, x in (("dq", q), ("dk", k), ("dv", v))}
    got = F.attn_prompt_backward(q, k, v, o, lse, dO, _dev(cu_q), _dev(cu_k), max(lq), out=out)
    _, _, want, A = attention_grad(q, k, v, cu_q, cu_k, d ** -0.5, dO)
    assert all((x[:5] == 3).all() for x in got.values())
    cut = lambda xs: {name: x[5:] for name, x in xs.items()}  # noqa: E731
    _check(cut(got), cut(want), cut(A), dtype, _S(q, k, d ** -0.5))


@pytest.mark.parametrize("d,Hq", [(64, 8), (128, 4)])
def test_rows_computed_again_outlast_the_waits(F, d, Hq):
    """An infinite key at 2000 of 3000: the queries before it in its tile are computed again, milliseconds of work, while the
    CTA's next blocks wait with a limit of half a millisecond."""
    lens = [3000] * 4
    cu = _dev(_cu(lens))
    n = sum(lens)
    q, k, v, dO = _inputs(lens, lens, Hq, Hq, d, "bf16", 3)
    o, lse = _forward(F, q, k, v, cu, cu, 3000)
    for b in range(4):
        v[3000 * b + 2000] = math.inf
    p = F.AttnParams(B=4, Hq=Hq, Hkv=Hq, d=d, dtype=F.FALCON_BF16, max_q=3000, tokens=n, k_tokens=n)
    ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
    got = [{"dq": torch.full_like(q, 3.0)} for _ in range(2)]
    try:
        for out, limit in zip(got, (0, 500_000)):
            F.falcon_test_hooks(wait_limit_ns=limit)
            F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, out, ws)
            assert F.falcon_workspace_status(ws) == F.FALCON_OK
    finally:
        F.falcon_test_hooks(0, False)
    x = got[0]["dq"].view(4, 3000, Hq, d)
    assert torch.isfinite(x[:, :2000]).all() and not torch.isfinite(x[:, 2000:]).any()
    assert torch.equal(got[1]["dq"].view(torch.int16), got[0]["dq"].view(torch.int16))


def test_no_queries_and_no_keys(F):
    """Keys that no query sees get zeros; queries without keys too; empty calls write nothing."""
    d = 64
    for dtype in ("bf16", "f32"):
        q, k, v, dO = _inputs([5, 0], [0, 70], 2, 2, d, dtype)
        cu_q, cu_k = _dev([0, 5, 5]), _dev([0, 0, 70])
        o, lse = _forward(F, q, k, v, cu_q, cu_k, 5)
        out = {n: torch.full_like(x, 3.0) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        got = F.attn_prompt_backward(q, k, v, o, lse, dO, cu_q, cu_k, 5, out=out)
        assert all(not x.any() for x in got.values())
        e = lambda x: x[:0]  # noqa: E731
        out = {n: torch.full_like(x, 3.0) for n, x in (("dk", k), ("dv", v))}
        got = F.attn_prompt_backward(e(q), k, v, e(o), e(lse), e(dO), _dev([0, 0, 0]), cu_k, 1, out=out)
        assert got["dq"].shape[0] == 0 and not got["dk"].any() and not got["dv"].any()
        got = F.attn_prompt_backward(q, e(k), e(v), o, lse, dO, cu_q, _dev([0, 0, 0]), 5)
        assert not got["dq"].any()
        F.attn_prompt_backward(e(q), e(k), e(v), e(o), e(lse), e(dO), _dev([0, 0]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_calls_without_queries_clear_the_status(F, dtype, d):
    q, k, v, dO = _inputs([5], [70], 2, 1, d, dtype)
    lse = torch.zeros(5, 2, device="cuda")
    for tokens, max_q in ((0, 3), (5, 0)):
        p = F.AttnParams(B=1, Hq=2, Hkv=1, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=max_q,
                         tokens=tokens, k_tokens=70)
        ws = F.alloc_workspace(F.falcon_attn_prompt_backward_workspace_size(p))
        ws.fill_(0xFF)
        out = {n: torch.full_like(k, 3.0) for n in ("dk", "dv")}
        F.falcon_attn_prompt_backward(p, q, k, v, _dev([0, tokens]), _dev([0, 70]), q, lse, dO, None, out, ws)
        assert F.falcon_workspace_status(ws) == F.FALCON_OK
        assert not out["dk"].any() and not out["dv"].any()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
def test_captured_calls_share_a_workspace(F, dtype, d):
    """Two graphs of different sizes over one workspace, replayed in turn with new inputs."""
    Hq, Hkv, calls = 4, 2, []
    most = 0
    for lens in ([300, 100], [129]):
        n = sum(lens)
        cu = _dev(_cu(lens))
        q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, dtype, n)
        p = F.AttnParams(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32,
                         max_q=max(lens), tokens=n, k_tokens=n)
        most = max(most, F.falcon_attn_prompt_backward_workspace_size(p))
        g = {name: torch.zeros_like(x) for name, x in (("dq", q), ("dk", k), ("dv", v))}
        calls.append((p, lens, cu, q, k, v, dO, g))
    ws = F.alloc_workspace(most)
    graphs = []
    for p, lens, cu, q, k, v, dO, g in calls:
        o, lse = _forward(F, q, k, v, cu, cu, max(lens))
        run = lambda: F.falcon_attn_prompt_backward(p, q, k, v, cu, cu, o, lse, dO, None, g, ws)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append((graph, o, lse))
    for seed in (100, 200):
        for (p, lens, cu, q, k, v, dO, g), (graph, o, lse) in zip(calls, graphs):
            for t, x in zip((q, k, v, dO), _inputs(lens, lens, Hq, Hkv, d, dtype, seed)):
                t.copy_(x)
            for t, x in zip((o, lse), _forward(F, q, k, v, cu, cu, max(lens))):
                t.copy_(x)
            for x in g.values():
                x.fill_(9.0)
            graph.replay()
        for (p, lens, cu, q, k, v, dO, g), (graph, o, lse) in zip(calls, graphs):
            want = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=max(lens))
            assert all(torch.equal(g[name], want[name]) for name in g)
    assert F.falcon_workspace_status(ws) == F.FALCON_OK


def test_differences_of_the_forward(F):
    """<dx, u> against (L(x + h u) - L(x - h u)) / 2 h of the fp32 forward, L = <o, dO> + <lse, dlse>: the step's
    h^2 / 6 of the third derivative, below 2^-10 of |dx| |u|, and two roundings of L, 2^-22 of sum |o dO| over h."""
    lens, Hq, Hkv, d, h = [90, 33], 4, 2, 64, 2.0 ** -7
    q, k, v, dO = _inputs(lens, lens, Hq, Hkv, d, "f32", 12)
    dlse = _rand(q.shape[:2], "f32", 13)
    cu = _dev(_cu(lens))

    def loss(q, k, v):
        o, lse = _forward(F, q, k, v, cu, cu, 90)
        return ((o.double() * dO).sum() + (lse.double() * dlse).sum()).item(), (o.double() * dO).abs().sum().item()

    o, lse = _forward(F, q, k, v, cu, cu, 90)
    g = F.attn_prompt_backward(q, k, v, o, lse, dO, cu, max_q=90, dlse=dlse)
    for name, at in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        u = _rand(x[at].shape, "f32", 20 + at)
        u = u / u.norm() * g[name].norm().sqrt()
        x[at] = x[at] + h * u
        hi, size = loss(*x)
        x[at] = x[at] - 2 * h * u
        lo, _ = loss(*x)
        want = (g[name].double() * u).sum().item()
        tol = 2.0 ** -10 * (g[name].norm() * u.norm()).item() + 2.0 ** -22 * size / h
        assert abs((hi - lo) / (2 * h) - want) <= tol


# ---------------------------------------------------------------- norm and rotation
def _norm_args(F, n, Hq, Hkv, d, rot, dtype, fused=0, seed=1):
    g = torch.Generator().manual_seed(seed)
    mk = lambda H, s: (_rand((n, H + fused, d), dtype, s) * (0.2 + 4.8 * torch.rand((n, 1, 1), generator=g).cuda()).to(  # noqa: E731
        DT[dtype]))[:, fused:]
    q, k, gq, gk = mk(Hq, 1), mk(Hkv, 2), _rand((n, Hq, d), dtype, 3), _rand((n, Hkv, d), dtype, 4)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g)).cuda(), (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    table = F.rope_table(*F.rope_frequencies(rot)[:1], 500) if rot else None
    pos = torch.randint(0, 500, (n,), generator=g).cuda() if rot else None
    return q, k, gq, gk, wq, wk, table, pos


def _check_rows(got, want, x, w, dy, dtype, norm):
    """Some thirty fp32 roundings of terms up to r |u|_max: 2^-19 of it for a row; bf16 rounds once more."""
    size = np.abs(dy).max(-1, keepdims=True) * 2
    if norm:
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        # mean(u x r) x r is at most the largest |u| times |x r| |x r|_rms: below sqrt(d) of it
        size = size * r * np.abs(w).max() * (1 + np.abs(x * r).max(-1, keepdims=True))
    tol = 2.0 ** -19 * size + (U * np.abs(want) if dtype == "bf16" else 0)
    assert (np.abs(got - want) <= tol + 1e-30).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,layout,norm,fused", [
    (1, 1, 1, 16, 16, "half", True, 0), (7, 12, 4, 64, 64, "half", True, 0), (33, 5, 5, 64, 32, "interleaved", True, 3),
    (19, 16, 2, 128, 128, "half", True, 2), (9, 3, 1, 128, 6, "half", True, 0), (9, 3, 1, 32, 10, "interleaved", True, 1),
    (5, 8, 8, 128, 50, "half", False, 0), (300, 17, 1, 32, 32, "half", True, 0), (4, 2, 2, 64, 0, "half", True, 0),
    (1300, 2, 1, 16, 8, "half", True, 0), (77, 12, 12, 64, 64, "interleaved", False, 0), (6000, 1, 1, 64, 64, "half", True, 1),
])
def test_norm_rope_gradients(F, dtype, n, Hq, Hkv, d, rot, layout, norm, fused):
    q, k, gq, gk, wq, wk, table, pos = _norm_args(F, n, Hq, Hkv, d, rot, dtype, fused)
    lay = F.FALCON_ROPE_HALF if layout == "half" else F.FALCON_ROPE_INTERLEAVED
    got = F.qk_norm_rope_backward(q, k, gq, gk, pos, table, wq, wk, norm=norm, layout=lay)
    assert set(got) == ({"dq", "dk", "dw_q", "dw_k"} if norm else {"dq", "dk"})
    for x, w, dy, a, b in ((q, wq, gq, "dq", "dw_q"), (k, wk, gk, "dk", "dw_k")):
        dx, dw = O.norm_rope_grad(_np(x), _np(w), 1e-6 if norm else None, _np(pos).astype(int) if rot else None,
                                  table.cpu().numpy() if rot else None, layout, _np(dy))
        _check_rows(_np(got[a]), dx, _np(x), _np(w), _np(dy), dtype, norm)
        if norm:
            # terms off by 2^-21 of their size; sums of a lane, of lanes and of CTAs: at most 64 roundings deep on the way
            r = 1 / np.sqrt((_np(x) ** 2).mean(-1, keepdims=True) + 1e-6)
            size = 2 * (np.abs(_np(dy)).max(-1, keepdims=True) * np.abs(_np(x) * r)).sum((0, 1))
            assert (np.abs(_np(got[b]) - dw) <= (2.0 ** -21 + 64 * 2.0 ** -24) * size).all()


def test_norm_rope_gradients_in_place_alone_and_at_odd_addresses(F):
    n, H, d = 37, 3, 64
    q, k, gq, gk, wq, wk, table, pos = _norm_args(F, n, H, H, d, 64, "bf16")
    want = F.qk_norm_rope_backward(q, k, gq, gk, pos, table, wq, wk)
    alone = F.qk_norm_rope_backward(q, None, gq, None, pos, table, wq)
    assert set(alone) == {"dq", "dw_q"} and torch.equal(alone["dq"], want["dq"])
    # other CTAs share the rows out: dw's order may be another
    assert torch.allclose(alone["dw_q"], want["dw_q"], rtol=0, atol=1e-5 * want["dw_q"].abs().max().item())
    gq2, gk2 = gq.clone(), gk.clone()
    got = F.qk_norm_rope_backward(q, k, gq2, gk2, pos, table, wq, wk, out={"dq": gq2, "dk": gk2})
    assert got["dq"].data_ptr() == gq2.data_ptr()
    assert all(torch.equal(got[m], want[m]) for m in want)
    # rows two bytes past a boundary, in place (pairs read from memory before a row is written)
    for layout in (F.FALCON_ROPE_HALF, F.FALCON_ROPE_INTERLEAVED):
        want = F.qk_norm_rope_backward(q, k, gq, gk, pos, table, wq, wk, layout=layout)
        buf = torch.full((n, H * d + 5), 2.0, dtype=torch.bfloat16, device="cuda")
        odd = buf[:, 1:1 + H * d].unflatten(1, (H, d))
        odd.copy_(gq)
        got = F.qk_norm_rope_backward(q, k, odd, gk, pos, table, wq, wk, out={"dq": odd}, layout=layout)
        for m in want:  # another order of the same roundings
            scale = want[m].float().abs().max()
            assert ((got[m].float() - want[m].float()).abs() <= 2 * U * want[m].float().abs() + 2.0 ** -17 * scale).all()
        assert (buf[:, 0] == 2).all() and (buf[:, 1 + H * d:] == 2).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_rope_gradients_of_positions_outside_the_table(F, layout):
    q = _rand((5, 2, 64), "f32", 5)
    g = _rand((5, 2, 64), "f32", 6)
    table = F.rope_table(F.rope_frequencies(32)[0], 10)
    pos = torch.tensor([-1, 0, 9, 10, 1 << 40]).cuda()
    lay = F.FALCON_ROPE_HALF if layout == "half" else F.FALCON_ROPE_INTERLEAVED
    got = F.qk_norm_rope_backward(q, None, g, None, pos, table, norm=False, layout=lay)
    bad = torch.isnan(got["dq"][..., :32]).all(-1)
    assert bad.tolist() == [[True, True], [False] * 2, [False] * 2, [True] * 2, [True] * 2]
    assert torch.isfinite(got["dq"][..., 32:]).all() and torch.isfinite(got["dq"][1:3]).all()
    got = F.qk_norm_rope_backward(q, None, g, None, pos, table, layout=lay)
    assert torch.isnan(got["dq"]).flatten(1).all(1).tolist() == [True, False, False, True, True]
    assert torch.isnan(got["dw_q"]).tolist() == [True] * 32 + [False] * 32  # dw_c is a sum of n_c alone


def test_norm_rope_gradients_of_extreme_rows(F):
    """Zero rows, rows of tiny values, rows whose square sum passes fp32's range, and no rows at all."""
    x = torch.zeros((4, 1, 64), device="cuda")
    x[1] = 1e-25
    x[2] = 1e30
    x[3] = _rand((1, 64), "f32", 1)
    g = _rand((4, 1, 64), "f32", 2)
    got = F.qk_norm_rope_backward(x, None, g, None)
    dx, dw = O.norm_rope_grad(_np(x), None, 1e-6, None, None, "half", _np(g))
    assert torch.allclose(got["dq"].double().cpu()[[0, 1, 3]], torch.from_numpy(dx)[[0, 1, 3]], rtol=2e-6, atol=1e-5)
    assert not got["dq"][2].any() and torch.isfinite(got["dw_q"]).all()
    rest = O.norm_rope_grad(_np(x)[[0, 1, 3]], None, 1e-6, None, None, "half", _np(g)[[0, 1, 3]])[1]
    assert np.abs(_np(got["dw_q"]) - rest).max() < 1e-5
    none = F.qk_norm_rope_backward(x[:0], x[:0], g[:0], g[:0])
    assert not none["dw_q"].any() and not none["dw_k"].any() and none["dq"].shape[0] == 0


def test_norm_rope_gradients_captured(F):
    """A captured call over a workspace that an eager call uses in between; the same bits each time."""
    q, k, gq, gk, wq, wk, table, pos = _norm_args(F, 700, 8, 2, 64, 64, "bf16")
    p = F.AttnParams(Hq=8, Hkv=2, d=64, dtype=F.FALCON_BF16, tokens=700, qk_norm=1, rot=64, rope_rows=500)
    ws = F.alloc_workspace(F.falcon_qk_norm_rope_backward_workspace_size(p))
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k)}
    dw = [torch.empty(64, device="cuda") for _ in range(2)]
    run = lambda: F.falcon_qk_norm_rope_backward(p, q, k, wq, wk, pos, table, gq, gk, g, *dw, ws)  # noqa: E731
    run()
    first = [x.clone() for x in (g["dq"], g["dk"], *dw)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for x in (g["dq"], g["dk"], *dw):
            x.fill_(4.0)
        ws.fill_(255)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, (g["dq"], g["dk"], *dw)))


# ---------------------------------------------------------------- together
def test_a_layer_end_to_end(F):
    """Norm, rotation and attention forward, then back to the fused projection, against fp64 differentiation of the
    same rounded intermediate rows: each operator's own tolerance carries to the next, 2^-5 of the norm overall."""
    lens, Hq, Hkv, d = [120, 77], 4, 2, 64
    n = sum(lens)
    x = _rand((n, Hq + 2 * Hkv, d), "bf16", 1)
    wq, wk = 1 + 0.1 * _rand((d,), "f32", 2), 1 + 0.1 * _rand((d,), "f32", 3)
    dO = _rand((n, Hq, d), "bf16", 4)
    table = F.rope_table(F.rope_frequencies(d)[0], 200)
    cu = _dev(_cu(lens))
    pos = torch.cat([torch.arange(m) for m in lens]).cuda()
    q, k, v = torch.split(x, [Hq, Hkv, Hkv], 1)
    qr, kr = F.qk_norm_rope(q, k, pos, table, wq, wk)
    o, lse = F.attn_prompt(qr, kr, v, cu, max_q=120, want_lse=True)
    dx = torch.empty_like(x)
    parts = dict(zip(("dq", "dk", "dv"), torch.split(dx, [Hq, Hkv, Hkv], 1)))
    a = F.attn_prompt_backward(qr, kr, v, o, lse, dO, cu, max_q=120, out={"dv": parts["dv"]})
    b = F.qk_norm_rope_backward(q, k, a["dq"], a["dk"], pos, table, wq, wk, out={m: parts[m] for m in ("dq", "dk")})

    X, W = x.double().requires_grad_(), [w.double().requires_grad_() for w in (wq, wk)]
    t = torch.view_as_complex(table.double().contiguous())[pos].unsqueeze(1)

    def rotated(y, w):
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * t
        return torch.cat([z.real, z.imag], -1)

    Q, K, V = rotated(X[:, :Hq], W[0]), rotated(X[:, Hq:Hq + Hkv], W[1]), X[:, Hq + Hkv:]
    loss, at = 0.0, 0
    for m in lens:
        s = slice(at, at + m)
        Kh, Vh = (y[s].repeat_interleave(Hq // Hkv, 1) for y in (K, V))
        sc = torch.einsum("ihd,jhd->hij", Q[s], Kh) * d ** -0.5
        sc = sc.masked_fill(~torch.ones((m, m), dtype=torch.bool, device="cuda").tril(), -math.inf)
        loss = loss + (torch.einsum("hij,jhd->ihd", sc.softmax(-1), Vh) * dO[s].double()).sum()
        at += m
    gx, gq, gk = torch.autograd.grad(loss, [X, *W])
    for got, want in ((dx, gx), (b["dw_q"], gq), (b["dw_k"], gk)):
        assert (got.double() - want).norm() <= 2.0 ** -5 * want.norm()
