"""The softmax-attention operators' gradients without a GPU: the oracle's pins,
and the refusals that the host gives before anything is enqueued (the addresses
handed in are never dereferenced)."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from attn_grad_ref import attention_grad
from oracle import softmax_attention as O


@pytest.fixture(scope="module")
def F():
    import __graft_entry__
    __graft_entry__.build()
    import chunked_delta_rule_gb300 as F
    return F


# ---------------------------------------------------------------- oracle pins
CU_Q, CU_K = [0, 4, 4, 9, 11], [0, 6, 8, 11, 11]


def _call(seed=0, Hq=4, Hkv=2, d=4):
    g = np.random.default_rng(seed)
    n, m = CU_Q[-1], CU_K[-1]
    return [g.standard_normal(s) for s in ((n, Hq, d), (m, Hkv, d), (m, Hkv, d), (n, Hq, d), (n, Hq))]


def test_attention_gradient_by_differences():
    q, k, v, dO, dlse = _call()

    def loss():
        o, lse = O.prompt(q, k, v, CU_Q, CU_K, 0.7)
        return (o * dO).sum() + (np.where(np.isfinite(lse), lse, 0) * dlse).sum()

    grads = O.prompt_grad(q, k, v, CU_Q, CU_K, 0.7, dO, dlse)
    g = np.random.default_rng(1)
    for x, dx in zip((q, k, v), grads):
        for _ in range(40):
            at = tuple(g.integers(0, s) for s in x.shape)
            old, h = x[at], 1e-6
            x[at] = old + h
            hi = loss()
            x[at] = old - h
            lo = loss()
            x[at] = old
            assert abs((hi - lo) / (2 * h) - dx[at]) < 1e-8


def test_attention_gradient_closed_forms():
    """One visible key: its weight is 1 whatever the scores, so dq = dk = 0 and dv = dO.  Equal scores of two keys: P = 1/2
    each, dS = (dP_0 - dP_1) / 4 up to sign."""
    q, k, v, dO = (np.random.default_rng(i).standard_normal((1, 1, 4)) for i in range(4))
    dq, dk, dv = O.prompt_grad(q, k, v, [0, 1], [0, 1], 1.0, dO)
    assert not dq.any() and not dk.any() and np.array_equal(dv, dO)
    k2, v2 = np.concatenate([k, k]), np.concatenate([v, 2 * v])
    dq, dk, dv = O.prompt_grad(q, k2, v2, [0, 1], [0, 2], 1.0, dO)
    e = ((v - 2 * v) * dO).sum() / 4
    assert np.allclose(dv, dO / 2) and np.allclose(dk, e * np.concatenate([q, -q])) and np.allclose(dq, 0)


def test_the_dense_reference_is_the_oracle():
    q, k, v, dO, dlse = _call(3)
    t = [torch.from_numpy(x) for x in (q, k, v, dO, dlse)]
    o, lse, g, A = attention_grad(*t[:3], CU_Q, CU_K, 0.7, t[3], t[4])
    want_o, want_lse = O.prompt(q, k, v, CU_Q, CU_K, 0.7)
    assert np.allclose(o.numpy(), want_o) and np.allclose(lse.numpy(), want_lse)
    for x, y in zip(("dq", "dk", "dv"), O.prompt_grad(q, k, v, CU_Q, CU_K, 0.7, dO, dlse)):
        assert np.allclose(g[x].numpy(), y, atol=1e-12) and (np.abs(y) <= A[x].numpy() + 1e-12).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("eps", [None, 0.1])
def test_norm_gradient_by_differences(layout, eps):
    g = np.random.default_rng(2)
    x, w, dy = g.standard_normal((3, 2, 8)), g.standard_normal(8), g.standard_normal((3, 2, 8))
    a = g.uniform(0, 6, (5, 3))
    table, pos = np.stack([np.cos(a), np.sin(a)], -1), [4, 0, 2]
    loss = lambda: (O.norm_rope(x, w, eps, pos, table, layout) * dy).sum()  # noqa: E731
    dx, dw = O.norm_rope_grad(x, w, eps, pos, table, layout, dy)
    for t, dt in ((x, dx), (w, dw)):
        if dt is None:
            continue
        for at in np.ndindex(t.shape):
            old, h = t[at], 1e-6
            t[at] = old + h
            hi = loss()
            t[at] = old - h
            lo = loss()
            t[at] = old
            assert abs((hi - lo) / (2 * h) - dt[at]) < 1e-7


# ---------------------------------------------------------------- refusals
X = [(i + 1) << 32 for i in range(16)]  # addresses far apart


def _p(F, **kw):
    base = dict(B=2, Hq=8, Hkv=2, d=64, dtype=F.FALCON_BF16, tokens=10, k_tokens=10, max_q=10, rope_rows=128)
    base.update(kw)
    return F.AttnParams(**base)


def _grads(F, **kw):
    base = dict(dq=X[8], dk=X[9], dv=X[10])
    base.update(kw)
    return F.falcon_attn_grads_t(**base)


def _attn(F, p, g, q=X[0], k=X[1], v=X[2], cu_q=X[3], cu_k=X[4], o=X[5], lse=X[6], dO=X[7], dlse=None, ws=X[11],
          n=1 << 40):
    F.falcon_attn_prompt_backward(p, q, k, v, cu_q, cu_k, o, lse, dO, dlse, g, ws, n, 0)


def _norm(F, p, g, q=X[0], k=X[1], w_q=None, w_k=None, pos=X[2], table=X[3], gq=X[4], gk=X[5], dw_q=X[6], dw_k=X[7],
          ws=X[11], n=1 << 40):
    F.falcon_qk_norm_rope_backward(p, q, k, w_q, w_k, pos, table, gq, gk, g, dw_q, dw_k, ws, n, 0)


def _refused(F, code, call, *args, **kw):
    with pytest.raises(F.FalconError) as e:
        call(F, *args, **kw)
    assert e.value.code == code


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=0), -1), (dict(Hkv=3), -1), (dict(Hkv=0), -1), (dict(d=48), -2), (dict(d=256), -2), (dict(dtype=2), -1),
    (dict(tokens=-1), -1), (dict(max_q=-1), -1), (dict(q_stride=511), -1), (dict(k_stride=-1), -1),
    (dict(v_stride=127), -1), (dict(o_stride=8), -1)])
def test_bad_params(F, kw, code):
    p = _p(F, **kw)
    _refused(F, code, _attn, p, _grads(F))
    _refused(F, code, _norm, p, _grads(F))
    assert F.falcon_attn_prompt_backward_workspace_size(p) == 0 == F.falcon_qk_norm_rope_backward_workspace_size(p)


@pytest.mark.parametrize("kw", [dict(dq_stride=511), dict(dk_stride=127), dict(dv_stride=-1), dict(do_stride=500)])
def test_bad_strides_of_gradients(F, kw):
    _refused(F, -1, _attn, _p(F), _grads(F, **kw))
    _refused(F, -1, _norm, _p(F, rot=64, qk_norm=1), _grads(F, **kw))


def test_attention_pointers_and_scale(F):
    p, g = _p(F), _grads(F)
    for name in ("q", "k", "v", "cu_q", "cu_k", "o", "lse", "dO"):
        _refused(F, -1, _attn, p, g, **{name: None})
    for name in ("q", "k", "v", "o", "dO"):
        _refused(F, -1, _attn, p, g, **{name: X[12] + 1})
    for name in ("cu_q", "lse", "dlse"):
        _refused(F, -1, _attn, p, g, **{name: X[12] + 2})
    _refused(F, -1, _attn, p, None)
    for kw in (dict(dk=None), dict(dv=None), dict(dq=None, dk=None, dv=None), dict(dq=X[8] + 1)):
        _refused(F, -1, _attn, p, _grads(F, **kw))
    for s in (-1.0, math.nan, math.inf):
        _refused(F, -1, _attn, _p(F, scale=s), g)
    _refused(F, -1, _attn, _p(F, B=0), g)


def test_attention_overlaps(F):
    """No gradient over what the call reads, over another gradient or over the workspace; rows may lie between rows of
    one stride."""
    p, size = _p(F), 10 * 8 * 64 * 2
    for x in (X[0], X[1], X[2], X[5], X[7], X[6], X[11], X[0] + size - 2, X[10]):
        _refused(F, -1, _attn, p, _grads(F, dq=x))
    for x in (X[0], X[1], X[2], X[5], X[7], X[8], X[10], X[11]):
        _refused(F, -1, _attn, p, _grads(F, dk=x))
    for x in (X[0], X[1], X[2], X[5], X[7], X[6], X[12]):
        _refused(F, -1, _attn, p, _grads(F), ws=x, dlse=X[12])
    fused = dict(dq=X[8], dk=X[8] + 1024, dv=X[8] + 1024 + 256, dq_stride=768, dk_stride=768, dv_stride=768)
    _refused(F, -3, _attn, p, _grads(F, **fused), ws=None)  # slices of one gradient: only the workspace is missed
    for kw in (dict(dk=X[8] + 1022), dict(dv=X[8] + 1024 + 254), dict(dv_stride=1024)):
        _refused(F, -1, _attn, p, _grads(F, **{**fused, **kw}), ws=None)


def test_workspaces(F):
    p, g = _p(F), _grads(F)
    n = F.falcon_attn_prompt_backward_workspace_size(p)
    assert n > 0 and n % 256 == 0
    for ws, size in ((None, n), (X[11], n - 1), (X[11] + 16, n)):
        _refused(F, -3, _attn, p, g, ws=ws, n=size)
    p = _p(F, rot=64, qk_norm=1)
    n = F.falcon_qk_norm_rope_backward_workspace_size(p)
    assert n > 0 and n % 256 == 0
    for ws, size in ((None, n), (X[11], n - 1), (X[11] + 16, n)):
        _refused(F, -3, _norm, p, g, ws=ws, n=size)


@pytest.mark.parametrize("n", [2**31 - 1, 2**31 - 1023, 2**33])
def test_sequences_past_32_bits(F, n):
    far = [(i + 1) << 46 for i in range(12)]
    args = dict(q=far[0], k=far[1], v=far[2], o=far[3], lse=far[4], dO=far[5], ws=far[6])
    g = _grads(F, dq=far[7], dk=far[8], dv=far[9])
    _refused(F, -2, _attn, _p(F, tokens=n, max_q=2**31 - 1), g, **args)
    _refused(F, -2, _attn, _p(F, k_tokens=n), g, **args)
    assert F.falcon_attn_prompt_backward_workspace_size(_p(F, tokens=n)) == 0


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=66), dict(rot=-2), dict(rot=2, rope_layout=2),
                                dict(rot=2, rope_rows=0), dict(qk_norm=1, norm_eps=0.0),
                                dict(qk_norm=1, norm_eps=float("nan"))])
def test_norm_settings(F, kw):
    _refused(F, -1, _norm, _p(F, **kw), _grads(F))


def test_norm_pointers_and_overlaps(F):
    p, g = _p(F, rot=64, qk_norm=1), _grads(F)
    for kw in (dict(gq=None, gk=None), dict(q=None), dict(k=None), dict(pos=None), dict(table=None), dict(q=X[0] + 1),
               dict(gk=X[5] + 1), dict(dw_q=X[6] + 2), dict(w_k=X[12] + 2)):
        _refused(F, -1, _norm, p, g, **kw)
    _refused(F, -1, _norm, p, None)
    for kw in (dict(dq=None), dict(dk=None), dict(dq=X[0]), dict(dq=X[1]), dict(dk=X[0]), dict(dq=X[4] + 64),
               dict(dq=X[5]), dict(dk=X[4]), dict(dk=X[8]), dict(dq=X[6] - 8), dict(dq=X[11]),
               dict(dq=X[4], dq_stride=1024)):
        _refused(F, -1, _norm, p, _grads(F, **kw))
    for kw in (dict(dw_k=X[6]), dict(dw_q=X[0]), dict(dw_k=X[4]), dict(dw_q=X[11]), dict(w_q=X[6]), dict(w_k=X[6] + 8),
               dict(ws=X[0]), dict(ws=X[5]), dict(ws=X[8])):
        _refused(F, -1, _norm, p, g, **kw)


def test_empty_calls_do_nothing(F):
    p = _p(F, tokens=0, k_tokens=0)
    _attn(F, p, _grads(F, dq=None, dk=None, dv=None), q=None, k=None, v=None, cu_q=None, cu_k=None, o=None, lse=None,
          dO=None, ws=None, n=0)
    _norm(F, p, _grads(F, dq=None, dk=None), q=None, k=None, pos=None, table=None, gq=None, gk=None, dw_q=None, dw_k=None,
          ws=None, n=0)


def test_struct_matches_the_header(F):
    assert ctypes.sizeof(F.falcon_attn_grads_t) == 56
    t = torch.zeros((4, 6, 64))
    g = F.make_attn_grads({"dq": t[:, :2], "dk": t[:, 2:4], "dv": None}, 9)
    assert (g.dq, g.dk, g.dv) == (t.data_ptr(), t.data_ptr() + 512, None)
    assert (g.dq_stride, g.dk_stride, g.dv_stride, g.do_stride) == (384, 384, 0, 9)
    assert F.make_attn_grads(None) is None


def test_helpers_refuse_other_layouts(F):
    q, kv = torch.zeros((4, 8, 64)), torch.zeros((4, 2, 64))
    lse, cu = torch.zeros((4, 8)), torch.tensor([0, 4], dtype=torch.int32)
    ok = dict(q=q, k=kv, v=kv, o=q, lse=lse, dO=q, cu_q=cu)
    for kw in (dict(o=q[:3]), dict(dO=q.bfloat16()), dict(lse=lse[:, :4]), dict(lse=lse.double()), dict(dlse=lse.T),
               dict(k=kv.bfloat16()), dict(cu_q=cu.long()), dict(v=kv[:3]), dict(dO=q[:1].expand(4, 8, 64)),
               dict(dO=q.transpose(1, 2)), dict(out={"dx": q}), dict(out={"dq": q[:3]}), dict(out={"dq": q.bfloat16()}),
               dict(out={"dk": kv.transpose(0, 1)}), dict(q=q.half(), o=q.half(), dO=q.half(), k=kv.half(), v=kv.half())):
        with pytest.raises(ValueError):
            F.attn_prompt_backward(**{**ok, **kw})
    ok = dict(q=q, k=kv, dq_out=q, dk_out=kv)
    for kw in (dict(dk_out=None), dict(dq_out=q[:3]), dict(dk_out=kv.bfloat16()), dict(w_q=torch.zeros(3)),
               dict(table=torch.zeros((4, 32, 2))), dict(out={"dv": kv}), dict(out={"dq": q.half()}),
               dict(dk_out=torch.zeros((4, 3, 64))[:, :2])):
        with pytest.raises(ValueError):
            F.qk_norm_rope_backward(**{**ok, **kw})
