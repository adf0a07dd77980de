"""Softmax-attention operators without a GPU: the oracle's pins, the rotary
frequencies, and the refusals that the host gives before anything is
enqueued (the addresses handed in are never dereferenced)."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import softmax_attention as O


@pytest.fixture(scope="module")
def F():
    import __graft_entry__
    __graft_entry__.build()
    import chunked_delta_rule_gb300 as F
    return F


# ---------------------------------------------------------------- oracle pins
def test_e4m3_encode_matches_torch():
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(4000) * 10.0 ** g.uniform(-4, 2.5, 4000), O.E4M3[:127], -O.E4M3[:127],
                        (O.E4M3[:126] + O.E4M3[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_encode(x), want)
    assert np.array_equal(O.e4m3_encode([np.inf, -np.inf, 1e9, np.nan]), [0x7E, 0xFE, 0x7E, 0x7F])


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (224.0, -1), (1.0, -8), (0.0, -126), (1e-38, -126),
                                   (3e38, 120)])
def test_scale_exponent(top, e):
    assert O.scale_exponent(np.array([top, -top / 3, np.inf, np.nan])) == e


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_depends_on_distance_alone(layout):
    """<R(m) q, R(n) k> is a function of m - n, and rotation keeps the length."""
    g = np.random.default_rng(1)
    d, f = 16, 10000.0 ** (-np.arange(8) / 8)
    a = np.arange(64)[:, None] * f
    table = np.stack([np.cos(a), np.sin(a)], -1)
    q, k = g.standard_normal((1, 1, d)), g.standard_normal((1, 1, d))
    dot = lambda m, n: (O.norm_rope(q, None, None, [m], table, layout)  # noqa: E731
                        * O.norm_rope(k, None, None, [n], table, layout)).sum()
    assert abs(dot(5, 2) - dot(40, 37)) < 1e-12 and abs(dot(7, 7) - (q * k).sum()) < 1e-12


def test_attend_is_the_mean_for_equal_scores():
    v = np.random.default_rng(2).standard_normal((5, 1, 4))
    o, lse = O.attend(np.zeros((2, 1, 4)), np.ones((5, 1, 4)), v, np.array([[1, 1, 1, 0, 0], [0] * 5], bool), 1.0)
    assert np.allclose(o[0, 0], v[:3, 0].mean(0)) and abs(lse[0, 0] - math.log(3)) < 1e-12
    assert not o[1].any() and lse[1, 0] == -np.inf


# ---------------------------------------------------------------- frequencies
def test_rope_frequencies(F):
    f, m = F.rope_frequencies(64, 10000.0)
    assert m == 1.0 and f.dtype == torch.float64 and f[0] == 1.0 and f.numel() == 32
    lin, _ = F.rope_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin, f / 4)
    ntk, _ = F.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and torch.allclose(ntk[-1], f[-1] / 4)
    y, m = F.rope_frequencies(64, scaling="yarn", factor=4.0, original_len=2048)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-15
    assert y[0] == f[0] and torch.allclose(y[-1], f[-1] / 4) and (y <= f).all() and (y >= f / 4).all()
    assert F.rope_frequencies(0)[0].numel() == 0
    for kw in (dict(scaling="other"), dict(scaling="yarn", factor=2.0), dict(scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            F.rope_frequencies(64, **kw)


# ---------------------------------------------------------------- refusals
X = [(i + 1) << 32 for i in range(12)]  # addresses far apart


def _p(F, **kw):
    base = dict(B=2, Hq=8, Hkv=2, d=64, dtype=F.FALCON_BF16, tokens=10, k_tokens=10, max_q=10, max_k=100, page=64,
                num_pages=9, max_pages=4, rope_rows=128)
    base.update(kw)
    return F.AttnParams(**base)


def _refused(F, code, call, *args):
    with pytest.raises(F.FalconError) as e:
        call(*args)
    assert e.value.code == code


BAD = [(dict(Hq=0), -1), (dict(Hkv=3), -1), (dict(Hkv=0), -1), (dict(d=48), -2), (dict(d=256), -2), (dict(dtype=2), -1),
       (dict(tokens=-1), -1), (dict(max_q=-1), -1), (dict(q_stride=511), -1), (dict(k_stride=-1), -1),
       (dict(v_stride=127), -1), (dict(o_stride=8), -1)]


@pytest.mark.parametrize("kw,code", BAD)
def test_every_operator_refuses_bad_params(F, kw, code):
    p, cache = _p(F, **kw), dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    _refused(F, code, F.falcon_qk_norm_rope, p, X[0], X[1], None, None, None, None, X[2], X[3], 0)
    _refused(F, code, F.falcon_kv_append, p, X[0], X[1], None, None, X[2], X[3], X[8], cache, 0)
    _refused(F, code, F.falcon_attn_decode, p, X[0], cache, X[8], X[1], X[2], None, X[9], 1 << 30, 0)
    _refused(F, code, F.falcon_attn_prompt, p, X[0], X[1], X[2], X[3], X[4], X[5], None, X[9], 256, 0)
    assert F.falcon_attn_decode_workspace_size(p) == 0 and F.falcon_attn_prompt_workspace_size(p) == 0


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=66), dict(rot=-2), dict(rot=2, rope_layout=2),
                                dict(rot=2, rope_rows=0), dict(qk_norm=1, norm_eps=0.0),
                                dict(qk_norm=1, norm_eps=float("nan"))])
def test_norm_and_rotation_settings(F, kw):
    cache = dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    p = _p(F, **kw)
    _refused(F, -1, F.falcon_qk_norm_rope, p, X[0], X[1], None, None, X[8], X[9], X[2], X[3], 0)
    _refused(F, -1, F.falcon_kv_append, p, X[0], X[1], None, X[9], X[2], X[3], X[8], cache, 0)


def test_qk_norm_rope_pointers(F):
    call, p = F.falcon_qk_norm_rope, _p(F, rot=64)
    _refused(F, -1, call, p, None, None, None, None, X[0], X[1], X[2], X[3], 0)     # nothing to do it to
    _refused(F, -1, call, p, X[0], X[1], None, None, X[4], X[5], None, X[3], 0)     # no output
    _refused(F, -1, call, p, X[0], X[1], None, None, None, X[5], X[2], X[3], 0)     # no positions
    _refused(F, -1, call, p, X[0], X[1], None, None, X[4], None, X[2], X[3], 0)     # no table
    _refused(F, -1, call, p, X[0] + 1, X[1], None, None, X[4], X[5], X[2], X[3], 0)  # half an element
    _refused(F, -1, call, p, X[0], X[1], None, None, X[4], X[5], X[0] + 64, X[3], 0)  # partly over its input
    _refused(F, -1, call, p, X[0], X[1], None, None, X[4], X[5], X[2], X[2], 0)     # outputs over one another
    fused = _p(F, q_stride=1024)
    _refused(F, -1, call, fused, X[0], X[1], None, None, None, None, X[0], X[3], 0)  # in place, other stride


def test_rows_that_share_bytes_in_a_fused_projection(F):
    """Rows of 8 + 2 + 2 heads of 64 bf16, 2048 elements apart.  What starts inside another operand's row, or runs into
    the next one, is refused."""
    call, p = F.falcon_qk_norm_rope, _p(F, q_stride=2048, k_stride=2048, o_stride=2048)
    q, k = X[0], X[0] + 8 * 64 * 2
    for out in (q + 2, q + 511 * 2, k, k + 127 * 2, k - 511 * 2, q + 2048 * 2 - 2, q + 2048 * 2 * 9 - 1022):
        _refused(F, -1, call, p, q, k, None, None, None, None, out, X[3], 0)
    _refused(F, -1, call, p, q, k, None, None, None, None, q, q + 2048 * 2 * 9, 0)   # dense k_out over the last row of q
    _refused(F, -1, call, _p(F, q_stride=2048, k_stride=2048, o_stride=1024), q, k, None, None, None, None, q, X[3], 0)
    p = _p(F, q_stride=2048, k_stride=2048, v_stride=2048, o_stride=2048)
    v = k + 128 * 2
    for out in (q, k - 2, v + 64 * 2, q - 511 * 2, v + 127 * 2):
        _refused(F, -1, F.falcon_attn_prompt, p, q, k, v, X[3], X[4], out, None, X[9], 256, 0)
    # keys of another number of rows: their whole span
    p = _p(F, q_stride=2048, k_stride=2048, v_stride=2048, o_stride=2048, k_tokens=11)
    _refused(F, -1, F.falcon_attn_prompt, p, q, k, v, X[3], X[4], v + 128 * 2, None, X[9], 256, 0)


def test_results_over_the_cache_or_the_workspace(F):
    """Neither a result nor the workspace may lie over what the call reads or over one another."""
    p, cache = _p(F), dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    n, last = F.falcon_attn_decode_workspace_size(p), 9 * 2 * 64 * 64 - 2  # of the codes
    dec = lambda q, o, lse, ws: _refused(F, -1, F.falcon_attn_decode, p, q, cache, X[8], X[1], o, lse, ws, n, 0)  # noqa: E731
    for at in X[4:8] + [X[4] + last, X[5] + last - 2]:
        dec(X[0], at, None, X[9])
        dec(X[0], X[2], at & ~3, X[9])
    for at in X[4:8] + [X[4] + 256, X[0], X[2], X[3]]:
        dec(X[0], X[2], X[3], at)
    dec(X[0], X[2], X[0], X[9])      # lse over the queries
    prompt = lambda o, lse, ws: _refused(F, -1, F.falcon_attn_prompt, p, X[0], X[1], X[2], X[3], X[4], o, lse, ws,  # noqa: E731
                                         256, 0)
    for at in X[0:3] + [X[5], X[6], X[0] + 10 * 8 * 64 * 2 - 256]:
        prompt(X[5], X[6], at)


@pytest.mark.parametrize("kw,code", [(dict(page=48), -2), (dict(page=256), -2), (dict(B=0), -1), (dict(num_pages=0), -1),
                                     (dict(max_pages=-1), -1)])
def test_cache_settings(F, kw, code):
    p, cache = _p(F, **kw), dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    _refused(F, code, F.falcon_kv_append, p, X[0], X[1], None, None, X[2], X[3], X[8], cache, 0)
    _refused(F, code, F.falcon_attn_decode, p, X[0], cache, X[8], X[1], X[2], None, X[9], 1 << 30, 0)


def test_cache_pointers(F):
    p, cache = _p(F), dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    for bad in (dict(k=None), dict(v_scale=None), dict(k=X[4] + 8), dict(v=X[4])):
        c = {**cache, **bad}
        _refused(F, -1, F.falcon_kv_append, p, X[0], X[1], None, None, X[2], X[3], X[8], c, 0)
    _refused(F, -1, F.falcon_kv_append, p, X[4], X[1], None, None, X[2], X[3], X[8], cache, 0)   # k is the cache
    _refused(F, -1, F.falcon_kv_append, p, X[0], X[1], None, None, None, X[3], X[8], cache, 0)
    _refused(F, -1, F.falcon_kv_append, p, X[0], X[1], None, None, X[2], X[3], None, cache, 0)
    _refused(F, -1, F.falcon_attn_decode, p, X[0], None, X[8], X[1], X[2], None, X[9], 1 << 30, 0)
    _refused(F, -1, F.falcon_attn_decode, p, X[0], cache, X[8], None, X[2], None, X[9], 1 << 30, 0)


def test_attention_workspace_scale_and_overlap(F):
    p, cache = _p(F), dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    n = F.falcon_attn_decode_workspace_size(p)
    assert n > 0 and n % 256 == 0 and F.falcon_attn_prompt_workspace_size(p) % 256 == 0
    for ws, size in ((None, n), (X[9], n - 1), (X[9] + 16, n)):
        _refused(F, -3, F.falcon_attn_decode, p, X[0], cache, X[8], X[1], X[2], None, ws, size, 0)
    for ws, size in ((None, 256), (X[9], 255), (X[9] + 16, 256)):
        _refused(F, -3, F.falcon_attn_prompt, p, X[0], X[1], X[2], X[3], X[4], X[5], None, ws, size, 0)
    for s in (-1.0, float("nan"), float("inf")):
        q = _p(F, scale=s)
        _refused(F, -1, F.falcon_attn_decode, q, X[0], cache, X[8], X[1], X[2], None, X[9], n, 0)
        _refused(F, -1, F.falcon_attn_prompt, q, X[0], X[1], X[2], X[3], X[4], X[5], None, X[9], 256, 0)
    _refused(F, -1, F.falcon_attn_decode, p, X[0], cache, X[8], X[1], X[0], None, X[9], n, 0)  # o over q
    _refused(F, -1, F.falcon_attn_prompt, p, X[0], X[1], X[2], X[3], X[4], X[1], None, X[9], 256, 0)  # o over k
    _refused(F, -1, F.falcon_attn_prompt, p, X[0], X[1], X[2], X[3], X[4], X[5], X[5] + 64, X[9], 256, 0)  # lse over o
    _refused(F, -1, F.falcon_attn_prompt, p, X[0], None, X[2], X[3], X[4], X[5], None, X[9], 256, 0)


FAR = [(i + 1) << 46 for i in range(10)]


@pytest.mark.parametrize("n", [2**31 - 1, 2**31 - 1023, 2**33])
def test_sequences_past_32_bits(F, n):
    """Rows and keys are numbered in 32 bits, whole tiles of them: longer sequences are refused, also where the bound is
    2^31 - 1 and the tokens say the rest."""
    cache = dict(zip(("k", "v", "k_scale", "v_scale"), FAR[4:8]))
    p = _p(F, tokens=n, k_tokens=10, max_q=2**31 - 1)
    _refused(F, -2, F.falcon_attn_prompt, p, FAR[0], FAR[1], FAR[2], FAR[3], FAR[8], FAR[5], None, FAR[9], 256, 0)
    _refused(F, -2, F.falcon_kv_append, p, FAR[0], FAR[1], None, None, FAR[2], FAR[3], FAR[8], cache, 0)
    p = _p(F, tokens=10, k_tokens=n)
    _refused(F, -2, F.falcon_attn_prompt, p, FAR[0], FAR[1], FAR[2], FAR[3], FAR[8], FAR[5], None, FAR[9], 256, 0)
    for kw in (dict(max_k=2**31 - 1, max_pages=2**25), dict(B=1 << 22, max_k=2**31 - 1, max_pages=1 << 10)):
        p = _p(F, **kw)
        _refused(F, -2, F.falcon_attn_decode, p, FAR[0], cache, FAR[8], FAR[1], FAR[2], None, FAR[9], 1 << 40, 0)


def test_heads_past_32_bits(F):
    p, cache = _p(F, Hq=1 << 25, Hkv=1 << 25), dict(zip(("k", "v", "k_scale", "v_scale"), FAR[4:8]))
    _refused(F, -2, F.falcon_qk_norm_rope, p, FAR[0], FAR[1], None, None, None, None, FAR[2], FAR[3], 0)
    _refused(F, -2, F.falcon_attn_prompt, p, FAR[0], FAR[1], FAR[2], FAR[3], FAR[8], FAR[5], None, FAR[9], 256, 0)
    _refused(F, -2, F.falcon_attn_decode, p, FAR[0], cache, FAR[8], FAR[1], FAR[2], None, FAR[9], 1 << 40, 0)


def test_empty_calls_do_nothing(F):
    """No tokens: accepted without a pointer, nothing is enqueued."""
    p, cache = _p(F, tokens=0), dict(zip(("k", "v", "k_scale", "v_scale"), X[4:8]))
    F.falcon_qk_norm_rope(p, None, None, None, None, None, None, None, None, 0)
    F.falcon_kv_append(p, None, None, None, None, None, None, X[8], cache, 0)
    F.falcon_attn_prompt(p, None, None, None, None, None, None, None, None, 0, 0)


def test_helpers_refuse_other_layouts(F):
    q = torch.zeros((4, 8, 64))
    with pytest.raises(ValueError):  # a broadcast token axis
        F.qk_norm_rope(q[:1].expand(4, 8, 64), None)
    with pytest.raises(ValueError):  # heads that are not dense
        F.qk_norm_rope(q.transpose(0, 1), None)
    with pytest.raises(ValueError):
        F.qk_norm_rope(q.half(), None)
    with pytest.raises(ValueError):  # a table without positions
        F.qk_norm_rope(q, None, None, torch.zeros((4, 32, 2)))
    with pytest.raises(ValueError):
        F.attn_prompt(q, q.bfloat16(), q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        F.attn_prompt(q, q, q, torch.zeros(2, dtype=torch.int64))
    cache = F.empty_kv_cache(2, 8, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        F.attn_decode(q, cache, torch.zeros((3, 1), dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        F.kv_append({**cache, "k": cache["k"].transpose(1, 2)}, q, q, torch.zeros(2, dtype=torch.int32),
                    torch.zeros(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32), 4)
