"""Softmax-attention operators on the GPU against the fp64 oracle.

Tolerances follow from the number formats.  A bf16 result is rounded once (at
most 2^-8 of it).  Norm and rotation are some twenty fp32 roundings: 2^-19 of
the row's largest value.  Attention weights are rounded to 11 bits (decode) or
8 bits (prompt, bf16) before they multiply the values, an error of at most
2^-11 or 2^-8 of the largest value in the sequence; an fp32 result carries the
scores' fp32 sums, 2e-5 of it.  Scales, and codes of rows that are neither
normed nor rotated, are exact; other codes lie within half a step (and the
fp32 error) of the true value.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

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


def _rand(shape, dtype, seed, spread=False, fused=0):
    """N(0, 1) rows [tokens, H, d]; fused: a slice of rows that are `fused` heads wider."""
    g = torch.Generator().manual_seed(seed)
    n, H, d = shape
    x = torch.randn((n, H + fused, d), generator=g)
    if spread:
        x = x * (0.2 + 4.8 * torch.rand((n, 1, 1), generator=g))
    x = x.to(DT[dtype]).cuda()
    return x[:, fused:] if fused else x


def _table(F, rot, rows, **kw):
    f, m = F.rope_frequencies(rot, **kw)
    return F.rope_table(f, rows, m), f, m


def _layout(F, name):
    return F.FALCON_ROPE_HALF if name == "half" else F.FALCON_ROPE_INTERLEAVED


# ---------------------------------------------------------------- table
def test_rope_table(F):
    t, f, m = _table(F, 32, 200001, scaling="yarn", factor=4.0, original_len=4096)
    a = np.arange(200001)[:, None] * f.numpy()
    want = np.stack([np.cos(a), np.sin(a)], -1) * np.float32(m).astype(np.float64)
    assert np.abs(_np(t) - want).max() < 2.0 ** -22


# ---------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,layout,norm,fused", [
    (1, 1, 1, 16, 16, "half", True, 0), (7, 12, 4, 64, 64, "half", True, 0), (33, 5, 5, 64, 32, "interleaved", True, 3),
    (19, 16, 2, 128, 128, "half", True, 2), (9, 3, 1, 128, 6, "half", True, 0), (9, 3, 1, 32, 10, "interleaved", True, 1),
    (5, 8, 8, 128, 50, "half", False, 0), (300, 17, 1, 32, 32, "half", True, 0), (4, 2, 2, 64, 0, "half", True, 0),
])
def test_qk_norm_rope(F, dtype, n, Hq, Hkv, d, rot, layout, norm, fused):
    q, k = _rand((n, Hq, d), dtype, 1, True, fused), _rand((n, Hkv, d), dtype, 2, True, fused)
    g = torch.Generator().manual_seed(3)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g)).cuda(), (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    table = _table(F, rot, 5000)[0] if rot else None
    pos = torch.randint(0, 5000, (n,), generator=g)
    qo, ko = F.qk_norm_rope(q, k, pos.cuda() if rot else None, table, wq, wk, norm=norm, layout=_layout(F, layout))
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        want = O.norm_rope(_np(x), _np(w) if norm else None, 1e-6 if norm else None, pos.numpy(),
                           table.cpu().numpy() if rot else None, layout)
        tol = 2.0 ** -19 * np.abs(want).max(-1, keepdims=True) + (U * np.abs(want) if dtype == "bf16" else 0)
        assert (np.abs(_np(y) - want) <= tol).all()


def test_qk_norm_rope_odd_addresses_in_place_and_alone(F):
    """Rows off the 16-byte boundaries, results over their inputs, q alone, and weights left out."""
    buf = torch.randn(1 + 6 * 200, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    q = buf[1:].view(6, 200)[:, :192].view(6, 3, 64)  # a row every 200 elements, 2 bytes past a boundary
    table = _table(F, 64, 100)[0]
    pos = torch.tensor([0, 99, 5, 5, 1, 50])
    want = O.norm_rope(_np(q), None, 1e-6, pos.numpy(), table.cpu().numpy(), "half")
    got, none = F.qk_norm_rope(q, None, pos.cuda(), table)
    assert none is None
    p = F.AttnParams(Hq=3, Hkv=3, d=64, dtype=F.FALCON_BF16, tokens=6, q_stride=200, o_stride=200, qk_norm=1, rot=64,
                     rope_rows=100)
    before = buf.clone()
    F.falcon_qk_norm_rope(p, q, None, None, None, pos.cuda(), table, q, None)
    for y in (got, q):
        assert (np.abs(_np(y) - want) <= U * np.abs(want) + 2.0 ** -19 * np.abs(want).max(-1, keepdims=True)).all()
    gap = torch.ones(1201, dtype=torch.bool)
    gap[1:].view(6, 200)[:, :192] = False
    assert torch.equal(buf[gap.cuda()], before[gap.cuda()])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_outside_the_table_are_nan(F, layout):
    q = _rand((5, 2, 64), "f32", 5)
    table = _table(F, 32, 10)[0]
    pos = torch.tensor([-1, 0, 9, 10, 1 << 40]).cuda()
    y = F.qk_norm_rope(q, None, pos, table, layout=_layout(F, layout))[0].cpu()
    bad = torch.isnan(y[..., :32]).all(-1)
    assert bad.tolist() == [[True, True], [False] * 2, [False] * 2, [True] * 2, [True] * 2]
    assert torch.isfinite(y[..., 32:]).all() and torch.isfinite(y[1:3]).all()


# ---------------------------------------------------------------- append
def _paged(lens, page, extra, seed):
    """A block table (int32, -1 past the end) over pages in a random order."""
    cols = max(-(-max(lens) // page), 1)
    used = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(used) + extra)
    bt, at = np.full((len(lens), cols), -1, np.int32), 0
    for b, u in enumerate(used):
        bt[b, :u] = order[at:at + u]
        at += u
    return bt, sum(used) + extra


def _garbage_cache(pages, Hkv, page, d, seed):
    """Bytes of every kind (NaN codes among them), scales around 2^0."""
    g = np.random.default_rng(seed)
    c = {n: g.integers(0, 256, (pages, Hkv, page, d)).astype(np.uint8) for n in ("k", "v")}
    c.update({n + "_scale": g.integers(110, 130, (pages, Hkv)).astype(np.uint8) for n in ("k", "v")})
    return c


def _cuda(cache):
    return {n: torch.from_numpy(a.copy()).cuda() for n, a in cache.items()}


def _check_codes(got, scale, x, slack):
    """got codes are nearest to x / scale (up to `slack` of it where fp32 rounds the other way)."""
    v, y = O.E4M3[got], x / scale
    with np.errstate(invalid="ignore"):
        step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3, -9)
        ok = np.abs(v - np.clip(y, -448, 448)) <= step / 2 + slack * np.abs(y).max(-1, keepdims=True)
    assert ok.all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx,Hkv,d,page,fused", [
    ([1, 1, 1], [0, 15, 16], 3, 64, 16, 0), ([40, 0, 1, 17], [5, 3, 0, 31], 2, 128, 32, 2),
    ([130, 64], [63, 64], 1, 32, 64, 0), ([3, 300], [126, 1], 2, 16, 128, 1), ([257], [0], 4, 128, 128, 0),
])
def test_append_exact(F, dtype, new, ctx, Hkv, d, page, fused):
    """Rows as they are: every byte of the cache as the oracle's, old codes re-rounded where a scale grows."""
    n = sum(new)
    k, v = _rand((n, Hkv, d), dtype, 6, True, fused), _rand((n, Hkv, d), dtype, 7, True, fused)
    lens = [a + b for a, b in zip(new, ctx)]
    bt, pages = _paged(lens, page, 2, 8)
    cache = _garbage_cache(pages, Hkv, page, d, 9)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    dev = _cuda(cache)
    F.kv_append(dev, k, v, torch.from_numpy(cu).cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                torch.from_numpy(bt).cuda(), max(new))
    want = O.append(cache, _np(k), _np(v), cu, ctx, bt)
    for name in want:
        got = dev[name].cpu().numpy()
        if name in "kv":  # NaN codes that are rounded again may change their sign
            nan = (want[name] & 127) == 127
            assert (((got & 127) == 127) == nan).all()
            got = np.where(nan, want[name], got)
        assert np.array_equal(got, want[name]), name


@pytest.mark.parametrize("dtype,new,page,d,rot,layout", [
    ("bf16", [1, 1], 64, 64, 64, "half"), ("bf16", [100, 37], 64, 128, 64, "interleaved"),
    ("f32", [33, 9], 16, 64, 20, "half"), ("bf16", [70, 5], 32, 32, 32, "half"), ("f32", [3], 128, 128, 128, "half"),
])
def test_append_norm_and_rotation_on_the_way(F, dtype, new, page, d, rot, layout):
    n, ctx = sum(new), [37, 0][:len(new)]
    k, v = _rand((n, 2, d), dtype, 10, True), _rand((n, 2, d), dtype, 11)
    w = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(12))).cuda()
    lens = [a + b for a, b in zip(new, ctx)]
    bt, pages = _paged(lens, page, 1, 13)
    table = _table(F, rot, max(lens))[0]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    cache = _garbage_cache(pages, 2, page, d, 14)
    dev = _cuda(cache)
    F.kv_append(dev, k, v, torch.from_numpy(cu).cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                torch.from_numpy(bt).cuda(), max(new), table, w, norm=True, layout=_layout(F, layout))
    pos = np.concatenate([c + np.arange(m) for c, m in zip(ctx, new)])
    kr = O.norm_rope(_np(k), _np(w), 1e-6, pos, table.cpu().numpy(), layout)
    want = O.append(cache, kr, _np(v), cu, ctx, bt)
    assert np.array_equal(dev["v"].cpu().numpy()[want["v"] & 127 != 127], want["v"][want["v"] & 127 != 127])
    assert np.array_equal(dev["v_scale"].cpu().numpy(), want["v_scale"])
    assert np.array_equal(dev["k_scale"].cpu().numpy(), want["k_scale"])
    codes = dev["k"].cpu().numpy()
    for b in range(len(new)):
        for i in range(new[b]):
            t = ctx[b] + i
            pg = bt[b, t // page]
            s = 2.0 ** (want["k_scale"][pg].astype(np.float64) - 127)
            _check_codes(codes[pg, :, t % page], s[:, None], kr[cu[b] + i], 2.0 ** -19)


def test_append_in_steps_keeps_what_was_there(F):
    """Token by token: every value stays within its rounding at the page's final scale (re-rounding by powers of
    two only touches what falls below the normal range: at most the smallest step, 2^-10 of the scale, each time)."""
    T, Hkv, d, page = 40, 2, 64, 16
    k = (_rand((T, Hkv, d), "bf16", 15) * torch.logspace(-3, 2, T).view(T, 1, 1).cuda()).bfloat16()
    bt, pages = _paged([T], page, 0, 16)
    cache = F.empty_kv_cache(pages, Hkv, page, d)
    for t in range(T):
        F.kv_append(cache, k[t:t + 1], k[t:t + 1], torch.tensor([0, 1], dtype=torch.int32).cuda(),
                    torch.tensor([t], dtype=torch.int32).cuda(), torch.from_numpy(bt).cuda(), 1)
    x = _np(k)
    for name in ("k", "v"):
        c = {n: a.cpu().numpy() for n, a in cache.items()}
        val, ok = O.cached(c, name, bt[0], T)
        s = 2.0 ** (c[name + "_scale"][bt[0, np.arange(T) // page]].astype(np.float64) - 127)
        assert ok.all() and (np.abs(val - x) <= 2.0 ** -4 * np.abs(x) + 2 ** -9 * s[:, :, None]).all()


def test_append_infinities_nan_zeros_and_pages_that_do_not_exist(F):
    d, page = 64, 16
    k = torch.zeros((4, 1, d), dtype=torch.bfloat16)
    k[1, 0, :3] = torch.tensor([float("inf"), -float("inf"), float("nan")])
    k[1, 0, 3] = 448.0
    cu = np.array([0, 1, 2, 3, 4], np.int32)
    bt = np.array([[0, -1], [1, -1], [-1, -1], [7, 3]], np.int32)  # sequence 2 has no page, 3's first is outside
    cache = _garbage_cache(4, 1, page, d, 17)
    dev = _cuda(cache)
    F.kv_append(dev, k.cuda(), k.cuda(), torch.from_numpy(cu).cuda(), torch.zeros(4, dtype=torch.int32).cuda(),
                torch.from_numpy(bt).cuda(), 1)
    want = O.append(cache, _np(k), _np(k), cu, [0] * 4, bt)
    for name in want:
        assert np.array_equal(dev[name].cpu().numpy(), want[name])
    assert want["k_scale"][0, 0] == 1 and want["k"][1, 0, 0, :4].tolist() == [0x7E, 0xFE, 0x7F, 0x7E]
    # more tokens than max_q allows, and a table that is too narrow: those tokens are not stored
    dev2 = _cuda(cache)
    F.kv_append(dev2, k.cuda(), k.cuda(), torch.tensor([0, 4], dtype=torch.int32).cuda(),
                torch.tensor([page - 1], dtype=torch.int32).cuda(), torch.tensor([[2]], dtype=torch.int32).cuda(), 2)
    for name in ("k", "v"):
        got = dev2[name].cpu().numpy()
        assert np.array_equal(got[[0, 1, 3]], cache[name][[0, 1, 3]]) and not (got[2, 0, page - 1] & 127).any()


# ---------------------------------------------------------------- decode
def _decode_case(F, lens, Hq, Hkv, d, page, dtype, seed, fused=0):
    bt, pages = _paged(lens, page, 3, seed)
    g = np.random.default_rng(seed)
    cache = _garbage_cache(pages, Hkv, page, d, seed + 1)  # slots past a sequence's end keep any byte, NaN too
    for n in ("k", "v"):
        cache[n + "_scale"][:] = 255  # pages that nothing uses: a NaN scale
    for b, L in enumerate(lens):
        for c in range(-(-L // page)):
            m = min(page, L - c * page)
            for n in ("k", "v"):
                cache[n][bt[b, c], :, :m] = O.e4m3_encode(g.standard_normal((Hkv, m, d)) * 100)
                cache[n + "_scale"][bt[b, c]] = g.integers(118, 122, Hkv)
    return bt, cache, _rand((len(lens), Hq, d), dtype, seed, fused=fused)


def _check_attention(o, lse, want, want_lse, vmax, dtype, step):
    o, lse = _np(o), _np(lse)
    tol = (U * np.abs(want) + step * vmax) if dtype == "bf16" else 2e-5 * vmax
    assert (np.abs(o - want) <= tol).all(), np.abs(o - want).max()
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), none)
    assert (np.abs(lse[~none] - want_lse[~none]) <= 2e-5 * (4 + np.abs(want_lse[~none]))).all()
    assert not o[none].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [
    ([1], 1, 1, 64, 16), ([0, 1, 63, 64, 65], 12, 12, 64, 64), ([5, 129, 1, 16], 8, 2, 128, 16),
    ([200, 0, 333], 16, 1, 32, 32), ([100, 17], 6, 2, 16, 128), ([1025, 700, 3], 16, 4, 128, 64),
    ([127, 128, 129], 20, 1, 64, 128), ([2500], 3, 3, 128, 64), ([4099, 1], 10, 2, 64, 16), ([3000], 40, 1, 128, 32),
])
def test_decode(F, dtype, lens, Hq, Hkv, d, page):
    bt, cache, q = _decode_case(F, lens, Hq, Hkv, d, page, dtype, 20 + len(lens) + d)
    o, lse = F.attn_decode(q, _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           max(lens), want_lse=True)
    want, want_lse = O.decode(_np(q), cache, bt, lens, d ** -0.5)
    _check_attention(o, lse, want, want_lse, 448 * 2.0 ** (121 - 127), dtype, 2.0 ** -11)


@pytest.mark.parametrize("d,B,n", [(16, 96, 12800), (128, 48, 6400)])
def test_decode_fp32_error_does_not_grow_with_the_keys(F, d, B, n):
    """The tensor cores cut sums off: 2^-24 of a sum a step in the mean.  A score has d / 16 steps of two products, a
    tile's weighted values two; queries and weights in two halves lose 2^-22 each, and as much is left for the rest:
    2^-24 (d / 8 + 12), however many keys a warp sums over."""
    Hq, Hkv, page = 6, 2, 128
    g = torch.Generator().manual_seed(33)
    k, v = ((torch.randn((B * n // page, Hkv, page, d), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
            for _ in "kv")
    scale = torch.full((B * n // page, Hkv), 120, dtype=torch.uint8, device="cuda")
    q = _rand((B, Hq, d), "f32", 34)
    cache = {"k": k.view(torch.uint8), "v": v.view(torch.uint8), "k_scale": scale, "v_scale": scale.clone()}
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    o, _ = F.attn_decode(q, cache, table, torch.full((B,), n, dtype=torch.int32, device="cuda"), n, want_lse=True)
    # [B, Hkv, n, d] and, for a key head's queries, [B, Hkv, Hq / Hkv, d]
    kd, vd = (x.double().view(B, n // page, Hkv, page, d).transpose(1, 2).reshape(B, Hkv, n, d) / 128 for x in (k, v))
    w = (q.double().view(B, Hkv, -1, d) @ kd.transpose(2, 3) * d ** -0.5).softmax(-1)
    want = (w @ vd).view(B, Hq, d)
    assert ((o.double() - want).norm() / want.norm()).item() < (d / 8 + 12) * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,lens", [(16, [333, 500, 70]), (64, [600, 1300, 520]), (128, [333, 500, 70]),
                                    (128, [600, 1300, 520])])
@pytest.mark.parametrize("ratio", [8, 16, 20, 24, 32, 60])
def test_decode_value_scales_far_apart(F, dtype, d, lens, ratio):
    """One page whose values are 2^ratio larger: the first or the last of a sequence with next to no weight (30 nats
    down), or with its share of the weight and one dim alone.  Weights are known to 11 bits (bf16) and everything else to
    2e-5, relative to sum_j p_j |v_j| of the element itself: nothing is lost to another page's scale."""
    Hq, Hkv, page = 6, 2, 16
    bt, pages = _paged(lens, page, 0, 90)
    g = np.random.default_rng(90 + d)
    cache = {n: O.e4m3_encode(g.standard_normal((pages, Hkv, page, d)) * f) for n, f in (("k", 3.0), ("v", 100.0))}
    cache["k_scale"] = np.full((pages, Hkv), 125, np.uint8)
    cache["v_scale"] = g.integers(118, 122, (pages, Hkv)).astype(np.uint8)
    for b, c in ((0, 0), (1, (lens[1] - 1) // page), (2, 1)):
        at = bt[b, c]
        cache["v_scale"][at] = 120 + ratio
        if b < 2:
            cache["k"][at] = 0
            cache["k"][at, :, :, 0] = O.e4m3_encode(-240.0)
        else:
            cache["v"][at, :, :, 1:] = 0
    q = _rand((3, Hq, d), dtype, 91)
    q[:, :, 0] = 4.0
    o, lse = F.attn_decode(q, _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           max(lens), 0.125, want_lse=True)
    want, want_lse = O.decode(_np(q), cache, bt, lens, 0.125)
    size, _ = O.decode(_np(q), {**cache, "v": cache["v"] & 127}, bt, lens, 0.125)
    tol = (2e-5 + (2.0 ** -11 if dtype == "bf16" else 0.0)) * size + (U * np.abs(want) if dtype == "bf16" else 0.0)
    assert (np.abs(_np(o) - want) <= tol).all(), (np.abs(_np(o) - want) / size).max()
    assert (np.abs(_np(lse) - want_lse) <= 2e-5 * (4 + np.abs(want_lse))).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_decode_many_small_weights(F, dtype, d):
    """131071 keys 22 nats under a strong one (2^-31.7 each) carry 3.7e-5 of the weight and, with larger values, a
    percent of the result.  fp32: weights in two halves 2^-22, at most 24 sums in a row of 2^-24 each."""
    n, page, at = 131072, 128, 70001
    g = torch.Generator().manual_seed(92)
    k = torch.zeros((n // page, 1, page, d))
    v = 300.0 + 100.0 * torch.rand((n // page, 1, page, d), generator=g)
    k[at // page, 0, at % page, 0], v[at // page, 0, at % page] = 44.0, 1.0
    codes = {x: y.to(torch.float8_e4m3fn).cuda() for x, y in (("k", k), ("v", v))}
    cache = {x: y.view(torch.uint8) for x, y in codes.items()}
    cache.update({x + "_scale": torch.full((n // page, 1), 127, dtype=torch.uint8, device="cuda") for x in "kv"})
    q = torch.zeros((1, 2, d), dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 4.0
    o, lse = F.attn_decode(q, cache, torch.arange(n // page, dtype=torch.int32, device="cuda")[None],
                           torch.tensor([n], dtype=torch.int32).cuda(), n, 0.125, want_lse=True)
    s = codes["k"].double().view(n, d)[:, 0] * 0.5
    want = torch.softmax(s, 0) @ codes["v"].double().view(n, d)
    tol = want * (U + 2.0 ** -11 if dtype == "bf16" else 2.0 ** -19)
    assert ((o[0].double() - want).abs() <= tol).all(), ((o[0].double() - want) / want).abs().max().item()
    assert (lse.double() - torch.logsumexp(s, 0)).abs().max().item() < 2e-5 * 26


def test_decode_strides_scale_and_bounds(F):
    """q a slice of a wider projection, o inside wider rows, a scale of its own, lengths past max_len, a page that
    does not exist, no lse, a workspace of garbage."""
    lens = [90, 33]
    bt, cache, q = _decode_case(F, lens, 4, 2, 64, 16, "bf16", 31, fused=3)
    bt[0, 2], bt[1, 0] = -1, 1 << 20
    rows = torch.full((2, 4 * 64 + 24), 7.0, dtype=torch.bfloat16).cuda()
    p = F.AttnParams(B=2, Hq=4, Hkv=2, d=64, dtype=F.FALCON_BF16, max_k=80, page=16, num_pages=cache["k"].shape[0],
                     max_pages=bt.shape[1], q_stride=q.stride(0), o_stride=280, scale=0.05)
    ws = torch.full((F.falcon_attn_decode_workspace_size(p),), 255, dtype=torch.uint8).cuda()
    F.falcon_attn_decode(p, q, _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                         rows, None, ws)
    want, want_lse = O.decode(_np(q), cache, bt, [80, 33], 0.05)
    got = rows[:, :256].reshape(2, 4, 64)
    _check_attention(got, torch.from_numpy(want_lse), want, want_lse, 7.0, "bf16", 2.0 ** -11)
    assert (rows[:, 256:] == 7).all()


def test_decode_large_scores_and_outliers(F):
    """Scores in the thousands (one key takes all the weight) and queries of very different sizes."""
    lens, d = [300, 300], 64
    bt, cache, q = _decode_case(F, lens, 4, 2, d, 64, "bf16", 33)
    q = (q * torch.tensor([1e4, 1e-6, 300.0, 1e-30]).view(1, 4, 1).cuda()).bfloat16()
    o, lse = F.attn_decode(q, _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           300, want_lse=True)
    want, want_lse = O.decode(_np(q), cache, bt, lens, d ** -0.5)
    o, lse = _np(o), _np(lse)
    # a score of size s is known to about 2^-22 s, so the weights to that
    slack = 2.0 ** -20 * np.abs(want_lse)[..., None] * 7
    assert (np.abs(o - want) <= U * np.abs(want) + 2.0 ** -11 * 7 + slack).all()
    assert (np.abs(lse - want_lse) <= 2e-5 * (4 + np.abs(want_lse))).all()


def test_cache_past_32_bits(F):
    """Pages that lie more than 2^32 bytes into the cache."""
    Hkv, page, d = 4, 128, 128
    pages = (1 << 32) // (Hkv * page * d) + 40
    n, lens = 200, [200]
    cache = {x: torch.empty((pages, Hkv, page, d), dtype=torch.uint8, device="cuda") for x in ("k", "v")}
    cache.update({x + "_scale": torch.zeros((pages, Hkv), dtype=torch.uint8, device="cuda") for x in ("k", "v")})
    bt = torch.tensor([[pages - 1, pages - 30]], dtype=torch.int32).cuda()
    k, v, q = _rand((n, Hkv, d), "bf16", 35), _rand((n, Hkv, d), "bf16", 36), _rand((1, 8, d), "bf16", 37)
    F.kv_append(cache, k, v, torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                bt, n)
    o, lse = F.attn_decode(q, cache, bt, torch.tensor(lens, dtype=torch.int32).cuda(), n, want_lse=True)
    at = bt[0].long()
    small = {x: cache[x][at].cpu().numpy() for x in cache}
    want, want_lse = O.decode(_np(q), small, np.array([[0, 1]]), lens, d ** -0.5)
    _check_attention(o, lse, want, want_lse, 5.0, "bf16", 2.0 ** -11)


@pytest.mark.parametrize("n,d", [(300, 64), (2000, 128)])
def test_decode_reports_a_wait_that_ran_out(F, n, d):
    """A load that is held back: the bounded waits give up, the call says so once, the next one is clean (one CTA a
    row, and rows in shares)."""
    bt, cache, q = _decode_case(F, [n, n], 4, 2, d, 64, "bf16", 38)
    dev, bt, ln = _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor([n, n], dtype=torch.int32).cuda()
    good = F.attn_decode(q, dev, bt, ln, n)
    p = F.AttnParams(B=2, Hq=4, Hkv=2, d=d, dtype=F.FALCON_BF16, max_k=n, page=64, num_pages=dev["k"].shape[0],
                     max_pages=bt.shape[1])
    ws = F.alloc_workspace(F.falcon_attn_decode_workspace_size(p))
    o = torch.zeros_like(q)
    F.falcon_test_hooks(2_000_000, True)
    try:
        F.falcon_attn_decode(p, q, dev, bt, ln, o, None, ws)
        assert F.falcon_workspace_status(ws) == F.FALCON_ERR_TIMEOUT
        assert F.falcon_workspace_status(ws) == F.FALCON_OK
        F.falcon_attn_decode(p, q, dev, bt, ln, o, None, ws)
        assert F.falcon_workspace_status(ws) == F.FALCON_OK and torch.equal(o, good)
    finally:
        F.falcon_test_hooks(0, False)


@pytest.mark.parametrize("lens", [[0, 0, 0], [3000, 0, 1, 0, 700], [1] * 300, list(range(0, 4000, 37))])
def test_decode_shares_of_uneven_lengths(F, lens):
    """Lengths known on the device only: none at all, most of them empty, one key each, every length in steps."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    bt, pages = _paged([max(n, 1) for n in lens], page, 0, 39)
    cols = -(-4000 // page)
    bt = np.pad(bt, ((0, 0), (0, cols - bt.shape[1])), constant_values=-1)
    g = torch.Generator(device="cuda").manual_seed(39)
    cache = {n: (torch.randn((pages, Hkv, page, d), generator=g, device="cuda") * 100).clamp(-448, 448)
             .to(torch.float8_e4m3fn).view(torch.uint8) for n in ("k", "v")}
    cache.update({n + "_scale": torch.randint(118, 122, (pages, Hkv), generator=g, device="cuda").to(torch.uint8)
                  for n in ("k", "v")})
    q = _rand((len(lens), Hq, d), "bf16", 39)
    o, lse = F.attn_decode(q, cache, torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 4000,
                           want_lse=True)
    at = torch.from_numpy(bt).cuda().long().clamp(min=0)

    def keys(n):  # [B, T, Hkv, d] in 64 bits
        x = cache[n].view(torch.float8_e4m3fn).double() * torch.exp2(cache[n + "_scale"].double() - 127)[..., None, None]
        return x[at].transpose(2, 3).reshape(len(lens), -1, Hkv, d)

    k, v = keys("k").repeat_interleave(Hq // Hkv, 2), keys("v").repeat_interleave(Hq // Hkv, 2)
    s = torch.einsum("bhd,bthd->bht", q.double(), k) * d ** -0.5
    n = torch.tensor(lens).cuda()
    s.masked_fill_(torch.arange(s.shape[2]).cuda() >= n[:, None, None], -float("inf"))
    want_lse = torch.logsumexp(s, -1)
    want = torch.einsum("bht,bthd->bhd", torch.exp(s - torch.where(n[:, None] > 0, want_lse, 0.0)[..., None]), v)
    _check_attention(o, lse, _np(want), _np(want_lse), 448 * 2.0 ** (121 - 127), "bf16", 2.0 ** -11)


# ---------------------------------------------------------------- prompt
def _prompt_case(lq, lk, Hq, Hkv, d, dtype, seed, fused=0):
    cq, ck = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32), np.concatenate([[0], np.cumsum(lk)]).astype(np.int32)
    q = _rand((int(cq[-1]), Hq, d), dtype, seed, fused=fused)
    k, v = _rand((int(ck[-1]), Hkv, d), dtype, seed + 1, fused=fused), _rand((int(ck[-1]), Hkv, d), dtype, seed + 2, fused=fused)
    return q, k, v, cq, ck


def _prompt(F, q, k, v, cq, ck, max_q=0):
    return F.attn_prompt(q, k, v, torch.from_numpy(cq).cuda(), torch.from_numpy(ck).cuda(), max_q, want_lse=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,d,fused", [
    ([1], [1], 1, 1, 64, 0), ([5, 1, 130], [5, 1, 130], 4, 2, 64, 0), ([100, 0, 30], [100, 7, 30], 3, 1, 128, 1),
    ([40, 3], [10, 0], 4, 4, 64, 0), ([7, 64], [200, 300], 8, 2, 128, 2), ([127, 128, 129], [127, 128, 129], 2, 2, 64, 0),
    ([256, 257], [256, 257], 2, 1, 128, 0), ([33, 70], [33, 70], 6, 3, 32, 1), ([50], [50], 2, 2, 16, 0),
    ([300], [137], 2, 1, 128, 0), ([1, 1, 1], [500, 64, 129], 12, 4, 64, 0), ([513], [513], 5, 5, 64, 0),
])
def test_prompt(F, dtype, lq, lk, Hq, Hkv, d, fused):
    q, k, v, cq, ck = _prompt_case(lq, lk, Hq, Hkv, d, dtype, 40 + d, fused)
    o, lse = _prompt(F, q, k, v, cq, ck, max(lq))
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    _check_attention(o, lse, want, want_lse, max(1.0, v.abs().max().item() if v.numel() else 1.0), dtype, 1.25 * U)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_prompt_of_more_blocks_than_fit(F, d):
    """Far more blocks of queries than the GPU holds at a time, some without rows, some without a key."""
    rng = np.random.default_rng(46)
    lq = [int(n) for n in rng.integers(0, 400, 40)]
    lk = [max(0, n + (0, 150, -n, -30, 1)[i % 5]) for i, n in enumerate(lq)]
    q, k, v, cq, ck = _prompt_case(lq, lk, 12, 4, d, "bf16", 47, 1)
    o, lse = _prompt(F, q, k, v, cq, ck, 512)
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    _check_attention(o, lse, want, want_lse, max(1.0, v.abs().max().item()), "bf16", 1.25 * U)
    again, _ = _prompt(F, q, k, v, cq, ck, 512)
    assert torch.equal(o, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_infinities_and_nan_in_masked_places(F, dtype, d):
    """What a query does not see does not reach it: NaN and infinity in a later token of its own sequence, in the
    next sequence, and in the rows past the last one."""
    lq = [150, 70]
    q, k, v, cq, ck = _prompt_case(lq, lq, 2, 1, d, dtype, 50)
    clean = _prompt(F, q, k, v, cq, ck, 150)
    k2, v2 = k.clone(), v.clone()
    k2[145], v2[145] = float("nan"), float("inf")       # seen by the last five queries of the first sequence
    k2[150 + 60], v2[150 + 60] = float("inf"), float("nan")
    o, lse = _prompt(F, q, k2, v2, cq, ck, 150)
    unseen = torch.ones(220, dtype=torch.bool)
    unseen[145:150] = unseen[210:220] = False
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    _check_attention(o[unseen], lse[unseen], want[unseen], want_lse[unseen], 5.0, dtype, 1.25 * U)
    assert torch.isnan(o[~unseen].float()).all()
    assert torch.isfinite(clean[0].float()).all()


def test_prompt_large_scores(F):
    """Scores in the hundreds, growing along the keys: the running maximum moves at every tile."""
    n, d = 700, 64
    q, k, v, cq, ck = _prompt_case([n], [n], 2, 2, d, "bf16", 55)
    k = (k * torch.linspace(0, 30, n).view(n, 1, 1).cuda()).bfloat16()
    q = (q * 4).bfloat16()
    o, lse = _prompt(F, q, k, v, cq, ck)
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    slack = 2.0 ** -20 * np.abs(want_lse)[..., None] * 5
    assert (np.abs(_np(o) - want) <= U * np.abs(want) + 1.25 * U * 5 + slack).all()
    assert (np.abs(_np(lse) - want_lse) <= 2e-5 * (4 + np.abs(want_lse))).all()


def test_prompt_all_scores_minus_infinity_and_lowest(F):
    """Keys whose every score is minus infinity weigh nothing; scores at the type's lowest value weigh alike."""
    q, k, v, cq, ck = _prompt_case([40], [40], 1, 1, 64, "f32", 57)
    q[:], k[:] = 0.0, 0.0
    q[:, :, 0], k[:, :, 0] = 1.0, -float("inf")
    k[30:, :, 0] = -3e38
    o, lse = _prompt(F, q, k, v, cq, ck)
    assert not o[:30].any() and torch.isneginf(lse[:30]).all()
    want = torch.stack([v[30:31 + i, 0].mean(0) for i in range(10)])
    assert (o[30:, 0] - want).abs().max() < 1e-4


def test_prompt_odd_addresses_and_wide_rows(F):
    """Rows off the 16-byte boundaries, o inside wider rows, token strides past 2^31 elements."""
    n, Hq, d = 20, 2, 64
    q, k, v, cq, ck = _prompt_case([13, 7], [13, 7], Hq, 1, d, "bf16", 60)
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    odd = torch.empty(1 + n * 129, dtype=torch.bfloat16, device="cuda")[1:].view(n, 129)[:, :128].view(n, Hq, d)
    odd.copy_(q)
    o, lse = _prompt(F, odd, k, v, cq, ck)
    _check_attention(o, lse, want, want_lse, 5.0, "bf16", 1.25 * U)
    step = (1 << 31) // 16
    far = torch.empty(step * n, dtype=torch.bfloat16, device="cuda").view(n, step)
    kw, vw, ow = far[:, :64].view(n, 1, d), far[:, 64:128].view(n, 1, d), far[:, 128:256]
    kw.copy_(k)
    vw.copy_(v)
    p = F.AttnParams(B=2, Hq=Hq, Hkv=1, d=d, dtype=F.FALCON_BF16, max_q=13, tokens=n, k_tokens=n, k_stride=step,
                     v_stride=step)
    lse = torch.empty((n, Hq), device="cuda")
    res = torch.full((n, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    p.o_stride = 200
    F.falcon_attn_prompt(p, q, kw, vw, torch.from_numpy(cq).cuda(), torch.from_numpy(ck).cuda(), res, lse,
                         F.alloc_workspace(F.falcon_attn_prompt_workspace_size(p)))
    _check_attention(res[:, :128].reshape(n, Hq, d), lse, want, want_lse, 5.0, "bf16", 1.25 * U)
    assert (res[:, 128:] == 3).all()
    del far, kw, vw, ow


def test_prompt_more_rows_than_a_head_count_divides(F):
    """A prompt longer than several tiles of queries and keys, every head group, against fp64 on the GPU."""
    n, Hq, Hkv, d = 1500, 4, 2, 128
    q, k, v, cq, ck = _prompt_case([n], [n], Hq, Hkv, d, "bf16", 62)
    o, lse = _prompt(F, q, k, v, cq, ck)
    s = torch.einsum("ihd,jhd->hij", q.double(), k.double().repeat_interleave(2, 1)) * d ** -0.5
    s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v.double().repeat_interleave(2, 1))
    _check_attention(o, lse, _np(want), _np(torch.logsumexp(s, -1).T), 5.0, "bf16", 1.25 * U)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_reports_a_wait_that_ran_out(F, d):
    """A load that is held back: the bounded waits give up, the call says so once, the next one is clean."""
    q, k, v, cq, ck = _prompt_case([300, 20], [300, 20], 2, 1, d, "bf16", 63)
    cu = torch.from_numpy(cq).cuda()
    good, lse = _prompt(F, q, k, v, cq, ck)
    p = F.AttnParams(B=2, Hq=2, Hkv=1, d=d, dtype=F.FALCON_BF16, max_q=300, tokens=320, k_tokens=320)
    ws = F.alloc_workspace(F.falcon_attn_prompt_workspace_size(p))
    o = torch.zeros_like(q)
    F.falcon_test_hooks(2_000_000, True)
    try:
        F.falcon_attn_prompt(p, q, k, v, cu, cu, o, None, ws)
        assert F.falcon_workspace_status(ws) == F.FALCON_ERR_TIMEOUT
        assert F.falcon_workspace_status(ws) == F.FALCON_OK and not o.any()
        F.falcon_attn_prompt(p, q, k, v, cu, cu, o, None, ws)
        assert F.falcon_workspace_status(ws) == F.FALCON_OK and torch.equal(o, good)
    finally:
        F.falcon_test_hooks(0, False)


@pytest.mark.parametrize("d", [16, 64, 128])
def test_prompt_fp32_error_does_not_grow_with_the_keys(F, d):
    """The tensor cores cut sums off: 2^-24 of a sum a step in the mean.  A score has d / 8 steps, a tile's weighted
    values 8 steps of three products: 2^-24 (16 + 24) at most, also at 2000 keys."""
    n, H = 2000, 3
    q, k, v, cq, ck = _prompt_case([n], [n], H, H, d, "f32", 65)
    o, _ = _prompt(F, q, k, v, cq, ck)
    s = torch.einsum("ihd,jhd->hij", q.double(), k.double()) * d ** -0.5
    s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v.double())
    assert ((o.double() - want).norm() / want.norm()).item() < 40 * 2.0 ** -24


@pytest.mark.parametrize("dtype,n,d", [("f32", 70, 64), ("bf16", 20, 64), ("bf16", 300, 32), ("bf16", 300, 128)])
def test_prompt_clears_the_status_of_a_new_workspace(F, dtype, n, d):
    """Whatever the workspace held before: after a call whose waits all came back its status is clean."""
    q, k, v, cq, ck = _prompt_case([n], [n], 2, 1, d, dtype, 64)
    cu = torch.from_numpy(cq).cuda()
    p = F.AttnParams(B=1, Hq=2, Hkv=1, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, max_q=n,
                     tokens=n, k_tokens=n)
    ws = torch.full((F.falcon_attn_prompt_workspace_size(p),), 1, dtype=torch.uint8, device="cuda")
    F.falcon_attn_prompt(p, q, k, v, cu, cu, torch.empty_like(q), None, ws)
    assert F.falcon_workspace_status(ws) == F.FALCON_OK


@pytest.mark.parametrize("d", [16, 32])
def test_prompt_small_dims_infinities_and_nan_in_masked_places(F, d):
    test_prompt_infinities_and_nan_in_masked_places(F, "bf16", d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,d", [(64, 64), (64, 128), (16, 32)])
def test_no_bound_on_the_rows_of_a_sequence(F, dtype, Hq, d):
    """max_q is an upper bound, 2^31 - 1 none at all: the same bits as with the longest length (192 sequence-heads
    times the tiles of 2^31 rows is a number that wraps to a grid)."""
    lq = [3, 130, 70]
    q, k, v, cq, ck = _prompt_case(lq, lq, Hq, 2, d, dtype, 66)
    o, lse = _prompt(F, q, k, v, cq, ck, max(lq))
    for bound in (2**31 - 1, 2**31 - 64, 1 << 20, 203):
        o2, lse2 = _prompt(F, q, k, v, cq, ck, bound)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(3, 1, 64), (2, 2, 128), (4, 2, 16)])
def test_many_prompts_under_a_loose_bound(F, dtype, Hq, Hkv, d):
    """Blocks dealt out by the tokens instead of the bound: lengths around multiples of a block and of zero, fewer and
    more keys than queries, the same bits as with the longest length."""
    lq = [0, 1, 127, 128, 129, 0, 0, 255, 256, 257, 63, 64, 65, 300, 2, 0, 511, 512, 5] + [3] * 40 + [0]
    lk = [max(0, n + (0, 150, -n, -30, 1)[i % 5]) for i, n in enumerate(lq)]
    q, k, v, cq, ck = _prompt_case(lq, lk, Hq, Hkv, d, dtype, 65, 1)
    o, lse = _prompt(F, q, k, v, cq, ck, 512)
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    _check_attention(o, lse, want, want_lse, max(1.0, v.abs().max().item()), dtype, 1.25 * U)
    for bound in (0, 2**31 - 1, 2048):
        o2, lse2 = _prompt(F, q, k, v, cq, ck, bound)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_rows_computed_again_in_every_grid(F, dtype, d):
    """An infinity in one dim of each third prompt's second value: the rows that see it are infinite there and right
    elsewhere, those that do not see it are right (some of both are computed again), the same bits whichever way the
    blocks are dealt out."""
    lq = [2 + 37 * i % 300 for i in range(90)]
    q, k, v, cq, ck = _prompt_case(lq, lq, 6, 2, d, dtype, 67)
    clean, clean_lse = _prompt(F, q, k, v, cq, ck, max(lq))
    hit = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for b in range(0, 90, 3):
        v[cq[b] + 1, :, 3] = float("inf")
        hit[cq[b] + 1:cq[b + 1]] = True
    got = [_prompt(F, q, k, v, cq, ck, bound) for bound in (max(lq), 2**31 - 1)]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    o, lse = got[0]
    rest = [i for i in range(d) if i != 3]
    assert torch.isinf(o[hit][:, :, 3]).all()
    # two roundings of the same rows: weights to 8 bits (bf16) in one of them, results to 8 bits in both
    tol = (2 * U + 1.25 * U) * 5 if dtype == "bf16" else 2e-5 * 5
    assert (o[hit][:, :, rest].float() - clean[hit][:, :, rest].float()).abs().max() <= tol
    assert (o[~hit].float() - clean[~hit].float()).abs().max() <= tol
    assert (lse - clean_lse).abs().max() <= 2e-5 * 10


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_loose_bound_costs_little(F, dtype, d):
    """256 prompts of 128 tokens, the longest length left out: within three times the call with it (some 35 times where
    every sequence had the blocks of all tokens)."""
    n, B = 128, 256
    q, k, v, cq, _ = _prompt_case([n] * B, [n] * B, 12, 12, d, dtype, 66)
    cu = torch.from_numpy(cq).cuda()
    assert _prompt_ms(F, q, k, v, cu, 0) < 3 * _prompt_ms(F, q, k, v, cu, n)


def test_no_bound_on_the_tokens_appended(F):
    lens, B = [3, 40, 17] * 6, 18
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    bt, pages = _paged(lens, 16, 0, 67)
    bt, ctx = torch.from_numpy(bt).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    k, v = (_rand((sum(lens), 2, 64), "bf16", 68 + i) for i in range(2))
    caches = [F.empty_kv_cache(pages, 2, 16, 64) for _ in range(2)]
    for cache, bound in zip(caches, (40, 2**31 - 1)):
        F.kv_append(cache, k, v, cu, ctx, bt, bound)
    assert all(torch.equal(caches[0][n], caches[1][n]) for n in caches[0])


def test_no_bound_on_the_keys(F):
    lens = [700, 90]
    bt, cache, q = _decode_case(F, lens, 8, 2, 64, 64, "bf16", 69)
    dev, bt, ln = _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    got = [F.attn_decode(q, dev, bt, ln, n, want_lse=True) for n in (11 * 64, 2**31 - 1)]
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prompt_rows_computed_again_are_no_timeout(F, d):
    """An infinity in one dim of an early value sends every later row through the definition.  That takes longer than a
    wait may (3 ms here), which is no reason for the waits of the same block to run out."""
    n, H = 4096, 24 if d < 128 else 4
    q, k, v, cq, _ = _prompt_case([n], [n], H, 2, d, "bf16", 93)
    v[5, :, 3] = float("inf")
    cu, o = torch.from_numpy(cq).cuda(), torch.empty_like(q)
    p = F.AttnParams(B=1, Hq=H, Hkv=2, d=d, dtype=F.FALCON_BF16, max_q=n, tokens=n, k_tokens=n)
    ws = F.alloc_workspace(F.falcon_attn_prompt_workspace_size(p))
    F.falcon_test_hooks(3_000_000, False)
    try:
        F.falcon_attn_prompt(p, q, k, v, cu, cu, o, None, ws)
        assert F.falcon_workspace_status(ws) == F.FALCON_OK
    finally:
        F.falcon_test_hooks(0, False)
    assert torch.isinf(o[5:, :, 3]).all() and torch.isfinite(o[:5]).all()
    rest = [i for i in range(d) if i != 3]
    for h in (0, H - 1):
        s = q[:, h].double() @ k[:, h * 2 // H].double().T * d ** -0.5
        s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -float("inf"))
        want = s.softmax(-1) @ v[:, h * 2 // H, rest].double()
        assert ((o[:, h, rest].double() - want).abs() <= U * want.abs() + 1.25 * U * 5).all()


def _prompt_ms(F, q, k, v, cu, max_q=None):
    """The quicker of two calls after a first one."""
    ms = []
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        a.record()
        F.attn_prompt(q, k, v, cu, max_q=q.shape[0] if max_q is None else max_q)
        b.record()
        b.synchronize()
        ms.append(a.elapsed_time(b))
    return min(ms[1:])


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_walk_of_a_row_ends_at_nan(F, d):
    """An early key that is NaN makes every later row NaN: computing those again ends there, so the call takes a few
    times as long as a clean one, not the some 1000 times that walking over every key of every row does."""
    n, H = 4096, 12
    q, k, v, cq, _ = _prompt_case([n], [n], H, 2, d, "bf16", 95)
    cu = torch.from_numpy(cq).cuda()
    clean = _prompt_ms(F, q, k, v, cu)
    k[5] = float("nan")
    assert _prompt_ms(F, q, k, v, cu) < 50 * clean
    o = F.attn_prompt(q, k, v, cu, max_q=n)
    assert torch.isfinite(o[:5]).all() and torch.isnan(o[5:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_prompt_scores_that_jump(F, dtype, d):
    """Scores that pass what a row has seen before by 60 to 2000 nats, at the start of a tile and inside one, for some of
    the rows; values of 2^30 beside them."""
    n = 700
    q, k, v, cq, ck = _prompt_case([n], [n], 2, 1, d, dtype, 94)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    q[::3, :, 0] = 0.25
    for at, jump in ((128, 100.0), (200, 60.0), (384, 300.0), (500, 2000.0)):
        k[at, :, 0] = jump * d ** 0.5
    v[100:140] *= 2.0 ** 30
    o, lse = _prompt(F, q, k, v, cq, ck)
    want, want_lse = O.prompt(_np(q), _np(k), _np(v), cq, ck, d ** -0.5)
    size, _ = O.prompt(_np(q), _np(k), np.abs(_np(v)), cq, ck, d ** -0.5)
    # weights to 8 bits (bf16), scores of size s to 2^-20 s
    tol = U * np.abs(want) + (1.25 * U + 2.0 ** -20 * np.abs(want_lse)[..., None]) * size
    if dtype == "f32":
        tol = (2e-5 + 2.0 ** -20 * np.abs(want_lse)[..., None]) * size
    assert (np.abs(_np(o) - want) <= tol).all(), (np.abs(_np(o) - want) / size).max()
    assert (np.abs(_np(lse) - want_lse) <= 2e-5 * (4 + np.abs(want_lse))).all()


@pytest.mark.parametrize("d", [32, 64])
def test_prompt_finite_jump_costs_no_second_pass(F, d):
    """Scores that jump by 160 nats from one key on, seen by most rows: finite scores need no row computed again (which
    took some hundred times as long)."""
    n, H = 4096, 12
    q, k, v, cq, _ = _prompt_case([n], [n], H, 2, d, "bf16", 96)
    q[:, :, 0], k[:, :, 0] = 8.0, 0.0
    cu = torch.from_numpy(cq).cuda()
    clean = _prompt_ms(F, q, k, v, cu)
    k[200:, :, 0] = 20.0 * d ** 0.5
    assert _prompt_ms(F, q, k, v, cu) < 20 * clean


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place_in_a_fused_projection(F, dtype):
    """q is normed where it lies between k and v of its token; k goes elsewhere, k and v stay as they were."""
    n, Hq, Hkv, d = 37, 6, 2, 64
    x = _rand((n, Hq + 2 * Hkv, d), dtype, 97)
    before, (table, pos) = x.clone(), (_table(F, d, 64)[0], torch.arange(n).cuda())
    q, k, _ = torch.split(x, [Hq, Hkv, Hkv], dim=1)
    want = F.qk_norm_rope(q, k, pos, table)
    p = F.AttnParams(Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16 if dtype == "bf16" else F.FALCON_F32, tokens=n, qk_norm=1,
                     rot=d, rope_rows=64, q_stride=x.stride(0), k_stride=x.stride(0), o_stride=x.stride(0))
    ko = torch.empty((n, Hkv, d), dtype=x.dtype, device="cuda")
    F.falcon_qk_norm_rope(p, q, k, None, None, pos, table, q, ko)
    assert torch.equal(q, want[0]) and torch.equal(ko, want[1]) and torch.equal(x[:, Hq:], before[:, Hq:])


@pytest.mark.parametrize("n,d", [(300, 64), (300, 32), (70, 128), (10, 64)])
def test_prompt_output_in_a_fused_buffer(F, n, d):
    """o lies between the rows of q, k and v."""
    Hq, Hkv = 6, 2
    x = _rand((n, 2 * Hq + 2 * Hkv, d), "bf16", 98)
    before = x.clone()
    q, k, v, o = torch.split(x, [Hq, Hkv, Hkv, Hq], dim=1)
    cu, st = torch.tensor([0, n], dtype=torch.int32).cuda(), x.stride(0)
    want = F.attn_prompt(q, k, v, cu)
    p = F.AttnParams(B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=F.FALCON_BF16, max_q=n, tokens=n, k_tokens=n, q_stride=st,
                     k_stride=st, v_stride=st, o_stride=st)
    F.falcon_attn_prompt(p, q, k, v, cu, cu, o, None, F.alloc_workspace(F.falcon_attn_prompt_workspace_size(p)))
    assert torch.equal(o, want) and torch.equal(x[:, :Hq + 2 * Hkv], before[:, :Hq + 2 * Hkv])


def test_decode_output_beside_the_queries(F):
    lens = [90, 33, 0]
    bt, cache, q = _decode_case(F, lens, 4, 2, 64, 16, "bf16", 99)
    dev, bt, ln = _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    want = F.attn_decode(q, dev, bt, ln, 96)
    x = torch.cat([q, torch.zeros_like(q)], 1)
    p = F.AttnParams(B=3, Hq=4, Hkv=2, d=64, dtype=F.FALCON_BF16, max_k=96, page=16, num_pages=dev["k"].shape[0],
                     max_pages=bt.shape[1], q_stride=512, o_stride=512)
    F.falcon_attn_decode(p, x, dev, bt, ln, x[:, 4:], None, F.alloc_workspace(F.falcon_attn_decode_workspace_size(p)))
    assert torch.equal(x[:, 4:], want) and torch.equal(x[:, :4], q)


# ---------------------------------------------------------------- streams, repeats, the pieces together
def test_same_bits_again_and_on_another_stream(F):
    lens = [700, 90]
    bt, cache, q = _decode_case(F, lens, 8, 2, 64, 64, "bf16", 70)
    dev, bt, ln = _cuda(cache), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    a = F.attn_decode(q, dev, bt, ln, 700)
    x = _prompt_case([300, 41], [300, 41], 4, 2, 64, "bf16", 71)
    b = _prompt(F, *x)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a2 = F.attn_decode(q, dev, bt, ln, 700, stream=side)
    cu = torch.from_numpy(x[3]).cuda()
    side.wait_stream(torch.cuda.current_stream())
    b2 = F.attn_prompt(*x[:3], cu, stream=side)
    side.synchronize()
    assert torch.equal(a, a2) and torch.equal(b, b2)


def test_decode_step_in_a_graph(F):
    """One captured step (append, then attention), replayed with new inputs in place."""
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    bt, pages = _paged([64] * B, page, 0, 72)
    bt = torch.from_numpy(bt).cuda()
    caches = [F.empty_kv_cache(pages, Hkv, page, d) for _ in range(2)]
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    ctx = torch.zeros(B, dtype=torch.int32).cuda()
    q, k, v = (torch.zeros((B, H, d), dtype=torch.bfloat16).cuda() for H in (Hq, Hkv, Hkv))
    table = _table(F, d, 64)[0]

    def step(cache):
        F.kv_append(cache, k, v, cu, ctx, bt, 1, table, norm=True)
        return F.attn_decode(q, cache, bt, ctx + 1, 64)

    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(F.empty_kv_cache(pages, Hkv, page, d))
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        out = step(caches[0])
    for t in range(20):
        for x, i in ((q, 0), (k, 1), (v, 2)):
            x.copy_(_rand(tuple(x.shape), "bf16", 100 + 3 * t + i))
        ctx.fill_(t)
        g.replay()
        assert torch.equal(out, step(caches[1])), t


def test_prompt_then_tokens(F):
    """A layer's whole way: prompt, append, then tokens one by one; every token's output is that of a prompt run over
    all of it, up to the cache's 8 bits (2^-4 of a key or value)."""
    T, n0, Hq, Hkv, d, page = 80, 61, 4, 2, 64, 16
    q, k, v = (_rand((T, H, d), "bf16", 80 + i) for i, H in enumerate((Hq, Hkv, Hkv)))
    table, pos = _table(F, d, T)[0], torch.arange(T).cuda()
    qr, kr = F.qk_norm_rope(q, k, pos, table)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32).cuda()  # noqa: E731
    i32 = lambda n: torch.tensor([n], dtype=torch.int32).cuda()  # noqa: E731
    whole = F.attn_prompt(qr, kr, v, cu(T))
    bt, pages = _paged([T], page, 0, 84)
    bt, cache = torch.from_numpy(bt).cuda(), F.empty_kv_cache(pages, Hkv, page, d)
    first = F.attn_prompt(qr[:n0].contiguous(), kr[:n0].contiguous(), v[:n0].contiguous(), cu(n0))
    assert torch.equal(first, whole[:n0])
    F.kv_append(cache, kr[:n0].contiguous(), v[:n0].contiguous(), cu(n0), i32(0), bt, n0)
    err = []
    for t in range(n0, T):
        F.kv_append(cache, k[t:t + 1], v[t:t + 1], cu(1), i32(t), bt, 1, table, norm=True)
        qt = F.qk_norm_rope(q[t:t + 1], None, pos[t:t + 1], table)[0]
        o = F.attn_decode(qt, cache, bt, i32(t + 1), T)
        err.append((o - whole[t:t + 1]).float())
    rel = (torch.cat(err).square().mean() / whole[n0:].float().square().mean()).sqrt().item()
    assert rel < 2.0 ** -4, rel
