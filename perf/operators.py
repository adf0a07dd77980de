"""The measured cases of the softmax-attention operators: the per-head norm
with rotary positions, the append to the 8-bit paged cache, attention of one
token per sequence over that cache, and causal attention over packed prompts.

``own`` selects between the plain torch form and the library's entry points.
Head counts and dims are the library's usual ones (12 heads of 64, 16 of 128)
and their grouped forms.
"""

import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 256 sequences: queries and keys of the new tokens
        dict(name="norm_rope_step", op="norm_rope", tokens=256, Hq=12, Hkv=12, d=64, rot=64, layout="half",
             dtype="bf16", fused=False, maxpos=4096),
        # packed prompts in fp32, half of each head rotated in pairs, out of one fused projection
        dict(name="norm_rope_packed", op="norm_rope", tokens=9984, Hq=12, Hkv=4, d=64, rot=32,
             layout="interleaved", dtype="f32", fused=True, maxpos=2048),
        # two prompts of 16384 tokens, wide heads, out of one fused projection
        dict(name="norm_rope_long", op="norm_rope", tokens=32768, Hq=16, Hkv=4, d=128, rot=128, layout="half",
             dtype="bf16", fused=True, maxpos=16384),
        # one decode step: every sequence appends the key and value of one token (norm and rotation on the way)
        dict(name="append_step", op="append", B=256, new=1, spread=0.0, ctx=1500, Hkv=12, d=64, page=64, rot=64,
             layout="half", norm=True, dtype="bf16", fused=False),
        # ragged chunks of prompts that continue half-filled pages
        dict(name="append_ragged", op="append", B=8, new=1027, spread=0.9, ctx=333, Hkv=4, d=128, page=64, rot=64,
             layout="interleaved", norm=True, dtype="bf16", fused=True),
        # two whole prompts, keys already normed and rotated by the pass over the queries
        dict(name="append_long", op="append", B=2, new=16384, spread=0.0, ctx=0, Hkv=16, d=128, page=64, rot=0,
             layout="half", norm=False, dtype="bf16", fused=False),
        # one token of one short conversation: latency
        dict(name="decode_one", op="decode", B=1, len=777, spread=0.0, Hq=12, Hkv=12, d=64, page=64, dtype="bf16"),
        # 256 conversations of different lengths, four queries to a key
        dict(name="decode_batch", op="decode", B=256, len=2048, spread=0.8, Hq=16, Hkv=4, d=128, page=64,
             dtype="bf16"),
        # two very long documents, eight queries to a key
        dict(name="decode_long", op="decode", B=2, len=131072, spread=0.1, Hq=16, Hkv=2, d=128, page=64,
             dtype="bf16"),
        # short ragged prompts in fp32, one with more queries than keys
        dict(name="prompt_short", op="prompt", B=7, new=333, spread=0.95, ctx=-40, Hq=12, Hkv=4, d=64, dtype="f32",
             fused=False),
        # a training-length batch of the 12-head layer
        dict(name="prompt_batch", op="prompt", B=8, new=2048, spread=0.0, ctx=0, Hq=12, Hkv=12, d=64, dtype="bf16",
             fused=True),
        # a long document, wide grouped heads
        dict(name="prompt_long", op="prompt", B=1, new=16384, spread=0.0, ctx=0, Hq=16, Hkv=4, d=128, dtype="bf16",
             fused=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    Hq, Hkv = rng.choice([(12, 12), (12, 4), (16, 16), (16, 4), (16, 2), (8, 1), (6, 2)])
    d = rng.choice([64, 64, 128, 128, 32, 16])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rope = dict(rot=rng.choice([d, d // 2, d // 4]), layout=rng.choice(["half", "interleaved"]))
    spread = rng.choice([0.0, 0.3, 0.9])
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["norm_rope", "append", "decode", "prompt"])
    if op == "norm_rope":
        return dict(op=op, tokens=_logint(rng, 1, 32768), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype,
                    fused=rng.random() < 0.5, maxpos=_logint(rng, 256, 65536), **rope)
    if op == "append":
        if rng.random() < 0.2:
            rope["rot"] = 0
        return dict(op=op, B=_logint(rng, 1, 256), new=rng.choice([1, _logint(rng, 1, 16384)]), spread=spread,
                    ctx=rng.choice([0, _logint(rng, 1, 4096)]), Hkv=Hkv, d=d, page=page, norm=rng.random() < 0.7,
                    dtype=dtype, fused=rng.random() < 0.5, **rope)
    if op == "decode":
        return dict(op=op, B=_logint(rng, 1, 256), len=_logint(rng, 1, 131072), spread=spread, Hq=Hq, Hkv=Hkv, d=d,
                    page=page, dtype=dtype)
    return dict(op=op, B=_logint(rng, 1, 16), new=_logint(rng, 1, 16384 if dtype == "bf16" else 2048), spread=spread,
                ctx=rng.choice([0, 0, _logint(rng, 1, 1024), -16]), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype,
                fused=rng.random() < 0.5)


def _within(case):
    """No more than the largest listed case of the operator, and room for the plain form's score matrix."""
    top = [work(c) for c in listed() if c["op"] == case["op"]]
    w = work(case)
    if w["bytes"] > max(t["bytes"] for t in top) or w["flops"] > max(t["flops"] for t in top):
        return False
    if case["op"] == "prompt":
        lq, lk = _prompt_lens(case)
        return case["B"] * case["Hq"] * max(lq) * max(max(lk), 1) <= 16 * 16384 ** 2
    if case["op"] == "decode":
        return case["B"] * case["len"] * case["Hkv"] * case["d"] <= 256 * 2048 * 4 * 128
    return True


def draw(rng):
    while True:
        case = _draw(rng)
        if _within(case):
            return case


def _ragged(B, top, spread):
    """Lengths between (1 - spread) top and top, the first one top: the same for every seed, so that work() knows them."""
    return [max(1, int(round(top * (1.0 - spread * ((b * 0.6180339887) % 1.0))))) for b in range(B)]


def _prompt_lens(case):
    """Query and key lengths: ctx > 0 keys before the prompt, ctx < 0 fewer keys than queries (rows that see none)."""
    lq = _ragged(case["B"], case["new"], case["spread"])
    return lq, [max(0, n + case["ctx"]) for n in lq]


def _pairs(lq, lk):
    """Visible (query, key) pairs of a causal sequence aligned at its end."""
    n = min(lq, lk)
    return n * (n + 1) // 2 + n * (lk - n)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "norm_rope":
        rows = case["tokens"] * (case["Hq"] + case["Hkv"])
        table = min(case["tokens"], case["maxpos"]) * case["rot"] * 4
        return {"bytes": 2 * rows * d * e + 8 * case["tokens"] + table + 8 * d, "flops": 7 * rows * d}
    if case["op"] == "append":
        new = _ragged(case["B"], case["new"], case["spread"])
        n, P = sum(new), case["page"]
        touched = sum(-(-(case["ctx"] + x) // P) - case["ctx"] // P for x in new)
        table = max(new) * case["rot"] * 4
        return {"bytes": 2 * n * case["Hkv"] * d * (e + 1) + touched * (4 + 2 * case["Hkv"]) + table + 8 * case["B"],
                "flops": 8 * n * case["Hkv"] * d}
    if case["op"] == "decode":
        lens = _ragged(case["B"], case["len"], case["spread"])
        pages = sum(-(-x // case["page"]) for x in lens)
        return {"bytes": 2 * sum(lens) * case["Hkv"] * d + pages * (4 + 2 * case["Hkv"])
                + case["B"] * case["Hq"] * (2 * d * e + 4), "flops": 4 * sum(lens) * case["Hq"] * d}
    lq, lk = _prompt_lens(case)
    return {"bytes": sum(lq) * case["Hq"] * (2 * d * e + 4) + 2 * sum(lk) * case["Hkv"] * d * e,
            "flops": 4 * case["Hq"] * d * sum(_pairs(a, b) for a, b in zip(lq, lk))}


# ------------------------------------------------------------------ inputs
def _cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _table(rows, rot, g):
    """Rotary table [rows, rot / 2, 2] of (cos, sin), frequencies stretched fourfold for long contexts."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / max(rot, 1)) / 4.0
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _rows(n, H, d, dtype, g):
    """Projected rows: N(0, 1) with a scale of its own for each token."""
    x = torch.randn((n, H, d), generator=g, device=DEV)
    x *= 0.2 + 4.8 * torch.rand((n, 1, 1), generator=g, device=DEV)
    return x.to(DT[dtype])


def _heads(n, counts, d, dtype, fused, g):
    """One tensor per entry of counts, [n, heads, d]: slices of one projection, or each on its own."""
    x = _rows(n, sum(counts), d, dtype, g)
    parts = list(torch.split(x, counts, dim=1))
    return parts if fused else [p.contiguous() for p in parts]


def _quantise(x):
    """Codes and power-of-two scale bytes of pages x [..., page, d]."""
    m, e = torch.frexp(x.abs().amax((-1, -2)))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m > 0, e, -126).clamp(-126, 127)
    codes = torch.ldexp(x, -e[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _cache(pages, Hkv, page, d, g, scale):
    k = torch.randn((pages, Hkv, page, d), generator=g, device=DEV)
    v = torch.randn((pages, Hkv, page, d), generator=g, device=DEV)
    s = scale * (0.2 + 1.8 * torch.rand((pages, 1, 1, 1), generator=g, device=DEV))
    kc, ks = _quantise(k * scale)
    vc, vs = _quantise(v * s)
    return {"k": kc, "v": vc, "k_scale": ks, "v_scale": vs}


def _block_table(lens, page, max_pages, g):
    """Pages in a random order, -1 past each sequence's last page; and the pages of the cache."""
    used = torch.tensor([-(-n // page) for n in lens], device=DEV)
    total = int(used.sum()) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.cumsum(used, 0) - used
    col = torch.arange(max_pages, device=DEV)
    at = (first[:, None] + col).clamp(max=total - 1)
    return torch.where(col < used[:, None], order[at], torch.full_like(order[at], -1)).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, d, dt = case["op"], case["d"], case["dtype"]
    s = {"case": case}
    if op == "norm_rope":
        n = case["tokens"]
        s["q"], s["k"] = _heads(n, [case["Hq"], case["Hkv"], case["Hkv"]], d, dt, case["fused"], g)[:2]
        s["wq"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
        s["wk"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
        start = torch.randint(0, case["maxpos"], (1,), generator=g, device=DEV)
        s["pos"] = (start + torch.arange(n, device=DEV)) % case["maxpos"]
        s["table"] = _table(case["maxpos"], case["rot"], g)
        s["q_out"] = torch.empty((n, case["Hq"], d), dtype=DT[dt], device=DEV)
        s["k_out"] = torch.empty((n, case["Hkv"], d), dtype=DT[dt], device=DEV)
    elif op == "append":
        new, page = _ragged(case["B"], case["new"], case["spread"]), case["page"]
        lens = [case["ctx"] + n for n in new]
        s["max_pages"] = -(-max(lens) // page)
        s["k"], s["v"] = _heads(sum(new), [case["Hkv"], case["Hkv"]], d, dt, case["fused"], g)
        s["wk"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        s["table"] = _table(max(lens), case["rot"], g) if case["rot"] else None
        s["cu"] = _cumulative(new)
        s["ctx"] = torch.full((case["B"],), case["ctx"], dtype=torch.int32, device=DEV)
        s["blocks"], pages = _block_table(lens, page, s["max_pages"], g)
        # the tokens cached before are smaller than many of the new ones: scales of half-filled pages grow
        s["cache"] = _cache(pages, case["Hkv"], page, d, g, 0.5)
    elif op == "decode":
        lens, page = _ragged(case["B"], case["len"], case["spread"]), case["page"]
        s["max_pages"] = -(-max(lens) // page)
        s["q"] = torch.randn((case["B"], case["Hq"], d), generator=g, device=DEV).to(DT[dt])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["blocks"], pages = _block_table(lens, page, s["max_pages"], g)
        s["cache"] = _cache(pages, case["Hkv"], page, d, g, 1.0)
        s["o"] = torch.empty((case["B"], case["Hq"], d), dtype=DT[dt], device=DEV)
        s["lse"] = torch.empty((case["B"], case["Hq"]), device=DEV)
    else:
        lq, lk = _prompt_lens(case)
        s["max_q"], s["max_k"] = max(lq), max(lk)
        if case["fused"] and lq == lk:
            s["q"], s["k"], s["v"] = _heads(sum(lq), [case["Hq"], case["Hkv"], case["Hkv"]], d, dt, True, g)
        else:
            s["q"] = _heads(sum(lq), [case["Hq"]], d, dt, False, g)[0]
            s["k"], s["v"] = _heads(sum(lk), [case["Hkv"], case["Hkv"]], d, dt, case["fused"], g)
        for n in ("q", "k"):  # as the norm leaves them
            x = s[n].float()
            s[n].copy_(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt())
        s["cu_q"], s["cu_k"] = _cumulative(lq), _cumulative(lk)
        s["o"] = torch.empty((sum(lq), case["Hq"], d), dtype=DT[dt], device=DEV)
        s["lse"] = torch.empty((sum(lq), case["Hq"]), device=DEV)
    if own:  # the params and the workspace that a program keeps from call to call
        s["plan"] = _plan(s)
    return s


# ------------------------------------------------------------------ the library
def _plan(s):
    import chunked_delta_rule_gb300 as F
    c = s["case"]
    kw = dict(d=c["d"], dtype=F.FALCON_BF16 if c["dtype"] == "bf16" else F.FALCON_F32)
    if c["op"] in ("norm_rope", "append"):
        kw.update(rot=c["rot"], rope_rows=s["table"].shape[0] if s["table"] is not None else 0, norm_eps=EPS,
                  rope_layout=F.FALCON_ROPE_HALF if c["layout"] == "half" else F.FALCON_ROPE_INTERLEAVED)
    if c["op"] == "norm_rope":
        return F, F.AttnParams(Hq=c["Hq"], Hkv=c["Hkv"], tokens=c["tokens"], qk_norm=1, q_stride=s["q"].stride(0),
                               k_stride=s["k"].stride(0), **kw), None
    if c["op"] == "append":
        return F, F.AttnParams(B=c["B"], Hq=c["Hkv"], Hkv=c["Hkv"], tokens=s["k"].shape[0], max_q=c["new"],
                               page=c["page"], num_pages=s["cache"]["k"].shape[0], max_pages=s["max_pages"],
                               qk_norm=int(c["norm"]), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0),
                               **kw), None
    if c["op"] == "decode":
        p = F.AttnParams(B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], max_k=c["len"], page=c["page"],
                         num_pages=s["cache"]["k"].shape[0], max_pages=s["max_pages"], **kw)
        n = F.falcon_attn_decode_workspace_size(p)
    else:
        p = F.AttnParams(B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], max_q=s["max_q"], max_k=s["max_k"],
                         tokens=s["q"].shape[0], k_tokens=s["k"].shape[0], q_stride=s["q"].stride(0),
                         k_stride=s["k"].stride(0), v_stride=s["v"].stride(0), **kw)
        n = F.falcon_attn_prompt_workspace_size(p)
    return F, p, F.alloc_workspace(n, DEV)


def _run_own(s):
    F, p, ws = s["plan"]
    op = s["case"]["op"]
    if op == "norm_rope":
        F.falcon_qk_norm_rope(p, s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["table"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        F.falcon_kv_append(p, s["k"], s["v"], s["wk"], s["table"], s["cu"], s["ctx"], s["blocks"], s["cache"])
        return s["cache"]
    if op == "decode":
        F.falcon_attn_decode(p, s["q"], s["cache"], s["blocks"], s["lens"], s["o"], s["lse"], ws)
    else:
        F.falcon_attn_prompt(p, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["o"], s["lse"], ws)
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ plain forms
def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _rotate(x, pos, table, layout):
    """x [n, H, d] fp32; the first 2 * table.shape[1] dims rotated by the angles of the positions."""
    half = table.shape[1]
    c, s = table[pos][:, None].unbind(-1)
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        head = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        head = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([head, x[..., 2 * half:]], -1)


def _plain_append(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    row = torch.arange(k.shape[0], device=DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = s["ctx"].long()[seq] + row - s["cu"].long()[seq]
    if c["norm"]:
        k = _norm(k, s["wk"])
    if c["rot"]:
        k = _rotate(k, pos, s["table"], c["layout"])
    P, Hkv = c["page"], c["Hkv"]
    # the pages that each sequence writes: M columns of its table, the last one again where it writes fewer
    ctx, n = s["ctx"].long(), s["cu"].long().diff()
    first = ctx // P
    M = (P - 1 + c["new"] - 1) // P + 1
    col = torch.minimum(first[:, None] + torch.arange(M, device=DEV), ((ctx + n - 1) // P)[:, None])
    page = s["blocks"].long().gather(1, col)  # [B, M]
    at, slot = (seq, pos // P - first[seq]), pos % P
    start = torch.where(col == first[:, None], (ctx % P)[:, None], 0)  # first slot written
    kept = (torch.arange(P, device=DEV) < start[..., None])[:, :, None, :, None]
    again = (torch.arange(c["B"], device=DEV)[:, None], col - first[:, None])
    for x, name in ((k, "k"), (v, "v")):
        a = x.abs()
        a = torch.where(torch.isfinite(a), a, 0).amax(-1)
        amax = torch.zeros((c["B"] * M, Hkv), device=DEV)
        amax = amax.scatter_reduce(0, (at[0] * M + at[1])[:, None].expand(-1, Hkv), a, "amax")
        m, e = torch.frexp(amax.view(c["B"], M, Hkv)[again])
        e = torch.where(m <= 0.875, e - 9, e - 8)
        e = torch.where(m > 0, e, -126).clamp(-126, 127)
        scale, codes = s["cache"][name + "_scale"].view(torch.uint8), s["cache"][name].view(torch.uint8)
        old = scale[page].int() - 127
        e = torch.where((start == 0)[..., None], e, torch.maximum(e, old))
        before = codes[page]
        held = torch.ldexp(before.view(torch.float8_e4m3fn).float(), (old - e)[..., None, None])
        held = torch.where(kept, held.to(torch.float8_e4m3fn).view(torch.uint8), before)
        codes[page] = held
        new = torch.ldexp(x, -e[at][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[page[at], :, slot] = new
        scale[page] = (e + 127).to(torch.uint8)
    return s["cache"]


def _softmax_values(scores, seen, v):
    """exp(scores - max) v / sum over the seen keys, and log sum exp; rows that see nothing give 0 and -inf. Overwrites scores."""
    scores.masked_fill_(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = scores.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v)
    o = torch.where(l > 0, o / l, 0.0)
    return o, (m + l.log())[..., 0]


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, d, P = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    at = s["blocks"].long().clamp(min=0)

    def keys(name):  # [B, Hkv, T, d]
        x = s["cache"][name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
        x *= s["cache"][name + "_scale"].view(torch.uint8)[at].view(torch.float8_e8m0fnu).float()[..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, d)

    k, v = keys("k"), keys("v")
    seen = torch.arange(k.shape[2], device=DEV) < s["lens"][:, None]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    scores = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    o, lse = _softmax_values(scores, seen[:, None, None], v)
    return {"o": o.reshape(B, Hq, d).to(DT[c["dtype"]]), "lse": lse.reshape(B, Hq)}


def _plain_prompt(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq.diff(), ck.diff()
    iq, ik = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    padded = lambda x, first, i: x[(first[:, None] + i).clamp(max=x.shape[0] - 1)].float()  # noqa: E731
    q = padded(s["q"], cq[:-1], iq).view(B, -1, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    k = padded(s["k"], ck[:-1], ik).permute(0, 2, 1, 3)[:, :, None]
    v = padded(s["v"], ck[:-1], ik).permute(0, 2, 1, 3)[:, :, None]
    seen = (ik <= iq[:, None] + (lk - lq)[:, None, None]) & (ik < lk[:, None, None])  # [B, Tq, Tk]
    o, lse = _softmax_values(torch.matmul(q * d ** -0.5, k.transpose(-1, -2)), seen[:, None, None], v)
    row = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cq[1:], row, right=True)
    at = row - cq[seq]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, d)[seq, at]
    return {"o": o.to(DT[c["dtype"]]), "lse": lse.permute(0, 3, 1, 2).reshape(B, -1, Hq)[seq, at]}


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "norm_rope":
        dt = DT[c["dtype"]]
        q, k = _norm(state["q"].float(), state["wq"]), _norm(state["k"].float(), state["wk"])
        return {"q": _rotate(q, state["pos"], state["table"], c["layout"]).to(dt),
                "k": _rotate(k, state["pos"], state["table"], c["layout"]).to(dt)}
    return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[c["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_rows(x, w, pos, table, layout):
    """Norm, then the rotation as a complex product."""
    x = x.double()
    if w is not None:
        x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    if table is None:
        return x
    turn = torch.view_as_complex(table.double().contiguous())[pos].unsqueeze(1)
    r = 2 * table.shape[1]
    y = x.clone()
    if layout == "half":
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous()) * turn
        y[..., :r] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_exponent(top):
    m, e = torch.frexp(top.double() / 448.0)
    return torch.where(top > 0, e - (m == 0.5).int(), -126).clamp(-126, 127)


def _exact_append(s):
    """Values over the scale, before they are rounded to 8 bits."""
    c, P = s["case"], s["case"]["page"]
    out = {n: s["cache"][n].float().double() for n in ("k", "v")}
    exps = {n: s["cache"][n + "_scale"].view(torch.uint8).int() - 127 for n in ("k", "v")}
    cu, blocks = s["cu"].tolist(), s["blocks"].tolist()
    pos = torch.cat([torch.arange(c["ctx"], c["ctx"] + b - a, device=DEV) for a, b in zip(cu, cu[1:])])
    new = {"k": _exact_rows(s["k"], s["wk"], pos, s["table"], c["layout"]), "v": s["v"].double()}
    for b, (first, end) in enumerate(zip(cu, cu[1:])):
        t = c["ctx"]
        while first < end:
            slot, page = t % P, blocks[b][t // P]
            n = min(P - slot, end - first)
            for name in ("k", "v"):
                x = new[name][first:first + n].transpose(0, 1)  # [Hkv, n, d]
                e = _exact_exponent(x.abs().amax((1, 2)))
                if slot:
                    before = exps[name][page]
                    e = torch.maximum(e, before)
                    out[name][page, :, :slot] *= torch.exp2((before - e).double())[:, None, None]
                out[name][page, :, slot:slot + n] = x * torch.exp2(-e.double())[:, None, None]
                exps[name][page] = e
            first, t = first + n, t + n
    return {"k": out["k"], "v": out["v"], "k_scale": torch.exp2(exps["k"].double()),
            "v_scale": torch.exp2(exps["v"].double())}


def _exact_attend(q, k, v, seen):
    """One sequence: q [n, Hq, d], k and v [T, Hkv, d], seen [n, T], all in 64 bits."""
    n, Hq, d = q.shape
    o, lse = torch.zeros_like(q), torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    some = seen.any(1)
    if n == 0 or k.shape[0] == 0:
        return o, lse
    for h in range(Hq):
        j = h // (Hq // k.shape[1])
        x = (q[:, h] @ k[:, j].T / math.sqrt(d)).masked_fill(~seen, -math.inf)
        z = torch.logsumexp(x, 1)
        y = torch.exp(x - torch.where(some, z, 0.0)[:, None]) @ v[:, j]
        o[:, h], lse[:, h] = torch.where(some[:, None], y, 0.0), torch.where(some, z, -math.inf)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return {"q": _exact_rows(s["q"], s["wq"], s["pos"], s["table"], case["layout"]),
                "k": _exact_rows(s["k"], s["wk"], s["pos"], s["table"], case["layout"])}
    if op == "append":
        # a page at a time: over some thousand pages this takes too long
        return _exact_append(s) if case["B"] * (case["new"] // case["page"] + 1) <= 4096 else None
    got = []
    if op == "decode":
        for b, n in enumerate(s["lens"].tolist()):
            at = s["blocks"][b, :-(-n // case["page"])].long()
            kv = []
            for name in ("k", "v"):
                e = s["cache"][name + "_scale"].view(torch.uint8)[at].double() - 127
                x = s["cache"][name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float().double()
                kv.append((x * torch.exp2(e)[..., None, None]).transpose(1, 2).reshape(-1, case["Hkv"], case["d"])[:n])
            got.append(_exact_attend(s["q"][b:b + 1].double(), *kv, torch.ones((1, n), dtype=torch.bool, device=DEV)))
    else:
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for a, b, i, j in zip(cq, cq[1:], ck, ck[1:]):
            seen = torch.ones((b - a, j - i), dtype=torch.bool, device=DEV).tril((j - i) - (b - a))
            got.append(_exact_attend(s["q"][a:b].double(), s["k"][i:j].double(), s["v"][i:j].double(), seen))
    return {"o": torch.cat([x[0] for x in got]), "lse": torch.cat([x[1] for x in got])}
