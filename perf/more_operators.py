"""The measured cases of the softmax-attention layers' backward pass: the
gradient of causal attention over packed prompts, which forms the weights
again from the log sums that the forward kept, and the gradient of the per-head
norm with rotary positions (the rows' and the norm weights').

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
        # one short sequence of the 12-head layer: latency
        dict(name="attn_one", op="attn", B=1, new=77, spread=0.0, ctx=0, Hq=12, Hkv=12, d=64, dtype="bf16",
             fused=True, dlse=False),
        # short ragged sequences in fp32 with fewer keys than queries: their first rows see none
        dict(name="attn_short", op="attn", B=7, new=333, spread=0.95, ctx=-40, Hq=12, Hkv=4, d=64, dtype="f32",
             fused=False, dlse=True),
        # small shared heads, queries that continue 500 earlier keys (a truncated backward over segments)
        dict(name="attn_continued", op="attn", B=4, new=1001, spread=0.3, ctx=500, Hq=8, Hkv=1, d=32, dtype="bf16",
             fused=False, dlse=False),
        # a training batch in fp32, wide heads
        dict(name="attn_fp32", op="attn", B=2, new=1024, spread=0.0, ctx=0, Hq=16, Hkv=16, d=128, dtype="f32",
             fused=True, dlse=False),
        # a training-length batch of the 12-head layer
        dict(name="attn_batch", op="attn", B=8, new=2048, spread=0.0, ctx=0, Hq=12, Hkv=12, d=64, dtype="bf16",
             fused=True, dlse=False),
        # packed documents of different lengths, four queries to a key, the log sums used by the loss too
        dict(name="attn_packed", op="attn", B=12, new=2048, spread=0.9, ctx=0, Hq=16, Hkv=4, d=128, dtype="bf16",
             fused=False, dlse=True),
        # few key heads and one sequence: the keys alone do not fill the GPU
        dict(name="attn_shared", op="attn", B=1, new=3000, spread=0.0, ctx=0, Hq=16, Hkv=2, d=64, dtype="bf16",
             fused=True, dlse=False),
        # a long document, wide grouped heads
        dict(name="attn_long", op="attn", B=1, new=16384, spread=0.0, ctx=0, Hq=16, Hkv=4, d=128, dtype="bf16",
             fused=False, dlse=False),
        # the rows of one short sequence
        dict(name="norm_one", op="norm", tokens=77, Hq=12, Hkv=12, d=64, rot=64, layout="half", dtype="bf16",
             fused=True, norm=True, maxpos=2048),
        # packed sequences in fp32, half of each head rotated in pairs
        dict(name="norm_packed", op="norm", tokens=9984, Hq=12, Hkv=4, d=64, rot=32, layout="interleaved",
             dtype="f32", fused=True, norm=True, maxpos=2048),
        # rotation alone (a layer without the norm)
        dict(name="norm_rotated", op="norm", tokens=16384, Hq=12, Hkv=12, d=64, rot=64, layout="half", dtype="bf16",
             fused=False, norm=False, maxpos=2048),
        # two documents of 16384 tokens, wide heads, out of and into one fused projection
        dict(name="norm_long", op="norm", tokens=32768, Hq=16, Hkv=4, d=128, rot=128, layout="half", dtype="bf16",
             fused=True, norm=True, maxpos=16384),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    Hq, Hkv = rng.choice([(12, 12), (12, 4), (16, 16), (16, 4), (16, 2), (8, 1), (6, 2)])
    d = rng.choice([64, 64, 128, 128, 32, 16])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.4:
        return dict(op="norm", tokens=_logint(rng, 1, 32768), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                    fused=rng.random() < 0.5, norm=rng.random() < 0.8, maxpos=_logint(rng, 256, 65536))
    return dict(op="attn", B=_logint(rng, 1, 16), new=_logint(rng, 1, 16384 if dtype == "bf16" else 2048),
                spread=rng.choice([0.0, 0.3, 0.9]), ctx=rng.choice([0, 0, _logint(rng, 1, 1024), -16]), Hq=Hq,
                Hkv=Hkv, d=d, dtype=dtype, fused=rng.random() < 0.5, dlse=rng.random() < 0.3)


def _within(case):
    """No more than the largest listed case of the operator, and room for the plain form's score matrices."""
    top = [work(c) for c in listed() if c["op"] == case["op"]]
    w = work(case)
    if w["bytes"] > max(t["bytes"] for t in top) or w["flops"] > max(t["flops"] for t in top):
        return False
    if case["op"] == "attn":
        lq, lk = _lens(case)
        # with a key or two the queries' and keys' gradients are differences of equal numbers: nothing to compare
        return max(lk) >= 16 and case["B"] * case["Hq"] * max(lq) * max(lk) <= 16 * 16384 ** 2
    return True


def draw(rng):
    while True:
        case = _draw(rng)
        if _within(case):
            return case


def _ragged(B, top, spread):
    """Lengths between (1 - spread) top and top, the first one top: the same for every seed, so that work() knows them."""
    return [max(1, int(round(top * (1.0 - spread * ((b * 0.6180339887) % 1.0))))) for b in range(B)]


def _lens(case):
    """Query and key lengths: ctx > 0 keys before the queries, ctx < 0 fewer keys than queries (rows that see none)."""
    lq = _ragged(case["B"], case["new"], case["spread"])
    return lq, [max(0, n + case["ctx"]) for n in lq]


def _pairs(lq, lk):
    """Visible (query, key) pairs of a causal sequence aligned at its end."""
    n = min(lq, lk)
    return n * (n + 1) // 2 + n * (lk - n)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "norm":
        rows = case["tokens"] * (case["Hq"] + case["Hkv"])
        table = min(case["tokens"], case["maxpos"]) * case["rot"] * 4
        # with the norm: x and dy in, dx out, the weights and their gradients; without: dy in, dx out
        if not case["norm"]:
            return {"bytes": 2 * rows * d * e + 8 * case["tokens"] + table, "flops": 3 * rows * d}
        return {"bytes": 3 * rows * d * e + 8 * case["tokens"] + table + 16 * d, "flops": 13 * rows * d}
    lq, lk = _lens(case)
    # q, o, do in, dq out, the log sums (and their gradients); k, v in, dk, dv out
    sums = 8 if case["dlse"] else 4
    return {"bytes": sum(lq) * case["Hq"] * (4 * d * e + sums) + 4 * sum(lk) * case["Hkv"] * d * e,
            "flops": 10 * case["Hq"] * d * sum(_pairs(a, b) for a, b in zip(lq, lk))}


# ------------------------------------------------------------------ inputs
def _cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _table(rows, rot):
    """Rotary table [rows, rot / 2, 2] of (cos, sin), frequencies stretched fourfold for long contexts."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / max(rot, 1)) / 4.0
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _rows(n, H, d, dtype, g, spread=4.8):
    """Rows N(0, 1) with a scale of its own for each token."""
    x = torch.randn((n, H, d), generator=g, device=DEV)
    x *= 0.2 + spread * torch.rand((n, 1, 1), generator=g, device=DEV)
    return x.to(DT[dtype])


def _heads(x, counts, fused):
    """One tensor per entry of counts, [n, heads, d]: slices of x, or each on its own."""
    parts = list(torch.split(x, counts, dim=1))
    return parts if fused else [p.contiguous() for p in parts]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d, dt, Hq, Hkv = case["d"], case["dtype"], case["Hq"], case["Hkv"]
    s = {"case": case}
    empty = lambda n, H: torch.empty((n, H, d), dtype=DT[dt], device=DEV)  # noqa: E731
    if case["op"] == "norm":
        n = case["tokens"]
        counts = [Hq, Hkv, Hkv]
        s["q"], s["k"] = _heads(_rows(n, sum(counts), d, dt, g), counts, case["fused"])[:2]
        s["wq"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        s["wk"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        start = torch.randint(0, case["maxpos"], (1,), generator=g, device=DEV)
        s["pos"] = (start + torch.arange(n, device=DEV)) % case["maxpos"]
        s["table"] = _table(case["maxpos"], case["rot"])
        s["dq_out"], s["dk_out"] = _rows(n, Hq, d, dt, g, 1.0), _rows(n, Hkv, d, dt, g, 1.0)
        s["dq"], s["dk"] = _heads(empty(n, sum(counts)), counts, case["fused"])[:2]
        s["dwq"] = torch.empty(d, device=DEV) if case["norm"] else None
        s["dwk"] = torch.empty(d, device=DEV) if case["norm"] else None
    else:
        lq, lk = _lens(case)
        n, m = sum(lq), sum(lk)
        s["max_q"], s["max_k"] = max(lq), max(lk)
        s["cu_q"], s["cu_k"] = _cumulative(lq), _cumulative(lk)
        if case["fused"] and lq == lk:
            counts = [Hq, Hkv, Hkv]
            s["q"], s["k"], s["v"] = _heads(_rows(n, sum(counts), d, dt, g), counts, True)
            s["dq"], s["dk"], s["dv"] = _heads(empty(n, sum(counts)), counts, True)
        else:
            s["q"] = _rows(n, Hq, d, dt, g)
            s["k"], s["v"] = _heads(_rows(m, 2 * Hkv, d, dt, g), [Hkv, Hkv], case["fused"])
            s["dq"] = empty(n, Hq)
            s["dk"], s["dv"] = _heads(empty(m, 2 * Hkv), [Hkv, Hkv], case["fused"])
        for name in ("q", "k"):  # as the norm leaves them
            x = s[name].float()
            s[name].copy_(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt())
        s["do"] = _rows(n, Hq, d, dt, g, 1.0)
        s["dlse"] = torch.randn((n, Hq), generator=g, device=DEV) if case["dlse"] else None
        s["o"], s["lse"] = _forward(s)  # what the forward kept
    if own:  # the params, the outputs' addresses and the workspace that a program keeps from call to call
        s["plan"] = _plan(s)
    return s


# ------------------------------------------------------------------ the library
def _plan(s):
    import chunked_delta_rule_gb300 as F
    c = s["case"]
    kw = dict(Hq=c["Hq"], Hkv=c["Hkv"], d=c["d"], dtype=F.FALCON_BF16 if c["dtype"] == "bf16" else F.FALCON_F32,
              q_stride=s["q"].stride(0), k_stride=s["k"].stride(0))
    if c["op"] == "norm":
        p = F.AttnParams(tokens=c["tokens"], qk_norm=int(c["norm"]), rot=c["rot"], rope_rows=s["table"].shape[0],
                         norm_eps=EPS, **kw,
                         rope_layout=F.FALCON_ROPE_HALF if c["layout"] == "half" else F.FALCON_ROPE_INTERLEAVED)
        grads = F.make_attn_grads({"dq": s["dq"], "dk": s["dk"]})
        size = F.falcon_qk_norm_rope_backward_workspace_size(p)
    else:
        p = F.AttnParams(B=c["B"], max_q=s["max_q"], tokens=s["q"].shape[0], k_tokens=s["k"].shape[0],
                         v_stride=s["v"].stride(0), **kw)
        grads = F.make_attn_grads({"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]})
        size = F.falcon_attn_prompt_backward_workspace_size(p)
    return F, p, grads, F.alloc_workspace(size, DEV)


def _run_own(s):
    F, p, grads, ws = s["plan"]
    if s["case"]["op"] == "norm":
        F.falcon_qk_norm_rope_backward(p, s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["table"], s["dq_out"],
                                       s["dk_out"], grads, s["dwq"], s["dwk"], ws)
        return {"dq": s["dq"], "dk": s["dk"], "dw_q": s["dwq"], "dw_k": s["dwk"]}
    F.falcon_attn_prompt_backward(p, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["o"], s["lse"], s["do"],
                                  s["dlse"], grads, ws)
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


# ------------------------------------------------------------------ plain forms
class _Padded:
    """The packed rows of a call as padded batches, and back; which keys a query sees."""

    def __init__(self, s):
        c = s["case"]
        self.B, self.Hq, self.Hkv, self.d = c["B"], c["Hq"], c["Hkv"], c["d"]
        cq, ck = s["cu_q"].long(), s["cu_k"].long()
        lq, lk = cq.diff(), ck.diff()
        iq, ik = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
        self.at_q, self.at_k = self._places(cq, iq, s["q"]), self._places(ck, ik, s["k"])
        self.back_q, self.back_k = self._back(cq, s["q"]), self._back(ck, s["k"])
        see = (ik <= iq[:, None] + (lk - lq)[:, None, None]) & (ik < lk[:, None, None]) & (iq < lq[:, None])[..., None]
        self.unseen = ~see[:, None, None]  # [B, 1, 1, Tq, Tk]

    @staticmethod
    def _places(cu, i, x):
        return (cu[:-1, None] + i).clamp(max=max(x.shape[0] - 1, 0))

    @staticmethod
    def _back(cu, x):
        row = torch.arange(x.shape[0], device=DEV)
        seq = torch.searchsorted(cu[1:], row, right=True)
        return seq, row - cu[seq]

    def queries(self, x):  # [n, Hq, d] -> [B, Hkv, G, Tq, d] fp32
        return x[self.at_q].float().view(self.B, -1, self.Hkv, self.Hq // self.Hkv, self.d).permute(0, 2, 3, 1, 4)

    def rows(self, x):  # [n, Hq] -> [B, Hkv, G, Tq, 1]
        return x[self.at_q].view(self.B, -1, self.Hkv, self.Hq // self.Hkv, 1).permute(0, 2, 3, 1, 4)

    def keys(self, x):  # [m, Hkv, d] -> [B, Hkv, 1, Tk, d] fp32
        return x[self.at_k].float().permute(0, 2, 1, 3)[:, :, None]

    def packed_queries(self, x):
        return x.permute(0, 3, 1, 2, 4).reshape(self.B, -1, self.Hq, x.shape[-1])[self.back_q]

    def packed_keys(self, x):  # [B, Hkv, Tk, d]
        return x.permute(0, 2, 1, 3)[self.back_k]


def _scores(s, pad):
    scores = torch.matmul(pad.queries(s["q"]) * s["case"]["d"] ** -0.5, pad.keys(s["k"]).transpose(-1, -2))
    return scores.masked_fill_(pad.unseen, -math.inf)


def _forward(s):
    """o and the log sums of the forward; rows that see no key give 0 and -inf."""
    dt = DT[s["case"]["dtype"]]
    if s["k"].shape[0] == 0:
        return torch.zeros_like(s["q"]), torch.full(s["q"].shape[:2], -math.inf, device=DEV)
    pad = _Padded(s)
    p = _scores(s, pad)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, torch.matmul(p, pad.keys(s["v"])) / total, 0.0)
    return pad.packed_queries(o).to(dt), pad.packed_queries(m + total.log())[..., 0].contiguous()


def _plain_attention(s):
    c = s["case"]
    dt, scale = DT[c["dtype"]], c["d"] ** -0.5
    if s["k"].shape[0] == 0:
        return {"dq": torch.zeros_like(s["q"]), "dk": torch.zeros_like(s["k"]), "dv": torch.zeros_like(s["v"])}
    pad = _Padded(s)
    lse = pad.rows(s["lse"])
    p = _scores(s, pad)
    p.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    do = pad.queries(s["do"])
    delta = (do * pad.queries(s["o"])).sum(-1, keepdim=True)
    if s["dlse"] is not None:
        delta = delta - pad.rows(s["dlse"])
    # the queries of all heads of a group beside one another: their sum is the product's own
    flat = lambda x: x.flatten(2, 3)  # noqa: E731
    dv = torch.matmul(flat(p).transpose(-1, -2), flat(do))
    p.mul_(torch.matmul(do, pad.keys(s["v"]).transpose(-1, -2)).sub_(delta))
    dq = torch.matmul(p, pad.keys(s["k"])) * scale
    dk = torch.matmul(flat(p).transpose(-1, -2), flat(pad.queries(s["q"]))) * scale
    return {"dq": pad.packed_queries(dq).to(dt), "dk": pad.packed_keys(dk).to(dt), "dv": pad.packed_keys(dv).to(dt)}


def _unrotate(g, pos, table, layout):
    """g [n, H, d] fp32 turned back by the angles of the positions."""
    half = table.shape[1]
    c, s = table[pos][:, None].unbind(-1)
    if layout == "half":
        a, b = g[..., :half], g[..., half:2 * half]
        head = torch.cat([a * c + b * s, b * c - a * s], -1)
    else:
        a, b = g[..., 0:2 * half:2], g[..., 1:2 * half:2]
        head = torch.stack([a * c + b * s, b * c - a * s], -1).flatten(-2)
    return torch.cat([head, g[..., 2 * half:]], -1)


def _plain_rows(s, x, dy, w):
    c = s["case"]
    g = _unrotate(dy.float(), s["pos"], s["table"], c["layout"])
    if not c["norm"]:
        return g.to(dy.dtype), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * r
    dw = (g * x).sum((0, 1))
    g = g * w
    return (r * (g - x * (g * x).mean(-1, keepdim=True))).to(dy.dtype), dw


def run(state):
    if own:
        return _run_own(state)
    if state["case"]["op"] == "attn":
        return _plain_attention(state)
    dq, dwq = _plain_rows(state, state["q"], state["dq_out"], state["wq"])
    dk, dwk = _plain_rows(state, state["k"], state["dk_out"], state["wk"])
    return {"dq": dq, "dk": dk, "dw_q": dwq, "dw_k": dwk}


# ------------------------------------------------------------------ 64 bits
def _exact_sequence(q, k, v, do, dlse):
    """One sequence: the softmax and its derivative in full, a head at a time; q, do [n, Hq, d], k, v [T, Hkv, d]."""
    n, Hq, d = q.shape
    T, Hkv = k.shape[:2]
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in (q, k, v))
    if n == 0 or T == 0:
        return dq, dk, dv
    hidden = torch.ones((n, T), dtype=torch.bool, device=DEV).triu(T - n + 1)
    for h in range(Hq):
        j = h // (Hq // Hkv)
        qh, kj, vj, g = q[:, h].double(), k[:, j].double(), v[:, j].double(), do[:, h].double()
        p = ((qh @ kj.T) / math.sqrt(d)).masked_fill_(hidden, -math.inf)
        p = torch.softmax(p, 1).nan_to_num_(0.0)  # rows that see nothing have no weights
        dv[:, j] += p.T @ g
        t = g @ vj.T
        t -= (p * t).sum(1, keepdim=True)
        if dlse is not None:
            t += dlse[:, h, None].double()
        t *= p
        dq[:, h] = (t @ kj) / math.sqrt(d)
        dk[:, j] += (t.T @ qh) / math.sqrt(d)
    return dq, dk, dv


def _exact_rows(s, x, dy, w):
    """The rotation's inverse as a complex product; the norm's derivative through y = w x / |x|_rms."""
    c = s["case"]
    g = dy.double().clone()
    turn = torch.view_as_complex(s["table"].double().contiguous())[s["pos"]].unsqueeze(1).conj()
    r = 2 * s["table"].shape[1]
    if c["layout"] == "half":
        z = torch.complex(g[..., :r // 2].contiguous(), g[..., r // 2:r].contiguous()) * turn
        g[..., :r // 2], g[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.view_as_complex(g[..., :r].reshape(*g.shape[:-1], r // 2, 2).contiguous()) * turn
        g[..., :r] = torch.view_as_real(z).flatten(-2)
    if not c["norm"]:
        return g, None
    x, w = x.double(), w.double()
    rms = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    dw = torch.einsum("nhd,nhd->d", g, x / rms)
    dx = g * w / rms - x * (g * w * x).sum(-1, keepdim=True) / (x.shape[-1] * rms ** 3)
    return dx, dw


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        dq, dwq = _exact_rows(s, s["q"], s["dq_out"], s["wq"])
        dk, dwk = _exact_rows(s, s["k"], s["dk_out"], s["wk"])
        return {"dq": dq, "dk": dk, "dw_q": dwq, "dw_k": dwk}
    lq, lk = _lens(case)
    if 10 * case["d"] * case["Hq"] * sum(a * b for a, b in zip(lq, lk)) > 8e12:  # past 20 seconds in 64 bits
        return None
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    got = [_exact_sequence(s["q"][a:b], s["k"][i:j], s["v"][i:j], s["do"][a:b],
                           s["dlse"][a:b] if case["dlse"] else None)
           for a, b, i, j in zip(cq, cq[1:], ck, ck[1:])]
    return {n: torch.cat([x[i] for x in got]) for i, n in enumerate(("dq", "dk", "dv"))}
