"""Python binding of libfalcon.so (GB300 Falcon fast-weight forward).

Argument marshalling only: every step of the forward runs in the CUDA
kernels behind the C ABI declared in ``include/falcon.h``.  The functions
keep the C names; tensors are ``torch.Tensor`` on the GPU (their
``data_ptr()`` is passed) or raw integer device pointers.  There is no CPU
fallback: importing this package without a built ``libfalcon.so`` raises.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfalcon.so")

FALCON_1, FALCON_1A, FALCON_2, FALCON_2A, FALCON_3, FALCON_3A = range(6)
FALCON_BF16, FALCON_F32 = 0, 1
FALCON_IMPL_AUTO, FALCON_IMPL_GENERIC, FALCON_IMPL_TC, FALCON_IMPL_SCAN = 0, 1, 2, 3
FALCON_PAIR_PREFIX, FALCON_PAIR_SAME_STEP = 0, 1
FALCON_PROLOGUE_L2NORM_QK, FALCON_PROLOGUE_GATE_LOGITS = 1, 2
FALCON_ROPE_HALF, FALCON_ROPE_INTERLEAVED = 0, 1
FALCON_OK = 0
FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED, FALCON_ERR_WORKSPACE = -1, -2, -3
FALCON_ERR_CUDA, FALCON_ERR_TIMEOUT = -4, -5

EXPORTED = [
    "falcon_workspace_size", "falcon_chunk_fwd", "falcon_recurrent_step",
    "falcon_masked_parallel_workspace_size", "falcon_masked_parallel_ref_gpu",
    "falcon_strerror", "falcon_version", "falcon_chunk_fwd_plan", "falcon_chunk_fwd_timed",
    "falcon_chunk_fwd_noalloc", "falcon_backward_workspace_size", "falcon_backward",
    "falcon_backward_carry",
    "falcon_varlen_workspace_size", "falcon_chunk_fwd_varlen", "falcon_workspace_status",
    "falcon_test_hooks", "falcon_rope_table", "falcon_qk_norm_rope", "falcon_kv_append",
    "falcon_attn_decode_workspace_size", "falcon_attn_decode", "falcon_attn_prompt_workspace_size",
    "falcon_attn_prompt",
]


class FalconError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} ({code})")


class falcon_params_t(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("window", ctypes.c_int32), ("eps", ctypes.c_float), ("eps_gamma", ctypes.c_float),
                ("variant", ctypes.c_int32), ("dtype", ctypes.c_int32), ("impl", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("prologue", ctypes.c_int32)]


class falcon_carry_t(ctypes.Structure):
    _fields_ = [("S", ctypes.c_void_p), ("k_prev", ctypes.c_void_p), ("win_x", ctypes.c_void_p),
                ("win_v", ctypes.c_void_p), ("pos", ctypes.c_void_p)]


class AttnParams(ctypes.Structure):
    """falcon_attn_params_t of the softmax-attention operators.  Fields left
    out are 0 (norm_eps 1e-6); an operator reads the ones that its entry in
    include/falcon.h names."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "B", "Hq", "Hkv", "d", "dtype", "qk_norm", "rot", "rope_layout", "rope_rows", "page", "num_pages",
        "max_pages", "max_q", "max_k")] + [("norm_eps", ctypes.c_float), ("scale", ctypes.c_float)] + [
        (n, ctypes.c_int64) for n in ("tokens", "k_tokens", "q_stride", "k_stride", "v_stride", "o_stride")]

    def __init__(self, B: int = 1, norm_eps: float = 1e-6, **kw):
        super().__init__(B=B, norm_eps=norm_eps, **kw)


class falcon_kv_cache_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfalcon.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    P, C, V, S = ctypes.POINTER(falcon_params_t), ctypes.POINTER(falcon_carry_t), ctypes.c_void_p, ctypes.c_size_t
    lib.falcon_workspace_size.argtypes = [P]
    lib.falcon_workspace_size.restype = S
    lib.falcon_chunk_fwd.argtypes = [P, V, V, V, V, V, C, V, C, V, S, V]
    lib.falcon_chunk_fwd.restype = ctypes.c_int
    lib.falcon_recurrent_step.argtypes = [P, V, V, V, V, V, C, V, V]
    lib.falcon_recurrent_step.restype = ctypes.c_int
    lib.falcon_masked_parallel_workspace_size.argtypes = [P]
    lib.falcon_masked_parallel_workspace_size.restype = S
    lib.falcon_masked_parallel_ref_gpu.argtypes = [P, V, V, V, V, V, V, V, V, S, V]
    lib.falcon_masked_parallel_ref_gpu.restype = ctypes.c_int
    lib.falcon_chunk_fwd_timed.argtypes = [P, V, V, V, V, V, C, V, C, V, S, V,
                                           ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32]
    lib.falcon_chunk_fwd_timed.restype = ctypes.c_int
    lib.falcon_chunk_fwd_noalloc.argtypes = [P, V, V, V, V, V, C, V, C, V]
    lib.falcon_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.falcon_chunk_fwd_plan.argtypes = [P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.falcon_chunk_fwd_plan.restype = ctypes.c_int
    lib.falcon_varlen_workspace_size.argtypes = [P]
    lib.falcon_varlen_workspace_size.restype = S
    lib.falcon_chunk_fwd_varlen.argtypes = [P, V, ctypes.c_int64, V, V, V, V, V, C, V, C, V, S, V]
    lib.falcon_chunk_fwd_varlen.restype = ctypes.c_int
    lib.falcon_backward_workspace_size.argtypes = [P]
    lib.falcon_backward_workspace_size.restype = S
    lib.falcon_backward.argtypes = [P, V, V, V, V, V, C, V, V, V, V, V, V, V, V, V, V, S, V]
    lib.falcon_backward.restype = ctypes.c_int
    lib.falcon_backward_carry.argtypes = [P, V, V, V, V, V, C, V, V, V, V, V, V, V, C, V, S, V]
    lib.falcon_backward_carry.restype = ctypes.c_int
    lib.falcon_workspace_status.argtypes = [V, V]
    lib.falcon_workspace_status.restype = ctypes.c_int
    lib.falcon_test_hooks.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    lib.falcon_test_hooks.restype = None
    A, K, I = ctypes.POINTER(AttnParams), ctypes.POINTER(falcon_kv_cache_t), ctypes.c_int32
    lib.falcon_rope_table.argtypes = [V, I, I, ctypes.c_float, V, V]
    lib.falcon_rope_table.restype = ctypes.c_int
    lib.falcon_qk_norm_rope.argtypes = [A, V, V, V, V, V, V, V, V, V]
    lib.falcon_qk_norm_rope.restype = ctypes.c_int
    lib.falcon_kv_append.argtypes = [A, V, V, V, V, V, V, V, K, V]
    lib.falcon_kv_append.restype = ctypes.c_int
    lib.falcon_attn_decode_workspace_size.argtypes = [A]
    lib.falcon_attn_decode_workspace_size.restype = S
    lib.falcon_attn_decode.argtypes = [A, V, K, V, V, V, V, V, S, V]
    lib.falcon_attn_decode.restype = ctypes.c_int
    lib.falcon_attn_prompt_workspace_size.argtypes = [A]
    lib.falcon_attn_prompt_workspace_size.restype = S
    lib.falcon_attn_prompt.argtypes = [A, V, V, V, V, V, V, V, V, S, V]
    lib.falcon_attn_prompt.restype = ctypes.c_int
    lib.falcon_strerror.argtypes = [ctypes.c_int]
    lib.falcon_strerror.restype = ctypes.c_char_p
    lib.falcon_version.argtypes = []
    lib.falcon_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


@dataclass
class Params:
    """Python mirror of falcon_params_t."""
    B: int
    T: int
    H: int
    dk: int
    dv: int
    chunk: int = 64
    window: int = 1
    eps: float = 1e-6
    eps_gamma: float = 1e-3
    variant: int = FALCON_1
    dtype: int = FALCON_BF16
    impl: int = FALCON_IMPL_AUTO
    pairing: int = FALCON_PAIR_PREFIX
    prologue: int = 0

    def c(self) -> falcon_params_t:
        return falcon_params_t(self.B, self.T, self.H, self.dk, self.dv, self.chunk, self.window,
                               self.eps, self.eps_gamma, self.variant, self.dtype, self.impl,
                               self.pairing, self.prologue)


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        try:
            import torch
            # torch.cuda.current_stream().cuda_stream without the Stream object (3 us a call)
            return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        except AttributeError:  # pragma: no cover
            return torch.cuda.current_stream().cuda_stream
        except Exception:  # pragma: no cover
            return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_carry(carry: dict | None) -> falcon_carry_t | None:
    """Carry dict {S, k_prev, win_x, win_v, pos} -> falcon_carry_t (fields may be None)."""
    if carry is None:
        return None
    return falcon_carry_t(_ptr(carry.get("S")), _ptr(carry.get("k_prev")), _ptr(carry.get("win_x")),
                          _ptr(carry.get("win_v")), _ptr(carry.get("pos")))


def strerror(code: int) -> str:
    return load_library().falcon_strerror(code).decode()


def falcon_version() -> str:
    return load_library().falcon_version().decode()


def falcon_workspace_size(p: Params) -> int:
    return int(load_library().falcon_workspace_size(ctypes.byref(p.c())))


def falcon_masked_parallel_workspace_size(p: Params) -> int:
    return int(load_library().falcon_masked_parallel_workspace_size(ctypes.byref(p.c())))


def falcon_chunk_fwd_plan(p: Params) -> tuple[int, int]:
    """(impl, launches) the chunk forward uses for params p."""
    impl, n = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().falcon_chunk_fwd_plan(ctypes.byref(p.c()), ctypes.byref(impl),
                                                 ctypes.byref(n)), "falcon_chunk_fwd_plan")
    return impl.value, n.value


def _check(code: int, where: str):
    if code != FALCON_OK:
        raise FalconError(code, where)


def falcon_chunk_fwd(p: Params, q, k, v, beta, lam, carry_in: dict | None, o,
                     carry_out: dict | None, workspace=None, workspace_bytes: int = 0, stream=None):
    lib = load_library()
    ci = make_carry(carry_in)
    co = make_carry(carry_out)
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = lib.falcon_chunk_fwd(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam),
                                ctypes.byref(ci) if ci is not None else None, _ptr(o),
                                ctypes.byref(co) if co is not None else None, _ptr(workspace),
                                workspace_bytes, _stream(stream))
    _check(code, "falcon_chunk_fwd")


def falcon_chunk_fwd_timed(p: Params, q, k, v, beta, lam, carry_in: dict | None, o,
                           carry_out: dict | None, workspace, workspace_bytes: int, stream,
                           events: list):
    """falcon_chunk_fwd recording torch.cuda.Event objects around each kernel."""
    lib = load_library()
    ci = make_carry(carry_in)
    co = make_carry(carry_out)
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    code = lib.falcon_chunk_fwd_timed(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                      _ptr(lam), ctypes.byref(ci) if ci is not None else None,
                                      _ptr(o), ctypes.byref(co) if co is not None else None,
                                      _ptr(workspace), workspace_bytes, _stream(stream), arr,
                                      len(events))
    _check(code, "falcon_chunk_fwd_timed")


def falcon_chunk_fwd_noalloc(p: Params, q, k, v, beta, lam, carry_in: dict | None, o,
                             carry_out: dict | None, stream=None):
    """falcon_chunk_fwd without a workspace argument, for callers that cannot
    allocate device memory: the library uses its own fixed scratch array."""
    lib = load_library()
    ci = make_carry(carry_in)
    co = make_carry(carry_out)
    code = lib.falcon_chunk_fwd_noalloc(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                        _ptr(lam), ctypes.byref(ci) if ci is not None else None,
                                        _ptr(o), ctypes.byref(co) if co is not None else None,
                                        _stream(stream))
    _check(code, "falcon_chunk_fwd_noalloc")


def falcon_workspace_status(workspace=None, stream=None) -> int:
    """Status code of the last tensor-core call that used ``workspace`` (None:
    the last falcon_chunk_fwd_noalloc call on the current device): FALCON_OK
    or FALCON_ERR_TIMEOUT.  Synchronises the stream; clears the word."""
    code = load_library().falcon_workspace_status(_ptr(workspace), _stream(stream))
    if code not in (FALCON_OK, FALCON_ERR_TIMEOUT):
        _check(code, "falcon_workspace_status")
    return code


def falcon_test_hooks(wait_limit_ns: int = 0, stall: bool = False) -> None:
    """Failure-detection test hook: the bounded-wait limit of later calls
    (0 = the default 2 s) and a one-shot stall of the next Falcon-1/1A
    tensor-core call's per-chunk kernel."""
    load_library().falcon_test_hooks(int(wait_limit_ns), 1 if stall else 0)


def falcon_recurrent_step(p: Params, q, k, v, beta, lam, carry: dict, o, stream=None):
    lib = load_library()
    c = make_carry(carry)
    code = lib.falcon_recurrent_step(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                     _ptr(lam), ctypes.byref(c) if c is not None else None, _ptr(o),
                                     _stream(stream))
    _check(code, "falcon_recurrent_step")


def falcon_masked_parallel_ref_gpu(p: Params, q, k, v, beta, lam, o, S_final, workspace,
                                   workspace_bytes: int = 0, stream=None):
    lib = load_library()
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = lib.falcon_masked_parallel_ref_gpu(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(beta), _ptr(lam), _ptr(o), _ptr(S_final),
                                              _ptr(workspace), workspace_bytes, _stream(stream))
    _check(code, "falcon_masked_parallel_ref_gpu")


def falcon_varlen_workspace_size(p: Params) -> int:
    return int(load_library().falcon_varlen_workspace_size(ctypes.byref(p.c())))


def falcon_chunk_fwd_varlen(p: Params, cu_seqlens, total_tokens: int, q, k, v, beta, lam,
                            carry_in: dict | None, o, carry_out: dict | None, workspace,
                            workspace_bytes: int = 0, stream=None):
    lib = load_library()
    ci = make_carry(carry_in)
    co = make_carry(carry_out)
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = lib.falcon_chunk_fwd_varlen(ctypes.byref(p.c()), _ptr(cu_seqlens), int(total_tokens), _ptr(q),
                                       _ptr(k), _ptr(v), _ptr(beta), _ptr(lam),
                                       ctypes.byref(ci) if ci is not None else None, _ptr(o),
                                       ctypes.byref(co) if co is not None else None, _ptr(workspace),
                                       workspace_bytes, _stream(stream))
    _check(code, "falcon_chunk_fwd_varlen")


def falcon_backward_workspace_size(p: Params) -> int:
    return int(load_library().falcon_backward_workspace_size(ctypes.byref(p.c())))


def falcon_backward(p: Params, q, k, v, beta, lam, carry_in: dict | None, dO, dS_final, dq, dk, dv,
                    dbeta, dlam, dS_in, dk_prev, workspace, workspace_bytes: int = 0, stream=None):
    lib = load_library()
    ci = make_carry(carry_in)
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = lib.falcon_backward(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam),
                               ctypes.byref(ci) if ci is not None else None, _ptr(dO), _ptr(dS_final),
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dlam), _ptr(dS_in),
                               _ptr(dk_prev), _ptr(workspace), workspace_bytes, _stream(stream))
    _check(code, "falcon_backward")


def falcon_backward_carry(p: Params, q, k, v, beta, lam, carry_in: dict | None, dO, dS_final, dq, dk, dv,
                          dbeta, dlam, dcarry: dict | None, workspace, workspace_bytes: int = 0, stream=None):
    """dcarry: dict of output buffers {S, k_prev, win_x, win_v} (any may be None)."""
    lib = load_library()
    ci = make_carry(carry_in)
    dc = make_carry(dcarry)
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = lib.falcon_backward_carry(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam),
                                     ctypes.byref(ci) if ci is not None else None, _ptr(dO), _ptr(dS_final),
                                     _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dlam),
                                     ctypes.byref(dc) if dc is not None else None, _ptr(workspace),
                                     workspace_bytes, _stream(stream))
    _check(code, "falcon_backward_carry")


def falcon_rope_table(inv_freq, rot: int, rows: int, mscale: float, table, stream=None):
    _check(load_library().falcon_rope_table(_ptr(inv_freq), rot, rows, mscale, _ptr(table), _stream(stream)),
           "falcon_rope_table")


def falcon_qk_norm_rope(p: AttnParams, q, k, w_q, w_k, positions, table, q_out, k_out, stream=None):
    code = load_library().falcon_qk_norm_rope(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k),
                                              _ptr(positions), _ptr(table), _ptr(q_out), _ptr(k_out),
                                              _stream(stream))
    _check(code, "falcon_qk_norm_rope")


def make_kv_cache(cache: dict | None) -> falcon_kv_cache_t | None:
    """Cache dict {k, v, k_scale, v_scale} -> falcon_kv_cache_t."""
    if cache is None:
        return None
    return falcon_kv_cache_t(_ptr(cache["k"]), _ptr(cache["v"]), _ptr(cache["k_scale"]), _ptr(cache["v_scale"]))


def falcon_kv_append(p: AttnParams, k, v, w_k, table, cu_new, ctx_lens, block_table, cache: dict, stream=None):
    c = make_kv_cache(cache)
    code = load_library().falcon_kv_append(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(w_k), _ptr(table), _ptr(cu_new),
                                           _ptr(ctx_lens), _ptr(block_table),
                                           ctypes.byref(c) if c is not None else None, _stream(stream))
    _check(code, "falcon_kv_append")


def falcon_attn_decode_workspace_size(p: AttnParams) -> int:
    return int(load_library().falcon_attn_decode_workspace_size(ctypes.byref(p)))


def falcon_attn_decode(p: AttnParams, q, cache: dict, block_table, lens, o, lse, workspace,
                       workspace_bytes: int = 0, stream=None):
    c = make_kv_cache(cache)
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = load_library().falcon_attn_decode(ctypes.byref(p), _ptr(q), ctypes.byref(c) if c is not None else None,
                                             _ptr(block_table), _ptr(lens), _ptr(o), _ptr(lse), _ptr(workspace),
                                             workspace_bytes, _stream(stream))
    _check(code, "falcon_attn_decode")


def falcon_attn_prompt_workspace_size(p: AttnParams) -> int:
    return int(load_library().falcon_attn_prompt_workspace_size(ctypes.byref(p)))


def falcon_attn_prompt(p: AttnParams, q, k, v, cu_q, cu_k, o, lse, workspace, workspace_bytes: int = 0,
                       stream=None):
    if workspace is not None and not workspace_bytes and not isinstance(workspace, int):
        workspace_bytes = workspace.numel() * workspace.element_size()
    code = load_library().falcon_attn_prompt(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k),
                                             _ptr(o), _ptr(lse), _ptr(workspace), workspace_bytes,
                                             _stream(stream))
    _check(code, "falcon_attn_prompt")


# ---------------------------------------------------------------- tensor helpers
def alloc_workspace(nbytes: int, device="cuda"):
    """A 256-byte aligned byte buffer (torch's caching allocator aligns to 512)."""
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def empty_carry(p: Params, device="cuda") -> dict:
    """Carry buffers for an output carry of params p."""
    import torch
    dt = torch.bfloat16 if p.dtype == FALCON_BF16 else torch.float32
    c = {"S": torch.empty((p.B, p.H, p.dk, p.dv), dtype=torch.float32, device=device),
         "k_prev": torch.empty((p.B, p.H, p.dk), dtype=dt, device=device),
         "pos": torch.empty((p.B, p.H), dtype=torch.int64, device=device)}
    if p.variant in (FALCON_3, FALCON_3A) and p.window > 1:
        c["win_x"] = torch.empty((p.B, p.H, p.window - 1, p.dk), dtype=dt, device=device)
        c["win_v"] = torch.empty((p.B, p.H, p.window - 1, p.dv), dtype=dt, device=device)
    return c


def chunk_forward(p: Params, q, k, v, beta, lam, carry_in: dict | None = None, want_carry=True,
                  stream=None):
    """Allocate o / carry_out / workspace with torch and call falcon_chunk_fwd."""
    import torch
    o = torch.empty((p.B, p.T, p.H, p.dv), dtype=q.dtype, device=q.device)
    co = empty_carry(p, q.device) if want_carry else None
    ws_n = falcon_workspace_size(p)
    ws = alloc_workspace(ws_n, q.device) if ws_n else None
    falcon_chunk_fwd(p, q, k, v, beta, lam, carry_in, o, co, ws, ws_n, stream)
    return o, co


def chunk_forward_varlen(p: Params, cu_seqlens, q, k, v, beta, lam, carry_in: dict | None = None,
                        want_carry=True, stream=None):
    """Packed sequences: q, k [total, H, dk], v [total, H, dv], cu_seqlens int32
    [B + 1] on the device; p.B = number of sequences, p.T >= the longest."""
    import torch
    total = q.shape[0]
    o = torch.empty((total, p.H, p.dv), dtype=q.dtype, device=q.device)
    co = empty_carry(p, q.device) if want_carry else None
    ws_n = falcon_varlen_workspace_size(p)
    ws = alloc_workspace(ws_n, q.device)
    falcon_chunk_fwd_varlen(p, cu_seqlens, total, q, k, v, beta, lam, carry_in, o, co, ws, ws_n, stream)
    return o, co


def masked_parallel(p: Params, q, k, v, beta, lam, stream=None):
    import torch
    o = torch.empty((p.B, p.T, p.H, p.dv), dtype=q.dtype, device=q.device)
    S = torch.empty((p.B, p.H, p.dk, p.dv), dtype=torch.float32, device=q.device)
    ws_n = falcon_masked_parallel_workspace_size(p)
    ws = alloc_workspace(ws_n, q.device)
    falcon_masked_parallel_ref_gpu(p, q, k, v, beta, lam, o, S, ws, ws_n, stream)
    return o, S



def backward(p: Params, q, k, v, beta, lam, dO, dS_final=None, carry_in: dict | None = None,
             stream=None) -> dict:
    """Allocate the gradients / workspace with torch and call falcon_backward_carry.

    Returns dq, dk, dv, dbeta, dlam, dS_in / dk_prev (gradients of the
    carried state and key) and, for Falcon-3/3A with W > 1, dwin_x / dwin_v
    (gradients of the carried window ring)."""
    import torch
    dev = q.device
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dbeta": torch.empty_like(beta), "dlam": torch.empty_like(lam),
         "dS_in": torch.empty((p.B, p.H, p.dk, p.dv), dtype=torch.float32, device=dev),
         "dk_prev": torch.empty((p.B, p.H, p.dk), dtype=q.dtype, device=dev)}
    dc = {"S": g["dS_in"], "k_prev": g["dk_prev"]}
    if p.variant in (FALCON_3, FALCON_3A) and p.window > 1:
        g["dwin_x"] = dc["win_x"] = torch.empty((p.B, p.H, p.window - 1, p.dk), dtype=q.dtype, device=dev)
        g["dwin_v"] = dc["win_v"] = torch.empty((p.B, p.H, p.window - 1, p.dv), dtype=q.dtype, device=dev)
    ws_n = falcon_backward_workspace_size(p)
    ws = alloc_workspace(ws_n, dev) if ws_n else None
    falcon_backward_carry(p, q, k, v, beta, lam, carry_in, dO, dS_final, g["dq"], g["dk"], g["dv"],
                          g["dbeta"], g["dlam"], dc, ws, ws_n, stream)
    return g


# ------------------------------------------------- softmax-attention layers: tensor helpers
def _attn_dtype(x) -> int:
    import torch
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"bf16 or fp32 tensors are wanted, not {x.dtype}")
    return FALCON_BF16 if x.dtype == torch.bfloat16 else FALCON_F32


def _token_stride(x, name: str) -> int:
    """Elements between tokens of x [tokens, H, d], whose heads and dims must be dense."""
    if x.dim() != 3 or (x.numel() and (x.stride(2) != 1 or (x.shape[1] > 1 and x.stride(1) != x.shape[2]))):
        raise ValueError(f"{name}: [tokens, heads, d] with dense heads is wanted, not shape {tuple(x.shape)} "
                         f"strides {x.stride()}")
    if x.shape[0] > 1 and x.stride(0) < x.shape[1] * x.shape[2]:
        raise ValueError(f"{name}: tokens that do not overlap are wanted, not strides {x.stride()}")
    return x.stride(0) if x.shape[0] > 1 else 0


def _on(stream):
    """Allocations made under it belong to ``stream``, on which the call runs."""
    import contextlib

    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) and stream else
                             torch.cuda.default_stream() if isinstance(stream, int) else stream)


def _like(x, ref, name: str, dtype=None):
    if x is not None and (x.device != ref.device or (dtype is not None and x.dtype != dtype)):
        raise ValueError(f"{name}: {dtype or ''} on {ref.device} is wanted, not {x.dtype} on {x.device}")
    if x is not None and dtype is not None and not x.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is wanted")


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq float64 [rot/2] on the CPU, mscale) of rotary positions,
    f_i = base^(-2i/rot), stretched for contexts ``factor`` times as long:

    * "linear": every frequency over factor (positions interpolated).
    * "ntk": base times factor^(rot/(rot-2)), so that the lowest frequency is
      divided by factor and the highest kept.
    * "yarn": per frequency between the two: those that turn more than
      beta_fast times over original_len tokens are kept, those that turn less
      than beta_slow times divided by factor, a linear ramp over the index in
      between; mscale = 0.1 ln(factor) + 1.
    """
    import math

    import torch
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if factor < 1.0:
        raise ValueError("factor >= 1 is wanted")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / max(rot, 1))
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        if original_len < 1:
            raise ValueError("yarn needs original_len")
        at = lambda turns: rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return f, 1.0


def rope_table(inv_freq, rows: int, mscale: float = 1.0, device="cuda", stream=None):
    """Rotary table [rows, rot/2, 2] (cos, sin) for falcon_qk_norm_rope / falcon_kv_append."""
    import torch
    with _on(stream):
        f = inv_freq.to(device=device, dtype=torch.float64).contiguous()
        t = torch.empty((rows, f.numel(), 2), dtype=torch.float32, device=device)
        falcon_rope_table(f, 2 * f.numel(), rows, mscale, t, stream)
    return t


def _rope_fields(d: int, table, layout: int, norm: bool, norm_eps: float) -> dict:
    if table is None:
        return dict(qk_norm=int(norm), norm_eps=norm_eps)
    if table.dim() != 3 or table.shape[2] != 2 or 2 * table.shape[1] > d:
        raise ValueError(f"table: [rows, rot/2, 2] with rot <= {d} is wanted, not {tuple(table.shape)}")
    return dict(qk_norm=int(norm), norm_eps=norm_eps, rot=2 * table.shape[1], rope_rows=table.shape[0],
                rope_layout=layout)


def qk_norm_rope(q, k, positions=None, table=None, w_q=None, w_k=None, norm: bool = True, norm_eps: float = 1e-6,
                 layout: int = FALCON_ROPE_HALF, stream=None):
    """Norm and rotation of q [tokens, Hq, d] and k [tokens, Hkv, d] (k may be
    None): returns (q_out, k_out), dense.  table None: no rotation.  Forward
    only: the results carry no gradient, also where an input requires one."""
    import torch
    _, Hq, d = q.shape
    p = AttnParams(Hq=Hq, Hkv=Hq if k is None else k.shape[1], d=d, dtype=_attn_dtype(q), tokens=q.shape[0],
                   q_stride=_token_stride(q, "q"), k_stride=0 if k is None else _token_stride(k, "k"),
                   **_rope_fields(d, table, layout, norm, norm_eps))
    if k is not None and (k.shape[0] != q.shape[0] or k.shape[2] != d or k.dtype != q.dtype):
        raise ValueError("q and k differ in tokens, head dim or dtype")
    if table is not None and (positions is None or positions.shape != (q.shape[0],)):
        raise ValueError("positions: int64 [tokens] is wanted with a table")
    _like(k, q, "k")
    for x, n, t in ((w_q, "w_q", torch.float32), (w_k, "w_k", torch.float32), (table, "table", torch.float32),
                    (positions, "positions", torch.int64)):
        _like(x, q, n, t)
    for x, n in ((w_q, "w_q"), (w_k, "w_k")):
        if x is not None and x.shape != (d,):
            raise ValueError(f"{n}: [d] is wanted")
    with _on(stream):
        qo = torch.empty((q.shape[0], Hq, d), dtype=q.dtype, device=q.device)
        ko = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        falcon_qk_norm_rope(p, q, k, w_q, w_k, positions, table, qo, ko, stream)
    return qo, ko


def empty_kv_cache(num_pages: int, Hkv: int, page: int, d: int, device="cuda") -> dict:
    """Buffers of a paged 8-bit cache: e4m3 codes and e8m0 scales as bytes."""
    import torch
    codes = lambda: torch.zeros((num_pages, Hkv, page, d), dtype=torch.uint8, device=device)  # noqa: E731
    scales = lambda: torch.zeros((num_pages, Hkv), dtype=torch.uint8, device=device)  # noqa: E731
    return {"k": codes(), "v": codes(), "k_scale": scales(), "v_scale": scales()}


def _cache_fields(cache: dict, block_table, ref) -> dict:
    import torch
    pages, Hkv, page, d = cache["k"].shape
    for n, shape in (("k", (pages, Hkv, page, d)), ("v", (pages, Hkv, page, d)), ("k_scale", (pages, Hkv)),
                     ("v_scale", (pages, Hkv))):
        x = cache[n]
        if tuple(x.shape) != shape or x.element_size() != 1 or not x.is_contiguous() or x.device != ref.device:
            raise ValueError(f"cache {n}: contiguous bytes {shape} on {ref.device} are wanted")
    _like(block_table, ref, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table: [B, max_pages] is wanted")
    return dict(Hkv=Hkv, d=d, page=page, num_pages=pages, max_pages=block_table.shape[1])


def kv_append(cache: dict, k, v, cu_new, ctx_lens, block_table, max_new: int, table=None, w_k=None,
              norm: bool = False, norm_eps: float = 1e-6, layout: int = FALCON_ROPE_HALF, stream=None) -> None:
    """Append k, v [tokens, Hkv, d] to the cache in place; cu_new int32 [B + 1],
    ctx_lens int32 [B], block_table int32 [B, max_pages]; max_new is at least
    the most tokens of one sequence.  No gradient passes through the cache."""
    import torch
    f = _cache_fields(cache, block_table, k)
    B = block_table.shape[0]
    if k.shape != v.shape or k.dtype != v.dtype or k.shape[1:] != (f["Hkv"], f["d"]):
        raise ValueError("k and v: [tokens, Hkv, d] of one dtype, as the cache's, are wanted")
    if cu_new.shape != (B + 1,) or ctx_lens.shape != (B,):
        raise ValueError("cu_new [B + 1] and ctx_lens [B] are wanted")
    _like(v, k, "v")
    for x, n, t in ((w_k, "w_k", torch.float32), (table, "table", torch.float32), (cu_new, "cu_new", torch.int32),
                    (ctx_lens, "ctx_lens", torch.int32)):
        _like(x, k, n, t)
    if w_k is not None and w_k.shape != (f["d"],):
        raise ValueError("w_k: [d] is wanted")
    p = AttnParams(B=B, Hq=f["Hkv"], dtype=_attn_dtype(k), tokens=k.shape[0], max_q=max_new,
                   k_stride=_token_stride(k, "k"), v_stride=_token_stride(v, "v"), **f,
                   **_rope_fields(f["d"], table, layout, norm, norm_eps))
    falcon_kv_append(p, k, v, w_k, table, cu_new, ctx_lens, block_table, cache, stream)


def attn_decode(q, cache: dict, block_table, lens, max_len: int, scale: float = 0.0, want_lse=False, stream=None):
    """One token per sequence: q [B, Hq, d], lens int32 [B] (at most max_len) -> o, or (o, lse).  Forward only: the
    results carry no gradient."""
    import torch
    f = _cache_fields(cache, block_table, q)
    if q.shape[0] != block_table.shape[0] or lens.shape != (q.shape[0],) or q.shape[2] != f["d"]:
        raise ValueError("q [B, Hq, d], block_table [B, max_pages] and lens [B] are wanted, d as the cache's")
    _like(lens, q, "lens", torch.int32)
    B, Hq, d = q.shape
    p = AttnParams(B=B, Hq=Hq, dtype=_attn_dtype(q), max_k=max_len, scale=scale, q_stride=_token_stride(q, "q"), **f)
    with _on(stream):
        o = torch.empty((B, Hq, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if want_lse else None
        if B > 0:
            ws = alloc_workspace(falcon_attn_decode_workspace_size(p), q.device)
            falcon_attn_decode(p, q, cache, block_table, lens, o, lse, ws, 0, stream)
    return (o, lse) if want_lse else o


def attn_prompt(q, k, v, cu_q, cu_k=None, max_q: int = 0, scale: float = 0.0, want_lse=False, stream=None):
    """Causal attention over packed prompts: q [tokens, Hq, d], k and v
    [k_tokens, Hkv, d], cu_q / cu_k int32 [B + 1] (cu_k None: cu_q), max_q at
    least the longest sequence's rows of q (0: all of them; the exact bound is
    the quickest) -> o, or (o, lse).  Forward only: the results carry no
    gradient, also where an input requires one."""
    import torch
    cu_k = cu_q if cu_k is None else cu_k
    if k.shape != v.shape or k.shape[2] != q.shape[2] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v: [k_tokens, Hkv, d] with q's d and dtype are wanted")
    if cu_q.dim() != 1 or cu_q.shape != cu_k.shape or cu_q.numel() < 2:
        raise ValueError("cu_q and cu_k: [B + 1] are wanted")
    _like(k, q, "k")
    _like(v, q, "v")
    _like(cu_q, q, "cu_q", torch.int32)
    _like(cu_k, q, "cu_k", torch.int32)
    n, Hq, d = q.shape
    p = AttnParams(B=cu_q.numel() - 1, Hq=Hq, Hkv=k.shape[1], d=d, dtype=_attn_dtype(q), max_q=max_q or n, tokens=n,
                   k_tokens=k.shape[0], scale=scale, q_stride=_token_stride(q, "q"),
                   k_stride=_token_stride(k, "k"), v_stride=_token_stride(v, "v"))
    with _on(stream):
        o = torch.empty((n, Hq, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((n, Hq), dtype=torch.float32, device=q.device) if want_lse else None
        ws = alloc_workspace(falcon_attn_prompt_workspace_size(p), q.device)
        falcon_attn_prompt(p, q, k, v, cu_q, cu_k, o, lse, ws, 0, stream)
    return (o, lse) if want_lse else o


load_library()
