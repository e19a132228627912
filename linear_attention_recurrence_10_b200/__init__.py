"""Gated DeltaNet (gated delta rule) token mixer for B200 -- Python binding.

Thin wrappers over the C ABI of include/gdr.h (libgdr.so, built in-tree by
``python -m linear_attention_recurrence_10_b200.build``).  Each wrapper only
turns torch tensors into pointers, strides and dtype codes and passes the
current CUDA stream; every step of the computation runs in the library's
kernels.  PyTorch is used for device memory and streams only.

    decode_step(q, k, v, g, beta, state, out, ...)        one token per sequence
    prefill_chunked(q, k, v, g, beta, cu_seqlens, out, ...)  packed varlen prompts
    rmsnorm_gated(o, z, out, ...)                          the output gate alone
    attn_decode_step(q, gate, k, v, k_cache, v_cache, cache_len, out, ...)
                                                           gated full-attention decode
    kv_append(k, v, k_pages, v_pages, ...)                  new tokens into a paged cache
    attn_paged(q, k_pages, v_pages, ...)                    new tokens attend over the pages
    kv_gather(k_pages, v_pages, ...)                        cached tokens read back
    moe_decode(x, w_router, w_gate_up, w_down, out, ...)    routed-expert MoE block
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from . import _abi
from ._abi import GDR_BF16, GDR_E4M3, GDR_F32

__all__ = ["GdrError", "decode_step", "decode_multi", "prefill_chunked", "prefill_chunked_noalloc",
           "prefill_noalloc_status", "prefill_workspace_size", "attn_decode_step",
           "attn_decode_workspace_size", "kv_append", "kv_gather", "attn_paged",
           "attn_paged_workspace_size", "moe_decode", "moe_workspace_size",
           "rmsnorm_gated", "version", "status_string"]


class GdrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        name = _abi.STATUS_NAMES.get(self.status, f"status {status}")
        super().__init__(f"{where}: {name}")


def _check(status: int, where: str):
    if status != 0:
        raise GdrError(status, where)


def _dtype_code(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    if t.dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"{what}: dtype {t.dtype} is not bf16 or fp32")


def _ptr(t):
    # A plain int: every pointer field and argument is declared void* (c_void_p).
    return None if t is None else t.data_ptr()


def _row_stride(t: torch.Tensor, what: str) -> int:
    """Row stride of a [rows, H, d] (or [rows, d]) tensor whose inner dims are packed."""
    if t.is_contiguous():
        return t.stride(0) if t.shape[0] > 1 else 0
    if t.dim() >= 2:
        inner = 1
        for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
            if size > 1 and stride != inner:
                raise ValueError(f"{what}: inner dimensions must be contiguous")
            inner *= size
    return int(t.stride(0)) if t.shape[0] > 1 else 0


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    # (Without a GPU the library's own checks run, and its launch fails.)
    elif device.type != "cuda" and torch.cuda.is_available():
        raise ValueError(f"tensors must be on a CUDA device, not {device}")
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _workspace(n_bytes: int, stream, device) -> torch.Tensor:
    """A workspace for one call on `stream` (None: the current one).

    It is allocated with that stream as the current one.  The allocator hands a freed block
    out again in the order of the stream it was allocated on: taken from another stream's,
    it could still be in use by work queued there, which `stream` does not wait for, and
    when the call returns it would go back to that stream while this one still uses it.
    """
    if stream is not None and device.type == "cuda":
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle != torch.cuda.current_stream(device).cuda_stream:
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(handle, device=device) if handle else
                          torch.cuda.default_stream(device))
            with torch.cuda.stream(stream):
                return torch.empty(n_bytes, dtype=torch.uint8, device=device)
    return torch.empty(n_bytes, dtype=torch.uint8, device=device)


def _f32_tensor(t, what):
    if t is not None and t.dtype != torch.float32:
        raise TypeError(f"{what} must be fp32")
    return t


def version() -> int:
    return _abi.lib().gdr_version()


def status_string(status: int) -> str:
    return _abi.lib().gdr_status_string(int(status)).decode()


def _gate_params(gate_params, H_v):
    """(A_log, dt_bias) fp32 [H_v] tensors, or None: see GDR_GATE_FROM_RAW."""
    if gate_params is None:
        return None, None
    A_log, dt_bias = gate_params
    for t, name in ((A_log, "A_log"), (dt_bias, "dt_bias")):
        _f32_tensor(t, name)
        if t.dim() != 1 or t.shape[0] != H_v or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 tensor of H_v entries")
    return A_log, dt_bias


def _decode_args(q, k, v, g, beta, state, out, z, norm_w, state_out, scale, eps_l2, eps_norm,
                 qk_l2norm, overlap_state_load, batch, gate_params=None):
    H_k, d = q.shape[1], q.shape[2]
    H_v = v.shape[1]
    for t, name in ((g, "g"), (beta, "beta"), (state, "state"), (norm_w, "norm_w")):
        _f32_tensor(t, name)
    if g.stride() != beta.stride():
        raise ValueError("g and beta must share one layout")
    so = state if state_out is None else _f32_tensor(state_out, "state_out")
    if state.stride() != so.stride():
        raise ValueError("state and state_out must share one layout")
    in_dtype = _dtype_code(q, "q")
    for t, name in ((k, "k"), (v, "v"), (z, "z")):
        if t is not None and _dtype_code(t, name) != in_dtype:
            raise TypeError(f"{name} must have the dtype of q")
    flags = _abi.GDR_DECODE_OVERLAP_STATE_LOAD if overlap_state_load else 0
    A_log, dt_bias = _gate_params(gate_params, H_v)
    if A_log is not None:
        flags |= _abi.GDR_GATE_FROM_RAW
    # One constructor call: ctypes fills the fields in C, a third of the cost of
    # assigning them one by one (this runs on every decode call).
    return _abi.DecodeArgs(
        batch=batch, H_k=H_k, H_v=H_v, d_k=d, d_v=v.shape[2],
        in_dtype=in_dtype, out_dtype=_dtype_code(out, "out"), qk_l2norm=int(bool(qk_l2norm)),
        scale=float(scale), eps_l2=float(eps_l2), eps_norm=float(eps_norm), flags=flags,
        q_stride=_row_stride(q, "q"), k_stride=_row_stride(k, "k"), v_stride=_row_stride(v, "v"),
        z_stride=_row_stride(z, "z") if z is not None else 0, gb_stride=_row_stride(g, "g"),
        out_stride=_row_stride(out, "out"), state_stride=_row_stride(state, "state"),
        q=_ptr(q), k=_ptr(k), v=_ptr(v), z=_ptr(z), g=_ptr(g), beta=_ptr(beta),
        state_in=_ptr(state), state_out=_ptr(so), norm_w=_ptr(norm_w), out=_ptr(out),
        A_log=_ptr(A_log), dt_bias=_ptr(dt_bias))


def decode_step(q, k, v, g, beta, state, out, *, z=None, norm_w=None, state_out=None,
                scale: float = 1.0, eps_l2: float = 1e-6, eps_norm: float = 1e-6,
                qk_l2norm: bool = True, overlap_state_load: bool = False,
                gate_params=None, stream=None) -> torch.Tensor:
    """Advance every sequence of the batch by one token (gdr_decode_step).

    q, k [B, H_k, d]; v, z [B, H_v, d] (bf16 or fp32, same dtype); g, beta
    [B, H_v] fp32; state [B, H_v, d, d] fp32, updated in place unless
    ``state_out`` is given; out [B, H_v, d] bf16 or fp32.  Batch rows may be
    strided views (e.g. one step of a [B, T, H, d] tensor).
    ``overlap_state_load``: GDR_DECODE_OVERLAP_STATE_LOAD -- only when the
    kernel queued just before this call does not write this state.
    ``gate_params`` = (A_log, dt_bias), fp32 [H_v]: g and beta then hold the
    raw projections a, b (GDR_GATE_FROM_RAW).
    """
    a = _decode_args(q, k, v, g, beta, state, out, z, norm_w, state_out, scale, eps_l2, eps_norm,
                     qk_l2norm, overlap_state_load, q.shape[0], gate_params)
    _check(_abi.lib().gdr_decode_step(ctypes.byref(a), _stream(stream, q.device)),
           "gdr_decode_step")
    return out


def decode_multi(q, k, v, g, beta, state, out, *, n_tokens: int, z=None, norm_w=None,
                 state_out=None, slots=None, status=None, scale: float = 1.0,
                 eps_l2: float = 1e-6, eps_norm: float = 1e-6, qk_l2norm: bool = True,
                 overlap_state_load: bool = False, gate_params=None,
                 stream=None) -> torch.Tensor:
    """Advance every sequence by ``n_tokens`` tokens in one call (gdr_decode_multi).

    Token-indexed tensors hold B * n_tokens rows, row b * n_tokens + t being
    token t of sequence b: q, k [B*T, H_k, d]; v, z [B*T, H_v, d]; g, beta
    [B*T, H_v]; out [B*T, H_v, d].  ``slots`` (int32 [B] on the device, or
    None) maps sequence b to its row of ``state`` [n_rows, H_v, d, d];
    ``status`` (int32 [1] on the device) receives GDR_ERR_INVALID_ARG if a
    slot is out of range.
    """
    rows = q.shape[0]
    if n_tokens < 1 or rows % n_tokens != 0:
        raise ValueError("q must hold batch * n_tokens rows")
    batch = rows // n_tokens
    a = _decode_args(q, k, v, g, beta, state, out, z, norm_w, state_out, scale, eps_l2, eps_norm,
                     qk_l2norm, overlap_state_load, batch, gate_params)
    m = _abi.DecodeMultiArgs()
    m.base = a
    m.n_tokens = int(n_tokens)
    m.n_slots = 0
    if slots is not None:
        if slots.dtype != torch.int32 or slots.dim() != 1 or slots.shape[0] != batch:
            raise ValueError("slots must be an int32 tensor of one entry per sequence")
        m.n_slots = state.shape[0]
    m.state_slot = _ptr(slots)
    m.status = _ptr(status)
    _check(_abi.lib().gdr_decode_multi(ctypes.byref(m), _stream(stream, q.device)),
           "gdr_decode_multi")
    return out


def _prefill_args(q, k, v, g, beta, cu_seqlens, out, cu_seqlens_host, z, norm_w,
                  initial_state, final_state, chunk, scale, eps_l2, eps_norm, qk_l2norm,
                  gate_params=None):
    n_tok, H_k, d = q.shape
    H_v = v.shape[1]
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu()
    host = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
    for t, name in ((g, "g"), (beta, "beta"), (initial_state, "initial_state"),
                    (final_state, "final_state"), (norm_w, "norm_w")):
        _f32_tensor(t, name)
    if g.stride() != beta.stride():
        raise ValueError("g and beta must share one layout")
    a = _abi.PrefillArgs()
    a.n_seq = len(cu_seqlens_host) - 1
    a.H_k, a.H_v, a.d_k, a.d_v = H_k, H_v, d, v.shape[2]
    a.chunk = int(chunk)
    a.in_dtype = _dtype_code(q, "q")
    for t, name in ((k, "k"), (v, "v"), (z, "z")):
        if t is not None and _dtype_code(t, name) != a.in_dtype:
            raise TypeError(f"{name} must have the dtype of q")
    a.out_dtype = _dtype_code(out, "out")
    a.qk_l2norm = int(bool(qk_l2norm))
    a.scale, a.eps_l2, a.eps_norm = float(scale), float(eps_l2), float(eps_norm)
    a.n_tok = n_tok
    a.q_stride, a.k_stride = _row_stride(q, "q"), _row_stride(k, "k")
    a.v_stride = _row_stride(v, "v")
    a.z_stride = _row_stride(z, "z") if z is not None else 0
    a.gb_stride = _row_stride(g, "g")
    a.out_stride = _row_stride(out, "out")
    a.q, a.k, a.v, a.z = _ptr(q), _ptr(k), _ptr(v), _ptr(z)
    a.g, a.beta = _ptr(g), _ptr(beta)
    a.cu_seqlens = _ptr(cu_seqlens)
    a.cu_seqlens_host = ctypes.cast(host, ctypes.POINTER(ctypes.c_int32))
    a.initial_state, a.final_state = _ptr(initial_state), _ptr(final_state)
    a.norm_w, a.out = _ptr(norm_w), _ptr(out)
    A_log, dt_bias = _gate_params(gate_params, H_v)
    if A_log is not None:
        a.flags = _abi.GDR_GATE_FROM_RAW
        a.A_log, a.dt_bias = _ptr(A_log), _ptr(dt_bias)
    return a, host


def prefill_workspace_size(q, k, v, g, beta, cu_seqlens, out, *, cu_seqlens_host=None,
                           z=None, chunk: int = 0, **_) -> int:
    a, host = _prefill_args(q, k, v, g, beta, cu_seqlens, out, cu_seqlens_host, z, None, None,
                            None, chunk, 1.0, 1e-6, 1e-6, True)
    n = ctypes.c_size_t(0)
    _check(_abi.lib().gdr_prefill_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "gdr_prefill_workspace_size")
    del host
    return int(n.value)


def prefill_chunked(q, k, v, g, beta, cu_seqlens, out, *, cu_seqlens_host=None, z=None,
                    norm_w=None, initial_state=None, final_state=None, chunk: int = 0,
                    workspace=None, scale: float = 1.0, eps_l2: float = 1e-6,
                    eps_norm: float = 1e-6, qk_l2norm: bool = True, gate_params=None,
                    stream=None) -> torch.Tensor:
    """Chunked prefill of packed variable-length sequences (gdr_prefill_chunked).

    q, k [n_tok, H_k, d]; v, z, out [n_tok, H_v, d]; g, beta [n_tok, H_v] fp32;
    cu_seqlens int32 [n_seq + 1] on the device (``cu_seqlens_host``: the same
    values on the host, read during the call); initial_state / final_state
    [n_seq, H_v, d, d] fp32 or None.  ``workspace``: a uint8 device tensor of
    at least prefill_workspace_size() bytes; allocated here when None.
    ``gate_params`` = (A_log, dt_bias), fp32 [H_v]: g and beta then hold the
    raw projections a, b (GDR_GATE_FROM_RAW).
    """
    a, host = _prefill_args(q, k, v, g, beta, cu_seqlens, out, cu_seqlens_host, z, norm_w,
                            initial_state, final_state, chunk, scale, eps_l2, eps_norm,
                            qk_l2norm, gate_params)
    L = _abi.lib()
    n = ctypes.c_size_t(0)
    _check(L.gdr_prefill_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "gdr_prefill_workspace_size")
    if workspace is None and n.value:
        workspace = _workspace(int(n.value), stream, q.device)
    ws_ptr = _ptr(workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(L.gdr_prefill_chunked(ctypes.byref(a), ws_ptr, ws_bytes, _stream(stream, q.device)),
           "gdr_prefill_chunked")
    del host
    return out


def prefill_chunked_noalloc(q, k, v, g, beta, cu_seqlens, out, *, cu_seqlens_host=None,
                            z=None, norm_w=None, initial_state=None, final_state=None,
                            chunk: int = 0, scale: float = 1.0, eps_l2: float = 1e-6,
                            eps_norm: float = 1e-6, qk_l2norm: bool = True, gate_params=None,
                            stream=None) -> torch.Tensor:
    """gdr_prefill_chunked_noalloc: the same prefill, with no workspace to pass and
    nothing allocated -- for callers that cannot allocate device memory here.
    At most 4096 sequences per call; calls must not overlap on the GPU (they
    share one scratch array per device).  Arguments as prefill_chunked."""
    a, host = _prefill_args(q, k, v, g, beta, cu_seqlens, out, cu_seqlens_host, z, norm_w,
                            initial_state, final_state, chunk, scale, eps_l2, eps_norm,
                            qk_l2norm, gate_params)
    _check(_abi.lib().gdr_prefill_chunked_noalloc(ctypes.byref(a), _stream(stream, q.device)),
           "gdr_prefill_chunked_noalloc")
    del host
    return out


def prefill_noalloc_status(stream=None) -> int:
    """The status word of the last prefill_chunked_noalloc call on the current
    device (gdr_prefill_noalloc_status): 0, or GDR_ERR_TIMEOUT if a bounded
    device wait gave up.  ``stream``: a torch CUDA stream (default: the current
    one), which is synchronised, since the value is read back to the host."""
    s = stream if stream is not None else torch.cuda.current_stream()
    host = torch.zeros(1, dtype=torch.int32).pin_memory()
    _check(_abi.lib().gdr_prefill_noalloc_status(host.data_ptr(), ctypes.c_void_p(s.cuda_stream)),
           "gdr_prefill_noalloc_status")
    s.synchronize()
    return int(host.item())


def rmsnorm_gated(o, z, out, *, w=None, eps: float = 1e-6, stream=None) -> torch.Tensor:
    """y = o / sqrt(mean(o^2) + eps) * w * z * sigmoid(z) over the last dim (gdr_rmsnorm_gated).

    o, z, out: [..., d] with packed rows; w [d] fp32 or None."""
    d = o.shape[-1]
    o2, z2, out2 = o.reshape(-1, d), z.reshape(-1, d), out.reshape(-1, d)
    if out2.data_ptr() != out.data_ptr():
        raise ValueError("out must be viewable as [rows, d]")
    _f32_tensor(w, "w")
    a = _abi.NormArgs()
    a.rows, a.d = o2.shape[0], d
    a.o_dtype, a.z_dtype = _dtype_code(o, "o"), _dtype_code(z, "z")
    a.out_dtype = _dtype_code(out, "out")
    a.eps = float(eps)
    a.o_stride, a.z_stride = _row_stride(o2, "o"), _row_stride(z2, "z")
    a.out_stride = _row_stride(out2, "out")
    a.o, a.z, a.w, a.out = _ptr(o2), _ptr(z2), _ptr(w), _ptr(out2)
    _check(_abi.lib().gdr_rmsnorm_gated(ctypes.byref(a), _stream(stream, o.device)),
           "gdr_rmsnorm_gated")
    return out


def _attn_args(q, gate, k, v, k_cache, v_cache, cache_len, out, kv_bound, rot_dim, rope_theta,
               scale):
    B, H_q, d = q.shape
    H_kv = k.shape[1]
    for t, name in ((q, "q"), (gate, "gate"), (k, "k"), (v, "v"), (k_cache, "k_cache"),
                    (v_cache, "v_cache")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bf16")
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dim() != 4 or t.shape[:2] != (B, H_kv) or t.shape[3] != d or not t.is_contiguous():
            raise ValueError(f"{name} must be a packed [batch, H_kv, max_len, d] tensor")
    if cache_len.dtype != torch.int32:
        raise TypeError("cache_len must be int32")
    return _abi.AttnDecodeArgs(
        batch=B, H_q=H_q, H_kv=H_kv, d=d, rot_dim=int(rot_dim), max_len=k_cache.shape[2],
        kv_bound=int(kv_bound), out_dtype=_dtype_code(out, "out"), rope_theta=float(rope_theta),
        scale=float(d ** -0.5 if scale is None else scale),
        q_stride=_row_stride(q, "q"), gate_stride=_row_stride(gate, "gate"),
        k_stride=_row_stride(k, "k"), v_stride=_row_stride(v, "v"),
        out_stride=_row_stride(out, "out"), q=_ptr(q), gate=_ptr(gate), k=_ptr(k), v=_ptr(v),
        k_cache=_ptr(k_cache), v_cache=_ptr(v_cache), cache_len=_ptr(cache_len), out=_ptr(out))


def attn_decode_workspace_size(q, gate, k, v, k_cache, v_cache, cache_len, out, *, kv_bound,
                               rot_dim=64, rope_theta=1e7, scale=None) -> int:
    a = _attn_args(q, gate, k, v, k_cache, v_cache, cache_len, out, kv_bound, rot_dim,
                   rope_theta, scale)
    n = ctypes.c_size_t(0)
    _check(_abi.lib().gdr_attn_decode_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "gdr_attn_decode_workspace_size")
    return int(n.value)


def attn_decode_step(q, gate, k, v, k_cache, v_cache, cache_len, out, *, kv_bound, rot_dim=64,
                     rope_theta=1e7, scale=None, workspace=None, stream=None) -> torch.Tensor:
    """One decode step of the gated full-attention layer (gdr_attn_decode_step).

    q, gate [B, H_q, 256]; k, v [B, H_kv, 256] (the new token, bf16);
    k_cache, v_cache [B, H_kv, max_len, 256] bf16 (row cache_len[b] receives the
    rotated key and the value); cache_len int32 [B] on the device; ``kv_bound``
    an upper bound of cache_len on the host; out [B, H_q, 256] bf16 or fp32.
    ``workspace``: a uint8 device tensor of attn_decode_workspace_size() bytes,
    allocated here when None.
    """
    a = _attn_args(q, gate, k, v, k_cache, v_cache, cache_len, out, kv_bound, rot_dim,
                   rope_theta, scale)
    L = _abi.lib()
    n = ctypes.c_size_t(0)
    _check(L.gdr_attn_decode_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "gdr_attn_decode_workspace_size")
    if workspace is None and n.value:
        workspace = _workspace(int(n.value), stream, q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(L.gdr_attn_decode_step(ctypes.byref(a), _ptr(workspace), ws_bytes,
                                  _stream(stream, q.device)), "gdr_attn_decode_step")
    return out


# The paged cache's calls run once per layer and generated token, where the marshalling is
# most of the time: the C structs are packed by struct (native layout) instead of field by
# field, and each tensor is asked as little as its checks need.
_KV_PAGES = "8i q 6P"
_PACK_APPEND = struct.Struct("@" + _KV_PAGES + " q 2i f i 4q 6P")
_PACK_GATHER = struct.Struct("@" + _KV_PAGES + " q 2i 2q 4P")
_PACK_ATTN = struct.Struct("@" + _KV_PAGES + " q 2i f i 4q 5P")


def _distinct_rows(t, what):
    """Row stride in the C ABI's terms: 0 for packed rows; rows must not be one row expanded."""
    if t.is_contiguous():
        return 0
    s = _row_stride(t, what)
    if s == 0 and t.shape[0] > 1:
        raise ValueError(f"{what}: rows are expanded, make it contiguous")
    return s


def _ptr0(t):
    return 0 if t is None else t.data_ptr()


def _kv_pages(k_pages, v_pages, page_table, cu_seqlens, k_scale, v_scale):
    """The paged cache as gdr_kv_pages: (its fields in order, H_kv, d, n_seq)."""
    dtype, shape = k_pages.dtype, k_pages.shape
    if dtype is torch.bfloat16:
        code = GDR_BF16
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale are given with float8_e4m3fn pages only")
    elif dtype is torch.float8_e4m3fn:
        code = GDR_E4M3
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise ValueError(f"float8_e4m3fn pages need {name}")
            if t.dtype is not torch.float32 or t.shape != shape[:3] or not t.is_contiguous():
                raise ValueError(f"{name} must be a packed fp32 [n_pages, H_kv, page_size] tensor")
    else:
        raise TypeError(f"k_pages: dtype {dtype} is not bf16 or float8_e4m3fn")
    if v_pages.dtype is not dtype:
        raise TypeError("k_pages and v_pages must have one dtype")
    if len(shape) != 4 or v_pages.shape != shape or not k_pages.is_contiguous() \
            or not v_pages.is_contiguous():
        raise ValueError("k_pages and v_pages must be packed [n_pages, H_kv, page_size, d] tensors")
    if page_table.dtype is not torch.int32 or cu_seqlens.dtype is not torch.int32:
        raise TypeError("page_table and cu_seqlens must be int32")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seq, table_width]")
    n_seq, width = page_table.shape
    table_stride = 0
    if not page_table.is_contiguous():
        if width > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table must have packed rows")
        table_stride = page_table.stride(0) if n_seq > 1 else 0
        if n_seq > 1 and table_stride < width:
            raise ValueError("page_table's rows must not overlap (an expanded table: make it "
                             "contiguous)")
    if cu_seqlens.shape != (n_seq + 1,) or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must hold n_seq + 1 entries")
    fields = (n_seq, shape[1], shape[3], shape[2], shape[0], width, code, 0, table_stride,
              k_pages.data_ptr(), v_pages.data_ptr(), _ptr0(k_scale), _ptr0(v_scale),
              page_table.data_ptr(), cu_seqlens.data_ptr())
    return fields, shape[1], shape[3], n_seq


def _rows_bf16(t, name, shape):
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bf16")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")


def _per_seq(t, name, n_seq):
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.shape != (n_seq,) or not t.is_contiguous():
        raise ValueError(f"{name} must hold n_seq entries")


def _status_word(status):
    if status is not None and (status.dtype is not torch.int32 or status.numel() < 1):
        raise TypeError("status must be int32")


# The current stream's handle without a Stream object around it, where torch has that call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


_no_change = contextlib.nullcontext()


def _made_current(index):
    """A context in which CUDA device `index` is the current one (a CPU's -1: no change)."""
    return _no_change if index < 0 or index == torch.cuda.current_device() else torch.cuda.device(index)


def _queue(f, name, packed, more, stream, *tensors):
    """Call library function f on one device's stream: all tensors' device, made current."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on one device: {tensors[0].device} and {t.device}")
    # (Without a GPU the library's own checks run, and its launch fails.)
    if index < 0 and torch.cuda.is_available():
        raise ValueError(f"{name}: tensors must be on a CUDA device, not {tensors[0].device}")
    if stream is None:
        handle = _raw_stream(index) if index >= 0 else 0
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    with _made_current(index):
        status = f(packed, *more, handle)
    if status:
        raise GdrError(status, name)


def kv_append(k, v, k_pages, v_pages, page_table, cu_seqlens, cache_len, *, k_scale=None,
              v_scale=None, q=None, q_out=None, rot_dim=64, rope_theta=1e7, status=None,
              stream=None):
    """Write the new tokens of packed sequences into a paged cache (gdr_kv_append).

    k, v [n_tok, H_kv, 256] bf16: sequence s's new tokens are rows
    cu_seqlens[s] .. cu_seqlens[s+1]-1, at positions cache_len[s] + i; k is rotated
    (first ``rot_dim`` dims).  k_pages, v_pages [n_pages, H_kv, page_size, 256]: bf16,
    or float8_e4m3fn with k_scale, v_scale [n_pages, H_kv, page_size] fp32, then each
    row is stored as codes of x / scale with scale = max|x| / 448.  page_table
    [n_seq, table_width], cu_seqlens [n_seq + 1], cache_len [n_seq]: int32 on the
    device; cache_len is not updated.  ``q``, ``q_out`` [n_tok, H_q, 256] bf16: q_out
    receives q rotated the same way (it may be q).  ``status``: a device int32,
    written only when a token has no valid page.  Returns q_out.
    """
    pages, H_kv, d, n_seq = _kv_pages(k_pages, v_pages, page_table, cu_seqlens, k_scale, v_scale)
    n = k.shape[0]
    kv_shape = (n, H_kv, d)
    _rows_bf16(k, "k", kv_shape)
    _rows_bf16(v, "v", kv_shape)
    H_q = q_stride = q_out_stride = 0
    if q is not None:
        if q_out is None or q.dim() != 3:
            raise ValueError("q [n_tok, H_q, d] and q_out are given together")
        H_q = q.shape[1]
        shape = (n, H_q, d)
        _rows_bf16(q, "q", shape)
        _rows_bf16(q_out, "q_out", shape)
        q_stride, q_out_stride = _distinct_rows(q, "q"), _distinct_rows(q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q and q_out are given together")
    _per_seq(cache_len, "cache_len", n_seq)
    _status_word(status)
    a = _PACK_APPEND.pack(*pages, n, H_q, int(rot_dim), rope_theta, 0, q_stride, q_out_stride,
                          _distinct_rows(k, "k"), _distinct_rows(v, "v"), _ptr0(q), k.data_ptr(),
                          v.data_ptr(), _ptr0(q_out), cache_len.data_ptr(), _ptr0(status))
    _queue(_abi.lib().gdr_kv_append, "gdr_kv_append", a, (), stream, k, v, k_pages, v_pages,
           page_table, cu_seqlens, cache_len, k_scale, v_scale, q, q_out, status)
    return q_out


def kv_gather(k_pages, v_pages, page_table, cu_seqlens, k_out, v_out, *, k_scale=None,
              v_scale=None, first=None, status=None, stream=None):
    """Read cached tokens back into packed rows (gdr_kv_gather).

    Row cu_seqlens[s] + i of k_out, v_out [n_tok, H_kv, 256] (bf16 or fp32; either may
    be None) receives token first[s] + i of sequence s (``first`` int32 [n_seq] on the
    device; None: from token 0).  The cache's tensors are those of kv_append.
    Returns (k_out, v_out).
    """
    pages, H_kv, d, n_seq = _kv_pages(k_pages, v_pages, page_table, cu_seqlens, k_scale, v_scale)
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("one of k_out and v_out is needed")
    n = some.shape[0]
    strides = []
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            strides.append(0)
            continue
        if t.dtype is not some.dtype:
            raise TypeError("k_out and v_out must have one dtype")
        if t.shape != (n, H_kv, d):
            raise ValueError(f"{name} must be [n_tok, H_kv, d]")
        strides.append(_distinct_rows(t, name))
    if first is not None:
        _per_seq(first, "first", n_seq)
    _status_word(status)
    a = _PACK_GATHER.pack(*pages, n, _dtype_code(some, "k_out"), 0, *strides, _ptr0(k_out),
                          _ptr0(v_out), _ptr0(first), _ptr0(status))
    _queue(_abi.lib().gdr_kv_gather, "gdr_kv_gather", a, (), stream, some, v_out, k_pages, v_pages,
           page_table, cu_seqlens, k_scale, v_scale, first, status)
    return k_out, v_out


def _attn_paged_args(q, k_pages, v_pages, page_table, cu_seqlens, cache_len, out, k_scale, v_scale,
                     gate, lse, scale):
    pages, H_kv, d, n_seq = _kv_pages(k_pages, v_pages, page_table, cu_seqlens, k_scale, v_scale)
    if q.dim() != 3:
        raise ValueError("q must be [n_tok, H_q, d]")
    n, H_q, _ = shape = q.shape
    _rows_bf16(q, "q", (n, H_q, d))
    gate_stride = lse_stride = 0
    if gate is not None:
        _rows_bf16(gate, "gate", shape)
        gate_stride = _distinct_rows(gate, "gate")
    if out.shape != shape:
        raise ValueError("out must have q's shape")
    if lse is not None:
        _f32_tensor(lse, "lse")
        if lse.shape != (n, H_q):
            raise ValueError("lse must be [n_tok, H_q]")
        lse_stride = _distinct_rows(lse, "lse")
    _per_seq(cache_len, "cache_len", n_seq)
    return _PACK_ATTN.pack(*pages, n, H_q, _dtype_code(out, "out"), d ** -0.5 if scale is None else scale,
                           0, _distinct_rows(q, "q"), gate_stride, _distinct_rows(out, "out"),
                           lse_stride, q.data_ptr(), _ptr0(gate), cache_len.data_ptr(),
                           out.data_ptr(), _ptr0(lse))


def attn_paged_workspace_size(q, k_pages, v_pages, page_table, cu_seqlens, cache_len, out, *,
                              k_scale=None, v_scale=None, gate=None, lse=None, scale=None) -> int:
    a = _attn_paged_args(q, k_pages, v_pages, page_table, cu_seqlens, cache_len, out, k_scale,
                         v_scale, gate, lse, scale)
    n = ctypes.c_size_t(0)
    with _made_current(q.get_device()):
        _check(_abi.lib().gdr_attn_paged_workspace_size(a, ctypes.byref(n)),
               "gdr_attn_paged_workspace_size")
    return int(n.value)


def attn_paged(q, k_pages, v_pages, page_table, cu_seqlens, cache_len, out, *, k_scale=None,
               v_scale=None, gate=None, lse=None, scale=None, workspace=None,
               stream=None) -> torch.Tensor:
    """The new tokens of packed sequences attend over their pages (gdr_attn_paged).

    q [n_tok, H_q, 256] bf16, rotated (kv_append's q_out): sequence s's new tokens are
    rows cu_seqlens[s] .. cu_seqlens[s+1]-1, the last tokens of its cache (append them
    first); row i attends tokens 0 .. cache_len[s] + i.  ``gate`` [n_tok, H_q, 256] bf16
    or None: the output is multiplied by sigmoid(gate).  out [n_tok, H_q, 256] bf16 or
    fp32; ``lse`` [n_tok, H_q] fp32 or None receives the log of the softmax sums.  The
    cache's tensors are those of kv_append.  ``workspace``: a uint8 device tensor of
    attn_paged_workspace_size() bytes (about 39 MB, whatever the lengths), allocated
    here when None; its first 4 bytes (int32) are the call's status word.
    """
    a = _attn_paged_args(q, k_pages, v_pages, page_table, cu_seqlens, cache_len, out, k_scale,
                         v_scale, gate, lse, scale)
    L = _abi.lib()
    if workspace is None:
        n = ctypes.c_size_t(0)
        with _made_current(q.get_device()):
            _check(L.gdr_attn_paged_workspace_size(a, ctypes.byref(n)),
                   "gdr_attn_paged_workspace_size")
        if n.value:
            workspace = _workspace(int(n.value), stream, q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _queue(L.gdr_attn_paged, "gdr_attn_paged", a, (_ptr0(workspace), ws_bytes), stream, q, k_pages,
           v_pages, page_table, cu_seqlens, cache_len, out, k_scale, v_scale, gate, lse, workspace)
    return out


def _moe_args(x, w_router, w_gate_up, w_down, out, top_k, shared, topk_idx, topk_w):
    n_tok, H = x.shape
    E = w_router.shape[0]
    I = w_gate_up.shape[1] // 2
    for t, name in ((x, "x"), (w_router, "w_router"), (w_gate_up, "w_gate_up"),
                    (w_down, "w_down")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bf16")
    for t, name, shape in ((w_router, "w_router", (E, H)), (w_gate_up, "w_gate_up", (E, 2 * I, H)),
                           (w_down, "w_down", (E, H, I))):
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a packed {list(shape)} tensor")
    ws_gate_up = ws_down = w_sgate = None
    SI = 0
    if shared is not None:
        ws_gate_up, ws_down, w_sgate = shared
        SI = ws_gate_up.shape[0] // 2
        for t, name, shape in ((ws_gate_up, "ws_gate_up", (2 * SI, H)), (ws_down, "ws_down", (H, SI)),
                               (w_sgate, "w_sgate", (H,))):
            if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a packed bf16 {list(shape)} tensor")
    if topk_idx is not None and topk_idx.dtype != torch.int32:
        raise TypeError("topk_idx must be int32")
    _f32_tensor(topk_w, "topk_w")
    return _abi.MoeArgs(
        n_tok=n_tok, hidden=H, n_exp=E, top_k=int(top_k), inter=I, s_inter=SI,
        out_dtype=_dtype_code(out, "out"), reserved=0,
        x_stride=_row_stride(x, "x"), out_stride=_row_stride(out, "out"),
        x=_ptr(x), w_router=_ptr(w_router), w_gate_up=_ptr(w_gate_up), w_down=_ptr(w_down),
        ws_gate_up=_ptr(ws_gate_up), ws_down=_ptr(ws_down), w_sgate=_ptr(w_sgate), out=_ptr(out),
        topk_idx=_ptr(topk_idx), topk_w=_ptr(topk_w))


def moe_workspace_size(x, w_router, w_gate_up, w_down, out, *, top_k=8, shared=None) -> int:
    a = _moe_args(x, w_router, w_gate_up, w_down, out, top_k, shared, None, None)
    n = ctypes.c_size_t(0)
    _check(_abi.lib().gdr_moe_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "gdr_moe_workspace_size")
    return int(n.value)


def moe_decode(x, w_router, w_gate_up, w_down, out, *, top_k=8, shared=None, topk_idx=None,
               topk_w=None, workspace=None, stream=None) -> torch.Tensor:
    """The routed-expert MoE block for a decode batch (gdr_moe_decode).

    x [n_tok, hidden] bf16; w_router [n_exp, hidden]; w_gate_up [n_exp, 2*inter,
    hidden] (gate rows, then up rows); w_down [n_exp, hidden, inter], all bf16;
    ``shared`` = (ws_gate_up [2*s_inter, hidden], ws_down [hidden, s_inter],
    w_sgate [hidden]) bf16 or None; out [n_tok, hidden] bf16 or fp32;
    ``topk_idx`` (int32) / ``topk_w`` (fp32) [n_tok, top_k] receive the routing.
    """
    a = _moe_args(x, w_router, w_gate_up, w_down, out, top_k, shared, topk_idx, topk_w)
    L = _abi.lib()
    n = ctypes.c_size_t(0)
    _check(L.gdr_moe_workspace_size(ctypes.byref(a), ctypes.byref(n)), "gdr_moe_workspace_size")
    if workspace is None and n.value:
        workspace = _workspace(int(n.value), stream, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(L.gdr_moe_decode(ctypes.byref(a), _ptr(workspace), ws_bytes, _stream(stream, x.device)),
           "gdr_moe_decode")
    return out
