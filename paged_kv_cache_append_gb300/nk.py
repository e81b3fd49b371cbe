"""Thin Python binding of the libnk C ABI (``include/nk.h``).

Argument marshalling only: every step of the hot path runs in libnk's CUDA
kernels.  Functions named ``nk_*`` mirror the C entry points one to one and
take raw integers for device pointers and streams; ``Pool`` is a convenience
wrapper that allocates the planes as torch tensors (device memory), keeps them
alive and passes ``torch.cuda.current_stream()``.  A call with ``stream=`` runs
on that stream: what it allocates (outputs, a workspace) belongs to it, and the
caller orders the given tensors' other uses against it.

There is no CPU fallback: ``load()`` raises when ``libnk.so`` has not been
built, and every call raises ``NkError`` on a non-zero status.
"""

from __future__ import annotations

import contextlib
import ctypes as C
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libnk.so")

NK_OK = 0
ERRORS = {-1: "NK_ERR_INVALID_ARG", -2: "NK_ERR_SHAPE", -3: "NK_ERR_RANGE",
          -4: "NK_ERR_UNSUPPORTED", -5: "NK_ERR_ALIGN", -6: "NK_ERR_CUDA", -7: "NK_ERR_WORKSPACE"}
STATUS_PAGE_RANGE, STATUS_FRONTIER, STATUS_TIMEOUT = 1, 2, 4
STATUS_TOKEN_RANGE, STATUS_PREFIX, STATUS_PAGES = 8, 16, 32
PROFILES = {"bf16": 0, "int8_g64": 1, "fp8_row": 2, "nvfp4_g16": 3, "k8v4": 4}
POOL_CHECK_BOUNDS = 1

SYMBOLS = ["nk_version", "nk_last_error", "nk_pool_plane_bytes", "nk_pool_capacity_bounds",
           "nk_pool_mtp_pages", "nk_pages_needed",
           "nk_pool_create", "nk_pool_destroy", "nk_paged_kv_append", "nk_decode_workspace_bytes",
           "nk_paged_decode_attention", "nk_paged_append_decode_attention",
           "nk_paged_decode_attention_noalloc",
           "nk_prefill_workspace_bytes", "nk_paged_prefill_attention",
           "nk_page_copy_columns", "nk_status_read", "nk_host_page_bytes", "nk_page_runs",
           "nk_pages_to_host", "nk_pages_from_host", "nk_selftest_bounded_wait",
           "nk_shared_decode_workspace_bytes", "nk_paged_shared_decode_attention", "nk_qk_norm_rope",
           "nk_paged_kv_append_rope", "nk_verify_drafts", "nk_diff_decode_workspace_bytes",
           "nk_paged_diff_decode_attention", "nk_diff_prefill_workspace_bytes", "nk_paged_diff_prefill_attention",
           "nk_residual_norm", "nk_pages_grow"]


class NkError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


class PoolDesc(C.Structure):
    _fields_ = [("profile", C.c_int32), ("num_layers", C.c_int32), ("num_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("max_context", C.c_int32),
                ("max_concurrency", C.c_int32), ("order", C.c_int32), ("flags", C.c_int32)]


class Rows(C.Structure):
    """nk_rows: element (token n, head h, dim d) at ptr[n * token_stride + h * head_stride + d]."""
    _fields_ = [("ptr", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class RopeDesc(C.Structure):
    _fields_ = [("cos_sin", C.c_void_p), ("positions", C.c_int32), ("rotary_dim", C.c_int32),
                ("layout", C.c_int32), ("eps", C.c_float), ("weight_offset", C.c_float),
                ("reserved", C.c_int32), ("q_weight", C.c_void_p), ("k_weight", C.c_void_p)]


class DiffDesc(C.Structure):
    """nk_diff"""
    _fields_ = [("lam", C.c_void_p), ("lambda_stride", C.c_int64), ("norm_weight", C.c_void_p), ("eps", C.c_float),
                ("out_scale", C.c_float)]


class BlockNormDesc(C.Structure):
    """nk_block_norm"""
    _fields_ = [("weight", C.c_void_p), ("post_weight", C.c_void_p), ("eps", C.c_float), ("weight_offset", C.c_float),
                ("scale", C.c_float), ("residual_scale", C.c_float), ("sigmoid_gate", C.c_int32),
                ("residual_fp32", C.c_int32)]


_lib = None
_P, _I, _F, _S, _L = C.c_void_p, C.c_int32, C.c_float, C.c_size_t, C.c_int64


def load(path: str | None = None) -> C.CDLL:
    """Loads libnk.so (raises RuntimeError when it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run paged_kv_cache_append_gb300.build.build()")
    lib = C.CDLL(p)
    sig = {
        "nk_version": (C.c_int, []),
        "nk_last_error": (C.c_char_p, []),
        "nk_pool_plane_bytes": (C.c_int, [C.POINTER(PoolDesc), _I, C.POINTER(_I), C.POINTER(_S), C.POINTER(_S)]),
        "nk_pool_capacity_bounds": (C.c_int, [C.POINTER(PoolDesc), C.POINTER(_I), C.POINTER(_I)]),
        "nk_pool_create": (C.c_int, [C.POINTER(PoolDesc), _I, C.POINTER(_P), C.POINTER(_P)]),
        "nk_pool_destroy": (C.c_int, [_P]),
        "nk_paged_kv_append": (C.c_int, [_P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _P]),
        "nk_pool_mtp_pages": (C.c_int, [_I, _I, _I, C.POINTER(_I)]),
        "nk_pages_needed": (C.c_int, [_I, _I, C.POINTER(_I)]),
        "nk_host_page_bytes": (C.c_int, [_P, C.POINTER(_S)]),
        "nk_page_runs": (C.c_int, [_P, _I, _P, _P, C.POINTER(_I)]),
        "nk_pages_to_host": (C.c_int, [_P, _P, _I, _P, _P]),
        "nk_pages_from_host": (C.c_int, [_P, _P, _I, _P, _P]),
        "nk_decode_workspace_bytes": (C.c_int, [_P, _I, _I, _I, C.POINTER(_S)]),
        "nk_paged_decode_attention": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _I, _I, _F, _P, _P, _P, _S, _P]),
        "nk_paged_append_decode_attention": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _P, _P, _I, _I, _F, _P, _P, _P,
                                                       _S, _P]),
        "nk_paged_decode_attention_noalloc": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _I, _I, _F, _P, _P, _P]),
        "nk_prefill_workspace_bytes": (C.c_int, [_P, _I, _I, _I, C.POINTER(_S)]),
        "nk_paged_prefill_attention": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _P, _I, _I, _F, _P, _P, _P, _S, _P]),
        "nk_page_copy_columns": (C.c_int, [_P, _I, _I, _I, _P]),
        "nk_status_read": (C.c_int, [C.POINTER(_I), _I, _P]),
        "nk_selftest_bounded_wait": (C.c_int, [_I, _P, _P]),
        "nk_shared_decode_workspace_bytes": (C.c_int, [_P, _I, _I, _I, C.POINTER(_S)]),
        "nk_paged_shared_decode_attention": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _P, _I, _I, _F, _P, _P, _L, _P, _S,
                                                       _P]),
        "nk_qk_norm_rope": (C.c_int, [C.POINTER(RopeDesc), _I, C.POINTER(Rows), _I, C.POINTER(Rows), _I, _P, _I,
                                      C.POINTER(Rows), C.POINTER(Rows), _P]),
        "nk_paged_kv_append_rope": (C.c_int, [_P, _I, _P, _P, _P, _P, C.POINTER(RopeDesc), C.POINTER(Rows),
                                              C.POINTER(Rows), C.POINTER(Rows), _I, _P, _I, _I, _P]),
        "nk_verify_drafts": (C.c_int, [_P, _L, _P, _L, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
        "nk_diff_decode_workspace_bytes": (C.c_int, [_P, _I, _I, _I, C.POINTER(_S)]),
        "nk_paged_diff_decode_attention": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _I, _I, _F, C.POINTER(DiffDesc), _P,
                                                     _P, _P, _S, _P]),
        "nk_diff_prefill_workspace_bytes": (C.c_int, [_P, _I, _I, _I, C.POINTER(_S)]),
        "nk_paged_diff_prefill_attention": (C.c_int, [_P, _I, _P, _I, _P, _P, _P, _P, _I, _I, _F, C.POINTER(DiffDesc),
                                                      _P, _P, _P, _S, _P]),
        "nk_residual_norm": (C.c_int, [C.POINTER(BlockNormDesc), _I, _I, _P, _L, _P, _L, _P, _L, _P, _L, _P, _L, _P]),
        "nk_pages_grow": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


def _check(rc: int) -> None:
    if rc != NK_OK:
        raise NkError(rc, load().nk_last_error().decode())


ORDERS = {"page_major": 0, "head_major": 1}


def make_desc(profile, num_layers, num_kv_heads, head_dim, max_context, max_concurrency,
              flags: int = 0, order: str = "page_major") -> PoolDesc:
    prof = PROFILES[profile] if isinstance(profile, str) else int(profile)
    return PoolDesc(prof, num_layers, num_kv_heads, head_dim, max_context, max_concurrency,
                    ORDERS[order], flags)


# ----------------------------------------------------------- C-named wrappers

def nk_version() -> int:
    return load().nk_version()


def nk_pool_plane_bytes(desc: PoolDesc, M: int):
    n = _I()
    b = (_S * 4)()
    rb = (_S * 4)()
    _check(load().nk_pool_plane_bytes(C.byref(desc), M, C.byref(n), b, rb))
    return n.value, list(b)[:n.value], list(rb)[:n.value]


def nk_pool_capacity_bounds(desc: PoolDesc):
    lo, hi = _I(), _I()
    _check(load().nk_pool_capacity_bounds(C.byref(desc), C.byref(lo), C.byref(hi)))
    return lo.value, hi.value


def nk_pool_create(desc: PoolDesc, M: int, plane_ptrs) -> int:
    arr = (_P * len(plane_ptrs))(*plane_ptrs)
    out = _P()
    _check(load().nk_pool_create(C.byref(desc), M, arr, C.byref(out)))
    return out.value


def nk_pool_destroy(pool: int) -> None:
    _check(load().nk_pool_destroy(pool))


def nk_paged_kv_append(pool, layer, block_tables, table_rows, write_pos, counts, k, v, B, T, stream):
    _check(load().nk_paged_kv_append(pool, layer, block_tables, table_rows, write_pos, counts,
                                     k, v, B, T, stream))


def nk_pool_mtp_pages(M, C_rows, draft_window) -> int:
    n = _I()
    _check(load().nk_pool_mtp_pages(M, C_rows, draft_window, C.byref(n)))
    return n.value


def nk_pages_needed(committed_frontier, provisional_frontier) -> int:
    n = _I()
    _check(load().nk_pages_needed(committed_frontier, provisional_frontier, C.byref(n)))
    return n.value


def nk_page_runs(page_ids):
    """Runs of consecutive physical ids: list of (first logical page, length)."""
    import numpy as np
    ids = np.ascontiguousarray(page_ids, dtype=np.int32)
    n = ids.size
    first = np.zeros(max(n, 1), np.int32)
    ln = np.zeros(max(n, 1), np.int32)
    nr = _I()
    _check(load().nk_page_runs(ids.ctypes.data, n, first.ctypes.data, ln.ctypes.data, C.byref(nr)))
    return [(int(first[r]), int(ln[r])) for r in range(nr.value)]


def nk_decode_workspace_bytes(pool, B, T, Hq) -> int:
    n = _S()
    _check(load().nk_decode_workspace_bytes(pool, B, T, Hq, C.byref(n)))
    return n.value


def nk_paged_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers, B, T, scale,
                              out, lse, workspace, workspace_bytes, stream):
    _check(load().nk_paged_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers,
                                            B, T, scale, out, lse, workspace, workspace_bytes, stream))


def nk_paged_append_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers, k, v, B,
                                     T, scale, out, lse, workspace, workspace_bytes, stream):
    _check(load().nk_paged_append_decode_attention(q, Hq, pool, layer, block_tables, table_rows,
                                                   frontiers, k, v, B, T, scale, out, lse, workspace,
                                                   workspace_bytes, stream))


def nk_paged_decode_attention_noalloc(q, Hq, pool, layer, block_tables, table_rows, frontiers, B, T,
                                      scale, out, lse, stream):
    _check(load().nk_paged_decode_attention_noalloc(q, Hq, pool, layer, block_tables, table_rows,
                                                    frontiers, B, T, scale, out, lse, stream))


def nk_prefill_workspace_bytes(pool, B, Tc, Hq) -> int:
    n = _S()
    _check(load().nk_prefill_workspace_bytes(pool, B, Tc, Hq, C.byref(n)))
    return n.value


def nk_paged_prefill_attention(q, Hq, pool, layer, block_tables, table_rows, prefix_len, chunk_len,
                               B, Tc, scale, out, lse, workspace, workspace_bytes, stream):
    _check(load().nk_paged_prefill_attention(q, Hq, pool, layer, block_tables, table_rows, prefix_len,
                                             chunk_len, B, Tc, scale, out, lse, workspace,
                                             workspace_bytes, stream))


def nk_shared_decode_workspace_bytes(pool, B, T, Hq) -> int:
    n = _S()
    _check(load().nk_shared_decode_workspace_bytes(pool, B, T, Hq, C.byref(n)))
    return n.value


def nk_paged_shared_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers, shared_pages,
                                     B, T, scale, out, lse, share_from, workspace, workspace_bytes, stream):
    _check(load().nk_paged_shared_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers,
                                                   shared_pages, B, T, scale, out, lse, share_from, workspace,
                                                   workspace_bytes, stream))


def nk_qk_norm_rope(rope, head_dim, q, Hq, k, H, positions, N, q_out, k_out, stream):
    """rope: RopeDesc; q, k, q_out, k_out: Rows or None."""
    _check(load().nk_qk_norm_rope(rope, head_dim, q, Hq, k, H, positions, N, q_out, k_out, stream))


def nk_paged_kv_append_rope(pool, layer, block_tables, table_rows, write_pos, counts, rope, k, v, q, Hq, q_out,
                            B, T, stream):
    """rope: RopeDesc; k, v, q: Rows (q may be None)."""
    _check(load().nk_paged_kv_append_rope(pool, layer, block_tables, table_rows, write_pos, counts, rope, k, v,
                                          q, Hq, q_out, B, T, stream))


def nk_verify_drafts(target, target_stride, draft, draft_stride, tokens, draft_len, uniforms, frontiers, B, K, V,
                     accepted, out_tokens, frontiers_out, stream):
    _check(load().nk_verify_drafts(target, target_stride, draft, draft_stride, tokens, draft_len, uniforms,
                                   frontiers, B, K, V, accepted, out_tokens, frontiers_out, stream))


def nk_diff_decode_workspace_bytes(pool, B, T, Hq) -> int:
    n = _S()
    _check(load().nk_diff_decode_workspace_bytes(pool, B, T, Hq, C.byref(n)))
    return n.value


def nk_paged_diff_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers, B, T, scale, diff, out,
                                   lse, workspace, workspace_bytes, stream):
    """diff: DiffDesc."""
    _check(load().nk_paged_diff_decode_attention(q, Hq, pool, layer, block_tables, table_rows, frontiers, B, T, scale,
                                                 diff, out, lse, workspace, workspace_bytes, stream))


def nk_diff_prefill_workspace_bytes(pool, B, Tc, Hq) -> int:
    n = _S()
    _check(load().nk_diff_prefill_workspace_bytes(pool, B, Tc, Hq, C.byref(n)))
    return n.value


def nk_paged_diff_prefill_attention(q, Hq, pool, layer, block_tables, table_rows, prefix_len, chunk_len, B, Tc, scale,
                                    diff, out, lse, workspace, workspace_bytes, stream):
    """diff: DiffDesc."""
    _check(load().nk_paged_diff_prefill_attention(q, Hq, pool, layer, block_tables, table_rows, prefix_len, chunk_len,
                                                  B, Tc, scale, diff, out, lse, workspace, workspace_bytes, stream))


def nk_residual_norm(norm, dim, N, y, y_stride, gate, gate_stride, residual, residual_stride, residual_out,
                     residual_out_stride, x_out, x_stride, stream):
    """norm: BlockNormDesc."""
    _check(load().nk_residual_norm(norm, dim, N, y, y_stride, gate, gate_stride, residual, residual_stride, residual_out,
                                   residual_out_stride, x_out, x_stride, stream))


def nk_pages_grow(pool, block_tables, table_rows, committed, counts, keep, mapped, mapped_out, free_pages, free_count,
                  free_count_out, B, T, frontiers, positions, slots, stream):
    _check(load().nk_pages_grow(pool, block_tables, table_rows, committed, counts, keep, mapped, mapped_out, free_pages,
                                free_count, free_count_out, B, T, frontiers, positions, slots, stream))


def nk_page_copy_columns(pool, src, dst, ncols, stream):
    _check(load().nk_page_copy_columns(pool, src, dst, ncols, stream))


def nk_status_read(clear: bool = True, stream=None) -> int:
    s = _I()
    _check(load().nk_status_read(C.byref(s), int(clear), stream))
    return s.value


def nk_selftest_bounded_wait(limit_us: int, waited_ns_ptr=None, stream=None) -> None:
    _check(load().nk_selftest_bounded_wait(int(limit_us), waited_ns_ptr, stream))


# ------------------------------------------------------------ torch wrapper

def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_raw_stream = None


def _current_stream(device: int) -> int:
    """Handle of the current stream of a device, without building a Stream object where torch can do without."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _stream(stream) -> int:
    import torch
    return stream.cuda_stream if stream is not None else _current_stream(torch.cuda.current_device())


def _on(stream):
    """Where a call on `stream` (None: the current one) makes its tensors: in
    that stream's order, so that the block they get is free by the time the
    call runs and is not handed out again before it has."""
    import torch
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _handle(stream, dev: int) -> int:
    """Stream handle of a call on device `dev`."""
    if stream is None:
        return _current_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: expected a stream of device {dev}, got one of device {stream.device_index}")
    return stream.cuda_stream


_pyargs = None


def _args():
    """The CPython module that checks and marshals tensor arguments (csrc/pyargs.c)."""
    global _pyargs
    if _pyargs is None:
        import torch

        try:
            from . import _pyargs as m
        except ImportError as e:
            raise RuntimeError("_pyargs is not built; run paged_kv_cache_append_gb300.build.build()") from e
        lib = load()
        m.init(*(C.cast(f, C.c_void_p).value for f in (
            lib.nk_qk_norm_rope, lib.nk_paged_kv_append_rope, lib.nk_paged_shared_decode_attention, lib.nk_verify_drafts,
            lib.nk_paged_diff_decode_attention, lib.nk_paged_diff_prefill_attention, lib.nk_residual_norm,
            lib.nk_pages_grow)), torch.bfloat16, torch.float32, torch.int32, torch.int64)
        _pyargs = m
    return _pyargs


class Rope:
    """Norm and rotation of head rows (nk.h, nk_rope).

    ``cos_sin`` is a contiguous fp32 CUDA tensor [positions, rotary_dim] whose
    row is the cosines of the rotary_dim / 2 angles, then their sines; the
    weights are bf16 [D] or None (no norm).  Keeps its tensors alive.
    """

    def __init__(self, cos_sin, rotary_dim: int, interleaved: bool = False, q_weight=None, k_weight=None,
                 eps: float = 1e-6, weight_offset: float = 0.0):
        import torch
        if cos_sin.dtype != torch.float32 or not cos_sin.is_cuda or not cos_sin.is_contiguous() \
                or cos_sin.dim() != 2 or cos_sin.shape[1] != rotary_dim:
            raise ValueError(f"cos_sin must be a contiguous fp32 CUDA tensor [positions, {rotary_dim}]")
        for w in (q_weight, k_weight):
            if w is not None and (w.dtype != torch.bfloat16 or w.device != cos_sin.device or w.dim() != 1
                                  or not w.is_contiguous()):
                raise ValueError("norm weights must be contiguous bf16 vectors on the table's device")
        if q_weight is not None and k_weight is not None and q_weight.numel() != k_weight.numel():
            raise ValueError("the norm weights must have one size")
        w = q_weight if q_weight is not None else k_weight
        self.cos_sin, self.q_weight, self.k_weight = cos_sin, q_weight, k_weight
        self.device = cos_sin.get_device()
        self.head_dim = 0 if w is None else w.numel()   # 0: any
        self.desc = RopeDesc(_ptr(cos_sin), cos_sin.shape[0], rotary_dim, int(interleaved), eps, weight_offset, 0,
                             _ptr(q_weight), _ptr(k_weight))
        self.address = C.addressof(self.desc)


def qk_norm_rope(q, k, positions, rope: Rope, q_out=None, k_out=None, stream=None):
    """Per-head norm and rotation of q [N, Hq, D] and k [N, H, D] (bf16, any
    token and head strides) at ``positions`` int32 [N]; returns (q_out, k_out),
    new contiguous tensors unless given (q_out may be q itself, k_out k)."""
    import torch
    dev = rope.device
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return qk_norm_rope(q, k, positions, rope, q_out, k_out, stream)
    at = _handle(stream, dev)
    if q_out is None or k_out is None:
        with _on(stream):
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _check((_pyargs or _args()).norm_rope(q, k, positions, q_out, k_out, rope.address, rope.head_dim, dev, at))
    return q_out, k_out


def _verify_outputs(target, frontiers):
    import torch
    B, K1, _ = target.shape
    out = torch.empty((B, K1), dtype=torch.int32, device=target.device)
    if frontiers is None:
        return torch.empty(B, dtype=torch.int32, device=target.device), out, None
    return torch.empty_like(frontiers), out, torch.empty_like(frontiers)


def verify_drafts(target, tokens, uniforms, draft=None, draft_len=None, frontiers=None, stream=None):
    """Verification of drafted tokens (nk.h, nk_verify_drafts).

    target fp32 [B, K+1, V] and draft fp32 [B, K, V] or None (their rows may be
    padded: any row stride, contiguous batches of rows), tokens int32 [B, K],
    uniforms fp32 [B, K+1], draft_len and frontiers int32 [B] or None.
    Returns (accepted [B], tokens [B, K+1], frontiers [B] or None), int32.
    """
    import torch
    dev = target.get_device()
    if dev < 0:
        raise ValueError("target: expected a CUDA tensor")
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return verify_drafts(target, tokens, uniforms, draft, draft_len, frontiers, stream)
    at = _handle(stream, dev)
    if stream is None:
        accepted, out, after = _verify_outputs(target, frontiers)
    else:
        with _on(stream):
            accepted, out, after = _verify_outputs(target, frontiers)
    _check((_pyargs or _args()).verify(target, draft, tokens, draft_len, uniforms, frontiers, accepted, out, after, dev,
                                       at))
    return accepted, out, after


class Diff:
    """What a differential attention has besides queries and pages (nk.h, nk_diff).

    ``lam`` is fp32: [heads] (the same for every token) or [..., heads], a row
    for each token of the call; ``norm_weight`` bf16 [2 D] or None (no norm).
    Keeps its tensors alive.
    """

    def __init__(self, lam, norm_weight=None, eps: float = 1e-5, out_scale: float = 1.0):
        import torch
        if lam.dtype != torch.float32 or not lam.is_cuda or not lam.is_contiguous() or lam.dim() < 1 \
                or lam.numel() < 1:
            raise ValueError("lam must be a contiguous fp32 CUDA tensor [..., heads]")
        if norm_weight is not None and (norm_weight.dtype != torch.bfloat16 or norm_weight.device != lam.device
                                        or norm_weight.dim() != 1 or not norm_weight.is_contiguous()):
            raise ValueError("norm_weight must be a contiguous bf16 vector on lam's device")
        self.lam, self.norm_weight = lam, norm_weight
        self.device, self.heads = lam.get_device(), lam.shape[-1]
        self.tokens = 0 if lam.dim() == 1 else lam.numel() // self.heads   # 0: the same for every token
        self.width = 0 if norm_weight is None else norm_weight.numel()     # 0: any
        self.desc = DiffDesc(_ptr(lam), self.heads if lam.dim() > 1 else 0, _ptr(norm_weight), eps, out_scale)
        self.address = C.addressof(self.desc)

    @classmethod
    def from_vectors(cls, q1, k1, q2, k2, lambda_init: float, heads: int, norm_weight=None, eps: float = 1e-5):
        """lambda = exp(q1 . k1) - exp(q2 . k2) + lambda_init from learned vectors [D] or [heads, D], once per
        model; the output is scaled by 1 - lambda_init."""
        import torch
        dot = [(a.double() * b.double()).sum(-1).exp() for a, b in ((q1, k1), (q2, k2))]
        lam = (dot[0] - dot[1] + lambda_init).to(torch.float32).expand(heads).contiguous()
        return cls(lam, norm_weight, eps, 1.0 - lambda_init)


class ResidualNorm:
    """Norms, gate and scales around a block (nk.h, nk_block_norm).

    ``weight`` and ``post_weight`` are bf16 [dim]; without ``weight`` only the
    residual is updated.  Keeps its tensors alive.
    """

    def __init__(self, weight, post_weight=None, eps: float = 1e-6, scale: float = 1.0, residual_scale: float = 1.0,
                 weight_offset: float = 0.0, sigmoid_gate: bool = False):
        import torch
        given = [w for w in (weight, post_weight) if w is not None]
        for w in given:
            if w.dtype != torch.bfloat16 or not w.is_cuda or w.device != given[0].device or w.dim() != 1 \
                    or not w.is_contiguous() or w.numel() != given[0].numel():
                raise ValueError("norm weights must be contiguous bf16 CUDA vectors of one size on one device")
        self.weight, self.post_weight = weight, post_weight
        self.dim = given[0].numel() if given else 0                  # 0: any
        self.device = given[0].get_device() if given else None      # None: any
        desc = (_ptr(weight), _ptr(post_weight), eps, weight_offset, scale, residual_scale, int(sigmoid_gate))
        self.descs = BlockNormDesc(*desc, 0), BlockNormDesc(*desc, 1)   # a bf16 residual, an fp32 one
        self.addresses = tuple(C.addressof(d) for d in self.descs)


def residual_norm(y, residual, norm: ResidualNorm, gate=None, out=None, residual_out=None, stream=None):
    """h = residual_scale * residual + scale * act(gate) * post(y) and x, its norm (nk.h, nk_residual_norm).

    y bf16 [N, dim] or [B, T, dim] or None; residual of the same sizes, bf16 or
    fp32; gate bf16 of the same sizes or [dim], or None.  Rows may be padded (any
    row stride, one for all tokens).  Returns (x, h): new contiguous tensors
    unless given (residual_out may be residual itself, out may be y); x is None
    without a weight.
    """
    import torch
    dev = residual.get_device()
    if dev < 0:
        raise ValueError("residual: expected a CUDA tensor")
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return residual_norm(y, residual, norm, gate, out, residual_out, stream)
    if norm.device is not None and norm.device != dev:
        raise ValueError("the norm weights are on another device than the residual")
    if norm.weight is None and out is not None:
        raise ValueError("out: there is no norm weight to make it with")
    at = _handle(stream, dev)
    if residual_out is None or (out is None and norm.weight is not None):
        with _on(stream):
            if residual_out is None:
                residual_out = torch.empty(residual.shape, dtype=residual.dtype, device=residual.device)
            if out is None and norm.weight is not None:
                out = torch.empty(residual.shape, dtype=torch.bfloat16, device=residual.device)
    wide = residual.dtype == torch.float32
    _check((_pyargs or _args()).residual_norm(norm.addresses[wide], norm.dim, y, residual, gate, out, residual_out,
                                              wide, dev, at))
    return out, residual_out


class Pool:
    """A typed growing KV pool whose planes are torch uint8 device tensors.

    ``planes[layer][i]`` follows nk.h's plane order [K code, V code, K scale,
    V scale]; ``tables`` etc. are int32 device tensors owned by the caller.
    """

    def __init__(self, profile: str, num_layers: int, num_kv_heads: int, head_dim: int,
                 max_context: int, max_concurrency: int, M: int, device="cuda",
                 check_bounds: bool = False, order: str = "page_major"):
        import torch
        self.profile, self.num_layers, self.H, self.D = profile, num_layers, num_kv_heads, head_dim
        self.S, self.C, self.M = max_context, max_concurrency, M
        self.L = -(-max_context // 64)
        self.order = order
        self.desc = make_desc(profile, num_layers, num_kv_heads, head_dim, max_context,
                              max_concurrency, POOL_CHECK_BOUNDS if check_bounds else 0, order)
        self.n_planes, self.plane_bytes, self.row_bytes = nk_pool_plane_bytes(self.desc, M)
        self.planes = [[torch.zeros(nb, dtype=torch.uint8, device=device) for nb in self.plane_bytes]
                       for _ in range(num_layers)]
        self.device = self.planes[0][0].get_device()
        ptrs = [p.data_ptr() for layer in self.planes for p in layer]
        self.handle = nk_pool_create(self.desc, M, ptrs)
        self._ws = None

    def close(self) -> None:
        if self.handle:
            nk_pool_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def kv_bytes_per_token_head(self) -> int:
        return int(sum(self.row_bytes))

    def append(self, layer, tables, table_rows, write_pos, k, v, counts=None, stream=None):
        B, T = k.shape[0], k.shape[1]
        nk_paged_kv_append(self.handle, layer, _ptr(tables), _ptr(table_rows), _ptr(write_pos),
                           _ptr(counts), _ptr(k), _ptr(v), B, T, _stream(stream))

    def workspace(self, B, T, Hq):
        """The workspace that ``decode`` and ``append_decode`` use unless given
        one: one for all calls of this pool, which then must not overlap."""
        import torch
        n = nk_decode_workspace_bytes(self.handle, B, T, Hq)
        if self._ws is None or self._ws.numel() < n:   # zero-filled once (split counters)
            self._ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=self.planes[0][0].device)
        return self._ws

    def decode(self, layer, q, tables, table_rows, frontiers, scale, out=None, lse=None,
               workspace=None, stream=None):
        import torch
        B, T, Hq, D = q.shape
        ws = workspace
        if out is None or lse is None or ws is None:
            with _on(stream):
                if out is None:
                    out = torch.empty_like(q)
                if lse is None:
                    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
                if ws is None:
                    ws = self.workspace(B, T, Hq)
        nk_paged_decode_attention(_ptr(q), Hq, self.handle, layer, _ptr(tables), _ptr(table_rows),
                                  _ptr(frontiers), B, T, float(scale), _ptr(out), _ptr(lse),
                                  _ptr(ws), ws.numel(), _stream(stream))
        return out, lse

    def append_decode(self, layer, q, k, v, tables, table_rows, frontiers, scale, out=None, lse=None,
                      workspace=None, stream=None):
        """Appends the T new tokens k, v [B, T, H, D] of every row at
        frontiers - T .. frontiers - 1, then attends (one launch)."""
        import torch
        B, T, Hq, D = q.shape
        ws = workspace
        if out is None or lse is None or ws is None:
            with _on(stream):
                if out is None:
                    out = torch.empty_like(q)
                if lse is None:
                    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
                if ws is None:
                    ws = self.workspace(B, T, Hq)
        nk_paged_append_decode_attention(_ptr(q), Hq, self.handle, layer, _ptr(tables), _ptr(table_rows),
                                         _ptr(frontiers), _ptr(k), _ptr(v), B, T, float(scale), _ptr(out),
                                         _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
        return out, lse

    def host_page_bytes(self) -> int:
        n = _S()
        _check(load().nk_host_page_bytes(self.handle, C.byref(n)))
        return n.value

    def pages_to_host(self, page_ids, host, stream=None):
        """Packs pages page_ids (logical order) into the uint8 host tensor
        `host` [n, host_page_bytes] (asynchronous when it is pinned)."""
        import numpy as np
        ids = np.ascontiguousarray(page_ids, dtype=np.int32)
        _check(load().nk_pages_to_host(self.handle, ids.ctypes.data, ids.size, host.data_ptr(),
                                       _stream(stream)))
        return host

    def pages_from_host(self, page_ids, host, stream=None):
        import numpy as np
        ids = np.ascontiguousarray(page_ids, dtype=np.int32)
        _check(load().nk_pages_from_host(self.handle, ids.ctypes.data, ids.size, host.data_ptr(),
                                         _stream(stream)))

    def prefill(self, layer, q, tables, table_rows, prefix_len, chunk_len, scale, out=None,
                lse=None, workspace=None, stream=None):
        import torch
        B, Tc, Hq, D = q.shape
        n = nk_prefill_workspace_bytes(self.handle, B, Tc, Hq)
        ws = workspace
        if out is None or lse is None or ws is None:
            with _on(stream):
                if out is None:
                    out = torch.zeros_like(q)
                if lse is None:
                    lse = torch.full((B, Tc, Hq), float("-inf"), dtype=torch.float32, device=q.device)
                if ws is None and n:   # split partials and counters, zero-filled once, kept for reuse
                    if getattr(self, "_pws", None) is None or self._pws.numel() < n:
                        self._pws = torch.zeros(n, dtype=torch.uint8, device=q.device)
                    ws = self._pws
        nk_paged_prefill_attention(_ptr(q), Hq, self.handle, layer, _ptr(tables), _ptr(table_rows),
                                   _ptr(prefix_len), _ptr(chunk_len), B, Tc, float(scale), _ptr(out),
                                   _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
        return out, lse

    def copy_columns(self, src, dst, ncols, stream=None):
        nk_page_copy_columns(self.handle, src, dst, ncols, _stream(stream))

    def append_rope(self, layer, tables, table_rows, write_pos, k, v, rope: Rope, q=None, q_out=None, counts=None,
                    stream=None):
        """Appends k, v [B, T, H, D] with the norm and rotation of k on the
        way, and returns q_out [B, T, Hq, D], the queries normed and rotated in
        the same launch (None without q).  k, v, q: bf16, any token and head
        strides, one token stride apart across rows; rows of q_out past a
        row's count are not written."""
        import torch
        dev = self.device
        if torch.cuda.current_device() != dev:
            with torch.cuda.device(dev):
                return self.append_rope(layer, tables, table_rows, write_pos, k, v, rope, q, q_out, counts, stream)
        if rope.device != dev:
            raise ValueError("the rotation table is on another device than the pool")
        at = _handle(stream, dev)
        if q is not None and q_out is None:
            with _on(stream):
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _check((_pyargs or _args()).append_rope(
            self.handle, self.H, self.D, self.C, self.L, layer, tables, table_rows, write_pos, k, v, q, q_out, counts,
            rope.address, rope.head_dim, dev, at))
        return q_out

    def shared_workspace(self, B, T, Hq):
        """A workspace for ``shared_decode`` (one per stream or captured graph that may overlap others)."""
        import torch
        n = nk_shared_decode_workspace_bytes(self.handle, B, T, Hq)
        return torch.empty(n, dtype=torch.uint8, device=self.planes[0][0].device)

    def shared_decode(self, layer, q, tables, table_rows, frontiers, shared_pages, scale, out=None, lse=None,
                      workspace=None, stream=None, share_from: int = -1):
        """``decode`` of a batch whose rows share their first ``shared_pages``
        (int32 device tensor of one value) pages, attended once for all rows
        from ``share_from`` of them on (-1: the library's choice, 0: always).
        ``workspace``: contiguous, of any type; without it one is allocated
        for this call."""
        import torch
        dev = self.device
        if torch.cuda.current_device() != dev:
            with torch.cuda.device(dev):
                return self.shared_decode(layer, q, tables, table_rows, frontiers, shared_pages, scale, out, lse,
                                          workspace, stream, share_from)
        at = _handle(stream, dev)
        ws = workspace
        if out is None or lse is None or ws is None:
            with _on(stream):
                if out is None:
                    out = torch.empty_like(q)
                if lse is None:
                    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
                if ws is None:
                    ws = self.shared_workspace(*q.shape[:3])
        _check((_pyargs or _args()).shared_decode(
            self.handle, self.D, self.C, self.L, layer, q, tables, table_rows, frontiers, shared_pages, float(scale),
            out, lse, share_from, ws, dev, at))
        return out, lse

    def diff_decode_workspace(self, B, T, Hq):
        """A workspace for ``diff_decode`` (one per stream or captured graph that may overlap others)."""
        import torch
        n = nk_diff_decode_workspace_bytes(self.handle, B, T, Hq)
        return torch.empty(n, dtype=torch.uint8, device=self.planes[0][0].device)

    def diff_prefill_workspace(self, B, Tc, Hq):
        """A workspace for ``diff_prefill`` (one per stream or captured graph that may overlap others)."""
        import torch
        n = nk_diff_prefill_workspace_bytes(self.handle, B, Tc, Hq)
        return torch.empty(n, dtype=torch.uint8, device=self.planes[0][0].device)

    def diff_decode(self, layer, q, tables, table_rows, frontiers, scale, diff: Diff, out=None, lse=None,
                    workspace=None, stream=None):
        """Differential attention of the T newest tokens of every row (nk.h,
        nk_paged_diff_decode_attention): q [B, T, Hq, D], head i's maps in query
        heads 2i and 2i + 1; returns out [B, T, Hq / 2, 2 D] and lse [B, T, Hq].
        Without ``workspace`` one is allocated for this call."""
        return self._diff(False, layer, q, tables, table_rows, frontiers, None, scale, diff, out, lse, workspace, stream)

    def diff_prefill(self, layer, q, tables, table_rows, prefix_len, chunk_len, scale, diff: Diff, out=None, lse=None,
                     workspace=None, stream=None):
        """Differential attention of prompt chunks (nk.h,
        nk_paged_diff_prefill_attention): q [B, Tc, Hq, D] as in ``diff_decode``;
        rows behind chunk_len are not written (0 and -inf in tensors that this
        call makes)."""
        return self._diff(True, layer, q, tables, table_rows, prefix_len, chunk_len, scale, diff, out, lse, workspace,
                          stream)

    def _diff(self, prefill, layer, q, tables, table_rows, lengths, chunk_len, scale, diff, out, lse, workspace, stream):
        import torch
        dev = self.device
        if torch.cuda.current_device() != dev:
            with torch.cuda.device(dev):
                return self._diff(prefill, layer, q, tables, table_rows, lengths, chunk_len, scale, diff, out, lse,
                                  workspace, stream)
        if diff.device != dev:
            raise ValueError("lam is on another device than the pool")
        at = _handle(stream, dev)
        ws = workspace
        if out is None or lse is None or ws is None:
            if len(q.shape) != 4 or q.shape[2] % 2:
                raise ValueError("q: expected [B, T, an even number of query heads, head_dim]")
            B, T, Hq, D = q.shape
            with _on(stream):
                if out is None:
                    make = torch.zeros if prefill else torch.empty
                    out = make((B, T, Hq // 2, 2 * D), dtype=torch.bfloat16, device=q.device)
                if lse is None:
                    lse = (torch.full((B, T, Hq), float("-inf"), dtype=torch.float32, device=q.device) if prefill
                           else torch.empty((B, T, Hq), dtype=torch.float32, device=q.device))
                if ws is None:
                    ws = (self.diff_prefill_workspace if prefill else self.diff_decode_workspace)(B, T, Hq)
        _check((_pyargs or _args()).diff(
            prefill, self.handle, self.D, self.C, self.L, layer, q, tables, table_rows, lengths, chunk_len, float(scale),
            diff.address, diff.heads, diff.tokens, diff.width, out, lse, ws, dev, at))
        return out, lse

    def free_pages(self):
        """The state of an empty pool for ``grow``: tables [C, L] (-1), mapped [C] (0), the stack of free pages [M]
        (all, page 0 on top) and their number [1], int32."""
        import torch
        kw = dict(dtype=torch.int32, device=self.planes[0][0].device)
        return (torch.full((self.C, self.L), -1, **kw), torch.zeros(self.C, **kw),
                torch.arange(self.M - 1, -1, -1, **kw), torch.full((1,), self.M, **kw))

    def grow(self, tables, table_rows, committed, mapped, free_pages, free_count, T, counts=None, keep=None,
             mapped_out=None, free_count_out=None, frontiers=None, positions=None, slots=None, stream=None):
        """Brings every row of the batch to the pages of its committed + count tokens (nk.h, nk_pages_grow).

        tables [C, L], mapped [C], free_pages [M] and free_count [1] are updated
        in place (mapped_out, free_count_out: written instead of mapped and
        free_count); committed, counts (None: T each) [B]; keep [C] or None.
        Returns (frontiers [B], positions [B, T], slots [B, T] int64): new tensors
        unless given; positions=False, slots=False: not made (None).
        """
        import torch
        dev = self.device
        if torch.cuda.current_device() != dev:
            with torch.cuda.device(dev):
                return self.grow(tables, table_rows, committed, mapped, free_pages, free_count, T, counts, keep,
                                 mapped_out, free_count_out, frontiers, positions, slots, stream)
        at = _handle(stream, dev)
        if frontiers is None or positions is None or slots is None:
            B = committed.shape[0]
            with _on(stream):
                if frontiers is None:
                    frontiers = torch.empty((B,), dtype=torch.int32, device=committed.device)
                if positions is None:
                    positions = torch.empty((B, T), dtype=torch.int32, device=committed.device)
                if slots is None:
                    slots = torch.empty((B, T), dtype=torch.int64, device=committed.device)
        positions, slots = (None if x is False else x for x in (positions, slots))
        _check((_pyargs or _args()).grow(
            self.handle, self.C, self.L, self.M, T, tables, table_rows, committed, counts, keep, mapped,
            mapped if mapped_out is None else mapped_out, free_pages, free_count,
            free_count if free_count_out is None else free_count_out, frontiers, positions, slots, dev, at))
        return frontiers, positions, slots
