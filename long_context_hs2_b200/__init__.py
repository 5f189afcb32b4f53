"""Python binding of libhs2, the sm_100a HySparse2 hybrid-block hot path.

Argument marshalling only: every function here forwards to the C ABI of
include/hs2.h with the same name, turning torch tensors into device pointers
and the current CUDA stream into a stream handle, and raises ``Hs2Error`` when
the library returns a non-OK status.  All computation runs in the library's
CUDA kernels; there is no fallback path.  Importing this package does not load
the library; the first call does, and fails loudly if ``libhs2.so`` has not
been built (``python -m long_context_hs2_b200.build``).
"""

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhs2.so")

HS2_OK = 0
HS2_KV_BF16 = 0
HS2_KV_FP8_E4M3 = 1

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error",
           4: "workspace", 5: "timeout", 6: "device index error"}

EXPORTED = ("hs2_bridge_kv", "hs2_full_attn_select_workspace", "hs2_full_attn_select",
            "hs2_full_attn_select_noalloc", "hs2_sparse_attn", "hs2_last_device_status",
            "hs2_status_string", "hs2_version", "hs2_set_stage_events",
            "hs2_set_fault_injection", "hs2_full_attn_select_blocks", "hs2_cp_workspace",
            "hs2_cp_attn_partial", "hs2_cp_lse_combine", "hs2_cp_rescale", "hs2_cp_select_local",
            "hs2_cp_merge_select", "hs2_set_phase_stamps", "hs2_add_rmsnorm", "hs2_fp8_gemm",
            "hs2_paged_append", "hs2_paged_attn", "hs2_paged_attn_workspace", "hs2_paged_evict")

# Global-timer stamps per CTA written by the fused full-attention kernel when enabled.
HS2_PHASES = 8

# Size of the scratch area built into the library for hs2_full_attn_select_noalloc.
HS2_NOALLOC_SCRATCH_BYTES = 16 << 20


class Hs2Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s failed: %s (%d)" % (fn, _STATUS.get(status, "?"), status))
        self.status = status


class hs2_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class hs2_paged_cache(ctypes.Structure):
    _fields_ = [("kv", hs2_kv_cache), ("weight", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libhs2.so and declares its signatures.  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libhs2.so is not built at %s; run python -m long_context_hs2_b200.build"
                           % path)
    lib = ctypes.CDLL(path)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    KV = ctypes.POINTER(hs2_kv_cache)
    lib.hs2_version.restype = i32
    lib.hs2_status_string.restype = ctypes.c_char_p
    lib.hs2_status_string.argtypes = [i32]
    lib.hs2_last_device_status.restype = i32
    lib.hs2_last_device_status.argtypes = [P]
    lib.hs2_bridge_kv.restype = i32
    lib.hs2_bridge_kv.argtypes = [P, i64, i32, P, i32, i32, i32, KV, i64, P]
    lib.hs2_full_attn_select_workspace.restype = sz
    lib.hs2_full_attn_select_workspace.argtypes = [i32, i32, i64, i32, i32, i32, i32, i32]
    lib.hs2_full_attn_select.restype = i32
    lib.hs2_full_attn_select.argtypes = [P, KV, i32, i32, i64, i32, i32, ctypes.c_float, i32, i32,
                                         i32, P, P, P, P, P, sz, P]
    lib.hs2_full_attn_select_blocks.restype = i32
    lib.hs2_full_attn_select_blocks.argtypes = [P, KV, i32, i32, i64, i32, i32, ctypes.c_float,
                                                i32, i32, i32, i32, P, P, P, P, P, sz, P]
    lib.hs2_cp_workspace.restype = sz
    lib.hs2_cp_workspace.argtypes = [i32, i32, i64, i32, i32, i32, i32, i32]
    lib.hs2_cp_attn_partial.restype = i32
    lib.hs2_cp_attn_partial.argtypes = [P, KV, i32, i32, i64, i64, i32, i32, ctypes.c_float, i32,
                                        P, P, P, sz, P]
    lib.hs2_cp_lse_combine.restype = i32
    lib.hs2_cp_lse_combine.argtypes = [P, i32, i64, P, P]
    lib.hs2_cp_rescale.restype = i32
    lib.hs2_cp_rescale.argtypes = [P, P, P, i64, i32, P]
    lib.hs2_cp_select_local.restype = i32
    lib.hs2_cp_select_local.argtypes = [P, KV, i32, i32, i64, i64, i64, i32, i32, ctypes.c_float,
                                        i32, i32, i32, P, P, P, P, sz, P]
    lib.hs2_cp_merge_select.restype = i32
    lib.hs2_cp_merge_select.argtypes = [P, P, i32, i32, i32, i64, i32, i32, P, P, P]
    lib.hs2_full_attn_select_noalloc.restype = i32
    lib.hs2_full_attn_select_noalloc.argtypes = [P, KV, i32, i32, i64, i32, i32, ctypes.c_float,
                                                 i32, i32, i32, P, P, P, P, P]
    lib.hs2_set_stage_events.restype = i32
    lib.hs2_set_fault_injection.restype = i32
    lib.hs2_set_fault_injection.argtypes = [ctypes.c_uint, ctypes.c_ulonglong]
    lib.hs2_set_phase_stamps.restype = i32
    lib.hs2_set_phase_stamps.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.hs2_set_stage_events.argtypes = [P, P]
    lib.hs2_sparse_attn.restype = i32
    lib.hs2_sparse_attn.argtypes = [P, KV, i32, i32, i64, i32, i32, ctypes.c_float, P, P, i32, i32,
                                    P, P]
    PC = ctypes.POINTER(hs2_paged_cache)
    lib.hs2_add_rmsnorm.restype = i32
    lib.hs2_add_rmsnorm.argtypes = [P, P, P, i64, i32, ctypes.c_float, P, P, P, P, P]
    lib.hs2_fp8_gemm.restype = i32
    lib.hs2_fp8_gemm.argtypes = [P, P, i64, P, P, i32, i32, P, P]
    lib.hs2_paged_append.restype = i32
    lib.hs2_paged_append.argtypes = [P, P, i64, i64, P, PC, i32, i32, i32, i32, P]
    lib.hs2_paged_attn_workspace.restype = sz
    lib.hs2_paged_attn_workspace.argtypes = [i32, i32, i32, i32]
    lib.hs2_paged_attn.restype = i32
    lib.hs2_paged_attn.argtypes = [P, PC, i32, i32, i32, i32, ctypes.c_float, i32, P, P, i32, P,
                                   sz, P]
    lib.hs2_paged_evict.restype = i32
    lib.hs2_paged_evict.argtypes = [PC, i32, i32, i32, i32, i32, i32, P, i32, P, P, P]
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the handle without a Stream object
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int):
    if st != HS2_OK:
        raise Hs2Error(fn, st)


def kv_cache(k, v, k_scale=None, v_scale=None) -> hs2_kv_cache:
    """The C struct of one layer's cache from device tensors (or raw pointers).
    The struct holds references to the tensors it was made from, so that their
    memory stays allocated for as long as the struct (or a CUDA graph that
    captured calls with it, while the caller keeps the struct) is in use."""
    c = hs2_kv_cache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale))
    c._tensors = (k, v, k_scale, v_scale)
    return c


def hs2_version() -> int:
    return load_library().hs2_version()


def hs2_status_string(status: int) -> str:
    return load_library().hs2_status_string(int(status)).decode()


def hs2_last_device_status(stream=None) -> int:
    """Synchronises `stream`; returns (and clears) the device status code."""
    return load_library().hs2_last_device_status(_stream(stream))


def hs2_bridge_kv(X, T: int, hidden: int, Wt, n_layers: int, D: int, out_dtype: int,
                  caches: Sequence[hs2_kv_cache], cache_row_offset: int = 0, stream=None):
    arr = (hs2_kv_cache * n_layers)(*caches)
    _check("hs2_bridge_kv", load_library().hs2_bridge_kv(
        _ptr(X), int(T), int(hidden), _ptr(Wt), int(n_layers), int(D), int(out_dtype), arr,
        int(cache_row_offset), _stream(stream)))


def hs2_full_attn_select_workspace(B, T, L, H, D, topk, window, dt) -> int:
    return int(load_library().hs2_full_attn_select_workspace(int(B), int(T), int(L), int(H), int(D),
                                                             int(topk), int(window), int(dt)))


def hs2_full_attn_select(Q, kv: hs2_kv_cache, B, T, L, H, D, scale, topk, window, dt, O, lse,
                         idx, n_sel, workspace, workspace_bytes: int, stream=None):
    _check("hs2_full_attn_select", load_library().hs2_full_attn_select(
        _ptr(Q), ctypes.byref(kv), int(B), int(T), int(L), int(H), int(D), float(scale), int(topk),
        int(window), int(dt), _ptr(O), _ptr(lse), _ptr(idx), _ptr(n_sel), _ptr(workspace),
        int(workspace_bytes), _stream(stream)))


def hs2_full_attn_select_blocks(Q, kv: hs2_kv_cache, B, T, L, H, D, scale, topk, window, block,
                                dt, O, lse, idx, n_sel, workspace, workspace_bytes: int,
                                stream=None):
    """hs2_full_attn_select with the block-level selection (blocks of `block`
    positions, topk/block of them kept) instead of the token-level one."""
    _check("hs2_full_attn_select_blocks", load_library().hs2_full_attn_select_blocks(
        _ptr(Q), ctypes.byref(kv), int(B), int(T), int(L), int(H), int(D), float(scale),
        int(topk), int(window), int(block), int(dt), _ptr(O), _ptr(lse), _ptr(idx), _ptr(n_sel),
        _ptr(workspace), int(workspace_bytes), _stream(stream)))


def hs2_full_attn_select_noalloc(Q, kv: hs2_kv_cache, B, T, L, H, D, scale, topk, window, dt,
                                 O, lse, idx, n_sel, stream=None):
    """hs2_full_attn_select without a workspace argument, for callers that cannot
    allocate device memory; the library's built-in scratch area is used instead."""
    _check("hs2_full_attn_select_noalloc", load_library().hs2_full_attn_select_noalloc(
        _ptr(Q), ctypes.byref(kv), int(B), int(T), int(L), int(H), int(D), float(scale),
        int(topk), int(window), int(dt), _ptr(O), _ptr(lse), _ptr(idx), _ptr(n_sel),
        _stream(stream)))


def hs2_sparse_attn(Q, kv: hs2_kv_cache, B, T, L, H, D, scale, idx, n_sel, slots, dt, O,
                    stream=None):
    _check("hs2_sparse_attn", load_library().hs2_sparse_attn(
        _ptr(Q), ctypes.byref(kv), int(B), int(T), int(L), int(H), int(D), float(scale),
        _ptr(idx), _ptr(n_sel), int(slots), int(dt), _ptr(O), _stream(stream)))


def hs2_set_stage_events(begin=None, end=None):
    """Sets (or, with no arguments, clears) the events that this thread's
    full-attention calls record around their partial-attention kernel.
    `begin`/`end` are torch.cuda.Event objects (timing enabled) or raw handles."""
    def handle(e):
        if e is None or isinstance(e, int):
            return e
        return e.cuda_event
    _check("hs2_set_stage_events", load_library().hs2_set_stage_events(handle(begin), handle(end)))


def hs2_set_phase_stamps(stamps=None, max_ctas: int = 0):
    """Tracing: the fused full-attention kernel writes HS2_PHASES global-timer
    stamps per CTA into `stamps` (a device uint64/int64 buffer of max_ctas *
    HS2_PHASES values); None turns them off."""
    _check("hs2_set_phase_stamps",
           load_library().hs2_set_phase_stamps(_ptr(stamps), int(max_ctas) if stamps is not None else 0))


def hs2_set_fault_injection(extra_arrivals: int = 0, wait_limit_ns: int = 0):
    """Test hook: the fused kernel's group barriers wait for `extra_arrivals`
    arrivals that never come and give up after `wait_limit_ns` (0: one second).
    With no arguments, restores the defaults."""
    _check("hs2_set_fault_injection",
           load_library().hs2_set_fault_injection(int(extra_arrivals), int(wait_limit_ns)))


# ------------------------------------------------ context parallelism --
def hs2_cp_workspace(B, T, L_local, H, D, topk, window, dt) -> int:
    return int(load_library().hs2_cp_workspace(int(B), int(T), int(L_local), int(H), int(D),
                                                int(topk), int(window), int(dt)))


def hs2_cp_attn_partial(Q, kv: hs2_kv_cache, B, T, L_local, q_pos_local, H, D, scale, dt, O, lse,
                        workspace, workspace_bytes: int, stream=None):
    _check("hs2_cp_attn_partial", load_library().hs2_cp_attn_partial(
        _ptr(Q), ctypes.byref(kv), int(B), int(T), int(L_local), int(q_pos_local), int(H), int(D),
        float(scale), int(dt), _ptr(O), _ptr(lse), _ptr(workspace), int(workspace_bytes),
        _stream(stream)))


def hs2_cp_lse_combine(lse_parts, G, n, lse, stream=None):
    _check("hs2_cp_lse_combine", load_library().hs2_cp_lse_combine(
        _ptr(lse_parts), int(G), int(n), _ptr(lse), _stream(stream)))


def hs2_cp_rescale(O_part, lse_part, lse, n, D, stream=None):
    _check("hs2_cp_rescale", load_library().hs2_cp_rescale(
        _ptr(O_part), _ptr(lse_part), _ptr(lse), int(n), int(D), _stream(stream)))


def hs2_cp_select_local(Q, kv: hs2_kv_cache, B, T, L_local, q_pos_local, key_pos0, H, D, scale,
                        topk, window, dt, lse, cand_score, cand_idx, workspace,
                        workspace_bytes: int, stream=None):
    _check("hs2_cp_select_local", load_library().hs2_cp_select_local(
        _ptr(Q), ctypes.byref(kv), int(B), int(T), int(L_local), int(q_pos_local), int(key_pos0),
        int(H), int(D), float(scale), int(topk), int(window), int(dt), _ptr(lse),
        _ptr(cand_score), _ptr(cand_idx), _ptr(workspace), int(workspace_bytes),
        _stream(stream)))


def hs2_cp_merge_select(cand_score, cand_idx, G, B, T, q_pos0, topk, window, idx, n_sel,
                        stream=None):
    _check("hs2_cp_merge_select", load_library().hs2_cp_merge_select(
        _ptr(cand_score), _ptr(cand_idx), int(G), int(B), int(T), int(q_pos0), int(topk),
        int(window), _ptr(idx), _ptr(n_sel), _stream(stream)))


# --------------------------------------------------- paged decode path --
# Tensors given to these calls must be contiguous (K and V of the append excepted),
# of the type the C ABI names, and on the current device, whose current stream the
# work is enqueued on; anything else raises Hs2Error (invalid argument).  E4M3
# codes are uint8 or float8_e4m3fn tensors, workspaces of any type of one byte.  Raw
# pointers are taken as they are.
_TYPES = {}


def _types():
    """The element types that each kind of argument may have."""
    if not _TYPES:
        import torch
        codes = (torch.uint8, torch.float8_e4m3fn)
        _TYPES.update(bf16=(torch.bfloat16,), f32=(torch.float32,), i32=(torch.int32,), e4m3=codes,
                      bytes=codes + (torch.int8,))
    return _TYPES


def _tensors(fn: str, specs):
    """Device pointers of (tensor, kind of element, least elements, contiguous) entries."""
    import torch
    types = _TYPES or _types()
    dev, out = None, []
    for t, kind, least, contiguous in specs:
        if t is None or isinstance(t, int):
            out.append(t)
            continue
        d = t.get_device()
        if dev is None and d >= 0:
            dev = torch.cuda.current_device()
        if (d != dev or t.dtype not in types[kind] or t.numel() < least
                or (contiguous and not t.is_contiguous())):
            raise Hs2Error(fn, 1)
        out.append(t.data_ptr())
    return out


def paged_cache(k, v, page_table, seq_len, k_scale=None, v_scale=None,
                weight=None) -> hs2_paged_cache:
    """The C struct of a paged cache: k, v [n_pages, page_size, kv_heads, D] (bf16, or E4M3
    with scales [n_pages, page_size, kv_heads]), page_table int32 [B, max_pages], seq_len
    int32 [B], weight fp32 [n_pages, page_size].  Like kv_cache, it keeps its tensors."""
    n_pages, page_size, heads, _ = k.shape
    if (v.shape != k.shape or v.dtype != k.dtype or page_table.dim() != 2
            or seq_len.numel() != page_table.shape[0]
            or (k_scale is None) != (v_scale is None)):
        raise Hs2Error("paged_cache", 1)
    rows, kind = n_pages * page_size, "bf16" if k_scale is None else "e4m3"
    p = _tensors("paged_cache", ((k, kind, 1, True), (v, kind, 1, True),
                                 (k_scale, "f32", rows * heads, True),
                                 (v_scale, "f32", rows * heads, True), (weight, "f32", rows, True),
                                 (page_table, "i32", 1, True), (seq_len, "i32", 1, True)))
    c = hs2_paged_cache(hs2_kv_cache(p[0], p[1], p[2], p[3]), p[4], p[5], p[6], n_pages, page_size,
                        page_table.shape[1])
    c._tensors = (k, v, page_table, seq_len, k_scale, v_scale, weight)
    c._shape = (page_table.shape[0], heads, k.shape[3], 0 if k_scale is None else 1)
    return c


def _check_cache(fn: str, cache, B, kv_heads, D, dt):
    # a struct made by paged_cache knows what its tensors hold
    shape = getattr(cache, "_shape", None)
    if shape is not None and (B > shape[0] or (kv_heads, D, dt) != shape[1:]):
        raise Hs2Error(fn, 1)


def hs2_add_rmsnorm(X, R, gamma, T, hidden, eps, sum=None, Y=None, Yq=None, Yq_scale=None,
                    stream=None):
    n = T * hidden
    p = _tensors("hs2_add_rmsnorm", ((X, "bf16", n, True), (R, "bf16", n, True),
                                     (gamma, "bf16", hidden, True), (sum, "bf16", n, True),
                                     (Y, "bf16", n, True), (Yq, "e4m3", n, True),
                                     (Yq_scale, "f32", T * ((hidden + 127) // 128), True)))
    _check("hs2_add_rmsnorm", load_library().hs2_add_rmsnorm(
        p[0], p[1], p[2], T, hidden, eps, p[3], p[4], p[5], p[6], _stream(stream)))


def hs2_fp8_gemm(A, A_scale, M, B, B_scale, N, K, C, stream=None):
    """C = A B^T in E4M3 with a scale per 1 x 128 of A and 128 x 128 of B; C bf16 [M, N]."""
    kb = (K + 127) // 128
    p = _tensors("hs2_fp8_gemm", ((A, "e4m3", M * K, True), (A_scale, "f32", M * kb, True),
                                  (B, "e4m3", N * K, True),
                                  (B_scale, "f32", (N + 127) // 128 * kb, True),
                                  (C, "bf16", M * N, True)))
    _check("hs2_fp8_gemm", load_library().hs2_fp8_gemm(p[0], p[1], M, p[2], p[3], N, K, p[4],
                                                       _stream(stream)))


def _row_elements(shape, stride) -> int:
    """Elements that lie one after another from the start of each row rows[r]; 0 where a row
    has gaps."""
    if len(shape) == 2:
        return shape[1] if stride[1] == 1 or shape[1] == 1 else 0
    n = 1
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] != 1 and stride[i] != n:
            return 0
        n *= shape[i]
    return n if len(shape) > 1 else 0


def hs2_paged_append(K, V, ld, n_rows, row_start, cache: hs2_paged_cache, B, kv_heads, D, dt,
                     stream=None):
    """K, V: the new rows, `ld` elements apart (views into a projection's output, for example)."""
    _check_cache("hs2_paged_append", cache, B, kv_heads, D, dt)
    n = n_rows * kv_heads * D
    for rows in (K, V):
        if isinstance(rows, int) or rows is None:
            continue
        shape, stride = rows.shape, rows.stride()
        if (shape[0] < n_rows or (n_rows > 1 and stride[0] != ld)
                or _row_elements(shape, stride) < kv_heads * D):
            raise Hs2Error("hs2_paged_append", 1)
    p = _tensors("hs2_paged_append", ((K, "bf16", n, False), (V, "bf16", n, False),
                                      (row_start, "i32", B + 1, True)))
    _check("hs2_paged_append", load_library().hs2_paged_append(
        p[0], p[1], ld, n_rows, p[2], ctypes.byref(cache), B, kv_heads, D, dt, _stream(stream)))


def hs2_paged_attn_workspace(B, H, kv_heads, D) -> int:
    return int(load_library().hs2_paged_attn_workspace(B, H, kv_heads, D))


def hs2_paged_attn(Q, cache: hs2_paged_cache, B, H, kv_heads, D, scale, dt, O, lse, accumulate,
                   workspace, workspace_bytes: int, stream=None):
    """One new token per sequence over its pages; `accumulate` adds each position's
    head-summed probability to the cache's weight."""
    _check_cache("hs2_paged_attn", cache, B, kv_heads, D, dt)
    n = B * H * D
    p = _tensors("hs2_paged_attn", ((Q, "bf16", n, True), (O, "bf16", n, True),
                                    (lse, "f32", B * H, True),
                                    (workspace, "bytes", workspace_bytes, True)))
    _check("hs2_paged_attn", load_library().hs2_paged_attn(
        p[0], ctypes.byref(cache), B, H, kv_heads, D, scale, dt, p[1], p[2],
        1 if accumulate else 0, p[3], workspace_bytes, _stream(stream)))


def hs2_paged_evict(cache: hs2_paged_cache, B, kv_heads, D, dt, topk, window, dst_table, kept,
                    new_len, stream=None, dst_max_pages=None):
    """Keeps the `topk` heaviest positions and the `window` most recent ones of every sequence,
    moved to the pages of dst_table int32 [B, dst_max_pages] (None: in place).  The width is
    the tensor's own; with a raw pointer it has to be given."""
    _check_cache("hs2_paged_evict", cache, B, kv_heads, D, dt)
    if dst_table is None:
        dst_max_pages = 0
    elif not isinstance(dst_table, int):
        if dst_table.dim() != 2 or dst_max_pages not in (None, dst_table.shape[1]):
            raise Hs2Error("hs2_paged_evict", 1)
        dst_max_pages = dst_table.shape[1]
    elif dst_max_pages is None:
        raise Hs2Error("hs2_paged_evict", 1)
    most = B * dst_max_pages
    p = _tensors("hs2_paged_evict", ((dst_table, "i32", most, True),
                                     (kept, "i32", B * (topk + window), True),
                                     (new_len, "i32", B, True)))
    _check("hs2_paged_evict", load_library().hs2_paged_evict(
        ctypes.byref(cache), B, kv_heads, D, dt, topk, window, p[0],
        dst_max_pages, p[1], p[2], _stream(stream)))
