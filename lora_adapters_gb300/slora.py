"""Thin ctypes binding of libslora.so (include/slora.h).

Every ``slora_*`` function here has the C function's name and arguments and
only marshals them; all work happens in the library.  ``Pool`` is a small
convenience wrapper over the same calls for torch tensors.

The library is loaded from this package directory (built by
``lora_adapters_gb300.build``).  If it is missing the import of the binding
fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
# SLORA_DEBUG=1 in the environment selects the build with bounds checks in
# every kernel (libslora_debug.so); either way the library must exist.
DEBUG = os.environ.get("SLORA_DEBUG", "") == "1"
LIB_PATH = os.path.join(HERE, "libslora_debug.so" if DEBUG else "libslora.so")

OK = 0
ERR_INVALID = -1
ERR_OOM = -2
ERR_EXISTS = -3
ERR_NOT_RESIDENT = -4
ERR_BUSY = -5
ERR_CUDA = -6
ERR_DEVICE = -7
ERR_TIMEOUT = -8
ERR_DEVICE_ASSERT = -9
F16, BF16 = 0, 1
MODE_AUTO, MODE_DECODE, MODE_PREFILL = 0, 1, 2

EXPORTED = (
    "slora_pool_create", "slora_pool_destroy", "slora_pages_alloc", "slora_pages_free",
    "slora_pool_info", "slora_adapter_load", "slora_adapter_evict", "slora_adapter_pages",
    "slora_build_segments", "slora_lora_apply", "slora_lora_apply_multi", "slora_device_status",
    "slora_pool_snapshot", "slora_timing_enable", "slora_timing_read", "slora_set_tc_threshold",
    "slora_last_error_string", "slora_lora_apply_noalloc", "slora_adapter_set_scale",
    "slora_lora_apply_bmm", "slora_bmm_scratch_bytes", "slora_set_tc_min_batch", "slora_debug_set_fault",
    "slora_debug_set_wait_limit", "slora_adapter_ready", "slora_build_segments_for",
    "slora_debug_poke_page_table",
    "slora_kv_array_ints", "slora_kv_create", "slora_kv_destroy", "slora_kv_set_rotary", "slora_kv_plan", "slora_kv_append",
    "slora_kv_attend",
)
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1
KV_MAX_REQUESTS = 4096
KV_MAX_HEAD_DIM = 256
FAULT_NONE, FAULT_PAGE_ALLOC, FAULT_COPY = 0, 1, 2


class SloraError(RuntimeError):
    def __init__(self, code: int, fn: str, msg: str):
        super().__init__(f"{fn} -> {code}: {msg}")
        self.code = code


class slora_segments(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("max_segs", ctypes.c_int32),
                ("perm", ctypes.c_void_p), ("seg_start", ctypes.c_void_p),
                ("seg_adapter", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("generation", ctypes.c_uint64)]


class slora_kv_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("layers", "heads_q", "heads_kv", "head_dim", "max_requests",
                                              "max_blocks")]


class slora_kv_batch(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("T", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("tok_req", ctypes.c_void_p),
                ("tok_pos", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("slot_stride", ctypes.c_int64),
                ("generation", ctypes.c_uint64)]


_lib = None
P = ctypes.c_void_p
I32, I64 = ctypes.c_int32, ctypes.c_int64
_SIGS = {
    "slora_pool_create": [ctypes.POINTER(P), P, I64, I32, I32, I32, I32, I32, I32, P, P, P, P],
    "slora_pool_destroy": [P],
    "slora_pages_alloc": [P, I64, P],
    "slora_pages_free": [P, I64, P],
    "slora_pool_info": [P, P, P, P, P],
    "slora_adapter_load": [P, I32, I32, P, P, ctypes.POINTER(P)],
    "slora_adapter_evict": [P, I32],
    "slora_adapter_set_scale": [P, I32, ctypes.c_float],
    "slora_adapter_ready": [P, I32, P],
    "slora_adapter_pages": [P, I32, P, I64, P],
    "slora_build_segments": [P, P, I32, ctypes.POINTER(slora_segments)],
    "slora_build_segments_for": [P, P, I32, P, ctypes.POINTER(slora_segments)],
    "slora_lora_apply": [P, ctypes.POINTER(slora_segments), I32, P, I64, P, I64, ctypes.c_float, I32],
    "slora_lora_apply_multi": [P, ctypes.POINTER(slora_segments), I32, P, P, P, P, P, ctypes.c_float, I32],
    "slora_lora_apply_bmm": [P, ctypes.POINTER(slora_segments), I32, P, I64, P, I64, ctypes.c_float],
    "slora_bmm_scratch_bytes": [P, ctypes.POINTER(ctypes.c_size_t)],
    "slora_device_status": [P, P],
    "slora_pool_snapshot": [P, P, ctypes.POINTER(ctypes.c_size_t)],
    "slora_timing_enable": [P, I32],
    "slora_timing_read": [P, I32, P, P, P, P],
    "slora_set_tc_threshold": [P, I32],
    "slora_set_tc_min_batch": [P, I32],
    "slora_debug_set_fault": [P, I32, I64],
    "slora_debug_set_wait_limit": [P, ctypes.c_uint32],
    "slora_debug_poke_page_table": [P, I64, I32, P],
    "slora_lora_apply_noalloc": [P, I32, I32, P, I64, P, I32, I32, P, P, I32, P, I32, P, I64, P, I64,
                                 ctypes.c_float, P, P],
    "slora_kv_array_ints": [P, ctypes.POINTER(slora_kv_config), P],
    "slora_kv_create": [ctypes.POINTER(P), P, ctypes.POINTER(slora_kv_config), P, P],
    "slora_kv_destroy": [P],
    "slora_kv_set_rotary": [P, I32, I32, P, ctypes.c_float],
    "slora_kv_plan": [P, I32, P, P, P, P, I64, I32, I32, ctypes.POINTER(slora_kv_batch)],
    "slora_kv_append": [P, ctypes.POINTER(slora_kv_batch), I32, P, I64, P, I64, P, I64, P, P, ctypes.c_float, P, I64],
    "slora_kv_attend": [P, ctypes.POINTER(slora_kv_batch), I32, P, I64, P, I64, ctypes.c_float, ctypes.c_float],
}


def lib() -> ctypes.CDLL:
    """Load libslora.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{os.path.basename(LIB_PATH)} not built at {LIB_PATH}: "
                              "run lora_adapters_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.slora_last_error_string.argtypes = []
        L.slora_last_error_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(rc: int, fn: str) -> int:
    if rc != OK:
        raise SloraError(rc, fn, slora_last_error_string())
    return rc


def _arr(values, ctype):
    return (ctype * len(values))(*values)


# ---- the C functions under their own names ------------------------------------
def slora_last_error_string() -> str:
    s = lib().slora_last_error_string()
    return s.decode() if s else ""


def slora_pool_create(d_pool: int, num_pages: int, page_elems: int, dtype: int, max_adapters: int,
                      max_rank: int, max_tokens: int, proj_in: Sequence[int], proj_out: Sequence[int],
                      compute_stream: int = 0, copy_stream: int = 0) -> int:
    out = P()
    _check(lib().slora_pool_create(ctypes.byref(out), d_pool or None, num_pages, page_elems, dtype,
                                   max_adapters, max_rank, max_tokens, len(proj_in),
                                   _arr(proj_in, I32), _arr(proj_out, I32),
                                   compute_stream or None, copy_stream or None), "slora_pool_create")
    return out.value


def slora_pool_destroy(pool: int) -> None:
    _check(lib().slora_pool_destroy(pool), "slora_pool_destroy")


def slora_pages_alloc(pool: int, n: int) -> np.ndarray:
    out = np.empty(max(n, 0), dtype=np.int32)
    _check(lib().slora_pages_alloc(pool, n, out.ctypes.data), "slora_pages_alloc")
    return out


def slora_pages_free(pool: int, pages) -> None:
    pages = np.ascontiguousarray(pages, dtype=np.int32)
    _check(lib().slora_pages_free(pool, pages.shape[0], pages.ctypes.data), "slora_pages_free")


def slora_pool_info(pool: int):
    free, num, ppr = I64(), I64(), I64()
    H = I32()
    _check(lib().slora_pool_info(pool, ctypes.byref(free), ctypes.byref(num), ctypes.byref(H),
                                 ctypes.byref(ppr)), "slora_pool_info")
    return {"free_pages": free.value, "num_pages": num.value, "page_elems": H.value,
            "pages_per_rank": ppr.value}


def slora_adapter_load(pool: int, adapter_id: int, rank: int, h_A: Optional[Sequence[int]],
                       h_B: Optional[Sequence[int]]) -> int:
    """h_A / h_B: host addresses per projection (or None on a planning pool). Returns the event."""
    ev = P()
    A = _arr(h_A, P) if h_A is not None else None
    B = _arr(h_B, P) if h_B is not None else None
    _check(lib().slora_adapter_load(pool, adapter_id, rank, A, B, ctypes.byref(ev)), "slora_adapter_load")
    return ev.value or 0


def slora_adapter_evict(pool: int, adapter_id: int) -> None:
    _check(lib().slora_adapter_evict(pool, adapter_id), "slora_adapter_evict")


def slora_adapter_ready(pool: int, adapter_id: int) -> bool:
    r = I32()
    _check(lib().slora_adapter_ready(pool, adapter_id, ctypes.byref(r)), "slora_adapter_ready")
    return bool(r.value)


def slora_adapter_set_scale(pool: int, adapter_id: int, scale: float) -> None:
    _check(lib().slora_adapter_set_scale(pool, adapter_id, float(scale)), "slora_adapter_set_scale")


def slora_adapter_pages(pool: int, adapter_id: int) -> np.ndarray:
    n = I64()
    _check(lib().slora_adapter_pages(pool, adapter_id, None, 0, ctypes.byref(n)), "slora_adapter_pages")
    out = np.empty(n.value, dtype=np.int32)
    _check(lib().slora_adapter_pages(pool, adapter_id, out.ctypes.data, n.value, ctypes.byref(n)),
           "slora_adapter_pages")
    return out


def slora_build_segments(pool: int, d_token_adapter: int, T: int) -> slora_segments:
    seg = slora_segments()
    _check(lib().slora_build_segments(pool, d_token_adapter or None, T, ctypes.byref(seg)),
           "slora_build_segments")
    return seg


def slora_build_segments_for(pool: int, d_token_adapter: int, T: int, h_token_adapter) -> slora_segments:
    """h_token_adapter: host int32 array of the same ids (or None)."""
    seg = slora_segments()
    h = None
    if h_token_adapter is not None:
        h_token_adapter = np.ascontiguousarray(h_token_adapter, dtype=np.int32)
        h = h_token_adapter.ctypes.data
    _check(lib().slora_build_segments_for(pool, d_token_adapter or None, T, h, ctypes.byref(seg)),
           "slora_build_segments_for")
    return seg


def slora_lora_apply(pool: int, seg: slora_segments, proj: int, d_x: int, ldx: int, d_y: int, ldy: int,
                     s: float, mode: int = MODE_AUTO) -> None:
    _check(lib().slora_lora_apply(pool, ctypes.byref(seg), proj, d_x, ldx, d_y, ldy, s, mode),
           "slora_lora_apply")


def slora_lora_apply_bmm(pool: int, seg: slora_segments, proj: int, d_x: int, ldx: int, d_y: int, ldy: int,
                         s: float) -> None:
    _check(lib().slora_lora_apply_bmm(pool, ctypes.byref(seg), proj, d_x, ldx, d_y, ldy, s), "slora_lora_apply_bmm")


def slora_bmm_scratch_bytes(pool: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().slora_bmm_scratch_bytes(pool, ctypes.byref(n)), "slora_bmm_scratch_bytes")
    return n.value


def slora_lora_apply_multi(pool: int, seg: slora_segments, projs: Sequence[int], d_x: Sequence[int],
                           ldx: Sequence[int], d_y: Sequence[int], ldy: Sequence[int], s: float,
                           mode: int = MODE_AUTO) -> None:
    n = len(projs)
    _check(lib().slora_lora_apply_multi(pool, ctypes.byref(seg), n, _arr(projs, I32), _arr(d_x, P),
                                        _arr(ldx, I64), _arr(d_y, P), _arr(ldy, I64), s, mode),
           "slora_lora_apply_multi")


def slora_device_status(pool: int) -> int:
    st = I32()
    _check(lib().slora_device_status(pool, ctypes.byref(st)), "slora_device_status")
    return st.value


def slora_pool_snapshot(pool: int) -> dict:
    n = ctypes.c_size_t()
    _check(lib().slora_pool_snapshot(pool, None, ctypes.byref(n)), "slora_pool_snapshot")
    buf = np.empty(n.value, dtype=np.uint8)
    _check(lib().slora_pool_snapshot(pool, buf.ctypes.data, ctypes.byref(n)), "slora_pool_snapshot")
    num_pages, free_pages = buf[:16].view(np.int64)
    max_adapters, stride = buf[16:24].view(np.int32)
    body = buf[24:].view(np.int32)
    owner = body[:num_pages]
    rank = body[num_pages:num_pages + max_adapters]
    pt = body[num_pages + max_adapters:].reshape(max_adapters, stride)
    return {"num_pages": int(num_pages), "free_pages": int(free_pages), "owner": owner, "rank": rank,
            "page_table": pt}


def slora_timing_enable(pool: int, enable: bool) -> None:
    _check(lib().slora_timing_enable(pool, 1 if enable else 0), "slora_timing_enable")


def slora_timing_read(pool: int) -> dict:
    cap = 16
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_double * cap)()
    launches = (ctypes.c_int64 * cap)()
    n = I32()
    _check(lib().slora_timing_read(pool, cap, names, ms, launches, ctypes.byref(n)), "slora_timing_read")
    return {names[i].decode(): (ms[i], launches[i]) for i in range(n.value)}


def slora_set_tc_threshold(pool: int, min_tokens: int) -> None:
    _check(lib().slora_set_tc_threshold(pool, min_tokens), "slora_set_tc_threshold")


def slora_set_tc_min_batch(pool: int, min_tokens: int) -> None:
    _check(lib().slora_set_tc_min_batch(pool, min_tokens), "slora_set_tc_min_batch")


def slora_debug_set_fault(pool: int, kind: int, nth: int) -> None:
    _check(lib().slora_debug_set_fault(pool, kind, nth), "slora_debug_set_fault")


def slora_debug_set_wait_limit(pool: int, polls: int) -> None:
    _check(lib().slora_debug_set_wait_limit(pool, polls), "slora_debug_set_wait_limit")


def slora_debug_poke_page_table(pool: int, entry: int, value: int) -> int:
    """Writes one device page-table entry (SLORA_DEBUG build only); returns the old value."""
    old = ctypes.c_int32(0)
    _check(lib().slora_debug_poke_page_table(pool, entry, value, ctypes.byref(old)), "slora_debug_poke_page_table")
    return old.value


NOALLOC_MAX_TOKENS = 2048


def slora_lora_apply_noalloc(d_pool: int, page_elems: int, dtype: int, d_page_table: int, pt_stride: int,
                             d_rank: int, max_adapters: int, proj_in: Sequence[int], proj_out: Sequence[int],
                             proj: int, d_token_adapter: int, T: int, d_x: int, ldx: int, d_y: int, ldy: int,
                             s: float, stream: int = 0, status: int = 0) -> None:
    """The allocation-free apply (every buffer caller-owned; see slora.h).

    status: address of one int32 (device or pinned host memory) that receives
    the call's device status on the stream, or 0 for none."""
    _check(lib().slora_lora_apply_noalloc(d_pool, page_elems, dtype, d_page_table, pt_stride, d_rank,
                                          max_adapters, len(proj_in), _arr(proj_in, I32), _arr(proj_out, I32),
                                          proj, d_token_adapter or None, T, d_x or None, ldx, d_y or None, ldy, s,
                                          stream or None, status or None), "slora_lora_apply_noalloc")


# ---- paged key-value cache -------------------------------------------------------------
def slora_kv_array_ints(pool: int, layers: int, heads_q: int, heads_kv: int, head_dim: int, max_requests: int,
                        max_blocks: int) -> int:
    n = I64()
    cfg = slora_kv_config(layers, heads_q, heads_kv, head_dim, max_requests, max_blocks)
    _check(lib().slora_kv_array_ints(pool or None, ctypes.byref(cfg), ctypes.byref(n)), "slora_kv_array_ints")
    return n.value


def slora_kv_create(pool: int, layers: int, heads_q: int, heads_kv: int, head_dim: int, max_requests: int,
                    max_blocks: int, d_table: int, d_arrays: int) -> int:
    out = P()
    cfg = slora_kv_config(layers, heads_q, heads_kv, head_dim, max_requests, max_blocks)
    _check(lib().slora_kv_create(ctypes.byref(out), pool or None, ctypes.byref(cfg), d_table or None,
                                 d_arrays or None), "slora_kv_create")
    return out.value


def slora_kv_destroy(kv: int) -> None:
    _check(lib().slora_kv_destroy(kv), "slora_kv_destroy")


def slora_kv_set_rotary(kv: int, rot_dim: int, layout: int, inv_freq: Sequence[float], mscale: float = 1.0) -> None:
    """inv_freq: rot_dim / 2 host floats, radians a position."""
    if len(inv_freq) < rot_dim // 2:
        raise ValueError(f"{rot_dim // 2} frequencies are needed, got {len(inv_freq)}")
    _check(lib().slora_kv_set_rotary(kv, rot_dim, layout, _arr([float(f) for f in inv_freq], ctypes.c_double),
                                     float(mscale)), "slora_kv_set_rotary")


def slora_kv_plan(kv: int, R: int, d_row: int, d_ctx: int, d_new: int, d_pages: int, n_pages: int, T: int,
                  max_new: int) -> slora_kv_batch:
    b = slora_kv_batch()
    _check(lib().slora_kv_plan(kv, R, d_row or None, d_ctx or None, d_new or None, d_pages or None, n_pages, T,
                               max_new, ctypes.byref(b)), "slora_kv_plan")
    return b


def slora_kv_append(kv: int, batch: slora_kv_batch, layer: int, d_q: int, ldq: int, d_k: int, ldk: int, d_v: int,
                    ldv: int, d_q_weight: int, d_k_weight: int, eps: float, d_q_out: int, ldqo: int) -> None:
    _check(lib().slora_kv_append(kv, ctypes.byref(batch), layer, d_q or None, ldq, d_k or None, ldk, d_v or None, ldv,
                                 d_q_weight or None, d_k_weight or None, eps, d_q_out or None, ldqo),
           "slora_kv_append")


def slora_kv_attend(kv: int, batch: slora_kv_batch, layer: int, d_q: int, ldq: int, d_out: int, ldo: int,
                    scale: float, softcap: float = 0.0) -> None:
    _check(lib().slora_kv_attend(kv, ctypes.byref(batch), layer, d_q or None, ldq, d_out or None, ldo, scale, softcap),
           "slora_kv_attend")


# ---- convenience wrapper for torch tensors -----------------------------------------
class Pool:
    """A pool over a torch device buffer (or a planning pool when device=None).

    buffer: the device buffer, a contiguous [num_pages, H] tensor of the
    pool's type (default: one is allocated)."""

    def __init__(self, num_pages: int, H: int, dtype: str, projections, max_adapters: int, max_rank: int,
                 max_tokens: int, device=None, compute_stream=None, copy_stream=None, buffer=None):
        import torch

        self.H, self.dtype = int(H), dtype
        self.projections = [(int(i), int(o)) for i, o in projections]
        self.tdtype = torch.float16 if dtype == "f16" else torch.bfloat16
        self.buffer = None
        d_pool, cs, ps = 0, 0, 0
        if device is not None:
            if buffer is None:
                buffer = torch.empty((int(num_pages), int(H)), dtype=self.tdtype, device=device)
            elif (buffer.dtype != self.tdtype or tuple(buffer.shape) != (num_pages, H) or not buffer.is_contiguous()
                  or not buffer.is_cuda):
                raise ValueError(f"buffer must be a contiguous CUDA tensor of {num_pages} x {H} {dtype} elements")
            self.buffer = buffer
            d_pool = self.buffer.data_ptr()
            self.compute_stream = compute_stream or torch.cuda.current_stream(device)
            self.copy_stream = copy_stream or torch.cuda.Stream(device)
            cs, ps = self.compute_stream.cuda_stream, self.copy_stream.cuda_stream
        self.handle = slora_pool_create(d_pool, num_pages, H, F16 if dtype == "f16" else BF16, max_adapters,
                                        max_rank, max_tokens, [i for i, _ in self.projections],
                                        [o for _, o in self.projections], cs, ps)
        self._arena = None
        self._arena_t = None
        self._arena_off = 0

    def close(self):
        if self.handle:
            slora_pool_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load(self, adapter_id: int, rank: int, weights=None) -> int:
        """weights: per projection (A rows [r, h_in], B rows [r, h_out]) uint16 arrays, or None.

        The arrays are copied into a pinned host arena that the asynchronous
        copies read from; the arena is reused only after the copy stream has
        drained (``sync_loads``), so callers may drop their arrays at once.
        """
        if weights is None:
            return slora_adapter_load(self.handle, adapter_id, rank, None, None)
        arrays = []
        for A, B in weights:
            arrays += [np.ascontiguousarray(A, dtype=np.uint16), np.ascontiguousarray(B, dtype=np.uint16)]
        need = sum(a.nbytes + 16 for a in arrays)
        if self._arena is None or self._arena_off + need > self._arena.nbytes:
            self.sync_loads()
            if self._arena is None or need > self._arena.nbytes:
                import torch

                size = max(need, 256 << 20)
                self._arena_t = torch.empty(size, dtype=torch.uint8).pin_memory()
                self._arena = self._arena_t.numpy()
        addrs = []
        base = self._arena.ctypes.data
        for a in arrays:
            off = (self._arena_off + 15) & ~15
            self._arena[off:off + a.nbytes] = a.view(np.uint8).reshape(-1)
            addrs.append(base + off)
            self._arena_off = off + a.nbytes
        return slora_adapter_load(self.handle, adapter_id, rank, addrs[0::2], addrs[1::2])

    def set_scale(self, adapter_id: int, scale: float) -> None:
        slora_adapter_set_scale(self.handle, adapter_id, scale)

    def sync_loads(self):
        if self.buffer is not None:
            self.copy_stream.synchronize()
        self._arena_off = 0

    def replay(self, ops, ranks, weights_of=None) -> dict:
        """Replay a workload's pool call sequence; returns the KV handles' page lists."""
        handles = {}
        for op in ops:
            if op[0] == "kv_alloc":
                handles[op[1]] = slora_pages_alloc(self.handle, op[2])
            elif op[0] == "kv_free":
                slora_pages_free(self.handle, handles[op[1]][np.asarray(op[2], dtype=np.int64)])
            elif op[0] == "load":
                a = op[1]
                w = weights_of(a) if weights_of is not None else None
                self.load(a, int(ranks[a]), w)
            elif op[0] == "evict":
                slora_adapter_evict(self.handle, op[1])
            else:
                raise ValueError(op)
        self.sync_loads()
        return handles

    def build_segments(self, token_adapter_dev) -> slora_segments:
        return slora_build_segments(self.handle, token_adapter_dev.data_ptr() if token_adapter_dev.numel() else 0,
                                    int(token_adapter_dev.numel()))

    def apply(self, seg, proj: int, x, y, s: float, mode: int = MODE_AUTO) -> None:
        slora_lora_apply(self.handle, seg, proj, x.data_ptr(), x.stride(0), y.data_ptr(), y.stride(0), s, mode)

    def apply_bmm(self, seg, proj: int, x, y, s: float) -> None:
        """The padded batched-matmul comparator (slora_lora_apply_bmm)."""
        slora_lora_apply_bmm(self.handle, seg, proj, x.data_ptr(), x.stride(0), y.data_ptr(), y.stride(0), s)

    def apply_multi(self, seg, projs, xs, ys, s: float, mode: int = MODE_AUTO) -> None:
        slora_lora_apply_multi(self.handle, seg, list(projs), [x.data_ptr() for x in xs],
                               [x.stride(0) for x in xs], [y.data_ptr() for y in ys],
                               [y.stride(0) for y in ys], s, mode)

    def snapshot(self) -> dict:
        return slora_pool_snapshot(self.handle)

    def status(self) -> int:
        return slora_device_status(self.handle)


class KVBatch:
    """A planned step.  The arrays of slora_kv_batch are views of the cache's
    ``arrays`` tensor, made when they are asked for (the cache's next plan
    overwrites them)."""

    __slots__ = ("raw", "ref", "R", "T", "_arrays", "_layout")

    def __init__(self, raw: slora_kv_batch, R: int, T: int, arrays, layout):
        self.raw, self.ref, self.R, self.T, self._arrays, self._layout = raw, ctypes.byref(raw), R, T, arrays, layout

    @property
    def q_start(self):
        return self._arrays.as_strided((self.R + 1,), (1,), self._layout[0])

    @property
    def kv_len(self):
        return self._arrays.as_strided((self.R,), (1,), self._layout[1])

    @property
    def tok_req(self):
        return self._arrays.as_strided((self.T,), (1,), self._layout[2])

    @property
    def tok_pos(self):
        return self._arrays.as_strided((self.T,), (1,), self._layout[3])

    @property
    def slots(self):
        _, _, _, _, at, layers, n = self._layout
        return self._arrays.as_strided((layers, 2, self.T), (2 * n, n, 1), at)


class KVCache:
    """A paged key-value cache over a Pool (slora_kv_* of slora.h).

    ``table`` is the block table [layers, 2, max_requests, max_blocks] (int32).
    Calls run on the pool's compute stream: tensors made on another stream are
    the caller's to order, as with every call on the pool.
    """

    def __init__(self, pool: Pool, layers: int, heads_q: int, heads_kv: int, head_dim: int, max_requests: int,
                 max_blocks: int):
        import torch

        self.handle = 0
        if pool.buffer is None:
            raise ValueError("a KV cache needs a pool with a device buffer")
        self.pool = pool
        self.heads_q, self.heads_kv, self.head_dim = heads_q, heads_kv, head_dim
        self.tokens_per_page = pool.H // max(1, heads_kv * head_dim)
        cfg = (layers, heads_q, heads_kv, head_dim, max_requests, max_blocks)
        n = slora_kv_array_ints(pool.handle, *cfg)     # also refuses what the cache cannot be
        i32 = dict(dtype=torch.int32, device=pool.buffer.device)
        # of the stream that writes them: memory that another one still uses is not theirs
        with torch.cuda.stream(pool.compute_stream):
            self.table = torch.empty((layers, 2, max_requests, max_blocks), **i32)
            self.arrays = torch.empty(n, **i32)
        self.handle = slora_kv_create(pool.handle, *cfg, self.table.data_ptr(), self.arrays.data_ptr())
        self._lib, self._int32, self._layout = lib(), torch.int32, None
        self._wq, self._wk = heads_q * head_dim, heads_kv * head_dim

    def close(self):
        if self.handle:
            if not self.pool.handle:
                raise RuntimeError("the pool was closed before its KV cache")
            slora_kv_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_rotary(self, rot_dim: int, inv_freq, interleaved: bool = False, mscale: float = 1.0) -> None:
        slora_kv_set_rotary(self.handle, rot_dim, ROTARY_INTERLEAVED if interleaved else ROTARY_HALF, inv_freq, mscale)

    def _i32(self, name, t):
        if t is None:
            return None
        if t.dtype is not self._int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor")
        return t.data_ptr() or None

    def _rows(self, name, t, T, cols):
        """(address, row stride) of at least T rows of `cols` contiguous elements."""
        shape, stride = t.shape, t.stride()
        if t.dtype is not self.pool.tdtype or len(shape) != 2 or shape[1] != cols or shape[0] < T or stride[1] != 1 or (
                not t.is_cuda):
            raise ValueError(f"{name} must be a CUDA {self.pool.dtype} tensor of {T} rows of {cols} contiguous elements")
        return t.data_ptr(), stride[0] if shape[0] > 1 else max(cols, stride[0])

    def _weight(self, name, t):
        if t is None:
            return None
        if t.dtype is not self.pool.tdtype or t.numel() != self.head_dim or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous CUDA {self.pool.dtype} tensor of {self.head_dim}")
        return t.data_ptr()

    def plan(self, ctx, new, pages, T: int, max_new: int, rows=None) -> KVBatch:
        """ctx, new, rows: int32 per request; pages: the opened blocks' pages in
        order (int32, [block][layer][K, V]); T: tokens the batch has room for."""
        R = ctx.numel()
        if new.numel() != R or (rows is not None and rows.numel() != R):
            raise ValueError("ctx, new and rows must have one entry per request")
        raw = slora_kv_batch()
        _check(self._lib.slora_kv_plan(self.handle, R, self._i32("rows", rows), self._i32("ctx", ctx),
                                       self._i32("new", new), self._i32("pages", pages),
                                       pages.numel() if pages is not None else 0, T, max_new, ctypes.byref(raw)),
               "slora_kv_plan")
        if self._layout is None:       # where the arrays lie, the same in every batch
            base = self.arrays.data_ptr()
            self._layout = (*((p - base) // 4 for p in (raw.q_start, raw.kv_len, raw.tok_req, raw.tok_pos, raw.slots)),
                            self.table.shape[0], raw.slot_stride)
        return KVBatch(raw, R, T, self.arrays, self._layout)

    def append(self, batch: KVBatch, layer: int, q, k, v, q_out=None, q_weight=None, k_weight=None,
               eps: float = 1e-6) -> None:
        """q [T, heads_q * head_dim] (rotated into q_out, or in place), k and v
        [T, heads_kv * head_dim] (stored); q_weight, k_weight [head_dim]."""
        T, wq, wk = batch.raw.T, self._wq, self._wk
        pq, ldq = self._rows("q", q, T, wq)
        pk, ldk = self._rows("k", k, T, wk)
        pv, ldv = self._rows("v", v, T, wk)
        po, ldo = (pq, ldq) if q_out is None else self._rows("q_out", q_out, T, wq)
        _check(self._lib.slora_kv_append(self.handle, batch.ref, layer, pq, ldq, pk, ldk, pv, ldv,
                                         self._weight("q_weight", q_weight), self._weight("k_weight", k_weight), eps,
                                         po, ldo), "slora_kv_append")

    def attend(self, batch: KVBatch, layer: int, q, out, scale: Optional[float] = None, softcap: float = 0.0) -> None:
        """out[t] = attention of token t's heads over its request's stored tokens
        (scale: 1 / sqrt(head_dim) by default)."""
        T = batch.raw.T
        pq, ldq = self._rows("q", q, T, self._wq)
        po, ldo = self._rows("out", out, T, self._wq)
        _check(self._lib.slora_kv_attend(self.handle, batch.ref, layer, pq, ldq, po, ldo,
                                         self.head_dim ** -0.5 if scale is None else scale, softcap), "slora_kv_attend")
