"""Thin ctypes binding over libsva.so (include/sva.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. torch is used for device memory and streams; tensors are passed by
data_ptr(), streams by their cudaStream_t handle. Any non-OK status raises
SvError with the library's own message. There is no fallback: if libsva.so is
missing or was built for another machine, loading it raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

import torch

from . import workloads as W

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsva.so")

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_WORKSPACE, SV_ERR_CUDA, \
    SV_ERR_DEVICE_FAULT = range(6)
SV_BF16, SV_F32 = 0, 1
SV_FLAG_BAD_BLOCK_INDEX, SV_FLAG_BAD_PAGE, SV_FLAG_WAIT_TIMEOUT, SV_FLAG_STALE_WORKSPACE, \
    SV_FLAG_NO_PAGE, SV_FLAG_BAD_LENGTH = 1, 2, 4, 8, 16, 32

SV_PATH_CUDA_CORES, SV_PATH_MMA_SYNC, SV_PATH_TCGEN05 = 0, 1, 2
ABI_VERSION = 4  # SV_ABI_VERSION the structures below match

EXPORTED = ("sv_abi_version", "sv_last_error", "sv_budget_blocks", "sv_workspace_bytes",
            "sv_clear_status", "sv_read_status", "sv_build_reps", "sv_score_blocks",
            "sv_select_blocks", "sv_score_select", "sv_sparse_attend", "sv_attend_plan",
            "sv_verify_layer", "sv_sparse_attend_noalloc", "sv_append_kv",
            "sv_selection_overlap", "sv_reset_workspace", "sv_verify_layer_host",
            "sv_build_tables", "sv_write_kv", "sv_prompt_workspace_bytes",
            "sv_prefix_workspace_bytes", "sv_prompt_attend", "sv_prefix_attend", "sv_norm_rope",
            "sv_rope_write_kv", "sv_kv4_page_bytes", "sv_write_kv4", "sv_read_kv4",
            "sv_build_reps_kv4", "sv_kv4_workspace_bytes", "sv_attend_kv4")


class SvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"sva status {status}: {msg}")
        self.status = status


class Shape(C.Structure):
    _fields_ = [("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("d", C.c_int),
                ("blk", C.c_int), ("T", C.c_int), ("dtype", C.c_int)]


class BudgetC(C.Structure):
    _fields_ = [("mode", C.c_int), ("fixed_blocks", C.c_int), ("short_ctx", C.c_int),
                ("floor_blocks", C.c_int), ("frac_mid", C.c_double), ("long_ctx", C.c_int),
                ("frac_long", C.c_double)]


class KV(C.Structure):
    _fields_ = [("k_pool", C.c_void_p), ("v_pool", C.c_void_p), ("block_table", C.c_void_p),
                ("nb_max", C.c_int), ("num_pages", C.c_int), ("ctx", C.c_int),
                ("seq_ctx", C.POINTER(C.c_int32))]


class Rope(C.Structure):
    _fields_ = [("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("table", C.c_void_p),
                ("eps", C.c_float), ("max_pos", C.c_int), ("rot", C.c_int), ("interleaved", C.c_int)]


class KV4(C.Structure):
    _fields_ = [("k_pool", C.c_void_p), ("v_pool", C.c_void_p), ("block_table", C.c_void_p),
                ("seq_ctx", C.c_void_p), ("k_exp", C.c_void_p), ("v_exp", C.c_void_p),
                ("nb_max", C.c_int), ("num_pages", C.c_int)]


class SelSlotC(C.Structure):
    _fields_ = [("sel", C.c_void_p), ("kmax", C.c_int), ("stamp", C.c_uint64)]


class SelSlot:
    """A selection cache slot (sv_sel_slot): the device selection [B, Hkv,
    kmax] int32 and the host-side stamp the library writes when a computing
    layer fills it and checks when a reuse layer reads it."""

    def __init__(self, B: int, Hkv: int, kmax: int, device="cuda"):
        self.tensor = torch.full((B, Hkv, max(kmax, 1)), -1, dtype=torch.int32, device=device)
        self.c = SelSlotC(self.tensor.data_ptr(), kmax, 0)

    def copy(self) -> "SelSlot":
        """A new slot holding a copy of this one's selection and stamp."""
        new = SelSlot.__new__(SelSlot)
        new.tensor = self.tensor.clone()
        new.c = SelSlotC(new.tensor.data_ptr(), self.c.kmax, self.c.stamp)
        return new

    @property
    def kmax(self) -> int:
        return self.c.kmax


class Plan(C.Structure):
    _fields_ = [("path", C.c_int), ("cluster", C.c_int), ("n_splits", C.c_int),
                ("blocks_per_split", C.c_int), ("ctas_per_sm", C.c_int),
                ("split_extra", C.c_int), ("streamk", C.c_int)]


_lib = None


def lib() -> C.CDLL:
    """Load libsva.so (once). Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "sparse_verification_attention_gb300.build_lib.build()")
        L = C.CDLL(LIB_PATH)
        vp, i, sz, ll = C.c_void_p, C.c_int, C.c_size_t, C.c_longlong
        sig = {
            "sv_abi_version": (i, []),
            "sv_last_error": (C.c_char_p, []),
            "sv_budget_blocks": (i, [C.POINTER(BudgetC), i, i]),
            "sv_workspace_bytes": (sz, [C.POINTER(Shape), i, i]),
            "sv_clear_status": (i, [vp, vp]),
            "sv_read_status": (i, [vp, C.POINTER(C.c_uint32), vp]),
            "sv_build_reps": (i, [C.POINTER(Shape), C.POINTER(KV), i, i, vp, vp]),
            "sv_score_blocks": (i, [C.POINTER(Shape), vp, vp, C.POINTER(KV), vp, vp]),
            "sv_select_blocks": (i, [C.POINTER(Shape), vp, i, i, vp, i, vp]),
            "sv_score_select": (i, [C.POINTER(Shape), vp, vp, C.POINTER(KV), C.POINTER(BudgetC),
                                    vp, i, C.POINTER(C.c_int), vp, sz, vp]),
            "sv_sparse_attend": (i, [C.POINTER(Shape), vp, C.POINTER(KV), vp, i, i, vp, vp,
                                     C.POINTER(C.c_int32), vp, vp, sz, vp]),
            "sv_attend_plan": (i, [C.POINTER(Shape), C.POINTER(KV), i, C.POINTER(Plan)]),
            "sv_verify_layer": (i, [C.POINTER(Shape), vp, C.POINTER(KV), vp, C.POINTER(BudgetC),
                                    vp, vp, C.POINTER(C.c_int32), i, C.POINTER(SelSlotC),
                                    C.POINTER(C.c_int), vp, vp, sz, vp]),
            "sv_sparse_attend_noalloc": (i, [C.POINTER(Shape), vp, C.POINTER(KV), vp, i, i, vp,
                                             vp, C.POINTER(C.c_int32), vp, vp, vp]),
            "sv_append_kv": (i, [C.POINTER(Shape), vp, vp, vp, i, i, vp, vp, vp, vp, vp, vp, vp,
                                 vp]),
            "sv_selection_overlap": (i, [vp, i, i, i, i, C.POINTER(C.c_int32), vp, vp, vp]),
            "sv_reset_workspace": (i, [C.POINTER(Shape), i, i, vp, sz, vp]),
            "sv_verify_layer_host": (i, [C.POINTER(Shape), vp, vp, C.POINTER(KV), vp,
                                         C.POINTER(BudgetC), vp, vp, vp, vp,
                                         C.POINTER(C.c_int32), i, C.POINTER(SelSlotC),
                                         C.POINTER(C.c_int), vp, vp, vp, sz, vp, vp, vp]),
            "sv_build_tables": (i, [i, i, vp, vp, vp, vp, i, i, vp, vp, vp, vp, vp, vp, i, vp, vp]),
            "sv_write_kv": (i, [C.POINTER(Shape), vp, ll, vp, ll, vp, i, vp, vp, i, vp, vp]),
            "sv_prompt_workspace_bytes": (sz, [C.POINTER(Shape), i]),
            "sv_prefix_workspace_bytes": (sz, [C.POINTER(Shape)]),
            "sv_prompt_attend": (i, [C.POINTER(Shape), vp, ll, i, vp, vp, vp, i, i, vp, vp, vp, vp,
                                     sz, vp]),
            "sv_prefix_attend": (i, [C.POINTER(Shape), vp, C.POINTER(KV), i, vp, vp,
                                     C.POINTER(C.c_int32), vp, vp, sz, vp]),
            "sv_norm_rope": (i, [C.POINTER(Shape), C.POINTER(Rope), vp, i, vp, ll, vp, ll, vp, ll, vp,
                                 ll, vp, vp]),
            "sv_rope_write_kv": (i, [C.POINTER(Shape), C.POINTER(Rope), vp, i, vp, ll, vp, ll, vp, ll,
                                     vp, ll, vp, vp, vp, i, vp, vp]),
            "sv_kv4_page_bytes": (sz, [C.POINTER(Shape)]),
            "sv_write_kv4": (i, [C.POINTER(Shape), vp, ll, vp, ll, vp, i, C.POINTER(KV4), vp, vp]),
            "sv_read_kv4": (i, [C.POINTER(Shape), C.POINTER(KV4), vp, i, vp, ll, vp, ll, vp, vp]),
            "sv_build_reps_kv4": (i, [C.POINTER(Shape), C.POINTER(KV4), vp, i, vp, vp, vp]),
            "sv_kv4_workspace_bytes": (sz, [C.POINTER(Shape)]),
            "sv_attend_kv4": (i, [C.POINTER(Shape), vp, C.POINTER(KV4), vp, i, i, vp, vp,
                                  C.POINTER(C.c_int32), vp, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        if L.sv_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI {L.sv_abi_version()}, the binding expects "
                               f"{ABI_VERSION}: rebuild it")
        _lib = L
    return _lib


def _check(status: int):
    if status != SV_OK:
        raise SvError(status, lib().sv_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return SV_BF16
    if t == torch.float32:
        return SV_F32
    raise ValueError(f"unsupported dtype {t}")


def make_shape(B, Hq, Hkv, d, blk, T, dtype) -> Shape:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return Shape(B, Hq, Hkv, d, blk, T, code)


def make_budget(b: W.Budget) -> BudgetC:
    return BudgetC(b.mode, b.fixed_blocks, b.short_ctx, b.floor_blocks, b.frac_mid, b.long_ctx,
                   b.frac_long)


def make_kv(k_pool: torch.Tensor, v_pool: Optional[torch.Tensor], block_table: torch.Tensor,
            ctx: int, seq_ctx: Optional[Sequence[int]] = None) -> KV:
    """The cache descriptor. seq_ctx (one prefix length per sequence, kept on
    the host) replaces the uniform ctx; the returned structure owns the
    array it points to, and keeps the tensors. The library reads B entries of
    seq_ctx, so it must have one per row of the block table."""
    kv = KV(k_pool.data_ptr(), None if v_pool is None else v_pool.data_ptr(),
            block_table.data_ptr(), block_table.shape[1], k_pool.shape[0], ctx)
    kv._tensors = k_pool, v_pool, block_table
    if seq_ctx is not None:
        if len(seq_ctx) != block_table.shape[0]:
            raise ValueError(f"seq_ctx has {len(seq_ctx)} entries for "
                             f"{block_table.shape[0]} sequences")
        arr = (C.c_int32 * len(seq_ctx))(*[int(c) for c in seq_ctx])
        kv._seq_ctx_keep = arr
        kv.seq_ctx = arr
    return kv


_parents_cache: dict = {}


def _parents(parents: Optional[Sequence[int]]):
    if parents is None:
        return None
    key = tuple(parents)
    arr = _parents_cache.get(key)
    if arr is None:  # the C array is only read during the call
        arr = (C.c_int32 * len(key))(*key)
        if len(_parents_cache) < 64:
            _parents_cache[key] = arr
    return arr


# ------------------------------------------------------------------ calls
def sv_abi_version() -> int:
    return lib().sv_abi_version()


def sv_budget_blocks(budget: W.Budget, ctx: int, nb: int) -> int:
    b = make_budget(budget)
    return lib().sv_budget_blocks(C.byref(b), ctx, nb)


def sv_workspace_bytes(shape: Shape, nb_max: int, kmax: int) -> int:
    return lib().sv_workspace_bytes(C.byref(shape), nb_max, kmax)


def alloc_workspace(shape: Shape, nb_max: int, kmax: int, device="cuda") -> torch.Tensor:
    n = sv_workspace_bytes(shape, nb_max, kmax)
    if n == 0:
        raise SvError(SV_ERR_INVALID_ARG, "invalid shape for a workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def sv_clear_status(ws: torch.Tensor, stream=None):
    _check(lib().sv_clear_status(_ptr(ws), _stream(stream)))


def sv_reset_workspace(shape: Shape, nb_max: int, kmax: int, ws: torch.Tensor, stream=None):
    """Zero the workspace's status word and per-(b, h) counts and flags (what
    a workspace needs after a call that raised SV_FLAG_WAIT_TIMEOUT)."""
    _check(lib().sv_reset_workspace(C.byref(shape), nb_max, kmax, _ptr(ws), ws.numel(),
                                    _stream(stream)))


def sv_read_status(ws: torch.Tensor, stream=None) -> int:
    """Device status flags (0 = clean). Does not raise on set flags."""
    v = C.c_uint32(0)
    lib().sv_read_status(_ptr(ws), C.byref(v), _stream(stream))
    return int(v.value)


def sv_build_reps(shape: Shape, kv: KV, first_block: int, n_blocks: int, reps: torch.Tensor,
                  stream=None):
    _check(lib().sv_build_reps(C.byref(shape), C.byref(kv), first_block, n_blocks, _ptr(reps),
                               _stream(stream)))


def sv_score_blocks(shape: Shape, q, reps, kv: KV, scores, stream=None):
    _check(lib().sv_score_blocks(C.byref(shape), _ptr(q), _ptr(reps), C.byref(kv), _ptr(scores),
                                 _stream(stream)))


def sv_select_blocks(shape: Shape, scores, nb: int, k: int, sel, kmax: int, stream=None):
    _check(lib().sv_select_blocks(C.byref(shape), _ptr(scores), nb, k, _ptr(sel), kmax,
                                  _stream(stream)))


def sv_score_select(shape: Shape, q, reps, kv: KV, budget: W.Budget, sel, kmax: int, ws,
                    stream=None) -> int:
    b = make_budget(budget)
    k = C.c_int(-1)
    _check(lib().sv_score_select(C.byref(shape), _ptr(q), _ptr(reps), C.byref(kv), C.byref(b),
                                 _ptr(sel), kmax, C.byref(k), _ptr(ws),
                                 0 if ws is None else ws.numel(), _stream(stream)))
    return k.value


def sv_sparse_attend(shape: Shape, q, kv: KV, sel, n_sel: int, sel_stride: int, draft_k, draft_v,
                     parents, out, ws, stream=None):
    _check(lib().sv_sparse_attend(C.byref(shape), _ptr(q), C.byref(kv), _ptr(sel), n_sel,
                                  sel_stride, _ptr(draft_k), _ptr(draft_v), _parents(parents),
                                  _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                  _stream(stream)))


def sv_sparse_attend_noalloc(shape: Shape, q, kv: KV, sel, n_sel: int, sel_stride: int, draft_k,
                             draft_v, parents, out, flags_out=None, stream=None):
    """sv_sparse_attend with the library's static scratch instead of a
    workspace, for callers that cannot allocate device memory. flags_out: an
    optional device uint32/int32 tensor of one element that receives the
    call's status flags. Calls whose GPU work overlaps race on the scratch."""
    _check(lib().sv_sparse_attend_noalloc(C.byref(shape), _ptr(q), C.byref(kv), _ptr(sel), n_sel,
                                          sel_stride, _ptr(draft_k), _ptr(draft_v),
                                          _parents(parents), _ptr(out), _ptr(flags_out),
                                          _stream(stream)))


def sv_append_kv(shape: Shape, k_pool, v_pool, block_table, seq_ctx, n_accept, accept_idx,
                 draft_k, draft_v, reps=None, ws=None, stream=None):
    """Append each sequence's accepted drafts to its paged cache (and rebuild
    the representatives of blocks that fill). seq_ctx, n_accept: device int32
    [B]; accept_idx: device int32 [B, T]."""
    _check(lib().sv_append_kv(C.byref(shape), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                              block_table.shape[1], k_pool.shape[0], _ptr(seq_ctx),
                              _ptr(n_accept), _ptr(accept_idx), _ptr(draft_k), _ptr(draft_v),
                              _ptr(reps), _ptr(ws), _stream(stream)))


def sv_selection_overlap(sels, k: int, parents, overlap0, by_distance, stream=None):
    """Overlaps of T per-draft selections. sels: device int32 [T, pairs, kmax]
    (each row ascending in its first k entries); overlap0, by_distance:
    device float32 [pairs, T], written."""
    T, pairs, kmax = sels.shape
    _check(lib().sv_selection_overlap(_ptr(sels), T, pairs, kmax, k, _parents(parents),
                                      _ptr(overlap0), _ptr(by_distance), _stream(stream)))


def sv_attend_plan(shape: Shape, kv: KV, n_sel: int) -> Plan:
    p = Plan()
    _check(lib().sv_attend_plan(C.byref(shape), C.byref(kv), n_sel, C.byref(p)))
    return p


def sv_verify_layer(shape: Shape, q, kv: KV, reps, budget: Optional[W.Budget], draft_k, draft_v,
                    parents, reuse: int, slot: Optional[SelSlot], out, ws, stream=None) -> int:
    b = None if budget is None else C.byref(make_budget(budget))
    k = C.c_int(-1)
    _check(lib().sv_verify_layer(C.byref(shape), _ptr(q), C.byref(kv), _ptr(reps), b,
                                 _ptr(draft_k), _ptr(draft_v), _parents(parents), int(reuse),
                                 None if slot is None else C.byref(slot.c), C.byref(k), _ptr(out),
                                 _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return k.value


def sv_verify_layer_host(shape: Shape, q_host, q, kv: KV, reps, budget: Optional[W.Budget],
                         dk_host, dv_host, draft_k, draft_v, parents, reuse: int,
                         slot: Optional[SelSlot], out_host, out, ws, stream=None,
                         copy_in_stream=None, copy_out_stream=None) -> int:
    """sv_verify_layer with q, draft K/V and the output in host memory
    (pinned tensors for asynchronous copies); q, draft_k, draft_v and out are
    the device buffers the call stages them through."""
    b = None if budget is None else C.byref(make_budget(budget))
    k = C.c_int(-1)
    ci = None if copy_in_stream is None else _stream(copy_in_stream)
    co = None if copy_out_stream is None else _stream(copy_out_stream)
    _check(lib().sv_verify_layer_host(
        C.byref(shape), _ptr(q_host), _ptr(q), C.byref(kv), _ptr(reps), b, _ptr(dk_host),
        _ptr(dv_host), _ptr(draft_k), _ptr(draft_v), _parents(parents), int(reuse),
        None if slot is None else C.byref(slot.c), C.byref(k), _ptr(out_host), _ptr(out), _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream), ci, co))
    return k.value


# ------------------------------------------------------------------ paged cache
# A decoding step makes these calls once per layer, and their kernels take a few
# microseconds: the checks read each attribute of a tensor once, and pointers and
# streams go to ctypes as plain integers.
_DTYPES = (torch.bfloat16, torch.float32)  # by dtype code


def _call(fn, tensors, stream, *args):
    """fn(*args, stream) with the tensors' device current. None stands for an
    argument that is left out; the others must lie on one CUDA device."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            dev = -1
            break
    if dev < 0:
        raise ValueError("the tensors of a call must lie on one CUDA device")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != SV_OK:
        _check(status)


def _ints(name: str, t: torch.Tensor, *shape) -> int:
    """The address of t, which must be a dense int32 tensor of this shape."""
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)}")
    return t.data_ptr()


def _dense(name: str, t: torch.Tensor, dtype: torch.dtype, *shape) -> int:
    """The address of t, which must be a dense tensor of the call's dtype and this shape."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of dtype {dtype} and of shape {list(shape)}")
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, dtype: torch.dtype, heads: int, d: int) -> int:
    """The distance of t's rows [n, heads, d], in elements; rows may be strided."""
    shape, stride = t.shape, t.stride()
    if t.dtype != dtype or len(shape) != 3 or shape[1] != heads or shape[2] != d or \
            (shape[0] and (stride[2] != 1 or (heads > 1 and stride[1] != d))):
        raise ValueError(f"{name} must be rows [n, {heads}, {d}] of dtype {dtype}, each row dense")
    return stride[0] if shape[0] > 1 else heads * d


def _row_array(name: str, t: torch.Tensor, dtype: torch.dtype, heads: int, d: int):
    """The number of t's rows [n, heads, d], their address and distance (see _rows)."""
    shape, stride = t.shape, t.stride()
    n = shape[0] if shape else 0
    if t.dtype != dtype or shape != (n, heads, d) or (n and (stride[2] != 1 or (heads > 1 and stride[1] != d))):
        raise ValueError(f"{name} must be rows [n, {heads}, {d}] of dtype {dtype}, each row dense")
    return n, t.data_ptr(), stride[0] if n > 1 else heads * d


def _same_device(dev: int, tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("the tensors of a call must lie on one CUDA device")


def _workspace(ws: Optional[torch.Tensor]):
    """Address and bytes of a workspace (or of a status word), None and 0 without one."""
    if ws is None:
        return None, 0
    n = ws.numel() * ws.element_size()
    if n < 4 or not ws.is_contiguous():
        raise ValueError("the workspace must be a dense tensor that holds a status word at least")
    return ws.data_ptr(), n


def sv_build_tables(blk: int, old_len, new_len, block_table, free_pages, free_count, free_count_out,
                    cu_new, slot_map, positions=None, pinned=None, ws=None, stream=None):
    """Pages for requests that go from old_len to new_len tokens, and the slots
    (and positions) of their new tokens. All tensors int32 on the device:
    old_len, new_len, pinned [B]; block_table [B, nb_max]; free_pages
    [num_pages], a stack of which free_count[0] entries are free; free_count_out
    [1] (may be free_count); cu_new [B + 1]; slot_map, positions [n_max]."""
    B, nb_max = block_table.shape
    (n_max,), (num_pages,) = slot_map.shape, free_pages.shape
    _call(lib().sv_build_tables,
          (old_len, new_len, pinned, block_table, free_pages, free_count, free_count_out, cu_new,
           slot_map, positions, ws), stream,
          B, blk, _ints("old_len", old_len, B), _ints("new_len", new_len, B),
          None if pinned is None else _ints("pinned", pinned, B),
          _ints("block_table", block_table, B, nb_max), nb_max, num_pages,
          _ints("free_pages", free_pages, num_pages), _ints("free_count", free_count, 1),
          _ints("free_count_out", free_count_out, 1), _ints("cu_new", cu_new, B + 1),
          _ints("slot_map", slot_map, n_max),
          None if positions is None else _ints("positions", positions, n_max), n_max, _workspace(ws)[0])


def sv_write_kv(shape: Shape, k, v, slot_map, k_pool, v_pool, ws=None, stream=None):
    """Store the rows k, v [n, Hkv, d] (slices of a fused projection are fine) at
    their slots of the paged cache; slots of -1 are skipped."""
    H, d, dtype = shape.Hkv, shape.d, _DTYPES[shape.dtype]
    ks, vs = _rows("k", k, dtype, H, d), _rows("v", v, dtype, H, d)
    n, pages = k.shape[0], k_pool.shape[0]
    if v.shape[0] != n:
        raise ValueError(f"{n} key rows and {v.shape[0]} value rows")
    pool = (pages, H, shape.blk, d)
    _call(lib().sv_write_kv, (k, v, slot_map, k_pool, v_pool, ws), stream, C.byref(shape),
          k.data_ptr(), ks, v.data_ptr(), vs, _ints("slot_map", slot_map, n), n,
          _dense("k_pool", k_pool, dtype, *pool), _dense("v_pool", v_pool, dtype, *pool), pages,
          _workspace(ws)[0])


def _alloc_zeroed(n: int, device) -> torch.Tensor:
    if n == 0:
        raise SvError(SV_ERR_INVALID_ARG, "invalid shape for a workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_prompt_workspace(shape: Shape, n_rows: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for sv_prompt_attend calls of up to n_rows rows."""
    return _alloc_zeroed(lib().sv_prompt_workspace_bytes(C.byref(shape), n_rows), device)


def alloc_prefix_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    """A zeroed workspace for sv_prefix_attend calls with this shape."""
    return _alloc_zeroed(lib().sv_prefix_workspace_bytes(C.byref(shape)), device)


def sv_prompt_attend(shape: Shape, q, k_pool, v_pool, block_table, seq_ctx, cu_q, out, ws,
                     stream=None):
    """Causal attention of the packed rows q [n, Hq, d] (rows may be strided)
    over the paged cache: rows cu_q[b] .. cu_q[b+1] are the last of the
    seq_ctx[b] cached tokens of sequence b. out: [n, Hq, d]."""
    B, Hq, d, dtype = shape.B, shape.Hq, shape.d, _DTYPES[shape.dtype]
    qs = _rows("q", q, dtype, Hq, d)
    n, pages, nb_max = q.shape[0], k_pool.shape[0], block_table.shape[-1]
    pool = (pages, shape.Hkv, shape.blk, d)
    _call(lib().sv_prompt_attend, (q, k_pool, v_pool, block_table, seq_ctx, cu_q, out, ws), stream,
          C.byref(shape), q.data_ptr(), qs, n, _dense("k_pool", k_pool, dtype, *pool),
          _dense("v_pool", v_pool, dtype, *pool), _ints("block_table", block_table, B, nb_max),
          nb_max, pages, _ints("seq_ctx", seq_ctx, B), _ints("cu_q", cu_q, B + 1),
          _dense("out", out, dtype, n, Hq, d), *_workspace(ws))


def _check_cache(shape: Shape, dtype: torch.dtype, k_pool, v_pool, table):
    """A descriptor's tensors must be a cache of this shape, for shape.B sequences at least."""
    pages = k_pool.shape
    if pages[1:] != (shape.Hkv, shape.blk, shape.d) or k_pool.dtype != dtype or not k_pool.is_contiguous():
        raise ValueError(f"the k_pool of kv must be contiguous, of dtype {dtype} and of shape "
                         f"[pages, {shape.Hkv}, {shape.blk}, {shape.d}]")
    if v_pool is not None and \
            (v_pool.shape != pages or v_pool.dtype != dtype or not v_pool.is_contiguous()):
        raise ValueError("the v_pool of kv must be as its k_pool")
    if table.shape[0] < shape.B or table.dtype != torch.int32 or not table.is_contiguous():
        raise ValueError(f"the block_table of kv must be contiguous, int32 and have {shape.B} rows")


def sv_prefix_attend(shape: Shape, q, kv: KV, n_shared: int, draft_k, draft_v, parents, out, ws,
                     stream=None):
    """sv_sparse_attend over every block for a batch whose sequences share
    their first n_shared blocks: those are read once for all of them."""
    B, T, d, dtype = shape.B, shape.T, shape.d, _DTYPES[shape.dtype]
    rows, drafts = (B, T, shape.Hq, d), (B, T, shape.Hkv, d)
    if parents is not None and len(parents) != T:
        raise ValueError(f"{len(parents)} draft parents for T={T} drafts")
    cache = getattr(kv, "_tensors", ())  # none in a descriptor filled by hand
    if cache:
        _check_cache(shape, dtype, *cache)
    _call(lib().sv_prefix_attend, (q, draft_k, draft_v, out, ws, *cache), stream, C.byref(shape),
          _dense("q", q, dtype, *rows), C.byref(kv), n_shared,
          _dense("draft_k", draft_k, dtype, *drafts), _dense("draft_v", draft_v, dtype, *drafts),
          _parents(parents), _dense("out", out, dtype, *rows), *_workspace(ws))


# ------------------------------------------------------------------ head norms, rotation, 4-bit cache
def rope_table(max_pos: int, rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines [max_pos, rot] fp32 of the plain rotation: pair i of
    position p turns by p * theta^(-2 i / rot). Angles are taken in 64 bits; a
    model with scaled frequencies makes its own table of this layout."""
    if max_pos < 1 or rot < 8 or rot % 8:
        raise ValueError("max_pos >= 1 and rot a positive multiple of 8")
    freq = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def make_rope(table: Optional[torch.Tensor] = None, rot: Optional[int] = None, interleaved: bool = False,
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
              eps: float = 1e-6) -> Rope:
    """The norm and rotation of a model's heads. table: fp32 [max_pos, rot] (see
    rope_table), None rotates nothing; weights [d], None norms nothing. The
    returned structure keeps the tensors."""
    if table is None:
        if rot:
            raise ValueError(f"a rotation of {rot} dims needs a table")
        max_pos, rot = 0, 0
    else:
        if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous() or \
                rot not in (None, table.shape[1]):
            raise ValueError(f"table must be a contiguous float32 tensor [max_pos, rot]{'' if rot is None else f', rot {rot}'}")
        max_pos, rot = table.shape
    r = Rope(None if q_weight is None else q_weight.data_ptr(),
             None if k_weight is None else k_weight.data_ptr(),
             None if table is None else table.data_ptr(), eps, max_pos, rot, int(interleaved))
    r._tensors = table, q_weight, k_weight
    return r


def _check_rope(rope: Rope, dtype: torch.dtype, d: int, dev: int):
    """The tensors of a rope descriptor against a call's heads and device; the descriptor
    remembers what it was last checked against."""
    fits = dtype, d, dev
    if getattr(rope, "_fits", None) == fits:
        return
    kept = getattr(rope, "_tensors", ())  # none in a descriptor filled by hand
    for w in kept[1:]:
        if w is not None and (w.dtype != dtype or w.shape != (d,) or not w.is_contiguous()):
            raise ValueError(f"norm weights must be contiguous, of dtype {dtype} and of shape [{d}]")
    _same_device(dev, kept)
    rope._fits = fits


def sv_norm_rope(shape: Shape, rope: Rope, positions, q, k, q_out, k_out, ws=None, stream=None):
    """Norm and rotate the heads of the rows q [n, Hq, d] (or None) and k [n, Hkv,
    d]; rows may be strided, q_out may be q and k_out k. positions: int32 [n],
    -1 leaves a row out (None when nothing is rotated)."""
    H, d, dtype = shape.Hkv, shape.d, _DTYPES[shape.dtype]
    n, kp, ks = _row_array("k", k, dtype, H, d)
    no, kop, kos = _row_array("k_out", k_out, dtype, H, d)
    if no != n:
        raise ValueError(f"{n} key rows and {no} rows to write")
    qp, qs, qop, qos = _q_rows(shape, dtype, n, q, q_out)
    _check_rope(rope, dtype, d, k.get_device())
    _call(lib().sv_norm_rope, (k, q, q_out, k_out, positions, ws), stream,
          C.byref(shape), C.byref(rope), None if positions is None else _ints("positions", positions, n),
          n, qp, qs, kp, ks, qop, qos, kop, kos, _workspace(ws)[0])


def _q_rows(shape: Shape, dtype: torch.dtype, n: int, q, q_out):
    """Addresses and strides of a call's query rows and of where they go."""
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out are given together")
    if q is None:
        return None, 0, None, 0
    nq, qp, qs = _row_array("q", q, dtype, shape.Hq, shape.d)
    no, qop, qos = _row_array("q_out", q_out, dtype, shape.Hq, shape.d)
    if nq != n or no != n:
        raise ValueError(f"{n} key rows, {nq} query rows and {no} rows to write")
    return qp, qs, qop, qos


def sv_rope_write_kv(shape: Shape, rope: Rope, positions, q, k, v, q_out, slot_map, k_pool, v_pool, ws=None,
                     stream=None):
    """sv_norm_rope with the keys, and the values v [n, Hkv, d] beside them, stored
    at their slots of the paged cache; q and q_out may be None."""
    H, d, dtype = shape.Hkv, shape.d, _DTYPES[shape.dtype]
    pages = k_pool.shape[0]
    n, kp, ks = _row_array("k", k, dtype, H, d)
    nv, vp, vs = _row_array("v", v, dtype, H, d)
    if nv != n:
        raise ValueError(f"{n} key rows and {nv} value rows")
    qp, qs, qop, qos = _q_rows(shape, dtype, n, q, q_out)
    pool = (pages, H, shape.blk, d)
    _check_rope(rope, dtype, d, k.get_device())
    _call(lib().sv_rope_write_kv, (k, v, q, q_out, positions, slot_map, k_pool, v_pool, ws), stream,
          C.byref(shape), C.byref(rope), None if positions is None else _ints("positions", positions, n),
          n, qp, qs, qop, qos, kp, ks, vp, vs, _ints("slot_map", slot_map, n),
          _dense("k_pool", k_pool, dtype, *pool), _dense("v_pool", v_pool, dtype, *pool), pages,
          _workspace(ws)[0])


def alloc_kv4_pool(shape: Shape, pages: int, device="cuda") -> torch.Tensor:
    """A zeroed pool of a 4-bit cache: uint8 [pages, Hkv, blk / 16, 9 d]."""
    if lib().sv_kv4_page_bytes(C.byref(shape)) == 0:
        _check(SV_ERR_INVALID_ARG)
    return torch.zeros(pages, shape.Hkv, shape.blk // 16, 9 * shape.d, dtype=torch.uint8, device=device)


def make_kv4(k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: Optional[torch.Tensor] = None,
             seq_ctx: Optional[torch.Tensor] = None, k_exp: Optional[torch.Tensor] = None,
             v_exp: Optional[torch.Tensor] = None) -> KV4:
    """The descriptor of a 4-bit cache. seq_ctx (int32 [B]) lies on the device; the
    row calls need neither it nor block_table. k_exp, v_exp: int32 [Hkv], the heads'
    exponents. The returned structure keeps the tensors."""
    ptr = [None if t is None else t.data_ptr() for t in (k_pool, v_pool, block_table, seq_ctx, k_exp, v_exp)]
    kv = KV4(*ptr, 0 if block_table is None else block_table.shape[-1], k_pool.shape[0])
    kv._tensors = k_pool, v_pool, block_table, seq_ctx, k_exp, v_exp
    return kv


def _check_kv4(shape: Shape, kv: KV4, seqs: bool, dev: int):
    """A descriptor's tensors, which must be a 4-bit cache of this shape on the call's
    device (and hold shape.B sequences); it remembers what it was last checked against."""
    fits = shape.Hkv, shape.blk, shape.d, shape.B if seqs else None, dev
    if getattr(kv, "_fits", None) == fits:
        return
    kept = getattr(kv, "_tensors", ())  # none in a descriptor filled by hand
    if not kept:
        return
    k_pool, v_pool, table, seq_ctx, k_exp, v_exp = kept
    pool = (k_pool.shape[0], shape.Hkv, shape.blk // 16, 9 * shape.d)
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t.dtype != torch.uint8 or t.shape != pool or not t.is_contiguous():
            raise ValueError(f"the {name} of kv must be contiguous, uint8 and of shape {list(pool)}")
    for name, t in (("k_exp", k_exp), ("v_exp", v_exp)):
        if t is not None:
            _ints(f"the {name} of kv", t, shape.Hkv)
    if seqs:
        if table is None or seq_ctx is None:
            raise ValueError("kv needs a block_table and seq_ctx for this call")
        _ints("the block_table of kv", table, shape.B, table.shape[-1])
        _ints("the seq_ctx of kv", seq_ctx, shape.B)
    _same_device(dev, kept)
    kv._fits = fits


def sv_write_kv4(shape: Shape, k, v, slot_map, kv: KV4, ws=None, stream=None):
    """Store the rows k, v [n, Hkv, d] (slices of a fused projection are fine) in 4
    bits at their slots; slots of -1 are skipped."""
    H, d, dtype = shape.Hkv, shape.d, _DTYPES[shape.dtype]
    n, kp, ks = _row_array("k", k, dtype, H, d)
    nv, vp, vs = _row_array("v", v, dtype, H, d)
    if nv != n:
        raise ValueError(f"{n} key rows and {nv} value rows")
    _check_kv4(shape, kv, False, k.get_device())
    _call(lib().sv_write_kv4, (k, v, slot_map, ws), stream, C.byref(shape), kp, ks, vp, vs,
          _ints("slot_map", slot_map, n), n, C.byref(kv), _workspace(ws)[0])


def sv_read_kv4(shape: Shape, kv: KV4, slot_map, k_out, v_out, ws=None, stream=None):
    """The rows k_out, v_out [n, Hkv, d] of the values at the slots of a 4-bit cache;
    rows of slots -1 stay as they are."""
    H, d, dtype = shape.Hkv, shape.d, _DTYPES[shape.dtype]
    n, kp, ks = _row_array("k_out", k_out, dtype, H, d)
    nv, vp, vs = _row_array("v_out", v_out, dtype, H, d)
    if nv != n:
        raise ValueError(f"{n} key rows and {nv} value rows")
    _check_kv4(shape, kv, False, k_out.get_device())
    _call(lib().sv_read_kv4, (k_out, v_out, slot_map, ws), stream, C.byref(shape), C.byref(kv),
          _ints("slot_map", slot_map, n), n, kp, ks, vp, vs, _workspace(ws)[0])


def sv_build_reps_kv4(shape: Shape, kv: KV4, max_blocks: int, reps, from_len=None, ws=None, stream=None):
    """Representatives of the blocks that sequences filled since they had from_len
    tokens (int32 [B], None: since the beginning), at most max_blocks each. reps:
    float32 [B, Hkv, nb_max, d]."""
    B = shape.B
    _check_kv4(shape, kv, True, reps.get_device())
    _call(lib().sv_build_reps_kv4, (reps, from_len, ws), stream,
          C.byref(shape), C.byref(kv), None if from_len is None else _ints("from_len", from_len, B),
          max_blocks, _dense("reps", reps, torch.float32, B, shape.Hkv, kv.nb_max, shape.d),
          _workspace(ws)[0])


def alloc_kv4_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    """A zeroed workspace for sv_attend_kv4 calls with this shape."""
    return _alloc_zeroed(lib().sv_kv4_workspace_bytes(C.byref(shape)), device)


def sv_attend_kv4(shape: Shape, q, kv: KV4, sel, draft_k, draft_v, parents, out, ws,
                  n_sel: Optional[int] = None, stream=None):
    """Verification attention over a 4-bit cache: every block when sel is None, else
    the first n_sel (all, when None) entries of the rows sel [B, Hkv, kmax]; -1
    entries hold nothing. T = 1 is a decoding step."""
    B, T, H, d, dtype = shape.B, shape.T, shape.Hkv, shape.d, _DTYPES[shape.dtype]
    rows, drafts = (B, T, shape.Hq, d), (B, T, H, d)
    if parents is not None and len(parents) != T:
        raise ValueError(f"{len(parents)} draft parents for T={T} drafts")
    stride = 0 if sel is None else sel.shape[-1]
    # an empty selection has no address, and none would mean every block: any other does, as no entry is read
    sel_ptr = None if sel is None else _ints("sel", sel, B, H, stride) or kv.block_table
    _check_kv4(shape, kv, True, q.get_device())
    _call(lib().sv_attend_kv4, (q, sel, draft_k, draft_v, out, ws), stream,
          C.byref(shape), _dense("q", q, dtype, *rows), C.byref(kv), sel_ptr,
          stride if n_sel is None else n_sel, stride, _dense("draft_k", draft_k, dtype, *drafts),
          _dense("draft_v", draft_v, dtype, *drafts), _parents(parents), _dense("out", out, dtype, *rows),
          *_workspace(ws))


VERIFY_COMPUTE, VERIFY_REUSE, VERIFY_FULL = 0, 1, 2  # sv_verify_layer's reuse values


class VerifySchedule:
    """Which sv_verify_layer mode a (step, layer) runs: every `full_period`-th
    step is a full verification over every block (the periodic full steps that
    partial verification interleaves; 0 = never); in the other steps layer l
    recomputes its selection when l % compute_every == 0 and reuses the last
    one otherwise."""

    def __init__(self, full_period: int = 0, compute_every: int = 1):
        if full_period < 0 or compute_every < 1:
            raise ValueError("full_period >= 0 and compute_every >= 1")
        self.full_period = full_period
        self.compute_every = compute_every

    def mode(self, step: int, layer: int = 0) -> int:
        if self.full_period and step % self.full_period == self.full_period - 1:
            return VERIFY_FULL
        return VERIFY_COMPUTE if layer % self.compute_every == 0 else VERIFY_REUSE
class LayerState:
    """Device-resident state of one verification layer: the paged KV cache,
    its block representatives, a selection cache slot and a workspace.

    Built from workloads.LayerInputs already on the device. Only allocation
    and marshalling happen here; the computation is the library's.
    """

    def __init__(self, wl: W.Workload, x: W.LayerInputs, kmax: Optional[int] = None,
                 build_reps: bool = True, stream=None, seq_ctx: Optional[Sequence[int]] = None):
        """seq_ctx: one prefix length per sequence (each at most wl.ctx, the
        length the block table is laid out for); wl.ctx for all when None."""
        self.wl, self.x = wl, x
        self.shape = make_shape(wl.B, wl.Hq, wl.Hkv, wl.d, wl.blk, wl.T, wl.torch_dtype)
        self.kv = make_kv(x.k_pool, x.v_pool, x.block_table, wl.ctx, seq_ctx)
        nb = wl.NB
        ctxs = [wl.ctx] if seq_ctx is None else list(seq_ctx)
        # the largest per-sequence budget: the selection rows' valid prefix
        self.k = max(sv_budget_blocks(wl.budget, c, c // wl.blk) for c in ctxs) if ctxs else 0
        self.kmax = self.k if kmax is None else kmax
        dev = x.q.device
        # [B, Hkv, nb_max, d]: the calls index representatives with the block
        # table's width as stride (a partial last block gets a row, unused)
        nb_max = max(x.block_table.shape[1], 1)
        self.reps = torch.zeros(wl.B, wl.Hkv, nb_max, wl.d, dtype=torch.float32, device=dev)
        self.slot = SelSlot(wl.B, wl.Hkv, self.kmax, device=dev)
        self.out = torch.empty_like(x.q)
        # sized for the budgeted selection and for a dense (all-block) pass
        # sized for the block table's width (nb_max), as the calls check it
        self.ws = alloc_workspace(self.shape, nb_max, max(self.kmax, nb, 1), device=dev)
        self.parents = None if wl.parents is None else list(wl.parents)
        if build_reps and nb:
            sv_build_reps(self.shape, self.kv, 0, nb, self.reps, stream)

    @property
    def sel(self) -> torch.Tensor:
        """The layer's selection (its slot's device tensor)."""
        return self.slot.tensor

    def verify(self, reuse: int = 0, sel_from: Optional["LayerState"] = None, stream=None):
        """One sv_verify_layer call; sel_from shares that layer's selection
        slot (inter-layer reuse)."""
        if sel_from is not None:
            self.slot = sel_from.slot
        sv_verify_layer(self.shape, self.x.q, self.kv, self.reps, self.wl.budget, self.x.draft_k,
                        self.x.draft_v, self.parents, reuse, self.slot, self.out, self.ws, stream)
        return self.out
