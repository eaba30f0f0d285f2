"""Paged-attention decode on GB300: Python binding of libpa103.so (include/pa.h).

This module only marshals arguments: every step of the decode (planning, page gather,
attention, split merge) runs in the library's CUDA kernels.  PyTorch tensors supply the
device memory and the current stream.  If the library has not been built the first call
raises; there is no fallback.

Build the library with ``python -m paged_kv_cache_work_gb300.build`` (or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = ["PaConfig", "PaError", "load", "workspace_size", "plan", "decode", "reduce",
           "decode_step_static", "STATIC_SCRATCH_BYTES", "append_kv", "gather_kv",
           "build_tables", "update_bounds", "score_blocks", "select_blocks",
           "decode_selected", "append_rotated", "dequant_kv", "PaRotary",
           "read_flags", "status_string", "config_for", "paged_attention", "LIB_PATH",
           "BF16", "FP16", "FP8_E4M3", "INT4", "SCALE_NONE", "SCALE_PER_TENSOR", "SCALE_PER_TOKEN",
           "SCALE_PER_BLOCK", "SCALE_AFFINE",
           "FLAG_BAD_LENGTHS", "FLAG_BAD_BLOCK_ID", "FLAG_WAIT_TIMEOUT", "FLAG_STALE_PLAN",
           "FLAG_BAD_SELECTION", "FLAG_NO_FREE_BLOCKS", "FLAG_BAD_FREE_LIST", "FLAG_BAD_POSITION",
           "EXPORTED_SYMBOLS",
           "MERGE_AUTO", "MERGE_IN_DECODE", "MERGE_IN_REDUCE"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa103.so")

# pa_status
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE = range(6)
# pa_dtype, pa_scale_mode, flags
BF16, FP16, FP8_E4M3, INT4 = 0, 1, 2, 3
SCALE_NONE, SCALE_PER_TENSOR, SCALE_PER_TOKEN, SCALE_PER_BLOCK, SCALE_AFFINE = 0, 1, 2, 3, 4
FLAG_BAD_LENGTHS, FLAG_BAD_BLOCK_ID, FLAG_WAIT_TIMEOUT, FLAG_STALE_PLAN = 1, 2, 4, 8
FLAG_BAD_SELECTION, FLAG_NO_FREE_BLOCKS, FLAG_BAD_FREE_LIST = 16, 32, 64
FLAG_BAD_POSITION = 128
MERGE_AUTO, MERGE_IN_DECODE, MERGE_IN_REDUCE = 0, 1, 2

EXPORTED_SYMBOLS = ("pa_workspace_size", "pa_plan", "pa_decode", "pa_reduce", "pa_read_flags",
                    "pa_status_string", "pa_decode_step_static", "pa_gather_kv", "pa_append_kv",
                    "pa_build_tables", "pa_update_bounds", "pa_score_blocks", "pa_select_blocks",
                    "pa_decode_selected", "pa_append_rotated", "pa_dequant_kv")

# Bytes of the device array behind pa_decode_step_static (PA_STATIC_SCRATCH_BYTES).
STATIC_SCRATCH_BYTES = 16 << 20


class PaConfig(ctypes.Structure):
    """Mirror of pa_config."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "max_q_len", "num_q_heads", "num_kv_heads", "head_dim", "block_size",
        "max_blocks_per_seq", "num_blocks", "q_dtype", "kv_dtype", "kv_scale_mode", "causal")] + [
        ("sm_scale", ctypes.c_float), ("num_ctas", ctypes.c_int32), ("grid_mult", ctypes.c_int32),
        ("split_merge", ctypes.c_int32)]


class PaRotary(ctypes.Structure):
    """Mirror of pa_rotary."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("cos_sin", ctypes.c_void_p), ("table_rows", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("num_axes", ctypes.c_int32),
                ("axis_pairs", ctypes.c_int32 * 3), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class PaError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (once).  Raises if it is missing: there is no CPU fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run python -m paged_kv_cache_work_gb300.build")
    L = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    cfgp = ctypes.POINTER(PaConfig)
    L.pa_workspace_size.argtypes = [cfgp, ctypes.POINTER(sz)]
    L.pa_plan.argtypes = [cfgp, vp, vp, vp, vp, sz, vp]
    L.pa_decode.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.pa_reduce.argtypes = [cfgp, vp, vp, vp, sz, vp]
    L.pa_read_flags.argtypes = [vp, sz, ctypes.POINTER(ctypes.c_int32), vp]
    for f in ("pa_workspace_size", "pa_plan", "pa_decode", "pa_reduce", "pa_read_flags"):
        getattr(L, f).restype = ctypes.c_int
    L.pa_decode_step_static.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.pa_decode_step_static.restype = ctypes.c_int
    L.pa_gather_kv.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp, vp, vp]
    L.pa_gather_kv.restype = ctypes.c_int
    L.pa_append_kv.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.pa_append_kv.restype = ctypes.c_int
    L.pa_build_tables.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.pa_build_tables.restype = ctypes.c_int
    i32 = ctypes.c_int32
    L.pa_update_bounds.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp]
    L.pa_update_bounds.restype = ctypes.c_int
    L.pa_score_blocks.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.pa_score_blocks.restype = ctypes.c_int
    L.pa_select_blocks.argtypes = [cfgp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    L.pa_select_blocks.restype = ctypes.c_int
    L.pa_decode_selected.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp,
                                     vp, vp]
    L.pa_decode_selected.restype = ctypes.c_int
    L.pa_append_rotated.argtypes = [cfgp, ctypes.POINTER(PaRotary)] + [vp] * 14
    L.pa_append_rotated.restype = ctypes.c_int
    L.pa_dequant_kv.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp, vp, vp]
    L.pa_dequant_kv.restype = ctypes.c_int
    L.pa_status_string.argtypes = [ctypes.c_int]
    L.pa_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _current_stream() -> int:
    """Handle of torch's current stream on the current device."""
    global _current_stream
    import torch
    stream = torch.cuda.current_stream().cuda_stream  # (initialises CUDA)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None:  # the same handle, without a Stream object: 0.2 us
        _current_stream = lambda: raw(device())  # noqa: E731  instead of 3 us on the host
    return stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(call: str, status: int):
    if status != OK:
        raise PaError(call, status)


def workspace_size(cfg: PaConfig) -> int:
    n = ctypes.c_size_t(0)
    _check("pa_workspace_size", load().pa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


_type_cache = None


def _types():
    """(current device, then the torch types of int32, int64 and fp32 arrays and, by pa_dtype,
    those of q and of a cache)."""
    global _type_cache
    if _type_cache is None:
        import torch
        cache = {BF16: (torch.bfloat16,), FP16: (torch.float16,),
                 FP8_E4M3: (torch.uint8, torch.float8_e4m3fn), INT4: (torch.uint8,)}
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _type_cache = device, (torch.int32,), (torch.int64,), (torch.float32,), cache
    device, i32, i64, f32, cache = _type_cache
    try:
        return device(), i32, i64, f32, cache
    except RuntimeError:  # no GPU: no tensor is on the current one
        return None, i32, i64, f32, cache


def _dense(call: str, device: int, count: int, t, dtypes) -> int:
    """Address of a contiguous tensor of at least `count` elements of one of `dtypes` on the
    current GPU (an int address passes as it is); PaError otherwise."""
    try:
        if t.dtype in dtypes and t.numel() >= count and t.is_contiguous() \
                and t.get_device() == device:
            return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return t
    raise PaError(call, ERR_INVALID_ARG)


def _columns(call: str, t) -> int:
    """The last dimension of a tensor that has one; PaError otherwise."""
    shape = getattr(t, "shape", None)
    if not shape:
        raise PaError(call, ERR_INVALID_ARG)
    return shape[-1]


def _maybe(call: str, device: int, count: int, t, dtypes) -> Optional[int]:
    return None if t is None else _dense(call, device, count, t, dtypes)


def _scale(call: str, device: int, cfg: PaConfig, t, f32) -> Optional[int]:
    """Address of one of a cache's scale arrays, as large as cfg's scale mode has it (a mode that
    the library refuses: whatever is given)."""
    mode = cfg.kv_scale_mode
    if mode == SCALE_NONE:
        return None
    if not 0 < mode <= SCALE_AFFINE:
        return _ptr(t)
    heads = cfg.num_blocks * cfg.num_kv_heads
    if mode == SCALE_AFFINE:  # pairs (step, low) in the queries' type
        return _dense(call, device, 2 * heads * cfg.block_size, t, _types()[4].get(cfg.q_dtype, ()))
    return _dense(call, device, (0, 1, heads * cfg.block_size, heads)[mode], t, f32)


def _cache_elements(cfg: PaConfig) -> int:
    """Elements (bytes, for a 4-bit cache) of a K or V cache."""
    n = cfg.num_blocks * cfg.block_size * cfg.num_kv_heads * cfg.head_dim
    return n // 2 if cfg.kv_dtype == INT4 else n


def plan(cfg: PaConfig, block_tables, context_lens, q_lens, ws, stream=None):
    _check("pa_plan", load().pa_plan(ctypes.byref(cfg), _ptr(block_tables), _ptr(context_lens),
                                     _ptr(q_lens), _ptr(ws), _nbytes(ws), _stream(stream)))


def decode(cfg: PaConfig, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
           q_lens, out, lse, ws, stream=None):
    dev, _, _, f32, _ = _types()
    name = "pa_decode"
    _check(name, load().pa_decode(
        ctypes.byref(cfg), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _scale(name, dev, cfg, k_scale, f32), _scale(name, dev, cfg, v_scale, f32),
        _ptr(block_tables), _ptr(context_lens), _ptr(q_lens), _ptr(out), _ptr(lse), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def reduce(cfg: PaConfig, out, lse, ws, stream=None):
    _check("pa_reduce", load().pa_reduce(ctypes.byref(cfg), _ptr(out), _ptr(lse), _ptr(ws),
                                         _nbytes(ws), _stream(stream)))


def read_flags(ws, stream=None) -> int:
    """Synchronise and return the device flags of the last step run in ``ws``."""
    f = ctypes.c_int32(0)
    st = load().pa_read_flags(_ptr(ws), _nbytes(ws), ctypes.byref(f), _stream(stream))
    if st not in (OK, ERR_DEVICE):
        raise PaError("pa_read_flags", st)
    return f.value


def decode_step_static(cfg: PaConfig, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                       context_lens, q_lens, out, lse, stream=None):
    """One decode step on the library's static device scratch, for callers that cannot
    allocate device memory (no workspace argument; see pa_decode_step_static in pa.h)."""
    dev, _, _, f32, _ = _types()
    name = "pa_decode_step_static"
    _check(name, load().pa_decode_step_static(
        ctypes.byref(cfg), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _scale(name, dev, cfg, k_scale, f32), _scale(name, dev, cfg, v_scale, f32),
        _ptr(block_tables), _ptr(context_lens), _ptr(q_lens), _ptr(out), _ptr(lse),
        _stream(stream)))


def gather_kv(cfg: PaConfig, k_cache, v_cache, block_tables, context_lens, k_out, v_out,
              max_rows: int, row_offsets=None, flags=None, stream=None):
    """Paged -> contiguous copy of the batch's K and V rows (see pa_gather_kv in pa.h):
    sequence b lands at rows row_offsets[b] .. row_offsets[b + 1] - 1 of k_out and v_out."""
    _check("pa_gather_kv", load().pa_gather_kv(
        ctypes.byref(cfg), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        _ptr(k_out), _ptr(v_out), int(max_rows), _ptr(row_offsets), _ptr(flags),
        _stream(stream)))


def append_kv(cfg: PaConfig, k_new, v_new, block_tables, context_lens, q_lens, k_cache, v_cache,
              k_scale=None, v_scale=None, flags=None, stream=None):
    """Write a step's new K/V rows into their pages, quantised for an fp8 or 4-bit cache (see
    pa_append_kv in pa.h): new row i of sequence b lands at position
    context_lens[b] - q_lens[b] + i.  Per-token scales, and a 4-bit cache's pairs (step, low)
    [num_blocks, Hkv, block_size, 2], are written into k_scale / v_scale; a page's one scale
    (SCALE_PER_BLOCK) is raised where a new row needs it, and the page's older codes follow."""
    dev, i32, _, f32, kinds = _types()
    name, B, row = "pa_append_kv", cfg.batch, cfg.num_kv_heads * cfg.head_dim
    kind, cache_kind = kinds.get(cfg.q_dtype, ()), kinds.get(cfg.kv_dtype, ())
    cache = _cache_elements(cfg)
    _check(name, load().pa_append_kv(
        ctypes.byref(cfg), _dense(name, dev, B * cfg.max_q_len * row, k_new, kind),
        _dense(name, dev, B * cfg.max_q_len * row, v_new, kind),
        _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32),
        _dense(name, dev, B, context_lens, i32), _dense(name, dev, B, q_lens, i32),
        _dense(name, dev, cache, k_cache, cache_kind), _dense(name, dev, cache, v_cache, cache_kind),
        _scale(name, dev, cfg, k_scale, f32), _scale(name, dev, cfg, v_scale, f32),
        _maybe(name, dev, 1, flags, i32), _stream(stream)))


def build_tables(cfg: PaConfig, context_lens, q_lens, held_blocks, block_tables, free_blocks,
                 free_count, new_held, new_free_count, slot_map=None, flags=None, stream=None):
    """Grow and shrink the rows of block_tables to the pages that context_lens need, out of and
    back into the free stack free_blocks[:free_count], and write the new tokens' slots (see
    pa_build_tables in pa.h).  The held and free counts after the call go to new_held and
    new_free_count, which are the next call's held_blocks and free_count."""
    dev, i32, i64, _, _ = _types()
    name, B = "pa_build_tables", cfg.batch
    _check(name, load().pa_build_tables(
        ctypes.byref(cfg), _dense(name, dev, B, context_lens, i32),
        _dense(name, dev, B, q_lens, i32), _dense(name, dev, B, held_blocks, i32),
        _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32),
        _dense(name, dev, cfg.num_blocks, free_blocks, i32), _dense(name, dev, 1, free_count, i32),
        _dense(name, dev, B, new_held, i32), _dense(name, dev, 1, new_free_count, i32),
        _maybe(name, dev, B * cfg.max_q_len, slot_map, i64),
        _maybe(name, dev, 1, flags, i32), _stream(stream)))


def update_bounds(cfg: PaConfig, k_new, block_tables, context_lens, q_lens, k_bounds, flags=None,
                  stream=None):
    """Widen the channel bounds k_bounds [num_blocks, Hkv, 2, D] of the pages that a step's new K
    rows go to (see pa_update_bounds in pa.h); a page whose first slot is new starts afresh."""
    dev, i32, _, _, kinds = _types()
    name, B, row = "pa_update_bounds", cfg.batch, cfg.num_kv_heads * cfg.head_dim
    kind = kinds.get(cfg.q_dtype, ())
    _check(name, load().pa_update_bounds(
        ctypes.byref(cfg), _dense(name, dev, B * cfg.max_q_len * row, k_new, kind),
        _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32),
        _dense(name, dev, B, context_lens, i32), _dense(name, dev, B, q_lens, i32),
        _dense(name, dev, cfg.num_blocks * row * 2, k_bounds, kind),
        _maybe(name, dev, 1, flags, i32), _stream(stream)))


def score_blocks(cfg: PaConfig, q, k_bounds, block_tables, context_lens, q_lens, scores,
                 flags=None, stream=None):
    """Upper bounds of the logits of every page for each new-token row and kv head, into scores
    [B, Sq, Hkv, max_blocks_per_seq]; -inf for pages the row does not see (see pa_score_blocks in
    pa.h)."""
    dev, i32, _, f32, kinds = _types()
    name, B, rows = "pa_score_blocks", cfg.batch, cfg.batch * cfg.max_q_len
    kind = kinds.get(cfg.q_dtype, ())
    _check(name, load().pa_score_blocks(
        ctypes.byref(cfg), _dense(name, dev, rows * cfg.num_q_heads * cfg.head_dim, q, kind),
        _dense(name, dev, cfg.num_blocks * cfg.num_kv_heads * 2 * cfg.head_dim, k_bounds, kind),
        _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32),
        _dense(name, dev, B, context_lens, i32), _dense(name, dev, B, q_lens, i32),
        _dense(name, dev, rows * cfg.num_kv_heads * cfg.max_blocks_per_seq, scores, f32),
        _maybe(name, dev, 1, flags, i32), _stream(stream)))


def select_blocks(cfg: PaConfig, scores, context_lens, q_lens, num_first: int, num_last: int,
                  selected, num_selected, flags=None, stream=None):
    """The best selected.shape[-1] pages of each row, ascending, the first num_first and the last
    num_last always among them (see pa_select_blocks in pa.h)."""
    dev, i32, _, f32, _ = _types()
    name, B = "pa_select_blocks", cfg.batch
    rows, top_k = B * cfg.max_q_len * cfg.num_kv_heads, _columns(name, selected)
    _check(name, load().pa_select_blocks(
        ctypes.byref(cfg), _dense(name, dev, rows * cfg.max_blocks_per_seq, scores, f32),
        _dense(name, dev, B, context_lens, i32), _dense(name, dev, B, q_lens, i32), top_k,
        int(num_first), int(num_last), _dense(name, dev, rows * top_k, selected, i32),
        _dense(name, dev, rows, num_selected, i32), _maybe(name, dev, 1, flags, i32),
        _stream(stream)))


def decode_selected(cfg: PaConfig, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                    context_lens, q_lens, selected, num_selected, out, lse=None, flags=None,
                    stream=None):
    """Attention of each row over its listed pages selected [B, Sq, Hkv, top_k], of which the
    first num_selected count (see pa_decode_selected in pa.h).  One launch, no workspace."""
    dev, i32, _, f32, kinds = _types()
    name, B, Hkv = "pa_decode_selected", cfg.batch, cfg.num_kv_heads
    rows, top_k = B * cfg.max_q_len, _columns(name, selected)
    kind, cache_kind = kinds.get(cfg.q_dtype, ()), kinds.get(cfg.kv_dtype, ())
    cache = cfg.num_blocks * cfg.block_size * Hkv * cfg.head_dim
    _check(name, load().pa_decode_selected(
        ctypes.byref(cfg), _dense(name, dev, rows * cfg.num_q_heads * cfg.head_dim, q, kind),
        _dense(name, dev, cache, k_cache, cache_kind),
        _dense(name, dev, cache, v_cache, cache_kind),
        _scale(name, dev, cfg, k_scale, f32), _scale(name, dev, cfg, v_scale, f32),
        _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32),
        _dense(name, dev, B, context_lens, i32), _dense(name, dev, B, q_lens, i32),
        _dense(name, dev, rows * Hkv * top_k, selected, i32),
        _dense(name, dev, rows * Hkv, num_selected, i32), top_k,
        _dense(name, dev, rows * cfg.num_q_heads * cfg.head_dim, out, kind),
        _maybe(name, dev, rows * cfg.num_q_heads, lse, f32),
        _maybe(name, dev, 1, flags, i32), _stream(stream)))


def _rows(call: str, device: int, tokens: int, heads: int, dim: int, t, dtypes):
    """(address, elements between tokens) of rows [B, Sq, heads, dim] that lie dense within a token
    (an address passes as it is, with 0: dense)."""
    try:
        shape, stride = t.shape, t.stride()
        if t.dtype in dtypes and t.get_device() == device and len(shape) == 4 and stride[3] == 1 \
                and shape[3] == dim and shape[2] == heads and (stride[2] == dim or heads == 1):
            b, sq = shape[0], shape[1]
            step = stride[1] if sq > 1 else stride[0] if b > 1 else 0
            # (tokens that share one row, as an expanded tensor's: 0 would say dense)
            if b * sq >= tokens and (step or b * sq == 1) and (b == 1 or sq == 1 or stride[0] == sq * step):
                return t.data_ptr(), step
    except AttributeError:
        if isinstance(t, int):
            return t, 0
    raise PaError(call, ERR_INVALID_ARG)


def append_rotated(cfg: PaConfig, q, k_new, v_new, block_tables, context_lens, q_lens, q_out,
                   k_cache, v_cache, k_scale=None, v_scale=None, *, cos_sin=None,
                   interleaved: bool = False, positions=None, axis_pairs=None, q_weight=None,
                   k_weight=None, eps: float = 1e-6, k_out=None, flags=None, stream=None):
    """Normalise (q_weight, k_weight) and rotate (cos_sin [positions, rotary_dim] fp32: cosines, then
    sines) a step's queries and keys, into q_out and k_out, and write its K/V rows into their pages,
    in one pass (see pa_append_rotated in pa.h).  q, k_new and v_new may be slices of one projection's
    output.  positions [axes, B, Sq] default to the cache positions; axis_pairs: how many of the
    rotated pairs follow each axis (either without cos_sin is refused).  With k_cache and v_cache None nothing goes into pages."""
    dev, i32, _, f32, kinds = _types()
    name, B, D = "pa_append_rotated", cfg.batch, cfg.head_dim
    kind, hq, hkv = kinds.get(cfg.q_dtype, ()), cfg.num_q_heads, cfg.num_kv_heads
    tokens = B * cfg.max_q_len
    table, rows, turned, where, axes, pairs = None, 0, 0, None, 0, (0, 0, 0)
    if cos_sin is not None:
        shape = getattr(cos_sin, "shape", ())
        if len(shape) != 2:
            raise PaError(name, ERR_INVALID_ARG)
        rows, turned = shape
        table = _dense(name, dev, rows * turned, cos_sin, f32)
        pairs = (turned // 2,) if axis_pairs is None else tuple(axis_pairs)
        axes = len(pairs)
        if not 1 <= axes <= 3:
            raise PaError(name, ERR_INVALID_ARG)
        pairs += (0,) * (3 - axes)
        if positions is not None:
            where = _dense(name, dev, axes * tokens, positions, i32)
    elif positions is not None or axis_pairs is not None:  # (of angles that were not given)
        raise PaError(name, ERR_INVALID_ARG)
    qp, qs = _rows(name, dev, tokens, hq, D, q, kind)
    kp, ks = _rows(name, dev, tokens, hkv, D, k_new, kind)
    vp = vs = blocks = kc = vc = k_sc = v_sc = None
    if k_cache is not None or v_cache is not None:
        cache_kind, cache = kinds.get(cfg.kv_dtype, ()), _cache_elements(cfg)
        vp, vs = _rows(name, dev, tokens, hkv, D, v_new, kind)
        blocks = _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32)
        kc, vc = _dense(name, dev, cache, k_cache, cache_kind), _dense(name, dev, cache, v_cache, cache_kind)
        if cfg.kv_scale_mode != SCALE_NONE:
            k_sc, v_sc = _scale(name, dev, cfg, k_scale, f32), _scale(name, dev, cfg, v_scale, f32)
    rotary = PaRotary(
        None if q_weight is None else _dense(name, dev, D, q_weight, kind),
        None if k_weight is None else _dense(name, dev, D, k_weight, kind), eps, turned,
        1 if interleaved else 0, table, rows, where, axes, pairs, qs, ks, vs or 0)
    _check(name, load().pa_append_rotated(
        ctypes.byref(cfg), ctypes.byref(rotary), qp, kp, vp, blocks, _dense(name, dev, B, context_lens, i32),
        _dense(name, dev, B, q_lens, i32), _dense(name, dev, tokens * hq * D, q_out, kind),
        None if k_out is None else _dense(name, dev, tokens * hkv * D, k_out, kind), kc, vc, k_sc, v_sc,
        None if flags is None else _dense(name, dev, 1, flags, i32), _stream(stream)))


def dequant_kv(cfg: PaConfig, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, k_out,
               v_out, max_rows: Optional[int] = None, row_offsets=None, flags=None, stream=None):
    """The batch's rows of an fp8 or 4-bit cache as values of q_dtype in contiguous buffers (see
    pa_dequant_kv in pa.h): sequence b lands at rows row_offsets[b] .. row_offsets[b + 1] - 1 of k_out
    and v_out, which have room for max_rows rows (by default what both hold)."""
    dev, i32, _, f32, kinds = _types()
    name, B, row = "pa_dequant_kv", cfg.batch, cfg.num_kv_heads * cfg.head_dim
    kind, cache_kind, cache = kinds.get(cfg.q_dtype, ()), kinds.get(cfg.kv_dtype, ()), _cache_elements(cfg)
    if max_rows is None:
        try:
            max_rows = min(k_out.numel(), v_out.numel()) // max(1, row)
        except AttributeError:
            raise PaError(name, ERR_INVALID_ARG) from None
    _check(name, load().pa_dequant_kv(
        ctypes.byref(cfg), _dense(name, dev, cache, k_cache, cache_kind),
        _dense(name, dev, cache, v_cache, cache_kind), _scale(name, dev, cfg, k_scale, f32),
        _scale(name, dev, cfg, v_scale, f32),
        _dense(name, dev, B * cfg.max_blocks_per_seq, block_tables, i32),
        _dense(name, dev, B, context_lens, i32), _dense(name, dev, max_rows * row, k_out, kind),
        _dense(name, dev, max_rows * row, v_out, kind), int(max_rows),
        _maybe(name, dev, B + 1, row_offsets, i32), _maybe(name, dev, 1, flags, i32), _stream(stream)))


_DT = {"bf16": BF16, "fp16": FP16, "fp8": FP8_E4M3, "int4": INT4}
_SM = {"none": SCALE_NONE, "tensor": SCALE_PER_TENSOR, "token": SCALE_PER_TOKEN,
       "block": SCALE_PER_BLOCK}


def config_for(inp: dict, num_ctas: int = 0, grid_mult: int = 0,
               split_merge: int = MERGE_AUTO) -> PaConfig:
    """pa_config of a problem laid out as workloads.make_inputs returns it.  With neither a
    grid size nor a multiplier given and the inputs on a GPU, the multiplier comes from the
    tuned table (grid_tune.lookup: 1 for shapes it does not list)."""
    w = inp["workload"]
    cfg = PaConfig(batch=w.batch, max_q_len=w.max_q_len, num_q_heads=w.num_q_heads,
                   num_kv_heads=w.num_kv_heads, head_dim=w.head_dim, block_size=w.block_size,
                   max_blocks_per_seq=inp["block_tables"].shape[1],
                   num_blocks=inp["k_cache"].shape[0], q_dtype=_DT[w.q_dtype],
                   kv_dtype=_DT[w.kv_dtype],
                   kv_scale_mode=_SM[w.scale_mode] if w.kv_dtype == "fp8" else
                   SCALE_AFFINE if w.kv_dtype == "int4" else SCALE_NONE,
                   causal=int(w.causal), sm_scale=float(inp["sm_scale"]), num_ctas=num_ctas,
                   grid_mult=grid_mult, split_merge=split_merge)
    q = inp["q"]
    if num_ctas == 0 and grid_mult == 0 and getattr(q, "is_cuda", False):
        import torch
        from . import grid_tune
        sms = torch.cuda.get_device_properties(q.device).multi_processor_count
        cfg.grid_mult = grid_tune.lookup(cfg, sms)
    return cfg


def paged_attention(inp: dict, out=None, lse=None, ws=None, cfg: Optional[PaConfig] = None,
                    stream=None):
    """One decode step (plan, decode, reduce) on tensors already on the GPU.

    Allocates out [B, Sq, Hq, D], lse [B, Sq, Hq] and the workspace with torch when they are
    not given.  Returns (out, lse, ws)."""
    import torch
    cfg = cfg if cfg is not None else config_for(inp)
    q = inp["q"]
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(workspace_size(cfg), dtype=torch.uint8, device=dev)
    plan(cfg, inp["block_tables"], inp["context_lens"], inp["q_lens"], ws, stream)
    decode(cfg, q, inp["k_cache"], inp["v_cache"], inp.get("k_scale"), inp.get("v_scale"),
           inp["block_tables"], inp["context_lens"], inp["q_lens"], out, lse, ws, stream)
    reduce(cfg, out, lse, ws, stream)
    return out, lse, ws
