"""Python binding of libuniprefill.so: UniPrefill's per-layer token-dropping hot path on GB300.

Each ``up_*`` function has the name and meaning of the C entry point declared in
include/uniprefill.h and does argument marshalling only (torch tensors -> device
pointers, sizes, the current CUDA stream); every step of the computation runs in
the library's CUDA kernels.  There is no CPU fallback: if the shared library is
missing or cannot be loaded, importing the binding's functions raises.

Paper: "UniPrefill: Universal Long-Context Prefill Acceleration via Block-wise
Dynamic Sparsification" (arXiv 2605.06221), sections 3.2-3.5.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libuniprefill.so")

UP_OK, UP_ERR_ARG, UP_ERR_SHAPE, UP_ERR_WORKSPACE, UP_ERR_CUDA, UP_ERR_DEVICE = range(6)
MAX_BLOCKS_PER_REQUEST = 8192
NOALLOC_MAX_TOKENS = 16384 * 1024

_c_p = ctypes.c_void_p
_i32, _i64, _f32, _f64, _sz, _u64 = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_size_t, ctypes.c_uint64

_SIGNATURES = {
    "up_max_blocks": (_i64, [_i32, _i64, _i32]),
    "up_score_workspace_bytes": (_sz, [_i32, _i64, _i32, _i32, _i32, _i32, _i32, _i64, _i32]),
    "up_compact_workspace_bytes": (_sz, [_i32, _i64]),
    "up_select_workspace_bytes": (_sz, [_i64]),
    "up_workspace_bytes": (_sz, [_i32, _i64, _i32, _i32, _i32, _i32, _i32, _i64]),
    "up_make_cu_blocks": (_i32, [_c_p, _i32, _i64, _i32, _c_p, _c_p, _c_p]),
    "up_score_blocks": (_i32, [_c_p, _c_p, _c_p, _i32, _i64, _i32, _i32, _i32, _i32, _i32, _f32,
                                _c_p, _i64, _c_p, _c_p, _c_p, _sz, _c_p, _c_p]),
    "up_select_topp": (_i32, [_c_p, _c_p, _c_p, _i32, _i64, _i64, _i32, _i32, _i32, _f64,
                               _c_p, _c_p, _c_p, _c_p, _sz, _c_p, _c_p]),
    "up_compact": (_i32, [_c_p, _c_p, _i32, _i64, _c_p, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                           _c_p, _c_p, _c_p, _c_p, _c_p, _i32, _i32, _c_p, _sz, _c_p, _c_p]),
    "up_compact_noalloc": (_i32, [_c_p, _c_p, _i32, _i64, _c_p, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                   _c_p, _c_p, _c_p, _c_p, _c_p, _i32, _i32, _c_p, _c_p]),
    "up_scatter_back": (_i32, [_c_p, _c_p, _c_p, _i64, _i32, _c_p, _c_p, _c_p]),
    "up_slot_mapping": (_i32, [_c_p, _c_p, _i32, _i64, _c_p, _c_p, _i32, _i32, _c_p, _c_p, _c_p]),
    "up_seqused": (_i32, [_c_p, _c_p, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p]),
    "up_read_status": (_i32, [_c_p, _c_p, _c_p]),
    "up_status_string": (ctypes.c_char_p, [_i32, _i32]),
    "up_kernel_launches": (_u64, []),
    "up_abi_version": (_i32, []),
    "up_debug_bounds": (_i32, []),
}

_SIGNATURES.update({
    "up_kv_scale_row": (_i32, [_i32]),
    "up_kv_write": (_i32, [_c_p, _c_p, _i64, _c_p, _i64, _c_p, _i64, _c_p, _c_p, _c_p]),
    "up_kv_read": (_i32, [_c_p, _c_p, _i64, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "up_paged_decode_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "up_paged_decode": (_i32, [_c_p, _i64, _c_p, _c_p, _c_p, _i32, _i32, _i32, _f32, _i32, _c_p, _c_p,
                               _c_p, _sz, _c_p, _c_p]),
})

_SIGNATURES.update({
    "up_rope_plan": (_i32, [_i32, _f64, _i32, _i32, _f64, _f64, _f64, _f64, _f64, _c_p]),
    "up_rope": (_i32, [_c_p, _c_p, _i64, _c_p, _i64, _i32, _c_p, _i64, _c_p, _i64, _i32, _i32, _c_p, _i64, _c_p, _i32,
                       _c_p, _c_p]),
    "up_kv_mass": (_i32, [_c_p, _i64, _c_p, _c_p, _c_p, _c_p, _i32, _i32, _i32, _f32, _c_p, _c_p, _f32, _c_p, _c_p, _c_p,
                          _c_p, _c_p]),
    "up_kv_evict": (_i32, [_c_p, _c_p, _i64, _i32, _i32, _c_p, _c_p, _c_p, _i32, _i32, _c_p, _i32, _i32, _c_p, _i64, _c_p,
                           _c_p, _c_p, _c_p]),
    "up_kv_move": (_i32, [_c_p, _c_p, _i32, _i32, _c_p, _i64, _c_p, _c_p, _c_p, _c_p, _c_p]),
})

KV_BF16, KV_E4M3 = 0, 1
ROPE_LAYOUTS = {"halves": 0, "pairs": 1}
# the scalings of rotary frequencies, with the turns over the trained length between which they blend
ROPE_SCALINGS = {"none": (0, 1.0, 2.0), "linear": (1, 1.0, 2.0), "bands": (2, 1.0, 4.0), "ramp": (3, 1.0, 32.0)}


class _KvCache(ctypes.Structure):
    """up_kv_cache"""
    _fields_ = [("k", _c_p), ("v", _c_p), ("k_scale", _c_p), ("v_scale", _c_p), ("num_blocks", _i64),
                ("stride_block", _i64), ("stride_head", _i64), ("stride_token", _i64),
                ("Hkv", ctypes.c_int32), ("B", ctypes.c_int32), ("dk", ctypes.c_int32), ("format", ctypes.c_int32)]


class RopeTable(ctypes.Structure):
    """up_rope_table: how the heads of a model turn (up_rope_plan)"""
    _fields_ = [("turns", _u64 * 128), ("gain", _f32), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32)]


_BF16, _E4M3, _U8, _I32, _I64 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32, torch.int64

_lib = None


def load_library(path=LIB_PATH):
    """Load libuniprefill.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libuniprefill.so not found at {path}; build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class UpError(RuntimeError):
    def __init__(self, code, where):
        msg = load_library().up_status_string(code, 0).decode()
        super().__init__(f"{where}: {msg}")
        self.code = code


def _check(code, where):
    if code != UP_OK:
        raise UpError(code, where)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:         # the current stream's handle without a Stream object (3 us of a small call)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _bf16(t):
    assert t.dtype == torch.bfloat16 and t.is_contiguous() and t.is_cuda
    return _p(t)


# ------------------------------------------------------------------------------------------ sizing

def up_max_blocks(R, T, G):
    return load_library().up_max_blocks(R, T, G)


def up_score_workspace_bytes(R, T, Hq, Hkv, dk, G, n, nb_cap, with_token_scores=False):
    return load_library().up_score_workspace_bytes(R, T, Hq, Hkv, dk, G, n, nb_cap, int(bool(with_token_scores)))


def up_compact_workspace_bytes(R, T):
    return load_library().up_compact_workspace_bytes(R, T)


def up_select_workspace_bytes(nb_cap):
    return load_library().up_select_workspace_bytes(nb_cap)


def up_workspace_bytes(R, T, Hq, Hkv, dk, G, n, nb_cap):
    return load_library().up_workspace_bytes(R, T, Hq, Hkv, dk, G, n, nb_cap)


# ------------------------------------------------------------------------------------------ the drop step

def up_make_cu_blocks(cu_seqlens, G, cu_blocks, dev_status, T=None, stream=None):
    R = cu_seqlens.numel() - 1
    T = int(T) if T is not None else None
    if T is None:
        raise ValueError("T (total tokens) is required: the binding never reads device memory back")
    _check(load_library().up_make_cu_blocks(_p(cu_seqlens), R, T, G, _p(cu_blocks), _p(dev_status), _stream(stream)),
           "up_make_cu_blocks")


def up_score_blocks(Q, K, cu_seqlens, G, n, cu_blocks, block_scores, ws, dev_status, token_scores=None,
                    sm_scale=None, stream=None):
    T, Hq, dk = Q.shape
    Hkv = K.shape[1]
    R = cu_seqlens.numel() - 1
    sm_scale = dk ** -0.5 if sm_scale is None else sm_scale
    _check(load_library().up_score_blocks(_bf16(Q), _bf16(K), _p(cu_seqlens), R, T, Hq, Hkv, dk, G, n, sm_scale,
                                          _p(cu_blocks), block_scores.numel(), _p(block_scores), _p(token_scores),
                                          _p(ws), ws.numel() * ws.element_size(), _p(dev_status), _stream(stream)),
           "up_score_blocks")


def up_select_topp(block_scores, cu_blocks, cu_seqlens, T, G, n, A, p, block_keep, token_keep, kstar, dev_status,
                   ws=None, stream=None):
    """ws: optional device workspace (up_select_workspace_bytes(block_scores.numel()) bytes); needed only
    for requests of more than MAX_BLOCKS_PER_REQUEST blocks."""
    R = cu_seqlens.numel() - 1
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().up_select_topp(_p(block_scores), _p(cu_blocks), _p(cu_seqlens), R, T, block_scores.numel(),
                                         G, n, A, float(p), _p(block_keep), _p(token_keep), _p(kstar), _p(ws), nbytes,
                                         _p(dev_status), _stream(stream)),
           "up_select_topp")


def up_compact(token_keep, cu_seqlens, kept_index, new_cu_seqlens, new_seq_lens, num_actual_tokens, ws, dev_status,
               hidden=None, out_hidden=None, positions=None, out_positions=None, slots=None, out_slots=None,
               kept_len=None, drop_layer=None, layer=0, stream=None):
    R = cu_seqlens.numel() - 1
    T = token_keep.numel()
    hdim = hidden.shape[1] if hidden is not None else 0
    L = drop_layer.numel() if drop_layer is not None else (kept_len.shape[0] if kept_len is not None else 0)
    _check(load_library().up_compact(_p(token_keep), _p(cu_seqlens), R, T, _p(hidden), hdim, _p(positions), _p(slots),
                                     _p(out_hidden), _p(out_positions), _p(out_slots), _p(kept_index),
                                     _p(new_cu_seqlens), _p(new_seq_lens), _p(num_actual_tokens), _p(kept_len),
                                     _p(drop_layer), L, layer, _p(ws), ws.numel() * ws.element_size(),
                                     _p(dev_status), _stream(stream)),
           "up_compact")


def up_compact_noalloc(token_keep, cu_seqlens, kept_index, new_cu_seqlens, new_seq_lens, num_actual_tokens,
                       dev_status, hidden=None, out_hidden=None, positions=None, out_positions=None, slots=None,
                       out_slots=None, kept_len=None, drop_layer=None, layer=0, stream=None):
    """up_compact for callers that cannot provide a device workspace: the library's own fixed scratch
    array is used instead (at most UP_NOALLOC_MAX_TOKENS tokens; calls that overlap on the GPU race)."""
    R = cu_seqlens.numel() - 1
    T = token_keep.numel()
    hdim = hidden.shape[1] if hidden is not None else 0
    L = drop_layer.numel() if drop_layer is not None else (kept_len.shape[0] if kept_len is not None else 0)
    _check(load_library().up_compact_noalloc(_p(token_keep), _p(cu_seqlens), R, T, _p(hidden), hdim, _p(positions),
                                             _p(slots), _p(out_hidden), _p(out_positions), _p(out_slots),
                                             _p(kept_index), _p(new_cu_seqlens), _p(new_seq_lens),
                                             _p(num_actual_tokens), _p(kept_len), _p(drop_layer), L, layer,
                                             _p(dev_status), _stream(stream)),
           "up_compact_noalloc")


def up_scatter_back(new_states, kept_index, num_actual_tokens, residual, dev_status, stream=None):
    """residual [T, hdim] receives the compacted rows new_states [T_upper <= T, hdim] (T_upper is
    passed as the bound of *num_actual_tokens)."""
    T, hdim = residual.shape
    assert new_states.shape[1] == hdim and new_states.shape[0] <= T
    _check(load_library().up_scatter_back(_bf16(new_states), _p(kept_index), _p(num_actual_tokens),
                                          new_states.shape[0], hdim, _bf16(residual), _p(dev_status),
                                          _stream(stream)),
           "up_scatter_back")


def up_slot_mapping(positions, cu_seqlens, block_table, B, slots, dev_status, num_tokens=None, stream=None):
    R = cu_seqlens.numel() - 1
    _check(load_library().up_slot_mapping(_p(positions), _p(cu_seqlens), R, positions.numel(), _p(num_tokens),
                                          _p(block_table), block_table.shape[1], B, _p(slots), _p(dev_status),
                                          _stream(stream)),
           "up_slot_mapping")


def up_seqused(kept_len, drop_layer, layer, orig_len, kv_len, seqused, stream=None):
    L, R = kept_len.shape
    _check(load_library().up_seqused(_p(kept_len), _p(drop_layer), L, R, layer, _p(orig_len), _p(kv_len),
                                     _p(seqused), _stream(stream)),
           "up_seqused")


# ------------------------------------------------------------------------------------------ the paged cache

def _kv_cache(k_cache, v_cache, k_scale, v_scale):
    """The up_kv_cache of tensors [num_blocks, Hkv, B, dk] (bf16, or float8_e4m3fn with uint8 scale tensors
    [num_blocks, Hkv, up_kv_scale_row(B)]); keys and values have the same shape and strides."""
    shape, strides, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    num_blocks, Hkv, B, dk = shape
    sb, sh, st, sd = strides
    assert v_cache.shape == shape and v_cache.stride() == strides and sd == 1
    assert v_cache.dtype == dtype and k_cache.is_cuda
    if dtype == _E4M3:
        rows = (num_blocks, Hkv, (B + 15) // 16 * 16)
        assert k_scale.shape == rows and v_scale.shape == rows and k_scale.is_contiguous() and v_scale.is_contiguous()
        assert k_scale.dtype == _U8 and v_scale.dtype == _U8
        return _KvCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), num_blocks, sb,
                        sh, st, Hkv, B, dk, KV_E4M3)
    assert dtype == _BF16
    return _KvCache(k_cache.data_ptr(), v_cache.data_ptr(), None, None, num_blocks, sb, sh, st, Hkv, B, dk, KV_BF16)


def _rows(t, T, heads, dk):
    """A bf16 tensor [T, heads, dk] whose tokens may lie at a stride (pointer, stride in elements)."""
    st, sh, sd = t.stride()
    assert t.shape == (T, heads, dk) and t.dtype == _BF16 and t.is_cuda
    assert (sd == 1 and (sh == dk or heads == 1)) or T == 0
    return t.data_ptr(), st


def up_kv_scale_row(B):
    return load_library().up_kv_scale_row(B)


def up_kv_write(k, v, slots, k_cache, v_cache, dev_status, k_scale=None, v_scale=None, num_tokens=None, stream=None):
    """k, v [T, Hkv, dk] (either may be None) into the rows that slots [T] int64 names."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    T = slots.numel()
    assert slots.dtype == _I64 and slots.is_contiguous()
    kp, ks = (None, 0) if k is None else _rows(k, T, cache.Hkv, cache.dk)
    vp, vs = (None, 0) if v is None else _rows(v, T, cache.Hkv, cache.dk)
    code = load_library().up_kv_write(ctypes.byref(cache), kp, ks, vp, vs, slots.data_ptr(), T, _p(num_tokens),
                                      dev_status.data_ptr(), _stream(stream))
    if code:
        raise UpError(code, "up_kv_write")


def up_kv_read(k_cache, v_cache, slots, k, v, dev_status, k_scale=None, v_scale=None, num_tokens=None, stream=None):
    """The rows that slots [T] int64 names to the packed streams k, v [T, Hkv, dk] (either may be None)."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    T = slots.numel()
    assert slots.dtype == _I64 and slots.is_contiguous()
    want = (T, cache.Hkv, cache.dk)
    assert (k is None or k.shape == want) and (v is None or v.shape == want)
    code = load_library().up_kv_read(ctypes.byref(cache), slots.data_ptr(), T, _p(num_tokens),
                                     None if k is None else _bf16(k), None if v is None else _bf16(v),
                                     dev_status.data_ptr(), _stream(stream))
    if code:
        raise UpError(code, "up_kv_read")


def up_paged_decode_workspace_bytes(R, Hq, Hkv, dk, B, max_blocks, window=0):
    return load_library().up_paged_decode_workspace_bytes(R, Hq, Hkv, dk, B, max_blocks, window)


def up_paged_decode(q, k_cache, v_cache, block_table, seqused, out, ws, dev_status, k_scale=None, v_scale=None,
                    lse=None, window=0, sm_scale=None, stream=None):
    """q [R, Hq, dk], one new token per request; block_table [R, max_blocks] int32; seqused [R] int32;
    out [R, Hq, dk]; ws of up_paged_decode_workspace_bytes(...) bytes; lse optional fp32 [R, Hq]."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    shape = q.shape
    R, Hq, dk = shape
    rows, max_blocks = block_table.shape
    assert dk == cache.dk and out.shape == shape
    assert block_table.dtype == _I32 and block_table.is_contiguous() and rows == R
    assert seqused.dtype == _I32 and seqused.is_contiguous() and seqused.numel() == R
    assert lse is None or (lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == (R, Hq))
    qp, qs = _rows(q, R, Hq, dk)
    code = load_library().up_paged_decode(qp, qs, ctypes.byref(cache), block_table.data_ptr(), seqused.data_ptr(), R,
                                          max_blocks, Hq, dk ** -0.5 if sm_scale is None else sm_scale, window,
                                          _bf16(out), _p(lse), ws.data_ptr(), ws.nbytes, dev_status.data_ptr(),
                                          _stream(stream))
    if code:
        raise UpError(code, "up_paged_decode")


# ------------------------------------------------------------------------------------------ rotary positions

def up_rope_plan(rot, theta=10000.0, layout="halves", scaling="none", factor=1.0, original_len=0, low=None, high=None,
                 gain=0.0):
    """The RopeTable of heads whose first `rot` numbers turn, in the layout "halves" or "pairs", with frequencies as they
    are ("none") or scaled: "linear", "bands" or "ramp" (up_rope_plan in include/uniprefill.h has the formulas; low and
    high, in turns over original_len, are 1 and 4 for bands and 1 and 32 for ramp unless given)."""
    kind, low0, high0 = ROPE_SCALINGS[scaling]
    plan = RopeTable()
    _check(load_library().up_rope_plan(rot, theta, ROPE_LAYOUTS[layout], kind, factor, original_len,
                                       low0 if low is None else low, high0 if high is None else high, gain,
                                       ctypes.byref(plan)), "up_rope_plan")
    return plan


def _launch(stream, *tensors):
    """The handle of a call's stream; its tensors, and the stream, belong to the current device, which is launched on."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise AssertionError("a tensor on another device than the current one")
    if stream is None:
        return _c_p(torch._C._cuda_getCurrentRawStream(device))
    assert stream.device.index == device
    return _c_p(stream.cuda_stream)


def up_rope(plan, positions, dev_status, q=None, q_out=None, k=None, k_out=None, num_tokens=None, transpose=False,
            stream=None):
    """q [T, Hq, dk] -> q_out, k [T, Hkv, dk] -> k_out (either pair may be None), turned by positions [T] int64;
    q_out may be q, and k_out k.  transpose: the gradient of that."""
    T = positions.numel()
    assert (q is None) == (q_out is None) and (k is None) == (k_out is None)
    assert positions.dtype is _I64 and positions.is_contiguous()
    assert num_tokens is None or num_tokens.dtype is _I32
    st = _launch(stream, positions, dev_status, q, q_out, k, k_out, num_tokens)
    Hq = Hkv = 0
    dk, qp, qs, qo, qos, kp, ks, ko, kos = 128, None, 0, None, 0, None, 0, None, 0
    if q is not None:
        _, Hq, dk = q.shape
        (qp, qs), (qo, qos) = _rows(q, T, Hq, dk), _rows(q_out, T, Hq, dk)
    if k is not None:
        Hkv = k.shape[1]
        dk = k.shape[2] if q is None else dk
        (kp, ks), (ko, kos) = _rows(k, T, Hkv, dk), _rows(k_out, T, Hkv, dk)
    code = load_library().up_rope(ctypes.byref(plan), qp, qs, qo, qos, Hq, kp, ks, ko, kos, Hkv, dk, positions.data_ptr(), T,
                                  _p(num_tokens), bool(transpose), dev_status.data_ptr(), st)
    if code:
        raise UpError(code, "up_rope")


# ------------------------------------------------------------------------------------------ eviction

def _int32(t, n):
    """n contiguous int32 numbers, or None"""
    if t is None:
        return None
    assert t.dtype is _I32 and t.is_contiguous() and t.numel() == n
    return t.data_ptr()


def _records(t, dtype, shape):
    """A cache's records, contiguous [num_blocks, Hkv, B], or None"""
    if t is None:
        return None
    assert t.dtype is dtype and t.is_contiguous() and t.shape == shape
    return t.data_ptr()


def up_kv_mass(q, k_cache, v_cache, block_table, seqused, lse, mass, born, dev_status, k_scale=None, v_scale=None,
               mass_out=None, counted=None, total=None, decay=1.0, sm_scale=None, stream=None):
    """mass_out (mass itself where None) <- decay * mass + the weights that q [R, Hq, dk] gave the cached rows, lse [R, Hq]
    being up_paged_decode's; mass [num_blocks, Hkv, B] fp32, born the same in int32; counted, total [R] int32."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    R, Hq, dk = q.shape
    rows, max_blocks = block_table.shape
    st = _launch(stream, q, k_cache, v_cache, block_table, seqused, lse, mass, mass_out, born, dev_status, k_scale, v_scale,
                 counted, total)
    shape = (cache.num_blocks, cache.Hkv, cache.B)
    mp, bp = _records(mass, torch.float32, shape), _records(born, _I32, shape)
    op = mp if mass_out is None else _records(mass_out, torch.float32, shape)
    assert dk == cache.dk and rows == R and lse.dtype is torch.float32 and lse.is_contiguous() and lse.shape == (R, Hq)
    qp, qs = _rows(q, R, Hq, dk)
    code = load_library().up_kv_mass(qp, qs, ctypes.byref(cache), _int32(block_table, R * max_blocks), _int32(seqused, R),
                                     lse.data_ptr(), R, max_blocks, Hq, dk ** -0.5 if sm_scale is None else sm_scale,
                                     _int32(counted, R), _int32(total, R), decay, mp, op, bp, dev_status.data_ptr(), st)
    if code:
        raise UpError(code, "up_kv_mass")


def up_kv_evict(mass, born, block_table, seqused, budget, moves, num_moves, new_len, dev_status, total=None, sinks=0,
                recent=0, stream=None):
    """Which rows of every request and head stay, budget [R] of them, and how they come to be the first:
    moves [R, Hkv, max_moves, 2] (from, to), num_moves [R, Hkv], new_len [R], all int32.  sinks and recent may be numbers of
    any size: no row's number is beyond 31 bits."""
    if not (0 <= sinks <= 0x7fffffff and 0 <= recent <= 0x7fffffff):       # (ctypes would cut them to 32 bits)
        sinks, recent = (max(-1, min(x, 0x7fffffff)) for x in (sinks, recent))
    shape = mass.shape
    num_blocks, Hkv, B = shape
    R, max_blocks = block_table.shape
    st = _launch(stream, mass, born, block_table, seqused, budget, moves, num_moves, new_len, dev_status, total)
    rows, heads, max_moves, two = moves.shape
    assert rows == R and heads == Hkv and two == 2
    code = load_library().up_kv_evict(_records(mass, torch.float32, shape), _records(born, _I32, shape), num_blocks, Hkv, B,
                                      _int32(block_table, R * max_blocks), _int32(seqused, R), _int32(budget, R), R, max_blocks,
                                      _int32(total, R), sinks, recent, _int32(moves, R * Hkv * max_moves * 2), max_moves,
                                      _int32(num_moves, R * Hkv), _int32(new_len, R), dev_status.data_ptr(), st)
    if code:
        raise UpError(code, "up_kv_evict")


def up_kv_move(k_cache, v_cache, block_table, moves, num_moves, dev_status, k_scale=None, v_scale=None, mass=None,
               born=None, stream=None):
    """Moves the rows of up_kv_evict's lists, with their records (mass and born, either may be None)."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    R, max_blocks = block_table.shape
    st = _launch(stream, k_cache, v_cache, block_table, moves, num_moves, dev_status, k_scale, v_scale, mass, born)
    shape = (cache.num_blocks, cache.Hkv, cache.B)
    rows, heads, max_moves, two = moves.shape
    assert rows == R and heads == cache.Hkv and two == 2
    code = load_library().up_kv_move(ctypes.byref(cache), _int32(block_table, R * max_blocks), R, max_blocks,
                                     _int32(moves, R * heads * max_moves * 2), max_moves, _int32(num_moves, R * heads),
                                     _records(mass, torch.float32, shape), _records(born, _I32, shape), dev_status.data_ptr(), st)
    if code:
        raise UpError(code, "up_kv_move")


# ------------------------------------------------------------------------------------------ status

def up_read_status(dev_status, stream=None):
    out = ctypes.c_int32(0)
    code = load_library().up_read_status(_p(dev_status), ctypes.byref(out), _stream(stream))
    if code not in (UP_OK, UP_ERR_DEVICE):
        _check(code, "up_read_status")
    return out.value


def up_status_string(code, device=False):
    return load_library().up_status_string(code, int(bool(device))).decode()


def up_kernel_launches():
    return int(load_library().up_kernel_launches())


def up_abi_version():
    return int(load_library().up_abi_version())


def up_debug_bounds():
    return int(load_library().up_debug_bounds())


from .step import DropStep  # noqa: E402,F401
