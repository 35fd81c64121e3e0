"""ctypes binding of ``libts.so`` (the C ABI declared in ``include/ts.h``).

Argument marshalling only: every step of the sparse-convolution path runs in
the library's HIP kernels.  PyTorch supplies device memory and the current
HIP stream.  Importing this module loads the in-tree ``libts.so`` and fails
loudly when it is missing -- there is no CPU fallback.

The ``ts_*`` functions mirror the C entry points one to one.  The small
classes below (``HashTable``, ``Kmap``) allocate the buffers the size queries
ask for and keep them alive next to the C structs that point into them.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
DEBUG_LIB_PATH = os.path.join(_HERE, "libts_debug.so")
# debug_binding() sets _LIB_OVERRIDE in a second instance of this module
LIB_PATH = globals().get("_LIB_OVERRIDE") or os.path.join(_HERE, "libts.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m convolution_voxelised_point_amd.build`")
_lib = ctypes.CDLL(LIB_PATH)

TS_OK, TS_ERR_INVALID_ARG, TS_ERR_UNSUPPORTED, TS_ERR_HIP = 0, 1, 2, 3
TS_F32, TS_F16, TS_BF16 = 0, 1, 2
TS_DATAFLOW_AUTO, TS_DATAFLOW_IMPLICIT_GEMM, TS_DATAFLOW_GATHER_SCATTER, TS_DATAFLOW_IMPLICIT_GEMM_PACKED = 0, 1, 2, 3
TS_DATAFLOW_FETCH_ON_DEMAND = 4
TS_FLAG_DUP, TS_FLAG_RANGE, TS_FLAG_FULL = 1, 2, 4
TS_KMAP_PAIRS, TS_KMAP_BWD, TS_KMAP_NATURAL, TS_KMAP_TARGET, TS_KMAP_TRANSPOSED = 1, 2, 4, 8, 16
TS_KMAP_GROUPS, TS_KMAP_NO_TABLE = 32, 64
TS_OP_FWD, TS_OP_DGRAD, TS_OP_WGRAD, TS_OP_TRANSPOSE = 0, 1, 2, 3
TS_POOL_MAX, TS_POOL_AVG = 0, 1
TS_TILE, TS_GTILE, TS_MAX_KVOL = 16, 128, 64
TS_NOALLOC_SCRATCH_BYTES = 4 << 20
TS_ACT8_BLOCK = 32
TS_DEBUG_SRC_ROW, TS_DEBUG_DST_ROW = 1, 2

_DT = {torch.float32: TS_F32, torch.float16: TS_F16, torch.bfloat16: TS_BF16}

_vp, _i64, _i32, _u32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32, ctypes.c_size_t


class TsRel(ctypes.Structure):
    _fields_ = [("n_dest_cap", _i64), ("n_tiles", _i64), ("n_dest", _vp), ("tile_mask", _vp),
                ("tile_rows", _vp), ("nbr", _vp), ("row_mask", _vp), ("n_gtiles", _i64), ("gcount", _vp),
                ("gsrc", _vp), ("gslot", _vp)]


class TsKmap(ctypes.Structure):
    _fields_ = [("ndim", ctypes.c_int32), ("ksize", ctypes.c_int32), ("stride", ctypes.c_int32),
                ("kvol", ctypes.c_int32), ("flags", ctypes.c_uint32), ("mirror_bwd", ctypes.c_int32),
                ("n_in", _i64), ("n_out_cap", _i64), ("n_out", _vp), ("fwd", TsRel), ("bwd", TsRel),
                ("pair_cap", _i64), ("pair_start", _vp), ("pair_in", _vp), ("pair_out", _vp),
                ("scratch", _vp), ("scratch_bytes", _sz)]


class TsAttn(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("hq", ctypes.c_int32), ("hk", ctypes.c_int32), ("d", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("scale", ctypes.c_float), ("cap", ctypes.c_float), ("nq", _i64),
                ("nk", _i64), ("n_sets", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("o_stride", _i64), ("q_starts", _vp), ("k_starts", _vp), ("slopes", _vp), ("q_coords", _vp),
                ("k_coords", _vp)]


class TsAct8(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp)]


class TsRope(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("d", ctypes.c_int32), ("ndim", ctypes.c_int32), ("pairs", ctypes.c_int32 * 3),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float), ("n", _i64), ("coords", _vp), ("freqs", _vp)]


class TsRopeHeads(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("x_stride", _i64), ("y_stride", _i64), ("dy_stride", _i64), ("dx_stride", _i64),
                ("x", _vp), ("w", _vp), ("y", _vp), ("dy", _vp), ("dx", _vp), ("dw", _vp)]


class TsGroups(ctypes.Structure):
    _fields_ = [("n_groups", ctypes.c_int32), ("n_rows", _i64), ("starts", _vp), ("rows", _vp), ("n_src", _i64)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_P = ctypes.POINTER(TsKmap)
_lib_status_string = _sig("ts_status_string", ctypes.c_char_p, [_i32])
_lib_version = _sig("ts_version", ctypes.c_char_p, [])
_lib_hash_capacity = _sig("ts_hash_capacity", _i64, [_i64, ctypes.c_double])
_lib_hash_table_bytes = _sig("ts_hash_table_bytes", _sz, [_i64])
_lib_hash_build = _sig("ts_hash_build", _i32, [_vp, _i64, _i32, _vp, _i64, _vp, _vp])
_lib_hash_query = _sig("ts_hash_query", _i32, [_vp, _i64, _i32, _vp, _i64, _vp, _vp])
_lib_support_scratch_bytes = _sig("ts_support_scratch_bytes", _sz, [_i64])
_lib_strided_support = _sig("ts_strided_support", _i32, [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _sz, _vp, _vp])
_lib_generative_scratch_bytes = _sig("ts_generative_scratch_bytes", _sz, [_i64, _i32, _i32])
_lib_generative_support = _sig("ts_generative_support", _i32,
                               [_vp, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp, _vp])
_lib_transposed_support = _sig("ts_transposed_support", _i32,
                               [_vp, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp, _vp])
_lib_voxelize_scratch_bytes = _sig("ts_voxelize_scratch_bytes", _sz, [_i64])
_lib_voxelize = _sig("ts_voxelize", _i32, [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp,
                                           _sz, _vp, _vp])
_lib_devoxelize = _sig("ts_devoxelize", _i32, [_vp, _i64, _vp, _i32, _vp, _i32, _vp])
_lib_kmap_bytes = _sig("ts_kmap_bytes", _sz, [_i64, _i64, _i32, _i32, _i32, _u32])
_lib_kmap_build = _sig("ts_kmap_build", _i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _u32,
                                               _vp, _sz, _P, _vp])
_lib_conv_workspace_bytes = _sig("ts_conv_workspace_bytes", _sz, [_P, _i32, _i32, _i32, _i32, _i32])
_lib_conv_pack_weights = _sig("ts_conv_pack_weights", _i32, [_P, _vp, _i32, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_conv_fwd = _sig("ts_conv_fwd", _i32, [_P, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_subm_conv_fwd = _sig("ts_subm_conv_fwd", _i32, [_P, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_conv_fwd_strided = _sig("ts_conv_fwd_strided", _i32,
                             [_vp, _i64, _i32, _vp, _i64, _i32, _i32, _u32, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _P,
                              _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_conv_fwd_generative = _sig("ts_conv_fwd_generative", _i32,
                                [_vp, _i64, _i32, _vp, _i64, _i32, _u32, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _sz, _P,
                                 _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_conv_transpose_fwd = _sig("ts_conv_transpose_fwd", _i32,
                               [_P, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_graph_conv_fwd = _sig("ts_graph_conv_fwd", _i32, [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _i32, _vp, _i32, _vp, _i32,
                                                       _i32, _vp, _vp])
_lib_pool_fwd = _sig("ts_pool_fwd", _i32, [_P, _vp, _i32, _vp, _i32, _i32, _i32, _vp])
_lib_conv_bwd_dgrad = _sig("ts_conv_bwd_dgrad", _i32, [_P, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp])
_lib_conv_bwd_wgrad = _sig("ts_conv_bwd_wgrad", _i32, [_P, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _sz, _vp])
_lib_conv_bwd_dgrad_noalloc = _sig("ts_conv_bwd_dgrad_noalloc", _i32, [_P, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _vp])
_A = ctypes.POINTER(TsAttn)
_lib_attn_workspace_bytes = _sig("ts_attn_workspace_bytes", _sz, [_A, _i32])
_lib_attn_fwd = _sig("ts_attn_fwd", _i32, [_A, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp])
_lib_attn_bwd = _sig("ts_attn_bwd", _i32, [_A, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp])
_C = ctypes.POINTER(TsAct8)
_lib_act_pack = _sig("ts_act_pack", _i32, [_vp, _i64, _i32, _i32, _C, _vp])
_lib_act_unpack = _sig("ts_act_unpack", _i32, [_C, _i64, _i32, _vp, _i32, _vp])
_lib_conv_wgrad_act8_workspace_bytes = _sig("ts_conv_wgrad_act8_workspace_bytes", _sz, [_P, _i32, _i32])
_lib_conv_bwd_wgrad_act8 = _sig("ts_conv_bwd_wgrad_act8", _i32, [_P, _C, _i32, _vp, _i32, _i32, _vp, _vp, _sz, _vp])
_lib_norm_fwd = _sig("ts_norm_fwd", _i32, [_vp, _vp, _vp, _i64, _i32, ctypes.c_float, _i32, _vp, _vp, _vp, _C, _C, _vp])
_lib_norm_workspace_bytes = _sig("ts_norm_workspace_bytes", _sz, [_i64, _i32])
_lib_norm_bwd = _sig("ts_norm_bwd", _i32, [_vp, _vp, _C, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _sz, _vp])
_R, _H = ctypes.POINTER(TsRope), ctypes.POINTER(TsRopeHeads)
_lib_rope_workspace_bytes = _sig("ts_rope_workspace_bytes", _sz, [_R, _i32, _i32])
_lib_rope_fwd = _sig("ts_rope_fwd", _i32, [_R, _H, _H, _vp])
_lib_rope_bwd = _sig("ts_rope_bwd", _i32, [_R, _H, _H, _vp, _sz, _vp])
_lib_route_workspace_bytes = _sig("ts_route_workspace_bytes", _sz, [_i64, _i32, _i32])
_lib_route_fwd = _sig("ts_route_fwd", _i32, [_vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp])
_lib_route_bwd = _sig("ts_route_bwd", _i32, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp])
_lib_combine_fwd = _sig("ts_combine_fwd", _i32, [_vp, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp])
_lib_combine_bwd = _sig("ts_combine_bwd", _i32, [_vp, _vp, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp])
_G = ctypes.POINTER(TsGroups)
_lib_group_fwd = _sig("ts_group_fwd", _i32, [_G, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp])
_lib_group_bwd_dgrad = _sig("ts_group_bwd_dgrad", _i32, [_G, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp])
_lib_group_wgrad_workspace_bytes = _sig("ts_group_wgrad_workspace_bytes", _sz, [_G, _i32, _i32])
_lib_group_bwd_wgrad = _sig("ts_group_bwd_wgrad", _i32, [_G, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _sz, _vp, _vp])
_lib_debug_violations = _sig("ts_debug_violations", _i32, [ctypes.POINTER(_u32)])

EXPORTED = ["ts_status_string", "ts_version", "ts_hash_capacity", "ts_hash_table_bytes", "ts_hash_build",
            "ts_hash_query", "ts_support_scratch_bytes", "ts_strided_support", "ts_generative_scratch_bytes",
            "ts_generative_support", "ts_transposed_support", "ts_voxelize_scratch_bytes", "ts_voxelize",
            "ts_devoxelize", "ts_kmap_bytes", "ts_kmap_build",
            "ts_conv_workspace_bytes", "ts_conv_pack_weights", "ts_conv_fwd", "ts_subm_conv_fwd", "ts_conv_fwd_strided",
            "ts_conv_fwd_generative", "ts_conv_transpose_fwd", "ts_pool_fwd", "ts_graph_conv_fwd", "ts_conv_bwd_dgrad",
            "ts_conv_bwd_wgrad", "ts_conv_bwd_dgrad_noalloc", "ts_attn_workspace_bytes", "ts_attn_fwd", "ts_attn_bwd",
            "ts_act_pack", "ts_act_unpack", "ts_conv_wgrad_act8_workspace_bytes", "ts_conv_bwd_wgrad_act8", "ts_norm_fwd",
            "ts_norm_workspace_bytes", "ts_norm_bwd", "ts_rope_workspace_bytes", "ts_rope_fwd", "ts_rope_bwd",
            "ts_route_workspace_bytes", "ts_route_fwd", "ts_route_bwd", "ts_combine_fwd", "ts_combine_bwd", "ts_group_fwd",
            "ts_group_bwd_dgrad", "ts_group_wgrad_workspace_bytes", "ts_group_bwd_wgrad", "ts_debug_violations"]


class TsError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {ts_status_string(status)} ({status})")
        self.status = status


def _check(st: int, what: str) -> None:
    if st != TS_OK:
        raise TsError(st, what)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "device tensors must be contiguous CUDA/HIP tensors"
    return ctypes.c_void_p(t.data_ptr())


def _rows(t: torch.Tensor):
    """Rows of [n][heads][d], the heads of a row adjacent."""
    assert t.is_cuda and _row_stride(t) is not None, "device tensors [n][heads][d] with adjacent heads"
    return ctypes.c_void_p(t.data_ptr())


def _row_stride(t: torch.Tensor) -> Optional[int]:
    """Elements between the rows of [n][heads][d], or None where the heads of a row are not adjacent."""
    if t.dim() != 3:
        return None
    n, h, d = t.shape
    row, head, one = t.stride()
    if (one != 1 and d > 1) or (head != d and h > 1):
        return None
    if n <= 1:
        return h * d
    return row if row >= h * d else None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    return _DT[t.dtype]


# ---------------------------------------------------------------- 1:1 wrappers
def ts_status_string(st: int) -> str:
    return _lib_status_string(st).decode()


def ts_debug_violations() -> int:
    """Bits raised by the bounds checks on the current device since the last
    call (the call waits for the device and clears them).  Only the
    bounds-check build has checks; the regular library raises TsError
    (unsupported)."""
    bits = _u32(0)
    _check(_lib_debug_violations(ctypes.byref(bits)), "ts_debug_violations")
    return int(bits.value)


def debug_binding():
    """A second instance of this binding over the bounds-check build
    ``libts_debug.so`` (the same entry points; every kernel checks the row
    indexes it reads from a map).  Raises ImportError when it is not built."""
    import importlib.util
    spec = importlib.util.spec_from_file_location(__name__ + "_debug", __file__)
    mod = importlib.util.module_from_spec(spec)
    mod._LIB_OVERRIDE = DEBUG_LIB_PATH
    spec.loader.exec_module(mod)
    return mod


def ts_version() -> str:
    return _lib_version().decode()


def ts_hash_capacity(n: int, rsv_ratio: float = 2.0) -> int:
    return int(_lib_hash_capacity(n, rsv_ratio))


def ts_hash_table_bytes(cap: int) -> int:
    return int(_lib_hash_table_bytes(cap))


def ts_hash_build(coords: torch.Tensor, table: torch.Tensor, cap: int, err_flags: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    ndim = coords.shape[1] - 1
    _check(_lib_hash_build(_p(coords), coords.shape[0], ndim, _p(table), cap, _p(err_flags), _stream(stream)),
           "ts_hash_build")


def ts_hash_query(table: torch.Tensor, cap: int, q: torch.Tensor, rows: torch.Tensor, stream=None) -> None:
    _check(_lib_hash_query(_p(table), cap, q.shape[1] - 1, _p(q), q.shape[0], _p(rows), _stream(stream)),
           "ts_hash_query")


def ts_support_scratch_bytes(n_in: int) -> int:
    return int(_lib_support_scratch_bytes(n_in))


def ts_strided_support(in_coords, stride, out_coords, n_out, out_table, out_cap, scratch, err_flags=None,
                       stream=None) -> None:
    _check(_lib_strided_support(_p(in_coords), in_coords.shape[0], in_coords.shape[1] - 1, stride, _p(out_coords),
                                _p(n_out), _p(out_table), out_cap, _p(scratch), scratch.numel(), _p(err_flags),
                                _stream(stream)), "ts_strided_support")


def ts_generative_scratch_bytes(n_in: int, ndim: int, ksize: int) -> int:
    return int(_lib_generative_scratch_bytes(n_in, ndim, ksize))


def ts_generative_support(in_coords, ksize, out_coords, n_out, out_table, out_cap, scratch, err_flags=None,
                          stream=None) -> None:
    _check(_lib_generative_support(_p(in_coords), in_coords.shape[0], in_coords.shape[1] - 1, ksize, _p(out_coords),
                                   out_coords.shape[0], _p(n_out), _p(out_table), out_cap, _p(scratch),
                                   scratch.numel(), _p(err_flags), _stream(stream)), "ts_generative_support")


def ts_transposed_support(in_coords, ksize, stride, out_coords, n_out, out_table, out_cap, scratch, err_flags=None,
                          stream=None) -> None:
    _check(_lib_transposed_support(_p(in_coords), in_coords.shape[0], in_coords.shape[1] - 1, ksize, stride,
                                   _p(out_coords), out_coords.shape[0], _p(n_out), _p(out_table), out_cap,
                                   _p(scratch), scratch.numel(), _p(err_flags), _stream(stream)),
           "ts_transposed_support")


def ts_voxelize_scratch_bytes(n: int) -> int:
    return int(_lib_voxelize_scratch_bytes(n))


def ts_voxelize(batch, pos, size, origin, feats, out_coords, n_out, out_table, out_cap, vox_of, out_feats, scratch,
                err_flags=None, stream=None) -> None:
    ndim = pos.shape[1]
    sz = (ctypes.c_float * ndim)(*[float(v) for v in size])
    og = (ctypes.c_float * ndim)(*[float(v) for v in origin])
    c = 0 if feats is None else feats.shape[1]
    _check(_lib_voxelize(_p(batch), _p(pos), pos.shape[0], ndim, sz, og, _p(feats), c, _p(out_coords), _p(n_out),
                         _p(out_table), out_cap, _p(vox_of), _p(out_feats), _p(scratch), scratch.numel(), _p(err_flags),
                         _stream(stream)), "ts_voxelize")


def ts_devoxelize(vox_of, vox_feats, point_feats, stream=None) -> None:
    _check(_lib_devoxelize(_p(vox_of), vox_of.shape[0], _p(vox_feats), vox_feats.shape[1], _p(point_feats),
                           _dt(vox_feats), _stream(stream)), "ts_devoxelize")


def ts_kmap_bytes(n_in: int, n_out_cap: int, ndim: int, ksize: int, stride: int, flags: int) -> int:
    return int(_lib_kmap_bytes(n_in, n_out_cap, ndim, ksize, stride, flags))


def ts_kmap_build(in_coords, in_table, in_cap, out_coords, n_out_cap, n_out, out_table, out_cap, ndim, ksize, stride,
                  flags, buf, kmap: TsKmap, stream=None) -> None:
    _check(_lib_kmap_build(_p(in_coords), in_coords.shape[0], _p(in_table), in_cap, _p(out_coords), n_out_cap,
                           _p(n_out), _p(out_table), out_cap, ndim, ksize, stride, flags, _p(buf), buf.numel(),
                           ctypes.byref(kmap), _stream(stream)), "ts_kmap_build")


def ts_conv_workspace_bytes(kmap: TsKmap, cin: int, cout: int, op: int, in_dtype: int, dataflow: int) -> int:
    return int(_lib_conv_workspace_bytes(ctypes.byref(kmap), cin, cout, op, in_dtype, dataflow))


def ts_conv_pack_weights(kmap, w, op, ws, stream=None) -> None:
    """Weights [kvol][cin][cout] packed into `ws` for a later call of `op`
    with TS_DATAFLOW_IMPLICIT_GEMM_PACKED."""
    _check(_lib_conv_pack_weights(ctypes.byref(kmap), _p(w), w.shape[1], w.shape[2], op, _dt(w), _p(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)), "ts_conv_pack_weights")


def ts_conv_fwd(kmap, x, w, y, dataflow=TS_DATAFLOW_AUTO, ws=None, stream=None, subm=False) -> None:
    f = _lib_subm_conv_fwd if subm else _lib_conv_fwd
    _check(f(ctypes.byref(kmap), _p(x), x.shape[1], _p(w), w.shape[2], _p(y), _dt(x), _dt(y), dataflow, _p(ws),
             0 if ws is None else ws.numel(), _stream(stream)), "ts_subm_conv_fwd" if subm else "ts_conv_fwd")


def ts_subm_conv_fwd(kmap, x, w, y, dataflow=TS_DATAFLOW_AUTO, ws=None, stream=None) -> None:
    ts_conv_fwd(kmap, x, w, y, dataflow, ws, stream, subm=True)


def ts_conv_fwd_strided(in_coords, in_table, in_cap, ksize, stride, kmap_flags, out_coords, n_out, out_table, out_cap,
                        err_flags, map_buf, kmap, x, w, y, dataflow=TS_DATAFLOW_AUTO, ws=None, stream=None) -> None:
    _check(_lib_conv_fwd_strided(_p(in_coords), in_coords.shape[0], in_coords.shape[1] - 1, _p(in_table), in_cap,
                                 ksize, stride, kmap_flags, _p(out_coords), _p(n_out), _p(out_table), out_cap,
                                 _p(err_flags), _p(map_buf), map_buf.numel(), ctypes.byref(kmap), _p(x), x.shape[1],
                                 _p(w), w.shape[2], _p(y), _dt(x), _dt(y), dataflow, _p(ws),
                                 0 if ws is None else ws.numel(), _stream(stream)), "ts_conv_fwd_strided")


def ts_conv_fwd_generative(in_coords, in_table, in_cap, ksize, kmap_flags, out_coords, n_out, out_table, out_cap,
                           err_flags, map_buf, kmap, x, w, y, dataflow=TS_DATAFLOW_AUTO, ws=None,
                           stream=None) -> None:
    """out_coords and y have the same row capacity (n_out_cap)."""
    assert out_coords.shape[0] == y.shape[0]
    _check(_lib_conv_fwd_generative(_p(in_coords), in_coords.shape[0], in_coords.shape[1] - 1, _p(in_table), in_cap,
                                    ksize, kmap_flags, _p(out_coords), out_coords.shape[0], _p(n_out),
                                    _p(out_table), out_cap, _p(err_flags), _p(map_buf), map_buf.numel(),
                                    ctypes.byref(kmap), _p(x), x.shape[1], _p(w), w.shape[2], _p(y), _dt(x), _dt(y),
                                    dataflow, _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "ts_conv_fwd_generative")


def ts_conv_transpose_fwd(kmap, x, w, y, dataflow=TS_DATAFLOW_AUTO, ws=None, stream=None) -> None:
    _check(_lib_conv_transpose_fwd(ctypes.byref(kmap), _p(x), x.shape[1], _p(w), w.shape[2], _p(y), _dt(x), _dt(y),
                                   dataflow, _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "ts_conv_transpose_fwd")


def ts_graph_conv_fwd(indptr, src, rel, n_src, n_rel, x, w, y, err_flags=None, stream=None) -> None:
    _check(_lib_graph_conv_fwd(_p(indptr), _p(src), _p(rel), indptr.shape[0] - 1, n_src, n_rel, _p(x), w.shape[1],
                               _p(w), w.shape[2], _p(y), _dt(w), _dt(y), _p(err_flags), _stream(stream)),
           "ts_graph_conv_fwd")


def ts_pool_fwd(kmap, x, y, mode=TS_POOL_MAX, stream=None) -> None:
    _check(_lib_pool_fwd(ctypes.byref(kmap), _p(x), x.shape[1], _p(y), _dt(x), _dt(y), mode, _stream(stream)),
           "ts_pool_fwd")


def ts_conv_bwd_dgrad(kmap, dy, w, dx, dataflow=TS_DATAFLOW_AUTO, ws=None, stream=None) -> None:
    _check(_lib_conv_bwd_dgrad(ctypes.byref(kmap), _p(dy), dy.shape[1], _p(w), dx.shape[1], _p(dx), _dt(dy), _dt(dx),
                               dataflow, _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "ts_conv_bwd_dgrad")


def ts_conv_bwd_dgrad_noalloc(kmap, dy, w, dx, stream=None) -> None:
    """dgrad with the library's static scratch instead of a workspace."""
    _check(_lib_conv_bwd_dgrad_noalloc(ctypes.byref(kmap), _p(dy), dy.shape[1], _p(w), dx.shape[1], _p(dx), _dt(dy),
                                       _dt(dx), _stream(stream)), "ts_conv_bwd_dgrad_noalloc")


def ts_conv_bwd_wgrad(kmap, x, dy, dw, ws, stream=None) -> None:
    _check(_lib_conv_bwd_wgrad(ctypes.byref(kmap), _p(x), x.shape[1], _p(dy), dy.shape[1], _dt(x), _p(dw), _p(ws),
                               ws.numel(), _stream(stream)), "ts_conv_bwd_wgrad")


def ts_attn_workspace_bytes(at: TsAttn, backward: bool) -> int:
    return int(_lib_attn_workspace_bytes(ctypes.byref(at), 1 if backward else 0))


def ts_attn_fwd(at: TsAttn, q, k, v, out, lse, ws=None, err_flags=None, stream=None) -> None:
    """q, k, v, out: rows `at.*_stride` elements apart."""
    _check(_lib_attn_fwd(ctypes.byref(at), _rows(q), _rows(k), _rows(v), _rows(out), _p(lse), _p(ws),
                         0 if ws is None else ws.numel(), _p(err_flags), _stream(stream)), "ts_attn_fwd")


def ts_attn_bwd(at: TsAttn, q, k, v, out, lse, dout, dq, dk, dv, ws, err_flags=None, stream=None) -> None:
    _check(_lib_attn_bwd(ctypes.byref(at), _rows(q), _rows(k), _rows(v), _rows(out), _p(lse), _rows(dout), _rows(dq),
                         _rows(dk), _rows(dv), _p(ws), 0 if ws is None else ws.numel(), _p(err_flags),
                         _stream(stream)), "ts_attn_bwd")


def _act(a: "Optional[Act8]"):
    return None if a is None else ctypes.byref(TsAct8(a.codes.data_ptr(), a.scales.data_ptr()))


def ts_act_pack(x, a: "Act8", stream=None) -> None:
    _check(_lib_act_pack(_p(x), x.shape[0], x.shape[1], _dt(x), _act(a), _stream(stream)), "ts_act_pack")


def ts_act_unpack(a: "Act8", x, stream=None) -> None:
    _check(_lib_act_unpack(_act(a), x.shape[0], x.shape[1], _p(x), _dt(x), _stream(stream)), "ts_act_unpack")


def ts_conv_wgrad_act8_workspace_bytes(kmap: TsKmap, cin: int, cout: int) -> int:
    return int(_lib_conv_wgrad_act8_workspace_bytes(ctypes.byref(kmap), cin, cout))


def ts_conv_bwd_wgrad_act8(kmap, x: "Act8", dy, dw, ws, stream=None) -> None:
    _check(_lib_conv_bwd_wgrad_act8(ctypes.byref(kmap), _act(x), x.codes.shape[1], _p(dy), dy.shape[1], _dt(dy), _p(dw),
                                    _p(ws), ws.numel(), _stream(stream)), "ts_conv_bwd_wgrad_act8")


def ts_norm_fwd(x, residual, w, eps, h=None, y=None, rstd=None, y8=None, h8=None, stream=None) -> None:
    _check(_lib_norm_fwd(_p(x), _p(residual), _p(w), x.shape[0], x.shape[1], eps, _dt(x), _p(h), _p(y), _p(rstd),
                         _act(y8), _act(h8), _stream(stream)), "ts_norm_fwd")


def ts_norm_workspace_bytes(n: int, c: int) -> int:
    return int(_lib_norm_workspace_bytes(n, c))


def ts_norm_bwd(dy, h, h8, w, rstd, dh, dx, dw, ws, stream=None) -> None:
    _check(_lib_norm_bwd(_p(dy), _p(h), _act(h8), _p(w), _p(rstd), _p(dh), dy.shape[0], dy.shape[1], _dt(dy), _p(dx),
                         _p(dw), _p(ws), 0 if ws is None else ws.numel(), _stream(stream)), "ts_norm_bwd")


# ---------------------------------------------------------------- owners of buffers
def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


def _zero_bytes(n: int, device) -> torch.Tensor:
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


class HashTable:
    """A coordinate table sized by the reserve ratio."""

    def __init__(self, coords: torch.Tensor, rsv_ratio: float = 2.0, err_flags: Optional[torch.Tensor] = None,
                 build: bool = True, stream=None):
        self.ndim = coords.shape[1] - 1
        self.cap = ts_hash_capacity(coords.shape[0], rsv_ratio)
        self.buf = _zero_bytes(ts_hash_table_bytes(self.cap), coords.device)  # a table starts zero-filled
        if build:
            ts_hash_build(coords, self.buf, self.cap, err_flags, stream)

    @classmethod
    def with_capacity(cls, ndim: int, cap: int, device) -> "HashTable":
        """An empty (zero-filled) table of `cap` block slots."""
        t = cls.__new__(cls)
        t.ndim, t.cap = ndim, cap
        t.buf = _zero_bytes(ts_hash_table_bytes(cap), device)
        return t

    def query(self, q: torch.Tensor, stream=None) -> torch.Tensor:
        rows = torch.empty(q.shape[0], dtype=torch.int32, device=q.device)
        ts_hash_query(self.buf, self.cap, q, rows, stream)
        return rows


class Kmap:
    """A built kernel map: the C struct plus the buffers it points into."""

    def __init__(self, struct: TsKmap, buf: torch.Tensor, keep=()):
        self.s = struct
        self.buf = buf
        self.keep = keep

    @property
    def kvol(self) -> int:
        return self.s.kvol

    def n_out(self) -> int:
        """Output row count (reads a device scalar: synchronises)."""
        base = self.buf.data_ptr()
        if self.s.n_out >= base and self.s.n_out < base + self.buf.numel():
            return int(self._view(self.s.n_out, torch.int64, 1)[0])
        for t in self.keep:
            if isinstance(t, torch.Tensor) and t.data_ptr() == self.s.n_out:
                return int(t[0])
        raise RuntimeError("n_out pointer not owned")

    def _view(self, ptr: int, dtype, count: int) -> torch.Tensor:
        off = ptr - self.buf.data_ptr()
        itemsize = torch.tensor([], dtype=dtype).element_size()
        assert 0 <= off and off + count * itemsize <= self.buf.numel()
        return self.buf[off:off + count * itemsize].view(dtype)

    def rel_arrays(self, which: str = "fwd") -> dict:
        """Device views of a relation's arrays (those the map holds)."""
        r = getattr(self.s, which)
        nt, kv, ng = r.n_tiles, self.s.kvol, r.n_gtiles
        out = {"row_mask": self._view(r.row_mask, torch.int64, r.n_dest_cap)}
        if r.nbr:
            out["tile_mask"] = self._view(r.tile_mask, torch.int64, nt)
            out["tile_rows"] = self._view(r.tile_rows, torch.int32, nt * TS_TILE)
            out["nbr"] = self._view(r.nbr, torch.int32, r.n_dest_cap * kv)
        if ng:
            out["gcount"] = self._view(r.gcount, torch.int32, ng * kv)
            out["gsrc"] = self._view(r.gsrc, torch.int32, ng * kv * TS_GTILE)
            out["gslot"] = self._view(r.gslot, torch.uint8, ng * kv * TS_GTILE)
        return out

    def pairs(self):
        """(pair_start[kvol+1], pair_in[P], pair_out[P]) on the host."""
        ps = self._view(self.s.pair_start, torch.int64, self.s.kvol + 1).cpu().numpy()
        P = int(ps[-1])
        pin = self._view(self.s.pair_in, torch.int32, max(P, 0)).cpu().numpy()
        pout = self._view(self.s.pair_out, torch.int32, max(P, 0)).cpu().numpy()
        return ps, pin, pout


def decode_rel(arrs: dict, kvol: int, transposed: bool = False) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Host decode of a relation into (in, out, offset) triples, walking the
    tiles (so every destination row must sit in exactly one tile slot).

    Used by tests; ``transposed`` marks a relation whose destinations are
    input rows."""
    rows = arrs["tile_rows"].cpu().numpy()
    rows = rows[rows >= 0].astype(np.int64)
    nbr = arrs["nbr"].cpu().numpy().reshape(-1, kvol)
    sub = nbr[rows]
    d, o = np.nonzero(sub >= 0)
    a = sub[d, o].astype(np.int32)
    b = rows[d].astype(np.int32)
    c = o.astype(np.int32)
    return (b, a, c) if transposed else (a, b, c)


def decode_groups(arrs: dict, kvol: int, transposed: bool = False) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Host decode of a relation's pair groups into (in, out, offset)
    triples (tile t, offset o: entries from 16 * sum of earlier offsets'
    whole groups, gcount of them).  Used by tests."""
    cnt = arrs["gcount"].cpu().numpy().reshape(-1, kvol).astype(np.int64)
    nt = cnt.shape[0]
    src = arrs["gsrc"].cpu().numpy().reshape(nt, kvol * TS_GTILE)
    slot = arrs["gslot"].cpu().numpy().reshape(nt, kvol * TS_GTILE).astype(np.int64)
    start = np.zeros_like(cnt)
    start[:, 1:] = np.cumsum((cnt[:, :-1] + 15) // 16 * 16, axis=1)
    t_idx, o_idx = np.nonzero(cnt > 0)
    a, b, c = [], [], []
    for t, o in zip(t_idx, o_idx):
        e0, n = start[t, o], cnt[t, o]
        a.append(src[t, e0:e0 + n])
        b.append(t * TS_GTILE + slot[t, e0:e0 + n])
        c.append(np.full(n, o, np.int64))
    if not a:
        z = np.zeros(0, np.int32)
        return z, z, z
    a, b, c = (np.concatenate(v).astype(np.int32) for v in (a, b, c))
    return (b, a, c) if transposed else (a, b, c)


def build_kmap(coords: torch.Tensor, table: HashTable, ksize: int, stride: int = 1, flags: int = 0,
               out_coords: Optional[torch.Tensor] = None, n_out: Optional[torch.Tensor] = None,
               out_table: Optional[HashTable] = None, stream=None) -> Kmap:
    """Allocate and build a kernel map (submanifold when stride == 1 and
    neither TS_KMAP_TARGET nor TS_KMAP_TRANSPOSED is set; otherwise over
    out_coords / n_out)."""
    ndim = coords.shape[1] - 1
    n_in = coords.shape[0]
    own_outputs = flags & (TS_KMAP_TARGET | TS_KMAP_TRANSPOSED)
    n_out_cap = n_in if (stride == 1 and not own_outputs) else out_coords.shape[0]
    nbytes = ts_kmap_bytes(n_in, n_out_cap, ndim, ksize, stride, flags)
    if nbytes == 0:
        raise TsError(TS_ERR_INVALID_ARG, "ts_kmap_bytes")
    buf = _bytes(nbytes, coords.device)
    km = TsKmap()
    ts_kmap_build(coords, table.buf, table.cap, out_coords, n_out_cap, n_out,
                  None if out_table is None else out_table.buf, 0 if out_table is None else out_table.cap,
                  ndim, ksize, stride, flags, buf, km, stream)
    return Kmap(km, buf, keep=(coords, table, out_coords, n_out, out_table))


def strided_support(coords: torch.Tensor, stride: int, rsv_ratio: float = 2.0, err_flags=None, stream=None):
    """(out_coords [capacity n_in], n_out device scalar, out table)."""
    n = coords.shape[0]
    out = torch.zeros_like(coords)
    n_out = torch.zeros(1, dtype=torch.int64, device=coords.device)
    table = HashTable(coords, rsv_ratio, build=False)
    scratch = _bytes(ts_support_scratch_bytes(n), coords.device)
    ts_strided_support(coords, stride, out, n_out, table.buf, table.cap, scratch, err_flags, stream)
    return out, n_out, table


def generative_table_capacity(n_in: int) -> int:
    """Block slots for the table of a generated support: four per input row
    (a site grid of surfaces spans about 1.3 blocks per input row for a 3^3
    kernel); a support that needs more raises TS_FLAG_FULL."""
    return ts_hash_capacity(n_in, 4.0)


def generative_support(coords: torch.Tensor, ksize: int, n_out_cap: Optional[int] = None, out_cap: Optional[int] = None,
                       err_flags=None, stream=None):
    """(out_coords [capacity n_out_cap, default n_in * ksize^ndim], n_out
    device scalar, out table of out_cap block slots, default
    generative_table_capacity(n_in))."""
    n, ndim = coords.shape[0], coords.shape[1] - 1
    if n_out_cap is None:
        n_out_cap = n * ksize ** ndim
    out = torch.zeros((n_out_cap, ndim + 1), dtype=torch.int32, device=coords.device)
    n_out = torch.zeros(1, dtype=torch.int64, device=coords.device)
    table = HashTable.with_capacity(ndim, generative_table_capacity(n) if out_cap is None else out_cap, coords.device)
    scratch = _bytes(ts_generative_scratch_bytes(n, ndim, ksize), coords.device)
    ts_generative_support(coords, ksize, out, n_out, table.buf, table.cap, scratch, err_flags, stream)
    return out, n_out, table


def transposed_support(coords: torch.Tensor, ksize: int, stride: int, n_out_cap: Optional[int] = None,
                       out_cap: Optional[int] = None, err_flags=None, stream=None):
    """(fine out_coords [capacity n_out_cap, default n_in * ksize^ndim], n_out
    device scalar, their table of out_cap block slots, default
    generative_table_capacity(n_in): the children of one input (k = s = 2)
    share one fine block)."""
    n, ndim = coords.shape[0], coords.shape[1] - 1
    if n_out_cap is None:
        n_out_cap = n * ksize ** ndim
    out = torch.zeros((n_out_cap, ndim + 1), dtype=torch.int32, device=coords.device)
    n_out = torch.zeros(1, dtype=torch.int64, device=coords.device)
    cap = generative_table_capacity(n) if out_cap is None else out_cap
    table = HashTable.with_capacity(ndim, cap, coords.device)
    scratch = _bytes(ts_generative_scratch_bytes(n, ndim, ksize), coords.device)
    ts_transposed_support(coords, ksize, stride, out, n_out, table.buf, table.cap, scratch, err_flags, stream)
    return out, n_out, table


def conv_transpose(kmap: Kmap, x: torch.Tensor, w: torch.Tensor, out_dtype=None, dataflow=TS_DATAFLOW_AUTO, ws=None,
                   stream=None) -> torch.Tensor:
    """ConvTranspose over the map's relation: y on the map's input rows."""
    out_dtype = out_dtype or x.dtype
    y = torch.empty((kmap.s.n_in, w.shape[2]), dtype=out_dtype, device=x.device)
    if ws is None:
        ws = workspace(kmap, w.shape[1], w.shape[2], TS_OP_TRANSPOSE, x.dtype, dataflow)
    ts_conv_transpose_fwd(kmap.s, x, w, y, dataflow, ws, stream)
    return y


def pool(kmap: Kmap, x: torch.Tensor, mode: int = TS_POOL_MAX, out_dtype=None, stream=None) -> torch.Tensor:
    """Max / average pooling over the map: y on the map's output rows."""
    y = torch.empty((kmap.s.n_out_cap, x.shape[1]), dtype=out_dtype or x.dtype, device=x.device)
    ts_pool_fwd(kmap.s, x, y, mode, stream)
    return y


def voxelize(pos: torch.Tensor, size, origin, feats: Optional[torch.Tensor] = None,
             batch: Optional[torch.Tensor] = None, rsv_ratio: float = 2.0, err_flags=None, stream=None):
    """(voxel coords [capacity n], n_out device scalar, voxel table, vox_of [n],
    mean features [capacity n] or None)."""
    n, ndim = pos.shape
    out = torch.zeros((max(n, 1), ndim + 1), dtype=torch.int32, device=pos.device)
    n_out = torch.zeros(1, dtype=torch.int64, device=pos.device)
    table = HashTable.with_capacity(ndim, ts_hash_capacity(n, rsv_ratio), pos.device)
    vox_of = torch.empty(max(n, 1), dtype=torch.int32, device=pos.device)
    of = None if feats is None else torch.empty((max(n, 1), feats.shape[1]), dtype=torch.float32, device=pos.device)
    scratch = _bytes(ts_voxelize_scratch_bytes(n), pos.device)
    ts_voxelize(batch, pos, size, origin, feats, out, n_out, table.buf, table.cap, vox_of, of, scratch, err_flags,
                stream)
    return out, n_out, table, vox_of[:n], of


def workspace(kmap: Kmap, cin: int, cout: int, op: int, dtype: torch.dtype, dataflow: int = TS_DATAFLOW_AUTO):
    n = ts_conv_workspace_bytes(kmap.s, cin, cout, op, _DT[dtype], dataflow)
    return _bytes(n, kmap.buf.device) if n > 0 else None


def conv_fwd(kmap: Kmap, x: torch.Tensor, w: torch.Tensor, out_dtype=None, dataflow=TS_DATAFLOW_AUTO, ws=None,
             stream=None) -> torch.Tensor:
    out_dtype = out_dtype or x.dtype
    y = torch.empty((kmap.s.n_out_cap, w.shape[2]), dtype=out_dtype, device=x.device)
    if ws is None:
        ws = workspace(kmap, w.shape[1], w.shape[2], TS_OP_FWD, x.dtype, dataflow)
    ts_conv_fwd(kmap.s, x, w, y, dataflow, ws, stream, subm=kmap.s.stride == 1 and not kmap.s.flags & TS_KMAP_TARGET)
    return y


def conv_dgrad(kmap: Kmap, dy: torch.Tensor, w: torch.Tensor, out_dtype=None, dataflow=TS_DATAFLOW_AUTO, ws=None,
               stream=None) -> torch.Tensor:
    out_dtype = out_dtype or dy.dtype
    dx = torch.empty((kmap.s.n_in, w.shape[1]), dtype=out_dtype, device=dy.device)
    if ws is None:
        ws = workspace(kmap, w.shape[1], w.shape[2], TS_OP_DGRAD, dy.dtype, dataflow)
    ts_conv_bwd_dgrad(kmap.s, dy, w, dx, dataflow, ws, stream)
    return dx


def conv_wgrad(kmap: Kmap, x: torch.Tensor, dy: torch.Tensor, ws=None, stream=None) -> torch.Tensor:
    dw = torch.empty((kmap.kvol, x.shape[1], dy.shape[1]), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(kmap, x.shape[1], dy.shape[1], TS_OP_WGRAD, x.dtype)
    ts_conv_bwd_wgrad(kmap.s, x, dy, dw, ws, stream)
    return dw


# ---------------------------------------------------------------- voxel-transformer operators
# These calls are short, so they check their tensors in one pass and hand plain
# addresses to the library.  A call on another stream runs with that stream as
# the current one, so that its buffers come from that stream's pool (a freed
# workspace is not handed out while the call still runs).
def _need(ok: bool, what: str) -> None:
    if not ok:
        raise TsError(TS_ERR_INVALID_ARG, what)


def _raw_stream(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """Rows of heads the library can take: dense copies of misaligned ones,
    unless their width or stride (the one it is told: that of a single row is
    its width) makes the library copy them itself."""
    if t.data_ptr() % 16 == 0 or t.shape[-1] % 8 or (_row_stride(t) or 0) % 8:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _flag_ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    _need(t.is_cuda and t.element_size() == 4 and t.numel() >= 1, "err_flags is a 32-bit device word")
    return t.data_ptr()


def attn_args(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
              k_starts: Optional[torch.Tensor] = None, scale: Optional[float] = None, cap: float = 0.0,
              slopes: Optional[torch.Tensor] = None, q_coords: Optional[torch.Tensor] = None,
              k_coords: Optional[torch.Tensor] = None, o_stride: Optional[int] = None) -> TsAttn:
    """The C description of an attention call, its tensors checked against
    each other.  scale defaults to 1 / sqrt(d); o_stride to dense rows."""
    qst, kst, vst = _row_stride(q), _row_stride(k), _row_stride(v)
    _need(qst is not None and kst is not None and vst is not None and q.is_cuda and k.is_cuda and v.is_cuda,
          "attention: q, k, v are device tensors [n][heads][d] with adjacent heads")
    nq, hq, d = q.shape
    nk, hk, dk = k.shape
    dtype = q.dtype
    _need(dk == d and v.shape == k.shape and k.dtype is dtype and v.dtype is dtype and dtype in _DT,
          "attention: q, k, v differ in width, type or keys")
    n_sets = q_starts.numel() - 1
    _need(n_sets >= 0 and q_starts.dtype is torch.int64 and q_starts.is_cuda and q_starts.is_contiguous(),
          "attention: starts are int64 [n_sets + 1]")
    if k_starts is not None:
        _need(k_starts.numel() - 1 == n_sets and k_starts.dtype is torch.int64 and k_starts.is_cuda
              and k_starts.is_contiguous(), "attention: starts are int64 [n_sets + 1]")
    ndim = 3
    if slopes is not None:
        _need(slopes.is_cuda and slopes.dtype is torch.float32 and slopes.is_contiguous() and slopes.numel() == hq,
              "attention: slopes are float32 [hq]")
        _need(q_coords is not None and q_coords.dim() == 2, "attention: slopes need coordinates")
        ndim = q_coords.shape[1] - 1
        for c, n in ((q_coords, nq), (q_coords if k_coords is None else k_coords, nk)):
            _need(c.is_cuda and c.dtype is torch.int32 and c.is_contiguous() and c.shape == (n, ndim + 1),
                  "attention: coordinates are int32 [n][ndim + 1]")
    else:
        q_coords = k_coords = None
    return TsAttn(_DT[dtype], hq, hk, d, ndim, 1.0 / d ** 0.5 if scale is None else scale, cap, nq, nk, n_sets, qst, kst,
                  vst, hq * d if o_stride is None else o_stride, q_starts.data_ptr(), _ptr(k_starts), _ptr(slopes),
                  _ptr(q_coords), _ptr(k_coords))


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
             k_starts: Optional[torch.Tensor] = None, scale: Optional[float] = None, cap: float = 0.0,
             slopes: Optional[torch.Tensor] = None, q_coords: Optional[torch.Tensor] = None,
             k_coords: Optional[torch.Tensor] = None, err_flags: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out [nq][hq][d], lse [nq][hq]): attention of each packed set's rows
    over its own keys (see ts_attn in ts.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return attn_fwd(q, k, v, q_starts, k_starts, scale, cap, slopes, q_coords, k_coords, err_flags)
    q, k, v = _aligned(q), _aligned(k), _aligned(v)
    at = attn_args(q, k, v, q_starts, k_starts, scale, cap, slopes, q_coords, k_coords)
    ref, dev = ctypes.byref(at), q.device
    out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty((at.nq, at.hq), dtype=torch.float32, device=dev)
    n = _lib_attn_workspace_bytes(ref, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    _check(_lib_attn_fwd(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), _ptr(ws), n,
                         _flag_ptr(err_flags), _raw_stream(q)), "ts_attn_fwd")
    return out, lse


def _laid_out_like(*tensors: torch.Tensor) -> list:
    """New tensors [n][heads][d] with the rows of the given ones; columns of one
    matrix where those are."""
    new, groups = [None] * len(tensors), {}
    for i, t in enumerate(tensors):
        n, h, d = t.shape
        if n < 2 or t.stride(0) == h * d:
            new[i] = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)
        else:
            groups.setdefault((n, t.stride(0), t.untyped_storage().data_ptr()), []).append((t.storage_offset(), i))
    for (n, stride, _), columns in groups.items():
        columns.sort()
        while columns:
            # as many as follow each other within a row
            first, _ = columns[0]
            end, taken = first, 0
            for at, i in columns:
                width = tensors[i].shape[1] * tensors[i].shape[2]
                if at < end or at + width > first + stride:
                    break
                end, taken = at + width, taken + 1
            t = tensors[columns[0][1]]
            whole = torch.empty((n - 1) * stride + end - first, dtype=t.dtype, device=t.device)
            for at, i in columns[:taken]:
                new[i] = whole.as_strided(tensors[i].shape, tensors[i].stride(), at - first)
            columns = columns[taken:]
    return new


def attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
             lse: torch.Tensor, q_starts: torch.Tensor, k_starts: Optional[torch.Tensor] = None,
             scale: Optional[float] = None, cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
             q_coords: Optional[torch.Tensor] = None, k_coords: Optional[torch.Tensor] = None,
             err_flags: Optional[torch.Tensor] = None, stream=None,
             into: Optional[Sequence[torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv) of attn_fwd with the same arguments, laid out like q, k, v:
    where those are columns of one matrix, so are the gradients.  They are
    written to the three tensors of `into`, or to new ones."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return attn_bwd(dout, q, k, v, out, lse, q_starts, k_starts, scale, cap, slopes, q_coords, k_coords, err_flags,
                            into=into)
    _need(out.shape == q.shape and dout.shape == q.shape and out.dtype is q.dtype and dout.dtype is q.dtype
          and out.is_cuda and dout.is_cuda, "attention: out and dout are like q")
    _need(lse.dtype is torch.float32 and lse.is_cuda and lse.is_contiguous() and lse.shape == q.shape[:2],
          "attention: lse is float32 [nq][hq]")
    like = (q, k, v)
    q, k, v, out, dout = (_aligned(t) for t in (q, k, v, out, dout))
    st = _row_stride(out)
    if st is None or _row_stride(dout) != st:
        dout, out = dout.contiguous(), out.contiguous()
        st = _row_stride(out)
    at = attn_args(q, k, v, q_starts, k_starts, scale, cap, slopes, q_coords, k_coords, st)
    ref = ctypes.byref(at)
    _need(into is None or (len(into) == 3 and all(
        g.is_cuda and g.dtype is t.dtype and g.shape == t.shape and g.stride() == t.stride()
        for g, t in zip(into, like))), "attention: dq, dk, dv are laid out like q, k, v")
    # their own buffers where q, k or v was copied or the library could not write there
    direct = into is not None and all(_aligned(g) is g and t is l for g, t, l in zip(into, (q, k, v), like))
    dq, dk, dv = into if direct else _laid_out_like(q, k, v)
    n = _lib_attn_workspace_bytes(ref, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    _check(_lib_attn_bwd(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ws), n, _flag_ptr(err_flags),
                         _raw_stream(q)), "ts_attn_bwd")
    if into is not None and not direct:
        for g, t in zip(into, (dq, dk, dv)):
            g.copy_(t)
        return tuple(into)
    return dq, dk, dv


class Act8(NamedTuple):
    """Activations in 8 bits: codes int8 [n][c], scales uint8 [n][ceil(c / 32)]."""
    codes: torch.Tensor
    scales: torch.Tensor

    @classmethod
    def empty(cls, n: int, c: int, device) -> "Act8":
        return cls(torch.empty((n, c), dtype=torch.int8, device=device),
                   torch.empty((n, -(-c // TS_ACT8_BLOCK)), dtype=torch.uint8, device=device))

    def check(self, n: int, c: int) -> None:
        a, s = self.codes, self.scales
        _need(a.dtype is torch.int8 and s.dtype is torch.uint8 and a.is_cuda and s.is_cuda and a.is_contiguous()
              and s.is_contiguous() and a.shape == (n, c) and s.shape == (n, -(-c // TS_ACT8_BLOCK)),
              "8-bit activations of [n][c]: codes int8 [n][c], scales uint8 [n][ceil(c / 32)]")


def _matrix(t: torch.Tensor, what: str, shape=None, dtype=None) -> None:
    _need(t.is_cuda and t.dim() == 2 and t.is_contiguous() and t.dtype in _DT and (shape is None or t.shape == shape)
          and (dtype is None or t.dtype is dtype), what)


def act_pack(x: torch.Tensor, stream=None) -> Act8:
    """x [n][c] in 8 bits (see ts_act8 in ts.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return act_pack(x)
    _matrix(x, "act_pack: a dense device matrix [n][c]")
    n, c = x.shape
    a = Act8.empty(n, c, x.device)
    _check(_lib_act_pack(x.data_ptr(), n, c, _DT[x.dtype], _act(a), _raw_stream(x)), "ts_act_pack")
    return a


def act_unpack(a: Act8, dtype: torch.dtype, stream=None) -> torch.Tensor:
    """The values `a` stands for, in `dtype`: exact in fp32, bf16 and the type they
    were packed from; in fp16 from another one rounded where its range ends."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return act_unpack(a, dtype)
    n, c = a.codes.shape
    a.check(n, c)
    _need(dtype in _DT, "act_unpack: a feature type")
    x = torch.empty((n, c), dtype=dtype, device=a.codes.device)
    _check(_lib_act_unpack(_act(a), n, c, x.data_ptr(), _DT[dtype], _raw_stream(x)), "ts_act_unpack")
    return x


def conv_wgrad_act8(kmap: Kmap, x: Act8, dy: torch.Tensor, stream=None) -> torch.Tensor:
    """conv_wgrad with the layer's input kept in 8 bits."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return conv_wgrad_act8(kmap, x, dy)
    cin = x.codes.shape[1]
    x.check(kmap.s.n_in, cin)
    _matrix(dy, "conv_wgrad_act8: dy is a dense device matrix [n_out][cout]")
    _need(dy.shape[0] >= kmap.s.n_out_cap, "conv_wgrad_act8: dy has the map's output rows")
    cout, ref = dy.shape[1], ctypes.byref(kmap.s)
    dw = torch.empty((kmap.kvol, cin, cout), dtype=torch.float32, device=dy.device)
    n = _lib_conv_wgrad_act8_workspace_bytes(ref, cin, cout)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dy.device)
    _check(_lib_conv_bwd_wgrad_act8(ref, _act(x), cin, dy.data_ptr(), cout, _DT[dy.dtype], dw.data_ptr(), ws.data_ptr(), n,
                                    _raw_stream(dy)), "ts_conv_bwd_wgrad_act8")
    return dw


class Norm(NamedTuple):
    """Results of norm_fwd: h (x itself without a residual), and those asked for."""
    h: torch.Tensor
    y: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]
    y8: Optional[Act8]
    h8: Optional[Act8]


def norm_fwd(x: torch.Tensor, w: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             want_y: bool = True, want_rstd: bool = True, y8: bool = False, h8: bool = False, stream=None) -> Norm:
    """Root-mean-square norm of x + residual (see ts_norm_fwd in ts.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return norm_fwd(x, w, residual, eps, want_y, want_rstd, y8, h8)
    _matrix(x, "norm_fwd: x is a dense device matrix [n][c]")
    n, c = x.shape
    if residual is not None:
        _matrix(residual, "norm_fwd: the residual is like x", x.shape, x.dtype)
    _need(w.is_cuda and w.dtype is torch.float32 and w.is_contiguous() and w.numel() == c, "norm_fwd: w is float32 [c]")
    h = None if residual is None else torch.empty_like(x)
    y = torch.empty_like(x) if want_y else None
    rstd = torch.empty(n, dtype=torch.float32, device=x.device) if want_rstd else None
    qy = Act8.empty(n, c, x.device) if y8 else None
    qh = Act8.empty(n, c, x.device) if h8 else None
    _check(_lib_norm_fwd(x.data_ptr(), _ptr(residual), w.data_ptr(), n, c, eps, _DT[x.dtype], _ptr(h), _ptr(y), _ptr(rstd),
                         _act(qy), _act(qh), _raw_stream(x)), "ts_norm_fwd")
    return Norm(x if h is None else h, y, rstd, qy, qh)


def norm_bwd(dy: torch.Tensor, h: Union[torch.Tensor, Act8], w: torch.Tensor, rstd: torch.Tensor,
             dh: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of norm_fwd from h or its 8-bit form; dx is also the residual's
    gradient, dh the gradient that reaches h past the norm."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return norm_bwd(dy, h, w, rstd, dh)
    _matrix(dy, "norm_bwd: dy is a dense device matrix [n][c]")
    n, c = dy.shape
    eight = isinstance(h, Act8)
    if eight:
        h.check(n, c)
    else:
        _matrix(h, "norm_bwd: h is like dy", dy.shape, dy.dtype)
    if dh is not None:
        _matrix(dh, "norm_bwd: dh is like dy", dy.shape, dy.dtype)
    for t, m in ((w, c), (rstd, n)):
        _need(t.is_cuda and t.dtype is torch.float32 and t.is_contiguous() and t.numel() == m,
              "norm_bwd: w is float32 [c], rstd float32 [n]")
    dx = torch.empty_like(dy)
    dw = torch.empty(c, dtype=torch.float32, device=dy.device)
    size = _lib_norm_workspace_bytes(n, c)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=dy.device)
    _check(_lib_norm_bwd(dy.data_ptr(), None if eight else h.data_ptr(), _act(h) if eight else None, w.data_ptr(),
                         rstd.data_ptr(), _ptr(dh), n, c, _DT[dy.dtype], dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), size,
                         _raw_stream(dy)), "ts_norm_bwd")
    return dx, dw


# ---------------------------------------------------------------- the rest of a voxel-transformer layer
def rope_freqs(pairs: Sequence[int], base: float = 100.0, device="cuda") -> torch.Tensor:
    """Frequencies for `pairs` channel pairs of each axis: base^(-i / m) radians a
    voxel for pair i of an axis with m."""
    return torch.cat([base ** (-torch.arange(m, dtype=torch.float64) / max(m, 1)) for m in pairs]).float().to(device)


_I3 = ctypes.c_int32 * 3


def _rope_args(like: torch.Tensor, coords: Optional[torch.Tensor], freqs: Optional[torch.Tensor], pairs: Sequence[int],
               eps: float, interleaved: bool) -> TsRope:
    n, _, d = like.shape
    pairs = tuple(pairs)
    _need(len(pairs) in (2, 3) and min(pairs) >= 0, "rope: pairs are the channel pairs of 2 or 3 axes")
    turned = sum(pairs)
    if turned > 0:
        _need(coords is not None and coords.is_cuda and coords.dtype is torch.int32 and coords.is_contiguous()
              and coords.shape == (n, len(pairs) + 1), "rope: coordinates are int32 [n][ndim + 1]")
        _need(freqs is not None and freqs.is_cuda and freqs.dtype is torch.float32 and freqs.is_contiguous()
              and freqs.numel() == turned, "rope: freqs are float32, one for each pair")
    else:
        coords = freqs = None
    _need(like.dtype in _DT, "rope: a feature type")
    return TsRope(_DT[like.dtype], d, len(pairs), _I3(*pairs), int(interleaved), eps, n, _ptr(coords), _ptr(freqs))


def _rope_rows(t: torch.Tensor, like: torch.Tensor, shape: Tuple[int, int, int], what: str) -> int:
    """_row_stride of a tensor of this shape and of like's type."""
    _need(t.shape == shape and t.dtype is like.dtype and t.is_cuda, what)
    n, h, d = shape
    row, head, one = t.stride()
    _need((one == 1 or d <= 1) and (head == d or h <= 1) and (row >= h * d or n <= 1), what)
    return row if n > 1 else h * d


def _rope_weight(w: Optional[torch.Tensor], d: int) -> None:
    _need(w is None or (w.is_cuda and w.dtype is torch.float32 and w.is_contiguous() and w.numel() == d),
          "rope: the norm's weights are float32 [d]")


def rope_fwd(q: torch.Tensor, k: Optional[torch.Tensor], coords: Optional[torch.Tensor], freqs: Optional[torch.Tensor],
             pairs: Sequence[int], wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
             interleaved: bool = False, into: Optional[Sequence[Optional[torch.Tensor]]] = None,
             stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Queries [n][hq][d] and keys [n][hk][d] (or None) of the same voxels, normalised
    where a weight is given and turned by their positions (see ts_rope in ts.h).  Written
    to the two tensors of `into`, which may be q and k themselves, or to new ones."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rope_fwd(q, k, coords, freqs, pairs, wq, wk, eps, interleaved, into)
    _need(q.dim() == 3, "rope: q is [n][heads][d]")
    args = _rope_args(q, coords, freqs, pairs, eps, interleaved)
    _need(into is None or len(into) == 2, "rope: results for q and k")
    yq, yk = into or (None, None)
    yq, side_q = _rope_fwd_side(q, q, wq, yq, into is None)
    yk, side_k = _rope_fwd_side(k, q, wk, yk, into is None)
    _check(_lib_rope_fwd(ctypes.byref(args), side_q, side_k, _raw_stream(q)), "ts_rope_fwd")
    return yq, yk


def _rope_fwd_side(x, q, w, y, new):
    if x is None:
        _need(y is None, "rope: a result without its input")
        return None, None
    _need(x.dim() == 3, "rope: k is [n][heads][d]")
    n, _, d = q.shape
    h = x.shape[1]
    st = _rope_rows(x, q, (n, h, d), "rope: q and k are device tensors [n][heads][d] of one type, with adjacent heads")
    _rope_weight(w, d)
    if new:
        y, yst = torch.empty((n, h, d), dtype=q.dtype, device=q.device), h * d
    else:
        _need(y is not None, "rope: results for q and k")
        yst = _rope_rows(y, q, (n, h, d), "rope: results are like q and k")
    return y, ctypes.byref(TsRopeHeads(h, st, yst, 0, 0, x.data_ptr(), _ptr(w), y.data_ptr()))


class RopeGrads(NamedTuple):
    """Gradients of rope_fwd's q, k, wq and wk (None where there is none)."""
    dq: torch.Tensor
    dk: Optional[torch.Tensor]
    dwq: Optional[torch.Tensor]
    dwk: Optional[torch.Tensor]


def rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
             coords: Optional[torch.Tensor], freqs: Optional[torch.Tensor], pairs: Sequence[int],
             wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
             into: Optional[Sequence[Optional[torch.Tensor]]] = None, stream=None) -> RopeGrads:
    """Gradients from those of rope_fwd's results and its inputs.  Written to the two
    tensors of `into`, which may be dq and dk themselves, or to new ones."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq, wk, eps, interleaved, into)
    _need(q.dim() == 3 and (dk is None) == (k is None), "rope: q is [n][heads][d], dk comes with k")
    args = ctypes.byref(_rope_args(q, coords, freqs, pairs, eps, interleaved))
    _need(into is None or len(into) == 2, "rope: results for q and k")
    yq, yk = into or (None, None)
    yq, dwq, side_q = _rope_bwd_side(dq, q, q, wq, yq, into is None)
    yk, dwk, side_k = _rope_bwd_side(dk, k, q, wk, yk, into is None)
    n = _lib_rope_workspace_bytes(args, q.shape[1], 0 if k is None else k.shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    _check(_lib_rope_bwd(args, side_q, side_k, _ptr(ws), n, _raw_stream(q)), "ts_rope_bwd")
    return RopeGrads(yq, yk, dwq, dwk)


def _rope_bwd_side(g, x, q, w, y, new):
    if x is None:
        _need(y is None, "rope: a result without its input")
        return None, None, None
    what = "rope: q, k and their gradients are device tensors [n][heads][d] of one type, with adjacent heads"
    _need(x.dim() == 3, what)
    n, _, d = q.shape
    h = x.shape[1]
    st, gst = _rope_rows(x, q, (n, h, d), what), _rope_rows(g, q, (n, h, d), what)
    _rope_weight(w, d)
    if new:
        y, yst = torch.empty((n, h, d), dtype=q.dtype, device=q.device), h * d
    else:
        _need(y is not None, "rope: results for q and k")
        yst = _rope_rows(y, q, (n, h, d), "rope: results are like q and k")
    # (a call without any heads launches nothing)
    dw = None if w is None else (torch.empty if h else torch.zeros)(d, dtype=torch.float32, device=q.device)
    return y, dw, ctypes.byref(TsRopeHeads(h, st, 0, gst, yst, x.data_ptr(), _ptr(w), None, g.data_ptr(), y.data_ptr(), _ptr(dw)))


class Route(NamedTuple):
    """What route_fwd returns: experts int32 and gates float32 [n][top]; the grouped rows'
    starts int64 [n_experts + 1] and rows int32 [n * top], and place int32 [n][top]."""
    experts: torch.Tensor
    gates: torch.Tensor
    starts: torch.Tensor
    rows: torch.Tensor
    place: torch.Tensor


def route_fwd(logits: torch.Tensor, top: int, over_all: bool = False, stream=None) -> Route:
    """Each row's `top` experts, their gates, and the pairs grouped by expert (see
    ts_route_fwd in ts.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route_fwd(logits, top, over_all)
    _matrix(logits, "route_fwd: logits are a dense device matrix [n][experts]")
    n, e = logits.shape
    _need(1 <= top <= e, "route_fwd: 1 <= top <= experts")
    dev = logits.device
    experts = torch.empty((n, top), dtype=torch.int32, device=dev)
    rows, place = torch.empty(n * top, dtype=torch.int32, device=dev), torch.empty_like(experts)
    gates = torch.empty((n, top), dtype=torch.float32, device=dev)
    starts = torch.empty(e + 1, dtype=torch.int64, device=dev)
    size = _lib_route_workspace_bytes(n, e, top)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _check(_lib_route_fwd(logits.data_ptr(), n, e, _DT[logits.dtype], top, int(over_all), experts.data_ptr(), gates.data_ptr(),
                          starts.data_ptr(), rows.data_ptr(), place.data_ptr(), _ptr(ws), size, _raw_stream(logits)), "ts_route_fwd")
    return Route(experts, gates, starts, rows, place)


def route_bwd(dgates: torch.Tensor, logits: torch.Tensor, route: Route, over_all: bool = False, stream=None) -> torch.Tensor:
    """Gradient of the logits from that of the gates."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route_bwd(dgates, logits, route, over_all)
    _matrix(logits, "route_bwd: logits are a dense device matrix [n][experts]")
    n, e = logits.shape
    top = route.experts.shape[1]
    for t, dt in ((dgates, torch.float32), (route.gates, torch.float32), (route.experts, torch.int32)):
        _need(t.is_cuda and t.dtype is dt and t.is_contiguous() and t.shape == (n, top), "route_bwd: gates, gradients, experts [n][top]")
    d = torch.empty_like(logits)
    _check(_lib_route_bwd(dgates.data_ptr(), logits.data_ptr(), route.experts.data_ptr(), route.gates.data_ptr(), n, e,
                          _DT[logits.dtype], top, int(over_all), d.data_ptr(), _raw_stream(logits)), "ts_route_bwd")
    return d


class Groups(NamedTuple):
    """Grouped rows (see ts_groups in ts.h): starts int64 [groups + 1], and int32 rows of x they
    read (None: grouped row p is row p)."""
    starts: torch.Tensor
    rows: Optional[torch.Tensor] = None


def _groups(g: Groups, x: Optional[torch.Tensor], n_rows: int) -> TsGroups:
    """Of n_rows grouped rows that read x (None: they read nothing by `rows`)."""
    starts, rows = g.starts, g.rows
    _need(starts.is_cuda and starts.dtype is torch.int64 and starts.is_contiguous() and starts.dim() == 1 and starts.numel() >= 2,
          "groups: starts are int64 [groups + 1]")
    _need(rows is None or (rows.is_cuda and rows.dtype is torch.int32 and rows.is_contiguous() and rows.shape == (n_rows,)),
          "groups: rows are int32, one for each grouped row")
    _need(x is None or rows is not None or x.shape[0] == n_rows, "groups: x has the grouped rows")
    return TsGroups(starts.numel() - 1, n_rows, starts.data_ptr(), _ptr(rows), 0 if x is None else x.shape[0])


def _experts(w: torch.Tensor, groups: TsGroups, cin: int, cout: Optional[int], like: torch.Tensor) -> None:
    _need(w.is_cuda and w.dim() == 3 and w.is_contiguous() and w.dtype is like.dtype and w.shape[:2] == (groups.n_groups, cin)
          and cout in (None, w.shape[2]), "groups: weights are a dense device tensor [groups][cin][cout]")


def _group_fwd(x, w, groups, glu, want_h, err_flags):
    _matrix(x, "group_fwd: x is a dense device matrix [n][cin]")
    p, (n, cin), dev = x.shape[0] if groups.rows is None else groups.rows.numel(), x.shape, x.device
    g = _groups(groups, x, p)
    _experts(w, g, cin, None, x)
    wide = w.shape[2]
    _need(not glu or wide % 2 == 0, "group_glu_fwd: weights have two columns for each result")
    cout = wide // 2 if glu else wide
    y = torch.empty((p, cout), dtype=x.dtype, device=dev)
    h = torch.empty((p, wide), dtype=x.dtype, device=dev) if want_h else None
    _check(_lib_group_fwd(ctypes.byref(g), x.data_ptr(), cin, w.data_ptr(), cout, _DT[x.dtype], int(glu), y.data_ptr(), _ptr(h),
                          _flag_ptr(err_flags), _raw_stream(x)), "ts_group_fwd")
    return y, h


def group_fwd(x: torch.Tensor, w: torch.Tensor, groups: Groups, err_flags: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """y[p] = x[rows[p]] w[e] for the grouped rows p of each group e (see ts_groups in ts.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_fwd(x, w, groups, err_flags)
    return _group_fwd(x, w, groups, False, False, err_flags)[0]


def group_glu_fwd(x: torch.Tensor, w: torch.Tensor, groups: Groups, want_h: bool = False,
                  err_flags: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(silu(a) b, h): a and b are the first and the last half of the columns of group_fwd, and h is
    both, for the backward pass (None unless want_h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_glu_fwd(x, w, groups, want_h, err_flags)
    return _group_fwd(x, w, groups, True, want_h, err_flags)


def _group_dgrad(dy, w, h, groups, err_flags, into=None):
    _matrix(dy, "group_dgrad: dy is a dense device matrix [grouped rows][cout]")
    p, cout = dy.shape
    g = _groups(Groups(groups.starts), None, p)
    _need(w.dim() == 3, "groups: weights are a dense device tensor [groups][cin][cout]")
    cin = w.shape[1]
    _experts(w, g, cin, cout, dy)
    if h is not None:
        _matrix(h, "group_glu_dgrad: h is what group_glu_fwd returned", (p, 2 * cin), dy.dtype)
    dx = torch.empty((p, cin if h is None else 2 * cin), dtype=dy.dtype, device=dy.device) if into is None else into
    if into is not None:
        _matrix(into, "group_glu_dgrad: the result is like h", (p, 2 * cin), dy.dtype)
    _check(_lib_group_bwd_dgrad(ctypes.byref(g), dy.data_ptr(), cout, w.data_ptr(), cin, _DT[dy.dtype], _ptr(h), dx.data_ptr(),
                                _flag_ptr(err_flags), _raw_stream(dy)), "ts_group_bwd_dgrad")
    return dx


def group_dgrad(dy: torch.Tensor, w: torch.Tensor, groups: Groups, err_flags: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Gradient of what each grouped row read; where rows of x are read by several, combine_fwd
    without gates adds them up."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_dgrad(dy, w, groups, err_flags)
    return _group_dgrad(dy, w, None, groups, err_flags)


def group_glu_dgrad(dy: torch.Tensor, w: torch.Tensor, h: torch.Tensor, groups: Groups, err_flags: Optional[torch.Tensor] = None,
                    into: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of h = (a, b), from that of the product with w that silu(a) b went into; written
    to `into` (which may be h) or to a new matrix."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_glu_dgrad(dy, w, h, groups, err_flags, into)
    return _group_dgrad(dy, w, h, groups, err_flags, into)


def group_wgrad(x: torch.Tensor, dy: torch.Tensor, groups: Groups, err_flags: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """float32 gradient of the weights [groups][cin][cout] from x and the gradient of group_fwd's result."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_wgrad(x, dy, groups, err_flags)
    _matrix(x, "group_wgrad: x is a dense device matrix [n][cin]")
    _matrix(dy, "group_wgrad: dy is a dense device matrix [grouped rows][cout]", dtype=x.dtype)
    p, cout = dy.shape
    g, cin = _groups(groups, x, p), x.shape[1]
    ref = ctypes.byref(g)
    dw = torch.empty((g.n_groups, cin, cout), dtype=torch.float32, device=x.device)
    size = _lib_group_wgrad_workspace_bytes(ref, cin, cout)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=x.device)
    _check(_lib_group_bwd_wgrad(ref, x.data_ptr(), cin, dy.data_ptr(), cout, _DT[x.dtype], dw.data_ptr(), ws.data_ptr(), size,
                                _flag_ptr(err_flags), _raw_stream(x)), "ts_group_bwd_wgrad")
    return dw


def _place(place: torch.Tensor, gates: Optional[torch.Tensor]) -> None:
    _need(place.is_cuda and place.dtype is torch.int32 and place.dim() == 2 and place.is_contiguous(), "combine: place is int32 [n][top]")
    _need(gates is None or (gates.is_cuda and gates.dtype is torch.float32 and gates.is_contiguous() and gates.shape == place.shape),
          "combine: gates are float32 [n][top]")


def combine_fwd(y: torch.Tensor, place: torch.Tensor, gates: Optional[torch.Tensor] = None,
                err_flags: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum over j of gates[t][j] y[place[t][j]] (see ts_combine_fwd in ts.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return combine_fwd(y, place, gates, err_flags)
    _matrix(y, "combine: y is a dense device matrix of grouped rows")
    _place(place, gates)
    (p, c), (n, top) = y.shape, place.shape
    out = torch.empty((n, c), dtype=y.dtype, device=y.device)
    _check(_lib_combine_fwd(y.data_ptr(), p, place.data_ptr(), _ptr(gates), n, top, c, _DT[y.dtype], out.data_ptr(),
                            _flag_ptr(err_flags), _raw_stream(y)), "ts_combine_fwd")
    return out


def combine_bwd(dout: torch.Tensor, y: torch.Tensor, place: torch.Tensor, gates: torch.Tensor,
                err_flags: Optional[torch.Tensor] = None, into: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dy, dgates) of combine_fwd; dy is written to `into` (which may be y, if no two places
    name the same row) or to a new matrix, whose rows that no place names are not written."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return combine_bwd(dout, y, place, gates, err_flags, into)
    _matrix(y, "combine: y is a dense device matrix of grouped rows")
    _place(place, gates)
    (p, c), (n, top) = y.shape, place.shape
    _matrix(dout, "combine: dout is like the result", (n, c), y.dtype)
    dy = torch.empty_like(y) if into is None else into
    _matrix(dy, "combine: dy is like y", y.shape, y.dtype)
    dgates = torch.empty((n, top), dtype=torch.float32, device=y.device)
    _check(_lib_combine_bwd(dout.data_ptr(), y.data_ptr(), p, place.data_ptr(), gates.data_ptr(), n, top, c, _DT[y.dtype],
                            dy.data_ptr(), dgates.data_ptr(), _flag_ptr(err_flags), _raw_stream(y)), "ts_combine_bwd")
    return dy, dgates
