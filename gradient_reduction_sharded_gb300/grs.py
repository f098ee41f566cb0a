"""Thin ctypes binding of libgrs (include/grs.h), same names as the C ABI.

Argument marshalling only: device pointers are passed as Python ints
(e.g. ``tensor.data_ptr()``) and streams as ``torch.cuda.Stream.cuda_stream``
ints.  Every computation happens in libgrs's CUDA kernels; if the library
is missing this module raises at import time — there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
# GRS_LIBRARY may name another build of the same library (e.g. a variant
# compiled with different tile constants); default: the in-tree build.
LIB_PATH = os.environ.get("GRS_LIBRARY") or os.path.join(_HERE, "libgrs.so")

GRS_REPLICA_AVG, GRS_PARTIAL_SUM, GRS_LOCAL_SHARD, GRS_ALREADY_REDUCED = 0, 1, 2, 3
GRS_OK = 0
GRS_ERR_INVALID_ARG = 1
GRS_ERR_UNSUPPORTED_COMPOSITION = 2
GRS_ERR_SHAPE = 3
GRS_ERR_ALIGNMENT = 4
GRS_ERR_CUDA = 5
GRS_ERR_TIMEOUT = 6
GRS_ERR_NONFINITE = 7
GRS_ERR_NO_DEVICE = 8
GRS_ERR_BOUNDS = 9
GRS_FEATURE_CHECKED = 1
GRS_PLAN_HOST_ONLY = 1
GRS_PLAN_FP32_GRADS = 2
GRS_TENSOR_FROZEN = 1
GRS_MAX_WORLD = 128
GRS_NOALLOC_SCRATCH_BYTES = 4 << 20
GRS_SMALL_MAX_TILES = 128
GRS_SMALL_MAX_BUFFERS = 256
GRS_DTYPE_BF16, GRS_DTYPE_FP32 = 0, 1
GRS_STATE_BLOCK = 256
GRS_MOE_MAX_EXPERTS = 1024
GRS_MAX_WIDTH = 1 << 30
GRS_QK_MAX_DIM = 1024
GRS_MAX_ROWS = (1 << 31) - (1 << 16)
GRS_MAX_ELEMENTS = 1 << 40

STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED_COMPOSITION", 3: "SHAPE",
                4: "ALIGNMENT", 5: "CUDA", 6: "TIMEOUT", 7: "NONFINITE", 8: "NO_DEVICE",
                9: "BOUNDS"}


class GrsError(RuntimeError):
    def __init__(self, status: int, func: str, msg: str):
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class grs_plan_info(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int32), ("n_buckets", ctypes.c_int32),
                ("world", ctypes.c_int32), ("tp", ctypes.c_int32),
                ("dp_replicate", ctypes.c_int32), ("dp_shard", ctypes.c_int32),
                ("dp", ctypes.c_int32), ("device", ctypes.c_int32),
                ("n_unique", ctypes.c_int64), ("n_rank_pad", ctypes.c_int64),
                ("n_state_pad", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("n_reduce_tiles", ctypes.c_int64), ("grad_bytes", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class grs_bucket_desc(ctypes.Structure):
    _fields_ = [("tag", ctypes.c_int32), ("copies", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("n_tensors", ctypes.c_int32),
                ("used", ctypes.c_int64), ("padded", ctypes.c_int64),
                ("shard_len", ctypes.c_int64), ("rank_offset", ctypes.c_int64),
                ("state_offset", ctypes.c_int64), ("n_segments", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class grs_segment_desc(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_int32), ("tp_index", ctypes.c_int32),
                ("bucket_offset", ctypes.c_int64), ("tensor_offset", ctypes.c_int64),
                ("numel", ctypes.c_int64), ("state_offset", ctypes.c_int64)]


class grs_tensor_desc(ctypes.Structure):
    _fields_ = [("bucket", ctypes.c_int32), ("owner", ctypes.c_int32),
                ("numel", ctypes.c_int64), ("per_rank", ctypes.c_int64),
                ("bucket_offset", ctypes.c_int64), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class grs_adamw(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("max_norm", ctypes.c_float), ("step", ctypes.c_int32),
                ("n_micro", ctypes.c_int32)]


class grs_tensors_info(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int32), ("device", ctypes.c_int32), ("n_elements", ctypes.c_int64),
                ("n_state", ctypes.c_int64), ("n_blocks", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]


class grs_norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("ld_dx", ctypes.c_int64), ("cols", ctypes.c_int32),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class grs_moe(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("top_k", ctypes.c_int32), ("expert_begin", ctypes.c_int32),
                ("expert_end", ctypes.c_int32), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class grs_experts(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("experts", ctypes.c_int32),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class grs_embedding(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("row_begin", ctypes.c_int32), ("row_end", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


class grs_qk_norm(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("ld_q", ctypes.c_int64), ("ld_k", ctypes.c_int64), ("ld_qo", ctypes.c_int64),
                ("ld_ko", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                      "(there is no CPU fallback)")
_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_P = ctypes.POINTER
_sig = {
    "grs_plan_create": ([_P(ctypes.c_int64), _P(ctypes.c_int32), ctypes.c_int32, ctypes.c_int32,
                         ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64,
                         ctypes.c_uint32, _P(_vp)], ctypes.c_int),
    "grs_plan_create_ex": ([_P(ctypes.c_int64), _P(ctypes.c_int32), _P(ctypes.c_uint32), ctypes.c_int32,
                            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                            ctypes.c_int64, ctypes.c_uint32, _P(_vp)], ctypes.c_int),
    "grs_plan_destroy": ([_vp], None),
    "grs_plan_shard_view": ([_vp, ctypes.c_int32, ctypes.c_int32, _P(_vp)], ctypes.c_int),
    "grs_plan_query": ([_vp, _P(grs_plan_info)], ctypes.c_int),
    "grs_bucket_info": ([_vp, ctypes.c_int32, _P(grs_bucket_desc)], ctypes.c_int),
    "grs_tensor_info": ([_vp, ctypes.c_int32, _P(grs_tensor_desc)], ctypes.c_int),
    "grs_segment_info": ([_vp, ctypes.c_int32, ctypes.c_int32, _P(grs_segment_desc)], ctypes.c_int),
    "grs_reduce_bucket": ([_vp, ctypes.c_int32, _P(_vp), _vp, ctypes.c_int32, ctypes.c_int32, _vp,
                           _vp], ctypes.c_int),
    "grs_reduce_all": ([_vp, _P(_vp), _vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp], ctypes.c_int),
    "grs_reduce_bucket_ex": ([_vp, ctypes.c_int32, _P(_vp), _vp, ctypes.c_int32, ctypes.c_int32, _vp,
                              ctypes.c_int32, _vp, _vp], ctypes.c_int),
    "grs_reduce_all_masked": ([_vp, _P(_vp), _vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp], ctypes.c_int),
    "grs_accumulate": ([_vp, ctypes.c_int32, _vp, _vp, _vp], ctypes.c_int),
    "grs_grad_norm_sq": ([_vp, _vp, ctypes.c_int32, _vp, ctypes.c_int32, _vp, _vp], ctypes.c_int),
    "grs_clip_adamw_step": ([_vp, _P(grs_adamw), _vp, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "grs_gather_params": ([_vp, _vp, _P(_vp), _vp], ctypes.c_int),
    "grs_clip_adamw_step_to_tensors": ([_vp, _P(grs_adamw), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
                                       ctypes.c_int),
    "grs_grad_norm_sq_masked": ([_vp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp], ctypes.c_int),
    "grs_clip_adamw_step_masked": ([_vp, _P(grs_adamw), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _vp], ctypes.c_int),
    "grs_check_device_errors": ([_vp, _vp], ctypes.c_int),
    "grs_selftest_bounded_wait": ([_vp, ctypes.c_int64, _vp], ctypes.c_int),
    "grs_check_already_reduced": ([_vp, _P(_vp), _vp], ctypes.c_int),
    "grs_state_to_logical": ([_vp, _vp, _vp, _vp], ctypes.c_int),
    "grs_state_from_logical": ([_vp, _vp, _vp, _vp], ctypes.c_int),
    "grs_grad_norm_sq_noalloc": ([_vp, _vp, ctypes.c_int32, _vp, _vp], ctypes.c_int),
    "grs_step_from_host": ([_vp, _P(grs_adamw), _P(_vp), _P(_vp), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                            _vp, _vp, _vp], ctypes.c_int),
    "grs_update_small": ([_vp, _P(grs_adamw), _P(_vp), _vp, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "grs_tensors_create": ([_P(ctypes.c_int64), ctypes.c_int32, ctypes.c_uint32, _P(_vp)], ctypes.c_int),
    "grs_tensors_destroy": ([_vp], None),
    "grs_tensors_query": ([_vp, _P(grs_tensors_info)], ctypes.c_int),
    "grs_tensors_offset": ([_vp, ctypes.c_int32, _P(ctypes.c_int64)], ctypes.c_int),
    "grs_tensors_norm_sq": ([_vp, _vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp], ctypes.c_int),
    "grs_tensors_adamw_step": ([_vp, _P(grs_adamw), _vp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "grs_tensors_adamw8_step": ([_vp, _P(grs_adamw), ctypes.c_uint64, _vp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp], ctypes.c_int),
    "grs_tensors_pack8": ([_vp] * 8, ctypes.c_int),
    "grs_tensors_unpack8": ([_vp] * 8, ctypes.c_int),
    "grs_tensors_check_device_errors": ([_vp, _vp], ctypes.c_int),
    "grs_layernorm_forward": ([_P(grs_norm)] + [_vp] * 7, ctypes.c_int),
    "grs_layernorm_backward": ([_P(grs_norm)] + [_vp] * 10, ctypes.c_int),
    "grs_layernorm_workspace_bytes": ([_P(grs_norm)], ctypes.c_int64),
    "grs_layernorm_check_device_errors": ([_vp], ctypes.c_int),
    "grs_selftest_layernorm_wait": ([_P(grs_norm)] + [_vp] * 9 + [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _vp], ctypes.c_int),
    "grs_moe_sort": ([_P(grs_moe)] + [_vp] * 6, ctypes.c_int),
    "grs_moe_workspace_bytes": ([_P(grs_moe)], ctypes.c_int64),
    "grs_moe_dispatch": ([_P(grs_moe)] + [_vp] * 4, ctypes.c_int),
    "grs_moe_dispatch_backward": ([_P(grs_moe)] + [_vp] * 4, ctypes.c_int),
    "grs_moe_combine": ([_P(grs_moe)] + [_vp] * 5, ctypes.c_int),
    "grs_moe_combine_backward": ([_P(grs_moe)] + [_vp] * 7, ctypes.c_int),
    "grs_operators_check_device_errors": ([_vp], ctypes.c_int),
    "grs_experts_forward": ([_P(grs_experts)] + [_vp] * 6, ctypes.c_int),
    "grs_experts_backward": ([_P(grs_experts)] + [_vp] * 8, ctypes.c_int),
    "grs_experts_workspace_bytes": ([_P(grs_experts)], ctypes.c_int64),
    "grs_selftest_experts_wait": ([_P(grs_experts)] + [_vp] * 7 + [ctypes.c_int32, ctypes.c_int32, _vp], ctypes.c_int),
    "grs_embedding_forward": ([_P(grs_embedding)] + [_vp] * 4, ctypes.c_int),
    "grs_embedding_backward": ([_P(grs_embedding)] + [_vp] * 5, ctypes.c_int),
    "grs_embedding_workspace_bytes": ([_P(grs_embedding)], ctypes.c_int64),
    "grs_rope_turns": ([_P(ctypes.c_double), ctypes.c_int32, _P(ctypes.c_uint64)], ctypes.c_int),
    "grs_qk_norm_forward": ([_P(grs_qk_norm)] + [_vp] * 9, ctypes.c_int),
    "grs_qk_norm_backward": ([_P(grs_qk_norm)] + [_vp] * 14, ctypes.c_int),
    "grs_qk_norm_workspace_bytes": ([_P(grs_qk_norm)], ctypes.c_int64),
    "grs_last_error": ([], ctypes.c_char_p),
    "grs_build_features": ([], ctypes.c_uint32),
}
for _name, (_args, _res) in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_sig)


def grs_last_error() -> str:
    return (_lib.grs_last_error() or b"").decode()


def grs_build_features() -> int:
    return int(_lib.grs_build_features())


def _check(status: int, func: str):
    if status != GRS_OK:
        raise GrsError(status, func, grs_last_error())


def pointer_array(seq: Sequence[Optional[int]]):
    """A reusable C array of device pointers: every call below that takes a
    pointer list also takes one of these as is (no conversion per call)."""
    return _ptrs(seq)


def _ptrs(seq: Sequence[Optional[int]]):
    if isinstance(seq, ctypes.Array):
        return seq
    arr = (_vp * max(1, len(seq)))()
    for i, p in enumerate(seq):
        arr[i] = None if p is None else int(p)
    return arr


def grs_plan_create(numels: Sequence[int], owners: Sequence[int], world: int, tp: int,
                    dp_replicate: int, dp_shard: int, bucket_bytes: int, flags: int = 0) -> int:
    n = len(numels)
    ne = (ctypes.c_int64 * max(1, n))(*numels)
    ow = (ctypes.c_int32 * max(1, n))(*owners)
    out = _vp()
    _check(_lib.grs_plan_create(ne, ow, n, world, tp, dp_replicate, dp_shard, bucket_bytes, flags,
                                ctypes.byref(out)), "grs_plan_create")
    return out.value


def grs_plan_create_ex(numels: Sequence[int], owners: Sequence[int], tensor_flags: Optional[Sequence[int]],
                       world: int, tp: int, dp_replicate: int, dp_shard: int, bucket_bytes: int,
                       flags: int = 0) -> int:
    n = len(numels)
    ne = (ctypes.c_int64 * max(1, n))(*numels)
    ow = (ctypes.c_int32 * max(1, n))(*owners)
    tf = None if tensor_flags is None else (ctypes.c_uint32 * max(1, n))(*tensor_flags)
    out = _vp()
    _check(_lib.grs_plan_create_ex(ne, ow, tf, n, world, tp, dp_replicate, dp_shard, bucket_bytes,
                                   flags, ctypes.byref(out)), "grs_plan_create_ex")
    return out.value


def grs_plan_shard_view(plan: int, shard: int, tp_index: int) -> int:
    out = _vp()
    _check(_lib.grs_plan_shard_view(plan, shard, tp_index, ctypes.byref(out)), "grs_plan_shard_view")
    return out.value


def grs_plan_destroy(plan: int) -> None:
    _lib.grs_plan_destroy(plan)


def _as_dict(s) -> Dict[str, int]:
    return {k: getattr(s, k) for k, _ in s._fields_}


def grs_plan_query(plan: int) -> Dict[str, int]:
    o = grs_plan_info()
    _check(_lib.grs_plan_query(plan, ctypes.byref(o)), "grs_plan_query")
    return _as_dict(o)


def grs_bucket_info(plan: int, bucket: int) -> Dict[str, int]:
    o = grs_bucket_desc()
    _check(_lib.grs_bucket_info(plan, bucket, ctypes.byref(o)), "grs_bucket_info")
    return _as_dict(o)


def grs_tensor_info(plan: int, tensor: int) -> Dict[str, int]:
    o = grs_tensor_desc()
    _check(_lib.grs_tensor_info(plan, tensor, ctypes.byref(o)), "grs_tensor_info")
    return _as_dict(o)


def grs_segment_info(plan: int, bucket: int, segment: int) -> Dict[str, int]:
    o = grs_segment_desc()
    _check(_lib.grs_segment_info(plan, bucket, segment, ctypes.byref(o)), "grs_segment_info")
    return _as_dict(o)


def grs_reduce_bucket(plan: int, bucket: int, rank_grads: Sequence[int], acc: int, accumulate: int,
                      emit_norm_partials: int, workspace: Optional[int], stream: int) -> None:
    _check(_lib.grs_reduce_bucket(plan, bucket, _ptrs(rank_grads), acc, accumulate,
                                  emit_norm_partials, workspace, stream), "grs_reduce_bucket")


def grs_reduce_bucket_ex(plan: int, bucket: int, rank_grads: Sequence[int], acc: int, accumulate: int,
                         emit_norm_partials: int, workspace: Optional[int], max_ctas: int,
                         wait_event: Optional[int], stream: int) -> None:
    """wait_event: a cudaEvent_t handle (torch.cuda.Event.cuda_event) or None."""
    _check(_lib.grs_reduce_bucket_ex(plan, bucket, _ptrs(rank_grads), acc, accumulate,
                                     emit_norm_partials, workspace, max_ctas, wait_event, stream),
           "grs_reduce_bucket_ex")


def grs_reduce_all(plan: int, rank_grads: Sequence[int], acc: int, accumulate: int,
                   emit_norm_partials: int, workspace: Optional[int], stream: int) -> None:
    _check(_lib.grs_reduce_all(plan, _ptrs(rank_grads), acc, accumulate, emit_norm_partials,
                               workspace, stream), "grs_reduce_all")


def grs_reduce_all_masked(plan: int, rank_grads: Sequence[int], acc: int, accumulate: int,
                          emit_norm_partials: int, d_tensor_used: int, workspace: Optional[int],
                          stream: int) -> None:
    _check(_lib.grs_reduce_all_masked(plan, _ptrs(rank_grads), acc, accumulate, emit_norm_partials,
                                      d_tensor_used, workspace, stream), "grs_reduce_all_masked")


def grs_accumulate(plan: int, bucket: int, acc: int, mb: int, stream: int) -> None:
    _check(_lib.grs_accumulate(plan, bucket, acc, mb, stream), "grs_accumulate")


def grs_grad_norm_sq(plan: int, acc: Optional[int], n_micro: int, workspace: int,
                     partials_ready: int, d_norm_sq: int, stream: int) -> None:
    _check(_lib.grs_grad_norm_sq(plan, acc, n_micro, workspace, partials_ready, d_norm_sq, stream),
           "grs_grad_norm_sq")


def make_adamw(lr, beta1, beta2, eps, weight_decay, max_norm, step, n_micro) -> grs_adamw:
    return grs_adamw(lr, beta1, beta2, eps, weight_decay, max_norm, step, n_micro)


def grs_clip_adamw_step(plan: int, hp: grs_adamw, d_norm_sq: Optional[int], acc: int, master: int,
                        m: int, v: int, params_bf16: int, stream: int) -> None:
    _check(_lib.grs_clip_adamw_step(plan, ctypes.byref(hp), d_norm_sq, acc, master, m, v,
                                    params_bf16, stream), "grs_clip_adamw_step")


def grs_clip_adamw_step_to_tensors(plan: int, hp: grs_adamw, d_norm_sq: Optional[int], acc: int,
                                   master: int, m: int, v: int, params_bf16: Optional[int],
                                   d_tensor_ptrs: int, stream: int) -> None:
    """d_tensor_ptrs: device address of an int64 array of per-tensor device
    pointers (0 = skip), e.g. ``torch.tensor(ptrs, dtype=torch.int64,
    device=...).data_ptr()``."""
    _check(_lib.grs_clip_adamw_step_to_tensors(plan, ctypes.byref(hp), d_norm_sq, acc, master, m, v,
                                               params_bf16, d_tensor_ptrs, stream),
           "grs_clip_adamw_step_to_tensors")


def grs_gather_params(plan: int, params_bf16: int, tensor_ptrs: Sequence[Optional[int]],
                      stream: int) -> None:
    _check(_lib.grs_gather_params(plan, params_bf16, _ptrs(tensor_ptrs), stream),
           "grs_gather_params")


def grs_step_from_host(plan: int, hp: grs_adamw, host_grads: Sequence[int], dev_stage: Sequence[int],
                       acc: int, master: int, m: int, v: int, params_bf16: int, workspace: int,
                       d_norm_sq: int, host_params: Optional[int], host_norm_sq: Optional[int],
                       stream: int) -> None:
    _check(_lib.grs_step_from_host(plan, ctypes.byref(hp), _ptrs(host_grads), _ptrs(dev_stage), acc,
                                   master, m, v, params_bf16, workspace, d_norm_sq, host_params,
                                   host_norm_sq, stream), "grs_step_from_host")


def grs_grad_norm_sq_noalloc(plan: int, acc: int, n_micro: int, d_norm_sq: int, stream: int) -> None:
    """Global squared norm with the library's static scratch (no workspace,
    no allocation); for callers that cannot allocate device memory."""
    _check(_lib.grs_grad_norm_sq_noalloc(plan, acc, n_micro, d_norm_sq, stream),
           "grs_grad_norm_sq_noalloc")


def grs_grad_norm_sq_masked(plan: int, acc: int, n_micro: int, d_tensor_used: int, workspace: int,
                            d_norm_sq: int, stream: int) -> None:
    _check(_lib.grs_grad_norm_sq_masked(plan, acc, n_micro, d_tensor_used, workspace, d_norm_sq, stream),
           "grs_grad_norm_sq_masked")


def grs_clip_adamw_step_masked(plan: int, hp: grs_adamw, d_norm_sq: Optional[int], acc: int, master: int,
                               m: int, v: int, params_bf16: int, d_tensor_used: int, d_tensor_steps: int,
                               workspace: int, stream: int) -> None:
    _check(_lib.grs_clip_adamw_step_masked(plan, ctypes.byref(hp), d_norm_sq, acc, master, m, v,
                                           params_bf16, d_tensor_used, d_tensor_steps, workspace, stream),
           "grs_clip_adamw_step_masked")


def grs_update_small(plan: int, hp: grs_adamw, rank_grads: Sequence[int], acc: int, master: int, m: int,
                     v: int, params_bf16: int, d_norm_sq: int, stream: int) -> None:
    """The whole update of a small plan in one launch; rank_grads holds
    n_micro * world buffers, microbatch-major."""
    _check(_lib.grs_update_small(plan, ctypes.byref(hp), _ptrs(rank_grads), acc, master, m, v, params_bf16,
                                 d_norm_sq, stream), "grs_update_small")


def grs_state_to_logical(plan: int, state: int, logical: int, stream: int) -> None:
    _check(_lib.grs_state_to_logical(plan, state, logical, stream), "grs_state_to_logical")


def grs_state_from_logical(plan: int, logical: int, state: int, stream: int) -> None:
    _check(_lib.grs_state_from_logical(plan, logical, state, stream), "grs_state_from_logical")


def grs_check_already_reduced(plan: int, rank_grads: Sequence[int], stream: int) -> None:
    _check(_lib.grs_check_already_reduced(plan, _ptrs(rank_grads), stream), "grs_check_already_reduced")


def grs_selftest_bounded_wait(plan: int, limit_ns: int, stream: int) -> None:
    _check(_lib.grs_selftest_bounded_wait(plan, limit_ns, stream), "grs_selftest_bounded_wait")


def grs_check_device_errors(plan: int, stream: int) -> int:
    """Returns the status (raises only for CUDA errors)."""
    st = _lib.grs_check_device_errors(plan, stream)
    if st == GRS_ERR_CUDA:
        _check(st, "grs_check_device_errors")
    return st


def grs_tensors_create(numels: Sequence[int], flags: int = 0) -> int:
    n = len(numels)
    ne = (ctypes.c_int64 * max(1, n))(*numels)
    out = _vp()
    _check(_lib.grs_tensors_create(ne, n, flags, ctypes.byref(out)), "grs_tensors_create")
    return out.value


def grs_tensors_destroy(tensors: int) -> None:
    _lib.grs_tensors_destroy(tensors)


def grs_tensors_query(tensors: int) -> Dict[str, int]:
    o = grs_tensors_info()
    _check(_lib.grs_tensors_query(tensors, ctypes.byref(o)), "grs_tensors_query")
    return _as_dict(o)


def grs_tensors_offset(tensors: int, tensor: int) -> int:
    o = ctypes.c_int64()
    _check(_lib.grs_tensors_offset(tensors, tensor, ctypes.byref(o)), "grs_tensors_offset")
    return o.value


def grs_tensors_norm_sq(tensors: int, d_grads: int, grad_dtype: int, n_micro: int, workspace: int, d_norm_sq: int,
                        stream: int) -> None:
    """d_grads (here and below): device address of an int64 array of
    per-tensor device pointers (0 = no gradient)."""
    _check(_lib.grs_tensors_norm_sq(tensors, d_grads, grad_dtype, n_micro, workspace, d_norm_sq, stream),
           "grs_tensors_norm_sq")


def grs_tensors_adamw_step(tensors: int, hp: grs_adamw, d_norm_sq: Optional[int], d_grads: int, grad_dtype: int,
                           master: int, m: int, v: int, d_params_bf16: Optional[int], stream: int) -> None:
    _check(_lib.grs_tensors_adamw_step(tensors, ctypes.byref(hp), d_norm_sq, d_grads, grad_dtype, master, m, v,
                                       d_params_bf16, stream), "grs_tensors_adamw_step")


def grs_tensors_adamw8_step(tensors: int, hp: grs_adamw, seed: int, d_norm_sq: Optional[int], d_grads: int,
                            grad_dtype: int, master: int, m8: int, m_scale: int, s8: int, s_scale: int,
                            d_params_bf16: Optional[int], stream: int) -> None:
    _check(_lib.grs_tensors_adamw8_step(tensors, ctypes.byref(hp), seed, d_norm_sq, d_grads, grad_dtype, master, m8,
                                        m_scale, s8, s_scale, d_params_bf16, stream), "grs_tensors_adamw8_step")


def grs_tensors_pack8(tensors: int, m: int, v: int, m8: int, m_scale: int, s8: int, s_scale: int,
                      stream: int) -> None:
    _check(_lib.grs_tensors_pack8(tensors, m, v, m8, m_scale, s8, s_scale, stream), "grs_tensors_pack8")


def grs_tensors_unpack8(tensors: int, m8: int, m_scale: int, s8: int, s_scale: int, m: int, v: int,
                        stream: int) -> None:
    _check(_lib.grs_tensors_unpack8(tensors, m8, m_scale, s8, s_scale, m, v, stream), "grs_tensors_unpack8")


def grs_tensors_check_device_errors(tensors: int, stream: int) -> int:
    """Returns the status (raises only for CUDA errors)."""
    st = _lib.grs_tensors_check_device_errors(tensors, stream)
    if st == GRS_ERR_CUDA:
        _check(st, "grs_tensors_check_device_errors")
    return st


def make_norm(rows: int, cols: int, eps: float, dtype: int, param_dtype: int, grad_dtype: int, ld_x: int = 0,
              ld_y: int = 0, ld_dy: int = 0, ld_dx: int = 0) -> grs_norm:
    return grs_norm(rows, ld_x, ld_y, ld_dy, ld_dx, cols, eps, dtype, param_dtype, grad_dtype, 0)


def grs_layernorm_forward(shape: grs_norm, x: int, w: Optional[int], b: Optional[int], y: int, mean: Optional[int],
                          rstd: Optional[int], stream: int) -> None:
    _check(_lib.grs_layernorm_forward(ctypes.byref(shape), x, w, b, y, mean, rstd, stream), "grs_layernorm_forward")


def grs_layernorm_backward(shape: grs_norm, dy: int, x: int, w: Optional[int], mean: int, rstd: int,
                           dx: Optional[int], dw: Optional[int], db: Optional[int], workspace: Optional[int],
                           stream: int) -> None:
    _check(_lib.grs_layernorm_backward(ctypes.byref(shape), dy, x, w, mean, rstd, dx, dw, db, workspace, stream),
           "grs_layernorm_backward")


def _bytes(n: int, func: str) -> int:
    if n < 0:
        raise GrsError(GRS_ERR_INVALID_ARG, func, grs_last_error())
    return n


def grs_layernorm_workspace_bytes(shape: grs_norm) -> int:
    return _bytes(int(_lib.grs_layernorm_workspace_bytes(ctypes.byref(shape))), "grs_layernorm_workspace_bytes")


def grs_layernorm_check_device_errors(stream: int) -> int:
    """Returns the status (raises only for CUDA errors)."""
    st = _lib.grs_layernorm_check_device_errors(stream)
    if st == GRS_ERR_CUDA:
        _check(st, "grs_layernorm_check_device_errors")
    return st


def grs_selftest_layernorm_wait(shape: grs_norm, dy: int, x: int, w: Optional[int], mean: int, rstd: int, dx: int,
                                dw: Optional[int], db: Optional[int], workspace: Optional[int], limit_ns: int,
                                quitter: int, quit_row: int, stream: int) -> None:
    _check(_lib.grs_selftest_layernorm_wait(ctypes.byref(shape), dy, x, w, mean, rstd, dx, dw, db, workspace, limit_ns,
                                            quitter, quit_row, stream), "grs_selftest_layernorm_wait")


def make_moe(tokens: int, top_k: int, n_experts: int, expert_begin: int, expert_end: int, hidden: int,
             dtype: int) -> grs_moe:
    """n_experts is what the router chooses from; the call's experts are
    [expert_begin, expert_end) of them."""
    if not 0 <= expert_begin < expert_end <= n_experts:
        raise GrsError(GRS_ERR_INVALID_ARG, "make_moe", "the expert range must lie in [0, n_experts)")
    return grs_moe(tokens, top_k, expert_begin, expert_end, hidden, dtype, 0)


def grs_moe_workspace_bytes(shape: grs_moe) -> int:
    return _bytes(int(_lib.grs_moe_workspace_bytes(ctypes.byref(shape))), "grs_moe_workspace_bytes")


def grs_moe_sort(shape: grs_moe, expert_ids: int, expert_offsets: int, row_slot: int, slot_row: int, workspace: int,
                 stream: int) -> None:
    _check(_lib.grs_moe_sort(ctypes.byref(shape), expert_ids, expert_offsets, row_slot, slot_row, workspace, stream),
           "grs_moe_sort")


def grs_moe_dispatch(shape: grs_moe, x: int, slot_row: int, xs: int, stream: int) -> None:
    _check(_lib.grs_moe_dispatch(ctypes.byref(shape), x, slot_row, xs, stream), "grs_moe_dispatch")


def grs_moe_dispatch_backward(shape: grs_moe, dxs: int, slot_row: int, dx: int, stream: int) -> None:
    _check(_lib.grs_moe_dispatch_backward(ctypes.byref(shape), dxs, slot_row, dx, stream), "grs_moe_dispatch_backward")


def grs_moe_combine(shape: grs_moe, ys: int, slot_row: int, weights: int, y: int, stream: int) -> None:
    _check(_lib.grs_moe_combine(ctypes.byref(shape), ys, slot_row, weights, y, stream), "grs_moe_combine")


def grs_moe_combine_backward(shape: grs_moe, dy: int, ys: int, slot_row: int, weights: int, dys: int, dweights: int,
                             stream: int) -> None:
    _check(_lib.grs_moe_combine_backward(ctypes.byref(shape), dy, ys, slot_row, weights, dys, dweights, stream),
           "grs_moe_combine_backward")


def grs_operators_check_device_errors(stream: int) -> int:
    """Returns the status (raises only for CUDA errors)."""
    st = _lib.grs_operators_check_device_errors(stream)
    if st == GRS_ERR_CUDA:
        _check(st, "grs_operators_check_device_errors")
    return st


def make_experts(rows: int, experts: int, in_features: int, out_features: int, dtype: int, grad_dtype: int, ld_x: int = 0,
                 ld_y: int = 0) -> grs_experts:
    return grs_experts(rows, ld_x, ld_y, experts, in_features, out_features, dtype, grad_dtype, 0)


def grs_experts_workspace_bytes(shape: grs_experts) -> int:
    return _bytes(int(_lib.grs_experts_workspace_bytes(ctypes.byref(shape))), "grs_experts_workspace_bytes")


def grs_experts_forward(shape: grs_experts, xs: int, w: int, offsets: int, ys: int, workspace: Optional[int], stream: int) -> None:
    _check(_lib.grs_experts_forward(ctypes.byref(shape), xs, w, offsets, ys, workspace, stream), "grs_experts_forward")


def grs_experts_backward(shape: grs_experts, dys: int, xs: Optional[int], w: Optional[int], offsets: int, dxs: Optional[int],
                         dw: Optional[int], workspace: Optional[int], stream: int) -> None:
    _check(_lib.grs_experts_backward(ctypes.byref(shape), dys, xs, w, offsets, dxs, dw, workspace, stream),
           "grs_experts_backward")


def grs_selftest_experts_wait(shape: grs_experts, dys: int, xs: Optional[int], w: Optional[int], offsets: int, dxs: Optional[int],
                              dw: Optional[int], workspace: Optional[int], quitter: int, quit_tile: int, stream: int) -> None:
    _check(_lib.grs_selftest_experts_wait(ctypes.byref(shape), dys, xs, w, offsets, dxs, dw, workspace, quitter, quit_tile, stream),
           "grs_selftest_experts_wait")


def make_embedding(tokens: int, row_begin: int, row_end: int, hidden: int, scale: float, dtype: int,
                   grad_dtype: int) -> grs_embedding:
    return grs_embedding(tokens, row_begin, row_end, hidden, scale, dtype, grad_dtype)


def grs_embedding_workspace_bytes(shape: grs_embedding) -> int:
    return _bytes(int(_lib.grs_embedding_workspace_bytes(ctypes.byref(shape))), "grs_embedding_workspace_bytes")


def grs_embedding_forward(shape: grs_embedding, ids: int, table: int, y: int, stream: int) -> None:
    _check(_lib.grs_embedding_forward(ctypes.byref(shape), ids, table, y, stream), "grs_embedding_forward")


def grs_embedding_backward(shape: grs_embedding, ids: int, dy: int, dtable: int, workspace: Optional[int], stream: int) -> None:
    _check(_lib.grs_embedding_backward(ctypes.byref(shape), ids, dy, dtable, workspace, stream), "grs_embedding_backward")


def make_qk_norm(tokens: int, q_heads: int, k_heads: int, head_dim: int, rotary_dim: int, eps: float, dtype: int, param_dtype: int,
                 grad_dtype: int, interleaved: bool = False, ld_q: int = 0, ld_k: int = 0, ld_qo: int = 0,
                 ld_ko: int = 0) -> grs_qk_norm:
    return grs_qk_norm(tokens, ld_q, ld_k, ld_qo, ld_ko, q_heads, k_heads, head_dim, rotary_dim, int(interleaved), eps, dtype,
                       param_dtype, grad_dtype, 0)


def grs_rope_turns(inv_freq: Sequence[float]) -> list:
    """The frequencies as fractions of 2^64 of a turn, for a device uint64 tensor."""
    n = len(inv_freq)
    out = (ctypes.c_uint64 * max(1, n))()
    _check(_lib.grs_rope_turns((ctypes.c_double * max(1, n))(*inv_freq), n, out), "grs_rope_turns")
    return list(out)[:n]


def grs_qk_norm_workspace_bytes(shape: grs_qk_norm) -> int:
    return _bytes(int(_lib.grs_qk_norm_workspace_bytes(ctypes.byref(shape))), "grs_qk_norm_workspace_bytes")


def grs_qk_norm_forward(shape: grs_qk_norm, q: Optional[int], k: Optional[int], wq: Optional[int], wk: Optional[int],
                        positions: Optional[int], turns: Optional[int], qo: Optional[int], ko: Optional[int], stream: int) -> None:
    _check(_lib.grs_qk_norm_forward(ctypes.byref(shape), q, k, wq, wk, positions, turns, qo, ko, stream), "grs_qk_norm_forward")


def grs_qk_norm_backward(shape: grs_qk_norm, dqo: Optional[int], dko: Optional[int], q: Optional[int], k: Optional[int],
                         wq: Optional[int], wk: Optional[int], positions: Optional[int], turns: Optional[int], dq: Optional[int],
                         dk: Optional[int], dwq: Optional[int], dwk: Optional[int], workspace: Optional[int], stream: int) -> None:
    _check(_lib.grs_qk_norm_backward(ctypes.byref(shape), dqo, dko, q, k, wq, wk, positions, turns, dq, dk, dwq, dwk, workspace,
                                     stream), "grs_qk_norm_backward")
