"""Python binding of libzero (the sharded mixed-precision AdamW step for GB300).

Thin ctypes marshalling over the C ABI declared in ``include/zero.h``: every
function has the C name and forwards plain integers (device pointers, sizes,
stream handles).  All arithmetic runs in the CUDA kernels of ``libzero.so``;
there is no Python or CPU fallback.  If the library has not been built, import
succeeds but the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libzero.so")

ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ECUDA, ZERO_ESTATE, ZERO_ERANGE, ZERO_ETIMEOUT, ZERO_ENOMEM = range(8)
ZERO_BF16, ZERO_FP16, ZERO_FP32 = 0, 1, 2
ZERO_MAX_RANKS = 128
ZERO_REPORT_GRAD_NORM = 1
(ZERO_OPT_STAGING, ZERO_OPT_WAIT_LIMIT_NS, ZERO_OPT_BULK_TILE, ZERO_OPT_BULK_STAGES,
 ZERO_OPT_LAST_STEP_KERNEL, ZERO_OPT_GATHER_STAGING, ZERO_OPT_GATHER_CHUNK,
 ZERO_OPT_GATHER_STAGES, ZERO_OPT_HOST_PIPELINE, ZERO_OPT_HOST_H2D_BYTES,
 ZERO_OPT_HOST_D2H_BYTES, ZERO_OPT_LAST_GATHER_IN_STEP, ZERO_OPT_OFFLOAD_DEFER,
 ZERO_OPT_UNIT_ORDER) = range(14)
ZERO_STAGING_REGISTER_LOADS, ZERO_STAGING_BULK, ZERO_STAGING_AUTO = range(3)
(ZERO_TABLE_TENSOR_OFFSET, ZERO_TABLE_UNITS, ZERO_TABLE_SHARD_SEGMENTS,
 ZERO_TABLE_BUCKET_SEGMENTS, ZERO_TABLE_STATE_LAYOUT, ZERO_TABLE_PARAM_CHUNKS) = range(6)
TABLE_COLS = {0: 1, 1: 7, 2: 6, 3: 5, 4: 4, 5: 10}
ZERO_WEIGHT_OUT_IN, ZERO_WEIGHT_IN_OUT = range(2)
ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_GELU_TANH, ZERO_ACT_GELU, ZERO_ACT_SILU = range(5)
ZERO_LINEAR_ACCUMULATE = 1
ZERO_GATED_ACCUMULATE = 1
ZERO_LINEAR_MAX_SIZE = 1073741824
ZERO_NORM_RMS, ZERO_NORM_LAYER = range(2)
ZERO_NORM_PRE, ZERO_NORM_POST = 1, 2
ZERO_NORM_MAX_DIM = 8192
ZERO_ADAMW_BLOCK = 256
ZERO_ADAMW_MAX_BLOCKS = 1073741824
ZERO_MUON_SCALE_NONE, ZERO_MUON_SCALE_ASPECT, ZERO_MUON_SCALE_RMS = range(3)
ZERO_MUON_NESTEROV = 1
ZERO_MUON_MAX_STEPS = 8
ZERO_MUON_MAX_MATRICES = 65536
ZERO_MUON_MAX_SIZE = 4194304
ZERO_MUON_MAX_SIDE = 65536
ZERO_MUON_BLOCK = 256
ZERO_MUON_OPT_WAIT_LIMIT_NS, ZERO_MUON_OPT_SMS = range(2)
ZERO_MUON_MAX_WAIT_NS = 30_000_000_000
STATUS_NAMES = {0: "ZERO_OK", 1: "ZERO_EINVAL", 2: "ZERO_EALIGN", 3: "ZERO_ECUDA",
                4: "ZERO_ESTATE", 5: "ZERO_ERANGE", 6: "ZERO_ETIMEOUT", 7: "ZERO_ENOMEM"}

EXPORTED = ["zero_plan_create", "zero_plan_create_per_param", "zero_plan_info", "zero_rank_state_elems", "zero_plan_tables",
            "zero_bind", "zero_bind_peer", "zero_step", "zero_step_finish", "zero_gather_layer",
            "zero_release_layer", "zero_memory_report", "zero_comm_report", "zero_set_scaler",
            "zero_read_state", "zero_restore_state", "zero_grad_norm",
            "zero_step_units_overlapped", "zero_bind_offload", "zero_offload_step",
            "zero_offload_finish", "zero_set_option", "zero_get_option",
            "zero_bind_host_staging", "zero_step_host", "zero_step_host_finish", "zero_grad_norm_host",
            "zero_step_gather_next",
            "zero_last_error", "zero_plan_destroy", "zero_step_range_noalloc",
            "zero_linear_workspace", "zero_linear", "zero_linear_backward", "zero_operators_check",
            "zero_gated_workspace", "zero_gated", "zero_gated_backward",
            "zero_block_norm", "zero_block_norm_workspace", "zero_block_norm_backward",
            "zero_adamw_create", "zero_adamw_info", "zero_adamw_bind", "zero_adamw_step",
            "zero_adamw_check", "zero_adamw_step_with", "zero_adamw_export", "zero_adamw_read", "zero_adamw_destroy",
            "zero_muon_create", "zero_muon_info", "zero_muon_set_option", "zero_muon_bind", "zero_muon_step",
            "zero_muon_check", "zero_muon_step_with", "zero_muon_read", "zero_muon_destroy"]
ZERO_NOALLOC_SCRATCH_BYTES = 256


class ZeroError(RuntimeError):
    def __init__(self, status: int, msg: str, result=None):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status
        self.result = result   # the step state read with a ZERO_ETIMEOUT report


class zero_hyper_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("max_grad_norm", ctypes.c_double), ("flags", ctypes.c_int64)]


class zero_scaler_t(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_double), ("growth_factor", ctypes.c_double),
                ("backoff_factor", ctypes.c_double), ("min_scale", ctypes.c_double),
                ("growth_interval", ctypes.c_int64), ("good_steps", ctypes.c_int64)]


class zero_plan_info_t(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int64), ("n_units", ctypes.c_int64),
                ("n_buckets", ctypes.c_int64), ("phi", ctypes.c_int64),
                ("phi_pad", ctypes.c_int64), ("shard", ctypes.c_int64),
                ("max_contrib_elems", ctypes.c_int64), ("max_unit_pad", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64), ("n_d", ctypes.c_int32),
                ("stage", ctypes.c_int32), ("dtype16", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("host_staging_bytes", ctypes.c_int64)]


class zero_step_result_t(ctypes.Structure):
    _fields_ = [("skipped", ctypes.c_int32), ("current", ctypes.c_int32),
                ("t", ctypes.c_int64), ("scale", ctypes.c_double),
                ("good_steps", ctypes.c_int64), ("skipped_total", ctypes.c_int64),
                ("finished", ctypes.c_int64), ("grad_norm", ctypes.c_double)]


class zero_mem_report_t(ctypes.Structure):
    _fields_ = [("logical", (ctypes.c_int64 * 3) * 4), ("logical_total", ctypes.c_int64 * 4),
                ("logical_ddp_fp32_grads", ctypes.c_int64),
                ("physical_state_bytes", ctypes.c_int64),
                ("physical_param16_bytes", ctypes.c_int64),
                ("physical_contrib_bytes", ctypes.c_int64),
                ("physical_gather_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]


class zero_comm_report_t(ctypes.Structure):
    _fields_ = [("per_collective", ctypes.c_int64), ("ddp", ctypes.c_int64),
                ("zero1", ctypes.c_int64), ("zero2", ctypes.c_int64), ("zero3", ctypes.c_int64),
                ("this_stage", ctypes.c_int64), ("bytes_per_elem", ctypes.c_int64),
                ("collectives_per_step", ctypes.c_int64)]


class zero_linear_t(ctypes.Structure):
    """One linear layer's sizes, strides (0: dense) and device pointers; see include/zero.h."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("rows", "in_features", "out_features")] +
                [(k, ctypes.c_int32) for k in ("dtype16", "layout", "activation", "flags")] +
                [(k, ctypes.c_int64) for k in ("ld_x", "ld_w", "ld_y", "ld_pre", "ld_residual", "ld_dy",
                                               "ld_dx", "ld_dw")] +
                [(k, ctypes.c_void_p) for k in ("x", "w", "bias", "residual", "y", "pre", "dy", "dx",
                                                "dw", "dbias")])


class zero_gated_t(ctypes.Structure):
    """The first half of a gated feed-forward block: sizes, strides (0: dense) and device pointers; see
    include/zero.h."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("rows", "in_features", "out_features")] +
                [(k, ctypes.c_int32) for k in ("dtype16", "layout", "activation", "flags")] +
                [(k, ctypes.c_int64) for k in ("ld_x", "ld_w_gate", "ld_w_up", "ld_h", "ld_gate", "ld_up", "ld_dh",
                                               "ld_dx", "ld_dw_gate", "ld_dw_up")] +
                [(k, ctypes.c_void_p) for k in ("x", "w_gate", "w_up", "b_gate", "b_up", "h", "gate", "up", "dh",
                                                "dx", "dw_gate", "dw_up", "db_gate", "db_up")])


class zero_block_norm_t(ctypes.Structure):
    """The norms around a block: sizes, strides (0: dense) and device pointers; see include/zero.h."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("rows", "dim")] +
                [(k, ctypes.c_int32) for k in ("dtype16", "kind", "norms", "reserved")] +
                [("rows_per_gate", ctypes.c_int64), ("eps", ctypes.c_double),
                 ("residual_scale", ctypes.c_double)] +
                [(k, ctypes.c_int64) for k in ("ld_h", "ld_x", "ld_y", "ld_z", "ld_gate", "ld_dy", "ld_dz",
                                               "ld_dx", "ld_dh", "ld_dgate")] +
                [(k, ctypes.c_void_p) for k in ("h", "x", "gate", "post_w", "post_b", "pre_w", "pre_b", "y",
                                                "z", "dy", "dz", "dx", "dh", "dgate", "dpost_w", "dpost_b",
                                                "dpre_w", "dpre_b")])


class zero_adamw_info_t(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in
                ("n_tensors", "elems", "n_blocks", "state_elems", "moment_bytes", "scale_bytes",
                 "workspace_bytes")]


class zero_muon_hyper_t(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_double) for k in ("lr", "momentum", "weight_decay", "eps")] +
                [("coefficients", (ctypes.c_double * 3) * ZERO_MUON_MAX_STEPS), ("steps", ctypes.c_int32),
                 ("scale", ctypes.c_int32), ("flags", ctypes.c_int64)])


class zero_muon_info_t(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("n_matrices", "n_contribs", "elems", "state_elems", "workspace_bytes")]


_lib = None
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int


def lib() -> ctypes.CDLL:
    """Load libzero.so; raises if it is missing (no fallback path exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libzero.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        st = _int
        L.zero_plan_create.restype = st
        L.zero_plan_create.argtypes = [_vp, _i64, _int, _int, _i64, _vp, _i64, _int,
                                       ctypes.POINTER(_vp)]
        L.zero_plan_create_per_param.restype = st
        L.zero_plan_create_per_param.argtypes = [_vp, _vp, _i64, _int, _vp, _i64, _int,
                                                 ctypes.POINTER(_vp)]
        L.zero_plan_info.restype = st
        L.zero_plan_info.argtypes = [_vp, ctypes.POINTER(zero_plan_info_t)]
        L.zero_rank_state_elems.restype = st
        L.zero_rank_state_elems.argtypes = [_vp, _int, ctypes.POINTER(_i64)]
        L.zero_plan_tables.restype = st
        L.zero_plan_tables.argtypes = [_vp, _int, _vp, _i64, ctypes.POINTER(_i64)]
        L.zero_bind.restype = st
        L.zero_bind.argtypes = [_vp, _int, _vp, _vp, _vp, _vp, _vp, _vp]
        L.zero_bind_peer.restype = st
        L.zero_bind_peer.argtypes = [_vp, _int, _vp]
        L.zero_step.restype = st
        L.zero_step.argtypes = [_vp, _vp, _i64, _i64, ctypes.POINTER(zero_hyper_t), _vp]
        L.zero_step_finish.restype = st
        L.zero_step_finish.argtypes = [_vp, _vp, ctypes.POINTER(zero_step_result_t)]
        L.zero_set_scaler.restype = st
        L.zero_set_scaler.argtypes = [_vp, ctypes.POINTER(zero_scaler_t), _vp]
        L.zero_read_state.restype = st
        L.zero_read_state.argtypes = [_vp, _vp, ctypes.POINTER(zero_step_result_t)]
        L.zero_step_units_overlapped.restype = st
        L.zero_step_units_overlapped.argtypes = [_vp, _vp, _i64, _vp, ctypes.POINTER(zero_hyper_t),
                                                 _vp, _vp, ctypes.POINTER(zero_step_result_t)]
        L.zero_bind_offload.restype = st
        L.zero_bind_offload.argtypes = [_vp, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.zero_offload_step.restype = st
        L.zero_offload_step.argtypes = [_vp, _vp, _i64, _i64, ctypes.POINTER(zero_hyper_t), _vp]
        L.zero_offload_finish.restype = st
        L.zero_offload_finish.argtypes = [_vp, _int, _vp, ctypes.POINTER(zero_step_result_t)]
        L.zero_step_gather_next.restype = st
        L.zero_step_gather_next.argtypes = [_vp, _vp, _i64, _i64, ctypes.POINTER(zero_hyper_t), _i64,
                                            _vp, _vp]
        L.zero_bind_host_staging.restype = st
        L.zero_bind_host_staging.argtypes = [_vp, _vp, _i64]
        L.zero_step_host.restype = st
        L.zero_step_host.argtypes = [_vp, _vp, _i64, _i64, ctypes.POINTER(zero_hyper_t), _vp, _vp]
        L.zero_grad_norm_host.restype = st
        L.zero_grad_norm_host.argtypes = [_vp, _vp, _i64, _i64, _vp]
        L.zero_step_host_finish.restype = st
        L.zero_step_host_finish.argtypes = [_vp, _vp, ctypes.POINTER(zero_step_result_t)]
        L.zero_grad_norm.restype = st
        L.zero_grad_norm.argtypes = [_vp, _vp, _i64, _i64, _vp]
        L.zero_set_option.restype = st
        L.zero_set_option.argtypes = [_vp, _int, _i64]
        L.zero_get_option.restype = st
        L.zero_get_option.argtypes = [_vp, _int, ctypes.POINTER(_i64)]
        L.zero_restore_state.restype = st
        L.zero_restore_state.argtypes = [_vp, ctypes.POINTER(zero_step_result_t), _vp]
        L.zero_gather_layer.restype = st
        L.zero_gather_layer.argtypes = [_vp, _i64, _vp, _vp]
        L.zero_release_layer.restype = st
        L.zero_release_layer.argtypes = [_vp, _i64]
        L.zero_memory_report.restype = st
        L.zero_memory_report.argtypes = [_vp, ctypes.POINTER(zero_mem_report_t)]
        L.zero_comm_report.restype = st
        L.zero_comm_report.argtypes = [_vp, ctypes.POINTER(zero_comm_report_t)]
        L.zero_last_error.restype = ctypes.c_char_p
        L.zero_last_error.argtypes = []
        L.zero_step_range_noalloc.restype = st
        L.zero_step_range_noalloc.argtypes = [_vp, _int, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, ctypes.POINTER(zero_hyper_t), _i64,
                                              ctypes.c_double, _vp, ctypes.POINTER(ctypes.c_int32)]
        L.zero_plan_destroy.restype = None
        L.zero_plan_destroy.argtypes = [_vp]
        L.zero_linear_workspace.argtypes = [ctypes.POINTER(zero_linear_t), _int, ctypes.POINTER(_i64)]
        L.zero_linear.argtypes = [ctypes.POINTER(zero_linear_t), _vp, _i64, _vp]
        L.zero_linear_backward.argtypes = [ctypes.POINTER(zero_linear_t), _vp, _i64, _vp]
        L.zero_operators_check.argtypes = [_vp]
        for f in (L.zero_linear_workspace, L.zero_linear, L.zero_linear_backward, L.zero_operators_check):
            f.restype = st
        L.zero_gated_workspace.argtypes = [ctypes.POINTER(zero_gated_t), _int, ctypes.POINTER(_i64)]
        L.zero_gated.argtypes = [ctypes.POINTER(zero_gated_t), _vp, _i64, _vp]
        L.zero_gated_backward.argtypes = [ctypes.POINTER(zero_gated_t), _vp, _i64, _vp]
        for f in (L.zero_gated_workspace, L.zero_gated, L.zero_gated_backward):
            f.restype = st
        L.zero_block_norm.argtypes = [ctypes.POINTER(zero_block_norm_t), _vp]
        L.zero_block_norm_workspace.argtypes = [ctypes.POINTER(zero_block_norm_t), ctypes.POINTER(_i64)]
        L.zero_block_norm_backward.argtypes = [ctypes.POINTER(zero_block_norm_t), _vp, _i64, _vp]
        for f in (L.zero_block_norm, L.zero_block_norm_workspace, L.zero_block_norm_backward):
            f.restype = st
        L.zero_adamw_create.argtypes = [_vp, _i64, _int, _int, _int, ctypes.POINTER(_vp)]
        L.zero_adamw_info.argtypes = [_vp, ctypes.POINTER(zero_adamw_info_t)]
        L.zero_adamw_bind.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
        L.zero_adamw_step.argtypes = [_vp, ctypes.POINTER(zero_hyper_t), ctypes.c_double, _vp]
        L.zero_adamw_check.argtypes = [_vp, _vp, _vp]
        L.zero_adamw_step_with.argtypes = [_vp, _vp, ctypes.POINTER(zero_hyper_t), _vp]
        L.zero_adamw_export.argtypes = [_vp, _vp, _vp, _vp]
        L.zero_adamw_read.argtypes = [_vp, _vp, ctypes.POINTER(zero_step_result_t)]
        for f in (L.zero_adamw_create, L.zero_adamw_info, L.zero_adamw_bind, L.zero_adamw_step,
                  L.zero_adamw_check, L.zero_adamw_step_with, L.zero_adamw_export, L.zero_adamw_read):
            f.restype = st
        L.zero_adamw_destroy.restype = None
        L.zero_adamw_destroy.argtypes = [_vp]
        L.zero_muon_create.argtypes = [_vp, _vp, _i64, _int, _int, ctypes.POINTER(_vp)]
        L.zero_muon_info.argtypes = [_vp, ctypes.POINTER(zero_muon_info_t)]
        L.zero_muon_set_option.argtypes = [_vp, _int, _i64]
        L.zero_muon_bind.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
        L.zero_muon_step.argtypes = [_vp, ctypes.POINTER(zero_muon_hyper_t), ctypes.c_double, _vp]
        L.zero_muon_check.argtypes = [_vp, _vp, ctypes.POINTER(zero_muon_hyper_t), _vp]
        L.zero_muon_step_with.argtypes = [_vp, _vp, ctypes.POINTER(zero_muon_hyper_t), _vp]
        L.zero_muon_read.argtypes = [_vp, _vp, ctypes.POINTER(zero_step_result_t)]
        for f in (L.zero_muon_create, L.zero_muon_info, L.zero_muon_set_option, L.zero_muon_bind, L.zero_muon_step,
                  L.zero_muon_check, L.zero_muon_step_with, L.zero_muon_read):
            f.restype = st
        L.zero_muon_destroy.restype = None
        L.zero_muon_destroy.argtypes = [_vp]
        _lib = L
    return _lib


def _check(status: int, result=None) -> None:
    if status != ZERO_OK:
        msg = lib().zero_last_error()
        raise ZeroError(status, msg.decode() if msg else "", result)


def _ptr_array(ptrs: Sequence[Optional[int]]):
    arr = (_vp * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = p or None
    return arr


def _i64_array(vals: Sequence[int]):
    arr = (_i64 * max(1, len(vals)))()
    for i, v in enumerate(vals):
        arr[i] = int(v)
    return arr


# --------------------------------------------------------------------------- C-named calls

def zero_plan_create(tensor_sizes: Sequence[int], n_d: int, stage: int, bucket_elems: int = 0,
                     unit_first: Optional[Sequence[int]] = None, dtype16: int = ZERO_BF16) -> int:
    sizes = _i64_array(tensor_sizes)
    units = _i64_array(unit_first) if unit_first else None
    out = _vp()
    _check(lib().zero_plan_create(sizes, len(tensor_sizes), n_d, stage, bucket_elems, units,
                                  len(unit_first) if unit_first else 0, dtype16,
                                  ctypes.byref(out)))
    return int(out.value)


def zero_plan_create_per_param(tensor_sizes: Sequence[int], dim0: Sequence[int], n_d: int,
                               unit_first: Optional[Sequence[int]] = None,
                               dtype16: int = ZERO_BF16) -> int:
    sizes = _i64_array(tensor_sizes)
    d0 = _i64_array(dim0)
    units = _i64_array(unit_first) if unit_first else None
    out = _vp()
    _check(lib().zero_plan_create_per_param(sizes, d0, len(tensor_sizes), n_d, units,
                                            len(unit_first) if unit_first else 0, dtype16,
                                            ctypes.byref(out)))
    return int(out.value)


def zero_plan_info(plan: int) -> zero_plan_info_t:
    info = zero_plan_info_t()
    _check(lib().zero_plan_info(plan, ctypes.byref(info)))
    return info


def zero_rank_state_elems(plan: int, rank: int) -> int:
    n = _i64()
    _check(lib().zero_rank_state_elems(plan, rank, ctypes.byref(n)))
    return int(n.value)


def zero_plan_tables(plan: int, which: int):
    """Returns a list of rows (tuples of ints)."""
    n = _i64()
    _check(lib().zero_plan_tables(plan, which, None, 0, ctypes.byref(n)))
    cols = TABLE_COLS[which]
    buf = (_i64 * max(1, n.value * cols))()
    _check(lib().zero_plan_tables(plan, which, buf, n.value * cols, ctypes.byref(n)))
    return [tuple(buf[i * cols:(i + 1) * cols]) for i in range(n.value)]


def zero_bind(plan: int, rank: int, master: Sequence[int], m: Sequence[int], v: Sequence[int],
              shard16: Optional[int], full16: Optional[int], workspace: int) -> None:
    _check(lib().zero_bind(plan, rank, _ptr_array(master), _ptr_array(m), _ptr_array(v),
                           shard16 or None, full16 or None, workspace or None))


def zero_bind_peer(plan: int, rank: int, shard16: int) -> None:
    _check(lib().zero_bind_peer(plan, rank, shard16 or None))


def zero_set_scaler(plan: int, scaler: Optional[zero_scaler_t], stream: int = 0) -> None:
    _check(lib().zero_set_scaler(plan, ctypes.byref(scaler) if scaler is not None else None,
                                 stream or None))


def zero_step(plan: int, grad_contribs: Sequence[int], which: int, hyper: zero_hyper_t,
              stream: int = 0) -> None:
    _check(lib().zero_step(plan, _ptr_array(grad_contribs), len(grad_contribs), which,
                           ctypes.byref(hyper), stream or None))


def zero_step_gather_next(plan: int, grad_contribs: Sequence[int], unit: int, hyper: zero_hyper_t,
                          next_unit: int, next_full16: int, stream: int = 0) -> None:
    _check(lib().zero_step_gather_next(plan, _ptr_array(grad_contribs), len(grad_contribs), unit,
                                       ctypes.byref(hyper), next_unit, next_full16 or None,
                                       stream or None))


def zero_grad_norm(plan: int, grad_contribs: Sequence[int], which: int, stream: int = 0) -> None:
    _check(lib().zero_grad_norm(plan, _ptr_array(grad_contribs), len(grad_contribs), which,
                                stream or None))


def zero_step_units_overlapped(plan: int, unit_contribs: Sequence[int], gather_bufs: Sequence[int],
                               hyper: zero_hyper_t, compute_stream: int, comm_stream: Optional[int],
                               wait: bool = True) -> Optional[zero_step_result_t]:
    """comm_stream None / 0: the one-stream schedule (unit u+1's gather inside unit u's step)."""
    res = zero_step_result_t() if wait else None
    _check(lib().zero_step_units_overlapped(plan, _ptr_array(unit_contribs), len(unit_contribs),
                                            _ptr_array(gather_bufs), ctypes.byref(hyper),
                                            compute_stream or None, comm_stream or None,
                                            ctypes.byref(res) if res is not None else None))
    return res


def zero_bind_offload(plan: int, rank: int, master: int, m: int, v: int, grad_host: int,
                      param16_host: int, shard16: Optional[int], full16: Optional[int],
                      workspace: int) -> None:
    _check(lib().zero_bind_offload(plan, rank, master or None, m or None, v or None,
                                   grad_host or None, param16_host or None, shard16 or None,
                                   full16 or None, workspace or None))


def zero_offload_step(plan: int, grad_contribs: Sequence[int], which: int, hyper: zero_hyper_t,
                      stream: int = 0) -> None:
    _check(lib().zero_offload_step(plan, _ptr_array(grad_contribs), len(grad_contribs), which,
                                   ctypes.byref(hyper), stream or None))


def zero_offload_finish(plan: int, threads: int, stream: int = 0,
                        wait: bool = True) -> Optional[zero_step_result_t]:
    res = zero_step_result_t() if wait else None
    _check(lib().zero_offload_finish(plan, threads, stream or None,
                                     ctypes.byref(res) if res is not None else None), res)
    return res


def zero_bind_host_staging(plan: int, staging: Sequence[int], bytes_each: int) -> None:
    _check(lib().zero_bind_host_staging(plan, _ptr_array(staging), bytes_each))


def zero_step_host(plan: int, host_contribs: Sequence[int], which: int, hyper: zero_hyper_t,
                   host_out16: int, stream: int = 0) -> None:
    _check(lib().zero_step_host(plan, _ptr_array(host_contribs), len(host_contribs), which,
                                ctypes.byref(hyper), host_out16 or None, stream or None))


def zero_grad_norm_host(plan: int, host_contribs: Sequence[int], which: int, stream: int = 0) -> None:
    _check(lib().zero_grad_norm_host(plan, _ptr_array(host_contribs), len(host_contribs), which,
                                     stream or None))


def zero_step_host_finish(plan: int, stream: int = 0) -> zero_step_result_t:
    """End a step that had zero_step_host calls (synchronises); returns the step state."""
    res = zero_step_result_t()
    _check(lib().zero_step_host_finish(plan, stream or None, ctypes.byref(res)), res)
    return res


def zero_step_finish(plan: int, stream: int = 0, wait: bool = True) -> Optional[zero_step_result_t]:
    """Enqueue the commit; with wait=True also read back the step state (synchronises)."""
    res = zero_step_result_t() if wait else None
    _check(lib().zero_step_finish(plan, stream or None,
                                  ctypes.byref(res) if res is not None else None), res)
    return res


def zero_restore_state(plan: int, state: zero_step_result_t, stream: int = 0) -> None:
    _check(lib().zero_restore_state(plan, ctypes.byref(state), stream or None))


def zero_read_state(plan: int, stream: int = 0) -> zero_step_result_t:
    res = zero_step_result_t()
    _check(lib().zero_read_state(plan, stream or None, ctypes.byref(res)), res)
    return res


def zero_set_option(plan: int, option: int, value: int) -> None:
    """ZERO_OPT_STAGING (ZERO_STAGING_REGISTER_LOADS / _BULK / _AUTO), ZERO_OPT_WAIT_LIMIT_NS,
    ZERO_OPT_BULK_TILE, ZERO_OPT_BULK_STAGES (0 = chosen from N_d); the gather's
    ZERO_OPT_GATHER_STAGING, ZERO_OPT_GATHER_CHUNK, ZERO_OPT_GATHER_STAGES (0 = default);
    ZERO_OPT_HOST_PIPELINE (host-buffer steps: 1 pipelined, 0 serial)."""
    _check(lib().zero_set_option(plan, option, int(value)))


def zero_get_option(plan: int, option: int) -> int:
    """An option's value in effect, or ZERO_OPT_LAST_STEP_KERNEL (1 staged, 0 register loads)."""
    v = _i64()
    _check(lib().zero_get_option(plan, option, ctypes.byref(v)))
    return v.value


def zero_gather_layer(plan: int, unit: int, full_unit16: int, stream: int = 0) -> None:
    _check(lib().zero_gather_layer(plan, unit, full_unit16 or None, stream or None))


def zero_release_layer(plan: int, unit: int) -> None:
    _check(lib().zero_release_layer(plan, unit))


def zero_memory_report(plan: int) -> zero_mem_report_t:
    rep = zero_mem_report_t()
    _check(lib().zero_memory_report(plan, ctypes.byref(rep)))
    return rep


def zero_comm_report(plan: int) -> zero_comm_report_t:
    rep = zero_comm_report_t()
    _check(lib().zero_comm_report(plan, ctypes.byref(rep)))
    return rep


def zero_last_error() -> str:
    msg = lib().zero_last_error()
    return msg.decode() if msg else ""


def zero_plan_destroy(plan: int) -> None:
    if plan:
        lib().zero_plan_destroy(plan)


def zero_step_range_noalloc(grad_contribs: Sequence[int], n: int, dtype16: int, master_in: int,
                            m_in: int, v_in: int, master_out: int, m_out: int, v_out: int,
                            out16: int, hyper: zero_hyper_t, t: int, loss_scale: float = 1.0,
                            stream: int = 0) -> int:
    """Fused step over one flat range without any workspace; returns the non-finite flag."""
    flag = ctypes.c_int32(0)
    _check(lib().zero_step_range_noalloc(_ptr_array(grad_contribs), len(grad_contribs), n, dtype16,
                                         master_in or None, m_in or None, v_in or None,
                                         master_out or None, m_out or None, v_out or None,
                                         out16 or None, ctypes.byref(hyper), t, loss_scale,
                                         stream or None, ctypes.byref(flag)))
    return int(flag.value)


def zero_linear_workspace(args: zero_linear_t, backward: bool = False) -> int:
    """Bytes of workspace that zero_linear (or zero_linear_backward) needs for these arguments."""
    n = _i64()
    _check(lib().zero_linear_workspace(ctypes.byref(args), int(backward), ctypes.byref(n)))
    return n.value


def zero_linear(args: zero_linear_t, workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().zero_linear(ctypes.byref(args), workspace or None, workspace_bytes, stream or None))


def zero_linear_backward(args: zero_linear_t, workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().zero_linear_backward(ctypes.byref(args), workspace or None, workspace_bytes,
                                      stream or None))


def zero_gated_workspace(args: zero_gated_t, backward: bool = False) -> int:
    """Bytes of workspace that zero_gated (or zero_gated_backward) needs for these arguments."""
    n = _i64()
    _check(lib().zero_gated_workspace(ctypes.byref(args), int(backward), ctypes.byref(n)))
    return n.value


def zero_gated(args: zero_gated_t, workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().zero_gated(ctypes.byref(args), workspace or None, workspace_bytes, stream or None))


def zero_gated_backward(args: zero_gated_t, workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().zero_gated_backward(ctypes.byref(args), workspace or None, workspace_bytes,
                                     stream or None))


def zero_operators_check(stream: int = 0) -> None:
    """Raises ZERO_ETIMEOUT if a bounded wait of an operator's kernel ran out since the last call."""
    _check(lib().zero_operators_check(stream or None))


def zero_block_norm(args: zero_block_norm_t, stream: int = 0) -> None:
    _check(lib().zero_block_norm(ctypes.byref(args), stream or None))


def zero_block_norm_workspace(args: zero_block_norm_t) -> int:
    """Bytes of workspace that zero_block_norm_backward needs for these arguments."""
    n = _i64()
    _check(lib().zero_block_norm_workspace(ctypes.byref(args), ctypes.byref(n)))
    return n.value


def zero_block_norm_backward(args: zero_block_norm_t, workspace: int, workspace_bytes: int,
                             stream: int = 0) -> None:
    _check(lib().zero_block_norm_backward(ctypes.byref(args), workspace or None, workspace_bytes,
                                          stream or None))


def zero_adamw_create(tensor_sizes: Sequence[int], state_bits: int, dtype16: int = ZERO_BF16,
                      grad_type: int = ZERO_BF16) -> int:
    out = _vp()
    _check(lib().zero_adamw_create(_i64_array(tensor_sizes), len(tensor_sizes), state_bits, dtype16,
                                   grad_type, ctypes.byref(out)))
    return int(out.value)


def zero_adamw_info(handle: int) -> zero_adamw_info_t:
    info = zero_adamw_info_t()
    _check(lib().zero_adamw_info(handle, ctypes.byref(info)))
    return info


def zero_adamw_bind(handle: int, params: Sequence[int], params16: Optional[Sequence[Optional[int]]],
                    grads: Sequence[int], m: int, v: int, scales: Optional[int], workspace: int,
                    t: int = 0, stream: int = 0) -> None:
    n = zero_adamw_info(handle).n_tensors
    for ptrs in (params, grads) + ((params16,) if params16 is not None else ()):
        if len(ptrs) != n:
            raise ValueError(f"zero_adamw_bind: {len(ptrs)} pointers for {n} tensors")
    _check(lib().zero_adamw_bind(handle, _ptr_array(params),
                                 _ptr_array(params16) if params16 is not None else None,
                                 _ptr_array(grads), m or None, v or None, scales or None,
                                 workspace or None, t, stream or None))


def zero_adamw_step(handle: int, hyper: zero_hyper_t, loss_scale: float = 1.0, stream: int = 0) -> None:
    _check(lib().zero_adamw_step(handle, ctypes.byref(hyper), loss_scale, stream or None))


def zero_adamw_check(handle: int, plan: int, stream: int = 0) -> None:
    """Make the optimizer's gradients part of the plan's step: its skip decision and its norm."""
    _check(lib().zero_adamw_check(handle, plan, stream or None))


def zero_adamw_step_with(handle: int, plan: int, hyper: zero_hyper_t, stream: int = 0) -> None:
    """The optimizer's part of the plan's open step, before its finish; see include/zero.h."""
    _check(lib().zero_adamw_step_with(handle, plan, ctypes.byref(hyper), stream or None))


def zero_adamw_export(handle: int, m_out: int, root_out: int, stream: int = 0) -> None:
    _check(lib().zero_adamw_export(handle, m_out or None, root_out or None, stream or None))


def zero_adamw_read(handle: int, stream: int = 0) -> zero_step_result_t:
    res = zero_step_result_t()
    _check(lib().zero_adamw_read(handle, stream or None, ctypes.byref(res)), res)
    return res


def zero_adamw_destroy(handle: int) -> None:
    if handle:
        lib().zero_adamw_destroy(handle)


def zero_muon_create(rows: Sequence[int], cols: Sequence[int], n_contribs: int = 1, dtype16: int = ZERO_BF16) -> int:
    if len(rows) != len(cols):
        raise ValueError(f"zero_muon_create: {len(rows)} row counts for {len(cols)} column counts")
    out = _vp()
    _check(lib().zero_muon_create(_i64_array(rows), _i64_array(cols), len(rows), n_contribs, dtype16, ctypes.byref(out)))
    return int(out.value)


def zero_muon_info(handle: int) -> zero_muon_info_t:
    info = zero_muon_info_t()
    _check(lib().zero_muon_info(handle, ctypes.byref(info)))
    return info


def zero_muon_set_option(handle: int, option: int, value: int) -> None:
    """ZERO_MUON_OPT_WAIT_LIMIT_NS, ZERO_MUON_OPT_SMS; see include/zero.h."""
    _check(lib().zero_muon_set_option(handle, option, int(value)))


def zero_muon_bind(handle: int, params: Optional[Sequence[Optional[int]]], params16: Optional[Sequence[Optional[int]]],
                   updates: Optional[Sequence[Optional[int]]], grads: Sequence[int], momentum: Sequence[int],
                   workspace: int, t: int = 0, stream: int = 0) -> None:
    """grads: contribution r of matrix i at r * n_matrices + i; see include/zero.h."""
    info = zero_muon_info(handle)
    n = info.n_matrices
    for ptrs in (params, params16, updates):
        if ptrs is not None and len(ptrs) != n:
            raise ValueError(f"zero_muon_bind: {len(ptrs)} pointers for {n} matrices")
    if len(momentum) != 2:
        raise ValueError("zero_muon_bind: the momentum has two halves")
    if len(grads) != n * info.n_contribs:
        raise ValueError(f"zero_muon_bind: {len(grads)} pointers for {info.n_contribs} contributions of {n} matrices")
    lists = [_ptr_array(ptrs) if ptrs is not None else None for ptrs in (params, params16, updates)]
    _check(lib().zero_muon_bind(handle, *lists, _ptr_array(grads), _ptr_array(momentum), workspace or None, t,
                                stream or None))


def zero_muon_step(handle: int, hyper: zero_muon_hyper_t, loss_scale: float = 1.0, stream: int = 0) -> None:
    _check(lib().zero_muon_step(handle, ctypes.byref(hyper), loss_scale, stream or None))


def zero_muon_check(handle: int, plan: int, hyper: zero_muon_hyper_t, stream: int = 0) -> None:
    """Form the momentum as part of the plan's step: its loss scale and its skip decision."""
    _check(lib().zero_muon_check(handle, plan, ctypes.byref(hyper), stream or None))


def zero_muon_step_with(handle: int, plan: int, hyper: zero_muon_hyper_t, stream: int = 0) -> None:
    """The optimizer's part of the plan's open step, before its finish; see include/zero.h."""
    _check(lib().zero_muon_step_with(handle, plan, ctypes.byref(hyper), stream or None))


def zero_muon_read(handle: int, stream: int = 0) -> zero_step_result_t:
    res = zero_step_result_t()
    _check(lib().zero_muon_read(handle, stream or None, ctypes.byref(res)), res)
    return res


def zero_muon_destroy(handle: int) -> None:
    if handle:
        lib().zero_muon_destroy(handle)


def muon_hyper(lr=2e-4, momentum=0.95, weight_decay=0.1, eps=1e-7, steps=5, coefficients=(3.4445, -4.7750, 2.0315),
               nesterov=True, scale=ZERO_MUON_SCALE_RMS) -> zero_muon_hyper_t:
    """coefficients: a, b, c, or one such triple for each step."""
    h = zero_muon_hyper_t(lr, momentum, weight_decay, eps, steps=steps, scale=scale,
                          flags=ZERO_MUON_NESTEROV if nesterov else 0)
    each = list(coefficients)
    if each and not hasattr(each[0], "__len__"):
        each = [each] * ZERO_MUON_MAX_STEPS
    if len(each) < steps:
        raise ValueError(f"muon_hyper: coefficients of {len(each)} steps for {steps}")
    for k, abc in enumerate(each[:ZERO_MUON_MAX_STEPS]):
        h.coefficients[k][:] = tuple(abc)
    return h


def hyper(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, max_grad_norm=0.0,
          report_grad_norm=False) -> zero_hyper_t:
    return zero_hyper_t(lr, beta1, beta2, eps, weight_decay, max_grad_norm,
                        ZERO_REPORT_GRAD_NORM if report_grad_norm else 0)


def scaler(scale=65536.0, growth_factor=2.0, backoff_factor=0.5, min_scale=1.0,
           growth_interval=1000, good_steps=0) -> zero_scaler_t:
    return zero_scaler_t(scale, growth_factor, backoff_factor, min_scale, growth_interval,
                         good_steps)
