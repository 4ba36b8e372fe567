"""ctypes loader of libbf16ops.so (argument types only; no computation here).

As with libbf16delta.so there is no fallback: if the shared library is missing and cannot be
built, loading fails with an error.
"""
from __future__ import annotations

import ctypes

from . import build as _build

c_u64, c_i64, c_u32, c_int = ctypes.c_uint64, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int
c_p, c_f, c_d = ctypes.c_void_p, ctypes.c_float, ctypes.c_double


class AdamWItem(ctypes.Structure):
    _fields_ = [("d_weight", c_p), ("d_out", c_p), ("d_grad", c_p), ("n", c_u64),
                ("first_block", c_u64), ("weight_decay", c_f), ("reserved", c_u32)]


class AdamWState(ctypes.Structure):
    _fields_ = [("d_m", c_p), ("d_v", c_p), ("d_m_scale", c_p), ("d_v_scale", c_p),
                ("d_master", c_p), ("blocks", c_u64)]


class AdamW(ctypes.Structure):
    _fields_ = [("state", AdamWState), ("d_control", c_p), ("d_chunks", c_p),
                ("d_partials", c_p), ("chunks", c_u64), ("weight_kind", c_u32),
                ("grad_dtype", c_u32), ("state_bits", c_u32), ("flags", c_u32), ("device", c_int)]


class AdamWStepArgs(ctypes.Structure):
    _fields_ = [("lr", c_f), ("d_lr", c_p), ("beta1", c_d), ("beta2", c_d), ("eps", c_f),
                ("max_norm", c_f), ("seed", c_u64)]


class Adapter(ctypes.Structure):
    _fields_ = [("d_down", c_p), ("d_up", c_p), ("ld_down", c_u64), ("ld_up", c_u64),
                ("d_grad_down", c_p), ("d_grad_up", c_p), ("ld_grad_down", c_u64),
                ("ld_grad_up", c_u64), ("rank", c_u32), ("scale", c_f)]


class AdapterSet(ctypes.Structure):
    _fields_ = [("d_table", c_p), ("k", c_u32), ("hidden", c_u32), ("out", c_u32),
                ("rank", c_u32), ("grad_dtype", c_u32), ("has_grads", c_u32),
                ("wide", c_u32), ("device", c_int)]


class AdapterRows(ctypes.Structure):
    _fields_ = [("d_perm", c_p), ("d_offsets", c_p), ("d_blocks", c_p), ("d_tiles", c_p * 3), ("d_ntiles", c_p),
                ("d_status", c_p),
                ("rows", c_u32), ("k", c_u32), ("device", c_int)]


class Logprobs(ctypes.Structure):
    _fields_ = [("d_logprobs", c_p), ("d_entropy", c_p), ("d_top_logprobs", c_p),
                ("d_top_tokens", c_p), ("d_saved", c_p), ("rows", c_u32), ("vocab", c_u32),
                ("top", c_u32), ("device", c_int)]


class Routing(ctypes.Structure):
    _fields_ = [("d_weights", c_p), ("d_experts", c_p), ("d_counts", c_p), ("d_probs", c_p),
                ("d_loss", c_p), ("d_real", c_p), ("d_partials", c_p), ("tokens", c_u32),
                ("experts", c_u32), ("k", c_u32), ("normalize", c_u32), ("device", c_int)]


# name -> (restype, argtypes); must match include/ops/bf16ops.h
SIGNATURES = {
    "bo_adamw_plan_size": (c_u64, [c_p, c_u32]),
    "bo_adamw_plan": (c_int, [c_p, c_u32, c_p, c_u32, c_u32, c_u32, c_u32, c_i64, c_p, c_u64, c_p,
                              c_p]),
    "bo_adamw_step": (c_int, [c_p, c_p, c_p]),
    "bo_adamw_norm": (c_int, [c_p, c_f, c_p]),
    "bo_adamw_moments": (c_int, [c_p, c_u32, c_p, c_p, c_p]),
    "bo_adapter_set_size": (c_u64, [c_u32]),
    "bo_adapter_set_init": (c_int, [c_p, c_u32, c_u32, c_u32, c_u32, c_p, c_u64, c_p, c_p]),
    "bo_adapter_rows_size": (c_u64, [c_u32, c_u32]),
    "bo_adapter_rows_init": (c_int, [c_p, c_u32, c_u32, c_p, c_u64, c_p, c_p, c_p]),
    "bo_adapter_forward": (c_int, [c_p, c_p, c_p, c_u64, c_p, c_u64, c_p, c_p]),
    "bo_adapter_low_rows": (c_u32, [c_p]),
    "bo_adapter_backward_workspace_size": (c_u64, [c_p, c_u32]),
    "bo_adapter_backward": (c_int, [c_p, c_p, c_p, c_u64, c_p, c_u64, c_p, c_p, c_u64, c_int, c_p,
                                    c_u64, c_p]),
    "bo_logprobs_size": (c_u64, [c_u32, c_u32, c_u32, c_u32]),
    "bo_logprobs_init": (c_int, [c_u32, c_u32, c_u32, c_u32, c_p, c_u64, c_p, c_p]),
    "bo_logprobs_forward": (c_int, [c_p, c_p, c_u32, c_u64, c_u32, c_p, c_u32, c_u64, c_f, c_p, c_u64,
                                    c_p]),
    "bo_logprobs_backward": (c_int, [c_p, c_p, c_u32, c_u64, c_u32, c_p, c_u64, c_p, c_u64, c_p, c_u64,
                                     c_p]),
    "bo_routing_size": (c_u64, [c_u32, c_u32, c_u32]),
    "bo_routing_init": (c_int, [c_u32, c_u32, c_u32, c_u32, c_p, c_u64, c_p, c_p]),
    "bo_routing_forward": (c_int, [c_p, c_p, c_u32, c_u64, c_u32, c_p, c_u64, c_p]),
    "bo_routing_backward": (c_int, [c_p, c_p, c_u32, c_u64, c_u32, c_p, c_u64, c_u64, c_f, c_p, c_p,
                                    c_p, c_u64, c_p]),
    "bo_status_string": (ctypes.c_char_p, [c_int]),
}

_lib = None


def path() -> str:
    return _build.OPS_LIB


def load():
    """Returns the loaded library, building it first when it is missing or stale."""
    global _lib
    if _lib is None:
        if not _build.up_to_date(_build.OPS_LIB):
            try:
                _build.build()
            except Exception as e:  # no fallback path exists
                raise RuntimeError(f"libbf16ops.so is missing and could not be built: {e}") from e
        lib = ctypes.CDLL(_build.OPS_LIB)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib
