"""ctypes mirror of include/moe.h and loader of the in-tree libmoe.so.

Argument marshalling only: every step of the branch runs in the HIP library.
Loading fails loudly if the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_LIB selects another build of the library (e.g. the host-sanitized one)
LIB_PATH = os.environ.get("MOE_LIB") or os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16 = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_HIP"}


class MoeConfig(C.Structure):
    _fields_ = [
        ("T", C.c_int64),
        ("d_model", C.c_int32), ("d_latent", C.c_int32), ("n_experts", C.c_int32),
        ("n_pools", C.c_int32), ("top_k", C.c_int32), ("d_ff", C.c_int32),
        ("n_shared", C.c_int32), ("d_ff_shared", C.c_int32), ("n_waves", C.c_int32),
        ("send_cap_num", C.c_int32), ("send_cap_den", C.c_int32),
        ("recv_cap_num", C.c_int32), ("recv_cap_den", C.c_int32),
        ("cap_send_rows", C.c_int64), ("cap_recv_rows", C.c_int64),
        ("dtype", C.c_int32), ("reserved", C.c_int32),
    ]


class MoePlan(C.Structure):
    _fields_ = [(n, C.c_int64) for n in (
        "tokens_per_wave", "cap_send", "cap_recv", "experts_per_pool", "elem_bytes",
        "row_bytes", "pool_block_bytes", "ids_offset", "pools_bytes", "expert_out_bytes",
        "max_expert_rows", "dispatch_ws_bytes", "experts_ws_bytes", "forward_ws_bytes",
        "dropless_rows", "dropless_dispatch_ws_bytes", "dropless_experts_ws_bytes",
        "dropless_forward_ws_bytes", "backward_rows", "experts_bwd_ws_bytes",
        "backward_ws_bytes", "dropless_backward_rows", "dropless_experts_bwd_ws_bytes",
        "dropless_backward_ws_bytes")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class MoeWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "w_latent", "w_router", "router_bias", "w_gate", "w_up", "w_down", "w_up_proj",
        "ws_gate", "ws_up", "ws_down")]


class MoeTaps(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "logits", "topk_idx", "gates", "pool_slot", "recv_slot", "pool_count",
        "expert_count", "bank_rows", "z", "pools", "expert_out", "y_latent")]


class MoeDroplessTaps(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "logits", "topk_idx", "gates", "row_of", "expert_offsets", "z", "xs", "expert_out",
        "y_latent")]


class MoeScoring(C.Structure):
    _fields_ = [("score", C.c_int32), ("n_groups", C.c_int32), ("top_groups", C.c_int32), ("group_top", C.c_int32),
                ("renormalise", C.c_int32), ("scale", C.c_float), ("reserved", C.c_int32)]


class MoeQuantGemm(C.Structure):
    _fields_ = [("M", C.c_int64), ("N", C.c_int64), ("K", C.c_int64), ("a", C.c_void_p), ("lda", C.c_int64),
                ("a_scale", C.c_void_p), ("a_scale_ld", C.c_int64), ("b", C.c_void_p), ("ldb", C.c_int64),
                ("b_scale", C.c_void_p), ("b_scale_ld", C.c_int64), ("c", C.c_void_p), ("ldc", C.c_int64),
                ("b_block_rows", C.c_int32), ("out_dtype", C.c_int32), ("reserved", C.c_int32)]


class MoeQuantExperts(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("q_gate", "s_gate", "q_up", "s_up", "q_down", "s_down")]


class MoeQuantWeights(C.Structure):
    _fields_ = ([(n, C.c_void_p) for n in ("q_latent", "s_latent", "w_router", "router_bias")]
                + [("experts", MoeQuantExperts)]
                + [(n, C.c_void_p) for n in ("q_shared_gate", "s_shared_gate", "q_shared_up", "s_shared_up", "q_output",
                                             "s_output")])


class MoeLinearArgs(C.Structure):
    _fields_ = [("M", C.c_int64), ("N", C.c_int64), ("K", C.c_int64), ("x", C.c_void_p), ("ldx", C.c_int64),
                ("w", C.c_void_p), ("ldw", C.c_int64), ("bias", C.c_void_p), ("residual", C.c_void_p),
                ("ldr", C.c_int64), ("y", C.c_void_p), ("ldy", C.c_int64), ("pre", C.c_void_p), ("ldp", C.c_int64),
                ("act", C.c_int32), ("bias_dtype", C.c_int32), ("out_dtype", C.c_int32), ("reserved", C.c_int32)]


class MoeLinearGrad(C.Structure):
    _fields_ = [("M", C.c_int64), ("N", C.c_int64), ("K", C.c_int64), ("dy", C.c_void_p), ("lddy", C.c_int64),
                ("pre", C.c_void_p), ("ldp", C.c_int64), ("x", C.c_void_p), ("ldx", C.c_int64), ("w", C.c_void_p),
                ("ldw", C.c_int64), ("dx", C.c_void_p), ("lddx", C.c_int64), ("dw", C.c_void_p), ("lddw", C.c_int64),
                ("db", C.c_void_p), ("act", C.c_int32), ("dy_dtype", C.c_int32), ("reserved", C.c_int32)]


class MoeOrthoArgs(C.Structure):
    _fields_ = [("batch", C.c_int64), ("M", C.c_int64), ("N", C.c_int64), ("g", C.c_void_p), ("ldg", C.c_int64),
                ("stride_g", C.c_int64), ("out", C.c_void_p), ("ldo", C.c_int64), ("stride_o", C.c_int64),
                ("coeffs", C.POINTER(C.c_float)), ("steps", C.c_int32), ("dtype", C.c_int32), ("eps", C.c_float),
                ("scale", C.c_float), ("reserved", C.c_int32)]


ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}

# exported symbols and their signatures
_P = C.c_void_p
SIGNATURES = {
    "moe_status_string": (C.c_char_p, [C.c_int]),
    "moe_version": (C.c_int32, []),
    "moe_make_plan": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoePlan)]),
    "moe_route": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P]),
    "moe_router_bias_ws_bytes": (C.c_int, [C.POINTER(MoeConfig), C.c_int32, C.POINTER(C.c_size_t)]),
    "moe_router_bias_update": (C.c_int, [C.POINTER(MoeConfig), _P, C.c_int32, _P, _P, _P, _P,
                                         C.c_size_t, _P]),
    "moe_router_bias_stage_count": (C.c_int32, []),
    "moe_router_bias_update_profiled": (C.c_int, [C.POINTER(MoeConfig), _P, C.c_int32, _P, _P, _P, _P,
                                                  C.c_size_t, _P, _P, C.c_int32]),
    "moe_dispatch": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                               _P, C.c_size_t, _P]),
    "moe_dispatch_noalloc": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_noalloc_scratch_bytes": (C.c_int64, []),
    "moe_experts": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P, _P,
                              C.c_size_t, _P]),
    "moe_combine": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P]),
    "moe_forward": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights), _P, _P,
                              C.POINTER(MoeTaps), _P, _P, C.c_size_t, _P]),
    "moe_forward_stage_count": (C.c_int32, []),
    "moe_forward_profiled": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights), _P, _P,
                                       C.POINTER(MoeTaps), _P, _P, C.c_size_t, _P,
                                       C.POINTER(C.c_void_p), C.c_int32]),
    "moe_dispatch_dropless": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P,
                                        C.c_size_t, _P]),
    "moe_experts_dropless": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P,
                                       C.c_size_t, _P]),
    "moe_combine_dropless": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P]),
    "moe_forward_dropless": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights), _P, _P,
                                       C.POINTER(MoeDroplessTaps), _P, _P, C.c_size_t, _P]),
    "moe_forward_dropless_stage_count": (C.c_int32, []),
    "moe_forward_dropless_profiled": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights),
                                                _P, _P, C.POINTER(MoeDroplessTaps), _P, _P,
                                                C.c_size_t, _P, C.POINTER(C.c_void_p),
                                                C.c_int32]),
    "moe_combine_backward": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_experts_backward": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                       _P, _P, _P, C.c_size_t, _P]),
    "moe_dispatch_backward": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P]),
    "moe_route_backward": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P]),
    "moe_backward_routed": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights),
                                      C.POINTER(MoeTaps), _P, _P, _P, _P, _P, _P, _P,
                                      C.c_size_t, _P]),
    "moe_backward_routed_stage_count": (C.c_int32, []),
    "moe_combine_backward_dropless": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P]),
    "moe_experts_backward_dropless": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P, _P, _P, _P,
                                                _P, _P, _P, _P, C.c_size_t, _P]),
    "moe_dispatch_backward_dropless": (C.c_int, [C.POINTER(MoeConfig), _P, _P, _P, _P]),
    "moe_backward_dropless": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights),
                                        C.POINTER(MoeDroplessTaps), _P, _P, _P, _P, _P, _P, _P,
                                        C.c_size_t, _P]),
    "moe_backward_dropless_profiled": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights),
                                                 C.POINTER(MoeDroplessTaps), _P, _P, _P, _P, _P,
                                                 _P, _P, C.c_size_t, _P, C.POINTER(C.c_void_p),
                                                 C.c_int32]),
    "moe_backward_routed_profiled": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights),
                                               C.POINTER(MoeTaps), _P, _P, _P, _P, _P, _P, _P,
                                               C.c_size_t, _P, C.POINTER(C.c_void_p),
                                               C.c_int32]),
    "moe_route_scored": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeScoring), _P, _P, _P, _P, _P]),
    "moe_route_scored_backward": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeScoring), _P, _P, _P, _P, _P]),
    "moe_quantize": (C.c_int, [C.c_int64, C.c_int64, _P, C.c_int64, C.c_int32, C.c_int32, C.c_int32, _P, _P, _P]),
    "moe_gemm_quant_ws_bytes": (C.c_int, [C.POINTER(MoeQuantGemm), C.POINTER(C.c_size_t)]),
    "moe_gemm_quant": (C.c_int, [C.POINTER(MoeQuantGemm), _P, C.c_size_t, _P]),
    "moe_experts_dropless_quant_ws_bytes": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(C.c_size_t)]),
    "moe_forward_dropless_quant_ws_bytes": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(C.c_size_t)]),
    "moe_forward_dropless_quant": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeScoring), C.POINTER(MoeQuantWeights), _P,
                                             _P, C.POINTER(MoeDroplessTaps), _P, _P, C.c_size_t, _P]),
    "moe_experts_dropless_quant": (C.c_int, [C.POINTER(MoeConfig), _P, _P, C.POINTER(MoeQuantExperts), _P, _P,
                                             C.c_size_t, _P]),
    "moe_linear_ws_bytes": (C.c_int, [C.POINTER(MoeLinearArgs), C.POINTER(C.c_size_t)]),
    "moe_linear": (C.c_int, [C.POINTER(MoeLinearArgs), _P, C.c_size_t, _P]),
    "moe_linear_backward_ws_bytes": (C.c_int, [C.POINTER(MoeLinearGrad), C.POINTER(C.c_size_t)]),
    "moe_linear_backward": (C.c_int, [C.POINTER(MoeLinearGrad), _P, C.c_size_t, _P]),
    "moe_forward_few_ws_bytes": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(C.c_size_t)]),
    "moe_forward_few": (C.c_int, [C.POINTER(MoeConfig), C.POINTER(MoeWeights), _P, _P, _P, _P, _P, _P, _P, C.c_size_t,
                                  _P]),
    "moe_orthogonalize_ws_bytes": (C.c_int, [C.POINTER(MoeOrthoArgs), C.POINTER(C.c_size_t)]),
    "moe_orthogonalize": (C.c_int, [C.POINTER(MoeOrthoArgs), _P, C.c_size_t, _P]),
}

STAGES = ["latent", "router", "topk", "assign", "scatter", "recv_bin", "expert_rows",
          "expert_gate_up", "expert_down", "combine", "shared_gate_up", "output"]
DROPLESS_STAGES = ["latent", "router", "topk", "sort", "scatter", "tiles", "expert_gate_up",
                   "expert_down", "combine", "shared_gate_up", "output"]
BIAS_STAGES = ["bias_range", "bias_hist", "bias_quantile", "bias_mean"]
BACKWARD_STAGES = ["combine_bwd", "layout", "gather", "dh", "swiglu_bwd", "du", "dw_down",
                   "dw_gate", "dw_up", "dispatch_bwd", "route_bwd"]

_lib = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Load libmoe.so (cached).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing; build it with `python -m routing_capacity_dispatch_amd.build`")
    lib = C.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")


def check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)
