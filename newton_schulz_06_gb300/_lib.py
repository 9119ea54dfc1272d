"""ctypes binding of libmuon's C ABI (include/muon.h): marshalling only.

Every function here forwards to the library with the same name; there is no
computation and no fallback.  What is loaded is libmuon_torch.so: libmuon.so's
code on the process's CUDA runtime (build.py).  If it has not been built the
first use raises, so a missing extension can never turn into a silent CPU path.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmuon_torch.so")

MUON_OK = 0
MUON_ERR_INVALID_ARG = -1
MUON_ERR_UNSUPPORTED = -2
MUON_ERR_NO_WORKSPACE = -3
MUON_ERR_CUDA = -4
MUON_ERR_TIMEOUT = -5
MUON_ERR_STATE = -6
MUON_F32 = 0
MUON_BF16 = 1
MUON_FULL = 0
MUON_BLOCKWISE = 1
MUON_DISTRIBUTED = 2
MUON_HOST_ONLY = -1
MUON_N_STAGES = 8
STAGE_NAMES = ("momentum", "norm", "normalise", "syrk1", "syrk2", "gemm",
               "update", "chain")

# Every entry point include/muon.h declares.
EXPORTS = ("muon_create", "muon_set_stream", "muon_register_params",
           "muon_workspace_size", "muon_set_workspace", "muon_step",
           "muon_sync", "muon_destroy", "muon_last_error",
           "muon_set_profiling", "muon_stage_times", "muon_last_launch_count",
           "muon_debug_set_exports", "muon_get_plan_info",
           "muon_step_noalloc", "muon_debug_wait_timeout", "muon_step_host",
           "muon_debug_check_chain_schedule", "muon_debug_set_chain_test",
           "muon_dist_configure", "muon_dist_momentum", "muon_dist_gram",
           "muon_dist_update",
           "muon_ckpt8_pack", "muon_ckpt8_unpack", "muon_layer_norm",
           "muon_layer_norm_grad_workspace", "muon_layer_norm_grad",
           "muon_weight_grad_workspace", "muon_weight_grad",
           "muon_route_workspace", "muon_route", "muon_route_grad",
           "muon_gated_ffn_workspace", "muon_gated_ffn",
           "muon_gated_ffn_grad_workspace", "muon_gated_ffn_grad",
           "muon_rotary", "muon_rotary_frequencies", "muon_dropout",
           "muon_ops_sync", "muon_debug_ops_wait_timeout",
           "muon_debug_ffn_wait_timeout")


class MuonParam(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld_w", ctypes.c_int64),
                ("ld_g", ctypes.c_int64), ("ld_m", ctypes.c_int64),
                ("w_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32)]


class MuonPlanInfo(ctypes.Structure):
    _fields_ = [("units", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("syrk_tiles", ctypes.c_int64), ("gemm_tiles", ctypes.c_int64),
                ("ew_tiles", ctypes.c_int64),
                ("useful_flops", ctypes.c_int64),
                ("executed_flops", ctypes.c_int64),
                ("chained_groups", ctypes.c_int64)]


def _struct(name, *groups):
    """A ctypes structure from (C type, "field names") groups in order."""
    return type(name, (ctypes.Structure,),
                {"_fields_": [(f, t) for t, names in groups for f in names.split()]})


_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_u64, _f64 = ctypes.c_uint64, ctypes.c_double
Ckpt8 = _struct("Ckpt8", (_vp, "q e"), (_i64, "ld_q ld_e"))
LayerNormArgs = _struct("LayerNormArgs", (_vp, "x weight bias y mean rstd"), (Ckpt8, "saved"),
                        (_i64, "rows cols ld_x ld_y"), (_i32, "x_dtype w_dtype"), (_f32, "eps"))
LayerNormGradArgs = _struct("LayerNormGradArgs",
                            (_vp, "dy x mean rstd weight dx dweight dbias"), (Ckpt8, "saved"),
                            (_i64, "rows cols ld_dy ld_x ld_dx"), (_i32, "x_dtype w_dtype"))
WeightGradArgs = _struct("WeightGradArgs", (_vp, "dy weight bias c g offsets"), (Ckpt8, "saved"),
                         (_i64, "rows n k experts ld_dy ld_c ld_g stride_c stride_g"),
                         (_i32, "g_dtype w_dtype"))
RouteArgs = _struct("RouteArgs",
                    (_vp, "logits mask indices weights counts offsets loss kept"),
                    (_i64, "tokens experts k ld_z"), (_i32, "z_dtype renormalise"),
                    (_f32, "coef"))
RouteGradArgs = _struct("RouteGradArgs",
                        (_vp, "logits indices weights counts kept dloss dweights dlogits"),
                        (_i64, "tokens experts k ld_z ld_dw ld_dz"),
                        (_i32, "z_dtype renormalise"), (_f32, "coef"))

GatedFfnArgs = _struct("GatedFfnArgs", (_vp, "x w_gate w_up w_down y gate up offsets"),
                       (_i64, "rows hidden inner experts ld_x ld_gate ld_up ld_down ld_y ld_kept "
                              "stride_gate stride_up stride_down"), (_i32, "activation"))
GatedFfnGradArgs = _struct("GatedFfnGradArgs",
                           (_vp, "dy x gate up w_gate w_up w_down dx dw_gate dw_up dw_down dgate dup h "
                                 "offsets"),
                           (_i64, "rows hidden inner experts ld_dy ld_x ld_kept ld_gate ld_up ld_down "
                                  "ld_dx ld_d ld_dw_gate ld_dw_up ld_dw_down stride_gate stride_up "
                                  "stride_down stride_dw_gate stride_dw_up stride_dw_down"),
                           (_i32, "activation g_dtype accumulate"))
RotaryTensor = _struct("RotaryTensor", (_vp, "x y"), (_i64, "heads x_batch x_seq x_head y_batch y_seq y_head"))
RotaryArgs = _struct("RotaryArgs", (RotaryTensor, "q k"), (_vp, "positions turns"),
                     (_i64, "batch seq head pairs stride_positions offset"),
                     (_i32, "x_dtype layout positions_64 inverse"), (_f32, "scale"))
DropoutArgs = _struct("DropoutArgs", (_vp, "x residual y counter"), (_i64, "rows cols ld_x ld_r ld_y"),
                      (_u64, "seed offset"), (_f64, "p"), (_i32, "x_dtype"))


def packer(cls):
    """struct.Struct that packs a structure's fields in order, nested ones in
    line (several times faster than filling the ctypes object): its bytes can
    be passed where a pointer to the structure is expected."""
    code = {_vp: "Q", _i64: "q", _i32: "i", _f32: "f", _u64: "Q", _f64: "d"}
    flat = []

    def walk(c, base):
        for name, t in c._fields_:
            at = base + getattr(c, name).offset
            if t in code:
                flat.append((at, ctypes.sizeof(t), code[t]))
            else:
                walk(t, at)

    walk(cls, 0)
    fmt, end = "<", 0
    for at, size, c in flat:
        fmt += f"{at - end}x" * (at > end) + c
        end = at + size
    return struct.Struct(fmt + f"{ctypes.sizeof(cls) - end}x" * (ctypes.sizeof(cls) > end))


class MuonError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"libmuon error {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmuon_torch.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m newton_schulz_06_gb300.build` (or "
            "__graft_entry__.build()); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    H = ctypes.c_void_p
    vp = ctypes.c_void_p
    i32 = ctypes.c_int
    f32 = ctypes.c_float
    sz = ctypes.c_size_t
    sig = {
        "muon_create": [ctypes.POINTER(H), i32, vp],
        "muon_set_stream": [H, vp],
        "muon_register_params": [H, i32, ctypes.POINTER(MuonParam)],
        "muon_workspace_size": [H, i32, i32, ctypes.POINTER(sz),
                                ctypes.POINTER(sz)],
        "muon_set_workspace": [H, vp, sz],
        "muon_step": [H, f32, f32, i32, i32, f32, f32, f32, i32, i32],
        "muon_sync": [H],
        "muon_destroy": [H],
        "muon_last_error": [H],
        "muon_set_profiling": [H, i32],
        "muon_stage_times": [H, ctypes.POINTER(f32), ctypes.POINTER(i32),
                             i32],
        "muon_last_launch_count": [H],
        "muon_debug_set_exports": [H, i32, ctypes.POINTER(vp),
                                   ctypes.POINTER(vp)],
        "muon_get_plan_info": [H, i32, i32, ctypes.POINTER(MuonPlanInfo)],
        "muon_step_noalloc": [ctypes.POINTER(MuonParam), f32, f32, i32, i32,
                              f32, f32, f32, vp, ctypes.c_char_p, sz],
        "muon_debug_wait_timeout": [H, vp, i32],
        "muon_debug_check_chain_schedule": [H, i32, i32],
        "muon_debug_set_chain_test": [H, i32],
        "muon_step_host": [H, i32, ctypes.POINTER(vp), ctypes.POINTER(vp), f32,
                           f32, i32, i32, f32, f32, f32, i32, i32],
        "muon_dist_configure": [H, i32, f32],
        "muon_dist_momentum": [H, f32, i32, vp],
        "muon_dist_gram": [H, vp, ctypes.c_int64, i32, i32],
        "muon_dist_update": [H, vp, ctypes.c_int64, i32, i32, vp, f32, f32, f32,
                             f32],
        # the operators' argument structures go by address (ctypes.byref)
        "muon_ckpt8_pack": [vp, i32, _i64, _i64, _i64, vp, vp, vp, sz],
        "muon_ckpt8_unpack": [vp, _i64, _i64, vp, i32, _i64, vp, vp, sz],
        "muon_layer_norm": [vp, vp, vp, sz],
        "muon_layer_norm_grad_workspace": [vp, ctypes.POINTER(sz)],
        "muon_layer_norm_grad": [vp, vp, sz, vp, vp, sz],
        "muon_weight_grad_workspace": [vp, ctypes.POINTER(sz)],
        "muon_weight_grad": [vp, vp, sz, vp, vp, sz],
        "muon_route_workspace": [vp, ctypes.POINTER(sz)],
        "muon_route": [vp, vp, sz, vp, vp, sz],
        "muon_route_grad": [vp, vp, vp, sz],
        "muon_gated_ffn_workspace": [vp, ctypes.POINTER(sz)],
        "muon_gated_ffn": [vp, vp, sz, vp, vp, sz],
        "muon_gated_ffn_grad_workspace": [vp, ctypes.POINTER(sz)],
        "muon_gated_ffn_grad": [vp, vp, sz, vp, vp, sz],
        "muon_rotary": [vp, vp, vp, sz],
        "muon_rotary_frequencies": [_i64, _f64, i32, _f64, _f64, _f64, _f64, vp, vp, vp, sz],
        "muon_dropout": [vp, vp, vp, sz],
        "muon_ops_sync": [vp, vp, sz],
        "muon_debug_ops_wait_timeout": [i32, vp, vp, sz],
        "muon_debug_ffn_wait_timeout": [i32, vp, vp, sz],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "muon_last_error" else i32
    _lib = L
    return L


def check(rc: int, handle=None) -> int:
    if rc < 0:
        msg = lib().muon_last_error(handle).decode(errors="replace")
        raise MuonError(rc, msg)
    return rc
