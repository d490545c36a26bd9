"""ctypes declarations of the libmuon C ABI (include/muon.h).

Loading is lazy: importing the package works without the library (e.g. to
use the workload generator), but every call into the library fails loudly
when libmuon.so has not been built.  There is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# MUON_LIB selects another build of the same library (e.g. the host
# AddressSanitizer build of build.py --asan); the default is the in-place one.
LIB_PATH = os.environ.get("MUON_LIB") or os.path.join(_HERE, "libmuon.so")

MUON_OK = 0
MUON_EINVAL = -1
MUON_EWORKSPACE = -2
MUON_EHIP = -3
MUON_EALIAS = -4
MUON_ECAPTURE = -5
MUON_ENONFINITE = -6

MUON_F32 = 0
MUON_BF16 = 1

MUON_SCALE_NONE = 0
MUON_SCALE_SQRT_MAX1 = 1

MUON_OPT_ZERO_CENTER = 1
MUON_OPT_NESTEROV = 2
MUON_OPT_NS_FIRST = 4

MUON_PHASES = 8
PHASE_NAMES = ("momentum_norm", "normalize_cast", "gram", "gram2_epilogue", "x_update", "apply",
               "adamw", "ns_fused")

EXPORTED = ("muon_workspace_bytes", "muon_step", "muon_step_ex", "muon_plan_create",
            "muon_plan_step", "muon_plan_destroy", "muon_orthogonalize",
            "muon_workspace_view",
            "muon_adamw_workspace_bytes", "muon_adamw_step",
            "muon_timing_enable", "muon_timing_read", "muon_status_string", "muon_version",
            "muon_step_noalloc", "muon_noalloc_scratch",
            "muon_act8_pack", "muon_act8_unpack",
            "muon_rmsnorm_act8", "muon_rmsnorm_act8_grad_workspace_bytes", "muon_rmsnorm_act8_grad",
            "muon_swiglu_act8", "muon_swiglu_act8_grad",
            "muon_act8_wgrad_workspace_bytes", "muon_act8_wgrad",
            "muon_embed", "muon_embed_grad_workspace_bytes", "muon_embed_grad",
            "muon_attention", "muon_attention_workspace_bytes", "muon_attention_grad_workspace_bytes", "muon_attention_grad",
            "muon_distill", "muon_policy")


class MuonMatrix(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("momentum", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("grad_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class MuonOptions(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class MuonOrtho(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("in_dtype", ctypes.c_int32)]


class MuonCoeff(ctypes.Structure):
    _fields_ = [("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float)]


class MuonAdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("step", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonWorkspaceView(ctypes.Structure):
    _fields_ = [("x_off", ctypes.c_size_t * 2), ("a_off", ctypes.c_size_t),
                ("c_off", ctypes.c_size_t), ("c_lo_off", ctypes.c_size_t), ("o_off", ctypes.c_size_t),
                ("nrm2_off", ctypes.c_size_t), ("rows_pad", ctypes.c_int64),
                ("cols_pad", ctypes.c_int64), ("m_pad", ctypes.c_int64),
                ("transposed", ctypes.c_int32), ("tile", ctypes.c_int32)]


# Training operators (ops.py)
class MuonAct8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64)]


def _int64s(*names):
    return [(n, ctypes.c_int64) for n in names]


class MuonRmsnorm(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("gain", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n", MuonAct8),
                ("rstd", ctypes.c_void_p),
                *_int64s("rows", "cols", "ld_x", "ld_residual", "ld_h", "ld_y"),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class MuonRmsnormGrad(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("dres", ctypes.c_void_p), ("gain", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p), ("n", MuonAct8), ("dx", ctypes.c_void_p),
                ("dgain", ctypes.c_void_p),
                *_int64s("rows", "cols", "ld_dy", "ld_dres", "ld_dx"),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonSwiglu(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("a", ctypes.c_void_p),
                ("gate8", MuonAct8), ("up8", MuonAct8),
                *_int64s("rows", "cols", "ld_gate", "ld_up", "ld_a"),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonSwigluGrad(ctypes.Structure):
    _fields_ = [("da", ctypes.c_void_p), ("gate8", MuonAct8), ("up8", MuonAct8),
                ("dgate", ctypes.c_void_p), ("dup", ctypes.c_void_p), ("a8", MuonAct8),
                *_int64s("rows", "cols", "ld_da", "ld_dgate", "ld_dup"),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonAct8Wgrad(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("x8", MuonAct8), ("col_gain", ctypes.c_void_p),
                ("dw", ctypes.c_void_p), *_int64s("tokens", "n", "k", "ld_dy", "ld_dw"),
                ("dw_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class MuonEmbed(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("out", ctypes.c_void_p),
                *_int64s("tokens", "vocab", "cols", "ld_table", "ld_out"),
                ("scale", ctypes.c_float), ("table_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32)]


class MuonEmbedGrad(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("dtable", ctypes.c_void_p),
                *_int64s("tokens", "vocab", "cols", "ld_dy", "ld_dtable"),
                ("scale", ctypes.c_float), ("dy_dtype", ctypes.c_int32),
                ("table_dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld_token", ctypes.c_int64), ("ld_head", ctypes.c_int64)]


_ATTENTION = [("starts", ctypes.c_void_p), ("k_starts", ctypes.c_void_p),
              *_int64s("tokens", "k_tokens", "sequences", "heads", "kv_heads", "dim", "ld_lse"),
              ("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("zero_rest", ctypes.c_int32),
              ("reserved", ctypes.c_int32)]


class MuonAttention(ctypes.Structure):
    _fields_ = [*((n, MuonHeads) for n in ("q", "k", "v", "o")), ("lse", ctypes.c_void_p), *_ATTENTION]


class MuonAttentionGrad(ctypes.Structure):
    _fields_ = [*((n, MuonHeads) for n in ("dout", "q", "k", "v", "o", "dq", "dk", "dv")),
                ("lse", ctypes.c_void_p), *_ATTENTION]


class MuonDistill(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("logits", "ids", "teacher", "weights", "loss", "dlogits")),
                *_int64s("tokens", "vocab", "top", "ld_logits", "ld_ids", "ld_teacher", "ld_dlogits"),
                ("temperature", ctypes.c_float), ("dtype", ctypes.c_int32), ("teacher_dtype", ctypes.c_int32),
                ("id_bytes", ctypes.c_int32)]


class MuonPolicy(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("logits", "actions", "old_logp", "advantages", "ref_logp", "weights",
                                                 "loss", "logp", "dlogits")),
                *_int64s("tokens", "vocab", "ld_logits", "ld_dlogits"),
                *((n, ctypes.c_float) for n in ("clip_low", "clip_high", "kl_coef", "temperature")),
                ("dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32)]


_lib = None


class LibMuonError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: libmuon status {status}: {status_string(status)}")


def load() -> ctypes.CDLL:
    """Load libmuon.so (built in place by ``build.py``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmuon.so not found at {LIB_PATH}; build it with "
                           "`python -m matrix_aware_optimizer_libmuon_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    lib.muon_workspace_bytes.argtypes = [P(MuonMatrix), ctypes.c_int64]
    lib.muon_workspace_bytes.restype = ctypes.c_size_t
    lib.muon_step.argtypes = [P(MuonMatrix), ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                              ctypes.c_float, ctypes.c_int, P(MuonCoeff), ctypes.c_int, ctypes.c_int,
                              ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.muon_step.restype = ctypes.c_int
    lib.muon_step_ex.argtypes = [P(MuonMatrix), ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                 ctypes.c_float, ctypes.c_int, P(MuonCoeff), ctypes.c_int,
                                 ctypes.c_int, ctypes.c_float, P(MuonOptions), ctypes.c_void_p,
                                 ctypes.c_size_t, ctypes.c_void_p]
    lib.muon_step_ex.restype = ctypes.c_int
    lib.muon_plan_create.argtypes = [P(MuonMatrix), ctypes.c_int64, ctypes.c_int, P(MuonCoeff),
                                     ctypes.c_int, ctypes.c_int, ctypes.c_float, P(MuonOptions),
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                     P(ctypes.c_void_p)]
    lib.muon_plan_create.restype = ctypes.c_int
    lib.muon_plan_step.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.muon_plan_step.restype = ctypes.c_int
    lib.muon_plan_destroy.argtypes = [ctypes.c_void_p]
    lib.muon_plan_destroy.restype = None
    lib.muon_orthogonalize.argtypes = [P(MuonOrtho), ctypes.c_int64, ctypes.c_int, P(MuonCoeff),
                                       ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p]
    lib.muon_orthogonalize.restype = ctypes.c_int
    lib.muon_workspace_view.argtypes = [P(MuonMatrix), ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                        P(MuonWorkspaceView)]
    lib.muon_workspace_view.restype = ctypes.c_int
    lib.muon_adamw_workspace_bytes.argtypes = [ctypes.c_int64]
    lib.muon_adamw_workspace_bytes.restype = ctypes.c_size_t
    lib.muon_adamw_step.argtypes = [P(MuonAdamWTensor), ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                    ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]
    lib.muon_adamw_step.restype = ctypes.c_int
    lib.muon_timing_enable.argtypes = [ctypes.c_int]
    lib.muon_timing_enable.restype = ctypes.c_int
    lib.muon_timing_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64)]
    lib.muon_timing_read.restype = ctypes.c_int
    lib.muon_status_string.argtypes = [ctypes.c_int]
    lib.muon_status_string.restype = ctypes.c_char_p
    lib.muon_step_noalloc.argtypes = [P(MuonMatrix), ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                      ctypes.c_float, ctypes.c_int, P(MuonCoeff), ctypes.c_int,
                                      ctypes.c_int, ctypes.c_float, ctypes.c_void_p]
    lib.muon_step_noalloc.restype = ctypes.c_int
    lib.muon_noalloc_scratch.argtypes = []
    lib.muon_noalloc_scratch.restype = ctypes.c_void_p
    i32, i64, size_t, ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    for name, res, args in (
            ("muon_act8_pack", ctypes.c_int, [ptr, i64, i32, i64, i64, P(MuonAct8), ptr]),
            ("muon_act8_unpack", ctypes.c_int, [P(MuonAct8), i64, i64, ptr, i64, i32, ptr]),
            ("muon_rmsnorm_act8", ctypes.c_int, [P(MuonRmsnorm), ptr]),
            ("muon_rmsnorm_act8_grad_workspace_bytes", size_t, [i64, i64]),
            ("muon_rmsnorm_act8_grad", ctypes.c_int, [P(MuonRmsnormGrad), ptr, size_t, ptr]),
            ("muon_swiglu_act8", ctypes.c_int, [P(MuonSwiglu), ptr]),
            ("muon_swiglu_act8_grad", ctypes.c_int, [P(MuonSwigluGrad), ptr]),
            ("muon_act8_wgrad_workspace_bytes", size_t, [P(MuonAct8Wgrad)]),
            ("muon_act8_wgrad", ctypes.c_int, [P(MuonAct8Wgrad), ptr, size_t, ptr]),
            ("muon_embed", ctypes.c_int, [P(MuonEmbed), ptr]),
            ("muon_embed_grad_workspace_bytes", size_t, [i64, i64, i64]),
            ("muon_embed_grad", ctypes.c_int, [P(MuonEmbedGrad), ptr, size_t, ptr]),
            ("muon_attention_workspace_bytes", size_t, [P(MuonAttention)]),
            ("muon_attention", ctypes.c_int, [P(MuonAttention), ptr, size_t, ptr]),
            ("muon_attention_grad_workspace_bytes", size_t, [P(MuonAttentionGrad)]),
            ("muon_attention_grad", ctypes.c_int, [P(MuonAttentionGrad), ptr, size_t, ptr]),
            ("muon_distill", ctypes.c_int, [P(MuonDistill), ptr]),
            ("muon_policy", ctypes.c_int, [P(MuonPolicy), ptr])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    lib.muon_version.argtypes = []
    lib.muon_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().muon_status_string(int(status)).decode()


def check(status: int, where: str) -> None:
    if status != MUON_OK:
        raise LibMuonError(status, where)
