"""Python binding of libmoe.so: the C ABI in include/moe.h, same names.

Argument marshalling only -- every step of the path runs in the library's
CUDA kernels. Device buffers are torch tensors (torch supplies memory and
streams); each wrapper checks dtype/device/contiguity/size, passes raw
pointers, and raises MoeError on a non-zero status. Importing this module
raises ImportError when the library has not been built: there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK = 0
MOE_ERR_ARG = -1
MOE_ERR_SHAPE = -2
MOE_ERR_CAPACITY = -3
MOE_ERR_CUDA = -4
MOE_ERR_NONFINITE = -5
MOE_ERR_STATE = -6
MOE_ERR_TIMEOUT = -7
MOE_ERR_INJECTED = -8
MOE_ERR_UNSUPPORTED = -9

MOE_PATH_AUTO, MOE_PATH_GEMV, MOE_PATH_GROUPED, MOE_PATH_GEMV_UNFUSED = 0, 1, 2, 3


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {moe_status_string(status)}: {detail}")


class moe_expert_shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("group", ctypes.c_int32)]


class moe_block_layout(ctypes.Structure):
    _fields_ = [("total", ctypes.c_uint64), ("d_offset", ctypes.c_uint64),
                ("gu_row_bytes", ctypes.c_uint32), ("d_row_bytes", ctypes.c_uint32)] + [
        (n, ctypes.c_uint32) for n in ("gu_q_gate", "gu_q_up", "gu_sz", "d_q", "d_sz")]


MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1
MOE_F32, MOE_F16 = 0, 1


class moe_route_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "n_groups", "top_groups", "group_rank", "renorm")] + [
        ("scale", ctypes.c_float)]


MOE_NORM_RMS, MOE_NORM_LAYER = 0, 1
MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_CHANNEL, MOE_GATE_ELEMENT = 0, 1, 2, 3
(MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_SIGMOID) = range(6)


class moe_norm_cfg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class moe_balance_cfg(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("coef", ctypes.c_float)]


class moe_block(ctypes.Structure):
    _fields_ = [("shape", moe_expert_shape)] + [
        (n, ctypes.c_int32) for n in ("experts", "top_k", "n_slots", "shared_inter")] + [
        ("norm", moe_norm_cfg), ("route", moe_route_cfg), ("scale", ctypes.c_float),
        ("residual_scale", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("norm_w", "norm_b", "gate_w", "gate_b", "route_bias", "pool", "slot_of",
                                       "shared_g", "shared_u", "shared_d", "post_w", "post_b")]


MOE_POLICY_DECAY, MOE_POLICY_LRU, MOE_POLICY_PINNED = 0, 1, 2


class moe_residency_cfg(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("slots", ctypes.c_int32), ("spares", ctypes.c_int32),
                ("max_ids_per_step", ctypes.c_int32), ("dry_run", ctypes.c_int32),
                ("block_bytes", ctypes.c_uint64), ("decay", ctypes.c_double),
                ("policy", ctypes.c_int32), ("pinned", ctypes.c_int32),
                ("profile", ctypes.c_void_p), ("log_ops", ctypes.c_int32)]


class moe_residency_op(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("kind", "stream", "event", "layer", "slot", "expert")]


MOE_OP_RECORD, MOE_OP_WAIT, MOE_OP_COPY, MOE_OP_PUBLISH = 0, 1, 2, 3


class moe_residency_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("steps", "hits", "misses", "evictions", "copies", "h2d_bytes", "prefetched",
                 "prefetch_copies")]


class moe_residency_event(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int64), ("layer", ctypes.c_int32),
                ("expert", ctypes.c_int32), ("slot", ctypes.c_int32),
                ("victim", ctypes.c_int32)]


if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is not built; run int4_routed_expert_moe_gb300.build.build()")
_lib = ctypes.CDLL(_LIB_PATH)

_F32, _F16, _I32, _U8 = torch.float32, torch.float16, torch.int32, torch.uint8
_FP8 = torch.float8_e4m3fn

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_SHAPE = ctypes.POINTER(moe_expert_shape)
_CFG = ctypes.POINTER(moe_route_cfg)
_NORM = ctypes.POINTER(moe_norm_cfg)
_BAL = ctypes.POINTER(moe_balance_cfg)
_BLOCK = ctypes.POINTER(moe_block)
_LL = ctypes.c_longlong
_F = ctypes.c_float

_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_version": (_I, []),
    "moe_expert_block_bytes": (_SZ, [_SHAPE]),
    "moe_expert_block_layout": (_I, [_SHAPE, ctypes.POINTER(moe_block_layout)]),
    "moe_pack_expert": (_I, [_SHAPE] + [_P] * 10),
    "moe_unpack_expert": (_I, [_SHAPE] + [_P] * 10),
    "moe_route": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_route_scored": (_I, [_CFG, _P, _I, ctypes.c_longlong, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_token_sort": (_I, [_P, _I, _I, _I, _P, _P, _P, _P]),
    "moe_forward_workspace_bytes": (_SZ, [_SHAPE, _I, _I, _I, _I]),
    "moe_expert_forward": (_I, [_SHAPE, _P, _I, _P, _P, _I, _I, _P, _P, _I, _P, _P, _P, _SZ, _I, _P]),
    "moe_expert_forward_zero_copy": (_I, [_SHAPE, _P, _I, _P, _P, _I, _I, _P, _P, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_layer_forward": (_I, [_SHAPE, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P, _SZ, _I, _P]),
    "moe_layer_forward_scored": (_I, [_SHAPE, _P, _CFG, _P, _I, ctypes.c_longlong, _I, _I, _I, _P, _P, _P, _P, _P, _I,
                                      _P, _P, _P, _SZ, _I, _P]),
    "moe_layer_forward_noalloc": (_I, [_SHAPE, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P]),
    "moe_layer_forward_noalloc_flags": (_I, [ctypes.POINTER(ctypes.c_int32), _P]),
    "moe_workspace_clear_flags": (_I, [_P, _P]),
    "moe_workspace_flags": (_I, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
    "moe_shared_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_shared_forward": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_quantize_fp8": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_matmul_fp8_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_matmul_fp8": (_I, [_P, _P, _I, _P, _P, _I, _I, _P, _P, _SZ, _P]),
    "moe_shared_fp8_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_shared_forward_fp8": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_norm": (_I, [_NORM, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_norm_residual": (_I, [_NORM, _P, _P, _I, _I, _I, _P, _P, _P, _I, _F, _F, _P, _P, _P, _P, _P, _P, _P]),
    "moe_linear_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_linear": (_I, [_P, _LL, _I, _I, _P, _I, _P, _I, _P, _LL, _P, _I, _LL, _P, _SZ, _P]),
    "moe_balance_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_balance_loss": (_I, [_BAL, _P, _I, _LL, _I, _I, _P, _I, _P, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_balance_loss_backward": (_I, [_BAL, _P, _I, _LL, _I, _I, _I, _P, _I, _P, _P, _P, _P, _LL, _I, _P]),
    "moe_block_workspace_bytes": (_SZ, [_BLOCK, _I]),
    "moe_block_forward": (_I, [_BLOCK, _P, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_residency_create": (_I, [ctypes.POINTER(moe_residency_cfg), _P, _P, _P, _P, _P,
                                  ctypes.POINTER(_P)]),
    "moe_residency_prepare": (_I, [_P, _I, _P, _I]),
    "moe_residency_prefetch": (_I, [_P, _I, _P, _I, ctypes.POINTER(ctypes.c_int)]),
    "moe_residency_get_stats": (_I, [_P, _I, ctypes.POINTER(moe_residency_stats)]),
    "moe_residency_trace": (_I, [_P, _P, _SZ, ctypes.POINTER(_SZ)]),
    "moe_residency_ops": (_I, [_P, _P, _SZ, ctypes.POINTER(_SZ)]),
    "moe_residency_slot_table": (_I, [_P, _I, _P]),
    "moe_residency_counts": (_I, [_P, _I, _P]),
    "moe_residency_inject_copy_failure": (_I, [_P, ctypes.c_int64]),
    "moe_residency_destroy": (None, [_P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


def lib_path() -> str:
    return _LIB_PATH


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(status).decode()


def moe_last_error() -> str:
    return _lib.moe_last_error().decode()


def moe_version() -> int:
    return _lib.moe_version()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where, moe_last_error())


def _shape(shape) -> moe_expert_shape:
    H, I, g = shape
    return moe_expert_shape(int(H), int(I), int(g))


def _stream(stream) -> int:
    if stream is None:  # torch.cuda.current_stream().cuda_stream, without making the Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor | None, dtype, name: str, numel: int | None = None, nullable=False):
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    try:  # the usual case in few steps; what is wrong is looked for below
        if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (numel is None or t.numel() >= numel):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t.data_ptr()


# ---- expert block layout (host) --------------------------------------------
def moe_expert_block_bytes(shape) -> int:
    s = _shape(shape)
    return _lib.moe_expert_block_bytes(ctypes.byref(s))


def moe_expert_block_layout(shape) -> dict:
    s = _shape(shape)
    out = moe_block_layout()
    _check(_lib.moe_expert_block_layout(ctypes.byref(s), ctypes.byref(out)), "moe_expert_block_layout")
    return {n: int(getattr(out, n)) for n, _ in moe_block_layout._fields_}


_ARRAY_ORDER = ("qp_gate", "qp_up", "qp_down", "s_gate", "z_gate", "s_up", "z_up",
                "s_down", "z_down")


def _np_ptr(a: np.ndarray) -> int:
    return a.ctypes.data


def moe_pack_expert(shape, arrays: dict, out: np.ndarray | None = None) -> np.ndarray:
    """Copies the canonical arrays of one expert into one block (host)."""
    H, I, g = shape
    nbytes = moe_expert_block_bytes(shape)
    if nbytes == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_pack_expert", f"invalid shape {shape}")
    want = {"qp_gate": ((I, H // 2), np.uint8), "qp_up": ((I, H // 2), np.uint8),
            "qp_down": ((H, I // 2), np.uint8)}
    for n in ("gate", "up"):
        want[f"s_{n}"] = want[f"z_{n}"] = ((I, H // g), np.float16)
    want["s_down"] = want["z_down"] = ((H, I // g), np.float16)
    arrs = []
    for n in _ARRAY_ORDER:
        a = np.ascontiguousarray(arrays[n])
        shp, dt = want[n]
        if a.shape != shp or a.dtype != dt:
            raise ValueError(f"{n}: expected {shp} {dt}, got {a.shape} {a.dtype}")
        arrs.append(a)
    if out is None:
        out = np.empty(nbytes, dtype=np.uint8)
    assert out.nbytes >= nbytes and out.flags.c_contiguous
    s = _shape(shape)
    _check(_lib.moe_pack_expert(ctypes.byref(s), *[_np_ptr(a) for a in arrs], _np_ptr(out)),
           "moe_pack_expert")
    return out


def moe_unpack_expert(shape, block: np.ndarray) -> dict:
    H, I, g = shape
    out = {"qp_gate": np.empty((I, H // 2), np.uint8), "qp_up": np.empty((I, H // 2), np.uint8),
           "qp_down": np.empty((H, I // 2), np.uint8)}
    for n in ("gate", "up"):
        out[f"s_{n}"] = np.empty((I, H // g), np.float16)
        out[f"z_{n}"] = np.empty((I, H // g), np.float16)
    out["s_down"] = np.empty((H, I // g), np.float16)
    out["z_down"] = np.empty((H, I // g), np.float16)
    block = np.ascontiguousarray(block, dtype=np.uint8)
    s = _shape(shape)
    _check(_lib.moe_unpack_expert(ctypes.byref(s), _np_ptr(block),
                                  *[_np_ptr(out[n]) for n in _ARRAY_ORDER]), "moe_unpack_expert")
    return out


# ---- GPU calls -------------------------------------------------------------
def moe_route(logits: torch.Tensor, k: int, renorm: bool, ids: torch.Tensor,
              weights: torch.Tensor, bad_tokens: torch.Tensor | None = None, stream=None) -> None:
    T, E = logits.shape
    _check(_lib.moe_route(_dev(logits, torch.float32, "logits"), T, E, k, int(bool(renorm)),
                          _dev(ids, torch.int32, "ids", T * k),
                          _dev(weights, torch.float32, "weights", T * k),
                          _dev(bad_tokens, torch.int32, "bad_tokens", 1, nullable=True),
                          _stream(stream)), "moe_route")


_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_RANKS = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}
_LOGIT_TYPES = {torch.float32: MOE_F32, torch.float16: MOE_F16}


def moe_route_config(score: str = "softmax", n_groups: int = 1, top_groups: int = 1, group_rank: str = "max",
                     renorm: bool = True, scale: float = 1.0) -> moe_route_cfg:
    """A scored router's settings (made once, passed to every call)."""
    return moe_route_cfg(_SCORES[score], int(n_groups), int(top_groups), _RANKS[group_rank], int(bool(renorm)),
                         float(scale))


def _logits(logits) -> tuple:
    """(pointer, type, row stride, T, E) of a router's logits: rows may be strided."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32 or float16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [T][E] with contiguous rows")
    T, E = logits.shape
    ld, step = logits.stride()
    if E > 1 and step != 1:
        raise ValueError("logits must be [T][E] with contiguous rows")
    return logits.data_ptr(), kind, ld if T > 1 else E, T, E


def moe_route_scored(cfg: moe_route_cfg, logits: torch.Tensor, k: int, bias: torch.Tensor | None,
                     ids: torch.Tensor, weights: torch.Tensor, bad_tokens: torch.Tensor | None = None,
                     stream=None) -> None:
    ptr, kind, ld, T, E = _logits(logits)
    n = T * k
    status = _lib.moe_route_scored(
        cfg, ptr, kind, ld, T, E, k, None if bias is None else _dev(bias, _F32, "bias", E), _dev(ids, _I32, "ids", n),
        _dev(weights, _F32, "weights", n), None if bad_tokens is None else _dev(bad_tokens, _I32, "bad_tokens", 1),
        _stream(stream))
    if status:
        _check(status, "moe_route_scored")


def moe_token_sort(ids: torch.Tensor, E: int, offsets: torch.Tensor, pair_tok: torch.Tensor,
                   pair_j: torch.Tensor, stream=None) -> None:
    T, k = ids.shape
    _check(_lib.moe_token_sort(_dev(ids, torch.int32, "ids"), T, k, E,
                               _dev(offsets, torch.int32, "offsets", E + 1),
                               _dev(pair_tok, torch.int32, "pair_tok", T * k),
                               _dev(pair_j, torch.int32, "pair_j", T * k),
                               _stream(stream)), "moe_token_sort")


def moe_forward_workspace_bytes(shape, T: int, k: int, E: int, path: int = MOE_PATH_AUTO) -> int:
    s = _shape(shape)
    return _lib.moe_forward_workspace_bytes(ctypes.byref(s), T, k, E, path)


def moe_expert_forward(shape, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, E: int,
                       pool: torch.Tensor, slot_of: torch.Tensor, n_slots: int,
                       y_shared: torch.Tensor | None, y: torch.Tensor, workspace: torch.Tensor,
                       path: int = MOE_PATH_AUTO, stream=None) -> None:
    H, I, g = shape
    T, k = ids.shape
    s = _shape(shape)
    bb = moe_expert_block_bytes(shape)
    _check(_lib.moe_expert_forward(
        ctypes.byref(s), _dev(x, torch.float16, "x", T * H), T,
        _dev(ids, torch.int32, "ids", T * k), _dev(weights, torch.float32, "weights", T * k), k, E,
        _dev(pool, torch.uint8, "pool", n_slots * bb), _dev(slot_of, torch.int32, "slot_of", E), n_slots,
        _dev(y_shared, torch.float16, "y_shared", T * H, nullable=True),
        _dev(y, torch.float16, "y", T * H), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), path, _stream(stream)), "moe_expert_forward")


def moe_expert_forward_zero_copy(shape, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, E: int,
                                 pool: torch.Tensor, slot_of: torch.Tensor, n_slots: int,
                                 host_src: torch.Tensor, y_shared: torch.Tensor | None, y: torch.Tensor,
                                 workspace: torch.Tensor, stream=None) -> None:
    """moe_expert_forward on the two-kernel GEMV path; experts with slot -1
    are read in place from host_src (pinned CPU uint8 [E][block])."""
    H, I, g = shape
    T, k = ids.shape
    s = _shape(shape)
    bb = moe_expert_block_bytes(shape)
    if not isinstance(host_src, torch.Tensor) or host_src.is_cuda or host_src.dtype != torch.uint8:
        raise TypeError("host_src must be a CPU uint8 tensor")
    if not host_src.is_contiguous() or host_src.numel() < E * bb:
        raise ValueError(f"host_src must be contiguous with >= {E * bb} bytes")
    _check(_lib.moe_expert_forward_zero_copy(
        ctypes.byref(s), _dev(x, torch.float16, "x", T * H), T,
        _dev(ids, torch.int32, "ids", T * k), _dev(weights, torch.float32, "weights", T * k), k, E,
        _dev(pool, torch.uint8, "pool", n_slots * bb), _dev(slot_of, torch.int32, "slot_of", E), n_slots,
        host_src.data_ptr(), _dev(y_shared, torch.float16, "y_shared", T * H, nullable=True),
        _dev(y, torch.float16, "y", T * H), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "moe_expert_forward_zero_copy")


def moe_layer_forward(shape, x: torch.Tensor, logits: torch.Tensor, k: int, renorm: bool,
                      ids: torch.Tensor, weights: torch.Tensor, pool: torch.Tensor,
                      slot_of: torch.Tensor, n_slots: int, y_shared: torch.Tensor | None,
                      y: torch.Tensor, workspace: torch.Tensor, path: int = MOE_PATH_AUTO,
                      stream=None) -> None:
    H, I, g = shape
    T, E = logits.shape
    s = _shape(shape)
    bb = moe_expert_block_bytes(shape)
    _check(_lib.moe_layer_forward(
        ctypes.byref(s), _dev(x, torch.float16, "x", T * H), _dev(logits, torch.float32, "logits"), T, E,
        k, int(bool(renorm)), _dev(ids, torch.int32, "ids", T * k), _dev(weights, torch.float32, "weights", T * k),
        _dev(pool, torch.uint8, "pool", n_slots * bb), _dev(slot_of, torch.int32, "slot_of", E), n_slots,
        _dev(y_shared, torch.float16, "y_shared", T * H, nullable=True), _dev(y, torch.float16, "y", T * H),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), path, _stream(stream)), "moe_layer_forward")


def moe_layer_forward_scored(shape, x: torch.Tensor, cfg: moe_route_cfg, logits: torch.Tensor, k: int,
                             bias: torch.Tensor | None, ids: torch.Tensor, weights: torch.Tensor,
                             pool: torch.Tensor, slot_of: torch.Tensor, n_slots: int,
                             y_shared: torch.Tensor | None, y: torch.Tensor, workspace: torch.Tensor,
                             path: int = MOE_PATH_AUTO, stream=None) -> None:
    """moe_route_scored, then moe_expert_forward on its ids and weights."""
    H, I, g = shape
    ptr, kind, ld, T, E = _logits(logits)
    s = _shape(shape)
    bb = moe_expert_block_bytes(shape)
    _check(_lib.moe_layer_forward_scored(
        ctypes.byref(s), _dev(x, torch.float16, "x", T * H), cfg, ptr, kind, ld, T, E, k,
        _dev(bias, torch.float32, "bias", E, nullable=True), _dev(ids, torch.int32, "ids", T * k),
        _dev(weights, torch.float32, "weights", T * k), _dev(pool, torch.uint8, "pool", n_slots * bb),
        _dev(slot_of, torch.int32, "slot_of", E), n_slots,
        _dev(y_shared, torch.float16, "y_shared", T * H, nullable=True), _dev(y, torch.float16, "y", T * H),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), path, _stream(stream)),
        "moe_layer_forward_scored")


def moe_layer_forward_noalloc(shape, x: torch.Tensor, logits: torch.Tensor, k: int, renorm: bool,
                              ids: torch.Tensor, weights: torch.Tensor, pool: torch.Tensor,
                              slot_of: torch.Tensor, n_slots: int, y_shared: torch.Tensor | None,
                              y: torch.Tensor, stream=None) -> None:
    """moe_layer_forward without a workspace (scratch is a fixed array inside the library)."""
    H, I, g = shape
    T, E = logits.shape
    s = _shape(shape)
    bb = moe_expert_block_bytes(shape)
    _check(_lib.moe_layer_forward_noalloc(
        ctypes.byref(s), _dev(x, torch.float16, "x", T * H), _dev(logits, torch.float32, "logits"), T, E,
        k, int(bool(renorm)), _dev(ids, torch.int32, "ids", T * k), _dev(weights, torch.float32, "weights", T * k),
        _dev(pool, torch.uint8, "pool", n_slots * bb), _dev(slot_of, torch.int32, "slot_of", E), n_slots,
        _dev(y_shared, torch.float16, "y_shared", T * H, nullable=True), _dev(y, torch.float16, "y", T * H),
        _stream(stream)), "moe_layer_forward_noalloc")


def moe_layer_forward_noalloc_flags(stream=None) -> int:
    """Error word of the last moe_layer_forward_noalloc call on the current device (synchronises)."""
    v = ctypes.c_int32(0)
    _check(_lib.moe_layer_forward_noalloc_flags(ctypes.byref(v), _stream(stream)), "moe_layer_forward_noalloc_flags")
    return v.value


def moe_workspace_clear_flags(workspace: torch.Tensor, stream=None) -> None:
    _check(_lib.moe_workspace_clear_flags(_dev(workspace, torch.uint8, "workspace"), _stream(stream)),
           "moe_workspace_clear_flags")


def moe_workspace_flags(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(_lib.moe_workspace_flags(_dev(workspace, torch.uint8, "workspace"), ctypes.byref(v),
                                    _stream(stream)), "moe_workspace_flags")
    return v.value


def moe_shared_workspace_bytes(T: int, H: int, Is: int) -> int:
    return _lib.moe_shared_workspace_bytes(T, H, Is)


def moe_shared_forward(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, wd: torch.Tensor,
                       y: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    T, H = x.shape
    Is = wg.shape[0]
    _check(_lib.moe_shared_forward(
        _dev(x, torch.float16, "x", T * H), T, H, Is, _dev(wg, torch.float16, "wg", Is * H),
        _dev(wu, torch.float16, "wu", Is * H), _dev(wd, torch.float16, "wd", H * Is),
        _dev(y, torch.float16, "y", T * H), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "moe_shared_forward")


# ---- FP8 non-routed path -----------------------------------------------------


def _nb(n: int) -> int:
    return (n + 127) >> 7


def moe_quantize_fp8(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, block_rows: int = 1,
                     stream=None) -> None:
    """x (fp16 [rows][cols]) to float8_e4m3fn codes q and scales
    [ceil(rows / block_rows)][ceil(cols / 128)]; block_rows 1 (activations) or 128 (weights)."""
    rows, cols = x.shape
    status = _lib.moe_quantize_fp8(_dev(x, _F16, "x"), rows, cols, block_rows, _dev(q, _FP8, "q", rows * cols),
                                   _dev(scales, _F32, "scales", -(-rows // max(1, block_rows)) * _nb(cols)),
                                   _stream(stream))
    if status:
        _check(status, "moe_quantize_fp8")


def moe_matmul_fp8_workspace_bytes(T: int, N: int, K: int) -> int:
    return _lib.moe_matmul_fp8_workspace_bytes(T, N, K)


def moe_matmul_fp8(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, y: torch.Tensor,
                   workspace: torch.Tensor, stream=None) -> None:
    """y [T][N] = x W^T from the codes xq [T][K], wq [N][K] and their scales."""
    T, K = xq.shape
    N, Kw = wq.shape
    if Kw != K:
        raise ValueError(f"xq has {K} columns, wq {Kw}")
    nb = _nb(K)
    status = _lib.moe_matmul_fp8(_dev(xq, _FP8, "xq"), _dev(xs, _F32, "xs", T * nb), T, _dev(wq, _FP8, "wq"),
                                 _dev(ws, _F32, "ws", _nb(N) * nb), N, K, _dev(y, _F16, "y", T * N),
                                 _dev(workspace, _U8, "workspace"), workspace.numel(), _stream(stream))
    if status:
        _check(status, "moe_matmul_fp8")


def moe_shared_fp8_workspace_bytes(T: int, H: int, Is: int) -> int:
    return _lib.moe_shared_fp8_workspace_bytes(T, H, Is)


def _shared_fp8_shapes(H: int, Is: int, w: dict) -> None:
    """ValueError for the operand that is too small, or would be read with a row pitch that is not its own."""
    for n, (rows, cols) in dict(g=(Is, H), u=(Is, H), d=(H, Is)).items():
        for name, shape, flat in (("w" + n, (rows, cols), False), ("s" + n, (_nb(rows), _nb(cols)), True)):
            t = w[name]
            if not isinstance(t, torch.Tensor):
                raise (ValueError if t is None else TypeError)(f"{name} must be a CUDA tensor")
            # Scales may come as rows end to end, and with rows to spare.
            if t.shape != shape and not (flat and t.numel() >= shape[0] * shape[1]
                                         and (t.dim() != 2 or t.shape[1] == shape[1])):
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def moe_shared_forward_fp8(x: torch.Tensor, wg: torch.Tensor, sg: torch.Tensor, wu: torch.Tensor, su: torch.Tensor,
                           wd: torch.Tensor, sd: torch.Tensor, y: torch.Tensor, workspace: torch.Tensor,
                           stream=None) -> None:
    """moe_shared_forward with float8_e4m3fn weights and their 128 x 128 block scales."""
    T, H = x.shape
    Is = wg.shape[0]
    up, down, sup, sdown = (Is, H), (H, Is), (_nb(Is), _nb(H)), (_nb(H), _nb(Is))
    try:  # the usual case in few steps
        usual = (wg.shape == wu.shape == up and wd.shape == down and sg.shape == su.shape == sup
                 and sd.shape == sdown)
    except AttributeError:
        usual = False
    if not usual:
        _shared_fp8_shapes(H, Is, dict(wg=wg, sg=sg, wu=wu, su=su, wd=wd, sd=sd))
    status = _lib.moe_shared_forward_fp8(
        _dev(x, _F16, "x"), T, H, Is, _dev(wg, _FP8, "wg"), _dev(sg, _F32, "sg"), _dev(wu, _FP8, "wu"),
        _dev(su, _F32, "su"), _dev(wd, _FP8, "wd"), _dev(sd, _F32, "sd"), _dev(y, _F16, "y", T * H),
        _dev(workspace, _U8, "workspace"), workspace.numel(), _stream(stream))
    if status:
        _check(status, "moe_shared_forward_fp8")


# ---- norms round a block -------------------------------------------------------
_NORMS = {"rms": MOE_NORM_RMS, "layer": MOE_NORM_LAYER}


def moe_norm_config(kind: str = "rms", eps: float = 1e-6, weight_offset: float = 0.0) -> moe_norm_cfg:
    """A norm's settings (made once, passed to every call)."""
    return moe_norm_cfg(_NORMS[kind], float(eps), float(weight_offset))


def _stream_type(t, name: str) -> int:
    """MOE_F16 or MOE_F32 of a residual stream."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    kind = _LOGIT_TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32 or float16, got {t.dtype}")
    return kind


def moe_norm(cfg: moe_norm_cfg, x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
             y: torch.Tensor | None = None, q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
             stream=None) -> None:
    """norm(x) of x [T][H] (float16 or float32) as float16 y, as float8_e4m3fn codes q with scales
    [T][ceil(H / 128)], or both."""
    kind = _stream_type(x, "x")
    T, H = x.shape
    n = T * H
    status = _lib.moe_norm(cfg, _dev(x, x.dtype, "x"), kind, T, H, _dev(w, _F16, "w", H),
                           None if b is None else _dev(b, _F16, "b", H), None if y is None else _dev(y, _F16, "y", n),
                           None if q is None else _dev(q, _FP8, "q", n),
                           None if scales is None else _dev(scales, _F32, "scales", T * _nb(H)), _stream(stream))
    if status:
        _check(status, "moe_norm")


def _gate(gate, T: int, H: int) -> tuple:
    """(pointer, kind): float32 [T] per token, float16 [H] per channel, float16 [T][H] per element."""
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a CUDA tensor")
    if gate.dtype is _F32 and gate.shape in ((T,), (T, 1)):
        return _dev(gate, _F32, "gate"), MOE_GATE_TOKEN
    if gate.dtype is _F16 and gate.shape == (H,):
        return _dev(gate, _F16, "gate"), MOE_GATE_CHANNEL
    if gate.dtype is _F16 and gate.shape == (T, H):
        return _dev(gate, _F16, "gate"), MOE_GATE_ELEMENT
    raise ValueError(f"gate must be float32 [{T}], float16 [{H}] or float16 [{T}][{H}], got {gate.dtype} "
                     f"{list(gate.shape)}")


def moe_norm_residual(cfg: moe_norm_cfg, branch: torch.Tensor, residual: torch.Tensor | None,
                      h: torch.Tensor | None, post_w: torch.Tensor | None = None, post_b: torch.Tensor | None = None,
                      gate: torch.Tensor | None = None, scale: float = 1.0, residual_scale: float = 1.0,
                      w: torch.Tensor | None = None, b: torch.Tensor | None = None, y: torch.Tensor | None = None,
                      q: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None) -> None:
    """h = residual_scale * residual + scale * gate * (branch or its norm with post_w); then, with y or q, the
    norm of h with w as moe_norm gives it. residual and h: float16 or float32 [T][H], of one type."""
    shape = branch.shape
    T, H = shape
    n = T * H
    typ, kind = _F16, MOE_F16
    for name, t in (("residual", residual), ("h", h)):
        if t is not None:
            kind = _stream_type(t, name)
            if t.shape != shape:
                raise ValueError(f"{name} must be [{T}][{H}], got {list(t.shape)}")
            typ = t.dtype
    pg, gk = (None, MOE_GATE_NONE) if gate is None else _gate(gate, T, H)
    status = _lib.moe_norm_residual(
        cfg, _dev(branch, _F16, "branch"), None if residual is None else _dev(residual, typ, "residual"), kind, T, H,
        None if post_w is None else _dev(post_w, _F16, "post_w", H),
        None if post_b is None else _dev(post_b, _F16, "post_b", H), pg, gk, scale, residual_scale,
        None if h is None else _dev(h, typ, "h"), None if w is None else _dev(w, _F16, "w", H),
        None if b is None else _dev(b, _F16, "b", H), None if y is None else _dev(y, _F16, "y", n),
        None if q is None else _dev(q, _FP8, "q", n),
        None if scales is None else _dev(scales, _F32, "scales", T * _nb(H)), _stream(stream))
    if status:
        _check(status, "moe_norm_residual")


# ---- FP16 product with its epilogue ----------------------------------------------
_ACTS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU,
         "gelu_tanh": MOE_ACT_GELU_TANH, "sigmoid": MOE_ACT_SIGMOID}


def _rows(t, name: str, shape: tuple, dtypes) -> tuple:
    """(pointer, row stride) of a [rows][columns] tensor whose rows may be strided."""
    try:  # the usual case in few steps
        if t.is_cuda and t.dtype in dtypes and t.is_contiguous() and t.shape == shape:
            return t.data_ptr(), shape[1]
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    ld, step = t.stride()
    rows, cols = shape
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld if rows > 1 else cols


_HALF, _HALF_OR_FLOAT = (_F16,), (_F16, _F32)


def moe_linear_workspace_bytes(T: int, N: int, K: int) -> int:
    return _lib.moe_linear_workspace_bytes(T, N, K)


def moe_linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None, y: torch.Tensor, workspace: torch.Tensor,
               act: str = "none", residual: torch.Tensor | None = None, stream=None) -> None:
    """y [T][N] (float16 or float32) = act(x W^T + bias) + residual, x [T][K] and w [N][K] float16, bias
    float32 [N], residual of y's type. Rows of x, y and residual may be strided."""
    shape = x.shape
    T, K = shape
    N, Kw = w.shape
    if Kw != K:
        raise ValueError(f"x has {K} columns, w {Kw}")
    px, ldx = _rows(x, "x", shape, _HALF)
    py, ldy = _rows(y, "y", (T, N), _HALF_OR_FLOAT)
    pr, ldr = (None, 0) if residual is None else _rows(residual, "residual", (T, N), (y.dtype,))
    status = _lib.moe_linear(px, ldx, T, K, _dev(w, _F16, "w"), N, None if bias is None else _dev(bias, _F32, "bias", N),
                             _ACTS[act], pr, ldr, py, _LOGIT_TYPES[y.dtype], ldy, _dev(workspace, _U8, "workspace"),
                             workspace.numel(), _stream(stream))
    if status:
        _check(status, "moe_linear")


# ---- balance loss ------------------------------------------------------------------
def moe_balance_config(score: str = "softmax", coef: float = 1.0) -> moe_balance_cfg:
    """A balance loss's settings (made once, passed to every call)."""
    return moe_balance_cfg(_SCORES[score], float(coef))


def moe_balance_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return _lib.moe_balance_workspace_bytes(T, E, S)


def _sequences(offsets) -> tuple:
    """(pointer, S) of the sequences' offsets; None: one sequence of all tokens."""
    if offsets is None:
        return None, 1
    return _dev(offsets, _I32, "offsets"), offsets.numel() - 1


def moe_balance_loss(cfg: moe_balance_cfg, logits: torch.Tensor, ids: torch.Tensor, offsets: torch.Tensor | None,
                     counts: torch.Tensor, tokens: torch.Tensor, mean: torch.Tensor | None,
                     loss: torch.Tensor | None, workspace: torch.Tensor, stream=None) -> None:
    """Per sequence: counts int32 [S][E] of the picks ids [T][k], tokens int32 [S] that count, mean float32
    [S][E] of the router's probabilities; loss float32 [1] of all."""
    ptr, kind, ld, T, E = _logits(logits)
    k = ids.shape[1]
    if ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}][k], got {list(ids.shape)}")
    po, S = _sequences(offsets)
    status = _lib.moe_balance_loss(
        cfg, ptr, kind, ld, T, E, _dev(ids, _I32, "ids"), k, po, S, _dev(counts, _I32, "counts", S * E),
        _dev(tokens, _I32, "tokens", S), None if mean is None else _dev(mean, _F32, "mean", S * E),
        None if loss is None else _dev(loss, _F32, "loss", 1), _dev(workspace, _U8, "workspace"), workspace.numel(),
        _stream(stream))
    if status:
        _check(status, "moe_balance_loss")


def moe_balance_loss_backward(cfg: moe_balance_cfg, logits: torch.Tensor, k: int, offsets: torch.Tensor | None,
                              counts: torch.Tensor, tokens: torch.Tensor, grad_loss: torch.Tensor | None,
                              dlogits: torch.Tensor, accumulate: bool = False, stream=None) -> None:
    """dlogits float32 [T][E] (rows may be strided) = the loss's gradient, or added to it; counts and tokens as
    moe_balance_loss left them."""
    ptr, kind, ld, T, E = _logits(logits)
    po, S = _sequences(offsets)
    pd, ldd = _rows(dlogits, "dlogits", (T, E), (_F32,))
    status = _lib.moe_balance_loss_backward(
        cfg, ptr, kind, ld, T, E, k, po, S, _dev(counts, _I32, "counts", S * E), _dev(tokens, _I32, "tokens", S),
        None if grad_loss is None else _dev(grad_loss, _F32, "grad_loss", 1), pd, ldd, int(bool(accumulate)),
        _stream(stream))
    if status:
        _check(status, "moe_balance_loss_backward")


# ---- a whole MoE block -------------------------------------------------------------
def moe_block_config(shape, k: int, norm: moe_norm_cfg, norm_w: torch.Tensor, gate_w: torch.Tensor,
                     route: moe_route_cfg, pool: torch.Tensor, slot_of: torch.Tensor, n_slots: int,
                     norm_b: torch.Tensor | None = None, gate_b: torch.Tensor | None = None,
                     route_bias: torch.Tensor | None = None, shared: tuple | None = None,
                     post_w: torch.Tensor | None = None, post_b: torch.Tensor | None = None, scale: float = 1.0,
                     residual_scale: float = 1.0) -> moe_block:
    """An MoE block's weights and settings (made once, passed to every call; it keeps the tensors). gate_w
    float16 [E][H]; shared: (wg, wu [Is][H], wd [H][Is]) float16 or None."""
    H, E = int(shape[0]), gate_w.shape[0]
    if gate_w.shape != (E, H):
        raise ValueError(f"gate_w must be [E][{H}], got {list(gate_w.shape)}")
    Is = 0
    if shared is not None:
        Is = shared[0].shape[0]
        for name, t, want in zip(("wg", "wu", "wd"), shared, ((Is, H), (Is, H), (H, Is))):
            if t.shape != want:
                raise ValueError(f"{name} must be {list(want)}, got {list(t.shape)}")
    vec = lambda t, name: None if t is None else _dev(t, _F16, name, H)
    per = lambda t, name: None if t is None else _dev(t, _F32, name, E)
    sg, su, sd = (None,) * 3 if shared is None else (_dev(t, _F16, n) for t, n in zip(shared, ("wg", "wu", "wd")))
    b = moe_block(_shape(shape), E, int(k), int(n_slots), Is, norm, route, float(scale), float(residual_scale),
                  _dev(norm_w, _F16, "norm_w", H), vec(norm_b, "norm_b"), _dev(gate_w, _F16, "gate_w"),
                  per(gate_b, "gate_b"), per(route_bias, "route_bias"),
                  _dev(pool, _U8, "pool", int(n_slots) * moe_expert_block_bytes(shape)), _dev(slot_of, _I32, "slot_of", E),
                  sg, su, sd, vec(post_w, "post_w"), vec(post_b, "post_b"))
    b.tensors = (norm_w, norm_b, gate_w, gate_b, route_bias, pool, slot_of, shared, post_w, post_b)
    return b


def moe_block_workspace_bytes(block: moe_block, T: int) -> int:
    return _lib.moe_block_workspace_bytes(block, T)


def moe_block_forward(block: moe_block, h: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                      workspace: torch.Tensor, logits: torch.Tensor | None = None, stream=None) -> None:
    """h [T][H] (float16 or float32) through norm, router, experts (and shared FFN) and residual sum, in place."""
    kind = _stream_type(h, "h")
    T, H = h.shape
    if H != block.shape.hidden:
        raise ValueError(f"h must be [T][{block.shape.hidden}], got {list(h.shape)}")
    n = T * block.top_k
    status = _lib.moe_block_forward(
        block, _dev(h, h.dtype, "h"), kind, T, _dev(ids, _I32, "ids", n), _dev(weights, _F32, "weights", n),
        None if logits is None else _dev(logits, _F32, "logits", T * block.experts), _dev(workspace, _U8, "workspace"),
        workspace.numel(), _stream(stream))
    if status:
        _check(status, "moe_block_forward")


# ---- residency manager -----------------------------------------------------
def moe_residency_create(cfg: dict, host_src: torch.Tensor | None, dev_pool: torch.Tensor | None,
                         dev_slot_of: torch.Tensor | None, compute=None, copy=None) -> int:
    policy = cfg.get("policy", MOE_POLICY_DECAY)
    if isinstance(policy, str):
        policy = {"decay": MOE_POLICY_DECAY, "lru": MOE_POLICY_LRU, "pinned": MOE_POLICY_PINNED}[policy]
    prof = cfg.get("profile")
    prof_arr = None
    if prof is not None:
        prof_arr = np.ascontiguousarray(np.asarray(prof, dtype=np.float64).reshape(-1))
        if prof_arr.size != int(cfg["layers"]) * int(cfg["experts"]):
            raise ValueError("profile must hold layers x experts values")
    c = moe_residency_cfg(int(cfg["layers"]), int(cfg["experts"]), int(cfg["slots"]),
                          int(cfg.get("spares", 0)), int(cfg["max_ids_per_step"]),
                          int(cfg.get("dry_run", 0)), int(cfg["block_bytes"]),
                          float(cfg["decay"]), int(policy), int(cfg.get("pinned", 0)),
                          prof_arr.ctypes.data if prof_arr is not None else None, int(cfg.get("log_ops", 0)))
    dry = bool(c.dry_run)
    src = pool = slot = None
    cs = cp = None
    if not dry:
        if host_src is None or not host_src.is_pinned():
            raise ValueError("host_src must be a pinned CPU tensor")
        src = host_src.data_ptr()
        pool = _dev(dev_pool, torch.uint8, "dev_pool")
        slot = _dev(dev_slot_of, torch.int32, "dev_slot_of", c.layers * c.experts)
        cs, cp = _stream(compute), _stream(copy)
    h = ctypes.c_void_p()
    _check(_lib.moe_residency_create(ctypes.byref(c), src, pool, slot, cs, cp, ctypes.byref(h)),
           "moe_residency_create")
    return h.value


def moe_residency_prepare(handle: int, layer: int, host_ids) -> None:
    a = np.ascontiguousarray(np.asarray(host_ids, dtype=np.int32).reshape(-1))
    _check(_lib.moe_residency_prepare(handle, layer, a.ctypes.data if a.size else None, a.size),
           "moe_residency_prepare")


def moe_residency_prefetch(handle: int, layer: int, host_ids) -> int:
    """Copy predicted misses into free spare slots; returns how many were copied."""
    a = np.ascontiguousarray(np.asarray(host_ids, dtype=np.int32).reshape(-1))
    n = ctypes.c_int(0)
    _check(_lib.moe_residency_prefetch(handle, layer, a.ctypes.data if a.size else None, a.size,
                                       ctypes.byref(n)), "moe_residency_prefetch")
    return int(n.value)


def moe_residency_get_stats(handle: int, layer: int = -1) -> dict:
    st = moe_residency_stats()
    _check(_lib.moe_residency_get_stats(handle, layer, ctypes.byref(st)), "moe_residency_get_stats")
    return {n: int(getattr(st, n)) for n, _ in moe_residency_stats._fields_}


def moe_residency_trace(handle: int) -> list:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_residency_trace(handle, None, 0, ctypes.byref(n)), "moe_residency_trace")
    buf = (moe_residency_event * max(1, n.value))()
    _check(_lib.moe_residency_trace(handle, buf, n.value, ctypes.byref(n)), "moe_residency_trace")
    return [(int(b.step), int(b.layer), int(b.expert), int(b.slot), int(b.victim))
            for b in buf[:n.value]]


def moe_residency_ops(handle: int) -> list:
    """Logged stream operations: (kind, stream, event, layer, slot, expert) tuples."""
    n = ctypes.c_size_t(0)
    _check(_lib.moe_residency_ops(handle, None, 0, ctypes.byref(n)), "moe_residency_ops")
    buf = (moe_residency_op * max(1, n.value))()
    _check(_lib.moe_residency_ops(handle, buf, n.value, ctypes.byref(n)), "moe_residency_ops")
    return [(o.kind, o.stream, o.event, o.layer, o.slot, o.expert) for o in buf[:n.value]]


def moe_residency_slot_table(handle: int, layer: int, E: int) -> np.ndarray:
    out = np.empty(E, dtype=np.int32)
    _check(_lib.moe_residency_slot_table(handle, layer, out.ctypes.data), "moe_residency_slot_table")
    return out


def moe_residency_counts(handle: int, layer: int, E: int) -> np.ndarray:
    out = np.empty(E, dtype=np.float64)
    _check(_lib.moe_residency_counts(handle, layer, out.ctypes.data), "moe_residency_counts")
    return out


def moe_residency_inject_copy_failure(handle: int, nth_copy: int) -> None:
    _check(_lib.moe_residency_inject_copy_failure(handle, nth_copy), "moe_residency_inject_copy_failure")


def moe_residency_destroy(handle: int) -> None:
    _lib.moe_residency_destroy(handle)
