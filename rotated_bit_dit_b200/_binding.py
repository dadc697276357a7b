"""ctypes binding of librbd.so: the same entry points as include/rbd.h.

Argument marshalling only.  Every computation runs in the library's CUDA
kernels; there is no Python or CPU fallback.  Tensors must be CUDA tensors on
the current device (others are refused before any launch); the current torch
stream is used unless `stream` is given.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

RBD_OK = 0
STATUS_NAMES = {0: "RBD_OK", 1: "RBD_ERR_INVALID_ARG", 2: "RBD_ERR_UNSUPPORTED", 3: "RBD_ERR_ALIGNMENT",
                4: "RBD_ERR_CUDA", 5: "RBD_ERR_DEVICE_TIMEOUT"}

EXPORTED = ("rbd_rot_quant_act", "rbd_norm_rot_quant_act", "rbd_lowrank_fused", "rbd_lowrank_down", "rbd_pack_weights_int4", "rbd_pack_weights_int8",
            "rbd_w4a4_linear", "rbd_w8a8_linear", "rbd_nvfp4_scale_bytes", "rbd_nvfp4_quant",
            "rbd_nvfp4_quant_noalloc", "rbd_nvfp4_linear", "rbd_kv4_encode", "rbd_kv4_decode", "rbd_qk_norm_rope", "rbd_rope_tables", "rbd_attn_workspace_bytes", "rbd_attn_quant", "rbd_attn_int8",
            "rbd_kv8_append", "rbd_kv8_read", "rbd_kv8_attn_workspace_bytes", "rbd_kv8_attn", "rbd_kv8_evict",
            "rbd_svdquant_workspace_bytes", "rbd_svdquant_fit",
            "rbd_check", "rbd_debug_timeout_probe", "rbd_status_string", "rbd_version")


class RbdError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


CODES_INT8 = 0   # activation code stored as a two's-complement int8
CODES_E4M3 = 1   # activation code stored as the E4M3 byte of the same value (4-bit codes)


class QCfg(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("rot_group", ctypes.c_int32), ("scale_group", ctypes.c_int32),
                ("code_format", ctypes.c_int32)]


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("ld", ctypes.c_void_p), ("l2t", ctypes.c_void_p),
                ("r", ctypes.c_int32), ("gate_mode", ctypes.c_int32), ("gate_col0", ctypes.c_int64),
                ("gate_col1", ctypes.c_int64), ("gate", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ldr", ctypes.c_int64), ("acc_debug", ctypes.c_void_p)]


class Kv8(ctypes.Structure):
    """rbd_kv8: the buffers of an 8-bit paged key/value cache."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("ldt", ctypes.c_int64), ("pages", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("seqs", ctypes.c_int64), ("heads", ctypes.c_int32), ("code_format", ctypes.c_int32)]


_LIB = None


def lib_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load librbd.so (building it first when absent).  Raises if it cannot be loaded."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"librbd.so not built: {path}")
        _build.build()
    lib = ctypes.CDLL(path)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    sigs = {
        "rbd_rot_quant_act": [vp, i64, i64, i64, QCfg, vp, vp, vp],
        "rbd_norm_rot_quant_act": [vp, i64, i64, i64, vp, vp, vp, ctypes.c_float, QCfg, vp, vp, vp],
        "rbd_lowrank_fused": [vp, i64, i64, i64, QCfg, vp, vp, vp, i32, vp, vp],
        "rbd_lowrank_down": [vp, i64, i64, i64, vp, i32, vp, vp],
        "rbd_pack_weights_int4": [vp, i64, i64, QCfg, vp, vp, vp],
        "rbd_pack_weights_int8": [vp, i64, i64, QCfg, vp, vp, vp],
        "rbd_w4a4_linear": [vp, vp, vp, vp, i64, i64, i64, QCfg, ctypes.POINTER(Epilogue), vp, i64, vp],
        "rbd_w8a8_linear": [vp, vp, vp, vp, i64, i64, i64, QCfg, ctypes.POINTER(Epilogue), vp, i64, vp],
        "rbd_nvfp4_quant": [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp],
        "rbd_nvfp4_quant_noalloc": [vp, i64, i64, i64, i32, vp, vp, vp, vp],
        "rbd_nvfp4_linear": [vp, vp, vp, vp, vp, vp, i64, i64, i64, ctypes.POINTER(Epilogue), vp, i64, vp],
        "rbd_kv4_encode": [vp, i64, i64, i64, i32, vp, vp, i64, i64, vp],
        "rbd_kv4_decode": [vp, vp, i64, i64, i64, i64, i32, vp, i64, vp],
        "rbd_qk_norm_rope": [vp, i64, i64, i64, vp, vp, vp, ctypes.c_float, vp, i64, vp],
        "rbd_rope_tables": [vp, i64, ctypes.c_double, vp, vp, vp],
        "rbd_attn_quant": [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp, vp],
        "rbd_attn_int8": [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i64, vp],
        "rbd_kv8_append": [ctypes.POINTER(Kv8), vp, vp, vp, i64, vp, i64, i64, vp],
        "rbd_kv8_read": [ctypes.POINTER(Kv8), vp, i64, vp, i64, vp, i64, vp],
        "rbd_kv8_attn": [ctypes.POINTER(Kv8), vp, vp, vp, i64, i64, i64, i32, ctypes.c_float, i64, vp, i64, vp, vp, i64,
                         i64, vp, i64, vp],
        "rbd_kv8_evict": [ctypes.POINTER(Kv8), vp, vp, i64, i64, i64, i64, i64, vp, i64, vp, vp, i64, i64, i64, vp, vp],
        "rbd_svdquant_fit": [vp, i64, i64, QCfg, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
        "rbd_check": [vp],
        "rbd_debug_timeout_probe": [i64, vp],
    }
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.rbd_nvfp4_scale_bytes.argtypes = [i64, i64]
    lib.rbd_nvfp4_scale_bytes.restype = i64
    lib.rbd_attn_workspace_bytes.argtypes = [i64, i64]
    lib.rbd_attn_workspace_bytes.restype = i64
    lib.rbd_kv8_attn_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32]
    lib.rbd_kv8_attn_workspace_bytes.restype = i64
    lib.rbd_svdquant_workspace_bytes.argtypes = [i64, i64, i32, i32, QCfg]
    lib.rbd_svdquant_workspace_bytes.restype = i64
    lib.rbd_status_string.argtypes = [ctypes.c_int]
    lib.rbd_status_string.restype = ctypes.c_char_p
    lib.rbd_version.argtypes = []
    lib.rbd_version.restype = ctypes.c_char_p
    _LIB = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    """Device address of t.  Every kernel launches on the current device, so a tensor that
    lives on another device is refused here, before any launch (its address would be
    dereferenced by the wrong GPU)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index is not None and t.device.index != cur:
        raise ValueError(f"tensor on {t.device} while cuda:{cur} is current; "
                         f"call under torch.cuda.device({t.device})")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ok(status: int, where: str):
    if status != RBD_OK:
        raise RbdError(status, where)


def _qcfg(bits: int, rot_group: int, scale_group: int, code_format: int = CODES_INT8) -> QCfg:
    return QCfg(bits, rot_group, scale_group, code_format)


def _rowstride(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D row-major tensor")
    return t.stride(0)


# ---------------------------------------------------------------- entry points
def rbd_rot_quant_act(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bits: int = 4,
                      rot_group: int = 256, scale_group: int = 0, stream=None, code_format: int = CODES_INT8) -> None:
    """x bf16 [M, K] -> codes [M, K] (one byte each, in code_format), scales float32 [M] or [M, K/64]."""
    M, K = x.shape
    _ok(load().rbd_rot_quant_act(_ptr(x), M, K, _rowstride(x), _qcfg(bits, rot_group, scale_group, code_format),
                                 _ptr(codes), _ptr(scales), _stream(stream)), "rbd_rot_quant_act")


def rbd_norm_rot_quant_act(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                           gamma: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                           scale: Optional[torch.Tensor] = None, eps: float = 1e-6, bits: int = 4,
                           rot_group: int = 256, scale_group: int = 0, stream=None,
                           code_format: int = CODES_INT8) -> None:
    """RMSNorm (optional gamma) and modulation x*(1 + scale) + shift, then rbd_rot_quant_act.
    gamma, shift, scale: bf16 [K] or None."""
    M, K = x.shape
    for name, v in (("gamma", gamma), ("shift", shift), ("scale", scale)):
        if v is not None and (v.numel() != K or not v.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bf16 vector of length K")
    _ok(load().rbd_norm_rot_quant_act(_ptr(x), M, K, _rowstride(x), _ptr(gamma), _ptr(shift), _ptr(scale),
                                      float(eps), _qcfg(bits, rot_group, scale_group, code_format), _ptr(codes),
                                      _ptr(scales), _stream(stream)), "rbd_norm_rot_quant_act")


def rbd_lowrank_fused(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, l1t: torch.Tensor,
                      ld: torch.Tensor, bits: int = 4, rot_group: int = 256, scale_group: int = 0,
                      stream=None, code_format: int = CODES_INT8) -> None:
    """rbd_rot_quant_act plus ld = X @ L1 (l1t = L1^T bf16 [r, K], ld bf16 [M, r])."""
    M, K = x.shape
    r = l1t.shape[0]
    if _rowstride(l1t) != K:
        raise ValueError("l1t must be a contiguous [r, K] tensor")
    _ok(load().rbd_lowrank_fused(_ptr(x), M, K, _rowstride(x), _qcfg(bits, rot_group, scale_group, code_format),
                                 _ptr(codes), _ptr(scales), _ptr(l1t), r, _ptr(ld), _stream(stream)),
        "rbd_lowrank_fused")


def rbd_lowrank_down(x: torch.Tensor, l1t: torch.Tensor, ld: torch.Tensor, stream=None) -> None:
    """ld = X @ L1 alone (l1t = L1^T bf16 [r, K], ld bf16 [M, r])."""
    M, K = x.shape
    r = l1t.shape[0]
    if _rowstride(l1t) != K:
        raise ValueError("l1t must be a contiguous [r, K] tensor")
    _ok(load().rbd_lowrank_down(_ptr(x), M, K, _rowstride(x), _ptr(l1t), r, _ptr(ld), _stream(stream)),
        "rbd_lowrank_down")


def rbd_pack_weights_int4(w: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, rot_group: int = 256,
                          scale_group: int = 0, stream=None) -> None:
    """w bf16 [N, K] -> packed uint8 [N, K/2], scales float32 [N] or [N, K/64]."""
    N, K = w.shape
    _ok(load().rbd_pack_weights_int4(_ptr(w), N, K, _qcfg(4, rot_group, scale_group), _ptr(packed),
                                     _ptr(scales), _stream(stream)), "rbd_pack_weights_int4")


def rbd_pack_weights_int8(w: torch.Tensor, w8: torch.Tensor, scales: torch.Tensor, rot_group: int = 256,
                          scale_group: int = 0, stream=None) -> None:
    """w bf16 [N, K] -> w8 int8 [N, K], scales float32 [N] or [N, K/64]."""
    N, K = w.shape
    _ok(load().rbd_pack_weights_int8(_ptr(w), N, K, _qcfg(8, rot_group, scale_group), _ptr(w8),
                                     _ptr(scales), _stream(stream)), "rbd_pack_weights_int8")


def make_epilogue(bias=None, ld=None, l2t=None, gate_mode: int = 0, gate_cols=(0, 0), gate=None,
                  residual=None, acc_debug=None) -> Epilogue:
    e = Epilogue()
    e.bias = _ptr(bias)
    e.ld = _ptr(ld)
    e.l2t = _ptr(l2t)
    e.r = 0 if ld is None else int(ld.shape[1])
    e.gate_mode = gate_mode
    e.gate_col0, e.gate_col1 = int(gate_cols[0]), int(gate_cols[1])
    e.gate = _ptr(gate)
    e.residual = _ptr(residual)
    e.ldr = 0 if residual is None else _rowstride(residual)
    e.acc_debug = _ptr(acc_debug)
    return e


def _linear(fn, where, codes, sx, w, sw, y, bits, rot_group, scale_group, epi, stream, code_format=CODES_INT8):
    M, K = codes.shape
    N = y.shape[1]
    e = epi if epi is not None else Epilogue()
    _ok(fn(_ptr(codes), _ptr(sx), _ptr(w), _ptr(sw), M, N, K, _qcfg(bits, rot_group, scale_group, code_format),
           ctypes.byref(e), _ptr(y), _rowstride(y), _stream(stream)), where)


def rbd_w4a4_linear(codes: torch.Tensor, sx: torch.Tensor, w_packed: torch.Tensor, sw: torch.Tensor,
                    y: torch.Tensor, scale_group: int = 0, epi: Optional[Epilogue] = None,
                    rot_group: int = 256, stream=None, code_format: int = CODES_INT8) -> None:
    """y bf16 [M, N] = epilogue(dequant(codes @ unpack(w_packed)^T)); codes in code_format (E4M3
    codes take the FP8 tensor-core path, group-64 scales only)."""
    _linear(load().rbd_w4a4_linear, "rbd_w4a4_linear", codes, sx, w_packed, sw, y, 4, rot_group,
            scale_group, epi, stream, code_format)


def rbd_w8a8_linear(codes: torch.Tensor, sx: torch.Tensor, w8: torch.Tensor, sw: torch.Tensor,
                    y: torch.Tensor, scale_group: int = 0, epi: Optional[Epilogue] = None,
                    rot_group: int = 256, stream=None) -> None:
    """y bf16 [M, N] = epilogue(dequant(codes @ w8^T))."""
    _linear(load().rbd_w8a8_linear, "rbd_w8a8_linear", codes, sx, w8, sw, y, 8, rot_group,
            scale_group, epi, stream)


def rbd_nvfp4_scale_bytes(rows: int, K: int) -> int:
    """Bytes of a tile-interleaved E4M3 block-scale buffer for `rows` rows of length K."""
    return int(load().rbd_nvfp4_scale_bytes(rows, K))


def rbd_nvfp4_quant(x: torch.Tensor, codes: torch.Tensor, block_scales: torch.Tensor, tensor_scale: torch.Tensor,
                    work: torch.Tensor, rot_group: int = 256, stream=None) -> None:
    """x bf16 [M, K] -> codes uint8 [M, K/2] (E2M1 pairs), block_scales uint8 (tile-interleaved E4M3,
    rbd_nvfp4_scale_bytes(M, K)), tensor_scale float32 [1]; work: 4 bytes of device scratch."""
    M, K = x.shape
    _ok(load().rbd_nvfp4_quant(_ptr(x), M, K, _rowstride(x), rot_group, _ptr(codes), _ptr(block_scales),
                               _ptr(tensor_scale), _ptr(work), _stream(stream)), "rbd_nvfp4_quant")


def rbd_nvfp4_quant_noalloc(x: torch.Tensor, codes: torch.Tensor, block_scales: torch.Tensor,
                            tensor_scale: torch.Tensor, rot_group: int = 256, stream=None) -> None:
    """rbd_nvfp4_quant with its scratch word in library-owned device memory (no scratch argument)."""
    M, K = x.shape
    _ok(load().rbd_nvfp4_quant_noalloc(_ptr(x), M, K, _rowstride(x), rot_group, _ptr(codes), _ptr(block_scales),
                                       _ptr(tensor_scale), _stream(stream)), "rbd_nvfp4_quant_noalloc")


def rbd_nvfp4_linear(xq, xbs, xgs, wq, wbs, wgs, y: torch.Tensor, epi: Optional[Epilogue] = None,
                     stream=None) -> None:
    """y bf16 [M, N] = epilogue(gs_x gs_w (Q_x . Q_w^T)) on the block-scaled FP4 tensor cores."""
    M, K2 = xq.shape
    N = y.shape[1]
    e = epi if epi is not None else Epilogue()
    _ok(load().rbd_nvfp4_linear(_ptr(xq), _ptr(xbs), _ptr(xgs), _ptr(wq), _ptr(wbs), _ptr(wgs), M, N, 2 * K2,
                                ctypes.byref(e), _ptr(y), _rowstride(y), _stream(stream)), "rbd_nvfp4_linear")


def rbd_check(stream=None) -> int:
    """Synchronise the stream and return the device status (0 = fine)."""
    return load().rbd_check(_stream(stream))


def rbd_debug_timeout_probe(timeout_ns: int, stream=None) -> None:
    _ok(load().rbd_debug_timeout_probe(int(timeout_ns), _stream(stream)), "rbd_debug_timeout_probe")


def rbd_status_string(status: int) -> str:
    return load().rbd_status_string(status).decode()


def rbd_version() -> str:
    return load().rbd_version().decode()


def rbd_kv4_encode(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, groups_per_band: int = 1,
                   slot0: int = 0, stream=None) -> None:
    """x bf16 [T, H*128] (row stride may be larger) -> cache slots (slot0 + t) mod capacity of
    codes uint8 [capacity, H, 64] and scales float32 [capacity, H, 3*groups_per_band]."""
    T = x.shape[0]
    capacity, H = codes.shape[0], codes.shape[1]
    _ok(load().rbd_kv4_encode(_ptr(x), T, H, _rowstride(x), groups_per_band, _ptr(codes), _ptr(scales),
                              capacity, slot0, _stream(stream)), "rbd_kv4_encode")


def rbd_kv4_decode(codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor, groups_per_band: int = 1,
                   slot0: int = 0, stream=None) -> None:
    """Cache slots (slot0 + t) mod capacity, t < y.shape[0] -> y bf16 [T, H*128]."""
    T = y.shape[0]
    capacity, H = codes.shape[0], codes.shape[1]
    _ok(load().rbd_kv4_decode(_ptr(codes), _ptr(scales), capacity, slot0, T, H, groups_per_band, _ptr(y),
                              _rowstride(y), _stream(stream)), "rbd_kv4_decode")


def rbd_qk_norm_rope(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, y: torch.Tensor,
                     gamma: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> None:
    """x bf16 [T, H*128] (row stride may be larger) -> y bf16 [T, H*128] (y may be x): per-head
    RMSNorm times gamma (bf16 [128] or None), then the RoPE turn by cos / sin float32 [T, 64]."""
    T = x.shape[0]
    if x.shape[1] % 128 or y.shape[0] != T or y.shape[1] != x.shape[1]:
        raise ValueError("x and y must be [T, H*128]")
    if cos.shape != (T, 64) or sin.shape != (T, 64) or not (cos.is_contiguous() and sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous [T, 64]")
    _ok(load().rbd_qk_norm_rope(_ptr(x), T, x.shape[1] // 128, _rowstride(x), _ptr(gamma), _ptr(cos), _ptr(sin),
                                eps, _ptr(y), _rowstride(y), _stream(stream)), "rbd_qk_norm_rope")


def rbd_rope_tables(pos: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, base: float = 10000.0,
                    stream=None) -> None:
    """pos int32 [T, 3] (time, height, width) -> cos, sin float32 [T, 64]."""
    T = pos.shape[0]
    if pos.dtype != torch.int32 or pos.shape != (T, 3) or not pos.is_contiguous():
        raise ValueError("pos must be contiguous int32 [T, 3]")
    if cos.shape != (T, 64) or sin.shape != (T, 64) or not (cos.is_contiguous() and sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous [T, 64]")
    _ok(load().rbd_rope_tables(_ptr(pos), T, base, _ptr(cos), _ptr(sin), _stream(stream)), "rbd_rope_tables")


def rbd_attn_workspace_bytes(Tk: int, H: int) -> int:
    """Bytes of device scratch rbd_attn_quant needs for Tk keys and H heads."""
    return int(load().rbd_attn_workspace_bytes(Tk, H))


def rbd_attn_quant(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, H: int, qc: torch.Tensor, sq: torch.Tensor,
                   kc: torch.Tensor, sk: torch.Tensor, vt: torch.Tensor, work: torch.Tensor, stream=None) -> None:
    """q bf16 [Tq, >=H*128], k / v bf16 [Tk, >=H*128] -> qc int8 [H, Tq, 128], sq float32 [H, Tq],
    kc int8 [H, Tk, 128], sk float32 [H, tkp], vt fp16 [H, 128, tkp] (tkp = sk.shape[1]);
    work: rbd_attn_workspace_bytes(Tk, H) bytes of device scratch."""
    Tq, Tk = q.shape[0], k.shape[0]
    tkp = sk.shape[1]
    if vt.shape[-1] != tkp:
        raise ValueError("sk and vt must share the padded key count")
    _ok(load().rbd_attn_quant(_ptr(q), _rowstride(q), _ptr(k), _rowstride(k), _ptr(v), _rowstride(v), Tq, Tk, H,
                              _ptr(qc), _ptr(sq), _ptr(kc), _ptr(sk), _ptr(vt), tkp, _ptr(work), _stream(stream)),
        "rbd_attn_quant")


def rbd_attn_int8(qc: torch.Tensor, sq: torch.Tensor, kc: torch.Tensor, sk: torch.Tensor, vt: torch.Tensor,
                  o: torch.Tensor, stream=None) -> None:
    """Attention on rbd_attn_quant's operands -> o bf16 [Tq, >=H*128]."""
    H, Tq = sq.shape
    Tk = kc.shape[1]
    _ok(load().rbd_attn_int8(_ptr(qc), _ptr(sq), _ptr(kc), _ptr(sk), _ptr(vt), Tq, Tk, H, sk.shape[1], _ptr(o),
                             _rowstride(o), _stream(stream)), "rbd_attn_int8")


def _at(t: torch.Tensor, cur: int) -> int:
    """Device address of a CUDA tensor on device `cur`, the current one (see _ptr)."""
    if t.get_device() != cur:
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        raise ValueError(f"tensor on {t.device} while cuda:{cur} is current; call under torch.cuda.device({t.device})")
    return t.data_ptr()


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, cur: int) -> int:
    """cudaStream_t of `stream`, or of the current stream of device `cur` (without making a Stream object of it,
    which costs as much as a launch)."""
    if stream is None:
        return _current_raw_stream(cur) if _current_raw_stream else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _kv8(table: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, code_format: int, cur: int) -> Kv8:
    """The rbd_kv8 of table int32 [seqs, pages per sequence], codes uint8 [pages, heads, 2, 64, 128] and
    scales float32 [pages, heads, 2]."""
    s = codes.shape
    if codes.dtype != torch.uint8 or len(s) != 5 or s[2] != 2 or s[3] != 64 or s[4] != 128 or not codes.is_contiguous():
        raise ValueError("codes must be contiguous uint8 [pages, heads, 2, 64, 128]")
    z = scales.shape
    if scales.dtype != torch.float32 or len(z) != 3 or z[0] != s[0] or z[1] != s[1] or z[2] != 2 or \
            not scales.is_contiguous():
        raise ValueError("scales must be contiguous float32 [pages, heads, 2]")
    t = table.shape
    if table.dtype != torch.int32 or len(t) != 2 or (t[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be row-major int32 [seqs, pages per sequence]")
    return Kv8(_at(codes, cur), _at(scales, cur), _at(table, cur), table.stride(0) if t[0] > 1 else t[1], s[0], t[1], t[0],
               s[1], code_format)


def _i32(t: torch.Tensor, count: int, what: str, cur: int) -> int:
    """Device address of a contiguous int32 vector of `count` elements."""
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != count or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 [{count}]")
    return _at(t, cur)


def _bf16_rows(t: torch.Tensor, cols: int, what: str) -> int:
    """Row stride of bf16 [rows, >= cols]."""
    s = t.shape
    if t.dtype != torch.bfloat16 or len(s) != 2 or s[1] < cols or t.stride(1) != 1:
        raise ValueError(f"{what} must be bf16 [rows, >= {cols}], rows contiguous")
    return t.stride(0) if s[0] > 1 else cols + -cols % 8       # a single row's stride means nothing


def _weights(t: torch.Tensor, seqs: int, heads: int, what: str):
    """(sequence stride, head stride, columns) of float32 [seqs, heads, columns]."""
    s = t.shape
    if t.dtype != torch.float32 or len(s) != 3 or s[0] != seqs or s[1] != heads or (s[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{what} must be float32 [{seqs}, {heads}, columns] with adjacent columns")
    return t.stride(0), (t.stride(1) if heads > 1 else max(t.stride(1), s[2])), s[2]


def _kv8_append(c: Kv8, cur: int, lens: int, cu: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    cols = c.heads * 128
    ldk, ldv = _bf16_rows(k, cols, "k"), _bf16_rows(v, cols, "v")
    rows = k.shape[0]
    if rows != v.shape[0]:
        raise ValueError("k and v differ in rows")
    _ok(load().rbd_kv8_append(c, lens, cu, _at(k, cur), ldk, _at(v, cur), ldv, rows, _raw_stream(stream, cur)),
        "rbd_kv8_append")


def rbd_kv8_append(k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                   codes: torch.Tensor, scales: torch.Tensor, code_format: int = CODES_INT8, stream=None) -> None:
    """k, v bf16 [rows, >= heads*128] -> tokens lens[b] .. of every sequence b, whose rows are cu[b] ..
    cu[b+1] - 1 (cu int32 [seqs + 1], lens int32 [seqs]; lens is not changed)."""
    cur = torch.cuda.current_device()
    c = _kv8(table, codes, scales, code_format, cur)
    _kv8_append(c, cur, _i32(lens, c.seqs, "lens", cur), _i32(cu, c.seqs + 1, "cu", cur), k, v, stream)


def _kv8_read(c: Kv8, cur: int, lens: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    cols = c.heads * 128
    s = k.shape
    if s != v.shape or len(s) != 3 or s[0] != c.seqs or s[2] != cols or k.dtype != torch.bfloat16 or \
            v.dtype != torch.bfloat16 or not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous bf16 [seqs, tokens, heads*128]")
    _ok(load().rbd_kv8_read(c, lens, s[1], _at(k, cur), cols, _at(v, cur), cols, _raw_stream(stream, cur)), "rbd_kv8_read")


def rbd_kv8_read(lens: torch.Tensor, table: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, k: torch.Tensor,
                 v: torch.Tensor, code_format: int = CODES_INT8, stream=None) -> None:
    """The last T tokens of every sequence -> k, v bf16 [seqs, T, heads*128] (contiguous; zeros in front of a
    sequence's first token)."""
    cur = torch.cuda.current_device()
    c = _kv8(table, codes, scales, code_format, cur)
    _kv8_read(c, cur, _i32(lens, c.seqs, "lens", cur), k, v, stream)


def rbd_kv8_attn_workspace_bytes(seqs: int, heads: int, q_heads: int, rows: int, max_len: int,
                                 weigh: bool = False) -> int:
    """Bytes of device scratch rbd_kv8_attn needs (-1 for bad sizes)."""
    return int(load().rbd_kv8_attn_workspace_bytes(seqs, heads, q_heads, rows, max_len, int(weigh)))


def _kv8_attn(c: Kv8, cur: int, lens: int, cu: int, q: torch.Tensor, o: torch.Tensor, q_heads: int,
              work: Optional[torch.Tensor], max_len: int, causal: bool, softmax_scale: float,
              weights_in: Optional[torch.Tensor], weights_out: Optional[torch.Tensor], stream=None) -> None:
    ldq, ldo = _bf16_rows(q, q_heads * 128, "q"), _bf16_rows(o, q_heads * 128, "o")
    rows = q.shape[0]
    if rows != o.shape[0]:
        raise ValueError("q and o differ in rows")
    w_in = w_out = None
    w_seq = w_head = 0
    if weights_in is not None or weights_out is not None:
        if weights_in is None or weights_out is None:
            raise ValueError("weights_in and weights_out go together")
        w_seq, w_head, width = _weights(weights_out, c.seqs, c.heads, "weights_out")
        if (weights_in is not weights_out and
                _weights(weights_in, c.seqs, c.heads, "weights_in") != (w_seq, w_head, width)) or width < max_len:
            raise ValueError("weights_in and weights_out must agree in shape and strides and hold max_len columns")
        w_in, w_out = _at(weights_in, cur), _at(weights_out, cur)
    _ok(load().rbd_kv8_attn(c, lens, cu, _at(q, cur), ldq, rows, q_heads, causal, softmax_scale, max_len, _at(o, cur), ldo,
                            w_in, w_out, w_seq, w_head, None if work is None else _at(work, cur),
                            0 if work is None else work.numel() * work.element_size(), _raw_stream(stream, cur)),
        "rbd_kv8_attn")


def rbd_kv8_attn(q: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, codes: torch.Tensor,
                 scales: torch.Tensor, o: torch.Tensor, q_heads: int, work: Optional[torch.Tensor], max_len: int,
                 causal: bool = True, softmax_scale: float = 128 ** -0.5, weights_in: Optional[torch.Tensor] = None,
                 weights_out: Optional[torch.Tensor] = None, code_format: int = CODES_INT8, stream=None) -> None:
    """q bf16 [rows, >= q_heads*128] -> o bf16, attention over the cached tokens; weights_in / weights_out
    float32 [seqs, heads, >= max_len] add up every key's attention weight (both or neither; the same one works).
    work: rbd_kv8_attn_workspace_bytes bytes of scratch (None for 0)."""
    cur = torch.cuda.current_device()
    c = _kv8(table, codes, scales, code_format, cur)
    _kv8_attn(c, cur, _i32(lens, c.seqs, "lens", cur), _i32(cu, c.seqs + 1, "cu", cur), q, o, q_heads, work, max_len,
              causal, softmax_scale, weights_in, weights_out, stream)


def rbd_kv8_evict(weights: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, codes: torch.Tensor,
                  scales: torch.Tensor, keep: int, recent: int, dst_table: torch.Tensor, kept: torch.Tensor,
                  weights_out: torch.Tensor, lens_out: torch.Tensor, code_format: int = CODES_INT8,
                  stream=None) -> None:
    """Keep min(lens, keep) tokens of every (sequence, head): the last `recent` ones and those of largest weight
    (weights float32 [seqs, heads, width >= lens]), quantised into the pages of dst_table int32 [seqs, >= ceil(keep / 64)]
    (none of them held by a sequence).  kept int32 [seqs, heads, keep] gets the positions (-1 behind them),
    weights_out float32 [seqs, heads, >= keep] their weights (zeros behind; may be weights), lens_out the new lengths."""
    cur = torch.cuda.current_device()
    c = _kv8(table, codes, scales, code_format, cur)
    w_seq, w_head, width = _weights(weights, c.seqs, c.heads, "weights")
    o_seq, o_head, width_out = _weights(weights_out, c.seqs, c.heads, "weights_out")
    d = dst_table.shape
    if dst_table.dtype != torch.int32 or len(d) != 2 or d[0] != c.seqs or d[1] * 64 < keep or \
            (d[1] > 1 and dst_table.stride(1) != 1):
        raise ValueError("dst_table must be row-major int32 [seqs, >= ceil(keep / 64)]")
    s = kept.shape
    if kept.dtype != torch.int32 or len(s) != 3 or s[0] != c.seqs or s[1] != c.heads or s[2] != keep or \
            not kept.is_contiguous():
        raise ValueError("kept must be contiguous int32 [seqs, heads, keep]")
    _ok(load().rbd_kv8_evict(c, _i32(lens, c.seqs, "lens", cur), _at(weights, cur), w_seq, w_head, width, keep, recent,
                             _at(dst_table, cur), dst_table.stride(0) if d[0] > 1 else d[1], _at(kept, cur),
                             _at(weights_out, cur), o_seq, o_head, width_out, _i32(lens_out, c.seqs, "lens_out", cur),
                             _raw_stream(stream, cur)), "rbd_kv8_evict")


def rbd_svdquant_fit(w: torch.Tensor, rank: int, omegas, bits: int = 4, rot_group: int = 256, scale_group: int = 0,
                     act_rms=None, stream=None):
    """The offline SVDQuant fit of a bf16 [N, K] CUDA weight.  omegas: float64 array-like
    [iters, K, rank + oversample] (the test matrices); act_rms: float64 [K] or None.
    Returns dict(q, scales (CUDA tensors of the kept iterate), l1 [K, rank], l2 [rank, N] (float64
    numpy), errs [iters] (float64 numpy), best).  Synchronous."""
    import numpy as np
    N, K = w.shape
    om = np.ascontiguousarray(omegas, dtype=np.float64)
    iters, k_, p = om.shape
    if k_ != K or p < rank:
        raise ValueError("omegas must be [iters, K, rank + oversample]")
    cfg = _qcfg(bits, rot_group, scale_group)
    nbytes = int(load().rbd_svdquant_workspace_bytes(N, K, rank, p - rank, cfg))
    if nbytes < 0:
        raise RbdError(2, "rbd_svdquant_workspace_bytes")
    dev = w.device
    work = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
    q = torch.empty((N, K // 2) if bits == 4 else (N, K), dtype=torch.uint8 if bits == 4 else torch.int8, device=dev)
    scales = torch.empty((N, K // 64) if scale_group else (N,), dtype=torch.float32, device=dev)
    l1 = np.zeros((K, rank), np.float64)
    l2 = np.zeros((rank, N), np.float64)
    errs = np.zeros(iters, np.float64)
    best = ctypes.c_int32(-1)
    ar = None if act_rms is None else np.ascontiguousarray(act_rms, dtype=np.float64)
    dp = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
    _ok(load().rbd_svdquant_fit(_ptr(w), N, K, cfg, rank, p - rank, iters, dp(om), dp(ar), _ptr(q), _ptr(scales),
                                dp(l1), dp(l2), dp(errs), ctypes.byref(best), _ptr(work), _stream(stream)),
        "rbd_svdquant_fit")
    return dict(q=q, scales=scales, l1=l1, l2=l2, errs=errs, best=int(best.value))
