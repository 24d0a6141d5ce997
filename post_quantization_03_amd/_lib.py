"""ctypes binding of libkq.so (include/kq.h). Argument marshalling only: every step runs in the
library's HIP kernels. Tensors supply device pointers; the stream is torch's current stream.

The library must be built (python -m post_quantization_03_amd.build); there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkq.so")

KQ_F32, KQ_BF16 = 0, 1
HG_FORM = {"diag": 0, "block": 1, "full": 2}
OP = {"hessian": 0, "rotate_in": 1, "hg_sqrt": 2, "rotate_out": 3, "cholinv": 4, "quantize": 5, "unrotate": 6,
      "loss": 7, "matvec": 8, "hg_lowrank": 9, "kfac_loss": 10, "cross": 11, "drift": 12, "mx_gemm": 13,
      "mx_gated": 14, "gated_forward": 15, "gated_backward": 16, "i8_gemm": 17, "i8_gated": 18, "grouped_gemm": 19,
      "grouped_gated": 20, "grouped_backward": 21, "norm_backward": 22}
ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
NORM = {"layer": 0, "rms": 1}
EXPORTS = ("kq_workspace_bytes", "kq_hessian_accum", "kq_rotate_in", "kq_hg_sqrt", "kq_rotate_out", "kq_cholinv",
           "kq_quantize_layer", "kq_sensitivity", "kq_unrotate", "kq_layer_loss", "kq_strerror", "kq_last_error",
           "kq_hadamard_order", "kq_version", "kq_allocate_bits", "kq_matvec_quantized",
           "kq_hg_extract", "kq_hg_lowrank", "kq_kfac_loss", "kq_quantize_layer_search",
           "kq_block_order", "kq_permute_blocks", "kq_cross_accum", "kq_drift_target", "kq_matvec_quantized_static",
           "kq_mx_quantize", "kq_mx_dequantize", "kq_mx_gemm", "kq_mx_gated", "kq_gated_forward", "kq_gated_backward",
           "kq_i8_quantize", "kq_i8_dequantize", "kq_i8_gemm", "kq_i8_gated", "kq_grouped_gemm", "kq_grouped_gated",
           "kq_grouped_backward", "kq_norm_forward", "kq_norm_backward")


class KQError(RuntimeError):
    def __init__(self, name: str, status: int, detail: str):
        super().__init__(f"{name} failed: status {status} ({strerror(status)}): {detail}")
        self.status = status


_lib = None
_i64, _vp, _f32, _int, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run `python -m post_quantization_03_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    sig = {
        "kq_workspace_bytes": (_sz, [_int, _i64, _i64, _i64, _int, _int, _int, _int, _i64]),
        "kq_hessian_accum": (_int, [_vp, _int, _i64, _i64, _i64, ctypes.c_double, ctypes.c_double, _vp, _vp, _sz, _vp]),
        "kq_rotate_in": (_int, [_vp, _int, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
        "kq_hg_sqrt": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
        "kq_rotate_out": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _i64, _vp, _vp, _sz, _vp]),
        "kq_cholinv": (_int, [_vp, _i64, _i64, ctypes.c_double, _vp, _vp, _vp, _sz, _vp]),
        "kq_quantize_layer": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _int, _int, _int, _vp, _vp, _vp, _vp, _vp, _sz,
                                     _vp]),
        "kq_sensitivity": (_int, [_vp, _i64, _i64, _vp, _int, _i64, _i64, _vp, _vp]),
        "kq_unrotate": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _int, _i64, _vp, _i64, _vp, _sz, _vp]),
        "kq_layer_loss": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
        "kq_strerror": (ctypes.c_char_p, [_int]),
        "kq_last_error": (ctypes.c_char_p, []),
        "kq_hadamard_order": (_i64, [_i64, ctypes.POINTER(_i64)]),
        "kq_version": (_int, []),
        "kq_allocate_bits": (_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64), _i64, ctypes.c_double, _int,
                                    _int, ctypes.POINTER(ctypes.c_int32)]),
        "kq_matvec_quantized": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _int, _vp, _vp, _vp, _int, _i64, _vp, _i64, _i64,
                                       _vp, _i64, _vp, _sz, _vp]),
        "kq_matvec_quantized_static": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _int, _vp, _vp, _vp, _int, _i64, _vp,
                                              _i64, _i64, _vp, _i64, _vp]),
        "kq_hg_extract": (_int, [_vp, _i64, _i64, _int, _i64, _vp, _vp]),
        "kq_block_order": (_int, [_vp, _i64, _i64, _i64, _vp, _vp]),
        "kq_cross_accum": (_int, [_vp, _vp, _int, _i64, _i64, _i64, _i64, ctypes.c_double, ctypes.c_double, _vp, _vp,
                                  _sz, _vp]),
        "kq_drift_target": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _sz, _vp]),
        "kq_permute_blocks": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _int, _int, _vp, _vp]),
        "kq_quantize_layer_search": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _int, _int, _int, _int, _vp, _vp, _vp,
                                            _vp, _vp, _sz, _vp]),
        "kq_hg_lowrank": (_int, [_vp, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
        "kq_kfac_loss": (_int, [_vp, _int, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _int, _i64, _vp, _vp, _sz,
                                _vp]),
        "kq_mx_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]),
        "kq_mx_dequantize": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _int, _i64, _vp]),
        "kq_mx_gemm": (_int, [_vp, _i64] * 4 + [_i64, _i64, _i64, _vp, _int, _i64, _vp, _sz, _vp]),
        "kq_mx_gated": (_int, [_vp, _i64] * 6 + [_i64, _i64, _i64, _int, _vp, _int, _i64, _vp, _sz, _vp]),
        "kq_gated_forward": (_int, [_vp, _i64] * 3 + [_int, _i64, _i64, _i64, _int] + [_vp, _i64] * 3 + [_vp, _sz, _vp]),
        "kq_gated_backward": (_int, [_vp, _i64] * 6 + [_int, _i64, _i64, _i64, _int] + [_vp, _i64] * 5 + [_vp, _sz, _vp]),
        "kq_i8_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _vp, _vp]),
        "kq_i8_dequantize": (_int, [_vp, _i64, _vp, _i64, _i64, _vp, _int, _i64, _vp]),
        "kq_i8_gemm": (_int, [_vp, _i64, _vp] * 2 + [_vp, _i64, _i64, _i64, _i64, _vp, _int, _i64, _vp, _sz, _vp]),
        "kq_i8_gated": (_int, [_vp, _i64, _vp] * 3 + [_vp, _i64, _i64, _i64, _i64, _int, _vp, _int, _i64, _vp, _sz, _vp]),
        "kq_grouped_gemm": (_int, [_vp, _i64] * 2 + [_vp, _i64, _int, _i64, _i64, _i64, _vp, _i64, _vp, _sz, _vp]),
        "kq_grouped_gated": (_int, [_vp, _i64] * 3 + [_vp, _i64, _int, _i64, _i64, _i64, _int] + [_vp, _i64] * 3 +
                             [_vp, _sz, _vp]),
        "kq_grouped_backward": (_int, [_vp, _i64] * 5 + [_vp, _i64, _int, _i64, _i64, _i64] + [_vp, _i64] * 3 + [_vp, _sz, _vp]),
        "kq_norm_forward": (_int, [_vp, _i64, _vp, _vp, _int, _i64, _i64, _int, _f32, _vp, _i64, _vp, _vp, _vp]),
        "kq_norm_backward": (_int, [_vp, _i64] * 2 + [_vp, _vp, _vp, _int, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def strerror(status: int) -> str:
    return lib().kq_strerror(status).decode()


def last_error() -> str:
    return lib().kq_last_error().decode()


def _check(name: str, status: int) -> None:
    if status != 0:
        raise KQError(name, status, last_error())


def _p(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ws(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _xdt(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return KQ_BF16
    if t.dtype == torch.float32:
        return KQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ----------------------------------------------------------------------------------- wrappers
def kq_workspace_bytes(op: str, o: int = 0, i: int = 0, n: int = 0, xdt: int = KQ_BF16, bits: int = 0,
                       group: int = 0, form: str = "diag", blk: int = 0) -> int:
    return int(lib().kq_workspace_bytes(OP[op], o, i, n, xdt, bits, group, HG_FORM[form], blk))


def kq_hadamard_order(d: int) -> tuple[int, int]:
    p2 = _i64(0)
    m = lib().kq_hadamard_order(d, ctypes.byref(p2))
    return int(m), int(p2.value)


def kq_hessian_accum(X, H, alpha: float, beta: float, ws=None, stream=None) -> None:
    n, d = X.shape
    w, wb = _ws(ws)
    _check("kq_hessian_accum", lib().kq_hessian_accum(_p(X), _xdt(X), n, d, X.stride(0), alpha, beta, _p(H), w, wb,
                                                      _stream(stream)))


def kq_rotate_in(Win, Wout, HX, sign_in, ws=None, stream=None) -> None:
    o, i = Win.shape
    w, wb = _ws(ws)
    _check("kq_rotate_in", lib().kq_rotate_in(_p(Win), _xdt(Win), Win.stride(0), _p(Wout), Wout.stride(0), o, i,
                                              _p(HX), _p(sign_in), w, wb, _stream(stream)))


def kq_rotate_in_hessian(HX, sign_in, ws=None, stream=None) -> None:
    """kq_rotate_in with no weights: HX <- U^T HX U."""
    i = HX.shape[0]
    w, wb = _ws(ws)
    _check("kq_rotate_in", lib().kq_rotate_in(None, KQ_F32, i, None, i, 0, i, _p(HX), _p(sign_in), w, wb,
                                              _stream(stream)))


def kq_hg_sqrt(HG, form: str, o: int, blk: int, S, Sinv, info, ws=None, stream=None) -> None:
    w, wb = _ws(ws)
    _check("kq_hg_sqrt", lib().kq_hg_sqrt(_p(HG), HG_FORM[form], o, blk, _p(S), _p(Sinv), _p(info), w, wb,
                                          _stream(stream)))


def kq_rotate_out(W, S, form: str, blk: int, sign_out, ws=None, stream=None) -> None:
    o, i = W.shape
    w, wb = _ws(ws)
    _check("kq_rotate_out", lib().kq_rotate_out(_p(W), o, i, W.stride(0), _p(S), HG_FORM[form], blk, _p(sign_out), w,
                                                wb, _stream(stream)))


def kq_cholinv(HX, damp: float, R, info, ws=None, stream=None) -> None:
    i = HX.shape[0]
    w, wb = _ws(ws)
    _check("kq_cholinv", lib().kq_cholinv(_p(HX), i, HX.stride(0), damp, _p(R), _p(info), w, wb, _stream(stream)))


def kq_quantize_layer(W, R, bits: int, group: int, block: int, codes, scale, offset, row_loss=None, ws=None,
                      stream=None) -> None:
    o, i = W.shape
    w, wb = _ws(ws)
    _check("kq_quantize_layer", lib().kq_quantize_layer(_p(W), o, i, W.stride(0), _p(R), R.stride(0), bits, group,
                                                        block, _p(codes), _p(scale), _p(offset), _p(row_loss), w, wb,
                                                        _stream(stream)))


def kq_quantize_layer_search(W, R, bits: int, group: int, block: int, candidates: int, codes, scale, offset,
                             row_loss=None, ws=None, stream=None) -> None:
    o, i = W.shape
    w, wb = _ws(ws)
    _check("kq_quantize_layer_search",
           lib().kq_quantize_layer_search(_p(W), o, i, W.stride(0), _p(R), R.stride(0), bits, group, block, candidates,
                                          _p(codes), _p(scale), _p(offset), _p(row_loss), w, wb, _stream(stream)))


def kq_block_order(H, width: int, order, stream=None) -> None:
    i = H.shape[0]
    _check("kq_block_order", lib().kq_block_order(_p(H), i, H.stride(0), width, _p(order), _stream(stream)))


def kq_permute_blocks(src, dst, width: int, axis: int, perm, stream=None) -> None:
    rows, cols = src.shape
    _check("kq_permute_blocks", lib().kq_permute_blocks(_p(src), src.stride(0), _p(dst), dst.stride(0), rows, cols,
                                                        width, axis, src.element_size(), _p(perm), _stream(stream)))


def kq_cross_accum(A, B, C, alpha: float, beta: float, ws=None, stream=None) -> None:
    n, d = A.shape
    if B.shape != A.shape or B.dtype != A.dtype:
        raise ValueError("kq_cross_accum: A and B must have the same shape and dtype")
    w, wb = _ws(ws)
    _check("kq_cross_accum", lib().kq_cross_accum(_p(A), _p(B), _xdt(A), n, d, A.stride(0), B.stride(0), alpha, beta,
                                                  _p(C), w, wb, _stream(stream)))


def kq_drift_target(W, C, R, Wt, ws=None, stream=None) -> None:
    o, i = W.shape
    w, wb = _ws(ws)
    _check("kq_drift_target", lib().kq_drift_target(_p(W), _xdt(W), W.stride(0), o, i, _p(C), C.stride(0), _p(R),
                                                    R.stride(0), _p(Wt), Wt.stride(0), w, wb, _stream(stream)))


def kq_sensitivity(HX, HG, form: str, o: int, blk: int, score, stream=None) -> None:
    i = HX.shape[0]
    _check("kq_sensitivity", lib().kq_sensitivity(_p(HX), i, HX.stride(0), _p(HG), HG_FORM[form], o, blk, _p(score),
                                                  _stream(stream)))


def kq_unrotate(Q, sign_in, sign_out, Sinv, form: str, blk: int, What, ws=None, stream=None) -> None:
    o, i = Q.shape
    w, wb = _ws(ws)
    _check("kq_unrotate", lib().kq_unrotate(_p(Q), o, i, Q.stride(0), _p(sign_in), _p(sign_out), _p(Sinv),
                                            HG_FORM[form], blk, _p(What), What.stride(0), w, wb, _stream(stream)))


def kq_matvec_quantized(codes, scale, offset, o: int, i: int, bits: int, group: int, sign_in, sign_out, Sinv,
                        form: str, blk: int, X, Y, ws=None, stream=None) -> None:
    """Y (nt x o) = W^ X^T for the tokens in the rows of X (nt x i), from the packed codes."""
    nt = X.shape[0]
    w, wb = _ws(ws)
    _check("kq_matvec_quantized", lib().kq_matvec_quantized(_p(codes), _p(scale), _p(offset), o, i, bits, group,
                                                            _p(sign_in), _p(sign_out), _p(Sinv), HG_FORM[form], blk,
                                                            _p(X), X.stride(0), nt, _p(Y), Y.stride(0), w, wb,
                                                            _stream(stream)))


def kq_matvec_quantized_static(codes, scale, offset, o: int, i: int, bits: int, group: int, sign_in, sign_out, Sinv,
                               form: str, blk: int, X, Y, stream=None) -> None:
    """kq_matvec_quantized on the library's fixed per-device scratch array (no workspace argument)."""
    nt = X.shape[0]
    _check("kq_matvec_quantized_static",
           lib().kq_matvec_quantized_static(_p(codes), _p(scale), _p(offset), o, i, bits, group, _p(sign_in),
                                            _p(sign_out), _p(Sinv), HG_FORM[form], blk, _p(X), X.stride(0), nt, _p(Y),
                                            Y.stride(0), _stream(stream)))


def kq_hg_extract(H, form: str, blk: int, HG, stream=None) -> None:
    o = H.shape[0]
    _check("kq_hg_extract", lib().kq_hg_extract(_p(H), o, H.stride(0), HG_FORM[form], blk, _p(HG), _stream(stream)))


def kq_hg_lowrank(G, k: int, q: int, omega, S, Sinv, HGhat, sigma, info, ws=None, stream=None) -> None:
    n, o = G.shape
    w, wb = _ws(ws)
    _check("kq_hg_lowrank", lib().kq_hg_lowrank(_p(G), n, o, G.stride(0), k, q, _p(omega), _p(S), _p(Sinv),
                                                _p(HGhat), _p(sigma), _p(info), w, wb, _stream(stream)))


def kq_kfac_loss(W, What, HX, HG, form: str, blk: int, loss, ws=None, stream=None) -> None:
    o, i = What.shape
    w, wb = _ws(ws)
    _check("kq_kfac_loss", lib().kq_kfac_loss(_p(W), _xdt(W), W.stride(0), _p(What), What.stride(0), o, i, _p(HX),
                                              HX.stride(0), _p(HG), HG_FORM[form], blk, _p(loss), w, wb,
                                              _stream(stream)))


def kq_layer_loss(W2, Q, HX2, row_loss, loss, ws=None, stream=None) -> None:
    o, i = W2.shape
    w, wb = _ws(ws)
    _check("kq_layer_loss", lib().kq_layer_loss(_p(W2), _p(Q), o, i, W2.stride(0), _p(HX2), HX2.stride(0),
                                                _p(row_loss), _p(loss), w, wb, _stream(stream)))


def kq_allocate_bits(scores, sizes, budget: float = 3.0, bmin: int = 2, bmax: int = 4):
    """Host call: bit-width per sublayer from the sensitivity scores (see include/kq.h)."""
    import numpy as np
    sc = np.ascontiguousarray(scores, dtype=np.float64)
    sz = np.ascontiguousarray(sizes, dtype=np.int64)
    out = np.zeros(len(sc), dtype=np.int32)
    _check("kq_allocate_bits", lib().kq_allocate_bits(sc.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                                      sz.ctypes.data_as(ctypes.POINTER(_i64)), len(sc), budget, bmin,
                                                      bmax, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))
    return out


# ------------------------------------------------- microscaled 4-bit products and the gated block
# These wrappers also check what the C calls cannot see: types, shapes, devices and the memory behind a
# view (rows are read in whole 16-byte pieces). A call on few tokens runs for a few microseconds on the
# GPU, so the checks read each tensor's attributes once and no device guard is entered on the current device.
_TORCH: tuple | None = None


def _torch() -> tuple:
    """torch.uint8, the raw current stream of a device, the current device, and torch dtype -> (kq_dtype,
    elements in 16 bytes): looked up at the first call and published whole, since two threads may come here at
    once."""
    global _TORCH
    if _TORCH is None:
        import torch
        raw, cur = (getattr(torch._C, k, None) for k in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        _TORCH = (torch.uint8, raw or (lambda d: torch.cuda.current_stream(d).cuda_stream), cur or torch.cuda.current_device,
                  {torch.float32: (KQ_F32, 4), torch.bfloat16: (KQ_BF16, 8)})
    return _TORCH


def _float(name: str, what: str, t):
    """(kq_dtype, elements in 16 bytes, device) of a tensor."""
    f = (_TORCH or _torch())[3].get(t.dtype)
    if f is None:
        raise TypeError(f"{name}: {what} has type {t.dtype}")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name}: {what} is not on a GPU")
    return f[0], f[1], d


def _matrix(name: str, what: str, t, rows: int, cols: int, dtype, per: int, whole: bool, dev: int):
    """Checks a row-major rows x cols matrix of `dtype` on device `dev`; returns (pointer, leading
    dimension). whole: its rows are read in pieces of `per` elements, the last one included."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {what} has type {t.dtype}, not {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: {what} has shape {tuple(t.shape)}, not {(rows, cols)}")
    if t.get_device() != dev:
        _other_device(name, what, t, dev)
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: {what} is not row-major")
    if rows <= 1:       # the stride of a single row is arbitrary: any legal one will do
        ld = -(-cols // per) * per
    if whole and cols % per and rows:
        end = t.storage_offset() + (rows - 1) * ld + -(-cols // per) * per
        if end * t.element_size() > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: the last row of {what} ends inside its 16 bytes, past the storage")
    return t.data_ptr(), ld


def _other_device(name: str, what: str, t, dev: int) -> None:
    if t.get_device() < 0:
        raise ValueError(f"{name}: {what} is not on a GPU")
    raise ValueError(f"{name}: operands on different devices: {what} on {t.device}, others on cuda:{dev}")


def _mx(name: str, what: str, codes, scales, cols: int, dev: int) -> tuple:
    """Checks a microscaled operand of `cols` columns; returns its four C arguments."""
    u8 = (_TORCH or _torch())[0]
    if codes.dtype is not u8 or scales.dtype is not u8:
        raise TypeError(f"{name}: {what} codes and scales have types {codes.dtype} and {scales.dtype}, not uint8")
    cs, ss = codes.shape, scales.shape
    if len(cs) != 2 or len(ss) != 2 or cs[0] != ss[0]:
        raise ValueError(f"{name}: {what} needs codes and scales with one row for each of the matrix")
    if codes.get_device() != dev:
        _other_device(name, what + " codes", codes, dev)
    if scales.get_device() != dev:
        _other_device(name, what + " scales", scales, dev)
    nblk = (cols + 31) // 32
    rows, wide, have = cs[0], (nblk + 3) // 4 * 4, ss[1]
    if cs[1] != 16 * nblk or not nblk <= have <= wide:
        raise ValueError(f"{name}: {what} of {cols} columns needs 16 * {nblk} bytes of codes and {nblk} scales a row "
                         f"(mx_empty), not {cs[1]} and {have}")
    (ldc, c1), (lds, s1) = codes.stride(), scales.stride()
    if c1 != 1 or (s1 != 1 and have > 1):
        raise ValueError(f"{name}: {what} is not row-major")
    if rows <= 1:
        ldc, lds = 16 * nblk, wide
    if have != wide and rows and scales.storage_offset() + (rows - 1) * lds + wide > scales.untyped_storage().nbytes():
        raise ValueError(f"{name}: the last scale row of {what} ends inside its 4 bytes, past the storage")
    return codes.data_ptr(), ldc, scales.data_ptr(), lds


def _workspace(name: str, ws, dev: int) -> tuple:
    if ws is None:
        return None, 0
    if ws.get_device() != dev:
        _other_device(name, "the workspace", ws, dev)
    if not ws.is_contiguous():      # its size in bytes would not be that of the memory behind it
        raise ValueError(f"{name}: the workspace is not contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _launch(name: str, fn, dev: int, stream, args: tuple) -> None:
    """fn(*args, stream) on device `dev`."""
    _, raw_stream, current_device, _ = _TORCH or _torch()
    if stream is None:
        s = raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{name}: the stream is on {stream.device}, the operands on cuda:{dev}")
    else:
        s = stream.cuda_stream
    if current_device() == dev:
        status = fn(*args, s)
    else:
        import torch
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status:
        raise KQError(name, status, last_error())


def _act(name: str, act: str) -> int:
    if act not in ACT:
        raise ValueError(f"{name}: activation {act!r} is none of {sorted(ACT)}")
    return ACT[act]


def mx_empty(rows: int, cols: int, device):
    """Buffers for a rows x cols matrix in the microscaled format: codes (16 bytes per 32 columns) and
    scales (one byte per 32 columns, rows padded to 4 bytes), both uint8, contents undefined."""
    import torch
    nblk = -(-cols // 32)
    return (torch.empty((rows, 16 * nblk), dtype=torch.uint8, device=device),
            torch.empty((rows, -(-nblk // 4) * 4), dtype=torch.uint8, device=device))


def kq_mx_quantize(X, codes, scales, stream=None) -> None:
    """X (rows x cols, fp32 or bf16) into codes and scales of mx_empty(rows, cols)."""
    name = "kq_mx_quantize"
    rows, cols = X.shape
    dt, per, dev = _float(name, "X", X)
    p, ld = _matrix(name, "X", X, rows, cols, X.dtype, per, False, dev)
    if codes.shape[0] != rows:
        raise ValueError(f"{name}: {codes.shape[0]} rows of codes for {rows} rows")
    _launch(name, lib().kq_mx_quantize, dev, stream, (p, dt, rows, cols, ld, *_mx(name, "the output", codes, scales, cols, dev)))


def kq_mx_dequantize(codes, scales, Y, stream=None) -> None:
    """The values that codes and scales stand for, into Y (rows x cols, fp32 or bf16)."""
    name = "kq_mx_dequantize"
    rows, cols = Y.shape
    dt, per, dev = _float(name, "Y", Y)
    p, ld = _matrix(name, "Y", Y, rows, cols, Y.dtype, per, False, dev)
    if codes.shape[0] != rows:
        raise ValueError(f"{name}: {codes.shape[0]} rows of codes for {rows} rows")
    _launch(name, lib().kq_mx_dequantize, dev, stream,
            (*_mx(name, "the input", codes, scales, cols, dev), rows, cols, p, dt, ld))


def kq_mx_gemm(Ac, As, Bc, Bs, i: int, Y, ws=None, stream=None) -> None:
    """Y (n x o, fp32 or bf16) = A B^T for microscaled A (n x i) and B (o x i)."""
    name = "kq_mx_gemm"
    n, o = Ac.shape[0], Bc.shape[0]
    dt, per, dev = _float(name, "Y", Y)
    p, ld = _matrix(name, "Y", Y, n, o, Y.dtype, per, False, dev)
    _launch(name, lib().kq_mx_gemm, dev, stream,
            (*_mx(name, "A", Ac, As, i, dev), *_mx(name, "B", Bc, Bs, i, dev), n, o, i, p, dt, ld,
             *_workspace(name, ws, dev)))


def kq_mx_gated(Xc, Xs, Gc, Gs, Uc, Us, i: int, act: str, H, ws=None, stream=None) -> None:
    """H (n x o, fp32 or bf16) = act(X G^T) * (X U^T) for microscaled X (n x i), G and U (o x i)."""
    name = "kq_mx_gated"
    n, o = Xc.shape[0], Gc.shape[0]
    if Uc.shape[0] != o:
        raise ValueError(f"{name}: {o} gate rows and {Uc.shape[0]} up rows")
    dt, per, dev = _float(name, "H", H)
    p, ld = _matrix(name, "H", H, n, o, H.dtype, per, False, dev)
    _launch(name, lib().kq_mx_gated, dev, stream,
            (*_mx(name, "X", Xc, Xs, i, dev), *_mx(name, "gate weights", Gc, Gs, i, dev),
             *_mx(name, "up weights", Uc, Us, i, dev), n, o, i, _act(name, act), p, dt, ld, *_workspace(name, ws, dev)))


def kq_gated_forward(X, Wg, Wu, act: str, H, A=None, B=None, ws=None, stream=None) -> None:
    """H = act(X Wg^T) * (X Wu^T); A and B, where given, take the two products. One type for all."""
    name = "kq_gated_forward"
    (n, i), o, t = X.shape, Wg.shape[0], X.dtype
    dt, per, dev = _float(name, "X", X)
    _launch(name, lib().kq_gated_forward, dev, stream,
            (*_matrix(name, "X", X, n, i, t, per, True, dev), *_matrix(name, "Wg", Wg, o, i, t, per, True, dev),
             *_matrix(name, "Wu", Wu, o, i, t, per, True, dev), dt, n, o, i, _act(name, act),
             *_matrix(name, "H", H, n, o, t, per, False, dev),
             *((None, 0) if A is None else _matrix(name, "A", A, n, o, t, per, False, dev)),
             *((None, 0) if B is None else _matrix(name, "B", B, n, o, t, per, False, dev)), *_workspace(name, ws, dev)))


def kq_gated_backward(dH, A, B, X, Wg, Wu, act: str, dA, dB, dX=None, dWg=None, dWu=None, ws=None, stream=None) -> None:
    """Gradients of kq_gated_forward from dH and the A and B that it kept: dA and dB always, dX, dWg and
    dWu where given (X may be None without weight gradients, Wg and Wu without dX)."""
    name = "kq_gated_backward"
    (n, o), t = dH.shape, dH.dtype
    if dX is not None and (Wg is None or Wu is None):
        raise ValueError(f"{name}: dX needs Wg and Wu")
    if (dWg is not None or dWu is not None) and X is None:
        raise ValueError(f"{name}: weight gradients need X")
    dt, per, dev = _float(name, "dH", dH)
    some = next((m for m in (dX, dWg, dWu, X, Wg, Wu) if m is not None), None)
    i = 1 if some is None else some.shape[1]

    def take(what, m, rows, cols, whole):
        return (None, 0) if m is None else _matrix(name, what, m, rows, cols, t, per, whole, dev)

    # dA and dB are also operands, of the products that follow
    _launch(name, lib().kq_gated_backward, dev, stream,
            (*take("dH", dH, n, o, False), *take("A", A, n, o, False), *take("B", B, n, o, False),
             *take("X", X, n, i, True), *take("Wg", Wg, o, i, True), *take("Wu", Wu, o, i, True), dt, n, o, i, _act(name, act),
             *take("dA", dA, n, o, True), *take("dB", dB, n, o, True), *take("dX", dX, n, i, False),
             *take("dWg", dWg, o, i, False), *take("dWu", dWu, o, i, False), *_workspace(name, ws, dev)))


# ------------------------------------- 8-bit integer products, products grouped by expert, norms
_WORDS: tuple | None = None


def _words() -> tuple:
    """torch.int8, torch.int32 and torch.float32, published whole as _torch's."""
    global _WORDS
    if _WORDS is None:
        import torch
        _WORDS = (torch.int8, torch.int32, torch.float32)
    return _WORDS


def _lead(name: str, what: str, t, whole: bool) -> tuple:
    """The operand that sets a call's type, device and two of its sizes, its attributes read once: (kq_dtype, torch dtype, elements in 16
    bytes, device, rows, cols, pointer, leading dimension), checked as _matrix does."""
    dtype = t.dtype
    f = (_TORCH or _torch())[3].get(dtype)
    if f is None:
        raise TypeError(f"{name}: {what} has type {dtype}")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: {what} is not on a GPU")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: {what} is not row-major")
    dt, per = f
    if rows <= 1:
        ld = -(-cols // per) * per
    if whole and cols % per and rows:
        end = t.storage_offset() + (rows - 1) * ld + -(-cols // per) * per
        if end * t.element_size() > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: the last row of {what} ends inside its 16 bytes, past the storage")
    return dt, dtype, per, dev, rows, cols, t.data_ptr(), ld


def _stack(name: str, what: str, t, e: int, o: int, cols: int, dtype, per: int, whole: bool, dev: int):
    """_matrix for e matrices o x cols one under the other; returns (pointer, leading dimension)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {what} has type {t.dtype}, not {dtype}")
    if t.shape != (e, o, cols):
        raise ValueError(f"{name}: {what} has shape {tuple(t.shape)}, not {(e, o, cols)}")
    if t.get_device() != dev:
        _other_device(name, what, t, dev)
    each, ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: {what} is not row-major")
    if o == 1:
        ld = each       # the stride of a single row is arbitrary
    elif e > 1 and each != o * ld:
        raise ValueError(f"{name}: the matrices of {what} do not lie one under the other")
    rows = e * o
    if rows <= 1:
        ld = -(-cols // per) * per
    if whole and cols % per and rows:
        end = t.storage_offset() + (rows - 1) * ld + -(-cols // per) * per
        if end * t.element_size() > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: the last row of {what} ends inside its 16 bytes, past the storage")
    return t.data_ptr(), ld


def _vector(name: str, what: str, t, shape: tuple, dtype, dev: int):
    """Checks a contiguous tensor of `shape`; returns its pointer (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {what} has type {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: {what} has shape {tuple(t.shape)}, not {shape}")
    if t.get_device() != dev:
        _other_device(name, what, t, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name}: {what} is not contiguous")
    return t.data_ptr()


def _offsets(name: str, t, experts: int, dev: int):
    return _vector(name, "offsets", t, (experts + 1,), (_WORDS or _words())[1], dev)


def _i8(name: str, what: str, codes, scales, rows: int, cols: int, dev: int) -> tuple:
    """Checks 8-bit codes and their scales; returns their three C arguments."""
    i8, _, f32 = _WORDS or _words()
    return *_matrix(name, what + " codes", codes, rows, cols, i8, 16, True, dev), _vector(name, what + " scales", scales, (rows,), f32, dev)


def _i8_weights(name: str, what: str, codes, scales, experts: int, o: int, i: int, dev: int) -> tuple:
    if not experts:
        return _i8(name, what, codes, scales, o, i, dev)
    i8, _, f32 = _WORDS or _words()
    return (*_stack(name, what + " codes", codes, experts, o, i, i8, 16, True, dev),
            _vector(name, what + " scales", scales, (experts, o), f32, dev))


def _experts(name: str, what: str, t) -> int:
    if t.dim() != 3:
        raise ValueError(f"{name}: {what} has shape {tuple(t.shape)}: with offsets it is a stack of matrices")
    return t.shape[0]


def i8_empty(rows: int, cols: int, device):
    """Buffers for a rows x cols matrix of 8-bit integers: codes (int8, rows starting on 16 bytes) and scales (a
    float a row), contents undefined."""
    import torch
    return (torch.empty((rows, -(-cols // 16) * 16), dtype=torch.int8, device=device)[:, :cols],
            torch.empty(rows, dtype=torch.float32, device=device))


def kq_i8_quantize(X, codes, scales, stream=None) -> None:
    """X (rows x cols, fp32 or bf16) into codes and scales of i8_empty(rows, cols)."""
    name = "kq_i8_quantize"
    dt, _, _, dev, rows, cols, p, ld = _lead(name, "X", X, False)
    _launch(name, lib().kq_i8_quantize, dev, stream, (p, dt, rows, cols, ld, *_i8(name, "output", codes, scales, rows, cols, dev)))


def kq_i8_dequantize(codes, scales, Y, stream=None) -> None:
    """The values that codes and scales stand for, into Y (rows x cols, fp32 or bf16)."""
    name = "kq_i8_dequantize"
    dt, _, _, dev, rows, cols, p, ld = _lead(name, "Y", Y, False)
    _launch(name, lib().kq_i8_dequantize, dev, stream, (*_i8(name, "input", codes, scales, rows, cols, dev), rows, cols, p, dt, ld))


def kq_i8_gemm(Ac, As, Bc, Bs, Y, offsets=None, ws=None, stream=None) -> None:
    """Y (n x o, fp32 or bf16) = A B^T for 8-bit A (n x i) and B (o x i, scales o); with offsets (experts + 1 int32)
    the rows of A are sorted by expert and B is experts x o x i, its scales experts x o."""
    name = "kq_i8_gemm"
    dt, _, _, dev, n, o, p, ld = _lead(name, "Y", Y, False)
    i, e = Ac.shape[1], 0 if offsets is None else _experts(name, "B codes", Bc)
    _launch(name, lib().kq_i8_gemm, dev, stream,
            (*_i8(name, "A", Ac, As, n, i, dev), *_i8_weights(name, "B", Bc, Bs, e, o, i, dev), _offsets(name, offsets, e, dev),
             e, n, o, i, p, dt, ld, *_workspace(name, ws, dev)))


def kq_i8_gated(Xc, Xs, Gc, Gs, Uc, Us, act: str, H, offsets=None, ws=None, stream=None) -> None:
    """H (n x o, fp32 or bf16) = act(X G^T) * (X U^T) for 8-bit X (n x i), G and U; offsets as for kq_i8_gemm."""
    name = "kq_i8_gated"
    dt, _, _, dev, n, o, p, ld = _lead(name, "H", H, False)
    i, e = Xc.shape[1], 0 if offsets is None else _experts(name, "gate codes", Gc)
    _launch(name, lib().kq_i8_gated, dev, stream,
            (*_i8(name, "X", Xc, Xs, n, i, dev), *_i8_weights(name, "gate", Gc, Gs, e, o, i, dev),
             *_i8_weights(name, "up", Uc, Us, e, o, i, dev), _offsets(name, offsets, e, dev), e, n, o, i, _act(name, act), p, dt,
             ld, *_workspace(name, ws, dev)))


def kq_grouped_gemm(X, W, offsets, Y, ws=None, stream=None) -> None:
    """Y_r = X_r W_k^T for the rows offsets[k] .. offsets[k + 1] - 1 of X (n x i); W: experts x o x i, offsets: experts + 1
    int32. Rows outside the offsets are left alone."""
    name = "kq_grouped_gemm"
    dt, t, per, dev, n, i, p, ld = _lead(name, "X", X, True)
    e, o, _ = W.shape
    _launch(name, lib().kq_grouped_gemm, dev, stream,
            (p, ld, *_stack(name, "W", W, e, o, i, t, per, True, dev),
             _offsets(name, offsets, e, dev), e, dt, n, o, i, *_matrix(name, "Y", Y, n, o, t, per, False, dev),
             *_workspace(name, ws, dev)))


def kq_grouped_gated(X, Wg, Wu, offsets, act: str, H, A=None, B=None, ws=None, stream=None) -> None:
    """kq_gated_forward for each expert's rows; Wg, Wu and offsets as kq_grouped_gemm's."""
    name = "kq_grouped_gated"
    dt, t, per, dev, n, i, p, ld = _lead(name, "X", X, True)
    e, o, _ = Wg.shape
    _launch(name, lib().kq_grouped_gated, dev, stream,
            (p, ld, *_stack(name, "Wg", Wg, e, o, i, t, per, True, dev),
             *_stack(name, "Wu", Wu, e, o, i, t, per, True, dev), _offsets(name, offsets, e, dev), e, dt, n, o, i,
             _act(name, act), *_matrix(name, "H", H, n, o, t, per, False, dev),
             *((None, 0) if A is None else _matrix(name, "A", A, n, o, t, per, False, dev)),
             *((None, 0) if B is None else _matrix(name, "B", B, n, o, t, per, False, dev)), *_workspace(name, ws, dev)))


def kq_grouped_backward(dY, X, W, offsets, dX=None, dW=None, dY2=None, W2=None, dW2=None, ws=None, stream=None) -> None:
    """Gradients of kq_grouped_gemm: dX and dW where given (W may be None without dX, X without weight gradients).
    With dY2 they are those of two products of the same X: dX the sum of both, dW2 the second's."""
    name = "kq_grouped_backward"
    if dX is not None and (W is None or (dY2 is not None and W2 is None)):
        raise ValueError(f"{name}: dX needs the weights")
    if (dW is not None or dW2 is not None) and X is None:
        raise ValueError(f"{name}: weight gradients need X")
    if dY2 is None and (W2 is not None or dW2 is not None):
        raise ValueError(f"{name}: W2 and dW2 go with dY2")
    dt, t, per, dev, n, o, p, ld = _lead(name, "dY", dY, True)
    e = offsets.shape[0] - 1 if offsets.dim() == 1 else 0
    some = next((m for m in (dX, dW, dW2, X, W, W2) if m is not None), None)
    i = 1 if some is None else some.shape[-1]

    def take(what, m, rows, cols, whole):
        return (None, 0) if m is None else _matrix(name, what, m, rows, cols, t, per, whole, dev)

    def stack(what, m, whole):
        return (None, 0) if m is None else _stack(name, what, m, e, o, i, t, per, whole, dev)

    _launch(name, lib().kq_grouped_backward, dev, stream,
            (p, ld, *stack("W", W, True), *take("dY2", dY2, n, o, True), *stack("W2", W2, True),
             *take("X", X, n, i, True), _offsets(name, offsets, e, dev), e, dt, n, o, i, *take("dX", dX, n, i, False),
             *stack("dW", dW, False), *stack("dW2", dW2, False), *_workspace(name, ws, dev)))


def _norm(name: str, kind: str) -> int:
    if kind not in NORM:
        raise ValueError(f"{name}: kind {kind!r} is none of {sorted(NORM)}")
    return NORM[kind]


def kq_norm_forward(X, gamma, beta, kind: str, eps: float, Y, mean=None, rstd=None, stream=None) -> None:
    """Y = norm(X) * gamma + beta over the rows of X (n x d), kind "layer" or "rms"; gamma and beta (d, X's type) may be None;
    mean and rstd (n floats), where given, take the statistics. Y may be X."""
    name = "kq_norm_forward"
    f32 = (_WORDS or _words())[2]
    dt, t, per, dev, n, d, p, ld = _lead(name, "X", X, False)
    _launch(name, lib().kq_norm_forward, dev, stream,
            (p, ld, _vector(name, "gamma", gamma, (d,), t, dev),
             _vector(name, "beta", beta, (d,), t, dev), dt, n, d, _norm(name, kind), eps,
             *_matrix(name, "Y", Y, n, d, t, per, False, dev), _vector(name, "mean", mean, (n,), f32, dev),
             _vector(name, "rstd", rstd, (n,), f32, dev)))


def kq_norm_backward(dY, X, gamma, mean, rstd, kind: str, dX=None, dgamma=None, dbeta=None, ws=None, stream=None) -> None:
    """Gradients of kq_norm_forward from dY and the mean (None will do for "rms") and rstd that it kept; dX may be dY or X."""
    name = "kq_norm_backward"
    f32 = (_WORDS or _words())[2]
    dt, t, per, dev, n, d, p, ld = _lead(name, "dY", dY, False)
    _launch(name, lib().kq_norm_backward, dev, stream,
            (p, ld, *_matrix(name, "X", X, n, d, t, per, False, dev),
             _vector(name, "gamma", gamma, (d,), t, dev), _vector(name, "mean", mean, (n,), f32, dev),
             _vector(name, "rstd", rstd, (n,), f32, dev), dt, n, d, _norm(name, kind),
             *((None, 0) if dX is None else _matrix(name, "dX", dX, n, d, t, per, False, dev)),
             _vector(name, "dgamma", dgamma, (d,), t, dev), _vector(name, "dbeta", dbeta, (d,), t, dev),
             *_workspace(name, ws, dev)))
