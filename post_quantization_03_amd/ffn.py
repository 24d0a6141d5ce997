"""Gated feed-forward block of a transformer layer on the GPU through the C ABI (include/kq.h):
y = Wd h, h = act(Wg x) * (Wu x).

Calibration (KronQ review page, Method: activation and gradient covariances of a layer come from one
calibration pass): the block's forward pass gives the down projection's input H, and the backward pass
from the gradient at H gives the output gradients of gate and up, whose covariances are their H_G:
  kq_gated_forward   H, and the pre-activations A, B
  kq_gated_backward  dA, dB (the gradient rows of gate and up), dX for the layers before
  kq_hessian_accum   dA^T dA / n, dB^T dB / n
  kq_hg_extract      their storage forms
quantize_gated then runs the per-layer solver on gate and up with these statistics.

Serving in microscaled 4-bit floating point (MXFeedForward): weights quantised once, tokens and
activations quantised per call, all to the nearest code (the solver's results are integer codes and do not
enter here); kq_mx_gated and kq_mx_gemm do the products.

Matrices are passed on as they are, so the rows of X, dH and the weights start on 16 bytes: a contiguous matrix
of another width is refused (KQError) and has to be copied into padded rows first.
Torch only allocates device memory and supplies the stream.
"""
from __future__ import annotations

import torch

from . import _lib as K
from .layer import LayerCfg, hg_factor_shape, quantize_layer


def _rows(n: int, d: int, like: torch.Tensor) -> torch.Tensor:
    """n x d of like's type, rows starting on 16 bytes."""
    per = 16 // like.element_size()
    return torch.empty((n, -(-d // per) * per), dtype=like.dtype, device=like.device)[:, :d]


def _ws(op: str, o: int, i: int, n: int, like: torch.Tensor) -> torch.Tensor:
    xdt = K.KQ_BF16 if like.dtype == torch.bfloat16 else K.KQ_F32
    return torch.empty(max(K.kq_workspace_bytes(op, o, i, n, xdt), 256), dtype=torch.uint8, device=like.device)


def _on(t: torch.Tensor, name: str):
    """t's device as the current one: the solver's calls launch on the current device and its stream."""
    return torch.cuda.device(K._float(name, "X", t)[2])


def _covariance(G: torch.Tensor, cfg: LayerCfg) -> torch.Tensor:
    """H_G = G^T G / n of gradient rows G (n x o) in cfg's storage form."""
    n, o = G.shape
    xdt = K.KQ_BF16 if G.dtype == torch.bfloat16 else K.KQ_F32
    H = torch.empty((o, o), dtype=torch.float64, device=G.device)
    ws = torch.empty(max(K.kq_workspace_bytes("hessian", 0, o, n, xdt), 256), dtype=torch.uint8, device=G.device)
    K.kq_hessian_accum(G, H, 1.0 / n, 0.0, ws)
    out = torch.empty(hg_factor_shape(o, cfg), dtype=torch.float32, device=G.device)
    K.kq_hg_extract(H, cfg.form, cfg.blk, out)
    return out


def calibrate_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, dH: torch.Tensor, act: str,
                    cfg: LayerCfg) -> dict:
    """Statistics of one calibration batch X (n x i) with the gradient dH (n x o) at the block's
    product: H (input of the down projection), dA and dB (gradient rows of gate and up), dX, and the
    gradient covariances HG_gate and HG_up in cfg's storage form."""
    n, i = X.shape
    if n == 0:
        raise ValueError("calibrate_gated: no tokens, no statistics")
    o = Wg.shape[0]
    with _on(X, "calibrate_gated"):
        H, A, B = _rows(n, o, X), _rows(n, o, X), _rows(n, o, X)
        K.kq_gated_forward(X, Wg, Wu, act, H, A, B, _ws("gated_forward", o, i, n, X))
        dA, dB, dX = _rows(n, o, X), _rows(n, o, X), _rows(n, i, X)
        K.kq_gated_backward(dH, A, B, X, Wg, Wu, act, dA, dB, dX, ws=_ws("gated_backward", o, i, n, X))
        return {"H": H, "dA": dA, "dB": dB, "dX": dX, "HG_gate": _covariance(dA, cfg), "HG_up": _covariance(dB, cfg)}


def quantize_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, dH: torch.Tensor, act: str, s: torch.Tensor,
                   t_gate: torch.Tensor, t_up: torch.Tensor, cfg: LayerCfg, verify: bool = False) -> dict:
    """Calibrates the block and quantises its gate and up projections with the per-layer solver:
    {"gate": ..., "up": ...} as quantize_layer returns them, and calibrate_gated's result."""
    cal = calibrate_gated(X, Wg, Wu, dH, act, cfg)
    with _on(X, "quantize_gated"):
        return {"gate": quantize_layer(X, Wg, cal["HG_gate"], s, t_gate, cfg, verify=verify),
                "up": quantize_layer(X, Wu, cal["HG_up"], s, t_up, cfg, verify=verify), "calibration": cal}


def mx_quantize(X: torch.Tensor) -> tuple:
    """(codes, scales) of X (rows x cols, fp32 or bf16) in the microscaled format."""
    codes, scales = K.mx_empty(X.shape[0], X.shape[1], X.device)
    K.kq_mx_quantize(X, codes, scales)
    return codes, scales


class MXFeedForward:
    """The block with microscaled 4-bit weights: Wg, Wu (o x i) and Wd (m x o), fp32 or bf16, are
    quantised here; a call quantises its tokens and the product H, and multiplies 4 bits by 4 bits."""

    def __init__(self, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, act: str = "silu"):
        if Wg.shape != Wu.shape or Wd.shape[1] != Wg.shape[0]:
            raise ValueError(f"MXFeedForward: weights of shapes {tuple(Wg.shape)}, {tuple(Wu.shape)} and {tuple(Wd.shape)}")
        if act not in K.ACT:
            raise ValueError(f"MXFeedForward: activation {act!r} is none of {sorted(K.ACT)}")
        self.o, self.i = Wg.shape
        self.m = Wd.shape[0]
        self.act = act
        self.gate, self.up, self.down = mx_quantize(Wg), mx_quantize(Wu), mx_quantize(Wd)

    def __call__(self, X: torch.Tensor) -> torch.Tensor:
        """Y (n x m) for tokens X (n x i), in X's type."""
        n = X.shape[0]
        if X.shape[1] != self.i:
            raise ValueError(f"MXFeedForward: tokens of width {X.shape[1]}, not {self.i}")
        H = _rows(n, self.o, X)
        K.kq_mx_gated(*mx_quantize(X), *self.gate, *self.up, self.i, self.act, H, _ws("mx_gated", self.o, self.i, n, X))
        Y = _rows(n, self.m, X)
        K.kq_mx_gemm(*mx_quantize(H), *self.down, self.o, Y, _ws("mx_gemm", self.m, self.o, n, X))
        return Y
