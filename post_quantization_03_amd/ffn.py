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

calibrate_norm_gated does the same from the hidden states, through the norm in front of the block (kq_norm_forward,
kq_norm_backward), to the gradient that the sublayers before it see.

Expert layers: calibrate_experts and quantize_experts do this for every expert over its own tokens, with the products grouped
by expert (kq_grouped_gated, kq_grouped_backward). Tokens come sorted by expert; the router and the sorting are the caller's.

Serving in microscaled 4-bit floating point (MXFeedForward): weights quantised once, tokens and
activations quantised per call, all to the nearest code (the solver's results are integer codes and do not
enter here); kq_mx_gated and kq_mx_gemm do the products. Int8FeedForward is the same in 8-bit integers with a scale for each
token and each output channel, of one block or of an expert layer's (kq_i8_gated, kq_i8_gemm).

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


def _ws(op: str, o: int, i: int, n: int, like: torch.Tensor, experts: int = 0) -> torch.Tensor:
    xdt = K.KQ_BF16 if like.dtype == torch.bfloat16 else K.KQ_F32
    return torch.empty(max(K.kq_workspace_bytes(op, o, i, n, xdt, group=experts), 256), dtype=torch.uint8, device=like.device)


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


def calibrate_norm_gated(X: torch.Tensor, gamma: torch.Tensor | None, beta: torch.Tensor | None, kind: str, eps: float,
                         Wg: torch.Tensor, Wu: torch.Tensor, dH: torch.Tensor, act: str, cfg: LayerCfg) -> dict:
    """calibrate_gated of the block behind a norm, from the hidden states X (n x i): its result, the norm's output N (the input
    of gate and up, which the solver takes as X), and the gradients through the norm: dX at the hidden states (in place
    of the block's own, which is dN), dgamma (None without gamma) and dbeta (None without beta)."""
    n, i = X.shape
    with _on(X, "calibrate_norm_gated"):
        N = _rows(n, i, X)
        mean, rstd = (torch.empty(n, dtype=torch.float32, device=X.device) for _ in range(2))
        K.kq_norm_forward(X, gamma, beta, kind, eps, N, mean, rstd)
        cal = calibrate_gated(N, Wg, Wu, dH, act, cfg)
        dX = _rows(n, i, X)
        dgamma, dbeta = (None if p is None else torch.empty_like(p) for p in (gamma, beta))
        K.kq_norm_backward(cal["dX"], X, gamma, mean, rstd, kind, dX, dgamma, dbeta, _ws("norm_backward", 0, i, n, X))
        return {**cal, "N": N, "dN": cal["dX"], "dX": dX, "dgamma": dgamma, "dbeta": dbeta}


def _spans(offsets: torch.Tensor, n: int) -> list:
    """(first row, end) of each expert's tokens, on the host (which waits for them)."""
    off = offsets.tolist()
    if any(b < a for a, b in zip(off, off[1:])) or off[0] < 0 or off[-1] > n:
        raise ValueError(f"offsets {off} do not ascend within {n} rows")
    return list(zip(off, off[1:]))


def calibrate_experts(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, offsets: torch.Tensor, dH: torch.Tensor, act: str,
                      cfg: LayerCfg) -> dict:
    """calibrate_gated for each expert: the tokens X (n x i) are sorted by expert, expert k's being rows offsets[k] ..
    offsets[k + 1] - 1 (experts + 1 int32 on the device), Wg and Wu are experts x o x i, dH n x o. H, dA, dB and dX are n-row
    matrices, HG_gate and HG_up lists with an entry for each expert, None for one without tokens. Rows outside the offsets are zero."""
    n, i = X.shape
    e, o, _ = Wg.shape
    with _on(X, "calibrate_experts"):
        spans = _spans(offsets, n)
        H, A, B, dA, dB, dX = (_rows(n, d, X).zero_() for d in (o, o, o, o, o, i))
        K.kq_grouped_gated(X, Wg, Wu, offsets, act, H, A, B, _ws("grouped_gated", o, i, n, X, e))
        r = slice(spans[0][0], spans[-1][1])
        K.kq_gated_backward(dH[r], A[r], B[r], None, None, None, act, dA[r], dB[r])
        K.kq_grouped_backward(dA, X, Wg, offsets, dX, dY2=dB, W2=Wu, ws=_ws("grouped_backward", o, i, n, X, e))
        hg = [[_covariance(G[a:b], cfg) if b > a else None for a, b in spans] for G in (dA, dB)]
        return {"H": H, "dA": dA, "dB": dB, "dX": dX, "HG_gate": hg[0], "HG_up": hg[1], "spans": spans}


def quantize_experts(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, offsets: torch.Tensor, dH: torch.Tensor, act: str,
                     s: torch.Tensor, t_gate: torch.Tensor, t_up: torch.Tensor, cfg: LayerCfg, verify: bool = False) -> dict:
    """Calibrates an expert layer and quantises every expert's gate and up projections with the per-layer solver on its own tokens:
    {"gate": [...], "up": [...]}, None for an expert without tokens, and calibrate_experts' result."""
    cal = calibrate_experts(X, Wg, Wu, offsets, dH, act, cfg)
    with _on(X, "quantize_experts"):
        out = {key: [quantize_layer(X[a:b], W[k], cal["HG_" + key][k], s, t, cfg, verify=verify) if b > a else None
                     for k, (a, b) in enumerate(cal["spans"])] for key, W, t in (("gate", Wg, t_gate), ("up", Wu, t_up))}
        return {**out, "calibration": cal}


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


def i8_quantize(X: torch.Tensor) -> tuple:
    """(codes, scales) of X (rows x cols, fp32 or bf16) in 8-bit integers, a scale for each row; of a stack of matrices, each
    one's rows."""
    if X.dim() == 3:
        e, o, i = X.shape
        codes, scales = i8_quantize(X.flatten(0, 1))
        return codes.unflatten(0, (e, o)), scales.view(e, o)
    codes, scales = K.i8_empty(X.shape[0], X.shape[1], X.device)
    K.kq_i8_quantize(X, codes, scales)
    return codes, scales


class Int8FeedForward:
    """The block with 8-bit integer weights, a scale for each output channel: Wg, Wu (o x i) and Wd (m x o), fp32 or bf16, or
    stacks of them for an expert layer (experts x o x i, experts x m x o), are quantised here; a call quantises its tokens and the
    product H, a scale for each token, and multiplies 8 bits by 8 bits."""

    def __init__(self, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, act: str = "silu"):
        if Wg.shape != Wu.shape or Wg.dim() not in (2, 3) or Wd.dim() != Wg.dim() or Wd.shape[-1] != Wg.shape[-2] or \
                Wd.shape[:-2] != Wg.shape[:-2]:
            raise ValueError(f"Int8FeedForward: weights of shapes {tuple(Wg.shape)}, {tuple(Wu.shape)} and {tuple(Wd.shape)}")
        if act not in K.ACT:
            raise ValueError(f"Int8FeedForward: activation {act!r} is none of {sorted(K.ACT)}")
        self.experts = Wg.shape[0] if Wg.dim() == 3 else 0
        self.o, self.i = Wg.shape[-2:]
        self.m = Wd.shape[-2]
        self.act = act
        self.gate, self.up, self.down = i8_quantize(Wg), i8_quantize(Wu), i8_quantize(Wd)

    def __call__(self, X: torch.Tensor, offsets: torch.Tensor | None = None) -> torch.Tensor:
        """Y (n x m) for tokens X (n x i), in X's type; of an expert layer the tokens are sorted by expert and offsets
        (experts + 1 int32 on the device) are their first rows. Rows outside the offsets are undefined."""
        n = X.shape[0]
        if X.shape[1] != self.i:
            raise ValueError(f"Int8FeedForward: tokens of width {X.shape[1]}, not {self.i}")
        if (offsets is None) != (self.experts == 0):
            raise ValueError(f"Int8FeedForward: offsets go with an expert layer, this one has {self.experts} experts")
        H = _rows(n, self.o, X)
        K.kq_i8_gated(*i8_quantize(X), *self.gate, *self.up, self.act, H, offsets, _ws("i8_gated", self.o, self.i, n, X, self.experts))
        Y = _rows(n, self.m, X)
        K.kq_i8_gemm(*i8_quantize(H), *self.down, Y, offsets, _ws("i8_gemm", self.m, self.o, n, X, self.experts))
        return Y
