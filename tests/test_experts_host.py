"""8-bit integer products, products grouped by expert and norms without a GPU: the oracle's definitions against
independent computations, and every refusal of the C entry points and of the Python wrappers."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import experts as oe
from post_quantization_03_amd import _lib as K
from post_quantization_03_amd import ffn

EINVAL, ESHAPE, EWORKSPACE = 1, 2, 6
P = ctypes.c_void_p(4096)        # a stand-in: refused calls never dereference it
ODD = ctypes.c_void_p(4097)
FOUR = ctypes.c_void_p(4100)


# ---------------------------------------------------------------------------------------- oracle
def test_oracle_quantiser_against_fractions():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 40)) * np.exp(3 * rng.standard_normal((6, 40)))).astype(np.float32)
    x[1] = np.round(x[1] * 4) / 4
    x[2, 0], x[2, 1:] = 127.0, np.arange(39) - 19.5          # ties, multiplier 1
    x[3] = 0.0
    x[4] *= np.float32(2.0 ** -100)
    x[5, 3] = np.inf
    codes, scales = oe.i8_quantize(x)
    for r in range(5):
        a = np.abs(x[r]).max()
        if a == 0:
            assert scales[r] == 0 and not codes[r].any()
            continue
        # both divisions rounded to fp32 by hand: half an ulp from the fraction
        m = np.float32(127) / a
        for got, want in ((scales[r], Fraction(float(a)) / 127), (m, Fraction(127) / Fraction(float(a)))):
            assert abs(Fraction(float(got)) - want) <= Fraction(float(np.spacing(got))) / 2
        for c, v in zip(codes[r], x[r]):
            q = Fraction(float(v)) * Fraction(float(m))
            assert abs(q - int(c)) <= Fraction(1, 2) and (abs(q - int(c)) != Fraction(1, 2) or c % 2 == 0)
        assert np.abs(codes[r]).max() == 127
    assert np.isnan(scales[5]) and not codes[5].any()
    assert oe.i8_quantize(np.full((1, 3), 2.0 ** -119 * (1 - 2.0 ** -24)))[1][0] == 0
    assert oe.i8_quantize(np.full((1, 3), 2.0 ** -119))[1][0] > 2.0 ** -126


def test_oracle_spans_of_any_contents():
    assert oe.spans([0, 3, 3, 7], 7) == [(0, 0, 3), (1, 3, 3), (2, 3, 7)]
    assert oe.spans([2, 1, 9, -4, 5], 7) == [(0, 2, 2), (1, 2, 7), (2, 7, 7), (3, 7, 7)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_oracle_norm_gradients_against_differences(kind):
    rng = np.random.default_rng(2)
    X, gamma, beta, dY = rng.standard_normal((5, 7)) + 0.5, rng.standard_normal(7), rng.standard_normal(7), rng.standard_normal((5, 7))
    _, m, r = oe.norm(X, gamma, beta, kind, 1e-3)
    grads = oe.norm_grad(dY, X, gamma, m, r, kind)
    h = 1e-6
    for k, g in enumerate(grads):
        V = rng.standard_normal(g.shape)

        def loss(t):
            p = [X, gamma, beta]
            p[k] = p[k] + t * V
            return (oe.norm(*p, kind, 1e-3)[0] * dY).sum()

        # central differences: h^2 times a third derivative of order 1e2, and 1e-16 / h of rounding
        assert abs((loss(h) - loss(-h)) / (2 * h) - (g * V).sum()) < 1e-7 * (1 + np.abs(g * V).sum())


def test_oracle_grouped_gradients_against_differences():
    rng = np.random.default_rng(3)
    X, W, off = rng.standard_normal((9, 4)), rng.standard_normal((3, 5, 4)), [1, 4, 4, 8]
    dY = rng.standard_normal((9, 5))
    dX, dW = oe.grouped_grad(dY, X, W, off)
    for p, g, k in ((X, dX, 0), (W, dW, 1)):
        V = rng.standard_normal(p.shape)
        f = lambda t: (oe.grouped(*(q + t * V * (j == k) if j == k else q for j, q in enumerate((X, W))), off)[0] * dY).sum()   # noqa: E731
        assert abs((f(0.5) - f(-0.5)) - (g * V).sum()) < 1e-12 * (1 + np.abs(g * V).sum())      # linear in each


# ------------------------------------------------------------------------------------- C refusals
def quantize(X=P, dt=0, rows=4, cols=40, ldx=40, c=P, ldc=48, s=P):
    return K.lib().kq_i8_quantize(X, dt, rows, cols, ldx, c, ldc, s, None)


def dequantize(c=P, ldc=48, s=P, rows=4, cols=40, Y=P, dt=0, ldy=40):
    return K.lib().kq_i8_dequantize(c, ldc, s, rows, cols, Y, dt, ldy, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_i8_conversion_refusals(call):
    for kw, st in ((dict(rows=-1), ESHAPE), (dict(cols=0), ESHAPE), (dict(dt=2), EINVAL), (dict(c=None), EINVAL),
                   (dict(s=None), EINVAL), (dict(ldc=32), ESHAPE), (dict(ldc=40), EINVAL), (dict(c=FOUR), EINVAL),
                   (dict(s=ODD), EINVAL), (dict(ldc=1 << 23), ESHAPE)):
        assert call(**kw) == st, kw
    name, ld = ("X", "ldx") if call is quantize else ("Y", "ldy")
    for kw, st in (({name: None}, EINVAL), ({ld: 36}, ESHAPE), ({ld: 42}, EINVAL), ({name: FOUR}, EINVAL),
                   ({ld: 44, "dt": 1}, EINVAL)):
        assert call(**kw) == st, kw
    assert call(rows=0) == 0      # nothing to do, nothing dereferenced


def i8_gemm(A=P, lda=48, sA=P, B=P, ldb=48, sB=P, off=None, e=0, n=4, o=8, i=40, Y=P, dt=0, ldy=8, ws=None, wb=0):
    return K.lib().kq_i8_gemm(A, lda, sA, B, ldb, sB, off, e, n, o, i, Y, dt, ldy, ws, wb, None)


def i8_gated(A=P, lda=48, sA=P, B=P, ldb=48, sB=P, U=P, ldu=48, sU=P, off=None, e=0, n=4, o=8, i=40, act=0, Y=P, dt=0, ldy=8,
             ws=None, wb=0):
    return K.lib().kq_i8_gated(A, lda, sA, B, ldb, sB, U, ldu, sU, off, e, n, o, i, act, Y, dt, ldy, ws, wb, None)


@pytest.mark.parametrize("call", [i8_gemm, i8_gated])
def test_i8_product_refusals(call):
    wide = dict(lda=1 << 17, ldb=1 << 17, **({"ldu": 1 << 17} if call is i8_gated else {}))
    for kw, st in ((dict(n=-1), ESHAPE), (dict(o=0), ESHAPE), (dict(i=0), ESHAPE), (dict(dt=7), EINVAL), (dict(A=None), EINVAL),
                   (dict(sA=None), EINVAL), (dict(B=None), EINVAL), (dict(sB=None), EINVAL), (dict(Y=None), EINVAL),
                   (dict(lda=32), ESHAPE), (dict(ldb=32), ESHAPE), (dict(ldb=56), EINVAL), (dict(A=FOUR), EINVAL), (dict(sB=ODD), EINVAL),
                   (dict(ldy=4), ESHAPE), (dict(ldy=9), EINVAL), (dict(ldy=12, dt=1), EINVAL), (dict(i=1 << 17, **wide), ESHAPE),
                   (dict(e=3), EINVAL), (dict(off=P, e=0), ESHAPE), (dict(off=P, e=4097), ESHAPE), (dict(off=ODD, e=2), EINVAL),
                   (dict(off=P, e=2, n=1 << 31), ESHAPE), (dict(off=P, e=1024, o=1 << 22, ldy=1 << 22), ESHAPE),
                   (dict(n=(1 << 31) + 1), ESHAPE)):
        assert call(**kw) == st, kw
    assert call(n=0) == 0 and call(n=0, off=P, e=2) == 0
    big = dict(n=300, o=200, i=9000, lda=9008, ldb=9008, ldy=200, **({"ldu": 9008} if call is i8_gated else {}))
    need = K.kq_workspace_bytes("i8_gemm" if call is i8_gemm else "i8_gated", 200, 9000, 300)
    assert need > 0
    for ws, wb in ((None, 0), (P, 64), (None, need), (FOUR, need), (P, need - 1)):
        assert call(ws=ws, wb=wb, **big) == EWORKSPACE, (ws, wb)
    if call is i8_gated:
        for kw in (dict(U=None), dict(sU=None), dict(act=4), dict(act=-1), dict(U=FOUR)):
            assert call(**kw) == EINVAL, kw
    large = dict(n=16384, o=4096, i=11008, off=P, e=8, lda=11008, ldb=11008, ldy=4096, **({"ldu": 11008} if call is i8_gated else {}))
    need = K.kq_workspace_bytes("i8_gemm" if call is i8_gemm else "i8_gated", 4096, 11008, 16384, group=8)
    for ws, wb in ((None, 0), (P, need - 1), (FOUR, need)):
        assert call(ws=ws, wb=wb, **large) == EWORKSPACE, (ws, wb)


def gg(X=P, ldx=16, W=P, ldw=16, off=P, e=3, dt=1, n=4, o=8, i=16, Y=P, ldy=8, ws=None, wb=0):
    return K.lib().kq_grouped_gemm(X, ldx, W, ldw, off, e, dt, n, o, i, Y, ldy, ws, wb, None)


def ggated(X=P, ldx=16, W=P, ldw=16, U=P, ldu=16, off=P, e=3, dt=1, n=4, o=8, i=16, act=0, Y=P, ldy=8, A=P, lda=8, B=P, ldb=8, ws=None,
           wb=0):
    return K.lib().kq_grouped_gated(X, ldx, W, ldw, U, ldu, off, e, dt, n, o, i, act, Y, ldy, A, lda, B, ldb, ws, wb, None)


@pytest.mark.parametrize("call", [gg, ggated])
def test_grouped_refusals(call):
    for kw, st in ((dict(n=-1), ESHAPE), (dict(o=0), ESHAPE), (dict(i=-3), ESHAPE), (dict(dt=2), EINVAL), (dict(X=None), EINVAL),
                   (dict(W=None), EINVAL), (dict(Y=None), EINVAL), (dict(off=None), EINVAL), (dict(off=ODD), EINVAL),
                   (dict(e=0), ESHAPE), (dict(e=-1), ESHAPE), (dict(e=4097), ESHAPE), (dict(ldx=8), ESHAPE), (dict(ldw=20), EINVAL),
                   (dict(ldy=12), EINVAL), (dict(ldx=1 << 22), ESHAPE), (dict(n=1 << 31), ESHAPE), (dict(e=4096, o=1 << 20), ESHAPE),
                   (dict(n=(1 << 31) - 511), ESHAPE), (dict(n=(1 << 31) - 512, o=1 << 16, ldy=1 << 16), ESHAPE)):
        assert call(**kw) == st, kw
    if call is ggated:
        for kw, st in ((dict(U=None), EINVAL), (dict(act=9), EINVAL), (dict(lda=4), ESHAPE), (dict(B=ODD), EINVAL)):
            assert call(**kw) == st, kw
    large = dict(n=16384, o=4096, i=11008, e=8, ldx=11008, ldw=11008, ldy=4096,
                 **({"ldu": 11008, "A": None, "B": None} if call is ggated else {}))
    need = K.kq_workspace_bytes("grouped_gemm" if call is gg else "grouped_gated", 4096, 11008, 16384, group=8)
    for ws, wb in ((None, 0), (P, need - 1), (FOUR, need)):
        assert call(ws=ws, wb=wb, **large) == EWORKSPACE, (ws, wb)
    assert call(n=0) == 0


def test_grouped_backward_refusals():
    def bwd(dY=P, lddy=8, W=P, ldw=16, dY2=P, lddy2=8, W2=P, ldw2=16, X=P, ldx=16, off=P, e=3, dt=1, n=4, o=8, i=16, dX=P, lddx=16,
            dW=P, lddw=16, dW2=P, lddw2=16):
        return K.lib().kq_grouped_backward(dY, lddy, W, ldw, dY2, lddy2, W2, ldw2, X, ldx, off, e, dt, n, o, i, dX, lddx, dW, lddw,
                                           dW2, lddw2, None, 0, None)

    for kw, st in ((dict(n=-1), ESHAPE), (dict(o=0), ESHAPE), (dict(dt=3), EINVAL), (dict(off=None), EINVAL), (dict(e=0), ESHAPE),
                   (dict(dY=None), EINVAL), (dict(W=None), EINVAL), (dict(dY2=None), EINVAL), (dict(W2=None), EINVAL),
                   (dict(X=None), EINVAL), (dict(lddy=4), ESHAPE), (dict(lddx=8), ESHAPE), (dict(lddw=20), EINVAL),
                   (dict(dW2=ODD), EINVAL), (dict(ldx=8), ESHAPE), (dict(n=1 << 31), ESHAPE),
                   (dict(e=4096, o=1 << 18, i=1 << 18, lddw=1 << 18, lddw2=1 << 18, ldx=1 << 18, lddx=1 << 18, ldw=1 << 18,
                         ldw2=1 << 18, lddy=1 << 18, lddy2=1 << 18, dX=None), ESHAPE)):
        assert bwd(**kw) == st, kw
    assert bwd(n=0, dW=None, dW2=None) == 0
    assert bwd(dX=None, dW=None, dW2=None, dY2=None, W2=None) == 0


@pytest.mark.parametrize("two", [False, True])
def test_grouped_backward_checks_all_before_it_launches(two):
    """A call whose weight gradients are refused (workspace, grid) enqueues nothing, dX neither: without a GPU a launch would come back as
    a HIP error instead of the refusal."""
    def bwd(n, e, o, i, ws, wb, dt=1):
        lo, li = -(-o // 8) * 8, -(-i // 8) * 8
        more = (P, lo, P, li) if two else (None, 0, None, 0)
        return K.lib().kq_grouped_backward(P, lo, P, li, *more, P, li, P, e, dt, n, o, i, P, li, P, li, P if two else None, li, ws, wb, None)

    # what the sizes are for: more split sums of dW than of dX; split sums of dW alone; of both, fp32
    for n, e, o, i, dt in ((6034, 2, 805, 1587, 1), (5001, 2, 371, 971, 1), (9000, 1, 40, 72, 1), (9000, 1, 40, 72, 0)):
        need = K.kq_workspace_bytes("grouped_backward", o, i, n, dt, group=e)
        assert need > 0
        for ws, wb in ((None, 0), (None, need), (FOUR, need), (P, need // 2 - 1)):
            assert bwd(n, e, o, i, ws, wb, dt) == EWORKSPACE, (n, e, o, i, dt, ws, wb)
    # 4 rows: few tiles of dX, 4096 experts' weight gradients past a launch
    assert bwd(4, 4096, 1 << 18, 1 << 18, P, 1 << 40) == ESHAPE


def test_norm_refusals():
    def fwd(X=P, ldx=16, g=P, b=P, dt=1, n=4, d=16, kind=0, eps=1e-5, Y=P, ldy=16, m=P, r=P):
        return K.lib().kq_norm_forward(X, ldx, g, b, dt, n, d, kind, eps, Y, ldy, m, r, None)

    for kw, st in ((dict(n=-1), ESHAPE), (dict(d=0), ESHAPE), (dict(dt=2), EINVAL), (dict(kind=2), EINVAL), (dict(kind=-1), EINVAL),
                   (dict(eps=0.0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=1e9), EINVAL),
                   (dict(X=None), EINVAL), (dict(Y=None), EINVAL), (dict(g=FOUR), EINVAL), (dict(b=ODD), EINVAL), (dict(m=ODD), EINVAL),
                   (dict(r=ODD), EINVAL), (dict(ldx=8), ESHAPE), (dict(ldy=20), EINVAL), (dict(X=FOUR), EINVAL),
                   (dict(ldx=1 << 21), ESHAPE), (dict(n=(1 << 31) + 1), ESHAPE)):
        assert fwd(**kw) == st, kw
    assert fwd(n=0) == 0

    def bwd(dY=P, lddy=16, X=P, ldx=16, g=P, m=P, r=P, dt=1, n=4, d=16, kind=0, dX=P, lddx=16, dg=P, db=P, ws=P, wb=1 << 20):
        return K.lib().kq_norm_backward(dY, lddy, X, ldx, g, m, r, dt, n, d, kind, dX, lddx, dg, db, ws, wb, None)

    need = K.kq_workspace_bytes("norm_backward", 0, 16, 4)
    for kw, st in ((dict(n=-1), ESHAPE), (dict(d=0), ESHAPE), (dict(dt=2), EINVAL), (dict(kind=5), EINVAL), (dict(dY=None), EINVAL),
                   (dict(X=None), EINVAL), (dict(r=None), EINVAL), (dict(m=None), EINVAL), (dict(m=ODD), EINVAL), (dict(g=FOUR), EINVAL),
                   (dict(dg=ODD), EINVAL), (dict(lddx=8), ESHAPE), (dict(lddy=20), EINVAL), (dict(ws=None), EWORKSPACE),
                   (dict(ws=FOUR), EWORKSPACE), (dict(wb=need - 1), EWORKSPACE)):
        assert bwd(**kw) == st, kw
    assert bwd(n=0, dg=None, db=None) == 0
    assert bwd(dX=None, dg=None, db=None, ws=None, wb=0) == 0


def test_workspace_sizes():
    for op in ("i8_gemm", "i8_gated"):
        assert K.kq_workspace_bytes(op, 4096, 4096, 32) == 0
        assert 0 < K.kq_workspace_bytes(op, 200, 9000, 300, group=4) <= 32 << 20
    for op in ("i8_gemm", "i8_gated", "grouped_gemm", "grouped_gated", "grouped_backward"):
        assert K.kq_workspace_bytes(op, 200, 100, 300, group=4) == 0        # small grouped products are not cut
        assert 0 < K.kq_workspace_bytes(op, 4096, 11008, 16384, group=8) <= 128 << 20
        assert K.kq_workspace_bytes(op, 4096, 11008, 16384, group=0) == 0 or op.startswith("i8")
        assert K.kq_workspace_bytes(op, 4096, 11008, 16384, group=5000) == 0
        assert K.kq_workspace_bytes(op, 4096, 11008, 1 << 40, group=8) == 0
    for d in (1, 100, 1000, 4096, 11008, 50000):
        for n in (1, 3, 333, 8192):
            for dt in (K.KQ_F32, K.KQ_BF16):
                assert 8 * d <= K.kq_workspace_bytes("norm_backward", 0, d, n, dt) <= 8 * d * 4096
    assert K.kq_workspace_bytes("norm_backward", 0, 64, 0) == 0


# -------------------------------------------------------------------------------- wrapper refusals
def test_wrappers_refuse_host_tensors_shapes_and_types():
    x, w = torch.zeros(4, 64), torch.zeros(3, 8, 64)
    off = torch.zeros(4, dtype=torch.int32)
    c, s = K.i8_empty(4, 60, "cpu")
    assert c.shape == (4, 60) and c.stride() == (64, 1) and s.shape == (4,)
    for call in (lambda: K.kq_i8_quantize(x, c, s), lambda: K.kq_i8_dequantize(c, s, x), lambda: K.kq_i8_gemm(c, s, c, s, x),
                 lambda: K.kq_grouped_gemm(x, w, off, x), lambda: K.kq_grouped_gated(x, w, w, off, "silu", x),
                 lambda: K.kq_grouped_backward(x, x, w, off, dX=x), lambda: K.kq_norm_forward(x, None, None, "layer", 1e-5, x),
                 lambda: K.kq_norm_backward(x, x, None, s, s, "rms", x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError, match="type"):
        K.kq_i8_quantize(x.double(), c, s)
    with pytest.raises(TypeError, match="type"):
        K.kq_grouped_gemm(x.half(), w, off, x)
    with pytest.raises(ValueError, match="stack of matrices"):
        K._experts("e", "B codes", c)
    assert K._experts("e", "B codes", c.unflatten(0, (2, 2))) == 2
    for bad, match in ((x.T, "GPU"), (x.double(), "type"), (x.to(torch.int32), "type")):
        with pytest.raises((TypeError, ValueError), match=match):
            K._lead("l", "X", bad, True)
    with pytest.raises(ValueError, match="needs the weights"):
        K.kq_grouped_backward(x, x, None, off, dX=x)
    with pytest.raises(ValueError, match="needs the weights"):
        K.kq_grouped_backward(x, x, w, off, dX=x, dY2=x)
    with pytest.raises(ValueError, match="need X"):
        K.kq_grouped_backward(x, None, w, off, dW=w)
    with pytest.raises(ValueError, match="go with dY2"):
        K.kq_grouped_backward(x, x, w, off, dW=w, dW2=w)


def test_stacks_and_vectors():
    t = torch.zeros(3, 8, 64)
    f32 = torch.float32
    assert K._stack("s", "W", t, 3, 8, 64, f32, 4, True, -1) == (t.data_ptr(), 64)
    pad = torch.zeros(3 * 8, 72)[:, :61].unflatten(0, (3, 8))
    assert K._stack("s", "W", pad, 3, 8, 61, f32, 4, True, -1)[1] == 72
    one = torch.zeros(3, 1, 128)[:, :, :64]
    assert K._stack("s", "W", one, 3, 1, 64, f32, 4, True, -1)[1] == 128
    for bad, match in ((torch.zeros(3, 16, 64)[:, :8], "under"), (torch.zeros(1, 8, 64).expand(3, 8, 64), "under"),
                       (torch.zeros(3, 64, 8).transpose(1, 2), "row-major"), (torch.zeros(3, 8, 60), "shape"),
                       (torch.zeros(3 * 8 * 64).as_strided((3, 8, 64), (8 * 64, 64, 1))[:, :, :64].to(torch.bfloat16), "type")):
        with pytest.raises((ValueError, TypeError), match=match):
            K._stack("s", "W", bad, 3, 8, 64, f32, 4, True, -1)
    short = torch.zeros(24 * 64 - 3).as_strided((3, 8, 61), (8 * 64, 64, 1))
    with pytest.raises(ValueError, match="past the storage"):
        K._stack("s", "W", short, 3, 8, 61, f32, 4, True, -1)
    with pytest.raises(ValueError, match="past the storage"):
        K._i8("q", "A", torch.zeros(4 * 48 - 5, dtype=torch.int8).as_strided((4, 40), (48, 1)), torch.zeros(4), 4, 40, -1)
    with pytest.raises(TypeError, match="int32"):
        K._offsets("o", torch.zeros(4, dtype=torch.int64), 3, -1)
    with pytest.raises(ValueError, match="shape"):
        K._offsets("o", torch.zeros(3, dtype=torch.int32), 3, -1)
    with pytest.raises(ValueError, match="contiguous"):
        K._offsets("o", torch.zeros(8, dtype=torch.int32)[::2], 3, -1)
    with pytest.raises(ValueError, match="activation"):
        K._act("a", "tanh")
    with pytest.raises(ValueError, match="kind"):
        K._norm("n", "batch")


# ----------------------------------------------------------------------------------------- drivers
def test_driver_refusals():
    from post_quantization_03_amd.layer import LayerCfg
    z = torch.zeros
    for shapes in (((8, 4), (8, 5), (4, 8)), ((8, 4), (8, 4), (4, 7)), ((3, 8, 4), (3, 8, 4), (4, 8)), ((3, 8, 4), (3, 8, 4), (2, 4, 8)),
                   ((8,), (8,), (8,))):
        with pytest.raises(ValueError, match="shapes"):
            ffn.Int8FeedForward(*(z(*s) for s in shapes))
    with pytest.raises(ValueError, match="activation"):
        ffn.Int8FeedForward(z(8, 4), z(8, 4), z(4, 8), "tanh")
    for bad in ([0, 5, 4], [-1, 2, 4], [0, 2, 11]):
        with pytest.raises(ValueError, match="ascend"):
            ffn._spans(torch.tensor(bad, dtype=torch.int32), 10)
    assert ffn._spans(torch.tensor([2, 2, 10], dtype=torch.int32), 10) == [(2, 2), (2, 10)]
    cfg = LayerCfg(bits=4, group=64, form="diag")
    with pytest.raises(ValueError, match="GPU"):
        ffn.calibrate_experts(z(4, 64), z(2, 8, 64), z(2, 8, 64), torch.tensor([0, 2, 4], dtype=torch.int32), z(4, 8), "silu", cfg)
    with pytest.raises(ValueError, match="GPU"):
        ffn.calibrate_norm_gated(z(4, 64), z(64), None, "layer", 1e-5, z(8, 64), z(8, 64), z(4, 8), "silu", cfg)


@pytest.mark.parametrize("have", [(False, False), (False, True), (True, False), (True, True)])
def test_norm_driver_without_weights(monkeypatch, have):
    """calibrate_norm_gated of a norm without gamma or beta: the norm's calls get None for them and for their gradients."""
    import contextlib

    from post_quantization_03_amd.layer import LayerCfg
    seen = {}
    monkeypatch.setattr(ffn, "_on", lambda t, name: contextlib.nullcontext())
    monkeypatch.setattr(ffn, "calibrate_gated", lambda N, *a: {"H": None, "dX": N})
    monkeypatch.setattr(K, "kq_norm_forward", lambda X, gamma, beta, *a: seen.update(gamma=gamma, beta=beta))
    monkeypatch.setattr(K, "kq_norm_backward", lambda dY, X, gamma, mean, rstd, kind, dX, dgamma, dbeta, ws: seen.update(
        gamma2=gamma, dgamma=dgamma, dbeta=dbeta))
    x, w, dh = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4, 8)
    gamma, beta = (torch.ones(64) if h else None for h in have)
    out = ffn.calibrate_norm_gated(x, gamma, beta, "rms", 1e-5, w, w, dh, "silu", LayerCfg(bits=4, group=64, form="diag"))
    assert seen["gamma"] is gamma and seen["gamma2"] is gamma and seen["beta"] is beta
    for key, p in (("dgamma", gamma), ("dbeta", beta)):
        assert out[key] is seen[key] and (out[key] is None) == (p is None)
        assert p is None or out[key].shape == p.shape


def test_drivers_run_on_their_tensors_device(monkeypatch):
    """Tensors on a device other than the current one: every call of the drivers runs with the tensors' device current."""
    import contextlib

    from post_quantization_03_amd.layer import LayerCfg

    class OnOne(torch.Tensor):
        def get_device(self):
            return 1

    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        current.append(d if isinstance(d, int) else 1)
        yield
        current.pop()

    def record(name):
        def call(*args, **kw):
            calls.append((name, current[-1]))
            return {}
        return call

    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("kq_gated_forward", "kq_gated_backward", "kq_hessian_accum", "kq_hg_extract", "kq_norm_forward", "kq_norm_backward",
                 "kq_grouped_gated", "kq_grouped_backward"):
        monkeypatch.setattr(K, name, record(name))
    monkeypatch.setattr(ffn, "quantize_layer", record("quantize_layer"))
    rows = ffn._rows
    monkeypatch.setattr(ffn, "_rows", lambda n, d, like: rows(n, d, like).as_subclass(OnOne))
    x, w, dh, gamma, ws = (torch.zeros(*s).as_subclass(OnOne) for s in ((4, 64), (8, 64), (4, 8), (64,), (3, 8, 64)))
    cfg = LayerCfg(bits=4, group=64, form="diag")
    ffn.calibrate_norm_gated(x, gamma, None, "rms", 1e-5, w, w, dh, "silu", cfg)
    assert calls == [(n, 1) for n in ["kq_norm_forward", "kq_gated_forward", "kq_gated_backward"] +
                     2 * ["kq_hessian_accum", "kq_hg_extract"] + ["kq_norm_backward"]]
    calls.clear()
    out = ffn.quantize_experts(x, ws, ws, torch.tensor([0, 1, 1, 4], dtype=torch.int32), dh, "silu", None, None, None, cfg)
    assert calls == [(n, 1) for n in ["kq_grouped_gated", "kq_gated_backward", "kq_grouped_backward"] +
                     4 * ["kq_hessian_accum", "kq_hg_extract"] + 4 * ["quantize_layer"]]
    assert out["gate"][1] is None and out["up"][1] is None and current == [0]
