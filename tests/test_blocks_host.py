"""Microscaled products and the gated block without a GPU: the oracle's definitions against independent
computations, and every refusal of the C entry points and of the Python wrappers."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import blocks as ob
from post_quantization_03_amd import _lib as K
from post_quantization_03_amd import ffn

EINVAL, ESHAPE, EWORKSPACE = 1, 2, 6
P = ctypes.c_void_p(4096)        # a stand-in: refused calls never dereference it
ODD = ctypes.c_void_p(4097)


# ---------------------------------------------------------------------------------------- oracle
def test_oracle_quantiser_on_hand_worked_blocks():
    x = np.zeros((1, 64))
    x[0, :8] = [6.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]     # scale 1; ties to the even code
    x[0, 32:36] = [7.9, 4.0, -6.9, 0.0]                          # scale 1; past 6 saturates
    codes, scales = ob.mx_quantize(x)
    assert scales.tolist() == [[127, 127]]
    v = ob.mx_values(codes, scales, 64)[0]
    assert v[:8].tolist() == [6.0, -0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0] and np.signbit(v[1])
    assert v[32:36].tolist() == [6.0, 4.0, -6.0, 0.0]
    assert codes[0, 0] == (7 | 8 << 4)          # column 0 in the low bits of byte 0, column 1 above it


def test_oracle_quantiser_scales():
    for top, byte in ((0.0, 0), (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125), (3.99, 126), (4.0, 127),
                      (3.4e38, 252), (np.inf, 255), (np.nan, 255)):
        x = np.zeros((1, 32))
        x[0, 5] = top
        codes, scales = ob.mx_quantize(x)
        assert scales[0, 0] == byte, top
        if byte == 255:
            assert not codes.any() and np.all(np.isnan(ob.mx_values(codes, scales, 32)))


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_oracle_gradients_against_differences(kind):
    rng = np.random.default_rng(1)
    X, Wg, Wu = rng.standard_normal((5, 7)), rng.standard_normal((6, 7)), rng.standard_normal((6, 7))
    dH = rng.standard_normal((5, 6))
    _, A, B = ob.gated(X, Wg, Wu, kind)
    _, _, dX, dWg, dWu = ob.gated_grad(dH, A, B, X, Wg, Wu, kind)
    h = 1e-6
    for k, g in enumerate((dX, dWg, dWu)):
        V = rng.standard_normal(g.shape)
        args = [X, Wg, Wu]

        def loss(t):
            a = list(args)
            a[k] = a[k] + t * V
            return (ob.gated(*a, kind)[0] * dH).sum()

        # central differences: h^2 times a third derivative of order 1e2, and 1e-16 / h of rounding
        assert abs((loss(h) - loss(-h)) / (2 * h) - (g * V).sum()) < 1e-7 * (1 + np.abs(g * V).sum())


# ------------------------------------------------------------------------------------- C refusals
def quantize(X=P, dt=0, rows=4, cols=40, ldx=40, c=P, ldc=32, s=P, lds=4):
    return K.lib().kq_mx_quantize(X, dt, rows, cols, ldx, c, ldc, s, lds, None)


def dequantize(c=P, ldc=32, s=P, lds=4, rows=4, cols=40, Y=P, dt=0, ldy=40):
    return K.lib().kq_mx_dequantize(c, ldc, s, lds, rows, cols, Y, dt, ldy, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_mx_conversion_refusals(call):
    for kw, st in ((dict(rows=-1), ESHAPE), (dict(cols=0), ESHAPE), (dict(dt=2), EINVAL), (dict(c=None), EINVAL),
                   (dict(s=None), EINVAL), (dict(ldc=16), ESHAPE), (dict(ldc=40), EINVAL), (dict(lds=1), ESHAPE),
                   (dict(lds=6), EINVAL), (dict(c=ctypes.c_void_p(4104)), EINVAL), (dict(s=ODD), EINVAL),
                   (dict(ldc=1 << 23), ESHAPE)):
        assert call(**kw) == st, kw
    name = "X" if call is quantize else "Y"
    ld = "ldx" if call is quantize else "ldy"
    for kw, st in (({name: None}, EINVAL), ({ld: 36}, ESHAPE), ({ld: 42}, EINVAL), ({name: ctypes.c_void_p(4100)}, EINVAL),
                   ({ld: 44, "dt": 1}, EINVAL)):
        assert call(**kw) == st, kw
    assert call(rows=0) == 0      # nothing to do, nothing dereferenced


def test_mx_product_refusals():
    lib = K.lib()

    def gemm(Ac=P, ldac=32, As=P, ldas=4, Bc=P, ldbc=32, Bs=P, ldbs=4, n=4, o=8, i=40, Y=P, dt=0, ldy=8, ws=None, wb=0):
        return lib.kq_mx_gemm(Ac, ldac, As, ldas, Bc, ldbc, Bs, ldbs, n, o, i, Y, dt, ldy, ws, wb, None)

    def gated(Ac=P, ldac=32, As=P, ldas=4, Bc=P, ldbc=32, Bs=P, ldbs=4, n=4, o=8, i=40, Y=P, dt=0, ldy=8, ws=None, wb=0,
              Uc=P, lduc=32, Us=P, ldus=4, act=0):
        return lib.kq_mx_gated(Ac, ldac, As, ldas, Bc, ldbc, Bs, ldbs, Uc, lduc, Us, ldus, n, o, i, act, Y, dt, ldy, ws, wb,
                               None)

    for call in (gemm, gated):
        for kw, st in ((dict(n=-1), ESHAPE), (dict(o=0), ESHAPE), (dict(i=0), ESHAPE), (dict(dt=7), EINVAL),
                       (dict(Ac=None), EINVAL), (dict(As=None), EINVAL), (dict(Bc=None), EINVAL), (dict(Bs=None), EINVAL),
                       (dict(Y=None), EINVAL), (dict(ldac=16), ESHAPE), (dict(ldbc=24), ESHAPE), (dict(ldbc=40), EINVAL),
                       (dict(ldas=5), EINVAL), (dict(ldy=4), ESHAPE), (dict(ldy=9), EINVAL), (dict(ldy=12, dt=1), EINVAL)):
            assert call(**kw) == st, (call.__name__, kw)
        big = dict(n=3000, o=6000, i=2000, ldac=1008, ldas=64, ldbc=1008, ldbs=64, ldy=6000)
        if call is gated:
            big.update(lduc=1008, ldus=64)
        need = K.kq_workspace_bytes("mx_gemm" if call is gemm else "mx_gated", 6000, 2000, 3000)
        for ws, wb in ((None, 0), (P, 64), (None, need), (ctypes.c_void_p(4100), need), (P, need - 1)):
            assert call(ws=ws, wb=wb, **big) == EWORKSPACE, (call.__name__, ws, wb)
        assert call(n=0) == 0
    for kw, st in ((dict(Uc=None), EINVAL), (dict(Us=None), EINVAL), (dict(lduc=16), ESHAPE), (dict(act=4), EINVAL),
                   (dict(act=-1), EINVAL)):
        assert gated(**kw) == st, kw


def test_gated_refusals():
    lib = K.lib()

    def fwd(X=P, ldx=16, G=P, ldg=16, U=P, ldu=16, dt=1, n=4, o=8, i=16, act=0, H=P, ldh=8, A=P, lda=8, B=P, ldb=8):
        return lib.kq_gated_forward(X, ldx, G, ldg, U, ldu, dt, n, o, i, act, H, ldh, A, lda, B, ldb, None, 0, None)

    for kw, st in ((dict(n=-1), ESHAPE), (dict(o=0), ESHAPE), (dict(i=-3), ESHAPE), (dict(dt=2), EINVAL), (dict(act=9), EINVAL),
                   (dict(X=None), EINVAL), (dict(G=None), EINVAL), (dict(U=None), EINVAL), (dict(H=None), EINVAL),
                   (dict(ldx=8), ESHAPE), (dict(ldg=20), EINVAL), (dict(ldu=8), ESHAPE), (dict(ldh=12), EINVAL),
                   (dict(lda=4), ESHAPE), (dict(B=ODD), EINVAL), (dict(ldx=1 << 22), ESHAPE)):
        assert fwd(**kw) == st, kw
    assert fwd(n=0) == 0

    def bwd(dH=P, lddh=8, A=P, lda=8, B=P, ldb=8, X=P, ldx=16, G=P, ldg=16, U=P, ldu=16, dt=1, n=4, o=8, i=16, act=0, dA=P,
            ldda=8, dB=P, lddb=8, dX=P, lddx=16, dG=P, lddg=16, dU=P, lddu=16):
        return lib.kq_gated_backward(dH, lddh, A, lda, B, ldb, X, ldx, G, ldg, U, ldu, dt, n, o, i, act, dA, ldda, dB, lddb,
                                     dX, lddx, dG, lddg, dU, lddu, None, 0, None)

    for kw, st in ((dict(n=-1), ESHAPE), (dict(dt=3), EINVAL), (dict(act=4), EINVAL), (dict(dH=None), EINVAL),
                   (dict(A=None), EINVAL), (dict(B=None), EINVAL), (dict(X=None), EINVAL), (dict(G=None), EINVAL),
                   (dict(U=None), EINVAL), (dict(dA=None), EINVAL), (dict(dB=None), EINVAL), (dict(lddh=4), ESHAPE),
                   (dict(ldda=12), EINVAL), (dict(lddx=8), ESHAPE), (dict(lddg=20), EINVAL), (dict(dU=ODD), EINVAL)):
        assert bwd(**kw) == st, kw
    assert bwd(n=0, dG=None, dU=None) == 0


def test_sizes_past_a_launch_are_refused():
    """Results and grids that no launch can hold come back as ESHAPE, before any workspace or GPU is asked for."""
    lib, far = K.lib(), 1 << 31

    def gemm(n, o, U=False):
        if U:
            return lib.kq_mx_gated(P, 32, P, 4, P, 32, P, 4, P, 32, P, 4, n, o, 40, 0, P, 0, o, None, 0, None)
        return lib.kq_mx_gemm(P, 32, P, 4, P, 32, P, 4, n, o, 40, P, 0, o, None, 0, None)

    for u in (False, True):
        for n, o in ((1, 1 << 28), (far, far), (far, 64), (far + 1, 64)):
            assert gemm(n, o, u) == ESHAPE, (n, o, u)
    assert K.kq_workspace_bytes("mx_gemm", far, 40, far) == 0
    for n, o in ((far + 1, 64), (far, 1 << 20)):
        assert lib.kq_gated_forward(P, 16, P, 16, P, 16, 1, n, o, 16, 0, P, o, None, 0, None, 0, None, 0, None) == ESHAPE
        assert lib.kq_gated_backward(P, o, P, o, P, o, P, 1 << 20, P, 1 << 20, P, 1 << 20, 1, n, o, 1 << 20, 0, P, o, P, o,
                                     P, 1 << 20, None, 0, None, 0, None, 0, None) == ESHAPE


def test_calibration_needs_tokens():
    from post_quantization_03_amd.layer import LayerCfg
    x, w = torch.zeros(0, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="no tokens"):
        ffn.calibrate_gated(x, w, w, torch.zeros(0, 8), "silu", LayerCfg(bits=4, group=64, form="diag"))


def test_workspace_sizes():
    for op in ("mx_gemm", "mx_gated"):
        assert K.kq_workspace_bytes(op, 4096, 4096, 32) == 0
        assert K.kq_workspace_bytes(op, 4096, 11008, 8192) >= (4096 + 8192) * 344


# -------------------------------------------------------------------------------- wrapper refusals
def test_wrappers_refuse_host_tensors_and_bad_types():
    x = torch.zeros(4, 64)
    c, s = K.mx_empty(4, 64, "cpu")
    assert c.shape == (4, 32) and s.shape == (4, 4)
    with pytest.raises(ValueError, match="GPU"):
        K.kq_mx_quantize(x, c, s)
    with pytest.raises(TypeError, match="type"):
        K.kq_mx_quantize(x.double(), c, s)
    with pytest.raises(ValueError, match="GPU"):
        K.kq_gated_forward(x, x, x, "silu", x)
    with pytest.raises(TypeError, match="type"):
        K.kq_gated_forward(x.half(), x, x, "silu", x)
    with pytest.raises(ValueError, match="needs Wg and Wu"):
        K.kq_gated_backward(x, x, x, None, None, None, "silu", x, x, dX=x)
    with pytest.raises(ValueError, match="need X"):
        K.kq_gated_backward(x, x, x, None, x, x, "silu", x, x, dWg=x)
    with pytest.raises(ValueError, match="shapes"):
        ffn.MXFeedForward(torch.zeros(8, 4), torch.zeros(8, 5), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="activation"):
        ffn.MXFeedForward(torch.zeros(8, 4), torch.zeros(8, 4), torch.zeros(4, 8), "tanh")


def test_first_calls_of_two_threads_at_any_point():
    """A second thread's first call at every line of the first thread's gets the same answer: a fresh copy of
    the module, whose lazy set-up is interrupted line by line."""
    import importlib.util
    import sys
    import threading

    spec = importlib.util.spec_from_file_location("fresh_lib", K.__file__)
    x = torch.zeros(4, 64)
    answers = []

    def call(mod):
        try:
            mod._float("first", "X", x)
        except Exception as e:      # noqa: BLE001  the answer: this tensor is refused for its device alone
            answers.append(f"{type(e).__name__}: {e}")

    def first(mod, stop):
        seen = 0

        def trace(frame, event, arg):
            nonlocal seen
            if frame.f_code.co_filename != K.__file__:
                return None
            if event == "line":
                if seen == stop:
                    other = threading.Thread(target=call, args=(mod,))
                    other.start()
                    other.join(20)
                    assert not other.is_alive()
                seen += 1
            return trace

        sys.settrace(trace)
        try:
            call(mod)
        finally:
            sys.settrace(None)
        return seen

    lines, stop = 1, 0
    while stop < lines:             # as many times as the first call has lines
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        t = threading.Thread(target=lambda: counts.append(first(mod, stop)))
        counts: list = []
        t.start()
        t.join(30)
        lines, stop = counts[0], stop + 1
    assert lines > 5
    assert set(answers) == {"ValueError: first: X is not on a GPU"}, set(answers)


def test_workspaces_whose_bytes_are_not_in_one_piece_are_refused():
    """A view counts values that it does not own: an expanded one (stride 0) claims bytes past its storage, a
    strided one bytes between its values."""
    whole = torch.empty(4096, dtype=torch.uint8)
    assert K._workspace("w", whole, -1) == (whole.data_ptr(), 4096)
    assert K._workspace("w", whole[256:].view(15, 256), -1) == (whole.data_ptr() + 256, 3840)
    assert K._workspace("w", whole[:1024].view(torch.float32), -1) == (whole.data_ptr(), 1024)
    for bad in (whole[:1].expand(4096), whole[::2], whole.view(64, 64).T, whole.view(64, 64)[:, :32]):
        with pytest.raises(ValueError, match="contiguous"):
            K._workspace("w", bad, -1)


def test_calibration_runs_on_its_tensors_device(monkeypatch):
    """Tensors on a device other than the current one: every call of the calibration, those of the older entry points
    among them (which launch on the current device), runs with the tensors' device current."""
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
    for name in ("kq_gated_forward", "kq_gated_backward", "kq_hessian_accum", "kq_hg_extract"):
        monkeypatch.setattr(K, name, record(name))
    monkeypatch.setattr(ffn, "quantize_layer", record("quantize_layer"))
    x, w, dh = (torch.zeros(*s).as_subclass(OnOne) for s in ((4, 64), (8, 64), (4, 8)))
    cfg = LayerCfg(bits=4, group=64, form="diag")
    ffn.calibrate_gated(x, w, w, dh, "silu", cfg)
    names = ["kq_gated_forward", "kq_gated_backward"] + 2 * ["kq_hessian_accum", "kq_hg_extract"]
    assert calls == [(n, 1) for n in names]
    calls.clear()
    ffn.quantize_gated(x, w, w, dh, "silu", None, None, None, cfg)
    assert calls == [(n, 1) for n in names + 2 * ["quantize_layer"]]
    assert current == [0]
    with pytest.raises(ValueError, match="not on a GPU"):
        ffn.calibrate_gated(torch.zeros(4, 64), w, w, dh, "silu", cfg)
