"""Norms on the GPU against the float64 oracle.

Bounds, with E = 2^-24. A sum over a row of d values has at most k = 72 + d / 1024 roundings one after another (a thread's own values,
then wavefront and work-group), so it is off by k E times the sum of magnitudes; 1 / d and the product with it add two.
Forward: the mean is off by em = (k + 3) E mean|x|; the mean of (x - m')^2 about m' = m + em is the variance plus em^2 and relatively
off by (k + 6) E; r is relatively off by half of the change of variance + eps, and by 4 E for its own roundings.
Backward takes mean and rstd as given: h is off by 3 E |h|, g by E |g|, the two means by their sums' bounds.
dgamma and dbeta: at most n + 8 roundings one after another.
"""
import numpy as np
import pytest

from oracle import experts as oe
from post_quantization_03_amd import _lib as K
from tests.gpu_util import host, say, torch_dev
from tests.test_gpu_blocks import HALF, check, get, mat, put
from tests.test_gpu_i8 import Workspace

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
EPS = 1e-5


def steps(d):
    return 72 + d / 1024


def forward_tols(x, gamma, beta, kind, dt):
    """(values, bounds) of Y, mean and rstd."""
    y, m, r = oe.norm(x, gamma, beta, kind, np.float64(np.float32(EPS)))
    k = steps(x.shape[1])
    em = (k + 3) * E * np.abs(x).mean(axis=1) if kind == "layer" else np.zeros(len(x))
    t = np.abs(x - m[:, None])
    var = (t * t).mean(axis=1)
    rr = 0.5 * (em ** 2 / (var + EPS) + (k + 7) * E) * 1.1 + 5 * E
    et = em[:, None] + E * (t + em[:, None])
    h = t * r[:, None]
    ey = np.abs(gamma) * (et * r[:, None] * (1 + rr[:, None]) + h * (rr[:, None] + 3 * E)) + 2 * E * (np.abs(y) + np.abs(beta))
    return (y, m, r), (ey + HALF[dt] * (np.abs(y) + ey) + 2.0 ** -126, em + E * np.abs(m) + 2.0 ** -126, rr * r)


def backward_tols(dy, x, gamma, m, r, kind, dt):
    """(values, bounds) of dX, dgamma and dbeta."""
    want = oe.norm_grad(dy, x, gamma, m, r, kind)
    n, d = x.shape
    k = steps(d)
    r = r[:, None]
    h, g = np.abs(x - m[:, None]) * r, np.abs(dy * gamma)
    c1, c0 = np.abs((dy * gamma * (x - m[:, None]) * r).mean(axis=1, keepdims=True)), np.abs((dy * gamma).mean(axis=1, keepdims=True))
    e1, e0 = (k + 8) * E * (g * h).mean(axis=1, keepdims=True), (k + 4) * E * g.mean(axis=1, keepdims=True)
    if kind == "rms":
        c0, e0 = 0 * c0, 0 * e0
    ex = r * (E * g + e0 + h * (e1 + 4 * E * c1) + 5 * E * (g + c0 + h * c1))
    eg, eb = (n + 12) * E * (np.abs(dy) * h).sum(axis=0), (n + 8) * E * np.abs(dy).sum(axis=0)
    return want, [e + HALF[dt] * (np.abs(w) + e) + 2.0 ** -126 for w, e in zip(want, (ex, eg, eb))]


def vector(a, dt):
    """Host values rounded to dt on the device; and as float64."""
    t, v = put(np.asarray(a)[None], dt)
    return t[0].contiguous(), v[0]


def case(n, d, dt, seed=0):
    rng = np.random.default_rng(1000 * n + d + seed)
    X = put(rng.standard_normal((n, d)) * np.exp(0.7 * rng.standard_normal((1, d))) + 0.5, dt, pad=1)
    dY = put(rng.standard_normal((n, d)) * np.exp(rng.standard_normal((1, d))), dt, pad=2)
    return X, dY, vector(1 + 0.3 * rng.standard_normal(d), dt), vector(rng.standard_normal(d), dt)


def padding_kept(t):
    return (host(t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)).float())[:, t.shape[1]:] == -77.0).all()


# every number of pieces a thread and threads a row, whole and ragged, and rows past the registers
WIDTHS = [(5, 1), (9, 3), (7, 8), (33, 31), (6, 256), (300, 257), (5, 512), (70, 513), (3, 1000), (333, 1000), (4, 1024), (9, 1025),
          (2, 2048), (1, 2050), (3, 4096), (1500, 4096), (2, 4097), (5, 8192), (2, 8200), (3, 11008), (4, 13824), (2, 16384), (3, 16390),
          (2, 32768), (70, 32780), (3, 50001)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", WIDTHS)
def test_forward_and_backward(n, d, dt, kind):
    torch, dev = torch_dev()
    say(f"norm n={n} d={d} {dt} {kind}")
    (X, x), (dY, dy), (gamma, gv), (beta, bv) = case(n, d, dt)
    Y = mat(n, d, dt, pad=1, fill=-77.0)
    mean, rstd = torch.full((n + 1,), -77.0, device=dev), torch.full((n + 1,), -77.0, device=dev)
    K.kq_norm_forward(X, gamma, beta, kind, EPS, Y, mean[:n], rstd[:n])
    want, tols = forward_tols(x, gv, bv, kind, dt)
    got = (get(Y), get(mean[:n]), get(rstd[:n]))
    for name, g, w, t in zip(("Y", "mean", "rstd"), got, want, tols):
        check(g, w, t, name)
    assert padding_kept(Y) and float(mean[n]) == -77.0 and float(rstd[n]) == -77.0
    w = Workspace("norm_backward", 0, d, n, dt)
    dX = mat(n, d, dt, pad=1, fill=-77.0)
    dg, db = (torch.full((d + 8,), -77.0, dtype=X.dtype, device=dev) for _ in range(2))
    K.kq_norm_backward(dY, X, gamma, mean[:n] if kind == "layer" else None, rstd[:n], kind, dX, dg[:d], db[:d], w.ws)
    want, tols = backward_tols(dy, x, gv, got[1], got[2], kind, dt)
    for name, t, v, tol in zip(("dX", "dgamma", "dbeta"), (dX, dg[:d], db[:d]), want, tols):
        check(get(t), v, tol, name)
    assert padding_kept(dX) and w.kept() and bool((dg[d:] == -77.0).all()) and bool((db[d:] == -77.0).all())
    # any subset has the same bits, on a workspace of other contents
    w.buf[:w.need] = 0
    dX2, dg2, db2 = mat(n, d, dt), torch.empty_like(dg[:d]), torch.empty_like(db[:d])
    K.kq_norm_backward(dY, X, gamma, mean[:n], rstd[:n], kind, dX2)
    K.kq_norm_backward(dY, X, gamma, mean[:n], rstd[:n], kind, dgamma=dg2, ws=w.ws)
    K.kq_norm_backward(dY, X, gamma, mean[:n], rstd[:n], kind, dbeta=db2, ws=w.ws)
    assert torch.equal(dX2, dX) and torch.equal(dg2, dg[:d]) and torch.equal(db2, db[:d])
    # in place: Y over X, dX over dY and over X
    Z = mat(n, d, dt)
    Z.copy_(X)
    K.kq_norm_forward(Z, gamma, beta, kind, EPS, Z)
    assert torch.equal(Z, Y)
    for over in (0, 1):
        a, b = mat(n, d, dt), mat(n, d, dt)
        a.copy_(dY), b.copy_(X)
        K.kq_norm_backward(a, b, gamma, mean[:n], rstd[:n], kind, (a, b)[over], dg2, db2, w.ws)
        assert torch.equal((a, b)[over], dX) and torch.equal(dg2, dg[:d]) and torch.equal(db2, db[:d])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(2053, 100), (2053, 500), (2053, 1000), (1100, 2000), (700, 2900), (700, 6000), (300, 11008), (300, 13824),
                                 (300, 16001), (300, 20000)])
def test_more_rows_than_work_groups_take_at_once(n, d, dt, kind):
    """Rows past the work-groups of the backward pass, not a multiple of them: the weights' sums go on from row to row, in every number of
    threads and pieces, with the next row loaded ahead and without room for it."""
    test_forward_and_backward(n, d, dt, kind)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1 << 20, (1 << 20) - 11])
def test_the_widest_rows(d, dt):
    """Rows of up to 2^20 values. Padding would take a row past the limit of leading dimensions, so it has none."""
    torch, dev = torch_dev()
    say(f"norm d={d} {dt}")
    rng = np.random.default_rng(d)
    X, x = put(rng.standard_normal((3, d)) * 2 + 0.5, dt)
    dY, dy = put(rng.standard_normal((3, d)), dt)
    (gamma, gv), (beta, bv) = vector(1 + 0.3 * rng.standard_normal(d), dt), vector(rng.standard_normal(d), dt)
    for kind in ("layer", "rms"):
        Y, mean, rstd = mat(3, d, dt), torch.empty(3, device=dev), torch.empty(3, device=dev)
        K.kq_norm_forward(X, gamma, beta, kind, EPS, Y, mean, rstd)
        want, tols = forward_tols(x, gv, bv, kind, dt)
        for name, t, w, tol in zip(("Y", "mean", "rstd"), (Y, mean, rstd), want, tols):
            check(get(t), w, tol, name)
        dX, dg, db = mat(3, d, dt), torch.empty_like(gamma), torch.empty_like(beta)
        K.kq_norm_backward(dY, X, gamma, mean, rstd, kind, dX, dg, db, Workspace("norm_backward", 0, d, 3, dt).ws)
        want, tols = backward_tols(dy, x, gv, get(mean), get(rstd), kind, dt)
        for name, t, w, tol in zip(("dX", "dgamma", "dbeta"), (dX, dg, db), want, tols):
            check(get(t), w, tol, name)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [100, 3000, 33000])
def test_without_weights(d, dt):
    (X, x), (dY, dy), _, _ = case(6, d, dt, 1)
    ones, zeros = np.ones(d), np.zeros(d)
    torch, dev = torch_dev()
    for kind in ("layer", "rms"):
        Y, mean, rstd = mat(6, d, dt), torch.empty(6, device=dev), torch.empty(6, device=dev)
        K.kq_norm_forward(X, None, None, kind, EPS, Y, mean, rstd)
        want, tols = forward_tols(x, ones, zeros, kind, dt)
        check(get(Y), want[0], tols[0], "Y")
        dX = mat(6, d, dt)
        K.kq_norm_backward(dY, X, None, mean, rstd, kind, dX)
        want, tols = backward_tols(dy, x, ones, get(mean), get(rstd), kind, dt)
        check(get(dX), want[0], tols[0], "dX")


@pytest.mark.parametrize("d", [64, 1000, 20000])
def test_large_mean_constant_and_special_rows(d):
    """A mean of 10^4 deviations keeps the variance's digits; a constant row gives beta; infinities and NaN stay in their rows."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(d)
    x = rng.standard_normal((7, d))
    x[0] += 1e4
    x[1] = 3.25
    x[2] = 0.0
    x[3, d // 2], x[4, 0] = np.inf, np.nan
    x[5] *= 1e15
    X, x = put(x, "f32")
    (gamma, gv), (beta, bv) = vector(1 + rng.standard_normal(d), "f32"), vector(rng.standard_normal(d), "f32")
    Y, mean, rstd = mat(7, d, "f32"), torch.empty(7, device=dev), torch.empty(7, device=dev)
    K.kq_norm_forward(X, gamma, beta, "layer", EPS, Y, mean, rstd)
    fine = [0, 1, 2, 5, 6]
    want, tols = forward_tols(x[fine], gv, bv, "layer", "f32")
    for name, g, w, t in zip(("Y", "mean", "rstd"), (get(Y), get(mean), get(rstd)), want, tols):
        check(g[fine], w, t, name)
    assert np.isnan(get(Y)[3:5]).all()
    assert np.array_equal(get(Y)[1:3], np.tile(bv, (2, 1)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 250, 1000, 4096, 8200, 20000, 40000])
def test_rows_whose_sums_pass_the_largest_number(d, dt):
    """Finite rows whose sum, or whose differences from the mean, pass 3.4e38: the mean keeps the bound of any other; r is zero where the
    squares pass, so that Y is beta and dX zero. A constant row's mean is that constant: differences t = c - m of a first mean m, off by at
    most (k + 3) E c, are exact, and their mean is t off by (k + 2) E t, less than E c / 2: m and it add up to c. Its r is a zero row's, or
    zero: t is zero, or at least an ulp of c, whose square passes."""
    torch, dev = torch_dev()
    say(f"norm of large values d={d} {dt}")
    rng = np.random.default_rng(d)
    x = rng.standard_normal((9, d))
    x[0] = 1e37
    x[1] = 10.0 ** rng.uniform(36, 38.4, d)
    x[2] = np.where(np.arange(d) % 2, 3e38, -3e38)
    x[3] = -3e38
    x[3, d // 3] = 3e38
    x[4] = 0.0
    x[5] = np.where(np.arange(d) < d // 2, 3e38, -3e38)
    x[6] = -3.3e38
    x[7] = 1e37
    x[7, d - 1] = np.inf
    X, x = put(x, dt)
    (gamma, gv), (beta, bv) = vector(1 + 0.3 * rng.standard_normal(d), dt), vector(rng.standard_normal(d), dt)
    dY, dy = put(rng.standard_normal((9, d)), dt)
    finite = [k for k in range(9) if k != 7]
    for kind in ("layer", "rms"):
        Y, mean, rstd = mat(9, d, dt), torch.empty(9, device=dev), torch.empty(9, device=dev)
        K.kq_norm_forward(X, gamma, beta, kind, EPS, Y, mean, rstd)
        want, tols = forward_tols(x[finite], gv, bv, kind, dt)
        check(get(mean)[finite], want[1], tols[1], "mean")
        check(get(Y)[[8]], want[0][-1:], tols[0][-1:], "Y of an ordinary row")
        zero, one = [1, 2, 3, 5], [0, 6]
        assert (get(rstd)[zero] == 0).all()
        if kind == "layer":
            assert np.array_equal(get(mean)[one], x[one, 0]) and np.isin(get(rstd)[one], [0, get(rstd)[4]]).all() and get(rstd)[4] > 300
            assert np.isnan(get(Y)[7]).all()
        else:
            assert (get(rstd)[one] == 0).all() and np.isnan(get(Y)[7, d - 1])
        assert np.array_equal(get(Y)[zero + one + [4]], np.tile(bv, (7, 1)))
        # gradients of the finite rows, whose values these are
        Xf, dYf, mf, rf = X[finite].contiguous(), dY[finite].contiguous(), mean[finite].contiguous(), rstd[finite].contiguous()
        a, b = mat(8, d, dt), mat(8, d, dt)
        a.copy_(Xf), b.copy_(dYf)
        dX, dg, db = mat(8, d, dt), torch.empty_like(gamma), torch.empty_like(gamma)
        K.kq_norm_backward(b, a, gamma, mf, rf, kind, dX, dg, db, Workspace("norm_backward", 0, d, 8, dt).ws)
        want, tols = backward_tols(dy[finite], x[finite], gv, get(mf), get(rf), kind, dt)
        for name, t, w, tol in zip(("dX", "dgamma", "dbeta"), (dX, dg, db), want, tols):
            check(get(t), w, tol, name)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(kind):
    """The fp32 kernel's gradients against central differences of the float64 forward pass along random directions: h^2 times a third
    derivative (of order 100 here), and the kernel's own bound with the statistics' rounding, 200 E relative, on top."""
    torch, dev = torch_dev()
    n, d, h = 30, 70, 1e-5
    (X, x), (dY, dy), (gamma, gv), (beta, bv) = case(n, d, "f32", 2)
    Y, mean, rstd = mat(n, d, "f32"), torch.empty(n, device=dev), torch.empty(n, device=dev)
    K.kq_norm_forward(X, gamma, beta, kind, EPS, Y, mean, rstd)
    dX, dg, db = mat(n, d, "f32"), torch.empty(d, device=dev), torch.empty(d, device=dev)
    K.kq_norm_backward(dY, X, gamma, mean, rstd, kind, dX, dg, db, Workspace("norm_backward", 0, d, n, "f32").ws)
    _, tols = backward_tols(dy, x, gv, get(mean), get(rstd), kind, "f32")
    rng = np.random.default_rng(5)
    size = (np.abs(dy) * (1 + np.abs(gv)) * (3 + np.abs(x))).sum()
    for k, (grad, tol) in enumerate(zip((get(dX), get(dg), get(db)), tols)):
        V = rng.standard_normal(grad.shape)

        def loss(t):
            p = [x, gv, bv]
            p[k] = p[k] + t * V
            return (oe.norm(*p, kind, EPS)[0] * dy).sum()

        diff = (loss(h) - loss(-h)) / (2 * h)
        slack = (tol * np.abs(V)).sum() + 200 * E * size * np.abs(V).max() + 100 * h * h * size * np.abs(V).max() ** 3 + 1e-14 * size / h
        assert abs(diff - (grad * V).sum()) <= slack, (k, diff, (grad * V).sum(), slack)


def test_no_rows():
    torch, dev = torch_dev()
    x, s = mat(0, 40, "bf16"), torch.empty(0, device=dev)
    dg, db = (torch.full((40,), -77.0, dtype=x.dtype, device=dev) for _ in range(2))
    K.kq_norm_forward(x, None, None, "layer", EPS, x, s, s)
    K.kq_norm_backward(x, x, None, s, s, "layer", x, dg, db)
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows are those of a call on these alone; sums over rows that are zero but the last."""
    torch, dev = torch_dev()
    n, d, k = 262501, 8200, 5
    say("norm offsets")
    X, dY, dX = mat(n, d, "bf16", fill=0.0), mat(n, d, "bf16", fill=0.0), mat(n, d, "bf16", fill=-77.0)
    torch.manual_seed(1)
    X[-k:].copy_(torch.randn(k, d, device=dev)), dY[-k:].copy_(torch.randn(k, d, device=dev))
    (gamma, gv), (beta, bv) = vector(np.ones(d), "bf16"), vector(np.linspace(-1, 1, d), "bf16")
    mean, rstd = torch.empty(n, device=dev), torch.empty(n, device=dev)
    K.kq_norm_forward(X, gamma, beta, "layer", EPS, dX, mean, rstd)
    want, tols = forward_tols(get(X[-k:]), gv, bv, "layer", "bf16")
    check(get(dX[-k:]), want[0], tols[0], "Y")
    assert bool((dX[:-k] == beta).all())
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    K.kq_norm_backward(dY, X, gamma, mean, rstd, "layer", dX, dg, db, Workspace("norm_backward", 0, d, n).ws)
    want, tols = backward_tols(get(dY[-k:]), get(X[-k:]), gv, get(mean[-k:]), get(rstd[-k:]), "layer", "bf16")
    for name, t, w, tol in zip(("dX", "dgamma", "dbeta"), (dX[-k:], dg, db), want, tols):
        check(get(t), w, tol, name)
    assert bool((dX[:-k] == 0).all())
