"""Products grouped by expert on the GPU. Operands are small whole numbers, so that every partial sum of a product is a whole
number below 2^24, which fp32 holds in any order: the result is the definition's rounded once and the tolerance
is zero. Ordinary values and the other activations: bounds of the gated block's tests."""
import numpy as np
import pytest

from oracle import blocks as ob
from oracle import experts as oe
from post_quantization_03_amd import _lib as K
from tests.gpu_util import host, say, torch_dev
from tests.test_gpu_blocks import E23, HALF, KINDS, check, gated_tol, get, mat, put
from tests.test_gpu_blocks_plans import generator, out, same, whole_numbers
from tests.test_gpu_i8 import Workspace, dealt, offsets

pytestmark = pytest.mark.gpu


def stack(e, o, i, dt, top, g):
    """e matrices of whole numbers one under the other, NaN in the padding; and as float64."""
    t, v = whole_numbers(e * o, i, dt, top, g)
    return t.as_strided((e, o, i), (o * t.stride(0), t.stride(0), 1)), v.view(e, o, i)


def space(op, o, i, n, dt, e):
    """The workspace that a call asks for, full of NaN."""
    return Workspace(op, o, i, n, dt, e).ws


def out_stack(e, o, i, dt):
    t = out(e * o, i, dt)
    return t, t.as_strided((e, o, i), (o * t.stride(0), t.stride(0), 1))


# few rows an expert, one expert with more, more experts than lanes; then tile shapes of 256, 128 and 64 rows (L, M, S) with K whole,
# split for all tiles, or for those behind the last full turn (mixed), of the plain or the gated product
FORWARD = [("few", "bf16", 1, 1, 40, 33), ("few", "bf16", 3, 4, 41, 100), ("few", "bf16", 64, 16, 70, 1000), ("few", "bf16", 90, 70, 40, 65),
           ("few", "bf16", 200, 150, 30, 100), ("few", "f32", 1, 1, 40, 33), ("few", "f32", 64, 16, 70, 1000), ("few", "f32", 300, 70, 40, 65),
           ("SD", "bf16", 100, 3, 33, 400), ("SD", "bf16", 500, 7, 130, 257), ("S", "bf16", 4100, 130, 70, 48), ("MD", "bf16", 3000, 5, 1100, 900),
           ("SD", "bf16", 25, 2, 1, 876), ("S mixed", "bf16", 110, 9, 7674, 1792), ("S mixed gated", "bf16", 51, 5, 7228, 1593),
           ("M", "bf16", 776, 12, 2812, 9), ("M", "bf16", 655, 10, 3306, 3), ("MD", "bf16", 4277, 2, 464, 3085),
           ("MD gated", "bf16", 1479, 2, 752, 3154), ("M mixed", "bf16", 5500, 3, 3126, 2463), ("M mixed gated", "bf16", 4873, 2, 1664, 1853),
           ("L", "bf16", 4011, 3, 2059, 548), ("L", "bf16", 2313, 3, 1609, 594), ("L split", "bf16", 5840, 2, 1483, 10880),
           ("L split gated", "bf16", 1539, 2, 2539, 11720), ("L mixed", "bf16", 8505, 2, 4325, 5866), ("L mixed gated", "bf16", 4273, 3, 4150, 4753),
           ("S", "f32", 517, 5, 130, 257), ("S", "f32", 1000, 3, 200, 72), ("S split", "f32", 92, 2, 2, 437), ("S mixed", "f32", 3637, 2, 1191, 755),
           ("S mixed gated", "f32", 3517, 3, 597, 633)]
# tiles with four slabs in LDS (MD, SD), whole and split, and lengths of K that end anywhere in the four; (may): cut for some row counts
FORWARD += [("L (may)", "bf16", 7077, 2, 2182, 1015), ("M (may)", "bf16", 5797, 2, 1282, 2045), ("M split", "bf16", 3493, 2, 635, 10706),
            ("MD (may)", "bf16", 2049, 4, 208, 8814), ("MD", "bf16", 5004, 2, 628, 228), ("MD split", "bf16", 1556, 2, 762, 4803),
            ("S (may)", "bf16", 194, 3, 289, 3165), ("S split", "bf16", 24, 2, 1, 1540), ("SD (may)", "bf16", 645, 10, 150, 6321),
            ("SD split", "bf16", 17, 2, 1, 3734), ("MD gated", "bf16", 1278, 2, 1259, 200), ("MD split gated", "bf16", 922, 2, 177, 6388),
            ("MD (may) gated", "bf16", 3331, 13, 134, 8278), ("SD (may) gated", "bf16", 257, 2, 62, 7247), ("M (may) gated", "bf16", 2655, 3, 1503, 2008),
            ("M split gated", "bf16", 3561, 2, 574, 5400), ("S (may) gated", "bf16", 129, 2, 146, 2513), ("S (may)", "f32", 129, 2, 211, 524)]
# few rows an expert, rows that begin at multiples of 128 bytes (their padding counted): wavefronts without a slab, with one, with several
FORWARD += [("few, spread", "bf16", n, 7, 100, i) for n in (1, 40) for i in (56, 120, 497, 504, 568, 1009, 1080, 4085)]
FORWARD += [("few, spread", "f32", n, 7, 100, i) for n in (1, 40) for i in (28, 57, 249, 252, 284, 1017, 2044)]
FORWARD += [("SD", "bf16", 300, 3, 200, i) for i in (129, 150, 192, 193, 256, 257, 319, 320, 321, 384, 449, 513)]


@pytest.mark.parametrize("plan,dt,n,e,o,i", FORWARD)
def test_grouped_forward_exact(plan, dt, n, e, o, i):
    """Whole numbers of at most 4: products of at most 16, 11720 of which sum to less than 2^18."""
    import torch
    say(f"grouped forward {plan} {dt} n={n} e={e} o={o} i={i}")
    g = generator(n + e + o + i)
    X, x = whole_numbers(n, i, dt, 4, g)
    (W, w), (U, u) = stack(e, o, i, dt, 4, g), stack(e, o, i, dt, 4, g)
    for off in (dealt(n, e, g), dealt(n, e, g, n // 4, n - n // 5), offsets([0] * e + [n])):
        a, b = torch.zeros((n, o), dtype=torch.float64, device=X.device), torch.zeros((n, o), dtype=torch.float64, device=X.device)
        inside = torch.zeros(n, dtype=torch.bool, device=X.device)
        for k, p, q in oe.spans(host(off), n):
            a[p:q], b[p:q], inside[p:q] = torch.mm(x[p:q], w[k].T), torch.mm(x[p:q], u[k].T), True
        Y, H, A, B, H2 = (out(n, o, dt) for _ in range(5))
        w1, w2 = Workspace("grouped_gemm", o, i, n, dt, e), Workspace("grouped_gated", o, i, n, dt, e)
        K.kq_grouped_gemm(X, W, off, Y, w1.ws)
        K.kq_grouped_gated(X, W, U, off, "relu", H, A, B, w2.ws)
        K.kq_grouped_gated(X, W, U, off, "relu", H2, B=None, ws=w2.ws)
        assert w1.kept() and w2.kept()
        assert torch.equal(H, H2)
        for t, want, name in ((Y, a, "Y"), (A, a, "A"), (B, b, "B"), (H, a.float().clamp(min=0) * b.float(), "H")):
            assert bool((t[~inside] == -77.0).all()), name + ": rows outside the offsets"
            t[~inside] = 0.0
            same(t, want, dt, name)
    # NaN in a row that no expert owns stays out; in one that some expert owns it stays in its row
    off = offsets([1] + [n] * e) if n > 1 else offsets([0] + [1] * e)
    X[0, i - 1], X[n - 1, 0] = float("nan"), float("nan")
    Y = out(n, o, dt)
    K.kq_grouped_gemm(X, W, off, Y, w1.ws)
    assert bool(torch.isnan(Y[n - 1]).all())
    if n > 1:
        assert bool((Y[0] == -77.0).all())
        same(Y[1:n - 1], torch.mm(x[1:n - 1], w[0].T), dt, "Y beside NaN")


@pytest.mark.parametrize("n,e,o,i", [(9, 1, 40, 33), (17, 1, 17, 130), (31, 1, 33, 257), (32, 1, 100, 64), (60, 3, 70, 1001), (200, 7, 41, 514),
                                     (90, 3, 16, 2047), (23, 1, 33, 257), (24, 1, 100, 64), (160, 7, 41, 514), (70, 3, 16, 2047)])
def test_grouped_few_rows_in_two_blocks_exact(n, e, o, i):
    """Few rows of fp32 in work-groups of 32 rows, two blocks of 16: means of 8 to 24 rows an expert; and just above, in tiles."""
    assert 8 * e < n <= 32 * e
    test_grouped_forward_exact("few, two blocks", "f32", n, e, o, i)


@pytest.mark.parametrize("dt,n", [("bf16", 1), ("bf16", 5000), ("bf16", 30000), ("f32", 5000), ("f32", 40000), ("f32", 120000)])
def test_the_most_experts(dt, n):
    """4096 experts, most of them empty, of few rows and of tiles: products, gated products and both gradients, exact."""
    torch, dev = torch_dev()
    e, o, i = 4096, 20, 40
    say(f"grouped, 4096 experts {dt} n={n}")
    g = generator(n)
    (X, x), (dY, dy) = whole_numbers(n, i, dt, 4, g), whole_numbers(n, o, dt, 4, g)
    (W, w), (U, u) = stack(e, o, i, dt, 4, g), stack(e, o, i, dt, 4, g)
    for off in (dealt(n, e, g), offsets([0] * 4000 + [n // 3] * 96 + [n])):
        k = torch.bucketize(torch.arange(n, device=dev), off[1:].long(), right=True)     # each row's expert
        a, b, dx = (torch.empty((n, d), dtype=torch.float64, device=dev) for d in (o, o, i))
        dw = torch.zeros((e, o, i), dtype=torch.float64, device=dev)
        for p in range(0, n, 2000):
            r = slice(p, min(p + 2000, n))
            a[r], b[r] = (x[r, None, :] * w[k[r]]).sum(2), (x[r, None, :] * u[k[r]]).sum(2)
            dx[r] = (dy[r, :, None] * w[k[r]]).sum(1)
            dw.index_add_(0, k[r], dy[r, :, None] * x[r, None, :])       # whole numbers below 2^53: the order does not matter
        Y, H, dX, (flat, dW) = out(n, o, dt), out(n, o, dt), out(n, i, dt), out_stack(e, o, i, dt)
        K.kq_grouped_gemm(X, W, off, Y, space("grouped_gemm", o, i, n, dt, e))
        K.kq_grouped_gated(X, W, U, off, "relu", H, ws=space("grouped_gated", o, i, n, dt, e))
        K.kq_grouped_backward(dY, X, W, off, dX, dW, ws=space("grouped_backward", o, i, n, dt, e))
        for t, want, name in ((Y, a, "Y"), (H, a.float().clamp(min=0) * b.float(), "H"), (dX, dx, "dX"), (flat, dw.view(e * o, i), "dW")):
            same(t, want, dt, name)


@pytest.mark.parametrize("n,e,o,i", [(50, 6, 40, 64), (300, 5, 70, 130)])
def test_any_offsets_stay_inside(n, e, o, i):
    """Offsets that decrease, are negative or lie past the rows are read as the header says, in every entry point."""
    import torch
    g = generator(n)
    X, x = whole_numbers(n, i, "bf16", 4, g)
    W, w = stack(e, o, i, "bf16", 4, g)
    dY, dy = whole_numbers(n, o, "bf16", 4, g)
    big = 2 ** 31 - 1
    for values in ([0] * (e + 1), [n] * (e + 1), [-5, n // 2, 3, n // 2 + 4, big, 7, n][:e + 1], [big] * (e + 1), [-big - 1] * e + [big],
                   [n // 3, 0, 0, n - 1, 2 * n, 0, 0][:e + 1]):
        off = offsets(values)
        Y, dX, (flat, dW) = out(n, o, "bf16"), out(n, i, "bf16"), out_stack(e, o, i, "bf16")
        K.kq_grouped_gemm(X, W, off, Y)
        K.kq_grouped_backward(dY, X, W, off, dX, dW)
        wy, inside = oe.grouped(host(x), host(w), values)
        wx, ww = oe.grouped_grad(host(dy), host(x), host(w), values)
        out_rows = torch.from_numpy(~inside).to(X.device)
        for t, want, name in ((Y, wy, "Y"), (dX, wx, "dX")):
            assert bool((t[out_rows] == -77.0).all()), name
            t[out_rows] = 0.0
            same(t, torch.from_numpy(want).to(X.device), "bf16", name)
        same(flat, torch.from_numpy(ww).to(X.device).view(e * o, i), "bf16", "dW")


# what each is there for: tile shapes and cuts of dX (of one product, of two) and of dW; two uncut S plans run in one launch
BACKWARD = [("one launch", "bf16", 1, 1, 40, 33), ("one launch", "bf16", 33, 3, 65, 70), ("one launch", "bf16", 64, 16, 70, 200),
            ("one launch", "bf16", 500, 70, 33, 65), ("one launch, dX cut", "bf16", 21, 2, 477, 1), ("one launch, dX cut", "bf16", 21, 7, 914, 1),
            ("dX M", "bf16", 263, 4, 41, 8360), ("dX M", "bf16", 643, 10, 2, 3470), ("dX2 M split", "bf16", 1564, 2, 1616, 1459),
            ("dX2 M mixed", "bf16", 1838, 2, 740, 8681), ("dX M split", "bf16", 1003, 2, 2830, 2059), ("dX M mixed", "bf16", 4747, 2, 1491, 3430),
            ("dX2 L split", "bf16", 2764, 2, 6048, 3195), ("dX2 L mixed", "bf16", 7189, 2, 1656, 6962), ("dX L mixed", "bf16", 10782, 2, 3298, 3479),
            ("dW L", "bf16", 915, 2, 935, 4375), ("dW L split", "bf16", 11824, 2, 941, 2069), ("dW M", "bf16", 66, 19, 66, 1748),
            ("dW M split", "bf16", 5001, 2, 371, 971), ("dW S split", "bf16", 907, 2, 1, 1), ("dW S split", "bf16", 9000, 1, 40, 72),
            ("some", "bf16", 104, 30, 1097, 67), ("some", "bf16", 3000, 5, 1100, 900),
            ("one launch", "f32", 1, 1, 40, 33), ("one launch", "f32", 64, 16, 70, 200), ("one launch", "f32", 517, 5, 130, 257),
            ("one launch, dX cut", "f32", 21, 2, 235, 1), ("dW split", "f32", 478, 2, 1, 1), ("some", "f32", 1000, 70, 40, 65),
            ("some", "f32", 3000, 2, 200, 100)]
# tiles with four slabs in LDS for dX (of one product, of two), whole and split, of K that ends anywhere in the four
BACKWARD += [("dX MD (may)", "bf16", 602, 4, 8716, 2763), ("dX MD", "bf16", 3211, 2, 466, 649), ("dX MD", "bf16", 2811, 2, 268, 1119),
             ("dX MD", "bf16", 544, 4, 328, 2694), ("dX MD", "bf16", 609, 2, 419, 3844), ("dX MD", "bf16", 1378, 2, 199, 2346),
             ("dX MD split", "bf16", 741, 2, 7885, 2530), ("dX SD (may)", "bf16", 257, 4, 5146, 409), ("dX SD", "bf16", 1091, 2, 452, 3),
             ("dX SD", "bf16", 920, 2, 265, 1), ("dX SD", "bf16", 948, 2, 333, 10), ("dX SD", "bf16", 1091, 2, 412, 1),
             ("dX SD", "bf16", 937, 2, 141, 4), ("dX SD split", "bf16", 80, 8, 4531, 66), ("dX2 MD (may)", "bf16", 2117, 11, 3496, 734),
             ("dX2 MD", "bf16", 1547, 2, 257, 1443), ("dX2 MD", "bf16", 1965, 2, 327, 1203), ("dX2 MD", "bf16", 959, 2, 397, 2050),
             ("dX2 MD", "bf16", 2468, 2, 129, 835), ("dX2 MD split", "bf16", 3924, 4, 4537, 491), ("dX2 SD (may)", "bf16", 129, 2, 4390, 951),
             ("dX2 SD", "bf16", 904, 2, 65, 4)]


@pytest.mark.parametrize("plan,dt,n,e,o,i", BACKWARD)
def test_grouped_backward_exact(plan, dt, n, e, o, i):
    """Whole numbers of at most 4: products of at most 16; 2 * 8716 and 11824 of them sum to less than 2^19."""
    import torch
    say(f"grouped backward {plan} {dt} n={n} e={e} o={o} i={i}")
    g = generator(n + e + o + i)
    X, x = whole_numbers(n, i, dt, 4, g)
    (dY, dy), (dZ, dz) = whole_numbers(n, o, dt, 4, g), whole_numbers(n, o, dt, 4, g)
    (W, w), (U, u) = stack(e, o, i, dt, 4, g), stack(e, o, i, dt, 4, g)
    space_ = Workspace("grouped_backward", o, i, n, dt, e)
    ws = space_.ws
    for off in (dealt(n, e, g), dealt(n, e, g, n // 4, n - n // 5), offsets([0] * e + [n])):
        d1, d2 = (torch.zeros((n, i), dtype=torch.float64, device=X.device) for _ in range(2))
        gw, gu = (torch.zeros((e, o, i), dtype=torch.float64, device=X.device) for _ in range(2))
        inside = torch.zeros(n, dtype=torch.bool, device=X.device)
        for k, p, q in oe.spans(host(off), n):
            d1[p:q], d2[p:q], inside[p:q] = torch.mm(dy[p:q], w[k]), torch.mm(dz[p:q], u[k]), True
            gw[k], gu[k] = torch.mm(dy[p:q].T, x[p:q]), torch.mm(dz[p:q].T, x[p:q])
        dX, dX1 = out(n, i, dt), out(n, i, dt)
        (fW, dW), (fU, dU), (f1, dW1) = (out_stack(e, o, i, dt) for _ in range(3))
        K.kq_grouped_backward(dY, X, W, off, dX, dW, dZ, U, dU, ws)
        K.kq_grouped_backward(dY, X, W, off, dX1, dW1, ws=ws)
        for t, want, name in ((dX, d1 + d2, "dX of two"), (dX1, d1, "dX")):
            assert bool((t[~inside] == -77.0).all()), name + ": rows outside the offsets"
            t[~inside] = 0.0
            same(t, want, dt, name)
        for t, want, name in ((fW, gw, "dW"), (f1, gw, "dW alone"), (fU, gu, "dW2")):
            same(t, want.view(e * o, i), dt, name)
        # any subset of the outputs has the same bits
        dX2, (_, dU2) = out(n, i, dt), out_stack(e, o, i, dt)
        K.kq_grouped_backward(dY, None, W, off, dX2, dY2=dZ, W2=U, ws=ws)
        K.kq_grouped_backward(dY, X, None, off, dY2=dZ, dW2=dU2, ws=ws)
        assert torch.equal(dX2[inside], dX[inside]) and torch.equal(dU2, dU)
        assert bool((dX2[~inside] == -77.0).all()) and space_.kept()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [20, 400])
def test_grouped_ordinary_values(n, dt):
    """Products and gradients of normal values, all activations, against float64 with the bounds of sums of k products."""
    torch, dev = torch_dev()
    e, o, i = 4, 90, 150
    rng = np.random.default_rng(n)
    X, x = put(rng.standard_normal((n, i)), dt)
    W, w = put(rng.standard_normal((e * o, i)) * 2 / np.sqrt(i), dt)
    U, u = put(rng.standard_normal((e * o, i)) / np.sqrt(i), dt)
    dY, dy = put(rng.standard_normal((n, o)), dt)
    W3, U3 = (t.as_strided((e, o, i), (o * t.stride(0), t.stride(0), 1)) for t in (W, U))
    w, u = w.reshape(e, o, i), u.reshape(e, o, i)
    off = [0, n // 3, n // 3, n - 5, n]
    a, b = oe.grouped(x, w, off)[0], oe.grouped(x, u, off)[0]
    da, db = i * E23 * oe.grouped(np.abs(x), np.abs(w), off)[0], i * E23 * oe.grouped(np.abs(x), np.abs(u), off)[0]
    for kind in KINDS:
        H, A, B = mat(n, o, dt), mat(n, o, dt), mat(n, o, dt)
        K.kq_grouped_gated(X, W3, U3, offsets(off), kind, H, A, B)
        check(get(A), a, da + HALF[dt] * (np.abs(a) + da), "A")
        check(get(B), b, db + HALF[dt] * (np.abs(b) + db), "B")
        check(get(H), ob.act(a, kind)[0] * b, gated_tol(a, b, da, db, kind, dt), "H")
    dX, dW = mat(n, i, dt), torch.empty((e, o, i + (-i) % 8), dtype=X.dtype, device=dev)[:, :, :i]
    K.kq_grouped_backward(dY, X, W3, offsets(off), dX, dW)
    wx, ww = oe.grouped_grad(dy, x, w, off)
    sx, sw = oe.grouped_grad(np.abs(dy), np.abs(x), np.abs(w), off)
    check(get(dX), wx, o * E23 * sx + HALF[dt] * (np.abs(wx) + o * E23 * sx), "dX")
    check(get(dW), ww, n * E23 * sw + HALF[dt] * (np.abs(ww) + n * E23 * sw), "dW")
    if dt == "f32":          # the kernel's gradients against differences of the product, which is linear in each operand
        for grad, k in ((get(dX), 0), (get(dW), 1)):
            V = rng.standard_normal(grad.shape)
            lo, hi = ([x + (k == 0) * s * V if k == 0 else x, w + s * V if k == 1 else w] for s in (-0.5, 0.5))
            diff = ((oe.grouped(*hi, off)[0] - oe.grouped(*lo, off)[0]) * dy).sum()
            assert abs(diff - (grad * V).sum()) <= ((o if k == 0 else n) * E23 + 2.0 ** -23) * np.abs((sx, sw)[k] * V).sum()


def test_no_rows():
    torch, dev = torch_dev()
    for dt in ("f32", "bf16"):
        W = mat(6 * 20, 24, dt, fill=1.0).unflatten(0, (6, 20))
        x, y = mat(0, 24, dt), mat(0, 20, dt)
        off = offsets([0] * 7)
        (f1, dW), (f2, dU) = out_stack(6, 20, 24, dt), out_stack(6, 20, 24, dt)
        K.kq_grouped_gemm(x, W, off, y)
        K.kq_grouped_gated(x, W, W, off, "silu", y)
        K.kq_grouped_backward(y, x, W, off, x, dW, y, W, dU)
        for f in (f1, f2):
            same(f, torch.zeros((120, 24), device=dev), dt, "dW")


def test_grouped_offsets_past_32_bits():
    """Tokens 64 KiB apart (4.3 GB in all) and stacked weights and gradients past 2^31 values."""
    torch, dev = torch_dev()
    n, o, i, e = 65700, 72, 40, 3
    g = generator(7)

    def wide(d, fill=None):
        t = torch.empty((n, 32768), dtype=torch.bfloat16, device=dev)[:, :d]
        t.copy_(torch.randint(-4, 5, (n, d), generator=g, device=dev)) if fill is None else t.fill_(fill)
        return t

    X, dY, (W, w) = wide(i), wide(o), stack(e, o, i, "bf16", 4, g)
    Y, dX, (fW, dW) = wide(o, -77.0), wide(i, -77.0), out_stack(e, o, i, "bf16")
    cut = 65600
    off = offsets([5, 20, cut, n])
    say("grouped offsets: tokens")
    K.kq_grouped_gemm(X, W, off, Y, space("grouped_gemm", o, i, n, "bf16", e))
    K.kq_grouped_backward(dY, X, W, off, dX, dW, ws=space("grouped_backward", o, i, n, "bf16", e))
    same(Y[cut:].contiguous(), torch.mm(X[cut:].double(), w[2].T), "bf16", "Y")
    same(dX[cut:].contiguous(), torch.mm(dY[cut:].double(), w[2]), "bf16", "dX")
    # up to 65580 products of at most 16: sums below 2^21
    same(fW, torch.cat([torch.mm(dY[p:q].double().T.contiguous(), X[p:q].double()) for p, q in ((5, 20), (20, cut), (cut, n))]), "bf16", "dW")
    assert bool((Y[:5] == -77.0).all()) and bool((dX[:5] == -77.0).all())
    del X, dY, Y, dX
    say("grouped offsets: weights")
    n, o, i, e = 600, 4104, 65544, 9
    W = torch.zeros((e, o, i), dtype=torch.bfloat16, device=dev)
    last = torch.randint(-4, 5, (o, i), generator=g, device=dev)
    W[e - 1].copy_(last)
    (X, x), (dY, dy) = whole_numbers(n, i, "bf16", 4, g), whole_numbers(n, o, "bf16", 4, g)
    Y, dX = out(n, o, "bf16"), out(n, i, "bf16")
    off = offsets([0, 100] + [100] * (e - 2) + [n])
    K.kq_grouped_gemm(X, W, off, Y, space("grouped_gemm", o, i, n, "bf16", e))
    same(Y[100:], torch.mm(x[100:], last.double().T), "bf16", "Y")
    W[0].copy_(last)
    K.kq_grouped_backward(dY, X, W, off, dX, W, ws=space("grouped_backward", o, i, n, "bf16", e))
    same(dX, torch.mm(dy, last.double()), "bf16", "dX")
    assert torch.equal(W[e - 1], torch.mm(dy[100:].T.contiguous(), x[100:]).bfloat16()) and bool((W[1:e - 1] == 0).all())


# --------------------------------------------------------------------- streams, graphs, two calls
@pytest.mark.parametrize("n", [20, 300])
def test_replayed_from_a_graph(n):
    """One graph of an expert layer's calls: every replay on new inputs and new offsets gives the eager result, with eager work
    between the replays."""
    torch, dev = torch_dev()
    e, o, i, dt = 5, 136, 264, "bf16"
    g = generator(n)
    X, dH = mat(n, i, dt, fill=0.0), mat(n, o, dt, fill=0.0)
    (W, _), (U, _) = stack(e, o, i, dt, 4, g), stack(e, o, i, dt, 4, g)
    gamma = torch.ones(i, dtype=X.dtype, device=dev)
    off = offsets([0] * (e + 1))
    wq = [K.i8_empty(e * o, i, dev) for _ in range(2)]
    for t, q in zip((W, U), wq):
        K.kq_i8_quantize(t.flatten(0, 1), *q)
    gq, uq = ((c.unflatten(0, (e, o)), s.view(e, o)) for c, s in wq)

    def buffers():
        return dict(N=mat(n, i, dt, fill=0.0), stats=[torch.empty(n, device=dev) for _ in range(2)], H=mat(n, o, dt, fill=0.0), A=mat(n, o, dt, fill=0.0),
                    B=mat(n, o, dt, fill=0.0), dA=mat(n, o, dt, fill=0.0), dB=mat(n, o, dt, fill=0.0), dN=mat(n, i, dt, fill=0.0),
                    dW=torch.empty_like(W), dU=torch.empty_like(U), dX=mat(n, i, dt, fill=0.0), dg=torch.empty_like(gamma), q=K.i8_empty(n, i, dev),
                    Q=mat(n, o, dt, fill=0.0), w=Workspace("norm_backward", 0, i, n, dt).ws)

    def run(b):
        K.kq_norm_forward(X, gamma, None, "rms", 1e-5, b["N"], rstd=b["stats"][1])
        K.kq_grouped_gated(b["N"], W, U, off, "silu", b["H"], b["A"], b["B"])
        K.kq_gated_backward(dH, b["A"], b["B"], None, None, None, "silu", b["dA"], b["dB"])
        K.kq_grouped_backward(b["dA"], b["N"], W, off, b["dN"], b["dW"], b["dB"], U, b["dU"])
        K.kq_norm_backward(b["dN"], X, gamma, None, b["stats"][1], "rms", b["dX"], b["dg"], ws=b["w"])
        K.kq_i8_quantize(b["N"], *b["q"])
        K.kq_i8_gated(*b["q"], *gq, *uq, "silu", b["Q"], off)

    cap, eager = buffers(), buffers()
    run(cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(cap)
    for rep in range(3):
        X.copy_(torch.randn(n, i, generator=g, device=dev))
        dH.copy_(torch.randn(n, o, generator=g, device=dev))
        off.copy_(dealt(n, e, g))
        run(eager)
        torch.cuda.synchronize()
        graph.replay()
        run(eager)
        torch.cuda.synchronize()
        for k in ("N", "H", "A", "B", "dA", "dB", "dN", "dW", "dU", "dX", "dg", "Q"):
            assert torch.equal(cap[k], eager[k]), (rep, k)
        assert torch.equal(cap["q"][0], eager["q"][0])


def test_two_streams_at_once():
    torch, dev = torch_dev()
    n, e, o, i = 300, 4, 520, 512
    g = generator(1)
    jobs = []
    for _ in range(2):
        X, x = whole_numbers(n, i, "bf16", 4, g)
        W, w = stack(e, o, i, "bf16", 4, g)
        off = dealt(n, e, g)
        want = torch.cat([torch.mm(x[p:q], w[k].T) for k, p, q in oe.spans(host(off), n)])
        jobs.append((X, W, off, out(n, o, "bf16"), want, torch.cuda.Stream(dev)))
    for _ in range(5):
        for X, W, off, Y, _, st in jobs:
            st.wait_stream(torch.cuda.current_stream())
            K.kq_grouped_gemm(X, W, off, Y, stream=st)
        torch.cuda.synchronize()
        for _, _, _, Y, want, _ in jobs:
            same(Y, want, "bf16", "Y")
            Y.fill_(0.0)
            Y.as_strided((n, Y.stride(0)), (Y.stride(0), 1))[:, o:] = -77.0


def test_the_same_call_gives_the_same_bits():
    """Ordinary values on tiles whose K is cut: every call, on a workspace of any contents, has the bits of the first."""
    torch, dev = torch_dev()
    n, e, o, i = 4400, 3, 1795, 3000
    torch.manual_seed(3)
    X, W = mat(n, i, "bf16"), torch.empty((e, o, i), dtype=torch.bfloat16, device=dev)
    X.copy_(torch.randn(n, i, device=dev)), W.copy_(torch.randn(e, o, i, device=dev))
    off, ws, first = offsets([0, 1900, 2500, n]), space("grouped_gemm", o, i, n, "bf16", e), None
    for fill in (0, 255, 7):
        if ws is not None:
            ws.fill_(fill)
        Y = mat(n, o, "bf16")
        K.kq_grouped_gemm(X, W, off, Y, ws)
        first = Y if first is None else first
        assert torch.equal(Y, first)
