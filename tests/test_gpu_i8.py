"""8-bit integer operators on the GPU against the definitions.

Sums of products of codes are whole numbers that int32 holds, so a product's result is fl32(sum) * fl32(sA sB), rounded to
fp32 and then to the output: the tolerance is zero, whatever the order of the sums. The gated block with max(a, 0) is one more
fp32 product of two such results. With the other activations the bounds are those of the gated block on dense
operands, a being off by three roundings of fp32.
"""
import numpy as np
import pytest

from oracle import blocks as ob
from oracle import experts as oe
from post_quantization_03_amd import _lib as K
from tests.gpu_util import host, say, torch_dev
from tests.test_gpu_blocks import KINDS, check, gated_tol, get, mat, put
from tests.test_gpu_blocks_plans import generator, out, same

pytestmark = pytest.mark.gpu


class Workspace:
    """Exactly the bytes that a call asks for, full of ones, with bytes behind that have to stay."""

    def __init__(self, op, o, i, n, dt="bf16", experts=0):
        torch, dev = torch_dev()
        self.need = K.kq_workspace_bytes(op, o, i, n, K.KQ_BF16 if dt == "bf16" else K.KQ_F32, group=experts)
        self.buf = torch.full((self.need + 4096,), 255, dtype=torch.uint8, device=dev)
        self.buf[self.need:] = 0xA5
        self.ws = self.buf[:self.need] if self.need else None

    def kept(self):
        return bool((self.buf[self.need:] == 0xA5).all())


# --------------------------------------------------------------------------------- quantisation
def special_rows(cols):
    """Rows with every kind of tie, with the ends of fp32's range and around the smallest scale."""
    rng = np.random.default_rng(cols)
    rows = [np.zeros(cols), -np.zeros(cols)]
    for e in (-118, -60, 0, 100, 120):
        r = rng.integers(-254, 255, cols) / 2.0           # halves: ties where the multiplier is a power of two
        r[cols // 2] = 127.0 * rng.choice([-1, 1])
        rows.append(r * 2.0 ** e)
    near = (rng.integers(-253, 254, cols) / 2.0) * (1 + rng.choice([-1, 0, 1], cols) * 2.0 ** -23)
    near[0] = 127.0
    rows.append(near)
    rows.append(rng.standard_normal(cols) * np.exp(2 * rng.standard_normal(cols)))
    rows.append(np.full(cols, 3.4028234e38))
    for top in (2.0 ** -119, 2.0 ** -119 * (1 - 2.0 ** -24), 2.0 ** -149):
        r = rng.uniform(-1, 1, cols) * top
        r[-1] = top
        rows.append(r)
    return np.array(rows).astype(np.float32)


# every number of pieces a thread and threads a row, whole and ragged, and rows past the registers
COLS = [1, 3, 7, 15, 16, 17, 100, 255, 512, 513, 1000, 1024, 1025, 2047, 2048, 2049, 4096, 4100, 8192, 8200, 11008, 13824, 16384, 16391,
        32768, 32770, 50001]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_quantise_and_back_exact(cols, dt):
    torch, dev = torch_dev()
    say(f"i8 quantise cols={cols} {dt}")
    x, v = put(special_rows(cols), dt, pad=1)
    rows = x.shape[0]
    codes, scales = oe.i8_quantize(v)
    ld = -(-cols // 16) * 16 + 16
    c = torch.full((rows + 2, ld), 0x5B, dtype=torch.int8, device=dev)
    s = torch.full((rows + 2,), -7.0, device=dev)
    K.kq_i8_quantize(x, c[:rows, :cols], s[:rows])
    hc, hs = host(c), host(s)
    assert np.array_equal(hs[:rows], scales, equal_nan=True)       # fp32's largest value is infinite as bf16
    assert np.array_equal(hc[:rows, :cols], codes)
    assert (hc[rows:] == 0x5B).all() and (hc[:, cols:] == 0x5B).all() and (hs[rows:] == -7.0).all()   # nothing else is written
    for kind in ("f32", "bf16"):
        y = mat(rows, cols, kind, pad=1, fill=-77.0)
        K.kq_i8_dequantize(c[:rows, :cols], s[:rows], y)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(oe.i8_values(codes, scales)).to(y.dtype).double().numpy()
        assert np.array_equal(get(y), want, equal_nan=True)
        assert (host(y.as_strided((rows, y.stride(0)), (y.stride(0), 1)).float())[:, cols:] == -77.0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [33, 1500, 5000, 60000])
def test_quantise_infinities_and_nan(cols, dt):
    torch, dev = torch_dev()
    x = np.random.default_rng(cols).standard_normal((6, cols)).astype(np.float32)
    x[0, cols - 1], x[1, 0], x[3, cols // 2], x[4, 3] = np.inf, np.nan, -np.inf, 3e38
    t, v = put(x, dt)
    c, s = K.i8_empty(6, cols, dev)
    K.kq_i8_quantize(t, c, s)
    codes, scales = oe.i8_quantize(v)
    assert np.array_equal(host(s), scales, equal_nan=True) and np.array_equal(host(c), codes)
    y = mat(6, cols, dt)
    K.kq_i8_dequantize(c, s, y)
    assert np.isnan(get(y)).all(axis=1).tolist() == [True, True, False, True, False, False]
    assert not np.isnan(get(y)[[2, 4, 5]]).any()


def test_every_code_and_single_rows():
    torch, dev = torch_dev()
    c = torch.arange(-128, 128, device=dev).to(torch.int8).repeat(5, 1)
    s = torch.tensor([1.0, 2.0 ** -126, 3e36, 0.0, 1.1], device=dev)
    for dt in ("f32", "bf16"):
        y = mat(5, 256, dt)
        K.kq_i8_dequantize(c, s, y)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(oe.i8_values(host(c), host(s))).to(y.dtype).double().numpy()
        assert np.array_equal(get(y), want)
    x = torch.randn(1, 64, device=dev)
    c, s = K.i8_empty(1, 64, dev)
    K.kq_i8_quantize(x, c, s)
    assert np.array_equal(host(c), oe.i8_quantize(get(x))[0])
    c0, s0 = K.i8_empty(0, 64, dev)
    K.kq_i8_quantize(x[:0], c0, s0)
    K.kq_i8_dequantize(c0, s0, x[:0])
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------- products
def operand(rows, cols, g, stack=0):
    """Random codes with stray bytes behind each row, and scales over many powers of two; a stack of matrices for
    several experts."""
    torch, dev = torch_dev()
    total = rows * max(stack, 1)
    c, s = K.i8_empty(total, cols, dev)
    c.as_strided((total, c.stride(0)), (c.stride(0), 1)).fill_(0x5B)
    c.copy_(torch.randint(-128, 128, (total, cols), generator=g, device=dev))
    s.copy_(torch.exp2(torch.randint(-20, 20, (total,), generator=g, device=dev).float()) *
            (1 + torch.rand(total, generator=g, device=dev)))
    if stack:
        return c.as_strided((stack, rows, cols), (rows * c.stride(0), c.stride(0), 1)), s.view(stack, rows)
    return c, s


def product(a, b):
    """The definition's fp32 result."""
    import torch
    sums = torch.mm(a[0].double(), b[0].double().T)
    return sums.float() * torch.outer(a[1], b[1])


# few tokens; tile shapes of 256, 128 and 64 rows, K whole, split for all tiles, or for those behind the last full turn
GEMM = [(1, 1, 1), (1, 41, 11008), (5, 100, 255), (16, 64, 256), (17, 130, 257), (32, 48, 1000), (33, 1, 1), (33, 1, 783),
        (65, 255, 100), (66, 256, 64), (255, 129, 511), (11182, 321, 2), (753, 976, 4977), (1444, 5455, 903),
        (2444, 3256, 953), (2553, 1613, 11112), (3209, 5104, 3210), (40, 50, 131071), (3, 20, 131071)]
# tiles with four slabs in LDS (MD, SD), whole and split, of long and short K; lengths of K that end anywhere in the four; S split
GEMM += [(961, 2080, 750), (2715, 1101, 392), (1131, 901, 8895), (33, 1, 3137), (33, 1, 4391), (200, 300, 8000)]
GEMM += [(70, 200, i) for i in (257, 300, 384, 385, 500, 512, 513, 639, 640, 641, 767, 768, 769, 896, 1025)]
GEMM += [(1100, 2100, i) for i in (512, 513, 640, 700, 768, 769, 897, 1024, 1151)]
GATED = [(1, 1, 1), (1, 41, 11008), (5, 100, 255), (16, 64, 256), (17, 130, 257), (32, 48, 1000), (33, 1, 1), (33, 1, 783),
         (65, 255, 100), (255, 129, 511), (197, 8230, 5), (489, 749, 5038), (1032, 3644, 801), (2638, 1597, 943),
         (1256, 1688, 11153), (3232, 2521, 3230)]
# few rows that begin at multiples of 128 bytes: wavefronts without a slab, with one, with several; the ends of the choice
SPREAD = [113, 128, 245, 896, 1017, 1024, 1152, 2160, 4090, 11008]
GEMM += [(n, 100, i) for n in (1, 7) for i in SPREAD] + [(16, 8192, 200), (16, 8193, 200), (8, 8193, 200), (9, 8193, 200)]
GATED += [(n, 100, i) for n in (1, 7) for i in SPREAD] + [(16, 4096, 200), (16, 4097, 200), (8, 4097, 200), (9, 4097, 200)]
GATED += [(1045, 1049, 773), (545, 2867, 393), (862, 585, 8107), (33, 1, 3137), (34, 1, 8495), (33, 1, 4391), (70, 200, 640)]


@pytest.mark.parametrize("n,o,i", GEMM)
def test_i8_gemm_exact(n, o, i):
    import torch
    say(f"i8 gemm n={n} o={o} i={i}")
    g = generator(n + o + i)
    a, b = operand(n, i, g), operand(o, i, g)
    if i == 131071:
        a[0].fill_(-128), b[0].fill_(-128)        # the largest sum there is: 131071 * 2^14 < 2^31
    want = product(a, b)
    for dt in ("f32", "bf16"):
        w, y = Workspace("i8_gemm", o, i, n, dt), out(n, o, dt)
        K.kq_i8_gemm(*a, *b, y, ws=w.ws)
        same(y, want, dt, "Y")
        assert w.kept()
    # a scale that is NaN: its row, its column
    r, c = n - 1, o // 2
    a[1][r], b[1][c] = float("nan"), float("nan")
    w, y = Workspace("i8_gemm", o, i, n), out(n, o, "f32")
    K.kq_i8_gemm(*a, *b, y, ws=w.ws)
    assert bool(torch.isnan(y[r]).all()) and bool(torch.isnan(y[:, c]).all())
    y[r], y[:, c] = want[r], want[:, c]
    same(y, want, "f32", "Y beside NaN")


@pytest.mark.parametrize("n,o,i", GATED)
def test_i8_gated_exact(n, o, i):
    say(f"i8 gated n={n} o={o} i={i}")
    g = generator(n + o + i)
    x, gate, up = operand(n, i, g), operand(o, i, g), operand(o, i, g)
    want = product(x, gate).clamp(min=0) * product(x, up)
    for dt in ("f32", "bf16"):
        w, h = Workspace("i8_gated", o, i, n, dt), out(n, o, dt)
        K.kq_i8_gated(*x, *gate, *up, "relu", h, ws=w.ws)
        same(h, want, dt, "H")
        assert w.kept()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 70])
def test_i8_gated_activations(n, kind, dt):
    torch, dev = torch_dev()
    o, i = 90, 200
    rng = np.random.default_rng(n)
    ops, vals = [], []
    for rows, std in ((n, 1.0), (o, 2 / np.sqrt(i)), (o, 1 / np.sqrt(i))):
        codes, scales = oe.i8_quantize(rng.standard_normal((rows, i)) * std)
        c, s = K.i8_empty(rows, i, dev)
        c.copy_(torch.from_numpy(codes)), s.copy_(torch.from_numpy(scales))
        ops += [c, s]
        vals.append(codes.astype(np.float64) * scales.astype(np.float64)[:, None])
    h = mat(n, o, dt)
    K.kq_i8_gated(*ops, kind, h, ws=Workspace("i8_gated", o, i, n, dt).ws)
    want, a, b = ob.gated(*vals, kind)
    da, db = 3 * 2.0 ** -24 * np.abs(a), 3 * 2.0 ** -24 * np.abs(b)      # the sum's, the scales' and their product's rounding
    check(get(h), want, gated_tol(a, b, da, db, kind, dt), "H")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1 << 22, (1 << 22) - 5])
def test_quantise_the_widest_rows(cols, dt):
    """Rows of 4 MiB of codes, the most that there are."""
    torch, dev = torch_dev()
    say(f"i8 quantise cols={cols} {dt}")
    torch.manual_seed(cols)
    x = mat(2, cols, dt)
    x.copy_(torch.randn(2, cols, device=dev))
    c, s = K.i8_empty(2, cols, dev)
    K.kq_i8_quantize(x, c, s)
    codes, scales = oe.i8_quantize(get(x))
    assert np.array_equal(host(c), codes) and np.array_equal(host(s), scales)
    y = mat(2, cols, dt)
    K.kq_i8_dequantize(c, s, y)
    assert torch.equal(y, torch.from_numpy(oe.i8_values(codes, scales)).to(dev).to(y.dtype))


@pytest.mark.parametrize("n", [3, 9000, 30000])
def test_i8_the_most_experts(n):
    """4096 experts, most of them empty, of few rows and of tiles."""
    torch, dev = torch_dev()
    e, o, i = 4096, 20, 100
    say(f"i8, 4096 experts n={n}")
    g = generator(n)
    a, b, u = operand(n, i, g), operand(o, i, g, e), operand(o, i, g, e)
    for off in (dealt(n, e, g), offsets([0] * 4000 + [n // 3] * 96 + [n])):
        k = torch.bucketize(torch.arange(n, device=dev), off[1:].long(), right=True)
        wa, wu = (torch.empty((n, o), device=dev) for _ in range(2))
        for p in range(0, n, 2000):
            r = slice(p, min(p + 2000, n))
            for t, m in ((wa, b), (wu, u)):
                t[r] = (a[0][r, None, :].double() * m[0][k[r]].double()).sum(2).float() * (a[1][r, None] * m[1][k[r]])
        y, h = out(n, o, "f32"), out(n, o, "f32")
        K.kq_i8_gemm(*a, *b, y, off, Workspace("i8_gemm", o, i, n, "f32", e).ws)
        K.kq_i8_gated(*a, *b, *u, "relu", h, off, Workspace("i8_gated", o, i, n, "f32", e).ws)
        same(y, wa, "f32", "Y")
        same(h, wa.clamp(min=0) * wu, "f32", "H")


# ---------------------------------------------------------------------------------- grouped products
def offsets(values):
    torch, dev = torch_dev()
    return torch.tensor(values, dtype=torch.int32, device=dev)


def dealt(n, e, g, first=0, last=None):
    """Offsets of rows dealt unevenly, some experts left empty."""
    import torch
    last = n if last is None else last
    cuts = torch.randint(first, last + 1, (e - 1,), generator=g, device=g.device).sort().values.int()
    ends = torch.tensor([first, last], dtype=torch.int32, device=g.device)
    off = torch.cat((ends[:1], cuts, ends[1:]))
    if e > 3:
        off[2] = off[1]
    return off


# few rows an expert, one expert with more than the others, more experts than lanes; then tile shapes with K whole, split, or split
# for the tiles behind the last full turn, of the plain or the gated product
GROUPS = [(1, 1, 40, 33), (3, 4, 41, 100), (64, 16, 70, 1000), (90, 70, 40, 65), (200, 150, 30, 100), (100, 3, 33, 400), (500, 7, 130, 257),
          (776, 12, 2812, 17), (3000, 5, 1100, 900), (4100, 130, 70, 48), (20, 2, 1, 2488), (300, 28, 2330, 3184), (163, 15, 2386, 5039),
          (655, 10, 3306, 3), (1738, 2, 1176, 6420), (843, 3, 1123, 6029), (4046, 2, 4429, 5540), (2866, 2, 2926, 4064), (3652, 2, 2320, 1370),
          (5633, 3, 724, 901), (8505, 2, 4325, 5866), (9239, 2, 2685, 5103), (9224, 18, 736, 9018)]
# plans that came with the tiles of four slabs, and what is left of the others
GROUPS += [(2531, 4, 3096, 2704), (4288, 19, 593, 8976), (4963, 4, 587, 467), (1442, 2, 675, 9089), (645, 37, 1713, 5097), (17, 2, 1, 3734),
           *((n, 7, 100, i) for n in (1, 40) for i in SPREAD), (18, 2, 3, 7229), (6972, 2, 1120, 2033), (1322, 7, 1092, 10533), (858, 2, 1770, 427),
           (2065, 2, 259, 11894), (257, 2, 62, 7247), (8798, 2, 208, 11469), (242, 28, 2330, 3184)]


@pytest.mark.parametrize("n,e,o,i", GROUPS)
def test_i8_grouped_exact(n, e, o, i):
    import torch
    say(f"i8 grouped n={n} e={e} o={o} i={i}")
    g = generator(n + e + o + i)
    a, b, u = operand(n, i, g), operand(o, i, g, e), operand(o, i, g, e)
    lists = [dealt(n, e, g), dealt(n, e, g, n // 4, n - n // 5), offsets([0] * e + [n])]     # all rows of one expert, too
    for off in lists:
        wa, wu = torch.zeros((n, o), device=g.device), torch.zeros((n, o), device=g.device)
        inside = torch.zeros(n, dtype=torch.bool, device=g.device)
        for k, p, q in oe.spans(host(off), n):
            rows = (a[0][p:q], a[1][p:q])
            wa[p:q], wu[p:q], inside[p:q] = product(rows, (b[0][k], b[1][k])), product(rows, (u[0][k], u[1][k])), True
        for dt in ("f32", "bf16"):
            y, h = out(n, o, dt), out(n, o, dt)
            w1, w2 = Workspace("i8_gemm", o, i, n, dt, e), Workspace("i8_gated", o, i, n, dt, e)
            K.kq_i8_gemm(*a, *b, y, off, w1.ws)
            K.kq_i8_gated(*a, *b, *u, "relu", h, off, w2.ws)
            assert w1.kept() and w2.kept()
            for t, want, name in ((y, wa, "Y"), (h, wa.clamp(min=0) * wu, "H")):
                assert bool((t[~inside] == -77.0).all()), name + ": rows outside the offsets"
                t[~inside] = 0.0
                same(t, want * inside.unsqueeze(1), dt, name)


def test_i8_offsets_past_32_bits():
    """More than 2^31 codes of tokens and of stacked weights: the last rows are those of a call on these alone."""
    torch, dev = torch_dev()
    n, o, i, e, k = 70, 262200, 2064, 4, 40
    g = generator(5)
    a, b = operand(n, i, g), (torch.zeros((e, o, i), dtype=torch.int8, device=dev), torch.ones((e, o), device=dev))
    last, sl = operand(o, i, g)
    b[0][e - 1].copy_(last), b[1][e - 1].copy_(sl)
    y = out(n, o, "bf16")
    say("i8 offsets: grouped weights")
    K.kq_i8_gemm(*a, *b, y, offsets([0, 10, 10, 30, n]), Workspace("i8_gemm", o, i, n, experts=e).ws)
    assert bool((y[:30] == 0).all())
    same(y[30:], product((a[0][30:], a[1][30:]), (last, sl)), "bf16", "Y")
    del b, y
    rows, cols = 1049600, 2064
    say("i8 offsets: quantise")
    x = mat(rows, cols, "bf16", fill=0.0)
    x[-k:].copy_(torch.randn(k, cols, device=dev))
    c, s = K.i8_empty(rows, cols, dev)
    K.kq_i8_quantize(x, c, s)
    want = oe.i8_quantize(get(x[-k:]))
    assert np.array_equal(host(c[-k:]), want[0]) and np.array_equal(host(s[-k:]), want[1]) and bool((s[:-k] == 0).all())
    x.fill_(-77.0)
    K.kq_i8_dequantize(c, s, x)
    assert np.array_equal(get(x[-k:]), torch.from_numpy(oe.i8_values(*want)).bfloat16().double().numpy())
    assert bool((x[:-k] == 0).all())
    del x
    say("i8 offsets: tokens")
    b = operand(100, cols, g)
    y = out(rows, 100, "bf16")
    K.kq_i8_gemm(c, s, *b, y, ws=Workspace("i8_gemm", 100, cols, rows).ws)
    same(y[-k:], product((c[-k:], s[-k:]), b), "bf16", "last rows")
    assert bool((y[:-k] == 0).all())
