"""Block operators on every way a product can be cut: tile shapes of 256, 128 and 64 rows (L, M, S), K whole, split
for all tiles, or split for the tiles behind the last full turn of the GPU only (mixed), and the products of few tokens.

Two kinds of test. Exact ones: operands are small multiples of a power of two, so that every partial sum of
a product, in any order, is such a multiple below 2^24 times it. fp32 then holds all of them, the result is
the definition's rounded once, and the tolerance is zero: one lost, doubled or misplaced column shows at any
length of K. Same-bits ones: ordinary values, where a result may not depend on what else is asked for, on the
workspace's contents, on other streams or on a replay.
"""
import numpy as np
import pytest

from post_quantization_03_amd import _lib as K
from post_quantization_03_amd import ffn
from post_quantization_03_amd.layer import LayerCfg
from tests.gpu_util import host, say, torch_dev
from tests.test_gpu_blocks import E23, check, get, mat, tdtype

pytestmark = pytest.mark.gpu


class Workspace:
    """Exactly the bytes that a call asks for, full of NaN, with bytes behind that have to stay."""

    def __init__(self, op, o, i, n, dt="bf16", fill=255):
        torch, dev = torch_dev()
        self.need = K.kq_workspace_bytes(op, o, i, n, K.KQ_BF16 if dt == "bf16" else K.KQ_F32)
        self.buf = torch.full((self.need + 4096,), fill, dtype=torch.uint8, device=dev)
        self.buf[self.need:] = 0xA5
        self.ws = self.buf[:self.need] if self.need else None

    def kept(self):
        return bool((self.buf[self.need:] == 0xA5).all())


def generator(seed):
    torch, dev = torch_dev()
    return torch.Generator(device=dev).manual_seed(seed)


def whole_numbers(rows, cols, dt, top, g):
    """Whole numbers of -top .. top on the device, NaN in the padding behind each row; and as float64."""
    torch, dev = torch_dev()
    t = mat(rows, cols, dt, pad=1)
    t.copy_(torch.randint(-top, top + 1, (rows, cols), generator=g, device=dev))
    return t, t.double()


def out(rows, cols, dt):
    return mat(rows, cols, dt, pad=1, fill=-77.0)


def same(got, want, dt, what):
    """Equal to the exact result rounded to dt, the padding as it was."""
    import torch
    w = want.float().to(tdtype(dt))
    bad = got != w
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}: " \
                                f"{got[bad][0].item()} for {w[bad][0].item()}"
    whole = got.as_strided((got.shape[0], got.stride(0)), (got.stride(0), 1))
    assert bool((whole[:, got.shape[1]:] == -77.0).all()), f"{what}: padding written"


# ------------------------------------------------------------------------------- microscaled, exact
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def mx_exact(rows, cols, low, spread, g):
    """A microscaled operand of random codes: block scales 2^(low - 127) or twice that, times a power 2^-spread ..
    2^spread of its own for each row. Returns codes, scales and float64 values."""
    torch, dev = torch_dev()
    nblk = -(-cols // 32)
    code = torch.randint(0, 16, (rows, nblk * 32), generator=g, device=dev)
    code[:, cols:] = 0
    scale = torch.randint(low, low + 2, (rows, nblk), generator=g, device=dev)
    scale += torch.randint(-spread, spread + 1, (rows, 1), generator=g, device=dev)
    c, s = K.mx_empty(rows, cols, dev)
    c.copy_(code[:, 0::2] | code[:, 1::2] << 4)
    s.fill_(0xEE)
    s[:, :nblk] = scale
    table = torch.tensor(VALUES, dtype=torch.float64, device=dev)
    v = table[code] * torch.exp2((scale - 127).double()).repeat_interleave(32, dim=1)
    return c, s, v[:, :cols]


# tile plan: sizes whose products are cut so
MX_GEMM = [("few", 1, 41, 11008), ("few", 16, 41, 1001), ("few", 17, 100, 11008), ("few", 32, 41, 1001),
           ("S", 49, 67, 35), ("S split", 50, 65, 4359), ("S split", 65, 130, 2000), ("M", 3151, 1938, 33),
           ("M split", 2731, 68, 9421), ("M split", 130, 4001, 7990), ("M mixed", 1287, 5950, 2406),
           ("L", 1694, 6991, 1049), ("L split", 17109, 136, 23215), ("L mixed", 1765, 9349, 5379)]
MX_GATED = [("few", 1, 41, 11008), ("few", 16, 41, 1001), ("few", 17, 100, 11008), ("few", 32, 41, 1001),
            ("S", 49, 67, 35), ("S split", 50, 65, 4359), ("M", 258, 10735, 34), ("M split", 66, 1513, 9276),
            ("M mixed", 6580, 577, 2332), ("L", 539, 9939, 1027), ("L split", 136, 8250, 21747),
            ("L mixed", 658, 11003, 6107)]


@pytest.mark.parametrize("plan,n,o,i", MX_GEMM)
def test_mx_gemm_exact(plan, n, o, i):
    """Values are multiples of 2^-2 (tokens) and 2^-1 (weights) of at most 6 and 12, so products are multiples of 2^-3 of
    at most 72, and 23215 of them sum to less than 2^21 = 2^24 * 2^-3. The rows' powers multiply whole
    results; the largest is below 2^(21 + 100), the smallest other than 0 2^(-3 - 100)."""
    import torch
    say(f"mx gemm exact {plan} n={n} o={o} i={i}")
    g = generator(n + o + i)
    (ac, as_, a), (bc, bs, b) = mx_exact(n, i, 126, 50, g), mx_exact(o, i, 127, 50, g)
    want = a @ b.T
    for dt in ("f32", "bf16"):
        w, y = Workspace("mx_gemm", o, i, n, dt), out(n, o, dt)
        K.kq_mx_gemm(ac, as_, bc, bs, i, y, w.ws)
        same(y, want, dt, "Y")
        assert w.kept()
    # a block that is NaN: the last of the last token's, the first of one weight's
    r, c = n - 1, o // 2
    as_[r, -(-i // 32) - 1], bs[c, 0] = 255, 255
    w, y = Workspace("mx_gemm", o, i, n), out(n, o, "f32")
    K.kq_mx_gemm(ac, as_, bc, bs, i, y, w.ws)
    assert bool(torch.isnan(y[r]).all()) and bool(torch.isnan(y[:, c]).all())
    y[r], y[:, c] = want[r].float(), want[:, c].float()
    same(y, want, "f32", "Y beside NaN")


@pytest.mark.parametrize("plan,n,o,i", MX_GATED)
def test_mx_gated_exact(plan, n, o, i):
    """Both products as above; with max(a, 0) the block is their product, rounded to fp32 and then to the output."""
    import torch
    say(f"mx gated exact {plan} n={n} o={o} i={i}")
    g = generator(n + o + i)
    x, gate, up = mx_exact(n, i, 126, 15, g), mx_exact(o, i, 127, 15, g), mx_exact(o, i, 127, 15, g)
    a, b = x[2] @ gate[2].T, x[2] @ up[2].T
    want = a.float().clamp(min=0) * b.float()
    for dt in ("f32", "bf16"):
        w, h = Workspace("mx_gated", o, i, n, dt), out(n, o, dt)
        K.kq_mx_gated(*x[:2], *gate[:2], *up[:2], i, "relu", h, w.ws)
        same(h, want, dt, "H")
        assert w.kept()
    r, c, d = n - 1, o // 2, o // 3
    x[1][r, -(-i // 32) - 1], gate[1][c, 0], up[1][d, -(-i // 32) - 1] = 255, 255, 255
    w, h = Workspace("mx_gated", o, i, n), out(n, o, "f32")
    K.kq_mx_gated(*x[:2], *gate[:2], *up[:2], i, "relu", h, w.ws)
    assert bool(torch.isnan(h[r]).all()) and bool(torch.isnan(h[:, [c, d]]).all())
    h[r], h[:, [c, d]] = want[r], want[:, [c, d]]
    same(h, want, "f32", "H beside NaN")


# ------------------------------------------------------------------------------------- dense, exact
FORWARD = [("few", "bf16", 1, 41, 11008), ("few", "bf16", 8, 700, 11007), ("few", "bf16", 33, 41, 1001), ("few", "bf16", 48, 100, 11008),
           ("few", "f32", 1, 41, 11008), ("few", "f32", 17, 100, 11007), ("few", "f32", 32, 41, 1001),
           ("S", "bf16", 49, 67, 35), ("S split", "bf16", 49, 66, 1103), ("M", "bf16", 200, 8507, 33), ("M split", "bf16", 68, 1387, 4789),
           ("M mixed", "bf16", 393, 8303, 676), ("L", "bf16", 515, 10110, 265), ("L split", "bf16", 138, 8431, 5537),
           ("L mixed", "bf16", 1498, 5461, 1474),
           ("S", "f32", 49, 67, 35), ("S split", "f32", 53, 65, 555), ("S mixed", "f32", 7380, 263, 298)]


@pytest.mark.parametrize("plan,dt,n,o,i", FORWARD)
def test_gated_forward_exact(plan, dt, n, o, i):
    """Whole numbers of at most 4: products of at most 16, 11008 of which sum to less than 2^18."""
    say(f"gated forward exact {plan} {dt} n={n} o={o} i={i}")
    g = generator(n + o + i)
    (X, x), (Wg, wg), (Wu, wu) = (whole_numbers(r, i, dt, 4, g) for r in (n, o, o))
    a, b = x @ wg.T, x @ wu.T
    w = Workspace("gated_forward", o, i, n, dt)
    H, A, B = (out(n, o, dt) for _ in range(3))
    K.kq_gated_forward(X, Wg, Wu, "relu", H, A, B, w.ws)
    same(A, a, dt, "A")
    same(B, b, dt, "B")
    same(H, a.float().clamp(min=0) * b.float(), dt, "H")
    assert w.kept()
    # NaN in the last token's last value, infinity in one weight's: their row and their column, nothing else
    import torch
    r, c, h = n - 1, o // 2, a.float().clamp(min=0) * b.float()
    X[r, i - 1], Wg[c, i - 1] = float("nan"), float("inf")
    K.kq_gated_forward(X, Wg, Wu, "relu", H, A, B, w.ws)
    for t, v, name in ((A, a, "A"), (B, b, "B"), (H, h, "H")):
        assert bool(torch.isnan(t[r]).all()), name
        t[r] = v[r].to(t.dtype)
        if name != "B":
            assert name == "H" or not bool(torch.isfinite(A[:r, c]).any())
            t[:, c] = v[:, c].to(t.dtype)
        same(t, v, dt, name + " beside NaN")


# plans of dX and of the weight gradients; two S plans run in one launch
BACKWARD = [("L split", "L split", "bf16", 5693, 2984, 651), ("L mixed", "L mixed", "bf16", 1943, 937, 8660),
            ("L mixed", "L", "bf16", 1694, 690, 9455), ("L", "M split", "bf16", 7657, 198, 1031),
            ("M mixed", "M mixed", "bf16", 647, 274, 10950), ("M split", "M", "bf16", 65, 2377, 2874),
            ("M split", "S split", "bf16", 2755, 2062, 70), ("M", "M", "bf16", 606, 65, 8428),
            ("M", "S split", "bf16", 5003, 65, 590), ("S", "L", "bf16", 258, 1165, 5020),
            ("S split", "M split", "bf16", 4937, 1387, 70), ("S split", "S split", "bf16", 464, 207, 33),
            ("S", "S split", "bf16", 386, 71, 34), ("S split", "S", "bf16", 51, 202, 33), ("S", "S", "bf16", 49, 67, 35),
            ("S split", "S split", "f32", 193, 97, 33), ("S split", "S mixed", "f32", 198, 10885, 143),
            ("S split", "S", "f32", 52, 97, 33), ("S mixed", "S split", "f32", 1197, 101, 3436),
            ("S mixed", "S mixed", "f32", 463, 199, 8249), ("S mixed", "S", "f32", 553, 102, 7258),
            ("S", "S split", "f32", 195, 66, 33), ("S", "S mixed", "f32", 205, 138, 10923), ("S", "S", "f32", 49, 67, 35),
            ("long", "long", "bf16", 11001, 40, 72), ("long", "long", "f32", 11001, 40, 72)]


@pytest.mark.parametrize("px,pw,dt,n,o,i", BACKWARD)
def test_gated_backward_exact(px, pw, dt, n, o, i):
    """Whole numbers of at most 3 (dH, A, B) and 4 (X, weights): with max(a, 0), dA and dB are at most 9, exact in
    bf16; the gradients' products are at most 36, and 2 * 11008 of them sum to less than 2^20."""
    say(f"gated backward exact {px} / {pw} {dt} n={n} o={o} i={i}")
    g = generator(n + o + i)
    (dH, dh), (A, a), (B, b) = (whole_numbers(n, o, dt, 3, g) for _ in range(3))
    (X, x), (Wg, wg), (Wu, wu) = (whole_numbers(r, i, dt, 4, g) for r in (n, o, o))
    da, db = dh * b * (a > 0), dh * a.clamp(min=0)
    want = {"dA": da, "dB": db, "dX": da @ wg + db @ wu, "dWg": da.T @ x, "dWu": db.T @ x}
    w = Workspace("gated_backward", o, i, n, dt)
    got = {k: out(*v.shape, dt) for k, v in want.items()}
    K.kq_gated_backward(dH, A, B, X, Wg, Wu, "relu", *got.values(), w.ws)
    for k in want:
        same(got[k], want[k], dt, k)
    assert w.kept()
    # NaN in one value of dH, X and Wg each: the rows and columns of the gradients that it enters, nothing else
    import torch
    dH[n - 1, o - 1], X[0, i - 1], Wg[o // 2, 0] = (float("nan"),) * 3
    K.kq_gated_backward(dH, A, B, X, Wg, Wu, "relu", *got.values(), w.ws)
    every = slice(None)
    for k, places in (("dA", [(n - 1, o - 1)]), ("dB", [(n - 1, o - 1)]), ("dX", [(n - 1, every), (every, 0)]),
                      ("dWg", [(o - 1, every), (every, i - 1)]), ("dWu", [(o - 1, every), (every, i - 1)])):
        for at in places:
            assert bool(torch.isnan(got[k][at]).all()), (k, at)
        for at in places:
            got[k][at] = want[k][at].to(got[k].dtype)
        same(got[k], want[k], dt, k + " beside NaN")


# ---------------------------------------------------------------------------------------- same bits
def normal(rows, cols, dt, std, g):
    torch, dev = torch_dev()
    t = mat(rows, cols, dt, pad=1)
    t.copy_(torch.randn((rows, cols), generator=g, device=dev) * std)
    return t


def backward_operands(n, o, i, dt, seed):
    g = generator(seed)
    return [normal(n, o, dt, 1.0, g) for _ in range(3)] + [normal(n, i, dt, 1.0, g)] + [normal(o, i, dt, i ** -0.5, g) for _ in range(2)]


# both plans S and split (one launch), both mixed, M with whole and split K
@pytest.mark.parametrize("dt,n,o,i", [("f32", 520, 264, 520), ("bf16", 464, 207, 33), ("f32", 463, 199, 8249),
                                      ("bf16", 1943, 937, 8660), ("bf16", 65, 2377, 2874)])
def test_each_gradient_alone_and_in_company(dt, n, o, i):
    """Every choice of the three optional gradients gives the bits of the full call."""
    import torch
    say(f"gradients in company {dt} n={n} o={o} i={i}")
    ops = backward_operands(n, o, i, dt, n)
    shapes = {"dA": (n, o), "dB": (n, o), "dX": (n, i), "dWg": (o, i), "dWu": (o, i)}

    def call(names):
        got = {k: out(*shapes[k], dt) for k in ("dA", "dB") + names}
        w = Workspace("gated_backward", o, i, n, dt)
        X = ops[3] if "dWg" in names or "dWu" in names else None
        W = ops[4:] if "dX" in names else [None, None]
        K.kq_gated_backward(*ops[:3], X, *W, "gelu", *(got.get(k) for k in shapes), w.ws)
        torch.cuda.synchronize()
        assert w.kept()
        return got

    full = call(("dX", "dWg", "dWu"))
    for names in (("dX",), ("dWg",), ("dWu",), ("dX", "dWg"), ("dX", "dWu"), ("dWg", "dWu"), ()):
        for k, t in call(names).items():
            assert torch.equal(t, full[k]), (names, k)


def block_calls(seed, fill=255):
    """Calls of all four products, each with a workspace of its own: (call, outputs). Every one lays out
    scales, splits K, or both."""
    torch, dev = torch_dev()
    g = generator(seed)
    calls, inputs, spaces = [], [], []

    def operand(rows, cols, std=1.0):
        x = normal(rows, cols, "f32", std, g)
        q = K.mx_empty(rows, cols, dev)
        K.kq_mx_quantize(x, *q)
        inputs.append(q[0])
        return q

    def space(*size):
        w = Workspace(*size, fill=fill)
        assert w.need > 0, size
        spaces.append(w)
        return w.ws

    for n, o, i in ((130, 4001, 7990), (65, 130, 2000)):
        a, b, y = operand(n, i), operand(o, i), out(n, o, "bf16")
        w = space("mx_gemm", o, i, n)
        calls.append((lambda stream=None, a=a, b=b, y=y, i=i, w=w: K.kq_mx_gemm(*a, *b, i, y, w, stream=stream), [y]))
    n, o, i = 66, 1513, 9276
    x, gate, up, h = operand(n, i), operand(o, i, i ** -0.5), operand(o, i, i ** -0.5), out(n, o, "f32")
    wg = space("mx_gated", o, i, n)
    calls.append((lambda stream=None: K.kq_mx_gated(*x, *gate, *up, 9276, "silu", h, wg, stream=stream), [h]))
    n, o, i = 68, 1387, 4789
    X, G, U = normal(n, i, "bf16", 1.0, g), normal(o, i, "bf16", i ** -0.5, g), normal(o, i, "bf16", i ** -0.5, g)
    H, A, B = (out(n, o, "bf16") for _ in range(3))
    wf = space("gated_forward", o, i, n)
    calls.append((lambda stream=None: K.kq_gated_forward(X, G, U, "silu", H, A, B, wf, stream=stream), [H, A, B]))
    m, p, q = 1500, 2000, 520
    ops = backward_operands(m, p, q, "bf16", seed + 1)
    grads = [out(m, p, "bf16"), out(m, p, "bf16"), out(m, q, "bf16"), out(p, q, "bf16"), out(p, q, "bf16")]
    wb = space("gated_backward", p, q, m)
    calls.append((lambda stream=None: K.kq_gated_backward(*ops, "silu", *grads, wb, stream=stream), grads))
    return calls, inputs + [X] + ops[:1], spaces


def snapshot(calls):
    return [t.clone() for _, outs in calls for t in outs]


def equal(got, want):
    import torch
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_a_workspace_held_before_does_not_matter():
    import torch
    seen = []
    for fill in (0, 255, 0x7F):
        calls, _, spaces = block_calls(7, fill)
        for call, _ in calls:
            call()
        torch.cuda.synchronize()
        seen.append(snapshot(calls))
        for w in spaces:
            assert w.kept()
    assert equal(seen[1], seen[0]) and equal(seen[2], seen[0])
    assert all(bool(torch.isfinite(t.float()).all()) for t in seen[0])


def test_two_streams_with_workspaces_of_their_own():
    """All products on two streams at once, in opposite orders, each with a workspace of its own."""
    torch, dev = torch_dev()
    sets = [block_calls(s)[0] for s in (11, 12)]
    want = []
    for calls in sets:
        for call, _ in calls:
            call()
        torch.cuda.synchronize()
        want.append(snapshot(calls))
    streams = [torch.cuda.Stream(dev) for _ in sets]
    for rep in range(5):
        for calls in sets:
            for _, outs in calls:
                for t in outs:
                    t.fill_(-77.0)
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        for a, b in zip(sets[0], reversed(sets[1])):
            a[0](stream=streams[0])
            b[0](stream=streams[1])
        torch.cuda.synchronize()
        for calls, w in zip(sets, want):
            assert equal(snapshot(calls), w), rep


def test_replays_of_products_that_use_workspaces():
    """All products in one graph: replays on new inputs, with NaN in the workspaces and eager calls of the
    same kind before each, give the eager bits."""
    torch, dev = torch_dev()
    (cap, cap_in, spaces), (eager, eager_in, _) = block_calls(21), block_calls(21)
    for call, _ in cap + eager:
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _ in cap:
            call()
    for rep in range(4):
        g = generator(100 + rep)
        for a, b in zip(cap_in, eager_in):
            if a.dtype == torch.uint8:      # other signs in the blocks that K does not end in
                a[:, :-16] ^= torch.randint(0, 2, (a.shape[0], a.shape[1] - 16), generator=g, device=dev, dtype=torch.uint8) * 0x88
            else:
                a.copy_(torch.randn(a.shape, generator=g, device=dev))
            b.copy_(a)
        for w in spaces:
            w.buf[:w.need].fill_(255)
        for call, _ in eager:
            call()
        torch.cuda.synchronize()
        graph.replay()
        for call, _ in eager:
            call()
        torch.cuda.synchronize()
        assert equal(snapshot(cap), snapshot(eager)), rep
        for w in spaces:
            assert w.kept()


def test_two_threads_with_streams_of_their_own():
    """All products from two host threads, each on a stream of its own."""
    import threading
    torch, dev = torch_dev()
    sets = [block_calls(s)[0] for s in (31, 32)]
    want = []
    for calls in sets:
        for call, _ in calls:
            call()
        torch.cuda.synchronize()
        want.append(snapshot(calls))
        for _, outs in calls:
            for t in outs:
                t.fill_(-77.0)
    torch.cuda.synchronize()
    errors = []

    def work(calls, stream):
        try:
            for _ in range(3):
                for call, _ in calls:
                    call(stream=stream)
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(calls, torch.cuda.Stream(dev))) for calls in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not errors
    for calls, w in zip(sets, want):
        assert equal(snapshot(calls), w)


@pytest.mark.parametrize("n", [1, 4, 130])
def test_served_block_replayed_from_a_graph(n):
    """MXFeedForward in a graph, its buffers and workspaces the graph's: replays on new tokens give the eager bits."""
    torch, dev = torch_dev()
    i, o, dt = 1024, 4032, "bf16"
    g = generator(n)
    block = ffn.MXFeedForward(normal(o, i, dt, i ** -0.5, g), normal(o, i, dt, i ** -0.5, g), normal(i, o, dt, o ** -0.5, g), "silu")
    X = normal(n, i, dt, 1.0, g)
    block(X)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = block(X)
    for rep in range(4):
        X.copy_(torch.randn((n, i), generator=g, device=dev))
        want = block(X)
        torch.cuda.synchronize()
        graph.replay()
        block(X)
        torch.cuda.synchronize()
        assert torch.equal(Y, want) and bool(torch.isfinite(Y.float()).all()), rep


# ----------------------------------------------------------------------------- refusals, calibration
def test_workspace_views_are_refused_on_the_device():
    torch, dev = torch_dev()
    c, s = K.mx_empty(130, 7990, dev)
    w, ws = K.mx_empty(4001, 7990, dev)
    need = K.kq_workspace_bytes("mx_gemm", 4001, 7990, 130)
    for bad in (torch.empty(1, dtype=torch.uint8, device=dev).expand(need), torch.empty(2 * need, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            K.kq_mx_gemm(c, s, w, ws, 7990, out(130, 4001, "bf16"), bad)


@pytest.mark.parametrize("dt,o,form,blk", [("bf16", 203, "full", 0), ("bf16", 192, "block", 64), ("f32", 192, "block", 64),
                                           ("f32", 203, "full", 0), ("bf16", 203, "diag", 0)])
def test_calibration_in_every_storage_form(dt, o, form, blk):
    """The covariances of calibrate_gated are those of its own gradient rows: n squares, summed in at least fp32
    (n 2^-23 of the sum of magnitudes) and rounded to fp32."""
    n, i = 333, 100
    g = generator(o)
    X, Wg, Wu, dH = normal(n, i, dt, 1.0, g), normal(o, i, dt, 0.1, g), normal(o, i, dt, 0.1, g), normal(n, o, dt, 1.0, g)
    cal = ffn.calibrate_gated(X, Wg, Wu, dH, "silu", LayerCfg(bits=4, form=form, blk=blk))
    for name, rows in (("HG_gate", get(cal["dA"])), ("HG_up", get(cal["dB"]))):
        want, mag = rows.T @ rows / n, np.abs(rows).T @ np.abs(rows) / n
        if form == "diag":
            want, mag = np.diag(want), np.diag(mag)
        if form == "block":
            want, mag = (np.array([m[k:k + blk, k:k + blk] for k in range(0, o, blk)]) for m in (want, mag))
        assert cal[name].shape == want.shape
        check(host(cal[name]).astype(np.float64), want, (n + 2) * E23 * mag, name)


def test_served_block_refuses_rows_off_16_bytes():
    """A contiguous matrix of a width that is no multiple of 16 bytes is refused, as every entry point does; the same
    values in padded rows are taken."""
    torch, dev = torch_dev()
    flat = torch.ones((40, 33), dtype=torch.bfloat16, device=dev)
    padded = mat(40, 33, "bf16")
    padded.copy_(flat)
    down = mat(33, 40, "bf16", fill=1.0)
    with pytest.raises(K.KQError, match="16 bytes"):
        ffn.MXFeedForward(flat, flat, down)
    block = ffn.MXFeedForward(padded, padded, down)
    with pytest.raises(K.KQError, match="16 bytes"):
        block(flat)
    assert block(padded).shape == (40, 33)
