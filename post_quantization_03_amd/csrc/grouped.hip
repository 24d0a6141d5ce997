// Products grouped by expert on dense operands, forward and backward (KronQ review page, Method: the activation and
// gradient statistics of a layer come from one calibration pass; an expert layer has them for each expert, over the
// tokens that its router sent there). Rows of X are sorted by expert, off[k] .. off[k + 1] - 1 being expert k's.
//
//   Y_r = X_r W_k^T                                 for each row r of expert k
//   H_r = act(X_r Wg_k^T) * (X_r Wu_k^T)
//   dX_r = dY_r W_k [+ dY2_r W2_k],  dW_k = sum over k's rows of dY_r^T X_r  [dW2_k likewise]
//
// Types, roundings and sums are those of the gated block (gated.hip).
#include "group.h"

namespace kq {

struct DenseRows {
    const void* p;
    int64_t ld;
    const char* what;
};

static kq_status rows_check(const char* who, kq_dtype dt, const DenseRows& m, int64_t cols) {
    if (!m.p) return fail(KQ_EINVAL, "%s: null %s", who, m.what);
    if (m.ld < cols) return fail(KQ_ESHAPE, "%s: leading dimension of %s too small", who, m.what);
    if (!aligned16(m.p) || m.ld % (dt == KQ_BF16 ? 8 : 4))
        return fail(KQ_EINVAL, "%s: rows of %s must be 16-byte aligned", who, m.what);
    if (m.ld > TL_LD_MAX / 4) return fail(KQ_ESHAPE, "%s: %s too large", who, m.what);
    return KQ_OK;
}

static const char* bytes_of(const void* p) { return static_cast<const char*>(p); }

template <int E, bool GATED>
static kq_status forward(const char* who, const Group& gr, const void* X, int64_t ldx, const void* W, int64_t ldw, const void* W2,
                         int64_t ldw2, int64_t n, int64_t o, int64_t i, int act, kq_dtype dt, void* Y, int64_t ldy, void* A,
                         int64_t lda, void* B, int64_t ldb, void* ws, size_t ws_bytes, hipStream_t st) {
    const int64_t es = E == EL_BF16 ? 2 : 4;
    if (group_few<E>(n, gr.experts)) {
        FewArgs f{};
        f.n = n; f.o = o; f.K = i;
        f.A = bytes_of(X); f.lda = ldx * es;
        f.B = bytes_of(W); f.ldb = ldw * es;
        f.B2 = bytes_of(W2); f.ldb2 = ldw2 * es;
        f.Y = Y; f.ldy = ldy; f.Y2 = A; f.ldy2 = lda; f.Y3 = B; f.ldy3 = ldb;
        f.dt = dt; f.act = act;
        return group_few_launch<E, GATED>(f, gr, st, who);
    }
    TileArgs g{};
    g.M = n; g.N = o; g.K = i;
    g.A = bytes_of(X); g.lda = ldx * es;
    g.B = bytes_of(W); g.ldb = ldw * es;
    g.B2 = bytes_of(W2); g.ldb2 = ldw2 * es;
    g.Y = Y; g.ldy = ldy; g.Y2 = A; g.ldy2 = lda; g.Y3 = B; g.ldy3 = ldb;
    g.dt = dt; g.act = act; g.pairs = 1;
    return group_launch<E, GATED ? TP_GATED : TP_PLAIN>(g, gr, ws, ws_bytes, st, who);
}

template <int E, int MODE>
static kq_status backward(const char* who, const Group& gr, const TileArgs& x, const TileArgs& w, int pairs, void* ws, size_t ws_bytes,
                          hipStream_t st) {
    if (x.Y && pairs && group_grads_together<E, MODE>(x, w, gr)) return group_grads_launch<E, MODE>(x, w, gr, pairs, ws, ws_bytes, st, who);
    // a refused call leaves dX alone too: the weight gradients are checked first, dX by its own launch before it enqueues anything
    GradPlan plan{};
    if (pairs) KQ_TRY((group_grad_prepare<E>(plan, w, gr, pairs, ws, ws_bytes, who)));
    if (x.Y) KQ_TRY((group_launch<E, MODE>(x, gr, ws, ws_bytes, st, who)));
    return pairs ? group_grad_launch<E>(w, plan, gr, pairs, ws, st, who) : KQ_OK;
}
template <int E>
static kq_status backward(const char* who, const Group& gr, const TileArgs& x, const TileArgs& w, int pairs, void* ws, size_t ws_bytes,
                          hipStream_t st) {
    return x.A2 ? backward<E, TP_GRAD_X>(who, gr, x, w, pairs, ws, ws_bytes, st)
                : backward<E, TP_GRAD_X1>(who, gr, x, w, pairs, ws, ws_bytes, st);
}

}  // namespace kq

using namespace kq;

template <int E>
static size_t grouped_ws_of(kq_op op, int64_t o, int64_t i, int64_t n, int64_t experts) {
    if (op == KQ_OP_GROUPED_BACKWARD) {
        // the most that any call of these sizes takes: dX of one product or of two, one weight gradient or two
        const size_t a = group_ws<E, TP_GRAD_X>(n, experts, i, o), b = group_ws<E, TP_GRAD_X1>(n, experts, i, o);
        const size_t w = group_grad_ws<E>(n, experts, o, i, 2);
        return a > b ? (a > w ? a : w) : b > w ? b : w;
    }
    if (group_few<E>(n, experts)) return 0;
    return op == KQ_OP_GROUPED_GATED ? group_ws<E, TP_GATED>(n, experts, o, i) : group_ws<E, TP_PLAIN>(n, experts, o, i);
}

size_t grouped_ws(kq_op op, int64_t o, int64_t i, int64_t n, kq_dtype dt, int64_t experts) {
    if (n <= 0 || o <= 0 || i <= 0 || experts <= 0 || experts > GROUP_MAX || n > GROUP_ROWS_MAX || !tile_sizes_ok(n, o > i ? o : i)) return 0;
    return dt == KQ_BF16 ? grouped_ws_of<EL_BF16>(op, o, i, n, experts) : grouped_ws_of<EL_F32>(op, o, i, n, experts);
}

extern "C" kq_status kq_grouped_gemm(const void* X, int64_t ldx, const void* W, int64_t ldw, const int32_t* offsets,
                                     int64_t experts, kq_dtype dt, int64_t n, int64_t o, int64_t i, void* Y, int64_t ldy,
                                     void* ws, size_t ws_bytes, kq_stream stream) {
    const char* who = "kq_grouped_gemm";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    KQ_TRY(group_check(who, offsets, experts, n, o));
    if (n == 0) return KQ_OK;
    KQ_TRY(rows_check(who, dt, DenseRows{X, ldx, "X"}, i));
    KQ_TRY(rows_check(who, dt, DenseRows{W, ldw, "W"}, i));
    KQ_TRY(rows_check(who, dt, DenseRows{Y, ldy, "Y"}, o));
    const Group gr{offsets, (int)experts, (int)n, (int)o};
    if (dt == KQ_BF16)
        return forward<EL_BF16, false>(who, gr, X, ldx, W, ldw, nullptr, 0, n, o, i, 0, dt, Y, ldy, nullptr, 0, nullptr, 0, ws,
                                      ws_bytes, hs(stream));
    return forward<EL_F32, false>(who, gr, X, ldx, W, ldw, nullptr, 0, n, o, i, 0, dt, Y, ldy, nullptr, 0, nullptr, 0, ws,
                                      ws_bytes, hs(stream));
}

extern "C" kq_status kq_grouped_gated(const void* X, int64_t ldx, const void* Wg, int64_t ldg, const void* Wu, int64_t ldu,
                                      const int32_t* offsets, int64_t experts, kq_dtype dt, int64_t n, int64_t o, int64_t i,
                                      kq_act act, void* H, int64_t ldh, void* A, int64_t lda, void* B, int64_t ldb, void* ws,
                                      size_t ws_bytes, kq_stream stream) {
    const char* who = "kq_grouped_gated";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (act < KQ_ACT_SILU || act > KQ_ACT_RELU) return fail(KQ_EINVAL, "%s: bad activation", who);
    KQ_TRY(group_check(who, offsets, experts, n, o));
    if (n == 0) return KQ_OK;
    KQ_TRY(rows_check(who, dt, DenseRows{X, ldx, "X"}, i));
    KQ_TRY(rows_check(who, dt, DenseRows{Wg, ldg, "Wg"}, i));
    KQ_TRY(rows_check(who, dt, DenseRows{Wu, ldu, "Wu"}, i));
    KQ_TRY(rows_check(who, dt, DenseRows{H, ldh, "H"}, o));
    if (A) KQ_TRY(rows_check(who, dt, DenseRows{A, lda, "A"}, o));
    if (B) KQ_TRY(rows_check(who, dt, DenseRows{B, ldb, "B"}, o));
    const Group gr{offsets, (int)experts, (int)n, (int)o};
    if (dt == KQ_BF16)
        return forward<EL_BF16, true>(who, gr, X, ldx, Wg, ldg, Wu, ldu, n, o, i, act, dt, H, ldh, A, lda, B, ldb, ws,
                                      ws_bytes, hs(stream));
    return forward<EL_F32, true>(who, gr, X, ldx, Wg, ldg, Wu, ldu, n, o, i, act, dt, H, ldh, A, lda, B, ldb, ws,
                                      ws_bytes, hs(stream));
}

extern "C" kq_status kq_grouped_backward(const void* dY, int64_t lddy, const void* W, int64_t ldw, const void* dY2, int64_t lddy2,
                                         const void* W2, int64_t ldw2, const void* X, int64_t ldx, const int32_t* offsets,
                                         int64_t experts, kq_dtype dt, int64_t n, int64_t o, int64_t i, void* dX, int64_t lddx,
                                         void* dW, int64_t lddw, void* dW2, int64_t lddw2, void* ws, size_t ws_bytes,
                                         kq_stream stream) {
    const char* who = "kq_grouped_backward";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    KQ_TRY(group_check(who, offsets, experts, n, o));
    const bool two = dW2 || dY2 || W2;
    if (dW) KQ_TRY(rows_check(who, dt, DenseRows{dW, lddw, "dW"}, i));
    if (dW2) KQ_TRY(rows_check(who, dt, DenseRows{dW2, lddw2, "dW2"}, i));
    if (n > 0) {
        if (dX || dW) KQ_TRY(rows_check(who, dt, DenseRows{dY, lddy, "dY"}, o));
        if (two && (dX || dW2)) KQ_TRY(rows_check(who, dt, DenseRows{dY2, lddy2, "dY2"}, o));
        if (dX) {
            KQ_TRY(rows_check(who, dt, DenseRows{dX, lddx, "dX"}, i));
            KQ_TRY(rows_check(who, dt, DenseRows{W, ldw, "W"}, i));
            if (two) KQ_TRY(rows_check(who, dt, DenseRows{W2, ldw2, "W2"}, i));
        }
        if (dW || dW2) KQ_TRY(rows_check(who, dt, DenseRows{X, ldx, "X"}, i));
    }
    const int64_t es = dt == KQ_BF16 ? 2 : 4;
    const Group gr{offsets, (int)experts, (int)n, (int)o};
    TileArgs x{}, w{};
    x.M = n; x.N = i; x.K = o;
    x.A = bytes_of(dY); x.lda = lddy * es; x.B = bytes_of(W); x.ldb = ldw * es;
    if (two) { x.A2 = bytes_of(dY2); x.lda2 = lddy2 * es; x.B2 = bytes_of(W2); x.ldb2 = ldw2 * es; }
    x.Y = n > 0 ? dX : nullptr; x.ldy = lddx; x.dt = dt; x.pairs = 1;
    w.M = o; w.N = i;
    w.A = bytes_of(dW ? dY : dY2); w.lda = (dW ? lddy : lddy2) * es;
    w.A2 = bytes_of(dY2); w.lda2 = lddy2 * es;
    w.B = bytes_of(X); w.ldb = ldx * es;
    w.Y = dW ? dW : dW2; w.ldy = dW ? lddw : lddw2; w.Y2 = dW2; w.ldy2 = lddw2; w.dt = dt;
    const int pairs = dW && dW2 ? 2 : dW || dW2 ? 1 : 0;
    return dt == KQ_BF16 ? backward<EL_BF16>(who, gr, x, w, pairs, ws, ws_bytes, hs(stream))
                         : backward<EL_F32>(who, gr, x, w, pairs, ws, ws_bytes, hs(stream));
}
