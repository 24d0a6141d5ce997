// Gated feed-forward block on dense operands, forward and backward (KronQ review page, Method: the activation
// and gradient statistics of a layer come from one calibration pass; the rows of X and H feed H_X, those
// of dA and dB feed H_G of the gate and up projections).
//
//   A = X Wg^T,  B = X Wu^T,  H = act(A) * B
//   dA = dH * B * act'(A),  dB = dH * act(A)
//   dX = dA Wg + dB Wu,  dWg = dA^T X,  dWu = dB^T X
//
// bf16 operands run on the bf16 matrix cores with fp32 sums; A and B are rounded to bf16 only where the
// caller keeps them, H is computed from the unrounded sums. dA and dB are rounded to the operands' type
// once, as outputs and as the operands of the three gradient products: bf16 matrix cores take bf16
// operands, and a second product with what the rounding leaves would double the matrix work. The roundings (2^-8
// relative at most, independent from element to element) add up to an error of the size of the result's own
// rounding, not below it: at 8192 tokens of 11008 x 4096 weights dX, dWg and dWu are 0.0024 relative (norm of the
// difference over the norm) off the products of unrounded dA and dB, of which rounding the results alone makes
// 0.0017; elements whose terms cancel are off by more of themselves. fp32 operands run on the fp32 matrix cores throughout
// and are not rounded.
#include "tile.h"

namespace kq {

// dA and dB, 16 bytes a lane and operand; HBM-bound: three matrices read, two written (8192 x 11008 bf16: 150 us for
// 902 MB, 6 TB/s, the inputs partly in the last-level cache). Apart from the products: in the
// products' tiles it would be computed again in each of the i / 256 tiles that read an element.
template <bool BF>
__global__ __launch_bounds__(256) void gated_grad_kernel(const void* dH, int64_t lddh, const void* A, int64_t lda,
                                                         const void* B, int64_t ldb, int64_t n, int64_t o, int act,
                                                         void* dA, int64_t ldda, void* dB, int64_t lddb) {
    constexpr int V = BF ? 8 : 4;
    const int64_t per = (o + V - 1) / V, total = n * per;
    auto load = [&](const void* P, int64_t ld, int64_t r, int64_t c, float (&v)[V]) {
        if constexpr (BF) {
            const uint16_t* p = static_cast<const uint16_t*>(P) + r * ld + c;
            if (c + V <= o) {
                const uint4 w = *reinterpret_cast<const uint4*>(p);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    v[2 * k] = __uint_as_float(u[k] << 16);
                    v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; k++) v[k] = c + k < o ? from_bf16(p[k]) : 0.0f;
            }
        } else {
            const float* p = static_cast<const float*>(P) + r * ld + c;
            if (c + V <= o) {
                const float4 w = *reinterpret_cast<const float4*>(p);
                v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
            } else {
#pragma unroll
                for (int k = 0; k < V; k++) v[k] = c + k < o ? p[k] : 0.0f;
            }
        }
    };
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
        const int64_t r = e / per, c = (e - r * per) * V;
        float h[V], a[V], b[V], da[V], db[V];
        load(dH, lddh, r, c, h);
        load(A, lda, r, c, a);
        load(B, ldb, r, c, b);
        with_act(act, [&](auto ACT) {
#pragma unroll
            for (int k = 0; k < V; k++) {
                float f, df;
                act_both<ACT.value>(a[k], f, df);
                da[k] = h[k] * b[k] * df;
                db[k] = h[k] * f;
            }
        });
        store_run<V>(dA, BF ? KQ_BF16 : KQ_F32, r * ldda + c, da, o - c);
        store_run<V>(dB, BF ? KQ_BF16 : KQ_F32, r * lddb + c, db, o - c);
    }
}

// zeros in a rows x cols matrix (gradients of no tokens)
__global__ __launch_bounds__(256) void zero_rows_kernel(char* p, int64_t rows, int64_t bytes, int64_t ld) {
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * (bytes / 2); e += (int64_t)gridDim.x * 256)
        *reinterpret_cast<uint16_t*>(p + e / (bytes / 2) * ld + e % (bytes / 2) * 2) = 0;
}

struct Dense {
    const void* p;
    int64_t ld;
    const char* what;
};

static kq_status dense_check(const char* who, kq_dtype dt, const Dense& m, int64_t rows, int64_t cols) {
    if (!m.p) return fail(KQ_EINVAL, "%s: null %s", who, m.what);
    if (m.ld < cols) return fail(KQ_ESHAPE, "%s: leading dimension of %s too small", who, m.what);
    if (!aligned16(m.p) || m.ld % (dt == KQ_BF16 ? 8 : 4))
        return fail(KQ_EINVAL, "%s: rows of %s must be 16-byte aligned", who, m.what);
    if (m.ld > TL_LD_MAX / 4 || rows > TL_ROWS_MAX) return fail(KQ_ESHAPE, "%s: %s too large", who, m.what);
    return KQ_OK;
}

static kq_status ws_check(const char* who, const void* ws, size_t have, size_t need) {
    if (!ws || have < need || !aligned16(ws)) return fail(KQ_EWORKSPACE, "%s: workspace too small or not aligned to 16 bytes", who);
    return KQ_OK;
}

static const char* bytes_of(const void* p) { return static_cast<const char*>(p); }

template <int E>
static kq_status gated_forward(const char* who, const void* X, int64_t ldx, const void* Wg, int64_t ldg, const void* Wu,
                               int64_t ldu, int64_t n, int64_t o, int64_t i, int act, kq_dtype dt, void* H, int64_t ldh,
                               void* A, int64_t lda, void* B, int64_t ldb, void* ws,
                               size_t ws_bytes, hipStream_t st) {
    const int64_t es = E == EL_BF16 ? 2 : 4;
    if (few_tokens<E>(n, o, i)) {
        FewArgs f{};
        f.n = n; f.o = o; f.K = i;
        f.A = bytes_of(X); f.lda = ldx * es;
        f.B = bytes_of(Wg); f.ldb = ldg * es;
        f.B2 = bytes_of(Wu); f.ldb2 = ldu * es;
        f.Y = H; f.ldy = ldh; f.Y2 = A; f.ldy2 = lda; f.Y3 = B; f.ldy3 = ldb;
        f.dt = dt; f.act = act;
        return few_launch<E, true>(f, st, who);
    }
    TileArgs g{};
    g.M = n; g.N = o; g.K = i;
    g.A = bytes_of(X); g.lda = ldx * es;
    g.B = bytes_of(Wg); g.ldb = ldg * es;
    g.B2 = bytes_of(Wu); g.ldb2 = ldu * es;
    g.Y = H; g.ldy = ldh; g.Y2 = A; g.ldy2 = lda; g.Y3 = B; g.ldy3 = ldb;
    g.dt = dt; g.act = act;
    const TilePlan plan = tile_plan<E, TP_GATED>(n, o, i);
    if (plan.part) KQ_TRY(ws_check(who, ws, ws_bytes, sizeof(float) * plan.part));
    return tile_launch<E, TP_GATED>(g, plan, 1, static_cast<float*>(ws), st, who);
}

}  // namespace kq

using namespace kq;

size_t gated_forward_ws(int64_t o, int64_t i, int64_t n, kq_dtype dt) {
    if (n <= 0 || o <= 0 || i <= 0 || !tile_sizes_ok(n, o) ||
        (dt == KQ_BF16 ? few_tokens<EL_BF16>(n, o, i) : few_tokens<EL_F32>(n, o, i))) return 0;
    return sizeof(float) * (dt == KQ_BF16 ? tile_plan<EL_BF16, TP_GATED>(n, o, i) : tile_plan<EL_F32, TP_GATED>(n, o, i)).part;
}

struct GradPlans {
    TilePlan w, x;
    size_t bytes;        // of split sums: shared by products that run one after another on the caller's stream
};
static GradPlans grad_plans(int64_t o, int64_t i, int64_t n, kq_dtype dt) {
    GradPlans p;
    p.w = dt == KQ_BF16 ? tile_plan<EL_BF16, TP_GRAD_W>(o, i, n) : tile_plan<EL_F32, TP_GRAD_W>(o, i, n);
    p.x = dt == KQ_BF16 ? tile_plan<EL_BF16, TP_GRAD_X>(n, i, o) : tile_plan<EL_F32, TP_GRAD_X>(n, i, o);
    p.bytes = sizeof(float) * (grads_together(p.x, p.w) ? p.x.part + p.w.part : p.x.part > p.w.part ? p.x.part : p.w.part);
    return p;
}

size_t gated_backward_ws(int64_t o, int64_t i, int64_t n, kq_dtype dt) {
    if (n <= 0 || o <= 0 || i <= 0 || !tile_sizes_ok(n, i) || !tile_sizes_ok(o, i)) return 0;
    return grad_plans(o, i, n, dt).bytes;
}

extern "C" kq_status kq_gated_forward(const void* X, int64_t ldx, const void* Wg, int64_t ldg, const void* Wu, int64_t ldu,
                                      kq_dtype dt, int64_t n, int64_t o, int64_t i, kq_act act, void* H, int64_t ldh,
                                      void* A, int64_t lda, void* B, int64_t ldb, void* ws, size_t ws_bytes,
                                      kq_stream stream) {
    const char* who = "kq_gated_forward";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (act < KQ_ACT_SILU || act > KQ_ACT_RELU) return fail(KQ_EINVAL, "%s: bad activation", who);
    if (n == 0) return KQ_OK;
    if (!tile_sizes_ok(n, o)) return fail(KQ_ESHAPE, "%s: result too large", who);
    KQ_TRY(dense_check(who, dt, Dense{X, ldx, "X"}, n, i));
    KQ_TRY(dense_check(who, dt, Dense{Wg, ldg, "Wg"}, o, i));
    KQ_TRY(dense_check(who, dt, Dense{Wu, ldu, "Wu"}, o, i));
    KQ_TRY(dense_check(who, dt, Dense{H, ldh, "H"}, n, o));
    if (A) KQ_TRY(dense_check(who, dt, Dense{A, lda, "A"}, n, o));
    if (B) KQ_TRY(dense_check(who, dt, Dense{B, ldb, "B"}, n, o));
    if (dt == KQ_BF16)
        return gated_forward<EL_BF16>(who, X, ldx, Wg, ldg, Wu, ldu, n, o, i, act, dt, H, ldh, A, lda, B, ldb, ws, ws_bytes,
                                      hs(stream));
    return gated_forward<EL_F32>(who, X, ldx, Wg, ldg, Wu, ldu, n, o, i, act, dt, H, ldh, A, lda, B, ldb, ws, ws_bytes,
                                      hs(stream));
}

extern "C" kq_status kq_gated_backward(const void* dH, int64_t lddh, const void* A, int64_t lda, const void* B, int64_t ldb,
                                       const void* X, int64_t ldx, const void* Wg, int64_t ldg, const void* Wu, int64_t ldu,
                                       kq_dtype dt, int64_t n, int64_t o, int64_t i, kq_act act, void* dA, int64_t ldda,
                                       void* dB, int64_t lddb, void* dX, int64_t lddx, void* dWg, int64_t lddg, void* dWu,
                                       int64_t lddu, void* ws, size_t ws_bytes, kq_stream stream) {
    const char* who = "kq_gated_backward";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (act < KQ_ACT_SILU || act > KQ_ACT_RELU) return fail(KQ_EINVAL, "%s: bad activation", who);
    if ((dX && !tile_sizes_ok(n, i)) || ((dWg || dWu) && !tile_sizes_ok(o, i)))
        return fail(KQ_ESHAPE, "%s: gradients too large", who);
    if (dWg) KQ_TRY(dense_check(who, dt, Dense{dWg, lddg, "dWg"}, o, i));
    if (dWu) KQ_TRY(dense_check(who, dt, Dense{dWu, lddu, "dWu"}, o, i));
    const hipStream_t st = hs(stream);
    const int64_t es = dt == KQ_BF16 ? 2 : 4;
    if (n == 0) {
        void* w[2] = {dWg, dWu};
        const int64_t l[2] = {lddg, lddu};
        for (int k = 0; k < 2; k++) {
            if (!w[k]) continue;
            const int64_t e = o * i * (es / 2);
            hipLaunchKernelGGL(zero_rows_kernel, dim3((unsigned)((e + 255) / 256 < 8192 ? (e + 255) / 256 : 8192)), dim3(256),
                               0, st, static_cast<char*>(w[k]), o, i * es, l[k] * es);
            KQ_TRY(check_launch(who));
        }
        return KQ_OK;
    }
    KQ_TRY(dense_check(who, dt, Dense{dH, lddh, "dH"}, n, o));
    KQ_TRY(dense_check(who, dt, Dense{A, lda, "A"}, n, o));
    KQ_TRY(dense_check(who, dt, Dense{B, ldb, "B"}, n, o));
    KQ_TRY(dense_check(who, dt, Dense{dA, ldda, "dA"}, n, o));
    KQ_TRY(dense_check(who, dt, Dense{dB, lddb, "dB"}, n, o));
    if (dX) {
        KQ_TRY(dense_check(who, dt, Dense{dX, lddx, "dX"}, n, i));
        KQ_TRY(dense_check(who, dt, Dense{Wg, ldg, "Wg"}, o, i));
        KQ_TRY(dense_check(who, dt, Dense{Wu, ldu, "Wu"}, o, i));
    }
    if (dWg || dWu) KQ_TRY(dense_check(who, dt, Dense{X, ldx, "X"}, n, i));
    GradPlans plans{};
    if (dX || dWg || dWu) {
        plans = grad_plans(o, i, n, dt);
        if (plans.bytes) KQ_TRY(ws_check(who, ws, ws_bytes, plans.bytes));
    }
    float* part = static_cast<float*>(ws);
    {
        const int64_t total = n * ((o + 16 / es - 1) / (16 / es));
        const dim3 grid((unsigned)((total + 255) / 256 < 65536 ? (total + 255) / 256 : 65536));
        if (dt == KQ_BF16)
            hipLaunchKernelGGL((gated_grad_kernel<true>), grid, dim3(256), 0, st, dH, lddh, A, lda, B, ldb, n, o, (int)act, dA,
                               ldda, dB, lddb);
        else
            hipLaunchKernelGGL((gated_grad_kernel<false>), grid, dim3(256), 0, st, dH, lddh, A, lda, B, ldb, n, o, (int)act,
                               dA, ldda, dB, lddb);
        KQ_TRY(check_launch(who));
    }
    TileArgs x{}, w{};
    x.M = n; x.N = i; x.K = o;
    x.A = bytes_of(dA); x.lda = ldda * es; x.B = bytes_of(Wg); x.ldb = ldg * es;
    x.A2 = bytes_of(dB); x.lda2 = lddb * es; x.B2 = bytes_of(Wu); x.ldb2 = ldu * es;
    x.Y = dX; x.ldy = lddx; x.dt = dt;
    w.M = o; w.N = i; w.K = n;
    w.A = bytes_of(dWg ? dA : dB); w.lda = (dWg ? ldda : lddb) * es;
    w.A2 = bytes_of(dB); w.lda2 = lddb * es;
    w.B = bytes_of(X); w.ldb = ldx * es;
    w.Y = dWg ? dWg : dWu; w.ldy = dWg ? lddg : lddu; w.Y2 = dWu; w.ldy2 = lddu; w.dt = dt;
    const int pairs = dWg && dWu ? 2 : 1;
    if (dX && (dWg || dWu) && grads_together(plans.x, plans.w)) {
        x.pairs = 1; x.part = part;
        w.pairs = pairs; w.part = part + plans.x.part;
        return dt == KQ_BF16 ? tile_launch_grads<EL_BF16>(x, plans.x, w, plans.w, st, who)
                             : tile_launch_grads<EL_F32>(x, plans.x, w, plans.w, st, who);
    }
    if (dX) {
        if (dt == KQ_BF16) KQ_TRY((tile_launch<EL_BF16, TP_GRAD_X>(x, plans.x, 1, part, st, who)));
        else KQ_TRY((tile_launch<EL_F32, TP_GRAD_X>(x, plans.x, 1, part, st, who)));
    }
    if (dWg || dWu) {
        if (dt == KQ_BF16) KQ_TRY((tile_launch<EL_BF16, TP_GRAD_W>(w, plans.w, pairs, part, st, who)));
        else KQ_TRY((tile_launch<EL_F32, TP_GRAD_W>(w, plans.w, pairs, part, st, who)));
    }
    return KQ_OK;
}
