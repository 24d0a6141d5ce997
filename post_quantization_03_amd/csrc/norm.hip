// The norm in front of a block, forward and backward (KronQ review page, Method: the activation and gradient statistics of a
// layer come from one calibration pass, which runs through the norm on its way to the sublayers before it).
//
//   layer   m = mean x, r = 1 / sqrt(mean (x - m)^2 + eps)      rms   m = 0, r = 1 / sqrt(mean x^2 + eps)
//   h = (x - m) r,  y = h gamma + beta
//   g = dy gamma,  dx = r (g - [layer: mean g] - h mean(g h)),  dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
//
// Both passes are bound by HBM: x is read once and y written once (8192 x 4096 bf16 27.7 us, 4.8 TB/s); dy and x are read once and dx written
// once (37 us, 5.4 TB/s, and 4.6 us for the sums of 512 work-groups' 17 MB); a copy of 4 GiB runs at 4.7 TB/s. A row stays in
// registers between its statistics and its results. All sums are fp32; the variance is taken of the differences from the
// mean, which keeps its digits where the mean is large against the deviation.
#include "rows.h"

namespace kq {

// gamma (1 where there is none) and beta (0) of the columns of piece c
template <bool BF>
__device__ __forceinline__ void norm_weights(const void* p, int64_t col, int64_t cols, float none, float (&v)[row_chunk<BF>()]) {
    if (p && col < cols) row_load<BF>(p, col, cols - col, v);
    else
#pragma unroll
        for (int e = 0; e < row_chunk<BF>(); e++) v[e] = none;
}

struct NormArgs {
    const void *X, *dY, *gamma, *beta;
    int64_t ldx, lddy, n, d;
    float eps;
    int layer;               // the mean is taken off
    void *Y;                 // or dX
    int64_t ldy;
    float *mean, *rstd;
    float *part;             // backward: rows of sums of dgamma, then of dbeta
};
// floats of a row of sums, and of its dgamma half: whole pieces of 8 columns
__host__ __device__ inline int64_t norm_part_half(int64_t d) { return (d + 7) / 8 * 8; }
__host__ __device__ inline int64_t norm_part_row(int64_t d) { return 2 * norm_part_half(d); }

// A row's sum is taken at 2^-21 of its size, which 2^20 finite values cannot pass the largest number at: a power of two in a fused multiply-add
// changes neither the bits nor the cost of a plain sum (below 2^-81 values lose digits, 2^-129 of the mean at most).
constexpr float NORM_SCALE = 0x1p-21f;
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) < __builtin_inff(); }
// The mean from that sum; of values next to the largest number rounding may lead past it.
__device__ __forceinline__ float norm_mean(float s, float width) {
    const float m = s / (width * NORM_SCALE);
    return is_finite(s) ? fminf(fmaxf(m, -__FLT_MAX__), __FLT_MAX__) : m;
}
// 1 / deviation from the sums q of the squares and of the differences from m, a first mean (0 for rms). The sum of the differences
// is what rounding left of the mean: it corrects m, and its square comes off the variance. A row of one value then has that value
// as its mean, where one ulp beside it would come out times up to 1 / sqrt(eps). Finite values whose differences are not (their squares
// then are infinite, and not NaN as those of a row with an infinity) leave m as it is.
__device__ __forceinline__ float norm_rstd(float& m, const float (&q)[2], float width, const NormArgs& g) {
    float var = q[0] / width;
    if (g.layer) {
        const float rest = q[1] / width;
        if (is_finite(rest) || var != __builtin_inff()) {
            m += rest;
            var = __builtin_fmaf(-rest, rest, var);      // infinite where the squares are
            if (var < 0.0f) var = 0.0f;
        }
    }
    return 1.0f / sqrtf(var + g.eps);
}
// What a value's difference is taken from: a row of r = 0 has h = 0, also where the difference is not finite.
__device__ __forceinline__ float norm_from(float m, float rs) { return rs == 0.0f ? 0.0f : m; }

template <bool BF, int T, int CH>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_forward_kernel(NormArgs g) {
    constexpr int V = row_chunk<BF>();
    __shared__ float sm[32];
    const RowAt<T> at;
    const float width = (float)g.d;
    for (int64_t r = at.first; r < g.n; r += at.step) {
        RowRegs<BF, T, CH> x;
        x.load(g.X, r * g.ldx, g.d, at.lane);
        float m = 0.0f;
        if (g.layer) {
            float s[1] = {0.0f};
            x.each([&](int, float v) { s[0] = __builtin_fmaf(v, NORM_SCALE, s[0]); });
            row_sum<T>(s, sm);
            m = norm_mean(s[0], width);
        }
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int64_t col = ((int64_t)c * T + at.lane) * V;
            float v[V];
            x.get(c, v);
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float t = col + e < g.d ? v[e] - m : 0.0f;
                q[0] += t * t;
                q[1] += t;
            }
        }
        row_sum<T>(q, sm);
        const float rs = norm_rstd(m, q, width, g);
        if (at.lane == 0) {
            if (g.mean) g.mean[r] = m;
            if (g.rstd) g.rstd[r] = rs;
        }
        m = norm_from(m, rs);
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int64_t col = ((int64_t)c * T + at.lane) * V;
            if (col >= g.d) continue;
            float v[V], w[V], b[V];
            x.get(c, v);
            norm_weights<BF>(g.gamma, col, g.d, 1.0f, w);
            norm_weights<BF>(g.beta, col, g.d, 0.0f, b);
#pragma unroll
            for (int e = 0; e < V; e++) v[e] = (v[e] - m) * rs * w[e] + b[e];
            store_run<V>(g.Y, BF ? KQ_BF16 : KQ_F32, r * g.ldy + col, v, g.d - col);
        }
    }
}

// Rows that the registers do not hold: read three times, the last two mostly from a cache (2048 x 28672 fp32: 136 us).
template <bool BF>
__global__ __launch_bounds__(1024) void norm_forward_long_kernel(NormArgs g) {
    constexpr int V = row_chunk<BF>();
    __shared__ float sm[32];
    const float width = (float)g.d;
    for (int64_t r = blockIdx.x; r < g.n; r += gridDim.x) {
        auto all = [&](auto&& f) {
            for (int64_t col = (int64_t)threadIdx.x * V; col < g.d; col += 1024 * V) {
                float v[V];
                row_load<BF>(g.X, r * g.ldx + col, g.d - col, v);
                f(col, v);
            }
        };
        float m = 0.0f;
        if (g.layer) {
            float s[1] = {0.0f};
            all([&](int64_t, float (&v)[V]) {
                for (int e = 0; e < V; e++) s[0] = __builtin_fmaf(v[e], NORM_SCALE, s[0]);
            });
            row_sum<1024>(s, sm);
            m = norm_mean(s[0], width);
        }
        float q[2] = {0.0f, 0.0f};
        all([&](int64_t col, float (&v)[V]) {
            for (int e = 0; e < V; e++) {
                const float t = col + e < g.d ? v[e] - m : 0.0f;
                q[0] += t * t;
                q[1] += t;
            }
        });
        row_sum<1024>(q, sm);
        const float rs = norm_rstd(m, q, width, g);
        if (threadIdx.x == 0) {
            if (g.mean) g.mean[r] = m;
            if (g.rstd) g.rstd[r] = rs;
        }
        m = norm_from(m, rs);
        all([&](int64_t col, float (&v)[V]) {
            float w[V], b[V];
            norm_weights<BF>(g.gamma, col, g.d, 1.0f, w);
            norm_weights<BF>(g.beta, col, g.d, 0.0f, b);
            for (int e = 0; e < V; e++) v[e] = (v[e] - m) * rs * w[e] + b[e];
            store_run<V>(g.Y, BF ? KQ_BF16 : KQ_F32, r * g.ldy + col, v, g.d - col);
        });
    }
}

// dX of a work-group's rows and its part of dgamma and dbeta, which stay in registers over its rows. The next row's loads are
// in flight while one is reduced and written.
template <bool BF, int T, int CH>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_backward_kernel(NormArgs g) {
    constexpr int V = row_chunk<BF>(), PER = T < 256 ? 256 / T : 1;
    __shared__ float sm[32];
    const RowAt<T> at;
    const float inv = 1.0f / (float)g.d;
    RowRegs<BF, T, CH> w;
    w.load_or(g.gamma, g.d, at.lane, BF ? 0x3F803F80u : 0x3F800000u);
    float dg[CH][V], db[CH][V];
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
        for (int e = 0; e < V; e++) dg[c][e] = db[c][e] = 0.0f;
    struct Row {
        RowRegs<BF, T, CH> x, y;
        float m, rs;
    };
    auto fetch = [&](Row& row, int64_t r) {
        row.x.load(g.X, r * g.ldx, g.d, at.lane);
        row.y.load(g.dY, r * g.lddy, g.d, at.lane);
        row.m = g.layer ? g.mean[r] : 0.0f;
        row.rs = g.rstd[r];
    };
    constexpr bool AHEAD = CH * V <= 24;      // with more the second row does not fit in registers
    Row row, next;
    if (AHEAD && at.first < g.n) fetch(row, at.first);
    for (int64_t r = at.first; r < g.n; r += at.step) {
        if (!AHEAD) fetch(row, r);
        else if (r + at.step < g.n) fetch(next, r + at.step);
        const float rs = row.rs, m = norm_from(row.m, rs);
        float s[2] = {0.0f, 0.0f};       // of g h and of g
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int64_t col = ((int64_t)c * T + at.lane) * V;
            float v[V], dy[V], u[V];
            row.x.get(c, v);
            row.y.get(c, dy);
            w.get(c, u);
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float h = col + e < g.d ? (v[e] - m) * rs : 0.0f, t = dy[e] * u[e];
                s[0] += t * h;
                s[1] += t;
                dg[c][e] += dy[e] * h;
                db[c][e] += dy[e];
            }
        }
        if (g.Y) {
            row_sum<T>(s, sm);
            const float c1 = s[0] * inv, c0 = g.layer ? s[1] * inv : 0.0f;
#pragma unroll
            for (int c = 0; c < CH; c++) {
                const int64_t col = ((int64_t)c * T + at.lane) * V;
                if (col >= g.d) continue;
                float v[V], dy[V], u[V];
                row.x.get(c, v);
                row.y.get(c, dy);
                w.get(c, u);
#pragma unroll
                for (int e = 0; e < V; e++) v[e] = rs * (dy[e] * u[e] - c0 - (v[e] - m) * rs * c1);
                store_run<V>(g.Y, BF ? KQ_BF16 : KQ_F32, r * g.ldy + col, v, g.d - col);
            }
        }
        if (AHEAD) row = next;
    }
    if (!g.part) return;
    if constexpr (PER > 1) {
        // the work-group's rows are those of its wavefronts: added in order, the last one writes
        __shared__ float both[2][T * CH * V];
        const int mine = (int)threadIdx.x / T;
        for (int k = 0; k < PER; k++) {
            if (mine == k)
#pragma unroll
                for (int c = 0; c < CH; c++)
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        float &a = both[0][(c * V + e) * T + at.lane], &b = both[1][(c * V + e) * T + at.lane];
                        a = dg[c][e] = k ? a + dg[c][e] : dg[c][e];
                        b = db[c][e] = k ? b + db[c][e] : db[c][e];
                    }
            __syncthreads();
        }
        if (mine != PER - 1) return;
    }
    float* p = g.part + blockIdx.x * norm_part_row(g.d);
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int64_t col = ((int64_t)c * T + at.lane) * V;
        if (col >= g.d) continue;        // rows of sums are padded to whole pieces
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            *reinterpret_cast<float4*>(p + col + e) = make_float4(dg[c][e], dg[c][e + 1], dg[c][e + 2], dg[c][e + 3]);
            *reinterpret_cast<float4*>(p + norm_part_half(g.d) + col + e) = make_float4(db[c][e], db[c][e + 1], db[c][e + 2], db[c][e + 3]);
        }
    }
}

// dX of rows that the registers do not hold: read twice (2048 x 28672 fp32: 275 us with the weights' gradients, 181 without).
template <bool BF>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(NormArgs g) {
    constexpr int V = row_chunk<BF>();
    __shared__ float sm[32];
    const float inv = 1.0f / (float)g.d;
    for (int64_t r = blockIdx.x; r < g.n; r += gridDim.x) {
        const float rs = g.rstd[r];
        float m = g.layer ? g.mean[r] : 0.0f;
        auto all = [&](auto&& f) {
            for (int64_t col = (int64_t)threadIdx.x * V; col < g.d; col += 1024 * V) {
                float h[V], t[V], w[V];
                row_load<BF>(g.X, r * g.ldx + col, g.d - col, h);
                row_load<BF>(g.dY, r * g.lddy + col, g.d - col, t);
                norm_weights<BF>(g.gamma, col, g.d, 1.0f, w);
                for (int e = 0; e < V; e++) {
                    h[e] = col + e < g.d ? (h[e] - m) * rs : 0.0f;
                    t[e] *= w[e];
                }
                f(col, h, t);
            }
        };
        float s[2] = {0.0f, 0.0f};
        all([&](int64_t, float (&h)[V], float (&t)[V]) {
            for (int e = 0; e < V; e++) {
                s[0] += t[e] * h[e];
                s[1] += t[e];
            }
        });
        row_sum<1024>(s, sm);
        // norm_from here and not before the first loop, whose loads would wait for r (2048 x 40000 bf16: 132 -> 135 us)
        m = norm_from(m, rs);
        const float c1 = g.layer && rs == 0.0f ? 0.0f : s[0] * inv, c0 = g.layer ? s[1] * inv : 0.0f;
        all([&](int64_t col, float (&h)[V], float (&t)[V]) {
            for (int e = 0; e < V; e++) t[e] = rs * (t[e] - c0 - h[e] * c1);
            store_run<V>(g.Y, BF ? KQ_BF16 : KQ_F32, r * g.ldy + col, t, g.d - col);
        });
    }
}

// dgamma and dbeta of rows that the registers do not hold: a work-group's four wavefronts take its rows in turn, 64 pieces of
// columns wide, and write a row of sums each.
template <bool BF>
__global__ __launch_bounds__(256) void norm_weights_long_kernel(NormArgs g) {
    constexpr int V = row_chunk<BF>();
    const int64_t col = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * V, mine = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6);
    if (col >= g.d) return;
    float dg[V], db[V];
    for (int e = 0; e < V; e++) dg[e] = db[e] = 0.0f;
    for (int64_t r = mine; r < g.n; r += (int64_t)gridDim.y * 4) {
        const float rs = g.rstd[r], mean = g.layer ? g.mean[r] : 0.0f;
        float v[V], dy[V];
        row_load<BF>(g.X, r * g.ldx + col, g.d - col, v);
        row_load<BF>(g.dY, r * g.lddy + col, g.d - col, dy);
        const float m = norm_from(mean, rs);
        for (int e = 0; e < V; e++) {
            dg[e] += dy[e] * ((v[e] - m) * rs);
            db[e] += dy[e];
        }
    }
    float* p = g.part + mine * norm_part_row(g.d) + col;
    for (int e = 0; e < V; e++) {
        p[e] = dg[e];
        p[norm_part_half(g.d) + e] = db[e];
    }
}

// The rows of sums added: 32 columns a work-group, 8 lanes of four columns by 32 lanes of rows r, r + 32, .., whose sums are added in
// lane order.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* part, int64_t rows, int64_t d, void* dgamma, void* dbeta, int dt) {
    __shared__ float sm[32][36];
    const int64_t half = norm_part_half(d), step = norm_part_row(d);
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int64_t col = (int64_t)blockIdx.x * 32 + 4 * x;       // of half, a multiple of 8
    void* out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    float4 s = make_float4(0, 0, 0, 0);
    if (col < half) {
        const float* p = part + blockIdx.y * half + col;
#pragma unroll 8
        for (int64_t r = y; r < rows; r += 32) {
            const float4 v = *reinterpret_cast<const float4*>(p + r * step);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
    }
    *reinterpret_cast<float4*>(&sm[y][4 * x]) = s;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    float t = sm[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < 32; k++) t += sm[k][threadIdx.x];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    if (c >= d) return;
    if (dt == KQ_BF16) static_cast<uint16_t*>(out)[c] = to_bf16(t);
    else static_cast<float*>(out)[c] = t;
}

// f(BF, T, CH, G) for the backward pass over rows of `cols` values, on G work-groups at most (each leaves a row of sums); CH = 0 as
// for with_rows. From the same kind of sweep: a row's sums and the row ahead take registers too, so there are fewer pieces a
// thread (8192 x 8192 bf16: 80 us on 512 threads with the row ahead, 94 without room for it, 98 on 1024; 4096 x 13824: 79, and 196
// on 1024, which spill).
template <typename F>
kq_status with_grad_rows(bool bf, int64_t cols, F&& f) {
    const int64_t pieces = (cols + (bf ? 7 : 3)) / (bf ? 8 : 4);
    auto go = [&](auto t, auto ch, auto g) { return bf ? f(std::true_type{}, t, ch, g) : f(std::false_type{}, t, ch, g); };
#define KQ_ROWS(T, CH, G) go(std::integral_constant<int, T>{}, std::integral_constant<int, CH>{}, std::integral_constant<int, G>{})
    if (pieces <= 64) return KQ_ROWS(64, 1, 512);
    if (pieces <= 128) return KQ_ROWS(64, 2, 512);
    if (pieces <= 256) return KQ_ROWS(256, 1, 1024);
    if (pieces <= 512) return KQ_ROWS(512, 1, 512);
    if (pieces <= 768) return KQ_ROWS(256, 3, 512);
    if (pieces <= 1536) return KQ_ROWS(512, 3, 256);
    if (pieces <= 2048) return KQ_ROWS(512, 4, 256);
    // of bf16 their sums alone would fill the registers
    if (pieces <= 4096 && !bf)
        return f(std::false_type{}, std::integral_constant<int, 512>{}, std::integral_constant<int, 8>{}, std::integral_constant<int, 256>{});
    return KQ_ROWS(1024, 0, 256);
#undef KQ_ROWS
}
// rows of sums
static int64_t norm_parts(int64_t n, int64_t d, bool bf) {
    int64_t parts = 0;
    with_grad_rows(bf, d, [&](auto, auto t, auto ch, auto most) {
        constexpr int T = decltype(t)::value;
        parts = decltype(ch)::value == 0 ? 4 * (n < 64 ? (n + 3) / 4 : 16)
                                         : (int64_t)row_groups<T>(n, decltype(most)::value);
        return KQ_OK;
    });
    return parts;
}

struct NormMatrix {
    const void* p;
    int64_t ld;
    const char* what;
};
static kq_status norm_check(const char* who, kq_dtype dt, const NormMatrix& m, int64_t n, int64_t d) {
    if (!m.p) return fail(KQ_EINVAL, "%s: null %s", who, m.what);
    if (m.ld < d) return fail(KQ_ESHAPE, "%s: leading dimension of %s too small", who, m.what);
    if (!aligned16(m.p) || m.ld % (dt == KQ_BF16 ? 8 : 4))
        return fail(KQ_EINVAL, "%s: rows of %s must be 16-byte aligned", who, m.what);
    if (m.ld > TL_LD_MAX / 4 || n > TL_ROWS_MAX) return fail(KQ_ESHAPE, "%s: %s too large", who, m.what);
    return KQ_OK;
}
static kq_status norm_args(const char* who, kq_dtype dt, int64_t n, int64_t d, kq_norm kind, const void* gamma, const void* beta) {
    if (n < 0 || d <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (kind != KQ_NORM_LAYER && kind != KQ_NORM_RMS) return fail(KQ_EINVAL, "%s: bad kind", who);
    if (!aligned16(gamma) || !aligned16(beta)) return fail(KQ_EINVAL, "%s: gamma and beta must be 16-byte aligned", who);
    return KQ_OK;
}
static bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace kq

using namespace kq;

size_t norm_backward_ws(int64_t d, int64_t n, kq_dtype dt) {
    if (n <= 0 || d <= 0) return 0;
    return sizeof(float) * (size_t)(norm_part_row(d) * norm_parts(n, d, dt == KQ_BF16));
}

extern "C" kq_status kq_norm_forward(const void* X, int64_t ldx, const void* gamma, const void* beta, kq_dtype dt, int64_t n,
                                     int64_t d, kq_norm kind, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                                     kq_stream stream) {
    const char* who = "kq_norm_forward";
    KQ_TRY(norm_args(who, dt, n, d, kind, gamma, beta));
    if (!(eps > 0.0f) || !(eps <= 1.0f)) return fail(KQ_EINVAL, "%s: eps must lie in (0, 1]", who);
    if (n == 0) return KQ_OK;
    KQ_TRY(norm_check(who, dt, NormMatrix{X, ldx, "X"}, n, d));
    KQ_TRY(norm_check(who, dt, NormMatrix{Y, ldy, "Y"}, n, d));
    if (!aligned4(mean) || !aligned4(rstd)) return fail(KQ_EINVAL, "%s: mean and rstd must be aligned to 4 bytes", who);
    NormArgs g{};
    g.X = X; g.ldx = ldx; g.gamma = gamma; g.beta = beta; g.n = n; g.d = d; g.eps = eps; g.layer = kind == KQ_NORM_LAYER;
    g.Y = Y; g.ldy = ldy; g.mean = mean; g.rstd = rstd;
    return with_rows(dt == KQ_BF16, d, [&](auto bf, auto t, auto ch) {
        constexpr bool BF = decltype(bf)::value;
        constexpr int T = decltype(t)::value, CH = decltype(ch)::value;
        if constexpr (CH == 0)
            hipLaunchKernelGGL((norm_forward_long_kernel<BF>), dim3(row_groups<1024>(n)), dim3(1024), 0, hs(stream), g);
        else
            hipLaunchKernelGGL((norm_forward_kernel<BF, T, CH>), dim3(row_groups<T>(n)), dim3(T < 256 ? 256 : T), 0, hs(stream), g);
        return check_launch(who);
    });
}

extern "C" kq_status kq_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* gamma, const float* mean,
                                      const float* rstd, kq_dtype dt, int64_t n, int64_t d, kq_norm kind, void* dX, int64_t lddx,
                                      void* dgamma, void* dbeta, void* ws, size_t ws_bytes, kq_stream stream) {
    const char* who = "kq_norm_backward";
    KQ_TRY(norm_args(who, dt, n, d, kind, gamma, nullptr));
    if (!aligned4(dgamma) || !aligned4(dbeta)) return fail(KQ_EINVAL, "%s: dgamma and dbeta must be aligned to 4 bytes", who);
    if (n > 0) {
        KQ_TRY(norm_check(who, dt, NormMatrix{dY, lddy, "dY"}, n, d));
        KQ_TRY(norm_check(who, dt, NormMatrix{X, ldx, "X"}, n, d));
        if (dX) KQ_TRY(norm_check(who, dt, NormMatrix{dX, lddx, "dX"}, n, d));
        if (!rstd || (kind == KQ_NORM_LAYER && !mean)) return fail(KQ_EINVAL, "%s: null statistics", who);
        if (!aligned4(mean) || !aligned4(rstd)) return fail(KQ_EINVAL, "%s: mean and rstd must be aligned to 4 bytes", who);
    }
    const bool weights = dgamma || dbeta;
    const int64_t parts = n > 0 ? norm_parts(n, d, dt == KQ_BF16) : 0;
    if (weights && n > 0 && (!ws || !aligned16(ws) || ws_bytes < sizeof(float) * (size_t)(norm_part_row(d) * parts)))
        return fail(KQ_EWORKSPACE, "%s: workspace too small or not aligned to 16 bytes", who);
    NormArgs g{};
    g.X = X; g.ldx = ldx; g.dY = dY; g.lddy = lddy; g.gamma = gamma; g.n = n; g.d = d; g.layer = kind == KQ_NORM_LAYER;
    g.Y = dX; g.ldy = lddx; g.mean = const_cast<float*>(mean); g.rstd = const_cast<float*>(rstd);
    g.part = weights ? static_cast<float*>(ws) : nullptr;
    const hipStream_t st = hs(stream);
    if (n > 0 && (dX || weights))
        KQ_TRY(with_grad_rows(dt == KQ_BF16, d, [&](auto bf, auto t, auto ch, auto most) {
            constexpr bool BF = decltype(bf)::value;
            constexpr int T = decltype(t)::value, CH = decltype(ch)::value;
            if constexpr (CH == 0) {
                // the weights' sums first: dX may overwrite what they read
                constexpr int64_t wide = 64 * row_chunk<BF>();
                if (weights)
                    hipLaunchKernelGGL((norm_weights_long_kernel<BF>), dim3((unsigned)((d + wide - 1) / wide), (unsigned)(parts / 4)),
                                       dim3(256), 0, st, g);
                KQ_TRY(check_launch(who));
                if (dX) hipLaunchKernelGGL((norm_backward_long_kernel<BF>), dim3(row_groups<1024>(n)), dim3(1024), 0, st, g);
            } else {
                hipLaunchKernelGGL((norm_backward_kernel<BF, T, CH>), dim3(row_groups<T>(n, decltype(most)::value)), dim3(T < 256 ? 256 : T), 0, st, g);
            }
            return check_launch(who);
        }));
    if (!weights) return KQ_OK;
    hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((d + 31) / 32), 2), dim3(256), 0, st, g.part, parts, d, dgamma, dbeta, (int)dt);
    return check_launch(who);
}
