// 8-bit integers with a scale for each row (KronQ review page, Limitations (3): the stored weights are multiplied at
// inference time; Goal: low-bit weights. Symmetric rounding, a scale for each token and each output channel): value =
// code * scale, codes -127 .. 127.
//
// Quantisation of a row with largest magnitude a: scale = a / 127 and m = 127 / a, both rounded to fp32; a code is the
// whole number nearest to the exact product x m, ties to the even one. x m + 1.5 * 2^23 in one fused
// multiply-add is that number in the low bits of the sum: fp32 values of that size are the whole numbers, so the sum's one rounding is
// the one wanted, where a rounded product could land on a half that the exact one misses. A row with a < 2^-119 (whose scale
// would be subnormal) has scale 0 and zero codes; one that holds an infinity or NaN has scale NaN and zero codes,
// so that it reads as NaN instead of as some finite value.
#include "group.h"
#include "rows.h"

namespace kq {

// One row a work-group (a wavefront for short rows) at a time, held in registers between the maximum and the codes: each value
// is read once, and HBM bounds the pass. MI355X: 8192 x 4096 bf16 16.9 us, 6.0 TB/s (101 MB, less than the last-level cache holds);
// 5120 x 13824 fp32 85 us, 4.2 TB/s, where a copy of 4 GiB runs at 4.7.
template <bool BF, int T, int CH>
__global__ __launch_bounds__(T < 256 ? 256 : T) void i8_quantize_kernel(const void* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
                                                                        int8_t* __restrict__ codes, int64_t ldc,
                                                                        float* __restrict__ scales) {
    constexpr int V = row_chunk<BF>();
    __shared__ float sm[16];
    const RowAt<T> at;
    for (int64_t r = at.first; r < rows; r += at.step) {
        RowRegs<BF, T, CH> x;
        x.load(X, r * ldx, cols, at.lane);
        // magnitudes order like their bit patterns, infinities and NaN last
        uint32_t top = 0;
        x.each([&](int, float v) {
            const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        });
        top = row_max<T>(top, sm);
        const bool bad = top >= 0x7F800000u, none = top < 0x04000000u;      // 2^-119
        const float a = __uint_as_float(top), m = bad || none ? 0.0f : 127.0f / a;
        if (at.lane == 0) scales[r] = bad ? __uint_as_float(0x7FC00000u) : none ? 0.0f : a / 127.0f;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int64_t col = ((int64_t)c * T + at.lane) * V;
            if (col >= cols) continue;
            float v[V];
            x.get(c, v);
            uint32_t w[V / 4];
#pragma unroll
            for (int k = 0; k < V / 4; k++) {
                uint32_t q[4];
#pragma unroll
                for (int e = 0; e < 4; e++) q[e] = __float_as_uint(__builtin_fmaf(v[4 * k + e], m, 12582912.0f));
                w[k] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[3], q[2], 0x0C0C0400u), __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u),
                                             0x05040100u);
                if (bad) w[k] = 0;       // NaN and infinity times 0
            }
            int8_t* p = codes + r * ldc + col;
            if (col + V <= cols) {
                if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t*>(p) = w[0];
            } else {
#pragma unroll
                for (int e = 0; e < V; e++)
                    if (col + e < cols) p[e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
            }
        }
    }
}

// Rows longer than the registers of a work-group hold: read twice, the second time mostly from a cache (2048 x 28672 fp32: 71 us for
// 294 MB, 4.1 TB/s).
template <bool BF>
__global__ __launch_bounds__(1024) void i8_quantize_long_kernel(const void* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
                                                                int8_t* __restrict__ codes, int64_t ldc, float* __restrict__ scales) {
    constexpr int V = row_chunk<BF>();
    __shared__ float sm[16];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        uint32_t top = 0;
        for (int64_t col = (int64_t)threadIdx.x * V; col < cols; col += 1024 * V) {
            float v[V];
            row_load<BF>(X, r * ldx + col, cols - col, v);
#pragma unroll
            for (int e = 0; e < V; e++) {
                const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
                top = b > top ? b : top;
            }
        }
        top = row_max<1024>(top, sm);
        const bool bad = top >= 0x7F800000u, none = top < 0x04000000u;
        const float a = __uint_as_float(top), m = bad || none ? 0.0f : 127.0f / a;
        if (threadIdx.x == 0) scales[r] = bad ? __uint_as_float(0x7FC00000u) : none ? 0.0f : a / 127.0f;
        for (int64_t col = (int64_t)threadIdx.x * V; col < cols; col += 1024 * V) {
            float v[V];
            row_load<BF>(X, r * ldx + col, cols - col, v);
#pragma unroll
            for (int e = 0; e < V; e++)
                if (col + e < cols)
                    codes[r * ldc + col + e] = bad ? (int8_t)0 : (int8_t)__float_as_uint(__builtin_fmaf(v[e], m, 12582912.0f));
        }
    }
}

// 16 bytes of output a lane, so that a wavefront's store is one run of 1 KiB; bound by HBM (8192 x 4096 bf16 17.2 us, 5.9 TB/s; 5120 x 13824
// fp32 68 us, 5.2 TB/s).
template <bool BF>
__global__ __launch_bounds__(256) void i8_dequantize_kernel(const int8_t* __restrict__ codes, int64_t ldc,
                                                            const float* __restrict__ scales, int64_t rows, int64_t cols,
                                                            void* __restrict__ Y, int64_t ldy) {
    constexpr int V = row_chunk<BF>();
    const int64_t per = (cols + V - 1) / V, total = rows * per;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += step) {
        const int64_t r = e / per, c = (e - r * per) * V;
        const int8_t* p = codes + r * ldc + c;       // the last piece of a row lies inside its 16 bytes
        const float s = scales[r];
        int32_t w[V / 4];
        if constexpr (BF) {
            const int2 q = *reinterpret_cast<const int2*>(p);
            w[0] = q.x; w[1] = q.y;
        } else {
            w[0] = *reinterpret_cast<const int32_t*>(p);
        }
        float v[V];
#pragma unroll
        for (int k = 0; k < V; k++) v[k] = (float)(int8_t)(w[k / 4] >> (8 * (k % 4))) * s;
        store_run<V>(Y, BF ? KQ_BF16 : KQ_F32, r * ldy + c, v, cols - c);
    }
}

struct I8Operand {
    const int8_t* c;
    int64_t ld;
    const float* s;
};

static kq_status i8_check(const char* who, const char* what, const I8Operand& m, int64_t rows, int64_t cols) {
    if (!m.c || !m.s) return fail(KQ_EINVAL, "%s: null %s", who, what);
    if (m.ld < cols) return fail(KQ_ESHAPE, "%s: leading dimension of %s too small", who, what);
    if (!aligned16(m.c) || m.ld % 16 || reinterpret_cast<uintptr_t>(m.s) % 4)
        return fail(KQ_EINVAL, "%s: rows of %s must be aligned to 16 bytes and scales to 4", who, what);
    if (m.ld > TL_LD_MAX || rows > TL_ROWS_MAX) return fail(KQ_ESHAPE, "%s: %s too large", who, what);
    return KQ_OK;
}

static kq_status i8_float_check(const char* who, const char* what, const void* p, kq_dtype dt, int64_t ld, int64_t cols) {
    if (!p) return fail(KQ_EINVAL, "%s: null %s", who, what);
    if (ld < cols) return fail(KQ_ESHAPE, "%s: leading dimension of %s too small", who, what);
    if (!aligned16(p) || ld % (dt == KQ_BF16 ? 8 : 4)) return fail(KQ_EINVAL, "%s: rows of %s must be 16-byte aligned", who, what);
    return KQ_OK;
}

// Products: int8 matrix cores on the tiles of tile.h, the scales in the epilogue. 8192 x 4096 x 11008 253 to 290 us by the box's clock, 2.5
// to 2.9 POP/s (the library's int8 product of these sizes 339 us); one token 9.0 us, 5.0 TB/s of weights.
// Sums of products of codes of up to 128 by magnitude stay below 2^31.
constexpr int64_t I8_WIDTH_MAX = (1 << 17) - 1;

template <bool GATED>
static TilePlan i8_plan(int64_t n, int64_t o, int64_t i) {
    return tile_plan<EL_I8, GATED ? TP_GATED : TP_PLAIN>(n, o, i);
}

template <bool GATED>
static kq_status i8_product(const char* who, const I8Operand& A, const I8Operand& B, const I8Operand& U, const int32_t* offsets,
                            int64_t experts, int64_t n, int64_t o, int64_t i, int act, void* Y, kq_dtype dt, int64_t ldy, void* ws,
                            size_t ws_bytes, hipStream_t st) {
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (act < KQ_ACT_SILU || act > KQ_ACT_RELU) return fail(KQ_EINVAL, "%s: bad activation", who);
    if (i > I8_WIDTH_MAX) return fail(KQ_ESHAPE, "%s: rows of more than %lld codes", who, (long long)I8_WIDTH_MAX);
    if (offsets) KQ_TRY(group_check(who, offsets, experts, n, o));
    else if (experts != 0) return fail(KQ_EINVAL, "%s: experts without offsets", who);
    if (n == 0) return KQ_OK;
    if (!tile_sizes_ok(n, o)) return fail(KQ_ESHAPE, "%s: result too large", who);
    const int64_t orows = offsets ? experts * o : o;
    KQ_TRY(i8_check(who, "tokens", A, n, i));
    KQ_TRY(i8_check(who, GATED ? "gate weights" : "weights", B, orows, i));
    if (GATED) KQ_TRY(i8_check(who, "up weights", U, orows, i));
    KQ_TRY(i8_float_check(who, "the output", Y, dt, ldy, o));
    const Group gr{offsets, (int)experts, (int)(n <= GROUP_ROWS_MAX ? n : 0), (int)o};
    if (offsets ? group_few<EL_I8>(n, experts) : few_tokens<EL_I8>(n, GATED ? 2 * o : o, i)) {
        FewArgs f{};
        f.n = n; f.o = o; f.K = i;
        f.A = reinterpret_cast<const char*>(A.c); f.lda = A.ld; f.fA = A.s;
        f.B = reinterpret_cast<const char*>(B.c); f.ldb = B.ld; f.fB = B.s;
        f.B2 = reinterpret_cast<const char*>(U.c); f.ldb2 = U.ld; f.fB2 = U.s;
        f.Y = Y; f.ldy = ldy; f.dt = dt; f.act = act;
        return offsets ? group_few_launch<EL_I8, GATED>(f, gr, st, who) : few_launch<EL_I8, GATED>(f, st, who);
    }
    constexpr int MODE = GATED ? TP_GATED : TP_PLAIN;
    TileArgs g{};
    g.M = n; g.N = o; g.K = i;
    g.A = reinterpret_cast<const char*>(A.c); g.lda = A.ld; g.fA = A.s;
    g.B = reinterpret_cast<const char*>(B.c); g.ldb = B.ld; g.fB = B.s;
    g.B2 = reinterpret_cast<const char*>(U.c); g.ldb2 = U.ld; g.fB2 = U.s;
    g.Y = Y; g.ldy = ldy; g.dt = dt; g.act = act; g.pairs = 1;
    if (offsets) return group_launch<EL_I8, MODE>(g, gr, ws, ws_bytes, st, who);
    const TilePlan plan = i8_plan<GATED>(n, o, i);
    if (plan.part && (!ws || !aligned16(ws) || ws_bytes < sizeof(float) * plan.part))
        return fail(KQ_EWORKSPACE, "%s: workspace too small or not aligned to 16 bytes", who);
    return tile_launch<EL_I8, MODE>(g, plan, 1, static_cast<float*>(ws), st, who);
}

}  // namespace kq

using namespace kq;

size_t i8_product_ws(int64_t o, int64_t i, int64_t n, bool gated, int64_t experts) {
    if (n <= 0 || o <= 0 || i <= 0 || !tile_sizes_ok(n, o) || experts < 0) return 0;
    if (experts) {
        if (experts > GROUP_MAX || n > GROUP_ROWS_MAX || group_few<EL_I8>(n, experts)) return 0;
        return gated ? group_ws<EL_I8, TP_GATED>(n, experts, o, i) : group_ws<EL_I8, TP_PLAIN>(n, experts, o, i);
    }
    if (few_tokens<EL_I8>(n, gated ? 2 * o : o, i)) return 0;
    return sizeof(float) * (gated ? i8_plan<true>(n, o, i) : i8_plan<false>(n, o, i)).part;
}

extern "C" kq_status kq_i8_quantize(const void* X, kq_dtype xdt, int64_t rows, int64_t cols, int64_t ldx, int8_t* codes,
                                    int64_t ldc, float* scales, kq_stream stream) {
    const char* who = "kq_i8_quantize";
    if (rows < 0 || cols <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (xdt != KQ_F32 && xdt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (rows == 0) return KQ_OK;
    KQ_TRY(i8_float_check(who, "X", X, xdt, ldx, cols));
    KQ_TRY(i8_check(who, "the output", I8Operand{codes, ldc, scales}, rows, cols));
    return with_rows(xdt == KQ_BF16, cols, [&](auto bf, auto t, auto ch) {
        constexpr bool BF = decltype(bf)::value;
        constexpr int T = decltype(t)::value, CH = decltype(ch)::value;
        if constexpr (CH == 0)
            hipLaunchKernelGGL((i8_quantize_long_kernel<BF>), dim3(row_groups<1024>(rows)), dim3(1024), 0, hs(stream), X, rows, cols,
                               ldx, codes, ldc, scales);
        else
            hipLaunchKernelGGL((i8_quantize_kernel<BF, T, CH>), dim3(row_groups<T>(rows)), dim3(T < 256 ? 256 : T), 0, hs(stream), X,
                               rows, cols, ldx, codes, ldc, scales);
        return check_launch(who);
    });
}

extern "C" kq_status kq_i8_dequantize(const int8_t* codes, int64_t ldc, const float* scales, int64_t rows, int64_t cols, void* Y,
                                      kq_dtype ydt, int64_t ldy, kq_stream stream) {
    const char* who = "kq_i8_dequantize";
    if (rows < 0 || cols <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (ydt != KQ_F32 && ydt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (rows == 0) return KQ_OK;
    KQ_TRY(i8_check(who, "the input", I8Operand{codes, ldc, scales}, rows, cols));
    KQ_TRY(i8_float_check(who, "Y", Y, ydt, ldy, cols));
    const int64_t v = ydt == KQ_BF16 ? 8 : 4, total = rows * ((cols + v - 1) / v);
    const unsigned grid = (unsigned)((total + 255) / 256 < 65536 ? (total + 255) / 256 : 65536);
    if (ydt == KQ_BF16)
        hipLaunchKernelGGL((i8_dequantize_kernel<true>), dim3(grid), dim3(256), 0, hs(stream), codes, ldc, scales, rows, cols, Y, ldy);
    else
        hipLaunchKernelGGL((i8_dequantize_kernel<false>), dim3(grid), dim3(256), 0, hs(stream), codes, ldc, scales, rows, cols, Y, ldy);
    return check_launch(who);
}

extern "C" kq_status kq_i8_gemm(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, const float* sB,
                                const int32_t* offsets, int64_t experts, int64_t n, int64_t o, int64_t i, void* Y, kq_dtype ydt,
                                int64_t ldy, void* ws, size_t ws_bytes, kq_stream stream) {
    return i8_product<false>("kq_i8_gemm", I8Operand{A, lda, sA}, I8Operand{B, ldb, sB}, I8Operand{}, offsets, experts, n, o, i, 0, Y,
                             ydt, ldy, ws, ws_bytes, hs(stream));
}

extern "C" kq_status kq_i8_gated(const int8_t* X, int64_t ldx, const float* sX, const int8_t* G, int64_t ldg, const float* sG,
                                 const int8_t* U, int64_t ldu, const float* sU, const int32_t* offsets, int64_t experts, int64_t n,
                                 int64_t o, int64_t i, kq_act act, void* H, kq_dtype hdt, int64_t ldh, void* ws, size_t ws_bytes,
                                 kq_stream stream) {
    return i8_product<true>("kq_i8_gated", I8Operand{X, ldx, sX}, I8Operand{G, ldg, sG}, I8Operand{U, ldu, sU}, offsets, experts, n, o,
                            i, act, H, hdt, ldh, ws, ws_bytes, hs(stream));
}
