// Rows held in registers, for operators that reduce over a row before they use it (i8.hip, norm.hip). Not part of the
// C ABI. T threads share a row, CH pieces of 16 bytes each (V values: 8 bf16 or 4 fp32): piece c of lane l holds
// columns (c T + l) V .., so that a load is one run of T * 16 bytes.
#pragma once

#include "tile.h"

namespace kq {

template <bool BF>
constexpr int row_chunk() { return BF ? 8 : 4; }

// the rows of this thread: rows first, first + step, ..
template <int T>
struct RowAt {
    int lane;
    int64_t first, step;
    __device__ __forceinline__ RowAt() {
        constexpr int PER = T < 256 ? 256 / T : 1;       // rows a work-group
        lane = PER > 1 ? (int)threadIdx.x % T : (int)threadIdx.x;
        first = (int64_t)blockIdx.x * PER + (PER > 1 ? (int)threadIdx.x / T : 0);
        step = (int64_t)gridDim.x * PER;
    }
};
template <int T>
unsigned row_groups(int64_t rows, int64_t most = 65536) {
    constexpr int PER = T < 256 ? 256 / T : 1;
    const int64_t n = (rows + PER - 1) / PER;
    return (unsigned)(n < most ? n : most);
}

template <bool BF>
__device__ __forceinline__ void row_unpack(const uint4& w, float (&v)[row_chunk<BF>()]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (BF) {
            v[2 * k] = __uint_as_float(u[k] << 16);
            v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        } else {
            v[k] = __uint_as_float(u[k]);
        }
    }
}

// One piece as it lies in memory, zeros behind the last of `left` values.
template <bool BF>
__device__ __forceinline__ uint4 row_piece(const void* X, int64_t off, int64_t left) {
    if (left >= row_chunk<BF>())
        return *reinterpret_cast<const uint4*>(static_cast<const char*>(X) + off * (BF ? 2 : 4));
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < row_chunk<BF>(); e++) {
        if (e >= left) continue;
        if constexpr (BF) u[e / 2] |= (uint32_t)static_cast<const uint16_t*>(X)[off + e] << (16 * (e % 2));
        else u[e] = static_cast<const uint32_t*>(X)[off + e];
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
template <bool BF>
__device__ __forceinline__ void row_load(const void* X, int64_t off, int64_t left, float (&v)[row_chunk<BF>()]) {
    row_unpack<BF>(row_piece<BF>(X, off, left), v);
}

template <bool BF, int T, int CH>
struct RowRegs {
    static constexpr int V = row_chunk<BF>();
    uint4 w[CH];
    __device__ __forceinline__ void load(const void* X, int64_t off, int64_t cols, int lane) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int64_t col = ((int64_t)c * T + lane) * V;
            w[c] = col < cols ? row_piece<BF>(X, off + col, cols - col) : make_uint4(0, 0, 0, 0);
        }
    }
    // the same for one row that all share, or `none` in every word where there is no row
    __device__ __forceinline__ void load_or(const void* P, int64_t cols, int lane, uint32_t none) {
        if (P) load(P, 0, cols, lane);
        else
#pragma unroll
            for (int c = 0; c < CH; c++) w[c] = make_uint4(none, none, none, none);
    }
    __device__ __forceinline__ void get(int c, float (&v)[V]) const { row_unpack<BF>(w[c], v); }
    // f(piece, value) for all values, zeros behind the last column among them
    template <typename F>
    __device__ __forceinline__ void each(F&& f) const {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            float v[V];
            get(c, v);
#pragma unroll
            for (int e = 0; e < V; e++) f(c, v[e]);
        }
    }
};

// Reductions over the T threads of a row, the result in all of them, in one order. sm: one word a wavefront and value, used by rows of
// several wavefronts (whose threads all come here together).
template <int T, int N, typename D, typename F>
__device__ __forceinline__ void row_reduce(D (&v)[N], D* sm, F&& f) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < N; k++) v[k] = f(v[k], __shfl_xor(v[k], d));
    if constexpr (T > 64) {
        constexpr int W = T / 64;
        __syncthreads();                 // the last reduction's words have been read
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < N; k++) sm[k * W + (threadIdx.x >> 6)] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; k++) {
            v[k] = sm[k * W];
            for (int w = 1; w < W; w++) v[k] = f(v[k], sm[k * W + w]);
        }
    }
}
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float* sm) {
    uint32_t a[1] = {v};
    row_reduce<T>(a, reinterpret_cast<uint32_t*>(sm), [](uint32_t x, uint32_t y) { return x > y ? x : y; });
    return a[0];
}
template <int T, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* sm) {
    row_reduce<T>(v, sm, [](float x, float y) { return x + y; });
}

// f(BF, T, CH) for rows of `cols` values, CH = 0 for rows that the registers of 512 threads do not hold. Chosen by a sweep of T and
// CH over widths of 512 to 13824 of both types (8192 or 4096 rows, MI355X): a wavefront a row as long as four pieces hold it, then 256
// threads, then 512; 1024 threads, of which a compute unit holds two rows, are slower (norm of 4096 x 11008 bf16: 37 us on 512 threads, 72
// on 1024; of 8192 x 5120: 33 on 256, 38 on 1024) but for the widest rows of bf16, whose 64 values a thread of 512 take too many registers
// (2048 x 28672: 69 us on 1024, 80 on 512).
template <typename F>
kq_status with_rows(bool bf, int64_t cols, F&& f) {
    const int64_t pieces = (cols + (bf ? 7 : 3)) / (bf ? 8 : 4);
    auto go = [&](auto t, auto ch) { return bf ? f(std::true_type{}, t, ch) : f(std::false_type{}, t, ch); };
#define KQ_ROWS(T, CH) go(std::integral_constant<int, T>{}, std::integral_constant<int, CH>{})
    if (pieces <= 64) return KQ_ROWS(64, 1);
    if (pieces <= 128) return KQ_ROWS(64, 2);
    if (pieces <= 256) return KQ_ROWS(64, 4);
    if (pieces <= 512) return KQ_ROWS(256, 2);
    if (pieces <= 768) return KQ_ROWS(256, 3);
    if (pieces <= 1024) return KQ_ROWS(256, 4);
    if (pieces <= 1536) return KQ_ROWS(512, 3);
    if (pieces <= 2048) return KQ_ROWS(512, 4);
    if (pieces <= 4096 && bf) return f(std::true_type{}, std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
    auto f32 = [&](auto ch) { return f(std::false_type{}, std::integral_constant<int, 512>{}, ch); };
    if (pieces <= 6 * 512) return f32(std::integral_constant<int, 6>{});
    if (pieces <= 8 * 512) return f32(std::integral_constant<int, 8>{});
    return KQ_ROWS(1024, 0);
#undef KQ_ROWS
}

}  // namespace kq
