// norm.cuh -- the root-mean-square norm with the residual's addition (spec_rms_norm), and with
// its output in 8 bits and one scale per row (spec_rms_norm_fp8).
//
//   y = x + r,   n = y g / sqrt(mean(y^2) + eps)
//
// A row is read once and held in registers: G threads take it in 16-byte vectors, keep y in
// fp32 (the sum is not rounded before the norm; only the copy of y that is written back is),
// and meet once, for the sum of squares and, in the 8-bit form, the largest |y g| -- the row's
// factor 1/sqrt(..) is positive, so the row's largest |n| is that factor times it, and one
// reduction serves both.  The scale is max|n| / 448 (at least 2^-126, so that its reciprocal is
// finite and a row of zeros needs no case of its own); codes are e4m3, rounded to nearest.  The factor
// and the scale's reciprocal are one fp32 product a value: a division a value would cost an issue-bound
// row its time, and moves no code except where n / scale lies within a few 2^-24 of the middle between
// two (6140 of 1.6 10^9 codes are the farther one; with n / scale divided in fp32, 12743).
// Bound by HBM: each input and output element crosses it once.
#pragma once

#include <cstdint>

#include "device_common.cuh"

namespace specverify {

struct NormParams {
    const void* x;         // [rows, d]
    const void* residual;  // [rows, d] or nullptr
    const void* gain;      // [d]
    void* out;             // [rows, d] in the input's type, or e4m3 codes
    void* out_residual;    // [rows, d]: y, or nullptr
    float* out_scale;      // [rows] (8-bit form)
    int rows, d;
    float eps;
};

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// Two e4m3 codes of (lo, hi), rounded to nearest even, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

// Two bf16 of (lo, hi), rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t c;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(c) : "f"(hi), "f"(lo));
    return c;
}

__device__ __forceinline__ uint4 load_once16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// The kVec values g[head + v kVec ..] of an array of d values on a 16-byte boundary, 0 < head < kVec,
// from the two aligned vectors that hold them (head is the row's, so the choice below is uniform);
// by single loads where the second would reach past the array.
template <class ET>
__device__ __forceinline__ uint4 load_shifted(const typename ET::storage* g, int head, int v, int d) {
    if ((v + 2) * ET::kVec > d) return ET::load_vec_unaligned(g + head + v * ET::kVec);
    const uint4* a = reinterpret_cast<const uint4*>(g) + v;
    const uint4 lo = __ldg(a), hi = __ldg(a + 1);
    uint32_t w[5];
    switch (head * static_cast<int>(sizeof(typename ET::storage)) / 4) {
        case 0: w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w; w[4] = hi.x; break;
        case 1: w[0] = lo.y; w[1] = lo.z; w[2] = lo.w; w[3] = hi.x; w[4] = hi.y; break;
        case 2: w[0] = lo.z; w[1] = lo.w; w[2] = hi.x; w[3] = hi.y; w[4] = hi.z; break;
        default: w[0] = lo.w; w[1] = hi.x; w[2] = hi.y; w[3] = hi.z; w[4] = hi.w; break;
    }
    if (sizeof(typename ET::storage) == 2 && (head & 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Stores of one 16-byte vector's worth of values, or of one value, in a type.
template <class ET>
struct NormOut;

template <>
struct NormOut<Bf16Elem> {
    __device__ __forceinline__ static void vec(uint16_t* p, const float (&f)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]),
                                                  bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
    }
    __device__ __forceinline__ static void one(uint16_t* p, float f) { *p = static_cast<uint16_t>(bf16_pair(f, 0.0f)); }
    __device__ __forceinline__ static void codes(uint8_t* p, const float (&f)[8]) {
        *reinterpret_cast<uint2*>(p) = make_uint2(e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16),
                                                  e4m3_pair(f[4], f[5]) | (e4m3_pair(f[6], f[7]) << 16));
    }
};

template <>
struct NormOut<F32Elem> {
    __device__ __forceinline__ static void vec(float* p, const float (&f)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
    __device__ __forceinline__ static void one(float* p, float f) { *p = f; }
    __device__ __forceinline__ static void codes(uint8_t* p, const float (&f)[4]) {
        *reinterpret_cast<uint32_t*>(p) = e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16);
    }
};

// The values of a vector in pairs, and back.
template <class ET>
__device__ __forceinline__ void widen_pairs(const uint4& v, uint64_t (&f)[ET::kVec / 2]) {
    float e[ET::kVec];
    ET::widen(v, e);
#pragma unroll
    for (int i = 0; i < ET::kVec / 2; ++i) f[i] = pack2(e[2 * i], e[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void unpack_pairs(const uint64_t (&v)[N], float (&f)[2 * N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
}

// max(a, |b|, |c|), NaN where one of them is.
__device__ __forceinline__ float max_magnitude(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Sums, products and the scaling go two values an instruction, and a pair's magnitudes into the
// largest in one: rows of bf16 to e4m3 without a residual are bound by issue otherwise (47337 x 5760:
// 181 us value by value, 159 so).  A block that takes several rows and loads the next while it norms
// one is slower than blocks of one row each (245): the SM's other blocks hide a row's latency already.
//
// One block per row, or kLanes (8, 16, 32) lanes of a warp per row, at most NV 16-byte vectors (kVec
// values) a thread.  kWhole: every row is whole vectors on 16-byte
// boundaries.  Otherwise (an odd d) a row has up to kVec - 1 values before its first boundary and
// after its last whole vector; they are one value each for the threads 0.. and 16.., and only the
// gain, which does not move with the row's boundary, is shifted into place (two loads from L1).  x, the
// residual and both outputs share a row's offset, so their boundaries are the same.
template <class ET, bool kFp8, int kLanes, int NV, int kMaxThreads, bool kWhole>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_kernel(NormParams p) {
    using S = typename ET::storage;
    constexpr int kVec = ET::kVec;
    static_assert(kWhole || kLanes == 0 || kLanes == 32, "the values outside the vectors take 24 threads");
    const int G = kLanes ? kLanes : static_cast<int>(blockDim.x);
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    int row = static_cast<int>(blockIdx.x), t = static_cast<int>(threadIdx.x);
    bool live = true;  // (a warp may hold rows behind the last: its lanes go along and write nothing)
    if constexpr (kLanes > 0) {
        row = static_cast<int>(blockIdx.x) * (kMaxThreads / kLanes) + t / kLanes;
        t %= kLanes;
        live = row < p.rows;
        row = min(row, p.rows - 1);
    }
    const long long at = static_cast<long long>(row) * p.d;
    const S* x = static_cast<const S*>(p.x) + at;
    const S* r = p.residual ? static_cast<const S*>(p.residual) + at : nullptr;
    const S* g = static_cast<const S*>(p.gain);
    int head = 0, nvec = p.d / kVec;
    int odd = -1;  // this thread's value outside the vectors
    if (!kWhole) {
        head = static_cast<int>((kVec - at % kVec) % kVec);
        if (head > p.d) head = p.d;
        nvec = (p.d - head) / kVec;
        const int tail0 = head + nvec * kVec;
        if (t < head) odd = t;
        else if (t >= 16 && t - 16 < p.d - tail0) odd = tail0 + t - 16;
    }

    grid_dependency();
    uint64_t y[NV][kVec / 2];  // pairs of values
    float y_odd = 0.0f;
    {
        uint4 vx[NV], vr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = t + k * G;
            vx[k] = v < nvec ? load_once16(x + head + v * kVec) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (r) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = t + k * G;
                vr[k] = v < nvec ? load_once16(r + head + v * kVec) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (!kWhole && odd >= 0) {
            y_odd = ET::load1(x + odd);
            if (r) y_odd += ET::load1(r + odd);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            widen_pairs<ET>(vx[k], y[k]);
            if (r) {
                uint64_t f[kVec / 2];
                widen_pairs<ET>(vr[k], f);
#pragma unroll
                for (int e = 0; e < kVec / 2; ++e) y[k][e] = add2(y[k][e], f[e]);
            }
        }
    }

    // y's copy out, its squares, and y g (which replaces y)
    uint64_t squares = 0ull;
    float most = 0.0f;  // the largest |y g|, or NaN
    S* const out_y = p.out_residual ? static_cast<S*>(p.out_residual) + at : nullptr;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = t + k * G;
        uint64_t f[kVec / 2];
        uint4 vg = make_uint4(0u, 0u, 0u, 0u);
        if (v < nvec) {
            if (out_y && live) {
                float e[kVec];
                unpack_pairs(y[k], e);
                NormOut<ET>::vec(out_y + head + v * kVec, e);
            }
            vg = kWhole || head == 0 ? __ldg(reinterpret_cast<const uint4*>(g + v * kVec)) : load_shifted<ET>(g, head, v, p.d);
        }
        widen_pairs<ET>(vg, f);
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {
            squares = fma2(y[k][e], y[k][e], squares);
            y[k][e] = mul2(y[k][e], f[e]);
            if (kFp8) {
                float lo, hi;
                unpack2(y[k][e], lo, hi);
                most = max_magnitude(most, lo, hi);
            }
        }
    }
    float sum, sum_hi;
    unpack2(squares, sum, sum_hi);
    sum += sum_hi;
    if (!kWhole && odd >= 0) {
        if (out_y && live) NormOut<ET>::one(out_y + odd, y_odd);
        sum = fmaf(y_odd, y_odd, sum);
        y_odd *= ET::load1(g + odd);
        if (kFp8) most = max_magnitude(most, y_odd, y_odd);
    }
    uint32_t top = __float_as_uint(most) & 0x7FFFFFFFu;  // as bits: NaN sorts above infinity, so it is kept
    constexpr int kSpan = kLanes ? kLanes : 32;
#pragma unroll
    for (int off = kSpan / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (kFp8 && kSpan == 32) top = __reduce_max_sync(0xffffffffu, top);
    if (kFp8 && kSpan < 32) {
#pragma unroll
        for (int off = kSpan / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    }
    if (!kLanes) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = G >> 5;
        if (lane == 0) {
            s_sum[warp] = sum;
            if (kFp8) s_max[warp] = top;
        }
        __syncthreads();
        sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (kFp8) top = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
    }
    const float factor = rsqrtf(sum / static_cast<float>(p.d) + p.eps);
    float scaling = factor;
    if (kFp8) {
        float scale = __uint_as_float(top) * factor / kE4m3Max;
        scale = scale < kMinScale ? kMinScale : scale;  // (NaN stays)
        if (t == 0 && live) p.out_scale[row] = scale;
        const float inverse = 1.0f / scale;
        scaling = factor * inverse;
        if (!(scaling <= 3.0e38f)) {  // (a row of zeros, whose y times infinity would be NaN; and NaN)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < kVec / 2; ++e) y[k][e] = mul2(y[k][e], pack2(factor, factor));
            y_odd *= factor;
            scaling = inverse;
        }
    }
    const uint64_t scaling2 = pack2(scaling, scaling);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = t + k * G;
        if (v >= nvec || !live) continue;
        float n[kVec];
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) unpack2(mul2(y[k][e], scaling2), n[2 * e], n[2 * e + 1]);
        if (kFp8) NormOut<ET>::codes(static_cast<uint8_t*>(p.out) + at + head + v * kVec, n);
        else NormOut<ET>::vec(static_cast<S*>(p.out) + at + head + v * kVec, n);
    }
    if (!kWhole && odd >= 0 && live) {
        if (kFp8) static_cast<uint8_t*>(p.out)[at + odd] = static_cast<uint8_t>(e4m3_pair(y_odd * scaling, 0.0f));
        else NormOut<ET>::one(static_cast<S*>(p.out) + at + odd, y_odd * scaling);
    }
}

}  // namespace specverify
