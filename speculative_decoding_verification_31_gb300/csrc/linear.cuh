// linear.cuh -- the matrix product with bias, activation and residual in its epilogue
// (spec_linear), on the tensor cores:
//
//   out[m, n] = act(s_x[m] s_w[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
//
// x [rows, K] and w [N, K] row-major (both K-major), bf16 x bf16 or e4m3 x e4m3, accumulated in
// fp32 in TMEM.  The weight takes the MMA's M side (128 output channels a tile, one TMEM lane
// and one epilogue thread each) and the tokens its N side (BN = 16 .. 256 columns), so that one
// kernel serves a single token, where the call is a stream of the weight through shared memory,
// and a full batch, where it is bound by the tensor cores; bias and weight scale are one
// register a thread, and a warp's stores run along a row of the output.
//   warp 0     one thread issues the TMA loads of the weight's and the tokens' 128-byte K slices
//              into a ring of stages (128-byte swizzle);
//   warp 1     allocates TMEM (two accumulators of BN columns); one thread issues tcgen05.mma;
//   warps 2-   the epilogue (four or eight warps), from tcgen05.ld.
// With fewer tiles than SMs the K axis is split over the CTAs of a cluster: each leaves its
// fp32 partial tile in its shared memory, and after a cluster barrier CTA r adds the columns
// of its share over the CTAs in rank order (so the result does not depend on timing) and runs
// the epilogue on them.  Every mbarrier wait is bounded as in the LM-head kernel.
#pragma once

#include <cooperative_groups.h>
#include <cstdint>

#include "device_common.cuh"
#include "tensor_core.cuh"

namespace specverify {

constexpr int kLinBM = 128;          // output channels per tile (TMEM lanes)
constexpr int kLinBK = 128;          // bytes of K per stage: one 128-byte swizzle row
constexpr uint32_t kLinStageW = kLinBM * kLinBK;
constexpr uint32_t kLinSmemMax = 227u * 1024u;
// K slices of a stage.  A warp's turn of the ring (wait, loads or MMAs, commit) weighs as much as a
// narrow tile's slice: two to a turn, 32 x 12288 x 4096 bf16 18.5 us (20.3 with one), 32 x 1024 x
// 1024 4.7 (5.4).  A tile of 128 columns is better off with twice the stages (128 x 8192 x 4096
// 18.9, 19.9 with two).
__host__ __device__ constexpr int lin_slices(int bn) { return bn >= 128 ? 1 : 2; }

__host__ __device__ constexpr uint32_t lin_slice_bytes(int bn) { return kLinStageW + static_cast<uint32_t>(bn) * kLinBK; }
__host__ __device__ constexpr uint32_t lin_stage_bytes(int bn) { return lin_slices(bn) * lin_slice_bytes(bn); }
// Epilogue warps: two for each 32-lane slice of TMEM where a tile has columns for both, so that the
// epilogue of a tile (its loads of the residual, activations and stores) takes less time than
// the products of the next.
__host__ __device__ constexpr int lin_epilogue_warps(int bn) { return bn >= 64 ? 8 : 4; }
__host__ __device__ constexpr int lin_threads(int bn) { return 64 + 32 * lin_epilogue_warps(bn); }
// columns (tokens) of a step of the epilogue, and the shared memory where they are turned into rows
__host__ __device__ constexpr int lin_step(int bn) { return bn < 32 ? bn : 32; }
__host__ __device__ constexpr uint32_t lin_turn_bytes(int bn) {
    return static_cast<uint32_t>(lin_epilogue_warps(bn) * lin_step(bn) * 32 * 4);
}
// stages that fit beside 1024 bytes of alignment slack, the epilogue's and the barriers
__host__ __device__ constexpr int lin_stages(int bn) {
    const int n = static_cast<int>((kLinSmemMax - 1024u - 512u - lin_turn_bytes(bn)) / lin_stage_bytes(bn));
    return n > 6 ? 6 : n;
}
constexpr uint32_t lin_smem(int bn) {
    return 1024u + static_cast<uint32_t>(lin_stages(bn)) * lin_stage_bytes(bn) + lin_turn_bytes(bn) + 512u;
}

// Instruction descriptor: D fp32 (bits 4-5 = 1); A and B formats at bits 7-9 and 10-12 (kind::f16:
// bf16 = 1; kind::f8f6f4: e4m3 = 0); both K-major; N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t lin_idesc(bool fp8, int bn) {
    return (1u << 4) | (fp8 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(bn >> 3) << 17) |
           (static_cast<uint32_t>(kLinBM >> 4) << 24);
}

// (By a whole warp, whose elected thread issues.)
template <bool kFp8>
__device__ __forceinline__ void lin_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    if (kFp8) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}

enum LinAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// v / (1 + e^-t).  2^x and the division are the special-function unit's: the denominator is at
// least 1, so their relative errors (about 2^-22 each, plus |t| 2^-23 where e^-t > 1) stay a few
// 2^-23 |v|, and an overflowing e^-t gives the limit 0.
__device__ __forceinline__ float lin_sigmoid_times(float v, float t) {
    return __fdividef(v, 1.0f + ex2_fast(-kLog2e * t));
}

// v Phi(v) = max(v, 0) - |v| Phi(-|v|).  For a >= 0, a Phi(-a) = s Q(s) e^{-a^2/2} with s = a / (1 + 0.26 a)
// in [0, 1/0.26): Q is smooth there and never near zero, so a polynomial fits it to a relative error
// (the nine coefficients below, Q(0) = 1/2, from a minimax fit against the scaled complementary error
// function on 0 <= a <= 14.2: 2.7e-8), and a negative v, where the result is this term alone, keeps its
// digits in the tail.  Off by (18 + 5 a + 1.2 a^2) 2^-24 of the term: reciprocal, power and polynomial,
// and the rounding of a^2 / 2, which is v's own.  Branch-free: with erff the epilogue of 4096 x 16384 x
// 256 e4m3 took 123 us.  Past |v| = 16 the term is zero; max(v, 0) = v / 2 + |v| / 2 keeps a NaN.
__device__ __forceinline__ float lin_gelu(float v) {
    const float a = fminf(fabsf(v), 16.0f);
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.26f, a, 1.0f)));
    const float s = a * t;
    float q = fmaf(6.36942332e-07f, s, -7.32871149e-06f);
    q = fmaf(q, s, 1.11066438e-05f);
    q = fmaf(q, s, 1.69870400e-04f);
    q = fmaf(q, s, -1.59907286e-04f);
    q = fmaf(q, s, -1.00966180e-02f);
    q = fmaf(q, s, 7.63486475e-02f);
    q = fmaf(q, s, -2.68942028e-01f);
    q = fmaf(q, s, 0.5f);
    return fmaf(0.5f, v, 0.5f * fabsf(v)) - (s * q) * ex2_fast(a * a * (-0.5f * kLog2e));
}

// The activation of W values; the choice is made once for all of them.  The tanh form of GELU is
// v sigmoid(2 sqrt(2/pi) (v + 0.044715 v^3)), since (1 + tanh z) / 2 = sigmoid(2z).
template <int W>
__device__ __forceinline__ void lin_activate(float (&v)[W], int act) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = v[i] > 0.0f || isnan(v[i]) ? v[i] : 0.0f;
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = lin_gelu(v[i]);
            break;
        case kActGeluTanh:
#pragma unroll
            for (int i = 0; i < W; ++i)
                v[i] = lin_sigmoid_times(v[i], 1.5957691216057308f * fmaf(0.044715f * v[i] * v[i], v[i], v[i]));
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = lin_sigmoid_times(v[i], v[i]);
            break;
        default: break;
    }
}

struct LinearParams {
    int rows, N;
    int bn;                   // tokens per tile (linear_pair_kernel)
    int kblocks;              // 128-byte slices of K
    int m_tiles, n_tiles;     // tiles of bn tokens and of 128 output channels
    int group;                // token tiles of one raster group
    int act;
    int vec;                  // rows of out and residual are whole groups of four on their boundaries
    int out_f32;              // type of out, bias and residual: fp32, or bf16
    const float* x_scale;     // [rows] (e4m3)
    const float* w_scale;     // [N] (e4m3)
    const void* bias;         // [N] or nullptr
    const void* residual;     // [rows, N] or nullptr
    void* out;                // [rows, N]
    int32_t* status;
};

// Tile index -> (token tile, channel tile): groups of `group` token tiles, within a group the
// channel tiles outermost, so that the CTAs at work share few slices of both operands.
__device__ __forceinline__ void lin_tile(const LinearParams& p, int tile, int& mt, int& nt) {
    const int per_group = p.group * p.n_tiles;
    const int g = tile / per_group, in = tile - g * per_group;
    const int width = min(p.group, p.m_tiles - g * p.group);
    nt = in / width;
    mt = g * p.group + in - nt * width;
}

__device__ __forceinline__ float lin_load(const void* base, long long i, bool f32) {
    if (f32) return static_cast<const float*>(base)[i];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
}

__device__ __forceinline__ void lin_store(void* base, long long i, bool f32, float v) {
    if (f32) {
        static_cast<float*>(base)[i] = v;
    } else {
        uint32_t c;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(c) : "f"(0.0f), "f"(v));
        static_cast<uint16_t*>(base)[i] = static_cast<uint16_t>(c);
    }
}

// The residual of W columns (tokens m .. m_end - 1 of one output channel n), as stored: every load in
// flight at once, none behind a branch (columns outside the output repeat one inside; m < m_end).
template <int W>
__device__ __forceinline__ void lin_residual(const LinearParams& p, uint32_t (&res)[W], int m, int m_end, int n) {
    const int last = m_end - 1 - m;
    const long long at = static_cast<long long>(m) * p.N + min(n, p.N - 1);
    if (p.out_f32) {
        const uint32_t* r = static_cast<const uint32_t*>(p.residual) + at;
#pragma unroll
        for (int i = 0; i < W; ++i) res[i] = r[static_cast<long long>(min(i, last)) * p.N];
    } else {
        const uint16_t* r = static_cast<const uint16_t*>(p.residual) + at;
#pragma unroll
        for (int i = 0; i < W; ++i) res[i] = r[static_cast<long long>(min(i, last)) * p.N];
    }
}

// The residual of a tile into L2 ahead of its epilogue: thread i of `threads` takes the rows m0 + i, ...
// Read by the epilogue itself it comes in pieces of 64 bytes of far-apart rows, which DRAM serves at
// a fraction of its rate.
__device__ __forceinline__ void lin_prefetch_residual(const LinearParams& p, int m0, int m_end, int n0, int channels, int i,
                                                      int threads) {
    if (!p.residual || n0 >= p.N) return;
    const int es = p.out_f32 ? 4 : 2;
    const uint32_t bytes = static_cast<uint32_t>(min(channels, p.N - n0) * es) & ~15u;
    for (int m = m0 + i; m < m_end; m += threads) {
        const char* at = static_cast<const char*>(p.residual) + (static_cast<long long>(m) * p.N + n0) * es;
        if (bytes && (reinterpret_cast<uintptr_t>(at) & 15u) == 0) prefetch_l2(at, bytes);
    }
}

template <int W, bool kF32, bool kGuard>
__device__ __forceinline__ void lin_write(const LinearParams& p, const float (&v)[W], int m, int m_end, int n) {
    const long long at = static_cast<long long>(m) * p.N + n;
    const bool n_ok = !kGuard || n < p.N;
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (n_ok && (!kGuard || m + i < m_end)) lin_store(p.out, at + static_cast<long long>(i) * p.N, kF32, v[i]);
}

// The epilogue of W columns (tokens m .. m_end - 1) of one output channel n: v holds the sums, res
// the residual.
template <int W>
__device__ __forceinline__ void lin_finish(const LinearParams& p, float (&v)[W], const uint32_t (&res)[W], int m,
                                           int m_end, int n, int lane, float ws, float bias) {
    if (p.x_scale) {
        const float xs = lane < W && m + lane < m_end ? __ldg(p.x_scale + m + lane) : 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = fmaf(v[i], __shfl_sync(0xffffffffu, xs, i) * ws, bias);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += bias;
    }
    lin_activate<W>(v, p.act);
    if (p.residual) {
        const int shift = p.out_f32 ? 0 : 16;
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += __uint_as_float(res[i] << shift);
    }
    const bool guard = m + W > m_end || n - lane + 32 > p.N;  // (uniform over the warp)
    if (p.out_f32) {
        if (guard) lin_write<W, true, true>(p, v, m, m_end, n);
        else lin_write<W, true, false>(p, v, m, m_end, n);
    } else {
        if (guard) lin_write<W, false, true>(p, v, m, m_end, n);
        else lin_write<W, false, false>(p, v, m, m_end, n);
    }
}

// ---- The epilogue of a step in rows: W tokens x 32 channels of a warp.  TMEM gives a lane one channel of
// every token: written out that way a step is a load of the residual, a store and their addresses
// for every value, and the epilogue is bound by issue.  With a residual the step is turned through
// shared memory instead, and a lane takes four channels of W / 4 tokens: loads and stores of 8 or 16
// bytes, and the token's scale one load instead of a shuffle a value.  (In the pair
// kernel without a residual the turn costs more than it saves: 4096 x 16384 x 256 bf16 42 us
// direct, 61 turned; with one, e4m3 and a shorter GELU, 172 and 139 (with the present one 155 turned).
// One CTA a tile, 1000 x 5000 x 256: 11.3 and 10.0.) ----

// Four values as stored.
template <bool kF32>
struct LinFour {
    using type = uint2;  // bf16
};
template <>
struct LinFour<true> {
    using type = uint4;
};

// The residual of a step, as stored; m < m_end.
template <int W, bool kF32>
__device__ __forceinline__ void lin_residual_rows(const LinearParams& p, typename LinFour<kF32>::type (&res)[W / 4], int m,
                                                  int m_end, int n4, int lane) {
    using T = typename LinFour<kF32>::type;
    const long long at = min(n4, p.N - 4);
#pragma unroll
    for (int k = 0; k < W / 4; ++k) {
        const long long i = static_cast<long long>(min(m + 4 * k + (lane >> 3), m_end - 1)) * p.N + at;
        res[k] = *reinterpret_cast<const T*>(static_cast<const char*>(p.residual) + i * (kF32 ? 4 : 2));
    }
}

// v: the sums of tokens m .. m + W - 1 for the channel of this lane; turn: the warp's shared memory
// [W][32]; ws, bias: of the channels n4 .. n4 + 3 that the lane writes.
template <int W, bool kF32>
__device__ __forceinline__ void lin_finish_rows(const LinearParams& p, const float (&v)[W],
                                                const typename LinFour<kF32>::type (&res)[W / 4], float* turn, int m, int m_end, int n4, int lane, const float (&ws)[4],
                                                const float (&bias)[4]) {
    __syncwarp();  // (the step before has been read)
#pragma unroll
    for (int i = 0; i < W; ++i) turn[i * 32 + lane] = v[i];
    __syncwarp();
    const int row = m + (lane >> 3);  // and every fourth after it
    float a[W];
#pragma unroll
    for (int k = 0; k < W / 4; ++k) {
        const float4 q = *reinterpret_cast<const float4*>(turn + (4 * k + (lane >> 3)) * 32 + (lane & 7) * 4);
        a[4 * k] = q.x;
        a[4 * k + 1] = q.y;
        a[4 * k + 2] = q.z;
        a[4 * k + 3] = q.w;
    }
    if (p.x_scale) {
        float xs[W / 4];
#pragma unroll
        for (int k = 0; k < W / 4; ++k) xs[k] = __ldg(p.x_scale + min(row + 4 * k, m_end - 1));
#pragma unroll
        for (int i = 0; i < W; ++i) a[i] = fmaf(a[i], xs[i / 4] * ws[i % 4], bias[i % 4]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) a[i] += bias[i % 4];
    }
    lin_activate<W>(a, p.act);
    const long long at = static_cast<long long>(row) * p.N + n4;
    const long long step = 4LL * p.N;
    const bool in = n4 < p.N;
    if constexpr (kF32) {
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
            float4 o = make_float4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
            if (p.residual) {
                o.x += __uint_as_float(res[k].x);
                o.y += __uint_as_float(res[k].y);
                o.z += __uint_as_float(res[k].z);
                o.w += __uint_as_float(res[k].w);
            }
            if (in && row + 4 * k < m_end) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at + k * step) = o;
        }
    } else {
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
            if (p.residual) {
                a[4 * k] += __uint_as_float(res[k].x << 16);
                a[4 * k + 1] += __uint_as_float(res[k].x & 0xFFFF0000u);
                a[4 * k + 2] += __uint_as_float(res[k].y << 16);
                a[4 * k + 3] += __uint_as_float(res[k].y & 0xFFFF0000u);
            }
            uint2 o;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(a[4 * k + 1]), "f"(a[4 * k]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(a[4 * k + 3]), "f"(a[4 * k + 2]));
            if (in && row + 4 * k < m_end) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at + k * step) = o;
        }
    }
}

// Weight scale and bias of the channels n4 .. n4 + 3.
__device__ __forceinline__ void lin_channels(const LinearParams& p, int n4, float (&ws)[4], float (&bias)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = min(n4 + i, p.N - 1);
        ws[i] = p.w_scale ? __ldg(p.w_scale + n) : 1.0f;
        bias[i] = p.bias ? lin_load(p.bias, n, p.out_f32 != 0) : 0.0f;
    }
}

// Wait (bounded) for an accumulator: lane 0 waits and the warp follows it, so that it stays converged
// for the .sync.aligned TMEM loads; then every lane observes the completed phase.
__device__ __forceinline__ bool lin_accumulator(uint64_t* bar, uint32_t phase, volatile int* abort, int lane) {
    int ok = 0;
    if (lane == 0) ok = mbar_wait(bar, phase, abort);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) {
        if (lane == 0) *abort = 1;
        return false;
    }
    volatile int never = 0;
    mbar_wait(bar, phase, &never);  // completed: returns at once
    __syncwarp();
    tmem_fence_after();
    return true;
}

// A tile's epilogue by one warp: columns c_first, c_first + kStep, ... (steps of kW) of the accumulator at
// `lanes`, 32 channels from n0, tokens m0 .. m_end - 1.  `wait` returns once the accumulator is complete
// (false: give up); what is read from memory is on its way before.
template <int kW, int kStep, bool kTurn, bool kF32, class Wait>
__device__ __forceinline__ bool lin_epilogue_as(const LinearParams& p, uint32_t lanes, float* turn, int bn, int c_first, int m0,
                                             int m_end, int n0, int lane, Wait wait) {
    if (p.vec && (kTurn || p.residual)) {
        const int n4 = n0 + (lane & 7) * 4;
        float ws[4], bias[4];
        lin_channels(p, n4, ws, bias);
        typename LinFour<kF32>::type res[2][kW / 4] = {};  // two steps in flight
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (p.residual && m0 + c_first + h * kStep < m_end)
                lin_residual_rows<kW, kF32>(p, res[h], m0 + c_first + h * kStep, m_end, n4, lane);
        if (!wait()) return false;
#pragma unroll 1
        for (int c = c_first; c < bn && m0 + c < m_end; c += 2 * kStep) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = m0 + c + h * kStep;
                if (c + h * kStep >= bn || m >= m_end) break;
                float v[kW];
                tmem_load<kW>(lanes + static_cast<uint32_t>(c + h * kStep), v);
                lin_finish_rows<kW, kF32>(p, v, res[h], turn, m, m_end, n4, lane, ws, bias);
                if (p.residual && m + 2 * kStep < m_end) lin_residual_rows<kW, kF32>(p, res[h], m + 2 * kStep, m_end, n4, lane);
            }
        }
    } else {
        const int n = n0 + lane;
        const float ws = p.w_scale && n < p.N ? __ldg(p.w_scale + n) : 1.0f;
        const float bias = p.bias && n < p.N ? lin_load(p.bias, n, p.out_f32 != 0) : 0.0f;
        uint32_t res[kW] = {};
        if (p.residual && m0 + c_first < m_end) lin_residual<kW>(p, res, m0 + c_first, m_end, n);
        if (!wait()) return false;
#pragma unroll 1
        for (int c = c_first; c < bn && m0 + c < m_end; c += kStep) {
            const int m = m0 + c;
            float v[kW];
            tmem_load<kW>(lanes + static_cast<uint32_t>(c), v);
            lin_finish<kW>(p, v, res, m, m_end, n, lane, ws, bias);
            if (p.residual && m + kStep < m_end) lin_residual<kW>(p, res, m + kStep, m_end, n);
        }
    }
    return true;
}

// kTurn: in rows with or without a residual.
template <int kW, int kStep, bool kTurn, class Wait>
__device__ __forceinline__ bool lin_epilogue(const LinearParams& p, uint32_t lanes, float* turn, int bn, int c_first, int m0,
                                             int m_end, int n0, int lane, Wait wait) {
    return p.out_f32 ? lin_epilogue_as<kW, kStep, kTurn, true>(p, lanes, turn, bn, c_first, m0, m_end, n0, lane, wait)
                     : lin_epilogue_as<kW, kStep, kTurn, false>(p, lanes, turn, bn, c_first, m0, m_end, n0, lane, wait);
}

// CTA `rank`'s share of a tile whose K was split over S CTAs: BN / S columns, a warp's all at once (so
// that the other CTAs' shared memory is waited for once), added in rank order, then the epilogue.
template <int BN, int S>
__device__ __forceinline__ void lin_reduce(const LinearParams& p, const float* part, int rank, int mt, int nt, int warp, int lane) {
    constexpr int kGroups = lin_epilogue_warps(BN) / 4;
    constexpr int kC = BN / S / kGroups;
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int slice = warp & 3, c = rank * (BN / S) + ((warp - 2) >> 2) * kC;
    const int n = nt * kLinBM + slice * 32 + lane;
    const int m = mt * BN + c, m_end = min(p.rows, m + kC);
    if (m >= m_end) return;
    float q[S][kC], v[kC] = {};
#pragma unroll
    for (int r = 0; r < S; ++r) {
        const float* from = cluster.map_shared_rank(part, r) + c * kLinBM + slice * 32 + lane;
#pragma unroll
        for (int i = 0; i < kC; ++i) q[r][i] = from[i * kLinBM];
    }
    const float ws = p.w_scale && n < p.N ? __ldg(p.w_scale + n) : 1.0f;
    const float bias = p.bias && n < p.N ? lin_load(p.bias, n, p.out_f32 != 0) : 0.0f;
    uint32_t res[kC] = {};
    if (p.residual) lin_residual<kC>(p, res, m, m_end, n);
#pragma unroll
    for (int r = 0; r < S; ++r)
#pragma unroll
        for (int i = 0; i < kC; ++i) v[i] += q[r][i];
    lin_finish<kC>(p, v, res, m, m_end, n, lane, ws, bias);
}

template <bool kFp8, int BN, bool kSplit>
__global__ void __launch_bounds__(lin_threads(BN), 1)
linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LinearParams p) {
    namespace cg = cooperative_groups;
    constexpr int kStages = lin_stages(BN);
    constexpr int kElems = kFp8 ? kLinBK : kLinBK / 2;   // K elements of a stage
    constexpr uint32_t kCols = 2 * BN < 32 ? 32 : 2 * BN;
    constexpr int kW = lin_step(BN);                     // columns of an epilogue step
    constexpr int kEpiWarps = lin_epilogue_warps(BN);
    extern __shared__ uint8_t lin_smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* stage_w = base;
    constexpr int kSlices = lin_slices(BN);
    uint8_t* stage_x = base + kStages * kSlices * kLinStageW;
    float* turn = reinterpret_cast<float*>(base + kStages * lin_stage_bytes(BN));  // the epilogue's
    uint64_t* full = reinterpret_cast<uint64_t*>(base + kStages * lin_stage_bytes(BN) + lin_turn_bytes(BN));
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* tdrain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdrain + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = kSplit ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
    const int rank = kSplit ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int tiles = p.m_tiles * p.n_tiles;
    const int first = static_cast<int>(blockIdx.x) / splits;
    const int step = static_cast<int>(gridDim.x) / splits;
    // this CTA's turns of the ring (a slice past the end of K is filled with zeros)
    const int turns = (p.kblocks + kSlices - 1) / kSlices;
    const int kb0 = static_cast<int>(static_cast<long long>(turns) * rank / splits);
    const int kb1 = static_cast<int>(static_cast<long long>(turns) * (rank + 1) / splits);

    if (threadIdx.x == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, kEpiWarps);  // one arrival per epilogue warp
        }
        mbar_init(tdrain, 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependency();

    if (warp == 0) {
        // ---- TMA producer ----
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        bool go = true;
        for (int tile = first; tile < tiles && go; tile += step) {
            int mt, nt;
            lin_tile(p, tile, mt, nt);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_mbar_wait(empty + stage, phase ^ 1u, abort)) {
                    go = false;
                    break;
                }
                warp_expect_tx(full + stage, lin_stage_bytes(BN));
#pragma unroll
                for (int h = 0; h < kSlices; ++h) {
                    const int at = stage * kSlices + h, k = (kb * kSlices + h) * kElems;
                    warp_tma_load_2d(&map_w, full + stage, stage_w + at * kLinStageW, k, nt * kLinBM);
                    warp_tma_load_2d(&map_x, full + stage, stage_x + at * (BN * kLinBK), k, mt * BN);
                }
                ++issued;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!go) {
            // let the loads in flight land before the CTA's shared memory goes away
            if (lane == 0) *abort = 1;
            const int pending = min(issued, kStages);
            for (int k = 0; k < pending; ++k) {
                if (--stage < 0) {
                    stage = kStages - 1;
                    phase ^= 1u;
                }
                volatile int never = 0;
                warp_mbar_wait(full + stage, phase, &never);
            }
            if (lane == 0) set_status(p.status, 4 /* SPEC_ETIMEOUT */);
        }
    } else if (warp == 1) {
        // ---- MMA issuer ----
        int stage = 0;
        uint32_t phase = 0;
        int t = 0;
        const uint32_t idesc = lin_idesc(kFp8, BN);
        bool go = true;
        for (int tile = first; tile < tiles && go; tile += step, ++t) {
            const int acc = t & 1;
            if (!warp_mbar_wait(tempty + acc, ((t >> 1) & 1u) ^ 1u, abort)) {
                go = false;
                break;
            }
            tmem_fence_after();
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_mbar_wait(full + stage, phase, abort)) {
                    go = false;
                    break;
                }
                tmem_fence_after();
#pragma unroll
                for (int h = 0; h < kSlices; ++h) {
                    const int at = stage * kSlices + h;
                    const uint64_t adesc = sw128_kmajor_desc(smem_addr(stage_w + at * kLinStageW));
                    const uint64_t bdesc = sw128_kmajor_desc(smem_addr(stage_x + at * (BN * kLinBK)));
#pragma unroll
                    for (int kk = 0; kk < kLinBK / 32; ++kk)  // 32 bytes of K per MMA
                        lin_mma<kFp8>(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, kb != kb0 || h != 0 || kk != 0);
                }
                warp_umma_commit(empty + stage);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!go) break;
            warp_umma_commit(tfull + acc);
        }
        if (!go && lane == 0) *abort = 1;
        warp_umma_commit(tdrain);  // no MMA may still write TMEM when it is freed
        volatile int never = 0;
        if (!warp_mbar_wait(tdrain, 0, &never) && lane == 0) set_status(p.status, 4 /* SPEC_ETIMEOUT */);
    } else {
        // ---- epilogue: TMEM lane slice (warp % 4) * 32, every (kEpiWarps / 4)-th step of columns ----
        const int slice = warp & 3, part_of = (warp - 2) >> 2;
        constexpr int kStep = kW * (kEpiWarps / 4);
        int t = 0;
        for (int tile = first; tile < tiles; tile += step, ++t) {
            const int acc = t & 1;
            int mt, nt;
            lin_tile(p, tile, mt, nt);
            const int m0 = mt * BN, m_end = min(p.rows, m0 + BN);
            const uint32_t lanes = tmem_base + (static_cast<uint32_t>(slice * 32) << 16) + static_cast<uint32_t>(acc * BN);
            auto wait = [&] { return lin_accumulator(tfull + acc, (t >> 1) & 1u, abort, lane); };
            bool ok;
            if (kSplit) {
                ok = wait();
                float* part = reinterpret_cast<float*>(base);  // [BN][128]; every load and MMA is done
#pragma unroll 1
                for (int c = part_of * kW; ok && c < BN && m0 + c < m_end; c += kStep) {
                    float v[kW];
                    tmem_load<kW>(lanes + static_cast<uint32_t>(c), v);
#pragma unroll
                    for (int i = 0; i < kW; ++i) part[(c + i) * kLinBM + slice * 32 + lane] = v[i];
                }
            } else {
                ok = lin_epilogue<kW, kStep, true>(p, lanes, turn + (warp - 2) * kW * 32, BN, part_of * kW, m0, m_end,
                                             nt * kLinBM + slice * 32, lane, wait);
            }
            if (!ok) break;
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty + acc);
        }
        if (*abort && lane == 0) set_status(p.status, 4 /* SPEC_ETIMEOUT */);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kCols) : "memory");
    }
    if (kSplit) {
        cg::this_cluster().sync();  // every CTA's partial tile is in its shared memory
        int mt, nt;
        lin_tile(p, first, mt, nt);
        const float* part = reinterpret_cast<const float*>(base);
        if (warp >= 2) {
            if (splits == 2) lin_reduce<BN, 2>(p, part, rank, mt, nt, warp, lane);
            else if (splits == 4) lin_reduce<BN, 4>(p, part, rank, mt, nt, warp, lane);
            else lin_reduce<BN, 8>(p, part, rank, mt, nt, warp, lane);
        }
        cg::this_cluster().sync();  // no CTA leaves while another reads its partial tile
    }
}

// ----------------------------------------------------------------------------------------
// Many tokens: the same product on CTA pairs.  A pair owns 256 channels x bn tokens, each CTA 128
// of the channels (its TMEM lanes) and the loads of half of the tokens' rows: 32 KB per K slice and
// CTA where one CTA alone would load 48 KB for a 128 x 256 tile.  The loads of both operands come
// from L2 at about 64 bytes a clock and SM, and with one CTA per tile they, not the tensor cores,
// were the bound (3328 x 4096 x 4096 bf16: 82 us; 1.28 GB through L2).
// ----------------------------------------------------------------------------------------

constexpr int kPairBN = 256;                              // most tokens of a tile
constexpr int kPairBM = 256;                              // channels of a tile
constexpr uint32_t kPairStage = kLinStageW + (kPairBN / 2) * kLinBK;  // bytes per CTA
constexpr int kPairStages = 6;
constexpr int kPairEpiWarps = 8;
constexpr unsigned long long kPairLandNs = 10000000ull;  // after a timeout: time for loads to land
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr uint32_t kPairTurn = kPairEpiWarps * 32 * 32 * 4;  // the epilogue's shared memory
constexpr uint32_t kPairSmem = 1024u + kPairStages * kPairStage + kPairTurn + 512u;

__host__ __device__ constexpr uint32_t pair_idesc(bool fp8, int bn) {
    return (1u << 4) | (fp8 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(bn >> 3) << 17) |
           (static_cast<uint32_t>(kPairBM >> 4) << 24);
}

// (By a whole warp, whose elected thread issues.)
template <bool kFp8>
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    if (kFp8) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}

// Launched in clusters of two.  p.bn: a multiple of 32; p.n_tiles counts tiles of 256 channels.
template <bool kFp8>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LinearParams p) {
    namespace cg = cooperative_groups;
    constexpr int kElems = kFp8 ? kLinBK : kLinBK / 2;
    constexpr int kW = 32;
    extern __shared__ uint8_t lin_smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* stage_w = base;
    uint8_t* stage_x = base + kPairStages * kLinStageW;
    float* turn = reinterpret_cast<float*>(base + kPairStages * kPairStage);  // the epilogue's
    uint64_t* full = reinterpret_cast<uint64_t*>(base + kPairStages * kPairStage + kPairTurn);  // (the even CTA's are used)
    uint64_t* empty = full + kPairStages;
    uint64_t* tfull = empty + kPairStages;
    uint64_t* tempty = tfull + 2;  // (the even CTA's are used)
    uint64_t* tdrain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdrain + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = p.m_tiles * p.n_tiles;
    const int first = static_cast<int>(blockIdx.x) / 2, step = static_cast<int>(gridDim.x) / 2;

    if (threadIdx.x == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 2 * kPairEpiWarps);  // every epilogue warp of both CTAs
        }
        mbar_init(tdrain, 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {  // TMEM of both CTAs: two accumulators of 256 columns
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    cluster.sync();  // both CTAs' barriers and TMEM are there
    tmem_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependency();

    if (warp == 0) {
        // ---- TMA producer: this CTA's channels, and its half of the tokens ----
        const uint32_t lead_full = pair_leader_addr(full);
        int stage = 0;
        uint32_t phase = 0;
        bool go = true;
        for (int tile = first; tile < tiles && go; tile += step) {
            int mt, nt;
            lin_tile(p, tile, mt, nt);
            for (int kb = 0; kb < p.kblocks; ++kb) {
                if (!warp_mbar_wait(empty + stage, phase ^ 1u, abort)) {
                    go = false;
                    break;
                }
                if (rank == 0) warp_expect_tx(full + stage, 2u * kLinStageW + static_cast<uint32_t>(p.bn) * kLinBK);
                const uint32_t bar = lead_full + static_cast<uint32_t>(stage * sizeof(uint64_t));
                tma_load_2d_pair(&map_w, bar, stage_w + stage * kLinStageW, kb * kElems, nt * kPairBM + rank * kLinBM);
                tma_load_2d_pair(&map_x, bar, stage_x + stage * (kPairBN / 2 * kLinBK), kb * kElems,
                                 mt * p.bn + rank * (p.bn / 2));
                if (++stage == kPairStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!go && lane == 0) {
            *abort = 1;
            // let the loads in flight land before the CTA's shared memory goes away (their
            // barriers may be the other CTA's, so by time: they take microseconds)
            const unsigned long long t0 = global_time_ns();
            while (global_time_ns() - t0 < kPairLandNs) __nanosleep(1000);
            set_status(p.status, 4 /* SPEC_ETIMEOUT */);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer (the even CTA's whole warp) ----
        if (rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int t = 0;
            const uint32_t idesc = pair_idesc(kFp8, p.bn);
            bool go = true;
            for (int tile = first; tile < tiles && go; tile += step, ++t) {
                const int acc = t & 1;
                if (!warp_mbar_wait(tempty + acc, ((t >> 1) & 1u) ^ 1u, abort)) {
                    go = false;
                    break;
                }
                tmem_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kPairBN);
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!warp_mbar_wait(full + stage, phase, abort)) {
                        go = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint64_t adesc = sw128_kmajor_desc(smem_addr(stage_w + stage * kLinStageW));
                    const uint64_t bdesc = sw128_kmajor_desc(smem_addr(stage_x + stage * (kPairBN / 2 * kLinBK)));
#pragma unroll
                    for (int kk = 0; kk < kLinBK / 32; ++kk)
                        pair_mma<kFp8>(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, kb != 0 || kk != 0);
                    umma_commit_pair(empty + stage);
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!go) break;
                umma_commit_pair(tfull + acc);
            }
            if (!go && lane == 0) *abort = 1;
            umma_commit_pair(tdrain);  // no MMA may still read shared memory or write TMEM below
        }
    } else {
        // ---- epilogue: TMEM lane slice (warp % 4) * 32, every second step of columns ----
        const int slice = warp & 3, part_of = (warp - 2) >> 2;
        const uint32_t lead_tempty = pair_leader_addr(tempty);
        auto prefetch = [&](int tile) {
            if (!p.residual || tile >= tiles) return;
            int mt, nt;
            lin_tile(p, tile, mt, nt);
            lin_prefetch_residual(p, mt * p.bn, min(p.rows, mt * p.bn + p.bn), nt * kPairBM + rank * kLinBM, kLinBM,
                                  static_cast<int>(threadIdx.x) - 64, 32 * kPairEpiWarps);
        };
        prefetch(first);
        int t = 0;
        for (int tile = first; tile < tiles; tile += step, ++t) {
            prefetch(tile + step);
            const int acc = t & 1;
            int mt, nt;
            lin_tile(p, tile, mt, nt);
            const int m0 = mt * p.bn, m_end = min(p.rows, m0 + p.bn);
            const uint32_t lanes = tmem_base + (static_cast<uint32_t>(slice * 32) << 16) + static_cast<uint32_t>(acc * kPairBN);
            auto wait = [&] { return lin_accumulator(tfull + acc, (t >> 1) & 1u, abort, lane); };
            if (!lin_epilogue<kW, kW * (kPairEpiWarps / 4), false>(p, lanes, turn + (warp - 2) * kW * 32, p.bn, part_of * kW, m0, m_end,
                                                            nt * kPairBM + rank * kLinBM + slice * 32, lane, wait))
                break;
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_tempty + static_cast<uint32_t>(acc * sizeof(uint64_t)));
        }
        if (*abort && lane == 0) set_status(p.status, 4 /* SPEC_ETIMEOUT */);
    }
    tmem_fence_before();
    __syncthreads();
    if (threadIdx.x == 32) {
        volatile int never = 0;
        if (!mbar_wait(tdrain, 0, &never)) set_status(p.status, 4 /* SPEC_ETIMEOUT */);
    }
    __syncwarp();
    cluster.sync();  // both CTAs are done with each other's barriers, shared memory and TMEM
    if (warp == 1) {
        __syncwarp();
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
    }
}

// ----------------------------------------------------------------------------------------
// One to four tokens: a stream of the weight.  The call is bound by HBM, and the tile kernel's start
// (barriers, TMEM, descriptors, the first trip of a ring) and end (the cluster's meeting) are time in
// which nothing streams; here plain loads go out in the first instructions.  A block takes 16
// channels at a time and its eight warps share K: lane (g, t) = (lane / 4, lane % 4) loads 16 bytes
// of channels g and g + 8 from its place in a 64-byte slice of K, and the same place of token g
// from shared memory; read as fragments of mma.sync (m16n8k16, fp32 sums) these are a permutation
// of K that both operands share, so no byte is moved again.  (The legacy instruction costs an
// issue slot here, nothing more; tensor throughput is not what bounds this.)  e4m3 is widened to
// fp16, which is exact.  The warps' sums meet in shared memory and are added in warp order.
// ----------------------------------------------------------------------------------------

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewChannels = 16;
constexpr int kFewMaxRows = 4;
constexpr int kFewBatch = 8;                    // slices of a warp in flight: two loads each
constexpr uint32_t kFewMaxSmem = 100u * 1024u;  // the tokens, as 16-bit values

// bytes of one token in shared memory: the row, in whole slices, and 64 bytes that move the next
// token to other banks
__host__ __device__ constexpr uint32_t few_stride(bool fp8, int K) {
    const uint32_t slice = fp8 ? 64u : 32u;  // elements
    return (static_cast<uint32_t>(K) + slice - 1) / slice * slice * 2u + 64u;
}

// Four e4m3 (one word) as two words of two fp16 each.
__device__ __forceinline__ void few_widen(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(w >> 16)));
}

template <bool kF16>
__device__ __forceinline__ void few_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    if constexpr (kF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool kFp8>
__global__ void __launch_bounds__(kFewThreads) linear_few_kernel(const uint8_t* x, const uint8_t* w, int K, LinearParams p) {
    extern __shared__ uint4 few_x[];  // [rows] tokens of few_stride bytes
    __shared__ float s_part[kFewWarps][kFewChannels * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const long long row_bytes = static_cast<long long>(K) * (kFp8 ? 1 : 2);
    const int slices = static_cast<int>((row_bytes + 63) / 64);
    const uint32_t stride = few_stride(kFp8, K);
    const uint8_t* xs = reinterpret_cast<const uint8_t*>(few_x) + static_cast<uint32_t>(g) * stride;
    const bool f32 = p.out_f32 != 0;
    const int groups = (p.N - 1) / kFewChannels + 1;

    uint4 va[kFewBatch], vb[kFewBatch];
    auto load = [&](int group, int s0) {  // slices s0, s0 + 8, .. of the group's channels g and g + 8
        const int n = min(group * kFewChannels + g, p.N - 1), n8 = min(group * kFewChannels + g + 8, p.N - 1);
        const uint8_t* a = w + n * row_bytes;
        const uint8_t* b = w + n8 * row_bytes;
#pragma unroll
        for (int k = 0; k < kFewBatch; ++k) {
            const long long at = static_cast<long long>(s0 + k * kFewWarps) * 64 + t * 16;
            const bool in = at < row_bytes;  // (rows are whole 16-byte vectors)
            va[k] = in ? ld_stream16(a + at) : make_uint4(0u, 0u, 0u, 0u);
            vb[k] = in ? ld_stream16(b + at) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int group = static_cast<int>(blockIdx.x);
    grid_dependency();
    load(group, warp);
    // the tokens, as 16-bit values, zeros behind the row
    {
        constexpr int kVec = kFp8 ? 16 : 8;
        const int per = static_cast<int>((stride - 64u) / (2 * kVec)), have = K / kVec;
        for (int i = threadIdx.x; i < p.rows * per; i += kFewThreads) {
            const int m = i / per, v = i - m * per;
            const uint4 q = v < have ? __ldg(reinterpret_cast<const uint4*>(x + m * row_bytes) + v) : make_uint4(0u, 0u, 0u, 0u);
            uint4* to = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(few_x) + static_cast<uint32_t>(m) * stride) +
                        v * (kFp8 ? 2 : 1);
            if constexpr (kFp8) {
                uint4 lo, hi;
                few_widen(q.x, lo.x, lo.y);
                few_widen(q.y, lo.z, lo.w);
                few_widen(q.z, hi.x, hi.y);
                few_widen(q.w, hi.z, hi.w);
                to[0] = lo;
                to[1] = hi;
            } else {
                to[0] = q;
            }
        }
    }
    __syncthreads();
    for (; group < groups; group += static_cast<int>(gridDim.x)) {
        float c[4] = {};
        for (int s0 = warp; s0 < slices; s0 += kFewWarps * kFewBatch) {
#pragma unroll
            for (int k = 0; k < kFewBatch; ++k) {
                const int s = s0 + k * kFewWarps;
                const bool in = g < p.rows && s < slices;
                if constexpr (kFp8) {
                    const uint4* q = reinterpret_cast<const uint4*>(xs + s * 128 + t * 32);
                    const uint4 x0 = in ? q[0] : make_uint4(0u, 0u, 0u, 0u), x1 = in ? q[1] : make_uint4(0u, 0u, 0u, 0u);
                    uint32_t a[8], b[8];
                    few_widen(va[k].x, a[0], a[1]);
                    few_widen(va[k].y, a[2], a[3]);
                    few_widen(va[k].z, a[4], a[5]);
                    few_widen(va[k].w, a[6], a[7]);
                    few_widen(vb[k].x, b[0], b[1]);
                    few_widen(vb[k].y, b[2], b[3]);
                    few_widen(vb[k].z, b[4], b[5]);
                    few_widen(vb[k].w, b[6], b[7]);
                    few_mma<true>(c, a[0], b[0], a[1], b[1], x0.x, x0.y);
                    few_mma<true>(c, a[2], b[2], a[3], b[3], x0.z, x0.w);
                    few_mma<true>(c, a[4], b[4], a[5], b[5], x1.x, x1.y);
                    few_mma<true>(c, a[6], b[6], a[7], b[7], x1.z, x1.w);
                } else {
                    const uint4* q = reinterpret_cast<const uint4*>(xs + s * 64 + t * 16);
                    const uint4 xv = in ? *q : make_uint4(0u, 0u, 0u, 0u);
                    few_mma<false>(c, va[k].x, vb[k].x, va[k].y, vb[k].y, xv.x, xv.y);
                    few_mma<false>(c, va[k].z, vb[k].z, va[k].w, vb[k].w, xv.z, xv.w);
                }
            }
            // the next slices, or the first of the next group, are on their way meanwhile
            if (s0 + kFewWarps * kFewBatch < slices) load(group, s0 + kFewWarps * kFewBatch);
            else if (group + static_cast<int>(gridDim.x) < groups) load(group + static_cast<int>(gridDim.x), warp);
        }
        // c: channels g, g and g + 8, g + 8 for tokens 2t, 2t + 1
        s_part[warp][(2 * t) * kFewChannels + g] = c[0];
        s_part[warp][(2 * t + 1) * kFewChannels + g] = c[1];
        s_part[warp][(2 * t) * kFewChannels + g + 8] = c[2];
        s_part[warp][(2 * t + 1) * kFewChannels + g + 8] = c[3];
        const int m = static_cast<int>(threadIdx.x) / kFewChannels, n = group * kFewChannels + static_cast<int>(threadIdx.x) % kFewChannels;
        const bool mine = m < p.rows && n < p.N;
        const long long at = static_cast<long long>(m) * p.N + n;
        const float bias = mine && p.bias ? lin_load(p.bias, n, f32) : 0.0f;
        const float res = mine && p.residual ? lin_load(p.residual, at, f32) : 0.0f;
        const float scale = mine && p.x_scale ? __ldg(p.x_scale + m) * __ldg(p.w_scale + n) : 1.0f;
        __syncthreads();
        if (mine) {
            float v[1] = {0.0f};
#pragma unroll
            for (int k = 0; k < kFewWarps; ++k) v[0] += s_part[k][threadIdx.x];
            v[0] = fmaf(v[0], scale, bias);
            lin_activate<1>(v, p.act);
            lin_store(p.out, at, f32, v[0] + res);
        }
        __syncthreads();
    }
}

}  // namespace specverify
