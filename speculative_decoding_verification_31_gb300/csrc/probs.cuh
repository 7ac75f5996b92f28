// probs.cuh -- the verify from probabilities and given random numbers (spec_verify_probs).
//
// Position i of sequence b is accepted while u_i q_i(d_i) < p_i(d_i); j is the first rejected
// position (or the sequence's draft length).  One token is drawn by inverting the running sum:
// with w(x) = max(0, p_j(x) - q_j(x)) at a rejection and w = p_j otherwise, the drawn token is
// the least x whose sum of w over [0, x] exceeds u_gamma times the sum over the whole row.
// u q is exact in fp64 (two 24-bit factors), so the accept test has no rounding at all; the
// running sums must not have a visible one either, since a draw falls next to a border between
// two tokens with a probability proportional to their error.
//
// One cluster of CTAs per sequence.  Every CTA repeats the accept tests (a few gathers) and
// sums its contiguous share of row j in chunks of kProbChunk tokens, one chunk per warp at a
// time.  Sums are pairs of fp32 (hi + lo: an exact difference p - q, compensated additions;
// 2^-38 of the sum at worst): fp64 additions run at 1/64 of fp32's rate here, and with only the
// reductions of lanes and chunks in fp64 the call took 65 us instead of 50 (B = 256, V = 152064,
// fp32; 6.2 of 6.8 TB/s).  Rows of bf16 halve the bytes and not the time: 41 us at that size, and at
// B = 200 33, or 24 where nothing is taken from p (floors 23, 18 and 9).  Neither memory nor a pipe is
// full then (issue 50 %, FMA 35 %); a warp adds and reduces a chunk with no load in flight.  An
// accumulator that begins above its bf16 values saves three of seven instructions an addition and
// 1 us of 42.
// Every warp stores its total into each CTA's shared memory, and after one cluster barrier each
// CTA knows them all; the CTA whose share holds the drawn token finds its chunk from the chunk
// sums it kept and reads that one chunk again.  No workspace, no atomics on global memory and no
// order that varies: the same inputs give the same token whatever else runs.
#pragma once

#include <cooperative_groups.h>
#include <climits>
#include <cstdint>

#include "device_common.cuh"

namespace specverify {

constexpr int kProbThreads = 256;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kProbMaxCluster = 16;
constexpr int kProbChunk = 1024;  // tokens of a warp's step (kChunk of the kernel: that, or half)

struct ProbParams {
    const void* target;       // [B, gamma+1, V]
    const void* draft;        // [B, gamma, V], or nullptr: q_i is one-hot at d_i
    const int32_t* tokens;    // [B, gamma]
    const float* uniforms;    // [B, gamma+1]
    const int32_t* lens;      // [B] draft lengths, or nullptr: gamma
    int B, gamma, V;
    int share;                // chunks of a CTA's share of the row
    int32_t* out_tokens;      // [B, gamma+1]
    int32_t* out_n;           // [B]
    int32_t* status;
};

// A sum of fp32 values as hi + lo.
struct PairSum {
    float hi, lo;
};

// a + b = s + e exactly, s the rounded sum.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = a + b;
    const float c = s - a;
    e = (a - (s - c)) + (b - c);
}

// The sum of two pairs, |lo| brought back to half a step of hi: off by a few 2^-48 of it.
__device__ __forceinline__ PairSum pair_plus(PairSum a, PairSum b) {
    float s, x;
    two_sum(a.hi, b.hi, s, x);
    x += a.lo + b.lo;
    const float hi = s + x;
    return PairSum{hi, x - (hi - s)};
}

__device__ __forceinline__ bool pair_exceeds(PairSum a, PairSum b) {
    float s, x;
    two_sum(a.hi, -b.hi, s, x);
    return s + (x + (a.lo - b.lo)) > 0.0f;
}

// A probability as the operator takes it: negative values and NaN count as zero.
__device__ __forceinline__ float prob_value(float v) { return fmaxf(v, 0.0f); }

// max(0, p - q) as its rounded value and the rounding error: with q held to p the difference is
// never negative, and (p - s) - q recovers the error exactly.
__device__ __forceinline__ PairSum prob_difference(float p, float q) {
    const float x = prob_value(p), y = fminf(prob_value(q), x);
    const float s = x - y;
    return PairSum{s, (x - s) - y};
}

// Two running pair sums a = (hi, lo) += max(0, p - q) of two tokens.
__device__ __forceinline__ void add_differences(uint64_t& hi, uint64_t& lo, float p0, float p1, float q0, float q1) {
    const float x0 = prob_value(p0), x1 = prob_value(p1);
    const uint64_t x = pack2(x0, x1), y = pack2(fminf(prob_value(q0), x0), fminf(prob_value(q1), x1));
    const uint64_t d = sub2(x, y);
    const uint64_t err = sub2(sub2(x, d), y);
    const uint64_t s = add2(hi, d), c = sub2(s, hi);
    const uint64_t e = add2(sub2(hi, sub2(s, c)), sub2(d, c));
    lo = add2(lo, add2(e, err));
    hi = s;
}

// How a chunk lies: wholly inside its row, every vector on a 16-byte boundary; the last chunk of a
// row of whole vectors; inside its row by a vector, p or q off the boundary; anything else.
enum class ChunkKind { kInside, kLast, kShifted, kOther };

// 16 bytes from `words` words and, if `half`, two bytes into the 32 of lo and hi.
__device__ __forceinline__ uint4 vec_within(const uint4& lo, const uint4& hi, int words, bool half) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = (words & 2) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = (words & 1) ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], half ? 16 : 0);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's tokens of a row off its boundary, all loads under way before the first is needed.  bf16:
// the vectors of tokens xb + (k 32 + lane) kVec.., each from two aligned ones.  fp32: 4-byte loads,
// a warp's side by side: word e of vector k is token xb + (4 k + e) 32 + lane.  (200 x 151669: bf16
// 73 -> 48 us, fp32 61 -> 46, against a vector's own loads by size, each behind its branches.)
template <class ET, int kBatch>
__device__ __forceinline__ void load_shifted_vecs(const typename ET::storage* row, int xb, int lane, uint4 (&v)[kBatch]) {
    if constexpr (ET::kVec == 8) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + xb + lane * ET::kVec);
        const uint4* a = reinterpret_cast<const uint4*>(at & ~uintptr_t{15});
        uint4 next[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            v[k] = __ldg(a + k * 32);
            next[k] = __ldg(a + k * 32 + ((at & 15u) ? 1 : 0));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = vec_within(v[k], next[k], static_cast<int>(at & 15u) >> 2, (at & 2u) != 0);
    } else {
        const uint32_t* a = reinterpret_cast<const uint32_t*>(row) + xb + lane;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            v[k] = make_uint4(__ldg(a + k * 128), __ldg(a + k * 128 + 32), __ldg(a + k * 128 + 64), __ldg(a + k * 128 + 96));
    }
}

// Vector of tokens x.. of a row that is not on a 16-byte boundary, or that ends inside it (zeros
// behind the end).
template <class ET>
__device__ __forceinline__ uint4 load_prob_vec_slow(const typename ET::storage* row, int x, int V) {
    if (x + ET::kVec <= V) return ET::load_vec_unaligned(row + x);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    constexpr int kPerWord = ET::kVec / 4;
#pragma unroll
    for (int e = 0; e < ET::kVec; ++e) {
        if (x + e >= V) continue;
        const uint32_t bits = __float_as_uint(ET::load1(row + x + e));
        if (kPerWord == 1) w[e] = bits;
        else w[e / 2] |= (e & 1) ? (bits & 0xFFFF0000u) : (bits >> 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class ET, ChunkKind kKind>
__device__ __forceinline__ uint4 load_prob_vec(const typename ET::storage* row, int x, int V) {
    if constexpr (kKind == ChunkKind::kInside) return ld_stream16(row + x);
    if constexpr (kKind == ChunkKind::kLast) return x < V ? ld_stream16(row + x) : make_uint4(0u, 0u, 0u, 0u);
    return load_prob_vec_slow<ET>(row, x, V);
}

// The raced row: p, and what is taken from it (a row of q, or 1 at one token, or nothing).
template <class ET>
struct ProbRow {
    const typename ET::storage* p;
    const typename ET::storage* q;  // nullptr: nothing is read
    int one_hot;                    // token whose q is 1 (-1: none)
    bool aligned;                   // both on 16-byte boundaries
};

template <class ET>
__device__ __forceinline__ ProbRow<ET> prob_row(const typename ET::storage* p, const typename ET::storage* q, int one_hot) {
    return ProbRow<ET>{p, q, one_hot, ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0};
}

// The weight of token x of the row.
template <class ET>
__device__ __forceinline__ PairSum prob_weight(const ProbRow<ET>& r, int x, int V) {
    if (x >= V) return PairSum{0.0f, 0.0f};
    return prob_difference(ET::load1(r.p + x), r.q ? ET::load1(r.q + x) : (x == r.one_hot ? 1.0f : 0.0f));
}

// Two tokens' probabilities as the operator takes them (prob_value, and y = min(q, p)): of word k
// of a vector, two fp32 or a word's two bf16, whose maximum and minimum need one instruction.
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_words(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sub_words(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t widen_words(uint32_t w) {
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Largest power of two up to m (0 when it is zero), at most 2^120.
__device__ __forceinline__ float leading_power(float m) {
    return fminf(__uint_as_float(__float_as_uint(m) & 0x7F800000u), 0x1p120f);
}

// acc + lo += x for two tokens.  acc began at a power of two that is at least half of every x, so
// acc >= x but for rounding, (acc + x) - acc is exact, and x less that is the sum's error: four
// instructions instead of seven for values in any order (two_sum).
__device__ __forceinline__ void add_descending(uint64_t& acc, uint64_t& lo, uint64_t x) {
    const uint64_t s = add2(acc, x);
    lo = add2(lo, sub2(x, sub2(s, acc)));
    acc = s;
}

__device__ __forceinline__ PairSum warp_sum(PairSum a) {
#pragma unroll 1
    for (int off = 16; off > 0; off >>= 1)
        a = pair_plus(a, PairSum{__shfl_xor_sync(0xffffffffu, a.hi, off), __shfl_xor_sync(0xffffffffu, a.lo, off)});
    return a;
}

// The lane's part of chunk c.  kBatch: 16-byte vectors of each row in flight per lane; kTaken: the
// row has a q.
template <class ET, int kChunk, int kBatch, ChunkKind kKind, bool kTaken>
__device__ __forceinline__ PairSum lane_sum(const ProbRow<ET>& r, int c, int V, int lane) {
    PairSum sum{0.0f, 0.0f};
    uint64_t hi = 0ull, lo = 0ull;
    const int x0 = c * kChunk, end = min(V, x0 + kChunk);
#pragma unroll 1
    for (int xb = x0; xb < end; xb += kBatch * 32 * ET::kVec) {
        const int x = xb + lane * ET::kVec;
        uint4 vp[kBatch], vq[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) vq[k] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kKind == ChunkKind::kShifted) {
            load_shifted_vecs<ET>(r.p, xb, lane, vp);
            if (kTaken && r.q) load_shifted_vecs<ET>(r.q, xb, lane, vq);
        } else {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) vp[k] = load_prob_vec<ET, kKind>(r.p, x + k * 32 * ET::kVec, V);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (kTaken && r.q) vq[k] = load_prob_vec<ET, kKind>(r.q, x + k * 32 * ET::kVec, V);
        }
        uint32_t any = 0u;  // filtered rows (top-k, top-p) hold long runs of p = 0
#pragma unroll
        for (int k = 0; k < kBatch; ++k) any |= vp[k].x | vp[k].y | vp[k].z | vp[k].w;
        if (!__any_sync(0xffffffffu, any != 0u)) continue;
        uint32_t wp[kBatch * 4], wq[kBatch * 4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            wp[4 * k] = vp[k].x, wp[4 * k + 1] = vp[k].y, wp[4 * k + 2] = vp[k].z, wp[4 * k + 3] = vp[k].w;
            wq[4 * k] = vq[k].x, wq[4 * k + 1] = vq[k].y, wq[4 * k + 2] = vq[k].z, wq[4 * k + 3] = vq[k].w;
            unsigned hot = static_cast<unsigned>(r.one_hot - (x + k * 32 * ET::kVec));
            if (kKind == ChunkKind::kShifted && ET::kVec == 4) {  // (see load_shifted_vecs)
                const int from = r.one_hot - xb - lane;
                hot = from % 32 == 0 ? static_cast<unsigned>(from / 32 - 4 * k) : 4u;
            }
            if (kTaken && hot < static_cast<unsigned>(ET::kVec)) {
                constexpr unsigned kPerWord = ET::kVec / 4;
                const uint32_t one = kPerWord == 1 ? 0x3F800000u : 0x3F80u << (16 * (hot % kPerWord));
#pragma unroll
                for (unsigned e = 0; e < 4; ++e)
                    if (hot / kPerWord == e) wq[4 * k + e] = one;
            }
        }
        if constexpr (ET::kVec == 8) {
            uint32_t most = 0u;  // (a difference rounded to bf16 keeps or raises its power of two)
#pragma unroll
            for (int e = 0; e < kBatch * 4; ++e) {
                wp[e] = max_words(wp[e], 0u);
                if (kTaken) wq[e] = min_words(max_words(wq[e], 0u), wp[e]);
                most = max_words(most, kTaken ? sub_words(wp[e], wq[e]) : wp[e]);
            }
            const float start = leading_power(fmaxf(__uint_as_float(most << 16), __uint_as_float(most & 0xFFFF0000u)));
            const uint64_t start2 = pack2(start, start);
            uint64_t acc = start2;
#pragma unroll
            for (int e = 0; e < kBatch * 4; ++e) {
                const uint64_t a = widen_words(wp[e]);
                if (kTaken) {
                    const uint64_t y = widen_words(wq[e]), d = sub2(a, y);
                    add_descending(acc, lo, d);
                    lo = add2(lo, sub2(sub2(a, d), y));
                } else {
                    add_descending(acc, lo, a);
                }
            }
            PairSum a, b;
            unpack2(sub2(acc, start2), a.hi, b.hi);  // (exact)
            sum = pair_plus(sum, pair_plus(PairSum{a.hi, 0.0f}, PairSum{b.hi, 0.0f}));
        } else {
#pragma unroll
            for (int e = 0; e < kBatch * 4; e += 2)
                add_differences(hi, lo, __uint_as_float(wp[e]), __uint_as_float(wp[e + 1]), __uint_as_float(wq[e]),
                                __uint_as_float(wq[e + 1]));
        }
    }
    PairSum a, b;
    unpack2(hi, a.hi, b.hi);
    unpack2(lo, a.lo, b.lo);
    return pair_plus(sum, pair_plus(a, b));
}

// The warp's sum of w over chunk c of the row (every lane gets it).
template <class ET, int kChunk, int kBatch, ChunkKind kKind>
__device__ __forceinline__ PairSum chunk_sum_as(const ProbRow<ET>& r, int c, int V, int lane) {
    const unsigned hot = static_cast<unsigned>(r.one_hot - c * kChunk);
    if (ET::kVec == 8 && !r.q && hot >= static_cast<unsigned>(kChunk))
        return warp_sum(lane_sum<ET, kChunk, kBatch, kKind, false>(r, c, V, lane));
    return warp_sum(lane_sum<ET, kChunk, kBatch, kKind, true>(r, c, V, lane));
}

// (out of line: their branches around the loads would cost the chunks inside their row a tenth)
template <class ET, int kChunk, int kBatch, ChunkKind kKind>
__device__ __noinline__ PairSum chunk_sum_apart(const ProbRow<ET>& r, int c, int V, int lane) {
    return chunk_sum_as<ET, kChunk, kBatch, kKind>(r, c, V, lane);
}

// By one warp: among `count` weights in token order, the first whose running sum (from `base`)
// exceeds t, or the last positive one when none does (u >= 1, NaN, or rounding); `base` becomes
// the sum before it.  With from_u, t is u (>= 0) times the sum of all weights, and is returned.
// -1: every weight is zero; -2: the sum is not finite.
__device__ __noinline__ int locate(const PairSum* weights, int count, PairSum& base, PairSum& t, bool from_u, float u) {
    const int lane = threadIdx.x & 31;
    const int each = (count + 31) >> 5;
    const int lo = lane * each, hi = min(count, lo + each);
    PairSum s{0.0f, 0.0f};
#pragma unroll 1
    for (int c = lo; c < hi; ++c) s = pair_plus(s, weights[c]);
    PairSum before{0.0f, 0.0f};
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const PairSum o{__shfl_up_sync(0xffffffffu, s.hi, off), __shfl_up_sync(0xffffffffu, s.lo, off)};
        if (lane >= off) s = pair_plus(o, s);
    }
    before.hi = __shfl_up_sync(0xffffffffu, s.hi, 1);
    before.lo = __shfl_up_sync(0xffffffffu, s.lo, 1);
    if (lane == 0) before = PairSum{0.0f, 0.0f};
    const PairSum whole{__shfl_sync(0xffffffffu, s.hi, 31), __shfl_sync(0xffffffffu, s.lo, 31)};
    if (whole.hi == 0.0f) return -1;
    if (!(whole.hi > 0.0f) || !isfinite(whole.hi + whole.lo)) return -2;
    if (from_u) {  // the fma gives the product's rounding error
        t.hi = u * whole.hi;
        t.lo = fmaf(u, whole.hi, -t.hi) + u * whole.lo;
    }
    PairSum run = pair_plus(base, before), first_base{}, last_base{};
    int first = INT_MAX, last = -1;
#pragma unroll 1
    for (int c = lo; c < hi; ++c) {
        const PairSum w = weights[c], next = pair_plus(run, w);
        if (w.hi > 0.0f) {
            last = c;
            last_base = run;
            if (first == INT_MAX && pair_exceeds(next, t)) {
                first = c;
                first_base = run;
            }
        }
        run = next;
    }
    const int f = __reduce_min_sync(0xffffffffu, first), l = __reduce_max_sync(0xffffffffu, last);
    const int at = f != INT_MAX ? f : l;
    const PairSum from = f != INT_MAX ? first_base : last_base;
    base.hi = __shfl_sync(0xffffffffu, from.hi, at / each);
    base.lo = __shfl_sync(0xffffffffu, from.lo, at / each);
    return at;
}

// kBatch, kMinBlocks: loads in flight per lane, and blocks that an SM must hold (see launch_probs).
template <class ET, int kChunk, int kBatch, int kMinBlocks>
__global__ void __launch_bounds__(kProbThreads, kMinBlocks) verify_probs_kernel(ProbParams p) {
    namespace cg = cooperative_groups;
    using S = typename ET::storage;
    constexpr int kShiftedBatch = ET::kVec == 8 && kMinBlocks > 3 ? 2 : 4;
    extern __shared__ PairSum s_chunk[];  // [share] sums of this CTA's chunks
    // the total of every warp of the cluster, in token order: of the residual, of p_j
    __shared__ PairSum s_warp[2][kProbMaxCluster * kProbWarps];
    __shared__ PairSum s_part[kProbWarps], s_rest;
    __shared__ int s_j, s_owner, s_c, s_first, s_last;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // (waited for before the first store into another CTA)
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / C;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const S* target = static_cast<const S*>(p.target) + static_cast<long long>(b) * (p.gamma + 1) * p.V;
    const S* draft = static_cast<const S*>(p.draft);
    if (draft) draft += static_cast<long long>(b) * p.gamma * p.V;
    const int32_t* tokens = p.tokens + static_cast<long long>(b) * p.gamma;
    const float* uniforms = p.uniforms + static_cast<long long>(b) * (p.gamma + 1);
    int32_t* out = p.out_tokens + static_cast<long long>(b) * (p.gamma + 1);

    grid_dependency();
    // the first rejected position (every CTA of the cluster finds the same one)
    const int len = p.lens ? __ldg(p.lens + b) : p.gamma;
    const float u_draw = __ldg(uniforms + p.gamma);
    int error = (len < 0 || len > p.gamma) ? 9 /* SPEC_EBADLEN */ : 0;
    if (threadIdx.x == 0) {
        s_j = len;
        s_first = INT_MAX;
        s_last = -1;
    }
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i < p.gamma; i += kProbThreads) {
        const int d = __ldg(tokens + i);  // (read before the length is known: one wait less)
        const float u = __ldg(uniforms + i);
        if (error || i >= len) break;
        if (d < 0 || d >= p.V) {
            bad = true;
            continue;
        }
        const float pd = prob_value(ET::load1(target + static_cast<long long>(i) * p.V + d));
        const float qd = draft ? prob_value(ET::load1(draft + static_cast<long long>(i) * p.V + d)) : 1.0f;
        if (!(static_cast<double>(u) * static_cast<double>(qd) < static_cast<double>(pd))) atomicMin(&s_j, i);
    }
    if (__syncthreads_or(bad)) error = 3 /* SPEC_EBADTOKEN */;
    cluster.barrier_wait();  // every CTA of the cluster has started
    const int j = s_j;
    int owner = -1;  // the warp of the cluster whose chunks hold the drawn token
    PairSum base{0.0f, 0.0f}, t{0.0f, 0.0f};  // (warp 0) the sum before it, and u W
    ProbRow<ET> row{};
    // warp w of CTA r takes the chunks [c0 + w per, c0 + (w + 1) per) of the CTA's share
    const int n_chunks = (p.V + kChunk - 1) / kChunk;
    const int c0 = rank * p.share;
    const int n = max(0, min(p.share, n_chunks - c0));
    const int per = (p.share + kProbWarps - 1) / kProbWarps;
    if (!error) {
        const bool residual = j < len;
        row = prob_row<ET>(target + static_cast<long long>(j) * p.V,
                           residual && draft ? draft + static_cast<long long>(j) * p.V : nullptr,
                           residual && !draft ? tokens[j] : -1);
        for (int slot = 0;; ++slot) {
            PairSum sum{0.0f, 0.0f};
            for (int c = warp * per; c < min(n, (warp + 1) * per); ++c) {
                PairSum s;
                if (row.aligned && (c0 + c + 1) * kChunk <= p.V)
                    s = chunk_sum_as<ET, kChunk, kBatch, ChunkKind::kInside>(row, c0 + c, p.V, lane);
                else if (row.aligned && p.V % ET::kVec == 0)
                    s = chunk_sum_apart<ET, kChunk, kBatch, ChunkKind::kLast>(row, c0 + c, p.V, lane);
                else if ((c0 + c + 1) * kChunk + ET::kVec <= p.V)
                    s = chunk_sum_apart<ET, kChunk, kShiftedBatch, ChunkKind::kShifted>(row, c0 + c, p.V, lane);
                else
                    s = chunk_sum_apart<ET, kChunk, kBatch, ChunkKind::kOther>(row, c0 + c, p.V, lane);
                if (lane == 0) s_chunk[c] = s;
                sum = pair_plus(sum, s);
            }
            // to every CTA's copy, a lane each
            if (lane < C) *cluster.map_shared_rank(&s_warp[slot][rank * kProbWarps + warp], lane) = sum;
            cluster.sync();  // every CTA has every total
            if (warp == 0) {
                const int o = locate(s_warp[slot], C * kProbWarps, base, t, true, u_draw < 0.0f ? 0.0f : u_draw);
                if (lane == 0) s_owner = o;
            }
            __syncthreads();
            owner = s_owner;
            if (owner != -1 || !residual || slot == 1) break;
            row = prob_row<ET>(row.p, nullptr, -1);  // p <= q everywhere: the draw is from p_j
        }
        if (owner < 0) error = 8 /* SPEC_EBADPROB */;
    }
    if (rank == 0) {
        for (int i = threadIdx.x; i <= p.gamma; i += kProbThreads)
            if (error) out[i] = -1;
            else if (i != j) out[i] = i < j ? tokens[i] : -1;
        if (threadIdx.x == 0) {
            p.out_n[b] = error ? -1 : j;
            if (error) set_status(p.status, error);
        }
    }
    if (owner < 0 || owner / kProbWarps != rank) return;
    // down to that warp's chunk, then to the token
    if (warp == 0) {
        const int begin = (owner % kProbWarps) * per;
        const int c = begin + (per > 1 ? locate(s_chunk + begin, min(n, begin + per) - begin, base, t, false, 0.0f) : 0);
        if (lane == 0) {
            s_c = c0 + c;
            s_rest = pair_plus(t, PairSum{-base.hi, -base.lo});  // u W less the sum before the chunk
        }
    }
    __syncthreads();
    // every thread two or four tokens of the chunk: their sums over the block, then their places
    constexpr int kPer = kChunk / kProbThreads;
    const int x0 = s_c * kChunk + static_cast<int>(threadIdx.x) * kPer;
    PairSum w[kPer], incl, run;
    static_assert(kPer == 4 || kPer == 2, "two or four tokens a thread");
#pragma unroll
    for (int e = 0; e < kPer; ++e) w[e] = prob_weight<ET>(row, x0 + e, p.V);
    incl = pair_plus(w[0], w[1]);
    if constexpr (kPer == 4) incl = pair_plus(incl, pair_plus(w[2], w[3]));
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const PairSum o{__shfl_up_sync(0xffffffffu, incl.hi, off), __shfl_up_sync(0xffffffffu, incl.lo, off)};
        if (lane >= off) incl = pair_plus(o, incl);
    }
    run.hi = __shfl_up_sync(0xffffffffu, incl.hi, 1);
    run.lo = __shfl_up_sync(0xffffffffu, incl.lo, 1);
    if (lane == 0) run = PairSum{0.0f, 0.0f};
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    t = s_rest;
#pragma unroll 1
    for (int k = 0; k < warp; ++k) run = pair_plus(run, s_part[k]);
    int first = INT_MAX, last = -1;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        run = pair_plus(run, w[e]);
        if (w[e].hi > 0.0f) {
            last = x0 + e;
            if (first == INT_MAX && pair_exceeds(run, t)) first = last;
        }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
        atomicMin(&s_first, first);
        atomicMax(&s_last, last);
    }
    __syncthreads();
    if (threadIdx.x == 0) out[j] = s_first != INT_MAX ? s_first : s_last;
}

}  // namespace specverify
