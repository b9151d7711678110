// select.cuh -- routing by scores: expert scores of given logits, a balance bias that steers
// the selection only, expert groups, top-k, renormalised and scaled weights; and the gradient
// of the weights at the logits.
//
//   s_e   = 1 / (1 + exp(-l_e))  or  exp(l_e - m) / sum_i exp(l_i - m)   over the live experts
//           (live: l_e > -inf; -inf and NaN are masked experts with score 0)
//   key_e = s_e + bias_e; without a bias the order of s is the order of l, so key_e = l_e
//   group g (E / n_group consecutive experts): its largest key, or the sum of its two largest
//           s + bias; the top_group best groups stay, ties to the lower group
//   experts: the k largest keys of the groups that stay, ties to the lower id; masked experts
//           come last (by id) and weigh 0
//   w_j   = scale * s_j / sum_i s_i (renorm)  or  scale * s_j
//
// The selection is the one that keys in 64 bits give. Keys are first formed in 32 bits with the
// fast exponential, whose distance from the 64-bit key is bounded (SEL_TOL_*). Where every
// decision of a token was clear of that bound the 32-bit selection is the 64-bit one; otherwise
// (about 1 token in 1000 of random logits; ties) the warp selects again with 64-bit keys
// (sel_exact).
//
// One warp per token, tokens in a grid-stride loop with the next row's logits in flight; lane i
// owns the EPT consecutive experts from i * EPT. With 256 experts a row is 1 KB and the work is
// some 400 warp instructions, so the kernel is bound by instructions, not bytes, and is built to
// spend few per key:
//   - a key carries its place in the lane in its lowest log2(EPT) mantissa bits (counted in the
//     bound), so a key and its expert sort as one float: min and max, nothing else;
//   - each lane sorts its keys once (19 exchanges for 8); a round of the top-k is then one
//     redux.sync over the lanes' heads, and the winning lane drops its head;
//   - a group's two largest keys are the heads of its lanes;
//   - the checks against the bound are made once, after the rounds, on the k winners' lanes.
// bf16 logits without a bias leave 16 mantissa bits free: the key carries the whole expert id and the
// 32-bit order is exact, ties included.
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <stdint.h>

namespace moe {

constexpr int SEL_MAX_K = 32;      // one selected expert per lane
constexpr int SEL_MAX_GROUPS = 32; // one group per lane

// Bounds on the gap of two 32-bit keys whose 64-bit order could differ (both keys' errors):
// sigmoid: the exponential's (2 + 1.17 |l|) ulp through s (1 - s) is at most 7.5e-8, the sum
//   1 + e adds 2^-24 s, the quotient 2 ulp: 3.8e-7 a key, 7.6e-7 for two;
// softmax: 3.2e-7 s_max a key from the exponential, and one factor common to all keys (the sum:
//   36 rounded additions and the terms' own errors, the reciprocal) of at most 4.1e-6: 4.8e-6;
// the sum with the bias rounds by 2^-24 of the key, the place by at most EPT 2^-23 of it.
constexpr float SEL_TOL_SIGMOID = 9.5367431640625e-7f; // 2^-20
constexpr float SEL_TOL_SOFTMAX = 7.62939453125e-6f;   // 2^-17, times the largest score
constexpr float SEL_TOL_KEY = 2.384185791015625e-7f;   // 2^-22, times the key
constexpr float SEL_TOL_ZERO = 1.0e-40f;               // a place in a zero or denormal key
__host__ __device__ constexpr float SEL_PLACE(int ept) { return ept * 1.1920928955078125e-7f; } // EPT 2^-23
// Masked or excluded experts' key, and the clamp of the others; a winner at or beyond SEL_EDGE
// (also a lane whose sorted keys ran out) sends the token to sel_exact.
constexpr float SEL_FAR = 3.0e38f;
constexpr float SEL_EDGE = 2.9e38f;

struct SelectArgs {
    const void *logits; // [T, E], row stride ld (elements)
    int64_t ld;
    const float *bias;  // [E] or nullptr
    int32_t *idx;       // [T, k]
    float *w;           // [T, k]
    const int32_t *n_rows; // rows from *n_rows on are left as they are; nullptr: all T
    int T, E, k;
    int sigmoid;
    int groups, gsz, keep, sum2;
    int renorm;
    float scale;
    int vec; // rows may be read in 16-byte pieces
};

__device__ __forceinline__ float sel_load(const float *p) { return *p; }
__device__ __forceinline__ float sel_load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// finite, -inf (masked: -inf and NaN) or the largest finite value (+inf)
__device__ __forceinline__ float sel_clean(float l)
{
    return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;
}

// Order-preserving integers of 64-bit keys: 0 is no candidate, 1 a masked expert; a NaN key (a
// NaN bias) counts as -inf.
__device__ __forceinline__ unsigned long long sel_ord64(double key)
{
    if (key != key) key = -INFINITY;
    const unsigned long long u = (unsigned long long)__double_as_longlong(key + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr unsigned long long SEL_MASKED = 1ull;

__device__ __forceinline__ float sel_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sel_min(float v)
{
    float r;
    asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sel_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Whether group `lane` stays, from the groups' values (lane g holds group g's): its rank among
// the values, ties to the lower group.
template <typename V>
__device__ __forceinline__ bool sel_group_stays(V gv, int groups, int keep, int lane)
{
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const V o = __shfl_sync(0xffffffffu, gv, g);
        rank += (o > gv || (o == gv && g < lane)) ? 1 : 0;
    }
    return lane < groups && rank < keep;
}

struct SelExact {
    int mine;     // the expert selected in round `lane` (lane < k)
    float m, sum; // softmax: the row's maximum and sum
};

// The selection with keys in 64 bits. key: E order words of this warp in shared memory.
template <typename LT>
__device__ __noinline__ SelExact sel_exact(const SelectArgs &a, const LT *row, unsigned long long *key,
                                           int lane)
{
    double m = -INFINITY, sum = 0.0;
    if (!a.sigmoid) {
        for (int e = lane; e < a.E; e += 32) m = fmax(m, (double)sel_clean(sel_load(row + e)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, off));
        for (int e = lane; e < a.E; e += 32) {
            const float l = sel_clean(sel_load(row + e));
            if (l > -INFINITY) sum += exp((double)l - m);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    auto value = [&](float l, int e) -> double { // s + bias of a live expert
        const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - m) / sum;
        const double v = a.bias != nullptr ? s + (double)a.bias[e] : s;
        return v == v ? v : -INFINITY;
    };
    uint32_t stay = 0xffffffffu;
    if (a.groups > 1) {
        double gv = -INFINITY;
        if (lane < a.groups) {
            double v1 = -INFINITY, v2 = -INFINITY;
            for (int i = 0; i < a.gsz; ++i) {
                const int e = lane * a.gsz + i;
                const float l = sel_clean(sel_load(row + e));
                if (!(l > -INFINITY)) continue;
                const double v = (a.bias != nullptr || a.sum2) ? value(l, e) : (double)l;
                if (v > v1) {
                    v2 = v1;
                    v1 = v;
                } else if (v > v2) {
                    v2 = v;
                }
            }
            gv = (a.sum2 && v2 > -INFINITY) ? v1 + v2 : v1;
        }
        stay = __ballot_sync(0xffffffffu, sel_group_stays(gv, a.groups, a.keep, lane));
    }
    for (int e = lane; e < a.E; e += 32) {
        const float l = sel_clean(sel_load(row + e));
        unsigned long long o = SEL_MASKED;
        if (l > -INFINITY) o = sel_ord64(a.bias != nullptr ? value(l, e) : (double)l);
        if (a.groups > 1 && !((stay >> (e / a.gsz)) & 1u)) o = 0;
        key[e] = o;
    }
    __syncwarp();
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        unsigned long long bo = 0;
        int be = 0x7fffffff;
        for (int e = lane; e < a.E; e += 32)
            if (key[e] > bo) {
                bo = key[e];
                be = e;
            }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const unsigned long long oo = __shfl_xor_sync(0xffffffffu, bo, off);
            const int oe = __shfl_xor_sync(0xffffffffu, be, off);
            if (oo > bo || (oo == bo && oe < be)) {
                bo = oo;
                be = oe;
            }
        }
        if (be >= a.E) be = 0; // not reached: at least k experts are candidates
        if (lane == j) mine = be;
        __syncwarp();
        if (lane == 0) key[be] = 0;
        __syncwarp();
    }
    return SelExact{mine, (float)m, sum > 0.0 ? (float)sum : 1.0f};
}

// Descending order of n keys (n = 2, 4, 8), by compare-exchange of minimum and maximum.
__device__ __forceinline__ void sel_cx(float &a, float &b)
{
    const float hi = fmaxf(a, b);
    b = fminf(a, b);
    a = hi;
}
template <int N> __device__ __forceinline__ void sel_sort(float *v)
{
    if constexpr (N == 2) {
        sel_cx(v[0], v[1]);
    } else if constexpr (N == 4) {
        sel_cx(v[0], v[2]); sel_cx(v[1], v[3]);
        sel_cx(v[0], v[1]); sel_cx(v[2], v[3]);
        sel_cx(v[1], v[2]);
    } else if constexpr (N == 8) {
        sel_cx(v[0], v[2]); sel_cx(v[1], v[3]); sel_cx(v[4], v[6]); sel_cx(v[5], v[7]);
        sel_cx(v[0], v[4]); sel_cx(v[1], v[5]); sel_cx(v[2], v[6]); sel_cx(v[3], v[7]);
        sel_cx(v[0], v[1]); sel_cx(v[2], v[3]); sel_cx(v[4], v[5]); sel_cx(v[6], v[7]);
        sel_cx(v[2], v[4]); sel_cx(v[3], v[5]);
        sel_cx(v[1], v[4]); sel_cx(v[3], v[6]);
        sel_cx(v[1], v[2]); sel_cx(v[3], v[4]); sel_cx(v[5], v[6]);
    }
}
// a: the eight largest of two descending runs of eight
__device__ __forceinline__ void sel_merge8(float *a, const float *b)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = fmaxf(a[i], b[7 - i]);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) sel_cx(a[i], a[i + d]);
}

// EPT consecutive logits of a row from e0 (beyond E: -inf)
template <int EPT, typename LT>
__device__ __forceinline__ void sel_load_row(const SelectArgs &a, const LT *row, int e0, float (&l)[EPT])
{
    constexpr int PV = 16 / (int)sizeof(LT); // values in 16 bytes
    if (EPT % PV == 0 && a.vec && e0 + EPT <= a.E) {
#pragma unroll
        for (int i = 0; i < EPT / PV; ++i) {
            const uint4 u = reinterpret_cast<const uint4 *>(row + e0)[i];
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < PV; ++q) {
                if (sizeof(LT) == 4)
                    l[(i * PV + q) % EPT] = __uint_as_float(uw[q & 3]);
                else
                    l[(i * PV + q) % EPT] = __uint_as_float((q & 1) ? (uw[q >> 1] & 0xffff0000u) : (uw[q >> 1] << 16));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) l[i] = e0 + i < a.E ? sel_load(row + e0 + i) : -INFINITY;
    }
}

// A score in 32 bits: the sigmoid, or exp(l - m) / sum with inv = 1 / sum.
__device__ __forceinline__ float sel_score(int sigmoid, float l, float m, float inv)
{
    return sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l)) : __expf(l - m) * inv;
}

// A group's value from its two largest keys (SEL_FAR: none). Without a bias the keys are logits and
// a sum is formed of their scores (the order is the same).
__device__ __forceinline__ float sel_group_value(const SelectArgs &a, bool biased, float v1, float v2,
                                                 float m, float inv)
{
    if (!a.sum2 || !(v1 > -SEL_EDGE)) return v1;
    if (biased) return v2 > -SEL_EDGE ? v1 + v2 : v1;
    return sel_score(a.sigmoid, v1, m, inv) + (v2 > -SEL_EDGE ? sel_score(a.sigmoid, v2, m, inv) : 0.0f);
}

// Threads per block and blocks per SM (the launch fills the SMs once).
__host__ __device__ constexpr int sel_threads(int ept) { return ept == 32 ? 128 : 256; }
__host__ __device__ constexpr int sel_blocks(int ept) { return ept <= 4 ? 4 : ept == 16 ? 2 : 3; }

// Dynamic shared memory, per warp: E 8-byte words (sel_exact's keys; the values of odd-sized
// groups), then 34 8-byte words (the rounds' winners).
template <int EPT, typename LT, bool BIASED>
__global__ void __launch_bounds__(sel_threads(EPT), sel_blocks(EPT)) route_select_kernel(const __grid_constant__ SelectArgs a)
{
    constexpr bool EXACT = !BIASED && (EPT == 1 || sizeof(LT) == 2); // keys order as 64 bits would
    constexpr bool IDS = EXACT && EPT > 1;                           // keys carry expert ids
    constexpr int D = EPT < 8 ? EPT : 8;                             // sorted keys kept per lane
    constexpr float TOL_KEY = EPT == 1 ? SEL_TOL_KEY : SEL_TOL_KEY + SEL_PLACE(EPT);
    extern __shared__ unsigned long long sel_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    unsigned long long *scratch = sel_smem + (size_t)warp * (a.E + 34);
    uint2 *pick = reinterpret_cast<uint2 *>(scratch + a.E);
    const int T = a.n_rows != nullptr ? min(a.T, *a.n_rows) : a.T;
    const int e0 = lane * EPT;
    const uint32_t below = (1u << lane) - 1u;
    const int step = gridDim.x * warps;
    int t = blockIdx.x * warps + warp;
    if (t >= T) return;

    const bool sums = a.groups > 1 && a.sum2;
    const bool need_sum = !a.sigmoid && (BIASED || sums || !a.renorm);
    const int lanes = a.groups > 1 ? a.gsz / EPT : 1; // lanes of a group, where it is whole lanes
    const bool whole = a.groups > 1 && a.gsz % EPT == 0 && (lanes & (lanes - 1)) == 0;
    const int my_group = whole ? lane / lanes : 0;
    float bias[BIASED && EPT <= 8 ? EPT : 1];
    if (BIASED && EPT <= 8) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) bias[i % (int)(sizeof(bias) / 4)] = e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
    }
    float next[EPT];
    sel_load_row(a, static_cast<const LT *>(a.logits) + (size_t)t * a.ld, e0, next);

    for (; t < T; t += step) {
        const LT *row = static_cast<const LT *>(a.logits) + (size_t)t * a.ld;
        float v[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) v[i] = fminf(fmaxf(next[i], -SEL_FAR), SEL_FAR); // NaN: masked
        if (t + step < T) sel_load_row(a, row + (size_t)step * a.ld, e0, next);
        bool bad = false;

        // softmax: the row's maximum and sum where anything but the order is needed
        float m = 0.0f, sum = 1.0f;
        if (need_sum) {
            m = v[0];
#pragma unroll
            for (int i = 1; i < EPT; ++i) m = fmaxf(m, v[i]);
            m = sel_max(m);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < EPT; ++i) s += __expf(v[i] - m);
            sum = sel_sum(s);
            bad = !(fabsf(m) < SEL_EDGE);
        }
        const float inv = __fdividef(1.0f, sum);
        if (BIASED) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const float b = EPT <= 8 ? bias[i % (int)(sizeof(bias) / 4)] : (e0 + i < a.E ? a.bias[e0 + i] : 0.0f);
                const float key = fminf(fmaxf(sel_score(a.sigmoid, v[i], m, inv) + b, -SEL_FAR), SEL_FAR);
                v[i] = v[i] > -SEL_EDGE ? key : -SEL_FAR;
            }
        }
        float tol = a.sigmoid ? SEL_TOL_SIGMOID : SEL_TOL_SOFTMAX * inv;
        if (!BIASED && sums) {
            // the scores of a group's two largest logits, each off by its place's EPT 2^-23 |l|
            // through the score's slope: |l| s (1 - s) < 0.23, |l| s < (|m| + 1) / sum
            tol += (a.sigmoid ? 1.0f : 2.0f * (fabsf(m) + 1.0f) * inv) * SEL_PLACE(EPT);
        }

        float gv = 0.0f;
        uint32_t stay = 0xffffffffu; // odd-sized groups: bit g
        if (a.groups > 1 && !whole) {
            // the keys through shared memory, lane g walks group g
            float *sv = reinterpret_cast<float *>(scratch);
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (e0 + i < a.E) sv[e0 + i] = v[i];
            __syncwarp();
            float v1 = -SEL_FAR, v2 = -SEL_FAR;
            if (lane < a.groups)
                for (int i = 0; i < a.gsz; ++i) {
                    const float x = sv[lane * a.gsz + i];
                    v2 = fmaxf(v2, fminf(v1, x));
                    v1 = fmaxf(v1, x);
                }
            __syncwarp();
            gv = sel_group_value(a, BIASED, v1, v2, m, inv);
            const bool st = sel_group_stays(gv, a.groups, a.keep, lane);
            stay = __ballot_sync(0xffffffffu, st);
            const float lo = sel_min(st ? gv : SEL_FAR), hi = sel_max(!st && lane < a.groups ? gv : -SEL_FAR);
            if ((BIASED || sums) && hi > -SEL_FAR && !(lo - hi > 2.0f * tol + SEL_TOL_KEY * (fabsf(lo) + fabsf(hi))))
                bad = true;
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (!((stay >> min((e0 + i) / a.gsz, 31)) & 1u)) v[i] = -SEL_FAR;
        }

        // the place (or id) into the lowest bits, then each lane's keys in descending order
        if (IDS) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) { // larger bits are larger for a positive key only
                const uint32_t u = __float_as_uint(v[i] + 0.0f) & 0xffff0000u;
                v[i] = __uint_as_float(u | (uint32_t)((u >> 31) ? e0 + i : 1023 - e0 - i));
            }
        } else if (EPT > 1) {
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                v[i] = __uint_as_float((__float_as_uint(v[i]) & ~(uint32_t)(EPT - 1)) | (uint32_t)i);
        }
        if constexpr (EPT <= 8) {
            sel_sort<EPT>(v);
        } else {
#pragma unroll
            for (int c = 0; c < EPT / 8; ++c) sel_sort<8>(v + 8 * c);
#pragma unroll
            for (int c = 1; c < EPT / 8; ++c) sel_merge8(v, v + 8 * c);
        }

        if (whole) {
            float v1 = v[0], v2 = EPT > 1 ? v[EPT > 1 ? 1 : 0] : -SEL_FAR;
            if (IDS) {
                v1 = __uint_as_float(__float_as_uint(v1) & 0xffff0000u);
                v2 = __uint_as_float(__float_as_uint(v2) & 0xffff0000u);
            }
            for (int off = 1; off < lanes; off <<= 1) {
                const float o1 = __shfl_xor_sync(0xffffffffu, v1, off);
                const float o2 = __shfl_xor_sync(0xffffffffu, v2, off);
                v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
                v1 = fmaxf(v1, o1);
            }
            gv = sel_group_value(a, BIASED, v1, v2, m, inv);
            // the group's rank: its lanes compare with the groups c, c + lanes, ... and add up
            int rank = 0;
            for (int g0 = 0; g0 < a.groups; g0 += lanes) { // every lane takes every turn
                const int g = g0 + (lane & (lanes - 1));
                const float o = __shfl_sync(0xffffffffu, gv, min(g, a.groups - 1) * lanes);
                if (g < a.groups) rank += (o > gv || (o == gv && g < my_group)) ? 1 : 0;
            }
            for (int off = 1; off < lanes; off <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, off);
            const bool in = my_group < a.groups, st = in && rank < a.keep;
            if (!EXACT || sums) {
                const float lo = sel_min(st ? gv : SEL_FAR), hi = sel_max(in && !st ? gv : -SEL_FAR);
                if (hi > -SEL_EDGE && !(lo - hi > (BIASED || sums ? 2.0f * tol : 0.0f) + TOL_KEY * (fabsf(lo) + fabsf(hi)) + SEL_TOL_ZERO))
                    bad = true;
            }
            if (!st) v[0] = -SEL_FAR;
        }

        const int rounds = EXACT ? a.k : a.k + 1; // one more: the best that is left out
#pragma unroll 1
        for (int j = 0; j < rounds; ++j) {
            const float top = sel_max(v[0]);
            const bool head = v[0] == top;
            const uint32_t all = __ballot_sync(0xffffffffu, head);
            if (head && !(all & below)) {
                pick[j] = make_uint2(__float_as_uint(top), (uint32_t)lane);
#pragma unroll
                for (int i = 0; i + 1 < D; ++i) v[i] = v[i + 1];
                // a lane that gave all its experts has no more; one that kept eight of more might
                v[D - 1] = EPT > D ? SEL_FAR : -SEL_FAR;
            }
        }
        __syncwarp();
        int mine = 0;
        const bool on = lane < a.k;
        if (on) {
            const uint2 p = pick[lane];
            const float key = __uint_as_float(p.x);
            if (!(fabsf(key) < SEL_EDGE)) bad = true;
            if (!EXACT) {
                const float after = __uint_as_float(pick[lane + 1].x);
                if (!(key - after > (BIASED ? tol : 0.0f) + TOL_KEY * (fabsf(key) + fabsf(after)) + SEL_TOL_ZERO)) bad = true;
            }
            if (IDS)
                mine = (p.x >> 31) ? (int)(p.x & 0xffffu) : 1023 - (int)(p.x & 0xffffu);
            else
                mine = (int)p.y * EPT + (EPT > 1 ? (int)(p.x & (uint32_t)(EPT - 1)) : 0);
        }
        __syncwarp(); // pick and scratch are free for the next token
        if (__any_sync(0xffffffffu, bad)) {
            const SelExact x = sel_exact(a, row, scratch, lane);
            mine = x.mine;
            m = x.m;
            sum = x.sum;
            __syncwarp();
        }

        // weights, once for the k selected on lanes 0 .. k - 1
        const float lj = on ? sel_clean(sel_load(row + mine)) : -INFINITY;
        const bool live = lj > -INFINITY;
        float u = 0.0f;
        if (a.sigmoid) {
            const float mn = fminf(lj, 0.0f);
            const float M = a.renorm ? sel_max(live ? mn : -INFINITY) : 0.0f; // keeps tiny scores' ratios
            if (live) u = __fdividef(expf(mn - M), 1.0f + expf(-fabsf(lj)));
        } else {
            const float M = a.renorm ? sel_max(lj) : m;
            if (live) u = a.renorm ? expf(lj - M) : __fdividef(expf(lj - M), sum);
        }
        if (a.renorm) {
            const float total = sel_sum(u);
            u = total > 0.0f ? __fdividef(u, total) : 0.0f;
        }
        if (on) {
            a.idx[(size_t)t * a.k + lane] = mine;
            a.w[(size_t)t * a.k + lane] = a.scale * u;
        }
    }
}

struct SelectBwdArgs {
    const void *logits; // [T, E], row stride ld
    int64_t ld;
    const int32_t *idx; // [T, k]
    const float *dw;    // [T, k]
    void *dlogits;      // [T, E] of the logits' type, row stride ldd
    int64_t ldd;
    const int32_t *n_rows;
    int T, E, k;
    int sigmoid, renorm;
    float scale;
    int vec; // rows of dlogits may be written in 16-byte pieces
};

__device__ __forceinline__ void sel_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void sel_store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// dL/dl of one token's weights, the selection held fixed, g_j = dL/dw_j and q_j = w_j / scale:
//   renorm, sigmoid:  dl_j = scale q_j (1 - s_j) (g_j - sum_i g_i q_i)
//   renorm, softmax:  dl_j = scale q_j (g_j - sum_i g_i q_i)
//   sigmoid:          dl_j = scale g_j s_j (1 - s_j)
//   softmax:          dl_e = scale p_e ([e = e_j] g_j - sum_i g_i p_i) for every live e
// and 0 elsewhere. One warp per token: the row is filled first, then the first k lanes write
// their experts' values (an id given twice gets the sum; an id outside [0, E) is skipped).
// Bound by the T E values written.
template <typename LT>
__global__ void __launch_bounds__(256) route_select_bwd_kernel(const __grid_constant__ SelectBwdArgs a)
{
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= a.T || (a.n_rows != nullptr && t >= *a.n_rows)) return;
    const LT *row = static_cast<const LT *>(a.logits) + (size_t)t * a.ld;
    LT *out = static_cast<LT *>(a.dlogits) + (size_t)t * a.ldd;
    const bool on = lane < a.k;
    const int id = on ? a.idx[(size_t)t * a.k + lane] : -1;
    const bool ok = id >= 0 && id < a.E;
    const float lj = ok ? sel_clean(sel_load(row + id)) : -INFINITY;
    const float g = ok ? a.scale * a.dw[(size_t)t * a.k + lane] : 0.0f;
    const bool live = lj > -INFINITY;

    float m = 0.0f, sum = 1.0f;
    const bool dense = !a.sigmoid && !a.renorm;
    if (dense) {
        m = -INFINITY;
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, sel_clean(sel_load(row + e)));
        m = sel_max(m);
        float s = 0.0f;
        for (int e = lane; e < a.E; e += 32) {
            const float l = sel_clean(sel_load(row + e));
            if (l > -INFINITY) s += expf(l - m);
        }
        sum = sel_sum(s);
        if (sum == 0.0f) sum = 1.0f;
    }
    float u = 0.0f, rest = 1.0f; // score up to the common factor; 1 - s of a sigmoid
    if (a.sigmoid) {
        const float mn = fminf(lj, 0.0f);
        const float M = a.renorm ? sel_max(live ? mn : -INFINITY) : 0.0f;
        const float d = 1.0f + expf(-fabsf(lj));
        if (live) {
            u = expf(mn - M) / d;
            rest = expf(fminf(-lj, 0.0f)) / d;
        }
    } else {
        const float M = a.renorm ? sel_max(lj) : m;
        if (live) u = a.renorm ? expf(lj - M) : expf(lj - M) / sum;
    }
    float dot = 0.0f;
    if (a.renorm) {
        const float total = sel_sum(u);
        u = total > 0.0f ? u / total : 0.0f;
    }
    if (a.renorm || dense) dot = sel_sum(u > 0.0f ? g * u : 0.0f);
    float d = 0.0f;
    if (u > 0.0f) d = dense ? g * u : u * rest * (g - dot);
    // an id given twice: each of its slots writes the sum of both
    float tot = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int oi = __shfl_sync(0xffffffffu, id, j);
        const float od = __shfl_sync(0xffffffffu, d, j);
        if (oi == id) tot += od;
    }
    if (dense) {
        for (int e = lane; e < a.E; e += 32) {
            const float l = sel_clean(sel_load(row + e));
            sel_store(out + e, l > -INFINITY ? -(expf(l - m) / sum) * dot : 0.0f);
        }
        tot -= u * dot;
    } else if (a.vec) {
        constexpr int PV = 16 / (int)sizeof(LT);
        for (int i = lane; i < a.E / PV; i += 32)
            reinterpret_cast<uint4 *>(out)[i] = make_uint4(0u, 0u, 0u, 0u);
    } else {
        for (int e = lane; e < a.E; e += 32) sel_store(out + e, 0.0f);
    }
    __syncwarp(); // the fill above is written before the selected experts' values
    if (ok) sel_store(out + id, tot);
}

} // namespace moe
