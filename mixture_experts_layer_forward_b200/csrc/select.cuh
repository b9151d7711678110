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
// the warp forms the token's keys again in 64 bits (sel_exact). Without a bias, and without
// sums over groups, the keys are the logits themselves and no bound is needed.
//
// One warp per token; lane i owns the EPT consecutive experts from i * EPT, so the lowest lane
// with the largest key holds the lowest expert id. k rounds: the lanes' own maxima (as
// order-preserving unsigned integers) meet in one redux.sync, the first lane that holds it
// gives up that expert. The weights are computed once for all k on the first k lanes.
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
// the sum with the bias rounds by 2^-24 of the key.
constexpr float SEL_TOL_SIGMOID = 9.5367431640625e-7f; // 2^-20
constexpr float SEL_TOL_SOFTMAX = 7.62939453125e-6f;   // 2^-17, times the largest score
constexpr float SEL_TOL_KEY = 2.384185791015625e-7f;   // 2^-22, times the key

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

// Order-preserving integers of keys. 0 is no candidate, 1 a masked expert; a NaN key (a NaN
// bias) counts as -inf.
__device__ __forceinline__ uint32_t sel_ord(float key)
{
    if (key != key) key = -INFINITY;
    const uint32_t u = __float_as_uint(key + 0.0f); // -0 and +0 are equal keys
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sel_unord(uint32_t o)
{
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ unsigned long long sel_ord64(double key)
{
    if (key != key) key = -INFINITY;
    const unsigned long long u = (unsigned long long)__double_as_longlong(key + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint32_t SEL_MASKED = 1u;
constexpr uint32_t SEL_NEG_INF = 0x007fffffu; // sel_ord(-inf)

__device__ __forceinline__ float sel_max(float v)
{
    return sel_unord(__reduce_max_sync(0xffffffffu, sel_ord(v)));
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

// The selection with keys in 64 bits. key: E order words of this warp in shared memory.
// Returns the expert selected in round `lane` (lane < k).
template <typename LT>
__device__ __noinline__ int sel_exact(const SelectArgs &a, const LT *row, unsigned long long *key,
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
    return mine;
}

// Dynamic shared memory: per warp E order words (sel_exact; the group values' scratch).
template <int EPT, typename LT>
__global__ void __launch_bounds__(256) route_select_kernel(const __grid_constant__ SelectArgs a)
{
    extern __shared__ unsigned long long sel_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= a.T || (a.n_rows != nullptr && t >= *a.n_rows)) return;
    const LT *row = static_cast<const LT *>(a.logits) + (size_t)t * a.ld;
    unsigned long long *scratch = sel_smem + (size_t)warp * a.E;
    const int e0 = lane * EPT;
    constexpr int PV = 16 / (int)sizeof(LT); // values in 16 bytes

    float l[EPT];
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
#pragma unroll
    for (int i = 0; i < EPT; ++i) l[i] = sel_clean(l[i]);

    const bool biased = a.bias != nullptr;
    const bool sum2 = a.groups > 1 && a.sum2;
    // softmax: the row's maximum and sum where anything but the order is needed
    float m = 0.0f, sum = 1.0f;
    if (!a.sigmoid && (biased || sum2 || !a.renorm)) {
        m = l[0];
#pragma unroll
        for (int i = 1; i < EPT; ++i) m = fmaxf(m, l[i]);
        m = sel_max(m);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) s += l[i] > -INFINITY ? __expf(l[i] - m) : 0.0f;
        sum = sel_sum(s);
        if (sum == 0.0f) sum = 1.0f; // every expert masked
    }
    const float inv = 1.0f / sum;
    float v[EPT]; // key, or s + bias where sums over groups need it
    if (biased || sum2) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            float s = a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l[i])) : __expf(l[i] - m) * inv;
            if (biased && e0 + i < a.E) s += a.bias[e0 + i];
            v[i] = s == s ? s : -INFINITY;
            if (!(l[i] > -INFINITY)) v[i] = -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) v[i] = l[i];
    }
    const float tol = a.sigmoid ? SEL_TOL_SIGMOID : SEL_TOL_SOFTMAX * inv;
    bool clear = true;

    bool stays = true; // this lane's experts (fast form), or bit g of stay_mask
    uint32_t stay_mask = 0xffffffffu;
    bool by_mask = false;
    if (a.groups > 1) {
        const int lanes = a.gsz / EPT;
        float gv;
        if (a.gsz % EPT == 0 && (lanes & (lanes - 1)) == 0) {
            // a group is `lanes` (a power of two) whole lanes: its two largest by butterflies
            float v1 = v[0], v2 = -INFINITY;
#pragma unroll
            for (int i = 1; i < EPT; ++i) {
                v2 = fmaxf(v2, fminf(v1, v[i]));
                v1 = fmaxf(v1, v[i]);
            }
            for (int off = 1; off < lanes; off <<= 1) {
                const float o1 = __shfl_xor_sync(0xffffffffu, v1, off);
                const float o2 = __shfl_xor_sync(0xffffffffu, v2, off);
                v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
                v1 = fmaxf(v1, o1);
            }
            gv = (sum2 && v2 > -INFINITY) ? v1 + v2 : v1;
            gv = __shfl_sync(0xffffffffu, gv, lane < a.groups ? lane * lanes : 0);
            by_mask = false;
        } else {
            // any other size: the values through shared memory, lane g walks group g
            float *sv = reinterpret_cast<float *>(scratch);
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (e0 + i < a.E) sv[e0 + i] = v[i];
            __syncwarp();
            float v1 = -INFINITY, v2 = -INFINITY;
            if (lane < a.groups)
                for (int i = 0; i < a.gsz; ++i) {
                    const float x = sv[lane * a.gsz + i];
                    v2 = fmaxf(v2, fminf(v1, x));
                    v1 = fmaxf(v1, x);
                }
            __syncwarp();
            gv = (sum2 && v2 > -INFINITY) ? v1 + v2 : v1;
            by_mask = true;
        }
        const bool st = sel_group_stays(gv, a.groups, a.keep, lane);
        stay_mask = __ballot_sync(0xffffffffu, st);
        if ((biased || sum2) && a.keep < a.groups) {
            // the border between the groups that stay and the others
            const float lo = sel_unord(__reduce_min_sync(0xffffffffu, st ? sel_ord(gv) : 0xffffffffu));
            const float hi = sel_unord(__reduce_max_sync(
                0xffffffffu, (!st && lane < a.groups) ? sel_ord(gv) : SEL_NEG_INF));
            const float bound = 2.0f * tol + SEL_TOL_KEY * (fabsf(lo) + fabsf(hi));
            if (hi > -INFINITY && !(lo - hi > bound)) clear = false;
        }
        if (!by_mask) stays = (stay_mask >> min(e0 / a.gsz, 31)) & 1u;
    }

    uint32_t o[EPT];
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const bool live = l[i] > -INFINITY;
        o[i] = live ? sel_ord(biased ? v[i] : l[i]) : SEL_MASKED;
        bool cand = stays && e0 + i < a.E;
        if (by_mask && cand) cand = (stay_mask >> ((e0 + i) / a.gsz)) & 1u;
        if (!cand) o[i] = 0;
        best = max(best, o[i]);
    }

    int mine = 0;
    float prev = 0.0f;
    const int rounds = biased ? a.k + 1 : a.k;
    for (int j = 0; j < rounds && clear; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int src = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        if (biased) {
            const float cur = sel_unord(top);
            if (j > 0 && top > SEL_NEG_INF && !(prev - cur > tol + SEL_TOL_KEY * (fabsf(prev) + fabsf(cur))))
                clear = false;
            prev = cur;
        }
        int e = 0;
        if (lane == src) {
            uint32_t nb = 0;
            bool found = false;
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                if (!found && o[i] == top) {
                    found = true;
                    e = e0 + i;
                    o[i] = 0;
                }
                nb = max(nb, o[i]);
            }
            best = nb;
        }
        e = __shfl_sync(0xffffffffu, e, src);
        if (lane == j) mine = e;
    }
    if (!clear) mine = sel_exact(a, row, scratch, lane);

    // weights, once for the k selected on lanes 0 .. k - 1
    const bool on = lane < a.k;
    const float lj = on ? sel_clean(sel_load(row + mine)) : -INFINITY;
    const bool live = lj > -INFINITY;
    float u = 0.0f;
    if (a.sigmoid) {
        const float mn = fminf(lj, 0.0f);
        const float M = a.renorm ? sel_max(live ? mn : -INFINITY) : 0.0f; // keeps tiny scores' ratios
        if (live) u = expf(mn - M) / (1.0f + expf(-fabsf(lj)));
    } else {
        const float M = a.renorm ? sel_max(lj) : m;
        if (live) u = a.renorm ? expf(lj - M) : expf(lj - M) / sum;
    }
    if (a.renorm) {
        const float total = sel_sum(u);
        u = total > 0.0f ? u / total : 0.0f;
    }
    if (on) {
        a.idx[(size_t)t * a.k + lane] = mine;
        a.w[(size_t)t * a.k + lane] = a.scale * u;
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
