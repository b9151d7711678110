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
// decision of a token was clear of that bound the 32-bit selection is the 64-bit one. Otherwise
// (about 5 tokens in 1000 of random fp32 logits) the groups' values, or the k + 1 winners' keys, are
// formed again in 64 bits and ordered by them; and where that does not settle it (ties around the
// last place, masked or infinite winners) the warp selects from scratch with 64-bit keys
// (sel_exact: some 10 us for a token, and the launch waits for it).
// Measured on the device: 16384 tokens, 256 experts in 8 groups, fp32, bias: 13 to 15 us (2.6 us of
// bytes at the measured copy rate), and 18 to 21 in one random batch of eight, where a token selects
// from scratch. Ties: bf16 logits with a bias of 0 (five of six warps settle winners in 64 bits, one
// token in 42 selects from scratch) 39 us, all logits equal 103 us. 8192 tokens, 64 experts, bf16:
// 3.8 us; one token: 3.7 us, 14 with all logits equal.
//
// LPT lanes per token (a warp, or eight lanes: four tokens per warp); lane i owns the EPT
// consecutive experts from i * EPT. With 256 experts a row is 1 KB and a token of a batch takes 386
// warp instructions with eight lanes, so the kernel is bound by instructions and their latency, not
// bytes, and is built to spend few per key:
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
// sigmoid: e = 2^(-l log2 e) is off by 2^-22.5 + 1.5 |l| 2^-24 of itself, which s (1 - s) takes to
//   at most 6.3e-8; the sum 1 + e adds 2^-24 s, the reciprocal 2^-23 s: 2.5e-7 a key, 5e-7 for two;
// softmax: 3.2e-7 s_max a key from the exponential, and one factor common to all keys (the sum:
//   36 rounded additions and the terms' own errors, the reciprocal) of at most 4.1e-6: 4.8e-6;
// the sum with the bias rounds by 2^-24 of the key, the place by at most EPT 2^-23 of it.
constexpr float SEL_TOL_SIGMOID = 9.5367431640625e-7f; // 2^-20
constexpr float SEL_TOL_SOFTMAX = 7.62939453125e-6f;   // 2^-17, times the largest score
constexpr float SEL_TOL_KEY = 2.384185791015625e-7f;   // 2^-22, times the key
constexpr float SEL_TOL_ZERO = 1.0e-40f;               // a place in a zero or denormal key
__host__ __device__ constexpr float SEL_PLACE(int ept) { return ept * 1.1920928955078125e-7f; } // EPT 2^-23
// Masked or excluded experts' key, and the clamp of the others; a winner at or beyond SEL_EDGE
// (also a lane whose sorted keys ran out) sends the token to sel_exact. A live expert's key is clamped
// at -SEL_LOW where a group's sum has to tell it from a masked one: keys below -SEL_NONE (places and
// ids in their lowest bits included) are no experts.
constexpr float SEL_FAR = 3.0e38f;
constexpr float SEL_NONE = 2.97e38f;
constexpr float SEL_LOW = 2.95e38f;
constexpr float SEL_EDGE = 2.9e38f;
constexpr float SEL_BIG = 1.0e38f; // a biased sum with a key at or beyond this: sel_exact

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
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// 2^x and 1 / x as the special function unit gives them (2^-22.5 and 2^-23 relative, denormal
// results 0)
__device__ __forceinline__ float sel_ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sel_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float SEL_LOG2E = 1.4426950408889634f;

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

// s + bias of a sigmoid score in 64 bits (a NaN bias: -inf)
__device__ __noinline__ double sel_value64(float l, float b)
{
    const double v = 1.0 / (1.0 + exp(-(double)l)) + (double)b;
    return v == v ? v : -INFINITY;
}

struct SelExact {
    int mine;     // the expert selected in round `lane` (lane < k)
    float m, sum; // softmax: the row's maximum and sum
};

// Over the LPT lanes of a token.
template <int LPT> __device__ __forceinline__ float sel_max_of(float v)
{
    if constexpr (LPT == 32) {
        return sel_max(v);
    } else {
#pragma unroll
        for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        return v;
    }
}
template <int LPT> __device__ __forceinline__ float sel_min_of(float v)
{
    return -sel_max_of<LPT>(-v);
}
template <int LPT> __device__ __forceinline__ float sel_sum_of(float v)
{
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

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
        const float b = a.bias != nullptr ? a.bias[e] : 0.0f;
        if (a.sigmoid) return sel_value64(l, b);
        const double v = exp((double)l - m) / sum + (double)b;
        return v == v ? v : -INFINITY;
    };
    // first the values (s + bias; without a bias and sums, the logits), for the groups
    const bool plain = a.bias == nullptr && !a.sum2;
    uint32_t stay = 0xffffffffu;
    if (a.groups > 1) {
        double *val = reinterpret_cast<double *>(key);
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) {
            const float l = sel_clean(sel_load(row + e));
            val[e] = !(l > -INFINITY) ? -INFINITY : plain ? (double)l : value(l, e);
        }
        __syncwarp();
        // `per` lanes (a power of two) walk a group's values, then add their findings
        int per = 1;
        while (per * 2 * a.groups <= 32) per *= 2;
        const int g = lane / per;
        double v1 = -INFINITY, v2 = -INFINITY;
        if (g < a.groups)
            for (int i = lane & (per - 1); i < a.gsz; i += per) {
                const double v = val[g * a.gsz + i];
                v2 = fmax(v2, fmin(v1, v));
                v1 = fmax(v1, v);
            }
        for (int off = 1; off < per; off <<= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, v1, off);
            const double o2 = __shfl_xor_sync(0xffffffffu, v2, off);
            v2 = fmax(fmin(v1, o1), fmax(v2, o2));
            v1 = fmax(v1, o1);
        }
        double gv = (a.sum2 && v2 > -INFINITY) ? v1 + v2 : v1;
        gv = __shfl_sync(0xffffffffu, gv, min(lane * per, 31)); // lane g: group g's
        stay = __ballot_sync(0xffffffffu, sel_group_stays(gv, a.groups, a.keep, lane));
        __syncwarp();
    }
    // then the order words; a lane's experts are lane, lane + 32, ...
    unsigned long long bo = 0;
    int be = lane;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) {
        const float l = sel_clean(sel_load(row + e));
        unsigned long long o = SEL_MASKED;
        if (l > -INFINITY)
            o = sel_ord64(a.bias == nullptr ? (double)l
                          : a.groups > 1    ? reinterpret_cast<double *>(key)[e]
                                            : value(l, e));
        if (a.groups > 1 && !((stay >> (e / a.gsz)) & 1u)) o = 0;
        key[e] = o;
        if (o > bo) {
            bo = o;
            be = e;
        }
    }
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        // the largest word, its two halves in turn, then the lowest id that has it
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(bo >> 32));
        const bool h = (uint32_t)(bo >> 32) == hi;
        const uint32_t lo = __reduce_max_sync(0xffffffffu, h ? (uint32_t)bo : 0u);
        const int win = (int)__reduce_min_sync(0xffffffffu, h && (uint32_t)bo == lo ? (uint32_t)be : 0x7fffffffu);
        if (lane == j) mine = win;
        if (be == win) { // its lane looks for its next
            key[win] = 0;
            bo = 0;
            for (int e = lane; e < a.E; e += 32)
                if (key[e] > bo) {
                    bo = key[e];
                    be = e;
                }
            if (bo == 0) be = lane;
        }
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

// a finite bias: beyond SEL_EDGE sel_exact decides; -inf (and NaN, which counts as it) is as good as
// a mask, but a finite one is not: it brings its group's sum down
__device__ __forceinline__ float sel_bias(float b)
{
    return b > -INFINITY ? fminf(fmaxf(b, -SEL_LOW), SEL_FAR) : -SEL_FAR;
}

// the expert id that an IDS key carries
__device__ __forceinline__ int sel_id(float key)
{
    const uint32_t u = __float_as_uint(key);
    return (u >> 31) ? (int)(u & 0xffffu) : 1023 - (int)(u & 0xffffu);
}

// A score in 32 bits: the sigmoid, or exp(l - m) / sum with inv = 1 / sum (the place in l's lowest
// bits may take it past m, and a large one past what an exponential holds).
__device__ __forceinline__ float sel_score(int sigmoid, float l, float m, float inv)
{
    return sigmoid ? sel_rcp(1.0f + sel_ex2(l * -SEL_LOG2E)) : sel_ex2(fminf(l - m, 0.0f) * SEL_LOG2E) * inv;
}

// A group's value from its two largest keys (-SEL_FAR: none). Without a bias the keys are logits and
// a sum is formed of their scores (the order is the same). bad: a sum that 32 bits may not hold, or one
// with a clamped key.
__device__ __forceinline__ float sel_group_value(const SelectArgs &a, bool biased, float v1, float v2,
                                                 float m, float inv, bool &bad)
{
    if (!a.sum2 || !(v1 > -SEL_NONE)) return v1;
    if (biased) {
        if (!(v2 > -SEL_NONE)) return v1;
        if (!(v1 < SEL_BIG && v2 > -SEL_BIG)) bad = true;
        return v1 + v2;
    }
    return sel_score(a.sigmoid, v1, m, inv) + (v2 > -SEL_NONE ? sel_score(a.sigmoid, v2, m, inv) : 0.0f);
}

// What a group's value may be off by beyond its scores' own bounds, relative to its keys, not to their
// sum: the two of a biased sum may cancel. (The sums with the biases, the keys' sum, this bound's and the
// values' difference round by 2^-24 each: together SEL_TOL_KEY.)
__device__ __forceinline__ float sel_group_error(const SelectArgs &a, bool biased, float tol_key, float gv,
                                                 float v1, float v2)
{
    const bool sum = biased && a.sum2 && v2 > -SEL_NONE;
    return sum ? tol_key * fabsf(v1) + tol_key * fabsf(v2) : tol_key * fabsf(gv);
}

// Threads per block and blocks per SM (the launch fills the SMs once).
__host__ __device__ constexpr int sel_threads(int lpt, int ept) { return ept == 32 ? 128 : 256; }
__host__ __device__ constexpr int sel_blocks(int lpt, int ept)
{
    return ept == 32 ? (lpt == 8 ? 6 : 3) : lpt == 8 || ept <= 4 ? 4 : ept == 16 ? 2 : 3;
}
// The bias in shared memory: lane i's EPT values, then (from 4) 4 more, so that 16-byte reads of
// eight lanes meet no bank twice.
__host__ __device__ constexpr int sel_bias_ld(int ept) { return ept >= 4 ? ept + 4 : ept; }
// Per warp: 8-byte words of scratch (64-bit keys; the values of odd-sized groups; with LPT = 8 and
// EPT >= 4 the rows of its four tokens, laid out as the bias), then 40 of the rounds' winners (up to
// LPT + 2 per token).
__host__ __device__ constexpr int sel_scratch(int lpt, int ept, int E)
{
    const int rows = lpt == 8 && ept >= 4 ? 16 * sel_bias_ld(ept) : 40; // 4 tokens x 8 lanes x ld floats
    return rows > E ? rows : E; // at least 40: the winners' 64-bit keys
}
__host__ __device__ constexpr int sel_smem(int lpt, int ept, int warps, int E, bool biased)
{
    return (biased ? lpt * sel_bias_ld(ept) * 4 : 0) + warps * (sel_scratch(lpt, ept, E + (E & 1)) + 40) * 8;
}

// LPT lanes per token (32, or 8: four tokens per warp), E <= LPT * EPT, k <= LPT. With LPT = 8 groups are
// whole lanes, a power of two of them, or there are none.
template <int LPT, int EPT, typename LT, bool BIASED>
__global__ void __launch_bounds__(sel_threads(LPT, EPT), sel_blocks(LPT, EPT))
    route_select_kernel(const __grid_constant__ SelectArgs a)
{
    constexpr bool EXACT = !BIASED && (EPT == 1 || sizeof(LT) == 2); // keys order as 64 bits would
    constexpr bool IDS = EXACT && EPT > 1;                           // keys carry expert ids
    constexpr int D = EPT < 8 ? EPT : 8;                             // sorted keys kept per lane
    constexpr float TOL_KEY = EPT == 1 ? SEL_TOL_KEY : SEL_TOL_KEY + SEL_PLACE(EPT);
    constexpr int BLD = sel_bias_ld(EPT);
    extern __shared__ uint4 sel_smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float *sbias = reinterpret_cast<float *>(sel_smem_raw);
    const int nscratch = sel_scratch(LPT, EPT, a.E + (a.E & 1)); // even: 16-byte rows
    unsigned long long *scratch =
        reinterpret_cast<unsigned long long *>(sbias + (BIASED ? LPT * BLD : 0)) + (size_t)warp * (nscratch + 40);
    const int sl = lane & (LPT - 1), seg = lane / LPT;
    uint2 *pick = reinterpret_cast<uint2 *>(scratch + nscratch) + seg * (LPT + 2);
    const int T = a.n_rows != nullptr ? min(a.T, *a.n_rows) : a.T;
    const int e0 = sl * EPT;
    const uint32_t rivals = ((1u << lane) - 1u) & (LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1u) << (seg * LPT));
    if (BIASED) {
        for (int e = threadIdx.x; e < LPT * EPT; e += blockDim.x)
            sbias[e / EPT * BLD + e % EPT] = e < a.E ? sel_bias(a.bias[e]) : 0.0f;
        __syncthreads();
    }
    const bool sums = a.groups > 1 && a.sum2;
    const bool need_sum = !a.sigmoid && (BIASED || sums || !a.renorm);
    const int lanes = a.groups > 1 ? a.gsz / EPT : 1; // lanes of a group, where it is whole lanes
    const bool whole = a.groups > 1 && (LPT == 8 || (a.gsz % EPT == 0 && (lanes & (lanes - 1)) == 0));
    const int my_group = whole ? sl / lanes : 0;
    constexpr int TPW = 32 / LPT; // tokens per warp

    for (int64_t tw = (int64_t)(blockIdx.x * warps + warp) * TPW; tw < T; tw += (int64_t)gridDim.x * warps * TPW) {
        const int t = (int)min(tw + seg, (int64_t)T - 1); // the last warp's spare lanes repeat a token
        const bool mine_too = tw + seg < T;
        const LT *row = static_cast<const LT *>(a.logits) + (size_t)t * a.ld;
        float v[EPT];
        if (LPT == 8 && EPT >= 4 && sizeof(LT) == 4 && a.vec && a.E == LPT * EPT) {
            // four whole fp32 rows, 512 consecutive bytes a time, through shared memory (a lane's own
            // values are EPT * 4 bytes apart from its neighbour's: 32 lines per load instead of 4)
            constexpr int Q = EPT >= 4 ? EPT / 4 : 1; // 16-byte pieces of a lane's values
            float *st = reinterpret_cast<float *>(scratch);
            float4 x[EPT >= 4 ? EPT / 4 : 1];
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int piece = i * 32 + lane, tok = piece / (8 * Q), at = piece % (8 * Q);
                const int tr = (int)min(tw + tok, (int64_t)T - 1);
                x[i] = reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + (size_t)tr * a.ld)[at];
            }
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int piece = i * 32 + lane, tok = piece / (8 * Q), at = piece % (8 * Q);
                *reinterpret_cast<float4 *>(st + (tok * 8 + at / Q) * BLD + at % Q * 4) = x[i];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float4 y = *reinterpret_cast<const float4 *>(st + lane * BLD + i * 4);
                v[(i * 4) % EPT] = y.x; v[(i * 4 + 1) % EPT] = y.y;
                v[(i * 4 + 2) % EPT] = y.z; v[(i * 4 + 3) % EPT] = y.w;
            }
            __syncwarp();
        } else {
            sel_load_row(a, row, e0, v);
        }
        if constexpr (BIASED) {
            // Every finite logit is live, the lowest too, and its bias may win: only -inf and NaN are
            // masked (a sigmoid and the test of its key need no clamp)
            if (!a.sigmoid) {
#pragma unroll
                for (int i = 0; i < EPT; ++i) v[i] = fminf(fmaxf(v[i], -INFINITY), SEL_FAR);
            }
        } else if (sums) { // a live logit has a score, if of 0, that counts for its group
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                v[i] = v[i] > -INFINITY ? fminf(fmaxf(v[i], -SEL_LOW), SEL_FAR) : -SEL_FAR;
        } else { // the order of the logits: below -SEL_EDGE sel_exact settles what is live
#pragma unroll
            for (int i = 0; i < EPT; ++i) v[i] = fminf(fmaxf(v[i], -SEL_FAR), SEL_FAR);
        }
        bool bad = false;

        // softmax: the row's maximum and sum where anything but the order is needed
        float m = 0.0f, sum = 1.0f;
        if (need_sum) {
            m = v[0];
#pragma unroll
            for (int i = 1; i < EPT; ++i) m = fmaxf(m, v[i]);
            // no live logit is below the floor, so the largest adds 1 and the sum is 0 only where every
            // expert is masked: no key is NaN
            m = fmaxf(sel_max_of<LPT>(m), -FLT_MAX);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < EPT; ++i) s += sel_ex2((v[i] - m) * SEL_LOG2E);
            sum = sel_sum_of<LPT>(s);
            bad = !(fabsf(m) < SEL_EDGE);
        }
        const float inv = sel_rcp(sum);
        if (BIASED) {
            float b[EPT];
            if constexpr (EPT >= 4) {
#pragma unroll
                for (int i = 0; i < EPT; i += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(sbias + sl * BLD + i);
                    b[i] = x.x; b[i + 1] = x.y; b[i + 2] = x.z; b[i + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPT; ++i) b[i] = sbias[sl * BLD + i];
            }
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < EPT; ++i)
                    v[i] = v[i] > -INFINITY ? sel_rcp(1.0f + sel_ex2(v[i] * -SEL_LOG2E)) + b[i] : -SEL_FAR;
            } else {
#pragma unroll
                for (int i = 0; i < EPT; ++i)
                    v[i] = v[i] > -INFINITY ? sel_ex2((v[i] - m) * SEL_LOG2E) * inv + b[i] : -SEL_FAR;
            }
        }
        float tol = a.sigmoid ? SEL_TOL_SIGMOID : SEL_TOL_SOFTMAX * inv;
        if (!BIASED && sums) {
            // the scores of a group's two largest logits, each off by its place's EPT 2^-23 |l|
            // through the score's slope: |l| s (1 - s) < 0.23, |l| s < (|m| + 1) / sum
            tol += (a.sigmoid ? 1.0f : 2.0f * (fabsf(m) + 1.0f) * inv) * SEL_PLACE(EPT);
        }

        if (LPT == 32 && a.groups > 1 && !whole) {
            // groups of any other size: the keys through shared memory, lane g walks group g
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
            const float gv = sel_group_value(a, BIASED, v1, v2, m, inv, bad);
            const bool st = sel_group_stays(gv, a.groups, a.keep, lane);
            const uint32_t stay = __ballot_sync(0xffffffffu, st);
            const float ge = sel_group_error(a, BIASED, SEL_TOL_KEY, gv, v1, v2);
            const float lo = sel_min_of<LPT>(st ? gv - ge : SEL_FAR);
            const float hi = sel_max_of<LPT>(!st && lane < a.groups ? gv + ge : -SEL_FAR);
            // (two groups at the clamp are as close as can be)
            if ((BIASED || sums) && hi > -SEL_NONE && !(lo - hi > 2.0f * tol)) bad = true;
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
            for (int c = 0; c < EPT / 8; ++c) {
                sel_sort<8>(v + 8 * c);
                if (c > 0) sel_merge8(v, v + 8 * c);
            }
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
            const float gv = sel_group_value(a, BIASED, v1, v2, m, inv, bad);
            // the group's rank: its lanes compare with the groups c, c + lanes, ... and add up
            auto rank_of = [&](auto x) {
                int rank = 0;
                for (int g0 = 0; g0 < a.groups; g0 += lanes) { // every lane takes every turn
                    const int g = g0 + (sl & (lanes - 1));
                    const auto o = __shfl_sync(0xffffffffu, x, min(g, a.groups - 1) * lanes, LPT);
                    if (g < a.groups) rank += (o > x || (o == x && g < my_group)) ? 1 : 0;
                }
                for (int off = 1; off < lanes; off <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, off);
                return rank;
            };
            const bool in = my_group < a.groups;
            const int rank = rank_of(gv); // every lane takes part, its group real or not
            bool st = in && rank < a.keep;
            if (!EXACT || sums) {
                const float ge = sel_group_error(a, BIASED, TOL_KEY, gv, v1, v2);
                const float lo = sel_min_of<LPT>(st ? gv - ge : SEL_FAR);
                const float hi = sel_max_of<LPT>(in && !st ? gv + ge : -SEL_FAR);
                const bool close =
                    hi > -SEL_NONE && !(lo - hi > (BIASED || sums ? 2.0f * tol : 0.0f) + SEL_TOL_ZERO);
                if (__any_sync(0xffffffffu, close)) {
                    // the groups' values again in 64 bits, from each lane's two largest (which are its two
                    // largest in 64 bits too, or the token goes to sel_exact)
                    const float third = EPT > 2 ? v[EPT > 2 ? 2 : 0] : -SEL_FAR;
                    const float second = EPT > 1 ? v[EPT > 1 ? 1 : 0] : -SEL_FAR;
                    const bool sure = !(third > -SEL_EDGE) ||
                                      second - third > tol + TOL_KEY * (fabsf(second) + fabsf(third)) + SEL_TOL_ZERO;
                    auto value = [&](float key) -> double {
                        if (!(key > -SEL_NONE)) return -INFINITY;
                        const int e = IDS ? sel_id(key) : e0 + (EPT > 1 ? (int)(__float_as_uint(key) & (uint32_t)(EPT - 1)) : 0);
                        const float l = sel_load(row + e);
                        return BIASED || sums ? sel_value64(l, BIASED ? a.bias[e] : 0.0f) : (double)l;
                    };
                    double d1 = value(v[0]), d2 = value(second);
                    if (d2 > d1) {
                        const double x = d1;
                        d1 = d2;
                        d2 = x;
                    }
                    for (int off = 1; off < lanes; off <<= 1) {
                        const double o1 = __shfl_xor_sync(0xffffffffu, d1, off);
                        const double o2 = __shfl_xor_sync(0xffffffffu, d2, off);
                        d2 = fmax(fmin(d1, o1), fmax(d2, o2));
                        d1 = fmax(d1, o1);
                    }
                    const double dg = sums && d2 > -INFINITY ? d1 + d2 : d1;
                    const int rank64 = rank_of(dg);
                    const bool st64 = in && rank64 < a.keep;
                    if (close) {
                        st = st64;
                        if (!sure || (!a.sigmoid && (BIASED || sums)) || !(fabsf(lo) < SEL_EDGE)) bad = true;
                    }
                }
            }
            if (!st) v[0] = -SEL_FAR;
        }

        auto round = [&](int j) {
            const float top = sel_max_of<LPT>(v[0]);
            const bool head = v[0] == top;
            const uint32_t all = __ballot_sync(0xffffffffu, head);
            if (head && !(all & rivals)) {
                pick[j] = make_uint2(__float_as_uint(top), (uint32_t)e0);
#pragma unroll
                for (int i = 0; i + 1 < D; ++i) v[i] = v[i + 1];
                // a lane that gave all its experts has no more; one that kept eight of more might
                v[D - 1] = EPT > D ? SEL_FAR : -SEL_FAR;
            }
        };
        const int rounds = EXACT ? a.k : a.k + 1; // one more: the best that is left out
#pragma unroll 1
        for (int j = 0; j < rounds; ++j) round(j);
        __syncwarp();
        auto expert = [&](uint2 p) {
            return IDS ? sel_id(__uint_as_float(p.x)) : (int)p.y + (EPT > 1 ? (int)(p.x & (uint32_t)(EPT - 1)) : 0);
        };
        auto apart = [&](float x, float y) { // surely in this order in 64 bits
            return x - y > (BIASED ? tol : 0.0f) + TOL_KEY * (fabsf(x) + fabsf(y)) + SEL_TOL_ZERO;
        };
        int mine = 0;
        const bool on = sl < a.k;
        bool close = false;
        if (on) {
            const uint2 p = pick[sl];
            const float key = __uint_as_float(p.x);
            if (!(fabsf(key) < SEL_EDGE)) bad = true;
            if (!EXACT && !apart(key, __uint_as_float(pick[sl + 1].x))) close = true;
            mine = expert(p);
        }
        uint32_t closes = 0;
        if (!EXACT) closes = __ballot_sync(0xffffffffu, close);
        if (!EXACT && closes) {
            // Winners too close to order in 32 bits: the first k + 1, if they are surely the k + 1
            // largest, again by their keys in 64 bits
            round(a.k + 1);
            __syncwarp();
            const float last = __uint_as_float(pick[a.k].x), after = __uint_as_float(pick[a.k + 1].x);
            const bool here = (closes & (LPT == 32 ? 0xffffffffu : ((1u << (LPT & 31)) - 1u) << (seg * LPT))) != 0;
            if (here && ((BIASED && !a.sigmoid) || !(last < SEL_EDGE && after < SEL_EDGE) ||
                         (last > -SEL_EDGE && !apart(last, after))))
                bad = true;
            double *d64 = reinterpret_cast<double *>(scratch) + seg * (LPT + 2);
            for (int j = sl; j <= a.k; j += LPT) {
                const uint2 p = pick[j];
                double d = -INFINITY;
                if (fabsf(__uint_as_float(p.x)) < SEL_EDGE) {
                    const int e = expert(p);
                    const float l = sel_load(row + e);
                    d = BIASED ? sel_value64(l, a.bias[e]) : (double)l;
                }
                d64[j] = d;
            }
            __syncwarp();
            int slot = -1, id = 0, slot2 = -1, id2 = 0; // ranks of entries sl and sl + LPT
            for (int j = sl; j <= a.k; j += LPT) {
                const double d = d64[j];
                const int e = expert(pick[j]);
                int rank = 0;
                for (int i = 0; i <= a.k; ++i)
                    rank += d64[i] > d || (d64[i] == d && (expert(pick[i]) < e || (expert(pick[i]) == e && i < j))) ? 1 : 0;
                if (j < LPT) {
                    slot = rank;
                    id = e;
                } else {
                    slot2 = rank;
                    id2 = e;
                }
            }
            __syncwarp();
            if (slot >= 0) pick[slot].y = (uint32_t)id;
            if (slot2 >= 0) pick[slot2].y = (uint32_t)id2;
            __syncwarp();
            if (here && on) mine = (int)pick[sl].y;
        }
        __syncwarp(); // pick and scratch are free for the next token
        uint32_t again = __ballot_sync(0xffffffffu, bad);
        while (again) { // one token at a time, the whole warp
            const int s = LPT == 32 ? 0 : (__ffs(again) - 1) / LPT;
            const int te = __shfl_sync(0xffffffffu, t, s * LPT);
            const SelExact x = sel_exact(a, static_cast<const LT *>(a.logits) + (size_t)te * a.ld, scratch, lane);
            const int xm = __shfl_sync(0xffffffffu, x.mine, sl);
            if (seg == s) {
                mine = xm;
                m = x.m;
                sum = x.sum;
            }
            __syncwarp();
            again &= LPT == 32 ? 0u : ~(((1u << (LPT & 31)) - 1u) << (s * LPT));
        }

        // weights, once for the k selected on the token's first k lanes
        const float lj = on ? sel_clean(sel_load(row + mine)) : -INFINITY;
        const bool live = lj > -INFINITY;
        float u = 0.0f;
        if (a.sigmoid) {
            const float mn = fminf(lj, 0.0f);
            const float M = a.renorm ? sel_max_of<LPT>(live ? mn : -INFINITY) : 0.0f; // keeps tiny scores' ratios
            if (live) u = __fdividef(expf(mn - M), 1.0f + expf(-fabsf(lj)));
        } else {
            const float M = a.renorm ? sel_max_of<LPT>(lj) : m;
            if (live) u = a.renorm ? expf(lj - M) : __fdividef(expf(lj - M), sum);
        }
        if (a.renorm) {
            const float total = sel_sum_of<LPT>(u);
            u = total > 0.0f ? __fdividef(u, total) : 0.0f;
        }
        if (on && mine_too) {
            a.idx[(size_t)t * a.k + sl] = mine;
            a.w[(size_t)t * a.k + sl] = a.scale * u;
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
