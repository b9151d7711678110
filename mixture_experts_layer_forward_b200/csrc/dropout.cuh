// dropout.cuh -- dropout from a counter-based generator, with the residual; the mask is never
// stored: the backward pass forms it again from the same seed and offset.
//
//   y_i = r_i + (u_i >= thr ? x_i * 65536 / (65536 - thr) : 0),   thr = 65536 p
//   dx_i =       u_i >= thr ? dy_i * 65536 / (65536 - thr) : 0
// u_i is 16 bits of the ten-round 4 x 32-bit counter generator of Salmon, Moraes, Dror and
// Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3" (2011): key = seed, counter = offset +
// i / 8 (64 bits, the upper two words 0); element i takes word (i % 8) / 2, its lower half for
// an even i. One counter serves eight elements, so a thread owns eight consecutive ones (one
// 16-byte piece of bf16). p is a multiple of 2^-16 and the scale is its own, so the mean is kept.
// Sums in fp32, one rounding. A dropped value is not multiplied, so an infinity or NaN there
// does not pass. Bound by the bytes read and written (8192 x 4096 bf16 with a residual: 31 us, 6.4 TB/s,
// the measured copy rate); without a residual the ten rounds, about 60 of 130 instructions for
// eight elements, come close to the bytes (27 us against 21).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "order.cuh"
#include "ptx.cuh"

namespace moe {

struct DropoutArgs {
    const void *x;
    const void *res;      // nullptr: none
    void *y;
    const unsigned long long *rng; // [2] on the device: seed, offset
    int64_t n;
    uint32_t thr;         // 0 .. 65536
    float scale;
};

__device__ __forceinline__ void dropout_bits(unsigned long long ctr, unsigned long long seed,
                                             uint32_t (&c)[4])
{
    c[0] = (uint32_t)ctr;
    c[1] = (uint32_t)(ctr >> 32);
    c[2] = 0u;
    c[3] = 0u;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long a = (unsigned long long)c[0] * 0xD2511F53u;
        const unsigned long long b = (unsigned long long)c[2] * 0xCD9E8D57u;
        const uint32_t n0 = (uint32_t)(b >> 32) ^ c[1] ^ k0;
        const uint32_t n2 = (uint32_t)(a >> 32) ^ c[3] ^ k1;
        c[1] = (uint32_t)b;
        c[3] = (uint32_t)a;
        c[0] = n0;
        c[2] = n2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Eight consecutive elements as loaded: 16 bytes of bf16, 32 of fp32.
template <typename DT> struct DropoutRaw {
    uint4 p[sizeof(DT) / 2];
    __device__ __forceinline__ void load(const DT *src)
    {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(DT) / 2); ++i) p[i] = reinterpret_cast<const uint4 *>(src)[i];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        if constexpr (sizeof(DT) == 2) {
            v[0] = bf16_lo(p[0].x); v[1] = bf16_hi(p[0].x); v[2] = bf16_lo(p[0].y); v[3] = bf16_hi(p[0].y);
            v[4] = bf16_lo(p[0].z); v[5] = bf16_hi(p[0].z); v[6] = bf16_lo(p[0].w); v[7] = bf16_hi(p[0].w);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(p[i].x); v[4 * i + 1] = __uint_as_float(p[i].y);
                v[4 * i + 2] = __uint_as_float(p[i].z); v[4 * i + 3] = __uint_as_float(p[i].w);
            }
        }
    }
};
__device__ __forceinline__ uint32_t dropout_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void dropout_store8(__nv_bfloat16 *p, const float (&v)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(dropout_pack(v[0], v[1]), dropout_pack(v[2], v[3]),
                                               dropout_pack(v[4], v[5]), dropout_pack(v[6], v[7]));
}
__device__ __forceinline__ void dropout_store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float dropout_load1(const float *p) { return *p; }
__device__ __forceinline__ float dropout_load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void dropout_store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void dropout_store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// v of group i: kept, scaled, plus r
__device__ __forceinline__ void dropout_apply(const DropoutArgs &a, unsigned long long seed,
                                              unsigned long long ctr, float (&v)[8], const float (&r)[8])
{
    uint32_t c[4];
    dropout_bits(ctr, seed, c);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = (c[q] & 0xffffu) >= a.thr ? fmaf(v[2 * q], a.scale, r[2 * q]) : r[2 * q];
        v[2 * q + 1] = (c[q] >> 16) >= a.thr ? fmaf(v[2 * q + 1], a.scale, r[2 * q + 1]) : r[2 * q + 1];
    }
}

// GROUPS groups of eight elements per thread and turn, their loads in flight together.
template <typename DT, bool RES, int GROUPS>
__global__ void __launch_bounds__(256) dropout_add_kernel(const __grid_constant__ DropoutArgs a)
{
    order_launch_dependents();
    order_wait();
    const DT *x = static_cast<const DT *>(a.x), *res = static_cast<const DT *>(a.res);
    DT *y = static_cast<DT *>(a.y);
    const unsigned long long seed = a.rng[0], offset = a.rng[1];
    const int64_t whole = a.n / 8, stride = (int64_t)gridDim.x * 256;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (; i + (GROUPS - 1) * stride < whole; i += GROUPS * stride) {
        DropoutRaw<DT> xr[GROUPS], rr[GROUPS];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            xr[g].load(x + (i + g * stride) * 8);
            if (RES) rr[g].load(res + (i + g * stride) * 8);
        }
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            float v[8], r[8];
            xr[g].values(v);
#pragma unroll
            for (int q = 0; q < 8; ++q) r[q] = 0.0f;
            if (RES) rr[g].values(r);
            dropout_apply(a, seed, offset + (unsigned long long)(i + g * stride), v, r);
            dropout_store8(y + (i + g * stride) * 8, v);
        }
    }
    for (; i < (a.n + 7) / 8; i += stride) { // the rest, and the elements behind the last whole group
        float v[8], r[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = r[q] = 0.0f;
        if (i < whole) {
            DropoutRaw<DT> xr, rr;
            xr.load(x + i * 8);
            if (RES) rr.load(res + i * 8);
            xr.values(v);
            if (RES) rr.values(r);
        } else {
#pragma unroll 1
            for (int q = 0; q < (int)(a.n - i * 8); ++q) {
                const float xv = dropout_load1(x + i * 8 + q), rv = RES ? dropout_load1(res + i * 8 + q) : 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j == q) {
                        v[j] = xv;
                        r[j] = rv;
                    }
            }
        }
        dropout_apply(a, seed, offset + (unsigned long long)i, v, r);
        if (i < whole) {
            dropout_store8(y + i * 8, v);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (i * 8 + q < a.n) dropout_store1(y + i * 8 + q, v[q]);
        }
    }
}

} // namespace moe
