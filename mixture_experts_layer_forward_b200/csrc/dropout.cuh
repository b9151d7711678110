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
// does not pass. Bound by the bytes read and written: ten rounds are about 60 instructions for
// eight elements.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

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

__device__ __forceinline__ float dropout_one(uint32_t u, uint32_t thr, float x, float scale, float r)
{
    return u >= thr ? fmaf(x, scale, r) : r;
}

__device__ __forceinline__ void dropout_load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void dropout_load8(const float *p, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void dropout_store8(__nv_bfloat16 *p, const float (&v)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
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

template <typename DT>
__global__ void __launch_bounds__(256) dropout_add_kernel(const DropoutArgs a)
{
    const DT *x = static_cast<const DT *>(a.x), *res = static_cast<const DT *>(a.res);
    DT *y = static_cast<DT *>(a.y);
    const unsigned long long seed = a.rng[0], offset = a.rng[1];
    const int64_t groups = (a.n + 7) / 8, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < groups; i += stride) {
        const bool whole = i * 8 + 8 <= a.n;
        float v[8], r[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = r[q] = 0.0f;
        if (whole) {
            dropout_load8(x + i * 8, v);
            if (res != nullptr) dropout_load8(res + i * 8, r);
        } else {
            for (int q = 0; q < 8; ++q)
                if (i * 8 + q < a.n) {
                    v[q] = dropout_load1(x + i * 8 + q);
                    if (res != nullptr) r[q] = dropout_load1(res + i * 8 + q);
                }
        }
        uint32_t c[4];
        dropout_bits(offset + (unsigned long long)i, seed, c);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = dropout_one(c[q] & 0xffffu, a.thr, v[2 * q], a.scale, r[2 * q]);
            v[2 * q + 1] = dropout_one(c[q] >> 16, a.thr, v[2 * q + 1], a.scale, r[2 * q + 1]);
        }
        if (whole) {
            dropout_store8(y + i * 8, v);
        } else {
            for (int q = 0; q < 8; ++q)
                if (i * 8 + q < a.n) dropout_store1(y + i * 8 + q, v[q]);
        }
    }
}

} // namespace moe
