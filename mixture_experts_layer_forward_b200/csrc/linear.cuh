// linear.cuh -- dense product with bias, activation and residual in its epilogue, on the
// 5th-generation tensor cores, and the products of its gradient.
//
//   z = x W + bias,  y = act(z) + residual           (SwiGLU: z = [g, u], y = silu(g) u + r)
//   dz = dy act'(z), dx = dz W^T, dW = x^T dz, dbias = sum over rows of dz
//
// All four products are one tile loop, D[m, n] = sum_k A[m, k] B[k, n], with each operand read
// as it is stored: K-major (k contiguous) or MN-major (m or n contiguous).
//   forward   A = x K-major;   B = W [K, N] MN-major, or W [N, K] K-major
//   dx        A = dz K-major;  B = W^T: W [K, N] K-major, or W [N, K] MN-major
//   dW        A and B MN-major: x^T dz [K, N], or dz^T x [N, K]
// Edges need no padding: copies past a tensor's end read zeros, and the epilogue stores only
// rows < M and columns < N.
//
// A block has ten warps: one issues TMA copies into a ring of 128-byte-swizzled stages (64 or 128
// values of k each), one issues tcgen05.mma (M = 128, N = BN, fp32 accumulators in TMEM), eight
// run the epilogue (each pair of warps shares 32 rows and splits the columns).
//   linear_kernel        persistent, one block per SM, two accumulators, so that a tile's
//                        epilogue runs beside the next tile's products.
//   linear_split_kernel  one tile per cluster of S blocks, each with 1/S of k; the blocks'
//                        accumulators meet through distributed shared memory, summed in rank
//                        order (deterministic), and each block finishes 1/S of the columns.
//                        For outputs of few tiles, where one block per tile would leave most
//                        SMs idle: a token or a decode batch (bound by reading W), router
//                        logits and weight gradients with few columns.
// Every wait is bounded as in the other kernels here: a block that gives up records the
// timeout, waits for its copies and products in flight, frees its TMEM and leaves.
//
// Measured (M x K x N), calls back to back: 4096^3 101 us, 1360 TFLOP/s (0.83 of the measured burst rate: the
// tensor pipe is busy 71 to 75% of the launch); 8192 x 4096 x 2 * 14336 SwiGLU 1.47 ms under the power cap (0.94 of
// the sustained rate), 1.28 ms cool; 4096 x 7168 x 256 fp32 24.2 us, bound by what an SM takes from L2 (64 KB per
// 128 x 128 x 128 step, 130 GB/s); 64 x 7168 x 2 * 2048 SwiGLU 16.3 us, 1 x 4096 x 4096 9.6 us (59 and 34 MB of W
// at 6.5 TB/s: 9 and 5 us, the rest start, reduction and end of the launch). Row strides that are not a multiple
// of 128 bytes cost up to half as much again while operands come from L2 (1003 x 1160 x 2568: 13.6 us of products
// against 9.1 at K = 1152).
#pragma once

#include "order.cuh"
#include "ptx.cuh"

namespace moe {

namespace lin {
constexpr int BM = 128;
constexpr int A_BOX = BM * 64 * 2; // 16 KB: 128 rows x 64 k, or two boxes of 64 columns x 64 k rows
constexpr int BOX = 64 * 64 * 2;   // 8 KB: 64 columns x 64 k rows of an MN-major operand
constexpr int THREADS = 320;       // TMA warp, MMA warp, 8 epilogue warps
constexpr int EPI_THREADS = 256;
// 64-value blocks of k in a stage: a narrow tile's products are shorter than the barrier's round trip,
// so its stages hold two
__host__ __device__ constexpr int sub(int bn) { return bn == 256 ? 1 : 2; }
__host__ __device__ constexpr int bk(int bn) { return 64 * sub(bn); }
__host__ __device__ constexpr int stage_bytes(int bn) { return sub(bn) * (A_BOX + bn * 128); }
__host__ __device__ constexpr int stages(int bn) { return 196608 / stage_bytes(bn); } // 4, 3, 4 for BN = 256, 128, 64
__host__ __device__ constexpr int num_bars(int bn) { return 2 * stages(bn) + 5; }
constexpr int TURN = 32 * 32 * 4; // one warp's 32 x 32 fp32 values on their way from rows per lane to rows in memory
__host__ __device__ constexpr int smem_bytes(int bn, bool split)
{
    return 1024 + stages(bn) * stage_bytes(bn) + (split ? 0 : 8 * TURN) + num_bars(bn) * 8 + 16;
}
// fp32 outputs: k values summed in one accumulator before its values are added up in registers. The
// tensor core truncates what it adds to the accumulator's size, so that errors add up with K. Measured,
// one accumulator against runs of 512: products of one sign 2.9e-5 against 9.4e-7 of the sum at
// K = 7168, 7.5e-5 against 9.9e-7 at 16384; of random signs 3.8e-6 against 4.7e-7 at K = 7168. bf16
// outputs keep one accumulator: their own rounding is 2^-8.
constexpr int PROMOTE_K = 512;
// Least limit of a wait, whatever moe_set_wait_timeout_ns asks for. Copies and products in flight take
// microseconds to land, so a block that gives up never leaves before its own have; and block 0, the first
// to be set up, has cleared the status word long before another block's wait can run out and record it.
constexpr int64_t LEAST_WAIT_NS = 100000000;
} // namespace lin

struct LinearArgs {
    int M, N;             // output rows and columns
    int m_tiles, n_tiles, k_blocks;
    int group_m;          // m tiles that share a run of n tiles (operands of a run stay in L2)
    int a_rows;           // rows of a K-major A box (M rounded up to 8, at most 128)
    int act;              // 0 SwiGLU, 1 GELU (tanh form), 2 ReLU, 3 identity
    int up_col;           // SwiGLU: first up column (= N); a tile holds BN/2 gate, BN/2 up columns
    const float *bias;    // [N] ([2N] for SwiGLU) or nullptr
    const __nv_bfloat16 *res; // [M, N], row stride ldr, or nullptr
    int64_t ldr;
    void *y;              // [M, N], row stride ldy
    int64_t ldy;
    int y_f32;
    __nv_bfloat16 *z;     // pre-activation [M, N or 2N], row stride ldz, or nullptr
    int64_t ldz;
    int splits;           // linear_split_kernel: blocks per cluster
    int full;             // 256-column tiles: those from this one on are worked as two halves
    int *status;
    int clear_status;     // block 0 clears the status word (the call's first launch with waits)
    int64_t timeout_ns;   // at least lin::LEAST_WAIT_NS
};

__device__ __forceinline__ void lin_load_bias8(const float *bias, float (&b)[8])
{
    const float4 x = reinterpret_cast<const float4 *>(bias)[0];
    const float4 y = reinterpret_cast<const float4 *>(bias)[1];
    b[0] = x.x; b[1] = x.y; b[2] = x.z; b[3] = x.w;
    b[4] = y.x; b[5] = y.y; b[6] = y.z; b[7] = y.w;
}

__device__ __forceinline__ uint32_t lin_pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint4 lin_pack8(const float (&v)[8])
{
    return make_uint4(lin_pack2(v[0], v[1]), lin_pack2(v[2], v[3]), lin_pack2(v[4], v[5]),
                      lin_pack2(v[6], v[7]));
}

// 2^x and 1 / x of the special function unit (2^-22.5 and 2^-23 relative; denormal results 0)
__device__ __forceinline__ float lin_ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lin_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float LIN_LOG2E = 1.4426950408889634f;
constexpr float LIN_GC2 = 1.5957691216057308f; // 2 sqrt(2 / pi): (1 + tanh(w)) / 2 = 1 / (1 + exp(-2 w))
constexpr float LIN_GK = 0.044715f;

__device__ __forceinline__ float lin_sigmoid(float z) { return lin_rcp(1.0f + lin_ex2(-LIN_LOG2E * z)); }
// the sigmoid of 2 sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float lin_gelu_gate(float z, float z2)
{
    return lin_rcp(1.0f + lin_ex2(z * fmaf(-LIN_LOG2E * LIN_GC2 * LIN_GK, z2, -LIN_LOG2E * LIN_GC2)));
}
__device__ __forceinline__ float lin_silu(float z) { return z * lin_sigmoid(z); }
__device__ __forceinline__ float lin_gelu(float z) { return z * lin_gelu_gate(z, z * z); }
// z within +-lim; a NaN stays one
__device__ __forceinline__ float lin_within(float z, float lim)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(lim));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-lim));
    return r;
}
// s + z s (1 - s) w', w' = 2 sqrt(2 / pi) (1 + 3 * 0.044715 z^2). At 30 the gate s is 0 or 1 to the last
// bit; further out the products would overflow against it (0 times infinity).
__device__ __forceinline__ float lin_gelu_grad(float z)
{
    z = lin_within(z, 30.0f);
    const float z2 = z * z, s = lin_gelu_gate(z, z2);
    return s * fmaf(z * (1.0f - s), fmaf(3.0f * LIN_GK * LIN_GC2, z2, LIN_GC2), 1.0f);
}

// The residual of eight columns (zeros outside the output).
__device__ __forceinline__ uint4 lin_res8(const LinearArgs &a, int row, int col)
{
    if (a.res == nullptr || row >= a.M || col >= a.N) return make_uint4(0u, 0u, 0u, 0u);
    return *reinterpret_cast<const uint4 *>(a.res + (size_t)row * a.ldr + col);
}

// Where eight consecutive output columns of one row go (z of SwiGLU: the up half up_col further).
struct LinOut {
    char *y;            // bf16 or fp32
    __nv_bfloat16 *z;   // nullptr: not wanted
    __device__ LinOut(const LinearArgs &a, int row, int col)
    {
        y = static_cast<char *>(a.y) + ((size_t)row * a.ldy + col) * (a.y_f32 ? 4 : 2);
        z = a.z != nullptr ? a.z + (size_t)row * a.ldz + col : nullptr;
    }
    __device__ void down(const LinearArgs &a, int rows)
    {
        y += (size_t)rows * a.ldy * (a.y_f32 ? 4 : 2);
        if (z != nullptr) z += (size_t)rows * a.ldz;
    }
};

// Eight consecutive columns of one row: v the accumulators (SwiGLU: v the gate's, u the up's), bv and
// bu the bias (zeros: none), r the residual.
__device__ __forceinline__ void lin_finish8(const LinearArgs &a, float (&v)[8], float (&u)[8],
                                            const float (&bv)[8], const float (&bu)[8], const uint4 &r,
                                            const LinOut &out)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += bv[i];
    if (out.z != nullptr) *reinterpret_cast<uint4 *>(out.z) = lin_pack8(v);
    if (a.act == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += bu[i];
        if (out.z != nullptr) *reinterpret_cast<uint4 *>(out.z + a.up_col) = lin_pack8(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lin_silu(v[i]) * u[i];
    } else if (a.act == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lin_gelu(v[i]);
    } else if (a.act == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
    }
    if (a.res != nullptr) {
        v[0] += bf16_lo(r.x); v[1] += bf16_hi(r.x); v[2] += bf16_lo(r.y); v[3] += bf16_hi(r.y);
        v[4] += bf16_lo(r.z); v[5] += bf16_hi(r.z); v[6] += bf16_lo(r.w); v[7] += bf16_hi(r.w);
    }
    if (a.y_f32) {
        reinterpret_cast<float4 *>(out.y)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(out.y)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(out.y) = lin_pack8(v);
    }
}

__device__ __forceinline__ void lin_tile(int w, const LinearArgs &a, int &mt, int &nt)
{
    const int per = a.group_m * a.n_tiles;
    const int g = w / per, r = w - g * per;
    const int m0 = g * a.group_m;
    const int gm = min(a.group_m, a.m_tiles - m0);
    mt = m0 + r % gm;
    nt = r / gm;
}

// One lane of a converged warp. The roles below run warp-wide, with only the copies and products
// themselves under this predicate: their operands then stay in uniform registers. (One-lane loops
// cost 90 to 130 cycles an instruction, which bound every tile: 0.31 us a k-block at BN = 256, 0.28
// at BN = 64, where the products take 0.27 and 0.07.)
__device__ __forceinline__ bool lin_elect()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Bounded wait of a whole warp (mbar_wait_bounded for all lanes alike).
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                         int64_t timeout_ns, int *status, int where)
{
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (true) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool late = (int64_t)(globaltimer_ns() - t0) > timeout_ns;
        if (__any_sync(0xffffffffu, late || *abort_flag != 0)) {
            if (late && *abort_flag == 0) {
                *abort_flag = 1;
                record_status(status, DEV_TIMEOUT, where);
            }
            return false;
        }
    }
}

// One work item of the persistent kernel: a tile, or half the columns of one. A last wave of tiles
// that would leave more than half of the blocks idle is worked in halves, one each
// (4096 x 4096 x 4096: 3.46 waves of tiles in the time of 3.5 instead of 4).
struct LinItem {
    int mt, n0, width; // row tile, first output column, accumulator columns
};
template <int BN> __device__ __forceinline__ LinItem lin_item(int w, const LinearArgs &a, int tc)
{
    LinItem it;
    int nt, off = 0;
    it.width = BN;
    if (BN == 256 && w >= a.full) {
        const int j = w - a.full;
        w = a.full + (j >> 1);
        off = (j & 1) * (tc / 2);
        it.width = BN / 2;
    }
    lin_tile(w, a, it.mt, nt);
    it.n0 = nt * tc + off;
    return it;
}

// The barriers and the two pipeline roles, shared by both kernels.
template <int BN, bool A_MN, bool B_MN> struct LinPipe {
    static constexpr int STAGES = lin::stages(BN);
    static constexpr int STAGE = lin::stage_bytes(BN);
    static constexpr int SUB = lin::sub(BN);
    static constexpr int SUB_BYTES = lin::A_BOX + BN * 128; // one 64-value block of k: A, then B
    static constexpr uint32_t IDESC =
        idesc_bf16_f32(lin::BM, BN, B_MN) | ((A_MN ? 1u : 0u) << 15);
    static constexpr uint32_t IDESC_HALF =
        idesc_bf16_f32(lin::BM, BN / 2, B_MN) | ((A_MN ? 1u : 0u) << 15);
    uint8_t *smem;
    uint32_t bar0;
    int s = 0;       // ring position
    uint32_t ph = 0;

    __device__ uint32_t full(int i) const { return bar0 + 8u * i; }
    __device__ uint32_t empty(int i) const { return bar0 + 8u * (STAGES + i); }
    __device__ uint32_t tfull(int i) const { return bar0 + 8u * (2 * STAGES + i); }
    __device__ uint32_t tempty(int i) const { return bar0 + 8u * (2 * STAGES + 2 + i); }
    __device__ uint32_t done() const { return bar0 + 8u * (2 * STAGES + 4); }
    __device__ void next()
    {
        if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
        }
    }
    __device__ void init_bars(bool two_sided)
    {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            if (two_sided) mbar_init(tempty(i), 8);
        }
        mbar_init(done(), 1);
        fence_mbar_init();
    }

    // TMA copies of k-blocks [kb0, kb1) of one item (one warp)
    __device__ bool produce(const CUtensorMap &tmA, const CUtensorMap &tmB, const LinearArgs &a,
                            const LinItem &w, int kb0, int kb1, volatile int *abort_flag, uint32_t &armed)
    {
        const bool gated = a.act == 0;
        const int mt = w.mt, n0 = w.n0;
        const int boxes = BN == 256 ? w.width / 64 : BN / 64; // 64 columns of B each
        const int gate = gated ? boxes / 2 : boxes;           // of them before the up columns
        const uint32_t bytes = SUB * ((A_MN ? lin::A_BOX : a.a_rows * 128) + boxes * lin::BOX);
        const uint32_t base = smem_u32(smem);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!lin_wait(empty(s), ph ^ 1u, abort_flag, a.timeout_ns, a.status, 500)) return false;
            armed |= 1u << s;
            if (lin_elect()) {
                mbar_arrive_expect_tx(full(s), bytes);
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    const uint32_t a_dst = base + s * STAGE + j * SUB_BYTES, b_dst = a_dst + lin::A_BOX;
                    const int k = (kb * SUB + j) * 64;
                    if (A_MN) {
                        tma_load_2d(a_dst, &tmA, full(s), mt * lin::BM, k);
                        tma_load_2d(a_dst + lin::BOX, &tmA, full(s), mt * lin::BM + 64, k);
                    } else {
                        tma_load_2d(a_dst, &tmA, full(s), k, mt * lin::BM);
                    }
                    if (B_MN || BN == 256) { // boxes of 64 columns (B_MN) or 64 rows
#pragma unroll
                        for (int i = 0; i < BN / 64; ++i) {
                            if (i >= boxes) break;
                            const int col = i >= gate ? a.up_col + n0 + (i - gate) * 64 : n0 + i * 64;
                            tma_load_2d(b_dst + i * lin::BOX, &tmB, full(s), B_MN ? col : k, B_MN ? k : col);
                        }
                    } else if (gated) { // box of BN / 2 rows
                        tma_load_2d(b_dst, &tmB, full(s), k, n0);
                        tma_load_2d(b_dst + BN / 2 * 128, &tmB, full(s), k, a.up_col + n0);
                    } else { // box of BN rows
                        tma_load_2d(b_dst, &tmB, full(s), k, n0);
                    }
                }
            }
            __syncwarp();
            next();
        }
        return true;
    }

    // every copy issued has landed before the block leaves (ph, s: the next copy's place)
    __device__ void drain(uint32_t armed, int64_t timeout_ns)
    {
        for (int i = 0; i < STAGES; ++i)
            if ((armed >> i) & 1u) {
                volatile int never = 0;
                lin_wait(full(i), i < s ? ph : ph ^ 1u, &never, timeout_ns, nullptr, 0);
            }
    }

    // the products of k-blocks [kb0, kb1) into d_tmem (one warp)
    __device__ bool multiply(const LinearArgs &a, uint32_t d_tmem, int width, int kb0, int kb1,
                             volatile int *abort_flag)
    {
        const uint32_t base = smem_u32(smem);
        const uint32_t idesc = BN == 256 && width != BN ? IDESC_HALF : IDESC;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!lin_wait(full(s), ph, abort_flag, a.timeout_ns, a.status, 510)) return false;
            tc_fence_after();
            if (lin_elect()) {
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    const uint32_t a_addr = base + s * STAGE + j * SUB_BYTES, b_addr = a_addr + lin::A_BOX;
                    // K-major: rows of 128 bytes, +32 bytes per 16 k; MN-major: 64-column blocks of
                    // 64 k rows, +16 rows per 16 k
                    const uint64_t ad = A_MN ? sw128_desc(a_addr, lin::BOX, 1024) : sw128_desc(a_addr, 16, 1024);
                    const uint64_t bd = B_MN ? sw128_desc(b_addr, lin::BOX, 1024) : sw128_desc(b_addr, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(d_tmem, ad + (uint64_t)((A_MN ? k * 2048 : k * 32) >> 4),
                                  bd + (uint64_t)((B_MN ? k * 2048 : k * 32) >> 4), idesc,
                                  (kb != kb0 || (j | k) != 0) ? 1u : 0u);
                }
                umma_commit(empty(s));
            }
            __syncwarp();
            next();
        }
        return true;
    }

    // the products of k-blocks [kb0, kb1) in runs of `run`, each into the accumulator of its turn
    __device__ bool multiply_runs(const LinearArgs &a, uint32_t tmem, int width, int kb0, int kb1, int run,
                                  int &it, volatile int *abort_flag)
    {
        for (int kb = kb0; kb < kb1; kb += run, ++it) {
            const int acc = it & 1;
            if (!lin_wait(tempty(acc), ((it >> 1) & 1) ^ 1, abort_flag, a.timeout_ns, a.status, 520)) return false;
            tc_fence_after();
            if (!multiply(a, tmem + acc * BN, width, kb, min(kb + run, kb1), abort_flag)) return false;
            if (lin_elect()) umma_commit(tfull(acc));
            __syncwarp();
        }
        return true;
    }
};

// 16 consecutive accumulator columns of this warp's 32 rows (one row per lane), to be waited for
// before they are used.
__device__ __forceinline__ void lin_ld16(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// A finished run's columns added to sum.
__device__ __forceinline__ void lin_add16(uint32_t taddr, float *sum)
{
    uint32_t r[16];
    lin_ld16(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] += __uint_as_float(r[i]);
}
__device__ __forceinline__ void lin_add32(uint32_t t_row, int c, float *sum)
{
    lin_add16(t_row + c * 32, sum);
    lin_add16(t_row + c * 32 + 16, sum + 16);
}

// PROMOTE: runs of lin::PROMOTE_K values of k are summed in registers (fp32 outputs).
template <int BN, bool A_MN, bool B_MN, bool PROMOTE>
__global__ void __launch_bounds__(lin::THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ LinearArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    LinPipe<BN, A_MN, B_MN> p;
    p.smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~static_cast<uintptr_t>(1023));
    float *turns = reinterpret_cast<float *>(p.smem + lin::stages(BN) * lin::stage_bytes(BN));
    uint64_t *bars = reinterpret_cast<uint64_t *>(turns + 8 * lin::TURN / 4);
    p.bar0 = smem_u32(bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + lin::num_bars(BN));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    order_launch_dependents();
    if (threadIdx.x == 0) {
        p.init_bars(true);
        *abort_flag = 0;
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 2 * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = BN == 256 ? 2 * a.m_tiles * a.n_tiles - a.full : a.m_tiles * a.n_tiles;
    const int tc = a.act == 0 ? BN / 2 : BN;
    const int run = PROMOTE ? lin::PROMOTE_K / lin::bk(BN) : a.k_blocks;
    order_wait();
    if (a.clear_status && blockIdx.x == 0 && threadIdx.x == 0) { // no wait has run out yet (LEAST_WAIT_NS)
        a.status[0] = DEV_OK;
        a.status[1] = 0;
    }

    if (warp == 0) {
        uint32_t armed = 0;
        for (int w = blockIdx.x; w < total; w += gridDim.x) {
            if (!p.produce(tmA, tmB, a, lin_item<BN>(w, a, tc), 0, a.k_blocks, abort_flag, armed)) break;
        }
        p.drain(armed, a.timeout_ns);
    } else if (warp == 1) {
        int it = 0;
        for (int w = blockIdx.x; w < total; w += gridDim.x)
            if (!p.multiply_runs(a, tmem, lin_item<BN>(w, a, tc).width, 0, a.k_blocks, run, it, abort_flag)) break;
        if (lin_elect()) umma_commit(p.done()); // every product is finished before TMEM is released
        __syncwarp();
        volatile int never = 0;
        lin_wait(p.done(), 0, &never, a.timeout_ns, a.status, 530);
    } else {
        const int q = warp & 3, half = warp >= 6 ? 1 : 0;
        const bool gated = a.act == 0;
        int it = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
            const LinItem item = lin_item<BN>(w, a, tc);
            const int mt = item.mt, wide = item.width;       // accumulator columns
            const int each = (gated ? wide / 2 : wide) / 2;  // output columns of a warp
            // A lane's accumulators are one row of 32 values (SwiGLU: 16 gate and 16 up columns); in
            // memory the warp takes whole rows' pieces, eight columns a lane, so that loads and stores
            // touch whole sectors of few lines (one row per lane: 32 lines an instruction). The values
            // change hands through shared memory, their 16-byte units exchanged by the row's low bits.
            // The loop over the rows stays rolled: its code runs a few times a launch, and unrolled it
            // took longer (a launch of one 128 x 256 tile, k = 64: 11.1 us, rolled 7.1).
            float *turn = turns + (warp - 2) * (lin::TURN / 4);
            const int psh = gated ? 1 : 2;                   // log2 of the lanes (8-column pieces) of a row
            const int piece = lane & ((1 << psh) - 1), up_unit = 4 + piece * 2;
            const int cols = 8 << psh;                       // output columns of a turn
            const int first = item.n0 + half * each;         // this warp's first column
            auto own_row = [&](const uint32_t (&own)[32]) {  // 32 values of row `lane` into the turn
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(turn + lane * 32 + ((i ^ (lane & 7)) << 2)) =
                        make_uint4(own[i * 4], own[i * 4 + 1], own[i * 4 + 2], own[i * 4 + 3]);
                __syncwarp();
            };
            const int rstep = 32 >> psh, row0 = mt * lin::BM + q * 32 + (lane >> psh);
            // the residual of this lane's rows of a turn, on its way one turn ahead (the first turn's
            // while the products run)
            uint4 res[4] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u),
                            make_uint4(0u, 0u, 0u, 0u)};
            auto fetch = [&](int col) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    res[i] = i < (1 << psh) ? lin_res8(a, row0 + i * rstep, col + piece * 8) : make_uint4(0u, 0u, 0u, 0u);
            };
            if (a.res != nullptr) fetch(first);
            auto rows_out = [&](int col, bool more) {        // the turn's 32 rows, columns col .. col + cols
                uint4 now[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = res[i];
                if (more && a.res != nullptr) fetch(col + cols);
                const int mine = col + piece * 8;
                if (mine >= a.N) return;
                float bv[8], bu[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) bv[i] = bu[i] = 0.0f;
                if (a.bias != nullptr) {
                    lin_load_bias8(a.bias + mine, bv);
                    if (gated) lin_load_bias8(a.bias + a.up_col + mine, bu);
                }
                LinOut out(a, row0, mine);
#pragma unroll 1
                for (int i = 0; i < (1 << psh); ++i) {
                    if (row0 + i * rstep >= a.M) break;
                    const int r = (lane >> psh) + i * rstep;
                    float v[8], u[8];
                    auto take = [&](int unit, float (&o)[8]) {
                        const float4 x = *reinterpret_cast<const float4 *>(turn + r * 32 + ((unit ^ (r & 7)) << 2));
                        const float4 y = *reinterpret_cast<const float4 *>(turn + r * 32 + (((unit + 1) ^ (r & 7)) << 2));
                        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
                        o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
                    };
                    take(piece * 2, v);
                    if (gated) take(up_unit, u);
                    lin_finish8(a, v, u, bv, bu, now[0], out);
                    out.down(a, rstep);
                    now[0] = now[1];
                    now[1] = now[2];
                    now[2] = now[3];
                }
            };
            if constexpr (PROMOTE) {
                // this warp's half of the accumulator's columns (SwiGLU: half of the gate's, of the up's)
                float sum[BN / 2];
#pragma unroll
                for (int i = 0; i < BN / 2; ++i) sum[i] = 0.0f;
                for (int kb = 0; kb < a.k_blocks; kb += run, ++it) {
                    const int acc = it & 1;
                    ok = lin_wait(p.tfull(acc), (it >> 1) & 1, abort_flag, a.timeout_ns, a.status, 540);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
                    if (gated) { // turns of 16 gate and 16 up columns
#pragma unroll
                        for (int c = 0; c < BN / 64; ++c) {
                            lin_add16(t_row + half * (BN / 4) + c * 16, sum + c * 32);
                            lin_add16(t_row + BN / 2 + half * (BN / 4) + c * 16, sum + c * 32 + 16);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < BN / 64; ++c)
                            lin_add32(t_row, half * (BN / 64) + c, sum + c * 32);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p.tempty(acc));
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) {
                    uint32_t own[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) own[i] = __float_as_uint(sum[c * 32 + i]);
                    own_row(own);
                    rows_out(first + c * cols, c + 1 < BN / 64);
                }
            } else {
                const int acc = it & 1;
                ok = lin_wait(p.tfull(acc), (it >> 1) & 1, abort_flag, a.timeout_ns, a.status, 540);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
                const uint32_t t_col = t_row + half * each;
#pragma unroll 1
                for (int c = 0; c < each; c += cols) {
                    if (first + c >= a.N) break;
                    uint32_t own[32];
                    if (gated) {
                        lin_ld16(t_col + c, own);
                        lin_ld16(t_col + wide / 2 + c, own + 16);
                    } else {
                        lin_ld16(t_col + c, own);
                        lin_ld16(t_col + c + 16, own + 16);
                    }
                    tmem_ld_wait();
                    own_row(own);
                    rows_out(first + c, c + cols < each);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p.tempty(acc));
                ++it;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * BN);
    }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The parked accumulators of linear_split_kernel, for reading by the block that finishes a slice of
// the columns: slices of BN / S columns one after the other (SwiGLU: a slice's gate half, then its up
// half), each a dense [128][columns] fp32 block, so that a peer's warp reads 1 KB of consecutive
// bytes (16-byte reads of scattered rows came to 7 bytes a cycle: 2.3 us for 64 rows at S = 4). The
// 16-byte units of a row are exchanged by the row's low bits against bank conflicts of the
// writers, whose lanes hold one row each.
struct LinPark {
    int wsh;    // log2 of the columns of a block of the layout
    int half;   // BN / 2 for SwiGLU, else BN
    bool gated;
    __device__ LinPark(int bn, int splits, bool gated_) : gated(gated_)
    {
        half = gated ? bn / 2 : bn;
        wsh = 31 - __clz(half / splits);
    }
    // float offset of the 16-byte unit that holds accumulator columns col .. col + 3 of a row
    __device__ int unit(int row, int col) const
    {
        const int up = col >= half ? 1 : 0, c = col - up * half;
        const int blk = gated ? (c >> wsh) * 2 + up : c >> wsh;
        const int u = (c & ((1 << wsh) - 1)) >> 2;
        return (((blk * lin::BM + row) << wsh)) + ((u ^ (row & ((1 << (wsh - 2)) - 1))) << 2);
    }
};

// One tile per cluster of a.splits blocks (launched with that cluster width).
template <int BN, bool A_MN, bool B_MN, bool PROMOTE>
__global__ void __launch_bounds__(lin::THREADS, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ LinearArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    LinPipe<BN, A_MN, B_MN> p;
    p.smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~static_cast<uintptr_t>(1023));
    constexpr int TMEM_COLS = PROMOTE ? 2 * BN : BN;
    static_assert(lin::BM * BN * 4 <= lin::stages(BN) * lin::stage_bytes(BN), "the parked tile fits the stages");
    uint64_t *bars = reinterpret_cast<uint64_t *>(p.smem + lin::stages(BN) * lin::stage_bytes(BN));
    p.bar0 = smem_u32(bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + lin::num_bars(BN));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = a.splits;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    order_launch_dependents();
    if (threadIdx.x == 0) {
        p.init_bars(true);
        *abort_flag = 0;
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int mt, nt;
    lin_tile(blockIdx.x / S, a, mt, nt);
    const int kb0 = (int)((int64_t)rank * a.k_blocks / S), kb1 = (int)((int64_t)(rank + 1) * a.k_blocks / S);
    const int run = PROMOTE ? lin::PROMOTE_K / lin::bk(BN) : kb1 - kb0;
    const bool gated = a.act == 0;
    const int tc = gated ? BN / 2 : BN;
    const int rows = min(lin::BM, a.M - mt * lin::BM);
    float *park = reinterpret_cast<float *>(p.smem);
    const LinPark lay(BN, S, gated);
    order_wait();
    if (a.clear_status && blockIdx.x == 0 && threadIdx.x == 0) { // no wait has run out yet (LEAST_WAIT_NS)
        a.status[0] = DEV_OK;
        a.status[1] = 0;
    }

    if (warp == 0) {
        uint32_t armed = 0;
        p.produce(tmA, tmB, a, LinItem{mt, nt * tc, BN}, kb0, kb1, abort_flag, armed);
        p.drain(armed, a.timeout_ns);
    } else if (warp == 1) {
        int it = 0;
        p.multiply_runs(a, tmem, BN, kb0, kb1, run, it, abort_flag);
        if (lin_elect()) umma_commit(p.done()); // every product issued is finished
        __syncwarp();
    } else {
        const int q = warp & 3, half = warp >= 6 ? 1 : 0;
        bool ok = true;
        const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16);
        if constexpr (PROMOTE) {
            float sum[BN / 2];
#pragma unroll
            for (int i = 0; i < BN / 2; ++i) sum[i] = 0.0f;
            int it = 0;
            for (int kb = kb0; ok && kb < kb1; kb += run, ++it) {
                const int acc = it & 1;
                ok = lin_wait(p.tfull(acc), (it >> 1) & 1, abort_flag, a.timeout_ns, a.status, 540);
                if (!ok) break;
                if (q * 32 < rows) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < BN / 64; ++c)
                        lin_add32(t_row + (uint32_t)(acc * BN), half * (BN / 64) + c, sum + c * 32);
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p.tempty(acc));
            }
            // the stages are free once every product has read them (an abort: once those issued have)
            volatile int never = 0;
            ok = lin_wait(p.done(), 0, &never, 2 * a.timeout_ns, a.status, 545);
            if (ok && q * 32 < rows) {
                const int row = q * 32 + lane;
#pragma unroll
                for (int i = 0; i < BN / 8; ++i)
                    *reinterpret_cast<float4 *>(park + lay.unit(row, half * (BN / 2) + i * 4)) =
                        make_float4(sum[i * 4], sum[i * 4 + 1], sum[i * 4 + 2], sum[i * 4 + 3]);
            }
        } else {
            // the products issued finish on their own: this wait ends with them, or runs out
            volatile int never = 0;
            ok = lin_wait(p.done(), 0, &never, 2 * a.timeout_ns, a.status, 540);
            if (ok && q * 32 < rows) {
                tc_fence_after();
                const int row = q * 32 + lane;
#pragma unroll 1
                for (int c = half * (BN / 64); c < (half + 1) * (BN / 64); ++c) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(t_row + c * 32, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(park + lay.unit(row, c * 32 + i * 4)) =
                            make_uint4(r[i * 4], r[i * 4 + 1], r[i * 4 + 2], r[i * 4 + 3]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (S > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
    if (warp >= 2) {
        // this block's 1/S of the tile's columns, eight at a time
        const int vsh = lay.wsh - 3; // log2 of the 8-column pieces of a row
        const uint32_t base = smem_u32(park);
        uint32_t peer[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) peer[s] = (S > 1 && s < S) ? mapa_shared(base, (uint32_t)s) : base;
        const int block0 = rank * (gated ? 2 : 1); // this slice's (gate) block of the layout
        for (int i = threadIdx.x - 64; i < (rows << vsh); i += lin::EPI_THREADS) {
            // 32 consecutive bytes of the layout: row, and the piece it holds there (its two 16-byte
            // units swapped in odd rows)
            const int row = i >> vsh, at = i & ((1 << vsh) - 1);
            const int piece = at ^ ((row >> 1) & ((1 << vsh) - 1));
            const int c = (rank << lay.wsh) + piece * 8;
            if (nt * tc + c >= a.N) continue;
            const uint4 res = lin_res8(a, mt * lin::BM + row, nt * tc + c);
            const uint32_t off = (uint32_t)(((block0 * lin::BM + row) << lay.wsh) + at * 8) * 4u;
            const uint32_t lo = off + ((row & 1) << 4), hi = off + (((row & 1) ^ 1) << 4);
            const uint32_t up = (uint32_t)(lin::BM << lay.wsh) * 4u;
            float v[8], u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.0f;
#pragma unroll
            for (int s0 = 0; s0 < 8; s0 += 4) { // four peers' parts in flight, added in rank order
                if (s0 >= S) break;
                float4 x[4][4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (s0 + s >= S) break;
                    x[s][0] = ld_cluster_f4(peer[s0 + s] + lo);
                    x[s][1] = ld_cluster_f4(peer[s0 + s] + hi);
                    if (gated) {
                        x[s][2] = ld_cluster_f4(peer[s0 + s] + lo + up);
                        x[s][3] = ld_cluster_f4(peer[s0 + s] + hi + up);
                    }
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (s0 + s >= S) break;
                    v[0] += x[s][0].x; v[1] += x[s][0].y; v[2] += x[s][0].z; v[3] += x[s][0].w;
                    v[4] += x[s][1].x; v[5] += x[s][1].y; v[6] += x[s][1].z; v[7] += x[s][1].w;
                    if (gated) {
                        u[0] += x[s][2].x; u[1] += x[s][2].y; u[2] += x[s][2].z; u[3] += x[s][2].w;
                        u[4] += x[s][3].x; u[5] += x[s][3].y; u[6] += x[s][3].z; u[7] += x[s][3].w;
                    }
                }
            }
            float bv[8], bu[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) bv[j] = bu[j] = 0.0f;
            if (a.bias != nullptr) {
                lin_load_bias8(a.bias + nt * tc + c, bv);
                if (gated) lin_load_bias8(a.bias + a.up_col + nt * tc + c, bu);
            }
            lin_finish8(a, v, u, bv, bu, res, LinOut(a, mt * lin::BM + row, nt * tc + c));
        }
    }
    if (S > 1) {
        __syncwarp();
        cluster_sync_all(); // no block leaves while a peer may still read its accumulators
    }
}

// ---------------------------------------------------------------------------------------
// the gradient at the pre-activation
// ---------------------------------------------------------------------------------------

struct LinearDzArgs {
    const void *dy; // [M, N] bf16 or fp32, row stride ldy
    int64_t ldy;
    int dy_f32;
    const __nv_bfloat16 *z; // [M, N or 2N], row stride ldz (identity: not read)
    int64_t ldz;
    __nv_bfloat16 *dz;      // [M, N or 2N] dense, or nullptr (only the column sums are wanted)
    float *part;            // [chunks, N or 2N] column sums of each row chunk, or nullptr
    int M, N;
    int rows;               // rows per chunk
};

// dz (bf16, the products' operand) and the column sums of the unrounded dz, in one pass over dy
// and z. A block has 32 x 8 threads: 32 vectors of eight columns, sixteen rows at a time (two a
// thread, their loads in flight together); the sums over a chunk's rows run in fp32 in a fixed order
// (rows of one thread, then the eight threads). Bound by the bytes of dy, z and dz.
template <int ACT, bool F32>
__global__ void __launch_bounds__(256, ACT == 0 ? 3 : 5) linear_dz_kernel(const __grid_constant__ LinearDzArgs a)
{
    constexpr bool GATED = ACT == 0;
    constexpr int ND = F32 ? 2 : 1; // 16-byte pieces of eight dy
    order_launch_dependents();
    order_wait();
    __shared__ float red[8][32][17];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int col = (blockIdx.x * 32 + tx) * 8;
    const int cols = GATED ? 2 * a.N : a.N;
    const int r1 = min(a.M, ((int)blockIdx.y + 1) * a.rows);
    float sg[8], su[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[i] = su[i] = 0.0f;
    struct Row {
        uint4 d[ND], g, u;
    };
    auto load = [&](int row, Row &x) {
        const char *p = static_cast<const char *>(a.dy) + ((size_t)row * a.ldy + col) * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < ND; ++i) x.d[i] = reinterpret_cast<const uint4 *>(p)[i];
        if (ACT != 3) {
            const __nv_bfloat16 *zr = a.z + (size_t)row * a.ldz + col;
            x.g = *reinterpret_cast<const uint4 *>(zr);
            if (GATED) x.u = *reinterpret_cast<const uint4 *>(zr + a.N);
        }
    };
    auto unpack = [](const uint4 &x, float (&v)[8]) {
        v[0] = bf16_lo(x.x); v[1] = bf16_hi(x.x); v[2] = bf16_lo(x.y); v[3] = bf16_hi(x.y);
        v[4] = bf16_lo(x.z); v[5] = bf16_hi(x.z); v[6] = bf16_lo(x.w); v[7] = bf16_hi(x.w);
    };
    auto use = [&](int row, const Row &x) {
        float d[8], g[8], u[8];
        if (F32) {
            d[0] = __uint_as_float(x.d[0].x); d[1] = __uint_as_float(x.d[0].y);
            d[2] = __uint_as_float(x.d[0].z); d[3] = __uint_as_float(x.d[0].w);
            d[4] = __uint_as_float(x.d[ND - 1].x); d[5] = __uint_as_float(x.d[ND - 1].y);
            d[6] = __uint_as_float(x.d[ND - 1].z); d[7] = __uint_as_float(x.d[ND - 1].w);
        } else {
            unpack(x.d[0], d);
        }
        if (ACT != 3) unpack(x.g, g);
        if (GATED) unpack(x.u, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (GATED) {
                // the gate's factors first: 0 where it is shut, so that no product overflows before them
                const float s = lin_sigmoid(g[i]);
                const float du = d[i] * (g[i] * s);
                d[i] *= u[i] * (s * fmaf(g[i], 1.0f - s, 1.0f));
                u[i] = du;
                su[i] += du;
            } else if (ACT == 1) {
                d[i] *= lin_gelu_grad(g[i]);
            } else if (ACT == 2) {
                d[i] = g[i] > 0.0f ? d[i] : 0.0f;
            }
            sg[i] += d[i];
        }
        if (a.dz != nullptr) {
            __nv_bfloat16 *o = a.dz + (size_t)row * cols + col;
            *reinterpret_cast<uint4 *>(o) = lin_pack8(d);
            if (GATED) *reinterpret_cast<uint4 *>(o + a.N) = lin_pack8(u);
        }
    };
    if (col < a.N) {
        int row = blockIdx.y * a.rows + ty;
        for (; row + 8 < r1; row += 16) {
            Row x, y;
            load(row, x);
            load(row + 8, y);
            use(row, x);
            use(row + 8, y);
        }
        if (row < r1) {
            Row x;
            load(row, x);
            use(row, x);
        }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        red[ty][tx][i] = sg[i];
        red[ty][tx][8 + i] = su[i];
    }
    __syncthreads();
    // 256 gate (or plain) sums, then 256 up sums
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const int v = threadIdx.x >> 3, i = threadIdx.x & 7;
        const int c = (blockIdx.x * 32 + v) * 8 + i;
        if (c < a.N) {
            float s = 0.0f;
#pragma unroll
            for (int y = 0; y < 8; ++y) s += red[y][v][h * 8 + i];
            a.part[(size_t)blockIdx.y * cols + h * a.N + c] = s;
        }
    }
}

struct LinearDbiasArgs {
    const float *part; // [chunks, cols]
    float *dbias;      // [cols]
    int chunks, cols;
};

// dbias[c] = the chunks' sums: eight threads a column take every eighth chunk in order, then the
// eight in order. A block has 32 columns.
__global__ void __launch_bounds__(256)
    linear_dbias_kernel(const __grid_constant__ LinearDbiasArgs a)
{
    order_launch_dependents();
    order_wait();
    __shared__ float red[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    float s = 0.0f;
    if (c < a.cols) {
#pragma unroll 8
        for (int i = ty; i < a.chunks; i += 8) s += a.part[(size_t)i * a.cols + c];
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < a.cols) {
        float t = 0.0f;
#pragma unroll
        for (int y = 0; y < 8; ++y) t += red[y][tx];
        a.dbias[c] = t;
    }
}

} // namespace moe
