// ops_api.cu -- the C ABI of the operators around the layer (include/moe.h): routing by scores,
// the dense product with its epilogue, dropout with the residual, and their gradients. This
// file only validates, plans and launches.
#include "moe.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "dropout.cuh"
#include "host.cuh"
#include "linear.cuh"
#include "select.cuh"

namespace {

using namespace moe;

// A launch in programmatic order (order.cuh).
template <typename A>
cudaError_t launch_ordered(void (*kern)(A), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args);
}

// ---------------------------------------------------------------------------------------
// routing by scores
// ---------------------------------------------------------------------------------------

moe_status check_select(const moe_select *s)
{
    if (s == nullptr) return MOE_ERR_INVALID_ARG;
    if (s->T < 0 || s->E <= 0 || s->top_k <= 0 || s->top_k > s->E) return MOE_ERR_INVALID_ARG;
    if (s->score != MOE_SCORE_SOFTMAX && s->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (s->group_score != MOE_GROUP_MAX && s->group_score != MOE_GROUP_SUM2) return MOE_ERR_INVALID_ARG;
    if (s->dtype != MOE_DTYPE_BF16 && s->dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (s->n_group <= 0 || s->top_group <= 0 || s->top_group > s->n_group || s->E % s->n_group != 0)
        return MOE_ERR_INVALID_ARG;
    // the groups that stay hold at least top_k experts
    if ((int64_t)(s->E / s->n_group) * s->top_group < s->top_k) return MOE_ERR_INVALID_ARG;
    if (s->ld != 0 && s->ld < s->E) return MOE_ERR_INVALID_ARG;
    if (!(s->scale > 0.0f) || !(s->scale <= 3.0e38f)) return MOE_ERR_INVALID_ARG;
    if (s->E > 1024 || s->top_k > SEL_MAX_K || s->n_group > SEL_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int dtype_bytes(int32_t d) { return d == MOE_DTYPE_F32 ? 4 : 2; }
bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % (unsigned)bytes) == 0; }

template <int LPT, int EPT, typename LT, bool BIASED>
cudaError_t launch_select(const SelectArgs &a, cudaStream_t st)
{
    constexpr int warps = sel_threads(LPT, EPT) / 32, per_block = warps * (32 / LPT);
    const int smem = sel_smem(LPT, EPT, warps, a.E, BIASED);
    static_assert(sel_smem(LPT, EPT, warps, LPT * EPT, BIASED) <= 48 * 1024, "no opt-in needed");
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const int64_t blocks = ((int64_t)a.T + per_block - 1) / per_block;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * sel_blocks(LPT, EPT));
    route_select_kernel<LPT, EPT, LT, BIASED><<<grid, warps * 32, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename LT, bool BIASED> cudaError_t launch_select_wide(const SelectArgs &a, cudaStream_t st)
{
    // Four tokens per warp where they fit (k <= 8, E <= 256, groups of whole lanes) and there are
    // enough of them: fewer instructions a token, but longer chains a lane. Measured on the device, a
    // warp each against eight lanes each: E = 256 (8 groups, bias) T = 4096 7.6 / 8.2 us, 8192 10.0 / 9.8,
    // 16384 16.8 / 14.0; E = 128 (the same) 6.2 / 7.0, 8.5 / 8.0, 13.6 / 10.5; E = 64 3.9 / 4.8, 5.6 / 4.6,
    // 8.8 / 6.2; E = 32 T = 2048 2.8 / 3.2, 4096 3.6 / 3.7, 8192 5.2 / 4.0; E = 16 2.8 / 3.0, 3.6 / 3.1,
    // 5.2 / 3.3; E = 8 2.6 / 2.6, 3.2 / 2.6, 4.5 / 2.7.
    int ept = 1;
    while (ept * 8 < a.E) ept *= 2;
    const int lanes = a.gsz / ept;
    const bool fits = a.k <= 8 && a.E <= 256 &&
                      (a.groups == 1 || (a.gsz % ept == 0 && (lanes & (lanes - 1)) == 0));
    if (fits && a.T >= (a.E <= 16 ? 4096 : 8192)) {
        switch (ept) {
        case 1: return launch_select<8, 1, LT, BIASED>(a, st);
        case 2: return launch_select<8, 2, LT, BIASED>(a, st);
        case 4: return launch_select<8, 4, LT, BIASED>(a, st);
        case 8: return launch_select<8, 8, LT, BIASED>(a, st);
        case 16: return launch_select<8, 16, LT, BIASED>(a, st);
        default: return launch_select<8, 32, LT, BIASED>(a, st);
        }
    }
    if (a.E <= 32) return launch_select<32, 1, LT, BIASED>(a, st);
    if (a.E <= 64) return launch_select<32, 2, LT, BIASED>(a, st);
    if (a.E <= 128) return launch_select<32, 4, LT, BIASED>(a, st);
    if (a.E <= 256) return launch_select<32, 8, LT, BIASED>(a, st);
    if (a.E <= 512) return launch_select<32, 16, LT, BIASED>(a, st);
    return launch_select<32, 32, LT, BIASED>(a, st);
}

template <typename LT> cudaError_t launch_select_any(const SelectArgs &a, cudaStream_t st)
{
    return a.bias != nullptr ? launch_select_wide<LT, true>(a, st) : launch_select_wide<LT, false>(a, st);
}

// ---------------------------------------------------------------------------------------
// dense product
// ---------------------------------------------------------------------------------------

std::atomic<int> g_linear_tile{0}, g_linear_split{0};

struct LinearDims {
    int64_t cols; // columns of W: N, or 2N for SwiGLU
    int64_t ldx, ldw, ldr, ldy, ldz;
};

moe_status check_linear(const moe_linear *p, LinearDims *d)
{
    if (p == nullptr) return MOE_ERR_INVALID_ARG;
    if (p->M < 0 || p->N <= 0 || p->K <= 0) return MOE_ERR_INVALID_ARG;
    if (p->act < MOE_ACT_SWIGLU || p->act > MOE_ACT_IDENTITY) return MOE_ERR_INVALID_ARG;
    if (p->w_layout != MOE_W_KN && p->w_layout != MOE_W_NK) return MOE_ERR_INVALID_ARG;
    if (p->out_dtype != MOE_DTYPE_BF16 && p->out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (p->N % 8 != 0 || p->K % 8 != 0) return MOE_ERR_UNSUPPORTED;
    if (p->M > (1 << 30) || p->N > (1 << 28) || p->K > (1 << 28)) return MOE_ERR_UNSUPPORTED;
    d->cols = p->act == MOE_ACT_SWIGLU ? 2 * (int64_t)p->N : p->N;
    const bool kn = p->w_layout == MOE_W_KN;
    const int64_t w_row = kn ? d->cols : p->K;
    if ((p->ldx != 0 && p->ldx < p->K) || (p->ldw != 0 && p->ldw < w_row) ||
        (p->ldr != 0 && p->ldr < p->N) || (p->ldy != 0 && p->ldy < p->N) ||
        (p->ldz != 0 && p->ldz < d->cols))
        return MOE_ERR_INVALID_ARG;
    d->ldx = p->ldx ? p->ldx : p->K;
    d->ldw = p->ldw ? p->ldw : w_row;
    d->ldr = p->ldr ? p->ldr : p->N;
    d->ldy = p->ldy ? p->ldy : p->N;
    d->ldz = p->ldz ? p->ldz : d->cols;
    const int yv = p->out_dtype == MOE_DTYPE_F32 ? 4 : 8;
    if (d->ldx % 8 || d->ldw % 8 || d->ldr % 8 || d->ldz % 8 || d->ldy % yv) return MOE_ERR_UNSUPPORTED;
    if (std::max({d->ldx, d->ldw, d->ldr, d->ldy, d->ldz}) >= (1LL << 38)) return MOE_ERR_UNSUPPORTED;
    const int64_t mt = ((int64_t)p->M + lin::BM - 1) / lin::BM;
    // tile counts of the three products in 32 bits
    const int64_t kt = (p->K + 63) / 64, ct = (d->cols + 63) / 64;
    if (mt * ct * 8 >= (1LL << 31) || mt * kt * 8 >= (1LL << 31) || kt * ct * 8 >= (1LL << 31))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// 2D bf16 [rows, cols] with row stride ld; box of 64 columns x box_rows rows, 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t ld,
              uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct LinearPlan {
    int bn;     // tile columns
    int splits; // 0: the persistent kernel; else blocks per cluster
};

// Tile width and k split by an estimate of one launch's time in microseconds, from measurements at
// 1 to 8192 rows (device time): a 64-value block of k of a 128 x BN tile takes 0.30, 0.19, 0.165 (BN = 256, 128,
// 64); a persistent launch pays start and last epilogue once (7.0, 5.5), a split one per tile, more of
// it for more rows and splits. Measured, the choice against the best of the others: 1 x 4096 x 4096
// (M x K x N) 9.7 (128 columns, 4 splits) / 10.4; 64 x 7168 x 2 * 2048 SwiGLU 16.1 (128, 4) / 19.2;
// 128 x 4096 x 4096 12.8 (64, 2) / 14.5; 512 x 4096 x 4096 21.3 (128) / 22.4; 4096 x 7168 x 256 fp32
// 22.2 (128, 2) / 25.9; 4096^3 104 (256) / 119. `wide`: 256-column tiles are possible (not for fp32
// outputs, whose sums are kept in registers).
LinearPlan plan_linear(int64_t M, int64_t n_out, bool gated, int64_t K, bool wide, int sms)
{
    const int ft = g_linear_tile.load(), fs = g_linear_split.load();
    LinearPlan best{wide ? 256 : 128, 0};
    double tbest = 1e300;
    const int64_t mt = (M + lin::BM - 1) / lin::BM;
    const double r = (M < lin::BM ? (double)M : (double)lin::BM) / 64.0;
    auto consider = [&](int bn, int s) {
        if (ft != 0 && (bn != ft || s != fs)) return;
        const int tc = gated ? bn / 2 : bn;
        const int64_t tiles = mt * ((n_out + tc - 1) / tc);
        const int64_t kb = (K + lin::bk(bn) - 1) / lin::bk(bn);
        if (s > kb) return;
        const double step = lin::sub(bn) * (bn == 256 ? 0.30 : bn == 128 ? 0.19 : 0.165);
        double t;
        if (s == 0) {
            const int64_t rest = tiles % sms;
            double waves = (double)((tiles + sms - 1) / sms);
            if (bn == 256 && tiles > sms && rest > 0 && 2 * rest <= sms) waves -= 0.4; // the last in halves
            t = (bn == 256 ? 7.0 : 5.5) + waves * kb * step;
        } else {
            const int64_t waves = (tiles * s + sms - 1) / sms;
            t = waves * (3.0 + 1.5 * r + (s - 1) * (0.5 + 0.47 * r) + (double)((kb + s - 1) / s) * step);
        }
        if (t < tbest) {
            tbest = t;
            best = LinearPlan{bn, s};
        }
    };
    if (wide) consider(256, 0);
    consider(128, 0);
    for (int s = 1; s <= 8; s *= 2) {
        consider(128, s);
        if (!gated) consider(64, s);
    }
    return best;
}

template <int BN, bool A_MN, bool B_MN, bool PROMOTE, bool SPLIT>
cudaError_t launch_linear_kernel(const CUtensorMap &ta, const CUtensorMap &tb, const LinearArgs &a, int sms,
                                 cudaStream_t st)
{
    void (*kern)(CUtensorMap, CUtensorMap, LinearArgs);
    if constexpr (SPLIT)
        kern = linear_split_kernel<BN, A_MN, B_MN, PROMOTE>;
    else
        kern = linear_kernel<BN, A_MN, B_MN, PROMOTE>;
    // dynamic shared memory, allowed once per device
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute((const void *)kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 lin::smem_bytes(BN, SPLIT));
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * a.splits : std::min<int64_t>(tiles, sms)));
    cfg.blockDim = dim3(lin::THREADS);
    cfg.dynamicSmemBytes = lin::smem_bytes(BN, SPLIT);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    // the next call's blocks are set up while this one's run (they wait for its end before they read)
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ta, tb, a);
}

template <bool A_MN, bool B_MN, bool PROMOTE>
cudaError_t launch_linear_plan(const LinearPlan &p, const CUtensorMap &ta, const CUtensorMap &tb,
                               const LinearArgs &a, int sms, cudaStream_t st)
{
    if (p.splits != 0)
        return p.bn == 128 ? launch_linear_kernel<128, A_MN, B_MN, PROMOTE, true>(ta, tb, a, sms, st)
                           : launch_linear_kernel<64, A_MN, B_MN, PROMOTE, true>(ta, tb, a, sms, st);
    if constexpr (!PROMOTE)
        if (p.bn == 256) return launch_linear_kernel<256, A_MN, B_MN, false, false>(ta, tb, a, sms, st);
    return launch_linear_kernel<128, A_MN, B_MN, PROMOTE, false>(ta, tb, a, sms, st);
}

// One product of the tile loop. A is [M, K] (K-major) or [K, M] (MN-major), B [N, K] or [K, N];
// `a` carries M, N, act, epilogue operands and the status word.
template <bool A_MN, bool B_MN>
cudaError_t launch_linear(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_cols, int64_t K,
                          LinearArgs a, cudaStream_t st)
{
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const bool gated = a.act == 0;
    const bool promote = a.y_f32 && K > lin::PROMOTE_K;
    const LinearPlan p = plan_linear(a.M, a.N, gated, K, !promote, sms);
    const int tc = gated ? p.bn / 2 : p.bn;
    a.k_blocks = (int)((K + lin::bk(p.bn) - 1) / lin::bk(p.bn));
    a.m_tiles = (a.M + lin::BM - 1) / lin::BM;
    a.n_tiles = (a.N + tc - 1) / tc;
    a.group_m = 16;
    a.splits = p.splits;
    a.a_rows = std::min(lin::BM, (a.M + 7) / 8 * 8);
    a.timeout_ns = std::max<int64_t>(g_timeout_ns.load(), lin::LEAST_WAIT_NS);
    // a last wave of at most half the SMs' tiles is worked in halves
    const int tiles = a.m_tiles * a.n_tiles, rest = tiles % sms;
    a.full = tiles > sms && 2 * rest <= sms ? tiles - rest : tiles;
    CUtensorMap ta, tb;
    const bool ok = (A_MN ? make_map(&ta, A, (uint64_t)K, (uint64_t)a.M, (uint64_t)lda, 64)
                          : make_map(&ta, A, (uint64_t)a.M, (uint64_t)K, (uint64_t)lda, (uint32_t)a.a_rows)) &&
                    (B_MN ? make_map(&tb, B, (uint64_t)K, (uint64_t)b_cols, (uint64_t)ldb, 64)
                          : make_map(&tb, B, (uint64_t)b_cols, (uint64_t)K, (uint64_t)ldb,
                                     p.bn == 256 ? 64u : (uint32_t)tc));
    if (!ok) return cudaErrorInvalidValue;
    if constexpr (!A_MN) // gradients of W are bf16
        if (promote) return launch_linear_plan<A_MN, B_MN, true>(p, ta, tb, a, sms, st);
    return launch_linear_plan<A_MN, B_MN, false>(p, ta, tb, a, sms, st);
}

template <int ACT> cudaError_t launch_dz_of(const LinearDzArgs &a, dim3 grid, cudaStream_t st)
{
    return a.dy_f32 ? launch_ordered(linear_dz_kernel<ACT, true>, grid, 256, 0, st, a)
                    : launch_ordered(linear_dz_kernel<ACT, false>, grid, 256, 0, st, a);
}

cudaError_t launch_dz(const LinearDzArgs &a, int act, int chunks, cudaStream_t st)
{
    const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)chunks);
    switch (act) {
    case MOE_ACT_SWIGLU: return launch_dz_of<MOE_ACT_SWIGLU>(a, grid, st);
    case MOE_ACT_GELU_TANH: return launch_dz_of<MOE_ACT_GELU_TANH>(a, grid, st);
    case MOE_ACT_RELU: return launch_dz_of<MOE_ACT_RELU>(a, grid, st);
    default: return launch_dz_of<MOE_ACT_IDENTITY>(a, grid, st);
    }
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Backward workspace: the status word; dz where it is not dy itself; the row chunks' column sums.
struct LinearBwdLayout {
    size_t dz, part, end;
    int chunks, rows;
    bool need_dz;
};

LinearBwdLayout linear_bwd_layout(const moe_linear *p, const LinearDims &d)
{
    LinearBwdLayout L{};
    L.need_dz = p->act != MOE_ACT_IDENTITY || p->out_dtype == MOE_DTYPE_F32;
    // one wave of blocks over the column blocks of 148 SMs, five per SM (SwiGLU three: more registers),
    // whole groups of 8 rows; 4096 x 6400 GELU: 31.0 us, against 36.9 with six per SM. Not the current
    // device's count: the workspace's size does not depend on a device, and sums are added in the same
    // order on each
    const int64_t cb = (p->N + 255) / 256;
    int64_t chunks = std::max<int64_t>(1, 148 * (p->act == MOE_ACT_SWIGLU ? 3 : 5) / cb);
    const int64_t groups = std::max<int64_t>(1, ((int64_t)p->M + 7) / 8);
    chunks = std::min(chunks, groups);
    L.rows = (int)((groups + chunks - 1) / chunks * 8);
    L.chunks = (int)std::max<int64_t>(1, ((int64_t)p->M + L.rows - 1) / L.rows);
    L.dz = 256;
    L.part = align256(L.dz + (L.need_dz ? (size_t)p->M * d.cols * 2 : 0));
    L.end = align256(L.part + (size_t)L.chunks * d.cols * 4);
    return L;
}

// ---------------------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------------------

// Groups per thread and turn: what keeps 64 to 96 bytes a thread in flight. Measured at 2^25
// elements, 1 / 2 / 4 groups: bf16 with a residual 36.7 / 31.4 / 38.9 us, without 32.2 / 29.5 / 27.4;
// fp32 61.9 / 66.1 / 64.7 and 44.4 / 51.6 / 55.6.
template <typename DT> cudaError_t launch_dropout(const DropoutArgs &a, cudaStream_t st)
{
    constexpr bool half = sizeof(DT) == 2;
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const int64_t blocks = ((a.n + 7) / 8 + 255) / 256;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * 8);
    return a.res != nullptr ? launch_ordered(dropout_add_kernel<DT, true, half ? 2 : 1>, grid, 256, 0, st, a)
                            : launch_ordered(dropout_add_kernel<DT, false, half ? 4 : 1>, grid, 256, 0, st, a);
}

} // namespace

extern "C" {

moe_status moe_route_select(const moe_select *s, const void *logits, const float *bias,
                            int32_t *topk_idx, float *topk_w, const int32_t *n_rows, void *stream)
{
    const moe_status c = check_select(s);
    if (c != MOE_OK) return c;
    if (s->T == 0) return MOE_OK;
    if (logits == nullptr || topk_idx == nullptr || topk_w == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, dtype_bytes(s->dtype)) || !aligned4(bias) || !aligned4(topk_idx) ||
        !aligned4(topk_w) || !aligned4(n_rows))
        return MOE_ERR_INVALID_ARG;
    SelectArgs a{};
    a.logits = logits;
    a.ld = s->ld ? s->ld : s->E;
    a.bias = bias;
    a.idx = topk_idx;
    a.w = topk_w;
    a.n_rows = n_rows;
    a.T = s->T;
    a.E = s->E;
    a.k = s->top_k;
    a.sigmoid = s->score == MOE_SCORE_SIGMOID;
    a.groups = s->n_group;
    a.gsz = s->E / s->n_group;
    a.keep = s->top_group;
    a.sum2 = s->group_score == MOE_GROUP_SUM2;
    a.renorm = s->renorm != 0;
    a.scale = s->scale;
    a.vec = aligned16(logits) && a.ld * dtype_bytes(s->dtype) % 16 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return to_status(s->dtype == MOE_DTYPE_F32 ? launch_select_any<float>(a, st)
                                               : launch_select_any<__nv_bfloat16>(a, st));
}

moe_status moe_route_select_backward(const moe_select *s, const void *logits, const int32_t *topk_idx,
                                     const float *dtopk_w, void *dlogits, const int32_t *n_rows,
                                     void *stream)
{
    const moe_status c = check_select(s);
    if (c != MOE_OK) return c;
    if (s->T == 0) return MOE_OK;
    if (logits == nullptr || topk_idx == nullptr || dtopk_w == nullptr || dlogits == nullptr)
        return MOE_ERR_INVALID_ARG;
    const int b = dtype_bytes(s->dtype);
    if (!aligned_to(logits, b) || !aligned_to(dlogits, b) || !aligned4(topk_idx) || !aligned4(dtopk_w) ||
        !aligned4(n_rows))
        return MOE_ERR_INVALID_ARG;
    SelectBwdArgs a{};
    a.logits = logits;
    a.ld = s->ld ? s->ld : s->E;
    a.idx = topk_idx;
    a.dw = dtopk_w;
    a.dlogits = dlogits;
    a.ldd = s->E;
    a.n_rows = n_rows;
    a.T = s->T;
    a.E = s->E;
    a.k = s->top_k;
    a.sigmoid = s->score == MOE_SCORE_SIGMOID;
    a.renorm = s->renorm != 0;
    a.scale = s->scale;
    a.vec = aligned16(dlogits) && (int64_t)s->E * b % 16 == 0;
    const unsigned grid = (unsigned)(((int64_t)a.T + 7) / 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (s->dtype == MOE_DTYPE_F32)
        route_select_bwd_kernel<float><<<grid, 256, 0, st>>>(a);
    else
        route_select_bwd_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    return to_status(cudaGetLastError());
}

size_t moe_linear_workspace_size(const moe_linear *p)
{
    LinearDims d;
    return check_linear(p, &d) == MOE_OK ? 256 : 0;
}

size_t moe_linear_backward_workspace_size(const moe_linear *p)
{
    LinearDims d;
    return check_linear(p, &d) == MOE_OK ? linear_bwd_layout(p, d).end : 0;
}

moe_status moe_linear_forward(const moe_linear *p, const moe_bf16 *x, const moe_bf16 *W, const float *bias,
                              const moe_bf16 *residual, void *y, moe_bf16 *z, void *ws, size_t ws_bytes,
                              void *stream)
{
    LinearDims d;
    const moe_status c = check_linear(p, &d);
    if (c != MOE_OK) return c;
    if (W == nullptr || ws == nullptr || (p->M > 0 && (x == nullptr || y == nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < 256) return MOE_ERR_WORKSPACE;
    if (!aligned16(x) || !aligned16(W) || !aligned16(bias) || !aligned16(residual) || !aligned16(y) ||
        !aligned16(z) || !aligned16(ws))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->M == 0) return to_status(cudaMemsetAsync(ws, 0, 8, st));
    LinearArgs a{};
    a.M = p->M;
    a.N = p->N;
    a.act = p->act;
    a.up_col = p->N;
    a.bias = bias;
    a.res = reinterpret_cast<const __nv_bfloat16 *>(residual);
    a.ldr = d.ldr;
    a.y = y;
    a.ldy = d.ldy;
    a.y_f32 = p->out_dtype == MOE_DTYPE_F32;
    a.z = reinterpret_cast<__nv_bfloat16 *>(z);
    a.ldz = d.ldz;
    a.status = static_cast<int *>(ws);
    a.clear_status = 1;
    return to_status(p->w_layout == MOE_W_KN
                         ? launch_linear<false, true>(x, d.ldx, W, d.ldw, d.cols, p->K, a, st)
                         : launch_linear<false, false>(x, d.ldx, W, d.ldw, d.cols, p->K, a, st));
}

moe_status moe_linear_backward(const moe_linear *p, const moe_bf16 *x, const moe_bf16 *W, const moe_bf16 *z,
                               const void *dy, moe_bf16 *dx, moe_bf16 *dW, float *dbias, void *ws,
                               size_t ws_bytes, void *stream)
{
    LinearDims d;
    const moe_status c = check_linear(p, &d);
    if (c != MOE_OK) return c;
    if (ws == nullptr || (dx == nullptr && dW == nullptr && dbias == nullptr)) return MOE_ERR_INVALID_ARG;
    if (p->M > 0 && (dy == nullptr || (p->act != MOE_ACT_IDENTITY && z == nullptr) ||
                     (dx != nullptr && W == nullptr) || (dW != nullptr && x == nullptr)))
        return MOE_ERR_INVALID_ARG;
    const LinearBwdLayout L = linear_bwd_layout(p, d);
    if (ws_bytes < L.end) return MOE_ERR_WORKSPACE;
    if (!aligned16(x) || !aligned16(W) || !aligned16(z) || !aligned16(dy) || !aligned16(dx) ||
        !aligned16(dW) || !aligned4(dbias) || !aligned16(ws))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (p->M == 0) { // no rows: the weights' gradients are zero
        e = cudaMemsetAsync(ws, 0, 8, st);
        if (e == cudaSuccess && dW != nullptr) e = cudaMemsetAsync(dW, 0, (size_t)p->K * d.cols * 2, st);
        if (e == cudaSuccess && dbias != nullptr) e = cudaMemsetAsync(dbias, 0, (size_t)d.cols * 4, st);
        return to_status(e);
    }
    char *w = static_cast<char *>(ws);
    const bool gemms = dx != nullptr || dW != nullptr;
    const bool make_dz = L.need_dz && gemms;
    float *part = reinterpret_cast<float *>(w + L.part);
    if (make_dz || dbias != nullptr) {
        LinearDzArgs z_{};
        z_.dy = dy;
        z_.ldy = d.ldy;
        z_.dy_f32 = p->out_dtype == MOE_DTYPE_F32;
        z_.z = reinterpret_cast<const __nv_bfloat16 *>(z);
        z_.ldz = d.ldz;
        z_.dz = make_dz ? reinterpret_cast<__nv_bfloat16 *>(w + L.dz) : nullptr;
        z_.part = dbias == nullptr ? nullptr : L.chunks == 1 ? dbias : part;
        z_.M = p->M;
        z_.N = p->N;
        z_.rows = L.rows;
        e = launch_dz(z_, p->act, L.chunks, st);
        if (e == cudaSuccess && dbias != nullptr && L.chunks > 1) {
            e = launch_ordered(linear_dbias_kernel, dim3((unsigned)((d.cols + 31) / 32)), 256, 0, st,
                               LinearDbiasArgs{part, dbias, L.chunks, (int)d.cols});
        }
    }
    if (!gemms) {
        if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0, 8, st);
        return to_status(e);
    }
    const void *g = make_dz ? static_cast<const void *>(w + L.dz) : dy;
    const int64_t ldg = make_dz ? d.cols : d.ldy;
    LinearArgs a{};
    a.act = MOE_ACT_IDENTITY;
    a.status = static_cast<int *>(ws);
    const bool kn = p->w_layout == MOE_W_KN;
    if (e == cudaSuccess && dx != nullptr) { // dx [M, K] = dz [M, cols] W^T
        LinearArgs b = a;
        b.M = p->M;
        b.N = p->K;
        b.y = dx;
        b.clear_status = 1;
        b.ldy = p->K;
        e = kn ? launch_linear<false, false>(g, ldg, W, d.ldw, p->K, d.cols, b, st)
               : launch_linear<false, true>(g, ldg, W, d.ldw, p->K, d.cols, b, st);
    }
    if (e == cudaSuccess && dW != nullptr) { // x^T dz [K, cols], or dz^T x [cols, K]
        LinearArgs b = a;
        b.M = kn ? p->K : (int)d.cols;
        b.N = kn ? (int)d.cols : p->K;
        b.y = dW;
        b.clear_status = dx == nullptr;
        b.ldy = b.N;
        e = kn ? launch_linear<true, true>(x, d.ldx, g, ldg, d.cols, p->M, b, st)
               : launch_linear<true, true>(g, ldg, x, d.ldx, p->K, p->M, b, st);
    }
    return to_status(e);
}

int moe_set_linear_plan(int tile_n, int splits)
{
    const bool ok = tile_n == 0 || (splits == 0 && (tile_n == 128 || tile_n == 256)) ||
                    ((tile_n == 64 || tile_n == 128) &&
                     (splits == 1 || splits == 2 || splits == 4 || splits == 8));
    if (!ok) return -1;
    g_linear_tile.store(tile_n);
    g_linear_split.store(splits);
    return 0;
}

moe_status moe_dropout_add(int64_t n, int32_t dtype, int32_t drop, const uint64_t *rng, const void *x,
                           const void *residual, void *y, void *stream)
{
    if (n < 0 || (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) || drop < 0 || drop > 65536 ||
        rng == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (x == nullptr || y == nullptr || !aligned16(x) || !aligned16(residual) || !aligned16(y) ||
        !aligned_to(rng, 8))
        return MOE_ERR_INVALID_ARG;
    DropoutArgs a{};
    a.x = x;
    a.res = residual;
    a.y = y;
    a.rng = reinterpret_cast<const unsigned long long *>(rng);
    a.n = n;
    a.thr = (uint32_t)drop;
    a.scale = a.thr < 65536u ? 65536.0f / (float)(65536u - a.thr) : 0.0f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return to_status(dtype == MOE_DTYPE_F32 ? launch_dropout<float>(a, st)
                                            : launch_dropout<__nv_bfloat16>(a, st));
}

moe_status moe_dropout_add_backward(int64_t n, int32_t dtype, int32_t drop, const uint64_t *rng,
                                    const void *dy, void *dx, void *stream)
{
    return moe_dropout_add(n, dtype, drop, rng, dy, nullptr, dx, stream);
}

} // extern "C"
