// sba.cu -- host side of the C ABI declared in include/sba.h: argument checks,
// TMA tensor-map encoding, launches and the device status word.  The kernels come from the
// .cuh files; those of the row operators, many and long to compile, are in units of their
// own (rows.cu).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/sba.h"
#include "attention.cuh"
#include "attention2.cuh"
#include "common.cuh"
#include "select.cuh"
#include "select_fused.cuh"
#include "score_lse.cuh"
#include "pair.cuh"
#include "producer.cuh"
#include "compensation.cuh"
#include "prune.cuh"
#include "residual_norm.cuh"
#include "rotary.cuh"
#include "int8_linear.cuh"

namespace {

constexpr uint64_t kDefaultWaitLimit = 1ull << 32;  // clock cycles, ~2 s at 2 GHz
uint64_t g_wait_limit = kDefaultWaitLimit;
int g_attn_kernel = SBA_ATTN_KERNEL_AUTO;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align_up_256(size_t x) { return (x + 255) & ~size_t(255); }

sba_status check_shape(int B, int H, int Npad, int D, int block) {
    if (B <= 0 || H <= 0 || Npad <= 0) return SBA_ERR_INVALID_ARG;
    if (B > 65535 || H > 65535) return SBA_ERR_UNSUPPORTED;
    if (D != 64 && D != 128) return SBA_ERR_UNSUPPORTED;
    if (block != 64) return SBA_ERR_UNSUPPORTED;
    if (Npad % block != 0) return SBA_ERR_INVALID_ARG;
    if (Npad > SBA_MAX_NPAD) return SBA_ERR_UNSUPPORTED;
    return SBA_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// [B*H, Npad, D] bf16 viewed as a 3-D tensor; box = 64 columns (128 B) x rows x 1,
// 128-byte swizzle (the canonical K-major / MN-major SW128 operand layout).
bool make_map(CUtensorMap* map, const void* base, int BH, int Npad, int D, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Npad, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Npad * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Row-major [rows][cols] bf16 as a 2-D tensor; box = 64 columns (128 B) x box_rows,
// 128-byte swizzle.
bool make_map_2d(CUtensorMap* map, const void* base, long long rows, int cols, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// The key means of one head sampled every `stride` blocks: [BH][nB][D] bf16 viewed as
// 3-D (D, floor(nB / stride), BH) with row pitch stride * D * 2 bytes; box 64 x 128 rows.
bool make_map_sample(CUtensorMap* map, const void* base, int BH, int nB, int D, int stride) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)(nB / stride), (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)stride * D * 2, (cuuint64_t)nB * D * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Where the epilogue stores the output when it goes straight to sequence shards.
struct ShardOut {
    int n;
    int h_total;
    int h_first;
    void* const* o;
    float* const* lse;  // NULL: no lse
};

// kbar / vbar (kMeanComp only): bf16 [BH][nBpad][D] block means for the compensation steps.
template <int D, int NS, int MODE = sba::kPlain>
sba_status launch_attention(const void* q, const void* k, const void* v, void* o, float* lse,
                            int B, int H, int Npad, const int32_t* valid_len,
                            const int32_t* kv_idx, const int32_t* kv_cnt, int kmax, int dense,
                            const int32_t* pair_order, float softmax_scale, cudaStream_t stream,
                            const void* kbar = nullptr, const void* vbar = nullptr, int nBpad = 0,
                            const ShardOut* shards = nullptr) {
    using SM = sba::AttnSmem<D, NS>;
    CUtensorMap tq, tk, tv, tkb, tvb;
    const int BH = B * H;
    if (!make_map(&tq, q, BH, Npad, D, 64) || !make_map(&tk, k, BH, Npad, D, 64) ||
        !make_map(&tv, v, BH, Npad, D, 64))
        return SBA_ERR_CUDA;
    if (MODE == sba::kMeanComp) {
        if (!make_map(&tkb, kbar, BH, nBpad, D, 64) || !make_map(&tvb, vbar, BH, nBpad, D, 64)) return SBA_ERR_CUDA;
    } else {
        tkb = tk;
        tvb = tv;
    }
    const void* fn = MODE == sba::kMeanComp      ? (const void*)sba::attn_comp_kernel<D, NS>
                     : MODE == sba::kFirstOrder ? (const void*)sba::attn_first_order_kernel<D, NS>
                                                : (const void*)sba::attn_kernel<D, NS>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kAlloc) != cudaSuccess)
        return SBA_ERR_CUDA;
    sba::AttnParams p;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.valid_len = valid_len;
    p.kv_idx = kv_idx;
    p.kv_cnt = kv_cnt;
    p.pair_order = pair_order;
    p.H = H;
    p.Npad = Npad;
    p.kmax = kmax;
    p.dense = dense;
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)D);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit = g_wait_limit;
    if (shards) {
        p.n_shards = shards->n;
        p.shard_len = Npad / shards->n;
        p.h_total = shards->h_total;
        p.h_first = shards->h_first;
        for (int i = 0; i < shards->n; ++i) {
            p.o_shard[i] = static_cast<__nv_bfloat16*>(shards->o[i]);
            p.lse_shard[i] = shards->lse ? shards->lse[i] : nullptr;
        }
    }
    dim3 grid((Npad / 64 + 1) / 2, H, B);
    if (MODE == sba::kMeanComp)
        sba::attn_comp_kernel<D, NS><<<grid, 192, SM::kAlloc, stream>>>(tq, tk, tv, tkb, tvb, p);
    else if (MODE == sba::kFirstOrder)
        sba::attn_first_order_kernel<D, NS><<<grid, 192, SM::kAlloc, stream>>>(tq, tk, tv, p);
    else
        sba::attn_kernel<D, NS><<<grid, 192, SM::kAlloc, stream>>>(tq, tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

// The CTA-pair kernel (D = 128): four query blocks per 2-SM cluster, two key blocks
// per step.
template <int NS>
sba_status launch_attention_pair(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                                 int Npad, const int32_t* valid_len, const int32_t* kv_idx, const int32_t* kv_cnt,
                                 int kmax, int dense, float softmax_scale, cudaStream_t stream) {
    using SM = sba::Attn2Smem<NS>;
    CUtensorMap tq, tk, tv;
    const int BH = B * H;
    if (!make_map(&tq, q, BH, Npad, 128, 64) || !make_map(&tk, k, BH, Npad, 128, 64) ||
        !make_map(&tv, v, BH, Npad, 128, 64))
        return SBA_ERR_CUDA;
    if (cudaFuncSetAttribute(sba::attn_pair_kernel<NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kAlloc) !=
        cudaSuccess)
        return SBA_ERR_CUDA;
    sba::AttnParams p;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.valid_len = valid_len;
    p.kv_idx = kv_idx;
    p.kv_cnt = kv_cnt;
    p.pair_order = nullptr;
    p.H = H;
    p.Npad = Npad;
    p.kmax = kmax;
    p.dense = dense;
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(128.0f);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit = g_wait_limit;
    const int nQ = Npad / 64;
    dim3 grid(2 * ((nQ + 3) / 4), H, B);
    sba::attn_pair_kernel<NS><<<grid, 320, SM::kAlloc, stream>>>(tq, tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

// Routing launches shared by both routers: pool Q and K (blocks, or NSUB
// sub-blocks per block), largest key norm, screened scores on the tensor cores
// (skipped when nothing is dropped), then the per-row top-k.  Arguments checked
// by the caller.
// With qmean/kmean given (fp64 block means [BH][nB][D], NSUB = 1), pooling is replaced
// by splitting those means for the screen, and the top-k re-scores from them.
template <int D, int NSUB>
sba_status run_select(const void* q, const void* k, int B, int H, int Npad, const int32_t* valid_len,
                      double sparsity, int budget, int kmax, int32_t* kv_idx, int32_t* kv_cnt,
                      void* workspace, cudaStream_t s, const double* qmean = nullptr,
                      const double* kmean = nullptr) {
    constexpr int BLK = 64 / NSUB;
    const size_t BH = (size_t)B * H;
    const int nB = Npad / 64;
    const int nP = nB * NSUB;
    sba::SelectWorkspace ws = sba::carve_select_workspace(workspace, BH, nB, D, NSUB);
    const long long pgroups = (long long)BH * nP;
    const int gpc = 256 / (D / 8);  // pooled rows per CTA
    const unsigned pool_grid = (unsigned)((pgroups + gpc - 1) / gpc);
    const long long rows = (long long)BH * nB;
    const int wpb = 8;              // top-k: one warp per routing row
    const size_t tsmem = sba::topk_smem(wpb, ws.ld);
    if (tsmem > 227 * 1024) return SBA_ERR_UNSUPPORTED;
    const unsigned tgrid = (unsigned)((rows + wpb - 1) / wpb);
    const auto* qb = static_cast<const __nv_bfloat16*>(q);
    const auto* kb = static_cast<const __nv_bfloat16*>(k);
    const bool need_scores = sparsity > 0.0;
    CUtensorMap tqh, tql, tkh, tkl, tks;
    const int sample_stride = nB / 128 > 1 ? nB / 128 : 1;  // the fused screen's range sample
    if (NSUB == 1 && BH > 65535) return SBA_ERR_UNSUPPORTED;  // grid.y of the fused screen
    if ((need_scores || NSUB == 1) &&
        (!make_map(&tqh, ws.qhi, (int)BH, nP, D, 128) || !make_map(&tql, ws.qlo, (int)BH, nP, D, 128) ||
         !make_map(&tkh, ws.khi, (int)BH, nP, D, 128) || !make_map(&tkl, ws.klo, (int)BH, nP, D, 128) ||
         (NSUB == 1 && !make_map_sample(&tks, ws.khi, (int)BH, nB, D, sample_stride))))
        return SBA_ERR_CUDA;
    if (qmean && kmean) {
        ws.qmean64 = const_cast<double*>(qmean);
        ws.kmean64 = const_cast<double*>(kmean);
        sba::split_means_kernel<D><<<pool_grid, 256, 0, s>>>(qmean, ws.qhi, ws.qlo, ws.qnorm, pgroups);
        sba::split_means_kernel<D><<<pool_grid, 256, 0, s>>>(kmean, ws.khi, ws.klo, ws.knorm, pgroups);
    } else {
        // Q and K in one launch: the CTAs past pool_grid pool K
        const sba::PoolSecond kside{kb, ws.kmean64, ws.khi, ws.klo, ws.knorm, pool_grid};
        sba::pool_kernel<D, BLK><<<2 * pool_grid, 256, 0, s>>>(qb, valid_len, H, Npad, ws.qmean64, ws.qhi, ws.qlo,
                                                               ws.qnorm, pgroups, kside);
    }
    sba::kmax_kernel<<<(unsigned)((BH + 7) / 8), 256, 0, s>>>(ws, valid_len, H, Npad, (int)BH, BLK);
    if (NSUB == 1) {
        // screen and top-k in one kernel; the rows it hands back finish in topk_rest_kernel
        using SM = sba::FusedSmem<D>;
        if (cudaFuncSetAttribute(sba::select_fused_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SM::kAlloc) != cudaSuccess ||
            cudaFuncSetAttribute(sba::topk_rest_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)tsmem) != cudaSuccess)
            return SBA_ERR_CUDA;
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
            return SBA_ERR_CUDA;
        const dim3 fgrid((unsigned)((nB + 127) / 128), (unsigned)BH);
        sba::select_fused_kernel<D><<<fgrid, sba::kFusedThreads, SM::kAlloc, s>>>(
            tqh, tql, tkh, tkl, tks, ws, valid_len, H, Npad, sample_stride, sparsity, budget, kmax, kv_idx, kv_cnt,
            g_wait_limit);
        using FS = sba::FinishSmem<D>;
        if (cudaFuncSetAttribute(sba::select_finish_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FS::kTotal) != cudaSuccess)
            return SBA_ERR_CUDA;
        sba::select_finish_kernel<D><<<(unsigned)((rows + sba::kFinishWarps - 1) / sba::kFinishWarps),
                                       32 * sba::kFinishWarps, FS::kTotal, s>>>(ws, valid_len, H, Npad, sparsity,
                                                                               budget, kmax, kv_idx, kv_cnt, rows);
        sba::topk_rest_kernel<D><<<(unsigned)(2 * sms), 32 * wpb, tsmem, s>>>(ws, valid_len, H, Npad, sparsity,
                                                                              budget, kmax, kv_idx, kv_cnt);
        return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
    } else if (need_scores) {
        // persistent: one CTA per SM over the (b, h, query tile) items
        using SM = sba::LseSmem<D>;
        if (cudaFuncSetAttribute(sba::score_lse_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SM::kAlloc) != cudaSuccess)
            return SBA_ERR_CUDA;
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
            return SBA_ERR_CUDA;
        const long long items = (long long)BH * ((nP + 127) / 128);
        const unsigned grid = (unsigned)(items < sms ? items : sms);
        sba::score_lse_kernel<D><<<grid, 320, SM::kAlloc, s>>>(tqh, tql, tkh, tkl, ws.scores, nB, ws.ld, valid_len,
                                                               H, Npad, (int)BH, g_wait_limit);
    }
    if (cudaFuncSetAttribute(sba::topk_kernel<D, NSUB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tsmem) !=
        cudaSuccess)
        return SBA_ERR_CUDA;
    sba::topk_kernel<D, NSUB><<<tgrid, 32 * wpb, tsmem, s>>>(ws, valid_len, H, Npad, sparsity, budget, kmax, kv_idx,
                                                             kv_cnt, rows);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

}  // namespace

extern "C" {

int32_t sba_keep_count(int32_t n_blocks, double sparsity) {
    return sba::keep_count(n_blocks, sparsity);
}

int32_t sba_keep_count_budget(int32_t n_blocks, double sparsity, int32_t budget) {
    if (budget < 1) return 0;
    return sba::keep_count_budget(n_blocks, sparsity, budget);
}

size_t sba_pool_select_workspace_size(int B, int H, int Npad, int D, int block) {
    if (check_shape(B, H, Npad, D, block) != SBA_OK) return 0;
    return sba::select_workspace_bytes((size_t)B * H, (size_t)Npad / block, (size_t)D);
}

sba_status sba_pool_select(const void* q, const void* k, int B, int H, int Npad, int D,
                           const int32_t* valid_len, int block, double sparsity, int kmax,
                           int32_t* kv_idx, int32_t* kv_cnt, void* workspace,
                           size_t workspace_bytes, void* stream) {
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (!q || !k || !kv_idx || !kv_cnt || !workspace) return SBA_ERR_INVALID_ARG;
    if (!(sparsity >= 0.0 && sparsity < 1.0)) return SBA_ERR_INVALID_ARG;
    const int nB = Npad / block;
    if (kmax < sba::keep_count(nB, sparsity)) return SBA_ERR_INVALID_ARG;
    if (workspace_bytes < sba::select_workspace_bytes((size_t)B * H, nB, D)) return SBA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(workspace) || !aligned16(valid_len))
        return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D == 128)
        return run_select<128, 1>(q, k, B, H, Npad, valid_len, sparsity, 1, kmax, kv_idx, kv_cnt, workspace, s);
    return run_select<64, 1>(q, k, B, H, Npad, valid_len, sparsity, 1, kmax, kv_idx, kv_cnt, workspace, s);
}

sba_status sba_pool_select_means(const double* qmean, const double* kmean, int B, int H, int Npad, int D,
                                 const int32_t* valid_len, int block, double sparsity, int kmax,
                                 int32_t* kv_idx, int32_t* kv_cnt, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (!qmean || !kmean || !kv_idx || !kv_cnt || !workspace) return SBA_ERR_INVALID_ARG;
    if (!(sparsity >= 0.0 && sparsity < 1.0)) return SBA_ERR_INVALID_ARG;
    const int nB = Npad / block;
    if (kmax < sba::keep_count(nB, sparsity)) return SBA_ERR_INVALID_ARG;
    if (workspace_bytes < sba::select_workspace_bytes((size_t)B * H, nB, D)) return SBA_ERR_INVALID_ARG;
    if (!aligned16(qmean) || !aligned16(kmean) || !aligned16(workspace) || !aligned16(valid_len))
        return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D == 128)
        return run_select<128, 1>(nullptr, nullptr, B, H, Npad, valid_len, sparsity, 1, kmax, kv_idx, kv_cnt,
                                  workspace, s, qmean, kmean);
    return run_select<64, 1>(nullptr, nullptr, B, H, Npad, valid_len, sparsity, 1, kmax, kv_idx, kv_cnt, workspace,
                             s, qmean, kmean);
}

sba_status sba_qk_norm_rope_pool(const void* x, const void* weight, const int32_t* pos, int B, int H, int Npad,
                                 int D, const int32_t* valid_len, int block, int rope_dim, double rope_base,
                                 float eps, void* out, double* means, void* stream) {
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (!x || !weight || !pos || !out) return SBA_ERR_INVALID_ARG;
    if (rope_dim < 0 || rope_dim > D || rope_dim % 6 != 0 || rope_dim / 6 > sba::kMaxRopePairs)
        return SBA_ERR_INVALID_ARG;
    if (!(rope_base > 0.0) || !std::isfinite(rope_base) || !(eps >= 0.f) || !std::isfinite(eps))
        return SBA_ERR_INVALID_ARG;
    if ((long long)B * H * (Npad / block) > 0x7fffffffll) return SBA_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(out) || !aligned16(weight) || !aligned16(means) || !aligned16(valid_len) ||
        (reinterpret_cast<uintptr_t>(pos) & 3u))
        return SBA_ERR_ALIGNMENT;
    sba::RopeFreqs f;
    const int da = rope_dim / 3;
    for (int i = 0; i < sba::kMaxRopePairs; ++i)
        f.inv_freq[i] = (da > 0 && 2 * i < da) ? (float)std::pow(rope_base, -2.0 * i / da) : 0.f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)((long long)B * H * (Npad / block));
    const auto* xb = static_cast<const __nv_bfloat16*>(x);
    const auto* wb = static_cast<const __nv_bfloat16*>(weight);
    auto* ob = static_cast<__nv_bfloat16*>(out);
    if (D == 128)
        sba::qk_norm_rope_pool_kernel<128><<<grid, 256, 0, s>>>(xb, wb, pos, valid_len, H, Npad, rope_dim, f, eps, ob,
                                                                means);
    else
        sba::qk_norm_rope_pool_kernel<64><<<grid, 256, 0, s>>>(xb, wb, pos, valid_len, H, Npad, rope_dim, f, eps, ob,
                                                               means);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

size_t sba_pool_select_lse_workspace_size(int B, int H, int Npad, int D, int block, int nsub) {
    if (check_shape(B, H, Npad, D, block) != SBA_OK || nsub != sba::kNsub) return 0;
    return sba::select_workspace_bytes((size_t)B * H, (size_t)Npad / block, (size_t)D, (size_t)nsub);
}

sba_status sba_pool_select_lse(const void* q, const void* k, int B, int H, int Npad, int D,
                               const int32_t* valid_len, int block, int nsub, double sparsity, int budget,
                               int kmax, int32_t* kv_idx, int32_t* kv_cnt, void* workspace,
                               size_t workspace_bytes, void* stream) {
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (nsub != sba::kNsub) return SBA_ERR_UNSUPPORTED;
    if (!q || !k || !kv_idx || !kv_cnt || !workspace) return SBA_ERR_INVALID_ARG;
    if (!(sparsity >= 0.0 && sparsity < 1.0) || budget < 1) return SBA_ERR_INVALID_ARG;
    const int nB = Npad / block;
    if (kmax < sba::keep_count_budget(nB, sparsity, budget)) return SBA_ERR_INVALID_ARG;
    if (workspace_bytes < sba::select_workspace_bytes((size_t)B * H, nB, D, nsub)) return SBA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(workspace) || !aligned16(valid_len))
        return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D == 128)
        return run_select<128, sba::kNsub>(q, k, B, H, Npad, valid_len, sparsity, budget, kmax, kv_idx, kv_cnt,
                                           workspace, s);
    return run_select<64, sba::kNsub>(q, k, B, H, Npad, valid_len, sparsity, budget, kmax, kv_idx, kv_cnt,
                                      workspace, s);
}

sba_status sba_block_means(const void* x, int B, int H, int Npad, int D, const int32_t* valid_len,
                           int block, double* out, void* stream) {
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (!x || !out) return SBA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(out) || !aligned16(valid_len)) return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long groups = (long long)B * H * (Npad / block);
    const int gpc = 256 / (D / 8);
    const unsigned grid = (unsigned)((groups + gpc - 1) / gpc);
    if (D == 128)
        sba::pool_kernel<128><<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), valid_len, H,
                                                   Npad, out, nullptr, nullptr, nullptr, groups,
                                                   sba::PoolSecond{nullptr, nullptr, nullptr, nullptr, nullptr, grid});
    else
        sba::pool_kernel<64><<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), valid_len, H,
                                                  Npad, out, nullptr, nullptr, nullptr, groups,
                                                   sba::PoolSecond{nullptr, nullptr, nullptr, nullptr, nullptr, grid});
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

static sba_status attention_common(const void* q, const void* k, const void* v, void* o, float* lse,
                                   int B, int H, int Npad, int D, const int32_t* valid_len,
                                   int block, const int32_t* kv_idx, const int32_t* kv_cnt,
                                   int kmax, int dense, const int32_t* pair_order,
                                   float softmax_scale, void* stream, void* comp_ws = nullptr,
                                   size_t comp_ws_bytes = 0, const ShardOut* shards = nullptr,
                                   bool first_order = false) {
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (!q || !k || !v || !o) return SBA_ERR_INVALID_ARG;
    if (!dense && (!kv_idx || !kv_cnt || kmax <= 0)) return SBA_ERR_INVALID_ARG;
    if (!std::isfinite(softmax_scale)) return SBA_ERR_INVALID_ARG;
    if ((long long)B * H * Npad > (1ll << 31)) return SBA_ERR_UNSUPPORTED;  // 3-D TMA row index
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(valid_len) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) ||
        (kv_idx && (reinterpret_cast<uintptr_t>(kv_idx) & 3u)) ||
        (kv_cnt && (reinterpret_cast<uintptr_t>(kv_cnt) & 3u)) ||
        (pair_order && (reinterpret_cast<uintptr_t>(pair_order) & 3u)))
        return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (comp_ws) {
        // compensated: the bf16 block means of K and V, then the attention with the
        // mean steps after the kept blocks
        if (dense) return SBA_ERR_INVALID_ARG;
        if (!aligned16(comp_ws)) return SBA_ERR_ALIGNMENT;
        const int nBpad = (Npad / 64 + 63) / 64 * 64;
        const size_t half = align_up_256((size_t)B * H * nBpad * D * 2);
        if (comp_ws_bytes < 2 * half) return SBA_ERR_INVALID_ARG;
        char* kbar = static_cast<char*>(comp_ws);
        char* vbar = kbar + half;
        const long long groups = (long long)B * H * nBpad;
        const int gpc = 256 / (D / 8);
        const unsigned mgrid = (unsigned)((groups + gpc - 1) / gpc);
        if (D == 128) {
            sba::block_mean_bf16_kernel<128><<<mgrid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(k), valid_len, H,
                                                                    Npad, nBpad, reinterpret_cast<__nv_bfloat16*>(kbar),
                                                                    groups);
            sba::block_mean_bf16_kernel<128><<<mgrid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(v), valid_len, H,
                                                                    Npad, nBpad, reinterpret_cast<__nv_bfloat16*>(vbar),
                                                                    groups);
            return launch_attention<128, 2, sba::kMeanComp>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt,
                                                            kmax, 0, pair_order, softmax_scale, s, kbar, vbar, nBpad);
        }
        sba::block_mean_bf16_kernel<64><<<mgrid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(k), valid_len, H, Npad,
                                                               nBpad, reinterpret_cast<__nv_bfloat16*>(kbar), groups);
        sba::block_mean_bf16_kernel<64><<<mgrid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(v), valid_len, H, Npad,
                                                               nBpad, reinterpret_cast<__nv_bfloat16*>(vbar), groups);
        return launch_attention<64, 4, sba::kMeanComp>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax,
                                                       0, pair_order, softmax_scale, s, kbar, vbar, nBpad);
    }
    if (first_order) {
        if (dense) return SBA_ERR_INVALID_ARG;
        if (D == 128)
            return launch_attention<128, 2, sba::kFirstOrder>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt,
                                                              kmax, 0, pair_order, softmax_scale, s);
        return launch_attention<64, 4, sba::kFirstOrder>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax,
                                                         0, pair_order, softmax_scale, s);
    }
    if (shards) {
        if (D == 128)
            return launch_attention<128, 2>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax, dense,
                                            pair_order, softmax_scale, s, nullptr, nullptr, 0, shards);
        return launch_attention<64, 4>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax, dense,
                                       pair_order, softmax_scale, s, nullptr, nullptr, 0, shards);
    }
    // the CTA-pair kernel only when chosen: on B200 it is slower than the query pairs on
    // every workload measured, dense included
    if (D == 128 && g_attn_kernel == SBA_ATTN_KERNEL_CTA_PAIR)
        return launch_attention_pair<4>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax, dense,
                                        softmax_scale, s);
    if (D == 128)
        return launch_attention<128, 2>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax,
                                        dense, pair_order, softmax_scale, s);
    return launch_attention<64, 4>(q, k, v, o, lse, B, H, Npad, valid_len, kv_idx, kv_cnt, kmax, dense,
                                   pair_order, softmax_scale, s);
}

sba_status sba_attention(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int Npad, int D, const int32_t* valid_len, int block,
                         const int32_t* kv_idx, const int32_t* kv_cnt, int kmax,
                         float softmax_scale, void* stream) {
    return attention_common(q, k, v, o, lse, B, H, Npad, D, valid_len, block, kv_idx, kv_cnt, kmax,
                            0, nullptr, softmax_scale, stream);
}

sba_status sba_attention_paired(const void* q, const void* k, const void* v, void* o, float* lse,
                                int B, int H, int Npad, int D, const int32_t* valid_len, int block,
                                const int32_t* kv_idx, const int32_t* kv_cnt, int kmax,
                                const int32_t* pair_order, float softmax_scale, void* stream) {
    if (!pair_order) return SBA_ERR_INVALID_ARG;
    return attention_common(q, k, v, o, lse, B, H, Npad, D, valid_len, block, kv_idx, kv_cnt, kmax,
                            0, pair_order, softmax_scale, stream);
}

sba_status sba_dense_attention(const void* q, const void* k, const void* v, void* o, float* lse,
                               int B, int H, int Npad, int D, const int32_t* valid_len,
                               float softmax_scale, void* stream) {
    return attention_common(q, k, v, o, lse, B, H, Npad, D, valid_len, 64, nullptr, nullptr, 0, 1,
                            nullptr, softmax_scale, stream);
}

sba_status sba_attention_to_shards(const void* q, const void* k, const void* v, void* const* o_shards,
                                   float* const* lse_shards, int n_shards, int h_total, int h_first, int B,
                                   int H, int Npad, int D, const int32_t* valid_len, int block,
                                   const int32_t* kv_idx, const int32_t* kv_cnt, int kmax,
                                   const int32_t* pair_order, float softmax_scale, void* stream) {
    if (!o_shards || n_shards < 1 || n_shards > sba::kMaxShards) return SBA_ERR_INVALID_ARG;
    if (Npad <= 0 || Npad % n_shards != 0 || h_first < 0 || H < 1 || h_total < h_first + H)
        return SBA_ERR_INVALID_ARG;
    for (int i = 0; i < n_shards; ++i) {
        if (!o_shards[i] || (lse_shards && !lse_shards[i])) return SBA_ERR_INVALID_ARG;
        if (!aligned16(o_shards[i]) || (lse_shards && (reinterpret_cast<uintptr_t>(lse_shards[i]) & 3u)))
            return SBA_ERR_ALIGNMENT;
    }
    if ((long long)B * h_total * (Npad / n_shards) > (1ll << 31)) return SBA_ERR_UNSUPPORTED;
    const ShardOut sh{n_shards, h_total, h_first, o_shards, lse_shards};
    // o is not written; any 16-byte aligned pointer passes the common checks
    return attention_common(q, k, v, o_shards[0], nullptr, B, H, Npad, D, valid_len, block, kv_idx, kv_cnt, kmax, 0,
                            pair_order, softmax_scale, stream, nullptr, 0, &sh);
}

size_t sba_mean_compensation_workspace_size(int B, int H, int Npad, int D, int block) {
    if (check_shape(B, H, Npad, D, block) != SBA_OK) return 0;
    const int nBpad = (Npad / 64 + 63) / 64 * 64;
    return 2 * align_up_256((size_t)B * H * nBpad * D * 2);
}

sba_status sba_attention_mean_compensated(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                                          int H, int Npad, int D, const int32_t* valid_len, int block,
                                          const int32_t* kv_idx, const int32_t* kv_cnt, int kmax,
                                          const int32_t* pair_order, float softmax_scale, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    if (!workspace) return SBA_ERR_INVALID_ARG;
    return attention_common(q, k, v, o, lse, B, H, Npad, D, valid_len, block, kv_idx, kv_cnt, kmax, 0,
                            pair_order, softmax_scale, stream, workspace, workspace_bytes);
}

sba_status sba_attention_compensated(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                                     int H, int Npad, int D, const int32_t* valid_len, int block,
                                     const int32_t* kv_idx, const int32_t* kv_cnt, int kmax,
                                     const int32_t* pair_order, float softmax_scale, void* stream) {
    return attention_common(q, k, v, o, lse, B, H, Npad, D, valid_len, block, kv_idx, kv_cnt, kmax, 0,
                            pair_order, softmax_scale, stream, nullptr, 0, nullptr, true);
}

sba_status sba_get_device_status(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SBA_ERR_CUDA;
    int word = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&word, sba::g_device_error, sizeof(int)) != cudaSuccess) return SBA_ERR_CUDA;
    if (cudaMemcpyToSymbol(sba::g_device_error, &zero, sizeof(int)) != cudaSuccess) return SBA_ERR_CUDA;
    if (word == sba::kErrTimeout) return SBA_ERR_TIMEOUT;
    if (word != 0) return SBA_ERR_DEVICE_FLAG;
    return SBA_OK;
}

void sba_set_wait_limit(uint64_t cycles) { g_wait_limit = cycles ? cycles : kDefaultWaitLimit; }

sba_status sba_set_attention_kernel(int which) {
    if (which != SBA_ATTN_KERNEL_AUTO && which != SBA_ATTN_KERNEL_QUERY_PAIRS && which != SBA_ATTN_KERNEL_CTA_PAIR)
        return SBA_ERR_INVALID_ARG;
    g_attn_kernel = which;
    return SBA_OK;
}

const char* sba_strerror(sba_status status) {
    switch (status) {
        case SBA_OK: return "ok";
        case SBA_ERR_INVALID_ARG: return "invalid argument";
        case SBA_ERR_UNSUPPORTED: return "unsupported shape or parameter";
        case SBA_ERR_ALIGNMENT: return "misaligned device pointer";
        case SBA_ERR_CUDA: return "CUDA call failed";
        case SBA_ERR_TIMEOUT: return "a kernel wait gave up";
        case SBA_ERR_DEVICE_FLAG: return "a kernel found an invalid routing entry or index";
        case SBA_ERR_SCRATCH_TOO_SMALL: return "problem needs more scratch than the fixed no-allocation buffer holds";
    }
    return "unknown status";
}

}  // extern "C"

// ---------------------------------------------------------------- token pruning
extern "C" int32_t sba_keep_token_count(int32_t n_tokens, double keep_ratio) {
    if (!(keep_ratio >= 0.0 && keep_ratio <= 1.0)) return 0;
    return sba::keep_tokens(n_tokens, keep_ratio);
}

extern "C" size_t sba_token_prune_workspace_size(int B, int N) {
    if (B <= 0 || N <= 0 || (long long)B * N > 0x7fffffffll) return 0;
    return align_up_256((size_t)B * N * sizeof(double));
}

extern "C" sba_status sba_token_prune_select(const void* x, int B, int N, int C, const int32_t* valid_len,
                                             double keep_ratio, int Npad_out, int32_t* idx, int32_t* valid_len_out,
                                             void* workspace, size_t workspace_bytes, void* stream) {
    if (B <= 0 || N <= 0 || C <= 0 || Npad_out <= 0) return SBA_ERR_INVALID_ARG;
    if ((long long)B * N > 0x7fffffffll || B > 65535 || C > (1 << 20)) return SBA_ERR_UNSUPPORTED;
    if (C % 8 != 0) return SBA_ERR_UNSUPPORTED;
    if (!x || !idx || !valid_len_out || !workspace) return SBA_ERR_INVALID_ARG;
    if (!(keep_ratio >= 0.0 && keep_ratio <= 1.0)) return SBA_ERR_INVALID_ARG;
    if (Npad_out < sba::keep_tokens(N, keep_ratio)) return SBA_ERR_INVALID_ARG;
    if (workspace_bytes < (size_t)B * N * sizeof(double)) return SBA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(workspace) || !aligned16(valid_len) ||
        (reinterpret_cast<uintptr_t>(idx) & 3u) || (reinterpret_cast<uintptr_t>(valid_len_out) & 3u))
        return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap tx;
    const long long rows = (long long)B * N;
    if (!make_map_2d(&tx, x, rows, C, sba::kNormRows)) return SBA_ERR_CUDA;
    if (cudaFuncSetAttribute(sba::token_norm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sba::kNormSmem) !=
        cudaSuccess)
        return SBA_ERR_CUDA;
    double* norm2 = static_cast<double*>(workspace);
    const unsigned grid = (unsigned)((rows + sba::kNormRows - 1) / sba::kNormRows);
    sba::token_norm_kernel<<<grid, 160, sba::kNormSmem, s>>>(tx, valid_len, N, C, rows, norm2, g_wait_limit);
    sba::prune_select_kernel<<<(unsigned)B, 1024, 0, s>>>(norm2, valid_len, N, keep_ratio, Npad_out, idx,
                                                           valid_len_out);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

extern "C" sba_status sba_gather_tokens(const void* src, int B, int H, int N, int row_bytes, const int32_t* idx,
                                        const int32_t* valid_len_out, int Npad_out, void* dst, void* stream) {
    if (B <= 0 || H <= 0 || N <= 0 || Npad_out <= 0 || row_bytes <= 0) return SBA_ERR_INVALID_ARG;
    if (row_bytes % 4 != 0) return SBA_ERR_UNSUPPORTED;
    if ((long long)B * H > 65535 || (long long)Npad_out * (row_bytes / 4) > 0x7fffffffll ||
        (long long)N * (row_bytes / 4) > 0x7fffffffll)
        return SBA_ERR_UNSUPPORTED;
    if (!src || !dst || !idx || !valid_len_out) return SBA_ERR_INVALID_ARG;
    const int unit = row_bytes % 16 == 0 ? 16 : 4;
    const uintptr_t am = (uintptr_t)unit - 1;
    if ((reinterpret_cast<uintptr_t>(src) & am) || (reinterpret_cast<uintptr_t>(dst) & am) ||
        (reinterpret_cast<uintptr_t>(idx) & 3u) || (reinterpret_cast<uintptr_t>(valid_len_out) & 3u))
        return SBA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long units = (long long)Npad_out * (row_bytes / unit);   // per (b, h)
    const dim3 grid((unsigned)((units + 4 * 256 - 1) / (4 * 256)), (unsigned)(B * H));
    const auto* sp = static_cast<const unsigned char*>(src);
    auto* dp = static_cast<unsigned char*>(dst);
    if (unit == 16)
        sba::gather_rows_kernel<16><<<grid, 256, 0, s>>>(sp, dp, idx, valid_len_out, H, N, row_bytes, Npad_out);
    else
        sba::gather_rows_kernel<4><<<grid, 256, 0, s>>>(sp, dp, idx, valid_len_out, H, N, row_bytes, Npad_out);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

// ---------------------------------------------------------------- query-block pairing
extern "C" size_t sba_pair_workspace_size(int B, int H, int Npad, int block) {
    if (check_shape(B, H, Npad, 64, block) != SBA_OK) return 0;
    return sba::pair_workspace_bytes((size_t)B * H, (size_t)Npad / block);
}

extern "C" sba_status sba_pair_query_blocks(const int32_t* kv_idx, const int32_t* kv_cnt, int B, int H,
                                            int Npad, int kmax, const int32_t* valid_len, int block,
                                            int32_t* pair_order, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    sba_status st = check_shape(B, H, Npad, 64, block);
    if (st != SBA_OK) return st;
    if (!kv_idx || !kv_cnt || !pair_order || !workspace || kmax <= 0) return SBA_ERR_INVALID_ARG;
    const int nQ = Npad / block;
    const size_t BH = (size_t)B * H;
    if (workspace_bytes < sba::pair_workspace_bytes(BH, nQ)) return SBA_ERR_INVALID_ARG;
    if (!aligned16(workspace) || !aligned16(valid_len) || (reinterpret_cast<uintptr_t>(kv_idx) & 3u) ||
        (reinterpret_cast<uintptr_t>(kv_cnt) & 3u) || (reinterpret_cast<uintptr_t>(pair_order) & 3u))
        return SBA_ERR_ALIGNMENT;
    const long long rows = (long long)BH * nQ;
    const int tiles_per_bh = (nQ + sba::kPairWarps - 1) / sba::kPairWarps;
    // every grid below is one dimension of at most 2^31 - 1 CTAs
    if ((rows + 7) / 8 > 0x7fffffffLL || (long long)BH * tiles_per_bh > 0x7fffffffLL) return SBA_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    sba::PairWorkspace ws = sba::carve_pair_workspace(workspace, BH, nQ);
    const unsigned wgrid = (unsigned)((rows + 7) / 8);   // 8 warps per 256-thread CTA
    sba::pair_bitmap_kernel<<<wgrid, 256, 8 * ((nQ + 31) / 32) * 4, s>>>(ws, kv_idx, kv_cnt, nQ, kmax, rows);
    const int W = (nQ + 31) / 32;
    const size_t psmem = (size_t)sba::kPairSpan * sba::pair_row_words(W) * 4;  // <= 144 x 132 x 4 = 76 KB
    if (cudaFuncSetAttribute(sba::pair_propose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)psmem) != cudaSuccess)
        return SBA_ERR_CUDA;
    sba::pair_propose_kernel<<<(unsigned)(BH * tiles_per_bh), 32 * sba::kPairWarps, psmem, s>>>(
        ws, kv_cnt, valid_len, H, nQ, tiles_per_bh);
    const size_t msmem = (size_t)2 * nQ * 4;  // <= 2 x 4096 x 4 = 32 KB
    if (cudaFuncSetAttribute(sba::pair_match_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)msmem) != cudaSuccess)
        return SBA_ERR_CUDA;
    sba::pair_match_kernel<<<(unsigned)BH, sba::kPairMatchThreads, msmem, s>>>(ws, valid_len, H, nQ, pair_order);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

// ---------------------------------------------------------------- routing without allocation
// Scratch for sba_pool_select_noalloc: a fixed array in device memory that every
// GPU loading this library holds until the process exits.  In host code its name is
// only a handle; host code resolves its device address with cudaGetSymbolAddress
// and passes that address to sba_pool_select as the workspace.
namespace {
constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;  // 16 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 64;
void* g_noalloc_ptr[kMaxDevices] = {};
std::mutex g_noalloc_mutex;

// Device address of the scratch array on the current device, resolved once per device
// (on the first call there, under the lock).
sba_status noalloc_scratch(void** out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SBA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    if (!g_noalloc_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return SBA_ERR_CUDA;
        g_noalloc_ptr[dev] = p;
    }
    *out = g_noalloc_ptr[dev];
    return SBA_OK;
}
}  // namespace

extern "C" size_t sba_noalloc_scratch_bytes(void) { return kNoAllocScratchBytes; }

extern "C" sba_status sba_pool_select_noalloc(const void* q, const void* k, int B, int H, int Npad,
                                              int D, const int32_t* valid_len, int block,
                                              double sparsity, int kmax, int32_t* kv_idx,
                                              int32_t* kv_cnt, void* stream) {
    // the argument checks of sba_pool_select first, so that a bad argument is reported
    // as such whatever the problem size
    sba_status st = check_shape(B, H, Npad, D, block);
    if (st != SBA_OK) return st;
    if (!q || !k || !kv_idx || !kv_cnt) return SBA_ERR_INVALID_ARG;
    if (!(sparsity >= 0.0 && sparsity < 1.0)) return SBA_ERR_INVALID_ARG;
    if (kmax < sba::keep_count(Npad / block, sparsity)) return SBA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(valid_len)) return SBA_ERR_ALIGNMENT;
    const size_t need = sba::select_workspace_bytes((size_t)B * H, (size_t)Npad / block, (size_t)D);
    if (need > kNoAllocScratchBytes) return SBA_ERR_SCRATCH_TOO_SMALL;
    void* scratch = nullptr;
    st = noalloc_scratch(&scratch);
    if (st != SBA_OK) return st;
    return sba_pool_select(q, k, B, H, Npad, D, valid_len, block, sparsity, kmax, kv_idx, kv_cnt,
                           scratch, kNoAllocScratchBytes, stream);
}

// ---------------------------------------------------------------- the block around the attention
namespace {

bool is_dtype(int d) { return d == SBA_DTYPE_BF16 || d == SBA_DTYPE_FP16 || d == SBA_DTYPE_FP32; }
int dtype_bytes(int d) { return d == SBA_DTYPE_FP32 ? 4 : 2; }
bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Whether rows at p + i * stride elements all start on 16 bytes.
bool rows16(const void* p, const int64_t* strides, int n, int width) {
    if (!aligned16(p)) return false;
    for (int i = 0; i < n; ++i)
        if ((strides[i] * width) % 16 != 0) return false;
    return true;
}
bool none_negative(const int64_t* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0) return false;
    return true;
}

// Whether an output may start at an input's address: the rows at the same places (strides of
// sample, token).
bool in_place(const void* in, const int64_t* si, const void* out, const int64_t* so, int B, int N, bool same_type) {
    return in != out || (same_type && (B == 1 || si[0] == so[0]) && (N == 1 || si[1] == so[1]));
}

sba_status dispatch_rows(const sba::RowParams& p, int x_dtype, int dtype, bool vec, cudaStream_t s) {
    if (x_dtype == SBA_DTYPE_BF16) return sba::run_rows<0, 0>(p, vec, s);
    if (x_dtype == SBA_DTYPE_FP16) return sba::run_rows<1, 1>(p, vec, s);
    if (dtype == SBA_DTYPE_BF16) return sba::run_rows<2, 0>(p, vec, s);
    if (dtype == SBA_DTYPE_FP16) return sba::run_rows<2, 1>(p, vec, s);
    return sba::run_rows<2, 2>(p, vec, s);
}

// Row-major [rows][K] 8-bit codes as a 2-D tensor; box = 128 codes x box_rows, 128-byte swizzle.
bool make_map_codes(CUtensorMap* map, const void* base, long long rows, int K, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// How a product runs: the pair kernel with tiles of 256 x bn (splits = 0), or the split
// kernel with tiles of 128 x bn and K in `splits` parts.
struct LinearPlan {
    int bn, splits;
};

// The plan of least estimated time, in microseconds.  The estimates follow what bounds each form:
// K steps of a tile (which are latency and issue up to about 128 columns and tensor work above), the
// epilogue that the next tile's steps hide or do not, the operands' way from L2, W's way from
// HBM; for the split kernel also the staged sums and the CTAs past one per SM, whose start
// costs more in clusters.  Constants fitted to 84 sizes (2 to 512 rows, 320 to 24576
// channels, 512 to 16384 codes) with every plan timed at each: the chosen plan took 1.5%
// longer than the fastest on average, 16% at worst.  Per size, splitting against the pair kernel:
// 2 x 24576 x 4096 codes 15.4 against 33 us, 128 x 320 x 16384 9.1 against 17 us; the
// other way at 128 x 5120 x 512 10.0 against 7.4 us and 512 x 5120 x 4096 22.7 against 14.6 us.
LinearPlan plan_linear(long long M, long long N, long long K, int sms) {
    const double ks = (double)((K + 127) / 128), hbm = (double)N * K / 6.5e6;
    LinearPlan best{256, 0};
    double least = 1e300;
    for (int bn = 64; bn <= 256; bn += 64) {
        const double tiles = (double)((M + 255) / 256) * (double)((N + bn - 1) / bn);
        const double waves = std::ceil(tiles / (sms / 2)), step = 0.021 + 0.0018 * bn, out = 3.0 + 0.0091 * bn;
        const double loop = std::fmax(std::fmax(ks * step + out + (waves - 1) * std::fmax(ks * step, out),
                                                tiles * ks * (256 + bn) * 128 / 14e6 + out), hbm);
        if (1.7 + loop < least) {
            least = 1.7 + loop;
            best = LinearPlan{bn, 0};
        }
    }
    // the split kernel's row tiles are a grid's second dimension; the pair kernel takes more
    if ((M + 127) / 128 > 65535) return best;
    const double box = M < 128 ? (double)((M + 7) / 8 * 8) : 128.0;
    for (int bn = 64; bn <= 128; bn += 64) {
        for (int splits = 1; splits <= 8 && (splits == 1 || ks >= 2 * splits); splits *= 2) {
            const double ctas = (double)((M + 127) / 128) * (double)((N + bn - 1) / bn) * splits, per = ctas / sms;
            const double part = std::ceil(ks / splits);
            const double sums = box * bn * (0.00062 / splits + (splits > 1 ? 0.0001 : 0.0));
            const double more = per > 1 ? (per - 1) * ((splits > 1 ? 3.8 : 0.13) + 0.5 * sums) : 0.0;
            const double loop = std::fmax(std::fmax(part * (0.072 + 0.001 * bn) * std::fmax(1.0, 0.59 * per),
                                                    ctas * part * (bn + box) * 128 / 7.2e6), hbm);
            const double est = 3.7 + (splits > 1 ? 0.95 : 0.0) + sums + more + loop;
            if (est < least) {
                least = est;
                best = LinearPlan{bn, splits};
            }
        }
    }
    return best;
}

// w radians, |w| <= 2^30, in turns, whole ones dropped: the nearest multiple of 2^-64, in 64 bits.  In
// integers: a product in floating point has its 64 digits used up by the whole turns of a large w
// (1e9 radians at position 2^31 were 0.09 radians off).
uint64_t turn_fraction(double w) {
    // 1 / (2 pi) * 2^192, lowest 64 bits first
    constexpr uint64_t inv_two_pi[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(w), &e), 53);  // |w| = m * 2^(e - 53)
    uint64_t product[5] = {};  // m / (2 pi) * 2^192: the turns are product * 2^(e - 245)
    for (int i = 0; i < 3; ++i) {
        const unsigned __int128 t = (unsigned __int128)m * inv_two_pi[i] + product[i];
        product[i] = (uint64_t)t;
        product[i + 1] = (uint64_t)(t >> 64);
    }
    const int drop = 181 - e;  // product's bits below 2^-64 of a turn: 151 at the least, since e <= 30
    if (drop > 255) return 0;
    const int i = drop / 64, b = drop % 64;
    uint64_t f = product[i] >> b | (b ? product[i + 1] << (64 - b) : 0);
    f += product[(drop - 1) / 64] >> ((drop - 1) % 64) & 1;
    return w < 0 ? 0 - f : f;
}

}  // namespace

extern "C" sba_status sba_residual_norm(const void* x, const void* y, void* x_out, void* out, float* out_scale,
                                        int x_dtype, int dtype, int B, int N, int C, const int64_t* strides,
                                        const int32_t* valid_len, int norm, const void* weight, const void* bias,
                                        int post_norm, const void* post_weight, const void* gate, const void* scale,
                                        const void* shift, int param_dtype, int G, const int32_t* index, float eps,
                                        void* stream) {
    if (B <= 0 || N <= 0 || C <= 0) return SBA_ERR_INVALID_ARG;
    if (!is_dtype(x_dtype) || !is_dtype(dtype) || !is_dtype(param_dtype)) return SBA_ERR_INVALID_ARG;
    if (!x || !strides || !none_negative(strides, 8)) return SBA_ERR_INVALID_ARG;
    if (norm < SBA_NORM_NONE || norm > SBA_NORM_RMS || post_norm < SBA_NORM_NONE || post_norm > SBA_NORM_RMS)
        return SBA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return SBA_ERR_INVALID_ARG;
    // what a step without its operand would mean
    if (y ? !x_out : (gate || post_norm || post_weight)) return SBA_ERR_INVALID_ARG;
    if (norm ? !out : (!y || out_scale || weight || bias || scale || shift)) return SBA_ERR_INVALID_ARG;
    if (post_weight && !post_norm) return SBA_ERR_INVALID_ARG;
    const bool modulated = gate || scale || shift;
    if (modulated && (G <= 0 || (!index && G < B))) return SBA_ERR_INVALID_ARG;
    if (C > SBA_MAX_CHANNELS || (long long)B * N > 0x7fffffffll) return SBA_ERR_UNSUPPORTED;
    if (x_dtype != dtype && x_dtype != SBA_DTYPE_FP32) return SBA_ERR_UNSUPPORTED;
    if (param_dtype != SBA_DTYPE_FP32 && param_dtype != dtype) return SBA_ERR_UNSUPPORTED;
    const int xw = dtype_bytes(x_dtype), hw = dtype_bytes(dtype), pw = dtype_bytes(param_dtype);
    if (!aligned_to(x, xw) || !aligned_to(y, hw) || !aligned_to(x_out, xw) || !aligned_to(out, out_scale ? 16 : hw) ||
        !aligned_to(out_scale, 4) || !aligned_to(weight, pw) || !aligned_to(bias, pw) || !aligned_to(post_weight, pw) ||
        !aligned_to(gate, pw) || !aligned_to(scale, pw) || !aligned_to(shift, pw) || !aligned_to(index, 4) ||
        !aligned_to(valid_len, 4))
        return SBA_ERR_ALIGNMENT;
    sba::RowParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x; p.y = y; p.r = x_out; p.h = out; p.h_scale = out_scale;
    p.valid_len = valid_len;
    p.index = modulated ? index : nullptr;
    if (p.index && cudaGetSymbolAddress(reinterpret_cast<void**>(&p.error), sba::g_device_error) != cudaSuccess)
        return SBA_ERR_CUDA;
    p.gate = gate; p.scale = scale; p.shift = shift;
    p.weight = weight; p.bias = bias; p.post_weight = post_weight;
    p.x_sb = strides[0]; p.x_sn = strides[1]; p.y_sb = strides[2]; p.y_sn = strides[3];
    p.r_sb = strides[4]; p.r_sn = strides[5]; p.h_sb = strides[6]; p.h_sn = strides[7];
    p.N = N; p.C = C; p.G = G;
    p.rows = (long long)B * N;
    p.x_end = static_cast<const char*>(x) + ((B - 1) * strides[0] + (N - 1) * strides[1] + C) * xw;
    if (y) p.y_end = static_cast<const char*>(y) + ((B - 1) * strides[2] + (N - 1) * strides[3] + C) * hw;
    p.norm = norm; p.post = post_norm; p.quant = out_scale != nullptr;
    p.Cq = (C + 15) / 16 * 16;
    if (p.quant && (p.h_sb % 16 || p.h_sn % 16)) return SBA_ERR_ALIGNMENT;
    if (y && (x_out == y || !in_place(x, strides, x_out, strides + 4, B, N, true))) return SBA_ERR_INVALID_ARG;
    if (norm && (out == x_out || !in_place(x, strides, out, strides + 6, B, N, !p.quant && x_dtype == dtype) ||
                 !in_place(y, strides + 2, out, strides + 6, B, N, !p.quant)))
        return SBA_ERR_INVALID_ARG;
    p.param32 = param_dtype == SBA_DTYPE_FP32;
    p.eps = eps;
    const bool vec = C % 8 == 0 && rows16(x, strides, 2, xw) && (!y || (rows16(y, strides + 2, 2, hw) &&
                     rows16(x_out, strides + 4, 2, xw))) && (!norm || p.quant || rows16(out, strides + 6, 2, hw)) &&
                     aligned_to(weight, 8 * pw) && aligned_to(bias, 8 * pw) && aligned_to(post_weight, 8 * pw) &&
                     aligned_to(gate, 8 * pw) && aligned_to(scale, 8 * pw) && aligned_to(shift, 8 * pw);
    return dispatch_rows(p, x_dtype, dtype, vec, static_cast<cudaStream_t>(stream));
}

extern "C" sba_status sba_token_quantize(const void* x, int dtype, int B, int H, int N, int D, const int64_t* strides,
                                         int8_t* codes, float* scales, void* stream) {
    if (B <= 0 || H <= 0 || N <= 0 || D <= 0) return SBA_ERR_INVALID_ARG;
    if (!is_dtype(dtype) || !x || !codes || !scales || !strides || !none_negative(strides, 3))
        return SBA_ERR_INVALID_ARG;
    if ((long long)H * D > SBA_MAX_CHANNELS || (long long)B * N > 0x7fffffffll) return SBA_ERR_UNSUPPORTED;
    const int w = dtype_bytes(dtype);
    if (!aligned_to(x, w) || !aligned16(codes) || !aligned_to(scales, 4)) return SBA_ERR_ALIGNMENT;
    if (static_cast<const void*>(codes) == x) return SBA_ERR_INVALID_ARG;
    sba::RowParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x; p.h = codes; p.h_scale = scales;
    p.x_sb = strides[0]; p.x_sh = strides[1]; p.x_sn = strides[2];
    p.x_end = static_cast<const char*>(x) + ((B - 1) * strides[0] + (N - 1) * strides[2] + D) * w;  // of plain rows
    p.D = H > 1 ? D : 0;
    p.N = N; p.C = H * D; p.G = 1;
    p.Cq = (p.C + 15) / 16 * 16;
    p.h_sn = p.Cq;
    p.h_sb = (long long)N * p.Cq;
    p.rows = (long long)B * N;
    p.quant = 1;
    const bool vec = D % 8 == 0 && rows16(x, strides, 3, w);
    return dispatch_rows(p, dtype, dtype, vec, static_cast<cudaStream_t>(stream));
}

extern "C" sba_status sba_int8_linear_plan(long long rows, int channels, int codes, int sms, int* columns, int* splits) {
    if (rows <= 0 || channels <= 0 || codes <= 0 || sms <= 1 || !columns || !splits) return SBA_ERR_INVALID_ARG;
    const LinearPlan plan = plan_linear(rows, channels, codes, sms);
    *columns = plan.bn;
    *splits = plan.splits;
    return SBA_OK;
}

extern "C" sba_status sba_int8_linear(const int8_t* a, const float* a_scale, const int8_t* w, const float* w_scale,
                                      int B, int N, int K, int M, const void* bias, const void* gate, int param_dtype,
                                      int G, const int32_t* index, int activation, const void* residual, void* out,
                                      int out_dtype, int heads, const int64_t* strides, void* stream) {
    if (B <= 0 || N <= 0 || K <= 0 || M <= 0 || heads < 0) return SBA_ERR_INVALID_ARG;
    if (!a || !a_scale || !w || !w_scale || !out || !strides || !none_negative(strides, 5)) return SBA_ERR_INVALID_ARG;
    if (!is_dtype(out_dtype) || !is_dtype(param_dtype)) return SBA_ERR_INVALID_ARG;
    if (activation < SBA_ACT_NONE || activation > SBA_ACT_SILU) return SBA_ERR_INVALID_ARG;
    if (heads > 0 && M % heads != 0) return SBA_ERR_INVALID_ARG;
    if (gate && (G <= 0 || (!index && G < B))) return SBA_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > SBA_MAX_INT8_K) return SBA_ERR_UNSUPPORTED;
    if (heads > 0 && (M / heads) % 32 != 0) return SBA_ERR_UNSUPPORTED;
    if (param_dtype != SBA_DTYPE_FP32 && param_dtype != out_dtype) return SBA_ERR_UNSUPPORTED;
    if ((long long)B * N > 0x7fffff00ll || M > (1 << 24)) return SBA_ERR_UNSUPPORTED;
    const int ow = dtype_bytes(out_dtype), pw = dtype_bytes(param_dtype);
    if (!aligned16(a) || !aligned16(w) || !aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(bias, pw) ||
        !aligned_to(gate, pw) || !aligned_to(residual, ow) || !aligned_to(out, ow) || !aligned_to(index, 4))
        return SBA_ERR_ALIGNMENT;
    if (out == static_cast<const void*>(a) || out == static_cast<const void*>(w)) return SBA_ERR_INVALID_ARG;
    if (out == residual && (heads > 0 || !in_place(residual, strides, out, strides + 2, B, 1, true) ||
                            (N > 1 && strides[1] != strides[4])))
        return SBA_ERR_INVALID_ARG;
    sba::LinearParams p;
    std::memset(&p, 0, sizeof(p));
    p.a_scale = a_scale; p.w_scale = w_scale; p.bias = bias; p.gate = gate; p.residual = residual;
    p.index = gate ? index : nullptr;
    p.out = out;
    p.res_sb = strides[0]; p.res_sn = strides[1];
    p.out_sb = strides[2]; p.out_sh = strides[3]; p.out_sn = strides[4];
    p.M = B * N; p.N = M; p.K = K;
    p.tokens = N;
    p.G = G;
    p.D = heads > 0 ? M / heads : 0;
    p.act = activation;
    p.out_type = out_dtype;
    p.param_type = param_dtype;
    // column groups of 4 and 8 start on 16 bytes in every row
    p.vec = aligned16(w_scale) && aligned16(bias) && rows16(out, strides + 2, 3, ow) &&
            (!residual || rows16(residual, strides, 2, ow)) && (!gate || (aligned16(gate) && (long long)M * pw % 16 == 0));
    p.wait_limit = g_wait_limit;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return SBA_ERR_CUDA;
    CUtensorMap ta, tw;
    const LinearPlan plan = plan_linear(p.M, p.N, K, sms);
    p.bn = plan.bn;
    const long long tiles_n = (p.N + p.bn - 1ll) / p.bn;
    if (plan.splits == 0) {
        const long long pair_tiles = (p.M + 255ll) / 256 * tiles_n;
        if (pair_tiles > 0x3fffffffll) return SBA_ERR_UNSUPPORTED;
        using SM = sba::PairSmem;
        p.stages = SM::stages(p.bn);
        if (!make_map_codes(&ta, a, p.M, K, 128) || !make_map_codes(&tw, w, M, K, p.bn / 2)) return SBA_ERR_CUDA;
        if (cudaFuncSetAttribute(sba::int8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kAlloc) !=
            cudaSuccess)
            return SBA_ERR_CUDA;
        const int clusters = (int)(pair_tiles < sms / 2 ? pair_tiles : sms / 2);
        sba::int8_pair_kernel<<<2 * clusters, sba::kPairThreads, SM::kAlloc, s>>>(ta, tw, p);
        return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
    }
    using SM = sba::SplitSmem;
    p.box_rows = p.M < 128 ? (p.M + 7) / 8 * 8 : 128;
    const int splits = plan.splits;
    const long long tiles_m = (p.M + 127ll) / 128, ctas = tiles_n * tiles_m * splits;  // tiles_n * splits < 2^22
    // CTAs share an SM's memory, up to three where there are that many
    const int per_sm = ctas > 2 * sms ? 3 : ctas > sms ? 2 : 1;
    p.stages = sba::kMaxStages;
    while (p.stages > 2 && (SM::alloc(p.bn, p.box_rows, p.stages) + 1024) * per_sm > 227 * 1024) --p.stages;
    const int smem = SM::alloc(p.bn, p.box_rows, p.stages);
    if (!make_map_codes(&ta, a, p.M, K, p.box_rows) || !make_map_codes(&tw, w, M, K, p.bn)) return SBA_ERR_CUDA;
    // the same limit for every size: a smaller one could come between another thread's limit and
    // its launch
    if (cudaFuncSetAttribute(sba::int8_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) !=
        cudaSuccess)
        return SBA_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(tiles_n * splits), (unsigned)tiles_m);
    cfg.blockDim = dim3(sba::kSplitThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sba::int8_split_kernel, ta, tw, p, splits) == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

extern "C" sba_status sba_rotary(const void* x, void* out, int dtype, const int32_t* pos, int axes, int B, int H, int N,
                                 int D, const int64_t* strides, int rope_dim, int layout, const double* inv_freq,
                                 const uint8_t* axis, float amplitude, int inverse, void* stream) {
    if (B <= 0 || H <= 0 || N <= 0 || D <= 0 || axes <= 0 || axes > 255) return SBA_ERR_INVALID_ARG;
    if (!is_dtype(dtype) || !x || !out || !pos || !strides || !inv_freq || !axis || !none_negative(strides, 6))
        return SBA_ERR_INVALID_ARG;
    if (layout != SBA_ROPE_INTERLEAVED && layout != SBA_ROPE_HALF) return SBA_ERR_INVALID_ARG;
    if (rope_dim <= 0 || rope_dim > D || rope_dim % 2 != 0 || !std::isfinite(amplitude)) return SBA_ERR_INVALID_ARG;
    if (rope_dim / 2 > sba::kMaxRotaryPairs || B > 65535 || H > 65535 || D > (1 << 20)) return SBA_ERR_UNSUPPORTED;
    for (int i = 0; i < rope_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1e9 || axis[i] >= axes) return SBA_ERR_INVALID_ARG;
    const int w = dtype_bytes(dtype);
    if (!aligned_to(x, w) || !aligned_to(out, w) || !aligned_to(pos, 4)) return SBA_ERR_ALIGNMENT;
    if (!in_place(x, strides, out, strides + 3, B, H, true) || (out == x && N > 1 && strides[2] != strides[5]))
        return SBA_ERR_INVALID_ARG;
    sba::RotaryParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x; p.out = out; p.pos = pos;
    p.x_sb = strides[0]; p.x_sh = strides[1]; p.x_sn = strides[2];
    p.o_sb = strides[3]; p.o_sh = strides[4]; p.o_sn = strides[5];
    p.H = H; p.N = N; p.D = D; p.axes = axes; p.pairs = rope_dim / 2;
    p.half = layout == SBA_ROPE_HALF;
    p.copy = rope_dim < D && out != x;
    p.fp16 = dtype == SBA_DTYPE_FP16;
    p.cos_amp = amplitude;
    p.sin_amp = inverse ? -amplitude : amplitude;
    for (int i = 0; i < p.pairs; ++i) {
        p.axis[i] = axis[i];
        p.turn[i] = turn_fraction(inv_freq[i]);
    }
    const bool vec = D % 16 == 0 && p.pairs % (p.half ? 8 : 4) == 0 && rows16(x, strides, 3, w) && rows16(out, strides + 3, 3, w);
    const long long per_token = vec ? D / 16 : (p.copy ? D - p.pairs : p.pairs);
    const long long gx = ((long long)N * per_token + 255) / 256;
    if (gx > 0x7fffffffll) return SBA_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return SBA_ERR_CUDA;
    // heads a thread takes with one set of sines: eight, fewer when that leaves SMs idle
    int hpc = 8;
    while (hpc > 1 && gx * B * ((H + hpc - 1) / hpc) < 4ll * sms) hpc /= 2;
    p.heads_per_cta = hpc;
    const dim3 grid((unsigned)gx, (unsigned)((H + hpc - 1) / hpc), (unsigned)B);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (vec) {
        if (dtype == SBA_DTYPE_FP32 && p.half) sba::rotary_vec_kernel<true, true><<<grid, 256, 0, s>>>(p);
        else if (dtype == SBA_DTYPE_FP32) sba::rotary_vec_kernel<true, false><<<grid, 256, 0, s>>>(p);
        else if (p.half) sba::rotary_vec_kernel<false, true><<<grid, 256, 0, s>>>(p);
        else sba::rotary_vec_kernel<false, false><<<grid, 256, 0, s>>>(p);
    } else {
        if (dtype == SBA_DTYPE_FP32) sba::rotary_any_kernel<true><<<grid, 256, 0, s>>>(p);
        else sba::rotary_any_kernel<false><<<grid, 256, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}
