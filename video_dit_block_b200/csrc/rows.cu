// rows.cu -- launches of the row operators (residual_norm.cuh).  Compiled once for each pair of
// types ROW_X (x and r) and ROW_H (y and h), given on the command line, side by side with
// the rest of the library: all pairs together take minutes.
#include <cuda_runtime.h>

#include "residual_norm.cuh"

#ifndef ROW_X
#define ROW_X 0
#define ROW_H 0
#endif

namespace sba {

template <int XT, int HT, bool WARP, int VPT, bool VEC, int KIND, bool P32 = true>
static sba_status launch_rows(const RowParams& p, int chunks, cudaStream_t s) {
    const auto kernel = residual_norm_kernel<XT, HT, WARP, VPT, VEC, KIND, P32>;
    const int threads = WARP ? 128 : (chunks + 32 * VPT - 1) / (32 * VPT) * 32;
    const long long ctas = WARP ? (p.rows + 3) / 4 : p.rows;
    long long grid = ctas;
    const size_t smem = VEC || !p.quant ? 0 : (size_t)threads * VPT * 8;  // the codes of the CTA's rows
    if (ctas > 128) {
        int dev = 0, sms = 0, resident = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, smem) != cudaSuccess || resident < 1)
            return SBA_ERR_CUDA;
        if (ctas > (long long)sms * resident) grid = (long long)sms * resident;
    }
    kernel<<<(unsigned)grid, threads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

// Which of the kernels with fixed steps a call is.  The rule: the steps of a block whose norms are
// modulated (scale and shift together, no bias), with the gated residual or without a y, and of one
// with a norm after the block (then without modulation); all other combinations take the general
// kernel.  What that leaves them at, 37800 rows of 5120 channels in bf16, as shares of the copy rate
// (20 launches after a pause): with kernels of their own, modulated norm 146 us (0.81), gated residual
// and modulated norm 252 (0.94), with codes 236 (0.88), fp32 stream with post norm, gate, RMS
// norm and weight 390 (0.91); in the general one, ungated residual, RMS norm and weight 253 (0.93),
// with the gate 273 (0.87), RMS norm and weight 170 (0.69), with codes 191 (0.46), layer norm, weight
// and bias 202 (0.59), these and modulation 255 (0.46), post norm and modulation 340 (0.70), fp32 h
// 304 (0.78).
static int row_kind(const RowParams& p) {
    if (!p.norm) return p.y ? kRowAny : p.D ? kRowQuantHeads : kRowQuant;
    const bool modulated = p.scale && p.shift && !p.bias;
    if (!p.y && modulated) return p.quant ? kRowNormQuant : kRowNorm;
    if (p.y && p.gate && !p.post && modulated) return p.quant ? kRowGateNormQuant : kRowGateNorm;
    if (p.y && p.gate && p.post && !p.scale && !p.shift && !p.quant) return kRowPostGateNorm;
    return kRowAny;
}

template <int XT, int HT, bool P32>
static sba_status run_kind(const RowParams& p, int chunks, cudaStream_t s) {
    switch (row_kind(p)) {
        case kRowNorm: return launch_rows<XT, HT, false, 4, true, kRowNorm, P32>(p, chunks, s);
        case kRowNormQuant: return launch_rows<XT, HT, false, 4, true, kRowNormQuant, P32>(p, chunks, s);
        case kRowGateNorm: return launch_rows<XT, HT, false, 4, true, kRowGateNorm, P32>(p, chunks, s);
        case kRowGateNormQuant: return launch_rows<XT, HT, false, 4, true, kRowGateNormQuant, P32>(p, chunks, s);
        case kRowPostGateNorm: return launch_rows<XT, HT, false, 4, true, kRowPostGateNorm, P32>(p, chunks, s);
    }
    return launch_rows<XT, HT, false, 4, true, kRowAny>(p, chunks, s);
}

// The warps of a row and the chunks of each thread.
template <int XT, int HT>
sba_status run_rows(const RowParams& p, bool vec, cudaStream_t s) {
    const int chunks = p.quant ? p.Cq / 8 : (p.C + 7) / 8;
    if (!vec) {
        // the row may start up to 7 channels into its first chunk, and its codes are read back
        // up to 4 bytes past their end.  No more chunks a thread than needed: each one's ends
        // cost (200,000 rows of 250 channels, gated residual and modulated norm: two chunks a
        // thread 296 to 336, four 607 us)
        const int most = chunks + 2;
        if (most <= 32) return launch_rows<XT, HT, true, 1, false, kRowAny>(p, most, s);
        if (most <= 64) return launch_rows<XT, HT, true, 2, false, kRowAny>(p, most, s);
        if (most <= 128) return launch_rows<XT, HT, true, 4, false, kRowAny>(p, most, s);
        if constexpr (XT == HT)
            if (row_kind(p) == kRowQuant && most <= 4096)
                return launch_rows<XT, HT, false, 4, false, kRowQuant>(p, most, s);
        if (most <= 1024) return launch_rows<XT, HT, false, 4, false, kRowAny>(p, most, s);
        return launch_rows<XT, HT, false, 9, false, kRowAny>(p, most, s);
    }
    if (chunks <= 32) return launch_rows<XT, HT, true, 1, true, kRowAny>(p, chunks, s);
    if (chunks <= 128) return launch_rows<XT, HT, true, 4, true, kRowAny>(p, chunks, s);
    if constexpr (XT == HT) {
        if (row_kind(p) == kRowQuant) return launch_rows<XT, HT, false, 4, true, kRowQuant>(p, chunks, s);
        if (row_kind(p) == kRowQuantHeads)
            return launch_rows<XT, HT, false, 4, true, kRowQuantHeads>(p, chunks, s);
    }
    if (chunks > 1024) return launch_rows<XT, HT, false, 8, true, kRowAny>(p, chunks, s);
    if constexpr (HT != kRowFp32) return p.param32 ? run_kind<XT, HT, true>(p, chunks, s) : run_kind<XT, HT, false>(p, chunks, s);
    return launch_rows<XT, HT, false, 4, true, kRowAny>(p, chunks, s);
}

template sba_status run_rows<ROW_X, ROW_H>(const RowParams&, bool, cudaStream_t);

}  // namespace sba
