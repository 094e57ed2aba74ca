// int8_linear.cuh -- products of 8-bit integer codes with one scale a token and one a
// channel: the projections of a transformer block, with their epilogue.
//
//   acc[m][n] = sum_k a[m][k] w[n][k]                  (exact, 32-bit integers)
//   v = acc * (a_scale[m] * w_scale[n]) + bias[n]
//   v = gelu_tanh(v) or silu(v)                        (optional)
//   out[m][n] = residual[m][n] + gate[g(m)][n] * v     (each optional; one rounding)
//
// tcgen05.mma kind::i8 with S32 accumulators in TMEM; both operands K-major in shared
// memory, 128 codes (one 128-byte swizzled row) per K step, brought by TMA, which fills
// what lies past the last row or code with zeros.
//
//   int8_pair_kernel  large products.  A cluster of two CTAs computes tiles of 256 x 256:
//                     cta_group::2 MMAs of M = 256, each CTA staging its 128 rows of A and
//                     its 128 rows of W, which halves the shared-memory traffic of W and
//                     leaves 64 bytes a clock of the 128.  Persistent: the accumulators of
//                     two tiles alternate in TMEM, so the eight epilogue warps finish one
//                     tile while the MMAs of the next run.
//   int8_split_kernel few rows or few tiles.  One CTA per 128 x 64 tile and K split; the
//                     splits of a tile form a cluster and add their integer sums through
//                     distributed shared memory (exact in any order).  With few rows it
//                     streams W once: HBM-bound.
//
// Every wait is bounded: on expiry the CTA records SBA_ERR_TIMEOUT, unwinds all roles,
// drains its own loads and MMAs and frees its TMEM.
#pragma once
#include <cstdint>
#include <cuda.h>

#include "attention2.cuh"      // mma_pair_commit_local, wait_drain
#include "residual_norm.cuh"   // unpack16, pack16

namespace sba {

enum LinearAct : int { kActNone = 0, kActGeluTanh = 1, kActSilu = 2 };

struct LinearParams {
    const float* a_scale;      // [M]
    const float* w_scale;      // [N]
    const void* bias;          // [N] or NULL
    const void* gate;          // [G][N] or NULL
    const void* residual;      // rows of N, or NULL
    const int32_t* index;      // [M] or NULL: row of the gate table
    void* out;
    long long res_sb, res_sn;  // strides in elements of a sample and a token
    long long out_sb, out_sn, out_sh;
    int M, N, K;               // rows, channels, codes
    int tokens;                // rows of a sample
    int G;
    int D;                     // out in head layout: channel n goes to head n / D; 0 = rows
    int act;
    int out_type, param_type;  // 0 bf16, 1 fp16, 2 fp32
    int vec;                   // rows and parameters allow 16-byte accesses
    int box_rows;              // rows of A loaded per tile (split kernel)
    unsigned long long wait_limit;
};

// ------------------------------------------------------------------- instructions
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_pair_s8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_s8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on an mbarrier of the cluster after reads of TMEM: released to the whole cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ------------------------------------------------------------------- epilogue
// What an output row needs.
struct LinearRow {
    float sa;
    const char* gate;
    const char* res;
    char* out;
};

__device__ __forceinline__ LinearRow linear_row(const LinearParams& p, int m) {
    LinearRow r;
    const int b = m / p.tokens, n = m - b * p.tokens;
    r.sa = p.a_scale[m];
    int g = b;
    if (p.index) {
        g = p.index[m];
        if (g < 0 || g >= p.G) {
            raise_device_error(kErrBadRouting);
            g = 0;
        }
    }
    r.gate = p.gate ? static_cast<const char*>(p.gate) + (long long)g * p.N * (p.param_type == 2 ? 4 : 2) : nullptr;
    const int w = p.out_type == 2 ? 4 : 2;
    r.res = p.residual ? static_cast<const char*>(p.residual) + (b * p.res_sb + n * p.res_sn) * w : nullptr;
    r.out = static_cast<char*>(p.out) + (b * p.out_sb + n * p.out_sn) * w;
    return r;
}

// U values (4 or 8) of type `type` at column n of a row.
template <int U>
__device__ __forceinline__ void linear_load(float (&f)[U], const char* row, int n, int type) {
    if (type == 2) {
#pragma unroll
        for (int i = 0; i < U; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(row + 4ll * (n + i));
            f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
        }
    } else if (U == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(row + 2ll * n);
        unpack16(w.x, type, f[0], f[1]);
        unpack16(w.y, type, f[2], f[3]);
        unpack16(w.z, type, f[U - 4], f[U - 3]);
        unpack16(w.w, type, f[U - 2], f[U - 1]);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 2ll * n);
        unpack16(w.x, type, f[0], f[1]);
        unpack16(w.y, type, f[2], f[3]);
    }
}
template <int U>
__device__ __forceinline__ void linear_store(char* row, long long n, const float (&f)[U], int type) {
    if (type == 2) {
#pragma unroll
        for (int i = 0; i < U; i += 4)
            *reinterpret_cast<float4*>(row + 4 * (n + i)) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else if (U == 8) {
        *reinterpret_cast<uint4*>(row + 2 * n) = make_uint4(pack16(f[0], f[1], type), pack16(f[2], f[3], type),
                                                            pack16(f[U - 4], f[U - 3], type),
                                                            pack16(f[U - 2], f[U - 1], type));
    } else {
        *reinterpret_cast<uint2*>(row + 2 * n) = make_uint2(pack16(f[0], f[1], type), pack16(f[2], f[3], type));
    }
}
__device__ __forceinline__ float linear_load1(const void* base, long long i, int type) {
    if (type == 2) return static_cast<const float*>(base)[i];
    float a, z;
    unpack16(static_cast<const uint16_t*>(base)[i], type, a, z);
    return a;
}

__device__ __forceinline__ float linear_act(float v, int act) {
    if (act == kActNone) return v;
    // v * sigmoid(t): silu takes t = v, the tanh form of GELU t = 2 sqrt(2/pi) (v + 0.044715 v^3)
    const float t = act == kActSilu ? v : v * fmaf(0.07135481282052155f, v * v, 1.5957691216057308f);
    return __fdividef(v, 1.f + __expf(-fmaxf(t, -80.f)));
}

// Columns n .. n + U - 1 of a row whose accumulators are `acc`, all of them inside N.
template <int U>
__device__ __forceinline__ void linear_finish(const LinearParams& p, const LinearRow& r, int n, const int* acc) {
    float v[U], t[U];
    linear_load<U>(t, reinterpret_cast<const char*>(p.w_scale), n, 2);
#pragma unroll
    for (int i = 0; i < U; ++i) v[i] = (float)acc[i] * (r.sa * t[i]);
    if (p.bias) {
        linear_load<U>(t, static_cast<const char*>(p.bias), n, p.param_type);
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] += t[i];
    }
    if (p.act) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = linear_act(v[i], p.act);
    }
    if (r.gate) {
        linear_load<U>(t, r.gate, n, p.param_type);
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] *= t[i];
    }
    if (r.res) {
        linear_load<U>(t, r.res, n, p.out_type);
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] += t[i];
    }
    linear_store<U>(r.out, p.D ? (n / p.D) * p.out_sh + n % p.D : (long long)n, v, p.out_type);
}
// One column, any alignment.
__device__ __forceinline__ void linear_finish1(const LinearParams& p, const LinearRow& r, int n, int acc) {
    float v = (float)acc * (r.sa * p.w_scale[n]);
    if (p.bias) v += linear_load1(p.bias, n, p.param_type);
    v = linear_act(v, p.act);
    if (r.gate) v *= linear_load1(r.gate, n, p.param_type);
    if (r.res) v += linear_load1(r.res, n, p.out_type);
    const long long at = p.D ? (n / p.D) * p.out_sh + n % p.D : (long long)n;
    if (p.out_type == 2) reinterpret_cast<float*>(r.out)[at] = v;
    else reinterpret_cast<uint16_t*>(r.out)[at] = (uint16_t)pack16(v, 0.f, p.out_type);
}

// ------------------------------------------------------------------- large products
struct PairSmem {
    static constexpr int kStages = 6;
    static constexpr int kABytes = 128 * 128, kWBytes = 128 * 128;
    static constexpr int kStageBytes = kABytes + kWBytes;
    static constexpr int kBars = kStages * kStageBytes;
    // barriers: full[6], peer[6], empty[6], acc_full[2], acc_empty[2], drain
    static constexpr int kNumBars = 3 * kStages + 5;
    static constexpr int kCtl = kBars + kNumBars * 8;
    static constexpr int kAlloc = kCtl + 16 + 1024;
};
constexpr int kPairThreads = 320;
constexpr int kPairGroup = 8;  // row tiles that walk the columns together

// Tile `i` of the walk: kPairGroup row tiles at a time, all their column tiles, rows fastest,
// so that the clusters at work share both operands in L2.
__device__ __forceinline__ void pair_tile(int i, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int per = kPairGroup * tiles_n;
    const int g = i / per, first = g * kPairGroup;
    const int rows = min(kPairGroup, tiles_m - first);
    const int j = i - g * per;
    tm = first + j % rows;
    tn = j / rows;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ LinearParams p) {
    using SM = PairSmem;
    constexpr int NS = SM::kStages;
    constexpr uint32_t kIdesc = idesc_s8_s32(256, 256);
    constexpr uint32_t kTmemCols = 512;  // two accumulators of 256 columns
    constexpr uint16_t kBoth = 0x3;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(sm), bars = base + SM::kBars;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_peer = [&](int s) { return bars + 8u * (NS + s); };
    auto bar_empty = [&](int s) { return bars + 8u * (2 * NS + s); };
    auto bar_af = [&](int s) { return bars + 8u * (3 * NS + s); };
    auto bar_ae = [&](int s) { return bars + 8u * (3 * NS + 2 + s); };
    const uint32_t bar_drain = bars + 8u * (3 * NS + 4);
    uint32_t* ctl = reinterpret_cast<uint32_t*>(sm + SM::kCtl);
    volatile uint32_t* abort_flag = ctl + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int tiles_m = (p.M + 255) / 256, tiles_n = (p.N + 255) / 256;
    const int tiles = tiles_m * tiles_n;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int ksteps = (p.K + 127) / 128;
    const uint64_t lim = p.wait_limit;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_peer(s), 1);
            mbar_init(bar_empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_af(s), 1);
            mbar_init(bar_ae(s), 16);  // eight epilogue warps of each CTA
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc_pair(smem_u32(ctl), kTmemCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl[0];
    int issued = 0;  // stages whose loads the producer has issued

    if (warp == 8) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmW);
            bool ok = true;
            for (int i = first; ok && i < tiles; i += step) {
                int tm, tn;
                pair_tile(i, tiles_m, tiles_n, tm, tn);
                const int ra = tm * 256 + rank * 128, rw = tn * 256 + rank * 128;
                for (int k = 0; k < ksteps; ++k) {
                    const int st = issued % NS;
                    if (issued >= NS && !wait_bounded(bar_empty(st), ((issued / NS) - 1) & 1, abort_flag, lim)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(bar_full(st), SM::kStageBytes);
                    tma_load_2d(base + st * SM::kStageBytes, &tmA, bar_full(st), k * 128, ra);
                    tma_load_2d(base + st * SM::kStageBytes + SM::kABytes, &tmW, bar_full(st), k * 128, rw);
                    ++issued;
                }
            }
        }
    } else if (warp == 9) {
        if (leader) {
            // -------------------------------------------------------- MMA issuer (pair)
            if (lane == 0) {
                const uint64_t da = smem_desc_sw128(base, 16, 1024);
                const uint64_t dw = smem_desc_sw128(base + SM::kABytes, 16, 1024);
                constexpr uint64_t kStep = SM::kStageBytes >> 4;
                bool ok = true;
                int it = 0, done = 0;
                for (int i = first; ok && i < tiles; i += step, ++done) {
                    const int buf = done & 1;
                    if (done >= 2 && !poll_bounded(bar_ae(buf), ((done >> 1) - 1) & 1, abort_flag, lim)) break;
                    tc_fence_after();
                    for (int k = 0; k < ksteps; ++k, ++it) {
                        const int st = it % NS;
                        const uint32_t par = (it / NS) & 1;
                        if (!poll_bounded(bar_full(st), par, abort_flag, lim) ||
                            !poll_bounded(bar_peer(st), par, abort_flag, lim)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // 32 codes an instruction
                            mma_pair_s8_ss(tmem + buf * 256, da + st * kStep + 2 * kk, dw + st * kStep + 2 * kk, kIdesc,
                                           (k > 0 || kk > 0) ? 1u : 0u);
                        mma_pair_commit(bar_empty(st), kBoth);
                    }
                    if (ok) mma_pair_commit(bar_af(buf), kBoth);
                }
            }
        } else if (lane == 0) {
            // -------------------------------------------------------- relay (CTA 1)
            // CTA 0's MMAs read this CTA's operands: tell it when each stage has landed.
            int it = 0;
            bool ok = true;
            for (int i = first; ok && i < tiles; i += step) {
                for (int k = 0; k < ksteps; ++k, ++it) {
                    const int st = it % NS;
                    if (!wait_bounded(bar_full(st), (it / NS) & 1, abort_flag, lim)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_remote(mapa_shared(bar_peer(st), 0));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue warps
        const int quad = warp & 3, half = warp >> 2;
        int done = 0;
        for (int i = first; i < tiles; i += step, ++done) {
            const int buf = done & 1;
            int tm, tn;
            pair_tile(i, tiles_m, tiles_n, tm, tn);
            const int m = tm * 256 + rank * 128 + quad * 32 + lane;
            const int n0 = tn * 256 + half * 128;
            LinearRow row;
            if (m < p.M) row = linear_row(p, m);
            if (!warp_wait_bounded(bar_af(buf), (done >> 1) & 1, abort_flag, lim)) break;
            tc_fence_after();
            const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * 256 + half * 128;
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t acc[32];
                __syncwarp();
                tmem_ld32(tl + 32 * ch, acc);
                tmem_wait_ld();
                const int n = n0 + 32 * ch;
                if (m >= p.M || n >= p.N) continue;
                const int* ai = reinterpret_cast<const int*>(acc);
                if (p.vec && n + 32 <= p.N) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) linear_finish<8>(p, row, n + 8 * q, ai + 8 * q);
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        if (n + q < p.N) linear_finish1(p, row, n + q, ai[q]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(bar_ae(buf), 0));
        }
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // this CTA's own copies land, and CTA 0's MMAs finish, before TMEM is freed
        if (warp == 8 && lane == 0) {
            for (int t = issued > NS ? issued - NS : 0; t < issued; ++t) wait_drain(bar_full(t % NS), (t / NS) & 1);
        }
        if (warp == 9 && lane == 0 && leader) {
            mma_pair_commit_local(bar_drain);
            wait_drain(bar_drain, 0);
        }
        __syncthreads();
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------- few rows or tiles
struct SplitSmem {
    static constexpr int kStages = 3, kBN = 64;
    static constexpr int kABytes = 128 * 128, kWBytes = kBN * 128;
    static constexpr int kStageBytes = kABytes + kWBytes;
    static constexpr int kPitch = kBN * 4 + 16;  // bytes a row of the staged sums
    static constexpr int kBars = kStages * kStageBytes;
    static constexpr int kCtl = kBars + (2 * kStages + 2) * 8;
    static constexpr int kAlloc = kCtl + 16 + 1024;
    static_assert(128 * kPitch <= kBars, "the sums are staged over the operand ring");
};
constexpr int kSplitThreads = 192;

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// grid (splits * column tiles, row tiles), cluster (splits, 1, 1).  Warps 0-3 move the sums
// out, warp 4 loads, warp 5 issues the MMAs; all of them share the last step.
__global__ void __launch_bounds__(kSplitThreads) int8_split_kernel(const __grid_constant__ CUtensorMap tmA,
                                                                   const __grid_constant__ CUtensorMap tmW,
                                                                   const __grid_constant__ LinearParams p, int splits) {
    using SM = SplitSmem;
    constexpr int NS = SM::kStages, BN = SM::kBN;
    constexpr uint32_t kIdesc = idesc_s8_s32(128, BN);
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(sm), bars = base + SM::kBars;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_empty = [&](int s) { return bars + 8u * (NS + s); };
    const uint32_t bar_acc = bars + 8u * (2 * NS), bar_drain = bars + 8u * (2 * NS + 1);
    uint32_t* ctl = reinterpret_cast<uint32_t*>(sm + SM::kCtl);
    volatile uint32_t* abort_flag = ctl + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
    const int n0 = (int)(blockIdx.x / splits) * BN, m0 = (int)blockIdx.y * 128;
    const int rows = min(128, p.M - m0);
    const int ksteps = (p.K + 127) / 128;
    const int k0 = (int)((long long)ksteps * rank / splits), k1 = (int)((long long)ksteps * (rank + 1) / splits);
    const uint64_t lim = p.wait_limit;
    const uint32_t bytes = (uint32_t)p.box_rows * 128 + SM::kWBytes;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), 1);
        }
        mbar_init(bar_acc, 1);
        mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 5) tmem_alloc(smem_u32(ctl), BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl[0];
    int issued = 0;
    bool ok = true;

    if (warp == 4) {
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmW);
            for (int k = k0; k < k1; ++k) {
                const int st = issued % NS;
                if (issued >= NS && !wait_bounded(bar_empty(st), ((issued / NS) - 1) & 1, abort_flag, lim)) break;
                // rows of A past box_rows stay as they are: their sums are never read
                mbar_arrive_expect_tx(bar_full(st), bytes);
                tma_load_2d(base + st * SM::kStageBytes + SM::kABytes, &tmW, bar_full(st), k * 128, n0);
                tma_load_2d(base + st * SM::kStageBytes, &tmA, bar_full(st), k * 128, m0);
                ++issued;
            }
        }
    } else if (warp == 5) {
        if (lane == 0) {
            const uint64_t da = smem_desc_sw128(base, 16, 1024);
            const uint64_t dw = smem_desc_sw128(base + SM::kABytes, 16, 1024);
            constexpr uint64_t kStep = SM::kStageBytes >> 4;
            for (int it = 0; it < k1 - k0; ++it) {
                const int st = it % NS;
                if (!poll_bounded(bar_full(st), (it / NS) & 1, abort_flag, lim)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_s8_ss(tmem, da + st * kStep + 2 * kk, dw + st * kStep + 2 * kk, kIdesc,
                              (it > 0 || kk > 0) ? 1u : 0u);
                mma_commit(bar_empty(st));
            }
            if (ok) mma_commit(bar_acc);
        }
    } else if (warp * 32 < rows) {
        ok = warp_wait_bounded(bar_acc, 0, abort_flag, lim);
        tc_fence_after();
        if (ok) {
            // every MMA is done, so the operand ring is free
            unsigned char* dst = sm + (warp * 32 + lane) * SM::kPitch;
            const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll
            for (int ch = 0; ch < BN / 32; ++ch) {
                uint32_t acc[32];
                tmem_ld32(tl + 32 * ch, acc);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4*>(dst + 128 * ch + 16 * q) =
                        make_uint4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 4 && lane == 0) {
            for (int t = issued > NS ? issued - NS : 0; t < issued; ++t) wait_drain(bar_full(t % NS), (t / NS) & 1);
        }
        if (warp == 5 && lane == 0) {
            mma_commit(bar_drain);
            wait_drain(bar_drain, 0);
        }
        __syncthreads();
    }
    if (splits > 1) cluster_sync();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, BN);

    // the splits' sums, four columns a thread, the tile's items dealt over the cluster
    if (!*abort_flag) {
        const int items = rows * (BN / 4);
        for (int i = rank * kSplitThreads + tid; i < items; i += splits * kSplitThreads) {
            const int r = i / (BN / 4), c = 4 * (i % (BN / 4));
            const int n = n0 + c;
            if (n >= p.N) continue;
            const uint32_t at = base + r * SM::kPitch + c * 4;
            int acc[4] = {0, 0, 0, 0};
            for (int s = 0; s < splits; ++s) {
                const int4 v = splits > 1 ? ld_cluster_int4(mapa_shared(at, s))
                                          : *reinterpret_cast<const int4*>(sm + r * SM::kPitch + c * 4);
                acc[0] += v.x;
                acc[1] += v.y;
                acc[2] += v.z;
                acc[3] += v.w;
            }
            const LinearRow row = linear_row(p, m0 + r);
            if (p.vec && n + 4 <= p.N) {
                linear_finish<4>(p, row, n, acc);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (n + q < p.N) linear_finish1(p, row, n + q, acc[q]);
            }
        }
    }
    if (splits > 1) cluster_sync();  // no CTA leaves while its sums may still be read
}

}  // namespace sba
