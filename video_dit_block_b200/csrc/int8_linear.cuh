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
//                     leaves it 64 bytes a clock of the 128.  Persistent: the accumulators of
//                     two tiles alternate in TMEM, so the eight epilogue warps finish one
//                     tile while the MMAs of the next run.  8192 x 5120 x 5120 codes, random ones,
//                     20 launches after a pause: 140 us, 0.94 of twice the measured bf16
//                     rate, with gate and residual 153.  Without a pause the power cap
//                     takes the clock to 1.3 GHz: 160 and 180.
//   int8_split_kernel few rows or few tiles.  One CTA per tile of 128 x bn and K split; the
//                     splits of a tile form a cluster and add their integer sums through
//                     distributed shared memory (exact in any order).  With few rows it
//                     streams W once.  2 rows, 24576 x 4096 codes, weights in turn that
//                     together exceed L2: 20.0 us, W's bytes (101 MB) at 0.77 of the copy
//                     rate; the rest goes, as far as the code shows, to the CTAs' start.
//                     (The same weight again and again is found in L2 in part: 14.7 us.)
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
    int bn;                    // columns of a tile: 64, 128, 192 or 256 (split kernel: 64 or 128)
    int stages;                // K steps in flight
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

// A tiled load whose bytes count on a barrier of either CTA of the pair (given by its
// shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
// The count goes ahead of the loads it announces and carries no data of this thread, so it is
// relaxed: a release at cluster scope made the producer wait for its loads (0.8 us a step
// in place of 0.3).
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t cluster_addr, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr),
                 "r"(bytes)
                 : "memory");
}

// True in one lane of a converged warp, the same one every time.  The MMAs and loads are issued
// behind it, from loops that the whole warp runs: behind `lane == 0` the compiler cannot know that
// one lane is left, and an MMA took 180 cycles to issue whatever its size; behind this it takes
// 80, less than a 128 x 256 x 32 needs (128).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A bounded wait by polling whose outcome is the same, and known to be the same, for the whole
// warp.
__device__ __forceinline__ bool warp_poll_bounded(uint32_t bar, uint32_t parity, volatile uint32_t* abort,
                                                  uint64_t limit) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (true) {
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
        bool stop = *abort != 0;
        if ((uint64_t)(clock64() - t0) > limit) {
            if (!stop) raise_device_error(kErrTimeout);
            *abort = 1u;
            stop = true;
        }
        if (__any_sync(0xffffffffu, stop)) return false;
    }
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

// U parameters (4 or 8) of type `type` at column n of a row.
template <int U>
__device__ __forceinline__ void linear_load(float (&f)[U], const char* row, int n, int type) {
    if (U > 8) {
#pragma unroll
        for (int i = 0; i < U; i += 8) {
            float g[8];
            linear_load<8>(g, row, n + i, type);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[(i + e) % U] = g[e];
        }
    } else if (type == 2) {
#pragma unroll
        for (int i = 0; i < U; i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + 4ll * (n + i)));
            f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
        }
    } else if (U == 8) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + 2ll * n));
        unpack16(w.x, type, f[0], f[1]);
        unpack16(w.y, type, f[2], f[3]);
        unpack16(w.z, type, f[U - 4], f[U - 3]);
        unpack16(w.w, type, f[U - 2], f[U - 1]);
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + 2ll * n));
        unpack16(w.x, type, f[0], f[1]);
        unpack16(w.y, type, f[2], f[3]);
    }
}
// Four values of a row of residuals (which may be the output: plain loads) or outputs.
__device__ __forceinline__ void linear_read4(float (&f)[4], const char* row, int n, int type) {
    if (type == 2) {
        const float4 a = *reinterpret_cast<const float4*>(row + 4ll * n);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 2ll * n);
        unpack16(w.x, type, f[0], f[1]);
        unpack16(w.y, type, f[2], f[3]);
    }
}
__device__ __forceinline__ void linear_write4(char* row, long long n, const float (&f)[4], int type) {
    if (type == 2) *reinterpret_cast<float4*>(row + 4 * n) = make_float4(f[0], f[1], f[2], f[3]);
    else *reinterpret_cast<uint2*>(row + 2 * n) = make_uint2(pack16(f[0], f[1], type), pack16(f[2], f[3], type));
}
__device__ __forceinline__ float linear_load1(const void* base, long long i, int type) {
    if (type == 2) return static_cast<const float*>(base)[i];
    float a, z;
    unpack16(static_cast<const uint16_t*>(base)[i], type, a, z);
    return a;
}

// v * sigmoid(t): silu takes t = v, the tanh form of GELU t = 2 sqrt(2/pi) (v + 0.044715 v^3).
// -t log2(e) is formed directly; an exponential that overflows ends in v * (1 / inf) = 0.
__device__ __forceinline__ float linear_act(float v, int act) {
    if (act == kActNone) return v;
    constexpr float kLog2e = 1.4426950408889634f;
    const float t = act == kActSilu ? -kLog2e * v
                                    : v * fmaf(-0.07135481282052155f * kLog2e, v * v, -1.5957691216057308f * kLog2e);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(t)));
    return v * r;
}

// v of columns n .. n + U - 1 of a row, before the residual; `sw` and `bias` are those
// columns' (bias 0 where there is none).  WIDE: all of them inside N, the gate's rows on 16
// bytes.
template <int U, bool WIDE>
__device__ __forceinline__ void linear_value(float (&v)[U], const LinearParams& p, const LinearRow& r, int n,
                                             const uint32_t* acc, const float* sw, const float* bias) {
#pragma unroll
    for (int i = 0; i < U; i += 4) {
        float4 s = make_float4(sw[0], sw[1], sw[2], sw[3]), b = make_float4(bias[0], bias[1], bias[2], bias[3]);
        if (U > 4) {  // from shared memory, aligned
            s = *reinterpret_cast<const float4*>(sw + i);
            b = *reinterpret_cast<const float4*>(bias + i);
        }
        v[i] = fmaf((float)(int)acc[i], r.sa * s.x, b.x);
        v[i + 1] = fmaf((float)(int)acc[i + 1], r.sa * s.y, b.y);
        v[i + 2] = fmaf((float)(int)acc[i + 2], r.sa * s.z, b.z);
        v[i + 3] = fmaf((float)(int)acc[i + 3], r.sa * s.w, b.w);
    }
    if (p.act) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = linear_act(v[i], p.act);
    }
    if (r.gate) {
        if (WIDE) {
            float t[U];
            linear_load<U>(t, r.gate, n, p.param_type);
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] *= t[i];
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (n + i < p.N) v[i] *= linear_load1(r.gate, n + i, p.param_type);
        }
    }
}
// The offset of column n in its output row.
__device__ __forceinline__ long long linear_col(const LinearParams& p, int n) {
    return p.D ? (n / p.D) * p.out_sh + n % p.D : (long long)n;
}
// One column, any alignment.
__device__ __forceinline__ void linear_finish1(const LinearParams& p, const LinearRow& r, int n, int acc) {
    const float bias = p.bias ? linear_load1(p.bias, n, p.param_type) : 0.f;
    float v = linear_act(fmaf((float)acc, r.sa * p.w_scale[n], bias), p.act);
    if (r.gate) v *= linear_load1(r.gate, n, p.param_type);
    if (r.res) v += linear_load1(r.res, n, p.out_type);
    const long long at = linear_col(p, n);
    if (p.out_type == 2) reinterpret_cast<float*>(r.out)[at] = v;
    else reinterpret_cast<uint16_t*>(r.out)[at] = (uint16_t)pack16(v, 0.f, p.out_type);
}

// ------------------------------------------------------------------- large products
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

constexpr int kMaxStages = 10;
struct PairSmem {
    static constexpr int kABytes = 128 * 128;  // 128 rows of A, then bn / 2 of W, a stage
    static constexpr int kRing = 6 * 32768;    // the operand ring: as many stages as fit
    // barriers: full[10], empty[10], acc_full[2], acc_empty[2], drain
    static constexpr int kBars = kRing;
    static constexpr int kCols = kBars + (2 * kMaxStages + 6) / 2 * 16;  // float [2 tiles][scale, bias][256]
    static constexpr int kOut = kCols + 2 * 2 * 256 * 4;                 // 2 KB an epilogue warp
    static constexpr int kCtl = kOut + 8 * 2048;
    static constexpr int kAlloc = kCtl + 16 + 1024;
    static __host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn / 2 * 128; }
    static __host__ __device__ constexpr int stages(int bn) {
        return kRing / stage_bytes(bn) < kMaxStages ? kRing / stage_bytes(bn) : kMaxStages;
    }
};
static_assert(PairSmem::kAlloc <= 227 * 1024, "one CTA's shared memory");
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

// A lane of an epilogue warp has a row of the accumulator, but 32 lanes storing to 32 rows
// take 32 cycles an access and held the tile back (11,600 cycles a tile; 25,000 with a
// residual).  So the rows pass through 2 KB of shared memory in pieces of 64 bytes a row
// (32 columns of 16 bits, 16 of fp32), and neighbouring lanes move neighbouring columns: 16
// bytes each, four lanes a row, or (rows off the 16-byte grid, or past the last column) one
// column each.  16-byte word j of row r stands at 4 r + (j ^ (r / 2 & 3)): eight lanes touch all
// banks either way.
__device__ __forceinline__ int pair_word(int r, int j) { return 4 * r + (j ^ ((r >> 1) & 3)); }

// The residual of the piece at column n, as this lane moves it in 16-byte accesses.
__device__ __forceinline__ void pair_fetch(uint4 (&res)[4], const LinearParams& p, const long long (&row)[4],
                                           const bool (&live)[4], int n, int lane) {
    const char* base = static_cast<const char*>(p.residual) + 16 * (lane & 3);
    const int w = p.out_type == 2 ? 4 : 2;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (live[r]) res[r] = *reinterpret_cast<const uint4*>(base + (row[r] + n) * w);
}

// The piece at column n column by column: the residual into the stage (LOAD), or the stage to the
// output.  Of 16 bits a lane has a column of every row, of fp32 one of every other row.
template <bool F32, bool LOAD>
__device__ __forceinline__ void pair_columns(const LinearParams& p, int m0, int n, uint4* stage, int lane) {
    const int c = F32 ? lane & 15 : lane;
    const bool in = n + c < p.N;
    const long long col = LOAD ? (long long)(n + c) : linear_col(p, n + c);
    int b = m0 / p.tokens, tk = m0 - b * p.tokens;  // the rows' sample and token
    if (F32 && lane >= 16 && ++tk == p.tokens) tk = 0, ++b;
    constexpr int R = F32 ? 16 : 32;
    char* at = reinterpret_cast<char*>(stage) + c % (F32 ? 4 : 8) * (F32 ? 4 : 2);
    auto place = [&](int i) { return at + 16 * pair_word(F32 ? 2 * i + (lane >> 4) : i, c / (F32 ? 4 : 8)); };
    uint32_t u[R];  // all read before any is written: the compiler cannot tell the two apart
    if (!LOAD) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            u[i] = F32 ? *reinterpret_cast<const uint32_t*>(place(i)) : *reinterpret_cast<const uint16_t*>(place(i));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool live = in && m0 + (F32 ? 2 * i + (lane >> 4) : i) < p.M;
        if (LOAD) {
            u[i] = 0;
            if (live) {
                const long long g = b * p.res_sb + tk * p.res_sn + col;
                u[i] = F32 ? static_cast<const uint32_t*>(p.residual)[g] : static_cast<const uint16_t*>(p.residual)[g];
            }
        } else if (live) {
            const long long g = b * p.out_sb + tk * p.out_sn + col;
            if (F32) static_cast<uint32_t*>(p.out)[g] = u[i];
            else static_cast<uint16_t*>(p.out)[g] = (uint16_t)u[i];
        }
        if (++tk == p.tokens) tk = 0, ++b;
        if (F32 && ++tk == p.tokens) tk = 0, ++b;
    }
    if (LOAD) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (F32) *reinterpret_cast<uint32_t*>(place(i)) = u[i];
            else *reinterpret_cast<uint16_t*>(place(i)) = (uint16_t)u[i];
        }
    }
}

// One piece from the accumulators of the lane's row to the output.  m0: the warp's first row.
template <bool F32, bool WIDE>
__device__ __forceinline__ void pair_piece(const LinearParams& p, const LinearRow& row, int m0, int n,
                                           const uint32_t* acc, const float* s_col, bool any_res, const uint4 (&res)[4],
                                           uint4* stage, const long long (&out_row)[4], const bool (&live)[4], int lane) {
    constexpr int U = F32 ? 16 : 32;
    float v[U];
    linear_value<U, WIDE>(v, p, row, n, acc, s_col, s_col + 256);
    if (any_res) {
        if (WIDE) {
#pragma unroll
            for (int r = 0; r < 4; ++r) stage[pair_word(8 * r + (lane >> 2), lane & 3)] = res[r];
        } else {
            pair_columns<F32, true>(p, m0, n, stage, lane);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 w = stage[pair_word(lane, j)];
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (F32) {
                    v[4 * j + e] += __uint_as_float(u[e]);
                } else {
                    float a, b;
                    unpack16(u[e], p.out_type, a, b);
                    v[U / 4 * j + 2 * e] += a;
                    v[U / 4 * j + 2 * e + 1] += b;
                }
            }
        }
    }
    // each word of the stage is rewritten by the lane that has just read it
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 w;
        if (F32) {
            w = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                           __float_as_uint(v[4 * j + 3]));
        } else {
            const float* f = v + U / 4 * j;
            w = make_uint4(pack16(f[0], f[1], p.out_type), pack16(f[2], f[3], p.out_type),
                           pack16(f[4 % (U / 4)], f[5 % (U / 4)], p.out_type),
                           pack16(f[6 % (U / 4)], f[7 % (U / 4)], p.out_type));
        }
        stage[pair_word(lane, j)] = w;
    }
    __syncwarp();
    if (WIDE) {
        const long long col = linear_col(p, n);
        char* base = static_cast<char*>(p.out) + 16 * (lane & 3);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint4 w = stage[pair_word(8 * r + (lane >> 2), lane & 3)];
            if (live[r]) *reinterpret_cast<uint4*>(base + (out_row[r] + col) * (F32 ? 4 : 2)) = w;
        }
    } else {
        pair_columns<F32, false>(p, m0, n, stage, lane);
    }
    __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ LinearParams p) {
    using SM = PairSmem;
    const int NS = p.stages, kStage = SM::stage_bytes(p.bn);
    const uint32_t idesc = idesc_s8_s32(256, p.bn);
    constexpr uint32_t kTmemCols = 512;  // two accumulators of 256 columns
    constexpr uint16_t kBoth = 0x3;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(sm), bars = base + SM::kBars;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
    auto bar_af = [&](int s) { return bars + 8u * (2 * kMaxStages + s); };
    auto bar_ae = [&](int s) { return bars + 8u * (2 * kMaxStages + 2 + s); };
    const uint32_t bar_drain = bars + 8u * (2 * kMaxStages + 4);
    uint32_t* ctl = reinterpret_cast<uint32_t*>(sm + SM::kCtl);
    volatile uint32_t* abort_flag = ctl + 1;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int tiles_m = (p.M + 255) / 256, tiles_n = (p.N + p.bn - 1) / p.bn;
    const int wr = p.bn / 2;  // rows of W a CTA stages, and columns an epilogue warp finishes
    const int tiles = tiles_m * tiles_n;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int ksteps = (p.K + 127) / 128;
    const uint64_t lim = p.wait_limit;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar_full(s), 2);  // CTA 0's counts both CTAs' loads
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
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl[0], 0);
    int issued = 0;  // stages whose loads the producer has issued

    if (warp == 8) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmW);
        }
        bool ok = true;
        int st = 0;          // stage, and the parity of its next wait
        uint32_t par = 1;
        for (int i = first; ok && i < tiles; i += step) {
            int tm, tn;
            pair_tile(i, tiles_m, tiles_n, tm, tn);
            const int ra = tm * 256 + rank * 128, rw = tn * p.bn + rank * wr;
            for (int k = 0; k < ksteps; ++k) {
                if (issued >= NS && !warp_poll_bounded(bar_empty(st), par, abort_flag, lim)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t full = mapa_shared(bar_full(st), 0);
                    mbar_arrive_expect_tx_cluster(full, SM::kABytes + wr * 128);
                    tma_load_2d_pair(base + st * kStage, &tmA, full, k * 128, ra);
                    tma_load_2d_pair(base + st * kStage + SM::kABytes, &tmW, full, k * 128, rw);
                }
                ++issued;
                if (++st == NS) st = 0, par ^= 1;
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer (pair)
        if (leader) {
            const uint64_t da = smem_desc_sw128(base, 16, 1024);
            const uint64_t dw = smem_desc_sw128(base + SM::kABytes, 16, 1024);
            const uint64_t step16 = (uint64_t)(kStage >> 4);
            bool ok = true;
            int st = 0, done = 0;
            uint32_t par = 0;
            uint64_t sa = da, sw = dw;
            for (int i = first; ok && i < tiles; i += step, ++done) {
                const int buf = done & 1;
                if (done >= 2 && !warp_poll_bounded(bar_ae(buf), ((done >> 1) - 1) & 1, abort_flag, lim)) break;
                tc_fence_after();
                for (int k = 0; k < ksteps; ++k) {
                    if (!warp_poll_bounded(bar_full(st), par, abort_flag, lim)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // 32 codes an instruction
                            mma_pair_s8_ss(tmem + buf * 256, sa + 2 * kk, sw + 2 * kk, idesc,
                                           (k > 0 || kk > 0) ? 1u : 0u);
                        mma_pair_commit(bar_empty(st), kBoth);
                    }
                    __syncwarp();
                    sa += step16, sw += step16;
                    if (++st == NS) st = 0, par ^= 1, sa = da, sw = dw;
                }
                if (ok && elect_one()) mma_pair_commit(bar_af(buf), kBoth);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue warps
        // (the four warps of a half pass the same named barriers whatever happens: a wait that
        // fails is carried to the end of its tile)
        const int quad = warp & 3, half = warp >> 2;
        int done = 0;
        bool failed = false;
        uint4* stage = reinterpret_cast<uint4*>(sm + SM::kOut) + warp * 128;
        for (int i = first; i < tiles; i += step, ++done) {
            const int buf = done & 1;
            int tm, tn;
            pair_tile(i, tiles_m, tiles_n, tm, tn);
            const int m = tm * 256 + rank * 128 + quad * 32 + lane;
            const int n0 = tn * p.bn + half * wr;
            const LinearRow row = linear_row(p, m < p.M ? m : p.M - 1);
            // while the MMAs run: the columns' scales and biases into shared memory, the first
            // piece of the residual into registers
            float* s_col = reinterpret_cast<float*>(sm + SM::kCols) + buf * 512 + half * 128;
            {
                const int c = quad * 32 + lane, n = n0 + c;
                const bool in = c < wr && n < p.N;
                s_col[c] = in ? p.w_scale[n] : 0.f;
                s_col[256 + c] = in && p.bias ? linear_load1(p.bias, n, p.param_type) : 0.f;
            }
            // the rows this lane moves: 8 i + lane / 4, 16 bytes at lane % 4 of each 64-byte piece
            long long out_row[4], res_row[4];
            bool live[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int mr = tm * 256 + rank * 128 + quad * 32 + 8 * r + (lane >> 2);
                const int b = mr / p.tokens, tk = mr - b * p.tokens;
                live[r] = mr < p.M;
                out_row[r] = b * p.out_sb + tk * p.out_sn;
                res_row[r] = b * p.res_sb + tk * p.res_sn;
            }
            named_bar_sync(1 + half, 128);
            const bool any_res = p.vec && p.residual;
            const int cols = p.out_type == 2 ? 16 : 32;
            uint4 res[4];  // the residual's piece that comes next
            auto fetch = [&](int n) {
                if (any_res && n < n0 + wr && n + cols <= p.N) pair_fetch(res, p, res_row, live, n, lane);
            };
            fetch(n0);
            if (!warp_wait_bounded(bar_af(buf), (done >> 1) & 1, abort_flag, lim)) failed = true;
            tc_fence_after();
            const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * 256 + half * wr;
#pragma unroll 1
            for (int ch = 0; 32 * ch < wr; ++ch) {
                uint32_t acc[32];
                const int n = n0 + 32 * ch;
                tmem_ld32(tl + 32 * ch, acc);
                tmem_wait_ld();
                if (failed || n >= p.N) continue;  // the same for the whole warp
                const int m0 = tm * 256 + rank * 128 + quad * 32;
                if (p.vec && n + 32 <= p.N) {
                    if (p.out_type == 2) {
                        pair_piece<true, true>(p, row, m0, n, acc, s_col + 32 * ch, any_res, res, stage, out_row, live,
                                               lane);
                        fetch(n + 16);
                        pair_piece<true, true>(p, row, m0, n + 16, acc + 16, s_col + 32 * ch + 16, any_res, res, stage,
                                               out_row, live, lane);
                    } else {
                        pair_piece<false, true>(p, row, m0, n, acc, s_col + 32 * ch, any_res, res, stage, out_row, live,
                                                lane);
                    }
                    fetch(n + 32);
                } else if (p.out_type == 2) {
                    pair_piece<true, false>(p, row, m0, n, acc, s_col + 32 * ch, p.residual, res, stage, out_row, live,
                                            lane);
                    pair_piece<true, false>(p, row, m0, n + 16, acc + 16, s_col + 32 * ch + 16, p.residual, res, stage,
                                            out_row, live, lane);
                } else {
                    pair_piece<false, false>(p, row, m0, n, acc, s_col + 32 * ch, p.residual, res, stage, out_row, live,
                                             lane);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(bar_ae(buf), 0));
        }
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    if (warp == 8 && lane == 0) ctl[2] = (uint32_t)issued;
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    // After an abort in either CTA both CTAs' loads land, and CTA 0's MMAs finish, before TMEM
    // is freed.  All roles are done, so the counts of loads stand; a stage that only one CTA
    // has loaded is completed by an arrival in the other's place.
    const bool aborted = ld_cluster_u32(mapa_shared(smem_u32(ctl + 1), 0)) | ld_cluster_u32(mapa_shared(smem_u32(ctl + 1), 1));
    if (aborted) {
        if (warp == 8 && lane == 0 && leader) {
            const int own = issued, peer = (int)ld_cluster_u32(mapa_shared(smem_u32(ctl + 2), 1));
            const int most = own > peer ? own : peer;
            for (int t = most > NS ? most - NS : 0; t < most; ++t) {
                if (t >= own || t >= peer) mbar_arrive(bar_full(t % NS));
                wait_drain(bar_full(t % NS), (t / NS) & 1);
            }
        }
        if (warp == 9 && leader && elect_one()) {  // the lane that issued the MMAs
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
// The MMAs read 128 rows of A a stage, but only the rows that exist are loaded, so with few
// rows the stages of A stand box_rows apart and each one's unused rows are its neighbours':
// their sums are never read.  W's stages come first, then A's, then room for the last one.
struct SplitSmem {
    static constexpr int kBars = 0;  // full[10], empty[10], acc, drain
    static constexpr int kCtl = (2 * kMaxStages + 2) * 8;
    static constexpr int kRing = 1024;
    static __host__ __device__ constexpr int stage_bytes(int bn, int box) { return (bn + box) * 128; }
    static __host__ __device__ constexpr int pitch(int bn) { return bn * 4 + 16; }  // bytes a row of the staged sums
    static __host__ __device__ constexpr int alloc(int bn, int box, int stages) {
        const int ring = stages * stage_bytes(bn, box) + (128 - box) * 128, sums = box * pitch(bn);
        return kRing + (ring > sums ? ring : sums) + 1024;
    }
};
static_assert(SplitSmem::kCtl + 16 <= SplitSmem::kRing, "barriers before the ring");
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
    const int NS = p.stages, BN = p.bn;
    const uint32_t idesc = idesc_s8_s32(128, BN);
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t bars = smem_u32(sm) + SM::kBars, ring = smem_u32(sm) + SM::kRing;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
    const uint32_t bar_acc = bars + 8u * (2 * kMaxStages), bar_drain = bars + 8u * (2 * kMaxStages + 1);
    uint32_t* ctl = reinterpret_cast<uint32_t*>(sm + SM::kCtl);
    volatile uint32_t* abort_flag = ctl + 1;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
    const int n0 = (int)(blockIdx.x / splits) * BN, m0 = (int)blockIdx.y * 128;
    const int rows = min(128, p.M - m0);
    const int ksteps = (p.K + 127) / 128;
    const int k0 = (int)((long long)ksteps * rank / splits), k1 = (int)((long long)ksteps * (rank + 1) / splits);
    const uint64_t lim = p.wait_limit;
    const int w_bytes = BN * 128, a_bytes = p.box_rows * 128, pitch = SM::pitch(BN);
    const uint32_t ring_a = ring + NS * w_bytes;

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
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl[0], 0);
    int issued = 0;
    bool ok = true;

    if (warp == 4) {
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmW);
        }
        int st = 0;          // stage, and the parity of its next wait
        uint32_t par = 1;
        for (int k = k0; k < k1; ++k) {
            if (issued >= NS && !warp_poll_bounded(bar_empty(st), par, abort_flag, lim)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar_full(st), (uint32_t)(w_bytes + a_bytes));
                tma_load_2d(ring + st * w_bytes, &tmW, bar_full(st), k * 128, n0);
                tma_load_2d(ring_a + st * a_bytes, &tmA, bar_full(st), k * 128, m0);
            }
            ++issued;
            if (++st == NS) st = 0, par ^= 1;
        }
    } else if (warp == 5) {
        const uint64_t da = smem_desc_sw128(ring_a, 16, 1024), dw = smem_desc_sw128(ring, 16, 1024);
        const uint64_t step_a = (uint64_t)(a_bytes >> 4), step_w = (uint64_t)(w_bytes >> 4);
        int st = 0;
        uint32_t par = 0;
        uint64_t sa = da, sw = dw;
        for (int k = k0; k < k1; ++k) {
            if (!warp_poll_bounded(bar_full(st), par, abort_flag, lim)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_s8_ss(tmem, sa + 2 * kk, sw + 2 * kk, idesc, (k > k0 || kk > 0) ? 1u : 0u);
                mma_commit(bar_empty(st));
            }
            __syncwarp();
            sa += step_a, sw += step_w;
            if (++st == NS) st = 0, par ^= 1, sa = da, sw = dw;
        }
        if (ok && elect_one()) mma_commit(bar_acc);
    } else if (warp * 32 < rows) {
        ok = warp_wait_bounded(bar_acc, 0, abort_flag, lim);
        tc_fence_after();
        if (ok) {
            // every MMA is done, so the operand ring is free
            unsigned char* dst = sm + SM::kRing + (warp * 32 + lane) * pitch;
            const bool stored = warp * 32 + lane < rows;
            const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            for (int ch = 0; ch < BN / 32; ++ch) {
                uint32_t acc[32];
                __syncwarp();
                tmem_ld32(tl + 32 * ch, acc);
                tmem_wait_ld();
                if (!stored) continue;
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
        if (warp == 5 && elect_one()) {  // the lane that issued the MMAs
            mma_commit(bar_drain);
            wait_drain(bar_drain, 0);
        }
        __syncthreads();
    }
    if (splits > 1) cluster_sync();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, BN);

    // the splits' sums: a thread keeps four columns, whose parameters it loads once, and walks the
    // rows that are dealt over the cluster
    const int groups = BN / 4, rows_at_once = kSplitThreads / groups;
    const int c = 4 * (tid % groups), n = n0 + c;
    if (!*abort_flag && n < p.N) {
        const bool whole = p.vec && n + 4 <= p.N;
        float sw[4], bias[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sw[q] = n + q < p.N ? p.w_scale[n + q] : 0.f;
            bias[q] = p.bias && n + q < p.N ? linear_load1(p.bias, n + q, p.param_type) : 0.f;
        }
        const long long col = linear_col(p, n);
#pragma unroll 2
        for (int r = rank * rows_at_once + tid / groups; r < rows; r += splits * rows_at_once) {
            const LinearRow row = linear_row(p, m0 + r);
            float res[4];
            if (whole && row.res) linear_read4(res, row.res, n, p.out_type);
            const uint32_t at = ring + r * pitch + c * 4;
            uint32_t acc[4] = {0, 0, 0, 0};
            for (int s = 0; s < splits; ++s) {
                const int4 v = splits > 1 ? ld_cluster_int4(mapa_shared(at, s))
                                          : *reinterpret_cast<const int4*>(sm + SM::kRing + r * pitch + c * 4);
                acc[0] += v.x;
                acc[1] += v.y;
                acc[2] += v.z;
                acc[3] += v.w;
            }
            if (whole) {
                float v[4];
                linear_value<4, true>(v, p, row, n, acc, sw, bias);
                if (row.res) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] += res[q];
                }
                linear_write4(row.out, col, v, p.out_type);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (n + q < p.N) linear_finish1(p, row, n + q, (int)acc[q]);
            }
        }
    }
    if (splits > 1) cluster_sync();  // no CTA leaves while its sums may still be read
}

}  // namespace sba
