// residual_norm.cuh -- the row operators around a transformer block: the gated residual of
// the block's output with an optional norm of that output, the norm of the new residual
// row with its modulation, and the 8-bit quantisation of a row.
//
// The page "MiniMax-H3 on 8xH200 benchmark" (news.paixiangai.cn), the kernel layer,
// lists an indexed AdaLN and a gated residual among its fused kernels; the formulas here
// are the usual ones.  Per row (b, n) of C channels, with g the row's modulation row
// (its sample's, or index[b][n]):
//   z = y, or post(y) * post_weight      r = x + gate[g] * z
//   layer norm:  u = (r - mean r) / sqrt(mean (r - mean r)^2 + eps)
//   RMS norm:    u = r / sqrt(mean r^2 + eps)
//   h = (u * weight + bias) * (1 + scale[g]) + shift[g]
//   quantised:   s = max|h| / 127,  code = nearest integer to fp32(h * fp32(127 / max|h|))
// All of it in fp32; r and h are rounded once, on their way out, and the norm reads the
// unrounded r.  The mean comes first and the squared distances from it second, both
// from registers, so a large common offset costs no digits.
//
// HBM-bound: x and y are read once, r and h written once; a row stays in the registers of
// its threads, VPT chunks of 8 channels each, all its loads issued before the first use.
// CTAs stay and walk the rows, the next row's loads in flight under this one's arithmetic.
// Rows of up to 1024 channels take a warp, wider ones a CTA of as many warps as they need.
// Arithmetic is in packed pairs: at 29 instructions a channel an earlier form was bound by
// issue, not by memory.  The parameter rows are shared by all rows of a sample and come from
// L1: they are the only loads that may allocate there, the streams bypass it.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/sba.h"
#include "common.cuh"

namespace sba {

enum RowNorm : int { kNormNone = 0, kNormLayer = 1, kNormRms = 2 };

struct RowParams {
    const void* x;
    const void* y;             // NULL: no residual step
    void* r;                   // the new residual rows (with y)
    void* h;                   // normed rows, or int8 codes
    float* h_scale;            // quantised: one scale a row
    const int32_t* valid_len;  // [B] or NULL
    const int32_t* index;      // [B][N] or NULL: row b of the modulation tables
    const void* gate;          // [G][C] each, or NULL
    const void* scale;
    const void* shift;
    const void* weight;        // [C] each, or NULL
    const void* bias;
    const void* post_weight;
    const char *x_end, *y_end;  // past the last byte of x and y (rows off the 16-byte grid)
    long long x_sb, x_sn, y_sb, y_sn, r_sb, r_sn, h_sb, h_sn;  // strides in elements
    long long x_sh;            // x in head layout: channel c is channel c % D of head c / D
    int D;                     // head dimension; 0 = plain rows
    int N, C, G;
    int Cq;                    // quantised: code columns, C rounded up to 16
    long long rows;            // B * N
    int norm, post, quant;
    int param32;               // parameters are fp32 (else the 16-bit type)
    float eps;
    int* error;                // the device's error word (with index)
};

// The launch for types XT, HT (as RowType); vec: rows and parameters on their wide grids.
template <int XT, int HT>
sba_status run_rows(const RowParams& p, bool vec, cudaStream_t s);

// Two 16-bit values of a 32-bit word as floats, and back (one rounding, to nearest even).
__device__ __forceinline__ void unpack16(uint32_t w, int fp16, float& a, float& b) {
    if (fp16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = f.x;
        b = f.y;
    } else {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int fp16) {
    if (fp16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Streaming 16-byte loads and stores: read and written once, kept out of L1.  Not through
// the read-only path, since the outputs may be the inputs.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void stg_stream(void* p, const uint4& v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// How a kernel holds its rows.  T: 0 bf16, 1 fp16, 2 fp32.
enum RowType : int { kRowBf16 = 0, kRowFp16 = 1, kRowFp32 = 2 };

// A thread's place in its row: chunk v of thread t holds the 8 channels from row_col on.  With
// VEC rows start on 16 bytes and C is a multiple of 8, so a chunk lies in the row (the first
// `live` ones) or past it.  Otherwise the chunks start `a` channels before the row, at the 16
// bytes that its first channel lies in, so that all but the row's two ends move in 16-byte
// accesses just the same; `a` differs from row to row.
struct RowPlace {
    int t, tpr, C, live, a;
};
template <bool VEC>
__device__ __forceinline__ int row_col(int v, const RowPlace& q) {
    return (v * q.tpr + q.t) * 8 - (VEC ? 0 : q.a);
}
template <bool VEC>
__device__ __forceinline__ bool row_full(int v, const RowPlace& q) {
    const int c = row_col<VEC>(v, q);
    return VEC ? v < q.live : c >= 0 && c + 8 <= q.C;
}
__device__ __forceinline__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Eight values of a row as loaded: one 16-byte word of 16-bit values, two of fp32.
template <int T>
struct Raw8 {
    static constexpr int kWords = T == kRowFp32 ? 2 : 1;
    uint4 w[kWords];
};

// Values outside the row are zeros.  W: bytes a value.
template <int T>
__device__ __forceinline__ Raw8<T> row_edge(const char* base, int c, int C) {
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool in = (unsigned)(c + e) < (unsigned)C;
        uint32_t x = 0;
        if (in) x = T == kRowFp32 ? reinterpret_cast<const uint32_t*>(base)[c + e] : reinterpret_cast<const uint16_t*>(base)[c + e];
        if (T == kRowFp32) u[e] = x;
        else if (e & 1) u[e / 2] |= x << 16;
        else u[e / 2] = x;
    }
    Raw8<T> r;
    r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    if (T == kRowFp32) r.w[Raw8<T>::kWords - 1] = make_uint4(u[4], u[5], u[6], u[7]);
    return r;
}
// Zeros for the values outside the row.
template <int T>
__device__ __forceinline__ void row_mask(Raw8<T>& r, int c, int C) {
    uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, 0, 0, 0, 0};
    if (T == kRowFp32) {
        const uint4 b = r.w[Raw8<T>::kWords - 1];
        u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool in = (unsigned)(c + e) < (unsigned)C;
        if (T == kRowFp32) u[e] = in ? u[e] : 0u;
        else u[e / 2] &= in ? 0xffffffffu : e & 1 ? 0x0000ffffu : 0xffff0000u;
    }
    r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    if (T == kRowFp32) r.w[Raw8<T>::kWords - 1] = make_uint4(u[4], u[5], u[6], u[7]);
}
// [lo, hi): the bytes of the whole tensor.  A row's first and last 16 bytes may hold its
// neighbours' values, which are read too and masked later; nothing outside the tensor is
// read.  (Its own two ends, and a tensor that starts elsewhere on the 16-byte grid than the chunks
// do, go value by value, in little code.)
template <int T, bool VEC>
__device__ __forceinline__ void row_load(Raw8<T>& raw, const char* base, int v, const RowPlace& q, const char* lo,
                                         const char* hi) {
    constexpr int W = T == kRowFp32 ? 4 : 2;
    const int c = row_col<VEC>(v, q);
    const char* p = base + c * W;
    if (VEC ? v < q.live : c < q.C && p >= lo && p + 8 * W <= hi && on16(p)) {
#pragma unroll
        for (int i = 0; i < Raw8<T>::kWords; ++i) raw.w[i] = ldg_stream(p + 16 * i);
    } else {
#pragma unroll
        for (int i = 0; i < Raw8<T>::kWords; ++i) raw.w[i] = make_uint4(0, 0, 0, 0);
        if (!VEC && c < q.C) {
#pragma unroll 1
            for (int e = 7; e >= 0; --e) {
                const bool in = (unsigned)(c + e) < (unsigned)q.C;
                uint4 &a = raw.w[0], &b = raw.w[Raw8<T>::kWords - 1];
                if (T == kRowFp32) {
                    b.w = b.z; b.z = b.y; b.y = b.x; b.x = a.w; a.w = a.z; a.z = a.y; a.y = a.x;
                    a.x = in ? reinterpret_cast<const uint32_t*>(base)[c + e] : 0u;
                } else {
                    a.w = a.w << 16 | a.z >> 16;
                    a.z = a.z << 16 | a.y >> 16;
                    a.y = a.y << 16 | a.x >> 16;
                    a.x = a.x << 16 | (in ? reinterpret_cast<const uint16_t*>(base)[c + e] : 0u);
                }
            }
        }
    }
}

// As four packed pairs of floats.
template <int T, bool VEC>
__device__ __forceinline__ void row_values(Raw8<T>& raw, uint64_t (&f)[4], int v, const RowPlace& q) {
    if (!VEC && !row_full<VEC>(v, q)) row_mask<T>(raw, row_col<VEC>(v, q), q.C);
    const uint4 a = raw.w[0], b = raw.w[Raw8<T>::kWords - 1];
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        if (T == kRowFp32) {
            lo = __uint_as_float(u[2 * i]);
            hi = __uint_as_float(u[2 * i + 1]);
        } else {
            unpack16(u[i], T, lo, hi);
        }
        f[i] = pack2(lo, hi);
    }
}

template <int T, bool VEC>
__device__ __forceinline__ void row_store(char* base, const uint64_t (&f)[4], int v, const RowPlace& q) {
    constexpr int W = T == kRowFp32 ? 4 : 2;
    float g[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(f[i], g[2 * i], g[2 * i + 1]);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = T == kRowFp32 ? __float_as_uint(g[i]) : i < 4 ? pack16(g[2 * i], g[2 * i + 1], T) : 0u;
    const int c = row_col<VEC>(v, q);
    char* p = base + c * W;
    if (row_full<VEC>(v, q) && (VEC || on16(p))) {
        stg_stream(p, make_uint4(u[0], u[1], u[2], u[3]));
        if (T == kRowFp32) stg_stream(p + 16, make_uint4(u[4], u[5], u[6], u[7]));
    } else if (!VEC && c < q.C) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if ((unsigned)(c + e) >= (unsigned)q.C) continue;
            if (T == kRowFp32) reinterpret_cast<uint32_t*>(base)[c + e] = u[e];
            else reinterpret_cast<uint16_t*>(base)[c + e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
        }
    }
}

// Eight parameters of the same columns, through L1: fp32, or 16-bit of type T16.  Columns
// outside the row give 0.
template <int T16, bool VEC>
__device__ __forceinline__ void param_load(uint64_t (&f)[4], const char* base, int param32, int v, const RowPlace& q) {
    float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int c = row_col<VEC>(v, q);
    if (VEC) {
        if (v < q.live) {
            if (param32) {
                // 32 bytes at once: two loads of 16 at a stride of 32 would each touch every line
                asm("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                    : "=f"(g[0]), "=f"(g[1]), "=f"(g[2]), "=f"(g[3]), "=f"(g[4]), "=f"(g[5]), "=f"(g[6]), "=f"(g[7])
                    : "l"(base + c * 4));
            } else {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(base + c * 2));
                unpack16(w.x, T16, g[0], g[1]);
                unpack16(w.y, T16, g[2], g[3]);
                unpack16(w.z, T16, g[4], g[5]);
                unpack16(w.w, T16, g[6], g[7]);
            }
        }
    } else if (c < q.C) {
        // the 16-byte words that the eight lie in, where those are all the row's, shifted; the
        // shift is the same for all threads
        const int PW = param32 ? 4 : 2, s = (int)((reinterpret_cast<uintptr_t>(base) + c * PW) & 15) / PW;
        const bool inside = c - s >= 0 && c - s + (param32 ? 12 : 16) <= q.C;
        const char* p = base + (c - s) * PW;
        if (!inside) {
            if (param32) {
                Raw8<kRowFp32> r = row_edge<kRowFp32>(base, c, q.C);
                row_values<kRowFp32, true>(r, f, v, q);
            } else {
                Raw8<T16 == kRowFp32 ? kRowBf16 : T16> r = row_edge<T16 == kRowFp32 ? kRowBf16 : T16>(base, c, q.C);
                row_values<T16 == kRowFp32 ? kRowBf16 : T16, true>(r, f, v, q);
            }
            return;
        }
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p)), y = __ldg(reinterpret_cast<const uint4*>(p + 16));
        uint32_t w[12] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, 0, 0, 0, 0};
        if (param32) {
            const uint4 z = __ldg(reinterpret_cast<const uint4*>(p + 32));
            w[8] = z.x; w[9] = z.y; w[10] = z.z; w[11] = z.w;
        }
        const int ws = param32 ? s : s >> 1;
        if (ws & 1) {
#pragma unroll
            for (int i = 0; i < 11; ++i) w[i] = w[i + 1];
        }
        if (ws & 2) {
#pragma unroll
            for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
        }
        if (param32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack16(s & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i], T16, g[2 * i], g[2 * i + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pack2(g[2 * i], g[2 * i + 1]);
}

// The larger of two values; a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum or maximum over the threads of a row: a warp's, or a CTA's.  `slot` alternates between
// calls, so one barrier per reduction suffices.
template <bool WARP, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*red)[32], int& slot) {
    if (MAX) {  // of values that are not negative: their bits are in their order, a NaN above all
        v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
    } else {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    if (!WARP) {
        // the slots past the CTA's warps hold zeros
        if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = v;
        __syncthreads();
        const float4* r = reinterpret_cast<const float4*>(red[slot]);
        for (int i = 0; i < (int)blockDim.x; i += 256) {  // eight warps
            const float4 a = r[i / 128], b = r[i / 128 + 1];
            const float w = MAX ? max_nan(max_nan(max_nan(a.x, a.y), max_nan(a.z, a.w)),
                                          max_nan(max_nan(b.x, b.y), max_nan(b.z, b.w)))
                                : ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
            v = i == 0 ? w : MAX ? max_nan(v, w) : v + w;
        }
        slot ^= 1;
    }
    return v;
}

// 1 / sqrt(mean of squares + eps) of the row's values (`centre`: about their mean, which is
// subtracted).  Columns past C hold 0 on entry and on return.
template <bool WARP, int VPT, bool VEC>
__device__ __forceinline__ float row_statistics(uint64_t (&f)[VPT][4], bool centre, const RowPlace& q, float inv_c,
                                                float eps, float (*red)[32], int& slot) {
    float a, b;
    if (centre) {
        uint64_t s = pack2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fadd2(s, f[v][i]);
        }
        unpack2(s, a, b);
        const float mean = row_reduce<WARP, false>(a + b, red, slot) * inv_c;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (VEC || row_full<VEC>(v, q)) {
                const float m = !VEC || v < q.live ? -mean : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) f[v][i] = fadd2(f[v][i], pack2(m, m));
            } else {
                const int c = row_col<VEC>(v, q);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[v][i] = fadd2(f[v][i], pack2((unsigned)(c + 2 * i) < (unsigned)q.C ? -mean : 0.f,
                                                   (unsigned)(c + 2 * i + 1) < (unsigned)q.C ? -mean : 0.f));
            }
        }
    }
    uint64_t s2 = pack2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = ffma2(f[v][i], f[v][i], s2);
    }
    unpack2(s2, a, b);
    return 1.f / sqrtf(row_reduce<WARP, false>(a + b, red, slot) * inv_c + eps);
}

__device__ __forceinline__ uint64_t row_mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A step of the row with one parameter: f = f a, f + a, or f + a z.
enum RowStep : int { kStepMul, kStepAdd, kStepGate };
template <int STEP, int T16, int VPT, bool VEC>
__device__ __forceinline__ void row_step(uint64_t (&f)[VPT][4], const uint64_t (&z)[VPT][4], const char* base,
                                         int param32, const RowPlace& q) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        uint64_t a[4];
        param_load<T16, VEC>(a, base, param32, v, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (STEP == kStepMul) f[v][i] = row_mul2(f[v][i], a[i]);
            if (STEP == kStepAdd) f[v][i] = fadd2(f[v][i], a[i]);
            if (STEP == kStepGate) f[v][i] = ffma2(a[i], z[v][i], f[v][i]);
        }
    }
}

// The calls a transformer block makes have kernels of their own: in the general one
// (kRowAny), which asks for every step as it goes, instruction fetch and issue cost more
// than memory does (37800 rows of 5120 channels in bf16, of the copy rate: the modulated norm
// 58%, with the gated residual 80%; on their own 81% and 94%, 146 and 252 us).
enum RowKind : int {
    kRowAny,
    kRowQuant,         // codes of plain rows
    kRowQuantHeads,    // codes of rows in head layout
    kRowNorm,          // norm with scale and shift
    kRowNormQuant,
    kRowGateNorm,      // gated residual, norm with scale and shift
    kRowGateNormQuant,
    kRowPostGateNorm,  // post norm, gated residual, norm without them
};

// The CTAs an SM that a kernel's registers leave room for.  16-bit rows without a y need few, and
// run faster at 80 registers (37800 x 5120, side by side: norm and modulation 144 us, with codes
// 155) than at 128 (149 and 176); fp32 rows and rows with a y would spill.
template <int XT, bool WARP, int VPT, int KIND>
constexpr int row_ctas() {
    if (WARP) return 4;
    if (VPT > 4 || KIND == kRowQuant || KIND == kRowQuantHeads) return 1;
    return XT != kRowFp32 && (KIND == kRowNorm || KIND == kRowNormQuant) ? 3 : 2;
}

// XT, HT: the types of x and r, and of y and h (as RowType).  WARP: four rows per CTA of four
// warps; otherwise a row per CTA, and as many CTAs as are resident.  P32: parameters in fp32.
template <int XT, int HT, bool WARP, int VPT, bool VEC, int KIND, bool P32>
__global__ void __launch_bounds__(WARP                  ? 128
                                  : KIND == kRowQuant || KIND == kRowQuantHeads ? 1024
                                  : VPT > 4                                     ? 512
                                                                                : 256,
                                  (row_ctas<XT, WARP, VPT, KIND>())) residual_norm_kernel(
    const __grid_constant__ RowParams p) {
    __shared__ __align__(16) float red[2][32];
    extern __shared__ __align__(16) unsigned char code_rows[];  // without VEC: a row's codes
    int slot = 0;
    const int tpr = WARP ? 32 : blockDim.x;
    unsigned char* codes = code_rows + (WARP ? (threadIdx.x >> 5) * (32 * VPT * 8) : 0);
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    constexpr int rpc = WARP ? 4 : 1;
    const uint32_t rows = (uint32_t)p.rows, N = (uint32_t)p.N, stride = gridDim.x * rpc;
    if (!WARP) {
        for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i >> 5][i & 31] = 0.f;
        __syncthreads();
    }
    constexpr bool kAny = KIND == kRowAny;
    const int param32 = kAny ? p.param32 : P32;  // a branch on it would part the loads of the chunks
    constexpr bool kGated = KIND == kRowGateNorm || KIND == kRowGateNormQuant || KIND == kRowPostGateNorm;
    constexpr bool kModulated = KIND == kRowNorm || KIND == kRowNormQuant || KIND == kRowGateNorm || KIND == kRowGateNormQuant;
    const bool has_y = kAny ? p.y != nullptr : kGated;
    const bool has_gate = kAny ? p.gate != nullptr : kGated;
    const bool has_post = kAny ? p.post != 0 : KIND == kRowPostGateNorm;
    const bool has_norm = kAny ? p.norm != 0 : KIND != kRowQuant && KIND != kRowQuantHeads;
    const bool has_scale = kAny ? p.scale != nullptr : kModulated;
    const bool has_shift = kAny ? p.shift != nullptr : kModulated;
    const bool quant = kAny ? p.quant != 0 : KIND == kRowQuant || KIND == kRowQuantHeads || KIND == kRowNormQuant || KIND == kRowGateNormQuant;
    const bool heads = kAny ? p.D != 0 : KIND == kRowQuantHeads;
    constexpr int XW = XT == kRowFp32 ? 4 : 2, HW = HT == kRowFp32 ? 4 : 2;
    RowPlace q{t, tpr, p.C, min(VPT, max(0, (p.C / 8 - t + tpr - 1) / tpr)), 0};
    const float inv_c = 1.f / (float)p.C;
    Raw8<XT> rx[VPT];
    Raw8<HT> ry[VPT];

    // A row's place in the tensors.  Rows step by the grid, within a sample by adding to the
    // addresses: finding each row anew took more instructions than a warp's channels did.
    struct At {
        uint32_t row, n;
        int b, len, a;
        const char *x, *y;
        char *r, *h;
    };
    const int h_width = quant ? 1 : HW;
    const long long dx = stride * p.x_sn * XW, dy = stride * p.y_sn * HW, dr = stride * p.r_sn * XW,
                    dh = stride * p.h_sn * h_width;
    // where the chunks start: by the narrowest tensor, the others mostly agree with it
    auto place = [&](At& a) {
        if (VEC || heads) a.a = 0;
        else if (XT == HT) a.a = (int)(reinterpret_cast<uintptr_t>(a.x) & 15) / XW;
        else if (has_y) a.a = (int)(reinterpret_cast<uintptr_t>(a.y) & 15) / HW;
        else if (!quant) a.a = (int)(reinterpret_cast<uintptr_t>(a.h) & 15) / HW;
        else a.a = (int)(reinterpret_cast<uintptr_t>(a.x) & 15) / XW;
    };
    auto seek = [&](At& a) {
        a.b = (int)(a.row / N);
        a.n = a.row - a.b * N;
        a.len = p.valid_len ? p.valid_len[a.b] : (int)N;
        a.x = static_cast<const char*>(p.x) + (a.b * p.x_sb + a.n * p.x_sn) * XW;
        a.y = static_cast<const char*>(p.y) + (a.b * p.y_sb + a.n * p.y_sn) * HW;
        a.r = static_cast<char*>(p.r) + (a.b * p.r_sb + a.n * p.r_sn) * XW;
        a.h = static_cast<char*>(p.h) + (a.b * p.h_sb + a.n * p.h_sn) * h_width;
        place(a);
    };
    auto step = [&](At& a) {
        a.row += stride;
        a.n += stride;
        if (a.n < N) {
            a.x += dx;
            a.y += dy;
            a.r += dr;
            a.h += dh;
            place(a);
        } else if (a.row < rows) {
            seek(a);
        }
    };
    // the loads of a row (padding is not read)
    auto load = [&](const At& a) {
        if (a.row >= rows || (int)a.n >= a.len) return;
        RowPlace qa = q;
        qa.a = a.a;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!heads) {
                row_load<XT, VEC>(rx[v], a.x, v, qa, static_cast<const char*>(p.x), p.x_end);
            } else if (VEC) {
                const int hd = row_col<true>(v, q) / p.D;
                // the head's row, moved back so that column c of it is channel c % D
                row_load<XT, VEC>(rx[v], a.x + hd * (p.x_sh - p.D) * XW, v, qa, nullptr, nullptr);
            } else {
                const int c = row_col<true>(v, q);
                uint32_t u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (c + e >= p.C) continue;
                    const char* at = a.x + ((c + e) / p.D * p.x_sh + (c + e) % p.D) * XW;
                    if (XW == 4) u[e] = *reinterpret_cast<const uint32_t*>(at);
                    else u[e / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(at) << (16 * (e & 1));
                }
                rx[v].w[0] = make_uint4(u[0], u[1], u[2], u[3]);
                if (XW == 4) rx[v].w[Raw8<XT>::kWords - 1] = make_uint4(u[4], u[5], u[6], u[7]);
            }
        }
        if (has_y) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) row_load<HT, VEC>(ry[v], a.y, v, qa, static_cast<const char*>(p.y), p.y_end);
        }
    };

    constexpr bool kAhead = VPT <= 4;  // registers for a second row
    At next;
    next.row = blockIdx.x * rpc + (WARP ? threadIdx.x >> 5 : 0);
    if (next.row >= rows) return;
    seek(next);
    load(next);
    while (next.row < rows) {
        const At at = next;
        q.a = at.a;
        step(next);
        uint64_t f[VPT][4];
        if ((int)at.n >= at.len) {
            // padding: zeros out, nothing read
#pragma unroll
            for (int i = 0; i < 4; ++i) f[0][i] = 0;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (has_y) row_store<XT, VEC>(at.r, f[0], v, q);
                if (has_norm && !quant) row_store<HT, VEC>(at.h, f[0], v, q);
            }
            if (quant) {
                for (int c = 16 * t; c < p.Cq; c += 16 * tpr) *reinterpret_cast<uint4*>(at.h + c) = make_uint4(0, 0, 0, 0);
                if (t == 0) p.h_scale[at.row] = 0.f;
            }
            load(next);
            continue;
        }

        // the row's modulation row
        int g = at.b;
        if (p.index) {
            g = p.index[at.row];
            if (g < 0 || g >= p.G) {
                if (t == 0) atomicCAS(p.error, 0, (int)kErrBadRouting);
                g = 0;
            }
        }
        const long long goff = (long long)g * p.C * (param32 ? 4 : 2);

        if (has_y) {
            uint64_t z[VPT][4];
#pragma unroll
            for (int v = 0; v < VPT; ++v) row_values<HT, VEC>(ry[v], z[v], v, q);
            float inv = 1.f;
            if (has_post) inv = row_statistics<WARP, VPT, VEC>(z, p.post == kNormLayer, q, inv_c, p.eps, red, slot);
            if (has_post) {
                const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[v][i] = row_mul2(z[v][i], inv2);
                }
                if (p.post_weight) row_step<kStepMul, HT, VPT, VEC>(z, z, static_cast<const char*>(p.post_weight), param32, q);
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) row_values<XT, VEC>(rx[v], f[v], v, q);
            if (has_gate) {
                row_step<kStepGate, HT, VPT, VEC>(f, z, static_cast<const char*>(p.gate) + goff, param32, q);
            } else {
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[v][i] = fadd2(f[v][i], z[v][i]);
                }
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) row_store<XT, VEC>(at.r, f[v], v, q);
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v) row_values<XT, VEC>(rx[v], f[v], v, q);
        }

        // the next row's loads run under this one's statistics and stores
        if (kAhead) load(next);

        if (has_norm) {
            const float inv = row_statistics<WARP, VPT, VEC>(f, p.norm == kNormLayer, q, inv_c, p.eps, red, slot);
            const uint64_t inv2 = pack2(inv, inv);
            uint64_t none[VPT][4];
            if (p.weight) row_step<kStepMul, HT, VPT, VEC>(f, none, static_cast<const char*>(p.weight), param32, q);
            if (!p.bias && has_scale) {
                // f inv (1 + scale) + shift in two steps: f (inv + inv scale) + shift
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    uint64_t a[4];
                    param_load<HT, VEC>(a, static_cast<const char*>(p.scale) + goff, param32, v, q);
                    if (has_shift) {
                        uint64_t s[4];
                        param_load<HT, VEC>(s, static_cast<const char*>(p.shift) + goff, param32, v, q);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[v][i] = ffma2(f[v][i], ffma2(a[i], inv2, inv2), s[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[v][i] = row_mul2(f[v][i], ffma2(a[i], inv2, inv2));
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[v][i] = row_mul2(f[v][i], inv2);
                }
                if (p.bias) row_step<kStepAdd, HT, VPT, VEC>(f, none, static_cast<const char*>(p.bias), param32, q);
                if (has_scale) {
#pragma unroll
                    for (int v = 0; v < VPT; ++v) {
                        uint64_t a[4];
                        param_load<HT, VEC>(a, static_cast<const char*>(p.scale) + goff, param32, v, q);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[v][i] = ffma2(f[v][i], a[i], f[v][i]);
                    }
                }
                if (has_shift)
                    row_step<kStepAdd, HT, VPT, VEC>(f, none, static_cast<const char*>(p.shift) + goff, param32, q);
            }
            if (!quant) {
#pragma unroll
                for (int v = 0; v < VPT; ++v) row_store<HT, VEC>(at.h, f[v], v, q);
            }
        }
        if (!quant) {
            if (!kAhead) load(next);
            continue;
        }

        // columns past C hold 0; a NaN becomes the row's scale
        float top = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                unpack2(f[v][i], lo, hi);
                asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(lo), "f"(hi));
            }
        }
        top = row_reduce<WARP, true>(top, red, slot);
        // below 2^-100 the reciprocal step would leave fp32's range: such a row counts as zero
        const bool zero = top < 7.888609052210118e-31f;
        const float inv = zero ? 0.f : __fdiv_rn(127.f, top);
        if (t == 0) p.h_scale[at.row] = zero ? 0.f : __fdiv_rn(top, 127.f);
        // Adding 1.5 * 2^23 to a product of at most 127 rounds it to the nearest integer, ties to
        // even, and leaves that integer in the low byte.  Both steps round by definition: packed,
        // the compiler makes one fused step of them, which decides some ties otherwise.
        constexpr float kMagic = 12582912.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            uint32_t code[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                unpack2(f[v][i], lo, hi);
                code[2 * i] = __float_as_uint(__fadd_rn(__fmul_rn(lo, inv), kMagic));
                code[2 * i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(hi, inv), kMagic));
            }
            uint2 w;
            w.x = __byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410);
            w.y = __byte_perm(__byte_perm(code[4], code[5], 0x0040), __byte_perm(code[6], code[7], 0x0040), 0x5410);
            const int k = (v * tpr + t) * 8;
            if (VEC) {
                if (k < p.Cq) *reinterpret_cast<uint2*>(at.h + k) = w;
            } else {
                *reinterpret_cast<uint2*>(codes + k) = w;
            }
        }
        if (!VEC) {
            // the codes stand `a` bytes late in shared memory: out in aligned words
            if (WARP) __syncwarp();
            else __syncthreads();
            for (int c = 16 * t; c < p.Cq; c += 16 * tpr) {
                const uint32_t* s = reinterpret_cast<const uint32_t*>(codes + c + (q.a & ~3));
                const int sh = 8 * (q.a & 3);
                *reinterpret_cast<uint4*>(at.h + c) =
                    make_uint4(__funnelshift_r(s[0], s[1], sh), __funnelshift_r(s[1], s[2], sh),
                               __funnelshift_r(s[2], s[3], sh), __funnelshift_r(s[3], s[4], sh));
            }
            if (WARP) __syncwarp();  // (a CTA's next row has a reduction before its codes)
        }
        if (!kAhead) load(next);
    }
}

}  // namespace sba
