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
// its TPR threads (VPT chunks of 8 channels each), all its loads issued before the first
// use.  The parameter rows are shared by all rows of a sample and come from L1: they are
// the only loads that may allocate there, the streams bypass it.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
    long long x_sb, x_sn, y_sb, y_sn, r_sb, r_sn, h_sb, h_sn;  // strides in elements
    long long x_sh;            // x in head layout: channel c is channel c % D of head c / D
    int D;                     // head dimension; 0 = plain rows
    int N, C, G;
    int Cq;                    // quantised: code columns, C rounded up to 16
    long long rows;            // B * N
    int norm, post, quant;
    int fp16;                  // 16-bit values are fp16 (else bf16)
    int param32;               // parameters are fp32 (else the 16-bit type)
    float eps;
};

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

// Eight values of a row as loaded: one 16-byte word of 16-bit values, or two of fp32.
template <bool F32>
struct Raw8 {
    uint4 w[F32 ? 2 : 1];
};

// The column of element e of chunk v of thread t: with VEC eight neighbours per thread,
// otherwise (rows whose address or length rules 16-byte accesses out) one neighbour per
// thread, so that a warp's single-element accesses coalesce.
template <int TPR, bool VEC>
__device__ __forceinline__ int row_col(int v, int t, int e) {
    return VEC ? (v * TPR + t) * 8 + e : (v * 8 + e) * TPR + t;
}

template <bool F32, int TPR, bool VEC>
__device__ __forceinline__ void row_load(Raw8<F32>& raw, const void* base, int v, int t, int C) {
    constexpr int W = F32 ? 4 : 2;
    if (VEC) {
        const int c = row_col<TPR, true>(v, t, 0);
        if (c < C) {
            const char* p = static_cast<const char*>(base) + (long long)c * W;
            raw.w[0] = ldg_stream(p);
            if (F32) raw.w[F32 ? 1 : 0] = ldg_stream(p + 16);
        }
    } else {
        uint32_t u[F32 ? 8 : 4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = row_col<TPR, false>(v, t, e);
            uint32_t val = 0;
            if (c < C) val = F32 ? static_cast<const uint32_t*>(base)[c] : static_cast<const uint16_t*>(base)[c];
            if (F32) u[F32 ? e : 0] = val;
            else if (e & 1) u[e >> 1] |= val << 16;
            else u[e >> 1] = val;
        }
        raw.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
        if (F32) raw.w[F32 ? 1 : 0] = make_uint4(u[F32 ? 4 : 0], u[F32 ? 5 : 0], u[F32 ? 6 : 0], u[F32 ? 7 : 0]);
    }
}

template <bool F32>
__device__ __forceinline__ void raw_to_float(const Raw8<F32>& raw, int fp16, float (&f)[8]) {
    if (F32) {
        const uint4 a = raw.w[0], b = raw.w[F32 ? 1 : 0];
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(u[e]);
    } else {
        const uint32_t u[4] = {raw.w[0].x, raw.w[0].y, raw.w[0].z, raw.w[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack16(u[e], fp16, f[2 * e], f[2 * e + 1]);
    }
}

// Eight parameters of the same columns, through L1.  Columns past C give 0.
template <int TPR, bool VEC>
__device__ __forceinline__ void param_load(float (&f)[8], const void* base, int param32, int fp16, int v, int t, int C) {
    if (VEC) {
        const int c = row_col<TPR, true>(v, t, 0);
        if (c >= C) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = 0.f;
        } else if (param32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + c);
            const float4 a = __ldg(p), b = __ldg(p + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + c));
            unpack16(w.x, fp16, f[0], f[1]);
            unpack16(w.y, fp16, f[2], f[3]);
            unpack16(w.z, fp16, f[4], f[5]);
            unpack16(w.w, fp16, f[6], f[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = row_col<TPR, false>(v, t, e);
            float a = 0.f, b;
            if (c < C) {
                if (param32) a = __ldg(static_cast<const float*>(base) + c);
                else unpack16(__ldg(static_cast<const uint16_t*>(base) + c), fp16, a, b);
            }
            f[e] = a;
        }
    }
}

template <bool F32, int TPR, bool VEC>
__device__ __forceinline__ void row_store(void* base, const float (&f)[8], int fp16, int v, int t, int C) {
    if (VEC) {
        const int c = row_col<TPR, true>(v, t, 0);
        if (c >= C) return;
        if (F32) {
            float* p = static_cast<float*>(base) + c;
            stg_stream(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                     __float_as_uint(f[3])));
            stg_stream(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                                         __float_as_uint(f[7])));
        } else {
            stg_stream(static_cast<uint16_t*>(base) + c,
                       make_uint4(pack16(f[0], f[1], fp16), pack16(f[2], f[3], fp16), pack16(f[4], f[5], fp16),
                                  pack16(f[6], f[7], fp16)));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = row_col<TPR, false>(v, t, e);
            if (c >= C) continue;
            if (F32) static_cast<float*>(base)[c] = f[e];
            else static_cast<uint16_t*>(base)[c] = (uint16_t)pack16(f[e], 0.f, fp16);
        }
    }
}

// Sum or maximum over the TPR threads of a row.  Rows of more than a warp own their CTA;
// `slot` alternates between calls, so one barrier per reduction suffices.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*red)[TPR / 32 > 0 ? TPR / 32 : 1], int& slot) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    if (TPR > 32) {
        const int w = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[slot][w] = v;
        __syncthreads();
        v = red[slot][0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) v = MAX ? fmaxf(v, red[slot][i]) : v + red[slot][i];
        slot ^= 1;
    }
    return v;
}

// 1 / sqrt(mean of squares + eps) of the row's values (`centre`: about their mean, which is
// subtracted).  Columns past C hold 0 on entry and on return.
template <int TPR, int VPT, bool VEC>
__device__ __forceinline__ float row_statistics(float (&f)[VPT][8], bool centre, int t, int C, float eps,
                                                float (*red)[TPR / 32 > 0 ? TPR / 32 : 1], int& slot) {
    const float inv_c = 1.f / (float)C;
    if (centre) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s += f[v][e];
        }
        const float mean = row_reduce<TPR, false>(s, red, slot) * inv_c;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (VEC ? row_col<TPR, true>(v, t, 0) < C : row_col<TPR, false>(v, t, e) < C) f[v][e] -= mean;
        }
    }
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(f[v][e], f[v][e], q);
    }
    return 1.f / sqrtf(row_reduce<TPR, false>(q, red, slot) * inv_c + eps);
}

// X32 / H32: x and r (y and h) are fp32, else 16-bit.  One CTA of max(TPR, 128) threads per
// max(1, 128 / TPR) rows.
template <bool X32, bool H32, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) residual_norm_kernel(const RowParams p) {
    constexpr int RPC = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[2][TPR / 32 > 0 ? TPR / 32 : 1];
    int slot = 0;
    const int t = TPR < 128 ? threadIdx.x % TPR : threadIdx.x;
    const long long row = (long long)blockIdx.x * RPC + (TPR < 128 ? threadIdx.x / TPR : 0);
    if (row >= p.rows) return;
    const int b = (int)(row / p.N), n = (int)(row % p.N);
    const int C = p.C;
    constexpr int XW = X32 ? 4 : 2, HW = H32 ? 4 : 2;
    char* rrow = static_cast<char*>(p.r) + (b * p.r_sb + n * p.r_sn) * XW;
    char* hrow = static_cast<char*>(p.h) + (b * p.h_sb + n * p.h_sn) * (p.quant ? 1 : HW);

    float f[VPT][8];
    if (p.valid_len && n >= p.valid_len[b]) {
        // padding: zeros out, nothing read
#pragma unroll
        for (int e = 0; e < 8; ++e) f[0][e] = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (p.y) row_store<X32, TPR, VEC>(rrow, f[0], p.fp16, v, t, C);
            if (p.norm && !p.quant) row_store<H32, TPR, VEC>(hrow, f[0], p.fp16, v, t, C);
        }
        if (p.quant) {
            for (int c = 16 * t; c < p.Cq; c += 16 * TPR) *reinterpret_cast<uint4*>(hrow + c) = make_uint4(0, 0, 0, 0);
            if (t == 0) p.h_scale[row] = 0.f;
        }
        return;
    }

    // every load of the row before any use
    Raw8<X32> rx[VPT];
    Raw8<H32> ry[VPT];
    const char* xrow = static_cast<const char*>(p.x) + (b * p.x_sb + n * p.x_sn) * XW;
    if (p.D == 0) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) row_load<X32, TPR, VEC>(rx[v], xrow, v, t, C);
    } else if (VEC) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = row_col<TPR, true>(v, t, 0), hd = c / p.D;
            // the head's row, moved back so that column c of it is channel c % D
            row_load<X32, TPR, VEC>(rx[v], xrow + (hd * p.x_sh - (long long)hd * p.D) * XW, v, t, C);
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            Raw8<X32>& raw = rx[v];
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = row_col<TPR, false>(v, t, e);
                u[e] = 0;
                if (c < C) {
                    const char* q = xrow + ((c / p.D) * p.x_sh + c % p.D) * XW;
                    u[e] = X32 ? *reinterpret_cast<const uint32_t*>(q) : *reinterpret_cast<const uint16_t*>(q);
                }
            }
            if (X32) {
                raw.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
                raw.w[X32 ? 1 : 0] = make_uint4(u[4], u[5], u[6], u[7]);
            } else {
                raw.w[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
            }
        }
    }
    if (p.y) {
        const char* yrow = static_cast<const char*>(p.y) + (b * p.y_sb + n * p.y_sn) * HW;
#pragma unroll
        for (int v = 0; v < VPT; ++v) row_load<H32, TPR, VEC>(ry[v], yrow, v, t, C);
    }
    // the row's modulation row
    int g = b;
    if (p.index) {
        g = p.index[(long long)b * p.N + n];
        if (g < 0 || g >= p.G) {
            if (t == 0) raise_device_error(kErrBadRouting);
            g = 0;
        }
    }
    const long long goff = (long long)g * C * (p.param32 ? 4 : 2);

    if (p.y) {
        float z[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            raw_to_float<H32>(ry[v], p.fp16, z[v]);
            if (VEC && row_col<TPR, true>(v, t, 0) >= C) {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[v][e] = 0.f;
            }
        }
        float inv = 1.f;
        if (p.post) inv = row_statistics<TPR, VPT, VEC>(z, p.post == kNormLayer, t, C, p.eps, red, slot);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float a[8];
            if (p.post) {
                if (p.post_weight) {
                    param_load<TPR, VEC>(a, p.post_weight, p.param32, p.fp16, v, t, C);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[v][e] *= inv * a[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[v][e] *= inv;
                }
            }
            raw_to_float<X32>(rx[v], p.fp16, f[v]);
            if (p.gate) {
                param_load<TPR, VEC>(a, static_cast<const char*>(p.gate) + goff, p.param32, p.fp16, v, t, C);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] = fmaf(a[e], z[v][e], f[v][e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] += z[v][e];
            }
            row_store<X32, TPR, VEC>(rrow, f[v], p.fp16, v, t, C);
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) raw_to_float<X32>(rx[v], p.fp16, f[v]);
    }
    if (!p.norm && !p.quant) return;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (VEC && row_col<TPR, true>(v, t, 0) >= C) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[v][e] = 0.f;
        }
    }

    if (p.norm) {
        const float inv = row_statistics<TPR, VPT, VEC>(f, p.norm == kNormLayer, t, C, p.eps, red, slot);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float a[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[v][e] *= inv;
            if (p.weight) {
                param_load<TPR, VEC>(a, p.weight, p.param32, p.fp16, v, t, C);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] *= a[e];
            }
            if (p.bias) {
                param_load<TPR, VEC>(a, p.bias, p.param32, p.fp16, v, t, C);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] += a[e];
            }
            if (p.scale) {
                param_load<TPR, VEC>(a, static_cast<const char*>(p.scale) + goff, p.param32, p.fp16, v, t, C);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] = fmaf(f[v][e], a[e], f[v][e]);
            }
            if (p.shift) {
                param_load<TPR, VEC>(a, static_cast<const char*>(p.shift) + goff, p.param32, p.fp16, v, t, C);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] += a[e];
            }
            if (!p.quant) row_store<H32, TPR, VEC>(hrow, f[v], p.fp16, v, t, C);
        }
    }
    if (!p.quant) return;

    // Columns past C hold 0 here or are masked below, so they change no maximum.
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[v][e]));
    }
    top = row_reduce<TPR, true>(top, red, slot);
    // below 2^-100 the reciprocal step would leave fp32's range: such a row counts as zero
    const bool zero = !(top >= 7.888609052210118e-31f);
    const float inv = zero ? 0.f : __fdiv_rn(127.f, top);
    if (t == 0) p.h_scale[row] = zero ? 0.f : __fdiv_rn(top, 127.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        int q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = __float2int_rn(__fmul_rn(f[v][e], inv));
        if (VEC) {
            const int c = row_col<TPR, true>(v, t, 0);
            if (c < p.Cq) {
                uint2 w;
                w.x = (q[0] & 255) | (q[1] & 255) << 8 | (q[2] & 255) << 16 | (uint32_t)q[3] << 24;
                w.y = (q[4] & 255) | (q[5] & 255) << 8 | (q[6] & 255) << 16 | (uint32_t)q[7] << 24;
                *reinterpret_cast<uint2*>(hrow + c) = w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = row_col<TPR, false>(v, t, e);
                if (c < p.Cq) hrow[c] = (char)q[e];
            }
        }
    }
}

}  // namespace sba
