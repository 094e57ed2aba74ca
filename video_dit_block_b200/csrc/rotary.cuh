// rotary.cuh -- rotary positions of attention inputs: adjacent ("interleaved") or split
// ("half") channel pairs, on the first rope_dim channels of each head, several position
// axes, any frequency per pair.
//
// The producer (producer.cuh) turns normed Q and K by the 3D rotation of the page
// "MiniMax-H3 on 8xH200 benchmark" (news.paixiangai.cn); this is the rotation by itself,
// for models that pair their channels or scale their frequencies otherwise.  Pair p =
// (u, v) of a token at position pos[a] on the pair's axis a turns by theta = pos[a] * w_p:
//   (u, v) -> amp * (u cos theta - v sin theta, u sin theta + v cos theta)
// (inverse: by -theta).  Channels past rope_dim are copied.  fp32 arithmetic, one rounding.
//
// Angles.  A turn is 2^64: F_p = round(w_p / 2 pi * 2^64), formed on the host, and pos * F_p
// modulo 2^64 drops whole turns exactly, so a position of 2^31 costs no more accuracy than
// position 1, whatever the frequency (2^-34 turns from the rounding of F_p, 2^-25 of the
// angle from its conversion to fp32).
//
// HBM-bound: x is read once and written once.  A thread owns 16 channels of one token in two
// runs of 8, such that its neighbours' runs are next to its own, takes their sines and
// cosines once and applies them to all heads of its chunk, four heads' loads in flight at a
// time (two of fp32).  Three CTAs an SM: with 40 heads of 128 bf16 channels, all turned, 119 to
// 121 us for 37824 tokens, the rate of a copy; two CTAs (no register limit) take 133, four 134 us.
// Widths off the vector form's multiples move value by value: 60 of 128 channels on three axes
// take 402 us where 96 take 122.
#pragma once
#include <cstdint>

#include "residual_norm.cuh"  // unpack16, pack16

namespace sba {

constexpr int kMaxRotaryPairs = 128;

struct RotaryParams {
    const void* x;
    void* out;
    const int32_t* pos;                      // [B][N][axes]
    long long x_sb, x_sh, x_sn, o_sb, o_sh, o_sn;  // strides in elements
    int H, N, D, axes, pairs;
    int heads_per_cta;
    int half, copy, fp16;                    // copy: channels past rope_dim are written
    float sin_amp, cos_amp;
    unsigned long long turn[kMaxRotaryPairs];
    unsigned char axis[kMaxRotaryPairs];
};

__device__ __forceinline__ void rotary_sincos(const RotaryParams& p, const int32_t* pos, int pair, float& s, float& c) {
    const unsigned long long a = (unsigned long long)(long long)pos[p.axis[pair]] * p.turn[pair];
    // the top 32 bits as a signed fraction of a turn; sincospif takes half turns
    sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);
    s *= p.sin_amp;
    c *= p.cos_amp;
}

// Eight consecutive values, 16-byte accesses.
template <bool F32>
struct Raw8Words {
    uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8Words<F32> rotary_load(const char* q) {
    Raw8Words<F32> r;
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) r.w[i] = ldg_stream(q + 16 * i);
    return r;
}
template <bool F32>
__device__ __forceinline__ void rotary_values(const Raw8Words<F32>& raw, int fp16, float (&f)[8]) {
    const uint4 a = raw.w[0], b = raw.w[F32 ? 1 : 0];
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        if (F32) {
            f[e] = __uint_as_float(u[e]);
            f[e + 1] = __uint_as_float(u[e + 1]);
        } else {
            unpack16(u[e / 2], fp16, f[e], f[e + 1]);
        }
    }
}
template <bool F32>
__device__ __forceinline__ void rotary_store(char* q, const float (&f)[8], int fp16) {
    if (F32) {
        stg_stream(q, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
        stg_stream(q + 16, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                                      __float_as_uint(f[7])));
    } else {
        stg_stream(q, make_uint4(pack16(f[0], f[1], fp16), pack16(f[2], f[3], fp16), pack16(f[4], f[5], fp16),
                                 pack16(f[6], f[7], fp16)));
    }
}

// Vector form: D a multiple of 16, pairs of 8 (half) or 4 (interleaved), rows 16-byte aligned.
// Thread t of the grid's x owns 16 channels of token t / (D / 16).
template <bool F32, bool HALF>
__global__ void __launch_bounds__(256, 3) rotary_vec_kernel(const __grid_constant__ RotaryParams p) {
    constexpr int W = F32 ? 4 : 2;
    constexpr int U = F32 ? 2 : 4;  // heads in flight
    const int tpt = p.D >> 4;       // threads per token
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int j = (int)(id % tpt);
    if (id / tpt >= p.N) return;
    const int n = (int)(id / tpt);
    const int b = blockIdx.z;
    const int h0 = blockIdx.y * p.heads_per_cta;
    const int h1 = min(p.H, h0 + p.heads_per_cta);
    // The two runs.  half: the pairs' first and second channels, or two runs to copy.
    // Interleaved: runs j and j + D / 16 of the row, each of four pairs or to copy.
    int c0 = 8 * j, c1;
    bool on0, on1;
    if (HALF) {
        on0 = on1 = c0 < p.pairs;
        if (!on0) c0 += p.pairs;
        c1 = on0 ? c0 + p.pairs : c0 + (p.D / 2 - p.pairs);
    } else {
        c1 = c0 + p.D / 2;
        on0 = c0 < 2 * p.pairs;
        on1 = c1 < 2 * p.pairs;
    }
    if (!p.copy && !on0 && !on1) return;
    const bool do0 = HALF || on0 || p.copy, do1 = HALF || on1 || p.copy;
    const char* x = static_cast<const char*>(p.x) + (b * p.x_sb + n * p.x_sn) * W;
    char* o = static_cast<char*>(p.out) + (b * p.o_sb + n * p.o_sn) * W;
    if (HALF && !on0) {
        for (int h = h0; h < h1; ++h) {
            const Raw8Words<F32> ra = rotary_load<F32>(x + (h * p.x_sh + c0) * W);
            const Raw8Words<F32> rb = rotary_load<F32>(x + (h * p.x_sh + c1) * W);
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) {
                stg_stream(o + (h * p.o_sh + c0) * W + 16 * i, ra.w[i]);
                stg_stream(o + (h * p.o_sh + c1) * W + 16 * i, rb.w[i]);
            }
        }
        return;
    }
    float s[8], c[8];
    const int32_t* pos = p.pos + ((long long)b * p.N + n) * p.axes;
    if (HALF || on0) {
#pragma unroll
        for (int e = 0; e < (HALF ? 8 : 4); ++e) rotary_sincos(p, pos, (HALF ? c0 : c0 / 2) + e, s[e], c[e]);
    }
    if (!HALF && on1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) rotary_sincos(p, pos, c1 / 2 + e, s[4 + e], c[4 + e]);
    }
    for (int h = h0; h < h1; h += U) {
        Raw8Words<F32> ra[U], rb[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (h + i < h1) {
                if (do0) ra[i] = rotary_load<F32>(x + ((h + i) * p.x_sh + c0) * W);
                if (do1) rb[i] = rotary_load<F32>(x + ((h + i) * p.x_sh + c1) * W);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (h + i >= h1) break;
            float a[8], d[8];
            rotary_values<F32>(ra[i], p.fp16, a);
            rotary_values<F32>(rb[i], p.fp16, d);
            if (HALF) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = a[e], v = d[e];
                    a[e] = fmaf(u, c[e], -v * s[e]);
                    d[e] = fmaf(u, s[e], v * c[e]);
                }
            } else {
                if (on0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float u = a[2 * e], v = a[2 * e + 1];
                        a[2 * e] = fmaf(u, c[e], -v * s[e]);
                        a[2 * e + 1] = fmaf(u, s[e], v * c[e]);
                    }
                }
                if (on1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float u = d[2 * e], v = d[2 * e + 1];
                        d[2 * e] = fmaf(u, c[4 + e], -v * s[4 + e]);
                        d[2 * e + 1] = fmaf(u, s[4 + e], v * c[4 + e]);
                    }
                }
            }
            if (do0) rotary_store<F32>(o + ((h + i) * p.o_sh + c0) * W, a, p.fp16);
            if (do1) rotary_store<F32>(o + ((h + i) * p.o_sh + c1) * W, d, p.fp16);
        }
    }
}

// Any size and alignment: a thread per (token, pair) or (token, copied channel).
template <bool F32>
__global__ void __launch_bounds__(256) rotary_any_kernel(const __grid_constant__ RotaryParams p) {
    const int units = p.copy ? p.D - p.pairs : p.pairs;  // the pairs, then the copied channels
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long n = id / units;
    const int j = (int)(id % units);
    if (n >= p.N) return;
    const int b = blockIdx.z;
    const int h0 = blockIdx.y * p.heads_per_cta;
    const int h1 = min(p.H, h0 + p.heads_per_cta);
    const bool turned = j < p.pairs;
    const int c0 = turned ? (p.half ? j : 2 * j) : p.pairs + j;
    const int c1 = turned ? (p.half ? p.pairs + j : 2 * j + 1) : c0;
    const long long xo = b * p.x_sb + n * p.x_sn, oo = b * p.o_sb + n * p.o_sn;
    auto load = [&](long long at) {
        if (F32) return static_cast<const float*>(p.x)[at];
        float a, z;
        unpack16(static_cast<const uint16_t*>(p.x)[at], p.fp16, a, z);
        return a;
    };
    auto store = [&](long long at, float f) {
        if (F32) static_cast<float*>(p.out)[at] = f;
        else static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack16(f, 0.f, p.fp16);
    };
    float s = 0.f, c = 1.f;
    if (turned) rotary_sincos(p, p.pos + ((long long)b * p.N + n) * p.axes, j, s, c);
    for (int h = h0; h < h1; ++h) {
        const float u = load(xo + h * p.x_sh + c0);
        if (!turned) {
            store(oo + h * p.o_sh + c0, u);
            continue;
        }
        const float v = load(xo + h * p.x_sh + c1);
        store(oo + h * p.o_sh + c0, fmaf(u, c, -v * s));
        store(oo + h * p.o_sh + c1, fmaf(u, s, v * c));
    }
}

}  // namespace sba
