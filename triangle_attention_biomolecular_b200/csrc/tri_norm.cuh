// tri_norm.cuh -- layer norm of pair rows (forward, backward, restore) and the
// 8-bit activation checkpoint it can write and read, sm_100a.
//
// All of it is bound by HBM: a forward row of C channels is read once and
// written once against some 8 operations a channel.  A row therefore stays in
// registers between its two reductions: G lanes share it, sixteen channels
// each, so that a 128-channel BF16 row is eight lanes with one 32-byte load
// apiece and a warp works on four rows at once.  The variance is the second
// pass over the registers (sum of (x - mean)^2), never E[x^2] - mean^2.
//
// The 8-bit form shares a power-of-two scale between 32 neighbouring channels.
// With such a scale value / scale and code * scale are exact, so a code depends
// on one rounding only and BF16 restores it without another.
//
// Measured at 768 x 768 rows of 128 channels, in bytes that must move over time
// (6.57 TB/s is the card's copy rate): forward FP32 to BF16 72 us, 6.4 TB/s; its
// backward 115 us, 6.6 TB/s; forward BF16 with the int8 form 64 us, 6.0 TB/s;
// restore 45 us, 5.2 TB/s; backward from the int8 form 76 us, 5.1 TB/s; these
// last two issue the most instructions per byte.  A second row on its way per
// lane gained nothing (the BF16 backward spilled: 22 to 27 us at 384 x 384 rows).
#pragma once

#include <cuda_fp8.h>

#include "sm100.cuh"

namespace tri {

enum : int { ACT_NONE = 0, ACT_INT8 = 1, ACT_E4M3 = 2 };

struct NormParams {
    int64_t R;
    int C;
    int lanes;       // lanes per row: a power of two up to 32, or 32 x (warps per row)
    float inv_c, eps;
    const void* x;
    int64_t xs;
    const void *w, *b;
    int w_bf16;
    void* y;
    int64_t ys;
    float* stats;
    uint8_t* codes;
    int64_t cs;
    uint8_t* exps;
    int64_t es;
    const void* dy;
    int64_t dys;
    void* dx;
    int64_t dxs;
    float* partial;  // [gridDim.x][2][C], or NULL; a single block writes dw and db themselves
    float *dw, *db;
};

// ---------------------------------------------------------------------------
// sixteen channels of a row
// ---------------------------------------------------------------------------
// How the lanes of a row share its channels.  kVec: lane g has 16 g .. 16 g + 15,
// moved in aligned vectors.  Rows that cannot be moved so are walked element by
// element, neighbouring lanes on neighbouring channels, with a stride that the
// compiler knows: by 4 lanes (up to 64 channels: 8 rows per warp; 400000 rows of 50
// BF16 channels take 35 us forward, 70 with a warp per row) or by whole warps, 512
// channels each, where lane l has l, l + 32, l + 64, ...  Rows of up to 256 (128)
// channels have kBy32Half (kBy32Quarter), eight (four) channels per lane in place of
// sixteen, since those that a lane does not have would cost their instructions and
// registers all the same: 200000 rows of 100 BF16 channels take 36 us forward and
// 47 us backward in place of 74 and 208, 209 FP32 channels 62 and 86 in place of 78
// and 105.  The 8-bit activation by itself takes rows of 65 to 128 channels by 8
// lanes (kBy8): 200000 rows of 100 in 27 us in place of 45; with the norm's sums
// beside it that mode needs too many registers (backward 72 us).
enum : int { kVec = 0, kBy4 = 4, kBy8 = 8, kBy32 = 32, kBy32Half = 33, kBy32Quarter = 34 };
// channels per lane, and the lanes' stride where they are not neighbours
__host__ __device__ constexpr int norm_n(int mode) {
    return mode == kBy32Quarter ? 4 : mode == kBy32Half ? 8 : 16;
}
__host__ __device__ constexpr int norm_stride(int mode) { return mode > kBy32 ? 32 : mode; }
template <int MODE>
__device__ __forceinline__ int norm_col(int g, int k) {
    if constexpr (MODE == kVec) return g * 16 + k;
    if constexpr (MODE == kBy4 || MODE == kBy8) return g + MODE * k;
    return (g >> 5) * 512 + (g & 31) + 32 * k;
}

__device__ __forceinline__ void ld_global_v8(const void* p, uint32_t* w) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Sixteen channels as loaded, kept apart from their conversion so that a row can
// be on its way while the one before it is worked on.  Channels that do not exist
// (past C, or of a row that does not exist) read as 0.
template <typename T, int MODE>
struct NormRow {
    uint32_t w[MODE == kVec && sizeof(T) == 2 ? 8 : norm_n(MODE)];
    __device__ __forceinline__ void load(const void* base, int64_t off, bool ok, int g, int G, int C) {
        const T* row = static_cast<const T*>(base) + off;
        if constexpr (MODE == kVec) {
            if (ok && g * 16 < C) {
                ld_global_v8(row + g * 16, w);
                if constexpr (sizeof(T) == 4) ld_global_v8(row + g * 16 + 8, w + 8);
            } else {
#pragma unroll
                for (uint32_t& x : w) x = 0u;
            }
        } else {
#pragma unroll
            for (int k = 0; k < norm_n(MODE); ++k) {
                const int c = norm_col<MODE>(g, k);
                w[k] = 0u;
                if (ok && c < C) {
                    if constexpr (sizeof(T) == 2)
                        w[k] = static_cast<uint32_t>(__bfloat16_as_ushort(row[c])) << 16;
                    else
                        w[k] = __float_as_uint(row[c]);
                }
            }
        }
    }
    __device__ __forceinline__ void values(float2 (&v)[norm_n(MODE) / 2]) const {
#pragma unroll
        for (int k = 0; k < norm_n(MODE) / 2; ++k) {
            if constexpr (MODE == kVec && sizeof(T) == 2)
                v[k] = bf16x2_to_f2(w[k]);
            else
                v[k] = make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        }
    }
};

template <typename T, int MODE>
__device__ __forceinline__ void store16(void* base, int64_t off, bool ok, int g, int G, int C,
                                        const float2 (&v)[norm_n(MODE) / 2]) {
    T* row = static_cast<T*>(base) + off;
    if constexpr (MODE == kVec) {
        if (ok && g * 16 < C) {
            uint32_t w[16];
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = pack_bf16(v[k].x, v[k].y);
                st_global_v8(row + g * 16, w);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    w[2 * k] = __float_as_uint(v[k].x);
                    w[2 * k + 1] = __float_as_uint(v[k].y);
                }
                st_global_v8(row + g * 16, w);
                st_global_v8(row + g * 16 + 8, w + 8);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < norm_n(MODE); ++k) {
            const int c = norm_col<MODE>(g, k);
            if (ok && c < C) row[c] = from_f32<T>(k & 1 ? v[k / 2].y : v[k / 2].x);
        }
    }
}

// w or b, `absent` where there is none: for a block's rows in shared memory, in
// the order in which the lanes read it without bank conflicts (VEC: the q-th four
// channels of lane g at 4 (q G + g), else channel c at c); for rows as wide as a
// block, in the registers of the one thread that needs it
__device__ __forceinline__ float norm_param(const void* p, int is_bf16, float absent, int c, int C) {
    if (!p || c >= C) return absent;
    return is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]) : static_cast<const float*>(p)[c];
}
template <int MODE, bool WIDE>
struct NormParam {
    float2 own[WIDE ? norm_n(MODE) / 2 : 1];
    const float* sh;
    __device__ __forceinline__ void init(const void* p, int is_bf16, float absent, int g, int G, int C, float* shared) {
        sh = shared;
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < norm_n(MODE) / 2; ++k)
                own[k] = make_float2(norm_param(p, is_bf16, absent, norm_col<MODE>(g, 2 * k), C),
                                     norm_param(p, is_bf16, absent, norm_col<MODE>(g, 2 * k + 1), C));
        } else {
            for (int x = threadIdx.x; x < norm_n(MODE) * G; x += blockDim.x) {
                const int lane = (x >> 2) & (G - 1), q = (x >> 2) / G;
                shared[x] = norm_param(p, is_bf16, absent, MODE == kVec ? lane * 16 + q * 4 + (x & 3) : x, C);
            }
        }
    }
    // channels 4 q .. 4 q + 3 of this lane
    __device__ __forceinline__ void get4(int q, int g, int G, float2& a, float2& b) const {
        if constexpr (WIDE) {
            a = own[2 * q];
            b = own[2 * q + 1];
        } else if constexpr (MODE == kVec) {
            const float4 v = *reinterpret_cast<const float4*>(sh + 4 * (q * G + g));
            a = make_float2(v.x, v.y);
            b = make_float2(v.z, v.w);
        } else {
            const float* s = sh + norm_col<MODE>(g, 4 * q);
            constexpr int kStride = norm_stride(MODE);
            a = make_float2(s[0], s[kStride]);
            b = make_float2(s[2 * kStride], s[3 * kStride]);
        }
    }
};

// ---------------------------------------------------------------------------
// the 8-bit form
// ---------------------------------------------------------------------------
// exponent byte of a block whose largest magnitude has the bits `amax`: the
// mantissa of Q (127 = 1.984375 x 2^6, 448 = 1.75 x 2^8) decides by a carry
// whether the next power of two is needed; 255 marks an infinity or NaN
template <int ACT>
__device__ __forceinline__ uint32_t act8_exp(uint32_t amax) {
    constexpr uint32_t kCarry = ACT == ACT_INT8 ? 0x7FFFFFu - 0x7E0000u : 0x7FFFFFu - 0x600000u;
    constexpr int kTop = ACT == ACT_INT8 ? 6 : 8;
    const int e = static_cast<int>((amax + kCarry) >> 23) - kTop;  // biased by 127
    return amax >= 0x7F800000u ? 255u : static_cast<uint32_t>(max(e, 1));
}
// 2^-e for an exponent byte (1 .. 249)
__device__ __forceinline__ float act8_inv(uint32_t eb) { return __uint_as_float((254u - eb) << 23); }
// 2^e; byte 255 gives infinity, which turns the code 0 into NaN
__device__ __forceinline__ float act8_scale(uint32_t eb) { return __uint_as_float(eb << 23); }

// two codes, a in the low byte
template <int ACT>
__device__ __forceinline__ uint32_t act8_code2(float a, float b, float inv) {
    if constexpr (ACT == ACT_INT8) {
        // adding 1.5 x 2^23 leaves the nearest integer (ties to even) in the low bits
        const float m = 12582912.f;
        const uint32_t lo = __float_as_uint(fmaf(a, inv, m)), hi = __float_as_uint(fmaf(b, inv, m));
        return __byte_perm(lo, hi, 0x0040) & 0xFFFFu;
    } else {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b * inv), "f"(a * inv));
        return r;
    }
}
template <int ACT>
__device__ __forceinline__ float act8_value(uint32_t byte) {
    if constexpr (ACT == ACT_INT8) {
        return static_cast<float>(static_cast<int8_t>(byte));
    } else {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
        return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xFFFFu)));
    }
}

// values of four codes in a word, times the scale
template <int ACT>
__device__ __forceinline__ void act8_value4(uint32_t w, float scale, float2* v) {
    const float2 s = make_float2(scale, scale);
    if constexpr (ACT == ACT_INT8) {
        // byte b of (w ^ 0x80808080) in the low bits of 2^23 is 2^23 + 128 + code
        const uint32_t u = w ^ 0x80808080u;
        const float2 off = make_float2(-8388736.f, -8388736.f);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = fmul2(fadd2(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u + 2 * k)),
                                           __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441u + 2 * k))),
                               off),
                         s);
    } else {
        uint32_t h0, h1;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
        v[0] = fmul2(__half22float2(*reinterpret_cast<__half2*>(&h0)), s);
        v[1] = fmul2(__half22float2(*reinterpret_cast<__half2*>(&h1)), s);
    }
}
// four codes in a word
template <int ACT>
__device__ __forceinline__ uint32_t act8_code4(float2 a, float2 b, float inv) {
    const float2 s = make_float2(inv, inv);
    if constexpr (ACT == ACT_INT8) {
        const float2 m = make_float2(12582912.f, 12582912.f);  // as in act8_code2
        a = ffma2(a, s, m);
        b = ffma2(b, s, m);
        const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        return act8_code2<ACT>(a.x, a.y, inv) | act8_code2<ACT>(b.x, b.y, inv) << 16;
    }
}
// the larger magnitude of three; a NaN stays one
__device__ __forceinline__ float absmax3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// this lane's sixteen channels, from channel c0 of their row on, into its 8-bit form; every lane of
// the warp calls it
template <int ACT, int MODE>
__device__ __forceinline__ void act8_emit(const NormParams& p, int64_t row, bool ok, int g, int G,
                                          const float2 (&u)[norm_n(MODE) / 2], int c0 = 0) {
    const int C = p.C - c0;
    uint8_t* codes = p.codes + row * p.cs + c0;
    uint8_t* exps = p.exps + row * p.es + c0 / 32;
    if constexpr (MODE == kVec) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = absmax3(m, u[k].x, u[k].y);
        uint32_t a = __float_as_uint(m) & 0x7FFFFFFFu;
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, a, 1);
        if (G > 1) a = max(a, other);  // two lanes share a block (C = 16: one lane is the row)
        const uint32_t eb = act8_exp<ACT>(a);
        const float inv = act8_inv(eb);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = act8_code4<ACT>(u[2 * q], u[2 * q + 1], inv);
            if (eb == 255u) w[q] = 0u;
        }
        if (ok && g * 16 < C) {
            *reinterpret_cast<uint4*>(codes + g * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            if ((g & 1) == 0) exps[g >> 1] = static_cast<uint8_t>(eb);
        }
    } else {
        constexpr int N = norm_n(MODE);
        float v[N];
        uint32_t a[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = k & 1 ? u[k / 2].y : u[k / 2].x;
#pragma unroll
        for (int k = 0; k < N; ++k) a[k] = __float_as_uint(v[k]) & 0x7FFFFFFFu;
        if constexpr (norm_stride(MODE) == 32) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (32 * k < p.C) a[k] = __reduce_max_sync(0xFFFFFFFFu, a[k]);
        } else {  // a block is several k of the row's lanes
            constexpr int kPer = 32 / norm_stride(MODE);
#pragma unroll
            for (int s = 0; s < N; s += kPer) {
#pragma unroll
                for (int k = 1; k < kPer; ++k) a[s] = max(a[s], a[s + k]);
#pragma unroll
                for (int m = 1; m < norm_stride(MODE); m *= 2) a[s] = max(a[s], __shfl_xor_sync(0xFFFFFFFFu, a[s], m));
#pragma unroll
                for (int k = 1; k < kPer; ++k) a[s + k] = a[s];
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = norm_col<MODE>(g, k);
            if (ok && c < C) {
                const uint32_t eb = act8_exp<ACT>(a[k]);
                const uint32_t code = eb == 255u ? 0u : act8_code2<ACT>(v[k], 0.f, act8_inv(eb));
                codes[c] = static_cast<uint8_t>(code);
                if ((c & 31) == 0) exps[c >> 5] = static_cast<uint8_t>(eb);
            }
        }
    }
}

// sixteen channels of the 8-bit form of a row, as loaded
template <int ACT, int MODE>
struct NormRow8 {
    uint32_t w[MODE == kVec ? 4 : norm_n(MODE)], e[MODE == kVec ? 1 : norm_n(MODE)];
    __device__ __forceinline__ void load(const NormParams& p, int64_t row, bool ok, int g, int G, int c0 = 0) {
        const int C = p.C - c0;
        const uint8_t* codes = p.codes + row * p.cs + c0;
        const uint8_t* exps = p.exps + row * p.es + c0 / 32;
        if constexpr (MODE == kVec) {
            w[0] = w[1] = w[2] = w[3] = e[0] = 0u;
            if (ok && g * 16 < C) {
                const uint4 c = *reinterpret_cast<const uint4*>(codes + g * 16);
                w[0] = c.x;
                w[1] = c.y;
                w[2] = c.z;
                w[3] = c.w;
                e[0] = exps[g >> 1];
            }
        } else {
#pragma unroll
            for (int k = 0; k < norm_n(MODE); ++k) {
                const int c = norm_col<MODE>(g, k);
                w[k] = e[k] = 0u;
                if (ok && c < C) {
                    w[k] = codes[c];
                    e[k] = exps[c >> 5];
                }
            }
        }
    }
    __device__ __forceinline__ void values(float2 (&v)[norm_n(MODE) / 2]) const {
        if constexpr (MODE == kVec) {
            const float s = act8_scale(e[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) act8_value4<ACT>(w[q], s, v + 2 * q);
        } else {
#pragma unroll
            for (int k = 0; k < norm_n(MODE) / 2; ++k)
                v[k] = make_float2(act8_value<ACT>(w[2 * k]) * act8_scale(e[2 * k]),
                                   act8_value<ACT>(w[2 * k + 1]) * act8_scale(e[2 * k + 1]));
        }
    }
};

// ---------------------------------------------------------------------------
// sums over the lanes of a row
//
// While the device error word is set the kernels here compute as usual but
// store nothing: a launch that returned early in some threads only (the word
// can be set while it starts) would leave others waiting at a barrier.
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;   // rows of up to 512 channels: 256 / G of them per block
constexpr int kNormMaxWarps = 16;   // rows of up to 8192 channels: one block, a warp per 512
// Blocks per SM.  A row on its way takes eight registers in BF16 and sixteen in FP32 or element by
// element, so those get the registers of a block less.  The 8-bit form beside it does not fit the 80
// registers that kBy32 has then and spills 80 to 88 bytes.  Two blocks without spills do better from
// FP32 (100000 rows of 387 with the int8 form 93 us in place of 110) and worse from BF16 (151 and
// 126) and without the 8-bit form (60 and 52; BF16 111 and 78).
__host__ __device__ constexpr int norm_fwd_blocks(int mode, bool f32) {
    return mode == kBy32Quarter ? 5 : mode == kBy32Half || (mode == kVec && !f32) ? 4 : 3;
}
__host__ __device__ constexpr int norm_bwd_per_sm(int mode) { return mode == kBy32Quarter ? 4 : mode == kBy32Half ? 3 : 2; }

// Sums over the G lanes of this lane's row, the same bits in every lane.  Rows
// of more than one warp meet in shared memory; `turn` alternates between two
// buffers, so one barrier per sum is enough.
template <bool WIDE>
__device__ __forceinline__ float2 row_sum2(float2 v, int G, float2 (*red)[kNormMaxWarps], int& turn) {
    for (int m = 1; m < 32 && m < G; m <<= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, m);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, m);
    }
    if constexpr (WIDE) {
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[turn][0];
        for (int w = 1; w < G / 32; ++w) {
            v.x += red[turn][w].x;
            v.y += red[turn][w].y;
        }
        turn ^= 1;
    }
    return v;
}
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, int G, float2 (*red)[kNormMaxWarps], int& turn) {
    if constexpr (WIDE) {
        return row_sum2<true>(make_float2(v, 0.f), G, red, turn).x;
    } else {
        for (int m = 1; m < 32 && m < G; m <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
        return v;
    }
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// ---------------------------------------------------------------------------
// forward; with RESTORE the row comes from its 8-bit form and its statistics
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int ACT, int MODE, bool RESTORE, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 32 * kNormMaxWarps : kNormThreads,
                                  WIDE ? 1 : norm_fwd_blocks(MODE, sizeof(TX) == 4 && !RESTORE))
    tri_norm_fwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 red[2][kNormMaxWarps];
    __shared__ __align__(16) float sh_w[WIDE ? 4 : 512], sh_b[WIDE ? 4 : 512];
    const bool dead = device_error_pending();
    constexpr int N = norm_n(MODE), N2 = N / 2;  // channels and pairs of them per lane
    const int G = MODE == kVec || WIDE ? p.lanes : norm_stride(MODE);
    const int g = WIDE ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (G - 1);
    const int per_block = WIDE ? 1 : kNormThreads / G, sub = WIDE ? 0 : threadIdx.x / G;
    int turn = 0;
    NormParam<MODE, WIDE> w, b;
    w.init(p.w, p.w_bf16, 1.f, g, G, p.C, sh_w);
    b.init(p.b, p.w_bf16, 0.f, g, G, p.C, sh_b);
    NormRow<TX, MODE> next;
    NormRow8<ACT, MODE> next8;
    float mean = 0.f, rstd = 0.f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
    int64_t base = static_cast<int64_t>(blockIdx.x) * per_block;
    // rows are loaded one round ahead, but for 8-bit rows byte by byte, whose 32 loads do not fit
    constexpr bool kAhead = MODE == kVec || !RESTORE;
    const auto load = [&](int64_t row) {
        if constexpr (RESTORE) {
            const bool ok = row < p.R;
            next8.load(p, row, ok, g, G);
            mean = ok ? p.stats[row] : 0.f;
            rstd = ok ? p.stats[p.R + row] : 0.f;
        } else {
            next.load(p.x, row * p.xs, row < p.R, g, G, p.C);
        }
    };
    if constexpr (kAhead) load(base + sub);
    if constexpr (!WIDE) __syncthreads();
    // the loop runs for whole blocks: rows past R are computed on zeros and not stored
    for (; base < p.R; base += step) {
        const int64_t row = base + sub;
        const bool st = row < p.R && !dead;
        float2 v[N2];
        if constexpr (RESTORE) {
            if constexpr (!kAhead) load(row);
            next8.values(v);
            const float m = mean, r = rstd;
            if constexpr (kAhead) load(row + step);
#pragma unroll
            for (int k = 0; k < N2; ++k) v[k] = fmul2(fadd2(v[k], splat(-m)), splat(r));
        } else {
            next.values(v);
            load(row + step);
            if constexpr (ACT != ACT_NONE) act8_emit<ACT, MODE>(p, row, st, g, G, v);
            float2 s = fadd2(v[0], v[1]);
#pragma unroll
            for (int k = 2; k < N2; ++k) s = fadd2(s, v[k]);
            mean = row_sum<WIDE>(s.x + s.y, G, red, turn) * p.inv_c;
            s = splat(0.f);
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                v[k] = fadd2(v[k], splat(-mean));
                if constexpr (MODE != kVec) {
                    if (norm_col<MODE>(g, 2 * k) >= p.C) v[k].x = 0.f;
                    if (norm_col<MODE>(g, 2 * k + 1) >= p.C) v[k].y = 0.f;
                }
                s = ffma2(v[k], v[k], s);
            }
            const float own = MODE != kVec || g * 16 < p.C ? s.x + s.y : 0.f;
            rstd = rsqrtf(fmaf(row_sum<WIDE>(own, G, red, turn), p.inv_c, p.eps));
            if (st && g == 0) {
                p.stats[row] = mean;
                p.stats[p.R + row] = rstd;
            }
#pragma unroll
            for (int k = 0; k < N2; ++k) v[k] = fmul2(v[k], splat(rstd));
        }
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            float2 wa, wb, ba, bb;
            w.get4(q, g, G, wa, wb);
            b.get4(q, g, G, ba, bb);
            v[2 * q] = ffma2(v[2 * q], wa, ba);
            v[2 * q + 1] = ffma2(v[2 * q + 1], wb, bb);
        }
        store16<TY, MODE>(p.y, row * p.ys, st, g, G, p.C, v);
    }
}

// A kernel launched with programmatic stream serialisation starts while the one
// before it still runs: grid_dependents_start there allows it (all its blocks have
// begun), grid_dependency_wait here returns once that kernel has ended and its
// writes are visible.
__device__ __forceinline__ void grid_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------------------
// backward: dx row by row, dw and db summed in registers over the block's rows
// ---------------------------------------------------------------------------
// The block's share of dw and db leaves as one partial sum; the shares are
// added in block order by tri_ordered_sum_kernel.  The number of blocks is a
// function of the sizes alone, and so is every order of additions.
template <typename TX, typename TY, int ACT, int MODE, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 32 * kNormMaxWarps : kNormThreads, WIDE ? 1 : norm_bwd_per_sm(MODE))
    tri_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 red[2][kNormMaxWarps];
    __shared__ __align__(16) float sums[WIDE ? 1 : kNormThreads / 32][2][WIDE ? 1 : 512];
    __shared__ __align__(16) float sh_w[WIDE ? 4 : 512];
    grid_dependents_start();
    const bool dead = device_error_pending();
    constexpr int N = norm_n(MODE), N2 = N / 2;  // channels and pairs of them per lane
    const int G = MODE == kVec || WIDE ? p.lanes : norm_stride(MODE);
    const int g = WIDE ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (G - 1);
    const int per_block = WIDE ? 1 : kNormThreads / G, sub = WIDE ? 0 : threadIdx.x / G;
    int turn = 0;
    NormParam<MODE, WIDE> w;
    w.init(p.w, p.w_bf16, 1.f, g, G, p.C, sh_w);
    float2 dw[N2], db[N2];
#pragma unroll
    for (int k = 0; k < N2; ++k) dw[k] = db[k] = splat(0.f);
    NormRow<TX, MODE> nx;
    NormRow8<ACT, MODE> nx8;
    NormRow<TY, MODE> nd;
    float mean, rstd;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
    int64_t base = static_cast<int64_t>(blockIdx.x) * per_block;
    constexpr bool kAhead = MODE == kVec || ACT == ACT_NONE;
    const auto load = [&](int64_t row) {
        const bool ok = row < p.R;
        if constexpr (ACT != ACT_NONE)
            nx8.load(p, row, ok, g, G);
        else
            nx.load(p.x, row * p.xs, ok, g, G, p.C);
        nd.load(p.dy, row * p.dys, ok, g, G, p.C);
        mean = ok ? p.stats[row] : 0.f;
        rstd = ok ? p.stats[p.R + row] : 0.f;
    };
    if constexpr (kAhead) load(base + sub);
    if constexpr (!WIDE) __syncthreads();
    for (; base < p.R; base += step) {
        const int64_t row = base + sub;
        const bool st = row < p.R && !dead;
        float2 h[N2], d[N2];
        if constexpr (!kAhead) load(row);
        if constexpr (ACT != ACT_NONE)
            nx8.values(h);
        else
            nx.values(h);
        nd.values(d);
        const float m = mean, r = rstd;
        if constexpr (kAhead) load(row + step);
        float2 sa = splat(0.f), sb = splat(0.f);
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            float2 ww[2];
            w.get4(q, g, G, ww[0], ww[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int k = 2 * q + x;
                h[k] = fmul2(fadd2(h[k], splat(-m)), splat(r));
                dw[k] = ffma2(d[k], h[k], dw[k]);
                db[k] = fadd2(db[k], d[k]);
                d[k] = fmul2(d[k], ww[x]);
                sa = fadd2(sa, d[k]);
                sb = ffma2(d[k], h[k], sb);
            }
        }
        if (p.dx) {
            const float2 s = row_sum2<WIDE>(make_float2(sa.x + sa.y, sb.x + sb.y), G, red, turn);
            const float2 c1 = splat(s.x * p.inv_c), c2 = splat(-s.y * p.inv_c);
            const float2 n1 = make_float2(-c1.x, -c1.y);
#pragma unroll
            for (int k = 0; k < N2; ++k) d[k] = fmul2(fadd2(d[k], ffma2(h[k], c2, n1)), splat(r));
            store16<TX, MODE>(p.dx, row * p.dxs, st, g, G, p.C, d);
        }
    }
    if (!p.partial) return;  // the same for every thread
    float* out_w = gridDim.x == 1 ? p.dw : p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.C;
    float* out_b = gridDim.x == 1 ? p.db : out_w + p.C;
    if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = norm_col<MODE>(g, k);
            if (c < p.C && !dead) {
                out_w[c] = k & 1 ? dw[k / 2].y : dw[k / 2].x;
                out_b[c] = k & 1 ? db[k / 2].y : db[k / 2].x;
            }
        }
    } else {
        // the rows of a warp, then the warps of the block
        for (int m = G; m < 32; m <<= 1) {
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                dw[k].x += __shfl_xor_sync(0xFFFFFFFFu, dw[k].x, m);
                dw[k].y += __shfl_xor_sync(0xFFFFFFFFu, dw[k].y, m);
                db[k].x += __shfl_xor_sync(0xFFFFFFFFu, db[k].x, m);
                db[k].y += __shfl_xor_sync(0xFFFFFFFFu, db[k].y, m);
            }
        }
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) < G) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                sums[warp][0][norm_col<MODE>(g, k)] = k & 1 ? dw[k / 2].y : dw[k / 2].x;
                sums[warp][1][norm_col<MODE>(g, k)] = k & 1 ? db[k / 2].y : db[k / 2].x;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) {
            const int which = c >= p.C, col = c - which * p.C;
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kNormThreads / 32; ++q) s += sums[q][which][col];
            if (!dead) (which ? out_b : out_w)[col] = s;
        }
    }
}

// out[i] = sum over q < nparts of part[q][i], i < n: the first n0 of them into
// out0, the rest into out1.  32 columns by 32 runs of q per block; each run is
// added in ascending q, the runs in ascending order.  part is written while this
// kernel runs, up to the wait: no __restrict__, which would promise that it does not
// change and let its loads pass the wait.
__global__ void __launch_bounds__(1024) tri_ordered_sum_kernel(const float* part, int nparts, int n, float* out0,
                                                               int n0, float* out1) {
    __shared__ float runs[32][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    grid_dependency_wait();
    const bool dead = device_error_pending();
    if (i < n)
        for (int q = run; q < nparts; q += 32) s += part[static_cast<int64_t>(q) * n + i];
    runs[run][lane] = s;
    __syncthreads();
    if (run == 0 && i < n && !dead) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 32; ++q) s += runs[q][lane];
        if (i < n0)
            out0[i] = s;
        else
            out1[i - n0] = s;
    }
}

// ---------------------------------------------------------------------------
// an activation into and out of its 8-bit form
// ---------------------------------------------------------------------------
// The lanes share a row as in the norm; rows of more than 512 channels are cut
// into pieces of 512, a warp each.  What hides the latency here is many warps: with
// a row loaded ahead, for which two blocks per SM less fit, 640 x 640 rows of 128
// BF16 channels packed in 36 us instead of 31 (5.2 TB/s; unpacking 27 us, 5.9 TB/s).
// Element by element, 20011 rows of 209 FP32 channels take 10.5 and 7.5 us, bound
// by their instructions.
__host__ __device__ constexpr int act8_blocks(int mode) { return mode == kVec ? 6 : 4; }  // per SM
template <typename TX, int ACT, int MODE, bool PACK>
__global__ void __launch_bounds__(kNormThreads, act8_blocks(MODE))
    tri_act8_kernel(const __grid_constant__ NormParams p) {
    const bool dead = device_error_pending();
    const int G = MODE == kVec ? p.lanes : norm_stride(MODE);
    const int g = static_cast<int>(threadIdx.x) & (G - 1), per_block = kNormThreads / G;
    const int pieces = (p.C + 511) / 512;
    const int64_t items = p.R * pieces, step = static_cast<int64_t>(gridDim.x) * per_block;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * per_block; base < items; base += step) {
        const int64_t item = base + threadIdx.x / G;
        const bool ok = item < items;
        int64_t row = item;
        int c0 = 0;
        if (pieces > 1) {
            row = item / pieces;
            c0 = static_cast<int>(item - row * pieces) * 512;
        }
        // a piece ends where the next one begins: the lanes cover no more than 512 channels
        float2 v[norm_n(MODE) / 2];
        if constexpr (PACK) {
            NormRow<TX, MODE> r;
            r.load(p.x, row * p.xs + c0, ok, g, G, p.C - c0);
            r.values(v);
            act8_emit<ACT, MODE>(p, row, ok && !dead, g, G, v, c0);
        } else {
            NormRow8<ACT, MODE> r;
            r.load(p, row, ok, g, G, c0);
            r.values(v);
            store16<TX, MODE>(p.y, row * p.ys + c0, ok && !dead, g, G, p.C - c0, v);
        }
    }
}

}  // namespace tri
