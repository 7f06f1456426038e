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
    float* partial;  // [gridDim.x][2][C], or NULL
};

// ---------------------------------------------------------------------------
// sixteen channels of a row
// ---------------------------------------------------------------------------
// The channels lane g of a row's G lanes owns: 16 g .. 16 g + 15 when the row
// can be moved in aligned vectors (VEC), else g, g + G, g + 2 G, ... so that
// neighbouring lanes still touch neighbouring elements.
template <bool VEC>
__device__ __forceinline__ int norm_col(int g, int G, int k) {
    return VEC ? g * 16 + k : g + G * k;
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

// channels that do not exist (past C, or of a row that does not exist) read as 0
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const void* base, int64_t off, bool ok, int g, int G, int C, float (&v)[16]) {
    const T* row = static_cast<const T*>(base) + off;
    if constexpr (VEC) {
        if (ok && g * 16 < C) {
            if constexpr (sizeof(T) == 2) {
                uint32_t w[8];
                ld_global_v8(row + g * 16, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[2 * k] = bf16lo(w[k]);
                    v[2 * k + 1] = bf16hi(w[k]);
                }
            } else {
                uint32_t w[16];
                ld_global_v8(row + g * 16, w);
                ld_global_v8(row + g * 16 + 8, w + 8);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(w[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int c = norm_col<VEC>(g, G, k);
            v[k] = ok && c < C ? to_f32(row[c]) : 0.f;
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store16(void* base, int64_t off, bool ok, int g, int G, int C, const float (&v)[16]) {
    T* row = static_cast<T*>(base) + off;
    if constexpr (VEC) {
        if (ok && g * 16 < C) {
            uint32_t w[16];
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
                st_global_v8(row + g * 16, w);
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(v[k]);
                st_global_v8(row + g * 16, w);
                st_global_v8(row + g * 16 + 8, w + 8);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int c = norm_col<VEC>(g, G, k);
            if (ok && c < C) row[c] = from_f32<T>(v[k]);
        }
    }
}

// w or b for this lane's channels, `absent` where there is none
template <bool VEC>
__device__ __forceinline__ void load_param16(const void* p, int is_bf16, float absent, int g, int G, int C,
                                             float (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int c = norm_col<VEC>(g, G, k);
        v[k] = absent;
        if (p && c < C)
            v[k] = is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]) : static_cast<const float*>(p)[c];
    }
}

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
__device__ __forceinline__ void act8_value4(uint32_t w, float scale, float* v) {
    if constexpr (ACT == ACT_INT8) {
        // byte b of (w ^ 0x80808080) in the low bits of 2^23 is 2^23 + 128 + code
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u + k)) - 8388736.f) * scale;
    } else {
        uint32_t h0, h1;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
        const float2 a = __half22float2(*reinterpret_cast<__half2*>(&h0));
        const float2 b = __half22float2(*reinterpret_cast<__half2*>(&h1));
        v[0] = a.x * scale;
        v[1] = a.y * scale;
        v[2] = b.x * scale;
        v[3] = b.y * scale;
    }
}

// this lane's sixteen channels into the 8-bit form of their row; every lane of the warp calls it
template <int ACT, bool VEC>
__device__ __forceinline__ void act8_emit(const NormParams& p, int64_t row, bool ok, int g, int G, const float (&v)[16]) {
    if constexpr (VEC) {
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) a = max(a, __float_as_uint(v[k]) & 0x7FFFFFFFu);
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, a, 1);
        if (G > 1) a = max(a, other);  // two lanes share a block (C = 16: one lane is the row)
        const uint32_t eb = act8_exp<ACT>(a);
        const float inv = act8_inv(eb);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = act8_code2<ACT>(v[4 * q], v[4 * q + 1], inv) | act8_code2<ACT>(v[4 * q + 2], v[4 * q + 3], inv) << 16;
            if (eb == 255u) w[q] = 0u;
        }
        if (ok && g * 16 < p.C) {
            *reinterpret_cast<uint4*>(p.codes + row * p.cs + g * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            if ((g & 1) == 0) p.exps[row * p.es + (g >> 1)] = static_cast<uint8_t>(eb);
        }
    } else {
        uint32_t a[16];
        const int per = G >= 32 ? 1 : 32 / G;  // consecutive k of one block
#pragma unroll
        for (int k = 0; k < 16; ++k) a[k] = __float_as_uint(v[k]) & 0x7FFFFFFFu;
#pragma unroll
        for (int s = 1; s < 16; s <<= 1)
            if (s < per) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if ((k & s) == 0) a[k] = a[k + s] = max(a[k], a[k + s]);
            }
        for (int m = 1; m < 32 && m < G; m <<= 1) {
#pragma unroll
            for (int k = 0; k < 16; ++k) a[k] = max(a[k], __shfl_xor_sync(0xFFFFFFFFu, a[k], m));
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int c = norm_col<VEC>(g, G, k);
            if (ok && c < p.C) {
                const uint32_t eb = act8_exp<ACT>(a[k]);
                const uint32_t code = eb == 255u ? 0u : act8_code2<ACT>(v[k], 0.f, act8_inv(eb));
                p.codes[row * p.cs + c] = static_cast<uint8_t>(code);
                if ((c & 31) == 0) p.exps[row * p.es + (c >> 5)] = static_cast<uint8_t>(eb);
            }
        }
    }
}

// the values the 8-bit form of a row stands for
template <int ACT, bool VEC>
__device__ __forceinline__ void act8_load16(const NormParams& p, int64_t row, bool ok, int g, int G, float (&v)[16]) {
    if constexpr (VEC) {
        if (ok && g * 16 < p.C) {
            const uint4 w = *reinterpret_cast<const uint4*>(p.codes + row * p.cs + g * 16);
            const float s = act8_scale(p.exps[row * p.es + (g >> 1)]);
            act8_value4<ACT>(w.x, s, v);
            act8_value4<ACT>(w.y, s, v + 4);
            act8_value4<ACT>(w.z, s, v + 8);
            act8_value4<ACT>(w.w, s, v + 12);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int c = norm_col<VEC>(g, G, k);
            v[k] = ok && c < p.C ? act8_value<ACT>(p.codes[row * p.cs + c]) * act8_scale(p.exps[row * p.es + (c >> 5)])
                                 : 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// sums over the lanes of a row
//
// While the device error word is set the kernels here compute as usual but
// store nothing: a launch that returned early in some threads only (the word
// can be set while it starts) would leave others waiting at a barrier.
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;   // rows of up to 512 channels: 256 / G of them per block
constexpr int kNormMaxWarps = 16;   // rows of up to 8192 channels: one block, a warp per 512

// Sums over the G lanes of this lane's row, the same bits in every lane.  Rows
// of more than one warp meet in shared memory; `turn` alternates between two
// buffers, so one barrier per sum is enough.
__device__ __forceinline__ float2 row_sum2(float2 v, int G, float2 (*red)[kNormMaxWarps], int& turn) {
    for (int m = 1; m < 32 && m < G; m <<= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, m);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, m);
    }
    if (G > 32) {
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

// ---------------------------------------------------------------------------
// forward; with RESTORE the row comes from its 8-bit form and its statistics
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int ACT, bool VEC, bool RESTORE>
__global__ void __launch_bounds__(512) tri_norm_fwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 red[2][kNormMaxWarps];
    const bool dead = device_error_pending();
    const int G = p.lanes;
    const int g = G > 32 ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (G - 1);
    const int per_block = blockDim.x / G, sub = threadIdx.x / G;
    int turn = 0;
    float w[16], b[16];
    load_param16<VEC>(p.w, p.w_bf16, 1.f, g, G, p.C, w);
    load_param16<VEC>(p.b, p.w_bf16, 0.f, g, G, p.C, b);
    // the loop runs for whole blocks: rows past R are computed on zeros and not stored
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * per_block; base < p.R;
         base += static_cast<int64_t>(gridDim.x) * per_block) {
        const int64_t row = base + sub;
        const bool ok = row < p.R, st = ok && !dead;
        float v[16], mean, rstd;
        if constexpr (RESTORE) {
            act8_load16<ACT, VEC>(p, row, ok, g, G, v);
            mean = ok ? p.stats[row] : 0.f;
            rstd = ok ? p.stats[p.R + row] : 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] -= mean;
        } else {
            load16<TX, VEC>(p.x, row * p.xs, ok, g, G, p.C, v);
            if constexpr (ACT != ACT_NONE) act8_emit<ACT, VEC>(p, row, st, g, G, v);
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) s += v[k];
            mean = row_sum2(make_float2(s, 0.f), G, red, turn).x * p.inv_c;
            s = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                v[k] = norm_col<VEC>(g, G, k) < p.C ? v[k] - mean : 0.f;
                s = fmaf(v[k], v[k], s);
            }
            rstd = rsqrtf(fmaf(row_sum2(make_float2(s, 0.f), G, red, turn).x, p.inv_c, p.eps));
            if (st && g == 0) {
                p.stats[row] = mean;
                p.stats[p.R + row] = rstd;
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = fmaf(v[k] * rstd, w[k], b[k]);
        store16<TY, VEC>(p.y, row * p.ys, st, g, G, p.C, v);
    }
}

// ---------------------------------------------------------------------------
// backward: dx row by row, dw and db summed in registers over the block's rows
// ---------------------------------------------------------------------------
// The block's share of dw and db leaves as one partial sum; the shares are
// added in block order by tri_ordered_sum_kernel.  The number of blocks is a
// function of the sizes alone, and so is every order of additions.
template <typename TX, typename TY, int ACT, bool VEC>
__global__ void __launch_bounds__(512) tri_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 red[2][kNormMaxWarps];
    __shared__ float sums[kNormThreads / 32][2][512];
    const bool dead = device_error_pending();
    const int G = p.lanes;
    const int g = G > 32 ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (G - 1);
    const int per_block = blockDim.x / G, sub = threadIdx.x / G;
    int turn = 0;
    float w[16], dw[16], db[16];
    load_param16<VEC>(p.w, p.w_bf16, 1.f, g, G, p.C, w);
#pragma unroll
    for (int k = 0; k < 16; ++k) dw[k] = db[k] = 0.f;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * per_block; base < p.R;
         base += static_cast<int64_t>(gridDim.x) * per_block) {
        const int64_t row = base + sub;
        const bool ok = row < p.R, st = ok && !dead;
        float h[16], d[16];
        if constexpr (ACT != ACT_NONE)
            act8_load16<ACT, VEC>(p, row, ok, g, G, h);
        else
            load16<TX, VEC>(p.x, row * p.xs, ok, g, G, p.C, h);
        load16<TY, VEC>(p.dy, row * p.dys, ok, g, G, p.C, d);
        const float mean = ok ? p.stats[row] : 0.f, rstd = ok ? p.stats[p.R + row] : 0.f;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            h[k] = (h[k] - mean) * rstd;
            dw[k] = fmaf(d[k], h[k], dw[k]);
            db[k] += d[k];
            d[k] *= w[k];
            s.x += d[k];
            s.y = fmaf(d[k], h[k], s.y);
        }
        if (p.dx) {
            s = row_sum2(s, G, red, turn);
            const float c1 = s.x * p.inv_c, c2 = s.y * p.inv_c;
#pragma unroll
            for (int k = 0; k < 16; ++k) d[k] = rstd * (d[k] - fmaf(h[k], c2, c1));
            store16<TX, VEC>(p.dx, row * p.dxs, st, g, G, p.C, d);
        }
    }
    if (!p.partial) return;  // the same for every thread
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.C;
    if (G > 32) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int c = norm_col<VEC>(g, G, k);
            if (c < p.C && !dead) {
                out[c] = dw[k];
                out[p.C + c] = db[k];
            }
        }
        return;
    }
    // the rows of a warp, then the warps of the block
    for (int m = G; m < 32; m <<= 1) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            dw[k] += __shfl_xor_sync(0xFFFFFFFFu, dw[k], m);
            db[k] += __shfl_xor_sync(0xFFFFFFFFu, db[k], m);
        }
    }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < G) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            sums[warp][0][norm_col<VEC>(g, G, k)] = dw[k];
            sums[warp][1][norm_col<VEC>(g, G, k)] = db[k];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) {
        const int which = c >= p.C, col = c - which * p.C;
        float s = 0.f;
        for (int q = 0; q < kNormThreads / 32; ++q) s += sums[q][which][col];
        if (!dead) out[c] = s;
    }
}

// out[i] = sum over q < nparts of part[q][i], i < n: the first n0 of them into
// out0, the rest into out1.  32 columns by 32 runs of q per block; each run is
// added in ascending q, the runs in ascending order.
__global__ void __launch_bounds__(1024) tri_ordered_sum_kernel(const float* __restrict__ part, int nparts, int n,
                                                               float* __restrict__ out0, int n0,
                                                               float* __restrict__ out1) {
    __shared__ float runs[32][33];
    const bool dead = device_error_pending();
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
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
// VEC: two lanes per block of 32 channels, sixteen each; else a warp per block.
template <typename TX, int ACT, bool VEC, bool PACK>
__global__ void __launch_bounds__(256) tri_act8_kernel(const __grid_constant__ NormParams p) {
    const bool dead = device_error_pending();
    constexpr int kLanes = VEC ? 2 : 32;
    const int nblk = (p.C + 31) / 32;
    const int64_t items = p.R * nblk;
    const int g = threadIdx.x % kLanes;
    constexpr int kPer = 256 / kLanes;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kPer; base < items;
         base += static_cast<int64_t>(gridDim.x) * kPer) {
        const int64_t it = base + threadIdx.x / kLanes;
        const int64_t row = it / nblk;
        const int blk = static_cast<int>(it - row * nblk);
        if constexpr (VEC) {
            const bool ok = it < items && blk * 32 + g * 16 < p.C;
            const int unit = blk * 2 + g;
            float v[16];
            if constexpr (PACK) {
                load16<TX, true>(p.x, row * p.xs, ok, unit, 2, p.C, v);
                act8_emit<ACT, true>(p, row, ok && !dead, unit, 2, v);
            } else {
                act8_load16<ACT, true>(p, row, ok, unit, 2, v);
                store16<TX, true>(p.y, row * p.ys, ok && !dead, unit, 2, p.C, v);
            }
        } else {
            const int c = blk * 32 + g;
            const bool ok = it < items && c < p.C;
            if constexpr (PACK) {
                const float v = ok ? to_f32(static_cast<const TX*>(p.x)[row * p.xs + c]) : 0.f;
                const uint32_t a = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
                const uint32_t eb = act8_exp<ACT>(a);
                if (ok && !dead) {
                    p.codes[row * p.cs + c] =
                        static_cast<uint8_t>(eb == 255u ? 0u : act8_code2<ACT>(v, 0.f, act8_inv(eb)));
                    if (g == 0) p.exps[row * p.es + blk] = static_cast<uint8_t>(eb);
                }
            } else if (ok && !dead) {
                static_cast<TX*>(p.y)[row * p.ys + c] = from_f32<TX>(
                    act8_value<ACT>(p.codes[row * p.cs + c]) * act8_scale(p.exps[row * p.es + blk]));
            }
        }
    }
}

}  // namespace tri
