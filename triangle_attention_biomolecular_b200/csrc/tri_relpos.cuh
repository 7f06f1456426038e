// tri_relpos.cuh -- learned relative position bias by buckets, sm_100a.
//
// Forward: bias[b,h,i,j] = table[bucket(b,i,j), h] (+ base), in the layout the
// attention reads.  A bucket serves all H heads, so a thread finds the buckets
// of eight neighbouring keys once and then writes 16 bytes per head; the table
// sits in shared memory.  Bound by the bytes of the bias.
//
// Backward: dtable[k,h] = sum of dbias over the positions of bucket k, read
// once.  No atomics: see tri_relpos_bwd_kernel.
#pragma once

#include "sm100.cuh"

namespace tri {

constexpr int kRelMaxEdges = 510;
// distances between the first and the last edge that get a table of their
// buckets in shared memory; wider edges are searched
constexpr int kRelLut = 2048;

struct RelposParams {
    int B, H, Nq, Nk, E;
    int nb;        // buckets, the one for different groups included
    int chunks;    // ceil(Nk / 8)
    int heads;     // heads per block (grid.y chunks of them)
    const void* table;
    int table_bf16;
    const int32_t* edges;
    const int32_t *pos_q, *pos_k, *grp_q, *grp_k;
    int64_t qs, ks;
    const __nv_bfloat16* base;
    int64_t bs[3];
    __nv_bfloat16* bias;
    int64_t os[3];
    const __nv_bfloat16* dbias;
    int64_t ds[3];
    int rows_per_task, row_tasks;  // backward: rows a warp walks, and tasks per column tile
    float* partial;                // backward: [gridDim.x][nb][H]
};

// Buckets of distances.  edges and lut are shared memory, filled by init (every
// thread of the block; a barrier follows).
struct RelposBuckets {
    const int32_t* edges;
    const uint16_t* lut;
    int E, lo, hi;
    bool table;

    // number of edges <= d
    __device__ __forceinline__ int search(int d) const {
        int n = 0;
#pragma unroll
        for (int s = 256; s > 0; s >>= 1)
            if (n + s <= E && edges[n + s - 1] <= d) n += s;
        return n;
    }
    __device__ __forceinline__ void init(int32_t* sh_edges, uint16_t* sh_lut, const RelposParams& p) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh_edges[e] = p.edges[e];
        __syncthreads();
        edges = sh_edges;
        lut = sh_lut;
        E = p.E;
        lo = sh_edges[0];
        hi = sh_edges[E - 1];
        const int64_t span = static_cast<int64_t>(hi) - lo + 2;
        table = span >= 2 && span <= kRelLut && lo != INT32_MIN;
        if (table) {
            lo -= 1;
            for (int x = threadIdx.x; x < static_cast<int>(span); x += blockDim.x)
                sh_lut[x] = static_cast<uint16_t>(search(lo + x));
        }
        __syncthreads();
    }
    __device__ __forceinline__ int operator()(int pk, int pq) const {
        // saturating: a difference past 32 bits lies beyond every edge (or, at the
        // lowest value, is compared as that value)
        int d;
        asm("sub.sat.s32 %0, %1, %2;" : "=r"(d) : "r"(pk), "r"(pq));
        return table ? lut[min(max(d, lo), hi) - lo] : search(d);
    }
};

constexpr int kRelThreads = 256;
constexpr int kRelHeads = 16;  // heads of the table a forward block holds

// words per table row: heads rounded up to 4, plus 4 so that neighbouring rows start in other banks
__host__ __device__ constexpr int relpos_pitch(int heads) { return (heads + 3) / 4 * 4 + 4; }
__host__ constexpr size_t relpos_fwd_smem(int nb, int heads) {
    return static_cast<size_t>(nb) * relpos_pitch(heads) * 4 + 512 * 4 + kRelLut * 2;
}

template <bool BASE>
__global__ void __launch_bounds__(kRelThreads) tri_relpos_fwd_kernel(const __grid_constant__ RelposParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const bool dead = device_error_pending();
    const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.H - h0);
    const int pitch = relpos_pitch(p.heads);
    float* tab = reinterpret_cast<float*>(smem);
    int32_t* sh_edges = reinterpret_cast<int32_t*>(smem + static_cast<size_t>(p.nb) * pitch * 4);
    uint16_t* sh_lut = reinterpret_cast<uint16_t*>(sh_edges + 512);
    for (int x = threadIdx.x; x < p.nb * pitch; x += kRelThreads) {
        const int r = x / pitch, h = x - r * pitch;
        float v = 0.f;
        if (h < nh) {
            const int64_t at = static_cast<int64_t>(r) * p.H + h0 + h;
            v = p.table_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.table)[at])
                             : static_cast<const float*>(p.table)[at];
        }
        tab[x] = v;
    }
    RelposBuckets bucket;
    bucket.init(sh_edges, sh_lut, p);  // ends with a barrier: the table is in place too

    const int items = p.B * p.Nq * p.chunks;  // < 2^31, checked on the host
    for (int64_t it64 = static_cast<int64_t>(blockIdx.x) * kRelThreads + threadIdx.x; it64 < items;
         it64 += static_cast<int64_t>(gridDim.x) * kRelThreads) {
        const int it = static_cast<int>(it64);
        const int bi = it / p.chunks, c = it - bi * p.chunks;
        const int b = bi / p.Nq, i = bi - b * p.Nq;
        const int j0 = c * 8, nj = min(8, p.Nk - j0);
        const int pq = p.pos_q[b * p.qs + i];
        const int gq = p.grp_q ? p.grp_q[b * p.qs + i] : 0;
        const int32_t* pk = p.pos_k + b * p.ks + j0;
        const int32_t* gk = p.grp_k ? p.grp_k + b * p.ks + j0 : nullptr;
        int at[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int xx = min(x, nj - 1);
            int k = bucket(pk[xx], pq);
            if (gk && gk[xx] != gq) k = p.E + 1;
            at[x] = k * pitch;
        }
        __nv_bfloat16* out = p.bias + b * p.os[0] + h0 * p.os[1] + i * p.os[2] + j0;
        const __nv_bfloat16* in = BASE ? p.base + b * p.bs[0] + h0 * p.bs[1] + i * p.bs[2] + j0 : nullptr;
        for (int h = 0; h < nh; h += 4) {
            float4 t[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) t[x] = *reinterpret_cast<const float4*>(tab + at[x] + h);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (h + q >= nh) break;
                float v[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = q == 0 ? t[x].x : q == 1 ? t[x].y : q == 2 ? t[x].z : t[x].w;
                __nv_bfloat16* o = out + (h + q) * p.os[1];
                const __nv_bfloat16* ib = BASE ? in + (h + q) * p.bs[1] : nullptr;
                if (nj == 8) {
                    if constexpr (BASE) {
                        const uint4 w = *reinterpret_cast<const uint4*>(ib);
                        v[0] += bf16lo(w.x); v[1] += bf16hi(w.x);
                        v[2] += bf16lo(w.y); v[3] += bf16hi(w.y);
                        v[4] += bf16lo(w.z); v[5] += bf16hi(w.z);
                        v[6] += bf16lo(w.w); v[7] += bf16hi(w.w);
                    }
                    if (!dead)
                        *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                                  pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x < nj && !dead) {
                            if constexpr (BASE) v[x] += __bfloat162float(ib[x]);
                            o[x] = __float2bfloat16_rn(v[x]);
                        }
                }
            }
        }
    }
}

// Backward.  A warp takes Hc heads (H rounded up to a power of two, at most 32)
// by S = 32 / Hc chunks of eight keys and walks down the rows i of its task; a
// lane keeps to one head and one chunk of keys.  Each lane owns a column of the
// warp's sums in shared memory, [bucket][lane]: no two lanes ever meet in a
// word (nor, 32 lanes to 32 banks, in a bank), so there are no atomics and
// every sum has one order.  Most chunks lie in one bucket as a whole (beyond
// the clipping distance, or in another chain): the bucket of the smallest and
// the largest position of the chunk tell, and the eight values then go into a
// register that is put down only when the bucket changes.
constexpr int kRelBwdWarps = 4;

__host__ constexpr size_t relpos_bwd_smem(int nb, int warps) {
    return static_cast<size_t>(warps) * nb * 32 * 4 + 512 * 4 + kRelLut * 2;
}

__global__ void __launch_bounds__(kRelBwdWarps * 32) tri_relpos_bwd_kernel(const __grid_constant__ RelposParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const bool dead = device_error_pending();
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sums = reinterpret_cast<float*>(smem);  // [warps][nb][32]
    int32_t* sh_edges = reinterpret_cast<int32_t*>(sums + static_cast<size_t>(warps) * p.nb * 32);
    uint16_t* sh_lut = reinterpret_cast<uint16_t*>(sh_edges + 512);
    for (int x = threadIdx.x; x < warps * p.nb * 32; x += blockDim.x) sums[x] = 0.f;
    RelposBuckets bucket;
    bucket.init(sh_edges, sh_lut, p);

    const int Hc = p.heads, S = 32 / Hc;
    const int h0 = blockIdx.y * Hc, h = h0 + lane / S, sub = lane % S;
    const bool head = h < p.H;
    const int tiles = (p.chunks + S - 1) / S;
    float* mine = sums + static_cast<size_t>(warp) * p.nb * 32 + lane;
    const int64_t tasks = static_cast<int64_t>(p.B) * tiles * p.row_tasks;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < tasks;
         t += static_cast<int64_t>(gridDim.x) * warps) {
        const int rt = static_cast<int>(t % p.row_tasks);
        const int64_t bt = t / p.row_tasks;
        const int tile = static_cast<int>(bt % tiles), b = static_cast<int>(bt / tiles);
        const int c = tile * S + sub;
        if (c >= p.chunks || !head) continue;  // no barrier or warp-wide step inside the walk
        const int j0 = c * 8, nj = min(8, p.Nk - j0);
        int pk[8], gk[8], pmin = INT32_MAX, pmax = INT32_MIN;
        bool one_group = true;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int xx = min(x, nj - 1);
            pk[x] = p.pos_k[b * p.ks + j0 + xx];
            gk[x] = p.grp_k ? p.grp_k[b * p.ks + j0 + xx] : 0;
            pmin = min(pmin, pk[x]);
            pmax = max(pmax, pk[x]);
            one_group &= gk[x] == gk[0];
        }
        const int i0 = rt * p.rows_per_task, i1 = min(p.Nq, i0 + p.rows_per_task);
        const __nv_bfloat16* src = p.dbias + b * p.ds[0] + h * p.ds[1] + j0;
        int cur = 0;
        float acc = 0.f;
        for (int i = i0; i < i1; ++i) {
            const int pq = p.pos_q[b * p.qs + i];
            const int gq = p.grp_q ? p.grp_q[b * p.qs + i] : 0;
            float v[8];
            const __nv_bfloat16* s = src + i * p.ds[2];
            if (nj == 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(s);
                v[0] = bf16lo(w.x); v[1] = bf16hi(w.x);
                v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
                v[4] = bf16lo(w.z); v[5] = bf16hi(w.z);
                v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
            } else {
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = x < nj ? __bfloat162float(s[x]) : 0.f;
            }
            int k0 = p.E + 1, k1 = k0;
            if (one_group && gk[0] == gq) {
                k0 = bucket(pmin, pq);
                k1 = bucket(pmax, pq);
            } else if (!one_group) {
                k1 = -1;
            }
            if (k0 == k1) {
                if (k0 != cur) {
                    mine[cur * 32] += acc;
                    acc = 0.f;
                    cur = k0;
                }
                acc += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            } else {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int k = gk[x] == gq ? bucket(pk[x], pq) : p.E + 1;
                    if (x < nj) mine[k * 32] += v[x];
                }
            }
        }
        mine[cur * 32] += acc;
    }
    __syncthreads();
    // the block's sums: over its warps, then over the chunks side by side
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.nb * p.H;
    for (int x = threadIdx.x; x < p.nb * Hc; x += blockDim.x) {
        const int k = x / Hc, hh = x - k * Hc;
        if (h0 + hh >= p.H) continue;
        float s = 0.f;
        for (int w = 0; w < warps; ++w)
            for (int q = 0; q < S; ++q) s += sums[(static_cast<size_t>(w) * p.nb + k) * 32 + hh * S + q];
        if (!dead) out[static_cast<int64_t>(k) * p.H + h0 + hh] = s;
    }
}

}  // namespace tri
