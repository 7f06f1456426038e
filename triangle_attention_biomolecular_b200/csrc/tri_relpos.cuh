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
// distances whose buckets are tabulated in shared memory
constexpr int kRelLut = 2048;

struct RelposParams {
    int B, H, Nq, Nk, E;
    int nb;        // buckets, the one for different groups included
    int chunks;    // ceil(Nk / 8)
    int heads;     // heads per block (grid.y chunks of them); backward: per warp
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
    int row_tasks;                 // backward: warps that share the rows of a column tile
    float* partial;                // backward: [gridDim.x][nb][H]
};

// Buckets of distances.  edges and lut are shared memory, filled by init (every
// thread of the block; a barrier follows).  Distances from lo to lo + kRelLut - 1
// are looked up: all there are (others are clamped to the ends) when the edges
// lie that close together, else the kRelLut around 0, and those outside are
// searched.
struct RelposBuckets {
    const int32_t* edges;
    const uint16_t* lut;
    int E, lo, size, dmin, dmax;

    // number of edges <= d; rarely needed, so one copy of the code
    __device__ __noinline__ int search(int d) const {
        int n = 0;
#pragma unroll 1
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
        const int first = sh_edges[0], last = sh_edges[E - 1];
        const int64_t span = static_cast<int64_t>(last) - first + 2;
        if (span >= 2 && span <= kRelLut && first != INT32_MIN) {
            lo = dmin = first - 1;
            dmax = last;
            size = static_cast<int>(span);
        } else {
            lo = -kRelLut / 2;
            size = kRelLut;
            dmin = INT32_MIN;
            dmax = INT32_MAX;
        }
        for (int x = threadIdx.x; x < size; x += blockDim.x) sh_lut[x] = static_cast<uint16_t>(search(lo + x));
        __syncthreads();
    }
    // pk - pq, saturating: a difference past 32 bits lies beyond every edge
    static __device__ __forceinline__ int distance(int pk, int pq) {
        int d;
        asm("sub.sat.s32 %0, %1, %2;" : "=r"(d) : "r"(pk), "r"(pq));
        return d;
    }
    __device__ __forceinline__ int of(int d) const {
        d = min(max(d, dmin), dmax);
        const uint32_t x = static_cast<uint32_t>(d) - static_cast<uint32_t>(lo);
        return x < static_cast<uint32_t>(size) ? lut[x] : search(d);
    }
    // eight at once, their look-ups in flight together
    __device__ __forceinline__ void of8(const int (&d)[8], int (&k)[8]) const {
        bool far[8], any = false;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int dx = min(max(d[x], dmin), dmax);
            const uint32_t at = static_cast<uint32_t>(dx) - static_cast<uint32_t>(lo);
            far[x] = at >= static_cast<uint32_t>(size);
            any |= far[x];
            k[x] = lut[far[x] ? 0u : at];
        }
        if (any) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (far[x]) k[x] = search(d[x]);
        }
    }
    // the distances of bucket k are least(k) <= d <= most(k)
    __device__ __forceinline__ int least(int k) const { return k > 0 ? edges[k - 1] : INT32_MIN; }
    __device__ __forceinline__ int most(int k) const { return k < E ? edges[k] - 1 : INT32_MAX; }
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
        // a chunk whose nearest and farthest key lie in one bucket needs no other look
        int key[8], at[8];
        int pmin = INT32_MAX, pmax = INT32_MIN;
        bool same = true, apart = true;  // all keys of the query's group; none
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int xx = min(x, nj - 1);
            key[x] = pk[xx];
            pmin = min(pmin, key[x]);
            pmax = max(pmax, key[x]);
            at[x] = gk && gk[xx] != gq;
            same &= !at[x];
            apart &= at[x] != 0;
        }
        const int first = apart ? p.E + 1 : bucket.of(RelposBuckets::distance(pmin, pq));
        const bool one = apart || (same && first == bucket.of(RelposBuckets::distance(pmax, pq)));
        if (one) {
#pragma unroll
            for (int x = 0; x < 8; ++x) at[x] = first * pitch;
        } else {
            int k[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) key[x] = RelposBuckets::distance(key[x], pq);
            bucket.of8(key, k);
#pragma unroll
            for (int x = 0; x < 8; ++x) at[x] = (at[x] ? p.E + 1 : k[x]) * pitch;
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

// Backward.  A warp takes S chunks of eight keys by 32 / S heads and walks down
// rows i; a lane keeps to one head and one chunk.  Each lane owns a column of the
// warp's sums in shared memory, [bucket][lane]: no two lanes ever meet in a word
// (nor, 32 lanes to 32 banks, in a bank), so there are no atomics and every sum
// has one order.
//
// Most chunks lie in one bucket as a whole (beyond the clipping distance, or in
// another group) or across one edge.  A lane therefore holds two neighbouring
// buckets in hand, each with a sum in a register, and the bounds that tell with two
// comparisons that a chunk lies within them; they are put down into the column
// when a chunk does not.  Rows are taken kRelRows at a time, so that their loads
// are in flight together; the few rows that need more than the registers are read
// again afterwards (from the cache) by one compact loop: unrolled into the walk,
// that code did not fit the instruction cache.  A task's batches of rows lie a
// whole round of tasks apart, since the rows near the diagonal cost the most.
constexpr int kRelBwdWarps = 4;
constexpr int kRelRows = 8;

__host__ constexpr size_t relpos_bwd_smem(int nb, int warps) {
    return static_cast<size_t>(warps) * nb * 32 * 4 + 512 * 4 + kRelLut * 2;
}

// the two buckets a lane has in hand: first and, if there is one, first + 1
struct RelposPair {
    int first, least, edge, most;  // distances least .. edge - 1 and edge .. most
    float sum0, sum1;
    __device__ __forceinline__ void take(const RelposBuckets& bucket, int k) {
        first = k;
        least = bucket.least(k);
        edge = k < bucket.E ? bucket.edges[k] : INT32_MAX;
        most = bucket.most(min(k + 1, bucket.E));
        sum0 = sum1 = 0.f;
    }
    __device__ __forceinline__ void put(float* column, int E) const {
        if (first < E) {
            column[first * 32] += sum0;
            column[(first + 1) * 32] += sum1;
        } else {
            column[E * 32] += sum0 + sum1;
        }
    }
    // a chunk across the edge
    __device__ __forceinline__ void split(const float (&v)[8], const int (&pk)[8], int pq) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const bool up = RelposBuckets::distance(pk[x], pq) >= edge;
            a += up ? 0.f : v[x];
            b += up ? v[x] : 0.f;
        }
        sum0 += a;
        sum1 += b;
    }
};

__device__ __forceinline__ void relpos_load8(const __nv_bfloat16* s, int n, uint4& w) {
    if (n == 8) {
        w = *reinterpret_cast<const uint4*>(s);
    } else {
        uint32_t v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = x < n ? __bfloat16_as_ushort(s[x]) : 0u;
        w = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}
__device__ __forceinline__ void relpos_values(const uint4& w, float (&v)[8]) {
    v[0] = bf16lo(w.x); v[1] = bf16hi(w.x);
    v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z); v[5] = bf16hi(w.z);
    v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}

__device__ __forceinline__ float relpos_sum8(const float (&v)[8]) {
    const float2 a = fadd2(make_float2(v[0], v[1]), make_float2(v[2], v[3]));
    const float2 b = fadd2(make_float2(v[4], v[5]), make_float2(v[6], v[7]));
    const float2 c = fadd2(a, b);
    return c.x + c.y;
}

__global__ void __launch_bounds__(kRelBwdWarps * 32, 5) tri_relpos_bwd_kernel(const __grid_constant__ RelposParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const bool dead = device_error_pending();
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sums = reinterpret_cast<float*>(smem);  // [warps][nb][32]
    int32_t* sh_edges = reinterpret_cast<int32_t*>(sums + static_cast<size_t>(warps) * p.nb * 32);
    uint16_t* sh_lut = reinterpret_cast<uint16_t*>(sh_edges + 512);
    for (int x = threadIdx.x; x < warps * p.nb * 8; x += blockDim.x)
        reinterpret_cast<float4*>(sums)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    RelposBuckets bucket;
    bucket.init(sh_edges, sh_lut, p);

    const int Hc = p.heads, S = 32 / Hc;
    const int h0 = blockIdx.y * Hc, h = h0 + lane / S, sub = lane % S;
    const int tiles = (p.chunks + S - 1) / S;
    float* mine = sums + static_cast<size_t>(warp) * p.nb * 32 + lane;
    const int64_t tasks = static_cast<int64_t>(p.B) * tiles * p.row_tasks;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < tasks;
         t += static_cast<int64_t>(gridDim.x) * warps) {
        const int rt = static_cast<int>(t % p.row_tasks);
        const int64_t bt = t / p.row_tasks;
        const int tile = static_cast<int>(bt % tiles), b = static_cast<int>(bt / tiles);
        const int c = tile * S + sub;
        if (c >= p.chunks || h >= p.H) continue;  // no barrier or warp-wide step inside the walk
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
        const __nv_bfloat16* src = p.dbias + b * p.ds[0] + h * p.ds[1] + j0;
        const int32_t* pos = p.pos_q + b * p.qs;
        const int32_t* grp = p.grp_q ? p.grp_q + b * p.qs : nullptr;
        RelposPair hand;
        hand.take(bucket, 0);
        float apart = 0.f;  // pairs of different groups
        for (int i0 = rt * kRelRows; i0 < p.Nq; i0 += p.row_tasks * kRelRows) {
            uint4 w[kRelRows];
            int pq[kRelRows], gq[kRelRows];
            const __nv_bfloat16* s = src + i0 * p.ds[2];
            const int rows = min(kRelRows, p.Nq - i0);
            if (rows == kRelRows) {
#pragma unroll
                for (int u = 0; u < kRelRows; ++u, s += p.ds[2]) {
                    pq[u] = pos[i0 + u];
                    gq[u] = grp ? grp[i0 + u] : 0;
                    relpos_load8(s, nj, w[u]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kRelRows; ++u, s += p.ds[2]) {
                    pq[u] = gq[u] = 0;
                    if (u < rows) {
                        pq[u] = pos[i0 + u];
                        gq[u] = grp ? grp[i0 + u] : 0;
                        relpos_load8(s, nj, w[u]);
                    }
                }
            }
            uint32_t more = 0;
#pragma unroll
            for (int u = 0; u < kRelRows; ++u) {
                if (u >= rows) break;
                const int lo = RelposBuckets::distance(pmin, pq[u]), hi = RelposBuckets::distance(pmax, pq[u]);
                float v[8];
                relpos_values(w[u], v);
                const float all = relpos_sum8(v);
                const bool other = one_group && gk[0] != gq[u];
                const bool fits = one_group && !other && lo >= hand.least && hi <= hand.most;
                const bool below = fits && hi < hand.edge, above = fits && lo >= hand.edge;
                apart += other ? all : 0.f;
                hand.sum0 += below ? all : 0.f;
                hand.sum1 += above ? all : 0.f;
                if (fits && !below && !above) hand.split(v, pk, pq[u]);
                if (!other && !fits) more |= 1u << u;
            }
            while (more) {
                const int i = i0 + __ffs(more) - 1;
                more &= more - 1;
                uint4 wi;
                float v[8];
                relpos_load8(src + i * p.ds[2], nj, wi);
                relpos_values(wi, v);
                const int q = pos[i], g = grp ? grp[i] : 0;
                if (one_group) {  // and of the row's group
                    const int lo = RelposBuckets::distance(pmin, q), hi = RelposBuckets::distance(pmax, q);
                    if (lo < hand.least || hi > hand.most) {
                        hand.put(mine, p.E);
                        hand.take(bucket, bucket.of(lo));
                    }
                    if (hi <= hand.most) {
                        hand.split(v, pk, q);
                        continue;
                    }
                }
                // key by key; in ascending order of buckets (the usual case) equal neighbours are
                // joined first, and what is left lies in different words
                int d[8], k[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) d[x] = RelposBuckets::distance(pk[x], q);
                bucket.of8(d, k);
                bool ascending = true;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (gk[x] != g) k[x] = p.E + 1;
                    if (x > 0) ascending &= k[x] >= k[x - 1];
                }
                if (ascending) {
                    float old[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        if (x < 7 && k[x] == k[min(x + 1, 7)]) {
                            v[min(x + 1, 7)] += v[x];
                            k[x] = -1;
                        }
                        old[x] = k[x] >= 0 ? mine[k[x] * 32] : 0.f;
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (k[x] >= 0) mine[k[x] * 32] = old[x] + v[x];
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x < nj) mine[k[x] * 32] += v[x];
                }
            }
        }
        hand.put(mine, p.E);
        if (p.grp_k) mine[(p.E + 1) * 32] += apart;
    }
    __syncthreads();
    // the block's sums: a warp per bucket, over the warps, then over the chunks side by side
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.nb * p.H;
#pragma unroll 4
    for (int k = warp; k < p.nb; k += warps) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += sums[(static_cast<size_t>(w) * p.nb + k) * 32 + lane];
        for (int m = 1; m < S; m <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
        if (sub == 0 && h < p.H && !dead) out[static_cast<int64_t>(k) * p.H + h] = s;
    }
}

}  // namespace tri
