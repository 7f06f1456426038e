// tri_relpos.cuh -- learned relative position bias by buckets, sm_100a.
//
// Forward: bias[b,h,i,j] = table[bucket(b,i,j), h] (+ base), in the layout the
// attention reads.  A bucket serves all H heads, so a thread finds the buckets
// of eight neighbouring keys once and then writes 16 bytes per head; the table
// sits in shared memory.  Bound by the bytes of the bias: 2048 x 2048 x 16 heads
// take 26 us, 5.2 TB/s of stores (20.4 us at the measured copy rate); 2 x 1031 x
// 1031 x 12 heads, which the L2 cache holds, 17 us, bound by their instructions.
//
// Backward: dtable[k,h] = sum of dbias over the positions of bucket k, read
// once.  No atomics: see tri_relpos_bwd_kernel.
#pragma once

#include "sm100.cuh"
#include "tri_norm.cuh"

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
    int row_tasks, run;            // backward: warps that share the rows of a column tile, in runs of batches
    float* partial;                // backward: [gridDim.x][nb][H]
};

// number of edges <= d
__device__ __forceinline__ int relpos_search(const int32_t* edges, int E, int d) {
    int n = 0;
#pragma unroll 1
    for (int s = 256; s > 0; s >>= 1)
        if (n + s <= E && edges[n + s - 1] <= d) n += s;
    return n;
}

// Buckets of distances.  edges and lut are shared memory, filled by init (every
// thread of the block; a barrier follows).  Distances from lo to lo + kRelLut - 1
// are looked up: all there are (others are clamped to the ends) when the edges
// lie that close together, else the kRelLut around 0, and those outside are
// searched.
struct RelposBuckets {
    const int32_t* edges;
    const uint16_t* lut;
    int E, lo, size, dmin, dmax;

    __device__ __forceinline__ int search(int d) const { return relpos_search(edges, E, d); }
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
        // each thread fills a run of neighbouring distances: one search, then steps from edge to edge
        const int run = (size + blockDim.x - 1) / blockDim.x, x0 = threadIdx.x * run;
        if (x0 < size) {
            int n = search(lo + x0);
            int up = n < E ? edges[n] : INT32_MAX;
            for (int x = x0; x < min(x0 + run, size); ++x) {
                while (n < E && up <= lo + x) up = ++n < E ? edges[n] : INT32_MAX;
                sh_lut[x] = static_cast<uint16_t>(n);
            }
        }
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
    // eight distances into their buckets, the look-ups in flight together
    __device__ __forceinline__ void of8(int (&k)[8]) const {
        bool far[8], any = false;
        int near[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const uint32_t at = static_cast<uint32_t>(min(max(k[x], dmin), dmax)) - static_cast<uint32_t>(lo);
            far[x] = at >= static_cast<uint32_t>(size);
            any |= far[x];
            near[x] = lut[far[x] ? 0u : at];
        }
        if (any) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (far[x]) near[x] = search(k[x]);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) k[x] = near[x];
    }
};

// Eight keys of a row, 16 bytes at once, of which n belong to the row (n < 8 only at
// its end): the others are read with them and count as 0.  Put together from
// smaller loads instead, the end of a row made every load wait for its value (2x).
__device__ __forceinline__ uint4 relpos_cut8(const uint4& w, int n) {
    const auto keep = [n](uint32_t v, int x) { return n >= x + 2 ? v : n == x + 1 ? v & 0xFFFFu : 0u; };
    return make_uint4(keep(w.x, 0), keep(w.y, 2), keep(w.z, 4), keep(w.w, 6));
}
__device__ __forceinline__ uint4 relpos_load8(const __nv_bfloat16* s, int n) {
    const uint4 w = *reinterpret_cast<const uint4*>(s);
    return n < 8 ? relpos_cut8(w, n) : w;
}
__device__ __forceinline__ void relpos_values(const uint4& w, float (&v)[8]) {
    v[0] = bf16lo(w.x); v[1] = bf16hi(w.x);
    v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z); v[5] = bf16hi(w.z);
    v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}
__device__ __forceinline__ void relpos_store8(__nv_bfloat16* s, int n, const uint4& w) {
    if (n == 8) {
        *reinterpret_cast<uint4*>(s) = w;
        return;
    }
    if (n & 4) *reinterpret_cast<uint2*>(s) = make_uint2(w.x, w.y);
    const uint32_t two = n & 4 ? w.z : w.x;
    if (n & 2) *reinterpret_cast<uint32_t*>(s + (n & 4)) = two;
    const uint32_t one = n == 7 ? w.w : n == 5 ? w.z : n == 3 ? w.y : w.x;
    if (n & 1) s[n - 1] = __ushort_as_bfloat16(static_cast<unsigned short>(one));
}

constexpr int kRelThreads = 256, kRelFwdBlocks = 4;  // per SM
constexpr int kRelHeads = 16;  // heads of the table a forward block holds

// The table in shared memory, read 8 bytes at a time: BF16 of four heads, or, where
// a base is added before the rounding, FP32 of two.  A row is an odd number of
// these, so that sixteen neighbouring rows start in sixteen different pairs of banks.
__host__ __device__ constexpr int relpos_pitch(int heads, bool base) {
    return (base ? (heads + 1) / 2 : (heads + 3) / 4) | 1;
}
__host__ constexpr size_t relpos_fwd_smem(int nb, int heads, bool base) {
    return static_cast<size_t>(nb) * relpos_pitch(heads, base) * 8 + 512 * 4 + kRelLut * 2;
}

// Forward.  A thread keeps to one chunk of eight keys and walks down the rows, as
// many rows at a step as all threads together hold; neighbouring threads take
// neighbouring chunks, so a warp's 16-byte stores lie side by side.  With the
// table in FP32 throughout, and every chunk looked up key by key, the two sizes
// above took 29 and 26 us; with warps split between the two ways, 28 and 19.
template <bool BASE>
__global__ void __launch_bounds__(kRelThreads, kRelFwdBlocks)
    tri_relpos_fwd_kernel(const __grid_constant__ RelposParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const bool dead = device_error_pending();
    const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.H - h0);
    const int pitch = relpos_pitch(p.heads, BASE);
    uint2* tab = reinterpret_cast<uint2*>(smem);
    int32_t* sh_edges = reinterpret_cast<int32_t*>(tab + static_cast<size_t>(p.nb) * pitch);
    uint16_t* sh_lut = reinterpret_cast<uint16_t*>(sh_edges + 512);
    {
        constexpr int kPer = BASE ? 2 : 4;  // heads per entry
        const int per_row = pitch * kPer;
        for (int x = threadIdx.x; x < p.nb * per_row; x += kRelThreads) {
            const int r = x / per_row, h = x - r * per_row;
            float v = 0.f;
            if (h < nh) {
                const int64_t at = static_cast<int64_t>(r) * p.H + h0 + h;
                v = p.table_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.table)[at])
                                 : static_cast<const float*>(p.table)[at];
            }
            if constexpr (BASE)
                reinterpret_cast<float*>(tab)[x] = v;
            else
                reinterpret_cast<__nv_bfloat16*>(tab)[x] = __float2bfloat16_rn(v);
        }
    }
    RelposBuckets bucket;
    bucket.init(sh_edges, sh_lut, p);  // ends with a barrier: the table is in place too

    // the grid holds at least one row of chunks (see the launch)
    const uint32_t id = blockIdx.x * kRelThreads + threadIdx.x, chunks = p.chunks;
    const int rstep = static_cast<int>(gridDim.x * kRelThreads / chunks), row0 = static_cast<int>(id / chunks);
    if (row0 >= rstep) return;  // no barrier follows
    const int j0 = static_cast<int>(id - row0 * chunks) * 8, nj = min(8, p.Nk - j0);
    int key[8], pmin = 0, pmax = 0, g0 = 0;
    bool one_group = true;
    const int32_t* gk = nullptr;
    int last_b = -1;
    for (int64_t row = row0; row < static_cast<int64_t>(p.B) * p.Nq; row += rstep) {
        const int b = static_cast<int>(row) / p.Nq, i = static_cast<int>(row) - b * p.Nq;
        if (b != last_b) {
            last_b = b;
            const int32_t* pk = p.pos_k + b * p.ks + j0;
            gk = p.grp_k ? p.grp_k + b * p.ks + j0 : nullptr;
            g0 = gk ? gk[0] : 0;
            one_group = true;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                key[x] = pk[min(x, nj - 1)];
                pmin = x ? min(pmin, key[x]) : key[x];
                pmax = x ? max(pmax, key[x]) : key[x];
                if (gk) one_group &= gk[min(x, nj - 1)] == g0;
            }
        }
        const int pq = p.pos_q[b * p.qs + i];
        const int gq = p.grp_q ? p.grp_q[b * p.qs + i] : 0;
        // a chunk whose nearest and farthest key lie in one bucket needs no other look
        int at[8];
        bool one = false;
        if (one_group) {
            at[0] = g0 == gq ? bucket.of(RelposBuckets::distance(pmin, pq)) : p.E + 1;
            one = g0 != gq || at[0] == bucket.of(RelposBuckets::distance(pmax, pq));
        }
        if (!one) {
#pragma unroll
            for (int x = 0; x < 8; ++x) at[x] = RelposBuckets::distance(key[x], pq);
            bucket.of8(at);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                if (!one_group && gk[min(x, nj - 1)] != gq) at[x] = p.E + 1;
                at[x] *= pitch;
            }
        } else {
            at[0] *= pitch;
#pragma unroll
            for (int x = 1; x < 8; ++x) at[x] = at[0];
        }
        // the short way only where the whole warp can take it: a split warp would go both
        one = __all_sync(__activemask(), one);
        __nv_bfloat16* out = p.bias + b * p.os[0] + h0 * p.os[1] + i * p.os[2] + j0;
        if constexpr (BASE) {
            const __nv_bfloat16* in = p.base + b * p.bs[0] + h0 * p.bs[1] + i * p.bs[2] + j0;
            for (int h = 0; h < nh; h += 2) {
                const bool two = h + 1 < nh;
                float u0[8], u1[8];
                relpos_values(relpos_load8(in, nj), u0);
                in += p.bs[1];
                relpos_values(two ? relpos_load8(in, nj) : make_uint4(0u, 0u, 0u, 0u), u1);
                in += p.bs[1];
                uint2 e = tab[at[0] + h / 2];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (x > 0 && !one) e = tab[at[x] + h / 2];
                    u0[x] += __uint_as_float(e.x);
                    u1[x] += __uint_as_float(e.y);
                }
                if (!dead) {
                    relpos_store8(out, nj, make_uint4(pack_bf16(u0[0], u0[1]), pack_bf16(u0[2], u0[3]),
                                                      pack_bf16(u0[4], u0[5]), pack_bf16(u0[6], u0[7])));
                    if (two)
                        relpos_store8(out + p.os[1], nj, make_uint4(pack_bf16(u1[0], u1[1]), pack_bf16(u1[2], u1[3]),
                                                                    pack_bf16(u1[4], u1[5]), pack_bf16(u1[6], u1[7])));
                }
                out += 2 * p.os[1];
            }
        } else if (one) {
            for (int h = 0; h < nh; h += 4) {
                const uint2 e = tab[at[0] + h / 4];
#pragma unroll
                for (int q = 0; q < 4; ++q, out += p.os[1]) {
                    const uint32_t w = __byte_perm(q < 2 ? e.x : e.y, 0u, q & 1 ? 0x3232 : 0x1010);
                    if (h + q < nh && !dead) relpos_store8(out, nj, make_uint4(w, w, w, w));
                }
            }
        } else {
            for (int h = 0; h < nh; h += 4) {
                uint2 e[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) e[x] = tab[at[x] + h / 4];
#pragma unroll
                for (int q = 0; q < 4; ++q, out += p.os[1]) {
                    uint32_t w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        w[x] = __byte_perm(q < 2 ? e[2 * x].x : e[2 * x].y, q < 2 ? e[2 * x + 1].x : e[2 * x + 1].y,
                                           q & 1 ? 0x7632 : 0x5410);
                    if (h + q < nh && !dead) relpos_store8(out, nj, make_uint4(w[0], w[1], w[2], w[3]));
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
// Most chunks lie in one bucket as a whole: beyond the first or the last edge, in
// another group, or between two edges far apart.  A lane therefore keeps five sums
// in registers, those of the first and the last bucket, of the pairs of different
// groups, and of two neighbouring buckets it has in hand, and only a chunk that
// none of them covers takes the slow way: its buckets are looked up key by key, and
// either become the two in hand or are added to the column.  kRelRows rows are
// taken at a time and loaded while the ones before are added up; where one sum takes
// them all it takes them in one step, else they are gone through one by one (and
// read again, from the cache) by a loop of their own, since unrolled into the walk
// that code did not fit the instruction cache.  Neighbouring warps take
// neighbouring keys of the same rows: with neighbouring rows instead, 2368 warps
// on rows far apart reached 1.1 TB/s.
//
// 2048 x 2048 x 16 heads: 55 us (44 us in one chain without gaps; floor 20.4 us).
// What bounds it is the latency of 16 warps per SM, as many as the columns and the
// registers leave room for (8 from 108 buckets on, fewer from 195 on); 24 warps
// spilled and took 98 us, and so did batches of two rows.  2 x 1031 x 1031 x 12 heads
// with edges out to 200000: 39 us, of which 17 are rows gone through one by one.
// 768 x 768 x 4 heads: 11 us, most of it latency.
constexpr int kRelBwdWarps = 8, kRelBwdBlocks = 2;  // per block, blocks per SM
constexpr int kRelRows = 4;
constexpr int kRelBwdSmem = 200 * 1024;  // the columns of as many warps as fit

__host__ constexpr size_t relpos_bwd_smem(int nb, int warps) {
    return static_cast<size_t>(warps) * nb * 32 * 4 + 512 * 4 + kRelLut * 2;
}
// blocks that an SM holds at once: two while the columns leave room for a second one (up to 107
// buckets), then one; a block takes 1 KB more than it asks for.  768 x 768 x 4 heads with 129
// buckets: 11.2 us; cut for two blocks where one fits, 17.6
__host__ constexpr int relpos_bwd_per_sm(size_t smem) {
    return kRelBwdBlocks * (smem + 1024) <= 228 * 1024 ? kRelBwdBlocks : 1;
}

__device__ __forceinline__ int relpos_cut(int64_t v) {
    return static_cast<int>(v < INT32_MIN ? INT32_MIN : v > INT32_MAX ? INT32_MAX : v);
}

// The two buckets a lane has in hand, first and first + 1 (first < E).  What they
// mean for the chunk's keys is kept in terms of the query's position q, so that a
// row costs comparisons and no saturating subtraction: the chunk lies within the
// two for qlo < q < qhi, and key x of it above the edge between them for q < t[x]
// (tmin .. tmax).  Bounds past 32 bits are cut to positions that then lie outside.
struct RelposPair {
    int first, qlo, qhi, tmin, tmax, t[8];
    float sum0, sum1;
    // n keys at positions pk, from their least to their greatest one
    __device__ __forceinline__ void take(const RelposBuckets& bucket, int k, const int32_t* pk, int n, int pmin,
                                         int pmax) {
        first = k;
        sum0 = sum1 = 0.f;
        asm volatile("" : "+l"(pk));  // keeps eight loop-invariant addresses out of the walk's registers
#pragma unroll
        for (int x = 0; x < 8; ++x)
            t[x] = relpos_cut(static_cast<int64_t>(pk[min(x, n - 1)]) - bucket.edges[k] + 1);
        tmin = relpos_cut(static_cast<int64_t>(pmin) - bucket.edges[k] + 1);
        tmax = relpos_cut(static_cast<int64_t>(pmax) - bucket.edges[k] + 1);
        qhi = k > 0 ? relpos_cut(static_cast<int64_t>(pmin) - bucket.edges[k - 1] + 1) : INT32_MAX;
        qlo = k + 1 < bucket.E ? relpos_cut(static_cast<int64_t>(pmax) - bucket.edges[k + 1]) : INT32_MIN;
    }
    __device__ __forceinline__ bool fits(int q) const { return q > qlo && q < qhi; }
    __device__ __forceinline__ void add(const float (&v)[8], int q) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            if (q < t[x])
                b += v[x];
            else
                a += v[x];
        }
        sum0 += a;
        sum1 += b;
    }
    __device__ __forceinline__ void put(float* column) const {
        column[first * 32] += sum0;
        column[(first + 1) * 32] += sum1;
    }
};

__device__ __forceinline__ float relpos_sum8(const float (&v)[8]) {
    const float2 a = fadd2(make_float2(v[0], v[1]), make_float2(v[2], v[3]));
    const float2 b = fadd2(make_float2(v[4], v[5]), make_float2(v[6], v[7]));
    const float2 c = fadd2(a, b);
    return c.x + c.y;
}

// kRelRows rows of a lane's chunk, as loaded
struct RelposBatch {
    uint4 w[kRelRows];
    int q[kRelRows], g[kRelRows];
    template <bool GROUPS>
    __device__ __forceinline__ void load(const __nv_bfloat16* s, int64_t step, const int32_t* pos, const int32_t* grp) {
#pragma unroll
        for (int u = 0; u < kRelRows; ++u, s += step) {
            w[u] = *reinterpret_cast<const uint4*>(s);
            q[u] = pos[u];
            g[u] = GROUPS ? grp[u] : 0;
        }
    }
};

template <bool GROUPS>
__global__ void __launch_bounds__(kRelBwdWarps * 32, kRelBwdBlocks)
    tri_relpos_bwd_kernel(const __grid_constant__ RelposParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    grid_dependents_start();
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
    const uint32_t tasks = static_cast<uint32_t>(p.B) * tiles * p.row_tasks;  // < 2^31, see the launch
    for (uint32_t task = blockIdx.x * warps + warp; task < tasks; task += gridDim.x * warps) {
        // neighbouring warps take neighbouring keys of the same rows
        const uint32_t br = task / tiles, tile = task - br * tiles;
        const int b = static_cast<int>(br / p.row_tasks), rt = static_cast<int>(br - b * p.row_tasks);
        const int c = static_cast<int>(tile) * S + sub;
        if (c >= p.chunks || h >= p.H) continue;  // no barrier or warp-wide step inside the walk
        const int j0 = c * 8, nj = min(8, p.Nk - j0);
        const int32_t* keys = p.pos_k + b * p.ks + j0;
        const int32_t* gkeys = GROUPS ? p.grp_k + b * p.ks + j0 : nullptr;
        const int32_t* pos = p.pos_q + b * p.qs;
        const int32_t* grp = GROUPS ? p.grp_q + b * p.qs : nullptr;
        const int g0 = GROUPS ? gkeys[0] : 0;
        bool one_group = true;
        RelposPair hand;
        int pmin = INT32_MAX, pmax = INT32_MIN;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int k = keys[min(x, nj - 1)];
            pmin = min(pmin, k);
            pmax = max(pmax, k);
            if (GROUPS) one_group &= gkeys[min(x, nj - 1)] == g0;
        }
        // all keys lie below the first edge for q > q0, above the last for q < qE
        const int q0 = one_group ? relpos_cut(static_cast<int64_t>(pmax) - sh_edges[0]) : INT32_MAX;
        const int qE = one_group ? relpos_cut(static_cast<int64_t>(pmin) - sh_edges[p.E - 1] + 1) : INT32_MIN;
        hand.take(bucket, 0, keys, nj, pmin, pmax);
        if (!one_group) hand.qhi = INT32_MIN;  // nothing fits
        float low = 0.f, high = 0.f, apart = 0.f;
        const __nv_bfloat16* src = p.dbias + b * p.ds[0] + h * p.ds[1] + j0;
        const int64_t step = p.ds[2];
        // a batch of rows, loaded while the one before it is added up
        RelposBatch next;
        // `run` batches in a row, then on past the runs of the other tasks
        const int jump = ((p.row_tasks - 1) * p.run + 1) * kRelRows;
        int i0 = rt * p.run * kRelRows, left = p.run;
        if (i0 + kRelRows <= p.Nq) next.load<GROUPS>(src + i0 * step, step, pos + i0, grp + i0);
        for (int i2; i0 < p.Nq; i0 = i2) {
            i2 = i0 + (--left ? kRelRows : jump);
            if (left == 0) left = p.run;
            if (i0 + kRelRows <= p.Nq) {
                RelposBatch now = next;
                if (i2 + kRelRows <= p.Nq) next.load<GROUPS>(src + i2 * step, step, pos + i2, grp + i2);
                int lo = now.q[0], hi = now.q[0];
                bool same = one_group, other = GROUPS && one_group;
#pragma unroll
                for (int u = 0; u < kRelRows; ++u) {
                    lo = min(lo, now.q[u]);
                    hi = max(hi, now.q[u]);
                    if (GROUPS) {
                        same &= now.g[u] == g0;
                        other &= now.g[u] != g0;
                    }
                }
                const bool is_low = same && lo > q0, is_high = same && hi < qE;
                const bool in = same && !is_low && !is_high && lo > hand.qlo && hi < hand.qhi;
                const bool below = in && lo >= hand.tmax, above = in && hi < hand.tmin;
                if (other || is_low || is_high || below || above) {
                    if (nj < 8) {
#pragma unroll
                        for (int u = 0; u < kRelRows; ++u) now.w[u] = relpos_cut8(now.w[u], nj);
                    }
                    float2 a[kRelRows];
#pragma unroll
                    for (int u = 0; u < kRelRows; ++u)
                        a[u] = fadd2(fadd2(bf16x2_to_f2(now.w[u].x), bf16x2_to_f2(now.w[u].y)),
                                     fadd2(bf16x2_to_f2(now.w[u].z), bf16x2_to_f2(now.w[u].w)));
#pragma unroll
                    for (int m = 1; m < kRelRows; m *= 2)
#pragma unroll
                        for (int u = 0; u < kRelRows; u += 2 * m) a[u] = fadd2(a[u], a[u + m]);
                    const float all = a[0].x + a[0].y;
                    apart += other ? all : 0.f;
                    low += is_low ? all : 0.f;
                    high += is_high ? all : 0.f;
                    hand.sum0 += below ? all : 0.f;
                    hand.sum1 += above ? all : 0.f;
                    continue;
                }
            }
#pragma unroll 1
            for (int i = i0; i < min(p.Nq, i0 + kRelRows); ++i) {
                const int q = pos[i], g = GROUPS ? grp[i] : 0;
                float v[8];
                relpos_values(relpos_load8(src + i * step, nj), v);
                if (one_group) {
                    const float all = relpos_sum8(v);
                    const bool other = GROUPS && g != g0;
                    const bool is_low = !other && q > q0, is_high = !other && q < qE;
                    apart += other ? all : 0.f;
                    low += is_low ? all : 0.f;
                    high += is_high ? all : 0.f;
                    if (other || is_low || is_high) continue;
                    if (hand.fits(q)) {
                        hand.add(v, q);
                        continue;
                    }
                }
                const int32_t* kp = keys;
                asm volatile("" : "+l"(kp));  // keeps what depends on it from being held through the walk
                int k[8], least = INT32_MAX, most = 0;
#pragma unroll
                for (int x = 0; x < 8; ++x) k[x] = RelposBuckets::distance(kp[min(x, nj - 1)], q);
                bucket.of8(k);
                bool ascending = true;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (GROUPS && !one_group && gkeys[min(x, nj - 1)] != g) k[x] = p.E + 1;
                    if (x > 0) ascending &= k[x] >= k[x - 1];
                    least = min(least, k[x]);
                    most = max(most, k[x]);
                }
                if (one_group && most - least <= 1) {  // two others to take in hand
                    hand.put(mine);
                    hand.take(bucket, min(least, p.E - 1), keys, nj, pmin, pmax);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        hand.sum0 += k[x] == hand.first ? v[x] : 0.f;
                        hand.sum1 += k[x] == hand.first ? 0.f : v[x];
                    }
                } else if (ascending) {
                    // the usual case: equal neighbours are joined first, and what is left lies in
                    // different words
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
        hand.put(mine);
        mine[0] += low;
        mine[p.E * 32] += high;
        if (GROUPS) mine[(p.E + 1) * 32] += apart;
    }
    __syncthreads();
    // the block's sums: word by word over the warps, then over the chunks side by side, starting
    // at another chunk for each bucket so that the lanes read different banks
    const int words = p.nb * 32;
#pragma unroll 3
    for (int x = threadIdx.x; x < words; x += blockDim.x) {
        float s[kRelBwdWarps];
#pragma unroll
        for (int w = 0; w < kRelBwdWarps; ++w) s[w] = w < warps ? sums[w * words + x] : 0.f;
#pragma unroll
        for (int m = 1; m < kRelBwdWarps; m *= 2)
#pragma unroll
            for (int w = 0; w < kRelBwdWarps; w += 2 * m) s[w] += s[w + m];
        sums[x] = s[0];
    }
    __syncthreads();
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.nb * p.H + h0;
    for (int x = threadIdx.x; x < p.nb * Hc; x += blockDim.x) {
        const int k = x / Hc, hh = x & (Hc - 1);
        float s = 0.f;
#pragma unroll 8
        for (int q = 0; q < S; ++q) s += sums[k * 32 + hh * S + ((q + k) & (S - 1))];
        if (h0 + hh < p.H && !dead) out[static_cast<int64_t>(k) * p.H + hh] = s;
    }
}

}  // namespace tri
