// pair_ops.cuh -- host side of the layer norm, the 8-bit activation and the
// relative position bias: argument checks, launch shapes and the exported entry
// points.  Part of api.cu's translation unit (one device error word).
#pragma once

namespace {

using tri::NormParams;
using tri::RelposParams;

bool type_ok(int t) { return t == TRI_TYPE_BF16 || t == TRI_TYPE_F32; }
int64_t type_bytes(int t) { return t == TRI_TYPE_F32 ? 4 : 2; }
bool aligned_to(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// rows of an array the library reads (out = false) or writes
tri_attn_status check_rows(const void* p, int64_t R, int64_t C, int64_t stride, int64_t elem, bool out) {
    if (!p && R > 0) return TRI_ATTN_ERR_NULL;
    if (stride < 0 || (out && R > 1 && stride < C)) return TRI_ATTN_ERR_STRIDE;
    if (!aligned_to(p, elem)) return TRI_ATTN_ERR_ALIGN;
    return TRI_ATTN_OK;
}
tri_attn_status check_act8(const tri_act8& a, int64_t R, int C, bool out) {
    if (a.kind != TRI_ACT8_INT8 && a.kind != TRI_ACT8_E4M3) return TRI_ATTN_ERR_UNSUPPORTED;
    tri_attn_status st = check_rows(a.codes, R, C, a.codes_stride, 1, out);
    return st ? st : check_rows(a.exps, R, (C + 31) / 32, a.exps_stride, 1, out);
}
constexpr int kNormMaxC = 16 * 32 * tri::kNormMaxWarps;
tri_attn_status check_norm_sizes(int64_t R, int C) {
    if (R < 0 || R > (int64_t{1} << 40) || C < 1) return TRI_ATTN_ERR_SHAPE;
    return C > kNormMaxC ? TRI_ATTN_ERR_UNSUPPORTED : TRI_ATTN_OK;
}

// rows that move in aligned 32-byte (codes: 16-byte) vectors of sixteen channels
bool vec_rows(const void* p, int64_t stride, int64_t elem) { return aligned_to(p, 32) && stride * elem % 32 == 0; }
bool vec_act8(const tri_act8& a) { return aligned_to(a.codes, 16) && a.codes_stride % 16 == 0; }

struct NormShape {
    int mode, lanes, threads;
    int64_t per_block;
};
// alone: the 8-bit activation by itself, whose rows of 65 to 128 channels go by 8 lanes (see kBy8)
NormShape norm_shape(int C, bool vec, bool alone = false) {
    const int units = (C + 15) / 16;
    NormShape s{};
    s.threads = tri::kNormThreads;
    s.mode = vec                ? tri::kVec
             : units <= 4       ? tri::kBy4
             : C <= 128         ? (alone ? tri::kBy8 : tri::kBy32Quarter)
             : C <= 256         ? tri::kBy32Half
                                : tri::kBy32;
    if (units > 32)
        s.lanes = s.threads = (units + 31) / 32 * 32;
    else if (!vec)
        s.lanes = tri::norm_stride(s.mode);
    else
        for (s.lanes = 1; s.lanes < units;) s.lanes *= 2;
    s.per_block = s.threads / s.lanes;
    return s;
}
// blocks of the backward: a function of the sizes, the alignment and of whether dw and db are
// wanted (sums) alone, like every order of additions there
int64_t norm_bwd_blocks(int64_t R, int C, bool vec, bool sums) {
    const NormShape s = norm_shape(C, vec);
    // few rows: one block goes through them, and the launch that adds up partial sums is saved
    // (64 rows of 128: 17.5 us of host time and 4.4 us of the device's, against 19.7 and 6.4);
    // without sums there is no such launch (128 rows of 128: 2.2 us, in one block 3.4)
    if (sums && R > 0 && R <= 4 * s.per_block) return 1;
    return std::min<int64_t>((R + s.per_block - 1) / s.per_block, 148 * (s.lanes > 32 ? 4 : tri::norm_bwd_per_sm(s.mode)));
}

void norm_params(NormParams& p, const tri_norm_fwd_args& a, const NormShape& s) {
    p.R = a.R;
    p.C = a.C;
    p.lanes = s.lanes;
    p.inv_c = 1.0f / static_cast<float>(a.C);
    p.eps = a.eps;
    p.x = a.x;
    p.xs = a.x_stride;
    p.w = a.w;
    p.b = a.b;
    p.w_bf16 = a.w_type == TRI_TYPE_BF16;
    p.y = a.y;
    p.ys = a.y_stride;
    p.stats = a.stats;
    p.codes = static_cast<uint8_t*>(a.act.codes);
    p.cs = a.act.codes_stride;
    p.exps = static_cast<uint8_t*>(a.act.exps);
    p.es = a.act.exps_stride;
}

// f(TX, TY) for the two element types, as default-constructed values
template <typename F>
void with_types(int tx, int ty, F&& f) {
    if (tx == TRI_TYPE_BF16)
        ty == TRI_TYPE_BF16 ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, float{});
    else
        ty == TRI_TYPE_BF16 ? f(float{}, __nv_bfloat16{}) : f(float{}, float{});
}
template <int V>
using Int = std::integral_constant<int, V>;
template <typename F>
void with_kind(int kind, F&& f) {
    if (kind == TRI_ACT8_INT8)
        f(Int<tri::ACT_INT8>{});
    else
        f(Int<tri::ACT_E4M3>{});
}
template <typename F>
void with_bool(bool v, F&& f) {
    v ? f(std::true_type{}) : f(std::false_type{});
}

// f(how the lanes share a row, whether a row takes a whole block)
template <bool ALONE, typename F>
void with_mode(const NormShape& s, F&& f) {
    constexpr int kTo128 = ALONE ? tri::kBy8 : tri::kBy32Quarter;
    if (s.lanes > 32)
        s.mode == tri::kVec ? f(Int<tri::kVec>{}, std::true_type{}) : f(Int<tri::kBy32>{}, std::true_type{});
    else if (s.mode == tri::kVec)
        f(Int<tri::kVec>{}, std::false_type{});
    else if (s.mode == tri::kBy4)
        f(Int<tri::kBy4>{}, std::false_type{});
    else if (s.mode == kTo128)
        f(Int<kTo128>{}, std::false_type{});
    else
        s.mode == tri::kBy32Half ? f(Int<tri::kBy32Half>{}, std::false_type{}) : f(Int<tri::kBy32>{}, std::false_type{});
}

// the ordered sum of partial sums, its launch overlapping the end of the kernel that writes them
void launch_ordered_sum(const float* part, int64_t nparts, int n, float* out0, int n0, float* out1, cudaStream_t cs) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((n + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = cs;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, tri::tri_ordered_sum_kernel, part, static_cast<int>(nparts), n, out0, n0, out1);
}

tri_attn_status launched() { return cudaGetLastError() == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA; }

tri_attn_status norm_fwd_impl(const tri_norm_fwd_args* a, bool restore, tri_attn_stream_t stream) {
    if (!a) return TRI_ATTN_ERR_NULL;
    tri_attn_status st = check_norm_sizes(a->R, a->C);
    if (st) return st;
    if (!type_ok(a->y_type) || (!restore && !type_ok(a->x_type)) || ((a->w || a->b) && !type_ok(a->w_type)))
        return TRI_ATTN_ERR_DTYPE;
    if (!restore && !(std::isfinite(a->eps) && a->eps >= 0.f)) return TRI_ATTN_ERR_SHAPE;
    const int64_t xe = type_bytes(a->x_type), ye = type_bytes(a->y_type), we = type_bytes(a->w_type);
    if (!restore && (st = check_rows(a->x, a->R, a->C, a->x_stride, xe, false))) return st;
    if ((st = check_rows(a->y, a->R, a->C, a->y_stride, ye, true))) return st;
    if ((st = check_rows(a->stats, a->R, 1, 1, 4, false))) return st;
    if (!aligned_to(a->w, we) || !aligned_to(a->b, we)) return TRI_ATTN_ERR_ALIGN;
    const bool act = restore || a->act.kind != TRI_ACT8_NONE;
    if (act && (st = check_act8(a->act, a->R, a->C, !restore))) return st;
    if ((st = ensure_device())) return st;
    if (a->R == 0) return TRI_ATTN_OK;
    const bool vec = a->C % 16 == 0 && vec_rows(a->y, a->y_stride, ye) && (!act || vec_act8(a->act)) &&
                     (restore || vec_rows(a->x, a->x_stride, xe));
    const NormShape s = norm_shape(a->C, vec);
    NormParams p{};
    norm_params(p, *a, s);
    const int per_sm = s.lanes > 32 ? 8 : tri::norm_fwd_blocks(s.mode, !restore && xe == 4);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((a->R + s.per_block - 1) / s.per_block, 148 * per_sm));
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    with_mode<false>(s, [&](auto m, auto wd) {
        constexpr int MODE = decltype(m)::value;
        constexpr bool WIDE = decltype(wd)::value;
        with_types(restore ? a->y_type : a->x_type, a->y_type, [&](auto tx, auto ty) {
            using TX = decltype(tx);
            using TY = decltype(ty);
            if (restore) {
                if constexpr (std::is_same<TX, TY>::value)
                    with_kind(a->act.kind, [&](auto k) {
                        tri::tri_norm_fwd_kernel<TX, TY, decltype(k)::value, MODE, true, WIDE>
                            <<<grid, s.threads, 0, cs>>>(p);
                    });
            } else if (!act) {
                tri::tri_norm_fwd_kernel<TX, TY, tri::ACT_NONE, MODE, false, WIDE><<<grid, s.threads, 0, cs>>>(p);
            } else {
                with_kind(a->act.kind, [&](auto k) {
                    tri::tri_norm_fwd_kernel<TX, TY, decltype(k)::value, MODE, false, WIDE>
                        <<<grid, s.threads, 0, cs>>>(p);
                });
            }
        });
    });
    return launched();
}

tri_attn_status act8_impl(const tri_act8_args* a, bool pack, tri_attn_stream_t stream) {
    if (!a) return TRI_ATTN_ERR_NULL;
    const int64_t R = a->R, xs = a->x_stride;
    const int C = a->C, x_type = a->x_type;
    const tri_act8& act = a->act;
    void* x = a->x;
    if (R < 0 || R > (int64_t{1} << 40) || C < 1 || C > (1 << 30)) return TRI_ATTN_ERR_SHAPE;
    if (!type_ok(x_type)) return TRI_ATTN_ERR_DTYPE;
    const int64_t xe = type_bytes(x_type);
    tri_attn_status st = check_rows(x, R, C, xs, xe, !pack);
    if (st || (st = check_act8(act, R, C, pack)) || (st = ensure_device())) return st;
    if (R == 0) return TRI_ATTN_OK;
    const bool vec = C % 16 == 0 && vec_rows(x, xs, xe) && vec_act8(act);
    const int pieces = (C + 511) / 512;
    NormParams p{};
    p.R = R;
    p.C = C;
    const NormShape s = norm_shape(std::min(C, 512), vec, true);
    p.lanes = s.lanes;
    p.x = x;
    p.xs = xs;
    p.y = x;
    p.ys = xs;
    p.codes = static_cast<uint8_t*>(act.codes);
    p.cs = act.codes_stride;
    p.exps = static_cast<uint8_t*>(act.exps);
    p.es = act.exps_stride;
    const int64_t per = tri::kNormThreads / p.lanes, items = R * pieces;
    const int per_sm = 2 * tri::act8_blocks(s.mode);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((items + per - 1) / per, 148 * per_sm));
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    with_mode<true>(s, [&](auto m, auto wd) {
        if constexpr (!decltype(wd)::value)  // pieces are no wider than a warp
            with_types(x_type, x_type, [&](auto tx, auto ty) {
                using TX = decltype(tx);
                if constexpr (std::is_same<TX, decltype(ty)>::value)
                    with_kind(act.kind, [&](auto k) {
                        with_bool(pack, [&](auto pk) {
                            tri::tri_act8_kernel<TX, decltype(k)::value, decltype(m)::value, decltype(pk)::value>
                                <<<grid, tri::kNormThreads, 0, cs>>>(p);
                        });
                    });
            });
    });
    return launched();
}

// ---------------------------------------------------------------------------
// relative position bias
// ---------------------------------------------------------------------------
tri_attn_status check_relpos_sizes(int B, int H, int Nq, int Nk, int E) {
    constexpr int kMost = 1 << 30;  // row and key numbers plus a step stay within 32 bits
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || E < 1 || Nq > kMost || Nk > kMost) return TRI_ATTN_ERR_SHAPE;
    if (static_cast<double>(B) * Nq * ((static_cast<int64_t>(Nk) + 7) / 8) >= 2147483648.0) return TRI_ATTN_ERR_SHAPE;
    return H > 4096 || E > tri::kRelMaxEdges ? TRI_ATTN_ERR_UNSUPPORTED : TRI_ATTN_OK;
}

// what both directions share; no CUDA call
tri_attn_status check_relpos(const tri_relpos_fwd_args& a) {
    tri_attn_status st = check_relpos_sizes(a.B, a.H, a.Nq, a.Nk, a.E);
    if (st) return st;
    if (!a.edges || !a.pos_q || !a.pos_k || !a.group_q != !a.group_k) return TRI_ATTN_ERR_NULL;
    if (a.q_stride < 0 || a.k_stride < 0) return TRI_ATTN_ERR_STRIDE;
    for (const void* ptr : {a.edges, a.pos_q, a.pos_k, a.group_q, a.group_k})
        if (!aligned_to(ptr, 4)) return TRI_ATTN_ERR_ALIGN;
    return TRI_ATTN_OK;
}

void relpos_params(RelposParams& p, const tri_relpos_fwd_args& a) {
    p.B = a.B;
    p.H = a.H;
    p.Nq = a.Nq;
    p.Nk = a.Nk;
    p.E = a.E;
    p.nb = a.E + 1 + (a.group_q ? 1 : 0);
    p.chunks = (a.Nk + 7) / 8;
    p.table = a.table;
    p.table_bf16 = a.table_type == TRI_TYPE_BF16;
    p.edges = a.edges;
    p.pos_q = a.pos_q;
    p.pos_k = a.pos_k;
    p.grp_q = a.group_q;
    p.grp_k = a.group_k;
    p.qs = a.q_stride;
    p.ks = a.k_stride;
}

// launch shape of the backward: a function of the sizes alone
struct RelposBwdShape {
    int heads, head_blocks, warps, row_tasks, run;
    unsigned grid;
    size_t smem;
};
RelposBwdShape relpos_bwd_shape(int B, int H, int Nq, int Nk, int nb) {
    RelposBwdShape s{};
    // a warp's lanes: 8 chunks of four heads, 16 of two or 32 of one, or fewer chunks where there
    // are no more; of these the one that leaves the fewest lanes without work, the narrowest first
    // (the fewer keys a warp spans, the fewer of its rows have one of them near the diagonal)
    const int chunks = (Nk + 7) / 8;
    int64_t fewest = INT64_MAX;
    for (int heads = 32; heads >= 1; heads /= 2) {
        const int side = 32 / heads;
        const int64_t lanes =
            static_cast<int64_t>((chunks + side - 1) / side) * side * ((H + heads - 1) / heads * heads);
        if (lanes < fewest && (heads <= 4 || side >= chunks)) {
            fewest = lanes;
            s.heads = heads;
        }
    }
    s.head_blocks = (H + s.heads - 1) / s.heads;
    const int S = 32 / s.heads;
    const int64_t tiles = static_cast<int64_t>(B) * ((chunks + S - 1) / S);
    s.warps = tri::kRelBwdWarps;
    while (s.warps > 1 && tri::relpos_bwd_smem(nb, s.warps) > tri::kRelBwdSmem) --s.warps;
    s.smem = tri::relpos_bwd_smem(nb, s.warps);
    const int64_t at_once = 148 * tri::relpos_bwd_per_sm(s.smem);  // blocks
    // as many tasks as warps run at once, each with at least one batch of rows; those with many
    // take two in a row, so that the buckets in hand last longer
    const int64_t want = std::max<int64_t>(1, at_once * s.warps / (tiles * s.head_blocks));
    const int64_t batches = (Nq + tri::kRelRows - 1) / tri::kRelRows;
    s.row_tasks = static_cast<int>(std::min(want, batches));
    s.run = static_cast<int>(std::min<int64_t>(2, batches / s.row_tasks));
    const int64_t tasks = tiles * s.row_tasks;  // < 2^31: at most one per warp at once, or B * chunks of them
    // a few tasks: one block, as in the norm (64 x 64 x 4 heads: 17 us of host time, the device's
    // 12.6 us, against 19 and 10.5)
    const int64_t blocks = std::min<int64_t>((tasks + s.warps - 1) / s.warps, at_once);
    s.grid = tasks <= 4 * s.warps ? 1u : static_cast<unsigned>(blocks);
    return s;
}

}  // namespace

extern "C" {

tri_attn_status tri_norm_fwd(const tri_norm_fwd_args* a, tri_attn_stream_t stream) {
    return norm_fwd_impl(a, false, stream);
}

tri_attn_status tri_norm_restore(const tri_norm_fwd_args* a, tri_attn_stream_t stream) {
    return norm_fwd_impl(a, true, stream);
}

size_t tri_norm_bwd_workspace_bytes(int64_t R, int C) {
    if (check_norm_sizes(R, C)) return 0;
    // never 0 for sizes that are valid
    const int64_t blocks = std::max(norm_bwd_blocks(R, C, false, true), norm_bwd_blocks(R, C, true, true));
    return static_cast<size_t>(std::max<int64_t>(1, blocks)) * 2 * C * sizeof(float);
}

tri_attn_status tri_norm_bwd(const tri_norm_bwd_args* a, tri_attn_stream_t stream) {
    if (!a) return TRI_ATTN_ERR_NULL;
    const tri_norm_fwd_args& f = a->f;
    tri_attn_status st = check_norm_sizes(f.R, f.C);
    if (st) return st;
    if (!type_ok(f.x_type) || !type_ok(f.y_type) || (f.w && !type_ok(f.w_type))) return TRI_ATTN_ERR_DTYPE;
    const int64_t xe = type_bytes(f.x_type), ye = type_bytes(f.y_type);
    const bool act = f.act.kind != TRI_ACT8_NONE;
    if (act ? (st = check_act8(f.act, f.R, f.C, false)) : (st = check_rows(f.x, f.R, f.C, f.x_stride, xe, false)))
        return st;
    if ((st = check_rows(a->dy, f.R, f.C, a->dy_stride, ye, false))) return st;
    if (a->dx && (st = check_rows(a->dx, f.R, f.C, a->dx_stride, xe, true))) return st;
    if ((st = check_rows(f.stats, f.R, 1, 1, 4, false))) return st;
    if (!a->dw != !a->db) return TRI_ATTN_ERR_NULL;
    if (!aligned_to(f.w, type_bytes(f.w_type)) || !aligned_to(a->dw, 4) || !aligned_to(a->db, 4))
        return TRI_ATTN_ERR_ALIGN;
    if (a->dw) {
        if (!a->workspace || a->workspace_bytes < tri_norm_bwd_workspace_bytes(f.R, f.C)) return TRI_ATTN_ERR_WORKSPACE;
        if (!aligned16(a->workspace)) return TRI_ATTN_ERR_ALIGN;
    }
    if ((st = ensure_device())) return st;
    if (!a->dx && !a->dw) return TRI_ATTN_OK;
    const bool vec = f.C % 16 == 0 && vec_rows(a->dy, a->dy_stride, ye) &&
                     (!a->dx || vec_rows(a->dx, a->dx_stride, xe)) &&
                     (act ? vec_act8(f.act) : vec_rows(f.x, f.x_stride, xe));
    const NormShape s = norm_shape(f.C, vec);
    const int64_t blocks = norm_bwd_blocks(f.R, f.C, vec, a->dw != nullptr);
    NormParams p{};
    norm_params(p, f, s);
    p.dy = a->dy;
    p.dys = a->dy_stride;
    p.dx = f.R ? a->dx : nullptr;
    p.dxs = a->dx_stride;
    p.partial = a->dw ? static_cast<float*>(a->workspace) : nullptr;
    p.dw = a->dw;
    p.db = a->db;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (blocks) {
        with_mode<false>(s, [&](auto m, auto wd) {
            constexpr int MODE = decltype(m)::value;
            constexpr bool WIDE = decltype(wd)::value;
            with_types(f.x_type, f.y_type, [&](auto tx, auto ty) {
                using TX = decltype(tx);
                using TY = decltype(ty);
                const unsigned grid = static_cast<unsigned>(blocks);
                if (!act)
                    tri::tri_norm_bwd_kernel<TX, TY, tri::ACT_NONE, MODE, WIDE><<<grid, s.threads, 0, cs>>>(p);
                else
                    with_kind(f.act.kind, [&](auto k) {
                        tri::tri_norm_bwd_kernel<TX, TY, decltype(k)::value, MODE, WIDE><<<grid, s.threads, 0, cs>>>(p);
                    });
            });
        });
    }
    if (a->dw && blocks != 1)  // with no rows: zeros
        launch_ordered_sum(p.partial, blocks, 2 * f.C, a->dw, f.C, a->db, cs);
    return launched();
}

tri_attn_status tri_act8_pack(const tri_act8_args* a, tri_attn_stream_t stream) { return act8_impl(a, true, stream); }

tri_attn_status tri_act8_unpack(const tri_act8_args* a, tri_attn_stream_t stream) {
    return act8_impl(a, false, stream);
}

tri_attn_status tri_relpos_fwd(const tri_relpos_fwd_args* a, tri_attn_stream_t stream) {
    if (!a) return TRI_ATTN_ERR_NULL;
    tri_attn_status st = check_relpos(*a);
    if (st) return st;
    if (!a->table) return TRI_ATTN_ERR_NULL;
    if (!type_ok(a->table_type)) return TRI_ATTN_ERR_DTYPE;
    if (!aligned_to(a->table, type_bytes(a->table_type))) return TRI_ATTN_ERR_ALIGN;
    if ((st = check_t4(a->bias)) || (a->base.ptr && (st = check_t4(a->base)))) return st;
    const int64_t extent[3] = {a->B, a->H, a->Nq};
    for (int x = 0; x < 3; ++x)
        if (extent[x] > 1 && a->bias.stride[x] < a->Nk) return TRI_ATTN_ERR_STRIDE;
    if ((st = ensure_device())) return st;
    RelposParams p{};
    relpos_params(p, *a);
    p.heads = std::min(a->H, tri::kRelHeads);
    p.base = static_cast<const __nv_bfloat16*>(a->base.ptr);
    p.bias = static_cast<__nv_bfloat16*>(a->bias.ptr);
    for (int x = 0; x < 3; ++x) {
        p.bs[x] = a->base.stride[x];
        p.os[x] = a->bias.stride[x];
    }
    // all blocks run at once, and hold at least one row of chunks
    const int64_t items = static_cast<int64_t>(a->B) * a->Nq * p.chunks, threads = tri::kRelThreads;
    // few rows: the heads go to blocks of their own, more than four halved, which leaves two to four
    // (one row of 4096 keys with 16 heads runs on 8 blocks in place of 2).  Table entries hold four
    // heads, but keeping to fours gains nothing: 8 x 64 with 5 heads and a base 4.0 us, by fours 4.8;
    // one row of 4096 keys with 12 heads 4.0 either way
    while (p.heads > 4 && (items + threads - 1) / threads * ((a->H + p.heads - 1) / p.heads) < 74) p.heads /= 2;
    const unsigned head_blocks = (a->H + p.heads - 1) / p.heads;
    const int64_t at_once =
        std::max<int64_t>(148 * tri::kRelFwdBlocks / head_blocks, (p.chunks + threads - 1) / threads);
    const dim3 grid(static_cast<unsigned>(std::min((items + threads - 1) / threads, at_once)), head_blocks);
    const size_t smem = tri::relpos_fwd_smem(p.nb, p.heads, p.base != nullptr);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    with_bool(p.base != nullptr, [&](auto v) {
        tri::tri_relpos_fwd_kernel<decltype(v)::value><<<grid, tri::kRelThreads, smem, cs>>>(p);
    });
    return launched();
}

size_t tri_relpos_bwd_workspace_bytes(int B, int H, int Nq, int Nk, int E, int groups) {
    if (check_relpos_sizes(B, H, Nq, Nk, E)) return 0;
    const int nb = E + 1 + (groups ? 1 : 0);
    return static_cast<size_t>(relpos_bwd_shape(B, H, Nq, Nk, nb).grid) * nb * H * sizeof(float);
}

tri_attn_status tri_relpos_bwd(const tri_relpos_bwd_args* a, tri_attn_stream_t stream) {
    if (!a) return TRI_ATTN_ERR_NULL;
    const tri_relpos_fwd_args& f = a->f;
    tri_attn_status st = check_relpos(f);
    if (st || (st = check_t4(a->dbias))) return st;
    if (!a->dtable) return TRI_ATTN_ERR_NULL;
    if (!aligned_to(a->dtable, 4)) return TRI_ATTN_ERR_ALIGN;
    if (!a->workspace ||
        a->workspace_bytes < tri_relpos_bwd_workspace_bytes(f.B, f.H, f.Nq, f.Nk, f.E, f.group_q != nullptr))
        return TRI_ATTN_ERR_WORKSPACE;
    if (!aligned16(a->workspace)) return TRI_ATTN_ERR_ALIGN;
    if ((st = ensure_device())) return st;
    RelposParams p{};
    relpos_params(p, f);
    const RelposBwdShape s = relpos_bwd_shape(f.B, f.H, f.Nq, f.Nk, p.nb);
    p.heads = s.heads;
    p.row_tasks = s.row_tasks;
    p.run = s.run;
    p.partial = s.grid == 1 ? a->dtable : static_cast<float*>(a->workspace);  // the same layout
    p.dbias = static_cast<const __nv_bfloat16*>(a->dbias.ptr);
    for (int x = 0; x < 3; ++x) p.ds[x] = a->dbias.stride[x];
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    with_bool(p.grp_q != nullptr, [&](auto v) {
        tri::tri_relpos_bwd_kernel<decltype(v)::value><<<dim3(s.grid, s.head_blocks), s.warps * 32, s.smem, cs>>>(p);
    });
    const int n = p.nb * f.H;
    if (s.grid > 1) launch_ordered_sum(p.partial, s.grid, n, a->dtable, n, nullptr, cs);
    return launched();
}

}  // extern "C"
