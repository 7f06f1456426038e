/*
 * tri_attn.h -- C ABI of the B200 (sm_100a) triangle-attention library
 * (libtriattn.so).  Plain pointers and sizes only; no framework types.
 *
 * What it computes.  Triangle attention around the starting node of an
 * AlphaFold3 / OpenFold3 Pairformer pair tensor: for batch b, pair row i,
 * head h and query j,
 *
 *   out[b,i,j,h,:] = sum_k softmax_k( scale * q[b,i,j,h,:].k[b,i,k,h,:]
 *                                     + bias[b,h,j,k] + mask[b,i,k] ) v[b,i,k,h,:]
 *
 * with ONE pair bias shared by all N rows i, so the work is cubic in the crop
 * size N and the bias gradient is a reduction over rows.  Pages this follows:
 *   (A) "16张H100，训练步提速1.73倍：TurboPairFormer为什么不是'装个包就能加速AlphaFold3'"
 *       (biocloudservice.com), sections "先看清'1.73倍'对应什么" (cubic cost) and
 *       "它优化了什么，而不是只'少存一点张量'" (the four gradients and the shared
 *       pair bias; the BF16 output-rounding residual with an FP32 correction);
 *   (B) "TurboPairFormer: более быстрое, стабильное и точное дообучение OpenFold3"
 *       (dev48.org), section "Как работает TurboPairFormer" (probabilities
 *       recomputed in the backward, residual compensation, fixed accumulation
 *       order giving bitwise-identical gradients).
 *
 * Ending-node orientation is the same operation on the transposed pair
 * tensor: pass every 5-D tensor (inputs AND outputs) with stride[1] and
 * stride[2] swapped.  bias and mask are always given in the attention's own
 * frame ((j,k) and (i,k)); the caller builds them from the transposed pair
 * representation, as AlphaFold does.
 *
 * Conventions (every entry point):
 *  - Ownership: the caller allocates and frees every buffer (inputs, outputs,
 *    saved forward state, workspace).  The library never allocates device or
 *    host memory for data, never frees, and never synchronises the stream.
 *  - Asynchrony: work is enqueued on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream).  Argument errors are detected on the host and
 *    returned before anything is enqueued; nothing is launched on error.
 *  - Device: the current CUDA device must be compute capability 10.0
 *    (B200, sm_100a); otherwise TRI_ATTN_ERR_ARCH.
 *  - Types: q, k, v, bias, dout, o, resid and all gradients are BF16; mask
 *    and lse are FP32.
 *  - Strides are in ELEMENTS.  The innermost (channel / key) stride must be 1;
 *    every other stride must be a non-negative multiple of 8 elements (16
 *    bytes) except the mask's, which may be anything (0 broadcasts).  Data
 *    pointers must be 16-byte aligned (mask: 4-byte).
 *  - Supported sizes: 1 <= B, 1 <= N <= 4096, 1 <= H, d in {32, 64}.
 *  - Rows whose every key is masked (all mask values <= -1e8) are outside
 *    the contract: their outputs are unspecified.
 *  - Determinism: for fixed inputs and shapes every output is bitwise
 *    identical from run to run (no floating-point atomics; every reduction
 *    has a fixed order independent of scheduling and SM count).
 *  - Thread safety: all entry points are reentrant.
 */
#ifndef TRI_ATTN_H
#define TRI_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TRI_ATTN_ABI_VERSION 1

/* A cudaStream_t without pulling in the CUDA headers. */
typedef struct CUstream_st *tri_attn_stream_t;

typedef enum {
    TRI_ATTN_OK = 0,
    TRI_ATTN_ERR_NULL = 1,           /* a required pointer is NULL                     */
    TRI_ATTN_ERR_SHAPE = 2,          /* a size or scalar out of range                  */
    TRI_ATTN_ERR_STRIDE = 3,         /* innermost stride != 1, or a stride that the call
                                        does not take                                */
    TRI_ATTN_ERR_ALIGN = 4,          /* a data pointer is not aligned as the call asks */
    TRI_ATTN_ERR_DTYPE = 5,          /* wrong element type                             */
    TRI_ATTN_ERR_UNSUPPORTED = 6,    /* a size past the call's limit (d not in {32, 64},
                                        N > 4096, C > 8192, ...) or an unknown option  */
    TRI_ATTN_ERR_WORKSPACE = 7,      /* workspace NULL or smaller than required        */
    TRI_ATTN_ERR_ARCH = 8,           /* current device is not sm_100                   */
    TRI_ATTN_ERR_CUDA = 9,           /* a CUDA runtime/driver call failed              */
    TRI_ATTN_ERR_DEVICE_TIMEOUT = 10, /* a kernel's bounded wait expired (see
                                        tri_attn_device_error)                        */
    TRI_ATTN_ERR_SCRATCH_LIMIT = 11  /* the sizes need more scratch than
                                        TRI_ATTN_STATIC_SCRATCH_BYTES (only from
                                        tri_attn_bwd_static_scratch)                 */
} tri_attn_status;

/* BF16 pair tensor [B,N,N,H,d]; stride[] = element strides of (b,i,j,h,c), c-stride 1. */
typedef struct {
    void *ptr;
    int64_t stride[5];
} tri_attn_tensor5;

/* BF16 bias / bias gradient [B,H,N,N]; stride[] = element strides of (b,h,j,k), k-stride 1. */
typedef struct {
    void *ptr;
    int64_t stride[4];
} tri_attn_tensor4;

/* FP32 additive mask [B,N,N] indexed (b,i,k); ptr may be NULL (no mask); any strides. */
typedef struct {
    const float *ptr;
    int64_t stride[3];
} tri_attn_mask;

/*
 * Forward arguments.
 *   q, k, v, bias, mask : inputs (read only)
 *   o     : output, BF16 round-to-nearest-even of the FP32 result O32
 *   resid : output, BF16 RNE of (O32 - float(o)), the output-rounding residual
 *           (page A, section "它优化了什么": saved so that the backward's softmax
 *           correction can be formed in FP32 from o + resid)
 *   lse   : output, FP32 log-sum-exp of each softmax row (natural log), a
 *           contiguous [B,H,N,N] array indexed (b,h,i,j)
 *   scale : multiplies q.k only; 0 means 1/sqrt(d)
 */
typedef struct {
    int B, N, H, d;
    float scale;
    tri_attn_tensor5 q, k, v;
    tri_attn_tensor4 bias;
    tri_attn_mask mask;
    tri_attn_tensor5 o, resid;
    float *lse;
} tri_attn_fwd_args;

/* Backward flag: form the softmax correction D from o alone, ignoring resid
 * (the uncompensated variant, for measuring what the residual buys). */
#define TRI_ATTN_BWD_NO_RESIDUAL 1u

/*
 * Backward arguments.
 *   f     : the forward's inputs plus its saved state (o, resid, lse), all read only
 *   dout  : upstream gradient of o (read only)
 *   dq, dk, dv : outputs, BF16, same layout rules as q
 *   dbias : output, BF16 [B,H,N,N], the sum over rows i of the score gradient
 *   workspace, workspace_bytes : caller-owned device scratch of at least
 *           tri_attn_bwd_workspace_bytes(B,N,H,d) bytes, 256-byte aligned;
 *           contents on entry are ignored and on exit are unspecified
 *   flags : 0, or TRI_ATTN_BWD_NO_RESIDUAL
 * No gradient is produced for mask.
 */
typedef struct {
    tri_attn_fwd_args f;
    tri_attn_tensor5 dout;
    tri_attn_tensor5 dq, dk, dv;
    tri_attn_tensor4 dbias;
    void *workspace;
    size_t workspace_bytes;
    unsigned flags;
} tri_attn_bwd_args;

/* Enqueue the forward on `stream`.  Returns TRI_ATTN_OK or the first argument
 * error found (nothing enqueued), or TRI_ATTN_ERR_CUDA if a launch failed. */
tri_attn_status tri_attn_fwd(const tri_attn_fwd_args *args, tri_attn_stream_t stream);

/* Bytes of device workspace tri_attn_bwd needs for these sizes (a pure
 * function of the sizes; 0 for invalid sizes).  No device access. */
size_t tri_attn_bwd_workspace_bytes(int B, int N, int H, int d);

/* Enqueue the backward (dq, dk, dv, dbias) on `stream`.  Same error rules as
 * tri_attn_fwd, plus TRI_ATTN_ERR_WORKSPACE. */
tri_attn_status tri_attn_bwd(const tri_attn_bwd_args *args, tri_attn_stream_t stream);

/* tri_attn_bwd with timing markers: `markers` is NULL or an array of four
 * cudaEvent_t handles (as void*) that are recorded on `stream` before the
 * D pre-pass, before the dq/dk/dv kernel, before the dbias kernel(s) and
 * after the last kernel, so a caller can time each phase with the events it
 * owns.  Otherwise identical to tri_attn_bwd. */
tri_attn_status tri_attn_bwd_marked(const tri_attn_bwd_args *args, tri_attn_stream_t stream,
                                    void *const *markers);

/* ---------------------------------------------------------------------------
 * Row shards: a 1-D split of the rows i across devices, the row sharding of
 * the pair representation in "Design-CP: Context Parallelism for Design of
 * Protein Nanoparticles" (gist.science summary), section "方法论", item
 * "1. 推理策略" (1D row sharding).  The problems of
 * different rows i are independent except for dBias, the sum over i of the
 * score gradient: each shard returns its share of that sum in FP32, and
 * tri_attn_dbias_sum adds the shares of all shards in a fixed order.
 *
 * A shard call covers rows i0 .. i0+rows-1 of the full problem:
 *   args->N            : the full N (the j and k extent; bias is [B,H,N,N])
 *   q,k,v,o,resid,dout,dq,dk,dv : point at row i0 (strides unchanged)
 *   mask.ptr           : points at row i0 (if not NULL)
 *   lse                : this shard's own contiguous FP32 [B,H,rows,N] array
 *   1 <= rows <= N, else TRI_ATTN_ERR_SHAPE.
 * With rows = N and no offset, tri_attn_fwd_rows equals tri_attn_fwd bit for
 * bit, and so do the o, resid, lse, dq, dk, dv of a shard and of the whole.
 * --------------------------------------------------------------------------- */
tri_attn_status tri_attn_fwd_rows(const tri_attn_fwd_args *args, int rows, tri_attn_stream_t stream);

/* Workspace bytes of tri_attn_bwd_rows (pure function; 0 for invalid sizes). */
size_t tri_attn_bwd_rows_workspace_bytes(int B, int rows, int N, int H, int d);

/* Number P of FP32 dBias partial sums tri_attn_bwd_rows writes for these sizes
 * (pure function, the same for every shard of equal rows; 0 if invalid). */
int tri_attn_bwd_rows_dbias_parts(int B, int rows, int N, int H, int d);

/* Backward of one shard: dq, dk, dv of its rows as tri_attn_bwd does, and its
 * share of dBias as P contiguous FP32 [B,H,N,N] arrays in dbias_parts
 * (caller-owned, 16-byte aligned, P * B*H*N*N floats, overwritten); their sum
 * is the shard's sum over its rows of the score gradient.  args->dbias is not
 * used.  Workspace: tri_attn_bwd_rows_workspace_bytes. */
tri_attn_status tri_attn_bwd_rows(const tri_attn_bwd_args *args, int rows, float *dbias_parts,
                                  tri_attn_stream_t stream);

/* dbias = BF16 RNE of the sum of nparts contiguous FP32 [B,H,N,N] arrays,
 * added in ascending index order (the shards' partials gathered in rank
 * order: every device that calls this on the same gathered array gets the
 * same bits).  parts 16-byte aligned; dbias strides as in tri_attn_bwd. */
tri_attn_status tri_attn_dbias_sum(const float *parts, int nparts, int B, int H, int N, tri_attn_tensor4 dbias,
                                   tri_attn_stream_t stream);

/* Size of the static scratch area of tri_attn_bwd_static_scratch, per device:
 * 64 MiB, enough for every size whose tri_attn_bwd_workspace_bytes is at most
 * that (for example B=1, N=768, H=4 at d=32 or d=64). */
#define TRI_ATTN_STATIC_SCRATCH_BYTES (64ull << 20)

/*
 * The backward without any device allocation.  The method's pages have no
 * counterpart to this: it is a service of the library, for callers that must
 * not allocate device memory on the path where the backward runs (an
 * application whose allocator owns all device memory, or a latency-critical
 * loop where cudaMalloc / cudaFree, which can synchronise the device, are not
 * allowed).  It runs exactly the kernels of tri_attn_bwd and returns the same
 * results, but its scratch is a fixed array of TRI_ATTN_STATIC_SCRATCH_BYTES
 * in the library's own device memory, reserved when the library's module for
 * it is loaded onto a device; args->workspace and args->workspace_bytes are
 * ignored.
 *   - Order of checks: the argument errors of tri_attn_bwd first (on the
 *     host, before any CUDA call), then the limit: sizes whose
 *     tri_attn_bwd_workspace_bytes(B,N,H,d) exceeds
 *     TRI_ATTN_STATIC_SCRATCH_BYTES are rejected with
 *     TRI_ATTN_ERR_SCRATCH_LIMIT before anything is enqueued.
 *   - Set-up: the first call on each device (the current device at the call)
 *     looks up the array's device address, which loads the module there; call
 *     it once on each device before any stream capture begins, so that this
 *     set-up happens outside a capture.  The address is kept per device
 *     together with the CUDA context it belongs to; after a device reset (a
 *     new context) the next call looks it up again, so that call is a set-up
 *     call too.
 *   - Initial contents: nothing in the scratch has to start at zero; every
 *     word the kernels read is written earlier in the same call.
 *   - Races: all calls on one device share the one array.  Two calls whose
 *     work can overlap on the device (different streams without an ordering
 *     event between them, or several host threads) race on it and produce
 *     wrong gradients; order them, for example on one stream.
 * Otherwise the same arguments and error rules as tri_attn_bwd.
 */
tri_attn_status tri_attn_bwd_static_scratch(const tri_attn_bwd_args *args, tri_attn_stream_t stream);

/* ---------------------------------------------------------------------------
 * Triangle multiplicative update: the contraction step.
 *
 * The pages name the Triangle Multiplicative Update as the second operation
 * TurboPairFormer optimises beside triangle attention (page A, opening
 * paragraph; page B, the paragraph introducing TurboPairFormer) without a
 * formula; read the AlphaFold way, its only cubic step contracts two projected
 * pair tensors over the third residue k, for every batch b and channel c:
 *   outgoing edges (flags 0):            x[b,c,i,j] = sum_k a[b,c,i,k] b[b,c,j,k]
 *   incoming edges (TRI_MUL_INCOMING):   x[b,c,i,j] = sum_k a[b,c,k,i] b[b,c,k,j]
 * The projections, gates and LayerNorms around it are per-position work of the
 * model and are not part of this call.
 *   a, b, x : BF16 [B,C,N,N], channel-first (the caller permutes the
 *             channel-last pair representation), strides as tri_attn_tensor4
 *             with (b, c, row, col) in place of (b, h, j, k): innermost stride
 *             1, the others non-negative multiples of 8 elements, pointers
 *             16-byte aligned
 *   x       : output, BF16 round-to-nearest-even of the FP32 sum
 * Sizes: 1 <= B, 1 <= C, B*C <= 65535, 1 <= N <= 16384.  Same ownership,
 * asynchrony, error and determinism rules as the attention calls.
 */
#define TRI_MUL_INCOMING 1u

typedef struct {
    int B, C, N;
    tri_attn_tensor4 a, b;
    tri_attn_tensor4 x;
    unsigned flags; /* 0 (outgoing edges) or TRI_MUL_INCOMING */
} tri_mul_fwd_args;

/* Backward of the contraction: given dx (the upstream gradient of x), writes
 *   outgoing:  da[i,k] = sum_j dx[i,j] b[j,k]     db[j,k] = sum_i dx[i,j] a[i,k]
 *   incoming:  da[k,i] = sum_j dx[i,j] b[k,j]     db[k,j] = sum_i dx[i,j] a[k,i]
 * (BF16 outputs from FP32 sums).  f.a, f.b and f.flags as in the forward;
 * f.x is not used. */
typedef struct {
    tri_mul_fwd_args f;
    tri_attn_tensor4 dx;
    tri_attn_tensor4 da, db;
} tri_mul_bwd_args;

tri_attn_status tri_mul_fwd(const tri_mul_fwd_args *args, tri_attn_stream_t stream);
tri_attn_status tri_mul_bwd(const tri_mul_bwd_args *args, tri_attn_stream_t stream);

/* ---------------------------------------------------------------------------
 * Gated output projection around the attention (no counterpart on the pages,
 * which describe the attention itself; the AlphaFold-style steps on either
 * side of it, fused):  for every pair position r,
 *     g = sigmoid(z[r,:] Wg),   y[r,:] = (g * o[r,:]) Wo
 *   z  : BF16 [R, 128], the attention block's pair input (cz = 128)
 *   o  : BF16 [R, 128], the attention output with heads concatenated (H*d = 128)
 *   wg : BF16 [128, 128] row-major, wg[cz][co];  wo: BF16 [128, 128], wo[co][cz]
 *   y  : BF16 [R, 128] output (RNE of the FP32 result)
 * Row strides in elements (multiples of 8); pointers 16-byte aligned; R >= 1.
 * No biases.  Same ownership, asynchrony and error rules as the other calls.
 */
typedef struct {
    int R;
    const void *z;
    int64_t z_stride;
    const void *o;
    int64_t o_stride;
    const void *wg, *wo;
    void *y;
    int64_t y_stride;
} tri_gate_fwd_args;

tri_attn_status tri_gate_fwd(const tri_gate_fwd_args *args, tri_attn_stream_t stream);

/* Backward of tri_gate_fwd for the upstream gradient dy (a = g * o):
 *     dA = dy Wo^T,  do = dA * g,  dl = dA * o * g * (1 - g),
 *     dz = dl Wg^T,  dWo = sum_r a^T dy,  dWg = sum_r z^T dl
 *   f      : the forward's arguments (f.y is not used)
 *   dy     : BF16 [R, 128] upstream gradient
 *   dz, d_o: BF16 [R, 128] outputs (overwritten)
 *   dwg    : FP32 [128, 128] row-major, dwg[cz][co] (overwritten)
 *   dwo    : FP32 [128, 128] row-major, dwo[co][cz] (overwritten)
 *   workspace, workspace_bytes : caller-owned device scratch of at least
 *            tri_gate_bwd_workspace_bytes(R) bytes, 16-byte aligned (partial
 *            weight-gradient sums of each CTA).
 * The weight gradients are summed in a fixed order, so repeated calls with the
 * same inputs give bitwise-identical results.  Strides, alignment and errors
 * as for tri_gate_fwd; TRI_ATTN_ERR_WORKSPACE if the workspace is NULL or too
 * small. */
typedef struct {
    tri_gate_fwd_args f;
    const void *dy;
    int64_t dy_stride;
    void *dz;
    int64_t dz_stride;
    void *d_o;
    int64_t do_stride;
    float *dwg, *dwo;
    void *workspace;
    size_t workspace_bytes;
} tri_gate_bwd_args;

/* Bytes of workspace tri_gate_bwd needs for R pair positions (pure function;
 * 0 for R < 1). */
size_t tri_gate_bwd_workspace_bytes(int R);

tri_attn_status tri_gate_bwd(const tri_gate_bwd_args *args, tri_attn_stream_t stream);

/* ---------------------------------------------------------------------------
 * The pair block's per-position steps around the attention (no counterpart on
 * the pages, which describe the attention itself): the layer norm in front of
 * it, an 8-bit form of an activation kept for the backward pass, and a learned
 * relative position bias in the layout the attention reads.  Ownership,
 * asynchrony, determinism and error rules as for the other calls.
 *
 * Element types: a field named *_type holds TRI_TYPE_BF16 or TRI_TYPE_F32
 * (else TRI_ATTN_ERR_DTYPE).  Rows are R rows of C channels with channel
 * stride 1 and the given row stride in elements: any stride of at least C for
 * what is written (so that rows do not overlap), any non-negative stride for
 * what is read.  Pointers need the alignment of their element type only;
 * 32-byte aligned data with row strides of a multiple of 32 bytes and C a
 * multiple of 16 runs fastest.  Outputs do not overlap inputs.  Channels past
 * C and rows past R are left as they were.  Sizes: 0 <= R (nothing to do at
 * 0, except that weight gradients are written as zeros), 1 <= C <= 8192.
 */
#define TRI_TYPE_BF16 0
#define TRI_TYPE_F32 1

#define TRI_ACT8_NONE 0
#define TRI_ACT8_INT8 1 /* codes are two's complement, -127 .. 127                  */
#define TRI_ACT8_E4M3 2 /* codes are e4m3 floats (no infinities), largest 448        */

/* Channels that share a scale: blocks start at multiples of 32 of a row, the
 * last one may be cut short by C. */
#define TRI_ACT8_BLOCK 32

/* An activation in 8 bits: codes [R,C] (one byte each, row stride in bytes)
 * and exponents [R, ceil(C/32)] (one byte each, row stride in bytes), both
 * with unit inner stride.  A block with largest magnitude m is stored under
 * the scale 2^e, e the least integer >= -126 with m <= Q 2^e, where Q = 127
 * (INT8) or 448 (E4M3); its exponent byte is e + 127.  Each code is the
 * nearest one to value / 2^e, ties to even, and stands for code * 2^e.  A
 * block that holds an infinity or a NaN gets the exponent byte 255 and codes
 * 0, and is restored as NaNs.  (Magnitudes within a code's half step of 2^128
 * are restored as 2^128, which is an infinity in both element types.)  kind TRI_ACT8_NONE: no activation is given. */
typedef struct {
    void *codes;
    int64_t codes_stride;
    void *exps;
    int64_t exps_stride;
    int kind;
} tri_act8;

/* Layer norm over the channels of each row, forward:
 *     mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps),
 *     y = (x - mean) * rstd * w + b
 * in FP32 (so |x - mean| stays below some 1e18, the root of its range).
 *   x     : [R,C] input;  w, b : contiguous [C] of type w_type, either may be
 *           NULL (1 and 0)
 *   y     : [R,C] output, rounded once from FP32
 *   stats : FP32, contiguous [2,R] output: the R means, then the R rstds
 *   act   : TRI_ACT8_NONE, or an output: x in 8 bits, for tri_norm_restore,
 *           tri_norm_bwd and tri_act8_unpack
 *   eps   : finite, not negative */
typedef struct {
    int64_t R;
    const void *x;
    int64_t x_stride;
    const void *w, *b;
    void *y;
    int64_t y_stride;
    float *stats;
    tri_act8 act;
    int C, x_type, w_type, y_type;
    float eps;
} tri_norm_fwd_args;

tri_attn_status tri_norm_fwd(const tri_norm_fwd_args *args, tri_attn_stream_t stream);

/* y of tri_norm_fwd once more, from what was kept of x: act and stats are
 * read, y is written; x, x_type and eps are not used. */
tri_attn_status tri_norm_restore(const tri_norm_fwd_args *args, tri_attn_stream_t stream);

/* Layer norm, backward, with h = (x - mean) * rstd and g = dy * w:
 *     dx = rstd * (g - mean_c(g) - h * mean_c(g h)),
 *     dw = sum_r dy h,   db = sum_r dy
 *   f      : the forward's R, C, w, w_type, stats, and x with x_type, or, with
 *            f.act.kind set, act in place of x (f.x is then not used); b, y and
 *            eps are not used
 *   dy     : [R,C] upstream gradient of type f.y_type
 *   dx     : [R,C] output of type f.x_type, or NULL
 *   dw, db : FP32 contiguous [C] outputs, or both NULL
 *   workspace, workspace_bytes : caller-owned device scratch of at least
 *            tri_norm_bwd_workspace_bytes(R, C) bytes, 16-byte aligned; not
 *            used when dw and db are NULL */
typedef struct {
    tri_norm_fwd_args f;
    const void *dy;
    int64_t dy_stride;
    void *dx;
    int64_t dx_stride;
    float *dw, *db;
    void *workspace;
    size_t workspace_bytes;
} tri_norm_bwd_args;

/* Bytes of workspace tri_norm_bwd needs (pure function of the sizes; 0 for
 * invalid ones). */
size_t tri_norm_bwd_workspace_bytes(int64_t R, int C);

tri_attn_status tri_norm_bwd(const tri_norm_bwd_args *args, tri_attn_stream_t stream);

/* Pack: act = x in 8 bits.  Unpack: x = the values act stands for, rounded to
 * x_type.  x is [R,C] of type x_type; 1 <= C <= 2^30. */
typedef struct {
    int64_t R;
    void *x;
    int64_t x_stride;
    tri_act8 act;
    int C, x_type;
} tri_act8_args;

tri_attn_status tri_act8_pack(const tri_act8_args *args, tri_attn_stream_t stream);
tri_attn_status tri_act8_unpack(const tri_act8_args *args, tri_attn_stream_t stream);

/* Learned relative position bias by buckets.  For batch b, query i, key j:
 *     delta  = pos_k[b,j] - pos_q[b,i]
 *     bucket = number of e with edges[e] <= delta                  (0 .. E)
 *              or E + 1, where groups are given and group_q[b,i] != group_k[b,j]
 *     bias[b,h,i,j] = table[bucket,h] (+ base[b,h,i,j])
 *   edges   : int32 [E], ascending (equal ones allowed), above -2^31;
 *             1 <= E <= 510
 *   pos_*   : int32 [B,Nq] and [B,Nk], unit inner stride, the given batch
 *             strides (0: shared by the batch); differences may pass 32 bits
 *   group_* : int32, laid out as pos_* with the same batch strides (chains,
 *             segments), or both NULL
 *   table   : [E + 1, H], or [E + 2, H] with groups; contiguous, of type table_type
 *   base    : BF16 [B,H,Nq,Nk] or ptr NULL;  bias : BF16 [B,H,Nq,Nk] output,
 *             rounded once from the FP32 sum.  Strides as for the attention's
 *             bias: innermost 1, the others non-negative multiples of 8
 *             elements, pointers 16-byte aligned; the bias's own rows must not
 *             overlap.  Elements of a padded row past Nk are left as they were;
 *             those of base in the same 16 bytes as the row's last key are read
 *             (and not used), so they must exist.
 * Sizes: 1 <= B, H, Nq, Nk, with Nq, Nk <= 2^30, B * Nq * ceil(Nk/8) < 2^31
 * and H <= 4096. */
typedef struct {
    int B, H, Nq, Nk, E, table_type;
    const void *table;
    const int32_t *edges;
    const int32_t *pos_q, *pos_k;
    const int32_t *group_q, *group_k;
    int64_t q_stride, k_stride;
    tri_attn_tensor4 base;
    tri_attn_tensor4 bias;
} tri_relpos_fwd_args;

tri_attn_status tri_relpos_fwd(const tri_relpos_fwd_args *args, tri_attn_stream_t stream);

/* Gradient of the table: dtable[k,h] = sum over b, i, j of bucket k of
 * dbias[b,h,i,j], FP32, contiguous, shaped as the table.
 *   f     : the forward's sizes, edges, positions and groups (table, base and
 *           bias are not used)
 *   dbias : BF16 [B,H,Nq,Nk], strides and the end of a row as for base
 *   workspace : caller-owned device scratch of at least
 *           tri_relpos_bwd_workspace_bytes(...) bytes, 16-byte aligned */
typedef struct {
    tri_relpos_fwd_args f;
    tri_attn_tensor4 dbias;
    float *dtable;
    void *workspace;
    size_t workspace_bytes;
} tri_relpos_bwd_args;

/* groups: nonzero if groups are given.  Pure function; 0 for invalid sizes. */
size_t tri_relpos_bwd_workspace_bytes(int B, int H, int Nq, int Nk, int E, int groups);

tri_attn_status tri_relpos_bwd(const tri_relpos_bwd_args *args, tri_attn_stream_t stream);

/* Static, NUL-terminated description of a status code. */
const char *tri_attn_strerror(tri_attn_status status);

/* Reads (and, if clear != 0, resets) the library's device error word on the
 * current device.  Every spin-wait inside the kernels is bounded; a wait that
 * expires records its site there and the kernel returns early instead of
 * hanging.  While the word is set, every later launch of the library's
 * kernels returns at once without computing (outputs untouched), until the
 * word is cleared here.  Synchronises the device.  Returns TRI_ATTN_OK,
 * TRI_ATTN_ERR_DEVICE_TIMEOUT (and stores the raw word in *word if non-NULL),
 * or TRI_ATTN_ERR_CUDA. */
tri_attn_status tri_attn_device_error(int clear, uint32_t *word);

/* Sets the bound of every kernel spin-wait, in nanoseconds of GPU global
 * timer (default 2e9 = 2 s).  Affects launches enqueued afterwards. */
void tri_attn_set_wait_limit_ns(uint64_t ns);

/* Test hook for the timeout path: enqueues a one-CTA kernel whose bounded
 * wait is on a barrier that nothing ever completes, so the wait must expire
 * (after the current limit) and record TRI_ATTN_ERR_DEVICE_TIMEOUT in the
 * device error word.  Faults nothing; the context stays usable. */
tri_attn_status tri_attn_selftest_expire_wait(tri_attn_stream_t stream);

/* TRI_ATTN_ABI_VERSION of the loaded library. */
int tri_attn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TRI_ATTN_H */
