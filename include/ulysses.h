/*
 * ulysses.h -- C ABI of the GB300 (sm_103a) Ulysses sequence-parallel hot path.
 *
 * The path (Transformers docs "Ulysses sequence parallelism", introduction and
 * its all-to-all diagram; Hugging Face Ulysses blog summary, "How Ulysses
 * Sequence Parallelism Works", steps 3-5):
 *   1. seq->head all-to-all: P sequence shards [N/P, H, d] become P head
 *      shards [N, H/P, d];
 *   2. local attention over every head shard, full sequence, causal, with
 *      GQA K/V sharing and optional packed-document masking; and its
 *      backward;
 *   3. head->seq all-to-all back.
 * On one GPU the P ranks are P virtual ranks: P contiguous shards inside one
 * device allocation, so the all-to-all is a device-local permutation.
 *
 * Conventions for every call:
 *  - Pointers named x_*, q, k, v, o, lse, dout, dq, dk, dv and workspace are
 *    DEVICE pointers owned by the caller; the library never allocates, frees
 *    or keeps them.  Host pointers are marked _host.
 *  - Every pointer must be 16-byte aligned (ULY_ERR_MISALIGNED otherwise).
 *  - Calls are asynchronous on `stream` (a cudaStream_t, NULL = legacy default
 *    stream) and never synchronise, except ulysses_get_device_status.
 *  - Arguments are validated on the host before anything is launched; on
 *    failure nothing is launched and the status says why.
 *  - dtype: ULY_BF16 (bf16 storage, fp32 accumulation) or ULY_FP32 (fp32
 *    throughout, the correctness path).
 *  - Layouts are row-major, outermost first:
 *      seq layout  : [P][B][N/P][H][d]   (P contiguous sequence shards)
 *      head layout : [P][B][N][H/P][d]   (P contiguous head shards)
 *      lse         : [S][B][Hq][N] fp32, natural logarithm of the row's sum
 *                    of exp(scaled scores)
 *    where S is the number of head shards an attention call covers.
 *  - Thread safety: calls on different streams with different buffers and
 *    workspaces may run concurrently.  The device status word is shared by
 *    all calls on a device.
 */
#ifndef ULYSSES_H
#define ULYSSES_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ULY_OK = 0,
    ULY_ERR_INVALID_ARG = 1, /* a size, count or flag is out of range */
    ULY_ERR_UNSUPPORTED = 2, /* valid for the method, not handled by this library */
    ULY_ERR_MISALIGNED = 3,  /* a pointer is not 16-byte aligned */
    ULY_ERR_OVERLAP = 4,     /* input and output buffers overlap */
    ULY_ERR_CUDA = 5,        /* a CUDA runtime/driver call failed */
    ULY_ERR_TIMEOUT = 6,     /* a device-side bounded wait ran out */
    ULY_ERR_WORKSPACE = 7,   /* workspace missing or smaller than required */
    ULY_ERR_SCRATCH_LIMIT = 8, /* sizes need more scratch than ulysses_attn_bwd_noalloc has */
    ULY_ERR_BOUNDS = 9        /* a bounds check of the debug build failed (see below) */
} uly_status;

typedef enum { ULY_BF16 = 0, ULY_FP32 = 1 } uly_dtype;

/* ---------------------------------------------------------------- swaps */

/*
 * seq->head all-to-all, emulated over P virtual ranks in one allocation.
 * Source: Transformers docs "Ulysses sequence parallelism", the all-to-all
 * diagram (rank r keeps every token and receives the contiguous head block
 * r); blog summary "How Ulysses Sequence Parallelism Works", step 3.
 *
 *   x_head[r][b][n][h][k] = x_seq[n / (N/P)][b][n % (N/P)][r*H/P + h][k]
 *
 * x_seq  : device, [P][B][N/P][H][d], read only.
 * x_head : device, [P][B][N][H/P][d], fully written.
 * B >= 1, N >= 1 with N % P == 0 (sequences are padded to a multiple of the
 * SP size), H % P == 0 (the number of heads must be divisible by the SP size),
 * 1 <= P <= H, d in {64, 128}.  The two buffers must not overlap.
 * The copy is exact (bit for bit) for either dtype.
 */
uly_status ulysses_seq_to_head(const void *x_seq, void *x_head, int64_t B, int64_t N, int32_t H,
                               int32_t d, int32_t P, uly_dtype dtype, void *stream);

/*
 * head->seq all-to-all: the exact inverse of ulysses_seq_to_head (the second
 * all-to-all of the same diagram; blog summary step 5).  It is also the
 * backward of seq->head, and seq->head is the backward of head->seq.
 *
 *   x_seq[s][b][t][r*H/P + h][k] = x_head[r][b][s*(N/P) + t][h][k]
 *
 * Same argument rules as ulysses_seq_to_head.
 */
uly_status ulysses_head_to_seq(const void *x_head, void *x_seq, int64_t B, int64_t N, int32_t H,
                               int32_t d, int32_t P, uly_dtype dtype, void *stream);

/*
 * A batch of up to four swaps in one launch, e.g. Q, K and V on their way to
 * the head layout (the all-to-all diagram moves them together), dQ, dK and dV
 * on their way back, or O going back while dO comes in.  Every tensor of the
 * batch shares B, N, d, P and dtype; each has its own head count H and its
 * own direction.  The results are those of the single calls, bit for bit.
 *
 * descs_host : host array of n_descs entries (1 <= n_descs <= 4), read before
 *              the call returns:
 *   src, dst : device buffers as in ulysses_seq_to_head (to_head = 1) or
 *              ulysses_head_to_seq (to_head = 0);
 *   H        : the tensor's head count, H % P == 0.
 * Same argument rules as ulysses_seq_to_head for every entry.  In addition no
 * entry's dst may overlap another entry's src or dst (ULY_ERR_OVERLAP): the
 * entries are copied concurrently.
 */
typedef struct {
    const void *src;
    void *dst;
    int32_t H;
    int32_t to_head;
} uly_swap_desc;

uly_status ulysses_swap_batch(const uly_swap_desc *descs_host, int32_t n_descs, int64_t B, int64_t N,
                              int32_t d, int32_t P, uly_dtype dtype, void *stream);

/* ------------------------------- norm, rotation and move of Q, K and V */

/*
 * Rotary position embedding of a call, read on the host before it returns.
 * Pair f (0 <= f < rot_dim/2) of a head turns by the angle
 *   t = positions[axis_host[f]][token] * inv_freq_host[f]
 * and is the values (f, f + rot_dim/2) of the head (interleaved = 0) or
 * (2f, 2f + 1) (interleaved = 1); values from rot_dim on are not rotated:
 *   (a, b) -> (a cos t - b sin t, b cos t + a sin t).
 * Any int64 position and any finite frequency is valid, negative ones too; the
 * angle is formed modulo a turn with an error below 2^-25 turns (the fp32
 * argument of the sine) plus |position| * (2^-62 + 2^-106 |inv_freq|) turns.
 */
typedef struct {
    const int64_t *positions;    /* device [num_axes][P][B][N/P] (8-byte aligned), or
                                    NULL: the token's index n in its sequence, every axis */
    const double *inv_freq_host; /* [rot_dim/2], finite; may be NULL if rot_dim = 0 */
    const int32_t *axis_host;    /* [rot_dim/2] values in [0, num_axes), or NULL: axis 0 */
    int32_t rot_dim;             /* 0 (no rotation) or a multiple of 16 up to d */
    int32_t num_axes;            /* 1..8 (time, height and width: 3) */
    int32_t interleaved;         /* 0 or 1 */
} uly_rope_desc;

/* Bytes of device workspace ulysses_qkv_norm_rope_bwd needs (0 if d is not supported). */
size_t ulysses_qkv_norm_rope_workspace_size(int32_t d);

/*
 * The step before the first all-to-all, and the all-to-all with it: an RMS
 * norm of every query and key head with a learned weight, the rotary position
 * embedding, and the seq->head move of Q, K and V, in one pass (the layer's
 * projection outputs are read once).  The pages leave the norm and the
 * embedding to the model; the move is ulysses_seq_to_head's.  For a head row
 * x of Q or K:
 *   y = rotate(w * x / sqrt(mean(x^2) + eps))
 * in fp32, rounded once; V is copied bit for bit.
 *
 * q_seq         : device [P][B][N/P][Hq][d], k_seq, v_seq with Hkv heads, read only.
 * q/k/v_stride  : elements from one token to the next, so that the three may
 *                 be views of one projection output [tokens][(Hq+2Hkv)*d];
 *                 0 = contiguous.  At least H*d, and a multiple of 16 bytes.
 * q_weight, k_weight : device [d], or both NULL (no norm, rotation only).
 * q_out, k_out, v_out : device, contiguous.  to_head = 1: the head layout
 *                 [P][B][N][H/P][d] (Hq % P == 0, Hkv % P == 0); to_head = 0:
 *                 the sequence layout.  No output may overlap an input or
 *                 another output.  v_seq and v_out may both be NULL.
 * N % P == 0, Hq % Hkv == 0, d in {64, 128}; P*B*(N/P) < 2^31 tokens;
 * eps >= 0.  One token (N = P = 1) is an ordinary call.
 */
uly_status ulysses_qkv_norm_rope_fwd(const void *q_seq, const void *k_seq, const void *v_seq,
                                     const void *q_weight, const void *k_weight, void *q_out, void *k_out,
                                     void *v_out, int64_t B, int64_t N, int32_t Hq, int32_t Hkv, int32_t d,
                                     int32_t P, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                     const uly_rope_desc *rope_host, float eps, int32_t to_head,
                                     uly_dtype dtype, void *stream);

/*
 * Its backward, head->seq move included.  With g = rotate^-1(dy), r = 1 /
 * sqrt(mean(x^2) + eps) and xhat = x r:
 *   dx = r (w * g - xhat mean(w * g * xhat)),   dw = sum over rows of g * xhat
 * dV is copied back bit for bit.
 *
 * q_seq, k_seq and their strides : the forward's inputs (not read, and may be
 *                 NULL, without a norm).
 * dq_out, dk_out, dv_out : device, gradients of the forward's outputs, in their layout.
 * dq_seq, dk_seq, dv_seq : device, written; strides as the inputs' above, so
 *                 that the three may be views of one buffer.  dv_out and
 *                 dv_seq may both be NULL.
 * dq_weight, dk_weight : device [d], written; each may be NULL.  Summed in
 *                 fp32 in an order that depends on the sizes alone.
 * workspace     : device, >= ulysses_qkv_norm_rope_workspace_size(d) bytes.
 * Calls that may run at the same time need workspaces of their own.
 */
uly_status ulysses_qkv_norm_rope_bwd(const void *q_seq, const void *k_seq, const void *q_weight,
                                     const void *k_weight, const void *dq_out, const void *dk_out,
                                     const void *dv_out, void *dq_seq, void *dk_seq, void *dv_seq,
                                     void *dq_weight, void *dk_weight, int64_t B, int64_t N, int32_t Hq,
                                     int32_t Hkv, int32_t d, int32_t P, int64_t q_stride, int64_t k_stride,
                                     int64_t dq_stride, int64_t dk_stride, int64_t dv_stride,
                                     const uly_rope_desc *rope_host, float eps, int32_t to_head,
                                     uly_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);

/* -------------------------------------------------- norms around a block */

/*
 * What stands between two blocks of a model (attention and its output
 * projection, or a feed-forward layer; the pages leave it to the model), in one
 * pass over the sequence-sharded tokens: the RMS norm behind a block, its gate
 * and residual scale, the sum with the residual stream, and the RMS norm before
 * the next block.  For a token's rows x (residual stream) and y (the block's
 * output):
 *   u = post_weight * y / sqrt(mean(y^2) + eps)    (u = y without post_weight)
 *   h = x + residual_scale * gate * u
 *   z = weight * h / sqrt(mean(h^2) + eps)
 * in fp32, h and z rounded once (z is formed from h before its rounding).
 * Without a block (y NULL: the norm before a model's first block) h is x.
 *
 * x, y           : device [P][B][N/P][D], read only; y may be NULL, then
 *                  post_weight, gate and h are NULL too.
 * weight, post_weight : device [D]; post_weight may be NULL (no norm behind the block).
 * gate           : device [gate_rows][D] or NULL: gate_rows = 1, one vector for
 *                  every token; gate_rows = B, one for each sequence; 0 with NULL.
 * h, z           : device, like x.  h may be NULL (the last norm of a model).
 * rstd           : device fp32 [2][P][B][N/P], 1/sqrt(mean + eps) of h and of y
 *                  (1 without post_weight) for the backward, or NULL.
 * No output may overlap an input or another output.
 * N % P == 0, B * N < 2^31 tokens, a row (D elements) a multiple of 16 bytes
 * and at most 32768 (ULY_ERR_UNSUPPORTED otherwise); eps >= 0.  One token
 * (N = P = 1) is an ordinary call.
 */
uly_status ulysses_residual_norm_fwd(const void *x, const void *y, const void *weight, const void *post_weight,
                                     const void *gate, int32_t gate_rows, float residual_scale, float eps, void *h,
                                     void *z, float *rstd, int64_t B, int64_t N, int32_t D, int32_t P,
                                     uly_dtype dtype, void *stream);

/* Bytes of device workspace ulysses_residual_norm_bwd needs, for either type (0 for sizes it would reject with both). */
size_t ulysses_residual_norm_workspace_size(int64_t B, int64_t N, int32_t D, int32_t P);

/*
 * Its backward.  With hhat and yhat the rows times their rstd (yhat = y without
 * post_weight):
 *   t  = dh + rstd_h (weight*dz - hhat mean(weight*dz*hhat)) = dx
 *   du = residual_scale * gate * t
 *   dy = rstd_y (post_weight*du - yhat mean(post_weight*du*yhat))   (dy = du without post_weight)
 *   dweight = sum dz*hhat,  dpost_weight = sum du*yhat,
 *   dgate = sum residual_scale * t * u over the tokens that share the gate.
 *
 * x, y, weight, post_weight, gate, gate_rows, residual_scale : as in the forward
 *                  (h is formed again from x and y); rstd : from the forward.
 * dh             : device, gradient of h from elsewhere, or NULL (none; without
 *                  a block it is what else the gradient of x holds).
 * dz             : device, gradient of z.
 * dx, dy         : device, like x, written; dy NULL if and only if y is.
 * dweight, dpost_weight [D], dgate [gate_rows][D] : device, written; each may be
 *                  NULL.  Summed in fp32 in an order that depends on the sizes alone.
 * workspace      : device, >= ulysses_residual_norm_workspace_size bytes; may be
 *                  NULL if all three are.  Calls that may run at the same time
 *                  need workspaces of their own.
 */
uly_status ulysses_residual_norm_bwd(const void *x, const void *y, const void *weight, const void *post_weight,
                                     const void *gate, int32_t gate_rows, float residual_scale, const float *rstd,
                                     const void *dh, const void *dz, void *dx, void *dy, void *dweight,
                                     void *dpost_weight, void *dgate, int64_t B, int64_t N, int32_t D, int32_t P,
                                     uly_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------ attention */

/*
 * Bytes of device workspace ulysses_attn_fwd (for_bwd = 0) or
 * ulysses_attn_bwd (for_bwd = 1) needs for these sizes.  Returns 0 for sizes
 * the call would reject.  num_docs = 0 means one document (no packing).
 */
size_t ulysses_attn_workspace_size(int64_t B, int64_t N, int32_t Hq_local, int32_t Hkv_local,
                                   int32_t d, int32_t num_shards, int32_t num_docs,
                                   int32_t for_bwd, uly_dtype dtype);

/*
 * The order in which the bf16 attention kernels walk the 128-row tiles of
 * a sequence (host only; no device work).  out[0 .. ceil(N/128)) receives
 * every tile index once, longest walk first.  Forward (for_bwd = 0): query
 * tiles, a tile's walk being the key tiles its rows may attend to (their
 * documents' keys, up to the row itself when causal); ties keep the later
 * tile first.  Backward (for_bwd = 1): key tiles, the walk being the query
 * tiles that may attend to the keys; ties keep the earlier tile first.
 * With packed documents a tile's walk follows its place in its document, so
 * the attention calls sort the tiles like this themselves (the order goes
 * into the workspace next to cu_seqlens); without documents the walk only
 * depends on the index and this is the kernels' index order.  Exposed for
 * inspection and tests.
 * out : host, ceil(N/128) int32.
 * Errors: ULY_ERR_INVALID_ARG for out == NULL, N < 1, causal or for_bwd not
 * 0/1, or cu_seqlens the attention calls would reject.
 */
uly_status ulysses_attn_tile_order(int64_t N, int32_t causal, const int32_t *cu_seqlens_host,
                                   int32_t num_docs, int32_t for_bwd, int32_t *out);

/*
 * Attention forward over `num_shards` consecutive head shards (blog summary,
 * step 4 "Local Attention": every rank attends over all N tokens for its
 * heads).  For shard s, batch b, local query head h (local KV head h / G,
 * G = Hq_local / Hkv_local), row i:
 *   s_ij  = softmax_scale * <q_i, k_j>            for allowed j
 *   lse_i = ln sum_j exp(s_ij)
 *   o_i   = sum_j exp(s_ij - lse_i) v_j
 * allowed: j <= i if causal; and doc(i) == doc(j) if cu_seqlens_host is not
 * NULL (packed documents, the block-diagonal mask of FlashAttention-style
 * varlen attention that the Transformers docs recommend for packing).
 *
 * q, o       : device, [num_shards][B][N][Hq_local][d]
 * k, v       : device, [num_shards][B][N][Hkv_local][d]
 * lse        : device fp32, [num_shards][B][Hq_local][N]
 * cu_seqlens_host : host int32 [num_docs + 1], 0 = cu[0] <= cu[1] <= ... <=
 *              cu[num_docs] = N, or NULL (one document).  Copied before return.
 * softmax_scale <= 0 selects 1/sqrt(d).
 * workspace  : device, >= ulysses_attn_workspace_size(..., for_bwd=0) bytes.
 * Requires Hq_local % Hkv_local == 0, d in {64, 128} (bf16: d == 128).
 */
uly_status ulysses_attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                            int64_t B, int64_t N, int32_t Hq_local, int32_t Hkv_local, int32_t d,
                            int32_t num_shards, int32_t causal, const int32_t *cu_seqlens_host,
                            int32_t num_docs, float softmax_scale, uly_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * Attention backward (the gradient of ulysses_attn_fwd, which training needs;
 * the Trainer discussion in the blog summary requires the gradients to be
 * correct).  With P_ij = exp(s_ij - lse_i) and D_i = <dO_i, O_i>:
 *   dV_j = sum_i P_ij dO_i
 *   dS_ij = P_ij (<dO_i, v_j> - D_i)
 *   dQ_i = softmax_scale sum_j dS_ij k_j
 *   dK_j = softmax_scale sum_i dS_ij q_i
 * dK and dV are summed over the G query heads sharing a KV head.
 *
 * q, k, v, o, lse : as returned/used by ulysses_attn_fwd (o and lse from it).
 * dout, dq        : device, like q.   dk, dv : device, like k.  All written.
 * workspace       : device, >= ulysses_attn_workspace_size(..., for_bwd=1);
 *                   holds fp32 scratch (D, scaled lse, the dQ accumulator).
 * Other arguments as in ulysses_attn_fwd.
 */
uly_status ulysses_attn_bwd(const void *q, const void *k, const void *v, const void *o,
                            const float *lse, const void *dout, void *dq, void *dk, void *dv,
                            int64_t B, int64_t N, int32_t Hq_local, int32_t Hkv_local, int32_t d,
                            int32_t num_shards, int32_t causal, const int32_t *cu_seqlens_host,
                            int32_t num_docs, float softmax_scale, uly_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * The swap -> attention -> swap pipeline without the swaps: attention over all
 * P head shards read straight from the sequence-sharded buffers, outputs
 * written straight back to them.  Same results as
 *   ulysses_seq_to_head(q/k/v) ; ulysses_attn_fwd(num_shards = P) ;
 *   ulysses_head_to_seq(o)
 * because on one device head shard r is just a strided view of the seq
 * buffer (the all-to-all moves data between GPUs; on one GPU it only
 * relabels rows).  Source: as ulysses_seq_to_head and ulysses_attn_fwd.
 *
 * q_seq, o_seq : device, [P][B][N/P][Hq][d]     k_seq, v_seq : [P][B][N/P][Hkv][d]
 * lse          : device fp32, [P][B][Hq/P][N]   (head shard r, local head h)
 * Hq, Hkv are the GLOBAL head counts; H % P == 0 for both (ULY_ERR_INVALID_ARG).
 * bf16 also needs (N/P) % 128 == 0 so that no 128-token tile straddles two
 * sequence shards (ULY_ERR_UNSUPPORTED otherwise).  workspace: as
 * ulysses_attn_workspace_size(B, N, Hq/P, Hkv/P, d, P, num_docs, 0, dtype).
 * Other arguments, validation and errors as ulysses_attn_fwd.
 */
uly_status ulysses_attn_fwd_seq(const void *q_seq, const void *k_seq, const void *v_seq, void *o_seq,
                                float *lse, int64_t B, int64_t N, int32_t Hq, int32_t Hkv, int32_t d,
                                int32_t P, int32_t causal, const int32_t *cu_seqlens_host,
                                int32_t num_docs, float softmax_scale, uly_dtype dtype, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * Backward of ulysses_attn_fwd_seq: dout_seq in, dq_seq / dk_seq / dv_seq out,
 * all in the sequence-sharded layout (the backward of the swaps is the
 * inverse swap, so no swap is needed here either).  workspace: as
 * ulysses_attn_workspace_size(B, N, Hq/P, Hkv/P, d, P, num_docs, 1, dtype).
 */
uly_status ulysses_attn_bwd_seq(const void *q_seq, const void *k_seq, const void *v_seq,
                                const void *o_seq, const float *lse, const void *dout_seq,
                                void *dq_seq, void *dk_seq, void *dv_seq, int64_t B, int64_t N,
                                int32_t Hq, int32_t Hkv, int32_t d, int32_t P, int32_t causal,
                                const int32_t *cu_seqlens_host, int32_t num_docs, float softmax_scale,
                                uly_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * ulysses_attn_bwd without a workspace, for callers that cannot allocate
 * device memory: code running inside an allocator's own hooks, a process
 * whose device memory pool is fixed up front, a plugin that is handed only
 * the tensors it works on, or a latency-critical path that must not take the
 * allocator's locks.  The pages have no counterpart: the method itself does
 * not care where scratch lives.
 *
 * Same arguments and results as ulysses_attn_bwd, minus workspace.  The fp32
 * scratch (lse*log2(e), D, the dQ accumulator, the cu_seqlens copy) lives in
 * one fixed 64 MiB device array inside the library; every GPU that loads
 * this part of the library holds those 64 MiB until the process exits.
 * Sizes whose scratch (ulysses_attn_workspace_size(..., for_bwd=1, ...))
 * exceeds 64 MiB return ULY_ERR_SCRATCH_LIMIT and launch nothing; for bf16
 * that is about 129,000 (shard x batch x query-head x padded-row) rows, e.g.
 * N = 8192 with 8 local query heads and 1 shard fits.
 * The call itself makes no cudaMalloc and calls no allocating library
 * routine.  The array is part of the library's device code, which the CUDA
 * runtime loads onto a device lazily: the first call on each device looks up
 * the array's device address, and that lookup loads the module, so the
 * driver reserves the 64 MiB (and the module's code) inside that first call.
 * A caller whose restricted context cannot afford that reservation (a fixed
 * pool with its memory already committed, an allocator hook) must make the
 * first call on each device outside that context, at start-up, and also
 * before any stream capture; later calls reserve nothing.
 * stream and every pointer must belong to the CURRENT device (the scratch
 * address is the current device's).  After cudaDeviceReset the cached
 * address is stale: do not call this entry point again in that process.
 * All calls share the array: calls that overlap on the GPU (other streams,
 * other threads) race and must not be issued; sequential calls are safe
 * because each one rewrites or clears every scratch byte it reads.
 */
uly_status ulysses_attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o,
                                    const float *lse, const void *dout, void *dq, void *dk, void *dv,
                                    int64_t B, int64_t N, int32_t Hq_local, int32_t Hkv_local,
                                    int32_t d, int32_t num_shards, int32_t causal,
                                    const int32_t *cu_seqlens_host, int32_t num_docs,
                                    float softmax_scale, uly_dtype dtype, void *stream);

/* ------------------------------------------------- sliding-window attention */

/*
 * Causal attention over a sliding window, with the first tokens of each
 * document staying visible (sinks): the attention of ulysses_attn_fwd with
 *   allowed: j <= i, doc(i) == doc(j), and
 *            i - j < window  or  j - start(doc(i)) < sinks
 * where start(doc) is the document's first token (0 without documents).
 * window >= N is plain causal attention.  Every row sees itself.
 *
 * q, o, k, v, lse, cu_seqlens_host, num_docs, softmax_scale : as in
 *              ulysses_attn_fwd; no output may overlap an input or another
 *              output.  K and V of every token must be finite, padding's too
 *              (zeros do): one that is not, at token j, may spoil rows that do not
 *              see it, of any document, since rows and keys are taken in tiles:
 *              those from j - 384 to j + window + 384; and, if j lies in one tile
 *              of 128 tokens with one of the first max(sinks, 32) of a document
 *              (sinks > 0), those from that document's start to 384 behind its end.
 * window >= 1, sinks >= 0, any size.
 * workspace  : device, >= ulysses_window_attn_workspace_size(..., for_bwd) bytes
 *              (num_docs = 0 without documents).  Calls that may run at the same
 *              time need workspaces of their own.  cu_seqlens_host is taken in
 *              before the call returns; a captured call replays with it.
 * Requires Hq_local % Hkv_local == 0, d in {64, 128} (bf16: d == 128).
 */
size_t ulysses_window_attn_workspace_size(int64_t B, int64_t N, int32_t Hq_local, int32_t Hkv_local, int32_t d,
                                          int32_t num_shards, int64_t window, int64_t sinks, int32_t num_docs,
                                          int32_t for_bwd, uly_dtype dtype);
uly_status ulysses_window_attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int64_t B,
                                   int64_t N, int32_t Hq_local, int32_t Hkv_local, int32_t d, int32_t num_shards,
                                   int64_t window, int64_t sinks, const int32_t *cu_seqlens_host, int32_t num_docs,
                                   float softmax_scale, uly_dtype dtype, void *workspace, size_t workspace_bytes,
                                   void *stream);

/*
 * Its backward: ulysses_attn_bwd's formulas over the same allowed pairs.  q, dout
 * and lse have to be finite too, or any gradient may be spoilt.  dK and dV (and dQ in fp32) are summed in an order
 * that depends on the arguments alone; in bf16 dQ is summed with fp32 atomics, as in
 * ulysses_attn_bwd, so its last bits may differ between calls.
 */
uly_status ulysses_window_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                   const void *dout, void *dq, void *dk, void *dv, int64_t B, int64_t N,
                                   int32_t Hq_local, int32_t Hkv_local, int32_t d, int32_t num_shards, int64_t window,
                                   int64_t sinks, const int32_t *cu_seqlens_host, int32_t num_docs,
                                   float softmax_scale, uly_dtype dtype, void *workspace, size_t workspace_bytes,
                                   void *stream);

/*
 * The same attention for one new token of every sequence, over a cache of keys
 * and values that already holds the token's own: sequence b has lens[b] tokens,
 * its new one at position lens[b] - 1, which sees the cache's tokens j with
 * lens[b] - 1 - j < window or j < sinks.
 *
 * q, o     : device [num_shards][B][1][Hq_local][d].  lse : device fp32 [num_shards][B][Hq_local][1].
 * k_cache, v_cache : device [num_shards][B][C][Hkv_local][d].  Token j lies in slot
 *            j, as long as the cache holds every token; once a sequence has more
 *            than C tokens the cache rolls (C >= sinks + window): token j lies in
 *            slot j for j < sinks, else in slot sinks + (j - sinks) mod (C - sinks)
 *            (the same slot while j < C).  Only the slots of tokens that are seen
 *            are read; the others may hold anything.
 * lens     : device int64 [B] (8-byte aligned), read on the device.  0: an empty sequence, o = 0
 *            and lse = -inf.  Negative, or more than C with C < sinks + window: the
 *            same, and ULY_ERR_INVALID_ARG from ulysses_get_device_status.
 * workspace: device, >= ulysses_window_attn_decode_workspace_size bytes.  Calls that
 *            may run at the same time need workspaces of their own.
 * window >= 1, sinks >= 0 (more than 2^30 counts as 2^30), C <= 2^30; other
 * rules as above.  The result has the same bits on every call.
 */
size_t ulysses_window_attn_decode_workspace_size(int64_t B, int64_t C, int32_t Hq_local, int32_t Hkv_local, int32_t d,
                                                 int32_t num_shards, int64_t window, int64_t sinks, uly_dtype dtype);
uly_status ulysses_window_attn_decode(const void *q, const void *k_cache, const void *v_cache, const int64_t *lens,
                                      void *o, float *lse, int64_t B, int64_t C, int32_t Hq_local, int32_t Hkv_local,
                                      int32_t d, int32_t num_shards, int64_t window, int64_t sinks,
                                      float softmax_scale, uly_dtype dtype, void *workspace, size_t workspace_bytes,
                                      void *stream);

/* --------------------------------------------------------- ring attention */

/*
 * Ring attention over P virtual ranks, the pages' alternative to Ulysses
 * ("Sequence Parallelism for Long-Context AI Training", "Advanced Scaling:
 * Ring Attention and Ulysses"; blog summary, "Comparing Ulysses and Ring
 * Attention"): rank r keeps its chunk of Q for ALL heads and the K/V chunks
 * travel round the ring; in P steps every query chunk meets every key chunk
 * (step k: query chunk r with key chunk (r - k) mod P; causal keeps only
 * r >= k after step 0), and the partial results are merged through their
 * log-sum-exp.  The result equals causal attention over all N tokens, i.e.
 * the same as the Ulysses path, without any head sharding.
 *
 * q_seq, o_seq, dout_seq, dq_seq : device, [P][B][N/P][Hq][d]
 * k_seq, v_seq, dk_seq, dv_seq   : device, [P][B][N/P][Hkv][d]
 * lse : device fp32, [P][B][Hq][N/P] (chunk, batch, head, position in chunk)
 * Hq, Hkv are the total head counts (ring attention does not shard heads).
 * N % P == 0; otherwise the rules of ulysses_attn_fwd on each chunk
 * (N/P tokens), without packed documents.
 * workspace : device, >= ulysses_ring_attn_workspace_size(..., for_bwd).
 * The backward uses the final o and lse of the forward.
 */
size_t ulysses_ring_attn_workspace_size(int64_t B, int64_t N, int32_t Hq, int32_t Hkv, int32_t d,
                                        int32_t P, int32_t for_bwd, uly_dtype dtype);
uly_status ulysses_ring_attn_fwd(const void *q_seq, const void *k_seq, const void *v_seq, void *o_seq,
                                 float *lse, int64_t B, int64_t N, int32_t Hq, int32_t Hkv, int32_t d,
                                 int32_t P, int32_t causal, float softmax_scale, uly_dtype dtype,
                                 void *workspace, size_t workspace_bytes, void *stream);
uly_status ulysses_ring_attn_bwd(const void *q_seq, const void *k_seq, const void *v_seq,
                                 const void *o_seq, const float *lse, const void *dout_seq,
                                 void *dq_seq, void *dk_seq, void *dv_seq, int64_t B, int64_t N,
                                 int32_t Hq, int32_t Hkv, int32_t d, int32_t P, int32_t causal,
                                 float softmax_scale, uly_dtype dtype, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* -------------------------------------------------------- sharded loss */

/* Bytes of device workspace ulysses_sharded_ce_loss needs (0 if invalid). */
size_t ulysses_sharded_ce_workspace_size(int64_t B, int64_t N, int32_t P);

/*
 * Next-token cross entropy of a sequence-parallel batch and its
 * good-token-weighted aggregation across the P ranks (Accelerate PR
 * "Deepspeed Ulysses/ALST integration", user API step 2: shift_labels, the
 * per-rank loss, all_gather of losses and good-token counts, then
 * sum_r loss_r * good_r / max(sum_r good_r, 1); the Transformers docs list
 * label shifting and loss aggregation among what the Trainer does for SP).
 *
 * Labels are shifted over the WHOLE sequence before sharding: the target of
 * the last token of rank r's chunk is the first label of rank r+1's chunk;
 * the last token of each sequence gets -100 (ignored).
 *
 * logits     : device, [P][B][N/P][V] (each rank's LM-head output), read.
 * labels     : device int64, [P][B][N/P], unshifted; -100 = ignored.  Values
 *              outside [0, V) other than -100 are ignored and reported as
 *              ULY_ERR_INVALID_ARG by ulysses_get_device_status.
 * dlogits    : device, like logits, or NULL.  If given, receives
 *              d total_loss / d logits = (softmax - onehot(target)) / max(T, 1)
 *              on good rows and 0 on ignored rows (T = all good tokens).
 * shard_loss : device fp32 [P]: rank r's mean CE over its good tokens (0 if none).
 * shard_good : device int64 [P]: rank r's good-token count.
 * total_loss : device fp32 [1]: the aggregated loss.
 * workspace  : device, >= ulysses_sharded_ce_workspace_size(B, N, P).
 * N % P == 0 (sequences padded to a multiple of the SP size).
 */
uly_status ulysses_sharded_ce_loss(const void *logits, const int64_t *labels, void *dlogits,
                                   float *shard_loss, int64_t *shard_good, float *total_loss,
                                   int64_t B, int64_t N, int32_t V, int32_t P, uly_dtype dtype,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * The LM head and ulysses_sharded_ce_loss in one, without the logits: the
 * same shifted labels, per-shard means and good-token-weighted total, of
 *   logits[row][v] = <hidden[row], weight[v]>
 * which are formed in pieces of rows with a label (as many as 2.5 GB of
 * workspace hold, at least 1024, at most 65536) and never kept: a long
 * sequence's logits and their gradient outweigh everything else the step holds
 * (at 65,536 tokens and a vocabulary of 151,936, 20 GB each in bf16).  Rows
 * without a label (ignored ones, and the last of each sequence) take no part:
 * their hidden values are not read.
 *
 * hidden     : device, [P][B][N/P][D].      weight : device, [V][D].
 * labels     : as in ulysses_sharded_ce_loss.
 * dhidden    : device, like hidden, or NULL: d total / d hidden (0 on rows without a label).
 * dweight    : device, like weight, or NULL: d total / d weight.
 * shard_loss, shard_good, total_loss : as in ulysses_sharded_ce_loss.
 * workspace  : device, >= ulysses_sharded_linear_ce_workspace_size(..., for_grad
 *              = 1 if dhidden or dweight is given) bytes.  Calls that may run
 *              at the same time need workspaces of their own.
 * Products are accumulated in fp32; softmax and loss are fp32.  bf16: the
 * label's term of a row's gradient, (p - 1) weight[label] and (p - 1) hidden, is
 * formed in fp32; of the other words' terms, p weight[v] and p hidden, the
 * softmax's numerators and, for dweight, the hidden rows divided by its
 * denominators are rounded to bf16; each gradient is rounded to bf16 once.
 * fp32: operands are taken as three bf16 parts each, off by less than 2^-26 of a
 * value or 2^-134, what is more (values above 3.39e38, bf16's largest, count as
 * infinite).  Numerators reach 2^48, and their sums with weight and hidden are
 * formed before the division: values above 2^58 may overflow.
 * D * element size a multiple of 16 bytes, D <= 65536, V <= 2^21
 * (ULY_ERR_UNSUPPORTED otherwise); N % P == 0.
 */
size_t ulysses_sharded_linear_ce_workspace_size(int64_t B, int64_t N, int32_t D, int32_t V, int32_t P,
                                                int32_t for_grad, uly_dtype dtype);
uly_status ulysses_sharded_linear_ce_loss(const void *hidden, const void *weight, const int64_t *labels,
                                          void *dhidden, void *dweight, float *shard_loss, int64_t *shard_good,
                                          float *total_loss, int64_t B, int64_t N, int32_t D, int32_t V,
                                          int32_t P, uly_dtype dtype, void *workspace, size_t workspace_bytes,
                                          void *stream);

/* ------------------------------------------------------------ diagnostics */

/*
 * Synchronises `stream`, then reads and clears the current device's status
 * word.  ULY_OK if no kernel reported a problem since the last read;
 * ULY_ERR_TIMEOUT if a bounded device-side wait ran out (the kernel then
 * stopped early and its outputs are invalid); ULY_ERR_BOUNDS if a kernel of
 * the debug build found an access outside its buffer (it skipped the access;
 * outputs are invalid); ULY_ERR_INVALID_ARG if a kernel rejected its launch
 * configuration; ULY_ERR_CUDA on a CUDA error.  If site_out is not NULL it
 * receives the id of the first site that reported (a wait, or 0x8000 plus
 * the id of an access).
 */
uly_status ulysses_get_device_status(void *stream, uint32_t *site_out);

/*
 * Sets the per-wait limit (nanoseconds, >= 1000) of every bounded device
 * wait launched afterwards by this process.  Default: 2 s.
 */
uly_status ulysses_set_wait_limit_ns(uint64_t limit_ns);

/*
 * Launches one tiny kernel whose mbarrier wait can never complete (nothing
 * arrives on it), with a limit of limit_ns.  The wait gives up, records
 * ULY_ERR_TIMEOUT in the device status word and the kernel returns.  Used by
 * tests of the timeout path; it faults nothing and hangs nothing.
 */
uly_status ulysses_selftest_wait_timeout(uint64_t limit_ns, void *stream);

/*
 * Debug build only (the library compiled with -DULY_DEBUG, which checks every
 * raw-pointer global access of the swap and attention kernels (the windowed ones
 * too), and those of the norm-rotation, residual-norm and LM-head loss kernels
 * whose place depends on data or on the schedule, against their buffers and
 * reports ULY_ERR_BOUNDS instead of making them): launches one tiny kernel whose
 * check is given an offset past its extent, touching no memory, so that the
 * reporting path can be tested.  The release build returns ULY_ERR_UNSUPPORTED and
 * launches nothing.
 */
uly_status ulysses_selftest_bounds(void *stream);

/* Human-readable name of a status code (static string). */
const char *ulysses_status_string(uly_status status);

/* Library version, major*10000 + minor*100 + patch. */
int32_t ulysses_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ULYSSES_H */
