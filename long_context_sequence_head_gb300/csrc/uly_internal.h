// Internal declarations shared by the library's translation units (host side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "uly_ptx.cuh"

namespace uly {

// cuTensorMapEncodeTiled, resolved through the runtime once per process.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// An NVTX push/pop range around one call of the C ABI, named after the call,
// so that profilers can attribute kernels to it.  NVTX 3 is header-only: with
// no tool attached a push or pop is a check of a null function pointer.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};
#define ULY_NVTX_RANGE() const ::uly::NvtxRange uly_nvtx_range_(__func__)

// Device status word of the current device (2 x u32: flags, first site).
unsigned *device_status_ptr();
uint64_t wait_limit_ns();
int num_sms();

// Rows [lo, hi) of the document holding token i (the whole sequence without documents).
inline void doc_range_host(const int32_t *cu, int num_docs, int64_t N, int64_t i, int64_t &lo, int64_t &hi)
{
    lo = 0;
    hi = N;
    if (cu == nullptr || num_docs <= 0)
        return;
    int a = 0, b = num_docs;
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (static_cast<int64_t>(cu[m]) <= i)
            a = m;
        else
            b = m;
    }
    lo = cu[a];
    hi = cu[a + 1];
}

// The 128-row tiles of a packed-document sequence in the order the bf16
// kernels walk them, longest walk first, so that no long walk is left to run
// on alone at the end of a launch (with documents the walk length follows a
// tile's place in its document, not its index).  Forward (bwd = false): query
// tiles, walk = the key tiles their rows may attend to, ties with the later
// tile first.  Backward: key tiles, walk = the query tiles that may attend to
// them, ties with the earlier tile first.  out: ceil(N/128) entries.
inline void tile_order_host(bool bwd, int64_t N, int causal, const int32_t *cu, int num_docs, int32_t *out)
{
    const int n = static_cast<int>((N + 127) / 128);
    std::vector<int64_t> walk(n);
    for (int t = 0; t < n; ++t) {
        const int64_t a = static_cast<int64_t>(t) * 128, b = std::min<int64_t>(a + 127, N - 1);
        int64_t lo_a, hi_a, lo_b, hi_b;
        doc_range_host(cu, num_docs, N, a, lo_a, hi_a);
        doc_range_host(cu, num_docs, N, b, lo_b, hi_b);
        const int64_t lo = (bwd && causal) ? a : lo_a;
        const int64_t hi = (!bwd && causal) ? b + 1 : hi_b;
        walk[t] = (hi - 1) / 128 - lo / 128 + 1;
        out[t] = bwd ? t : n - 1 - t;
    }
    std::stable_sort(out, out + n, [&](int32_t x, int32_t y) { return walk[x] > walk[y]; });
}

// Problems interleaved per group of the grid: the fewest that make a group's
// work per SM at least 1.5 times the longest single work unit, so that the
// last group's longest units do not run on alone at the end of the launch.
inline int group_for(int64_t work_per_problem, int64_t longest_unit, int64_t nprob)
{
    if (work_per_problem <= 0)
        return 1;
    int64_t g = (3 * longest_unit * num_sms() + 2 * work_per_problem - 1) / (2 * work_per_problem);
    if (g > nprob)
        g = nprob;
    return g < 1 ? 1 : static_cast<int>(g);
}

// Launches a kernel that calls grid_wait(): its blocks may be set up while the
// kernel before it on the stream finishes, which hides a launch of small ones.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), int64_t grid, int block, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

inline WaitCfg wait_cfg() { return WaitCfg{device_status_ptr(), wait_limit_ns()}; }

// ---------------------------------------------------------------- swap
// seq layout [P][B][N/P][H][d] <-> head layout [P][B][N][H/P][d].
cudaError_t launch_swap(bool to_head, const void *src, void *dst, int64_t B, int64_t N, int H, int d, int P,
                        int esize, cudaStream_t stream);

// Up to kSwapMaxBatch tensors with common B, N, d, P and element size in one
// launch; each has its own head count and direction.
constexpr int kSwapMaxBatch = 4;
struct SwapDesc {
    const void *src;
    void *dst;
    int H;
    int to_head;
};
cudaError_t launch_swap_batch(const SwapDesc *descs, int n, int64_t B, int64_t N, int d, int P, int esize,
                              cudaStream_t stream);

// ----------------------------------------------------------- attention
// Where the rows of an attention tensor live.
//   head layout (seq == 0): [S][B][N][H][d], shard-major, what the swap writes;
//   seq layout  (seq == 1): [P][B][N/P][P*H][d], the sequence-sharded buffer
//     before the swap: head shard r of local head h is global head r*H + h,
//     token n sits in sequence shard n / (N/P) at position n % (N/P).
// Row (sb, n, h) with sb = shard*B + batch.
struct RowLayout {
    int seq;
    int B;
    int64_t Np;  // N / P (seq layout)
    int P;       // head shards == sequence shards (seq layout)

    __host__ __device__ int64_t off(int64_t N, int64_t sb, int64_t n, int H, int h, int d) const
    {
        if (!seq)
            return ((sb * N + n) * H + h) * static_cast<int64_t>(d);
        const int64_t r = sb / B, b = sb % B, s = n / Np, t = n % Np;
        return (((s * B + b) * Np + t) * (static_cast<int64_t>(H) * P) + r * H + h) * static_cast<int64_t>(d);
    }
    // coordinates {head, token, batch, outer} of the 5-D tensor map of this
    // layout for a tile of rows starting at token n0 (which never straddles a
    // sequence shard in the seq layout)
    __host__ __device__ void tile(int64_t sb, int64_t n0, int H, int h, int &c1, int &c2, int &c3, int &c4) const
    {
        const int r = static_cast<int>(sb / B), b = static_cast<int>(sb % B);
        c3 = b;
        if (!seq) {
            c1 = h;
            c2 = static_cast<int>(n0);
            c4 = r;
        } else {
            c1 = r * H + h;
            c2 = static_cast<int>(n0 % Np);
            c4 = static_cast<int>(n0 / Np);
        }
    }
};

// How the backward of a windowed attention is cut into units (window_attn.cu):
// a key tile and the query tiles that see it.  A tile with sinks is seen by
// every later row of its document; that walk, past the window's, is cut into
// extra units, whose sums of the sinks' dK and dV are joined afterwards.
struct WindowUnits {
    int sink_tiles = 0;          // without documents: tiles 0 .. sink_tiles-1 have sinks
    int extra = 0;               // extra units of each (without documents)
    int n_units = 0;             // of a problem
    int n_joins = 0;             // tiles to join
    int64_t work = 0, longest = 0;  // query tiles walked by a problem's units, and by its longest
    int slots = 0;               // partial sums of a problem
    int rows = 0;                // keys of a slot
    const int4 *units = nullptr; // device, with documents: {key tile, first query tile, query tiles, slot * 2 + extra or -1}
    const int4 *joins = nullptr; // device, with documents: {first key, keys, first slot, slots}
    float *part = nullptr;       // [problem][slot][2][rows][d] fp32: dK, dV
    // bf16 with up to kWindowSinksApart sinks: window_sinks.cu takes their dK and dV in
    // documents with rows past their window, in chunks of row tiles; up to kWindowSinks
    // also what they add to the dQ of those rows (it sets the accumulator), so that no
    // unit is extra.  Device, three each: {first row tile, past the last, document's start
    // or -1 for no sinks, sinks}, {slot of the sinks in their first key tile, from a key
    // tile's to the next one's, last row tile that the main kernel walks for the first key
    // tile, for the second}, {document's end, first row tile whose dQ is this document's to
    // set, 0, 0}
    const int4 *chunks = nullptr;
    int n_chunks = 0;
    int sinks = 0;  // of a document in the chunks, at most
};
constexpr int kWindowSinks = 64, kWindowSinksApart = 320;

// The last query tile that sees key tile t through the window, without documents.
__host__ __device__ inline int window_end(int64_t N, int window, int tile, int t)
{
    const int64_t next = (static_cast<int64_t>(t) + 1) * tile, last = next < N ? next - 1 : N - 1;
    return static_cast<int>((last + window < N ? last + window - 1 : N - 1) / tile);
}

// Unit `rank` of a problem: {key tile, first query tile, query tiles, slot * 2 +
// extra or -1}.  Extra units come first (with documents: the longest units).
__device__ __forceinline__ int4 window_unit(const WindowUnits &wu, int64_t N, int window, int tile, int rank)
{
    if (wu.units != nullptr)
        return wu.units[rank];
    const int tiles = static_cast<int>((N + tile - 1) / tile), n_extra = wu.sink_tiles * wu.extra;
    if (rank < n_extra) {
        const int t = rank / wu.extra, e = rank % wu.extra, m0 = window_end(N, window, tile, t) + 1;
        const int lo = m0 + static_cast<int>(static_cast<int64_t>(tiles - m0) * e / wu.extra);
        const int hi = m0 + static_cast<int>(static_cast<int64_t>(tiles - m0) * (e + 1) / wu.extra);
        return make_int4(t, lo, hi - lo, (t * (1 + wu.extra) + 1 + e) * 2 + 1);
    }
    const int t = rank - n_extra;
    const bool sinks = t < wu.sink_tiles;
    const int end = sinks && wu.extra == 0 ? tiles - 1 : window_end(N, window, tile, t);
    return make_int4(t, t, end - t + 1, sinks && wu.extra > 0 ? t * (1 + wu.extra) * 2 : -1);
}

struct AttnShape {
    int window = 0, sinks = 0;  // sliding window (0: none) and first tokens that stay visible
    WindowUnits units;          // backward with a window
    int64_t SB;      // num_shards * B (independent (shard, batch) problems)
    int64_t N;       // tokens
    int Hq, Hkv, d;  // per shard
    int causal;
    const int32_t *cu_dev;  // device cu_seqlens [num_docs+1] or nullptr
    const int32_t *cu_host; // the same on the host (valid during the call) or nullptr
    int32_t *order_dev;     // with documents: device room for a 128-row tile order [ceil(N/128)], else nullptr
    int num_docs;
    float scale;      // softmax scale
    RowLayout L;     // where q/k/v/o/dout/dq/dk/dv rows live
    // buffer extents in elements, for the bounds checks of debug builds
    int64_t q_elems;    // q, o, dout, dq
    int64_t kv_elems;   // k, v, dk, dv
    int64_t lse_elems;  // lse (and the per-row fp32 scratch)
    unsigned *status;   // device status word
};

// 5-D bf16 tensor map {d, H, T, B, outer} over a row-major
// [outer][B][T][H][d] buffer, box {64, 1, rows, 1, 1}, 128-byte swizzle.
CUresult make_rows_map_bf16(CUtensorMap *map, const void *base, const AttnShape &s, int H, int rows = 128);

cudaError_t launch_attn_fwd_f32(const AttnShape &s, const float *q, const float *k, const float *v, float *o,
                                float *lse, cudaStream_t stream);
cudaError_t launch_attn_bwd_f32(const AttnShape &s, const float *q, const float *k, const float *v,
                                const float *o, const float *lse, const float *dout, float *dq, float *dk,
                                float *dv, float *ws_D, cudaStream_t stream);

cudaError_t launch_attn_fwd_bf16(const AttnShape &s, const void *q, const void *k, const void *v, void *o,
                                 float *lse, cudaStream_t stream);

// bf16 backward scratch (fp32): lse2/D [SB][Hq][Npad], dq_acc [SB][Hq][Npad][d]
struct BwdScratch {
    float *lse2;
    float *D;
    float *dq_acc;
    int64_t Npad;
};
cudaError_t launch_window_sinks(const AttnShape &s, const void *q, const void *k, const void *v, const void *dout,
                                const BwdScratch &scr, cudaStream_t stream);
cudaError_t launch_attn_bwd_bf16(const AttnShape &s, const void *q, const void *k, const void *v, const void *o,
                                 const float *lse, const void *dout, void *dq, void *dk, void *dv,
                                 const BwdScratch &scr, cudaStream_t stream);

cudaError_t launch_window_fwd_bf16(const AttnShape &s, const void *q, const void *k, const void *v, void *o,
                                   float *lse, cudaStream_t stream);

// fp32 with a sliding window; part of window_attn.cu's units (key tiles of 64).
constexpr int kWindowTileF32 = 64;
cudaError_t launch_window_fwd_f32(const AttnShape &s, const float *q, const float *k, const float *v, float *o,
                                  float *lse, cudaStream_t stream);
cudaError_t launch_window_bwd_f32(const AttnShape &s, const float *q, const float *k, const float *v, const float *o,
                                  const float *lse, const float *dout, float *dq, float *dk, float *dv, float *ws_D,
                                  cudaStream_t stream);

// Sliding-window attention (window_attn.cu): workspace of a call, and the call
// itself on arguments that were checked.
size_t window_attn_workspace(int64_t B, int64_t N, int Hq, int Hkv, int d, int S, int64_t window, int64_t sinks,
                             int num_docs, bool bwd, int esize);
cudaError_t window_attn_fwd(AttnShape s, const void *q, const void *k, const void *v, void *o, float *lse, int esize,
                            void *workspace, cudaStream_t stream);
cudaError_t window_attn_bwd(AttnShape s, const void *q, const void *k, const void *v, const void *o, const float *lse,
                            const void *dout, void *dq, void *dk, void *dv, int esize, void *workspace,
                            cudaStream_t stream);

// One new token of every sequence over a cache (window_decode.cu).
struct WindowDecodeParams {
    const void *q, *k, *v;  // [SB][Hq][d], [SB][C][Hkv][d]
    const int64_t *lens;    // [B]
    void *o;
    float *lse;             // [SB][Hq]
    int64_t SB, C;
    int B, Hq, Hkv;
    int window, sinks;
    float scale_log2;
    // set by the launch: query heads of a KV head, groups of them, blocks a group is spread over
    int G, parts, splits;
    float *part, *stats;    // [SB][Hq][splits][d], [SB][Hq][splits][2]
    unsigned *status;
};
size_t window_decode_workspace(int64_t SB, int64_t C, int Hq, int Hkv, int d, int64_t window, int64_t sinks, int esize);
cudaError_t launch_window_decode(WindowDecodeParams &p, int d, int esize, void *workspace, cudaStream_t s);

cudaError_t launch_selftest_timeout(uint64_t limit_ns, cudaStream_t stream);

// -------------------------------------------- norm, rotation and move of Q, K, V
// Most blocks of a backward launch, and so most weight-gradient partials.
constexpr int kNormRopeMaxBlocks = 1280;
constexpr int kNormRopeMaxHalf = 64;

struct NormRopeParams {
    // near side: the sequence layout, token strides in elements.  The backward
    // reads q and k for the norm; v only tells it that there is a V.
    const void *q, *k, *v;
    int64_t qs, ks, vs;
    // far side: outputs of the forward, gradients read by the backward
    void *qo, *ko, *vo;
    // backward: gradients of q, k and v, token strides in elements
    void *dq, *dk, *dv;
    int64_t dqs, dks, dvs;
    const void *wq, *wk;  // norm weights [d], both or neither
    void *dwq, *dwk;      // their gradients, each may be null
    float *partial;       // [blocks][2][d]
    const int64_t *positions;  // [axes][P][B][N/P] or null
    int axes;
    int64_t tokens;            // P * B * N/P
    int64_t N;
    int Np, B;  // tokens per shard, sequences
    int Hq, Hkv, Hqp, Hkvp;
    int to_head;
    int half;  // rot / 2
    float eps;
    // set by the launch: tokens that are worked on whole, runs of a token, parts
    // of the other tokens and the runs of a part, and 2^32 / (H/P) rounded up (0
    // for H/P = 1)
    int64_t whole;
    int runs, splits, runs_per_split;
    unsigned magic_q, magic_k;
    uint64_t turn[kNormRopeMaxHalf];  // inv_freq / 2 pi as a 64-bit fraction of a turn
    uint8_t axis[kNormRopeMaxHalf];
};
uint64_t turn_fraction(double inv_freq);
cudaError_t launch_norm_rope(NormRopeParams &p, int d, bool inter, bool bwd, int esize, cudaStream_t s);

// ------------------------------------------------- norms around a block
struct ResidualNormParams {
    const void *x, *y;           // residual stream, block output (null: none)
    const void *w1, *w2, *gate;  // norm weights, the gate's rows; w2 and gate may be null
    void *h, *z;                 // forward outputs; h may be null
    float *rstd_out;             // forward: [2][T] or null
    const float *rstd;           // backward
    const void *dh, *dz;         // dh may be null
    void *dx, *dy;
    void *dw1, *dw2, *dgate;     // each may be null
    float scale, eps;
    int64_t T;    // tokens
    int64_t run;  // neighbouring tokens that share a gate: N/P with a gate for every sequence, else T
    int gates;    // rows of gate: 0, 1 or B
    int D;
    // set by the launch: warps of a group and the lanes a row has in a warp, groups of
    // a block, rows it works on at once (backward; 0 for one), rows of a slot, slots of the ring
    int warps, lanes, groups, parts, slot_rows, slots;
    int block_rows;        // rows of a block, with a gate for every sequence
    float *part1, *partA;  // the blocks' sums: [blocks][D], [blocks + runs][D]
    int64_t part1_elems, partA_elems;
    WaitCfg w;
};
// How rows are laid over a block's threads.
struct ResidualNormPlan {
    int chunks, warps, lanes, groups, parts, slot_rows, slots, blocks, block_rows, threads;
    size_t smem;
};
cudaError_t launch_residual_norm_f32(const ResidualNormParams &p, const ResidualNormPlan &q, bool bwd, cudaStream_t s);
size_t residual_norm_workspace(int64_t T, int64_t Np, int D);
cudaError_t launch_residual_norm(ResidualNormParams &p, bool bwd, int esize, void *workspace, cudaStream_t s);

// ------------------------------------------------------- sharded loss
cudaError_t launch_sharded_ce(const void *logits, const int64_t *labels, void *dlogits, float *shard_loss,
                              int64_t *shard_good, float *total, int64_t B, int64_t N, int64_t V, int P, int esize,
                              void *workspace, cudaStream_t stream);
size_t sharded_ce_workspace(int64_t B, int64_t N, int P);

// ------------------------------------------ LM head and sharded loss in one
cudaError_t launch_sharded_linear_ce(const void *hidden, const void *weight, const int64_t *labels, void *dhidden,
                                     void *dweight, float *shard_loss, int64_t *shard_good, float *total, int64_t B,
                                     int64_t N, int D, int V, int P, int esize, void *workspace, cudaStream_t stream);
size_t sharded_linear_ce_workspace(int64_t B, int64_t N, int D, int V, int P, bool grad, int esize);

}  // namespace uly

#include <ulysses.h>

namespace uly {

// Validated attention calls (ulysses_api.cu), shared by the C entry points
// and the ring-attention orchestration.
uly_status attn_fwd_impl(const void *q, const void *k, const void *v, void *o, float *lse, int64_t B, int64_t N,
                         int32_t Hq_local, int32_t Hkv_local, int32_t d, int32_t num_shards, int32_t causal,
                         const int32_t *cu_seqlens_host, int32_t num_docs, float softmax_scale, uly_dtype dtype,
                         void *workspace, size_t workspace_bytes, void *stream, RowLayout L);
uly_status attn_bwd_impl(const void *q, const void *k, const void *v, const void *o, const float *lse,
                         const void *dout, void *dq, void *dk, void *dv, int64_t B, int64_t N, int32_t Hq_local,
                         int32_t Hkv_local, int32_t d, int32_t num_shards, int32_t causal,
                         const int32_t *cu_seqlens_host, int32_t num_docs, float softmax_scale, uly_dtype dtype,
                         void *workspace, size_t workspace_bytes, void *stream, RowLayout L);
RowLayout head_rows(int64_t B, int64_t N, int32_t S);

// ring attention (ring.cu)
size_t ring_workspace_size(int64_t B, int64_t N, int Hq, int Hkv, int d, int P, bool bwd, uly_dtype dt);
uly_status ring_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int64_t B, int64_t N, int Hq,
                    int Hkv, int d, int P, int causal, float scale, uly_dtype dt, void *workspace, size_t ws_bytes,
                    cudaStream_t s);
uly_status ring_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dout,
                    void *dq, void *dk, void *dv, int64_t B, int64_t N, int Hq, int Hkv, int d, int P, int causal,
                    float scale, uly_dtype dt, void *workspace, size_t ws_bytes, cudaStream_t s);

}  // namespace uly
