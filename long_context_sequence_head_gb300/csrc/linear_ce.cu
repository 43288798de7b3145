// The LM head's product and the sequence-parallel loss in one operator: next-
// token cross entropy of hidden states h [P][B][N/P][D] under a head weight
// W [V][D], with the labels shifted over the whole sequence and the ranks'
// losses weighted by their good tokens as in sharded_loss.cu, and the
// gradients of the total with respect to h and W.  The logits
//   x_rv = <h_r, w_v>
// are never kept: the good rows are taken in pieces of a few thousand, and
// for each piece
//   1. logits   x = h W^T; every (row, column tile) leaves its maximum c (in
//               units of log2), its sum s of e = 2^(x log2 e - c), the row's
//               target logit, and e itself in the piece buffer;
//   2. rows     C = max c, S = sum s 2^(c - C); loss = ln S + (C ln 2 - x_y);
//               e becomes g = softmax - onehot = e 2^(c - C) / S - [v == y];
//   3. dh       = g W / T for the piece's rows;
//   4. dW      += g^T h / T, in fp32 across the pieces, rounded once at the end.
// That is three products instead of the four that recomputing the logits from
// a kept log-sum-exp would take.  Rows without a label are left out before the
// first product: the good rows are gathered next to each other.
#include "linear_ce.h"

namespace uly {
namespace {

// Rows of a piece: as many as hold kPieceBytes of exponentials and gradients (2
// bytes a value, 10 in fp32), at least 1024 and at most 65,536.  dW is carried
// from piece to piece in fp32: at D = 2560 and V = 151,936 its 1.6 GB read and
// written are 0.46 ms beside 12 ms of products for a piece of 8448 rows.
constexpr int64_t kPieceBytes = int64_t(2500) << 20;
// Vocabularies above this take 512 threads a row, others 128.  Whole calls with
// 512 / 128, us: 4096 rows x 16,000 words (D = 256) 194 / 175, x 3208 107 / 86;
// 1024 rows x 50,257 (D = 776) 320 / 327, 512 x 32,000 90 / 97.
constexpr int kLongRow = 24576;

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xffffu); }

__device__ __forceinline__ float2 f16x2_values(uint32_t b)
{
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(b));
    return make_float2(lo, hi);
}

// Three bf16 parts of x: x1 + x2 + x3 = x up to 2^-26 |x|.
struct Parts {
    uint16_t p[3];
};
__device__ __forceinline__ Parts split3(float x)
{
    Parts r;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        r.p[i] = bf16_bits(x);
        x -= bf16_value(r.p[i]);
    }
    return r;
}

// Eight values as planes, 16 bytes each, `plane` elements apart.
__device__ __forceinline__ void store_planes(uint16_t *out, int64_t plane, const float (&x)[8])
{
    Parts q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        q[j] = split3(x[j]);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = q[2 * j].p[i] | static_cast<uint32_t>(q[2 * j + 1].p[i]) << 16;
        *reinterpret_cast<uint4 *>(out + i * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Eight values of an fp32 row of D values (a multiple of 4), zeros past its end.
__device__ __forceinline__ void load8(const float *row, int i, int D, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(row + i);
    const float4 b = i + 4 < D ? *reinterpret_cast<const float4 *>(row + i + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The totals of a call without gradients.
__global__ void __launch_bounds__(1024) totals_kernel(const CeTotals t)
{
    grid_wait();
    __shared__ float2 part[32];
    for (int r = 0; r < t.P; ++r) {
        const float *base = t.row_loss + r * t.per_shard;
        float2 s = make_float2(0.f, 0.f);
        for (int64_t i = threadIdx.x; i < t.per_shard; i += 1024)
            s = two_sum(s, make_float2(base[i], 0.f));
        s = warp_two_sum(s);
        if (lane_id() == 0)
            part[warp_id()] = s;
        __syncthreads();
        if (warp_id() == 0)
            ce_shard(t, r, warp_two_sum(part[lane_id()]));
        __syncthreads();
    }
    if (warp_id() == 0)
        ce_total(t);
}

// One block: the labels shifted over the whole sequence, each shard's good
// rows, and the good rows in order (index[i] = row of the i-th one).  A row's
// loss starts as 0.  Labels out of range are reported and ignored.  8192 rows a
// round of about 6 us, against 8 ms of products behind as many rows.
__global__ void __launch_bounds__(1024) labels_kernel(const int64_t *__restrict__ labels, int32_t *__restrict__ shifted,
                                                      unsigned long long *__restrict__ good,
                                                      float *__restrict__ row_loss, int32_t *__restrict__ index,
                                                      int *__restrict__ n_good, unsigned rows, unsigned Np, unsigned B,
                                                      int P, int V, unsigned *status)
{
    constexpr int kEach = 8;
    __shared__ int warp_sum[32];
    grid_next();
    for (int r = threadIdx.x; r < P; r += 1024)
        good[r] = 0;
    __syncthreads();
    int done = 0;
    for (int64_t base = 0; base < rows; base += 1024 * kEach) {
        const int64_t first = base + static_cast<int64_t>(threadIdx.x) * kEach;
        int32_t y[kEach];
        int mine = 0;
        // place in the shard's sequence; the next token is the next row, or,
        // at the end of a shard, the first of the same sequence in the next
        unsigned t = static_cast<unsigned>(first < rows ? first : 0) % Np;
#pragma unroll
        for (int i = 0; i < kEach; ++i, ++t) {
            y[i] = -100;
            if (first + i >= rows)
                continue;
            if (t == Np)
                t = 0;
            const int64_t next = first + i + 1 + (t + 1 == Np ? static_cast<int64_t>(B - 1) * Np : 0);
            if (next < rows) {
                const int64_t lab = labels[next];
                if (lab >= 0 && lab < V)
                    y[i] = static_cast<int32_t>(lab);
                else if (lab != -100)
                    atomicOr(status, kDevBadArg);
            }
            mine += y[i] >= 0;
        }
        // places of this thread's good rows among all
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane_id() >= o ? v : 0;
        }
        if (lane_id() == 31)
            warp_sum[warp_id()] = upto;
        __syncthreads();
        int sum = warp_sum[lane_id()];  // every warp scans the 32 sums
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane_id() >= o ? v : 0;
        }
        const int before = __shfl_sync(0xffffffffu, sum, warp_id() > 0 ? warp_id() - 1 : 0);
        int at = done + upto - mine + (warp_id() > 0 ? before : 0);
        done += __shfl_sync(0xffffffffu, sum, 31);
        // a warp's 256 rows are of one shard, mostly
        const int64_t w0 = base + static_cast<int64_t>(warp_id()) * 32 * kEach;
        const unsigned r0 = static_cast<unsigned>(w0 < rows ? w0 : 0) / (Np * B);
        const bool one = w0 + 32 * kEach <= static_cast<int64_t>(r0 + 1) * Np * B;
        if (one && lane_id() == 31 && upto > 0)
            atomicAdd(&good[r0], static_cast<unsigned long long>(upto));
        if (first + kEach <= rows) {
#pragma unroll
            for (int i = 0; i < kEach; i += 4) {
                *reinterpret_cast<int4 *>(shifted + first + i) = make_int4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                *reinterpret_cast<float4 *>(row_loss + first + i) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (first + i >= rows)
                continue;
            if (first + kEach > rows) {
                shifted[first + i] = y[i];
                row_loss[first + i] = 0.f;
            }
            if (y[i] >= 0) {
                index[at++] = static_cast<int32_t>(first + i);
                if (!one)
                    atomicAdd(&good[static_cast<unsigned>(first + i) / (Np * B)], 1ull);
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        *n_good = done;
}

// Eight values of row `row`, columns [i, i + 8), to the products' layout.
template <bool kSplit>
__device__ __forceinline__ void lay8(const void *src, int64_t row, int i, int D, uint16_t *out, int64_t to, int64_t pitch,
                                     int64_t plane)
{
    if constexpr (kSplit) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (src)
            load8(static_cast<const float *>(src) + row * D, i, D, x);
        store_planes(out + to * pitch + i, plane, x);
    } else {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (src)
            x = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + row * D + i);
        *reinterpret_cast<uint4 *>(out + to * pitch + i) = x;
    }
}

// The piece's hidden rows next to each other (fp32: as planes), with their
// labels; zeros up to a multiple of 64 rows, where dW's contraction ends.  The
// first piece also clears the gradient of the rows without a label: its row r
// then stands for row r of the call too.  A thread takes eight values.
template <bool kSplit>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ CeArgs a, const void *__restrict__ hidden,
                                                     const int32_t *__restrict__ shifted, int32_t *__restrict__ label,
                                                     uint16_t *__restrict__ out, int64_t ldh, int64_t rows)
{
    grid_wait();
    grid_next();
    const int cnt = ce_piece_rows(a), vecs = (a.D + 7) / 8;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, r = at / vecs;
    const int i = static_cast<int>(at - r * vecs) * 8;
    if (a.base == 0 && a.dh != nullptr && r < rows && shifted[r] < 0) {
        uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.dh) + (r * a.D + i) * (kSplit ? 4 : 2));
        to[0] = make_uint4(0, 0, 0, 0);
        if (kSplit && i + 4 < a.D)
            to[1] = make_uint4(0, 0, 0, 0);
    }
    if (r >= (cnt + kCeStep - 1) / kCeStep * kCeStep)
        return;
    const bool live = r < cnt;
    const int64_t src = live ? a.index[a.base + r] : 0;
    if (i == 0)
        label[r] = live ? shifted[src] : -1;
    lay8<kSplit>(live ? hidden : nullptr, src, i, a.D, out, r, ldh, ldh * a.rows);
}

// fp32 weight as planes.
__global__ void __launch_bounds__(256) split_weight_kernel(const float *__restrict__ w, int D, int V,
                                                           uint16_t *__restrict__ out, int64_t ldw)
{
    grid_wait();
    grid_next();
    const int vecs = (D + 7) / 8;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, v = at / vecs;
    if (v < V)
        lay8<true>(w, v, static_cast<int>(at - v * vecs) * 8, D, out, v, ldw, ldw * V);
}

// One CTA per row of the piece, or several that share a row's columns where
// there are few rows: the row's loss, and with a gradient e -> g, in place in
// bf16, to planes in fp32.  e stays relative to its own columns'
// maximum until here, as fp16 (2^-11 of e; below 2^-14 of that maximum the
// error is 2^-25 of it): stored as bf16, g would be rounded to 8 bits twice.
// Memory-bound: 5,734 rows of 151,936 in 0.55 ms, 6.3 TB/s; 4,830 of 50,257 in
// 0.16 ms, 6.1 TB/s (the row's statistics are joined while its first values are
// on their way; loaded after them it took 0.18).
template <bool kSplit, int kRowThreads>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ CeArgs a, uint16_t *__restrict__ g,
                                                           const int32_t *__restrict__ label,
                                                           float *__restrict__ row_loss, int parts)
{
    grid_wait();
    grid_next();
    const int cnt = ce_piece_rows(a), r = blockIdx.x / parts, part = blockIdx.x % parts;
    if (r >= (cnt + kCeStep - 1) / kCeStep * kCeStep)
        return;
    uint16_t *grow = g + r * a.ldg;
    const int64_t plane = a.ldg * a.rows;
    if (r >= cnt) {
        if (a.keep)
            for (int v = (part * kRowThreads + threadIdx.x) * 8; v < a.V; v += parts * kRowThreads * 8)
#pragma unroll
                for (int i = 0; i < (kSplit ? 3 : 1); ++i)
                    *reinterpret_cast<uint4 *>(grow + i * plane + v) = make_uint4(0, 0, 0, 0);
        return;
    }
    constexpr int kWarps = kRowThreads / 32;
    constexpr int kAhead = kSplit ? 2 : 4;  // vectors of 8 values loaded before the first is used
    __shared__ float red[2][kWarps];
    const int v_step = parts * kRowThreads * 8, v_first = (part * kRowThreads + threadIdx.x) * 8;
    struct Eight {
        uint4 v[kSplit ? 2 : 1];
    } next[kAhead];
    auto fetch = [&](int v0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = v0 + i * v_step;
            if (v < a.V) {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.e) +
                                                                   (r * a.ldg + v) * (kSplit ? 4 : 2));
                next[i].v[0] = src[0];
                if constexpr (kSplit)
                    next[i].v[1] = src[1];
            }
        }
    };
    if (a.keep)
        fetch(v_first);  // on its way while the row's statistics are joined
    const float2 *stats = a.stats + static_cast<int64_t>(r) * a.stat_tiles;
    float C = -INFINITY;
    for (int t = threadIdx.x; t < a.stat_tiles; t += kRowThreads)
        C = fmaxf(C, stats[t].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        C = fmaxf(C, __shfl_xor_sync(0xffffffffu, C, o));
    if (lane_id() == 0)
        red[0][warp_id()] = C;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
        C = fmaxf(C, red[0][w]);
    float S = 0.f;
    for (int t = threadIdx.x; t < a.stat_tiles; t += kRowThreads)
        S += stats[t].y * exp2f(stats[t].x - C);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        S += __shfl_xor_sync(0xffffffffu, S, o);
    if (lane_id() == 0)
        red[1][warp_id()] = S;
    __syncthreads();
    S = 0.f;
    for (int w = 0; w < kWarps; ++w)
        S += red[1][w];
    const int y = label[r];
    if (part == 0 && threadIdx.x == 0)  // ln S + C ln 2 - x_y, with C taken out of x_y before anything is rounded
        row_loss[a.index[a.base + r]] = (log2f(S) - fmaf(a.target[r], kLog2e, -C)) * kLn2;
    if (!a.keep)
        return;
    const float inv = 1.f / S;
    for (int v0 = v_first; v0 < a.V; v0 += kAhead * v_step) {
        Eight now[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            now[i] = next[i];
        fetch(v0 + kAhead * v_step);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = v0 + i * v_step;
            if (v >= a.V)
                break;
            const float f = exp2f(stats[v / kCeStatCols].x - C) * inv;
            float x[8];
            const uint32_t w[4] = {now[i].v[0].x, now[i].v[0].y, now[i].v[0].z, now[i].v[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (kSplit) {
                    x[j] = __uint_as_float(w[j]);
                } else {
                    const float2 p = f16x2_values(w[j]);
                    x[2 * j] = p.x, x[2 * j + 1] = p.y;
                }
            }
            if constexpr (kSplit) {
                const uint4 h = now[i].v[1];
                x[4] = __uint_as_float(h.x), x[5] = __uint_as_float(h.y), x[6] = __uint_as_float(h.z),
                x[7] = __uint_as_float(h.w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = x[j] * f - (v + j == y ? 1.f : 0.f);
            if constexpr (kSplit)
                store_planes(grow + v, plane, x);
            else
                *reinterpret_cast<uint4 *>(grow + v) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        }
    }
}

size_t up(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
    size_t good, n_good, shifted, row_loss, index, label, target, stats, h, w, e, g, acc, partial, total;
    int64_t ldh, ldg;
    int rows, stat_tiles;
};

Layout layout(int64_t B, int64_t N, int D, int V, int P, bool grad, int esize)
{
    Layout L = {};
    const int64_t T = B * N;
    const bool split = esize == 4;
    L.ldg = (V + 63) / 64 * 64;
    const int64_t fit = std::max<int64_t>(1024, kPieceBytes / (L.ldg * (split ? 10 : 2)) / kCeTile * kCeTile);
    L.rows = static_cast<int>(std::min<int64_t>(std::min<int64_t>(fit, 65536), (T + 63) / 64 * 64));
    L.ldh = (D + 63) / 64 * 64;
    L.stat_tiles = (V + kCeStatCols - 1) / kCeStatCols;
    const size_t planes = split ? 3 : 1, kept = static_cast<size_t>(L.rows) * L.ldg;
    size_t o = 0;
    auto take = [&](size_t &at, size_t bytes) { at = o, o += up(bytes); };
    take(L.good, sizeof(unsigned long long) * P);
    take(L.n_good, sizeof(int));
    take(L.shifted, sizeof(int32_t) * T);
    take(L.row_loss, sizeof(float) * T);
    take(L.index, sizeof(int32_t) * T);
    take(L.label, sizeof(int32_t) * L.rows);
    take(L.target, sizeof(float) * L.rows);
    take(L.stats, sizeof(float2) * L.rows * static_cast<size_t>(L.stat_tiles));
    take(L.h, planes * L.rows * L.ldh * 2);
    if (split)
        take(L.w, planes * V * L.ldh * 2);
    if (grad) {
        take(L.g, planes * kept * 2);
        L.e = L.g;  // bf16: e becomes g in place
        if (split)
            take(L.e, kept * 4);
        const size_t tiles = static_cast<size_t>((V + kCeTile - 1) / kCeTile) * ((D + kCeTile - 1) / kCeTile);
        if (T > L.rows)
            take(L.acc, sizeof(float) * kCeTileFloats * tiles);
        take(L.partial, sizeof(float) * kCeTileFloats *
                            std::max(ce_most_parts(kCeDh, L.rows, D, V), ce_most_parts(kCeDw, L.rows, D, V)));
    }
    L.total = o;
    return L;
}

template <bool kSplit>
cudaError_t run(const void *hidden, const void *weight, const int64_t *labels, void *dhidden, void *dweight,
                float *shard_loss, int64_t *shard_good, float *total, int64_t B, int64_t N, int D, int V, int P,
                uint8_t *ws, cudaStream_t s)
{
    constexpr int kEsize = kSplit ? 4 : 2;
    const bool grad = dhidden || dweight;
    const Layout L = layout(B, N, D, V, P, grad, kEsize);
    const int64_t rows = B * N;
    auto *good = reinterpret_cast<unsigned long long *>(ws + L.good);
    auto *shifted = reinterpret_cast<int32_t *>(ws + L.shifted);
    auto *row_loss = reinterpret_cast<float *>(ws + L.row_loss);
    auto *index = reinterpret_cast<int32_t *>(ws + L.index);
    auto *label = reinterpret_cast<int32_t *>(ws + L.label);
    auto *g = reinterpret_cast<uint16_t *>(ws + L.g);
    CeArgs a = {};
    a.n_good = reinterpret_cast<int *>(ws + L.n_good);
    a.rows = L.rows;
    a.D = D;
    a.V = V;
    a.ldg = L.ldg;
    a.e = ws + L.e;
    a.index = index;
    a.label = label;
    a.stats = reinterpret_cast<float2 *>(ws + L.stats);
    a.stat_tiles = L.stat_tiles;
    a.target = reinterpret_cast<float *>(ws + L.target);
    a.keep = grad;
    a.dh = dhidden;
    a.dw = dweight;
    a.acc = reinterpret_cast<float *>(ws + L.acc);
    a.partial = reinterpret_cast<float *>(ws + L.partial);
    // Few rows: each goes to several blocks, of at least two vectors a thread.
    const int parts = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(V / (2 * 8 * (V > kLongRow ? 512 : 128)), 4 * num_sms() / std::max<int64_t>(1, rows))));
    a.totals = CeTotals{row_loss, good, rows / P, P, shard_loss, total, shard_good};
    labels_kernel<<<1, 1024, 0, s>>>(labels, shifted, good, row_loss, index, a.n_good, static_cast<unsigned>(rows),
                                     static_cast<unsigned>(N / P), static_cast<unsigned>(B), P, V,
                                     device_status_ptr());
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const void *w = weight;
    int64_t ldw = D;
    const int64_t vecs = (D + 7) / 8;
    if (kSplit) {
        w = ws + L.w;
        ldw = L.ldh;
        e = launch_after(split_weight_kernel, (static_cast<int64_t>(V) * vecs + 255) / 256, 256, 0, s,
                         static_cast<const float *>(weight), D, V, reinterpret_cast<uint16_t *>(ws + L.w), ldw);
    }
    for (int64_t base = 0; base < rows; base += L.rows) {
        a.base = base;
        const int64_t blocks = ((base == 0 ? std::max<int64_t>(rows, L.rows) : L.rows) * vecs + 255) / 256;
        if (e == cudaSuccess)
            e = launch_after(gather_kernel<kSplit>, blocks, 256, 0, s, a, hidden, shifted, label,
                             reinterpret_cast<uint16_t *>(ws + L.h), L.ldh, rows);
        if (e == cudaSuccess)
            e = launch_ce_product(kCeLogits, a, ws + L.h, L.ldh, w, ldw, g, kEsize, s);
        if (e == cudaSuccess)
            e = launch_after(V > kLongRow ? rows_kernel<kSplit, 512> : rows_kernel<kSplit, 128>,
                             static_cast<int64_t>(L.rows) * parts, V > kLongRow ? 512 : 128, 0, s, a, g, label, row_loss,
                             parts);
        // the last product of a call makes the totals beside its own work
        const bool end = base + L.rows >= rows;
        a.make_totals = end && !dweight;
        if (e == cudaSuccess && dhidden)
            e = launch_ce_product(kCeDh, a, ws + L.h, L.ldh, w, ldw, g, kEsize, s);
        a.make_totals = end;
        if (e == cudaSuccess && dweight)
            e = launch_ce_product(kCeDw, a, ws + L.h, L.ldh, w, ldw, g, kEsize, s);
        if (e != cudaSuccess)
            return e;
    }
    if (e == cudaSuccess && !grad)
        e = launch_after(totals_kernel, 1, 1024, 0, s, a.totals);
    return e;
}

}  // namespace

size_t sharded_linear_ce_workspace(int64_t B, int64_t N, int D, int V, int P, bool grad, int esize)
{
    return layout(B, N, D, V, P, grad, esize).total;
}

cudaError_t launch_sharded_linear_ce(const void *hidden, const void *weight, const int64_t *labels, void *dhidden,
                                     void *dweight, float *shard_loss, int64_t *shard_good, float *total, int64_t B,
                                     int64_t N, int D, int V, int P, int esize, void *workspace, cudaStream_t s)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (esize == 2)
        return run<false>(hidden, weight, labels, dhidden, dweight, shard_loss, shard_good, total, B, N, D, V, P, ws,
                          s);
    return run<true>(hidden, weight, labels, dhidden, dweight, shard_loss, shard_good, total, B, N, D, V, P, ws, s);
}

}  // namespace uly
