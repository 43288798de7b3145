// The LM head's product and the sequence-parallel loss in one operator: next-
// token cross entropy of hidden states h [P][B][N/P][D] under a head weight
// W [V][D], with the labels shifted over the whole sequence and the ranks'
// losses weighted by their good tokens as in sharded_loss.cu, and the
// gradients of the total with respect to h and W.  The logits
//   x_rv = <h_r, w_v>
// are never kept: the good rows are taken in pieces of at most kPieceRows, and
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
#include "uly_internal.h"

namespace uly {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kStatCols = 64;

template <typename T>
struct Types;
template <>
struct Types<uint16_t> {
    using E = uint16_t;  // fp16 bits of e, then bf16 bits of g
};
template <>
struct Types<float> {
    using E = float;
};

__device__ __forceinline__ float ld(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ void st(uint16_t *p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xffffu); }
__device__ __forceinline__ void st(float *p, float v) { *p = v; }

__device__ __forceinline__ uint16_t half_bits(float v)
{
    uint16_t r;
    asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float half_value(uint16_t b)
{
    float r;
    asm("cvt.f32.f16 %0, %1;" : "=f"(r) : "h"(b));
    return r;
}

// Rows of the piece starting at good row `base`: device data, since the number
// of good rows is.
__device__ __forceinline__ int piece_count(const int *n_good, int64_t base, int rows)
{
    const int64_t left = *n_good - base;
    return left <= 0 ? 0 : (left < rows ? static_cast<int>(left) : rows);
}

// Good rows in order: index[i] = row of the i-th one, n_good = how many.
__global__ void __launch_bounds__(1024) compact_kernel(const int32_t *__restrict__ shifted, int64_t rows,
                                                       int32_t *__restrict__ index, int *__restrict__ n_good)
{
    __shared__ int warp_sum[32];
    int done = 0;
    for (int64_t base = 0; base < rows; base += 1024) {
        const int64_t r = base + threadIdx.x;
        const bool good = r < rows && shifted[r] >= 0;
        const unsigned mask = __ballot_sync(0xffffffffu, good);
        if (lane_id() == 0)
            warp_sum[warp_id()] = __popc(mask);
        __syncthreads();
        int before = done, all = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp_id() ? warp_sum[w] : 0;
            all += warp_sum[w];
        }
        if (good)
            index[before + __popc(mask & ((1u << lane_id()) - 1u))] = static_cast<int32_t>(r);
        done += all;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        *n_good = done;
}

// The piece's hidden rows next to each other, zeros up to a multiple of 64.
template <typename T>
__global__ void gather_kernel(const T *__restrict__ hidden, const int32_t *__restrict__ index,
                              const int *__restrict__ n_good, int64_t base, int rows, int D, T *__restrict__ out)
{
    const int cnt = piece_count(n_good, base, rows), r = blockIdx.x;
    if (r >= (cnt + 63) / 64 * 64)
        return;
    const uint4 *src = r < cnt ? reinterpret_cast<const uint4 *>(hidden + static_cast<int64_t>(index[base + r]) * D) : nullptr;
    uint4 *dst = reinterpret_cast<uint4 *>(out + static_cast<int64_t>(r) * D);
    for (int i = threadIdx.x; i < D * static_cast<int>(sizeof(T)) / 16; i += blockDim.x)
        dst[i] = src ? src[i] : make_uint4(0, 0, 0, 0);
}

// Zero gradient of the rows without a label.
template <typename T>
__global__ void zero_ignored_kernel(const int32_t *__restrict__ shifted, int D, T *__restrict__ dhidden)
{
    const int64_t r = blockIdx.x;
    if (shifted[r] >= 0)
        return;
    uint4 *dst = reinterpret_cast<uint4 *>(dhidden + r * D);
    for (int i = threadIdx.x; i < D * static_cast<int>(sizeof(T)) / 16; i += blockDim.x)
        dst[i] = make_uint4(0, 0, 0, 0);
}

enum { kLogits = 0, kDh = 1, kDw = 2 };

struct GemmArgs {
    const void *h, *w;  // gathered rows [rows][D], weight [V][D]
    void *g;            // [rows][ldg]
    int64_t ldg;
    const int32_t *index, *shifted;
    const int *n_good;
    int64_t base;
    int rows, D, V;
    float2 *stats;  // [rows][stat_tiles] (c, s)
    int stat_tiles;
    float *target;  // [rows] target logits
    int keep;       // logits: keep e
    void *dh, *dw;
    float *acc;  // [V][D] across pieces
};

// C[m][n] = sum_k A(m, k) B(n, k), 64 x 64 tiles, 4 x 4 a thread.
template <typename T, int kMode>
__global__ void __launch_bounds__(256) gemm_kernel(const __grid_constant__ GemmArgs a)
{
    using E = typename Types<T>::E;
    const int cnt = piece_count(a.n_good, a.base, a.rows);
    const bool last = a.base + a.rows >= *a.n_good;
    if (kMode != kDw && static_cast<int>(blockIdx.y) * 64 >= cnt)
        return;
    if (kMode == kDw && cnt == 0 && a.base > 0)
        return;
    const int M = kMode == kDw ? a.V : cnt, N = kMode == kLogits ? a.V : a.D;
    const int K = kMode == kLogits ? a.D : (kMode == kDh ? a.V : cnt);
    const T *h = static_cast<const T *>(a.h), *w = static_cast<const T *>(a.w);
    E *g = static_cast<E *>(a.g);
    __shared__ float As[16][65], Bs[16][65];
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float c[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            // k fastest for the operands whose rows run along k
            const int kf = i % 16, rf = i / 16, rs = i % 64, ks = i / 64;
            if (kMode == kDw) {
                const int m = m0 + rs, k = k0 + ks;
                As[ks][rs] = m < M && k < K ? ld(g + k * a.ldg + m) : 0.f;
            } else {
                const int m = m0 + rf, k = k0 + kf;
                const bool in = m < M && k < K;
                As[kf][rf] = !in ? 0.f : (kMode == kLogits ? ld(h + static_cast<int64_t>(m) * a.D + k) : ld(g + m * a.ldg + k));
            }
            if (kMode == kLogits) {
                const int n = n0 + rf, k = k0 + kf;
                Bs[kf][rf] = n < N && k < K ? ld(w + static_cast<int64_t>(n) * a.D + k) : 0.f;
            } else {
                const int n = n0 + rs, k = k0 + ks;
                Bs[ks][rs] = n < N && k < K ? ld((kMode == kDh ? w : h) + static_cast<int64_t>(k) * a.D + n) : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    c[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], c[i][j]);
        __syncthreads();
    }
    const float inv_t = 1.f / static_cast<float>(*a.n_good > 1 ? *a.n_good : 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i;
        if (kMode == kLogits) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mx = fmaxf(mx, n0 + tx * 4 + j < N ? c[i][j] : -INFINITY);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float c2 = mx * kLog2e;
            const int y = m < M ? a.shifted[a.index[a.base + m]] : -1;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n >= N)
                    continue;
                const float e = exp2f(fmaf(c[i][j], kLog2e, -c2));
                sum += e;
                if (m >= M)
                    continue;
                if (n == y)
                    a.target[m] = c[i][j];
                if (a.keep) {
                    if constexpr (sizeof(E) == 2)
                        g[m * a.ldg + n] = half_bits(e);
                    else
                        g[m * a.ldg + n] = e;
                }
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (tx == 0 && m < M)
                a.stats[static_cast<int64_t>(m) * a.stat_tiles + blockIdx.x] = make_float2(c2, sum);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (m >= M || n >= N)
                    continue;
                if (kMode == kDh) {
                    st(static_cast<T *>(a.dh) + static_cast<int64_t>(a.index[a.base + m]) * a.D + n, c[i][j] * inv_t);
                } else {
                    const int64_t o = static_cast<int64_t>(m) * a.D + n;
                    const float v = c[i][j] + (a.base > 0 ? a.acc[o] : 0.f);
                    if (last)
                        st(static_cast<T *>(a.dw) + o, v * inv_t);
                    else
                        a.acc[o] = v;
                }
            }
        }
    }
}

// One CTA per row of the piece: the row's loss, and with the gradient e -> g.
template <typename T>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ GemmArgs a, float *__restrict__ row_loss)
{
    using E = typename Types<T>::E;
    const int cnt = piece_count(a.n_good, a.base, a.rows), r = blockIdx.x;
    if (r >= (cnt + 63) / 64 * 64)
        return;
    E *g = static_cast<E *>(a.g) + r * a.ldg;
    if (r >= cnt) {
        if (a.keep)
            for (int v = threadIdx.x; v < a.V; v += 256)
                g[v] = 0;
        return;
    }
    __shared__ float red[2][8];
    const float2 *stats = a.stats + static_cast<int64_t>(r) * a.stat_tiles;
    float C = -INFINITY;
    for (int t = threadIdx.x; t < a.stat_tiles; t += 256)
        C = fmaxf(C, stats[t].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        C = fmaxf(C, __shfl_xor_sync(0xffffffffu, C, o));
    if (lane_id() == 0)
        red[0][warp_id()] = C;
    __syncthreads();
    for (int w = 0; w < 8; ++w)
        C = fmaxf(C, red[0][w]);
    float S = 0.f;
    for (int t = threadIdx.x; t < a.stat_tiles; t += 256)
        S += stats[t].y * exp2f(stats[t].x - C);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        S += __shfl_xor_sync(0xffffffffu, S, o);
    if (lane_id() == 0)
        red[1][warp_id()] = S;
    __syncthreads();
    S = 0.f;
    for (int w = 0; w < 8; ++w)
        S += red[1][w];
    const int row = a.index[a.base + r];
    const int y = a.shifted[row];
    if (threadIdx.x == 0)
        row_loss[row] = (log2f(S) - fmaf(a.target[r], kLog2e, -C)) * kLn2;
    if (!a.keep)
        return;
    const float inv = 1.f / S;
    for (int v = threadIdx.x; v < a.V; v += 256) {
        const float f = exp2f(stats[v / kStatCols].x - C) * inv;
        if constexpr (sizeof(E) == 2)
            st(g + v, half_value(g[v]) * f - (v == y ? 1.f : 0.f));
        else
            g[v] = g[v] * f - (v == y ? 1.f : 0.f);
    }
}

constexpr int kPieceRows = 8192;
size_t up(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
    size_t good, n_good, shifted, row_loss, index, target, stats, h, g, acc, total;
    int64_t ldg;
    int rows, stat_tiles;
};

Layout layout(int64_t B, int64_t N, int D, int V, int P, bool grad, int esize)
{
    Layout L = {};
    const int64_t T = B * N;
    L.rows = static_cast<int>(std::min<int64_t>(kPieceRows, (T + 63) / 64 * 64));
    L.ldg = (V + 63) / 64 * 64;
    L.stat_tiles = (V + kStatCols - 1) / kStatCols;
    size_t o = 0;
    auto take = [&](size_t &at, size_t bytes) { at = o, o += up(bytes); };
    take(L.good, sizeof(unsigned long long) * P);
    take(L.n_good, sizeof(int));
    take(L.shifted, sizeof(int32_t) * T);
    take(L.row_loss, sizeof(float) * T);
    take(L.index, sizeof(int32_t) * T);
    take(L.target, sizeof(float) * L.rows);
    take(L.stats, sizeof(float2) * L.rows * static_cast<size_t>(L.stat_tiles));
    take(L.h, static_cast<size_t>(L.rows) * D * esize);
    if (grad) {
        take(L.g, static_cast<size_t>(L.rows) * L.ldg * esize);
        if (T > L.rows)
            take(L.acc, sizeof(float) * static_cast<size_t>(V) * D);
    }
    L.total = o;
    return L;
}

template <typename T>
cudaError_t run(const void *hidden, const void *weight, const int64_t *labels, void *dhidden, void *dweight,
                float *shard_loss, int64_t *shard_good, float *total, int64_t B, int64_t N, int D, int V, int P,
                uint8_t *ws, cudaStream_t s)
{
    const bool grad = dhidden || dweight;
    const Layout L = layout(B, N, D, V, P, grad, sizeof(T));
    const int64_t rows = B * N;
    auto *good = reinterpret_cast<unsigned long long *>(ws + L.good);
    auto *shifted = reinterpret_cast<int32_t *>(ws + L.shifted);
    auto *row_loss = reinterpret_cast<float *>(ws + L.row_loss);
    GemmArgs a = {};
    a.h = ws + L.h;
    a.w = weight;
    a.g = ws + L.g;
    a.ldg = L.ldg;
    a.index = reinterpret_cast<int32_t *>(ws + L.index);
    a.shifted = shifted;
    a.n_good = reinterpret_cast<int *>(ws + L.n_good);
    a.rows = L.rows;
    a.D = D;
    a.V = V;
    a.stats = reinterpret_cast<float2 *>(ws + L.stats);
    a.stat_tiles = L.stat_tiles;
    a.target = reinterpret_cast<float *>(ws + L.target);
    a.keep = grad;
    a.dh = dhidden;
    a.dw = dweight;
    a.acc = reinterpret_cast<float *>(ws + L.acc);
    cudaError_t e = launch_shift_count(labels, shifted, good, B, N, P, V, s);
    if (e == cudaSuccess)
        e = cudaMemsetAsync(row_loss, 0, sizeof(float) * rows, s);
    if (e != cudaSuccess)
        return e;
    compact_kernel<<<1, 1024, 0, s>>>(shifted, rows, reinterpret_cast<int32_t *>(ws + L.index),
                                      reinterpret_cast<int *>(ws + L.n_good));
    if (dhidden)
        zero_ignored_kernel<T><<<static_cast<unsigned>(rows), 128, 0, s>>>(shifted, D, static_cast<T *>(dhidden));
    const unsigned mt = (L.rows + 63) / 64, vt = (V + 63) / 64, dt = (D + 63) / 64;
    for (int64_t base = 0; base < rows; base += L.rows) {
        a.base = base;
        gather_kernel<T><<<L.rows, 128, 0, s>>>(static_cast<const T *>(hidden), a.index, a.n_good, base, L.rows, D,
                                                reinterpret_cast<T *>(ws + L.h));
        gemm_kernel<T, kLogits><<<dim3(vt, mt), 256, 0, s>>>(a);
        rows_kernel<T><<<L.rows, 256, 0, s>>>(a, row_loss);
        if (dhidden)
            gemm_kernel<T, kDh><<<dim3(dt, mt), 256, 0, s>>>(a);
        if (dweight)
            gemm_kernel<T, kDw><<<dim3(dt, vt), 256, 0, s>>>(a);
    }
    return launch_shard_totals(row_loss, good, shard_loss, shard_good, total, B, N, P, s);
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
        return run<uint16_t>(hidden, weight, labels, dhidden, dweight, shard_loss, shard_good, total, B, N, D, V, P,
                             ws, s);
    return run<float>(hidden, weight, labels, dhidden, dweight, shard_loss, shard_good, total, B, N, D, V, P, ws, s);
}

}  // namespace uly
