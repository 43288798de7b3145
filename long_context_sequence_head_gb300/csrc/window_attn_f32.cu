// fp32 sliding-window attention with sinks, forward and backward (SIMT FFMA;
// TF32 tensor cores cannot meet the fp32 path's 1e-5).  Definitions as in
// window_attn.cu and attn_f32.cu.
//
// Tiles of 64 rows x 64 keys, 256 threads as 16 x 16.  A product of two tiles
// over d gives a thread 4 x 4 values from 8 shared loads of 16 bytes per 64 FFMA;
// products with P or dS give it 4 rows x d/16 columns.  Tiles are padded by 4
// floats a row, so that 8 neighbouring rows lie in different banks.  Shared
// memory and issue bound these kernels: at 8192 tokens of 8 heads of 64, window 1024,
// the forward takes 0.64 ms, the backward 1.89 ms, with the shared loads' pipe 59 and 68
// % busy and the FFMA pipe 46 and 49 %.  Loads of the next tile are not overlapped.
#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kT = kWindowTileF32;
constexpr int kThreads = 256;
constexpr int kPad = 4;
constexpr int kPitchP = kT + kPad;

// [lo, hi): the document of token i.
__device__ __forceinline__ void doc_bounds(const AttnShape &s, int64_t i, int64_t &lo, int64_t &hi)
{
    lo = 0;
    hi = s.N;
    if (s.cu_dev == nullptr)
        return;
    int a = 0, b = s.num_docs;
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (static_cast<int64_t>(s.cu_dev[m]) <= i)
            a = m;
        else
            b = m;
    }
    lo = s.cu_dev[a];
    hi = s.cu_dev[a + 1];
}

// The key tiles of a tile of rows: those of its first row's sinks, then those
// from its first row's window up to the last row.
struct KeyWalk {
    int sink, n_sink, lo, n;

    __device__ __forceinline__ KeyWalk(const AttnShape &s, int64_t q0)
    {
        const int64_t last = min(q0 + kT, s.N) - 1;
        int64_t start, end;
        doc_bounds(s, q0, start, end);
        const int64_t first = max(start, q0 - s.window + 1), sink_end = min(start + s.sinks, first);
        lo = static_cast<int>(first / kT);
        sink = static_cast<int>(start / kT);
        n_sink = sink_end > start ? static_cast<int>(min((sink_end - 1) / kT + 1, first / kT)) - sink : 0;
        n = n_sink + static_cast<int>(last / kT) - lo + 1;
    }
    __device__ __forceinline__ int64_t key0(int j) const
    {
        return static_cast<int64_t>(j < n_sink ? sink + j : lo + j - n_sink) * kT;
    }
};

// What row i of a document [start, ...) sees.
struct RowMask {
    int64_t start, row;
    int window, sinks;

    __device__ __forceinline__ bool sees(int64_t j) const
    {
        return j >= start && j <= row && (row - j < window || j - start < sinks);
    }
    // it sees no key but its own: dS is 0, and not what two sums of the same terms differ by
    __device__ __forceinline__ bool alone() const { return row == start || (window == 1 && sinks == 0); }
};

// 64 rows of a tensor of H heads (head layout) from token n0 on; rows past N are
// zero.  All of a thread's loads are on their way at once.
template <int D>
__device__ __forceinline__ void load_tile(float *dst, const float *src, const AttnShape &s, int64_t sb, int64_t n0,
                                          int H, int h, [[maybe_unused]] int64_t extent)
{
    constexpr int kPer = D / 4, kRows = kThreads / kPer;  // threads of a row, rows at once
    const int r0 = threadIdx.x / kPer, c = threadIdx.x % kPer * 4;
    const int64_t first = ((sb * s.N + n0 + r0) * H + h) * D + c, step = static_cast<int64_t>(kRows) * H * D;
    float4 v[kT / kRows];
#pragma unroll
    for (int i = 0; i < kT / kRows; ++i) {
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n0 + r0 + i * kRows < s.N && ULY_IN_BOUNDS(s.status, first + i * step, 4, extent, 0x63))
            v[i] = *reinterpret_cast<const float4 *>(src + first + i * step);
    }
#pragma unroll
    for (int i = 0; i < kT / kRows; ++i)
        *reinterpret_cast<float4 *>(dst + (r0 + i * kRows) * (D + kPad) + c) = v[i];
}

// x[i][c] = <a row ty + 16 i, b row tx + 16 c>
template <int D>
__device__ __forceinline__ void rows_by_rows(const float *a, const float *b, int tx, int ty, float (&x)[4][4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            x[i][c] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 u[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = *reinterpret_cast<const float4 *>(a + (ty + 16 * i) * (D + kPad) + k);
            w[i] = *reinterpret_cast<const float4 *>(b + (tx + 16 * i) * (D + kPad) + k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[i][c] = fmaf(u[i].x, w[c].x, x[i][c]);
                x[i][c] = fmaf(u[i].y, w[c].y, x[i][c]);
                x[i][c] = fmaf(u[i].z, w[c].z, x[i][c]);
                x[i][c] = fmaf(u[i].w, w[c].w, x[i][c]);
            }
    }
}

// acc[i][.] += sum over j of p[j][4 ty + i] m[j][columns 4 tx + 64 c ..]: p holds
// the products' index j as rows (kPitchP apart).
template <int D>
__device__ __forceinline__ void add_product(const float *p, const float *m, int tx, int ty, float (&acc)[4][D / 16])
{
#pragma unroll 4
    for (int j = 0; j < kT; ++j) {
        const float4 w = *reinterpret_cast<const float4 *>(p + j * kPitchP + 4 * ty);
        const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float4 v = *reinterpret_cast<const float4 *>(m + j * (D + kPad) + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][4 * c] = fmaf(f[i], v.x, acc[i][4 * c]);
                acc[i][4 * c + 1] = fmaf(f[i], v.y, acc[i][4 * c + 1]);
                acc[i][4 * c + 2] = fmaf(f[i], v.z, acc[i][4 * c + 2]);
                acc[i][4 * c + 3] = fmaf(f[i], v.w, acc[i][4 * c + 3]);
            }
        }
    }
}

// over the 16 lanes that share a row
__device__ __forceinline__ float row_max(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D>
constexpr size_t tile_bytes() { return sizeof(float) * kT * (D + kPad); }

// Writes 4 rows (4 ty + i) x D/16 columns of a thread.
template <int D>
__device__ __forceinline__ void store_rows(float *dst, const float (&acc)[4][D / 16], const float (&f)[4],
                                           const AttnShape &s, int64_t sb, int64_t n0, int H, int h, int tx, int ty,
                                           [[maybe_unused]] int64_t extent)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + 4 * ty + i;
        if (n >= s.N)
            continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int64_t off = s.L.off(s.N, sb, n, H, h, D) + 64 * c + 4 * tx;
            if (ULY_IN_BOUNDS(s.status, off, 4, extent, 0x64))
                *reinterpret_cast<float4 *>(dst + off) =
                    make_float4(acc[i][4 * c] * f[i], acc[i][4 * c + 1] * f[i], acc[i][4 * c + 2] * f[i],
                                acc[i][4 * c + 3] * f[i]);
        }
    }
}

// One block: 64 rows of one query head.  P goes through shared memory as
// [key][row]; a row's maximum and sum live with the 16 threads that made its
// scores (rows ty + 16 i), its output with those of rows 4 ty + i, so the
// rescaling factors go through shared memory too.
template <int D>
__global__ void __launch_bounds__(kThreads) window_fwd_f32_kernel(const __grid_constant__ AttnShape s,
                                                                  const float *__restrict__ q,
                                                                  const float *__restrict__ k,
                                                                  const float *__restrict__ v, float *__restrict__ o,
                                                                  float *__restrict__ lse)
{
    extern __shared__ __align__(16) float sm[];
    constexpr int kTile = kT * (D + kPad);
    float *sQ = sm, *sK = sm + kTile, *sV = sm + 2 * kTile, *sP = sm + 3 * kTile, *sF = sP + kT * kPitchP;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tiles = (s.N + kT - 1) / kT;
    const int64_t q0 = blockIdx.x % tiles * kT;
    const int h = static_cast<int>(blockIdx.x / tiles % s.Hq);
    const int64_t sb = blockIdx.x / tiles / s.Hq;
    const int kvh = h / (s.Hq / s.Hkv);
    load_tile<D>(sQ, q, s, sb, q0, s.Hq, h, s.q_elems);
    RowMask mask[4];
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mask[i].row = min(q0 + ty + 16 * i, s.N - 1);
        mask[i].window = s.window;
        mask[i].sinks = s.sinks;
        int64_t end;
        doc_bounds(s, mask[i].row, mask[i].start, end);
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            acc[i][c] = 0.f;
    }
    const KeyWalk walk(s, q0);
    for (int j = 0; j < walk.n; ++j) {
        const int64_t key0 = walk.key0(j);
        __syncthreads();
        load_tile<D>(sK, k, s, sb, key0, s.Hkv, kvh, s.kv_elems);
        load_tile<D>(sV, v, s, sb, key0, s.Hkv, kvh, s.kv_elems);
        __syncthreads();
        float x[4][4];
        rows_by_rows<D>(sQ, sK, tx, ty, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[i][c] = mask[i].sees(key0 + tx + 16 * c) ? x[i][c] * s.scale : -INFINITY;
                top = fmaxf(top, x[i][c]);
            }
            top = fmaxf(m[i], row_max(top));
            const float ref = top == -INFINITY ? 0.f : top;  // no key so far
            const float f = expf(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = expf(x[i][c] - ref);
                sum += p;
                sP[(tx + 16 * c) * kPitchP + ty + 16 * i] = p;
            }
            l[i] = l[i] * f + row_sum(sum);
            m[i] = top;
            if (tx == 0)
                sF[ty + 16 * i] = f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = sF[4 * ty + i];
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
                acc[i][c] *= f;
        }
        add_product<D>(sP, sV, tx, ty, acc);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = q0 + ty + 16 * i, li = (sb * s.Hq + h) * s.N + row;
        if (tx == 0) {
            sF[ty + 16 * i] = 1.f / l[i];
            if (row < s.N && ULY_IN_BOUNDS(s.status, li, 1, s.lse_elems, 0x65))
                lse[li] = m[i] + logf(l[i]);
        }
    }
    __syncthreads();
    const float f[4] = {sF[4 * ty], sF[4 * ty + 1], sF[4 * ty + 2], sF[4 * ty + 3]};
    store_rows<D>(o, acc, f, s, sb, q0, s.Hq, h, tx, ty, s.q_elems);
}

// D_i = <dO_i, O_i>, one warp a row.
template <int D>
__global__ void __launch_bounds__(kThreads) window_pre_f32_kernel(const __grid_constant__ AttnShape s,
                                                                  const float *__restrict__ o,
                                                                  const float *__restrict__ dout,
                                                                  float *__restrict__ Dv)
{
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (w >= s.SB * s.Hq * s.N)
        return;
    const int64_t i = w % s.N, sb = w / s.N / s.Hq;
    const int h = static_cast<int>(w / s.N % s.Hq);
    const int64_t off = s.L.off(s.N, sb, i, s.Hq, h, D);
    if (!ULY_IN_BOUNDS(s.status, off, D, s.q_elems, 0x66) || !ULY_IN_BOUNDS(s.status, w, 1, s.lse_elems, 0x67))
        return;
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        part = fmaf(dout[off + lane_id() + 32 * e], o[off + lane_id() + 32 * e], part);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        part += __shfl_xor_sync(0xffffffffu, part, x);
    if (lane_id() == 0)
        Dv[w] = part;
}

// One block: dQ of 64 rows of one query head, over the forward's walk.
template <int D>
__device__ __forceinline__ void window_dq(const AttnShape &s, int64_t block, float *sm, const float *__restrict__ q,
                                          const float *__restrict__ k, const float *__restrict__ v,
                                          const float *__restrict__ lse, const float *__restrict__ dout,
                                          const float *__restrict__ Dv, float *__restrict__ dq)
{
    constexpr int kTile = kT * (D + kPad);
    float *sQ = sm, *sO = sm + kTile, *sK = sm + 2 * kTile, *sV = sm + 3 * kTile, *sP = sm + 4 * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tiles = (s.N + kT - 1) / kT;
    const int64_t q0 = block % tiles * kT;
    const int h = static_cast<int>(block / tiles % s.Hq);
    const int64_t sb = block / tiles / s.Hq;
    const int kvh = h / (s.Hq / s.Hkv);
    load_tile<D>(sQ, q, s, sb, q0, s.Hq, h, s.q_elems);
    load_tile<D>(sO, dout, s, sb, q0, s.Hq, h, s.q_elems);
    RowMask mask[4];
    float L[4], Di[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mask[i].row = min(q0 + ty + 16 * i, s.N - 1);
        mask[i].window = s.window;
        mask[i].sinks = s.sinks;
        int64_t end;
        doc_bounds(s, mask[i].row, mask[i].start, end);
        const int64_t li = (sb * s.Hq + h) * s.N + mask[i].row;
        const bool ok = ULY_IN_BOUNDS(s.status, li, 1, s.lse_elems, 0x68);
        L[i] = ok ? lse[li] : 0.f;
        Di[i] = ok ? Dv[li] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            acc[i][c] = 0.f;
    }
    const KeyWalk walk(s, q0);
    for (int j = 0; j < walk.n; ++j) {
        const int64_t key0 = walk.key0(j);
        __syncthreads();
        load_tile<D>(sK, k, s, sb, key0, s.Hkv, kvh, s.kv_elems);
        load_tile<D>(sV, v, s, sb, key0, s.Hkv, kvh, s.kv_elems);
        __syncthreads();
        float x[4][4], y[4][4];
        rows_by_rows<D>(sQ, sK, tx, ty, x);
        rows_by_rows<D>(sO, sV, tx, ty, y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = mask[i].sees(key0 + tx + 16 * c) ? expf(x[i][c] * s.scale - L[i]) : 0.f;
                sP[(tx + 16 * c) * kPitchP + ty + 16 * i] = mask[i].alone() ? 0.f : p * (y[i][c] - Di[i]);
            }
        __syncthreads();
        add_product<D>(sP, sK, tx, ty, acc);
    }
    const float f[4] = {s.scale, s.scale, s.scale, s.scale};
    store_rows<D>(dq, acc, f, s, sb, q0, s.Hq, h, tx, ty, s.q_elems);
}

// One block: dK and dV of 64 keys of one KV head, or its unit's part of them,
// over the query tiles of the unit and the heads of the group.
template <int D>
__device__ __forceinline__ void window_dkv(const AttnShape &s, int64_t block, float *sm, const float *__restrict__ q,
                                           const float *__restrict__ k, const float *__restrict__ v,
                                           const float *__restrict__ lse, const float *__restrict__ dout,
                                           const float *__restrict__ Dv, float *__restrict__ dk,
                                           float *__restrict__ dv)
{
    constexpr int kTile = kT * (D + kPad);
    float *sK = sm, *sV = sm + kTile, *sQ = sm + 2 * kTile, *sO = sm + 3 * kTile, *sP = sm + 4 * kTile,
          *sS = sP + kT * kPitchP;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t prob = block % (s.SB * s.Hkv);
    const int4 unit = window_unit(s.units, s.N, s.window, kT, static_cast<int>(block / (s.SB * s.Hkv)));
    const int kvh = static_cast<int>(prob % s.Hkv), G = s.Hq / s.Hkv;
    const int64_t sb = prob / s.Hkv, k0 = static_cast<int64_t>(unit.x) * kT;
    load_tile<D>(sK, k, s, sb, k0, s.Hkv, kvh, s.kv_elems);
    load_tile<D>(sV, v, s, sb, k0, s.Hkv, kvh, s.kv_elems);
    // rows that see the keys tx + 16 c: [key, end)
    int64_t end[4];
    bool alone[4];  // its own row sees no other key
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int64_t key = k0 + tx + 16 * c;
        end[c] = 0;
        alone[c] = false;
        if (key < s.N) {
            int64_t start;
            doc_bounds(s, key, start, end[c]);
            alone[c] = key == start || (s.window == 1 && s.sinks == 0);
            if (key >= start + s.sinks)
                end[c] = min(end[c], key + s.window);
        }
    }
    float aK[4][D / 16], aV[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            aK[i][c] = aV[i][c] = 0.f;
    for (int it = 0; it < unit.z * G; ++it) {
        const int h = kvh * G + it % G;
        const int64_t q0 = static_cast<int64_t>(unit.y + it / G) * kT;
        __syncthreads();
        load_tile<D>(sQ, q, s, sb, q0, s.Hq, h, s.q_elems);
        load_tile<D>(sO, dout, s, sb, q0, s.Hq, h, s.q_elems);
        float L[4], Di[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t li = (sb * s.Hq + h) * s.N + min(q0 + ty + 16 * i, s.N - 1);
            const bool ok = ULY_IN_BOUNDS(s.status, li, 1, s.lse_elems, 0x69);
            L[i] = ok ? lse[li] : 0.f;
            Di[i] = ok ? Dv[li] : 0.f;
        }
        __syncthreads();
        float x[4][4], y[4][4];
        rows_by_rows<D>(sQ, sK, tx, ty, x);
        rows_by_rows<D>(sO, sV, tx, ty, y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int64_t row = q0 + ty + 16 * i, key = k0 + tx + 16 * c;
                const bool one = alone[c] && row == key;  // P = 1 and dS = 0, whatever the roundings
                const float p = one ? 1.f : row >= key && row < end[c] ? expf(x[i][c] * s.scale - L[i]) : 0.f;
                sP[(ty + 16 * i) * kPitchP + tx + 16 * c] = p;
                sS[(ty + 16 * i) * kPitchP + tx + 16 * c] = one ? 0.f : p * (y[i][c] - Di[i]);
            }
        __syncthreads();
        add_product<D>(sP, sO, tx, ty, aV);
        add_product<D>(sS, sQ, tx, ty, aK);
    }
    // a tile whose walk is cut: the sums of its last document's sinks go to the unit's slot
    int64_t first = 0, past = 0;
    if (unit.w >= 0) {
        int64_t start, hi;
        doc_bounds(s, min(k0 + kT, s.N) - 1, start, hi);
        first = max(start, k0);
        past = min(start + s.sinks, s.N);
    }
    [[maybe_unused]] const int64_t extent = s.SB * s.Hkv * s.units.slots * 2 * s.units.rows * D;
    const int64_t other = static_cast<int64_t>(s.units.rows) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t key = k0 + 4 * ty + i;
        if (key >= s.N)
            continue;
        const bool sums = key >= first && key < past;
        if (!sums && unit.w >= 0 && (unit.w & 1))
            continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int col = 64 * c + 4 * tx;
            const float4 a = make_float4(aK[i][4 * c], aK[i][4 * c + 1], aK[i][4 * c + 2], aK[i][4 * c + 3]);
            const float4 b = make_float4(aV[i][4 * c], aV[i][4 * c + 1], aV[i][4 * c + 2], aV[i][4 * c + 3]);
            if (sums) {
                const int64_t off =
                    ((prob * s.units.slots + (unit.w >> 1)) * 2 * s.units.rows + key - first) * D + col;
                if (ULY_IN_BOUNDS(s.status, off, other + 4, extent, 0x6a)) {
                    *reinterpret_cast<float4 *>(s.units.part + off) = a;
                    *reinterpret_cast<float4 *>(s.units.part + off + other) = b;
                }
            } else {
                const int64_t off = s.L.off(s.N, sb, key, s.Hkv, kvh, D) + col;
                if (ULY_IN_BOUNDS(s.status, off, 4, s.kv_elems, 0x6b)) {
                    *reinterpret_cast<float4 *>(dk + off) =
                        make_float4(a.x * s.scale, a.y * s.scale, a.z * s.scale, a.w * s.scale);
                    *reinterpret_cast<float4 *>(dv + off) = b;
                }
            }
        }
    }
}

// The blocks of dK and dV, whose walks are the longer ones, then those of dQ: a short
// sequence has too few of either to fill the GPU (509 tokens of 2 x 4 heads of 64: 76 us,
// 109 in two launches).  Heads of 64 let two blocks share an SM, for which their
// registers have to spill a little: 3.6 ms against 4.1 at 8192 tokens under a window of
// 1024, but 86 us at 509 tokens, so that grids of one block an SM keep theirs.
template <int D, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) window_bwd_f32_kernel(const __grid_constant__ AttnShape s,
                                                                  int64_t dkv_blocks, const float *__restrict__ q,
                                                                  const float *__restrict__ k,
                                                                  const float *__restrict__ v,
                                                                  const float *__restrict__ lse,
                                                                  const float *__restrict__ dout,
                                                                  const float *__restrict__ Dv, float *__restrict__ dq,
                                                                  float *__restrict__ dk, float *__restrict__ dv)
{
    extern __shared__ __align__(16) float sm[];
    if (blockIdx.x < dkv_blocks)
        window_dkv<D>(s, blockIdx.x, sm, q, k, v, lse, dout, Dv, dk, dv);
    else
        window_dq<D>(s, blockIdx.x - dkv_blocks, sm, q, k, v, lse, dout, Dv, dq);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t grid, size_t smem, cudaStream_t st, Args... args)
{
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess)
        return e;
    kernel<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(args...);
    return cudaGetLastError();
}

constexpr size_t kPBytes = sizeof(float) * kT * kPitchP;

template <int D>
cudaError_t fwd(const AttnShape &s, const float *q, const float *k, const float *v, float *o, float *lse,
                cudaStream_t st)
{
    const int64_t tiles = (s.N + kT - 1) / kT;
    return launch(window_fwd_f32_kernel<D>, tiles * s.Hq * s.SB, 3 * tile_bytes<D>() + kPBytes + kT * sizeof(float), st,
                  s, q, k, v, o, lse);
}

template <int D>
cudaError_t bwd(const AttnShape &s, const float *q, const float *k, const float *v, const float *o, const float *lse,
                const float *dout, float *dq, float *dk, float *dv, float *Dv, cudaStream_t st)
{
    const int64_t tiles = (s.N + kT - 1) / kT, rows = s.SB * s.Hq * s.N;
    cudaError_t e = launch(window_pre_f32_kernel<D>, (rows * 32 + kThreads - 1) / kThreads, 0, st, s, o, dout, Dv);
    const int64_t dkv = s.units.n_units * s.SB * s.Hkv, blocks = dkv + tiles * s.Hq * s.SB;
    if (e == cudaSuccess)
        e = launch(blocks <= num_sms() ? window_bwd_f32_kernel<D, 1> : window_bwd_f32_kernel<D, D == 64 ? 2 : 1>, blocks,
                   4 * tile_bytes<D>() + 2 * kPBytes, st, s, dkv, q, k, v, lse, dout,
                   static_cast<const float *>(Dv), dq, dk, dv);
    return e;
}

}  // namespace

cudaError_t launch_window_fwd_f32(const AttnShape &s, const float *q, const float *k, const float *v, float *o,
                                  float *lse, cudaStream_t stream)
{
    return s.d == 64 ? fwd<64>(s, q, k, v, o, lse, stream) : fwd<128>(s, q, k, v, o, lse, stream);
}

cudaError_t launch_window_bwd_f32(const AttnShape &s, const float *q, const float *k, const float *v, const float *o,
                                  const float *lse, const float *dout, float *dq, float *dk, float *dv, float *ws_D,
                                  cudaStream_t stream)
{
    return s.d == 64 ? bwd<64>(s, q, k, v, o, lse, dout, dq, dk, dv, ws_D, stream)
                     : bwd<128>(s, q, k, v, o, lse, dout, dq, dk, dv, ws_D, stream);
}

}  // namespace uly
