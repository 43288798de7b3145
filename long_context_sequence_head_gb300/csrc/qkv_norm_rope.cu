// RMS norm of every query and key head, rotary position embedding and the
// seq->head move of Q, K and V in one pass over the projection's output, and
// its backward.  For a head row x (d values), its weight w and its token's
// positions p_a on the axes a:
//   r    = 1 / sqrt(mean(x^2) + eps)          xhat = x r
//   y    = R(p) (w * xhat)                    R: a rotation of each pair of values
//   pair f (values f and f + rot/2, or 2f and 2f + 1):
//     (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = p_axis(f) * inv_freq(f)
// Backward, with g = R(p)^T dy (the rotation by -t):
//   dw   = sum over rows of g * xhat
//   dx   = r (w * g - xhat mean(w * g * xhat))
// Everything between the load and the store is fp32 and rounded once.
//
// Angles.  t / 2 pi is wanted modulo one turn.  inv_freq / 2 pi, reduced to
// [0, 1), is held as a 64-bit fraction F; F * p modulo 2^64 (one 64-bit
// integer product that wraps) is then the turn's fraction, exact up to
// p * 2^-53 of a turn (the rounding of inv_freq / 2 pi itself), for negative
// positions too.  A product in fp32 would be off by 0.06 rad at a million.
//
// Memory-bound: reads and writes every value once; a warp takes one token's
// rows, 16 bytes a lane, so that the cosines and sines of the token are made
// once and shared by its heads.
#include <cmath>

#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &u, float (&x)[Vec<T>::kN])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            x[k] = __uint_as_float(w[k]);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[Vec<T>::kN])
{
    if constexpr (sizeof(T) == 2)
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    else
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

struct Token {
    int64_t m;  // row of the sequence layout: ((s * B + b) * Np + t)
    int64_t n;  // index in its sequence
    int b;
};

__device__ __forceinline__ Token token_of(const NormRopeParams &p, uint32_t m)
{
    const uint32_t sb = m / static_cast<uint32_t>(p.Np), t = m - sb * static_cast<uint32_t>(p.Np);
    const uint32_t s = sb / static_cast<uint32_t>(p.B);
    return Token{m, static_cast<int64_t>(s) * p.Np + t, static_cast<int>(sb - s * p.B)};
}

// Offset (elements) of head h of a tensor of H heads in the far layout: the
// head layout [P][B][N][H/P][d] or the sequence layout, contiguous.
__device__ __forceinline__ int64_t far_off(const NormRopeParams &p, const Token &k, int H, int Hp, int h, int d)
{
    if (!p.to_head)
        return (k.m * H + h) * d;
    const int r = h / Hp;
    return (((static_cast<int64_t>(r) * p.B + k.b) * p.N + k.n) * Hp + (h - r * Hp)) * d;
}

// cos and sin of the token's rot/2 angles into the warp's shared table
__device__ __forceinline__ void angles(const NormRopeParams &p, const Token &k, float2 *table, int lane)
{
    __syncwarp();  // the last token's reads are done
    for (int f = lane; f < p.half; f += 32) {
        const int64_t pos = p.positions ? p.positions[p.axis[f] * p.tokens + k.m] : k.n;
        const uint64_t frac = p.turn[f] * static_cast<uint64_t>(pos);
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int64_t>(frac)) * 0x1p-63f, &sn, &cs);  // in (-1, 1] half turns
        table[f] = make_float2(cs, sn);
    }
    __syncwarp();
}

// This lane's part of the rotation: values e0 .. e0 + n-1 of the row.
// y_j = x_j * c_j + partner_j * s_j; for the half-split pairs the partner is
// the same place of another lane, for the interleaved pairs the neighbour.
template <typename T, bool kInter>
struct Rot {
    static constexpr int kN = Vec<T>::kN;
    float c[kN], s[kN];
    int partner;  // lane holding the partner values (this lane: none)

    __device__ __forceinline__ void load(const NormRopeParams &p, const float2 *table, int e0, int lane)
    {
        partner = lane;
#pragma unroll
        for (int j = 0; j < kN; ++j)
            c[j] = 1.f, s[j] = 0.f;
        if (e0 >= 2 * p.half)
            return;
        if (kInter) {
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float2 v = table[(e0 + j) >> 1];
                c[j] = v.x;
                s[j] = (j & 1) ? v.y : -v.y;
            }
        } else {
            const bool low = e0 < p.half;
            partner = low ? lane + p.half / kN : lane - p.half / kN;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float2 v = table[(low ? e0 : e0 - p.half) + j];
                c[j] = v.x;
                s[j] = low ? -v.y : v.y;
            }
        }
    }
    // kBack: the transpose (rotation by the negative angle)
    template <bool kBack>
    __device__ __forceinline__ void apply(float (&x)[kN]) const
    {
        float o[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j)
            o[j] = kInter ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner);
#pragma unroll
        for (int j = 0; j < kN; ++j)
            x[j] = fmaf(x[j], c[j], kBack ? -o[j] * s[j] : o[j] * s[j]);
    }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, int kD, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int kN = Vec<T>::kN, kLanes = kD / kN, kRows = 32 / kLanes;
    __shared__ float2 table[kWarps][kD / 2];
    const int warp = warp_id(), lane = lane_id();
    const int e0 = (lane % kLanes) * kN, sub = lane / kLanes;
    float wq[kN], wk[kN];
    if (kNorm) {
        unpack<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(p.wq) + e0), wq);
        unpack<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(p.wk) + e0), wk);
    }
    const int rows = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    const int64_t units = p.tokens * p.splits;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const Token k = token_of(p, static_cast<uint32_t>(u / p.splits));
        const int part = static_cast<int>(u % p.splits);
        const int r0 = part * p.rows_per_split, r1 = min(rows, r0 + p.rows_per_split);
        Rot<T, kInter> rot;
        if (r0 < p.Hq + p.Hkv)
            angles(p, k, table[warp], lane);
        rot.load(p, table[warp], e0, lane);
        for (int rb = r0; rb < r1; rb += kRows) {
            const int r = rb + sub;
            const bool live = r < r1;
            const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
            const int h = is_q ? r : (is_v ? r - p.Hq - p.Hkv : r - p.Hq);
            const T *src = static_cast<const T *>(is_q ? p.q : (is_v ? p.v : p.k)) +
                           k.m * (is_q ? p.qs : (is_v ? p.vs : p.ks)) + static_cast<int64_t>(h) * kD + e0;
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (live)
                raw = *reinterpret_cast<const uint4 *>(src);
            float x[kN];
            unpack<T>(raw, x);
            if (kNorm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    ss = fmaf(x[j], x[j], ss);
                const float rstd = 1.f / sqrtf(row_sum<kLanes>(ss) * (1.f / kD) + p.eps);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    x[j] *= rstd * (is_q ? wq[j] : wk[j]);
            }
            rot.template apply<false>(x);
            if (live) {
                T *dst = static_cast<T *>(is_q ? p.qo : (is_v ? p.vo : p.ko)) +
                         far_off(p, k, is_q ? p.Hq : p.Hkv, is_q ? p.Hqp : p.Hkvp, h, kD) + e0;
                *reinterpret_cast<uint4 *>(dst) = is_v ? raw : pack<T>(x);
            }
        }
    }
}

template <typename T, int kD, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int kN = Vec<T>::kN, kLanes = kD / kN, kRows = 32 / kLanes;
    __shared__ float2 table[kWarps][kD / 2];
    __shared__ float sums[kWarps][2][kD];
    const int warp = warp_id(), lane = lane_id();
    const int e0 = (lane % kLanes) * kN, sub = lane / kLanes;
    float wq[kN], wk[kN], aq[kN], ak[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j)
        aq[j] = ak[j] = 0.f;
    if (kNorm) {
        unpack<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(p.wq) + e0), wq);
        unpack<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(p.wk) + e0), wk);
    }
    const int rows = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    const int64_t units = p.tokens * p.splits;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const Token k = token_of(p, static_cast<uint32_t>(u / p.splits));
        const int part = static_cast<int>(u % p.splits);
        const int r0 = part * p.rows_per_split, r1 = min(rows, r0 + p.rows_per_split);
        Rot<T, kInter> rot;
        if (r0 < p.Hq + p.Hkv)
            angles(p, k, table[warp], lane);
        rot.load(p, table[warp], e0, lane);
        for (int rb = r0; rb < r1; rb += kRows) {
            const int r = rb + sub;
            const bool live = r < r1;
            const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
            const int h = is_q ? r : (is_v ? r - p.Hq - p.Hkv : r - p.Hq);
            const T *dy = static_cast<const T *>(is_q ? p.qo : (is_v ? p.vo : p.ko)) +
                          far_off(p, k, is_q ? p.Hq : p.Hkv, is_q ? p.Hqp : p.Hkvp, h, kD) + e0;
            uint4 raw = make_uint4(0, 0, 0, 0), rawx = raw;
            if (live) {
                raw = *reinterpret_cast<const uint4 *>(dy);
                if (kNorm && !is_v)
                    rawx = *reinterpret_cast<const uint4 *>(static_cast<const T *>(is_q ? p.q : p.k) +
                                                            k.m * (is_q ? p.qs : p.ks) +
                                                            static_cast<int64_t>(h) * kD + e0);
            }
            float g[kN];
            unpack<T>(raw, g);
            rot.template apply<true>(g);
            if (kNorm) {
                float x[kN];
                unpack<T>(rawx, x);
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    ss = fmaf(x[j], x[j], ss);
                const float rstd = 1.f / sqrtf(row_sum<kLanes>(ss) * (1.f / kD) + p.eps);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    x[j] *= rstd;
                    const float gx = g[j] * x[j];
                    if (live && is_q)
                        aq[j] += gx;
                    else if (live && !is_v)
                        ak[j] += gx;
                    const float w = is_q ? wq[j] : wk[j];
                    dot = fmaf(w, gx, dot);
                    g[j] *= w;
                }
                dot = row_sum<kLanes>(dot) * (1.f / kD);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    g[j] = rstd * fmaf(-x[j], dot, g[j]);
            }
            if (live) {
                T *dst = static_cast<T *>(is_q ? p.dq : (is_v ? p.dv : p.dk)) +
                         k.m * (is_q ? p.dqs : (is_v ? p.dvs : p.dks)) + static_cast<int64_t>(h) * kD + e0;
                *reinterpret_cast<uint4 *>(dst) = is_v ? raw : pack<T>(g);
            }
        }
    }
    if constexpr (kNorm) {
        // the block's weight-gradient partial: row slots within the warp, then the
        // warps, always in the same order
#pragma unroll
        for (int j = 0; j < kN; ++j) {
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1) {
                aq[j] += __shfl_xor_sync(0xffffffffu, aq[j], o);
                ak[j] += __shfl_xor_sync(0xffffffffu, ak[j], o);
            }
            if (sub == 0) {
                sums[warp][0][e0 + j] = aq[j];
                sums[warp][1][e0 + j] = ak[j];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kD; i += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                s += sums[w][i / kD][i % kD];
            p.partial[static_cast<int64_t>(blockIdx.x) * 2 * kD + i] = s;
        }
    }
}

// dw[i] = sum over the blocks' partials, in block order within each of 32
// strided runs and then over the runs: the same order on every launch.
template <typename T>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float *__restrict__ partial, int blocks, int d,
                                                            T *__restrict__ dwq, T *__restrict__ dwk)
{
    __shared__ float run[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    for (int b = threadIdx.y; b < blocks; b += 32)
        s += partial[static_cast<int64_t>(b) * 2 * d + col];
    run[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0)
        return;
    s = 0.f;
    for (int k = 0; k < 32; ++k)
        s += run[k][threadIdx.x];
    T *dw = col < d ? dwq : dwk;
    if (dw == nullptr)
        return;
    if constexpr (sizeof(T) == 2)
        dw[col % d] = static_cast<T>(pack_bf16x2(s, 0.f) & 0xffffu);
    else
        dw[col % d] = s;
}

template <typename T, int kD, bool kInter, bool kNorm>
cudaError_t run(NormRopeParams &p, bool bwd, cudaStream_t s)
{
    constexpr int kRows = 32 / (kD / Vec<T>::kN);
    const int rows = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    // few tokens: a token's rows go to several warps
    const int64_t want = static_cast<int64_t>(num_sms()) * 16;
    int splits = static_cast<int>(std::min<int64_t>((rows + kRows - 1) / kRows, (want + p.tokens - 1) / p.tokens));
    p.rows_per_split = ((rows + splits - 1) / splits + kRows - 1) / kRows * kRows;
    p.splits = (rows + p.rows_per_split - 1) / p.rows_per_split;
    const int64_t need = (p.tokens * p.splits + kWarps - 1) / kWarps;
    int64_t grid = std::min<int64_t>(need, static_cast<int64_t>(num_sms()) * 8);
    if (!bwd) {
        norm_rope_fwd_kernel<T, kD, kInter, kNorm><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    grid = std::min<int64_t>(grid, kNormRopeMaxBlocks);
    norm_rope_bwd_kernel<T, kD, kInter, kNorm><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    if (kNorm && (p.dwq || p.dwk))
        norm_rope_dw_kernel<T><<<2 * kD / 32, dim3(32, 32), 0, s>>>(p.partial, static_cast<int>(grid), kD,
                                                                    static_cast<T *>(p.dwq), static_cast<T *>(p.dwk));
    return cudaGetLastError();
}

template <typename T, int kD>
cudaError_t run_d(NormRopeParams &p, bool inter, bool bwd, cudaStream_t s)
{
    const bool norm = p.wq != nullptr;
    if (inter)
        return norm ? run<T, kD, true, true>(p, bwd, s) : run<T, kD, true, false>(p, bwd, s);
    return norm ? run<T, kD, false, true>(p, bwd, s) : run<T, kD, false, false>(p, bwd, s);
}

}  // namespace

uint64_t turn_fraction(double inv_freq)
{
    double t = inv_freq * 0.15915494309189533577;  // turns per position
    t -= std::floor(t);
    const double f = std::ldexp(t, 64);
    return f >= 18446744073709551616.0 ? 0ull : static_cast<uint64_t>(f);
}

cudaError_t launch_norm_rope(NormRopeParams &p, int d, bool inter, bool bwd, int esize, cudaStream_t s)
{
    if (esize == 2)
        return d == 64 ? run_d<uint16_t, 64>(p, inter, bwd, s) : run_d<uint16_t, 128>(p, inter, bwd, s);
    return d == 64 ? run_d<float, 64>(p, inter, bwd, s) : run_d<float, 128>(p, inter, bwd, s);
}

}  // namespace uly
