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
// Memory-bound: every value is read and written once.  A warp takes one
// token's rows, so that its cosines and sines are made once and shared by its
// heads; a lane holds the two chunks of a row (8 bytes each) whose values turn
// with each other, so that the rotation needs no exchange between lanes; the
// next kUnroll rows are loaded before the first is used.
#include <cmath>

#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;

// A row of kD values over kLanes lanes: two chunks of kC values each, as kP
// pairs for the packed fp32 arithmetic.
template <typename T, int kD_>
struct Shape {
    static constexpr int kD = kD_;
    static constexpr int kC = 8 / sizeof(T);
    static constexpr int kP = kC / 2;
    static constexpr int kLanes = kD / (2 * kC);
    static constexpr int kRows = 32 / kLanes;  // rows a warp takes at once
};

template <typename T>
__device__ __forceinline__ void unpack(const uint2 &u, float2 *x)
{
    if constexpr (sizeof(T) == 2) {
        x[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
        x[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    } else {
        x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    }
}

template <typename T>
__device__ __forceinline__ uint2 pack(const float2 *x)
{
    if constexpr (sizeof(T) == 2)
        return make_uint2(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y));
    else
        return make_uint2(__float_as_uint(x[0].x), __float_as_uint(x[0].y));
}

__device__ __forceinline__ float2 swap(float2 v) { return make_float2(v.y, v.x); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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

// Heads of one tensor on the far side: the head layout [P][B][N][H/P][d] or
// the sequence layout, contiguous.  h / (H/P) by a product: exact below 65536.
struct Far {
    int64_t first, rank;  // this token's offset in rank 0, and between ranks (elements)
    unsigned magic;
    int per;

    __device__ __forceinline__ Far(const NormRopeParams &p, const Token &k, int H, int Hp, unsigned magic_, int d)
        : magic(magic_), per(Hp)
    {
        if (p.to_head) {
            first = (k.b * p.N + k.n) * Hp * d;
            rank = p.N * p.B * Hp * d;
        } else {
            first = k.m * H * d;
            rank = 0;
        }
    }
    __device__ __forceinline__ int64_t at(int h, int d) const
    {
        const int r = magic ? static_cast<int>(__umulhi(static_cast<unsigned>(h), magic)) : h;
        return first + r * rank + static_cast<int64_t>(h - r * per) * d;
    }
};

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

// Where a lane's chunks lie.  Half-split pairs: lanes below half / kC hold
// values f.. and half + f.. that turn with each other, the others two chunks
// of the part that does not turn.  Interleaved pairs: neighbouring chunks.
template <typename S, bool kInter>
__device__ __forceinline__ void chunk_places(int half, int i, int &lo, int &hi)
{
    if (kInter) {
        lo = 2 * i * S::kC;
        hi = lo + S::kC;
    } else if (i * S::kC < half) {
        lo = i * S::kC;
        hi = half + lo;
    } else {
        lo = half + i * S::kC;
        hi = lo + (S::kD - 2 * half) / 2;
    }
}

// The rotation of a lane's chunks: lo' = lo c_lo + o s_lo, hi' = hi c_hi + o s_hi,
// where o is the other chunk (half-split) or the chunk with its pairs swapped
// (interleaved).  kBack: its transpose.
template <typename S, bool kInter, bool kBack>
struct Turn {
    float2 cl[S::kP], sl[S::kP], ch[S::kP], sh[S::kP];
    bool turns;  // both chunks do or neither (rot is a multiple of 16): an infinity must not meet a zero sine

    __device__ __forceinline__ Turn(const float2 *table, int half, int lo, int hi)
    {
        const float sign = kBack ? -1.f : 1.f;
        turns = kInter ? lo < 2 * half : lo < half;
#pragma unroll
        for (int j = 0; j < S::kP; ++j) {
            cl[j] = ch[j] = both(1.f);
            sl[j] = sh[j] = both(0.f);
            if (!turns)
                continue;
            if (kInter) {
                const float2 t = table[lo / 2 + j], u = table[hi / 2 + j];
                cl[j] = both(t.x);
                ch[j] = both(u.x);
                sl[j] = make_float2(-sign * t.y, sign * t.y);
                sh[j] = make_float2(-sign * u.y, sign * u.y);
            } else {
                const float2 t = table[lo + 2 * j], u = table[lo + 2 * j + 1];
                cl[j] = ch[j] = make_float2(t.x, u.x);
                sl[j] = make_float2(-sign * t.y, -sign * u.y);
                sh[j] = make_float2(sign * t.y, sign * u.y);
            }
        }
    }
    // the rotation of w * x as one of x (the norm's weight taken in)
    __device__ __forceinline__ void weigh(const float2 *wl, const float2 *wh)
    {
#pragma unroll
        for (int j = 0; j < S::kP; ++j) {
            cl[j] = fmul2(cl[j], wl[j]);
            ch[j] = fmul2(ch[j], wh[j]);
            sl[j] = fmul2(sl[j], kInter ? swap(wl[j]) : wh[j]);
            sh[j] = fmul2(sh[j], kInter ? swap(wh[j]) : wl[j]);
        }
    }
    __device__ __forceinline__ void apply(float2 *lo, float2 *hi) const
    {
#pragma unroll
        for (int j = 0; j < S::kP; ++j) {
            const float2 a = lo[j], b = hi[j];
            lo[j] = fmul2(a, cl[j]);
            hi[j] = fmul2(b, ch[j]);
            if (turns) {
                lo[j] = ffma2(kInter ? swap(a) : b, sl[j], lo[j]);
                hi[j] = ffma2(kInter ? swap(b) : a, sh[j], hi[j]);
            }
        }
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

template <typename T, typename S>
__device__ __forceinline__ void load_weights(const void *w, int lo, int hi, float2 *wl, float2 *wh)
{
    unpack<T>(*reinterpret_cast<const uint2 *>(static_cast<const T *>(w) + lo), wl);
    unpack<T>(*reinterpret_cast<const uint2 *>(static_cast<const T *>(w) + hi), wh);
}

struct Raw {
    uint2 lo, hi;
};

template <typename T>
__device__ __forceinline__ Raw load_row(const T *row, int lo, int hi)
{
    return Raw{*reinterpret_cast<const uint2 *>(row + lo), *reinterpret_cast<const uint2 *>(row + hi)};
}

template <typename T>
__device__ __forceinline__ void store_row(T *row, int lo, int hi, const Raw &v)
{
    *reinterpret_cast<uint2 *>(row + lo) = v.lo;
    *reinterpret_cast<uint2 *>(row + hi) = v.hi;
}

// A unit is one token and a run [r0, r1) of its rows: Q's heads, K's, V's.
struct Run {
    int q0, q1, k0, k1, v0, v1;

    __device__ __forceinline__ Run(const NormRopeParams &p, int part)
    {
        const int r0 = part * p.rows_per_split, r1 = r0 + p.rows_per_split, kv = p.Hq + p.Hkv;
        q0 = min(r0, p.Hq), q1 = min(r1, p.Hq);
        k0 = max(r0 - p.Hq, 0), k1 = min(r1 - p.Hq, p.Hkv);
        v0 = max(r0 - kv, 0), v1 = p.v ? min(r1 - kv, p.Hkv) : 0;
    }
};

// heads [h0, h1): load kUnroll of this lane's rows, then hand them on
template <typename S, typename Load, typename Use>
__device__ __forceinline__ void for_heads(int h0, int h1, int sub, Load load, Use use)
{
    using R = decltype(load(0));
    for (int hb = h0; hb < h1; hb += kUnroll * S::kRows) {
        R raw[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = hb + i * S::kRows + sub;
            raw[i] = load(h < h1 ? h : h0);  // past the end: a row that is there
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (hb + i * S::kRows < h1) {
                const int h = hb + i * S::kRows + sub;
                use(h, h < h1, raw[i]);
            }
    }
}

template <typename T, int kD, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p)
{
    using S = Shape<T, kD>;
    __shared__ float2 table[kWarps][kD / 2];
    const int warp = warp_id(), lane = lane_id(), sub = lane / S::kLanes;
    int lo, hi;
    chunk_places<S, kInter>(p.half, lane % S::kLanes, lo, hi);
    const int64_t units = p.tokens * p.splits;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const Token k = token_of(p, static_cast<uint32_t>(u / p.splits));
        const Run run(p, static_cast<int>(u % p.splits));
        if (run.v0 == 0)
            angles(p, k, table[warp], lane);
        auto heads = [&](int h0, int h1, const void *in, int64_t stride, void *out, int H, int Hp, unsigned magic,
                         const void *w) {
            if (h0 >= h1)
                return;
            Turn<S, kInter, false> turn(table[warp], p.half, lo, hi);
            if (kNorm) {
                float2 wl[S::kP], wh[S::kP];
                load_weights<T, S>(w, lo, hi, wl, wh);
                turn.weigh(wl, wh);
            }
            const T *src = static_cast<const T *>(in) + k.m * stride;
            const Far far(p, k, H, Hp, magic, kD);
            for_heads<S>(
                h0, h1, sub, [&](int h) { return load_row<T>(src + static_cast<int64_t>(h) * kD, lo, hi); },
                [&](int h, bool live, const Raw &raw) {
                    float2 a[S::kP], b[S::kP];
                    unpack<T>(raw.lo, a);
                    unpack<T>(raw.hi, b);
                    float rstd = 1.f;
                    if (kNorm) {
                        float2 ss = both(0.f);
#pragma unroll
                        for (int j = 0; j < S::kP; ++j)
                            ss = ffma2(b[j], b[j], ffma2(a[j], a[j], ss));
                        rstd = rsqrtf(row_sum<S::kLanes>(ss.x + ss.y) * (1.f / kD) + p.eps);
                    }
                    turn.apply(a, b);
                    if (kNorm) {
#pragma unroll
                        for (int j = 0; j < S::kP; ++j) {
                            a[j] = fmul2(a[j], both(rstd));
                            b[j] = fmul2(b[j], both(rstd));
                        }
                    }
                    if (live)
                        store_row<T>(static_cast<T *>(out) + far.at(h, kD), lo, hi, Raw{pack<T>(a), pack<T>(b)});
                });
        };
        heads(run.q0, run.q1, p.q, p.qs, p.qo, p.Hq, p.Hqp, p.magic_q, p.wq);
        heads(run.k0, run.k1, p.k, p.ks, p.ko, p.Hkv, p.Hkvp, p.magic_k, p.wk);
        if (run.v0 < run.v1) {
            const T *src = static_cast<const T *>(p.v) + k.m * p.vs;
            const Far far(p, k, p.Hkv, p.Hkvp, p.magic_k, kD);
            for_heads<S>(
                run.v0, run.v1, sub, [&](int h) { return load_row<T>(src + static_cast<int64_t>(h) * kD, lo, hi); },
                [&](int h, bool live, const Raw &raw) {
                    if (live)
                        store_row<T>(static_cast<T *>(p.vo) + far.at(h, kD), lo, hi, raw);
                });
        }
    }
}

template <typename T, int kD, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p)
{
    using S = Shape<T, kD>;
    __shared__ float2 table[kWarps][kD / 2];
    const int warp = warp_id(), lane = lane_id(), sub = lane / S::kLanes;
    int lo, hi;
    chunk_places<S, kInter>(p.half, lane % S::kLanes, lo, hi);
    // this lane's part of dw: [q, k][lo, hi]
    float2 dw[2][2][S::kP];
#pragma unroll
    for (int j = 0; j < S::kP; ++j)
        dw[0][0][j] = dw[0][1][j] = dw[1][0][j] = dw[1][1][j] = both(0.f);
    const int64_t units = p.tokens * p.splits;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const Token k = token_of(p, static_cast<uint32_t>(u / p.splits));
        const Run run(p, static_cast<int>(u % p.splits));
        if (run.v0 == 0)
            angles(p, k, table[warp], lane);
        auto heads = [&](int h0, int h1, const void *in, int64_t stride, const void *dy, void *dx, int64_t dstride,
                         int H, int Hp, unsigned magic, const void *w, float2 (&sum)[2][S::kP]) {
            if (h0 >= h1)
                return;
            const Turn<S, kInter, true> turn(table[warp], p.half, lo, hi);
            float2 wl[S::kP], wh[S::kP];
            if (kNorm)
                load_weights<T, S>(w, lo, hi, wl, wh);
            const T *src = static_cast<const T *>(in) + (kNorm ? k.m * stride : 0);
            T *dst = static_cast<T *>(dx) + k.m * dstride;
            const Far far(p, k, H, Hp, magic, kD);
            struct Two {
                Raw dy, x;
            };
            for_heads<S>(
                h0, h1, sub,
                [&](int h) {
                    Two t;
                    t.dy = load_row<T>(static_cast<const T *>(dy) + far.at(h, kD), lo, hi);
                    if (kNorm)
                        t.x = load_row<T>(src + static_cast<int64_t>(h) * kD, lo, hi);
                    return t;
                },
                [&](int h, bool live, const Two &raw) {
                    float2 g[2][S::kP];
                    unpack<T>(raw.dy.lo, g[0]);
                    unpack<T>(raw.dy.hi, g[1]);
                    turn.apply(g[0], g[1]);
                    if (kNorm) {
                        float2 x[2][S::kP], ss = both(0.f), dot = both(0.f), gx[2][S::kP];
                        unpack<T>(raw.x.lo, x[0]);
                        unpack<T>(raw.x.hi, x[1]);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int j = 0; j < S::kP; ++j) {
                                const float2 w2 = c ? wh[j] : wl[j];
                                ss = ffma2(x[c][j], x[c][j], ss);
                                gx[c][j] = fmul2(g[c][j], x[c][j]);
                                dot = ffma2(w2, gx[c][j], dot);
                                g[c][j] = fmul2(w2, g[c][j]);
                            }
                        const float rstd = rsqrtf(row_sum<S::kLanes>(ss.x + ss.y) * (1.f / kD) + p.eps);
                        // mean(w g xhat) r: what x loses, before the last factor r
                        const float m = row_sum<S::kLanes>(dot.x + dot.y) * (1.f / kD) * rstd * rstd;
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int j = 0; j < S::kP; ++j) {
                                if (live)
                                    sum[c][j] = ffma2(gx[c][j], both(rstd), sum[c][j]);
                                g[c][j] = fmul2(ffma2(x[c][j], both(-m), g[c][j]), both(rstd));
                            }
                    }
                    if (live)
                        store_row<T>(dst + static_cast<int64_t>(h) * kD, lo, hi, Raw{pack<T>(g[0]), pack<T>(g[1])});
                });
        };
        heads(run.q0, run.q1, p.q, p.qs, p.qo, p.dq, p.dqs, p.Hq, p.Hqp, p.magic_q, p.wq, dw[0]);
        heads(run.k0, run.k1, p.k, p.ks, p.ko, p.dk, p.dks, p.Hkv, p.Hkvp, p.magic_k, p.wk, dw[1]);
        if (run.v0 < run.v1) {
            T *dst = static_cast<T *>(p.dv) + k.m * p.dvs;
            const Far far(p, k, p.Hkv, p.Hkvp, p.magic_k, kD);
            for_heads<S>(
                run.v0, run.v1, sub,
                [&](int h) { return load_row<T>(static_cast<const T *>(p.vo) + far.at(h, kD), lo, hi); },
                [&](int h, bool live, const Raw &raw) {
                    if (live)
                        store_row<T>(dst + static_cast<int64_t>(h) * kD, lo, hi, raw);
                });
        }
    }
    if constexpr (kNorm) {
        // the block's weight-gradient partial: row slots within the warp, then the
        // warps, always in the same order
        __shared__ float sums[kWarps][2][kD];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < S::kP; ++j) {
                    float2 v = dw[t][c][j];
#pragma unroll
                    for (int o = S::kLanes; o < 32; o <<= 1) {
                        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
                        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
                    }
                    if (sub == 0)
                        *reinterpret_cast<float2 *>(&sums[warp][t][(c ? hi : lo) + 2 * j]) = v;
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
    constexpr int kRows = Shape<T, kD>::kRows;
    const int rows = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    // few tokens: a token's rows go to several warps
    const int64_t want = static_cast<int64_t>(num_sms()) * 16;
    int splits = static_cast<int>(std::min<int64_t>((rows + kRows - 1) / kRows, (want + p.tokens - 1) / p.tokens));
    p.rows_per_split = ((rows + splits - 1) / splits + kRows - 1) / kRows * kRows;
    p.splits = (rows + p.rows_per_split - 1) / p.rows_per_split;
    p.magic_q = p.Hqp == 1 ? 0u : 0xffffffffu / p.Hqp + 1;
    p.magic_k = p.Hkvp == 1 ? 0u : 0xffffffffu / p.Hkvp + 1;
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
