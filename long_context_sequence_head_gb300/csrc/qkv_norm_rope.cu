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
// [0, 1), is held as a 64-bit fraction F; F * p modulo 2^64 (one 64-bit integer
// product that wraps) is then the turn's fraction, exact up to |p| times F's own
// error, 2^-62 and 2^-106 of inv_freq, for negative positions too.  A product in fp32
// would be off by 0.06 rad at a million.  The upper 32 bits go to the sine in fp32,
// which rounds them by up to 2^-26 of a turn.
//
// Memory-bound: every value is read and written once.  A warp takes one
// token's rows, so that its cosines and sines are made once and shared by its
// heads; a lane holds the two chunks of a row (8 bytes each) whose values turn
// with each other, so that the rotation needs no exchange between lanes.  Rows
// come in runs, by bulk copies into shared memory that each warp keeps for
// itself: what is in flight costs no registers, and while a warp works on its
// run those of the SM's other warps are on their way.
#include <cmath>

#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Rows of a run (bytes) and resident blocks per SM; a warp has one run on its way.
// Where little is computed per byte (fp32, or no norm) fewer runs on their way are
// better, or reads and writes get into each other's way.  us with the caches emptied
// before each call, bf16: 64K tokens, 32 + 8 + 8 heads of 128; fp32: 32K tokens, 16 +
// 4 + 4.
//   forward, normed   249 (6 KB x 5 blocks), 259 (6 KB x 6), 261 (4 KB x 5), 264 (6
//                     KB x 4), 286 (4 KB x 4), 257 (two runs a warp, 4 KB x 4, which
//                     take 42 us at 8K tokens instead of 44)
//   not normed        249 (4 KB x 4), 256 (4 KB x 5), 268 (6 KB x 5)
//   fp32              132 (4 KB x 4), 131 (4 KB x 5), 138 (6 KB x 5)
//   backward, normed  359 (4 KB x 5), 364 (x 4), over 430 with 2 KB or spills
//   not normed        246 (4 KB x 4), 258 (x 5), 274 (x 3)
//   fp32              180 (4 KB x 4), 190 (x 5), 195 (x 3)
template <typename T, bool kNorm>
constexpr bool kLight = sizeof(T) == 4 || !kNorm;
template <typename T, bool kNorm>
struct Fwd {
    static constexpr int kRun = kLight<T, kNorm> ? 4096 : 6144;
    static constexpr int kBlocks = kLight<T, kNorm> ? 4 : 5;
};
template <typename T, bool kNorm>
struct Bwd {
    static constexpr int kRun = 4096;
    static constexpr int kBlocks = kLight<T, kNorm> ? 4 : 5;
};

// A row of kD values over kLanes lanes: two chunks of kC values each, as kP
// pairs for the packed fp32 arithmetic.
template <typename T, int kD_, int kRunBytes_>
struct Shape {
    static constexpr int kRunBytes = kRunBytes_;
    static constexpr int kD = kD_;
    static constexpr int kC = 8 / sizeof(T);
    static constexpr int kP = kC / 2;
    static constexpr int kLanes = kD / (2 * kC);
    static constexpr int kRows = 32 / kLanes;  // rows a warp takes at once
    static constexpr int kRun = kRunBytes / (kD * sizeof(T));  // rows of a run
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
    uint32_t m;  // row of the sequence layout: ((s * B + b) * Np + t)
    uint32_t n;  // index in its sequence
    int b;
};

// Heads of one tensor on the far side: the head layout [P][B][N][H/P][d] or
// the sequence layout, contiguous.  h / (H/P) by a product: exact below 65536.
struct Far {
    int64_t first, rank;  // this token's offset in rank 0, and between ranks (elements)
    unsigned magic;
    int per;

    __device__ __forceinline__ Far() {}
    __device__ __forceinline__ Far(const NormRopeParams &p, const Token &k, int H, int Hp, unsigned magic_, int d)
        : magic(magic_), per(Hp)
    {
        if (p.to_head) {
            first = (k.b * p.N + k.n) * static_cast<int64_t>(Hp) * d;
            rank = p.N * p.B * Hp * d;
        } else {
            first = static_cast<int64_t>(k.m) * H * d;
            rank = 0;
        }
    }
    __device__ __forceinline__ int rank_of(int h) const
    {
        return magic ? static_cast<int>(__umulhi(static_cast<unsigned>(h), magic)) : h;
    }
    __device__ __forceinline__ int64_t at(int h, int d) const
    {
        const int r = rank_of(h);
        return first + r * rank + (h - r * per) * d;
    }
};

// The frequencies and their axes, in shared memory: lanes that index the kernel's
// parameters at different places are served one by one.
template <int kD>
struct Freqs {
    uint64_t turn[kD / 2];
    uint8_t axis[kD / 2];

    __device__ __forceinline__ void load(const NormRopeParams &p)
    {
        for (int i = threadIdx.x; i < p.half; i += kThreads) {
            turn[i] = p.turn[i];
            axis[i] = p.axis[i];
        }
    }
};

// Extents (elements) of a near tensor of H heads whose tokens are `stride` apart,
// for the bounds checks of debug builds.
[[maybe_unused]] __device__ __forceinline__ int64_t near_extent(const NormRopeParams &p, int64_t stride, int H, int d)
{
    return (p.tokens - 1) * stride + static_cast<int64_t>(H) * d;
}

// cos and sin of a token's rot/2 angles in the warp's shared table.  A lane
// makes at most two; the positions of the next token are read while this one
// is worked on.
template <int kD>
struct Angles {
    int64_t pos[2];
    uint32_t held, made;  // the token whose positions these are, and the one the table is of

    __device__ __forceinline__ Angles() : held(~0u), made(~0u) {}
    __device__ __forceinline__ void read(const NormRopeParams &p, const Freqs<kD> &fr, uint32_t m, int lane,
                                         [[maybe_unused]] unsigned *status)
    {
        held = m;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (lane + 32 * i >= p.half)
                continue;
            const int64_t off = fr.axis[lane + 32 * i] * p.tokens + m;
            if (ULY_IN_BOUNDS(status, off, 1, p.axes * p.tokens, 0x41))
                pos[i] = p.positions[off];
        }
    }
    // true if the table is new; `next`: the warp's next token
    __device__ __forceinline__ bool make(const NormRopeParams &p, const Freqs<kD> &fr, const Token &k, uint32_t next,
                                         float2 *table, int lane, unsigned *status)
    {
        if (made == k.m)
            return false;
        made = k.m;
        if (p.positions && held != k.m)
            read(p, fr, k.m, lane, status);
        __syncwarp();  // the last token's reads are done
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int f = lane + 32 * i;
            if (f < p.half) {
                const uint64_t frac = fr.turn[f] * static_cast<uint64_t>(p.positions ? pos[i] : k.n);
                float sn, cs;
                // its upper 32 bits, as half turns in [-1, 1)
                sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f, &sn, &cs);
                table[f] = make_float2(cs, sn);
            }
        }
        __syncwarp();
        if (p.positions && next < p.tokens)
            read(p, fr, next, lane, status);
        return true;
    }
};

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
// (interleaved).  kBack: its transpose.  Without a weight the half-split pairs
// have c_lo = c_hi and s_lo = -s_hi, and are held once.
template <typename S, bool kInter, bool kBack, bool kWeighed>
struct Turn {
    static constexpr bool kOnce = !kInter && !kWeighed;
    float2 cl[S::kP], sl[S::kP], ch[kOnce ? 1 : S::kP], sh[kOnce ? 1 : S::kP];
    bool turns;  // both chunks do or neither (rot is a multiple of 16): an infinity must not meet a zero sine

    __device__ __forceinline__ void load(const float2 *table, int half, int lo, int hi)
    {
        const float sign = kBack ? -1.f : 1.f;
        turns = kInter ? lo < 2 * half : lo < half;
#pragma unroll
        for (int j = 0; j < S::kP; ++j) {
            float2 t = make_float2(1.f, 0.f), u = t;
            if (turns)
                t = table[kInter ? lo / 2 + j : lo + 2 * j], u = table[kInter ? hi / 2 + j : lo + 2 * j + 1];
            cl[j] = kInter ? both(t.x) : make_float2(t.x, u.x);
            sl[j] = kInter ? make_float2(-sign * t.y, sign * t.y) : make_float2(-sign * t.y, -sign * u.y);
            if constexpr (!kOnce) {
                ch[j] = kInter ? both(u.x) : cl[j];
                sh[j] = kInter ? make_float2(-sign * u.y, sign * u.y) : make_float2(-sl[j].x, -sl[j].y);
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
            hi[j] = fmul2(b, kOnce ? cl[j] : ch[kOnce ? 0 : j]);
            if (turns) {
                lo[j] = ffma2(kInter ? swap(a) : b, sl[j], lo[j]);
                hi[j] = ffma2(kInter ? swap(b) : a, kOnce ? make_float2(-sl[j].x, -sl[j].y) : sh[kOnce ? 0 : j], hi[j]);
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

// A place in a warp's list of runs.  Unit u (a token, or a part of a token's
// runs) goes to warp u modulo the number of warps, so that all warps work on
// neighbouring memory.  A unit's runs are kRun rows each of the token's list:
// Q's heads, then K's, then V's.  The first `whole` tokens are units of their
// own, the others come in parts.
template <typename S>
struct Cursor {
    uint32_t u, units, stride;
    int r, end;  // this run, and the first run past the unit
    Token k;

    __device__ __forceinline__ Cursor(const NormRopeParams &p, uint32_t warp, uint32_t warps)
        : u(warp), units(static_cast<uint32_t>(p.whole + (p.tokens - p.whole) * p.splits)), stride(warps)
    {
        enter(p);
    }
    static __device__ __forceinline__ int rows(const NormRopeParams &p) { return p.Hq + (p.v ? 2 : 1) * p.Hkv; }
    __device__ __forceinline__ bool more() const { return u < units; }
    __device__ __forceinline__ void enter(const NormRopeParams &p)
    {
        uint32_t m = u;
        r = 0;
        end = p.runs;
        if (u >= static_cast<uint32_t>(p.whole)) {
            const uint32_t at = u - static_cast<uint32_t>(p.whole), token = at / p.splits;
            m = static_cast<uint32_t>(p.whole) + token;
            r = static_cast<int>(at - token * p.splits) * p.runs_per_split;
            end = min(p.runs, r + p.runs_per_split);
        }
        const uint32_t sb = m / static_cast<uint32_t>(p.Np), s = sb / static_cast<uint32_t>(p.B);
        k = Token{m, s * p.Np + (m - sb * p.Np), static_cast<int>(sb - s * p.B)};
    }
    // to the next run
    __device__ __forceinline__ void step(const NormRopeParams &p)
    {
        if (++r < end)
            return;
        u += stride;
        if (more())
            enter(p);
    }
    __device__ __forceinline__ int row0() const { return r * S::kRun; }
    __device__ __forceinline__ int row1(const NormRopeParams &p) const { return min(rows(p), (r + 1) * S::kRun); }
    // heads [h0, h1) of tensor t in this run; `at`: the run's row of head h0
    __device__ __forceinline__ void heads(const NormRopeParams &p, int t, int &h0, int &h1, int &at) const
    {
        const int first = t == 0 ? 0 : (t == 1 ? p.Hq : p.Hq + p.Hkv);
        h0 = max(row0() - first, 0);
        h1 = min(row1(p) - first, t ? p.Hkv : p.Hq);
        at = first + h0 - row0();
    }
    __device__ __forceinline__ Far far(const NormRopeParams &p, int t) const
    {
        return t ? Far(p, k, p.Hkv, p.Hkvp, p.magic_k, S::kD) : Far(p, k, p.Hq, p.Hqp, p.magic_q, S::kD);
    }
};

// Where a warp's run lands: kParts times kRunBytes, and the barrier of its copies.
template <int kParts, int kRunBytes>
struct Landing {
    uint8_t *data;
    uint64_t *bar;

    __device__ __forceinline__ Landing(uint8_t *smem, int warp, int lane)
    {
        data = smem + warp * (kParts * kRunBytes);
        bar = reinterpret_cast<uint64_t *>(smem + kWarps * (kParts * kRunBytes)) + warp;
        if (lane == 0) {
            mbar_init(bar, 1);
            fence_mbar_init();
        }
        __syncwarp();
    }
    static constexpr int kBytes = kWarps * (kParts * kRunBytes + 8);
};

template <typename T, int kD, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads, Fwd<T, kNorm>::kBlocks)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p, const WaitCfg wait)
{
    constexpr int kRunBytes = Fwd<T, kNorm>::kRun;
    using S = Shape<T, kD, kRunBytes>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 table[kWarps][kD / 2];
    __shared__ __align__(16) T weights[2][kD];
    __shared__ Freqs<kD> freqs;
    const int warp = warp_id(), lane = lane_id(), sub = lane / S::kLanes;
    freqs.load(p);
    if (kNorm) {
        for (int i = threadIdx.x; i < kD; i += kThreads) {
            weights[0][i] = static_cast<const T *>(p.wq)[i];
            weights[1][i] = static_cast<const T *>(p.wk)[i];
        }
    }
    __syncthreads();
    const Landing<1, kRunBytes> run(smem, warp, lane);
    int lo, hi;
    chunk_places<S, kInter>(p.half, lane % S::kLanes, lo, hi);
    Cursor<S> now(p, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
    Cursor<S> ahead = now;
    auto fetch = [&] {  // a copy per tensor
        if (lane == 0)
            mbar_expect_tx(run.bar, (ahead.row1(p) - ahead.row0()) * kD * sizeof(T));
        __syncwarp();
        int h0, h1, row;
        ahead.heads(p, lane, h0, h1, row);
        if (lane < 3 && h0 < h1) {
            const T *src = static_cast<const T *>(lane == 0 ? p.q : (lane == 1 ? p.k : p.v));
            const int64_t stride = lane == 0 ? p.qs : (lane == 1 ? p.ks : p.vs), off = ahead.k.m * stride + h0 * kD;
            // (a check that fails is reported and the first token's rows are copied, which the barrier counts on)
            if (ULY_IN_BOUNDS(wait.status, off, (h1 - h0) * kD, near_extent(p, stride, lane ? p.Hkv : p.Hq, kD), 0x42))
                src += off;
            bulk_g2s(run.data + row * kD * sizeof(T), src, (h1 - h0) * kD * sizeof(T), run.bar);
        }
        ahead.step(p);
    };
    if (ahead.more())
        fetch();
    uint32_t phase = 0;
    Angles<kD> at;
    int last = -1;
    Turn<S, kInter, false, kNorm> turn;
    Far far;
    while (now.more()) {
        if (now.row0() < p.Hq + p.Hkv && at.make(p, freqs, now.k, now.k.m + now.stride, table[warp], lane,
                                                  wait.status))
            last = -1;
        if (!__all_sync(0xffffffffu, mbar_wait(run.bar, phase, wait, 0xb1)))
            break;
        phase ^= 1;
        const T *data = reinterpret_cast<const T *>(run.data);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            int h0, h1, row;
            now.heads(p, t, h0, h1, row);
            if (h0 >= h1)
                continue;
            if (t != last) {
                last = t;
                turn.load(table[warp], p.half, lo, hi);
                if constexpr (kNorm) {
                    const Raw raw = load_row<T>(weights[t], lo, hi);
                    float2 wl[S::kP], wh[S::kP];
                    unpack<T>(raw.lo, wl);
                    unpack<T>(raw.hi, wh);
                    turn.weigh(wl, wh);
                }
            }
            far = now.far(p, t);
            T *out = static_cast<T *>(t ? p.ko : p.qo);
            const T *rows = data + (row - h0) * kD;
#pragma unroll 2
            for (int hb = h0; hb < h1; hb += S::kRows) {
                const int h = hb + sub;
                const Raw raw = load_row<T>(rows + min(h, h1 - 1) * kD, lo, hi);
                float2 x[S::kP], y[S::kP];
                unpack<T>(raw.lo, x);
                unpack<T>(raw.hi, y);
                float rstd = 1.f;
                if (kNorm) {
                    float2 ss = both(0.f), st = ss;
#pragma unroll
                    for (int j = 0; j < S::kP; ++j) {
                        ss = ffma2(x[j], x[j], ss);
                        st = ffma2(y[j], y[j], st);
                    }
                    ss = fadd2(ss, st);
                    rstd = rsqrtf(row_sum<S::kLanes>(ss.x + ss.y) * (1.f / kD) + p.eps);
                }
                turn.apply(x, y);
                if (kNorm) {
#pragma unroll
                    for (int j = 0; j < S::kP; ++j) {
                        x[j] = fmul2(x[j], both(rstd));
                        y[j] = fmul2(y[j], both(rstd));
                    }
                }
                if (h < h1 && ULY_IN_BOUNDS(wait.status, far.at(h, kD), kD, p.tokens * (t ? p.Hkv : p.Hq) * kD, 0x43))
                    store_row<T>(out + far.at(h, kD), lo, hi, Raw{pack<T>(x), pack<T>(y)});
            }
        }
        int h0, h1, row;
        now.heads(p, 2, h0, h1, row);
        if (h0 < h1) {
            far = now.far(p, 2);
#pragma unroll 2
            for (int h = h0 + sub; h < h1; h += S::kRows)
                if (ULY_IN_BOUNDS(wait.status, far.at(h, kD), kD, p.tokens * p.Hkv * kD, 0x44))
                    store_row<T>(static_cast<T *>(p.vo) + far.at(h, kD), lo, hi,
                                 load_row<T>(data + (row + h - h0) * kD, lo, hi));
        }
        __syncwarp();  // the run is read
        if (ahead.more())
            fetch();
        now.step(p);
    }
    if (now.more())  // after a wait that ran out: the copies still on their way (bounded)
        mbar_wait(run.bar, phase, wait, 0xbf);
}

template <typename T, int kD, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads, Bwd<T, kNorm>::kBlocks)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, const WaitCfg wait)
{
    constexpr int kRunBytes = Bwd<T, kNorm>::kRun;
    using S = Shape<T, kD, kRunBytes>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 table[kWarps][kD / 2];
    __shared__ __align__(16) T weights[2][kD];
    __shared__ Freqs<kD> freqs;
    const int warp = warp_id(), lane = lane_id(), sub = lane / S::kLanes;
    freqs.load(p);
    if (kNorm) {
        for (int i = threadIdx.x; i < kD; i += kThreads) {
            weights[0][i] = static_cast<const T *>(p.wq)[i];
            weights[1][i] = static_cast<const T *>(p.wk)[i];
        }
    }
    __syncthreads();
    constexpr int kParts = kNorm ? 2 : 1;  // a run of dy and one of x
    const Landing<kParts, kRunBytes> run(smem, warp, lane);
    int lo, hi;
    chunk_places<S, kInter>(p.half, lane % S::kLanes, lo, hi);
    // the warp's part of dw, kept between runs: [q, k][slot][d]
    constexpr int kSlots = S::kRows < 2 ? 1 : 2;
    constexpr int kSums = kNorm ? 2 * kSlots * kD : 2;
    __shared__ float2 sums[kWarps][kSums / 2];
    if (kNorm)
        for (int i = lane; i < kSums / 2; i += 32)
            sums[warp][i] = both(0.f);
    __syncwarp();
    Cursor<S> now(p, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
    Cursor<S> ahead = now;
    auto fetch = [&] {
        // Lanes 0, 1, 2 (mod 4): dy of Q, K and V, a copy per rank; lanes 3 and 7: x of Q and K
        uint8_t *to = run.data;
        const int row0 = ahead.row0(), row1 = ahead.row1(p), xrows = max(min(row1, p.Hq + p.Hkv) - row0, 0);
        if (lane == 0)
            mbar_expect_tx(run.bar, (row1 - row0 + (kNorm ? xrows : 0)) * kD * sizeof(T));
        __syncwarp();
        const int kind = lane & 3, t = kind < 3 ? kind : lane >> 2;
        int h0, h1, row;
        ahead.heads(p, t, h0, h1, row);
        if (kind < 3) {
            const Far far = ahead.far(p, t);
            const T *src = static_cast<const T *>(t == 0 ? p.qo : (t == 1 ? p.ko : p.vo));
            for (int i = far.rank_of(h0) + (lane >> 2); h0 < h1; i += 8) {
                const int a = max(h0, i * far.per), b = min(h1, (i + 1) * far.per);
                if (a >= b)
                    break;
                const bool ok = ULY_IN_BOUNDS(wait.status, far.at(a, kD), (b - a) * kD,
                                              p.tokens * (t ? p.Hkv : p.Hq) * kD, 0x45);
                bulk_g2s(to + (row + a - h0) * kD * sizeof(T), src + (ok ? far.at(a, kD) : 0), (b - a) * kD * sizeof(T),
                         run.bar);
            }
        } else if (kNorm && t < 2 && h0 < h1) {
            const int64_t stride = t ? p.ks : p.qs, off = ahead.k.m * stride + h0 * kD;
            const bool ok =
                ULY_IN_BOUNDS(wait.status, off, (h1 - h0) * kD, near_extent(p, stride, t ? p.Hkv : p.Hq, kD), 0x46);
            bulk_g2s(to + kRunBytes + row * kD * sizeof(T), static_cast<const T *>(t ? p.k : p.q) + (ok ? off : 0),
                     (h1 - h0) * kD * sizeof(T), run.bar);
        }
        ahead.step(p);
    };
    if (ahead.more())
        fetch();
    uint32_t phase = 0;
    Angles<kD> at;
    Turn<S, kInter, true, false> turn;
    while (now.more()) {
        if (now.row0() < p.Hq + p.Hkv && at.make(p, freqs, now.k, now.k.m + now.stride, table[warp], lane,
                                                  wait.status))
            turn.load(table[warp], p.half, lo, hi);
        if (!__all_sync(0xffffffffu, mbar_wait(run.bar, phase, wait, 0xb2)))
            break;
        phase ^= 1;
        const T *data = reinterpret_cast<const T *>(run.data);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            int h0, h1, row;
            now.heads(p, t, h0, h1, row);
            if (h0 >= h1)
                continue;
            const int64_t stride = t ? p.dks : p.dqs, near = static_cast<int64_t>(now.k.m) * stride;
            T *out = static_cast<T *>(t ? p.dk : p.dq);
            const T *rows = data + (row - h0) * kD, *xrows = rows + kRunBytes / sizeof(T);
            float2 w[2][S::kP], sum[2][S::kP];
            if (kNorm) {
                const Raw raw = load_row<T>(weights[t], lo, hi);
                unpack<T>(raw.lo, w[0]);
                unpack<T>(raw.hi, w[1]);
            }
#pragma unroll
            for (int j = 0; j < S::kP; ++j)
                sum[0][j] = sum[1][j] = both(0.f);
#pragma unroll 1
            for (int hb = h0; hb < h1; hb += S::kRows) {
                const int h = hb + sub, hr = min(h, h1 - 1);
                const bool live = h < h1;
                const Raw raw = load_row<T>(rows + hr * kD, lo, hi);
                float2 g[2][S::kP];
                unpack<T>(raw.lo, g[0]);
                unpack<T>(raw.hi, g[1]);
                turn.apply(g[0], g[1]);
                if (kNorm) {
                    const Raw rawx = load_row<T>(xrows + hr * kD, lo, hi);
                    float2 x[2][S::kP], ss[2] = {both(0.f), both(0.f)}, dot[2] = {both(0.f), both(0.f)};
                    unpack<T>(rawx.lo, x[0]);
                    unpack<T>(rawx.hi, x[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < S::kP; ++j) {
                            ss[c] = ffma2(x[c][j], x[c][j], ss[c]);
                            dot[c] = ffma2(w[c][j], fmul2(g[c][j], x[c][j]), dot[c]);
                        }
                    ss[0] = fadd2(ss[0], ss[1]);
                    dot[0] = fadd2(dot[0], dot[1]);
                    const float rstd = rsqrtf(row_sum<S::kLanes>(ss[0].x + ss[0].y) * (1.f / kD) + p.eps);
                    // mean(w g xhat) r: what x loses, before the last factor r
                    const float m = row_sum<S::kLanes>(dot[0].x + dot[0].y) * (1.f / kD) * rstd * rstd;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < S::kP; ++j) {
                            if (live)
                                sum[c][j] = ffma2(fmul2(g[c][j], x[c][j]), both(rstd), sum[c][j]);
                            g[c][j] = fmul2(ffma2(x[c][j], both(-m), fmul2(w[c][j], g[c][j])), both(rstd));
                        }
                }
                if (live && ULY_IN_BOUNDS(wait.status, near + h * kD, kD,
                                          near_extent(p, stride, t ? p.Hkv : p.Hq, kD), 0x47))
                    store_row<T>(out + near + h * kD, lo, hi, Raw{pack<T>(g[0]), pack<T>(g[1])});
            }
            if (kNorm) {
                float *to = reinterpret_cast<float *>(sums[warp]) + (t * kSlots + sub) * kD;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < S::kP; ++j) {
                        float2 v = sum[c][j];
#pragma unroll
                        for (int o = 16; o >= S::kLanes * kSlots; o >>= 1)
                            v = fadd2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                                                     __shfl_xor_sync(0xffffffffu, v.y, o)));
                        if (sub < kSlots) {
                            float2 *place = reinterpret_cast<float2 *>(to + (c ? hi : lo) + 2 * j);
                            *place = fadd2(*place, v);
                        }
                    }
            }
        }
        int h0, h1, row;
        now.heads(p, 2, h0, h1, row);
        if (h0 < h1) {
            const int64_t near = static_cast<int64_t>(now.k.m) * p.dvs;
#pragma unroll 2
            for (int h = h0 + sub; h < h1; h += S::kRows)
                if (ULY_IN_BOUNDS(wait.status, near + h * kD, kD, near_extent(p, p.dvs, p.Hkv, kD), 0x48))
                    store_row<T>(static_cast<T *>(p.dv) + near + h * kD, lo, hi,
                                 load_row<T>(data + (row + h - h0) * kD, lo, hi));
        }
        __syncwarp();  // the run is read
        if (ahead.more())
            fetch();
        now.step(p);
    }
    if (now.more())  // after a wait that ran out: the copies still on their way (bounded)
        mbar_wait(run.bar, phase, wait, 0xbf);
    if constexpr (kNorm) {
        // the block's weight-gradient partial: row slots and warps, always in the same order
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kD; i += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int k = 0; k < kSlots; ++k)
                    v += reinterpret_cast<const float *>(sums[w])[(i / kD * kSlots + k) * kD + i % kD];
            const int64_t off = static_cast<int64_t>(blockIdx.x) * 2 * kD + i;
            if (ULY_IN_BOUNDS(wait.status, off, 1, kNormRopeMaxBlocks * 2 * kD, 0x49))
                p.partial[off] = v;
        }
    }
}

// dw[i] = sum over the blocks' partials: 128 strided runs of them, in block
// order, then the runs, always in the same order.  A block takes 8 values and
// has its loads on their way together: 2 us behind the backward, 4 with blocks of
// 32 values and loads one by one.
constexpr int kDwCols = 8, kDwRuns = 128;
template <typename T>
__global__ void __launch_bounds__(kDwCols *kDwRuns) norm_rope_dw_kernel(const float *__restrict__ partial, int blocks,
                                                                       int d, T *__restrict__ dwq,
                                                                       T *__restrict__ dwk)
{
    __shared__ float run[kDwCols][kDwRuns + 1];
    grid_wait();
    const int tx = threadIdx.x % kDwCols, ty = threadIdx.x / kDwCols;
    constexpr int kAhead = 6;
    float s = 0.f;
    for (int b0 = ty; b0 < blocks; b0 += kDwRuns * kAhead) {
        float v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int b = b0 + kDwRuns * i;
            v[i] = b < blocks ? partial[static_cast<int64_t>(b) * 2 * d + blockIdx.x * kDwCols + tx] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            s += v[i];
    }
    run[tx][ty] = s;
    __syncthreads();
    if (warp_id() >= kDwCols)
        return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kDwRuns; k += 32)
        s += run[warp_id()][lane_id() + k];
    s = row_sum<32>(s);
    const int col = blockIdx.x * kDwCols + warp_id();
    T *dw = col < d ? dwq : dwk;
    if (dw == nullptr || lane_id() != 0)
        return;
    if constexpr (sizeof(T) == 2)
        dw[col % d] = static_cast<T>(pack_bf16x2(s, 0.f) & 0xffffu);
    else
        dw[col % d] = s;
}

template <typename T, int kD, bool kInter, bool kNorm>
cudaError_t run(NormRopeParams &p, bool bwd, cudaStream_t s)
{
    constexpr int kFwdRun = Fwd<T, kNorm>::kRun, kBwdRun = Bwd<T, kNorm>::kRun;
    const int kRun = (bwd ? kBwdRun : kFwdRun) / static_cast<int>(kD * sizeof(T));
    const int runs = (p.Hq + (p.v ? 2 : 1) * p.Hkv + kRun - 1) / kRun;
    p.runs = runs;
    const int64_t resident = static_cast<int64_t>(num_sms()) * (bwd ? Bwd<T, kNorm>::kBlocks : Fwd<T, kNorm>::kBlocks);
    // Tokens that are fewer than the warps come in the parts that end first:
    // rounds of parts x runs of a part.  So do the backward's last tokens, when
    // every warp has had the same number of whole ones: 2048 tokens of 32 + 8 + 8
    // heads 25.3 us (parts for as many warps as there are 31.5), 4095 fp32 ones of
    // 12 + 6 + 6 25.1 (all whole 27.4).  In the forward the parts' angles cost
    // what their rounds save (8192 tokens 43.7 us either way; caches emptied).
    const int64_t warps = resident * kWarps;
    p.whole = bwd || p.tokens < warps ? p.tokens / warps * warps : p.tokens;
    const int64_t rest = p.tokens - p.whole;
    p.runs_per_split = runs;
    int64_t best = INT64_MAX;
    for (int64_t k = 1; rest > 0 && k <= std::min<int64_t>(runs, (warps + rest - 1) / rest); ++k) {
        const int64_t per = (runs + k - 1) / k, parts = (runs + per - 1) / per;
        const int64_t time = (rest * parts + warps - 1) / warps * per;
        if (time < best) {
            best = time;
            p.runs_per_split = static_cast<int>(per);
        }
    }
    p.splits = (runs + p.runs_per_split - 1) / p.runs_per_split;
    if (p.splits == 1)
        p.whole = p.tokens;
    p.magic_q = p.Hqp == 1 ? 0u : 0xffffffffu / p.Hqp + 1;
    p.magic_k = p.Hkvp == 1 ? 0u : 0xffffffffu / p.Hkvp + 1;
    const int64_t grid = std::min<int64_t>((p.whole + (p.tokens - p.whole) * p.splits + kWarps - 1) / kWarps, resident);
    if (!bwd) {
        auto kernel = norm_rope_fwd_kernel<T, kD, kInter, kNorm>;
        constexpr int smem = Landing<1, kFwdRun>::kBytes;
        static_assert(smem <= 40 * 1024, "with the static part, what a launch may take without asking");
        kernel<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(p, wait_cfg());
        return cudaGetLastError();
    }
    if (grid > kNormRopeMaxBlocks)
        return cudaErrorInvalidConfiguration;
    auto kernel = norm_rope_bwd_kernel<T, kD, kInter, kNorm>;
    constexpr int smem = Landing<kNorm ? 2 : 1, kBwdRun>::kBytes;
    static_assert(smem + static_cast<int>(sizeof(float)) * 24 * kD <= 48 * 1024, "as above");
    kernel<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(p, wait_cfg());
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    if (kNorm && (p.dwq || p.dwk))
        return launch_after(norm_rope_dw_kernel<T>, 2 * kD / kDwCols, kDwCols * kDwRuns, 0, s, p.partial,
                            static_cast<int>(grid), kD, static_cast<T *>(p.dwq), static_cast<T *>(p.dwk));
    return cudaSuccess;
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

// The part of v behind the point as a 64-bit fraction, modulo 1.
static uint64_t fraction(double v)
{
    const double f = std::ldexp(std::fabs(v - std::trunc(v)), 64);
    return v < 0 ? 0 - static_cast<uint64_t>(f) : static_cast<uint64_t>(f);
}

// inv_freq / 2 pi in three parts: the product with the nearest double of 1 / 2 pi,
// that product's rounding error, and the product with what is left of 1 / 2 pi
// (0.159154943091895335768883763372514362...).  Each part is cut to 64 bits, and the
// last one's rounding and what it leaves out are below 2^-108 of inv_freq.
uint64_t turn_fraction(double inv_freq)
{
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double p = inv_freq * kHi;
    return fraction(p) + fraction(std::fma(inv_freq, kHi, -p)) + fraction(inv_freq * kLo);
}

cudaError_t launch_norm_rope(NormRopeParams &p, int d, bool inter, bool bwd, int esize, cudaStream_t s)
{
    if (esize == 2)
        return d == 64 ? run_d<uint16_t, 64>(p, inter, bwd, s) : run_d<uint16_t, 128>(p, inter, bwd, s);
    return d == 64 ? run_d<float, 64>(p, inter, bwd, s) : run_d<float, 128>(p, inter, bwd, s);
}

}  // namespace uly
