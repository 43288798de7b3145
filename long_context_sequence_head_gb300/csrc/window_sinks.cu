// The sinks' part of the sliding-window backward (bf16) in documents with rows past
// their window, and the first values of the accumulator of dQ that the main kernel
// (attn_bwd_bf16.cu) adds to.
//
// Every later row of a document sees its up to 64 first keys.  Their dK and dV are
// sums over the whole document, many times the other keys' in magnitude, so what
// bf16 takes from P and dS there stands out: an element of such a row was up to 0.6
// of the whole dK's rms off at 64K tokens under 4 sinks.  Here P and dS go into the
// second products as two bf16 parts each (2^-17 of their value).
//   dQ_i  = sum over the sinks of dS_is k_s, past the main kernel's walk
//   dK_s  = sum_i dS_is q_i,  dV_s = sum_i P_is dO_i   (fp32, a slot for each block)
// One pass over Q and dO, 16 sinks at a time; the accumulator has to be set to zero
// in any case, so that the pass costs the reads: bound by HBM, 8 bytes an element of Q.
// 64K tokens of 32 heads 348 us, 6.1 TB/s (zeroing the accumulator alone takes 160).
// A warp takes 16 rows of a 128-row tile on mma.sync (16 x 16 pieces of 4 to 64
// keys: too narrow for a tcgen05 tile of 128); tiles of Q and dO come through two
// cp.async buffers.
#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kBM = 128, kD = 128;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kKeys = 16;                 // sinks at a time
constexpr int kRowBytes = kD * 2;
constexpr int kTile = kBM * kRowBytes;    // 32 KB

struct Smem {
    static constexpr int kK = 0;                              // [64][128] bf16
    static constexpr int kV = kK + kWindowSinks * kRowBytes;
    static constexpr int kBuf = kV + kWindowSinks * kRowBytes;  // [2][Q, dO]
    static constexpr int kStats = kBuf + 4 * kTile;           // [2][lse2, D][128]
    static constexpr int kTotal = kStats + 2 * 2 * kBM * 4;
};

struct Params {
    const uint16_t *q, *k, *v, *dout;
    const float *lse2, *Dv;  // [SB][Hq][Npad]
    float *acc;              // [SB][Hq][Npad/128][32][128][4]
    float *part;             // the units' slots
    const int4 *chunks;      // three a chunk, see WindowUnits
    int64_t SB, N, Npad;
    int Hq, Hkv, G, slots, rows;
    int pass;  // wide: groups of keys of a block
    float scale_log2;
    int64_t q_elems, kv_elems;
    unsigned *status;
};

__device__ __forceinline__ uint32_t tile_at(int r, int unit) { return r * kRowBytes + ((unit ^ (r & 7)) << 4); }

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool read)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(read ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// c += a b: a 16 x 16, b 16 x 8, c 16 x 8 (rows lane/4 and + 8, columns 2 (lane%4) and + 1)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A pair of values as two bf16 pairs whose sum is 2^-17 of it off.
__device__ __forceinline__ void two_parts(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x, y);
    lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

__global__ void __launch_bounds__(kThreads, 1) window_sinks_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = warp_id(), lane = lane_id();
    const int64_t nprob = p.SB * p.Hkv, prob = blockIdx.x % nprob;
    const int chunk = static_cast<int>(blockIdx.x / nprob);
    const int kvh = static_cast<int>(prob % p.Hkv);
    const int64_t sb = prob / p.Hkv;
    // {first row tile, past the last, document's start or -1, sinks}, {slot of the first key tile's sinks, from
    // it to the second's, last row tile that the main kernel walks for each}, {document's end, first row tile to set}
    const int4 a = p.chunks[3 * chunk], b = p.chunks[3 * chunk + 1], c = p.chunks[3 * chunk + 2];
    const int64_t tiles = p.Npad / kBM;
    [[maybe_unused]] const int64_t acc_elems = p.SB * p.Hq * p.Npad * kD;
    if (a.z < 0) {  // rows that see no sink past their window
        for (int g = 0; g < p.G; ++g) {
            const int64_t off = ((sb * p.Hq + kvh * p.G + g) * tiles + a.x) * (kBM * kD);
            const int64_t n = static_cast<int64_t>(a.y - a.x) * (kBM * kD);
            if (!ULY_IN_BOUNDS(p.status, off, n, acc_elems, 0x33))
                break;
            for (int64_t i = threadIdx.x; i < n / 4; i += kThreads)
                reinterpret_cast<float4 *>(p.acc + off)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    const uint32_t base = smem_u32(smem);
    // the sinks' keys and values, zeros behind them
    const int groups = (a.w + kKeys - 1) / kKeys;
    for (int i = threadIdx.x; i < groups * kKeys * 16; i += kThreads) {
        const int r = i / 16, unit = i % 16;
        const int64_t off = ((sb * p.N + a.z + r) * p.Hkv + kvh) * kD + unit * 8;
        const bool in = r < a.w && ULY_IN_BOUNDS(p.status, off, 8, p.kv_elems, 0x34);
        copy16(base + Smem::kK + tile_at(r, unit), p.k + (in ? off : 0), in);
        copy16(base + Smem::kV + tile_at(r, unit), p.v + (in ? off : 0), in);
    }
    const int steps = (a.y - a.x) * p.G;  // (row tile, head of the group)
    auto load = [&](int step) {
        if (step < steps) {
            const int64_t row0 = static_cast<int64_t>(a.x + step / p.G) * kBM;
            const int h = kvh * p.G + step % p.G;
            const uint32_t to = base + Smem::kBuf + (step & 1) * 2 * kTile;
            for (int i = threadIdx.x; i < kBM * 16; i += kThreads) {
                const int r = i / 16, unit = i % 16;
                const int64_t off = ((sb * p.N + row0 + r) * p.Hq + h) * kD + unit * 8;
                const bool in = row0 + r < p.N && ULY_IN_BOUNDS(p.status, off, 8, p.q_elems, 0x35);
                copy16(to + tile_at(r, unit), p.q + (in ? off : 0), in);
                copy16(to + kTile + tile_at(r, unit), p.dout + (in ? off : 0), in);
            }
            const int64_t at = (sb * p.Hq + h) * p.Npad + row0 + threadIdx.x % kBM;
            const bool ok = ULY_IN_BOUNDS(p.status, at, 1, p.SB * p.Hq * p.Npad, 0x36);
            copy4(base + Smem::kStats + ((step & 1) * 2 * kBM + threadIdx.x) * 4,
                  (threadIdx.x < kBM ? p.lse2 : p.Dv) + (ok ? at : 0), ok);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int second = (a.z / kBM + 1) * kBM - a.z;  // sinks in the first key tile
    const int r0 = warp * 16 + (lane >> 2);          // this lane's rows of a tile: r0 and r0 + 8
    for (int g = 0; g < groups; ++g) {
        float dk[kD / 8][4], dv[kD / 8][4];  // sinks lane/4 and + 8 of the group
#pragma unroll
        for (int n = 0; n < kD / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dk[n][e] = dv[n][e] = 0.f;
        load(0);
        for (int step = 0; step < steps; ++step) {
            load(step + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            const int m = a.x + step / p.G, h = kvh * p.G + step % p.G;
            const uint32_t q_at = base + Smem::kBuf + (step & 1) * 2 * kTile, d_at = q_at + kTile;
            const uint32_t k_at = base + Smem::kK + g * kKeys * kRowBytes, v_at = k_at + Smem::kV - Smem::kK;
            const float *stats = reinterpret_cast<const float *>(smem + Smem::kStats) + (step & 1) * 2 * kBM;
            float s[2][4] = {}, dp[2][4] = {};
            const int a_row = warp * 16 + (lane & 15), a_unit = lane >> 4;                // A: 16 rows, two halves
            const int b_row = (lane & 7) + ((lane >> 4) << 3), b_unit = (lane >> 3) & 1;  // B: keys by columns
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
                uint32_t x[4], y[4];
                ldmatrix4(q_at + tile_at(a_row, 2 * kk + a_unit), x);
                ldmatrix4(k_at + tile_at(b_row, 2 * kk + b_unit), y);
                mma(s[0], x, y[0], y[1]);
                mma(s[1], x, y[2], y[3]);
                ldmatrix4(d_at + tile_at(a_row, 2 * kk + a_unit), x);
                ldmatrix4(v_at + tile_at(b_row, 2 * kk + b_unit), y);
                mma(dp[0], x, y[0], y[1]);
                mma(dp[1], x, y[2], y[3]);
            }
            // P and dS in two parts: [part][tile of 8 keys][rows 0-7, 8-15]
            uint32_t P[2][2][2], S[2][2][2];
            const int64_t row0 = static_cast<int64_t>(m) * kBM;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = r0 + 8 * half;
                    float pr[2], ds[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = g * kKeys + 8 * n + 2 * (lane & 3) + e;  // of the document
                        const bool sees = key < a.w && row0 + r >= a.z + key && row0 + r < c.x;
                        pr[e] = sees ? ex2_approx(fmaf(s[n][2 * half + e], p.scale_log2, -stats[r])) : 0.f;
                        ds[e] = sees ? pr[e] * (dp[n][2 * half + e] - stats[kBM + r]) : 0.f;
                    }
                    two_parts(pr[0], pr[1], P[0][n][half], P[1][n][half]);
                    two_parts(ds[0], ds[1], S[0][n][half], S[1][n][half]);
                }
            // dQ: rows x d, from the group's keys that the main kernel does not walk
            uint32_t sh[4], sl[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int key = g * kKeys + 8 * n + 2 * (lane & 3);
                const uint32_t keep = (m > (key < second ? b.z : b.w) ? 0xffffu : 0u) |
                                      (m > (key + 1 < second ? b.z : b.w) ? 0xffff0000u : 0u);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    sh[2 * n + half] = S[0][n][half] & keep;
                    sl[2 * n + half] = S[1][n][half] & keep;
                }
            }
            const int64_t acc_off = ((sb * p.Hq + h) * tiles + m) * (kBM * kD);
            const bool acc_ok = m >= c.y && ULY_IN_BOUNDS(p.status, acc_off, kBM * kD, acc_elems, 0x37);
            // transposed B: two tiles of 8 columns
            const int t_row = (lane & 7) + (((lane >> 3) & 1) << 3), t_unit = lane >> 4;
#pragma unroll
            for (int n = 0; n < kD / 8; n += 2) {
                uint32_t y[4];
                ldmatrix4_t(k_at + tile_at(t_row, n + t_unit), y);
                float x[2][4] = {};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(x[e], sh, y[2 * e], y[2 * e + 1]);
                    mma(x[e], sl, y[2 * e], y[2 * e + 1]);
                    // columns 8 (n + e) + 2 (lane%4): half of a group of four
                    float *to = p.acc + acc_off + (2 * (n + e) + ((lane & 3) >> 1)) * (kBM * 4) + (lane & 1) * 2;
                    float2 *lo = reinterpret_cast<float2 *>(to + r0 * 4);
                    float2 *hi = reinterpret_cast<float2 *>(to + (r0 + 8) * 4);
                    if (!acc_ok)
                        continue;
                    if (g > 0) {
                        x[e][0] += lo->x, x[e][1] += lo->y;
                        x[e][2] += hi->x, x[e][3] += hi->y;
                    }
                    *lo = make_float2(x[e][0], x[e][1]);
                    *hi = make_float2(x[e][2], x[e][3]);
                }
            }
            // dK and dV: keys x d, from the warp's 16 rows
            uint32_t st[2][4], pt[2][4];
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // keys 0-7 / 8-15 (e & 1), rows 0-7 / 8-15 (e >> 1)
                    st[part][e] = transposed(S[part][e & 1][e >> 1]);
                    pt[part][e] = transposed(P[part][e & 1][e >> 1]);
                }
#pragma unroll
            for (int n = 0; n < kD / 8; n += 2) {
                uint32_t y[4];
                ldmatrix4_t(q_at + tile_at(warp * 16 + t_row, n + t_unit), y);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(dk[n + e], st[0], y[2 * e], y[2 * e + 1]);
                    mma(dk[n + e], st[1], y[2 * e], y[2 * e + 1]);
                }
                ldmatrix4_t(d_at + tile_at(warp * 16 + t_row, n + t_unit), y);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(dv[n + e], pt[0], y[2 * e], y[2 * e + 1]);
                    mma(dv[n + e], pt[1], y[2 * e], y[2 * e + 1]);
                }
            }
            __syncthreads();  // the buffer is read: it may be filled again
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // the warps' sums, in order, to the chunk's slots: [warp][dK, dV][16][128]
        float *sums = reinterpret_cast<float *>(smem + Smem::kBuf);
        static_assert(kWarps * 2 * kKeys * kD * 4 <= 4 * kTile, "the warps' sums fit");
#pragma unroll
        for (int n = 0; n < kD / 8; ++n)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float *to = sums + ((warp * 2) * kKeys + (lane >> 2) + 8 * half) * kD + 8 * n + 2 * (lane & 3);
                *reinterpret_cast<float2 *>(to) = make_float2(dk[n][2 * half], dk[n][2 * half + 1]);
                *reinterpret_cast<float2 *>(to + kKeys * kD) = make_float2(dv[n][2 * half], dv[n][2 * half + 1]);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kKeys * kD; i += kThreads) {
            const int which = i / (kKeys * kD), key = g * kKeys + i / kD % kKeys, col = i % kD;
            if (key >= a.w)
                continue;
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                t += sums[w * 2 * kKeys * kD + i];
            const int slot = key < second ? b.x : b.x + b.y, at = key < second ? key : key - second;
            const int64_t off = (((prob * p.slots + slot) * 2 + which) * p.rows + at) * kD + col;
            if (ULY_IN_BOUNDS(p.status, off, 1, nprob * p.slots * 2 * p.rows * kD, 0x38))
                p.part[off] = t;
        }
        __syncthreads();
    }
}

// More sinks: dK and dV alone, dQ is the main kernel's.  A warp has 16 keys and all
// rows, scores are formed with the keys as the rows of the products (K and V in
// registers), which is also how the second products take them.  Shared memory binds:
// every warp reads every row of Q and dO twice, 16 KB a 16 x 16 piece's products.
// 64K tokens of 32 heads: about 0.7 ms for 128 sinks.
struct Wide {
    static constexpr int kK = 0;                          // [128][128] bf16
    static constexpr int kV = kK + kWarps * kKeys * kRowBytes;
    static constexpr int kBuf = kV + kWarps * kKeys * kRowBytes;  // [2][Q, dO]
    static constexpr int kStats = kBuf + 4 * kTile;       // [2][lse2, D][128]
    static constexpr int kTotal = kStats + 2 * 2 * kBM * 4;
};

__global__ void __launch_bounds__(kThreads, 1) window_sinks_wide_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = warp_id(), lane = lane_id();
    const int64_t nprob = p.SB * p.Hkv, prob = blockIdx.x % nprob;
    const int chunk = static_cast<int>(blockIdx.x / nprob);
    const int kvh = static_cast<int>(prob % p.Hkv);
    const int64_t sb = prob / p.Hkv;
    const int4 a = p.chunks[3 * chunk], b = p.chunks[3 * chunk + 1], c = p.chunks[3 * chunk + 2];
    const int first = blockIdx.y * p.pass * kKeys, last = min(first + p.pass * kKeys, a.w);
    if (first >= last)
        return;
    const uint32_t base = smem_u32(smem);
    for (int i = threadIdx.x; i < kWarps * kKeys * 16; i += kThreads) {
        const int r = i / 16, unit = i % 16;
        const int64_t off = ((sb * p.N + a.z + first + r) * p.Hkv + kvh) * kD + unit * 8;
        const bool in = first + r < last && ULY_IN_BOUNDS(p.status, off, 8, p.kv_elems, 0x39);
        copy16(base + Wide::kK + tile_at(r, unit), p.k + (in ? off : 0), in);
        copy16(base + Wide::kV + tile_at(r, unit), p.v + (in ? off : 0), in);
    }
    const int steps = (a.y - a.x) * p.G;  // (row tile, head of the group)
    auto load = [&](int step) {
        if (step < steps) {
            const int64_t row0 = static_cast<int64_t>(a.x + step / p.G) * kBM;
            const int h = kvh * p.G + step % p.G;
            const uint32_t to = base + Wide::kBuf + (step & 1) * 2 * kTile;
            for (int i = threadIdx.x; i < kBM * 16; i += kThreads) {
                const int r = i / 16, unit = i % 16;
                const int64_t off = ((sb * p.N + row0 + r) * p.Hq + h) * kD + unit * 8;
                const bool in = row0 + r < p.N && ULY_IN_BOUNDS(p.status, off, 8, p.q_elems, 0x3a);
                copy16(to + tile_at(r, unit), p.q + (in ? off : 0), in);
                copy16(to + kTile + tile_at(r, unit), p.dout + (in ? off : 0), in);
            }
            const int64_t at = (sb * p.Hq + h) * p.Npad + row0 + threadIdx.x % kBM;
            const bool ok = ULY_IN_BOUNDS(p.status, at, 1, p.SB * p.Hq * p.Npad, 0x3b);
            copy4(base + Wide::kStats + ((step & 1) * 2 * kBM + threadIdx.x) * 4,
                  (threadIdx.x < kBM ? p.lse2 : p.Dv) + (ok ? at : 0), ok);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(0);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const bool mine = first + warp * kKeys < last && warp < p.pass;
    uint32_t ka[kD / 16][4], va[kD / 16][4];
#pragma unroll
    for (int kk = 0; kk < kD / 16; ++kk) {
        const uint32_t at = tile_at(warp * kKeys + (lane & 15), 2 * kk + (lane >> 4));
        ldmatrix4(base + Wide::kK + at, ka[kk]);
        ldmatrix4(base + Wide::kV + at, va[kk]);
    }
    float dk[kD / 8][4], dv[kD / 8][4];  // keys lane/4 and + 8 of the warp's
#pragma unroll
    for (int n = 0; n < kD / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            dk[n][e] = dv[n][e] = 0.f;
    const int key0 = first + warp * kKeys + (lane >> 2);
    for (int step = 0; step < steps; ++step) {
        load(step + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const int64_t row0 = static_cast<int64_t>(a.x + step / p.G) * kBM;
        const uint32_t q_at = base + Wide::kBuf + (step & 1) * 2 * kTile, d_at = q_at + kTile;
        const float *stats = reinterpret_cast<const float *>(smem + Wide::kStats) + (step & 1) * 2 * kBM;
        if (mine) {
#pragma unroll 1
            for (int slab = 0; slab < kBM; slab += 16) {
                float s[2][4] = {}, dp[2][4] = {};
                const int b_row = slab + (lane & 7) + ((lane >> 4) << 3), b_unit = (lane >> 3) & 1;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                    uint32_t y[4];
                    ldmatrix4(q_at + tile_at(b_row, 2 * kk + b_unit), y);
                    mma(s[0], ka[kk], y[0], y[1]);
                    mma(s[1], ka[kk], y[2], y[3]);
                    ldmatrix4(d_at + tile_at(b_row, 2 * kk + b_unit), y);
                    mma(dp[0], va[kk], y[0], y[1]);
                    mma(dp[1], va[kk], y[2], y[3]);
                }
                uint32_t P[2][4], S[2][4];  // [part]: keys x rows, as the second products' left operand
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int r = slab + 8 * n + 2 * (lane & 3);
                    const float2 l2 = *reinterpret_cast<const float2 *>(stats + r);
                    const float2 D2 = *reinterpret_cast<const float2 *>(stats + kBM + r);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int key = key0 + 8 * half;
                        float pr[2], ds[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int64_t row = row0 + r + e;
                            const bool sees = key < last && row >= a.z + key && row < c.x;
                            const float x = fmaf(s[n][2 * half + e], p.scale_log2, -(e ? l2.y : l2.x));
                            pr[e] = sees ? ex2_approx(x) : 0.f;
                            ds[e] = sees ? pr[e] * (dp[n][2 * half + e] - (e ? D2.y : D2.x)) : 0.f;
                        }
                        two_parts(pr[0], pr[1], P[0][2 * n + half], P[1][2 * n + half]);
                        two_parts(ds[0], ds[1], S[0][2 * n + half], S[1][2 * n + half]);
                    }
                }
                const int t_row = slab + (lane & 7) + (((lane >> 3) & 1) << 3), t_unit = lane >> 4;
#pragma unroll
                for (int n = 0; n < kD / 8; n += 2) {
                    uint32_t y[4];
                    ldmatrix4_t(q_at + tile_at(t_row, n + t_unit), y);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mma(dk[n + e], S[0], y[2 * e], y[2 * e + 1]);
                        mma(dk[n + e], S[1], y[2 * e], y[2 * e + 1]);
                    }
                    ldmatrix4_t(d_at + tile_at(t_row, n + t_unit), y);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mma(dv[n + e], P[0], y[2 * e], y[2 * e + 1]);
                        mma(dv[n + e], P[1], y[2 * e], y[2 * e + 1]);
                    }
                }
            }
        }
        __syncthreads();  // the buffer is read: it may be filled again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int key = key0 + 8 * half, pos = a.z % kBM + key, t = pos / kBM;
        if (!mine || key >= last)
            continue;
        const int at = t ? pos % kBM : key;
        const int64_t off = ((prob * p.slots + b.x + t * b.y) * 2 * p.rows + at) * kD + 2 * (lane & 3);
        if (!ULY_IN_BOUNDS(p.status, off, (p.rows + 1) * kD - 6, nprob * p.slots * 2 * p.rows * kD, 0x3c))
            continue;
#pragma unroll
        for (int n = 0; n < kD / 8; ++n) {
            *reinterpret_cast<float2 *>(p.part + off + 8 * n) = make_float2(dk[n][2 * half], dk[n][2 * half + 1]);
            *reinterpret_cast<float2 *>(p.part + off + p.rows * kD + 8 * n) =
                make_float2(dv[n][2 * half], dv[n][2 * half + 1]);
        }
    }
}

}  // namespace

cudaError_t launch_window_sinks(const AttnShape &s, const void *q, const void *k, const void *v, const void *dout,
                                const BwdScratch &scr, cudaStream_t stream)
{
    Params p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.dout = static_cast<const uint16_t *>(dout);
    p.lse2 = scr.lse2;
    p.Dv = scr.D;
    p.acc = scr.dq_acc;
    p.part = s.units.part;
    p.chunks = s.units.chunks;
    p.SB = s.SB;
    p.N = s.N;
    p.Npad = scr.Npad;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.G = s.Hq / s.Hkv;
    p.slots = s.units.slots;
    p.rows = s.units.rows;
    p.scale_log2 = s.scale * 1.4426950408889634f;
    p.q_elems = s.q_elems;
    p.kv_elems = s.kv_elems;
    p.status = s.status;
    const bool wide = s.sinks > kWindowSinks;
    const int groups = (s.units.sinks + kKeys - 1) / kKeys, passes = wide ? (groups + kWarps - 1) / kWarps : 1;
    p.pass = (groups + passes - 1) / passes;
    cudaError_t e = cudaFuncSetAttribute(window_sinks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kTotal);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(window_sinks_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide::kTotal);
    if (e == cudaSuccess && wide)
        e = cudaMemsetAsync(p.acc, 0, static_cast<size_t>(s.SB) * s.Hq * p.Npad * kD * sizeof(float), stream);
    if (e != cudaSuccess || s.units.n_chunks == 0)
        return e;
    const dim3 grid(static_cast<unsigned>(s.units.n_chunks * s.SB * s.Hkv), passes);
    if (wide)
        window_sinks_wide_kernel<<<grid, kThreads, Wide::kTotal, stream>>>(p);
    else
        window_sinks_kernel<<<grid, kThreads, Smem::kTotal, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace uly
