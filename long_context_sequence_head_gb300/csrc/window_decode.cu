// Sliding-window attention with sinks for one new token of every sequence over
// a key/value cache.
//
// The token (position len - 1) sees the cache's tokens j with len - 1 - j <
// window or j < sinks.  Token j lies in slot j while it fits; a cache of C >=
// sinks + window slots may roll: slot(j) = j for j < sinks, else sinks + (j -
// sinks) mod (C - sinks), which overwrites only what no later token sees.  A
// sequence's visible tokens form one list, sinks first; blocks take equal runs
// of it.
//
// Bound by HBM: every visible key and value is read once, 512 bytes a token and
// KV head in bf16, for 4 d operations per query head.  With up to 8 query heads
// a KV head the arithmetic (mma.sync: the operands are 16 x 16 pieces that four
// warps take independently, too small for a tcgen05 tile) stays far below the
// bytes' time.  Every warp streams its own steps of 16 tokens through a ring of
// cp.async copies, without block-wide waits, so that 2 x 4 warps an SM have up
// to 128 KB on their way.
//   S = Q K^T      (heads x tokens, heads padded to 16: rows 8.. are zero)
//   O^T += V^T P^T (d x heads): P leaves the first product in the layout that the
//                  second takes as its B operand.
// The running maximum is raised only when a score exceeds it by 2^8, as in the
// forward kernel, so most steps exchange nothing between lanes.  Slots that are
// not in the list are neither read nor multiplied.
#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kD = 128;        // bf16
constexpr int kStep = 16;      // tokens a warp takes at once
constexpr int kStages = 3;
constexpr int kRowBytes = kD * 2;
constexpr int kTileBytes = kStep * kRowBytes;  // 4 KB of K, and of V
constexpr int kHeads = 8;      // query heads of a unit, bf16
constexpr int kHeadsF32 = 4;   // fp32
constexpr float kRaise = 8.f;  // log2 units
constexpr int kSplitMax = 64;
constexpr int kClusterMax = 8;  // blocks that join their sums through shared memory

// A sequence's visible tokens: `sinks` first ones, then `n - sinks` of the window.
struct List {
    int n, sinks;   // all, and those before the window
    int plain;      // of the window's tokens, those that lie in slot = token
    int first;      // slot of the first of them
    int base, ring; // the others: sink_slots + (base + i) mod ring
    int sink_slots;

    __device__ __forceinline__ List(const WindowDecodeParams &p, int b, bool &bad)
    {
        const int64_t len = p.lens[b];
        n = sinks = plain = first = base = 0;
        ring = static_cast<int>(p.C - p.sinks);
        sink_slots = p.sinks;
        bad = len < 0 || (len > p.C && p.C < static_cast<int64_t>(p.sinks) + p.window);
        if (bad || len == 0)
            return;
        const int64_t from = len > p.window ? len - p.window : 0;
        sinks = static_cast<int>(from < p.sinks ? from : p.sinks);
        n = sinks + static_cast<int>(len - from);
        if (from < p.sinks) {
            first = static_cast<int>(from);
            plain = static_cast<int>((len < p.sinks ? len : p.sinks) - from);
        } else {
            base = static_cast<int>((from - p.sinks) % ring);
        }
    }
    __device__ __forceinline__ int slot(int t) const
    {
        if (t < sinks)
            return t;
        t -= sinks;
        if (t < plain)
            return first + t;
        t += base - plain;
        return sink_slots + (t >= ring ? t - ring : t);
    }
};

struct Unit {
    int sb, kvh, h0, heads, split;  // first query head and how many

    __device__ __forceinline__ Unit(const WindowDecodeParams &p, int heads_max)
    {
        int64_t u = blockIdx.x;
        split = static_cast<int>(u % p.splits);
        u /= p.splits;
        const int part = static_cast<int>(u % p.parts);
        u /= p.parts;
        kvh = static_cast<int>(u % p.Hkv);
        sb = static_cast<int>(u / p.Hkv);
        h0 = kvh * p.G + part * heads_max;
        heads = min(heads_max, p.G - part * heads_max);
    }
};

// ------------------------------------------------------------- results
// A block's sums (relative to m, in log2 units) go to the output, or to its
// split's part of the workspace: [sb][Hq][split] rows of d values, then m and l.
template <typename T, int D, bool kDone = false>
__device__ __forceinline__ void put(const WindowDecodeParams &p, const Unit &u, int head, int col, const float *x,
                                    int count, float m, float l)
{
    const int64_t row = static_cast<int64_t>(u.sb) * p.Hq + u.h0 + head;
    if (kDone || p.splits == 1) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        if (!ULY_IN_BOUNDS(p.status, row * D + col, count, p.SB * p.Hq * D, 0x71))
            return;
        for (int i = 0; i < count; i += 2) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + row * D + col + i) =
                    pack_bf16x2(x[i] * inv, x[i + 1] * inv);
            else
                *reinterpret_cast<float2 *>(static_cast<float *>(p.o) + row * D + col + i) =
                    make_float2(x[i] * inv, x[i + 1] * inv);
        }
        if (col == 0)
            p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
        return;
    }
    const int64_t at = row * p.splits + u.split;
    if (!ULY_IN_BOUNDS(p.status, at * D + col, count, p.SB * p.Hq * p.splits * D, 0x72))
        return;
    for (int i = 0; i < count; i += 2)
        *reinterpret_cast<float2 *>(p.part + at * D + col + i) = make_float2(x[i], x[i + 1]);
    if (col == 0)
        *reinterpret_cast<float2 *>(p.stats + 2 * at) = make_float2(m, l);
}

// One warp a (sequence, query head): the splits' sums, in order.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_combine_kernel(const __grid_constant__ WindowDecodeParams p)
{
    grid_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp_id();
    if (row >= p.SB * p.Hq)
        return;
    const int lane = lane_id();
    float2 ml[kSplitMax / 32];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSplitMax / 32; ++i) {
        const int s = lane + 32 * i;
        ml[i] = s < p.splits ? *reinterpret_cast<const float2 *>(p.stats + 2 * (row * p.splits + s))
                             : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, f[kSplitMax / 32];
#pragma unroll
    for (int i = 0; i < kSplitMax / 32; ++i) {
        f[i] = exp2f(ml[i].x - ref);
        l = fmaf(ml[i].y, f[i], l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, o);
    float acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        acc[e] = 0.f;
    for (int s = 0; s < p.splits; ++s) {
        const float w = __shfl_sync(0xffffffffu, s < 32 ? f[0] : f[1], s & 31);
#pragma unroll
        for (int e = 0; e < D / 32; e += 2) {
            const float2 x =
                *reinterpret_cast<const float2 *>(p.part + (row * p.splits + s) * D + lane * (D / 32) + e);
            acc[e] = fmaf(w, x.x, acc[e]);
            acc[e + 1] = fmaf(w, x.y, acc[e + 1]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if (!ULY_IN_BOUNDS(p.status, row * D + lane * (D / 32), D / 32, p.SB * p.Hq * D, 0x73))
        return;
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
        const int64_t at = row * D + lane * (D / 32) + e;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + at) =
                pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        else
            *reinterpret_cast<float2 *>(static_cast<float *>(p.o) + at) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    }
    if (lane == 0)
        p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

// ---------------------------------------------------------------- bf16
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b: a 16 x 16 (rows lane/4, +8), b 16 x 8 (columns lane/4), c 16 x 8
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-byte unit `unit` of row `r` of a 16-row tile, spread over the banks.
__device__ __forceinline__ uint32_t tile_at(int r, int unit) { return r * kRowBytes + ((unit ^ (r & 7)) << 4); }

// Reads of another block's shared memory (a shared::cluster address).
__device__ __forceinline__ float2 ld_cluster(uint32_t at)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// kCluster: the blocks of a unit are one cluster, which joins their sums through
// shared memory; otherwise they go through the workspace.
template <bool kCluster>
__global__ void __launch_bounds__(kThreads, 2) window_decode_bf16_kernel(const __grid_constant__ WindowDecodeParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = warp_id(), lane = lane_id();
    const Unit u(p, kHeads);
    bool bad;
    const List list(p, u.sb % p.B, bad);
    if (bad && threadIdx.x == 0 && u.split == 0)
        atomicOr(p.status, kDevBadArg);
    // this block's steps of 16 tokens; its warps take every kWarps-th
    const int steps = (list.n + kStep - 1) / kStep;
    const int step0 = static_cast<int>(static_cast<int64_t>(steps) * u.split / p.splits);
    const int step1 = static_cast<int>(static_cast<int64_t>(steps) * (u.split + 1) / p.splits);
    uint8_t *ring = smem + warp * kStages * 2 * kTileBytes;
    const int64_t pitch = static_cast<int64_t>(p.Hkv) * kD;  // from a token to the next
    const int64_t origin = static_cast<int64_t>(u.sb) * p.C * pitch + u.kvh * kD;
    auto load = [&](int i, int stage) {  // the warp's i-th step
        const int step = step0 + warp + i * kWarps;
        if (step < step1) {
            const uint32_t k_at = smem_u32(ring + stage * 2 * kTileBytes), v_at = k_at + kTileBytes;
#pragma unroll
            for (int j = 0; j < kStep / 2; ++j) {  // two tokens an instruction, 16 lanes each
                const int r = 2 * j + (lane >> 4), unit = lane & 15, t = step * kStep + r;
                const bool in = t < list.n;
                const int64_t off = origin + (in ? list.slot(t) : 0) * pitch + unit * 8;
                const bool ok = in && ULY_IN_BOUNDS(p.status, off, 8, p.SB * p.C * pitch, 0x74);
                cp_async16(k_at + tile_at(r, unit), static_cast<const uint16_t *>(p.k) + (ok ? off : 0), ok);
                cp_async16(v_at + tile_at(r, unit), static_cast<const uint16_t *>(p.v) + (ok ? off : 0), ok);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        load(i, i);
    // Q's rows as the A operand: head lane/4 (rows 8.. are zero), columns 16 kk + 2 (lane%4) and + 8
    uint32_t q0[kD / 16], q2[kD / 16];
    {
        const int head = lane >> 2;
        const int64_t row = (static_cast<int64_t>(u.sb) * p.Hq + u.h0 + (head < u.heads ? head : 0)) * kD;
        const bool ok = ULY_IN_BOUNDS(p.status, row, kD, p.SB * p.Hq * kD, 0x75);
        const uint32_t *q = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.q) + row) + (lane & 3);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
            q0[kk] = ok && head < u.heads ? q[8 * kk] : 0u;
            q2[kk] = ok && head < u.heads ? q[8 * kk + 4] : 0u;
        }
    }
    float o[kD / 16][4];  // O^T: rows 16 i + lane/4 (+8) of d, heads 2 (lane%4) + {0, 1}
#pragma unroll
    for (int i = 0; i < kD / 16; ++i)
        o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m = -INFINITY, l = 0.f;  // of head lane/4: maximum; this lane's share of the sum
    const int mine = step1 - step0 > warp ? (step1 - step0 - warp + kWarps - 1) / kWarps : 0;
    int stage = 0;
    for (int i = 0; i < mine; ++i) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        load(i + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        const uint32_t k_at = smem_u32(ring + stage * 2 * kTileBytes), v_at = k_at + kTileBytes;
        float s[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
            // matrices: tokens 0-7 and 8-15 of columns 16 kk .. and 16 kk + 8 ..
            uint32_t b[4];
            ldmatrix4(k_at + tile_at((lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)), b);
            mma16816(s[0], q0[kk], 0u, q2[kk], 0u, b[0], b[1]);
            mma16816(s[1], q0[kk], 0u, q2[kk], 0u, b[2], b[3]);
        }
        const int t0 = (step0 + warp + i * kWarps) * kStep + 2 * (lane & 3);
        float x[4] = {s[0][0] * p.scale_log2, s[0][1] * p.scale_log2, s[1][0] * p.scale_log2, s[1][1] * p.scale_log2};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t0 + (e >> 1) * 8 + (e & 1) >= list.n)
                x[e] = -INFINITY;
        const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(0xffffffffu, top > m + kRaise || (m == -INFINITY && top > m))) {
            float raised = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            raised = fmaxf(raised, __shfl_xor_sync(0xffffffffu, raised, 2));
            raised = fmaxf(raised, m);
            const float f = raised == -INFINITY ? 1.f : exp2f(m - raised);
            m = raised;
            l *= f;
            const float f0 = __shfl_sync(0xffffffffu, f, (lane & 3) * 8), f1 = __shfl_sync(0xffffffffu, f, (lane & 3) * 8 + 4);
#pragma unroll
            for (int j = 0; j < kD / 16; ++j) {
                o[j][0] *= f0, o[j][2] *= f0;
                o[j][1] *= f1, o[j][3] *= f1;
            }
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = ex2_approx(x[e] - ref);
            l += x[e];
        }
        const uint32_t p0 = pack_bf16x2(x[0], x[1]), p1 = pack_bf16x2(x[2], x[3]);
#pragma unroll
        for (int j = 0; j < kD / 16; ++j) {
            // V^T: rows d 16 j .. and + 8, columns tokens 0-7 and 8-15
            uint32_t a[4];
            ldmatrix4_t(v_at + tile_at((lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)), a);
            mma16816(o[j], a[0], a[1], a[2], a[3], p0, p1);
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    if constexpr (!kCluster)
        grid_next();
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    __syncthreads();
    // the warps' sums, brought to the block's maximum: [warp][head][d], then m and l
    float *sums = reinterpret_cast<float *>(smem);
    constexpr int kPitch = kD + 4;
    float2 *stats = reinterpret_cast<float2 *>(sums + kWarps * kHeads * kPitch);
    if ((lane & 3) == 0)
        stats[warp * kHeads + (lane >> 2)] = make_float2(m, l);
#pragma unroll
    for (int j = 0; j < kD / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sums[(warp * kHeads + 2 * (lane & 3) + (e & 1)) * kPitch + 16 * j + (lane >> 2) + (e >> 1) * 8] = o[j][e];
    __syncthreads();
    const int head = threadIdx.x / 16, col = threadIdx.x % 16 * 8;
    if (!kCluster && head >= u.heads)
        return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        top = fmaxf(top, stats[w * kHeads + head].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f, x[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float2 ml = stats[w * kHeads + head];
        const float f = exp2f(ml.x - ref);
        total = fmaf(ml.y, f, total);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = fmaf(sums[(w * kHeads + head) * kPitch + col + e], f, x[e]);
    }
    if constexpr (kCluster) {
        // this block's sums for the others, behind what its own threads still read;
        // then every block writes its share of the output, from all of theirs
        float *mine = reinterpret_cast<float *>(stats + kWarps * kHeads);
        float2 *mine_stats = reinterpret_cast<float2 *>(mine + kHeads * kD);
        *reinterpret_cast<float4 *>(mine + head * kD + col) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(mine + head * kD + col + 4) = make_float4(x[4], x[5], x[6], x[7]);
        if (col == 0)
            mine_stats[head] = make_float2(top, total);
        cluster_sync_all();
        for (int i = u.split * kThreads + static_cast<int>(threadIdx.x); i < u.heads * (kD / 2);
             i += p.splits * kThreads) {
            const int h = i / (kD / 2), at = i % (kD / 2) * 2;
            float2 ml[kClusterMax], v[kClusterMax];
            float most = -INFINITY;
#pragma unroll
            for (int b = 0; b < kClusterMax; ++b) {
                ml[b] = make_float2(-INFINITY, 0.f);
                v[b] = make_float2(0.f, 0.f);
                if (b < p.splits) {
                    ml[b] = ld_cluster(cluster_addr(mine_stats + h, b));
                    v[b] = ld_cluster(cluster_addr(mine + h * kD + at, b));
                }
            }
#pragma unroll
            for (int b = 0; b < kClusterMax; ++b)
                most = fmaxf(most, ml[b].x);
            const float against = most == -INFINITY ? 0.f : most;
            float sum = 0.f, y[2] = {};
#pragma unroll
            for (int b = 0; b < kClusterMax; ++b) {
                const float f = exp2f(ml[b].x - against);
                sum = fmaf(ml[b].y, f, sum);
                y[0] = fmaf(v[b].x, f, y[0]);
                y[1] = fmaf(v[b].y, f, y[1]);
            }
            put<uint16_t, kD, true>(p, u, h, at, y, 2, most, sum);
        }
        cluster_sync_all();  // no block's memory goes while another reads it
    } else {
        put<uint16_t, kD>(p, u, head, col, x, 8, top, total);
    }
}

// ---------------------------------------------------------------- fp32
// Eight lanes a token, so that a warp takes four tokens at once; every group of
// eight keeps maximum, sum and output of its own tokens for up to four heads,
// and the block joins its 16 groups at the end.
template <int D>
__global__ void __launch_bounds__(kThreads) window_decode_f32_kernel(const __grid_constant__ WindowDecodeParams p)
{
    constexpr int kE = D / 8, kGroups = kThreads / 8;
    __shared__ __align__(16) float sums[kGroups][D];
    __shared__ float2 stats[kHeadsF32][kGroups];
    const int group = threadIdx.x / 8, lane = threadIdx.x % 8;
    const Unit u(p, kHeadsF32);
    bool bad;
    const List list(p, u.sb % p.B, bad);
    if (bad && threadIdx.x == 0 && u.split == 0)
        atomicOr(p.status, kDevBadArg);
    const int t1 = static_cast<int>(static_cast<int64_t>(list.n) * (u.split + 1) / p.splits);
    const int t0 = static_cast<int>(static_cast<int64_t>(list.n) * u.split / p.splits);
    const int64_t pitch = static_cast<int64_t>(p.Hkv) * D;
    const int64_t origin = static_cast<int64_t>(u.sb) * p.C * pitch + u.kvh * D;
    float q[kHeadsF32][kE], o[kHeadsF32][kE], m[kHeadsF32], l[kHeadsF32];
#pragma unroll
    for (int h = 0; h < kHeadsF32; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        const int64_t row = (static_cast<int64_t>(u.sb) * p.Hq + u.h0 + (h < u.heads ? h : 0)) * D;
        const bool ok = ULY_IN_BOUNDS(p.status, row, D, p.SB * p.Hq * D, 0x76);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            q[h][e] = ok ? static_cast<const float *>(p.q)[row + (e / 4) * 32 + lane * 4 + e % 4] : 0.f;
            o[h][e] = 0.f;
        }
    }
    // every lane of a warp goes round as often, so that all of them meet in the shuffles
    for (int t = t0 + group; t - group < t1; t += kGroups) {
        const bool in = t < t1;
        const int64_t off = origin + (in ? list.slot(t) : 0) * pitch + lane * 4;
        const bool ok = in && ULY_IN_BOUNDS(p.status, off, D - 28, p.SB * p.C * pitch, 0x77);
        float k[kE], v[kE];
#pragma unroll
        for (int e = 0; e < kE; e += 4) {
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 a = ok ? *reinterpret_cast<const float4 *>(static_cast<const float *>(p.k) + off + 8 * e) : zero;
            const float4 b = ok ? *reinterpret_cast<const float4 *>(static_cast<const float *>(p.v) + off + 8 * e) : zero;
            k[e] = a.x, k[e + 1] = a.y, k[e + 2] = a.z, k[e + 3] = a.w;
            v[e] = b.x, v[e + 1] = b.y, v[e + 2] = b.z, v[e + 3] = b.w;
        }
#pragma unroll
        for (int h = 0; h < kHeadsF32; ++h) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e)
                s = fmaf(q[h][e], k[e], s);
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            if (!in)
                continue;
            s *= p.scale_log2;
            const float top = fmaxf(m[h], s);
            const float f = exp2f(m[h] - top), w = exp2f(s - top);
            m[h] = top;
            l[h] = fmaf(l[h], f, w);
#pragma unroll
            for (int e = 0; e < kE; ++e)
                o[h][e] = fmaf(w, v[e], o[h][e] * f);
        }
    }
    grid_next();
#pragma unroll
    for (int h = 0; h < kHeadsF32; ++h)
        if (lane == 0)
            stats[h][group] = make_float2(m[h], l[h]);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeadsF32; ++h) {
        float top = -INFINITY, total = 0.f;
        for (int g = 0; g < kGroups; ++g)
            top = fmaxf(top, stats[h][g].x);
        const float ref = top == -INFINITY ? 0.f : top;
        for (int g = 0; g < kGroups; ++g)
            total = fmaf(stats[h][g].y, exp2f(stats[h][g].x - ref), total);
        const float f = exp2f(m[h] - ref);
#pragma unroll
        for (int e = 0; e < kE; ++e)
            sums[group][(e / 4) * 32 + lane * 4 + e % 4] = o[h][e] * f;
        __syncthreads();
        if (h < u.heads && threadIdx.x < D / 2) {
            float x[2] = {};
            for (int g = 0; g < kGroups; ++g) {
                x[0] += sums[g][2 * threadIdx.x];
                x[1] += sums[g][2 * threadIdx.x + 1];
            }
            put<float, D>(p, u, h, 2 * static_cast<int>(threadIdx.x), x, 2, top, total);
        }
        __syncthreads();
    }
}

// Blocks a (sequence, KV head, group of query heads) is spread over, and whether
// they are a cluster, which joins their sums without a second launch.  Two blocks
// fit an SM; a block's start and end cost about as much as 200 tokens, the second
// launch as 250.  64 units of 1,028 tokens: 9.5 us as clusters of 4 (256 blocks, one
// wave), 12.9 of 8, 18.3 with one block each; 256 units of 4,100: 78 us with one
// block each, 87 to 110 as clusters of 2 to 8.
struct Spread {
    int splits;
    bool cluster;
};

Spread spread_for(int64_t units, int64_t C, int64_t window, int64_t sinks, int esize)
{
    const int64_t keys = std::min(C, sinks + window), room = 2 * num_sms();
    const int64_t most = std::min<int64_t>(kSplitMax, (keys + kWarps * kStep - 1) / (kWarps * kStep));
    Spread best{1, false};
    int64_t least = 0;
    for (int n = 1; n <= most; ++n) {
        const bool cluster = esize == 2 && n > 1 && n <= kClusterMax;
        const int64_t cost = (units * n + room - 1) / room * ((keys + n - 1) / n + 200) + (n > 1 && !cluster ? 250 : 0);
        if (n == 1 || cost < least) {
            least = cost;
            best = Spread{n, cluster};
        }
    }
    return best;
}

int parts_of(int G, int esize) { return esize == 2 ? (G + kHeads - 1) / kHeads : (G + kHeadsF32 - 1) / kHeadsF32; }

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

}  // namespace

size_t window_decode_workspace(int64_t SB, int64_t C, int Hq, int Hkv, int d, int64_t window, int64_t sinks, int esize)
{
    const Spread n = spread_for(SB * Hkv * parts_of(Hq / Hkv, esize), C, window, sinks, esize);
    const size_t rows = static_cast<size_t>(SB) * Hq * n.splits;
    return n.splits == 1 || n.cluster ? kAlign : up(rows * d * sizeof(float)) + up(rows * 2 * sizeof(float));
}

cudaError_t launch_window_decode(WindowDecodeParams &p, int d, int esize, void *workspace, cudaStream_t s)
{
    p.G = p.Hq / p.Hkv;
    p.parts = parts_of(p.G, esize);
    const Spread spread = spread_for(p.SB * p.Hkv * p.parts, p.C, p.window, p.sinks, esize);
    p.splits = spread.splits;
    const size_t rows = static_cast<size_t>(p.SB) * p.Hq * p.splits;
    p.part = static_cast<float *>(workspace);
    p.stats = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + up(rows * d * sizeof(float)));
    const int64_t grid = p.SB * p.Hkv * p.parts * p.splits;
    cudaError_t e;
    if (esize == 2) {
        constexpr size_t smem = static_cast<size_t>(kWarps) * kStages * 2 * kTileBytes;
        static_assert(smem >= kHeads * (kWarps * ((kD + 4) * sizeof(float) + sizeof(float2)) + kD * sizeof(float) +
                                        sizeof(float2)),
                      "the joined sums fit");
        auto kernel = spread.cluster ? window_decode_bf16_kernel<true> : window_decode_bf16_kernel<false>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess)
            return e;
        if (spread.cluster) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(grid));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = smem;
            cfg.stream = s;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            return cudaLaunchKernelEx(&cfg, kernel, p);
        }
        kernel<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(p);
    } else if (d == 64) {
        window_decode_f32_kernel<64><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    } else {
        window_decode_f32_kernel<128><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1)
        return e;
    const int64_t blocks = (p.SB * p.Hq + kWarps - 1) / kWarps;
    return esize == 2 ? launch_after(window_combine_kernel<uint16_t, 128>, blocks, kThreads, 0, s, p)
           : d == 64  ? launch_after(window_combine_kernel<float, 64>, blocks, kThreads, 0, s, p)
                      : launch_after(window_combine_kernel<float, 128>, blocks, kThreads, 0, s, p);
}

}  // namespace uly
