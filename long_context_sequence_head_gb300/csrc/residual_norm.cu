// What stands between two blocks of a model, in one pass over the tokens: the
// RMS norm behind a block, its gate and residual scale, the sum with the
// residual stream, and the RMS norm before the next block:
//   r2 = 1/sqrt(mean y^2 + eps),  yh = y r2,  u = w2 yh   (u = y without w2)
//   h  = x + a g u,               r1 = 1/sqrt(mean h^2 + eps),  z = w1 h r1
// and its backward, from dh and dz (hh = h r1, everything but the statistics
// formed again from x and y):
//   gz = w1 dz,  t = dh + r1 (gz - hh mean(gz hh)) = dx
//   dy = r2 (c t - yh mean(c t yh)) with c = a g w2,   or a g t without w2
//   dw1 = sum dz hh;  A = sum t yh over the rows of a gate:
//   dw2 = sum over gates a g A,  dg = a w2 A
// All arithmetic is fp32; every output is rounded once (z comes from h before
// its rounding).
//
// Both directions are bound by HBM: 4 (forward) and 6 (backward) values move
// per element, against 8 and about 20 operations.  A block takes a contiguous
// run of rows.  One warp copies them, a few rows ahead, into a ring in shared
// memory (contiguous rows: one bulk copy a tensor and stage), so that the bytes
// on their way do not depend on registers; the other warps hold a row (or
// several short ones) between them, 16 bytes a lane, each thread the same
// columns of every row, so that the columns' sums stay in registers.  The
// backward's three row sums (S1 = sum gz hh, S2 = sum c yh b, S3 = sum c yh hh
// with b = dh + r1 gz, so that sum c t yh = S2 - r1 mean(gz hh) S3) cross the
// row's warps in one exchange.
#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kMaxWarps = 16;   // of a row
constexpr int kMaxThreads = 32 * (kMaxWarps + 1);
constexpr int kMaxStages = 8;
constexpr int kJoinLanes = 8;   // slots a column's sum is spread over

// Elements of a 16-byte chunk as fp32 pairs.
template <typename T>
struct Chunk {
    static constexpr int kE = 16 / sizeof(T);
    static constexpr int kP = kE / 2;
    float2 v[kP];

    __device__ __forceinline__ void unpack(const uint4 &u)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            v[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
            v[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
        }
    }
    __device__ __forceinline__ uint4 pack() const
    {
        if constexpr (sizeof(T) == 2)
            return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                              pack_bf16x2(v[3].x, v[3].y));
        else
            return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                              __float_as_uint(v[1].y));
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The rows of a block in stages of at most p.rows rows that share a gate.
struct Stages {
    int64_t row, end, run_end;
    int64_t run;

    __device__ __forceinline__ explicit Stages(const ResidualNormParams &p)
    {
        row = p.T * blockIdx.x / gridDim.x;
        end = p.T * (blockIdx.x + 1) / gridDim.x;
        run = row / p.run;
        run_end = (run + 1) * p.run;
    }
    __device__ __forceinline__ bool more() const { return row < end; }
    __device__ __forceinline__ int count(const ResidualNormParams &p) const
    {
        const int64_t last = run_end < end ? run_end : end;
        return last - row < p.rows ? static_cast<int>(last - row) : p.rows;
    }
    // true if the next stage has another gate
    __device__ __forceinline__ bool next(const ResidualNormParams &p, int n)
    {
        row += n;
        if (row < run_end)
            return false;
        ++run;
        run_end += p.run;
        return true;
    }
};

struct Smem {
    uint64_t *full, *empty;
    volatile int *abort;
    float4 *sums;   // [groups][2][kMaxWarps]
    uint8_t *w1, *w2, *gate, *ring;

    __device__ __forceinline__ Smem(uint8_t *base, int row_bytes, int groups)
    {
        full = reinterpret_cast<uint64_t *>(base);
        empty = full + kMaxStages;
        abort = reinterpret_cast<volatile int *>(empty + kMaxStages);
        sums = reinterpret_cast<float4 *>(base + 256);
        w1 = base + 256 + groups * 2 * kMaxWarps * sizeof(float4);
        w2 = w1 + row_bytes;
        gate = w2 + row_bytes;
        ring = gate + row_bytes;
    }
};

// The copying warp: rows of n_in tensors, stage by stage.
template <int kIn>
__device__ __forceinline__ void copy_rows(const ResidualNormParams &p, const Smem &sm, const uint8_t *const *in,
                                          int row_bytes)
{
    Stages st(p);
    int k = 0;
    for (; st.more() && !*sm.abort; ++k) {
        const int slot = k % p.stages, n = st.count(p);
        if (!mbar_wait(&sm.empty[slot], ((k / p.stages) & 1) ^ 1, p.w, 0xa1)) {
            *sm.abort = 1;
            break;
        }
        uint8_t *dst = sm.ring + static_cast<size_t>(slot) * kIn * p.rows * row_bytes;
        const uint32_t bytes = static_cast<uint32_t>(n) * row_bytes;
        int tensors = 0;
#pragma unroll
        for (int t = 0; t < kIn; ++t)
            tensors += in[t] != nullptr;
        const bool ok = ULY_IN_BOUNDS(p.w.status, st.row, n, p.T, 0x51);
        mbar_expect_tx(&sm.full[slot], ok ? tensors * bytes : 0);
#pragma unroll
        for (int t = 0; t < kIn; ++t)
            if (ok && in[t] != nullptr)
                bulk_g2s(dst + static_cast<size_t>(t) * p.rows * row_bytes, in[t] + st.row * row_bytes, bytes,
                         &sm.full[slot]);
        st.next(p, n);
    }
    if (*sm.abort)  // wait (bounded) for the copies that are on their way
        for (int i = k > p.stages ? k - p.stages : 0; i < k; ++i)
            mbar_wait(&sm.full[i % p.stages], (i / p.stages) & 1, p.w, 0xaf);
}

// Sums over the lanes (and warps) that hold a row.  lanes: a power of two up
// to 32, or 32 with `warps` > 1; every thread of the row gets the same bits.
template <int kN>
struct RowSum {
    float4 *slots;
    int lanes, warps, group, parity = 0;

    __device__ __forceinline__ void operator()(float (&s)[kN])
    {
        for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kN; ++i)
                s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
        if (warps == 1)
            return;
        float4 *at = slots + parity * kMaxWarps;
        parity ^= 1;
        const int w = warp_id() - group * warps;
        if (lane_id() == 0)
            at[w] = make_float4(s[0], kN > 1 ? s[kN > 1 ? 1 : 0] : 0.f, kN > 2 ? s[kN > 2 ? 2 : 0] : 0.f, 0.f);
        named_bar_sync(1 + group, warps * 32);
        float4 total = at[0];
        for (int i = 1; i < warps; ++i) {
            const float4 o = at[i];
            total.x += o.x, total.y += o.y, total.z += o.z;
        }
        s[0] = total.x;
        if constexpr (kN > 1)
            s[1] = total.y;
        if constexpr (kN > 2)
            s[2] = total.z;
    }
};

// Copies a row of weights into shared memory (the threads that work on rows).
__device__ __forceinline__ void load_weights(uint8_t *dst, const void *src, int64_t row, int row_bytes, int threads)
{
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(src) + row * row_bytes);
    for (int i = threadIdx.x; i < row_bytes / 16; i += threads)
        reinterpret_cast<uint4 *>(dst)[i] = from[i];
}

__device__ __forceinline__ bool set_up(const Smem &sm, const ResidualNormParams &p, int threads)
{
    if (threadIdx.x == threads) {  // lane 0 of the copying warp
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], threads / 32);
        }
        *sm.abort = 0;
        fence_mbar_init();
    }
    return threadIdx.x >= threads;
}

__device__ __forceinline__ void await(const Smem &sm, const ResidualNormParams &p, int k, unsigned site)
{
    // after a wait that ran out the loop goes on without waiting: its outputs
    // are invalid and the status says so
    if (!*sm.abort && !mbar_wait(&sm.full[k % p.stages], (k / p.stages) & 1, p.w, site))
        *sm.abort = 1;
}

__device__ __forceinline__ uint4 ld_chunk(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// kC: chunks a thread holds of its row.  kPost: a norm behind the block.
// kFirst: no block before this norm (y is null).
template <typename T, int kC, bool kPost, bool kFirst>
__global__ void __launch_bounds__(kMaxThreads) residual_norm_fwd_kernel(const __grid_constant__ ResidualNormParams p)
{
    constexpr int kIn = kFirst ? 1 : 2, kP = Chunk<T>::kP;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int row_bytes = p.D * static_cast<int>(sizeof(T)), nvec = row_bytes / 16;
    const int groups = p.lanes < 32 ? 1 : p.rows;  // rows that are summed over several warps
    const Smem sm(smem_raw, row_bytes, groups);
    const int threads = static_cast<int>(blockDim.x) - 32;
    const bool copies = set_up(sm, p, threads);
    if (!copies) {
        load_weights(sm.w1, p.w1, 0, row_bytes, threads);
        if (kPost)
            load_weights(sm.w2, p.w2, 0, row_bytes, threads);
    }
    __syncthreads();
    if (copies) {
        if (lane_id() == 0) {
            const uint8_t *in[kIn];
            in[0] = static_cast<const uint8_t *>(p.x);
            if constexpr (!kFirst)
                in[1] = static_cast<const uint8_t *>(p.y);
            copy_rows<kIn>(p, sm, in, row_bytes);
        }
        return;
    }
    const int mine = threadIdx.x / p.per_row, cl = threadIdx.x % p.per_row;
    const int group = p.lanes < 32 ? 0 : mine;
    RowSum<1> sum{sm.sums + group * 2 * kMaxWarps, p.lanes, p.lanes < 32 ? 1 : p.per_row / 32, group};
    const bool gated = !kFirst && p.gate != nullptr;
    const float inv_d = 1.f / static_cast<float>(p.D);
    bool turn = true;
    Stages st(p);
    for (int k = 0; st.more(); ++k) {
        const int n = st.count(p), slot = k % p.stages;
        if (turn && gated) {  // this run's gate
            named_bar_sync(15, threads);
            load_weights(sm.gate, p.gate, p.gates > 1 ? st.run % p.gates : 0, row_bytes, threads);
            named_bar_sync(15, threads);
        }
        await(sm, p, k, 0xa2);
        const bool live = mine < n;
        const uint8_t *from = sm.ring + static_cast<size_t>(slot) * kIn * p.rows * row_bytes +
                              static_cast<size_t>(mine) * row_bytes;
        Chunk<T> x[kC], y[kFirst ? 1 : kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int at = cl + c * p.per_row;
            const bool in = live && at < nvec;
            x[c].unpack(in ? ld_chunk(from + at * 16) : make_uint4(0, 0, 0, 0));
            if constexpr (!kFirst)
                y[c].unpack(in ? ld_chunk(from + static_cast<size_t>(p.rows) * row_bytes + at * 16)
                               : make_uint4(0, 0, 0, 0));
        }
        __syncwarp();
        if (lane_id() == 0)
            mbar_arrive(&sm.empty[slot]);
        float r2 = 1.f;
        if constexpr (kPost) {
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    q = ffma2(y[c].v[e], y[c].v[e], q);
            float s[1] = {q.x + q.y};
            sum(s);
            r2 = 1.f / sqrtf(fmaf(s[0], inv_d, p.eps));
        }
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int at = cl + c * p.per_row;
            if constexpr (!kFirst) {
                const float2 f = both(p.scale * r2);
                Chunk<T> w, g;
                const bool in = at < nvec;
                if (kPost)
                    w.unpack(in ? ld_chunk(sm.w2 + at * 16) : make_uint4(0, 0, 0, 0));
                if (gated)
                    g.unpack(in ? ld_chunk(sm.gate + at * 16) : make_uint4(0, 0, 0, 0));
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    float2 u = fmul2(y[c].v[e], f);
                    if (kPost)
                        u = fmul2(u, w.v[e]);
                    x[c].v[e] = gated ? ffma2(u, g.v[e], x[c].v[e]) : fadd2(u, x[c].v[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < kP; ++e)
                q = ffma2(x[c].v[e], x[c].v[e], q);
        }
        float s[1] = {q.x + q.y};
        sum(s);
        const float r1 = 1.f / sqrtf(fmaf(s[0], inv_d, p.eps));
        if (live && ULY_IN_BOUNDS(p.w.status, st.row + mine, 1, p.T, 0x52)) {
            const int64_t row = (st.row + mine) * row_bytes;
            if (cl == 0 && p.rstd_out) {
                p.rstd_out[st.row + mine] = r1;
                p.rstd_out[p.T + st.row + mine] = r2;
            }
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int at = cl + c * p.per_row;
                if (at >= nvec)
                    continue;
                if (!kFirst && p.h)
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.h) + row + at * 16) = x[c].pack();
                Chunk<T> w;
                w.unpack(ld_chunk(sm.w1 + at * 16));
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    x[c].v[e] = fmul2(fmul2(x[c].v[e], both(r1)), w.v[e]);
                *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.z) + row + at * 16) = x[c].pack();
            }
        }
        turn = st.next(p, n);
    }
}

// kC: as above.  Up to one chunk a thread what both passes over a row need (before
// and after its sums) stays in registers; with more it is formed again from the
// stage, which is then released after the second pass.
template <typename T, int kC, bool kPost, bool kFirst>
__global__ void __launch_bounds__(kMaxThreads) residual_norm_bwd_kernel(const __grid_constant__ ResidualNormParams p)
{
    constexpr int kIn = kFirst ? 3 : 4, kP = Chunk<T>::kP, kE = Chunk<T>::kE;
    constexpr bool kHold = kC == 1;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int row_bytes = p.D * static_cast<int>(sizeof(T)), nvec = row_bytes / 16;
    const int groups = p.lanes < 32 ? 1 : p.rows;
    const Smem sm(smem_raw, row_bytes, groups);
    const int threads = static_cast<int>(blockDim.x) - 32;
    const bool copies = set_up(sm, p, threads);
    if (!copies) {
        load_weights(sm.w1, p.w1, 0, row_bytes, threads);
        if (kPost)
            load_weights(sm.w2, p.w2, 0, row_bytes, threads);
    }
    __syncthreads();
    if (copies) {
        if (lane_id() == 0) {
            const uint8_t *in[kIn];
            in[0] = static_cast<const uint8_t *>(p.x);
            in[1] = static_cast<const uint8_t *>(p.dz);
            in[2] = static_cast<const uint8_t *>(p.dh);
            if constexpr (!kFirst)
                in[3] = static_cast<const uint8_t *>(p.y);
            copy_rows<kIn>(p, sm, in, row_bytes);
        }
        return;
    }
    const int mine = threadIdx.x / p.per_row, cl = threadIdx.x % p.per_row;
    const int group = p.lanes < 32 ? 0 : mine;
    RowSum<kPost ? 3 : 1> sum{sm.sums + group * 2 * kMaxWarps, p.lanes, p.lanes < 32 ? 1 : p.per_row / 32, group};
    const bool gated = !kFirst && p.gate != nullptr;
    const bool has_dh = p.dh != nullptr;
    const float inv_d = 1.f / static_cast<float>(p.D);
    const size_t pitch = static_cast<size_t>(p.rows) * row_bytes;  // of a stage's tensors
    float2 a1[kC][kP], aA[kFirst ? 1 : kC][kP];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int e = 0; e < kP; ++e) {
            a1[c][e] = make_float2(0.f, 0.f);
            if constexpr (!kFirst)
                aA[c][e] = make_float2(0.f, 0.f);
        }
    // writes a thread's sums of its columns and takes them back to zero
    auto flush = [&](float *base, int64_t slot, [[maybe_unused]] int64_t extent, float2(*a)[kP],
                     [[maybe_unused]] unsigned site) {
        if (mine >= p.rows)  // a row of fewer lanes than a warp, and no other row beside it
            return;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int at = cl + c * p.per_row;
            const int64_t off = (slot * p.rows + mine) * p.D + static_cast<int64_t>(at) * kE;
            if (at < nvec && ULY_IN_BOUNDS(p.w.status, off, kE, extent, site))
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    *reinterpret_cast<float2 *>(base + off + 2 * e) = a[c][e];
#pragma unroll
            for (int e = 0; e < kP; ++e)
                a[c][e] = make_float2(0.f, 0.f);
        }
    };
    bool turn = true;
    Stages st(p);
    float r1 = 0.f, r2 = 0.f;  // of the next stage's row, read a stage ahead
    auto statistics = [&](const Stages &s) {
        r1 = r2 = 0.f;
        if (s.more() && mine < s.count(p) && ULY_IN_BOUNDS(p.w.status, s.row + mine, 1, p.T, 0x53)) {
            r1 = p.rstd[s.row + mine];
            r2 = kPost ? p.rstd[p.T + s.row + mine] : 1.f;
        }
    };
    statistics(st);
    for (int k = 0; st.more(); ++k) {
        const int n = st.count(p), slot = k % p.stages;
        if (turn && gated) {
            named_bar_sync(15, threads);
            load_weights(sm.gate, p.gate, p.gates > 1 ? st.run % p.gates : 0, row_bytes, threads);
            named_bar_sync(15, threads);
        }
        const int64_t row0 = st.row, run = st.run;
        const float m1 = r1, m2 = r2;
        turn = st.next(p, n);
        statistics(st);
        await(sm, p, k, 0xa3);
        const bool live = mine < n;
        const uint8_t *from = sm.ring + slot * kIn * pitch + static_cast<size_t>(mine) * row_bytes;
        // hh, yh, b = dh + r1 w1 dz and f = a g w2 (what yh has in h) of one chunk
        auto form = [&](int c, Chunk<T> &hh, Chunk<T> &yh, Chunk<T> &b, Chunk<T> &f, Chunk<T> &dz, Chunk<T> &w) {
            const int at = cl + c * p.per_row;
            const bool in = live && at < nvec;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            hh.unpack(in ? ld_chunk(from + at * 16) : zero);
            dz.unpack(in ? ld_chunk(from + pitch + at * 16) : zero);
            b.unpack(in && has_dh ? ld_chunk(from + 2 * pitch + at * 16) : zero);
            w.unpack(in ? ld_chunk(sm.w1 + at * 16) : zero);
            if constexpr (!kFirst) {
                yh.unpack(in ? ld_chunk(from + 3 * pitch + at * 16) : zero);
                Chunk<T> o;
                if (gated)
                    f.unpack(in ? ld_chunk(sm.gate + at * 16) : zero);
                if (kPost)
                    o.unpack(in ? ld_chunk(sm.w2 + at * 16) : zero);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    f.v[e] = gated ? fmul2(f.v[e], both(p.scale)) : both(p.scale);
                    if (kPost) {
                        f.v[e] = fmul2(f.v[e], o.v[e]);
                        yh.v[e] = fmul2(yh.v[e], both(m2));
                    }
                    hh.v[e] = ffma2(f.v[e], yh.v[e], hh.v[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                hh.v[e] = fmul2(hh.v[e], both(m1));
                w.v[e] = fmul2(w.v[e], dz.v[e]);
                b.v[e] = ffma2(w.v[e], both(m1), b.v[e]);
            }
        };
        Chunk<T> hh, yh, b, f, dz, gz;
        float2 q1 = make_float2(0.f, 0.f), q2 = q1, q3 = q1;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            form(c, hh, yh, b, f, dz, gz);
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                q1 = ffma2(gz.v[e], hh.v[e], q1);
                a1[c][e] = ffma2(dz.v[e], hh.v[e], a1[c][e]);
                if constexpr (kPost) {
                    const float2 fy = fmul2(f.v[e], yh.v[e]);
                    q2 = ffma2(fy, b.v[e], q2);
                    q3 = ffma2(fy, hh.v[e], q3);
                }
            }
        }
        auto release = [&]() {
            __syncwarp();
            if (lane_id() == 0)
                mbar_arrive(&sm.empty[slot]);
        };
        if (kHold)
            release();
        float s[kPost ? 3 : 1];
        s[0] = q1.x + q1.y;
        if constexpr (kPost) {
            s[1] = q2.x + q2.y;
            s[2] = q3.x + q3.y;
        }
        sum(s);
        const float k1 = m1 * (s[0] * inv_d);
        float k2 = 0.f;
        if constexpr (kPost)
            k2 = m2 * (fmaf(-k1, s[2], s[1]) * inv_d);
        const bool store = live && ULY_IN_BOUNDS(p.w.status, row0 + mine, 1, p.T, 0x54);
        const int64_t out = (row0 + mine) * row_bytes;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int at = cl + c * p.per_row;
            const bool in = store && at < nvec;
            if (!kHold)
                form(c, hh, yh, b, f, dz, gz);
            Chunk<T> t;
#pragma unroll
            for (int e = 0; e < kP; ++e)
                t.v[e] = ffma2(hh.v[e], both(-k1), b.v[e]);
            if (in)
                *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.dx) + out + at * 16) = t.pack();
            if constexpr (!kFirst) {
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    aA[c][e] = ffma2(t.v[e], yh.v[e], aA[c][e]);
                    t.v[e] = fmul2(t.v[e], f.v[e]);
                    if constexpr (kPost)
                        t.v[e] = ffma2(yh.v[e], both(-k2), fmul2(t.v[e], both(m2)));
                }
                if (in)
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.dy) + out + at * 16) = t.pack();
            }
        }
        if (!kHold)
            release();
        if constexpr (!kFirst)
            if ((turn || !st.more()) && p.partA)
                flush(p.partA, blockIdx.x + run, p.partA_elems, aA, 0x55);
    }
    if (p.part1)
        flush(p.part1, blockIdx.x, p.part1_elems, a1, 0x56);
}

// The weights' gradients from the blocks' sums, in an order that depends on the
// sizes alone: a block takes 32 columns, kJoinLanes threads a column.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinLanes) residual_norm_join_kernel(const __grid_constant__ ResidualNormParams p,
                                                                             int blocks)
{
    __shared__ float part[kJoinLanes][33];
    const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const bool in = col < p.D;
    // the sum of rows [first, last) of a buffer of D columns, for the threads with j = 0
    auto column = [&](const float *base, int64_t first, int64_t last, int64_t extent) {
        (void)extent;
        float s = 0.f;
        if (in)
            for (int64_t r = first + j; r < last; r += kJoinLanes)
                if (ULY_IN_BOUNDS(p.w.status, r * p.D + col, 1, extent, 0x57))
                    s += base[r * p.D + col];
        return s;
    };
    auto across = [&](float s) {
        part[j][lane] = s;
        __syncthreads();
        float t = part[0][lane];
#pragma unroll
        for (int i = 1; i < kJoinLanes; ++i)
            t += part[i][lane];
        __syncthreads();
        return t;
    };
    auto value = [&](const void *w, int64_t at) {
        if constexpr (sizeof(T) == 2)
            return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(w)[at]) << 16);
        else
            return static_cast<const float *>(w)[at];
    };
    auto write = [&](void *w, int64_t at, float v) {
        if (in && j == 0) {
            if constexpr (sizeof(T) == 2)
                static_cast<uint16_t *>(w)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
            else
                static_cast<float *>(w)[at] = v;
        }
    };
    if (p.dw1)
        write(p.dw1, col, across(column(p.part1, 0, static_cast<int64_t>(blocks) * p.rows, p.part1_elems)));
    if (!p.dw2 && !p.dgate)
        return;
    auto block_of = [&](int64_t row) { return ((row + 1) * blocks - 1) / p.T; };
    const int64_t runs = (p.T + p.run - 1) / p.run;
    const int gates = p.gates > 1 ? p.gates : 1;
    float dw2 = 0.f;
    for (int b = 0; b < gates; ++b) {
        float s = 0.f;
        for (int64_t run = b; run < runs; run += gates) {
            const int64_t lo = block_of(run * p.run), hi = block_of((run + 1) * p.run - 1);
            s += column(p.partA, (lo + run) * p.rows, (hi + run + 1) * p.rows, p.partA_elems);
        }
        const float A = p.scale * across(s);
        if (p.dgate && in)
            write(p.dgate, b * static_cast<int64_t>(p.D) + col, p.w2 ? A * value(p.w2, col) : A);
        if (in)
            dw2 = p.gate ? fmaf(value(p.gate, b * static_cast<int64_t>(p.D) + col), A, dw2) : dw2 + A;
    }
    if (p.dw2)
        write(p.dw2, col, dw2);
}

// How rows are laid over a block's threads.
struct Plan {
    int chunks, per_row, lanes, rows, stages, blocks, threads;
    size_t smem;
};

Plan plan_for(int64_t T, int64_t run, int row_bytes, int tensors)
{
    Plan q;
    const int nvec = row_bytes / 16;
    q.chunks = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
    const int need = (nvec + q.chunks - 1) / q.chunks;
    q.per_row = 1;
    if (need > 32)
        q.per_row = (need + 31) / 32 * 32;
    else
        while (q.per_row < need)
            q.per_row *= 2;
    q.lanes = q.per_row < 32 ? q.per_row : 32;
    // several short rows at once, as many as fill 256 threads, but no more than a gate's run holds
    q.rows = 1;
    while (q.rows * 2 * q.per_row <= 256 && q.rows * 2 <= run && (q.per_row <= 32 || q.rows < 8))
        q.rows *= 2;
    q.threads = (q.rows * q.per_row + 31) / 32 * 32 + 32;
    const int stage = tensors * q.rows * row_bytes;
    const size_t fixed = 256 + static_cast<size_t>(q.lanes < 32 ? 1 : q.rows) * 2 * kMaxWarps * sizeof(float4) +
                         3 * static_cast<size_t>(row_bytes);
    // two or three blocks an SM, and in all about 100 KB (their stages) on the way
    const int per_sm = q.threads <= 384 ? 2 : 1;
    const size_t room = (per_sm == 2 ? 110 : 220) * 1024 - fixed;
    int64_t stages = static_cast<int64_t>(room) / stage;
    q.stages = static_cast<int>(stages < 1 ? 1 : stages > kMaxStages ? kMaxStages : stages);
    while (q.stages > 2 && static_cast<int64_t>(q.stages - 1) * stage * per_sm >= 128 * 1024)
        --q.stages;
    q.smem = fixed + static_cast<size_t>(q.stages) * stage;
    const int64_t most = (T + q.rows - 1) / q.rows;
    q.blocks = static_cast<int>(std::min<int64_t>(most, static_cast<int64_t>(num_sms()) * per_sm));
    return q;
}

template <typename T, int kC>
cudaError_t launch_main(const ResidualNormParams &p, const Plan &q, bool bwd, cudaStream_t s)
{
    using Kernel = void (*)(const ResidualNormParams);
    Kernel k;
    if (bwd)
        k = !p.y ? residual_norm_bwd_kernel<T, kC, false, true>
                 : p.w2 ? residual_norm_bwd_kernel<T, kC, true, false> : residual_norm_bwd_kernel<T, kC, false, false>;
    else
        k = !p.y ? residual_norm_fwd_kernel<T, kC, false, true>
                 : p.w2 ? residual_norm_fwd_kernel<T, kC, true, false> : residual_norm_fwd_kernel<T, kC, false, false>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(q.smem));
    if (e != cudaSuccess)
        return e;
    k<<<q.blocks, q.threads, q.smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const ResidualNormParams &p, const Plan &q, bool bwd, cudaStream_t s)
{
    cudaError_t e = q.chunks == 1 ? launch_main<T, 1>(p, q, bwd, s)
                                  : q.chunks == 2 ? launch_main<T, 2>(p, q, bwd, s) : launch_main<T, 4>(p, q, bwd, s);
    if (e != cudaSuccess || !bwd || !(p.part1 || p.partA))
        return e;
    residual_norm_join_kernel<T><<<static_cast<unsigned>((p.D + 31) / 32), 32 * kJoinLanes, 0, s>>>(p, q.blocks);
    return cudaGetLastError();
}

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// Bytes of the blocks' sums: those of w1, then those of the gates' runs.
void partial_bytes(const Plan &q, int64_t T, int64_t run, int D, size_t &one, size_t &gates)
{
    const int64_t runs = (T + run - 1) / run;
    one = up(static_cast<size_t>(q.blocks) * q.rows * D * sizeof(float));
    gates = up(static_cast<size_t>(q.blocks + runs) * q.rows * D * sizeof(float));
}

}  // namespace

size_t residual_norm_workspace(int64_t T, int64_t Np, int D)
{
    // the largest of the element types, gates shared or a sequence's own, block or none before the norm
    size_t most = 0;
    for (int es = 2; es <= 4; es += 2)
        for (int shared = 0; shared < 2; ++shared)
            for (int tensors = 3; tensors <= 4; ++tensors) {
                const int64_t run = shared ? T : Np;
                size_t one, gates;
                partial_bytes(plan_for(T, run, D * es, tensors), T, run, D, one, gates);
                most = std::max(most, one + gates);
            }
    return most;
}

cudaError_t launch_residual_norm(ResidualNormParams &p, bool bwd, int esize, void *workspace, cudaStream_t s)
{
    const int tensors = (bwd ? 3 : 1) + (p.y ? 1 : 0);
    const Plan q = plan_for(p.T, p.run, p.D * esize, tensors);
    p.per_row = q.per_row;
    p.lanes = q.lanes;
    p.rows = q.rows;
    p.stages = q.stages;
    p.w = wait_cfg();
    if (bwd && workspace) {
        size_t one, gates;
        partial_bytes(q, p.T, p.run, p.D, one, gates);
        p.part1_elems = static_cast<int64_t>(one / sizeof(float));
        p.partA_elems = static_cast<int64_t>(gates / sizeof(float));
        p.part1 = p.dw1 ? static_cast<float *>(workspace) : nullptr;
        p.partA = p.dw2 || p.dgate ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + one) : nullptr;
    }
    return esize == 2 ? launch_typed<uint16_t>(p, q, bwd, s) : launch_typed<float>(p, q, bwd, s);
}

}  // namespace uly
