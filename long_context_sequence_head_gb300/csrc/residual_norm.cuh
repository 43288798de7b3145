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
// per element, against 8 and about 20 operations.  Rows come in slots of one long
// row or several short ones (contiguous, one bulk copy a tensor); a block takes every
// gridDim-th slot, or a contiguous run of rows where every sequence has a gate of its
// own.  One warp copies slots into a ring in shared memory, so that the bytes on their
// way do not depend on registers; groups of one or more warps, each with slots of its
// own, take a row at a time, a thread 16 bytes by 16 bytes of the same columns of
// every row, so that the columns' sums stay in registers.  Few warps a row and several
// rows at once: ten warps on one row of 2560 spent most of their time in its sums
// (64K rows: forward 455 us, backward 642; now 203 and 300, HBM's time for the bytes
// 198 and 297).
//   The backward's three row sums (S1 = sum gz hh, S2 = sum c yh b, S3 = sum c yh hh
// with b = dh + r1 gz, so that sum c t yh = S2 - r1 mean(gz hh) S3) cross a group's
// warps in one exchange; what both passes over a row need is formed again from the
// slot, which costs less than the registers to hold it.
#pragma once

#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kMaxWarps = 15;   // that work on rows; with the copying one 16, which have 128 registers a thread
constexpr int kMaxThreads = 32 * (kMaxWarps + 1);
constexpr int kMaxSlots = 32;
constexpr int kMaxRows = 32;    // of a slot
constexpr int kJoinLanes = 16;  // blocks a column's sum is spread over

// Shared memory by 32-bit addresses: pointers to it would take 64 bits of the
// registers that the columns' sums need.
__device__ __forceinline__ uint4 ld_shared(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint64_t *barrier_at(uint32_t at)
{
    return static_cast<uint64_t *>(__cvta_shared_to_generic(at));
}

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
    // fp32 values in shared memory
    __device__ __forceinline__ void read(uint32_t at)
    {
#pragma unroll
        for (int i = 0; i < kP; i += 2) {
            const uint4 f = ld_shared(at + 8 * i);
            v[i] = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
            v[i + 1] = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
        }
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The rows of a block in slots of at most p.slot_rows rows.  Where all rows share
// one gate, the blocks' slots alternate, so that all of them work on neighbouring
// memory; with a gate for every sequence a block takes a run of rows, in slots
// that share one.
struct Slots {
    uint32_t row, end, run_end, step;  // fewer than 2^31 rows
    uint32_t run;

    __device__ __forceinline__ explicit Slots(const ResidualNormParams &p)
    {
        if (p.gates > 1) {
            row = blockIdx.x * p.block_rows;
            end = min(row + p.block_rows, static_cast<uint32_t>(p.T));
            run = row / static_cast<uint32_t>(p.run);
            run_end = (run + 1) * static_cast<uint32_t>(p.run);
        } else {
            row = blockIdx.x * p.slot_rows;
            end = run_end = static_cast<uint32_t>(p.T);
            run = 0;
        }
        step = gridDim.x * p.slot_rows;
    }
    __device__ __forceinline__ bool more() const { return row < end; }
    __device__ __forceinline__ int count(const ResidualNormParams &p) const
    {
        return static_cast<int>(min(min(run_end, end) - row, static_cast<uint32_t>(p.slot_rows)));
    }
    // the next slot (with one gate: the block's n-th from here); true if it has another gate
    __device__ __forceinline__ bool next(const ResidualNormParams &p, int rows, int n = 1)
    {
        if (p.gates <= 1) {
            row += n * step;  // below 2^31 + 15 * 152 * 32
            return false;
        }
        row += rows;
        if (row < run_end)
            return false;
        ++run;
        run_end += static_cast<uint32_t>(p.run);
        return true;
    }
};

// Shared memory (addresses): barriers, the groups' sums, the slots' statistics, w1
// as given, f = residual_scale * gate * post_weight in fp32, the ring.
struct Smem {
    uint32_t full, empty;  // [kMaxSlots] each
    uint32_t abort;
    uint32_t sums;         // [groups][2][warps] of 16 bytes
    uint32_t stats;        // backward: [slots][2][kMaxRows]
    uint32_t w1;
    uint32_t f;
    uint32_t scratch;      // backward: [parts][D], the sums on their way out of a block
    uint32_t ring;

    static constexpr int kHead = 16 * kMaxSlots + 128;
    static __host__ __device__ size_t fixed(int D, int row_bytes, int parts, int stat_slots)
    {
        return kHead + static_cast<size_t>(2) * kMaxWarps * 16 +
               static_cast<size_t>(stat_slots) * 2 * kMaxRows * sizeof(float) + row_bytes +
               static_cast<size_t>(1 + parts) * D * 4;
    }
    __device__ __forceinline__ Smem(const void *base, const ResidualNormParams &p, int row_bytes)
    {
        full = smem_u32(base);
        empty = full + 8 * kMaxSlots;
        abort = empty + 8 * kMaxSlots;
        sums = full + kHead;
        stats = sums + 2 * kMaxWarps * 16;
        w1 = stats + (p.rstd ? p.slots * 2 * kMaxRows * 4 : 0);
        f = w1 + row_bytes;
        scratch = f + p.D * 4;
        ring = scratch + p.parts * p.D * 4;
    }
    __device__ __forceinline__ bool aborted() const { return ld_shared_f32(abort) != 0.f; }
    __device__ __forceinline__ void set_aborted(bool on) const
    {
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(abort), "f"(on ? 1.f : 0.f) : "memory");
    }
};

__device__ __forceinline__ bool phase_done(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The copying warp, which starts before the block meets: slots of kIn tensors' rows
// (some may be null); kStats: with each row's two statistics, by 4-byte copies that
// arrive on the same barrier.  A lane copies for a group: one lane for all of them
// took 0.3 us a slot, 71 us for 32,768 rows of 512 that now take 29 (2 x 3,021 of 776
// backward: 34, now 27).  Slots are filled in order: whichever was free first made 64K
// rows of 2560 take 217 us instead of 207.
template <int kIn, bool kStats>
__device__ __forceinline__ void copy_rows(const ResidualNormParams &p, const Smem &sm, const uint8_t *const *in,
                                          int row_bytes)
{
    const int lane = lane_id();
    // Every group has slots of its own: one that others fill in turn would let a
    // group see the parity of a copy two phases back as its own.
    const int own = p.slots / p.groups;
    Slots st(p);
    auto skip = [&](int n) {
        if (p.gates <= 1)
            st.next(p, 0, n);
        else
            for (int i = 0; i < n && st.more(); ++i)
                st.next(p, st.count(p));
    };
    int tensors = 0;
#pragma unroll
    for (int t = 0; t < kIn; ++t)
        tensors += in[t] != nullptr;
    int turns = 0, at = 0;
    uint32_t phase = 0;
    auto copy = [&]() {  // the group's next slot
        const int slot = lane * own + at, n = st.count(p);
        const uint32_t full = sm.full + 8 * slot;
        const bool ok = ULY_IN_BOUNDS(p.w.status, st.row, n, p.T, 0x51);
        const uint32_t dst = sm.ring + slot * kIn * p.slot_rows * row_bytes;
        const uint32_t bytes = static_cast<uint32_t>(n) * row_bytes;
        mbar_expect_tx(barrier_at(full), ok ? tensors * bytes : 0);
#pragma unroll
        for (int t = 0; t < kIn; ++t)
            if (ok && in[t] != nullptr)
                bulk_g2s(__cvta_shared_to_generic(dst + t * p.slot_rows * row_bytes),
                         in[t] + static_cast<int64_t>(st.row) * row_bytes, bytes, barrier_at(full));
        if (kStats) {
            const uint32_t to = sm.stats + slot * 2 * kMaxRows * 4;
            for (int r = 0; ok && r < n; ++r) {
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + r * 4), "l"(p.rstd + st.row + r)
                             : "memory");
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + (kMaxRows + r) * 4),
                             "l"(p.rstd + p.T + st.row + r)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(full) : "memory");
        }
        ++turns;
        if (++at == own) {
            at = 0;
            phase ^= 1;
        }
        skip(p.groups);
    };
    bool todo = false;
    if (lane < p.groups) {
        skip(lane);
        if (st.more())
            copy();
        todo = st.more();
    }
    __syncwarp();
    __syncthreads();  // no more until the weights are there
    int idle = 0, next = 0;  // the group whose slot comes next
    uint64_t since = 0;
    while (__any_sync(0xffffffffu, todo)) {
        const bool ready = todo && phase_done(barrier_at(sm.empty + 8 * (lane * own + at)), phase ^ 1);
        const uint32_t free = __ballot_sync(0xffffffffu, ready);
        const int run = __ffs(~(free >> next | free << (p.groups - next))) - 1;  // in order
        const int count = min(run, p.groups);
        if (lane < p.groups && (lane >= next ? lane - next : lane - next + p.groups) < count) {
            copy();
            todo = st.more();
        }
        if (count > 0) {
            next = next + count < p.groups ? next + count : next + count - p.groups;
            idle = 0;
            continue;
        }
        if (++idle % 64 != 0)
            continue;
        bool stop = sm.aborted();
        if (idle == 64) {
            since = globaltimer_ns();
        } else if (!stop && globaltimer_ns() - since > p.w.limit_ns) {
            stop = true;
            if (lane == 0)
                record_timeout(p.w, 0xa1);
        }
        if (__any_sync(0xffffffffu, stop)) {
            sm.set_aborted(true);
            break;
        }
    }
    __syncwarp();
    if (sm.aborted())  // wait (bounded) for the copies that are on their way
        for (int i = turns > own ? turns - own : 0; i < turns; ++i)
            mbar_wait(barrier_at(sm.full + 8 * (lane * own + i % own)), (i / own) & 1, p.w, 0xaf);
}

// Sums over the lanes (and the group's warps) that hold a row.  lanes: a power of
// two up to 32; every thread of the row gets the same bits.
template <int kN>
struct RowSum {
    uint32_t slots;  // shared memory, [2][warps]
    int lanes, warps, group, warp, parity = 0;

    __device__ __forceinline__ void operator()(float (&s)[kN])
    {
        for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kN; ++i)
                s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
        if (warps == 1)
            return;
        const uint32_t at = slots + parity * warps * 16;
        parity ^= 1;
        if (lane_id() == 0)
            st_shared(at + warp * 16, make_uint4(__float_as_uint(s[0]), __float_as_uint(s[kN > 1 ? 1 : 0]),
                                                 __float_as_uint(s[kN > 2 ? 2 : 0]), 0u));
        named_bar_sync(1 + group, warps * 32);
        float4 total = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < warps; i += 5) {  // five loads on their way at once
            uint4 o[5];
#pragma unroll
            for (int j = 0; j < 5; ++j)
                o[j] = i + j < warps ? ld_shared(at + (i + j) * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                total.x += __uint_as_float(o[j].x);
                total.y += __uint_as_float(o[j].y);
                total.z += __uint_as_float(o[j].z);
            }
        }
        s[0] = total.x;
        if constexpr (kN > 1)
            s[1] = total.y;
        if constexpr (kN > 2)
            s[2] = total.z;
    }
};

// The threads that work on rows: which rows, which columns, and what they share.
template <typename T, int kIn, int kSums>
struct Worker {
    const ResidualNormParams &p;
    const Smem &sm;
    int threads, row_bytes, nvec;
    int group, sub, col, width;  // group of warps, row of those its warp holds at once, first chunk, chunks from one to the next
    RowSum<kSums> sum;

    __device__ __forceinline__ Worker(const ResidualNormParams &p_, const Smem &sm_, int threads_)
        : p(p_), sm(sm_), threads(threads_), row_bytes(p_.D * static_cast<int>(sizeof(T))), nvec(row_bytes / 16)
    {
        group = warp_id() / p.warps;
        const int warp = warp_id() - group * p.warps;
        sub = lane_id() / p.lanes;
        col = p.lanes < 32 ? lane_id() % p.lanes : warp * 32 + lane_id();
        width = p.lanes < 32 ? p.lanes : p.warps * 32;
        sum.slots = sm.sums + group * 2 * p.warps * 16;
        sum.lanes = p.lanes;
        sum.warps = p.warps;
        sum.group = group;
        sum.warp = warp;
    }
    // f for the rows of a run, and w1 with it at the start
    template <bool kStart>
    __device__ __forceinline__ void load_f(uint32_t run) const
    {
        const T *gate = static_cast<const T *>(p.gate), *w2 = static_cast<const T *>(p.w2);
        if (gate && p.gates > 1)
            gate += static_cast<int64_t>(run % p.gates) * p.D;
        for (int i = threadIdx.x; i < nvec; i += threads) {
            uint4 raw[3];  // on their way together
            if (kStart)
                raw[0] = static_cast<const uint4 *>(p.w1)[i];
            if (gate)
                raw[1] = reinterpret_cast<const uint4 *>(gate)[i];
            if (w2)
                raw[2] = reinterpret_cast<const uint4 *>(w2)[i];
            if (kStart)
                st_shared(sm.w1 + 16 * i, raw[0]);
            Chunk<T> f, w;
#pragma unroll
            for (int e = 0; e < Chunk<T>::kP; ++e)
                f.v[e] = both(p.scale);
#pragma unroll
            for (int k = 1; k < 3; ++k) {
                if (k == 1 ? gate == nullptr : w2 == nullptr)
                    continue;
                w.unpack(raw[k]);
#pragma unroll
                for (int e = 0; e < Chunk<T>::kP; ++e)
                    f.v[e] = fmul2(f.v[e], w.v[e]);
            }
#pragma unroll
            for (int e = 0; e < Chunk<T>::kP; ++e)
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sm.f + (i * Chunk<T>::kE + 2 * e) * 4),
                             "f"(f.v[e].x), "f"(f.v[e].y)
                             : "memory");
        }
    }
    // Goes through the block's slots: body(first row, row in slot, live, slot memory,
    // slot number) for the rows of this group's, end_of_run(run) for every thread.
    template <bool kSub, bool kGated, typename Body, typename EndOfRun>
    __device__ __forceinline__ void go(unsigned site, Body body, EndOfRun end_of_run)
    {
        Slots st(p);
        const int pitch = p.slot_rows * row_bytes;
        auto rows_of = [&](int slot, uint32_t phase, uint32_t row0, int n) {
            // after a wait that ran out the loop goes on without waiting: its outputs
            // are invalid and the status says so
            if (!sm.aborted() && !mbar_wait(barrier_at(sm.full + 8 * slot), phase, p.w, site))
                sm.set_aborted(true);
            const uint32_t at = sm.ring + slot * kIn * pitch;
            if constexpr (kSub) {
                for (int r = 0; r < n; r += 32 / p.lanes) {
                    const bool live = r + sub < n;
                    body(row0, r + sub, live, at + (live ? r + sub : 0) * row_bytes, slot);
                }
            } else {
                for (int r = 0; r < n; ++r)
                    body(row0, r, true, at + r * row_bytes, slot);
            }
            __syncwarp();
            if (lane_id() == 0)
                mbar_arrive(barrier_at(sm.empty + 8 * slot));
        };
        const int own = p.slots / p.groups, first_slot = group * own;
        int at = 0;
        uint32_t phase = 0;
        auto advance = [&]() {
            if (++at == own) {
                at = 0;
                phase ^= 1;
            }
        };
        if constexpr (!kGated) {  // a group's slots are evenly spaced
            for (st.next(p, 0, group); st.more();) {
                const uint32_t row0 = st.row;
                const int n = st.count(p);
                st.next(p, n, p.groups);
                rows_of(first_slot + at, phase, row0, n);
                advance();
            }
            end_of_run(0);
        } else {
            // all threads meet at the end of each run, to change the gate together
            // (set_up loaded the first); between, a group's slots are evenly spaced
            int whose = 0;
            bool turn = false;
            while (st.more()) {
                const uint32_t run = st.run;
                if (turn) {
                    named_bar_sync(15, threads);
                    load_f<false>(run);
                    named_bar_sync(15, threads);
                }
                // slots left in the run, and how many of them come before this group's next
                const uint32_t last = min(st.run_end, st.end);
                const int left = static_cast<int>((last - st.row + p.slot_rows - 1) / p.slot_rows);
                const int before = group >= whose ? group - whose : group - whose + p.groups;
                const bool ours = before < left;
                const uint32_t row0 = ours ? st.row + before * p.slot_rows : last;
                const int n = static_cast<int>(min(last - row0, static_cast<uint32_t>(p.slot_rows)));
                st.row = row0 + n;
                whose = ours ? (group + 1 == p.groups ? 0 : group + 1) : (whose + left) % p.groups;
                if (ours) {
                    rows_of(first_slot + at, phase, row0, n);
                    advance();
                }
                turn = st.row == last;
                if (turn) {
                    end_of_run(run);
                    ++st.run;
                    st.run_end += static_cast<uint32_t>(p.run);
                }
            }
        }
    }
};

// The copying warp sets up the barriers and leaves (true); the others load w1 and
// the first f, and wait for it.
template <typename T, int kIn, int kSums>
__device__ __forceinline__ bool set_up(const ResidualNormParams &p, const Smem &sm, int threads, int copies_arrive,
                                       const Worker<T, kIn, kSums> &me)
{
    if (threadIdx.x >= threads) {
        if (threadIdx.x == threads) {
            for (int i = 0; i < p.slots; ++i) {
                mbar_init(barrier_at(sm.full + 8 * i), copies_arrive);
                mbar_init(barrier_at(sm.empty + 8 * i), p.warps);
            }
            sm.set_aborted(false);
            fence_mbar_init();
        }
        __syncwarp();
        return true;
    }
    const int nvec = p.D * static_cast<int>(sizeof(T)) / 16;
    if (kIn == 4 && p.dh == nullptr)  // the copies leave its place in the slots as it is
        for (int i = threadIdx.x; i < p.slots * p.slot_rows * nvec; i += threads) {
            const int slot = i / (p.slot_rows * nvec);
            st_shared(sm.ring + 16 * (i + (3 * slot + 2) * p.slot_rows * nvec), make_uint4(0, 0, 0, 0));
        }
    me.template load_f<true>(Slots(p).run);
    __syncthreads();
    return false;
}

// kC: chunks a thread holds of its row; all but the last are there for every
// thread.  kSub: short rows, several a warp (kC = 1).  kY, kPost: a block before
// this norm, and a norm behind the block.  kGated: a gate for every sequence.
template <typename T, int kC, bool kSub, bool kPost, bool kY, bool kGated>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_fwd_kernel(
    const __grid_constant__ ResidualNormParams p)
{
    constexpr int kIn = 2, kP = Chunk<T>::kP, kE = Chunk<T>::kE;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int row_bytes = p.D * static_cast<int>(sizeof(T)), nvec = row_bytes / 16;
    const Smem sm(smem_raw, p, row_bytes);
    const int threads = static_cast<int>(blockDim.x) - 32;
    Worker<T, kIn, 1> me(p, sm, threads);
    if (set_up(p, sm, threads, 1, me)) {
        const uint8_t *in[kIn] = {static_cast<const uint8_t *>(p.x), static_cast<const uint8_t *>(p.y)};
        copy_rows<kIn, false>(p, sm, in, row_bytes);
        return;
    }
    const int pitch = p.slot_rows * row_bytes;  // of a slot's tensors
    const float inv_d = 1.f / static_cast<float>(p.D);
    me.template go<kSub, kGated>(
        0xa2,
        [&](uint32_t row0, int r, bool live, uint32_t from, int) {
            // the block's output is read from the slot as often as it is needed; only
            // the sum with the stream stays in registers
            Chunk<T> x[kC], y;
            auto there = [&](int c) { return (!kSub || live) && (c < kC - 1 || me.col + c * me.width < nvec); };
            float s[1], r2 = 1.f;
            if constexpr (kPost) {
                float2 q = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    if (!there(c))
                        continue;
                    y.unpack(ld_shared(from + pitch + (me.col + c * me.width) * 16));
#pragma unroll
                    for (int e = 0; e < kP; ++e)
                        q = ffma2(y.v[e], y.v[e], q);
                }
                s[0] = q.x + q.y;
                me.sum(s);
                r2 = rsqrtf(fmaf(s[0], inv_d, p.eps));
            }
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                if (!there(c))
                    continue;
                const int at = me.col + c * me.width;
                x[c].unpack(ld_shared(from + at * 16));
                if constexpr (kY) {
                    Chunk<T> f;
                    f.read(sm.f + at * kE * 4);
                    y.unpack(ld_shared(from + pitch + at * 16));
#pragma unroll
                    for (int e = 0; e < kP; ++e) {
                        const float2 yh = kPost ? fmul2(y.v[e], both(r2)) : y.v[e];
                        x[c].v[e] = ffma2(yh, f.v[e], x[c].v[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    q = ffma2(x[c].v[e], x[c].v[e], q);
            }
            s[0] = q.x + q.y;
            me.sum(s);
            const float r1 = rsqrtf(fmaf(s[0], inv_d, p.eps));
            if (!live || !ULY_IN_BOUNDS(p.w.status, row0 + r, 1, p.T, 0x52))
                return;
            const int64_t out = static_cast<int64_t>(row0 + r) * row_bytes;
            if (me.col == 0 && p.rstd_out) {
                p.rstd_out[row0 + r] = r1;
                p.rstd_out[p.T + row0 + r] = r2;
            }
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int at = me.col + c * me.width;
                if (!there(c))
                    continue;
                if (kY && p.h)
                    __stcs(reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.h) + out + at * 16), x[c].pack());
                Chunk<T> w;
                w.unpack(ld_shared(sm.w1 + at * 16));
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    x[c].v[e] = fmul2(fmul2(x[c].v[e], both(r1)), w.v[e]);
                __stcs(reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.z) + out + at * 16), x[c].pack());
            }
        },
        [](uint32_t) {});
}

// With one chunk a thread what both passes over a row need stays in registers; with
// more it is formed again (two held chunks spill: 64K rows of 2560 324 us, not 300).
template <typename T, int kC, bool kSub, bool kPost, bool kY, bool kGated>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_bwd_kernel(
    const __grid_constant__ ResidualNormParams p)
{
    constexpr int kIn = 4, kP = Chunk<T>::kP, kE = Chunk<T>::kE;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int row_bytes = p.D * static_cast<int>(sizeof(T)), nvec = row_bytes / 16;
    const Smem sm(smem_raw, p, row_bytes);
    const int threads = static_cast<int>(blockDim.x) - 32;
    Worker<T, kIn, kPost ? 3 : 1> me(p, sm, threads);
    if (set_up(p, sm, threads, 2, me)) {
        const uint8_t *in[kIn] = {static_cast<const uint8_t *>(p.x), static_cast<const uint8_t *>(p.dz),
                                  static_cast<const uint8_t *>(p.dh), static_cast<const uint8_t *>(p.y)};
        copy_rows<kIn, true>(p, sm, in, row_bytes);
        return;
    }
    const uint32_t w_at = sm.w1 + me.col * 16, f_at = sm.f + me.col * kE * 4;
    const int pitch = p.slot_rows * row_bytes;  // of a slot's tensors
    const float inv_d = 1.f / static_cast<float>(p.D);
    float2 a1[kC][kP], aA[kC][kP];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int e = 0; e < kP; ++e)
            a1[c][e] = aA[c][e] = make_float2(0.f, 0.f);
    // writes the block's sums of its columns, of all its groups in order, as one
    // row, and takes the threads' own back to zero
    auto flush = [&](float *base, int64_t row, [[maybe_unused]] int64_t extent, float2(&a)[kC][kP],
                     [[maybe_unused]] unsigned site) {
        if (p.parts == 0) {  // one row at once: the threads' columns are the block's
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int at = me.col + c * me.width;
                const int64_t off = row * p.D + static_cast<int64_t>(at) * kE;
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    if (at < nvec && ULY_IN_BOUNDS(p.w.status, off + 2 * e, 2, extent, site))
                        *reinterpret_cast<float2 *>(base + off + 2 * e) = a[c][e];
                    a[c][e] = make_float2(0.f, 0.f);
                }
            }
            return;
        }
        const uint32_t mine = sm.scratch + (me.group * (32 / p.lanes) + me.sub) * p.D * 4;
        named_bar_sync(15, threads);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int at = me.col + c * me.width;
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                if (at < nvec)
                    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(mine + (at * kE + 2 * e) * 4),
                                 "f"(a[c][e].x), "f"(a[c][e].y)
                                 : "memory");
                a[c][e] = make_float2(0.f, 0.f);
            }
        }
        named_bar_sync(15, threads);
        for (int i = threadIdx.x; i < p.D; i += threads) {
            float t = ld_shared_f32(sm.scratch + i * 4);
            for (int j = 1; j < p.parts; ++j)
                t += ld_shared_f32(sm.scratch + (j * p.D + i) * 4);
            if (ULY_IN_BOUNDS(p.w.status, row * p.D + i, 1, extent, site))
                base[row * p.D + i] = t;
        }
    };
    me.template go<kSub, kGated>(
        0xa3,
        [&](uint32_t row0, int r, bool live, uint32_t from, int slot) {
            const uint32_t stats = sm.stats + (slot * 2 * kMaxRows + r) * 4;
            const float m1 = live ? ld_shared_f32(stats) : 0.f, m2 = live && kPost ? ld_shared_f32(stats + kMaxRows * 4) : 0.f;
            constexpr bool kHold = kC == 1;
            auto there = [&](int c) { return (!kSub || live) && (c < kC - 1 || me.col + c * me.width < nvec); };
            const uint32_t x_at = from + me.col * 16, dz_at = x_at + pitch, dh_at = dz_at + pitch, y_at = dh_at + pitch;
            auto read_y = [&](int c, Chunk<T> &yh) {
                yh.unpack(ld_shared(y_at + c * me.width * 16));
                if (kPost)
#pragma unroll
                    for (int e = 0; e < kP; ++e)
                        yh.v[e] = fmul2(yh.v[e], both(m2));
            };
            // hh, yh, b = dh + r1 w1 dz and f of one chunk
            auto form = [&](int c, Chunk<T> &hh, Chunk<T> &yh, Chunk<T> &b, Chunk<T> &f, Chunk<T> &dz, Chunk<T> &gz) {
                const int at = c * me.width * 16;
                hh.unpack(ld_shared(x_at + at));
                if constexpr (kY) {
                    f.read(f_at + c * me.width * kE * 4);
                    read_y(c, yh);
#pragma unroll
                    for (int e = 0; e < kP; ++e)
                        hh.v[e] = ffma2(f.v[e], yh.v[e], hh.v[e]);
                }
                dz.unpack(ld_shared(dz_at + at));
                gz.unpack(ld_shared(w_at + at));
                b.unpack(ld_shared(dh_at + at));
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    hh.v[e] = fmul2(hh.v[e], both(m1));
                    gz.v[e] = fmul2(gz.v[e], dz.v[e]);
                    b.v[e] = ffma2(gz.v[e], both(m1), b.v[e]);
                }
            };
            constexpr int kKept = kHold ? kC : 1;
            Chunk<T> hh[kKept], b[kKept], yh, f, dz, gz;
            float2 q1 = make_float2(0.f, 0.f), q2 = q1, q3 = q1;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int i = kHold ? c : 0;
                if (!there(c))
                    continue;
                form(c, hh[i], yh, b[i], f, dz, gz);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    q1 = ffma2(gz.v[e], hh[i].v[e], q1);
                    a1[c][e] = ffma2(dz.v[e], hh[i].v[e], a1[c][e]);
                    if constexpr (kPost) {
                        const float2 fy = fmul2(f.v[e], yh.v[e]);
                        q2 = ffma2(fy, b[i].v[e], q2);
                        q3 = ffma2(fy, hh[i].v[e], q3);
                    }
                }
            }
            float s[kPost ? 3 : 1];
            s[0] = q1.x + q1.y;
            if constexpr (kPost) {
                s[1] = q2.x + q2.y;
                s[2] = q3.x + q3.y;
            }
            me.sum(s);
            const float k1 = m1 * (s[0] * inv_d);
            float k2 = 0.f;
            if constexpr (kPost)
                k2 = m2 * (fmaf(-k1, s[2], s[1]) * inv_d);
            if (!live || !ULY_IN_BOUNDS(p.w.status, row0 + r, 1, p.T, 0x54))
                return;
            const int64_t out = static_cast<int64_t>(row0 + r) * row_bytes + me.col * 16;
            uint8_t *dx = static_cast<uint8_t *>(p.dx) + out, *dy = static_cast<uint8_t *>(p.dy) + out;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int i = kHold ? c : 0, at = c * me.width * 16;
                if (!there(c))
                    continue;
                if constexpr (!kHold) {
                    form(c, hh[i], yh, b[i], f, dz, gz);
                } else if constexpr (kY) {
                    f.read(f_at + c * me.width * kE * 4);
                    read_y(c, yh);
                }
                Chunk<T> t;
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    t.v[e] = ffma2(hh[i].v[e], both(-k1), b[i].v[e]);
                __stcs(reinterpret_cast<uint4 *>(dx + at), t.pack());
                if constexpr (kY) {
#pragma unroll
                    for (int e = 0; e < kP; ++e) {
                        aA[c][e] = ffma2(t.v[e], yh.v[e], aA[c][e]);
                        t.v[e] = fmul2(t.v[e], f.v[e]);
                        if constexpr (kPost)
                            t.v[e] = ffma2(yh.v[e], both(-k2), fmul2(t.v[e], both(m2)));
                    }
                    __stcs(reinterpret_cast<uint4 *>(dy + at), t.pack());
                }
            }
        },
        [&](uint32_t run) {
            if (p.partA)
                flush(p.partA, blockIdx.x + run, p.partA_elems, aA, 0x55);
        });
    grid_next();
    if (p.part1)
        flush(p.part1, blockIdx.x, p.part1_elems, a1, 0x56);
}

// The weights' gradients from the blocks' sums, in an order that depends on the
// sizes alone: a block takes 32 columns of dweight (y = 0) or of the gates and
// dpost_weight (y = 1), kJoinLanes threads a column.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinLanes) residual_norm_join_kernel(const __grid_constant__ ResidualNormParams p,
                                                                             int blocks)
{
    __shared__ float part[kJoinLanes][33];
    grid_wait();
    const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const bool in = col < p.D;
    // rows first, first + step, .. below last of a buffer of D columns
    auto column = [&](const float *base, int64_t first, int64_t last, int step, [[maybe_unused]] int64_t extent) {
        float s = 0.f;
        if (in)
#pragma unroll 4
            for (int64_t r = first; r < last; r += step)
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
    auto put = [&](void *w, int64_t at, float v) {
        if constexpr (sizeof(T) == 2)
            static_cast<uint16_t *>(w)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
        else
            static_cast<float *>(w)[at] = v;
    };
    auto write = [&](void *w, int64_t at, float v) {
        if (in && j == 0)
            put(w, at, v);
    };
    if (blockIdx.y == 0) {
        if (p.dw1)
            write(p.dw1, col, across(column(p.part1, j, blocks, kJoinLanes, p.part1_elems)));
        return;
    }
    if (!p.dw2 && !p.dgate)
        return;
    if (p.gates <= 1) {  // one run, every block has a row of it
        const float A = p.scale * across(column(p.partA, j, blocks, kJoinLanes, p.partA_elems));
        if (p.dgate && in)
            write(p.dgate, col, p.w2 ? A * value(p.w2, col) : A);
        if (p.dw2 && in)
            write(p.dw2, col, p.gate ? A * value(p.gate, col) : A);
        return;
    }
    if (p.gates >= kJoinLanes) {  // gates enough for one a warp, eight of a warp's at once
        constexpr int kAt = 8;
        float dw2 = 0.f;
        const int runs = static_cast<int>(p.T / p.run);
        auto rows_of = [&](int run, int64_t &lo, int64_t &hi) {  // the run's rows of partA
            const uint32_t first = static_cast<uint32_t>(run) * static_cast<uint32_t>(p.run);
            lo = static_cast<int64_t>(first / p.block_rows) + run;
            hi = static_cast<int64_t>((first + static_cast<uint32_t>(p.run) - 1) / p.block_rows) + run + 1;
        };
        for (int b0 = j; b0 < p.gates; b0 += kAt * kJoinLanes) {
            float s[kAt];
            int64_t lo[kAt], hi[kAt];
#pragma unroll
            for (int e = 0; e < kAt; ++e) {
                const int b = b0 + e * kJoinLanes;
                s[e] = 0.f;
                lo[e] = hi[e] = 0;
                if (b < p.gates) {
                    rows_of(b, lo[e], hi[e]);
                    if (in && ULY_IN_BOUNDS(p.w.status, lo[e] * p.D + col, 1, p.partA_elems, 0x6c))
                        s[e] = p.partA[lo[e] * p.D + col];
                }
            }
#pragma unroll
            for (int e = 0; e < kAt; ++e) {
                const int b = b0 + e * kJoinLanes;
                if (b >= p.gates)
                    break;
                s[e] += column(p.partA, lo[e] + 1, hi[e], 1, p.partA_elems);
                for (int run = b + p.gates; run < runs; run += p.gates) {
                    int64_t l, h;
                    rows_of(run, l, h);
                    s[e] += column(p.partA, l, h, 1, p.partA_elems);
                }
                if (!in)
                    continue;
                const float A = p.scale * s[e];
                const int64_t at = b * static_cast<int64_t>(p.D) + col;
                if (p.dgate)
                    put(p.dgate, at, p.w2 ? A * value(p.w2, col) : A);
                if (p.dw2)
                    dw2 = fmaf(value(p.gate, at), A, dw2);
            }
        }
        if (p.dw2)
            write(p.dw2, col, across(dw2));
        return;
    }
    // a gate's runs, several at once where there are fewer than threads a column
    const int runs_of = static_cast<int>(p.T / p.run / p.gates);  // runs of a gate
    const int at_once = runs_of < kJoinLanes ? runs_of : kJoinLanes, share = kJoinLanes / at_once;
    float dw2 = 0.f;
    for (int b = 0; b < p.gates; ++b) {
        float s = 0.f;
        if (j < at_once * share)
            for (int i = j / share; i < runs_of; i += at_once) {
                const uint32_t run = b + static_cast<uint32_t>(i) * p.gates, first = run * static_cast<uint32_t>(p.run);
                const uint32_t lo = first / p.block_rows, hi = (first + static_cast<uint32_t>(p.run) - 1) / p.block_rows;
                s += column(p.partA, static_cast<int64_t>(lo) + run + j % share, static_cast<int64_t>(hi) + run + 1, share,
                            p.partA_elems);
            }
        const float A = p.scale * across(s);
        const int64_t at = b * static_cast<int64_t>(p.D) + col;
        if (p.dgate && in)
            write(p.dgate, at, p.w2 ? A * value(p.w2, col) : A);
        if (p.dw2 && in)
            dw2 = fmaf(value(p.gate, at), A, dw2);
    }
    if (p.dw2)
        write(p.dw2, col, dw2);
}

template <typename T, int kC, bool kSub, bool kPost, bool kY, bool kGated>
auto kernel_of(bool bwd) -> void (*)(const ResidualNormParams)
{
    return bwd ? residual_norm_bwd_kernel<T, kC, kSub, kPost, kY, kGated>
               : residual_norm_fwd_kernel<T, kC, kSub, kPost, kY, kGated>;
}

template <typename T, int kC, bool kSub>
auto kernel_for(const ResidualNormParams &p, bool bwd) -> void (*)(const ResidualNormParams)
{
    const bool gated = p.gates > 1;
    if (p.w2)
        return gated ? kernel_of<T, kC, kSub, true, true, true>(bwd) : kernel_of<T, kC, kSub, true, true, false>(bwd);
    if (p.y)
        return gated ? kernel_of<T, kC, kSub, false, true, true>(bwd) : kernel_of<T, kC, kSub, false, true, false>(bwd);
    return kernel_of<T, kC, kSub, false, false, false>(bwd);
}

template <typename T>
cudaError_t launch_residual_norm_typed(const ResidualNormParams &p, const ResidualNormPlan &q, bool bwd, cudaStream_t s)
{
    void (*k)(const ResidualNormParams) = nullptr;
    switch (q.chunks) {
    case 1: k = q.lanes < 32 ? kernel_for<T, 1, true>(p, bwd) : kernel_for<T, 1, false>(p, bwd); break;
    case 2: k = kernel_for<T, 2, false>(p, bwd); break;
    case 3: k = kernel_for<T, 3, false>(p, bwd); break;
    case 4: k = kernel_for<T, 4, false>(p, bwd); break;
    case 5: k = kernel_for<T, 5, false>(p, bwd); break;
    }
    if (k == nullptr)
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(q.smem));
    if (e != cudaSuccess)
        return e;
    k<<<q.blocks, q.threads, q.smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !bwd || !(p.part1 || p.partA))
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.D + 31) / 32), 2);
    cfg.blockDim = dim3(32 * kJoinLanes);
    cfg.stream = s;
    cudaLaunchAttribute early[1];  // its blocks may be set up while the kernel above ends
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, residual_norm_join_kernel<T>, p, q.blocks);
}

}  // namespace
}  // namespace uly
