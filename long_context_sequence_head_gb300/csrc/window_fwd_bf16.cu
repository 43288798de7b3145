// Sliding-window attention with sinks, forward, bf16 in, fp32 accumulate, on the
// 5th-generation tensor cores, head_dim 128.
//
// Row i of a document that starts at s sees the keys [max(s, i - window + 1), i]
// and [s, s + sinks).  The arithmetic of a tile is that of attn_fwd_bf16.cu: two
// query heads of a GQA group share every K/V tile, online softmax in base 2 with
// lazy rescaling (the running maximum is kept until a row's exponentials would
// pass 2^8), P overwrites S in TMEM and is the A operand of P V.
//
// A head without a partner takes two neighbouring tiles of rows instead, whose walk is
// one key tile longer: 8 such heads of 32,768 tokens, window 4096, 667 us, 1040 with a
// tile a block.  Not where there is an SM for every tile (16 heads of 1024 tokens,
// window 512: 23 us, 26 in pairs).
//
// What differs is the walk: a tile of 128 rows takes the key tiles of its window
// and its sinks.  Up to 32 sinks are one tile of 32 keys that starts at the
// document's first, instead of 128 that hold a few; more are whole tiles.  Window
// tiles start at multiples of 128: 9 of them under a window of 1024.
//   64K tokens, 32 heads, window 4096, 4 sinks 3.24 ms, 1310 TFLOP/s of allowed pairs
// (6 % more are computed in boundary tiles); 8K, window 1024: 152 us, 850 TFLOP/s (160
// with whole tiles of sinks), of which a block's start and end take about a third.  At
// 16K tokens under a window of 4096 the tensor pipe is busy 57 % of the cycles and the
// exponentials' 29 %: between them and the full forward's 1,500 TFLOP/s are start and end
// of walks of 34 tiles, 8 to 10 us a block of 60.  A block that stays on its SM and takes tile after tile, the
// next one's Q and first K loaded and its first S made meanwhile, was slower: with two
// Q buffers and three K/V slots 3.50 ms and 155 us (the slots bind), with three Q
// tiles taken in turn and four slots 3.79 ms and 175 us (the second head waits for the
// first one's output to leave its Q tile).
//
// Warp roles (320 threads), TMEM and shared memory as in attn_fwd_bf16.cu.
#include "uly_internal.h"

namespace uly {
namespace {

constexpr int kBM = 128;          // query rows per tile
constexpr int kBN = 128;          // keys per tile
constexpr int kD = 128;           // head dim
constexpr int kSlots = 4;         // K/V ring slots
constexpr int kFew = 32;          // keys of a narrow tile of sinks
constexpr int kTileBytes = kBM * kD * 2;  // 32 KB
constexpr int kChunk = kBM * 64 * 2;      // one 64-column swizzled chunk: 16 KB
constexpr int kThreads = 320;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

struct Smem {
    static constexpr int kQ = 0;
    static constexpr int kSlot0 = 2 * kTileBytes;
    static constexpr int kBars = kSlot0 + kSlots * kTileBytes;
    static constexpr int kTotal = kBars + 256;
};

struct Params {
    int64_t SB, N;
    int Hq, Hkv, G, n_qtiles;
    int units, pair_units;  // of the call; those of two heads come first
    bool tall;              // single heads take two tiles of rows
    const int32_t *cu;
    int num_docs;
    int window, sinks;
    float scale_log2;
    float *lse;
    int64_t lse_elems;      // extent for the bounds checks of debug builds
    const int32_t *order;   // with documents: query tiles, longest walk first
    WaitCfg w;
    RowLayout L;
};

__device__ __forceinline__ void doc_range(const Params &p, int i, int &lo, int &hi)
{
    lo = 0;
    hi = static_cast<int>(p.N);
    if (p.cu == nullptr)
        return;
    int a = 0, b = p.num_docs;
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (p.cu[m] <= i)
            a = m;
        else
            b = m;
    }
    lo = p.cu[a];
    hi = p.cu[a + 1];
}

// A block's rows and the key tiles it walks.
struct Unit {
    int sb, kvh, h0;  // first head
    bool two;         // heads, or tiles of rows
    int q0, down;     // first row; rows from the first tile to the second (0: two heads)
    int start;        // of the first row's document
    int n_sink;       // tiles of its sinks: one narrow one, or whole ones from tile `sink` on
    int sink, lo;     // first whole tile of sinks, first tile of the window
    int n;            // tiles

    // Pairs of heads come first, then the single heads of an odd group.
    __device__ __forceinline__ Unit(const Params &p, int u)
    {
        const int pairs = p.G / 2;
        two = u < p.pair_units;
        int pair = pairs, rest = u - p.pair_units;
        if (two) {
            pair = u % pairs;
            rest = u / pairs;
        }
        down = !two && p.tall ? kBM : 0;
        const int n_ranks = down ? (p.n_qtiles + 1) / 2 : p.n_qtiles;
        const int rank = rest % n_ranks, prob = rest / n_ranks;
        kvh = prob % p.Hkv;
        sb = prob / p.Hkv;
        h0 = kvh * p.G + 2 * pair;
        q0 = p.order != nullptr ? p.order[down ? p.n_qtiles + rank : rank] : n_ranks - 1 - rank;
        if (down) {
            q0 *= 2;
            two = q0 + 1 < p.n_qtiles;
        }
        q0 *= kBM;
        const int last = min(q0 + (two ? down : 0) + kBM, static_cast<int>(p.N)) - 1;
        int end;
        doc_range(p, q0, start, end);
        const int first = max(start, q0 - p.window + 1), sink_end = min(start + p.sinks, first);
        lo = first / kBN;
        sink = start / kBN;
        n_sink = sink_end > start ? min((sink_end - 1) / kBN + 1, lo) - sink : 0;
        if (n_sink > 0 && p.sinks <= kFew)
            n_sink = 1;
        n = n_sink + last / kBN - lo + 1;
    }
    __device__ __forceinline__ int head(int t) const { return down ? h0 : h0 + t; }
    __device__ __forceinline__ bool narrow(const Params &p, int j) const { return j < n_sink && p.sinks <= kFew; }
    __device__ __forceinline__ int key0(const Params &p, int j) const
    {
        return j >= n_sink ? (lo + j - n_sink) * kBN : p.sinks <= kFew ? start : (sink + j) * kBN;
    }
};

// Of 32 neighbouring keys, those in [lo, hi) (both relative to the first) as bits.
__device__ __forceinline__ uint32_t key_bits(int lo, int hi)
{
    lo = min(max(lo, 0), 32);
    hi = min(max(hi, 0), 32);
    const uint32_t below_hi = hi == 32 ? ~0u : (1u << hi) - 1u, below_lo = lo == 32 ? ~0u : (1u << lo) - 1u;
    return below_hi & ~below_lo;
}

// What a row sees: [w_lo, hi) and [lo, s_hi).
struct Row {
    int lo, s_hi, w_lo, hi;

    __device__ __forceinline__ uint32_t columns(int base) const
    {
        return key_bits(w_lo - base, hi - base) | key_bits(lo - base, s_hi - base);
    }
};

// The softmax of one tile of S (columns in TMEM at tS), P written over it, O (tO)
// and l rescaled where the maximum rose.
struct Softmax {
    float m, l;

    __device__ __forceinline__ static float row_max(const float (&pm)[8])
    {
        return fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7])));
    }
    __device__ __forceinline__ static float total(const float2 (&rs)[4])
    {
        const float2 a = fadd2(fadd2(rs[0], rs[1]), fadd2(rs[2], rs[3]));
        return a.x + a.y;
    }
    // raises m to a tile's maximum where that exceeds it by more than `slack`; the factor
    // of l and O
    __device__ __forceinline__ float raise(float mx, float scale_log2, float slack, bool &rescale)
    {
        const float cand = mx * scale_log2;
        if (!(cand > m + slack))
            return 1.f;
        const float alpha = ex2_approx(m - cand);
        rescale = m != -INFINITY;
        m = cand;
        return alpha;
    }
    __device__ __forceinline__ float2 shift() const
    {
        const float r = m == -INFINITY ? 0.f : m;
        return make_float2(-r, -r);
    }
};

__device__ __forceinline__ float2 exp_pair(uint32_t a, uint32_t b, float2 scale, float2 shift)
{
    const float2 x = ffma2(make_float2(__uint_as_float(a), __uint_as_float(b)), scale, shift);
    return make_float2(ex2_approx(x.x), ex2_approx(x.y));
}

__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_bf16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                           const __grid_constant__ CUtensorMap tm_k_few, const __grid_constant__ CUtensorMap tm_v_few,
                           const __grid_constant__ Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Smem::kBars);
    uint64_t *q_full = bars;                      // [2] heads
    uint64_t *kv_full = bars + 2;                 // [kSlots]
    uint64_t *kv_empty = kv_full + kSlots;        // [kSlots]
    uint64_t *s_full = kv_empty + kSlots;         // [2]
    uint64_t *p_full = s_full + 2;                // [2]
    uint64_t *o_done = s_full + 4;                // [2]
    uint64_t *drain = s_full + 6;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = warp_id();
    const int lane = lane_id();
    const Unit x(p, static_cast<int>(blockIdx.x));

    if (warp == 8 && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);  // one elected arrival per softmax warp
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    if (warp == 8) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_o);
            int c1, c2, c3, c4, loads = 0;
            auto load_q = [&](int t) {
                uint8_t *dst = smem + Smem::kQ + t * kTileBytes;
                mbar_expect_tx(&q_full[t], kTileBytes);
                p.L.tile(x.sb, x.q0 + t * x.down, p.Hq, x.head(t), c1, c2, c3, c4);
                tma_load_5d(dst, &tm_q, &q_full[t], 0, c1, c2, c3, c4);
                tma_load_5d(dst + kChunk, &tm_q, &q_full[t], 64, c1, c2, c3, c4);
            };
            bool ok = true;
            load_q(0);
            for (int j = 0; ok && j < x.n; ++j) {
                const bool few = x.narrow(p, j);
                const int key0 = x.key0(p, j);
                for (int which = 0; which < 2; ++which) {
                    const int slot = loads % kSlots;
                    ok = !*abort_flag && mbar_wait(&kv_empty[slot], ((loads / kSlots) & 1) ^ 1, p.w, 0xb2);
                    if (!ok)
                        break;
                    uint8_t *dst = smem + Smem::kSlot0 + slot * kTileBytes;
                    const CUtensorMap *tm = few ? (which ? &tm_v_few : &tm_k_few) : (which ? &tm_v : &tm_k);
                    mbar_expect_tx(&kv_full[slot], few ? kFew * kD * 2 : kTileBytes);
                    p.L.tile(x.sb, key0, p.Hkv, x.kvh, c1, c2, c3, c4);
                    tma_load_5d(dst, tm, &kv_full[slot], 0, c1, c2, c3, c4);
                    tma_load_5d(dst + kChunk, tm, &kv_full[slot], 64, c1, c2, c3, c4);
                    if (loads++ == 0 && x.two)
                        load_q(1);  // behind the first K, which the first head waits for
                }
            }
            if (!ok || *abort_flag) {
                *abort_flag = 1;
                // wait (bounded) for every load this thread started
                mbar_wait(&q_full[0], 0, p.w, 0xbf);
                if (x.two && loads > 0)
                    mbar_wait(&q_full[1], 0, p.w, 0xbf);
                for (int i = loads > kSlots ? loads - kSlots : 0; i < loads; ++i)
                    mbar_wait(&kv_full[i % kSlots], (i / kSlots) & 1, p.w, 0xbf);
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id_qk = idesc_bf16(kBM, kBN, false, false), id_few = idesc_bf16(kBM, kFew, false, false);
            const uint32_t id_pv = idesc_bf16(kBM, kD, false, true);
            const uint32_t sQ = smem_u32(smem + Smem::kQ), sSlot0 = smem_u32(smem + Smem::kSlot0);
            auto issue_qk = [&](int t, int slot, bool few) {
                const uint32_t q = sQ + t * kTileBytes, k = sSlot0 + slot * kTileBytes;
                const uint32_t id = few ? id_few : id_qk;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kChunk + (kk & 3) * 32;
                    mma_ss(tbase + t * 128, desc_sw128(q + off, 16, 1024), desc_sw128(k + off, 16, 1024), id, kk > 0);
                }
                mma_commit(&s_full[t]);
            };
            auto issue_pv = [&](int t, int slot, bool acc, bool few) {
                const uint32_t v = sSlot0 + slot * kTileBytes;
                auto step = [&](int kk) {
                    mma_ts(tbase + 256 + t * 128, tbase + t * 128 + kk * 8,
                           desc_sw128(v + kk * 16 * 128, kChunk, 1024), id_pv, (acc || kk > 0) ? 1u : 0u);
                };
#pragma unroll
                for (int kk = 0; kk < kFew / 16; ++kk)
                    step(kk);
                if (!few)
#pragma unroll
                    for (int kk = kFew / 16; kk < kBN / 16; ++kk)
                        step(kk);
            };
            bool ok = mbar_wait(&kv_full[0], 0, p.w, 0xb3);
            for (int t = 0; ok && t < (x.two ? 2 : 1); ++t) {
                ok = mbar_wait(&q_full[t], 0, p.w, 0xb4);
                tc_fence_after();
                if (ok)
                    issue_qk(t, 0, x.narrow(p, 0));
            }
            if (ok)
                mma_commit(&kv_empty[0]);
            for (int j = 0; ok && j < x.n; ++j) {
                const int it_v = 2 * j + 1, it_k = 2 * j + 2;
                const int slot_v = it_v % kSlots, slot_k = it_k % kSlots;
                const bool more = j + 1 < x.n, few = x.narrow(p, j);  // no tile behind the first is narrow
                ok = mbar_wait(&kv_full[slot_v], (it_v / kSlots) & 1, p.w, 0xb5) &&
                     mbar_wait(&p_full[0], j & 1, p.w, 0xb6);
                if (!ok)
                    break;
                tc_fence_after();
                issue_pv(0, slot_v, j > 0, few);
                if (more) {
                    ok = mbar_wait(&kv_full[slot_k], (it_k / kSlots) & 1, p.w, 0xb8);
                    if (!ok)
                        break;
                    tc_fence_after();
                    issue_qk(0, slot_k, false);
                } else {
                    mma_commit(&o_done[0]);
                }
                if (x.two) {
                    ok = mbar_wait(&p_full[1], j & 1, p.w, 0xb9);
                    if (!ok)
                        break;
                    tc_fence_after();
                    issue_pv(1, slot_v, j > 0, few);
                }
                mma_commit(&kv_empty[slot_v]);
                if (more) {
                    if (x.two)
                        issue_qk(1, slot_k, false);
                    mma_commit(&kv_empty[slot_k]);
                } else {
                    mma_commit(&o_done[1]);
                }
            }
            if (!ok) {
                *abort_flag = 1;
                mma_commit(&o_done[0]);  // nobody waits for what will not come
                mma_commit(&o_done[1]);
            }
            mma_commit(drain);
            mbar_wait(drain, 0, p.w, 0xbe);
        }
    } else {
        // ------------------------------------------------ softmax warps
        const int t = warp >> 2;  // head 0 or 1 of the pair
        const int wq = warp & 3;  // TMEM lane quarter
        const int r = wq * 32 + lane;
        const uint32_t tS = tbase + t * 128 + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t tO = tbase + 256 + t * 128 + (static_cast<uint32_t>(wq * 32) << 16);
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
        if (t == 0 || x.two) {
            const int row = x.q0 + t * x.down + r;
            Row see;
            {
                const int at = min(row, static_cast<int>(p.N) - 1);
                int end;
                doc_range(p, at, see.lo, end);
                see.hi = at + 1;
                see.w_lo = max(see.lo, at - p.window + 1);
                see.s_hi = see.lo;
                if (see.lo + p.sinks >= see.w_lo)
                    see.w_lo = see.lo;
                else
                    see.s_hi = see.lo + p.sinks;
            }
            Softmax sm{-INFINITY, 0.f};
            bool ok = true;
            int j = 0;
            if (x.narrow(p, 0)) {
                // the sinks of the first row's document: rows of later ones see none of
                // them, and this row's are not looked for among the window's tiles
                ok = mbar_wait_warp(&s_full[t], 0, p.w, 0xc1 + t);
                tc_fence_after();
                uint32_t v[32];
                tmem_ld32p(tS, v);
                tmem_ld_wait();
                tmem_ld_fence32p(v);
                const bool mine = see.lo == x.start;  // the narrow tile starts with the first row's document
                const int w_lo = max(see.lo, see.hi - p.window), seen = mine ? min(p.sinks, w_lo - see.lo) : 0;
                float pm[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    pm[e] = -INFINITY;
#pragma unroll
                for (int c = 0; c < kFew; ++c) {
                    if (c >= seen)
                        v[c] = __float_as_uint(-INFINITY);
                    pm[c & 7] = fmaxf(pm[c & 7], __uint_as_float(v[c]));
                }
                sm.m = Softmax::row_max(pm) * p.scale_log2;
                const float2 shift = sm.shift();
                float2 rs[4] = {};
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < kFew; c += 2) {
                    const float2 e = exp_pair(v[c], v[c + 1], sl2, shift);
                    rs[(c >> 1) & 3] = fadd2(rs[(c >> 1) & 3], e);
                    pk[c >> 1] = pack_bf16x2(e.x, e.y);
                }
                sm.l = Softmax::total(rs);
                tmem_st16p(tS, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[t]);
                ++j;
                if (mine) {
                    see.w_lo = w_lo;
                    see.s_hi = see.lo;
                }
            }
            for (; ok && j < x.n; ++j) {
                ok = mbar_wait_warp(&s_full[t], j & 1, p.w, 0xc1 + t);
                if (!ok)
                    break;
                tc_fence_after();
                uint32_t v[kBN];  // S row, then P row (fp32 bit patterns)
#pragma unroll
                for (int cb = 0; cb < kBN; cb += 32)
                    tmem_ld32p(tS + cb, v + cb);
                tmem_ld_wait();
#pragma unroll
                for (int cb = 0; cb < kBN; cb += 32)
                    tmem_ld_fence32p(v + cb);
                const int key0 = x.key0(p, j);
                const bool masked = !((key0 >= see.w_lo && key0 + kBN <= see.hi) ||
                                      (key0 >= see.lo && key0 + kBN <= see.s_hi));
                const bool empty = (key0 >= see.hi || key0 + kBN <= see.w_lo) &&
                                   (key0 >= see.s_hi || key0 + kBN <= see.lo);
                if (masked) {
#pragma unroll
                    for (int cb = 0; cb < kBN; cb += 32) {
                        const uint32_t keep = see.columns(key0 + cb);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(keep >> c & 1u))
                                v[cb + c] = __float_as_uint(-INFINITY);
                    }
                }
                // Speculate that the running maximum still holds: the exponentials
                // against it all stay <= 2^8 exactly when the lazy rule keeps it, and
                // their sum <= 2^8 proves it (see attn_fwd_bf16.cu).
                float2 rs[4] = {};
                float alpha = 1.f, sum;
                bool rescale = false;
                const bool first = __any_sync(0xffffffffu, sm.m == -INFINITY && !empty);
                if (!first) {
                    const float2 shift = sm.shift();
#pragma unroll
                    for (int c = 0; c < kBN; c += 2) {
                        const float2 e = exp_pair(v[c], v[c + 1], sl2, shift);
                        rs[(c >> 1) & 3] = fadd2(rs[(c >> 1) & 3], e);
                        v[c] = __float_as_uint(e.x);
                        v[c + 1] = __float_as_uint(e.y);
                    }
                }
                sum = Softmax::total(rs);
                if (first) {
                    // S, masked above, is still in registers
                    float pm[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pm[e] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < kBN; ++c)
                        pm[c & 7] = fmaxf(pm[c & 7], __uint_as_float(v[c]));
                    alpha = sm.raise(Softmax::row_max(pm), p.scale_log2, kRescaleThreshold, rescale);
                    const float2 shift = sm.shift();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        rs[e] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const float2 e = exp_pair(v[half * 64 + c], v[half * 64 + c + 1], sl2, shift);
                            rs[(c >> 1) & 3] = fadd2(rs[(c >> 1) & 3], e);
                            pk[c >> 1] = pack_bf16x2(e.x, e.y);
                        }
                        tmem_st32p(tS + half * 32, pk);
                    }
                    sum = Softmax::total(rs);
                } else if (__any_sync(0xffffffffu, !(sum <= 256.f))) {
                    // exact: row maximum of S, then the exponentials, 64 columns at a time
                    float pm[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pm[e] = -INFINITY;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        tmem_ld32p(tS + half * 64, v);
                        tmem_ld32p(tS + half * 64 + 32, v + 32);
                        tmem_ld_wait();
                        tmem_ld_fence32p(v);
                        tmem_ld_fence32p(v + 32);
                        const uint32_t keep[2] = {masked ? see.columns(key0 + half * 64) : ~0u,
                                                  masked ? see.columns(key0 + half * 64 + 32) : ~0u};
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            pm[c & 7] = fmaxf(pm[c & 7], keep[c >> 5] >> (c & 31) & 1u ? __uint_as_float(v[c])
                                                                                       : -INFINITY);
                    }
                    // A row whose first tile held few of its keys (its sinks, a window's last
                    // ones) may have a maximum so low that every later tile's sum passes the
                    // bound without a score 2^8 above it: raised here whatever the slack, it
                    // comes this way once.  16K tokens of 8 heads, window 4096, 4 sinks, keys
                    // that no query prefers: 206 us, 307 with the lazy rule here too; 64K of 32
                    // heads 3.40 ms for 5.14.
                    alpha = sm.raise(Softmax::row_max(pm), p.scale_log2, 0.f, rescale);
                    const float2 shift = sm.shift();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        rs[e] = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        tmem_ld32p(tS + half * 64, v);
                        tmem_ld32p(tS + half * 64 + 32, v + 32);
                        tmem_ld_wait();
                        tmem_ld_fence32p(v);
                        tmem_ld_fence32p(v + 32);
                        const uint32_t keep[2] = {masked ? see.columns(key0 + half * 64) : ~0u,
                                                  masked ? see.columns(key0 + half * 64 + 32) : ~0u};
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const uint32_t inf = __float_as_uint(-INFINITY);
                            const float2 e = exp_pair(keep[c >> 5] >> (c & 31) & 1u ? v[c] : inf,
                                                      keep[c >> 5] >> (c & 31) & 2u ? v[c + 1] : inf, sl2, shift);
                            rs[(c >> 1) & 3] = fadd2(rs[(c >> 1) & 3], e);
                            pk[c >> 1] = pack_bf16x2(e.x, e.y);
                        }
                        // P of S columns half*64.. lands on S columns this thread has read
                        tmem_st32p(tS + half * 32, pk);
                    }
                    sum = Softmax::total(rs);
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            pk[c] = pack_bf16x2(__uint_as_float(v[half * 64 + 2 * c]),
                                                __uint_as_float(v[half * 64 + 2 * c + 1]));
                        tmem_st32p(tS + half * 32, pk);
                    }
                }
                sm.l = sm.l * alpha + sum;
                if (__any_sync(0xffffffffu, rescale)) {
                    const float a = rescale ? alpha : 1.f;
#pragma unroll
                    for (int cb = 0; cb < kD; cb += 32) {
                        uint32_t o32[32];
                        tmem_ld32p(tO + cb, o32);
                        tmem_ld_wait();
                        tmem_ld_fence32p(o32);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o32[c] = __float_as_uint(__uint_as_float(o32[c]) * a);
                        tmem_st32p(tO + cb, o32);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[t]);
            }
            if (!ok)
                *abort_flag = 1;
            // O epilogue: row r, normalised to bf16, into this head's Q tile (free once
            // its products are complete) in the layout of the tensor map; one thread
            // stores the tile
            const bool have_o = mbar_wait_warp(&o_done[t], 0, p.w, 0xc3 + t) && ok;
            uint8_t *stage = smem + Smem::kQ + t * kTileBytes;
            if (have_o) {
                tc_fence_after();
                const float inv = 1.f / sm.l;
#pragma unroll
                for (int cb = 0; cb < kD; cb += 32) {
                    uint32_t o32[32];
                    tmem_ld32p(tO + cb, o32);
                    tmem_ld_wait();
                    tmem_ld_fence32p(o32);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int part = cb / 8 + q;  // 16-byte unit of the row, 0..15
                        const uint4 val = make_uint4(
                            pack_bf16x2(__uint_as_float(o32[8 * q]) * inv, __uint_as_float(o32[8 * q + 1]) * inv),
                            pack_bf16x2(__uint_as_float(o32[8 * q + 2]) * inv, __uint_as_float(o32[8 * q + 3]) * inv),
                            pack_bf16x2(__uint_as_float(o32[8 * q + 4]) * inv, __uint_as_float(o32[8 * q + 5]) * inv),
                            pack_bf16x2(__uint_as_float(o32[8 * q + 6]) * inv, __uint_as_float(o32[8 * q + 7]) * inv));
                        *reinterpret_cast<uint4 *>(stage + (part >> 3) * kChunk + r * 128 +
                                                   (((part & 7) ^ (r & 7)) << 4)) = val;
                    }
                }
                fence_async_smem();
                if (row < p.N) {
                    const int64_t li = (static_cast<int64_t>(x.sb) * p.Hq + x.head(t)) * p.N + row;
                    if (ULY_IN_BOUNDS(p.w.status, li, 1, p.lse_elems, 0x12))
                        p.lse[li] = (sm.m + __log2f(sm.l)) * 0.69314718055994530942f;
                }
            }
            named_bar_sync(1 + t, 128);  // the head's four warps have staged their rows
            if (r == 0 && have_o) {
                int c1, c2, c3, c4;
                p.L.tile(x.sb, x.q0 + t * x.down, p.Hq, x.head(t), c1, c2, c3, c4);
                tma_store_5d(&tm_o, stage, 0, c1, c2, c3, c4);
                tma_store_5d(&tm_o, stage + kChunk, 64, c1, c2, c3, c4);
                bulk_commit();
                bulk_wait_read<0>();  // the tile is read before the block's shared memory goes
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9)
        tmem_dealloc(tbase, 512);
}

}  // namespace

cudaError_t launch_window_fwd_bf16(const AttnShape &s, const void *q, const void *k, const void *v, void *o,
                                   float *lse, cudaStream_t stream)
{
    if (s.d != kD)
        return cudaErrorInvalidValue;
    CUtensorMap tq, tk, tv, to, tkf, tvf;
    if (make_rows_map_bf16(&tq, q, s, s.Hq) != CUDA_SUCCESS || make_rows_map_bf16(&tk, k, s, s.Hkv) != CUDA_SUCCESS ||
        make_rows_map_bf16(&tv, v, s, s.Hkv) != CUDA_SUCCESS || make_rows_map_bf16(&to, o, s, s.Hq) != CUDA_SUCCESS ||
        make_rows_map_bf16(&tkf, k, s, s.Hkv, kFew) != CUDA_SUCCESS ||
        make_rows_map_bf16(&tvf, v, s, s.Hkv, kFew) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    Params p;
    p.SB = s.SB;
    p.N = s.N;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.G = s.Hq / s.Hkv;
    p.n_qtiles = static_cast<int>((s.N + kBM - 1) / kBM);
    p.pair_units = static_cast<int>(s.SB * s.Hkv * (p.G / 2) * p.n_qtiles);
    const int64_t singles = p.G % 2 ? s.SB * s.Hkv : 0;
    p.tall = p.pair_units + singles * p.n_qtiles > num_sms();
    p.units = p.pair_units + static_cast<int>(singles * (p.tall ? (p.n_qtiles + 1) / 2 : p.n_qtiles));
    p.cu = s.cu_dev;
    p.num_docs = s.num_docs;
    p.window = s.window;
    p.sinks = s.sinks;
    p.scale_log2 = s.scale * 1.4426950408889634f;
    p.lse = lse;
    p.lse_elems = s.lse_elems;
    p.order = s.order_dev;
    p.w = wait_cfg();
    p.L = s.L;
    const size_t smem = Smem::kTotal + 1024;
    const cudaError_t e = cudaFuncSetAttribute(window_fwd_bf16_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess)
        return e;
    window_fwd_bf16_kernel<<<p.units, kThreads, smem, stream>>>(tq, tk, tv, to, tkf, tvf, p);
    return cudaGetLastError();
}

}  // namespace uly
