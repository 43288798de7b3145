// The three matrix products of the fused LM-head loss on the 5th-generation
// tensor cores, one persistent kernel per product.
//
// A CTA pair owns a 256 x 256 output tile (fewer columns where D asks for it):
// each CTA loads its 128 rows of A and its 128 columns of B (TMA, 128-byte
// swizzle), one thread of the pair issues tcgen05.mma.cta_group::2 (M = 256, N =
// 256), and each CTA's TMEM holds 128 rows of the fp32 result, twice, so that
// one tile is written out while the next is formed.  A pair reads half of what
// two single CTAs would: 64 bytes a clock and SM from L2 at full rate.  The
// operands come as they lie: a matrix whose rows run along the contraction is
// K-major, one whose rows run along the output (W in dh; e and h in dW) is
// MN-major.
//
// Measured (5,734 rows with labels, D = 2560, V = 151,936, bf16): logits 2.52
// ms, dh 2.54, dW 2.47, that is 1.75 to 1.81 PFLOP/s against 1.90 of the
// library's product in a burst; back to back the card's power limit sets the
// clock (the same products of a constant matrix take 2.1 ms).  At D = 776 and V =
// 50,257 (4,830 rows) the tensor cores are busy 0.64 to 0.76 of 289, 287 and 277
// us: a step of 64 brings 32 KB to every SM, which at 64 bytes a clock takes the
// 512 clocks of its products.  With half the products issued the three take 269,
// 311 and 252 us, with half the loads 251, 242 and 248; narrower tiles (224
// columns) and a sixth stage change nothing.
//
// Warps 0-15 write results out (TMEM lane quarter warp % 4, columns 64 (warp /
// 4) ..): the logits' exponentials take longer than a short contraction's
// products, and four warps a scheduler hide each other's latencies where two
// do not.  Warp 16 loads, warp 17 issues products.
//
// Tiles beyond the last full round over the pairs are split along the
// contraction when that saves more than joining them costs: each into as many
// equal runs as there are pairs for, every pair leaves its fp32 tile in
// `partial`, and a second kernel adds the runs in order.  The pairs on one run
// of neighbouring tiles read the same panels at the same time; an even spread
// of all steps over all pairs, which lets them drift apart, took 415 us where
// no split took 251 (dh of 4,500 rows, 72 tiles on 76 pairs, D = 776, V =
// 50,257), since every tile then reads its panels from DRAM.  The split depends
// on the sizes and the number of good rows alone, so results repeat bit for bit.
//
// The tensor cores' accumulation rounds toward zero: a sum shrinks by up to
// 2^-24 of itself with every instruction (16 values of the contraction).  Over
// D = 2560 that moved the loss by 2.2e-6 of its value, over V = 151936 it
// would move dh by 4e-4.  So an accumulator is taken out of TMEM after
// kChunkSteps steps and summed in registers, with ordinary rounding, while the
// next one fills: after 512 values for the logits, whose error the loss shows
// undiminished, after 4096 for the gradients, which are rounded to bf16.
//
// fp32 (kSplit): every operand is three bf16 planes (x = x1 + x2 + x3 up to
// 2^-26 of x) and a product is the six plane products above 2^-24, smallest
// first; an accumulator takes 64 values of the contraction (24 instructions).  A
// step's planes are loaded once for all six: the first two of A and B have two
// stages, the third, which the first two products alone use, one.  With loads of
// their own for every product the call of 2048 rows x 1024 x 32,000 took 1.54 ms
// instead of 1.32, 4096 x 2048 x 32,000 5.94 instead of 5.10.
#include <atomic>

#include "linear_ce.h"

namespace uly {
namespace {

constexpr int kStages = 5;
constexpr int kHalf = 128;                               // rows of A, columns of B per CTA
constexpr int kOperandBytes = kHalf * kCeStep * 2;       // 16 KB
constexpr int kStageBytes = 2 * kOperandBytes;           // this CTA's part
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kCols = kCeStatCols;                       // columns per writing warp
constexpr int kWarpStaging = 32 * 128;                   // 32 rows of 128 bytes
constexpr int kBars = 2 * kStages + 5;
constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kWarpStaging + 8 * kBars + 16 + 1024;
constexpr int kThird = 2;  // fp32: barrier of the third planes' stage, behind those of the two other stages
constexpr int kCeMaxDevices = 64;
// Least steps of a run, and steps a split must save: a step takes 0.34 us (fp32:
// six products, 2 us), the runs' tiles and the join 10 to 20 us.  Whole calls
// with a gain of 32 / 64 / 128, us: 300 rows x 2048 x 5000 62 / 74 / 72, 1180 x 496
// x 3440 52 / 57 / 57, 256 x 352 x 6410 43 / 43 / 64, 6765 x 200 x 3208 110 / 103 /
// 111; in fp32 with runs of 2 and a gain of 12 / 8 and 32: 32 rows x 256 x 1000
// 52 / 78, 32 x 1096 x 1656 84 / 129, 3000 x 448 x 2000 146 / 178.
__host__ __device__ constexpr int min_run(bool split) { return split ? 2 : 8; }
__host__ __device__ constexpr int split_gain(bool split) { return split ? 12 : 32; }

static_assert(kStages * 2 >= 10 && kStages > kThird, "fp32: ten operands of a step and the next");

template <int kWhat, bool kSplit>
constexpr int kChunkSteps = kSplit ? 1 : (kWhat == kCeLogits ? 8 : 64);

// ------------------------------------------------------------- schedule
struct Plan {
    int mt, nt, kb;   // tiles along the rows and columns of the result, steps of the contraction
    int cols;         // columns of a tile
    int whole;        // tiles [0, whole) are done by one pair each
    int rem, runs;    // the others, each in so many runs (0: none)
};

// Runs of each of the tiles left over from full rounds; 0: those are done whole too.
__host__ __device__ inline int ce_runs(int64_t tiles, int kb, int pairs, bool split)
{
    const int rem = static_cast<int>(tiles % pairs);
    if (rem == 0)
        return 0;
    int runs = pairs / rem;
    runs = runs < kb / min_run(split) ? runs : kb / min_run(split);
    return runs > 1 && kb - kb / runs > split_gain(split) ? runs : 0;
}

template <int kWhat, bool kSplit>
__device__ __forceinline__ Plan make_plan(const CeArgs &a, int cnt, int pairs)
{
    Plan p;
    const int M = kWhat == kCeDw ? a.V : cnt, N = kWhat == kCeLogits ? a.V : a.D;
    const int K = kWhat == kCeLogits ? a.D : (kWhat == kCeDh ? a.V : cnt);
    p.mt = (M + kCeTile - 1) / kCeTile;
    p.kb = (K + kCeStep - 1) / kCeStep;
    p.nt = (N + kCeTile - 1) / kCeTile;
    // D in equal tiles: 776 as four of 224 instead of three of 256 and one of 8 (of
    // 208, whose rows start off 64 bytes, 2 % slower)
    p.cols = kWhat == kCeLogits ? kCeTile : ((N + p.nt - 1) / p.nt + 31) / 32 * 32;
    const int tiles = p.mt * p.nt;
    p.runs = kWhat == kCeLogits ? 0 : ce_runs(tiles, p.kb, pairs, kSplit);  // a softmax needs whole sums
    p.rem = p.runs > 0 ? tiles % pairs : 0;
    p.whole = tiles - p.rem;
    return p;
}

// One tile, or a run of a tile's steps, in the order a pair takes them.  The
// loader, the issuer and the writers walk the same list.
struct Unit {
    int tile, k0, k1;
    bool part;  // a run: its tile goes to the pair's place in `partial`
};

struct Units {
    Plan p;
    int pair, pairs, next_tile;
    bool run;  // the pair's run is still to come

    __device__ Units(const Plan &plan, int pair_, int pairs_)
        : p(plan), pair(pair_), pairs(pairs_), next_tile(pair_), run(pair_ < plan.rem * plan.runs)
    {
    }
    __device__ __forceinline__ bool next(Unit &u)
    {
        if (next_tile < p.whole) {
            u = Unit{next_tile, 0, p.kb, false};
            next_tile += pairs;
            return true;
        }
        if (!run)
            return false;
        run = false;
        const int r = pair / p.rem;
        u = Unit{p.whole + pair - r * p.rem, static_cast<int>(static_cast<int64_t>(p.kb) * r / p.runs),
                 static_cast<int>(static_cast<int64_t>(p.kb) * (r + 1) / p.runs), true};
        return true;
    }
};

// Tile order.  Logits: rows fastest, so that a round over the pairs reads a
// few column panels of W once against all rows, which stay in L2.  dh and dW:
// columns (D) fastest, so that e, the large operand, is read once a round.
template <int kWhat>
__device__ __forceinline__ void tile_origin(const Plan &p, int tile, int &m0, int &n0)
{
    if (kWhat == kCeLogits) {
        n0 = tile / p.mt * p.cols;
        m0 = tile % p.mt * kCeTile;
    } else {
        m0 = tile / p.nt * kCeTile;
        n0 = tile % p.nt * p.cols;
    }
}

// A tile's fp32 values in memory, as the writers hold them: per CTA and warp
// 16 groups of 4 columns, each 32 rows x 16 bytes, so that a warp's access is
// 512 bytes in a row.
__device__ __forceinline__ float4 *tile_slot(float *buf, int64_t slot, int cta, int warp, int lane,
                                             [[maybe_unused]] int64_t slots, [[maybe_unused]] unsigned *status)
{
    if (!ULY_IN_BOUNDS(status, slot, 1, slots, 0x64))
        slot = 0;  // there is one where there is a slot to ask for
    return reinterpret_cast<float4 *>(buf + slot * kCeTileFloats) + (cta * kEpiWarps + warp) * (kCols / 4 * 32) + lane;
}

// ------------------------------------------------------------ writing out
// 16 bytes of a row: four fp32 values or eight bf16 ones.
template <bool kF32>
__device__ __forceinline__ uint4 unit(const float *v)
{
    if constexpr (kF32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
}

// The warp's 32 rows x 64 columns (row = lane) to memory, 128 bytes of a row
// per 8 lanes: through shared memory, units of 16 bytes permuted within the
// row so that neither side meets a bank conflict.  row: where this lane's row
// goes, negative: nowhere; the tensor has `rows`.  Columns from `limit` on are not
// written (a multiple of 16 bytes).
template <bool kF32>
__device__ __forceinline__ void store_rows(const float (&x)[kCols], void *out, int row, [[maybe_unused]] int64_t rows,
                                           int64_t pitch, int col0, int limit, uint8_t *staging, int lane,
                                           [[maybe_unused]] unsigned *status)
{
    constexpr int kPer = kF32 ? 4 : 8;  // values per unit
#pragma unroll
    for (int part = 0; part < kCols / (8 * kPer); ++part) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            *reinterpret_cast<uint4 *>(staging + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                unit<kF32>(x + (part * 8 + u) * kPer);
        }
        __syncwarp();
        const int u = lane & 7, col = col0 + (part * 8 + u) * kPer;
        uint8_t *to = static_cast<uint8_t *>(out) + static_cast<int64_t>(col) * (16 / kPer);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), at = __shfl_sync(0xffffffffu, row, r);
            const uint4 val = *reinterpret_cast<const uint4 *>(staging + r * 128 + ((u ^ (r & 7)) << 4));
            if (at >= 0 && col < limit && ULY_IN_BOUNDS(status, at * pitch + col, kPer, rows * pitch, 0x61))
                *reinterpret_cast<uint4 *>(to + at * (pitch * (16 / kPer))) = val;
        }
        __syncwarp();
    }
}

// The exponentials to their buffer by TMA, a box of 32 rows x 64 columns in the
// swizzled layout of the map, in fp32 one for each plane.
template <bool kSplit>
__device__ __forceinline__ void store_exponentials(const CeArgs &a, const CUtensorMap *te, float (&x)[kCols], int row0,
                                                   int col0, uint8_t *staging, int lane)
{
#pragma unroll
    for (int plane = 0; plane < (kSplit ? 3 : 1); ++plane) {
        if (lane == 0)
            bulk_wait_read<0>();  // what was staged before is on its way
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint4 q = unit<false>(x + u * 8);
            *reinterpret_cast<uint4 *>(staging + lane * 128 + ((u ^ (lane & 7)) << 4)) = q;
            if (kSplit && plane < 2) {  // what is left for the next planes
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[u * 8 + 2 * i] -= __uint_as_float(w[i] << 16);
                    x[u * 8 + 2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(te, staging, col0, plane * a.rows + row0);
            bulk_commit();
        }
    }
}

// Logits: the row's sum of e = 2^(x log2 e - c) over this warp's columns, its
// target's logit, and e itself.  c is 0 as long as the columns' largest x log2 e
// lies within kCeFree of it, otherwise that maximum, rounded so that another
// c changes e by a power of two alone.  The rows between the piece's last and the
// end of its step of 64 have h = 0 and leave e = 1, finite values that meet zeros
// in dW.
template <bool kSplit>
__device__ __forceinline__ void finish_logits(const CeArgs &a, const CUtensorMap *te, float (&x)[kCols], int cnt, int m,
                                              int col0, uint8_t *staging, int lane)
{
    if (col0 >= a.V || m - lane >= (cnt + kCeStep - 1) / kCeStep * kCeStep)
        return;
    const bool live = m < cnt;
    const int y = live ? a.label[m] : -1;
    if (y >= col0 && y < col0 + kCols && ULY_IN_BOUNDS(a.status, m, 1, a.rows, 0x62)) {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (y == col0 + j)
                a.target[m] = x[j];
    }
    if (col0 + kCols > a.V) {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (col0 + j >= a.V)
                x[j] = -INFINITY;
    }
    float pm[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        pm[j] = x[j];
#pragma unroll
    for (int j = 8; j < kCols; ++j)
        pm[j & 7] = fmaxf(pm[j & 7], x[j]);
    const float top = kLog2e * fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])),
                                     fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7])));
    // columns of -inf alone have no maximum to take out: their exponentials are 0
    const float c = fabsf(top) <= kCeFree ? 0.f : rintf(top), out = c == -INFINITY ? 0.f : -c;
    const float2 l2 = make_float2(kLog2e, kLog2e), c2 = make_float2(out, out);
    float2 ps[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < kCols; j += 2) {
        const float2 t = ffma2(make_float2(x[j], x[j + 1]), l2, c2);
        x[j] = ex2_approx(t.x);
        x[j + 1] = ex2_approx(t.y);
        ps[(j >> 1) & 3] = fadd2(ps[(j >> 1) & 3], make_float2(x[j], x[j + 1]));
    }
    const float2 s = fadd2(fadd2(ps[0], ps[1]), fadd2(ps[2], ps[3]));
    const int64_t stat = static_cast<int64_t>(m) * a.stat_tiles + col0 / kCeStatCols;
    if (live && ULY_IN_BOUNDS(a.status, stat, 1, static_cast<int64_t>(a.rows) * a.stat_tiles, 0x63))
        a.stats[stat] = make_float2(c, s.x + s.y);
    if (a.keep)
        store_exponentials<kSplit>(a, te, x, m - lane, col0, staging, lane);
}

// Where row m of dh (its place in hidden) or dW goes; negative past the end.
template <int kWhat>
__device__ __forceinline__ int grad_row(const CeArgs &a, int cnt, int m)
{
    if (m >= (kWhat == kCeDh ? cnt : a.V))
        return -1;
    return kWhat == kCeDh ? a.index[a.base + m] : m;
}

// What row m of the result is multiplied by: 1 / T, and in dh the softmax's 1 / S.
template <int kWhat>
__device__ __forceinline__ float grad_scale(const CeArgs &a, int cnt, int m)
{
    const int n = *a.n_good;
    const float inv = 1.f / static_cast<float>(n > 1 ? n : 1);
    return kWhat == kCeDh ? (m < cnt ? inv * a.row_scale[m] : 0.f) : inv;
}

// kN bf16 values of a row, from column col0 on, times f; `row` may end within them.
template <int kN>
__device__ __forceinline__ void add_scaled(float *x, float f, const uint16_t *row, int col0, int D)
{
    constexpr int kOnce = kN < 16 ? kN : 16;  // registers are short: more loads on their way spill
#pragma unroll
    for (int j0 = 0; j0 < kN; j0 += kOnce) {
        uint4 q[kOnce / 8];
#pragma unroll
        for (int j = 0; j < kOnce; j += 8)
            q[j / 8] = col0 + j0 + j < D ? *reinterpret_cast<const uint4 *>(row + col0 + j0 + j)
                                         : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kOnce; j += 8)
            add_scaled8(x + j0 + j, f, q[j / 8]);
    }
}

// The label's term of a row of dh, l w_y / T, for kN columns (bf16).
struct LabelWord {
    int64_t at;  // of w_y
    float f;     // l / T; 0 where there is no row

    __device__ __forceinline__ LabelWord(const CeArgs &a, int cnt, int m)
    {
        const int n = *a.n_good;
        at = m < cnt ? static_cast<int64_t>(a.label[m]) * a.D : 0;
        f = m < cnt ? a.label_grad[m] / static_cast<float>(n > 1 ? n : 1) : 0.f;
        if (!ULY_IN_BOUNDS(a.status, at, a.D, static_cast<int64_t>(a.V) * a.D, 0x65))
            at = 0;
    }
    template <int kN>
    __device__ __forceinline__ void add(const CeArgs &a, float *x, int col0) const
    {
        if (f != 0.f)
            add_scaled<kN>(x, f, a.weight + at, col0, a.D);
    }
};

// The labels' terms of dW (bf16): to word m0 + lane the rows r with that label
// among [r0, r1) (multiples of 64, a chunk of the contraction) give l_r h_r, those of
// a group of kCeGroup rows in one.  Which rows concern the warp's 32 words is marked
// by a bit each, 1024 rows to a load.  Their places, as offsets to r0, are listed for
// each word in the warp's staging memory while the products run; then each lane
// takes its own, so that as many rows' loads are on their way as words have one.
// dW of 5,734 rows of 151,936 takes 2 % longer with these terms, 11 % where every
// label was read instead of the marks: 23 KB a tile and warp, into an SM whose
// operands already fill its way to L2.
constexpr int kListed = kCeAlone * (kChunkSteps<kCeDw, false> * kCeStep / kCeGroup + 1);
static_assert(kListed * 64 + 128 <= kWarpStaging, "lists and their lengths");
struct LabelRows {
    uint16_t *list;  // [kListed][32]
    int *count;      // [32]

    __device__ __forceinline__ explicit LabelRows(uint8_t *staging)
        : list(reinterpret_cast<uint16_t *>(staging + 128)), count(reinterpret_cast<int *>(staging))
    {
    }
    __device__ __noinline__ void collect(const CeArgs &a, int m0, int r0, int r1, int lane) const
    {
        const uint32_t *marks = a.marks + static_cast<int64_t>(m0 / 32) * a.mark_pitch;
        count[lane] = 0;
        __syncwarp();
        for (int w0 = r0 / 32; w0 < r1 / 32; w0 += 32) {
            // each lane has the marks of 32 rows and takes them one by one
            uint32_t mark = w0 + lane < r1 / 32 ? marks[w0 + lane] : 0;
            while (__any_sync(0xffffffffu, mark != 0)) {
                const bool live = mark != 0;
                const int row = (w0 + lane) * 32 + __ffs(mark) - 1;
                const int word = live ? a.label[row] - m0 : -1;
                const unsigned same = __match_any_sync(0xffffffffu, word);
                const int before = __popc(same & ((1u << lane) - 1));
                const int place = live ? count[word] + before : 0;
                __syncwarp();
                if (live) {
                    list[place * 32 + word] = static_cast<uint16_t>(row - r0);
                    if (before == 0)
                        count[word] += __popc(same);
                }
                __syncwarp();
                mark &= mark - 1;
            }
        }
    }
    __device__ __forceinline__ void take(const CeArgs &a, float (&x)[kCols], int r0, int col0, int lane) const
    {
        const int n = count[lane];
        for (int i = 0; i < n; ++i) {
            const int r = r0 + list[i * 32 + lane], slot = a.label_slot[r];
            const float l = a.label_grad[r];
            if (!ULY_IN_BOUNDS(a.status, slot < 0 ? ~slot : slot, 1, slot < 0 ? a.all_rows : a.places, 0x66))
                continue;
            if (slot < 0) {
                add_scaled<kCols>(x, l, a.hidden + static_cast<int64_t>(~slot) * a.D, col0, a.D);
            } else {
                const float *sum = a.label_sum + static_cast<int64_t>(slot) * a.D + col0;
                constexpr int kOnce = 8;
#pragma unroll
                for (int j0 = 0; j0 < kCols; j0 += kOnce) {
                    float4 v[kOnce / 4];
#pragma unroll
                    for (int j = 0; j < kOnce; j += 4)
                        v[j / 4] = col0 + j0 + j < a.D ? *reinterpret_cast<const float4 *>(sum + j0 + j)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < kOnce; j += 4) {
                        x[j0 + j] += v[j / 4].x, x[j0 + j + 1] += v[j / 4].y;
                        x[j0 + j + 2] += v[j / 4].z, x[j0 + j + 3] += v[j / 4].w;
                    }
                }
            }
        }
        __syncwarp();
    }
};

// dh and dW: scaled and rounded once.  dW over several pieces is kept
// in fp32 until the last one.
template <int kWhat, bool kSplit>
__device__ __forceinline__ void finish_grad(const CeArgs &a, float (&x)[kCols], int cnt, int tile, int m, int col0,
                                            int cta, int warp, int limit, const LabelWord &word, uint8_t *staging,
                                            int lane)
{
    if (kWhat == kCeDw && a.base > 0) {
        const float4 *acc = tile_slot(a.acc, tile, cta, warp, lane, a.acc_slots, a.status);
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j) {
            const float4 v = acc[j * 32];
            x[4 * j] += v.x, x[4 * j + 1] += v.y, x[4 * j + 2] += v.z, x[4 * j + 3] += v.w;
        }
    }
    if (kWhat == kCeDw && a.base + a.rows < *a.n_good) {
        float4 *acc = tile_slot(a.acc, tile, cta, warp, lane, a.acc_slots, a.status);
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j)
            acc[j * 32] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        return;
    }
    const float inv = grad_scale<kWhat>(a, cnt, m);
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        x[j] *= inv;
    if (kWhat == kCeDh && !kSplit && col0 < limit)
        word.add<kCols>(a, x, col0);
    store_rows<kSplit>(x, kWhat == kCeDh ? a.dh : a.dw, grad_row<kWhat>(a, cnt, m), kWhat == kCeDh ? a.all_rows : a.V,
                       a.D, col0, min(limit, a.D), staging, lane, a.status);
}

// The call's totals by one warp alone.
__device__ __noinline__ void totals_by_warp(const CeTotals &t)
{
    for (int r = 0; r < t.P; ++r) {
        const float *base = t.row_loss + r * t.per_shard;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int64_t i = lane_id(); i < t.per_shard; i += 32)
            s = two_sum(s, make_float2(base[i], 0.f));
        ce_shard(t, r, warp_two_sum(s));
    }
    ce_total(t);
}

template <int kWhat, bool kSplit>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ce_product_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                      const __grid_constant__ CUtensorMap te, const __grid_constant__ CeArgs a, const WaitCfg w)
{
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint8_t *staging = smem + kStages * kStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + kEpiWarps * kWarpStaging);
    uint64_t *empty = full + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(drain + 1);
    volatile uint32_t *abort_flag = tmem_ptr + 1;
    const int warp = warp_id(), lane = lane_id();
    const int cta = static_cast<int>(cluster_ctarank());
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kEpiWarps) {
        if (lane == 0) {
            prefetch_tmap(&ta);
            prefetch_tmap(&tb);
        }
        __syncwarp();
        tmem_alloc_pair(tmem_ptr, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the other CTA's barriers are set up
    tc_fence_after();
    const uint32_t tbase = *tmem_ptr;
    grid_wait();
    grid_next();
    const int cnt = ce_piece_rows(a);
    Plan plan = make_plan<kWhat, kSplit>(a, cnt, pairs);
    if (cnt == 0 && (kWhat != kCeDw || a.base > 0))
        plan.whole = plan.rem = 0;  // nothing to do; dW without any row is written as zeros by the first piece
    // a narrow MN-major B: one block of 64 columns per CTA instead of two
    const bool second_block = plan.cols / 2 > 64;
    const uint32_t b_bytes = second_block ? kOperandBytes : kOperandBytes / 2;

    if (warp == kEpiWarps) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            // A step's instructions are what a pair can lose time on: one
            // thread loads and one issues, and a step of 64 is 512 cycles of
            // products.  So stages and parities are counted, addresses kept.
            const uint32_t bar0 = cluster_addr(&full[0], 0);
            auto ready = [&](int i, uint32_t par) {
                return mbar_try_wait(&empty[i], par) || (!*abort_flag && mbar_wait(&empty[i], par, w, 0xa1));
            };
            auto load_a = [&](uint8_t *to, uint32_t bar, int m, int kc, int plane) {
                if (kWhat == kCeDw) {
                    tma_load_3d_pair(to, &ta, bar, m, kc, plane);
                    tma_load_3d_pair(to + kOperandBytes / 2, &ta, bar, m + 64, kc, plane);
                } else {
                    tma_load_3d_pair(to, &ta, bar, kc, m, plane);
                }
            };
            auto load_b = [&](uint8_t *to, uint32_t bar, int n, int kc, int plane) {
                if (kWhat != kCeLogits) {
                    tma_load_3d_pair(to, &tb, bar, n, kc, plane);
                    if (second_block)
                        tma_load_3d_pair(to + kOperandBytes / 2, &tb, bar, n + 64, kc, plane);
                } else {
                    tma_load_3d_pair(to, &tb, bar, kc, n, plane);
                }
            };
            Units units(plan, pair, pairs);
            Unit u;
            uint32_t it = 0, s = 0, parity = 1;
            bool ok = true;
            while (ok && units.next(u)) {
                int m0, n0;
                tile_origin<kWhat>(plan, u.tile, m0, n0);
                m0 += cta * kHalf;
                n0 += cta * (plan.cols / 2);
                for (int k = u.k0; ok && k < u.k1; ++k) {
                    const int kc = k * kCeStep;
                    if constexpr (kSplit) {
                        ok = ready(s, parity);
                        if (!ok)
                            break;
                        if (cta == 0)
                            mbar_expect_tx(&full[s], 4 * (kOperandBytes + b_bytes));
                        for (int plane = 0; plane < 2; ++plane) {
                            uint8_t *to = smem + (4 * s + 2 * plane) * kOperandBytes;
                            load_a(to, bar0 + 8 * s, m0, kc, plane);
                            load_b(to + kOperandBytes, bar0 + 8 * s, n0, kc, plane);
                        }
                        ok = ready(kThird, (it & 1) ^ 1);
                        if (!ok)
                            break;
                        if (cta == 0)
                            mbar_expect_tx(&full[kThird], 2 * (kOperandBytes + b_bytes));
                        load_a(smem + 8 * kOperandBytes, bar0 + 8 * kThird, m0, kc, 2);
                        load_b(smem + 9 * kOperandBytes, bar0 + 8 * kThird, n0, kc, 2);
                        ++it;
                        s ^= 1;
                        parity ^= s == 0;
                    } else {
                        ok = ready(s, parity);
                        if (!ok)
                            break;
                        if (cta == 0)
                            mbar_expect_tx(&full[s], 2 * (kOperandBytes + b_bytes));
                        uint8_t *to = smem + s * kStageBytes;
                        load_a(to, bar0 + 8 * s, m0, kc, 0);
                        load_b(to + kOperandBytes, bar0 + 8 * s, n0, kc, 0);
                        ++it;
                        if (++s == kStages) {
                            s = 0;
                            parity ^= 1;
                        }
                    }
                }
            }
            // the last uses of the stages: their releases arrive from CTA 0, and this CTA stays until they have
            constexpr uint32_t ring = kSplit ? 2 : kStages;
            const uint32_t last = it > ring ? it - ring : 0;
            for (uint32_t i = last; ok && i < it; ++i)
                ok = mbar_wait(&empty[i % ring], (i / ring) & 1, w, 0xa6);
            if (kSplit && ok && it > 0)
                ok = mbar_wait(&empty[kThird], (it - 1) & 1, w, 0xa6);
            if (!ok) {
                *abort_flag = 1;
                // wait (bounded) for the loads still in flight; CTA 0 holds their barriers
                if (cta == 0) {
                    for (uint32_t i = last; i < it; ++i)
                        mbar_wait(&full[i % ring], (i / ring) & 1, w, 0xaf);
                    if (kSplit)  // and the step that was begun
                        mbar_wait(&full[s], parity ^ 1, w, 0xaf);
                    if (kSplit && it > 0)
                        mbar_wait(&full[kThird], (it - 1) & 1, w, 0xaf);
                }
            }
            // CTA 1 has followed the products up to here, so that this wait, too, is short
            if (cta == 1)
                mbar_wait(drain, 0, w, 0xa4);
        }
    } else if (warp == kEpiWarps + 1) {
        // ------------------------------------------------ products
        if (lane == 0 && cta == 0) {
            const uint32_t idesc = idesc_bf16(256, plan.cols, kWhat == kCeDw, kWhat != kCeLogits);
            Units units(plan, pair, pairs);
            Unit u;
            uint32_t s = 0, parity = 0, chunk = 0;
            // A and B of a step's first instruction, were they at the ring's start
            const uint64_t da0 = kWhat == kCeDw ? desc_sw128(smem_u32(smem), kOperandBytes / 2, 1024)
                                                : desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t db0 = kWhat != kCeLogits ? desc_sw128(smem_u32(smem), kOperandBytes / 2, 1024)
                                                    : desc_sw128(smem_u32(smem), 16, 1024);
            auto multiply = [&](uint32_t d, uint64_t da, uint64_t db, bool add) {
                constexpr uint32_t a_next = (kWhat == kCeDw ? 2048 : 32) / 16;
                constexpr uint32_t b_next = (kWhat != kCeLogits ? 2048 : 32) / 16;
#pragma unroll
                for (int kk = 0; kk < kCeStep / 16; ++kk)
                    mma_ss_pair(d, da + kk * a_next, db + kk * b_next, idesc, (add || kk > 0) ? 1u : 0u);
            };
            constexpr uint32_t slot = kOperandBytes / 16;
            uint32_t third = 0;  // parity
            bool ok = true;
            while (ok && units.next(u)) {
                int left = u.k1 - u.k0;  // steps of this unit
                while (ok && left > 0) {
                    constexpr int most = kChunkSteps<kWhat, kSplit>;
                    const int n = left < most ? left : most;  // steps of this accumulation
                    const uint32_t acc = chunk & 1, d = tbase + acc * 256;
                    if (*abort_flag || !mbar_wait_cluster(&acc_empty[acc], ((chunk >> 1) & 1) ^ 1, w, 0xa2)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int i = 0; i < n; ++i) {
                        ok = mbar_wait(&full[s], parity, w, 0xa3) &&
                             (!kSplit || mbar_wait(&full[kThird], third, w, 0xa3));
                        if (!ok)
                            break;
                        tc_fence_after();
                        if constexpr (kSplit) {
                            const uint64_t a1 = da0 + 4 * s * slot, b1 = db0 + (4 * s + 1) * slot;
                            const uint64_t a2 = a1 + 2 * slot, b2 = b1 + 2 * slot;
                            multiply(d, a1, db0 + 9 * slot, i > 0);
                            multiply(d, da0 + 8 * slot, b1, true);
                            mma_commit_pair(&empty[kThird]);
                            third ^= 1;
                            multiply(d, a2, b2, true);
                            multiply(d, a1, b2, true);
                            multiply(d, a2, b1, true);
                            multiply(d, a1, b1, true);
                            mma_commit_pair(&empty[s]);
                            s ^= 1;
                            parity ^= s == 0;
                        } else {
                            multiply(d, da0 + 2 * s * slot, db0 + (2 * s + 1) * slot, i > 0);
                            mma_commit_pair(&empty[s]);
                            if (++s == kStages) {
                                s = 0;
                                parity ^= 1;
                            }
                        }
                    }
                    if (!ok)
                        break;
                    mma_commit_pair(&acc_full[acc]);
                    ++chunk;
                    left -= n;
                }
            }
            if (!ok)
                *abort_flag = 1;
            mma_commit_pair(drain);
        }
        if (kWhat != kCeLogits && cta == 1 && pair == 0 && a.make_totals)
            totals_by_warp(a.totals);  // this CTA's issuer has nothing else to do
        __syncwarp();
        if (lane == 0 && cta == 0)
            mbar_wait(drain, 0, w, 0xa4);  // every product and release is through
    } else {
        // ------------------------------------------------ results
        Units units(plan, pair, pairs);
        Unit u;
        uint32_t chunk = 0;
        const int col = (warp >> 2) * kCols;
        uint8_t *stage = staging + warp * kWarpStaging;
        bool ok = true;
        while (ok && units.next(u)) {
            int m0, n0;
            tile_origin<kWhat>(plan, u.tile, m0, n0);
            const int m = m0 + cta * kHalf + (warp & 3) * 32 + lane;
            float x[kCols];
            constexpr int per = kChunkSteps<kWhat, kSplit>;
            const int chunks = (u.k1 - u.k0 + per - 1) / per;
            if (chunks == 0) {
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    x[j] = 0.f;
            }
            [[maybe_unused]] LabelWord word(a, kWhat == kCeDh && !kSplit && !u.part ? cnt : 0, m);
            const bool words = kWhat == kCeDw && !kSplit && m - lane < a.V && col < plan.cols && n0 + col < a.D;
            for (int c = 0; c < chunks; ++c, ++chunk) {
                const uint32_t acc = chunk & 1;
                const int r0 = (u.k0 + c * per) * kCeStep;  // dW: the chunk's first row
                const LabelRows rows(stage);
                if (words)  // while the products run
                    rows.collect(a, m - lane, r0, min(r0 + per * kCeStep, u.k1 * kCeStep), lane);
                if (!mbar_wait_warp(&acc_full[acc], (chunk >> 1) & 1, w, 0xa5)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t = tbase + acc * 256 + col + (static_cast<uint32_t>((warp & 3) * 32) << 16);
                if (c == 0) {
                    uint32_t *v = reinterpret_cast<uint32_t *>(x);
#pragma unroll
                    for (int j = 0; j < kCols; j += 32)
                        tmem_ld32p(t + j, v + j);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < kCols; j += 32)
                        tmem_ld_fence32p(v + j);
                } else {
#pragma unroll
                    for (int j = 0; j < kCols; j += 16) {
                        uint32_t v[16];
                        tmem_ld16_wait(t + j, v);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 s = fadd2(make_float2(x[j + i], x[j + i + 1]),
                                                   make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                            x[j + i] = s.x;
                            x[j + i + 1] = s.y;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster_relaxed(cluster_addr(&acc_empty[acc], 0));
                if (words)
                    rows.take(a, x, r0, n0 + col, lane);
            }
            if (!ok)
                break;
            if (u.part) {
                if (kWhat == kCeDh && m - lane >= cnt)
                    continue;  // nobody reads these rows
                float4 *slot = tile_slot(a.partial, pair, cta, warp, lane, a.partial_slots, a.status);
#pragma unroll
                for (int j = 0; j < kCols / 4; ++j)
                    slot[j * 32] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            } else if constexpr (kWhat == kCeLogits) {
                finish_logits<kSplit>(a, &te, x, cnt, m, n0 + col, stage, lane);
            } else {
                finish_grad<kWhat, kSplit>(a, x, cnt, u.tile, m, n0 + col, cta, warp, n0 + plan.cols, word, stage,
                                           lane);
            }
        }
        if (!ok)
            *abort_flag = 1;
        if (kWhat == kCeLogits && lane == 0)
            bulk_wait_read<0>();  // staged rows are read before the CTA's shared memory goes
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs are done with each other's memory and TMEM
    tc_fence_after();
    if (warp == kEpiWarps)
        tmem_dealloc_pair(tbase, 512);
}

// Adds the runs of the split tiles, in the order of the contraction.  An item
// is 32 rows x 64 columns of one tile: a warp takes 8 columns (fp32: 4; one
// 16-byte store a row) of one of kGroups shares of the runs, and the shares'
// sums are added in order.  Where a few tiles are split, each into dozens of
// runs, 1024 threads share them out (12 rows, D = 112, V = 138,259: the whole
// call 76 us, with one group 91); where dozens are, each has two or three runs
// and one group will do (28 tiles: 9 us, with four groups 22).
template <bool kSplit>
constexpr int kJoinCols = kSplit ? 4 : 8;
template <bool kSplit>
constexpr int kJoinGroups = kSplit ? 2 : 4;
template <bool kSplit, int kGroups>
constexpr int kJoinThreads = kGroups * (kCols / kJoinCols<kSplit>) * 32;
template <int kWhat, bool kSplit, int kGroups>
__global__ void __launch_bounds__(kJoinThreads<kSplit, kGroups>) ce_join_kernel(const __grid_constant__ CeArgs a,
                                                                               int pairs)
{
    constexpr int kPart = kJoinCols<kSplit>, kVecs = kPart / 4, kParts = kCols / kPart;
    static_assert(kJoinThreads<kSplit, kGroups> <= 1024, "a block");
    __shared__ float sums[kGroups > 1 ? kGroups - 1 : 1][kParts][kPart][32];
    grid_wait();
    grid_next();
    const int cnt = ce_piece_rows(a);
    if (cnt == 0)
        return;
    const Plan p = make_plan<kWhat, kSplit>(a, cnt, pairs);
    const int part = warp_id() % kParts, group = warp_id() / kParts, lane = lane_id();
    for (int item = blockIdx.x; item < p.rem * 2 * kEpiWarps; item += gridDim.x) {
        const int slab = item % kEpiWarps, cta = item / kEpiWarps % 2, split = item / (2 * kEpiWarps);
        const int tile = p.whole + split;
        int m0, n0;
        tile_origin<kWhat>(p, tile, m0, n0);
        const int m_slab = m0 + cta * kHalf + (slab & 3) * 32, col = n0 + (slab >> 2) * kCols + part * kPart;
        const int limit = min(n0 + p.cols, a.D);
        if (m_slab >= (kWhat == kCeDh ? cnt : a.V) || n0 + (slab >> 2) * kCols >= limit)
            continue;  // the whole block agrees
        float x[kPart];
#pragma unroll
        for (int j = 0; j < kPart; ++j)
            x[j] = 0.f;
        const int each = (p.runs + kGroups - 1) / kGroups, r0 = group * each, r1 = min(p.runs, r0 + each);
#pragma unroll 4
        for (int r = r0; r < r1; ++r) {
            const float4 *slot = tile_slot(a.partial, r * p.rem + split, cta, slab, lane, a.partial_slots, a.status);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const float4 v = slot[(part * kVecs + j) * 32];
                x[4 * j] += v.x, x[4 * j + 1] += v.y, x[4 * j + 2] += v.z, x[4 * j + 3] += v.w;
            }
        }
        if constexpr (kGroups > 1) {
            __syncthreads();  // the last item's sums are read
            if (group > 0)
#pragma unroll
                for (int j = 0; j < kPart; ++j)
                    sums[group - 1][part][j][lane] = x[j];
            __syncthreads();
            if (group > 0)
                continue;
        }
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g)
#pragma unroll
            for (int j = 0; j < kPart; ++j)
                x[j] += sums[g][part][j][lane];
        const bool more = a.base + a.rows < *a.n_good;  // rows to come
        if (kWhat == kCeDw && (a.base > 0 || more)) {
            float4 *acc = tile_slot(a.acc, tile, cta, slab, lane, a.acc_slots, a.status) + part * kVecs * 32;
            if (a.base > 0)
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const float4 v = acc[j * 32];
                    x[4 * j] += v.x, x[4 * j + 1] += v.y, x[4 * j + 2] += v.z, x[4 * j + 3] += v.w;
                }
            if (more) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    acc[j * 32] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                continue;
            }
        }
        const int row = grad_row<kWhat>(a, cnt, m_slab + lane);
        const float inv = grad_scale<kWhat>(a, cnt, m_slab + lane);
#pragma unroll
        for (int j = 0; j < kPart; ++j)
            x[j] *= inv;
        if constexpr (kWhat == kCeDh && !kSplit) {
            if (col < limit)
                LabelWord(a, cnt, m_slab + lane).template add<kPart>(a, x, col);
        }
        if (row >= 0 && col < limit &&
            ULY_IN_BOUNDS(a.status, static_cast<int64_t>(row) * a.D + col, kSplit ? 4 : 8,
                          (kWhat == kCeDh ? a.all_rows : a.V) * a.D, 0x67))
            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(kWhat == kCeDh ? a.dh : a.dw) +
                                       (static_cast<int64_t>(row) * a.D + col) * (kSplit ? 4 : 2)) = unit<kSplit>(x);
    }
}

// --------------------------------------------------------------- host
bool encode(CUtensorMap *map, CUtensorMapDataType type, int esize, int rank, const void *base, int64_t cols,
            int64_t rows, int64_t pitch, int planes, int box_cols, int box_rows)
{
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                          static_cast<cuuint64_t>(planes)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * esize, static_cast<cuuint64_t>(pitch) * rows * esize};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return tensor_map_encoder()(map, type, rank, const_cast<void *>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Box of a K-major operand: 64 values of the contraction x 128 rows; of an
// MN-major one: 64 columns x 64 values of the contraction.
bool make_map(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t pitch, int planes, int box_rows)
{
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 3, base, cols, rows, pitch, planes, 64, box_rows);
}

// Box of the exponentials on their way out: 64 columns x 32 rows; the planes
// lie below each other.
bool make_exp_map(CUtensorMap *map, const CeArgs &a, int planes)
{
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 2, a.e, a.ldg, static_cast<int64_t>(a.rows) * planes, a.ldg,
                  1, 64, 32);
}

template <int kWhat, bool kSplit>
cudaError_t launch(const CeArgs &a, const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &te,
                   cudaStream_t s)
{
    auto kernel = ce_product_kernel<kWhat, kSplit>;
    // Pairs resident at once (the schedule gives each an equal share), asked
    // for once per device; two threads that ask at the same time find the same.
    static std::atomic<int> known[kCeMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kCeMaxDevices)
        return cudaErrorInvalidDevice;
    int pairs = known[dev].load();
    if (pairs == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess)
            return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (num_sms() / 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
        if (e != cudaSuccess)
            return e;
        pairs = std::max(1, std::min(std::min(pairs, num_sms() / 2), kCeMaxPairs));
        known[dev].store(pairs);
    }
    e = launch_after(kernel, 2 * pairs, kThreads, kSmem, s, ta, tb, te, a, wait_cfg());
    if constexpr (kWhat != kCeLogits) {
        // Most tiles that any number of good rows could leave to be joined: at
        // most half the pairs are (two runs each).  dW's tiles are known here,
        // and fewer rows shorten its contraction and split it less.
        const int K = kWhat == kCeDh ? a.V : a.rows, kb = (K + kCeStep - 1) / kCeStep;
        const int nt = (a.D + kCeTile - 1) / kCeTile;
        const int tiles = ((kWhat == kCeDh ? a.rows : a.V) + kCeTile - 1) / kCeTile * nt;
        int most = kb > split_gain(kSplit) ? std::min(tiles, pairs / 2) : 0;
        if (kWhat == kCeDw && ce_runs(tiles, kb, pairs, kSplit) == 0)
            most = 0;
        const int items = most * 2 * kEpiWarps;
        constexpr int kMany = kJoinGroups<kSplit>;
        if (e == cudaSuccess && items > 0)
            e = items <= 2 * num_sms()
                    ? launch_after(ce_join_kernel<kWhat, kSplit, kMany>, items, kJoinThreads<kSplit, kMany>, 0, s, a,
                                   pairs)
                    : launch_after(ce_join_kernel<kWhat, kSplit, 1>, std::min(items, 8 * num_sms()),
                                   kJoinThreads<kSplit, 1>, 0, s, a, pairs);
    }
    return e;
}

template <bool kSplit>
cudaError_t product(CeProduct what, const CeArgs &a, const void *h, int64_t ldh, const void *w, int64_t ldw,
                    cudaStream_t s)
{
    constexpr int planes = kSplit ? 3 : 1;
    CUtensorMap ta, tb, te = {};  // te: the logits' exponentials alone
    bool ok;
    switch (what) {
    case kCeLogits:
        ok = make_map(&ta, h, a.D, a.rows, ldh, planes, kHalf) &&
             make_map(&tb, w, a.D, a.V, ldw, planes, kHalf);
        ok = ok && (!a.keep || make_exp_map(&te, a, planes));
        return ok ? launch<kCeLogits, kSplit>(a, ta, tb, te, s) : cudaErrorInvalidValue;
    case kCeDh:
        ok = make_map(&ta, a.e, a.V, a.rows, a.ldg, planes, kHalf) && make_map(&tb, w, a.D, a.V, ldw, planes, kCeStep);
        return ok ? launch<kCeDh, kSplit>(a, ta, tb, te, s) : cudaErrorInvalidValue;
    default:
        ok = make_map(&ta, a.e, a.V, a.rows, a.ldg, planes, kCeStep) &&
             make_map(&tb, h, a.D, a.rows, ldh, planes, kCeStep);
        return ok ? launch<kCeDw, kSplit>(a, ta, tb, te, s) : cudaErrorInvalidValue;
    }
}

}  // namespace

int ce_most_parts(CeProduct what, int rows, int D, int V, int esize)
{
    const int64_t mt = ((what == kCeDw ? V : rows) + kCeTile - 1) / kCeTile, nt = (D + kCeTile - 1) / kCeTile;
    const int64_t kb = ((what == kCeDw ? rows : V) + kCeStep - 1) / kCeStep;
    const bool split = esize == 4;
    if (kb <= split_gain(split))
        return 0;
    return static_cast<int>(std::min<int64_t>(kCeMaxPairs, mt * nt * (kb / min_run(split))));
}

cudaError_t launch_ce_product(CeProduct what, const CeArgs &a, const void *h, int64_t ldh, const void *w, int64_t ldw,
                              int esize, cudaStream_t s)
{
    return esize == 2 ? product<false>(what, a, h, ldh, w, ldw, s) : product<true>(what, a, h, ldh, w, ldw, s);
}

}  // namespace uly
