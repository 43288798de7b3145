// Shared by the two translation units of the fused LM-head loss: linear_ce.cu
// (rows, pieces, host) and linear_ce_gemm.cu (the three matrix products).
#pragma once

#include "uly_internal.h"

namespace uly {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

// The products run on CTA pairs: 256 x 256 output tiles, 64 values of the
// contraction per step.
constexpr int kCeTile = 256;
constexpr int kCeStep = 64;
constexpr int kCeStatCols = 64;  // columns behind one (c, s) of the softmax
constexpr int kCeMaxPairs = 80;
// Columns whose largest exponential lies within 2^+-kCeFree need no maximum taken
// out: sums of 2^21 such, and their products with values below 2^58, stay within
// fp32; exponentials are lost 2^-78 below the least such maximum, and of h / S
// values of h below 2^-57 (in fp32 their last 16 bits below 2^-33).
constexpr float kCeFree = 48.f;
// Rows that are searched for equal labels together, and how many with one label stay
// alone.
constexpr int kCeGroup = 256, kCeAlone = 2;
// floats a pair leaves for one tile
constexpr int64_t kCeTileFloats = static_cast<int64_t>(kCeTile) * kCeTile;

enum CeProduct {
    kCeLogits = 0,  // x  = h W^T   [rows][V]
    kCeDh = 1,      // dh = e W     [rows][D], rows scaled by 1 / S
    kCeDw = 2,      // dW = e^T h'  [V][D], h' = h / S
};

// What a call returns beside the gradients.
struct CeTotals {
    const float *row_loss;
    const unsigned long long *good;  // [P] good rows
    int64_t per_shard;               // rows
    int P;
    float *shard_loss, *total;
    int64_t *shard_good;
};

struct CeArgs {
    int *n_good;            // good rows of the whole call (device)
    int64_t base;           // first good row of the piece
    int rows;               // rows a piece may have
    int D, V;
    int64_t ldg;            // row pitch of e, elements
    uint16_t *e;            // [planes][rows][ldg] exponentials; at the label 0 (fp32: their difference to S)
    const int32_t *index;   // good row -> row of hidden
    const int32_t *label;   // [rows] of the piece
    float2 *stats;          // [rows][stat_tiles] (c, s)
    int stat_tiles;
    float *target;          // [rows] logits of the labels
    float *row_scale;       // [rows] 1 / S
    float *label_grad;      // bf16: [rows] of the piece, l = p - 1 at the label
    // bf16, with dW (else null): which rows of a block of kCeGroup have one label, see group_labels
    uint32_t *marks;        // [words / 32][mark_pitch] a bit for a row alone or the first of several, by its label
    int mark_pitch;
    int32_t *label_slot;    // [rows] place of the several rows' sum of l h; of a row that is alone ~(row of hidden)
    int32_t *label_next;    // [rows] the next of the several, -1: none
    int32_t *label_first;   // [places] the first of the several
    int32_t *label_left;    // [places] how many are still to come
    float *label_sum;       // [places][D]
    const uint16_t *hidden, *weight;  // bf16: as the caller gave them
    int keep;               // with a gradient: keep e
    void *dh, *dw;
    float *acc;             // dW over the pieces, in tiles (see tile_slot)
    float *partial;         // tiles split over the contraction
    int make_totals;        // this product's idle warp makes the totals
    CeTotals totals;
    // for the bounds checks of debug builds
    int64_t all_rows;                            // of hidden
    int64_t acc_slots, partial_slots, places;    // of acc and partial, in tiles; of label_sum
    unsigned *status;                            // device status word
};

// A sum held as hi + lo: 48 bits without the slow 64-bit units.
__device__ __forceinline__ float2 two_sum(float2 s, float2 v)
{
    const float hi = s.x + v.x, t = hi - s.x;
    if (!isfinite(hi))
        return make_float2(hi, 0.f);
    const float err = (s.x - (hi - t)) + (v.x - t) + s.y + v.y;
    const float top = hi + err;
    return make_float2(top, err - (top - hi));
}

__device__ __forceinline__ float2 warp_two_sum(float2 s)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s = two_sum(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    return s;
}

// Shard r's mean over its good rows from the sum of its rows' losses, and the
// total sum_r loss_r good_r / max(sum_r good_r, 1): by one warp, every sum in
// one order.
__device__ __forceinline__ void ce_shard(const CeTotals &t, int r, float2 sum)
{
    if (lane_id() == 0) {
        const long long n = static_cast<long long>(t.good[r]);
        const double all = static_cast<double>(sum.x) + sum.y;
        t.shard_loss[r] = n > 0 ? static_cast<float>(all / static_cast<double>(n)) : 0.f;
        t.shard_good[r] = n;
    }
}

__device__ __forceinline__ void ce_total(const CeTotals &t)
{
    __syncwarp();  // lane 0's shard means
    double num = 0.0;
    long long den = 0;
    for (int k = lane_id(); k < t.P; k += 32) {
        const long long n = static_cast<long long>(t.good[k]);
        num += static_cast<double>(t.shard_loss[k]) * static_cast<double>(n);
        den += n;
    }
    for (int o = 16; o > 0; o >>= 1) {
        num += __shfl_xor_sync(0xffffffffu, num, o);
        den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    if (lane_id() == 0)
        *t.total = static_cast<float>(num / static_cast<double>(den > 1 ? den : 1));
}

// Eight bf16 values from memory times f, added to x.
__device__ __forceinline__ void add_scaled8(float *x, float f, const uint4 &q)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = ffma2(make_float2(f, f), make_float2(__uint_as_float(w[j] << 16),
                                                              __uint_as_float(w[j] & 0xffff0000u)),
                               make_float2(x[2 * j], x[2 * j + 1]));
        x[2 * j] = v.x;
        x[2 * j + 1] = v.y;
    }
}

// Rows of the piece: device data, since the number of good rows is.
__device__ __forceinline__ int ce_piece_rows(const CeArgs &a)
{
    const int64_t left = *a.n_good - a.base;
    return left <= 0 ? 0 : (left < a.rows ? static_cast<int>(left) : a.rows);
}

// Most tiles that a product may leave in `partial` (host, for the workspace).
int ce_most_parts(CeProduct what, int rows, int D, int V, int esize);

// esize: 2 (bf16) or 4 (fp32, the operands as three bf16 planes each).  h: the
// piece's rows (dW: divided by S); w: the weight; ldh, ldw: row pitches in
// elements.
cudaError_t launch_ce_product(CeProduct what, const CeArgs &a, const void *h, int64_t ldh, const void *w, int64_t ldw,
                              int esize, cudaStream_t s);

}  // namespace uly
