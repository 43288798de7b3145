// The LM head's product and the sequence-parallel loss in one operator: next-
// token cross entropy of hidden states h [P][B][N/P][D] under a head weight
// W [V][D], with the labels shifted over the whole sequence and the ranks'
// losses weighted by their good tokens as in sharded_loss.cu, and the
// gradients of the total with respect to h and W.  The logits
//   x_rv = <h_r, w_v>
// are never kept: the good rows are taken in pieces of a few thousand, and
// for each piece
//   1. logits   x = h W^T; every (row, 64 columns) leaves c, the sum s of
//               e = 2^(x log2 e - c), the row's target logit, and e itself;
//   2. rows     C = max c, S = sum s 2^(c - C); loss = ln S + (C ln 2 - x_y);
//               l = (e_y - S) / S, then e_y = 0; h' = h / S;
//   3. dh       = (e W / S + l w_y) / T for the piece's rows;
//   4. dW      += (e^T h' + l h at the rows' labels) / T, in fp32 across the
//               pieces, rounded once at the end.
// The label's term l = p - 1 is most of a row's gradient.  In bf16 it stays in fp32
// and meets w_y and h as they were given, where a product's result is written out;
// only the other words' terms have rounded operands.  With the label's value
// rounded among e, or h' carrying its term, dW was 0.0020 and 0.0024 of its norm
// off at 5,734 rows of 151,936, of which its own rounding is 0.0017.  (fp32: e has
// three parts, at the label of (e_y - S), and no rounding is left to take out.)
// c is 0 for all columns of nearly every row, so that e already is the softmax's
// numerator and is used as it lies: the division by S goes to dh's rows and to
// h, and of e only the label's value is touched.  Rewriting e as the logits'
// gradient, softmax - onehot, took 0.55 of 8.9 ms at 5,734 rows of 151,936 and
// 0.16 of 1.08 at 4,830 of 50,257; a row whose logits leave +-33 still has its
// values brought to one c, by powers of two.
// That is three products instead of the four that recomputing the logits from
// a kept log-sum-exp would take.  Rows without a label are left out before the
// first product: the good rows are gathered next to each other.
#include "linear_ce.h"

namespace uly {
namespace {

// Rows of a piece: as many as hold kPieceBytes of exponentials (2 bytes a value,
// 6 in fp32), at least 1024 and at most 65,536.  dW is carried from piece to
// piece in fp32: at D = 2560 and V = 151,936 its 1.6 GB read and written are 0.46
// ms beside 12 ms of products for a piece of 8448 rows.
constexpr int64_t kPieceBytes = int64_t(2500) << 20;
constexpr int kRowThreads = 128;

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xffffu); }

// Three bf16 parts of x: x1 + x2 + x3 = x up to 2^-26 |x|.
struct Parts {
    uint16_t p[3];
};
__device__ __forceinline__ Parts split3(float x)
{
    Parts r;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        r.p[i] = bf16_bits(x);
        x -= bf16_value(r.p[i]);
    }
    return r;
}

// Eight values as planes, 16 bytes each, `plane` elements apart.
__device__ __forceinline__ void store_planes(uint16_t *out, int64_t plane, const float (&x)[8])
{
    Parts q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        q[j] = split3(x[j]);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = q[2 * j].p[i] | static_cast<uint32_t>(q[2 * j + 1].p[i]) << 16;
        *reinterpret_cast<uint4 *>(out + i * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Eight values of an fp32 row of D values (a multiple of 4), zeros past its end.
__device__ __forceinline__ void load8(const float *row, int i, int D, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(row + i);
    const float4 b = i + 4 < D ? *reinterpret_cast<const float4 *>(row + i + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The totals of a call without gradients.
__global__ void __launch_bounds__(1024) totals_kernel(const CeTotals t)
{
    grid_wait();
    __shared__ float2 part[32];
    for (int r = 0; r < t.P; ++r) {
        const float *base = t.row_loss + r * t.per_shard;
        float2 s = make_float2(0.f, 0.f);
        for (int64_t i = threadIdx.x; i < t.per_shard; i += 1024)
            s = two_sum(s, make_float2(base[i], 0.f));
        s = warp_two_sum(s);
        if (lane_id() == 0)
            part[warp_id()] = s;
        __syncthreads();
        if (warp_id() == 0)
            ce_shard(t, r, warp_two_sum(part[lane_id()]));
        __syncthreads();
    }
    if (warp_id() == 0)
        ce_total(t);
}

// One block: the labels shifted over the whole sequence, each shard's good
// rows, and the good rows in order (index[i] = row of the i-th one).  A row's
// loss starts as 0.  Labels out of range are reported and ignored.  8192 rows a
// round of about 6 us, against 8 ms of products behind as many rows.
__global__ void __launch_bounds__(1024) labels_kernel(const int64_t *__restrict__ labels, int32_t *__restrict__ shifted,
                                                      unsigned long long *__restrict__ good,
                                                      float *__restrict__ row_loss, int32_t *__restrict__ index,
                                                      int *__restrict__ n_good, unsigned rows, unsigned Np, unsigned B,
                                                      int P, int V, unsigned *status)
{
    constexpr int kEach = 8;
    __shared__ int warp_sum[32];
    grid_next();
    for (int r = threadIdx.x; r < P; r += 1024)
        good[r] = 0;
    __syncthreads();
    int done = 0;
    for (int64_t base = 0; base < rows; base += 1024 * kEach) {
        const int64_t first = base + static_cast<int64_t>(threadIdx.x) * kEach;
        int32_t y[kEach];
        int mine = 0;
        // place in the shard's sequence; the next token is the next row, or,
        // at the end of a shard, the first of the same sequence in the next
        unsigned t = static_cast<unsigned>(first < rows ? first : 0) % Np;
#pragma unroll
        for (int i = 0; i < kEach; ++i, ++t) {
            y[i] = -100;
            if (first + i >= rows)
                continue;
            if (t == Np)
                t = 0;
            const int64_t next = first + i + 1 + (t + 1 == Np ? static_cast<int64_t>(B - 1) * Np : 0);
            if (next < rows) {
                const int64_t lab = labels[next];
                if (lab >= 0 && lab < V)
                    y[i] = static_cast<int32_t>(lab);
                else if (lab != -100)
                    atomicOr(status, kDevBadArg);
            }
            mine += y[i] >= 0;
        }
        // places of this thread's good rows among all
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane_id() >= o ? v : 0;
        }
        if (lane_id() == 31)
            warp_sum[warp_id()] = upto;
        __syncthreads();
        int sum = warp_sum[lane_id()];  // every warp scans the 32 sums
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane_id() >= o ? v : 0;
        }
        const int before = __shfl_sync(0xffffffffu, sum, warp_id() > 0 ? warp_id() - 1 : 0);
        int at = done + upto - mine + (warp_id() > 0 ? before : 0);
        done += __shfl_sync(0xffffffffu, sum, 31);
        // a warp's 256 rows are of one shard, mostly
        const int64_t w0 = base + static_cast<int64_t>(warp_id()) * 32 * kEach;
        const unsigned r0 = static_cast<unsigned>(w0 < rows ? w0 : 0) / (Np * B);
        const bool one = w0 + 32 * kEach <= static_cast<int64_t>(r0 + 1) * Np * B;
        if (one && lane_id() == 31 && upto > 0)
            atomicAdd(&good[r0], static_cast<unsigned long long>(upto));
        if (first + kEach <= rows) {
#pragma unroll
            for (int i = 0; i < kEach; i += 4) {
                *reinterpret_cast<int4 *>(shifted + first + i) = make_int4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                *reinterpret_cast<float4 *>(row_loss + first + i) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (first + i >= rows)
                continue;
            if (first + kEach > rows) {
                shifted[first + i] = y[i];
                row_loss[first + i] = 0.f;
            }
            if (y[i] >= 0) {
                if (ULY_IN_BOUNDS(status, at, 1, rows, 0x51))
                    index[at] = static_cast<int32_t>(first + i);
                ++at;
                if (!one)
                    atomicAdd(&good[static_cast<unsigned>(first + i) / (Np * B)], 1ull);
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        *n_good = done;
}

// Eight values of row `row`, columns [i, i + 8), to the products' layout.
template <bool kSplit>
__device__ __forceinline__ void lay8(const void *src, int64_t row, int i, int D, uint16_t *out, int64_t to,
                                     int64_t pitch, int64_t plane)
{
    if constexpr (kSplit) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (src)
            load8(static_cast<const float *>(src) + row * D, i, D, x);
        store_planes(out + to * pitch + i, plane, x);
    } else {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (src)
            x = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + row * D + i);
        *reinterpret_cast<uint4 *>(out + to * pitch + i) = x;
    }
}

__host__ __device__ inline int ce_groups(int rows) { return (rows + kCeGroup - 1) / kCeGroup; }

// bf16, with dW: which of the piece's rows [r0, r0 + kCeGroup) have one label.  The
// terms l_r h_r of dW of more than kCeAlone go as one, since a frequent word's
// thousands of rows would otherwise all meet in the one warp that writes its row of
// dW: 4,830 rows of 50,257 words with frequencies as 1 / rank 1.4 ms a call, 1.06
// like this, 0.97 with all words as frequent; one word throughout 2.0 and 1.0.
// Thread i looks for row i's label among the block's 256.
__device__ __forceinline__ void group_labels(const CeArgs &a, int cnt, int r0, const int32_t *shifted)
{
    static_assert(kCeGroup == 256, "a thread a row");
    __shared__ __align__(16) int label[kCeGroup];
    __shared__ int places[kCeGroup / 32];
    const int i = threadIdx.x, r = r0 + i;
    const int64_t src = r < cnt ? a.index[a.base + r] : 0;
    const int y = r < cnt ? shifted[src] : -1;
    label[i] = y;
    // the marks of these rows, 8 of 32 a piece
    for (int w = i; w < (a.V + 31) / 32; w += kCeGroup) {
        uint4 *mark = reinterpret_cast<uint4 *>(a.marks + static_cast<int64_t>(w) * a.mark_pitch + r0 / 32);
        mark[0] = mark[1] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    int first = kCeGroup, next = kCeGroup, count = 0;
    for (int j = 0; j < min(kCeGroup, cnt - r0); j += 4) {
        const int4 q = *reinterpret_cast<const int4 *>(label + j);
        const int v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (v[k] == y) {
                ++count;
                first = min(first, j + k);
                if (j + k > i)
                    next = min(next, j + k);
            }
        }
    }
    const bool several = y >= 0 && count > kCeAlone, stands = several && first == i;
    const unsigned mask = __ballot_sync(0xffffffffu, stands);
    if (lane_id() == 0)
        places[warp_id()] = __popc(mask);
    __syncthreads();  // the marks are cleared, too
    int slot = r0 / 2 + __popc(mask & ((1u << lane_id()) - 1));
    for (int w = 0; w < warp_id(); ++w)
        slot += places[w];
    if (stands) {
        a.label_first[slot] = r;
        a.label_left[slot] = count;
        label[i] = slot;  // nobody compares labels any more
    }
    __syncthreads();
    if (y < 0)
        return;
    const int64_t mark = static_cast<int64_t>(y / 32) * a.mark_pitch + r / 32;
    if ((stands || !several) &&
        ULY_IN_BOUNDS(a.status, mark, 1, static_cast<int64_t>((a.V + 31) / 32) * a.mark_pitch, 0x52))
        atomicOr(&a.marks[mark], 1u << (r % 32));
    a.label_slot[r] = several ? label[first] : static_cast<int32_t>(~src);
    a.label_next[r] = next < kCeGroup ? r0 + next : -1;
}

// The piece's hidden rows next to each other (fp32: as planes), with their
// labels; zeros up to a multiple of 64 rows, where dW's contraction ends.  The
// first piece also clears the gradient of the rows without a label: its row r
// then stands for row r of the call too.  A thread takes eight values.  The first
// blocks group the labels.
template <bool kSplit>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ CeArgs a, const void *__restrict__ hidden,
                                                     const int32_t *__restrict__ shifted, int32_t *__restrict__ label,
                                                     uint16_t *__restrict__ out, int64_t ldh, int64_t rows)
{
    grid_wait();
    grid_next();
    const int cnt = ce_piece_rows(a), vecs = (a.D + 7) / 8;
    const int groups = !kSplit && a.marks != nullptr ? ce_groups(a.rows) : 0;
    if (static_cast<int>(blockIdx.x) < groups) {
        group_labels(a, cnt, blockIdx.x * kCeGroup, shifted);
        return;
    }
    const int64_t at = (static_cast<int64_t>(blockIdx.x) - groups) * blockDim.x + threadIdx.x, r = at / vecs;
    const int i = static_cast<int>(at - r * vecs) * 8;
    if (a.base == 0 && a.dh != nullptr && r < rows && shifted[r] < 0 &&
        ULY_IN_BOUNDS(a.status, r * a.D + i, kSplit ? 4 : 8, rows * a.D, 0x53)) {
        uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.dh) + (r * a.D + i) * (kSplit ? 4 : 2));
        to[0] = make_uint4(0, 0, 0, 0);
        if (kSplit && i + 4 < a.D)
            to[1] = make_uint4(0, 0, 0, 0);
    }
    if (r >= (cnt + kCeStep - 1) / kCeStep * kCeStep)
        return;
    const bool live = r < cnt;
    const int64_t src = live ? a.index[a.base + r] : 0;
    if (!ULY_IN_BOUNDS(a.status, src * a.D + i, kSplit ? 4 : 8, rows * a.D, 0x54) ||
        !ULY_IN_BOUNDS(a.status, r * ldh + i, 8, ldh * a.rows, 0x55))
        return;
    if (i == 0)
        label[r] = live ? shifted[src] : -1;
    lay8<kSplit>(live ? hidden : nullptr, src, i, a.D, out, r, ldh, ldh * a.rows);
}

// fp32 weight as planes.
__global__ void __launch_bounds__(256) split_weight_kernel(const float *__restrict__ w, int D, int V,
                                                           uint16_t *__restrict__ out, int64_t ldw)
{
    grid_wait();
    grid_next();
    const int vecs = (D + 7) / 8;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, v = at / vecs;
    if (v < V)
        lay8<true>(w, v, static_cast<int>(at - v * vecs) * 8, D, out, v, ldw, ldw * V);
}

// bf16, with dW, by the block of each row with others of its label in its group, once
// its l is written: the last of them to come sums all their terms l h, in the order
// of the rows, so that sums repeat bit for bit.
__device__ __forceinline__ void sum_label_terms(const CeArgs &a, int slot)
{
    __shared__ int last;
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicSub(&a.label_left[slot], 1) == 1;
        __threadfence();
    }
    __syncthreads();
    if (!last)
        return;
    constexpr int kAhead = 4;  // rows on their way together
    for (int col = threadIdx.x * 8; col < a.D; col += kRowThreads * 8) {
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int r = a.label_first[slot]; r >= 0;) {
            uint4 q[kAhead];
            float l[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool live = r >= 0;
                int64_t row = live ? a.index[a.base + r] : 0;
                if (!ULY_IN_BOUNDS(a.status, row, 1, a.all_rows, 0x57))
                    row = 0;
                q[k] = live ? *reinterpret_cast<const uint4 *>(a.hidden + row * a.D + col) : make_uint4(0, 0, 0, 0);
                l[k] = live ? __ldcg(&a.label_grad[r]) : 0.f;
                r = live ? a.label_next[r] : -1;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                add_scaled8(sum, l[k], q[k]);
        }
        if (!ULY_IN_BOUNDS(a.status, static_cast<int64_t>(slot) * a.D + col, 8, a.places * a.D, 0x56))
            continue;
        float4 *to = reinterpret_cast<float4 *>(a.label_sum + static_cast<int64_t>(slot) * a.D + col);
        to[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        to[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
}

// Softmax statistics of some columns: C and S of sum e = S 2^C, and the least c.
struct Stat {
    float C, S, least;

    // a C of -inf is that of no columns, with S = 0
    __device__ __forceinline__ void join(float c, float s, float l)
    {
        const float m = fmaxf(C, c);
        S = (C == m ? S : S * exp2f(C - m)) + (c == m ? s : s * exp2f(c - m));
        C = m;
        least = fminf(least, l);
    }
};

// One block per row of the piece: its loss, and with a gradient the row's scale
// 1 / S, the label's term, the row of h' (where dW is wanted), and e on one c where
// it is not yet.  32 registers a thread, so that blocks are set up beside the
// logits' product (with 40 the loss of 64 rows takes 154 us instead of 150.5).
template <bool kSplit>
__global__ void __launch_bounds__(kRowThreads, 16) rows_kernel(const __grid_constant__ CeArgs a,
                                                           const void *__restrict__ hidden,
                                                           const int32_t *__restrict__ label,
                                                           float *__restrict__ row_loss, uint16_t *__restrict__ out,
                                                           int64_t ldh)
{
    grid_wait();
    grid_next();
    const int cnt = ce_piece_rows(a), r = blockIdx.x;
    if (r >= cnt)
        return;
    constexpr int kWarps = kRowThreads / 32;
    __shared__ Stat red[kWarps];
    const float2 *stats = a.stats + static_cast<int64_t>(r) * a.stat_tiles;
    Stat st = {-INFINITY, 0.f, INFINITY};
#pragma unroll 4
    for (int t = threadIdx.x; t < a.stat_tiles; t += kRowThreads) {
        const float2 v = stats[t];
        st.join(v.x, v.y, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xffffffffu, st.C, o), s = __shfl_xor_sync(0xffffffffu, st.S, o);
        st.join(c, s, __shfl_xor_sync(0xffffffffu, st.least, o));
    }
    if (lane_id() == 0)
        red[warp_id()] = st;
    __syncthreads();
    st = red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
        st.join(red[w].C, red[w].S, red[w].least);
    const int y = label[r];
    const int64_t row = a.index[a.base + r];
    if (!ULY_IN_BOUNDS(a.status, row, 1, a.all_rows, 0x58) || !ULY_IN_BOUNDS(a.status, y, 1, a.V, 0x59))
        return;  // the whole block agrees
    const int slot = !kSplit && a.marks != nullptr ? a.label_slot[r] : -1;
    if (threadIdx.x == 0) {
        // ln S + C ln 2 - x_y, with the whole powers of two taken out of x_y before anything is rounded
        const uint32_t bits = __float_as_uint(st.S), exponent = bits >> 23;
        const bool normal = exponent > 0 && exponent < 255;
        const float k = normal ? static_cast<float>(static_cast<int>(exponent) - 127) : 0.f;
        const float m = normal ? __uint_as_float((bits & 0x007fffffu) | 0x3f800000u) : st.S;
        row_loss[row] = (log2f(m) - fmaf(a.target[r], kLog2e, -(st.C + k))) * kLn2;
    }
    if (!a.keep)
        return;
    const float g = ex2_approx(fmaf(a.target[r], kLog2e, -st.C)) - st.S, scale = 1.f / st.S;  // g: (p - 1) S
    uint16_t *erow = a.e + r * a.ldg;
    const int64_t plane = a.ldg * a.rows;
    if (st.least < st.C) {
        for (int v = threadIdx.x * 8; v < a.V; v += kRowThreads * 8) {
            const float f = exp2f(stats[v / kCeStatCols].x - st.C);
#pragma unroll
            for (int i = 0; i < (kSplit ? 3 : 1); ++i) {
                uint4 *at = reinterpret_cast<uint4 *>(erow + i * plane + v);
                uint4 q = *at;
                uint32_t *w = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = pack_bf16x2(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xffff0000u) * f);
                *at = q;
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.row_scale[r] = scale;
        if constexpr (kSplit) {
            const Parts q = split3(g);
#pragma unroll
            for (int i = 0; i < 3; ++i)
                erow[i * plane + y] = q.p[i];
        } else {
            a.label_grad[r] = g * scale;
            erow[y] = 0;
        }
    }
    if (a.dw == nullptr)
        return;
    for (int i = threadIdx.x * 8; i < a.D; i += kRowThreads * 8) {
        float x[8];
        if constexpr (kSplit) {
            load8(static_cast<const float *>(hidden) + row * a.D, i, a.D, x);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] *= scale;
            store_planes(out + r * ldh + i, ldh * a.rows, x);
        } else {
            const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(hidden) + row * a.D + i);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint32_t to[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                to[j] = pack_bf16x2(__uint_as_float(w[j] << 16) * scale, __uint_as_float(w[j] & 0xffff0000u) * scale);
            *reinterpret_cast<uint4 *>(out + r * ldh + i) = make_uint4(to[0], to[1], to[2], to[3]);
        }
    }
    if (!kSplit && slot >= 0)
        sum_label_terms(a, slot);
}

size_t up(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
    size_t good, n_good, shifted, row_loss, index, label, target, row_scale, label_grad, stats, h, w, e, acc, partial;
    size_t marks, label_slot, label_next, label_first, label_left, label_sum, total;
    int64_t ldh, ldg, acc_slots, partial_slots, places;
    int rows, stat_tiles;
};

Layout layout(int64_t B, int64_t N, int D, int V, int P, bool grad, int esize)
{
    Layout L = {};
    const int64_t T = B * N;
    const bool split = esize == 4;
    L.ldg = (V + 63) / 64 * 64;
    const int64_t fit = std::max<int64_t>(1024, kPieceBytes / (L.ldg * (split ? 6 : 2)) / kCeTile * kCeTile);
    L.rows = static_cast<int>(std::min<int64_t>(std::min<int64_t>(fit, 65536), (T + 63) / 64 * 64));
    L.ldh = (D + 63) / 64 * 64;
    L.stat_tiles = (V + kCeStatCols - 1) / kCeStatCols;
    const size_t planes = split ? 3 : 1, kept = static_cast<size_t>(L.rows) * L.ldg;
    size_t o = 0;
    auto take = [&](size_t &at, size_t bytes) { at = o, o += up(bytes); };
    take(L.good, sizeof(unsigned long long) * P);
    take(L.n_good, sizeof(int));
    take(L.shifted, sizeof(int32_t) * T);
    take(L.row_loss, sizeof(float) * T);
    take(L.index, sizeof(int32_t) * T);
    take(L.label, sizeof(int32_t) * L.rows);
    take(L.target, sizeof(float) * L.rows);
    take(L.row_scale, sizeof(float) * L.rows);
    take(L.label_grad, sizeof(float) * L.rows);
    take(L.stats, sizeof(float2) * L.rows * static_cast<size_t>(L.stat_tiles));
    take(L.h, planes * static_cast<size_t>(L.rows) * L.ldh * 2);
    if (split)
        take(L.w, planes * V * L.ldh * 2);
    if (grad) {
        take(L.e, planes * kept * 2);
        const size_t tiles = static_cast<size_t>((V + kCeTile - 1) / kCeTile) * ((D + kCeTile - 1) / kCeTile);
        L.acc_slots = T > L.rows ? tiles : 0;
        take(L.acc, sizeof(float) * kCeTileFloats * L.acc_slots);
        L.partial_slots =
            std::max(ce_most_parts(kCeDh, L.rows, D, V, esize), ce_most_parts(kCeDw, L.rows, D, V, esize));
        take(L.partial, sizeof(float) * kCeTileFloats * L.partial_slots);
        if (!split) {
            const size_t groups = ce_groups(L.rows);
            L.places = groups * (kCeGroup / 2);  // sums of two rows at least
            take(L.marks, sizeof(uint32_t) * (kCeGroup / 32) * groups * ((V + 31) / 32));
            take(L.label_slot, sizeof(int32_t) * L.rows);
            take(L.label_next, sizeof(int32_t) * L.rows);
            take(L.label_first, sizeof(int32_t) * L.places);
            take(L.label_left, sizeof(int32_t) * L.places);
            take(L.label_sum, sizeof(float) * L.places * D);
        }
    }
    L.total = o;
    return L;
}

template <bool kSplit>
cudaError_t run(const void *hidden, const void *weight, const int64_t *labels, void *dhidden, void *dweight,
                float *shard_loss, int64_t *shard_good, float *total, int64_t B, int64_t N, int D, int V, int P,
                uint8_t *ws, cudaStream_t s)
{
    constexpr int kEsize = kSplit ? 4 : 2;
    const bool grad = dhidden || dweight;
    const Layout L = layout(B, N, D, V, P, grad, kEsize);
    const int64_t rows = B * N;
    auto *good = reinterpret_cast<unsigned long long *>(ws + L.good);
    auto *shifted = reinterpret_cast<int32_t *>(ws + L.shifted);
    auto *row_loss = reinterpret_cast<float *>(ws + L.row_loss);
    auto *index = reinterpret_cast<int32_t *>(ws + L.index);
    auto *label = reinterpret_cast<int32_t *>(ws + L.label);
    auto *h = reinterpret_cast<uint16_t *>(ws + L.h);
    CeArgs a = {};
    a.n_good = reinterpret_cast<int *>(ws + L.n_good);
    a.rows = L.rows;
    a.D = D;
    a.V = V;
    a.ldg = L.ldg;
    a.e = reinterpret_cast<uint16_t *>(ws + L.e);
    a.index = index;
    a.label = label;
    a.stats = reinterpret_cast<float2 *>(ws + L.stats);
    a.stat_tiles = L.stat_tiles;
    a.target = reinterpret_cast<float *>(ws + L.target);
    a.row_scale = reinterpret_cast<float *>(ws + L.row_scale);
    a.keep = grad;
    a.label_grad = reinterpret_cast<float *>(ws + L.label_grad);
    a.marks = !kSplit && dweight ? reinterpret_cast<uint32_t *>(ws + L.marks) : nullptr;
    a.mark_pitch = ce_groups(L.rows) * (kCeGroup / 32);
    a.label_slot = reinterpret_cast<int32_t *>(ws + L.label_slot);
    a.label_next = reinterpret_cast<int32_t *>(ws + L.label_next);
    a.label_first = reinterpret_cast<int32_t *>(ws + L.label_first);
    a.label_left = reinterpret_cast<int32_t *>(ws + L.label_left);
    a.label_sum = reinterpret_cast<float *>(ws + L.label_sum);
    a.hidden = static_cast<const uint16_t *>(hidden);
    a.weight = static_cast<const uint16_t *>(weight);
    a.dh = dhidden;
    a.dw = dweight;
    a.acc = reinterpret_cast<float *>(ws + L.acc);
    a.partial = reinterpret_cast<float *>(ws + L.partial);
    a.totals = CeTotals{row_loss, good, rows / P, P, shard_loss, total, shard_good};
    a.all_rows = rows;
    a.acc_slots = L.acc_slots;
    a.partial_slots = L.partial_slots;
    a.places = L.places;
    a.status = device_status_ptr();
    labels_kernel<<<1, 1024, 0, s>>>(labels, shifted, good, row_loss, index, a.n_good, static_cast<unsigned>(rows),
                                     static_cast<unsigned>(N / P), static_cast<unsigned>(B), P, V,
                                     device_status_ptr());
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const void *w = weight;
    int64_t ldw = D;
    const int64_t vecs = (D + 7) / 8;
    if (kSplit) {
        w = ws + L.w;
        ldw = L.ldh;
        e = launch_after(split_weight_kernel, (static_cast<int64_t>(V) * vecs + 255) / 256, 256, 0, s,
                         static_cast<const float *>(weight), D, V, reinterpret_cast<uint16_t *>(ws + L.w), ldw);
    }
    for (int64_t base = 0; base < rows; base += L.rows) {
        a.base = base;
        const int64_t blocks = ((base == 0 ? std::max<int64_t>(rows, L.rows) : L.rows) * vecs + 255) / 256 +
                               (a.marks != nullptr ? ce_groups(L.rows) : 0);
        if (e == cudaSuccess)
            e = launch_after(gather_kernel<kSplit>, blocks, 256, 0, s, a, hidden, shifted, label, h, L.ldh, rows);
        if (e == cudaSuccess)
            e = launch_ce_product(kCeLogits, a, h, L.ldh, w, ldw, kEsize, s);
        if (e == cudaSuccess)
            e = launch_after(rows_kernel<kSplit>, L.rows, kRowThreads, 0, s, a, hidden, label, row_loss, h, L.ldh);
        // the last product of a call makes the totals beside its own work
        const bool end = base + L.rows >= rows;
        a.make_totals = end && !dweight;
        if (e == cudaSuccess && dhidden)
            e = launch_ce_product(kCeDh, a, h, L.ldh, w, ldw, kEsize, s);
        a.make_totals = end;
        if (e == cudaSuccess && dweight)
            e = launch_ce_product(kCeDw, a, h, L.ldh, w, ldw, kEsize, s);
        if (e != cudaSuccess)
            return e;
    }
    if (e == cudaSuccess && !grad)
        e = launch_after(totals_kernel, 1, 1024, 0, s, a.totals);
    return e;
}

}  // namespace

size_t sharded_linear_ce_workspace(int64_t B, int64_t N, int D, int V, int P, bool grad, int esize)
{
    return layout(B, N, D, V, P, grad, esize).total;
}

cudaError_t launch_sharded_linear_ce(const void *hidden, const void *weight, const int64_t *labels, void *dhidden,
                                     void *dweight, float *shard_loss, int64_t *shard_good, float *total, int64_t B,
                                     int64_t N, int D, int V, int P, int esize, void *workspace, cudaStream_t s)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (esize == 2)
        return run<false>(hidden, weight, labels, dhidden, dweight, shard_loss, shard_good, total, B, N, D, V, P, ws,
                          s);
    return run<true>(hidden, weight, labels, dhidden, dweight, shard_loss, shard_good, total, B, N, D, V, P, ws, s);
}

}  // namespace uly
