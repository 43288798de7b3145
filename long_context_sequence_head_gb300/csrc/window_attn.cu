// Sliding-window attention with sinks over the Ulysses head shards: how a call
// is cut into work, and the small kernels around the attention kernels
// (window_fwd_bf16.cu, attn_bwd_bf16.cu, window_attn_f32.cu).
//
// Row i of a document that starts at s sees the keys j <= i of its document
// with i - j < window, and the document's first `sinks` keys.
//   Forward: a tile of rows walks the tiles of its window and of its sinks; all
// tiles cost about the same, so the grid needs no order without documents.
//   Backward: a key tile walks the query tiles that see it.  Through the window
// these are window/tile + 1, but a tile with sinks is seen by every later row:
// 512 tiles at 64K tokens against 33 under a window of 4096, which would run on
// alone at the end.  Up to 64 sinks in bf16 a kernel that goes over the rows takes
// what lies past the window (window_sinks.cu).  Otherwise that walk is cut into
// extra units of about the window's length, which add to dQ as any unit does; their
// dK and dV are fp32 sums, or in bf16 up to 320 sinks window_sinks.cu's.
// window_join_kernel adds such sums in order.
#include <new>

#include "uly_internal.h"

namespace uly {
namespace {

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// ------------------------------------------------------------- staging
// Host integers into device memory by kernel arguments: a captured call replays
// with the values it was given, which a copy from pageable memory would not.
constexpr int kStage = 4000;
struct StageParams {
    int32_t *dst;
    int n;
    int32_t v[kStage];
};

__global__ void __launch_bounds__(256) stage_kernel(const __grid_constant__ StageParams p)
{
    for (int i = threadIdx.x; i < p.n; i += 256)
        p.dst[i] = p.v[i];
}

cudaError_t stage(const std::vector<int32_t> &host, int32_t *dst, cudaStream_t s)
{
    StageParams p;
    for (size_t at = 0; at < host.size(); at += kStage) {
        p.dst = dst + at;
        p.n = static_cast<int>(std::min<size_t>(kStage, host.size() - at));
        std::copy_n(host.begin() + at, p.n, p.v);
        stage_kernel<<<1, 256, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// ---------------------------------------------------------------- units
// Tiles of a walk through the window alone.
int64_t window_tiles(int64_t window, int tile) { return (window + tile - 2) / tile + 1; }

// How the walks of tiles with sinks are cut.  At most 64 extra units a document,
// so that their sums stay small (64 tiles of 128 keys: 8 MB a problem); many
// sinks are many tiles, which balance each other.
struct Cut {
    int64_t tiles_with_sinks;  // of a document, at most
    int64_t length, most;

    Cut(int64_t window, int64_t sinks, bool docs, int tile)
        : tiles_with_sinks(sinks > 0 ? (sinks + tile - 1) / tile + (docs ? 1 : 0) : 0),
          length(std::max<int64_t>(4, window_tiles(window, tile))),
          most(tiles_with_sinks > 0 ? 64 / tiles_with_sinks : 0)
    {
    }
    int extra(int64_t past) const
    {
        return past <= length / 2 ? 0 : static_cast<int>(std::min(most, (past + length - 1) / length));
    }
};

// In bf16: in documents with rows past their window the dK and dV of up to 320 sinks
// are window_sinks.cu's, however few tokens there are for each: with P and dS in one
// bf16 part an element of dK was 0.47 of its rms off with 130 sinks of 64K tokens, 0.3
// with 300 of 24K, and dV of 65 sinks in documents of 2,000 to 3,900 tokens four times
// the bound that two parts keep.  64K tokens under a window of 4096 take 11 ms with 513
// sinks, 12 with 130 and 13.8 with 300 apart; 8K tokens, window 128, 130 sinks 214 us
// (121 in one part), 32K, window 512, 300 sinks 954 (472).
bool apart(int64_t sinks, int tile) { return tile == 128 && sinks > 0 && sinks <= kWindowSinksApart; }

// Row tiles of a chunk of window_sinks.cu: as short as leaves a problem 64 of them, but
// with many sinks (whose sums are large) 4 for each SM in all; and whole waves.
int chunk_tiles(int64_t N, int64_t sinks, int64_t nprob)
{
    const int64_t sms = num_sms();
    int64_t most = sinks <= kWindowSinks ? 64 : std::clamp<int64_t>(4 * sms / nprob, 4, 64);
    if (most * nprob > sms)
        most = std::max<int64_t>(4, most * nprob / sms * sms / nprob);
    return static_cast<int>(std::max<int64_t>(2, ((N + 127) / 128 + most - 1) / most));
}

// Most units, slots, joins and chunks of a problem whose documents are not known.
// Documents follow one another, so that the tiles that each spans beside its first are
// n - 1 at most in all: of documents with as many as a cut (or window_sinks.cu) takes
// there are only so many, and what goes with their length is counted once, not for
// each (8 problems of 64K tokens, window 64, 320 sinks, 500 documents: 1.3 GB of sums, 5.0
// with every document as long as all).
void unit_bounds(int64_t N, int64_t window, int64_t sinks, int num_docs, int tile, int64_t nprob, int64_t &units,
                 int64_t &slots, int64_t &joins, int64_t &chunks)
{
    const Cut cut(window, sinks, num_docs > 0, tile);
    const int64_t n = (N + tile - 1) / tile, beside = n - 1, tws = cut.tiles_with_sinks;
    // only a document longer than the window has rows past it, and a tile's window ends
    // `within` tiles behind it
    const int64_t long_docs = num_docs > 0 ? std::min<int64_t>(num_docs, N / (window + 1)) : 1;
    const int64_t within = (window + tile - 2) / tile;
    auto documents = [&](int64_t past) { return std::min(long_docs, beside / (within + past)); };
    // a walk is cut from length / 2 + 1 tiles past the window on
    const int64_t walks = cut.most > 0 ? std::min(n, tws * documents(cut.length / 2 + 1)) : 0;
    const int64_t extra = std::min(walks * cut.most, walks + tws * beside / cut.length);
    units = n + extra;
    joins = walks;
    slots = joins + extra;
    chunks = 0;
    if (apart(sinks, tile)) {
        // a document that walks past its first tile's window has chunks of its own beside
        // those of the rows between; documents may share a tile
        const int64_t own = documents(1), len = chunk_tiles(N, sinks, nprob), pieces = (n + len - 1) / len;
        chunks = pieces + 3 * own + 1;
        joins = std::min(n, tws * own);
        slots = 2 * joins + tws * (beside / len);
    }
}

struct Units {
    WindowUnits u;
    std::vector<int32_t> list;  // with documents or sinks apart: units, joins and chunks, four integers each
};

// The units with the sinks' work apart, with documents or without.
Units make_units_apart(int64_t N, int window, int sinks, const int32_t *cu, int num_docs, int64_t nprob)
{
    constexpr int tile = 128;
    const Cut cut(window, sinks, num_docs > 0, tile);
    const bool wide = sinks > kWindowSinks;
    Units r;
    WindowUnits &u = r.u;
    const int n = static_cast<int>((N + tile - 1) / tile), len = chunk_tiles(N, sinks, nprob);
    u.rows = std::min(sinks, tile);
    std::vector<int4> units, joins, chunks;
    auto fill = [&](int from, int to) {  // row tiles that only need zeros for their dQ
        for (; !wide && from < to; from += len)
            chunks.insert(chunks.end(), {make_int4(from, std::min(from + len, to), -1, 0), make_int4(0, 0, 0, 0),
                                         make_int4(0, 0, 0, 0)});
    };
    int done = 0;  // row tiles whose dQ is set
    for (int t = 0; t < n; ++t) {
        const int64_t k0 = static_cast<int64_t>(t) * tile, last = std::min(k0 + tile, N) - 1;
        int64_t lo, hi;
        doc_range_host(cu, num_docs, N, last, lo, hi);
        auto end_of = [&](int64_t key) { return static_cast<int>((std::min(key + window, hi) - 1) / tile); };
        const int end = end_of(last), all = static_cast<int>((hi - 1) / tile);
        const bool sink = lo + sinks > k0;
        const int past = wide && sink ? all - end : 0, extra = cut.extra(past);
        const int walk = end - t + 1 + (extra == 0 ? past : 0);
        u.work += end - t + 1 + past;
        units.push_back(make_int4(t, t, walk, -1));
        // the document's first tile, whose walk ends first
        const int first = static_cast<int>(lo / tile);
        if (!sink || all <= end_of(static_cast<int64_t>(first) * tile + tile - 1))
            continue;
        units.back().w = u.slots * 2;
        for (int e = 0; e < extra; ++e) {
            const int from = static_cast<int>(static_cast<int64_t>(past) * e / extra);
            const int to = static_cast<int>(static_cast<int64_t>(past) * (e + 1) / extra);
            units.push_back(make_int4(t, end + 1 + from, to - from, 1));
        }
        const int pieces = (all - first + len) / len;
        const int64_t from_key = std::max(lo, k0);
        joins.push_back(make_int4(static_cast<int>(from_key),
                                  static_cast<int>(std::min(std::min(lo + sinks, k0 + tile), hi) - from_key), u.slots,
                                  1 + pieces));
        if (t == first) {
            // without the keys of a tile that another document ends: a walk of one tile,
            // of its own unit
            const int64_t whole = hi == N ? N : hi / tile * tile;
            const int64_t next_last = std::min(k0 + 2 * tile, N) - 1;
            const int count = static_cast<int>(std::min(lo + sinks, whole) - lo);
            u.sinks = std::max(u.sinks, count);
            fill(done, first);
            for (int i = 0; i < pieces; ++i) {
                const int from = first + i * len;
                chunks.insert(chunks.end(),
                              {make_int4(from, std::min(from + len, all + 1), static_cast<int>(lo), count),
                               make_int4(u.slots + 1 + i, 1 + pieces, end, end_of(next_last)),
                               make_int4(static_cast<int>(hi), std::max(done, first), 0, 0)});
            }
            done = all + 1;
        }
        u.slots += 1 + pieces;
    }
    fill(done, n);
    std::stable_sort(units.begin(), units.end(), [](const int4 &a, const int4 &b) { return a.z > b.z; });
    u.longest = units[0].z;
    u.n_units = static_cast<int>(units.size());
    u.n_joins = static_cast<int>(joins.size());
    u.n_chunks = static_cast<int>(chunks.size() / 3);
    for (const std::vector<int4> *v : {&units, &joins, &chunks})
        for (const int4 &x : *v)
            r.list.insert(r.list.end(), {x.x, x.y, x.z, x.w});
    return r;
}

Units make_units(int64_t N, int window, int sinks, const int32_t *cu, int num_docs, int tile, int64_t nprob)
{
    // (a sequence without rows past its window needs no list of units)
    if (apart(sinks, tile) && (num_docs > 0 || window_end(N, window, tile, 0) < (N - 1) / tile))
        return make_units_apart(N, window, sinks, cu, num_docs, nprob);
    Units r;
    WindowUnits &u = r.u;
    const Cut cut(window, sinks, num_docs > 0, tile);
    const int n = static_cast<int>((N + tile - 1) / tile);
    u.rows = std::min(sinks, tile);
    if (num_docs == 0) {
        u.sink_tiles = static_cast<int>((std::min<int64_t>(sinks, N) + tile - 1) / tile);
        u.extra = u.sink_tiles > 0 ? cut.extra(n - 1 - window_end(N, window, tile, 0)) : 0;
        u.n_units = n + u.sink_tiles * u.extra;
        u.n_joins = u.extra > 0 ? u.sink_tiles : 0;
        u.slots = u.n_joins * (1 + u.extra);
        for (int t = 0; t < n; ++t) {
            const int64_t walk = window_end(N, window, tile, t) - t + 1, whole = n - t;
            const bool sink = t < u.sink_tiles;
            u.work += sink ? whole : walk;
            u.longest = std::max<int64_t>(
                u.longest, sink && u.extra > 0 ? std::max(walk, (whole - walk + u.extra - 1) / u.extra)
                                               : sink ? whole : walk);
        }
        return r;
    }
    std::vector<int4> units, joins;
    for (int t = 0; t < n; ++t) {
        const int64_t k0 = static_cast<int64_t>(t) * tile, last = std::min(k0 + tile, N) - 1;
        int64_t lo, hi;
        doc_range_host(cu, num_docs, N, last, lo, hi);
        const int end = static_cast<int>((std::min(last + window, hi) - 1) / tile);
        const bool sink = lo + sinks > k0 && sinks > 0;
        const int past = sink ? static_cast<int>((hi - 1) / tile) - end : 0;
        const int extra = cut.extra(past);
        u.work += end - t + 1 + past;
        if (extra == 0) {
            units.push_back(make_int4(t, t, end - t + 1 + past, -1));
            continue;
        }
        units.push_back(make_int4(t, t, end - t + 1, u.slots * 2));
        for (int e = 0; e < extra; ++e) {
            const int a = static_cast<int>(static_cast<int64_t>(past) * e / extra);
            const int b = static_cast<int>(static_cast<int64_t>(past) * (e + 1) / extra);
            units.push_back(make_int4(t, end + 1 + a, b - a, (u.slots + 1 + e) * 2 + 1));
        }
        const int64_t first = std::max(lo, k0);
        joins.push_back(make_int4(static_cast<int>(first),
                                  static_cast<int>(std::min(std::min(lo + sinks, k0 + tile), N) - first), u.slots,
                                  1 + extra));
        u.slots += 1 + extra;
    }
    std::stable_sort(units.begin(), units.end(), [](const int4 &a, const int4 &b) { return a.z > b.z; });
    u.longest = units[0].z;
    u.n_units = static_cast<int>(units.size());
    u.n_joins = static_cast<int>(joins.size());
    for (const std::vector<int4> *v : {&units, &joins})
        for (const int4 &x : *v)
            r.list.insert(r.list.end(), {x.x, x.y, x.z, x.w});
    return r;
}

// Query tiles of `rows` rows in the order of their walks, the longest first.
void tile_order(int64_t N, int window, int sinks, const int32_t *cu, int num_docs, int rows, int32_t *out)
{
    const int n = static_cast<int>((N + rows - 1) / rows);
    std::vector<int64_t> walk(n);
    for (int t = 0; t < n; ++t) {
        const int64_t a = static_cast<int64_t>(t) * rows, b = std::min<int64_t>(a + rows - 1, N - 1);
        int64_t lo, hi;
        doc_range_host(cu, num_docs, N, a, lo, hi);
        const int64_t first = std::max(lo, a - window + 1), sink_end = std::min(lo + sinks, first);
        walk[t] = b / 128 - first / 128 + 1;
        if (sink_end > lo)
            walk[t] += std::min((sink_end - 1) / 128 + 1, first / 128) - lo / 128;
        out[t] = t;
    }
    std::stable_sort(out, out + n, [&](int32_t x, int32_t y) { return walk[x] > walk[y]; });
}

// ------------------------------------------------------------ workspace
//   cu_seqlens and, behind it, the forward's orders of tiles and of pairs of them
//   (with documents) or the backward's units, joins and chunks; backward: as ulysses_attn_bwd's scratch, then the
//   slots of fp32 sums
struct Layout {
    size_t cu = 0, list = 0, list_ints = 0, lse2 = 0, D = 0, acc = 0, part = 0, total = 0;
    int64_t Npad = 0;
    int64_t units = 0, slots = 0, joins = 0, chunks = 0;
};

Layout layout(int64_t SB, int64_t N, int Hq, int Hkv, int d, int64_t window, int64_t sinks, int num_docs, bool bwd,
              int esize)
{
    Layout L;
    const int tile = esize == 2 ? 128 : kWindowTileF32;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up(bytes);
        return at;
    };
    if (bwd)
        unit_bounds(N, window, sinks, num_docs, tile, SB * Hkv, L.units, L.slots, L.joins, L.chunks);
    if (num_docs > 0 || L.chunks > 0) {
        L.cu = take((static_cast<size_t>(num_docs) + 1) * sizeof(int32_t));
        L.list_ints = bwd ? static_cast<size_t>(L.units + L.joins + 3 * L.chunks) * 4
                          : static_cast<size_t>((N + 127) / 128 + (N + 255) / 256);
        L.list = take(L.list_ints * sizeof(int32_t));
    }
    L.Npad = (N + 127) / 128 * 128;
    if (bwd) {
        const size_t rows = static_cast<size_t>(SB) * Hq * L.Npad;
        if (esize == 2) {
            L.lse2 = take(rows * sizeof(float));
            L.D = take(rows * sizeof(float));
            L.acc = take(rows * d * sizeof(float));
        } else {
            L.D = take(static_cast<size_t>(SB) * Hq * N * sizeof(float));
        }
        L.part = take(static_cast<size_t>(SB) * Hkv * L.slots * 2 * std::min<int64_t>(sinks, tile) * d * sizeof(float));
    }
    L.total = std::max(off, kAlign);
    return L;
}

// ---------------------------------------------------------------- join
// dK and dV of the sinks whose walk was cut: the sums of their tile's slots, in
// order.  Blocks take a (tile, problem) and one of its keys; of 2 d threads the first d
// sum dK, the others dV.
template <typename T>
__global__ void __launch_bounds__(256) window_join_kernel(const __grid_constant__ AttnShape s, T *__restrict__ dk,
                                                          T *__restrict__ dv, int tile)
{
    const WindowUnits &wu = s.units;
    const int col = threadIdx.x % s.d;
    const bool second = static_cast<int>(threadIdx.x) >= s.d;
    const int64_t nprob = s.SB * s.Hkv;
    const int64_t prob = blockIdx.x % nprob;
    const int t = static_cast<int>(blockIdx.x / nprob);
    const int kvh = static_cast<int>(prob % s.Hkv);
    const int64_t sb = prob / s.Hkv;
    int4 join;  // {first key, keys, first slot, slots}
    if (wu.joins != nullptr) {
        join = wu.joins[t];
    } else {
        const int64_t first = static_cast<int64_t>(t) * tile, end = min(s.N, static_cast<int64_t>(s.sinks));
        join = make_int4(static_cast<int>(first), static_cast<int>(min(end - first, static_cast<int64_t>(tile))),
                         t * (1 + wu.extra), 1 + wu.extra);
    }
    [[maybe_unused]] const int64_t extent = nprob * wu.slots * 2 * wu.rows * s.d;
    const int64_t step = static_cast<int64_t>(2) * wu.rows * s.d;  // from a slot to the next
    for (int r = blockIdx.y; r < join.y; r += gridDim.y) {
        const int64_t first = (prob * wu.slots + join.z) * step + ((second ? wu.rows : 0) + r) * s.d + col;
        float sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < join.w; ++i)
            if (ULY_IN_BOUNDS(s.status, first + i * step, 1, extent, 0x61))
                sum += wu.part[first + i * step];
        if (!second)
            sum *= s.scale;
        const int64_t off = s.L.off(s.N, sb, join.x + r, s.Hkv, kvh, s.d) + col;
        if (!ULY_IN_BOUNDS(s.status, off, 1, s.kv_elems, 0x62))
            break;
        T *out = second ? dv : dk;
        if constexpr (sizeof(T) == 2)
            out[off] = static_cast<T>(pack_bf16x2(sum, 0.f));
        else
            out[off] = sum;
    }
}

template <typename T>
cudaError_t launch_join(const AttnShape &s, void *dk, void *dv, int tile, cudaStream_t stream)
{
    if (s.units.n_joins == 0)
        return cudaSuccess;
    const dim3 grid(static_cast<unsigned>(s.units.n_joins * s.SB * s.Hkv), s.units.rows);  // at most 128
    window_join_kernel<T><<<grid, 2 * s.d, 0, stream>>>(s, static_cast<T *>(dk), static_cast<T *>(dv), tile);
    return cudaGetLastError();
}

}  // namespace

size_t window_attn_workspace(int64_t B, int64_t N, int Hq, int Hkv, int d, int S, int64_t window, int64_t sinks,
                             int num_docs, bool bwd, int esize)
{
    return layout(B * S, N, Hq, Hkv, d, window, sinks, num_docs, bwd, esize).total;
}

cudaError_t window_attn_fwd(AttnShape s, const void *q, const void *k, const void *v, void *o, float *lse, int esize,
                            void *workspace, cudaStream_t stream)
try {
    const Layout L = layout(s.SB, s.N, s.Hq, s.Hkv, s.d, s.window, s.sinks, s.num_docs, false, esize);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (s.cu_host) {
        const size_t list = (L.list - L.cu) / sizeof(int32_t);
        std::vector<int32_t> host(list + L.list_ints);
        std::copy(s.cu_host, s.cu_host + s.num_docs + 1, host.begin());
        tile_order(s.N, s.window, s.sinks, s.cu_host, s.num_docs, 128, host.data() + list);
        tile_order(s.N, s.window, s.sinks, s.cu_host, s.num_docs, 256, host.data() + list + (s.N + 127) / 128);
        s.cu_dev = reinterpret_cast<int32_t *>(ws + L.cu);
        s.order_dev = reinterpret_cast<int32_t *>(ws + L.list);
        const cudaError_t e = stage(host, reinterpret_cast<int32_t *>(ws + L.cu), stream);
        if (e != cudaSuccess)
            return e;
    }
    if (esize == 2)
        return launch_window_fwd_bf16(s, q, k, v, o, lse, stream);
    return launch_window_fwd_f32(s, static_cast<const float *>(q), static_cast<const float *>(k),
                                 static_cast<const float *>(v), static_cast<float *>(o), lse, stream);
} catch (const std::bad_alloc &) {
    return cudaErrorMemoryAllocation;
}

cudaError_t window_attn_bwd(AttnShape s, const void *q, const void *k, const void *v, const void *o, const float *lse,
                            const void *dout, void *dq, void *dk, void *dv, int esize, void *workspace,
                            cudaStream_t stream)
try {
    const int tile = esize == 2 ? 128 : kWindowTileF32;
    const Layout L = layout(s.SB, s.N, s.Hq, s.Hkv, s.d, s.window, s.sinks, s.num_docs, true, esize);
    Units units = make_units(s.N, s.window, s.sinks, s.cu_host, s.num_docs, tile, s.SB * s.Hkv);
    if (units.u.slots > L.slots || units.u.n_units > L.units || units.u.n_joins > L.joins ||
        units.u.n_chunks > L.chunks)
        return cudaErrorInvalidValue;  // the bounds above hold, so this is never reached
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    s.units = units.u;
    s.units.part = reinterpret_cast<float *>(ws + L.part);
    if (!units.list.empty()) {
        const size_t list = (L.list - L.cu) / sizeof(int32_t);
        std::vector<int32_t> host(list);
        if (s.cu_host) {
            std::copy(s.cu_host, s.cu_host + s.num_docs + 1, host.begin());
            s.cu_dev = reinterpret_cast<int32_t *>(ws + L.cu);
        }
        host.insert(host.end(), units.list.begin(), units.list.end());
        s.units.units = reinterpret_cast<int4 *>(ws + L.list);
        s.units.joins = s.units.units + s.units.n_units;
        if (s.units.n_chunks > 0)
            s.units.chunks = s.units.joins + s.units.n_joins;
        const cudaError_t e = stage(host, reinterpret_cast<int32_t *>(ws + L.cu), stream);
        if (e != cudaSuccess)
            return e;
    }
    if (esize == 2) {
        BwdScratch scr;
        scr.lse2 = reinterpret_cast<float *>(ws + L.lse2);
        scr.D = reinterpret_cast<float *>(ws + L.D);
        scr.dq_acc = reinterpret_cast<float *>(ws + L.acc);
        scr.Npad = L.Npad;
        const cudaError_t e = launch_attn_bwd_bf16(s, q, k, v, o, lse, dout, dq, dk, dv, scr, stream);
        return e != cudaSuccess ? e : launch_join<uint16_t>(s, dk, dv, tile, stream);
    }
    const cudaError_t e = launch_window_bwd_f32(
        s, static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v),
        static_cast<const float *>(o), lse, static_cast<const float *>(dout), static_cast<float *>(dq),
        static_cast<float *>(dk), static_cast<float *>(dv), reinterpret_cast<float *>(ws + L.D), stream);
    return e != cudaSuccess ? e : launch_join<float>(s, dk, dv, tile, stream);
} catch (const std::bad_alloc &) {
    return cudaErrorMemoryAllocation;
}

}  // namespace uly
