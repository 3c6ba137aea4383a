// mla_dense.cuh -- what the dense MLA attention kernels share: which keys a row
// sees, the tiles, the device-side division of the work and the partial results
// of tiles that several workers share.
//
// Rows and tiles.  The n new tokens of a sequence times the H query heads are
// n * H query rows over ONE set of keys, flattened as m = i * H + h; a tile is
// kM consecutive rows of one sequence, whatever H is (128 heads: a token a
// tile; 16 heads: 8 tokens).  Token i sees vis(i) = clamp(L - n + i + 1, 0, L)
// keys: all of them, or the last `window` and the first `sinks` of them.
//
// Units.  A tile's keys are read in units of `unit` consecutive positions: the
// sinks' units, then the window's (or all of them), so that a block of kN keys
// never holds a unit that no row of the tile sees.
//
// Work.  Lengths are known on the device only, so the workers (CTAs or CTA
// pairs) divide it themselves: a tile costs its blocks plus kTileCost, worker g
// of G takes the costs [g C / G, (g + 1) C / G) of the total C, and a cut inside
// a tile falls on a block.  Every worker finds its two cuts with two block-wide
// scans, one over the sequences' tile counts and one over the tiles' costs; no
// launch and no buffer is spent on a schedule.  A tile that is cut leaves one
// partial result (O / l and lse in fp32) per worker in the caller's workspace, at
// most two a worker, which a second kernel joins in a fixed order.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace dsa {

constexpr int kDenseMaxWorkers = 160;     // bound of the workers, whatever the GPU

struct DenseShape {
    int rows, num_heads, batch, next_n;
    int window;                 // keys before a row's own end that it sees; < 0: all
    int sinks;                  // first keys that stay visible
    int cap;                    // positions the block table can address
    const int32_t* seq_lens;
    const int32_t* cum_q;       // null: next_n rows a sequence
};

// A latent cache as the kernels read it.
struct DenseCache {
    const uint8_t* vals;
    int64_t vps, vts;
    const uint8_t* scs;         // null: bf16
    int64_t sps, sts;
    const int32_t* bt;
    int64_t bt_stride;
    int page_kv, num_pages;
};

// Partial results of cut tiles: slot s holds slot_rows x (d_v + 1) floats (O / l,
// then lse) and its record.
struct DenseSlot {
    int32_t row0;               // first flattened row of the call (row * H + head)
    int32_t nrows;
    int32_t flags;              // bit 0: used, bit 1: the tile begins here, bit 2: it ends here
    int32_t pad;
};
struct DensePartials {
    float* o;
    float* lse;
    DenseSlot* slots;
    int slot_rows;
    int d_v;
};

// Rows of a sequence that the call holds, [begin, begin + n), kept inside it whatever cum_q
// holds; *q_len: its new tokens (more than n where the call's rows end before them).
__device__ __forceinline__ void dense_seq_rows(const DenseShape& s, int b, int* begin, int* n, int* q_len)
{
    if (s.cum_q) {
        const int c0 = s.cum_q[b], c1 = s.cum_q[b + 1];
        const int lo = min(max(c0, 0), s.rows);
        const int hi = min(max(c1, lo), s.rows);
        *begin = lo;
        *n = hi - lo;
        *q_len = max(c1 - lo, *n);
    } else {
        const long long lo = static_cast<long long>(b) * s.next_n;
        *begin = static_cast<int>(lo < s.rows ? lo : s.rows);
        const long long left = s.rows - lo;
        *n = static_cast<int>(left < 0 ? 0 : (left < s.next_n ? left : s.next_n));
        *q_len = s.next_n;
    }
}

// Keys of one token: [0, sink) and [lo, hi), sink <= lo.
struct DenseKeys {
    int sink, lo, hi;
};
__device__ __forceinline__ DenseKeys dense_keys(const DenseShape& s, int L, int n, int i)
{
    DenseKeys k;
    const int vis = visible_len(L, n, i);
    k.lo = s.window < 0 ? 0 : max(0, vis - s.window);
    k.hi = min(vis, s.cap);
    k.sink = min(s.sinks, k.lo);
    return k;
}

struct DenseTile {
    int seq, row0;              // sequence, first flattened row of the call
    int L, n, m0, nrows;        // context length, new tokens, first row within the sequence, rows
    DenseKeys first, last;      // keys of the tile's first and last token
    int su, wu0, nu, nblk;      // sink units, first window unit, units, blocks
    bool over;                  // the last token sees positions past the block table
};

__device__ __forceinline__ int dense_tiles_of(const DenseShape& s, int n, int kM)
{
    return static_cast<int>((static_cast<long long>(n) * s.num_heads + kM - 1) / kM);
}

// (The functions that walk tiles are called, not inlined: every role of a kernel
// walks, and a kernel whose code outgrows the instruction cache waits for it.)
template <int kM, int kN>
__device__ __noinline__ DenseTile dense_tile(const DenseShape& s, int unit, int seq, int begin, int rows, int n, int L, int t)
{
    DenseTile tile;
    DenseTile* o = &tile;
    const int H = s.num_heads;
    o->seq = seq;
    o->L = L;
    o->n = n;
    o->m0 = t * kM;
    o->nrows = static_cast<int>(min(static_cast<long long>(kM), static_cast<long long>(rows) * H - o->m0));
    o->row0 = begin * H + o->m0;
    o->first = dense_keys(s, L, n, o->m0 / H);
    const int i1 = (o->m0 + o->nrows - 1) / H;
    o->last = dense_keys(s, L, n, i1);
    o->over = visible_len(L, n, i1) > s.cap;
    const int end = (o->last.hi + unit - 1) / unit;
    o->wu0 = min(o->first.lo / unit, end);
    // the first row's sinks end before its window, the last row's may reach further
    o->su = min((min(o->last.sink, o->last.hi) + unit - 1) / unit, o->wu0);
    o->nu = o->su + end - o->wu0;
    o->nblk = (o->nu * unit + kN - 1) / kN;
    return tile;
}

// First position of unit k of the tile.
__device__ __forceinline__ int dense_unit_pos(const DenseTile& t, int unit, int k)
{
    return (k < t.su ? k : t.wu0 + k - t.su) * unit;
}

// Bit c set where position base + c (c < 32) is one of the keys k.
__device__ __forceinline__ uint32_t dense_mask32(const DenseKeys& k, int base)
{
    auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
    return (below(k.hi - base) & ~below(k.lo - base)) | below(min(k.sink, k.hi) - base);
}

// A place in the work: block `blk` of tile `tile` of sequence `seq`.
struct DenseCut {
    int seq, tile, blk;
};

// Exclusive block-wide prefix sum; *total receives the sum.  `tmp`: one word per warp plus one.
template <int kThreads>
__device__ __forceinline__ long long dense_scan(long long v, long long* tmp, long long* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        tmp[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long y = tmp[w];
        before += w < warp ? y : 0;
        all += y;
    }
    *total = all;
    return before + x - v;
}

// A place in the tiles' order: tile `tile` of the `tiles` of sequence `seq`, whose rows of the call,
// new tokens and length stand beside it.
struct DenseWalk {
    int seq, tile, tiles, begin, rows, n, L;
};
// The first sequence from `seq` on that has tiles (`seq` = batch: none), at its tile 0.
static __device__ __noinline__ DenseWalk dense_enter(const DenseShape& s, int kM, int seq)
{
    DenseWalk w;
    w.tile = w.tiles = w.begin = w.rows = w.n = w.L = 0;
#pragma unroll 1
    for (w.seq = seq; w.seq < s.batch; ++w.seq) {
        dense_seq_rows(s, w.seq, &w.begin, &w.rows, &w.n);
        w.tiles = dense_tiles_of(s, w.rows, kM);
        if (w.tiles > 0) {
            w.L = max(s.seq_lens[w.seq], 0);
            return w;
        }
    }
    w.tiles = 0;
    return w;
}
__device__ __forceinline__ void dense_next(const DenseShape& s, int kM, DenseWalk* w)
{
    if (++w->tile >= w->tiles)
        *w = dense_enter(s, kM, w->seq + 1);
}

// The cuts [cut[0], cut[1]) of worker g of `workers`, found by all threads of a
// CTA; `scratch` holds kThreads + 40 long longs of shared memory, free afterwards.  A cut
// leaves at least kMinBlocks blocks on either side; tiles of fewer than twice as many are
// not cut.
template <int kM, int kN, int kTileCost, int kMinBlocks, int kThreads>
__device__ void dense_divide(const DenseShape& s, int unit, int g, int workers, long long* scratch, DenseCut* cut)
{
    long long* tmp = scratch;                         // 32 + 1 words
    int* pre = reinterpret_cast<int*>(scratch + 40);  // tiles before each thread's sequences
    const int tid = threadIdx.x;
    const int per_seq = (s.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per_seq, s.batch), b1 = min(b0 + per_seq, s.batch);
    long long mine = 0, tiles = 0, cost_total = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        int begin, rows, n;
        dense_seq_rows(s, b, &begin, &rows, &n);
        mine += dense_tiles_of(s, rows, kM);
    }
    pre[tid] = static_cast<int>(dense_scan<kThreads>(mine, tmp, &tiles));
    __syncthreads();
    // this thread's tiles [t0, t1) and their cost
    const int T = static_cast<int>(tiles);
    const int per = (T + kThreads - 1) / kThreads;
    const int t0 = min(tid * per, T), t1 = min(t0 + per, T);
    DenseWalk at{};
    mine = 0;
    if (t0 < t1) {
        int lo = 0, hi = kThreads - 1;                // last thread with pre <= t0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= t0)
                lo = mid;
            else
                hi = mid - 1;
        }
        int skip = t0 - pre[lo];
        at = dense_enter(s, kM, lo * per_seq);
        while (skip >= at.tiles && at.seq < s.batch) {
            skip -= at.tiles;
            at = dense_enter(s, kM, at.seq + 1);
        }
        at.tile = skip;
    }
    DenseWalk w = at;
    DenseTile ti;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
        ti = dense_tile<kM, kN>(s, unit, w.seq, w.begin, w.rows, w.n, w.L, w.tile);
        mine += ti.nblk + kTileCost;
        if (t + 1 < t1)
            dense_next(s, kM, &w);
    }
    const long long before = dense_scan<kThreads>(mine, tmp, &cost_total);
    // as many workers as there are tiles, or pieces worth a worker
    workers = static_cast<int>(min(static_cast<long long>(workers),
                                   max(tiles, cost_total / (kMinBlocks + kTileCost))));
    workers = max(workers, 1);
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const long long pos = cost_total * (g + e) / workers;
        if (tid == 0 && pos >= cost_total)
            cut[e] = DenseCut{s.batch, 0, 0};
        if (pos < before || pos >= before + mine)
            continue;
        // the tile at this cost: its cut, on a block that leaves enough on either side
        w = at;
        long long left = pos - before;
        while (true) {
            ti = dense_tile<kM, kN>(s, unit, w.seq, w.begin, w.rows, w.n, w.L, w.tile);
            if (left < ti.nblk + kTileCost)
                break;
            left -= ti.nblk + kTileCost;
            dense_next(s, kM, &w);
        }
        int blk = max(0, static_cast<int>(left) - kTileCost);
        if (ti.nblk < 2 * kMinBlocks)
            blk = 2 * left < ti.nblk + kTileCost ? 0 : ti.nblk;
        else if (blk < kMinBlocks)
            blk = 0;
        else if (ti.nblk - blk < kMinBlocks)
            blk = ti.nblk;
        if (blk == ti.nblk && blk > 0) {
            dense_next(s, kM, &w);
            blk = 0;
        } else if (ti.nblk == 0 && 2 * left >= kTileCost) {
            dense_next(s, kM, &w);
        }
        cut[e] = DenseCut{w.seq, w.seq < s.batch ? w.tile : 0, blk};
    }
    __syncthreads();
}

// A worker's pieces in order: tiles from cut[0] to cut[1], the first and the
// last of them possibly in part.
struct DensePiece {
    DenseTile t;
    int blk0, blk1;             // blocks of this piece
    int slot;                   // partial slot, or -1 if the piece is a whole tile
};
template <int kM, int kN>
struct DensePieces {
    const DenseShape& s;
    const int unit;
    const DenseCut end;
    DenseWalk w;
    int blk, count, worker;

    __device__ __forceinline__ DensePieces(const DenseShape& sh, int u, int g, const DenseCut* cut)
        : s(sh), unit(u), end(cut[1]), blk(cut[0].blk), count(0), worker(g)
    {
        w = dense_enter(s, kM, cut[0].seq);
        w.tile = cut[0].tile;
    }
    __device__ __forceinline__ bool next(DensePiece* p)
    {
        if (w.seq >= s.batch || w.seq > end.seq || (w.seq == end.seq && w.tile > end.tile))
            return false;
        const bool at_end = w.seq == end.seq && w.tile == end.tile;
        if (at_end && blk >= end.blk)
            return false;
        p->t = dense_tile<kM, kN>(s, unit, w.seq, w.begin, w.rows, w.n, w.L, w.tile);
        p->blk0 = blk;
        p->blk1 = at_end ? end.blk : p->t.nblk;
        p->slot = p->blk0 == 0 && p->blk1 == p->t.nblk ? -1 : 2 * worker + (count > 0 ? 1 : 0);
        ++count;
        blk = 0;
        dense_next(s, kM, &w);
        return true;
    }
};

}  // namespace dsa
