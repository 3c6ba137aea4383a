// mla_dense_tc.cu -- dense MLA attention over a paged latent cache on the tcgen05
// tensor cores: d_v 512, d_qk 512 or 576, FP8 (e4m3 + token scale) or bf16 latents,
// any head count, pages that are multiples of 32 tokens.
//
//   s_j = c q . k_j,  out = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j),
//   v_j = the first 512 elements of k_j
//
// Bound by the tensor cores: a pair of a query row and a key costs 2 (d_qk + 512)
// flops against (d_qk + 4) bytes a key for 128 rows.
// Measured: 1024 new tokens x 128 heads over 16384 keys, 576 / 512, FP8: 2.66 ms in bursts
// (1.70 PFLOP/s, tensor pipe 72 % active), 2.85-2.93 ms back to back at the card's power limit;
// 64 single tokens x 128 heads over 8K-131K keys: 0.88 and 0.93-0.99 ms.  What bounds a block of
// 128 keys is the softmax's chain on eight warps: about 3000 cycles with all that stands between blocks,
// against 2176 of MMAs.
//
// One cluster of two CTAs owns a tile of 128 query rows and walks its keys with
// cta_group::2 MMAs of M = 128, 64 rows a CTA.  That shape leaves each CTA's results
// with both lane halves of its TMEM in use (rows x the first half of N in lanes 0-63,
// the second half in lanes 64-127), so the 64 x 512 fp32 output takes 256 columns and
// the scores fit beside it; each CTA runs the softmax of its own rows with nothing to
// exchange but barriers, and the pair shares the key tiles (each CTA fetches half
// the keys for S and half the value dims for O).  Measured with the issuing loop under
// elect.sync: N = 128 and N = 256 both run at 0.99 of the fp8 rate.
//
// FP8 latents are multiplied as they lie in the cache (no widening pass, TMA from the
// pages to the swizzled tiles).  q and P keep their precision as sums of two e4m3
// numbers, x = hi + lo: hi = e4m3(x), lo = e4m3(x - hi) hold 8 significant bits, all
// of a bf16, so S = Q_hi K + Q_lo K is exact but for elements below 2^-10 of their
// row's largest (absolute error 2^-17 of that).  Two fp8 MMAs take as long as one 16-bit
// MMA.  The token scale multiplies the fp32 scores; for O it is folded into P, and the
// running maximum m is taken over score + log2 of the scale, so that P x scale stays inside
// e4m3 whatever the scales are (those below 2^-72 leave it at its lower end).  P x scale is off by at most 2^-9 of itself (a
// bf16 by 2^-8), plus what is below e4m3's last step, 2^-16 of the row's largest: that is
// rounded up or down by an offset that varies with the key, so that it is right on average, and m
// goes down again where a long context lies far below an early key.
//
// bf16 latents use kind::f16, Q and P in bf16, and tiles of 64 keys (the same bytes): a
// block of 128 keys is two of them, one after the other, under one softmax (blocks of 64
// took the latency of its softmax twice).
//
//   warp 0     K tiles: TMA, half the block's keys, all dims
//   warp 1     V tiles: TMA, all keys, this CTA's 256 value dims; zeroes the rows that
//              no (or not every) query row may see where they could hold NaN
//   warp 2     even CTA: issues every MMA, S(j + 2) before O(j)
//   warp 3     the block's token scales, their maximum, its positions and whether a
//              mask is needed
//   warps 4-11 softmax, 4 threads a row; O's rescaling and the epilogue; a piece's Q rows:
//              per-row power of two, split, swizzled tiles
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "mla_dense.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kM = 128;                  // query rows of a pair
constexpr int kThreads = 384;
// Tokens a TMA box, the unit in which keys are read.  (Boxes of 64 take half the TMA issues but leave
// more unseen keys in a window's blocks: window 128, 64 rows of 128 heads 20.5 against 22.5 us;
// 512, 2749 tokens x 64 heads 304 against 313; a 1024-token chunk at 16384 x 128 heads 2.92 against
// 2.96 ms; the same within 1 % past 6000 keys.)
constexpr int kUnit = 32;
constexpr int kTileCost = 3;             // Q's preparation and the epilogue, in blocks
constexpr int kMinBlocks = 4;
constexpr int kQBytes = 64 * 576 * 2;    // hi and lo parts, or bf16
constexpr int kKBytes = 36864;           // one K stage: 64 x 576 e4m3 or 32 x 576 bf16
constexpr int kVBytes = 32768;           // one V stage: 128 x 256 e4m3 or 64 x 256 bf16
constexpr int kPBytes = 16384;           // hi and lo parts of 64 x 128, or 64 x 128 bf16 in two tiles
constexpr int kOffK = kQBytes;
constexpr int kOffV = kOffK + 2 * kKBytes;
constexpr int kOffP = kOffV + 2 * kVBytes;
constexpr int kOffMeta = kOffP + kPBytes;
constexpr uint32_t kSCol = 256;          // TMEM: O in columns 0-255, two score buffers of 64
constexpr uint32_t kTmemCols = 512;
constexpr float kGrow = 1.75f;           // FP8: the reference m follows the block's maximum up past 2^1.75 (bf16: 2^8) ...
constexpr float kHead = 7.f;             // ... and P is held times 2^7: at most 2^8.75 < 448
// ... and down to the recent blocks' maximum (which fades by kFade a block) where that is kGap or
// more below and the rounding of P could be seen: u holds the sum of the squares of the blocks' largest
// P over 2^7, less kNoise a block.  A key's rounding has a variance of 2^-20 at most, a block's 2^-13:
// u < 0 is more than 2^-21 of sum P^2, an error of 2^-10.5 of the row's rms; where a maximum within
// kGap comes back every kGap / kFade blocks it is 2^-10 at most.  (A chunk of 1024 tokens at 16384, 128
// heads, takes 2 % longer than without falling, and 2 % more with kNoise four times this.)
constexpr float kGap = 2.f, kFade = 0.25f, kNoise = 0.015625f;
constexpr float kDeep = 24.f;            // at most so far at a time: O and l stay inside fp32
constexpr uint32_t kFarBits = 0x01400000u;   // neighbours' scales whose bits differ by more, 2^2.5 or so, are far apart

// Barriers of a CTA.  Those that tell the MMA warp what is ready (K, V, P and Q
// tiles, score buffers and O free) count both CTAs' arrivals in the even CTA.
enum Bar {
    kKFull = 0, kKEmpty = 2, kVLand = 4, kVFull = 6, kVEmpty = 8, kSFull = 10, kSEmpty = 12, kMFull = 14,
    kMEmpty = 16, kPFull = 18, kPvDone = 19, kQFull = 20, kOFree = 21, kDrain = 22, kGFull = 24,
    kGEmpty = 26, kBars = 28
};

// What the softmax needs of a piece; nblk < 0: no more.
struct PieceInfo {
    int nblk, row0, m0, nrows, L, n, slot, flags, seq;
};
struct Meta {
    float scale[2][128];
    float lgp[2][64];            // log2 of the larger scale of two neighbours
    float mx[4][64];
    int8_t qe[2][64];
    int unit[2][4];
    int edge[2];                 // bit 0: a mask is needed, bit 1: neighbours' scales far apart
    uint64_t bar[kBars];
    DenseCut cut[2];
    PieceInfo piece[2];
    uint32_t tmem;
    int abort;
};
constexpr int kSmem = kOffMeta + static_cast<int>(sizeof(Meta));
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct TcParams {
    DenseShape s;
    DenseCache c;
    const __nv_bfloat16* q;
    int rope;                            // d_qk == 576
    float scale_log2;                    // |softmax_scale| * log2(e)
    uint32_t flip;                       // sign bits to flip in two bf16 of q (negative softmax_scale)
    uint32_t nan;                        // bits to set in two bf16 of q (softmax_scale is NaN: q becomes NaN)
    __nv_bfloat16* out;
    float* lse;
    DensePartials part;
    int32_t* status;
};

// ------------------------------------------------------------- PTX, two-CTA

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

template <bool kFp8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (kFp8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
                     "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
                     "r"(idesc), "r"(accumulate)
                     : "memory");
}

// One arrival on the barrier at this offset in both CTAs when all MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

// Arrive on a barrier of the pair's even CTA (a cluster address).  What the arrival
// announces lies in the arriving CTA's own memory, where that CTA's half of the MMA
// reads it, and was ordered before: shared memory by a proxy fence, TMEM by
// tcgen05.wait and a fence.
__device__ __forceinline__ void arrive_even(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// TMA to this CTA's memory that counts its bytes on a barrier of the pair's even CTA.
__device__ __forceinline__ void tma_pair_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3)
{
    asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
                 : "memory");
}

// Bounded wait of a whole warp that also ends when another role of the CTA gave up.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort)
{
    const uint64_t t0 = global_timer_ns();
    bool ok = false;
    while (true) {
        for (int i = 0; i < 32 && !ok; ++i)
            ok = mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, ok))
            return true;
        const bool late = *abort != 0 || global_timer_ns() - t0 > kWaitLimitNs;
        if (__any_sync(0xffffffffu, late)) {
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    return wait_slow(bar, parity, abort);
}

// Named barrier among `count` threads; true for all of them if `x` is for any.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t count, bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(count), "r"(x ? 1u : 0u)
                 : "memory");
    return r != 0;
}

// log2 of a scale's magnitude, given as bits, from above by at most 0.09; kLeastScale at least, because
// the probabilities' sum is held without the scale, 2^-lg times larger: up to 2^(8.75 + 72 + 24)
// a key, where the reference fell by kDeep, and 2^127 for four million such keys.
constexpr float kLeastScale = -72.f;
__device__ __forceinline__ float log2_above(uint32_t bits)
{
    return fmaxf(kLeastScale, fmaf(static_cast<float>(static_cast<int>(bits)), 0x1p-23f, -126.91f));
}

// x -> hi + lo in e4m3, two values at a time.
__device__ __forceinline__ void split_e4m3(__half2 x, uint32_t* hi, uint32_t* lo)
{
    const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 back(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3));
    const __half2 rest = __hsub2(x, back);                        // exact
    *hi = h;
    *lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
}

// A page id and the token in it of position pos of sequence seq; page = num_pages
// (out of the map's range: the box is filled with zeros) where there is none.
struct Place {
    int page, token;
};
__device__ __noinline__ Place place_of(const DenseCache& c, int seq, int pos, int cap)
{
    Place o{c.num_pages, 0};
    if (pos >= 0 && pos < cap) {
        const int lp = pos / c.page_kv;
        const int pg = c.bt[static_cast<int64_t>(seq) * c.bt_stride + lp];
        o.token = pos - lp * c.page_kv;
        if (pg >= 0 && pg < c.num_pages)
            o.page = pg;
    }
    return o;
}

// The bf16 latents' values at dims [dim, dim + 32) that are infinite or NaN in a key that the row sees
// and another row of its tile does not (the V warp makes such a value 0): bit per dim.  The keys
// before the first token's end, from the last one's start on and in the first one's sinks
// are seen by all.
__device__ __noinline__ uint32_t masked_infinities(const TcParams& p, const PieceInfo& pi, const DenseKeys& row, int dim)
{
    const DenseKeys first = dense_keys(p.s, pi.L, pi.n, pi.m0 / p.s.num_heads);
    const DenseKeys last = dense_keys(p.s, pi.L, pi.n, (pi.m0 + pi.nrows - 1) / p.s.num_heads);
    uint32_t found = 0;
    auto look = [&](int from, int to) {
        for (int x = from; x < to; ++x) {
            if ((x < row.lo && x >= row.sink) || (x < first.hi && (x >= last.lo || x < first.sink)))
                continue;
            const Place at = place_of(p.c, pi.seq, x, p.s.cap);
            if (at.page >= p.c.num_pages)
                continue;
            const uint4* v = reinterpret_cast<const uint4*>(p.c.vals + at.page * p.c.vps + at.token * p.c.vts + dim * 2);
            for (int i = 0; i < 4; ++i) {
                const uint4 w4 = v[i];
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                for (int e = 0; e < 4; ++e)
                    found |= ((w[e] & 0x7F80u) == 0x7F80u ? 1u : 0u) << (8 * i + 2 * e) |
                             ((w[e] & 0x7F800000u) == 0x7F800000u ? 2u : 0u) << (8 * i + 2 * e);
            }
        }
    };
    look(max(first.hi, 0), row.hi);
    look(row.lo, min(last.lo, min(first.hi, row.hi)));
    look(first.sink, min(row.sink, min(first.hi, row.lo)));
    return found;
}

// The blocks of a worker's pieces, one after another.
template <int kN>
struct BlockWalk {
    DensePieces<kM, kN> pieces;
    DensePiece pc;
    int j;
    bool more;
    __device__ __forceinline__ BlockWalk(const DenseShape& s, int unit, int worker, const DenseCut* cut)
        : pieces(s, unit, worker, cut), j(0)
    {
        enter();
    }
    __device__ __forceinline__ void enter()
    {
        do
            more = pieces.next(&pc);
        while (more && pc.blk0 >= pc.blk1);
        if (more)
            j = pc.blk0;
    }
    __device__ __forceinline__ bool first() const { return j == pc.blk0; }
    __device__ __forceinline__ bool last() const { return j + 1 >= pc.blk1; }
    __device__ __forceinline__ void step()
    {
        if (++j >= pc.blk1)
            enter();
    }
};

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_dense_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_r, const TcParams p)
{
    constexpr int kN = 128;                      // keys a block
    constexpr int U = kUnit;
    static_assert(U == 32, "a lane a token");
    constexpr int kSub = kFp8 ? 1 : 2;           // K and V tiles (sub-blocks) a block
    constexpr int kSN = kN / kSub;               // keys a sub-block
    constexpr int kKR = kSN / 2;                 // K rows of a CTA
    constexpr int kMain = kFp8 ? 4 : 8;          // 128-byte chunks of the first 512 dims
    constexpr int kVC = kMain / 2;               // chunks of a CTA's 256 value dims
    extern __shared__ __align__(1024) uint8_t smem[];
    Meta& mt = *reinterpret_cast<Meta*>(smem + kOffMeta);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const DenseShape& s = p.s;
    volatile int* abort = &mt.abort;
    const uint32_t bars = smem_u32(mt.bar);
    auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
    const uint32_t even_bars = mapa_shared(bars, 0);             // the even CTA's barriers
    auto even = [&](int i) -> uint32_t { return even_bars + 8u * static_cast<uint32_t>(i); };

    pdl_wait();
    pdl_launch_dependents();                     // the joining kernel may be set up meanwhile
    if (smem_u32(smem) & 1023u) {                // the swizzled tiles need it; both CTAs of a pair agree
        if (tid == 0 && p.status)
            atomicOr(p.status, DSA_DEV_TIMEOUT);
        return;
    }
    if (rank == 0 && tid < 2)
        p.part.slots[2 * pair + tid] = DenseSlot{0, 0, 0, 0};
    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int n = i == kSEmpty || i == kSEmpty + 1 || i == kPFull || i == kOFree || i == kQFull ? 16
                          : i == kMEmpty || i == kMEmpty + 1 || i == kGEmpty || i == kGEmpty + 1 ? 8
                          : i == kVFull || i == kVFull + 1 ? 2 : 1;
            mbar_init(bar(i), n);
        }
        mt.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&mt.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    dense_divide<kM, kN, kTileCost, kMinBlocks, kThreads>(s, U, pair, pairs, reinterpret_cast<long long*>(smem), mt.cut);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();                              // barriers of both CTAs are ready
    tc_fence_after_sync();
    const uint32_t tmem = mt.tmem;
    DensePieces<kM, kN> pieces(s, U, pair, mt.cut);
    DensePiece pc;
    constexpr int per_block = kN / U;            // units a block
    constexpr int per_sub = kSN / U;             // units a sub-block

    if (warp == 0) {
        // ================================ K tiles ===============================
        constexpr int ku = kKR / U;                              // units of this CTA's keys
        constexpr int main_loads = ku == 1 ? 1 : kMain;              // whole-row boxes, or a box a chunk
        const int per = main_loads + (kFp8 && p.rope ? 1 : 0);
        const uint32_t bytes = kFp8 ? (p.rope ? 36864u : 32768u) : (p.rope ? 36864u : 32768u);
        const int lu = lane / per, lc = lane % per;              // this lane's unit and load
        const bool mine = lu < ku;
        int n = 0;
        bool ok = true;
        while (ok && pieces.next(&pc)) {
            for (int j = pc.blk0 * kSub; j < pc.blk1 * kSub; ++j, ++n) {
                const int k = j * per_sub + rank * ku + lu;
                Place pl{p.c.num_pages, 0};
                if (mine && k < pc.t.nu)
                    pl = place_of(p.c, pc.t.seq, dense_unit_pos(pc.t, U, k), s.cap);
                const int st = n & 1;
                ok = wait_bar(bar(kKEmpty + st), ((n >> 1) & 1) ^ 1, abort);
                if (!ok)
                    break;
                // the even CTA's barrier counts both CTAs' bytes
                if (lane == 0 && rank == 0)
                    mbar_arrive_expect_tx(bar(kKFull + st), 2 * bytes);
                __syncwarp();
                if (mine) {
                    const uint32_t dst = smem_u32(smem + kOffK + st * kKBytes);
                    if (lc < main_loads)
                        tma_pair_4d(dst + (ku == 1 ? 0 : lc * (kKR * 128) + lu * (U * 128)), &tm_k, even(kKFull + st), 0,
                                    pl.token, lc, pl.page);
                    else
                        tma_pair_3d(dst + kMain * kKR * 128 + lu * (U * 64), &tm_r, even(kKFull + st), 0, pl.token, pl.page);
                }
            }
        }
        // nothing of these copies is in flight when the CTAs end: the even CTA sees
        // both CTAs' land; after a wait that gave up they get the time to
        if (rank == 0)
            for (int i = max(0, n - 2); i < n; ++i)
                mbar_wait(bar(kKFull + (i & 1)), (i >> 1) & 1);
        if (!ok) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 100000u) {
            }
        }
    } else if (warp == 1) {
        // ================================ V tiles ===============================
        // two walks: the blocks to fetch and, behind it, the blocks that have landed
        BlockWalk<kN> get(s, U, pair, mt.cut), land(s, U, pair, mt.cut);
        int n = 0, ln = 0, gsub = 0, lsub = 0;
        bool ok = true;
        auto fetch = [&]() {
            Place pl{p.c.num_pages, 0};
            const int k = get.j * per_block + gsub * per_sub + lane;
            if (lane < per_sub && k < get.pc.t.nu)
                pl = place_of(p.c, get.pc.t.seq, dense_unit_pos(get.pc.t, U, k), s.cap);
            const int st = n & 1;
            ok = wait_bar(bar(kVEmpty + st), ((n >> 1) & 1) ^ 1, abort);
            if (!ok)
                return;
            if (lane == 0)
                mbar_arrive_expect_tx(bar(kVLand + st), kVBytes);
            __syncwarp();
            if (lane < per_sub)
                tma_load_4d(smem_u32(smem + kOffV + st * kVBytes) + lane * (kVC * U * 128), &tm_v, bar(kVLand + st), 0,
                            pl.token, rank * kVC, pl.page);
            ++n;
            if (++gsub == kSub) {
                gsub = 0;
                get.step();
            }
        };
        auto announce = [&]() {
            ok = wait_bar(bar(kVLand + (ln & 1)), (ln >> 1) & 1, abort);
            if (!ok)
                return;
            {
                const int st = ln & 1, k0 = land.j * per_block + lsub * per_sub;
                uint8_t* tile = smem + kOffV + st * kVBytes;
                const DenseTile& t = land.pc.t;
                bool wrote = false;
                for (int u = 0; u < per_sub; ++u) {
                    const int k = k0 + u;
                    if (k >= t.nu)
                        break;                                   // zeros already
                    const int pos = dense_unit_pos(t, U, k);
                    if (pos + U <= t.first.hi && (pos >= t.last.lo || pos + U <= t.first.sink))
                        continue;                                // every row sees all of it
                    // rows that no query row sees become zeros, rows that some do not
                    // see too if they hold infinities or NaN (0 x NaN is NaN; who sees a NaN
                    // has it in its score, who sees an infinity with a score of -inf gets its
                    // NaN with the results)
                    wrote = true;
                    constexpr int kSeg = kVC * 8;                // 16-byte segments a row
                    for (int e = lane; e < U * kSeg; e += 32) {
                        const int row = e / kSeg, seg = e % kSeg;
                        const int x = pos + row;
                        const bool some = x < t.last.hi && (x >= t.first.lo || x < t.last.sink);
                        const bool every = x < t.first.hi && (x >= t.last.lo || x < t.first.sink);
                        uint4* at = reinterpret_cast<uint4*>(tile + u * (kVC * U * 128) + (seg >> 3) * (U * 128) +
                                                             row * 128 + (seg & 7) * 16);
                        bool bad = !some;
                        if (some && !every) {
                            const uint4 v = *at;
                            if (kFp8) {
                                const uint32_t nan = 0x7F7F7F7Fu;
                                bad = (__vcmpeq4(v.x & nan, nan) | __vcmpeq4(v.y & nan, nan) | __vcmpeq4(v.z & nan, nan) |
                                       __vcmpeq4(v.w & nan, nan)) != 0;
                            } else {
                                const uint32_t ex = 0x7F807F80u;
                                bad = (__vcmpeq2(v.x & ex, ex) | __vcmpeq2(v.y & ex, ex) | __vcmpeq2(v.z & ex, ex) |
                                       __vcmpeq2(v.w & ex, ex)) != 0;
                            }
                        }
                        if (bad)
                            *at = make_uint4(0, 0, 0, 0);
                    }
                }
                if (wrote)
                    fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    arrive_even(even(kVFull + st));
            }
            ++ln;
            if (++lsub == kSub) {
                lsub = 0;
                land.step();
            }
        };
        // fetch 0, 1, announce 0, then announce n + 1, fetch n + 2, ...: a block is announced
        // before the warp waits for the stage of the one after it
#pragma unroll 1
        for (int i = 0; ok && land.more; ++i) {
            if (i >= 2)
                announce();
            if (ok && i != 2 && get.more)
                fetch();
        }
        for (int i = max(0, n - 2); i < n; ++i)
            mbar_wait(bar(kVLand + (i & 1)), (i >> 1) & 1);
    } else if (warp == 2) {
        // ============================ MMAs (even CTA) ===========================
        // S(n + 2) is issued before O(n): it needs nothing of P(n), and the tensor cores
        // work on it while P(n) is on its way.
        // (S's MMAs are issued by a rolled loop over the 128-byte chunks: unrolled, its code
        // pushes the softmax's out of the instruction cache, 2.97 instead of 2.88 ms for 1024
        // tokens x 128 heads at 16384.)
        BlockWalk<kN> sw(s, U, pair, mt.cut), ow(s, U, pair, mt.cut);
        int nq = 0, nv = 0, sp = 0, op = 0;
        bool ok = rank == 0;
        const uint64_t sw128 = make_smem_desc(0, 16, 1024, kLayoutSw128);
        const uint64_t sw64 = make_smem_desc(0, 16, 512, kLayoutSw64);
        // V is read MN-major: 64-dim blocks of bf16 lie U rows apart
        const uint64_t vdesc = make_smem_desc(0, U * 128, 1024, kLayoutSw128);
        const uint32_t idesc_s = kFp8 ? make_idesc(0, 0, 0, 128, 128) : make_idesc(1, 1, 0, 128, 64);
        const uint32_t idesc_o = kFp8 ? make_idesc(0, 0, 1, 128, 256) : make_idesc(1, 1, 1, 128, 256);
        const uint32_t base = smem_u32(smem);
        const int rope = p.rope;
        int nk = 0, nw = 0;                                      // sub-blocks of K and V used
        auto issue_s = [&]() {
            const int b = nq & 1;
            const uint32_t ph = (nq >> 1) & 1;
            ok = (!sw.first() || wait_bar(bar(kQFull), sp & 1, abort)) && wait_bar(bar(kSEmpty + b), ph ^ 1, abort);
#pragma unroll 1
            for (int sub = 0; ok && sub < kSub; ++sub, ++nk) {
                const int kb_i = nk & 1;
                ok = wait_bar(bar(kKFull + kb_i), (nk >> 1) & 1, abort);
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint32_t kb = base + kOffK + kb_i * kKBytes;
                    const uint32_t d = tmem + kSCol + 64u * b + 32u * sub;
                    if constexpr (kFp8) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const uint64_t qd = sw128 + ((base + c * 8192) >> 4), kd = sw128 + ((kb + c * 8192) >> 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                mma_pair<kFp8>(d, qd + 2 * i, kd + 2 * i, idesc_s, c + i > 0 ? 1u : 0u);
                                mma_pair<kFp8>(d, qd + (kQBytes / 2 >> 4) + 2 * i, kd + 2 * i, idesc_s, 1u);
                            }
                        }
                        if (rope) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t off = 32768 + i * 32;
                                const uint64_t bd = sw64 + ((kb + off) >> 4);
                                mma_pair<kFp8>(d, sw64 + ((base + off) >> 4), bd, idesc_s, 1u);
                                mma_pair<kFp8>(d, sw64 + ((base + kQBytes / 2 + off) >> 4), bd, idesc_s, 1u);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 8 + rope; ++c) {
                            const uint64_t qd = sw128 + ((base + c * 8192) >> 4), kd = sw128 + ((kb + c * 4096) >> 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_pair<kFp8>(d, qd + 2 * i, kd + 2 * i, idesc_s, c + i > 0 ? 1u : 0u);
                        }
                    }
                    commit_pair(bar(kKEmpty + kb_i));
                    if (sub == kSub - 1)
                        commit_pair(bar(kSFull + b));
                }
                __syncwarp();
            }
            if (!ok)
                return;
            ++nq;
            sp += sw.last() ? 1 : 0;
            sw.step();
        };
        auto issue_o = [&]() {
            const bool begins = ow.first();
            ok = (!begins || wait_bar(bar(kOFree), (op & 1) ^ 1, abort)) && wait_bar(bar(kPFull), nv & 1, abort);
#pragma unroll 1
            for (int sub = 0; ok && sub < kSub; ++sub, ++nw) {
                const int b = nw & 1;
                ok = wait_bar(bar(kVFull + b), (nw >> 1) & 1, abort);
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint32_t vb = base + kOffV + b * kVBytes, pb = base + kOffP + (kFp8 ? 0 : sub * 8192);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        constexpr int kStep = kSN / 4;                   // keys an MMA
                        const uint32_t at = vb + (ks * kStep / U) * (kVC * U * 128) + (ks * kStep % U) * 128;
                        const uint32_t acc = !begins || ks > 0 || sub > 0 ? 1u : 0u;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint64_t bd = vdesc + ((at + hf * (kFp8 ? 1 : 2) * U * 128) >> 4);
                            mma_pair<kFp8>(tmem + hf * 128, sw128 + ((pb + ks * 32) >> 4), bd, idesc_o, acc);
                            if (kFp8)
                                mma_pair<kFp8>(tmem + hf * 128, sw128 + ((pb + 8192 + ks * 32) >> 4), bd, idesc_o, 1u);
                        }
                    }
                    if (sub == kSub - 1)
                        commit_pair(bar(kPvDone));
                    commit_pair(bar(kVEmpty + b));
                }
                __syncwarp();
            }
            if (!ok)
                return;
            ++nv;
            op += ow.last() ? 1 : 0;
            ow.step();
        };
        // (a piece's Q is written once the piece before has its last P)
#pragma unroll 1
        while (ok && ow.more) {
            if (sw.more && nq < nv + 3 && (nq == nv || !sw.first()))
                issue_s();
            else
                issue_o();
        }
        // every MMA is done before the CTAs give their TMEM back
        if (rank == 0) {
            if (elect_one())
                commit_pair(bar(kDrain));
            __syncwarp();
            mbar_wait(bar(kDrain), 0);
        }
    } else if (warp == 3) {
        // ===================== token scales, positions, masks ===================
        int n = 0, g = 0;
        bool ok = true;
        auto publish = [&](int nblk) {
            ok = wait_bar(bar(kGEmpty + (g & 1)), ((g >> 1) & 1) ^ 1, abort);
            if (!ok)
                return;
            if (lane == 0) {
                const DenseTile& t = pc.t;
                PieceInfo& o = mt.piece[g & 1];
                o.nblk = nblk;
                if (nblk >= 0) {
                    o.row0 = t.row0;
                    o.m0 = t.m0;
                    o.nrows = t.nrows;
                    o.L = t.L;
                    o.n = t.n;
                    o.slot = pc.slot;
                    o.seq = t.seq;
                    o.flags = 1 | (pc.blk0 == 0 ? 2 : 0) | (pc.blk1 == t.nblk ? 4 : 0);
                    // the piece's q rows to L2: they are read a few blocks later
                    const int rows = min(64, t.nrows - rank * 64);
                    if (nblk > 0 && rows > 0) {
                        const uint32_t row_bytes = p.rope ? 1152u : 1024u;
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                         reinterpret_cast<const uint8_t*>(p.q) + (static_cast<int64_t>(t.row0) + rank * 64) * row_bytes),
                                     "r"(rows * row_bytes)
                                     : "memory");
                    }
                }
                mbar_arrive(bar(kGFull + (g & 1)));
            }
            __syncwarp();
            ++g;
        };
        while (ok) {
            const bool more = pieces.next(&pc);
            publish(more ? pc.blk1 - pc.blk0 : -1);
            if (!more || !ok)
                break;
            const DenseTile& t = pc.t;
            // lane u < per_block holds unit u of block j: its place, fetched a block ahead
            auto unit_pos = [&](int j) -> int {
                const int k = j * per_block + lane;
                return lane < per_block && k < t.nu ? dense_unit_pos(t, U, k) : -1;
            };
            auto scales = [&](const Place& pl, int pos, float (&v)[4]) {
                if (!kFp8)
                    return;
                // lane e finds unit e's row of scales, every lane reads the keys 32 e + lane
                const uint64_t mine = pl.page < p.c.num_pages
                                          ? reinterpret_cast<uint64_t>(p.c.scs + pl.page * p.c.sps + pl.token * p.c.sts) : 0;
                const int64_t step = lane * p.c.sts;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t row = __shfl_sync(0xffffffffu, mine, e);
                    const int x = __shfl_sync(0xffffffffu, pos, e) + lane;
                    const bool some = x < t.last.hi && (x >= t.first.lo || x < t.last.sink);
                    // (-0 marks a key that no row sees)
                    v[e] = some && row ? *reinterpret_cast<const float*>(row + step) : -0.f;
                }
            };
            if (pc.blk0 < pc.blk1 && t.over && rank == 0 && lane == 0 && p.status)
                atomicOr(p.status, DSA_DEV_BAD_INDEX);
            // A turn fetches block j's scales (v) and block j + 1's pages, and writes block j - 1's
            // scales (w).  Turns come in pairs, so that nothing has to move from v to w: a move
            // would wait for the loads.  Long contexts' scales come from HBM: without the two
            // turns' lead and the hint to L2 the softmax waited 1000 cycles a block for them.
            int pos = -1, pos1 = pc.blk0 < pc.blk1 ? unit_pos(pc.blk0) : -1;
            Place pl{p.c.num_pages, 0}, pl1 = place_of(p.c, t.seq, pos1, s.cap);
            float va[4] = {0.f, 0.f, 0.f, 0.f}, vb[4] = {0.f, 0.f, 0.f, 0.f};
            auto turn = [&](int j, const float (&w)[4], float (&v)[4]) {
                scales(pl1, pos1, v);
                const int pos2 = j + 1 < pc.blk1 ? unit_pos(j + 1) : -1;
                const Place pl2 = place_of(p.c, t.seq, pos2, s.cap);
                if (kFp8 && pl2.page < p.c.num_pages) {          // its scales to L2 meanwhile
                    const uint8_t* sc = p.c.scs + pl2.page * p.c.sps + pl2.token * p.c.sts;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(sc));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(sc + (U / 2) * p.c.sts));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(sc + (U - 1) * p.c.sts));
                }
                if (j > pc.blk0) {
                    const bool bad = pos >= 0 && pl.page >= p.c.num_pages;
                    const bool whole = pos >= 0 && pos + U <= t.first.hi && (pos >= t.last.lo || pos + U <= t.first.sink);
                    const bool edge = __any_sync(0xffffffffu, lane < per_block && (bad || !whole));
                    if (bad && rank == 0 && p.status)
                        atomicOr(p.status, DSA_DEV_BAD_INDEX);
                    // even lanes take the pairs of keys 0-63, odd lanes those of 64-127
                    const bool odd = lane & 1;
                    bool far = false;
                    float lg[2];
                    if (kFp8) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = __float_as_uint(odd ? w[2 + e] : w[e]);
                            const uint32_t o = __shfl_xor_sync(0xffffffffu, __float_as_uint(odd ? w[e] : w[2 + e]), 1);
                            // magnitudes as bits, which differ by about 2^23 log2 of their ratio
                            const uint32_t ax = x & 0x7FFFFFFFu, ao = o & 0x7FFFFFFFu, hi = max(ax, ao);
                            far |= hi - min(ax, ao) > kFarBits && x != 0x80000000u && o != 0x80000000u;
                            lg[e] = log2_above(hi);
                        }
                        far = __any_sync(0xffffffffu, far);
                    }
                    const int st = n & 1;
                    ok = wait_bar(bar(kMEmpty + st), ((n >> 1) & 1) ^ 1, abort);
                    if (!ok)
                        return;
                    if (lane < per_block)
                        mt.unit[st][lane] = pos >= 0 && !bad ? pos : -1;
                    if (kFp8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mt.scale[st][e * 32 + lane] = w[e];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            mt.lgp[st][((odd ? 2 : 0) + e) * 16 + (lane >> 1)] = lg[e];
                    }
                    if (lane == 0)
                        mt.edge[st] = (edge ? 1 : 0) | (far ? 2 : 0);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(kMFull + st));
                    ++n;
                }
                pos = pos1;
                pos1 = pos2;
                pl = pl1;
                pl1 = pl2;
            };
#pragma unroll 1
            for (int j = pc.blk0; ok && j <= pc.blk1; j += 2) {
                turn(j, va, vb);
                if (ok && j < pc.blk1)
                    turn(j + 1, vb, va);
            }
        }
    } else {
        // ================================ softmax ===============================
        // Thread (quarter, lane, half): row r = TMEM lane mod 64, keys 32 half + 64 (lane
        // >= 64) of the block (bf16: half as many), value dims 256 (lane >= 64) + 128 half.
        constexpr int kC = 32;                                   // scores of a thread
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const int tl = quarter * 32 + lane, r = tl & 63, side = tl >> 6;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        // (bf16: the two halves are the two sub-blocks)
        const int key0 = kFp8 ? side * 64 + half * 32 : half * 64 + side * 32;
        const int bar_id = 1 + (quarter & 1);                    // the four warps of 32 rows
        float* mx_mine = &mt.mx[side * 2 + half][r];
        // Q of a piece (the MMAs that read the piece's before it are done)
        const int qw = warp - 4, segs = p.rope ? 72 : 64;        // rows 8 qw .. + 7; 16-byte segments a row
        auto load_q = [&](const PieceInfo& pi, int which) {
            const __nv_bfloat16* src = p.q + (static_cast<int64_t>(pi.row0) + rank * 64) * (segs * 8);
            const int nrows = pi.nrows - rank * 64;
            // two rows a turn, the next two on their way
            uint4 v[2][3];
            auto fetch = [&](int r0, uint4 (&o)[2][3]) {
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        const int sg = e * 32 + lane;
                        o[a][e] = make_uint4(0, 0, 0, 0);
                        if (sg < segs && r0 + a < nrows)
                            o[a][e] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r0 + a) * (segs * 8) + sg * 8);
                    }
            };
            fetch(qw * 8, v);
#pragma unroll 1
            for (int r0 = qw * 8; r0 < qw * 8 + 8; r0 += 2) {
                uint4 nx[2][3];
                fetch(r0 + 2 < qw * 8 + 8 ? r0 + 2 : nrows, nx);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int qr = r0 + a;
                    float sc = 1.f;
                    if (kFp8) {
                        // max |q| of the row: bit patterns of non-negative bf16 order like their values
                        uint32_t m2 = 0;
#pragma unroll
                        for (int e = 0; e < 3; ++e) {
                            m2 = __vmaxu2(m2, __vmaxu2(v[a][e].x & 0x7FFF7FFFu, v[a][e].y & 0x7FFF7FFFu));
                            m2 = __vmaxu2(m2, __vmaxu2(v[a][e].z & 0x7FFF7FFFu, v[a][e].w & 0x7FFF7FFFu));
                        }
                        const int top = static_cast<int>(__reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16)));
                        // times 2^e the largest, (1 + m / 128) 2^(E - 127), lies in [224, 448]; a row
                        // with infinities or NaN becomes NaN as a whole, and so its scores (but not
                        // what stands for the scores of keys that it does not see)
                        int e2 = min(100, ((top & 0x7F) <= 96 ? 135 : 134) - (top >> 7));   // -120 at least
                        e2 = top == 0 || top >= 0x7F80 ? 0 : e2;
                        if (lane == 0)
                            mt.qe[which & 1][qr] = static_cast<int8_t>(e2);
                        sc = top >= 0x7F80 ? __int_as_float(0x7FC00000) : __int_as_float((127 + e2) << 23);
                    }
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        const int sg = e * 32 + lane;
                        if (sg >= segs)
                            continue;
                        const uint32_t w[4] = {(v[a][e].x ^ p.flip) | p.nan, (v[a][e].y ^ p.flip) | p.nan,
                                               (v[a][e].z ^ p.flip) | p.nan, (v[a][e].w ^ p.flip) | p.nan};
                        if constexpr (kFp8) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                split_e4m3(__floats2half2_rn(__uint_as_float(w[i] << 16) * sc,
                                                             __uint_as_float(w[i] & 0xFFFF0000u) * sc), &hi[i], &lo[i]);
                            // 8 bytes of dims 8 sg: main chunk sg / 16, or the 64-byte rope rows
                            uint32_t off;
                            if (e < 2)
                                off = (sg >> 4) * 8192 + swizzled_offset(qr, (sg & 15) >> 1, 128) + (sg & 1) * 8;
                            else
                                off = 32768 + swizzled_offset(qr, (sg - 64) >> 1, 64) + (sg & 1) * 8;
                            *reinterpret_cast<uint2*>(smem + off) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                            *reinterpret_cast<uint2*>(smem + kQBytes / 2 + off) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                        } else {
                            *reinterpret_cast<uint4*>(smem + (sg >> 3) * 8192 + swizzled_offset(qr, sg & 7, 128)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        v[a][e] = nx[a][e];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                arrive_even(even(kQFull));
        };
        int n = 0, piece = 0;
        bool ok = true;
        // (every warp of the softmax leaves the loop where the others do: they meet at
        // named barriers)
        auto piece_info = [&](int g) -> int {
            ok = wait_bar(bar(kGFull + (g & 1)), (g >> 1) & 1, abort);
            return named_bar_or(3, 256, !ok) ? -1 : mt.piece[g & 1].nblk;
        };
        // turn g: the blocks of piece g, Q of piece g + 1, the results of piece g
        int nblk = 0;
#pragma unroll 1
        for (int g = -1; nblk >= 0; ++g) {
            const PieceInfo& pi = mt.piece[g & 1];
            const int m = rank * 64 + r;
            const DenseKeys keys = g >= 0 && m < pi.nrows ? dense_keys(s, pi.L, pi.n, (pi.m0 + m) / s.num_heads) : DenseKeys{0, 0, 0};
            float m_run = -INFINITY, l_run = 0.f, rf = 0.f;
            float n_run = 0.f;                                   // bf16: the sum of the rounded P
            float rec = -INFINITY, u = 0.f;                      // FP8: what the reference goes down by
            bool inf_seen = false;                               // bf16: a score of -inf where a mask is needed
            for (int j = 0; j < nblk; ++j, ++n) {
                const int b = n & 1;
                const uint32_t ph = (n >> 1) & 1;
                uint32_t ra[kC];
                if (ok)
                    ok = wait_bar(bar(kSFull + b), ph, abort);
                if (ok && j == 0) {                              // (read before the score buffer is given back)
                    const int e2 = kFp8 ? mt.qe[piece & 1][r] : 0;
                    rf = fmaxf(p.scale_log2 * __int_as_float((127 - e2) << 23), __int_as_float(1));   // (times -inf it stays -inf)
                }
                if (ok) {
                    tc_fence_after_sync();
                    tmem_ld_32x32b_x32(lane_base + kSCol + 64u * b + half * kC, ra);
                    tmem_ld_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        arrive_even(even(kSEmpty + b));
                    ok = wait_bar(bar(kMFull + b), ph, abort);
                }
                float f = 1.f;
                uint32_t ph4[kFp8 ? 8 : 16], pl4[8];
                const int edge = ok ? mt.edge[b] : 0;
                // The probabilities of the block, twice: blocks that need no mask and whose scales
                // are near one another (all but a few) take code without either, because what a
                // loop steps over still has to be fetched.
                auto probabilities = [&](auto cold) {
                constexpr bool kCold = decltype(cold)::value;
                // scores times the token scales
                uint64_t x2[kC / 2];
                const ulonglong2* sc4 = reinterpret_cast<const ulonglong2*>(&mt.scale[b][key0]);
#pragma unroll
                for (int i = 0; i < kC / 4; ++i) {
                    x2[2 * i] = pack_f32x2(__uint_as_float(ra[4 * i]), __uint_as_float(ra[4 * i + 1]));
                    x2[2 * i + 1] = pack_f32x2(__uint_as_float(ra[4 * i + 2]), __uint_as_float(ra[4 * i + 3]));
                    if constexpr (kFp8) {
                        const ulonglong2 sv = sc4[i];
                        x2[2 * i] = mul_f32x2(x2[2 * i], sv.x);
                        x2[2 * i + 1] = mul_f32x2(x2[2 * i + 1], sv.y);
                    }
                }
                uint32_t see = 0xFFFFFFFFu;
                if (kCold && (edge & 1)) {
                    const int base = mt.unit[b][key0 / U];
                    see = base < 0 ? 0u : dense_mask32(keys, base + key0 % U);
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) {
                        float2 x = unpack_f32x2(x2[i]);
                        if (!kFp8)
                            inf_seen |= (x.x == -INFINITY && (see >> (2 * i) & 1u)) || (x.y == -INFINITY && (see >> (2 * i + 1) & 1u));
                        x.x = see >> (2 * i) & 1u ? x.x : -INFINITY;
                        x.y = see >> (2 * i + 1) & 1u ? x.y : -INFINITY;
                        x2[i] = pack_f32x2(x.x, x.y);
                    }
                }
                float mblk = -INFINITY;
                if (kFp8 && !(kCold && (edge & 2))) {
                    // score + log2 of the scale, of the larger scale of two neighbours (at most 2.6 too high)
                    const ulonglong2* lg4 = reinterpret_cast<const ulonglong2*>(&mt.lgp[b][key0 / 2]);
                    const uint64_t rf2 = pack_f32x2(rf, rf);
                    float m1 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kC / 8; ++i) {
                        const ulonglong2 lg = lg4[i];
                        const float2 a0 = unpack_f32x2(x2[4 * i]), a1 = unpack_f32x2(x2[4 * i + 1]);
                        const float2 a2 = unpack_f32x2(x2[4 * i + 2]), a3 = unpack_f32x2(x2[4 * i + 3]);
                        const float2 y0 = unpack_f32x2(fma_f32x2(pack_f32x2(fmaxf(a0.x, a0.y), fmaxf(a1.x, a1.y)), rf2, lg.x));
                        const float2 y1 = unpack_f32x2(fma_f32x2(pack_f32x2(fmaxf(a2.x, a2.y), fmaxf(a3.x, a3.y)), rf2, lg.y));
                        mblk = fmaxf(fmaxf(mblk, y0.x), y0.y);
                        m1 = fmaxf(fmaxf(m1, y1.x), y1.y);
                    }
                    mblk = fmaxf(mblk, m1);
                } else if (kFp8) {
                    // neighbours' scales far apart: each key's own
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) {
                        const float2 x = unpack_f32x2(x2[i]);
                        const float2 sc = *reinterpret_cast<const float2*>(&mt.scale[b][key0 + 2 * i]);
                        mblk = fmaxf(mblk, fmaf(x.x, rf, log2_above(__float_as_uint(sc.x) & 0x7FFFFFFFu)));
                        mblk = fmaxf(mblk, fmaf(x.y, rf, log2_above(__float_as_uint(sc.y) & 0x7FFFFFFFu)));
                    }
                } else {
                    float m1 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) {
                        const float2 x = unpack_f32x2(x2[i]);
                        mblk = fmaxf(mblk, x.x);
                        m1 = fmaxf(m1, x.y);
                    }
                    mblk = fmaxf(mblk, m1) * rf;
                }
                named_bar_sync(bar_id, 128);                     // the block before has been read
                *mx_mine = mblk;
                named_bar_sync(bar_id, 128);
                mblk = fmaxf(fmaxf(mt.mx[0][r], mt.mx[1][r]), fmaxf(mt.mx[2][r], mt.mx[3][r]));
                rec = fmaxf(mblk, rec - kFade);
                const bool fall = kFp8 && u < 0.f && rec < m_run - kGap && mblk > -INFINITY;
                if (mblk > m_run + (kFp8 ? kGrow : 8.f) || fall) {
                    const float to = fall ? fmaxf(rec, m_run - kDeep) : mblk;
                    f = m_run == -INFINITY ? 1.f : ex2_approx(m_run - to);
                    l_run *= f;
                    n_run *= f;
                    u = fall ? f * f : u * f * f;                // (the sum held 1 at least before it fell)
                    m_run = to;
                }
                const float m_use = m_run == -INFINITY ? 0.f : (kFp8 ? m_run - kHead : m_run);
                // What P's last step, 2^-9, rounds: every other key gets the same offset of up to half
                // a step either way, another one in each of the row's threads and in each block, so
                // that P of 2^-10 and less do not all become 0 (131072 such keys 12 nats below one: 13 %
                // of the result were lost).  0 stays 0.
                uint64_t dither = 0;
                if constexpr (kFp8) {
                    const float top = ex2_approx(mblk - (m_use + kHead));
                    u = fmaf(top, top, u - kNoise);
                    const uint32_t at = static_cast<uint32_t>(j) * 0x9E3779B9u + static_cast<uint32_t>(side * 2 + half) * 0x20000000u;
                    auto offset = [&](uint32_t k) -> float {     // 2^-9 to 2^-8, less the middle
                        return __uint_as_float((at + k) >> 9 | 0x3B000000u) - 0.0029296875f;
                    };
                    dither = pack_f32x2(offset(0), offset(0x80000000u));
                }
                {
                    const uint64_t rf2 = pack_f32x2(rf, rf), neg = pack_f32x2(-m_use, -m_use);
                    uint64_t l2 = pack_f32x2(0.f, 0.f), n2 = l2;
#pragma unroll
                    for (int i = 0; i < kC / 4; ++i) {
                        uint32_t hi[2], lo[2];
                        ulonglong2 sv = make_ulonglong2(0, 0);
                        if constexpr (kFp8)
                            sv = sc4[i];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 y = unpack_f32x2(fma_f32x2(x2[2 * i + e], rf2, neg));
                            const uint64_t pp = pack_f32x2(ex2_approx(y.x), ex2_approx(y.y));     // -inf -> 0
                            l2 = add_f32x2(l2, pp);
                            const float2 w = unpack_f32x2(kFp8 ? fma_f32x2(pp, e == 0 ? sv.x : sv.y, dither) : pp);
                            if constexpr (kFp8) {
                                split_e4m3(__floats2half2_rn(w.x, w.y), &hi[e], &lo[e]);
                            } else {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(w.x, w.y);
                                const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
                                ph4[2 * i + e] = u;
                                n2 = add_f32x2(n2, pack_f32x2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)));
                            }
                        }
                        if constexpr (kFp8) {
                            ph4[i] = hi[0] | hi[1] << 16;
                            pl4[i] = lo[0] | lo[1] << 16;
                        }
                    }
                    const float2 ls = unpack_f32x2(l2);
                    l_run += ls.x + ls.y;
                    if constexpr (!kFp8) {
                        const float2 ns = unpack_f32x2(n2);
                        n_run += ns.x + ns.y;
                    }
                }
                if (kCold && kFp8 && (edge & 1)) {
                    // an unseen token's scale may be infinite or NaN: its P bytes become zeros
#pragma unroll
                    for (int i = 0; i < kC / 4; ++i) {
                        const uint32_t nib = see >> (4 * i) & 15u;
                        const uint32_t keep = (nib & 1u ? 0xFFu : 0u) | (nib & 2u ? 0xFF00u : 0u) |
                                              (nib & 4u ? 0xFF0000u : 0u) | (nib & 8u ? 0xFF000000u : 0u);
                        ph4[i] &= keep;
                        pl4[i] &= keep;
                    }
                }
                };
                if (edge == 0)
                    probabilities(std::false_type{});
                else
                    probabilities(std::true_type{});
                if (ok) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(kMEmpty + b));
                    // P(n - 1) and O of the blocks before are done with
                    ok = wait_bar(bar(kPvDone), (n & 1) ^ 1, abort);
                }
                if (ok) {
                    if (__builtin_expect(__any_sync(0xffffffffu, f != 1.f) && j > 0, 0)) {
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[16];
                            const uint32_t at = lane_base + half * 128 + c * 16;
                            tmem_ld_32x32b_x16(at, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st_32x32b_x16(at, o);
                        }
                        tmem_st_wait();
                    }
                    // FP8: 32 bytes of the row in the tile of each part; bf16: 64 in its sub-block's
                    uint8_t* pt = smem + kOffP + (kFp8 ? 0 : half * 8192);
                    const int ch = side * 4 + (kFp8 ? half * 2 : 0);
#pragma unroll
                    for (int i = 0; i < (kFp8 ? 2 : 4); ++i)
                        *reinterpret_cast<uint4*>(pt + swizzled_offset(r, ch + i, 128)) =
                            make_uint4(ph4[4 * i], ph4[4 * i + 1], ph4[4 * i + 2], ph4[4 * i + 3]);
                    if constexpr (kFp8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<uint4*>(pt + 8192 + swizzled_offset(r, ch + i, 128)) =
                                make_uint4(pl4[4 * i], pl4[4 * i + 1], pl4[4 * i + 2], pl4[4 * i + 3]);
                    }
                    fence_proxy_async_smem();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        arrive_even(even(kPFull));
                }
            }
            // ---- the piece's rows: O / l, lse
            // the next piece's Q, while O of the last block is being formed
            const int next = piece_info(g + 1);
            if (next > 0 && ok)
                load_q(mt.piece[(g + 1) & 1], piece + (nblk > 0 ? 1 : 0));
            if (g < 0) {
                nblk = next;
                continue;
            }
            const bool any = nblk > 0, row_ok = m < pi.nrows;
            const int slot = pi.slot;
            const int64_t row = static_cast<int64_t>(pi.row0) + m;
            named_bar_sync(bar_id, 128);
            *mx_mine = inf_seen ? -l_run : l_run;                // (sums of probabilities: the sign is free)
            named_bar_sync(bar_id, 128);
            const float l = (fabsf(mt.mx[0][r]) + fabsf(mt.mx[1][r])) + (fabsf(mt.mx[2][r]) + fabsf(mt.mx[3][r]));
            if (!kFp8)
                inf_seen = (signbit(mt.mx[0][r]) || signbit(mt.mx[1][r]) || signbit(mt.mx[2][r]) || signbit(mt.mx[3][r])) && row_ok;
            if (any && ok)
                ok = wait_bar(bar(kPvDone), (n & 1) ^ 1, abort);
            const bool some = l > 0.f || l != l;                 // NaN stays NaN
            float inv = some ? 1.f / l : 0.f;
            if constexpr (!kFp8) {
                // O is divided by the sum of the P that it was formed with, so that a row with a
                // single heavy key does not carry that P's rounding; lse keeps the unrounded sum
                named_bar_sync(bar_id, 128);
                *mx_mine = n_run;
                named_bar_sync(bar_id, 128);
                inv = some ? 1.f / ((mt.mx[0][r] + mt.mx[1][r]) + (mt.mx[2][r] + mt.mx[3][r])) : 0.f;
            }
            if (any && ok)
                tc_fence_after_sync();
            // 64 bytes a row at a time, turned in this warp's 2 KB of the P tile (the part of its
            // own 32 rows, which no warp of the other 32 writes and whose next P follows the next
            // block's barriers), so that four lanes store a row's
            const int dim0 = side * 256 + half * 128;
            const bool live = any && ok;
            uint8_t* turn = smem + kOffP + (half * 8192) + (quarter & 1) * 4096 + side * 2048;
            const int trow = (quarter * 32 & 63) + (lane >> 2);          // this lane's first row of a store
            const bool whole = slot < 0;
            const int turns = whole ? 4 : 8;                             // 32 bf16 or 16 fp32 columns each
            uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(p.out + (static_cast<int64_t>(pi.row0) + rank * 64 + trow) * 512 + dim0)
                                 : reinterpret_cast<uint8_t*>(p.part.o + (static_cast<int64_t>(slot) * p.part.slot_rows +
                                                                          rank * 64 + trow) * 512 + dim0);
            const int64_t pitch = whole ? 1024 : 2048;
#pragma unroll 1
            for (int c = 0; c < turns; ++c) {
                uint32_t o[32];
                __syncwarp();
                if (live) {
                    if (whole)
                        tmem_ld_32x32b_x32(lane_base + half * 128 + c * 32, o);
                    else
                        tmem_ld_32x32b_x16(lane_base + half * 128 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(o));
                    tmem_ld_wait();
                    if (c == turns - 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0)
                            arrive_even(even(kOFree));
                    }
                }
                // (a row without a sum has zeros here, or NaN where it saw infinities)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    o[i] = live ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
                if constexpr (!kFp8) {
                    if (inf_seen) {
                        const uint32_t nan = masked_infinities(p, pi, keys, dim0 + (whole ? c * 32 : (c >> 1) * 32)) >>
                                             (whole ? 0 : (c & 1) * 16);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = nan >> i & 1u ? 0x7FC00000u : o[i];
                    }
                }
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                        o[i] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4*>(turn + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) =
                        make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int lr = i * 8 + (lane >> 2);                  // row of the warp's 32
                    const uint4 v = *reinterpret_cast<const uint4*>(turn + lr * 64 + (((lane & 3) ^ (lr >> 1 & 3)) << 4));
                    if (rank * 64 + trow + i * 8 < pi.nrows)
                        *reinterpret_cast<uint4*>(dst + i * 8 * pitch + c * 64 + (lane & 3) * 16) = v;
                }
            }
            if (side == 0 && half == 0 && row_ok) {
                const float m_use = m_run == -INFINITY ? 0.f : (kFp8 ? m_run - kHead : m_run);
                // l's exponent meets m before its fraction's logarithm: they may nearly cancel
                int ex;
                const float fr = frexpf(l, &ex);
                const float z = some ? ((m_use + static_cast<float>(ex)) + log2f(fr)) * 0.69314718055994531f : -INFINITY;
                if (slot < 0)
                    p.lse[row] = z;
                else
                    p.part.lse[static_cast<int64_t>(slot) * p.part.slot_rows + m] = z;
            }
            if (slot >= 0 && rank == 0 && tid == 4 * 32)
                p.part.slots[slot] = DenseSlot{pi.row0, pi.nrows, pi.flags, 0};
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(kGEmpty + (g & 1)));
            piece += any ? 1 : 0;
            nblk = next;
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();                              // neither CTA touches the other's memory any more
    tc_fence_after_sync();
    if (tid == 0 && *abort && p.status)
        atomicOr(p.status, DSA_DEV_TIMEOUT);
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    cluster_sync();
}

}  // namespace

bool mla_dense_tc_supported(const DenseArgs& a)
{
    const dsa_paged_cache* c = a.kv;
    constexpr int64_t most = int64_t(1) << 40;           // a tensor map's strides lie below
    return a.d_v == 512 && (a.d_qk == 512 || a.d_qk == 576) && c->page_kv % 32 == 0 &&
           c->val_token_stride < most && c->val_page_stride < most;
}

dsa_status launch_mla_dense_tc(const DenseArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    const dsa_paged_cache* c = a.kv;
    const bool fp8 = c->fmt == DSA_KV_FP8_E4M3;
    const int sub = fp8 ? 128 : 64;          // keys a K tile
    TcParams p;
    p.s = dense_shape(a);
    p.c = dense_cache(c);
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.rope = a.d_qk == 576;
    const float scale = a.softmax_scale * 1.4426950408889634f;
    const float mag = scale < 0.f ? -scale : scale;
    p.scale_log2 = scale != scale ? 0.f : mag;
    p.flip = scale < 0.f ? 0x80008000u : 0u;
    p.nan = scale != scale ? 0x7FFF7FFFu : 0u;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.status = a.status;
    int pairs = dev.sm_count / 2;
    pairs = pairs < kDenseMaxWorkers / 2 ? pairs : kDenseMaxWorkers / 2;
    p.part = dense_partials(a, pairs, kM);
    // the pages as [page][128-byte chunk of a row][token][128 bytes]
    const CUtensorMapDataType dt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t elems = fp8 ? 128 : 64;
    const int chunks = fp8 ? 4 : (p.rope ? 9 : 8);
    const uint64_t dims[4] = {elems, static_cast<uint64_t>(c->page_kv), static_cast<uint64_t>(chunks),
                              static_cast<uint64_t>(c->num_pages)};
    const uint64_t strides[3] = {static_cast<uint64_t>(c->val_token_stride), 128,
                                 static_cast<uint64_t>(c->val_page_stride)};
    const uint32_t box = kUnit;
    const uint32_t kbox[4] = {static_cast<uint32_t>(elems), box,
                              static_cast<uint32_t>(kUnit == sub / 2 ? chunks : 1), 1};
    const uint32_t vbox[4] = {static_cast<uint32_t>(elems), box, static_cast<uint32_t>(fp8 ? 2 : 4), 1};
    CUtensorMap tm_k, tm_v, tm_r;
    dsa_status st = encode_tiled(&tm_k, dt, 4, c->values, dims, strides, kbox, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == DSA_OK)
        st = encode_tiled(&tm_v, dt, 4, c->values, dims, strides, vbox, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != DSA_OK)
        return st;
    tm_r = tm_k;
    if (fp8 && p.rope) {
        // the last 64 dims of a row
        const uint64_t rdims[3] = {64, static_cast<uint64_t>(c->page_kv), static_cast<uint64_t>(c->num_pages)};
        const uint64_t rstr[2] = {static_cast<uint64_t>(c->val_token_stride), static_cast<uint64_t>(c->val_page_stride)};
        const uint32_t rbox[3] = {64, box, 1};
        st = encode_tiled(&tm_r, dt, 3, static_cast<const uint8_t*>(c->values) + 512, rdims, rstr, rbox,
                          CU_TENSOR_MAP_SWIZZLE_64B);
        if (st != DSA_OK)
            return st;
    }
    auto kern = fp8 ? mla_dense_tc_kernel<true> : mla_dense_tc_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
        return cuda_fail(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, tm_r, p);
    if (e != cudaSuccess)
        return cuda_fail(e);
    st = check_launch();
    if (st != DSA_OK || !dense_may_cut(a, kM, 128, kUnit, kMinBlocks))
        return st;
    return launch_dense_join(p.part, pairs, a, dev, stream);
}

}  // namespace dsa
