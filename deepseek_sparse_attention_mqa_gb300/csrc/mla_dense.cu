// mla_dense.cu -- dense MLA attention over a paged latent cache, any shape: the
// mma.sync kernel for shapes and page sizes that the tcgen05 kernel does not
// take, and the kernel that joins the partial results of cut tiles (both
// kernels').
//
//   s_j = c q . k_j over the keys j a row sees,  out = sum_j softmax(s)_j v_j,
//   lse = ln sum_j exp(s_j),  v_j = the first d_v elements of k_j
//
// One pass over the keys with a running maximum m and sum l (base 2): O and l are
// multiplied by 2^(m_old - m_new) when m grows.  A CTA of 8 warps owns a tile of
// 64 query rows (kM) and walks its keys in blocks of 32 (kN): the block's rows are
// fetched through the block table and widened to bf16 in shared memory (exact for
// e4m3 codes; the token scale is applied to the fp32 scores and probabilities),
// S = Q K^T with m16n8k16 (4 warps of rows x 2 of keys), the softmax in fp32 with
// four threads a row, P as the sum of two bf16 (off by 2^-17; one bf16's rounding, the
// size of the output's own, made results up to 1.5 times as far off as the output's
// rounding alone), and O += P V with every warp owning d_v / 8 columns of all 64 rows, in
// registers.  Bound by its load - multiply - softmax chain, four
// barriers and 1.7 us a block of 80-element rows (two decode rows of 4 heads, 317 keys: 24 us).
// With 576 / 512 latents in pages of 16: 1024 tokens x 128 heads at 16384 37.4 ms (121 TFLOP/s), 64
// decode rows x 128 heads at 8192 2.04 ms (the tcgen05 kernel with pages of 32: 2.92 ms and 0.14).  It is
// the kernel that is right for every shape, not the fast one.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "host.h"
#include "mla_dense.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kM = 64;                // query rows a tile
constexpr int kN = 32;                // keys a block (and a unit)
constexpr int kThreads = 256;
constexpr int kTileCost = 2;
// A cut costs a second launch and its loads, about ten blocks; contexts of up to 1024 keys
// stay whole (two decode rows of 4 heads: 1023 keys whole 63 us, 1100 keys cut 42 us, so that the
// border is on the safe side).
constexpr int kMinBlocks = 16;
constexpr int kPPitch = kN + 8;       // bf16 elements a row of P
constexpr int kSPitch = kN + 1;       // floats a row of S

struct GeneralParams {
    DenseShape s;
    DenseCache c;
    const __nv_bfloat16* q;
    int d_qk, d_v;
    float scale_log2;                 // softmax_scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    DensePartials part;
    int32_t* status;
};

struct GeneralSmem {
    int k, p, sc, stat, scratch, total;
};
__host__ __device__ inline GeneralSmem general_smem(int d_qk)
{
    GeneralSmem m;
    const int pitch = (d_qk + 8) * 2;
    m.k = kM * pitch;                                  // Q comes first
    m.p = m.k + kN * pitch;
    m.sc = m.p + 2 * kM * kPPitch * 2;                 // S, fp32
    m.stat = m.sc + kM * kSPitch * 4;                  // per-row factors, per-token scales and flags
    m.scratch = m.stat + (kM + 3 * kN) * 4;
    m.scratch = (m.scratch + 15) / 16 * 16;
    m.total = m.scratch + 40 * 8 + kThreads * 4 + 2 * static_cast<int>(sizeof(DenseCut));
    return m;
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 e4m3 codes -> 8 bf16 (exact).
__device__ __forceinline__ uint4 e4m3x8_to_bf16x8(uint2 v)
{
    const uint32_t w[2] = {v.x, v.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t pair = static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Any of the 8 bf16 values infinite or NaN (all exponent bits set).
__device__ __forceinline__ bool nonfinite8(const uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
    return bad;
}

// kNT: n8 tiles of O columns per warp; kPre: 8-element chunks of a row that a thread
// fetches a block ahead (0: rows too long for the registers)
template <bool kFp8, int kNT, int kPre>
__global__ void __launch_bounds__(kThreads, 1) mla_dense_general_kernel(const GeneralParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const GeneralSmem lay = general_smem(p.d_qk);
    const int pitch = p.d_qk + 8;                                    // bf16 elements
    __nv_bfloat16* sQ = reinterpret_cast<__nv_bfloat16*>(smem);
    uint8_t* sK = smem + lay.k;
    __nv_bfloat16* sP = reinterpret_cast<__nv_bfloat16*>(smem + lay.p);
    float* sS = reinterpret_cast<float*>(smem + lay.sc);
    float* sFac = reinterpret_cast<float*>(smem + lay.stat);         // [kM]
    float* sScale = sFac + kM;                                       // [kN] token scale
    int* sValid = reinterpret_cast<int*>(sScale + kN);               // [kN] the token's page exists
    int* sBad = sValid + kN;                                         // [kN] infinities or NaN in its row
    DenseCut* sCut = reinterpret_cast<DenseCut*>(smem + lay.scratch + 40 * 8 + kThreads * 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DenseShape& s = p.s;
    pdl_wait();
    pdl_launch_dependents();                                         // the joining kernel may be set up meanwhile
    if (p.part.slots && tid < 2)
        p.part.slots[2 * blockIdx.x + tid] = DenseSlot{0, 0, 0, 0};
    dense_divide<kM, kN, kTileCost, kMinBlocks, kThreads>(s, kN, blockIdx.x, gridDim.x,
                                              reinterpret_cast<long long*>(smem + lay.scratch), sCut);
    DensePieces<kM, kN> pieces(s, kN, blockIdx.x, sCut);
    DensePiece pc;
    const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aP = smem_u32(sP);
    const int wr = (warp & 3) * 16, wk = (warp >> 2) * 16;           // this warp's rows and keys of S
    const int srow = tid >> 2, squad = tid & 3;                      // softmax: four threads a row, 8 keys each
    const int col0 = warp * kNT * 8;                                 // this warp's O columns

    while (pieces.next(&pc)) {
        const DenseTile& t = pc.t;
        if (t.over && tid == 0 && p.status)
            atomicOr(p.status, DSA_DEV_BAD_INDEX);
        __syncthreads();
        // Q rows (zeros past the tile)
        const int per_row = p.d_qk / 8;
        for (int e = tid; e < kM * per_row; e += kThreads) {
            const int r = e / per_row, c = e % per_row;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < t.nrows)
                v = *reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(t.row0) + r) * p.d_qk + c * 8);
            *reinterpret_cast<uint4*>(sQ + r * pitch + c * 8) = v;
        }
        const bool row_ok = srow < t.nrows;
        const DenseKeys keys = row_ok ? dense_keys(s, t.L, t.n, (t.m0 + srow) / s.num_heads) : DenseKeys{0, 0, 0};
        float o[4][kNT][4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < kNT; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[a][b][i] = 0.f;
        float m_run = -INFINITY, l_run = 0.f;

        // The row of a block's token (tid / 8), its scale and, for short rows, this thread's
        // chunks of it, fetched while the block before is worked on.
        const int tok = tid >> 3, part = tid & 7;
        const uint8_t* src = nullptr;
        float scale = 0.f;
        uint4 pre[kPre > 0 ? kPre : 1];
        auto load = [&](const uint8_t* row, int c) -> uint4 {
            if (!kFp8)
                return *reinterpret_cast<const uint4*>(row + c * 16);
            const uint2 v = *reinterpret_cast<const uint2*>(row + c * 8);
            return make_uint4(v.x, v.y, 0, 0);
        };
        auto fetch = [&](int j) {
            src = nullptr;
            scale = 0.f;
            if (j >= pc.blk1)
                return;
            const int pos = dense_unit_pos(t, kN, j) + tok;
            if (pos < t.last.hi && (pos >= t.first.lo || pos < t.last.sink)) {
                const int page = p.c.bt[static_cast<int64_t>(t.seq) * p.c.bt_stride + pos / p.c.page_kv];
                if (page >= 0 && page < p.c.num_pages) {
                    src = p.c.vals + page * p.c.vps + (pos % p.c.page_kv) * p.c.vts;
                    scale = kFp8 ? *reinterpret_cast<const float*>(p.c.scs + page * p.c.sps + (pos % p.c.page_kv) * p.c.sts)
                                 : 1.f;
                } else if (part == 0 && p.status) {
                    atomicOr(p.status, DSA_DEV_BAD_INDEX);
                }
            }
#pragma unroll
            for (int e = 0; e < kPre; ++e)
                pre[e] = src && part + 8 * e < per_row ? load(src, part + 8 * e) : make_uint4(0, 0, 0, 0);
        };
        fetch(pc.blk0);

        for (int j = pc.blk0; j < pc.blk1; ++j) {
            __syncthreads();                                         // the block before is used up
            const int base = dense_unit_pos(t, kN, j);
            // keys of the block that some row sees, and that every row sees
            bool bad = false;
            {
                const int pos = base + tok;
                const bool every = pos < t.first.hi && (pos >= t.last.lo || pos < t.first.sink);
                auto put = [&](int c, uint4 v) {
                    if (kFp8)
                        v = e4m3x8_to_bf16x8(make_uint2(v.x, v.y));
                    if (src && !every)
                        bad |= nonfinite8(v);
                    *reinterpret_cast<uint4*>(sK + (tok * pitch + c * 8) * 2) = v;
                };
                if (kPre > 0) {
#pragma unroll
                    for (int e = 0; e < kPre; ++e)
                        if (part + 8 * e < per_row)
                            put(part + 8 * e, pre[e]);
                } else {
                    for (int c = part; c < per_row; c += 8)
                        put(c, src ? load(src, c) : make_uint4(0, 0, 0, 0));
                }
                bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 24) & 0xFFu) != 0;   // the token's 8 lanes
                if (part == 0) {
                    sScale[tok] = scale;
                    sValid[tok] = src != nullptr;
                    sBad[tok] = bad;
                }
                fetch(j + 1);                                    // flies while this block is worked on
            }
            const int any_bad = __syncthreads_or(bad);
            // ---- S = Q K^T
            {
                float sacc[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sacc[b][i] = 0.f;
                const uint32_t qa = aQ + ((wr + (lane & 15)) * pitch + (lane >> 4) * 8) * 2;
                // B fragments of two n8 tiles: keys wk + 0-7 and 8-15, both halves of k
                const uint32_t ka = aK + ((wk + (lane & 7) + ((lane >> 4) << 3)) * pitch + ((lane >> 3) & 1) * 8) * 2;
                for (int k = 0; k < p.d_qk; k += 16) {
                    uint32_t a[4], b[4];
                    ldsm_x4(a, qa + k * 2);
                    ldsm_x4(b, ka + k * 2);
                    mma_bf16(sacc[0], a, b[0], b[1]);
                    mma_bf16(sacc[1], a, b[2], b[3]);
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sS[(wr + (lane >> 2) + (i >> 1) * 8) * kSPitch + wk + b * 8 + (lane & 3) * 2 + (i & 1)] = sacc[b][i];
            }
            __syncthreads();
            // ---- softmax: thread (row, quad) has keys quad * 8 .. + 7
            {
                uint32_t see = dense_mask32(keys, base) >> (squad * 8);
                float x[8], mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int kk = squad * 8 + c;
                    const bool on = (see >> c & 1u) && sValid[kk];
                    see &= on ? 0xFFFFFFFFu : ~(1u << c);
                    x[c] = on ? sS[srow * kSPitch + kk] * (p.scale_log2 * (kFp8 ? sScale[kk] : 1.f)) : -INFINITY;
                    mx = fmaxf(mx, x[c]);
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m_run, mx);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float f = m_run == -INFINITY ? 1.f : ex2_approx(m_run - m_use);
                m_run = m_new;
                float sum = 0.f;
                uint32_t pk[4], pl[4];
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    float pv[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float pr = ex2_approx(x[c + e] - m_use);          // a key not seen: 2^-inf = 0
                        sum += pr;
                        // (0 times a seen token's infinite scale is NaN, an unseen token's scale is no matter)
                        pv[e] = see >> (c + e) & 1u ? pr * (kFp8 ? sScale[squad * 8 + c + e] : 1.f) : 0.f;
                    }
                    const __nv_bfloat162 b = __floats2bfloat162_rn(pv[0], pv[1]);
                    const __nv_bfloat162 d = __floats2bfloat162_rn(pv[0] - __low2float(b), pv[1] - __high2float(b));
                    pk[c >> 1] = *reinterpret_cast<const uint32_t*>(&b);
                    pl[c >> 1] = *reinterpret_cast<const uint32_t*>(&d);
                }
                l_run = l_run * f + sum;
                *reinterpret_cast<uint4*>(sP + srow * kPPitch + squad * 8) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                *reinterpret_cast<uint4*>(sP + (kM + srow) * kPPitch + squad * 8) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                if (squad == 0)
                    sFac[srow] = f;
            }
            // a row that not every query row sees may hold infinities or NaN: as
            // values they become zeros (0 x NaN is NaN); who sees a NaN has it in P, and
            // who sees an infinity, with P = 0 where its score is -inf, gets the NaN here
            if (any_bad) {
                for (int kk = 0; kk < kN; ++kk) {
                    if (!sBad[kk])
                        continue;
#pragma unroll
                    for (int a = 0; a < 8; ++a) {
                        const int r = (a >> 1) * 16 + (a & 1) * 8 + (lane >> 2);
                        if (r >= t.nrows || !(dense_mask32(dense_keys(s, t.L, t.n, (t.m0 + r) / s.num_heads), base) >> kk & 1u))
                            continue;
#pragma unroll
                        for (int b = 0; b < kNT; ++b) {
                            const int c = col0 + b * 8 + (lane & 3) * 2;
                            if (c >= p.d_v)
                                continue;
                            const uint32_t v = *reinterpret_cast<const uint32_t*>(sK + (kk * pitch + c) * 2);
                            if ((v & 0x7F80u) == 0x7F80u)
                                o[a >> 1][b][2 * (a & 1)] = __int_as_float(0x7FC00000);
                            if ((v & 0x7F800000u) == 0x7F800000u)
                                o[a >> 1][b][2 * (a & 1) + 1] = __int_as_float(0x7FC00000);
                        }
                    }
                }
                __syncthreads();
                for (int e = tid; e < kN * per_row; e += kThreads)
                    if (sBad[e / per_row])
                        *reinterpret_cast<uint4*>(sK + (e / per_row * pitch + e % per_row * 8) * 2) = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
            // ---- O = O f + P V
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const float f0 = sFac[a * 16 + (lane >> 2)], f1 = sFac[a * 16 + 8 + (lane >> 2)];
                if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
                    for (int b = 0; b < kNT; ++b) {
                        o[a][b][0] *= f0;
                        o[a][b][1] *= f0;
                        o[a][b][2] *= f1;
                        o[a][b][3] *= f1;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2 * (kN / 16); ++e) {                  // both parts of P
                const int k = (e >> 1) * 16;
                uint32_t a[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ldsm_x4(a[i], aP + (((e & 1) * kM + i * 16 + (lane & 15)) * kPPitch + k + (lane >> 4) * 8) * 2);
#pragma unroll
                for (int b = 0; b < kNT; b += 2) {
                    if (col0 + b * 8 >= p.d_v)                          // whole warp: d_v is a multiple of 16
                        continue;
                    uint32_t v[4];
                    ldsm_x4_trans(v, aK + ((k + (lane & 15)) * pitch + col0 + b * 8 + (lane >> 4) * 8) * 2);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mma_bf16(o[i][b], a[i], v[0], v[1]);
                        mma_bf16(o[i][b + 1], a[i], v[2], v[3]);
                    }
                }
            }
        }
        // ---- the tile's rows, or this worker's part of them
        __syncthreads();                                             // every warp has read the last block's factors
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
        const bool some = l_run > 0.f || l_run != l_run;               // NaN stays NaN
        const float lse = some ? (m_run == -INFINITY ? l_run : (m_run + log2f(l_run)) * 0.69314718055994531f) : -INFINITY;
        if (squad == 0) {
            sFac[srow] = some ? 1.f / l_run : 0.f;
            if (row_ok) {
                if (pc.slot < 0)
                    p.lse[static_cast<int64_t>(t.row0) + srow] = lse;
                else
                    p.part.lse[static_cast<int64_t>(pc.slot) * p.part.slot_rows + srow] = lse;
            }
        }
        if (tid == 0 && pc.slot >= 0)
            p.part.slots[pc.slot] = DenseSlot{t.row0, t.nrows, 1 | (pc.blk0 == 0 ? 2 : 0) | (pc.blk1 == t.nblk ? 4 : 0), 0};
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = a * 16 + hh * 8 + (lane >> 2);
                if (r >= t.nrows)
                    continue;
                const float inv = sFac[r];
#pragma unroll
                for (int b = 0; b < kNT; ++b) {
                    const int c = col0 + b * 8 + (lane & 3) * 2;
                    if (c >= p.d_v)
                        continue;
                    const float x = o[a][b][2 * hh] * inv, y = o[a][b][2 * hh + 1] * inv;
                    if (pc.slot < 0) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                        *reinterpret_cast<__nv_bfloat162*>(p.out + (static_cast<int64_t>(t.row0) + r) * p.d_v + c) = v;
                    } else {
                        *reinterpret_cast<float2*>(p.part.o + (static_cast<int64_t>(pc.slot) * p.part.slot_rows + r) * p.d_v + c) =
                            make_float2(x, y);
                    }
                }
            }
    }
}

// Joins the parts of cut tiles: out = sum_i w_i O_i / sum_i w_i with w_i =
// exp(lse_i - max), lse = max + ln sum_i w_i, in a fixed order (no atomics).  Every CTA
// reads the slots' records and lists the cut tiles' rows, in groups: eight rows of a
// tile of up to kFewParts parts, a warp each, or one row of a tile of more, every
// eighth part of it a warp's, whose sums are added in order.  Group k
// belongs to CTA k mod grid.  What it costs is its chain of loads (records; lse and O
// together), so the parts of a row are in flight at once.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFewParts = 8;
constexpr int kChunks = kDenseMaxWorkers / 32;           // parts of a row, 32 at a time
__global__ void __launch_bounds__(kJoinThreads) mla_dense_join_kernel(const DensePartials part, int workers,
                                                                      __nv_bfloat16* out, float* lse)
{
    __shared__ int s_flags[2 * kDenseMaxWorkers], s_row0[2 * kDenseMaxWorkers], s_nrows[2 * kDenseMaxWorkers];
    __shared__ int s_before[kDenseMaxWorkers + 1];       // groups of the tiles that workers before this one begin
    __shared__ int s_nparts[kDenseMaxWorkers];
    __shared__ uint32_t s_used[kChunks], s_ends[kChunks];    // bit per worker: its first slot is used / ends a tile
    __shared__ float4 s_acc[kJoinWarps][128];            // d_v <= 512
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    for (int i = threadIdx.x; i < 2 * workers; i += kJoinThreads) {
        const DenseSlot r = part.slots[i];
        s_flags[i] = r.flags;
        s_row0[i] = r.row0;
        s_nrows[i] = r.nrows;
    }
    __syncthreads();
    // the slot in which worker g begins a tile that it does not end, or -1
    auto begin_slot = [&](int g) -> int {
        return (s_flags[2 * g] & 7) == 3 ? 2 * g : (s_flags[2 * g + 1] & 7) == 3 ? 2 * g + 1 : -1;
    };
    if (warp < kChunks) {
        const int g = warp * 32 + lane;
        const int f = g < workers ? s_flags[2 * g] : 0;
        const uint32_t used = __ballot_sync(0xffffffffu, f & 1), ends = __ballot_sync(0xffffffffu, f & 4);
        if (lane == 0) {
            s_used[warp] = used;
            s_ends[warp] = ends;
        }
    }
    __syncthreads();
    // bits of the workers of chunk c that have a part of the tile that worker g begins: the
    // used first slots after g, up to the first that ends a tile (a worker between may have
    // got no piece)
    auto parts_of = [&](int g, int c, bool* open) -> uint32_t {
        const int from = g + 1 - 32 * c;                 // the first bit of this chunk
        const uint32_t after = !*open || from >= 32 ? 0u : from <= 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << from;
        const uint32_t e = s_ends[c] & after;
        if (e)
            *open = false;
        return s_used[c] & after & (e ? (e ^ (e - 1u)) : 0xFFFFFFFFu);
    };
    for (int g = threadIdx.x; g < workers; g += kJoinThreads) {
        const int slot = begin_slot(g);
        int n = 0, groups = 0;
        if (slot >= 0) {
            bool open = true;
            n = 1;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                n += __popc(parts_of(g, c, &open));
            groups = n <= kFewParts ? (s_nrows[slot] + kJoinWarps - 1) / kJoinWarps : s_nrows[slot];
        }
        s_nparts[g] = n;
        s_before[g + 1] = groups;
    }
    __syncthreads();
    if (threadIdx.x < 32) {                              // prefix sum, 32 workers at a time
        int base = 0;
        for (int g0 = 0; g0 < workers; g0 += 32) {
            const int g = g0 + lane;
            int x = g < workers ? s_before[g + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o)
                    x += y;
            }
            if (g < workers)
                s_before[g + 1] = base + x;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0)
            s_before[0] = 0;
    }
    __syncthreads();
    const int groups = s_before[workers];
    auto add = [](float4& a, float w, const float4& v) {
        a.x = fmaf(w, v.x, a.x);
        a.y = fmaf(w, v.y, a.y);
        a.z = fmaf(w, v.z, a.z);
        a.w = fmaf(w, v.w, a.w);
    };
    auto store = [&](int64_t row, int col, const float4& v) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(out + row * part.d_v + col) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    };
    for (int k = blockIdx.x; k < groups; k += gridDim.x) {
        int lo = 0, hi = workers - 1;                    // the last worker with s_before <= k
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_before[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int slot = begin_slot(lo), nparts = s_nparts[lo];
        if (nparts <= kFewParts) {
            const int r = (k - s_before[lo]) * kJoinWarps + warp;
            if (r >= s_nrows[slot])
                continue;
            int mine = slot;                             // lane i: the slot of part i
            for (int h = lo + 1, i = 1; i < nparts; ++h)
                if (s_flags[2 * h] & 1) {
                    mine = lane == i ? 2 * h : mine;
                    ++i;
                }
            const float z = lane < nparts ? part.lse[static_cast<int64_t>(mine) * part.slot_rows + r] : -INFINITY;
            float4 first[2][4];                          // the first two parts' O fly with the lse
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float* src = part.o + (static_cast<int64_t>(__shfl_sync(0xffffffffu, mine, i)) * part.slot_rows + r) * part.d_v;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    first[i][c] = c * 128 + lane * 4 < part.d_v ? *reinterpret_cast<const float4*>(src + c * 128 + lane * 4)
                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mx = z;
#pragma unroll
            for (int o = kFewParts / 2; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = __shfl_sync(0xffffffffu, mx, 0);
            const float use = mx == -INFINITY ? 0.f : mx;
            const float w = lane < nparts ? expf(z - use) : 0.f;
            float total = w;
#pragma unroll
            for (int o = kFewParts / 2; o > 0; o >>= 1)
                total += __shfl_xor_sync(0xffffffffu, total, o);
            total = __shfl_sync(0xffffffffu, total, 0);
            const bool some = total > 0.f || total != total;           // NaN stays NaN
            const float inv = some ? 1.f / total : 0.f;
            float4 acc[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i) * inv;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    add(acc[c], wi, first[i][c]);
            }
            for (int i = 2; i < nparts; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i) * inv;
                const float* src = part.o + (static_cast<int64_t>(__shfl_sync(0xffffffffu, mine, i)) * part.slot_rows + r) * part.d_v;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c * 128 + lane * 4 < part.d_v)
                        add(acc[c], wi, *reinterpret_cast<const float4*>(src + c * 128 + lane * 4));
            }
            const int64_t row = static_cast<int64_t>(s_row0[slot]) + r;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c * 128 + lane * 4 < part.d_v)
                    store(row, c * 128 + lane * 4, acc[c]);
            if (lane == 0)
                lse[row] = some ? mx + logf(total) : -INFINITY;
            continue;
        }
        // part 0 is the slot in which the tile begins; part (c, bit) worker 32 c + bit's first slot.
        // Lane l of every warp weighs the parts (c, l), warp w sums the parts (c, w + 8 q).
        const int r = k - s_before[lo];
        uint32_t bits[kChunks];
        float z[kChunks], mx;
        const float z0 = part.lse[static_cast<int64_t>(slot) * part.slot_rows + r];
        mx = z0;
        bool open = true;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            bits[c] = parts_of(lo, c, &open);
            z[c] = bits[c] >> lane & 1u ? part.lse[static_cast<int64_t>(2 * (32 * c + lane)) * part.slot_rows + r] : -INFINITY;
        }
        float4 acc[4];
        const float* src0 = part.o + (static_cast<int64_t>(slot) * part.slot_rows + r) * part.d_v;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[c] = warp == 0 && c * 128 + lane * 4 < part.d_v ? *reinterpret_cast<const float4*>(src0 + c * 128 + lane * 4)
                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            mx = fmaxf(mx, z[c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float use = mx == -INFINITY ? 0.f : mx;
        float total = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            z[c] = bits[c] >> lane & 1u ? expf(z[c] - use) : 0.f;      // the weights
            total += z[c];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            total += __shfl_xor_sync(0xffffffffu, total, o);
        const float w0 = expf(z0 - use);
        total += w0;
        const bool some = total > 0.f || total != total;
        const float inv = some ? 1.f / total : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 v = acc[c];
            acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            add(acc[c], w0 * inv, v);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float4 v[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int bit = warp + 8 * q;
                const float* src = part.o + (static_cast<int64_t>(2 * (32 * c + bit)) * part.slot_rows + r) * part.d_v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[q][e] = (bits[c] >> bit & 1u) && e * 128 + lane * 4 < part.d_v
                                  ? *reinterpret_cast<const float4*>(src + e * 128 + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float w = __shfl_sync(0xffffffffu, z[c], warp + 8 * q) * inv;
                if (bits[c] >> (warp + 8 * q) & 1u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        add(acc[e], w, v[q][e]);
            }
        }
        __syncthreads();                                 // the row before has been written
#pragma unroll
        for (int c = 0; c < 4; ++c)
            s_acc[warp][c * 32 + lane] = acc[c];
        __syncthreads();
        const int64_t row = static_cast<int64_t>(s_row0[slot]) + r;
        if (threadIdx.x < 128 && threadIdx.x * 4 < part.d_v) {
            float4 t = s_acc[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w)
                add(t, 1.f, s_acc[w][threadIdx.x]);
            store(row, threadIdx.x * 4, t);
        }
        if (threadIdx.x == 0)
            lse[row] = some ? mx + logf(total) : -INFINITY;
    }
}

template <class... T>
cudaError_t launch_pdl(void (*kern)(T...), dim3 grid, int threads, int smem, cudaStream_t stream, T... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool kFp8>
void (*general_kernel(int d_qk, int d_v))(GeneralParams)
{
    if (d_v <= 128)
        return d_qk <= 128 ? mla_dense_general_kernel<kFp8, 2, 2> : mla_dense_general_kernel<kFp8, 2, 0>;
    return d_v <= 256 ? mla_dense_general_kernel<kFp8, 4, 0> : mla_dense_general_kernel<kFp8, 8, 0>;
}

}  // namespace

DenseShape dense_shape(const DenseArgs& a)
{
    DenseShape s;
    s.rows = a.rows;
    s.num_heads = a.num_heads;
    s.batch = a.batch;
    s.next_n = a.next_n;
    s.window = a.window;
    s.sinks = a.sinks;
    s.cap = a.kv->max_pages_per_seq * a.kv->page_kv;
    s.seq_lens = a.seq_lens;
    s.cum_q = a.cum_q;
    return s;
}

DenseCache dense_cache(const dsa_paged_cache* c)
{
    DenseCache d{};
    d.vals = static_cast<const uint8_t*>(c->values);
    d.vps = c->val_page_stride;
    d.vts = c->val_token_stride;
    d.scs = c->fmt == DSA_KV_FP8_E4M3 ? static_cast<const uint8_t*>(c->scales) : nullptr;
    d.sps = c->sc_page_stride;
    d.sts = c->sc_token_stride;
    d.bt = c->block_table;
    d.bt_stride = c->bt_row_stride;
    d.page_kv = c->page_kv;
    d.num_pages = c->num_pages;
    return d;
}

// The workspace: slots' O, then their lse, then their records.  The slots hold
// kDenseMaxWorkers x 2 x 64 rows however the kernel divides them (64-row tiles by
// one CTA, or 128-row tiles by a CTA pair), or fewer where the call has fewer rows.
int64_t dense_slot_rows(int rows, int num_heads, int tile_rows)
{
    const int64_t all = static_cast<int64_t>(rows) * num_heads;
    return all < tile_rows ? all : tile_rows;
}

size_t dense_workspace_bytes(int rows, int num_heads, int d_v)
{
    const int64_t a = dense_slot_rows(rows, num_heads, 64) * 2 * kDenseMaxWorkers;
    const int64_t b = dense_slot_rows(rows, num_heads, 128) * 2 * (kDenseMaxWorkers / 2);
    const int64_t n = a > b ? a : b;
    return static_cast<size_t>(n * 4 * (d_v + 1) + 2 * kDenseMaxWorkers * static_cast<int64_t>(sizeof(DenseSlot)) + 32);
}

DensePartials dense_partials(const DenseArgs& a, int workers, int tile_rows)
{
    DensePartials p;
    p.slot_rows = static_cast<int>(dense_slot_rows(a.rows, a.num_heads, tile_rows));
    p.d_v = a.d_v;
    const int64_t n = static_cast<int64_t>(2) * workers * p.slot_rows;
    p.o = static_cast<float*>(a.workspace);
    p.lse = p.o + n * a.d_v;
    p.slots = reinterpret_cast<DenseSlot*>(reinterpret_cast<uintptr_t>(p.lse + n + 3) & ~uintptr_t(15));
    return p;
}

// Whether any tile of the call can be cut: a window bounds a tile's blocks.
bool dense_may_cut(const DenseArgs& a, int tile_rows, int block_keys, int unit, int min_blocks)
{
    const int64_t cap = static_cast<int64_t>(a.kv->max_pages_per_seq) * a.kv->page_kv;
    int64_t keys = cap;
    if (a.window >= 0) {
        // the tile's tokens, their window and the sinks, each range with a unit at either end
        const int64_t tokens = (tile_rows + a.num_heads - 1) / a.num_heads + 1;
        const int64_t w = static_cast<int64_t>(a.window) + tokens + 2 * unit;
        const int64_t k = static_cast<int64_t>(a.sinks) + unit;
        keys = w + k < cap ? w + k : cap;
    }
    return (keys + block_keys - 1) / block_keys + 1 >= 2 * min_blocks;
}

dsa_status launch_dense_join(const DensePartials& part, int workers, const DenseArgs& a, const DeviceInfo& dev,
                             cudaStream_t stream)
{
    // a CTA a group of rows (eight, or one of many parts), as many as run at once and no more than
    // the call has rows
    const int64_t rows = static_cast<int64_t>(a.rows) * a.num_heads;
    const int64_t most = static_cast<int64_t>(dev.sm_count) * 4;
    const cudaError_t e = launch_pdl(mla_dense_join_kernel, dim3(static_cast<unsigned>(rows < most ? rows : most)),
                                     kJoinThreads, 0, stream, part, workers, static_cast<__nv_bfloat16*>(a.out), a.lse);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

dsa_status launch_mla_dense_general(const DenseArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    GeneralParams p;
    p.s = dense_shape(a);
    p.c = dense_cache(a.kv);
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.d_qk = a.d_qk;
    p.d_v = a.d_v;
    p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.status = a.status;
    const bool fp8 = a.kv->fmt == DSA_KV_FP8_E4M3;
    const int smem = general_smem(a.d_qk).total;
    if (smem > dev.max_smem_optin)
        return DSA_ERR_UNSUPPORTED;
    const int workers = dev.sm_count < kDenseMaxWorkers ? dev.sm_count : kDenseMaxWorkers;
    p.part = dense_partials(a, workers, kM);
    auto kern = fp8 ? general_kernel<true>(a.d_qk, a.d_v) : general_kernel<false>(a.d_qk, a.d_v);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = launch_pdl(kern, dim3(workers), kThreads, smem, stream, p);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const dsa_status st = check_launch();
    if (st != DSA_OK || !dense_may_cut(a, kM, kN, kN, kMinBlocks))
        return st;
    return launch_dense_join(p.part, workers, a, dev, stream);
}

}  // namespace dsa
