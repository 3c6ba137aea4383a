// gather.cu -- read ranges of a paged cache back as dense rows, the inverse of the
// quantise / scatter: row cum_rows[b] + i of the output is
//   decode(cache[b][starts[b] + i]) * scale
// from FP8 (e4m3 codes, an fp32 scale a token), MXFP4 (e2m1 codes, a ue8m0 scale
// per 32 elements) or bf16 pages to fp32 or bf16 rows.  The product is formed in
// fp32 and rounded once, so an fp32 output is exact for MXFP4 and within half a
// step for FP8.
//
// HBM-bound: a row of D elements is read once (D + 4, D / 2 + D / 32 or 2 D bytes)
// and written once.  A CTA owns a run of output rows: one thread a row finds its
// sequence, its place in the cache and its scale, then the rows' elements are moved in
// chunks of 16 output bytes (8 bf16 or 4 fp32), eight chunks a thread at a time, all loads
// before the first store.  A row's chunks belong to consecutive lanes, so a warp's loads and
// its stores are contiguous whatever the formats: 1.07 M rows of 576 e4m3 to bf16 take 281 us,
// 0.81 M rows of 64 e2m1 to fp32 49 us (an earlier form with 16-byte loads, and so stores 32 or
// 128 bytes apart, 322 and 111).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "host.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

struct GatherParams {
    const uint8_t* vals;
    int64_t vps, vts;
    const uint8_t* scs;
    int64_t sps, sts;
    const int32_t* bt;
    int64_t bt_stride;
    int max_pages, page_kv, num_pages, D;
    const int32_t* cum;
    const int32_t* starts;
    int batch;
    void* out;
    int64_t out_stride;
    int out_rows;
    int rows_per_cta;
    uint32_t recip;              // 2^32 / chunks of a row, rounded up
    int32_t* status;
};

// `n` elements (8 or 4) of a chunk's raw bytes -> fp32.
template <int kFmt, int n>
__device__ __forceinline__ void decode_chunk(const uint32_t (&w)[4], float (&f)[n])
{
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        float2 v;
        if constexpr (kFmt == DSA_KV_FP8_E4M3) {
            const __nv_fp8x2_storage_t pair = static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
            v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3)));
        } else if constexpr (kFmt == DSA_KV_MXFP4) {
            // e2m1: 0 and 0.5 (codes 0, 1), else (1 + m / 2) 2^(e - 1): the code's three
            // low bits moved to an fp32's exponent and top mantissa bit, times 2^126
            const uint32_t b = w[0] >> (8 * i);
            const uint32_t lo = ((b & 7u) << 22) | ((b & 8u) << 28), hi = ((b & 0x70u) << 18) | ((b & 0x80u) << 24);
            constexpr float up = 8.507059173023462e37f;      // 2^126
            v = make_float2(__uint_as_float(lo) * up, __uint_as_float(hi) * up);
        } else {
            v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

// `bytes` (2, 4, 8 or 16) from an address aligned to them; read once, so not kept.
template <int bytes>
__device__ __forceinline__ void load_raw(const uint8_t* src, uint32_t (&w)[4])
{
    if constexpr (bytes == 2) {
        w[0] = __ldcs(reinterpret_cast<const unsigned short*>(src));
    } else if constexpr (bytes == 4) {
        w[0] = __ldcs(reinterpret_cast<const unsigned int*>(src));
    } else if constexpr (bytes == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

constexpr int kMaxRows = 256;        // rows a CTA
constexpr int kInFlight = 8;

template <int kFmt, bool kBf16>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const GatherParams p)
{
    constexpr int kE = kBf16 ? 8 : 4;                    // elements a chunk
    constexpr int kBytes = kFmt == DSA_KV_FP8_E4M3 ? kE : kFmt == DSA_KV_MXFP4 ? kE / 2 : 2 * kE;
    __shared__ const uint8_t* s_src[kMaxRows];           // null: a row of zeros
    __shared__ const uint8_t* s_sc[kMaxRows];            // MXFP4: the row's block scales
    __shared__ float s_scale[kMaxRows];                  // FP8: the token's scale
    __shared__ bool s_on[kMaxRows];                      // the row belongs to a range
    const int chunks = p.D / kE;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
    const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.out_rows - row0));
    if (threadIdx.x < rows) {
        const int r = static_cast<int>(row0) + threadIdx.x;
        // the sequence of output row r: the last b with cum[b] <= r, if r < cum[b + 1]
        int lo = 0, hi = p.batch;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cum[mid] <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        const bool on = lo < p.batch && p.cum[lo] <= r;
        const uint8_t* src = nullptr;
        s_scale[threadIdx.x] = 1.f;
        if (on) {
            const int64_t pos = (p.starts ? p.starts[lo] : 0) + static_cast<int64_t>(r) - p.cum[lo];
            const int64_t lp = pos >= 0 ? pos / p.page_kv : p.max_pages;
            const int page = lp < p.max_pages ? p.bt[lo * p.bt_stride + lp] : -1;
            if (page >= 0 && page < p.num_pages) {
                const int64_t row = pos - lp * p.page_kv;
                src = p.vals + page * p.vps + row * p.vts;
                const uint8_t* sc = p.scs + page * p.sps + row * p.sts;
                if constexpr (kFmt == DSA_KV_FP8_E4M3)
                    s_scale[threadIdx.x] = *reinterpret_cast<const float*>(sc);
                if constexpr (kFmt == DSA_KV_MXFP4)
                    s_sc[threadIdx.x] = sc;
            } else if (p.status) {
                atomicOr(p.status, DSA_DEV_BAD_PAGE);     // its row becomes zeros
            }
        }
        s_src[threadIdx.x] = src;
        s_on[threadIdx.x] = on;
    }
    __syncthreads();
    const int items = rows * chunks;                      // < 2^18
    for (int i0 = threadIdx.x; i0 < items; i0 += kThreads * kInFlight) {
        uint32_t w[kInFlight][4], ex[kInFlight];
        int rr[kInFlight], cc[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int it = i0 + k * kThreads;
            // it / chunks: exact for it < 2^18 and a reciprocal rounded up to 2^-32
            rr[k] = chunks == 1 ? it : static_cast<int>(__umulhi(static_cast<uint32_t>(it), p.recip));
            cc[k] = it - rr[k] * chunks;
            w[k][0] = w[k][1] = w[k][2] = w[k][3] = 0;
            ex[k] = 127;
            const uint8_t* src = it < items ? s_src[rr[k]] : nullptr;
            if (src) {
                load_raw<kBytes>(src + cc[k] * kBytes, w[k]);
                if constexpr (kFmt == DSA_KV_MXFP4)
                    ex[k] = s_sc[rr[k]][cc[k] * kE / 32];
            }
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            if (i0 + k * kThreads >= items || !s_on[rr[k]])
                continue;                                 // outside every sequence: left as it was
            float scale = 1.f;
            if constexpr (kFmt == DSA_KV_FP8_E4M3)
                scale = s_scale[rr[k]];
            if constexpr (kFmt == DSA_KV_MXFP4)           // 2^(e - 127); 255 is NaN, 0 the subnormal 2^-127
                scale = __uint_as_float(ex[k] == 255u ? 0x7FC00000u : ex[k] == 0u ? 0x00400000u : ex[k] << 23);
            const int64_t at = (row0 + rr[k]) * p.out_stride + cc[k] * kE;
            if constexpr (kBf16 && kFmt == DSA_KV_BF16) {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
            } else {
                float f[kE];
                decode_chunk<kFmt, kE>(w[k], f);
                if constexpr (kFmt != DSA_KV_BF16)
#pragma unroll
                    for (int i = 0; i < kE; ++i)
                        f[i] *= scale;
                if constexpr (kBf16) {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                        o[i] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(f[0], f[1], f[2], f[3]);
                }
            }
        }
    }
}

}  // namespace

dsa_status launch_kv_gather(const GatherArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    const dsa_paged_cache* c = a.cache;
    GatherParams p;
    p.vals = static_cast<const uint8_t*>(c->values);
    p.vps = c->val_page_stride;
    p.vts = c->val_token_stride;
    p.scs = static_cast<const uint8_t*>(c->scales);
    p.sps = c->sc_page_stride;
    p.sts = c->sc_token_stride;
    p.bt = c->block_table;
    p.bt_stride = c->bt_row_stride;
    p.max_pages = c->max_pages_per_seq;
    p.page_kv = c->page_kv;
    p.num_pages = c->num_pages;
    p.D = c->head_dim;
    p.cum = a.cum_rows;
    p.starts = a.starts;
    p.batch = a.batch;
    p.out = a.out;
    p.out_stride = a.out_stride;
    p.out_rows = a.out_rows;
    p.status = a.status;
    const int chunk = a.bf16 ? 8 : 4;
    // rows a CTA: about two rounds of kInFlight chunks a thread, so that finding the rows is
    // spread over more of them (one round: 52 instead of 50 us for MXFP4, four: 289 instead of
    // 282 for FP8, in turn); fewer where the call would not fill the GPU
    const int chunks = c->head_dim / chunk;
    int per = 2 * kThreads * kInFlight / chunks;
    per = per < 1 ? 1 : per > kMaxRows ? kMaxRows : per;
    while (per > 8 && static_cast<int64_t>(a.out_rows) < static_cast<int64_t>(per) * dev.sm_count * 2)
        per = (per + 1) / 2;
    p.rows_per_cta = per;
    p.recip = static_cast<uint32_t>((0x100000000ull + chunks - 1) / chunks);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.out_rows) + per - 1) / per));
    if (c->fmt == DSA_KV_FP8_E4M3) {
        if (a.bf16)
            kv_gather_kernel<DSA_KV_FP8_E4M3, true><<<grid, kThreads, 0, stream>>>(p);
        else
            kv_gather_kernel<DSA_KV_FP8_E4M3, false><<<grid, kThreads, 0, stream>>>(p);
    } else if (c->fmt == DSA_KV_MXFP4) {
        if (a.bf16)
            kv_gather_kernel<DSA_KV_MXFP4, true><<<grid, kThreads, 0, stream>>>(p);
        else
            kv_gather_kernel<DSA_KV_MXFP4, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
        if (a.bf16)
            kv_gather_kernel<DSA_KV_BF16, true><<<grid, kThreads, 0, stream>>>(p);
        else
            kv_gather_kernel<DSA_KV_BF16, false><<<grid, kThreads, 0, stream>>>(p);
    }
    return check_launch();
}

}  // namespace dsa
