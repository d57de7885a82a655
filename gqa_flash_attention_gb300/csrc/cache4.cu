// sdp_cache4_append and sdp_cache4_gather: the 4-bit paged cache's writer, and its reader into
// 16-bit rows (cache4.cuh has the layout).
//
// Writing a group of 64 channels x_c:  b = bf16(min x),  s = bf16(max(0, (max x - b) / 15)),
// n_c = clamp(rint((x_c - b) / s), 0, 15), 0 where s = 0. The quotient is a true division: inputs
// of few bits often lie exactly on a border between two codes, where a product with 1 / s falls
// on either side.
//
// Both kernels are HBM-bound elementwise passes: a warp takes one token and runs over its 2 Hkv
// rows (K heads, then V heads), D/8 lanes a row, each lane one 16-byte access on the 16-bit side
// and one 4-byte word of eight codes on the other, so a row's codes are one 64- or 128-byte
// access. The token's sequence and page are looked up once a warp.
#include <cuda_runtime.h>

#include <cstdint>

#include "cache4.cuh"
#include "sdp.h"
#include "sixteen.cuh"

namespace {

using sdp::Cache4View;
using sdp::find_sequence;
using sdp::pack8;
using sdp::unpack8;

constexpr int kWarps = 4;
constexpr int kUnroll = 4;
constexpr unsigned FULL = 0xffffffffu;

struct RowsParams {
    Cache4View c;
    uint16_t *k, *v;                   // 16-bit rows: read by append, written by gather
    long long k_st, k_sh, v_st, v_sh;  // token and head strides in elements
    const int *cu, *lens;              // gather: lens is null, rows of a sequence are its tokens from 0
    unsigned int *status;
    int nseq, tokens;
    int rows_per_warp;
};

// A minimum / maximum that keeps NaN (fminf would drop it).
__device__ __forceinline__ float min_nan(float a, float b)
{
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Where a token lives: false (and a status code) for bad offsets or a page outside the pool.
__device__ __forceinline__ bool locate(const RowsParams &p, int token, int lane, long long *page, int *place)
{
    const int s = find_sequence(p.cu, p.nseq, token, lane);
    if (s >= p.nseq)
        return false;  // in no sequence: left as it is
    const int first = __ldg(p.cu + s), end = __ldg(p.cu + s + 1);
    bool ok = first >= 0 && end <= p.tokens;
    int pos = ok ? token - first : 0;
    if (ok && p.lens != nullptr) {
        const int before = __ldg(p.lens + s) - (end - first);  // tokens that were there already
        ok = before >= 0;
        pos = ok && pos <= INT32_MAX - before ? pos + before : INT32_MAX;
    }
    const int slot = ok ? pos / p.c.page_size : 0;
    if (!ok || slot >= p.c.max_pages) {
        if (lane == 0)
            atomicCAS(p.status, 0u, sdp::kBadSeqlens);
        return false;
    }
    const int id = __ldg(p.c.table + s * p.c.table_stride + slot);
    if (id < 0 || id >= p.c.num_pages) {
        if (lane == 0)
            atomicCAS(p.status, 0u, sdp::kBadPages);
        return false;
    }
    *page = id;
    *place = pos - slot * p.c.page_size;
    return true;
}

// Block 0 looks all offsets over: a token of a sequence with bad ones may belong to none.
__device__ __forceinline__ void check_offsets(const RowsParams &p)
{
    if (blockIdx.x != 0)
        return;
    for (int i = threadIdx.x; i < p.nseq; i += 32 * kWarps) {
        const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
        if (a < 0 || b < a || b > p.tokens)
            atomicCAS(p.status, 0u, sdp::kBadSeqlens);
    }
}

template <int D>
struct WarpItem {
    static constexpr int LPR = D / 8, RPP = 32 / LPR;
    int token, r0, r1;
    bool valid;
    __device__ __forceinline__ explicit WarpItem(const RowsParams &p)
    {
        const int rows = 2 * p.c.Hkv;
        const int runs = (rows + p.rows_per_warp - 1) / p.rows_per_warp;
        const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        valid = item < static_cast<long long>(p.tokens) * runs;
        token = static_cast<int>(item / runs);
        r0 = static_cast<int>(item - static_cast<long long>(token) * runs) * p.rows_per_warp;
        r1 = min(rows, r0 + p.rows_per_warp);
    }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kWarps) cache4_append_kernel(const RowsParams p)
{
    using W = WarpItem<D>;
    const int lane = threadIdx.x & 31;
    check_offsets(p);
    const W it(p);
    if (!it.valid)
        return;
    const int sub = lane / W::LPR, c0 = (lane % W::LPR) * 8;
    auto src = [&](int r) {
        return reinterpret_cast<const uint4 *>(r < p.c.Hkv ? p.k + it.token * p.k_st + r * p.k_sh + c0
                                                           : p.v + it.token * p.v_st + (r - p.c.Hkv) * p.v_sh + c0);
    };
    uint4 v[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int r = it.r0 + i * W::RPP + sub;
        if (r < it.r1)
            v[i] = __ldg(src(r));
    }
    long long page;
    int place;
    if (!locate(p, it.token, lane, &page, &place))
        return;
    for (int r0 = it.r0; r0 < it.r1; r0 += kUnroll * W::RPP) {
        if (r0 != it.r0) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int r = r0 + i * W::RPP + sub;
                if (r < it.r1)
                    v[i] = __ldg(src(r));
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (r0 + i * W::RPP >= it.r1)
                break;  // the same for the whole warp
            const int r = r0 + i * W::RPP + sub;
            const bool live = r < it.r1;
            float x[8];
            unpack8<BF16>(live ? v[i] : make_uint4(0u, 0u, 0u, 0u), x);
            float lo = x[0], hi = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) {
                lo = min_nan(lo, x[e]);
                hi = max_nan(hi, x[e]);
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) {  // eight lanes hold a group
                lo = min_nan(lo, __shfl_xor_sync(FULL, lo, off));
                hi = max_nan(hi, __shfl_xor_sync(FULL, hi, off));
            }
            const __nv_bfloat16 b16 = __float2bfloat16_rn(lo);
            const float b = __bfloat162float(b16);
            const __nv_bfloat16 s16 = __float2bfloat16_rn(max_nan(__fdiv_rn(__fsub_rn(hi, b), 15.f), 0.f));
            const float s = __bfloat162float(s16);
            uint32_t codes = 0;
            if (s != 0.f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[e], b), s)), 0.f), 15.f);
                    codes |= static_cast<uint32_t>(static_cast<int>(n)) << (4 * e);
                }
            }
            if (live) {
                const bool is_k = r < p.c.Hkv;
                const long long row = (page * p.c.Hkv + (is_k ? r : r - p.c.Hkv)) * p.c.page_size + place;
                uint8_t *out = is_k ? p.c.k_codes : p.c.v_codes;
                *reinterpret_cast<uint32_t *>(out + row * (D / 2) + c0 / 2) = codes;
                if (c0 % sdp::kCacheGroup == 0) {
                    uint32_t *sc = is_k ? p.c.k_scales : p.c.v_scales;
                    sc[row * (D / sdp::kCacheGroup) + c0 / sdp::kCacheGroup] =
                        static_cast<uint32_t>(__bfloat16_as_ushort(s16)) |
                        (static_cast<uint32_t>(__bfloat16_as_ushort(b16)) << 16);
                }
            }
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kWarps) cache4_gather_kernel(const RowsParams p)
{
    using W = WarpItem<D>;
    const int lane = threadIdx.x & 31;
    check_offsets(p);
    const W it(p);
    if (!it.valid)
        return;
    long long page;
    int place;
    if (!locate(p, it.token, lane, &page, &place))
        return;
    const int sub = lane / W::LPR, c0 = (lane % W::LPR) * 8;
    for (int r0 = it.r0; r0 < it.r1; r0 += kUnroll * W::RPP) {
        uint32_t codes[kUnroll], pair[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = r0 + i * W::RPP + sub;
            if (r < it.r1) {
                const bool is_k = r < p.c.Hkv;
                const long long row = (page * p.c.Hkv + (is_k ? r : r - p.c.Hkv)) * p.c.page_size + place;
                codes[i] = __ldg(reinterpret_cast<const uint32_t *>((is_k ? p.c.k_codes : p.c.v_codes) +
                                                                    row * (D / 2) + c0 / 2));
                pair[i] = __ldg((is_k ? p.c.k_scales : p.c.v_scales) + row * (D / sdp::kCacheGroup) +
                                c0 / sdp::kCacheGroup);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = r0 + i * W::RPP + sub;
            if (r < it.r1) {
                const float s = __uint_as_float(pair[i] << 16), b = __uint_as_float(pair[i] & 0xffff0000u);
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)  // s * code is exact in fp32 (8 + 4 bits): one rounding, then the store's
                    x[e] = fmaf(s, static_cast<float>((codes[i] >> (4 * e)) & 15u), b);
                uint16_t *out = r < p.c.Hkv ? p.k + it.token * p.k_st + r * p.k_sh + c0
                                            : p.v + it.token * p.v_st + (r - p.c.Hkv) * p.v_sh + c0;
                *reinterpret_cast<uint4 *>(out) = pack8<BF16>(x);
            }
        }
    }
}

// The checks that both calls share; fills p.
int rows_params(RowsParams &p, const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales,
                int num_pages, int page_size, const int *block_table, long long table_stride, int max_pages,
                const void *k, long long k_st, long long k_sh, const void *v, long long v_st, long long v_sh,
                const int *cu, const int *lens, bool with_lens, int nseq, int tokens, int Hkv, int D, int dtype)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (nseq <= 0 || tokens < 0 || Hkv <= 0 || num_pages <= 0 || max_pages <= 0 || page_size <= 0 ||
        page_size % 16 != 0 || table_stride < 0)
        return SDP_ERR_INVALID_ARG;
    if (tokens == 0)
        return SDP_OK;
    if (k_codes == nullptr || k_scales == nullptr || v_codes == nullptr || v_scales == nullptr ||
        block_table == nullptr || k == nullptr || v == nullptr || cu == nullptr || (with_lens && lens == nullptr))
        return SDP_ERR_INVALID_ARG;
    using sdp::is_aligned;
    if (!is_aligned(k_codes, 16) || !is_aligned(k_scales, 16) || !is_aligned(v_codes, 16) ||
        !is_aligned(v_scales, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(block_table, 4) ||
        !is_aligned(cu, 4) || !is_aligned(lens, 4) || k_st % 8 != 0 || k_sh % 8 != 0 || v_st % 8 != 0 || v_sh % 8 != 0)
        return SDP_ERR_ALIGNMENT;
    if (static_cast<long long>(max_pages) * page_size > INT32_MAX || Hkv > INT32_MAX / 2)
        return SDP_ERR_OVERFLOW;
    p.c.k_codes = static_cast<uint8_t *>(const_cast<void *>(k_codes));
    p.c.v_codes = static_cast<uint8_t *>(const_cast<void *>(v_codes));
    p.c.k_scales = static_cast<uint32_t *>(const_cast<void *>(k_scales));
    p.c.v_scales = static_cast<uint32_t *>(const_cast<void *>(v_scales));
    p.c.table = block_table;
    p.c.table_stride = table_stride;
    p.c.num_pages = num_pages;
    p.c.page_size = page_size;
    p.c.max_pages = max_pages;
    p.c.Hkv = Hkv;
    p.k = static_cast<uint16_t *>(const_cast<void *>(k));
    p.v = static_cast<uint16_t *>(const_cast<void *>(v));
    p.k_st = k_st;
    p.k_sh = k_sh;
    p.v_st = v_st;
    p.v_sh = v_sh;
    p.cu = cu;
    p.lens = with_lens ? lens : nullptr;
    p.nseq = nseq;
    p.tokens = tokens;
    return SDP_OK;
}

// Device, status word and the split of the rows over warps: one pass a warp while that leaves
// SMs without a full set of warps, then as many rows as share a token's look-up.
int plan(RowsParams &p, int D, unsigned *blocks)
{
    int dev = 0, sms = 0;
    int rc = sdp::current_device(&dev, &sms);
    if (rc != SDP_OK)
        return rc;
    if ((rc = sdp::status_word(dev, &p.status)) != SDP_OK)
        return rc;
    const int rpp = 256 / D;
    const long long rows = 2LL * p.c.Hkv, passes = (rows + rpp - 1) / rpp;
    long long per = p.tokens * passes / (static_cast<long long>(sms) * 32);
    per = per < 1 ? 1 : (per > passes ? passes : per);
    p.rows_per_warp = static_cast<int>(per * rpp);
    const long long runs = (rows + p.rows_per_warp - 1) / p.rows_per_warp;
    const long long n = (p.tokens * runs + kWarps - 1) / kWarps;
    if (n > INT32_MAX)
        return SDP_ERR_OVERFLOW;
    *blocks = static_cast<unsigned>(n);
    return SDP_OK;
}

}  // namespace

extern "C" int sdp_cache4_append(void *k_codes, void *k_scales, void *v_codes, void *v_scales, int num_pages,
                                 int page_size, const int *block_table, long long table_stride, int max_pages,
                                 const void *k, long long k_st, long long k_sh, const void *v, long long v_st,
                                 long long v_sh, const int *cu_seqlens, const int *cache_lens, int nseq, int tokens,
                                 int Hkv, int D, int dtype, void *stream)
{
    RowsParams p{};
    int rc = rows_params(p, k_codes, k_scales, v_codes, v_scales, num_pages, page_size, block_table, table_stride,
                         max_pages, k, k_st, k_sh, v, v_st, v_sh, cu_seqlens, cache_lens, true, nseq, tokens, Hkv, D,
                         dtype);
    if (rc != SDP_OK || tokens == 0)
        return rc;
    unsigned blocks = 0;
    if ((rc = plan(p, D, &blocks)) != SDP_OK)
        return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int threads = 32 * kWarps;
    if (D == 128 && dtype == SDP_BF16)
        cache4_append_kernel<128, true><<<blocks, threads, 0, st>>>(p);
    else if (D == 128)
        cache4_append_kernel<128, false><<<blocks, threads, 0, st>>>(p);
    else if (dtype == SDP_BF16)
        cache4_append_kernel<256, true><<<blocks, threads, 0, st>>>(p);
    else
        cache4_append_kernel<256, false><<<blocks, threads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}

extern "C" int sdp_cache4_gather(const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales,
                                 int num_pages, int page_size, const int *block_table, long long table_stride,
                                 int max_pages, void *k, long long k_st, long long k_sh, void *v, long long v_st,
                                 long long v_sh, const int *cu_seqlens, int nseq, int tokens, int Hkv, int D,
                                 int dtype, void *stream)
{
    RowsParams p{};
    int rc = rows_params(p, k_codes, k_scales, v_codes, v_scales, num_pages, page_size, block_table, table_stride,
                         max_pages, k, k_st, k_sh, v, v_st, v_sh, cu_seqlens, nullptr, false, nseq, tokens, Hkv, D,
                         dtype);
    if (rc != SDP_OK || tokens == 0)
        return rc;
    unsigned blocks = 0;
    if ((rc = plan(p, D, &blocks)) != SDP_OK)
        return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int threads = 32 * kWarps;
    if (D == 128 && dtype == SDP_BF16)
        cache4_gather_kernel<128, true><<<blocks, threads, 0, st>>>(p);
    else if (D == 128)
        cache4_gather_kernel<128, false><<<blocks, threads, 0, st>>>(p);
    else if (dtype == SDP_BF16)
        cache4_gather_kernel<256, true><<<blocks, threads, 0, st>>>(p);
    else
        cache4_gather_kernel<256, false><<<blocks, threads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}
