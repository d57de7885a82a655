// sdp_cache4_append and sdp_cache4_gather: the 4-bit paged cache's writer, and its reader into
// 16-bit rows (cache4.cuh has the layout).
//
// Writing a group of 64 channels x_c:  b = bf16(min x),  s = bf16(max(0, (max x - b) / 15)),
// n_c = clamp(rint((x_c - b) / s), 0, 15), 0 where s = 0. The quotient is correctly rounded: inputs
// of few bits often lie exactly on a border between two codes, where a product with 1 / s alone
// falls on either side. One correctly rounded reciprocal serves the group, and each quotient is
// corrected by its exact remainder (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): three operations an element where a division takes a dozen. The
// extremes are found on the 16-bit pairs as loaded, minimum and negated maximum in one register.
//
// Both kernels are elementwise passes over HBM at about half of its rate: 62529 tokens of 2 heads of 256
// channels take 43 us written and 32 us read back where the bytes alone take 24 us each (apart, in runs of
// calls; 42.6 and 29.4 us under ncu). The writer issues 2.7 instructions a cycle of 4, its integer units half
// busy: a group costs a reduction, a division and a reciprocal before its elements begin. The reader waits for
// its loads (5.5 of some 10 stalled warps an issue), with the 32 warps an SM that plan() gives it. A warp takes a few
// consecutive tokens and runs over their 2 Hkv rows each (K heads, then V heads), D/16 lanes a row. A lane
// holds two chunks of eight channels of one group, each one 16-byte access on the 16-bit side and one 4-byte
// word of codes on the other, so that four lanes share what a group costs. (With one chunk a lane, eight
// lanes a group, the two took 65 and 46 us, cold, with four 75 and 40, and with two 46 and 36: half the warps
// with twice the registers leave the loads' latency open.) Each lane looks up the place of one of the warp's tokens (a chain of
// dependent loads, which one token a warp left exposed).
#include <cuda_runtime.h>

#include <cstdint>

#include "cache4.cuh"
#include "ptx.cuh"
#include "sdp.h"
#include "sixteen.cuh"

namespace {

using sdp::Cache4View;
using sdp::mul2;
using sdp::unpack8;

constexpr int kWarps = 4;
constexpr int kUnroll = 2;           // passes whose loads a warp issues at once
constexpr int kChunks = 2;           // of eight channels a lane, all of one group
constexpr int kLanes = 8 / kChunks;  // of a group
constexpr int kStep = 8 * kLanes;    // channels from one of a lane's chunks to the next
constexpr int kMaxPasses = 32;      // of a warp that takes several tokens
constexpr unsigned FULL = 0xffffffffu;

struct RowsParams {
    Cache4View c;
    uint16_t *k, *v;                   // 16-bit rows: read by append, written by gather
    long long k_st, k_sh, v_st, v_sh;  // token and head strides in elements
    const int *cu, *lens;              // gather: lens is null, rows of a sequence are its tokens from 0
    unsigned int *status;
    int nseq, tokens;
    int tokens_per_warp;  // consecutive tokens a warp takes, up to 32
    int per_warp;         // passes of a token that a warp runs through
};

// Where this lane's token (token0 + lane, one of `n`) lives, as its row of head 0 in the pool's
// [pages * Hkv * page_size] rows; -1 where it is in no sequence, or (with a status code) for bad offsets and
// pages outside the pool. Called by a whole warp: the first token's sequence is searched by all lanes
// together, 32 candidates a step (two trips to memory for 1024 sequences); the others' are near it.
__device__ __forceinline__ long long locate(const RowsParams &p, int token0, int n, int lane)
{
    int lo = 0;
    for (int len = p.nseq; len > 1;) {  // the last sequence that begins at or before token0 lies in [lo, lo + len)
        const int step = (len + 31) / 32;
        const bool before = lane * step < len && __ldg(p.cu + lo + lane * step) <= token0;
        const unsigned m = __ballot_sync(FULL, before);
        const int used = m == 0u ? 0 : (31 - __clz(m)) * step;
        lo += used;
        len = min(step, len - used);
    }
    const int token = token0 + lane;
    if (lane >= n)
        return -1;
    int next = __ldg(p.cu + lo + 1);
    while (token >= next && lo + 1 < p.nseq)  // over empty sequences too
        next = __ldg(p.cu + ++lo + 1);
    if (token < __ldg(p.cu + lo))
        return -1;
    const int first = __ldg(p.cu + lo), end = next;
    if (token >= end)
        return -1;  // in no sequence: left as it is
    bool ok = first >= 0 && end <= p.tokens && first <= token;
    int pos = ok ? token - first : 0;
    if (ok && p.lens != nullptr) {
        const int len = __ldg(p.lens + lo);
        ok = len >= end - first;
        pos += ok ? len - (end - first) : 0;  // below len
    }
    const int slot = ok ? pos / p.c.page_size : 0;
    if (!ok || slot >= p.c.max_pages) {
        atomicCAS(p.status, 0u, sdp::kBadSeqlens);
        return -1;
    }
    const int id = __ldg(p.c.table + lo * p.c.table_stride + slot);
    if (id < 0 || id >= p.c.num_pages) {
        atomicCAS(p.status, 0u, sdp::kBadPages);
        return -1;
    }
    return static_cast<long long>(id) * p.c.Hkv * p.c.page_size + (pos - slot * p.c.page_size);
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

// A warp's share: tokens [token0, + n) and of each the passes [pass0, pass1), RPP rows a pass (K's
// heads, then V's). Passes are numbered through, token by token.
template <int D>
struct Share {
    static constexpr int LPR = D / 64 * kLanes, RPP = 32 / LPR;
    int token0, pass0, per_token, count;
    int passes_k;  // K's passes of a token (V's are as many)
    __device__ __forceinline__ explicit Share(const RowsParams &p)
    {
        passes_k = (p.c.Hkv + RPP - 1) / RPP;
        const int runs = (2 * passes_k + p.per_warp - 1) / p.per_warp;
        const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        const long long group = item / runs;
        pass0 = static_cast<int>(item - group * runs) * p.per_warp;
        per_token = min(2 * passes_k, pass0 + p.per_warp) - pass0;
        const long long t0 = group * p.tokens_per_warp;
        token0 = static_cast<int>(min(static_cast<long long>(p.tokens), t0));
        count = min(p.tokens_per_warp, p.tokens - token0) * per_token;
    }
    __device__ __forceinline__ int tokens() const { return count / per_token; }
};

// A place in a share's passes: the token (index in the share), K or V, and this lane's head (-1 past the last).
template <int D>
struct Cursor {
    int token, y;
    __device__ __forceinline__ explicit Cursor(const Share<D> &sh) : token(0), y(sh.pass0) {}
    __device__ __forceinline__ void next(const Share<D> &sh)
    {
        if (++y == sh.pass0 + sh.per_token) {
            y = sh.pass0;
            ++token;
        }
    }
    __device__ __forceinline__ bool is_k(const Share<D> &sh) const { return y < sh.passes_k; }
    __device__ __forceinline__ int head(const RowsParams &p, const Share<D> &sh, int sub) const
    {
        const int h = (y < sh.passes_k ? y : y - sh.passes_k) * Share<D>::RPP + sub;
        return h < p.c.Hkv ? h : -1;
    }
};

// First of a lane's channels in its row: a group's lanes take its chunks of eight channels in turn, so that each
// access of the lanes together is in one piece.
__device__ __forceinline__ int first_channel(int lane_of_row)
{
    return lane_of_row / kLanes * sdp::kCacheGroup + lane_of_row % kLanes * 8;
}

// Minimum of two pairs of 16-bit floats that keeps NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// t / s correctly rounded, from the correctly rounded reciprocal of s.
__device__ __forceinline__ float quotient(float t, float s, float inv)
{
    const float q = __fmul_rn(t, inv);
    return __fmaf_rn(__fmaf_rn(-q, s, t), inv, q);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kWarps) cache4_append_kernel(const RowsParams p)
{
    using S = Share<D>;
    const int lane = threadIdx.x & 31;
    check_offsets(p);
    const S sh(p);
    if (sh.count <= 0)
        return;
    const int sub = lane / S::LPR, c0 = first_channel(lane % S::LPR);
    uint4 v[kUnroll][kChunks];
    Cursor<D> ahead(sh), at(sh);
    int to_load = sh.count;
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = to_load > 0 ? ahead.head(p, sh, sub) : -1;
            const long long t = sh.token0 + ahead.token;
            const uint16_t *src =
                (ahead.is_k(sh) ? p.k + t * p.k_st + h * p.k_sh : p.v + t * p.v_st + h * p.v_sh) + c0;
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
                v[i][x] = h < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4 *>(src + x * kStep));
            ahead.next(sh);
            --to_load;
        }
    };
    load();
    const long long my_row = locate(p, sh.token0, sh.tokens(), lane);
    for (int x0 = 0; x0 < sh.count; x0 += kUnroll) {
        uint4 now[kUnroll][kChunks];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
                now[i][x] = v[i][x];
        if (to_load > 0)
            load();
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (x0 + i >= sh.count)
                break;  // the same for the whole warp
            const long long row0 = __shfl_sync(FULL, my_row, at.token);
            const int h = at.head(p, sh, sub);
            const bool is_k = at.is_k(sh);
            at.next(sh);
            uint32_t w[4 * kChunks];
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
                w[4 * x] = now[i][x].x, w[4 * x + 1] = now[i][x].y, w[4 * x + 2] = now[i][x].z, w[4 * x + 3] = now[i][x].w;
            // (minimum, - maximum) of the group, in the type of the rows: exact
            constexpr uint32_t SIGNS = 0x80008000u;
            uint32_t lo = w[0], hi = w[0] ^ SIGNS;
#pragma unroll
            for (int j = 1; j < 4 * kChunks; ++j) {
                lo = min2_nan<BF16>(lo, w[j]);
                hi = min2_nan<BF16>(hi, w[j] ^ SIGNS);
            }
            uint32_t both = min2_nan<BF16>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1)
                both = min2_nan<BF16>(both, __shfl_xor_sync(FULL, both, off));
            const float2 ends = sdp::unpack16<BF16>(both);
            const uint32_t b16 = __bfloat16_as_ushort(__float2bfloat16_rn(ends.x));
            const float b = __uint_as_float(b16 << 16);
            const float span = __fsub_rn(-ends.y, b);
            uint32_t codes[kChunks] = {}, s16;
            if (span > 1e-28f && span < 1e30f) {
                const float q15 = quotient(span, 15.f, 1.f / 15.f);
                s16 = __bfloat16_as_ushort(__float2bfloat16_rn(q15));
                const float s = __uint_as_float(s16 << 16), inv = __frcp_rn(s);
                const uint64_t s2 = sdp::ptx::f2_pack(-s, -s), inv2 = sdp::ptx::f2_pack(inv, inv);
                const uint64_t b2 = sdp::ptx::f2_pack(-b, -b), big = sdp::ptx::f2_pack(8388608.f, 8388608.f);
                uint32_t bytes[4 * kChunks];
#pragma unroll
                for (int j = 0; j < 4 * kChunks; ++j) {
                    const float2 f = sdp::unpack16<BF16>(w[j]);
                    const uint64_t t = sdp::ptx::f2_add(sdp::ptx::f2_pack(f.x, f.y), b2);
                    uint64_t q = mul2(t, inv2);
                    q = sdp::ptx::f2_fma(sdp::ptx::f2_fma(q, s2, t), inv2, q);  // t / s, correctly rounded
                    float q0, q1;
                    sdp::ptx::f2_unpack(q, q0, q1);
                    // below 15.5 always (s >= (1 - 2^-9) span / 15); below 0 where b was rounded up. 2^23 + q
                    // rounds to the code, ties to even
                    const uint64_t r = sdp::ptx::f2_add(sdp::ptx::f2_pack(fmaxf(q0, 0.f), fmaxf(q1, 0.f)), big);
                    float r0, r1;
                    sdp::ptx::f2_unpack(r, r0, r1);
                    bytes[j] = __float_as_uint(fmaf(r1 - 8388608.f, 16.f, r0));  // both codes in the low byte
                }
#pragma unroll
                for (int x = 0; x < kChunks; ++x)
                    codes[x] = __byte_perm(__byte_perm(bytes[4 * x], bytes[4 * x + 1], 0x0040),
                                           __byte_perm(bytes[4 * x + 2], bytes[4 * x + 3], 0x0040), 0x5410);
            } else {  // a constant group, a NaN, or a scale whose reciprocal or remainders leave fp32's range
                const float q15 = __fdiv_rn(span, 15.f);
                s16 = __bfloat16_as_ushort(__float2bfloat16_rn(q15 < 0.f ? 0.f : q15));  // NaN stays
                const float s = __uint_as_float(s16 << 16);
                if (s != 0.f) {
#pragma unroll
                    for (int x = 0; x < kChunks; ++x) {
                        float f[8];
                        unpack8<BF16>(now[i][x], f);
#pragma unroll 1
                        for (int e = 0; e < 8; ++e) {
                            const float n = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(f[e], b), s)), 0.f), 15.f);
                            codes[x] |= static_cast<uint32_t>(static_cast<int>(n)) << (4 * e);
                        }
                    }
                }
            }
            if (h >= 0 && row0 >= 0) {
                const long long row = row0 + static_cast<long long>(h) * p.c.page_size;
                uint8_t *dst = (is_k ? p.c.k_codes : p.c.v_codes) + row * (D / 2) + c0 / 2;
#pragma unroll
                for (int x = 0; x < kChunks; ++x)
                    *reinterpret_cast<uint32_t *>(dst + x * kStep / 2) = codes[x];
                if (c0 % sdp::kCacheGroup == 0)
                    (is_k ? p.c.k_scales : p.c.v_scales)[row * (D / sdp::kCacheGroup) + c0 / sdp::kCacheGroup] =
                        s16 | (b16 << 16);
            }
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kWarps) cache4_gather_kernel(const RowsParams p)
{
    using S = Share<D>;
    const int lane = threadIdx.x & 31;
    check_offsets(p);
    const S sh(p);
    if (sh.count <= 0)
        return;
    const long long my_row = locate(p, sh.token0, sh.tokens(), lane);
    const int sub = lane / S::LPR, c0 = first_channel(lane % S::LPR);
    Cursor<D> at(sh);
    for (int x0 = 0; x0 < sh.count; x0 += kUnroll) {
        uint32_t codes[kUnroll][kChunks], pair[kUnroll];
        uint16_t *out[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const long long row0 = __shfl_sync(FULL, my_row, at.token & 31);
            const int h = x0 + i < sh.count ? at.head(p, sh, sub) : -1;
            const bool is_k = at.is_k(sh);
            out[i] = nullptr;
            if (h >= 0 && row0 >= 0) {
                const long long row = row0 + static_cast<long long>(h) * p.c.page_size;
                const uint8_t *src = (is_k ? p.c.k_codes : p.c.v_codes) + row * (D / 2) + c0 / 2;
#pragma unroll
                for (int x = 0; x < kChunks; ++x)
                    codes[i][x] = __ldg(reinterpret_cast<const uint32_t *>(src + x * kStep / 2));
                pair[i] = __ldg((is_k ? p.c.k_scales : p.c.v_scales) + row * (D / sdp::kCacheGroup) +
                                c0 / sdp::kCacheGroup);
                const long long t = sh.token0 + at.token;
                out[i] = (is_k ? p.k + t * p.k_st + h * p.k_sh : p.v + t * p.v_st + h * p.v_sh) + c0;
            }
            at.next(sh);
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (out[i] == nullptr)
                continue;
            const float s = __uint_as_float(pair[i] << 16), b = __uint_as_float(pair[i] & 0xffff0000u);
            const uint64_t s2 = sdp::ptx::f2_pack(s, s), b2 = sdp::ptx::f2_pack(b, b);
            const uint64_t big = sdp::ptx::f2_pack(-8388608.f, -8388608.f);
#pragma unroll
            for (int x = 0; x < kChunks; ++x) {
                // a byte a code, then a code as 2^23 + n less 2^23; s * n is exact in fp32 (8 + 4 bits): one rounding,
                // then the store's
                const uint32_t even = codes[i][x] & 0x0f0f0f0fu, odd = (codes[i][x] >> 4) & 0x0f0f0f0fu;
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t n = sdp::ptx::f2_pack(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7550 | j)),
                                                         __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7550 | j)));
                    float lo, hi;
                    sdp::ptx::f2_unpack(sdp::ptx::f2_fma(s2, sdp::ptx::f2_add(n, big), b2), lo, hi);
                    o[j] = sdp::pack16<BF16>(lo, hi);
                }
                *reinterpret_cast<uint4 *>(out[i] + x * kStep) = make_uint4(o[0], o[1], o[2], o[3]);
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

// Device, status word and the split of the passes over warps: one pass a warp while that leaves SMs
// without a full set of warps, then a token's passes, then several tokens that share one look-up.
int plan(RowsParams &p, int D, unsigned *blocks)
{
    int dev = 0, sms = 0;
    int rc = sdp::current_device(&dev, &sms);
    if (rc != SDP_OK)
        return rc;
    if ((rc = sdp::status_word(dev, &p.status)) != SDP_OK)
        return rc;
    const int rpp = 32 / (D / 64 * kLanes);
    const long long passes = 2LL * ((p.c.Hkv + rpp - 1) / rpp);
    long long per = p.tokens * passes / (static_cast<long long>(sms) * 32);
    per = per < 1 ? 1 : per;
    p.per_warp = static_cast<int>(per < passes ? per : passes);
    // enough passes a warp to pay for the look-up, while every SM keeps its warps
    long long share = per / passes < kMaxPasses / passes ? per / passes : kMaxPasses / passes;
    p.tokens_per_warp = static_cast<int>(share < 1 ? 1 : (share > 32 ? 32 : share));
    const long long runs = (passes + p.per_warp - 1) / p.per_warp;
    const long long groups = (static_cast<long long>(p.tokens) + p.tokens_per_warp - 1) / p.tokens_per_warp;
    const long long n = (groups * runs + kWarps - 1) / kWarps;
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
