// The norm of every query and key head and the rotation by position, in one pass over both (sdp_qk_norm_rope), with
// the keys and values written into the pages of a 16-bit cache on the way (sdp_cache16_append).
//
// For the row x of one token and head (D channels), with weight w (the norm is left out where
// there is none):
//
//     y_c = x_c * w_c / sqrt(sum_j x_j^2 / D + eps)
//
// and for pair i of the first R channels, (y_i, y_{i + R/2}) or, interleaved, (y_2i, y_2i+1):
//
//     (a, b) -> m * (a cos t - b sin t, a sin t + b cos t),   t = position * f_i.
//
// Everything is in fp32, rounded once when the row is stored. Squares of bf16 values can leave fp32's
// range, and the norm's factor, applied last, would then meet an infinity: such a row (found by one test
// of its mean square) is brought near 1 by a power of two first, which the factor takes along.
//
// Angles: fp32 products lose the angle at far positions (position 1e6 leaves an error of 0.06
// rad), so the table holds each frequency in turns per position as a 64-bit binary fraction,
// u_i = f_i / (2 pi) * 2^64: position * u_i modulo 2^64 is the fraction of a turn, exactly as
// far as u_i is, and its upper 32 bits, read as a signed number, are the angle in units of
// 2^-31 half turns for sincospif. The product costs three integer multiplications.
//
// The work is HBM-bound: each element is read and written once, and at full bandwidth an SM has
// about 170 issue slots for a 512-byte pass of a warp. So what a row's channels share over a token's
// heads is folded once: with A = w cos (w outside the rotation) and B = -+ w' sin for the partner's
// weight w', an element is r * (A x + B x'), r the row's norm factor, in packed pairs of fp32; the
// partner x' travels as it was loaded (four 32-bit shuffles a row). A warp takes one token and a run
// of its passes (32 / (D / 8) rows of q or of k, one 16-byte load a lane), kPassUnroll passes' loads
// in flight; the token's R/2 cosines and sines are computed once for the run, spread over the lanes,
// and read back from shared memory. 39253 tokens of 34 heads at D = 256 take 233 us, 86 % of the copy
// rate. (With the weights applied and fp32 values shuffled row by row they took 348 us.)
//
// Appending (34332 tokens of 36 heads at D = 256: 219 us, 85 % of the copy rate; 3095 of 96 heads at D = 128: 32 us, 69 %) adds
// the look-up of a token's place, whose trips to memory run beside the first rows' loads, the position's and the
// frequencies' (one after the other, 34.4 us for the second). Rows loaded one at a time, as they are consumed, instead of
// kPassUnroll at once: 275 us for the first.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "sdp_internal.h"
#include "sixteen.cuh"

namespace sdp {
namespace rope {

constexpr int kWarps = 4;
constexpr int kPassUnroll = 4;
constexpr unsigned FULL = 0xffffffffu;
// Rows whose mean square (with eps) lies between are normed as they are: their squares do not vanish, and times any
// weight up to 2^100 they stay finite. The others, which only bf16 can hold (or zeros without an eps), are brought
// near 1 by a power of two first.
constexpr float MEAN_LOW = 0x1p-80f, MEAN_HIGH = 0x1p40f;

struct RopeParams {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    // strides in elements: batch, token, head
    long long qs[3], ks[3], qos[3], kos[3];
    const void *positions;
    long long ps[2];  // batch, token
    const unsigned long long *turns;
    const void *wq, *wk;
    float mscale, eps;
    int S, Hq, Hkv, R;
    int tokens;         // B * S
    int passes_q, passes;  // of a token: q's, and q's and k's
    int per_warp;          // passes a warp runs through
};

// The cache that rows are appended to (CACHE): k and v pools [num_pages, Hkv, page_size, D].
struct CacheDest {
    uint16_t *k, *v_pool;
    const uint16_t *v;  // the new tokens' values
    long long v_st, v_sh;
    const int *cu, *lens, *table;
    long long table_stride;
    unsigned int *status;
    int nseq, num_pages, page_size, max_pages, Hkv;
    int passes_k;  // q's and k's passes of a token, which come before v's
    int positions_64;
};

// w: eight weights at channel c0 of `base`, 16-bit or fp32.
template <bool BF16, bool W32>
__device__ __forceinline__ void load_weights(const void *base, int c0, float (&w)[8])
{
    if constexpr (W32) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(base) + c0));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(base) + c0 + 4));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + c0)), w);
    }
}

// Where a token goes in the cache.
struct Place {
    int position;  // in its sequence; -1: the token is in no sequence (or in a bad one)
    int id, at;    // the page, as the table has it, and the place in it
};

// Where `token` goes. Called by a whole warp: its sequence is searched by all lanes together, 32 candidates a step, and what
// belongs to the last 31 comes in the same trip to memory. (A short call's time is its chain of such trips: this one, the
// table's, and then the rows' way out.) Status codes for bad offsets and lengths.
__device__ __forceinline__ Place locate(const CacheDest &c, int token, int tokens)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = c.nseq;  // the last sequence that begins at or before the token lies in [lo, lo + n)
    while (n > 31) {
        const int step = (n + 31) / 32;
        const bool before = lane * step < n && __ldg(c.cu + lo + lane * step) <= token;
        const unsigned m = __ballot_sync(FULL, before);
        const int used = m == 0u ? 0 : (31 - __clz(m)) * step;
        lo += used;
        n = min(step, n - used);
    }
    const int mine = __ldg(c.cu + lo + min(lane, n)), my_len = __ldg(c.lens + lo + min(lane, n - 1));
    const unsigned m = __ballot_sync(FULL, lane < n && mine <= token);
    const int used = m == 0u ? 0 : 31 - __clz(m);
    const int first = __shfl_sync(FULL, mine, used), end = __shfl_sync(FULL, mine, used + 1);
    const int len = __shfl_sync(FULL, my_len, used);
    Place r{-1, -1, 0};
    if (token < first || token >= end)
        return r;  // in no sequence: left as it is
    const bool ok = first >= 0 && end <= tokens && len >= end - first;
    const int place = ok ? token - first + (len - (end - first)) : 0;  // below len
    const int slot = place / c.page_size;
    if (!ok || slot >= c.max_pages) {
        if (lane == 0)
            atomicCAS(c.status, 0u, kBadSeqlens);
        return r;
    }
    r.position = place;
    r.id = __ldg(c.table + (lo + used) * c.table_stride + slot);  // (looked at by `row_of`: the angles are computed meanwhile)
    r.at = place - slot * c.page_size;
    return r;
}

// Its place in head 0's rows of the pool ([pages * Hkv * page_size] rows), or -1 and a status code where the page is outside.
__device__ __forceinline__ long long row_of(const CacheDest &c, const Place &p)
{
    if (p.id < 0 || p.id >= c.num_pages) {
        if ((threadIdx.x & 31) == 0)
            atomicCAS(c.status, 0u, kBadPages);
        return -1;
    }
    return static_cast<long long>(p.id) * c.Hkv * c.page_size + p.at;
}

// CACHE: k's rows go to their pages, v's are copied to theirs (a third segment of a token's passes), and a token's
// position is its place in its sequence unless positions are given (of the type that positions_64 tells).
template <int D, bool BF16, bool W32, bool POS64, bool INTERLEAVED, bool CACHE>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const RopeParams p, const CacheDest c)
{
    constexpr int LPR = D / 8;     // lanes a row
    constexpr int RPP = 32 / LPR;  // rows a pass
    __shared__ float2 cs_all[kWarps][D / 2];
    if constexpr (CACHE) {  // launched while the kernel before it ends; the attention over the cache may be likewise
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int runs = (p.passes + p.per_warp - 1) / p.per_warp;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (item >= static_cast<long long>(p.tokens) * runs)
        return;
    const int token = static_cast<int>(item / runs);
    const int pass0 = static_cast<int>(item - static_cast<long long>(token) * runs) * p.per_warp;
    const int pass1 = min(p.passes, pass0 + p.per_warp);
    const int b = CACHE ? 0 : token / p.S, s = CACHE ? token : token - b * p.S;
    float2 *cs = cs_all[warp];

    const int sub = lane / LPR, c0 = (lane % LPR) * 8;
    const uint16_t *q = p.q + b * p.qs[0] + s * p.qs[1] + c0;
    const uint16_t *k = p.k + b * p.ks[0] + s * p.ks[1] + c0;
    // The run as a segment of q's heads and one of k's (and one of v's): first head, heads left from it.
    const bool q_first = pass0 < p.passes_q;
    const int end_q = min(pass1, p.passes_q);
    const int end_k = CACHE ? min(pass1, c.passes_k) : pass1;  // v's passes come last, as many as k's
    const uint16_t *src;
    long long step;
    int left;  // rows from this lane's first on: live while > 0
    uint4 v[kPassUnroll];
    auto load = [&]() {  // the next kPassUnroll passes' rows
#pragma unroll
        for (int i = 0; i < kPassUnroll; ++i) {
            v[i] = left > 0 ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0u, 0u, 0u, 0u);
            src += step;
            left -= RPP;
        }
    };
    auto open = [&](bool of_q) {
        const int h0 = (of_q ? pass0 : max(0, pass0 - p.passes_q)) * RPP + sub;
        const int h1 = of_q ? min(p.Hq, end_q * RPP) : min(p.Hkv, (end_k - p.passes_q) * RPP);
        step = (of_q ? p.qs[2] : p.ks[2]);
        src = (of_q ? q : k) + h0 * step;
        step *= RPP;
        left = h1 - h0;
        load();
    };
    [[maybe_unused]] auto open_v = [&]() {
        const int h0 = max(0, pass0 - c.passes_k) * RPP + sub;
        const int h1 = min(p.Hkv, (pass1 - c.passes_k) * RPP);
        src = c.v + s * c.v_st + c0 + h0 * c.v_sh;
        step = c.v_sh * RPP;
        left = h1 - h0;
        load();
    };
    // the first rows' loads run while the angles (and the place in the cache) are computed
    if (!CACHE || pass0 < c.passes_k)
        open(q_first);
    else
        open_v();
    // and so do those of the frequencies (as many as half of the shorter heads has) and of the position, where it is given
    const int half = p.R / 2;
    [[maybe_unused]] const bool turned = half > 0 && (!CACHE || pass0 < c.passes_k);
    unsigned long long turns[2] = {0, 0};
    long long given = 0;
    if (CACHE && turned) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (lane + 32 * x < half)
                turns[x] = __ldg(p.turns + lane + 32 * x);
        const long long at = s * p.ps[1];
        if (p.positions != nullptr)
            given = c.positions_64 != 0 ? static_cast<const long long *>(p.positions)[at] : static_cast<const int *>(p.positions)[at];
    }
    Place place{0, 0, 0};
    if constexpr (CACHE) {
        if (blockIdx.x == 0) {  // all offsets: a token of a sequence with bad ones may belong to none
            const int warps = static_cast<int>(min(static_cast<long long>(p.tokens) * runs, static_cast<long long>(kWarps)));  // with work
            for (int i = threadIdx.x; i < c.nseq; i += 32 * warps) {
                const int x = __ldg(c.cu + i), y = __ldg(c.cu + i + 1);
                if (x < 0 || y < x || y > p.tokens)
                    atomicCAS(c.status, 0u, kBadSeqlens);
            }
        }
        place = locate(c, token, p.tokens);
        if (place.position < 0)
            return;
    }

    if (turned) {
        const long long at = b * p.ps[0] + s * p.ps[1];
        const long long pos = CACHE ? (p.positions == nullptr ? place.position : given)
                              : POS64 ? static_cast<const long long *>(p.positions)[at]
                                      : static_cast<const int *>(p.positions)[at];
        for (int i = lane; i < half; i += 32) {
            const unsigned long long per = CACHE && i < 64 ? (i < 32 ? turns[0] : turns[1]) : __ldg(p.turns + i);
            const unsigned long long turn = static_cast<unsigned long long>(pos) * per;
            float sn, c;
            sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &c);  // 2^-31
            cs[i] = make_float2(c * p.mscale, sn * p.mscale);
        }
        __syncwarp();
    }
    // this lane's pairs: interleaved, pairs c0/2 .. +3 of its own channels; else pairs c0 .. +7 of
    // its channels and those R/2 away, which lane +- R/16 of the same row holds
    const bool turns_here = c0 < p.R;
    const bool upper = c0 >= half;
    const int partner_c0 = INTERLEAVED || !turns_here ? c0 : upper ? c0 - half : c0 + half;
    const int partner = lane + (partner_c0 - c0) / 8;
    uint64_t fa[4], fb[4];  // the factors A and B of the lane's channels, for q or for k
    auto factors = [&](bool of_q) {
        const void *wb = of_q ? p.wq : p.wk;
        float w[8], wp[8], x[8], y[8];
        if (wb != nullptr) {
            load_weights<BF16, W32>(wb, c0, w);
            load_weights<BF16, W32>(wb, partner_c0, wp);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float we = wb != nullptr ? w[e] : 1.f;
            x[e] = we;
            y[e] = 0.f;
            if (turns_here) {
                const float2 t = INTERLEAVED ? cs[c0 / 2 + e / 2] : cs[(upper ? c0 - half : c0) + e];
                const float wo = wb != nullptr ? wp[INTERLEAVED ? e ^ 1 : e] : 1.f;
                x[e] = we * t.x;
                // the partner's sign: - sin for a pair's first channel, + sin for its second
                y[e] = wo * ((INTERLEAVED ? (e & 1) : upper) ? t.y : -t.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[i] = sdp::ptx::f2_pack(x[2 * i], x[2 * i + 1]);
            fb[i] = sdp::ptx::f2_pack(y[2 * i], y[2 * i + 1]);
        }
    };

    auto mean_square = [&](const uint64_t (&x)[4]) {
        uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j)
            sq = sdp::ptx::f2_fma(x[j], x[j], sq);
        float s0, s1;
        sdp::ptx::f2_unpack(sq, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1)
            ss += __shfl_xor_sync(FULL, ss, off);
        return ss * (1.f / D);
    };
    // y = A x + B x' of the row x, whose words are w; `down`: a pair that x has been multiplied by, or an int
    auto weigh = [&](const uint64_t (&x)[4], uint64_t (&y)[4], const uint32_t (&w)[4], auto down) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            y[j] = mul2(x[j], fa[j]);
        if (half == 0)
            return;
        uint32_t o[4];
        if constexpr (!INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = __shfl_sync(FULL, w[j], partner);
        }
        if (!turns_here)  // outside the rotation B is no factor: 0 times an infinity is NaN
            return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint64_t other;
            if constexpr (INTERLEAVED) {
                float lo, hi;
                sdp::ptx::f2_unpack(x[j], lo, hi);
                other = sdp::ptx::f2_pack(hi, lo);
            } else {
                const float2 f = sdp::unpack16<BF16>(o[j]);
                other = sdp::ptx::f2_pack(f.x, f.y);
                if constexpr (sizeof(down) == 8)
                    other = mul2(other, down);
            }
            y[j] = sdp::ptx::f2_fma(other, fb[j], y[j]);
        }
    };

    for (int seg = q_first ? 0 : 1; seg < 2; ++seg) {
        const bool of_q = seg == 0;
        const int passes = of_q ? end_q - pass0 : end_k - max(pass0, p.passes_q);
        if (passes <= 0)
            break;
        if (of_q != q_first)
            open(of_q);
        factors(of_q);
        const bool normed = (of_q ? p.wq : p.wk) != nullptr;
        const int h0 = (of_q ? pass0 : max(0, pass0 - p.passes_q)) * RPP + sub;
        int live = (of_q ? min(p.Hq, end_q * RPP) : min(p.Hkv, (end_k - p.passes_q) * RPP)) - h0;
        uint16_t *dst;
        long long dst_step;
        if (of_q) {
            dst = p.q_out + b * p.qos[0] + s * p.qos[1] + h0 * p.qos[2] + c0;
            dst_step = p.qos[2] * RPP;
        } else if constexpr (CACHE) {
            const long long row = row_of(c, place);
            dst = c.k + (row + static_cast<long long>(h0) * c.page_size) * D + c0;
            dst_step = static_cast<long long>(c.page_size) * D * RPP;
            if (row < 0)
                live = 0;  // the page is not there
        } else {
            dst = p.k_out + b * p.kos[0] + s * p.kos[1] + h0 * p.kos[2] + c0;
            dst_step = p.kos[2] * RPP;
        }
        for (int pass = 0; pass < passes; pass += kPassUnroll) {
            uint4 now[kPassUnroll];
#pragma unroll
            for (int i = 0; i < kPassUnroll; ++i)
                now[i] = v[i];
            if (pass + kPassUnroll < passes)
                load();
#pragma unroll
            for (int i = 0; i < kPassUnroll; ++i) {
                if (pass + i >= passes)
                    break;  // the same for the whole warp
                const uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
                uint64_t x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = sdp::unpack16<BF16>(w[j]);
                    x[j] = sdp::ptx::f2_pack(f.x, f.y);
                }
                weigh(x, y, w, 0);
                if (normed) {
                    const float t = mean_square(x) + p.eps;
                    float r = rsqrtf(t);
                    if constexpr (BF16) {
                        const bool odd = live > 0 && !(t > MEAN_LOW && t < MEAN_HIGH);
                        if (__any_sync(FULL, odd)) {
                            float mx = sqrtf(p.eps);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = sdp::unpack16<BF16>(w[j]);
                                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                            }
#pragma unroll
                            for (int off = LPR / 2; off > 0; off >>= 1)
                                mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
                            // 2^-e for mx in [2^e, 2^(e + 1)), where both are normal numbers
                            const int e = min(126, max(-126, static_cast<int>(__float_as_uint(mx) >> 23) - 127));
                            const float down = odd ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f;
                            const uint64_t down2 = sdp::ptx::f2_pack(down, down);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[j] = mul2(x[j], down2);
                            weigh(x, y, w, down2);
                            const float scaled = rsqrtf(mean_square(x) + p.eps * down * down);
                            r = odd ? scaled : r;  // a row's bits do not depend on its neighbours in the warp
                        }
                    }
                    const uint64_t rr = sdp::ptx::f2_pack(r, r);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[j] = mul2(y[j], rr);
                }
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    sdp::ptx::f2_unpack(y[j], lo, hi);
                    o[j] = sdp::pack16<BF16>(lo, hi);
                }
                if (live > 0)
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                dst += dst_step;
                live -= RPP;
            }
        }
    }
    if constexpr (CACHE) {
        const int passes = pass1 - max(pass0, c.passes_k);
        if (passes <= 0)
            return;
        const long long row = row_of(c, place);
        if (row < 0)
            return;
        if (pass0 < c.passes_k)
            open_v();
        const int h0 = max(0, pass0 - c.passes_k) * RPP + sub;
        int live = min(p.Hkv, (pass1 - c.passes_k) * RPP) - h0;
        uint16_t *dst = c.v_pool + (row + static_cast<long long>(h0) * c.page_size) * D + c0;
        const long long dst_step = static_cast<long long>(c.page_size) * D * RPP;
        for (int pass = 0; pass < passes; pass += kPassUnroll) {
            uint4 now[kPassUnroll];
#pragma unroll
            for (int i = 0; i < kPassUnroll; ++i)
                now[i] = v[i];
            if (pass + kPassUnroll < passes)
                load();
#pragma unroll
            for (int i = 0; i < kPassUnroll; ++i) {
                if (live > 0)
                    *reinterpret_cast<uint4 *>(dst) = now[i];
                dst += dst_step;
                live -= RPP;
            }
        }
    }
}

}  // namespace rope
}  // namespace sdp
