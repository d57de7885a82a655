// The join of the parts that the 16-bit cache attention leaves in the workspace.
#pragma once

#include "cache16.cuh"
#include "ptx.cuh"
#include "sdp_fwd_kernel.cuh"

namespace sdp {

namespace c16 {

constexpr int JOIN_THREADS = 128;
// A part's weight beside the largest is positive, however small: an infinity among its values (of a drafted token, where add_odd
// has put it onto the part) stays one, as in a row that is not joined. 2^-149 of bf16's largest value is 2^-21, of a sum that is
// divided by 1 or more.
constexpr float LEAST = 0x1p-149f;

// Where a row's parts of one problem are: the word the problem's first run left, and the row's place in a part.
struct Parts {
    int2 word;  // first run, parts (1: whole, by rows of q)
    int row;
    const float *whole;
};

}  // namespace c16

// Adds up the parts of every row that has more than one, the prefix's first, in the order of the runs, and writes the rows
// that see nothing. A warp has a row (SHARE = 1) or, with few rows, whose problems are cut into many parts, the four
// warps of a block have one, every fourth part each.
template <int D, bool BF16, int SHARE>
__global__ void __launch_bounds__(c16::JOIN_THREADS) cache16_join_kernel(const __grid_constant__ Cache16Params p)
{
    using namespace c16;
    constexpr int V = D / 128;  // float4 a lane
    __shared__ float4 y_all[SHARE][32 * V];
    // (what is launched early by this reads nothing before this kernel has ended)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int all = p.nseq * p.n * p.Hq;
    const int row = SHARE == 1 ? blockIdx.x * (JOIN_THREADS / 32) + warp : blockIdx.x;
    const bool in = row < all;
    const int tok = in ? row / p.Hq : 0, head = in ? row - tok * p.Hq : 0;
    const int s = tok / p.n, t = tok - s * p.n;
    const Span sp = span_of(p, p.ngroups + s);
    // its two problems: of the sequence, and of the prefix
    const int kv = head / p.G, g = head - kv * p.G, hb = g / p.heads, h = g - hb * p.heads;
    const int heads = kv * p.head_blocks + hb, all_heads = p.Hkv * p.head_blocks;
    const int2 *join_o = nullptr, *join_p = nullptr;
    Parts po{}, pp{};
    if (sp.tiles > 0) {
        const int b = t / p.toks_o;
        join_o = p.joins_o + (static_cast<long long>(s) * p.blocks_o + b) * all_heads + heads;
        po = Parts{make_int2(0, 0), (t - b * p.toks_o) * p.heads + h, p.rows_o};
    }
    if (sp.lo > 0) {
        const int2 range = group_range(p, share_of(p, s).g);
        const int at = tok - range.x * p.n, b = at / p.toks_p;
        join_p = p.joins_p + (static_cast<long long>(range.x) * p.blocks_p + b) * all_heads + heads;
        pp = Parts{make_int2(0, 0), (at - b * p.toks_p) * p.heads + h, p.rows_p};
    }
    // What is above runs beside the attention's end. Every thread waits for that end: what follows on the
    // stream waits for this kernel alone.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!in)
        return;
    uint2 *const out = reinterpret_cast<uint2 *>(p.o + static_cast<long long>(row) * D);
    const bool writes = SHARE == 1 || warp == 0;
    if (sp.hi == 0) {
        if (sp.bad) {
            if (lane == 0)
                atomicCAS(p.status, 0u, kBadSeqlens);
            return;
        }
        if (writes) {
            for (int i = 0; i < V; ++i)
                out[i * 32 + lane] = make_uint2(0u, 0u);
            if (lane == 0 && p.lse != nullptr)
                p.lse[row] = -INFINITY;
        }
        return;
    }
    if (join_o != nullptr)
        po.word = *join_o;
    if (join_p != nullptr)
        pp.word = *join_p;
    // written already; or a word was never written (a wait ran out, and the status says so)
    if (join_p == nullptr && po.word.y == 1)
        return;
    auto bad = [&](const int2 *join, int2 w) { return join != nullptr && (w.y < 1 || w.x < 0 || w.y > p.sms - w.x); };
    if (bad(join_o, po.word) || bad(join_p, pp.word))
        return;
    const int parts = pp.word.y + po.word.y;
    float mx = -INFINITY, sum = 0.f;
    float4 y[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    // 32 parts at a time: lane x has where part x is, its m and l
#pragma unroll 1
    for (int x0 = 0; x0 < parts; x0 += 32) {
        const int x = min(x0 + lane, parts - 1);
        const bool of_p = x < pp.word.y;
        const Parts &a = of_p ? pp : po;
        const int i = of_p ? x : x - pp.word.y;
        const float *at, *ml;
        int step;  // from m to l
        if (a.word.y == 1) {
            at = a.whole + static_cast<long long>(row) * D;
            ml = a.whole + static_cast<long long>(all) * D + 2LL * row;
            step = 1;
        } else {  // the first begins the problem (slot 1 of its run), the others continue it (slot 0)
            at = p.parts + (2 * (a.word.x + i) + (i == 0 ? 1 : 0)) * part_floats<D>(p.part_rows);
            ml = at + p.part_rows * D + a.row;
            at += a.row * D;
            step = p.part_rows;
        }
        const float m = ml[0], l = x0 + lane < parts ? ml[step] : 0.f;
        float top = m;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
        const float next = fmaxf(mx, top), by = mx == -INFINITY ? 0.f : fmaxf(ptx::ex2(mx - next), LEAST);
        mx = next;
        // 1: the part holds 0, or NaN
        const float w = (m == -INFINITY ? 1.f : fmaxf(ptx::ex2(m - mx), LEAST)) * l;
        float total = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            total += __shfl_xor_sync(FULL, total, d);
        sum = fmaf(sum, by, total);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            y[v].x *= by;
            y[v].y *= by;
            y[v].z *= by;
            y[v].w *= by;
        }
        const int n = min(32, parts - x0);
#pragma unroll 4
        for (int j = SHARE == 1 ? 0 : warp; j < n; j += SHARE) {
            const float f = __shfl_sync(FULL, w, j);
            const float4 *const src =
                reinterpret_cast<const float4 *>(__shfl_sync(FULL, reinterpret_cast<unsigned long long>(at), j)) + lane;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 z = src[32 * v];
                y[v].x = fmaf(f, z.x, y[v].x);
                y[v].y = fmaf(f, z.y, y[v].y);
                y[v].z = fmaf(f, z.z, y[v].z);
                y[v].w = fmaf(f, z.w, y[v].w);
            }
        }
    }
    if constexpr (SHARE > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            y_all[warp][v * 32 + lane] = y[v];
        __syncthreads();
        if (warp != 0)
            return;
#pragma unroll
        for (int w = 1; w < SHARE; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 z = y_all[w][v * 32 + lane];
                y[v].x += z.x;
                y[v].y += z.y;
                y[v].z += z.z;
                y[v].w += z.w;
            }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v)
        out[v * 32 + lane] = make_uint2(pack16<BF16>(y[v].x * inv, y[v].y * inv), pack16<BF16>(y[v].z * inv, y[v].w * inv));
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = sum == 0.f ? -INFINITY : (mx + ptx::lg2(sum)) * LN2;
}

}  // namespace sdp
