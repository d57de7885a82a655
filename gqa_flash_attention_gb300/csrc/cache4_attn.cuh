// Attention of each sequence's last n tokens over the paged 4-bit cache (sdp_fwd_cache4):
//
//     row i of sequence s is at position p = len_s - n + i and sees the keys j <= p, with a window
//     W > 0 only those with j > p - W or j < sinks;
//     O = softmax(scale * Q K^T) V over them, LSE = ln sum exp; a row that sees none: 0 and -inf.
//
// The G query heads of a KV head and the n rows are the columns of one problem per (sequence, KV
// head): 8 * NT columns a CTA, so that the codes are unpacked once for all of them.
//
// Bound: HBM, 4.5 bits a channel once per KV head. The tensor work is small but the codes have to
// pass through registers, so the kernel is built to keep the instructions per code few:
//
//   K: value = s n + b per (token, 64 channels), so the score of a group is
//        s * sum_c q_c n_c + b * sum_c q_c.
//      Codes enter the MMA as they are: two of a 32-bit word (channels c and c + 4: any pairing
//      will do, the queries are laid out to match) become a register by one shift and one and/or.
//      bf16: 0x4300 | n is 128 + n exactly; the 128 is taken out with b (b - 128 s). fp16: n in
//      the low bits is the subnormal n * 2^-24 exactly; s takes the 2^24.
//   V: with the group's s folded into the weights, sum_t (p_t s_t) (n_tc - 8) + sum_t p_t (b_t + 8 s_t).
//      n - 8 in bf16 is 128 + n less 136, exactly: O is a sum of many small terms of both signs, and
//      with the 128 left in (and taken out at the end, as for a score) it lost up to 7e-3 of O over
//      32768 keys. p_t s_t as two bf16 (high part and remainder, 2^-17 relative: fp16's range would
//      not hold p s, and one bf16 would cost more than the output's rounding) in two MMAs.
//   S = K Q^T with 16 tokens by 8 columns (m16n8k16), O = V^T P with 16 channels by 8 columns:
//   few columns fill the n side. p turns from S's layout (token rows) to P's (column rows) by
//   movmatrix on the two halves of its 32 bits.
//
// Each warp streams 32-token tiles through a ring of its own (bulk copies of the codes' and scales'
// contiguous runs, NSTAGE tiles in flight, one mbarrier a stage; no barrier with other warps) and
// keeps its own running maximum, sum and O in registers. The maximum moves only when a score
// exceeds it by more than 8 (base 2), found by a vote, so most tiles need no reduction.
//
// Work split: all sequences' tiles are numbered sequence by sequence, KV head by KV head, and cut
// into equal runs, one a CTA (the lengths are on the device, so each CTA finds its run from them);
// a run's tiles of one (sequence, KV head) go round the CTA's warps and their states are joined
// through shared memory. A problem that lies in one CTA's run is written directly; the parts of
// the others go to the workspace in fp32 and cache4_merge_kernel joins them in a fixed order.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cache4.cuh"
#include "ptx.cuh"
#include "sdp_launch.h"
#include "sixteen.cuh"

namespace sdp {

struct Cache4AttnParams {
    const uint16_t *q;
    uint16_t *o;
    float *lse;
    const uint8_t *k_codes, *v_codes;
    const uint32_t *k_scales, *v_scales;
    const int *table, *lens;
    float *workspace;
    unsigned int *status;
    unsigned long long timeout_ns;
    long long table_stride;
    int num_pages, page_size, max_pages;
    int nseq, n, Hq, Hkv, G;
    int window, sinks;  // window 0: every key
    int chunks;         // column chunks of 8 * NT
    int ctas;           // CTAs that share the tiles (the merge sees the same number)
    int no_copies;      // test hook: no copy is issued, every wait runs out
    float c;            // scale * log2(e)
};

namespace c4 {

constexpr int TILE = 32;  // tokens a warp step
constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr unsigned FULL = 0xffffffffu;
constexpr float RESCALE = 8.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr unsigned kSlotNeverFilled = 3;  // the status word's site of a load that did not land

// Which tiles of a sequence its rows see: the sinks' tiles, then those from the first row's
// window start to the end.
struct Span {
    int len;       // valid length, 0 for an empty or a bad one
    int t_lo, ns;  // first tile of the window, tiles of the sinks before it
    int count;
    bool bad;
    __device__ __forceinline__ int tile(int e) const { return e < ns ? e : t_lo + e - ns; }
};

__device__ __forceinline__ Span span_of(const Cache4AttnParams &p, int s)
{
    Span r;
    const int len = __ldg(p.lens + s);
    r.bad = len < 0 || len > p.max_pages * p.page_size;  // the host keeps the product in 31 bits
    r.len = r.bad ? 0 : len;
    const long long lo = p.window > 0 ? static_cast<long long>(r.len) - p.n - p.window + 1 : 0;
    r.t_lo = lo > 0 ? static_cast<int>(lo / TILE) : 0;
    const int sinks = p.window > 0 ? min(p.sinks, r.len) : 0;
    r.ns = min(sinks / TILE + (sinks % TILE != 0), r.t_lo);
    r.count = r.len > 0 ? r.ns + (r.len + TILE - 1) / TILE - r.t_lo : 0;
    return r;
}

// Block-wide: the number of tiles of all problems (returned), and where the one numbered at(total)
// lies: its sequence and its place among the sequence's tiles. scratch: WARPS + 2 words.
template <class At>
__device__ __forceinline__ long long find_place(const Cache4AttnParams &p, int per_tile, long long *scratch, At &&at,
                                                int *s_out, long long *off_out)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.nseq + THREADS - 1) / THREADS;
    const long long first = static_cast<long long>(tid) * per;
    const int s0 = static_cast<int>(min(static_cast<long long>(p.nseq), first));
    const int s1 = static_cast<int>(min(static_cast<long long>(p.nseq), first + per));
    long long sum = 0;
    for (int s = s0; s < s1; ++s)
        sum += span_of(p, s).count;
    sum *= per_tile;
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(FULL, incl, d);
        if (lane >= d)
            incl += x;
    }
    if (lane == 31)
        scratch[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp)
            before += scratch[w];
        total += scratch[w];
    }
    incl += before;
    long long excl = incl - sum;
    const long long x = at(total);
    if (x >= excl && x < incl) {
        for (int s = s0; s < s1; ++s) {
            const long long n = static_cast<long long>(span_of(p, s).count) * per_tile;
            if (x < excl + n) {
                scratch[WARPS] = s;
                scratch[WARPS + 1] = x - excl;
                break;
            }
            excl += n;
        }
    }
    __syncthreads();
    *s_out = static_cast<int>(scratch[WARPS]);
    *off_out = scratch[WARPS + 1];
    return total;
}

// First tile of CTA i's run.
__device__ __forceinline__ long long run_start(long long total, int i, int n) { return total * i / n; }

// CTAs with work: every one of them has at least a tile.
__device__ __forceinline__ int busy_ctas(const Cache4AttnParams &p, long long total)
{
    return total < p.ctas ? static_cast<int>(total) : p.ctas;
}

// Floats of one part in the workspace: O [columns][D], then m and l of each column.
template <int D, int NT>
__host__ __device__ constexpr int part_floats()
{
    return 8 * NT * (D + 2);
}

template <int D, int NT>
struct Smem {
    static constexpr int GQ = D / kCacheGroup;
    static constexpr int CODE = TILE * D / 2;    // bytes of a tile's K (or V) codes
    static constexpr int SCALE = TILE * GQ * 4;  // and of its scales
    static constexpr int STAGE = 2 * (CODE + SCALE);
    static constexpr int NSTAGE = D == 128 ? 4 : 2;
    static constexpr int COLS = 8 * NT;
    static constexpr int O_SLOT = COLS * D * 4;
    static constexpr int O_SLOTS = WARPS / 2;
    static constexpr int QF = (D / 16) * NT * 32 * 8;
    static constexpr int RING = 0;
    static constexpr int O_BUF = RING + WARPS * NSTAGE * STAGE;
    static constexpr int Q_FRAG = O_BUF + O_SLOTS * O_SLOT;
    static constexpr int QSUM = Q_FRAG + QF;         // [GQ][COLS] floats
    static constexpr int ML = QSUM + GQ * COLS * 4;  // [2][WARPS][COLS] floats
    static constexpr int SCRATCH = ML + 2 * WARPS * COLS * 4;
    static constexpr int BARS = SCRATCH + 8 * (WARPS + 4);
    static constexpr int FLAG = BARS + 8 * WARPS * NSTAGE;
    static constexpr int BYTES = FLAG + 16;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static_assert(STAGE % 128 == 0 && O_BUF % 16 == 0 && Q_FRAG % 16 == 0 && SCRATCH % 8 == 0, "alignment");
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Codes i of the two 16-bit halves of w as a pair of 16-bit floats (128 + n in bf16; the fp16
// subnormal n * 2^-24 with magic 0).
template <uint32_t MAGIC>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i)
{
    return ((w >> (4 * i)) & 0x000f000fu) | MAGIC;
}

// The same pair as bf16 n - 8.
__device__ __forceinline__ uint32_t centred_pair(uint32_t w, int i)
{
    const uint32_t u = code_pair<0x43004300u>(w, i);
    const uint32_t c = 0x43084308u;  // 136
    __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u), *reinterpret_cast<const __nv_bfloat162 *>(&c));
    return *reinterpret_cast<uint32_t *>(&d);
}

__device__ __forceinline__ float scale_of(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float bias_of(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) that completes on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}

// A walk over a CTA's run, segment by segment (the run's tiles of one problem).
struct Walk {
    Span sp;
    int s, u;             // sequence; problem in it: KV head * chunks + chunk
    int e0, e1;           // tiles [e0, e1) of the problem
    long long off, left;  // position in the sequence's tiles, tiles left in the run
    __device__ __forceinline__ void segment(const Cache4AttnParams &p)
    {
        // empty sequences are passed over; `left` counts tiles that exist, so one follows
        while (off >= static_cast<long long>(sp.count) * p.Hkv * p.chunks) {
            off = 0;
            sp = span_of(p, ++s);
        }
        u = static_cast<int>(off / sp.count);
        e0 = static_cast<int>(off - static_cast<long long>(u) * sp.count);
        e1 = static_cast<int>(min(static_cast<long long>(sp.count), e0 + left));
    }
    __device__ __forceinline__ void start(const Cache4AttnParams &p, int s_, long long off_, long long left_)
    {
        s = s_;
        off = off_;
        left = left_;
        sp = span_of(p, s);
        if (left > 0)
            segment(p);
    }
    __device__ __forceinline__ void next(const Cache4AttnParams &p)
    {
        off += e1 - e0;
        left -= e1 - e0;
        if (left > 0)
            segment(p);
    }
};

// Waits up to the limit for the phase of `bar`; false when it ran out.
static __device__ __noinline__ bool wait_stage_slow(uint32_t bar, uint32_t parity, unsigned long long timeout_ns)
{
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer_ns() - t0 > timeout_ns)
            return false;
    return true;
}

__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, unsigned long long timeout_ns)
{
    return ptx::mbar_try_wait(bar, parity) || wait_stage_slow(bar, parity, timeout_ns);
}

}  // namespace c4

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(c4::THREADS, 1) cache4_attn_kernel(const Cache4AttnParams p)
{
    using namespace c4;
    using M = Smem<D, NT>;
    constexpr int GQ = M::GQ, COLS = M::COLS;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row8 = lane >> 2, quad = lane & 3;  // an MMA fragment's row (or column n) and place in it
    volatile int *failed = reinterpret_cast<volatile int *>(smem + M::FLAG);
    long long *scratch = reinterpret_cast<long long *>(smem + M::SCRATCH);
    float *qsum = reinterpret_cast<float *>(smem + M::QSUM);
    float *m_all = reinterpret_cast<float *>(smem + M::ML), *l_all = m_all + WARPS * COLS;
    const uint32_t ring = sbase + M::RING + warp * M::NSTAGE * M::STAGE;
    const uint8_t *ring_p = smem + M::RING + warp * M::NSTAGE * M::STAGE;
    const uint32_t bars = sbase + M::BARS + 8 * warp * M::NSTAGE;

    if (tid == 0)
        *failed = 0;
    if (lane == 0) {
        for (int i = 0; i < M::NSTAGE; ++i)
            ptx::mbar_init(bars + 8 * i, 1);
        ptx::fence_barrier_init();
    }
    // where this CTA's run of tiles starts
    int s_first = 0;
    long long off_first = 0;
    const int per_tile = p.Hkv * p.chunks;
    const long long total = find_place(
        p, per_tile, scratch,
        [&](long long t) -> long long {
            const int n = busy_ctas(p, t);
            return static_cast<int>(blockIdx.x) < n ? run_start(t, blockIdx.x, n) : -1;
        },
        &s_first, &off_first);
    const int busy = busy_ctas(p, total);
    if (static_cast<int>(blockIdx.x) >= busy)
        return;
    const long long run0 = run_start(total, blockIdx.x, busy);
    const long long run_len = run_start(total, blockIdx.x + 1, busy) - run0;

    // ---- copies: tile e of the walk's segment into stage `st`
    auto issue = [&](const Walk &w, int e, int st) {
        if (p.no_copies)
            return;
        const uint32_t bar = bars + 8 * st;
        if (lane == 0)
            expect_tx(bar, M::STAGE);
        __syncwarp();
        const int g = w.u / p.chunks;
        const int tok0 = w.sp.tile(e) * TILE;
        // a 32-token tile lies in one page where the page size is a multiple of 32, else in halves
        const int pieces = (p.page_size & 31) == 0 ? 1 : 2;
        if (lane < 4 * pieces) {
            const int part = lane & 3, half = lane >> 2;  // K codes, K scales, V codes, V scales
            const int tokens = TILE / pieces;
            const int tok = tok0 + half * tokens;
            const int slot = tok / p.page_size;
            // a half behind the last page is copied from that page and masked
            const int last = (w.sp.len - 1) / p.page_size;
            int id = __ldg(p.table + w.s * p.table_stride + min(slot, last));
            if (id < 0 || id >= p.num_pages) {
                atomicCAS(p.status, 0u, kBadPages);
                id = 0;
            }
            const long long row = (static_cast<long long>(id) * p.Hkv + g) * p.page_size + (tok - slot * p.page_size);
            const uint32_t base = ring + st * M::STAGE + (part >= 2 ? M::CODE + M::SCALE : 0);
            if (part & 1)
                bulk_load(base + M::CODE + half * tokens * GQ * 4, (part == 1 ? p.k_scales : p.v_scales) + row * GQ,
                          tokens * GQ * 4, bar);
            else
                bulk_load(base + half * tokens * (D / 2), (part == 0 ? p.k_codes : p.v_codes) + row * (D / 2),
                          tokens * (D / 2), bar);
        }
    };

    Walk ahead;  // the copies' place in the run
    ahead.start(p, s_first, off_first, run_len);
    int ae = ahead.e0 + warp;  // this warp's next tile to copy
    auto next_ahead = [&]() -> bool {  // moves to a segment with a tile of this warp's
        while (ahead.left > 0 && ae >= ahead.e1) {
            ahead.next(p);
            ae = ahead.e0 + warp;
        }
        return ahead.left > 0;
    };
    int in_flight = 0;
    for (; in_flight < M::NSTAGE && next_ahead(); ++in_flight) {
        issue(ahead, ae, in_flight);
        ae += WARPS;
    }
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto step_stage = [&]() {
        if (++stage == M::NSTAGE) {
            stage = 0;
            phase ^= 1u;
        }
    };

    Walk w;
    w.start(p, s_first, off_first, run_len);
    while (w.left > 0) {
        const int g = w.u / p.chunks, chunk = w.u - g * p.chunks;
        const int r_base = chunk * COLS, R = p.n * p.G;
        auto row_of = [&](int r) {  // the (sequence, row, head) row of column r in q, o and lse
            return (static_cast<long long>(w.s) * p.n + r / p.G) * p.Hq + g * p.G + r % p.G;
        };
        // ---- the queries as B fragments, and their sums over each group
        {
            uint2 *qf = reinterpret_cast<uint2 *>(smem + M::Q_FRAG);
            for (int i = tid; i < (D / 16) * NT * 32; i += THREADS) {
                const int ks = i / (NT * 32), nt = (i / 32) % NT, l = i & 31;
                const int r = r_base + nt * 8 + (l >> 2);
                uint2 f = make_uint2(0u, 0u);
                if (r < R) {
                    const int c0 = (ks / 4) * kCacheGroup + (l & 3) * 16 + ((ks & 3) / 2) * 8 + 2 * (ks & 1);
                    const uint16_t *src = p.q + row_of(r) * D + c0;
                    f.x = __ldg(src) | (static_cast<uint32_t>(__ldg(src + 4)) << 16);
                    f.y = __ldg(src + 1) | (static_cast<uint32_t>(__ldg(src + 5)) << 16);
                }
                qf[i] = f;
            }
            for (int i = warp; i < COLS * GQ; i += WARPS) {
                const int col = i / GQ, gq = i - col * GQ, r = r_base + col;
                float v = 0.f;
                if (r < R) {
                    const float2 x = unpack16<BF16>(__ldg(
                        reinterpret_cast<const uint32_t *>(p.q + row_of(r) * D + gq * kCacheGroup + 2 * lane)));
                    v = x.x + x.y;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    v += __shfl_xor_sync(FULL, v, o);
                if (lane == 0)
                    qsum[gq * COLS + col] = v;
            }
        }
        __syncthreads();

        float o[D / 16][NT][4], m[NT][2], l[NT][2], corr[NT][GQ];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int gq = 0; gq < GQ; ++gq)
                corr[nt][gq] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
        }
        // positions of the chunk's first and last column
        const int pos_lo = w.sp.len - p.n + r_base / p.G;
        const int pos_hi = w.sp.len - p.n + min(p.n - 1, (r_base + COLS - 1) / p.G);

        for (int e = w.e0 + warp; e < w.e1; e += WARPS) {
            if (ok && !__all_sync(FULL, wait_stage(bars + 8 * stage, phase, p.timeout_ns))) {
                ok = false;
                *failed = 1;
                if (lane == 0)
                    atomicCAS(p.status, 0u, kSlotNeverFilled | (blockIdx.x << 8));
                // this warp's copies land (waited for with a limit again) before the CTA may exit
                for (; in_flight > 0 && !p.no_copies; --in_flight) {
                    wait_stage(bars + 8 * stage, phase, p.timeout_ns);
                    step_stage();
                }
            }
            if (!ok)
                continue;
            const uint8_t *kc = ring_p + stage * M::STAGE, *vc = kc + M::CODE + M::SCALE;
            const uint32_t *ksc = reinterpret_cast<const uint32_t *>(kc + M::CODE);
            const uint32_t *vsc = reinterpret_cast<const uint32_t *>(vc + M::CODE);
            const uint2 *qf = reinterpret_cast<const uint2 *>(smem + M::Q_FRAG);
            const int tok0 = w.sp.tile(e) * TILE;
            const bool whole = tok0 + TILE - 1 <= pos_lo &&
                               (p.window == 0 || tok0 > pos_hi - p.window || tok0 + TILE <= p.sinks);
            // MMA row r (and r + 8) of a 16-token chunk is token ta (and ta + 8), so that P's
            // rows 2 quad, 2 quad + 1, 2 quad + 8, 2 quad + 9 are tokens quad + {0, 4, 8, 12}
            const int ta = (row8 >> 1) + ((row8 & 1) << 2);

            // ---- scores
            float s[2][NT][4];
#pragma unroll
            for (int mc = 0; mc < 2; ++mc)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[mc][nt][0] = s[mc][nt][1] = s[mc][nt][2] = s[mc][nt][3] = 0.f;
#pragma unroll
            for (int gq = 0; gq < GQ; ++gq) {
                float acc[2][NT][4];
                uint2 wa[2], wb[2];
#pragma unroll
                for (int mc = 0; mc < 2; ++mc) {
                    const uint8_t *at = kc + (mc * 16 + ta) * (D / 2) + gq * 32 + quad * 8;
                    wa[mc] = *reinterpret_cast<const uint2 *>(at);
                    wb[mc] = *reinterpret_cast<const uint2 *>(at + 8 * (D / 2));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        acc[mc][nt][0] = acc[mc][nt][1] = acc[mc][nt][2] = acc[mc][nt][3] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint2 b[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        b[nt] = qf[((gq * 4 + j) * NT + nt) * 32 + lane];
#pragma unroll
                    for (int mc = 0; mc < 2; ++mc) {
                        const uint32_t x = j < 2 ? wa[mc].x : wa[mc].y, y = j < 2 ? wb[mc].x : wb[mc].y;
                        constexpr uint32_t MAGIC = BF16 ? 0x43004300u : 0u;
                        const int h = 2 * (j & 1);
                        const uint32_t a0 = code_pair<MAGIC>(x, h), a1 = code_pair<MAGIC>(y, h);
                        const uint32_t a2 = code_pair<MAGIC>(x, h + 1), a3 = code_pair<MAGIC>(y, h + 1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (BF16)
                                mma_bf16(acc[mc][nt], a0, a1, a2, a3, b[nt].x, b[nt].y);
                            else
                                mma_f16(acc[mc][nt], a0, a1, a2, a3, b[nt].x, b[nt].y);
                        }
                    }
                }
#pragma unroll
                for (int mc = 0; mc < 2; ++mc) {
                    const uint32_t pa = ksc[(mc * 16 + ta) * GQ + gq], pb = ksc[(mc * 16 + ta + 8) * GQ + gq];
                    float sa = scale_of(pa), ba = bias_of(pa), sb = scale_of(pb), bb = bias_of(pb);
                    if constexpr (BF16) {
                        ba = fmaf(-128.f, sa, ba);
                        bb = fmaf(-128.f, sb, bb);
                    } else {
                        sa *= 16777216.f;  // 2^24
                        sb *= 16777216.f;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 qs = *reinterpret_cast<const float2 *>(qsum + gq * COLS + nt * 8 + 2 * quad);
                        float(&d)[4] = s[mc][nt];
                        d[0] = fmaf(sa, acc[mc][nt][0], fmaf(ba, qs.x, d[0]));
                        d[1] = fmaf(sa, acc[mc][nt][1], fmaf(ba, qs.y, d[1]));
                        d[2] = fmaf(sb, acc[mc][nt][2], fmaf(bb, qs.x, d[2]));
                        d[3] = fmaf(sb, acc[mc][nt][3], fmaf(bb, qs.y, d[3]));
                    }
                }
            }
            // ---- base-2 scores; keys a column does not see drop out
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mc = 0; mc < 2; ++mc)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[mc][nt][i] *= p.c;
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = r_base + nt * 8 + 2 * quad + i;
                        const int at = w.sp.len - p.n + min(p.n - 1, r / p.G);
                        const int from = p.window > 0 ? at - p.window : -1;  // keys past it are in the window
#pragma unroll
                        for (int mc = 0; mc < 2; ++mc)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int j = tok0 + mc * 16 + ta + 8 * x;
                                if (j > at || (j <= from && j >= p.sinks))
                                    s[mc][nt][i + 2 * x] = -INFINITY;
                            }
                    }
                }
            }
            // ---- running maximum: moved when some score is more than RESCALE above it
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    over |= fmaxf(fmaxf(s[0][nt][i], s[0][nt][i + 2]), fmaxf(s[1][nt][i], s[1][nt][i + 2])) >
                            m[nt][i] + RESCALE;
            if (__any_sync(FULL, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float a[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(fmaxf(s[0][nt][i], s[0][nt][i + 2]), fmaxf(s[1][nt][i], s[1][nt][i + 2]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            x = fmaxf(x, __shfl_xor_sync(FULL, x, off));
                        const float next = fmaxf(m[nt][i], x);
                        a[i] = next == m[nt][i] ? 1.f : ptx::ex2(m[nt][i] - next);
                        m[nt][i] = next;
                        l[nt][i] *= a[i];
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[i][nt][0] *= a[0];
                        o[i][nt][1] *= a[1];
                        o[i][nt][2] *= a[0];
                        o[i][nt][3] *= a[1];
                    }
                    // corr belongs to column row8, whose factor lanes with quad = row8 / 2 hold
                    const float x0 = __shfl_sync(FULL, a[0], row8 >> 1), x1 = __shfl_sync(FULL, a[1], row8 >> 1);
                    const float f = (row8 & 1) ? x1 : x0;
#pragma unroll
                    for (int gq = 0; gq < GQ; ++gq)
                        corr[nt][gq] *= f;
                }
            }
            // ---- weights, and their turn into P's layout
            float pb[2][NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
                const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                for (int mc = 0; mc < 2; ++mc) {
                    const float p0 = ptx::ex2(s[mc][nt][0] - m0), p1 = ptx::ex2(s[mc][nt][1] - m1);
                    const float p2 = ptx::ex2(s[mc][nt][2] - m0), p3 = ptx::ex2(s[mc][nt][3] - m1);
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                    const uint32_t u2 = __float_as_uint(p2), u3 = __float_as_uint(p3);
                    const uint32_t l0 = movmatrix(__byte_perm(u0, u1, 0x5410));
                    const uint32_t h0 = movmatrix(__byte_perm(u0, u1, 0x7632));
                    const uint32_t l1 = movmatrix(__byte_perm(u2, u3, 0x5410));
                    const uint32_t h1 = movmatrix(__byte_perm(u2, u3, 0x7632));
                    pb[mc][nt][0] = __uint_as_float(__byte_perm(l0, h0, 0x5410));
                    pb[mc][nt][1] = __uint_as_float(__byte_perm(l0, h0, 0x7632));
                    pb[mc][nt][2] = __uint_as_float(__byte_perm(l1, h1, 0x5410));
                    pb[mc][nt][3] = __uint_as_float(__byte_perm(l1, h1, 0x7632));
                }
            }
            // ---- O += V^T P
#pragma unroll
            for (int mc = 0; mc < 2; ++mc) {
#pragma unroll
                for (int gq = 0; gq < GQ; ++gq) {
                    uint32_t v[4];
                    float sc[4], bi[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = mc * 16 + quad + 4 * i;
                        v[i] = *reinterpret_cast<const uint32_t *>(vc + t * (D / 2) + gq * 32 + row8 * 4);
                        const uint32_t pr = vsc[t * GQ + gq];
                        sc[i] = scale_of(pr);
                        bi[i] = fmaf(8.f, sc[i], bias_of(pr));
                    }
                    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float pi = pb[mc][nt][i];
                            // a key that no column sees has weight 0, whatever its place in the pool holds
                            const bool out = !whole && pi == 0.f;
                            x[i] = out ? 0.f : pi * sc[i];
                            corr[nt][gq] = out ? corr[nt][gq] : fmaf(pi, bi[i], corr[nt][gq]);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            hi[nt][i] = pack16<true>(x[2 * i], x[2 * i + 1]);
                            lo[nt][i] = pack16<true>(x[2 * i] - __uint_as_float(hi[nt][i] << 16),
                                                     x[2 * i + 1] - __uint_as_float(hi[nt][i] & 0xffff0000u));
                        }
                    }
                    // halves of the words: codes 0-3 of two tokens, codes 4-7 of two tokens
                    const uint32_t x01 = __byte_perm(v[0], v[1], 0x5410), y01 = __byte_perm(v[0], v[1], 0x7632);
                    const uint32_t x23 = __byte_perm(v[2], v[3], 0x5410), y23 = __byte_perm(v[2], v[3], 0x7632);
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        const uint32_t w01 = mt < 2 ? x01 : y01, w23 = mt < 2 ? x23 : y23;
                        const int h = 2 * (mt & 1);
                        const uint32_t a0 = centred_pair(w01, h), a1 = centred_pair(w01, h + 1);
                        const uint32_t a2 = centred_pair(w23, h), a3 = centred_pair(w23, h + 1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_bf16(o[gq * 4 + mt][nt], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
                            mma_bf16(o[gq * 4 + mt][nt], a0, a1, a2, a3, lo[nt][0], lo[nt][1]);
                        }
                    }
                }
            }
            // ---- the stage is free: its next tile
            __syncwarp();
            if (next_ahead()) {
                issue(ahead, ae, stage);
                ae += WARPS;
            } else {
                --in_flight;
            }
            step_stage();
        }

        // ---- join the warps: maximum and sum of each column, then O
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][i] += __shfl_xor_sync(FULL, l[nt][i], off);
                if (row8 == 0) {
                    m_all[warp * COLS + nt * 8 + 2 * quad + i] = m[nt][i];
                    l_all[warp * COLS + nt * 8 + 2 * quad + i] = l[nt][i];
                }
            }
        __syncthreads();
        const int parts = min(WARPS, w.e1 - w.e0);  // warps that had a tile
        float *obuf = reinterpret_cast<float *>(smem + M::O_BUF);
        if (warp < parts) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2], cg[GQ][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = -INFINITY;
                    for (int x = 0; x < parts; ++x)
                        mx = fmaxf(mx, m_all[x * COLS + nt * 8 + 2 * quad + i]);
                    f[i] = m[nt][i] == -INFINITY ? 0.f : ptx::ex2(m[nt][i] - mx);
                }
#pragma unroll
                for (int gq = 0; gq < GQ; ++gq) {
                    float c = corr[nt][gq];
                    c += __shfl_xor_sync(FULL, c, 1);
                    c += __shfl_xor_sync(FULL, c, 2);
                    cg[gq][0] = __shfl_sync(FULL, c, 8 * quad);      // column 2 quad
                    cg[gq][1] = __shfl_sync(FULL, c, 8 * quad + 4);  // column 2 quad + 1
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        o[i][nt][x] = (o[i][nt][x] + cg[i / 4][x & 1]) * f[x & 1];
            }
            if (warp >= M::O_SLOTS) {
                float *dst = obuf + (warp - M::O_SLOTS) * COLS * D;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            dst[((i * NT + nt) * 4 + x) * 32 + lane] = o[i][nt][x];
            }
        }
        if (parts > M::O_SLOTS)
            __syncthreads();
        if (warp < M::O_SLOTS && warp < parts) {
            float *dst = obuf + warp * COLS * D;
            const bool more = warp + M::O_SLOTS < parts;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float *at = dst + ((i * NT + nt) * 4 + x) * 32 + lane;
                        *at = more ? o[i][nt][x] + *at : o[i][nt][x];
                    }
        }
        __syncthreads();
        // ---- sum over the slots; eight channels of a column a thread
        {
            const long long unit0 = run0 + (run_len - w.left) - w.e0;  // the problem's first tile among all
            const bool direct = w.e0 == 0 && w.e1 == w.sp.count;
            // a part that continues a problem is this CTA's first segment, one that begins it its last
            const int slot = unit0 < run0 ? 0 : 1;
            float *part = p.workspace + (static_cast<long long>(blockIdx.x) * 2 + slot) * part_floats<D, NT>();
            const int slots = min(parts, M::O_SLOTS);
            for (int it = tid; it < GQ * NT * 64; it += THREADS) {
                const int ln = it & 31, par = (it >> 5) & 1, nt = (it >> 6) % NT, gq = it / (64 * NT);
                const int col = nt * 8 + 2 * (ln & 3) + par, r = r_base + col;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = 0.f;
                for (int sl = 0; sl < slots; ++sl) {
                    const float *src = obuf + sl * COLS * D + ln;
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            y[2 * mt + x] += src[(((gq * 4 + mt) * NT + nt) * 4 + 2 * x + par) * 32];
                }
                if (r >= R || *failed)
                    continue;
                float mx = -INFINITY, sum = 0.f;
                for (int x = 0; x < parts; ++x)
                    mx = fmaxf(mx, m_all[x * COLS + col]);
                for (int x = 0; x < parts; ++x) {
                    const float mw = m_all[x * COLS + col];
                    // a warp whose keys were all out of sight holds 0 (or, after a NaN score, NaN)
                    sum += l_all[x * COLS + col] * (mw == -INFINITY ? 1.f : ptx::ex2(mw - mx));
                }
                const int c0 = gq * kCacheGroup + (ln >> 2) * 8;
                if (direct) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees no key: 0 and -inf
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] *= inv;
                    *reinterpret_cast<uint4 *>(p.o + row_of(r) * D + c0) = pack8<BF16>(y);
                    if (c0 == 0 && p.lse != nullptr)
                        p.lse[row_of(r)] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(part + col * D + c0);
                    dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                    dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                    if (c0 == 0) {
                        part[COLS * D + col] = mx;
                        part[COLS * D + COLS + col] = sum;
                    }
                }
            }
        }
        __syncthreads();  // the buffers serve the next segment
        w.next(p);
    }
}

// Joins the parts of every problem that more than one CTA worked on, in the order of the CTAs, and
// writes the rows of empty sequences. One block a problem, one warp a column.
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(c4::THREADS) cache4_merge_kernel(const Cache4AttnParams p)
{
    using namespace c4;
    constexpr int COLS = 8 * NT, V = D / 32;
    __shared__ long long both[2][WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_seq = p.Hkv * p.chunks;
    const int s = blockIdx.x / per_seq, u = blockIdx.x - s * per_seq;
    const int g = u / p.chunks, chunk = u - g * p.chunks;
    const Span sp = span_of(p, s);
    const int R = p.n * p.G, r_base = chunk * COLS;
    auto row_of = [&](int r) { return (static_cast<long long>(s) * p.n + r / p.G) * p.Hq + g * p.G + r % p.G; };
    if (sp.count == 0) {
        if (sp.bad) {
            if (threadIdx.x == 0)
                atomicCAS(p.status, 0u, kBadSeqlens);
            return;
        }
        for (int col = warp; col < COLS && r_base + col < R; col += WARPS) {
            const long long row = row_of(r_base + col);
            for (int i = lane; i < D / 8; i += 32)
                reinterpret_cast<uint4 *>(p.o + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (lane == 0 && p.lse != nullptr)
                p.lse[row] = -INFINITY;
        }
        return;
    }
    // tiles before this sequence, and in all
    long long before = 0, total = 0;
    {
        long long a = 0, t = 0;
        for (int i = threadIdx.x; i < p.nseq; i += THREADS) {
            const long long n = span_of(p, i).count;
            t += n;
            a += i < s ? n : 0;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            a += __shfl_xor_sync(FULL, a, off);
            t += __shfl_xor_sync(FULL, t, off);
        }
        if (lane == 0) {
            both[0][warp] = a;
            both[1][warp] = t;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            before += both[0][i];
            total += both[1][i];
        }
    }
    before *= per_seq;
    total *= per_seq;
    const long long u0 = before + static_cast<long long>(u) * sp.count, u1 = u0 + sp.count;
    const int busy = busy_ctas(p, total);
    // the CTA whose run holds tile x: the largest i with run_start(i) <= x
    const int i0 = static_cast<int>(((u0 + 1) * busy - 1) / total), i1 = static_cast<int>((u1 * busy - 1) / total);
    if (i0 == i1)
        return;  // written by the CTA itself
    constexpr int PART = part_floats<D, NT>();
    // part x (CTA i0 + x): the first begins the problem (slot 1), the others continue it (slot 0)
    auto part = [&](int x) { return p.workspace + (2LL * (i0 + x) + (x == 0 ? 1 : 0)) * PART; };
    const int parts = i1 - i0 + 1;
    for (int col = warp; col < COLS && r_base + col < R; col += WARPS) {
        float mx = -INFINITY;
        for (int x = lane; x < parts; x += 32)
            mx = fmaxf(mx, part(x)[COLS * D + col]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
        float sum = 0.f, y[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            y[i] = 0.f;
        for (int x0 = 0; x0 < parts; x0 += 32) {
            float f = 0.f;
            if (x0 + lane < parts) {
                const float mw = part(x0 + lane)[COLS * D + col];
                f = mw == -INFINITY ? 1.f : ptx::ex2(mw - mx);  // 1: the part holds 0, or NaN
                sum += f * part(x0 + lane)[COLS * D + COLS + col];
            }
            const int end = min(32, parts - x0);
#pragma unroll 4
            for (int x = 0; x < end; ++x) {
                const float fx = __shfl_sync(FULL, f, x);
                const float4 *src = reinterpret_cast<const float4 *>(part(x0 + x) + col * D) + lane * (V / 4);
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    const float4 t = src[i];
                    y[4 * i] = fmaf(fx, t.x, y[4 * i]);
                    y[4 * i + 1] = fmaf(fx, t.y, y[4 * i + 1]);
                    y[4 * i + 2] = fmaf(fx, t.z, y[4 * i + 2]);
                    y[4 * i + 3] = fmaf(fx, t.w, y[4 * i + 3]);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            sum += __shfl_xor_sync(FULL, sum, off);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long row = row_of(r_base + col);
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + row * D) + lane * (V / 2);
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            dst[i] = pack16<BF16>(y[2 * i] * inv, y[2 * i + 1] * inv);
        if (lane == 0 && p.lse != nullptr)
            p.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
}

template <int D, bool BF16, int NT>
cudaError_t launch_cache4_attn(const Cache4AttnParams &p, cudaStream_t st)
{
    using M = c4::Smem<D, NT>;
    static unsigned long long done = 0;
    auto kern = cache4_attn_kernel<D, BF16, NT>;
    cudaError_t e = set_smem_once(kern, M::BYTES, done);
    if (e != cudaSuccess)
        return e;
    kern<<<p.ctas, c4::THREADS, M::BYTES, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    cache4_merge_kernel<D, BF16, NT><<<p.nseq * p.Hkv * p.chunks, c4::THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

// One per (head dim, dtype): 8 or, wide, 16 columns a CTA.
cudaError_t cache4_attn_d128_fp16(const Cache4AttnParams &p, bool wide, cudaStream_t st);
cudaError_t cache4_attn_d128_bf16(const Cache4AttnParams &p, bool wide, cudaStream_t st);
cudaError_t cache4_attn_d256_fp16(const Cache4AttnParams &p, bool wide, cudaStream_t st);
cudaError_t cache4_attn_d256_bf16(const Cache4AttnParams &p, bool wide, cudaStream_t st);

}  // namespace sdp
