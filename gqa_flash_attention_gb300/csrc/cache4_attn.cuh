// Attention of each sequence's last n tokens over the paged 4-bit cache (sdp_fwd_cache4):
//
//     row i of sequence s is at position p = len_s - n + i and sees the keys j <= p, with a window
//     W > 0 only those with j > p - W or j < sinks;
//     O = softmax(scale * Q K^T) V over them, LSE = ln sum exp; a row that sees none: 0 and -inf.
//
// The G query heads of a KV head and the n rows are the columns of one problem per (sequence, KV
// head): 8 * NT columns a warp, so that the codes are unpacked once for all of them.
//
// Bound: HBM, 4.5 bits a channel once per KV head. The tensor work is small, but the codes have to
// pass through registers, so the kernel is built to keep the instructions per code few. Both
// products run in fp16 whatever the type of q, because a code needs no arithmetic to be an fp16
// number: two codes of a 32-bit word (channels c and c + 4: any pairing will do, the queries and
// the output are laid out to match) are the subnormals n * 2^-24 after one "and", or n * 2^-20
// where they lie four bits up, so eight codes take one shift and four "and"s. (bf16 has only seven
// bits below its exponent: 128 + n took a shift a pair, a larger bias term and, for V, a
// subtraction.)
//
//   K: value = s n + b per (token, 64 channels), so the score of a group is
//        s * sum_c q_c n_c + b * sum_c q_c.
//      A row of q comes as fp16 times a power of two that brings its largest channel into
//      [2^14, 2^15), odd channels over 16: every bf16 or fp16 channel down to 2^-25 of the largest
//      keeps all its bits, and the score's factor takes the power back. The bias terms come from
//      one more MMA, in bf16, whose A operand is the (s, b) words as they lie in memory and whose B
//      operand holds the group sums of q in three bf16 parts.
//   V: with the group's s folded into the weights, sum_t (p_t s_t) n_tc + sum_t p_t b_t; the second
//      sum stays in fp32. p s in fp16 is taken against a power of two S that bounds the scales seen
//      so far (O is rescaled when one exceeds it, as for the running maximum): at the most 2^15,
//      full precision down to 2^-20 S, and below that off by 2^-31 S at the most. One fp16 (2^-12 on
//      average) for bf16 outputs, as fine as the weights of a prefill; for fp16 outputs, whose own
//      rounding is no coarser, a second one holds what the first left out.
//
//   S = K Q^T with 16 tokens by 8 columns (m16n8k16), O = V^T P with 16 channels by 8 columns:
//   few columns fill the n side. p s turns from S's layout (token rows) to P's (column rows) by one
//   movmatrix.
//
// What bounds it now (64 ragged sequences, window 4096, D = 128, 4 columns: 53.3 us with the join): the
// latency between dependent instructions at four warps a scheduler, with half of the integer units' and
// 60 % of the issue slots' rate in use; O, the ring and a tile's fragments leave registers for no more
// warps. DRAM is at 42 % and the tensor pipe at 17 %. With 16 columns at D = 256 (two warps a scheduler) the
// slots are 32 % busy: 55.5 us for 8 x 16384 keys, of which the attention alone takes 51 us and the join of
// 76 parts a problem 15 us where nothing runs beside it. More than 16 columns (heads of a group times rows)
// are several problems, each of which reads and unpacks the sequence again: there, in bf16, 16 columns take 51 us,
// 32 take 76 and 64 take 127. (The products on tcgen05 with e4m3 codes, the unpacked codes
// passing through tensor and shared memory between warps of different roles, took 89 and 76 us: a tile's
// chain of hand-overs is longer than its share of the copy rate, and neither two CTAs an SM nor deeper
// rings hid it.)
//
// Work split: all sequences' tiles of 32 tokens are numbered sequence by sequence, KV head by KV
// head (each problem with OVERHEAD positions more for its start), and cut into equal runs, one a
// warp: the lengths are on the device, so each warp finds its run from them. Warps share nothing:
// each streams its K and V tiles through a ring of its own (bulk copies of the codes' and scales'
// contiguous runs, one mbarrier a slot), keeps its own running maximum, sum and O in registers, and
// so ragged batches of short sequences keep every warp busy. (With a CTA's warps going round one
// problem's tiles and joining through shared memory, the 64 ragged sequences took 150 us: CTAs with
// many short problems ran twice as long as the others.) The maximum moves only when a score exceeds
// it by more than 8 (base 2), found by a vote, so most tiles need no reduction. A problem that lies
// in one run is written directly; the parts of the others go to the workspace in fp32 and
// cache4_merge_kernel joins them in a fixed order.
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
    int2 *joins;             // behind the parts: of each problem its first run and its parts (0: written directly)
    unsigned int *status;
    unsigned long long timeout_ns;
    long long table_stride;
    int num_pages, page_size, max_pages;
    int nseq, n, Hq, Hkv, G;
    int window, sinks;  // window 0: every key
    int chunks;         // column chunks of 8 * NT
    int runs;           // warps that share the tiles (the merge sees the same number)
    int part_cols;      // columns of a part in the workspace: the live ones of a chunk
    int no_copies;      // test hook: no copy is issued, every wait runs out
    float c;            // scale * log2(e)
};

namespace c4 {

constexpr int TILE = 32;     // tokens a warp step
// Tiles that a problem's start and end cost as much as: with 1, 2, 3, 5 the 64 ragged sequences took 57.7, 54.1, 56.7,
// 56.6 us, 4 x 32768 keys with 4 rows 80.5, 78.5, 78.1, 78.4, 256 x 600 keys 65.5, 65.6, 69.5, 69.8.
constexpr int OVERHEAD = 2;
constexpr int MERGE_THREADS = 256;
constexpr unsigned FULL = 0xffffffffu;
constexpr float RESCALE = 8.f;               // weights stay below 2^8 of the reference
constexpr float RANGE = 64.f;                // p = 1 with the largest scale is stored as 64 at most, so 2^8 of it fits fp16
constexpr float CODE_UNIT = 16777216.f / RANGE;  // of an O accumulator: codes are n * 2^-24
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

// Positions of one problem of a sequence, and of all its problems.
__device__ __forceinline__ long long problem_length(const Span &sp) { return sp.count > 0 ? sp.count + OVERHEAD : 0; }

// Runs with work: every one of them has at least a position.
__device__ __forceinline__ int busy_runs(const Cache4AttnParams &p, long long total)
{
    return total < p.runs ? static_cast<int>(total) : p.runs;
}

// First position of run i.
__device__ __forceinline__ long long run_start(long long total, int i, int n) { return total * i / n; }

// Floats of one part in the workspace: O [columns][D] (over its own l, so that no part is larger than the
// values it joins), then m and l of each column, in all a
// multiple of 4 (O is stored 16 bytes at a time) whatever the number of columns.
template <int D>
__host__ __device__ constexpr long long part_floats(int cols)
{
    return static_cast<long long>(cols) * (D + 4);
}

// Warps a CTA, by the registers that are left: O alone
// takes D / 16 * NT * 4 registers a thread.
template <int D, int NT>
struct Plan {
    static constexpr int GQ = D / kCacheGroup;
    static constexpr int WARPS = D == 128 ? (NT == 1 ? 16 : 12) : (NT == 1 ? 12 : 8);
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int COLS = 8 * NT;
    static constexpr int CODE = TILE * D / 2;    // bytes of a tile's K (or V) codes
    static constexpr int SCALE = TILE * GQ * 4;  // and of its scales
    static constexpr int SLOT = CODE + SCALE;
    // More slots leave less L1 to what does not fit the registers: with all that fit (5, 6, 3 and 4) the 64 ragged
    // sequences took 54.1 instead of 53.5 us, 4 x 32768 keys with 4 rows 78.5 instead of 76.2, 8 x 16384 at D = 256
    // 55.6 instead of 53.9.
    static constexpr int NSLOT = 3;
    static constexpr int KSTEPS = D / 16;
    // steps that hold the three bf16 parts (24 bits) of each group's sum of q, eight (s, b) pairs a step
    static constexpr int BIAS_STEPS = GQ == 2 ? 1 : 2;
    static constexpr int QF = (KSTEPS + BIAS_STEPS) * NT * 32 * 8;  // B fragments of a warp
    static constexpr int Q_FRAG = WARPS * NSLOT * SLOT;
    static constexpr int PREFIX = Q_FRAG + WARPS * QF;  // THREADS + WARPS long longs
    static constexpr int BARS = PREFIX + 8 * (THREADS + WARPS);
    static constexpr int BYTES = BARS + 8 * WARPS * NSLOT;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static_assert(SLOT % 128 == 0 && Q_FRAG % 16 == 0 && PREFIX % 8 == 0, "alignment");
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

// Codes i and i + 4 of a word as two fp16 numbers: the subnormals n * 2^-24 for even i, and n * 2^-20, with no
// shift of their own, for odd i.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i)
{
    return (i < 2 ? w : w >> 8) & ((i & 1) ? 0x00f000f0u : 0x000f000fu);
}

// Pairs of fp16: a * b, a * b + c.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The larger of each 16-bit half.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

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

// A walk over a run, segment by segment (the run's tiles of one problem). Segments without a tile
// (the run ends inside a problem's start) are passed over.
struct Walk {
    Span sp;
    int s, u;             // sequence; problem in it: KV head * chunks + chunk
    int e0, e1;           // tiles [e0, e1) of the problem
    long long off, left;  // position in the sequence's problems, positions left in the run
    __device__ __forceinline__ void find(const Cache4AttnParams &p)
    {
        while (left > 0) {
            const long long len = problem_length(sp);
            if (off >= len * p.Hkv * p.chunks) {  // `left` counts positions that exist: a sequence follows
                off -= len * p.Hkv * p.chunks;
                sp = span_of(p, ++s);
                continue;
            }
            u = static_cast<int>(off / len);
            const long long in = off - u * len, take = min(left, len - in);
            e0 = static_cast<int>(max(0ll, in - OVERHEAD));
            e1 = static_cast<int>(in + take - OVERHEAD);
            off += take;
            left -= take;
            if (e1 > e0)
                return;
        }
        e0 = e1 = 0;
        s = -1;
    }
    __device__ __forceinline__ bool done() const { return s < 0; }
};

// Waits up to the limit for the phase of `bar`; false when it ran out.
static __device__ __noinline__ bool wait_slot_slow(uint32_t bar, uint32_t parity, unsigned long long timeout_ns)
{
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer_ns() - t0 > timeout_ns)
            return false;
    return true;
}

__device__ __forceinline__ bool wait_slot(uint32_t bar, uint32_t parity, unsigned long long timeout_ns)
{
    return ptx::mbar_try_wait(bar, parity) || wait_slot_slow(bar, parity, timeout_ns);
}

}  // namespace c4

// One tile's scores to weights to O (see the top of the file). MASKED: some column does not see
// some key of the tile, or the tile ends past the sequence.
template <int D, bool BF16, int NT>
struct Tile {
    static constexpr int PARTS = BF16 ? 1 : 2;  // fp16 parts of a weight

    using P = c4::Plan<D, NT>;
    static constexpr int GQ = P::GQ;
    float o[D / 16][NT][4], m[NT][2], l[NT][2], corr[NT][2][GQ];
    float f[NT][2];         // of the columns: from a score's units to base 2
    uint32_t s_bits;        // V's scales so far are at most this bf16, a power of two (or 0)
    float x_mul;            // RANGE / it

    __device__ __forceinline__ void clear()
    {
        s_bits = 0;
        x_mul = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int gq = 0; gq < GQ; ++gq)
                corr[nt][0][gq] = corr[nt][1][gq] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
        }
    }

    // s = scores in base 2 of the K tile at kc: rows ta, ta + 8 of each 16-token chunk, columns
    // 2 quad, 2 quad + 1.
    __device__ __forceinline__ void scores(float (&s)[2][NT][4], const uint8_t *kc, const uint2 *qf, int lane)
    {
        using namespace c4;
        const int row8 = lane >> 2, quad = lane & 3;
        // MMA row r (and r + 8) of a 16-token chunk is token ta (and ta + 8), so that P's
        // rows 2 quad, 2 quad + 1, 2 quad + 8, 2 quad + 9 are tokens quad + {0, 4, 8, 12}
        const int ta = (row8 >> 1) + ((row8 & 1) << 2);
        const uint32_t *ksc = reinterpret_cast<const uint32_t *>(kc + P::CODE);
        // the bias terms
#pragma unroll
        for (int mc = 0; mc < 2; ++mc) {
            const uint32_t wa = ksc[(mc * 16 + ta) * GQ + quad % GQ], wb = ksc[(mc * 16 + ta + 8) * GQ + quad % GQ];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s[mc][nt][0] = s[mc][nt][1] = s[mc][nt][2] = s[mc][nt][3] = 0.f;
#pragma unroll
                for (int st = 0; st < P::BIAS_STEPS; ++st) {
                    const uint2 b = qf[((P::KSTEPS + st) * NT + nt) * 32 + lane];
                    mma_bf16(s[mc][nt], wa, wb, wa, wb, b.x, b.y);
                }
            }
        }
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
                    const int h = 2 * (j & 1);
                    const uint32_t a0 = code_pair(x, h), a1 = code_pair(y, h);
                    const uint32_t a2 = code_pair(x, h + 1), a3 = code_pair(y, h + 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(acc[mc][nt], a0, a1, a2, a3, b[nt].x, b[nt].y);
                }
            }
#pragma unroll
            for (int mc = 0; mc < 2; ++mc) {
                const float sa = scale_of(ksc[(mc * 16 + ta) * GQ + gq]), sb = scale_of(ksc[(mc * 16 + ta + 8) * GQ + gq]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    s[mc][nt][0] = fmaf(sa, acc[mc][nt][0], s[mc][nt][0]);
                    s[mc][nt][1] = fmaf(sa, acc[mc][nt][1], s[mc][nt][1]);
                    s[mc][nt][2] = fmaf(sb, acc[mc][nt][2], s[mc][nt][2]);
                    s[mc][nt][3] = fmaf(sb, acc[mc][nt][3], s[mc][nt][3]);
                }
            }
        }
#pragma unroll
        for (int mc = 0; mc < 2; ++mc)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[mc][nt][i] *= f[nt][i & 1];
    }

    // Keys that a column does not see drop out: key tok0 + ... against positions first + r / G.
    __device__ __forceinline__ void mask(float (&s)[2][NT][4], const Cache4AttnParams &p, int tok0, int first, int r_base,
                                         int lane)
    {
        const int row8 = lane >> 2, quad = lane & 3, ta = (row8 >> 1) + ((row8 & 1) << 2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = nt * 8 + 2 * quad + i;
                const int at = first + min(p.n - 1, (r_base + col) / p.G);
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

    // The running maximum moves when some score is more than RESCALE above it; then s becomes the weights.
    __device__ __forceinline__ void weights(float (&s)[2][NT][4])
    {
        using namespace c4;
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
#pragma unroll
                for (int gq = 0; gq < GQ; ++gq) {
                    corr[nt][0][gq] *= a[0];
                    corr[nt][1][gq] *= a[1];
                }
            }
        }
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
                s[mc][nt][0] = p0;
                s[mc][nt][1] = p1;
                s[mc][nt][2] = p2;
                s[mc][nt][3] = p3;
            }
        }
    }

    // O += V^T P of the V tile at vc with the weights w. MASKED: a key that a column does not see has
    // weight 0 there, whatever scale its place in the pool holds.
    template <bool MASKED>
    __device__ __forceinline__ void output(const float (&w)[2][NT][4], const uint8_t *vc, int lane)
    {
        using namespace c4;
        const int row8 = lane >> 2, quad = lane & 3, ta = (row8 >> 1) + ((row8 & 1) << 2);
        // ---- scales of the tokens ta, ta + 8 of each chunk, and their bound
        uint32_t sb[2][2][GQ];
        uint32_t top = 0;
#pragma unroll
        for (int mc = 0; mc < 2; ++mc)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t *at = reinterpret_cast<const uint32_t *>(vc + P::CODE) + (mc * 16 + ta + 8 * x) * GQ;
                if constexpr (GQ == 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(at);
                    sb[mc][x][0] = v.x, sb[mc][x][1] = v.y, sb[mc][x][2] = v.z, sb[mc][x][3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(at);
                    sb[mc][x][0] = v.x, sb[mc][x][1] = v.y;
                }
                bool seen = !MASKED;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    seen |= w[mc][nt][2 * x] != 0.f || w[mc][nt][2 * x + 1] != 0.f;
#pragma unroll
                for (int gq = 0; gq < GQ; ++gq)
                    top = max_halves(top, seen ? sb[mc][x][gq] : 0u);
            }
        if (__any_sync(FULL, (top & 0xffffu) > s_bits)) {  // (a scale below zero, too: its bits are above)
            uint32_t mx = 0;
#pragma unroll
            for (int mc = 0; mc < 2; ++mc)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    bool seen = !MASKED;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        seen |= w[mc][nt][2 * x] != 0.f || w[mc][nt][2 * x + 1] != 0.f;
#pragma unroll
                    for (int gq = 0; gq < GQ; ++gq) {
                        const uint32_t b = sb[mc][x][gq] & 0x7fffu;
                        mx = max(mx, seen && b < 0x7f80u ? b : 0u);  // one that is not finite bounds nothing
                    }
                }
            mx = __reduce_max_sync(FULL, mx);
            if (mx > s_bits) {
                // the power of two above it, kept where RANGE over it is a normal number
                const uint32_t next = max(8u, min(254u, (mx >> 7) + 1)) << 7;
                const float bound = __uint_as_float(next << 16), ratio = __uint_as_float(s_bits << 16) / bound;
                s_bits = next;
                x_mul = RANGE / bound;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            o[i][nt][x] *= ratio;
            }
        }
#pragma unroll
        for (int mc = 0; mc < 2; ++mc) {
            // the weights as two fp16, and where they are not 0
            uint32_t hi[NT][2], lo[NT][2], live[NT][2];
            if constexpr (PARTS == 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = w[mc][nt][2 * x], p1 = w[mc][nt][2 * x + 1];
                        hi[nt][x] = pack16<false>(p0, p1);
                        const float2 h = unpack16<false>(hi[nt][x]);
                        lo[nt][x] = pack16<false>(p0 - h.x, p1 - h.y);
                        if constexpr (MASKED)
                            live[nt][x] = (p0 != 0.f ? 0xffffu : 0u) | (p1 != 0.f ? 0xffff0000u : 0u);
                    }
            }
#pragma unroll
            for (int gq = 0; gq < GQ; ++gq) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = *reinterpret_cast<const uint32_t *>(vc + (mc * 16 + quad + 4 * i) * (D / 2) + gq * 32 + row8 * 4);
                uint32_t pw[PARTS][NT][2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float sc = scale_of(sb[mc][x][gq]) * x_mul, bi = bias_of(sb[mc][x][gq]);
                    const uint32_t s2 = PARTS == 2 ? pack16<false>(sc, sc) : 0u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float y[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float pi = w[mc][nt][2 * x + i];
                            const bool out = MASKED && pi == 0.f;
                            if constexpr (PARTS == 1)
                                y[i] = out ? 0.f : pi * sc;
                            corr[nt][i][gq] = out ? corr[nt][i][gq] : fmaf(pi, bi, corr[nt][i][gq]);
                        }
                        if constexpr (PARTS == 1) {
                            pw[0][nt][x] = movmatrix(pack16<false>(y[0], y[1]));
                        } else {
                            // w * s rounded, and what that left out
                            uint32_t a = hmul2(hi[nt][x], s2);
                            uint32_t b = hfma2(lo[nt][x], s2, hfma2(hi[nt][x], s2, a ^ 0x80008000u));
                            if constexpr (MASKED) {
                                a &= live[nt][x];
                                b &= live[nt][x];
                            }
                            pw[0][nt][x] = movmatrix(a);
                            pw[PARTS - 1][nt][x] = movmatrix(b);
                        }
                    }
                }
                // halves of the words: codes 0-3 of two tokens, codes 4-7 of two tokens
                const uint32_t x01 = __byte_perm(v[0], v[1], 0x5410), y01 = __byte_perm(v[0], v[1], 0x7632);
                const uint32_t x23 = __byte_perm(v[2], v[3], 0x5410), y23 = __byte_perm(v[2], v[3], 0x7632);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const uint32_t w01 = mt < 2 ? x01 : y01, w23 = mt < 2 ? x23 : y23;
                    const int h = 2 * (mt & 1);
                    const uint32_t a0 = code_pair(w01, h), a1 = code_pair(w01, h + 1);
                    const uint32_t a2 = code_pair(w23, h), a3 = code_pair(w23, h + 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < PARTS; ++i)
                            mma_f16(o[gq * 4 + mt][nt], a0, a1, a2, a3, pw[i][nt][0], pw[i][nt][1]);
                }
            }
        }
    }
};

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(c4::Plan<D, NT>::THREADS, 1) cache4_attn_kernel(const Cache4AttnParams p)
{
    using namespace c4;
    using P = Plan<D, NT>;
    constexpr int GQ = P::GQ, WARPS = P::WARPS, THREADS = P::THREADS;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row8 = lane >> 2, quad = lane & 3;  // an MMA fragment's row (or column n) and place in it
    const uint32_t ring = sbase + warp * P::NSLOT * P::SLOT;
    const uint8_t *ring_p = smem + warp * P::NSLOT * P::SLOT;
    uint2 *qf = reinterpret_cast<uint2 *>(smem + P::Q_FRAG + warp * P::QF);
    const uint32_t bars = sbase + P::BARS + 8 * warp * P::NSLOT;

    if (lane == 0) {
        for (int i = 0; i < P::NSLOT; ++i)
            ptx::mbar_init(bars + 8 * i, 1);
        ptx::fence_barrier_init();
    }
    // ---- where this warp's run starts: prefix sums of the sequences' positions, a few sequences a thread
    const int run = warp * gridDim.x + blockIdx.x;  // consecutive runs lie on different SMs, so that few runs use many
    // positions in all, from the warps' sums (which stay where they are)
    auto positions = [&]() {
        const long long *warp_sum = reinterpret_cast<const long long *>(smem + P::PREFIX) + THREADS;
        long long total = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i)
            total += warp_sum[i];
        return total;
    };
    Walk ahead;  // the copies' place in the run
    {
        long long *prefix = reinterpret_cast<long long *>(smem + P::PREFIX), *warp_sum = prefix + THREADS;
        const int per_tile = p.Hkv * p.chunks;
        const int per = (p.nseq + THREADS - 1) / THREADS;
        const long long first = static_cast<long long>(tid) * per;
        const int s0 = static_cast<int>(min(static_cast<long long>(p.nseq), first));
        const int s1 = static_cast<int>(min(static_cast<long long>(p.nseq), first + per));
        long long sum = 0;
        for (int s = s0; s < s1; ++s)
            sum += problem_length(span_of(p, s));
        sum *= per_tile;
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(FULL, incl, d);
            if (lane >= d)
                incl += x;
        }
        prefix[tid] = incl - sum;  // within the warp
        if (lane == 31)
            warp_sum[warp] = incl;
        __syncthreads();
        const long long total = positions();
        const int busy = busy_runs(p, total);
        if (run >= busy)
            return;
        const long long x = run_start(total, run, busy);
        ahead.left = run_start(total, run + 1, busy) - x;
        // the last thread whose sequences start at or before x
        long long before = 0;
        int w0 = 0;
        while (before + warp_sum[w0] <= x)
            before += warp_sum[w0++];
        const unsigned at = __ballot_sync(FULL, before + prefix[w0 * 32 + lane] <= x);
        const int owner = w0 * 32 + 31 - __clz(at);
        ahead.off = x - before - prefix[owner];
        ahead.s = owner * per;
        ahead.sp = span_of(p, ahead.s);
        ahead.find(p);  // passes over whole sequences where a thread has several
    }
    Walk w = ahead;

    // ---- copies. A tile's K part, then its V part, go to the ring's next slot. The page id of the
    // next tile is loaded a tile ahead, so that no copy waits for it.
    const int pieces = (p.page_size & 31) == 0 ? 1 : 2;  // a 32-token tile lies in one page, or in halves
    const int piece_tokens = TILE / pieces;
    const int half = pieces == 1 ? 0 : (lane >> 1) & 1;  // lane: codes or scales (bit 0) of a piece (bit 1)
    int ae = ahead.e0;                                   // the next tile to copy
    int page_id = 0, page_off = 0;
    auto look_up = [&]() {
        if (ahead.done())
            return;
        int tok = ahead.sp.tile(ae) * TILE + half * piece_tokens;
        // A half between the sinks and the first row's window may lie in a page that is no longer there. The tile's
        // other half, which some row sees, is copied in its place, and masked.
        if (p.window > 0 && tok >= p.sinks && tok + piece_tokens + p.n - 1 <= ahead.sp.len - p.window)
            tok ^= piece_tokens;
        const int slot = tok / p.page_size;
        page_off = tok - slot * p.page_size;
        // a half behind the last page is copied from that page and masked
        page_id = __ldg(p.table + ahead.s * p.table_stride + min(slot, (ahead.sp.len - 1) / p.page_size));
    };
    look_up();
    bool is_v = false;  // the next part to copy
    auto issue = [&](int slot) {
        if (!p.no_copies) {
            const uint32_t bar = bars + 8 * slot;
            if (lane == 0)
                expect_tx(bar, P::SLOT);
            __syncwarp();
            if (lane < 2 * pieces) {
                int id = page_id;
                if (id < 0 || id >= p.num_pages) {
                    atomicCAS(p.status, 0u, kBadPages);
                    id = 0;
                }
                const long long row =
                    (static_cast<long long>(id) * p.Hkv + ahead.u / p.chunks) * p.page_size + page_off;
                const uint32_t base = ring + slot * P::SLOT;
                if (lane & 1)
                    bulk_load(base + P::CODE + half * piece_tokens * GQ * 4, (is_v ? p.v_scales : p.k_scales) + row * GQ,
                              piece_tokens * GQ * 4, bar);
                else
                    bulk_load(base + half * piece_tokens * (D / 2), (is_v ? p.v_codes : p.k_codes) + row * (D / 2),
                              piece_tokens * (D / 2), bar);
            }
        }
        if (is_v) {
            if (++ae >= ahead.e1) {
                ahead.find(p);
                ae = ahead.e0;
            }
            look_up();
        }
        is_v = !is_v;
    };
    int in_flight = 0;
    for (; in_flight < P::NSLOT && !ahead.done(); ++in_flight)
        issue(in_flight);
    int slot = 0;
    uint32_t phase = 0;
    auto step_slot = [&]() {
        if (++slot == P::NSLOT) {
            slot = 0;
            phase ^= 1u;
        }
    };
    // the next part has landed; false (and the warp stops) when its wait ran out
    auto landed = [&]() -> bool {
        if (__all_sync(FULL, wait_slot(bars + 8 * slot, phase, p.timeout_ns)))
            return true;
        if (lane == 0)
            atomicCAS(p.status, 0u, kSlotNeverFilled | (blockIdx.x << 8));
        // this warp's copies land (waited for with a limit again) before the CTA may exit
        for (; in_flight > 0 && !p.no_copies; --in_flight) {
            wait_slot(bars + 8 * slot, phase, p.timeout_ns);
            step_slot();
        }
        return false;
    };
    // the slot just read takes the next part
    auto refill = [&]() {
        __syncwarp();
        if (!ahead.done())
            issue(slot);
        else
            --in_flight;
        step_slot();
    };

    const int R = p.n * p.G;
    Tile<D, BF16, NT> t;
    for (; !w.done(); w.find(p)) {
        const int g = w.u / p.chunks, r_base = (w.u - g * p.chunks) * P::COLS;
        auto row_of = [&](int r) {  // the (sequence, row, head) row of column r in q, o and lse
            return (static_cast<long long>(w.s) * p.n + r / p.G) * p.Hq + g * p.G + r % p.G;
        };
        // ---- the queries as B fragments: lane (column row8, quad) holds 16 channels of each group
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = r_base + nt * 8 + row8;
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (r < R ? row_of(r) : 0) * D) + quad * 2;
            uint4 x[GQ][2];
            float mx = 0.f;
            bool odd = false;  // an infinity or a NaN
#pragma unroll
            for (int gq = 0; gq < GQ; ++gq)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[gq][j] = r < R ? __ldg(src + gq * 8 + j) : make_uint4(0u, 0u, 0u, 0u);
                    float v[8];
                    unpack8<BF16>(x[gq][j], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        mx = fmaxf(mx, fabsf(v[i]));
                        odd |= !(fabsf(v[i]) <= 3.4028235e38f);
                    }
                }
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
            odd = (__ballot_sync(FULL, odd) >> (lane & ~3)) & 15u;
            // The power of two that brings the row's largest into [2^14, 2^15): in fp16 every channel down to 2^-25
            // of it keeps its 11 bits, a sixteenth of it, too.
            const int ex = max(-126, min(126, 141 - static_cast<int>(__float_as_uint(mx) >> 23)));
            const float factor = mx == 0.f || odd ? 1.f : __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
            const float back = odd ? __uint_as_float(0x7fc00000u) : p.c * 16777216.f / factor;  // 2^24 of the codes
            t.f[nt][0] = __shfl_sync(FULL, back, 8 * quad);
            t.f[nt][1] = __shfl_sync(FULL, back, 8 * quad + 4);
            float sum[GQ];
#pragma unroll
            for (int gq = 0; gq < GQ; ++gq) {
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[8];
                    unpack8<BF16>(x[gq][j], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[i] = odd ? 0.f : v[i] * factor;
                        a += v[i];
                    }
                    // channels (c, c + 4) pair up, as the codes of a word do; odd ones meet codes times 16
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[((gq * 4 + 2 * j + i) * NT + nt) * 32 + lane] =
                            make_uint2(pack16<false>(v[2 * i], v[2 * i + 4]),
                                       pack16<false>(v[2 * i + 1] * 0.0625f, v[2 * i + 5] * 0.0625f));
                }
                a += __shfl_xor_sync(FULL, a, 1);
                a += __shfl_xor_sync(FULL, a, 2);
                sum[gq] = a * 5.9604644775390625e-8f;  // 2^-24
            }
            // the bias step's B operand: k pair j holds (0, part j / GQ of group j % GQ's sum)
#pragma unroll
            for (int st = 0; st < P::BIAS_STEPS; ++st) {
                uint32_t b[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = st * 8 + x * 4 + quad;
                    float a = sum[0];
#pragma unroll
                    for (int gq = 1; gq < GQ; ++gq)
                        a = j % GQ == gq ? sum[gq] : a;
                    const int which = j / GQ;
                    const float p0 = __bfloat162float(__float2bfloat16_rn(a));
                    const float p1 = __bfloat162float(__float2bfloat16_rn(a - p0));
                    const float part = which == 0 ? p0 : which == 1 ? p1 : which == 2 ? (a - p0) - p1 : 0.f;
                    b[x] = pack16<true>(0.f, part);
                }
                qf[((P::KSTEPS + st) * NT + nt) * 32 + lane] = make_uint2(b[0], b[1]);
            }
        }
        __syncwarp();

        t.clear();
        const int first = w.sp.len - p.n;  // position of row 0
        const int pos_lo = first + r_base / p.G;
        const int pos_hi = first + min(p.n - 1, (r_base + P::COLS - 1) / p.G);
        for (int e = w.e0; e < w.e1; ++e) {
            const int tok0 = w.sp.tile(e) * TILE;
            const bool whole = tok0 + TILE - 1 <= pos_lo &&
                               (p.window == 0 || tok0 > pos_hi - p.window || tok0 + TILE <= p.sinks);
            float s[2][NT][4];
            if (!landed())
                return;
            t.scores(s, ring_p + slot * P::SLOT, qf, lane);
            refill();
            if (!whole)
                t.mask(s, p, tok0, first, r_base, lane);
            t.weights(s);
            if (!landed())
                return;
            if (whole)
                t.template output<false>(s, ring_p + slot * P::SLOT, lane);
            else
                t.template output<true>(s, ring_p + slot * P::SLOT, lane);
            refill();
        }

        // ---- the segment's result: a lane holds channels 8 row8 .. + 7 of each group, of columns
        // 2 quad and 2 quad + 1
        const bool direct = w.e0 == 0 && w.e1 == w.sp.count;
        if (w.e0 == 0 && lane == 0) {  // for the join
            int parts = 0;
            if (!direct) {  // the run ends in the problem, whose last tile some run after it holds
                const long long total = positions();
                const int busy = busy_runs(p, total);
                const long long last = run_start(total, run + 1, busy) + (w.sp.count - w.e1) - 1;
                parts = static_cast<int>(((last + 1) * busy - 1) / total) - run + 1;
            }
            p.joins[w.s * p.Hkv * p.chunks + w.u] = make_int2(run, parts);
        }
        const float bound = __uint_as_float(t.s_bits << 16);
        // a part that continues a problem is this run's first segment, one that begins it its last
        float *part = p.workspace + (static_cast<long long>(run) * 2 + (w.e0 == 0 ? 1 : 0)) * part_floats<D>(p.part_cols);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = t.l[nt][i];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    sum += __shfl_xor_sync(FULL, sum, off);
                const int col = nt * 8 + 2 * quad + i, r = r_base + col;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees no key: 0 and -inf
#pragma unroll
                for (int gq = 0; gq < GQ; ++gq) {
                    float c = t.corr[nt][i][gq];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        c += __shfl_xor_sync(FULL, c, off);
                    float y[8];
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int x = 0; x < 2; ++x)  // odd channels' codes came times 16
                            y[2 * mt + x] =
                                fmaf(t.o[gq * 4 + mt][nt][2 * x + i] * (inv * (x == 0 ? CODE_UNIT : CODE_UNIT / 16.f)), bound, c * inv);
                    if (r >= R)
                        continue;
                    const int c0 = gq * kCacheGroup + row8 * 8;
                    if (direct) {
                        *reinterpret_cast<uint4 *>(p.o + row_of(r) * D + c0) = pack8<BF16>(y);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(part + col * D + c0);
                        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                    }
                }
                if (r < R && row8 == 0) {
                    if (!direct) {
                        part[p.part_cols * D + col] = t.m[nt][i];
                        part[p.part_cols * (D + 1) + col] = sum;
                    } else if (p.lse != nullptr) {
                        p.lse[row_of(r)] = sum == 0.f ? -INFINITY : (t.m[nt][i] + log2f(sum)) * kLn2;
                    }
                }
            }
        }
    }
}

// Joins the parts of every problem that more than one run shares, in the order of the runs, and
// writes the rows of empty sequences. A block takes one column of a problem, its eight warps every eighth
// part each, so that the parts of a long problem (76 at eight sequences of 16384 keys) are read at once and not one
// after the other; or (ONE, with many problems, of a few parts each) a column a warp. The attention leaves each
// problem's first run and parts: with every block finding them from the lengths, 2048 blocks took 11 us and 8192 took 42.
template <int D, bool BF16, int NT, bool ONE>
__global__ void __launch_bounds__(c4::MERGE_THREADS) cache4_merge_kernel(const Cache4AttnParams p)
{
    using namespace c4;
    constexpr int WARPS = MERGE_THREADS / 32, V = D / 128;  // V float4 a lane
    __shared__ float4 y_all[ONE ? 1 : WARPS][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_seq = p.Hkv * p.chunks, pc = p.part_cols;
    const int blocks = ONE ? (pc + WARPS - 1) / WARPS : pc;  // of a problem
    const int problem = blockIdx.x / blocks, at = blockIdx.x - problem * blocks;
    const int col = ONE ? at * WARPS + warp : at;
    const int s = problem / per_seq, u = problem - s * per_seq;
    const int g = u / p.chunks, r = (u - g * p.chunks) * 8 * NT + col;
    const Span sp = span_of(p, s);
    // What is above runs beside the attention's end. Every thread waits for that end: what follows on the
    // stream waits for this kernel alone.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (col >= pc || r >= p.n * p.G)
        return;
    const long long row = (static_cast<long long>(s) * p.n + r / p.G) * p.Hq + g * p.G + r % p.G;
    if (sp.count == 0) {
        if (sp.bad) {
            if (lane == 0)
                atomicCAS(p.status, 0u, kBadSeqlens);
            return;
        }
        if ((ONE || warp == 0) && lane < D / 8)
            reinterpret_cast<uint4 *>(p.o + row * D)[lane] = make_uint4(0u, 0u, 0u, 0u);
        if ((ONE || warp == 0) && lane == 0 && p.lse != nullptr)
            p.lse[row] = -INFINITY;
        return;
    }
    const int2 join = p.joins[problem];
    const int i0 = join.x, parts = join.y;
    // nothing to join; or the word was never written (a wait ran out, and the status says so)
    if (parts < 2 || i0 < 0 || parts > p.runs - i0)
        return;
    // part x (run i0 + x): the first begins the problem (slot 1), the others continue it (slot 0)
    auto part = [&](int x) { return p.workspace + (2LL * (i0 + x) + (x == 0 ? 1 : 0)) * part_floats<D>(pc); };
    auto m_of = [&](int x) { return part(x)[pc * D + col]; };
    auto l_of = [&](int x) { return part(x)[pc * (D + 1) + col]; };
    // every warp finds the maximum and the sum for itself
    const float m0 = lane < parts ? m_of(lane) : -INFINITY, l0 = lane < parts ? l_of(lane) : 0.f;
    float mx = m0;
    for (int x = lane + 32; x < parts; x += 32)
        mx = fmaxf(mx, m_of(x));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
    // 1: the part holds 0, or NaN
    auto weight = [&](float mw, float lw) { return (mw == -INFINITY ? 1.f : ptx::ex2(mw - mx)) * lw; };
    float sum = weight(m0, l0);
    for (int x = lane + 32; x < parts; x += 32)
        sum += weight(m_of(x), l_of(x));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        sum += __shfl_xor_sync(FULL, sum, off);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float4 y[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = ONE ? 0 : warp; x < parts; x += ONE ? 1 : WARPS) {
        const float4 *src = reinterpret_cast<const float4 *>(part(x) + col * D);
        const float f = weight(m_of(x), l_of(x)) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float4 t = src[i * 32 + lane];
            y[i].x = fmaf(f, t.x, y[i].x);
            y[i].y = fmaf(f, t.y, y[i].y);
            y[i].z = fmaf(f, t.z, y[i].z);
            y[i].w = fmaf(f, t.w, y[i].w);
        }
    }
    if constexpr (!ONE) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            y_all[warp][i * 32 + lane] = y[i];
        __syncthreads();
        if (warp != 0)
            return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 t = y_all[w][i * 32 + lane];
                y[i].x += t.x;
                y[i].y += t.y;
                y[i].z += t.z;
                y[i].w += t.w;
            }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        reinterpret_cast<uint2 *>(p.o + row * D)[i * 32 + lane] =
            make_uint2(pack16<BF16>(y[i].x, y[i].y), pack16<BF16>(y[i].z, y[i].w));
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

template <int D, bool BF16, int NT>
cudaError_t launch_cache4_attn(Cache4AttnParams p, int sms, cudaStream_t st)
{
    using P = c4::Plan<D, NT>;
    static unsigned long long done = 0;
    auto kern = cache4_attn_kernel<D, BF16, NT>;
    cudaError_t e = set_smem_once(kern, P::BYTES, done);
    if (e != cudaSuccess)
        return e;
    p.runs = sms * P::WARPS;
    kern<<<sms, P::THREADS, P::BYTES, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    // the blocks of the join start where the attention's CTAs end, not when the last one has
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    // a column a warp once that still gives every SM two blocks
    const int problems = p.nseq * p.Hkv * p.chunks;
    const bool one = problems >= 2 * sms;
    constexpr int WARPS = c4::MERGE_THREADS / 32;
    config.gridDim = dim3(problems * (one ? (p.part_cols + WARPS - 1) / WARPS : p.part_cols));
    config.blockDim = dim3(c4::MERGE_THREADS);
    config.stream = st;
    config.attrs = &early;
    config.numAttrs = 1;
    return one ? cudaLaunchKernelEx(&config, cache4_merge_kernel<D, BF16, NT, true>, p)
               : cudaLaunchKernelEx(&config, cache4_merge_kernel<D, BF16, NT, false>, p);
}

// One per (head dim, dtype): 8 columns a warp up to that many, else 16.
cudaError_t cache4_attn_d128_fp16(const Cache4AttnParams &p, int sms, cudaStream_t st);
cudaError_t cache4_attn_d128_bf16(const Cache4AttnParams &p, int sms, cudaStream_t st);
cudaError_t cache4_attn_d256_fp16(const Cache4AttnParams &p, int sms, cudaStream_t st);
cudaError_t cache4_attn_d256_bf16(const Cache4AttnParams &p, int sms, cudaStream_t st);

}  // namespace sdp
