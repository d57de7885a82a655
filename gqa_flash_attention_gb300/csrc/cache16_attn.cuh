// Attention of each sequence's last n tokens over the paged 16-bit cache, for batches whose sequences share prefixes
// (sdp_fwd_cache16):
//
//     row i of sequence s is at position p = len_s - n + i and sees the keys j <= p;
//     O = softmax(scale * Q K^T) V over them, LSE = ln sum exp; a row that sees none: 0 and -inf.
//
// The sequences of a group have their first P tokens in common. Softmax over a union of key sets is the sum of
// the sets' own results, each (m, l, O) weighed by 2^(m - max m) l, so there are two kinds of problems:
//
//   - (group, KV head, block): the prefix's keys, read once, for the rows of ALL sequences of the group, 128 a block.
//     Every row sees all of them: a matrix product of as many rows as the batch has, where one sequence alone has
//     the few rows of its group of heads;
//   - (sequence, KV head, block): the keys behind the prefix (all of them for a sequence that shares none).
//
// Both run through the pipeline of the windowed forward (window_kernel.cuh): the G query heads of a KV head and the
// tokens are the 128 lanes of S = Q K^T and O += P V on tcgen05 with both accumulators in tensor memory, 128-key tiles
// through a ring of shared memory (TMA boxes that lie in one page each), one thread a row for the softmax, a
// warpgroup of its own that writes a unit's rows while the next unit runs. Scores, weights and sums are fp32, the
// weights are rounded to the 16-bit type for P V as there. A decoding problem has few live rows: the products are
// padded to 128 lanes (a tile takes 1024 cycles of the tensor core at D = 128 and some 2700 of its share of HBM), the
// softmax is skipped by warps without a live row.
//
// Work split: the problems' tiles are numbered through, groups first, and cut into equal runs, one a CTA; the lengths
// are on the device, so each CTA finds its run from them. A problem that one run holds whole, and whose rows share no
// prefix, is written directly; everything else goes to the workspace in fp32 and cache16_join_kernel adds a row's
// parts up in a fixed order.
//
// What no row sees does not reach a result: scores are selected away, weights are 0, and as 0 times an infinity is
// NaN, rows of V before a problem's first key or behind its last (another sequence's, or never written) are zeroed in
// shared memory or left out of the product. A drafted token's V is seen by some rows of its problem only: where it
// holds values that are not finite these are taken out of the product too, and added to the rows that see them when
// they are written.
#pragma once

#include "sdp_fwd_kernel.cuh"
#include "sdp_internal.h"
#include "sixteen.cuh"

namespace sdp {

struct Cache16AttnParams {
    uint16_t *o;
    float *lse;
    const uint16_t *v;  // the pool (read directly where a value is not finite)
    const int *table, *lens, *prefix_table, *prefix_lens, *cu_groups;
    long long table_stride, prefix_stride;
    int num_pages, page_size, max_pages, prefix_pages;
    int nseq, ngroups, n, Hq, Hkv, G;
    int heads;          // query heads of a block: G, or 128 of a larger group
    int head_blocks;    // blocks of heads of a KV head
    int toks_p, toks_o;  // tokens of a block: of a prefix, of a sequence
    int blocks_o;       // blocks of a sequence's n tokens
    int box;            // keys of a TMA box: they lie in one page
    int part_rows;      // rows of a part in the workspace
    float *parts;       // two a run: the problem it continues and the one it begins
    float *rows_o, *rows_p;  // [nseq * n * Hq][D], then (m, l) of each: problems that one run holds whole
    int2 *joins_o, *joins_p;  // of each problem its first run and its parts (1: whole)
    unsigned int *status;
    unsigned long long timeout_ns;
    int no_copies;  // test hook: no copy is issued, every wait runs out
    float c;        // scale * log2(e)
};

namespace c16 {

constexpr int TILE = 128;
constexpr int OVERHEAD = 2;  // tiles that a problem's start and end cost as much as
constexpr int THREADS = 384;
constexpr int MERGE_THREADS = 256;
constexpr unsigned FULL = 0xffffffffu;

// A group that a sequence shares a prefix with: the prefix's length, 0 for none.
struct Share {
    int g, P;
    bool bad;
};

__device__ __forceinline__ int2 group_range(const Cache16AttnParams &p, int g)
{
    return p.cu_groups == nullptr ? make_int2(0, p.nseq) : make_int2(__ldg(p.cu_groups + g), __ldg(p.cu_groups + g + 1));
}

// The prefix of group g, whose sequences are [r.x, r.y). A group of one sequence has nothing to share.
__device__ __forceinline__ Share prefix_of(const Cache16AttnParams &p, int g, int2 r)
{
    const int P = __ldg(p.prefix_lens + g);
    const bool order = 0 <= r.x && r.x <= r.y && r.y <= p.nseq;
    Share s{g, 0, !order || P < 0 || P > p.prefix_pages * p.page_size};  // the host keeps the product in 31 bits
    if (!s.bad && r.y - r.x > 1)
        s.P = P;
    return s;
}

__device__ __forceinline__ Share share_of(const Cache16AttnParams &p, int s)
{
    if (p.ngroups == 0)
        return Share{-1, 0, false};
    int g = 0;
    if (p.cu_groups != nullptr)
        for (int len = p.ngroups; len > 1;) {  // the last group that begins at or before s
            const int h = len / 2;
            if (__ldg(p.cu_groups + g + h) <= s) {
                g += h;
                len -= h;
            } else {
                len = h;
            }
        }
    const int2 r = group_range(p, g);
    Share a = prefix_of(p, g, r);
    if (s < r.x || s >= r.y)
        a.P = 0;
    return a;
}

// One entry of the list of problems: a group (entries 0 .. ngroups - 1) or a sequence. Its problems are alike: keys
// [lo, hi) in `tiles` tiles from key k0, for each block of heads of each KV head and each block of `toks` tokens.
struct Span {
    int tiles, problems;
    int lo, hi, k0;
    int first, toks;  // the tokens of q
    bool bad;
};

static __device__ __noinline__ Span span_of(const Cache16AttnParams &p, int e)
{
    Span r{};
    if (e < p.ngroups) {
        const int2 at = group_range(p, e);
        const Share s = prefix_of(p, e, at);
        r.bad = s.bad;
        r.hi = s.P;
        if (s.P > 0) {
            r.first = at.x * p.n;
            r.toks = (at.y - at.x) * p.n;
            r.problems = p.Hkv * p.head_blocks * ((r.toks + p.toks_p - 1) / p.toks_p);
            r.tiles = (s.P + TILE - 1) / TILE;
        }
        return r;
    }
    const int s = e - p.ngroups, len = __ldg(p.lens + s);
    const Share a = share_of(p, s);
    r.bad = len < 0 || len > p.max_pages * p.page_size;  // (the join reports it, and leaves the rows)
    r.hi = r.bad ? 0 : len;
    // a sequence whose first row does not see the whole prefix goes through its own pages
    r.lo = a.P > 0 && r.hi >= a.P + p.n - 1 ? a.P : 0;
    r.k0 = r.lo & -p.box;
    r.first = s * p.n;
    r.toks = p.n;
    r.problems = p.Hkv * p.head_blocks * p.blocks_o;
    r.tiles = r.hi > r.lo ? (r.hi - r.k0 + TILE - 1) / TILE : 0;
    return r;
}

__device__ __forceinline__ long long entry_length(const Span &s)
{
    return s.tiles > 0 ? static_cast<long long>(s.problems) * (s.tiles + OVERHEAD) : 0;
}

// Positions cut into n runs: run i begins at floor(total * i / n).
struct Cut {
    long long total, q;
    int r, n;
    __device__ __forceinline__ Cut(long long positions, int most) : total(positions)
    {
        n = total < most ? static_cast<int>(total) : most;
        const int d = max(n, 1);
        // (a 64-bit division takes a few hundred cycles of a launch's first microseconds)
        q = total <= 0xffffffffll ? static_cast<uint32_t>(total) / static_cast<uint32_t>(d) : total / d;
        r = static_cast<int>(total - q * d);
    }
    __device__ __forceinline__ long long start(int i) const { return i * q + i * r / n; }
    __device__ __forceinline__ int run_of(long long x) const { return static_cast<int>(((x + 1) * n - 1) / total); }
};

// Floats of a part: O [rows][D] (over its own l, so that no part is larger than the values it joins), then m and l of
// each row, in all a multiple of 8 (O is stored 32 bytes at a time).
template <int D>
__host__ __device__ constexpr long long part_floats(int rows)
{
    return static_cast<long long>(rows) * (D + 8);
}

constexpr int DEST_DIRECT = -1, DEST_ROWS = -2;  // else the part's number

// A unit: a run's tiles of one problem. n < 0: none, nor any after it.
struct __align__(16) Unit {
    int n, tile0;       // tiles, and the first one's first key
    int lo, hi;         // keys that a row may see
    int q_tok, toks;    // the block's first token in q, and its tokens
    int head, live;     // its first query head, and its heads
    int kv, pos0;       // the KV head; position of the first token (of a prefix: hi - 1, every row's)
    int table, prefix;  // row of the block table, or of the prefixes'
    int dest, unused[3];
};

template <int D>
struct Plan {
    using L = Layout<D>;
    static constexpr int QB = D == 128 ? 2 : 1;  // query tiles in shared memory
    static constexpr int CPT = L::CHUNKS_PER_TILE;
    static constexpr int UNITS = 4;  // units looked up ahead
    static constexpr int BAR_AREA = 384;
    static constexpr int NSLOTS = (L::SMEM_LIMIT - BAR_AREA - 2 * TILE * 4 - UNITS * 64 - 1024 - QB * L::Q_BYTES) / L::CHUNK_BYTES;
    // q_full[QB], q_free[QB], slot_full[NS], slot_empty[NS], s_full[NB], p_full[NB], o_done[ring], final[2], o_free,
    // sum_full, sum_free, odd_full, unit_full[UNITS], unit_free[UNITS]
    static constexpr int NBARS = 2 * QB + 2 * NSLOTS + 2 * L::NSBUF + O_DONE_RING + 2 + 4 + 2 * UNITS;
    static constexpr int BAR_OFF = QB * L::Q_BYTES + NSLOTS * L::CHUNK_BYTES;
    static constexpr int HOLDER_OFF = BAR_OFF + 8 * NBARS;  // TMEM address, abort flag, mask of keys that are not finite
    static constexpr int SUM_OFF = BAR_OFF + BAR_AREA;      // m and l of a unit's rows
    static constexpr int UNIT_OFF = SUM_OFF + 2 * TILE * 4;
    static constexpr int SMEM_BYTES = UNIT_OFF + UNITS * 64 + 1024;
    static_assert(HOLDER_OFF + 12 <= BAR_OFF + BAR_AREA, "barrier area");
    static_assert(SMEM_BYTES <= L::SMEM_LIMIT, "shared memory");
    static_assert(sizeof(Unit) == 64 && UNIT_OFF % 16 == 0, "unit ring");
    static_assert(8 * (THREADS + THREADS / 32) + THREADS * static_cast<int>(sizeof(Span)) <= NSLOTS * L::CHUNK_BYTES, "the sums of the problems' lengths");
    // ring parity across units of any lengths: as the windowed kernel's, whose order of waits this one has
    static_assert(NSLOTS >= 4 && L::NSBUF <= 3, "ring parity soundness across units");
};

// Keys [0, n) of 32 as a bit mask.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Which halves of a pair are infinities or NaN, as a mask over their bits.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    return ((w & E) == E ? 0xffffu : 0u) | ((w & (E << 16)) == (E << 16) ? 0xffff0000u : 0u);
}

// Eight words to a 32-byte boundary: a whole sector of a row.
__device__ __forceinline__ void st_global_v8(void *at, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_of(const uint32_t (&s)[32], int i)
{
    return pack2<BF16>(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
}

__device__ __forceinline__ uint64_t f2_of(const uint32_t (&s)[32], int i)
{
    return ptx::f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
}

// The values of keys pos0 + 1 + b (bit b of `odd`, all of which the row sees) that are not finite, and so were left out of
// the product, onto a row that has been written: whatever their weights, which are positive, these decide.
template <int D, bool BF16>
static __device__ __noinline__ void add_odd(const Cache16AttnParams &p, const Unit &un, uint32_t odd, char *row, bool direct)
{
    for (; odd != 0u; odd &= odd - 1u) {
        const int key = un.pos0 + __ffs(odd), page = key / p.page_size;
        const int id = p.table[un.table * p.table_stride + page];
        if (id < 0 || id >= p.num_pages)
            return;
        const uint16_t *v = p.v + ((static_cast<long long>(id) * p.Hkv + un.kv) * p.page_size + (key - page * p.page_size)) * D;
        for (int i = 0; i < D; ++i) {
            const uint32_t w = v[i];
            if (not_finite<BF16>(w) == 0u)
                continue;
            const float x = unpack16<BF16>(w).x;
            if (direct) {
                uint16_t *o = reinterpret_cast<uint16_t *>(row) + i;
                *o = static_cast<uint16_t>(pack2<BF16>(unpack16<BF16>(*o).x + x, 0.f));
            } else {
                reinterpret_cast<float *>(row)[i] += x;
            }
        }
    }
}

}  // namespace c16

template <int D, bool BF16>
__global__ void __launch_bounds__(c16::THREADS, 1)
    cache16_attn_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qo,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const Cache16AttnParams p)
{
    using namespace c16;
    using L = Layout<D>;
    using PL = Plan<D>;
    constexpr int NS = PL::NSLOTS;
    constexpr int NB = L::NSBUF;
    constexpr int CPT = PL::CPT;
    constexpr int QB = PL::QB;
    constexpr uint32_t IDESC_S = ptx::idesc_f16_f32acc(128, TILE, BF16, false);
    constexpr uint32_t IDESC_PV = ptx::idesc_f16_f32acc(128, 128, BF16, true);

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_addr + pad;
    const uint32_t s_q0 = sbase;  // query tile b at s_q0 + b * Q_BYTES
    const uint32_t s_ring = sbase + QB * L::Q_BYTES;
    const uint32_t q_full0 = sbase + PL::BAR_OFF;  // + 8 b
    const uint32_t q_free0 = q_full0 + 8u * QB;    // + 8 b: the S MMAs that read query tile b last are done
    const uint32_t slot_full0 = q_free0 + 8u * QB;
    const uint32_t slot_empty0 = slot_full0 + 8u * NS;
    const uint32_t s_full0 = slot_empty0 + 8u * NS;
    const uint32_t p_full0 = s_full0 + 8u * NB;
    const uint32_t o_done0 = p_full0 + 8u * NB;
    const uint32_t final0 = o_done0 + 8u * O_DONE_RING;
    const uint32_t o_free = final0 + 16u;     // the unit's O has been read
    const uint32_t sum_full = o_free + 8u;    // its rows' m and l are there
    const uint32_t sum_free = sum_full + 8u;
    const uint32_t odd_full = sum_free + 8u;  // the mask of its keys that are not finite is there
    const uint32_t unit_full0 = odd_full + 8u, unit_free0 = unit_full0 + 8u * PL::UNITS;  // + 8 (i % UNITS)
    float *const row_m = reinterpret_cast<float *>(smem + PL::SUM_OFF), *const row_l = row_m + TILE;
    Unit *const ring = reinterpret_cast<Unit *>(smem + PL::UNIT_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + PL::HOLDER_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile uint32_t *odd_keys = tmem_holder + 2;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int run = static_cast<int>(blockIdx.x);

    if (threadIdx.x == 0) {
        for (int b = 0; b < QB; ++b) {
            ptx::mbar_init(q_full0 + 8u * b, 1);
            ptx::mbar_init(q_free0 + 8u * b, 1);
        }
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(slot_full0 + 8u * s, 1);
            ptx::mbar_init(slot_empty0 + 8u * s, 1);
        }
        for (int i = 0; i < NB; ++i) {
            ptx::mbar_init(s_full0 + 8u * i, 1);
            ptx::mbar_init(p_full0 + 8u * i, 4);  // one arrival a softmax warp
        }
        for (int i = 0; i < O_DONE_RING; ++i)
            ptx::mbar_init(o_done0 + 8u * i, 1);
        ptx::mbar_init(final0, 1);
        ptx::mbar_init(final0 + 8u, 1);
        ptx::mbar_init(o_free, 4);
        ptx::mbar_init(sum_full, 4);
        ptx::mbar_init(sum_free, 4);
        ptx::mbar_init(odd_full, 1);
        for (int i = 0; i < PL::UNITS; ++i) {
            ptx::mbar_init(unit_full0 + 8u * i, 1);
            ptx::mbar_init(unit_free0 + 8u * i, 11);  // the warps that read it
        }
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 4 && lane == 0) {
        ptx::prefetch_tmap(&tm_qp);
        ptx::prefetch_tmap(&tm_qo);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == 5) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_holder), L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    // The join's blocks may be launched: they find no room beside a CTA of this kernel (its registers), so they start on
    // the SMs whose CTA has ended, and wait there for the last one.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- the lengths of all entries, summed up: each thread has some consecutive ones. In the ring, which is not in
    // use before the first unit is known.
    const int entries = p.ngroups + p.nseq;
    const int per = (entries + THREADS - 1) / THREADS;
    long long *const prefix = reinterpret_cast<long long *>(smem + QB * L::Q_BYTES), *const warp_sum = prefix + THREADS;
    Span *const stash = reinterpret_cast<Span *>(warp_sum + THREADS / 32);  // (of thread e's first entry, where that is e)
    {
        const int e0 = min(entries, static_cast<int>(threadIdx.x) * per), e1 = min(entries, e0 + per);
        long long sum = 0;
        for (int e = e0; e < e1; ++e) {
            const Span s = span_of(p, e);
            if (e == static_cast<int>(threadIdx.x))
                stash[e] = s;
            sum += entry_length(s);
            if (s.bad && e < p.ngroups && run == 0)
                atomicCAS(p.status, 0u, static_cast<unsigned>(SITE_SEQLENS));
        }
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(FULL, incl, d);
            if (lane >= d)
                incl += x;
        }
        prefix[threadIdx.x] = incl - sum;  // within the warp
        if (lane == 31)
            warp_sum[warp] = incl;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // A whole warp's bounded wait. The limit holds a tile: who waits for `tiles` of them waits that much longer.
    auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t site, int tiles = 1) -> bool {
        return __all_sync(FULL, ptx::mbar_try_wait(bar, parity) ||
                                    wait_slow(bar, parity, abort_flag, p.status, p.timeout_ns * tiles, site));
    };
    auto drain = [&](uint32_t bar, uint32_t parity) {  // of what this warp issued itself
        wait_drain(bar, parity, p.timeout_ns);
    };
    auto arrive = [&](uint32_t bar) {  // once a warp
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar);
    };
    auto take = [&](int i, Unit &un) -> bool {  // unit i; false at the end or when a wait ran out
        const int at = i % PL::UNITS;
        if (!wait_all(unit_full0 + 8u * at, (i / PL::UNITS) & 1, SITE_Q_FULL))
            return false;
        un = ring[at];
        arrive(unit_free0 + 8u * at);
        return un.n >= 0;
    };

    if (warp >= 4 && warp < 8) {
        if (warp == 4) {
            // ------------------------------------------------------ TMA producer
            if (!p.no_copies) {  // whole warp; one elected lane issues
                int slot = 0, last_n = 1;
                uint32_t ph = 0, armed_mask = 0, armed_par = 0, q_armed = 0, q_par = 0;
                bool ok = true;
                Unit un;
                for (int k = 0; ok && take(k, un); ++k) {
                    const int b = k % QB;
                    if (k >= QB && !(ok = wait_all(q_free0 + 8u * b, ((k - QB) / QB) & 1, SITE_Q_FULL, last_n)))
                        break;
                    last_n = un.n;
                    const int box_toks = un.prefix ? p.toks_p : p.toks_o;
                    ptx::mbar_arrive_expect_tx_w(q_full0 + 8u * b, box_toks * p.heads * D * 2);
                    const CUtensorMap *const tq = un.prefix ? &tm_qp : &tm_qo;
#pragma unroll
                    for (int c = 0; c < D / L::BOX_COLS; ++c)
                        ptx::tma_load_3d_w(s_q0 + b * L::Q_BYTES + c * L::BOX_BYTES, tq, q_full0 + 8u * b, c * L::BOX_COLS,
                                           un.head, un.q_tok);
                    q_armed |= 1u << b;
                    q_par = (q_par & ~(1u << b)) | (((k / QB) & 1u) << b);
                    // Lane i has the page of a tile's box i and the place there; boxes without a key below `hi` are not
                    // loaded. The look-ups of a tile run while the one before it is copied.
                    const int *const table = un.prefix ? p.prefix_table + un.table * p.prefix_stride
                                                       : p.table + un.table * p.table_stride;
                    struct Boxes {
                        int n, plane, off;
                    };
                    auto look_up = [&](int j) {
                        Boxes r{0, 0, 0};
                        const int tok0 = un.tile0 + j * TILE;
                        const int keys = min(un.hi - tok0, TILE);
                        if (j >= un.n || keys <= 0)
                            return r;
                        r.n = (keys + p.box - 1) / p.box;
                        if (lane < r.n) {
                            const int tok = tok0 + lane * p.box, at = tok / p.page_size;
                            int id = __ldg(table + at);
                            if (id < 0 || id >= p.num_pages) {
                                atomicCAS(p.status, 0u, kBadPages);
                                id = 0;
                            }
                            r.plane = id * p.Hkv + un.kv;
                            r.off = tok - at * p.page_size;
                        }
                        return r;
                    };
                    // K_0, then K_{t + 1} (if any) and V_t for each tile: one loop, for the sake of the instruction cache
                    Boxes next{}, last_k{}, before{};
                    int looked = 0;  // tiles looked up
#pragma unroll 1
                    for (int x = -1; ok && x < 2 * un.n; ++x) {
                        const bool of_k = x <= 0 || ((x & 1) && (x + 1) / 2 < un.n);
                        if (of_k) {
                            before = last_k;
                            last_k = next;
                            next = look_up(looked++);
                        }
                        if (x < 0)
                            continue;
                        const CUtensorMap *const map = of_k ? &tm_k : &tm_v;
                        const Boxes &t = of_k || (x == 2 * un.n - 1) ? last_k : before;
#pragma unroll 1
                        for (int ch = 0; ch < CPT; ++ch) {
                            if (!(ok = wait_all(slot_empty0 + 8u * slot, ph ^ 1u, SITE_SLOT_EMPTY)))
                                break;
                            const uint32_t full = slot_full0 + 8u * slot;
                            ptx::mbar_arrive_expect_tx_w(full, t.n * p.box * 256);
                            uint32_t dst = s_ring + slot * L::CHUNK_BYTES;
#pragma unroll 1
                            for (int i = 0; i < t.n; ++i) {
                                const int plane = __shfl_sync(FULL, t.plane, i), off = __shfl_sync(FULL, t.off, i);
                                ptx::tma_load_3d_w(dst, map, full, ch * 128, off, plane);
                                ptx::tma_load_3d_w(dst + L::BOX_BYTES, map, full, ch * 128 + L::BOX_COLS, off, plane);
                                dst += p.box * 128;
                            }
                            armed_mask |= 1u << slot;
                            armed_par = (armed_par & ~(1u << slot)) | (ph << slot);
                            if (++slot == NS) {
                                slot = 0;
                                ph ^= 1u;
                            }
                        }
                    }
                }
                // Every copy this warp issued lands before the CTA may exit.
#pragma unroll 1
                for (int b = 0; b < QB; ++b)
                    if (q_armed & (1u << b))
                        drain(q_full0 + 8u * b, (q_par >> b) & 1u);
#pragma unroll 1
                for (int s = 0; s < NS; ++s)
                    if (armed_mask & (1u << s))
                        drain(slot_full0 + 8u * s, (armed_par >> s) & 1u);
            }
        } else if (warp == 5) {
            // ------------------------------------------- S = Q K^T issuer
            const uint64_t dk = ptx::smem_desc_sw128(s_ring, 16, 1024);
            bool issued = false, ok = true;
            int g0 = 0, pos0 = 0;  // tiles and ring chunks of the earlier units
            Unit un;
            for (int k = 0; ok && take(k, un); ++k) {
                const int n = un.n, b = k % QB;
                const uint64_t dq = ptx::smem_desc_sw128(s_q0 + b * L::Q_BYTES, 16, 1024);
                if (!(ok = wait_all(q_full0 + 8u * b, (k / QB) & 1, SITE_Q_FULL)))
                    break;
                for (int t = 0; ok && t < n; ++t) {
                    const int gt = g0 + t;
                    const int p0 = pos0 + pos_k<CPT>(t);
                    if (gt >= NB) {  // buffer gt % NB held P of tile gt - NB: its PV must have read it
                        const int pv = gt - NB;
                        if (!(ok = wait_all(o_done0 + 8u * (pv % O_DONE_RING), (pv / O_DONE_RING) & 1, SITE_O_DONE)))
                            break;
                    }
                    const uint32_t d_tmem = tmem + L::TM_S + (gt % NB) * TILE;
#pragma unroll 1
                    for (int ch = 0; ch < CPT; ++ch) {
                        const int pos = p0 + ch, slot = pos % NS;
                        if (!(ok = wait_all(slot_full0 + 8u * slot, (pos / NS) & 1, SITE_SLOT_FULL)))
                            break;
                        ptx::tc_fence_after();
                        const uint64_t kslot = dk + static_cast<uint64_t>((slot * L::CHUNK_BYTES) >> 4);
                        const uint64_t qch = dq + static_cast<uint64_t>((2 * ch * L::BOX_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t off = ((kk >> 2) * L::BOX_BYTES + (kk & 3) * 32) >> 4;
                            ptx::mma_ss_w(d_tmem, qch + off, kslot + off, IDESC_S, (ch | kk) != 0);
                        }
                        issued = true;
                        ptx::mma_commit_w(slot_empty0 + 8u * slot);
                    }
                    if (!ok)
                        break;
                    ptx::mma_commit_w(s_full0 + 8u * (gt % NB));
                }
                if (!ok)
                    break;
                ptx::mma_commit_w(q_free0 + 8u * b);  // query tile b may take unit k + QB's Q
                g0 += n;
                pos0 += 2 * CPT * n;
            }
            if (issued) {  // all of this warp's MMAs complete before TMEM is freed
                ptx::mma_commit_w(final0);
                drain(final0, 0);
            }
        } else if (warp == 6) {
            // ------------------------------------------ O += P V issuer
            const uint64_t dv = ptx::smem_desc_sw128(s_ring, L::BOX_BYTES, 1024);
            bool issued = false, ok = true;
            int g0 = 0, pos0 = 0;
            Unit un;
            for (int k = 0; ok && take(k, un); ++k) {
                const int n = un.n;
                uint32_t odd = 0;     // keys that only some rows see and whose V is not finite
                uint32_t onto = 0;    // O holds something of this unit
                const int own = un.pos0 + 1;  // the first such key
                for (int j = 0; ok && j < n; ++j) {
                    const int gj = g0 + j;
                    const int buf = gj % NB;
                    const int p0 = pos0 + pos_v<CPT>(j, n);
                    if constexpr (CPT == 1) {  // V_j's slot first, off the P_j -> PV_j path
                        if (!(ok = wait_all(slot_full0 + 8u * (p0 % NS), (p0 / NS) & 1, SITE_SLOT_FULL)))
                            break;
                    }
                    if (!(ok = wait_all(p_full0 + 8u * buf, (gj / NB) & 1, SITE_P_FULL)))
                        break;
                    // a unit's first PV overwrites O: the previous unit's rows must have been read
                    if (j == 0 && k > 0 && !(ok = wait_all(o_free, (k - 1) & 1, SITE_O_DONE)))
                        break;
                    ptx::tc_fence_after();
                    // Rows of the tile that hold keys. The product takes the steps of 16 rows that have any; what else these
                    // hold, before the first key or behind the last, is zeroed.
                    const int key0 = un.tile0 + j * TILE;
                    const int r0 = max(0, un.lo - key0), r1 = min(TILE, un.hi - key0);
                    const int kk0 = r0 / 16, kk1 = r1 > r0 ? (r1 + 15) / 16 : 0;
                    const bool ragged = r1 > r0 && ((r0 | r1) & 15) != 0;
                    const int a0 = max(r0, own - key0), a1 = un.prefix || p.n == 1 ? 0 : r1;  // keys that some rows do not see
                    const uint32_t a_tmem = tmem + L::TM_S + buf * TILE;
#pragma unroll 1
                    for (int ch = 0; ch < CPT; ++ch) {
                        const int pos = p0 + ch;
                        const int slot = pos % NS;
                        if constexpr (CPT != 1) {
                            if (!(ok = wait_all(slot_full0 + 8u * slot, (pos / NS) & 1, SITE_SLOT_FULL)))
                                break;
                            ptx::tc_fence_after();
                        }
                        if (ragged || a1 > a0) {
                            const uint32_t at = s_ring + slot * L::CHUNK_BYTES;
                            const int half = lane >> 4;  // a row's 256 bytes by 16 lanes
                            const uint32_t unit = ((lane >> 3) & 1) * L::BOX_BYTES + (lane & 7) * 16;
                            for (int r = kk0 * 16 + half; r < r0; r += 2)
                                st_shared_v4(at + r * 128 + unit, 0u, 0u, 0u, 0u);
                            for (int r = r1 + half; r < kk1 * 16; r += 2)
                                st_shared_v4(at + r * 128 + unit, 0u, 0u, 0u, 0u);
                            for (int r = a0; r < a1; r += 2) {
                                uint32_t w[4], x[4], any = 0;
                                const uint32_t addr = at + min(r + half, a1 - 1) * 128 + unit;
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                             : "r"(addr));
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    x[i] = not_finite<BF16>(w[i]);
                                    any |= x[i];
                                }
                                const unsigned hit = __ballot_sync(FULL, any != 0u);
                                if (hit != 0u) {
                                    if (any != 0u && r + half < a1)
                                        st_shared_v4(addr, w[0] & ~x[0], w[1] & ~x[1], w[2] & ~x[2], w[3] & ~x[3]);
                                    const int bit = key0 + r - own;  // 0 .. 30
                                    if (hit & 0xffffu)
                                        odd |= 1u << bit;
                                    if ((hit >> 16) != 0u && r + 1 < a1)
                                        odd |= 1u << (bit + 1);
                                }
                            }
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                        }
                        const uint64_t vslot = dv + static_cast<uint64_t>((slot * L::CHUNK_BYTES) >> 4);
                        if (kk0 == 0 && kk1 == 8) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                ptx::mma_ts_w(tmem + L::TM_O + ch * 128, a_tmem + kk * 8, vslot + ((kk * 2048) >> 4), IDESC_PV,
                                              kk == 0 ? onto : 1u);
                        } else {
#pragma unroll 1
                            for (int kk = kk0; kk < kk1; ++kk)
                                ptx::mma_ts_w(tmem + L::TM_O + ch * 128, a_tmem + kk * 8, vslot + ((kk * 2048) >> 4), IDESC_PV,
                                              onto | (kk > kk0 ? 1u : 0u));
                        }
                        issued = true;
                        ptx::mma_commit_w(slot_empty0 + 8u * slot);
                    }
                    if (!ok)
                        break;
                    onto |= kk1 > kk0 ? 1u : 0u;
                    ptx::mma_commit_w(o_done0 + 8u * (gj % O_DONE_RING));
                }
                if (!ok)
                    break;
                if (lane == 0)
                    *odd_keys = odd;  // the last unit's has been read: its O is free
                arrive(odd_full);
                g0 += n;
                pos0 += 2 * CPT * n;
            }
            if (issued) {
                ptx::mma_commit_w(final0 + 8u);
                drain(final0 + 8u, 0);
            }
        } else {
            // ------------------------------------------ the run's units, ahead of the other warps
            long long total = 0, before = 0;
#pragma unroll
            for (int i = 0; i < THREADS / 32; ++i)
                total += warp_sum[i];
            const Cut cut(total, gridDim.x);
            long long off = 0, left = 0;  // position in the entry's problems, positions left in the run
            int e = 0;
            if (run < cut.n) {
                const long long x = cut.start(run);
                left = cut.start(run + 1) - x;
                int w0 = 0;  // the last thread whose entries start at or before x
                while (before + warp_sum[w0] <= x)
                    before += warp_sum[w0++];
                const unsigned at = __ballot_sync(FULL, before + prefix[w0 * 32 + lane] <= x);
                const int owner = w0 * 32 + 31 - __clz(at);
                off = x - before - prefix[owner];
                e = owner * per;
            }
            int base = -32;  // the lanes have entries base .. base + 31
            bool fresh = true;  // the next problem is the one at `off` of entry e, else those below say which
            int u = 0, in = 0, b = 0, blocks = 1, heads = 0, hb = 0, kv = 0;
            const int blocks_p = (p.n + p.toks_p - 1) / p.toks_p, all_heads = p.Hkv * p.head_blocks;
            Span mine{};
            int longest = 1;  // of the units so far: its end may be what a place in the ring waits for
            for (int i = 0;; ++i) {
                Unit un;
                un.n = -1;
                bool first_run = false;
                int tiles_after = 0;
                int2 *join = nullptr;
                while (left > 0) {
                    if (e >= base + 32) {
                        const int at = min(e + lane, entries - 1);
                        mine = base < 0 && per == 1 ? stash[at] : span_of(p, at);  // (later the ring is in use)
                        base = e;
                    }
                    const int from = e - base;
                    const int tiles = __shfl_sync(FULL, mine.tiles, from), problems = __shfl_sync(FULL, mine.problems, from);
                    const int len = tiles + OVERHEAD;
                    if (fresh) {  // which of the entry's problems the run begins with
                        if (tiles == 0 || off >= static_cast<long long>(len) * problems) {
                            off -= tiles == 0 ? 0 : static_cast<long long>(len) * problems;
                            ++e;  // the positions left exist: an entry follows
                            continue;
                        }
                        u = off <= 0x7fffffffll ? static_cast<int>(off) / len : static_cast<int>(off / len);
                        in = static_cast<int>(off - static_cast<long long>(u) * len);
                        off = 0;
                    }
                    const int first = __shfl_sync(FULL, mine.first, from), toks = __shfl_sync(FULL, mine.toks, from);
                    un.prefix = e < p.ngroups;
                    const int block = un.prefix ? p.toks_p : p.toks_o;
                    if (fresh) {
                        blocks = (toks + block - 1) / block;
                        b = u % blocks;
                        heads = u / blocks;
                        kv = heads / p.head_blocks;
                        hb = heads - kv * p.head_blocks;
                        fresh = false;
                    }
                    // the problem's positions [in, in + take_n)
                    const int take_n = static_cast<int>(min(left, static_cast<long long>(len - in)));
                    const int t0 = max(0, in - OVERHEAD), t1 = in + take_n - OVERHEAD;
                    left -= take_n;
                    const int lo = __shfl_sync(FULL, mine.lo, from), hi = __shfl_sync(FULL, mine.hi, from);
                    const int k0 = __shfl_sync(FULL, mine.k0, from);
                    un.kv = kv;
                    un.n = t1 - t0;
                    un.tile0 = k0 + t0 * TILE;
                    un.lo = lo;
                    un.q_tok = first + b * block;
                    un.toks = min(block, toks - b * block);
                    un.head = un.kv * p.G + hb * p.heads;
                    un.live = min(p.heads, p.G - hb * p.heads);
                    un.table = un.prefix ? e : e - p.ngroups;
                    un.pos0 = un.prefix ? hi - 1 : hi - p.n + b * block;
                    // no row of the block sees a key behind its last token's own
                    un.hi = un.prefix ? hi : min(hi, un.pos0 + un.toks);
                    const bool whole = t0 == 0 && t1 == tiles;
                    const bool joined = un.prefix || lo > 0;
                    un.dest = !whole ? 2 * run + (t0 == 0 ? 1 : 0) : joined ? DEST_ROWS : DEST_DIRECT;
                    first_run = t0 == 0;
                    tiles_after = tiles - t1;
                    join = un.prefix ? p.joins_p : p.joins_o;
                    join += (static_cast<long long>(un.prefix ? first / p.n * blocks_p : un.table * p.blocks_o) + b) * all_heads + heads;
                    // on to the next problem, where the run has positions left
                    in = 0;
                    kv = un.kv;
                    if (++b == blocks) {
                        b = 0;
                        ++heads;
                        if (++hb == p.head_blocks) {
                            hb = 0;
                            ++kv;
                        }
                    }
                    if (kv == p.Hkv) {
                        fresh = true;
                        ++e;
                    }
                    if (un.n <= 0) {  // the run ends inside the problem's start
                        un.n = -1;
                        continue;
                    }
                    break;
                }
                const int at = i % PL::UNITS;
                if (i >= PL::UNITS && !wait_all(unit_free0 + 8u * at, (i / PL::UNITS - 1) & 1, SITE_Q_FULL, longest))
                    break;
                longest = max(longest, un.n);
                if (lane == 0) {
                    ring[at] = un;
                    ptx::mbar_arrive(unit_full0 + 8u * at);
                    if (un.n >= 0 && first_run)  // for the join; the problem's last tile lies in this run or in one after it
                        *join = make_int2(run, tiles_after == 0 ? 1 : cut.run_of(cut.start(run + 1) + tiles_after - 1) - run + 1);
                }
                if (un.n < 0)
                    break;
            }
        }
    } else if (warp < 4) {
        // --------------------------------------- softmax / correction
        const int row = threadIdx.x;  // row within the tile = TMEM lane
        const int row_tok = row / p.heads, row_head = row - row_tok * p.heads;
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t t_s = tmem + lane_off + L::TM_S;
        const uint32_t t_o = tmem + lane_off + L::TM_O;
        const float c = p.c;  // not 0
        const uint64_t c2 = ptx::f2_pack(c, c);
        const uint32_t unseen = c > 0.f ? 0xff800000u : 0x7f800000u;  // -inf or inf
        bool ok = true;
        int g0 = 0;
        Unit un;
        for (int k = 0; ok && take(k, un); ++k) {
            const int n = un.n;
            const bool idle = warp * 32 >= un.toks * p.heads;  // no live row in the warp
            const bool dead = row_tok >= un.toks || row_head >= un.live;
            // the row sees keys [lo, pos]
            const int pos = min(un.hi - 1, un.prefix ? un.pos0 : un.pos0 + row_tok);
            float m_used = -INFINITY, l = 0.f;
            bool s_seen = false;  // S_j's barrier was seen complete while tile j-1 ended
            for (int j = 0; j < n; ++j) {
                const int gj = g0 + j;
                const int buf = gj % NB;
                if (!__all_sync(FULL, s_seen)) {
                    if (!(ok = wait_all(s_full0 + 8u * buf, (gj / NB) & 1, SITE_S_FULL)))
                        break;
                }
                s_seen = false;
                if (idle) {  // whatever its lanes of P hold meets no other row
                    arrive(p_full0 + 8u * buf);
                    continue;
                }
                ptx::tc_fence_after();
                const uint32_t ts = t_s + buf * TILE;
                // Columns [w0, w1) hold the tile's keys: the product takes no others.
                const int k0 = un.tile0 + j * TILE;
                const int w0 = max(0, un.lo - k0) & -64, w1 = min(TILE, (un.hi - k0 + 63) & -64);
                // Scores of keys that a row does not see become -inf (times c)
                const int hi = pos + 1 - k0, lo = un.lo - k0;
                if (__any_sync(FULL, hi < w1 || lo > w0)) {
#pragma unroll 1
                    for (int w = w0; w < w1; w += 32) {
                        const uint32_t vis = below(hi - w) & ~below(lo - w);
                        if (__all_sync(FULL, vis == 0xffffffffu))
                            continue;
                        uint32_t s[32];
                        ptx::tmem_ld32(ts + w, s);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            s[i] = (vis & (1u << i)) ? s[i] : unseen;
                        ptx::tmem_st32(ts + w, s);
                    }
                    ptx::tmem_wait_st();
                }
                // Two passes over the tile, 32 scores at a time, the next ones on their way meanwhile.
                uint32_t a[32], b[32];
                auto largest = [&](const uint32_t (&s)[32], float &mx0, float &mx1) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float x0, x1, x2, x3;
                        ptx::f2_unpack(mul2(f2_of(s, i), c2), x0, x1);
                        ptx::f2_unpack(mul2(f2_of(s, i + 2), c2), x2, x3);
                        mx0 = ptx::max3(mx0, x0, x1);
                        mx1 = ptx::max3(mx1, x2, x3);
                    }
                };
                float mx0 = -INFINITY, mx1 = -INFINITY;
                if (w0 < w1)
                    ptx::tmem_ld32(ts + w0, a);
#pragma unroll 1
                for (int w = w0; w < w1; w += 64) {
                    ptx::tmem_wait_ld();
                    ptx::tmem_ld32(ts + w + 32, b);
                    largest(a, mx0, mx1);
                    ptx::tmem_wait_ld();
                    ptx::tmem_ld32(ts + (w + 64 < w1 ? w + 64 : w0), a);  // (the second pass begins with the first scores)
                    largest(b, mx0, mx1);
                }
                // -inf while the row has seen no key (and its weights are 2^(-inf - 0) = 0); a dead row's maximum stays there
                const float m_tile = fmaxf(mx0, mx1);
                const float m_new = !dead && m_tile > m_used + RESCALE_THRESHOLD ? m_tile : m_used;
                const float alpha = m_new == m_used ? 1.f : ptx::ex2(m_used - m_new);
                const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
                const uint64_t negm2 = ptx::f2_pack(neg_m, neg_m);
                uint64_t sum01 = ptx::f2_pack(0.f, 0.f), sum23 = sum01;
                auto weights = [&](const uint32_t (&s)[32], uint32_t to) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float x0, x1, x2, x3;
                        ptx::f2_unpack(ptx::f2_fma(f2_of(s, 2 * i), c2, negm2), x0, x1);
                        ptx::f2_unpack(ptx::f2_fma(f2_of(s, 2 * i + 2), c2, negm2), x2, x3);
                        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1), p2 = ptx::ex2(x2), p3 = ptx::ex2(x3);
                        sum01 = ptx::f2_add(sum01, ptx::f2_pack(p0, p1));
                        sum23 = ptx::f2_add(sum23, ptx::f2_pack(p2, p3));
                        pk[i] = pack2<BF16>(p0, p1);
                        pk[i + 1] = pack2<BF16>(p2, p3);
                    }
                    ptx::tmem_st16(to, pk);  // P overwrites scores that both passes have read
                };
#pragma unroll 1
                for (int w = w0; w < w1; w += 64) {
                    ptx::tmem_wait_ld();
                    ptx::tmem_ld32(ts + w + 32, b);
                    weights(a, ts + w / 2);
                    ptx::tmem_wait_ld();
                    if (w + 64 < w1)
                        ptx::tmem_ld32(ts + w + 64, a);
                    weights(b, ts + w / 2 + 16);
                }
                // Poll S_{j+1}'s barrier now (same unit), so the answer returns while P_j is stored and handed off.
                s_seen = j + 1 < n && ptx::mbar_test_wait(s_full0 + 8u * ((gj + 1) % NB), ((gj + 1) / NB) & 1);
                float sum0, sum1, sum2, sum3;
                ptx::f2_unpack(sum01, sum0, sum1);
                ptx::f2_unpack(sum23, sum2, sum3);
                ptx::tmem_wait_st();
                l = fmaf(l, alpha, (sum0 + sum1) + (sum2 + sum3));

                // Rescale O only in warps where some row's maximum moved (they wait for PV_{gj-1}).
                if (j > 0 && __any_sync(FULL, alpha != 1.f)) {
                    const int pv = gj - 1;
                    if (!(ok = wait_all(o_done0 + 8u * (pv % O_DONE_RING), (pv / O_DONE_RING) & 1, SITE_O_DONE)))
                        break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        ptx::tmem_ld32(t_o + 32 * cc, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        ptx::tmem_st32(t_o + 32 * cc, o);
                    }
                    ptx::tmem_wait_st();
                }
                ptx::tc_fence_before();
                arrive(p_full0 + 8u * buf);
                m_used = m_new;
            }
            if (!ok)
                break;
            if (k > 0 && !(ok = wait_all(sum_free, (k - 1) & 1, SITE_O_DONE)))
                break;
            row_m[row] = m_used;
            row_l[row] = l;
            arrive(sum_full);
            g0 += n;
        }
    } else {
        // --------------------------------------- rows' ends: O over l, to the output or to the workspace
        const int w4 = warp & 3, row = w4 * 32 + lane;
        const int row_tok = row / p.heads, row_head = row - row_tok * p.heads;
        const uint32_t t_o = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + L::TM_O;
        bool ok = true;
        int g0 = 0;
        Unit un;
        for (int k = 0; ok && take(k, un); ++k) {
            const int n = un.n, last = g0 + n - 1;
            if (!(ok = wait_all(sum_full, k & 1, SITE_O_DONE, n)))
                break;
            const float m = row_m[row], l = row_l[row];
            arrive(sum_free);
            if (!(ok = wait_all(o_done0 + 8u * (last % O_DONE_RING), (last / O_DONE_RING) & 1, SITE_O_DONE)) ||
                !(ok = wait_all(odd_full, k & 1, SITE_O_DONE)))
                break;
            const uint32_t odd = *odd_keys;
            if (w4 * 32 < un.toks * p.heads) {
                ptx::tc_fence_after();
                const bool none = l == 0.f;  // the row saw no key
                const float inv = 1.f / l;
                // the row of q and o, -1 where there is none
                const int at = row_tok < un.toks && row_head < un.live ? (un.q_tok + row_tok) * p.Hq + un.head + row_head : -1;
                const bool slot = un.dest >= 0, direct = un.dest == DEST_DIRECT;
                float *const part = slot ? p.parts + un.dest * part_floats<D>(p.part_rows) : un.prefix ? p.rows_p : p.rows_o;
                char *const to = direct ? reinterpret_cast<char *>(p.o + static_cast<long long>(at) * D)
                                        : reinterpret_cast<char *>(part + static_cast<long long>(slot ? row : at) * D);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    ptx::tmem_ld32(t_o + c0, o);
                    ptx::tmem_wait_ld();
                    if (at >= 0) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = none ? 0u : __float_as_uint(__uint_as_float(o[x]) * inv);
                        if (direct) {
#pragma unroll
                            for (int x = 0; x < 32; x += 8)
                                reinterpret_cast<uint4 *>(to + 2 * c0)[x / 8] = make_uint4(
                                    pack_of<BF16>(o, x), pack_of<BF16>(o, x + 2), pack_of<BF16>(o, x + 4), pack_of<BF16>(o, x + 6));
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; x += 8)
                                st_global_v8(to + 4 * (c0 + x), &o[x]);
                        }
                    }
                    __syncwarp();
                }
                ptx::tc_fence_before();
                arrive(o_free);
                if (at >= 0) {
                    if (odd != 0u)
                        add_odd<D, BF16>(p, un, odd & below(row_tok), to, direct);
                    if (direct) {
                        if (p.lse != nullptr)
                            p.lse[at] = none ? -INFINITY : (m + log2f(l)) * LN2;
                    } else if (slot) {
                        part[static_cast<long long>(p.part_rows) * D + row] = m;
                        part[static_cast<long long>(p.part_rows) * (D + 1) + row] = l;
                    } else {
                        reinterpret_cast<float2 *>(part + static_cast<long long>(p.nseq) * p.n * p.Hq * D)[at] = make_float2(m, l);
                    }
                }
            } else {
                arrive(o_free);
            }
            g0 += n;
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// Adds up the parts of every row that has more than one, the prefix's first, in the order of the runs, and writes the
// rows that see nothing. A row by the eight warps of a block, every eighth part each, so that a long problem's parts are
// read at once; or (ONE, with many rows, of a few parts each) a row a warp.
template <int D, bool BF16, bool ONE>
__global__ void __launch_bounds__(c16::MERGE_THREADS) cache16_join_kernel(const Cache16AttnParams p, int runs)
{
    using namespace c16;
    constexpr int WARPS = MERGE_THREADS / 32, V = D / 128;  // V float4 a lane
    __shared__ float4 y_all[ONE ? 1 : WARPS][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long all = static_cast<long long>(p.nseq) * p.n * p.Hq;
    const long long row = ONE ? static_cast<long long>(blockIdx.x) * WARPS + warp : blockIdx.x;
    const bool in = row < all;
    const int tok = in ? static_cast<int>(row / p.Hq) : 0, head = in ? static_cast<int>(row - static_cast<long long>(tok) * p.Hq) : 0;
    const int s = tok / p.n;
    const int kv = head / p.G, hb = (head - kv * p.G) / p.heads, h = head - kv * p.G - hb * p.heads;
    const Span sp = span_of(p, p.ngroups + s);
    const int t = tok - s * p.n, heads = kv * p.head_blocks + hb, all_heads = p.Hkv * p.head_blocks;
    // the row's place in its two problems
    const int2 *join_o = nullptr, *join_p = nullptr;
    int row_o = 0, row_p = 0;
    if (sp.tiles > 0) {
        const int b = t / p.toks_o;
        join_o = p.joins_o + (static_cast<long long>(s) * p.blocks_o + b) * all_heads + heads;
        row_o = (t - b * p.toks_o) * p.heads + h;
    }
    if (sp.lo > 0) {
        const int first = group_range(p, share_of(p, s).g).x, at = tok - first * p.n, b = at / p.toks_p;
        join_p = p.joins_p + (static_cast<long long>(first) * ((p.n + p.toks_p - 1) / p.toks_p) + b) * all_heads + heads;
        row_p = (at - b * p.toks_p) * p.heads + h;
    }
    // What is above runs beside the attention's end. Every thread waits for that end: what follows on the
    // stream waits for this kernel alone.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!in)
        return;
    if (sp.hi == 0) {
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
    const int2 jo = join_o != nullptr ? *join_o : make_int2(0, 0), jp = join_p != nullptr ? *join_p : make_int2(0, 0);
    // written already; or a word was never written (a wait ran out, and the status says so)
    if (join_p == nullptr && jo.y == 1)
        return;
    if (jo.y < (join_o != nullptr ? 1 : 0) || jo.x < 0 || jo.y > runs - jo.x || jp.y < (join_p != nullptr ? 1 : 0) ||
        jp.x < 0 || jp.y > runs - jp.x)
        return;
    const int parts = jp.y + jo.y;
    struct Part {
        const float *o;
        float m, l;
    };
    auto part = [&](int x) {
        const bool of_p = x < jp.y;
        const int2 j = of_p ? jp : jo;
        Part r;
        if (j.y == 1) {  // whole: by rows of q
            const float *at = of_p ? p.rows_p : p.rows_o;
            const float2 ml = reinterpret_cast<const float2 *>(at + all * D)[row];
            r.o = at + row * D;
            r.m = ml.x;
            r.l = ml.y;
        } else {  // the first begins the problem (slot 1 of its run), the others continue it (slot 0)
            const int i = of_p ? x : x - jp.y, r0 = of_p ? row_p : row_o;
            const float *at = p.parts + (2LL * (j.x + i) + (i == 0 ? 1 : 0)) * part_floats<D>(p.part_rows);
            r.o = at + static_cast<long long>(r0) * D;
            r.m = at[static_cast<long long>(p.part_rows) * D + r0];
            r.l = at[static_cast<long long>(p.part_rows) * (D + 1) + r0];
        }
        return r;
    };
    // every warp finds the maximum and the sum for itself
    const Part mine = part(min(lane, parts - 1));
    float mx = mine.m;
    for (int x = lane + 32; x < parts; x += 32)
        mx = fmaxf(mx, part(x).m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
    // 1: the part holds 0, or NaN
    auto weight = [&](const Part &a) { return (a.m == -INFINITY ? 1.f : ptx::ex2(a.m - mx)) * a.l; };
    float sum = lane < parts ? weight(mine) : 0.f;
    for (int x = lane + 32; x < parts; x += 32)
        sum += weight(part(x));
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
        const Part a = part(x);
        const float4 *src = reinterpret_cast<const float4 *>(a.o);
        const float f = weight(a) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float4 w = src[i * 32 + lane];
            y[i].x = fmaf(f, w.x, y[i].x);
            y[i].y = fmaf(f, w.y, y[i].y);
            y[i].z = fmaf(f, w.z, y[i].z);
            y[i].w = fmaf(f, w.w, y[i].w);
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
                const float4 x = y_all[w][i * 32 + lane];
                y[i].x += x.x;
                y[i].y += x.y;
                y[i].z += x.z;
                y[i].w += x.w;
            }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        reinterpret_cast<uint2 *>(p.o + row * D)[i * 32 + lane] =
            make_uint2(pack16<BF16>(y[i].x, y[i].y), pack16<BF16>(y[i].z, y[i].w));
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * LN2;
}

struct Cache16Maps {
    CUtensorMap q_prefix, q_own, k, v;
};

template <int D, bool BF16>
cudaError_t launch_cache16_attn(const Cache16Maps &m, const Cache16AttnParams &p, int sms, cudaStream_t st)
{
    using PL = c16::Plan<D>;
    static unsigned long long done = 0;
    auto kern = cache16_attn_kernel<D, BF16>;
    cudaError_t e = set_smem_once(kern, PL::SMEM_BYTES, done);
    if (e != cudaSuccess)
        return e;
    kern<<<sms, c16::THREADS, PL::SMEM_BYTES, st>>>(m.q_prefix, m.q_own, m.k, m.v, p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    // the blocks of the join start where the attention's CTAs end, not when the last one has
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    const long long rows = static_cast<long long>(p.nseq) * p.n * p.Hq;
    constexpr int WARPS = c16::MERGE_THREADS / 32;
    const bool one = rows >= 2LL * sms * WARPS;  // a row a warp once that still gives every SM two blocks
    config.gridDim = dim3(static_cast<unsigned>(one ? (rows + WARPS - 1) / WARPS : rows));
    config.blockDim = dim3(c16::MERGE_THREADS);
    config.stream = st;
    config.attrs = &early;
    config.numAttrs = 1;
    return one ? cudaLaunchKernelEx(&config, cache16_join_kernel<D, BF16, true>, p, sms)
               : cudaLaunchKernelEx(&config, cache16_join_kernel<D, BF16, false>, p, sms);
}

// One per (head dim, dtype).
cudaError_t cache16_attn_d128_fp16(const Cache16Maps &m, const Cache16AttnParams &p, int sms, cudaStream_t st);
cudaError_t cache16_attn_d128_bf16(const Cache16Maps &m, const Cache16AttnParams &p, int sms, cudaStream_t st);
cudaError_t cache16_attn_d256_fp16(const Cache16Maps &m, const Cache16AttnParams &p, int sms, cudaStream_t st);
cudaError_t cache16_attn_d256_bf16(const Cache16Maps &m, const Cache16AttnParams &p, int sms, cudaStream_t st);

}  // namespace sdp
