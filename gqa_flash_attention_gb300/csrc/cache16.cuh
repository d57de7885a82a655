// The attention over the paged 16-bit cache (sdp_fwd_cache16): what its kernels share. cache16_attn.cuh says how
// they work together.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "sdp_internal.h"
#include "sixteen.cuh"

namespace sdp {

struct Cache16Params {
    uint16_t *o;
    float *lse;
    const uint16_t *v;  // the pool (read directly where a value is not finite)
    const int *table, *lens, *prefix_table, *prefix_lens, *cu_groups;
    long long table_stride, prefix_stride;
    int num_pages, page_size, max_pages, prefix_pages;
    unsigned page_inverse;  // of page_size / 16, times 2^32
    int nseq, ngroups, n, Hq, Hkv, G;
    // query heads of a block (G, or 128 of a larger group), blocks of them a KV head; tokens of a block, of a prefix and of a
    // sequence; blocks of a sequence's n tokens, by its own problems and by a prefix's
    int heads, head_blocks, toks_p, toks_o, blocks_o, blocks_p;
    int box, box_log2;  // keys of a TMA box, a power of two of which lie in one page (of V: not more than a slot's)
    int sms;
    int part_rows;            // rows of a part in the workspace
    float *parts;             // two a run: the problem it continues and the one it begins
    float *rows_o, *rows_p;   // [nseq * n * Hq][D], then (m, l) of each: problems that one run holds whole
    int2 *joins_o, *joins_p;  // of each problem its first run and its parts (1: whole)
    unsigned int *status;
    unsigned long long timeout_ns;
    int no_copies, no_units;  // test hooks: no copy is issued, no unit is published; every wait runs out
    float c;        // scale * log2(e), not 0
};

namespace c16 {

constexpr int TILE = 128;    // keys of a tile
// Tiles that a problem's start and end cost as much as. (1, 2, 3: 60 in four groups 56.0, 56.1, 56.6 us, 129 sequences of 30 keys
// behind 5851, D = 128, 39, 43, 49; 256 x 16k at D = 256 129.6, 132.7 with 1 and 2, 205 of 100 keys there 74, 70.)
constexpr int OVERHEAD = 1;
constexpr unsigned FULL = 0xffffffffu;
// How far behind a problem's last key the first key of a box is formed: boxes are looked up 32 at a time, from a tile that has
// keys on, and have TILE keys at most. All keys that tables and prefixes could hold end that much below 2^31.
constexpr int KEYS_BEHIND = 32 * TILE;

// What a CTA's waits share, in shared memory.
struct Waits {
    unsigned long long timeout_ns;
    unsigned int *status;
    volatile int abort;
};

// A whole warp's bounded wait for the phase of `bar` with that parity; false when the CTA is given up. The limit holds a tile:
// who waits for `tiles` of them waits that much longer. But for the first look it is out of line, like all that is not in
// a tile's own way: what the warps of a CTA run at the same time has to fit the instruction cache. (Unrolled and
// inlined, 200 KB of code in all, a tile took 6400 cycles at D = 256 instead of 3600, most of them instruction fetches.)
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, Waits *w, uint32_t site, int tiles)
{
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(FULL, ptx::mbar_try_wait(bar, parity)))
            return true;
        if ((it & 15u) != 0)
            continue;
        const bool late = ptx::globaltimer_ns() - t0 > w->timeout_ns * tiles;
        if (__any_sync(FULL, late || w->abort)) {
            if (late) {
                w->abort = 1;
                const uint32_t cta = blockIdx.x < 0xFFFFFFu ? blockIdx.x : 0xFFFFFFu;
                atomicCAS(w->status, 0u, site | (cta << 8));
            }
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, Waits *w, uint32_t site, int tiles)
{
    return __all_sync(FULL, ptx::mbar_try_wait(bar, parity)) || wait_long(bar, parity, w, site, tiles);
}

// Waits for what this warp issued itself, which always completes.
static __device__ __noinline__ void wait_own(uint32_t bar, uint32_t parity, Waits *w)
{
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity) && ptx::globaltimer_ns() - t0 <= w->timeout_ns) {
    }
}

// A group that a sequence shares a prefix with: the prefix's length, 0 for none.
struct Share {
    int g, P;
    bool bad;
};

__device__ __forceinline__ int2 group_range(const Cache16Params &p, int g)
{
    return p.cu_groups == nullptr ? make_int2(0, p.nseq) : make_int2(__ldg(p.cu_groups + g), __ldg(p.cu_groups + g + 1));
}

// The prefix of group g, whose sequences are [r.x, r.y). A single sequence's is read from the prefix's pages too: its own need
// not hold it, and how many sequences a group has is known on the device alone.
__device__ __forceinline__ Share prefix_of(const Cache16Params &p, int g, int2 r)
{
    const int P = __ldg(p.prefix_lens + g);
    const bool order = 0 <= r.x && r.x <= r.y && r.y <= p.nseq;
    Share s{g, 0, !order || P < 0 || P > p.prefix_pages * p.page_size};  // the host keeps the product in 31 bits
    if (!s.bad && r.y > r.x)
        s.P = P;
    return s;
}

__device__ __forceinline__ Share share_of(const Cache16Params &p, int s)
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
// [lo, hi) in `tiles` tiles from key k0, for each KV head and each block of its heads and of the tokens.
struct Span {
    int tiles, problems;
    int lo, hi, k0;
    int seq, toks, blocks;  // the first sequence, the tokens of q, and their blocks
    bool bad;
};

// (Inline: out of line, the parameters would be read through memory, which they reach cold.)
__device__ __forceinline__ Span span_of(const Cache16Params &p, int e)
{
    Span r{};
    int block;
    if (e < p.ngroups) {
        const int2 at = group_range(p, e);
        const Share s = prefix_of(p, e, at);
        r.bad = s.bad;
        r.hi = s.P;
        r.seq = at.x;
        r.toks = s.P > 0 ? (at.y - at.x) * p.n : 0;
        block = p.toks_p;
    } else {
        const int s = e - p.ngroups, len = __ldg(p.lens + s);
        const Share a = share_of(p, s);
        r.bad = len < 0 || len > p.max_pages * p.page_size;  // (the join reports it, and leaves the rows)
        r.hi = r.bad ? 0 : len;
        // a sequence whose first row does not see the whole prefix goes through its own pages
        r.lo = a.P > 0 && r.hi >= a.P + p.n - 1 ? a.P : 0;
        r.seq = s;
        r.toks = p.n;
        block = p.toks_o;
    }
    r.blocks = (r.toks + block - 1) / block;
    r.problems = p.Hkv * p.head_blocks * r.blocks;
    r.k0 = r.lo & -p.box;
    r.tiles = r.hi > r.lo ? (r.hi - r.k0 + TILE - 1) / TILE : 0;
    return r;
}

// The host keeps the positions of all entries, and so an entry's, in 31 bits. (Offsets of groups that are not in order could
// pass that all the same: sums stop there.)
constexpr unsigned MOST = 0x7fffffffu;

__device__ __forceinline__ unsigned entry_length(const Span &s)
{
    return s.tiles > 0 ? static_cast<unsigned>(s.problems) * static_cast<unsigned>(s.tiles + OVERHEAD) : 0u;
}

// Positions cut into n runs: run i begins at floor(total * i / n).
struct Cut {
    unsigned total, q, r, n;
    __device__ __forceinline__ Cut(unsigned positions, unsigned most) : total(positions)
    {
        n = min(total, most);
        q = total / max(n, 1u);
        r = total - q * n;
    }
    __device__ __forceinline__ unsigned start(unsigned i) const { return i * q + i * r / n; }
    // The run of position x. (Once a problem that several runs share, out of a tile's way.)
    __device__ __forceinline__ int run_of(unsigned x) const
    {
        return static_cast<int>((static_cast<unsigned long long>(x + 1) * n - 1) / total);
    }
};

constexpr int DEST_DIRECT = -1, DEST_ROWS = -2;  // else the part's number

// A unit: a run's tiles of one problem. n < 0: none, nor any after it.
struct __align__(16) Unit {
    int n, tile0;       // tiles, and the first one's first key
    int lo, hi;         // keys that a row may see
    int q_tok, toks;    // the block's first token in q, and its tokens
    int head, live;     // its first query head, and its heads
    int kv, pos0;       // the KV head; position of the first token (of a prefix: hi - 1, every row's)
    int table;          // row of the block table, or ~ of the prefixes'
    int dest;
    int join, after;  // if it begins the problem: where the join finds what became of that (else -1), and the tiles that other runs have
    int unused[2];
    __device__ __forceinline__ bool prefix() const { return table < 0; }
};

// The sum of the lanes up to one's own, MOST at most.
__device__ __forceinline__ unsigned sum_to_lane(unsigned x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(FULL, x, d);
        x = min(x + (lane >= d ? y : 0u), MOST);
    }
    return x;
}

// The runs, as a CTA sees them: `begin` by all threads of the CTA, `start` and `next` by one warp.
template <int THREADS>
struct Runs {
    // What `begin` leaves in shared memory for `start`, where the copies' ring is later: the warp that reads it is the one that lets
    // copies begin.
    struct Shared {
        unsigned prefix[THREADS];
        Span first[THREADS];  // thread e's first entry, where that is e
    };
    int entries, per;
    Cut cut{0, 1};
    unsigned upto;  // lane w: the entries' lengths before warp w's

    // The lengths of all entries, summed up: each thread has some consecutive ones. `sums` has a word a warp, which every warp
    // reads behind the only __syncthreads(), when another may be copying already: no copy lands there.
    __device__ __forceinline__ void begin(const Cache16Params &p, Shared &sh, unsigned *sums)
    {
        const int tid = threadIdx.x, lane = tid & 31;
        entries = p.ngroups + p.nseq;
        per = (entries + THREADS - 1) / THREADS;
        const int e0 = min(entries, tid * per), e1 = min(entries, e0 + per);
        unsigned sum = 0;
#pragma unroll 1
        for (int e = e0; e < e1; ++e) {
            const Span s = span_of(p, e);
            if (e == tid)
                sh.first[e] = s;
            sum = min(sum + entry_length(s), MOST);
            if (s.bad && e < p.ngroups && blockIdx.x == 0)
                atomicCAS(p.status, 0u, kBadSeqlens);
        }
        const unsigned incl = sum_to_lane(sum);
        sh.prefix[tid] = incl - sum;  // within the warp
        if (lane == 31)
            sums[tid >> 5] = incl;
        ptx::fence_proxy_async_smem();  // (these stores come before the copies that land on `sh`)
        __syncthreads();
        // the warps' sums, a lane each
        const unsigned of_warp = lane < THREADS / 32 ? sums[lane] : 0u;
        const unsigned all = sum_to_lane(of_warp);
        cut = Cut(__shfl_sync(FULL, all, 31), p.sms);
        upto = all - of_warp;
    }

    // The walk over run `run`, problem by problem, by a whole warp.
    int left;         // positions left in the run
    int e, base;      // entry; the lanes have entries base .. base + 31
    unsigned skip;    // positions of entry e before the run
    Span mine, at;    // the lane's entry; entry e
    int in, b, block, heads, hb, kv;  // position in the problem; its block, KV head and block of heads, and both as one

    __device__ __forceinline__ void start(const Cache16Params &p, const Shared &sh)
    {
        const int lane = threadIdx.x & 31;
        const unsigned run = blockIdx.x, over = run * cut.r / cut.n;  // (start(run); start(run + 1) needs no division of its own)
        const unsigned x = run * cut.q + over;
        left = static_cast<int>(cut.q + (run * cut.r - over * cut.n + cut.r >= cut.n ? 1u : 0u));
        // the last warp, and the last thread of it, whose entries start at or before x
        const int w0 = 31 - __clz(__ballot_sync(FULL, lane < THREADS / 32 && upto <= x));
        const unsigned before = __shfl_sync(FULL, upto, w0);
        const unsigned hit = __ballot_sync(FULL, before + sh.prefix[w0 * 32 + lane] <= x);
        const int owner = w0 * 32 + 31 - __clz(hit);
        skip = x - before - sh.prefix[owner];
        base = owner * per;
        const int of_lane = min(base + lane, entries - 1);
        mine = per == 1 ? sh.first[of_lane] : span_of(p, of_lane);
        e = base - 1;
        kv = p.Hkv;  // done with entry e
        ptx::fence_proxy_async_smem();  // and so do these reads: lane 0 publishes the first unit behind them
        __syncwarp();
    }

    // The next unit.
    __device__ __forceinline__ Unit next(const Cache16Params &p)
    {
        const int lane = threadIdx.x & 31;
        Unit un;
        un.n = un.join = -1;
#pragma unroll 1
        while (left > 0) {
#pragma unroll 1
            while (kv == p.Hkv) {  // on to the next entry (the positions left exist: one follows)
                if (++e >= base + 32) {
                    base = e;
                    mine = span_of(p, min(e + lane, entries - 1));
                }
                const int from = e - base;
                at.tiles = __shfl_sync(FULL, mine.tiles, from);
                at.blocks = __shfl_sync(FULL, mine.blocks, from);
                at.lo = __shfl_sync(FULL, mine.lo, from);
                at.hi = __shfl_sync(FULL, mine.hi, from);
                at.k0 = __shfl_sync(FULL, mine.k0, from);
                at.seq = __shfl_sync(FULL, mine.seq, from);
                at.toks = __shfl_sync(FULL, mine.toks, from);
                if (at.tiles == 0)
                    continue;
                const int len = at.tiles + OVERHEAD;
                kv = heads = b = hb = in = 0;
                block = e < p.ngroups ? p.toks_p : p.toks_o;
                if (skip > 0) {  // the run's first problem
                    const unsigned all = static_cast<unsigned>(len) * static_cast<unsigned>(at.blocks * p.Hkv * p.head_blocks);
                    if (skip >= all) {
                        skip -= all;
                        kv = p.Hkv;
                        continue;
                    }
                    kv = heads = static_cast<int>(skip) / len;
                    in = static_cast<int>(skip) - heads * len;
                    skip = 0;
                    if (at.blocks > 1) {
                        const int first = heads;
                        kv = heads = first / at.blocks;
                        b = first - heads * at.blocks;
                    }
                    if (p.head_blocks > 1) {
                        kv = heads / p.head_blocks;
                        hb = heads - kv * p.head_blocks;
                    }
                }
            }
            // the problem's positions [in, in + take)
            const int take = min(left, at.tiles + OVERHEAD - in);
            const int t0 = max(0, in - OVERHEAD), t1 = in + take - OVERHEAD;
            left -= take;
            in = 0;
            const bool prefix = e < p.ngroups;
            un.table = prefix ? ~e : e - p.ngroups;
            un.n = t1 - t0;
            un.tile0 = at.k0 + t0 * TILE;
            un.lo = at.lo;
            un.kv = kv;
            un.head = kv * p.G + hb * p.heads;
            un.live = min(p.heads, p.G - hb * p.heads);
            un.q_tok = at.seq * p.n + b * block;
            un.toks = min(block, at.toks - b * block);
            un.hi = at.hi;
            un.pos0 = at.hi - 1;
            if (!prefix) {  // no row of the block sees a key behind its last token's own
                un.pos0 = at.hi - p.n + b * block;
                un.hi = min(un.hi, un.pos0 + un.toks);
            }
            const bool whole = t0 == 0 && t1 == at.tiles, joined = prefix || at.lo > 0;
            un.dest = !whole ? 2 * static_cast<int>(blockIdx.x) + (t0 == 0 ? 1 : 0) : joined ? DEST_ROWS : DEST_DIRECT;
            un.join = -1;
            un.after = at.tiles - t1;
            if (t0 == 0 && un.n > 0)  // the problem's place among those of its group (from its first sequence on) or sequence
                un.join = (at.seq * (prefix ? p.blocks_p : p.blocks_o) + b) * (p.Hkv * p.head_blocks) + heads;
            // on to the next problem
            if (++b == at.blocks) {
                b = 0;
                ++heads;
                if (++hb == p.head_blocks) {
                    hb = 0;
                    ++kv;
                }
            }
            if (un.n > 0)
                break;
            un.n = -1;  // the run ends inside the problem's start
        }
        return un;
    }

    // A problem's parts, of which the first ends with this run, `after` tiles before the problem's end.
    __device__ __forceinline__ int parts_of(int after) const
    {
        const int run = static_cast<int>(blockIdx.x);
        return after == 0 ? 1 : cut.run_of(cut.start(run + 1) + after - 1) - run + 1;
    }
};

// Floats of a part: O [rows][D] (over its own l, so that no part is larger than the values it joins), then m and l of
// each row, in all a multiple of 8 (O is stored 32 bytes at a time).
template <int D>
__host__ __device__ constexpr long long part_floats(int rows)
{
    return static_cast<long long>(rows) * (D + 8);
}

// Keys [0, n) of 32 as a bit mask.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Which halves of a pair are infinities or NaN, as a mask over their bits.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    return ((w & E) == E ? 0xffffu : 0u) | ((w & (E << 16)) == (E << 16) ? 0xffff0000u : 0u);
}

// Channels [c0, D) in steps of `step` of the values of keys pos0 + 1 + b of sequence s (bit b of `odd`, all of which the row
// sees) that are not finite, and so were left out of the product, onto a row that has been written (`direct`: in 16 bits):
// whatever their weights, which are positive, these decide.
template <int D, bool BF16>
static __device__ __noinline__ void add_odd(const Cache16Params &p, int s, int kv, int pos0, uint32_t odd, void *row,
                                            bool direct, int c0, int step)
{
#pragma unroll 1
    for (; odd != 0u; odd &= odd - 1u) {
        const int key = pos0 + __ffs(odd), page = key / p.page_size;
        const int id = p.table[s * p.table_stride + page];
        if (id < 0 || id >= p.num_pages)
            return;
        const uint16_t *v = p.v + ((static_cast<long long>(id) * p.Hkv + kv) * p.page_size + (key - page * p.page_size)) * D;
#pragma unroll 1
        for (int i = c0; i < D; i += step) {
            const uint32_t w = v[i];
            if (not_finite<BF16>(w) == 0u)
                continue;
            const float x = unpack16<BF16>(w).x;
            if (direct) {
                uint16_t *o = static_cast<uint16_t *>(row) + i;
                *o = static_cast<uint16_t>(pack16<BF16>(unpack16<BF16>(*o).x + x, 0.f));
            } else {
                static_cast<float *>(row)[i] += x;
            }
        }
    }
}

// The page of a token among its sequence's. (A division by an unknown number takes some 30 instructions; the product with the
// inverse, rounded down, is the quotient or one less.)
__device__ __forceinline__ int page_at(const Cache16Params &p, int tok)
{
    const int q = static_cast<int>(__umulhi(static_cast<unsigned>(tok >> 4), p.page_inverse));
    return q + ((q + 1) * p.page_size <= tok ? 1 : 0);
}

// The pages of a unit's boxes, 32 boxes at a time: lane i has that of box 32 batch + i, and the place in it. Boxes without a
// key that a row may see have none. The page is loaded when this is called, and looked at by `planes_of` when its boxes are next.
struct Pages {
    int id, off;
};

__device__ __forceinline__ Pages pages_of(const Cache16Params &p, const Unit &un, int batch)
{
    const int tok = un.tile0 + (batch * 32 + static_cast<int>(threadIdx.x & 31)) * p.box;
    Pages r{-1, -1};
    if (un.n > 0 && tok < min(un.hi, un.tile0 + un.n * TILE)) {
        const int at = page_at(p, tok);
        r.off = tok - at * p.page_size;
        r.id = __ldg((un.prefix() ? p.prefix_table + ~un.table * p.prefix_stride : p.table + un.table * p.table_stride) + at);
    }
    return r;
}

// Their planes in the pool; that of page 0, and a status code, for one outside it.
__device__ __forceinline__ int planes_of(const Cache16Params &p, const Unit &un, const Pages &at)
{
    int id = at.id;
    if (id < 0 || id >= p.num_pages) {
        if (at.off >= 0)
            atomicCAS(p.status, 0u, kBadPages);
        id = 0;
    }
    return id * p.Hkv + un.kv;
}

// A warp's copies of a unit's K (or V) through a ring of slots, each C channels of a tile's 128 keys as C / 64 boxes of 16 KB.
// The warp's lanes have the pages of `planes`.
struct Ring {
    uint32_t base, full0, empty0;  // the first slot and its barriers
    int slots, slot;
    uint32_t ph, armed, armed_par;
};

// A tile of a unit: its boxes with keys (the first one in lane first % 32), and the lanes' planes and places.
struct Tile {
    int first, n;
    int plane, off;
};

__device__ __forceinline__ Tile tile_of(const Cache16Params &p, const Unit &un, int j, int plane, int off)
{
    const int keys = min(un.hi - un.tile0 - j * TILE, TILE);
    return Tile{j * (TILE >> p.box_log2), keys > 0 ? (keys + p.box - 1) >> p.box_log2 : 0, plane, off};
}

// A tile's copies. A slot of K has 64 channels of all keys, one of V all channels of VK keys; a box has 64 channels, and a lane
// has a box. (One place for both: what a unit's copies run through is fetched from behind the instruction cache each time
// where units are short. A loop over the boxes took 130 cycles a box, lanes of their own take 55.) False when a wait ran out.
template <int D, int VK>
__device__ __forceinline__ bool copy_tile(const Cache16Params &p, const CUtensorMap *map, bool of_k, Ring &r, Waits *waits, const Tile &t)
{
    const int lane = threadIdx.x & 31;
    const int rows = t.n << p.box_log2, keys = of_k ? TILE : VK, box_log2 = min(p.box_log2, of_k ? 7 : 6);
    const int slot_bytes = of_k ? TILE * 128 : VK * D * 2, across = of_k ? 0 : D == 128 ? 1 : 2;  // 2^across boxes side by side
    static_assert(TILE == 128 && VK == 64, "the largest box");
    const int key = (lane >> across) << box_log2, box = lane & ((1 << across) - 1);  // this lane's box
#pragma unroll 1
    for (int s = 0; s < (of_k ? D / 64 : TILE / VK); ++s) {
        if (!wait_warp(r.empty0 + 8u * r.slot, r.ph ^ 1u, waits, 2 /* a slot that does not empty */, 1))
            return false;
        const uint32_t full = r.full0 + 8u * r.slot;
        const int k0 = of_k ? 0 : s * VK, n = max(0, min(rows - k0, keys));  // (rows is a multiple of the boxes)
        ptx::mbar_arrive_expect_tx_w(full, n << (7 + across));
        const int from = t.first + ((k0 + key) >> p.box_log2);
        const int z = __shfl_sync(FULL, t.plane, from & 31), y = __shfl_sync(FULL, t.off, from & 31) + ((k0 + key) & (p.box - 1));
        __syncwarp();
        if (key < n)
            ptx::tma_load_3d(r.base + r.slot * slot_bytes + key * 128 + box * (keys * 128), map, full, (of_k ? s : box) * 64, y, z);
        __syncwarp();
        r.armed |= 1u << r.slot;
        r.armed_par = (r.armed_par & ~(1u << r.slot)) | (r.ph << r.slot);
        if (++r.slot == r.slots) {
            r.slot = 0;
            r.ph ^= 1u;
        }
    }
    return true;
}

// Every copy that this warp issued lands before the CTA may exit.
__device__ __forceinline__ void land(const Ring &r, Waits *waits)
{
#pragma unroll 1
    for (int s = 0; s < r.slots; ++s)
        if (r.armed & (1u << s))
            wait_own(r.full0 + 8u * s, (r.armed_par >> s) & 1u, waits);
}

// A slot of V, rows of some keys in BOXES boxes of 64 channels, before the product, by a whole warp: rows [z0, r0) and [r1, z1)
// are zeroed, and of rows [a0, a1) the values that are not finite. Returns which of these rows had such: bit row + bit0.
template <bool BF16, int BOXES>
static __device__ __noinline__ uint32_t clean_rows(uint32_t slot, int box_bytes, int z0, int r0, int r1, int z1, int a0, int a1,
                                                   int bit0)
{
    constexpr int LANES = 8 * BOXES, ROWS = 32 / LANES;  // lanes a row, of 16 bytes each; rows at a time
    const int lane = threadIdx.x & 31, sub = lane / LANES;
    const uint32_t unit = slot + ((lane >> 3) % BOXES) * box_bytes + (lane & 7) * 16;
    auto store = [](uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    };
#pragma unroll 1
    for (int r = z0 + sub; r < r0; r += ROWS)
        store(unit + r * 128, 0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int r = r1 + sub; r < z1; r += ROWS)
        store(unit + r * 128, 0u, 0u, 0u, 0u);
    uint32_t odd = 0;
#pragma unroll 1
    for (int r = a0 + sub; r < a1; r += ROWS) {
        uint32_t w[4], x[4];
        const uint32_t at = unit + r * 128;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = not_finite<BF16>(w[i]);
        if ((x[0] | x[1] | x[2] | x[3]) != 0u) {
            store(at, w[0] & ~x[0], w[1] & ~x[1], w[2] & ~x[2], w[3] & ~x[3]);
            odd |= 1u << (r + bit0);  // 0 .. 30
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    return __reduce_or_sync(FULL, odd);
}

}  // namespace c16
}  // namespace sdp
