// Attention of each sequence's last n tokens over the paged 16-bit cache, for batches whose sequences share prefixes
// (sdp_fwd_cache16):
//
//     row i of sequence s is at position p = len_s - n + i and sees the keys j <= p;
//     O = softmax(scale * Q K^T) V over them, LSE = ln sum exp; a row that sees none: 0 and -inf.
//
// The sequences of a group have their first P tokens in common. Softmax over a union of key sets is the sum of
// the sets' own results, each (m, l, O) weighed by 2^(m - max m) l, so there are two kinds of problems:
//
//   - (group, KV head, block): the prefix's keys, for the rows of ALL sequences of the group, 128 a block, each of which reads them once.
//     Every row sees all of them: a matrix product of as many rows as the batch has, where one sequence alone has
//     the few rows of its group of heads;
//   - (sequence, KV head, block): the keys behind the prefix (all of them for a sequence that shares none).
//
// Both run through one pipeline: the G query heads of a KV head and the tokens are the 128 lanes of S = Q K^T and O += P V
// on tcgen05, with both accumulators in tensor memory; 128-key tiles come by TMA through rings of shared memory, in
// boxes that lie in one page each; a thread has a row of the softmax; a warpgroup of its own writes a unit's rows while the
// next unit runs. Scores, weights and sums are fp32; the weights are rounded to the 16-bit type for the product with V
// (half a step of theirs each, beside inputs that are rounded alike). A decoding problem has few live rows, and its
// products are padded to 128 lanes: a tile takes 1024 cycles of the tensor core at D = 128, and 2800 of an SM's share
// of HBM; warps without a live row skip the softmax.
//
// What a tile costs. The four warps of a softmax need 2000 to 2300 cycles for a tile's two passes, of which 1024 are
// the exponentials' (16 a cycle and SM), so two groups of four warps take the tiles in turn, and what one needs of
// the other, the rows' maxima, goes from tile to tile through shared memory between the two passes. P is handed over in
// halves, so that its product with V begins while the second one is computed. What remains is the chain S -> softmax -> PV ->
// S of the tile that takes the same buffer (2 at D = 256, which leaves no tensor memory for a third, 3 at D = 128): 1700
// cycles a tile at D = 128, 3050 at D = 256, where shared memory's 128 bytes a cycle alone would need 2560 (S reads Q and
// K, PV reads V, the copies write both). HBM's share is 2800 and 5600 cycles a tile that nobody else reads.
//
// Work split: the problems' tiles are numbered through, groups first, and cut into equal runs, one a CTA, a problem's start
// and end counting as OVERHEAD tiles more; the lengths are on the device, so each CTA finds its run from them. A problem
// that one run holds whole, and whose rows share no prefix, is written as it ends; what else there is, is joined
// by cache16_join.cuh's kernel, which starts as CTAs end. Results do not depend on the order in which CTAs run.
//
// Blocks of 256 rows by CTA pairs, each CTA with its own 128 rows and half of every tile of K and V, would halve the copies and what
// S and PV read of them: not built. (One CTA has no room for two blocks: one's O and S buffers fill tensor memory at D = 256.)
//
// What a problem's start and end cost. Each runs through some 30 KB of code once (look-up, copies, masks, cleaning, rows' ends), and
// with sixteen warps at seven kinds of work that is more than the instruction cache nearest them keeps: straight code then
// takes some 10 cycles an instruction, and what counts is how much of it there is, and on whose way. So units are looked up
// ahead by a warp that has time (on the copier's own way a problem of one tile took 8000 cycles, so 5000), both copiers
// run through one place, each box of a slot is a lane's, and the rows' ends are two loops of a few lines.
//
// 64 sequences behind 8192 shared tokens, 10 to 2000 of their own, 32 heads over 8, D = 128: 45 us, where HBM alone takes 24;
// 256 behind 16384, 32 heads over 2, D = 256: 130 us, where the tensor cores alone take 72; eight of 16384 tokens that share
// nothing, D = 256: 51 us (5.2 TB/s), where HBM takes 40; 32 behind 4001, 32 heads of their own, D = 128: 39 us, HBM 14. A launch
// needs some 9000 cycles (5 us) before its first copy and the join 4 to 8 us after the last tile.
//
// Keys outside [lo, hi) of a problem share its first and last tiles. Their scores are replaced before any arithmetic, whatever
// they hold (NaN too); their rows of V are zeroed in shared memory or left out of the product. A drafted token's V is seen by
// some rows of its problem only: where it holds values that are not finite these are taken out of the product too, and added
// to the rows that see them when they are written.
#pragma once

#include "cache16_join.cuh"
#include "sdp_fwd_kernel.cuh"

namespace sdp {

namespace c16 {

constexpr int THREADS = 512;

template <int D>
struct Plan {
    using L = Layout<D>;
    static constexpr int QB = D == 128 ? 2 : 1;  // query tiles in shared memory
    static constexpr int UNITS = 4;              // units looked up ahead
    // K and V have rings of their own, so that whoever waits for a slot has seen what it held before: its barrier is one phase
    // away at most. A slot of K has 128 keys by KC channels, one of V VK keys by all channels. At D = 256, where 160 KB are 1.25
    // tiles, 8 x 16k takes 51.4 us with 6 and 2 slots and 52.4 with 4 and 3 (256 x 16k 130.5 with both); with V in 5 slots of 32 keys
    // 256 x 16k took 144 us where it took 137, with K in 2 of 128 channels 141.
    static constexpr int KC = 64, VC = D, VK = 64;
    static constexpr int NK = D == 128 ? 4 : 6, NV = D == 128 ? 5 : 2, NS = NK + NV;
    static constexpr int K_SLOT = KC * 256, V_SLOT = VC * VK * 2;
    static constexpr int BAR_AREA = 512;
    // q_full[QB], q_free[QB], slot_full[NS], slot_empty[NS], s_full[NB], p_full[NB][2], o_done[ring], final[2], o_free,
    // sum_full, sum_free, odd_full, unit_full[UNITS], unit_free[UNITS], max_full[2][4]
    static constexpr int NBARS = 2 * QB + 2 * NS + 3 * L::NSBUF + O_DONE_RING + 2 + 4 + 2 * UNITS + 8;
    static constexpr int RING_OFF = QB * L::Q_BYTES, V_OFF = RING_OFF + NK * K_SLOT;
    static constexpr int BAR_OFF = V_OFF + NV * V_SLOT;
    static constexpr int HOLDER_OFF = BAR_OFF + 8 * NBARS;  // TMEM address, -, mask of keys that are not finite, whether O holds anything, Waits
    static constexpr int SUM_OFF = BAR_OFF + BAR_AREA;      // the rows' maxima so far; of a unit, their m and l from the two groups of softmax warps
    static constexpr int UNIT_OFF = SUM_OFF + 4 * TILE * 4;
    static constexpr int TOTALS_OFF = UNIT_OFF + UNITS * static_cast<int>(sizeof(Unit));  // of the entries of each warp (Runs::begin)
    static constexpr int SMEM_BYTES = TOTALS_OFF + THREADS / 32 * 4;
    static_assert(HOLDER_OFF % 8 == 0 && HOLDER_OFF + 24 + sizeof(Waits) <= BAR_OFF + BAR_AREA, "barrier area");
    static_assert(SMEM_BYTES <= L::SMEM_LIMIT, "shared memory");
    static_assert(sizeof(Unit) % 16 == 0 && UNIT_OFF % 16 == 0, "unit ring");
    static_assert(sizeof(Runs<THREADS>::Shared) <= BAR_OFF - RING_OFF, "the sums of the problems' lengths");
    static_assert(TOTALS_OFF >= V_OFF + NV * V_SLOT, "copies land below");
};

// Eight words to a 32-byte boundary, a whole sector of a row, if `live`.
__device__ __forceinline__ void st_global_v8(void *at, const uint32_t *w, uint32_t live)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t@p st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t}" ::"l"(at),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(live)
                 : "memory");
}

// Four, to 16 bytes.
__device__ __forceinline__ void st_global_v4(void *at, const uint32_t *w, uint32_t live)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(at), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(live)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}

template <int N>
__device__ __forceinline__ uint64_t f2_of(const uint32_t (&s)[N], int i)
{
    return ptx::f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
}

}  // namespace c16

template <int D, bool BF16>
__global__ void __launch_bounds__(c16::THREADS, 1)
    cache16_attn_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qo,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ Cache16Params p)
{
    using namespace c16;
    using L = Layout<D>;
    using PL = Plan<D>;
    constexpr int NS = PL::NS;
    constexpr int NB = L::NSBUF;
    constexpr int QB = PL::QB;
    constexpr uint32_t IDESC_S = ptx::idesc_f16_f32acc(128, TILE, BF16, false);
    constexpr uint32_t IDESC_PV = ptx::idesc_f16_f32acc(128, PL::VC, BF16, true);

    extern __shared__ __align__(1024) uint8_t smem[];  // (there is no room to align it by hand)
    const uint32_t sbase = ptx::smem_addr(smem);
    if ((sbase & 1023u) != 0u) {
        atomicCAS(p.status, 0u, SITE_SLOT_FULL);
        return;
    }
    const uint32_t s_q0 = sbase;  // query tile b at s_q0 + b * Q_BYTES
    const uint32_t s_k = sbase + PL::RING_OFF, s_v = sbase + PL::V_OFF;
    const uint32_t q_full0 = sbase + PL::BAR_OFF;  // + 8 b
    const uint32_t q_free0 = q_full0 + 8u * QB;    // + 8 b: the S MMAs that read query tile b last are done
    const uint32_t slot_full0 = q_free0 + 8u * QB;
    const uint32_t slot_empty0 = slot_full0 + 8u * NS;
    const uint32_t s_full0 = slot_empty0 + 8u * NS;
    const uint32_t p_full0 = s_full0 + 8u * NB;  // + 16 (tile % NB) + 8 (its half)
    const uint32_t o_done0 = p_full0 + 16u * NB;
    const uint32_t final0 = o_done0 + 8u * O_DONE_RING;
    const uint32_t o_free = final0 + 16u;     // the unit's O has been read
    const uint32_t sum_full = o_free + 8u;    // its rows' m and l are there
    const uint32_t sum_free = sum_full + 8u;
    const uint32_t odd_full = sum_free + 8u;  // the mask of its keys that are not finite is there
    const uint32_t unit_full0 = odd_full + 8u, unit_free0 = unit_full0 + 8u * PL::UNITS;  // + 8 (i % UNITS)
    const uint32_t max_full0 = unit_free0 + 8u * PL::UNITS;  // + 32 (tile % 2) + 8 (warp of a group)
    float *const row_max = reinterpret_cast<float *>(smem + PL::SUM_OFF), *const row_m = row_max + TILE, *const row_l = row_m + TILE;
    Unit *const ring = reinterpret_cast<Unit *>(smem + PL::UNIT_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + PL::HOLDER_OFF);
    Waits *const waits = reinterpret_cast<Waits *>(tmem_holder + 6);
    volatile uint32_t *odd_keys = tmem_holder + 2;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int run = static_cast<int>(blockIdx.x);

    if (warp == 15) {  // (the first warps have entries to look up)
        // one arrival each, but for p_full, o_free and sum_free, where four warps arrive, sum_full (eight) and unit_free (all)
        constexpr int P0 = 2 * QB + 2 * NS + NB, P1 = P0 + 2 * NB, SUM = P1 + O_DONE_RING + 2;
        for (int i = lane; i < PL::NBARS; i += 32) {
            const bool four = (i >= P0 && i < P1) || i == SUM || i == SUM + 2;
            const bool readers = i >= SUM + 4 + PL::UNITS && i < SUM + 4 + 2 * PL::UNITS;  // unit_free: all warps
            ptx::mbar_init(q_full0 + 8u * i, four ? 4 : i == SUM + 1 ? 8 : readers ? 16 : 1);
        }
        if (lane == 0) {
            waits->abort = 0;
            waits->status = p.status;
            waits->timeout_ns = p.timeout_ns;
        }
        __syncwarp();
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
    // Up to here the CTA has run beside the end of what is before it on the stream (the append, or another call's join, which let
    // it start). What follows may be launched from here on, as its own first reads are of what was there for this kernel; it
    // finds no room beside a CTA, so it starts where there is none or it has ended, and waits there for the last one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    using R = Runs<THREADS>;
    R::Shared &sums = *reinterpret_cast<R::Shared *>(smem + PL::RING_OFF);
    R runs;
    ptx::tc_fence_before();
    runs.begin(p, sums, reinterpret_cast<unsigned *>(smem + PL::TOTALS_OFF));
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    if (blockIdx.x >= runs.cut.n) {  // nothing left for this one
        if (warp == 5)
            ptx::tmem_dealloc(tmem, L::TMEM_COLS);
        return;
    }

    auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t site, int tiles = 1) {
        return wait_warp(bar, parity, waits, site, tiles);
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

    if (warp == 4 || warp == 7) {
        // ------------------------------------------ the copies of Q and K (warp 4), and of V
        const bool of_k = warp == 4;
        Ring r{of_k ? s_k : s_v, slot_full0 + (of_k ? 0u : 8u * PL::NK), slot_empty0 + (of_k ? 0u : 8u * PL::NK), of_k ? PL::NK : PL::NV, 0, 0, 0, 0};
        uint32_t q_armed = 0, q_par = 0;
        int longest = 1;  // of the units so far: its end may be what is waited for
        const int tiles = p.box / 4;  // of a batch of 32 boxes
        Unit un, next_un;
        un.n = 0;
        Pages now{}, next{};
        // (the unit before the first has no tiles: one place for what the loop does ahead)
#pragma unroll 1
        for (int k = -1;; ++k) {
            const int b = k % QB;
            if (of_k && k >= 0) {
                if (k >= QB && !wait_all(q_free0 + 8u * b, ((k - QB) / QB) & 1, SITE_Q_FULL, longest))
                    break;
                longest = max(longest, un.n);
                if (!p.no_copies) {
                    ptx::mbar_arrive_expect_tx_w(q_full0 + 8u * b, (un.prefix() ? p.toks_p : p.toks_o) * p.heads * D * 2);
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c)
                        ptx::tma_load_3d_w(s_q0 + b * L::Q_BYTES + c * L::BOX_BYTES, un.prefix() ? &tm_qp : &tm_qo, q_full0 + 8u * b, c * 64,
                                           un.head, un.q_tok);
                    q_armed |= 1u << b;
                    q_par = (q_par & ~(1u << b)) | (((k / QB) & 1u) << b);
                }
            }
            int j = 0;
            bool ok = true, more = true;
#pragma unroll 1
            do {
                const int plane = planes_of(p, un, now), off = now.off, end = min(un.n, j + tiles);
                // the next batch's pages, of this unit or of the one behind it, are looked up while this one is copied
                const bool same = end < un.n;
                if (!same && !(more = take(k + 1, next_un)))
                    next_un.n = -1;  // (also where a wait ran out and there is none: no page of it is looked up)
                next = pages_of(p, same ? un : next_un, same ? end / tiles : 0);
#pragma unroll 1
                for (; ok && j < end; ++j)
                    ok = p.no_copies || copy_tile<D, PL::VK>(p, of_k ? &tm_k : &tm_v, of_k, r, waits, tile_of(p, un, j, plane, off));
                now = next;
            } while (ok && j < un.n);
            if (!ok || !more)
                break;
            un = next_un;
        }
#pragma unroll 1
        for (int b = 0; b < QB; ++b)
            if (q_armed & (1u << b))
                wait_own(q_full0 + 8u * b, (q_par >> b) & 1u, waits);
        land(r, waits);
    } else if (warp == 5) {
        // ------------------------------------------- S = Q K^T issuer
        const uint64_t dk = ptx::smem_desc_sw128(s_k, 16, 1024);
        bool issued = false, ok = true;
        int g0 = 0, slot = 0;  // tiles of the earlier units, and the next slot
        uint32_t ph = 0;
        Unit un;
        for (int k = 0; ok && take(k, un); ++k) {
            const int n = un.n, b = k % QB;
            const uint64_t dq = ptx::smem_desc_sw128(s_q0 + b * L::Q_BYTES, 16, 1024);
            if (!(ok = wait_all(q_full0 + 8u * b, (k / QB) & 1, SITE_Q_FULL)))
                break;
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const int gt = g0 + t;
                if (gt >= NB) {  // buffer gt % NB held P of tile gt - NB: its PV must have read it
                    const int pv = gt - NB;
                    if (!(ok = wait_all(o_done0 + 8u * (pv % O_DONE_RING), (pv / O_DONE_RING) & 1, SITE_O_DONE)))
                        break;
                }
                const uint32_t d_tmem = tmem + L::TM_S + (gt % NB) * TILE;
#pragma unroll 1
                for (int ch = 0; ch < D / PL::KC; ++ch) {
                    if (!(ok = wait_all(slot_full0 + 8u * slot, ph, SITE_SLOT_FULL)))
                        break;
                    ptx::tc_fence_after();
                    const uint64_t kslot = dk + static_cast<uint64_t>((slot * PL::K_SLOT) >> 4);
                    const uint64_t qch = dq + static_cast<uint64_t>((ch * (PL::KC / 64) * L::BOX_BYTES) >> 4);
#pragma unroll
                    for (int kk = 0; kk < PL::KC / 16; ++kk) {
                        const uint32_t at = ((kk >> 2) * L::BOX_BYTES + (kk & 3) * 32) >> 4;
                        ptx::mma_ss_w(d_tmem, qch + at, kslot + at, IDESC_S, (ch | kk) != 0);
                    }
                    issued = true;
                    ptx::mma_commit_w(slot_empty0 + 8u * slot);
                    if (++slot == PL::NK) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok)
                    break;
                ptx::mma_commit_w(s_full0 + 8u * (gt % NB));
            }
            if (!ok)
                break;
            ptx::mma_commit_w(q_free0 + 8u * b);  // query tile b may take unit k + QB's Q
            g0 += n;
        }
        if (issued) {  // all of this warp's MMAs complete before TMEM is freed
            ptx::mma_commit_w(final0);
            wait_own(final0, 0, waits);
        }
    } else if (warp == 6) {
        // ------------------------------------------ O += P V issuer
        const uint64_t dv = ptx::smem_desc_sw128(s_v, PL::VK * 128, 1024);
        bool issued = false, ok = true;
        int g0 = 0, slot = 0;
        uint32_t ph = 0;
        Unit un;
        for (int k = 0; ok && take(k, un); ++k) {
            const int n = un.n;
            uint32_t odd = 0;     // keys that only some rows see and whose V is not finite
            uint32_t onto = 0;    // O holds something of this unit
            const int own = un.pos0 + 1;  // the first such key
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int gj = g0 + j;
                const int buf = gj % NB;
                // Rows of the tile that hold keys. The product takes the steps of 16 rows that have any; what else these
                // hold, before the first key or behind the last, is zeroed.
                const int key0 = un.tile0 + j * TILE;
                const int r0 = max(0, un.lo - key0), r1 = min(TILE, un.hi - key0);
                const int kk0 = r0 / 16, kk1 = r1 > r0 ? (r1 + 15) / 16 : 0;
                const bool ragged = r1 > r0 && ((r0 | r1) & 15) != 0;
                const int a0 = max(r0, own - key0), a1 = un.prefix() || p.n == 1 ? 0 : r1;  // keys that some rows do not see
                const uint32_t a_tmem = tmem + L::TM_S + buf * TILE;
                // (before P is there: V lands while the softmax is at work)
                if (ragged || a1 > a0) {
                    int at = slot;
                    uint32_t at_ph = ph;
#pragma unroll 1
                    for (int v0 = 0; ok && v0 < TILE; v0 += PL::VK) {
                        auto in = [&](int x) { return max(0, min(x - v0, PL::VK)); };
                        const int z0 = in(kk0 * 16), y0 = in(r0), y1 = in(r1), z1 = in(kk1 * 16), b0 = in(a0), b1 = in(a1);
                        if ((z0 < y0 || y1 < z1 || b0 < b1) && (ok = wait_all(slot_full0 + 8u * (PL::NK + at), at_ph, SITE_SLOT_FULL)))
                            odd |= clean_rows<BF16, D / 64>(s_v + at * PL::V_SLOT, PL::VK * 128, z0, y0, y1, z1, b0, b1, key0 + v0 - own);
                        if (++at == PL::NV) {
                            at = 0;
                            at_ph ^= 1u;
                        }
                    }
                    if (!ok)
                        break;
                }
                if (!(ok = wait_all(p_full0 + 16u * buf, (gj / NB) & 1, SITE_P_FULL)))
                    break;
                // a unit's first PV overwrites O: the previous unit's rows must have been read
                if (j == 0 && k > 0 && !(ok = wait_all(o_free, (k - 1) & 1, SITE_O_DONE)))
                    break;
#pragma unroll 1
                for (int v0 = 0; v0 < TILE; v0 += PL::VK) {
                    if (v0 == TILE / 2 && !(ok = wait_all(p_full0 + 16u * buf + 8u, (gj / NB) & 1, SITE_P_FULL)))
                        break;
                    if (!(ok = wait_all(slot_full0 + 8u * (PL::NK + slot), ph, SITE_SLOT_FULL)))
                        break;
                    ptx::tc_fence_after();
                    const uint64_t vslot = dv + static_cast<uint64_t>((slot * PL::V_SLOT) >> 4);
                    const int q0 = max(kk0, v0 / 16), q1 = min(kk1, (v0 + PL::VK) / 16);
                    if (q1 - q0 == PL::VK / 16) {
#pragma unroll
                        for (int kk = 0; kk < PL::VK / 16; ++kk)
                            ptx::mma_ts_w(tmem + L::TM_O, a_tmem + v0 / 2 + kk * 8, vslot + ((kk * 2048) >> 4), IDESC_PV,
                                          kk == 0 ? onto | (q0 > kk0 ? 1u : 0u) : 1u);
                    } else {
#pragma unroll 1
                        for (int kk = q0; kk < q1; ++kk)
                            ptx::mma_ts_w(tmem + L::TM_O, a_tmem + kk * 8, vslot + (((kk * 16 - v0) * 128) >> 4), IDESC_PV,
                                          onto | (kk > kk0 ? 1u : 0u));
                    }
                    issued = true;
                    ptx::mma_commit_w(slot_empty0 + 8u * (PL::NK + slot));
                    if (++slot == PL::NV) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok)
                    break;
                onto |= kk1 > kk0 ? 1u : 0u;
                ptx::mma_commit_w(o_done0 + 8u * (gj % O_DONE_RING));
            }
            if (!ok)
                break;
            if (lane == 0) {  // the last unit's have been read: its O is free
                *odd_keys = odd;
                odd_keys[1] = onto;
            }
            arrive(odd_full);
            g0 += n;
        }
        if (issued) {
            ptx::mma_commit_w(final0 + 8u);
            wait_own(final0 + 8u, 0, waits);
        }
    } else if (warp < 4 || warp >= 12) {
        // --------------------------------------- softmax / correction: warps 0 to 3 have the even tiles, 12 to 15 the odd ones
        const int group = warp < 4 ? 0 : 1, w4 = warp & 3;
        const int row = w4 * 32 + lane;  // row within the tile = TMEM lane
        const int row_tok = row / p.heads, row_head = row - row_tok * p.heads;
        const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
        const uint32_t t_s = tmem + lane_off + L::TM_S;
        const uint32_t t_o = tmem + lane_off + L::TM_O;
        const float c = p.c;  // not 0
        const uint64_t c2 = ptx::f2_pack(c, c);
        const uint32_t unseen = c > 0.f ? 0xff800000u : 0x7f800000u;  // -inf or inf
        const uint32_t max_mine = max_full0 + 32u * group + 8u * w4, max_other = max_full0 + 32u * (group ^ 1) + 8u * w4;
        bool ok = true;
        int g0 = 0;
        Unit un;
        for (int k = 0; ok && take(k, un); ++k) {
            const int n = un.n;
            const bool idle = w4 * 32 >= un.toks * p.heads;  // no live row in the warp
            const bool dead = row_tok >= un.toks || row_head >= un.live;
            // the row sees keys [lo, pos]
            const int pos = min(un.hi - 1, un.prefix() ? un.pos0 : un.pos0 + row_tok);
            // The rows' maxima go from tile to tile, from one group to the other: it is tile gj's turn.
            auto turn = [&](int gj) { return gj == 0 || wait_all(max_other, ((gj - 1) >> 1) & 1, SITE_S_FULL); };
            float m_used = -INFINITY, l = 0.f;  // l: of this group's tiles, in units of 2^m_used
            for (int j = (g0 + group) & 1; j < n; j += 2) {
                const int gj = g0 + j;
                const int buf = gj % NB;
                if (!(ok = wait_all(s_full0 + 8u * buf, (gj / NB) & 1, SITE_S_FULL)))
                    break;
                if (idle) {  // whatever its lanes of P hold meets no other row
                    if (!(ok = turn(gj)))
                        break;
                    arrive(max_mine);
                    arrive(p_full0 + 16u * buf);
                    arrive(p_full0 + 16u * buf + 8u);
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
                if (!(ok = turn(gj)))
                    break;
                const float m_old = j > 0 ? row_max[row] : -INFINITY;
                const float m_new = !dead && m_tile > m_old + RESCALE_THRESHOLD ? m_tile : m_old;
                row_max[row] = m_new;
                arrive(max_mine);
                const float alpha = m_new == m_old ? 1.f : ptx::ex2(m_old - m_new);  // of O, which has the tiles before
                l *= m_new == m_used ? 1.f : ptx::ex2(m_used - m_new);
                m_used = m_new;
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
                // P is handed over in halves, for its product to begin with the first one
#pragma unroll 1
                for (int w = 0; w < TILE; w += TILE / 2) {
                    if (w >= w0 && w < w1) {
                        ptx::tmem_wait_ld();
                        ptx::tmem_ld32(ts + w + 32, b);
                        weights(a, ts + w / 2);
                        ptx::tmem_wait_ld();
                        if (w + 64 < w1)
                            ptx::tmem_ld32(ts + w + 64, a);
                        weights(b, ts + w / 2 + 16);
                        ptx::tmem_wait_st();
                    }
                    ptx::tc_fence_before();
                    arrive(p_full0 + 16u * buf + w / 8);
                }
                float sum0, sum1, sum2, sum3;
                ptx::f2_unpack(sum01, sum0, sum1);
                ptx::f2_unpack(sum23, sum2, sum3);
                l += (sum0 + sum1) + (sum2 + sum3);
            }
            if (!ok)
                break;
            const bool latest = ((g0 + n - 1) & 1) == group;
            if (!latest) {  // the other group has the last tile, and the maximum of all
                if (!(ok = turn(g0 + n)))
                    break;
                if (l != 0.f)
                    l *= ptx::ex2(m_used - row_max[row]);
            }
            if (k > 0 && !(ok = wait_all(sum_free, (k - 1) & 1, SITE_O_DONE)))
                break;
            if (latest)
                row_m[row] = m_used;
            row_l[group * TILE + row] = l;
            arrive(sum_full);
            g0 += n;
        }
        ptx::tmem_wait_ld();  // (where a wait ran out)
    } else {
        // --------------------------------------- rows' ends: O over l, to the output or to the workspace; and the run's units, looked
        // up ahead by warp 11, whose rows are the last that a small unit has
        const int w4 = warp & 3, row = w4 * 32 + lane;
        const int row_tok = row / p.heads, row_head = row - row_tok * p.heads;
        const uint32_t t_o = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + L::TM_O;
        bool ok = true;
        int g0 = 0;
        Unit un;
        int published = 0, longest = 1;  // units, and the tiles of the longest: its end may be what is waited for
        bool more = warp == 11 && p.no_units == 0;
        if (more)
            runs.start(p, sums);
        for (int k = 0;; ++k) {
#pragma unroll 1
            for (; more && published < k + PL::UNITS; ++published) {
                const Unit next = runs.next(p);
                const int at = published % PL::UNITS;
                if (published >= PL::UNITS && !wait_all(unit_free0 + 8u * at, (published / PL::UNITS - 1) & 1, SITE_Q_FULL, longest)) {
                    ok = false;
                    break;
                }
                more = next.n >= 0;
                longest = max(longest, next.n);
                if (lane == 0) {
                    ring[at] = next;
                    ptx::mbar_arrive(unit_full0 + 8u * at);
                }
            }
            if (!ok || !take(k, un))
                break;
            const int n = un.n, last = g0 + n - 1;
            if (threadIdx.x == 8 * 32 && un.join >= 0)
                (un.prefix() ? p.joins_p : p.joins_o)[un.join] = make_int2(run, runs.parts_of(un.after));
            if (!(ok = wait_all(sum_full, k & 1, SITE_O_DONE, n)))
                break;
            const float m = row_m[row], l = row_l[row] + row_l[TILE + row];
            arrive(sum_free);
            if (!(ok = wait_all(o_done0 + 8u * (last % O_DONE_RING), (last / O_DONE_RING) & 1, SITE_O_DONE)) ||
                !(ok = wait_all(odd_full, k & 1, SITE_O_DONE)))
                break;
            const uint32_t odd = *odd_keys, onto = odd_keys[1];
            if (w4 * 32 < un.toks * p.heads) {
                ptx::tc_fence_after();
                const bool none = l == 0.f;  // the row saw no key, and its O is 0
                const float inv = none ? 0.f : 1.f / l;
                // the row of q and o, -1 where there is none
                const int at = row_tok < un.toks && row_head < un.live ? (un.q_tok + row_tok) * p.Hq + un.head + row_head : -1;
                const bool slot = un.dest >= 0, direct = un.dest == DEST_DIRECT;
                float *const part = slot ? p.parts + un.dest * part_floats<D>(p.part_rows) : un.prefix() ? p.rows_p : p.rows_o;
                char *const to = direct ? reinterpret_cast<char *>(p.o + static_cast<long long>(at) * D)
                                        : reinterpret_cast<char *>(part + static_cast<long long>(slot ? row : at) * D);
                if (onto == 0u) {  // no product was made
                    const uint32_t zeros[16] = {};
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16)
                        ptx::tmem_st16(t_o + c0, zeros);
                    ptx::tmem_wait_st();
                }
                // 16 channels at a time in loops that the instruction buffers hold: straight code, run once a unit, is fetched as it
                // runs, at some 9 cycles an instruction, and the next unit's first product waits for this.
                auto read = [&](int c0, uint32_t (&o)[16]) {
                    tmem_ld16(t_o + c0, o);
                    ptx::tmem_wait_ld();
                    if (c0 + 16 == D) {
                        ptx::tc_fence_before();
                        arrive(o_free);
                    }
                };
                const uint64_t inv2 = ptx::f2_pack(inv, inv);
                const uint32_t live = at >= 0 ? 1u : 0u;
                if (direct) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t o[16], w[8];
                        read(c0, o);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float y0, y1;
                            ptx::f2_unpack(mul2(f2_of(o, 2 * x), inv2), y0, y1);
                            w[x] = pack2<BF16>(y0, y1);
                        }
                        st_global_v4(to + 2 * c0, w, live);  // (o lies on 16 bytes, the workspace's rows on 32)
                        st_global_v4(to + 2 * c0 + 16, w + 4, live);
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t o[16], w[16];
                        read(c0, o);
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            float y0, y1;
                            ptx::f2_unpack(mul2(f2_of(o, x), inv2), y0, y1);
                            w[x] = __float_as_uint(y0);
                            w[x + 1] = __float_as_uint(y1);
                        }
                        st_global_v8(to + 4 * c0, w, live);
                        st_global_v8(to + 4 * c0 + 32, w + 8, live);
                    }
                }
                if (at >= 0) {
                    if (odd != 0u)
                        add_odd<D, BF16>(p, un.table, un.kv, un.pos0, odd & below(row_tok), to, direct, 0, 1);
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

struct Cache16Maps {
    CUtensorMap q_prefix, q_own, k, v;  // Q by the boxes of a block of a prefix and of a sequence
};

template <int D, bool BF16>
cudaError_t launch_cache16_attn(const Cache16Maps &m, const Cache16Params &p, cudaStream_t st)
{
    using PL = c16::Plan<D>;
    static unsigned long long done = 0;
    const cudaError_t e = set_smem_once(cache16_attn_kernel<D, BF16>, PL::SMEM_BYTES, done);
    if (e != cudaSuccess)
        return e;
    // Both start where CTAs of the kernel before them end (if that one lets them), not when the last one has.
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    auto launch = [&](auto kern, unsigned grid, int threads, int bytes, const auto &...args) {
        cudaLaunchConfig_t config{};
        config.gridDim = dim3(grid);
        config.blockDim = dim3(threads);
        config.dynamicSmemBytes = bytes;
        config.stream = st;
        config.attrs = &early;
        config.numAttrs = 1;
        return cudaLaunchKernelEx(&config, kern, args...);
    };
    const cudaError_t f =
        launch(cache16_attn_kernel<D, BF16>, p.sms, c16::THREADS, PL::SMEM_BYTES, m.q_prefix, m.q_own, m.k, m.v, p);
    if (f != cudaSuccess)
        return f;
    const unsigned rows = static_cast<unsigned>(p.nseq * p.n * p.Hq);
    constexpr int WARPS = c16::JOIN_THREADS / 32;
    // A row a warp once that still gives every SM two blocks: 2048 rows of 64 x 8k in 45.3 us (a row a block: 47.3), 8192 of 256 x 16k in
    // 130 (140); below, a row a block: 256 rows of 8 x 16k, nine parts each, in 52.4 us (a row a warp: 54.5).
    return rows >= 2u * p.sms * WARPS
               ? launch(cache16_join_kernel<D, BF16, 1>, (rows + WARPS - 1) / WARPS, c16::JOIN_THREADS, 0, p)
               : launch(cache16_join_kernel<D, BF16, WARPS>, rows, c16::JOIN_THREADS, 0, p);
}

// One per (head dim, dtype).
cudaError_t cache16_attn_d128_fp16(const Cache16Maps &m, const Cache16Params &p, cudaStream_t st);
cudaError_t cache16_attn_d128_bf16(const Cache16Maps &m, const Cache16Params &p, cudaStream_t st);
cudaError_t cache16_attn_d256_fp16(const Cache16Maps &m, const Cache16Params &p, cudaStream_t st);
cudaError_t cache16_attn_d256_bf16(const Cache16Maps &m, const Cache16Params &p, cudaStream_t st);

}  // namespace sdp
