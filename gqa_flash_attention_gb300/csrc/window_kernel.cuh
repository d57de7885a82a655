// Attention with a sliding window and first tokens that stay visible (sdp_fwd_window,
// sdp_fwd_varlen_window): a query row at position p of its sequence sees the keys j <= p with
// j > p - W or j < sinks. A sequence's rows are its last sq positions (p = skv - sq + i), so the
// same call serves a whole prompt and a chunk behind a cached prefix.
//
// Arithmetic and roles are those of the single-CTA kernel (sdp_fwd_kernel.cuh): 128-row query
// tiles, 128-key tiles through a TMA ring, S = Q K^T and O += P V on tcgen05 with both
// accumulators in tensor memory, one thread a row for the softmax with a lazily moved maximum. As
// there, scores, weights and sums are fp32 and the weights are rounded to the 16-bit type for P V, whose
// operands have one type: half a step of each weight (2^-9 of it in bf16), of the order of the output's own rounding.
// What the window changes:
//
//  - A unit (query tile, head) reads only the tiles of the sinks and those from its first row's
//    window start to its last row's own key: min(p, W) / 128 + 2 of them, whatever the length.
//  - Units are short (W = 1024: 10 tiles), so set-up, tear-down and the first loads would take a
//    third of the time: the kernel is persistent, one CTA an SM, with the next unit's Q and K/V
//    loads and first scores running during the current unit's end (barrier phases and ring
//    positions count across units). Units cost alike and neighbours share their K/V, so CTA c
//    takes units c, c + C, c + 2C, ... with no counter to claim from, the same in a captured
//    graph. A warpgroup of its own writes a unit's rows while the softmax warps are with the next
//    unit, and a warp of its own looks the units up ahead: with both done by the softmax warps, 7.8 us
//    passed at each unit's end at D = 256 (1.1 us a tile), and 12 packed prompts (W = 1024, D = 256)
//    took 903 us instead of 789, 16384 rows (W = 4096, D = 128) 697 instead of 634. A launch of one unit
//    a CTA at most has no next unit to go on with, and the hand-overs cost it 1.8 us of 8.3: it
//    runs without them (WINDOW_ONE). (The figures of these comments are of 20 calls in a row; in runs of hundreds
//    the clocks settle lower, at 800 instead of 724 us for the prompts and 690 instead of 634 for the 16384 rows.) O leaves tensor memory 32 columns at a time, stored as it comes: taken
//    out whole first, which frees it earlier, the first was slower (812 us), its unrolled code larger.
//  - What bounds a tile at D = 256 is shared memory: the products read Q, K and V there and the copies write
//    K and V, 320 KB a tile, where an SM moves 128 bytes a cycle (2560 cycles; 2570 measured; the products alone
//    take 2048). At D = 128 a tile takes 1210 to 1390 cycles, with 160 KB (1280 cycles), products of 1024 and a
//    softmax chain of about as long: which of them is the bound has not been told apart, since what shortens
//    one adds hand-overs (below). So at D = 256 two CTAs
//    run as a pair (WINDOW_PAIR): two heads of a group have the same window, each CTA holds half of
//    each K and V tile, and one product of 256 rows reads both halves: 12 packed prompts 786 -> 724 us. At
//    D = 128 the pair's hand-overs between
//    CTAs cost more than the copies saved (634 -> 704 us), so it keeps to one CTA. (Half of a tile's keys
//    a thread, in two softmax warpgroups, took 699 us; handing P over in four parts, which a pair of the
//    dense kernel gains from, 750 us for the prompts.)
//  - Only the tiles that cut a window or the diagonal (two or three a unit, plus the sinks') are
//    masked, from four 32-bit words of visible keys a row; the others run without a test.
//  - A row may see nothing in a tile, or at all (more rows than keys): its maximum stays -inf, its
//    weights 0, and at the end O = 0 and LSE = -inf.
//  - Masked weights are exactly 0, but 0 times an infinity or a NaN in V is NaN: a row whose O is
//    not finite is computed again from the keys it sees alone (recompute_row), so what lies outside
//    a window stays outside. Rows that are finite pay one multiply-add an element. A row computed
//    again takes 10 (D = 128) to 13 us (D = 256) for every 32 keys, which over a long window is longer
//    than any wait of the pipeline may last, so it is only marked in O while units run, and computed once
//    the CTA's last unit is written, when no warp waits for another. (9000 rows of 8 heads that all see an
//    infinity in 4000 keys: 112 ms, of finite values 0.11.)
#pragma once

#include "sdp_fwd_pair.cuh"

namespace sdp {

struct WindowParams {
    KernelParams k;  // as the other forward kernels take it (causal 0: the compact list in sequence order)
    const void *q, *kk, *v;
    // element strides of a plane (head) and of a row
    long long q_plane, q_row, kv_plane, kv_row;
    int window, sinks;
    int pack_sq;  // > 0: a group's query heads run as one head of G * pack_sq rows
};

// How a launch runs: a unit a CTA, several a CTA with a warpgroup that writes their rows, or the latter by pairs of
// CTAs.
enum WindowForm { WINDOW_ONE, WINDOW_MANY, WINDOW_PAIR };

template <int D, bool PAIR>
struct WindowLayout {
    using L = Layout<D>;
    using PL = PairLayout<D>;
    static constexpr int BAR_AREA = 512;
    // Query tiles in shared memory: two at D=128 (the next unit's Q loads while this unit runs),
    // one at D=256 (two would leave too few ring slots).
    static constexpr int QB = D == 128 ? 2 : 1;
    static constexpr int SLOT_BYTES = PAIR ? PL::HALF_BYTES : L::CHUNK_BYTES;
    static constexpr int CPT = PAIR ? 1 : L::CHUNKS_PER_TILE;  // slots a K tile (or a V tile)
    static constexpr int NSLOTS = (L::SMEM_LIMIT - BAR_AREA - 2 * L::BM * 4 - 4 * 48 - 1024 - QB * L::Q_BYTES) / SLOT_BYTES;
    // q_full[QB], slot_full[NS], slot_empty[NS], s_full[NB], p_full[NB], o_done[ring], final[2],
    // q_free[QB], o_free, sum_full[2], sum_free[2], unit_full[UNITS], unit_free[UNITS]
    static constexpr int UNITS = 4;  // units looked up ahead
    static constexpr int NBARS = QB + 2 * NSLOTS + 2 * L::NSBUF + O_DONE_RING + 2 + QB + 1 + 4 + 2 * UNITS;
    static constexpr int BAR_OFF = QB * L::Q_BYTES + NSLOTS * SLOT_BYTES;
    static constexpr int HOLDER_OFF = BAR_OFF + 8 * NBARS;  // TMEM address, then the abort flag
    static constexpr int SUM_OFF = BAR_OFF + BAR_AREA;  // two units' row factors, for the rows' ends
    static constexpr int UNIT_OFF = SUM_OFF + 2 * L::BM * 4;
    static constexpr int UNIT_AREA = UNITS * 48;
    static constexpr int SMEM_BYTES = UNIT_OFF + UNIT_AREA + 1024;
    static_assert(HOLDER_OFF + 8 <= BAR_OFF + BAR_AREA, "barrier area");
    static_assert(SMEM_BYTES <= L::SMEM_LIMIT, "shared memory");
    // Ring parity across units of any lengths (global load positions): the S issuer waits for
    // PV_{t-NSBUF} before its K slot and, with two chunks a tile, the PV issuer for P_j before its V
    // chunks, which the persistent kernel of the dense forward has checked by enumeration.
    static_assert(NSLOTS >= 4 && L::NSBUF <= 3, "ring parity soundness across units");
};

// Keys [0, n) of 32 as a bit mask.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// The mark of a row to be computed again, in its first element: a NaN in both types, and no other row that has been
// written holds one.
constexpr uint16_t ROW_AGAIN = 0x7fff;

// One row again, over the keys it sees alone: key ranges [0, a1) and [b0, b1) of the row's K/V plane.
// Called by a whole warp (the rare path of rows whose O is not finite). 32 keys a step, one a lane, for
// the scores; then each lane adds its D / 32 channels of their V rows.
template <int D, bool BF16>
static __device__ __noinline__ void recompute_row(const uint16_t *q, const uint16_t *k, const uint16_t *v, long long kv_row,
                                                  int a1, int b0, int b1, float c, uint16_t *o, float *lse)
{
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.f;
    const int n = a1 + max(0, b1 - b0);
    for (int t = 0; t < n; t += 32) {
        const int e = t + lane;
        const bool live = e < n;
        const long long key = e < a1 ? e : b0 + (e - a1);
        float s = 0.f;
        if (live) {
            const uint4 *kr = reinterpret_cast<const uint4 *>(k + key * kv_row), *qr = reinterpret_cast<const uint4 *>(q);
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = __ldg(kr + i), y = __ldg(qr + i);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float2 f, g;
                    if constexpr (BF16) {
                        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&xs[w]));
                        g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&ys[w]));
                    } else {
                        f = __half22float2(*reinterpret_cast<const __half2 *>(&xs[w]));
                        g = __half22float2(*reinterpret_cast<const __half2 *>(&ys[w]));
                    }
                    s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
                }
            }
            s *= c;
        }
        float mx = live ? s : -INFINITY;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float next = fmaxf(m, mx);
        const float ref = next == -INFINITY ? 0.f : next;
        const float alpha = m == -INFINITY ? 0.f : ptx::ex2(m - ref);
        m = next;
        const float w = live ? ptx::ex2(s - ref) : 0.f;
        float sum = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = (l == 0.f ? 0.f : l * alpha) + sum;
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = t == 0 ? 0.f : acc[i] * alpha;
        for (int x = 0; x < 32 && t + x < n; ++x) {
            const float wx = __shfl_sync(0xffffffffu, w, x);
            const long long kx = t + x < a1 ? t + x : b0 + (t + x - a1);
            const uint16_t *vr = v + kx * kv_row + lane * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint16_t u = __ldg(vr + i);
                float f;
                if constexpr (BF16)
                    f = __uint_as_float(static_cast<uint32_t>(u) << 16);
                else
                    f = __half2float(*reinterpret_cast<const __half *>(&u));
                acc[i] = fmaf(wx, f, acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; i += 2)
        *reinterpret_cast<uint32_t *>(o + lane * V + i) = pack2<BF16>(acc[i] / l, acc[i + 1] / l);
    if (lane == 0 && lse != nullptr)
        *lse = (m + ptx::lg2(l)) * LN2;
}

// Warpgroups: softmax, then the loading and issuing warps, then (OVERLAP) those that write the rows. Registers a
// thread of each with OVERLAP: the block launches with WINDOW_LAUNCH_REGS each, and the softmax takes what the
// second group gives back.
constexpr int WINDOW_LAUNCH_REGS = 168, WINDOW_SOFTMAX_REGS = 232, WINDOW_ISSUE_REGS = 104;
static_assert(WINDOW_SOFTMAX_REGS + WINDOW_ISSUE_REGS <= 2 * WINDOW_LAUNCH_REGS, "registers of the launch");
constexpr int window_threads(bool overlap) { return overlap ? 384 : 256; }

// OVERLAP: a warpgroup of its own writes a unit's rows while the softmax goes on with the next unit; without it the
// softmax warps do.
template <int D, bool BF16, bool VARLEN, WindowForm FORM>
__global__ void __launch_bounds__(window_threads(FORM != WINDOW_ONE), 1)
    window_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const WindowParams wp)
{
    constexpr bool PAIR = FORM == WINDOW_PAIR, OVERLAP = FORM != WINDOW_ONE;
    using L = Layout<D>;
    using PL = PairLayout<D>;
    using WL = WindowLayout<D, PAIR>;
    const KernelParams &p = wp.k;
    constexpr int NS = WL::NSLOTS;
    constexpr int NB = L::NSBUF;
    constexpr int CPT = WL::CPT;
    constexpr int QB = WL::QB;
    constexpr uint32_t IDESC_S = ptx::idesc_f16_f32acc(128, L::BN, BF16, false);
    constexpr uint32_t IDESC_PV = ptx::idesc_f16_f32acc(128, 128, BF16, true);
    constexpr uint32_t IDESC_S2 = ptx::idesc_f16_f32acc(256, L::BN, BF16, false);
    constexpr uint32_t IDESC_PV2 = ptx::idesc_f16_f32acc(256, D, BF16, true);
    const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
    const bool leader = rank == 0;  // issues the pair's products; its barriers count both CTAs' loads and arrivals

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_addr + pad;
    const uint32_t s_q0 = sbase;  // query tile b at s_q0 + b * Q_BYTES
    const uint32_t s_ring = sbase + QB * L::Q_BYTES;
    const uint32_t bar0 = sbase + WL::BAR_OFF;
    const uint32_t q_full0 = bar0;  // + 8 b
    const uint32_t slot_full0 = bar0 + 8u * QB;
    const uint32_t slot_empty0 = slot_full0 + 8u * NS;
    const uint32_t s_full0 = slot_empty0 + 8u * NS;
    const uint32_t p_full0 = s_full0 + 8u * NB;
    const uint32_t o_done0 = p_full0 + 8u * NB;
    const uint32_t final0 = o_done0 + 8u * O_DONE_RING;
    const uint32_t q_free0 = final0 + 16u;  // + 8 b: the S MMAs that read query tile b last are done
    const uint32_t o_free = q_free0 + 8u * QB;
    const uint32_t sum_full0 = o_free + 8u;  // + 8 (unit & 1): its row factors are there
    const uint32_t sum_free0 = sum_full0 + 16u;
    const uint32_t unit_full0 = sum_free0 + 16u, unit_free0 = unit_full0 + 8u * WL::UNITS;  // + 8 (i % UNITS)
    float *const row_factor = reinterpret_cast<float *>(smem + WL::SUM_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + WL::HOLDER_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // A unit's geometry: Q/O and K/V planes, its first row within its sequence (q0) and in the row
    // coordinate (q_row), the first K/V row, the sequence's rows, the position of its row 0, and its
    // tiles: ns of the sinks, then those from t_lo, n in all. n = 0: no key (its rows get O = 0 and
    // LSE = -inf); n < 0: nothing to do, in the ring: nor in any unit after it.
    struct __align__(16) Unit {
        int z_q, z_kv, q0, q_row, kv_row0, sq, pos0, t_lo, ns, n, unused[2];
        __device__ __forceinline__ int tile(int j) const { return j < ns ? j : t_lo + j - ns; }
    };
    int from = 0, before = 0;  // a sequence, and the tiles of those before it
    auto unit_of = [&](int u) {  // by a whole warp
        Unit r{};
        r.n = -1;
        const int hi = u % p.G;
        u /= p.G;
        if constexpr (VARLEN) {
            if (p.n_tiles > 0) {
                // Tile t of the list of those that exist, in sequence order: its sequence, from the sums of their
                // tiles, 32 sequences a step. A CTA's units move on through the list, so the search goes on from
                // the last one's place.
                const int t = u % p.n_tiles, g = u / p.n_tiles;
                const VarlenScan v{p.cu_q, p.cu_k, p.nseq, p.n_qtiles, p.Sq, p.Skv};
                if (t < before)
                    from = before = 0;
                int found = -1;
                for (; from < p.nseq; from += 32) {
                    bool bad;
                    const int tiles = varlen_tiles(v, from + lane, bad);
                    int incl = tiles;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int x = __shfl_up_sync(0xffffffffu, incl, d);
                        if (lane >= d)
                            incl += x;
                    }
                    incl += before;
                    const unsigned hit = __ballot_sync(0xffffffffu, incl - tiles <= t && t < incl);
                    if (hit != 0u) {
                        const int src = __ffs(hit) - 1;
                        found = ((from + src) * p.Hkv + g) * p.n_qtiles + t - __shfl_sync(0xffffffffu, incl - tiles, src);
                        break;
                    }
                    before = __shfl_sync(0xffffffffu, incl, 31);
                }
                if (found < 0)
                    return r;  // a slot past the last query tile
                u = found;
            }
        }
        const int qt = u % p.n_qtiles, bg = u / p.n_qtiles;
        const int b = bg / p.Hkv, g = bg - b * p.Hkv;
        r.z_q = VARLEN ? g * p.G + hi : b * p.Hq + g * p.G + hi;
        r.z_kv = VARLEN ? g : bg;
        r.q0 = qt * L::BM;
        const SeqGeom sg = seq_geom(p, b);
        if (!sg.ok) {
            if (lane == 0) {
                const uint32_t cta = blockIdx.x < 0xFFFFFFu ? blockIdx.x : 0xFFFFFFu;
                atomicCAS(p.status, 0u, SITE_SEQLENS | (cta << 8));
            }
            return r;
        }
        r.sq = sg.sq;
        if (r.q0 >= sg.sq)
            return r;  // a tile past the end of a shorter sequence
        r.q_row = sg.q_row0 + r.q0;
        r.kv_row0 = sg.kv_row0;
        r.pos0 = sg.skv - (wp.pack_sq > 0 ? wp.pack_sq : sg.sq);
        // positions of the tile's first and last row
        const int p_lo = r.pos0 + (wp.pack_sq > 0 ? 0 : r.q0);
        const int p_hi = r.pos0 + (wp.pack_sq > 0 ? wp.pack_sq - 1 : min(r.q0 + L::BM, sg.sq) - 1);
        r.n = 0;
        if (p_hi < 0)
            return r;
        r.t_lo = max(0, p_lo - wp.window + 1) / L::BN;
        r.ns = min((min(wp.sinks, p_hi + 1) + L::BN - 1) / L::BN, r.t_lo);
        r.n = r.ns + p_hi / L::BN + 1 - r.t_lo;
        return r;
    };

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
            ptx::mbar_init(p_full0 + 8u * i, PAIR ? 8 : 128);
        }
        for (int i = 0; i < O_DONE_RING; ++i)
            ptx::mbar_init(o_done0 + 8u * i, 1);
        ptx::mbar_init(final0, 1);
        ptx::mbar_init(final0 + 8u, 1);
        ptx::mbar_init(o_free, PAIR ? 8 : 4);  // one arrival a warp of the rows' ends
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(sum_full0 + 8u * b, 128);
            ptx::mbar_init(sum_free0 + 8u * b, 4);
        }
        for (int i = 0; i < WL::UNITS; ++i) {
            ptx::mbar_init(unit_full0 + 8u * i, 1);
            ptx::mbar_init(unit_free0 + 8u * i, leader ? 11 : 9);  // the warps that read it
        }
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 4 && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == 5) {
        if constexpr (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_addr(tmem_holder), L::TMEM_COLS);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_addr(tmem_holder), L::TMEM_COLS);
            ptx::tmem_relinquish();
        }
    }
    // OVERLAP: warp 7 looks up the units blockIdx.x, + gridDim.x, ... ahead of the others (in a batch of odd lengths
    // that takes a search and a few dependent loads) and hands those with rows on through a ring. Else a CTA has
    // one unit, which every warp looks up. k counts those with tiles.
    if (VARLEN && p.n_tiles > 0 && blockIdx.x == 0 && warp == 7) {  // all offsets: a bad sequence has no unit
        const VarlenScan v{p.cu_q, p.cu_k, p.nseq, p.n_qtiles, p.Sq, p.Skv};
        for (int i = lane; i < p.nseq; i += 32) {
            bool bad;
            varlen_tiles(v, i, bad);
            if (bad)
                atomicCAS(p.status, 0u, static_cast<unsigned>(SITE_SEQLENS));
        }
    }
    int u = static_cast<int>(blockIdx.x);
    auto next_unit = [&]() {
        Unit r;
        r.n = -1;
        while (u < p.units && r.n < 0) {
            r = unit_of(u);
            u += static_cast<int>(gridDim.x);
        }
        return r;
    };
    Unit ahead;
    if (!OVERLAP || warp == 7)
        ahead = next_unit();  // while tensor memory is allocated
    ptx::tc_fence_before();
    if constexpr (PAIR)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // Bounded waits as in the forward kernels, but inline: a call in a branch with registers of its own
    // (setmaxnreg) does not assemble. The limit holds a tile: who waits for `tiles` of them waits that much longer
    // (and stops with the others when the tile's own wait has run out).
    auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t site, int tiles = 1, bool peer = false) -> bool {
        // peer: the other CTA arrives, too
        auto try_wait = [&]() {
            if constexpr (PAIR)
                return peer ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
            else
                return ptx::mbar_try_wait(bar, parity);
        };
        bool done = try_wait();
        if (!__all_sync(0xffffffffu, done)) {
            const uint64_t t0 = ptx::globaltimer_ns();
            for (uint32_t it = 1; !__all_sync(0xffffffffu, done = try_wait()); ++it) {
                if ((it & 15u) != 0)
                    continue;
                const bool late = static_cast<float>(ptx::globaltimer_ns() - t0) > static_cast<float>(p.timeout_ns) * tiles;
                if (__any_sync(0xffffffffu, late || *abort_flag)) {
                    if (late && !done) {
                        *abort_flag = 1;
                        const uint32_t cta = blockIdx.x < 0xFFFFFFu ? blockIdx.x : 0xFFFFFFu;
                        atomicCAS(p.status, 0u, site | (cta << 8));
                    }
                    return false;
                }
            }
        }
        return true;
    };
    auto drain = [&](uint32_t bar, uint32_t parity) {  // of what this warp issued itself
        const uint64_t t0 = ptx::globaltimer_ns();
        while (!ptx::mbar_try_wait(bar, parity) && ptx::globaltimer_ns() - t0 <= p.timeout_ns) {
        }
    };

    // a warp's arrival on a barrier of the leader
    auto arrive_leader = [&](uint32_t bar) {
        __syncwarp();
        if (lane != 0)
            return;
        if constexpr (!PAIR)
            ptx::mbar_arrive(bar);
        else if (leader)
            ptx::mbar_arrive(bar);
        else
            ptx::mbar_arrive_cluster(ptx::map_to_rank(bar, 0));
    };
    // on a barrier, of a pair in both CTAs, once this warp's products so far are done
    auto commit = [&](uint32_t bar) {
        if constexpr (PAIR)
            ptx::mma_commit_pair_w(bar);
        else
            ptx::mma_commit_w(bar);
    };
    Unit *const ring = reinterpret_cast<Unit *>(smem + WL::UNIT_OFF);
    auto take = [&](int i, Unit &un) -> bool {  // unit i; false at the end or when a wait ran out
        if constexpr (!OVERLAP) {
            un = ahead;
            return i == 0 && un.n >= 0;
        }
        const int at = i % WL::UNITS;
        if (!wait_all(unit_full0 + 8u * at, (i / WL::UNITS) & 1, SITE_Q_FULL))
            return false;
        un = ring[at];
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(unit_free0 + 8u * at);
        return un.n >= 0;
    };
    auto o_tile_of = [&](const Unit &un) {
        return static_cast<uint16_t *>(p.o) + un.z_q * wp.q_plane + static_cast<long long>(un.q_row) * wp.q_row;
    };
    auto lse_of = [&](const Unit &un, int row) {
        return p.lse == nullptr ? nullptr : p.lse + static_cast<size_t>(un.z_q) * p.Sq + un.q_row + row;
    };
    auto no_key = [&](const Unit &un, int row) {  // the row of a unit without tiles
        if (un.q0 + row >= un.sq)
            return;
        for (int i = 0; i < D / 8; ++i)
            reinterpret_cast<uint4 *>(o_tile_of(un) + row * wp.q_row)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse != nullptr)
            *lse_of(un, row) = -INFINITY;
    };
    // A unit's rows, 32 of them by each of four warps (w4): O, complete with tile `last`, times inv_l (negative: the
    // row saw no key) to global memory, and O's tensor memory to the next unit's first PV. `marked` is set where a
    // row has to be computed again.
    auto write_rows = [&](const Unit &un, int w4, int last, float inv_l, bool &marked) -> bool {
        const int row = w4 * 32 + lane;
        const uint32_t t_o = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + L::TM_O;
        uint16_t *const o_tile = o_tile_of(un);
        const bool row_ok = un.q0 + row < un.sq, none = inv_l < 0.f;
        if (!wait_all(o_done0 + 8u * (last % O_DONE_RING), (last / O_DONE_RING) & 1, SITE_O_DONE))
            return false;
        ptx::tc_fence_after();
        float probe = 0.f;  // NaN once an element of the row is not finite
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            ptx::tmem_ld32(t_o + 32 * cc, o);
            ptx::tmem_wait_ld();
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float a = __uint_as_float(o[2 * i]), b = __uint_as_float(o[2 * i + 1]);
                probe = fmaf(a, 0.f, fmaf(b, 0.f, probe));
                pk[i] = none ? 0u : pack2<BF16>(a * inv_l, b * inv_l);
            }
            // four lanes' rows by four 16-byte units, transposed in two exchanges: lane l then holds
            // unit l & 3 of the rows l, l ^ 1, l ^ 2 and l ^ 3, and the four write 64 bytes of a row at once
            const bool odd = lane & 1, high = lane & 2;
            uint32_t own[2][4], next[2][4], out[4][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t u0 = pk[8 * h + x], u1 = pk[8 * h + 4 + x];
                    own[h][x] = odd ? u1 : u0;
                    next[h][x] = __shfl_xor_sync(0xffffffffu, odd ? u0 : u1, 1);
                }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                out[0][x] = high ? own[1][x] : own[0][x];
                out[1][x] = high ? next[1][x] : next[0][x];
                out[2][x] = __shfl_xor_sync(0xffffffffu, high ? own[0][x] : own[1][x], 2);
                out[3][x] = __shfl_xor_sync(0xffffffffu, high ? next[0][x] : next[1][x], 2);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (un.q0 + (row ^ i) < un.sq)
                    reinterpret_cast<uint4 *>(o_tile + (row ^ i) * wp.q_row)[4 * cc + (lane & 3)] =
                        make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]);
        }
        ptx::tc_fence_before();
        arrive_leader(o_free);
        const bool again = row_ok && !none && probe != 0.f;
        if (__any_sync(0xffffffffu, again)) {
            __syncwarp();  // the row's stores, by other lanes, before its mark
            if (again)
                o_tile[row * wp.q_row] = ROW_AGAIN;
            marked = true;
        }
        return true;
    };
    // The marked ones of the rows that this warp has written (the others hold no NaN), from the keys that they see.
    auto write_again = [&](const Unit &un, int w4) {
        const int row = w4 * 32 + lane;
        const bool mine = un.q0 + row < un.sq && o_tile_of(un)[row * wp.q_row] == ROW_AGAIN;
        for (unsigned left = __ballot_sync(0xffffffffu, mine); left != 0u; left &= left - 1u) {
            const int r = w4 * 32 + __ffs(left) - 1;
            const int at = un.pos0 + (wp.pack_sq > 0 ? (un.q0 + r) % wp.pack_sq : un.q0 + r);
            const int b0 = max(0, at - wp.window + 1);
            const long long q_off = un.z_q * wp.q_plane + static_cast<long long>(un.q_row + r) * wp.q_row;
            const long long kv_off = un.z_kv * wp.kv_plane + static_cast<long long>(un.kv_row0) * wp.kv_row;
            recompute_row<D, BF16>(static_cast<const uint16_t *>(wp.q) + q_off,
                                   static_cast<const uint16_t *>(wp.kk) + kv_off,
                                   static_cast<const uint16_t *>(wp.v) + kv_off, wp.kv_row, min(wp.sinks, b0), b0,
                                   at + 1, p.c, static_cast<uint16_t *>(p.o) + q_off,
                                   lse_of(un, r));
        }
    };
    if (warp >= 4 && warp < 8) {
        if constexpr (OVERLAP)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(WINDOW_ISSUE_REGS));
        if (warp == 4) {
            // ------------------------------------------------------ TMA producer
            if (!(p.debug_flags & DEBUG_NO_LOADS)) {  // whole warp; one elected lane issues
                int slot = 0, k = 0;
                uint32_t ph = 0, armed_mask = 0, armed_par = 0, q_armed = 0, q_par = 0;
                bool ok = true;
                auto load_box = [&](uint32_t dst, const CUtensorMap *map, uint32_t full, int x, int y, int z) {
                    if constexpr (PAIR)
                        ptx::tma_load_3d_pair_w(dst, map, full, x, y, z);
                    else
                        ptx::tma_load_3d_w(dst, map, full, x, y, z);
                };
                Unit un;
                for (int i = 0; ok && take(i, un); ++i) {
                    const int n = un.n;
                    if (n == 0)
                        continue;
                    const int b = k % QB;
                    if (k >= QB && !(ok = wait_all(q_free0 + 8u * b, ((k - QB) / QB) & 1, SITE_Q_FULL)))
                        break;
                    const uint32_t q_full = PAIR ? ptx::map_to_rank(q_full0 + 8u * b, 0) : q_full0 + 8u * b;
                    if (leader)
                        ptx::mbar_arrive_expect_tx_w(q_full0 + 8u * b, (PAIR ? 2 : 1) * L::Q_BYTES);
#pragma unroll
                    for (int c = 0; c < D / L::BOX_COLS; ++c)
                        load_box(s_q0 + b * L::Q_BYTES + c * L::BOX_BYTES, &tm_q, q_full, c * L::BOX_COLS, un.q_row, un.z_q);
                    q_armed |= 1u << b;
                    q_par = (q_par & ~(1u << b)) | (((k / QB) & 1u) << b);
                    // a K or V tile; of a pair each CTA loads its 64 keys of K and its half of V's columns
                    auto load_tile = [&](bool of_k, int j) -> bool {
                        const CUtensorMap *map = of_k ? &tm_k : &tm_v;
#pragma unroll
                        for (int ch = 0; ch < CPT; ++ch) {
                            if (!wait_all(slot_empty0 + 8u * slot, ph ^ 1u, SITE_SLOT_EMPTY))
                                return false;
                            const uint32_t own = slot_full0 + 8u * slot, full = PAIR ? ptx::map_to_rank(own, 0) : own;
                            if (leader)
                                ptx::mbar_arrive_expect_tx_w(own, (PAIR ? 2 : 1) * WL::SLOT_BYTES);
                            const uint32_t dst = s_ring + slot * WL::SLOT_BYTES;
                            const int y = un.kv_row0 + un.tile(j) * L::BN, r = static_cast<int>(rank);
                            if constexpr (!PAIR) {
                                load_box(dst, map, full, ch * 128, y, un.z_kv);
                                load_box(dst + L::BOX_BYTES, map, full, ch * 128 + L::BOX_COLS, y, un.z_kv);
                            } else if (of_k) {
#pragma unroll
                                for (int c = 0; c < D / 64; ++c)
                                    load_box(dst + c * PL::K_BOX_BYTES, map, full, c * 64, y + 64 * r, un.z_kv);
                            } else {
#pragma unroll
                                for (int c = 0; c < D / 128; ++c)
                                    load_box(dst + c * PL::V_BOX_BYTES, map, full, r * (D / 2) + c * 64, y, un.z_kv);
                            }
                            armed_mask |= 1u << slot;
                            armed_par = (armed_par & ~(1u << slot)) | (ph << slot);
                            if (++slot == NS) {
                                slot = 0;
                                ph ^= 1u;
                            }
                        }
                        return true;
                    };
                    ok = load_tile(true, 0);
                    for (int j = 0; ok && j < n; ++j) {
                        if (j + 1 < n)
                            ok = load_tile(true, j + 1);
                        if (ok)
                            ok = load_tile(false, j);
                    }
                    ++k;
                }
                // Every copy this thread issued lands before the CTA may exit (a pair's count on the leader's
                // barriers: its products have waited for them, and after a wait that ran out both CTAs linger).
                if constexpr (!PAIR) {
                    for (int b = 0; b < QB; ++b)
                        if (q_armed & (1u << b))
                            drain(q_full0 + 8u * b, (q_par >> b) & 1u);
                    for (int s = 0; s < NS; ++s)
                        if (armed_mask & (1u << s))
                            drain(slot_full0 + 8u * s, (armed_par >> s) & 1u);
                }
            }
        } else if (warp == 5 && leader) {
            // ------------------------------------------- S = Q K^T issuer
            const uint64_t dk = ptx::smem_desc_sw128(s_ring, 16, 1024);
            bool issued = false, ok = true;
            int g0 = 0, pos0 = 0, k = 0;  // tiles and ring chunks of the earlier units
            Unit un;
            for (int i = 0; ok && take(i, un); ++i) {
                const int n = un.n;
                if (n == 0)
                    continue;
                const int b = k % QB;
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
#pragma unroll
                    for (int ch = 0; ch < CPT; ++ch) {
                        const int pos = p0 + ch;
                        if (!(ok = wait_all(slot_full0 + 8u * (pos % NS), (pos / NS) & 1, SITE_SLOT_FULL)))
                            break;
                    }
                    if (!ok)
                        break;
                    ptx::tc_fence_after();
                    const uint32_t d_tmem = tmem + L::TM_S + (gt % NB) * L::BN;
#pragma unroll
                    for (int ch = 0; ch < CPT; ++ch) {
                        const int slot = (p0 + ch) % NS;
                        const uint64_t kslot = dk + static_cast<uint64_t>((slot * WL::SLOT_BYTES) >> 4);
                        if constexpr (PAIR) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t box = kk >> 2, off = (kk & 3) * 32;
                                ptx::mma_ss_pair_w(d_tmem, dq + ((box * PL::Q_BOX_BYTES + off) >> 4),
                                                   kslot + ((box * PL::K_BOX_BYTES + off) >> 4), IDESC_S2, kk != 0);
                            }
                            issued = true;
                            ptx::mma_commit_pair_w(slot_empty0 + 8u * slot);
                            continue;
                        }
                        const uint64_t qch = dq + static_cast<uint64_t>((2 * ch * L::BOX_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t off = ((kk >> 2) * L::BOX_BYTES + (kk & 3) * 32) >> 4;
                            ptx::mma_ss_w(d_tmem, qch + off, kslot + off, IDESC_S, (ch | kk) != 0);
                        }
                        issued = true;
                        ptx::mma_commit_w(slot_empty0 + 8u * slot);
                    }
                    commit(s_full0 + 8u * (gt % NB));
                }
                if (!ok)
                    break;
                commit(q_free0 + 8u * b);  // query tile b may take unit k + QB's Q
                g0 += n;
                pos0 += 2 * CPT * n;
                ++k;
            }
            if (issued) {  // all of this thread's MMAs complete before TMEM is freed
                commit(final0);
                drain(final0, 0);
            }
        } else if (warp == 6 && leader) {
            // ------------------------------------------ O += P V issuer
            const uint64_t dv = ptx::smem_desc_sw128(s_ring, L::BOX_BYTES, 1024);
            bool issued = false, ok = true;
            int g0 = 0, pos0 = 0, k = 0;
            Unit un;
            for (int i = 0; ok && take(i, un); ++i) {
                const int n = un.n;
                if (n == 0)
                    continue;
                for (int j = 0; ok && j < n; ++j) {
                    const int gj = g0 + j;
                    const int buf = gj % NB;
                    const int p0 = pos0 + pos_v<CPT>(j, n);
                    if constexpr (CPT == 1) {  // V_j's slot first, off the P_j -> PV_j path
                        if (!(ok = wait_all(slot_full0 + 8u * (p0 % NS), (p0 / NS) & 1, SITE_SLOT_FULL)))
                            break;
                    }
                    if (!(ok = wait_all(p_full0 + 8u * buf, (gj / NB) & 1, SITE_P_FULL, 1, PAIR)))
                        break;
                    // a unit's first PV overwrites O: the previous unit's epilogue must have read it
                    if (j == 0 && k > 0 && !(ok = wait_all(o_free, (k - 1) & 1, SITE_O_DONE, 1, PAIR)))
                        break;
                    ptx::tc_fence_after();
                    const uint32_t a_tmem = tmem + L::TM_S + buf * L::BN;
#pragma unroll
                    for (int ch = 0; ch < CPT; ++ch) {
                        const int pos = p0 + ch;
                        const int slot = pos % NS;
                        if constexpr (CPT != 1) {
                            if (!(ok = wait_all(slot_full0 + 8u * slot, (pos / NS) & 1, SITE_SLOT_FULL)))
                                break;
                            ptx::tc_fence_after();
                        }
                        const uint64_t vslot = dv + static_cast<uint64_t>((slot * WL::SLOT_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            if constexpr (PAIR)
                                ptx::mma_ts_pair_w(tmem + L::TM_O, a_tmem + kk * 8, vslot + ((kk * 2048) >> 4), IDESC_PV2,
                                                   (j > 0) || (kk > 0));
                            else
                                ptx::mma_ts_w(tmem + L::TM_O + ch * 128, a_tmem + kk * 8, vslot + ((kk * 2048) >> 4),
                                              IDESC_PV, (j > 0) || (kk > 0));
                        }
                        issued = true;
                        commit(slot_empty0 + 8u * slot);
                    }
                    if (!ok)
                        break;
                    commit(o_done0 + 8u * (gj % O_DONE_RING));
                }
                g0 += n;
                pos0 += 2 * CPT * n;
                ++k;
            }
            if (issued) {
                commit(final0 + 8u);
                drain(final0 + 8u, 0);
            }
        } else if (OVERLAP && (!PAIR || warp == 7)) {
            // ------------------------------------------ the units, ahead of the others
            int longest = 1;  // of the units so far: its end may be what a place in the ring waits for
            for (int i = 0;; ++i) {
                if (i > 0)
                    ahead = next_unit();
                const int at = i % WL::UNITS;
                if (i >= WL::UNITS && !wait_all(unit_free0 + 8u * at, (i / WL::UNITS - 1) & 1, SITE_Q_FULL, longest))
                    break;
                longest = max(longest, ahead.n);
                if (lane == 0) {
                    ring[at] = ahead;
                    ptx::mbar_arrive(unit_full0 + 8u * at);
                }
                if (ahead.n < 0)
                    break;
            }
        }
    } else if (warp < 4) {
        // --------------------------------------- softmax / correction
        if constexpr (OVERLAP)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(WINDOW_SOFTMAX_REGS));
        const int row = threadIdx.x;  // query row within the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t t_s = tmem + lane_off + L::TM_S;
        const uint32_t t_o = tmem + lane_off + L::TM_O;
        const float c = p.c;
        bool ok = true;
        int g0 = 0, k = 0;
        Unit un;
        for (int i = 0; ok && take(i, un); ++i) {
            const int n = un.n;
            if (n == 0) {
                if constexpr (!OVERLAP)
                    no_key(un, row);
                continue;
            }
            // this row's position; keys [0, pos] and (> pos - window or < sinks) are visible
            const int pos = un.pos0 + (wp.pack_sq > 0 ? (un.q0 + row) % wp.pack_sq : un.q0 + row);
            float m_used = -INFINITY, l = 0.f;
            bool s_seen = false;  // S_j's barrier was seen complete while tile j-1 ended
            for (int j = 0; j < n; ++j) {
                const int gj = g0 + j;
                const int buf = gj % NB;
                if (!__all_sync(0xffffffffu, s_seen)) {
                    if (!(ok = wait_all(s_full0 + 8u * buf, (gj / NB) & 1, SITE_S_FULL)))
                        break;
                }
                ptx::tc_fence_after();
                const uint32_t ts = t_s + buf * L::BN;
                uint32_t sr[128];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    ptx::tmem_ld32(ts + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * q]));
                ptx::tmem_wait_ld();
                float s[128];
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    s[i] = __uint_as_float(sr[i]);

                // Only a tile that holds a key some row of the warp must not see is masked: the
                // masked scores come out scaled (-inf where not seen), the others as they are.
                const int k0 = un.tile(j) * L::BN;
                const int hi = pos + 1 - k0, lo = pos - wp.window + 1 - k0, sk = wp.sinks - k0;  // i < hi && (i >= lo || i < sk)
                const bool masked = __any_sync(0xffffffffu, hi < L::BN || (lo > 0 && sk < L::BN));
                if (masked) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t vis = below(hi - 32 * w) & (~below(lo - 32 * w) | below(sk - 32 * w));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            s[32 * w + i] = (vis & (1u << i)) ? s[32 * w + i] * c : -INFINITY;
                    }
                }
                const float ce = masked ? 1.f : c;
                float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
                if (ce >= 0.f) {
#pragma unroll
                    for (int i = 4; i < 124; i += 8) {
                        mx0 = ptx::max3(mx0, s[i], s[i + 1]);
                        mx1 = ptx::max3(mx1, s[i + 2], s[i + 3]);
                        mx2 = ptx::max3(mx2, s[i + 4], s[i + 5]);
                        mx3 = ptx::max3(mx3, s[i + 6], s[i + 7]);
                    }
                    mx0 = ptx::max3(mx0, s[124], s[125]);
                    mx1 = ptx::max3(mx1, s[126], s[127]);
                    mx0 = ptx::max3(mx0, mx1, fmaxf(mx2, mx3));
                } else {
#pragma unroll
                    for (int i = 4; i < 124; i += 8) {
                        mx0 = ptx::min3(mx0, s[i], s[i + 1]);
                        mx1 = ptx::min3(mx1, s[i + 2], s[i + 3]);
                        mx2 = ptx::min3(mx2, s[i + 4], s[i + 5]);
                        mx3 = ptx::min3(mx3, s[i + 6], s[i + 7]);
                    }
                    mx0 = ptx::min3(mx0, s[124], s[125]);
                    mx1 = ptx::min3(mx1, s[126], s[127]);
                    mx0 = ptx::min3(mx0, mx1, fminf(mx2, mx3));
                }
                // -inf while the row has seen no key (and its weights are 2^(-inf - 0) = 0)
                const float m_tile = mx0 * ce;
                const float m_new = m_tile > m_used + RESCALE_THRESHOLD ? m_tile : m_used;
                const float alpha = m_new == m_used ? 1.f : ptx::ex2(m_used - m_new);
                const float neg_m = m_new == -INFINITY ? 0.f : -m_new;

                uint32_t pk[64];
                const uint64_t c2 = ptx::f2_pack(ce, ce), negm2 = ptx::f2_pack(neg_m, neg_m);
                uint64_t sum01 = ptx::f2_pack(0.f, 0.f), sum23 = sum01;
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    float x0, x1, x2, x3;
                    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[2 * i], s[2 * i + 1]), c2, negm2), x0, x1);
                    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[2 * i + 2], s[2 * i + 3]), c2, negm2), x2, x3);
                    const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1), p2 = ptx::ex2(x2), p3 = ptx::ex2(x3);
                    sum01 = ptx::f2_add(sum01, ptx::f2_pack(p0, p1));
                    sum23 = ptx::f2_add(sum23, ptx::f2_pack(p2, p3));
                    pk[i] = pack2<BF16>(p0, p1);
                    pk[i + 1] = pack2<BF16>(p2, p3);
                }
                // Poll S_{j+1}'s barrier now (same unit), so the answer returns while P_j is
                // stored and handed off.
                s_seen = j + 1 < n && ptx::mbar_test_wait(s_full0 + 8u * ((gj + 1) % NB), ((gj + 1) / NB) & 1);
                float sum0, sum1, sum2, sum3;
                ptx::f2_unpack(sum01, sum0, sum1);
                ptx::f2_unpack(sum23, sum2, sum3);
                ptx::tmem_st32(ts, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
                ptx::tmem_st32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
                ptx::tmem_wait_st();
                l = fmaf(l, alpha, (sum0 + sum1) + (sum2 + sum3));

                // Rescale O only in warps where some row's maximum moved (they wait for PV_{gj-1}).
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
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
                if constexpr (PAIR)
                    arrive_leader(p_full0 + 8u * buf);
                else
                    ptx::mbar_arrive(p_full0 + 8u * buf);
                m_used = m_new;
            }
            if (!ok)
                break;

            // the row's end: its log-sum-exp, and its factor for O
            const float inv_l = l == 0.f ? -1.f : 1.f / l;  // -1: the row saw no key
            if (p.lse != nullptr && un.q0 + row < un.sq)
                *lse_of(un, row) = l == 0.f ? -INFINITY : (m_used + ptx::lg2(l)) * LN2;
            if constexpr (OVERLAP) {
                const int b = k & 1;
                if (k >= 2 && !(ok = wait_all(sum_free0 + 8u * b, ((k >> 1) - 1) & 1, SITE_O_DONE)))
                    break;
                row_factor[b * L::BM + row] = inv_l;
                ptx::mbar_arrive(sum_full0 + 8u * b);
            } else {
                bool marked = false;
                if (!(ok = write_rows(un, warp, g0 + n - 1, inv_l, marked)))
                    break;
                if (marked)
                    write_again(un, warp);
            }
            g0 += n;
            ++k;
        }
    } else {
        // --------------------------------------- rows' ends: O times its factor, to global memory
        const int w4 = warp & 3, row = w4 * 32 + lane;
        bool ok = true, marked = false;
        int g0 = 0, k = 0;
        Unit un;
        for (int i = 0; ok && take(i, un); ++i) {
            const int n = un.n;
            if (n == 0) {
                no_key(un, row);
                continue;
            }
            const int b = k & 1;
            if (!(ok = wait_all(sum_full0 + 8u * b, (k >> 1) & 1, SITE_O_DONE, n)))
                break;
            const float inv_l = row_factor[b * L::BM + row];
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(sum_free0 + 8u * b);
            if (!(ok = write_rows(un, w4, g0 + n - 1, inv_l, marked)))
                break;
            g0 += n;
            ++k;
        }
        if (marked && !*abort_flag) {  // (the ring is done with: the units are looked up again)
            for (un = next_unit(); un.n >= 0; un = next_unit())
                if (un.n > 0)
                    write_again(un, w4);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) {
        // After a wait that ran out copies may be on their way to the pair; give them time before it exits.
        if (*abort_flag) {
            for (int i = 0; i < 100; ++i)
                ptx::nanosleep_ns(1000);
        }
        // Neither CTA leaves while the other may still signal its barriers or read its shared or tensor memory.
        ptx::cluster_sync();
    }
    if (warp == 5) {
        __syncwarp();
        ptx::tc_fence_after();
        if constexpr (PAIR)
            ptx::tmem_dealloc_pair(tmem, L::TMEM_COLS);
        else
            ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

template <int D, bool BF16>
cudaError_t launch_window(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream)
{
    const bool vl = p.k.cu_q != nullptr;
    const int sms = p.k.num_sms;
    // With a unit a CTA at most there is no next one to go on with, and the hand-over costs its latency (8.3 -> 10.1 us).
    // Pairs are two heads of a group; what they gain at D = 256 and cost at D = 128 is at the top of the file.
    const bool pairs = D == 256 && p.k.G % 2 == 0 && sms > 1 && !(p.k.debug_flags & DEBUG_SINGLE_CTA);
    const WindowForm form = p.k.units <= sms ? WINDOW_ONE : pairs ? WINDOW_PAIR : WINDOW_MANY;
    static unsigned long long set[2][3] = {};
    auto go = [&](auto kern, auto layout, const CUtensorMap &k) -> cudaError_t {
        constexpr int BYTES = decltype(layout)::SMEM_BYTES;
        cudaError_t e = set_smem_once(kern, BYTES, set[vl][form]);
        if (e != cudaSuccess)
            return e;
        cudaLaunchAttribute cluster{};
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim.x = form == WINDOW_PAIR ? 2 : 1;
        cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
        cudaLaunchConfig_t config{};
        const int most = form == WINDOW_PAIR ? sms / 2 * 2 : sms;
        config.gridDim = dim3(p.k.units < most ? p.k.units : most);
        config.blockDim = dim3(window_threads(form != WINDOW_ONE));
        config.dynamicSmemBytes = BYTES;
        config.stream = stream;
        config.attrs = &cluster;
        config.numAttrs = form == WINDOW_PAIR ? 1 : 0;
        return cudaLaunchKernelEx(&config, kern, m.q, k, m.v, p);
    };
    using Single = WindowLayout<D, false>;
    if constexpr (D == 256) {
        using Pair = WindowLayout<D, true>;
        if (form == WINDOW_PAIR)
            return vl ? go(window_kernel<D, BF16, true, WINDOW_PAIR>, Pair{}, m.k_half)
                      : go(window_kernel<D, BF16, false, WINDOW_PAIR>, Pair{}, m.k_half);
    }
    if (form == WINDOW_ONE)
        return vl ? go(window_kernel<D, BF16, true, WINDOW_ONE>, Single{}, m.k)
                  : go(window_kernel<D, BF16, false, WINDOW_ONE>, Single{}, m.k);
    return vl ? go(window_kernel<D, BF16, true, WINDOW_MANY>, Single{}, m.k)
              : go(window_kernel<D, BF16, false, WINDOW_MANY>, Single{}, m.k);
}

}  // namespace sdp
