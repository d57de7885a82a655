// Entry points of the attention over the 16-bit paged cache (cache16_attn.cuh): checks, the launch shape, the tensor maps
// and the dispatch on (head dim, dtype).
#include <algorithm>
#include <cmath>

#include "cache16_attn.cuh"
#include "sdp.h"

namespace {

constexpr int kMaxRows = 32;  // a bit each in the mask of a unit's keys whose V is not finite

struct Shape {
    int heads, head_blocks, toks_p, toks_o, blocks_o, blocks_p, part_rows, sms;
    // the workspace: parts; rows and joins of the sequences, then of the prefixes
    long long rows_o, rows_p, joins_o, joins_p, bytes;
};

// Sections of the workspace begin on 32 bytes of it, after at most 16 bytes that its own start lacks.
long long align32(long long x) { return (x + 31) / 32 * 32; }

// keys, prefix_keys: the most that a sequence's table and a prefix's can hold.
int shape_of(int nseq, int rows, int Hq, int Hkv, int D, int dtype, int ngroups, long long keys, long long prefix_keys, Shape *sh)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (nseq <= 0 || rows <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || ngroups < 0)
        return SDP_ERR_INVALID_ARG;
    if (rows > kMaxRows)
        return SDP_ERR_UNSUPPORTED;
    // 31 bits for a row of q and for an entry of the list of problems
    const long long tokens = static_cast<long long>(nseq) * rows;
    if (tokens > INT32_MAX / Hq || nseq > 1 << 30 || ngroups > 1 << 29)
        return SDP_ERR_OVERFLOW;
    const int G = Hq / Hkv;
    sh->heads = std::min(G, sdp::c16::TILE);
    sh->head_blocks = (G + sh->heads - 1) / sh->heads;
    sh->toks_p = sdp::c16::TILE / sh->heads;
    sh->toks_o = std::min(rows, sh->toks_p);
    sh->blocks_o = (rows + sh->toks_o - 1) / sh->toks_o;
    sh->blocks_p = (rows + sh->toks_p - 1) / sh->toks_p;
    const int most = ngroups > 0 ? static_cast<int>(std::min<long long>(sh->toks_p, tokens)) : sh->toks_o;
    sh->part_rows = most * sh->heads;
    // 31 bits for the positions that the work is cut by, whatever the lengths: tiles, and what the problems' ends count
    auto positions = [](long long k) { return static_cast<double>(k / sdp::c16::TILE + 1 + sdp::c16::OVERHEAD); };
    const double own_blocks = static_cast<double>(nseq) * sh->blocks_o, shared_blocks = static_cast<double>(tokens) / sh->toks_p + ngroups;
    if ((own_blocks * positions(keys) + (ngroups > 0 ? shared_blocks * positions(prefix_keys) : 0.0)) * Hkv * sh->head_blocks > INT32_MAX)
        return SDP_ERR_OVERFLOW;
    int dev = 0;
    const int rc = sdp::current_device(&dev, &sh->sms);
    if (rc != SDP_OK)
        return rc;
    const long long part = D == 128 ? sdp::c16::part_floats<128>(sh->part_rows) : sdp::c16::part_floats<256>(sh->part_rows);
    const long long problems = static_cast<long long>(nseq) * Hkv * sh->head_blocks;
    const long long whole = ngroups > 0 ? align32(tokens * Hq * (D + 2) * 4) : 0;  // O, m and l of every row
    sh->rows_o = align32(2 * sh->sms * part * 4);
    sh->rows_p = sh->rows_o + whole;
    sh->joins_o = sh->rows_p + whole;
    sh->joins_p = sh->joins_o + align32(problems * sh->blocks_o * static_cast<long long>(sizeof(int2)));
    sh->bytes = sh->joins_p + (ngroups > 0 ? align32(problems * sh->blocks_p * static_cast<long long>(sizeof(int2)))
                                           : 0);
    sh->bytes += 16;
    return SDP_OK;
}

}  // namespace

extern "C" long long sdp_fwd_cache16_workspace_bytes(int nseq, int rows, int Hq, int Hkv, int D, int dtype, int ngroups)
{
    Shape sh;
    const int rc = shape_of(nseq, rows, Hq, Hkv, D, dtype, ngroups, 0, 0, &sh);
    return rc != SDP_OK ? rc : sh.bytes;
}

extern "C" int sdp_fwd_cache16(const void *q, const void *k_cache, const void *v_cache, int num_pages, int page_size,
                               const int *block_table, long long table_stride, int max_pages, const int *cache_lens,
                               const int *prefix_table, long long prefix_stride, int prefix_pages,
                               const int *prefix_lens, const int *cu_groups, int ngroups, void *o, float *lse, int nseq,
                               int rows, int Hq, int Hkv, int D, float scale, int dtype, void *workspace,
                               unsigned long long workspace_bytes, void *stream)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_table == nullptr || cache_lens == nullptr ||
        o == nullptr || workspace == nullptr)
        return SDP_ERR_INVALID_ARG;
    const float c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // of powers of two
    if (num_pages <= 0 || page_size <= 0 || page_size % 16 != 0 || max_pages <= 0 || table_stride < 0 ||
        !std::isfinite(c) || o == q || o == k_cache || o == v_cache || ngroups < 0)
        return SDP_ERR_INVALID_ARG;
    if (ngroups > 0 && (prefix_table == nullptr || prefix_lens == nullptr || prefix_pages <= 0 || prefix_stride < 0 ||
                        (cu_groups == nullptr && ngroups != 1)))
        return SDP_ERR_INVALID_ARG;
    using sdp::is_aligned;
    if (!is_aligned(q, 16) || !is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(o, 16) ||
        !is_aligned(lse, 4) || !is_aligned(block_table, 4) || !is_aligned(cache_lens, 4) || !is_aligned(prefix_table, 4) ||
        !is_aligned(prefix_lens, 4) || !is_aligned(cu_groups, 4) || !is_aligned(workspace, 16))
        return SDP_ERR_ALIGNMENT;
    // 31 bits for the indexes of keys, and of those looked up behind the last one, and for a page's row of heads
    constexpr long long most = INT32_MAX - sdp::c16::KEYS_BEHIND;
    if (static_cast<long long>(max_pages) * page_size > most ||
        (ngroups > 0 && static_cast<long long>(prefix_pages) * page_size > most) || num_pages > INT32_MAX / std::max(Hkv, 1))
        return SDP_ERR_OVERFLOW;
    Shape sh;
    int rc = shape_of(nseq, rows, Hq, Hkv, D, dtype, ngroups, static_cast<long long>(max_pages) * page_size,
                      static_cast<long long>(prefix_pages) * page_size, &sh);
    if (rc != SDP_OK)
        return rc;
    if (workspace_bytes < static_cast<unsigned long long>(sh.bytes))
        return SDP_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if ((rc = sdp::current_device(&dev, &sms)) != SDP_OK)
        return rc;
    sdp::Cache16Params p{};
    if ((rc = sdp::status_word(dev, &p.status)) != SDP_OK)
        return rc;
    const int box = std::min(page_size & -page_size, 128);  // the largest power of two that divides a page
    const long long tokens = static_cast<long long>(nseq) * rows, planes = static_cast<long long>(num_pages) * Hkv;
    sdp::Cache16Maps m;
    if ((rc = sdp::tensor_map_tokens(&m.q_prefix, q, dtype, D, tokens, Hq, sh.heads, sh.toks_p)) != SDP_OK ||
        (rc = sdp::tensor_map_tokens(&m.q_own, q, dtype, D, tokens, Hq, sh.heads, sh.toks_o)) != SDP_OK ||
        (rc = sdp::tensor_map(&m.k, k_cache, dtype, D, page_size, planes, box)) != SDP_OK ||
        (rc = sdp::tensor_map(&m.v, v_cache, dtype, D, page_size, planes, std::min(box, 64))) != SDP_OK)
        return rc;
    char *const ws = static_cast<char *>(workspace) + (sdp::is_aligned(workspace, 32) ? 0 : 16);
    p.o = static_cast<uint16_t *>(o);
    p.lse = lse;
    p.v = static_cast<const uint16_t *>(v_cache);
    p.table = block_table;
    p.lens = cache_lens;
    p.prefix_table = prefix_table;
    p.prefix_lens = prefix_lens;
    p.cu_groups = cu_groups;
    p.table_stride = table_stride;
    p.prefix_stride = prefix_stride;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.page_inverse = page_size == 16 ? 0xffffffffu : static_cast<unsigned>((1ull << 32) / (page_size / 16));
    p.max_pages = max_pages;
    p.prefix_pages = prefix_pages;
    p.nseq = nseq;
    p.ngroups = ngroups;
    p.n = rows;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.heads = sh.heads;
    p.head_blocks = sh.head_blocks;
    p.toks_p = sh.toks_p;
    p.toks_o = sh.toks_o;
    p.blocks_o = sh.blocks_o;
    p.blocks_p = sh.blocks_p;
    p.box = box;
    for (p.box_log2 = 4; (1 << p.box_log2) < box;)
        ++p.box_log2;
    p.sms = sms;
    p.part_rows = sh.part_rows;
    p.parts = reinterpret_cast<float *>(ws);
    p.rows_o = reinterpret_cast<float *>(ws + sh.rows_o);
    p.rows_p = reinterpret_cast<float *>(ws + sh.rows_p);
    p.joins_o = reinterpret_cast<int2 *>(ws + sh.joins_o);
    p.joins_p = reinterpret_cast<int2 *>(ws + sh.joins_p);
    p.timeout_ns = sdp::wait_timeout_ns();
    p.no_copies = sdp::debug_flags() & 1;
    p.no_units = sdp::debug_flags() & 256;
    p.c = c != 0.f ? c : 1e-37f;  // (scores of 0, where those that a row does not see are still -inf)
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (D == 128)
        e = dtype == SDP_BF16 ? sdp::cache16_attn_d128_bf16(m, p, st) : sdp::cache16_attn_d128_fp16(m, p, st);
    else
        e = dtype == SDP_BF16 ? sdp::cache16_attn_d256_bf16(m, p, st) : sdp::cache16_attn_d256_fp16(m, p, st);
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}
