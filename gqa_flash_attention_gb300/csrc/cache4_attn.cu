// Entry points of the attention over the 4-bit paged cache (cache4_attn.cuh): checks, the launch
// shape and the dispatch on (head dim, dtype, columns a warp).
#include <cmath>

#include "cache4_attn.cuh"
#include "sdp.h"

namespace {

constexpr int kMaxRows = 32;

struct Shape {
    bool wide;  // 16 columns a warp, else 8
    int chunks, sms, part_cols;
    long long parts_bytes, workspace_bytes;
};

int shape_of(int nseq, int rows, int Hq, int Hkv, int D, int dtype, Shape *sh)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (nseq <= 0 || rows <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return SDP_ERR_INVALID_ARG;
    if (rows > kMaxRows)
        return SDP_ERR_UNSUPPORTED;
    const long long columns = static_cast<long long>(Hq / Hkv) * rows;
    sh->wide = columns > 8;
    const long long chunks = sh->wide ? (columns + 15) / 16 : 1;
    if (static_cast<long long>(nseq) * Hkv > INT32_MAX || chunks * 16 > INT32_MAX / (static_cast<long long>(nseq) * Hkv))
        return SDP_ERR_OVERFLOW;
    sh->chunks = static_cast<int>(chunks);
    int dev = 0, sms = 0;
    const int rc = sdp::current_device(&dev, &sms);
    if (rc != SDP_OK)
        return rc;
    sh->sms = sms;
    const int most = sh->wide ? 16 : 8;
    sh->part_cols = columns < most ? static_cast<int>(columns) : most;
    // two parts a warp: the problem it continues and the one it begins
    const int warps = D == 128 ? (sh->wide ? sdp::c4::Plan<128, 2>::WARPS : sdp::c4::Plan<128, 1>::WARPS)
                               : (sh->wide ? sdp::c4::Plan<256, 2>::WARPS : sdp::c4::Plan<256, 1>::WARPS);
    sh->parts_bytes = 2LL * sms * warps * 4 *
                      (D == 128 ? sdp::c4::part_floats<128>(sh->part_cols) : sdp::c4::part_floats<256>(sh->part_cols));
    sh->workspace_bytes = sh->parts_bytes + static_cast<long long>(nseq) * Hkv * chunks * static_cast<long long>(sizeof(int2));
    return SDP_OK;
}

}  // namespace

extern "C" long long sdp_fwd_cache4_workspace_bytes(int nseq, int rows, int Hq, int Hkv, int D, int dtype)
{
    Shape sh;
    const int rc = shape_of(nseq, rows, Hq, Hkv, D, dtype, &sh);
    return rc != SDP_OK ? rc : sh.workspace_bytes;
}

extern "C" int sdp_fwd_cache4(const void *q, const void *k_codes, const void *k_scales, const void *v_codes,
                              const void *v_scales, int num_pages, int page_size, const int *block_table,
                              long long table_stride, int max_pages, const int *cache_lens, void *o, float *lse,
                              int nseq, int rows, int Hq, int Hkv, int D, float scale, int dtype, int window,
                              int sinks, void *workspace, unsigned long long workspace_bytes, void *stream)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (q == nullptr || k_codes == nullptr || k_scales == nullptr || v_codes == nullptr || v_scales == nullptr ||
        block_table == nullptr || cache_lens == nullptr || o == nullptr || workspace == nullptr)
        return SDP_ERR_INVALID_ARG;
    if (num_pages <= 0 || page_size <= 0 || page_size % 16 != 0 || max_pages <= 0 || table_stride < 0 || window < 0 ||
        sinks < 0 || !std::isfinite(scale) || o == q)
        return SDP_ERR_INVALID_ARG;
    using sdp::is_aligned;
    if (!is_aligned(q, 16) || !is_aligned(k_codes, 16) || !is_aligned(k_scales, 16) || !is_aligned(v_codes, 16) ||
        !is_aligned(v_scales, 16) || !is_aligned(o, 16) || !is_aligned(lse, 4) || !is_aligned(block_table, 4) ||
        !is_aligned(cache_lens, 4) || !is_aligned(workspace, 16))
        return SDP_ERR_ALIGNMENT;
    // 31 bits for token indexes up to a tile past the end
    if (static_cast<long long>(max_pages) * page_size > INT32_MAX - 64)
        return SDP_ERR_OVERFLOW;
    Shape sh;
    int rc = shape_of(nseq, rows, Hq, Hkv, D, dtype, &sh);
    if (rc != SDP_OK)
        return rc;
    if (workspace_bytes < static_cast<unsigned long long>(sh.workspace_bytes))
        return SDP_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if ((rc = sdp::current_device(&dev, &sms)) != SDP_OK)
        return rc;
    sdp::Cache4AttnParams p{};
    if ((rc = sdp::status_word(dev, &p.status)) != SDP_OK)
        return rc;
    p.q = static_cast<const uint16_t *>(q);
    p.o = static_cast<uint16_t *>(o);
    p.lse = lse;
    p.k_codes = static_cast<const uint8_t *>(k_codes);
    p.v_codes = static_cast<const uint8_t *>(v_codes);
    p.k_scales = static_cast<const uint32_t *>(k_scales);
    p.v_scales = static_cast<const uint32_t *>(v_scales);
    p.table = block_table;
    p.lens = cache_lens;
    p.workspace = static_cast<float *>(workspace);
    p.joins = reinterpret_cast<int2 *>(static_cast<char *>(workspace) + sh.parts_bytes);
    p.timeout_ns = sdp::wait_timeout_ns();
    p.table_stride = table_stride;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.nseq = nseq;
    p.n = rows;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.window = window;
    p.sinks = sinks;
    p.chunks = sh.chunks;
    p.part_cols = sh.part_cols;
    p.no_copies = sdp::debug_flags() & 1;
    p.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (D == 128)
        e = dtype == SDP_BF16 ? sdp::cache4_attn_d128_bf16(p, sh.sms, st) : sdp::cache4_attn_d128_fp16(p, sh.sms, st);
    else
        e = dtype == SDP_BF16 ? sdp::cache4_attn_d256_bf16(p, sh.sms, st) : sdp::cache4_attn_d256_fp16(p, sh.sms, st);
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}
