// sdp_cache16_append: checks, the launch shape and the dispatch of the kernel in qk_norm_rope.cuh with a cache.
//
// One pass over HBM: q's rows are read and written normed and turned, k's go into their pages so, v's as they are. Apart
// (sdp_qk_norm_rope, then a copy of k and v into the pages) k would be written and read once more.
#include "qk_norm_rope.cuh"
#include "sdp.h"

namespace {

using namespace sdp::rope;

template <int D, bool BF16>
cudaError_t launch(const RopeParams &p, const CacheDest &c, bool w32, bool interleaved, unsigned blocks, cudaStream_t st)
{
    auto go = [&](auto kern) {
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t config{};
        config.gridDim = dim3(blocks);
        config.blockDim = dim3(32 * kWarps);
        config.stream = st;
        config.attrs = &early;
        config.numAttrs = 1;
        return cudaLaunchKernelEx(&config, kern, p, c);
    };
    if (w32)
        return interleaved ? go(qk_norm_rope_kernel<D, BF16, true, false, true, true>)
                           : go(qk_norm_rope_kernel<D, BF16, true, false, false, true>);
    return interleaved ? go(qk_norm_rope_kernel<D, BF16, false, false, true, true>)
                       : go(qk_norm_rope_kernel<D, BF16, false, false, false, true>);
}

}  // namespace

extern "C" int sdp_cache16_append(void *k_cache, void *v_cache, int num_pages, int page_size, const int *block_table,
                                  long long table_stride, int max_pages, const void *q, long long q_st, long long q_sh,
                                  void *q_out, long long qo_st, long long qo_sh, const void *k, long long k_st,
                                  long long k_sh, const void *v, long long v_st, long long v_sh, const int *cu_seqlens,
                                  const int *cache_lens, int nseq, int tokens, const void *positions, long long p_st,
                                  int positions_64, const unsigned long long *turns, int rot_dim, float mscale,
                                  const void *q_weight, const void *k_weight, int weight_fp32, float eps,
                                  int interleaved, int Hq, int Hkv, int D, int dtype, void *stream)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (nseq <= 0 || tokens < 0 || Hq < 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || page_size % 16 != 0 ||
        max_pages <= 0 || table_stride < 0 || rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0)
        return SDP_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !(eps <= 3.0e38f) || !(mscale >= -3.0e38f && mscale <= 3.0e38f))
        return SDP_ERR_INVALID_ARG;
    if (tokens == 0)
        return SDP_OK;
    if (k_cache == nullptr || v_cache == nullptr || block_table == nullptr || k == nullptr || v == nullptr ||
        cu_seqlens == nullptr || cache_lens == nullptr || (Hq > 0 && (q == nullptr || q_out == nullptr)) ||
        (rot_dim > 0 && turns == nullptr) || k_cache == v_cache)
        return SDP_ERR_INVALID_ARG;
    using sdp::is_aligned;
    for (long long s : {q_st, q_sh, qo_st, qo_sh, k_st, k_sh, v_st, v_sh})
        if (s % 8 != 0)
            return SDP_ERR_ALIGNMENT;
    for (const void *x : {static_cast<const void *>(k_cache), static_cast<const void *>(v_cache), q,
                          static_cast<const void *>(q_out), k, v, q_weight, k_weight})
        if (!is_aligned(x, 16))
            return SDP_ERR_ALIGNMENT;
    if (!is_aligned(block_table, 4) || !is_aligned(cu_seqlens, 4) || !is_aligned(cache_lens, 4) ||
        !is_aligned(turns, 8) || !is_aligned(positions, positions_64 ? 8 : 4))
        return SDP_ERR_ALIGNMENT;
    if (static_cast<long long>(max_pages) * page_size > INT32_MAX || static_cast<long long>(Hq) + 2LL * Hkv > INT32_MAX)
        return SDP_ERR_OVERFLOW;
    int dev = 0, sms = 0;
    int rc = sdp::current_device(&dev, &sms);
    if (rc != SDP_OK)
        return rc;

    RopeParams p{};
    CacheDest c{};
    // The split of the passes over warps is qk_norm_rope's, with v's passes behind k's. (It counts on 32 warps an SM, of which 16 to 20
    // are resident, and a token's last run may be short: 3095 tokens of 48 passes are runs of 30 and 18.)
    const int rpp = 256 / D;
    const long long passes_q = (Hq + static_cast<long long>(rpp) - 1) / rpp;
    const long long passes_kv = (Hkv + static_cast<long long>(rpp) - 1) / rpp;
    const long long passes = passes_q + 2 * passes_kv;
    long long per = tokens * passes / (static_cast<long long>(sms) * 32);
    per = per < 1 ? 1 : (per > passes ? passes : per);
    const long long runs = (passes + per - 1) / per;
    const long long blocks = (tokens * runs + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX)
        return SDP_ERR_OVERFLOW;
    if ((rc = sdp::status_word(dev, &c.status)) != SDP_OK)
        return rc;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.qs[1] = q_st;
    p.qs[2] = q_sh;
    p.ks[1] = k_st;
    p.ks[2] = k_sh;
    p.qos[1] = qo_st;
    p.qos[2] = qo_sh;
    p.positions = positions;
    p.ps[1] = p_st;
    p.turns = turns;
    p.wq = q_weight;
    p.wk = k_weight;
    p.mscale = mscale;
    p.eps = eps;
    p.S = tokens;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.R = rot_dim;
    p.tokens = tokens;
    p.passes_q = static_cast<int>(passes_q);
    p.passes = static_cast<int>(passes);
    p.per_warp = static_cast<int>(per);
    c.k = static_cast<uint16_t *>(k_cache);
    c.v_pool = static_cast<uint16_t *>(v_cache);
    c.v = static_cast<const uint16_t *>(v);
    c.v_st = v_st;
    c.v_sh = v_sh;
    c.cu = cu_seqlens;
    c.lens = cache_lens;
    c.table = block_table;
    c.table_stride = table_stride;
    c.nseq = nseq;
    c.num_pages = num_pages;
    c.page_size = page_size;
    c.max_pages = max_pages;
    c.Hkv = Hkv;
    c.passes_k = static_cast<int>(passes_q + passes_kv);
    c.positions_64 = positions_64;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool w32 = weight_fp32 != 0, il = interleaved != 0;
    const unsigned g = static_cast<unsigned>(blocks);
    cudaError_t e;
    if (D == 128)
        e = dtype == SDP_BF16 ? launch<128, true>(p, c, w32, il, g, st) : launch<128, false>(p, c, w32, il, g, st);
    else
        e = dtype == SDP_BF16 ? launch<256, true>(p, c, w32, il, g, st) : launch<256, false>(p, c, w32, il, g, st);
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}
