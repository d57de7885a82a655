// sdp_qk_norm_rope: checks, the launch shape and the dispatch of the kernel in qk_norm_rope.cuh without a cache.
#include "qk_norm_rope.cuh"
#include "sdp.h"

namespace {

using namespace sdp::rope;

template <int D, bool BF16, bool W32, bool POS64>
cudaError_t launch(const RopeParams &p, bool interleaved, unsigned blocks, cudaStream_t st)
{
    if (interleaved)
        qk_norm_rope_kernel<D, BF16, W32, POS64, true, false><<<blocks, 32 * kWarps, 0, st>>>(p, CacheDest{});
    else
        qk_norm_rope_kernel<D, BF16, W32, POS64, false, false><<<blocks, 32 * kWarps, 0, st>>>(p, CacheDest{});
    return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch(const RopeParams &p, bool w32, bool pos64, bool interleaved, unsigned blocks, cudaStream_t st)
{
    if (w32)
        return pos64 ? launch<D, BF16, true, true>(p, interleaved, blocks, st)
                     : launch<D, BF16, true, false>(p, interleaved, blocks, st);
    return pos64 ? launch<D, BF16, false, true>(p, interleaved, blocks, st)
                 : launch<D, BF16, false, false>(p, interleaved, blocks, st);
}

}  // namespace

extern "C" int sdp_qk_norm_rope(const void *q, long long q_sb, long long q_ss, long long q_sh, const void *k,
                                long long k_sb, long long k_ss, long long k_sh, void *q_out, long long qo_sb,
                                long long qo_ss, long long qo_sh, void *k_out, long long ko_sb, long long ko_ss,
                                long long ko_sh, const void *positions, long long p_sb, long long p_ss,
                                int positions_64, const unsigned long long *turns, int rot_dim, float mscale,
                                const void *q_weight, const void *k_weight, int weight_fp32, float eps,
                                int interleaved, int B, int S, int Hq, int Hkv, int D, int dtype, void *stream)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (B < 0 || S < 0 || Hq < 0 || Hkv < 0 || rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0)
        return SDP_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !(eps <= 3.0e38f) || !(mscale >= -3.0e38f && mscale <= 3.0e38f))
        return SDP_ERR_INVALID_ARG;
    if (B == 0 || S == 0 || Hq + static_cast<long long>(Hkv) == 0)
        return SDP_OK;
    if ((Hq > 0 && (q == nullptr || q_out == nullptr)) || (Hkv > 0 && (k == nullptr || k_out == nullptr)))
        return SDP_ERR_INVALID_ARG;
    if (rot_dim > 0 && (positions == nullptr || turns == nullptr))
        return SDP_ERR_INVALID_ARG;
    using sdp::is_aligned;
    const long long strides[12] = {q_sb, q_ss, q_sh, k_sb, k_ss, k_sh, qo_sb, qo_ss, qo_sh, ko_sb, ko_ss, ko_sh};
    for (long long s : strides)
        if (s % 8 != 0)
            return SDP_ERR_ALIGNMENT;
    if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(q_out, 16) || !is_aligned(k_out, 16) ||
        !is_aligned(q_weight, 16) || !is_aligned(k_weight, 16) || !is_aligned(turns, 8) ||
        !is_aligned(positions, positions_64 ? 8 : 4))
        return SDP_ERR_ALIGNMENT;
    const long long tokens = static_cast<long long>(B) * S;
    const long long heads = static_cast<long long>(Hq) + Hkv;
    if (tokens > INT32_MAX || heads > INT32_MAX)
        return SDP_ERR_OVERFLOW;
    int dev = 0, sms = 0;
    const int rc = sdp::current_device(&dev, &sms);
    if (rc != SDP_OK)
        return rc;

    RopeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = strides[i];
        p.ks[i] = strides[3 + i];
        p.qos[i] = strides[6 + i];
        p.kos[i] = strides[9 + i];
    }
    p.positions = positions;
    p.ps[0] = p_sb;
    p.ps[1] = p_ss;
    p.turns = turns;
    p.wq = q_weight;
    p.wk = k_weight;
    p.mscale = mscale;
    p.eps = eps;
    p.S = S;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.R = rot_dim;
    p.tokens = static_cast<int>(tokens);
    // Passes a warp: one while that leaves SMs without a full set of warps, then as many as share a
    // token's angles and factors.
    const int rpp = 256 / D;
    const long long passes_q = (Hq + static_cast<long long>(rpp) - 1) / rpp;
    const long long passes = passes_q + (Hkv + static_cast<long long>(rpp) - 1) / rpp;
    long long per = tokens * passes / (static_cast<long long>(sms) * 32);
    per = per < 1 ? 1 : (per > passes ? passes : per);
    p.passes_q = static_cast<int>(passes_q);
    p.passes = static_cast<int>(passes);
    p.per_warp = static_cast<int>(per);
    const long long runs = (passes + per - 1) / per;
    const long long blocks = (tokens * runs + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX)
        return SDP_ERR_OVERFLOW;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool w32 = weight_fp32 != 0, p64 = positions_64 != 0, il = interleaved != 0;
    const unsigned g = static_cast<unsigned>(blocks);
    cudaError_t e;
    if (D == 128)
        e = dtype == SDP_BF16 ? launch<128, true>(p, w32, p64, il, g, st) : launch<128, false>(p, w32, p64, il, g, st);
    else
        e = dtype == SDP_BF16 ? launch<256, true>(p, w32, p64, il, g, st) : launch<256, false>(p, w32, p64, il, g, st);
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}
