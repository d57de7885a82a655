// Entry points of the sliding-window attention (window_kernel.cuh): checks, tensor maps and the
// launch shape.
#include <algorithm>
#include <cmath>

#include "sdp.h"
#include "sdp_internal.h"
#include "window_kernel.cuh"
#include "window_launch.h"

namespace {

constexpr int kDebugNoPack = 4;
constexpr int kDebugFullVarlenGrid = 32;

int common_checks(const void *q, const void *k, const void *v, const void *o, const float *lse, int D, float scale,
                  int window, int sinks)
{
    if (q == nullptr || k == nullptr || v == nullptr || o == nullptr)
        return SDP_ERR_INVALID_ARG;
    if (window <= 0 || sinks < 0 || !std::isfinite(scale) || o == q || o == k || o == v)
        return SDP_ERR_INVALID_ARG;
    using sdp::is_aligned;
    if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(o, 16) || !is_aligned(lse, 4))
        return SDP_ERR_ALIGNMENT;
    return SDP_OK;
}

// Device, status word and what every launch carries.
int fill(sdp::WindowParams &p, const void *q, const void *k, const void *v, void *o, float *lse, float scale, int window,
         int sinks)
{
    int dev = 0;
    int rc = sdp::current_device(&dev, &p.k.num_sms);
    if (rc != SDP_OK)
        return rc;
    if ((rc = sdp::status_word(dev, &p.k.status)) != SDP_OK)
        return rc;
    p.q = q;
    p.kk = k;
    p.v = v;
    p.k.o = o;
    p.k.lse = lse;
    p.k.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // scale * log2(e)
    p.k.timeout_ns = sdp::wait_timeout_ns();
    p.k.debug_flags = sdp::debug_flags();
    p.k.kv_splits = 1;
    // positions lie within 2^30 of 0, so larger values say the same, and sums with them stay in 32 bits
    p.window = std::min(window, 1 << 30);
    p.sinks = std::min(sinks, 1 << 30);
    return SDP_OK;
}

int run(const sdp::LaunchMaps &m, const sdp::WindowParams &p, int D, int dtype, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (D == 128)
        e = dtype == SDP_BF16 ? sdp::window_d128_bf16(m, p, st) : sdp::window_d128_fp16(m, p, st);
    else
        e = dtype == SDP_BF16 ? sdp::window_d256_bf16(m, p, st) : sdp::window_d256_fp16(m, p, st);
    return e == cudaSuccess ? SDP_OK : sdp::record_cuda_error(e);
}

}  // namespace

extern "C" int sdp_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv,
                              int Sq, int Skv, int D, float scale, int dtype, int window, int sinks, void *stream)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Skv <= 0 || Hq % Hkv != 0)
        return SDP_ERR_INVALID_ARG;
    int rc = common_checks(q, k, v, o, lse, D, scale, window, sinks);
    if (rc != SDP_OK)
        return rc;
    // Few rows (decoding, drafted tokens): a group's query heads as one head of G * Sq rows, the same
    // memory, so that they share a tile and its K/V loads.
    const int G = Hq / Hkv;
    const bool pack = G > 1 && Sq < 128 && static_cast<long long>(G) * Sq <= INT32_MAX &&
                      !(sdp::debug_flags() & kDebugNoPack);
    const int rows = pack ? G * Sq : Sq, heads = pack ? Hkv : Hq;
    const long long n_qtiles = (static_cast<long long>(rows) + 127) / 128;
    const long long planes_q = static_cast<long long>(B) * heads, planes_kv = static_cast<long long>(B) * Hkv;
    if (Sq >= 1 << 30 || Skv >= 1 << 30 || planes_q > INT32_MAX || planes_kv > INT32_MAX ||
        planes_q > INT32_MAX / n_qtiles)
        return SDP_ERR_OVERFLOW;
    sdp::WindowParams p{};
    if ((rc = fill(p, q, k, v, o, lse, scale, window, sinks)) != SDP_OK)
        return rc;
    sdp::LaunchMaps m;
    if ((rc = sdp::tensor_map(&m.q, q, dtype, D, rows, planes_q, 128)) != SDP_OK ||
        (rc = sdp::tensor_map(&m.k, k, dtype, D, Skv, planes_kv, 128)) != SDP_OK ||
        (rc = sdp::tensor_map(&m.k_half, k, dtype, D, Skv, planes_kv, 64)) != SDP_OK ||
        (rc = sdp::tensor_map(&m.v, v, dtype, D, Skv, planes_kv, 128)) != SDP_OK)
        return rc;
    p.k.Hq = heads;
    p.k.Hkv = Hkv;
    p.k.G = pack ? 1 : G;
    p.k.Sq = rows;
    p.k.Skv = Skv;
    p.k.n_qtiles = static_cast<int>(n_qtiles);
    p.k.units = static_cast<int>(planes_q * n_qtiles);
    p.q_plane = static_cast<long long>(rows) * D;
    p.q_row = D;
    p.kv_plane = static_cast<long long>(Skv) * D;
    p.kv_row = D;
    p.pack_sq = pack ? Sq : 0;
    return run(m, p, D, dtype, stream);
}

extern "C" int sdp_fwd_varlen_window(const void *q, const void *k, const void *v, void *o, float *lse,
                                     const int *cu_seqlens_q, const int *cu_seqlens_k, int nseq, int Hq, int Hkv,
                                     int total_q, int total_k, int max_seqlen_q, int D, float scale, int dtype,
                                     int window, int sinks, void *stream)
{
    if (dtype != SDP_FP16 && dtype != SDP_BF16)
        return SDP_ERR_UNSUPPORTED;
    if (D != 128 && D != 256)
        return SDP_ERR_UNSUPPORTED;
    if (nseq <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0)
        return SDP_ERR_INVALID_ARG;
    if (total_q == 0)
        return SDP_OK;  // no query rows (empty tensors may have null pointers): nothing to compute
    if (cu_seqlens_q == nullptr || cu_seqlens_k == nullptr || max_seqlen_q == 0)
        return SDP_ERR_INVALID_ARG;
    // A batch without a single key (empty tensors may have null pointers): its rows get O = 0 and LSE = -inf, and
    // the maps of K and V, from which nothing is loaded, are made over q.
    if (total_k == 0)
        k = v = q;
    int rc = common_checks(q, k, v, o, lse, D, scale, window, sinks);
    if (rc != SDP_OK)
        return rc;
    if (!sdp::is_aligned(cu_seqlens_q, 4) || !sdp::is_aligned(cu_seqlens_k, 4))
        return SDP_ERR_ALIGNMENT;
    const long long n_qtiles = (static_cast<long long>(max_seqlen_q) + 127) / 128;
    const long long units = static_cast<long long>(nseq) * Hq;
    if (total_q >= 1 << 30 || total_k >= 1 << 30 || max_seqlen_q >= 1 << 30 || units > INT32_MAX / n_qtiles)
        return SDP_ERR_OVERFLOW;
    sdp::WindowParams p{};
    if ((rc = fill(p, q, k, v, o, lse, scale, window, sinks)) != SDP_OK)
        return rc;
    const long long kv_rows = total_k > 0 ? total_k : 1;
    sdp::LaunchMaps m;
    if ((rc = sdp::tensor_map_thd(&m.q, q, dtype, D, total_q, Hq, 128)) != SDP_OK ||
        (rc = sdp::tensor_map_thd(&m.k, k, dtype, D, kv_rows, Hkv, 128)) != SDP_OK ||
        (rc = sdp::tensor_map_thd(&m.k_half, k, dtype, D, kv_rows, Hkv, 64)) != SDP_OK ||
        (rc = sdp::tensor_map_thd(&m.v, v, dtype, D, kv_rows, Hkv, 128)) != SDP_OK)
        return rc;
    p.k.Hq = Hq;
    p.k.Hkv = Hkv;
    p.k.G = Hq / Hkv;
    p.k.Sq = total_q;
    p.k.Skv = total_k;
    p.k.n_qtiles = static_cast<int>(n_qtiles);
    p.k.cu_q = cu_seqlens_q;
    p.k.cu_k = cu_seqlens_k;
    p.k.nseq = nseq;
    const long long slots = std::min(static_cast<long long>(nseq) * n_qtiles,
                                     (static_cast<long long>(total_q) + 127LL * nseq) / 128);
    const bool compact = !(p.k.debug_flags & kDebugFullVarlenGrid);
    p.k.n_tiles = compact ? static_cast<int>(slots) : 0;
    p.k.units = static_cast<int>(compact ? slots * Hq : units * n_qtiles);
    p.q_plane = D;
    p.q_row = static_cast<long long>(Hq) * D;
    p.kv_plane = D;
    p.kv_row = static_cast<long long>(Hkv) * D;
    return run(m, p, D, dtype, stream);
}
