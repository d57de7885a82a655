// Instantiation of the 16-bit cache attention: head dim 256, bf16 I/O.
#include "cache16_attn.cuh"

namespace sdp {

cudaError_t cache16_attn_d256_bf16(const Cache16Maps &m, const Cache16AttnParams &p, int sms, cudaStream_t st)
{
    return launch_cache16_attn<256, true>(m, p, sms, st);
}

}  // namespace sdp
