// Instantiation of the 4-bit cache attention: head dim 128, bf16 I/O.
#include "cache4_attn.cuh"

namespace sdp {

cudaError_t cache4_attn_d128_bf16(const Cache4AttnParams &p, bool wide, int sms, cudaStream_t st)
{
    return wide ? launch_cache4_attn<128, true, 2>(p, sms, st) : launch_cache4_attn<128, true, 1>(p, sms, st);
}

}  // namespace sdp
