// Instantiation of the 4-bit cache attention: head dim 128, fp16 I/O.
#include "cache4_attn.cuh"

namespace sdp {

cudaError_t cache4_attn_d128_fp16(const Cache4AttnParams &p, int sms, cudaStream_t st)
{
    const int columns = p.n * p.G;
    return columns <= 8 ? launch_cache4_attn<128, false, 1>(p, sms, st)
                        : launch_cache4_attn<128, false, 2>(p, sms, st);
}

}  // namespace sdp
