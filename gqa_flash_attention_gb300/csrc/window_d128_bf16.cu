// Instantiation of the sliding-window kernel: head dim 128, bf16 I/O.
#include "window_kernel.cuh"
#include "window_launch.h"

namespace sdp {

cudaError_t window_d128_bf16(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream)
{
    return launch_window<128, true>(m, p, stream);
}

}  // namespace sdp
