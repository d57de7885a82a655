// Instantiation of the sliding-window kernel: head dim 256, fp16 I/O.
#include "window_kernel.cuh"
#include "window_launch.h"

namespace sdp {

cudaError_t window_d256_fp16(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream)
{
    return launch_window<256, false>(m, p, stream);
}

}  // namespace sdp
