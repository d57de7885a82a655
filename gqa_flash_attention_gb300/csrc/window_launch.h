// Launchers of the sliding-window kernels, one translation unit per (head dim, dtype).
#pragma once

#include "sdp_launch.h"

namespace sdp {

struct WindowParams;

cudaError_t window_d128_fp16(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream);
cudaError_t window_d128_bf16(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream);
cudaError_t window_d256_fp16(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream);
cudaError_t window_d256_bf16(const LaunchMaps &m, const WindowParams &p, cudaStream_t stream);

}  // namespace sdp
