// Internal services of sdp_api.cu for the other entry points of libsdp.so. Not part of
// the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sdp {

// Codes that kernels put in the low byte of a device's status word for faults of their inputs
// (a wait that ran out puts its site there, 1..6).
constexpr unsigned kBadSeqlens = 7;
constexpr unsigned kBadPages = 8;

// Records `e` for sdp_last_cuda_error() and returns SDP_ERR_CUDA.
int record_cuda_error(cudaError_t e);

// The current device's index and SM count; SDP_ERR_UNSUPPORTED off sm_103.
int current_device(int *dev, int *sms);

// The status word of `dev` that sdp_poll_status() reads, allocated and zeroed on first use
// (synchronously: outside stream capture).
int status_word(int dev, unsigned int **status);

// Upper bound of any wait inside a kernel, and the test hooks, of launches made now.
unsigned long long wait_timeout_ns();
int debug_flags();

// Cached 3-D tensor maps over 16-bit tensors (64 columns x box_rows rows x 1 plane, 128-byte
// swizzle): [planes, rows, D] contiguous, and (token, head, dim) with plane = head.
int tensor_map(CUtensorMap *map, const void *base, int dtype, int D, long long rows, long long planes,
               unsigned box_rows);
int tensor_map_thd(CUtensorMap *map, const void *base, int dtype, int D, long long rows, long long heads,
                   unsigned box_rows);

inline bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace sdp
