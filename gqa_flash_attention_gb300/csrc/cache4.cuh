// The paged cache held in 4 bits: layout and helpers shared by its kernels.
//
// A pool of num_pages pages, each holding page_size tokens of every KV head:
//
//     k_codes, v_codes    uint8 [num_pages, Hkv, page_size, D / 2]: channel 2i in the low and
//                         2i + 1 in the high half of byte i
//     k_scales, v_scales  bf16 [num_pages, Hkv, page_size, D / 64, 2]: scale s and bias b of 64 channels
//
// and code n stands for s * n + b: 4.5 bits a channel. bf16 holds any fp16 or bf16 range; b's
// rounding costs 2^-9 of the group's minimum, s's at most 15 * 2^-9 of a step.
//
// Token t of sequence i is at place t % page_size of page block_table[i][t / page_size].
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sdp_internal.h"

namespace sdp {

constexpr int kCacheGroup = 64;

struct Cache4View {
    uint8_t *k_codes, *v_codes;
    uint32_t *k_scales, *v_scales;  // (scale, bias) pairs: scale in the low half
    const int *table;
    long long table_stride;
    int num_pages, page_size, max_pages, Hkv;
};

// Index s with cu[s] <= t < cu[s + 1] of non-decreasing offsets cu[0..n], found by all 32 lanes
// together, 32 candidates a step (two trips to memory for up to 1024 sequences, where a binary
// search makes ten); n when t lies outside. t is the same in every lane.
__device__ __forceinline__ int find_sequence(const int *cu, int n, int t, int lane)
{
    int lo = 0, len = n;  // the answer lies in [lo, lo + len)
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int i = lo + lane * step;
        // sequences that begin at or before t form a prefix of the candidates
        const bool before = lane * step < len && __ldg(cu + i) <= t;
        const unsigned m = __ballot_sync(0xffffffffu, before);
        if (m == 0u)
            return n;
        const int used = (31 - __clz(m)) * step;
        lo += used;
        len = min(step, len - used);
        if (step == 1)
            break;
    }
    return lo < n && __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : n;
}

}  // namespace sdp
