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

}  // namespace sdp
