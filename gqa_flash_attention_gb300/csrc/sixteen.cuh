// Conversions between packed 16-bit pairs and fp32, shared by the memory-bound kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace sdp {

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t u)
{
    if constexpr (BF16) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<__half2 *>(&u));
    }
}

// Rounded to nearest even; `lo` is the pair's first element.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if constexpr (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    } else {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
}

// Eight consecutive 16-bit elements.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<BF16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack16<BF16>(x[0], x[1]), pack16<BF16>(x[2], x[3]), pack16<BF16>(x[4], x[5]),
                      pack16<BF16>(x[6], x[7]));
}

// a * b on packed pairs of fp32, each rounded as a scalar product.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

}  // namespace sdp
