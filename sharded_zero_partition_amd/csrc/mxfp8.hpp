// mxfp8.hpp -- element types and the block scales of MXFP8 (device translation units only).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zero_partition.h"

namespace zp {

// Types behind the ABI's dtype numbers.
template <int D>
struct Type;
template <>
struct Type<ZERO_DTYPE_FP16> {
    typedef uint16_t elem;
    static __device__ __forceinline__ float wide(uint16_t x) { return float(__builtin_bit_cast(_Float16, x)); }
    static __device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, _Float16(x)); }
};
template <>
struct Type<ZERO_DTYPE_BF16> {
    typedef uint16_t elem;
    static __device__ __forceinline__ float wide(uint16_t x) { return __builtin_bit_cast(float, uint32_t(x) << 16); }
    static __device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, __bf16(x)); }
};
template <>
struct Type<ZERO_DTYPE_FP32> {
    typedef float elem;
    static __device__ __forceinline__ float wide(float x) { return x; }
};
template <>
struct Type<ZERO_DTYPE_MXFP8> {
    typedef uint8_t elem;
};

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float number(uint32_t x) { return __builtin_bit_cast(float, x); }

// The scale byte of a block whose largest magnitude has the bits `top`: the
// least s >= 1 with top 2^(127 - s) <= 448 = 1.75 2^8.  The exponent of top less
// 8, and one more when its fraction is above 1.75.
__device__ __forceinline__ int scale_of(uint32_t top) {
    const int e = int((top + 0x1FFFFFu) >> 23) - 8;
    return e > 1 ? e : 1;
}

// 2^(s - 127).  s = 0 is 2^-127, below the normal range.
__device__ __forceinline__ float scale_value(int s) {
    const uint32_t b = uint32_t(s) << 23;
    return number(b > 0x00400000u ? b : 0x00400000u);
}

// The multiplier into a block's range, 2^(127 - s), exact for any value but
// those that fall below fp32's normal range.
__device__ __forceinline__ float into_block(int s) { return number(uint32_t(254 - s) << 23); }

}  // namespace zp
