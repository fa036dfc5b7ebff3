// Conversions of the 8-bit calls, and the launchers that apex4_gemm_e4m3
// chooses among.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"

namespace apex4 {
namespace e4m3 {

template <bool BF16>
__device__ inline float from16(uint16_t b)
{
    if (BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
    return (float)__builtin_bit_cast(_Float16, b);
}

// round to nearest, ties to even; bf16 by arithmetic on the bits (a NaN keeps a mantissa bit)
template <bool BF16>
__device__ inline uint16_t to16(float v)
{
    if (!BF16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    if (v != v) return (uint16_t)((b >> 16) | 0x40);
    return (uint16_t)((b + 0x7fff + ((b >> 16) & 1)) >> 16);
}

}  // namespace e4m3

size_t e4m3_tiled_workspace_bytes(const E4m3Problem& p);
hipError_t launch_e4m3_tiled(const E4m3Problem& p, hipStream_t stream);

}  // namespace apex4
