// Conversions of the 8-bit calls, and the launchers that apex4_gemm_e4m3
// chooses among.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layers.h"
#include "quant_rule.h"

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

struct Eight {
    float v[8];
};

template <bool BF16>
__device__ inline Eight load8(const uint16_t* p)
{
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Eight e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e.v[2 * i] = from16<BF16>((uint16_t)w[i]);
        e.v[2 * i + 1] = from16<BF16>((uint16_t)(w[i] >> 16));
    }
    return e;
}

__device__ inline float absmax(const Eight& e)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(e.v[i]));
    return m;
}

// The codes of 8 values: the correctly rounded fp32 quotient by the scale, kept
// within the largest E4M3 number (a scale that is a subnormal number may be
// rounded down so far that the quotient is above it), rounded to nearest even.
// A NaN, and an infinity by its infinite scale, stays a NaN (the comparison is
// false for it); in a block of zeros s is 0 and the value itself says which.
__device__ inline uint2 codes8(const Eight& e, float s)
{
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = s > 0.0f ? e.v[i] / s : e.v[i] + 0.0f;
        q[i] = fabsf(v) > 448.0f ? copysignf(448.0f, v) : v;
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// The scale of a block of 128 that 16 neighbouring lanes hold: max / 448.
__device__ inline float block_scale(const Eight& e)
{
    return qrule::group_max<16>(absmax(e)) / 448.0f;
}

}  // namespace e4m3

size_t e4m3_tiled_workspace_bytes(const E4m3Problem& p);
// At most 16 rows and 32 MB of weights, in one launch (launch_e4m3_rows, x null
// for operands that are quantized already).
bool e4m3_rows_supports(const E4m3Problem& p);
hipError_t launch_e4m3_tiled(const E4m3Problem& p, hipStream_t stream);

}  // namespace apex4
