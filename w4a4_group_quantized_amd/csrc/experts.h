// What the kernels of the experts' W4A4 network share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layers.h"
#include "quant_rule.h"

namespace apex4 {

// One of the network's two products, over the rows sorted by expert.
struct ExpertsProduct {
    const int32_t* offsets;   // [E + 1] first sorted row of every expert
    const int32_t* order;     // [R] slot of a sorted row; its token is slot / k
    const uint8_t* qx;        // gate and up: [rows, K/2] by token; down: by sorted row
    const float* sx;          // [., K/128]
    const uint8_t* qw;        // [E, N, K/2]
    const float* sw;          // [E, N, K/128]
    int64_t rows;             // tokens
    int32_t k, E, N, K;
    _Float16* h;              // gate and up: [R, N/2]
    float* d;                 // down: [parts, R, N]
    int32_t parts;            // K in this many parts (gate and up: 1)
    int64_t part_stride;      // R N
};

// The scale of a group of 128 values that 16 neighbouring lanes hold (the rule
// of apex4_quantize_act); not finite where one of them is not, which the codes
// cannot say.  The largest magnitude is taken as fp16 bits, which order NaN
// above infinity and that above the numbers (fmaxf drops a NaN).
template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v)
{
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
__device__ inline float experts_scale(const qrule::half8& v)
{
    typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
    const uint4 w = __builtin_bit_cast(uint4, v);
    auto two = [](uint32_t p) { return __builtin_bit_cast(ushort2v, p & 0x7FFF7FFFu); };
    const uint32_t both = __builtin_bit_cast(
        uint32_t, __builtin_elementwise_max(__builtin_elementwise_max(two(w.x), two(w.y)),
                                            __builtin_elementwise_max(two(w.z), two(w.w))));
    uint32_t m = max(both & 0xFFFF, both >> 16);
    m = dpp_max<0xB1>(m);             // quad swaps, half-row and row mirrors
    m = dpp_max<0x4E>(m);
    m = dpp_max<0x141>(m);
    m = dpp_max<0x140>(m);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)m) / 7.0f;
}

// silu(g) u, kept within fp16; NaN where g or u is infinite or NaN (the last sum is 0 for numbers)
__device__ inline _Float16 experts_h(float g, float u)
{
    const float v = g / (1.0f + expf(-g)) * u;
    return (_Float16)(fminf(fmaxf(v, -65504.0f), 65504.0f) + fmaf(0.0f, g, 0.0f * u));
}

// A few tokens (experts_token.hip): the whole network in two launches; h: [R, I].
bool experts_token_supports(const ExpertsProblem& p);
hipError_t launch_experts_token(const ExpertsProblem& p, _Float16* h, hipStream_t stream);

// K parts of the down product
int experts_parts(int64_t R, int32_t E, int32_t H, int32_t I);

void launch_experts_tiled(const ExpertsProduct& a, bool up, int64_t R, hipStream_t stream);

}  // namespace apex4
