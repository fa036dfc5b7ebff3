// What the kernels of the experts' W4A4 network share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layers.h"

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

// silu(g) u, kept within fp16
__device__ inline _Float16 experts_h(float g, float u)
{
    const float v = g / (1.0f + expf(-g)) * u;
    return (_Float16)fminf(fmaxf(v, -65504.0f), 65504.0f);
}

// A few tokens (experts_token.hip): the whole network in two launches; h: [R, I].
bool experts_token_supports(const ExpertsProblem& p);
hipError_t launch_experts_token(const ExpertsProblem& p, _Float16* h, hipStream_t stream);

// K parts of the down product
int experts_parts(int64_t R, int32_t E, int32_t H, int32_t I);

void launch_experts_tiled(const ExpertsProduct& a, bool up, int64_t R, hipStream_t stream);

}  // namespace apex4
