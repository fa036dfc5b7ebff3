// Launchers of the routing, expert and 8-bit calls (include/apex4.h), shared by
// their API file and their kernels.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "internal.h"

namespace apex4 {

// Compute units of the current device (0 where that cannot be asked).
int compute_units();

// Routing of tokens to experts (apex4_route, its argument names).
struct RouteProblem {
    const void* logits;
    int32_t type;
    int64_t M;
    int32_t E, k;
    bool sigmoid;
    const float* bias;
    int32_t n_group, keep, top;
    bool renormalize;
    float scale;
    int32_t* ids;
    float* gates;
};
hipError_t launch_route(const RouteProblem& p, hipStream_t stream);

// The experts' W4A4 network (apex4_experts_w4a4, its argument names; R = M k).
struct ExpertsProblem {
    const void* x;
    const int32_t* ids;
    const float* gates;
    int64_t M;
    int32_t k, E, H, I;
    const uint8_t* qw_gu;
    const float* s_gu;
    const uint8_t* qw_down;
    const float* s_down;
    void* y16;
    float* y32;
    void* ws;
};
size_t experts_workspace_bytes(int64_t M, int32_t k, int32_t E, int32_t H, int32_t I);
hipError_t launch_experts(const ExpertsProblem& p, hipStream_t stream);

// 8-bit floating point operands with a scale for each block of 128.
struct E4m3Problem {
    const uint8_t* qa;    // [M, K]
    const float* sa;      // [M, K/128]
    const uint8_t* qw;    // [N, K]
    const float* sw;      // [ceil(N/128), K/128]
    int32_t M, N, K;
    bool bf16;            // type of y: bf16, else fp16
    void* y;              // [M, N]
    float* y32;           // [M, N] or null
    void* ws;             // e4m3_workspace_bytes, or null
};
size_t e4m3_workspace_bytes(const E4m3Problem& p);
hipError_t launch_gemm_e4m3(const E4m3Problem& p, hipStream_t stream);
// the smallest calls, which quantize the rows x (of y's type) themselves
bool e4m3_rows_quantizes(const E4m3Problem& p);
hipError_t launch_e4m3_rows(const E4m3Problem& p, const void* x, hipStream_t stream);
hipError_t launch_quantize_e4m3(const void* x, bool bf16, int64_t rows, int64_t K, void* q8, float* s,
                                hipStream_t stream);
hipError_t launch_pack_e4m3(const void* w, bool bf16, int64_t N, int64_t K, void* q8, float* s, hipStream_t stream);

}  // namespace apex4
