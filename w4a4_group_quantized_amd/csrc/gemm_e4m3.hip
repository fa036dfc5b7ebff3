// Linear layers in 8-bit floating point (OCP E4M3) with a scale for each
// block of 128, on gfx950: the quantizers and the product
//
//     y[m, n] = sum_j s_a[m, j] s_w[n / 128, j] sum_{k in block j} qa[m, k] qw[n, k]
//
// The block sums come from the FP8 matrix instruction (v_mfma_scale_f32_*_f8f6f4
// with unit block scales), the sum over blocks is one fp32 fma per output and
// block.  The instruction adds the products of 8 neighbouring k aligned to the
// largest of them and drops what lies below 2^-13 of it (measured: beside
// 2^16 a product of 2^3 stays and one of 2^2 is lost, in one run of 8 only);
// between those runs its sums are fp32.  That is the price of the FP8 rate: a
// run may be off by 7 * 2^-13 of its largest product.  Of the sum of |products|
// that was 1e-6 for normal values (64 x 144 x 4096) and 2.4e-4, half a rounding
// to fp16, where every run held one product of the largest codes beside small
// ones; where the products cancel it is that much of more than the result.
// Widening the codes for the fp16 instruction would halve the matrix rate.
#include "gemm_e4m3.h"
#include "layers.h"

namespace apex4 {
namespace {

using e4m3::Eight;
using e4m3::absmax;
using e4m3::block_scale;
using e4m3::codes8;
using e4m3::load8;

// Activations: a scale for 128 columns of a row, 16 lanes a block.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_e4m3_kernel(const uint16_t* __restrict__ x, int64_t n8,
                                                            uint2* __restrict__ q, float* __restrict__ s)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    Eight e = {};
    if (t < n8) e = load8<BF16>(x + t * 8);
    const float scale = block_scale(e);
    if (t < n8) {
        q[t] = codes8(e, scale);
        if ((t & 15) == 0) s[t / 16] = scale;
    }
}

// Weights: a scale for 128 x 128, one workgroup a block (the last block of
// rows may be short).
template <bool BF16>
__global__ __launch_bounds__(256) void pack_e4m3_kernel(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                        uint8_t* __restrict__ q, float* __restrict__ s)
{
    __shared__ float part[4];
    const int64_t kb = K / 128, nb = blockIdx.x / kb, j = blockIdx.x - nb * kb;
    const int c = (threadIdx.x & 15) * 8, r0 = threadIdx.x >> 4;
    Eight e[8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = nb * 128 + r0 + 16 * i;
        e[i] = Eight{};
        if (n < N) e[i] = load8<BF16>(w + n * K + j * 128 + c);
        m = fmaxf(m, absmax(e[i]));
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float scale = m / 448.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = nb * 128 + r0 + 16 * i;
        if (n < N) *reinterpret_cast<uint2*>(q + n * K + j * 128 + c) = codes8(e[i], scale);
    }
    if (threadIdx.x == 0) s[nb * kb + j] = scale;
}

}  // namespace

hipError_t launch_quantize_e4m3(const void* x, bool bf16, int64_t rows, int64_t K, void* q8, float* s,
                                hipStream_t stream)
{
    const int64_t n8 = rows * (K / 8);
    const unsigned blocks = (unsigned)((n8 + 255) / 256);
    const uint16_t* in = static_cast<const uint16_t*>(x);
    uint2* q = static_cast<uint2*>(q8);
    if (bf16) quantize_e4m3_kernel<true><<<blocks, 256, 0, stream>>>(in, n8, q, s);
    else quantize_e4m3_kernel<false><<<blocks, 256, 0, stream>>>(in, n8, q, s);
    return hipGetLastError();
}

hipError_t launch_pack_e4m3(const void* w, bool bf16, int64_t N, int64_t K, void* q8, float* s, hipStream_t stream)
{
    const unsigned blocks = (unsigned)((N + 127) / 128 * (K / 128));
    const uint16_t* in = static_cast<const uint16_t*>(w);
    uint8_t* q = static_cast<uint8_t*>(q8);
    if (bf16) pack_e4m3_kernel<true><<<blocks, 256, 0, stream>>>(in, N, K, q, s);
    else pack_e4m3_kernel<false><<<blocks, 256, 0, stream>>>(in, N, K, q, s);
    return hipGetLastError();
}

size_t e4m3_workspace_bytes(const E4m3Problem& p) { return e4m3_rows_supports(p) ? 0 : e4m3_tiled_workspace_bytes(p); }

hipError_t launch_gemm_e4m3(const E4m3Problem& p, hipStream_t stream)
{
    return e4m3_rows_supports(p) ? launch_e4m3_rows(p, nullptr, stream) : launch_e4m3_tiled(p, stream);
}

}  // namespace apex4
