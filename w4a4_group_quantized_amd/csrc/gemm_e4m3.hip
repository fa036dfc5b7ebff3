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
// between those runs its sums are fp32.  That is the price of the FP8 rate:
// about 2e-5 of the sum of |products|, a tenth of the rounding of the output to
// fp16 and less of bf16's; widening the codes for the fp16 instruction would
// halve the matrix rate.
#include "gemm_e4m3.h"
#include "internal.h"
#include "rows_stream.h"

namespace apex4 {
namespace {

using e4m3::from16;
using e4m3::to16;

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
__device__ inline uint2 codes8(const Eight& e, float s)
{
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s > 0.0f ? fminf(fmaxf(e.v[i] / s, -448.0f), 448.0f) : 0.0f;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Activations: a scale for 128 columns of a row, 16 lanes a block.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_e4m3_kernel(const uint16_t* __restrict__ x, int64_t n8,
                                                            uint2* __restrict__ q, float* __restrict__ s)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    Eight e = {};
    if (t < n8) e = load8<BF16>(x + t * 8);
    float m = absmax(e);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float scale = m / 448.0f;
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

// Few rows: 16 weight rows a workgroup, passes of up to 64 activation rows.
template <bool BF16>
__global__ __launch_bounds__(rows::THREADS) void e4m3_rows_kernel(E4m3Problem a)
{
    using namespace rows;
    __shared__ Shared<true> sh;
    const int n0 = blockIdx.x * ROWS;
    const int64_t K = a.K, G = K / 128;
    auto wrow = [&](int r) { return n0 + r < a.N ? a.qw + (n0 + r) * K : nullptr; };
    auto swrow = [&](int r) { return n0 + r < a.N ? a.sw + (n0 + r) / 128 * G : nullptr; };
    const int lane = threadIdx.x & 63;
    uint16_t* y = static_cast<uint16_t*>(a.y);
    auto pass = [&](auto tc, int m0) {
        constexpr int TILES = decltype(tc)::value;
        const uint8_t* xrow[TILES];
        const float* sarow[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const int64_t m = m0 + 16 * i + (lane & 15);
            xrow[i] = m < a.M ? a.qa + m * K : nullptr;
            sarow[i] = m < a.M ? a.sa + m * G : nullptr;
        }
        stream<true, TILES>(sh, a.K, wrow, swrow, xrow, sarow);
        for (int j = threadIdx.x; j < TILES * 256; j += THREADS) {
            const int t = j >> 8, m = m0 + 16 * t + ((j >> 4) & 15), c = j & 15;
            if (m < a.M && n0 + c < a.N) {
                float v = sh.red[0][t][(16 * (c >> 2) + ((j >> 4) & 15)) * 4 + (c & 3)];
                asm volatile("" : "+v"(v));   // y is the rounding of y32
                y[(int64_t)m * a.N + n0 + c] = to16<BF16>(v);
                if (a.y32) a.y32[(int64_t)m * a.N + n0 + c] = v;
            }
        }
        __syncthreads();   // sh.red is written again
    };
    for (int m0 = 0; m0 < a.M; m0 += 64) {
        if (a.M - m0 <= 16) pass(std::integral_constant<int, 1>{}, m0);
        else if (a.M - m0 <= 32) pass(std::integral_constant<int, 2>{}, m0);
        else pass(std::integral_constant<int, 4>{}, m0);
    }
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

// Up to 16 rows and 32 MB of weights: one launch without partial sums (16 x 4096
// x 4096: 11.6 us a call, 14.3 in tiles with a reduction; 16 x 28672 x 8192: 64
// us, 39 in tiles).
static bool few_rows(const E4m3Problem& p) { return p.M <= 16 && (int64_t)p.N * p.K <= (1 << 25); }

size_t e4m3_workspace_bytes(const E4m3Problem& p) { return few_rows(p) ? 0 : e4m3_tiled_workspace_bytes(p); }

hipError_t launch_gemm_e4m3(const E4m3Problem& p, hipStream_t stream)
{
    if (!few_rows(p)) return launch_e4m3_tiled(p, stream);
    const unsigned blocks = (unsigned)((p.N + rows::ROWS - 1) / rows::ROWS);
    if (p.bf16) e4m3_rows_kernel<true><<<blocks, rows::THREADS, 0, stream>>>(p);
    else e4m3_rows_kernel<false><<<blocks, rows::THREADS, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace apex4
