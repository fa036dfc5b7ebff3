// The 8-bit block-scaled product for up to 16 activation rows and at most 32 MB
// of weights on gfx950: one launch, which quantizes the rows itself where
// they are few.
//
//     D[n, m] = sum_j s_w s_a[m, j] sum_{k in block j} w[n, k] x[m, k]
//
// Such a call takes a few microseconds, of which launches are the most: the
// three of quantizing, tiles with a K split and their sum took 15 us for one
// row of 4096 x 4096, 3 us of which is reading the weights.
//
// A workgroup of 4 waves owns 16 weight rows and walks K in items of 512 bytes
// a row.  The 8 KB of an item come in with 16-byte loads that cover 512
// consecutive bytes of a row, four items ahead (32 KB in flight a workgroup),
// go through LDS once to change lanes (piece c of a row at c ^ row, so that the
// reads of 16 rows at one column touch every bank once), and each wave
// multiplies its block of 128 of the item.  The weights are the A operand, so a
// lane holds one activation row m = lane & 15 and four weight rows: s_a is one
// value per lane and block.  The four waves' sums meet in LDS, in wave order.
#include "gemm_e4m3.h"
#include "layers.h"

namespace apex4 {
namespace {

using e4m3::Eight;
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int ROWS = 16;         // weight rows per workgroup, activation rows at most
constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int ITEM = 512;        // bytes per row and item
constexpr int GPI = ITEM / 128;  // blocks per item: one per wave
constexpr int AHEAD = 4;         // items in flight
constexpr int PAD = 16;          // bytes between quantized rows: their reads fall on different banks
static_assert(GPI == WAVES && AHEAD % 2 == 0, "one block per wave, two buffers");

struct RowsArgs {
    E4m3Problem p;
    const void* x;               // QUANT: [M, K] fp16 or bf16
};

__host__ __device__ inline int quant_lds(const E4m3Problem& p) { return p.M * (p.K + PAD) + p.M * (p.K / 128) * 4; }

// NX > 0: quantizes x, NX chunks of 8 values a thread; 0: reads p.qa, p.sa
template <bool BF16, int NX>
__global__ __launch_bounds__(THREADS) void e4m3_rows_kernel(RowsArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t sw_w[2][ROWS * ITEM];
    __shared__ float sw_s[2][GPI][ROWS];
    __shared__ float red[WAVES][64 * 4];
    extern __shared__ __attribute__((aligned(16))) uint8_t xq[];
    const E4m3Problem& p = a.p;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * ROWS, M = p.M, K = p.K, G = K / 128;
    const int items = (K + ITEM - 1) / ITEM;

    // the rows to quantize are asked for first: what is asked for after them
    // stays in flight while their codes are made
    const int n8 = M * (K / 8);
    Eight xv[NX ? NX : 1];
#pragma unroll
    for (int j = 0; j < NX; ++j)
        xv[j] = e4m3::load8<BF16>(static_cast<const uint16_t*>(a.x) + 8 * (int64_t)min(tid + j * THREADS, n8 - 1));

    // this thread's two pieces of an item, rows tid / 32 and 8 + tid / 32, and
    // for the first threads one scale
    const int crow = tid >> 5, piece = tid & 31;
    const uint8_t* const w0 = n0 + crow < p.N ? p.qw + (int64_t)(n0 + crow) * K : nullptr;
    const uint8_t* const w1 = n0 + crow + 8 < p.N ? p.qw + (int64_t)(n0 + crow + 8) * K : nullptr;
    const int srow = tid / GPI, sg = tid % GPI;
    const float* const sp =
        tid < ROWS * GPI && n0 + srow < p.N ? p.sw + (int64_t)((n0 + srow) / 128) * G : nullptr;
    uint4 rw[AHEAD][2];
    float rs[AHEAD];
    auto load = [&](int t, int slot) {
        const int pos = t * ITEM + piece * 16;
        const bool in = pos < K;
        rw[slot][0] = in && w0 ? *reinterpret_cast<const uint4*>(w0 + pos) : make_uint4(0, 0, 0, 0);
        rw[slot][1] = in && w1 ? *reinterpret_cast<const uint4*>(w1 + pos) : make_uint4(0, 0, 0, 0);
        rs[slot] = sp && t * GPI + sg < G ? sp[t * GPI + sg] : 0.0f;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(i, i);

    const int stride = K + PAD;
    float* xs = reinterpret_cast<float*>(xq + M * stride);
    if constexpr (NX > 0) {
#pragma unroll
        for (int j = 0; j < NX; ++j) {
            const int i = tid + j * THREADS;
            if (i >= n8) break;
            const float scale = e4m3::block_scale(xv[j]);
            const int m = i / (K / 8), c = i - m * (K / 8);
            *reinterpret_cast<uint2*>(xq + m * stride + 8 * c) = e4m3::codes8(xv[j], scale);
            if ((c & 15) == 0) xs[m * G + (c >> 4)] = scale;
        }
        __syncthreads();
    }

    const int m = lane & 15, kg = lane >> 4;
    v4f acc = {};
    for (int t0 = 0; t0 < items; t0 += AHEAD)
#pragma unroll
        for (int h = 0; h < AHEAD; ++h) {
            const int t = t0 + h;
            if (t >= items) break;
            const int b = h & 1;
            *reinterpret_cast<uint4*>(sw_w[b] + crow * ITEM + (piece ^ crow) * 16) = rw[h][0];
            *reinterpret_cast<uint4*>(sw_w[b] + (crow + 8) * ITEM + (piece ^ (crow + 8)) * 16) = rw[h][1];
            if (tid < ROWS * GPI) sw_s[b][sg][srow] = rs[h];
            load(t + AHEAD, h);                          // (past K: zeros, nothing is read)
            const int g = t * GPI + wave, pos = g * 128 + 16 * kg;
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            float sa = 0.0f;
            if (m < M && g < G) {
                if constexpr (NX > 0) {
                    x0 = *reinterpret_cast<const uint4*>(xq + m * stride + pos);
                    x1 = *reinterpret_cast<const uint4*>(xq + m * stride + pos + 64);
                    sa = xs[m * G + g];
                } else {
                    x0 = *reinterpret_cast<const uint4*>(p.qa + (int64_t)m * K + pos);
                    x1 = *reinterpret_cast<const uint4*>(p.qa + (int64_t)m * K + pos + 64);
                    sa = p.sa[(int64_t)m * G + g];
                }
            }
            __syncthreads();
            // buffer b is written again two items on, after the next barrier
            const uint8_t* f = sw_w[b] + m * ITEM;       // (weight row lane & 15)
            const uint4 f0 = *reinterpret_cast<const uint4*>(f + ((8 * wave + kg) ^ m) * 16);
            const uint4 f1 = *reinterpret_cast<const uint4*>(f + ((8 * wave + kg + 4) ^ m) * 16);
            const v4f sw = *reinterpret_cast<const v4f*>(&sw_s[b][wave][4 * kg]);
            auto join = [](uint4 u, uint4 v) {
                return v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
            };
            const v4f P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(f0, f1), join(x0, x1), v4f{}, 0, 0, 0,
                                                                           127, 0, 127);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = fmaf(sw[r] * sa, P[r], acc[r]);
        }

    *reinterpret_cast<v4f*>(&red[wave][lane * 4]) = acc;
    __syncthreads();
    // weight row c of activation row r: lane 16 (c >> 2) + r, element c & 3
    const int r = tid >> 4, c = tid & 15;
    if (r < M && n0 + c < p.N) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += red[w][(16 * (c >> 2) + r) * 4 + (c & 3)];
        asm volatile("" : "+v"(v));   // y is the rounding of y32
        const int64_t o = (int64_t)r * p.N + n0 + c;
        static_cast<uint16_t*>(p.y)[o] = e4m3::to16<BF16>(v);
        if (p.y32) p.y32[o] = v;
    }
}

template <int NX>
hipError_t launch(const RowsArgs& a, hipStream_t stream)
{
    const unsigned blocks = (unsigned)((a.p.N + ROWS - 1) / ROWS);
    const int lds = NX ? quant_lds(a.p) : 0;
    if (a.p.bf16) e4m3_rows_kernel<true, NX><<<blocks, THREADS, lds, stream>>>(a);
    else e4m3_rows_kernel<false, NX><<<blocks, THREADS, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

// One launch without partial sums against tiles with a reduction: 16 x 4096 x
// 4096 11.6 us a call and 14.3, 16 x 28672 x 8192 64 us and 39.  Just past the
// end, 45 MB, weights from memory: 16 x 4096 x 11008 23.2 us and 20.6, 16 x
// 11008 x 4096 19.7 and 18.8; one row 21.1 and 19.6, and 14.5 and 17.4, so that
// one row could go further where K is short (1 x 14336 x 8192 24.5 and 30.1).
bool e4m3_rows_supports(const E4m3Problem& p) { return p.M <= ROWS && (int64_t)p.N * p.K <= (1 << 25); }

// Every workgroup makes the codes of all rows: up to 64 values a thread.
bool e4m3_rows_quantizes(const E4m3Problem& p)
{
    return e4m3_rows_supports(p) && (int64_t)p.M * p.K <= 8 * 8 * THREADS;
}

hipError_t launch_e4m3_rows(const E4m3Problem& p, const void* x, hipStream_t stream)
{
    const RowsArgs a{p, x};
    if (!x) return launch<0>(a, stream);
    return (int64_t)p.M * p.K <= 2 * 8 * THREADS ? launch<2>(a, stream) : launch<8>(a, stream);
}

}  // namespace apex4
