// Weight rows streamed past a few activation rows on gfx950: the product of
// the decode-sized calls of the experts' W4A4 network and of the 8-bit
// block-scaled linear layer.  Device code shared by experts.hip and
// gemm_e4m3.hip.
//
//     D[n, m] = sum_j s_w s_a[m, j] sum_{k in group j} w[n, k] x[m, k]
//
// A workgroup of 4 waves owns 16 weight rows and walks K in items of 512
// bytes a row (1024 INT4 codes or 512 FP8 ones).  The 8 KB of an item come in
// with 16-byte loads that cover 512 consecutive bytes of a row, four items
// ahead (32 KB in flight a workgroup, several workgroups a CU), go through
// LDS once to change lanes, and each wave multiplies its quarter of the
// item's K: two groups of 128 INT4 codes (int8 MFMA on the widened nibbles)
// or one group of FP8 codes.  The MFMA takes the weights as its A operand, so
// a lane holds ONE activation row m = lane & 15 and four consecutive weight
// rows: s_a is one value per lane and group.  The four waves' sums meet in
// LDS, in wave order.
//
// LDS rows are 528 bytes: 16 rows at one column lie 16 bytes apart modulo the
// banks, so the fragment reads have no conflicts.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace apex4 {
namespace rows {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int ROWS = 16;         // weight rows per workgroup
constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int ITEM = 512;        // bytes per row and item
constexpr int STRIDE = ITEM + 16;
constexpr int AHEAD = 4;         // items in flight
constexpr int MAX_TILES = 4;     // tiles of 16 activation rows per pass

template <bool F8>
struct Shared {
    static constexpr int GPI = F8 ? ITEM / 128 : ITEM / 64;   // groups per item
    uint8_t w[2][ROWS * STRIDE];
    float sw[2][GPI][ROWS];      // (FP8: one scale per 128 weight rows, kept per row all the same)
    float red[WAVES][MAX_TILES][64 * 4];
};

__device__ inline v4i widen_lo(uint4 w)
{
    return v4i{(int)((w.x << 4) & 0xF0F0F0F0u), (int)(w.x & 0xF0F0F0F0u), (int)((w.y << 4) & 0xF0F0F0F0u),
               (int)(w.y & 0xF0F0F0F0u)};
}
__device__ inline v4i widen_hi(uint4 w)
{
    return v4i{(int)((w.z << 4) & 0xF0F0F0F0u), (int)(w.z & 0xF0F0F0F0u), (int)((w.w << 4) & 0xF0F0F0F0u),
               (int)(w.w & 0xF0F0F0F0u)};
}

__device__ inline v8i join(uint4 a, uint4 b)
{
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// One pass over K.  `wrow(r)`: the address of weight row r (0..15) of the
// workgroup, or null for none (zeros).  `swrow(r)`: its K/128 scales (rows of
// one FP8 block share theirs).  xrow[t], sarow[t]: this lane's activation row
// lane & 15 of tile t and its scales, null for none.  After it, sh.red holds
// the finished sums: red[0][t][lane * 4 + r] is D of weight row 4 (lane >> 4)
// + r and activation row 16 t + (lane & 15).
template <bool F8, int TILES, typename WRow, typename SRow>
__device__ inline void stream(Shared<F8>& sh, int K, WRow wrow, SRow swrow, const uint8_t* const (&xrow)[TILES],
                              const float* const (&sarow)[TILES])
{
    constexpr int GPI = Shared<F8>::GPI;
    constexpr int GPW = GPI / WAVES;                    // groups per wave and item
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rowbytes = F8 ? K : K / 2;
    const int G = K / 128;
    const int items = (rowbytes + ITEM - 1) / ITEM;

    // this thread's two chunks of an item: rows tid / 32 and 8 + tid / 32
    const int crow = tid >> 5, ccol = (tid & 31) * 16;
    const uint8_t* const w0 = wrow(crow);
    const uint8_t* const w1 = wrow(crow + 8);
    // and, for the first threads, one scale of an item
    const int srow = tid / GPI, sg = tid % GPI;
    const float* const sp = tid < ROWS * GPI ? swrow(srow) : nullptr;

    uint4 rw[AHEAD][2];
    float rs[AHEAD];
    auto load = [&](int t, int slot) {
        const int pos = t * ITEM + ccol;
        const bool in = pos < rowbytes;
        rw[slot][0] = in && w0 ? *reinterpret_cast<const uint4*>(w0 + pos) : make_uint4(0, 0, 0, 0);
        rw[slot][1] = in && w1 ? *reinterpret_cast<const uint4*>(w1 + pos) : make_uint4(0, 0, 0, 0);
        const int g = t * GPI + sg;
        rs[slot] = sp && g < G ? sp[g] : 0.0f;
    };
    // this wave's part of an item of the activation rows: 128 bytes a row
    const int fkb = lane >> 4;
    uint4 xa[TILES][2];
    float sa[TILES][GPW];
    auto load_x = [&](int t) {
        const int pos = t * ITEM + 128 * wave + 16 * fkb;
        const int g = t * GPI + GPW * wave;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const bool in = pos < rowbytes && xrow[i];
            xa[i][0] = in ? *reinterpret_cast<const uint4*>(xrow[i] + pos) : make_uint4(0, 0, 0, 0);
            xa[i][1] = in && pos + 64 < rowbytes ? *reinterpret_cast<const uint4*>(xrow[i] + pos + 64)
                                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < GPW; ++q) sa[i][q] = g + q < G && sarow[i] ? sarow[i][g + q] : 0.0f;
        }
    };

    v4f acc[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(i, i);

    for (int t0 = 0; t0 < items; t0 += AHEAD)
#pragma unroll
        for (int h = 0; h < AHEAD; ++h) {
            const int t = t0 + h;
            if (t >= items) break;
            const int b = h & 1;                        // (AHEAD is even)
            *reinterpret_cast<uint4*>(sh.w[b] + crow * STRIDE + ccol) = rw[h][0];
            *reinterpret_cast<uint4*>(sh.w[b] + (crow + 8) * STRIDE + ccol) = rw[h][1];
            if (tid < ROWS * GPI) sh.sw[b][sg][srow] = rs[h];
            load(t + AHEAD, h);                         // (past K: zeros, nothing is read)
            load_x(t);
            __syncthreads();
            // buffer b is written again two items on, after the next barrier
            const uint8_t* f = sh.w[b] + (lane & 15) * STRIDE + 128 * wave + 16 * fkb;
            const uint4 f0 = *reinterpret_cast<const uint4*>(f);
            const uint4 f1 = *reinterpret_cast<const uint4*>(f + 64);
            v4f sw[GPW];
#pragma unroll
            for (int q = 0; q < GPW; ++q) sw[q] = *reinterpret_cast<const v4f*>(&sh.sw[b][GPW * wave + q][4 * fkb]);
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                if constexpr (F8) {
                    const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        join(f0, f1), join(xa[i][0], xa[i][1]), v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 127, 0, 127);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(sw[0][r] * sa[i][0], p[r], acc[i][r]);
                } else {
                    v4i p[2];
                    p[0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(widen_lo(f0), widen_lo(xa[i][0]), v4i{}, 0, 0, 0);
                    p[1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(widen_lo(f1), widen_lo(xa[i][1]), v4i{}, 0, 0, 0);
                    p[0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(widen_hi(f0), widen_hi(xa[i][0]), p[0], 0, 0, 0);
                    p[1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(widen_hi(f1), widen_hi(xa[i][1]), p[1], 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < GPW; ++q)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][r] = fmaf(sw[q][r] * sa[i][q], (float)p[q][r], acc[i][r]);
                }
            }
        }

    // the waves' sums, added in wave order (INT4: with the 2^-8 of the widened codes)
#pragma unroll
    for (int i = 0; i < TILES; ++i) *reinterpret_cast<v4f*>(&sh.red[wave][i][lane * 4]) = acc[i];
    __syncthreads();
    for (int i = wave; i < TILES; i += WAVES) {
        v4f s = *reinterpret_cast<const v4f*>(&sh.red[0][i][lane * 4]);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const v4f*>(&sh.red[w][i][lane * 4]);
        if (!F8) s *= 0.00390625f;
        *reinterpret_cast<v4f*>(&sh.red[0][i][lane * 4]) = s;
    }
    __syncthreads();
}

}  // namespace rows
}  // namespace apex4
