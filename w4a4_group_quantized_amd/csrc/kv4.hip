// Rotary positions, and the writes and reads of the 4-bit key/value cache
// (include/apex4.h: apex4_rope, apex4_kv4_append, apex4_kv4_read).
#include "attention.h"
#include "quant_rule.h"
#include "rotary.h"

namespace apex4 {
namespace {

// One token a workgroup: the sines of its pairs once, then its heads, D / 16
// lanes a head.
template <int TYPE>
__global__ __launch_bounds__(256) void rope_kernel(RopeProblem p)
{
    __shared__ double2 table[512];
    const int64_t t = blockIdx.x;
    rotary::fill(table, p.turn, rotary::position(p.turn, t));
    __syncthreads();
    const int lanes = p.D / 16;
    for (int i = threadIdx.x; i < p.H * lanes; i += 256) {
        const int h = i / lanes, j = i - h * lanes;
        const rotary::Runs r = rotary::runs(p.turn, j);
        const int64_t x = t * p.ldx + (int64_t)h * p.D, y = t * p.ldy + (int64_t)h * p.D;
        float a[16], b[16];
        rotary::load8<TYPE>(p.x, x + r.first, a);
        rotary::load8<TYPE>(p.x, x + r.second, a + 8);
        rotary::turn16(p.turn, table, j, a, b);
        rotary::store8<TYPE>(p.y, y + r.first, b);
        rotary::store8<TYPE>(p.y, y + r.second, b + 8);
    }
}

// max over the LANES neighbouring lanes of a head; the bits of absolute values
// rank them, with infinities and then NaN above every number
template <int LANES>
__device__ inline uint32_t head_max(uint32_t v)
{
    const auto step = [&](uint32_t o) { v = v > o ? v : o; };
    step(__builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false));
    if (LANES >= 8) step(__builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false));
    if (LANES >= 16) step(__builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false));
    return v;
}

// The scale and the nibbles (code + 8) of one head, 16 numbers a lane: the
// quantization rule of apex4_quantize_act with the head as the group.  4-bit
// codes have no NaN: a head with a number that is not finite gets a NaN scale.
template <int LANES>
__device__ inline float quantize16(const float (&x)[16], uint32_t& first, uint32_t& second)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffff;
        m = m > b ? m : b;
    }
    m = head_max<LANES>(m);
    if (m >= 0x7f800000) {
        first = second = 0x88888888;
        return __builtin_nanf("");
    }
    const float s = __builtin_bit_cast(float, m) / 7.0f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float c = s > 0.0f ? fminf(fmaxf(rintf(x[i] / s), -8.0f), 7.0f) : 0.0f;
        w[i / 8] |= (uint32_t)((int)c + 8) << (4 * (i % 8));
    }
    first = w[0], second = w[1];
    return s;
}

// The byte of a page's values that holds dims r and r + 16 of the 32 from 32 v
// on, r = 0: see include/apex4.h.  Byte r lies r * D / 8 further on.
__device__ inline int64_t value_byte(int off, int v, int D)
{
    return (int64_t)(off >> 4) * 8 * D + ((off >> 2) & 3) * 2 * D + 4 * v + (off & 3);
}

// One token a workgroup (or one of its `parts` shares of the heads): queries
// turned, keys turned and stored, values stored, D / 16 lanes a head.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void append_kernel(Kv4AppendProblem p, int parts)
{
    constexpr int LANES = D / 16, TYPE = BF16 ? 2 : 1;
    __shared__ double2 table[D / 2];
    const int64_t t = blockIdx.x / parts;
    const int part = blockIdx.x - (int)(t * parts);
    if (p.turn.positions) {
        rotary::fill(table, p.turn, rotary::position(p.turn, t));
        __syncthreads();
    }
    const Kv4Cache& c = p.cache;
    const int64_t slot = p.slots[t];
    const int64_t pg = slot >> c.shift;
    const bool stored = slot >= 0 && pg < c.pages;
    const int off = (int)(slot & (c.page - 1));
    const int heads = p.Hq + 2 * c.Hkv;
    for (int i = part * 256 + threadIdx.x; i < heads * LANES; i += parts * 256) {
        const int h = i / LANES, j = i % LANES;
        float a[16], b[16];
        if (h < p.Hq) {
            const rotary::Runs r = rotary::runs(p.turn, j);
            const int64_t x = t * p.ldq + (int64_t)h * D, y = (t * p.Hq + h) * D;
            rotary::load8<TYPE>(p.q, x + r.first, a);
            rotary::load8<TYPE>(p.q, x + r.second, a + 8);
            rotary::turn16(p.turn, table, j, a, b);
            rotary::store8<TYPE>(p.q_out, y + r.first, b);
            rotary::store8<TYPE>(p.q_out, y + r.second, b + 8);
        } else if (!stored) {
            continue;
        } else if (h < p.Hq + c.Hkv) {
            const int g = h - p.Hq;
            const rotary::Runs r = rotary::runs(p.turn, j);
            const int64_t x = t * p.ldk + (int64_t)g * D;
            rotary::load8<TYPE>(p.k, x + r.first, a);
            rotary::load8<TYPE>(p.k, x + r.second, a + 8);
            rotary::turn16(p.turn, table, j, a, b);
            uint32_t w0, w1;
            const float s = quantize16<LANES>(b, w0, w1);
            const int64_t row = (pg * c.Hkv + g) * c.page + off;
            uint32_t* out = reinterpret_cast<uint32_t*>(c.k_codes + row * (D / 2));
            out[r.first / 8] = w0;
            out[r.second / 8] = w1;
            if (j == 0) c.k_scales[row] = s;
        } else {
            const int g = h - p.Hq - c.Hkv;
            const int64_t x = t * p.ldv + (int64_t)g * D + 16 * j;
            rotary::load8<TYPE>(p.v, x, a);
            rotary::load8<TYPE>(p.v, x + 8, a + 8);
            uint32_t w0, w1;
            const float s = quantize16<LANES>(a, w0, w1);
            // lane j holds 16 dims of one nibble half: lanes 2 v and 2 v + 1 exchange words, and
            // write the bytes of r = 0..7 and 8..15
            const uint32_t other = __builtin_amdgcn_update_dpp(0, j & 1 ? w0 : w1, 0xB1, 0xF, 0xF, false);
            const uint32_t low = j & 1 ? other : w0, high = j & 1 ? w1 : other;
            const int64_t page = pg * c.Hkv + g;
            uint8_t* out = c.v_codes + page * c.page * (D / 2) + value_byte(off, j / 2, D) + (j & 1) * D;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                out[r * (D / 8)] = (uint8_t)(((low >> (4 * r)) & 15) | ((high >> (4 * r)) & 15) << 4);
            if (j == 0) c.v_scales[page * c.page + off] = s;
        }
    }
}

// 16 dims of one key and value head a lane.
template <int TYPE>
__global__ __launch_bounds__(256) void read_kernel(Kv4ReadProblem p, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const Kv4Cache& c = p.cache;
    const int lanes = c.D / 16;
    const int64_t row = i / lanes, t = row / c.Hkv;
    const int j = (int)(i - row * lanes), g = (int)(row - t * c.Hkv);
    const int64_t slot = p.slots[t], pg = slot >> c.shift;
    const int off = (int)(slot & (c.page - 1));
    float k[16] = {}, v[16] = {};
    if (slot >= 0 && pg < c.pages) {
        const int64_t page = pg * c.Hkv + g, at = page * c.page + off;
        const float ks = c.k_scales[at], vs = c.v_scales[at];
        const uint2 w = *reinterpret_cast<const uint2*>(c.k_codes + at * (c.D / 2) + 8 * j);
        const uint8_t* in = c.v_codes + page * c.page * (c.D / 2) + value_byte(off, j / 2, c.D);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            k[e] = (float)((int)((e < 8 ? w.x >> (4 * e) : w.y >> (4 * e - 32)) & 15) - 8) * ks;
            v[e] = (float)((int)((in[e * (c.D / 8)] >> (4 * (j & 1))) & 15) - 8) * vs;
        }
    }
    const int64_t y = row * c.D + 16 * j;
    rotary::store8<TYPE>(p.k, y, k);
    rotary::store8<TYPE>(p.k, y + 8, k + 8);
    rotary::store8<TYPE>(p.v, y, v);
    rotary::store8<TYPE>(p.v, y + 8, v + 8);
}

template <bool BF16>
hipError_t append(const Kv4AppendProblem& p, hipStream_t stream)
{
    const int items = (p.Hq + 2 * p.cache.Hkv) * (p.cache.D / 16);
    const int parts = p.T <= 256 ? (items + 255) / 256 : 1;
    const unsigned blocks = (unsigned)(p.T * parts);
    switch (p.cache.D) {
    case 64: append_kernel<BF16, 64><<<blocks, 256, 0, stream>>>(p, parts); break;
    case 128: append_kernel<BF16, 128><<<blocks, 256, 0, stream>>>(p, parts); break;
    default: append_kernel<BF16, 256><<<blocks, 256, 0, stream>>>(p, parts); break;   // checked by the caller
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeProblem& p, hipStream_t stream)
{
    const unsigned blocks = (unsigned)p.T;
    switch (p.type) {
    case 0: rope_kernel<0><<<blocks, 256, 0, stream>>>(p); break;
    case 1: rope_kernel<1><<<blocks, 256, 0, stream>>>(p); break;
    default: rope_kernel<2><<<blocks, 256, 0, stream>>>(p); break;
    }
    return hipGetLastError();
}

hipError_t launch_kv4_append(const Kv4AppendProblem& p, hipStream_t stream)
{
    return p.bf16 ? append<true>(p, stream) : append<false>(p, stream);
}

hipError_t launch_kv4_read(const Kv4ReadProblem& p, hipStream_t stream)
{
    const int64_t n = p.T * p.cache.Hkv * (p.cache.D / 16);
    const unsigned blocks = (unsigned)((n + 255) / 256);
    switch (p.type) {
    case 0: read_kernel<0><<<blocks, 256, 0, stream>>>(p, n); break;
    case 1: read_kernel<1><<<blocks, 256, 0, stream>>>(p, n); break;
    default: read_kernel<2><<<blocks, 256, 0, stream>>>(p, n); break;
    }
    return hipGetLastError();
}

}  // namespace apex4
