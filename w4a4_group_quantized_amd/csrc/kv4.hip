// Rotary positions, and the writes and reads of the 4-bit key/value cache
// (include/apex4.h: apex4_rope, apex4_kv4_append, apex4_kv4_read).
//
// All three are bound by bytes where there are many tokens, and by the launch
// where there are few (2 to 5 us on the GPU for one token to 64).  A token's heads
// share the sines of its pairs, so a workgroup takes one token; a head is D / 16
// lanes, which hold both numbers of their pairs (turned in place if asked) and
// find the head's largest number by lane moves.  Measured: 4096 tokens x 64 heads
// x 128 bf16 turned in 22 us (6.0 TB/s, the last-level cache holds part of it);
// 4096 tokens of 64 query and 8 key heads appended in 30 us (160 MB, 5.3 TB/s);
// 65521 tokens of 8 heads read in 49 to 58 us one call after the other (340 MB, 5.8-7.0
// TB/s), in 77 where other work's lines are in the caches (4.4 TB/s).  fp32 heads of 128
// and all of 256 keep to the caches (see read): 65521 tokens of 8 heads of 128 in
// fp32 165 us (3.7 TB/s).
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

// Stores a value head whose lane r of 16 has the numbers r + 16 h, h < N: by way
// of `lds` (the head's own, 16-byte aligned), so that a lane writes 16 neighbouring
// bytes at a time (written where the lanes have them, 64 neighbouring bytes a
// head and store, the call took half as long again).
template <int TYPE, int N, bool FAR>
__device__ inline void store_values(void* base, int64_t at, int r, const float (&v)[N], uint32_t* lds)
{
    constexpr int WORDS = (TYPE == 0 ? 16 : 8) * N, EACH = WORDS / 16;      // of the head, of a lane
    if (TYPE == 0) {
#pragma unroll
        for (int h = 0; h < N; ++h) lds[r + 16 * h] = __builtin_bit_cast(uint32_t, v[h]);
    } else {
        // lanes r and r + 1 exchange: the even one writes the pairs of even h, the odd one of odd h
#pragma unroll
        for (int h = 0; h < N; h += 2) {
            const uint32_t a = e4m3::to16<TYPE == 2>(v[h]), b = e4m3::to16<TYPE == 2>(v[h + 1]);
            const uint32_t other = __builtin_amdgcn_update_dpp(0, r & 1 ? a : b, 0xB1, 0xF, 0xF, false);
            lds[8 * h + (r & 1 ? 7 + (r + 1) / 2 : r / 2)] = r & 1 ? other | b << 16 : a | other << 16;
        }
    }
    // (the 16 lanes are of one wave)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    uint32_t* out = static_cast<uint32_t*>(base) + at / (TYPE == 0 ? 1 : 2) + r * EACH;
    if (EACH == 2) {
        rotary::put<FAR>(out, *reinterpret_cast<const uint2*>(lds + r * EACH));
    } else {
#pragma unroll
        for (int e = 0; e < EACH; e += 4)
            rotary::put<FAR>(out + e, *reinterpret_cast<const uint4*>(lds + r * EACH + e));
    }
}

// 16 lanes a head: of its key D / 16 neighbours each, of its value the numbers r +
// 16 h, whose bytes lie together in the cache (with those of three other tokens).
template <int TYPE, int D, int ROWS, bool FAR>
__global__ __launch_bounds__(256) void read_kernel(Kv4ReadProblem p, int n)
{
    constexpr int N = D / 16, WORDS = TYPE == 0 ? D : D / 2;
    __shared__ __attribute__((aligned(16))) uint32_t lds[16][ROWS][WORDS + 4];
    const int first = blockIdx.x * 16 * ROWS + threadIdx.x / 16, r = threadIdx.x % 16;
    const Kv4Cache& c = p.cache;
    int64_t slot[ROWS];
    int g[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = min(first + 16 * i, n - 1), t = (unsigned)row / (unsigned)c.Hkv;
        g[i] = row - t * c.Hkv;
        slot[i] = p.slots[t];
    }
    uint32_t kw[ROWS][(N + 7) / 8], vw[ROWS][N / 2];
    float ks[ROWS], vs[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        // (a slot that is none reads the cache's first token, and counts it as zeros)
        const bool live = slot[i] >= 0 && (slot[i] >> c.shift) < c.pages;
        const int64_t pg = live ? slot[i] >> c.shift : 0;
        const int off = live ? (int)(slot[i] & (c.page - 1)) : 0;
        const int64_t page = pg * c.Hkv + g[i], at = page * c.page + off;
        const uint8_t* keys = c.k_codes + at * (D / 2) + r * (N / 2);
        const uint32_t* values = reinterpret_cast<const uint32_t*>(c.v_codes + page * c.page * (D / 2) + (off >> 4) * 8 * D +
                                                                   (((off >> 2) & 3) * 16 + r) * (D / 8));
        if (N == 4) {
            kw[i][0] = *reinterpret_cast<const uint16_t*>(keys);
        } else {
#pragma unroll
            for (int e = 0; e < N / 8; ++e) kw[i][e] = reinterpret_cast<const uint32_t*>(keys)[e];
        }
#pragma unroll
        for (int e = 0; e < N / 2; ++e) vw[i][e] = values[e];
        ks[i] = c.k_scales[at], vs[i] = c.v_scales[at];
        if (!live) ks[i] = vs[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = first + 16 * i;
        if (row >= n) break;
        float k[N], v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) k[e] = (float)((int)((kw[i][e / 8] >> (4 * (e % 8))) & 15) - 8) * ks[i];
        // byte off % 4 of each word: the number of the even h in its low half, of the odd one in its high half
        const int shift = 8 * (int)(slot[i] & 3);
#pragma unroll
        for (int h = 0; h < N; ++h) v[h] = (float)((int)((vw[i][h / 2] >> (shift + 4 * (h & 1))) & 15) - 8) * vs[i];
        const int64_t y = (int64_t)row * D;
        if (N == 4) {
            if (TYPE == 0) {
                rotary::put<FAR>(static_cast<float*>(p.k) + y + N * r,
                                 __builtin_bit_cast(uint4, make_float4(k[0], k[1], k[2], k[3])));
            } else {
                const uint32_t a = e4m3::to16<TYPE == 2>(k[0]) | (uint32_t)e4m3::to16<TYPE == 2>(k[1]) << 16;
                const uint32_t b = e4m3::to16<TYPE == 2>(k[2]) | (uint32_t)e4m3::to16<TYPE == 2>(k[3]) << 16;
                rotary::put<FAR>(static_cast<uint16_t*>(p.k) + y + N * r, make_uint2(a, b));
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; e += 8) rotary::store8<TYPE, FAR>(p.k, y + N * r + e, k + e);
        }
        store_values<TYPE, N, FAR>(p.v, y, r, v, lds[threadIdx.x / 16][i]);
    }
}

template <int TYPE, int D>
void read(const Kv4ReadProblem& p, hipStream_t stream)
{
    // several heads' loads in flight where there are enough of them
    constexpr int ROWS = 2;
    const int n = (int)(p.T * p.cache.Hkv);
    const unsigned blocks = (unsigned)((n + 16 * ROWS - 1) / (16 * ROWS));
    // More than 128 MB, half the last-level cache, are stored past it (65521 tokens of
    // 8 heads, 268 MB, 79 us to 55; 49152 and a copy of them 147 to 128; of 67 MB the
    // read gains a few percent and a copy of it loses more: 38.6 to 40.8).  Only heads
    // of up to 256 bytes, which a store of 16 lanes writes whole: in pieces such
    // stores cost far more (heads of 256 in fp32 96 us to 322).
    constexpr int64_t head = D * (TYPE == 0 ? 4 : 2);
    if (head <= 256 && 2 * n * head > (int64_t(1) << 27)) read_kernel<TYPE, D, ROWS, head <= 256><<<blocks, 256, 0, stream>>>(p, n);
    else read_kernel<TYPE, D, ROWS, false><<<blocks, 256, 0, stream>>>(p, n);
}

template <int TYPE>
hipError_t read(const Kv4ReadProblem& p, hipStream_t stream)
{
    switch (p.cache.D) {
    case 64: read<TYPE, 64>(p, stream); break;
    case 128: read<TYPE, 128>(p, stream); break;
    default: read<TYPE, 256>(p, stream); break;    // checked by the caller
    }
    return hipGetLastError();
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
    switch (p.type) {
    case 0: return read<0>(p, stream);
    case 1: return read<1>(p, stream);
    default: return read<2>(p, stream);
    }
}

}  // namespace apex4
