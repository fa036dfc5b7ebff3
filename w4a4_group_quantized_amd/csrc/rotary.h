// Rotary positions on the GPU, shared by the rotary call and the cache's
// append.  Device functions only.
//
// A pair (a, b) of a head is turned by theta = position * frequency:
//     (a cos theta - b sin theta, b cos theta + a sin theta)
// Angles grow with the position (10^6 radians at position 10^6 for the fastest
// pair), where fp32 keeps no more than a sixteenth of a radian: angle, reduction
// to a quarter turn, sine, cosine and the products are all fp64, so what comes
// out is the pair rounded once, and an appended key's 4-bit codes do not depend
// on how the sine was computed.  On gfx950 an fp64 fma costs a vector
// instruction's slot like an fp32 one; the sine and cosine of a token's pairs
// are computed once for all its heads.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "gemm_e4m3.h"

namespace apex4 {
namespace rotary {

// sine and cosine of an angle: the angle less its nearest multiple of pi / 2
// (the multiple in two parts), then the Taylor series on [-pi/4, pi/4], whose
// first terms left out are r^17/17! and r^16/16! < 2^-49
__device__ inline double2 cos_sin(double angle)
{
    const double n = rint(angle * 0.63661977236758134308);
    double r = fma(-n, 1.57079632679489661923, angle);
    r = fma(-n, 6.12323399573676603587e-17, r);
    const double z = r * r;
    double s = -1.0 / 1307674368000.0;                                  // -1/15!
    s = fma(s, z, 1.0 / 6227020800.0);
    s = fma(s, z, -1.0 / 39916800.0);
    s = fma(s, z, 1.0 / 362880.0);
    s = fma(s, z, -1.0 / 5040.0);
    s = fma(s, z, 1.0 / 120.0);
    s = fma(s, z, -1.0 / 6.0);
    s = fma(s * z, r, r);
    double c = -1.0 / 87178291200.0;                                    // -1/14!
    c = fma(c, z, 1.0 / 479001600.0);
    c = fma(c, z, -1.0 / 3628800.0);
    c = fma(c, z, 1.0 / 40320.0);
    c = fma(c, z, -1.0 / 720.0);
    c = fma(c, z, 1.0 / 24.0);
    c = fma(c, z, -0.5);
    c = fma(c, z, 1.0);
    const int q = (int)((int64_t)n & 3);
    const double cq = q & 1 ? s : c, sq = q & 1 ? c : s;
    return make_double2(q == 1 || q == 2 ? -cq : cq, q & 2 ? -sq : sq);
}

// The position of token t, kept within 32 bits: beyond them the angle's own
// rounding leaves little of it.
__device__ inline double position(const Rotation& turn, int64_t t)
{
    const int64_t p = turn.positions[t], most = 0x7fffffff;
    return (double)(p > most ? most : p < -most ? -most : p);
}

// (scaled) cosines and sines of one token's pairs, by the whole workgroup; the
// caller synchronizes
__device__ inline void fill(double2* table, const Rotation& turn, double pos)
{
    for (int i = threadIdx.x; i < turn.rotary / 2; i += blockDim.x) {
        const double2 cs = cos_sin(pos * turn.freqs[i]);
        table[i] = make_double2(cs.x * turn.scale, cs.y * turn.scale);
    }
}

// A head of D numbers is shared by D / 16 lanes.  Lane j holds two runs of 8,
// starting at first(j) and second(j): both halves of its pairs, so that a head
// may be turned in place, or 16 neighbours.
struct Runs {
    int first, second;
};
__device__ inline Runs runs(const Rotation& turn, int j)
{
    if (turn.positions && !turn.interleaved && j < turn.rotary / 16) return {8 * j, 8 * j + turn.rotary / 2};
    return {16 * j, 16 * j + 8};
}

// turns the 16 numbers of lane j (before[0..7], before[8..15]: its two runs)
__device__ inline void turn16(const Rotation& turn, const double2* table, int j, const float (&before)[16],
                              float (&after)[16])
{
    const bool live = turn.positions && j < turn.rotary / 16;
    if (live && turn.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double2 cs = table[8 * j + i];
            const double a = before[2 * i], b = before[2 * i + 1];
            after[2 * i] = (float)fma(a, cs.x, -(b * cs.y));
            after[2 * i + 1] = (float)fma(b, cs.x, a * cs.y);
        }
    } else if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double2 cs = table[8 * j + i];
            const double a = before[i], b = before[8 + i];
            after[i] = (float)fma(a, cs.x, -(b * cs.y));
            after[8 + i] = (float)fma(b, cs.x, a * cs.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) after[i] = before[i];
    }
}

// 8 numbers of type TYPE (APEX4_F32, APEX4_F16, APEX4_BF16), 16-byte aligned
template <int TYPE>
__device__ inline void load8(const void* base, int64_t at, float* v)
{
    if (TYPE == 0) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const e4m3::Eight e = e4m3::load8<TYPE == 2>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e.v[i];
    }
}

// A store of two or four words; FAR: past the caches (what is written is more
// than they hold, so that nothing would find it there).
template <bool FAR>
__device__ inline void put(void* out, uint2 v)
{
    typedef uint32_t Two __attribute__((ext_vector_type(2)));
    if (FAR) __builtin_nontemporal_store(Two{v.x, v.y}, static_cast<Two*>(out));
    else *static_cast<uint2*>(out) = v;
}
template <bool FAR>
__device__ inline void put(void* out, uint4 v)
{
    typedef uint32_t Four __attribute__((ext_vector_type(4)));
    if (FAR) __builtin_nontemporal_store(Four{v.x, v.y, v.z, v.w}, static_cast<Four*>(out));
    else *static_cast<uint4*>(out) = v;
}

template <int TYPE, bool FAR = false>
__device__ inline void store8(void* base, int64_t at, const float* v)
{
    if (TYPE == 0) {
        float* p = static_cast<float*>(base) + at;
        put<FAR>(p, __builtin_bit_cast(uint4, make_float4(v[0], v[1], v[2], v[3])));
        put<FAR>(p + 4, __builtin_bit_cast(uint4, make_float4(v[4], v[5], v[6], v[7])));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3::to16<TYPE == 2>(v[2 * i]) | (uint32_t)e4m3::to16<TYPE == 2>(v[2 * i + 1]) << 16;
        put<FAR>(static_cast<uint16_t*>(base) + at, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

}  // namespace rotary
}  // namespace apex4
