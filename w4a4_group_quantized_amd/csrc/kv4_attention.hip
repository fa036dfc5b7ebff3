// Attention over the 4-bit key/value cache (include/apex4.h:
// apex4_kv4_attention).
//
// A wave takes 16 RT rows (a row is one query head of one token; the heads that
// share a key head are rows beside each other) and 64 cached tokens at a time:
//
//     S = K Q^T   tokens x rows    v_mfma_f32_16x16x32_f16
//     t = S s_k scale log2(e) + log2(s_v),  w = 2^(t - M)
//     O += V^T w  numbers x rows   the same instruction, w rounded to fp16
//     l += w / s_v
//
// M follows the row's running maximum of t, so the weights that the matrix unit sees
// carry the values' scales and the largest of them is 2^7 to 2^15 whatever those are:
// M is the maximum less 7 when it moves, and moves only when a tile exceeds that
// maximum by 8, which keeps the rescaling of O out of most tiles.  fp16's smallest
// step is then 2^-31 of the largest weight or less; with weights of at most 1 it was
// 2^-24, and thousands of tokens below half of that beside a large one left O, but
// not l.  l (of the weights before they are rounded) and M are fp32.
//
// Codes go to the matrix unit nearly as they lie: the nibble u = c + 8 in bits
// 4..7 of an fp16 is the subnormal number u 2^-20, which the instruction takes
// exactly, so eight codes cost seven instructions.  The accumulators of S start at
// -8 sum(q), and 8 sum(w) comes from one more matrix instruction whose first
// operand is 8 everywhere.  Nibbles in bits 0..3 (u 2^-24) would cost five, but
// the instruction adds eight neighbouring products aligned to the largest
// product of their exponent fields and drops what lies more than 24 bits below:
// with u 2^-24 that is 2^-14 of the largest weight for every product, and
// 131072 tokens with weights of all sizes came out 2.5 times further off than by
// the rounding of w; with u 2^-20 it is 2^-18, and does not show.
//
// Operands come straight from memory in the order that the instruction wants:
// a lane's 32 numbers of a key are D/8 neighbouring bytes, and the values' layout
// puts a lane's 4 tokens of all its numbers side by side.  S leaves the matrix
// unit with 4 tokens of one row in a lane, which is how the second product wants
// w: nothing goes through LDS but a token's three factors.
//
// Few rows (decoding): bound by the cache's bytes.  64 sequences of up to 8192
// tokens at random, 8 key heads of 128, 64 query heads: 62 us (5.3 TB/s of a
// read's 5.7-6.2); of 4096 each, several layers in turn, 60 us (4.8 TB/s); one of
// 131071 tokens 33 us with the join's 4 (5.1 TB/s in the first launch).  A wave
// alone takes 1.3 us for 64 tokens, 420 vector instructions of which unpacking is 224.
// Many rows (prompts): 4096 tokens, 64 and 8 heads, 300 us (917 TFLOP/s of 275 GFLOP
// seen; the library's plain product of 8192^3 reaches 1164).  The vector ALU is
// busy 59% of the time and the matrix unit 39%, and on a SIMD the two overlap little
// (64 matrix instructions of one wave beside 256 fmas of another take 1.4 times as
// long as either alone): the sum is the bound.
#include <algorithm>

#include "attention.h"
#include "kv4_cut.h"
#include "layers.h"
#include "rotary.h"

namespace apex4 {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr float kTiny = 0x1p-80f;      // the least scale of values: 2^15 / kTiny, 2^30 times, stays finite
constexpr float kLazy = 8.0f, kRoom = 7.0f;     // (fp16 holds weights of 2^(kLazy + kRoom))

// How a call is cut (launch_kv4_attention).
struct Plan {
    int tiles;          // row tiles of a sequence and key head that the grid holds (workgroups stride over more);
                        // 0: as many as each sequence has (see place)
    bool share;         // the workgroups share all units of the call evenly and leave the sums of the row tiles
                        // that they have parts of; else each takes whole row tiles
    bool sorted;        // (whole tiles) the longest of at most kSorted sequences first
    float* part_o;      // [2 workgroups, rows of a tile, D], sums relative to their M
    float2* part_ml;    // [2 workgroups, rows of a tile] of (M, l)
    struct Split* splits;
};

// A row tile that several workgroups share.  Each of them keeps two records: of
// the one that it goes on with, and of the one that it begins and others end.
struct Split {
    int64_t q0;         // first query of the sequence
    int row0, rows;     // first row and live rows of the tile (rows 0: no record)
    int g;              // key head
    int first, last;    // its workgroups
};

__device__ inline half8 mfma_operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_bit_cast(half8, make_uint4(a, b, c, d));
}

__device__ inline float4v mfma(half8 a, half8 b, float4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// the operand that is 8 everywhere
__device__ inline half8 eights() { return mfma_operand(0x00800080, 0x00800080, 0x00800080, 0x00800080); }

// over the four lanes that hold a row (16 lanes apart).  The swaps exchange halves
// and rows of two registers, here of one value's copies: then each lane has its
// own and the other's.  (Written out: of the builtins' results the compiler kept
// only the first.)
__device__ inline float row_max(float x)
{
    float y = x;
    asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    x = y = fmaxf(x, y);
    asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    return fmaxf(x, y);
}
__device__ inline float row_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// The numbers of one row and its place in the batch.
struct Sequence {
    int b;
    int64_t q0;         // its first query
    int n, kv;          // queries, cached tokens
};

__device__ inline Sequence sequence(const Kv4AttentionProblem& p, int b)
{
    Sequence s{b, b, 1, 0};
    if (p.cu_q) {
        const int64_t from = max(0, p.cu_q[b]), to = min(p.T, (int64_t)p.cu_q[b + 1]);
        s.q0 = from;
        s.n = (int)max((int64_t)0, to - from);
    }
    s.kv = (int)min((int64_t)max(0, p.kv_lens[b]), p.cols << p.cache.shift);
    return s;
}

// the tokens [lo, hi) that query i sees
__device__ inline int seen_hi(const Kv4AttentionProblem& p, const Sequence& s, int i)
{
    return p.causal ? max(0, s.kv - s.n + i + 1) : s.kv;
}
__device__ inline int seen_lo(const Kv4AttentionProblem& p, const Sequence& s, int i)
{
    return p.window ? max(0, s.kv - s.n + i + 1 - p.window) : 0;
}

// What a wave holds of its rows.
template <int D, int RT>
struct Rows {
    half8 q[RT][D / 32];
    float4v bias[RT];       // -8 sum(q) 2^-20
    float unit[RT];         // the power of two that was taken out of the query
    int lo[RT], hi[RT];
    float4v o[RT][D / 16];  // sums of w u 2^-20
    float4v w[RT];          // 8 sum(w) 2^-20
    float m[RT], l[RT];
};

// numbers of a key that lane quad `quad` holds in matrix instruction f
template <int D>
__device__ inline int key_number(int quad, int f)
{
    if (D == 64) return 16 * quad + 8 * f;
    return 128 * (f / 4) + 32 * quad + 8 * (f % 4);
}

template <int D, int RT>
struct RawRows {
    uint4 q[RT][D / 32];
};

template <int D, int RT>
__device__ inline void fetch_rows(const Kv4AttentionProblem& p, const Sequence& s, int g, int row0, RawRows<D, RT>& raw)
{
    const int lane = threadIdx.x & 63, quad = lane >> 4;
    const int share = p.share;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + 16 * rt + (lane & 15);
        const bool live = row < s.n * share;
        const int i = row / share;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + (s.q0 + i) * p.ldq + (int64_t)(g * share + row - i * share) * D;
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
            raw.q[rt][f] = make_uint4(0, 0, 0, 0);
            if (live) raw.q[rt][f] = *reinterpret_cast<const uint4*>(q + key_number<D>(quad, f));
        }
    }
}

template <bool BF16, int D, int RT>
__device__ inline void make_rows(const Kv4AttentionProblem& p, const Sequence& s, int row0, const RawRows<D, RT>& raw,
                                 Rows<D, RT>& r)
{
    const int lane = threadIdx.x & 63;
    const int share = p.share;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + 16 * rt + (lane & 15);
        const bool live = row < s.n * share;
        const int i = live ? row / share : 0;
        float x[D / 4], most = 0.0f;
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
            const uint32_t words[4] = {raw.q[rt][f].x, raw.q[rt][f].y, raw.q[rt][f].z, raw.q[rt][f].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[8 * f + k] = e4m3::from16<BF16>((uint16_t)(words[k / 2] >> (16 * (k % 2))));
                most = fmaxf(most, fabsf(x[8 * f + k]));
            }
        }
        most = row_max(most);
        // rows outside fp16's comfortable range are brought to 16..32 by a power of two (a bf16
        // number is exact in fp16 down to 2^-16, here 2^-10 of the row's largest at the least; smaller
        // ones are off by up to 2^-25, 2^-19 of the largest)
        int e = 0;
        if (!(most >= 0x1p-6f && most < 0x1p14f) && most > 0.0f && most < INFINITY) e = 5 - __builtin_amdgcn_frexp_expf(most);
        r.unit[rt] = __builtin_amdgcn_ldexpf(1.0f, -e);
        r.bias[rt] = float4v{};
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
            half8 v;
            constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = (_Float16)__builtin_amdgcn_ldexpf(x[8 * f + order[k]], e);
            r.q[rt][f] = v;
            r.bias[rt] = mfma(mfma_operand(0x80808080, 0x80808080, 0x80808080, 0x80808080), v, r.bias[rt]);
        }
        r.lo[rt] = live ? seen_lo(p, s, i) : 0;
        r.hi[rt] = live ? seen_hi(p, s, i) : 0;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) r.o[rt][t] = float4v{};
        r.w[rt] = float4v{};
        r.m[rt] = -INFINITY;
        r.l[rt] = 0.0f;
    }
}

// Codes of 64 tokens as they come from memory, 16 tokens a row of the array.
template <int D>
struct Codes {
    uint32_t w[4][D / 32];
};

// ONCE: for one row tile, so they need not stay in the caches (where sequences share
// pages the time is the same): what they would push out is read again sooner (64 sequences of 4096
// tokens in each of five layers in turn 66.5 us a layer to 60, 8 of 4096 in 34
// layers 17.7 to 16.5; but 143 MB read by one call after the other 34 to 35.5).
template <bool ONCE, typename T>
__device__ inline T load(const uint8_t* p)
{
    const T* at = reinterpret_cast<const T*>(p);
    return ONCE ? __builtin_nontemporal_load(at) : *at;
}
typedef uint32_t Two __attribute__((ext_vector_type(2)));
typedef uint32_t Four __attribute__((ext_vector_type(4)));

template <int D, bool ONCE>
__device__ inline void load_codes(Codes<D>& c, int s, const uint8_t* p)
{
    if (D == 64) {
        const Two a = load<ONCE, Two>(p);
        c.w[s][0] = a.x, c.w[s][1] = a.y;
    } else {
#pragma unroll
        for (int k = 0; k < D / 128; ++k) {
            const Four a = load<ONCE, Four>(p + (D / 128 == 2 ? 64 * k : 0));
            c.w[s][4 * k] = a.x, c.w[s][4 * k + 1] = a.y, c.w[s][4 * k + 2] = a.z, c.w[s][4 * k + 3] = a.w;
        }
    }
}

// (a lane's values are D/8 neighbouring bytes)
template <int D, bool ONCE>
__device__ inline void load_values(Codes<D>& c, int s, const uint8_t* p)
{
    if (D == 256) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Four a = load<ONCE, Four>(p + 16 * k);
            c.w[s][4 * k] = a.x, c.w[s][4 * k + 1] = a.y, c.w[s][4 * k + 2] = a.z, c.w[s][4 * k + 3] = a.w;
        }
    } else {
        load_codes<D, ONCE>(c, s, p);
    }
}

constexpr uint32_t kNibble = 0x00F000F0;

// a word of eight codes as a key's operand, and two of values as the operands of
// their low and high numbers
__device__ inline half8 key_operand(uint32_t u)
{
    return mfma_operand(u << 4 & kNibble, u & kNibble, u >> 4 & kNibble, u >> 8 & kNibble);
}
__device__ inline uint2 value_low(uint32_t u) { return make_uint2(u << 4 & kNibble, u >> 4 & kNibble); }
__device__ inline uint2 value_high(uint32_t u) { return make_uint2(u & kNibble, u >> 8 & kNibble); }

// A token's three factors, in arrays of N: of its scores, log2 of its values'
// scale, and that scale's reciprocal; for a place that holds none, what makes its
// weight zero.  A scale that is not finite shows through the second: a row that
// does not see the token multiplies the third by zero.
__device__ inline float key_factor(bool valid, float ks, float factor) { return valid ? ks * factor : 0.0f; }
template <int N>
__device__ inline void put_value_factors(float* factors, int at, bool valid, float vs)
{
    const float v = vs < kTiny ? kTiny : vs;               // (a NaN stays)
    factors[N + at] = valid ? __builtin_amdgcn_logf(v) : -INFINITY;
    factors[2 * N + at] = valid && v < INFINITY ? __builtin_amdgcn_rcpf(v) : 0.0f;
}

// Scores of 16 NS tokens times their factors; top: the largest that a lane has
// of its rows.
template <int D, int RT, int NS>
__device__ inline void exponents(float4v (&x)[RT][NS], const float* factors, float (&top)[RT])
{
    const int quad = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) top[rt] = -INFINITY;
#pragma unroll
    for (int sub = 0; sub < NS; ++sub) {
        const float4v kf = *reinterpret_cast<const float4v*>(factors + 16 * sub + 4 * quad);
        const float4v ls = *reinterpret_cast<const float4v*>(factors + 16 * NS + 16 * sub + 4 * quad);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[rt][sub][i] = fmaf(x[rt][sub][i], kf[i], ls[i]);
                top[rt] = fmaxf(top[rt], x[rt][sub][i]);
            }
        }
    }
}

// The same where some row does not see all the tokens from t0 on.
template <int D, int RT, int NS>
__device__ inline void mask(const Rows<D, RT>& r, float4v (&x)[RT][NS], const float* factors, int t0, float (&top)[RT])
{
    const int quad = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) top[rt] = -INFINITY;
#pragma unroll
    for (int sub = 0; sub < NS; ++sub) {
        const float4v ls = *reinterpret_cast<const float4v*>(factors + 16 * NS + 16 * sub + 4 * quad);
        const int t = t0 + 16 * sub + 4 * quad;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool seen = (t + i < r.hi[rt]) & (t + i >= r.lo[rt]) & (ls[i] != -INFINITY);
                x[rt][sub][i] = seen ? x[rt][sub][i] : -INFINITY;
                top[rt] = fmaxf(top[rt], x[rt][sub][i]);
            }
        }
    }
}

// Moves the rows' M where a tile is far above it, with what is relative to it.
template <int D, int RT>
__device__ inline void raise(Rows<D, RT>& r, float (&top)[RT])
{
    bool above = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        top[rt] = row_max(top[rt]) - (kLazy + kRoom);
        above |= top[rt] > r.m[rt];
    }
    if (!__any(above)) return;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float m = top[rt] > r.m[rt] ? top[rt] + kLazy : r.m[rt];
        const float old = m == r.m[rt] ? 1.0f : __builtin_amdgcn_exp2f(r.m[rt] - m);
        r.m[rt] = m;
        r.l[rt] *= old;
        r.w[rt] *= old;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) r.o[rt][t] *= old;
    }
}

// Exponents to weights, the operands of the second product.  fp16, because the codes
// are exact beside it and bf16 would hold 3 bits less: a weight is off by 2^-11 of
// itself.  Outputs in fp16 are 2.6 to 2.8 10^-4 of the largest off for it, and 2.0 to
// 2.1 with weights in fp32 (the outputs' own rounding).
template <int D, int RT, int NS>
__device__ inline void weights(Rows<D, RT>& r, const float4v (&x)[RT][NS], const float* factors, half8 (&w)[RT][NS / 2])
{
    const int quad = (threadIdx.x & 63) >> 4;
    float m[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) m[rt] = r.m[rt] == -INFINITY ? 0.0f : r.m[rt];
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) {
        uint32_t packed[RT][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int sub = 2 * i + half;
            const float4v iv = *reinterpret_cast<const float4v*>(factors + 32 * NS + 16 * sub + 4 * quad);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    e[k] = __builtin_amdgcn_exp2f(x[rt][sub][k] - m[rt]);
                    r.l[rt] = fmaf(e[k], iv[k], r.l[rt]);
                }
                // (codes of tokens 0 and 2, and 1 and 3, share a register)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    packed[rt][2 * half + k] = __builtin_bit_cast(uint32_t, __builtin_convertvector((float2v{e[k], e[k + 2]}), half2v));
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            w[rt][i] = mfma_operand(packed[rt][0], packed[rt][1], packed[rt][2], packed[rt][3]);
    }
}

template <int D, int RT, int NS>
__device__ inline void unscale(const Rows<D, RT>& r, float4v (&x)[RT][NS])
{
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int sub = 0; sub < NS; ++sub) x[rt][sub] *= r.unit[rt];
}

template <int RT>
__device__ inline bool any_scaled(const float (&unit)[RT])
{
    bool scaled = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) scaled |= unit[rt] != 1.0f;
    return __any(scaled);
}

__device__ inline void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

constexpr float kLog2e = 1.44269504f;

// The tokens [from, to) in tiles of 64, `step` apart, each unpacked by the wave
// for itself; `factors`: 192 floats of the wave.  The rows are fetched and made
// in the shadow of the first tokens' loads.
template <bool BF16, int D, int RT>
__device__ inline void attend(const Kv4AttentionProblem& p, const Sequence& s, int g, int row0, int from, int to, int step,
                              int lo_max, int hi_min, Rows<D, RT>& r, float* factors)
{
    // (a lane reads a value of 256 numbers in two pieces, which would fetch its lines twice)
    constexpr bool ONCE = RT == 1 && D <= 128;
    const Kv4Cache& c = p.cache;
    const int lane = threadIdx.x & 63, quad = lane >> 4;
    const int32_t* table = p.table + s.b * p.cols;
    const int last = (int)p.cols - 1;
    const float factor = p.scale * kLog2e * 0x1p20f;
    const int key_at = (lane & 15) * (D / 2) + quad * (D == 64 ? 8 : 16), value_at = lane * (D / 8);

    // The tile ahead, and the row in the cache of the lane's token of it (row 0 where there
    // is none).  (Two tiles ahead do not fit the registers of the larger rows, and gained
    // nothing for the smaller ones.)
    struct Ahead {
        Codes<D> k, v;
        float ks, vs;
        int64_t row;
        bool valid;
    } a;
    int page = 0;
    const auto look = [&](int t) { page = table[min((t + lane) >> c.shift, last)]; };
    const auto locate = [&](int t) {
        a.valid = t + lane < to && page >= 0 && page < c.pages;
        a.row = a.valid ? (((int64_t)page * c.Hkv + g) << c.shift) + ((t + lane) & (c.page - 1)) : 0;
    };
    const auto base = [&](int sub) {
        const uint32_t low = __builtin_amdgcn_readlane((uint32_t)a.row, 16 * sub);
        const uint32_t high = __builtin_amdgcn_readlane((uint32_t)(a.row >> 32), 16 * sub);
        return (int64_t)((uint64_t)high << 32 | low) * (D / 2);
    };
    const auto load_k = [&]() {
        a.ks = c.k_scales[a.row];
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) load_codes<D, ONCE>(a.k, sub, c.k_codes + base(sub) + key_at);
    };
    const auto load_v = [&]() {
        a.vs = c.v_scales[a.row];
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) load_values<D, ONCE>(a.v, sub, c.v_codes + base(sub) + value_at);
    };
    RawRows<D, RT> raw;
    look(from);
    fetch_rows<D, RT>(p, s, g, row0, raw);
    locate(from);
    look(from + step);
    load_k();
    load_v();
    make_rows<BF16, D, RT>(p, s, row0, raw, r);
    const bool scaled = any_scaled(r.unit);

    for (int t0 = from; t0 < to; t0 += step) {
        factors[lane] = key_factor(a.valid, a.ks, factor);
        put_value_factors<64>(factors, lane, a.valid, a.vs);
        const bool edge = t0 + 64 > hi_min || t0 < lo_max || !__all(a.valid);
        wave_sync();
        float4v x[RT][4];
        // (four accumulators between two instructions on the same one)
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
#pragma unroll
            for (int sub = 0; sub < 4; ++sub) {
                const half8 key = key_operand(a.k.w[sub][f]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt][sub] = mfma(key, r.q[rt][f], f == 0 ? r.bias[rt] : x[rt][sub]);
            }
        }
        locate(t0 + step);
        look(t0 + 2 * step);
        load_k();
        if (scaled) unscale<D, RT>(r, x);
        float top[RT];
        exponents<D, RT>(x, factors, top);
        if (edge) mask<D, RT>(r, x, factors, t0, top);
        raise<D, RT>(r, top);
        half8 w[RT][2];
        weights<D, RT>(r, x, factors, w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) r.w[rt] = mfma(eights(), w[rt][i], r.w[rt]);
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const uint2 b0 = value_low(a.v.w[2 * i][n]), b1 = value_low(a.v.w[2 * i + 1][n]);
                const uint2 c0 = value_high(a.v.w[2 * i][n]), c1 = value_high(a.v.w[2 * i + 1][n]);
                const half8 even = mfma_operand(b0.x, b0.y, b1.x, b1.y), odd = mfma_operand(c0.x, c0.y, c1.x, c1.y);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    r.o[rt][2 * n] = mfma(even, w[rt][i], r.o[rt][2 * n]);
                    r.o[rt][2 * n + 1] = mfma(odd, w[rt][i], r.o[rt][2 * n + 1]);
                }
            }
        }
        load_v();
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) r.l[rt] = row_sum(r.l[rt]);
}

// A tile of 64 tokens as operands, in the order in which the lanes take them.
template <int D>
struct Tile {
    uint4 k[4][D / 32][64];         // [16 tokens][32 numbers][lane]
    uint2 v[2][D / 16][64][2];      // [32 tokens][16 numbers][lane][16 tokens]
    float factors[192];
};

// Asks the scheduler to keep the reads of N operands AHEAD before the RT matrix
// instructions that take each (it kept two: 326 us for the prompt against 303).
template <int N, int RT>
__device__ inline void reads_ahead()
{
    constexpr int AHEAD = 6;
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, RT, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
}

// The same for a workgroup whose waves have rows of their own: wave i unpacks
// tokens 16 i .. of each tile into LDS for all of them, a tile ahead.  from, to:
// what some row of the workgroup sees.
template <int D, int RT>
__device__ inline void attend_shared(const Kv4AttentionProblem& p, const Sequence& s, int g, int from, int to, int lo_max,
                                     int hi_min, Rows<D, RT>& r, Tile<D>* tiles)
{
    const Kv4Cache& c = p.cache;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, quad = lane >> 4;
    const int32_t* table = p.table + s.b * p.cols;
    const int last = (int)p.cols - 1;
    const float factor = p.scale * kLog2e * 0x1p20f;
    const int key_at = (lane & 15) * (D / 2) + quad * (D == 64 ? 8 : 16), value_at = lane * (D / 8);
    const bool scaled = any_scaled(r.unit);

    int page = 0;
    bool valid = false;
    Codes<D> k, v;                  // (the first row only)
    float ks = 0.0f, vs = 0.0f;
    // the wave's 16 tokens of the tile at t are of one page
    const auto look = [&](int t) { page = table[min((t + 16 * wave) >> c.shift, last)]; };
    const auto load = [&](int t) {
        const int first = t + 16 * wave, at = __builtin_amdgcn_readfirstlane(page);
        const bool some = first < to && at >= 0 && at < c.pages;
        const int64_t row = some ? (((int64_t)at * c.Hkv + g) << c.shift) + (first & (c.page - 1)) : 0;
        valid = some && first + (lane & 15) < to;
        load_codes<D, false>(k, 0, c.k_codes + row * (D / 2) + key_at);
        load_values<D, false>(v, 0, c.v_codes + row * (D / 2) + value_at);
        ks = c.k_scales[row + (lane & 15)];
        vs = c.v_scales[row + (lane & 15)];
    };
    const auto unpack = [&](Tile<D>& tile) {
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
            tile.k[wave][f][lane] = __builtin_bit_cast(uint4, key_operand(k.w[0][f]));
            tile.v[wave >> 1][2 * f][lane][wave & 1] = value_low(v.w[0][f]);
            tile.v[wave >> 1][2 * f + 1][lane][wave & 1] = value_high(v.w[0][f]);
        }
        if (lane < 16) {
            tile.factors[16 * wave + lane] = key_factor(valid, ks, factor);
            put_value_factors<64>(tile.factors, 16 * wave + lane, valid, vs);
        }
    };
    __syncthreads();                // (the rows before are done with the tiles)
    if (from < to) {
        look(from);
        load(from);
        look(from + 64);
        unpack(tiles[0]);
        load(from + 64);
        look(from + 128);
    }
    int at = 0;
    for (int t0 = from; t0 < to; t0 += 64, at ^= 1) {
        __syncthreads();
        // (what the load before this one brought; the tile that it replaces was read before the barrier)
        unpack(tiles[at ^ 1]);
        load(t0 + 128);
        look(t0 + 192);
        const Tile<D>& tile = tiles[at];
        float4v x[RT][4];
        // (four accumulators between two instructions on the same one)
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
#pragma unroll
            for (int sub = 0; sub < 4; ++sub) {
                const half8 a = __builtin_bit_cast(half8, tile.k[sub][f][lane]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt][sub] = mfma(a, r.q[rt][f], f == 0 ? r.bias[rt] : x[rt][sub]);
            }
        }
        reads_ahead<4 * (D / 32), RT>();
        const bool edge = t0 + 64 > hi_min || t0 < lo_max || __any(tile.factors[64 + lane] == -INFINITY);
        __builtin_amdgcn_sched_barrier(0);
        if (scaled) unscale<D, RT>(r, x);
        float top[RT];
        exponents<D, RT>(x, tile.factors, top);
        if (edge) mask<D, RT>(r, x, tile.factors, t0, top);
        raise<D, RT>(r, top);
        half8 w[RT][2];
        weights<D, RT>(r, x, tile.factors, w);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) r.w[rt] = mfma(eights(), w[rt][i], r.w[rt]);
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                const half8 a = __builtin_bit_cast(half8, *reinterpret_cast<const uint4*>(&tile.v[i][n][lane][0]));
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) r.o[rt][n] = mfma(a, w[rt][i], r.o[rt][n]);
            }
        }
        reads_ahead<2 * (D / 16), RT>();
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) r.l[rt] = row_sum(r.l[rt]);
}

// numbers 16 t + 4 quad .. + 3 of a lane's row, held in units of 2^-20, times `by`
template <int D, int RT>
__device__ inline float4v row_values(const Rows<D, RT>& r, int rt, int t, float by)
{
    return (r.o[rt][t] - r.w[rt][0]) * by;
}

template <bool BF16>
__device__ inline void store4(void* out, int64_t at, float4v v)
{
    uint2 w;
    w.x = e4m3::to16<BF16>(v[0]) | (uint32_t)e4m3::to16<BF16>(v[1]) << 16;
    w.y = e4m3::to16<BF16>(v[2]) | (uint32_t)e4m3::to16<BF16>(v[3]) << 16;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
}

__device__ inline float log_sum(float m, float l) { return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.693147181f; }

// The row tile of workgroup x, of R rows: key heads beside each other, then the
// tiles of a sequence, then the sequences.  Uneven sequences (a prompt beside
// decoding ones) have a tile k of sequence b at floor(its first row / R) + b + k:
// no two at one place, and at most B places empty.
struct Place {
    int b, g, k;        // k outside the sequence's tiles: an empty place
};
template <int R>
__device__ inline Place place(const Kv4AttentionProblem& p, int tiles, int x)
{
    const int g = x % p.cache.Hkv;
    x /= p.cache.Hkv;
    if (tiles) return {x / tiles, g, x % tiles};
    const auto first = [&](int b) { return (int)(min(sequence(p, b).q0, p.T) * p.share / R) + b; };
    int b = 0;
    for (int n = p.B; n > 1;) {                            // the last of n that begins at or before x, 64 at a time
        const int step = (n + 63) / 64, at = (threadIdx.x & 63) * step;
        const int upto = max(1, __popcll(__ballot(at < n && first(min(b + at, p.B - 1)) <= x))) - 1;
        b += upto * step;
        n = min(step, n - upto * step);
    }
    b = __builtin_amdgcn_readfirstlane(b);
    return {b, g, x - first(b)};
}

// Few rows: the waves of a workgroup have the same rows and every fourth 64
// tokens; their sums meet in LDS.  256 tokens of a row tile are a unit (kUnit).
template <int D, int RT>
struct Meeting {
    float factors[kWaves][192];
    float sums[kWaves][16 * RT][D + 4];
    float2 tops[kWaves][16 * RT];
};

// Units [u0, u1) of a row tile, counted from the token `base`.  slot < 0: those
// are all, and the rows are written; else the sums go to the workspace.
template <bool BF16, int D, int RT>
__device__ inline void few_rows(const Kv4AttentionProblem& p, const Plan& plan, const Sequence& s, int g, int row0, int base,
                                int u0, int u1, int slot, Meeting<D, RT>& lds)
{
    constexpr int R = 16 * RT;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int share = p.share, all = s.n * share;
    const int i0 = row0 / share, i1 = min(row0 + R - 1, all - 1) / share;
    // (tokens that no row of the tile sees are passed over)
    const int from = max(base + u0 * kUnit, seen_lo(p, s, i0) & ~(kUnit - 1)) + 64 * wave;
    const int to = (int)min((int64_t)seen_hi(p, s, i1), base + (int64_t)u1 * kUnit);
    Rows<D, RT> r;
    attend<BF16, D, RT>(p, s, g, row0, from, to, kUnit, seen_lo(p, s, i1), seen_hi(p, s, i0), r, lds.factors[wave]);
    __syncthreads();                                       // (the rows before are out of LDS)
    if (lane < 16) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) lds.tops[wave][16 * rt + lane] = make_float2(r.m[rt], r.l[rt]);
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = 16 * rt + (lane & 15);
        float m = lds.tops[0][row].x;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) m = fmaxf(m, lds.tops[v][row].x);
        const float by = (r.m[rt] == m ? 1.0f : __builtin_amdgcn_exp2f(r.m[rt] - m)) * 0x1p20f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
            *reinterpret_cast<float4v*>(&lds.sums[wave][row][16 * t + 4 * (lane >> 4)]) = row_values(r, rt, t, by);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < R * (D / 4); e += 64 * kWaves) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        if (row0 + row >= all) break;
        float m = lds.tops[0][row].x, l = 0.0f;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) m = fmaxf(m, lds.tops[v][row].x);
        float4v o = {};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const float2 ml = lds.tops[v][row];
            l += ml.y * (ml.x == m ? 1.0f : __builtin_amdgcn_exp2f(ml.x - m));
            o += *reinterpret_cast<const float4v*>(&lds.sums[v][row][d]);
        }
        if (slot < 0) {
            const int i = (row0 + row) / share;
            const int64_t at = (s.q0 + i) * p.Hq + g * share + (row0 + row - i * share);
            store4<BF16>(p.out, at * D + d, o * (l == 0.0f ? 0.0f : 1.0f / l));
            if (p.lse && d == 0) p.lse[at] = log_sum(m, l);
        } else {
            *reinterpret_cast<float4v*>(plan.part_o + ((int64_t)slot * R + row) * D + d) = o;
            if (d == 0) plan.part_ml[slot * R + row] = make_float2(m, l);
        }
    }
}

// The first token of a sequence's first unit, its row tiles, the units of one.
struct Extent {
    int base, tiles, units;
};
template <int R>
__device__ inline Extent extent(const Kv4AttentionProblem& p, const Sequence& s)
{
    const int base = seen_lo(p, s, 0) & ~(kUnit - 1);
    // (at least one: rows that see nothing are written too)
    return {base, (s.n * p.share + R - 1) / R, max(1, (s.kv - base + kUnit - 1) / kUnit)};
}

// Many rows: every wave has rows of its own and walks all the tokens they see.
// (Unpacking for itself, without LDS and barriers, it takes 355 us for the prompt
// against 322 on one box; 64 rows a wave do not fit the registers: 650 us.)
// UNEVEN: the batch may hold sequences of few rows (an instance of its own: the
// prompt takes 325 us with both in one against 302).
template <bool BF16, int D, int RT, bool UNEVEN>
__global__ __launch_bounds__(256, 2) void rows_kernel(Kv4AttentionProblem p, Plan plan)
{
    __shared__ union __attribute__((aligned(16))) {
        Tile<D> buffers[2];
        Meeting<D, 1> meeting;
    } lds;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Place own = place<16 * RT * kWaves>(p, UNEVEN ? 0 : plan.tiles, blockIdx.x);
    const Sequence s = sequence(p, own.b);
    const int g = own.g, share = p.share, all = s.n * share, tiles = (all + 16 * RT * kWaves - 1) / (16 * RT * kWaves);
    if (own.k < 0) return;
    if (UNEVEN && all <= 16) {
        // A decoding sequence beside a prompt: its tokens for all waves (63 of 4096
        // tokens and a prompt of 512 take 64 us, with the rows in one wave 164).
        const Extent e = extent<16>(p, s);
        if (own.k < e.tiles) few_rows<BF16, D, 1>(p, plan, s, g, 0, e.base, 0, e.units, -1, lds.meeting);
        return;
    }
    for (int k = own.k; k < tiles; k += UNEVEN ? tiles : plan.tiles) {
        // (the last rows see the most tokens: first)
        const int top = (tiles - 1 - k) * kWaves * 16 * RT, row0 = top + wave * 16 * RT;
        Rows<D, RT> r;
        RawRows<D, RT> raw;
        fetch_rows<D, RT>(p, s, g, row0, raw);
        make_rows<BF16, D, RT>(p, s, row0, raw, r);
        const int i0 = row0 / share, i1 = min(row0 + 16 * RT - 1, all - 1) / share;
        const int end = min(top + kWaves * 16 * RT, all) - 1;
        attend_shared<D, RT>(p, s, g, seen_lo(p, s, top / share) & ~63, seen_hi(p, s, end / share), seen_lo(p, s, i1),
                             seen_hi(p, s, i0), r, lds.buffers);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int row = row0 + 16 * rt + (lane & 15);
            if (row >= all) continue;
            const int i = row / share;
            const int64_t at = (s.q0 + i) * p.Hq + g * share + (row - i * share);
            const float by = r.l[rt] == 0.0f ? 0.0f : 1.0f / r.l[rt];
#pragma unroll
            for (int t = 0; t < D / 16; ++t)           // (1 / l may be so large that 2^20 times it is beyond fp32)
                store4<BF16>(p.out, at * D + 16 * t + 4 * (lane >> 4), row_values(r, rt, t, 0x1p20f) * by);
            if (p.lse && lane < 16) p.lse[at] = log_sum(r.m[rt], r.l[rt]);
        }
    }
}

// sum over the workgroup; `lds`: a number a wave
__device__ inline int64_t block_sum(int64_t x, int64_t* lds)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) x += lds[v];
    return x;
}

template <bool BF16, int D, int RT>
__global__ __launch_bounds__(256, 2) void few_kernel(Kv4AttentionProblem p, Plan plan)
{
    constexpr int R = 16 * RT;
    __shared__ __attribute__((aligned(16))) Meeting<D, RT> lds;
    const int Hkv = p.cache.Hkv;
    if (!plan.share) {
        Place own = place<R>(p, plan.tiles, blockIdx.x);
        if (plan.sorted) {
            // in place of sequence b the b-th longest
            __shared__ __attribute__((aligned(16))) int lengths[kSorted];
            __shared__ int chosen;
            const int b = threadIdx.x;
            int mine = -1, rank = 0;
            if (b < p.B) mine = extent<R>(p, sequence(p, b)).units;
            lengths[b] = mine;
            __syncthreads();
            for (int i = 0; i < p.B; i += 4) {
                const int4 other = *reinterpret_cast<const int4*>(lengths + i);
                rank += (other.x > mine || (other.x == mine && i < b)) + (other.y > mine || (other.y == mine && i + 1 < b)) +
                        (other.z > mine || (other.z == mine && i + 2 < b)) + (other.w > mine || (other.w == mine && i + 3 < b));
            }
            if (b < p.B && rank == own.b) chosen = b;
            __syncthreads();
            own.b = __builtin_amdgcn_readfirstlane(chosen);
        }
        const Sequence s = sequence(p, own.b);
        const Extent e = extent<R>(p, s);
        if (own.k < 0) return;
        for (int k = own.k; k < e.tiles; k += plan.tiles ? plan.tiles : e.tiles)
            few_rows<BF16, D, RT>(p, plan, s, own.g, k * R, e.base, 0, e.units, -1, lds);
        return;
    }
    // Units of all sequences in a row, an even share for each workgroup.
    __shared__ int64_t sums[kWaves];
    __shared__ int64_t before;
    __shared__ int start;
    const auto units = [&](int b) {
        const Sequence s = sequence(p, b);
        const Extent e = extent<R>(p, s);
        return (int64_t)Hkv * e.tiles * e.units;
    };
    int64_t total = 0;
    for (int b = threadIdx.x; b < p.B; b += 64 * kWaves) total += units(b);
    total = block_sum(total, sums);
    const int64_t each = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x);
    int64_t u = blockIdx.x * each;
    const int64_t end = min(total, u + each);
    if (threadIdx.x == 0) plan.splits[2 * blockIdx.x].rows = plan.splits[2 * blockIdx.x + 1].rows = 0;
    if (u >= end) return;
    // the sequence that holds unit u
    int64_t seen = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64 * kWaves) {
        const int b = b0 + threadIdx.x, lane = threadIdx.x & 63;
        const int64_t mine = b < p.B ? units(b) : 0;
        int64_t upto = mine;                               // (with the lanes before)
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t x = __shfl_up(upto, o);
            if (lane >= o) upto += x;
        }
        __syncthreads();
        if (lane == 63) sums[threadIdx.x >> 6] = upto;
        __syncthreads();
        int64_t ahead = seen;
        for (int v = 0; v < kWaves; ++v) {
            if (v < (int)(threadIdx.x >> 6)) ahead += sums[v];
            seen += sums[v];
        }
        if (ahead + upto - mine <= u && u < ahead + upto) before = ahead + upto - mine, start = b;
        if (seen > u) break;
    }
    __syncthreads();
    int b = start;
    int64_t rest = u - before;                             // units of the sequence before u
    while (u < end) {
        const Sequence s = sequence(p, b);
        const Extent e = extent<R>(p, s);
        const int64_t whole = (int64_t)e.tiles * e.units;
        if (rest >= Hkv * whole) {
            rest -= Hkv * whole;
            ++b;
            continue;
        }
        const int g = (int)(rest / whole), k = (int)((rest - g * whole) / e.units);
        const int u0 = (int)(rest - g * whole - (int64_t)k * e.units);
        const int n = (int)min((int64_t)(e.units - u0), end - u);
        int slot = -1;
        if (n < e.units) {
            slot = 2 * blockIdx.x + (u0 == 0);
            const int rows = min(R, s.n * p.share - k * R);
            const int64_t at = u - u0;                     // its first unit
            if (threadIdx.x == 0) plan.splits[slot] = {s.q0, k * R, rows, g, (int)(at / each), (int)((at + e.units - 1) / each)};
        }
        few_rows<BF16, D, RT>(p, plan, s, g, k * R, e.base, u0, u0 + n, slot, lds);
        u += n;
        rest += n;
    }
}

// The sums of the row tiles that several workgroups share, in the order of the
// tokens.  The workgroups here stand for those: each takes every n-th row of the
// tiles that it was one of n for.  PARTS waves a row, WAVES in all.
template <bool BF16, int D, int RT, int WAVES, int PARTS>
__global__ __launch_bounds__(64 * WAVES) void join_kernel(Kv4AttentionProblem p, Plan plan)
{
    constexpr int EACH = D / 64, R = 16 * RT;
    static_assert(PARTS == 1 || PARTS == WAVES, "");
    __shared__ float sums[PARTS][D];
    __shared__ float2 tops[PARTS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int part = PARTS == 1 ? 0 : wave;
    const int share = p.share;
    const Split records[2] = {plan.splits[2 * blockIdx.x], plan.splits[2 * blockIdx.x + 1]};
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const Split& s = records[which];
        if (s.rows == 0) continue;
        const int n = s.last - s.first + 1;
        // (the first workgroup's sums are its second ones)
        const auto slot = [&](int i) { return (int64_t)(2 * (s.first + i) + (i == 0)) * R; };
        for (int row = (int)blockIdx.x - s.first + (PARTS == 1 ? wave * n : 0); row < s.rows; row += n * (WAVES / PARTS)) {
            // one pass over the wave's parts with a maximum of its own
            float m = -INFINITY, l = 0.0f, o[EACH] = {};
#pragma unroll 4
            for (int i = part; i < n; i += PARTS) {
                const float2 ml = plan.part_ml[slot(i) + row];
                const float* from = plan.part_o + (slot(i) + row) * D + lane * EACH;
                const float top = fmaxf(m, ml.x);
                const float old = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
                const float by = ml.x == top ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top);
                l = l * old + ml.y * by;
#pragma unroll
                for (int e = 0; e < EACH; ++e) o[e] = o[e] * old + from[e] * by;
                m = top;
            }
            if (PARTS > 1) {
                __syncthreads();                           // (the row before is out of LDS)
#pragma unroll
                for (int e = 0; e < EACH; ++e) sums[part][lane * EACH + e] = o[e];
                if (lane == 0) tops[part] = make_float2(m, l);
                __syncthreads();
                if (part != 0) continue;
#pragma unroll
                for (int v = 0; v < PARTS; ++v) m = fmaxf(m, tops[v].x);
                l = 0.0f;
#pragma unroll
                for (int e = 0; e < EACH; ++e) o[e] = 0.0f;
#pragma unroll
                for (int v = 0; v < PARTS; ++v) {
                    const float2 ml = tops[v];
                    const float by = ml.x == m ? 1.0f : __builtin_amdgcn_exp2f(ml.x - m);
                    l += ml.y * by;
#pragma unroll
                    for (int e = 0; e < EACH; ++e) o[e] += sums[v][lane * EACH + e] * by;
                }
            }
            const float by = l == 0.0f ? 0.0f : 1.0f / l;
            const int i = (s.row0 + row) / share;
            const int64_t at = (s.q0 + i) * p.Hq + s.g * share + (s.row0 + row - i * share);
#pragma unroll
            for (int e = 0; e < EACH; ++e)
                static_cast<uint16_t*>(p.out)[at * D + lane * EACH + e] = e4m3::to16<BF16>(o[e] * by);
            if (p.lse && lane == 0) p.lse[at] = log_sum(m, l);
        }
    }
}

Cut cut(const Kv4AttentionProblem& p)
{
    const int cus = compute_units();
    return kv4_cut(p.T, p.B, p.cache.Hkv, p.share, p.cache.D, p.max_q, p.max_kv, p.window, cus > 0 ? cus : 256);
}

template <bool BF16, int D, int RT>
hipError_t launch(const Kv4AttentionProblem& p, const Cut& c, const Plan& plan, hipStream_t stream)
{
    const unsigned blocks = (unsigned)c.blocks;
    if constexpr (RT == row_tiles(D)) {
        if (c.rows) {
            if (c.tiles) rows_kernel<BF16, D, RT, false><<<blocks, 256, 0, stream>>>(p, plan);
            else rows_kernel<BF16, D, RT, true><<<blocks, 256, 0, stream>>>(p, plan);
            return hipGetLastError();
        }
    }
    few_kernel<BF16, D, RT><<<blocks, 256, 0, stream>>>(p, plan);
    if (c.share) {
        if (c.deep) join_kernel<BF16, D, RT, 16, 16><<<blocks, 1024, 0, stream>>>(p, plan);
        else join_kernel<BF16, D, RT, 8, 1><<<blocks, 512, 0, stream>>>(p, plan);
    }
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch(const Kv4AttentionProblem& p, const Cut& c, const Plan& plan, hipStream_t stream)
{
    switch (p.cache.D) {
    case 64: return c.rt == 1 ? launch<BF16, 64, 1>(p, c, plan, stream) : launch<BF16, 64, 2>(p, c, plan, stream);
    case 128: return c.rt == 1 ? launch<BF16, 128, 1>(p, c, plan, stream) : launch<BF16, 128, 2>(p, c, plan, stream);
    default: return launch<BF16, 256, 1>(p, c, plan, stream);
    }
}

// the workspace: sums of two row tiles a workgroup, their (M, l), records of them
size_t parts(const Cut& c) { return (size_t)c.blocks * 2 * 16 * c.rt; }

}  // namespace

size_t kv4_attention_workspace_bytes(const Kv4AttentionProblem& p)
{
    const Cut c = cut(p);
    return c.share ? parts(c) * (p.cache.D + 2) * 4 + 2 * (size_t)c.blocks * sizeof(Split) : 0;
}

hipError_t launch_kv4_attention(const Kv4AttentionProblem& p, hipStream_t stream)
{
    const Cut c = cut(p);
    Plan plan{c.tiles, c.share, c.sorted, nullptr, nullptr, nullptr};
    if (c.share) {
        plan.part_o = static_cast<float*>(p.ws);
        plan.part_ml = reinterpret_cast<float2*>(plan.part_o + parts(c) * p.cache.D);
        plan.splits = reinterpret_cast<Split*>(plan.part_ml + parts(c));
    }
    return p.bf16 ? launch<true>(p, c, plan, stream) : launch<false>(p, c, plan, stream);
}

}  // namespace apex4
