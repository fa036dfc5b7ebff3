// Routing of tokens to experts on gfx950: scores, groups, top-k and gates of
// one token per wave.
//
//     p_e = softmax_E(l)_e  or  1 / (1 + exp(-l_e));   key c_e = p_e + bias_e
//
// and the k experts of the largest keys, after the groups with the largest
// sums of their one or two best keys were kept.  Without a bias the scores
// rise with the logits, so the experts are ranked by the logits themselves,
// as 32-bit integers in the order of the floats; with a bias, and for the
// sums of two scores, ranks depend on computed values, and those are held in
// 64 bits so that two scores next to each other do not change places by a
// rounding.  Ties go to the lowest index.  A masked expert (logit or key -inf
// or NaN) has the rank key 0, below every live one.
//
// What bounds it: vector instructions.  A wave holds its row in registers (E / 64
// values a lane) and reads it once; 16384 rows of 256 experts are 16 rows a SIMD,
// so every 100 instructions a row are 3 us.  Hence
//   - the scores' exp and reciprocal are written out (a sigmoid in 64 bits is
//     about 26 instructions here, over 60 from the library);
//   - lane moves are DPP (moves through LDS, 130 a row, were two thirds of the
//     first kernel's 38 us; the row takes 29 now);
//   - a round of "largest key of the wave" runs on 32 bits: the keys rounded to
//     fp32, in the order of the numbers.  Rounding keeps the order, so the
//     largest key is among the lanes that hold the largest rounded one; only
//     where those are several do the 64-bit keys and the indices decide;
//   - up to 4 values a lane are sorted once, and a round looks at each lane's
//     first only.
// What is left is paid once a row for the whole wave: of 1080 instructions a
// row the groups' step takes 370, and the rounds most of the rest (one 32-bit
// score a value, 64 bits for the gates only).  Rows that shared a wave would
// share them; that is not built.
#include "layers.h"

namespace apex4 {
namespace {

constexpr int WAVES = 4;      // rows per workgroup
constexpr int MAX_E = 1024;

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t M;
    int32_t E, k;
    int32_t type;             // APEX4_F32, APEX4_F16, APEX4_BF16
    int32_t n_group, gsize, keep, top;
    uint32_t gmagic;          // floor(2^32 / gsize) + 1: e / gsize = (e * gmagic) >> 32 for e < 2^16
    bool sigmoid, renormalize;
    float scale;
    int32_t* ids;
    float* gates;
};

__device__ inline float load_logit(const RouteArgs& a, int64_t i)
{
    if (a.type == 0) return static_cast<const float*>(a.logits)[i];
    if (a.type == 1) return (float)static_cast<const _Float16*>(a.logits)[i];
    return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(a.logits)[i] << 16);
}

// integers in the order of the numbers, 0 for none of them (-inf is not 0)
__device__ inline uint32_t ordered(float x)
{
    x += 0.0f;                // -0 ranks as 0
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b >> 31 ? ~b : b | 0x80000000u;
}
template <int CTRL, int ROWS>
__device__ inline int dpp(int old, int x)
{
    return __builtin_amdgcn_update_dpp(old, x, CTRL, ROWS, 0xF, false);
}
constexpr int SWAP1 = 0xB1, SWAP2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140, BCAST15 = 0x142, BCAST31 = 0x143;

template <int CTRL, int ROWS>
__device__ inline double dpp(double old, double x)
{
    const int2 o = __builtin_bit_cast(int2, old), v = __builtin_bit_cast(int2, x);
    return __builtin_bit_cast(double, make_int2(dpp<CTRL, ROWS>(o.x, v.x), dpp<CTRL, ROWS>(o.y, v.y)));
}

__device__ inline uint32_t wave_max(uint32_t v)
{
    v = max(v, (uint32_t)dpp<SWAP1, 0xF>(0, (int)v));
    v = max(v, (uint32_t)dpp<SWAP2, 0xF>(0, (int)v));
    v = max(v, (uint32_t)dpp<HALF_MIRROR, 0xF>(0, (int)v));
    v = max(v, (uint32_t)dpp<MIRROR, 0xF>(0, (int)v));
    v = max(v, (uint32_t)dpp<BCAST15, 0xA>(0, (int)v));
    v = max(v, (uint32_t)dpp<BCAST31, 0xC>(0, (int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// (the same tree for every row: the sum does not depend on where a row lies)
__device__ inline double wave_sum(double v)
{
    v += dpp<SWAP1, 0xF>(0.0, v);
    v += dpp<SWAP2, 0xF>(0.0, v);
    v += dpp<HALF_MIRROR, 0xF>(0.0, v);
    v += dpp<MIRROR, 0xF>(0.0, v);
    v += dpp<BCAST15, 0xA>(0.0, v);
    v += dpp<BCAST31, 0xC>(0.0, v);
    const int2 b = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double,
                              make_int2(__builtin_amdgcn_readlane(b.x, 63), __builtin_amdgcn_readlane(b.y, 63)));
}

// exp(x) for x <= 1000 (above 709.8: infinity): x = n ln 2 + r, |r| <= ln 2 / 2, by the Taylor series of
// exp(r) (its 14th power is below 4e-18).  -inf and what underflows give 0.
__device__ inline double exp64(double x)
{
    x = fmax(x, -746.0);
    const double n = rint(x * 1.4426950408889634);
    double r = fma(n, -6.93147180369123816490e-01, x);     // ln 2 in two parts, the first of 33 bits (fdlibm's)
    r = fma(n, -1.90821492927058770002e-10, r);
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / x for 1 <= x: the hardware's estimate and two Newton steps (not on the estimate 0 of an infinite x)
__device__ inline double reciprocal(double x)
{
    double y = __builtin_amdgcn_rcp(x);
    y = fma(fma(-x, y, 1.0), y, y);
    y = fma(fma(-x, y, 1.0), y, y);
    return x > 1.7e308 ? 0.0 : y;
}

__device__ inline double sigmoid64(double x) { return reciprocal(1.0 + exp64(fmin(-x, 1000.0))); }

// 32-bit scores: within 1e-6 of the 64-bit ones (below)
__device__ inline float exp32(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ inline float sigmoid32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp32(-x)); }

template <int CTRL, int ROWS>
__device__ inline float dpp(float old, float x)
{
    return __builtin_bit_cast(
        float, dpp<CTRL, ROWS>(__builtin_bit_cast(int, old), __builtin_bit_cast(int, x)));
}
__device__ inline double read_lane(double x, int l)
{
    const int2 b = __builtin_bit_cast(int2, x);
    return __builtin_bit_cast(double,
                              make_int2(__builtin_amdgcn_readlane(b.x, l), __builtin_amdgcn_readlane(b.y, l)));
}
__device__ inline float read_lane(float x, int l)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}
__device__ inline float from_ordered(uint32_t k)
{
    return __builtin_bit_cast(float, k >> 31 ? k & 0x7FFFFFFFu : ~k);
}

// What the scores of a row are taken against: softmax's maximum and sum.
struct Row {
    double high, total;
};

// The choice of a row: lane j's j-th expert, -1 for none.  V: values per lane
// (E <= 64 V).  WIDE: ranks by computed keys (a bias), else by the logits.
// GROUPS: 0 none, 1 a group's score is its best key, 2 the sum of its two best.
// T: the type of computed keys.  In 32 bits a key is within 1e-6 max(1, |key|)
// of its value (exp within |x| 2^-24 relative, a factor that the slope of the
// score cancels for large |x|; the sum of a softmax within 1e-6; one rounding
// by the bias), and `sure` says whether no two keys that decide were nearer to
// each other than four times that, and every kept group is above every dropped
// one by more than their keys may be off by.  If not, the caller asks again in 64
// bits: about one row in a few hundred, where all of them in 64 bits took 41 us
// instead of 29 (16384 rows of 256 experts in 8 groups).
template <int V, bool WIDE, int GROUPS, typename T>
__device__ inline int choose(const RouteArgs& a, int64_t row, const float (&x)[V], const Row& of, T* values, bool& sure)
{
    constexpr bool SORT = V <= 4, EXACT = std::is_same<T, double>::value;
    const int lane = threadIdx.x & 63;
    const float masked = -__builtin_inff();
    const T none = -(T)__builtin_inff();
    auto score = [&](float l) -> T {
        if constexpr (EXACT) return a.sigmoid ? sigmoid64((double)l) : exp64((double)l - of.high) * reciprocal(of.total);
        else return a.sigmoid ? sigmoid32(l) : exp32(l - (float)of.high) * __builtin_amdgcn_rcpf((float)of.total);
    };
    auto near = [&](T high, T low) {
        const T size = low < 0 ? -low : low;
        return !EXACT && !(high - low > (T)4e-6 * (size > 1 ? size : (T)1));
    };
    // key: the rank key rounded to fp32, as an integer in its order, 0 for a
    // masked expert; val: the key (a score, or its group's share)
    uint32_t key[V];
    T val[V];
    int idx[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 64 + lane;
        idx[i] = e;
        val[i] = (T)x[i];
        if (WIDE || GROUPS == 2) {
            val[i] = score(x[i]);
            if (WIDE && e < a.E) val[i] += (T)a.bias[e];
        }
        const bool live = x[i] != masked && val[i] == val[i] && val[i] != none;
        key[i] = live ? ordered(WIDE ? (float)val[i] : x[i]) : 0;
        if (GROUPS) values[e] = live ? val[i] : none;
    }
    if (GROUPS) {
        // `share` lanes read a group's values (one wave wrote them: no
        // barrier, only the order of its own LDS accesses)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        auto larger = [](T p, T q) { return p > q ? p : q; };
        auto smaller = [](T p, T q) { return p > q ? q : p; };
        T b1 = none, b2 = none;
        const int share = a.n_group <= 8 ? 8 : a.n_group <= 16 ? 4 : a.n_group <= 32 ? 2 : 1;
        const int mine = lane / share;
        if (mine < a.n_group) {
            const T* g = values + mine * a.gsize;
            for (int j = lane & (share - 1); j < a.gsize; j += share) {
                const T v = g[j];
                if (GROUPS == 2) b2 = larger(b2, smaller(b1, v));
                b1 = larger(b1, v);
            }
        }
        auto merge = [&](T o1, T o2) {
            if (GROUPS == 2) b2 = larger(smaller(b1, o1), larger(b2, o2));
            b1 = larger(b1, o1);
        };
        if (share >= 2) merge(dpp<SWAP1, 0xF>(none, b1), dpp<SWAP1, 0xF>(none, b2));
        if (share >= 4) merge(dpp<SWAP2, 0xF>(none, b1), dpp<SWAP2, 0xF>(none, b2));
        if (share >= 8) merge(dpp<HALF_MIRROR, 0xF>(none, b1), dpp<HALF_MIRROR, 0xF>(none, b2));
        T sum = GROUPS == 2 && b2 != none ? b1 + b2 : b1;
        // (two keys near the ends of fp32 have a sum outside it, which is still above that of a dead group)
        const T most = (T)3.402823466e38f;
        if (!EXACT && b1 != none) sum = larger(-most, smaller(most, sum));
        int ahead = 0;        // groups before this one
        for (int j = 0; j < a.n_group; ++j) {
            const T other = read_lane(sum, j * share);
            ahead += other > sum || (other == sum && j < mine);
        }
        const uint64_t kept = __ballot(mine < a.n_group && ahead < a.keep);
        if (!EXACT && (WIDE || GROUPS == 2)) {
            // Every kept group has to be above every dropped one by more than
            // what both may be off by.  That goes with the keys, which may
            // cancel in the sum: 1e-6 max(1, |key|) each, and the roundings of
            // the sum and of the two lines below, 2^-24 of it each.  (At the
            // ends of fp32 the bounds are infinite: not sure.)  The least
            // bound of the kept ones as integers, by its complement.
            auto size = [](T key) { return key > 1 ? key : key < -1 ? -key : (T)1; };
            T off = (T)1.5e-6 * size(b1);
            if (GROUPS == 2 && b2 != none) off += (T)1.5e-6 * size(b2);
            const bool in = kept >> lane & 1, dropped = !in && mine < a.n_group && b1 != none;
            const uint32_t low = ~wave_max(in ? ~ordered((float)(sum - off)) : 0);
            const uint32_t best = wave_max(dropped ? ordered((float)(sum + off)) : 0);
            if (low <= best) sure = false;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t e = i * 64 + lane;
            const uint32_t g = a.gsize > 1 ? __umulhi(e, a.gmagic) : e;
            if (!(kept >> (g * share & 63) & 1)) key[i] = 0;
        }
    }
    // lists in descending order, equal keys by index (neighbours change places
    // only where the later one is larger)
    constexpr bool BY_VAL = WIDE && EXACT;   // the rounded keys alone do not decide
    if (SORT) {
#pragma unroll
        for (int phase = 0; phase < V; ++phase)
#pragma unroll
            for (int i = phase & 1; i + 1 < V; i += 2) {
                const uint32_t k0 = key[i], k1 = key[i + 1];
                const T v0 = val[i], v1 = val[i + 1];
                const int i0 = idx[i], i1 = idx[i + 1];
                const bool swap = k1 > k0 || (BY_VAL && k1 == k0 && k1 != 0 && v1 > v0);
                key[i] = swap ? k1 : k0;
                key[i + 1] = swap ? k0 : k1;
                if (BY_VAL) {
                    val[i] = swap ? v1 : v0;
                    val[i + 1] = swap ? v0 : v1;
                }
                idx[i] = swap ? i1 : i0;
                idx[i + 1] = swap ? i0 : i1;
            }
    }

    int my_id = -1;
    T before = -none;
    // (32-bit keys: one round more, whose key only has to be far enough below)
    const int rounds = WIDE && !EXACT ? a.k + 1 : a.k;
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = key[0];
        T best_val = val[0];
        int e = idx[0];
        if (!SORT) {
#pragma unroll
            for (int i = 1; i < V; ++i)
                if (key[i] > best || (BY_VAL && key[i] == best && val[i] > best_val)) {
                    best = key[i];
                    best_val = val[i];
                    e = idx[i];
                }
        }
        const uint32_t top = wave_max(best);
        if (top == 0) break;  // nothing live is left
        if (WIDE && !EXACT) {
            const T t = (T)from_ordered(top);
            if (near(before, t)) sure = false;
            before = t;
            if (!sure || j == a.k) break;
        }
        uint64_t who = __ballot(best == top);
        if (who & (who - 1)) {
            // several: by the 64-bit keys, then the lowest index
            bool in = best == top;
            if (BY_VAL) {
                T m = in ? best_val : none;
#pragma unroll
                for (int o = 32; o >= 1; o >>= 1) {
                    const T other = __shfl_xor(m, o);
                    m = other > m ? other : m;
                }
                in = in && best_val == m;
            }
            int low = in ? e : MAX_E;
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) low = min(low, __shfl_xor(low, o));
            who = __ballot(in && e == low);
        }
        const int winner = __builtin_ctzll(who);
        const int chosen = __builtin_amdgcn_readlane(e, winner);
        if (lane == j) my_id = chosen;
        if (SORT) {
            // the winner's list moves up
#pragma unroll
            for (int i = 0; i < V; ++i) {
                key[i] = lane == winner ? (i + 1 < V ? key[i + 1] : 0) : key[i];
                if (i + 1 < V) {
                    idx[i] = lane == winner ? idx[i + 1] : idx[i];
                    if (BY_VAL) val[i] = lane == winner ? val[i + 1] : val[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (idx[i] == chosen) key[i] = 0;
        }
    }
    return my_id;
}

template <int V, bool WIDE, int GROUPS>
__global__ __launch_bounds__(64 * WAVES) void route_kernel(RouteArgs a)
{
    __shared__ double values[GROUPS ? WAVES : 1][GROUPS ? 64 * V : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = (int64_t)blockIdx.x * WAVES + wave;
    if (row >= a.M) return;   // (whole waves; no workgroup barrier below)

    float x[V];
    const float masked = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 64 + lane;
        float v = e < a.E ? load_logit(a, row * a.E + e) : masked;
        v = v != v ? masked : v;
        x[i] = fminf(v, 3.402823466e38f);
    }
    constexpr bool COMPUTED = WIDE || GROUPS == 2;
    Row of{0.0, 1.0};
    if (!a.sigmoid && (COMPUTED || !a.renormalize)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, ordered(x[i]));
        const float top = from_ordered(wave_max(m));
        of.high = top == masked ? 0.0 : (double)top;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) s += exp64((double)x[i] - of.high);
        of.total = wave_sum(s);
        if (of.total == 0.0) of.total = 1.0;   // nothing live
    }
    bool sure = true;
    int my_id = 0;
    if (COMPUTED) my_id = choose<V, WIDE, GROUPS>(a, row, x, of, reinterpret_cast<float*>(values[GROUPS ? wave : 0]), sure);
    if (!COMPUTED || !sure) my_id = choose<V, WIDE, GROUPS>(a, row, x, of, values[GROUPS ? wave : 0], sure);

    // gates of the chosen, in 64 bits.  Renormalised softmax scores depend on
    // the chosen logits alone, taken against the largest of them, so that the
    // chosen ones do not underflow beside a logit that no group kept.
    const bool live = my_id >= 0;
    float my_x = masked;
    if (live) my_x = fminf(load_logit(a, row * a.E + my_id), 3.402823466e38f);
    double g = 0.0;
    if (a.renormalize && !a.sigmoid) {
        const float top = from_ordered(wave_max(ordered(my_x)));
        g = live ? exp64((double)my_x - (double)top) : 0.0;
    } else if (live) {
        g = a.sigmoid ? sigmoid64((double)my_x) : exp64((double)my_x - of.high) * reciprocal(of.total);
    }
    if (a.renormalize) {
        const double s = wave_sum(g);
        g = s > 0.0 ? g / s : 0.0;
    }
    if (lane < a.k) {
        a.ids[row * a.k + lane] = my_id;
        a.gates[row * a.k + lane] = (float)(g * (double)a.scale);
    }
}

template <int V>
hipError_t launch_v(const RouteArgs& a, hipStream_t stream)
{
    const unsigned blocks = (unsigned)((a.M + WAVES - 1) / WAVES);
    const int groups = a.n_group > 1 ? a.top : 0;
    const bool wide = a.bias != nullptr;
#define APEX4_ROUTE(W, G)                                                            \
    if (wide == W && groups == G) {                                                  \
        route_kernel<V, W, G><<<blocks, 64 * WAVES, 0, stream>>>(a);                 \
        return hipGetLastError();                                                    \
    }
    APEX4_ROUTE(false, 0) APEX4_ROUTE(false, 1) APEX4_ROUTE(false, 2)
    APEX4_ROUTE(true, 0) APEX4_ROUTE(true, 1) APEX4_ROUTE(true, 2)
#undef APEX4_ROUTE
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_route(const RouteProblem& p, hipStream_t stream)
{
    RouteArgs a{};
    a.logits = p.logits;
    a.bias = p.bias;
    a.M = p.M;
    a.E = p.E;
    a.k = p.k;
    a.type = p.type;
    a.n_group = p.n_group;
    a.gsize = p.E / p.n_group;
    a.keep = p.keep;
    a.top = p.top;
    a.gmagic = (uint32_t)((1ull << 32) / a.gsize + 1);
    a.sigmoid = p.sigmoid;
    a.renormalize = p.renormalize;
    a.scale = p.scale;
    a.ids = p.ids;
    a.gates = p.gates;
    if (p.E <= 64) return launch_v<1>(a, stream);
    if (p.E <= 128) return launch_v<2>(a, stream);
    if (p.E <= 256) return launch_v<4>(a, stream);
    if (p.E <= 512) return launch_v<8>(a, stream);
    return launch_v<16>(a, stream);
}

}  // namespace apex4
