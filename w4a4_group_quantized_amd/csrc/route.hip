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
// What bounds it: a wave holds its row in registers (E / 64 values a lane)
// and reads it once; the k rounds of "largest key of the wave" are the time.
// Each round is one 6-step butterfly on the key alone: the lane that holds it
// comes from a ballot, and only a tie takes a second butterfly on the index.
#include "internal.h"

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

// integers in the order of the numbers, 0 for none of them
__device__ inline uint32_t ordered(float x)
{
    x += 0.0f;                // -0 ranks as 0
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ inline uint64_t ordered(double x)
{
    x += 0.0;
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

template <typename T>
__device__ inline T wave_max(T v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const T w = __shfl_xor(v, o);
        v = w > v ? w : v;
    }
    return v;
}

__device__ inline double wave_sum(double v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// V: values per lane (E <= 64 V).  WIDE: ranks by computed 64-bit keys (a
// bias), else by the logits.  GROUPS: 0 none, 1 a group's score is its best
// rank key's value, 2 the sum of its two best.
template <int V, bool WIDE, int GROUPS>
__global__ __launch_bounds__(64 * WAVES) void route_kernel(RouteArgs a)
{
    typedef typename std::conditional<WIDE, uint64_t, uint32_t>::type Key;
    __shared__ double values[GROUPS ? WAVES : 1][GROUPS ? 64 * V : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = (int64_t)blockIdx.x * WAVES + wave;
    if (row >= a.M) return;   // (whole waves; no workgroup barrier below)

    float x[V];
    Key key[V];
    const float masked = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 64 + lane;
        float v = e < a.E ? load_logit(a, row * a.E + e) : masked;
        v = v != v ? masked : v;
        x[i] = fminf(v, 3.402823466e38f);
    }
    // row maximum and sum of exponentials, where a score needs them
    double high = 0.0, total = 1.0;
    const bool all_scores = WIDE || GROUPS == 2;
    if (!a.sigmoid && (all_scores || !a.renormalize)) {
        float m = masked;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
        m = wave_max(m);
        high = m == masked ? 0.0 : (double)m;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) s += exp((double)x[i] - high);
        total = wave_sum(s);
        if (total == 0.0) total = 1.0;   // nothing live
    }
    auto score = [&](float l) { return a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - high) / total; };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 64 + lane;
        double val = (double)x[i];
        if (all_scores) {
            val = score(x[i]);
            if (WIDE && e < a.E) val += (double)a.bias[e];
        }
        const bool live = x[i] != masked && val == val && val != -__builtin_inf();
        if constexpr (WIDE) key[i] = live ? ordered(val) : 0;
        else key[i] = live ? ordered(x[i]) : 0;
        if (GROUPS) values[wave][e] = live ? val : -__builtin_inf();
    }
    if (GROUPS) {
        // lane g reads group g's values (one wave wrote them: no barrier,
        // only the order of its own LDS accesses)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const double none = -__builtin_inf();
        double b1 = none, b2 = none;
        if (lane < a.n_group) {
            const double* g = values[wave] + lane * a.gsize;
            for (int j = 0; j < a.gsize; ++j) {
                const double v = g[j];
                if (GROUPS == 2) b2 = v > b1 ? b1 : v > b2 ? v : b2;
                b1 = v > b1 ? v : b1;
            }
        }
        const double mine = GROUPS == 2 && b2 != none ? b1 + b2 : b1;
        int ahead = 0;        // groups before this one
        for (int j = 0; j < a.n_group; ++j) {
            const double other = __shfl(mine, j);
            ahead += other > mine || (other == mine && j < lane);
        }
        const uint64_t kept = __ballot(lane < a.n_group && ahead < a.keep);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t e = i * 64 + lane;
            const uint32_t g = __umulhi(e, a.gmagic);
            if (a.gsize > 1 ? !(kept >> (g & 63) & 1) : !(kept >> (e & 63) & 1)) key[i] = 0;
        }
    }

    int my_id = -1;           // lane j: the j-th choice
    float my_x = masked;
    for (int j = 0; j < a.k; ++j) {
        Key best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const Key top = wave_max(best);
        if (top == 0) break;  // nothing live is left
        const bool have = best == top;
        const uint64_t who = __ballot(have);
        int e = at * 64 + lane;
        if ((who & (who - 1)) == 0) {
            e = __shfl(e, __ffsll((unsigned long long)who) - 1);
        } else {
            // a tie: the lowest index
            int low = have ? e : MAX_E;
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) low = min(low, __shfl_xor(low, o));
            e = low;
        }
        float l = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i == e >> 6) {
                l = x[i];
                if (lane == (e & 63)) key[i] = 0;
            }
        l = __shfl(l, e & 63);
        if (lane == j) {
            my_id = e;
            my_x = l;
        }
    }

    // gates of the chosen, in 64 bits.  Renormalised softmax scores depend on
    // the chosen logits alone, taken against the largest of them, so that the
    // chosen ones do not underflow beside a logit that no group kept.
    const bool live = my_id >= 0;
    double g = 0.0;
    if (a.renormalize && !a.sigmoid) {
        const float m = wave_max(my_x);
        g = live ? exp((double)my_x - (double)m) : 0.0;
    } else if (live) {
        g = score(my_x);
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
