// The experts' W4A4 feed-forward network over routed tokens on gfx950.
//
//     g, u = W4A4(x_m, gate_up_e);  h = f16(silu(g) u);  d = W4A4(h, down_e);
//     y_m = sum_j gates[m, j] d_(m, j)        for the slots (m, j), e = ids[m, j]
//
// Slots are put in the order of their experts once (plan_kernel: the sorted
// row of every slot and the first row of every expert), the activation codes
// are quantized per token, and the products run per expert over its rows.
#include "experts.h"
#include "layers.h"
#include "quant_rule.h"

namespace apex4 {
namespace {

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// The workspace, in this order.
struct Parts {
    int32_t* offsets;    // [E + 1] first sorted row of every expert; [E]: the live rows
    int32_t* order;      // [R] slot of a sorted row (rows past offsets[E]: unset)
    int32_t* place;      // [R] sorted row of a slot, -1 for a slot without an expert
    uint8_t* xq;         // [M, H/2] codes of x
    float* xs;           // [M, H/128]
    _Float16* h;         // [R, I]
    uint8_t* hq;         // [R, I/2]
    float* hs;           // [R, I/128]
    float* d;            // [parts, R, H], the down product's K parts
    int parts;
    size_t bytes;
};

Parts parts_of(void* ws, int64_t M, int32_t k, int32_t E, int32_t H, int32_t I)
{
    const int64_t R = M * k;
    uint8_t* p = static_cast<uint8_t*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t* q = p + at;
        at += align256(bytes);
        return q;
    };
    Parts w;
    w.offsets = reinterpret_cast<int32_t*>(take((size_t)(E + 1) * 4));
    w.order = reinterpret_cast<int32_t*>(take((size_t)R * 4));
    w.place = reinterpret_cast<int32_t*>(take((size_t)R * 4));
    w.xq = take((size_t)M * (H / 2));
    w.xs = reinterpret_cast<float*>(take((size_t)M * (H / 128) * 4));
    w.h = reinterpret_cast<_Float16*>(take((size_t)R * I * 2));
    w.hq = take((size_t)R * (I / 2));
    w.hs = reinterpret_cast<float*>(take((size_t)R * (I / 128) * 4));
    w.parts = experts_parts(R, E, H, I);
    w.d = reinterpret_cast<float*>(take((size_t)w.parts * R * H * 4));
    w.bytes = at;
    return w;
}

// The slots in the order of their experts, and in slot order within one: a
// counting sort without a word between workgroups.  Workgroup e reads all R
// ids, counts those below e and those equal to e (its first row), and reads
// them again to place its own; the ids stay in L2.  Each wave takes a
// contiguous run of slots, so that only the waves' counts cross the barrier.
constexpr int PLAN_WAVES = 16;
constexpr int PLAN_READS = 8;   // ids a lane asks for together
// The workgroups past the experts quantize x meanwhile (the rule of
// apex4_quantize_act, a chunk of 8 values a thread).
__global__ __launch_bounds__(64 * PLAN_WAVES) void plan_kernel(const int32_t* __restrict__ ids, int32_t R, int32_t E,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ order,
                                                               int32_t* __restrict__ place,
                                                               const qrule::half8* __restrict__ x, int64_t n8,
                                                               uint32_t* __restrict__ xq, float* __restrict__ xs)
{
    __shared__ int below[PLAN_WAVES], equal[PLAN_WAVES];
    if (blockIdx.x >= E) {
        const int64_t t = (int64_t)(blockIdx.x - E) * (64 * PLAN_WAVES) + threadIdx.x;
        if (t >= n8) return;      // (whole groups of 16 lanes)
        const qrule::half8 v = x[t];
        const float scale = experts_scale(v);
        xq[t] = qrule::quantize8(v, scale, scale != 0.0f);
        if ((t & 15) == 0) xs[t / 16] = scale;
        return;
    }
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = ((R + PLAN_WAVES - 1) / PLAN_WAVES + 63) / 64 * 64;
    const int64_t first = (int64_t)wave * per;
    const int last = (int)min((int64_t)R, first + per);
    int lt = 0, eq = 0;
    for (int64_t s0 = first + lane; s0 < last; s0 += 64 * PLAN_READS) {
        int id[PLAN_READS];
#pragma unroll
        for (int i = 0; i < PLAN_READS; ++i) id[i] = ids[min(s0 + 64 * i, (int64_t)R - 1)];
#pragma unroll
        for (int i = 0; i < PLAN_READS; ++i) {
            const int64_t s = s0 + 64 * i;
            const bool in = s < last;
            lt += in && id[i] >= 0 && id[i] < e;
            eq += in && id[i] == e;
            // slots without an expert: one workgroup says so
            if (in && e == 0 && (id[i] < 0 || id[i] >= E)) place[s] = -1;
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        lt += __shfl_xor(lt, o);
        eq += __shfl_xor(eq, o);
    }
    if (lane == 0) {
        below[wave] = lt;
        equal[wave] = eq;
    }
    __syncthreads();
    int row = 0, count = 0;
    for (int w = 0; w < PLAN_WAVES; ++w) {
        row += below[w];
        if (w < wave) row += equal[w];
        count += equal[w];
    }
    if (threadIdx.x == 0) {
        offsets[e] = row;
        if (e == E - 1) offsets[E] = row + count;
    }
    if (equal[wave] == 0) return;
    for (int64_t s0 = first + lane; s0 - lane < last; s0 += 64 * PLAN_READS) {
        int id[PLAN_READS];
#pragma unroll
        for (int i = 0; i < PLAN_READS; ++i) id[i] = ids[min(s0 + 64 * i, (int64_t)R - 1)];
#pragma unroll
        for (int i = 0; i < PLAN_READS; ++i) {
            const int64_t s = s0 + 64 * i;
            const bool mine = s < last && id[i] == e;
            const uint64_t who = __ballot(mine);
            if (mine) {
                const int r = row + __popcll(who & ((1ull << lane) - 1));
                order[r] = (int)s;
                place[s] = r;
            }
            row += __popcll(who);
        }
    }
}

// h to codes and scales, a chunk of 8 values a thread (rows without a slot too: nothing reads them)
__global__ __launch_bounds__(256) void quantize_h_kernel(const qrule::half8* __restrict__ h, int64_t n8,
                                                         uint32_t* __restrict__ hq, float* __restrict__ hs)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= n8) return;          // (whole groups of 16 lanes)
    const qrule::half8 v = h[t];
    const float scale = experts_scale(v);
    hq[t] = qrule::quantize8(v, scale, scale != 0.0f);
    if ((t & 15) == 0) hs[t / 16] = scale;
}

// y = the sum of a token's slots, in slot order, of each slot's K parts, in
// their order; one rounding to fp16 at the end.
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ d, const int32_t* __restrict__ place,
                                                      const float* __restrict__ gates, int32_t k, int32_t H,
                                                      int32_t parts, int64_t part_stride,
                                                      int64_t n4, _Float16* __restrict__ y16, float* __restrict__ y32)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= n4) return;
    const int per = H / 4;
    const int64_t m = t / per;
    const int c = (int)(t - m * per) * 4;
    typedef float v4f __attribute__((ext_vector_type(4)));
    v4f s = {};
    // eight slots' rows at a time, so that their reads are under way together
    for (int j0 = 0; j0 < k; j0 += 8) {
        int r[8];
        float g[8];
        v4f v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = j0 + j < k ? place[m * k + j0 + j] : -1;
            g[j] = r[j] >= 0 ? gates[m * k + j0 + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = r[j] >= 0 ? *reinterpret_cast<const v4f*>(d + (int64_t)r[j] * H + c) : v4f{};
        for (int p = 1; p < parts; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r[j] >= 0) v[j] += *reinterpret_cast<const v4f*>(d + p * part_stride + (int64_t)r[j] * H + c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = fmaf(g[j], v[j][i], s[i]);
    }
    typedef _Float16 half4 __attribute__((ext_vector_type(4)));
    half4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = s[i];
        asm volatile("" : "+v"(v));   // y16 is the fp16 rounding of y32
        o[i] = (_Float16)v;
        if (y32) y32[m * H + c + i] = v;
    }
    *reinterpret_cast<half4*>(y16 + m * H + c) = o;
}

}  // namespace

size_t experts_workspace_bytes(int64_t M, int32_t k, int32_t E, int32_t H, int32_t I)
{
    return parts_of(nullptr, M, k, E, H, I).bytes;
}

hipError_t launch_experts(const ExpertsProblem& p, hipStream_t stream)
{
    const Parts w = parts_of(p.ws, p.M, p.k, p.E, p.H, p.I);
    const int32_t R = (int32_t)(p.M * p.k);
    if (experts_token_supports(p)) return launch_experts_token(p, w.h, stream);
    const int64_t n8 = p.M * (p.H / 8);
    const unsigned chunks = (unsigned)((n8 + 64 * PLAN_WAVES - 1) / (64 * PLAN_WAVES));
    plan_kernel<<<p.E + chunks, 64 * PLAN_WAVES, 0, stream>>>(p.ids, R, p.E, w.offsets, w.order, w.place,
                                                              static_cast<const qrule::half8*>(p.x), n8,
                                                              reinterpret_cast<uint32_t*>(w.xq), w.xs);
    ExpertsProduct a{};
    a.offsets = w.offsets;
    a.order = w.order;
    a.k = p.k;
    a.E = p.E;
    a.qx = w.xq;
    a.sx = w.xs;
    a.qw = p.qw_gu;
    a.sw = p.s_gu;
    a.N = 2 * p.I;
    a.K = p.H;
    a.h = w.h;
    a.rows = p.M;
    a.parts = 1;
    launch_experts_tiled(a, true, R, stream);
    const int64_t h8 = (int64_t)R * (p.I / 8);
    quantize_h_kernel<<<(unsigned)((h8 + 255) / 256), 256, 0, stream>>>(
        reinterpret_cast<const qrule::half8*>(w.h), h8, reinterpret_cast<uint32_t*>(w.hq), w.hs);
    a.qx = w.hq;
    a.sx = w.hs;
    a.qw = p.qw_down;
    a.sw = p.s_down;
    a.N = p.H;
    a.K = p.I;
    a.d = w.d;
    a.parts = w.parts;
    a.part_stride = (int64_t)R * p.H;
    launch_experts_tiled(a, false, R, stream);
    const int64_t n4 = p.M * (p.H / 4);
    combine_kernel<<<(unsigned)((n4 + 255) / 256), 256, 0, stream>>>(w.d, w.place, p.gates, p.k, p.H, w.parts,
                                                                     (int64_t)R * p.H, n4,
                                                                     static_cast<_Float16*>(p.y16), p.y32);
    return hipGetLastError();
}

}  // namespace apex4
