// Attention over the 4-bit key/value cache (include/apex4.h:
// apex4_kv4_attention), one wave a query head.
#include <climits>

#include "attention.h"
#include "rotary.h"

namespace apex4 {
namespace {

template <bool BF16, int D>
__global__ __launch_bounds__(64) void row_kernel(Kv4AttentionProblem p, int rows)
{
    __shared__ float qs[D];
    __shared__ float ps[64];
    const int lane = threadIdx.x;
    const int row0 = blockIdx.x % rows, h = blockIdx.x / rows % p.Hq, b = blockIdx.x / rows / p.Hq;
    const Kv4Cache& c = p.cache;
    int64_t q0 = b, q1 = b + 1;
    if (p.cu_q) {
        q0 = max(0, p.cu_q[b]);
        q1 = min(p.T, (int64_t)p.cu_q[b + 1]);
    }
    const int64_t len = q1 - q0;
    const int64_t kv = min((int64_t)max(0, p.kv_lens[b]), p.cols << c.shift);
    const int g = h / (p.Hq / c.Hkv);
    for (int64_t i = row0; i < len; i += rows) {
        const int64_t at = ((q0 + i) * p.Hq + h) * D;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + (q0 + i) * p.ldq + (int64_t)h * D;
        __syncthreads();
        for (int d = lane; d < D; d += 64) qs[d] = e4m3::from16<BF16>(q[d]) * p.scale;
        __syncthreads();
        const int64_t pos = kv - len + i;
        const int64_t hi = p.causal ? min(kv, pos + 1) : kv;
        const int64_t lo = p.window ? max((int64_t)0, pos - p.window + 1) : 0;
        float m = -INFINITY, l = 0.0f, acc[D / 64] = {};
        for (int64_t t0 = lo & ~63ll; t0 < hi; t0 += 64) {
            const int64_t t = t0 + lane;
            const int64_t pg = t < kv ? p.table[b * p.cols + (t >> c.shift)] : -1;
            const bool seen = t >= lo && t < hi && pg >= 0 && pg < c.pages;
            float s = -INFINITY, vs = 0.0f;
            if (seen) {
                const int64_t r = ((pg * c.Hkv + g) << c.shift) + (t & (c.page - 1));
                const uint8_t* k = c.k_codes + r * (D / 2);
                float dot = 0.0f;
                for (int d = 0; d < D / 2; ++d) {
                    dot = fmaf(qs[2 * d], (float)((int)(k[d] & 15) - 8), dot);
                    dot = fmaf(qs[2 * d + 1], (float)((int)(k[d] >> 4) - 8), dot);
                }
                s = dot * c.k_scales[r];
                vs = c.v_scales[r];
            }
            float top = s;
            for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            const float next = fmaxf(m, top);
            const float from = next == -INFINITY ? 0.0f : next, old = expf(m - from);
            const float w = seen ? expf(s - from) : 0.0f;
            float sum = w;
            for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
            l = l * old + sum;
            m = next;
            __syncthreads();
            ps[lane] = seen ? w * vs : 0.0f;
            __syncthreads();
            for (int e = 0; e < D / 64; ++e) acc[e] *= old;
            for (int k = 0; k < 64; ++k) {
                const int64_t tk = t0 + k;
                if (tk < lo || tk >= hi) continue;
                const int64_t pk = p.table[b * p.cols + (tk >> c.shift)];
                if (pk < 0 || pk >= c.pages) continue;
                const int off = (int)(tk & (c.page - 1));
                const uint8_t* v = c.v_codes + (pk * c.Hkv + g) * c.page * (D / 2) + (off >> 4) * 8 * D;
                for (int e = 0; e < D / 64; ++e) {
                    const int d = lane + 64 * e;
                    const int by = v[(((off >> 2) & 3) * 16 + d % 16) * (D / 8) + d / 32 * 4 + (off & 3)];
                    acc[e] = fmaf(ps[k], (float)(((d & 16 ? by >> 4 : by) & 15) - 8), acc[e]);
                }
            }
        }
        for (int e = 0; e < D / 64; ++e)
            static_cast<uint16_t*>(p.out)[at + lane + 64 * e] = e4m3::to16<BF16>(l == 0.0f ? 0.0f : acc[e] / l);
        if (p.lse && lane == 0) p.lse[(q0 + i) * p.Hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
    }
}

template <bool BF16>
hipError_t rows(const Kv4AttentionProblem& p, hipStream_t stream)
{
    const unsigned blocks = (unsigned)((int64_t)p.B * p.Hq * p.max_q);
    switch (p.cache.D) {
    case 64: row_kernel<BF16, 64><<<blocks, 64, 0, stream>>>(p, p.max_q); break;
    case 128: row_kernel<BF16, 128><<<blocks, 64, 0, stream>>>(p, p.max_q); break;
    default: row_kernel<BF16, 256><<<blocks, 64, 0, stream>>>(p, p.max_q); break;
    }
    return hipGetLastError();
}

}  // namespace

size_t kv4_attention_workspace_bytes(const Kv4AttentionProblem&) { return 0; }

hipError_t launch_kv4_attention(const Kv4AttentionProblem& p, hipStream_t stream)
{
    return p.bf16 ? rows<true>(p, stream) : rows<false>(p, stream);
}

}  // namespace apex4
