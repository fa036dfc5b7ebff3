// C ABI of the rotary, cache and attention calls (include/apex4.h: apex4_rope
// and the kv4 calls): host-side argument checks, then the launch on the
// caller's stream.  Every check runs before anything is launched.
#include "apex4.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxTokens = (int64_t(1) << 24) - 1;      // a launch has fewer than 2^32 threads
constexpr int64_t kMaxStride = int64_t(1) << 32;
constexpr int32_t kMaxHeads = 1024;

apex4_status to_status(hipError_t e) { return e == hipSuccess ? APEX4_OK : APEX4_ERR_HIP; }

bool half_type(int32_t t) { return t == APEX4_F16 || t == APEX4_BF16; }

bool heads_ok(int64_t T, int32_t H) { return T >= 0 && T <= kMaxTokens && H >= 1 && H <= kMaxHeads; }

// rows of `H` heads of `D` numbers, `ld` apart
bool stride_ok(int64_t ld, int32_t H, int32_t D) { return ld >= (int64_t)H * D && ld < kMaxStride; }

bool rotation_ok(int32_t R, int32_t D, double scale)
{
    return R >= 16 && R <= D && R % 16 == 0 && std::isfinite(scale);
}

bool head_dim_ok(int32_t D) { return D == 64 || D == 128 || D == 256; }

bool page_ok(int32_t page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }

// sizes of a cache: APEX4_OK, or what refuses them
apex4_status cache_sizes(int64_t pages, int32_t page, int32_t Hkv, int32_t D)
{
    if (pages < 1 || pages >= (int64_t(1) << 31) || page < 1 || Hkv < 1 || Hkv > kMaxHeads || D < 1)
        return APEX4_ERR_INVALID_ARG;
    return head_dim_ok(D) && page_ok(page) ? APEX4_OK : APEX4_ERR_UNSUPPORTED;
}

apex4::Kv4Cache make_cache(const void* k_codes, const float* k_scales, const void* v_codes, const float* v_scales,
                           int64_t pages, int32_t page, int32_t Hkv, int32_t D)
{
    apex4::Kv4Cache c{};
    c.k_codes = static_cast<uint8_t*>(const_cast<void*>(k_codes));
    c.k_scales = const_cast<float*>(k_scales);
    c.v_codes = static_cast<uint8_t*>(const_cast<void*>(v_codes));
    c.v_scales = const_cast<float*>(v_scales);
    c.pages = pages;
    c.Hkv = Hkv;
    c.D = D;
    c.page = page;
    while ((1 << c.shift) < page) ++c.shift;
    return c;
}

bool cache_given(const apex4::Kv4Cache& c) { return c.k_codes && c.k_scales && c.v_codes && c.v_scales; }

bool cache_aligned(const apex4::Kv4Cache& c)
{
    return aligned(c.k_codes, 16) && aligned(c.k_scales, 16) && aligned(c.v_codes, 16) && aligned(c.v_scales, 16);
}

// sizes of an attention call (T or B may be 0)
apex4_status attention_sizes(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q, int32_t max_kv)
{
    if (!heads_ok(T, Hq) || B < 0 || B > 65536 || Hkv < 1 || Hq % Hkv != 0 || D < 1) return APEX4_ERR_INVALID_ARG;
    if (T * Hq >= (int64_t(1) << 30) || (int64_t)B * Hkv >= (int64_t(1) << 23) || max_q < 1 || max_kv < 1)
        return APEX4_ERR_INVALID_ARG;
    return head_dim_ok(D) ? APEX4_OK : APEX4_ERR_UNSUPPORTED;
}

apex4::Kv4AttentionProblem attention_problem(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q,
                                             int32_t max_kv)
{
    apex4::Kv4AttentionProblem p{};
    p.T = T;
    p.B = B;
    p.Hq = Hq;
    p.share = Hq / Hkv;
    p.cache.Hkv = Hkv;
    p.cache.D = D;
    // (no fewer than the mean, no more than there are)
    const int64_t mean = B > 0 ? (T + B - 1) / B : 1;
    p.max_q = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(std::max<int64_t>(max_q, mean), T)));
    p.max_kv = std::min(max_kv, 1 << 30);
    return p;
}

}  // namespace

extern "C" {

apex4_status apex4_rope(const void* x, int32_t type, int64_t T, int32_t H, int32_t D, int64_t ldx,
                        const int64_t* positions, const double* freqs, int32_t R, int32_t interleaved, double scale,
                        void* y, int64_t ldy, void* stream)
{
    if (!heads_ok(T, H) || D < 16 || D > 1024 || D % 16 != 0 || !rotation_ok(R, D, scale) || !stride_ok(ldx, H, D) ||
        !stride_ok(ldy, H, D))
        return APEX4_ERR_INVALID_ARG;
    if (type != APEX4_F32 && !half_type(type)) return APEX4_ERR_UNSUPPORTED;
    if (T == 0) return APEX4_OK;
    if (!x || !positions || !freqs || !y) return APEX4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(positions, 8) || !aligned(freqs, 8) || ldx % 8 || ldy % 8)
        return APEX4_ERR_ALIGNMENT;
    apex4::RopeProblem p{};
    p.x = x;
    p.type = type;
    p.T = T;
    p.H = H;
    p.D = D;
    p.ldx = ldx;
    p.turn = {positions, freqs, R, interleaved != 0, scale};
    p.y = y;
    p.ldy = ldy;
    return to_status(apex4::launch_rope(p, static_cast<hipStream_t>(stream)));
}

apex4_status apex4_kv4_append(const void* q, const void* k, const void* v, int32_t type, int64_t T, int32_t Hq,
                              int32_t Hkv, int32_t D, int64_t ldq, int64_t ldk, int64_t ldv,
                              const int64_t* positions, const double* freqs, int32_t R, int32_t interleaved,
                              double scale, const int64_t* slots, int64_t pages, int32_t page, void* k_codes,
                              float* k_scales, void* v_codes, float* v_scales, void* q_out, void* stream)
{
    const apex4_status sizes = cache_sizes(pages, page, Hkv, D);
    if (sizes != APEX4_OK) return sizes;
    if (T < 0 || T > kMaxTokens || Hq < 0 || Hq > kMaxHeads || !stride_ok(ldk, Hkv, D) || !stride_ok(ldv, Hkv, D))
        return APEX4_ERR_INVALID_ARG;
    if (R != 0 && !rotation_ok(R, D, scale)) return APEX4_ERR_INVALID_ARG;
    if (Hq > 0 && (R == 0 || !stride_ok(ldq, Hq, D))) return APEX4_ERR_INVALID_ARG;
    if (!half_type(type)) return APEX4_ERR_UNSUPPORTED;
    if (T == 0) return APEX4_OK;
    const apex4::Kv4Cache c = make_cache(k_codes, k_scales, v_codes, v_scales, pages, page, Hkv, D);
    if (!k || !v || !slots || !cache_given(c)) return APEX4_ERR_INVALID_ARG;
    if ((R != 0) != (positions != nullptr) || (R != 0) != (freqs != nullptr)) return APEX4_ERR_INVALID_ARG;
    if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr)) return APEX4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(slots, 8) ||
        !aligned(positions, 8) || !aligned(freqs, 8) || !cache_aligned(c) || (Hq > 0 && ldq % 8) || ldk % 8 || ldv % 8)
        return APEX4_ERR_ALIGNMENT;
    apex4::Kv4AppendProblem p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.bf16 = type == APEX4_BF16;
    p.T = T;
    p.Hq = Hq;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.turn = {positions, freqs, R, interleaved != 0, scale};
    p.slots = slots;
    p.cache = c;
    p.q_out = q_out;
    return to_status(apex4::launch_kv4_append(p, static_cast<hipStream_t>(stream)));
}

apex4_status apex4_kv4_read(const void* k_codes, const float* k_scales, const void* v_codes, const float* v_scales,
                            int64_t pages, int32_t page, int32_t Hkv, int32_t D, const int64_t* slots, int64_t T,
                            int32_t type, void* k, void* v, void* stream)
{
    const apex4_status sizes = cache_sizes(pages, page, Hkv, D);
    if (sizes != APEX4_OK) return sizes;
    if (T < 0 || T > kMaxTokens || T * Hkv >= (int64_t(1) << 28)) return APEX4_ERR_INVALID_ARG;
    if (type != APEX4_F32 && !half_type(type)) return APEX4_ERR_UNSUPPORTED;
    if (T == 0) return APEX4_OK;
    apex4::Kv4ReadProblem p{};
    p.cache = make_cache(k_codes, k_scales, v_codes, v_scales, pages, page, Hkv, D);
    if (!cache_given(p.cache) || !slots || !k || !v) return APEX4_ERR_INVALID_ARG;
    if (!cache_aligned(p.cache) || !aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return APEX4_ERR_ALIGNMENT;
    p.slots = slots;
    p.T = T;
    p.type = type;
    p.k = k;
    p.v = v;
    return to_status(apex4::launch_kv4_read(p, static_cast<hipStream_t>(stream)));
}

size_t apex4_kv4_attention_workspace_size(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q,
                                          int32_t max_kv)
{
    if (attention_sizes(T, B, Hq, Hkv, D, max_q, max_kv) != APEX4_OK || T == 0 || B == 0) return 0;
    return apex4::kv4_attention_workspace_bytes(attention_problem(T, B, Hq, Hkv, D, max_q, max_kv));
}

apex4_status apex4_kv4_attention(const void* q, int32_t type, int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                 int64_t ldq, const int32_t* cu_q, const int32_t* kv_lens, const int32_t* table,
                                 int64_t cols, const void* k_codes, const float* k_scales, const void* v_codes,
                                 const float* v_scales, int64_t pages, int32_t page, float scale, int32_t causal,
                                 int32_t window, int32_t max_q, int32_t max_kv, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream)
{
    apex4_status st = attention_sizes(T, B, Hq, Hkv, D, max_q, max_kv);
    if (st == APEX4_OK) st = cache_sizes(pages, page, Hkv, D);
    if (st != APEX4_OK) return st;
    if (!stride_ok(ldq, Hq, D) || cols < 1 || cols > (int64_t(1) << 30) / page || !std::isfinite(scale))
        return APEX4_ERR_INVALID_ARG;
    if (window < 0 || (window > 0 && !causal) || (!cu_q && T != B)) return APEX4_ERR_INVALID_ARG;
    if (!half_type(type)) return APEX4_ERR_UNSUPPORTED;
    const size_t need = apex4_kv4_attention_workspace_size(T, B, Hq, Hkv, D, max_q, max_kv);
    if (workspace_bytes < need || (need > 0 && !workspace)) return APEX4_ERR_WORKSPACE;
    if (T == 0 || B == 0) return APEX4_OK;
    apex4::Kv4AttentionProblem p = attention_problem(T, B, Hq, Hkv, D, max_q, max_kv);
    p.cache = make_cache(k_codes, k_scales, v_codes, v_scales, pages, page, Hkv, D);
    if (!q || !kv_lens || !table || !o || !cache_given(p.cache)) return APEX4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) ||
        !aligned(table, 4) || !cache_aligned(p.cache) || !aligned(workspace, 16) || ldq % 8)
        return APEX4_ERR_ALIGNMENT;
    p.q = q;
    p.bf16 = type == APEX4_BF16;
    p.ldq = ldq;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.table = table;
    p.cols = cols;
    p.scale = scale;
    p.causal = causal != 0;
    p.window = std::min(window, 1 << 30);      // (all tokens; positions less a window stay within 32 bits)
    p.out = o;
    p.lse = lse;
    p.ws = workspace;
    return to_status(apex4::launch_kv4_attention(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
