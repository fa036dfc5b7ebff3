// C ABI of the sparse-layer and 8-bit calls (include/apex4.h: apex4_route,
// apex4_experts_w4a4 and the e4m3 calls): host-side argument checks, then the
// launch on the caller's stream.  Every check runs before anything is launched,
// so a rejected call touches neither the device's work nor the caller's memory
// (a workspace size asks the runtime which device is current).
#include "apex4.h"

#include <atomic>
#include <cmath>
#include <cstdint>

#include "layers.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// elements of one tensor and rows of one call: a launch has fewer than 2^32
// threads along a dimension (8 elements, or 64 threads a row)
constexpr uint64_t kMaxElements = uint64_t(1) << 34;
constexpr int64_t kMaxRows = int64_t(1) << 26;
constexpr int64_t kMaxTokens = int64_t(1) << 25;   // of apex4_route: 64 threads each, rounded up to four
// outputs of an 8-bit product: more do not fit the memory, and tiles are counted in 32 bits
constexpr uint64_t kMaxOutputs = uint64_t(1) << 37;

apex4_status to_status(hipError_t e) { return e == hipSuccess ? APEX4_OK : APEX4_ERR_HIP; }

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

bool half_type(int32_t t) { return t == APEX4_F16 || t == APEX4_BF16; }

// sizes of the experts' network that apex4_experts_w4a4 takes (M may be 0)
bool experts_sizes(int64_t M, int32_t k, int64_t E, int64_t H, int64_t I)
{
    if (M < 0 || M > kMaxDim || k < 1 || k > 64 || E < 1 || E > 1024) return false;
    if (H <= 0 || I <= 0 || H > kMaxDim || I > kMaxDim || H % 128 != 0 || I % 128 != 0) return false;
    const uint64_t lim = uint64_t(1) << 32;
    if (M * k > kMaxDim || (uint64_t)(M * k) * (uint64_t)I >= kMaxElements) return false;
    return 2 * (uint64_t)I * (uint64_t)H < lim && (uint64_t)(M + k) * (uint64_t)H < lim;
}

// sizes of an 8-bit product (M or N may be 0)
bool e4m3_sizes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || M > kMaxRows || N > kMaxRows || K <= 0 || K % 128 != 0 || K >= (int64_t(1) << 23)) return false;
    if ((uint64_t)M * N >= kMaxOutputs) return false;
    return (uint64_t)M * K < kMaxElements && (uint64_t)N * K < kMaxElements;
}

apex4::E4m3Problem e4m3_problem(int64_t M, int64_t N, int64_t K)
{
    apex4::E4m3Problem p{};
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    return p;
}

apex4_status check_e4m3_quantize(const void* x, int32_t type, int64_t rows, int64_t K, const void* q, const float* s)
{
    if (!e4m3_sizes(rows, 0, K)) return APEX4_ERR_INVALID_ARG;
    if (!half_type(type)) return APEX4_ERR_UNSUPPORTED;
    if (rows == 0) return APEX4_OK;
    if (!x || !q || !s) return APEX4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(q, 8) || !aligned(s, 4)) return APEX4_ERR_ALIGNMENT;
    return APEX4_OK;
}

}  // namespace

int apex4::compute_units()
{
    // cached per device (relaxed atomics: any thread may write the same value)
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0 && hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess)
        cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

extern "C" {

apex4_status apex4_route(const void* logits, int32_t logits_type, int64_t M, int64_t E, int32_t score,
                         const float* bias, int32_t n_group, int32_t topk_group, int32_t group_top, int32_t k,
                         int32_t renormalize, float scale, int32_t* ids, float* gates, void* stream)
{
    if (M < 0 || M > kMaxTokens || E < 1 || E > 1024 || k < 1 || k > 64) return APEX4_ERR_INVALID_ARG;
    if (n_group < 1 || n_group > 64 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
        return APEX4_ERR_INVALID_ARG;
    if (k > topk_group * (E / n_group) || (group_top != 1 && group_top != 2) || !std::isfinite(scale))
        return APEX4_ERR_INVALID_ARG;
    if (score != APEX4_SCORE_SOFTMAX && score != APEX4_SCORE_SIGMOID) return APEX4_ERR_INVALID_ARG;
    if (logits_type != APEX4_F32 && !half_type(logits_type)) return APEX4_ERR_UNSUPPORTED;
    if (M == 0) return APEX4_OK;
    if (!logits || !ids || !gates) return APEX4_ERR_INVALID_ARG;
    if (!aligned(logits, logits_type == APEX4_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) ||
        !aligned(gates, 4))
        return APEX4_ERR_ALIGNMENT;
    apex4::RouteProblem p{};
    p.logits = logits;
    p.type = logits_type;
    p.M = M;
    p.E = static_cast<int32_t>(E);
    p.k = k;
    p.sigmoid = score == APEX4_SCORE_SIGMOID;
    p.bias = bias;
    p.n_group = n_group;
    p.keep = topk_group;
    p.top = group_top;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    p.ids = ids;
    p.gates = gates;
    return to_status(apex4::launch_route(p, static_cast<hipStream_t>(stream)));
}

size_t apex4_experts_workspace_size(int64_t M, int32_t k, int64_t E, int64_t H, int64_t I, int32_t group)
{
    if (!experts_sizes(M, k, E, H, I) || group != 128 || M == 0) return 0;
    return apex4::experts_workspace_bytes(M, k, static_cast<int32_t>(E), static_cast<int32_t>(H),
                                          static_cast<int32_t>(I));
}

apex4_status apex4_experts_w4a4(const void* x_f16, const int32_t* ids, const float* gates, int64_t M, int32_t k,
                                int64_t E, int64_t H, int64_t I, int32_t group, const void* qw_gate_up,
                                const float* s_gate_up, const void* qw_down, const float* s_down, void* y_f16,
                                float* y_f32, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!experts_sizes(M, k, E, H, I) || group <= 0) return APEX4_ERR_INVALID_ARG;
    if (group != 128) return APEX4_ERR_UNSUPPORTED;
    const size_t need = apex4_experts_workspace_size(M, k, E, H, I, group);
    if (workspace_bytes < need || (need > 0 && !workspace)) return APEX4_ERR_WORKSPACE;
    if (M == 0) return APEX4_OK;
    if (!x_f16 || !ids || !gates || !qw_gate_up || !s_gate_up || !qw_down || !s_down || !y_f16)
        return APEX4_ERR_INVALID_ARG;
    if (!aligned(x_f16, 16) || !aligned(ids, 4) || !aligned(gates, 4) || !aligned(qw_gate_up, 16) ||
        !aligned(s_gate_up, 4) || !aligned(qw_down, 16) || !aligned(s_down, 4) || !aligned(y_f16, 16) ||
        !aligned(y_f32, 4) || !aligned(workspace, 256))
        return APEX4_ERR_ALIGNMENT;
    apex4::ExpertsProblem p{};
    p.x = x_f16;
    p.ids = ids;
    p.gates = gates;
    p.M = M;
    p.k = k;
    p.E = static_cast<int32_t>(E);
    p.H = static_cast<int32_t>(H);
    p.I = static_cast<int32_t>(I);
    p.qw_gu = static_cast<const uint8_t*>(qw_gate_up);
    p.s_gu = s_gate_up;
    p.qw_down = static_cast<const uint8_t*>(qw_down);
    p.s_down = s_down;
    p.y16 = y_f16;
    p.y32 = y_f32;
    p.ws = workspace;
    return to_status(apex4::launch_experts(p, static_cast<hipStream_t>(stream)));
}

apex4_status apex4_quantize_e4m3(const void* x, int32_t x_type, int64_t rows, int64_t K, void* q8, float* s,
                                 void* stream)
{
    const apex4_status st = check_e4m3_quantize(x, x_type, rows, K, q8, s);
    if (st != APEX4_OK || rows == 0) return st;
    return to_status(
        apex4::launch_quantize_e4m3(x, x_type == APEX4_BF16, rows, K, q8, s, static_cast<hipStream_t>(stream)));
}

apex4_status apex4_pack_weight_e4m3(const void* w, int32_t w_type, int64_t N, int64_t K, void* q8, float* s,
                                    void* stream)
{
    const apex4_status st = check_e4m3_quantize(w, w_type, N, K, q8, s);
    if (st != APEX4_OK || N == 0) return st;
    return to_status(
        apex4::launch_pack_e4m3(w, w_type == APEX4_BF16, N, K, q8, s, static_cast<hipStream_t>(stream)));
}

size_t apex4_gemm_e4m3_workspace_size(int64_t M, int64_t N, int64_t K)
{
    if (!e4m3_sizes(M, N, K) || M == 0 || N == 0) return 0;
    return apex4::e4m3_workspace_bytes(e4m3_problem(M, N, K));
}

apex4_status apex4_gemm_e4m3(const void* qa8, const float* s_a, const void* qw8, const float* s_w, int64_t M,
                             int64_t N, int64_t K, int32_t y_type, void* y, float* y_f32, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    if (!e4m3_sizes(M, N, K)) return APEX4_ERR_INVALID_ARG;
    if (!half_type(y_type)) return APEX4_ERR_UNSUPPORTED;
    const size_t need = apex4_gemm_e4m3_workspace_size(M, N, K);
    if (workspace_bytes < need || (need > 0 && !workspace)) return APEX4_ERR_WORKSPACE;
    if (M == 0 || N == 0) return APEX4_OK;
    if (!qa8 || !s_a || !qw8 || !s_w || !y) return APEX4_ERR_INVALID_ARG;
    if (!aligned(qa8, 16) || !aligned(s_a, 4) || !aligned(qw8, 16) || !aligned(s_w, 4) || !aligned(y, 2) ||
        !aligned(y_f32, 4) || !aligned(workspace, 16))
        return APEX4_ERR_ALIGNMENT;
    apex4::E4m3Problem p = e4m3_problem(M, N, K);
    p.qa = static_cast<const uint8_t*>(qa8);
    p.sa = s_a;
    p.qw = static_cast<const uint8_t*>(qw8);
    p.sw = s_w;
    p.bf16 = y_type == APEX4_BF16;
    p.y = y;
    p.y32 = y_f32;
    p.ws = workspace;
    return to_status(apex4::launch_gemm_e4m3(p, static_cast<hipStream_t>(stream)));
}

size_t apex4_linear_e4m3_workspace_size(int64_t M, int64_t N, int64_t K)
{
    if (!e4m3_sizes(M, N, K) || M == 0 || N == 0) return 0;
    if (apex4::e4m3_rows_quantizes(e4m3_problem(M, N, K))) return 0;
    return align256((size_t)M * K) + align256((size_t)M * (K / 128) * 4) + apex4_gemm_e4m3_workspace_size(M, N, K);
}

apex4_status apex4_linear_e4m3(const void* x, int32_t x_type, const void* qw8, const float* s_w, int64_t M,
                               int64_t N, int64_t K, void* y, float* y_f32, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    if (!e4m3_sizes(M, N, K)) return APEX4_ERR_INVALID_ARG;
    if (!half_type(x_type)) return APEX4_ERR_UNSUPPORTED;
    const size_t need = apex4_linear_e4m3_workspace_size(M, N, K);
    if (workspace_bytes < need || (need > 0 && !workspace)) return APEX4_ERR_WORKSPACE;
    if (M == 0 || N == 0) return APEX4_OK;
    if (!x || !qw8 || !s_w || !y) return APEX4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(qw8, 16) || !aligned(s_w, 4) || !aligned(y, 2) || !aligned(y_f32, 4) ||
        !aligned(workspace, 256))
        return APEX4_ERR_ALIGNMENT;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    apex4::E4m3Problem p = e4m3_problem(M, N, K);
    p.qw = static_cast<const uint8_t*>(qw8);
    p.sw = s_w;
    p.bf16 = x_type == APEX4_BF16;
    p.y = y;
    p.y32 = y_f32;
    if (apex4::e4m3_rows_quantizes(p)) return to_status(apex4::launch_e4m3_rows(p, x, st));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t qa_bytes = align256((size_t)M * K), sa_bytes = align256((size_t)M * (K / 128) * 4);
    float* sa = reinterpret_cast<float*>(ws + qa_bytes);
    const hipError_t e = apex4::launch_quantize_e4m3(x, p.bf16, M, K, ws, sa, st);
    if (e != hipSuccess) return APEX4_ERR_HIP;
    p.qa = ws;
    p.sa = sa;
    p.ws = ws + qa_bytes + sa_bytes;
    return to_status(apex4::launch_gemm_e4m3(p, st));
}

}  // extern "C"
