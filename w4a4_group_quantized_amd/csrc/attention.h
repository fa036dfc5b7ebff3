// Launchers of the rotary, cache and attention calls (include/apex4.h), shared
// by their API file and their kernels.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace apex4 {

// Rotary positions: pairs of the first `rotary` numbers of every head turned by
// position * freqs[i], and scaled (apex4_rope, its argument names).
struct Rotation {
    const int64_t* positions;   // [T], null: no rotation
    const double* freqs;        // [rotary / 2]
    int32_t rotary;
    bool interleaved;
    double scale;
};

struct RopeProblem {
    const void* x;
    int32_t type;
    int64_t T;
    int32_t H, D;
    int64_t ldx;
    Rotation turn;
    void* y;
    int64_t ldy;
};
hipError_t launch_rope(const RopeProblem& p, hipStream_t stream);

// The 4-bit cache (layout in include/apex4.h).
struct Kv4Cache {
    uint8_t* k_codes;
    float* k_scales;
    uint8_t* v_codes;
    float* v_scales;
    int64_t pages;
    int32_t Hkv, D, page;       // page: tokens of one page, 16 * 2^n
    int32_t shift;              // log2(page)
};

struct Kv4AppendProblem {
    const void *q, *k, *v;      // q null: keys and values only (Hq is 0 then)
    bool bf16;
    int64_t T;
    int32_t Hq;
    int64_t ldq, ldk, ldv;
    Rotation turn;
    const int64_t* slots;
    Kv4Cache cache;
    void* q_out;                // [T, Hq, D]
};
hipError_t launch_kv4_append(const Kv4AppendProblem& p, hipStream_t stream);

struct Kv4ReadProblem {
    Kv4Cache cache;
    const int64_t* slots;
    int64_t T;
    int32_t type;
    void *k, *v;                // [T, Hkv, D]
};
hipError_t launch_kv4_read(const Kv4ReadProblem& p, hipStream_t stream);

struct Kv4AttentionProblem {
    const void* q;
    bool bf16;
    int64_t T;
    int32_t B, Hq;
    int32_t share;              // query heads of a key head
    int64_t ldq;
    const int32_t* cu_q;        // null: one query a sequence (T == B)
    const int32_t* kv_lens;
    const int32_t* table;       // [B, cols]
    int64_t cols;
    Kv4Cache cache;
    float scale;
    bool causal;
    int32_t window;             // 0: none
    int32_t max_q, max_kv;      // what to split the work for
    void* out;                  // [T, Hq, D]
    float* lse;                 // [T, Hq] or null
    void* ws;
};
size_t kv4_attention_workspace_bytes(const Kv4AttentionProblem& p);
hipError_t launch_kv4_attention(const Kv4AttentionProblem& p, hipStream_t stream);

}  // namespace apex4
