// The experts' W4A4 network for a few tokens (decoding) on gfx950, in two
// launches: gate and up of every chosen expert, then all the down products of
// a column block with the weighted sum over the experts.
//
// Such a call is the stream of the chosen experts' weights and the chain of
// small steps around it.  Launches of their own for the order of the slots, the
// codes of x, a product, the codes of h, a product and the sum took 50 us for one
// token and 8 of 64 experts (4096 x 1408; 74 MB of weights, 14 us at the rate
// of a large copy), of which the two products were 36; this way it takes 27.
// Here
//   - no plan: a wave looks at the at most 64 ids itself.  An entry is an
//     expert with the tokens that name it, one slot a token (a token that names
//     it again gives another entry); the matrix instruction's 16 activation
//     rows are the tokens;
//   - every workgroup quantizes the activations it needs (x, or h of all
//     slots) into LDS while its weights are on their way: a few dozen values
//     a thread, from L2;
//   - weights come by direct-to-LDS copies into a buffer of each wave's own,
//     16 rows by 512 bytes (1024 codes) at a time, so that no barrier stands
//     between a wave and its stream;
//   - the down launch walks all entries for its 16 columns.  Which wave takes
//     an item goes by the entries of all tokens, so each item's sums are stored
//     by slot, over the codes that the item alone has read, and a token's are
//     added at the end in the order of its slots: its result does not depend
//     on what other tokens name.
// LDS: piece c (16 bytes) of a row sits at c ^ row, so that the 16 rows' reads
// of one column touch every bank once.
#include "experts.h"
#include "layers.h"
#include "quant_rule.h"

namespace apex4 {
namespace {

using qrule::half8;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int TOKENS = 16;           // tokens of a call at most
constexpr int SLOTS = 64;            // and slots
constexpr int ITEM = 512;            // bytes of a row per item
constexpr int PIECE = 16 * ITEM;     // bytes of an item
constexpr int GPI = ITEM / 64;       // groups per item
constexpr int BUF = PIECE + GPI * 64; // an item in LDS: its codes, its scales
constexpr int UP_WAVES = 4, DOWN_WAVES = 8;
constexpr int BUFS = 2;              // buffers of a wave
constexpr int OOB = (int)0x80000000; // past every buffer: reads zeros
constexpr int PAD = 16;              // bytes between activation rows: their reads fall on different banks

struct Entries {
    signed char slot[SLOTS][TOKENS];  // of an entry's token; ~(its first slot) for a token that does not name it
    signed char entry[SLOTS];         // of a slot, -1 for none
};

// The entries, found by every wave for itself (lane s is slot s), so that it
// can ask for its weights before any barrier.
struct Found {
    int id;               // of this lane's slot, below 0 for a dead one
    int entry;            // of this lane's slot
    uint64_t leads;       // the first slots of the entries
    int n;
    __device__ int expert(int y) const
    {
        uint64_t l = leads;
        for (; y > 0; --y) l &= l - 1;
        return __builtin_amdgcn_readlane(id, __builtin_ctzll(l));
    }
};

// (id: of this lane's slot, -1 past the slots)
__device__ inline Found find_entries(int id, int R, int k, int E)
{
    const int lane = threadIdx.x & 63;
    Found f;
    f.id = id;
    const bool live = f.id >= 0 && f.id < E;
    if (!live) f.id = -1 - lane;      // like no other
    int rank = 0;                     // this token's earlier slots of the same expert
    int lead = lane;                  // the first slot of the entry
    if (R > 1) {
        // slots of one token, back from this one
        const int at = lane % k;
        for (int d = 1; d < k; ++d) rank += __shfl(f.id, lane - d) == f.id && d <= at;
        if (R > k)
            for (int s = R - 1; s >= 0; --s)
                if (__builtin_amdgcn_readlane(f.id, s) == f.id && __builtin_amdgcn_readlane(rank, s) == rank) lead = s;
    }
    f.leads = __ballot(live && lead == lane);
    f.entry = live ? __popcll(f.leads & ((1ull << lead) - 1)) : -1;
    f.n = __popcll(f.leads);
    return f;
}

// the tables that the products look into (one wave)
__device__ inline void write_entries(Entries& t, const Found& f, int k)
{
    const int lane = threadIdx.x & 63;
    const int none = (~lane & 255) * 0x01010101;
    if (f.leads >> lane & 1) *reinterpret_cast<int4*>(t.slot[f.entry]) = make_int4(none, none, none, none);
    t.entry[lane] = (signed char)f.entry;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (f.entry >= 0) t.slot[f.entry][lane / k] = (signed char)lane;
}

__device__ inline v4i widen_lo(v4i w)
{
    return v4i{(int)(((uint32_t)w[0] << 4) & 0xF0F0F0F0u), (int)((uint32_t)w[0] & 0xF0F0F0F0u),
               (int)(((uint32_t)w[1] << 4) & 0xF0F0F0F0u), (int)((uint32_t)w[1] & 0xF0F0F0F0u)};
}
__device__ inline v4i widen_hi(v4i w)
{
    return v4i{(int)(((uint32_t)w[2] << 4) & 0xF0F0F0F0u), (int)((uint32_t)w[2] & 0xF0F0F0F0u),
               (int)(((uint32_t)w[3] << 4) & 0xF0F0F0F0u), (int)((uint32_t)w[3] & 0xF0F0F0F0u)};
}

// Item `it` (bytes it ITEM .. of 16 weight rows) into a wave's buffer: copy j
// brings rows 2 j and 2 j + 1.  `rows`: the first row of each run of 8 rows
// (gate and up rows lie apart).
__device__ inline void copy_item(uint8_t* dst, const uint8_t* rows0, const uint8_t* rows8, int rowbytes, int it)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = 2 * j + (lane >> 5);
        const int pos = it * ITEM + (((lane & 31) ^ r) * 16);
        const uint8_t* base = j < 4 ? rows0 : rows8;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, 8 * rowbytes, 0x00020000),
            (lds_void*)(dst + j * 1024), 16, pos < rowbytes ? (r & 7) * rowbytes + pos : OOB, 0, 0, 0);
    }
}

// The scales of an item's groups into [group][weight row] after its codes: lane
// l of copy j brings row l & 15 of group 4 j + (l >> 4) (past the row: zeros).
__device__ inline void copy_scales(uint8_t* dst, const float* rows0, const float* rows8, int G, int it)
{
    const int lane = threadIdx.x & 63, r = lane & 15;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int g = it * GPI + 4 * j + (lane >> 4);
        const int64_t far = r < 8 ? 0 : (rows8 - rows0) * 4;
        // (gate and up rows of one expert: less than 2^31 bytes apart)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(rows0), (short)0,
                                              (int)((rows8 - rows0) * 4 + 8 * G * 4), 0x00020000),
            (lds_void*)(dst + PIECE + j * 256), 4, g < G ? (int)far + ((r & 7) * G + g) * 4 : OOB, 0, 0, 0);
    }
}

// Workgroup barrier for what was stored to LDS; copies in flight stay in flight.
__device__ inline void lds_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A thread's values to quantize, asked for before anything else: chunks of 8
// at tid, tid + threads, ..
template <int NX>
__device__ inline void load_chunks(half8 (&v)[NX], const half8* x, int n8, int threads)
{
#pragma unroll
    for (int c = 0; c < NX; ++c) v[c] = x[min((int)threadIdx.x + c * threads, n8 - 1)];
}

// acc[r] += sum over the item's groups of sa4(q)[r] s_w[q] P, P of activation row 4 (lane >> 4) + r and weight row
// lane & 15.  `x`: the codes of this lane's activation row lane & 15 at the item's first byte; `left`: bytes of the
// row from there.
template <typename Scale>
__device__ inline void item_products(v4f& acc, const uint8_t* buf, const uint8_t* x, int left, Scale sa4)
{
    const int lane = threadIdx.x & 63, row = lane & 15, kg = lane >> 4;
    const float* sw = reinterpret_cast<const float*>(buf + PIECE) + row;
    const int groups = min(GPI, left / 64);
    // four groups at a time, their reads together and then their products: one
    // after the other each group waits for LDS and for the matrix unit (an item
    // took 0.7 us); all eight unrolled, a launch of a few microseconds fetches
    // more code than it saves
#pragma unroll 1
    for (int q0 = 0; q0 < groups; q0 += 4) {
        v4i w[4], a[4], P[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = min(q0 + i, groups - 1);
            w[i] = *reinterpret_cast<const v4i*>(buf + row * ITEM + ((4 * q + kg) ^ row) * 16);
            a[i] = *reinterpret_cast<const v4i*>(x + 64 * q + 16 * kg);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            P[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(widen_lo(a[i]), widen_lo(w[i]), v4i{}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            P[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(widen_hi(a[i]), widen_hi(w[i]), P[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (q0 + i >= groups) break;
            const v4f s = sa4(q0 + i);
            const float sn = sw[16 * (q0 + i)];
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = fmaf(s[r] * sn, (float)P[i][r], acc[r]);
        }
    }
}

// This item's copies have landed: all but the 10 of the item after it (8 of
// codes, 2 of scales).  Items past the last are fetched too, as zeros from no
// address, so that this count always holds.
__device__ inline void wait_copies()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xF70 | 10);
    asm volatile("" ::: "memory");
}

struct TokenArgs {
    ExpertsProblem p;
    int G;                // groups of the launch's K
    int M4;               // tokens, in fours
};

// LDS of the gate-and-up launch beside the waves' buffers: the codes of x
// (rows of H/2 + PAD bytes), their scales as [G][16].
__host__ __device__ inline int up_lds(const TokenArgs& a)
{
    return (int)a.p.M * (a.p.H / 2 + PAD) + a.G * 64;
}

// A wave walks all of K for 8 gate rows and the 8 up rows of the same columns
// of h: no sum crosses waves, and the codes of x are made once for 4 of them.
template <int NX>
__global__ __launch_bounds__(UP_WAVES * 64) void token_up_kernel(TokenArgs a, _Float16* __restrict__ h)
{
    // (objects of their own: the compiler then tells the copies in flight from
    // the other buffer's reads and the stores of the codes)
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[UP_WAVES * BUF];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[UP_WAVES * BUF];
    extern __shared__ __attribute__((aligned(16))) uint8_t xq[];
    __shared__ Entries t;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int M = (int)a.p.M, k = a.p.k, H = a.p.H, I = a.p.I, G = a.G, R = M * k;
    const int stride = H / 2 + PAD;
    float* xs = reinterpret_cast<float*>(xq + M * stride);

    const int n8 = M * (H / 8);
    // (the ids first: what is asked for before them is waited for with them)
    int id = a.p.ids[min(lane, R - 1)];
    half8 v[NX];
    load_chunks(v, static_cast<const half8*>(a.p.x), n8, UP_WAVES * 64);
    id = lane < R ? id : -1;
    const Found f = find_entries(id, R, k, a.p.E);
    const int blocks = I / 8, block = blockIdx.x * UP_WAVES + wave, y = block / blocks;
    if (blockIdx.x * UP_WAVES >= f.n * blocks) return;
    const bool live = y < f.n;
    const int e = live ? f.expert(y) : 0, n0 = (block - y * blocks) * 8;
    const int rowbytes = H / 2, items = live ? (rowbytes + ITEM - 1) / ITEM : 0;
    const uint8_t* gate = a.p.qw_gu + ((int64_t)e * 2 * I + n0) * rowbytes;
    const uint8_t* up = gate + (int64_t)I * rowbytes;
    const int wr = lane & 15;
    const float* sgate = a.p.s_gu + ((int64_t)e * 2 * I + n0) * G;
    auto fetch = [&](uint8_t* buf, int it) {
        copy_item(buf + wave * BUF, gate, up, rowbytes, it);
        copy_scales(buf + wave * BUF, sgate, sgate + (int64_t)I * G, G, it);
    };
    // (a wave without an entry: rows of expert 0)
    fetch(buf0, 0);
    fetch(buf1, 1);

    // the codes of x beside them
#pragma unroll
    for (int j = 0; j < NX; ++j) {
        const int i = tid + j * UP_WAVES * 64;
        if (i >= n8) break;
        const float scale = experts_scale(v[j]);
        const int m = i / (H / 8), c = i - m * (H / 8);
        *reinterpret_cast<uint32_t*>(xq + m * stride + 4 * c) = qrule::quantize8(v[j], scale, scale != 0.0f);
        if ((c & 15) == 0) xs[(c >> 4) * 16 + m] = scale;
    }
    for (int i = tid; i < G * 16; i += UP_WAVES * 64)
        if ((i & 15) >= M) xs[i] = 0.0f;
    if (wave == 0) write_entries(t, f, k);
    lds_barrier();

    v4f acc = {};
    const uint8_t* xrow = xq + (wr < M ? wr : 0) * stride;
    for (int i0 = 0; i0 < items; i0 += BUFS) {
#pragma unroll
        for (int b = 0; b < BUFS; ++b) {
            const int it = i0 + b;
            wait_copies();
            if (it < items)
                item_products(acc, (b ? buf1 : buf0) + wave * BUF, xrow + it * ITEM, rowbytes - it * ITEM, [&](int q) {
                    return *reinterpret_cast<const v4f*>(xs + (it * GPI + q) * 16 + 4 * (lane >> 4));
                });
            asm volatile("" ::: "memory");
            fetch(b ? buf1 : buf0, it + BUFS);
        }
    }
    __builtin_amdgcn_s_waitcnt(0xF70);   // no copy outlives the wave
    if (!live) return;
    // lane 16 (m >> 2) + n, register m & 3: activation row m and weight row n (gate rows 0..7, up rows 8..15)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float u = __shfl(acc[r], lane + 8);
        const int m = 4 * (lane >> 4) + r;
        const int s = m < M && wr < 8 ? t.slot[y][m] : -1;
        if (s >= 0) h[(int64_t)s * I + n0 + wr] = experts_h(acc[r] * 0.00390625f, u * 0.00390625f);
    }
}

// LDS of the down launch beside the waves' buffers: the codes of h (rows of
// I/2 + PAD bytes by slot), their scales as [entry][G][M4].
__host__ __device__ inline int down_lds(const TokenArgs& a)
{
    const int R = (int)a.p.M * a.p.k;
    return R * (a.p.I / 2 + PAD) + R * a.G * a.M4 * 4;
}

template <int NX>
__global__ __launch_bounds__(DOWN_WAVES * 64) void token_down_kernel(TokenArgs a, const _Float16* __restrict__ h)
{
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[DOWN_WAVES * BUF];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[DOWN_WAVES * BUF];
    extern __shared__ __attribute__((aligned(16))) uint8_t hq[];
    __shared__ Entries t;
    __shared__ float gates[SLOTS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int M = (int)a.p.M, k = a.p.k, H = a.p.H, I = a.p.I, G = a.G, R = M * k, M4 = a.M4;
    const int stride = I / 2 + PAD;
    float* tab = reinterpret_cast<float*>(hq + R * stride);

    const int n8 = R * (I / 8);
    int id = a.p.ids[min(lane, R - 1)];
    half8 v[NX];
    load_chunks(v, reinterpret_cast<const half8*>(h), n8, DOWN_WAVES * 64);
    const float gate = a.p.gates[min(lane, R - 1)];
    id = lane < R ? id : -1;
    const Found f = find_entries(id, R, k, a.p.E);
    const int n0 = blockIdx.x * 16, rowbytes = I / 2, per = (rowbytes + ITEM - 1) / ITEM, items = f.n * per;
    const int wr = lane & 15;
    auto fetch = [&](uint8_t* buf, int item) {
        int en = item / per, it = item - en * per;
        if (item >= items) {
            en = 0;
            it = per;                            // past the rows: zeros
        }
        const int64_t first = (int64_t)f.expert(en) * H + n0;
        const uint8_t* w = a.p.qw_down + first * rowbytes;
        const float* sd = a.p.s_down + first * G;
        copy_item(buf + wave * BUF, w, w + 8 * (int64_t)rowbytes, rowbytes, it);
        copy_scales(buf + wave * BUF, sd, sd + 8 * G, G, it);
    };
    if (f.n == 0) {                              // nothing live: zeros
        for (int i = tid; i < M * 16; i += DOWN_WAVES * 64) {
            const int64_t o = (int64_t)(i >> 4) * H + n0 + (i & 15);
            static_cast<_Float16*>(a.p.y16)[o] = (_Float16)0.0f;
            if (a.p.y32) a.p.y32[o] = 0.0f;
        }
        return;
    }
    fetch(buf0, wave);
    fetch(buf1, wave + DOWN_WAVES);

    if (wave == 0) write_entries(t, f, k);
    lds_barrier();

    // the codes of h, and its scales (those of tokens that do not name an entry stay unset: what the matrix
    // instruction makes of their rows is not stored)
#pragma unroll
    for (int j = 0; j < NX; ++j) {
        const int i = tid + j * DOWN_WAVES * 64;
        if (i >= n8) break;
        const int s = i / (I / 8), c = i - s * (I / 8), en = t.entry[s];
        if (en < 0) continue;                    // (16 neighbouring lanes share a slot; its h is not set)
        const float scale = experts_scale(v[j]);
        *reinterpret_cast<uint32_t*>(hq + s * stride + 4 * c) = qrule::quantize8(v[j], scale, scale != 0.0f);
        if ((c & 15) == 0) tab[(en * G + (c >> 4)) * M4 + s / k] = scale;
    }
    if (wave == 0) gates[lane] = gate;
    lds_barrier();

    // the sums of item `it` for slot s: 16 floats in place of the codes that they were made of
    auto sums = [&](int s, int it) { return reinterpret_cast<float*>(hq + s * stride + it * ITEM); };
    for (int i0 = wave; i0 < items; i0 += BUFS * DOWN_WAVES) {
#pragma unroll
        for (int b = 0; b < BUFS; ++b) {
            const int item = i0 + b * DOWN_WAVES;
            const bool mine = item < items;
            const int en = item / per, it = item - en * per;
            v4f acc = {};
            int four = -1;
            wait_copies();
            if (mine) {
                // the slots of this lane's activation row (one that no token gives takes another's codes) and of
                // its four rows of sums
                int s = t.slot[en][wr];
                s ^= s >> 31;
                four = *reinterpret_cast<const int*>(&t.slot[en][4 * (lane >> 4)]);
                item_products(acc, (b ? buf1 : buf0) + wave * BUF, hq + s * stride + it * ITEM, rowbytes - it * ITEM,
                              [&](int q) {
                                  v4f v = {};
                                  if (4 * (lane >> 4) < M4)
                                      v = *reinterpret_cast<const v4f*>(tab + (en * G + it * GPI + q) * M4 +
                                                                        4 * (lane >> 4));
                                  return v;
                              });
            }
            asm volatile("" ::: "memory");
            fetch(b ? buf1 : buf0, item + BUFS * DOWN_WAVES);
            // (after the next copies: the sums are the end of the item's chain)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int to = (signed char)(four >> (8 * r));
                if (to >= 0) sums(to, it)[wr] = acc[r];
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0xF70);           // no copy outlives its buffer
    __syncthreads();
    // each slot's sum with its gate, 0 for a dead one; then each token's, in the order of its slots
    float* red = reinterpret_cast<float*>(buf0);  // the buffers are done with
#pragma unroll 1
    for (int i = tid; i < R * 16; i += DOWN_WAVES * 64) {
        const int s = i >> 4;
        float d = 0.0f;
#pragma unroll 1
        for (int it = 0; it < per; ++it) d += sums(s, it)[i & 15];
        red[i] = t.entry[s] >= 0 ? gates[s] * (d * 0.00390625f) : 0.0f;
    }
    __syncthreads();
    if (tid < 16 * TOKENS) {
        const int m = tid >> 4, c = tid & 15;
        if (m < M) {
            float v = 0.0f;
#pragma unroll 1
            for (int j0 = 0; j0 < k; j0 += 8) {
                float d[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = red[(m * k + min(j0 + j, k - 1)) * 16 + c];
#pragma unroll
                for (int j = 0; j < 8; ++j) v += j0 + j < k ? d[j] : 0.0f;
            }
            asm volatile("" : "+v"(v));          // y16 is the fp16 rounding of y32
            const int64_t o = (int64_t)m * H + n0 + c;
            static_cast<_Float16*>(a.p.y16)[o] = (_Float16)v;
            if (a.p.y32) a.p.y32[o] = v;
        }
    }
}

}  // namespace

static TokenArgs token_args(const ExpertsProblem& p, int K)
{
    TokenArgs a{};
    a.p = p;
    a.G = K / 128;
    a.M4 = ((int)p.M + 3) / 4 * 4;
    return a;
}

bool experts_token_supports(const ExpertsProblem& p)
{
    if (p.M > TOKENS || p.M * p.k > SLOTS || p.H > 16384 || p.I > 16384) return false;
    // what a workgroup quantizes, and its LDS beside buffers and entries: two workgroups of the first launch on a CU, one of the second
    if (p.M * p.H > 32768 || p.M * p.k * p.I > 32768) return false;
    return up_lds(token_args(p, p.H)) <= 10 * 1024 && down_lds(token_args(p, p.I)) <= 22 * 1024;
}

template <int NX_UP, int NX_DOWN>
static hipError_t launch_token(const ExpertsProblem& p, _Float16* h, hipStream_t stream)
{
    const TokenArgs up = token_args(p, p.H), down = token_args(p, p.I);
    const unsigned blocks = (unsigned)(p.M * p.k * (p.I / 8));
    token_up_kernel<NX_UP><<<(blocks + UP_WAVES - 1) / UP_WAVES, UP_WAVES * 64, up_lds(up), stream>>>(up, h);
    token_down_kernel<NX_DOWN><<<p.H / 16, DOWN_WAVES * 64, down_lds(down), stream>>>(down, h);
    return hipGetLastError();
}

hipError_t launch_experts_token(const ExpertsProblem& p, _Float16* h, hipStream_t stream)
{
    // chunks of 8 values that a thread quantizes
    const bool small_x = p.M * p.H <= 2 * 8 * UP_WAVES * 64, small_h = p.M * p.k * p.I <= 3 * 8 * DOWN_WAVES * 64;
    if (small_x) return small_h ? launch_token<2, 3>(p, h, stream) : launch_token<2, 8>(p, h, stream);
    return small_h ? launch_token<16, 3>(p, h, stream) : launch_token<16, 8>(p, h, stream);
}

}  // namespace apex4
