// The 8-bit block-scaled product (apex4_gemm_e4m3) in LDS tiles on gfx950.
#include "gemm_e4m3.h"
#include "layers.h"

namespace apex4 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int KB = 128;          // K values (bytes of a row) of a block

struct TileArgs {
    E4m3Problem p;
    int tiles_n, tiles_m;
    // The last `tail` tiles run as `parts` parts of K each (part q: stages
    // [q G / parts, (q + 1) G / parts)) into part[q][tile][BM][BN]; a
    // reduction adds them in part order.
    int tail, parts;
    float* part;
};

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes)
{
    // raw buffer: loads past `bytes` return zeros
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// 16 bytes a lane from memory straight to 1 KB of LDS
__device__ inline void copy_1k(const uint8_t* src, uint32_t bytes, uint8_t* dst, int voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(src, bytes), (lds_void*)dst, 16, voff, soff, 0, 0);
}

// Every copy of the stage has landed (vmcnt(0)) and every wave is done with
// the other buffer; no memory access moves across.
__device__ inline void stage_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    // (the builtin, which the compiler counts: an inline-asm wait would make
    // it wait for the next stage's copies before the first fragment read)
    __builtin_amdgcn_s_waitcnt(0xF70);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// (row block, column block) of a tile: bands of 4 row blocks, walked column by
// column, so that the 32 tiles that an XCD has in flight share 4 blocks of x
// and 8 of w
__device__ inline void tile_coords(const TileArgs& a, int tile, int& by, int& bx)
{
    const int band = 4 * a.tiles_n, g = tile / band, local = tile - g * band;
    const int rows = min(4, a.tiles_m - 4 * g);
    by = 4 * g + local % rows;
    bx = local / rows;
}

// WN x WM waves, each NT tiles of 16 weight rows by MT tiles of 16 activation
// rows; WPS: waves per SIMD that registers and LDS leave room for.
// KST: blocks of K per stage.
template <bool BF16, int WN, int WM, int NT, int MT, int WPS, int KST>
__global__ __launch_bounds__(WN* WM * 64, WPS) void e4m3_tile_kernel(TileArgs a)
{
    constexpr int BN = WN * NT * 16, BM = WM * MT * 16, WAVES = WN * WM;
    constexpr int RB = KST * KB;                     // bytes of a row per stage
    constexpr int LPR = RB / 16, RPC = 64 / LPR;     // lanes per row, rows per 1 KB copy
    constexpr int STEP = WAVES * RPC;                // rows that the waves' copies bring at a time
    constexpr int LOADS = (BN + BM) / STEP;          // 1 KB copies per wave and stage
    static_assert(BN % STEP == 0 && BM % STEP == 0, "a copy step is of w or of x");
    constexpr int STAGE = (BN + BM) * RB;
    // (objects of their own: the compiler then tells the copies in flight from
    // the reads of the other buffers)
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;
    const E4m3Problem& p = a.p;

    // full tiles first, then the parts of the others, part by part; XCD b mod 8
    // walks a contiguous range of the tiles in either (with the parts' tiles in
    // launch order each L2 fetches most of both operands: 515 x 4008 x 11008 49
    // us instead of 41, 300 x 8192 x 8192 59 instead of 54, 256 x 4096 x 4096
    // 14.6 and 15.8; a contiguous range of all parts' tiles 40, 54 and 21)
    const int full = a.tiles_n * a.tiles_m - a.tail;
    int lin = blockIdx.x, kpart = 0;
    const bool split = lin >= full;
    if (split) {
        kpart = (lin - full) / a.tail;
        lin = (lin - full) % a.tail;
    }
    const int per = (split ? a.tail : full) >> 3;
    if (lin < per * 8) lin = (lin & 7) * per + (lin >> 3);
    if (split) lin += full;
    int by, bx;
    tile_coords(a, lin, by, bx);
    const int m0 = by * BM, n0 = bx * BN;
    const int K = p.K, G = K / KB;
    const int all = (G + KST - 1) / KST;             // stages of all of K
    const int s0 = split ? kpart * all / a.parts : 0;
    const int stages = split ? (kpart + 1) * all / a.parts - s0 : all;
    const int rows_m = min(BM, p.M - m0), rows_n = min(BN, p.N - n0);
    const __amdgpu_buffer_rsrc_t rSA = buffer_of(p.sa + (int64_t)m0 * G, (uint32_t)rows_m * G * 4);
    const int nblk = n0 / 128, nblks = (rows_n + 127) / 128;
    const __amdgpu_buffer_rsrc_t rSW = buffer_of(p.sw + (int64_t)nblk * G, (uint32_t)nblks * G * 4);

    // Copy j of this wave brings rows RPC (j WAVES + wave) .. of the stage's BN
    // rows of w and BM rows of x; lane l fetches chunk (l % LPR) ^ (row & KEY) of
    // row l / LPR, so that the fragment reads of 16 rows at one column touch every
    // bank once.  A descriptor per copy, so that one lane offset serves all of
    // them and rows past the end read zeros.
    const uint8_t* src[LOADS];
    uint32_t bytes[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        const int r = j * STEP;
        const bool w = r < BN;
        const int first = w ? r : r - BN;
        const int left = max(0, (w ? rows_n : rows_m) - first);
        src[j] = w ? p.qw + (int64_t)(n0 + first) * K : p.qa + (int64_t)(m0 + first) * K;
        bytes[j] = __builtin_amdgcn_readfirstlane((uint32_t)min(left, STEP) * K);
    }
    constexpr int KEY = LPR < 16 ? LPR - 1 : 15;      // bits of the row that place its chunks
    const int lrow = RPC * wave + lane / LPR, lchunk = (lane % LPR) ^ (lrow & KEY);
    auto copy = [&](uint8_t* dst, int t, int j0, int j1) {
#pragma unroll
        for (int j = j0; j < j1; ++j) {
            // (steps of fewer than 16 rows: the row's upper bit comes from the step)
            const int chunk = lchunk ^ (j * STEP & KEY);
            // (more blocks a stage than K has left: those stay out)
            const bool out = KST > 1 && (s0 + t) * KST + chunk / 8 >= G;
            copy_1k(src[j], bytes[j], dst + (j * WAVES + wave) * 1024, out ? (int)0x80000000 : lrow * K + chunk * 16,
                    (s0 + t) * RB);
        }
    };

    // scales of four blocks at a time: one register set, reloaded as soon as
    // the last of the four has given its values
    uint32_t saoff[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) saoff[i] = (uint32_t)(wm * MT * 16 + i * 16 + (lane & 15)) * G * 4;
    const uint32_t swoff = (uint32_t)(wn * NT * 16 / 128) * G * 4;
    v4f sa[MT], sw;
    auto load_scales = [&](int block) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
            sa[i] = __builtin_bit_cast(
                v4f, __builtin_amdgcn_raw_buffer_load_b128(rSA, (int)saoff[i] + (s0 * KST + block) * 4, 0, 0));
        sw = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rSW, (int)swoff + (s0 * KST + block) * 4, 0, 0));
    };

    // Fragment offsets: row lane & 15, chunks (lane >> 4) + 4 j (any split of
    // the block's K over the lanes will do, alike for both operands).  A
    // 16-byte LDS read serves lanes 0-3, 12-15 and 20-27 in one cycle, then
    // the others: with neighbouring chunks in neighbouring lane groups their
    // 16 rows lie in 16 different places of the 256 bytes (chunks 2 (lane >>
    // 4) + j took two cycles).
    const int row = lane & 15, key = row & KEY;
    int foff[KST][2];
#pragma unroll
    for (int q = 0; q < KST; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) foff[q][j] = row * RB + ((8 * q + (lane >> 4) + 4 * j) ^ key) * 16;
    const int wbase = wn * NT * 16 * RB, xbase = (BN + wm * MT * 16) * RB;

    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{};

    auto frag = [&](const uint8_t* b, int q) {
        const v4i lo = *reinterpret_cast<const v4i*>(b + foff[q][0]);
        const v4i hi = *reinterpret_cast<const v4i*>(b + foff[q][1]);
        return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    auto compute = [&](const uint8_t* b, int q, const float (&S)[MT], auto&& issue) {
        v8i x[MT], w[2];
        v4f P[2][MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) x[i] = frag(b + xbase + i * 16 * RB, q);
        w[0] = frag(b + wbase, q);
#pragma unroll
        for (int j = 0; j <= NT; ++j) {
            issue(j);
            if (j + 1 < NT) w[(j + 1) & 1] = frag(b + wbase + (j + 1) * 16 * RB, q);
            // the products of w tile j beside the fold of tile j - 1, kept in
            // this order: left alone, the compiler folds each product at once
            // and waits for the matrix unit
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if (j < NT)
                    P[j & 1][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[j & 1], x[i], v4f{}, 0, 0, 0, 127,
                                                                                  0, 127);
                if (j > 0)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j - 1][r] = fmaf(S[i], P[(j - 1) & 1][i][r], acc[i][j - 1][r]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    load_scales(0);
    copy(buf0, 0, 0, LOADS);
    for (int t0 = 0; t0 < stages; t0 += 4) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int t = t0 + h;
            if (t >= stages) break;
            stage_barrier();
            // the next stage's copies, two beside each of the first w tiles,
            // the rest at once (past the last stage: a stage again, into a
            // buffer that is not read)
            auto issue = [&](int j) {
                if (2 * j < LOADS)
                    copy(h & 1 ? buf0 : buf1, t + 1 < stages ? t + 1 : 0, 2 * j,
                         j == NT ? LOADS : min(2 * j + 2, LOADS));
            };
#pragma unroll
            for (int q = 0; q < KST; ++q) {
                const int o = (KST * h + q) & 3;
                float S[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) S[i] = sa[i][o] * sw[o];
                if (o == 3) load_scales(t * KST + q + 1);
                if (KST > 1 && (s0 + t) * KST + q >= G) continue;
                if (q == 0) compute(h & 1 ? buf1 : buf0, q, S, issue);
                else compute(h & 1 ? buf1 : buf0, q, S, [](int) {});
            }
        }
    }

    stage_barrier();      // the copies in flight land before this LDS is used for anything else
    if (split) {
        float* out = a.part + ((size_t)kpart * a.tail + lin - full) * (BM * BN);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *reinterpret_cast<v4f*>(out + (size_t)(wm * MT * 16 + i * 16 + (lane & 15)) * BN + wn * NT * 16 +
                                        j * 16 + 4 * (lane >> 4)) = acc[i][j];
        return;
    }

    // --- epilogue: a lane holds 4 neighbouring columns of 16 rows per tile;
    // the wave's MT*16 x NT*16 outputs go through LDS (its own part of the
    // stage buffers, 8-byte pieces, piece c of row m at c ^ m modulo the pieces) and leave
    // in 16-byte stores that cover whole rows of the tile.  (Stored from the
    // accumulators, 2 bytes a lane, they took 30 us a tile.) ---
    constexpr int ROW = NT * 16 * 2;                  // bytes of a row of the wave's tile
    constexpr int PM = ROW / 8 < 16 ? ROW / 8 - 1 : 15;   // pieces that a row's place is spread over
    static_assert(MT * 16 * ROW * WAVES <= 2 * STAGE, "the waves' tiles in LDS");
    constexpr int PER_BUF = STAGE / (MT * 16 * ROW);  // waves per stage buffer
    uint8_t* out = (wave < PER_BUF ? buf0 : buf1) + (wave % PER_BUF) * MT * 16 * ROW;
    const int c0 = n0 + wn * NT * 16, r0 = m0 + wm * MT * 16;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int lm = i * 16 + (lane & 15), m = r0 + lm;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint16_t h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = acc[i][j][r];
                asm volatile("" : "+v"(v));           // y is the rounding of y32
                h[r] = e4m3::to16<BF16>(v);
                const int n = c0 + j * 16 + 4 * (lane >> 4) + r;
                if (p.y32 && m < p.M && n < p.N) p.y32[(int64_t)m * p.N + n] = v;
            }
            *reinterpret_cast<uint2*>(out + lm * ROW + ((4 * j + (lane >> 4)) ^ (lm & PM)) * 8) =
                make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        }
    }
    uint16_t* y = static_cast<uint16_t*>(p.y);
    if (p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0) {
        constexpr int OL = ROW / 16;                  // lanes per row
#pragma unroll 4
        for (int q = lane; q < MT * 16 * OL; q += 64) {
            const int lm = q / OL, c = 2 * (q % OL);
            const uint2 u = *reinterpret_cast<const uint2*>(out + lm * ROW + (c ^ (lm & PM)) * 8);
            const uint2 v = *reinterpret_cast<const uint2*>(out + lm * ROW + ((c + 1) ^ (lm & PM)) * 8);
            const int m = r0 + lm, n = c0 + 4 * c;
            if (m < p.M && n < p.N)
                *reinterpret_cast<uint4*>(y + (int64_t)m * p.N + n) = make_uint4(u.x, u.y, v.x, v.y);
        }
    } else {
        // rows that start anywhere: 2 bytes a lane
        for (int q = lane; q < MT * 16 * NT * 16; q += 64) {
            const int lm = q / (NT * 16), c = q % (NT * 16), m = r0 + lm, n = c0 + c;
            if (m < p.M && n < p.N)
                y[(int64_t)m * p.N + n] =
                    *reinterpret_cast<const uint16_t*>(out + lm * ROW + ((c >> 2) ^ (lm & PM)) * 8 + (c & 3) * 2);
        }
    }
}

// y of the tiles that ran in parts of K: the parts' sums in part order.  One
// thread per 4 columns of a tile row.
template <bool BF16, int BN, int BM>
__global__ __launch_bounds__(256) void e4m3_reduce_kernel(TileArgs a)
{
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    constexpr int PER = BM * BN / 4;
    if (idx >= (int64_t)a.tail * PER) return;
    const int t = (int)(idx / PER), rem = (int)(idx - (int64_t)t * PER);
    const int row = rem / (BN / 4), col = (rem - row * (BN / 4)) * 4;
    const E4m3Problem& p = a.p;
    int by, bx;
    tile_coords(a, a.tiles_n * a.tiles_m - a.tail + t, by, bx);
    const int m = by * BM + row, n0 = bx * BN + col;
    if (m >= p.M || n0 >= p.N) return;
    const float* src = a.part + (size_t)t * (BM * BN) + row * BN + col;
    v4f s = *reinterpret_cast<const v4f*>(src);
    for (int q = 1; q < a.parts; ++q) s += *reinterpret_cast<const v4f*>(src + (size_t)q * a.tail * (BM * BN));
    uint16_t* y = static_cast<uint16_t*>(p.y) + (int64_t)m * p.N + n0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float v = s[r];
        asm volatile("" : "+v"(v));                   // y is the rounding of y32
        if (n0 + r < p.N) {
            y[r] = e4m3::to16<BF16>(v);
            if (p.y32) p.y32[(int64_t)m * p.N + n0 + r] = v;
        }
    }
}

// The tile shapes, and how a call is cut: the shape and the number of K parts
// of the last tiles with the least modelled time.  The model's numbers are
// measured on 256 compute units: a block (128 of K) of a CU that holds all the
// workgroups it can, and of one that holds a single one, which waits for its
// copies; 5.5 TB/s for the operands, 12 TB/s for weights read again by another
// row of tiles; the shorter of the two times hides to two thirds under the
// longer; 4 TB/s for writing the partial sums and reading them again, and 1 us
// for that launch.  For few rows what counts is how much of a weight row one
// copy covers: 16 x 28672 x 8192 (235 MB, weights from HBM) takes 57 us with
// 128 bytes of 128 rows a stage, 47 with 256 bytes of 64 and 43 (5.5 TB/s)
// with 512 bytes of 64; beyond 32 rows the codes of x take their part of the
// copies, and 128 bytes of 128 weight rows are as good (64 x 28672 x 8192: 62
// us both).  Many rows: 4096 x 8192 x 8192 260 us in tiles of 256 x 256, 321 in
// 128 x 128, 419 in 128 x 64.
struct Shape {
    int bn, bm, per_cu;          // weight rows, activation rows, workgroups that fit a CU
    double loaded_us, alone_us;  // one block of K
};
constexpr int SHAPES = 5;
constexpr Shape kShapes[SHAPES] = {
    {256, 256, 1, 2.0, 1.6}, {128, 128, 2, 1.25, 0.78}, {128, 64, 3, 1.09, 0.6}, {64, 32, 3, 0.6, 0.45}, {64, 16, 2, 0.4, 0.32}};

struct Cut {
    int shape, tail, parts;
    size_t bytes;
};

Cut choose(const E4m3Problem& p, int cus)
{
    const int G = p.K / KB;
    const bool can_split = cus > 0;
    if (!can_split) cus = 256;
    Cut best{0, 0, 1, 0};
    double best_us = 0.0;
    for (int c = 0; c < SHAPES; ++c) {
        const Shape& s = kShapes[c];
        const int64_t tiles = (int64_t)((p.M + s.bm - 1) / s.bm) * ((p.N + s.bn - 1) / s.bn);
        const int64_t slots = (int64_t)cus * s.per_cu;
        const int64_t tail = tiles % slots;
        for (int parts = 1; parts <= 8 && parts <= (G + 3) / 4; ++parts) {
            if (parts > 1 && (tail == 0 || !can_split)) break;
            const int64_t per = (tail * parts + cus - 1) / cus, rest = per % s.per_cu;   // last workgroups per CU
            double last = (double)(per / s.per_cu) * s.loaded_us;
            if (rest) {
                const double share = s.loaded_us * (double)rest / s.per_cu;
                last += share > s.alone_us ? share : s.alone_us;
            }
            double us = (double)(tiles / slots) * G * s.loaded_us + last * ((G + parts - 1) / parts);
            const double w = (double)p.N * p.K, rows = (p.M + s.bm - 1) / s.bm;
            const double read = (w + (double)p.M * p.K + 2.0 * p.M * p.N) / 5.5e6 + (rows - 1) * w / 12e6;
            us = us > read ? us + 0.35 * read : read + 0.35 * us;
            const int64_t mem = parts > 1 ? tail * parts * s.bm * s.bn * 4 : 0;
            if (mem) us += 1.0 + (double)mem / 4e6;
            if (best_us == 0.0 || us < best_us) {
                best_us = us;
                best = Cut{c, parts > 1 ? (int)tail : 0, parts, (size_t)mem};
            }
        }
    }
    return best;
}

template <bool BF16, int WN, int WM, int NT, int MT, int WPS, int KST = 1>
hipError_t launch_shape(TileArgs a, hipStream_t stream)
{
    constexpr int BN = WN * NT * 16, BM = WM * MT * 16;
    a.tiles_m = (a.p.M + BM - 1) / BM;
    a.tiles_n = (a.p.N + BN - 1) / BN;
    const int64_t grid = (int64_t)a.tiles_m * a.tiles_n + (int64_t)a.tail * (a.parts - 1);
    e4m3_tile_kernel<BF16, WN, WM, NT, MT, WPS, KST><<<(unsigned)grid, WN * WM * 64, 0, stream>>>(a);
    if (a.tail) {
        const int64_t n = (int64_t)a.tail * (BM * BN / 4);
        e4m3_reduce_kernel<BF16, BN, BM><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_cut(const TileArgs& a, int shape, hipStream_t stream)
{
    if (shape == 0) return launch_shape<BF16, 2, 4, 8, 4, 2>(a, stream);
    if (shape == 1) return launch_shape<BF16, 2, 2, 4, 4, 2>(a, stream);
    if (shape == 2) return launch_shape<BF16, 4, 1, 2, 4, 3>(a, stream);
    if (shape == 3) return launch_shape<BF16, 4, 1, 1, 2, 3, 2>(a, stream);
    return launch_shape<BF16, 4, 1, 1, 1, 2, 4>(a, stream);
}

}  // namespace

size_t e4m3_tiled_workspace_bytes(const E4m3Problem& p) { return choose(p, compute_units()).bytes; }

hipError_t launch_e4m3_tiled(const E4m3Problem& p, hipStream_t stream)
{
    const Cut cut = choose(p, compute_units());
    TileArgs a{};
    a.p = p;
    a.tail = cut.tail;
    a.parts = cut.parts;
    a.part = static_cast<float*>(p.ws);
    return p.bf16 ? launch_cut<true>(a, cut.shape, stream) : launch_cut<false>(a, cut.shape, stream);
}

}  // namespace apex4
