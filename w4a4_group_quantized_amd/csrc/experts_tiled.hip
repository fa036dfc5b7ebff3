// The experts' W4A4 products (apex4_experts_w4a4) in LDS tiles on gfx950.
//
// A workgroup computes BN weight rows of one expert by BM of its rows.  The
// packed nibbles go straight from memory to LDS (stages of SB bytes a row, SB /
// 64 groups of 128 codes), two stage buffers, the copies of the next stage
// issued beside the first products of this one; the scales of the stage's
// groups come in by 4-byte copies, turned so that group and row index the
// buffer.  A wave reads 16 bytes a lane of 16 rows, widens the nibbles to the
// int8 values 16 c ((w << 4) & 0xF0F0F0F0 and w & 0xF0F0F0F0, the two halves
// of a 32-code run, alike for both operands) and feeds v_mfma_i32_16x16x64_i8
// twice a group.  The weights are the A operand, so a lane holds one
// activation row and four consecutive weight rows; the products of tile j are
// issued beside the rescale of tile j - 1.
//
// What bounds it: for long runs of rows the vector ALU (99% busy at 512 rows an
// expert, 4096 x 2816: 650 us, 1160 TOPS): it widens both operands, converts,
// multiplies the scales and adds, 25 instructions a 16x16 tile and group (12
// of them the rescale, 9 the widening), 100 clocks against 32 of its matrix
// instructions.  (Scale products from the fp32 matrix instruction: 758 us, it
// does not run beside the vector ALU.  Activations stored as bytes, which
// leaves 6 of the 9 out: 672 and 710 us, twice the bytes to copy.  The micro-scaling
// instruction, with the weights split into two 2-bit E2M1 operands and the
// activations as E2M3, returns the same sums in fp32 for 27% fewer vector
// instructions, but its 96-byte groups cost more in copies and LDS than that:
// 725 us.)  The dense kernel of this rule has fewer: it widens once a workgroup,
// on the way into LDS, and takes the scale products from one bf16 matrix
// instruction on exact splits; neither is built here.  For few rows it is the
// stream of the weights (355 MB in 80 us, 4.4 TB/s, at 2.5 rows an expert).
#include "experts.h"
#include "layers.h"

namespace apex4 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int SB = 128;              // bytes of a row per stage (256 took as long at 2.5 rows an expert, with less room)
constexpr int GS = SB / 64;          // groups per stage
constexpr int LPR = SB / 16, RPC = 64 / LPR;   // lanes per row, rows per 1 KB copy
constexpr int KEY = LPR - 1;         // bits of the row that place its chunks
constexpr int OOB = (int)0x80000000; // past every buffer: reads zeros

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// 16 (4) bytes a lane from memory straight to 1 KB (256 bytes) of LDS
__device__ inline void copy16(const void* src, uint32_t bytes, uint8_t* dst, int voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(src, bytes), (lds_void*)dst, 16, voff, soff, 0, 0);
}
__device__ inline void copy4(const void* src, uint32_t bytes, uint8_t* dst, int voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(src, bytes), (lds_void*)dst, 4, voff, soff, 0, 0);
}

// every copy has landed and every wave is done with the other buffer
__device__ inline void stage_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xF70);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
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

// The expert and the tile of unit `unit`: expert e has ceil(rows / BM) *
// tiles_n units, the row tiles of one column tile next to each other.  False
// past the last unit.  Every wave searches by itself: 64 experts a step.
__device__ inline bool find_tile(const int32_t* __restrict__ offsets, int E, int tiles_n, int bm, int unit, int& e,
                                 int& first, int& count, int& mt, int& nt)
{
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int at = e0 + lane;
        const int lo = at < E ? offsets[at] : 0, hi = at < E ? offsets[at + 1] : 0;
        const int row_tiles = (hi - lo + bm - 1) / bm;
        int sum = row_tiles * tiles_n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(sum, o);
            if (lane >= o) sum += v;
        }
        const uint64_t past = __ballot(sum > unit);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            e = e0 + l;
            first = __shfl(lo, l);
            count = __shfl(hi, l) - first;
            const int tiles = __shfl(row_tiles, l);
            const int local = unit - (__shfl(sum, l) - tiles * tiles_n);
            mt = local % tiles;
            nt = local / tiles;
            return true;
        }
        unit -= __shfl(sum, 63);
    }
    return false;
}

// UP: gate and up rows in alternating tiles of 16, h out; else d out.
// WN x WM waves, each NT tiles of 16 weight rows by MT tiles of 16 rows.
template <bool UP, int WN, int WM, int NT, int MT, int WPS>
__global__ __launch_bounds__(WN* WM * 64, WPS) void experts_tile_kernel(ExpertsProduct a)
{
    constexpr int BN = WN * NT * 16, BM = WM * MT * 16, WAVES = WN * WM;
    constexpr int WCOPIES = BN / RPC / WAVES;                  // per wave and stage
    constexpr int XCOPIES = (BM / RPC + WAVES - 1) / WAVES;
    constexpr int WS = BN / 64, XS = (BM + 63) / 64;           // scale copies per group
    constexpr int SCOPIES = (GS * (WS + XS) + WAVES - 1) / WAVES;
    constexpr int DATA = (BN + BM) * SB;
    constexpr int STAGE = DATA + GS * 256 * (WS + XS);
    static_assert(BN % (RPC * WAVES) == 0 && BN % 64 == 0, "copies of the weights divide among the waves");
    static_assert(!UP || NT % 2 == 0, "a wave holds gate and up");
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;

    // XCD b mod 8 walks a contiguous range of units
    int unit = blockIdx.x;
    const int per = (int)gridDim.x >> 3;
    if (unit < per * 8) unit = (unit & 7) * per + (unit >> 3);
    // (UP: one part)
    const int units = UP ? (int)gridDim.x : (int)gridDim.x / a.parts, kpart = UP ? 0 : unit / units;
    if (!UP) unit -= kpart * units;
    int e, first, count, mt, nt;
    if (!find_tile(a.offsets, a.E, (a.N + BN - 1) / BN, BM, unit, e, first, count, mt, nt)) return;
    e = __builtin_amdgcn_readfirstlane(e);
    first = __builtin_amdgcn_readfirstlane(first);
    count = __builtin_amdgcn_readfirstlane(count);
    const int m0 = __builtin_amdgcn_readfirstlane(mt) * BM, n0 = __builtin_amdgcn_readfirstlane(nt) * BN;
    const int rowbytes = a.K / 2, G = a.K / 128, half = a.N / 2;
    const int all = (G + GS - 1) / GS;
    const int s0 = UP ? 0 : kpart * all / a.parts, stages = UP ? all : (kpart + 1) * all / a.parts - s0;
    const uint8_t* qw = a.qw + (int64_t)e * a.N * rowbytes;
    const float* sw = a.sw + (int64_t)e * a.N * G;
    // weight row of row r of the tile (a.N and more: none)
    auto weight_row = [&](int r) {
        return UP ? ((r >> 4) & 1 ? half : 0) + (n0 >> 1) + (r >> 5) * 16 + (r & 15) : n0 + r;
    };
    // activation row of row r of the tile, -1 for none, counted from the base below
    auto act_row = [&](int r) {
        const int m = m0 + r;
        if (r >= BM || m >= count) return -1;
        return UP ? a.order[first + m] / a.k : r;
    };
    const int64_t base = UP ? 0 : first + m0;
    const int64_t base_rows = UP ? a.rows : min(BM, count - m0);
    const uint8_t* qx = a.qx + base * rowbytes;
    const float* sx = a.sx + base * G;

    // --- the copies of this wave: RPC rows of SB bytes each, lane l chunk
    // (l % LPR) ^ row of row l / LPR (the fragment reads then touch every bank
    // once); groups that K does not have stay out ---
    const int lrow = RPC * wave + lane / LPR;
    const int chunk = (lane % LPR) ^ (lrow & KEY);
    const int wvoff = (lane / LPR) * rowbytes + chunk * 16;
    const uint8_t* wsrc[WCOPIES];
    uint32_t wbytes[WCOPIES];
#pragma unroll
    for (int j = 0; j < WCOPIES; ++j) {
        const int row = weight_row(RPC * (j * WAVES + wave));
        wsrc[j] = qw + (int64_t)row * rowbytes;
        wbytes[j] = __builtin_amdgcn_readfirstlane(row < a.N ? RPC * rowbytes : 0);
    }
    auto copy_w = [&](uint8_t* dst, int t) {
        t += s0;
        const bool out = t * GS + chunk / 4 >= G;
#pragma unroll
        for (int j = 0; j < WCOPIES; ++j)
            copy16(wsrc[j], wbytes[j], dst + (j * WAVES + wave) * 1024, out ? OOB : wvoff, t * SB);
    };
    copy_w(buf0, 0);      // (before the rows are looked up: their way is longer)
    int xvoff[XCOPIES];
#pragma unroll
    for (int j = 0; j < XCOPIES; ++j) {
        const int r = act_row(RPC * (j * WAVES + wave) + lane / LPR);
        xvoff[j] = r < 0 ? OOB : r * rowbytes + chunk * 16;
    }
    // scale copies: of 64 rows and one group each; copy c is of group c % GS
    int svoff[SCOPIES];
#pragma unroll
    for (int j = 0; j < SCOPIES; ++j) {
        const int s = (j * WAVES + wave) / GS;
        int r;
        if (s < WS) {
            r = weight_row(64 * s + lane);
            if (r >= a.N) r = -1;
        } else {
            r = act_row(64 * (s - WS) + lane);
        }
        svoff[j] = r < 0 ? OOB : r * G * 4;
    }
    const uint32_t xbytes = (uint32_t)(base_rows * rowbytes), sxbytes = (uint32_t)(base_rows * G * 4);
    auto copy_x = [&](uint8_t* dst, int t) {
        t += s0;
        const bool out = t * GS + chunk / 4 >= G;
#pragma unroll
        for (int j = 0; j < XCOPIES; ++j)
            if (j * WAVES + wave < BM / RPC)
                copy16(qx, xbytes, dst + BN * SB + (j * WAVES + wave) * 1024, out ? OOB : xvoff[j], t * SB);
#pragma unroll
        for (int j = 0; j < SCOPIES; ++j) {
            const int c = j * WAVES + wave, s = c / GS, g = c % GS;
            if (s < WS + XS)
                copy4(s < WS ? sw : sx, s < WS ? (uint32_t)a.N * G * 4 : sxbytes,
                      dst + DATA + (g * (WS + XS) + s) * 256, t * GS + g >= G ? OOB : svoff[j], (t * GS + g) * 4);
        }
    };

    const int row = lane & 15, kg = lane >> 4, key = row & KEY;
    int foff[GS];
#pragma unroll
    for (int g = 0; g < GS; ++g) foff[g] = row * SB + ((4 * g + kg) ^ key) * 16;

    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{};

    auto compute = [&](const uint8_t* b, int t, auto&& issue) {
        const uint8_t* wb = b + wn * NT * 16 * SB;
        const uint8_t* xb = b + (BN + wm * MT * 16) * SB;
#pragma unroll
        for (int g = 0; g < GS; ++g) {
            if (g > 0 && (s0 + t) * GS + g >= G) break;
            const float* scales = reinterpret_cast<const float*>(b + DATA + g * (WS + XS) * 256);
            const float* sws = scales + wn * NT * 16 + 4 * kg;
            const float* sas = scales + 64 * WS + wm * MT * 16 + row;
            v4i xlo[MT], xhi[MT], wf[2];
            v4f sw4[2];
            float sa[MT];
            v4i P[2][MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const v4i f = *reinterpret_cast<const v4i*>(xb + i * 16 * SB + foff[g]);
                xlo[i] = widen_lo(f);
                xhi[i] = widen_hi(f);
                sa[i] = sas[16 * i];
            }
            wf[0] = *reinterpret_cast<const v4i*>(wb + foff[g]);
            if (g == 0) issue();
#pragma unroll
            for (int j = 0; j <= NT; ++j) {
                if (j + 1 < NT) wf[(j + 1) & 1] = *reinterpret_cast<const v4i*>(wb + (j + 1) * 16 * SB + foff[g]);
                if (j < NT) sw4[j & 1] = *reinterpret_cast<const v4f*>(sws + 16 * j);
                v4i wlo, whi;
                if (j < NT) {
                    wlo = widen_lo(wf[j & 1]);
                    whi = widen_hi(wf[j & 1]);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (j < NT) {
                        P[j & 1][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wlo, xlo[i], v4i{}, 0, 0, 0);
                        P[j & 1][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(whi, xhi[i], P[j & 1][i], 0, 0, 0);
                    }
                    if (j > 0)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][j - 1][r] = fmaf(sa[i] * sw4[(j - 1) & 1][r], (float)P[(j - 1) & 1][i][r],
                                                    acc[i][j - 1][r]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };

    copy_x(buf0, 0);
    for (int t0 = 0; t0 < stages; t0 += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = t0 + h;
            if (t >= stages) break;
            stage_barrier();
            // (past the last stage: the first again, into a buffer that is not read)
            compute(h ? buf1 : buf0, t, [&]() {
                copy_w(h ? buf0 : buf1, t + 1 < stages ? t + 1 : 0);
                copy_x(h ? buf0 : buf1, t + 1 < stages ? t + 1 : 0);
            });
        }
    }
    stage_barrier();      // the copies in flight land before the workgroup ends

    // --- epilogue (2^-8: the widened codes) ---
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + wm * MT * 16 + i * 16 + row;
        if (m >= count) continue;
        if constexpr (UP) {
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                uint32_t h[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    h[r] = __builtin_bit_cast(uint16_t, experts_h(acc[i][j][r] * 0.00390625f,
                                                                  acc[i][j + 1][r] * 0.00390625f));
                const int c = (n0 >> 1) + (wn * NT + j) * 8 + 4 * kg;
                if (c < half)
                    *reinterpret_cast<uint2*>(a.h + (int64_t)(first + m) * half + c) =
                        make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int n = n0 + (wn * NT + j) * 16 + 4 * kg;
                if (n < a.N)
                    *reinterpret_cast<v4f*>(a.d + kpart * a.part_stride + (int64_t)(first + m) * a.N + n) = acc[i][j] * 0.00390625f;
            }
        }
    }
}

constexpr int BN = 128;      // weight rows of a tile

// at most this many tiles of rows: a partial one per expert with rows
int64_t row_tiles(int64_t R, int32_t E, int bm) { return R / bm + (R < E ? R : E); }

// Three workgroups a CU in both shapes.  64 rows from a mean of 12 rows an
// expert on (hidden 4096, 1408 between): with 64 experts, 16 rows each 106 us
// for gate and up against 116 of 32-row tiles, 512 rows each 650 against 790;
// 2.5 rows each 94 against 80.  48 rows took as long or longer but for one
// size (301 tokens, 2 of 8 experts, 4096 x 11008: 317 us a call against 329;
// 512 rows each 1263 against 1186).  Tiles of 128 x 128 and 256 x 256 were
// slower at every size (512 rows: 660 and 800), with fewer waves a SIMD to
// fill the vector ALU.
bool tall_tiles(int64_t R, int32_t E) { return R / (R < E ? R : E) > 12; }

// Tiles of 128 weight rows by 16 MT activation rows, 4 waves.
template <int MT>
void launch_shape(const ExpertsProduct& a, bool up, int64_t R, hipStream_t stream)
{
    const unsigned grid = (unsigned)(row_tiles(R, a.E, 16 * MT) * ((a.N + BN - 1) / BN)) * a.parts;
    if (up) experts_tile_kernel<true, 4, 1, 2, MT, 3><<<grid, 256, 0, stream>>>(a);
    else experts_tile_kernel<false, 4, 1, 2, MT, 3><<<grid, 256, 0, stream>>>(a);
}

}  // namespace

// Two parts of K where all the tiles of the down product find room at once
// (three a CU) and K is long: 301 tokens, 2 of 8 experts, 4096 x 11008 338 us
// a call undivided, 329 in two parts, 325 in three; 200 tokens, 1024 x 4096 55,
// 47 and 49.  Where they do not, the parts' sums cost more than they fill (600
// tokens, 4 of 16 experts, 4096 x 1408: 132 and 148).
int experts_parts(int64_t R, int32_t E, int32_t H, int32_t I)
{
    const int64_t units = row_tiles(R, E, tall_tiles(R, E) ? 64 : 32) * ((H + BN - 1) / BN);
    return units <= 3 * (int64_t)compute_units() && I / 128 >= 16 ? 2 : 1;
}

void launch_experts_tiled(const ExpertsProduct& a, bool up, int64_t R, hipStream_t stream)
{
    if (tall_tiles(R, a.E)) launch_shape<4>(a, up, R, stream);
    else launch_shape<2>(a, up, R, stream);
}

}  // namespace apex4
