// How an attention call over the 4-bit cache is cut (kv4_attention.hip), from its
// sizes alone.  Host code without HIP, so that it can be tested where there is no GPU.
#pragma once
#include <algorithm>
#include <cstdint>

namespace apex4 {

constexpr int kWaves = 4;                // of a workgroup
constexpr int kUnit = 64 * kWaves;       // tokens that a workgroup of few rows takes at once
constexpr int kSorted = 256;             // sequences that a workgroup sorts: one a thread
constexpr int64_t kMaxBlocks = (1 << 24) - 1;

// Row tiles of 16 that a wave has where it has rows of its own: two, one for heads of
// 256 numbers, whose sums take twice the registers.
constexpr int row_tiles(int D) { return D == 256 ? 1 : 2; }

struct Cut {
    bool rows;                  // waves have rows of their own
    bool share, sorted;         // (see Plan in kv4_attention.hip)
    int rt, tiles;              // row tiles of 16 a wave; places of a sequence and key head (0: numbered over the batch)
    int64_t blocks;
    bool deep;                  // a row tile may be in many parts
};

// T queries of B sequences, Hkv key heads with `share` query heads each, of D numbers;
// max_q, max_kv, window: include/apex4.h (max_q at least the mean); cus: compute units.
inline Cut kv4_cut(int64_t T, int32_t B, int32_t Hkv, int32_t share, int32_t D, int32_t max_q, int32_t max_kv,
                   int32_t window, int cus)
{
    const int64_t all = (int64_t)max_q * share, pairs = (int64_t)B * Hkv;
    Cut c{};
    c.rt = all <= 16 ? 1 : row_tiles(D);
    // Row tiles of R rows: max_q's for every sequence, or fewer places where the
    // tokens can fill no more (63 decoding sequences and a prompt of 4096: 373 us
    // against 889, a prompt of 512: 64 against 566).  Workgroups stride over what passes the grid's 2^32 threads.
    const auto tile = [&](int64_t R) {
        const int64_t each = (all + R - 1) / R, places = (T * share / R + B) * Hkv;
        const bool uneven = places < pairs * each && places <= kMaxBlocks;
        c.tiles = uneven ? 0 : (int)std::max<int64_t>(1, std::min<int64_t>(each, kMaxBlocks / pairs));
        c.blocks = uneven ? places : pairs * c.tiles;
    };
    tile(16 * c.rt * kWaves);
    c.rows = all > 16 * c.rt && 2 * c.blocks >= 3 * cus;
    if (!c.rows) tile(16 * c.rt);
    if (c.rows) return c;
    // Row tiles of more than 5 units are shared where whole ones leave room for two
    // workgroups a compute unit: 1 x 2048 tokens of 32 heads 11.5 us against 14, 1 x
    // 131071 of 8 heads 34.5 against 675; up to 5 units the second launch costs more
    // (1 x 517 of 32 heads 11.6 us against 8.7), and where the chip is full without it
    // the starts of the parts do (64 x 4096 of 8 heads 54 us against 50).
    // (The tokens that a tile sees count, with a window fewer than those cached.)
    const int64_t seen = window ? std::min<int64_t>(max_kv, (int64_t)window + 16 * c.rt / share) : max_kv;
    const int64_t units = (seen + kUnit - 1) / kUnit, total = c.blocks * units;
    if (units > 5 && c.blocks < 2 * cus) {
        c.share = true;
        c.blocks = std::min<int64_t>(total, 2 * cus);
        // (16 waves for each row where a tile is in more than 8 parts)
        c.deep = units * c.blocks > 8 * total;
    }
    // Whole ones of uneven sequences: the longest first (64 x up to 8192 tokens of 8
    // heads 77 us to 66; not for few units, 64 x up to 512 10 us to 12).
    c.sorted = !c.share && c.tiles && units > 5 && B > 1 && B <= kSorted;
    return c;
}

}  // namespace apex4
