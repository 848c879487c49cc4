// attention_plan.h -- which variant of the attention kernels a call runs: rules on sizes, types
// and alignment, with both sides measured.  Arithmetic of the host alone.
#pragma once

#include <cstdint>

namespace nvfp4 {

// ---- rotary positions ---------------------------------------------------------------

constexpr int64_t kRopeStream = (int64_t)128 << 20;
struct RopePlan {
    bool stream;  // past the caches, where the tensor is larger than they are
    int width;    // elements of a piece
};
inline RopePlan rope_plan(int64_t t, int64_t heads, int64_t d, int64_t pairs) {
    return {t * heads * d * 2 > kRopeStream, pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : 2};
}

// ---- rows of the cache ----------------------------------------------------------------

// Threads of a workgroup, by the blocks there are: 8003 rows of 8 x 128 written and read at 256 /
// 512: 19.8 / 19.0 us, 16 rows: 5.9 / 6.5.
constexpr int kRowThreads = 256, kRowThreadsMany = 512;
constexpr int64_t kRowsMany = 256 * kRowThreadsMany;  // a workgroup a CU
inline int kv_rows_threads(int64_t blocks) { return blocks >= kRowsMany ? kRowThreadsMany : kRowThreads; }

// ---- decode -----------------------------------------------------------------------------

constexpr int64_t kAttnRows = 16;         // query rows of a matrix product
constexpr int64_t kAttnBlock = 64;        // tokens that a wave takes at a time
constexpr int64_t kAttnParts = 512;       // parts that the tokens of all sequences are split into, about
constexpr int64_t kAttnPartsLong = 768;   // the same where they are long
constexpr int64_t kAttnPartsNarrow = 1024;  // the same for heads of up to 64
constexpr int64_t kAttnLong = 4096;       // tokens of a long part, of a sequence twice as long
constexpr int64_t kAttnMinPart = 256;     // fewest tokens of a part
constexpr int64_t kAttnWhole = 1024;      // tokens of a sequence (by the table) that is not split
constexpr int64_t kAttnShared = (int64_t)1 << 18;  // tokens times KV heads from which rows share a read
constexpr int64_t kJoinMany = 1024;       // rows of the output that are joined by a wave each
struct DecodePlan {
    int width;         // of the kernel: 64, 128 or 256
    bool two;          // two products' worths of rows a workgroup
    bool once;         // no other workgroup reads a block
    bool packed;       // rows lie in LDS as they do in memory
    bool large;        // long parts: three workgroups a CU
    bool join;         // a second launch
    int join_waves;    // of a row of the output there
    int64_t row_tiles, split, least, units;  // parts of all sequences, about; fewest blocks of a part; most parts
};
inline DecodePlan decode_plan(int64_t b, int64_t t, int64_t q_heads, int64_t heads, int64_t d, int64_t cap) {
    DecodePlan p{};
    const int64_t rows = t * (q_heads / heads);  // that share a KV head
    p.width = d <= 64 ? 64 : d <= 128 ? 128 : 256;
    // More rows than one product takes: two share a read of the cache where that is much (by the
    // table's size; heads of 256 have no registers for it).  4 x 8 rows over 32 sequences of
    // 8192: 79 us, 114 apart; 4 x 8 over 8 of 8192: 29.6, 34.5; 4 x 8 over 16 of 1024: 16.4, 14.3 (not taken).
    p.two = rows > kAttnRows && d <= 128 && b * heads * cap >= kAttnShared;
    const int64_t tile = p.two ? 2 * kAttnRows : kAttnRows;
    p.row_tiles = (rows + tile - 1) / tile;
    p.once = p.row_tiles == 1;
    p.packed = d % 32 != 0 || 2 * d <= p.width;
    // Long parts (by the table's size, the lengths being on the device) of unequal sequences are
    // better off with three workgroups a CU and cut finer, so that the last ones end together; short
    // ones with four, whose beginnings overlap.  64 sequences to 16384: 119 us against 128; 4 to 131072: 113
    // against 123; 256 to 2048: 89 against 74 (not taken).  Equal long sequences, which the host cannot
    // tell, lose by it: 64 of 16384 each 203 against 196, 4 of 131072 122 against 106, 32 of 8192
    // (32 / 8 heads) 66 against 57.
    // Heads of 64 have half the bytes a wave, so five workgroups a CU and more parts: 32 of 8192:
    // 43 us with 1024 parts, 49 with 512, 47 with 2048.
    const int64_t hrs = heads * p.row_tiles;
    p.large = cap >= 2 * kAttnLong && b * hrs * cap >= kAttnLong * kAttnParts;
    p.split = p.two ? kAttnParts : d <= 64 ? kAttnPartsNarrow : p.large ? kAttnPartsLong : kAttnParts;  // (two: slots twice as large)
    // the most workgroups that lengths up to the table's can ask for
    p.units = (p.split + hrs - 1) / hrs + b;
    // Sequences of up to kAttnWhole stay whole, which saves the second launch (16 of 1000: 12.6 us
    // against 15.0; one alone: 11.9 against 10.7, and 3 us less of the host).
    const int64_t least = cap <= kAttnWhole ? kAttnWhole : kAttnMinPart;
    p.least = least / kAttnBlock;
    const int64_t each = (cap + least - 1) / least;
    if (each * b < p.units) p.units = each * b;
    p.join = each > 1;
    p.join_waves = b * t * q_heads < kJoinMany ? 4 : 1;
    return p;
}

// ---- prompts ------------------------------------------------------------------------------

// Workgroups that share the keys of a tile of rows, by the average sequence: two a CU in all, of 256
// keys or more, where the tiles are few and the keys many.  32 / 8 heads of 128, one sequence of 1 row
// behind 8191 keys: 19.3 us, unshared 95.9; 128 behind 1920: 21.8, 31.1; 512 behind 7680: 87, 110; but
// 700 behind 1300 (tiles for 192 CUs): 44, 33; 4 of 100 behind 1000: 30, 23 (not taken).
constexpr int64_t kPrefillGroups = 512, kPrefillKeys = 256, kPrefillLong = 1536;
constexpr int64_t kPrefillRows = 512 * 129;  // of the parts together
inline int64_t prefill_tiles(int64_t tq, int64_t per, int64_t heads, int64_t b) {
    return b * (((tq / b > 1 ? tq / b : 1) * per + 127) / 128) * heads;
}
// Whether the heads of a group in one tile save one tile in twenty or more.
inline bool prefill_packs(int64_t tq, int64_t q_heads, int64_t heads, int64_t b) {
    return 20 * prefill_tiles(tq, q_heads / heads, heads, b) <= 19 * prefill_tiles(tq, 1, q_heads, b);
}
inline int64_t prefill_parts(int64_t tq, int64_t tk, int64_t q_heads, int64_t heads, int64_t b) {
    const int64_t nk = tk / b;
    const int64_t most = kPrefillGroups / (prefill_packs(tq, q_heads, heads, b) ? prefill_tiles(tq, q_heads / heads, heads, b)
                                                                                : prefill_tiles(tq, 1, q_heads, b));
    if (most < 4 || nk < kPrefillLong) return 1;
    int64_t n = nk / kPrefillKeys < most ? nk / kPrefillKeys : most;
    if (n > 64) n = 64;
    const int64_t room = kPrefillRows / (tq * q_heads);  // of the workspace
    return n < room ? n : room > 1 ? room : 1;
}

struct PrefillPlan {
    int width;      // of the kernel: 64, 128 or 256
    int keys;       // of a tile
    int waves;      // of a workgroup
    int split;      // groups of waves that share a tile's keys
    bool pack;      // the rows of all heads of a group lie in one tile
    int64_t parts;  // workgroups that share a tile's keys
};
inline PrefillPlan prefill_plan(int64_t tq, int64_t tk, int64_t q_heads, int64_t heads, int64_t d, int64_t b, bool causal,
                                bool workspace) {
    // The workgroup, by the average sequence (the lengths themselves are on the device), measured
    // with 32 heads of 128:
    //   * few tiles of rows for the CUs, or few and of unequal work (causal, no long prefix): 128
    //     rows, the keys split (1 prompt of 1024: 21.9 us, 27.8 unsplit; of 2048: 44.6, 53.2; but 4 of 512: 27.9, 24.4; 4 of 300 behind 2000: 68, 66);
    //   * long ones: 256 rows (2 of 2048: 73.5 us, 80.2 with 128 rows; 4 of 300 behind 2000: 58,
    //     66; but 64 of 256: 126, 103);
    //   * others: 128 rows.  (Heads of 64, bound by the softmax's arithmetic, gain nothing from
    //     256 rows: 32 of 1500: 582 us, 421.)
    PrefillPlan p{d <= 64 ? 64 : d <= 128 ? 128 : 256, 64, 4, 1, false, 1};
    const int64_t nq = tq / b > 1 ? tq / b : 1, nk = tk / b, tiles = prefill_tiles(tq, 1, q_heads, b);
    // The heads of a group share a tile where that saves tiles, and these are more than the CUs or the
    // keys are shared too (32 / 8 heads of 128: 128 of 16 rows 20.0 us, 51 apart; 64 of 30 behind
    // 500 keys 39, 81; 16 of 16 behind 4000 60, 99; 8 of 520 behind 1000 115, 121; but one of 61 8.1,
    // 7.2; 8 of 32 behind 1000 26.6, 21.4: a wave beside it slows the chain of a tile's keys).
    p.parts = workspace ? prefill_parts(tq, tk, q_heads, heads, b) : 1;
    p.pack = prefill_packs(tq, q_heads, heads, b) && (p.parts > 1 || tiles > 256);
    if (p.pack || p.parts > 1) {
        if (p.width == 256) p.keys = 32;
        return p;
    }
    const bool split = (tiles <= 256 && nk >= 128) || (tiles <= 512 && nk >= 1024 && nq >= 128 && causal && 2 * tk <= 3 * tq);
    if (p.width <= 128) {
        if (split) p.waves = 8, p.split = 2;
        else if (p.width == 128 && nq >= 256 && nk >= 1024) p.waves = 8;
    } else if (tiles > 256) {
        // Two workgroups a CU where there are more than one (16 / 8 heads: a prompt of 8192
        // 506 us, 757 with one; 64 of 128 62, 79; but 2 of 66 behind 506, 35 / 7 heads, 37.6, 33.2).
        p.keys = 32;
    }
    return p;
}

}  // namespace nvfp4
