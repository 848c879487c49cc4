// skinny_w4.h -- pieces of the kernels that stream NVFP4 weight rows against a
// few bf16 rows (weight-only products for decode): the per-lane loads of one
// K chunk and the split of an fp32 value into two bf16 halves.
//
// A wave works on fragments of 16 weight rows and 16 activation rows.  Lane l
// (row r = l % 16, group g = l / 16) holds, per chunk of 128 columns, columns
// 32 g .. 32 g + 31 of its weight row (16 bytes) and of its activation row,
// and feeds four v_mfma_f32_16x16x32_bf16 slices from them: the same order of
// K on both operands.  The product lands with activation row l % 16 and weight
// rows 4 (l / 16) .. + 3 in lane l.
#pragma once

#include "device_common.h"
#include "gemm_common.h"

namespace nvfp4 {

constexpr int kChunk = 128;  // columns of a K chunk

// The lane's 32 weight codes of chunk c of the row at `row` (K/2 bytes long),
// zeros past K.  WHOLE: K is a multiple of 128.
template <bool WHOLE>
__device__ __forceinline__ u32x4 load_w4(const uint8_t* row, int c, int g, int rowb) {
    const int kb = c * 64 + g * 16;
    if (WHOLE) return *(const u32x4*)(row + kb);
    const int left = rowb - kb;  // K is a multiple of 16: rowb of 8
    const u32x2 lo = left >= 8 ? *(const u32x2*)(row + kb) : u32x2{0u, 0u};
    const u32x2 hi = left >= 16 ? *(const u32x2*)(row + kb + 8) : u32x2{0u, 0u};
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// Their two block scales (bytes 0 and 1), zero past K.  sf: the matrix's scale
// buffer at the row's own offset (scale_row_off); nblk = K / 16.
template <bool WHOLE>
__device__ __forceinline__ uint32_t load_s4(const uint8_t* sf, int c, int g, int nblk) {
    const int blk = c * 8 + 2 * g;  // even: both blocks sit in one column group of 4
    if (WHOLE) return *(const uint16_t*)(sf + (blk >> 2) * 512 + (blk & 3));
    if (blk >= nblk) return 0u;
    const uint32_t v = *(const uint16_t*)(sf + (blk >> 2) * 512 + (blk & 3));
    return blk + 1 < nblk ? v : v & 0xFFu;
}

// Offset of a row's scales in the swizzled layout (column group 0).
__device__ __forceinline__ int64_t scale_row_off(int64_t row, int cpa4) {
    return (row >> 7) * cpa4 * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4;
}

// The lane's 32 bf16 activations of chunk c, as four slices of 8; zeros past K
// and where `row` is null (an absent row: nothing is read).
template <bool WHOLE>
__device__ __forceinline__ void load_x16(u32x4 v[4], const uint16_t* row, int c, int g, int K) {
    const int k0 = c * kChunk + g * 32;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if (row && (WHOLE || k0 + 8 * j < K)) v[j] = *(const u32x4*)(row + k0 + 8 * j);
    }
}

// f = hi + lo + (at most 2^-16 of f): two bf16 values, each rounded to nearest
// even.  A non-finite f keeps its value in hi and a zero in lo.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(a, b);
    const float ra = a - bf16_lo(hi), rb = b - bf16_hi(hi);
    lo = pack_bf16x2(ra == ra ? ra : 0.0f, rb == rb ? rb : 0.0f);
}

}  // namespace nvfp4
