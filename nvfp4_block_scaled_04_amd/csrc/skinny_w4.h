// skinny_w4.h -- pieces of the kernels that stream NVFP4 weight rows against a
// few bf16 rows (weight-only products for decode).
//
// A wave works on fragments of 16 weight rows and 16 activation rows.  Lane l
// (row r = l % 16, group g = l / 16) holds, per chunk of 128 columns, columns
// 32 g .. 32 g + 31 of its weight row (16 bytes) and of its activation row,
// and feeds four v_mfma_f32_16x16x32_f16 slices from them: the same order of
// K on both operands.  The product lands with activation row l % 16 and weight
// rows 4 (l / 16) .. + 3 in lane l.
//
// Why fp16: e2m1 times a ue4m3 scale is exact in it and takes half the
// instructions that exact bf16 weights take (one conversion and one packed
// multiplication for two codes).  The activations, bf16 or fp32, become fp16
// when they are put into LDS, scaled by a power of two per row and chunk that
// brings the largest of the 128 columns to [2^14, 2^15): a bf16 value keeps all
// its bits down to 2^-29 of that largest one, and what lies below is off by less
// than 2^-38 of it (a truncation at fp16's least value, 2^-24), far under the fp32
// sums' own rounding.  The chunk's product is scaled back as it is added to the fp32
// accumulators.
//
// The weights come through LDS: every wave has a ring of K chunks of its own, into
// which buffer loads write directly (no registers, no address arithmetic: the
// lane's row is a 32-bit offset that never changes, the chunk a scalar one).  A
// load instruction takes 64 contiguous bytes of 16 rows, lane by lane; the
// fragment is read from LDS in the matrix instruction's order.  A ring runs empty
// where a block of activations is put into LDS: its loads are older than the ring's,
// in a loop, so the compiler's wait for them is for every load under way.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "gemm_common.h"

namespace nvfp4 {

constexpr int kChunk = 128;               // columns of a K chunk
constexpr uint32_t kNoRow = 0x80000000u;  // offset of what is not there: reads zeros (resources are smaller)

__device__ __forceinline__ u32x4 buf_load16(__amdgpu_buffer_rsrc_t rs, uint32_t vo, int so) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)vo, so, 0));
}

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(const lds_byte*)p; }

// ---- activations in LDS ----------------------------------------------------
// A workgroup's waves share the activation rows: `nr` rows of a block of chunks
// sit in LDS as fp16, [chunk][nr][256 bytes], a row of a chunk in 16 pieces of 16
// bytes (8 columns), piece q of row R in slot q ^ R, so that the 16 lanes of a read
// (one piece of 16 rows) touch every bank once; and their inverse scales,
// [chunk][nr] floats.  Loading the rows into each wave's registers from memory
// instead makes them four of every five bytes in flight in a CU and halves the
// rate at which weights arrive.
__device__ __forceinline__ int piece_off(int R, int q) { return R * 256 + ((q ^ R) & 15) * 16; }

// All-reduce over the 16 lanes of a DPP row: the neighbour in a pair, the other
// pair of a quad, the mirrored quad of 8, the mirrored half of 16.
template <typename T, typename F>
__device__ __forceinline__ T row16(T v, F f) {
    auto step = [&](auto ctl) {
        const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctl)::value, 0xF, 0xF, true);
        v = f(v, __builtin_bit_cast(T, o));
    };
    step(std::integral_constant<int, 0xB1>{});
    step(std::integral_constant<int, 0x4E>{});
    step(std::integral_constant<int, 0x141>{});
    step(std::integral_constant<int, 0x140>{});
    return v;
}
__device__ __forceinline__ float row16_max(float v) {
    return row16(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}

// One thread's part of a block on its way from memory to LDS: NV times 8 columns
// of a row of a chunk, the 16 lanes of a DPP row having the chunk between them.
// WIDE: x is fp32 and gives two rows, its high and its low fp16 half (the low one
// `split` rows after the high one); otherwise x is bf16.
template <int NV, bool WIDE>
struct XBlock {
    u32x4 v[NV][WIDE ? 2 : 1];
    uint32_t vo[NV];   // byte offset of the columns in chunk 0 of x
    int c0[NV], ce[NV];  // chunk of x at k0 = 0, end of its range (0: no part in the block)
    int at[NV];        // local chunk and row: lc * nr + R
    int row[NV];

    // Local chunk lc of the block at k0 is chunk first(lc) + k0 of x, up to end(lc);
    // off(R): byte offset of row R in x (rows loaded: nl); nr: rows in LDS.
    template <typename O, typename F, typename E>
    __device__ __forceinline__ void prepare(int nl, int nr, int nlc, int t, int nt, O off, F first, E end) {
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int i = t + u * nt, lc = i / (nl * 16), R = i % (nl * 16) >> 4;
            c0[u] = first(lc);
            ce[u] = lc < nlc ? end(lc) : 0;
            vo[u] = off(R) + (i & 15) * (WIDE ? 32 : 16);
            at[u] = lc * nr + R;
            row[u] = R;
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, int k0, int K, int t) {
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int c = c0[u] + k0;
            const bool in = c < ce[u] && c * kChunk + (t & 15) * 8 < K;  // columns past K are zeros
#pragma unroll
            for (int h = 0; h < (WIDE ? 2 : 1); h++)
                v[u][h] = buf_load16(x, in ? vo[u] + (uint32_t)c * (WIDE ? 512 : 256) + 16 * h : kNoRow, 0);
        }
    }
    __device__ __forceinline__ void store(uint8_t* xs, float* inv, int split, int k0, int t) const {
#pragma unroll
        for (int u = 0; u < NV; u++) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                f[i] = WIDE ? bits_f(v[u][(WIDE ? 1 : 0) * (i >> 2)][i & 3]) : i & 1 ? bf16_hi(v[u][0][i >> 1]) : bf16_lo(v[u][0][i >> 1]);
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) m = __builtin_fmaxf(m, __builtin_fabsf(f[i]));
            m = row16_max(m);
            // biased exponent of the largest value (255 for an infinity, whose row
            // keeps its finite values finite), not below that of 2^-112
            int e = (int)(f_bits(m) >> 23);
            e = e < 15 ? 15 : e;
            const float sc = bits_f((uint32_t)(127 + 14 + 127 - e) << 23);  // 2^(14 - exponent)
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] *= sc;
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const auto hv = __builtin_amdgcn_cvt_pkrtz(f[2 * i], f[2 * i + 1]);
                h[i] = __builtin_bit_cast(uint32_t, hv);
                if (WIDE) {  // an infinity's low half is 0
                    const float r0 = f[2 * i] - (float)hv[0], r1 = f[2 * i + 1] - (float)hv[1];
                    l[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(r0 == r0 ? r0 : 0.0f, r1 == r1 ? r1 : 0.0f));
                }
            }
            if (c0[u] + k0 >= ce[u]) continue;
            uint8_t* const d = xs + (at[u] - row[u]) * 256;
            *(u32x4*)(d + piece_off(row[u], t & 15)) = u32x4{h[0], h[1], h[2], h[3]};
            if (WIDE) *(u32x4*)(d + piece_off(row[u] + split, t & 15)) = u32x4{l[0], l[1], l[2], l[3]};
            if ((t & 15) == 0) inv[at[u]] = bits_f((uint32_t)(e - 14) << 23);  // 2^(exponent - 14)
        }
    }
};

// The lane's addresses of its four pieces of row R in LDS (chunk 0 of a block), and
// of the inverse scale of row Rs.
struct XLane {
    uint32_t a[4], s;
    __device__ __forceinline__ void set(const uint8_t* xs, const float* inv, int R, int Rs, int g) {
#pragma unroll
        for (int j = 0; j < 4; j++) a[j] = lds_addr(xs) + piece_off(R, 4 * g + j);
        s = lds_addr(inv) + Rs * 4;
    }
    // the lane's 32 columns of the chunk whose rows start at row `at` of the block
    __device__ __forceinline__ void read(f16x8 (&x)[4], float& inv, int at) const {
        asm volatile(
            "ds_read_b128 %0, %5\n\tds_read_b128 %1, %6\n\tds_read_b128 %2, %7\n\tds_read_b128 %3, %8\n\tds_read_b32 %4, %9\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(inv)
            : "v"(a[0] + at * 256), "v"(a[1] + at * 256), "v"(a[2] + at * 256), "v"(a[3] + at * 256), "v"(s + at * 4)
            : "memory");
    }
};

// ---- the weight ring of a wave ----------------------------------------------
// Rows of a fragment: tile t takes rows 4 (t % 8) .. + 3 of each of the four 32-row
// quarters of band t / 8 (128 rows).  The scale layout keeps those 16 rows' scales
// of a column group in 64 contiguous bytes; of 16 consecutive rows they would be a
// quarter of 256 bytes (read alone, codes and scales of 8 experts of 16384 x 5120:
// 78.5 us with consecutive rows, 72.8 us with whole lines of scales).
__device__ __forceinline__ int band_row(int tile, int r) { return (tile >> 3) * 128 + (r >> 2) * 32 + (tile & 7) * 4 + (r & 3); }

// NF fragments of 16 weight rows, D chunks in LDS.  `aim` points the loads at a
// matrix and rows, `issue` starts the load of a chunk into the next free slot,
// `take` waits for the oldest one, and run through `consume` multiplies it.  The
// reads of a slot and their wait are one piece of assembly, so that between two
// blocks of activations they wait for the slot's own loads (by the count of loads
// issued since) and not, as the compiler would have it, for every load into LDS.
template <int NF, int D>
struct W4Ring {
    static_assert(NF == 1 || NF == 2, "one scale load covers two fragments");
    static constexpr int SLOT = NF * 1024 + 256;  // codes of NF fragments; scales of two
    static constexpr int BYTES = D * SLOT, DEPTH = D;
    __amdgpu_buffer_rsrc_t w, s;
    uint32_t vw[NF], vs;   // the lane's source offsets of a load
    uint32_t rw, rs;       // the lane's LDS addresses in slot 0
    uint8_t* base;
    int head, tail, ahead; // slot to fill, slot to consume, chunks under way or waiting

    __device__ __forceinline__ void init(uint8_t* ring, int lane) {
        const int r = lane & 15, g = lane >> 4;
        base = ring;
        rw = lds_addr(ring) + r * 64 + ((g ^ swz(r)) << 4);
        rs = lds_addr(ring) + NF * 1024 + (g >> 1) * 64 + ((r & 3) * 4 + (r >> 2)) * 4 + (g & 1) * 2;
        head = tail = ahead = 0;
    }
    // Fragment f: rows first[f] + band_row(tile, 0 .. 15) of the matrix, those from
    // end[f] on read as the last one before it; the codes' offsets count from row0.
    __device__ __forceinline__ void aim(__amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales, const int (&first)[NF],
                                        const int (&end)[NF], int tile, int row0, int rowb, int cpa4, int lane) {
        w = codes;
        s = scales;
        // codes: lane l loads row l / 4's slot l % 4, which holds piece (l % 4) ^ swz(row)
        const int lr = lane >> 2;
#pragma unroll
        for (int f = 0; f < NF; f++) {
            const int x = first[f] + band_row(tile, lr);
            vw[f] = (uint32_t)((x < end[f] ? x : end[f] - 1) - row0) * (uint32_t)rowb + (((lane & 3) ^ swz(lr)) << 4);
        }
        // scales: a dword (4 blocks) per fragment, column group of the chunk and row,
        // in the order of memory (NF = 1: the upper half of the wave loads the same
        // again)
        const int f = NF == 2 && lane >= 32 ? NF - 1 : 0;
        int row = first[f] + band_row(tile, (lane & 3) * 4 + (lane >> 2 & 3));
        row = row < end[f] ? row : end[f] - 1;
        vs = (uint32_t)((row >> 7) * cpa4 * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (lane >> 4 & 1) * 512);
    }
    __device__ __forceinline__ void issue(int c) {
        lds_byte* const dst = (lds_byte*)base + head * SLOT;
#pragma unroll
        for (int f = 0; f < NF; f++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(w, (__attribute__((address_space(3))) void*)(dst + f * 1024), 16, vw[f], c * 64, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(s, (__attribute__((address_space(3))) void*)(dst + NF * 1024), 4, vs, c * 1024, 0, 0);
        head = head + 1 == D ? 0 : head + 1;
        ahead++;
    }
    // The oldest chunk's operands; its slot is free afterwards.
    __device__ __forceinline__ void take(u32x4 (&cw)[NF], uint32_t (&cs)[NF]) {
        // its loads are done when at most those of the chunks after it are left
        if (ahead == D) wait_vmcnt<(D - 1) * (NF + 1)>();
        else wait_vmcnt<0>();
        const uint32_t aw = rw + tail * SLOT, as = rs + tail * SLOT;
        if constexpr (NF == 1)
            asm volatile("ds_read_b128 %0, %2\n\tds_read_u16 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(cw[0]), "=&v"(cs[0])
                         : "v"(aw), "v"(as)
                         : "memory");
        else
            asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:1024\n\tds_read_u16 %2, %5\n\tds_read_u16 %3, %5 offset:128\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(cw[0]), "=&v"(cw[1]), "=&v"(cs[0]), "=&v"(cs[1])
                         : "v"(aw), "v"(as)
                         : "memory");
        tail = tail + 1 == D ? 0 : tail + 1;
        ahead--;
    }
};

// acc[f][i] += fragment f times activation tile i over the chunks [b0, b1) of a
// ring; next() starts the load of the chunk that comes after those under way, if
// there is one.  x: the lane's rows, chunk b0 at row `at` of the block, a chunk
// every `step` rows.  WHOLE: K is a multiple of 128; otherwise the scales of blocks
// past K count as zero (their codes may be the next row's).
template <int XT, bool WHOLE, int NF, int D, typename F>
__device__ __forceinline__ void consume(W4Ring<NF, D>& ring, f32x4 (&acc)[NF][XT], const XLane (&x)[XT], int at, int step, int b0,
                                        int b1, int g, int K, F next) {
    for (int c = b0; c < b1; c++) {
        u32x4 cw[NF];
        uint32_t cs[NF];
        ring.take(cw, cs);
        next();
        f16x8 xv[XT][4];
        float inv[XT];
#pragma unroll
        for (int i = 0; i < XT; i++) x[i].read(xv[i], inv[i], at);
        at += step;
        if (!WHOLE) {
            const int left = K - c * kChunk - 32 * g;
            const uint32_t keep = left >= 32 ? 0xFFFFu : left >= 16 ? 0xFFu : 0u;
#pragma unroll
            for (int f = 0; f < NF; f++) cs[f] &= keep;
        }
        f32x4 t[NF][XT];
#pragma unroll
        for (int f = 0; f < NF; f++) {
            const f16x2 s2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(cs[f], 1.0f, false);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const f16x8 wv = dequant8(word(cw[f], j), s2[j >> 1]);
#pragma unroll
                for (int i = 0; i < XT; i++)
                    t[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, xv[i][j], j ? t[f][i] : f32x4{0, 0, 0, 0}, 0, 0, 0);
            }
        }
#pragma unroll
        for (int f = 0; f < NF; f++)
#pragma unroll
            for (int i = 0; i < XT; i++) acc[f][i] += t[f][i] * inv[i];
    }
}

}  // namespace nvfp4
