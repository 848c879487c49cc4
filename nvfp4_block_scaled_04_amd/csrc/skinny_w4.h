// skinny_w4.h -- pieces of the kernels that stream NVFP4 weight rows against a
// few bf16 rows (weight-only products for decode), and the split of an fp32
// value into two bf16 halves.
//
// A wave works on fragments of 16 weight rows and 16 activation rows.  Lane l
// (row r = l % 16, group g = l / 16) holds, per chunk of 128 columns, columns
// 32 g .. 32 g + 31 of its weight row (16 bytes) and of its activation row,
// and feeds four v_mfma_f32_16x16x32_bf16 slices from them: the same order of
// K on both operands.  The product lands with activation row l % 16 and weight
// rows 4 (l / 16) .. + 3 in lane l.
//
// The weights come through LDS: every wave has a ring of K chunks of its own, into
// which buffer loads write directly (no registers, no address arithmetic: the
// lane's row is a 32-bit offset that never changes, the chunk a scalar one).  A
// load instruction takes 64 contiguous bytes of 16 rows, lane by lane; the
// fragment is read from LDS in the matrix instruction's order.
#pragma once

#include "device_common.h"
#include "gemm_common.h"

namespace nvfp4 {

constexpr int kChunk = 128;               // columns of a K chunk
constexpr uint32_t kNoRow = 0x80000000u;  // offset of what is not there: reads zeros (resources are smaller)

__device__ __forceinline__ u32x4 buf_load16(__amdgpu_buffer_rsrc_t rs, uint32_t vo, int so) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)vo, so, 0));
}

// f = hi + lo + (at most 2^-16 of f): two bf16 values, each rounded to nearest
// even.  A non-finite f keeps its value in hi and a zero in lo.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(a, b);
    const float ra = a - bf16_lo(hi), rb = b - bf16_hi(hi);
    lo = pack_bf16x2(ra == ra ? ra : 0.0f, rb == rb ? rb : 0.0f);
}

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(const lds_byte*)p; }

// ---- activations in LDS ----------------------------------------------------
// A workgroup's waves share the activation rows: `nr` rows of a block of chunks
// sit in LDS, [chunk][nr][256 bytes], a row of a chunk in 16 pieces of 16 bytes (8
// columns), piece q of row R in slot q ^ R, so that the 16 lanes of a read (one
// piece of 16 rows) touch every bank once.  Loading the rows into each wave's
// registers from memory instead makes them four of every five bytes in flight
// in a CU and halves the rate at which weights arrive.
__device__ __forceinline__ int piece_off(int R, int q) { return R * 256 + ((q ^ R) & 15) * 16; }

// One thread's part of a block, NV pieces of 16 bytes, on its way from memory to
// LDS.  Local chunk lc of the block is chunk lo(lc) of K, or none where that is
// negative; off(R) is the byte offset of row R in x.  Columns past K are zeros.
template <int NV>
struct XBlock {
    u32x4 v[NV];

    template <typename O, typename F>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, O off, int nr, int nlc, int K, int t, int nt, F lo) {
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int i = t + u * nt, lc = i / (nr * 16), R = i % (nr * 16) >> 4;
            const int c = lc < nlc ? lo(lc) : -1, col = c * kChunk + (i & 15) * 8;
            v[u] = buf_load16(x, c >= 0 && col < K ? off(R) + 2 * col : kNoRow, 0);
        }
    }
    __device__ __forceinline__ void store(uint8_t* dst, int nr, int nlc, int t, int nt) const {
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int i = t + u * nt, lc = i / (nr * 16), R = i % (nr * 16) >> 4;
            if (lc < nlc) *(u32x4*)(dst + lc * nr * 256 + piece_off(R, i & 15)) = v[u];
        }
    }
};

// The lane's addresses of its four pieces of a row in LDS (chunk 0 of a block).
struct XLane {
    uint32_t a[4];
    __device__ __forceinline__ void set(const uint8_t* xs, int R, int g) {
#pragma unroll
        for (int j = 0; j < 4; j++) a[j] = lds_addr(xs) + piece_off(R, 4 * g + j);
    }
    // the lane's 32 columns of the chunk at byte `at` of the block
    __device__ __forceinline__ void read(bf16x8 (&x)[4], int at) const {
        asm volatile(
            "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
            : "v"(a[0] + at), "v"(a[1] + at), "v"(a[2] + at), "v"(a[3] + at)
            : "memory");
    }
};

// ---- the weight ring of a wave ----------------------------------------------
// NF fragments of 16 weight rows, D chunks in LDS.  `aim` points the loads at a
// matrix and rows, `issue` starts the load of a chunk into the next free slot,
// `take` waits for the oldest one, and run through `consume` multiplies it.  The
// reads of a slot and their wait are one piece of assembly, so that they wait for
// the slot's own loads (by the count of loads issued since) and not, as the
// compiler would have it, for every load into LDS.
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
        rs = lds_addr(ring) + NF * 1024 + r * 8 + 2 * g;
        head = tail = ahead = 0;
    }
    // row0[f]: first row of fragment f
    __device__ __forceinline__ void aim(__amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales, const int (&row0)[NF], int rowb,
                                        int cpa4, int lane) {
        w = codes;
        s = scales;
        // codes: lane l loads row l / 4's slot l % 4, which holds piece (l % 4) ^ swz(row)
        const int lr = lane >> 2;
#pragma unroll
        for (int f = 0; f < NF; f++)
            vw[f] = (uint32_t)(row0[f] + lr) * (uint32_t)rowb + (((lane & 3) ^ swz(lr)) << 4);
        // scales: a dword (4 blocks) per fragment, row and column group of the chunk
        // (NF = 1: the upper half of the wave loads the same again)
        const int sr = (lane & 31) >> 1;
        const int row = (NF == 2 && lane >= 32 ? row0[NF - 1] : row0[0]) + sr;
        vs = (uint32_t)((row >> 7) * cpa4 * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (lane & 1) * 512);
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
// there is one.  x: the lane's rows, chunk b0 at byte x_at, a chunk every x_step
// bytes.  WHOLE: K is a multiple of 128; otherwise the scales of blocks past K
// count as zero (their codes may be the next row's).
template <int XT, bool WHOLE, int NF, int D, typename F>
__device__ __forceinline__ void consume(W4Ring<NF, D>& ring, f32x4 (&acc)[NF][XT], const XLane (&x)[XT], int x_at, int x_step, int b0,
                                        int b1, int g, int K, F next) {
    for (int c = b0; c < b1; c++) {
        u32x4 cw[NF];
        uint32_t cs[NF];
        ring.take(cw, cs);
        next();
        bf16x8 xv[XT][4];
#pragma unroll
        for (int i = 0; i < XT; i++) x[i].read(xv[i], x_at);
        x_at += x_step;
        if (!WHOLE) {
            const int left = K - c * kChunk - 32 * g;
            const uint32_t keep = left >= 32 ? 0xFFFFu : left >= 16 ? 0xFFu : 0u;
#pragma unroll
            for (int f = 0; f < NF; f++) cs[f] &= keep;
        }
#pragma unroll
        for (int f = 0; f < NF; f++) {
            const float s0 = __builtin_amdgcn_cvt_f32_fp8(cs[f], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(cs[f], 1);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bf16x8 wv = dequant8_bf16(word(cw[f], j), j < 2 ? s0 : s1);
#pragma unroll
                for (int i = 0; i < XT; i++)
                    acc[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv[i][j], acc[f][i], 0, 0, 0);
            }
        }
    }
}

}  // namespace nvfp4
