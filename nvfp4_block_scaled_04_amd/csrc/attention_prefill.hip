// attention_prefill.hip -- attention of whole prompts, packed one after the
// other: grouped heads, causal or full, keys that reach further back than the queries.
//
// For a query row i of a sequence, over the keys j that it sees:
//   s_j = q_i . k_j, p_j = 2^(s_j * c - m), out_i = sum p_j v_j / sum p_j,
// c = scale * log2(e), one pass over the keys with the running maximum m and sum.
//
// A workgroup of four or eight waves takes 128 or 256 rows of one head (or of the heads of a group),
// a wave 32 of them (see prefill_plan).  64 keys and values at a time (32 for most heads
// of 256) go straight from memory into LDS (two buffers), swizzled at their source so that neither
// product's reads collide in the banks.  Both products run on 32x32x16 bf16 MFMAs, transposed:
//   S^T[key, row] = K Q^T: a lane owns one row (and half of the keys), so the softmax
//   needs one exchange between lanes, and only where the maximum moves;
//   O^T[column, row] = V^T P^T: V^T comes from transposing LDS reads, in the order of
//   keys in which a lane holds its column of S^T, so P stays where it is.
// What bounds it: a prompt of 8192, 40 heads of 128, 600 us, 1.14 PFLOP/s: the card's power (on zeros
// 480 us; the library's product of 8192^3 runs at 1.24-1.32 on such data, 1.76 on zeros); heads of 64
// the softmax's arithmetic; short prompts the chain of a tile's keys.  Where few rows meet many
// keys, workgroups share the keys (prefill_parts).
// Sums, maximum and both products' sums are fp32; P is rounded to bf16 (V's range is
// bf16's), off by 2^-8 of itself at most, as the output is.  No P is above one (kLag), so that sums of
// values near bf16's largest stay within fp32 as far as a softmax in fp32 goes.
#include <type_traits>

#include "gemm_common.h"
#include "internal.h"

namespace nvfp4 {

namespace {

// LDS: two tiles of K and two of V for each of SPLIT groups of waves, the queries behind them where
// eight waves have rows of their own.  With 32 keys a wave's queries are as large as a tile, and
// four waves take a tile more.
template <int D, int KEYS, int NW, int SPLIT>
constexpr int lds_bytes() {
    return 4 * SPLIT * KEYS * D * 2 + (NW / SPLIT == 8 ? 8 * 64 * D : KEYS == 32 ? 64 * D : 0);
}

// A row's maximum m is moved only where a score exceeds it by more than kLag, to the largest score (on a
// grid on which m + kLag is exact); a probability is 2^(score - m - kLag), one at most.  (2^kLag times a
// value of 2^120 would pass fp32.)
constexpr int kLag = 8;

struct PParams {
    const uint16_t *q, *k, *v;
    uint16_t* out;
    float* lse;                // [tq, Hq] or null
    float* part;               // [parts, tq, Hq, D + 4] sums, maximum, sum of the probabilities
    const int32_t *cu_q, *cu_k;
    int64_t q_stride, k_stride, v_stride, out_stride;
    float c;                   // scale * log2(e)
    int b, tq, tk, Hq, H, G, d, causal, parts;
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// A sequence's rows and keys; offsets that do not ascend or leave the tensors are clamped.
struct Seq {
    int q0, nq, k0, nk;
};

__device__ __forceinline__ Seq seq_at(const PParams& p, int i) {
    Seq s;
    s.q0 = clamp_to(p.cu_q[i], 0, p.tq);
    s.nq = clamp_to(p.cu_q[i + 1], s.q0, p.tq) - s.q0;
    s.k0 = clamp_to(p.cu_k[i], 0, p.tk);
    s.nk = clamp_to(p.cu_k[i + 1], s.k0, p.tk) - s.k0;
    return s;
}

// The sequence and tile of rows (`per` heads each) of unit `unit`; a sequence's last tiles, which have the
// most keys, come first.
template <int ROWS>
__device__ __forceinline__ bool find_tile(const PParams& p, int unit, int per, Seq& s, int& tile) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base < p.b; base += 64) {
        const int i = base + lane;
        Seq mine = {};
        if (i < p.b) mine = seq_at(p, i);
        const int n = (mine.nq * per + ROWS - 1) / ROWS;
        const int sum = wave_scan(n);
        const uint64_t hit = __ballot(before + sum > unit);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            s.q0 = __builtin_amdgcn_readlane(mine.q0, l);
            s.nq = __builtin_amdgcn_readlane(mine.nq, l);
            s.k0 = __builtin_amdgcn_readlane(mine.k0, l);
            s.nk = __builtin_amdgcn_readlane(mine.nk, l);
            tile = before + __builtin_amdgcn_readlane(sum, l) - 1 - unit;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// 16-byte chunk c of row r of a staged tile lies in chunk c ^ swizzle(r): K so that 16
// consecutive rows put one chunk into 16 bank groups, V so that four rows put
// 64 bytes into four.
template <int D>
__device__ __forceinline__ int swizzle_k(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
template <int D>
__device__ __forceinline__ int swizzle_v(int r) { return D == 64 ? (r & 2) << 1 : (r & 3) << 2; }

// 16 bytes a lane from a raw buffer into LDS, lane after lane from `lds` on.  In assembly, since
// behind its own intrinsic the compiler waits for these loads at every LDS read, also of the
// other buffer.  (It writes no register; the compiler's own waits count it as one load more,
// which only makes them longer.  The s_nop covers m0 and a descriptor that a vector instruction has
// just written.)
__device__ __forceinline__ void load_to_lds(const u32x4& rsrc, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(rsrc), "s"(lds) : "memory", "m0");
}

__device__ __forceinline__ u32x4 raw_buffer(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)base;
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// NW: waves of a workgroup.  Eight waves sit two to a SIMD and take turns (sweep_paired).
// SPLIT: 1: each wave has 32 rows of its own; 2: the second four waves have the rows of
// the first, which take every other tile of keys, and the halves are joined at the end.
// PARTS: p.parts workgroups share a tile's keys, in stretches, and k_join_parts joins them.
// PACK: the rows of all heads of a group lie in one tile, one after the other (row n is head n % G of
// its token n / G), and share the keys that it reads.
// KEYS: of a tile.  With 32, two workgroups of heads of 256 share a CU (512 registers and 160 KB),
// with 64, one has them alone.  (With 32, 33 registers spill, 55 with PACK: before and behind the
// loop over the keys and in the second pass, none in the loop.)
template <int D, int KEYS, int NW, int SPLIT, bool PARTS, bool PACK>
__global__ __launch_bounds__(64 * NW, D * KEYS <= 128 * 64 ? 2 : 1) void k_attn_prefill(PParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int NS = KEYS / 32, NP = KEYS / 16;
    constexpr int CH = D / 8;                   // chunks of a row
    constexpr int TILE = KEYS * D * 2;          // bytes of a tile of K (of V)
    constexpr int OWN = 32 * D * 2;             // of a wave's 32 rows
    constexpr int GW = NW / SPLIT;              // waves of a group, which share tiles
    constexpr int LOADS = KEYS * CH / (64 * GW);  // of a lane, of K (of V)
    constexpr int ROWS = GW * 32;
    extern __shared__ __align__(16) uint8_t smem[];  // lds_bytes
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = SPLIT == 1 ? 0 : wave / GW, gw = SPLIT == 1 ? wave : wave % GW;
    const int l32 = lane & 31, hi = lane >> 5;

    // Workgroups are dealt to the 8 XCDs in turn: where the heads split evenly, an XCD
    // has KV heads of its own, whose keys and values stay in its L2.
    const int heads = PACK ? p.H : p.Hq, group = PACK ? p.G : 1;  // (heads of a row)
    int head, unit, part = 0;
    if (p.H % 8 == 0) {
        const int per = heads / 8, r = blockIdx.x >> 3;
        head = (blockIdx.x & 7) * per + r % per;
        unit = r / per;
    } else {
        head = blockIdx.x % heads;
        unit = blockIdx.x / heads;
    }
    if constexpr (PARTS) {
        part = unit % p.parts;
        unit /= p.parts;
    }
    Seq sq;
    int tile;
    if (!find_tile<ROWS>(p, unit, group, sq, tile)) return;
    const int kv = PACK ? head : head / p.G;
    if (PACK) head *= p.G;                      // the row's first
    const int nrows = sq.nq * group;
    auto token = [&](int row) { return PACK ? row / p.G : row; };
    const int back = sq.nk - sq.nq;             // row i sees the keys up to i + back
    const int row0 = tile * ROWS;
    int keys = sq.nk;                           // that any row of the tile sees
    if (p.causal) {
        const int last = row0 + ROWS < nrows ? row0 + ROWS : nrows;
        keys = clamp_to(token(last - 1) + 1 + back, 0, sq.nk);
    }

    const uint16_t* const kb = p.k + (int64_t)sq.k0 * p.k_stride + kv * p.d;
    const uint16_t* const vb = p.v + (int64_t)sq.k0 * p.v_stride + kv * p.d;
    lds_u8* const lds = (lds_u8*)smem + grp * 4 * TILE;  // the group's tiles
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds + gw * 1024;
    // a lane's offsets into a tile in memory: a row past the last one ends behind the buffer by
    // itself, a chunk past d is sent there
    uint32_t off_k[LOADS], off_v[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
        const int piece = (i * GW + gw) * 64 + lane;
        const int r = piece / CH, at = piece % CH;
        const int ck = at ^ swizzle_k<D>(r), cv = at ^ swizzle_v<D>(r);
        off_k[i] = ck * 8 < p.d ? (uint32_t)(r * (int)p.k_stride + ck * 8) * 2u : 0xFFFFFFF0u;
        off_v[i] = cv * 8 < p.d ? (uint32_t)(r * (int)p.v_stride + cv * 8) * 2u : 0xFFFFFFF0u;
    }
    // the group's n-th tile of keys
    int tile0 = 0, tile1 = (keys + KEYS - 1) / KEYS;
    if constexpr (PARTS) {
        const int all_tiles = tile1;
        tile0 = (int)((int64_t)all_tiles * part / p.parts);
        tile1 = (int)((int64_t)all_tiles * (part + 1) / p.parts);
    }
    auto key_of = [&](int n) { return PARTS ? (tile0 + n) * KEYS : (n * SPLIT + grp) * KEYS; };
    auto stage = [&](const uint16_t* base, int64_t stride, const uint32_t (&off)[LOADS], int key0, uint32_t to) {
        const int rows = sq.nk - key0 < KEYS ? sq.nk - key0 : KEYS;  // at least 1; later rows come as zeros
        const u32x4 rs = raw_buffer(base + key0 * stride, (uint32_t)(((rows - 1) * stride + p.d) * 2));
#pragma unroll
        for (int i = 0; i < LOADS; i++) load_to_lds(rs, off[i], __builtin_amdgcn_readfirstlane(lds0 + to + i * GW * 1024));
    };
    auto stage_k = [&](int n) { stage(kb, p.k_stride, off_k, key_of(n), (n & 1) * TILE); };
    auto stage_v = [&](int n) { stage(vb, p.v_stride, off_v, key_of(n), (2 + (n & 1)) * TILE); };
    auto tiles_of = [&](int upto) { return (upto + KEYS * (SPLIT - grp) - 1) / (KEYS * SPLIT); };  // of the group, of the keys below
    const int tiles = PARTS ? tile1 - tile0 : tiles_of(keys), steps = PARTS ? tiles : (keys + KEYS * SPLIT - 1) / (KEYS * SPLIT);
    if (tiles > 0) stage_k(0);

    // The wave's 32 rows of q go through LDS too, in whole lines (fragments straight from memory
    // would touch every line four times): behind the tiles, or, with four waves a
    // group, where tiles after the first of K will be.
    const int first = row0 + gw * 32;
    lds_u8* const mine_q = lds + (GW == 8 ? 4 * TILE + gw * OWN : KEYS == 32 ? (1 + gw) * TILE : (gw < 2 ? TILE : 3 * TILE) + (gw & 1) * OWN);
    {
        const int rows = nrows - first;  // those behind the sequence come as zeros
        const int t0 = token(first), t1 = token(first + (rows < 32 ? rows : 32) - 1);
        const u32x4 rs = raw_buffer(p.q + (int64_t)(sq.q0 + t0) * p.q_stride + head * p.d,
                                    rows > 0 ? (uint32_t)(((t1 - t0) * p.q_stride + group * p.d) * 2) : 0u);
#pragma unroll
        for (int i = 0; i < 32 * CH / 64; i++) {
            const int piece = i * 64 + lane;
            const int r = piece / CH, c = (piece % CH) ^ swizzle_k<D>(r);
            const int t = PACK ? token(first + r) - t0 : r, h = PACK ? first + r - (t + t0) * p.G : 0;
            load_to_lds(rs, c * 8 < p.d && (!PACK || r < rows) ? (uint32_t)(t * (int)p.q_stride + h * p.d + c * 8) * 2u : 0xFFFFFFF0u,
                        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)mine_q + i * 1024));
        }
    }
    const int mine = first + l32;
    const int end = mine >= nrows ? 0 : p.causal ? clamp_to(token(mine) + back + 1, 0, sq.nk) : sq.nk;  // keys below it are seen
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    bf16x8 q[D / 16];
#pragma unroll
    for (int s = 0; s < D / 16; s++)
        q[s] = *(const __attribute__((address_space(3))) bf16x8*)(mine_q + l32 * D * 2 + ((2 * s + hi) ^ swizzle_k<D>(l32)) * 16);
    // (waited for here, not at every use in the loop)
#pragma unroll
    for (int s = 0; s < D / 16; s++) asm volatile("" : "+v"(q[s]));
    // (some lie where the first tile of V goes)
    if constexpr (KEYS == 32) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // keys that all rows of the wave see, and that any sees (rows past the sequence count as its last)
    int all = sq.nk, any = sq.nk;
    if (p.causal) {
        all = clamp_to(token(first) + back + 1, 0, sq.nk);
        any = clamp_to(token((first + 32 < nrows ? first + 32 : nrows) - 1) + 1 + back, 0, sq.nk);
    }
    if (first >= nrows) any = 0;

    f32x16 o[D / 32];
    float m = neg_inf(), l = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; i++) o[i] = f32x16{};

    // a lane's V rows: 4 hi + (lane & 15) / 4 (+ 8 i)
    const int vr = (lane & 15) >> 2;
    constexpr int VA = D / 32 < 4 ? D / 32 : 4;  // (the swizzle stays within 16 chunks)
    int vat[VA];
#pragma unroll
    for (int i = 0; i < VA; i++) {
        const int c = 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        vat[i] = (4 * hi + vr) * D * 2 + (c ^ swizzle_v<D>(vr)) * 16 + (lane & 1) * 8;
    }
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x4 __attribute__((ext_vector_type(4)));

    // S^T of tile n: s[j] the keys 32 j .. of it
    auto scores = [&](int n, f32x16 (&s)[NS]) {
        lds_u8* const kt = lds + (n & 1) * TILE;
#pragma unroll
        for (int j = 0; j < NS; j++) {
            s[j] = f32x16{};
#pragma unroll
            for (int i = 0; i < D / 16; i++) {
                const int r = 32 * j + l32;
                const bf16x8 a = *(const __attribute__((address_space(3))) bf16x8*)(kt + r * D * 2 + ((2 * (i % 8) + hi) ^ swizzle_k<D>(r)) * 16 + i / 8 * 256);
                s[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[i], s[j], 0, 0, 0);
            }
        }
    };
    // its probabilities: pf[f] the keys 16 f .. of it.  FAR: by far_score in the rows whose scores are
    // that large.
    auto soften = [&](auto FAR, int n, f32x16 (&s)[NS], bf16x8 (&pf)[NP]) {
        const int key0 = key_of(n);
        if (key0 + KEYS > all) {
#pragma unroll
            for (int e = 0; e < 16 * NS; e++)
                if (key0 + 32 * (e >> 4) + 8 * ((e & 15) >> 2) + 4 * hi + (e & 3) >= end) s[e >> 4][e & 15] = neg_inf();
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < 16 * NS; e++) top = __builtin_fmaxf(top, s[e >> 4][e & 15]);
        top *= p.c;
        // (moved by the row alone, so that its bits do not depend on the rows beside it)
        if (__any(top > m + kLag)) {
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float to = top > m + kLag ? (top + kLag) - kLag : m;
            const float a = to == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= a;
#pragma unroll
            for (int i = 0; i < D / 32; i++) o[i] *= a;
        }
        const float most = m == neg_inf() ? 0.0f : m;
        float base = most + kLag, c = p.c;
        if constexpr (FAR) {
            const bool far = __builtin_fabsf(most) >= kFarScore;
#pragma unroll
            for (int e = 0; e < 16 * NS; e++) s[e >> 4][e & 15] = far ? far_score(s[e >> 4][e & 15], c, most) : s[e >> 4][e & 15];
            base = far ? kLag : base;
            c = far ? 1.0f : c;
        }
        float sum = 0.0f;
#pragma unroll
        for (int f = 0; f < NP; f++) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[f >> 1][8 * (f & 1) + 2 * e], c, -base));
                const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[f >> 1][8 * (f & 1) + 2 * e + 1], c, -base));
                sum += p0 + p1;
                w[e] = pack_bf16x2(p0, p1);
            }
            pf[f] = __builtin_bit_cast(bf16x8, w);
        }
        l += sum;
    };
    auto v_frag = [&](lds_u8* vt, int f, int i) {  // V^T of the keys 16 f .. and the columns 32 i ..
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(vt + vat[i % VA] + i / VA * 256 + 16 * f * D * 2));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(vt + vat[i % VA] + i / VA * 256 + (16 * f + 8) * D * 2));
        const bf16x4 x = __builtin_bit_cast(bf16x4, a), y = __builtin_bit_cast(bf16x4, b);
        return bf16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    };
    auto add_values = [&](int n, const bf16x8 (&pf)[NP]) {
        lds_u8* const vt = lds + (2 + (n & 1)) * TILE;
#pragma unroll
        for (int f = 0; f < NP; f++)
#pragma unroll
            for (int i = 0; i < D / 32; i++) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_frag(vt, f, i), pf[f], o[i], 0, 0, 0);
    };

    // One pass over the keys, each wave by itself between the tiles' barriers.  CAREFUL: a value
    // that is not finite behind a mask, which 0 times it would carry into the rows that do not
    // see it, is kept out of the product and handed to the rows that do; scores past kFarScore.
    auto sweep = [&](auto CAREFUL) {
        if (tiles > 0) stage_v(0);
        for (int n = 0; n < steps; n++) {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the tile is there, the other buffers have been read
            if (n + 1 < tiles) {
                stage_k(n + 1);
                stage_v(n + 1);
            }
            const int key0 = key_of(n);
            if (key0 >= any) continue;
            f32x16 s[NS];
            bf16x8 pf[NP];
            scores(n, s);
            soften(CAREFUL, n, s, pf);
            if constexpr (!CAREFUL) {
                add_values(n, pf);
            } else {
                lds_u8* const vt = lds + (2 + (n & 1)) * TILE;
#pragma unroll 1
                for (int f = 0; f < NP; f++)
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        u32x4 w = __builtin_bit_cast(u32x4, v_frag(vt, f, i));
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u;
                            if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu;
                        }
                        bf16x8 pv = pf[0];
                        pv = f == 1 ? pf[1] : f == 2 ? pf[2 % NP] : f == 3 ? pf[3 % NP] : pv;
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), pv, o[i], 0, 0, 0);
                    }
                u16x2 big = {};
#pragma unroll 1
                for (int i = lane; i < TILE / 16; i += 64) {
                    const u32x4 w = *(const __attribute__((address_space(3))) u32x4*)(vt + i * 16);
#pragma unroll
                    for (int e = 0; e < 4; e++) big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, w[e] & 0x7FFF7FFFu));
                }
                if (__any((big[0] > big[1] ? big[0] : big[1]) >= 0x7F80)) {
#pragma unroll 1
                    for (int r = 0; r < KEYS; r++)
#pragma unroll
                        for (int i = 0; i < D / 32; i++)
#pragma unroll
                            for (int e = 0; e < 16; e++) {
                                const int col = 32 * i + 8 * (e >> 2) + 4 * hi + (e & 3);
                                const uint16_t bits = *(const __attribute__((address_space(3))) uint16_t*)(
                                    vt + r * D * 2 + ((col >> 3) ^ swizzle_v<D>(r)) * 16 + (col & 7) * 2);
                                if ((bits & 0x7F80) == 0x7F80 && key0 + r < end) o[i][e] += bits_f((uint32_t)bits << 16);
                            }
                }
            }
        }
    };

    // The same with two waves of a SIMD in step: while one runs the products of a tile (V of the
    // one before, then K of this), the other runs the softmax of its own, so that the matrix
    // pipe is always fed.  A barrier ends each half of a step; the second four waves are half a
    // step behind.  Step n stages K of n + 1 and V of n, which are read a step later, into buffers
    // last read in the step before.
    auto sweep_paired = [&]() {
        const bool behind = wave >= NW / 2;
        const int own = tiles_of(any);  // tiles that the wave sees
        f32x16 s[NS];
        bf16x8 pf[NP];
        auto end_half = [&](auto LANDED) {
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (LANDED) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        auto feed = [&](int n) {
            if (n + 1 < tiles) stage_k(n + 1);
            if (n < tiles) stage_v(n);
        };
        // LDS reads run ahead of the products: the compiler alone puts each right before its use
        auto products = [&](int n) {
            add_values(n - 1, pf);
            scores(n, s);
            constexpr int NV = D / 32 * NP, NK = D / 16 * NS;  // products of each
            __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
            for (int i = 0; i < NV - 4; i++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
#pragma unroll
            for (int i = 0; i < NK - 8; i++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
        };
        // Step n: K of tile n meets the queries, V of tile n - 1 the probabilities.
        end_half(std::true_type{});  // K of tile 0 is there
        int n = 0;
        if (own > 0) {
            feed(0);
            if (!behind) {
                scores(0, s);
                end_half(std::false_type{});
                soften(std::false_type{}, 0, s, pf);
                end_half(std::true_type{});
                for (n = 1; n < own; n++) {
                    feed(n);
                    products(n);
                    end_half(std::false_type{});
                    soften(std::false_type{}, n, s, pf);
                    end_half(std::true_type{});
                }
                feed(n);
                add_values(n - 1, pf);
                end_half(std::false_type{});
            } else {
                end_half(std::false_type{});
                scores(0, s);
                end_half(std::true_type{});
                for (n = 1; n < own; n++) {
                    feed(n);
                    soften(std::false_type{}, n - 1, s, pf);
                    end_half(std::false_type{});
                    products(n);
                    end_half(std::true_type{});
                }
                feed(n);
                soften(std::false_type{}, n - 1, s, pf);
                end_half(std::false_type{});
                add_values(n - 1, pf);
            }
            end_half(std::true_type{});
            n++;
        }
        for (; n <= steps; n++) {  // tiles that only other waves see
            feed(n);
            end_half(std::false_type{});
            end_half(std::true_type{});
        }
    };
    if constexpr (NW == 8) sweep_paired();
    else sweep(std::false_type{});

    // Again, carefully, where an output is not finite or a row's scores are so large that their maximum's
    // rounding counts (a maximum that was as far below has left nothing, or what is not finite).
    bool again = m != neg_inf() && __builtin_fabsf(m) >= kFarScore;
#pragma unroll
    for (int i = 0; i < D / 32; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) again |= (f_bits(o[i][e]) & 0x7F800000u) == 0x7F800000u;
    __attribute__((address_space(3))) int* const flags = (__attribute__((address_space(3))) int*)smem;
    again = __any(again);
    __syncthreads();
    if (lane == 0) flags[wave] = again;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; i++) again |= flags[i] != 0;
    if (again) {
        __syncthreads();
        m = neg_inf();
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; i++) o[i] = f32x16{};
        if (tiles > 0) stage_k(0);
        sweep(std::true_type{});
    }

    __syncthreads();  // the tiles have been read
    if constexpr (SPLIT == 2) {  // the second group's sums to the first, lane by lane
        lds_u8* const all_lds = (lds_u8*)smem;
        __attribute__((address_space(3))) f32x4* const sums = (__attribute__((address_space(3))) f32x4*)(all_lds + (4 + gw) * TILE) + lane;
        __attribute__((address_space(3))) float* const stats = (__attribute__((address_space(3))) float*)(all_lds + 2 * TILE + gw * 512) + lane;
        if (grp == 1) {
#pragma unroll
            for (int i = 0; i < D / 32; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) sums[(4 * i + e) * 64] = f32x4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
            stats[0] = m;
            stats[64] = l;
        }
        __syncthreads();
        if (grp == 1) return;
        const float m1 = stats[0], to = __builtin_fmaxf(m, m1);
        const float a0 = to == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m - to), a1 = to == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m1 - to);
        l = l * a0 + stats[64] * a1;
        m = to;
#pragma unroll
        for (int i = 0; i < D / 32; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const f32x4 v = sums[(4 * i + e) * 64];
#pragma unroll
                for (int j = 0; j < 4; j++) o[i][4 * e + j] = o[i][4 * e + j] * a0 + v[j] * a1;
            }
    }
    const float den = l + __shfl_xor(l, 32);
    if constexpr (PARTS) {
        if (mine >= nrows) return;
        const int t = token(mine);
        float* const to = p.part + (((int64_t)part * p.tq + sq.q0 + t) * p.Hq + head + (mine - t * group)) * (D + 4);
#pragma unroll
        for (int i = 0; i < D / 32; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) *(f32x4*)(to + 32 * i + 8 * e + 4 * hi) = f32x4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
        if (hi == 0) {
            to[D] = m;
            to[D + 1] = den;
        }
        return;
    }
    const float by = den == 0.0f ? 0.0f : 1.0f / den;
    if (p.lse && hi == 0 && mine < nrows)
        p.lse[(int64_t)(sq.q0 + token(mine)) * p.Hq + head + (mine - token(mine) * group)] = (m + __builtin_log2f(den * (1 << kLag))) * 0.69314718055994530942f;
    // the rows leave through LDS, in whole lines
    lds_u8* const mo = lds + gw * OWN;
#pragma unroll
    for (int c = 0; c < D / 32; c++)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            *(__attribute__((address_space(3))) u32x2*)(mo + l32 * D * 2 + ((4 * c + (e >> 2)) ^ swizzle_k<D>(l32)) * 16 + 8 * hi) =
                u32x2{pack_bf16x2(o[c][e] * by, o[c][e + 1] * by), pack_bf16x2(o[c][e + 2] * by, o[c][e + 3] * by)};
#pragma unroll
    for (int i = 0; i < 32 * CH / 64; i++) {
        const int piece = i * 64 + lane;
        const int r = piece / CH, c = piece % CH;
        const u32x4 w = *(const __attribute__((address_space(3))) u32x4*)(mo + r * D * 2 + (c ^ swizzle_k<D>(r)) * 16);
        const int t = token(first + r);
        if (first + r < nrows && c * 8 < p.d)
            *(u32x4*)(p.out + (int64_t)(sq.q0 + t) * p.out_stride + (head + (first + r - t * group)) * p.d + c * 8) = w;
    }
#endif
}

// Joins the parts of the rows' keys: a wave for a head's row, its lanes side by side over the
// columns and then over the parts.
template <int D>
__global__ __launch_bounds__(256) void k_join_parts(PParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int row = (int)(at / p.Hq), head = (int)(at - (int64_t)row * p.Hq);
    if (row >= p.tq) return;
    bool live = false;  // rows outside the sequences stay as they are
    for (int base = 0; base < p.b && !live; base += 64) {
        const int i = base + lane;
        Seq s = {};
        if (i < p.b) s = seq_at(p, i);
        live = __any(row >= s.q0 && row < s.q0 + s.nq);
    }
    if (!live) return;
    constexpr int CT = D / 4, GROUPS = 64 / CT;
    const int c = (lane % CT) * 4, grp = lane / CT;
    const int64_t stride = (int64_t)p.tq * p.Hq * (D + 4);
    const float* const first = p.part + at * (D + 4);
    const float own = lane < p.parts ? first[lane * stride + D] : neg_inf();
    float den = lane < p.parts ? first[lane * stride + D + 1] : 0.0f;
    float top = own;
#pragma unroll
    for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
    const float weight = top == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(own - top);
    den *= weight;
#pragma unroll
    for (int o = 32; o; o >>= 1) den += __shfl_xor(den, o);
    f32x4 acc = {};
    for (int s0 = 0; s0 < p.parts; s0 += GROUPS) {  // (all lanes, since they hold the weights)
        const int s = s0 + grp < p.parts ? s0 + grp : p.parts - 1;
        const float a = __shfl(weight, s);
        const f32x4 x = *(const f32x4*)(first + s * stride + c);
        if (s0 + grp < p.parts) acc += a * x;
    }
#pragma unroll
    for (int o = 32; o >= CT; o >>= 1)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[j] += __shfl_xor(acc[j], o);
    const float by = den == 0.0f ? 0.0f : 1.0f / den;
    if (lane < CT && c < p.d)
        *(u32x2*)(p.out + row * p.out_stride + head * p.d + c) = u32x2{pack_bf16x2(acc[0] * by, acc[1] * by), pack_bf16x2(acc[2] * by, acc[3] * by)};
    if (p.lse && lane == 0) p.lse[at] = (top + __builtin_log2f(den * (1 << kLag))) * 0.69314718055994530942f;
}

template <int D, int KEYS, int NW, int SPLIT>
hipError_t launch(PParams& p, hipStream_t st) {
    const int64_t units = p.tq / (NW / SPLIT * 32) + p.b;  // tiles that no sequence has return at once
    k_attn_prefill<D, KEYS, NW, SPLIT, false, false><<<dim3((unsigned)(units * p.Hq)), 64 * NW, lds_bytes<D, KEYS, NW, SPLIT>(), st>>>(p);
    return hipGetLastError();
}

// The groups' rows in one tile (pack), p.parts workgroups to a tile.
template <int D>
hipError_t launch_few(PParams& p, bool pack, hipStream_t st) {
    const int64_t units = ((int64_t)p.tq * (pack ? p.G : 1) / 128 + p.b) * p.parts;
    const dim3 grid((unsigned)(units * (pack ? p.H : p.Hq)));
    constexpr int KEYS = D <= 128 ? 64 : 32, lds = lds_bytes<D, KEYS, 4, 1>();
    if (p.parts == 1) {
        k_attn_prefill<D, KEYS, 4, 1, false, true><<<grid, 256, lds, st>>>(p);
        return hipGetLastError();
    }
    if (pack) k_attn_prefill<D, KEYS, 4, 1, true, true><<<grid, 256, lds, st>>>(p);
    else k_attn_prefill<D, KEYS, 4, 1, true, false><<<grid, 256, lds, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_join_parts<D><<<dim3((unsigned)(((int64_t)p.tq * p.Hq + 3) / 4)), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_prefill(const AttnPrefillArgs& a, hipStream_t st) {
    PParams p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.out = a.out; p.lse = a.lse; p.cu_q = a.cu_q; p.cu_k = a.cu_k;
    p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride; p.out_stride = a.out_stride;
    p.c = a.scale * 1.44269504088896340736f;
    p.b = (int)a.b; p.tq = (int)a.tq; p.tk = (int)a.tk; p.Hq = (int)a.q_heads; p.H = (int)a.heads;
    p.G = p.Hq / p.H; p.d = (int)a.d; p.causal = a.causal;
    p.part = (float*)a.ws;
    const PrefillPlan plan = prefill_plan(a.tq, a.tk, a.q_heads, a.heads, a.d, a.b, a.causal != 0, a.ws != nullptr);
    p.parts = (int)plan.parts;
    if (plan.pack || plan.parts > 1) {
        if (plan.width == 64) return launch_few<64>(p, plan.pack, st);
        return plan.width == 128 ? launch_few<128>(p, plan.pack, st) : launch_few<256>(p, plan.pack, st);
    }
    if (plan.width == 64) return plan.split == 2 ? launch<64, 64, 8, 2>(p, st) : launch<64, 64, 4, 1>(p, st);
    if (plan.width == 128) {
        if (plan.split == 2) return launch<128, 64, 8, 2>(p, st);
        return plan.waves == 8 ? launch<128, 64, 8, 1>(p, st) : launch<128, 64, 4, 1>(p, st);
    }
    return plan.keys == 32 ? launch<256, 32, 4, 1>(p, st) : launch<256, 64, 4, 1>(p, st);
}

}  // namespace nvfp4
