// attention_decode.hip -- attention of a few tokens a sequence over the paged
// NVFP4 cache.
//
// For a query row n of a KV head (new token, head of the group), over its tokens j:
//   x_j = q_n . K_j * scale, p_j = exp(x_j - m), out_n = sum p_j V_j / sum p_j,
// one pass with the running maximum m (in base 2) and sum.  It is bound by the bytes
// of the cache (d * 9/8 a token, head and both tensors), so a workgroup serves 16 or 32
// rows of a KV head with one read, and the tokens of a sequence are split over
// workgroups where there are few sequences; a second launch joins the parts.  64 sequences
// of up to 16384, 64 / 8 heads of 128 (631 MB): 119 us, 5.3 TB/s, of 16384 each (1.2 GB) 203, 6.0 TB/s,
// what reads alone reach; 32 heads over one of 32768 (38 MB): 13 us, of which 6 are the bytes', and 4
// of the join.
//
// A wave takes 64 tokens at a time, staged in LDS of its own (16 bytes a lane, straight from
// memory, no barriers): one block, whose next loads start when the last read of it has
// come, and the other waves of the SIMD hide that wait (two blocks a wave would halve
// the workgroups of a CU).  Both products run on 16x16x32 fp16 MFMAs:
//   X^T[token, n] = K Q^T: a lane's A operand is 8 codes of a token (8 columns);
//   O^T[column, n] = V^T P^T: a transposing LDS read of 4-bit values hands a lane 16
//   tokens of one column, in the order in which its rows of X^T hold them, so P goes
//   from one product into the other without crossing lanes.
// e2m1 * ue4m3 is exact in fp16.  q enters as fp16 scaled by a power of two per row (exact
// down to 2^-28 of the row's largest, off by up to 2^-39 of it below); P is rounded to fp16 (kLag).
// Maximum, sum and both products' sums are fp32.
#include "gemm_common.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kBlock = kAttnBlock;  // tokens a wave takes at a time
constexpr int kRows = kAttnRows;    // query rows of a matrix product
// A row's maximum m, in whole powers of two, is moved where a score exceeds it by more than kLag; a
// probability is 2^(score - m + kUp), 2^15 at most, which fp16 holds to 2^-11 of itself down to 2^-26
// of the largest and to 2^-37 of the largest below.  (At m itself with a lag of 8 fp16 ends at 2^-25,
// and a key 17 above many others, in natural units, took their share away.)  A smaller lag moves more
// often: 64 sequences of up to 16384 with 0 / 2 / 8: 123 / 121 / 119 us, 4 x 8 rows over 32 of 8192
// 79.3 / 78.3 / 76.6.
constexpr int kLag = 2, kUp = 15 - kLag;
constexpr float kDown = 1.0f / (1 << kUp);
constexpr int kAttnLdsLong = 54272;  // LDS of a workgroup, three of which fit a CU

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

struct DParams {
    const uint16_t* q;        // [b, T, Hq, d], q_stride from token to token
    const uint8_t *kv, *sf;
    const float* gs;
    const int32_t* table;     // [b, table_pages]
    const int32_t* lengths;   // [b]
    uint16_t* out;
    float* lse;               // [b, T, Hq] or null
    int2* plan;               // [b] parts and first slot of a sequence
    float* part;              // slots of kRows * (D + 2) floats
    int64_t page_codes, page_sf;  // bytes of a page
    int64_t q_stride;
    float scale2;             // scale * log2(e)
    int b, T, Hq, H, G, d, pages, table_pages, page_log2, row_tiles, cap;
    int split, least;  // parts of all sequences, about; fewest blocks of a part
};

template <int D>
struct Stage {
    static constexpr int CODES = kBlock * D / 2;                // bytes of K (of V)
    static constexpr int SF = D / 16 * kBlock;                  // bytes of K's scales (of V's)
    static constexpr int OFF_V = CODES, OFF_SF = 2 * CODES;
    static constexpr int SF_LOADS = (2 * SF + 1023) / 1024;
    static constexpr int BYTES = 2 * CODES + SF_LOADS * 1024;
    static constexpr int WAVE = BYTES + 2 * SF;                 // the block, then V's scales as fp16
};

// V's 16-byte chunk c of row r lies in chunk c ^ swizzle(r), so that the 16 rows of a
// transposing read lie in different banks.
template <int D>
__device__ __forceinline__ int swizzle(int r) { return (r / (512 / D)) & (D / 32 - 1); }

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Which sequence, part and (head, row tile) a workgroup has, and how long the parts
// are: the tokens of all sequences are shared out evenly over about p.split
// workgroups, so that the time does not hang on the longest sequence.  Every wave works it
// out from the lengths (on the device, so that a captured graph follows them).
struct Work {
    int seq, len, parts, part, slot, hr;  // slot: the sequence's first unit of the workspace
};

__device__ __forceinline__ int seq_len(const DParams& p, int i) {
    const int v = p.lengths[i];
    return v < 0 ? 0 : v > p.cap ? p.cap : v;
}

__device__ __forceinline__ bool find_work(const DParams& p, Work& w) {
    const int lane = threadIdx.x & 63;
    const int hrs = p.H * p.row_tiles;
    const int unit = blockIdx.x / hrs;
    w.hr = blockIdx.x - unit * hrs;
    int64_t total = 0;  // in blocks; 64 lengths add up to less than 2^31
    int first = 0;
    for (int base = 0; base < p.b; base += 64) {
        const int v = base + lane < p.b ? seq_len(p, base + lane) : 0;
        if (base == 0) first = v;
        total += __builtin_amdgcn_readlane(wave_scan((v + kBlock - 1) / kBlock), 63);
    }
    int64_t chunk64 = (int64_t)((uint64_t)(total * hrs + p.split - 1) / (uint32_t)p.split);
    chunk64 = chunk64 < p.least ? p.least : chunk64;
    const uint32_t chunk = chunk64 > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)chunk64;
    int before = 0, slots = 0;
    for (int base = 0; base < p.b; base += 64) {
        const int i = base + lane;
        const int len = base == 0 ? first : i < p.b ? seq_len(p, i) : 0;
        const uint32_t blocks = (uint32_t)(len + kBlock - 1) / kBlock;
        const int n = i < p.b ? (blocks <= chunk ? 1 : (int)((blocks + chunk - 1) / chunk)) : 0;
        const int m = n > 1 ? n : 0;
        const int sn = wave_scan(n), sm = wave_scan(m);
        const uint64_t hit = __ballot(before + sn > unit);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            w.seq = base + l;
            w.len = __builtin_amdgcn_readlane(len, l);
            w.parts = __builtin_amdgcn_readlane(n, l);
            w.part = unit - before - (__builtin_amdgcn_readlane(sn, l) - w.parts);
            w.slot = slots + __builtin_amdgcn_readlane(sm, l) - __builtin_amdgcn_readlane(m, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(sn, 63);
        slots += __builtin_amdgcn_readlane(sm, 63);
    }
    return false;
}

// The pages of a wave's next 16 blocks: lane 4 k + i has the one of group i (16 tokens) of
// block k, -1 for a group behind the part's end or on no page.
__device__ __forceinline__ int load_pages(const DParams& p, const int32_t* row, int tok, int end) {
    const int lane = threadIdx.x & 63;
    const int t = tok + (lane >> 2) * (kWaves * kBlock) + 16 * (lane & 3);
    if (t >= end) return -1;
    const int id = row[t >> p.page_log2];
    return (uint32_t)id < (uint32_t)p.pages ? id : -1;
}

// Starts a block's loads into LDS.  id: its groups' pages (page 0 in the place of none).
// ONCE: no other workgroup reads the block (one tile of rows), so it passes the caches by
// (streaming policy): 64 sequences of 16384, 1.2 GB: 203 us a call, 220 without; of up to 16384 119, 129.
// PACKED: rows lie in LDS as they do in memory, where the 16 rows of a group are 8 d bytes in one
// piece, for a d that is no multiple of 32 (a row alone does not begin on 16 bytes) or half of D
// (32 sequences of 8192, heads of 32: 33 us, 39 with rows of D; but of 96, 64 of up to 8192: 72, 67).
template <int D, bool ONCE, bool PACKED>
__device__ __forceinline__ void stage_block(const DParams& p, const int (&id)[4], int tok, int head, lds_u8* st) {
    using S = Stage<D>;
    constexpr int CH = D / 32;             // 16-byte chunks of a row
    constexpr int ROWS = 64 / CH;          // rows of a load
    const int lane = threadIdx.x & 63;
    const int d = p.d;
    const uint32_t rb = d >> 1;
    const int mask = (1 << p.page_log2) - 1;
    const uint32_t r = lane / CH, c = lane % CH;
    if constexpr (PACKED) {
        const int per = d >> 1;  // 16-byte pieces of a group
        const int64_t plane = ((int64_t)head << p.page_log2) * rb, to_v = ((int64_t)p.H << p.page_log2) * rb;
        uint64_t at[4];  // of a group's first piece, less the pieces before it
#pragma unroll
        for (int i = 0; i < 4; i++)
            at[i] = (uint64_t)(p.kv + id[i] * p.page_codes + plane + (uint32_t)((tok + 16 * i) & mask) * rb) - i * per * 16;
#pragma unroll
        for (int j = 0; j < S::CODES / 1024; j++) {
            if (j * 64 >= 4 * per) break;
            // (a lane past the last piece repeats it, behind the rows)
            const int piece = j * 64 + lane < 4 * per ? j * 64 + lane : 4 * per - 1;
            uint64_t from = at[0];
#pragma unroll
            for (int i = 1; i < 4; i++) from = piece >= i * per ? at[i] : from;
            const uint8_t* const src = (const uint8_t*)from + piece * 16;
#pragma unroll
            for (int which = 0; which < 2; which++)
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + (which ? to_v : 0)),
                                                 (__attribute__((address_space(3))) void*)(st + which * S::OFF_V + j * 1024), 16, 0, ONCE ? 2 : 0);
        }
    }
#pragma unroll
    for (int which = 0; which < (PACKED ? 0 : 2); which++) {
        const int64_t plane = ((int64_t)(which * p.H + head) << p.page_log2) * rb;
#pragma unroll
        for (int j = 0; j < S::CODES / 1024; j++) {
            // rows j * ROWS .. of the block: within a group, or two groups
            auto at = [&](int group) { return p.kv + id[group] * p.page_codes + plane + (uint32_t)((tok + 16 * group) & mask) * rb; };
            uint32_t cc = which ? c ^ swizzle<D>(j * ROWS + r) : c;
            cc = cc * 32 < (uint32_t)d ? cc : 0;
            const uint8_t* src;
            if constexpr (D == 64) src = (r < 16 ? at(2 * j) : at(2 * j + 1)) + ((r & 15) * rb + cc * 16);
            else src = at(j * ROWS / 16) + ((j * ROWS % 16 + r) * rb + cc * 16);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(st + which * S::OFF_V + j * 1024), 16, 0, ONCE ? 2 : 0);
        }
    }
    const int blocks = d >> 4;
    auto at = [&](int group) { return p.sf + id[group] * p.page_sf + ((tok + 16 * group) & mask); };
    const uint8_t* const a = lane & 1 ? at(1) : at(0);
    const uint8_t* const b = lane & 1 ? at(3) : at(2);
    const uint8_t* const base = lane & 2 ? b : a;
#pragma unroll
    for (int j = 0; j < S::SF_LOADS; j++) {
        const int piece = j * 64 + lane;
        if (S::SF_LOADS > 1 || D == 128 || lane < 2 * S::SF / 16) {
            const int which = piece * 16 >= S::SF;
            const int blk = (piece - which * (S::SF / 16)) >> 2;
            const uint8_t* src = base + ((int64_t)((which * p.H + head) * blocks + (blk < blocks ? blk : 0)) << p.page_log2);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(st + S::OFF_SF + j * 1024), 16, 0, ONCE ? 2 : 0);
        }
    }
}

// Four ue4m3 scales of a dword as fp16.
__device__ __forceinline__ f16x4 scales4(uint32_t w) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
    return f16x4{a[0], a[1], b[0], b[1]};
}

// 8 codes of a dword times four pairs of scales.
__device__ __forceinline__ f16x8 dequant8_pairs(uint32_t w, f16x8 s) {
    const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * f16x2{s[0], s[1]};
    const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * f16x2{s[2], s[3]};
    const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * f16x2{s[4], s[5]};
    const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * f16x2{s[6], s[7]};
    return f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Transposing reads of N blocks of 16 columns of a lane's row, two to a 16-byte chunk, and
// the wait for them (the compiler puts a wait for every load under way before its own
// intrinsic).  sw: the row's swizzle, in bytes.
template <int D, int OFF, int N>
__device__ __forceinline__ void read_columns(uint32_t at, uint32_t sw, u32x2 (&v)[N]) {
    static_assert(N == 4 || N == 8, "");
    constexpr int BASE = D == 256 && OFF % 128 ? 64 : 0, CONST = OFF - BASE;
    const uint32_t a0 = at + (BASE ^ sw), a1 = at + ((BASE + 16) ^ sw);
    if constexpr (N == 4) {
        asm volatile("ds_read_b64_tr_b4 %0, %4 offset:%6\n\tds_read_b64_tr_b4 %1, %4 offset:%7\n\t"
                     "ds_read_b64_tr_b4 %2, %5 offset:%6\n\tds_read_b64_tr_b4 %3, %5 offset:%7\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]) : "v"(a0), "v"(a1), "n"(CONST), "n"(CONST + 8) : "memory");
    } else {
        const uint32_t a2 = at + ((BASE + 32) ^ sw), a3 = at + ((BASE + 48) ^ sw);
        asm volatile("ds_read_b64_tr_b4 %0, %8 offset:%12\n\tds_read_b64_tr_b4 %1, %8 offset:%13\n\t"
                     "ds_read_b64_tr_b4 %2, %9 offset:%12\n\tds_read_b64_tr_b4 %3, %9 offset:%13\n\t"
                     "ds_read_b64_tr_b4 %4, %10 offset:%12\n\tds_read_b64_tr_b4 %5, %10 offset:%13\n\t"
                     "ds_read_b64_tr_b4 %6, %11 offset:%12\n\tds_read_b64_tr_b4 %7, %11 offset:%13\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
                     : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(CONST), "n"(CONST + 8) : "memory");
    }
}

// NT: products' worths of query rows of a workgroup, which share the dequantized keys and values.
// (PACKED: a workgroup of a CU fewer, for the registers of its addresses: spilled, whose reloads
// wait for the loads in flight, 64 sequences of up to 8192 with heads of 96 took 113 us, 72 so.)
template <int D, int NT, bool ONCE, bool PACKED>
__global__ __launch_bounds__(kThreads, NT == 2 ? (D <= 64 ? 3 : 2) : D <= 64 ? (PACKED ? 4 : 5) : D <= 128 ? (PACKED ? 3 : 4) : 2) void k_attn_decode(DParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    using S = Stage<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int d = p.d;
    const int pitch = PACKED ? d >> 1 : D / 2;  // bytes of a row in LDS
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    Work w;
    if (!find_work(p, w)) return;
    w.seq = __builtin_amdgcn_readfirstlane(w.seq);
    const int rt = w.hr % p.row_tiles, head = w.hr / p.row_tiles;
    int chunk = (w.len + w.parts - 1) / w.parts;
    chunk = (chunk + kBlock - 1) / kBlock * kBlock;
    const int t0 = w.part * chunk;
    const int t1 = w.len - t0 < chunk ? w.len : t0 + chunk;  // may lie before t0
    const int32_t* const row = p.table + (int64_t)w.seq * p.table_pages;

    // the row's queries, under way while the first block's pages and loads are worked out
    constexpr int ROWS = NT * kRows;
    constexpr int QW = D / 32;
    int limit[NT];  // tokens a row sees
    const int step = kWaves * kBlock;
    int tok = t0 + wave * kBlock;
    int ids = load_pages(p, row, tok, t1), ids_next = load_pages(p, row, tok + 16 * step, t1);
    u32x4 raw[NT][QW];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int r = rt * ROWS + t * kRows + n;
        const bool live = r < p.T * p.G;
        const int qt = live ? r / p.G : 0;
        const uint16_t* const src = p.q + ((int64_t)w.seq * p.T + qt) * p.q_stride + (head * p.G + (live ? r - qt * p.G : 0)) * d;
        limit[t] = w.len - (p.T - 1 - qt);
#pragma unroll
        for (int s = 0; s < QW; s++) {
            const int col = g * (D / 4) + 8 * s;
            raw[t][s] = u32x4{};
            if (live && col < d) raw[t][s] = *(const u32x4*)(src + col);
        }
    }
    const float gs_k = p.gs[0], gs_v = p.gs[1];

    uint8_t* const mine = smem + wave * S::WAVE;
    lds_u8* const st = (lds_u8*)mine;
    uint8_t* const vs16 = mine + S::BYTES;
    int k = 0;          // of the 16 blocks that `ids` knows
    uint32_t bad = 0;   // groups of the block behind the end or on no page
    auto start = [&](int at) {  // the loads of the wave's block at `at`, whose pages are those of block k
        int id[4];
        bad = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int v = __builtin_amdgcn_readlane(ids, 4 * k + i);
            bad |= v < 0 ? 1u << i : 0u;
            id[i] = v < 0 ? 0 : v;
        }
        stage_block<D, ONCE, PACKED>(p, id, at, head, st);
    };
    if (tok < t1) start(tok);

    // scaled to fp16
    f16x8 q[NT][QW];
    float to_x[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < QW; s++) {
            const uint32_t v[4] = {raw[t][s][0], raw[t][s][1], raw[t][s][2], raw[t][s][3]};
            const uint32_t a = absmax_bits_bf16x8(v);
            top = a > top ? a : top;
        }
        uint32_t o = __shfl_xor(top, 16);
        top = o > top ? o : top;
        o = __shfl_xor(top, 32);
        top = o > top ? o : top;
        int e = top ? top >> 7 : 127;  // the largest one's exponent goes to 14
        e = e < 15 ? 15 : e > 254 ? 254 : e;
        const float up = bits_f((uint32_t)(268 - e > 254 ? 254 : 268 - e) << 23);
        const float inv = bits_f((uint32_t)(e - 14) << 23);
        to_x[t] = __builtin_fmaxf(inv * (p.scale2 / gs_k), 0x1p-126f);  // not 0: -inf times it is -inf
#pragma unroll
        for (int s = 0; s < QW; s++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                q[t][s][2 * j] = (_Float16)(bf16_lo(raw[t][s][j]) * up);
                q[t][s][2 * j + 1] = (_Float16)(bf16_hi(raw[t][s][j]) * up);
            }
    }

    // a lane's row of 16 values for the transposing reads
    constexpr int VN = D == 64 ? 4 : 8;
    const int vrow = 16 * g + n;
    const uint32_t vat = (uint32_t)(uintptr_t)st + vrow * pitch;
    const uint32_t vsw = PACKED ? 0 : swizzle<D>(vrow) * 16;

    float m[NT], l[NT];
    f32x4 o[NT][D / 16];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        m[t] = neg_inf();
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; i++) o[t][i] = f32x4{};
    }

    for (; tok < t1; tok += step) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint32_t none = bad;
        const bool masked = tok + kBlock > w.len - p.T + 1 || tok + kBlock > t1 || none;

        // V's scales to fp16
#pragma unroll
        for (int j = 0; j < (S::SF + 511) / 512; j++) {
            const int at = j * 512 + lane * 8;  // 8 tokens of a block of columns
            if (at < S::SF) {
                const u32x2 vb = *(const u32x2*)(mine + S::OFF_SF + S::SF + at);
                f16x4 v0 = scales4(vb[0]), v1 = scales4(vb[1]);
                const int t = at & 63;
                if (masked) {
                    const bool gone = (none >> (t >> 4)) & 1;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        if (gone || tok + t + e >= t1) v0[e] = (_Float16)0.0f;
                        if (gone || tok + t + 4 + e >= t1) v1[e] = (_Float16)0.0f;
                    }
                }
                if ((at >> 6) * 16 >= d) v0 = v1 = f16x4{};
                *(f16x8*)(vs16 + 2 * at) = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        }

        // X^T = K Q^T: row n of tile i is token 4 n + i, whose scales of a block of columns are
        // byte i of a dword
        f16x2 ksc[4][D / 128 ? D / 128 : 1];  // [i][pair of blocks]
        {
            uint32_t kb[D / 64];
#pragma unroll
            for (int c = 0; c < D / 64; c++) {
                kb[c] = *(const uint32_t*)(mine + S::OFF_SF + (g * (D / 64) + c) * kBlock + 4 * n);
                if ((g * (D / 64) + c) * 16 >= d) kb[c] = 0;
            }
            if constexpr (D == 64) {
                const f16x4 v = scales4(kb[0]);
#pragma unroll
                for (int i = 0; i < 4; i++) ksc[i][0] = f16x2{v[i], v[i]};
            } else {
#pragma unroll
                for (int c = 0; c < D / 128; c++) {
                    const f16x4 a = scales4(kb[2 * c]), b = scales4(kb[2 * c + 1]);
#pragma unroll
                    for (int i = 0; i < 4; i++) ksc[i][c] = f16x2{a[i], b[i]};
                }
            }
        }
        f32x4 x[NT][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
            for (int t = 0; t < NT; t++) x[t][i] = f32x4{};
            const uint8_t* const kr = mine + (4 * n + i) * pitch + g * (D / 8);
            uint32_t kw[QW];
            if constexpr (D == 64) {
                const u32x2 v = *(const u32x2*)kr;
                kw[0] = v[0]; kw[1] = v[1];
            } else {
#pragma unroll
                for (int c = 0; c < QW / 4; c++) {
                    u32x4 v;
                    if constexpr (PACKED) {
                        const u32x2 a = *(const u32x2*)(kr + 16 * c), b = *(const u32x2*)(kr + 16 * c + 8);
                        v = u32x4{a[0], a[1], b[0], b[1]};
                    } else {
                        v = *(const u32x4*)(kr + 16 * c);
                    }
#pragma unroll
                    for (int j = 0; j < 4; j++) kw[4 * c + j] = v[j];
                }
            }
#pragma unroll
            for (int c = 0; c < QW; c++) {
                const f16x8 kf = dequant8(kw[c], ksc[i][c >> 2][(c >> 1) & 1]);
#pragma unroll
                for (int t = 0; t < NT; t++) x[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[t][c], x[t][i], 0, 0, 0);
            }
        }
        u32x2 vw[D / 16 / VN][VN];
        read_columns<D, S::OFF_V>(vat, vsw, vw[0]);
        if constexpr (D == 256) read_columns<D, S::OFF_V + 64>(vat, vsw, vw[1]);
        // (that waited for every read of the block, so the next one's loads may come)
        if (tok + step < t1) {
            if (++k == 16) {
                k = 0;
                ids = ids_next;
                ids_next = load_pages(p, row, tok + 17 * step, t1);
            }
            start(tok + step);
        }
        f16x8 pf[NT][2];  // token 16 g + j in place j
#pragma unroll
        for (int t = 0; t < NT; t++) {
            if (masked) {
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int at = tok + 16 * g + 4 * e + i;
                        if (at >= limit[t] || at >= t1 || ((none >> g) & 1)) x[t][i][e] = neg_inf();
                    }
            }
            // (moved by the row alone, so that its bits do not depend on the rows beside it)
            float top = x[t][0][0];
#pragma unroll
            for (int i = 1; i < 16; i++) top = __builtin_fmaxf(top, x[t][i >> 2][i & 3]);
            top *= to_x[t];
            if (__any(top > m[t] + kLag)) {
                top = __builtin_fmaxf(top, __shfl_xor(top, 16));
                top = __builtin_fmaxf(top, __shfl_xor(top, 32));
                const float to = top > m[t] + kLag ? __builtin_rintf(top) : m[t];
                const float a = to == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m[t] - to);
                m[t] = to;
                l[t] *= a;
#pragma unroll
                for (int i = 0; i < D / 16; i++) o[t][i] *= a;
            }
            const float most = m[t] == neg_inf() ? 0.0f : m[t];
            float base = most - kUp, by = to_x[t];
            if (__any(__builtin_fabsf(most) >= kFarScore)) {  // (by the row alone too)
                const bool far = __builtin_fabsf(most) >= kFarScore;
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const float v = x[t][i >> 2][i & 3];
                    x[t][i >> 2][i & 3] = far ? far_score(v, by, most) : v;
                }
                base = far ? -kUp : base;
                by = far ? 1.0f : by;
            }
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][j & 3][j >> 2], by, -base));
                sum += e;
                pf[t][j >> 3][j & 7] = (_Float16)e;
            }
            l[t] += sum;
        }

        // O^T += V^T P^T
#pragma unroll
        for (int b = 0; b < D / 16; b++) {
            const u32x2 v = vw[b / VN][b % VN];
            const f16x8 s0 = *(const f16x8*)(vs16 + 128 * b + 32 * g), s1 = *(const f16x8*)(vs16 + 128 * b + 32 * g + 16);
            const f16x8 v0 = dequant8_pairs(v[0], s0), v1 = dequant8_pairs(v[1], s1);
#pragma unroll
            for (int t = 0; t < NT; t++) {
                o[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[t][0], o[t][b], 0, 0, 0);
                o[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[t][1], o[t][b], 0, 0, 0);
            }
        }
    }

    // the waves' parts, through LDS: [wave][n][D + 4], the last four: m, l
    constexpr int PITCH = D + 4;
    __syncthreads();
    float* const all = (float*)smem;
#pragma unroll
    for (int t = 0; t < NT; t++) {
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        float* const my = all + (wave * ROWS + t * kRows + n) * PITCH;
#pragma unroll
        for (int b = 0; b < D / 16; b++) *(f32x4*)(my + 16 * b + 4 * g) = o[t][b];
        if (g == 0) { my[D] = m[t]; my[D + 1] = l[t]; }
    }
    __syncthreads();
    const float out_scale = 1.0f / gs_v;
    float* const slot = p.part + ((int64_t)(w.slot + w.part) * p.H * p.row_tiles + w.hr) * (ROWS * (D + 2));
    if (w.hr == 0 && w.part == 0 && threadIdx.x == 0) p.plan[w.seq] = make_int2(w.parts, w.slot);
    constexpr int CT = D / 4;  // threads of a row, four columns each
    for (int i = threadIdx.x; i < ROWS * CT; i += kThreads) {
        const int nn = i / CT, c = (i - nn * CT) * 4;
        const int rr = rt * ROWS + nn;
        if (rr >= p.T * p.G) continue;
        float mm[kWaves], top = neg_inf();
#pragma unroll
        for (int v = 0; v < kWaves; v++) {
            mm[v] = all[(v * ROWS + nn) * PITCH + D];
            top = __builtin_fmaxf(top, mm[v]);
        }
        f32x4 sum = {};
        float den = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; v++) {
            const float* const src = all + (v * ROWS + nn) * PITCH;
            const float a = top == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(mm[v] - top);
            den += a * src[D + 1];
            sum += a * *(const f32x4*)(src + c);
        }
        if (w.parts > 1) {
            *(f32x4*)(slot + nn * D + c) = sum;
            if (c == 0) {
                slot[ROWS * D + nn] = top;
                slot[ROWS * D + ROWS + nn] = den;
            }
        } else {
            const int tt = rr / p.G;
            const int64_t orow = ((int64_t)w.seq * p.T + tt) * p.Hq + head * p.G + rr - tt * p.G;
            const float by = den == 0.0f ? 0.0f : 1.0f / den;  // (times out_scale it may be subnormal)
            if (c < d) *(u32x2*)(p.out + orow * d + c) = u32x2{pack_bf16x2(sum[0] * by * out_scale, sum[1] * by * out_scale), pack_bf16x2(sum[2] * by * out_scale, sum[3] * by * out_scale)};
            if (p.lse && c == 0) p.lse[orow] = (top + __builtin_log2f(den * kDown)) * 0.69314718055994530942f;
        }
    }
#endif
}

// Joins the parts of the sequences that have several.  WAVES: waves of a row of the output, whose
// threads lie side by side over the columns and then over the parts: four where the rows are few,
// one where they fill the card (most sequences have few parts then): the whole call for 256
// sequences of up to 2048, 64 heads, 80.2 us with four, 77.4 with one; for one of 32768, 32 heads,
// 16.6 and 18.5.
template <int D, int NT, int WAVES>
__global__ __launch_bounds__(kThreads) void k_attn_join(DParams p) {
    constexpr int ROWS = NT * kRows;
    constexpr int THREADS = 64 * WAVES, AT_ONCE = kWaves / WAVES;  // threads of a row, rows of a workgroup
    constexpr int CT = D / 4, GROUPS = THREADS / CT;  // threads of a part's row, parts at a time
    __shared__ float weights[AT_ONCE][kAttnPartsNarrow + 64];
    __shared__ float red[2 * kWaves];
    __shared__ __align__(16) float all_sums[AT_ONCE][GROUPS * D];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int own = wave / WAVES, t = threadIdx.x - own * THREADS;
    const int orow = blockIdx.x * AT_ONCE + own;
    if (orow >= p.b * p.T * p.Hq) return;
    float* const weight = weights[own];
    float* const sums = all_sums[own];
    auto sync = [] {
        if constexpr (WAVES > 1) __syncthreads();
        else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (a wave's own LDS accesses stay in order)
    };
    const int seq = orow / (p.T * p.Hq), rem = orow - seq * (p.T * p.Hq);
    const int2 plan = p.plan[seq];
    const int n = plan.x;
    if (n <= 1) return;
    const int tt = rem / p.Hq, qh = rem - tt * p.Hq;
    const int head = qh / p.G, r = tt * p.G + qh - head * p.G;
    const int hrs = p.H * p.row_tiles, rt = r / ROWS, nn = r - rt * ROWS;
    const int64_t stride = (int64_t)hrs * (ROWS * (D + 2));
    const float* const first = p.part + (int64_t)plan.y * stride + (int64_t)(head * p.row_tiles + rt) * (ROWS * (D + 2));
    // the first parts' rows, under way while the weights are worked out
    constexpr int AHEAD = 8;
    const int c = (t % CT) * 4, grp = t / CT;
    const float* src = first + (int64_t)(grp < n ? grp : 0) * stride + nn * D + c;
    f32x4 x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; i++) x[i] = *(const f32x4*)(src + (grp + i * GROUPS < n ? i * GROUPS * stride : 0));
    float top = neg_inf();
    for (int s = t; s < n; s += THREADS) {
        const float m = first[s * stride + ROWS * D + nn];
        weight[s] = m;
        top = __builtin_fmaxf(top, m);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
    if constexpr (WAVES > 1) {
        if (lane == 0) red[wave] = top;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kWaves; v++) top = __builtin_fmaxf(top, red[v]);
    }
    float den = 0.0f;
    for (int s = t; s < n; s += THREADS) {
        const float a = top == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(weight[s] - top);
        weight[s] = a;
        den += a * first[s * stride + ROWS * D + ROWS + nn];
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) den += __shfl_xor(den, o);
    if (WAVES > 1 && lane == 0) red[kWaves + wave] = den;
    sync();
    if constexpr (WAVES > 1) {
        den = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; v++) den += red[kWaves + v];
    }
    f32x4 acc = {};
#pragma unroll
    for (int i = 0; i < AHEAD; i++)
        if (grp + i * GROUPS < n) acc += weight[grp + i * GROUPS] * x[i];
    for (int s = grp + AHEAD * GROUPS; s < n; s += GROUPS) acc += weight[s] * *(const f32x4*)(src + (int64_t)(s - grp) * stride);
    *(f32x4*)(sums + grp * D + c) = acc;
    sync();
    if (t >= CT) return;
    acc = f32x4{};
#pragma unroll
    for (int i = 0; i < GROUPS; i++) acc += *(const f32x4*)(sums + i * D + c);
    const float by = den == 0.0f ? 0.0f : 1.0f / den, out_scale = 1.0f / p.gs[1];
    if (c < p.d) *(u32x2*)(p.out + (int64_t)orow * p.d + c) = u32x2{pack_bf16x2(acc[0] * by * out_scale, acc[1] * by * out_scale), pack_bf16x2(acc[2] * by * out_scale, acc[3] * by * out_scale)};
    if (p.lse && t == 0) p.lse[orow] = (top + __builtin_log2f(den * kDown)) * 0.69314718055994530942f;
}

template <int D, int NT>
hipError_t launch(const DParams& p, const DecodePlan& plan, hipStream_t st) {
    constexpr int merge = kWaves * NT * kRows * (D + 4) * 4;
    constexpr int need = kWaves * Stage<D>::WAVE > merge ? kWaves * Stage<D>::WAVE : merge;
    const int lds = D > 64 && plan.large && need < kAttnLdsLong ? kAttnLdsLong : need;
    const dim3 grid((unsigned)(plan.units * p.H * p.row_tiles));
    if (plan.once && !plan.packed) k_attn_decode<D, NT, true, false><<<grid, kThreads, lds, st>>>(p);
    else if (plan.once) k_attn_decode<D, NT, true, true><<<grid, kThreads, lds, st>>>(p);
    else if (!plan.packed) k_attn_decode<D, NT, false, false><<<grid, kThreads, lds, st>>>(p);
    else k_attn_decode<D, NT, false, true><<<grid, kThreads, lds, st>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !plan.join) return e;
    const int rows_out = p.b * p.T * p.Hq;
    if (plan.join_waves == kWaves) k_attn_join<D, NT, kWaves><<<dim3((unsigned)rows_out), kThreads, 0, st>>>(p);
    else k_attn_join<D, NT, 1><<<dim3((unsigned)((rows_out + kWaves - 1) / kWaves)), kThreads, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_decode(const AttnDecodeArgs& a, hipStream_t st) {
    DParams p{};
    p.q = a.q; p.kv = a.kv; p.sf = a.kv_sf; p.gs = a.kv_gs; p.table = a.block_table; p.lengths = a.lengths;
    p.out = a.out; p.lse = a.lse; p.q_stride = a.q_stride;
    p.plan = (int2*)a.ws;
    p.part = (float*)((char*)a.ws + (a.b * 8 + 255) / 256 * 256);
    p.page_codes = a.page * a.heads * a.d;
    p.page_sf = 2 * a.page * a.heads * (a.d / 16);
    p.scale2 = a.scale * 1.44269504088896340736f;
    p.b = (int)a.b; p.T = (int)a.t; p.H = (int)a.heads; p.Hq = (int)a.q_heads; p.G = p.Hq / p.H; p.d = (int)a.d;
    p.pages = (int)a.pages; p.table_pages = (int)a.table_pages;
    p.page_log2 = __builtin_ctzll((unsigned long long)a.page);
    p.cap = (int)(a.table_pages * a.page);
    const DecodePlan plan = decode_plan(a.b, a.t, a.q_heads, a.heads, a.d, p.cap);
    p.row_tiles = (int)plan.row_tiles;
    p.split = (int)plan.split;
    p.least = (int)plan.least;
    if (plan.width == 64) return plan.two ? launch<64, 2>(p, plan, st) : launch<64, 1>(p, plan, st);
    if (plan.width == 128) return plan.two ? launch<128, 2>(p, plan, st) : launch<128, 1>(p, plan, st);
    return launch<256, 1>(p, plan, st);
}

}  // namespace nvfp4
