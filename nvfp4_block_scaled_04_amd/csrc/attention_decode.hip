// attention_decode.hip -- attention of a few tokens a sequence over the paged
// NVFP4 cache.
//
// For a query row n of a KV head (new token, head of the group), over its tokens j:
//   x_j = q_n . K_j * scale, p_j = exp(x_j - m), out_n = sum p_j V_j / sum p_j,
// one pass with the running maximum m (in base 2) and sum.  It is bound by the bytes
// of the cache (d * 9/8 a token, head and both tensors), so a workgroup serves up to
// 16 rows of a KV head with one read, and the tokens of a sequence are split over
// workgroups where there are few sequences; a second launch joins the parts.
//
// A wave takes 64 tokens at a time, staged in its own LDS ring (16 bytes a lane, straight
// from memory, no barriers).  Both products run on 16x16x32 fp16 MFMAs:
//   X^T[token, n] = K Q^T: a lane's A operand is 8 codes of a token (8 columns);
//   O^T[column, n] = V^T P^T: a transposing LDS read of 4-bit values hands a lane 16
//   tokens of one column, in the order in which its rows of X^T hold them, so P goes
//   from one product into the other without crossing lanes.
// e2m1 * ue4m3 is exact in fp16.  q enters as fp16 scaled by a power of two per row (exact
// down to 2^-28 of the row's largest, off by up to 2^-39 of it below); P is rounded to fp16, off
// by 2^-11 of itself at most.  Maximum, sum and both products' sums are fp32.
#include "gemm_common.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kBlock = 64;        // tokens a wave takes at a time
constexpr int kRows = 16;         // query rows of a workgroup
constexpr int kStages = 2;

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

struct DParams {
    const uint16_t* q;        // [b, T, Hq, d]
    const uint8_t *kv, *sf;
    const float* gs;
    const int32_t* table;     // [b, table_pages]
    const int32_t* lengths;   // [b]
    uint16_t* out;
    float* lse;               // [b, T, Hq] or null
    int2* plan;               // [b] parts and first slot of a sequence
    float* part;              // slots of kRows * (D + 2) floats
    int64_t page_codes, page_sf;  // bytes of a page
    float scale2;             // scale * log2(e)
    int b, T, Hq, H, G, d, pages, table_pages, page_log2, row_tiles, cap;
};

template <int D>
struct Stage {
    static constexpr int CODES = kBlock * D / 2;                // bytes of K (of V)
    static constexpr int SF = D / 16 * kBlock;                  // bytes of K's scales (of V's)
    static constexpr int OFF_V = CODES, OFF_SF = 2 * CODES;
    static constexpr int LOADS = 2 * CODES / 1024, SF_LOADS = (2 * SF + 1023) / 1024;
    static constexpr int BYTES = 2 * CODES + SF_LOADS * 1024;
    static constexpr int WAVE = kStages * BYTES + 4 * SF;       // the ring, then the scales as fp16
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Which sequence, part and (head, row tile) a workgroup has, and how long the parts
// are: the tokens of all sequences are shared out evenly over about kAttnParts
// workgroups, so that the time does not hang on the longest sequence.  Every wave works it
// out from the lengths (on the device, so that a captured graph follows them).
struct Work {
    int seq, len, parts, part, slot, hr;  // slot: the sequence's first unit of the workspace
};

__device__ __forceinline__ int seq_len(const DParams& p, int i) {
    const int v = p.lengths[i];
    return v < 0 ? 0 : v > p.cap ? p.cap : v;
}

__device__ __forceinline__ int parts_of(int len, int64_t chunk) {
    const int n = (int)((len + chunk - 1) / chunk);
    return n < 1 ? 1 : n;
}

__device__ __forceinline__ bool find_work(const DParams& p, Work& w) {
    const int lane = threadIdx.x & 63;
    const int hrs = p.H * p.row_tiles;
    const int unit = blockIdx.x / hrs;
    w.hr = blockIdx.x - unit * hrs;
    int64_t total = 0;
    int first = 0;
    for (int i = lane; i < p.b; i += 64) {
        const int v = seq_len(p, i);
        if (i == lane) first = v;
        total += v;
    }
    total = wave_sum64(total);
    int64_t chunk = (total * hrs + kAttnParts - 1) / kAttnParts;
    chunk = chunk < kAttnMinPart ? kAttnMinPart : chunk;
    chunk = (chunk + kBlock - 1) / kBlock * kBlock;
    int before = 0, slots = 0;
    for (int base = 0; base < p.b; base += 64) {
        const int i = base + lane;
        const int len = i < p.b ? (base ? seq_len(p, i) : first) : 0;
        const int n = i < p.b ? parts_of(len, chunk) : 0;
        const int m = n > 1 ? n : 0;
        int sn = n, sm = m;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const int a = __shfl_up(sn, o), c = __shfl_up(sm, o);
            if (lane >= o) { sn += a; sm += c; }
        }
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

// Pages of a block's four groups of 16 tokens; bits of `bad`: a group behind the part's end
// or on no page (its loads go to page 0).
struct Pages {
    int id[4];
    uint32_t bad;
};

__device__ __forceinline__ Pages find_pages(const DParams& p, const int32_t* pages, int tok, int end) {
    // constant memory to the compiler, so that the uniform reads are scalar ones
    const auto* const row = (const __attribute__((address_space(4))) int32_t*)pages;
    Pages g;
    g.bad = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int t = tok + 16 * i;
        const int at = t < end ? t : end - 1;
        int id = row[at < 0 ? 0 : at >> p.page_log2];
        if (t >= end || (uint32_t)id >= (uint32_t)p.pages) {
            g.bad |= 1u << i;
            id = 0;
        }
        g.id[i] = id;
    }
    return g;
}

__device__ __forceinline__ int pick(const int (&id)[4], int i) {
    const int a = i & 1 ? id[1] : id[0], b = i & 1 ? id[3] : id[2];
    return i & 2 ? b : a;
}

template <int D>
__device__ __forceinline__ void stage_block(const DParams& p, const Pages& g, int tok, int head, lds_u8* st) {
    using S = Stage<D>;
    constexpr int CH = D / 32;  // 16-byte chunks of a row
    const int lane = threadIdx.x & 63;
    const int rb = p.d >> 1;
    const int mask = (1 << p.page_log2) - 1;
#pragma unroll
    for (int which = 0; which < 2; which++) {
        const uint8_t* const base = p.kv + (((int64_t)(which * p.H + head)) << p.page_log2) * rb;
#pragma unroll
        for (int j = 0; j < S::LOADS / 2; j++) {
            const int piece = j * 64 + lane;
            const int t = piece / CH, c = piece % CH;
            const int id = pick(g.id, t >> 4);
            const uint8_t* src = base + id * p.page_codes + (int64_t)(((tok + t) & mask) * rb + (c * 32 < p.d ? c * 16 : 0));
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(st + which * S::OFF_V + j * 1024), 16, 0, 0);
        }
    }
    const int blocks = p.d >> 4;
#pragma unroll
    for (int j = 0; j < S::SF_LOADS; j++) {
        const int piece = j * 64 + lane;
        if (piece * 16 < 2 * S::SF) {
            const int which = piece * 16 >= S::SF;
            const int rem = piece - which * (S::SF / 16);
            const int blk = (rem >> 2) < blocks ? rem >> 2 : 0, grp = rem & 3;
            const uint8_t* src = p.sf + pick(g.id, grp) * p.page_sf +
                                 ((((int64_t)(which * p.H + head)) * blocks + blk) << p.page_log2) + ((tok + 16 * grp) & mask);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(st + S::OFF_SF + j * 1024), 16, 0, 0);
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

template <int D>
__global__ __launch_bounds__(kThreads, 2) void k_attn_decode(DParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    using S = Stage<D>;
    extern __shared__ __align__(16) uint8_t smem[];
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

    // the row's queries, scaled to fp16
    const int r = rt * kRows + n;
    const bool live = r < p.T * p.G;
    const int qt = live ? r / p.G : 0;
    const int64_t qrow = ((int64_t)w.seq * p.T + qt) * p.Hq + head * p.G + (live ? r - qt * p.G : 0);
    constexpr int QW = D / 32;
    f16x8 q[QW];
    float inv;
    {
        u32x4 raw[QW];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < QW; s++) {
            const int col = g * (D / 4) + 8 * s;
            raw[s] = u32x4{};
            if (live && col < p.d) raw[s] = *(const u32x4*)(p.q + qrow * p.d + col);
            const uint32_t v[4] = {raw[s][0], raw[s][1], raw[s][2], raw[s][3]};
            const uint32_t a = absmax_bits_bf16x8(v);
            top = a > top ? a : top;
        }
        uint32_t o = __shfl_xor(top, 16);
        top = o > top ? o : top;
        o = __shfl_xor(top, 32);
        top = o > top ? o : top;
        int e = top >> 7;           // the largest one's exponent goes to 14
        e = e < 15 ? 15 : e > 254 ? 254 : e;
        const float up = bits_f((uint32_t)(268 - e > 254 ? 254 : 268 - e) << 23);
        inv = bits_f((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int s = 0; s < QW; s++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                q[s][2 * j] = (_Float16)(bf16_lo(raw[s][j]) * up);
                q[s][2 * j + 1] = (_Float16)(bf16_hi(raw[s][j]) * up);
            }
    }
    const float to_x = inv * (p.scale2 / p.gs[0]);
    const int limit = w.len - (p.T - 1 - qt);  // tokens this row sees

    uint8_t* const mine = smem + wave * S::WAVE;
    lds_u8* const ring = (lds_u8*)mine;
    uint8_t* const ks16 = mine + kStages * S::BYTES;
    uint8_t* const vs16 = ks16 + 2 * S::SF;

    float m = neg_inf(), l = 0.0f;
    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; i++) o[i] = f32x4{};

    const int step = kWaves * kBlock;
    int tok = t0 + wave * kBlock;
    Pages cur = find_pages(p, row, tok, t1), next = find_pages(p, row, tok + step, t1);
    if (tok < t1) stage_block<D>(p, cur, tok, head, ring);
    if (tok + step < t1) stage_block<D>(p, next, tok + step, head, ring + S::BYTES);
    int s = 0;
    for (; tok < t1; tok += step, s ^= 1) {
        const Pages after = find_pages(p, row, tok + 2 * step, t1);
        if (tok + step < t1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::LOADS + S::SF_LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint8_t* const st = mine + s * S::BYTES;
        const bool masked = tok + kBlock > w.len - p.T + 1 || tok + kBlock > t1 || cur.bad;

        // scales to fp16: K's as they lie, V's in the order of a lane's tokens
#pragma unroll
        for (int j = 0; j < (S::SF + 511) / 512; j++) {
            const int at = j * 512 + lane * 8;  // 8 tokens of a block
            if (at < S::SF) {
                const u32x2 kb = *(const u32x2*)(st + S::OFF_SF + at), vb = *(const u32x2*)(st + S::OFF_SF + S::SF + at);
                f16x4 k0 = scales4(kb[0]), k1 = scales4(kb[1]), v0 = scales4(vb[0]), v1 = scales4(vb[1]);
                const int t = at & 63, blk = at >> 6;
                if (masked) {
                    const bool none = (cur.bad >> (t >> 4)) & 1;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        if (none || tok + t + e >= t1) v0[e] = (_Float16)0.0f;
                        if (none || tok + t + 4 + e >= t1) v1[e] = (_Float16)0.0f;
                    }
                }
                if (blk * 16 >= p.d) k0 = k1 = v0 = v1 = f16x4{};
                *(f16x4*)(ks16 + 2 * at) = k0;
                *(f16x4*)(ks16 + 2 * at + 8) = k1;
                uint8_t* const vd = vs16 + 128 * blk + 8 * (t >> 4);
                *(f16x4*)(vd + 32 * ((t >> 2) & 3)) = v0;
                *(f16x4*)(vd + 32 * (((t >> 2) & 3) + 1)) = v1;
            }
        }

        // X^T = K Q^T
        float x[16];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f32x4 acc = {};
            const uint8_t* const kr = st + (16 * i + n) * (D / 2) + g * (D / 8);
            const uint8_t* const ksr = ks16 + (g * (D / 64) * kBlock + 16 * i + n) * 2;
            uint32_t kw[QW];
            if constexpr (D == 64) {
                const u32x2 v = *(const u32x2*)kr;
                kw[0] = v[0]; kw[1] = v[1];
            } else {
#pragma unroll
                for (int c = 0; c < QW / 4; c++) {
                    const u32x4 v = *(const u32x4*)(kr + 16 * c);
#pragma unroll
                    for (int j = 0; j < 4; j++) kw[4 * c + j] = v[j];
                }
            }
#pragma unroll
            for (int c = 0; c < QW; c++) {
                const _Float16 sc = *(const _Float16*)(ksr + (c >> 1) * kBlock * 2);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(dequant8(kw[c], sc), q[c], acc, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 4; e++) x[4 * i + e] = acc[e] * to_x;
        }
        if (masked) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int t = tok + 16 * i + 4 * g + e;
                    if (t >= limit || t >= t1 || ((cur.bad >> i) & 1)) x[4 * i + e] = neg_inf();
                }
        }
        // a row's maximum is moved only where a score exceeds it by more than 2^8 (by the row
        // alone, so that its bits do not depend on the rows beside it)
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; i++) top = __builtin_fmaxf(top, x[i]);
        if (__any(top > m + 8.0f)) {
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float to = top > m + 8.0f ? top : m;
            const float a = to == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= a;
#pragma unroll
            for (int i = 0; i < D / 16; i++) o[i] *= a;
        }
        const float base = m == neg_inf() ? 0.0f : m;
        f16x8 pf[2];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float e = __builtin_amdgcn_exp2f(x[i] - base);
            sum += e;
            pf[i >> 3][i & 7] = (_Float16)e;
        }
        l += sum;

        // O^T += V^T P^T
        const int vrow = 16 * (n >> 2) + 4 * g + (n & 3);
#pragma unroll
        for (int b = 0; b < D / 16; b++) {
            typedef int i32x2 __attribute__((ext_vector_type(2)));
            const i32x2 vw = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (__attribute__((address_space(3))) i32x2*)(ring + s * S::BYTES + S::OFF_V + vrow * (D / 2) + 8 * b));
            const f16x8 s0 = *(const f16x8*)(vs16 + 128 * b + 32 * g), s1 = *(const f16x8*)(vs16 + 128 * b + 32 * g + 16);
            o[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(dequant8_pairs((uint32_t)vw[0], s0), pf[0], o[b], 0, 0, 0);
            o[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(dequant8_pairs((uint32_t)vw[1], s1), pf[1], o[b], 0, 0, 0);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage has been read
        if (tok + 2 * step < t1) stage_block<D>(p, after, tok + 2 * step, head, ring + s * S::BYTES);
        cur = next;
        next = after;
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // the waves' parts, through LDS: [wave][n][D + 4], the last four: m, l
    constexpr int PITCH = D + 4;
    __syncthreads();
    float* const all = (float*)smem;
    float* const my = all + (wave * kRows + n) * PITCH;
#pragma unroll
    for (int b = 0; b < D / 16; b++) *(f32x4*)(my + 16 * b + 4 * g) = o[b];
    if (g == 0) { my[D] = m; my[D + 1] = l; }
    __syncthreads();
    const float out_scale = 1.0f / p.gs[1];
    float* const slot = p.part + ((int64_t)(w.slot + w.part) * p.H * p.row_tiles + w.hr) * (kRows * (D + 2));
    if (w.hr == 0 && w.part == 0 && threadIdx.x == 0) p.plan[w.seq] = make_int2(w.parts, w.slot);
    constexpr int CT = D / 4;  // threads of a row, four columns each
    for (int i = threadIdx.x; i < kRows * CT; i += kThreads) {
        const int nn = i / CT, c = (i - nn * CT) * 4;
        const int rr = rt * kRows + nn;
        if (rr >= p.T * p.G) continue;
        float mm[kWaves], top = neg_inf();
#pragma unroll
        for (int v = 0; v < kWaves; v++) {
            mm[v] = all[(v * kRows + nn) * PITCH + D];
            top = __builtin_fmaxf(top, mm[v]);
        }
        f32x4 sum = {};
        float den = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; v++) {
            const float* const src = all + (v * kRows + nn) * PITCH;
            const float a = top == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(mm[v] - top);
            den += a * src[D + 1];
            sum += a * *(const f32x4*)(src + c);
        }
        if (w.parts > 1) {
            *(f32x4*)(slot + nn * D + c) = sum;
            if (c == 0) {
                slot[kRows * D + nn] = top;
                slot[kRows * D + kRows + nn] = den;
            }
        } else {
            const int tt = rr / p.G;
            const int64_t orow = ((int64_t)w.seq * p.T + tt) * p.Hq + head * p.G + rr - tt * p.G;
            const float by = den == 0.0f ? 0.0f : out_scale / den;
            if (c < p.d) *(u32x2*)(p.out + orow * p.d + c) = u32x2{pack_bf16x2(sum[0] * by, sum[1] * by), pack_bf16x2(sum[2] * by, sum[3] * by)};
            if (p.lse && c == 0) p.lse[orow] = (top + __builtin_log2f(den)) * 0.69314718055994530942f;
        }
    }
#endif
}

// Joins the parts of the sequences that have several: a workgroup a (sequence, head,
// row tile), a wave every fourth row.
template <int D>
__global__ __launch_bounds__(kThreads) void k_attn_join(DParams p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int hrs = p.H * p.row_tiles;
    const int seq = blockIdx.x / hrs, hr = blockIdx.x - seq * hrs;
    const int2 plan = p.plan[seq];
    if (plan.x <= 1) return;
    const int rt = hr % p.row_tiles, head = hr / p.row_tiles;
    const int64_t stride = (int64_t)hrs * (kRows * (D + 2));
    const float* const first = p.part + (int64_t)plan.y * stride + (int64_t)hr * (kRows * (D + 2));
    const float out_scale = 1.0f / p.gs[1];
    constexpr int E = D / 64;
    for (int nn = wave; nn < kRows && rt * kRows + nn < p.T * p.G; nn += kWaves) {
        float top = neg_inf();
        for (int s = lane; s < plan.x; s += 64) top = __builtin_fmaxf(top, first[s * stride + kRows * D + nn]);
#pragma unroll
        for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
        float den = 0.0f, acc[E] = {};
        for (int s0 = 0; s0 < plan.x; s0 += 64) {
            float a = 0.0f;
            if (s0 + lane < plan.x) {
                const float* const ml = first + (s0 + lane) * stride + kRows * D + nn;
                a = top == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(ml[0] - top);
                den += a * ml[kRows];
            }
            const int k = plan.x - s0 < 64 ? plan.x - s0 : 64;
            for (int s = 0; s < k; s++) {
                const float as = __shfl(a, s);
                const float* const src = first + (s0 + s) * stride + nn * D + lane * E;
#pragma unroll
                for (int e = 0; e < E; e++) acc[e] += as * src[e];
            }
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) den += __shfl_xor(den, o);
        const int rr = rt * kRows + nn, tt = rr / p.G;
        const int64_t orow = ((int64_t)seq * p.T + tt) * p.Hq + head * p.G + rr - tt * p.G;
        const float by = den == 0.0f ? 0.0f : out_scale / den;
#pragma unroll
        for (int e = 0; e < E; e++)
            if (lane * E + e < p.d) p.out[orow * p.d + lane * E + e] = (uint16_t)f32_to_bf16_rne(acc[e] * by);
        if (p.lse && lane == 0) p.lse[orow] = (top + __builtin_log2f(den)) * 0.69314718055994530942f;
    }
}

template <int D>
hipError_t launch(const DParams& p, int64_t grid, bool join, hipStream_t st) {
    constexpr int lds = kWaves * Stage<D>::WAVE > kWaves * kRows * (D + 4) * 4 ? kWaves * Stage<D>::WAVE : kWaves * kRows * (D + 4) * 4;
    k_attn_decode<D><<<dim3((unsigned)grid), kThreads, lds, st>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !join) return e;
    k_attn_join<D><<<dim3((unsigned)(p.b * p.H * p.row_tiles)), kThreads, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_decode(const AttnDecodeArgs& a, hipStream_t st) {
    DParams p{};
    p.q = a.q; p.kv = a.kv; p.sf = a.kv_sf; p.gs = a.kv_gs; p.table = a.block_table; p.lengths = a.lengths;
    p.out = a.out; p.lse = a.lse;
    p.plan = (int2*)a.ws;
    p.part = (float*)((char*)a.ws + (a.b * 8 + 255) / 256 * 256);
    p.page_codes = a.page * a.heads * a.d;
    p.page_sf = 2 * a.page * a.heads * (a.d / 16);
    p.scale2 = a.scale * 1.44269504088896340736f;
    p.b = (int)a.b; p.T = (int)a.t; p.H = (int)a.heads; p.Hq = (int)a.q_heads; p.G = p.Hq / p.H; p.d = (int)a.d;
    p.pages = (int)a.pages; p.table_pages = (int)a.table_pages;
    p.page_log2 = __builtin_ctzll((unsigned long long)a.page);
    p.row_tiles = (p.T * p.G + kRows - 1) / kRows;
    p.cap = (int)(a.table_pages * a.page);
    // the most workgroups that lengths up to the table's can ask for
    const int64_t hrs = (int64_t)p.H * p.row_tiles;
    int64_t units = (kAttnParts + hrs - 1) / hrs + p.b;
    const int64_t each = (p.cap + kAttnMinPart - 1) / kAttnMinPart;
    if (each * p.b < units) units = each * p.b;
    const bool join = each > 1;
    if (a.d <= 64) return launch<64>(p, units * hrs, join, st);
    if (a.d <= 128) return launch<128>(p, units * hrs, join, st);
    return launch<256>(p, units * hrs, join, st);
}

}  // namespace nvfp4
