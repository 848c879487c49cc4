// moe_small.hip -- a whole mixture-of-experts layer for a few tokens in two
// launches, on NVFP4 expert weights and bf16 tokens.
//
// What is computed (n tokens x, router logits, E experts of H -> I -> H):
//   chosen(i) = the top_k experts by (logit descending, index ascending) among
//               logits that are neither NaN nor -inf
//   w(i, e)   = softmax or sigmoid of the logit (/ the chosen ones' sum)
//   [g, u]    = alpha13[e] * x[i] @ W13[e]^T,   a = g / (1 + e^-g) * u
//   out[i]    = sum_e w(i, e) * alpha2[e] * a @ W2[e]^T
//
// First launch (k_moe_up): one workgroup per 16 gate and 16 up rows of an
// expert.  It routes for itself (a token's logits are one load per lane), finds
// the tokens that chose its expert, and streams the 32 weight rows once against
// up to 16 of them.  The activation leaves multiplied by the unnormalised
// routing weight and alpha2, so the second launch is one long product.
// Second launch (k_moe_down): one workgroup per 16 output columns; its K axis is
// the chosen experts' I axes laid end to end, dealt to the waves in contiguous
// ranges.  Each wave adds an expert's product into its own fp32 accumulators of
// all tokens in LDS, and the waves' accumulators are summed in wave order: no
// atomics, the same result on every call.
//
// Bound: the chosen experts' weights are read once (9/16 byte an element), the
// rest is small; the kernels are built to keep weight loads in flight.
#include "device_common.h"
#include "gemm_common.h"
#include "internal.h"
#include "skinny_w4.h"

namespace nvfp4 {
namespace {

constexpr int kNone = 255;       // rank of a token that did not choose the expert
constexpr int kUpWaves = 8;
constexpr int kDownWaves = 16;

struct EParams {
    const uint16_t* x;         // [T, H]
    const void* logits;        // [T, E]
    const uint8_t* w13;        // [E, 2I, H/2]
    const uint8_t* w13_sf;
    const float* alpha13;
    const uint8_t* w2;         // [E, H, I/2]
    const uint8_t* w2_sf;
    const float* alpha2;
    uint16_t* out;             // [T, H]
    int32_t* ids;              // [T, k]
    float* weights;            // [T, k]
    float* raw;                // [T, k] unnormalised weights
    uint16_t* act_hi;          // [T * k, I], row t * k + slot
    uint16_t* act_lo;
    int64_t w13_sfsz, w2_sfsz; // scale bytes of one expert
    int T, H, I, E, k;
    int lg_bf16, sigmoid, renorm;
    int by_slot;               // workgroup row y is the y-th chosen expert (else expert y)
    int tiles, xcd_chunk;
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Logit of expert j of token t; NaN and j >= E read as -inf (never chosen).
__device__ __forceinline__ float load_logit(const EParams& p, int t, int j) {
    if (j >= p.E) return neg_inf();
    const int64_t at = (int64_t)t * p.E + j;
    const float v = p.lg_bf16 ? bf16_lo((uint32_t)((const uint16_t*)p.logits)[at]) : ((const float*)p.logits)[at];
    return v == v ? v : neg_inf();
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Unnormalised weight of a chosen expert with logit l of a token whose largest
// logit is top; lg: the lane's logits of that token.  Softmax: exp(l - top),
// divided by the sum over all experts unless the chosen ones' sum divides it
// later.  Sigmoid, to be divided by the chosen ones' sum: every value scaled by
// exp(-min(top, 0)), so that very negative logits keep their ratios.
template <int NR>
__device__ __forceinline__ float route_weight(const EParams& p, float l, float top, const float lg[NR]) {
    if (!p.sigmoid) {
        const float u = expf(l - top);
        if (p.renorm) return u;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; i++) s += expf(lg[i] - top);
        return u / wave_sum(s);
    }
    if (l >= 0.0f) return 1.0f / (1.0f + expf(-l));
    const float base = p.renorm ? __builtin_fminf(top, 0.0f) : 0.0f;
    return expf(l - base) / (1.0f + expf(l));
}

// Tile index of blockIdx.x: XCD x (workgroups are dealt round-robin) takes the
// x-th contiguous eighth, so tiles that share scale lines share an L2.
__device__ __forceinline__ int tile_of(const EParams& p) {
    const int b = blockIdx.x;
    return p.xcd_chunk ? (b & 7) * p.xcd_chunk + (b >> 3) : b;
}

// NR: logits a lane holds of one token (ceil(E / 64)).
template <int NR, bool WHOLE>
__global__ __launch_bounds__(64 * kUpWaves) void k_moe_up(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass only needs the launch stub
    __shared__ uint8_t rank_of[64];          // slot in which a token chose this expert, or kNone
    __shared__ float weight_of[64];          // its unnormalised weight
    __shared__ uint64_t active[NR];          // experts that any token chose (by_slot)
    __shared__ int members[64];
    __shared__ f32x4 part[kUpWaves][2][64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int tile = tile_of(p);
    const bool teller = blockIdx.x == 0;     // writes its expert's routing results

    // 1. the expert of this workgroup
    int e = blockIdx.y;
    if (p.by_slot) {
        if (t < NR) active[t] = 0;
        __syncthreads();
        for (int tok = wave; tok < p.T; tok += kUpWaves) {
            float lg[NR];
#pragma unroll
            for (int i = 0; i < NR; i++) lg[i] = load_logit(p, tok, lane + 64 * i);
            uint64_t got[NR] = {};
            for (int j = 0; j < p.k; j++) {
                float m = lg[0];
#pragma unroll
                for (int i = 1; i < NR; i++) m = __builtin_fmaxf(m, lg[i]);
                m = wave_max(m);
                if (m == neg_inf()) break;
                bool done = false;
#pragma unroll
                for (int i = 0; i < NR; i++) {  // the lowest index that holds the maximum
                    const uint64_t at = __ballot(lg[i] == m);
                    if (!done && at) {
                        done = true;
                        const int l = __builtin_ctzll(at);
                        got[i] |= (uint64_t)1 << l;
                        if (lane == l) lg[i] = neg_inf();
                    }
                }
            }
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < NR; i++)
                    if (got[i]) atomicOr((unsigned long long*)&active[i], (unsigned long long)got[i]);
            }
        }
        __syncthreads();
        int left = blockIdx.y;  // the e-th set bit
        e = -1;
#pragma unroll
        for (int i = 0; i < NR; i++) {
            uint64_t bits = active[i];
            const int n = __builtin_popcountll(bits);
            if (e < 0 && left < n) {
                for (int q = 0; q < left; q++) bits &= bits - 1;
                e = 64 * i + __builtin_ctzll(bits);
            }
            left -= n;
        }
        e = __builtin_amdgcn_readfirstlane(e);
    }

    // 2. the tokens that chose it: e is in slot `better` of a token if `better`
    //    of its logits come before e's
    for (int tok = wave; tok < p.T; tok += kUpWaves) {
        float lg[NR];
        float mx = neg_inf();
        int able = 0;
#pragma unroll
        for (int i = 0; i < NR; i++) {
            lg[i] = load_logit(p, tok, lane + 64 * i);
            mx = __builtin_fmaxf(mx, lg[i]);
            able += __builtin_popcountll(__ballot(lg[i] > neg_inf()));
        }
        if (teller && blockIdx.y == 0 && lane < p.k && lane >= able) {  // slots left over
            p.ids[tok * p.k + lane] = -1;
            p.raw[tok * p.k + lane] = 0.0f;
        }
        if (e < 0) continue;
        float le = neg_inf();
        int better = 0;
#pragma unroll
        for (int i = 0; i < NR; i++)
            if (e >> 6 == i) le = __shfl(lg[i], e & 63);
#pragma unroll
        for (int i = 0; i < NR; i++)
            better += __builtin_popcountll(__ballot(lg[i] > le || (lg[i] == le && lane + 64 * i < e)));
        const bool in = le > neg_inf() && better < p.k;
        float u = 0.0f;
        if (in) {
            u = route_weight<NR>(p, le, wave_max(mx), lg);
            if (teller && lane == 0) {
                p.ids[tok * p.k + better] = e;
                p.raw[tok * p.k + better] = u;
            }
        }
        if (lane == 0) {
            rank_of[tok] = (uint8_t)(in ? better : kNone);
            weight_of[tok] = u;
        }
    }
    if (e < 0) return;
    __syncthreads();
    const bool mem = lane < p.T && rank_of[lane < p.T ? lane : 0] != kNone;
    const uint64_t mask = __ballot(mem);
    const int n = __builtin_popcountll(mask);
    if (n == 0) return;
    if (wave == 0 && mem) members[__builtin_popcountll(mask & (((uint64_t)1 << lane) - 1))] = lane;
    __syncthreads();

    // 3. 16 gate and 16 up rows against the members, 16 at a time
    const int r = lane & 15, g = lane >> 4;
    const int rowb = p.H / 2, nblk = p.H / 16, cpa4 = (nblk + 3) / 4;
    const int nch = (p.H + kChunk - 1) / kChunk;
    const int per = (nch + kUpWaves - 1) / kUpWaves;
    const int c0 = wave * per, c1 = c0 + per < nch ? c0 + per : nch;
    const int row = tile * 16 + r;  // I is a multiple of 16: always a row
    const uint8_t* const W = p.w13 + (int64_t)e * 2 * p.I * rowb;
    const uint8_t* const S = p.w13_sf + (int64_t)e * p.w13_sfsz;
    const uint8_t* const B[2] = {W + (int64_t)row * rowb, W + (int64_t)(p.I + row) * rowb};
    const uint8_t* const F[2] = {S + scale_row_off(row, cpa4), S + scale_row_off(p.I + row, cpa4)};
    const float a13 = p.alpha13[e], a2 = p.alpha2[e];
    for (int m0 = 0; m0 < n; m0 += 16) {
        const uint16_t* const X = m0 + r < n ? p.x + (int64_t)members[m0 + r] * p.H : nullptr;
        f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
        constexpr int U = 4;  // chunks whose loads are in flight together
        for (int cb = c0; cb < c1; cb += U) {
            u32x4 w[U][2], xv[U][4];
            uint32_t s[U][2];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int c = cb + u < c1 ? cb + u : c1 - 1;  // past the range: reload, never used
#pragma unroll
                for (int f = 0; f < 2; f++) {
                    w[u][f] = load_w4<WHOLE>(B[f], c, g, rowb);
                    s[u][f] = load_s4<WHOLE>(F[f], c, g, nblk);
                }
                load_x16<WHOLE>(xv[u], X, c, g, p.H);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (cb + u >= c1) break;
#pragma unroll
                for (int f = 0; f < 2; f++) {
                    const float s0 = __builtin_amdgcn_cvt_f32_fp8(s[u][f], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(s[u][f], 1);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dequant8_bf16(word(w[u][f], j), j < 2 ? s0 : s1),
                                                                         __builtin_bit_cast(bf16x8, xv[u][j]), acc[f], 0, 0, 0);
                }
            }
        }
        part[wave][0][lane] = acc[0];
        part[wave][1][lane] = acc[1];
        __syncthreads();
        if (wave == 0 && m0 + r < n) {  // the waves' sums in wave order; lane: token r, columns 4 g ..
            f32x4 sg = part[0][0][lane], su = part[0][1][lane];
#pragma unroll
            for (int v = 1; v < kUpWaves; v++) {
                sg += part[v][0][lane];
                su += part[v][1][lane];
            }
            const int tok = members[m0 + r];
            const float wt = weight_of[tok] * a2;
            float a[4];
#pragma unroll
            for (int v = 0; v < 4; v++) {
                const float gt = a13 * sg[v];
                a[v] = gt / (1.0f + expf(-gt)) * (a13 * su[v]) * wt;
            }
            uint32_t h0, l0, h1, l1;
            split_bf16x2(a[0], a[1], h0, l0);
            split_bf16x2(a[2], a[3], h1, l1);
            const int64_t at = (int64_t)(tok * p.k + rank_of[tok]) * p.I + tile * 16 + 4 * g;
            *(u32x2*)(p.act_hi + at) = u32x2{h0, h1};
            *(u32x2*)(p.act_lo + at) = u32x2{l0, l1};
        }
        __syncthreads();
    }
#endif
}

template <bool WHOLE>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __align__(4) uint8_t rank_of[256 * 64];  // [E][T] slot, or kNone
    __shared__ int active[256];                    // the chosen experts, ascending
    __shared__ uint32_t chosen[8];                 // bit e % 32 of word e / 32
    __shared__ float sums[kDownWaves][64][17];     // each wave's [token][column] sums (padded rows)
    __shared__ float inv[64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int tile = tile_of(p);
    const int np = p.T * p.k;

    for (int i = t; i < (p.E * p.T + 3) / 4; i += 64 * kDownWaves) ((uint32_t*)rank_of)[i] = 0xFFFFFFFFu;
    for (int i = lane; i < 64 * 17; i += 64) (&sums[wave][0][0])[i] = 0.0f;
    if (t < 8) chosen[t] = 0;
    __syncthreads();
    for (int i = t; i < np; i += 64 * kDownWaves) {
        const int e = p.ids[i];
        if (e >= 0) {
            rank_of[e * p.T + i / p.k] = (uint8_t)(i % p.k);
            atomicOr(&chosen[e >> 5], 1u << (e & 31));
        }
    }
    if (t < p.T) {
        float s = 0.0f;
        for (int j = 0; j < p.k; j++) s += p.raw[t * p.k + j];
        const float v = p.renorm && p.ids[t * p.k] >= 0 ? 1.0f / s : 1.0f;
        inv[t] = v;
        if (blockIdx.x == 0)
            for (int j = 0; j < p.k; j++) p.weights[t * p.k + j] = p.raw[t * p.k + j] * v;
    }
    __syncthreads();
    int nact = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t w = chosen[i];
        if (t < 32 && (w >> t & 1)) active[nact + __builtin_popcount(w & ((1u << t) - 1))] = 32 * i + t;
        nact += __builtin_popcount(w);
    }
    __syncthreads();

    const int r = lane & 15, g = lane >> 4;
    const int rowb = p.I / 2, nblk = p.I / 16, cpa4 = (nblk + 3) / 4;
    const int nch = (p.I + kChunk - 1) / kChunk;
    const int row = tile * 16 + r;  // H is a multiple of 16
    const int total = nact * nch;
    const int q0 = (int)((int64_t)total * wave / kDownWaves), q1 = (int)((int64_t)total * (wave + 1) / kDownWaves);
    for (int q = q0; q < q1;) {
        const int at = q / nch, e = __builtin_amdgcn_readfirstlane(active[at]);
        const int c0 = q - at * nch, c1 = q1 - at * nch < nch ? q1 - at * nch : nch;  // this expert's chunks
        q += c1 - c0;
        const uint8_t* const B = p.w2 + ((int64_t)e * p.H + row) * rowb;
        const uint8_t* const F = p.w2_sf + (int64_t)e * p.w2_sfsz + scale_row_off(row, cpa4);
        const int rk = lane < p.T ? rank_of[e * p.T + lane] : kNone;
        uint64_t left = __ballot(rk != kNone);
        while (left) {  // up to 16 of its tokens at a time: lane r takes the r-th
            uint64_t rest = left;
            for (int i = 0; i < r; i++) rest &= rest - 1;
            const int tok = rest ? __builtin_ctzll(rest) : -1;
            for (int i = 0; i < 16; i++) left &= left - 1;
            const int slot = __shfl(rk, tok < 0 ? 0 : tok);
            const int64_t pair = tok < 0 ? 0 : (int64_t)(tok * p.k + slot) * p.I;
            const uint16_t* const XH = tok < 0 ? nullptr : p.act_hi + pair;
            const uint16_t* const XL = tok < 0 ? nullptr : p.act_lo + pair;
            f32x4 acc = {0, 0, 0, 0};
            constexpr int U = 2;
            for (int cb = c0; cb < c1; cb += U) {
                u32x4 w[U], xh[U][4], xl[U][4];
                uint32_t s[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int c = cb + u < c1 ? cb + u : c1 - 1;
                    w[u] = load_w4<WHOLE>(B, c, g, rowb);
                    s[u] = load_s4<WHOLE>(F, c, g, nblk);
                    load_x16<WHOLE>(xh[u], XH, c, g, p.I);
                    load_x16<WHOLE>(xl[u], XL, c, g, p.I);
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (cb + u >= c1) break;
                    const float s0 = __builtin_amdgcn_cvt_f32_fp8(s[u], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(s[u], 1);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const bf16x8 wv = dequant8_bf16(word(w[u], j), j < 2 ? s0 : s1);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, xh[u][j]), acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, xl[u][j]), acc, 0, 0, 0);
                    }
                }
            }
            if (tok >= 0) {
#pragma unroll
                for (int v = 0; v < 4; v++) sums[wave][tok][4 * g + v] += acc[v];
            }
        }
    }
    __syncthreads();
    for (int i = t; i < p.T * 16; i += 64 * kDownWaves) {
        const int tok = i >> 4, col = i & 15;
        float s = sums[0][tok][col];
#pragma unroll
        for (int v = 1; v < kDownWaves; v++) s += sums[v][tok][col];
        p.out[(int64_t)tok * p.H + tile * 16 + col] = (uint16_t)pack_bf16x2(s * inv[tok], 0.0f);
    }
#endif
}

template <int NR>
void launch_up(const EParams& p, dim3 grid, hipStream_t st) {
    if (p.H % kChunk == 0) k_moe_up<NR, true><<<grid, 64 * kUpWaves, 0, st>>>(p);
    else k_moe_up<NR, false><<<grid, 64 * kUpWaves, 0, st>>>(p);
}

}  // namespace

hipError_t launch_moe_small(const MoeSmallArgs& a, hipStream_t st) {
    EParams p{};
    p.x = a.x; p.logits = a.logits; p.lg_bf16 = a.logits_bf16;
    p.w13 = a.w13; p.w13_sf = a.w13_sf; p.alpha13 = a.alpha13;
    p.w2 = a.w2; p.w2_sf = a.w2_sf; p.alpha2 = a.alpha2;
    p.out = a.out; p.ids = a.ids; p.weights = a.weights;
    p.T = a.t; p.H = a.h; p.I = a.inter; p.E = a.E; p.k = a.top_k;
    p.sigmoid = a.sigmoid; p.renorm = a.renorm;
    p.raw = (float*)a.ws;  // T * k <= 1024 floats in the first 4 KiB
    p.act_hi = (uint16_t*)((char*)a.ws + 4096);
    p.act_lo = p.act_hi + (int64_t)a.t * a.top_k * a.inter;
    p.w13_sfsz = (int64_t)((2 * a.inter + 127) / 128 * 128) * ((a.h / 16 + 3) / 4 * 4);
    p.w2_sfsz = (int64_t)((a.h + 127) / 128 * 128) * ((a.inter / 16 + 3) / 4 * 4);
    // fewer pairs than experts: a workgroup row per chosen expert, else one per expert
    p.by_slot = a.t * a.top_k < a.E;
    const int rows = p.by_slot ? a.t * a.top_k : a.E;
    p.tiles = a.inter / 16;
    p.xcd_chunk = p.tiles % 8 == 0 ? p.tiles / 8 : 0;
    const dim3 grid((unsigned)p.tiles, (unsigned)rows);
    const int nr = (a.E + 63) / 64;
    if (nr == 1) launch_up<1>(p, grid, st);
    else if (nr == 2) launch_up<2>(p, grid, st);
    else launch_up<4>(p, grid, st);
    p.tiles = a.h / 16;
    p.xcd_chunk = p.tiles % 8 == 0 ? p.tiles / 8 : 0;
    if (a.inter % kChunk == 0) k_moe_down<true><<<dim3((unsigned)p.tiles), 64 * kDownWaves, 0, st>>>(p);
    else k_moe_down<false><<<dim3((unsigned)p.tiles), 64 * kDownWaves, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace nvfp4
