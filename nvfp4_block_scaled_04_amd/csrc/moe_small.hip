// moe_small.hip -- a whole mixture-of-experts layer for a few tokens in two
// launches (three beyond 32 tokens), on NVFP4 expert weights and bf16 tokens.
//
// What is computed (tokens x, router logits, E experts of H -> I -> H):
//   chosen(i) = the top_k experts by (logit descending, index ascending) among
//               logits that are neither NaN nor -inf
//   w(i, e)   = softmax or sigmoid of the logit (/ the chosen ones' sum)
//   [g, u]    = alpha13[e] * x[i] @ W13[e]^T,   a = g / (1 + e^-g) * u
//   out[i]    = sum_e w(i, e) * alpha2[e] * a @ W2[e]^T
//
// First launch (k_moe_up): every workgroup routes for itself, once -- 16 lanes a
// token, top_k rounds of a maximum over DPP -- and then walks its share of the
// (chosen expert, 16 gate and 16 up rows) items.  A wave streams an item's 32
// weight rows once against up to 16 of the tokens that chose the expert; with
// few items, the K axis of one is split over S waves.  The activation leaves
// multiplied by w(i, e) and alpha2, so the second launch is one long product.
// Second launch (k_moe_down): a workgroup has 128 output columns, 16 a wave, and
// a share of the K axis, which is the chosen experts' I axes laid end to end.  Its
// waves walk the same chunks and share the activations in LDS; each adds an
// expert's product into the fp32 sums of its own columns, and of the several
// workgroups of a column tile the last to finish (beyond 32 tokens, a launch of its
// own) adds their sums in the order of the shares: no atomic sums, the same result
// on every call.
//
// Bound: the chosen experts' weights (9/16 byte an element), the rest is small.  They
// are read once where up to 32 tokens (second launch: 16) chose an expert, and again
// for every 32 (16) more, from the caches if they fit there: 64 tokens that all choose
// the same 4 experts of 4096 x 2048 take 59 + 81 us and read 78 + 41 MB past the L2s,
// for 38 + 19 MB of weights.
#include "device_common.h"
#include "gemm_common.h"
#include "internal.h"
#include "skinny_w4.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 8;    // of either kernel's workgroups; two of them share a CU
constexpr int kThreads = 64 * kWaves;
constexpr int kXBytes = 16 << 10;  // LDS for activations: 4 chunks of 16 rows, 64 of one
constexpr int kInvBytes = kXBytes / 64;  // a float per row and chunk
typedef W4Ring<2, 3> UpRing;       // with x and the tables, LDS for two workgroups a CU

// Second launch: up to 32 tokens, two workgroups of 8 waves share a CU; beyond, the
// sums take the LDS, and one workgroup of 16 waves has a CU where there are enough
// columns for that (64 tokens over 32 experts of 4096 x 2048: 53 us, 67 with 8
// waves; 61 tokens over 60 of 2064 x 1104, too few: 53 us, 41 with 8 waves).
template <int NW>
struct DownShape {
    typedef W4Ring<1, NW == 8 ? 4 : 3> Ring;
    static constexpr int kX = NW == 8 ? 16 << 10 : 24 << 10;  // LDS for activations
    static constexpr int kInv = kX / 64;                      // a float per row and chunk
    static constexpr int kPitch = 16 * NW + 4;                // floats of a token's row of sums
    static constexpr int kFixed = NW * Ring::BYTES + kX + kInv;
};

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
    void* routes;              // Routes, from the first launch for the second
    int32_t* arrived;          // [8 * ceil(H/128)] shares of a column tile that are done (k_moe_down)
    float* act;                // [T * k, I], row t * k + slot: w(i, e) * alpha2 * a
    float* part;               // [8 * ceil(H/128), shares, T, 16] partial sums (k_moe_down with shares > 1)
    int64_t w13_sfsz, w2_sfsz; // scale bytes of one expert
    int T, H, I, E, k;
    int lg_bf16, sigmoid, renorm;
    int shares;                // most workgroups that share a column tile (k_moe_down)
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ float row16_sum(float v) {
    return row16(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ int row16_min(int v) {
    return row16(v, [](int a, int b) { return a < b ? a : b; });
}

// The value of lane l ^ 8 within a row of 16 (DPP row_ror:8).
__device__ __forceinline__ float row_half(float v) {
    return bits_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f_bits(v), 0x128, 0xF, 0xF, true));
}

// What the launches know of the routing: the chosen experts, ascending, each
// packed with its number of tokens and the start of their list, and the lists of
// (token, slot), tokens ascending.  The first launch makes it in LDS and leaves a
// copy in the workspace for the second.
struct alignas(16) Routes {
    uint32_t act[256];    // expert | tokens << 8 | first of the list << 16
    uint16_t list[1024];  // token << 4 | slot
    int32_t nact;
};
static_assert(sizeof(Routes) <= 4096, "room in the workspace");
__device__ __forceinline__ int act_expert(uint32_t a) { return a & 255; }
__device__ __forceinline__ int act_tokens(uint32_t a) { return a >> 8 & 255; }
__device__ __forceinline__ int act_first(uint32_t a) { return a >> 16; }

// Exclusive prefix sum over a wave; total: the whole sum.
__device__ __forceinline__ int wave_prefix(int v, int& total) {
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int u = __shfl_up(s, o);
        if ((int)(threadIdx.x & 63) >= o) s += u;
    }
    total = __shfl(s, 63);
    return s - v;
}

// NR: logits a lane holds of a token (E <= 16 NR).
// Bound: the reads of W13 where there is enough of it (16 tokens of 8 experts of
// 5120 x 8192, about 333 MB: 88 us, 3.8 TB/s; 64 tokens of 32 experts of 4096 x 2048,
// 302 MB: 77 us, 3.9 TB/s; a copy of 2 GiB moves 4.9, reads alone 5.2 to 5.9), and the
// routing, the first loads and the waves' sums otherwise (7 to 8 us of one token's 18.5
// for 47 MB, and of the 22.4 of 4 tokens over 128 experts of 2048 x 768).  Items are dealt
// whole, so a grid that they do not fill or just exceed waits for the last: 61 tokens
// over 60 experts of 2064 x 1104 are 540 items for 512 workgroups, 154 MB in 69 us, and
// about 174 items of 256 workgroups leave a third of them idle in the case of 4 tokens.
// 20 registers spill at four waves a SIMD (25 where H % 128 != 0), which shows as 6 to 25
// MB written a call, up to 2 of them the activations.
template <int NR, bool WHOLE>
__global__ __launch_bounds__(kThreads, 4) void k_moe_up(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass only needs the launch stub
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const rings = smem;                             // the waves' weight rings; then the parts' sums
    uint8_t* const xs = smem + kWaves * UpRing::BYTES;       // x of a block of chunks
    float* const inv = (float*)(xs + kXBytes);               // their inverse scales
    Routes& R = *(Routes*)(xs + kXBytes + kInvBytes);
    float* const weight_of = (float*)(&R + 1);               // [T * k]
    int16_t* const choice = (int16_t*)(weight_of + p.T * p.k);  // [T][k]
    int* const count = (int*)rings;                          // [256] tokens of an expert (before the rings are used)
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);

    // 1. routing: 16 lanes a token, its logits in registers (the first tokens' are on
    //    their way while the counts are cleared; bf16 ones the compiler loads one after
    //    another, 2 us of 28 at 256 experts)
    const int l16 = lane & 15;
    auto load_logits = [&](int tok, float (&lg)[NR]) {
#pragma unroll
        for (int i = 0; i < NR; i++) {
            const int j = l16 + 16 * i;
            lg[i] = neg_inf();
            if (tok < p.T && j < p.E) {
                const int64_t at = (int64_t)tok * p.E + j;
                lg[i] = p.lg_bf16 ? bf16_lo((uint32_t)((const uint16_t*)p.logits)[at]) : ((const float*)p.logits)[at];
            }
        }
    };
    float lg[NR];
    load_logits(wave * 4 + (lane >> 4), lg);
    if (t < 256) count[t] = 0;
    if (blockIdx.x == 0)
        for (int i = t; i < (p.H + 127) / 128 * 8; i += kThreads) p.arrived[i] = 0;
    __syncthreads();
    for (int t0 = wave * 4; t0 < p.T; t0 += kWaves * 4) {
        const int tok = t0 + (lane >> 4);
        if (t0 >= kWaves * 4) load_logits(tok, lg);
#pragma unroll
        for (int i = 0; i < NR; i++) lg[i] = lg[i] == lg[i] ? lg[i] : neg_inf();  // NaN is never chosen
        float top = lg[0];
#pragma unroll
        for (int i = 1; i < NR; i++) top = __builtin_fmaxf(top, lg[i]);
        top = row16_max(top);
        float den = 1.0f;
        if (!p.sigmoid && !p.renorm) {
            den = 0.0f;
#pragma unroll
            for (int i = 0; i < NR; i++) den += lg[i] == neg_inf() ? 0.0f : expf(lg[i] - top);
            den = row16_sum(den);
        }
        int mine = -1;            // lane j of the token keeps the expert of slot j
        float ml = neg_inf();
        for (int j = 0; j < p.k; j++) {
            float m = lg[0];
#pragma unroll
            for (int i = 1; i < NR; i++) m = __builtin_fmaxf(m, lg[i]);
            m = row16_max(m);
            int at = p.E;  // the lowest index that holds the maximum
#pragma unroll
            for (int i = NR - 1; i >= 0; i--)
                if (lg[i] == m) at = l16 + 16 * i;
            at = row16_min(at);
            if (m > neg_inf() && l16 == j) {
                mine = at;
                ml = m;
            }
#pragma unroll
            for (int i = 0; i < NR; i++)
                if (l16 + 16 * i == at) lg[i] = neg_inf();
        }
        // its weight.  Softmax: exp(l - top) over the sum of all, or of the chosen
        // ones.  Sigmoid over the chosen ones' sum: every value is scaled by
        // exp(-min(top, 0)), so that very negative logits keep their ratios.
        float u = 0.0f;
        if (mine >= 0) {
            if (!p.sigmoid) u = expf(ml - top) / den;
            else if (ml >= 0.0f) u = 1.0f / (1.0f + expf(-ml));
            else u = expf(ml - (p.renorm ? __builtin_fminf(top, 0.0f) : 0.0f)) / (1.0f + expf(ml));
        }
        if (p.renorm) {
            const float s = row16_sum(u);
            if (mine >= 0) u /= s;
        }
        if (tok < p.T && l16 < p.k) {
            weight_of[tok * p.k + l16] = u;
            choice[tok * p.k + l16] = (int16_t)mine;
            if (mine >= 0) atomicAdd(&count[mine], 1);
            if (blockIdx.x == 0) {
                p.ids[tok * p.k + l16] = mine;
                p.weights[tok * p.k + l16] = u;
            }
        }
    }
    __syncthreads();
    // the chosen experts: every wave writes the same list and reads back its own
    int nact = 0, pairs = 0, most = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        const int n = e0 + lane < p.E ? count[e0 + lane] : 0;
        const uint64_t some = __ballot(n > 0);
        int sum;
        const int first = pairs + wave_prefix(n, sum);
        if (n > 0)
            R.act[nact + __builtin_popcountll(some & (((uint64_t)1 << lane) - 1))] =
                (uint32_t)(e0 + lane) | (uint32_t)n << 8 | (uint32_t)first << 16;
        nact += __builtin_popcountll(some);
        pairs += sum;
        most = most > n ? most : n;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const int u = __shfl_xor(most, o);
        most = most > u ? most : u;
    }
    nact = __builtin_amdgcn_readfirstlane(nact);
    most = __builtin_amdgcn_readfirstlane(most);
    __builtin_amdgcn_wave_barrier();
    // an expert's tokens, lane by lane, into its place of the list
    auto list_tokens = [&](uint32_t a) {
        int slot = -1;
        if (lane < p.T)
            for (int j = 0; j < p.k; j++)
                if (choice[lane * p.k + j] == act_expert(a)) slot = j;
        const uint64_t in = __ballot(slot >= 0);
        if (slot >= 0) R.list[act_first(a) + __builtin_popcountll(in & (((uint64_t)1 << lane) - 1))] = (uint16_t)(lane << 4 | slot);
        __builtin_amdgcn_wave_barrier();
    };
    if (blockIdx.x == gridDim.x - 1) {  // the copy for the second launch
        if (t == 0) R.nact = nact;
        for (int i = wave; i < nact; i += kWaves) list_tokens(R.act[i]);
        __syncthreads();
        for (int i = t; i < (int)sizeof(Routes) / 4; i += kThreads) ((uint32_t*)p.routes)[i] = ((const uint32_t*)&R)[i];
    }
    __syncthreads();  // count shares the rings' LDS

    // 2. items: (chosen expert, up to 8 / S tiles of 16 gate and 16 up rows), the K
    //    axis of a tile split over S waves: as many as give every wave something,
    //    as long as LDS holds a chunk of x for each part
    const int r = lane & 15, g = lane >> 4;
    const int rowb = p.H / 2, cpa4 = (p.H / 16 + 3) / 4;
    const int nch = (p.H + kChunk - 1) / kChunk;
    const int tiles = (p.I + 127) / 128 * 8;
    const int rows_most = most < 32 ? most : 32;
    int S = 1;
    while (S < kWaves && nact * tiles * S * 2 <= (int)gridDim.x * kWaves && 2 * S * rows_most * 256 <= kXBytes) S *= 2;
    const int ipw = kWaves / S, sub = wave / S, part_of = wave % S;
    const int gpe = (tiles + ipw - 1) / ipw, items = nact * gpe;  // groups of an expert, of all
    const int cps = (nch + S - 1) / S;                            // chunks of a part
    const int c0 = cps * part_of < nch ? cps * part_of : nch, c1 = c0 + cps < nch ? c0 + cps : nch;
    const int G = gridDim.x, b = blockIdx.x;
    // S workgroups cover the 8 tiles of a band of 128 rows, whose scales share
    // lines: they are neighbours on one XCD (workgroups are dealt round-robin)
    const int w0 = G % (8 * S) == 0 ? (b / 8 / S * 8 + b % 8) * S + b / 8 % S : b;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, (uint32_t)(p.T * p.H * 2));
    UpRing ring;
    ring.init(rings + wave * UpRing::BYTES, lane);
    for (int idx = w0; idx < items; idx += G) {
        const int ai = idx / gpe, tile = (idx - ai * gpe) * ipw + sub;
        const uint32_t a = (uint32_t)__builtin_amdgcn_readfirstlane((int)R.act[ai]);
        const int e = act_expert(a), n = act_tokens(a);
        const uint16_t* const list = R.list + act_first(a);
        list_tokens(a);  // every wave the same
        const bool live = tile < tiles;
        const float a13 = p.alpha13[e], a2 = p.alpha2[e];
        ring.aim(make_rsrc(p.w13 + (int64_t)e * 2 * p.I * rowb, (uint32_t)(2 * p.I * rowb)),
                 make_rsrc(p.w13_sf + (int64_t)e * p.w13_sfsz, (uint32_t)p.w13_sfsz),
                 {0, p.I}, {p.I, 2 * p.I}, live ? tile : 0, 0, rowb, cpa4, lane);
        // XT tiles of 16 tokens at a time, the first of them the m0-th
        auto pass = [&](auto xt, int m0) {
            constexpr int XT = decltype(xt)::value;
            const int nr = n - m0 < 16 * XT ? n - m0 : 16 * XT;  // rows of x
            const int cb = kXBytes / (nr * 256) / S;             // chunks of every part in a block
            if (idx != w0 || m0) __syncthreads();  // nobody is at the previous pass's LDS any more
            int ca = c0;
            auto next = [&]() {
                if (ca < c1) ring.issue(ca++);
            };
            if (live)
                for (int u = 0; u < UpRing::DEPTH; u++) next();
            XBlock<kXBytes / 16 / kThreads, false> xb;
            xb.prepare(
                nr, nr, S * cb, t, kThreads, [&](int R_) { return (uint32_t)((list[m0 + R_] >> 4) * p.H * 2); },
                [&](int lc) { return cps * (lc / cb) + lc % cb; },
                [&](int lc) { return cps * (lc / cb + 1) < nch ? cps * (lc / cb + 1) : nch; });
            xb.load(rx, 0, p.H, t);
            XLane xl[XT];
#pragma unroll
            for (int i = 0; i < XT; i++) {
                const int row = 16 * i + r < nr ? 16 * i + r : nr - 1;  // absent: any row
                xl[i].set(xs, inv, row, row, g);
            }
            f32x4 acc[2][XT];
#pragma unroll
            for (int f = 0; f < 2; f++)
#pragma unroll
                for (int i = 0; i < XT; i++) acc[f][i] = f32x4{0, 0, 0, 0};
            for (int k0 = 0; k0 < cps; k0 += cb) {
                if (k0) __syncthreads();  // the previous block is consumed
                xb.store(xs, inv, 0, k0, t);
                __syncthreads();
                if (k0 + cb < cps) xb.load(rx, k0 + cb, p.H, t);  // the next block is on its way while this one is used
                const int b0 = c0 + k0, b1 = b0 + cb < c1 ? b0 + cb : c1;
                if (live) consume<XT, WHOLE>(ring, acc, xl, part_of * cb * nr, nr, b0, b1, g, p.H, next);
            }
            if (S > 1) {  // the parts' sums, in part order
                __syncthreads();
                f32x4* const part = (f32x4*)rings;
#pragma unroll
                for (int f = 0; f < 2; f++)
#pragma unroll
                    for (int i = 0; i < XT; i++) part[((f * XT + i) * kWaves + wave) * 64 + lane] = acc[f][i];
                __syncthreads();
                if (part_of != 0) return;
                for (int v = 1; v < S; v++)
#pragma unroll
                    for (int f = 0; f < 2; f++)
#pragma unroll
                        for (int i = 0; i < XT; i++) acc[f][i] += part[((f * XT + i) * kWaves + wave + v) * 64 + lane];
            }
#pragma unroll
            for (int i = 0; i < XT; i++) {
                const int col = band_row(tile, 4 * g);  // lane: its token, columns col .. col + 3 (I is a multiple of 16)
                if (!live || 16 * i + r >= nr || col >= p.I) continue;
                const int it = list[m0 + 16 * i + r], pair = (it >> 4) * p.k + (it & 15);
                const float wt = weight_of[pair] * a2;
                float v4[4];
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    const float gt = a13 * acc[0][i][v];
                    v4[v] = gt / (1.0f + expf(-gt)) * (a13 * acc[1][i][v]) * wt;
                }
                *(f32x4*)(p.act + (int64_t)pair * p.I + col) = f32x4{v4[0], v4[1], v4[2], v4[3]};
            }
        };
        if (n <= 16) {
            pass(std::integral_constant<int, 1>{}, 0);
        } else {
            for (int m0 = 0; m0 < n; m0 += 32) pass(std::integral_constant<int, 2>{}, m0);
        }
    }
#endif
}

// Shares of the second launch's K axis, of 12 chunks at least (4 tokens over 128
// experts of 2048 x 768: 17.9 us, of 4, 8 or 16 chunks at least 21.3, 20.4, 21.4).
constexpr int kShareChunks = 12;
__device__ __forceinline__ int shares_of(int total, int most) {
    return total >= kShareChunks * most ? most : total < kShareChunks ? 1 : total / kShareChunks;
}
// Tokens up to which k_moe_down adds the shares itself (16 tokens of 8 experts of
// 5120 x 8192: 50.3 us, with a launch of its own 52.8; 64 tokens of 32 experts of
// 4096 x 2048: 66 us, 59.2).
constexpr int kOwnSum = 32;

// Workgroup (16 NW output columns, share of the K axis): a wave has 16 columns to
// itself, and all walk the same (expert, chunk) range.
// Bound: the reads of W2 and the step from expert to expert (16 tokens of 8 experts
// of 5120 x 8192, 167 MB: 50.3 us, 3.3 TB/s; 64 of 32 of 4096 x 2048, 151 MB: 53.4 us,
// 2.8 TB/s); with few bytes the chain of routes, first weights, sums and their
// exchange (one token, 24 MB: 14.1 us; 4 tokens over 128 of 2048 x 768, 26 MB: 17.9).
// The compiler holds the ring's state per lane, since both pass forms share it: the
// weight loads of a chunk sit in loops over distinct lane values (one turn each), which
// costs VALU instructions (22 to 31 an MFMA, 14 to 24 in k_moe_up), and 14 registers spill.
template <int NW, bool WHOLE>
__global__ __launch_bounds__(64 * NW, 4) void k_moe_down(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef DownShape<NW> Shape;
    typedef typename Shape::Ring Ring;
    constexpr int kThreads = 64 * NW, kXBytes = Shape::kX, D = Ring::DEPTH, kSumPitch = Shape::kPitch;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const rings = smem;                             // the waves' weight rings
    uint8_t* const xs = smem + NW * Ring::BYTES;             // activations of a block of chunks
    float* const inv = (float*)(xs + kXBytes);               // their inverse scales
    Routes& R = *(Routes*)(xs + kXBytes + Shape::kInv);
    float* const sums = (float*)(&R + 1);                    // [T][kSumPitch]: sums of every token and column
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);

    for (int i = t; i < (int)sizeof(Routes) / 4; i += kThreads) ((uint32_t*)&R)[i] = ((const uint32_t*)p.routes)[i];
    for (int i = t; i < p.T * kSumPitch; i += kThreads) sums[i] = 0.0f;
    __syncthreads();
    const int nact = __builtin_amdgcn_readfirstlane(R.nact);

    const int r = lane & 15, g = lane >> 4;
    const int rowb = p.I / 2, cpa4 = (p.I / 16 + 3) / 4;
    const int nch = (p.I + kChunk - 1) / kChunk;
    const int total = nact * nch;
    const int shares = shares_of(total, p.shares);  // the rest of the workgroups has nothing to do
    const int share = blockIdx.y;
    if (share >= shares) return;
    const int tile = blockIdx.x * NW + wave;  // the wave's 16 columns: band_row(tile, 0 .. 15)
    const int mine0 = (wave >> 3) * 128 + (wave & 7) * 4;  // the first of them in sums; 32 apart from 4 to 4
    const bool live = band_row(tile, 0) < p.H;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.act, (uint32_t)(p.T * p.k * p.I * 4));
    const int q0 = (int)((int64_t)total * share / shares), q1 = (int)((int64_t)total * (share + 1) / shares);
    // A pass: the chunks of [q0, q1) that lie in one expert, with up to 16 of its
    // tokens (8 where it has no more).
    struct Pass {
        int at, m0;
    };
    const int last = (q1 - 1) / nch;  // place of the range's last expert
    auto act_of = [&](int at) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)R.act[at]); };
    auto after = [&](Pass q) {
        q.m0 += 16;
        if (q.m0 >= act_tokens(act_of(q.at))) q = Pass{q.at + 1, 0};
        return q;
    };
    auto begin_of = [&](int at) { return q0 > at * nch ? q0 - at * nch : 0; };
    auto end_of = [&](int at) { return q1 - at * nch < nch ? q1 - at * nch : nch; };
    auto tokens_of = [&](Pass q) {
        const int n = act_tokens(act_of(q.at)) - q.m0;
        return n < 16 ? n : 16;
    };
    Ring ring;
    ring.init(rings + wave * Ring::BYTES, lane);
    Pass aimed = {q0 / nch, 0};
    int ca = 0, ce = 0;
    auto aim = [&]() {
        ca = ce = 0;
        if (!live || aimed.at > last) return;
        const int e = act_expert(act_of(aimed.at));
        ring.aim(make_rsrc(p.w2 + (int64_t)e * p.H * rowb, (uint32_t)(p.H * rowb)),
                 make_rsrc(p.w2_sf + (int64_t)e * p.w2_sfsz, (uint32_t)p.w2_sfsz), {0}, {p.H}, tile, 0, rowb, cpa4, lane);
        ca = begin_of(aimed.at);
        ce = end_of(aimed.at);
    };
    auto next = [&]() {
        while (ca == ce && aimed.at <= last) {
            aimed = after(aimed);
            aim();
        }
        if (ca < ce) ring.issue(ca++);
    };
    // chunks of a block: what LDS holds and one piece a thread fills
    auto block_of = [&](int nt) { return kXBytes / (nt * 512) < kThreads / (nt * 16) ? kXBytes / (nt * 512) : kThreads / (nt * 16); };
    XBlock<1, true> xb;
    auto prepare = [&](Pass q) {  // rows in LDS: the tokens' high halves, then their low ones
        const int nt = tokens_of(q), end = end_of(q.at), begin = begin_of(q.at);
        const uint16_t* const list = R.list + act_first(act_of(q.at)) + q.m0;
        xb.prepare(
            nt, 2 * nt, block_of(nt), t, kThreads,
            [&](int i) { return (uint32_t)(((list[i] >> 4) * p.k + (list[i] & 15)) * p.I * 4); },
            [&](int lc) { return begin + lc; }, [&](int) { return end; });
    };
    Pass cur = {q0 / nch, 0};
    if (total > 0) {
        aim();
        for (int u = 0; u < D; u++) next();
        prepare(cur);
        xb.load(rx, 0, p.I, t);
    }
    while (total > 0 && cur.at <= last) {
        const Pass nxt = after(cur);
        const int c0 = begin_of(cur.at), c1 = end_of(cur.at);
        const int nt = tokens_of(cur), nr = 2 * nt, cb = block_of(nt);
        // XT = 1: up to 8 tokens, lanes r < 8 with their activations' high halves and
        // the others with the low ones; XT = 2: up to 16, a tile of each
        auto pass = [&](auto xt) {
            constexpr int XT = decltype(xt)::value, NT = 8 * XT;
            XLane xl[XT];
            const int tl = (r & (NT - 1)) < nt ? r & (NT - 1) : nt - 1;  // absent: any row
            if constexpr (XT == 1) {
                xl[0].set(xs, inv, (r >> 3) * nt + tl, tl, g);
            } else {
                xl[0].set(xs, inv, tl, tl, g);
                xl[1].set(xs, inv, nt + tl, tl, g);
            }
            f32x4 acc[1][XT];
#pragma unroll
            for (int i = 0; i < XT; i++) acc[0][i] = f32x4{0, 0, 0, 0};
            for (int b0 = c0; b0 < c1; b0 += cb) {
                const int b1 = b0 + cb < c1 ? b0 + cb : c1;
                __syncthreads();  // the previous block is consumed
                xb.store(xs, inv, nt, b0 - c0, t);
                __syncthreads();
                // the next block is on its way while this one is used
                if (b1 < c1) {
                    xb.load(rx, b1 - c0, p.I, t);
                } else if (nxt.at <= last) {
                    prepare(nxt);
                    xb.load(rx, 0, p.I, t);
                }
                if (live) consume<XT, WHOLE>(ring, acc, xl, 0, nr, b0, b1, g, p.I, next);
            }
            const int it = R.list[act_first(act_of(cur.at)) + cur.m0 + tl];
#pragma unroll
            for (int v = 0; v < 4; v++) {
                const float s = acc[0][0][v] + (XT == 1 ? row_half(acc[0][0][v]) : acc[0][XT - 1][v]);
                if (r < nt) sums[(it >> 4) * kSumPitch + mine0 + 32 * g + v] += s;
            }
        };
        if (nt <= 8) pass(std::integral_constant<int, 1>{});
        else pass(std::integral_constant<int, 2>{});
        cur = nxt;
    }
    // the wave's own columns (no other wave of the workgroup has touched them), four
    // of a token at a time: item i is token i / 4, quarter i % 4
    if (!live) return;
    auto mine = [&](int i) { return *(const f32x4*)&sums[(i >> 2) * kSumPitch + mine0 + (i & 3) * 32]; };
    auto put = [&](int i, f32x4 v) {
        const int col = band_row(tile, 4 * (i & 3));
        if (col < p.H)  // H is a multiple of 16
            *(u32x2*)(p.out + (int64_t)(i >> 2) * p.H + col) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
    if (shares == 1) {
        for (int i = lane; i < p.T * 4; i += 64) put(i, mine(i));
        return;
    }
    // several workgroups have these columns: each leaves its sums in memory.  Up to
    // kOwnSum tokens the wave that finds the others done adds them, in the order of
    // the shares; beyond, k_moe_sum does, since one wave would take 13 us to (64
    // tokens, 16 shares).  Device-scope stores and loads (sc1) pass by the XCDs' own
    // L2s, so no cache is written back or dropped; the stores are waited for before
    // the count.
    constexpr int kDevice = 16;
    const int n16 = p.T * 64;  // bytes of a share's sums of this tile
    const __amdgpu_buffer_rsrc_t part = make_rsrc(p.part + (int64_t)tile * p.shares * p.T * 16, (uint32_t)(shares * n16));
    for (int i = lane; i < p.T * 4; i += 64) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, mine(i)), part, i * 16, share * n16, kDevice);
    }
    if (p.T > kOwnSum) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int before = 0;
    if (lane == 0) before = __hip_atomic_fetch_add(&p.arrived[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(before) != shares - 1) return;
    asm volatile("" ::: "memory");
    for (int i = lane; i < p.T * 4; i += 64) {
        f32x4 s = {0, 0, 0, 0};
        constexpr int U = 16;  // loads in flight together
        for (int v0 = 0; v0 < shares; v0 += U) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; u++)  // past the last share: past the resource, zeros
                v[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(part, i * 16 + (v0 + u) * n16, 0, kDevice));
#pragma unroll
            for (int u = 0; u < U; u++) s += __builtin_bit_cast(f32x4, v[u]);
        }
        put(i, s);
    }
#endif
}

// The shares' sums in their order, where k_moe_down leaves them: four columns of a
// token a thread.
__global__ __launch_bounds__(256) void k_moe_sum(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int shares = shares_of(((const Routes*)p.routes)->nact * ((p.I + kChunk - 1) / kChunk), p.shares);
    if (shares == 1) return;  // written already
    const int n4 = p.T * 4;  // float4s of a share's sums of a tile
    const int id = blockIdx.x * 256 + threadIdx.x;
    const int tile = id / n4, i = id % n4, col = band_row(tile, 4 * (i & 3));
    if (tile >= (p.H + 127) / 128 * 8 || col >= p.H) return;
    const f32x4* const P = (const f32x4*)p.part + (int64_t)tile * p.shares * n4 + i;
    f32x4 s = {0, 0, 0, 0};
    constexpr int U = 16;  // loads in flight together
    for (int v0 = 0; v0 < shares; v0 += U) {
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; u++) v[u] = v0 + u < shares ? P[(int64_t)(v0 + u) * n4] : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < U; u++) s += v[u];
    }
    *(u32x2*)(p.out + (int64_t)(i >> 2) * p.H + col) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
#endif
}

template <int NR>
void launch_up(const EParams& p, int grid, size_t lds, hipStream_t st) {
    if (p.H % kChunk == 0) k_moe_up<NR, true><<<grid, kThreads, lds, st>>>(p);
    else k_moe_up<NR, false><<<grid, kThreads, lds, st>>>(p);
}

template <int NW>
void launch_down(EParams p, int cus, int most_shares, hipStream_t st) {
    typedef DownShape<NW> Shape;
    // enough workgroups for every CU, as far as the partial sums have room
    const int cols = (p.H + 16 * NW - 1) / (16 * NW);
    p.shares = (p.T <= 32 ? 2 : 1) * cus / cols;
    if (p.shares > most_shares) p.shares = most_shares;
    if (p.shares < 1) p.shares = 1;
    const size_t lds = Shape::kFixed + sizeof(Routes) + (size_t)p.T * Shape::kPitch * 4;
    const dim3 grid((unsigned)cols, (unsigned)p.shares);
    if (p.I % kChunk == 0) k_moe_down<NW, true><<<grid, 64 * NW, lds, st>>>(p);
    else k_moe_down<NW, false><<<grid, 64 * NW, lds, st>>>(p);
    if (p.T > kOwnSum && p.shares > 1) k_moe_sum<<<(unsigned)(((p.H + 127) / 128 * 8 * p.T * 4 + 255) / 256), 256, 0, st>>>(p);
}

}  // namespace

hipError_t launch_moe_small(const MoeSmallArgs& a, hipStream_t st) {
    const int cus = device_cus();
    if (cus <= 0) return hipErrorInvalidDevice;
    EParams p{};
    p.x = a.x; p.logits = a.logits; p.lg_bf16 = a.logits_bf16;
    p.w13 = a.w13; p.w13_sf = a.w13_sf; p.alpha13 = a.alpha13;
    p.w2 = a.w2; p.w2_sf = a.w2_sf; p.alpha2 = a.alpha2;
    p.out = a.out; p.ids = a.ids; p.weights = a.weights;
    p.T = a.t; p.H = a.h; p.I = a.inter; p.E = a.E; p.k = a.top_k;
    p.sigmoid = a.sigmoid; p.renorm = a.renorm;
    p.w13_sfsz = (int64_t)((2 * a.inter + 127) / 128 * 128) * ((a.h / 16 + 3) / 4 * 4);
    p.w2_sfsz = (int64_t)((a.h + 127) / 128 * 128) * ((a.inter / 16 + 3) / 4 * 4);
    // workspace: the activations, the partial sums of the second
    // launch (kMoePartRows rows of h), the tiles' counters
    const int64_t acts = (int64_t)a.t * a.top_k * a.inter;
    p.act = (float*)a.ws;
    p.part = p.act + acts;
    p.routes = p.part + (int64_t)kMoePartRows * ((a.h + 127) / 128 * 128);
    p.arrived = (int32_t*)((char*)p.routes + 4096);
    const int most = a.t * a.top_k < a.E ? a.t * a.top_k : a.E;  // experts that can be chosen
    // first launch: two workgroups a CU, one where that leaves a wave fewer than 8
    // chunks (one token over 8 experts of 5120 x 8192: 16.8 us against 19.0; at 40
    // chunks a wave, 92 against 90), or one per tile if there are fewer
    const int64_t items = (int64_t)most * ((a.inter + 127) / 128 * 8);
    const bool few = items * ((a.h + kChunk - 1) / kChunk) < 8 * (int64_t)(2 * cus * kWaves);
    const int wgs = few ? cus : 2 * cus;
    const int grid = (int)(items < wgs ? items : wgs);
    const size_t lds = kWaves * UpRing::BYTES + kXBytes + kInvBytes + sizeof(Routes) + (size_t)a.t * a.top_k * 6;
    if (a.E <= 16) launch_up<1>(p, grid, lds, st);
    else if (a.E <= 64) launch_up<4>(p, grid, lds, st);
    else if (a.E <= 128) launch_up<8>(p, grid, lds, st);
    else launch_up<16>(p, grid, lds, st);
    const int shares = kMoePartRows / a.t < 32 ? kMoePartRows / a.t : 32;
    if (a.t > 32 && (a.h + 255) / 256 * shares >= cus) launch_down<16>(p, cus, shares, st);
    else launch_down<8>(p, cus, shares, st);
    return hipGetLastError();
}

}  // namespace nvfp4
