// moe_small.hip -- a whole mixture-of-experts layer for a few tokens in two
// launches, on NVFP4 expert weights and bf16 tokens.
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
// workgroups of a column tile the last to finish adds their sums in the order of
// the shares: no atomic sums, the same result on every call.
//
// Bound: the chosen experts' weights are read once (9/16 byte an element), the
// rest is small; the kernels are built to keep weight loads in flight.
#include "device_common.h"
#include "gemm_common.h"
#include "internal.h"
#include "skinny_w4.h"

#include <type_traits>

namespace nvfp4 {
namespace {

constexpr int kWaves = 8;    // of either kernel's workgroups; two of them share a CU
constexpr int kThreads = 64 * kWaves;
constexpr int kXBytes = 16 << 10;  // LDS for activations: 4 chunks of 16 rows, 64 of one
constexpr int kSumPitch = 132;     // floats of a token's row of sums (128 columns, padded)
typedef W4Ring<2, 3> UpRing;       // with x and the tables, LDS for two workgroups a CU

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
    int32_t* arrived;          // [H/16] shares of a column tile that are done (k_moe_down)
    uint16_t* act_hi;          // [T * k, I], row t * k + slot
    uint16_t* act_lo;
    float* part;               // [H/16, shares, T, 16] partial sums (k_moe_down with shares > 1)
    int64_t w13_sfsz, w2_sfsz; // scale bytes of one expert
    int T, H, I, E, k;
    int lg_bf16, sigmoid, renorm;
    int shares;                // most workgroups that share a column tile (k_moe_down)
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

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
    int32_t most;         // most tokens on one expert
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
template <int NR, bool WHOLE>
__global__ __launch_bounds__(kThreads, 4) void k_moe_up(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass only needs the launch stub
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const rings = smem;                             // the waves' weight rings; then the parts' sums
    uint8_t* const xs = smem + kWaves * UpRing::BYTES;       // x of a block of chunks
    Routes& R = *(Routes*)(xs + kXBytes);
    float* const weight_of = (float*)(&R + 1);               // [T * k]
    int16_t* const choice = (int16_t*)(weight_of + p.T * p.k);  // [T][k]
    int* const count = (int*)rings;                          // [256] tokens of an expert (before the rings are used)
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);

    // 1. routing: 16 lanes a token, its logits in registers
    if (t < 256) count[t] = 0;
    if (blockIdx.x == 0)
        for (int i = t; i < p.H / 16; i += kThreads) p.arrived[i] = 0;
    __syncthreads();
    const int l16 = lane & 15;
    for (int t0 = wave * 4; t0 < p.T; t0 += kWaves * 4) {
        const int tok = t0 + (lane >> 4);
        float lg[NR];
#pragma unroll
        for (int i = 0; i < NR; i++) {
            const int j = l16 + 16 * i;
            lg[i] = neg_inf();
            if (tok < p.T && j < p.E) {
                const int64_t at = (int64_t)tok * p.E + j;
                const float v = p.lg_bf16 ? bf16_lo((uint32_t)((const uint16_t*)p.logits)[at]) : ((const float*)p.logits)[at];
                lg[i] = v == v ? v : neg_inf();  // NaN is never chosen
            }
        }
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
    if (wave == 0) {
        int na = 0, pairs = 0, most = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const int n = e0 + lane < p.E ? count[e0 + lane] : 0;
            int sum;
            const int first = pairs + wave_prefix(n, sum);
            const uint64_t some = __ballot(n > 0);
            if (n > 0)
                R.act[na + __builtin_popcountll(some & (((uint64_t)1 << lane) - 1))] =
                    (uint32_t)(e0 + lane) | (uint32_t)n << 8 | (uint32_t)first << 16;
            na += __builtin_popcountll(some);
            pairs += sum;
            most = most > n ? most : n;
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const int u = __shfl_xor(most, o);
            most = most > u ? most : u;
        }
        if (lane == 0) {
            R.nact = na;
            R.most = most;
        }
    }
    __syncthreads();
    const int nact = __builtin_amdgcn_readfirstlane(R.nact);
    for (int i = wave; i < nact; i += kWaves) {  // an expert's tokens, lane by lane
        const uint32_t a = R.act[i];
        int slot = -1;
        if (lane < p.T)
            for (int j = 0; j < p.k; j++)
                if (choice[lane * p.k + j] == act_expert(a)) slot = j;
        const uint64_t in = __ballot(slot >= 0);
        if (slot >= 0) R.list[act_first(a) + __builtin_popcountll(in & (((uint64_t)1 << lane) - 1))] = (uint16_t)(lane << 4 | slot);
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = t; i < (int)sizeof(Routes) / 4; i += kThreads) ((uint32_t*)p.routes)[i] = ((const uint32_t*)&R)[i];

    // 2. items: (chosen expert, up to 8 / S tiles of 16 gate and 16 up rows), the K
    //    axis of a tile split over S waves: as many as give every wave something,
    //    as long as LDS holds a chunk of x for each part
    const int r = lane & 15, g = lane >> 4;
    const int rowb = p.H / 2, cpa4 = (p.H / 16 + 3) / 4;
    const int nch = (p.H + kChunk - 1) / kChunk;
    const int tiles = p.I / 16;
    const int most = __builtin_amdgcn_readfirstlane(R.most), rows_most = most < 32 ? most : 32;
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
        const bool live = tile < tiles;
        const float a13 = p.alpha13[e], a2 = p.alpha2[e];
        ring.aim(make_rsrc(p.w13 + (int64_t)e * 2 * p.I * rowb, (uint32_t)(2 * p.I * rowb)),
                 make_rsrc(p.w13_sf + (int64_t)e * p.w13_sfsz, (uint32_t)p.w13_sfsz),
                 {live ? tile * 16 : 0, p.I + (live ? tile * 16 : 0)}, rowb, cpa4, lane);
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
            XBlock<kXBytes / 16 / kThreads> xb;
            auto load_block = [&](int k0) {
                xb.load(rx, [&](int i) { return (uint32_t)((list[m0 + i] >> 4) * p.H * 2); }, nr, S * cb, p.H, t, kThreads, [&](int lc) {
                    const int q = lc / cb, c = cps * q + k0 + lc - q * cb;
                    return k0 + lc - q * cb < cps && c < nch ? c : -1;
                });
            };
            load_block(0);
            XLane xl[XT];
#pragma unroll
            for (int i = 0; i < XT; i++) xl[i].set(xs, 16 * i + r < nr ? 16 * i + r : nr - 1, g);  // absent: any row
            f32x4 acc[2][XT];
#pragma unroll
            for (int f = 0; f < 2; f++)
#pragma unroll
                for (int i = 0; i < XT; i++) acc[f][i] = f32x4{0, 0, 0, 0};
            for (int k0 = 0; k0 < cps; k0 += cb) {
                if (k0) __syncthreads();  // the previous block is consumed
                xb.store(xs, nr, S * cb, t, kThreads);
                __syncthreads();
                if (k0 + cb < cps) load_block(k0 + cb);  // the next block is on its way while this one is used
                const int b0 = c0 + k0, b1 = b0 + cb < c1 ? b0 + cb : c1;
                if (live) consume<XT, WHOLE>(ring, acc, xl, part_of * cb * nr * 256, nr * 256, b0, b1, g, p.H, next);
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
                if (!live || 16 * i + r >= nr) continue;  // lane: its token, columns 4 g .. 4 g + 3 of the tile
                const int it = list[m0 + 16 * i + r], pair = (it >> 4) * p.k + (it & 15);
                const float wt = weight_of[pair] * a2;
                float v4[4];
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    const float gt = a13 * acc[0][i][v];
                    v4[v] = gt / (1.0f + expf(-gt)) * (a13 * acc[1][i][v]) * wt;
                }
                uint32_t h0, l0, h1, l1;
                split_bf16x2(v4[0], v4[1], h0, l0);
                split_bf16x2(v4[2], v4[3], h1, l1);
                const int64_t at = (int64_t)pair * p.I + tile * 16 + 4 * g;
                *(u32x2*)(p.act_hi + at) = u32x2{h0, h1};
                *(u32x2*)(p.act_lo + at) = u32x2{l0, l1};
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

// Workgroup (128 output columns, share of the K axis): wave w has columns 16 w ..
// + 15 to itself, and all walk the same (expert, chunk) range.
template <int D, bool WHOLE>
__global__ __launch_bounds__(kThreads, 4) void k_moe_down(EParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef W4Ring<1, D> Ring;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const rings = smem;                             // the waves' weight rings
    uint8_t* const xs = smem + kWaves * Ring::BYTES;         // activations of a block of chunks
    Routes& R = *(Routes*)(xs + kXBytes);
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
    // shares of at least 4 chunks; the rest of the workgroups has nothing to do
    const int shares = total < 4 * p.shares ? (total < 4 ? 1 : total / 4) : p.shares;
    const int share = blockIdx.y;
    if (share >= shares) return;
    const int tile = blockIdx.x * kWaves + wave, tiles = p.H / 16;
    const bool live = tile < tiles;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.act_hi, (uint32_t)(p.T * p.k * p.I * 4));  // both halves
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
                 make_rsrc(p.w2_sf + (int64_t)e * p.w2_sfsz, (uint32_t)p.w2_sfsz), {tile * 16}, rowb, cpa4, lane);
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
    XBlock<kXBytes / 16 / kThreads> xb;
    auto load_block = [&](Pass q, int b0) {  // rows: the tokens' high halves, then their low ones
        const int nt = tokens_of(q), cb = kXBytes / (nt * 512), end = end_of(q.at);
        const uint16_t* const list = R.list + act_first(act_of(q.at)) + q.m0;
        xb.load(
            rx,
            [&](int i) {
                const int lo = i >= nt, it = list[i - lo * nt];
                return (uint32_t)(((it >> 4) * p.k + (it & 15) + lo * p.T * p.k) * p.I * 2);
            },
            2 * nt, cb, p.I, t, kThreads, [&](int lc) { return b0 + lc < end ? b0 + lc : -1; });
    };
    Pass cur = {q0 / nch, 0};
    if (total > 0) {
        aim();
        for (int u = 0; u < D; u++) next();
        load_block(cur, begin_of(cur.at));
    }
    while (total > 0 && cur.at <= last) {
        const Pass nxt = after(cur);
        const int c0 = begin_of(cur.at), c1 = end_of(cur.at);
        const int nt = tokens_of(cur), nr = 2 * nt, cb = kXBytes / (nr * 256);
        // XT = 1: up to 8 tokens, lanes r < 8 with their activations' high halves and
        // the others with the low ones; XT = 2: up to 16, a tile of each
        auto pass = [&](auto xt) {
            constexpr int XT = decltype(xt)::value, NT = 8 * XT;
            XLane xl[XT];
            const int tl = (r & (NT - 1)) < nt ? r & (NT - 1) : nt - 1;  // absent: any row
            if constexpr (XT == 1) {
                xl[0].set(xs, (r >> 3) * nt + tl, g);
            } else {
                xl[0].set(xs, tl, g);
                xl[1].set(xs, nt + tl, g);
            }
            f32x4 acc[1][XT];
#pragma unroll
            for (int i = 0; i < XT; i++) acc[0][i] = f32x4{0, 0, 0, 0};
            for (int b0 = c0; b0 < c1; b0 += cb) {
                const int b1 = b0 + cb < c1 ? b0 + cb : c1;
                __syncthreads();  // the previous block is consumed
                xb.store(xs, nr, cb, t, kThreads);
                __syncthreads();
                // the next block is on its way while this one is used
                if (b1 < c1) load_block(cur, b1);
                else if (nxt.at <= last) load_block(nxt, begin_of(nxt.at));
                if (live) consume<XT, WHOLE>(ring, acc, xl, 0, nr * 256, b0, b1, g, p.I, next);
            }
            const int it = R.list[act_first(act_of(cur.at)) + cur.m0 + tl];
#pragma unroll
            for (int v = 0; v < 4; v++) {
                const float s = acc[0][0][v] + (XT == 1 ? row_half(acc[0][0][v]) : acc[0][XT - 1][v]);
                if (r < nt) sums[(it >> 4) * kSumPitch + wave * 16 + 4 * g + v] += s;
            }
        };
        if (nt <= 8) pass(std::integral_constant<int, 1>{});
        else pass(std::integral_constant<int, 2>{});
        cur = nxt;
    }
    // the wave's own columns (no other wave of the workgroup has touched them)
    if (!live) return;
    uint16_t* const O = p.out + tile * 16;
    const int col = lane & 15;
    if (shares == 1) {
        for (int tok = lane >> 4; tok < p.T; tok += 4)
            O[(int64_t)tok * p.H + col] = (uint16_t)pack_bf16x2(sums[tok * kSumPitch + wave * 16 + col], 0.0f);
        return;
    }
    // several workgroups have these columns: each leaves its sums in memory, and
    // the wave that finds the others done adds them, in the order of the shares.
    // Device-scope stores and loads (sc1) pass by the XCDs' own L2s, so no cache
    // is written back or dropped; the stores are waited for before the count.
    constexpr int kDevice = 16;
    const int n16 = p.T * 64;  // bytes of a share's sums of this tile
    const __amdgpu_buffer_rsrc_t part = make_rsrc(p.part + (int64_t)tile * p.shares * p.T * 16, (uint32_t)(shares * n16));
    for (int i = lane; i < p.T * 4; i += 64) {
        const f32x4 v = *(const f32x4*)&sums[(i >> 2) * kSumPitch + wave * 16 + (i & 3) * 4];
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), part, i * 16, share * n16, kDevice);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int before = 0;
    if (lane == 0) before = __hip_atomic_fetch_add(&p.arrived[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(before) != shares - 1) return;
    asm volatile("" ::: "memory");
    for (int i = lane; i < p.T * 4; i += 64) {
        f32x4 s = {0, 0, 0, 0};
        constexpr int U = 8;  // loads in flight together
        for (int v0 = 0; v0 < shares; v0 += U) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; u++)  // past the last share: past the resource, zeros
                v[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(part, i * 16 + (v0 + u) * n16, 0, kDevice));
#pragma unroll
            for (int u = 0; u < U; u++) s += __builtin_bit_cast(f32x4, v[u]);
        }
        *(u32x2*)(O + (int64_t)(i >> 2) * p.H + (i & 3) * 4) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    }
#endif
}

template <int NR>
void launch_up(const EParams& p, int grid, size_t lds, hipStream_t st) {
    if (p.H % kChunk == 0) k_moe_up<NR, true><<<grid, kThreads, lds, st>>>(p);
    else k_moe_up<NR, false><<<grid, kThreads, lds, st>>>(p);
}

template <int D>
void launch_down(const EParams& p, dim3 grid, size_t tables, hipStream_t st) {
    const size_t lds = kWaves * W4Ring<1, D>::BYTES + kXBytes + (size_t)p.T * kSumPitch * 4 + tables;
    if (p.I % kChunk == 0) k_moe_down<D, true><<<grid, kThreads, lds, st>>>(p);
    else k_moe_down<D, false><<<grid, kThreads, lds, st>>>(p);
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
    // workspace: the activations' two halves, the partial sums of the second
    // launch (kMoePartRows rows of h), the tiles' counters
    const int64_t acts = (int64_t)a.t * a.top_k * a.inter;
    p.act_hi = (uint16_t*)a.ws;
    p.act_lo = p.act_hi + acts;
    p.part = (float*)(p.act_lo + acts);
    p.routes = p.part + (int64_t)kMoePartRows * a.h;
    p.arrived = (int32_t*)((char*)p.routes + 4096);
    const int most = a.t * a.top_k < a.E ? a.t * a.top_k : a.E;  // experts that can be chosen
    const size_t tables = sizeof(Routes);
    // first launch: two workgroups a CU, or one per tile if there are fewer
    const int64_t items = (int64_t)most * (a.inter / 16);
    const int grid = (int)(items < 2 * cus ? items : 2 * cus);
    const size_t lds = kWaves * UpRing::BYTES + kXBytes + tables + (size_t)a.t * a.top_k * 6;
    if (a.E <= 16) launch_up<1>(p, grid, lds, st);
    else if (a.E <= 64) launch_up<4>(p, grid, lds, st);
    else if (a.E <= 128) launch_up<8>(p, grid, lds, st);
    else launch_up<16>(p, grid, lds, st);
    // second launch: two workgroups a CU as far as the partial sums have room
    const int cols = (a.h + 127) / 128;
    p.shares = 2 * cus / cols;
    if (p.shares > 32) p.shares = 32;
    if (p.shares > kMoePartRows / a.t) p.shares = kMoePartRows / a.t;
    if (p.shares < 1) p.shares = 1;
    // the ring's depth by what LDS has left beside the sums: two workgroups a CU up
    // to 32 tokens, one with a deeper ring beyond
    if (a.t <= 32) launch_down<4>(p, dim3((unsigned)cols, (unsigned)p.shares), tables, st);
    else launch_down<8>(p, dim3((unsigned)cols, (unsigned)p.shares), tables, st);
    return hipGetLastError();
}

}  // namespace nvfp4
