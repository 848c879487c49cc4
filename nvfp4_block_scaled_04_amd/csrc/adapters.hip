// adapters.hip -- low-rank adapters of many requests beside a shared NVFP4
// projection: the projection onto the ranks (any number of rows) and the
// weight-only decode product with the adapters' second half in its epilogue.
// (The prefill product is the block-scaled GEMM's adapter epilogue, gemm.hip.)
//
// What is computed, a = adapter[i] (none outside [0, L)):
//   d[i, :]   = scaling[a] * x[i] @ A[a]^T                      (k_adapter_down)
//   out[i, :] = alpha * x[i] @ dequant(W)^T + d[i] @ B[a]^T (+ bias)
//
// Rows may use any adapters in any order.  A wave finds the distinct adapters of
// its 16 rows by ballots over their ids: the first row not yet served names one,
// all rows that share it are served together, the other rows enter the product
// as zeros.  So an adapter is read once per 16 rows, whatever the order, and
// rows without one cost nothing.  d stays in fp32 and enters the second product
// as two bf16 halves (2^-16 of d), the adapters' own bf16 values are exact.
#include "device_common.h"
#include "gemm_common.h"
#include "internal.h"
#include "skinny_w4.h"

namespace nvfp4 {
namespace {

constexpr int kAdWaves = 8;  // K ranges of a workgroup

struct AParams {
    const uint16_t* x;         // [M, K]
    const uint8_t* b;          // [N, K/2]
    const uint8_t* b_sf;
    const float* alpha;        // [1]
    const uint16_t* la;        // [L, R, K]
    const uint16_t* lb;        // [L, N, R]
    const int32_t* adapter;    // [M]
    const float* scaling;      // [L] or null
    const uint16_t* bias;      // [N] or null
    uint16_t* out;             // [M, N]
    float* d;                  // [M, R]
    int64_t M, N, K;
    int R, L;
    int cpa4, nblk;
};

// Adapter of row m, or -1 (rows past M, ids outside [0, L)).
__device__ __forceinline__ int adapter_of(const AParams& p, int64_t m) {
    if (m >= p.M) return -1;
    const int a = p.adapter[m];
    return a >= 0 && a < p.L ? a : -1;
}

// Workgroup (rank group x, 16-row tile y, share z of the tile's distinct
// adapters): RT tiles of 16 ranks, K split over the waves.
template <int RT>
__global__ __launch_bounds__(64 * kAdWaves) void k_adapter_down(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass only needs the launch stub
    __shared__ f32x4 part[kAdWaves][RT][64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t m = (int64_t)blockIdx.y * 16 + r;
    const int id = adapter_of(p, m);
    const int p0 = blockIdx.x * 16 * RT;
    const int nsl = (int)((p.K + 31) / 32);  // slices of 32 columns
    const int s0 = (int)((int64_t)nsl * wave / kAdWaves), s1 = (int)((int64_t)nsl * (wave + 1) / kAdWaves);
    uint32_t rem = (uint32_t)(__ballot(id >= 0) & 0xFFFF);
    if (blockIdx.z == 0 && wave == 0 && m < p.M && id < 0) {  // rows without an adapter
        for (int c = p0 + g; c < p0 + 16 * RT && c < p.R; c += 4) p.d[m * p.R + c] = 0.0f;
    }
    for (int j = 0; rem; j++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(rem));
        const bool mine = id == a;
        rem &= ~(uint32_t)__ballot(mine);
        if (j % (int)gridDim.z != (int)blockIdx.z) continue;
        f32x4 acc[RT];
        const uint16_t* A[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            acc[i] = f32x4{0, 0, 0, 0};
            const int c = p0 + 16 * i + r < p.R ? p0 + 16 * i + r : p.R - 1;  // past R: never stored
            A[i] = p.la + ((int64_t)a * p.R + c) * p.K + 8 * g;
        }
        const uint16_t* const X = p.x + (mine ? m : 0) * p.K + 8 * g;
        constexpr int U = 4;  // slices whose loads are in flight together
        for (int sb = s0; sb < s1; sb += U) {
            u32x4 xv[U], av[U][RT];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int s = sb + u < s1 ? sb + u : s1 - 1;  // past the range: reload, never used
                const bool in = 32 * s + 8 * g < p.K;
                xv[u] = u32x4{0, 0, 0, 0};
                if (in && mine) xv[u] = *(const u32x4*)(X + 32 * s);
#pragma unroll
                for (int i = 0; i < RT; i++) {
                    av[u][i] = u32x4{0, 0, 0, 0};
                    if (in) av[u][i] = *(const u32x4*)(A[i] + 32 * s);
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (sb + u >= s1) break;
#pragma unroll
                for (int i = 0; i < RT; i++)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av[u][i]),
                                                                     __builtin_bit_cast(bf16x8, xv[u]), acc[i], 0, 0, 0);
            }
        }
        // the waves' partial sums, in wave order; lane: row r, ranks 4 g .. 4 g + 3
#pragma unroll
        for (int i = 0; i < RT; i++) part[wave][i][lane] = acc[i];
        __syncthreads();
        if (wave < RT) {
            f32x4 s = part[0][wave][lane];
#pragma unroll
            for (int v = 1; v < kAdWaves; v++) s += part[v][wave][lane];
            const int c = p0 + 16 * wave + 4 * g;
            if (mine && c < p.R) *(f32x4*)(p.d + m * p.R + c) = s * (p.scaling ? p.scaling[a] : 1.0f);  // R % 8 == 0
        }
        __syncthreads();
    }
#endif
}

// Weight-only product of 16 TT rows and 16 weight rows, the K chunks split over
// the waves; the tiles' distinct adapters are dealt to the waves too.
template <int TT, bool WHOLE>
__global__ __launch_bounds__(64 * kAdWaves) void k_w4a16_adapters(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ f32x4 part[kAdWaves][TT][64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * TT);
    const int64_t brow = n0 + r < p.N ? n0 + r : p.N - 1;
    const int rowb = (int)(p.K / 2);
    const uint8_t* const B = p.b + brow * rowb;
    const uint8_t* const F = p.b_sf + scale_byte_off(brow, 2 * g, p.cpa4);
    const uint16_t* X[TT];
    int id[TT];
#pragma unroll
    for (int i = 0; i < TT; i++) {
        const int64_t m = m0 + 16 * i + r;
        X[i] = m < p.M ? p.x + m * p.K + 32 * g : nullptr;
        id[i] = adapter_of(p, m);
    }
    const int nch = (int)((p.K + kChunk - 1) / kChunk);
    const int c0 = nch * wave / kAdWaves, c1 = nch * (wave + 1) / kAdWaves;
    f32x4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; i++) acc[i] = f32x4{0, 0, 0, 0};
    constexpr int U = TT == 1 ? 4 : 2;  // chunks whose loads are in flight together
    for (int cb = c0; cb < c1; cb += U) {
        u32x4 w[U], xv[U][TT][4];
        uint32_t s[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = cb + u < c1 ? cb + u : c1 - 1;  // past the range: reload, never used
            const int left = (int)p.K - c * kChunk - 32 * g;
            w[u] = u32x4{0, 0, 0, 0};
            s[u] = 0;
            if (WHOLE || left >= 32) w[u] = *(const u32x4*)(B + c * 64 + g * 16);
            else if (left >= 16) {
                const u32x2 h = *(const u32x2*)(B + c * 64 + g * 16);
                w[u] = u32x4{h.x, h.y, 0, 0};
            }
            if (WHOLE || left > 0) s[u] = *(const uint16_t*)(F + (int64_t)c * 1024) & (WHOLE || left >= 32 ? 0xFFFFu : 0xFFu);
#pragma unroll
            for (int i = 0; i < TT; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    xv[u][i][j] = u32x4{0, 0, 0, 0};
                    if (X[i] && (WHOLE || left > 8 * j)) xv[u][i][j] = *(const u32x4*)(X[i] + c * kChunk + 8 * j);
                }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (cb + u >= c1) break;
            const float f0 = __builtin_amdgcn_cvt_f32_fp8(s[u], 0), f1 = __builtin_amdgcn_cvt_f32_fp8(s[u], 1);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bf16x8 wv = dequant8_bf16(word(w[u], j), j < 2 ? f0 : f1);
#pragma unroll
                for (int i = 0; i < TT; i++)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, xv[u][i][j]), acc[i], 0, 0, 0);
            }
        }
    }
    const float alpha = p.alpha[0];
    int turn = 0;  // distinct adapters seen, over all row tiles
#pragma unroll
    for (int i = 0; i < TT; i++) {
        acc[i] *= alpha;
        uint32_t rem = (uint32_t)(__ballot(id[i] >= 0) & 0xFFFF);
        for (; rem; turn++) {
            const int a = __builtin_amdgcn_readlane(id[i], __builtin_ctz(rem));
            const bool mine = id[i] == a;
            rem &= ~(uint32_t)__ballot(mine);
            if (turn % kAdWaves != wave) continue;
            const uint16_t* const LB = p.lb + ((int64_t)a * p.N + brow) * p.R + 8 * g;
            const float* const D = p.d + (mine ? m0 + 16 * i + r : 0) * p.R + 8 * g;
            for (int k0 = 0; k0 < p.R; k0 += 32) {
                u32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0}, lv = {0, 0, 0, 0};
                if (k0 + 8 * g < p.R) {
                    lv = *(const u32x4*)(LB + k0);
                    if (mine) {
                        const f32x4 d0 = *(const f32x4*)(D + k0), d1 = *(const f32x4*)(D + k0 + 4);
                        uint32_t h[4], l[4];
                        split_bf16x2(d0[0], d0[1], h[0], l[0]);
                        split_bf16x2(d0[2], d0[3], h[1], l[1]);
                        split_bf16x2(d1[0], d1[1], h[2], l[2]);
                        split_bf16x2(d1[2], d1[3], h[3], l[3]);
                        hi = u32x4{h[0], h[1], h[2], h[3]};
                        lo = u32x4{l[0], l[1], l[2], l[3]};
                    }
                }
                const bf16x8 bv = __builtin_bit_cast(bf16x8, lv);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, __builtin_bit_cast(bf16x8, hi), acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, __builtin_bit_cast(bf16x8, lo), acc[i], 0, 0, 0);
            }
        }
    }
    // the waves' partial sums, in wave order; wave i takes row tile i
#pragma unroll
    for (int i = 0; i < TT; i++) part[wave][i][lane] = acc[i];
    __syncthreads();
    const int64_t m = m0 + 16 * wave + r;
    if (wave >= TT || m >= p.M) return;
    f32x4 s = part[0][wave][lane];
#pragma unroll
    for (int v = 1; v < kAdWaves; v++) s += part[v][wave][lane];
    uint16_t* const O = p.out + m * p.N;
    const int64_t n = n0 + 4 * g;
    float y[4];
#pragma unroll
    for (int v = 0; v < 4; v++) {
        y[v] = s[v];
        if (p.bias && n + v < p.N) y[v] += bf16_lo((uint32_t)p.bias[n + v]);
    }
    if ((p.N & 3) == 0 && n + 3 < p.N) {
        *(u32x2*)(O + n) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    } else {
#pragma unroll
        for (int v = 0; v < 4; v++)
            if (n + v < p.N) O[n + v] = (uint16_t)pack_bf16x2(y[v], 0.0f);
    }
#endif
}

AParams params(const AdapterArgs& a) {
    AParams p{};
    p.x = a.x; p.la = a.lora_a; p.lb = a.lora_b; p.adapter = a.adapter; p.scaling = a.scaling; p.d = a.d;
    p.M = a.m; p.N = a.n; p.K = a.k; p.R = (int)a.r; p.L = (int)a.n_adapters;
    p.nblk = (int)(a.k / 16);
    p.cpa4 = (p.nblk + 3) / 4;
    return p;
}

}  // namespace

hipError_t launch_adapter_down(const AdapterArgs& a, hipStream_t st) {
    const AParams p = params(a);
    const unsigned rows = (unsigned)((a.m + 15) / 16);
    const unsigned ranks = (unsigned)((a.r + 15) / 16);
    // few rows: a workgroup per rank tile and distinct adapter, since the
    // adapters' reads are the work; many rows: up to four rank tiles on one
    // read of x, and two workgroups share a row tile's adapters
    if (a.m <= 64) k_adapter_down<1><<<dim3(ranks, rows, a.m < 16 ? (unsigned)a.m : 16u), 64 * kAdWaves, 0, st>>>(p);
    else if (ranks == 1) k_adapter_down<1><<<dim3(1, rows, 2), 64 * kAdWaves, 0, st>>>(p);
    else if (ranks == 2) k_adapter_down<2><<<dim3(1, rows, 2), 64 * kAdWaves, 0, st>>>(p);
    else k_adapter_down<4><<<dim3((ranks + 3) / 4, rows, 2), 64 * kAdWaves, 0, st>>>(p);
    return hipGetLastError();
}

template <int TT>
static void launch_w4(const AParams& p, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 16 * TT - 1) / (16 * TT)));
    if (p.K % kChunk == 0) k_w4a16_adapters<TT, true><<<grid, 64 * kAdWaves, 0, st>>>(p);
    else k_w4a16_adapters<TT, false><<<grid, 64 * kAdWaves, 0, st>>>(p);
}

hipError_t launch_w4a16_adapters(const AdapterArgs& a, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                                 const uint16_t* bias, uint16_t* out, hipStream_t st) {
    AParams p = params(a);
    p.b = b; p.b_sf = b_sf; p.alpha = alpha; p.bias = bias; p.out = out;
    if (a.m <= 16) launch_w4<1>(p, st);
    else if (a.m <= 32) launch_w4<2>(p, st);
    else launch_w4<4>(p, st);
    return hipGetLastError();
}

}  // namespace nvfp4
