// adapters.hip -- low-rank adapters of many requests beside a shared NVFP4
// projection: the projection onto the ranks (any number of rows) and the
// weight-only decode products with the adapters' second half.
// (The prefill product is the block-scaled GEMM's adapter epilogue, gemm.hip.)
//
// What is computed, a = adapter[i] (none outside [0, L)):
//   d[i, :]   = scaling[a] * x[i] @ A[a]^T                      (k_adapter_down)
//   out[i, :] = alpha * x[i] @ dequant(W)^T + d[i] @ B[a]^T (+ bias)
//
// Rows may use any adapters in any order.  A wave finds the distinct adapters of
// its rows by ballots over their ids: the first row not yet served names one, all
// rows that share it are served together.  So an adapter is read once per tile of
// rows, whatever the order, and rows without one cost nothing.  The other rows of
// the tile are multiplied beside them (as zeros, an adapter's values may be
// infinite), and their products are left out by selection.  d stays in fp32 and
// enters the second product as two bf16 halves (2^-16 of d); the adapters' own
// bf16 values are exact.
//
// Bound: for decode the weight and the adapters that the batch uses, each read
// once; the projections are short, so their parts are spread over as many waves
// as there are and every load of a step is under way at once.
#include "device_common.h"
#include "gemm_common.h"
#include "internal.h"
#include "skinny_w4.h"

namespace nvfp4 {
namespace {

constexpr int kAdWaves = 8;  // K ranges of a workgroup (k_w4a16_adapters), waves of k_w4_wide

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
    // k_w4_wide: partial sums and counters of the workgroups that share a tile
    float* part;
    int32_t* arrived;
    int shares;
};

// Adapter of row m, or -1 (rows past M, ids outside [0, L)).
__device__ __forceinline__ int adapter_of(const AParams& p, int64_t m) {
    if (m >= p.M) return -1;
    const int a = p.adapter[m];
    return a >= 0 && a < p.L ? a : -1;
}

// Four columns n .. n + 3 of output row m: the bias, bf16.
__device__ __forceinline__ void store4(const AParams& p, int64_t m, int64_t n, f32x4 y) {
    uint16_t* const O = p.out + m * p.N;
#pragma unroll
    for (int v = 0; v < 4; v++)
        if (p.bias && n + v < p.N) y[v] += bf16_lo((uint32_t)p.bias[n + v]);
    if ((p.N & 3) == 0 && n + 3 < p.N) {
        *(u32x2*)(O + n) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    } else {
#pragma unroll
        for (int v = 0; v < 4; v++)
            if (n + v < p.N) O[n + v] = (uint16_t)pack_bf16x2(y[v], 0.0f);
    }
}

// Eight fp32 values as two bf16 fragments hi + lo (zeros where not `on`).
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, bool on, bf16x8& hi, bf16x8& lo) {
    uint32_t h[4], l[4];
    split_bf16x2(a[0], a[1], h[0], l[0]);
    split_bf16x2(a[2], a[3], h[1], l[1]);
    split_bf16x2(b[0], b[1], h[2], l[2]);
    split_bf16x2(b[2], b[3], h[3], l[3]);
    const u32x4 z = {0u, 0u, 0u, 0u};
    hi = __builtin_bit_cast(bf16x8, on ? u32x4{h[0], h[1], h[2], h[3]} : z);
    lo = __builtin_bit_cast(bf16x8, on ? u32x4{l[0], l[1], l[2], l[3]} : z);
}

// Workgroup (group of 16 RT ranks x, tile of 16 TT rows y, share z of the tile's
// distinct adapters): K split over NW waves, slices of 32 columns.  Many rows
// take TT = 2: an adapter's A is then read once per 32 rows.
template <int RT, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void k_adapter_down(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass only needs the launch stub
    __shared__ f32x4 part[NW][RT * TT][64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * TT);
    if (p.arrived && blockIdx.x + blockIdx.y + blockIdx.z == 0)  // for the product that follows
        for (int i = t; i < kAdCounters; i += 64 * NW) p.arrived[i] = 0;
    int id[TT];         // adapter of the lane's row of each 16
    uint32_t rem = 0;   // rows of the tile not yet served
#pragma unroll
    for (int i = 0; i < TT; i++) {
        id[i] = adapter_of(p, m0 + 16 * i + r);
        rem |= (uint32_t)(__ballot(id[i] >= 0) & 0xFFFF) << (16 * i);
    }
    const int p0 = blockIdx.x * 16 * RT;
    const int nsl = (int)((p.K + 31) / 32);
    const int s0 = nsl * wave / NW, s1 = nsl * (wave + 1) / NW;
    if (blockIdx.z == 0 && wave == 0) {  // rows without an adapter
#pragma unroll
        for (int i = 0; i < TT; i++)
            if (m0 + 16 * i + r < p.M && id[i] < 0)
                for (int c = p0 + g; c < p0 + 16 * RT && c < p.R; c += 4) p.d[(m0 + 16 * i + r) * p.R + c] = 0.0f;
    }
    for (int j = 0; rem; j++) {
        const int lead = __builtin_ctz(rem);
        int a = __builtin_amdgcn_readlane(id[0], lead & 15);
        if (TT == 2 && lead >= 16) a = __builtin_amdgcn_readlane(id[TT - 1], lead & 15);
#pragma unroll
        for (int i = 0; i < TT; i++) rem &= ~((uint32_t)(__ballot(id[i] == a) & 0xFFFF) << (16 * i));
        if (j % (int)gridDim.z != (int)blockIdx.z) continue;
        f32x4 acc[RT][TT];
        const uint16_t* A[RT];
        const uint16_t* X[TT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int c = p0 + 16 * i + r < p.R ? p0 + 16 * i + r : p.R - 1;  // past R: never stored
            A[i] = p.la + ((int64_t)a * p.R + c) * p.K + 8 * g;
#pragma unroll
            for (int q = 0; q < TT; q++) acc[i][q] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < TT; i++) X[i] = p.x + (id[i] == a ? m0 + 16 * i + r : 0) * p.K + 8 * g;
        constexpr int U = RT + TT <= 2 ? 8 : RT + TT <= 4 ? 5 : 3;  // slices whose loads are in flight together
        for (int sb = s0; sb < s1; sb += U) {
            u32x4 xv[U][TT], av[U][RT];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int s = sb + u < s1 ? sb + u : s1 - 1;  // past the range: reload, never used
                const bool in = 32 * s + 8 * g < p.K;
#pragma unroll
                for (int i = 0; i < TT; i++) {
                    xv[u][i] = u32x4{0, 0, 0, 0};
                    if (in && id[i] == a) xv[u][i] = *(const u32x4*)(X[i] + 32 * s);
                }
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
#pragma unroll
                    for (int q = 0; q < TT; q++)
                        acc[i][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, av[u][i]), __builtin_bit_cast(bf16x8, xv[u][q]), acc[i][q], 0, 0, 0);
            }
        }
        // the waves' partial sums, in wave order; lane: row r, ranks 4 g .. 4 g + 3
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int q = 0; q < TT; q++) part[wave][i * TT + q][lane] = acc[i][q];
        __syncthreads();
        if (wave < RT * TT) {
            f32x4 s = part[0][wave][lane];
#pragma unroll
            for (int v = 1; v < NW; v++) s += part[v][wave][lane];
            const int c = p0 + 16 * (wave / TT) + 4 * g, q = wave % TT;
            const bool mine = (TT == 2 && q ? id[TT - 1] : id[0]) == a;
            if (mine && c < p.R) *(f32x4*)(p.d + (m0 + 16 * q + r) * p.R + c) = s * (p.scaling ? p.scaling[a] : 1.0f);  // R % 8 == 0
        }
    }
#endif
}

// Weight-only product of up to 16 rows and 16 weight rows, the K chunks split over
// the waves, and so are the rows' distinct adapters, whose loads come first (the
// first weight loads are under way meanwhile).
template <bool WHOLE>
__global__ __launch_bounds__(64 * kAdWaves) void k_w4a16_adapters(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ f32x4 part[kAdWaves][64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t brow = n0 + r < p.N ? n0 + r : p.N - 1;
    const int rowb = (int)(p.K / 2);
    const uint8_t* const B = p.b + brow * rowb + g * 16;
    const uint8_t* const F = p.b_sf + scale_byte_off(brow, 2 * g, p.cpa4);
    const uint16_t* const X = r < p.M ? p.x + r * p.K + 32 * g : nullptr;
    const int id = adapter_of(p, r);
    const int nch = (int)((p.K + kChunk - 1) / kChunk);
    const int c0 = nch * wave / kAdWaves, c1 = nch * (wave + 1) / kAdWaves;
    constexpr int U = 4;  // chunks whose loads are in flight together
    u32x4 w[U], xv[U][4];
    uint32_t s[U];
    auto load_w = [&](int cb) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            int c = cb + u < c1 ? cb + u : c1 - 1;  // past the range: reload, never used
            c = c < 0 ? 0 : c;                      // a wave without chunks
            const int left = (int)p.K - c * kChunk - 32 * g;
            w[u] = u32x4{0, 0, 0, 0};
            s[u] = 0;
            if (WHOLE || left >= 32) w[u] = *(const u32x4*)(B + c * 64);
            else if (left >= 16) {
                const u32x2 h = *(const u32x2*)(B + c * 64);
                w[u] = u32x4{h.x, h.y, 0, 0};
            }
            if (WHOLE || left > 0) s[u] = *(const uint16_t*)(F + (int64_t)c * 1024) & (WHOLE || left >= 32 ? 0xFFFFu : 0xFFu);
        }
    };
    load_w(c0);
    f32x4 ad = {0, 0, 0, 0};
    uint32_t rem = (uint32_t)(__ballot(id >= 0) & 0xFFFF);
    for (int turn = 0; rem; turn++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(rem));
        rem &= ~(uint32_t)__ballot(id == a);
        if (turn % kAdWaves != wave) continue;
        const uint16_t* const LB = p.lb + ((int64_t)a * p.N + brow) * p.R + 8 * g;
        const float* const D = p.d + (id == a ? r : 0) * p.R + 8 * g;
        for (int k0 = 0; k0 < p.R; k0 += 32) {
            const bool in = k0 + 8 * g < p.R;
            const int k = in ? k0 : 0;
            const u32x4 bv = *(const u32x4*)(LB + k - (in ? 0 : 8 * g));
            const f32x4 d0 = *(const f32x4*)(D + k - (in ? 0 : 8 * g)), d1 = *(const f32x4*)(D + k - (in ? 0 : 8 * g) + 4);
            bf16x8 hi, lo;
            split8(d0, d1, in && id == a, hi, lo);
            const bf16x8 ol = __builtin_bit_cast(bf16x8, in ? bv : u32x4{0, 0, 0, 0});
            f32x4 z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ol, hi, f32x4{0, 0, 0, 0}, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ol, lo, z, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < 4; v++) ad[v] += id == a ? z[v] : 0.0f;
        }
    }
    f32x4 acc = {0, 0, 0, 0};
    for (int cb = c0; cb < c1; cb += U) {
        if (cb != c0) load_w(cb);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = cb + u < c1 ? cb + u : c1 - 1, left = (int)p.K - c * kChunk - 32 * g;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                xv[u][j] = u32x4{0, 0, 0, 0};
                if (X && (WHOLE || left > 8 * j)) xv[u][j] = *(const u32x4*)(X + c * kChunk + 8 * j);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (cb + u >= c1) break;
            const float f0 = __builtin_amdgcn_cvt_f32_fp8(s[u], 0), f1 = __builtin_amdgcn_cvt_f32_fp8(s[u], 1);
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dequant8_bf16(word(w[u], j), j < 2 ? f0 : f1),
                                                              __builtin_bit_cast(bf16x8, xv[u][j]), acc, 0, 0, 0);
        }
    }
    // the waves' partial sums, in wave order
    part[wave][lane] = acc * p.alpha[0] + ad;
    __syncthreads();
    if (wave != 0 || r >= p.M) return;
    f32x4 y = part[0][lane];
#pragma unroll
    for (int v = 1; v < kAdWaves; v++) y += part[v][lane];
    store4(p, r, n0 + 4 * g, y);
#endif
}

// Weight-only product of 16 XT rows and 256 columns, a share of the K axis and of
// the rows' distinct adapters: a wave has 32 columns to itself (two fragments, 128
// columns apart), the waves share x in LDS.  Of several workgroups of one tile
// each leaves its sums in memory and the last to finish adds them, wave by wave, in
// the order of the shares.
constexpr int kWideX = 32 << 10;  // LDS for x: 2 chunks of 64 rows; and 64 ranks of d
constexpr int kWideD = 68;        // floats of a row of d there (64 ranks, padded)
typedef W4Ring<2, 3> WideRing;

template <int XT, bool WHOLE>
__global__ __launch_bounds__(64 * kAdWaves, 2) void k_w4_wide(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __align__(16) uint8_t rings[kAdWaves * WideRing::BYTES];
    __shared__ __align__(16) uint8_t xs[kWideX];
    __shared__ float inv[kWideX / 256];
    static_assert(64 * kWideD * 4 <= kWideX, "64 ranks of 64 rows fit");
    constexpr int kThreads = 64 * kAdWaves;
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.z * (16 * XT);
    const int n0 = (int)blockIdx.x * 256, N = (int)p.N, K = (int)p.K;
    const int nr = (int)(p.M - m0 < 16 * XT ? p.M - m0 : 16 * XT);
    const int share = blockIdx.y, shares = p.shares;

    // this share's chunks, the first of them under way
    const int rowb = K / 2, nch = (K + kChunk - 1) / kChunk;
    const int c0 = nch * share / shares, c1 = nch * (share + 1) / shares;
    WideRing ring;
    ring.init(rings + wave * WideRing::BYTES, lane);
    const int nrows = N - n0 < 256 ? N - n0 : 256;
    ring.aim(make_rsrc(p.b + (int64_t)n0 * rowb, (uint32_t)(nrows * rowb)),
             make_rsrc(p.b_sf, (uint32_t)((p.N + 127) / 128 * p.cpa4 * 512)), {n0, n0 + 128}, {n0 + nrows, n0 + nrows}, wave, n0, rowb,
             p.cpa4, lane);
    int ca = c0;
    auto next = [&]() {
        if (ca < c1) ring.issue(ca++);
    };
    for (int u = 0; u < WideRing::DEPTH; u++) next();

    // 1. the adapters, 64 ranks of d in LDS at a time
    int col[2];  // the lane's row of B in each fragment (past N: the last one, never stored)
#pragma unroll
    for (int f = 0; f < 2; f++) {
        const int c = n0 + 128 * f + band_row(wave, r);
        col[f] = c < N ? c : N - 1;
    }
    const int id = lane < nr ? adapter_of(p, m0 + lane) : -1;  // lane: row of the tile
    f32x4 ad[2][XT];
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int i = 0; i < XT; i++) ad[f][i] = f32x4{0, 0, 0, 0};
    const uint64_t some = __ballot(id >= 0);
    for (int k0 = 0; some && k0 < p.R; k0 += 64) {
        float* const ds = (float*)xs;
        __syncthreads();
        for (int i = t; i < nr * 16; i += kThreads) {
            const int k = k0 + (i & 15) * 4;
            *(f32x4*)(ds + (i >> 4) * kWideD + (i & 15) * 4) =
                k < p.R ? *(const f32x4*)(p.d + (m0 + (i >> 4)) * p.R + k) : f32x4{0, 0, 0, 0};
        }
        __syncthreads();
        // this share's adapters in turn, the next one's B under way
        uint64_t rem = some;
        int turn = 0;
        auto find = [&]() {  // the next adapter of this share, or -1
            while (rem) {
                const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
                rem &= ~__ballot(id == a);
                if (turn++ % shares == share) return a;
            }
            return -1;
        };
        u32x4 bv[2][2][2];  // [buffer][fragment][32 ranks]
        auto load_b = [&](int buf, int a) {
#pragma unroll
            for (int f = 0; f < 2; f++)
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    const int k = k0 + 32 * s + 8 * g;
                    bv[buf][f][s] = *(const u32x4*)(p.lb + ((int64_t)a * p.N + col[f]) * p.R + (k < p.R ? k : 0));
                }
        };
        auto use = [&](int buf, int a) {
            const uint64_t mine = __ballot(id == a);
#pragma unroll
            for (int i = 0; i < XT; i++) {
                const uint32_t m16 = (uint32_t)(mine >> (16 * i)) & 0xFFFF;
                if (!m16) continue;
                const bool on = m16 >> r & 1;
                f32x4 z[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    const bool in = k0 + 32 * s + 8 * g < p.R;
                    const float* const d = ds + (16 * i + r) * kWideD + 32 * s + 8 * g;
                    bf16x8 hi, lo;
                    split8(*(const f32x4*)d, *(const f32x4*)(d + 4), on && in, hi, lo);
#pragma unroll
                    for (int f = 0; f < 2; f++) {
                        const bf16x8 ol = __builtin_bit_cast(bf16x8, in ? bv[buf][f][s] : u32x4{0u, 0u, 0u, 0u});
                        z[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ol, hi, z[f], 0, 0, 0);
                        z[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ol, lo, z[f], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int f = 0; f < 2; f++)
#pragma unroll
                    for (int v = 0; v < 4; v++) ad[f][i][v] += on ? z[f][v] : 0.0f;
            }
        };
        int a0 = find();
        if (a0 >= 0) load_b(0, a0);
        while (a0 >= 0) {
            const int a1 = find();
            if (a1 >= 0) load_b(1, a1);
            use(0, a0);
            if (a1 < 0) break;
            a0 = find();
            if (a0 >= 0) load_b(0, a0);
            use(1, a1);
        }
    }

    // 2. the shared projection
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + m0 * p.K, (uint32_t)(nr * K * 2));
    const int cb = kWideX / (nr * 256);  // chunks of a block
    XBlock<kWideX / 16 / kThreads, false> xb;
    xb.prepare(nr, nr, cb, t, kThreads, [&](int R) { return (uint32_t)(R * K * 2); }, [&](int lc) { return c0 + lc; },
               [&](int) { return c1; });
    xb.load(rx, 0, K, t);
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
    for (int b0 = c0; b0 < c1; b0 += cb) {
        __syncthreads();  // the previous block, or d, is consumed
        xb.store(xs, inv, 0, b0 - c0, t);
        __syncthreads();
        if (b0 + cb < c1) xb.load(rx, b0 + cb - c0, K, t);  // the next block is on its way while this one is used
        consume<XT, WHOLE>(ring, acc, xl, 0, nr, b0, b0 + cb < c1 ? b0 + cb : c1, g, K, next);
    }

    // 3. lane: row 16 i + r, columns n0 + 128 f + band_row(wave, 4 g) .. + 3
    const float alpha = p.alpha[0];
    auto put = [&](int f, int i, f32x4 y) {
        const int n = n0 + 128 * f + band_row(wave, 4 * g);
        if (16 * i + r < nr && n < N) store4(p, m0 + 16 * i + r, n, y);
    };
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int i = 0; i < XT; i++) {
            acc[f][i] = acc[f][i] * alpha + ad[f][i];
            if (shares == 1) put(f, i, acc[f][i]);
        }
    if (shares == 1) return;
    // device-scope stores and loads (sc1) pass by the XCDs' own L2s; the stores are
    // waited for before the count
    constexpr int kDevice = 16, kWave = 2 * XT * 1024;  // bytes of a wave's sums
    const int64_t place = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * kAdWaves + wave;
    const __amdgpu_buffer_rsrc_t part = make_rsrc((uint8_t*)p.part + place * shares * kWave, (uint32_t)(shares * kWave));
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int i = 0; i < XT; i++)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[f][i]), part,
                                                   share * kWave + (f * XT + i) * 1024 + lane * 16, 0, kDevice);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int before = 0;
    if (lane == 0) before = __hip_atomic_fetch_add(&p.arrived[place], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(before) != shares - 1) return;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int i = 0; i < XT; i++) {
            f32x4 y = {0, 0, 0, 0};
            constexpr int U = 16;  // loads in flight together
            for (int v0 = 0; v0 < shares; v0 += U) {
                u32x4 v[U];
#pragma unroll
                for (int u = 0; u < U; u++)  // past the last share: past the resource, zeros
                    v[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                         part, (v0 + u) * kWave + (f * XT + i) * 1024 + lane * 16, 0, kDevice));
#pragma unroll
                for (int u = 0; u < U; u++) y += __builtin_bit_cast(f32x4, v[u]);
            }
            put(f, i, y);
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
    AParams p = params(a);
    p.arrived = a.counters;
    const unsigned ranks = (unsigned)((a.r + 15) / 16);
    if (a.m <= 64) {
        // few rows: a workgroup per 16 ranks and distinct adapter, since the
        // adapters' reads are the work
        k_adapter_down<1, 1, 16><<<dim3(ranks, (unsigned)((a.m + 15) / 16), a.m < 16 ? (unsigned)a.m : 16u), 1024, 0, st>>>(p);
        return hipGetLastError();
    }
    // many rows: up to four tiles of ranks on one read of x, an adapter's A once per
    // 32 rows, and two workgroups share a row tile's adapters (a prompt's end falls
    // inside a tile)
    const unsigned rows = (unsigned)((a.m + 31) / 32);
    if (ranks == 1) k_adapter_down<1, 2, 16><<<dim3(1, rows, 2), 1024, 0, st>>>(p);
    else if (ranks == 2) k_adapter_down<2, 2, 16><<<dim3(1, rows, 2), 1024, 0, st>>>(p);
    else k_adapter_down<4, 2, 8><<<dim3((ranks + 3) / 4, rows, 2), 512, 0, st>>>(p);
    return hipGetLastError();
}

template <int XT>
static void launch_wide(AParams p, int cus, bool split, hipStream_t st) {
    const int cols = (int)((p.N + 255) / 256), rows = (int)((p.M + 16 * XT - 1) / (16 * XT)), nch = (int)((p.K + kChunk - 1) / kChunk);
    // one workgroup a CU; a share has 2 chunks at least
    p.shares = split && cols * rows * kAdWaves <= kAdCounters ? cus / (cols * rows) : 1;
    if (p.shares > nch / 2) p.shares = nch / 2;
    if (p.shares < 1) p.shares = 1;
    const dim3 grid((unsigned)cols, (unsigned)p.shares, (unsigned)rows);
    if (p.K % kChunk == 0) k_w4_wide<XT, true><<<grid, 64 * kAdWaves, 0, st>>>(p);
    else k_w4_wide<XT, false><<<grid, 64 * kAdWaves, 0, st>>>(p);
}

hipError_t launch_w4a16_adapters(const AdapterArgs& a, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                                 const uint16_t* bias, uint16_t* out, float* part, hipStream_t st) {
    AParams p = params(a);
    p.b = b; p.b_sf = b_sf; p.alpha = alpha; p.bias = bias; p.out = out;
    p.part = part; p.arrived = a.counters;
    const int cus = device_cus();
    if (cus <= 0) return hipErrorInvalidDevice;
    if (a.m <= 16) {
        const dim3 grid((unsigned)((p.N + 15) / 16));
        if (p.K % kChunk == 0) k_w4a16_adapters<true><<<grid, 64 * kAdWaves, 0, st>>>(p);
        else k_w4a16_adapters<false><<<grid, 64 * kAdWaves, 0, st>>>(p);
    } else if (a.m <= 32) {
        launch_wide<2>(p, cus, part != nullptr, st);
    } else {
        launch_wide<4>(p, cus, part != nullptr, st);
    }
    return hipGetLastError();
}

}  // namespace nvfp4
