// adapters.hip -- low-rank adapters of many requests beside a shared NVFP4
// projection: the projection onto the ranks (any number of rows) and the
// weight-only decode products with the adapters' second half.
// (The prefill product is the block-scaled GEMM's adapter epilogue, gemm.hip.)
//
// What is computed, a = adapter[i] (none outside [0, L)):
//   d[i, :]   = scaling[a] * x[i] @ A[a]^T                     (k_adapter_down)
//   out[i, :] = alpha * x[i] @ dequant(W)^T + d[i] @ B[a]^T (+ bias)
//
// Rows may use any adapters in any order.  A wave finds the distinct adapters of
// its rows by ballots over their ids: the first row not yet served names one, all
// rows that share it are served together.  So an adapter is read once per tile of
// rows, whatever the order, and rows without one cost nothing.  The other rows of
// the tile are multiplied beside them and their products left out by selection (an
// adapter's values may be infinite).  d is a sum and kept in fp32; it enters
// the second product as three bf16 parts that add up to it (split_bf16x3), beside the
// adapters' own bf16 values.
//
// Bound: for decode the weight and the adapters that the batch uses; the projections
// are short, so their parts are spread over as many waves as there are and every load
// of a step is under way at once.  The projection runs before the product, though only
// the product's last step needs d: its time (6.5 to 17 us for up to 64 rows) is added.
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
    // k_w4_wide: partial sums of the workgroups that share a tile
    float* part;
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

// Eight bf16 values, or zeros.
__device__ __forceinline__ bf16x8 b8(const uint16_t* b, bool on) {
    const u32x4 v = *(const u32x4*)b;
    return __builtin_bit_cast(bf16x8, on ? v : u32x4{0u, 0u, 0u, 0u});
}

// Eight values of d in their three parts, or zeros.
__device__ __forceinline__ void d8(const float* d, bool on, bf16x8 (&part)[3]) {
    const f32x4 zero = {0, 0, 0, 0}, lo = *(const f32x4*)d, hi = *(const f32x4*)(d + 4);
    split_bf16x3(on ? lo : zero, on ? hi : zero, part);
}

// A wave's ring of slices in LDS: NT tiles of 16 bf16 rows, 32 columns (64 bytes)
// a slice, D slices.  A load instruction takes 64 contiguous bytes of a row in four
// neighbouring lanes; taken straight into the matrix instruction's lanes (one row
// each) the same bytes come from L2 at a third of the rate (35 against 106 KB/us
// and CU).
template <int NT, int D>
struct RowRing {
    static_assert(NT <= 6, "operands of take");
    static constexpr int SLOT = NT * 1024, BYTES = D * SLOT;
    __amdgpu_buffer_rsrc_t src[NT];
    uint32_t vo[NT];  // the lane's source offset
    uint32_t rd;      // the lane's LDS address in slot 0
    uint8_t* base;
    int head, tail, ahead;

    __device__ __forceinline__ void init(uint8_t* ring, int lane) {
        base = ring;
        rd = lds_addr(ring) + (lane & 15) * 64 + (((lane >> 4) ^ swz(lane & 15)) << 4);
        head = tail = ahead = 0;
    }
    // rows of tile i: `rows` rows of K columns at `p` (past them: the last one); a
    // lane that is not `on` gets zeros and reads nothing, by an offset past the
    // source's end (16 rows of 2^24 bytes at most, and no sum with a slice's
    // offset wraps)
    __device__ __forceinline__ void aim(int i, const uint16_t* p, int rows, int64_t K, int lane, bool on = true) {
        const int lr = lane >> 2, row = lr < rows ? lr : rows - 1;
        src[i] = make_rsrc(p, (uint32_t)(rows * K * 2));
        vo[i] = on ? (uint32_t)(row * K * 2) + (((lane & 3) ^ swz(lr)) << 4) : 0x80000000u;
    }
    __device__ __forceinline__ void issue(int s) {
        lds_byte* const dst = (lds_byte*)base + head * SLOT;
#pragma unroll
        for (int i = 0; i < NT; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(src[i], (__attribute__((address_space(3))) void*)(dst + i * 1024), 16, vo[i], s * 64, 0, 0);
        head = head + 1 == D ? 0 : head + 1;
        ahead++;
    }
    __device__ __forceinline__ void take(bf16x8 (&v)[NT]) {
        if (ahead == D) wait_vmcnt<(D - 1) * NT>();
        else wait_vmcnt<0>();
        const uint32_t a = rd + tail * SLOT;
        if constexpr (NT == 2)
            asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:1024\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1]) : "v"(a) : "memory");
        else if constexpr (NT == 3)
            asm volatile("ds_read_b128 %0, %3\n\tds_read_b128 %1, %3 offset:1024\n\tds_read_b128 %2, %3 offset:2048\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]) : "v"(a) : "memory");
        else if constexpr (NT == 4)
            asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:1024\n\tds_read_b128 %2, %4 offset:2048\n\t"
                         "ds_read_b128 %3, %4 offset:3072\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]) : "v"(a) : "memory");
        else {
            static_assert(NT == 6, "operands");
            asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %1, %6 offset:1024\n\tds_read_b128 %2, %6 offset:2048\n\t"
                         "ds_read_b128 %3, %6 offset:3072\n\tds_read_b128 %4, %6 offset:4096\n\tds_read_b128 %5, %6 offset:5120\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]) : "v"(a) : "memory");
        }
        tail = tail + 1 == D ? 0 : tail + 1;
        ahead--;
    }
};

// Workgroup (group of 16 RT ranks x, tile of 16 TT rows y, share z of the tile's
// distinct adapters): K split over NW waves, slices of 32 columns.
// Bound: few rows, the latency of a first read and the adapters' bytes (64 rows, 48
// adapters of 64 x 8192: 50 MB in 15-17 us, 3 TB/s; one row 6.6 us); many rows, the
// reads of x and A through L2 (8192 x 5120, rank 32: 84 MB of x in 38 to 50 us, 2 TB/s;
// 128 rows of 4096 with 8 adapters of rank 16 in any order: 20 us, the two workgroups of
// a row tile serve four adapters each in turn).
template <int RT, int TT, int NW, int D>
__global__ __launch_bounds__(64 * NW) void k_adapter_down(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass only needs the launch stub
    constexpr int NT = RT + TT;
    typedef RowRing<NT, D> Ring;
    static_assert(Ring::BYTES >= RT * TT * 1024, "the partial sums take the rings' place");
    __shared__ __align__(16) uint8_t rings[NW * Ring::BYTES];
    f32x4* const part = (f32x4*)rings;  // [NW][RT * TT][64]
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * TT);
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
                for (int c = p0 + 4 * g; c < p0 + 16 * RT && c < p.R; c += 16)
                    *(f32x4*)(p.d + (m0 + 16 * i + r) * p.R + c) = f32x4{0, 0, 0, 0};
    }
    Ring ring;
    ring.init(rings + wave * Ring::BYTES, lane);
    for (int j = 0; rem; j++) {
        const int lead = __builtin_ctz(rem);
        int a = __builtin_amdgcn_readlane(id[0], lead & 15);
        if (TT == 2 && lead >= 16) a = __builtin_amdgcn_readlane(id[TT - 1], lead & 15);
#pragma unroll
        for (int i = 0; i < TT; i++) rem &= ~((uint32_t)(__ballot(id[i] == a) & 0xFFFF) << (16 * i));
        if (j % (int)gridDim.z != (int)blockIdx.z) continue;
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int c = p0 + 16 * i < p.R ? p0 + 16 * i : p.R - 1;  // past R: never stored
            ring.aim(i, p.la + ((int64_t)a * p.R + c) * p.K, p.R - c < 16 ? p.R - c : 16, p.K, lane);
        }
#pragma unroll
        for (int i = 0; i < TT; i++) {
            const int64_t first = m0 + 16 * i < p.M ? m0 + 16 * i : p.M - 1;
            // other adapters' rows, and those past M, are zeros
            ring.aim(RT + i, p.x + first * p.K, (int)(p.M - first < 16 ? p.M - first : 16), p.K, lane, __shfl(id[i], lane >> 2) == a);
        }
        f32x4 acc[RT][TT];
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int q = 0; q < TT; q++) acc[i][q] = f32x4{0, 0, 0, 0};
        __syncthreads();  // the previous adapter's sums are read
#pragma unroll
        for (int u = 0; u < D; u++)
            if (s0 + u < s1) ring.issue(s0 + u);
        for (int s = s0; s < s1; s++) {
            bf16x8 v[NT];
            ring.take(v);
            if (s + D < s1) ring.issue(s + D);
            if (32 * s + 8 * g >= p.K) {  // past K (K % 32 == 16): the next row's, or nothing
#pragma unroll
                for (int i = 0; i < NT; i++) v[i] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
            }
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int q = 0; q < TT; q++) acc[i][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[i], v[RT + q], acc[i][q], 0, 0, 0);
        }
        // the waves' partial sums, in wave order; lane: row r, ranks 4 g .. 4 g + 3
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int q = 0; q < TT; q++) part[(wave * RT * TT + i * TT + q) * 64 + lane] = acc[i][q];
        __syncthreads();
        if (wave < RT * TT) {
            f32x4 s = part[wave * 64 + lane];
#pragma unroll
            for (int v = 1; v < NW; v++) s += part[(v * RT * TT + wave) * 64 + lane];
            const int c = p0 + 16 * (wave / TT) + 4 * g, q = wave % TT;
            const bool mine = (TT == 2 && q ? id[TT - 1] : id[0]) == a;
            if (mine && c < p.R) {  // R % 8 == 0
                s *= p.scaling ? p.scaling[a] : 1.0f;
                *(f32x4*)(p.d + (m0 + 16 * q + r) * p.R + c) = s;
            }
        }
    }
#endif
}

// Weight-only product of up to 16 TT rows and 16 weight rows, the K chunks split
// over the waves, and so are the rows' distinct adapters, whose loads come first
// (the first weight loads are under way meanwhile).  Bound: the latency of one step
// of loads (4096 x 4096, 9.4 MB: one row 7 us, 16 rows with 16 adapters 10 us; 23 rows
// of 1000 x 2608 9 us), and for more rows every workgroup's own reads of x.
template <int TT, bool WHOLE>
__global__ __launch_bounds__(64 * kAdWaves) void k_w4a16_adapters(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ f32x4 part[kAdWaves][TT][64];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t brow = n0 + r < p.N ? n0 + r : p.N - 1;
    const int rowb = (int)(p.K / 2);
    const uint8_t* const B = p.b + brow * rowb + g * 16;
    const uint8_t* const F = p.b_sf + scale_byte_off(brow, 2 * g, p.cpa4);
    const uint16_t* X[TT];
    int id[TT];
#pragma unroll
    for (int i = 0; i < TT; i++) {
        X[i] = 16 * i + r < p.M ? p.x + (16 * i + r) * p.K + 32 * g : nullptr;
        id[i] = adapter_of(p, 16 * i + r);
    }
    const int nch = (int)((p.K + kChunk - 1) / kChunk);
    const int c0 = nch * wave / kAdWaves, c1 = nch * (wave + 1) / kAdWaves;
    constexpr int U = TT == 1 ? 4 : 2;  // chunks whose loads are in flight together
    u32x4 w[U], xv[U][TT][4];
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
    f32x4 ad[TT];
    int turn = 0;  // distinct adapters seen, over all 16-row tiles
#pragma unroll
    for (int i = 0; i < TT; i++) {
        ad[i] = f32x4{0, 0, 0, 0};
        uint32_t rem = (uint32_t)(__ballot(id[i] >= 0) & 0xFFFF);
        for (; rem; turn++) {
            const int a = __builtin_amdgcn_readlane(id[i], __builtin_ctz(rem));
            const bool mine = id[i] == a;
            rem &= ~(uint32_t)__ballot(mine);
            if (turn % kAdWaves != wave) continue;
            const uint16_t* const LB = p.lb + ((int64_t)a * p.N + brow) * p.R;
            const float* const D = p.d + (mine ? 16 * i + r : 0) * p.R;
            for (int k0 = 0; k0 < p.R; k0 += 32) {
                const bool in = k0 + 8 * g < p.R;
                const int k = in ? k0 + 8 * g : 0;
                const bf16x8 ol = b8(LB + k, in);
                bf16x8 dv[3];
                d8(D + k, in && mine, dv);
                f32x4 z = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 3; j++) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ol, dv[j], z, 0, 0, 0);
#pragma unroll
                for (int v = 0; v < 4; v++) ad[i][v] += mine ? z[v] : 0.0f;
            }
        }
    }
    f32x4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; i++) acc[i] = f32x4{0, 0, 0, 0};
    for (int cb = c0; cb < c1; cb += U) {
        if (cb != c0) load_w(cb);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = cb + u < c1 ? cb + u : c1 - 1, left = (int)p.K - c * kChunk - 32 * g;
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
    // the waves' partial sums, in wave order; wave i takes row tile i
#pragma unroll
    for (int i = 0; i < TT; i++) part[wave][i][lane] = acc[i] * p.alpha[0] + ad[i];
    __syncthreads();
    if (wave >= TT || 16 * wave + r >= p.M) return;
    f32x4 y = part[0][wave][lane];
#pragma unroll
    for (int v = 1; v < kAdWaves; v++) y += part[v][wave][lane];
    store4(p, 16 * wave + r, n0 + 4 * g, y);
#endif
}

// Weight-only product of 16 XT rows and 256 columns, a share of the K axis and of
// the rows' distinct adapters: a wave has 32 columns to itself (two fragments, 128
// columns apart), the waves share x in LDS.  Where several workgroups share a tile,
// each leaves its sums in memory for k_wide_sum (a launch more, 4.2 us; with the last
// of them adding all this one took 37.7 us instead of 30).  Bound: three
// parts in turn, the first loads and the sums, the adapters, the K loop (64 rows, 5120
// x 8192, 48 adapters of rank 64: 30 us for 58 MB, 1.9 TB/s; 22 without the adapters'
// part, 20 without the K loop; beyond 64 rows 128 x 4096 x 4096 21 us, 256 29).
constexpr int kWideX = 32 << 10;  // LDS for x: 2 chunks of 64 rows; and 64 ranks of d
constexpr int kWideD = 200;       // bf16 of a row of d there (64 ranks' three parts, padded)
typedef W4Ring<2, 3> WideRing;

template <int XT, bool WHOLE>
__global__ __launch_bounds__(64 * kAdWaves, 2) void k_w4_wide(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __align__(16) uint8_t rings[kAdWaves * WideRing::BYTES];
    __shared__ __align__(16) uint8_t xs[kWideX];
    __shared__ float inv[kWideX / 256];
    static_assert(64 * kWideD * 2 <= kWideX, "64 ranks of 64 rows fit");
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
        uint16_t* const ds = (uint16_t*)xs;
        __syncthreads();
        for (int i = t; i < nr * 8; i += kThreads) {  // 8 ranks of a row
            const int q = i & 7, k = k0 + q * 8;
            bf16x8 dv[3];
            d8(p.d + (m0 + (i >> 3)) * p.R + (k < p.R ? k : 0), k < p.R, dv);
#pragma unroll
            for (int j = 0; j < 3; j++) *(bf16x8*)(ds + (i >> 3) * kWideD + j * 64 + q * 8) = dv[j];
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
                    const uint16_t* const d = ds + (16 * i + r) * kWideD + 32 * s + 8 * g;
#pragma unroll
                    for (int j = 0; j < 3; j++) {
                        const bf16x8 dv = b8(d + 64 * j, on && in);
#pragma unroll
                        for (int f = 0; f < 2; f++) {
                            const bf16x8 ol = __builtin_bit_cast(bf16x8, in ? bv[buf][f][s] : u32x4{0u, 0u, 0u, 0u});
                            z[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ol, dv, z[f], 0, 0, 0);
                        }
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
    // its sums of the rows, [share][row][N rounded up to 4]
    const int64_t np = (p.N + 3) / 4 * 4;
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int i = 0; i < XT; i++) {
            const int n = n0 + 128 * f + band_row(wave, 4 * g);
            if (16 * i + r < nr && n < N) *(f32x4*)(p.part + ((int64_t)share * p.M + m0 + 16 * i + r) * np + n) = acc[f][i];
        }
#endif
}

// The shares' sums, in their order, four columns a thread.
__global__ __launch_bounds__(256) void k_wide_sum(AParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int64_t np4 = (p.N + 3) / 4, all = p.M * np4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= all) return;
    const f32x4* const P = (const f32x4*)p.part + i;
    f32x4 y = {0, 0, 0, 0};
    constexpr int U = 16;  // loads in flight together
    for (int v0 = 0; v0 < p.shares; v0 += U) {
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; u++) v[u] = v0 + u < p.shares ? P[(v0 + u) * all] : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < U; u++) y += v[u];
    }
    store4(p, i / np4, i % np4 * 4, y);
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
    const unsigned ranks = (unsigned)((a.r + 15) / 16), rows = (unsigned)((a.m + 15) / 16);
    const int cus = device_cus();
    if (cus <= 0) return hipErrorInvalidDevice;
    if (a.m <= 64) {
        // few rows: a workgroup per 16 ranks and distinct adapter, since the
        // adapters' reads are the work (64 rows of 8192, 12 adapters of rank 64: 11.4
        // us, with two workgroups for a row tile's adapters 71.8)
        k_adapter_down<1, 1, 16, 4><<<dim3(ranks, rows, a.m < 16 ? (unsigned)a.m : 16u), 1024, 0, st>>>(p);
        return hipGetLastError();
    }
    // Many rows: two workgroups share a row tile's adapters (a prompt's end falls
    // inside a tile), and the tiles are the smallest that leave one workgroup a CU
    // (its rings fill the LDS): 16 rows and 16 ranks, then two or three tiles of
    // ranks on one read of x, then 32 rows (half the reads of A).  us, 16 ranks
    // against more at 16 rows: 128 x 4096 rank 64 7.7 : 11.6, 1024 x 4096 rank 32
    // 9.2 : 11.0, 2048 x 4096 rank 32 17.0 : 11.4.  16 rows against 32: 1024 x 4096
    // rank 64 13.8 : 17.4, 2048 x 4096 rank 64 24.7 : 18.5, 4096 x 5120 rank 16
    // 18.2 : 14.2, 8192 x 5120 rank 32 49.8 : 42.9.
    const unsigned few = (unsigned)cus / 2;
    if (rows * ranks <= few) k_adapter_down<1, 1, 16, 4><<<dim3(ranks, rows, 2), 1024, 0, st>>>(p);
    else if (ranks >= 2 && ranks <= 3 && rows * ((ranks + 1) / 2) <= few)
        k_adapter_down<2, 1, 16, 3><<<dim3((ranks + 1) / 2, rows, 2), 1024, 0, st>>>(p);
    else if (ranks >= 4 && rows * ((ranks + 2) / 3) <= few) k_adapter_down<3, 1, 16, 2><<<dim3((ranks + 2) / 3, rows, 2), 1024, 0, st>>>(p);
    else if (ranks == 1) k_adapter_down<1, 2, 16, 3><<<dim3(1, (rows + 1) / 2, 2), 1024, 0, st>>>(p);
    else if (ranks == 2) k_adapter_down<2, 2, 16, 2><<<dim3(1, (rows + 1) / 2, 2), 1024, 0, st>>>(p);
    else k_adapter_down<4, 2, 8, 3><<<dim3((ranks + 3) / 4, (rows + 1) / 2, 2), 512, 0, st>>>(p);
    return hipGetLastError();
}

template <int XT>
static void launch_wide(AParams p, int cus, hipStream_t st) {
    const int64_t cols = (p.N + 255) / 256, rows = (p.M + 16 * XT - 1) / (16 * XT), nch = (p.K + kChunk - 1) / kChunk;
    // one workgroup a CU, as far as the partial sums have room; a share has 2
    // chunks at least
    int64_t shares = p.part ? cus / (cols * rows) : 1;
    const int64_t room = kAdPartBytes / (p.M * ((p.N + 3) / 4 * 16));
    if (shares > room) shares = room;
    if (shares > nch / 2) shares = nch / 2;
    p.shares = (int)(shares < 1 ? 1 : shares);
    const dim3 grid((unsigned)cols, (unsigned)p.shares, (unsigned)rows);
    if (p.K % kChunk == 0) k_w4_wide<XT, true><<<grid, 64 * kAdWaves, 0, st>>>(p);
    else k_w4_wide<XT, false><<<grid, 64 * kAdWaves, 0, st>>>(p);
    if (p.shares > 1) k_wide_sum<<<dim3((unsigned)((p.M * ((p.N + 3) / 4) + 255) / 256)), 256, 0, st>>>(p);
}

template <int TT>
static void launch_narrow(const AParams& p, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + 15) / 16));
    if (p.K % kChunk == 0) k_w4a16_adapters<TT, true><<<grid, 64 * kAdWaves, 0, st>>>(p);
    else k_w4a16_adapters<TT, false><<<grid, 64 * kAdWaves, 0, st>>>(p);
}

hipError_t launch_w4a16_adapters(const AdapterArgs& a, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                                 const uint16_t* bias, uint16_t* out, float* part, hipStream_t st) {
    AParams p = params(a);
    p.b = b; p.b_sf = b_sf; p.alpha = alpha; p.bias = bias; p.out = out;
    p.part = part;
    const int cus = device_cus();
    if (cus <= 0) return hipErrorInvalidDevice;
    // Small weights: 16 columns a workgroup, whose waves read the rows themselves
    // (one launch, no sums between workgroups).  It is ahead while every workgroup is
    // resident at once and a wave's K range is one step of loads; larger weights
    // take the shared tiles.  us, this form against the tiles: 16 rows, 1024 x 1024
    // 6.8 : 10.2, 4096 x 4096 9.0 : 14.0, 8192 x 4096 14.2 : 16.2, 5120 x 8192 24.2 :
    // 16.2, 16384 x 1024 23.4 : 13.4; 32 rows, 2048 x 2048 6.9 : 12.6, 4096 x 4096
    // 13.0 : 17.9, 8192 x 4096 21.8 : 20.4; 64 rows, 4096 x 4096 21.5 : 26.0,
    // 8192 x 4096 40.8 : 27.9.  (The rule gives away up to 2.6 us for 1 to 16 rows
    // of a weight of few columns and 8192 in K: 2048 x 8192, 1 row, 8.4 : 11.0.)
    if (a.m <= 64 && a.k <= 4 * kAdWaves * kChunk && a.n <= (a.m <= 16 ? 8192 : 4096)) {
        if (a.m <= 16) launch_narrow<1>(p, st);
        else if (a.m <= 32) launch_narrow<2>(p, st);
        else launch_narrow<4>(p, st);
    }
    else if (a.m <= 16) launch_wide<1>(p, cus, st);
    else if (a.m <= 32) launch_wide<2>(p, cus, st);
    else launch_wide<4>(p, cus, st);
    return hipGetLastError();
}

}  // namespace nvfp4
