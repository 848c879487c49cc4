// rope_cache.hip -- what a layer does between its qkv projection and its
// attention: rotary positions with several axes, and the rows of the paged NVFP4
// cache, written (quantized) and read back.
//
// All three are bound by their bytes.  A thread reads 32 bytes (16 bf16, of K and of V
// for the cache), works on them in registers and writes them, neighbours side by side:
// 20280 tokens of 48 x 128 turn at 6.0 TB/s (read and written, 83 us), 8003 rows of K
// and V of 8 x 128 are quantized into the cache in 8.7 us (42 MB, 4.8 TB/s) and read
// back in 10.6 (4.0 TB/s).
#include "gemm_common.h"
#include "internal.h"
#include "quant_block.h"

namespace nvfp4 {

namespace {

// ---- rotary positions -----------------------------------------------------------

constexpr int kRopeAngles = 2048;  // (cos, sin) pairs of a workgroup's tokens

// Threads of a workgroup: one that streams has less to wait for at its barrier if it is small
// (20280 tokens of 48 x 128 at 128 / 256 threads: 82.9 / 86.5 us), where few tokens fill part of
// the card their angles want more threads (16 tokens: 3.8 / 3.5 us).
constexpr int rope_threads(bool stream) { return stream ? 128 : 256; }

struct RParams {
    const uint16_t* x;
    uint16_t* out;
    const int32_t* pos;      // [axes, t]
    const float* inv_freq;   // [rot / 2]
    int64_t x_stride, out_stride;
    int t, heads, d, rot, tokens;
    int ends[kRopeAxes];     // first pair past axis a
};

// A piece: W elements of bf16.
template <int W>
struct Piece { typedef uint32_t type __attribute__((ext_vector_type(W / 2))); };
template <>
struct Piece<2> { typedef uint32_t type; };
__device__ __forceinline__ uint32_t dword(uint32_t v, int) { return v; }
__device__ __forceinline__ void set_dword(uint32_t& v, int, uint32_t to) { v = to; }
template <typename V>
__device__ __forceinline__ uint32_t dword(const V& v, int j) { return v[j]; }
template <typename V>
__device__ __forceinline__ void set_dword(V& v, int j, uint32_t to) { v[j] = to; }

// Two pieces.  Halves: a holds x1 of W pairs, b their x2 (ca: the W).  Else a holds
// W / 2 pairs (ca), b as many others (cb).
template <bool HALVES, int W>
__device__ __forceinline__ void rotate(typename Piece<W>::type& a, typename Piece<W>::type& b, const float2* ca, const float2* cb) {
#pragma unroll
    for (int j = 0; j < W / 2; j++) {
        const uint32_t aj = dword(a, j), bj = dword(b, j);
        if (HALVES) {
            const float2 c0 = ca[2 * j], c1 = ca[2 * j + 1];
            const float p0 = bf16_lo(aj), p1 = bf16_hi(aj), q0 = bf16_lo(bj), q1 = bf16_hi(bj);
            set_dword(a, j, pack_bf16x2(p0 * c0.x - q0 * c0.y, p1 * c1.x - q1 * c1.y));
            set_dword(b, j, pack_bf16x2(q0 * c0.x + p0 * c0.y, q1 * c1.x + p1 * c1.y));
        } else {
            const float2 c0 = ca[j], c1 = cb[j];
            const float p0 = bf16_lo(aj), q0 = bf16_hi(aj), p1 = bf16_lo(bj), q1 = bf16_hi(bj);
            set_dword(a, j, pack_bf16x2(p0 * c0.x - q0 * c0.y, q0 * c0.x + p0 * c0.y));
            set_dword(b, j, pack_bf16x2(p1 * c1.x - q1 * c1.y, q1 * c1.x + p1 * c1.y));
        }
    }
}

// (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin) in fp32, rounded once to bf16.
// The angle pos * inv_freq is formed in fp64 turns and reduced to half a turn before
// it becomes fp32: at position 2^20 an fp32 product would be off by 0.06 radians.  A
// workgroup makes the angles of its tokens once, for all their heads.  A thread takes two
// pieces of W elements, in the same place of the rotated part's halves, so that eight threads
// cover whole lines.  W: 8, or what divides the pairs, so that the second half begins on a piece.
// STREAM: past the caches, where the tensor is larger than they are.
template <bool HALVES, bool STREAM, int W>
__global__ __launch_bounds__(rope_threads(STREAM)) void k_rope_axes(RParams p) {
    constexpr int kThreads = rope_threads(STREAM);
    __shared__ float2 cs[kRopeAngles];
    const int t0 = blockIdx.x * p.tokens;
    const int nt = p.t - t0 < p.tokens ? p.t - t0 : p.tokens;
    const int half = p.rot >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int tok = i / half, pair = i - tok * half;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kRopeAxes - 1; a++) axis += pair >= p.ends[a];
        const double turns = (double)p.pos[(int64_t)axis * p.t + t0 + tok] * (double)p.inv_freq[pair] * 0.15915494309189533577;
        const float r = (float)(2.0 * (turns - __builtin_rint(turns)));  // half turns, in [-1, 1]
        cs[i] = make_float2(cospif(r), sinpif(r));
    }
    __syncthreads();
    typedef typename Piece<W>::type piece;
    const int units = p.d / (2 * W), turned = p.rot / (2 * W);  // two pieces each; the first `turned` are rotated
    const int per = p.heads * units;
    for (int i = threadIdx.x; i < nt * per; i += kThreads) {
        const int tok = i / per, r = i - tok * per;
        const int head = r / units, u = r - head * units;
        const bool turn = u < turned;
        const int64_t e = (int64_t)head * p.d;
        // element offsets of the unit's pieces
        const int o0 = turn ? u * W : u * 2 * W;
        const int o1 = turn ? half + u * W : u * 2 * W + W;
        const uint16_t* const src = p.x + (t0 + tok) * p.x_stride + e;
        uint16_t* const dst = p.out + (t0 + tok) * p.out_stride + e;
        piece a = STREAM ? __builtin_nontemporal_load((const piece*)(src + o0)) : *(const piece*)(src + o0);
        piece b = STREAM ? __builtin_nontemporal_load((const piece*)(src + o1)) : *(const piece*)(src + o1);
        if (turn) {
            const float2* const c = cs + tok * half;
            if (HALVES) rotate<true, W>(a, b, c + u * W, nullptr);
            else rotate<false, W>(a, b, c + u * (W / 2), c + (half >> 1) + u * (W / 2));
        }
        if (STREAM) {
            __builtin_nontemporal_store(a, (piece*)(dst + o0));
            __builtin_nontemporal_store(b, (piece*)(dst + o1));
        } else {
            *(piece*)(dst + o0) = a;
            *(piece*)(dst + o1) = b;
        }
    }
}

// ---- the cache --------------------------------------------------------------------

struct CParams {
    const uint16_t *k, *v;   // append: [t, heads, d]
    uint16_t *ko, *vo;       // read
    const int32_t* slots;
    const float* gs;
    uint8_t *kv, *sf;
    int64_t k_stride, v_stride, nslots;
    int t, heads, d, page_log2;
};

// One block (16 elements) of a head's row a thread, of K and of V; consecutive threads take the
// blocks of a row, then the heads, then the tokens.  At most 2^31 blocks: their index stays in
// 32 bits.
template <bool READ>
__global__ __launch_bounds__(kRowThreadsMany) void k_kv_rows(CParams p) {
    const uint32_t blocks = (uint32_t)p.d >> 4;
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    const uint32_t row = i / blocks;
    const int blk = (int)(i - row * blocks);
    const uint32_t tok32 = row / (uint32_t)p.heads;
    const int head = (int)(row - tok32 * (uint32_t)p.heads);
    const int64_t tok = tok32;
    if (tok >= p.t) return;
    const int slot = p.slots[tok];
    if (slot < 0 || slot >= p.nslots) return;
    // the head's rows of K and of V on the page, and the row's place among them
    const int64_t plane = (int64_t)(slot >> p.page_log2) * 2 * p.heads + head;
    const int off = slot & ((1 << p.page_log2) - 1);
    int64_t code[2], sf[2];
#pragma unroll
    for (int w = 0; w < 2; w++) {
        const int64_t r = plane + w * p.heads;
        code[w] = (((r << p.page_log2) + off) * p.d >> 1) + blk * 8;
        sf[w] = ((r * blocks + blk) << p.page_log2) + off;
    }
    const int64_t at[2] = {tok * p.k_stride + head * p.d + blk * 16, tok * p.v_stride + head * p.d + blk * 16};
    const float gs[2] = {p.gs[0], p.gs[1]};
    if (!READ) {
        u32x4 r[2][2];
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const u32x4* const src = (const u32x4*)((w ? p.v : p.k) + at[w]);
            r[w][0] = src[0];
            r[w][1] = src[1];
        }
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const u32x4 none[2] = {};
            float f[16];
            const float amax = process_block<V_BF16>(r[w], none, f);
            const uint32_t s = ue4m3_encode(div6(amax) * gs[w]);
            const float ds = ue4m3_decode(s);
            uint32_t w0, w1;
            pack_block(f, ds == 0.0f ? 0.0f : gs[w] / ds, w0, w1);
            *(u32x2*)(p.kv + code[w]) = u32x2{w0, w1};
            p.sf[sf[w]] = (uint8_t)s;
        }
    } else {
        u32x2 c[2];
        uint8_t s8[2];
#pragma unroll
        for (int w = 0; w < 2; w++) {
            c[w] = *(const u32x2*)(p.kv + code[w]);
            s8[w] = p.sf[sf[w]];
        }
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const float s = ue4m3_decode(s8[w]);
            // code * scale is exact; its quotient by gs, correctly rounded by one correction
            // step from the reciprocal (Markstein), then rounded to bf16
            const float rcp = 1.0f / gs[w];
            u32x4* const dst = (u32x4*)((w ? p.vo : p.ko) + at[w]);
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            if (!(gs[w] >= 0x1p-112f && gs[w] <= 0x1p112f)) {  // where a step of it could leave fp32's normal numbers
#pragma unroll 1
                for (int j = 0; j < 8; j++) {
                    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((j < 4 ? c[w][0] : c[w][1]) >> 8 * (j & 3), 1.0f, 0);
                    ((uint32_t*)dst)[j] = pack_bf16x2(v[0] * s / gs[w], v[1] * s / gs[w]);
                }
                continue;
            }
            u32x4 y[2];
            auto put = [&](int j, f32x2 v) {
                const float a = v[0] * s, b = v[1] * s;
                const float qa = a * rcp, qb = b * rcp;
                y[j >> 2][j & 3] = pack_bf16x2(__builtin_fmaf(__builtin_fmaf(-qa, gs[w], a), rcp, qa),
                                               __builtin_fmaf(__builtin_fmaf(-qb, gs[w], b), rcp, qb));
            };
#pragma unroll
            for (int h = 0; h < 2; h++) {
                put(4 * h + 0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w][h], 1.0f, 0));
                put(4 * h + 1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w][h], 1.0f, 1));
                put(4 * h + 2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w][h], 1.0f, 2));
                put(4 * h + 3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w][h], 1.0f, 3));
            }
            dst[0] = y[0];
            dst[1] = y[1];
        }
    }
}

}  // namespace

template <int W>
static void rope(const RParams& p, bool interleaved, bool stream, dim3 grid, hipStream_t st) {
    const int threads = rope_threads(stream);
    if (interleaved) {
        if (stream) k_rope_axes<false, true, W><<<grid, threads, 0, st>>>(p);
        else k_rope_axes<false, false, W><<<grid, threads, 0, st>>>(p);
    } else {
        if (stream) k_rope_axes<true, true, W><<<grid, threads, 0, st>>>(p);
        else k_rope_axes<true, false, W><<<grid, threads, 0, st>>>(p);
    }
}

hipError_t launch_rope_axes(const RopeArgs& a, hipStream_t st) {
    RParams p{};
    p.x = a.x; p.out = a.out; p.pos = a.positions; p.inv_freq = a.inv_freq;
    p.x_stride = a.x_stride; p.out_stride = a.out_stride;
    p.t = (int)a.t; p.heads = (int)a.heads; p.d = (int)a.d; p.rot = (int)a.rot;
    int end = 0;
    for (int i = 0; i < kRopeAxes; i++) {
        end += i < a.axes ? a.sections[i] : 0;
        p.ends[i] = i < a.axes - 1 ? end : 1 << 30;
    }
    // a few pieces a thread, while the workgroups still fill the card several times
    const RopePlan plan = rope_plan(a.t, a.heads, a.d, a.rot / 2);
    const int threads = rope_threads(plan.stream);
    const int64_t per = a.heads * (a.d / 16);  // (pairs of 16-byte pieces)
    int64_t tokens = per >= 4 * threads ? 1 : 4 * threads / per;
    const int64_t most = kRopeAngles / (a.rot / 2);
    if (tokens > most) tokens = most;
    while (tokens > 1 && (a.t + tokens - 1) / tokens < 1024) tokens >>= 1;
    p.tokens = (int)tokens;
    const dim3 grid((unsigned)((a.t + tokens - 1) / tokens));
    if (plan.width == 8) rope<8>(p, a.interleaved, plan.stream, grid, st);
    else if (plan.width == 4) rope<4>(p, a.interleaved, plan.stream, grid, st);
    else rope<2>(p, a.interleaved, plan.stream, grid, st);
    return hipGetLastError();
}

hipError_t launch_kv_rows(const KvRowsArgs& a, hipStream_t st) {
    CParams p{};
    p.k = a.k; p.v = a.v; p.ko = a.k_out; p.vo = a.v_out; p.slots = a.slots; p.gs = a.kv_gs;
    p.kv = a.kv; p.sf = a.kv_sf; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
    p.nslots = a.pages * a.page; p.t = (int)a.t; p.heads = (int)a.heads; p.d = (int)a.d;
    p.page_log2 = __builtin_ctzll((unsigned long long)a.page);
    const int64_t n = a.t * a.heads * (a.d / 16);
    const int threads = kv_rows_threads(n);
    const dim3 grid((unsigned)((n + threads - 1) / threads));
    if (a.read) k_kv_rows<true><<<grid, threads, 0, st>>>(p);
    else k_kv_rows<false><<<grid, threads, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace nvfp4
