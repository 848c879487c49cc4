// abi.cpp -- the extern "C" entry points declared in include/nvfp4.h,
// include/nvfp4_serving.h and include/nvfp4_attention.h: argument validation (before anything is enqueued) and dispatch to the
// kernel launchers.  The library allocates no memory and keeps no state.
#include <hip/hip_runtime.h>

#include "../../include/nvfp4.h"
#include "../../include/nvfp4_serving.h"
#include "../../include/nvfp4_attention.h"
#include "internal.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool dim_ok(int64_t v) { return v >= 1 && v <= kMaxDim; }

int launch_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_LAUNCH_FAILED; }

// Sizes must keep every per-item element count and every grid dimension in
// range of the kernels' 32-bit tile indices.
bool quant_sizes_ok(int64_t b, int64_t m, int64_t K) {
    if (!dim_ok(b) || !dim_ok(m) || !dim_ok(K)) return false;
    if (b > 65535) return false;
    int64_t nrt = (m + 127) / 128, nct = (K + 63) / 64;
    if (nrt > 65535 || nct > ((int64_t)1 << 31) - 1) return false;
    if (nrt * nct > ((int64_t)1 << 31) - 1) return false;
    return true;
}

// Bytes of a swizzled scale buffer for `rows` rows of `nblk` blocks:
// pad_up(rows,128) * pad_up(nblk,4).  The GEMM kernels address a scale
// buffer through a 32-bit buffer descriptor with 32-bit signed per-step
// offsets, so each one must stay below 2^31 bytes.
bool gemm_sf_ok(int64_t rows, int64_t nblk) {
    return ((rows + 127) / 128 * 128) * ((nblk + 3) / 4 * 4) < ((int64_t)1 << 31);
}

}  // namespace

extern "C" {

static int quantize_check(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                          float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                          uint8_t* out_fp4, uint8_t* out_sf) {
    if (!x || !global_scale || !out_fp4 || !out_sf) return NVFP4_NULL_POINTER;
    if (x_dtype != NVFP4_BF16 && x_dtype != NVFP4_F32) return NVFP4_BAD_DTYPE;
    if (gs_mode != NVFP4_GS_STATIC && gs_mode != NVFP4_GS_DYNAMIC) return NVFP4_UNSUPPORTED;
    if (k < 16 || k % 16 != 0 || !quant_sizes_ok(1, m, k)) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(out_fp4) || !aligned16(out_sf) ||
        (pre_quant_scale && !aligned16(pre_quant_scale)) || ((uintptr_t)global_scale & 3u) ||
        ((uintptr_t)gs_other & 3u) || ((uintptr_t)alpha & 3u))
        return NVFP4_MISALIGNED;
    return NVFP4_OK;
}

// Arguments already checked by quantize_check.
static int quantize_launch(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                           float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                           uint8_t* out_fp4, uint8_t* out_sf, float* ws, void* stream) {
    nvfp4::QuantizeArgs a{};
    a.x = x; a.x_dtype = x_dtype; a.pqs = pre_quant_scale; a.mask = nullptr;
    a.gs = global_scale; a.out_fp4 = out_fp4; a.out_sf = out_sf;
    a.b = 1; a.m = m; a.k_in = k; a.silu = false; a.dynamic = gs_mode == NVFP4_GS_DYNAMIC;
    a.gs_other = gs_other; a.alpha_out = alpha;
    a.ws = a.dynamic ? ws : nullptr;
    return launch_status(nvfp4::launch_quantize(a, (hipStream_t)stream));
}

static int quantize_common(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                           float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                           uint8_t* out_fp4, uint8_t* out_sf, float* ws, void* stream) {
    const int st = quantize_check(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, gs_other, alpha,
                                  out_fp4, out_sf);
    if (st != NVFP4_OK) return st;
    return quantize_launch(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, gs_other, alpha, out_fp4,
                           out_sf, ws, stream);
}

int nvfp4_quantize(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                   float* global_scale, int gs_mode, uint8_t* out_fp4, uint8_t* out_sf,
                   void* stream) {
    return quantize_common(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, nullptr, nullptr,
                           out_fp4, out_sf, nullptr, stream);
}

int nvfp4_quantize_alpha(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                         float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                         uint8_t* out_fp4, uint8_t* out_sf, void* stream) {
    if (!gs_other || !alpha) return NVFP4_NULL_POINTER;
    return quantize_common(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, gs_other, alpha,
                           out_fp4, out_sf, nullptr, stream);
}

int nvfp4_quantize_ws(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                      float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                      uint8_t* out_fp4, uint8_t* out_sf, void* workspace, int64_t workspace_bytes,
                      void* stream) {
    if (!gs_other != !alpha) return NVFP4_NULL_POINTER;
    if (gs_mode == NVFP4_GS_DYNAMIC) {
        if (!workspace) return NVFP4_NULL_POINTER;
        if (workspace_bytes < NVFP4_QUANTIZE_WS_BYTES) return NVFP4_BAD_SHAPE;
        if (!aligned16(workspace)) return NVFP4_MISALIGNED;
    }
    static_assert(NVFP4_QUANTIZE_WS_BYTES >= nvfp4::kQuantizeWsFloats * 4, "workspace holds the partials");
    return quantize_common(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, gs_other, alpha,
                           out_fp4, out_sf, (float*)workspace, stream);
}

int nvfp4_quantize_noalloc(const void* x, int x_dtype, int64_t m, int64_t k, const void* pre_quant_scale,
                           float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                           uint8_t* out_fp4, uint8_t* out_sf, void* stream) {
    if (!gs_other != !alpha) return NVFP4_NULL_POINTER;
    // every argument is checked before the device is touched (symbol lookup)
    const int st = quantize_check(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, gs_other, alpha,
                                  out_fp4, out_sf);
    if (st != NVFP4_OK) return st;
    float* ws = nullptr;
    if (gs_mode == NVFP4_GS_DYNAMIC && nvfp4::scratch_for_current_device(&ws) != hipSuccess)
        return NVFP4_LAUNCH_FAILED;
    return quantize_launch(x, x_dtype, m, k, pre_quant_scale, global_scale, gs_mode, gs_other, alpha, out_fp4,
                           out_sf, ws, stream);
}

static int lora_down_common(const void* x, int64_t m, int64_t k, const void* pre_quant_scale, const void* l2,
                            int64_t r, float* global_scale, int gs_mode, uint8_t* out_fp4, uint8_t* out_sf, void* d,
                            bool prepared, void* stream) {
    if (!x || !pre_quant_scale || !l2 || !global_scale || !out_fp4 || !out_sf || !d) return NVFP4_NULL_POINTER;
    if (gs_mode != NVFP4_GS_STATIC && gs_mode != NVFP4_GS_DYNAMIC) return NVFP4_UNSUPPORTED;
    if (r <= 0 || r % 32 != 0 || r > 128) return NVFP4_BAD_RANK;
    if (k < 16 || k % 16 != 0 || !quant_sizes_ok(1, m, k)) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(pre_quant_scale) || !aligned16(l2) || !aligned16(out_fp4) ||
        !aligned16(out_sf) || !aligned16(d) || ((uintptr_t)global_scale & 3u))
        return NVFP4_MISALIGNED;
    nvfp4::QuantizeArgs a{};
    a.x = x; a.x_dtype = NVFP4_BF16; a.pqs = pre_quant_scale; a.mask = nullptr;
    a.gs = global_scale; a.out_fp4 = out_fp4; a.out_sf = out_sf;
    a.b = 1; a.m = m; a.k_in = k; a.silu = false; a.dynamic = gs_mode == NVFP4_GS_DYNAMIC;
    return launch_status(nvfp4::launch_quantize_lora(a, (const uint16_t*)l2, (uint16_t*)d, (int)r, prepared,
                                                      (hipStream_t)stream));
}

int nvfp4_quantize_lora_down(const void* x, int64_t m, int64_t k, const void* pre_quant_scale,
                             const void* l2, int64_t r, float* global_scale, int gs_mode, uint8_t* out_fp4,
                             uint8_t* out_sf, void* d, void* stream) {
    return lora_down_common(x, m, k, pre_quant_scale, l2, r, global_scale, gs_mode, out_fp4, out_sf, d, false,
                            stream);
}

int nvfp4_lora_down_prepare(const void* pre_quant_scale, const void* l2, int64_t r, int64_t k, void* w_out,
                            void* stream) {
    if (!pre_quant_scale || !l2 || !w_out) return NVFP4_NULL_POINTER;
    if (r <= 0 || r % 32 != 0 || r > 128) return NVFP4_BAD_RANK;
    if (k < 16 || k % 16 != 0 || !dim_ok(k)) return NVFP4_BAD_SHAPE;
    if (!aligned16(pre_quant_scale) || !aligned16(l2) || !aligned16(w_out)) return NVFP4_MISALIGNED;
    return launch_status(nvfp4::launch_lora_split((const uint16_t*)pre_quant_scale, (const uint16_t*)l2,
                                                  (uint16_t*)w_out, (int)r, k, (hipStream_t)stream));
}

int nvfp4_quantize_lora_down_prepared(const void* x, int64_t m, int64_t k, const void* pre_quant_scale,
                                      const void* w_prepared, int64_t r, float* global_scale, int gs_mode,
                                      uint8_t* out_fp4, uint8_t* out_sf, void* d, void* stream) {
    return lora_down_common(x, m, k, pre_quant_scale, w_prepared, r, global_scale, gs_mode, out_fp4, out_sf, d,
                            true, stream);
}

// The batched forms (k_in: the input row width, 2K for silu): every check of
// the call, then the launch; with_ws: the *_ws forms (gs_other / alpha and,
// in DYNAMIC mode, the workspace).
static int batched_common(const void* x, int64_t b, int64_t m, int64_t k_in, bool silu, const int32_t* mask,
                          float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                          uint8_t* out_fp4, uint8_t* out_sf, bool with_ws, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    if (!x || !global_scale || !out_fp4 || !out_sf) return NVFP4_NULL_POINTER;
    if (!gs_other != !alpha) return NVFP4_NULL_POINTER;
    if (gs_mode != NVFP4_GS_STATIC && gs_mode != NVFP4_GS_DYNAMIC) return NVFP4_UNSUPPORTED;
    int64_t k = k_in;
    if (silu) {
        if (k_in < 32 || k_in % 2 != 0 || (k_in / 2) % 16 != 0) return NVFP4_BAD_SHAPE;
        k = k_in / 2;
    }
    if (k < 16 || k % 16 != 0 || !quant_sizes_ok(b, m, k)) return NVFP4_BAD_SHAPE;
    const bool use_ws = with_ws && gs_mode == NVFP4_GS_DYNAMIC;
    if (use_ws) {
        if (!workspace) return NVFP4_NULL_POINTER;
        if (workspace_bytes < NVFP4_BATCHED_WS_BYTES(b, m, k)) return NVFP4_BAD_SHAPE;
    }
    if (!aligned16(x) || !aligned16(out_fp4) || !aligned16(out_sf) || ((uintptr_t)global_scale & 3u) ||
        ((uintptr_t)mask & 3u) || ((uintptr_t)gs_other & 3u) || ((uintptr_t)alpha & 3u) ||
        (use_ws && !aligned16(workspace)))
        return NVFP4_MISALIGNED;
    nvfp4::QuantizeArgs a{};
    a.x = x; a.x_dtype = NVFP4_BF16; a.pqs = nullptr; a.mask = mask;
    a.gs = global_scale; a.out_fp4 = out_fp4; a.out_sf = out_sf;
    a.b = b; a.m = m; a.k_in = k_in; a.silu = silu; a.dynamic = gs_mode == NVFP4_GS_DYNAMIC;
    a.gs_other = gs_other; a.alpha_out = alpha;
    a.ws = use_ws ? (float*)workspace : nullptr;
    // silu with room for h after the partials: silu is evaluated once
    if (silu && use_ws && workspace_bytes >= NVFP4_SILU_WS_BYTES(b, m, k))
        a.hbuf = (uint16_t*)((char*)workspace + (NVFP4_BATCHED_WS_BYTES(b, m, k) + 255) / 256 * 256);
    return launch_status(nvfp4::launch_quantize(a, (hipStream_t)stream));
}

static_assert(NVFP4_BATCHED_WS_BYTES(1, 1, 16) >= nvfp4::kQuantizeWsFloats * 4, "the flat amax pass's partials fit");

int nvfp4_quantize_masked_batched(const void* x, int64_t b, int64_t m, int64_t k,
                                  const int32_t* mask, float* global_scale, int gs_mode,
                                  uint8_t* out_fp4, uint8_t* out_sf, void* stream) {
    return batched_common(x, b, m, k, false, mask, global_scale, gs_mode, nullptr, nullptr, out_fp4, out_sf,
                          false, nullptr, 0, stream);
}

int nvfp4_quantize_masked_batched_ws(const void* x, int64_t b, int64_t m, int64_t k, const int32_t* mask,
                                     float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                                     uint8_t* out_fp4, uint8_t* out_sf, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
    return batched_common(x, b, m, k, false, mask, global_scale, gs_mode, gs_other, alpha, out_fp4, out_sf,
                          true, workspace, workspace_bytes, stream);
}

int silu_mul_nvfp4_quantize(const void* x, int64_t b, int64_t m, int64_t k2, const int32_t* mask,
                            float* global_scale, int gs_mode, uint8_t* out_fp4, uint8_t* out_sf,
                            void* stream) {
    return batched_common(x, b, m, k2, true, mask, global_scale, gs_mode, nullptr, nullptr, out_fp4, out_sf,
                          false, nullptr, 0, stream);
}

int silu_mul_nvfp4_quantize_ws(const void* x, int64_t b, int64_t m, int64_t k2, const int32_t* mask,
                               float* global_scale, int gs_mode, const float* gs_other, float* alpha,
                               uint8_t* out_fp4, uint8_t* out_sf, void* workspace, int64_t workspace_bytes,
                               void* stream) {
    return batched_common(x, b, m, k2, true, mask, global_scale, gs_mode, gs_other, alpha, out_fp4, out_sf,
                          true, workspace, workspace_bytes, stream);
}

static_assert(NVFP4_GEMM_WS_BYTES == nvfp4::kGemmWsBytes, "GEMM workspace size");

// Every check of a GEMM call; fills g when they pass.
static int gemm_check(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                      const float* alpha, const int32_t* mask, const void* bias, const void* d,
                      const void* l1, void* out, int64_t E, int64_t m, int64_t n, int64_t k,
                      int64_t r, void* ws, int64_t ws_bytes, nvfp4::GemmArgs& g) {
    if (!a || !b || !a_sf || !b_sf || !alpha || !out) return NVFP4_NULL_POINTER;
    if (!dim_ok(E) || !dim_ok(m) || !dim_ok(n) || k < 16 || k % 16 != 0 || k > kMaxDim)
        return NVFP4_BAD_SHAPE;
    if (E > 65535 || ((m + 63) / 64) * ((n + 63) / 64) > ((int64_t)1 << 31) - 1) return NVFP4_BAD_SHAPE;
    // the GEMM kernels address one FP4 matrix with 32-bit byte offsets
    if (m * (k / 2) > ((int64_t)1 << 32) - 64 || n * (k / 2) > ((int64_t)1 << 32) - 64) return NVFP4_UNSUPPORTED;
    if (!gemm_sf_ok(m, k / 16) || !gemm_sf_ok(n, k / 16)) return NVFP4_UNSUPPORTED;
    if (!aligned16(a) || !aligned16(b) || !aligned16(a_sf) || !aligned16(b_sf) || !aligned16(out) ||
        ((uintptr_t)alpha & 3u) || (bias && !aligned16(bias)) || (d && !aligned16(d)) ||
        (l1 && !aligned16(l1)) || ((uintptr_t)mask & 3u))
        return NVFP4_MISALIGNED;
    if (ws && ws_bytes < NVFP4_GEMM_WS_BYTES) return NVFP4_BAD_SHAPE;
    if (ws && !aligned16(ws)) return NVFP4_MISALIGNED;
    g.a = a; g.b = b; g.a_sf = a_sf; g.b_sf = b_sf; g.alpha = alpha; g.mask = mask;
    g.bias = (const uint16_t*)bias; g.d = (const uint16_t*)d; g.l1 = (const uint16_t*)l1;
    g.out = (uint16_t*)out; g.E = E; g.m = m; g.n = n; g.k = k; g.r = r;
    g.ws = (float*)ws;
    return NVFP4_OK;
}

static int gemm_common(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                       const float* alpha, const int32_t* mask, const void* bias, const void* d,
                       const void* l1, void* out, int64_t E, int64_t m, int64_t n, int64_t k,
                       int64_t r, void* ws, int64_t ws_bytes, void* stream) {
    nvfp4::GemmArgs g{};
    const int st = gemm_check(a, b, a_sf, b_sf, alpha, mask, bias, d, l1, out, E, m, n, k, r, ws, ws_bytes, g);
    if (st != NVFP4_OK) return st;
    return launch_status(nvfp4::launch_gemm(g, (hipStream_t)stream));
}

int nvfp4_gemm(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
               const float* alpha, const void* bias, void* out, int64_t m, int64_t n, int64_t k,
               void* stream) {
    return gemm_common(a, b, a_sf, b_sf, alpha, nullptr, bias, nullptr, nullptr, out, 1, m, n, k, 0,
                       nullptr, 0, stream);
}

int nvfp4_gemm_ws(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                  const float* alpha, const void* bias, void* out, int64_t m, int64_t n, int64_t k,
                  void* workspace, int64_t workspace_bytes, void* stream) {
    return gemm_common(a, b, a_sf, b_sf, alpha, nullptr, bias, nullptr, nullptr, out, 1, m, n, k, 0,
                       workspace, workspace_bytes, stream);
}

int nvfp4_gemm_grouped_masked(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf,
                              const uint8_t* b_sf, const float* alpha, const int32_t* mask,
                              void* out, int64_t E, int64_t m, int64_t n, int64_t k, void* stream) {
    if (!mask) return NVFP4_NULL_POINTER;
    return gemm_common(a, b, a_sf, b_sf, alpha, mask, nullptr, nullptr, nullptr, out, E, m, n, k, 0,
                       nullptr, 0, stream);
}

int nvfp4_gemm_grouped_masked_ws(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf,
                                 const uint8_t* b_sf, const float* alpha, const int32_t* mask,
                                 void* out, int64_t E, int64_t m, int64_t n, int64_t k,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
    if (!mask) return NVFP4_NULL_POINTER;
    return gemm_common(a, b, a_sf, b_sf, alpha, mask, nullptr, nullptr, nullptr, out, E, m, n, k, 0,
                       workspace, workspace_bytes, stream);
}

int nvfp4_gemm_grouped_masked_silu_quantize(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf,
                                            const uint8_t* b_sf, const float* alpha, const int32_t* mask,
                                            const float* global_scale, int64_t E, int64_t m, int64_t n2,
                                            int64_t k, uint8_t* out_fp4, uint8_t* out_sf, void* stream) {
    if (!a || !b || !a_sf || !b_sf || !alpha || !mask || !global_scale || !out_fp4 || !out_sf)
        return NVFP4_NULL_POINTER;
    if (!dim_ok(E) || !dim_ok(m) || !dim_ok(n2) || k < 16 || k % 16 != 0 || k > kMaxDim) return NVFP4_BAD_SHAPE;
    if (n2 % 2 != 0 || n2 / 2 < 16 || (n2 / 2) % 16 != 0 || !quant_sizes_ok(E, m, n2 / 2)) return NVFP4_BAD_SHAPE;
    if (E > 65535 || ((m + 127) / 128) * ((n2 / 2 + 63) / 64) > ((int64_t)1 << 31) - 1) return NVFP4_BAD_SHAPE;
    if (m * (k / 2) > ((int64_t)1 << 32) - 64 || n2 * (k / 2) > ((int64_t)1 << 32) - 64) return NVFP4_UNSUPPORTED;
    if (!gemm_sf_ok(m, k / 16) || !gemm_sf_ok(n2, k / 16)) return NVFP4_UNSUPPORTED;
    if (!aligned16(a) || !aligned16(b) || !aligned16(a_sf) || !aligned16(b_sf) || !aligned16(out_fp4) ||
        !aligned16(out_sf) || ((uintptr_t)alpha & 3u) || ((uintptr_t)mask & 3u) || ((uintptr_t)global_scale & 3u))
        return NVFP4_MISALIGNED;
    nvfp4::GemmArgs g{};
    g.a = a; g.b = b; g.a_sf = a_sf; g.b_sf = b_sf; g.alpha = alpha; g.mask = mask;
    g.E = E; g.m = m; g.n = n2; g.k = k;
    nvfp4::SiluQuantOut q{out_fp4, out_sf, global_scale};
    return launch_status(nvfp4::launch_gemm_silu_quantize(g, q, (hipStream_t)stream));
}

int nvfp4_gemm_svdquant(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                        const float* alpha, const void* d, const void* l1, const void* bias,
                        void* out, int64_t m, int64_t n, int64_t k, int64_t r, void* stream) {
    if (!d || !l1) return NVFP4_NULL_POINTER;
    if (r <= 0 || r % 32 != 0 || r > 4096) return NVFP4_BAD_RANK;
    return gemm_common(a, b, a_sf, b_sf, alpha, nullptr, bias, d, l1, out, 1, m, n, k, r, nullptr, 0, stream);
}

int nvfp4_gemm_svdquant_ws(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                           const float* alpha, const void* d, const void* l1, const void* bias,
                           void* out, int64_t m, int64_t n, int64_t k, int64_t r, void* workspace,
                           int64_t workspace_bytes, void* stream) {
    if (!d || !l1) return NVFP4_NULL_POINTER;
    if (r <= 0 || r % 32 != 0 || r > 4096) return NVFP4_BAD_RANK;
    return gemm_common(a, b, a_sf, b_sf, alpha, nullptr, bias, d, l1, out, 1, m, n, k, r, workspace,
                       workspace_bytes, stream);
}

int nvfp4_gemm_w4a16(const void* a, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                     const void* bias, void* out, int64_t m, int64_t n, int64_t k, void* stream) {
    if (!a || !b || !b_sf || !alpha || !out) return NVFP4_NULL_POINTER;
    if (!dim_ok(m) || !dim_ok(n) || k < 16 || k % 16 != 0 || k > kMaxDim) return NVFP4_BAD_SHAPE;
    if ((m + 15) / 16 > 65535 || (n + 15) / 16 > ((int64_t)1 << 31) - 1) return NVFP4_BAD_SHAPE;
    if (!aligned16(a) || !aligned16(b) || !aligned16(b_sf) || !aligned16(out) || ((uintptr_t)alpha & 3u) ||
        (bias && !aligned16(bias)))
        return NVFP4_MISALIGNED;
    nvfp4::GemmArgs g{};
    g.a = (const uint8_t*)a; g.b = b; g.b_sf = b_sf; g.alpha = alpha;
    g.bias = (const uint16_t*)bias; g.out = (uint16_t*)out;
    g.E = 1; g.m = m; g.n = n; g.k = k;
    return launch_status(nvfp4::launch_gemm_w4a16(g, (hipStream_t)stream));
}

int nvfp4_linear_small(const void* x, int64_t m, int64_t k, const uint8_t* b, const uint8_t* b_sf,
                       const float* gs_b, const void* bias, void* out, int64_t n, float* gs_out, void* stream) {
    if (!x || !b || !b_sf || !gs_b || !out) return NVFP4_NULL_POINTER;
    if (!dim_ok(m) || !dim_ok(n) || k < 16 || k % 16 != 0 || k > kMaxDim) return NVFP4_BAD_SHAPE;
    if (m > nvfp4::kLinearSmallMaxRows || k % 128 != 0 || k > nvfp4::kLinearSmallMaxK) return NVFP4_UNSUPPORTED;
    if ((n + 15) / 16 > ((int64_t)1 << 31) - 1 || !gemm_sf_ok(n, k / 16)) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(b) || !aligned16(b_sf) || !aligned16(out) || ((uintptr_t)gs_b & 3u) ||
        ((uintptr_t)gs_out & 3u) || (bias && !aligned16(bias)))
        return NVFP4_MISALIGNED;
    nvfp4::LinearSmallArgs a{};
    a.x = x; a.b = b; a.b_sf = b_sf; a.gs_b = gs_b; a.bias = (const uint16_t*)bias;
    a.out = (uint16_t*)out; a.gs_out = gs_out; a.m = m; a.n = n; a.k = k;
    return launch_status(nvfp4::launch_linear_small(a, (hipStream_t)stream));
}

int mxfp4_quantize(const void* x, int x_dtype, int64_t m, int64_t k, uint8_t* out_fp4, uint8_t* out_sf,
                   void* stream) {
    if (!x || !out_fp4 || !out_sf) return NVFP4_NULL_POINTER;
    if (x_dtype != NVFP4_BF16 && x_dtype != NVFP4_F32) return NVFP4_BAD_DTYPE;
    if (k < 32 || k % 32 != 0 || !quant_sizes_ok(1, m, k)) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(out_fp4) || !aligned16(out_sf)) return NVFP4_MISALIGNED;
    nvfp4::MxQuantizeArgs a{x, x_dtype, out_fp4, out_sf, m, k};
    return launch_status(nvfp4::launch_quantize_mx(a, (hipStream_t)stream));
}

int mxfp4_gemm(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf, const float* alpha,
               const void* bias, void* out, int64_t m, int64_t n, int64_t k, void* stream) {
    if (!a || !b || !a_sf || !b_sf || !out) return NVFP4_NULL_POINTER;
    if (!dim_ok(m) || !dim_ok(n) || k < 32 || k % 32 != 0 || k > kMaxDim) return NVFP4_BAD_SHAPE;
    if (((m + 127) / 128) * ((n + 127) / 128) > ((int64_t)1 << 31) - 1) return NVFP4_BAD_SHAPE;
    if (m * (k / 2) > ((int64_t)1 << 32) - 64 || n * (k / 2) > ((int64_t)1 << 32) - 64) return NVFP4_UNSUPPORTED;
    if (!gemm_sf_ok(m, k / 32) || !gemm_sf_ok(n, k / 32)) return NVFP4_UNSUPPORTED;
    if (!aligned16(a) || !aligned16(b) || !aligned16(a_sf) || !aligned16(b_sf) || !aligned16(out) ||
        ((uintptr_t)alpha & 3u) || (bias && !aligned16(bias)))
        return NVFP4_MISALIGNED;
    nvfp4::GemmArgs g{};
    g.a = a; g.b = b; g.a_sf = a_sf; g.b_sf = b_sf; g.alpha = alpha;
    g.bias = (const uint16_t*)bias; g.out = (uint16_t*)out;
    g.E = 1; g.m = m; g.n = n; g.k = k;
    return launch_status(nvfp4::launch_gemm_mx(g, (hipStream_t)stream));
}

int nvfp4_alpha(const float* gs_a, const float* gs_b, float* alpha, int64_t count, void* stream) {
    if (!gs_a || !gs_b || !alpha) return NVFP4_NULL_POINTER;
    if (!dim_ok(count)) return NVFP4_BAD_SHAPE;
    if (((uintptr_t)gs_a & 3u) || ((uintptr_t)gs_b & 3u) || ((uintptr_t)alpha & 3u))
        return NVFP4_MISALIGNED;
    return launch_status(nvfp4::launch_alpha(gs_a, gs_b, alpha, count, (hipStream_t)stream));
}

static_assert(4096 == nvfp4::kMoePartRows * 4 && nvfp4::kMoePartRows >= NVFP4_MOE_SMALL_MAX_TOKENS,
              "the workspace holds the partial sums");

int nvfp4_moe_small(const void* x, int64_t t, int64_t h, const void* logits, int logits_dtype, int64_t E,
                    int64_t top_k, int score, int renormalize, const uint8_t* w13, const uint8_t* w13_sf,
                    const float* alpha13, const uint8_t* w2, const uint8_t* w2_sf, const float* alpha2,
                    int64_t inter, void* out, int32_t* topk_ids, float* topk_weights, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    if (!x || !logits || !w13 || !w13_sf || !alpha13 || !w2 || !w2_sf || !alpha2 || !out || !topk_ids ||
        !topk_weights || !workspace)
        return NVFP4_NULL_POINTER;
    if (logits_dtype != NVFP4_BF16 && logits_dtype != NVFP4_F32) return NVFP4_BAD_DTYPE;
    if (!dim_ok(t) || !dim_ok(E) || !dim_ok(top_k) || top_k > E) return NVFP4_BAD_SHAPE;
    if (!dim_ok(h) || h % 16 != 0 || !dim_ok(inter) || inter % 16 != 0) return NVFP4_BAD_SHAPE;
    if (t > NVFP4_MOE_SMALL_MAX_TOKENS || E > NVFP4_MOE_SMALL_MAX_EXPERTS || top_k > NVFP4_MOE_SMALL_MAX_TOP_K)
        return NVFP4_UNSUPPORTED;
    if (score != NVFP4_ROUTE_SOFTMAX && score != NVFP4_ROUTE_SIGMOID) return NVFP4_UNSUPPORTED;
    // 32-bit offsets: one expert's weights (2 inter x h codes) and scales, the
    // tokens, the activations' two halves
    if (inter > (((int64_t)1 << 31) - 1) / h || t * h * 2 >= ((int64_t)1 << 31) ||
        t * top_k * inter * 4 >= ((int64_t)1 << 31) || !gemm_sf_ok(2 * inter, h / 16) || !gemm_sf_ok(h, inter / 16))
        return NVFP4_UNSUPPORTED;
    if (workspace_bytes < NVFP4_MOE_SMALL_WS_BYTES(t, top_k, h, inter)) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(logits) || !aligned16(w13) || !aligned16(w13_sf) || !aligned16(w2) ||
        !aligned16(w2_sf) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)alpha13 & 3u) ||
        ((uintptr_t)alpha2 & 3u) || ((uintptr_t)topk_ids & 3u) || ((uintptr_t)topk_weights & 3u))
        return NVFP4_MISALIGNED;
    nvfp4::MoeSmallArgs a{};
    a.x = (const uint16_t*)x; a.logits = logits; a.logits_bf16 = logits_dtype == NVFP4_BF16;
    a.sigmoid = score == NVFP4_ROUTE_SIGMOID; a.renorm = renormalize != 0;
    a.w13 = w13; a.w13_sf = w13_sf; a.alpha13 = alpha13;
    a.w2 = w2; a.w2_sf = w2_sf; a.alpha2 = alpha2;
    a.out = (uint16_t*)out; a.ids = topk_ids; a.weights = topk_weights; a.ws = workspace;
    a.t = (int)t; a.h = (int)h; a.inter = (int)inter; a.E = (int)E; a.top_k = (int)top_k;
    return launch_status(nvfp4::launch_moe_small(a, (hipStream_t)stream));
}

static_assert(nvfp4::kAdPartBytes == NVFP4_GEMM_WS_BYTES, "the workspace holds the partial sums");

// The adapters' own arguments, and the workspace that holds d.
static int adapters_check(const void* x, const void* lora_a, const void* lora_b, const int32_t* adapter,
                          const float* scaling, int64_t m, int64_t n, int64_t k, int64_t r, int64_t n_adapters,
                          const void* workspace, int64_t workspace_bytes) {
    if (!x || !lora_a || !lora_b || !adapter || !workspace) return NVFP4_NULL_POINTER;
    if (r < 8 || r % 8 != 0 || r > NVFP4_ADAPTERS_MAX_RANK) return NVFP4_BAD_RANK;
    if (!dim_ok(m) || !dim_ok(n) || !dim_ok(n_adapters) || k < 16 || k % 16 != 0 || k > kMaxDim)
        return NVFP4_BAD_SHAPE;
    // the grids hold that many: workgroups of 16 rows are taken for few tiles only
    if (m > (int64_t)1 << 20) return NVFP4_BAD_SHAPE;
    // 32-bit offsets into one adapter's B, and into 64 rows of x, A or the weight
    if (n * r >= (int64_t)1 << 32 || k > ((int64_t)1 << 23)) return NVFP4_UNSUPPORTED;
    if (workspace_bytes < NVFP4_ADAPTERS_WS_BYTES(m, r)) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(lora_a) || !aligned16(lora_b) || !aligned16(workspace) ||
        ((uintptr_t)adapter & 3u) || ((uintptr_t)scaling & 3u))
        return NVFP4_MISALIGNED;
    return NVFP4_OK;
}

static nvfp4::AdapterArgs adapter_args(const void* x, const void* lora_a, const void* lora_b,
                                       const int32_t* adapter, const float* scaling, int64_t m, int64_t n,
                                       int64_t k, int64_t r, int64_t n_adapters, void* workspace) {
    nvfp4::AdapterArgs a{};
    a.x = (const uint16_t*)x; a.lora_a = (const uint16_t*)lora_a; a.lora_b = (const uint16_t*)lora_b;
    a.adapter = adapter; a.scaling = scaling; a.d = (float*)workspace;
    a.m = m; a.n = n; a.k = k; a.r = r; a.n_adapters = n_adapters;
    return a;
}

// The workspace: d, and, where it is large enough, the partial sums.
static void* adapter_parts(void* workspace, int64_t workspace_bytes, int64_t m, int64_t r) {
    const int64_t own = NVFP4_ADAPTERS_WS_BYTES(m, r);
    return workspace_bytes >= own + NVFP4_GEMM_WS_BYTES ? (char*)workspace + own : nullptr;
}

int nvfp4_linear_adapters(const void* x, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                          const void* lora_a, const void* lora_b, const int32_t* adapter, const float* scaling,
                          const void* bias, void* out, int64_t m, int64_t n, int64_t k, int64_t r,
                          int64_t n_adapters, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!b || !b_sf || !alpha || !out) return NVFP4_NULL_POINTER;
    const int st = adapters_check(x, lora_a, lora_b, adapter, scaling, m, n, k, r, n_adapters, workspace,
                                  workspace_bytes);
    if (st != NVFP4_OK) return st;
    if (!gemm_sf_ok(n, k / 16)) return NVFP4_UNSUPPORTED;
    if (!aligned16(b) || !aligned16(b_sf) || !aligned16(out) || ((uintptr_t)alpha & 3u) || (bias && !aligned16(bias)))
        return NVFP4_MISALIGNED;
    const nvfp4::AdapterArgs a = adapter_args(x, lora_a, lora_b, adapter, scaling, m, n, k, r, n_adapters, workspace);
    const hipError_t e = nvfp4::launch_adapter_down(a, (hipStream_t)stream);
    if (e != hipSuccess) return launch_status(e);
    return launch_status(nvfp4::launch_w4a16_adapters(a, b, b_sf, alpha, (const uint16_t*)bias, (uint16_t*)out,
                                                      (float*)adapter_parts(workspace, workspace_bytes, m, r),
                                                      (hipStream_t)stream));
}

int nvfp4_gemm_adapters(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                        const float* alpha, const void* x, const void* lora_a, const void* lora_b,
                        const int32_t* adapter, const float* scaling, const void* bias, void* out, int64_t m,
                        int64_t n, int64_t k, int64_t r, int64_t n_adapters, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    int st = adapters_check(x, lora_a, lora_b, adapter, scaling, m, n, k, r, n_adapters, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    void* const part = adapter_parts(workspace, workspace_bytes, m, r);  // the split-tail schedule's partial tiles
    nvfp4::GemmArgs g{};
    st = gemm_check(a, b, a_sf, b_sf, alpha, nullptr, bias, nullptr, nullptr, out, 1, m, n, k, 0, part,
                    NVFP4_GEMM_WS_BYTES, g);
    if (st != NVFP4_OK) return st;
    const nvfp4::AdapterArgs ad = adapter_args(x, lora_a, lora_b, adapter, scaling, m, n, k, r, n_adapters, workspace);
    const hipError_t e = nvfp4::launch_adapter_down(ad, (hipStream_t)stream);
    if (e != hipSuccess) return launch_status(e);
    g.r = r; g.ad_d = ad.d; g.ad_b = ad.lora_b; g.adapter = adapter; g.n_adapters = n_adapters;
    return launch_status(nvfp4::launch_gemm(g, (hipStream_t)stream));
}

static_assert(nvfp4::kRopeAxes == NVFP4_ROPE_MAX_AXES && 2 * nvfp4::kAttnPartsNarrow == NVFP4_ATTENTION_MAX_SLOTS,
              "the header's limits are the kernels'");

// Rows of heads [t, heads, d] with a stride from token to token, in elements.
static bool rows_ok(int64_t t, int64_t heads, int64_t d, int64_t stride) {
    return dim_ok(t) && dim_ok(heads) && dim_ok(d) && heads * d <= NVFP4_ATTENTION_MAX_STRIDE && stride >= heads * d &&
           stride <= NVFP4_ATTENTION_MAX_STRIDE && stride % 8 == 0;
}

int rope_axes(const void* x, int64_t x_stride, void* out, int64_t out_stride, int64_t t, int64_t heads, int64_t d,
              const int32_t* positions, const float* inv_freq, const int32_t* sections, int axes, int interleaved,
              void* stream) {
    if (!x || !out || !positions || !inv_freq || !sections) return NVFP4_NULL_POINTER;
    if (!rows_ok(t, heads, d, x_stride) || !rows_ok(t, heads, d, out_stride) || d % 16 != 0) return NVFP4_BAD_SHAPE;
    if (axes < 1) return NVFP4_BAD_SHAPE;
    if (axes > NVFP4_ROPE_MAX_AXES || d > NVFP4_ROPE_MAX_DIM) return NVFP4_UNSUPPORTED;
    if (t * heads > ((int64_t)1 << 36) / d) return NVFP4_UNSUPPORTED;  // the grid: at most a thread per 32 elements
    nvfp4::RopeArgs a{};
    int64_t pairs = 0;
    for (int i = 0; i < axes; i++) {
        if (sections[i] < 0) return NVFP4_BAD_SHAPE;
        a.sections[i] = sections[i];
        pairs += sections[i];
    }
    if (pairs < 2 || pairs % 2 != 0 || 2 * pairs > d) return NVFP4_BAD_SHAPE;
    if (!aligned16(x) || !aligned16(out) || ((uintptr_t)positions & 3u) || ((uintptr_t)inv_freq & 3u))
        return NVFP4_MISALIGNED;
    a.x = (const uint16_t*)x; a.out = (uint16_t*)out; a.positions = positions; a.inv_freq = inv_freq;
    a.t = t; a.heads = heads; a.d = d; a.rot = 2 * pairs; a.x_stride = x_stride; a.out_stride = out_stride;
    a.axes = axes; a.interleaved = interleaved != 0;
    return launch_status(nvfp4::launch_rope_axes(a, (hipStream_t)stream));
}

// The cache's own sizes.
static int cache_check(int64_t heads, int64_t d, int64_t pages, int64_t page) {
    if (!dim_ok(heads) || !dim_ok(pages) || d < 16 || d % 16 != 0) return NVFP4_BAD_SHAPE;
    if (page < 16 || (page & (page - 1)) != 0) return NVFP4_BAD_SHAPE;
    if (d > NVFP4_KV_MAX_DIM || page > NVFP4_KV_MAX_PAGE || heads * d > NVFP4_ATTENTION_MAX_STRIDE) return NVFP4_UNSUPPORTED;
    return NVFP4_OK;
}

static int kv_rows(bool read, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t t,
                   int64_t heads, int64_t d, const int32_t* slots, const float* kv_gs, uint8_t* kv, uint8_t* kv_sf,
                   int64_t pages, int64_t page, void* stream) {
    if (!k || !v || !slots || !kv_gs || !kv || !kv_sf) return NVFP4_NULL_POINTER;
    const int st = cache_check(heads, d, pages, page);
    if (st != NVFP4_OK) return st;
    if (!rows_ok(t, heads, d, k_stride) || !rows_ok(t, heads, d, v_stride)) return NVFP4_BAD_SHAPE;
    if (t * heads > ((int64_t)1 << 35) / d) return NVFP4_UNSUPPORTED;  // the grid: a thread per 16 elements of both
    if (!aligned16(k) || !aligned16(v) || !aligned16(kv) || !aligned16(kv_sf) || ((uintptr_t)slots & 3u) ||
        ((uintptr_t)kv_gs & 3u))
        return NVFP4_MISALIGNED;
    nvfp4::KvRowsArgs a{};
    a.read = read;
    a.k = (const uint16_t*)k; a.v = (const uint16_t*)v; a.k_out = (uint16_t*)k; a.v_out = (uint16_t*)v;
    a.slots = slots; a.kv_gs = kv_gs; a.kv = kv; a.kv_sf = kv_sf;
    a.t = t; a.heads = heads; a.d = d; a.pages = pages; a.page = page; a.k_stride = k_stride; a.v_stride = v_stride;
    return launch_status(nvfp4::launch_kv_rows(a, (hipStream_t)stream));
}

int nvfp4_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t t, int64_t heads,
                    int64_t d, const int32_t* slots, const float* kv_gs, uint8_t* kv, uint8_t* kv_sf, int64_t pages,
                    int64_t page, void* stream) {
    return kv_rows(false, k, k_stride, v, v_stride, t, heads, d, slots, kv_gs, kv, kv_sf, pages, page, stream);
}

int nvfp4_kv_read(const uint8_t* kv, const uint8_t* kv_sf, const float* kv_gs, int64_t pages, int64_t page,
                  const int32_t* slots, int64_t t, int64_t heads, int64_t d, void* k, int64_t k_stride, void* v,
                  int64_t v_stride, void* stream) {
    return kv_rows(true, k, k_stride, v, v_stride, t, heads, d, slots, kv_gs, (uint8_t*)kv, (uint8_t*)kv_sf, pages,
                   page, stream);
}

// (times log2(e) it is finite)
static bool scale_ok(float scale) { return scale > 0.0f && scale <= 2.0e38f; }

int nvfp4_attention_decode(const void* q, int64_t q_stride, int64_t b, int64_t t, int64_t q_heads, const uint8_t* kv,
                           const uint8_t* kv_sf, const float* kv_gs, int64_t heads, int64_t d, int64_t pages,
                           int64_t page, const int32_t* block_table, int64_t table_pages, const int32_t* lengths,
                           float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream) {
    if (!q || !kv || !kv_sf || !kv_gs || !block_table || !lengths || !out || !workspace) return NVFP4_NULL_POINTER;
    const int st = cache_check(heads, d, pages, page);
    if (st != NVFP4_OK) return st;
    if (!dim_ok(b) || !dim_ok(t) || !dim_ok(q_heads) || !dim_ok(table_pages) || q_heads % heads != 0)
        return NVFP4_BAD_SHAPE;
    if (q_stride < q_heads * d || q_stride % 8 != 0 || q_stride > NVFP4_ATTENTION_MAX_STRIDE) return NVFP4_BAD_SHAPE;
    if (!scale_ok(scale) || b > NVFP4_ATTENTION_MAX_BATCH || t > NVFP4_ATTENTION_MAX_TOKENS ||
        q_heads * d > NVFP4_ATTENTION_MAX_STRIDE || table_pages > (((int64_t)1 << 30) / page))
        return NVFP4_UNSUPPORTED;
    if (b * t * q_heads > (int64_t)1 << 23) return NVFP4_UNSUPPORTED;  // the grids: below 2^32 threads
    if (workspace_bytes < NVFP4_ATTENTION_WS_BYTES(b, d)) return NVFP4_BAD_SHAPE;
    if (!aligned16(q) || !aligned16(kv) || !aligned16(kv_sf) || !aligned16(out) || !aligned16(workspace) ||
        ((uintptr_t)kv_gs & 3u) || ((uintptr_t)block_table & 3u) || ((uintptr_t)lengths & 3u) || ((uintptr_t)lse & 3u))
        return NVFP4_MISALIGNED;
    nvfp4::AttnDecodeArgs a{};
    a.q = (const uint16_t*)q; a.kv = kv; a.kv_sf = kv_sf; a.kv_gs = kv_gs; a.block_table = block_table;
    a.lengths = lengths; a.out = (uint16_t*)out; a.lse = lse; a.ws = workspace;
    a.b = b; a.t = t; a.q_heads = q_heads; a.heads = heads; a.d = d; a.pages = pages; a.page = page;
    a.table_pages = table_pages; a.q_stride = q_stride; a.scale = scale;
    return launch_status(nvfp4::launch_attention_decode(a, (hipStream_t)stream));
}

int attention_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, int64_t tq, int64_t tk, int64_t q_heads, int64_t heads, int64_t d,
                      const int32_t* cu_q, const int32_t* cu_k, int64_t b, float scale, int causal, void* out,
                      int64_t out_stride, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!q || !k || !v || !cu_q || !cu_k || !out) return NVFP4_NULL_POINTER;
    if (d < 16 || d % 16 != 0 || !rows_ok(tq, q_heads, d, q_stride) || !rows_ok(tk, heads, d, k_stride) ||
        !rows_ok(tk, heads, d, v_stride) || !rows_ok(tq, q_heads, d, out_stride) || !dim_ok(b) || q_heads % heads != 0)
        return NVFP4_BAD_SHAPE;
    if (!scale_ok(scale) || d > NVFP4_KV_MAX_DIM || b > NVFP4_ATTENTION_MAX_BATCH ||
        (tq / 128 + b) * q_heads >= (int64_t)1 << 23)  // the grid: below 2^32 threads
        return NVFP4_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace) ||
        ((uintptr_t)cu_q & 3u) || ((uintptr_t)cu_k & 3u) || ((uintptr_t)lse & 3u))
        return NVFP4_MISALIGNED;
    if (workspace) {
        const int64_t parts = nvfp4::prefill_parts(tq, tk, q_heads, heads, b);
        if (parts > 1 && workspace_bytes < parts * tq * q_heads * ((d <= 64 ? 64 : d <= 128 ? 128 : 256) + 4) * 4)
            return NVFP4_BAD_SHAPE;
    }
    nvfp4::AttnPrefillArgs a{};
    a.q = (const uint16_t*)q; a.k = (const uint16_t*)k; a.v = (const uint16_t*)v; a.out = (uint16_t*)out; a.lse = lse;
    a.ws = workspace; a.cu_q = cu_q; a.cu_k = cu_k; a.b = b; a.tq = tq; a.tk = tk; a.q_heads = q_heads; a.heads = heads; a.d = d;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.out_stride = out_stride;
    a.scale = scale; a.causal = causal != 0;
    return launch_status(nvfp4::launch_attention_prefill(a, (hipStream_t)stream));
}

}  // extern "C"
