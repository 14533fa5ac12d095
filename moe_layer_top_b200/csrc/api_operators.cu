// C ABI of the stand-alone operators: the RMS norm, the E4M3 row format and
// the (grouped) matrix products.  Every argument is checked before anything
// is enqueued.
#include <math.h>

#include "api_internal.h"
#include "grouped.h"
#include "moe_b200.h"
#include "rows.h"

namespace {

using moe::api_fail;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_result(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();  // reported here; not left behind for another caller's check
  return api_fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A [rows, cols] tensor of `elem`-byte elements with `ld` elements between rows: 16-byte aligned rows.
int check_rows(const char* what, const char* name, const void* p, int64_t ld, int64_t cols, int elem) {
  if (!p) return api_fail(MOE_ERR_INVALID, "%s: %s is NULL", what, name);
  if (!aligned(p, 16)) return api_fail(MOE_ERR_INVALID, "%s: %s is not 16-byte aligned", what, name);
  if (ld < cols || (ld * elem) % 16 || ld > (int64_t(1) << 38))
    return api_fail(MOE_ERR_INVALID, "%s: row stride %lld of %s (at least %lld columns, a multiple of 16 bytes)", what,
                    static_cast<long long>(ld), name, static_cast<long long>(cols));
  return MOE_OK;
}

#define MOE_TRY(call)                \
  do {                               \
    const int rc_ = (call);          \
    if (rc_ != MOE_OK) return rc_;   \
  } while (0)

int check_norm_shape(const char* what, int32_t T, int32_t H) {
  if (T < 0) return api_fail(MOE_ERR_INVALID, "%s: T = %d < 0", what, T);
  if (H <= 0 || H % 8 || H > moe::kMaxNormH)
    return api_fail(MOE_ERR_INVALID, "%s: H = %d is not a multiple of 8 in [8, %d]", what, H, moe::kMaxNormH);
  return MOE_OK;
}

// Sizes common to the matrix products.  (The kernels round positions up to their tiles in 32 bits: hence 2^30.)
int check_product(const char* what, int32_t M, int32_t G, int32_t N, int32_t K, bool fp8, const int32_t* offsets,
                  const int32_t* status) {
  constexpr int32_t kMost = 1 << 30;
  if (M < 0) return api_fail(MOE_ERR_INVALID, "%s: M = %d < 0", what, M);
  if (M > kMost || N > kMost || K > kMost)
    return api_fail(MOE_ERR_INVALID, "%s: M = %d, N = %d or K = %d above 2^30", what, M, N, K);
  if (G < 1 || G > 1024) return api_fail(MOE_ERR_INVALID, "%s: G = %d outside [1, 1024]", what, G);
  if (N <= 0 || N % 8) return api_fail(MOE_ERR_INVALID, "%s: N = %d is not a positive multiple of 8", what, N);
  if (K <= 0 || K % (fp8 ? 16 : 8))
    return api_fail(MOE_ERR_INVALID, "%s: K = %d is not a positive multiple of %d", what, K, fp8 ? 16 : 8);
  if (!offsets && G != 1) return api_fail(MOE_ERR_INVALID, "%s: offsets may be NULL for one group only (G = %d)", what, G);
  if (!aligned(offsets, 4)) return api_fail(MOE_ERR_INVALID, "%s: offsets is not 4-byte aligned", what);
  if (!aligned(status, 4)) return api_fail(MOE_ERR_INVALID, "%s: status is not 4-byte aligned", what);
  const int64_t tiles = (static_cast<int64_t>(M) / 128 + G) * ((static_cast<int64_t>(N > K ? N : K) + 127) / 128);
  const int64_t dw_tiles = static_cast<int64_t>(G) * ((N + 127) / 128) * ((K + 127) / 128);
  if (tiles >= (int64_t(1) << 30) || dw_tiles >= (int64_t(1) << 30))
    return api_fail(MOE_ERR_INVALID, "%s: more than 2^30 tiles (M = %d, G = %d, N = %d, K = %d)", what, M, G, N, K);
  return MOE_OK;
}

int check_out_dtype(const char* what, int32_t dtype) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32)
    return api_fail(MOE_ERR_UNSUPPORTED, "%s: out_dtype %d (MOE_DTYPE_BF16 or MOE_DTYPE_FP32)", what, dtype);
  return MOE_OK;
}

int run_product(moe::GroupedProblem& p, const char* what, void* stream) {
  MOE_TRY(moe::api_device_check(&p.num_sms));
  if (!p.status) {
    const cudaError_t e = moe::operator_status_word(&p.status);
    if (e != cudaSuccess) return cuda_result(e, what);
  }
  return cuda_result(moe::launch_grouped(p, static_cast<cudaStream_t>(stream)), what);
}

int matmul_fp8(const char* what, const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
               const int32_t* offsets, int32_t M, int32_t G, int32_t N, int32_t K, void* y, int64_t ldy,
               int32_t out_dtype, int32_t* status, void* stream) {
  MOE_TRY(check_product(what, M, G, N, K, true, offsets, status));
  MOE_TRY(check_out_dtype(what, out_dtype));
  if (M == 0) return MOE_OK;
  const int out_bytes = out_dtype == MOE_DTYPE_FP32 ? 4 : 2;
  MOE_TRY(check_rows(what, "x", x, K, K, 1));
  MOE_TRY(check_rows(what, "w", w, K, K, 1));
  MOE_TRY(check_rows(what, "y", y, ldy, N, out_bytes));
  if (!x_scale || !w_scale || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return api_fail(MOE_ERR_INVALID, "%s: x_scale and w_scale are required, 4-byte aligned", what);
  moe::GroupedProblem p{};
  p.kind = moe::kGroupedFwd;
  p.fp8 = true;
  p.M = M, p.G = G, p.N = N, p.K = K;
  p.offsets = offsets;
  p.a = x, p.lda = K;
  p.b = w;
  p.a_scale = x_scale, p.b_scale = w_scale;
  p.out = y, p.ldo = ldy;
  p.out_f32 = out_dtype == MOE_DTYPE_FP32;
  p.status = status;
  return run_product(p, what, stream);
}

}  // namespace

extern "C" {

int moe_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* residual_out, int64_t ldo,
                 const void* weight, float eps, int32_t T, int32_t H, void* y, int64_t ldy, uint8_t* codes,
                 float* scales, float* rstd, void* stream) {
  const char* what = "rms_norm";
  MOE_TRY(check_norm_shape(what, T, H));
  if (!(eps >= 0.0f) || eps == INFINITY) return api_fail(MOE_ERR_INVALID, "%s: eps must be finite and >= 0", what);
  if (T == 0) return MOE_OK;  // nothing to read or write; buffers of zero rows may be NULL
  if (!residual != !residual_out) return api_fail(MOE_ERR_INVALID, "%s: give residual and residual_out, or neither", what);
  if (!y && !codes && !residual && !rstd) return api_fail(MOE_ERR_INVALID, "%s: no output is asked for", what);
  if (!codes != !scales) return api_fail(MOE_ERR_INVALID, "%s: give codes and scales, or neither", what);
  if (codes && H % 16) return api_fail(MOE_ERR_INVALID, "%s: FP8 rows need H %% 16 == 0 (H = %d)", what, H);
  MOE_TRY(check_rows(what, "x", x, ldx, H, 2));
  MOE_TRY(check_rows(what, "weight", weight, H, H, 2));
  if (residual) {
    MOE_TRY(check_rows(what, "residual", residual, ldr, H, 2));
    MOE_TRY(check_rows(what, "residual_out", residual_out, ldo, H, 2));
  }
  if (y) MOE_TRY(check_rows(what, "y", y, ldy, H, 2));
  if (codes) MOE_TRY(check_rows(what, "codes", codes, H, H, 1));
  if (!aligned(scales, 4) || !aligned(rstd, 4))
    return api_fail(MOE_ERR_INVALID, "%s: scales and rstd must be 4-byte aligned", what);
  MOE_TRY(moe::api_device_check(nullptr));
  moe::RmsNormArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x), a.ldx = ldx;
  a.residual = static_cast<const __nv_bfloat16*>(residual), a.ldr = ldr;
  a.residual_out = static_cast<__nv_bfloat16*>(residual_out), a.ldo = ldo;
  a.weight = static_cast<const __nv_bfloat16*>(weight);
  a.y = static_cast<__nv_bfloat16*>(y), a.ldy = ldy;
  a.codes = codes, a.scales = scales, a.rstd = rstd;
  a.eps = eps, a.T = T, a.H = H;
  return cuda_result(moe::launch_rms_norm(a, static_cast<cudaStream_t>(stream)), what);
}

size_t moe_rms_norm_backward_workspace_size(int32_t T, int32_t H) {
  if (check_norm_shape("rms_norm_backward", T, H) != MOE_OK) return 0;
  return static_cast<size_t>(moe::rms_norm_backward_blocks(T, H)) * static_cast<size_t>(H) * sizeof(float);
}

int moe_rms_norm_backward(const void* dy, int64_t lddy, const void* s, int64_t lds, const void* weight,
                          const float* rstd, const void* dresidual, int64_t lddres, int32_t T, int32_t H, void* dx,
                          int64_t lddx, float* dweight, void* ws, size_t ws_bytes, void* stream) {
  const char* what = "rms_norm_backward";
  MOE_TRY(check_norm_shape(what, T, H));
  if (!dweight || !aligned(dweight, 4)) return api_fail(MOE_ERR_INVALID, "%s: dweight is required, 4-byte aligned", what);
  if (T > 0) {
    MOE_TRY(check_rows(what, "dy", dy, lddy, H, 2));
    MOE_TRY(check_rows(what, "s", s, lds, H, 2));
    MOE_TRY(check_rows(what, "weight", weight, H, H, 2));
    MOE_TRY(check_rows(what, "dx", dx, lddx, H, 2));
    if (dresidual) MOE_TRY(check_rows(what, "dresidual", dresidual, lddres, H, 2));
    if (!rstd || !aligned(rstd, 4)) return api_fail(MOE_ERR_INVALID, "%s: rstd is required, 4-byte aligned", what);
    if (!ws || !aligned(ws, 16)) return api_fail(MOE_ERR_INVALID, "%s: ws is required, 16-byte aligned", what);
  }
  const int blocks = moe::rms_norm_backward_blocks(T, H);
  const size_t need = static_cast<size_t>(blocks) * static_cast<size_t>(H) * sizeof(float);
  if (ws_bytes < need)
    return api_fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_bytes, need);
  MOE_TRY(moe::api_device_check(nullptr));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return cuda_result(cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * sizeof(float), st), what);
  moe::RmsNormBackwardArgs a{};
  a.dy = static_cast<const __nv_bfloat16*>(dy), a.lddy = lddy;
  a.s = static_cast<const __nv_bfloat16*>(s), a.lds = lds;
  a.weight = static_cast<const __nv_bfloat16*>(weight);
  a.rstd = rstd;
  a.dresidual = static_cast<const __nv_bfloat16*>(dresidual), a.ldres = lddres;
  a.dx = static_cast<__nv_bfloat16*>(dx), a.lddx = lddx;
  a.partials = static_cast<float*>(ws);
  a.T = T, a.H = H;
  return cuda_result(moe::launch_rms_norm_backward(a, dweight, blocks, st), what);
}

int moe_quantize_rows_fp8(const void* x, int64_t ldx, int64_t rows, int32_t cols, uint8_t* codes, float* scales,
                          void* stream) {
  const char* what = "quantize_rows_fp8";
  if (rows < 0 || rows >= (int64_t(1) << 31) || cols <= 0 || cols % 16 || cols > (1 << 20))
    return api_fail(MOE_ERR_INVALID, "%s: rows = %lld, cols = %d (cols a multiple of 16 up to 2^20)", what,
                    static_cast<long long>(rows), cols);
  if (rows * ((cols + 127) / 128) >= (int64_t(1) << 35))
    return api_fail(MOE_ERR_INVALID, "%s: more than 2^35 scale groups", what);
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_rows(what, "x", x, ldx, cols, 2));
  MOE_TRY(check_rows(what, "codes", codes, cols, cols, 1));
  if (!scales || !aligned(scales, 4)) return api_fail(MOE_ERR_INVALID, "%s: scales is required, 4-byte aligned", what);
  MOE_TRY(moe::api_device_check(nullptr));
  return cuda_result(moe::launch_quantize_rows(x, ldx, rows, cols, codes, scales, static_cast<cudaStream_t>(stream)),
                     what);
}

int moe_dequantize_rows_fp8(const uint8_t* codes, const float* scales, int64_t rows, int32_t cols, void* x,
                            int64_t ldx, void* stream) {
  const char* what = "dequantize_rows_fp8";
  if (rows < 0 || rows >= (int64_t(1) << 31) || cols <= 0 || cols % 16 || cols > (1 << 20))
    return api_fail(MOE_ERR_INVALID, "%s: rows = %lld, cols = %d (cols a multiple of 16 up to 2^20)", what,
                    static_cast<long long>(rows), cols);
  if (rows * ((cols + 127) / 128) >= (int64_t(1) << 35))
    return api_fail(MOE_ERR_INVALID, "%s: more than 2^35 scale groups", what);
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_rows(what, "x", x, ldx, cols, 2));
  MOE_TRY(check_rows(what, "codes", codes, cols, cols, 1));
  if (!scales || !aligned(scales, 4)) return api_fail(MOE_ERR_INVALID, "%s: scales is required, 4-byte aligned", what);
  MOE_TRY(moe::api_device_check(nullptr));
  return cuda_result(moe::launch_dequantize_rows(codes, scales, rows, cols, x, ldx, static_cast<cudaStream_t>(stream)),
                     what);
}

int moe_matmul_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale, int32_t M,
                   int32_t N, int32_t K, void* y, int64_t ldy, int32_t out_dtype, int32_t* status, void* stream) {
  return matmul_fp8("matmul_fp8", x, x_scale, w, w_scale, nullptr, M, 1, N, K, y, ldy, out_dtype, status, stream);
}

int moe_grouped_matmul_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                           const int32_t* offsets, int32_t M, int32_t G, int32_t N, int32_t K, void* y, int64_t ldy,
                           int32_t out_dtype, int32_t* status, void* stream) {
  return matmul_fp8("grouped_matmul_fp8", x, x_scale, w, w_scale, offsets, M, G, N, K, y, ldy, out_dtype, status,
                    stream);
}

int moe_grouped_matmul(const void* x, int64_t ldx, const void* w, const int32_t* offsets, int32_t M, int32_t G,
                       int32_t N, int32_t K, void* y, int64_t ldy, int32_t out_dtype, int32_t* status, void* stream) {
  const char* what = "grouped_matmul";
  MOE_TRY(check_product(what, M, G, N, K, false, offsets, status));
  MOE_TRY(check_out_dtype(what, out_dtype));
  if (M == 0) return MOE_OK;
  MOE_TRY(check_rows(what, "x", x, ldx, K, 2));
  MOE_TRY(check_rows(what, "w", w, K, K, 2));
  MOE_TRY(check_rows(what, "y", y, ldy, N, out_dtype == MOE_DTYPE_FP32 ? 4 : 2));
  moe::GroupedProblem p{};
  p.kind = moe::kGroupedFwd;
  p.M = M, p.G = G, p.N = N, p.K = K;
  p.offsets = offsets;
  p.a = x, p.lda = ldx;
  p.b = w;
  p.out = y, p.ldo = ldy;
  p.out_f32 = out_dtype == MOE_DTYPE_FP32;
  p.status = status;
  return run_product(p, what, stream);
}

int moe_grouped_matmul_dx(const void* dy, int64_t lddy, const void* w, const int32_t* offsets, int32_t M, int32_t G,
                          int32_t N, int32_t K, void* dx, int64_t lddx, int32_t out_dtype, int32_t* status,
                          void* stream) {
  const char* what = "grouped_matmul_dx";
  MOE_TRY(check_product(what, M, G, N, K, false, offsets, status));
  MOE_TRY(check_out_dtype(what, out_dtype));
  if (M == 0) return MOE_OK;
  MOE_TRY(check_rows(what, "dy", dy, lddy, N, 2));
  MOE_TRY(check_rows(what, "w", w, K, K, 2));
  MOE_TRY(check_rows(what, "dx", dx, lddx, K, out_dtype == MOE_DTYPE_FP32 ? 4 : 2));
  moe::GroupedProblem p{};
  p.kind = moe::kGroupedDx;
  p.M = M, p.G = G, p.N = N, p.K = K;
  p.offsets = offsets;
  p.a = dy, p.lda = lddy;
  p.b = w;
  p.out = dx, p.ldo = lddx;
  p.out_f32 = out_dtype == MOE_DTYPE_FP32;
  p.status = status;
  return run_product(p, what, stream);
}

int moe_grouped_matmul_dw(const void* dy, int64_t lddy, const void* x, int64_t ldx, const int32_t* offsets, int32_t M,
                          int32_t G, int32_t N, int32_t K, void* dw, int32_t out_dtype, int32_t accumulate,
                          int32_t* status, void* stream) {
  const char* what = "grouped_matmul_dw";
  MOE_TRY(check_product(what, M, G, N, K, false, offsets, status));
  MOE_TRY(check_out_dtype(what, out_dtype));
  if (accumulate != 0 && accumulate != 1) return api_fail(MOE_ERR_INVALID, "%s: accumulate must be 0 or 1", what);
  if (accumulate && out_dtype != MOE_DTYPE_FP32)
    return api_fail(MOE_ERR_UNSUPPORTED, "%s: only an fp32 gradient can be accumulated into", what);
  if (M > 0) {
    MOE_TRY(check_rows(what, "dy", dy, lddy, N, 2));
    MOE_TRY(check_rows(what, "x", x, ldx, K, 2));
  }
  MOE_TRY(check_rows(what, "dw", dw, K, K, out_dtype == MOE_DTYPE_FP32 ? 4 : 2));
  if (M == 0 && accumulate) return MOE_OK;
  moe::GroupedProblem p{};
  p.kind = moe::kGroupedDw;
  p.M = M, p.G = G, p.N = N, p.K = K;
  p.offsets = offsets;
  p.a = dy, p.lda = lddy;
  p.b = x, p.ldb = ldx;
  p.out = dw, p.ldo = K;
  p.out_f32 = out_dtype == MOE_DTYPE_FP32;
  p.accumulate = accumulate != 0;
  p.status = status;
  return run_product(p, what, stream);
}

}  // extern "C"
