// Host-side launchers of the row operators (internal to the library).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct RmsNormArgs {
  const __nv_bfloat16* x;
  long long ldx;
  const __nv_bfloat16* residual;  // or NULL
  long long ldr;
  __nv_bfloat16* residual_out;    // with residual; may be the same rows
  long long ldo;
  const __nv_bfloat16* weight;    // [H]
  __nv_bfloat16* y;               // or NULL
  long long ldy;
  uint8_t* codes;                 // or NULL: E4M3 [T, H]
  float* scales;                  // with codes: [ceil(H / 128), T]
  float* rstd;                    // or NULL: [T]
  float eps;
  int T, H;
};

struct RmsNormBackwardArgs {
  const __nv_bfloat16* dy;
  long long lddy;
  const __nv_bfloat16* s;         // the rows that were normalised
  long long lds;
  const __nv_bfloat16* weight;
  const float* rstd;
  const __nv_bfloat16* dresidual; // or NULL
  long long ldres;
  __nv_bfloat16* dx;
  long long lddx;
  float* partials;                // [blocks, H]
  int T, H;
};

constexpr int kMaxNormH = 16384;

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream);

// blocks of the backward kernel (each leaves one row of weight-gradient partial sums)
int rms_norm_backward_blocks(int T, int H);
cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, float* dweight, int blocks, cudaStream_t stream);

cudaError_t launch_quantize_rows(const void* x, long long ldx, long long rows, int cols, uint8_t* codes,
                                 float* scales, cudaStream_t stream);
cudaError_t launch_dequantize_rows(const uint8_t* codes, const float* scales, long long rows, int cols, void* x,
                                   long long ldx, cudaStream_t stream);

}  // namespace moe
