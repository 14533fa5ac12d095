// Host-side launchers of the grouped matrix products (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// which of the three products of y[r] = x[r] . w[group(r)]^T runs
enum GroupedKind {
  kGroupedFwd = 0,  // y  [M, N]    = x  [M, K] . w[g]^T
  kGroupedDx = 1,   // dx [M, K]    = dy [M, N] . w[g]
  kGroupedDw = 2,   // dw [G, N, K] = dy_g^T . x_g
};

struct GroupedProblem {
  int kind;
  bool fp8;                // kGroupedFwd only: E4M3 codes with block scales
  int M, G, N, K;
  const int32_t* offsets;  // [G + 1] on the device, or NULL: one group of all M rows
  const void* a;           // x (fwd), dy (dx, dw)
  long long lda;           // elements between its rows
  const void* b;           // w (fwd, dx), x (dw)
  long long ldb;           // dw: elements between the rows of x
  const float* a_scale;    // fp8: [ceil(K / 128), M]
  const float* b_scale;    // fp8: [G, ceil(N / 128), ceil(K / 128)]
  void* out;
  long long ldo;           // fwd, dx: elements between the rows of out
  bool out_f32;            // else bf16
  bool accumulate;         // dw with out_f32: add to out
  int* status;             // device status word
  int num_sms;
};

cudaError_t launch_grouped(const GroupedProblem& p, cudaStream_t stream);
cudaError_t launch_grouped_fp8(const GroupedProblem& p, cudaStream_t stream);
// split: two pairs share a tile's K blocks; as many such clusters as fp8_pair_split_clusters says are resident at once
cudaError_t launch_grouped_fp8_pair(const GroupedProblem& p, bool split, cudaStream_t stream);
cudaError_t fp8_pair_split_clusters(int* count);

}  // namespace moe
