// Row operators in front of the FP8 products: the RMS norm with the
// residual's addition (bf16 and / or E4M3 output) and its backward pass, and
// the E4M3 row format by itself (quantise, read back).
//
//   forward : s = bf16(x + residual) (or x), r = 1 / sqrt(mean(s^2) + eps),
//             y = bf16(s * r * w), and per (row, 128 columns) of y the
//             power-of-two scale and E4M3 codes of the layer's own rule.
//   backward: n = s * r, a = dy * w:
//             dx = r * (a - n * mean(a * n)) + dresidual, dw = sum_t dy * n.
//
// The norm is taken of the stored (bf16) sum, so the backward pass, which
// reads that sum, differentiates the function that ran.  Codes are those of
// the rounded y, so they equal what quantising y afterwards would give.  All
// sums are fp32.  Everything here is bound by HBM: one pass, the row stays in
// registers between the sum and the output, 16 bytes per access.
#include "common.cuh"
#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kMaxRowThreads = 1024;
constexpr int kMaxBackwardBlocks = 296;  // two per SM; fixed, so that the workspace does not depend on the device

struct alignas(16) bf16x8 {
  __nv_bfloat162 h[4];
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const bf16x8 b = *reinterpret_cast<const bf16x8*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(b.h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  bf16x8 b;
#pragma unroll
  for (int i = 0; i < 4; ++i) b.h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return *reinterpret_cast<const uint4*>(&b);
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the `warps` warps of a block that share a row (all of them): one
// barrier per call, `buf` alternates between two slots so that a following
// call may start before every thread has read this one's.
__device__ __forceinline__ float block_sum(float v, int warps, float* buf) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

// Scale and E4M3 codes of the 128-column group that this thread's half-warp
// holds, 8 columns each (columns past the row's end are zeros).  The scale
// is that of the finite values; a value that is not finite becomes the NaN
// code (E4M3 has no infinity, and saturating would hide it).
__device__ __forceinline__ uint2 quantize8(const float (&f)[8], float* scale_out) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(f[i]);
    amax = fmaxf(amax, a <= 3.402823466e38f ? a : 0.f);  // false for NaN and infinity
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = act_scale_from_amax(amax);
  const float inv = pow2_recip(scale);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fabsf(f[i]) <= 3.402823466e38f ? f[i] * inv : __int_as_float(0x7fc00000);
  uint2 c;
  c.x = static_cast<uint32_t>(f32x2_to_e4m3x2(q[0], q[1])) | (static_cast<uint32_t>(f32x2_to_e4m3x2(q[2], q[3])) << 16);
  c.y = static_cast<uint32_t>(f32x2_to_e4m3x2(q[4], q[5])) | (static_cast<uint32_t>(f32x2_to_e4m3x2(q[6], q[7])) << 16);
  *scale_out = scale;
  return c;
}

// ----------------------------------------------------------------------------
// forward: blockDim.x threads per row (a multiple of 32), V vectors of 8
// columns each; blockDim.y rows per block when one warp covers a row.
// ----------------------------------------------------------------------------
template <int V>
__global__ void __launch_bounds__(kMaxRowThreads) rms_norm_kernel(const RmsNormArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sums[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= a.T) return;  // whole warps: blockDim.x is a multiple of 32, blockDim.y > 1 only with one warp per row
  const int vecs = a.H / 8;
  const __nv_bfloat16* xr = a.x + row * a.ldx;
  uint4 u[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    u[i] = make_uint4(0, 0, 0, 0);
    w[i] = make_uint4(0, 0, 0, 0);
    if (v < vecs) u[i] = ld16(xr + 8 * v);
  }
  if (a.residual) {
    const __nv_bfloat16* rr = a.residual + row * a.ldr;
    __nv_bfloat16* so = a.residual_out + row * a.ldo;
    uint4 r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      r[i] = make_uint4(0, 0, 0, 0);
      if (v < vecs) r[i] = ld16(rr + 8 * v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      float f[8], g[8];
      unpack8(u[i], f);
      unpack8(r[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
      u[i] = pack8(f);  // the sum is rounded to bf16 once, as it is stored
      if (v < vecs) *reinterpret_cast<uint4*>(so + 8 * v) = u[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < vecs) w[i] = ld16(a.weight + 8 * v);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    unpack8(u[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
  }
  ss = block_sum(ss, blockDim.x >> 5, sums);
  // the exact square root and division: one of each per row
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    float f[8], g[8];
    unpack8(u[i], f);
    unpack8(w[i], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * g[j];
    const uint4 y = pack8(f);
    if (a.y && v < vecs) *reinterpret_cast<uint4*>(a.y + row * a.ldy + 8 * v) = y;
    if (a.codes) {
      unpack8(y, f);
      float scale;
      const uint2 c = quantize8(f, &scale);
      if (v < vecs) {
        *reinterpret_cast<uint2*>(a.codes + row * a.H + 8 * v) = c;
        if ((v & 15) == 0) a.scales[static_cast<long long>(v >> 4) * a.T + row] = scale;
      }
    }
  }
}

// ----------------------------------------------------------------------------
// backward: a block walks rows (grid stride) and keeps its columns' weight
// gradient in registers; each block writes one row of partial sums, which the
// second kernel adds in block order, so the result does not depend on timing.
// ----------------------------------------------------------------------------
template <int V, bool kRes>
__global__ void __launch_bounds__(kMaxRowThreads) rms_norm_backward_kernel(const RmsNormBackwardArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sums[2][32];
  const int vecs = a.H / 8;
  const int warps = blockDim.x >> 5;
  float acc[V][8];
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    w[i] = make_uint4(0, 0, 0, 0);
    if (v < vecs) w[i] = ld16(a.weight + 8 * v);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  uint4 d[V], s[V], r[V];
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      d[i] = s[i] = r[i] = make_uint4(0, 0, 0, 0);
      if (v < vecs) {
        d[i] = ld16(a.dy + row * a.lddy + 8 * v);
        s[i] = ld16(a.s + row * a.lds + 8 * v);
        if constexpr (kRes) r[i] = ld16(a.dresidual + row * a.ldres + 8 * v);
      }
    }
  };
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int buf = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    load(row);
    const float rstd = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float df[8], sf[8], wf[8];
      unpack8(d[i], df);
      unpack8(s[i], sf);
      unpack8(w[i], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = sf[j] * rstd;
        acc[i][j] = fmaf(df[j], n, acc[i][j]);
        dot = fmaf(df[j] * wf[j], n, dot);
      }
    }
    const float c = block_sum(dot, warps, sums[buf]) * inv_h;
    buf ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      float df[8], sf[8], wf[8], rf[8];
      unpack8(d[i], df);
      unpack8(s[i], sf);
      unpack8(w[i], wf);
      unpack8(r[i], rf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = sf[j] * rstd;
        const float g = rstd * fmaf(-n, c, df[j] * wf[j]);
        df[j] = kRes ? g + rf[j] : g;
      }
      if (v < vecs) *reinterpret_cast<uint4*>(a.dx + row * a.lddx + 8 * v) = pack8(df);
    }
  }
  float* part = a.partials + static_cast<long long>(blockIdx.x) * a.H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < vecs) {
      float4* p = reinterpret_cast<float4*>(part + 8 * v);
      p[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      p[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// dweight[h] = sum over the partial rows: 32 columns per block, 32 row strides, then a fixed tree
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partials, int rows, int H, float* out) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float part[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (col < H)
    for (int r = threadIdx.y; r < rows; r += 32) v += partials[static_cast<long long>(r) * H + col];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  const float s = warp_sum(part[threadIdx.x][threadIdx.y]);  // column threadIdx.y of the block
  const int c = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < H) out[c] = s;
}

// ----------------------------------------------------------------------------
// the row format by itself: a half-warp quantises one 128-column group
// ----------------------------------------------------------------------------
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __nv_bfloat16* x, long long ldx, long long rows,
                                                            int cols, uint8_t* codes, float* scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int groups = (cols + 127) / 128;
  const long long items = rows * groups;
  const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
  const bool in = item < items;  // uniform over a half-warp; all lanes take part in the shuffles
  const long long row = in ? item / groups : 0;
  const int g = in ? static_cast<int>(item - row * groups) : 0;
  const int col = g * 128 + (threadIdx.x & 15) * 8;
  const bool live = in && col < cols;
  uint4 u = make_uint4(0, 0, 0, 0);
  if (live) u = ld16(x + row * ldx + col);
  float f[8];
  unpack8(u, f);
  float scale;
  const uint2 c = quantize8(f, &scale);
  if (live) *reinterpret_cast<uint2*>(codes + row * cols + col) = c;
  if (in && (threadIdx.x & 15) == 0) scales[static_cast<long long>(g) * rows + row] = scale;
}

// 16 codes per thread; the scale is a power of two, so bf16 holds the value exactly (subnormals of
// bf16 aside, which the scale's floor of 2^-42 keeps out of reach)
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const uint8_t* codes, const float* scales,
                                                              long long rows, int cols, __nv_bfloat16* x,
                                                              long long ldx) {
  pdl_launch_dependents();
  pdl_wait();
  const int per_row = cols / 16;
  const long long item = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (item >= rows * per_row) return;
  const long long row = item / per_row;
  const int col = static_cast<int>(item - row * per_row) * 16;
  const uint4 u = *reinterpret_cast<const uint4*>(codes + row * cols + col);
  const float s = scales[static_cast<long long>(col >> 7) * rows + row];
  const uint32_t words[4] = {u.x, u.y, u.z, u.w};
  uint4 out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      __nv_fp8x4_e4m3 q;
      q.__x = words[2 * h + j];
      const float4 v = static_cast<float4>(q);
      f[4 * j] = v.x * s;
      f[4 * j + 1] = v.y * s;
      f[4 * j + 2] = v.z * s;
      f[4 * j + 3] = v.w * s;
    }
    out[h] = pack8(f);
  }
  uint4* dst = reinterpret_cast<uint4*>(x + row * ldx + col);
  dst[0] = out[0];
  dst[1] = out[1];
}

// threads per row: the row's vectors over V per thread, whole warps
int row_threads(int vecs, int v) { return ((vecs + v - 1) / v + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream) {
  const int vecs = a.H / 8;
  const int v = vecs > 1024 ? 2 : 1;
  const int tx = row_threads(vecs, v);
  const int ty = tx == 32 ? 8 : 1;
  const dim3 block(tx, ty);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + ty - 1) / ty);
  if (v == 1) return launch_pdl(rms_norm_kernel<1>, dim3(grid), block, 0, stream, a);
  return launch_pdl(rms_norm_kernel<2>, dim3(grid), block, 0, stream, a);
}

int rms_norm_backward_blocks(int T) { return T < kMaxBackwardBlocks ? T : kMaxBackwardBlocks; }

cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, float* dweight, int blocks, cudaStream_t stream) {
  const int vecs = a.H / 8;
  const int v = vecs > 1024 ? 2 : 1;
  const int tx = row_threads(vecs, v);
  cudaError_t e;
  if (a.dresidual)
    e = v == 1 ? launch_pdl(rms_norm_backward_kernel<1, true>, dim3(blocks), dim3(tx), 0, stream, a)
               : launch_pdl(rms_norm_backward_kernel<2, true>, dim3(blocks), dim3(tx), 0, stream, a);
  else
    e = v == 1 ? launch_pdl(rms_norm_backward_kernel<1, false>, dim3(blocks), dim3(tx), 0, stream, a)
               : launch_pdl(rms_norm_backward_kernel<2, false>, dim3(blocks), dim3(tx), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(column_sum_kernel, dim3((a.H + 31) / 32), dim3(32, 32), 0, stream,
                    static_cast<const float*>(a.partials), blocks, a.H, dweight);
}

cudaError_t launch_quantize_rows(const void* x, long long ldx, long long rows, int cols, uint8_t* codes,
                                 float* scales, cudaStream_t stream) {
  const long long threads = rows * ((cols + 127) / 128) * 16;
  return launch_pdl(quantize_rows_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, stream,
                    static_cast<const __nv_bfloat16*>(x), ldx, rows, cols, codes, scales);
}

cudaError_t launch_dequantize_rows(const uint8_t* codes, const float* scales, long long rows, int cols, void* x,
                                   long long ldx, cudaStream_t stream) {
  const long long threads = rows * (cols / 16);
  return launch_pdl(dequantize_rows_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, stream,
                    codes, scales, rows, cols, static_cast<__nv_bfloat16*>(x), ldx);
}

}  // namespace moe
