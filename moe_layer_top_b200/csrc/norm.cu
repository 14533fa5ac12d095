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
// registers between the sum and the output, 16 bytes per access.  On a B200
// (6551 GB/s of copy): 8192 x 7168 with residual and FP8 output 63 us, 0.99 of
// the copy rate; backward of 16384 x 4096 with a residual gradient 86 us, 0.96;
// quantising 8192 x 7168 34 us, 0.79; reading it back 29 us, 0.94.  The
// backward pass of narrow rows is further off: 32768 x 512 24 us, 0.63.
#include "common.cuh"
#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kMaxRowThreads = 1024;

struct alignas(16) bf16x8 {
  __nv_bfloat162 h[4];
};

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  bf16x8 b;
#pragma unroll
  for (int i = 0; i < 4; ++i) b.h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return *reinterpret_cast<const uint4*>(&b);
}

// infinities -> the largest finite number of their sign
__device__ __forceinline__ uint4 finite8(const uint4& u) {
  bf16x8 b = *reinterpret_cast<const bf16x8*>(&u);
  const __nv_bfloat162 most = __bfloat162bfloat162(__ushort_as_bfloat16(0x7f7f));
#pragma unroll
  for (int i = 0; i < 4; ++i) b.h[i] = __hmax2_nan(__hmin2_nan(b.h[i], most), __hneg2(most));
  return *reinterpret_cast<const uint4*>(&b);
}

// Two fp32 lanes in one register pair: half the instructions of these kernels, which issue at 70 % of the peak rate
// (each lane is rounded as the scalar operation would be).
using f2 = unsigned long long;
__device__ __forceinline__ f2 both(float v) {
  f2 r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float2 halves(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
// a pair of bf16 numbers (the first in the low half) in fp32
__device__ __forceinline__ f2 widen(uint32_t u) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(u << 16), "r"(u & 0xffff0000u));
  return r;
}
__device__ __forceinline__ uint32_t narrow(f2 v) {
  const float2 t = halves(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(t.x, t.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// words of a 16-byte vector
struct alignas(16) Words {
  uint32_t u[4];
};
__device__ __forceinline__ Words words(const uint4& v) { return *reinterpret_cast<const Words*>(&v); }
__device__ __forceinline__ uint4 vec(const Words& w) { return *reinterpret_cast<const uint4*>(&w); }
// bf16(a + b), rounded once
__device__ __forceinline__ uint32_t add_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
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
// holds, 8 bf16 columns each (columns past the row's end are zeros).  Without
// their signs bf16 numbers compare as integers, infinity and NaN above the
// rest, so the largest is found two at a time without conversions; only a
// group whose largest is not finite looks again: the scale is that of the
// finite values, and a value that is not finite becomes the NaN code (E4M3 has
// no infinity, and saturating would hide it).
__device__ __forceinline__ uint2 quantize8(const uint4& u, float* scale_out) {
  constexpr uint32_t kAbs = 0x7fff7fffu, kInf = 0x7f80u;
  uint32_t m = __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  uint32_t top = max(m & 0xffffu, m >> 16);
  const bool odd = top >= kInf;  // the same on all lanes of the half-warp
  Words w = words(u);
  if (__any_sync(0xffffffffu, odd)) {
    uint32_t finite = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w.u[i] & 0x7fffu, hi = w.u[i] >> 16 & 0x7fffu;
      if (lo < kInf) finite = max(finite, lo);
      else w.u[i] |= 0x7fffu;
      if (hi < kInf) finite = max(finite, hi);
      else w.u[i] |= 0x7fff0000u;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) finite = max(finite, __shfl_xor_sync(0xffffffffu, finite, o));
    top = finite;
  }
  f2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = widen(w.u[i]);
  const float scale = act_scale_from_amax(__uint_as_float(top << 16));
  const float inv = pow2_recip(scale);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = halves(mul2(f[i], both(inv)));
    c[i] = f32x2_to_e4m3x2(q.x, q.y);
  }
  *scale_out = scale;
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// ----------------------------------------------------------------------------
// forward: blockDim.x threads per row (a multiple of 32), V vectors of 8
// columns each; blockDim.y rows per block when one warp covers a row.
// ----------------------------------------------------------------------------
template <int V>
__global__ void __launch_bounds__(V == 4 ? kMaxNormH / 32 : kMaxRowThreads) rms_norm_kernel(const RmsNormArgs a) {
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
      Words sum = words(u[i]);
      const Words add = words(r[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum.u[j] = add_bf16(sum.u[j], add.u[j]);  // rounded once, as it is stored
      u[i] = vec(sum);
      if (v < vecs) *reinterpret_cast<uint4*>(so + 8 * v) = u[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < vecs) w[i] = ld16(a.weight + 8 * v);
  }
  f2 squares = both(0.f);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const Words x = words(u[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) squares = fma2(widen(x.u[j]), widen(x.u[j]), squares);
  }
  const float ss = block_sum(halves(squares).x + halves(squares).y, blockDim.x >> 5, sums);
  // the exact square root and division: one of each per row
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    Words f = words(u[i]);
    const Words g = words(w[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.u[j] = narrow(mul2(mul2(widen(f.u[j]), both(rstd)), widen(g.u[j])));
    const uint4 y = vec(f);
    if (a.y && v < vecs) *reinterpret_cast<uint4*>(a.y + row * a.ldy + 8 * v) = y;
    if (a.codes) {
      float scale;
      const uint2 c = quantize8(y, &scale);
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
// The next row's loads are in flight while a row's sum is formed (V = 1).  Up to 512
// columns a warp holds a row by itself and 16 of them share a block (then the
// block adds their columns through shared memory first); otherwise the whole
// block holds one row.
// ----------------------------------------------------------------------------
template <int V, bool kRes>
__global__ void __launch_bounds__(kMaxRowThreads) rms_norm_backward_kernel(const RmsNormBackwardArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sums[2][32];
  extern __shared__ float columns[];  // blockDim.y > 1: [blockDim.y][H]
  const int vecs = a.H / 8;
  const int warps = blockDim.x >> 5;
  const long long first_row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  f2 acc[V][4];
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    w[i] = make_uint4(0, 0, 0, 0);
    if (v < vecs) w[i] = ld16(a.weight + 8 * v);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);
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
  constexpr bool kAhead = V == 1;  // with two vectors per thread the copies do not fit the registers
  float next_rstd = 0.f;
  if (kAhead && first_row < a.T) {
    load(first_row);
    next_rstd = a.rstd[first_row];
  }
  for (long long row = first_row; row < a.T; row += step) {
    if (!kAhead) {
      load(row);
      next_rstd = a.rstd[row];
    }
    const float rstd = next_rstd;
    f2 dots = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Words dw = words(d[i]), sw = words(s[i]), ww = words(w[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 g = widen(dw.u[j]), n = mul2(widen(sw.u[j]), both(rstd));
        acc[i][j] = fma2(g, n, acc[i][j]);
        dots = fma2(mul2(g, widen(ww.u[j])), n, dots);
      }
    }
    // the next row is under way while this one's sum is formed
    uint4 cd[V], cs[V], cr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      cd[i] = d[i];
      cs[i] = s[i];
      cr[i] = r[i];
    }
    if (kAhead && row + step < a.T) {
      load(row + step);
      next_rstd = a.rstd[row + step];
    }
    const float c = block_sum(halves(dots).x + halves(dots).y, warps, sums[buf]) * inv_h;
    buf ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      const Words dw = words(cd[i]), sw = words(cs[i]), ww = words(w[i]), rw = words(cr[i]);
      Words o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 n = mul2(widen(sw.u[j]), both(rstd));
        const f2 g = fma2(n, both(-c), mul2(widen(dw.u[j]), widen(ww.u[j])));
        o.u[j] = narrow(kRes ? fma2(g, both(rstd), widen(rw.u[j])) : mul2(g, both(rstd)));
      }
      if (v < vecs) *reinterpret_cast<uint4*>(a.dx + row * a.lddx + 8 * v) = vec(o);
    }
  }
  float* part = a.partials + static_cast<long long>(blockIdx.x) * a.H;
  if (blockDim.y > 1) part = columns + threadIdx.y * a.H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < vecs) {
      float4* p = reinterpret_cast<float4*>(part + 8 * v);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 lo = halves(acc[i][2 * j]), hi = halves(acc[i][2 * j + 1]);
        p[j] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
  if (blockDim.y > 1) {
    __syncthreads();
    const int threads = blockDim.x * blockDim.y;
    for (int h = threadIdx.y * blockDim.x + threadIdx.x; h < a.H; h += threads) {
      float v = 0.f;
      for (int y = 0; y < static_cast<int>(blockDim.y); ++y) v += columns[y * a.H + h];
      a.partials[static_cast<long long>(blockIdx.x) * a.H + h] = v;
    }
  }
}

// The same for wide rows, the next kStages - 1 rows under way: each thread copies its own vectors into shared memory
// (cp.async) and reads them back, so the copies need no registers and no barrier.
__device__ __forceinline__ void copy16(uint4* dst, const __nv_bfloat16* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <int V, int kStages, bool kRes>
__global__ void __launch_bounds__(kMaxRowThreads) rms_norm_backward_wide_kernel(const RmsNormBackwardArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sums[2][32];
  extern __shared__ uint4 ring[];  // [stage][dy, s, dresidual][vector of a thread][thread]
  constexpr int kTensors = kRes ? 3 : 2;
  const int vecs = a.H / 8;
  const int warps = blockDim.x >> 5;
  const long long step = gridDim.x;
  auto slot = [&](int stage, int tensor, int i) {
    return ring + (static_cast<size_t>(stage * kTensors + tensor) * V + i) * blockDim.x + threadIdx.x;
  };
  auto fetch = [&](long long row, int stage) {
    if (row < a.T) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v < vecs) {
          copy16(slot(stage, 0, i), a.dy + row * a.lddy + 8 * v);
          copy16(slot(stage, 1, i), a.s + row * a.lds + 8 * v);
          if constexpr (kRes) copy16(slot(stage, 2, i), a.dresidual + row * a.ldres + 8 * v);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  long long row = blockIdx.x;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(row + k * step, k);
  float next_rstd = row < a.T ? a.rstd[row] : 0.f;
  f2 acc[V][4];
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    w[i] = make_uint4(0, 0, 0, 0);
    if (v < vecs) w[i] = ld16(a.weight + 8 * v);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);
  }
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int buf = 0, stage = 0;
  for (; row < a.T; row += step) {
    const float rstd = next_rstd;
    if (row + step < a.T) next_rstd = a.rstd[row + step];
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    uint4 d[V], s[V];
    f2 dots = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = static_cast<int>(i * blockDim.x + threadIdx.x) < vecs;
      d[i] = in ? *slot(stage, 0, i) : make_uint4(0, 0, 0, 0);
      s[i] = in ? *slot(stage, 1, i) : make_uint4(0, 0, 0, 0);
      const Words dw = words(d[i]), sw = words(s[i]), ww = words(w[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 g = widen(dw.u[j]), n = mul2(widen(sw.u[j]), both(rstd));
        acc[i][j] = fma2(g, n, acc[i][j]);
        dots = fma2(mul2(g, widen(ww.u[j])), n, dots);
      }
    }
    // the stage that the previous row left
    fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    const float c = block_sum(halves(dots).x + halves(dots).y, warps, sums[buf]) * inv_h;
    buf ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v >= vecs) break;
      const Words dw = words(d[i]), sw = words(s[i]), ww = words(w[i]);
      Words rw{}, o;
      if constexpr (kRes) rw = words(*slot(stage, 2, i));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 n = mul2(widen(sw.u[j]), both(rstd));
        const f2 g = fma2(n, both(-c), mul2(widen(dw.u[j]), widen(ww.u[j])));
        o.u[j] = narrow(kRes ? fma2(g, both(rstd), widen(rw.u[j])) : mul2(g, both(rstd)));
      }
      *reinterpret_cast<uint4*>(a.dx + row * a.lddx + 8 * v) = vec(o);
    }
    if (++stage == kStages) stage = 0;
  }
  float* part = a.partials + static_cast<long long>(blockIdx.x) * a.H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < vecs) {
      float4* p = reinterpret_cast<float4*>(part + 8 * v);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 lo = halves(acc[i][2 * j]), hi = halves(acc[i][2 * j + 1]);
        p[j] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
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
template <int kItems>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __nv_bfloat16* x, long long ldx, long long rows,
                                                            int cols, int block_rows, uint8_t* codes, float* scales) {
  pdl_launch_dependents();
  pdl_wait();
  // a block takes kItems * 16 groups of `block_rows` rows, or of a part of one row (block_rows = 1)
  const int groups = (cols + 127) / 128;
  const int parts = (groups + kItems * 16 - 1) / (kItems * 16);  // blocks of a row
  const long long row0 = block_rows > 1 ? static_cast<long long>(blockIdx.x) * block_rows : blockIdx.x / parts;
  const int group0 = block_rows > 1 ? 0 : static_cast<int>(blockIdx.x % parts) * kItems * 16;
  const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
  long long row[kItems];
  int g[kItems];
  bool in[kItems];
  uint4 u[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int item = i * 16 + half;
    const int r = block_rows > 1 ? item / groups : 0;
    row[i] = row0 + r;
    g[i] = group0 + item - r * groups;
    in[i] = (block_rows == 1 || r < block_rows) && row[i] < rows && g[i] < groups;  // uniform over a half-warp
    u[i] = make_uint4(0, 0, 0, 0);
    if (in[i] && g[i] * 128 + 8 * l < cols) u[i] = ld16(x + row[i] * ldx + g[i] * 128 + 8 * l);
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    float scale;
    const uint2 c = quantize8(u[i], &scale);  // all lanes take part in the shuffles
    const int col = g[i] * 128 + 8 * l;
    if (in[i] && col < cols) *reinterpret_cast<uint2*>(codes + row[i] * cols + col) = c;
    if (in[i] && l == 0) scales[static_cast<long long>(g[i]) * rows + row[i]] = scale;
  }
}

// 16 codes per thread; the scale is a power of two, so bf16 holds the value exactly (subnormals of bf16 aside, which
// the scale's floor of 2^-42 keeps out of reach), but for one: from 248 * 2^120 on a row's largest number is rounded up
// to the code of 256 at a scale of 2^120, and 2^128 is past bf16.  What is past bf16's largest finite number is read
// back as that number, so that a finite row stays finite; NaN stays NaN.
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const uint8_t* codes, const float* scales,
                                                              long long rows, int cols, __nv_bfloat16* x,
                                                              long long ldx) {
  pdl_launch_dependents();
  pdl_wait();
  const int per_row = cols / 16;
  const long long item = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (item >= rows * per_row) return;
  // (a 64-bit division takes longer than the rest of the thread's work)
  const long long row = item < (1ll << 32) ? static_cast<uint32_t>(item) / static_cast<uint32_t>(per_row)
                                           : item / per_row;
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
    out[h] = finite8(pack8(f));
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
  // Few rows: a thread per vector, the shortest way through one row.  Many: up to four vectors per thread, so that
  // an SM has more rows in flight (T = 8192, H = 7168, residual and FP8 output: 88 us with one, 63 us with four).
  const int v = a.T <= 2 * 148 ? (vecs > 1024 ? 2 : 1) : (vecs > 64 ? 4 : (vecs > 32 ? 2 : 1));
  const int tx = row_threads(vecs, v);
  const int ty = tx == 32 ? 8 : 1;
  const dim3 block(tx, ty);
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.T) + ty - 1) / ty));
  if (v == 1) return launch_pdl(rms_norm_kernel<1>, grid, block, 0, stream, a);
  if (v == 2) return launch_pdl(rms_norm_kernel<2>, grid, block, 0, stream, a);
  return launch_pdl(rms_norm_kernel<4>, grid, block, 0, stream, a);
}

namespace {

constexpr int kWideSmem = 200 * 1024;
static_assert(4 * 3 * 2 * 544 * 16 > kWideSmem && 2 * 3 * 2 * 1024 * 16 <= kWideSmem && 3 * 2 * 2 * 1024 * 16 <= kWideSmem,
              "stages of the wide backward kernel");

// the backward kernel's block: threads per row, rows at a time, vectors per thread
struct BackwardShape {
  int tx, ty, v;
};

BackwardShape backward_shape(int H) {
  const int vecs = H / 8;
  if (vecs <= 64) return {32, 16, vecs > 32 ? 2 : 1};
  const int v = vecs > 1024 ? 2 : 1;
  return {row_threads(vecs, v), 1, v};
}

template <int V, int kStages, bool kRes>
cudaError_t launch_wide(const RmsNormBackwardArgs& a, int blocks, int threads, size_t smem, cudaStream_t stream) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(rms_norm_backward_wide_kernel<V, kStages, kRes>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kWideSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return launch_pdl(rms_norm_backward_wide_kernel<V, kStages, kRes>, dim3(blocks), dim3(threads), smem, stream, a);
}

template <bool kRes>
cudaError_t launch_backward_rows(const RmsNormBackwardArgs& a, int blocks, cudaStream_t stream) {
  const BackwardShape b = backward_shape(a.H);
  const size_t stage = static_cast<size_t>(kRes ? 3 : 2) * b.v * b.tx * 16;
  if (b.ty == 1 && b.v == 2) {  // two vectors per thread leave no registers to load ahead (16384 x 16384: 437 us, this way 380)
    // as many stages as fit: from 544 threads on three of three tensors or four of two, at 1024 two and three
    constexpr int kMost = kRes ? 3 : 4;
    if (kMost * stage <= kWideSmem) return launch_wide<2, kMost, kRes>(a, blocks, b.tx, kMost * stage, stream);
    return launch_wide<2, kMost - 1, kRes>(a, blocks, b.tx, (kMost - 1) * stage, stream);
  }
  // With one vector two rows ahead are better than one where a block has many rows, unless there are three tensors
  // to read (T = 16384, H = 7168: 117 us instead of 132, with a residual gradient 174 instead of 155; T = 1024: 13.8
  // and 12.9 us).
  if constexpr (!kRes)
    if (b.ty == 1 && a.T >= 12 * blocks) return launch_wide<1, 3, kRes>(a, blocks, b.tx, 3 * stage, stream);
  const size_t smem = b.ty > 1 ? static_cast<size_t>(b.ty) * a.H * sizeof(float) : 0;  // at most 32 KB
  if (b.v == 1)
    return launch_pdl(rms_norm_backward_kernel<1, kRes>, dim3(blocks), dim3(b.tx, b.ty), smem, stream, a);
  return launch_pdl(rms_norm_backward_kernel<2, kRes>, dim3(blocks), dim3(b.tx, b.ty), smem, stream, a);
}

}  // namespace

// Enough blocks for about 1024 threads per SM, or one per SM that does not fit twice; fixed numbers, so that neither
// the workspace nor the order of the sums depends on the device.
int rms_norm_backward_blocks(int T, int H) {
  const BackwardShape b = backward_shape(H);
  const int threads = b.tx * b.ty;
  const int most = 148 * (1024 / threads > 8 ? 8 : 1024 / threads);
  const int want = T / b.ty + (T % b.ty != 0);
  return want < most ? want : most;
}

cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, float* dweight, int blocks, cudaStream_t stream) {
  const cudaError_t e =
      a.dresidual ? launch_backward_rows<true>(a, blocks, stream) : launch_backward_rows<false>(a, blocks, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(column_sum_kernel, dim3((a.H + 31) / 32), dim3(32, 32), 0, stream,
                    static_cast<const float*>(a.partials), blocks, a.H, dweight);
}

cudaError_t launch_quantize_rows(const void* x, long long ldx, long long rows, int cols, uint8_t* codes,
                                 float* scales, cudaStream_t stream) {
  const int groups = (cols + 127) / 128;
  // four groups per half-warp where there is work for every SM (8192 x 7168: 44 us with one, 34 us with four)
  const int items = rows * groups >= 148 * 8 * 64 ? 4 : 1;
  const int block_rows = groups < items * 16 ? items * 16 / groups : 1;
  const long long blocks = block_rows > 1 ? (rows + block_rows - 1) / block_rows
                                          : rows * ((groups + items * 16 - 1) / (items * 16));
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
  if (items == 4)
    return launch_pdl(quantize_rows_kernel<4>, grid, dim3(256), 0, stream, xb, ldx, rows, cols, block_rows, codes,
                      scales);
  return launch_pdl(quantize_rows_kernel<1>, grid, dim3(256), 0, stream, xb, ldx, rows, cols, block_rows, codes,
                    scales);
}

cudaError_t launch_dequantize_rows(const uint8_t* codes, const float* scales, long long rows, int cols, void* x,
                                   long long ldx, cudaStream_t stream) {
  const long long threads = rows * (cols / 16);
  return launch_pdl(dequantize_rows_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, stream,
                    codes, scales, rows, cols, static_cast<__nv_bfloat16*>(x), ldx);
}

}  // namespace moe
