// Matrix products grouped by expert with ragged sizes, on the 5th-generation
// tensor cores (tcgen05, sm_100a).  Group g owns rows [off[g], off[g + 1]):
//
//   forward : y[r, :]  = x[r, :] . w[g]^T          (bf16, or E4M3 with scales)
//   dx      : dx[r, :] = dy[r, :] . w[g]
//   dw      : dw[g]    = dy_g^T . x_g               (reduction over g's rows)
//
// One group of all rows is the plain product.  No operand is copied, padded
// or transposed in memory: the tensor core reads K-major tiles (x, dy, and w
// in the forward product) and MN-major tiles (w in dx; dy and x in dw) alike,
// so every product takes the tensors as they lie.  Row tiles start at any
// row; a tile that runs past its group's end computes rows of the next group
// and does not store them.  In dw the rows are the reduction axis: the rows
// past the group's end in its last stage are cleared in shared memory.
//
// FP8: per 128-deep K block the accumulator is promoted into fp32 registers
// with the product of the row's scale and the weight block's scale.
//
// One CTA per SM, persistent over 128 x 128 tiles, 10 warps: TMA producer,
// MMA issuer, two groups of four epilogue warps (64 columns each).
#include <cudaTypedefs.h>

#include "common.cuh"
#include "grouped.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kMaxGroups = 1024;
constexpr int kTile = 128;                       // rows and columns of a tile
constexpr int kOperandBytes = kTile * 128;       // one operand of a stage: 128 rows (or columns) x 128 bytes
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 5;
constexpr int kOutPitch = 144;                   // 128 bytes of a row + 16: rows spread over the banks
constexpr int kOutBytes = kEpiWarps * 32 * kOutPitch;
constexpr int kTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kReserve = 1024 + kTableBytes;     // barriers, then the group tables
constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kReserve + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

// wait-site codes reported in the status word (low byte)
constexpr int kWhereProducer = 0x41, kWhereMma = 0x42, kWhereEpilogue = 0x43, kWhereDrain = 0x44;

struct Args {
  int M, G;
  int rows;          // output rows of a group: N (dw); otherwise the group's own rows
  int cols;          // output columns
  int red;           // reduction length (fwd: K, dx: N; dw: the group's rows)
  int n_tiles;       // column tiles
  int box_rows;      // fwd, dx: rows of one TMA box of A
  const int32_t* offsets;
  const float* a_scale;
  const float* b_scale;
  void* out;
  long long ldo;
  int out_f32, accumulate;
  int* status;
};

// Bounded wait: polls the barrier, looking at the abort flag and the clock
// only now and then (reading the clock costs more than a poll).
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int where) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31) == 0) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
        *abort = 1;
        report_status(status, MOE_STATUS_WAIT_TIMEOUT | where);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                              int where) {
  const bool ok = wait_bar(bar, parity, abort, status, where);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* map, uint64_t* bar, int x, int y, int z,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// fp32 add of `bytes` from shared into global memory (each element one addition)
__device__ __forceinline__ void bulk_add_f32(void* dst, const void* smem_src, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(smem_src)), "r"(bytes)
               : "memory");
}

// Descriptor of an MN-major operand written by TMA with the 128-byte swizzle
// as boxes of 64 columns (128 bytes) x 64 rows of the reduction axis: the
// leading byte offset (bits 16-29) is the distance of two 64-column boxes,
// the stride byte offset (bits 32-45) that of two 8-row groups.  16 rows of
// the reduction axis further is + 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

struct Tile {
  int g, row0, rows, col0;  // first output row (fwd, dx: of the batch; dw: of the group), rows to store, first column
  int red0, red;            // dw: the group's first row and row count; otherwise 0 and the reduction length
};

// Group tables in shared memory: off[g] (clamped to [0, M]: no access leaves
// the tensors whatever the offsets hold) and the first tile of each group.
// Returns the number of tiles.  All threads of the block take part.
template <int Kind>
__device__ __forceinline__ int build_tables(const Args& a, int* off, int* first, int* scan) {
  for (int i = threadIdx.x; i <= a.G; i += kThreads) {
    int v = a.offsets ? a.offsets[i] : (i ? a.M : 0);
    off[i] = v < 0 ? 0 : (v > a.M ? a.M : v);
  }
  if constexpr (Kind == kGroupedDw) {
    __syncthreads();
    return a.G * ((a.rows + kTile - 1) / kTile) * a.n_tiles;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  int n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    const int rows = g < a.G ? off[g + 1] - off[g] : 0;
    n[j] = rows > 0 ? (rows + kTile - 1) / kTile * a.n_tiles : 0;
    sum += n[j];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int base = incl - sum, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += scan[w];
    total += scan[w];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    if (g < a.G) first[g] = base;
    base += n[j];
  }
  __syncthreads();
  return total;
}

template <int Kind>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* off, const int* first, int t) {
  Tile r;
  int m;
  if constexpr (Kind == kGroupedDw) {
    const int per_row = a.n_tiles, per_group = ((a.rows + kTile - 1) / kTile) * per_row;
    r.g = t / per_group;
    const int i = t - r.g * per_group;
    m = i / per_row;
    r.col0 = (i - m * per_row) * kTile;
    r.row0 = m * kTile;
    r.rows = min(kTile, a.rows - r.row0);
    r.red0 = off[r.g];
    r.red = max(0, off[r.g + 1] - r.red0);
  } else {
    int lo = 0, hi = a.G;  // the last group whose first tile is <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= t) lo = mid; else hi = mid;
    }
    r.g = lo;
    const int i = t - first[lo];
    m = i / a.n_tiles;
    r.col0 = (i - m * a.n_tiles) * kTile;
    r.row0 = off[lo] + m * kTile;
    r.rows = min(kTile, off[lo + 1] - r.row0);
    r.red0 = 0;
    r.red = a.red;
  }
  return r;
}

template <int Kind, bool kFP8>
struct Cfg {
  static constexpr int kRed = kFP8 ? 128 : 64;   // reduction elements per stage
  static constexpr bool kMnA = Kind == kGroupedDw;
  static constexpr bool kMnB = Kind != kGroupedFwd;
  // bf16: a tile accumulates in one buffer; FP8: one buffer per K block
  static constexpr int kAccBufs = kFP8 ? 4 : 2;
  static constexpr int kTmemCols = kAccBufs * kTile;
  static constexpr uint32_t kIdesc =
      make_idesc(kTile, kTile, kFP8) | (kMnA ? 1u << 15 : 0u) | (kMnB ? 1u << 16 : 0u);
};

template <int Kind, bool kFP8>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const Args args) {
  using C = Cfg<Kind, kFP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + static_cast<size_t>(kStages) * kStageBytes;
  uint8_t* reserve = staging + kOutBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(reserve);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + C::kAccBufs;
  uint64_t* drain = acc_empty + C::kAccBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scan = reinterpret_cast<int*>(reserve + 512);
  int* off = reinterpret_cast<int*>(reserve + 1024);
  int* first = off + kMaxGroups + 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  const int num_tiles = build_tables<Kind>(args, off, first, scan);  // ends with a block barrier
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        const Tile tl = tile_at<Kind>(args, off, first, t);
        const int boxes = Kind == kGroupedDw ? 0 : (tl.rows + args.box_rows - 1) / args.box_rows;
        const uint32_t bytes =
            kOperandBytes + (Kind == kGroupedDw ? kOperandBytes : boxes * args.box_rows * 128);
        for (int k = 0; k < tl.red; k += C::kRed) {
          if (!wait_bar(&empty[stage], phase ^ 1u, abort_flag, args.status, kWhereProducer)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + static_cast<size_t>(stage) * kStageBytes;
          uint8_t* b = a + kOperandBytes;
          mbar_arrive_expect_tx(&full[stage], bytes);
          if constexpr (Kind == kGroupedDw) {
            tma_load_2d(a, &tm_a, &full[stage], tl.row0, tl.red0 + k, pol);
            tma_load_2d(a + 8192, &tm_a, &full[stage], tl.row0 + 64, tl.red0 + k, pol);
            tma_load_2d(b, &tm_b, &full[stage], tl.col0, tl.red0 + k, pol);
            tma_load_2d(b + 8192, &tm_b, &full[stage], tl.col0 + 64, tl.red0 + k, pol);
          } else {
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(a + i * args.box_rows * 128, &tm_a, &full[stage], k, tl.row0 + i * args.box_rows, pol);
            if constexpr (Kind == kGroupedFwd) {
              tma_load_3d(b, &tm_b, &full[stage], k, tl.col0, tl.g, pol);
            } else {
              tma_load_3d(b, &tm_b, &full[stage], tl.col0, k, tl.g, pol);
              tma_load_3d(b + 8192, &tm_b, &full[stage], tl.col0 + 64, k, tl.g, pol);
            }
          }
          ++fills;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // let every copy already issued land before the CTA tears down
        for (int s = 0; s < kStages; ++s) {
          const long long n_s = fills / kStages + (s < fills % kStages ? 1 : 0);
          if (n_s > 0) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&full[s], static_cast<uint32_t>((n_s - 1) & 1)) &&
                   globaltimer_ns() - t0 < kWaitTimeoutNs) {
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (the whole warp walks, lane 0 issues)
    int stage = 0, abuf = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
      const Tile tl = tile_at<Kind>(args, off, first, t);
      if (tl.red == 0) continue;
      if constexpr (!kFP8) {
        if (!warp_wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereMma)) break;
      }
      for (int k = 0; k < tl.red; k += C::kRed) {
        ok = warp_wait_bar(&full[stage], phase, abort_flag, args.status, kWhereMma);
        if (!ok) break;
        if constexpr (kFP8) {
          ok = warp_wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereMma);
          if (!ok) break;
        }
        uint8_t* st = smem + static_cast<size_t>(stage) * kStageBytes;
        int steps = 4;
        if constexpr (Kind == kGroupedDw) {
          const int valid = tl.red - k;
          if (valid < 64) {
            // the group ends inside this stage: clear the rows behind it up to the next step of 16
            // (the swizzle permutes 16-byte pieces inside a 128-byte row only, so whole rows are cleared)
            steps = (valid + 15) / 16;
            const int dead = 16 * steps - valid;
            for (int i = lane; i < 4 * dead * 8; i += 32) {
              const int box = i / (dead * 8), r = i / 8 % dead, c = i & 7;
              *reinterpret_cast<uint4*>(st + box * 8192 + (valid + r) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t d = tmem_base + static_cast<uint32_t>(abuf * kTile);
          const uint32_t a = smem_u32(st), b = a + kOperandBytes;
          for (int s = 0; s < steps; ++s) {
            const uint64_t ad = C::kMnA ? smem_desc_mn_sw128(a + 2048 * s) : smem_desc_sw128(a + 32 * s);
            const uint64_t bd = C::kMnB ? smem_desc_mn_sw128(b + 2048 * s) : smem_desc_sw128(b + 32 * s);
            if constexpr (kFP8)
              mma_fp8(d, ad, bd, C::kIdesc, s > 0 ? 1u : 0u);
            else
              mma_bf16(d, ad, bd, C::kIdesc, (k > 0 || s > 0) ? 1u : 0u);
          }
          mma_commit(&empty[stage]);
          if constexpr (kFP8) mma_commit(&acc_full[abuf]);
        }
        __syncwarp();
        if constexpr (kFP8) {
          if (++abuf == C::kAccBufs) {
            abuf = 0;
            aphase ^= 1u;
          }
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if constexpr (!kFP8) {
        if (lane == 0) mma_commit(&acc_full[abuf]);
        if (++abuf == C::kAccBufs) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
    }
    // every MMA this thread issued has completed once `drain` flips
    // (waited on even after an abort: TMEM must not be freed under a running MMA)
    if (lane == 0) {
      mma_commit(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0)) {
        if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
          report_status(args.status, MOE_STATUS_WAIT_TIMEOUT | kWhereDrain);
          break;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    const int g = (warp - 2) >> 2;        // column half
    const int row = 32 * q + lane;        // accumulator row
    uint8_t* out_row = staging + static_cast<size_t>(threadIdx.x - 64) * kOutPitch;
    const uint32_t lane_addr = (static_cast<uint32_t>(32 * q) << 16) + 64u * g;
    int abuf = 0;
    uint32_t aphase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
      const Tile tl = tile_at<Kind>(args, off, first, t);
      const bool warp_live = 32 * q < tl.rows && tl.col0 + 64 * g < args.cols;  // this warp has something to store
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      if constexpr (kFP8) {
        const int kb_n = (tl.red + 127) / 128;
        const float* sa = args.a_scale + tl.row0 + (row < tl.rows ? row : 0);
        const float* sb =
            args.b_scale + (static_cast<long long>(tl.g) * args.n_tiles + tl.col0 / kTile) * kb_n;
        float sa0 = warp_live ? *sa : 0.f, sb0 = *sb;
        for (int kb = 0; kb < kb_n; ++kb) {
          const float f = sa0 * sb0;
          if (kb + 1 < kb_n) {  // the next block's scales, ahead of the wait
            if (warp_live) sa0 = sa[static_cast<long long>(kb + 1) * args.M];
            sb0 = sb[kb + 1];
          }
          ok = warp_wait_bar(&acc_full[abuf], aphase, abort_flag, args.status, kWhereEpilogue);
          if (!ok) break;
          tc_fence_after();
          if (warp_live) {
            const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * kTile);
            uint32_t v[2][16];
            tmem_ld16u(d, v[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_wait_ld();
              if (c + 1 < 4) tmem_ld16u(d + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 16; i += 2)
                ffma2f(acc[16 * c + i], acc[16 * c + i + 1], v[c & 1][i], v[c & 1][i + 1], f);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[abuf]);
          if (++abuf == C::kAccBufs) {
            abuf = 0;
            aphase ^= 1u;
          }
        }
        if (!ok) break;
      } else if (tl.red > 0) {
        ok = warp_wait_bar(&acc_full[abuf], aphase, abort_flag, args.status, kWhereEpilogue);
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * kTile);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[16];
            tmem_ld16(d + 16 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[16 * c + i] = v[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[abuf]);
        if (++abuf == C::kAccBufs) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      // store: the thread's row goes through shared memory as bulk copies of up to 128 bytes
      const int col = tl.col0 + 64 * g;
      const int width = min(64, args.cols - col);
      // (a group without rows adds nothing to an accumulated gradient)
      if (row < tl.rows && width > 0 && !(args.accumulate && tl.red == 0)) {
        const long long at = (Kind == kGroupedDw
                                  ? (static_cast<long long>(tl.g) * args.rows + tl.row0 + row) * args.cols
                                  : (static_cast<long long>(tl.row0) + row) * args.ldo) + col;
        if (args.out_f32) {
          float* dst = static_cast<float*>(args.out) + at;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int w = min(32, width - 32 * h);
            if (w <= 0) break;
            bulk_wait_read_all();  // the previous copy has read the staging row
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4*>(out_row)[i] = make_float4(acc[32 * h + 4 * i], acc[32 * h + 4 * i + 1],
                                                                  acc[32 * h + 4 * i + 2], acc[32 * h + 4 * i + 3]);
            fence_proxy_async_smem();
            if (args.accumulate)
              bulk_add_f32(dst + 32 * h, out_row, 4 * w);
            else
              bulk_store(dst + 32 * h, out_row, 4 * w);
            bulk_commit();
          }
        } else {
          bulk_wait_read_all();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint4 u;
            __nv_bfloat162* h2 = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
            for (int j = 0; j < 4; ++j) h2[j] = __floats2bfloat162_rn(acc[8 * i + 2 * j], acc[8 * i + 2 * j + 1]);
            reinterpret_cast<uint4*>(out_row)[i] = u;
          }
          fence_proxy_async_smem();
          bulk_store(static_cast<__nv_bfloat16*>(args.out) + at, out_row, 2 * width);
          bulk_commit();
        }
      }
    }
    bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// tensor map of [batches, rows, cols] with `ld` elements between rows (batches > 0: rows * ld between batches),
// box = 128 bytes x box_rows, 128-byte swizzle; what lies outside reads as zero
bool make_map(CUtensorMap* map, const void* base, int batches, long long rows, long long cols, long long ld,
              int elem_bytes, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const CUtensorMapDataType dt = elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(batches)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * elem_bytes,
                           static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(rows) * elem_bytes};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem_bytes), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, dt, batches > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The dynamic shared memory limit is a property of the kernel on each device.
template <auto kKernel>
cudaError_t allow_smem(size_t bytes) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <int Kind, bool kFP8>
cudaError_t launch_tiles(const GroupedProblem& p, cudaStream_t s) {
  constexpr auto kern = grouped_kernel<Kind, kFP8>;
  cudaError_t e = allow_smem<kern>(kSmemBytes);
  if (e != cudaSuccess) return e;
  const int elem = kFP8 ? 1 : 2;
  Args a{};
  a.M = p.M;
  a.G = p.G;
  a.rows = p.N;
  a.cols = Kind == kGroupedFwd ? p.N : p.K;
  a.red = Kind == kGroupedFwd ? p.K : p.N;
  a.n_tiles = (a.cols + kTile - 1) / kTile;
  a.offsets = p.offsets;
  a.a_scale = p.a_scale;
  a.b_scale = p.b_scale;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.accumulate = p.accumulate;
  a.status = p.status;
  a.box_rows = 16;
  CUtensorMap tm_a, tm_b;
  long long tiles;
  if (Kind == kGroupedDw) {
    // an empty batch has no rows to map: its tiles load nothing
    const void* base_a = p.M > 0 ? p.a : p.out;
    const void* base_b = p.M > 0 ? p.b : p.out;
    const long long rows = p.M > 0 ? p.M : 1;
    if (!make_map(&tm_a, base_a, 0, rows, p.N, p.M > 0 ? p.lda : p.N, 2, 64)) return cudaErrorInvalidValue;
    if (!make_map(&tm_b, base_b, 0, rows, p.K, p.M > 0 ? p.ldb : p.K, 2, 64)) return cudaErrorInvalidValue;
    tiles = static_cast<long long>(p.G) * ((p.N + kTile - 1) / kTile) * a.n_tiles;
  } else {
    if (!make_map(&tm_a, p.a, 0, p.M, Kind == kGroupedFwd ? p.K : p.N, p.lda, elem, a.box_rows))
      return cudaErrorInvalidValue;
    if (!make_map(&tm_b, p.b, p.G, p.N, p.K, p.K, elem, Kind == kGroupedFwd ? kTile : 64))
      return cudaErrorInvalidValue;
    tiles = (static_cast<long long>(p.M) / kTile + (p.M < p.G ? p.M : p.G)) * a.n_tiles;
  }
  const unsigned grid = static_cast<unsigned>(tiles < p.num_sms ? tiles : p.num_sms);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, s, tm_a, tm_b, a);
}

}  // namespace

cudaError_t launch_grouped(const GroupedProblem& p, cudaStream_t stream) {
  switch (p.kind) {
    case kGroupedFwd: return p.fp8 ? launch_tiles<kGroupedFwd, true>(p, stream) : launch_tiles<kGroupedFwd, false>(p, stream);
    case kGroupedDx: return launch_tiles<kGroupedDx, false>(p, stream);
    default: return launch_tiles<kGroupedDw, false>(p, stream);
  }
}

}  // namespace moe
