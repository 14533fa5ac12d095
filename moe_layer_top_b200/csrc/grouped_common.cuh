// Device and host pieces shared by the grouped matrix products.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "grouped.h"
#include "kernels.h"

namespace moe {

constexpr int kGroupedThreads = 320;  // TMA producer warp, MMA warp, two groups of four epilogue warps
constexpr int kGroupedEpiWarps = 8;
constexpr int kMaxGroups = 1024;
constexpr int kGroupTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kGroupedReserve = 1024 + kGroupTableBytes;  // barriers, then the group tables
constexpr int kSmemMax = 232448;                          // dynamic shared memory of a block on sm_100

// wait-site codes reported in the status word (low byte)
constexpr int kWhereGroupedProducer = 0x41, kWhereGroupedMma = 0x42, kWhereGroupedEpilogue = 0x43,
              kWhereGroupedDrain = 0x44;

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

// After an abort: let every copy already issued into the ring land before the CTA tears down.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, long long fills) {
  for (int s = 0; s < stages; ++s) {
    const long long n_s = fills / stages + (s < fills % stages ? 1 : 0);
    if (n_s > 0) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&full[s], static_cast<uint32_t>((n_s - 1) & 1)) &&
             globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
  }
}

// Wait (bounded) until `drain`, committed after a thread's last MMA, has flipped.
__device__ __forceinline__ void drain_mma(uint64_t* drain, int* status) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(drain, 0)) {
    if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
      report_status(status, MOE_STATUS_WAIT_TIMEOUT | kWhereGroupedDrain);
      break;
    }
  }
}

// --------------------------------------------------------------------------
// clusters of two CTAs (tcgen05 cta_group::2).  Loads name no multicast.
// --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// shared::cluster address of the same shared-memory offset in CTA `rank`
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(smem_u32(p)), "r"(rank));
  return out;
}

// Arrive on a barrier of either CTA.  The arrivals hand over TMEM columns that have been read into registers
// (ordered by the tcgen05 fences) or shared memory that the async proxy reads, no generic writes: the default
// CTA-scope release is enough, where a cluster-scope one would wait for the thread's memory traffic each time
// (measured: it doubled the FP8 products' time per K block).
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// the same behind generic writes to shared memory (made visible to the async proxy before)
__device__ __forceinline__ void arrive_in_cluster_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// TMA tile loads.  kPair: issued by either CTA of a pair, the bytes counted on the barrier whose
// shared::cluster address is `bar` (the leader's); otherwise `bar` is this CTA's own.
template <bool kPair>
__device__ __forceinline__ void load_2d(void* dst, const void* map, uint32_t bar, int x, int y, uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

template <bool kPair>
__device__ __forceinline__ void load_3d(void* dst, const void* map, uint32_t bar, int x, int y, int z,
                                        uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

template <bool kPair>
__device__ __forceinline__ void load_4d(void* dst, const void* map, uint32_t bar, int x, int y, int z, int w,
                                        uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
        : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tmem_alloc_for(uint32_t* dst_smem, uint32_t ncols) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  }
}

template <bool kPair>
__device__ __forceinline__ void tmem_free_for(uint32_t taddr, uint32_t ncols) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}

template <bool kPair>
__device__ __forceinline__ void mma_bf16_for(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_bf16(d, a, b, idesc, acc);
}

template <bool kPair>
__device__ __forceinline__ void mma_fp8_for(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_fp8(d, a, b, idesc, acc);
}

// arrive on `bar` of every CTA of the pair (or of this CTA) once this thread's MMAs so far are done
template <bool kPair>
__device__ __forceinline__ void commit_for(uint64_t* bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    mma_commit(bar);
}

// TMA tile stores from shared memory (made visible to the async proxy before), tracked by the issuing thread's bulk
// groups; what lies outside the tensor is not written.  kAdd: fp32 addition to what is there, once per element.
template <bool kAdd>
__device__ __forceinline__ void store_3d(const void* map, const void* src, int x, int y, int z) {
  if constexpr (kAdd)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Row `lane` of a warp's 32 x 128-byte staging box, as the 128-byte swizzle lays it out: 16-byte piece c goes to
// c ^ (lane mod 8), so that the lanes of a store spread over all banks.
__device__ __forceinline__ void stage_row(uint8_t* box, int lane, const uint4 (&piece)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = piece[c];
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// Group tables in shared memory: off[g] (clamped to [0, M]: no access leaves
// the tensors whatever the offsets hold) and, with `first`, the first tile of
// each group, where a group has ceil(rows / row_tile) * per_row_tile tiles.
// Returns their number.  All threads of the block take part; ends with a
// block barrier.
__device__ __forceinline__ int build_group_tables(const int32_t* offsets, int M, int G, int row_tile, int per_row_tile,
                                                  int* off, int* first, int* scan) {
  for (int i = threadIdx.x; i <= G; i += kGroupedThreads) {
    const int v = offsets ? offsets[i] : (i ? M : 0);
    off[i] = v < 0 ? 0 : (v > M ? M : v);
  }
  __syncthreads();
  if (first == nullptr) return 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    const int rows = g < G ? off[g + 1] - off[g] : 0;
    n[j] = rows > 0 ? (rows + row_tile - 1) / row_tile * per_row_tile : 0;
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
  for (int w = 0; w < kGroupedThreads / 32; ++w) {
    if (w < warp) base += scan[w];
    total += scan[w];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    if (g < G) first[g] = base;
    base += n[j];
  }
  __syncthreads();
  return total;
}

// the group of tile t: the last one whose first tile is <= t
__device__ __forceinline__ int group_of_tile(const int* first, int G, int t) {
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// --------------------------------------------------------------------------
// host side
// --------------------------------------------------------------------------
// tensor map of an output [batches, rows, cols] (bf16 or fp32) for store_3d: boxes of 128 bytes x 32 rows
bool make_store_map(CUtensorMap* map, void* base, int batches, long long rows, long long cols, long long ld, bool f32);

// tensor map of bf16 [batches, rows, cols] whose box is 64 rows of 2 x 64 columns, the second 64 columns 8192 bytes
// behind the first (dimensions: column in a run of 64, row, run, batch); cols must be a multiple of 64
bool make_wide_map(CUtensorMap* map, const void* base, int batches, long long rows, long long cols, long long ld);

// tensor map of [batches, rows, cols] with `ld` elements between rows (rows * ld between batches; batches = 0:
// two dimensions), box = 128 bytes x box_rows, 128-byte swizzle; what lies outside reads as zero
bool make_grouped_map(CUtensorMap* map, const void* base, int batches, long long rows, long long cols, long long ld,
                      int elem_bytes, int box_rows);

// Tensor maps of the same rows with boxes of 16, 32, 64, 96 and 128 rows, so that a stage's rows are one TMA
// instruction: a second and third one for smaller boxes cost more than the rows that a larger box loads in vain
// (the row loads of 32768 x 1536 over 128 groups: 361 us as boxes of 64 and 16, 255 us as boxes of 128).
struct RowMaps {
  CUtensorMap map[5];
};
__host__ __device__ constexpr int row_map_index(int rows) {  // the smallest box that holds `rows` (1 .. 128)
  return rows <= 16 ? 0 : (rows <= 32 ? 1 : (rows <= 64 ? 2 : (rows <= 96 ? 3 : 4)));
}
__host__ __device__ constexpr int row_map_rows(int index) { return index == 0 ? 16 : 32 * index; }
bool make_row_maps(RowMaps* maps, const void* base, long long rows, long long cols, long long ld, int elem_bytes);

// The dynamic shared memory limit is a property of a kernel on each device.
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

// Launch with programmatic stream serialisation (see launch_pdl) as clusters of two CTAs; `pairs` clusters at most.
template <auto kKernel, typename... Args>
cudaError_t launch_pairs(long long pairs, size_t smem, cudaStream_t stream, const Args&... args) {
  static int fit[64] = {};  // clusters that are resident at once (the SMs of a GPC need not pair up evenly)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kGroupedThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  if (fit[dev] == 0) {
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg);
    if (e != cudaSuccess) return e;
    fit[dev] = n > 0 ? n : 1;
  }
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (pairs < fit[dev] ? pairs : fit[dev])));
  return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

}  // namespace moe
