// Device and host pieces shared by the grouped matrix products.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "grouped.h"
#include "kernels.h"

namespace moe {

constexpr int kGroupedEpiWarps = 8;  // two groups of four, besides the TMA producer and the MMA issuer
constexpr int kMaxGroups = 1024;
constexpr int kGroupTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kGroupedReserve = 1024 + kGroupTableBytes;  // barriers, then the group tables
constexpr int kSmemMax = 232448;                          // dynamic shared memory of a block on sm_100

// How a tile is computed: by one CTA, by a pair of CTAs (cta_group::2), or by a cluster that shares its reduction.
enum GroupedMode { kModeSingle = 0, kModePair = 1, kModeSplit = 2 };

// floats between two rows of a split tile's partial sums: 16-byte stores of a warp's rows spread over all banks
constexpr int kPartialPitch = 132;

// wait-site codes reported in the status word (low byte)
constexpr int kWhereGroupedProducer = 0x41, kWhereGroupedMma = 0x42, kWhereGroupedEpilogue = 0x43,
              kWhereGroupedDrain = 0x44;

// Bounded wait: polls the barrier, looking at the abort flag and the clock every 256 polls only.  `beat`, for a wait
// that spans a whole reduction: the number of stages that this CTA's producer has filled, which goes on counting as
// long as the reduction goes on; the limit then holds for the time since it was last seen to have changed.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int where,
                                         const volatile uint32_t* beat = nullptr) {
  uint64_t t0 = 0;
  uint32_t seen = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255) == 0) {
      if (*abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (beat != nullptr && *beat != seen) {
        seen = *beat;
        t0 = now;
      }
      if (now - t0 > kWaitTimeoutNs) {
        *abort = 1;
        report_status(status, MOE_STATUS_WAIT_TIMEOUT | where);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                              int where, const volatile uint32_t* beat = nullptr) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;  // the common case, without the bookkeeping
  const bool ok = wait_bar(bar, parity, abort, status, where, beat);
  return __all_sync(0xffffffffu, ok);
}

// The same for a barrier that a thread of another CTA arrives on behind writes of its own (arrive_in_cluster_release):
// acquired at cluster scope, or the writes would not be ordered.
__device__ __forceinline__ bool warp_wait_peer(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                               int where) {
  if (!warp_wait_bar(bar, parity, abort, status, where)) return false;
  uint32_t ok;  // true at once: the phase is over, and the next one begins when this thread goes on
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return true;
}

// One lane of a converged warp.  The producer and the issuer walk as whole warps and elect a lane for each batch of
// instructions: what a warp computes alike then stays in uniform registers, where a loop inside `if (lane == 0)`
// moves every descriptor and address there for each instruction (about 100 cycles per TMA or MMA instruction).
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
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

// All threads of the cluster take part.  The aligned form wants whole warps that are converged, which loops and
// branches with a count of their own per lane in front of it do not promise.
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// shared::cluster address of the same shared-memory offset in CTA `rank`
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(smem_u32(p)), "r"(rank));
  return out;
}

// Arrive on a barrier of either CTA without ordering the thread's other memory accesses.  The arrivals hand over
// TMEM columns that are in registers by then (tcgen05.wait::ld) or shared memory that the async proxy wrote and
// reads, no generic writes.  A cluster-scope release here waits for the thread's memory traffic each time: the FP8
// product of 8192 x 4096 x 7168 took 531 us with it and 318 us without.
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
  __syncwarp();  // an aligned instruction, as the barriers above
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

// arrive on `bar` of every CTA of the pair (or of this CTA) once this thread's MMAs so far are done; `lead` is the
// pair's first rank in its cluster
template <bool kPair>
__device__ __forceinline__ void commit_for(uint64_t* bar, int lead = 0) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3 << lead))
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

// Row `lane` of a warp's staging box of 32 rows x 16 kPieces bytes (128 or 64), as the swizzle of that width lays it out:
// 16-byte piece c of row r goes to c ^ (r mod 8), or c ^ (r / 2 mod 4), so that a store's lanes spread over all banks.
template <int kPieces>
__device__ __forceinline__ void stage_row(uint8_t* box, int lane, const uint4 (&piece)[kPieces]) {
  static_assert(kPieces == 8 || kPieces == 4, "swizzle width");
  const int x = kPieces == 8 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
  for (int c = 0; c < kPieces; ++c) *reinterpret_cast<uint4*>(box + lane * 16 * kPieces + ((c ^ x) << 4)) = piece[c];
}

// Values that an asynchronous TMEM load delivers may be used from here on: placed behind tcgen05.wait::ld, it keeps the
// compiler from moving their uses in front of the wait.
__device__ __forceinline__ void pin16(uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]),
                 "+r"(v[i + 6]), "+r"(v[i + 7]));
}
__device__ __forceinline__ void pin32(uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]),
                 "+r"(v[i + 6]), "+r"(v[i + 7]));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// (a0, a1) <- (d0, d1) * (f0, f1) + (a0, a1), each correctly rounded; d as raw fp32 words
__device__ __forceinline__ void ffma2v(float& a0, float& a1, uint32_t d0, uint32_t d1, float f0, float f1) {
  asm("{\n\t.reg .b64 ra, rd, rf;\n\t"
      "mov.b64 ra, {%0, %1};\n\t"
      "mov.b64 rd, {%2, %3};\n\t"
      "mov.b64 rf, {%4, %5};\n\t"
      "fma.rn.f32x2 ra, rd, rf, ra;\n\t"
      "mov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "r"(d0), "r"(d1), "f"(f0), "f"(f1));
}

__device__ __forceinline__ float4 load_in_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void store_in_cluster(uint32_t addr, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// Stores 16 accumulator columns of tiles whose columns are output rows: lane `lane` holds column `col` of rows
// 0 .. 15 at out[at + row * ldo + col], of which `rows` are stored, and columns below `cols` (a multiple of 8).  All
// lanes of the warp take part.  bf16: four neighbouring lanes exchange what they have of four rows, so that each
// stores four columns of one: 8 bytes per lane, 64 bytes of each of four rows per instruction.
__device__ __forceinline__ void store_columns16(const float (&v)[16], void* out, long long at, long long ldo, int col,
                                                int cols, int rows, bool f32) {
  const int lane = threadIdx.x & 31;
  if (f32) {
    float* o = static_cast<float*>(out) + at + col;
    if (col < cols) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < rows) o[i * ldo] = v[i];
    }
    return;
  }
  uint32_t u[8], w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t mine = pack_bf16(v[2 * i], v[2 * i + 1]);  // rows 2 i and 2 i + 1 of this column
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
    u[i] = lane & 1 ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 2 ? u[2 * j] : u[2 * j + 1], 2);
    w[2 * j] = lane & 2 ? got : u[2 * j];
    w[2 * j + 1] = lane & 2 ? u[2 * j + 1] : got;
  }
  const int r = lane & 3;  // this lane's rows: r + 4 j
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + at + r * ldo + (col & ~3);
  if (col < cols) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r + 4 * j < rows) *reinterpret_cast<uint2*>(o + 4 * j * ldo) = make_uint2(w[2 * j], w[2 * j + 1]);
  }
}

// The sum of a split tile: every CTA of the cluster has its partial sums [rows][kPartialPitch] at `smem`; CTA `cta`
// adds its part of the elements up in rank order (so the result does not depend on timing) and stores them at
// out[at + row * ldo + column], cols a multiple of 8.  Eight reads of other CTAs' shared memory are under way at a
// time: one after the other their latency is most of a small product's time (333 x 2056 x 1616 bf16 11.6 us that way).
template <int kThreads, int kMost>
__device__ __forceinline__ void add_partials_of(const uint8_t* smem, int cta, int splits, int rows, int cols, void* out,
                                                long long at, long long ldo, bool out_f32, bool accumulate) {
  constexpr int kItems = 8 / kMost;
  const int quads = cols / 4, n = rows * quads, step = splits * kThreads;
  uint32_t part[kMost];
#pragma unroll
  for (int s = 0; s < kMost; ++s) part[s] = in_cta(smem, s < splits ? s : 0);
  for (int i0 = cta * kThreads + threadIdx.x; i0 < n; i0 += kItems * step) {
    float4 p[kItems][kMost];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int i = i0 + u * step;
      const int r = i / quads, c = (i - r * quads) * 4;
#pragma unroll
      for (int s = 0; s < kMost; ++s)
        if (i < n && s < splits) p[u][s] = load_in_cluster(part[s] + (r * kPartialPitch + c) * 4);
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int i = i0 + u * step;
      if (i >= n) break;
      const int r = i / quads, c = (i - r * quads) * 4;
      float4 v = p[u][0];
#pragma unroll
      for (int s = 1; s < kMost; ++s) {
        if (s >= splits) break;
        v.x += p[u][s].x;
        v.y += p[u][s].y;
        v.z += p[u][s].z;
        v.w += p[u][s].w;
      }
      const long long o = at + r * ldo + c;
      if (out_f32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
        if (accumulate) {
          const float4 b = *dst;
          v = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
        }
        *dst = v;
      } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + o) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
      }
    }
  }
}

template <int kThreads>
__device__ __forceinline__ void add_partials(const uint8_t* smem, int cta, int splits, int rows, int cols, void* out,
                                             long long at, long long ldo, bool out_f32, bool accumulate) {
  if (splits == 2) add_partials_of<kThreads, 2>(smem, cta, 2, rows, cols, out, at, ldo, out_f32, accumulate);
  else if (splits <= 4) add_partials_of<kThreads, 4>(smem, cta, splits, rows, cols, out, at, ldo, out_f32, accumulate);
  else add_partials_of<kThreads, 8>(smem, cta, splits, rows, cols, out, at, ldo, out_f32, accumulate);
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

// Group tables in shared memory: off[g], the offsets clamped to [0, M] and made ascending (off[g] is the largest of
// the first g + 1), so that no group leaves the tensors or takes another's rows whatever they hold; and, with
// `first`, the first tile of each group, where a group has ceil(rows / row_tile) * per_row_tile tiles.  Returns their
// number.  All threads of the block take part; ends with a block barrier.
template <int kThreads>
__device__ __forceinline__ int build_group_tables(const int32_t* offsets, int M, int G, int row_tile, int per_row_tile,
                                                  int* off, int* first, int* scan) {
  static_assert(4 * kThreads >= kMaxGroups + 1 && kThreads / 32 <= 32, "four entries per thread");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (G == 1) {  // no scans on the way of a plain product
    const int a = offsets ? min(max(offsets[0], 0), M) : 0;
    const int b = offsets ? max(a, min(max(offsets[1], 0), M)) : M;
    if (threadIdx.x == 0) {
      off[0] = a;
      off[1] = b;
      if (first != nullptr) first[0] = 0;
    }
    __syncthreads();
    return (b - a + row_tile - 1) / row_tile * per_row_tile;
  }
  // inclusive scan of a value per thread over the block: returns the value of the thread before (`none` for the first)
  auto scan_before = [&](int v, int none, auto op) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = op(v, u);
    }
    if (lane == 31) scan[warp] = v;
    int before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = none;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = op(before, scan[w]);
    return before;
  };
  int o[4], top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    const int v = g > G ? 0 : (offsets ? offsets[g] : (g ? M : 0));
    top = max(top, min(max(v, 0), M));
    o[j] = top;
  }
  const int before = scan_before(top, 0, [](int x, int y) { return max(x, y); });
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    if (g <= G) off[g] = max(o[j], before);
  }
  __syncthreads();
  if (first == nullptr) return 0;
  int n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    const int rows = g < G ? off[g + 1] - off[g] : 0;
    n[j] = (rows + row_tile - 1) / row_tile * per_row_tile;
    sum += n[j];
  }
  int base = scan_before(sum, 0, [](int x, int y) { return x + y; });
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = 4 * threadIdx.x + j;
    if (g < G) first[g] = base;
    base += n[j];
  }
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += scan[w];
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
// tensor map of an output [batches, rows, cols] (bf16 or fp32) for store_3d: boxes of 128 or 64 bytes x 32 rows, with
// the swizzle of that width
bool make_store_map(CUtensorMap* map, void* base, int batches, long long rows, long long cols, long long ld, bool f32,
                    int box_bytes);

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
// (those that M rows can need; a box beyond them is not described)
bool make_row_maps(RowMaps* maps, const void* base, long long rows, long long cols, long long ld, int elem_bytes);

// Once per kernel and device: allow its dynamic shared memory, and check that it is launched with at least `regs`
// registers per thread.
template <auto kKernel>
cudaError_t prepare_kernel(size_t smem, int regs) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, kKernel)) != cudaSuccess) return e;
  if (attr.numRegs < regs) return cudaErrorInvalidKernelImage;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

// Clusters of `size` CTAs of the prepared kernel that are resident at once (the SMs of a GPC need not divide evenly);
// asked once per size and device.
template <auto kKernel>
cudaError_t resident_clusters(int threads, int size, size_t smem, int* count) {
  static int fit[64][9] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || size > 8) return cudaErrorInvalidValue;
  if (fit[dev][size] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg)) != cudaSuccess) return e;
    fit[dev][size] = n > 0 ? n : 1;
  }
  *count = fit[dev][size];
  return cudaSuccess;
}

// Launch clusters of `size` CTAs with programmatic stream serialisation (see launch_pdl).  persistent: no more than
// are resident at once.
template <auto kKernel, typename... Args>
cudaError_t launch_clusters(int threads, int size, long long clusters, bool persistent, size_t smem,
                            cudaStream_t stream, const Args&... args) {
  if (persistent) {
    int most = 0;
    const cudaError_t e = resident_clusters<kKernel>(threads, size, smem, &most);
    if (e != cudaSuccess) return e;
    if (clusters > most) clusters = most;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * size));
  return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

// Row tiles of `tile` rows that M rows in G groups come to: exact for one group, otherwise an estimate (the host does
// not see the offsets): every group that can have rows ends in half a tile.
inline long long row_tiles(long long M, long long G, int tile) {
  const long long groups = M < G ? M : G;
  if (G == 1) return (M + tile - 1) / tile;
  const long long n = M / tile + (groups + 1) / 2;
  return n > groups ? n : groups;
}

// CTAs that share a tile's reduction: as many as leave each at least four stages and let all clusters be resident at
// once; 1 if there is nothing to share.  kKernel is prepared if more than 1.  (Sixteen clusters of eight need not fit
// 148 SMs: one row by 2048 x 7168 in FP8 takes 12.5 us in two rounds of clusters of eight and 7.7 us in one of seven.)
template <auto kKernel>
cudaError_t choose_splits(long long tiles, int sms, int stages, int threads, size_t smem, int* splits) {
  *splits = 1;
  for (int s = 8; s > 1; --s) {
    if (tiles * s > sms || stages < 4 * s) continue;
    int most = 0;
    cudaError_t e = prepare_kernel<kKernel>(smem, 0);
    if (e == cudaSuccess) e = resident_clusters<kKernel>(threads, s, smem, &most);
    if (e != cudaSuccess) return e;
    if (tiles > most) continue;
    *splits = s;
    break;
  }
  return cudaSuccess;
}

}  // namespace moe
