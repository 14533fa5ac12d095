// FP8 matrix products with block scales, many rows per group: tiles of two SMs.
//
// A cluster of two CTAs computes 256 rows x 256 columns (tcgen05
// cta_group::2), 32 KB into each SM per 128-deep K block.  The rows fill the
// MMA's M side: an epilogue thread then holds one row, and its factor for a K
// block is one number.  Every K block has its own accumulator in TMEM (two, of
// 256 columns), which the epilogue adds into fp32 registers times the two
// scales while the tensor core works on the next block: the hand-over of these
// accumulators bounds the kernel: a K block takes about 830 cycles, of which
// the products take 512, the rest is the way from commit over both CTAs'
// epilogues back to the issuer, with room for two accumulators only
// (8192 x 4096 x 7168: 211 to 217 us, 2200 TFLOP/s; a plain FP8 product without scales
// per block needs none of it and takes 168 us).
//
// Row tiles start at any row; a tile that runs past its group's end computes
// rows of the next group and does not store them; no more rows than the group
// has are loaded, rounded up to a box of 16, 32, 64, 96 or 128.
//
// kSplit: a cluster of four, two such pairs, each with half of the K blocks; one tile per cluster.  Each pair then
// finishes one half of the columns: the sums of the other half go through distributed shared memory (pushed: reading
// them from the other pair's took 28 us instead of 25 for 256 x 5120 x 7168).
//
// Persistent, three warpgroups per CTA: the first holds the TMA producer, the
// MMA issuer (of a pair's leader) and two warps that multiply the scales and lay
// the factors of four K blocks at a time into shared memory; the other two are
// the epilogue and take over the registers that the first does without.  (An
// epilogue thread must have no global load under way: its hand-offs wait for
// it, 1 to 2 us in every block that loaded a scale.)
#include "grouped_common.cuh"

namespace moe {

namespace {

constexpr int kThreads = 384;
constexpr int kProducerRegs = 104, kEpilogueRegs = 200;  // 128 * 104 + 256 * 200 = 384 * 168, what the launch has
constexpr int kLaunchRegs = 168;
// The scales' factors go through a ring of batches in shared memory: [column half][slot][K block][row].
constexpr int kBatch = 4, kBatches = 3;
constexpr int kScaleBytes = 2 * kBatches * kBatch * 128 * 4;

struct Args {
  int M, G, N;
  int k_blocks;
  int n_tiles;
  const int32_t* offsets;
  const float* x_scale;
  const float* w_scale;
  void* out;
  long long ldo;
  int out_f32;
  int* status;
};

constexpr int kTile = 256;                                  // rows and columns of a tile
constexpr int kStageBytes = 32768;                          // this CTA's 128 rows and 128 weight rows x 128 bytes
constexpr int kAccBufs = 2;
constexpr int kTmemCols = kAccBufs * kTile;
constexpr int kCols = kTile / 2;                            // columns of an epilogue warpgroup
constexpr int kOutBytes = kGroupedEpiWarps * 4096;          // a box of 32 rows x 128 bytes per epilogue warp
constexpr int kStages = (kSmemMax - 1024 - kGroupedReserve - kScaleBytes - kOutBytes) / kStageBytes;
constexpr size_t kSmemBytes =
    static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kScaleBytes + kGroupedReserve + 1024;
constexpr uint32_t kIdesc = make_idesc(kTile, kTile, true);
static_assert(kStages >= 4, "ring depth");

constexpr int kChunk = 16;  // columns of one TMEM load (8 are as good; with 32 the same product takes 257 us)

struct Tile {
  int g, row0, rows, col0;  // first row of the batch, rows to store, first column
};

__device__ __forceinline__ Tile tile_at(const Args& a, const int* off, const int* first, int t) {
  Tile r;
  r.g = group_of_tile(first, a.G, t);
  const int i = t - first[r.g];
  const int m = i / a.n_tiles;
  r.col0 = (i - m * a.n_tiles) * kTile;
  r.row0 = off[r.g] + m * kTile;
  r.rows = min(kTile, off[r.g + 1] - r.row0);
  return r;
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_fp8_pair_kernel(const __grid_constant__ RowMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_out, const Args args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + static_cast<size_t>(kStages) * kStageBytes;
  float* factors = reinterpret_cast<float*>(staging + kOutBytes);
  uint8_t* reserve = staging + kOutBytes + kScaleBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(reserve);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kAccBufs;
  uint64_t* factor_full = acc_empty + kAccBufs;    // [column half][slot]
  uint64_t* factor_empty = factor_full + 2 * kBatches;
  uint64_t* drain = factor_empty + 2 * kBatches;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scan = reinterpret_cast<int*>(reserve + 640);
  int* off = reinterpret_cast<int*>(reserve + 1024);
  int* first = off + kMaxGroups + 4;
  static_assert((2 * kStages + 2 * kAccBufs + 4 * kBatches + 1) * 8 + 8 <= 640, "barriers overlap the scan buffer");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_rank());
  const int rank = cta & 1;                      // half of the tile
  const int part = kSplit ? cta >> 1 : 0;        // half of the K blocks
  const int lead = kSplit ? cta & ~1 : 0;        // the pair's leader in the cluster
  const bool leader = rank == 0;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kAccBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kGroupedEpiWarps);
    }
    for (int b = 0; b < 2 * kBatches; ++b) {
      mbar_init(&factor_full[b], 1);
      mbar_init(&factor_empty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x.map[0]);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) tmem_alloc_for<true>(tmem_slot, kTmemCols);
  pdl_wait();
  tc_fence_before();
  const int num_tiles = build_group_tables<kThreads>(args.offsets, args.M, args.G, kTile, args.n_tiles, off, first,
                                                     scan);
  cluster_barrier();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  constexpr int kCluster = kSplit ? 4 : 2;
  const int first_tile = static_cast<int>(blockIdx.x) / kCluster;
  const int stride = static_cast<int>(gridDim.x) / kCluster;  // kSplit: no cluster takes a second tile
  const int kb0 = kSplit ? args.k_blocks * part / 2 : 0;
  const int kb1 = kSplit ? args.k_blocks * (part + 1) / 2 : args.k_blocks;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp == 0) {
      // ---------------------------------------------------------------- producer (of each CTA)
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at(args, off, first, t);
        auto loaded = [&](int r) {  // rows that CTA r loads
          const int n = min(128, tl.rows - 128 * r);
          return n > 0 ? row_map_rows(row_map_index(n)) : 0;
        };
        const int rows = loaded(rank);
        const CUtensorMap* map = &tm_x.map[rows > 0 ? row_map_index(rows) : 0];
        const uint32_t bytes = (loaded(0) + loaded(1)) * 128 + 32768;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = warp_wait_bar(&empty[stage], phase ^ 1u, abort_flag, args.status, kWhereGroupedProducer);
          if (!ok) break;
          if (elect_lane()) {
            uint8_t* a = smem + static_cast<size_t>(stage) * kStageBytes;
            if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
            const uint32_t bar = in_cta(&full[stage], lead);
            if (rows > 0) load_2d<true>(a, map, bar, kb * 128, tl.row0 + 128 * rank, pol);
            load_3d<true>(a + 16384, &tm_w, bar, kb * 128, tl.col0 + 128 * rank, tl.g, pol);
          }
          __syncwarp();
          ++fills;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) drain_copies(full, kStages, fills);  // the leader's barriers count both CTAs' copies
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      if (leader) {
        int stage = 0, abuf = 0;
        uint32_t phase = 0, aphase = 0;
        bool ok = true;
        for (int t = first_tile; t < num_tiles && ok; t += stride) {
          for (int kb = kb0; kb < kb1; ++kb) {
            // (the operands are there long before the accumulator is: wait for that last)
            const uint32_t d = tmem_base + static_cast<uint32_t>(abuf * kTile);
            const uint32_t a = smem_u32(smem + static_cast<size_t>(stage) * kStageBytes);
            const uint64_t ad = smem_desc_sw128(a), bd = smem_desc_sw128(a + 16384);
            ok = warp_wait_bar(&full[stage], phase, abort_flag, args.status, kWhereGroupedMma) &&
                 warp_wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereGroupedMma);
            if (!ok) break;
            tc_fence_after();
            if (elect_lane()) {
#pragma unroll
              for (int s = 0; s < 4; ++s) mma_fp8_for<true>(d, ad + 2 * s, bd + 2 * s, kIdesc, s > 0 ? 1u : 0u);
              commit_for<true>(&acc_full[abuf], lead);
              commit_for<true>(&empty[stage], lead);
            }
            __syncwarp();
            if (++abuf == kAccBufs) {
              abuf = 0;
              aphase ^= 1u;
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // every MMA that the elected lanes issued has completed once `drain` flips
        // (waited on even after an abort: TMEM must not be freed under a running MMA)
        if (elect_lane()) commit_for<true>(drain, lead);
        __syncwarp();
        drain_mma(drain, args.status);
      }
    } else if (warp >= 2) {
      // ---------------------------------------------------------------- factors of column half warp - 2
      const int g = warp - 2;
      const int n_blocks = (args.N + 127) / 128;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at(args, off, first, t);
        const int n = min((tl.col0 + kCols * g) / 128, n_blocks - 1);
        const float* w = args.w_scale + (static_cast<long long>(tl.g) * n_blocks + n) * args.k_blocks;
        const float* x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = args.x_scale + tl.row0 + min(128 * rank + lane + 32 * i, tl.rows - 1);
        for (int kb = kb0; kb < kb1; kb += kBatch) {
          float xs[kBatch][4], ws[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int k = min(kb + j, kb1 - 1);
            ws[j] = w[k];
#pragma unroll
            for (int i = 0; i < 4; ++i) xs[j][i] = x[i][static_cast<long long>(k) * args.M];
          }
          ok = warp_wait_bar(&factor_empty[g * kBatches + slot], phase ^ 1u, abort_flag, args.status,
                             kWhereGroupedProducer);
          if (!ok) break;
          float* f = factors + (g * kBatches + slot) * kBatch * 128 + lane;
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[j * 128 + 32 * i] = xs[j][i] * ws[j];
          __syncwarp();
          if (elect_lane()) mbar_arrive(&factor_full[g * kBatches + slot]);
          if (++slot == kBatches) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
    if (kSplit) {  // where the pairs meet
      cluster_barrier();
      cluster_barrier();
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    const int g = (warp - 4) >> 2;        // column half
    const int row = 32 * q + lane;        // accumulator row
    uint8_t* out_box = staging + static_cast<size_t>(warp - 4) * 4096;
    const uint32_t lane_addr = (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(kCols * g);
    const uint32_t empty_bar = in_cta(acc_empty, lead);
    const float* my_factors = factors + g * kBatches * kBatch * 128 + row;
    uint32_t fphase = 0;
    int slot = 0;
    int abuf = 0;
    uint32_t aphase = 0;
    bool ok = true, met = false;  // kSplit: met the other pair
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at(args, off, first, t);
      const int rows = tl.rows - 128 * rank;            // of this CTA's half
      const int col = tl.col0 + kCols * g;           // first column of this thread
      const bool live = 32 * q < rows && col < args.N;  // this warp has something to store
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      for (int kb = kb0; kb < kb1 && ok; kb += kBatch) {
        // the factors of the next blocks
        ok = warp_wait_bar(&factor_full[g * kBatches + slot], fphase, abort_flag, args.status, kWhereGroupedEpilogue);
        if (!ok) break;
        float f[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) f[j] = my_factors[(slot * kBatch + j) * 128];
        __syncwarp();
        if (elect_lane()) mbar_arrive(&factor_empty[g * kBatches + slot]);
        if (++slot == kBatches) {
          slot = 0;
          fphase ^= 1u;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (kb + j >= kb1) break;
          ok = warp_wait_bar(&acc_full[abuf], aphase, abort_flag, args.status, kWhereGroupedEpilogue);
          if (!ok) break;
          tc_fence_after();
          // chunk c + 1 is read from TMEM while chunk c is scaled and added; the buffer goes back to the tensor core
          // as soon as its last chunk is in registers
          const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * kTile);
          uint32_t v[2][kChunk];
          if (live) tmem_ld16u(d, v[0]);
#pragma unroll
          for (int c = 0; c < kCols / kChunk; ++c) {
            if (live) {
              tmem_wait_ld();
              pin16(v[c & 1]);
              if (c + 1 < kCols / kChunk) tmem_ld16u(d + kChunk * (c + 1), v[(c + 1) & 1]);
            }
            if (c + 1 == kCols / kChunk) {
              tc_fence_before();
              __syncwarp();
              if (elect_lane()) arrive_in_cluster(empty_bar + 8 * abuf);
            }
            if (live) {
#pragma unroll
              for (int i = 0; i < kChunk; i += 2)
                ffma2f(acc[kChunk * c + i], acc[kChunk * c + i + 1], v[c & 1][i], v[c & 1][i + 1], f[j]);
            }
          }
          if (++abuf == kAccBufs) {
            abuf = 0;
            aphase ^= 1u;
          }
        }
      }
      if (!ok) break;
      if constexpr (kSplit) {
        // each pair finishes one column half: the other half's sums go to the CTA with the same rows in the other
        // pair, into its ring, which is idle behind the first barrier
        const int mine = row * kPartialPitch * 4;
        __syncwarp();
        cluster_barrier();
        if (live && g != part) {
          const uint32_t p = in_cta(smem + mine, cta ^ 2);
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            store_in_cluster(p + 4 * c, make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]));
        }
        __syncwarp();
        cluster_barrier();
        met = true;
        if (g != part) continue;
        if (live) {
          const float4* p = reinterpret_cast<const float4*>(smem + mine);
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float4 v = p[c / 4];
            acc[c] += v.x;
            acc[c + 1] += v.y;
            acc[c + 2] += v.z;
            acc[c + 3] += v.w;
          }
        }
      }
      if (!live) continue;
      if (32 * q + 32 <= rows) {
        // 128 bytes of each row go through shared memory as one TMA store of the warp's 32 rows (it leaves out
        // what lies behind the last column)
        auto store_box = [&](int c, const uint4 (&piece)[8]) {
          if (lane == 0) bulk_wait_read_all();  // the previous store has read the box
          __syncwarp();
          stage_row(out_box, lane, piece);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            store_3d<false>(&tm_out, out_box, col + c, tl.row0 + 128 * rank + 32 * q, 0);
            bulk_commit();
          }
        };
        if (args.out_f32) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            if (col + c >= args.N) break;
            uint4 piece[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float* f = acc + c + 4 * i;
              piece[i] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                    __float_as_uint(f[3]));
            }
            store_box(c, piece);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 64) {
            if (col + c >= args.N) break;
            uint4 piece[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) piece[i] = pack_bf16x8(acc + c + 8 * i);
            store_box(c, piece);
          }
        }
      } else if (row < rows) {
        // the group ends inside the warp's rows: each thread stores its own (N is a multiple of 8)
        const long long at = (static_cast<long long>(tl.row0) + 128 * rank + row) * args.ldo + col;
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          if (col + c >= args.N) break;
          const float* f = acc + c;
          if (args.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(args.out) + at + c);
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
          } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.out) + at + c) = pack_bf16x8(f);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    if (kSplit && !met) {
      cluster_barrier();
      cluster_barrier();
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_barrier();  // the leader's MMAs read this CTA's shared memory: leave together
  if (warp == 1) {
    tc_fence_after();
    tmem_free_for<true>(tmem_base, kTmemCols);
  }
}

template <bool kSplit>
cudaError_t launch_tiles(const GroupedProblem& p, cudaStream_t s) {
  constexpr auto kern = grouped_fp8_pair_kernel<kSplit>;
  // the register split waits for ever if the kernel is launched with fewer registers than it redistributes
  const cudaError_t e = prepare_kernel<kern>(kSmemBytes, kLaunchRegs);
  if (e != cudaSuccess) return e;
  Args a{};
  a.M = p.M;
  a.G = p.G;
  a.N = p.N;
  a.k_blocks = (p.K + 127) / 128;
  a.n_tiles = (p.N + kTile - 1) / kTile;
  a.offsets = p.offsets;
  a.x_scale = p.a_scale;
  a.w_scale = p.b_scale;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.status = p.status;
  RowMaps tm_x{};
  CUtensorMap tm_w, tm_out;
  if (!make_row_maps(&tm_x, p.a, p.M, p.K, p.lda, 1) ||
      !make_grouped_map(&tm_w, p.b, p.G, p.N, p.K, p.K, 1, 128) ||
      !make_store_map(&tm_out, p.out, 1, p.M, p.N, p.ldo, p.out_f32, 128))
    return cudaErrorInvalidValue;
  const long long tiles = (static_cast<long long>(p.M) / kTile + (p.M < p.G ? p.M : p.G)) * a.n_tiles;
  return launch_clusters<kern>(kThreads, kSplit ? 4 : 2, tiles, !kSplit, kSmemBytes, s, tm_x, tm_w, tm_out, a);
}

}  // namespace

cudaError_t launch_grouped_fp8_pair(const GroupedProblem& p, bool split, cudaStream_t s) {
  return split ? launch_tiles<true>(p, s) : launch_tiles<false>(p, s);
}

cudaError_t fp8_pair_split_clusters(int* count) {
  constexpr auto kern = grouped_fp8_pair_kernel<true>;
  const cudaError_t e = prepare_kernel<kern>(kSmemBytes, kLaunchRegs);
  return e != cudaSuccess ? e : resident_clusters<kern>(kThreads, 4, kSmemBytes, count);
}

}  // namespace moe
