// FP8 (E4M3) matrix products with block scales, grouped by expert with ragged
// sizes, on the 5th-generation tensor cores (tcgen05, sm_100a):
//
//   y[r, n] = sum over 128-deep K blocks b of
//             x_scale[b, r] * w_scale[g(r), n / 128, b] * (x_b[r] . w_b[g(r), n])
//
// One group of all rows is the plain product.  The rows fill the MMA's M side:
// an epilogue thread then holds one row and its factor for a K block is one
// number (on the N side it would need one per column).  Every K block has its
// own accumulator in TMEM, which the epilogue adds into fp32 registers times
// the two scales while the tensor core works on the next blocks.
//
// Row tiles start at any row; a tile that runs past its group's end computes
// rows of the next group and does not store them; no more rows than the group
// has are loaded, rounded up to a box of 16, 32, 64, 96 or 128.
//
// kPair: a cluster of two CTAs computes 256 x 256 (cta_group::2), 32 KB into
// each SM per K block.  kSingle: one CTA computes 128 x 128.  kSplit: a
// cluster of up to eight CTAs shares the K blocks of one 128 x 128 tile, each
// leaves its partial sums in shared memory and all add a part of them up, in
// rank order: a product of a few rows then streams its weights through all
// SMs instead of one per 128 columns.
//
// Persistent (kSplit: one tile per cluster), three warpgroups per CTA: the
// first holds the TMA producer, the MMA issuer (of the leader CTA) and two
// warps that multiply the scales and lay the factors of four K blocks at a time
// into shared memory; the other two are the epilogue and take over the
// registers that the first does without.  (An epilogue thread must have no
// global load under way: its hand-offs wait for it, 1 to 2 us in every block
// that loaded a scale.)
#include "grouped_common.cuh"

namespace moe {

namespace {

constexpr int kThreads = 384;
constexpr int kProducerRegs = 56, kEpilogueRegs = 224;  // 128 * 56 + 256 * 224 = 384 * 168, what the launch has
constexpr int kLaunchRegs = 168;
// The scales' factors go through a ring of batches in shared memory: [column half][slot][K block][row].
constexpr int kBatch = 4, kBatches = 3;
constexpr int kScaleBytes = 2 * kBatches * kBatch * 128 * 4;

struct Args {
  int M, G, N;
  int k_blocks;
  int n_tiles;
  int splits;        // kSplit: CTAs per cluster
  const int32_t* offsets;
  const float* x_scale;
  const float* w_scale;
  void* out;
  long long ldo;
  int out_f32;
  int* status;
};

template <int Mode>
struct Cfg {
  static constexpr bool kPair = Mode == kModePair;
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTile = 128 * kCtas;            // rows and columns of a tile
  static constexpr int kStageBytes = 32768;            // this CTA's 128 rows and 128 weight rows x 128 bytes
  static constexpr int kAccBufs = kPair ? 2 : 4;
  static constexpr int kTmemCols = kAccBufs * kTile;
  static constexpr int kCols = kTile / 2;              // columns of an epilogue warpgroup
  static constexpr int kOutBytes = Mode == kModeSplit ? 0 : kGroupedEpiWarps * 4096;  // 32 rows x 128 bytes per warp
  static constexpr int kStages = (kSmemMax - 1024 - kGroupedReserve - kScaleBytes - kOutBytes) / kStageBytes;
  static constexpr size_t kSmemBytes =
      static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kScaleBytes + kGroupedReserve + 1024;
  static constexpr uint32_t kIdesc = make_idesc(kTile, kTile, true);
  static_assert(kStages >= 4, "ring depth");
  static_assert(kStages * kStageBytes >= 128 * kPartialPitch * 4, "partial sums fit the ring");
};

constexpr int kChunk = 16;  // columns of one TMEM load
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&v)[16]) { tmem_ld16u(taddr, v); }
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld32(taddr, v); }
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&v)[8]) { tmem_ld8u(taddr, v); }
__device__ __forceinline__ void pin(uint32_t (&v)[8]) {
  asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]));
}
__device__ __forceinline__ void pin(uint32_t (&v)[16]) { pin16(v); }
__device__ __forceinline__ void pin(uint32_t (&v)[32]) { pin32(v); }

struct Tile {
  int g, row0, rows, col0;  // first row of the batch, rows to store, first column
};

template <int Mode>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* off, const int* first, int t) {
  using C = Cfg<Mode>;
  Tile r;
  r.g = group_of_tile(first, a.G, t);
  const int i = t - first[r.g];
  const int m = i / a.n_tiles;
  r.col0 = (i - m * a.n_tiles) * C::kTile;
  r.row0 = off[r.g] + m * C::kTile;
  r.rows = min(C::kTile, off[r.g + 1] - r.row0);
  return r;
}

template <int Mode>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_fp8_kernel(const __grid_constant__ RowMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_out, const Args args) {
  using C = Cfg<Mode>;
  constexpr bool kPair = C::kPair, kSplit = Mode == kModeSplit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + static_cast<size_t>(C::kStages) * C::kStageBytes;
  float* factors = reinterpret_cast<float*>(staging + C::kOutBytes);
  uint8_t* reserve = staging + C::kOutBytes + kScaleBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(reserve);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kAccBufs;
  uint64_t* factor_full = acc_empty + C::kAccBufs;    // [column half][slot]
  uint64_t* factor_empty = factor_full + 2 * kBatches;
  uint64_t* drain = factor_empty + 2 * kBatches;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scan = reinterpret_cast<int*>(reserve + 640);
  int* off = reinterpret_cast<int*>(reserve + 1024);
  int* first = off + kMaxGroups + 4;
  static_assert((2 * C::kStages + 2 * C::kAccBufs + 4 * kBatches + 1) * 8 + 8 <= 640, "barriers overlap the scan buffer");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = kPair || kSplit ? static_cast<int>(cluster_rank()) : 0;  // rank in the cluster
  const int rank = kPair ? cta : 0;                                        // half of the tile
  const bool leader = rank == 0;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kGroupedEpiWarps * C::kCtas);
    }
    for (int b = 0; b < 2 * kBatches; ++b) {
      mbar_init(&factor_full[b], 1);
      mbar_init(&factor_empty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x.map[4]);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) tmem_alloc_for<kPair>(tmem_slot, C::kTmemCols);
  pdl_wait();
  tc_fence_before();
  const int num_tiles = build_group_tables<kThreads>(args.offsets, args.M, args.G, C::kTile, args.n_tiles, off, first,
                                                     scan);
  if constexpr (kPair) cluster_barrier();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int cluster_size = kSplit ? args.splits : C::kCtas;
  const int first_tile = static_cast<int>(blockIdx.x) / cluster_size;
  const int stride = static_cast<int>(gridDim.x) / cluster_size;  // kSplit: no cluster takes a second tile
  const int kb0 = kSplit ? args.k_blocks * cta / args.splits : 0;
  const int kb1 = kSplit ? args.k_blocks * (cta + 1) / args.splits : args.k_blocks;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------------- producer (of each CTA)
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at<Mode>(args, off, first, t);
        auto loaded = [&](int r) {  // rows that CTA r loads
          const int n = min(128, tl.rows - 128 * r);
          return n > 0 ? row_map_rows(row_map_index(n)) : 0;
        };
        const int rows = loaded(rank);
        const CUtensorMap* map = &tm_x.map[rows > 0 ? row_map_index(rows) : 0];
        const uint32_t bytes = kPair ? (loaded(0) + loaded(1)) * 128 + 32768 : rows * 128 + 16384;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bar(&empty[stage], phase ^ 1u, abort_flag, args.status, kWhereGroupedProducer)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + static_cast<size_t>(stage) * C::kStageBytes;
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t bar = kPair ? in_cta(&full[stage], 0) : smem_u32(&full[stage]);
          if (rows > 0) load_2d<kPair>(a, map, bar, kb * 128, tl.row0 + 128 * rank, pol);
          load_3d<kPair>(a + 16384, &tm_w, bar, kb * 128, tl.col0 + 128 * rank, tl.g, pol);
          ++fills;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) drain_copies(full, C::kStages, fills);  // the leader's barriers count both CTAs' copies
    } else if (warp == 1 && lane == 0 && leader) {
      // ---------------------------------------------------------------- MMA issuer
      int stage = 0, abuf = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereGroupedMma) &&
               wait_bar(&full[stage], phase, abort_flag, args.status, kWhereGroupedMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(abuf * C::kTile);
          const uint32_t a = smem_u32(smem + static_cast<size_t>(stage) * C::kStageBytes), b = a + 16384;
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_fp8_for<kPair>(d, smem_desc_sw128(a + 32 * s), smem_desc_sw128(b + 32 * s), C::kIdesc, s > 0 ? 1u : 0u);
          commit_for<kPair>(&acc_full[abuf]);
          commit_for<kPair>(&empty[stage]);
          if (++abuf == C::kAccBufs) {
            abuf = 0;
            aphase ^= 1u;
          }
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every MMA this thread issued has completed once `drain` flips
      // (waited on even after an abort: TMEM must not be freed under a running MMA)
      commit_for<kPair>(drain);
      drain_mma(drain, args.status);
    } else if (warp >= 2) {
      // ---------------------------------------------------------------- factors of column half warp - 2
      const int g = warp - 2;
      const int n_blocks = (args.N + 127) / 128;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at<Mode>(args, off, first, t);
        const int n = min((tl.col0 + C::kCols * g) / 128, n_blocks - 1);
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
          if (lane == 0) mbar_arrive(&factor_full[g * kBatches + slot]);
          if (++slot == kBatches) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    const int g = (warp - 4) >> 2;        // column half
    const int row = 32 * q + lane;        // accumulator row
    uint8_t* out_box = staging + static_cast<size_t>(warp - 4) * 4096;
    const uint32_t lane_addr = (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(C::kCols * g);
    const uint32_t empty_bar = kPair ? in_cta(acc_empty, 0) : smem_u32(acc_empty);
    const float* my_factors = factors + g * kBatches * kBatch * 128 + row;
    uint32_t fphase = 0;
    int slot = 0;
    int abuf = 0;
    uint32_t aphase = 0;
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at<Mode>(args, off, first, t);
      const int rows = tl.rows - 128 * rank;            // of this CTA's half
      const int col = tl.col0 + C::kCols * g;           // first column of this thread
      const bool live = 32 * q < rows && col < args.N;  // this warp has something to store
      float acc[C::kCols];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i] = 0.f;
      for (int kb = kb0; kb < kb1 && ok; kb += kBatch) {
        // the factors of the next blocks
        ok = warp_wait_bar(&factor_full[g * kBatches + slot], fphase, abort_flag, args.status, kWhereGroupedEpilogue);
        if (!ok) break;
        float f[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) f[j] = my_factors[(slot * kBatch + j) * 128];
        __syncwarp();
        if (lane == 0) mbar_arrive(&factor_empty[g * kBatches + slot]);
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
          const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * C::kTile);
          uint32_t v[2][kChunk];
          if (live) load_chunk(d, v[0]);
#pragma unroll
          for (int c = 0; c < C::kCols / kChunk; ++c) {
            if (live) {
              tmem_wait_ld();
              pin(v[c & 1]);
              if (c + 1 < C::kCols / kChunk) load_chunk(d + kChunk * (c + 1), v[(c + 1) & 1]);
            }
            if (c + 1 == C::kCols / kChunk) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_in_cluster(empty_bar + 8 * abuf);
            }
            if (live) {
#pragma unroll
              for (int i = 0; i < kChunk; i += 2)
                ffma2f(acc[kChunk * c + i], acc[kChunk * c + i + 1], v[c & 1][i], v[c & 1][i + 1], f[j]);
            }
          }
          if (++abuf == C::kAccBufs) {
            abuf = 0;
            aphase ^= 1u;
          }
        }
      }
      if (!ok) break;
      if constexpr (kSplit) {
        // this CTA's share of the sums, for all CTAs of the cluster (the ring is idle: its last MMA is done)
        if (live && row < rows) {
          float* p = reinterpret_cast<float*>(smem) + row * kPartialPitch + C::kCols * g;
#pragma unroll
          for (int c = 0; c < C::kCols; c += 4)
            *reinterpret_cast<float4*>(p + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        }
        continue;
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
          for (int c = 0; c < C::kCols; c += 32) {
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
          for (int c = 0; c < C::kCols; c += 64) {
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
        for (int c = 0; c < C::kCols; c += 8) {
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
    if (!kSplit && lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (kSplit) {
    cluster_barrier();  // every CTA's partial sums are written
    if (first_tile < num_tiles) {
      const Tile tl = tile_at<Mode>(args, off, first, first_tile);
      add_partials<kThreads>(smem, cta, args.splits, min(tl.rows, 128), min(128, args.N - tl.col0), args.out,
                             static_cast<long long>(tl.row0) * args.ldo + tl.col0, args.ldo, args.out_f32, false);
    }
    cluster_barrier();  // no CTA leaves before the others have read its sums
  } else if constexpr (kPair) {
    cluster_barrier();  // the leader's MMAs read this CTA's shared memory: leave together
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_free_for<kPair>(tmem_base, C::kTmemCols);
  }
}

template <int Mode>
cudaError_t launch_tiles(const GroupedProblem& p, int splits, cudaStream_t s) {
  using C = Cfg<Mode>;
  constexpr auto kern = grouped_fp8_kernel<Mode>;
  // the register split waits for ever if the kernel is launched with fewer registers than it redistributes
  cudaError_t e = prepare_kernel<kern>(C::kSmemBytes, kLaunchRegs);
  if (e != cudaSuccess) return e;
  Args a{};
  a.M = p.M;
  a.G = p.G;
  a.N = p.N;
  a.k_blocks = (p.K + 127) / 128;
  a.n_tiles = (p.N + C::kTile - 1) / C::kTile;
  a.splits = splits;
  a.offsets = p.offsets;
  a.x_scale = p.a_scale;
  a.w_scale = p.b_scale;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.status = p.status;
  RowMaps tm_x;
  CUtensorMap tm_w, tm_out;
  if (!make_row_maps(&tm_x, p.a, p.M, p.K, p.lda, 1) ||
      !make_grouped_map(&tm_w, p.b, p.G, p.N, p.K, p.K, 1, 128) ||
      !make_store_map(&tm_out, p.out, 1, p.M, p.N, p.ldo, p.out_f32))
    return cudaErrorInvalidValue;
  const long long tiles = (static_cast<long long>(p.M) / C::kTile + (p.M < p.G ? p.M : p.G)) * a.n_tiles;
  if constexpr (Mode == kModeSingle) {
    const unsigned grid = static_cast<unsigned>(tiles < p.num_sms ? tiles : p.num_sms);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), C::kSmemBytes, s, tm_x, tm_w, tm_out, a);
  } else {
    return launch_clusters<kern>(kThreads, splits, tiles, Mode == kModePair, C::kSmemBytes, s, tm_x, tm_w, tm_out, a);
  }
}

}  // namespace

cudaError_t launch_grouped_fp8(const GroupedProblem& p, cudaStream_t stream) {
  const long long single = row_tiles(p.M, p.G, 128) * ((p.N + 127) / 128);
  const int splits = choose_splits(single, p.num_sms, (p.K + 127) / 128);
  if (splits > 1) return launch_tiles<kModeSplit>(p, splits, stream);
  // A pair takes 1.25 times as long for a K block of its 256 x 256 tile as a CTA for its 128 x 128 (0.6 against
  // 0.48 us), so it wins unless the larger tiles leave SMs idle or rows empty: N = 4096, K = 7168: 512 rows 31 us
  // in single tiles, 37 in pairs; 1024 rows 57 and 38 us.
  const int sms = p.num_sms, pairs = p.num_sms / 2;
  const long long pair = row_tiles(p.M, p.G, 256) * ((p.N + 255) / 256);
  const bool use_pair = 5 * ((pair + pairs - 1) / pairs) <= 4 * ((single + sms - 1) / sms);
  return use_pair ? launch_tiles<kModePair>(p, 2, stream) : launch_tiles<kModeSingle>(p, 1, stream);
}

}  // namespace moe
