// FP8 (E4M3) matrix products with block scales, grouped by expert with ragged
// sizes, on the 5th-generation tensor cores (tcgen05, sm_100a):
//
//   y[r, n] = sum over 128-deep K blocks b of
//             x_scale[b, r] * w_scale[g(r), n / 128, b] * (x_b[r] . w_b[g(r), n])
//
// One group of all rows is the plain product.  Every K block has its own
// accumulator in TMEM, which the epilogue adds into fp32 registers times the
// two scales while the tensor core works on the next blocks.
//
// This file: few rows per group (grouped_fp8_pair.cu has the tiles for many).
// The weights fill the M side and up to 128 rows
// of the group the N side, which comes in steps of 16: a tile of a few rows
// costs the tensor core little (a 128 x 128 tile of 2 rows held the memory
// stream back: 512 rows over 256 groups of 7168 x 2048 took 613 us that way,
// 500 this way, and 467, 0.99 of HBM, with the deeper ring below).  An epilogue thread holds one column of up to 64 rows; the
// rows' factors are read from shared memory, the same for all lanes.
// kSplit: a cluster of up to eight CTAs shares the K blocks of one such tile,
// each leaves its partial sums in shared memory and all add a part of them
// up, in rank order: a product of a few rows streams its weights through all
// SMs instead of one per 128 columns.
//
// Row tiles start at any row; a tile that runs past its group's end computes
// rows of the next group and does not store them; no more rows than the group
// has are loaded, rounded up to a box of 16, 32, 64, 96 or 128.
//
// Persistent (kSplit: one tile per cluster), three warpgroups per CTA: the
// first holds the TMA producer, the MMA issuer and a warp that multiplies the
// scales and lays the factors of four K blocks at a time into shared memory;
// the other two are the epilogue.  (An epilogue thread must have no global load
// under way: its hand-offs wait for it, 1 to 2 us in every block that loaded a
// scale.)
#include "grouped_common.cuh"

namespace moe {

namespace {

constexpr int kThreads = 384;
// The scales' factors go through a ring of batches in shared memory: [slot][K block][row].
constexpr int kBatch = 4, kBatches = 3;
constexpr int kScaleBytes = kBatches * kBatch * 128 * 4;
constexpr int kTile = 128;            // columns, and most rows, of a tile
constexpr int kAccBufs = 4;
constexpr int kTmemCols = kAccBufs * kTile;
constexpr int kHalf = kTile / 2;      // most rows of an epilogue warpgroup
// K blocks lie one behind the other in a ring of bytes, each as long as its tile's rows need (128 weight rows and a
// box of 16 to 128 rows, 128 bytes each): eleven blocks of up to 16 rows are under way at a time, six of 128 (4096
// skewed rows over 256 groups of 7168 x 2048: 571 us, 593 with six of any size; 512 rows 467 and 497 us).  kSplit,
// whose CTAs all start on their only tile at once, has six of any size: more only delay the first (1 x 4096 x 7168:
// 9.9 us instead of 9.4).
constexpr int kWeightBytes = 16384;
constexpr int kMostBytes = kWeightBytes + 128 * 128;  // of a block
constexpr int kRingBytes = (kSmemMax - 1024 - kGroupedReserve - kScaleBytes) / 2048 * 2048;
constexpr int kMostStages = 12;                       // blocks in the ring
constexpr size_t kSmemBytes = static_cast<size_t>(kRingBytes) + kScaleBytes + kGroupedReserve + 1024;
static_assert(kRingBytes >= 6 * kMostBytes, "ring depth");
static_assert(kRingBytes >= 128 * kPartialPitch * 4, "partial sums fit the ring");

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

struct Tile {
  int g, col0;           // first column
  int row0, rows, n;     // first row, rows to store, and the MMA's N
};

__device__ __forceinline__ Tile tile_at(const Args& a, const int* off, const int* first, int t) {
  Tile r;
  r.g = group_of_tile(first, a.G, t);
  const int i = t - first[r.g];
  const int row0 = off[r.g], rows = off[r.g + 1] - row0;
  const int parts = (rows + kTile - 1) / kTile;
  const int each = ((rows + parts - 1) / parts + 15) / 16 * 16;  // equal parts, <= kTile
  const int p = i / a.n_tiles;
  r.col0 = (i - p * a.n_tiles) * kTile;
  r.row0 = row0 + p * each;
  r.rows = min(each, rows - p * each);  // at least one: rows > (parts - 1) * kTile >= (parts - 1) * each
  r.n = (r.rows + 15) / 16 * 16;        // (no more than the box that holds the rows)
  return r;
}

// bytes that are loaded for one K block of a tile
__device__ __forceinline__ int block_bytes(const Tile& tl) {
  return kWeightBytes + row_map_rows(row_map_index(tl.rows)) * 128;
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_fp8_kernel(const __grid_constant__ RowMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const Args args) {
  constexpr int kStages = kSplit ? 6 : kMostStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* factors = reinterpret_cast<float*>(smem + kRingBytes);
  uint8_t* reserve = reinterpret_cast<uint8_t*>(factors) + kScaleBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(reserve);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kAccBufs;
  uint64_t* factor_full = acc_empty + kAccBufs;
  uint64_t* factor_empty = factor_full + kBatches;
  uint64_t* drain = factor_empty + kBatches;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* lengths = reinterpret_cast<int*>(reserve + 512);  // of the ring's blocks (the producer's own)
  int* scan = reinterpret_cast<int*>(reserve + 640);
  int* off = reinterpret_cast<int*>(reserve + 1024);
  int* first = off + kMaxGroups + 4;
  static_assert((2 * kStages + 2 * kAccBufs + 2 * kBatches + 1) * 8 + 8 <= 512, "barriers overlap the lengths");
  static_assert(kMostStages * 4 <= 128, "lengths overlap the scan buffer");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = kSplit ? static_cast<int>(cluster_rank()) : 0;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kAccBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kGroupedEpiWarps);
    }
    for (int b = 0; b < kBatches; ++b) {
      mbar_init(&factor_full[b], 1);
      mbar_init(&factor_empty[b], kGroupedEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x.map[0]);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) tmem_alloc_for<false>(tmem_slot, kTmemCols);
  pdl_wait();
  tc_fence_before();
  const int num_tiles =
      build_group_tables<kThreads>(args.offsets, args.M, args.G, kTile, args.n_tiles, off, first, scan);
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int cluster_size = kSplit ? args.splits : 1;
  const int first_tile = static_cast<int>(blockIdx.x) / cluster_size;
  const int stride = static_cast<int>(gridDim.x) / cluster_size;  // kSplit: no cluster takes a second tile
  const int kb0 = kSplit ? args.k_blocks * cta / args.splits : 0;
  const int kb1 = kSplit ? args.k_blocks * (cta + 1) / args.splits : args.k_blocks;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_normal();
    int stage = 0;
    long long fills = 0;
    int pos = 0, used = 0, held = 0;  // where the next block goes; bytes and blocks not yet given back
    int oldest = 0;
    uint32_t phase = 0;               // of the oldest block's barrier (kSplit: of the stage's)
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at(args, off, first, t);
      const int box = row_map_index(tl.rows);
      const int bytes = block_bytes(tl);
      for (int kb = kb0; kb < kb1; ++kb) {
        if constexpr (kSplit) {
          ok = warp_wait_bar(&empty[stage], phase ^ 1u, abort_flag, args.status, kWhereGroupedProducer);
          if (!ok) break;
          pos = stage * kMostBytes;
        } else {
          const bool wrap = pos + bytes > kRingBytes;  // a block lies in one piece; the gap before it is its own
          const int gap = wrap ? kRingBytes - pos : 0;
          while (held == kStages || used + gap + bytes > kRingBytes) {
            ok = warp_wait_bar(&empty[oldest], phase, abort_flag, args.status, kWhereGroupedProducer);
            if (!ok) break;
            used -= lengths[oldest];
            --held;
            if (++oldest == kStages) {
              oldest = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (wrap) pos = 0;
          __syncwarp();  // the length just read may be that of the slot written next
          if (elect_lane()) lengths[stage] = gap + bytes;
          used += gap + bytes;
          ++held;
        }
        if (elect_lane()) {
          uint8_t* a = smem + pos;
          const uint32_t bar = smem_u32(&full[stage]);
          mbar_arrive_expect_tx(&full[stage], bytes);
          load_3d<false>(a, &tm_w, bar, kb * 128, tl.col0, tl.g, pol);
          load_2d<false>(a + kWeightBytes, &tm_x.map[box], bar, kb * 128, tl.row0, pol);
        }
        __syncwarp();
        pos += bytes;
        ++fills;
        if (++stage == kStages) {
          stage = 0;
          if (kSplit) phase ^= 1u;
        }
      }
    }
    if (!ok) drain_copies(full, kStages, fills);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    int stage = 0, pos = 0, abuf = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at(args, off, first, t);
      const int bytes = block_bytes(tl);
      const uint32_t idesc = make_idesc(kTile, 0, true) | (static_cast<uint32_t>(tl.n >> 3) << 17);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = warp_wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereGroupedMma) &&
             warp_wait_bar(&full[stage], phase, abort_flag, args.status, kWhereGroupedMma);
        if (!ok) break;
        tc_fence_after();
        if (kSplit) pos = stage * kMostBytes;  // as the producer does
        else if (pos + bytes > kRingBytes) pos = 0;
        if (elect_lane()) {
          const uint32_t d = tmem_base + static_cast<uint32_t>(abuf * kTile);
          const uint32_t a = smem_u32(smem + pos);
          const uint64_t ad = smem_desc_sw128(a), bd = smem_desc_sw128(a + kWeightBytes);
#pragma unroll
          for (int s = 0; s < 4; ++s) mma_fp8(d, ad + 2 * s, bd + 2 * s, idesc, s > 0 ? 1u : 0u);  // + 32 bytes
          mma_commit(&acc_full[abuf]);
          mma_commit(&empty[stage]);
        }
        __syncwarp();
        pos += bytes;
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
    if (elect_lane()) mma_commit(drain);
    __syncwarp();
    drain_mma(drain, args.status);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ factors
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at(args, off, first, t);
      const float* w = args.w_scale +
                       (static_cast<long long>(tl.g) * args.n_tiles + tl.col0 / kTile) * args.k_blocks;
      const float* x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = args.x_scale + tl.row0 + min(lane + 32 * i, tl.rows - 1);
      for (int kb = kb0; kb < kb1; kb += kBatch) {
        float xs[kBatch][4], ws[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int k = min(kb + j, kb1 - 1);
          ws[j] = w[k];
#pragma unroll
          for (int i = 0; i < 4; ++i) xs[j][i] = 32 * i < tl.rows ? x[i][static_cast<long long>(k) * args.M] : 0.f;
        }
        ok = warp_wait_bar(&factor_empty[slot], phase ^ 1u, abort_flag, args.status, kWhereGroupedProducer);
        if (!ok) break;
        float* f = factors + slot * kBatch * 128 + lane;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j * 128 + 32 * i] = xs[j][i] * ws[j];
        __syncwarp();
        if (elect_lane()) mbar_arrive(&factor_full[slot]);
        if (++slot == kBatches) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue: lanes are columns of y
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    const int g = (warp - 4) >> 2;        // row half
    const uint32_t lane_addr = static_cast<uint32_t>(32 * q) << 16;
    int slot = 0, abuf = 0;
    uint32_t fphase = 0, aphase = 0;
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at(args, off, first, t);
      const int half = (tl.n / 2 + 15) / 16 * 16;  // this group's rows: [half * g, half * g + half), in chunks of 16
      const int col = tl.col0 + 32 * q + lane;
      const int mine = tl.col0 + 32 * q < args.N ? min(half, tl.rows - half * g) : 0;  // rows to store
      const int chunks = (max(mine, 0) + 15) / 16;
      float acc[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf; ++i) acc[i] = 0.f;
      for (int kb = kb0; kb < kb1 && ok; kb += kBatch) {
        ok = warp_wait_bar(&factor_full[slot], fphase, abort_flag, args.status, kWhereGroupedEpilogue);
        if (!ok) break;
        const float* f = factors + slot * kBatch * 128 + half * g;
        for (int j = 0; j < kBatch && kb + j < kb1; ++j, f += 128) {
          ok = warp_wait_bar(&acc_full[abuf], aphase, abort_flag, args.status, kWhereGroupedEpilogue);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * kTile + half * g);
          uint32_t v[2][16];
          if (chunks > 0) tmem_ld16u(d, v[0]);
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c) {
            if (c >= chunks) break;
            tmem_wait_ld();
            pin16(v[c & 1]);
            if (c + 1 < kHalf / 16 && c + 1 < chunks) tmem_ld16u(d + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 s = *reinterpret_cast<const float4*>(f + 16 * c + i);
              ffma2v(acc[16 * c + i], acc[16 * c + i + 1], v[c & 1][i], v[c & 1][i + 1], s.x, s.y);
              ffma2v(acc[16 * c + i + 2], acc[16 * c + i + 3], v[c & 1][i + 2], v[c & 1][i + 3], s.z, s.w);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (elect_lane()) mbar_arrive(&acc_empty[abuf]);
          if (++abuf == kAccBufs) {
            abuf = 0;
            aphase ^= 1u;
          }
        }
        __syncwarp();
        if (elect_lane()) mbar_arrive(&factor_empty[slot]);
        if (++slot == kBatches) {
          slot = 0;
          fphase ^= 1u;
        }
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < kHalf / 16; ++c) {
        if (c >= chunks) break;
        if constexpr (kSplit) {
          // this CTA's share of the sums, for all CTAs of the cluster (the ring is idle: its last MMA is done)
          float* p = reinterpret_cast<float*>(smem) + (half * g + 16 * c) * kPartialPitch + 32 * q + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (16 * c + i < mine) p[i * kPartialPitch] = acc[16 * c + i];
        } else {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = acc[16 * c + i];
          store_columns16(v, args.out, (static_cast<long long>(tl.row0) + half * g + 16 * c) * args.ldo, args.ldo, col,
                          args.N, mine - 16 * c, args.out_f32);
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (kSplit) {
    cluster_barrier();  // every CTA's partial sums are written
    if (first_tile < num_tiles) {
      const Tile tl = tile_at(args, off, first, first_tile);
      add_partials<kThreads>(smem, cta, args.splits, tl.rows, min(kTile, args.N - tl.col0), args.out,
                             static_cast<long long>(tl.row0) * args.ldo + tl.col0, args.ldo, args.out_f32, false);
    }
    cluster_barrier();  // no CTA leaves before the others have read its sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_free_for<false>(tmem_base, kTmemCols);
  }
}

template <bool kSplit>
cudaError_t launch_columns(const GroupedProblem& p, int splits, cudaStream_t s) {
  constexpr auto kern = grouped_fp8_kernel<kSplit>;
  const cudaError_t e = prepare_kernel<kern>(kSmemBytes, 0);
  if (e != cudaSuccess) return e;
  Args a{};
  a.M = p.M;
  a.G = p.G;
  a.N = p.N;
  a.k_blocks = (p.K + 127) / 128;
  a.n_tiles = (p.N + kTile - 1) / kTile;
  a.splits = splits;
  a.offsets = p.offsets;
  a.x_scale = p.a_scale;
  a.w_scale = p.b_scale;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.status = p.status;
  RowMaps tm_x{};
  CUtensorMap tm_w;
  if (!make_row_maps(&tm_x, p.a, p.M, p.K, p.lda, 1) || !make_grouped_map(&tm_w, p.b, p.G, p.N, p.K, p.K, 1, 128))
    return cudaErrorInvalidValue;
  const long long tiles = (static_cast<long long>(p.M) / kTile + (p.M < p.G ? p.M : p.G)) * a.n_tiles;
  if constexpr (kSplit) {
    return launch_clusters<kern>(kThreads, splits, tiles, false, kSmemBytes, s, tm_x, tm_w, a);
  } else {
    const unsigned grid = static_cast<unsigned>(tiles < p.num_sms ? tiles : p.num_sms);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, s, tm_x, tm_w, a);
  }
}

}  // namespace

cudaError_t launch_grouped_fp8(const GroupedProblem& p, cudaStream_t stream) {
  const long long single = row_tiles(p.M, p.G, 128) * ((p.N + 127) / 128);
  int splits;
  const cudaError_t e = choose_splits<grouped_fp8_kernel<true>>(single, p.num_sms, (p.K + 127) / 128, kThreads,
                                                                kSmemBytes, &splits);
  if (e != cudaSuccess) return e;
  if (splits > 1) return launch_columns<true>(p, splits, stream);
  // A pair computes its 256 x 256 tile in the time that a CTA takes for 128 x 128, so it wins unless the larger tiles
  // leave SMs idle (N = 4096, K = 7168: 512 rows 32 us in pairs and 34 in single tiles, 1024 rows 33 and 64 us) or
  // most of their rows empty: single tiles fit a group's rows in steps of 16.
  const int sms = p.num_sms, pairs = p.num_sms / 2;
  const long long pair = row_tiles(p.M, p.G, 256) * ((p.N + 255) / 256);
  const bool use_pair = p.M / p.G > 128 && (pair + pairs - 1) / pairs <= (single + sms - 1) / sms;
  // Few such tiles and a long reduction: two pairs share each one's K blocks (256 x 5120 x 7168: 24 us, 30 without;
  // 640 x 2560 x 4096 17.7 and 19.7; 256 x 7168 x 2048 16 and 13).
  bool split_pair = false;
  if (p.M / p.G > 128 && 2 * pair <= pairs && p.K >= 32 * 128) {
    int most = 0;
    const cudaError_t err = fp8_pair_split_clusters(&most);
    if (err != cudaSuccess) return err;
    split_pair = pair <= most;
  }
  return use_pair || split_pair ? launch_grouped_fp8_pair(p, split_pair, stream) : launch_columns<false>(p, 1, stream);
}

}  // namespace moe
