// bf16 matrix products grouped by expert with ragged sizes, on the
// 5th-generation tensor cores (tcgen05, sm_100a).  Group g owns rows
// [off[g], off[g + 1]):
//
//   forward : y[r, :]  = x[r, :] . w[g]^T
//   dx      : dx[r, :] = dy[r, :] . w[g]
//   dw      : dw[g]    = dy_g^T . x_g               (reduction over g's rows)
//
// No operand is copied, padded or transposed in memory: the tensor core reads
// K-major tiles (x, dy, and w in the forward product) and MN-major tiles (w in
// dx; dy and x in dw) alike, so every product takes the tensors as they lie.
//
// forward, dx: the weight fills the MMA's M side and the group's rows its N
// side, because N comes in steps of 16 or 32 and M only whole: a group's rows
// are cut into equal tiles of at most 256 (128), each rounded up by less than a
// step, so a ragged group wastes little and one row costs little more than
// its weights.  A tile that runs past its group's end computes rows of the
// next group and does not store them.
// dw: the rows are the reduction axis; those past the group's end in its last
// stage are cleared in shared memory before the MMA reads them.
//
// kPair: a cluster of two CTAs computes a 256 x 256 tile (cta_group::2): each
// SM loads 128 of the 256 A rows and half of the B rows, so a stage moves 32 KB
// into an SM for 512 cycles of MMA, which the shared-memory port keeps up with
// (a 128 x 256 tile of one SM needs 48 KB).  kSingle: one CTA computes
// 128 x 128: more and smaller tiles for small problems.
//
// kSplit: a cluster of up to eight CTAs shares the reduction of one 128 x 128
// tile, each leaves its partial sums in shared memory and all add a part of
// them up, in rank order: where tiles are few, all SMs stream operands.
//
// Persistent (kSplit: one tile per cluster), 10 warps per CTA: TMA producer,
// MMA issuer (of the leader CTA), eight epilogue warps; the accumulator is
// double-buffered in TMEM, so a tile's stores run under the next tile's
// products.
//
// On a B200: 8192 x 4096 x 4096 forward and dx 176 us (1560 TFLOP/s, 0.95 of
// the measured peak), dw 191 us; 32768 rows over 128 experts of 4096 x 1536
// forward and dx 400 us, dw 500 us; 512 rows over the same experts 243 us,
// 0.99 of HBM.  Forward and dx of that training batch are bound by the power
// limit (dx: a launch by itself 377 us at 1965 MHz, back to back 477 us at
// 1005 MHz).  dw is not: by itself it takes 519 us at 1965 MHz, the tensor
// pipe 39 % active and DRAM at half its rate.  Its reductions are four stages
// long, and it waits between them: stores and products hardly overlap (278 us
// without its stores, 273 without its products).
#include "grouped_common.cuh"

namespace moe {

namespace {

struct Args {
  int M, G;
  int m_rows;        // rows of the MMA's M side: N (fwd, dw), K (dx)
  int m_tiles;
  int cols;          // dw: K
  int n_tiles;       // dw: column tiles
  int red;           // fwd: K, dx: N
  const int32_t* offsets;
  void* out;
  long long ldo;     // fwd, dx: elements between rows of out
  int splits;        // kModeSplit: CTAs per cluster
  int out_f32, accumulate;
  int wide_a, wide_b;  // an MN-major operand's 128 columns are one box (its row is a multiple of 64 columns)
  int* status;
};

constexpr int kThreads = 320;

template <int Kind, int Mode>
struct Cfg {
  static constexpr bool kPair = Mode == kModePair;
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kMTile = 128 * kCtas;
  static constexpr int kNTile = 128 * kCtas;           // most N columns of a tile
  static constexpr int kABytes = 16384;                // 128 rows x 128 bytes
  static constexpr int kBBytes = 16384;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr bool kMnA = Kind != kGroupedFwd;
  static constexpr bool kMnB = Kind == kGroupedDw;
  static constexpr int kTmemCols = 2 * kNTile;
  // dw: each epilogue warp stages boxes of 32 rows x 64 bytes for TMA stores (128 bytes would cost a stage of the
  // ring, and the short reductions need them: dw of 32768 rows over 128 experts 525 us with five, 510 with six)
  static constexpr int kOutBytes = Kind == kGroupedDw && Mode != kModeSplit ? kGroupedEpiWarps * 2048 : 0;
  static constexpr int kStages = (kSmemMax - 1024 - kGroupedReserve - kOutBytes) / kStageBytes;
  static constexpr size_t kSmemBytes =
      static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kGroupedReserve + 1024;
  static constexpr uint32_t kIdesc =
      make_idesc(kMTile, 0, false) | (kMnA ? 1u << 15 : 0u) | (kMnB ? 1u << 16 : 0u);
  static_assert(kStages >= 4 && kStages <= 16, "ring depth");
  static_assert(kStages * kStageBytes >= 128 * kPartialPitch * 4, "partial sums fit the ring");
};

struct Tile {
  int g;
  int m0;         // first row of the M side
  int n0, n;      // first N column (fwd, dx: row of the batch; dw: column of out) and the MMA's N
  int valid;      // N columns to store
  int red0, red;  // dw: the group's first row and row count; otherwise 0 and the reduction length
};

template <int Kind, int Mode>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* off, const int* first, int t) {
  using C = Cfg<Kind, Mode>;
  Tile r;
  if constexpr (Kind == kGroupedDw) {
    const int per_group = a.m_tiles * a.n_tiles;
    r.g = t / per_group;
    const int i = t - r.g * per_group;
    const int m = i / a.n_tiles;
    r.m0 = m * C::kMTile;
    r.n0 = (i - m * a.n_tiles) * C::kNTile;
    r.n = C::kNTile;
    r.valid = min(C::kNTile, a.cols - r.n0);
    r.red0 = off[r.g];
    r.red = off[r.g + 1] - r.red0;
  } else {
    r.g = group_of_tile(first, a.G, t);
    const int i = t - first[r.g];
    const int row0 = off[r.g], rows = off[r.g + 1] - row0;
    const int parts = (rows + C::kNTile - 1) / C::kNTile;
    constexpr int kStep = 16 * C::kCtas;  // granularity of N: each CTA of a pair loads half in boxes of 16
    const int each = ((rows + parts - 1) / parts + kStep - 1) / kStep * kStep;  // <= kNTile
    const int p = i / a.m_tiles;
    r.m0 = (i - p * a.m_tiles) * C::kMTile;
    r.n0 = row0 + p * each;
    r.n = each;
    r.valid = min(each, rows - p * each);  // at least one: rows > (parts - 1) * kNTile >= (parts - 1) * each
    r.red0 = 0;
    r.red = a.red;
  }
  return r;
}

template <int Kind, int Mode>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_bf16_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ RowMaps tm_b,
                        const __grid_constant__ CUtensorMap tm_out, const Args args) {
  using C = Cfg<Kind, Mode>;
  constexpr bool kPair = C::kPair, kSplit = Mode == kModeSplit;
  // dw in a pair: a stage in which the group ends is counted, and cleared, by each CTA for itself, and the peer
  // tells the leader when its half is ready (that for every stage cost 11 % of 8192 x 4096 x 4096)
  constexpr bool kTails = kPair && Kind == kGroupedDw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + static_cast<size_t>(C::kStages) * C::kStageBytes;
  uint8_t* reserve = staging + C::kOutBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(reserve);
  uint64_t* empty = full + C::kStages;
  uint64_t* peer_full = empty + C::kStages;
  uint64_t* tail_full = peer_full + C::kStages;
  uint64_t* acc_full = tail_full + C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* beat = tmem_slot + 2;  // stages that the producer has filled
  int* scan = reinterpret_cast<int*>(reserve + 640);
  int* off = reinterpret_cast<int*>(reserve + 1024);
  int* first = off + kMaxGroups + 4;
  static_assert((4 * C::kStages + 5) * 8 + 12 <= 640, "barriers overlap the scan buffer");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = kPair || kSplit ? static_cast<int>(cluster_rank()) : 0;  // rank in the cluster
  const int rank = kPair ? cta : 0;                                        // half of the tile
  const bool leader = rank == 0;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&peer_full[s], 1);
      mbar_init(&tail_full[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kGroupedEpiWarps * C::kCtas);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *beat = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b.map[0]);
  }
  if (warp == 1) tmem_alloc_for<kPair>(tmem_slot, C::kTmemCols);
  pdl_wait();
  tc_fence_before();
  int num_tiles = build_group_tables<kThreads>(args.offsets, args.M, args.G, C::kNTile, args.m_tiles, off,
                                               Kind == kGroupedDw ? nullptr : first, scan);
  if constexpr (Kind == kGroupedDw) num_tiles = args.G * args.m_tiles * args.n_tiles;
  if constexpr (kPair) cluster_barrier();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int cluster_size = kSplit ? args.splits : C::kCtas;
  const int first_tile = static_cast<int>(blockIdx.x) / cluster_size;
  const int stride = static_cast<int>(gridDim.x) / cluster_size;  // kSplit: no cluster takes a second tile
  // the part of a tile's reduction that this CTA takes
  auto red_begin = [&](const Tile& tl) { return kSplit ? (tl.red + 63) / 64 * cta / args.splits * 64 : 0; };
  auto red_end = [&](const Tile& tl) {
    return kSplit ? min(tl.red, (tl.red + 63) / 64 * (cta + 1) / args.splits * 64) : tl.red;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (of each CTA)
    // dw: the rows are read again by every tile of their group, the gradient passing by is not read (8192 x 4096 x
    // 4096: 194 us, 199 without the hint; on the weights or rows of the other two it costs up to 5 %)
    const uint64_t pol = Kind == kGroupedDw ? policy_evict_last() : policy_evict_normal();
    int stage = 0;
    uint32_t phase = 0;
    long long fills = 0;
    uint32_t tails = 0, tail_odd = 0;  // kTails: stages with tails of the peer's own, and the parity of their number
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at<Kind, Mode>(args, off, first, t);
      const int m0 = tl.m0 + 128 * rank;
      const int half = tl.n / C::kCtas;           // N columns that this CTA loads
      const int n0 = tl.n0 + half * rank;
      const int box = row_map_index(half);        // fwd, dx: one box holds them (dw: boxes of 64 columns)
      const uint32_t bytes = C::kABytes + (Kind == kGroupedDw ? half : row_map_rows(box)) * 128;
      const int k1 = red_end(tl);
      for (int k = red_begin(tl); k < k1; k += 64) {
        ok = warp_wait_bar(&empty[stage], phase ^ 1u, abort_flag, args.status, kWhereGroupedProducer);
        if (!ok) break;
        if (elect_lane()) {
          *beat = static_cast<uint32_t>(fills) + 1;
          uint8_t* a = smem + static_cast<size_t>(stage) * C::kStageBytes;
          uint8_t* b = a + C::kABytes;
          uint32_t bar = smem_u32(&full[stage]);
          if (kTails && k + 64 > tl.red) {  // the group ends here: each CTA counts its own copies
            uint64_t* own = leader ? &full[stage] : &tail_full[stage];
            mbar_arrive_expect_tx(own, bytes);
            bar = in_cta(own, rank);
          } else if (kPair) {               // copies of both CTAs count on the leader's barrier
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
            bar = in_cta(&full[stage], 0);
          } else {
            mbar_arrive_expect_tx(&full[stage], bytes);
          }
          if constexpr (Kind == kGroupedFwd) {
            load_3d<kPair>(a, &tm_a, bar, k, m0, tl.g, pol);
          } else {
            const int y = tl.red0 + k, z = Kind == kGroupedDx ? tl.g : 0;
            if (args.wide_a) {
              load_4d<kPair>(a, &tm_a, bar, 0, y, m0 >> 6, z, pol);
            } else {
              load_3d<kPair>(a, &tm_a, bar, m0, y, z, pol);
              load_3d<kPair>(a + 8192, &tm_a, bar, m0 + 64, y, z, pol);
            }
          }
          if constexpr (Kind != kGroupedDw) {
            load_2d<kPair>(b, &tm_b.map[box], bar, k, n0, pol);
          } else if (args.wide_b) {
            load_4d<kPair>(b, &tm_b.map[0], bar, 0, tl.red0 + k, n0 >> 6, 0, pol);
          } else {
            load_3d<kPair>(b, &tm_b.map[0], bar, n0, tl.red0 + k, 0, pol);
            load_3d<kPair>(b + 8192, &tm_b.map[0], bar, n0 + 64, tl.red0 + k, 0, pol);
          }
        }
        __syncwarp();
        if (kTails && k + 64 > tl.red) {
          tails |= 1u << stage;
          tail_odd ^= 1u << stage;
        }
        ++fills;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && leader) drain_copies(full, C::kStages, fills);  // the leader's barriers count both CTAs' copies
    if (kTails && !ok && !leader) {                         // but for the peer's tails
      for (int i = 0; i < C::kStages; ++i)
        if (tails >> i & 1u) drain_copies(&tail_full[i], 1, 2 - (tail_odd >> i & 1u));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    int stage = 0, abuf = 0;
    uint32_t phase = 0, aphase = 0;
    uint32_t tails = 0;  // kTails: phase of each stage's tail barriers
    bool ok = true;
    auto next_stage = [&](int n) {
      stage += n;
      while (stage >= C::kStages) {
        stage -= C::kStages;
        phase ^= 1u;
      }
    };
    // the rows behind the group's end in a stage with `live` of them, cleared up to the next step of 16
    // (the swizzle permutes 16-byte pieces inside a 128-byte row only, so whole rows are cleared)
    auto clear_tail = [&](uint8_t* st, int live) {
      const int dead = (live + 15) / 16 * 16 - live;
      for (int i = lane; i < 4 * dead * 8; i += 32) {
        const int box = i / (dead * 8), r = i / 8 % dead, c = i & 7;
        *reinterpret_cast<uint4*>(st + box * 8192 + (live + r) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    if (leader) {
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at<Kind, Mode>(args, off, first, t);
        const int k0 = red_begin(tl), k1 = red_end(tl);
        if (k0 >= k1) continue;
        ok = warp_wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereGroupedMma);
        if (!ok) break;
        const uint32_t idesc = C::kIdesc | (static_cast<uint32_t>(tl.n >> 3) << 17);
        const uint32_t d = tmem_base + static_cast<uint32_t>(abuf * C::kNTile);
        for (int k = k0; k < k1; k += 64) {
          ok = warp_wait_bar(&full[stage], phase, abort_flag, args.status, kWhereGroupedMma);
          if (!ok) break;
          uint8_t* st = smem + static_cast<size_t>(stage) * C::kStageBytes;
          int steps = 4;
          if (Kind == kGroupedDw && k + 64 > tl.red) {
            steps = (tl.red - k + 15) / 16;
            clear_tail(st, tl.red - k);
            if constexpr (kTails) {
              ok = warp_wait_peer(&peer_full[stage], tails >> stage & 1u, abort_flag, args.status, kWhereGroupedMma);
              if (!ok) break;
              tails ^= 1u << stage;
            }
          }
          tc_fence_after();
          if (elect_lane()) {
            const uint32_t a = smem_u32(st), b = a + C::kABytes;
            const uint64_t ad = C::kMnA ? smem_desc_mn_sw128(a) : smem_desc_sw128(a);
            const uint64_t bd = C::kMnB ? smem_desc_mn_sw128(b) : smem_desc_sw128(b);
#pragma unroll
            for (int s = 0; s < 4; ++s) {  // 16 of the reduction further: 2048 bytes (MN-major) or 32
              if (Kind == kGroupedDw && s >= steps) break;
              mma_bf16_for<kPair>(d, ad + (C::kMnA ? 128 : 2) * s, bd + (C::kMnB ? 128 : 2) * s, idesc,
                                  (k > k0 || s > 0) ? 1u : 0u);
            }
            commit_for<kPair>(&empty[stage]);
          }
          __syncwarp();
          next_stage(1);
        }
        if (!ok) break;
        if (elect_lane()) commit_for<kPair>(&acc_full[abuf]);
        __syncwarp();
        abuf ^= 1;
        if (abuf == 0) aphase ^= 1u;
      }
    } else if constexpr (kTails) {
      // the peer's tails: cleared here, then handed to the leader
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at<Kind, Mode>(args, off, first, t);
        next_stage(tl.red / 64);
        if (tl.red % 64 == 0) continue;
        ok = warp_wait_bar(&tail_full[stage], tails >> stage & 1u, abort_flag, args.status, kWhereGroupedMma, beat);
        if (!ok) break;
        tails ^= 1u << stage;
        clear_tail(smem + static_cast<size_t>(stage) * C::kStageBytes, tl.red % 64);
        if (lane == 0) arrive_in_cluster_release(in_cta(&peer_full[stage], 0));
        next_stage(1);
      }
    }
    // every MMA that the elected lane issued has completed once `drain` flips
    // (waited on even after an abort: TMEM must not be freed under a running MMA)
    if (leader) {
      if (elect_lane()) commit_for<kPair>(drain);
      __syncwarp();
      drain_mma(drain, args.status);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    const int g = (warp - 2) >> 2;        // the two groups share the accumulator's columns
    const int row = 32 * q + lane;        // accumulator row
    const uint32_t lane_addr = static_cast<uint32_t>(32 * q) << 16;
    uint8_t* out_box = staging + static_cast<size_t>(warp - 2) * 2048;
    const uint32_t empty_bar = kPair ? in_cta(acc_empty, 0) : smem_u32(acc_empty);
    int abuf = 0;
    uint32_t aphase = 0;
    for (int t = first_tile; t < num_tiles; t += stride) {
      const Tile tl = tile_at<Kind, Mode>(args, off, first, t);
      const int m = tl.m0 + 128 * rank + row;                // row of the M side
      const bool live = tl.m0 + 128 * rank + 32 * q < args.m_rows;  // this warp has something to store
      const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * C::kNTile);
      const bool any = red_begin(tl) < red_end(tl);  // otherwise there is no accumulator: zeros
      if (any) {
        // (over a tile's whole reduction: up to 2^30 long, seconds)
        if (!warp_wait_bar(&acc_full[abuf], aphase, abort_flag, args.status, kWhereGroupedEpilogue, beat)) break;
        tc_fence_after();
      }
      if constexpr (Kind != kGroupedDw) {
        // a lane holds one output column of every row
        if (live) {
          const int chunks = (tl.valid + 15) / 16;
          for (int c = g; c < chunks; c += 2) {
            __syncwarp();  // the stores branch by lane; a TMEM load wants the warp converged
            float v[16];
            if (any) {
              uint32_t u[16];
              tmem_ld16u(d + 16 * c, u);
              tmem_wait_ld();
              pin16(u);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = 0.f;
            }
            const int n = min(16, tl.valid - 16 * c);
            if constexpr (kSplit) {
              // this CTA's share of the sums, for all CTAs of the cluster (the ring is idle: its last MMA is done)
              float* p = reinterpret_cast<float*>(smem) + 16 * c * kPartialPitch + row;
#pragma unroll
              for (int i = 0; i < 16; ++i) p[i * kPartialPitch] = v[i];
            } else {
              store_columns16(v, args.out, (static_cast<long long>(tl.n0) + 16 * c) * args.ldo, args.ldo, m, args.m_rows,
                              n, args.out_f32);
            }
          }
        }
        if (any) {
          tc_fence_before();
          __syncwarp();
          if (elect_lane()) arrive_in_cluster(empty_bar + 8 * abuf);
        }
      } else {
        // a lane holds a row: 64 bytes of each go through shared memory as one TMA store of the warp's 32 rows
        // (it leaves out what lies behind the last row and column)
        constexpr int kCols = C::kNTile / 2;  // columns of this group
        const int step = args.out_f32 ? 16 : 32;
        // a group without rows adds nothing to an accumulated gradient
        const int end = live && !(args.accumulate && tl.red == 0) ? min(kCols, tl.valid - g * kCols) : 0;
        if constexpr (kSplit) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            if (c >= end) break;
            uint32_t v[32];
            if (any) {
              tmem_ld32(d + g * kCols + c, v);
              tmem_wait_ld();
              pin32(v);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
            uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<float*>(smem) + row * kPartialPitch + g * kCols + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        for (int c = 0; !kSplit && c < end; c += step) {
          __syncwarp();  // as above: one lane stores
          const int col = g * kCols + c;
          uint4 piece[4];
          if (args.out_f32) {
            uint32_t v[16];
            if (any) {
              tmem_ld16u(d + col, v);
              tmem_wait_ld();
              pin16(v);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) piece[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            uint32_t v[32];
            if (any) {
              tmem_ld32(d + col, v);
              tmem_wait_ld();
              pin32(v);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float f[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[8 * i + j]);
              piece[i] = pack_bf16x8(f);
            }
          }
          if (lane == 0) bulk_wait_read_all();  // the previous store has read the box
          __syncwarp();
          stage_row(out_box, lane, piece);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int m_first = tl.m0 + 128 * rank + 32 * q;
            if (args.accumulate)
              store_3d<true>(&tm_out, out_box, tl.n0 + col, m_first, tl.g);
            else
              store_3d<false>(&tm_out, out_box, tl.n0 + col, m_first, tl.g);
            bulk_commit();
          }
        }
        if (any) {
          tc_fence_before();
          __syncwarp();
          if (elect_lane()) arrive_in_cluster(empty_bar + 8 * abuf);
        }
      }
      if (any) {
        abuf ^= 1;
        if (abuf == 0) aphase ^= 1u;
      }
    }
    if (Kind == kGroupedDw && !kSplit && lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (kSplit) {
    cluster_barrier();  // every CTA's partial sums are written
    if (first_tile < num_tiles) {
      const Tile tl = tile_at<Kind, Mode>(args, off, first, first_tile);
      if constexpr (Kind == kGroupedDw) {
        if (!(args.accumulate && tl.red == 0))
          add_partials<kThreads>(smem, cta, args.splits, min(128, args.m_rows - tl.m0), tl.valid, args.out,
                                 (static_cast<long long>(tl.g) * args.m_rows + tl.m0) * args.cols + tl.n0, args.cols,
                                 args.out_f32, args.accumulate);
      } else {
        add_partials<kThreads>(smem, cta, args.splits, tl.valid, min(128, args.m_rows - tl.m0), args.out,
                               static_cast<long long>(tl.n0) * args.ldo + tl.m0, args.ldo, args.out_f32, false);
      }
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

template <int Kind, int Mode>
cudaError_t launch_tiles(const GroupedProblem& p, int splits, cudaStream_t s) {
  using C = Cfg<Kind, Mode>;
  constexpr auto kern = grouped_bf16_kernel<Kind, Mode>;
  cudaError_t e = prepare_kernel<kern>(C::kSmemBytes, 0);
  if (e != cudaSuccess) return e;
  Args a{};
  a.M = p.M;
  a.G = p.G;
  a.m_rows = Kind == kGroupedDx ? p.K : p.N;
  a.m_tiles = (a.m_rows + C::kMTile - 1) / C::kMTile;
  a.cols = p.K;
  a.n_tiles = (p.K + C::kNTile - 1) / C::kNTile;
  a.red = Kind == kGroupedFwd ? p.K : p.N;
  a.splits = splits;
  a.offsets = p.offsets;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.accumulate = p.accumulate;
  a.status = p.status;
  CUtensorMap tm_a, tm_out{};
  RowMaps tm_b{};
  long long tiles;
  bool ok;
  if constexpr (Kind == kGroupedDw) {
    // an empty batch has no rows to map: its tiles load nothing
    const long long rows = p.M > 0 ? p.M : 1;
    const void* dy = p.M > 0 ? p.a : p.out;
    const void* x = p.M > 0 ? p.b : p.out;
    const long long lddy = p.M > 0 ? p.lda : p.N, ldx = p.M > 0 ? p.ldb : p.K;
    a.wide_a = p.N % 64 == 0;
    a.wide_b = p.K % 64 == 0;
    ok = (a.wide_a ? make_wide_map(&tm_a, dy, 1, rows, p.N, lddy) : make_grouped_map(&tm_a, dy, 1, rows, p.N, lddy, 2, 64)) &&
         (a.wide_b ? make_wide_map(&tm_b.map[0], x, 1, rows, p.K, ldx)
                   : make_grouped_map(&tm_b.map[0], x, 1, rows, p.K, ldx, 2, 64)) &&
         make_store_map(&tm_out, p.out, p.G, p.N, p.K, p.K, p.out_f32, 64);
    tiles = static_cast<long long>(p.G) * a.m_tiles * a.n_tiles;
  } else {
    a.wide_a = Kind == kGroupedDx && p.K % 64 == 0;
    ok = (a.wide_a ? make_wide_map(&tm_a, p.b, p.G, p.N, p.K, p.K)
                   : make_grouped_map(&tm_a, p.b, p.G, p.N, p.K, p.K, 2, Kind == kGroupedFwd ? 128 : 64)) &&
         make_row_maps(&tm_b, p.a, p.M, a.red, p.lda, 2);
    tiles = (static_cast<long long>(p.M) / C::kNTile + (p.M < p.G ? p.M : p.G)) * a.m_tiles;
  }
  if (!ok) return cudaErrorInvalidValue;
  if constexpr (Mode == kModeSingle) {
    const unsigned grid = static_cast<unsigned>(tiles < p.num_sms ? tiles : p.num_sms);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), C::kSmemBytes, s, tm_a, tm_b, tm_out, a);
  } else {
    return launch_clusters<kern>(kThreads, splits, tiles, Mode == kModePair, C::kSmemBytes, s, tm_a, tm_b, tm_out, a);
  }
}

template <int Kind>
cudaError_t dispatch(const GroupedProblem& p, cudaStream_t s) {
  const long long m = Kind == kGroupedDx ? p.K : p.N;
  auto tiles = [&](int tile) {
    const long long m_tiles = (m + tile - 1) / tile;
    return Kind == kGroupedDw ? p.G * m_tiles * ((p.K + tile - 1) / tile) : row_tiles(p.M, p.G, tile) * m_tiles;
  };
  const long long red = Kind == kGroupedFwd ? p.K : (Kind == kGroupedDx ? p.N : p.M / p.G);
  using C = Cfg<Kind, kModeSplit>;
  int splits;
  const cudaError_t e = choose_splits<grouped_bf16_kernel<Kind, kModeSplit>>(
      tiles(128), p.num_sms, static_cast<int>((red + 63) / 64), kThreads, C::kSmemBytes, &splits);
  if (e != cudaSuccess) return e;
  if (splits > 1) return launch_tiles<Kind, kModeSplit>(p, splits, s);
  // a stage takes a pair about as long for its 256 x 256 tile as a CTA for its 128 x 128, so the pairs win where
  // the larger tiles do not need more rounds over the SMs
  const long long single_rounds = (tiles(128) + p.num_sms - 1) / p.num_sms;
  const long long pair_rounds = (tiles(256) + p.num_sms / 2 - 1) / (p.num_sms / 2);
  return pair_rounds < single_rounds || (pair_rounds == single_rounds && pair_rounds > 1)
             ? launch_tiles<Kind, kModePair>(p, 2, s)
             : launch_tiles<Kind, kModeSingle>(p, 1, s);
}

}  // namespace

namespace {

bool encode(CUtensorMap* map, CUtensorMapDataType type, int dims, const void* base, const cuuint64_t* size,
            const cuuint64_t* strides, const cuuint32_t* box,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, type, dims, const_cast<void*>(base), size, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cuuint64_t u64(long long v) { return static_cast<cuuint64_t>(v); }

}  // namespace

bool make_grouped_map(CUtensorMap* map, const void* base, int batches, long long rows, long long cols, long long ld,
                      int elem_bytes, int box_rows) {
  const cuuint64_t size[3] = {u64(cols), u64(rows), u64(batches)};
  const cuuint64_t strides[2] = {u64(ld * elem_bytes), u64(ld * rows * elem_bytes)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem_bytes), static_cast<cuuint32_t>(box_rows), 1};
  return encode(map, elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                batches > 0 ? 3 : 2, base, size, strides, box);
}

bool make_wide_map(CUtensorMap* map, const void* base, int batches, long long rows, long long cols, long long ld) {
  const cuuint64_t size[4] = {64, u64(rows), u64(cols / 64), u64(batches)};
  const cuuint64_t strides[3] = {u64(ld * 2), 128, u64(ld * rows * 2)};
  const cuuint32_t box[4] = {64, 64, 2, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, size, strides, box);
}

bool make_store_map(CUtensorMap* map, void* base, int batches, long long rows, long long cols, long long ld, bool f32,
                    int box_bytes) {
  const long long elem = f32 ? 4 : 2;
  const cuuint64_t size[3] = {u64(cols), u64(rows), u64(batches)};
  const cuuint64_t strides[2] = {u64(ld * elem), u64(ld * rows * elem)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_bytes / elem), 32, 1};
  return encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, size, strides,
                box, box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_row_maps(RowMaps* maps, const void* base, long long rows, long long cols, long long ld, int elem_bytes) {
  const int most = row_map_index(rows < 128 ? static_cast<int>(rows) : 128);  // no tile has more rows than there are
  for (int i = 0; i <= most; ++i)
    if (!make_grouped_map(&maps->map[i], base, 0, rows, cols, ld, elem_bytes, row_map_rows(i))) return false;
  return true;
}

cudaError_t launch_grouped(const GroupedProblem& p, cudaStream_t stream) {
  if (p.fp8) return launch_grouped_fp8(p, stream);
  switch (p.kind) {
    case kGroupedFwd: return dispatch<kGroupedFwd>(p, stream);
    case kGroupedDx: return dispatch<kGroupedDx>(p, stream);
    default: return dispatch<kGroupedDw>(p, stream);
  }
}

}  // namespace moe
