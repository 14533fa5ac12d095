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
// each SM per K block; otherwise one CTA computes 128 x 128.
//
// Persistent, 10 warps per CTA: TMA producer, MMA issuer (of the leader CTA),
// two groups of four epilogue warps.
#include "grouped_common.cuh"

namespace moe {

namespace {

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

template <bool kPair>
struct Cfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTile = 128 * kCtas;            // rows and columns of a tile
  static constexpr int kStageBytes = 32768;            // this CTA's 128 rows and 128 weight rows x 128 bytes
  static constexpr int kAccBufs = kPair ? 2 : 4;
  static constexpr int kTmemCols = kAccBufs * kTile;
  static constexpr int kCols = kTile / 2;              // columns of an epilogue group
  static constexpr int kOutBytes = kGroupedEpiWarps * 4096;  // a box of 32 rows x 128 bytes per epilogue warp
  static constexpr int kStages = (kSmemMax - 1024 - kGroupedReserve - kOutBytes) / kStageBytes;
  static constexpr size_t kSmemBytes =
      static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kGroupedReserve + 1024;
  static constexpr uint32_t kIdesc = make_idesc(kTile, kTile, true);
  static_assert(kStages >= 4, "ring depth");
};

struct Tile {
  int g, row0, rows, col0;  // first row of the batch, rows to store, first column
};

template <bool kPair>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* off, const int* first, int t) {
  using C = Cfg<kPair>;
  Tile r;
  r.g = group_of_tile(first, a.G, t);
  const int i = t - first[r.g];
  const int m = i / a.n_tiles;
  r.col0 = (i - m * a.n_tiles) * C::kTile;
  r.row0 = off[r.g] + m * C::kTile;
  r.rows = min(C::kTile, off[r.g + 1] - r.row0);
  return r;
}

template <bool kPair>
__global__ void __launch_bounds__(kGroupedThreads, 1)
    grouped_fp8_kernel(const __grid_constant__ RowMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_out, const Args args) {
  using C = Cfg<kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + static_cast<size_t>(C::kStages) * C::kStageBytes;
  uint8_t* reserve = staging + C::kOutBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(reserve);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kAccBufs;
  uint64_t* drain = acc_empty + C::kAccBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scan = reinterpret_cast<int*>(reserve + 640);
  int* off = reinterpret_cast<int*>(reserve + 1024);
  int* first = off + kMaxGroups + 4;
  static_assert((2 * C::kStages + 2 * C::kAccBufs + 1) * 8 + 8 <= 640, "barriers overlap the scan buffer");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
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
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x.map[4]);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) tmem_alloc_for<kPair>(tmem_slot, C::kTmemCols);
  pdl_wait();
  tc_fence_before();
  const int num_tiles =
      build_group_tables(args.offsets, args.M, args.G, C::kTile, args.n_tiles, off, first, scan);
  if constexpr (kPair) cluster_barrier();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int first_tile = static_cast<int>(blockIdx.x) / C::kCtas, stride = static_cast<int>(gridDim.x) / C::kCtas;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (of each CTA)
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        const Tile tl = tile_at<kPair>(args, off, first, t);
        auto loaded = [&](int r) {  // rows that CTA r loads
          const int n = min(128, tl.rows - 128 * r);
          return n > 0 ? row_map_rows(row_map_index(n)) : 0;
        };
        const int rows = loaded(rank);
        const CUtensorMap* map = &tm_x.map[rows > 0 ? row_map_index(rows) : 0];
        const uint32_t bytes = kPair ? (loaded(0) + loaded(1)) * 128 + 32768 : rows * 128 + 16384;
        for (int kb = 0; kb < args.k_blocks; ++kb) {
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
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (leader && lane == 0) {
      int stage = 0, abuf = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true;
      for (int t = first_tile; t < num_tiles && ok; t += stride) {
        for (int kb = 0; kb < args.k_blocks; ++kb) {
          ok = wait_bar(&full[stage], phase, abort_flag, args.status, kWhereGroupedMma) &&
               wait_bar(&acc_empty[abuf], aphase ^ 1u, abort_flag, args.status, kWhereGroupedMma);
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
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    const int g = (warp - 2) >> 2;        // column half
    const int row = 32 * q + lane;        // accumulator row
    uint8_t* out_box = staging + static_cast<size_t>(warp - 2) * 4096;
    const uint32_t lane_addr = (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(C::kCols * g);
    const uint32_t empty_bar = kPair ? in_cta(acc_empty, 0) : smem_u32(acc_empty);
    const int kb_n = args.k_blocks;
    const int n_blocks = (args.N + 127) / 128;
    int abuf = 0;
    uint32_t aphase = 0;
    bool ok = true;
    for (int t = first_tile; t < num_tiles && ok; t += stride) {
      const Tile tl = tile_at<kPair>(args, off, first, t);
      const int rows = tl.rows - 128 * rank;            // of this CTA's half
      const int col = tl.col0 + C::kCols * g;           // first column of this thread
      const bool live = 32 * q < rows && col < args.N;  // this warp has something to store
      const long long grow = static_cast<long long>(tl.row0) + 128 * rank + row;
      float acc[C::kCols];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i] = 0.f;
      const float* sx = args.x_scale + (live && row < rows ? grow : 0);
      const float* sw =
          args.w_scale + (live ? (static_cast<long long>(tl.g) * n_blocks + col / 128) * kb_n : 0);
      // the scales of block kb are loaded two blocks ahead of their use
      float x0 = *sx, w0 = *sw, x1 = 0.f, w1 = 0.f;
      if (kb_n > 1) {
        x1 = sx[args.M];
        w1 = sw[1];
      }
      for (int kb = 0; kb < kb_n; ++kb) {
        const float f = x0 * w0;
        x0 = x1;
        w0 = w1;
        if (kb + 2 < kb_n) {
          x1 = sx[static_cast<long long>(kb + 2) * args.M];
          w1 = sw[kb + 2];
        }
        ok = warp_wait_bar(&acc_full[abuf], aphase, abort_flag, args.status, kWhereGroupedEpilogue);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          // chunk c + 1 is read from TMEM while chunk c is scaled and added
          const uint32_t d = tmem_base + lane_addr + static_cast<uint32_t>(abuf * C::kTile);
          uint32_t v[2][16];
          tmem_ld16u(d, v[0]);
#pragma unroll
          for (int c = 0; c < C::kCols / 16; ++c) {
            tmem_wait_ld();
            if (c + 1 < C::kCols / 16) tmem_ld16u(d + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              ffma2f(acc[16 * c + i], acc[16 * c + i + 1], v[c & 1][i], v[c & 1][i + 1], f);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_in_cluster(empty_bar + 8 * abuf);
        if (++abuf == C::kAccBufs) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) break;
      if (!live) continue;
      if (32 * q + 32 <= rows) {
        // 128 bytes of each row go through shared memory as one TMA store of the warp's 32 rows (it leaves out
        // what lies behind the last column)
        const int step = args.out_f32 ? 32 : 64;
#pragma unroll
        for (int c = 0; c < C::kCols; c += 32) {
          if (c % step == 0 && col + c < args.N) {
            uint4 piece[8];
            if (args.out_f32) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float* f = acc + c + 4 * i;
                piece[i] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                      __float_as_uint(f[3]));
              }
            } else if (c + 64 <= C::kCols) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float* f = acc + (c + 64 <= C::kCols ? c : 0) + 8 * i;
                piece[i] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                      pack_bf16(f[6], f[7]));
              }
            }
            if (lane == 0) bulk_wait_read_all();  // the previous store has read the box
            __syncwarp();
            stage_row(out_box, lane, piece);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              store_3d<false>(&tm_out, out_box, col + c, tl.row0 + 128 * rank + 32 * q, 0);
              bulk_commit();
            }
          }
        }
      } else if (row < rows) {
        // the group ends inside the warp's rows: each thread stores its own (N is a multiple of 8)
        const long long at = grow * args.ldo + col;
#pragma unroll
        for (int c = 0; c < C::kCols; c += 8) {
          if (col + c < args.N) {
            const float* f = acc + c;
            if (args.out_f32) {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(args.out) + at + c);
              o[0] = make_float4(f[0], f[1], f[2], f[3]);
              o[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.out) + at + c) =
                  make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (kPair)
    cluster_barrier();  // the leader's MMAs read this CTA's shared memory: leave together
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free_for<kPair>(tmem_base, C::kTmemCols);
  }
}

template <bool kPair>
cudaError_t launch_tiles(const GroupedProblem& p, cudaStream_t s) {
  using C = Cfg<kPair>;
  constexpr auto kern = grouped_fp8_kernel<kPair>;
  cudaError_t e = allow_smem<kern>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  Args a{};
  a.M = p.M;
  a.G = p.G;
  a.N = p.N;
  a.k_blocks = (p.K + 127) / 128;
  a.n_tiles = (p.N + C::kTile - 1) / C::kTile;
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
  if constexpr (kPair) {
    return launch_pairs<kern>(tiles, C::kSmemBytes, s, tm_x, tm_w, tm_out, a);
  } else {
    const unsigned grid = static_cast<unsigned>(tiles < p.num_sms ? tiles : p.num_sms);
    return launch_pdl(kern, dim3(grid), dim3(kGroupedThreads), C::kSmemBytes, s, tm_x, tm_w, tm_out, a);
  }
}

}  // namespace

cudaError_t launch_grouped_fp8(const GroupedProblem& p, cudaStream_t stream) {
  const bool pair = p.M / p.G >= 128 &&
                    static_cast<long long>(p.M) / 256 * ((p.N + 255) / 256) >= p.num_sms / 2;
  return pair ? launch_tiles<true>(p, stream) : launch_tiles<false>(p, stream);
}

}  // namespace moe
