// Weight gradients of the ragged products, on CTA pairs: for every expert e
//   dB[e][k, n] = sum over its rows t of A[t, k] D[t, n],   dbias[e][n] = sum of D[t, n],
// offsets[e] <= t < offsets[e+1] read on the device: the dW = X^T dY of a linear layer
// ("为什么我们要死磕GEMM" (kwkr.cn), section 3.2) for rows sorted by expert. An expert
// without rows gets zeros.
//
// Tiles are 256 x 256 of one expert's gradient; the reduction runs over its rows in blocks
// of 64, both operands read as they lie (MN-major: 64 columns x 64 rows per box). Rows of
// the last block past the expert's end belong to the next expert and must count as zeros in
// both operands (0 * NaN is NaN): that block is loaded in boxes of 32, 16, .. 1 rows, the
// expert's rows from where they are and the rest from rows past T, which TMA fills with
// zeros. The extra copies are issued once per tile.
//
// Tiles go round-robin over the clusters; the tiles of a ragged last wave are split along
// the rows into S pieces, summed in row order by the last to finish (deterministic).
// Roles as in gemm_grouped.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.cuh"
#include "operands.cuh"
#include "ragged.cuh"
#include "ragged.h"
#include "sm100.cuh"

namespace smg {

namespace {
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 32 * kEpiWarp0 + kEpiThreads;
constexpr int kEpiCols = 128;  // tile columns per epilogue warp
constexpr int kTileN = 256;
constexpr int kTcols = 512;
constexpr int kBK = 64, kStages = 6;
constexpr int kOpBytes = 128 * kBK * 2;  // one CTA's operand tile of a stage
constexpr int kStageBytes = 2 * kOpBytes;

// One piece of a tile: rows kb0*64 .. of expert e; unit >= 0 marks a piece of a split tile.
struct WItem {
  int tile, e, mt, nt, row0, cnt, kb0, kb1, unit;
};

struct WSched {
  int tiles, split_tiles, splits, per_group, P;
};

struct WIter {
  int next_dp, cluster;
  bool unit_pending;

  __device__ __forceinline__ void init(const WSched& s, int c) {
    cluster = c;
    next_dp = c;
    unit_pending = c < s.split_tiles * s.splits;
  }
  __device__ __forceinline__ void fill(const WgradParams& p, const WSched& s, const int* bound, WItem& it) {
    it.e = it.tile / s.per_group;
    TileSched ts{};
    ts.m_tiles = p.m_tiles;
    ts.n_tiles = p.n_tiles;
    ts.group_m = p.m_tiles < 8 ? p.m_tiles : 8;
    tile_coords(ts, it.tile - it.e * s.per_group, it.mt, it.nt);
    it.row0 = bound[it.e];
    it.cnt = bound[it.e + 1] - it.row0;
  }
  __device__ __forceinline__ bool next(const WgradParams& p, const WSched& s, const int* bound, WItem& it) {
    if (unit_pending) {
      unit_pending = false;
      it.tile = s.tiles - s.split_tiles + cluster / s.splits;
      fill(p, s, bound, it);
      const int kbn = (it.cnt + kBK - 1) / kBK, piece = cluster % s.splits;
      it.kb0 = static_cast<int>(static_cast<long long>(piece) * kbn / s.splits);
      it.kb1 = static_cast<int>(static_cast<long long>(piece + 1) * kbn / s.splits);
      it.unit = cluster;
      return true;
    }
    if (next_dp < s.tiles - s.split_tiles) {
      it.tile = next_dp;
      next_dp += s.P;
      fill(p, s, bound, it);
      it.kb0 = 0;
      it.kb1 = (it.cnt + kBK - 1) / kBK;
      it.unit = -1;
      return true;
    }
    return false;
  }
};
}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    gemm_ragged_wgrad_kernel(const __grid_constant__ WgradMaps maps, const __grid_constant__ WgradParams p) {
  constexpr int SLOT = 128 * kTileN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem_base - smem_u32(smem_raw));
  const uint32_t bar_base = smem_base + kStages * kStageBytes;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (kStages + s); };
  auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * kStages + b); };
  auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * kStages + 2 + b); };
  const uint32_t drain_bar = bar_base + 8u * (2 * kStages + 4);
  uint8_t* misc = smem_gen + kStages * kStageBytes + 8 * (2 * kStages + 5);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* reduce_flag = reinterpret_cast<volatile int*>(misc + 8);
  int* bound = reinterpret_cast<int*>(misc + 16);  // [E + 1]
  int* tile0 = bound + p.E + 1;                    // [E + 1], unused here

  const uint32_t warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), kTcols);
    tmem_relinquish_pair();
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 3) build_group_table(p.offsets, p.E, p.T, 256, lane, bound, tile0);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t limit = p.wait_limit_cycles;

  WSched s;
  s.per_group = p.m_tiles * p.n_tiles;
  s.tiles = s.per_group * p.E;
  s.P = static_cast<int>(gridDim.x >> 1);
  {
    // The last wave's R tiles are split when each piece keeps at least 8 blocks.
    const int R = s.tiles % s.P;
    s.split_tiles = 0;
    s.splits = 1;
    if (R > 0) {
      int min_kb = 1 << 30;
      for (int e = (s.tiles - R) / s.per_group; e < p.E; ++e) {
        const int kb = (bound[e + 1] - bound[e] + kBK - 1) / kBK;
        min_kb = kb < min_kb ? kb : min_kb;
      }
      const int S = min(s.P / R, min_kb / 8);
      if (S >= 2) {
        s.split_tiles = R;
        s.splits = S;
      }
    }
  }

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    WIter wi;
    wi.init(s, cluster);
    WItem it;
    while (ok && wi.next(p, s, bound, it)) {
      const int a_col = it.mt * 256 + static_cast<int>(rank) * 128;
      const int d_col = it.nt * kTileN + static_cast<int>(rank) * 128;
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        const bool w = mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, limit);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        const uint32_t sa = smem_base + stage * kStageBytes;
        const uint32_t leader_full = mapa_shared(full_bar(stage), 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * kStageBytes);
          // Rows `row`.. of both operands (two 64-column boxes each) to block row r.
          auto load = [&](int box, int r, int row) {
            const uint32_t dst = sa + r * 128;
            tma_load_2d_pair(dst, &maps.a[box], leader_full, a_col, row);
            tma_load_2d_pair(dst + kBK * 128, &maps.a[box], leader_full, a_col + 64, row);
            tma_load_2d_pair(dst + kOpBytes, &maps.d[box], leader_full, d_col, row);
            tma_load_2d_pair(dst + kOpBytes + kBK * 128, &maps.d[box], leader_full, d_col + 64, row);
          };
          const int row = it.row0 + kb * kBK;
          const int valid = it.cnt - kb * kBK;
          if (valid >= kBK) {
            load(0, 0, row);
          } else {
            int r = 0;
#pragma unroll 1
            for (int box = 1, n = 32; box < kWgradBoxes; ++box, n >>= 1)
              if (valid & n) {
                load(box, r, row + r);
                r += n;
              }
#pragma unroll 1
            for (int box = kWgradBoxes - 1, n = 1; box >= 1; --box, n <<= 1)
              if (r & n) {
                load(box, r, p.T);  // past the last row: zeros
                r += n;
              }
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && rank == 0 && lane == 0) {
      int st = stage;
      uint32_t ph = phase;
      volatile int no_abort = 0;
      for (long long i = 0; i < issued && i < kStages; ++i) {
        if (--st < 0) { st = kStages - 1; ph ^= 1u; }
        mbar_wait(full_bar(st), ph, &no_abort, limit);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    bool ok = true;
    WIter wi;
    wi.init(s, cluster);
    WItem it;
    while (ok && wi.next(p, s, bound, it)) {
      if (it.kb1 == it.kb0) continue;  // an expert without rows: the epilogue writes zeros
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, limit))) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * kTileN;
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, abort_flag, limit))) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_base + stage * kStageBytes;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            umma_f16_pair(d_tmem, operand_desc<128, kBK>(sa, 1, k), operand_desc<128, kBK>(sa + kOpBytes, 1, k),
                          p.idesc, (kb > it.kb0 || k > 0) ? 1u : 0u);
          umma_commit_pair(empty_bar(stage), 0x3);
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) umma_commit_pair(tfull_bar(acc), 0x3);
      __syncwarp();
      ++local;
    }
    if (elect_one()) umma_commit_pair(drain_bar, 0x1);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(drain_bar, 0, &no_abort, limit);
  } else if (warp >= kEpiWarp0) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int r_local = q * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const int epi_tid = threadIdx.x - kEpiWarp0 * 32;
    const int c_base = ((warp - kEpiWarp0) >> 2) * kEpiCols;
    int local = 0;
    bool dead = false;
    WIter wi;
    wi.init(s, cluster);
    WItem it;
    while (wi.next(p, s, bound, it)) {
      char* out = static_cast<char*>(p.C) + static_cast<long long>(it.e) * p.stride_c * (p.c_dtype == 0 ? 4 : 2);
      const EpiArgs e{p.K, p.N, nullptr, 0, 0, out, p.c_dtype, p.ldc};
      const int row = it.mt * 256 + static_cast<int>(rank) * 128 + r_local;
      const int col0 = it.nt * kTileN + c_base;
      if (it.kb1 == it.kb0) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 1
        for (int c = 0; c < kEpiCols / 32; ++c) epi_store_row32(e, row, col0 + c * 32, v);
        continue;
      }
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      if (!dead) dead = !mbar_wait(tfull_bar(acc), acc_phase, abort_flag, limit);
      dead = __any_sync(0xffffffffu, dead);
      const uint32_t tacc = tmem_base + lane_addr + acc * kTileN + c_base;
      const bool split = it.unit >= 0;
      float* my_slot = split ? p.slots + (static_cast<size_t>(it.unit) * 2 + rank) * SLOT : nullptr;
      if (!dead) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kEpiCols / 32; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32_sync(tacc + c * 32, r);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          if (split) slot_store<32>(my_slot, r_local, c_base + c * 32, v);
          else epi_store_row32(e, row, col0 + c * 32, v);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
      }
      if (split) {
        const int r_tail = it.tile - (s.tiles - s.split_tiles);
        __threadfence();
        named_barrier_sync(1, kEpiThreads);
        if (epi_tid == 0) {
          const bool any_dead = *abort_flag != 0;
          const int old = any_dead ? -1 : counter_arrive(p.counters + r_tail * 2 + rank, p.gen, s.splits);
          *reduce_flag = (!any_dead && old == s.splits - 1);
        }
        named_barrier_sync(1, kEpiThreads);
        if (*reduce_flag) {
          __threadfence();
#pragma unroll 1
          for (int c = 0; c < kEpiCols / 32; ++c) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 1
            for (int pc = 0; pc < s.splits; ++pc)
              slot_accumulate<32>(p.slots + ((static_cast<size_t>(r_tail) * s.splits + pc) * 2 + rank) * SLOT, r_local,
                                  c_base + c * 32, v);
            epi_store_row32(e, row, col0 + c * 32, v);
          }
        }
        named_barrier_sync(1, kEpiThreads);
      }
      ++local;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem_base, kTcols);
}

namespace {
// Column sums of one expert's rows of D: a CTA takes 64 columns, warp w the rows w, w + 8,
// ..; the eight partial sums are added in warp order (deterministic).
template <bool BF16>
__global__ void __launch_bounds__(256) ragged_dbias_kernel(const uint16_t* __restrict__ D, long long ldd, int T, int N,
                                                           const int* __restrict__ offsets, float* __restrict__ db) {
  __shared__ int sh_bound[2][8];
  __shared__ float part[8][64];
  pdl_launch_dependents();
  pdl_wait();
  const int e = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Bounds as in the group table: offsets clamped to [0, T] and to their running maximum.
  int lo = 0;
  for (int i = threadIdx.x; i <= e; i += 256) lo = max(lo, min(max(offsets[i], 0), T));
  lo = __reduce_max_sync(0xffffffffu, lo);
  if (lane == 0) sh_bound[0][warp] = lo;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) lo = max(lo, sh_bound[0][w]);
  const int hi = max(lo, min(max(offsets[e + 1], 0), T));
  const int col = blockIdx.x * 64 + 2 * lane;
  float s0 = 0.0f, s1 = 0.0f;
  auto add = [&](uint32_t w) {
    float2 f;
    if constexpr (BF16) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    else f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    s0 += f.x;
    s1 += f.y;
  };
  if (col + 1 < N) {
#pragma unroll 8
    for (int t = lo + warp; t < hi; t += 8)
      add(__ldg(reinterpret_cast<const unsigned int*>(D + static_cast<long long>(t) * ldd + col)));
  } else if (col < N) {
    for (int t = lo + warp; t < hi; t += 8) add(D[static_cast<long long>(t) * ldd + col]);
  }
  part[warp][2 * lane] = s0;
  part[warp][2 * lane + 1] = s1;
  __syncthreads();
  const int c = threadIdx.x, n = blockIdx.x * 64 + c;
  if (c < 64 && n < N) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w][c];
    db[static_cast<long long>(e) * N + n] = s;
  }
}

constexpr int kSmem = 1024 + kStages * kStageBytes + 8 * (2 * kStages + 5) + 16 +
                      2 * (kRaggedMaxGroups + 1) * static_cast<int>(sizeof(int));
static_assert(kSmem <= 232448, "shared memory budget");

cudaLaunchConfig_t config(int clusters, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}
}  // namespace

int wgrad_max_clusters() {
  static std::atomic<int> cached{-1};
  int n = cached.load();
  if (n >= 0) return n;
  n = 0;
  if (smem_opt_in<gemm_ragged_wgrad_kernel>(kSmem) == cudaSuccess) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(1, nullptr, attr);
    if (cudaOccupancyMaxActiveClusters(&n, gemm_ragged_wgrad_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
  }
  cached.store(n);
  return n;
}

cudaError_t launch_gemm_ragged_wgrad(const WgradMaps& m, const WgradParams& p, int clusters, cudaStream_t stream) {
  cudaError_t e = smem_opt_in<gemm_ragged_wgrad_kernel>(kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(clusters, stream, attr);
  add_pdl_attr(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, gemm_ragged_wgrad_kernel, m, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_ragged_dbias(const void* D, bool bf16, long long ldd, int T, int N, const int* offsets, int E,
                                float* db, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((N + 63) / 64, E, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  add_pdl_attr(cfg, attr);
  const uint16_t* d = static_cast<const uint16_t*>(D);
  const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, ragged_dbias_kernel<true>, d, ldd, T, N, offsets, db)
                             : cudaLaunchKernelEx(&cfg, ragged_dbias_kernel<false>, d, ldd, T, N, offsets, db);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

unsigned take_error_word_wgrad() { return take_error_word(); }

}  // namespace smg
