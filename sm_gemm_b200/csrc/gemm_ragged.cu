// Products of rows sorted by expert with their experts' matrices, on CTA pairs:
//   C[t, n] = act( sum_k A[t, k] B[e, k, n] + bias[e, n] ),  offsets[e] <= t < offsets[e+1],
// 16-bit operands with FP32 accumulation, or int8 codes with exact int32 accumulation and a
// scale per row and per column, C = act( sa[t] sb[e, n] sum + bias[e, n] ). The offsets are
// read on the device (they are a router's output), so the host neither waits for them nor
// knows the tiles: a batching of many small products in one launch ("为什么我们要死磕GEMM"
// (kwkr.cn), section 5.3) without its host-side size arrays. The dense int8 product is the
// case of one group.
//
// The features are the MMA's M and the rows its N (C^T = B^T A^T): a tile is 256 features
// (128 per CTA) by up to TN rows of one expert, and since the instruction's N is any
// multiple of 32, a ragged expert pays for its rows rounded up to 32, not to 128 or 256.
// An expert's rows are cut into ceil(rows / TN) tiles of equal width. Rows of a tile past
// the expert's end are the next expert's (or zeros past T): they only feed accumulator
// columns that are never stored. K past the end of an expert's matrix is zero-filled by
// the 3-D tensor map.
//
// Every CTA builds the group table (row bounds and first tiles) from the offsets in shared
// memory, and from the tile count the schedule: whole waves of tiles round-robin over the
// clusters, the ragged last wave cut along K (stream-K ranges, partials summed in K order
// by the last contributor: deterministic, no CTA waits for another).
//
// Roles as in gemm_grouped.cu: warp 0 TMA producer, warp 1 MMA issuer (rank-0 CTA), warp 2
// TMEM allocator, warp 3 group table, warps 4-11 epilogue.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.cuh"
#include "ragged.h"
#include "operands.cuh"
#include "ragged.cuh"
#include "sm100.cuh"

namespace smg {

namespace {
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 32 * kEpiWarp0 + kEpiThreads;
constexpr int kStageWarpBytes = 2048;  // epilogue transposition buffer per warp
constexpr int kWBytes = 128 * 128;     // one CTA's weight tile of a stage: 128 features x 128 bytes of K

// One tile: rows tok0 .. tok0 + ntok - 1 of expert e (MMA N = width), features from 256 ft.
struct RItem {
  int e, tok0, ntok, width, ft;
};

__device__ __forceinline__ RItem locate(const RaggedParams& p, const int* bound, const int* tile0, int tn, int t) {
  const int u = t / p.n_ft;
  int lo = 0, hi = p.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile0[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  RItem it;
  it.e = lo;
  const int r0 = bound[lo], r1 = bound[lo + 1];
  const int w = tile_width(r1 - r0, tn);
  TileSched ts{};
  ts.m_tiles = tile0[lo + 1] - tile0[lo];
  ts.n_tiles = p.n_ft;
  ts.group_m = ts.m_tiles < 8 ? ts.m_tiles : 8;
  int mt;
  tile_coords(ts, t - tile0[lo] * p.n_ft, mt, it.ft);
  it.tok0 = r0 + mt * w;
  it.ntok = r1 - it.tok0 < w ? r1 - it.tok0 : w;
  it.width = (it.ntok + 31) & ~31;
  return it;
}

// The schedule of `tiles` tiles of kb K blocks over P clusters: whole waves data-parallel,
// the R tiles of a ragged last wave as one stream-K range cut evenly over the clusters, at
// least min_kb blocks each.
__device__ __forceinline__ TileSched make_sched(int tiles, int kb, int P, int min_kb) {
  TileSched s{};
  s.m_tiles = tiles;
  s.n_tiles = 1;
  s.kb_total = kb;
  s.num_ctas = P;
  s.group_m = 1;
  const int R = tiles % P;
  s.dp_tiles = tiles;
  s.sk_iters = 0;
  s.sk_ctas = P;
  if (R > 0) {
    const long long iters = static_cast<long long>(R) * kb;
    long long c = iters / min_kb;
    if (c > P) c = P;
    if (c > R) {
      s.dp_tiles = tiles - R;
      s.sk_iters = iters;
      s.sk_ctas = static_cast<int>(c);
    }
  }
  return s;
}

// 32 features (lanes) x 32 rows of C^T in registers -> C: scale, bias, activation, cast,
// transposition through this warp's 2 KB buffer, 16-byte stores of whole row segments.
// f0: the warp's first feature; row0: first row; nrow: rows to store (<= 32).
template <bool I8>
__device__ __forceinline__ void emit_chunk(const RaggedParams& p, uint8_t* buf, int lane, int e, int f0, int row0,
                                           int nrow, const uint32_t (&r)[32]) {
  const int f = f0 + lane;
  const bool live = f < p.N;
  float v[32];
  if (p.kb_total == 0) {  // no products: C = act(bias)
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
  } else if constexpr (I8) {
    const float sb = live ? __ldg(p.sb + static_cast<long long>(e) * p.N + f) : 0.0f;
    const float sa = lane < nrow ? __ldg(p.sa + row0 + lane) : 0.0f;
    // int32 -> FP32 rounds sums of 2^24 and more to nearest (relative error 2^-24).
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = static_cast<float>(static_cast<int>(r[j])) * (sb * __shfl_sync(0xffffffffu, sa, j));
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
  }
  float b = 0.0f;
  if (p.bias != nullptr && live) b = load_bias(static_cast<const char*>(p.bias) +
                                               static_cast<long long>(e) * p.N * (p.bias_dtype == 0 ? 4 : 2),
                                               p.bias_dtype, f);
  if (p.act != 0 && p.c_dtype == 0) {
    // FP32 output: activation in double, one copy of the code (see epi_bias_act32_f64).
#pragma unroll 1
    for (int j = 0; j < 32; ++j) {
      const float y = __double2float_rn(act_apply_f64(static_cast<double>(v[0]) + static_cast<double>(b), p.act));
#pragma unroll
      for (int k = 0; k < 31; ++k) v[k] = v[k + 1];
      v[31] = y;
    }
  } else {
    if (p.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += b;
    }
    if (p.act == 1) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 y = act_apply2(make_float2(v[2 * j], v[2 * j + 1]), 1);
        v[2 * j] = y.x;
        v[2 * j + 1] = y.y;
      }
    } else if (p.act == 2) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 y = act_apply2(make_float2(v[2 * j], v[2 * j + 1]), 2);
        v[2 * j] = y.x;
        v[2 * j + 1] = y.y;
      }
    }
  }
  const bool whole = f0 + 32 <= p.N;
  if (p.c_dtype == 0) {
    float* C = static_cast<float*>(p.C);
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 rows of 128 bytes at a time
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) reinterpret_cast<float*>(buf)[j * 32 + lane] = v[16 * h + j];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + (lane >> 3), c = 4 * (lane & 7);
        const float4 x = reinterpret_cast<const float4*>(buf)[row * 8 + (lane & 7)];
        if (16 * h + row < nrow) {
          float* dst = C + static_cast<long long>(row0 + 16 * h + row) * p.ldc + f0 + c;
          if (whole) {
            *reinterpret_cast<float4*>(dst) = x;
          } else {
            const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (f0 + c + q < p.N) dst[q] = y[q];
          }
        }
      }
    }
  } else {
    // Lane pairs exchange halves so that each 32-bit word holds two neighbouring features
    // of one row: the even lane keeps row 2j, the odd lane row 2j + 1.
    const bool odd = lane & 1;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float give = odd ? v[2 * j] : v[2 * j + 1];
      const float got = __shfl_xor_sync(0xffffffffu, give, 1);
      const float lo = odd ? got : v[2 * j], hi = odd ? v[2 * j + 1] : got;
      uint32_t w;
      if (p.c_dtype == 1) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
        w = *reinterpret_cast<const uint32_t*>(&t);
      } else {
        const __half2 t = __floats2half2_rn(lo, hi);
        w = *reinterpret_cast<const uint32_t*>(&t);
      }
      reinterpret_cast<uint32_t*>(buf)[(2 * j + (odd ? 1 : 0)) * 16 + (lane >> 1)] = w;
    }
    __syncwarp();
    uint16_t* C = static_cast<uint16_t*>(p.C);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + (lane >> 2), c = 8 * (lane & 3);
      const uint4 x = reinterpret_cast<const uint4*>(buf)[row * 4 + (lane & 3)];
      if (row < nrow) {
        uint16_t* dst = C + static_cast<long long>(row0 + row) * p.ldc + f0 + c;
        if (whole) {
          *reinterpret_cast<uint4*>(dst) = x;
        } else {
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (f0 + c + q < p.N) dst[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
        }
      }
    }
  }
}

// Partial sums of a split tile: FP32 partials add as floats, int32 partials as integers.
template <bool I8>
__device__ __forceinline__ void slot_add32(const float* slot, int r_local, int col0, uint32_t (&v)[32]) {
  const uint4* s4 = reinterpret_cast<const uint4*>(slot);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint4 t = __ldcg(s4 + ((col0 >> 2) + q) * 128 + r_local);
    const uint32_t x[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if constexpr (I8) v[4 * q + h] += x[h];
      else v[4 * q + h] = __float_as_uint(__uint_as_float(v[4 * q + h]) + __uint_as_float(x[h]));
    }
  }
}
}  // namespace

template <bool I8, int TN, int STAGES>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_ragged_kernel(const __grid_constant__ RaggedMaps maps, const __grid_constant__ RaggedParams p) {
  constexpr int X_BYTES = (TN / 2) * 128;
  constexpr int STAGE_BYTES = kWBytes + X_BYTES;
  constexpr int BKE = I8 ? 128 : 64;  // elements of K per block of 128 bytes
  constexpr int SLOT = 128 * TN;
  constexpr int TCOLS = 2 * TN;       // two accumulators
  constexpr int kMinKb = 4;           // fewest K blocks of a stream-K piece

  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem_base - smem_u32(smem_raw));
  uint8_t* staging = smem_gen + STAGES * STAGE_BYTES;
  const uint32_t bar_base = smem_base + STAGES * STAGE_BYTES + kEpiWarps * kStageWarpBytes;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * STAGES + 2 + b); };
  const uint32_t drain_bar = bar_base + 8u * (2 * STAGES + 4);
  uint8_t* misc = smem_gen + STAGES * STAGE_BYTES + kEpiWarps * kStageWarpBytes + 8 * (2 * STAGES + 5);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* reduce_flag = reinterpret_cast<volatile int*>(misc + 8);
  int* bound = reinterpret_cast<int*>(misc + 16);  // [E + 1]
  int* tile0 = bound + p.E + 1;                    // [E + 1]

  const uint32_t warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
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
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.w);
#pragma unroll
    for (int i = 0; i < 3; ++i) tma_prefetch_desc(&maps.x[i]);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), TCOLS);
    tmem_relinquish_pair();
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 3) build_group_table(p.offsets, p.E, p.T, TN, lane, bound, tile0);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrive or copy targets them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const TileSched s = make_sched(tile0[p.E] * p.n_ft, p.kb_total, static_cast<int>(gridDim.x >> 1), kMinKb);
  const uint64_t limit = p.wait_limit_cycles;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    WorkIter wi;
    wi.init(s, cluster);
    Seg seg;
    while (ok && wi.next(s, seg)) {
      const RItem it = locate(p, bound, tile0, TN, seg.tile);
      const int rows = it.width >> 1;  // this CTA's half of the tile's rows: a multiple of 16
      const int w_row = it.ft * 256 + static_cast<int>(rank) * 128;
      const int x_row = it.tok0 + static_cast<int>(rank) * rows;
      const uint32_t tx_bytes = 2u * (kWBytes + rows * 128);
      for (int kb = seg.kb0; kb < seg.kb1; ++kb) {
        const bool w = mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, limit);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        const uint32_t sw = smem_base + stage * STAGE_BYTES;
        const uint32_t sx = sw + kWBytes;
        const uint32_t leader_full = mapa_shared(full_bar(stage), 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), tx_bytes);
          const int k0 = kb * BKE;
          if (!I8 && p.w_mn_major) {
            tma_load_3d_pair(sw, &maps.w, leader_full, w_row, k0, it.e);
            tma_load_3d_pair(sw + 64 * 128, &maps.w, leader_full, w_row + 64, k0, it.e);
          } else {
            tma_load_3d_pair(sw, &maps.w, leader_full, k0, w_row, it.e);
          }
          int r = 0;
#pragma unroll 1
          for (; r + 64 <= rows; r += 64) tma_load_2d_pair(sx + r * 128, &maps.x[0], leader_full, k0, x_row + r);
          if (rows & 32) {
            tma_load_2d_pair(sx + r * 128, &maps.x[1], leader_full, k0, x_row + r);
            r += 32;
          }
          if (rows & 16) tma_load_2d_pair(sx + r * 128, &maps.x[2], leader_full, k0, x_row + r);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && rank == 0 && lane == 0) {
      // Wait (bounded, independent of the abort flag) for copies still in flight.
      int st = stage;
      uint32_t ph = phase;
      volatile int no_abort = 0;
      for (long long i = 0; i < issued && i < STAGES; ++i) {
        if (--st < 0) { st = STAGES - 1; ph ^= 1u; }
        mbar_wait(full_bar(st), ph, &no_abort, limit);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    bool ok = true;
    WorkIter wi;
    wi.init(s, cluster);
    Seg seg;
    while (ok && wi.next(s, seg)) {
      const RItem it = locate(p, bound, tile0, TN, seg.tile);
      const uint32_t idesc = p.idesc | (static_cast<uint32_t>(it.width >> 3) << 17);
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, limit))) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * TN;
      for (int kb = seg.kb0; kb < seg.kb1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, abort_flag, limit))) { ok = false; break; }
        tc_fence_after();
        const uint32_t sw = smem_base + stage * STAGE_BYTES;
        const uint32_t sx = sw + kWBytes;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t accum = (kb > seg.kb0 || k > 0) ? 1u : 0u;
            const uint64_t xd = sdesc_sw128(sx + 32 * k, 16, 1024);
            if constexpr (I8) umma_i8_pair(d_tmem, sdesc_sw128(sw + 32 * k, 16, 1024), xd, idesc, accum);
            else umma_f16_pair(d_tmem, operand_desc<128, 64>(sw, p.w_mn_major, k), xd, idesc, accum);
          }
          umma_commit_pair(empty_bar(stage), 0x3);
        }
        __syncwarp();
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
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
    const int half = (warp - kEpiWarp0) >> 2;  // takes 32-row chunks half, half + 2, ...
    const int r_local = q * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const int epi_tid = threadIdx.x - kEpiWarp0 * 32;
    uint8_t* buf = staging + (warp - kEpiWarp0) * kStageWarpBytes;
    int local = 0;
    bool dead = false;
    WorkIter wi;
    wi.init(s, cluster);
    Seg seg;
    while (wi.next(s, seg)) {
      const RItem it = locate(p, bound, tile0, TN, seg.tile);
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      if (!dead) dead = !mbar_wait(tfull_bar(acc), acc_phase, abort_flag, limit);
      dead = __any_sync(0xffffffffu, dead);
      const int f0 = it.ft * 256 + static_cast<int>(rank) * 128 + q * 32;
      const int chunks = it.width >> 5;
      const uint32_t tacc = tmem_base + lane_addr + acc * TN;
      const bool whole = seg.kb0 == 0 && seg.kb1 == s.kb_total;
      auto emit = [&](int c, const uint32_t(&r)[32]) {
        const int n = it.ntok - 32 * c;
        if (f0 < p.N) emit_chunk<I8>(p, buf, static_cast<int>(lane), it.e, f0, it.tok0 + 32 * c, n < 32 ? n : 32, r);
      };
      float* my_slot = p.slots + ((static_cast<size_t>(cluster) * 2 + seg.slot) * 2 + rank) * SLOT;
      if (!dead) {
        tc_fence_after();
#pragma unroll 1
        for (int c = half; c < chunks; c += 2) {
          uint32_t r[32];
          tmem_ld_32x32b_x32_sync(tacc + c * 32, r);
          if (whole) {
            emit(c, r);
          } else {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
            slot_store<32>(my_slot, r_local, c * 32, v);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
      }
      if (!whole) {
        // The last contributor to the tile (per rank) sums the partials in K order.
        const long long t_sk = seg.tile - s.dp_tiles;
        const int c_lo = sk_owner(s, t_sk * s.kb_total);
        const int c_hi = sk_owner(s, (t_sk + 1) * s.kb_total - 1);
        __threadfence();
        named_barrier_sync(1, kEpiThreads);
        if (epi_tid == 0) {
          const bool any_dead = *abort_flag != 0;
          const int n = c_hi - c_lo + 1;  // every cluster's range is non-empty
          const int old = any_dead ? -1 : counter_arrive(p.counters + t_sk * 2 + rank, p.gen, n);
          *reduce_flag = (!any_dead && old == n - 1);
        }
        named_barrier_sync(1, kEpiThreads);
        if (*reduce_flag) {
          __threadfence();
#pragma unroll 1
          for (int c = half; c < chunks; c += 2) {
            uint32_t v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
#pragma unroll 1
            for (int cc = c_lo; cc <= c_hi; ++cc) {
              const float* src = p.slots + ((static_cast<size_t>(cc) * 2 + sk_slot_of(s, cc, t_sk)) * 2 + rank) * SLOT;
              slot_add32<I8>(src, r_local, c * 32, v);
            }
            emit(c, v);
          }
        }
        named_barrier_sync(1, kEpiThreads);
      }
      ++local;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer stays resident until the rank-0 MMA issuer has drained
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem_base, TCOLS);
}

namespace {
constexpr int kWideStages = 6, kNarrowStages = 9;

template <int TN, int STAGES>
constexpr int smem_bytes(int E) {
  return 1024 + STAGES * (kWBytes + (TN / 2) * 128) + kEpiWarps * kStageWarpBytes + 8 * (2 * STAGES + 5) + 16 +
         2 * (E + 1) * static_cast<int>(sizeof(int));
}
static_assert(smem_bytes<256, kWideStages>(kRaggedMaxGroups) <= 232448, "shared memory budget");
static_assert(smem_bytes<64, kNarrowStages>(kRaggedMaxGroups) <= 232448, "shared memory budget");

template <bool I8, int TN, int STAGES>
cudaLaunchConfig_t config(int clusters, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<TN, STAGES>(kRaggedMaxGroups);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <bool I8, int TN, int STAGES>
int max_clusters_of() {
  if (smem_opt_in<gemm_ragged_kernel<I8, TN, STAGES>>(smem_bytes<TN, STAGES>(kRaggedMaxGroups)) != cudaSuccess) return 0;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config<I8, TN, STAGES>(1, nullptr, attr);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_ragged_kernel<I8, TN, STAGES>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}

template <bool I8, int TN, int STAGES>
cudaError_t launch_of(const RaggedMaps& m, const RaggedParams& p, int clusters, cudaStream_t stream) {
  cudaError_t e = smem_opt_in<gemm_ragged_kernel<I8, TN, STAGES>>(smem_bytes<TN, STAGES>(kRaggedMaxGroups));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<I8, TN, STAGES>(clusters, stream, attr);
  add_pdl_attr(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, gemm_ragged_kernel<I8, TN, STAGES>, m, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}
}  // namespace

int ragged_max_clusters() {
  static std::atomic<int> cached{-1};
  int n = cached.load();
  if (n >= 0) return n;
  const int c[4] = {max_clusters_of<false, 256, kWideStages>(), max_clusters_of<false, 64, kNarrowStages>(),
                    max_clusters_of<true, 256, kWideStages>(), max_clusters_of<true, 64, kNarrowStages>()};
  n = c[0];
  for (int i = 1; i < 4; ++i) n = c[i] < n ? c[i] : n;
  cached.store(n);
  return n;
}

cudaError_t launch_gemm_ragged(const RaggedMaps& m, const RaggedParams& p, bool i8, bool narrow, int clusters,
                               cudaStream_t stream) {
  if (i8)
    return narrow ? launch_of<true, 64, kNarrowStages>(m, p, clusters, stream)
                  : launch_of<true, 256, kWideStages>(m, p, clusters, stream);
  return narrow ? launch_of<false, 64, kNarrowStages>(m, p, clusters, stream)
                : launch_of<false, 256, kWideStages>(m, p, clusters, stream);
}

unsigned take_error_word_ragged() { return take_error_word(); }

}  // namespace smg
