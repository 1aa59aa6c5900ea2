// Building blocks of the ragged products: the group table read from device offsets, 3-D
// tensor copies for a CTA of a pair and the int8 MMA.
#pragma once

#include "sm100.cuh"

namespace smg {

// As tma_load_2d_pair, from a 3-D tensor map.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t c0,
                                                 int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// As tma_store_2d, through a 3-D tensor map.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// D[tmem] (+)= A * B over a CTA pair, signed 8-bit integers, int32 accumulate (K = 32).
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// Instruction descriptor of kind::i8: both operands signed, S32 accumulator.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Rows of one token tile: a group of `cnt` rows is cut into equal tiles of at most `tn`,
// a multiple of 32.
__device__ __forceinline__ int tile_width(int cnt, int tn) {
  const int nt = (cnt + tn - 1) / tn;
  return nt == 0 ? 32 : ((cnt + nt - 1) / nt + 31) & ~31;
}

// Row bounds by one warp: bound[e] .. bound[e+1] are the rows of group e. Offsets are clamped
// to [0, T] and to their running maximum, so that no offset makes two groups write one row
// or any row outside the matrices.
__device__ __forceinline__ void group_bounds(const int* offsets, int E, int T, uint32_t lane, int* bound) {
  if (offsets == nullptr) {  // one group
    if (lane < 2) bound[lane] = lane == 0 ? 0 : T;
    return;
  }
  auto clamp_t = [&](int v) { return v < 0 ? 0 : (v > T ? T : v); };
  int run = 0;
  for (int base = 0; base <= E; base += 32) {
    const int i = base + static_cast<int>(lane);
    int v = i <= E ? clamp_t(offsets[i]) : 0;
    v = v > run ? v : run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (static_cast<int>(lane) >= d && o > v) v = o;
    }
    if (i <= E) bound[i] = v;
    run = __shfl_sync(0xffffffffu, v, 31);
  }
}

// First token tile of every group by one warp (after group_bounds): tile0[E] is their number.
__device__ __forceinline__ void group_tiles(const int* bound, int E, int cap, uint32_t lane, int* tile0) {
  int tiles = 0;
  if (lane == 0) tile0[0] = 0;
  for (int base = 0; base < E; base += 32) {
    const int i = base + static_cast<int>(lane);
    int nt = 0;
    if (i < E) {
      const int cnt = bound[i + 1] - bound[i];
      const int w = tile_width(cnt, cap);
      nt = (cnt + w - 1) / w;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, nt, d);
      if (static_cast<int>(lane) >= d) nt += o;
    }
    if (i < E) tile0[i + 1] = tiles + nt;
    tiles += __shfl_sync(0xffffffffu, nt, 31);
  }
}

}  // namespace smg
