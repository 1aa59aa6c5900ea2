// Building blocks of the ragged products: the group table read from device offsets, 3-D
// tensor copies for a CTA of a pair and the int8 MMA.
#pragma once

#include "epilogue.cuh"
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

// 32 TMEM lanes x 32 columns as MMA fragments: register 16 h + 4 c + k of thread t holds lane
// 16 h + t / 4 (+ 8 for k >= 2), column 8 c + 2 (t % 4) + (k & 1). Both halves' loads are in
// flight before the wait.
__device__ __forceinline__ void tmem_ld_fragments_sync(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}

// Four 8 x 8 matrices of 16-bit elements, each stored transposed: thread t holds row t / 4,
// columns 2 (t % 4), + 1 of each; lane l's address takes column l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// What the CTAs of a launch agree on, computed by each from the offsets.
struct RaggedPlan {
  int tiles;     // of all groups and features
  int width;     // the widest tile's rows, rounded up to 32
  int stream_k;  // tiles cut along K (a static schedule) instead of drawn one by one
};

// Tile heights to choose from: 256, 192, 128, 96, 64, 32 rows.
__host__ __device__ __forceinline__ int next_cap(int cap) { return cap - (cap > 128 ? 64 : 32); }

// Cycles per K block of the launch's waves of tiles of `width` rows (see choose_cap).
__host__ __device__ __forceinline__ unsigned wave_cycles(int tiles, int width, int P) {
  return static_cast<unsigned>((tiles + P - 1) / P) * static_cast<unsigned>(256 + width);
}

// Whether fewer tiles than clusters are cut along K: worth it when the time saved by the
// idle clusters' help, t (1 - tiles / P) for tiles of t cycles, exceeds the fix-up of a cut
// tile (partials written, arrival, read back by the last contributor, its epilogue).
__host__ __device__ __forceinline__ int cut_along_k(int tiles, int width, int kb, int P, int force) {
  if (force != 0) return force == 2;
  if (tiles >= P || tiles == 0) return 0;
  const float t = static_cast<float>(kb) * static_cast<float>(256 + width);
  return t * static_cast<float>(P - tiles) > (6000.0f + 100.0f * static_cast<float>(width)) * static_cast<float>(P);
}

// Rows of one token tile: a group of `cnt` rows is cut into equal tiles of at most `tn`,
// a multiple of 32.
__host__ __device__ __forceinline__ int tile_width(int cnt, int tn) {
  const int nt = (cnt + tn - 1) / tn;
  return nt == 0 ? 32 : ((cnt + nt - 1) / nt + 31) & ~31;
}

// The group table by one warp, in shared memory: bound[e] .. bound[e+1] are the rows of group
// e, w32[e] its tiles' height in units of 32 rows, tile0[e] its first token tile (tile0[E] =
// their number). Offsets are clamped to [0, T] and to their running maximum, so that no
// offset makes two groups write one row or any row outside the matrices. With cap == 0 only
// the bounds are written. Returns the greatest tile height.
__device__ __forceinline__ int group_table(const int* offsets, int E, int T, int cap, uint32_t lane, int* bound,
                                           uint8_t* w32, int* tile0) {
  auto clamp_t = [&](int v) { return v < 0 ? 0 : (v > T ? T : v); };
  int run = offsets == nullptr ? 0 : clamp_t(offsets[0]), tiles = 0, width = 32;
  if (lane == 0) {
    bound[0] = run;
    if (cap != 0) tile0[0] = 0;
  }
#pragma unroll 1
  for (int base = 0; base < E; base += 32) {
    const int i = base + static_cast<int>(lane);
    int v = i < E ? (offsets == nullptr ? T : clamp_t(offsets[i + 1])) : 0;
    v = v > run ? v : run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (static_cast<int>(lane) >= d && o > v) v = o;
    }
    int prev = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) prev = run;
    run = __shfl_sync(0xffffffffu, v, 31);
    if (i < E) bound[i + 1] = v;
    if (cap == 0) continue;
    const int cnt = v - prev;
    int w = 32, nt = cnt > 0 ? 1 : 0;
    if (cnt > 32) {
      w = tile_width(cnt, cap);
      nt = (cnt + w - 1) / w;
    }
    width = w > width ? w : width;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, nt, d);
      if (static_cast<int>(lane) >= d) nt += o;
    }
    if (i < E) {
      tile0[i + 1] = tiles + nt;
      w32[i] = static_cast<uint8_t>(w >> 5);
    }
    tiles += __shfl_sync(0xffffffffu, nt, 31);
  }
  return __reduce_max_sync(0xffffffffu, width);
}

// Activations of 16-bit outputs for a pair of values: as act_apply2, with one reciprocal for
// both, 1 / (d0 d1) (the denominators are in [1, 2]): three special-function operations per
// pair instead of four, which bound the epilogue. Two more roundings of 2^-24.
__device__ __forceinline__ float2 x_sigmoid_pair(float2 x, float2 z) {
  const float2 t = __fmul2_rn(make_float2(fabsf(z.x), fabsf(z.y)), make_float2(-1.4426950408889634f, -1.4426950408889634f));
  const bool tiny0 = t.x < -120.0f, tiny1 = t.y < -120.0f;
  float e0 = exp2_sfu(tiny0 ? t.x + 64.0f : t.x);
  float e1 = exp2_sfu(tiny1 ? t.y + 64.0f : t.y);
  if (tiny0) e0 *= 5.421010862427522e-20f;  // 2^-64
  if (tiny1) e1 *= 5.421010862427522e-20f;
  float2 d = __fadd2_rn(make_float2(1.0f, 1.0f), make_float2(e0, e1));
  d = make_float2(fminf(d.x, 2.0f), fminf(d.y, 2.0f));  // a NaN (kept by x below) must not reach the pair's other row
  const float r = rcp_sfu(d.x * d.y);
  const float2 xe = __fmul2_rn(x, make_float2(z.x >= 0.0f ? 1.0f : e0, z.y >= 0.0f ? 1.0f : e1));
  return __fmul2_rn(xe, __fmul2_rn(make_float2(r, r), make_float2(d.y, d.x)));
}

// Activation of FP32 outputs, in FP32: the exponent's product |z| log2 e is carried in two
// terms, so the result's relative error stays below 2^-20 plus that of z itself (exact for
// SiLU; 2^-22 relative for GeLU, i.e. |z| 2^-22 in the factor e^-|z| of its negative tail). In
// double precision it was within an FP32 ulp, but took 40 us where the product takes 4
// (474 rows of 40 int8 experts, 440 x 1301).
__device__ __forceinline__ float x_sigmoid_accurate(float x, float z) {
  const float a = fabsf(z);
  const float hi = __fmul_rn(a, -1.4426950408889634f);
  const float lo = __fmaf_rn(a, -1.4426950408889634f, -hi) - a * 1.925963033500011e-8f;  // log2 e = 1.4426950216.. + 1.9e-8
  const bool tiny = hi < -120.0f;
  float e = exp2_sfu(tiny ? hi + 64.0f : hi);
  if (tiny) e *= 5.421010862427522e-20f;  // 2^-64
  e = a < 200.0f ? __fmaf_rn(e, lo * 0.6931471805599453f, e) : 0.0f;
  const float r = __frcp_rn(1.0f + e);
  return z >= 0.0f ? x * r : (x * e) * r;
}

__device__ __forceinline__ float act_accurate(float x, int act) {
  return x_sigmoid_accurate(x, act == 1 ? x * fmaf(kGeluB, x * x, kGeluA) : x);
}

__device__ __forceinline__ float2 act_pair(float2 x, int act) {
  if (act == 1) {
    const float2 p = __ffma2_rn(make_float2(kGeluB, kGeluB), __fmul2_rn(x, x), make_float2(kGeluA, kGeluA));
    return x_sigmoid_pair(x, __fmul2_rn(x, p));
  }
  return x_sigmoid_pair(x, x);
}

}  // namespace smg
