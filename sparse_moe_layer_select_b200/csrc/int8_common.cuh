// int8_common.cuh -- the groups' tiles and the epilogue arithmetic shared by the
// two 8-bit integer product kernels.
#pragma once
#include <cuda_fp16.h>

#include "../../include/moe_rows.h"
#include "int8_ptx.cuh"
#include "rows.cuh"
#include "rows_kernels.h"
#include "status.cuh"

namespace moe {
namespace int8 {

constexpr int kMaxGroups = 512;
constexpr int kStageK = 128;  // K elements of a pipeline stage: one 128-byte swizzle row

// One tile of the output: up to the tile's rows of one group by a block of channels.
struct alignas(16) Work {
  int group, row0, nrows, ctile;
};

// Running sums over the groups: first_tile[g] = tiles of the groups before g,
// first_row[g] = their first row, clamped to [0, M] and made non-decreasing, so
// that offsets that no sort wrote cannot lead outside the matrices.  Called by
// every thread of the CTA; the sums are warp 0's, visible after the next barrier.
__device__ __forceinline__ void group_tiles(const Int8GemmParams &p, int tile_rows, int *first_tile,
                                            int *first_row) {
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x; g <= p.G; g += blockDim.x)  // one round trip for all of them
    first_row[g] = p.offsets ? p.offsets[g] : (g == 0 ? 0 : p.M);
  __syncthreads();
  if (threadIdx.x < 32) {
    int tiles = 0, top = 0;
    for (int g0 = 0; g0 < p.G; g0 += 32) {
      const int g = g0 + lane;
      int lo = 0, hi = 0;
      if (g < p.G) {
        lo = first_row[g];
        hi = first_row[g + 1];
      }
      __syncwarp();  // read before it is overwritten below
      bool bad = g < p.G && (lo < 0 || hi < lo || hi > p.M);
      lo = min(max(lo, 0), p.M);
      hi = min(max(hi, 0), p.M);
      // running maximum of the group ends: a group starts where the last one ended
      int end = hi;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, end, off);
        if (lane >= off) end = max(end, y);
      }
      end = max(end, top);
      int start = __shfl_up_sync(0xffffffffu, end, 1);
      if (lane == 0) start = top;
      if (g == 0) start = lo;
      start = min(max(start, lo), end);
      int nt = g < p.G ? (end - start + tile_rows - 1) / tile_rows : 0;
      int sum = nt;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      if (g < p.G) {
        first_tile[g] = tiles + sum - nt;
        first_row[g] = start;
      }
      if (g == p.G - 1) first_row[p.G] = end;
      tiles += __shfl_sync(0xffffffffu, sum, 31);
      top = __shfl_sync(0xffffffffu, end, 31);
      if (bad) record_status(p.status, MOE_ERR_DEVICE_BOUNDS, SITE_GROUP_OFFSETS);
    }
    if (lane == 0) first_tile[p.G] = tiles;
  }
}

// The tile of an item, by a search over the groups.
__device__ __forceinline__ Work find_work(const Int8GemmParams &p, int tile_rows, int item,
                                          const int *first_tile, const int *first_row) {
  const int ti = item / p.n_ctiles;
  int lo = 0, hi = p.G - 1;  // the last group whose first tile is <= ti
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_tile[mid] <= ti) lo = mid;
    else hi = mid - 1;
  }
  Work w;
  w.group = lo;
  w.row0 = first_row[lo] + (ti - first_tile[lo]) * tile_rows;
  w.nrows = min(tile_rows, first_row[lo + 1] - w.row0);
  w.ctile = item - ti * p.n_ctiles;
  return w;
}

// The tiles of a CTA's items (first, first + step, ...), the first kListed of them found
// by all threads at once when the kernel starts: a search by the thread that issues the
// loads, between two items, cost a third of the time of items of 64 KB of weights
// (256 groups, N = 2048, K = 512, 512 rows: 62 us against 41).
constexpr int kListed = 256;
struct ItemList {
  const Work *list;  // shared
  const int *first_tile, *first_row;
  int first, step;

  // tile of the CTA's i-th item
  __device__ __forceinline__ Work operator()(const Int8GemmParams &p, int tile_rows, int i) const {
    return i < kListed ? list[i]
                       : find_work(p, tile_rows, first + i * step, first_tile, first_row);
  }
};
__device__ __forceinline__ void list_items(const Int8GemmParams &p, int tile_rows, int first,
                                           int step, int n_items, const int *first_tile,
                                           const int *first_row, Work *list) {
  for (int i = threadIdx.x; i < kListed && first + i * step < n_items; i += blockDim.x)
    list[i] = find_work(p, tile_rows, first + i * step, first_tile, first_row);
}

// g sigmoid(g) by the fast exponential and quotient, whose documented bounds give: for g > 0 a
// few units in the last place; for g < 0 about 5 + 1.2 |g| of them (2 + 1.173 |g| of the
// exponential, which is nearly all of the denominator, 2 of the quotient): 17 at -10, 100 at
// -80, relative error 1.2e-5.  Below g = -87, where the denominator passes 2^126, it is 0 (the
// value itself is under 2e-36 there).
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

// Two accumulators of one row, converted and scaled by the row's scale and then by their
// channels' (each step rounded; the products two to an instruction).
__device__ __forceinline__ void scaled2(uint32_t a0, uint32_t a1, float sa, float s0, float s1,
                                        float *v0, float *v1) {
  const float f0 = static_cast<float>(static_cast<int>(a0));
  const float f1 = static_cast<float>(static_cast<int>(a1));
  asm("{\n\t.reg .b64 a, s, c;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 s, {%4, %4};\n\t"
      "mov.b64 c, {%5, %6};\n\t"
      "mul.rn.f32x2 a, a, s;\n\t"
      "mul.rn.f32x2 a, a, c;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(*v0), "=f"(*v1)
      : "f"(f0), "f"(f1), "f"(sa), "f"(s0), "f"(s1));
}

// fp16 outputs beyond the type's range become infinite: the largest magnitudes so far of
// a pair of columns (NaN, which a row without a scale gives, does not count).
__device__ __forceinline__ uint32_t larger_half2(uint32_t largest, uint32_t two) {
  const __half2 a = *reinterpret_cast<const __half2 *>(&largest);
  const __half2 b = __habs2(*reinterpret_cast<const __half2 *>(&two));
  const __half2 m = __hmax2(a, b);
  return *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ bool half2_overflows(uint32_t largest) {
  return (largest & 0xffffu) == 0x7c00u || (largest >> 16) == 0x7c00u;
}

}  // namespace int8
}  // namespace moe
