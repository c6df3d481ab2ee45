// rows.cuh -- element types and row access shared by the row kernels
// (expert-order copies and sums, 8-bit quantization).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {
namespace rows {

// N elements of T as they lie in memory, moved by the widest loads that the
// size allows (16 bytes at most per instruction).
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Chunk {
  T v[N];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Chunk c (elements [c N, c N + N)) of a row of d elements; elements past the
// row's end read as zero and are never touched.
template <typename T, int N>
__device__ __forceinline__ Chunk<T, N> load_chunk(const T *row, int c, int d) {
  Chunk<T, N> r;
  const int e0 = c * N;
  if (N == 1 || e0 + N <= d) {
    r = *reinterpret_cast<const Chunk<T, N> *>(row + e0);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = e0 + i < d ? row[e0 + i] : from_f32<T>(0.f);
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void store_chunk(T *row, int c, int d, const Chunk<T, N> &r) {
  const int e0 = c * N;
  if (N == 1 || e0 + N <= d) {
    *reinterpret_cast<Chunk<T, N> *>(row + e0) = r;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i < d) row[e0 + i] = r.v[i];
  }
}

}  // namespace rows
}  // namespace moe
