// rows.cuh -- element types and row access shared by the row kernels
// (expert-order copies and sums, 8-bit quantization).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {
namespace rows {

// N adjacent elements of T, kept as they lie in memory, in 32-bit words: a 16-bit
// element is only taken out of its word where its value is used.  (Held as an
// array of elements, each one costs a register of its own as soon as a chunk at a
// row's end is put together from single loads: 122 registers instead of 64 for
// eight bf16 chunks in flight, and half the bandwidth.)
template <typename T, int N>
struct Chunk {
  static constexpr int kWords = (N * static_cast<int>(sizeof(T)) + 3) / 4;
  uint32_t w[kWords];
};

template <typename T>
__device__ __forceinline__ float word_f32(uint32_t word, int e);  // element e of its word
template <>
__device__ __forceinline__ float word_f32<float>(uint32_t word, int) {
  return __uint_as_float(word);
}
template <>
__device__ __forceinline__ float word_f32<__nv_bfloat16>(uint32_t word, int e) {
  return __uint_as_float((e & 1) ? word & 0xffff0000u : word << 16);
}
template <>
__device__ __forceinline__ float word_f32<__half>(uint32_t word, int e) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>((e & 1) ? word >> 16 : word)));
}

template <typename T, int N>
__device__ __forceinline__ float element(const Chunk<T, N> &c, int e) {  // e: compile-time
  return word_f32<T>(c.w[sizeof(T) == 4 ? e : e / 2], e);
}

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

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<float>(float lo, float) { return __float_as_uint(lo); }

// The values rounded to T.
template <typename T, int N>
__device__ __forceinline__ Chunk<T, N> rounded(const float (&v)[N]) {
  Chunk<T, N> c;
#pragma unroll
  for (int i = 0; i < Chunk<T, N>::kWords; ++i) {
    if (sizeof(T) == 4) c.w[i] = __float_as_uint(v[i]);
    else c.w[i] = pack2<T>(v[2 * i], 2 * i + 1 < N ? v[(2 * i + 1) % N] : 0.f);
  }
  return c;
}

// Chunk c (elements [c N, c N + N)) of a row of d elements; elements past the
// row's end read as zero and are never touched.
template <typename T, int N>
__device__ __forceinline__ Chunk<T, N> load_chunk(const T *row, int c, int d) {
  constexpr int kBytes = N * static_cast<int>(sizeof(T));
  Chunk<T, N> r;
  const int e0 = c * N;
  if (N == 1 || e0 + N <= d) {
    const void *p = row + e0;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = static_cast<const uint4 *>(p)[i];
        r.w[4 * i] = v.x;
        r.w[4 * i + 1] = v.y;
        r.w[4 * i + 2] = v.z;
        r.w[4 * i + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = *static_cast<const uint2 *>(p);
      r.w[0] = v.x;
      r.w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      r.w[0] = *static_cast<const uint32_t *>(p);
    } else {
      r.w[0] = *static_cast<const uint16_t *>(p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < Chunk<T, N>::kWords; ++i) r.w[i] = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (e0 + e >= d) break;
      if constexpr (sizeof(T) == 4)
        r.w[e] = *reinterpret_cast<const uint32_t *>(row + e0 + e);
      else
        r.w[e / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(row + e0 + e))
                      << (16 * (e & 1));
    }
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void store_chunk(T *row, int c, int d, const Chunk<T, N> &r) {
  constexpr int kBytes = N * static_cast<int>(sizeof(T));
  const int e0 = c * N;
  if (N == 1 || e0 + N <= d) {
    void *p = row + e0;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        static_cast<uint4 *>(p)[i] =
            make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *static_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    } else if constexpr (kBytes == 4) {
      *static_cast<uint32_t *>(p) = r.w[0];
    } else {
      *static_cast<uint16_t *>(p) = static_cast<uint16_t>(r.w[0]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (e0 + e >= d) break;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<uint32_t *>(row + e0 + e) = r.w[e];
      else
        *reinterpret_cast<uint16_t *>(row + e0 + e) =
            static_cast<uint16_t>(r.w[e / 2] >> (16 * (e & 1)));
    }
  }
}

}  // namespace rows
}  // namespace moe
