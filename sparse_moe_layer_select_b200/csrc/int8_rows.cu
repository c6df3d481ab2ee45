// int8_rows.cu -- rows quantized to 8-bit integers, one scale per row:
//
//   s = max(amax(|v|) / 127, 2^-126)  (1 for a row of zeros),  r = 1 / s,
//   code = rint(v r)
//
// every step one correctly rounded fp32 operation (ties to even), so that the
// codes of a row are the same wherever they are computed.  The floor keeps r
// finite for rows of subnormal values.  A row that holds an infinity or NaN has
// no scale: it gets the scale NaN and codes of zero, which makes every product
// of it NaN.
//
// Bound by HBM: one read of the row, one byte per element written.  A row stays
// in registers between its maximum and its codes.  With an inverse permutation
// (dispatch) a token's codes are computed once and stored to the expert-order
// row of each of its slots.
#include <initializer_list>
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"
#include "status.cuh"

namespace moe {

namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kRegChunks = 16;  // chunks a lane keeps: rows of up to 512 chunks are read once

template <int N>
struct alignas(N) Codes {
  int8_t v[N];
};

template <typename T, int N>
__device__ __forceinline__ uint32_t chunk_amax_bits(const Chunk<T, N> &c, uint32_t m) {
  // |v| >= 0 orders as its bits do, with infinity and then NaN above every finite value
#pragma unroll
  for (int e = 0; e < N; ++e) m = max(m, __float_as_uint(fabsf(to_f32(c.v[e]))));
  return m;
}

template <typename T, int N>
__device__ __forceinline__ Codes<N> chunk_codes(const Chunk<T, N> &c, float r) {
  Codes<N> q;
#pragma unroll
  for (int e = 0; e < N; ++e)
    q.v[e] = static_cast<int8_t>(__float2int_rn(__fmul_rn(to_f32(c.v[e]), r)));
  return q;
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t *row, int c, int d, const Codes<N> &q) {
  const int e0 = c * N;
  if (N == 1 || e0 + N <= d) {
    *reinterpret_cast<Codes<N> *>(row + e0) = q;
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e0 + e < d) row[e0 + e] = q.v[e];
  }
}

// Scale and reciprocal of a row from the bits of its largest magnitude; false
// for a row that has none (the caller stores zero codes).
__device__ __forceinline__ bool row_scale(uint32_t amax_bits, float *scale, float *rcp) {
  if (amax_bits >= 0x7f800000u) {
    *scale = __uint_as_float(0x7fc00000u);
    *rcp = 0.f;
    return false;
  }
  const float amax = __uint_as_float(amax_bits);
  const float s = amax > 0.f ? fmaxf(__fdiv_rn(amax, 127.f), 0x1p-126f) : 1.f;
  *scale = s;
  *rcp = __frcp_rn(s);
  return true;
}

// One warp per row; DISPATCH: the row's codes go to row inv[t * k + j] of each slot j.
template <typename T, int N, bool DISPATCH>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T *__restrict__ x, int64_t x_stride, int n_rows,
                    const int32_t *__restrict__ n_valid, const int32_t *__restrict__ inv, int k,
                    int d, int chunks, int8_t *__restrict__ codes, int64_t c_stride,
                    float *__restrict__ scales, int *status) {
  const int lane = threadIdx.x & 31;
  const int warps = (gridDim.x * kThreads) >> 5;
  const int rows_in = n_valid != nullptr ? min(n_rows, *n_valid) : n_rows;
  for (int t = (blockIdx.x * kThreads + threadIdx.x) >> 5; t < rows_in; t += warps) {
    const T *row = x + t * x_stride;
    const bool keep = chunks <= 32 * kRegChunks;
    Chunk<T, N> v[kRegChunks];
    uint32_t m = 0;
    if (keep) {
#pragma unroll
      for (int i = 0; i < kRegChunks; ++i)
        if (lane + 32 * i < chunks) v[i] = load_chunk<T, N>(row, lane + 32 * i, d);
#pragma unroll
      for (int i = 0; i < kRegChunks; ++i)
        if (lane + 32 * i < chunks) m = chunk_amax_bits(v[i], m);
    } else {
      for (int c = lane; c < chunks; c += 32) m = chunk_amax_bits(load_chunk<T, N>(row, c, d), m);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    float scale, rcp;
    const bool finite = row_scale(m, &scale, &rcp);
    auto put = [&](int c, const Chunk<T, N> &val) {
      Codes<N> q;
      if (finite) {
        q = chunk_codes(val, rcp);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) q.v[e] = 0;
      }
      if (!DISPATCH) {
        store_codes<N>(codes + t * c_stride, c, d, q);
      } else {
        for (int j = 0; j < k; ++j) {
          const int r = inv[static_cast<int64_t>(t) * k + j];
          if (r >= 0 && r < n_rows * k)
            store_codes<N>(codes + r * c_stride, c, d, q);
        }
      }
    };
    if (keep) {
#pragma unroll
      for (int i = 0; i < kRegChunks; ++i)
        if (lane + 32 * i < chunks) put(lane + 32 * i, v[i]);
    } else {
      for (int c = lane; c < chunks; c += 32) put(c, load_chunk<T, N>(row, c, d));
    }
    if (!DISPATCH) {
      if (lane == 0) scales[t] = scale;
    } else if (lane < k) {
      const int r = inv[static_cast<int64_t>(t) * k + lane];
      if (r >= 0 && r < n_rows * k) scales[r] = scale;
      else if (r != kNotRouted) record_status(status, MOE_ERR_DEVICE_BOUNDS, SITE_INVERSE_ROW);
    }
  }
}

int blocks_for_rows(int rows) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int want = (rows + kThreads / 32 - 1) / (kThreads / 32);
  return want < sms * 8 ? want : sms * 8;
}

template <typename T, int N>
cudaError_t launch_typed(const void *x, int64_t x_stride, int rows, const int32_t *n_valid,
                         const int32_t *inv, int k, int d, int8_t *codes, int64_t c_stride,
                         float *scales, int *status, cudaStream_t s) {
  const int chunks = (d + N - 1) / N;
  const int grid = blocks_for_rows(rows);
  const T *xp = static_cast<const T *>(x);
  if (inv != nullptr)
    quantize_kernel<T, N, true><<<grid, kThreads, 0, s>>>(xp, x_stride, rows, n_valid, inv, k, d,
                                                          chunks, codes, c_stride, scales, status);
  else
    quantize_kernel<T, N, false><<<grid, kThreads, 0, s>>>(xp, x_stride, rows, n_valid, inv, k, d,
                                                           chunks, codes, c_stride, scales, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_by_chunk(const void *x, int64_t x_stride, int rows, const int32_t *n_valid,
                            const int32_t *inv, int k, int d, int8_t *codes, int64_t c_stride,
                            float *scales, int *status, cudaStream_t s) {
  // rows that all start on a 16-byte boundary move in 8-element chunks (c_stride is a
  // multiple of 16)
  if ((x_stride * static_cast<int64_t>(sizeof(T))) % 16 == 0)
    return launch_typed<T, 8>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride, scales,
                              status, s);
  if (x_stride % 2 == 0)
    return launch_typed<T, 2>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride, scales,
                              status, s);
  return launch_typed<T, 1>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride, scales, status,
                            s);
}

}  // namespace

cudaError_t launch_quantize_int8(int dtype, const void *x, int64_t x_stride, int rows,
                                 const int32_t *n_valid, const int32_t *inv, int k, int d,
                                 int8_t *codes, int64_t c_stride, float *scales, int *status,
                                 cudaStream_t s) {
  switch (dtype) {
    case MOE_DTYPE_BF16:
      return launch_by_chunk<__nv_bfloat16>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride,
                                            scales, status, s);
    case MOE_DTYPE_F16:
      return launch_by_chunk<__half>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride, scales,
                                     status, s);
    default:
      return launch_by_chunk<float>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride, scales,
                                    status, s);
  }
}

}  // namespace moe
