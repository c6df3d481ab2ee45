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
// row of each of its slots.  32768 x 2048 bf16: 31 us (6.4 TB/s), to 8 experts each 112 us
// (6.0 TB/s).
#include <initializer_list>
#include <type_traits>

#include "../../include/moe_rows.h"
#include "pdl.cuh"
#include "rows.cuh"
#include "rows_kernels.h"
#include "status.cuh"

namespace moe {

namespace {

using namespace rows;

template <typename T, int N>
__device__ __forceinline__ uint32_t chunk_amax_bits(const Chunk<T, N> &c, uint32_t m) {
  // |v| >= 0 orders as its bits do, with infinity and then NaN above every finite value
#pragma unroll
  for (int e = 0; e < N; ++e) m = max(m, __float_as_uint(fabsf(element(c, e))));
  return m;
}

// Codes of a chunk, four to a word, the first in the low byte.
template <int N>
struct Codes {
  uint32_t w[(N + 3) / 4];
};

template <typename T, int N>
__device__ __forceinline__ Codes<N> chunk_codes(const Chunk<T, N> &c, float r) {
  Codes<N> q;
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i) q.w[i] = 0;
#pragma unroll
  for (int e = 0; e < N; ++e)
    q.w[e / 4] |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(element(c, e), r))) & 0xffu)
                  << (8 * (e & 3));
  return q;
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t *row, int c, int d, const Codes<N> &q) {
  const int e0 = c * N;
  if (N == 1 || e0 + N <= d) {
    void *p = row + e0;
    if constexpr (N == 16) *static_cast<uint4 *>(p) = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
    else if constexpr (N == 8) *static_cast<uint2 *>(p) = make_uint2(q.w[0], q.w[1]);
    else if constexpr (N == 2) *static_cast<uint16_t *>(p) = static_cast<uint16_t>(q.w[0]);
    else row[e0] = static_cast<int8_t>(q.w[0]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (e0 + e >= d) break;
      row[e0 + e] = static_cast<int8_t>(q.w[e / 4] >> (8 * (e & 3)));
    }
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

// TPR threads per row, each holding up to R chunks of it; longer rows (KEEP false)
// are read a second time for their codes.  DISPATCH: the row's codes go to row
// inv[t * k + j] of each slot j.
template <typename T, int N, int TPR, int R, bool KEEP, bool DISPATCH>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    quantize_kernel(const T *__restrict__ x, int64_t x_stride, int n_rows,
                    const int32_t *__restrict__ n_valid, const int32_t *__restrict__ inv, int k,
                    int d, int chunks, int8_t *__restrict__ codes, int64_t c_stride,
                    float *__restrict__ scales, int *status) {
  early_start();
  constexpr int kBlock = TPR < 128 ? 128 : TPR;
  constexpr int kWarps = TPR / 32;
  __shared__ uint32_t warp_max[kBlock / 32];
  const int lane = threadIdx.x % TPR;
  const int64_t t = blockIdx.x * static_cast<int64_t>(kBlock / TPR) + threadIdx.x / TPR;
  // (threads of one row leave together, and a block of several warps per row has one row)
  if (t >= n_rows || (n_valid != nullptr && t >= *n_valid)) return;
  const T *row = x + t * x_stride;
  // the row of lane j's slot: loaded beside the row, given out by shuffles below
  int dest = kNotRouted;
  if (DISPATCH && (threadIdx.x & 31) < k) {
    dest = inv[t * k + (threadIdx.x & 31)];
    if (dest < 0 || dest >= n_rows * k) {
      if (dest != kNotRouted && lane < k)
        record_status(status, MOE_ERR_DEVICE_BOUNDS, SITE_INVERSE_ROW);
      dest = kNotRouted;
    }
  }
  Chunk<T, N> v[R] = {};
  uint32_t m = 0;
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (lane + TPR * i < chunks) v[i] = load_chunk<T, N>(row, lane + TPR * i, d);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (lane + TPR * i < chunks) m = chunk_amax_bits(v[i], m);
  } else {
    for (int c = lane; c < chunks; c += TPR) m = chunk_amax_bits(load_chunk<T, N>(row, c, d), m);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < kWarps ? warp_max[threadIdx.x & 31] : 0);
  }
  float scale, rcp;
  const bool finite = row_scale(m, &scale, &rcp);
  // (every lane of the warp takes part, also where its chunk is past the row's end)
  auto put = [&](int c, const Chunk<T, N> &val) {
    Codes<N> q = chunk_codes(val, rcp);
    if (!finite) {
#pragma unroll
      for (int i = 0; i < (N + 3) / 4; ++i) q.w[i] = 0;
    }
    if (!DISPATCH) {
      if (c < chunks) store_codes<N>(codes + t * c_stride, c, d, q);
    } else {
      for (int j = 0; j < k; ++j) {
        const int r = __shfl_sync(0xffffffffu, dest, j);
        if (c < chunks && r >= 0) store_codes<N>(codes + r * c_stride, c, d, q);
      }
    }
  };
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if ((lane & ~31) + TPR * i < chunks) put(lane + TPR * i, v[i]);
  } else {
    for (int c = lane; (c & ~31) < chunks; c += TPR) {
      Chunk<T, N> again{};
      if (c < chunks) again = load_chunk<T, N>(row, c, d);
      put(c, again);
    }
  }
  if (!DISPATCH) {
    if (lane == 0) scales[t] = scale;
  } else if (lane < k && dest >= 0) {
    scales[dest] = scale;
  }
}

constexpr int kFewRows = 512;

template <typename T, int N, int TPR, int R, bool KEEP>
cudaError_t launch_shape(const void *x, int64_t x_stride, int rows, const int32_t *n_valid,
                         const int32_t *inv, int k, int d, int8_t *codes, int64_t c_stride,
                         float *scales, int *status, cudaStream_t s) {
  constexpr int kBlock = TPR < 128 ? 128 : TPR;
  const int chunks = (d + N - 1) / N;
  const unsigned grid = (static_cast<unsigned>(rows) + kBlock / TPR - 1) / (kBlock / TPR);
  const T *xp = static_cast<const T *>(x);
  return launch_early(inv != nullptr ? quantize_kernel<T, N, TPR, R, KEEP, true>
                                     : quantize_kernel<T, N, TPR, R, KEEP, false>,
                      grid, kBlock, 0, s, 0, xp, x_stride, rows, n_valid, inv, k, d, chunks, codes,
                      c_stride, scales, status);
}

// Threads per row by the row's chunks, so that a thread holds four chunks at most and
// a short row does not leave most of a warp idle; with few rows a block each, so that
// they spread over the SMs (64 rows of 2048 copied to 8 experts each: 4.5 us with a warp
// per row, 3.3 with 128 threads).
template <typename T, int N>
cudaError_t launch_typed(const void *x, int64_t x_stride, int rows, const int32_t *n_valid,
                         const int32_t *inv, int k, int d, int8_t *codes, int64_t c_stride,
                         float *scales, int *status, cudaStream_t s) {
  const int chunks = (d + N - 1) / N;
#define MOE_QUANTIZE(TPR, R, KEEP)                                                             \
  launch_shape<T, N, TPR, R, KEEP>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride, scales, \
                                   status, s)
  if (rows <= kFewRows && chunks > 32 && chunks <= 128 * 2) return MOE_QUANTIZE(128, 2, true);
  if (chunks <= 32 * 2) return MOE_QUANTIZE(32, 2, true);
  if (chunks <= 32 * 4) return MOE_QUANTIZE(32, 4, true);
  if (chunks <= 128 * 4) return MOE_QUANTIZE(128, 4, true);
  if (chunks <= 512 * 4) return MOE_QUANTIZE(512, 4, true);
  return MOE_QUANTIZE(512, 1, false);
#undef MOE_QUANTIZE
}

template <typename T>
cudaError_t launch_by_chunk(const void *x, int64_t x_stride, int rows, const int32_t *n_valid,
                            const int32_t *inv, int k, int d, int8_t *codes, int64_t c_stride,
                            float *scales, int *status, cudaStream_t s) {
  // rows that all start on a 16-byte boundary move in chunks of 32 bytes (c_stride is a
  // multiple of 16, so their codes are stored 8 or 16 at a time)
  if ((x_stride * static_cast<int64_t>(sizeof(T))) % 16 == 0)
    return launch_typed<T, 32 / sizeof(T)>(x, x_stride, rows, n_valid, inv, k, d, codes, c_stride,
                                           scales, status, s);
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
