// int8_gemv.cu -- the product of 8-bit integers (int8_gemm.cu) for a few rows, as a
// single token's decode step has them.
//
// A warp takes two channels of b (SwiGLU: a gate channel and its up channel) and up to R
// rows of a: every lane multiplies 16 bytes of K at a time (four byte products to an
// instruction, exact int32 sums), the lanes' sums are added, and a lane per row scales
// and stores.  Without a pipeline to fill, tensor memory to allocate or a cluster to
// bring together, a call costs little more than its bytes: the weights are read once per
// R rows, spread over all SMs.  Groups have one row per block (R = 1); a group's rows
// then share its weights through L2.
#include <algorithm>
#include <type_traits>

#include "int8_common.cuh"
#include "pdl.cuh"

namespace moe {

namespace {

using namespace int8;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// 16 bytes of a row of K, zero past its end (the bytes between rows are not read).
__device__ __forceinline__ uint4 load16(const int8_t *row, int k0, int K) {
  if (k0 + 16 <= K) return *reinterpret_cast<const uint4 *>(row + k0);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k0 + i < K)
      w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k0 + i])) << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// The group of row r, or -1: the first group whose end lies past it (offsets clamped to
// [0, M]; group ends count as running maxima, as in group_tiles).  One warp.
__device__ __forceinline__ int group_of(const Int8GemmParams &p, int r) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kMaxGroups / 32;
  int end[kPer];  // of group 32 i + lane: all loads first, one round trip
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    end[i] = 32 * i + lane < p.G ? p.offsets[32 * i + lane + 1] : 0;
  const int start = p.offsets[0];
  int found = -1;
#pragma unroll
  for (int i = kPer - 1; i >= 0; --i) {
    const unsigned past = __ballot_sync(0xffffffffu, 32 * i + lane < p.G && min(end[i], p.M) > r);
    if (past != 0) found = 32 * i + __ffs(past) - 1;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = 32 * i + lane;
      if (g < p.G) {
        const int lo = p.offsets[g];
        if (lo < 0 || end[i] < lo || end[i] > p.M)
          record_status(p.status, MOE_ERR_DEVICE_BOUNDS, SITE_GROUP_OFFSETS);
      }
    }
  }
  return r < start ? -1 : found;
}

template <typename TO, bool SWIGLU, int R>
__global__ void __launch_bounds__(kThreads)
    int8_gemv_kernel(const Int8GemmParams p, const int8_t *__restrict__ a, int64_t a_stride,
                     const int8_t *__restrict__ b, int64_t b_stride) {
  constexpr int U = R == 1 ? 4 : 2;  // pieces of 512 bytes of K in flight
  early_start();
  const int lane = threadIdx.x & 31;
  const int pair = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int c0 = SWIGLU ? pair : 2 * pair;  // the output channel, or the first of two
  const int r0 = blockIdx.y * R;
  const int group = p.offsets != nullptr ? group_of(p, r0) : 0;
  if (c0 >= p.N || group < 0) return;
  const bool two = SWIGLU || c0 + 1 < p.N;
  const int64_t row_b = static_cast<int64_t>(group) * p.b_rows + c0;
  const int8_t *b0 = b + row_b * b_stride;
  const int8_t *b1 = two ? b0 + (SWIGLU ? p.N : 1) * b_stride : b0;
  const int rows = min(R, p.M - r0);
  int acc[2][R] = {};
  for (int k0 = lane * 16; k0 - lane * 16 < p.K; k0 += 512 * U) {
    uint4 w0[U], w1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w0[u] = w1[u] = make_uint4(0, 0, 0, 0);
      if (k0 + 512 * u < p.K) {
        w0[u] = load16(b0, k0 + 512 * u, p.K);
        w1[u] = load16(b1, k0 + 512 * u, p.K);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 512 * u >= p.K) break;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (R > 1 && r >= rows) break;
        const uint4 v = load16(a + (r0 + r) * a_stride, k0 + 512 * u, p.K);
        acc[0][r] = dot16(v, w0[u], acc[0][r]);
        acc[1][r] = dot16(v, w1[u], acc[1][r]);
      }
    }
  }
  int sum0 = 0, sum1 = 0;  // of row r0 + lane
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int s0 = __reduce_add_sync(0xffffffffu, acc[0][r]);
    const int s1 = __reduce_add_sync(0xffffffffu, acc[1][r]);
    if (lane == r) {
      sum0 = s0;
      sum1 = s1;
    }
  }
  if (lane >= rows) return;
  const int r = r0 + lane;
  const float sa = p.sa[r];
  float v0 = static_cast<float>(sum0) * sa * p.sb[row_b];
  float v1 = two ? static_cast<float>(sum1) * sa * p.sb[row_b + (SWIGLU ? p.N : 1)] : 0.f;
  if (SWIGLU) v0 = silu(v0) * v1;
  TO *out = static_cast<TO *>(p.out) + r * p.out_stride + c0;
  out[0] = rows::from_f32<TO>(v0);
  if (!SWIGLU && two) out[1] = rows::from_f32<TO>(v1);
  if (std::is_same<TO, __half>::value) {
    const float m = SWIGLU ? fabsf(v0) : fmaxf(fabsf(v0), fabsf(v1));
    if (__half2float(__float2half_rn(m)) == INFINITY)
      record_status(p.status, MOE_ERR_DEVICE_BOUNDS, SITE_H_FP16_RANGE);
  }
}

template <typename TO, bool SWIGLU>
cudaError_t launch_typed(const Int8GemmParams &p, const void *a, int64_t a_stride, const void *b,
                         int64_t b_stride, cudaStream_t s) {
  const int pairs = SWIGLU ? p.N : (p.N + 1) / 2;
  const int R = p.offsets != nullptr || p.M == 1 ? 1 : p.M == 2 ? 2 : 4;
  const dim3 grid((pairs + kWarps - 1) / kWarps, (p.M + R - 1) / R);
  auto kernel = R == 1 ? int8_gemv_kernel<TO, SWIGLU, 1>
                       : R == 2 ? int8_gemv_kernel<TO, SWIGLU, 2> : int8_gemv_kernel<TO, SWIGLU, 4>;
  return launch_early(kernel, grid, kThreads, 0, s, 0, p, static_cast<const int8_t *>(a), a_stride,
                      static_cast<const int8_t *>(b), b_stride);
}

}  // namespace

cudaError_t launch_int8_gemv(const Int8GemmParams &p, int out_type, bool swiglu, const void *a,
                             int64_t a_stride, const void *b, int64_t b_stride, cudaStream_t s) {
  switch (out_type) {
    case MOE_DTYPE_BF16:
      return swiglu ? launch_typed<__nv_bfloat16, true>(p, a, a_stride, b, b_stride, s)
                    : launch_typed<__nv_bfloat16, false>(p, a, a_stride, b, b_stride, s);
    case MOE_DTYPE_F16:
      return swiglu ? launch_typed<__half, true>(p, a, a_stride, b, b_stride, s)
                    : launch_typed<__half, false>(p, a, a_stride, b, b_stride, s);
    default:
      return swiglu ? launch_typed<float, true>(p, a, a_stride, b, b_stride, s)
                    : launch_typed<float, false>(p, a, a_stride, b, b_stride, s);
  }
}

}  // namespace moe
