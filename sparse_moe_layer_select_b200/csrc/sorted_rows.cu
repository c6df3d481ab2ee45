// sorted_rows.cu -- token rows to expert order and back, with the router's
// weights, and the gradients of both and of the router's logits.
//
// With inv[t, j] the expert-order row of token t's slot j (-1: not routed):
//
//   dispatch           x_perm[inv[t, j], :] = x[t, :]
//   dispatch backward  dx[t, :] = sum_j d_x_perm[inv[t, j], :]  (+ add[t, :])
//   combine            y[t, :] = s sum_j w[t, j] o[inv[t, j], :]  (+ shared[t, :])
//   combine backward   d_o[inv[t, j], :] = s w[t, j] dy[t, :]
//                      d_w[t, j] = s <dy[t, :], o[inv[t, j], :]>
//   route backward     with p = w normalised over the slots (w_j = sigmoid(l_j) /
//                      sum_i sigmoid(l_i)):  dl_j = p_j sigmoid(-l_j) (dw_j - sum_i dw_i p_i);
//                      not normalised:       dl_j = sigmoid(l_j) sigmoid(-l_j) dw_j
//
// All of them move far more bytes than they compute and are bound by HBM, at
// small batches by latency.  They go by the inverse permutation, token by
// token, so that each token row is read (or written) once and every sum runs
// in slot order: the results do not depend on the launch.  Sums are held in
// fp32 and rounded once.  An inv entry outside [-1, T k) is skipped and
// reported, so no row index reaches memory unchecked.
#include "../../include/moe_rows.h"
#include "pdl.cuh"
#include "rows.cuh"
#include "rows_kernels.h"
#include "status.cuh"

#include <initializer_list>
#include <type_traits>
#include <utility>

namespace moe {

namespace {

using namespace rows;

// (128: at 55 registers a thread, blocks of 256 leave an eighth of the SM's threads unused;
// combine of 16384 x 4096, top-16: 409 us, with 128 372)
constexpr int kThreads = 128;

// The expert-order row of a slot, or -1.
__device__ __forceinline__ int checked_row(int r, int n, int *status) {
  if (r >= 0 && r < n) return r;
  if (r != kNotRouted) record_status(status, MOE_ERR_DEVICE_BOUNDS, SITE_INVERSE_ROW);
  return -1;
}

// Chunks of one row that a thread handles, 32 apart: more than one where a chunk is too
// small to keep enough bytes in flight.
template <int N>
constexpr int kPieces = N == 8 ? 1 : 2;

// Token and first chunk of this thread's item: T x chunks items, or for several pieces
// T x (warps of 32 * pieces chunks).  (32-bit division where it will do.)
template <int U>
__device__ __forceinline__ bool item_of(int n_tokens, int chunks, int *t, int *c) {
  const int per_row = U == 1 ? chunks : (chunks + 32 * U - 1) / (32 * U) * 32;
  const int64_t total = static_cast<int64_t>(n_tokens) * per_row;
  const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  if (i >= total) return false;
  if (total <= 0xffffffffLL) *t = static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row);
  else *t = static_cast<int>(i / per_row);
  const int at = static_cast<int>(i - static_cast<int64_t>(*t) * per_row);
  *c = U == 1 ? at : (at & ~31) * U + (at & 31);
  return true;
}

// Slots whose rows a thread has in flight at once: 128 bytes of loads (twice as many were
// a fifth slower: fewer threads fit).
template <typename T, int N>
constexpr int kBatch = sizeof(T) * N * kPieces<N> * 16 <= 128 ? 16
                                                              : 128 / (sizeof(T) * N * kPieces<N>);

// Entries [j0, j0 + B) of a token's k slots, four to a load where every token's slots
// start on a 16-byte boundary; `none` past the last.
template <int B, typename V>
__device__ __forceinline__ void load_slots(const V *slots, int j0, int k, V none, V (&out)[B]) {
  static_assert(sizeof(V) == 4, "four entries to 16 bytes");
  if (B % 4 == 0 && k % 4 == 0) {
#pragma unroll
    for (int j = 0; j < B; j += 4) {
      V four[4] = {none, none, none, none};
      if (j0 + j < k) {
        const uint4 v = *reinterpret_cast<const uint4 *>(slots + j0 + j);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) four[q] = *reinterpret_cast<const V *>(&w[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) out[(j + q) % B] = four[q];
    }
  } else {
#pragma unroll
    for (int j = 0; j < B; ++j) out[j] = j0 + j < k ? slots[j0 + j] : none;
  }
}

// One thread per item: a load per piece, up to k stores of each.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
    dispatch_kernel(const T *__restrict__ x, int64_t x_stride, const int32_t *__restrict__ inv,
                    int n_tokens, int k, int d, int chunks, T *__restrict__ x_perm,
                    int64_t p_stride, int *status) {
  constexpr int U = kPieces<N>;
  early_start();
  int t, c0;
  if (!item_of<U>(n_tokens, chunks, &t, &c0)) return;
  Chunk<T, N> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (U == 1 || c0 + 32 * u < chunks) v[u] = load_chunk<T, N>(x + t * x_stride, c0 + 32 * u, d);
  const int32_t *slots = inv + static_cast<int64_t>(t) * k;
  for (int j0 = 0; j0 < k; j0 += 8) {
    int r[8];
    load_slots(slots, j0, k, kNotRouted, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = checked_row(r[j], n_tokens * k, status);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (r[j] >= 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (U == 1 || c0 + 32 * u < chunks)
            store_chunk<T, N>(x_perm + r[j] * p_stride, c0 + 32 * u, d, v[u]);
      }
  }
}

// One thread per item: up to k loads of each piece, kBatch of them in flight, summed in
// slot order.  y may be add itself: a chunk is read before the same thread overwrites
// it.  Bound by HBM: 16384 x 4096, top-16, bf16: 358 us when repeated on the same rows (6.75
// TB/s: some of them are still in L2), 370 to 394 on rows that change (6.1 to 6.5); the
// gradient of the copy (no weights) 325 us, 7.0 TB/s.  How many blocks fit on an SM decides
// that: 64 registers (weighted) and 56 (not).  At 64, 21 of the 27 weighted forms spill: 16
// bytes for 16-bit inputs in chunks of eight, 68 in chunks of two, 8 to 48 in single elements;
// none of the others does.  With 72 registers and no spills they are slower all the same: 368
// against 358 us there, 368 against 352 (8192 x 4096 bf16, chunks of two), 1381 against 1154
// (4097, single elements), 271 against 268 (fp32, single elements); fp32 in chunks of two 215
// against 217.  At 56 and 48 the spills cost more.
template <typename TI, typename TO, int N, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, WEIGHTED ? 8 : 9)
    to_tokens_kernel(const TI *__restrict__ o, int64_t o_stride, const TI *add,
                     int64_t add_stride, const int32_t *__restrict__ inv,
                     const float *__restrict__ w, int n_tokens, int k, int d, int chunks,
                     float scale, TO *y, int64_t y_stride, int *status) {
  constexpr int U = kPieces<N>;
  constexpr int B = kBatch<TI, N>;
  early_start();
  int t, c0;
  if (!item_of<U>(n_tokens, chunks, &t, &c0)) return;
  const int64_t s0 = static_cast<int64_t>(t) * k;
  float acc[U][N];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[u][e] = 0.f;
  for (int j0 = 0; j0 < k; j0 += B) {
    Chunk<TI, N> v[B][U];
    unsigned routed = 0;
    {
      int r[B];
      load_slots(inv + s0, j0, k, kNotRouted, r);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        r[j] = checked_row(r[j], n_tokens * k, status);
        if (r[j] >= 0) routed |= 1u << j;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (r[j] >= 0 && (U == 1 || c0 + 32 * u < chunks))
            v[j][u] = load_chunk<TI, N>(o + r[j] * o_stride, c0 + 32 * u, d);
          else
            v[j][u] = Chunk<TI, N>{};
        }
      }
    }
    float wj[B];
    if (WEIGHTED) load_slots(w + s0, j0, k, 0.f, wj);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      // a slot that is not routed adds 0 times 0, whatever its weight holds
      const float f = !WEIGHTED ? 1.f : (routed >> j & 1) ? wj[j] : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) acc[u][e] = fmaf(f, element(v[j][u], e), acc[u][e]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (U > 1 && c0 + 32 * u >= chunks) break;
    if (WEIGHTED) {
#pragma unroll
      for (int e = 0; e < N; ++e) acc[u][e] *= scale;
    }
    if (add != nullptr) {
      const Chunk<TI, N> a = load_chunk<TI, N>(add + t * add_stride, c0 + 32 * u, d);
#pragma unroll
      for (int e = 0; e < N; ++e) acc[u][e] += element(a, e);
    }
    store_chunk<TO, N>(y + t * y_stride, c0 + 32 * u, d, rounded<TO, N>(acc[u]));
  }
}

// One warp per slot: the slot's d_o row and its dot product, up to 64 bytes of each of
// the two rows in flight per lane.  Those are summed by themselves before they join the lane's
// sum (in one chain of d / 32 terms, 8192 products of one sign were off by 62 roundings, 32768
// by 249; now 7 and 16).  d_o may be o itself: a chunk is read before the same lane overwrites it.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const T *__restrict__ dy, int64_t dy_stride, const T *o,
                            int64_t o_stride, const int32_t *__restrict__ inv,
                            const float *__restrict__ w, int n_slots, int k, int d, int chunks,
                            float scale, T *d_o, int64_t do_stride, float *__restrict__ d_w,
                            int *status) {
  early_start();
  constexpr int B = 64 / (sizeof(T) * N) < 8 ? 64 / (sizeof(T) * N) : 8;
  const int lane = threadIdx.x & 31;
  const int64_t slot = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  if (slot >= n_slots) return;
  const int i = static_cast<int>(slot);
  const int r = checked_row(inv[i], n_slots, status);
  if (r < 0) {
    if (lane == 0) d_w[i] = 0.f;
    return;
  }
  const float g = scale * w[i];
  const T *dy_row = dy + (i / k) * dy_stride;
  const T *o_row = o + r * o_stride;
  T *do_row = d_o + r * do_stride;
  float dot = 0.f;
  for (int c0 = lane; c0 < chunks; c0 += 32 * B) {
    Chunk<T, N> a[B], b[B];
#pragma unroll
    for (int q = 0; q < B; ++q)
      if (c0 + 32 * q < chunks) {
        b[q] = load_chunk<T, N>(o_row, c0 + 32 * q, d);
        a[q] = load_chunk<T, N>(dy_row, c0 + 32 * q, d);
      }
    float piece = 0.f;
#pragma unroll
    for (int q = 0; q < B; ++q)
      if (c0 + 32 * q < chunks) {
        float out[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float f = element(a[q], e);
          piece = fmaf(f, element(b[q], e), piece);
          out[e] = g * f;
        }
        store_chunk<T, N>(do_row, c0 + 32 * q, d, rounded<T, N>(out));
      }
    dot += piece;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
  if (lane == 0) d_w[i] = scale * dot;
}

// Half a warp per token (k <= 16).  The normalised weights are a softmax of
// log sigmoid(l) over the slots, taken with its maximum out, so that a row whose scores
// all underflow still has its weights.  The row of d_logits is written whole: zeros,
// then the selected experts' entries (an expert that a row names twice gets the sum).
// (A warp per token was slower, 14.4 against 10 us for 32768 x 256: each waits for the
// same two round trips.)
template <int VEC>
__global__ void __launch_bounds__(kThreads)
    route_backward_kernel(const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                          const float *__restrict__ d_w, int n_tokens, int E, int k, int norm,
                          float *__restrict__ d_logits, int *status) {
  early_start();
  const int lane = threadIdx.x & 15;
  const int64_t t = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 4;
  const bool live = t < n_tokens;  // (the other half of the warp may be)
  float *row = d_logits + t * E;
  int e = kNotRouted;
  float g = 0.f;
  if (live && lane < k) {
    e = topk_idx[t * k + lane];
    g = d_w[t * k + lane];
    if (e < 0 || e >= E) {
      if (e != kNotRouted) record_status(status, MOE_ERR_DEVICE_BOUNDS, SITE_PERMUTE_EXPERT_ID);
      e = kNotRouted;
    }
  }
  const bool on = e >= 0;
  const float l = on ? logits[t * E + e] : 0.f;
  if (!on) g = 0.f;
  if (live)
    for (int c = lane * VEC; c < E; c += 16 * VEC) {
      if (VEC == 4) *reinterpret_cast<float4 *>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      else row[c] = 0.f;
    }
  const float q = 1.f / (1.f + expf(l));  // sigmoid(-l)
  float dl;
  if (norm) {
    const float ls = on ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : -INFINITY;
    float m = ls;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float p = on ? expf(ls - m) : 0.f;
    float sum = p, dot = p * g;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
      dot += __shfl_xor_sync(0xffffffffu, dot, off);
    }
    dl = p / sum * q * (g - dot / sum);
  } else {
    dl = q / (1.f + expf(-l)) * g;
  }
  float total = 0.f;
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl_sync(0xffffffffu, e, j, 16);
    const float dj = __shfl_sync(0xffffffffu, dl, j, 16);
    if (ej == e) total += dj;
  }
  __syncwarp();  // the row's zeros are written
  if (on) row[e] = total;
}

// Threads of a kernel that goes by item_of.
template <int N>
int64_t items(int T, int chunks) {
  constexpr int U = kPieces<N>;
  return static_cast<int64_t>(T) * (U == 1 ? chunks : (chunks + 32 * U - 1) / (32 * U) * 32);
}

unsigned all_blocks(int64_t threads) {
  return static_cast<unsigned>((threads + kThreads - 1) / kThreads);
}

// Elements per chunk: 8 where every row starts on a 16-byte boundary, 2 where
// row strides are even (rows then start on a boundary of two elements), else
// one (the base pointers are 16-byte aligned by the callers' check).
int chunk_elems(std::initializer_list<std::pair<int64_t, int>> strides) {
  bool v8 = true, v2 = true;
  for (const auto &s : strides) {
    v8 = v8 && (s.first * elem_size(s.second)) % 16 == 0;
    v2 = v2 && s.first % 2 == 0;
  }
  return v8 ? 8 : v2 ? 2 : 1;
}

template <typename F>
cudaError_t by_type(int dtype, F &&f) {
  switch (dtype) {
    case MOE_DTYPE_BF16: return f(__nv_bfloat16());
    case MOE_DTYPE_F16: return f(__half());
    default: return f(float());
  }
}

template <typename F>
cudaError_t by_chunk(int n, F &&f) {
  switch (n) {
    case 8: return f(std::integral_constant<int, 8>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, 1>());
  }
}

}  // namespace

cudaError_t launch_dispatch(int dtype, const void *x, int64_t x_stride, const int32_t *inv, int T,
                            int k, int d, void *x_perm, int64_t p_stride, int *status,
                            cudaStream_t s) {
  return by_type(dtype, [&](auto tag) {
    using Ty = decltype(tag);
    return by_chunk(chunk_elems({{x_stride, dtype}, {p_stride, dtype}}), [&](auto n) {
      constexpr int N = decltype(n)::value;
      const int chunks = (d + N - 1) / N;
      return launch_early(dispatch_kernel<Ty, N>, all_blocks(items<N>(T, chunks)), kThreads, 0, s,
                          0, static_cast<const Ty *>(x), x_stride, inv, T, k, d, chunks,
                          static_cast<Ty *>(x_perm), p_stride, status);
    });
  });
}

cudaError_t launch_to_tokens(int in_type, const void *o, int64_t o_stride, const void *add,
                             int64_t add_stride, const int32_t *inv, const float *w, int T, int k,
                             int d, float scale, int out_type, void *y, int64_t y_stride,
                             int *status, cudaStream_t s) {
  const int n_elems = chunk_elems(
      {{o_stride, in_type}, {add ? add_stride : 0, in_type}, {y_stride, out_type}});
  return by_type(in_type, [&](auto ti) {
    return by_type(out_type, [&](auto to) {
      return by_chunk(n_elems, [&](auto n) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int N = decltype(n)::value;
        const int chunks = (d + N - 1) / N;
        const unsigned grid = all_blocks(items<N>(T, chunks));
        const TI *op = static_cast<const TI *>(o), *ap = static_cast<const TI *>(add);
        TO *yp = static_cast<TO *>(y);
        return launch_early(w != nullptr ? to_tokens_kernel<TI, TO, N, true>
                                         : to_tokens_kernel<TI, TO, N, false>,
                            grid, kThreads, 0, s, 0, op, o_stride, ap, add_stride, inv, w, T, k, d,
                            chunks, scale, yp, y_stride, status);
      });
    });
  });
}

cudaError_t launch_combine_backward(int dtype, const void *dy, int64_t dy_stride, const void *o,
                                    int64_t o_stride, const int32_t *inv, const float *w, int T,
                                    int k, int d, float scale, void *d_o, int64_t do_stride,
                                    float *d_w, int *status, cudaStream_t s) {
  const int n_elems = chunk_elems({{dy_stride, dtype}, {o_stride, dtype}, {do_stride, dtype}});
  return by_type(dtype, [&](auto tag) {
    using Ty = decltype(tag);
    return by_chunk(n_elems, [&](auto n) {
      constexpr int N = decltype(n)::value;
      const int chunks = (d + N - 1) / N;
      return launch_early(combine_backward_kernel<Ty, N>,
                          all_blocks(static_cast<int64_t>(T) * k * 32), kThreads, 0, s, 0,
                          static_cast<const Ty *>(dy), dy_stride, static_cast<const Ty *>(o),
                          o_stride, inv, w, T * k, k, d, chunks, scale, static_cast<Ty *>(d_o),
                          do_stride, d_w, status);
    });
  });
}

cudaError_t launch_route_backward(const float *logits, const int32_t *topk_idx, const float *d_w,
                                  int T, int E, int k, int norm, float *d_logits, int *status,
                                  cudaStream_t s) {
  const unsigned grid = all_blocks(static_cast<int64_t>(T) * 16);
  return launch_early(E % 4 == 0 ? route_backward_kernel<4> : route_backward_kernel<1>, grid,
                      kThreads, 0, s, 0, logits, topk_idx, d_w, T, E, k, norm, d_logits, status);
}

}  // namespace moe
