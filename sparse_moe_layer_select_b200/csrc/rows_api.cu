// rows_api.cu -- the entry points of include/moe_rows.h, for training and for 8-bit
// integer products: expert order with its inverse, rows to experts and back,
// their gradients, quantized rows and their products.  Argument checks and
// launches only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe_rows.h"
#include "rows_kernels.h"
#include "status.cuh"

namespace {

using namespace moe;

static_assert(MOE_DTYPE_BF16 == 0 && MOE_DTYPE_F16 == 1 && MOE_DTYPE_F32 == 2, "elem_size");

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool good(const void *p) { return p != nullptr && aligned16(p); }
inline bool dtype_ok(int32_t t) { return t >= MOE_DTYPE_BF16 && t <= MOE_DTYPE_F32; }
inline size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The longest row: element and chunk numbers are 32-bit on the device, and loops step past
// the row's end.
constexpr int kMaxRow = 1 << 30;

// The dims of calls that only move rows: T, d_model, E and k.
moe_status check_rows(const moe_dims_t *dims) {
  if (dims == nullptr || dims->struct_size != sizeof(moe_dims_t)) return MOE_ERR_INVALID_ARG;
  const int k = dims->num_experts_per_tok, E = dims->num_experts;
  if (dims->T < 0) return MOE_ERR_INVALID_ARG;
  if (dims->d_model < 1 || dims->d_model > kMaxRow) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (E < 1 || E > 512 || k < 1 || k > 16 || k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
  // (slot numbers are 32-bit, and the index rounds them up to whole chunks)
  if (static_cast<int64_t>(dims->T) * k > INT32_MAX - kIndexChunk) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// A status header that may be left out (null), else 256-byte aligned.
moe_status check_header(const void *ws) {
  return (reinterpret_cast<uintptr_t>(ws) & 255) == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// Output rows may replace input rows where each element takes the place of its own input
// (same type and stride): any other way, threads would overwrite rows not yet read.
bool in_place_ok(const void *in, int32_t in_dtype, int64_t in_stride, const void *out,
                 int32_t out_dtype, int64_t out_stride) {
  return in != out || (in_dtype == out_dtype && in_stride == out_stride);
}

int64_t slots(const moe_dims_t *dims) {
  return static_cast<int64_t>(dims->T) * dims->num_experts_per_tok;
}

struct SortLayout {
  size_t hist, tiles, total;
};

// The layout of a batch with `nchunks` chunk histograms.
SortLayout sort_layout(const moe_dims_t *dims, int64_t nchunks) {
  const size_t n = static_cast<size_t>(dims->T) * dims->num_experts_per_tok;
  SortLayout L;
  L.hist = a256(sizeof(WsHeader));
  L.tiles = L.hist + a256(static_cast<size_t>(nchunks) * dims->num_experts * sizeof(int));
  L.total = L.tiles + a256(((n + kBlockM - 1) / kBlockM + dims->num_experts) * sizeof(Tile));
  return L;
}

moe_status launched(cudaError_t e, int launches) {
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(launches);
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_sort_workspace_size(const moe_dims_t *dims) {
  // for every batch of up to T tokens: one just below a step of the chunk size has more chunks
  if (check_rows(dims) != MOE_OK) return 0;
  return sort_layout(dims, index_chunks_upto(slots(dims))).total;
}

moe_status moe_sort(const moe_dims_t *dims, const int32_t *topk_idx, int32_t *counts,
                    int32_t *offsets, int32_t *perm, int32_t *inv, int32_t dtype, const void *x,
                    int64_t x_stride, void *x_perm, int64_t x_perm_stride, void *ws,
                    size_t ws_bytes, void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK) return st;
  if (dims->T == 0) {  // no rows: nothing to order, and the (empty) other arrays may be null
    if (!good(counts) || !good(offsets)) return MOE_ERR_INVALID_ARG;
    set_last_launch_count(0);
    const size_t bytes = static_cast<size_t>(dims->num_experts) * sizeof(int32_t);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cudaMemsetAsync(counts, 0, bytes, s) == cudaSuccess &&
                   cudaMemsetAsync(offsets, 0, bytes + sizeof(int32_t), s) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  if (!good(topk_idx) || !good(counts) || !good(offsets) || !good(perm) || !good(inv))
    return MOE_ERR_INVALID_ARG;
  if ((x == nullptr) != (x_perm == nullptr)) return MOE_ERR_INVALID_ARG;
  const int T = dims->T, d = dims->d_model, E = dims->num_experts, k = dims->num_experts_per_tok;
  if (x != nullptr && (!dtype_ok(dtype) || !aligned16(x) || !aligned16(x_perm) || x_stride < d ||
                       x_perm_stride < d))
    return MOE_ERR_INVALID_ARG;
  if (ws == nullptr || (st = check_header(ws)) != MOE_OK) return MOE_ERR_INVALID_ARG;
  const SortLayout L = sort_layout(dims, index_chunks(slots(dims)));
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  set_last_launch_count(0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char *b = static_cast<char *>(ws);
  int *header = reinterpret_cast<int *>(b);
  int launches = 0;
  if (launch_index_cleared(topk_idx, T, k, E, reinterpret_cast<int *>(b + L.hist),
                           reinterpret_cast<Tile *>(b + L.tiles), header, counts, offsets, perm,
                           inv, s, &launches) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (x != nullptr) {
    if (launch_dispatch(dtype, x, x_stride, inv, T, k, d, x_perm, x_perm_stride, header, s) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    ++launches;
  }
  set_last_launch_count(launches);
  return MOE_OK;
}

moe_status moe_dispatch(const moe_dims_t *dims, int32_t dtype, const void *x, int64_t x_stride,
                        const int32_t *inv, void *x_perm, int64_t x_perm_stride, void *ws,
                        void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK || dims->T == 0) return st;
  const int d = dims->d_model;
  if (!dtype_ok(dtype) || !good(x) || !good(inv) || !good(x_perm) || x_stride < d ||
      x_perm_stride < d)
    return MOE_ERR_INVALID_ARG;
  if ((st = check_header(ws)) != MOE_OK) return st;
  set_last_launch_count(0);
  return launched(launch_dispatch(dtype, x, x_stride, inv, dims->T, dims->num_experts_per_tok, d,
                                  x_perm, x_perm_stride, static_cast<int *>(ws),
                                  static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_dispatch_backward(const moe_dims_t *dims, int32_t in_dtype, const void *d_x_perm,
                                 int64_t d_x_perm_stride, const int32_t *inv, const void *add,
                                 int64_t add_stride, int32_t out_dtype, void *d_x,
                                 int64_t d_x_stride, void *ws, void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK || dims->T == 0) return st;
  const int d = dims->d_model;
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype) || !good(d_x_perm) || !good(inv) || !good(d_x) ||
      !aligned16(add) || d_x_perm_stride < d || d_x_stride < d || (add && add_stride < d) ||
      !in_place_ok(add, in_dtype, add_stride, d_x, out_dtype, d_x_stride))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_header(ws)) != MOE_OK) return st;
  set_last_launch_count(0);
  return launched(launch_to_tokens(in_dtype, d_x_perm, d_x_perm_stride, add, add_stride, inv,
                                   nullptr, dims->T, dims->num_experts_per_tok, d, 1.f, out_dtype,
                                   d_x, d_x_stride, static_cast<int *>(ws),
                                   static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_combine(const moe_dims_t *dims, int32_t in_dtype, const void *o, int64_t o_stride,
                       const int32_t *inv, const float *topk_w, const void *shared,
                       int64_t shared_stride, int32_t out_dtype, void *y, int64_t y_stride,
                       void *ws, void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK || dims->T == 0) return st;
  const int d = dims->d_model;
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype) || !good(o) || !good(inv) || !good(topk_w) ||
      !good(y) || !aligned16(shared) || o_stride < d || y_stride < d ||
      (shared && shared_stride < d) ||
      !in_place_ok(shared, in_dtype, shared_stride, y, out_dtype, y_stride))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_header(ws)) != MOE_OK) return st;
  set_last_launch_count(0);
  return launched(launch_to_tokens(in_dtype, o, o_stride, shared, shared_stride, inv, topk_w,
                                   dims->T, dims->num_experts_per_tok, d,
                                   dims->routed_scaling_factor, out_dtype, y, y_stride,
                                   static_cast<int *>(ws), static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_combine_backward(const moe_dims_t *dims, int32_t dtype, const void *d_y,
                                int64_t d_y_stride, const void *o, int64_t o_stride,
                                const int32_t *inv, const float *topk_w, void *d_o,
                                int64_t d_o_stride, float *d_topk_w, void *ws, void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK || dims->T == 0) return st;
  const int d = dims->d_model;
  if (!dtype_ok(dtype) || !good(d_y) || !good(o) || !good(inv) || !good(topk_w) || !good(d_o) ||
      !good(d_topk_w) || d_y_stride < d || o_stride < d || d_o_stride < d)
    return MOE_ERR_INVALID_ARG;
  if (!in_place_ok(o, dtype, o_stride, d_o, dtype, d_o_stride)) return MOE_ERR_INVALID_ARG;
  if ((st = check_header(ws)) != MOE_OK) return st;
  set_last_launch_count(0);
  return launched(launch_combine_backward(dtype, d_y, d_y_stride, o, o_stride, inv, topk_w,
                                          dims->T, dims->num_experts_per_tok, d,
                                          dims->routed_scaling_factor, d_o, d_o_stride, d_topk_w,
                                          static_cast<int *>(ws),
                                          static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_route_backward(const moe_dims_t *dims, const float *logits, const int32_t *topk_idx,
                              const float *d_topk_w, float *d_logits, void *ws, void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK || dims->T == 0) return st;
  if (!good(logits) || !good(topk_idx) || !good(d_topk_w) || !good(d_logits))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_header(ws)) != MOE_OK) return st;
  set_last_launch_count(0);
  return launched(launch_route_backward(logits, topk_idx, d_topk_w, dims->T, dims->num_experts,
                                        dims->num_experts_per_tok, dims->norm_topk_prob ? 1 : 0,
                                        d_logits, static_cast<int *>(ws),
                                        static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_quantize_int8(int32_t rows, int32_t cols, int32_t dtype, const void *x,
                             int64_t x_stride, const int32_t *n_rows, int8_t *codes,
                             int64_t codes_stride, float *scales, void *stream) {
  if (rows < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (cols < 1 || cols > kMaxRow) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!good(x) || !good(codes) || !good(scales) || (reinterpret_cast<uintptr_t>(n_rows) & 3) ||
      x_stride < cols || codes_stride < cols || codes_stride % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  set_last_launch_count(0);
  return launched(launch_quantize_int8(dtype, x, x_stride, rows, n_rows, nullptr, 1, cols, codes,
                                       codes_stride, scales, nullptr,
                                       static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_dispatch_int8(const moe_dims_t *dims, int32_t dtype, const void *x,
                             int64_t x_stride, const int32_t *inv, int8_t *codes,
                             int64_t codes_stride, float *scales, void *ws, void *stream) {
  moe_status st = check_rows(dims);
  if (st != MOE_OK || dims->T == 0) return st;
  const int d = dims->d_model;
  if (!dtype_ok(dtype) || !good(x) || !good(inv) || !good(codes) || !good(scales) ||
      x_stride < d || codes_stride < d || codes_stride % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if ((st = check_header(ws)) != MOE_OK) return st;
  set_last_launch_count(0);
  return launched(launch_quantize_int8(dtype, x, x_stride, dims->T, nullptr, inv,
                                       dims->num_experts_per_tok, d, codes, codes_stride, scales,
                                       static_cast<int *>(ws), static_cast<cudaStream_t>(stream)),
                  1);
}

moe_status moe_matmul_int8(const moe_int8_matmul_t *m, void *ws, size_t ws_bytes, void *stream) {
  if (m == nullptr || m->struct_size != sizeof(moe_int8_matmul_t)) return MOE_ERR_INVALID_ARG;
  if (m->M < 0 || !dtype_ok(m->out_dtype) || (m->flags & ~MOE_INT8_SWIGLU))
    return MOE_ERR_INVALID_ARG;
  const bool swiglu = (m->flags & MOE_INT8_SWIGLU) != 0;
  const int64_t b_rows = static_cast<int64_t>(swiglu ? 2 : 1) * m->N;
  // K: the int32 sums cannot overflow (128 * 128 K < 2^31)
  if (m->N < 1 || m->K < 1 || m->K > 131071 || m->G < 1 || m->G > 512)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  // row and item numbers are 32-bit on the device
  if (m->M > INT32_MAX - 256) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int64_t tiles = (static_cast<int64_t>(m->M) + 127) / 128 + m->G;
  if (m->G * b_rows + 256 >= (int64_t(1) << 31) ||
      tiles * ((m->N + 127) / 128) >= (int64_t(1) << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (m->M == 0) return MOE_OK;
  if (m->offsets == nullptr && m->G != 1) return MOE_ERR_INVALID_ARG;
  if (!good(m->a) || !good(m->b) || !good(m->a_scale) || !good(m->b_scale) || !good(m->out) ||
      (reinterpret_cast<uintptr_t>(m->offsets) & 3))
    return MOE_ERR_INVALID_ARG;
  if (m->a_stride < m->K || m->b_stride < m->K || m->a_stride % 16 != 0 || m->b_stride % 16 != 0 ||
      m->out_stride < m->N)
    return MOE_ERR_INVALID_ARG;
  if (m->a_stride >= (int64_t(1) << 40) || m->b_stride >= (int64_t(1) << 40))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ws == nullptr || check_header(ws) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  set_last_launch_count(0);
  int sms = 0, clusters = 0;
  if (current_device_setup(&sms, &clusters) != cudaSuccess) return MOE_ERR_CUDA;
  Int8GemmParams p{};
  p.status = static_cast<int *>(ws);
  p.offsets = m->offsets;
  p.sa = m->a_scale;
  p.sb = m->b_scale;
  p.out = m->out;
  p.out_stride = m->out_stride;
  p.M = m->M;
  p.N = m->N;
  p.K = m->K;
  p.G = m->G;
  p.b_rows = static_cast<int>(b_rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // CUDA cores for a single row, and for few rows while their products are.  us there / on
  // tensor cores: 1 row, N = 1024, K = 2048: 2.4 / 6.3; 16 rows: 5.6 / 6.8; 1 row, N = 4096,
  // K = 8192: 7.4 / 10.8; 4 rows: 16.7 / 11.3; rows of 8 experts, SwiGLU, N = 512, K = 2048:
  // 6.6 / 14.5, of 32: 16.5 / 15.3.
  if (m->M == 1 || (m->M <= 16 && m->M * b_rows * m->K <= (int64_t(1) << 25)))
    return launched(launch_int8_gemv(p, m->out_dtype, swiglu, m->a, m->a_stride, m->b, m->b_stride,
                                     s),
                    1);
  // CTA pairs where the groups fill their 256-row tiles well enough; the other kernel brings
  // in the weights once and spends no products on rows that are not there, but a tile of many
  // rows keeps its epilogue longer than a short K keeps its loads.  us on 128-row tiles and on
  // pairs, 256 groups: N = 2048, K = 512: 61 / 73 at 32 rows each, 73 / 78 at 48, 87 / 79 at
  // 64, 101 / 79 at 80; SwiGLU, N = 512, K = 2048: 105 / 127 at 64, 113 / 125 at 96, 131 / 127
  // at 109.  One matrix goes to the other kernel's 32-row tiles while they find an SM each:
  // 512 rows, N = 1024, K = 2048: 9.7 / 11.0; 314 rows, N = 138, K = 1091: 7.9 / 11.7; 95 rows,
  // N = K = 4096: 14.3 / 15.1.
  const bool small = m->offsets == nullptr &&
                     (m->M + 31) / 32 * int64_t((m->N + 127) / 128) <= sms;
  const bool pairs =
      clusters > 0 && !small && m->M >= int64_t(m->K <= 1024 ? 56 : 104) * m->G;
  return launched(pairs ? launch_int8_pair(p, m->out_dtype, swiglu, m->a, m->a_stride, m->b,
                                           m->b_stride, clusters, s)
                        : launch_int8_gemm(p, m->out_dtype, swiglu, m->a, m->a_stride, m->b,
                                           m->b_stride, sms, s),
                  1);
}

}  // extern "C"
