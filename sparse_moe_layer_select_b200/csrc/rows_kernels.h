// rows_kernels.h -- launch interface of the row kernels (expert order, its gradients,
// 8-bit rows) and of the 8-bit integer products, beside kernels.h.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "kernels.h"

namespace moe {

// Site ids of these kernels (status.cuh has the others).
constexpr int SITE_INVERSE_ROW = 22;    // inverse-permutation entry outside [-1, T k)
constexpr int SITE_GROUP_OFFSETS = 23;  // group offsets that decrease or leave [0, rows]

// launch_index into a workspace header that the call zeroes first.
cudaError_t launch_index_cleared(const int32_t *topk_idx, int T, int k, int E, int *chunk_hist,
                                 Tile *tiles, int *header, int32_t *counts, int32_t *offsets,
                                 int32_t *perm, int32_t *inv, cudaStream_t s, int *launches);

// Bytes of one element of a moe_dtype.
inline int elem_size(int dtype) { return dtype == 2 ? 4 : 2; }  // 2: MOE_DTYPE_F32

// Row kernels by the inverse permutation inv [T, k] (sorted_rows.cu); strides in
// elements; status: the status word of a workspace header, or null.
cudaError_t launch_dispatch(int dtype, const void *x, int64_t x_stride, const int32_t *inv, int T,
                            int k, int d, void *x_perm, int64_t p_stride, int *status,
                            cudaStream_t s);
// y[t] = scale sum_j w[t, j] o[inv[t, j]] + add[t]; w null: sum_j o[inv[t, j]] + add[t].
cudaError_t launch_to_tokens(int in_type, const void *o, int64_t o_stride, const void *add,
                             int64_t add_stride, const int32_t *inv, const float *w, int T, int k,
                             int d, float scale, int out_type, void *y, int64_t y_stride,
                             int *status, cudaStream_t s);
cudaError_t launch_combine_backward(int dtype, const void *dy, int64_t dy_stride, const void *o,
                                    int64_t o_stride, const int32_t *inv, const float *w, int T,
                                    int k, int d, float scale, void *d_o, int64_t do_stride,
                                    float *d_w, int *status, cudaStream_t s);
cudaError_t launch_route_backward(const float *logits, const int32_t *topk_idx, const float *d_w,
                                  int T, int E, int k, int norm, float *d_logits, int *status,
                                  cudaStream_t s);
// int8 codes and fp32 scales of rows (int8_rows.cu); inv non-null: the codes of row t go to
// rows inv[t, j] (codes and scales then have rows * k rows).
cudaError_t launch_quantize_int8(int dtype, const void *x, int64_t x_stride, int rows,
                                 const int32_t *n_valid, const int32_t *inv, int k, int d,
                                 int8_t *codes, int64_t c_stride, float *scales, int *status,
                                 cudaStream_t s);

// Product of 8-bit integers (int8_gemm.cu).
struct Int8GemmParams {
  int *status;             // workspace header (status word)
  const int32_t *offsets;  // [G + 1] first row of each group, or null (one group: all rows)
  const float *sa;         // [M] row scales
  const float *sb;         // [G * b_rows] channel scales
  void *out;
  int64_t out_stride;      // elements
  int M, N, K, G;
  int b_rows;              // rows of b per group: N, or 2 N (SwiGLU: gate, then up)
  int n_ctiles;            // channel tiles (set by the launcher)
  int tma_out;             // pair kernel: output rows are a multiple of 16 bytes apart
  int tma_clips;           // and N channels are a multiple of 16 bytes
  int ksplit;              // rows kernel: CTAs of a cluster, each with a share of K
  int ring, boxes;         // pair kernel: pipeline stages, output boxes per epilogue warp
};
// On CTA pairs; clusters: pairs that can be resident at once.
cudaError_t launch_int8_pair(Int8GemmParams p, int out_type, bool swiglu, const void *a,
                             int64_t a_stride, const void *b, int64_t b_stride, int clusters,
                             cudaStream_t s);
cudaError_t launch_int8_gemm(Int8GemmParams p, int out_type, bool swiglu, const void *a,
                             int64_t a_stride, const void *b, int64_t b_stride, int sms,
                             cudaStream_t s);

// For a few rows, on CUDA cores (int8_gemv.cu).
cudaError_t launch_int8_gemv(const Int8GemmParams &p, int out_type, bool swiglu, const void *a,
                             int64_t a_stride, const void *b, int64_t b_stride, cudaStream_t s);

// Per-device set-up on the current device (once), its SM count and how many CTA pairs
// can be resident at once (moe_api.cu).
cudaError_t current_device_setup(int *sms, int *clusters);
// Store map of a [rows, cols] matrix of a moe_dtype, `stride` elements between rows:
// boxes of 64 bytes x 32 rows, 64-byte swizzle.
bool encode_out_map(CUtensorMap *m, const void *ptr, int dtype, uint64_t rows, uint64_t cols,
                    uint64_t stride);
// 2-D uint8 tensor map of [rows, cols] with `stride` bytes between rows: boxes of
// 128 bytes x box_rows, 128-byte swizzle, zero fill.
bool encode_map_u8(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint64_t stride,
                   uint32_t box_rows);

}  // namespace moe
