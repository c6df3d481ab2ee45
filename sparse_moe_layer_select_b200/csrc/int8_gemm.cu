// int8_gemm.cu -- products of 8-bit integers with a scale for each row of both
// operands, for one matrix or for the experts' matrices:
//
//   out[r, c] = (sum_k a[r, k] b[g, c, k]) sa[r] sb[g, c]      rows r of group g
//   SwiGLU:     out[r, c] = silu(gate) up, gate and up the products with b[g, c]
//               and b[g, N + c]
//
// The sums are exact (int32); they are rounded to fp32 once, then each product
// and the output are rounded once.  Groups are runs of rows: group g owns rows
// offsets[g] .. offsets[g + 1] - 1 (expert order).
//
// int8_rows_kernel: the weights' channels are the M side of the MMA (128 per
// tile, tcgen05 kind::i8, M = 128) and the rows are its N side, as many columns
// as the tile has rows (rounded up to 16, at most 128).  With few rows per group
// every weight byte is brought into shared memory once and the tensor core does
// no work on empty rows.  One persistent CTA per SM: warp 0 loads by TMA, warp 1
// issues the MMAs, warps 2-5 drain the accumulators (two, in turn).  The tile
// list is not stored anywhere: every CTA sums the groups' tile counts from the
// offsets, and finds an item's group by a search over those sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "int8_common.cuh"
#include "pdl.cuh"

namespace moe {

namespace {

using namespace int8;

constexpr int kThreads = 192;
constexpr int kTileChannels = 128;
constexpr int kTileRows = 128;
constexpr int kRowBox = 32;                  // rows of one TMA box of a
constexpr int kBBytes = kTileChannels * kStageK;
constexpr int kABytes = kTileRows * kStageK;
constexpr int kTmemCols = 512;

template <bool SWIGLU>
struct Smem {
  static constexpr int stages = SWIGLU ? 4 : 6;
  static constexpr int b_bytes = (SWIGLU ? 2 : 1) * kBBytes;
  static constexpr int a_off = stages * b_bytes;
  static constexpr int bar_off = a_off + stages * kABytes;
  // full[stages], empty[stages], acc_full[2], acc_empty[2], drain
  static constexpr int n_bars = 2 * stages + 5;
  static constexpr int tmem_slot_off = bar_off + n_bars * 8;
  static constexpr int first_tile_off = tmem_slot_off + 16;  // kMaxGroups + 1 ints
  static constexpr int first_row_off = first_tile_off + (kMaxGroups + 4) * 4;
  static constexpr int total = first_row_off + (kMaxGroups + 4) * 4;
};
static_assert(Smem<true>::total + 1024 <= 232448 && Smem<false>::total + 1024 <= 232448,
              "shared memory budget");

template <typename TO, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    int8_rows_kernel(const __grid_constant__ Int8GemmParams p,
                     const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b) {
  using S = Smem<SWIGLU>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::bar_off);
  uint64_t *empty = full + S::stages;
  uint64_t *acc_full = empty + S::stages;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::tmem_slot_off);
  int *first_tile = reinterpret_cast<int *>(smem + S::first_tile_off);
  int *first_row = reinterpret_cast<int *>(smem + S::first_row_off);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  early_start();
  group_tiles(p, kTileRows, first_tile, first_row);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_items = first_tile[p.G] * p.n_ctiles;
  const int n_kb = (p.K + kStageK - 1) / kStageK;
  constexpr int kAccStride = SWIGLU ? 256 : 128;  // TMEM columns of one accumulator set

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long long issued = 0;
      int group = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x) {
        const Work w = find_work(p, kTileRows, item, first_tile, first_row, group);
        const int boxes = (w.nrows + kRowBox - 1) / kRowBox;
        const int brow = w.group * p.b_rows + (w.ctile * kTileChannels);
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1, p.status, SITE_GEMM_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], S::b_bytes + boxes * kRowBox * kStageK);
          uint8_t *b_dst = smem + s * S::b_bytes;
          uint8_t *a_dst = smem + S::a_off + s * kABytes;
          tma_load_2d(b_dst, &tm_b, &full[s], kb * kStageK, brow);
          if (SWIGLU) tma_load_2d(b_dst + kBBytes, &tm_b, &full[s], kb * kStageK, brow + p.N);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(a_dst + b * kRowBox * kStageK, &tm_a, &full[s], kb * kStageK,
                        w.row0 + b * kRowBox);
          ++issued;
          if (++s == S::stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // every load has landed before the CTA exits
      for (long long n = issued > S::stages ? issued - S::stages : 0; n < issued; ++n)
        if (!mbar_wait(&full[n % S::stages], static_cast<uint32_t>((n / S::stages) & 1), p.status,
                       SITE_GEMM_DRAIN))
          break;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      int group = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x) {
        const Work w = find_work(p, kTileRows, item, first_tile, first_row, group);
        const uint32_t idesc = idesc_i8_s32(kTileChannels, (w.nrows + 15) / 16 * 16);
        if (!mbar_wait(&acc_empty[acc], aph ^ 1, p.status, SITE_GEMM_MMA_ACC_EMPTY)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kAccStride;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!mbar_wait(&full[s], ph, p.status, SITE_GEMM_MMA_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b0 = smem_u32(smem + s * S::b_bytes);
          const uint32_t a0 = smem_u32(smem + S::a_off + s * kABytes);
#pragma unroll
          for (int kk = 0; kk < kStageK / 32; ++kk) {
            umma_i8_ss(d_tmem, smem_desc_sw128(b0 + kk * 32), smem_desc_sw128(a0 + kk * 32), idesc,
                       (kb | kk) != 0);
            if (SWIGLU)
              umma_i8_ss(d_tmem + 128, smem_desc_sw128(b0 + kBBytes + kk * 32),
                         smem_desc_sw128(a0 + kk * 32), idesc, (kb | kk) != 0);
          }
          umma_commit(&empty[s]);
          if (++s == S::stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(&acc_full[acc]);
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
      }
      umma_commit(drain);
      mbar_wait(drain, 0, p.status, SITE_GEMM_DRAIN);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;  // this warp's quarter of the accumulator's lanes
    int acc = 0;
    uint32_t aph = 0;
    int group = 0;
    float amax = 0.f;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const Work w = find_work(p, kTileRows, item, first_tile, first_row, group);
      const int chan = (w.ctile * kTileChannels) + q * 32 + lane;
      const bool on = chan < p.N;
      const float *sb = p.sb + static_cast<int64_t>(w.group) * p.b_rows + chan;
      const float sb0 = on ? sb[0] : 0.f;
      const float sb1 = SWIGLU && on ? sb[p.N] : 0.f;
      if (!mbar_wait(&acc_full[acc], aph, p.status, SITE_GEMM_EPI_ACC_FULL)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * kAccStride;
      TO *out = static_cast<TO *>(p.out) + static_cast<int64_t>(w.row0) * p.out_stride + chan;
      for (int c = 0; c < w.nrows; c += 16) {
        uint32_t d0[16], d1[16];
        tmem_ld_32x32b_x16(taddr + c, d0);
        if (SWIGLU) tmem_ld_32x32b_x16(taddr + 128 + c, d1);
        const float sa_lane = c + (lane & 15) < w.nrows ? p.sa[w.row0 + c + (lane & 15)] : 0.f;
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float sa = __shfl_sync(0xffffffffu, sa_lane, i);
          float v = static_cast<float>(static_cast<int>(d0[i])) * sa * sb0;
          if (SWIGLU) v = silu(v) * (static_cast<float>(static_cast<int>(d1[i])) * sa * sb1);
          if (on && c + i < w.nrows) {
            out[(c + i) * p.out_stride] = rows::from_f32<TO>(v);
            amax = fmaxf(amax, fabsf(v));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1;
      }
    }
    if (std::is_same<TO, __half>::value && __half2float(__float2half_rn(amax)) == INFINITY)
      record_status(p.status, MOE_ERR_DEVICE_BOUNDS, SITE_H_FP16_RANGE);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <typename TO, bool SWIGLU>
cudaError_t launch_rows(const Int8GemmParams &p, const CUtensorMap &a, const CUtensorMap &b,
                        int grid, cudaStream_t s) {
  return launch_early(int8_rows_kernel<TO, SWIGLU>, grid, kThreads, Smem<SWIGLU>::total + 1024, s,
                      p, a, b);
}

template <typename TO>
cudaError_t set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(int8_rows_kernel<TO, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<false>::total + 1024);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(int8_rows_kernel<TO, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Smem<true>::total + 1024);
}

}  // namespace

cudaError_t int8_gemm_set_attributes() {
  cudaError_t e = set_attributes<__nv_bfloat16>();
  if (e == cudaSuccess) e = set_attributes<__half>();
  if (e == cudaSuccess) e = set_attributes<float>();
  return e;
}

cudaError_t launch_int8_gemm(Int8GemmParams p, int out_type, bool swiglu, const void *a,
                             int64_t a_stride, const void *b, int64_t b_stride, int sms,
                             cudaStream_t s) {
  CUtensorMap ma, mb;
  if (!encode_map_u8(&ma, a, p.M, p.K, a_stride, kRowBox) ||
      !encode_map_u8(&mb, b, static_cast<uint64_t>(p.G) * p.b_rows, p.K, b_stride, kTileChannels))
    return cudaErrorInvalidValue;
  p.n_ctiles = (p.N + kTileChannels - 1) / kTileChannels;
  // at most this many tiles (the device knows the groups' rows)
  const int64_t tiles = (static_cast<int64_t>(p.M) + kTileRows - 1) / kTileRows + p.G - 1;
  const int grid = static_cast<int>(std::min<int64_t>(sms, tiles * p.n_ctiles));
  switch (out_type) {
    case MOE_DTYPE_BF16:
      return swiglu ? launch_rows<__nv_bfloat16, true>(p, ma, mb, grid, s)
                    : launch_rows<__nv_bfloat16, false>(p, ma, mb, grid, s);
    case MOE_DTYPE_F16:
      return swiglu ? launch_rows<__half, true>(p, ma, mb, grid, s)
                    : launch_rows<__half, false>(p, ma, mb, grid, s);
    default:
      return swiglu ? launch_rows<float, true>(p, ma, mb, grid, s)
                    : launch_rows<float, false>(p, ma, mb, grid, s);
  }
}

}  // namespace moe
