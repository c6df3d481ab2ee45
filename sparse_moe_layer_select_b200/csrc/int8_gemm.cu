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
// int8_rows_kernel (few rows per group; int8_gemm_pair.cu has the other case): the
// weights' channels are the M side of the MMA (128 per tile, tcgen05 kind::i8,
// M = 128) and the rows are its N side, as many columns as the tile has rows
// (rounded up to 16, at most TR).  A weight byte is brought into shared memory once for
// every TR rows of its group: once for groups of up to 128 rows; ceil(M / 32) times for one
// matrix of M rows, whose tiles have 32 so that they spread over more SMs (from L2 after the
// first: 64 x 4096 x 8192 takes 19 us, 95 x 4096 x 4096 14.4, against 5 and 3 at HBM speed).
// The tensor core does no work on empty rows; the weights' bytes bound it.
// One persistent CTA per SM: warp 0 loads by TMA, warp 1 issues the MMAs, warps 2-5
// and 6-9 drain the two accumulators, each set every second item: an item of few rows
// is waiting for memory (its scales), and with one set that took longer than a short
// item's weights (K = 512: 62 us for 268 MB).  The tile list is not stored anywhere:
// every CTA sums the groups' tile counts from the offsets and finds its items' groups
// by a search over those sums, before it starts.
//
// One matrix (TR = 32; groups: TR = 128) with fewer tiles than SMs is cut along K as
// well: a cluster of up to 8 CTAs takes a tile, each a share of K, and sends its
// integer sums to the CTA that owns their rows (through distributed shared memory;
// integers, so the order of the sums does not matter).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "int8_common.cuh"
#include "pdl.cuh"

namespace moe {

namespace {

using namespace int8;

constexpr int kThreads = 320;
constexpr int kTileChannels = 128;
constexpr int kRowBox = 32;  // rows of one TMA box of a
constexpr int kBBytes = kTileChannels * kStageK;

template <bool SWIGLU, int TR>
struct Smem {
  static constexpr int n_acc = SWIGLU ? 2 : 1;  // accumulators of a tile: gate and up
  static constexpr int stages = TR == 32 ? (SWIGLU ? 5 : 10) : (SWIGLU ? 4 : 6);
  static constexpr int a_bytes = TR * kStageK;
  static constexpr int b_bytes = n_acc * kBBytes;
  static constexpr int a_off = stages * b_bytes;
  static constexpr int sums_off = a_off + stages * a_bytes;  // sums received (TR = 32 only)
  static constexpr int bar_off = sums_off + (TR == 32 ? n_acc * TR * kTileChannels * 4 : 0);
  // full[stages], empty[stages], acc_full[2], acc_empty[2], drain, sums_full
  static constexpr int n_bars = 2 * stages + 6;
  static constexpr int tmem_slot_off = bar_off + n_bars * 8;
  static constexpr int first_tile_off = tmem_slot_off + 16;  // kMaxGroups + 1 ints
  static constexpr int first_row_off = first_tile_off + (kMaxGroups + 4) * 4;
  static constexpr int list_off = (first_row_off + (kMaxGroups + 4) * 4 + 15) / 16 * 16;
  static constexpr int total = list_off + kListed * static_cast<int>(sizeof(Work));
  static constexpr int tmem_cols = 2 * n_acc * TR;  // two accumulator sets
  static_assert(total + 1024 <= 232448, "shared memory budget");
};

template <typename TO, bool SWIGLU, int TR>
__global__ void __launch_bounds__(kThreads, 1)
    int8_rows_kernel(const __grid_constant__ Int8GemmParams p,
                     const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b) {
  using S = Smem<SWIGLU, TR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::bar_off);
  uint64_t *empty = full + S::stages;
  uint64_t *acc_full = empty + S::stages;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint64_t *sums_full = drain + 1;
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
    mbar_init(sums_full, 4 * p.ksplit);  // the epilogue warps of every CTA of the cluster
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(tmem_slot, S::tmem_cols);
    tmem_relinquish();
  }
  wait_for_kernels_ahead();
  group_tiles(p, TR, first_tile, first_row);
  tc_fence_before();
  __syncthreads();
  const int n_items = first_tile[p.G] * p.n_ctiles;
  const int first = blockIdx.x / p.ksplit;
  const int step = gridDim.x / p.ksplit;
  Work *list = reinterpret_cast<Work *>(smem + S::list_off);
  list_items(p, TR, first, step, n_items, first_tile, first_row, list);
  const ItemList items{list, first_tile, first_row, first, step};
  const int count = first < n_items ? (n_items - first + step - 1) / step : 0;  // its items
  __syncthreads();
  if (p.ksplit > 1) cluster_sync();  // the others' barriers are ready before any arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_kb = (p.K + kStageK - 1) / kStageK;
  constexpr int kAccStride = S::n_acc * TR;  // TMEM columns of one accumulator set
  // this CTA's share of K (all of it without a cluster), the same items for a whole cluster
  const int rank = p.ksplit > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int kb0 = static_cast<int>(static_cast<int64_t>(n_kb) * rank / p.ksplit);
  const int kb1 = static_cast<int>(static_cast<int64_t>(n_kb) * (rank + 1) / p.ksplit);

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      for (int i = 0; ok && i < count; ++i) {
        const Work w = items(p, TR, i);
        const int boxes = (w.nrows + kRowBox - 1) / kRowBox;
        const int brow = w.group * p.b_rows + (w.ctile * kTileChannels);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1, p.status, SITE_GEMM_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], S::b_bytes + boxes * kRowBox * kStageK);
          uint8_t *b_dst = smem + s * S::b_bytes;
          uint8_t *a_dst = smem + S::a_off + s * S::a_bytes;
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
      bool ok = true;
      for (int i = 0; ok && i < count; ++i) {
        const Work w = items(p, TR, i);
        const uint32_t idesc = idesc_i8_s32(kTileChannels, (w.nrows + 15) / 16 * 16);
        if (!mbar_wait(&acc_empty[acc], aph ^ 1, p.status, SITE_GEMM_MMA_ACC_EMPTY)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kAccStride;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[s], ph, p.status, SITE_GEMM_MMA_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b0 = smem_u32(smem + s * S::b_bytes);
          const uint32_t a0 = smem_u32(smem + S::a_off + s * S::a_bytes);
#pragma unroll
          for (int kk = 0; kk < kStageK / 32; ++kk) {
            umma_i8_ss(d_tmem, smem_desc_sw128(b0 + kk * 32), smem_desc_sw128(a0 + kk * 32), idesc,
                       kb != kb0 || kk != 0);
            if (SWIGLU)
              umma_i8_ss(d_tmem + TR, smem_desc_sw128(b0 + kBBytes + kk * 32),
                         smem_desc_sw128(a0 + kk * 32), idesc, kb != kb0 || kk != 0);
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
    const int q = warp & 3;            // this warp's quarter of the accumulator's lanes
    const int set = (warp - 2) >> 2;   // its accumulator: every second item's
    uint32_t aph = 0;
    float amax = 0.f;
    // (an item's scales are loaded while the set's item before it is worked on)
    Work next{};
    float next_sb0 = 0.f, next_sb1 = 0.f, next_sa[TR / 32];
    auto fetch = [&](int i) {
      if (i >= count) return;
      next = items(p, TR, i);
      const int chan = next.ctile * kTileChannels + q * 32 + lane;
      if (chan < p.N) {
        const float *sb = p.sb + static_cast<int64_t>(next.group) * p.b_rows + chan;
        next_sb0 = sb[0];
        if (SWIGLU) next_sb1 = sb[p.N];
      }
#pragma unroll
      for (int u = 0; u < TR / 32; ++u)
        next_sa[u] = 32 * u + lane < next.nrows ? p.sa[next.row0 + 32 * u + lane] : 0.f;
    };
    fetch(set);
    for (int it = set; it < count; it += 2) {
      const Work w = next;
      const int chan = (w.ctile * kTileChannels) + q * 32 + lane;
      const bool on = chan < p.N;
      const float sb0 = next_sb0, sb1 = next_sb1;
      float sa_lane[TR / 32];
#pragma unroll
      for (int i = 0; i < TR / 32; ++i) sa_lane[i] = next_sa[i];
      fetch(it + 2);
      if (!mbar_wait(&acc_full[set], aph, p.status, SITE_GEMM_EPI_ACC_FULL)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + set * kAccStride;
      TO *out = static_cast<TO *>(p.out) + static_cast<int64_t>(w.row0) * p.out_stride + chan;
      if (TR == 32 && p.ksplit > 1) {  // (one item per cluster)
        // sums_off: [sender][accumulator][row of the owner's][channel]
        const int per = 32 / p.ksplit;  // rows of the tile that each CTA finishes
        const uint32_t sums = smem_u32(smem + S::sums_off);
        const int at = q * 32 + lane;
#pragma unroll
        for (int u = 0; u < S::n_acc; ++u) {
          for (int c = 0; c < w.nrows; c += 16) {
            uint32_t d[16];
            tmem_ld_32x32b_x16(taddr + u * TR + c, d);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int owner = (c + i) / per;
              const int slot = (rank * S::n_acc + u) * per + (c + i - owner * per);
              st_shared_cluster(map_shared_rank(sums + (slot * kTileChannels + at) * 4, owner),
                                d[i]);
            }
          }
        }
        fence_cluster();
        __syncwarp();
        if (lane < p.ksplit) mbar_arrive_release_cluster(map_shared_rank(smem_u32(sums_full), lane));
        if (!mbar_wait(sums_full, 0, p.status, SITE_GEMM_EPI_ACC_FULL)) break;
        fence_cluster();
        const int *recv = reinterpret_cast<const int *>(smem + S::sums_off) + at;
        for (int i = 0; i < per && rank * per + i < w.nrows; ++i) {
          int total[2] = {0, 0};
          for (int r = 0; r < p.ksplit; ++r)
#pragma unroll
            for (int u = 0; u < S::n_acc; ++u)
              total[u] += recv[((r * S::n_acc + u) * per + i) * kTileChannels];
          const int row = rank * per + i;
          const float sa = p.sa[w.row0 + row];
          float v = static_cast<float>(total[0]) * sa * sb0;
          if (SWIGLU) v = silu(v) * (static_cast<float>(total[1]) * sa * sb1);
          if (on) {
            out[row * p.out_stride] = rows::from_f32<TO>(v);
            amax = fmaxf(amax, fabsf(v));
          }
        }
        break;
      }
#pragma unroll
      for (int c = 0; c < TR; c += 16) {
        if (c >= w.nrows) break;
        uint32_t d0[16], d1[16];
        tmem_ld_32x32b_x16(taddr + c, d0);
        if (SWIGLU) tmem_ld_32x32b_x16(taddr + TR + c, d1);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float sa = __shfl_sync(0xffffffffu, sa_lane[c / 32], c % 32 + i);
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
      if (lane == 0) mbar_arrive(&acc_empty[set]);
      aph ^= 1;
    }
    if (std::is_same<TO, __half>::value && __half2float(__float2half_rn(amax)) == INFINITY)
      record_status(p.status, MOE_ERR_DEVICE_BOUNDS, SITE_H_FP16_RANGE);
  }

  tc_fence_before();
  __syncthreads();
  if (p.ksplit > 1) cluster_sync();  // no CTA leaves while another may still write to it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::tmem_cols);
  }
}

template <typename TO, bool SWIGLU, int TR>
cudaError_t launch_rows(const Int8GemmParams &p, const CUtensorMap &a, const CUtensorMap &b,
                        int grid, cudaStream_t s) {
  return launch_early(int8_rows_kernel<TO, SWIGLU, TR>, grid, kThreads,
                      Smem<SWIGLU, TR>::total + 1024, s, p.ksplit, p, a, b);
}

template <typename TO, bool SWIGLU, int TR>
cudaError_t set_one() {
  return cudaFuncSetAttribute(int8_rows_kernel<TO, SWIGLU, TR>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Smem<SWIGLU, TR>::total + 1024);
}

template <typename TO>
cudaError_t set_attributes() {
  cudaError_t e = set_one<TO, false, 32>();
  if (e == cudaSuccess) e = set_one<TO, false, 128>();
  if (e == cudaSuccess) e = set_one<TO, true, 32>();
  if (e == cudaSuccess) e = set_one<TO, true, 128>();
  return e;
}

template <typename TO>
cudaError_t launch_typed(const Int8GemmParams &p, bool swiglu, int tile_rows, const CUtensorMap &a,
                         const CUtensorMap &b, int grid, cudaStream_t s) {
  if (tile_rows == 32)
    return swiglu ? launch_rows<TO, true, 32>(p, a, b, grid, s)
                  : launch_rows<TO, false, 32>(p, a, b, grid, s);
  return swiglu ? launch_rows<TO, true, 128>(p, a, b, grid, s)
                : launch_rows<TO, false, 128>(p, a, b, grid, s);
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
  const int tile_rows = p.offsets == nullptr ? 32 : 128;
  p.n_ctiles = (p.N + kTileChannels - 1) / kTileChannels;
  // at most this many tiles (the device knows the groups' rows)
  const int64_t tiles = (static_cast<int64_t>(p.M) + tile_rows - 1) / tile_rows + p.G - 1;
  p.ksplit = 1;
  if (p.offsets == nullptr) {
    // The tiles are known here: K is cut while SMs would be idle, if it is long enough to
    // pay for the cluster.  us without / with: 1 row, N = 1024, K = 2048, 8 ways: 7.5 / 5.9;
    // 1 row, N = 4096, K = 8192, 4 ways: 21.9 / 10.3; 2 ways: 256 rows, N = 1024, K = 2048:
    // 9.6 / 11.9, 64 rows, N = 4096, K = 8192: 23.7 / 19.1.  (Clusters of 8 for up to 8
    // tiles only: more of them do not fit on the GPU at once with a CTA per SM, and 16 took
    // twice as long as 8.)
    const int n_kb = (p.K + kStageK - 1) / kStageK;
    const int64_t all = tiles * p.n_ctiles;
    if (all <= 8 && n_kb >= 16) p.ksplit = 8;
    else if (all * 4 <= sms && n_kb >= 12) p.ksplit = 4;
    else if (all * 2 <= sms && n_kb >= 48) p.ksplit = 2;
  }
  const int grid = static_cast<int>(std::min<int64_t>(sms, tiles * p.n_ctiles * p.ksplit));
  switch (out_type) {
    case MOE_DTYPE_BF16: return launch_typed<__nv_bfloat16>(p, swiglu, tile_rows, ma, mb, grid, s);
    case MOE_DTYPE_F16: return launch_typed<__half>(p, swiglu, tile_rows, ma, mb, grid, s);
    default: return launch_typed<float>(p, swiglu, tile_rows, ma, mb, grid, s);
  }
}

}  // namespace moe
