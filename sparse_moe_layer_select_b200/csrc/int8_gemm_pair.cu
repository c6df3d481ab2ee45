// int8_gemm_pair.cu -- the product of 8-bit integers (int8_gemm.cu) on CTA pairs,
// for groups that fill 256-row tiles.
//
// A cluster of two SMs computes a tile of 256 rows by 256 channels (SwiGLU: 128
// gate and the 128 up channels of the same outputs) with tcgen05.mma.cta_group::2
// kind::i8, M = 256: each SM holds its own 128 rows of a and half of the channels'
// rows of b, so every byte brought into shared memory feeds 256 rows or columns.
// The rows are the accumulator's lanes, so a lane of the epilogue owns a row: it reads
// 32 columns at a time, the next 32 in flight, scales them by its row's scale and the
// channels' scales (staged in shared memory per tile) and packs 64 bytes of output; a
// warp's 32 rows of them go out as one TMA box.  (Plain stores, by way of shared memory
// or not, and TMA boxes of 8 warps were slower: the epilogue is bound by the load/store
// pipe, and with 8 warps each box waited for the last one's read.)  Boxes that cross the
// end of a group, and outputs whose rows are no multiple of 16 bytes apart, are stored
// from shared memory row by row.
//
// 16384 x 2048 x 4096: 88 to 92 us in a burst, 3.0e15 operations a second; 109 in a loop of a
// second, which the power cap holds at 1.2 to 1.4 GHz.  262144 rows of 256 experts of unequal
// size, one launch (in such a loop): gate/up with SwiGLU (N = 512, K = 2048) 485 us (600), down
// (N = 2048, K = 512) 338 (416); of 1024 rows each 455 and 317, as one group 420 and 300.
// At 96 registers a thread (the most for 576 threads) three of the six forms spill 4 to 12
// bytes: fp32 without SwiGLU, bf16 and fp16 with it.
//
// Warps: 0 loads (TMA), 1 MMA issue (leader CTA), 2-17 epilogue, four to a quarter of
// the lanes, each with a quarter of the columns.  Barriers as in moe_gemm_pair.cu's
// down GEMM: both CTAs' loads complete on the leader's full[s], commits go to both CTAs.
// No TMA or bulk copy uses cluster multicast.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "int8_common.cuh"
#include "pdl.cuh"

namespace moe {

namespace {

using namespace int8;

constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTileRows = 256;
constexpr int kHalfRows = 128;                 // rows of a, and of b, per CTA
constexpr int kOpBytes = kHalfRows * kStageK;  // 16 KB
constexpr int kBoxBytes = 32 * 64;             // one output box: 64 bytes of 32 rows
constexpr int kTmemCols = 512;
constexpr int kAccStride = 256;

// Shared memory: the barriers and tables first, then (on a 1024-byte boundary) the ring of
// `ring` stages and the epilogue warps' boxes, `boxes` each.  Long sums need the deeper
// ring, short ones a second box (a tile is then finished sooner than a box is stored):
// 5 stages and one box each, or 4 and two.  Product of 131072 rows, 128 groups: 209 us
// against 225 at K = 2048 (SwiGLU, fp32 out, N = 512), 178 against 156 at K = 512
// (fp16 out, N = 2048).
constexpr int kShortK = 1024;
constexpr int kMaxRing = 5;
struct Smem {
  static constexpr int tmem_slot_off = 0;
  static constexpr int bar_off = 16;
  // full[kMaxRing], empty[kMaxRing], acc_full[2], acc_empty[2], drain
  static constexpr int n_bars = 2 * kMaxRing + 5;
  static constexpr int scale_off = bar_off + (n_bars + 1) * 8;  // 64 channel scales per warp
  static constexpr int first_tile_off = scale_off + kEpiWarps * 64 * 4;
  static constexpr int first_row_off = first_tile_off + (kMaxGroups + 4) * 4;
  static constexpr int list_off = (first_row_off + (kMaxGroups + 4) * 4 + 15) / 16 * 16;
  static constexpr int ring_off =
      (list_off + kListed * static_cast<int>(sizeof(Work)) + 1023) / 1024 * 1024;
  static constexpr int bytes(int ring, int boxes) {
    return ring_off + ring * 2 * kOpBytes + boxes * kEpiWarps * kBoxBytes;
  }
};
static_assert(Smem::bytes(5, 1) + 1024 <= 232448 && Smem::bytes(4, 2) + 1024 <= 232448,
              "shared memory budget");
static_assert(Smem::scale_off % 16 == 0, "alignment");

// Issues the load of piece i of a tile: 32 accumulator columns, for SwiGLU 16 gate
// columns and the 16 up columns of the same outputs.
template <bool SWIGLU>
__device__ __forceinline__ void load_piece(uint32_t taddr, int i, uint32_t (&d)[32]) {
  if (SWIGLU) {
    uint32_t(&lo)[16] = *reinterpret_cast<uint32_t(*)[16]>(&d[0]);
    uint32_t(&hi)[16] = *reinterpret_cast<uint32_t(*)[16]>(&d[16]);
    tmem_ld_32x32b_x16(taddr + 16 * i, lo);
    tmem_ld_32x32b_x16(taddr + 128 + 16 * i, hi);
  } else {
    tmem_ld_32x32b_x32(taddr + 32 * i, d);
  }
}

// The outputs of a piece: 32 columns, or 16 (SwiGLU).  sc: the warp's channel scales,
// 64 of them (SwiGLU: 32 gate scales, 32 up scales).
template <bool SWIGLU>
__device__ __forceinline__ void scaled_piece(const uint32_t (&d)[32], int i, float sa,
                                             const float *sc, float (&v)[32]) {
  constexpr int kOut = SWIGLU ? 16 : 32;
#pragma unroll
  for (int c = 0; c < kOut; c += 4) {
    const float4 s = *reinterpret_cast<const float4 *>(sc + kOut * i + c);
    scaled2(d[c], d[c + 1], sa, s.x, s.y, &v[c], &v[c + 1]);
    scaled2(d[c + 2], d[c + 3], sa, s.z, s.w, &v[c + 2], &v[c + 3]);
    if (SWIGLU) {
      const float4 u = *reinterpret_cast<const float4 *>(sc + 32 + kOut * i + c);
      float up[4];
      scaled2(d[(16 + c) % 32], d[(17 + c) % 32], sa, u.x, u.y, &up[0], &up[1]);
      scaled2(d[(18 + c) % 32], d[(19 + c) % 32], sa, u.z, u.w, &up[2], &up[3]);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[c + q] = silu(v[c + q]) * up[q];
    }
  }
}

}  // namespace

template <typename TO, bool SWIGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    int8_pair_kernel(const __grid_constant__ Int8GemmParams p,
                     const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_out) {
  using S = Smem;
  constexpr int kTileChannels = SWIGLU ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int ring = p.ring;
  uint8_t *sA = smem + S::ring_off;
  uint8_t *sB = sA + ring * kOpBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::bar_off);
  uint64_t *empty = full + kMaxRing;
  uint64_t *acc_full = empty + kMaxRing;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::tmem_slot_off);
  int *first_tile = reinterpret_cast<int *>(smem + S::first_tile_off);
  int *first_row = reinterpret_cast<int *>(smem + S::first_row_off);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 32) {
    for (int s = 0; s < ring; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  wait_for_kernels_ahead();
  group_tiles(p, kTileRows, first_tile, first_row);
  tc_fence_before();
  __syncthreads();
  const int n_items = first_tile[p.G] * p.n_ctiles;
  const int first = blockIdx.x >> 1;
  const int step = gridDim.x >> 1;
  Work *list = reinterpret_cast<Work *>(smem + S::list_off);
  list_items(p, kTileRows, first, step, n_items, first_tile, first_row, list);
  const ItemList items{list, first_tile, first_row, first, step};
  const int count = first < n_items ? (n_items - first + step - 1) / step : 0;  // its items
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_kb = (p.K + kStageK - 1) / kStageK;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t leader_full0 = map_shared_rank(smem_u32(&full[0]), 0);
      int s = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      for (int i = 0; ok && i < count; ++i) {
        const Work w = items(p, kTileRows, i);
        const int arow = w.row0 + static_cast<int>(rank) * kHalfRows;
        // SwiGLU: the leader loads the gate channels, its peer the up channels
        const int brow = w.group * p.b_rows + w.ctile * kTileChannels +
                         static_cast<int>(rank) * (SWIGLU ? p.N : kHalfRows);
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1, p.status, SITE_GEMM_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[s], 4 * kOpBytes);  // both CTAs' boxes
          const uint32_t bar = leader_full0 + s * 8;
          tma_load_2d_pair(sA + s * kOpBytes, &tm_a, bar, kb * kStageK, arow);
          tma_load_2d_pair(sB + s * kOpBytes, &tm_b, bar, kb * kStageK, brow);
          ++issued;
          if (++s == ring) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // the leader's full[] counts both CTAs' bytes; its peer stays until the closing
      // cluster barrier, which the leader reaches after they have landed
      if (leader)
        for (long long n = issued > ring ? issued - ring : 0; n < issued; ++n)
          if (!mbar_wait(&full[n % ring], static_cast<uint32_t>((n / ring) & 1), p.status,
                         SITE_GEMM_DRAIN))
            break;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && lane == 0) {
      constexpr uint32_t idesc = idesc_i8_s32(2 * kHalfRows, 256);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int i = 0; ok && i < count; ++i) {
        if (!mbar_wait(&acc_empty[acc], aph ^ 1, p.status, SITE_GEMM_MMA_ACC_EMPTY)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kAccStride;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!mbar_wait(&full[s], ph, p.status, SITE_GEMM_MMA_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * kOpBytes);
          const uint32_t b0 = smem_u32(sB + s * kOpBytes);
#pragma unroll
          for (int kk = 0; kk < kStageK / 32; ++kk)
            umma_i8_ss_pair(d_tmem, smem_desc_sw128(a0 + kk * 32), smem_desc_sw128(b0 + kk * 32),
                            idesc, (kb | kk) != 0);
          umma_commit_pair_multicast(&empty[s], 0x3);
          if (++s == ring) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit_pair_multicast(&acc_full[acc], 0x3);
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
      }
      umma_commit_pair_multicast(drain, 0x1);
      mbar_wait(drain, 0, p.status, SITE_GEMM_DRAIN);
    }
    __syncwarp();
  } else {
    constexpr int kWarpCols = kTileChannels / 4;               // outputs of this warp per row
    constexpr int kPieceCols = kWarpCols / 2;
    constexpr int kCols = 64 / static_cast<int>(sizeof(TO));   // columns of an output box
    constexpr int kVec = 16 / static_cast<int>(sizeof(TO));
    const int q = warp & 3;              // this warp's quarter of the accumulator's lanes
    const int part = (warp - 2) >> 2;    // and its quarter of the columns
    const uint32_t leader_acc_empty0 = map_shared_rank(smem_u32(&acc_empty[0]), 0);
    uint8_t *box = sB + ring * kOpBytes + (warp - 2) * p.boxes * kBoxBytes;
    uint32_t which = 0;  // the box to fill next
    float *sc = reinterpret_cast<float *>(smem + S::scale_off) + (warp - 2) * 64;
    TO *out = static_cast<TO *>(p.out);
    const int warp_row = static_cast<int>(rank) * kHalfRows + q * 32;  // within the tile
    int acc = 0;
    uint32_t aph = 0;
    uint32_t largest = 0;  // of the fp16 outputs, even and odd columns
    // a tile's scales are loaded while the tile before it is worked on
    Work next{};
    float next_sb[2], next_sa = 0.f;
    auto fetch = [&](int i) {
      if (i >= count) return;
      next = items(p, kTileRows, i);
      const float *sb = p.sb + static_cast<int64_t>(next.group) * p.b_rows;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int chan =
            next.ctile * kTileChannels + part * kWarpCols + lane + (SWIGLU ? 0 : 32 * u);
        next_sb[u] = chan < p.N ? sb[(SWIGLU ? u * p.N : 0) + chan] : 0.f;
      }
      next_sa = warp_row + lane < next.nrows ? p.sa[next.row0 + warp_row + lane] : 0.f;
    };
    fetch(0);
    for (int it = 0; it < count; ++it) {
      const Work w = next;
      const float sa = next_sa;
      const int chan0 = w.ctile * kTileChannels + part * kWarpCols;
      const int row0 = w.row0 + warp_row;
      const bool any = warp_row < w.nrows && chan0 < p.N;
      __syncwarp();  // the previous tile's scales have been read
#pragma unroll
      for (int i = 0; i < 2; ++i) sc[i * 32 + lane] = next_sb[i];
      __syncwarp();
      fetch(it + 1);
      if (!mbar_wait(&acc_full[acc], aph, p.status, SITE_GEMM_EPI_ACC_FULL)) break;
      tc_fence_after();
      if (any) {
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                               acc * kAccStride + part * kWarpCols;
        uint32_t d[2][32], words[16];
        load_piece<SWIGLU>(taddr, 0, d[0]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tmem_ld_wait_for(d[i]);
          if (i == 0) {
            load_piece<SWIGLU>(taddr, 1, d[1]);
          } else {  // the accumulator has been read: the next tile's products may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_acc_empty0 + acc * 8);
          }
          float v[32];
          scaled_piece<SWIGLU>(d[i], i, sa, sc, v);
#pragma unroll
          for (int c = 0; c < kPieceCols; ++c) {
            const int at = (i * kPieceCols + c) % kCols;  // column of the box
            if (sizeof(TO) == 4) words[at % 16] = __float_as_uint(v[c]);
            else if (c % 2 == 0) words[at / 2] = rows::pack2<TO>(v[c], v[(c + 1) % 32]);
            if (std::is_same<TO, __half>::value && c % 2 == 0)
              largest = larger_half2(largest, words[at / 2]);
            if (at + 1 < kCols) continue;
            // a box is filled; it goes through shared memory, in the 64-byte swizzle
            const int cb = i * kPieceCols + c + 1 - kCols;
            if (lane == 0) {  // the store that last used this box has read it
              if (p.boxes == 2) bulk_wait_read_le1();
              else bulk_wait_read_all();
            }
            __syncwarp();
            uint8_t *const here = box + which * kBoxBytes;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4 *>(here + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(words[4 * u], words[4 * u + 1], words[4 * u + 2], words[4 * u + 3]);
            if (warp_row + 32 <= w.nrows && p.tma_out && (chan0 + cb + kCols <= p.N || p.tma_clips)) {
              // whole rows of a group: one TMA store (which leaves out channels past N, in
              // steps of 16 bytes)
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tm_out, here, chan0 + cb, row0);
                bulk_commit_group();
              }
              which ^= p.boxes - 1;
              continue;
            }
            __syncwarp();
            const int live = min(32, w.nrows - warp_row);
            if (p.tma_out && chan0 + cb + kCols <= p.N) {  // 64-byte pieces of 8 rows a store
              const int vec = lane & 3;
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int r = 8 * u + (lane >> 2);
                if (r >= live) break;
                *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(row0 + r) * p.out_stride +
                                           chan0 + cb + vec * kVec) =
                    *reinterpret_cast<const uint4 *>(here + r * 64 +
                                                     ((vec ^ ((r >> 1) & 3)) << 4));
              }
            } else {  // rows on no 16-byte boundary, or the last channels: a lane per element
              const int e = lane % kCols;
              if (chan0 + cb + e < p.N) {
                for (int r = lane / kCols; r < live; r += 32 / kCols) {
                  const uint8_t *src = here + r * 64 + (((e / kVec) ^ ((r >> 1) & 3)) << 4) +
                                       e % kVec * static_cast<int>(sizeof(TO));
                  out[static_cast<int64_t>(row0 + r) * p.out_stride + chan0 + cb + e] =
                      *reinterpret_cast<const TO *>(src);
                }
              }
            }
          }
        }
      }
      if (!any && lane == 0) mbar_arrive_cluster(leader_acc_empty0 + acc * 8);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1;
      }
    }
    if (lane == 0) bulk_wait_all();  // this warp's stores are complete
    if (std::is_same<TO, __half>::value && half2_overflows(largest))
      record_status(p.status, MOE_ERR_DEVICE_BOUNDS, SITE_H_FP16_RANGE);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still read its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

namespace {

template <typename TO, bool SWIGLU>
cudaError_t set_one() {
  return cudaFuncSetAttribute(int8_pair_kernel<TO, SWIGLU>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              std::max(Smem::bytes(5, 1), Smem::bytes(4, 2)) + 1024);
}

template <typename TO, bool SWIGLU>
cudaError_t launch_one(const Int8GemmParams &p, const CUtensorMap &a, const CUtensorMap &b,
                       const CUtensorMap &out, int grid, cudaStream_t s) {
  return launch_early(int8_pair_kernel<TO, SWIGLU>, grid, kThreads,
                      Smem::bytes(p.ring, p.boxes) + 1024, s, 0, p, a, b, out);
}

}  // namespace

cudaError_t int8_pair_set_attributes() {
  cudaError_t e = set_one<__nv_bfloat16, false>();
  if (e == cudaSuccess) e = set_one<__nv_bfloat16, true>();
  if (e == cudaSuccess) e = set_one<__half, false>();
  if (e == cudaSuccess) e = set_one<__half, true>();
  if (e == cudaSuccess) e = set_one<float, false>();
  if (e == cudaSuccess) e = set_one<float, true>();
  return e;
}

cudaError_t launch_int8_pair(Int8GemmParams p, int out_type, bool swiglu, const void *a,
                             int64_t a_stride, const void *b, int64_t b_stride, int clusters,
                             cudaStream_t s) {
  CUtensorMap ma, mb, mo;
  if (!encode_map_u8(&ma, a, p.M, p.K, a_stride, kHalfRows) ||
      !encode_map_u8(&mb, b, static_cast<uint64_t>(p.G) * p.b_rows, p.K, b_stride, kHalfRows))
    return cudaErrorInvalidValue;
  p.tma_out = p.out_stride * elem_size(out_type) % 16 == 0;
  p.tma_clips = static_cast<int64_t>(p.N) * elem_size(out_type) % 16 == 0;
  if (p.tma_out && !encode_out_map(&mo, p.out, out_type, p.M, p.N, p.out_stride))
    return cudaErrorInvalidValue;
  if (!p.tma_out) mo = ma;  // not used
  p.ring = p.K <= kShortK ? 4 : kMaxRing;
  p.boxes = p.K <= kShortK ? 2 : 1;
  const int channels = swiglu ? 128 : 256;
  p.n_ctiles = (p.N + channels - 1) / channels;
  const int64_t tiles = (static_cast<int64_t>(p.M) + kTileRows - 1) / kTileRows + p.G - 1;
  const int grid = 2 * static_cast<int>(std::min<int64_t>(clusters, tiles * p.n_ctiles));
  switch (out_type) {
    case MOE_DTYPE_BF16:
      return swiglu ? launch_one<__nv_bfloat16, true>(p, ma, mb, mo, grid, s)
                    : launch_one<__nv_bfloat16, false>(p, ma, mb, mo, grid, s);
    case MOE_DTYPE_F16:
      return swiglu ? launch_one<__half, true>(p, ma, mb, mo, grid, s)
                    : launch_one<__half, false>(p, ma, mb, mo, grid, s);
    default:
      return swiglu ? launch_one<float, true>(p, ma, mb, mo, grid, s)
                    : launch_one<float, false>(p, ma, mb, mo, grid, s);
  }
}

}  // namespace moe
