// bnn_fp8_gemm / bnn_fp8_grouped_gemm: matrix products of e4m3 operands with a
// float32 scale for each block of 128 (include/bnn.h has the format).
//
//   y[i,j] = sum_b xs[b,i] ws[j/128,b] sum_{e in block b} xq[i,e] wq[j,e] (+ bias[j])
//
// Both kernels (this file: few rows; fp8_gemm_tile.cu: more) run the inner sums
// on tcgen05.mma kind::f8f6f4 (K = 32, four per block of 128) and start a fresh
// accumulator for every block of k: the block's sum is read from tensor memory
// and added, times its scales, to float32 accumulators in registers.  The
// scales are arbitrary float32 numbers, so the tensor cores' own block scaling
// (powers of two) cannot apply them.
#include <cooperative_groups.h>

#include "fp8_common.cuh"

namespace {

using bnn::fp8::Args;
using bnn::tc::mbar_arrive;
using bnn::tc::mbar_expect_tx;
using bnn::tc::mma_commit;
using bnn::tc::smem_u32;
using bnn::tc::sw128_desc;
using bnn::tc::tma_load_2d;
using bnn::tc::tmem_ld16;
using bnn::tc::tmem_wait_ld;

// ---------------------------------------------------------------------------
// Few rows: weights on the tensor-memory lanes.
//
// Tile: 128 weight rows (one scale block: the weight scale of a block of k is
// one number for the CTA) x BN activation rows as the MMA's N, so a handful of
// rows costs a handful of columns and the weights stream once at whatever rate
// HBM gives.  Stages of one block of k (128 bytes a row, one 128-byte-swizzled
// TMA box per operand).  When the tiles leave SMs idle, a cluster of KS CTAs
// splits the blocks of k and adds its partial sums in rank order through
// distributed shared memory: the order is fixed, so results are reproducible.
//
// Roles: a TMA thread; an MMA thread; four epilogue warps, each 32 weight rows:
// they read a block's BN sums (tcgen05.ld), scale and add them.  The scales of
// the BN rows reach every lane through a per-warp line of shared memory, loaded
// ahead from global memory (coalesced: the scale matrix is block-major).
//
// Launched with programmatic dependent launch: the weights' first stages are
// fetched before the wait for the kernel ahead (not for groups, whose tiles
// depend on the offsets).
// ---------------------------------------------------------------------------
constexpr int kTm = 128;                    // weight rows of a tile
constexpr int kBlockBytes = 128;            // bytes of a row's block of k
constexpr int kEpi = 128;                   // epilogue threads
constexpr int kThreads = kEpi + 64;         // + TMA warp + MMA warp
constexpr int kTmaWarp = kEpi / 32, kMmaWarp = kTmaWarp + 1;
constexpr int kAhead = 4;                   // blocks whose activation scales are in flight

template <int BN>
struct Cfg {
  static constexpr uint32_t kStageBytes = (kTm + BN) * kBlockBytes;
  static constexpr int kStages = 5;                                  // two CTAs an SM (up to 113 KiB each)
  static constexpr int kBufs = 128 / BN;                               // accumulators in tensor memory
  static constexpr uint32_t kTmemCols = BN * kBufs;                  // 128: two CTAs (and the next kernel's) fit the 512
  static constexpr size_t kSmem = kStages * kStageBytes + 1024;
};
static_assert(Cfg<16>::kStageBytes % 1024 == 0 && Cfg<32>::kStageBytes % 1024 == 0, "swizzle atoms stay aligned");

template <int BN, int KS, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 2)
fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                  const float* __restrict__ xs, const float* __restrict__ ws, const float* __restrict__ bias,
                  const int64_t* __restrict__ offsets, int groups, int64_t rows, int64_t n, int kb,
                  void* __restrict__ out, int out_type, unsigned int* errors) {
  static_assert(KS == 1 || !GROUPED, "a split cluster takes one tile");
  namespace cg = cooperative_groups;
  using C = Cfg<BN>;
  constexpr int S = C::kStages, NB = C::kBufs;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], part_full[NB], part_empty[NB];
  __shared__ uint32_t tmem_holder;
  __shared__ int any_bad;
  __shared__ __align__(16) float scales[4][2][BN];
  __shared__ bnn::fp8::Groups<GROUPED ? BNN_MAX_GROUPS : 1> map;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem);
  const int rank = KS > 1 ? static_cast<int>(blockIdx.x % KS) : 0;
  const int wtiles = static_cast<int>((n + kTm - 1) / kTm);
  const int b0 = static_cast<int>(static_cast<int64_t>(kb) * rank / KS);
  const int b1 = static_cast<int>(static_cast<int64_t>(kb) * (rank + 1) / KS);

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bnn::tc::mbar_init(smem_u32(&full_bar[i]), 1);
      bnn::tc::mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      bnn::tc::mbar_init(smem_u32(&part_full[i]), 1);
      bnn::tc::mbar_init(smem_u32(&part_empty[i]), 4);
    }
    any_bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid == kTmaWarp * 32) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_holder)),
                 "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
  }
  if (GROUPED) {
    bnn::pdl_wait();  // the offsets may come from the preceding kernel
    if (warp == 0) bnn::fp8::build_groups<BN>(map, offsets, groups, rows, lane);
  } else if (tid == 0) {
    map.start[0] = 0;
    map.start[1] = static_cast<int>(rows);
    map.first[0] = 0;
    map.first[1] = static_cast<int>((rows + BN - 1) / BN);
  }
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
  const uint32_t tmem = tmem_holder;
  bnn::pdl_trigger();
  const int64_t tiles = static_cast<int64_t>(map.first[groups]) * wtiles;
  const int64_t step = gridDim.x / KS, tile0 = blockIdx.x / KS;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA copies
    uint32_t it = 0;  // stages issued
    bool ok = true, waited = GROUPED;
    for (int64_t tile = tile0; tile < tiles && ok; tile += step) {
      const bnn::fp8::Tile t = bnn::fp8::tile_at<BN>(tile, groups, map.start, map.first, wtiles);
      const int wrow = t.group * static_cast<int>(n) + t.wtile * kTm;
      int b = b0;
      if (!waited) {  // the first stages' weights, then the wait, then their activations
        const int ahead = min(S, b1 - b0);
        for (int i = 0; i < ahead; ++i) {
          if (bnn::fp8::elected()) {
            mbar_expect_tx(smem_u32(&full_bar[i]), C::kStageBytes);
            tma_load_2d(ring + i * C::kStageBytes, &tmap_w, (b0 + i) * kBlockBytes, wrow, smem_u32(&full_bar[i]));
          }
          __syncwarp();
        }
        bnn::pdl_wait();
        for (int i = 0; i < ahead; ++i) {
          if (bnn::fp8::elected())
            tma_load_2d(ring + i * C::kStageBytes + kTm * kBlockBytes, &tmap_x, (b0 + i) * kBlockBytes, t.row,
                        smem_u32(&full_bar[i]));
          __syncwarp();
        }
        b += ahead;
        it = static_cast<uint32_t>(ahead);
        waited = true;
      }
      for (; b < b1; ++b, ++it) {
        const int st = static_cast<int>(it % S);
        if (it >= static_cast<uint32_t>(S))
          ok = bnn::fp8::wait(smem_u32(&empty_bar[st]), (it / S + 1) & 1u, errors);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (bnn::fp8::elected()) {
          const uint32_t dst = ring + st * C::kStageBytes, bar = smem_u32(&full_bar[st]);
          mbar_expect_tx(bar, C::kStageBytes);
          tma_load_2d(dst, &tmap_w, b * kBlockBytes, wrow, bar);
          tma_load_2d(dst + kTm * kBlockBytes, &tmap_x, b * kBlockBytes, t.row, bar);
        }
        __syncwarp();
      }
    }
    // the CTA must not retire with copies in flight
    for (uint32_t c = it >= static_cast<uint32_t>(S) ? it - S : 0; c < it; ++c)
      bnn::tc::mbar_drain(smem_u32(&full_bar[c % S]), (c / S) & 1u, errors);
    if (KS > 1) {
      __syncwarp();
      cluster.sync();
      cluster.sync();
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    if (!GROUPED) bnn::pdl_wait();  // before the first bounded wait (for copies that start after it)
    constexpr uint32_t word = bnn::fp8::mma_word(kTm, BN);
    uint32_t it = 0;
    bool ok = true;
    for (int64_t tile = tile0; tile < tiles && ok; tile += step) {
      for (int b = b0; b < b1; ++b, ++it) {
        const int st = static_cast<int>(it % S), pb = static_cast<int>(it % NB);
        if (it >= static_cast<uint32_t>(NB))
          ok = bnn::fp8::wait(smem_u32(&part_empty[pb]), (it / NB + 1) & 1u, errors);
        if (ok) ok = bnn::fp8::wait(smem_u32(&full_bar[st]), (it / S) & 1u, errors);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
        if (bnn::fp8::elected()) {
          const uint64_t ad = sw128_desc(ring + st * C::kStageBytes);
          const uint64_t bd = sw128_desc(ring + st * C::kStageBytes + kTm * kBlockBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            asm volatile(
                "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem + pb * BN),
                "l"(ad + static_cast<uint64_t>(2 * kk)), "l"(bd + static_cast<uint64_t>(2 * kk)), "r"(word),
                "r"(kk > 0 ? 1u : 0u));
          mma_commit(smem_u32(&empty_bar[st]));
          mma_commit(smem_u32(&part_full[pb]));
        }
        __syncwarp();
      }
    }
    // every MMA issued has completed before the CTA's memory is given back
    for (uint32_t c = it >= static_cast<uint32_t>(S) ? it - S : 0; c < it; ++c)
      bnn::tc::mbar_drain(smem_u32(&empty_bar[c % S]), (c / S) & 1u, errors);
    if (KS > 1) {
      __syncwarp();
      cluster.sync();
      cluster.sync();
    }
  } else {
    // ------------------------------------------------------------ scale and add
    if (!GROUPED) bnn::pdl_wait();  // the activation scales may come from the preceding kernel
    constexpr int PL = (BN + 31) / 32;  // rows' scales a lane loads per block
    uint32_t it = 0;
    bool ok = true;
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    const int64_t nb = wtiles;
    for (int64_t tile = tile0; tile < tiles; tile += step) {
      const bnn::fp8::Tile t = bnn::fp8::tile_at<BN>(tile, groups, map.start, map.first, wtiles);
      const float* wsp = ws + (t.group * nb + t.wtile) * kb;
      const int live = min(BN, t.end - t.row);
      float acc[BN];
#pragma unroll
      for (int c = 0; c < BN; ++c) acc[c] = 0.0f;
      // both scales of the blocks ahead, multiplied when used: a product here would wait for its loads
      float px[kAhead][PL], pw[kAhead];
      auto load = [&](int b, int a) {
        pw[a] = b < b1 ? __ldg(wsp + b) : 0.0f;
#pragma unroll
        for (int p = 0; p < PL; ++p) {
          const int c = lane + 32 * p;
          px[a][p] = b < b1 && c < live ? __ldg(xs + b * rows + t.row + c) : 0.0f;
        }
      };
#pragma unroll
      for (int a = 0; a < kAhead; ++a) load(b0 + a, a);
      for (int b = b0; b < b1 && ok; b += kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (b + a < b1 && ok) {
            float* line = scales[warp][a & 1];
#pragma unroll
            for (int p = 0; p < PL; ++p)
              if (lane + 32 * p < BN) line[lane + 32 * p] = px[a][p] * pw[a];
            load(b + a + kAhead, a);
            const int pb = static_cast<int>(it % NB);
            ok = bnn::fp8::wait(smem_u32(&part_full[pb]), (it / NB) & 1u, errors);
            ok = __all_sync(0xffffffffu, ok);
            __syncwarp();  // every lane's part of `line` is written
            if (ok) {
              asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
#pragma unroll
              for (int c0 = 0; c0 < BN; c0 += 16) {
                uint32_t r[16];
                tmem_ld16(tmem + lanes + pb * BN + c0, r);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                  const float4 s = *reinterpret_cast<const float4*>(line + c0 + c);
                  acc[c0 + c] = fmaf(__uint_as_float(r[c]), s.x, acc[c0 + c]);
                  acc[c0 + c + 1] = fmaf(__uint_as_float(r[c + 1]), s.y, acc[c0 + c + 1]);
                  acc[c0 + c + 2] = fmaf(__uint_as_float(r[c + 2]), s.z, acc[c0 + c + 2]);
                  acc[c0 + c + 3] = fmaf(__uint_as_float(r[c + 3]), s.w, acc[c0 + c + 3]);
                }
              }
              asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
              __syncwarp();  // also orders this block's reads of `line` before its next writes
              if (lane == 0) mbar_arrive(smem_u32(&part_empty[pb]));
            }
            ++it;
          }
        }
      }
      const int64_t j = static_cast<int64_t>(t.wtile) * kTm + tid;
      const float bj = bias && j < n ? __ldg(bias + j) : 0.0f;
      if (KS == 1) {
        if (!ok) break;
        if (j < n) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (c < live) bnn::fp8::store_one(out, out_type, (t.row + c) * n + j, acc[c] + bj);
        }
      } else {
        // the cluster's sums: rank r adds columns [r BN / KS, (r + 1) BN / KS) of all ranks, in rank order
        constexpr int kCols = BN / KS;
        float* recv = reinterpret_cast<float*>(smem);
        cluster.sync();  // every CTA's tensor core is done with its stages
        if (!ok && lane == 0)
          for (int q = 0; q < KS; ++q) atomicExch(cluster.map_shared_rank(&any_bad, q), 1);
#pragma unroll
        for (int c = 0; c < BN; ++c)
          cluster.map_shared_rank(recv, c / kCols)[(rank * kCols + c % kCols) * kEpi + tid] = acc[c];
        cluster.sync();  // every share has landed
        if (j < n && !any_bad) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            float y = 0.0f;
#pragma unroll
            for (int q = 0; q < KS; ++q) y += recv[(q * kCols + c) * kEpi + tid];
            if (rank * kCols + c < live)
              bnn::fp8::store_one(out, out_type, (t.row + rank * kCols + c) * n + j, y + bj);
          }
        }
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::kTmemCols));
}

// k = 0: every sum is empty.
__global__ void fp8_empty_kernel(const float* __restrict__ bias, const int64_t* __restrict__ offsets, int groups,
                                 int64_t rows, int64_t n, void* __restrict__ out, int out_type) {
  int64_t lo = 0, hi = rows;
  if (offsets) {
    lo = max(int64_t{0}, min(rows, offsets[0]));
    hi = lo;
    for (int g = 1; g <= groups; ++g) hi = max(hi, min(rows, offsets[g]));
  }
  for (int64_t i = lo * n + blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < hi * n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    bnn::fp8::store_one(out, out_type, i, bias ? bias[i % n] : 0.0f);
}

bnn_status gemm_empty(const Args& a) {
  fp8_empty_kernel<<<2 * bnn::sm_count(), 256, 0, a.stream>>>(a.bias, a.offsets, a.groups, a.rows, a.n, a.out,
                                                              a.out_type);
  return bnn::check_launch();
}

template <int BN, int KS, bool GROUPED>
bnn_status launch_narrow(const Args& a) {
  const int64_t wtiles = (a.n + kTm - 1) / kTm;
  // groups: at most one ragged tile each beside the full ones
  const int64_t rtiles = GROUPED ? a.rows / BN + (a.rows < a.groups ? a.rows : a.groups) : (a.rows + BN - 1) / BN;
  const int64_t tiles = rtiles * wtiles, slots = 2 * bnn::sm_count();
  const int64_t ctas = KS > 1 ? tiles * KS : (tiles < slots ? tiles : slots);
  // grid limits, and stages counted in 32 bits
  if (ctas > INT32_MAX || (tiles + slots - 1) / slots * a.kb >= (int64_t{1} << 31)) return BNN_ERR_INVALID_ARG;
  CUtensorMap tw, tx;
  const uint64_t pitch = static_cast<uint64_t>(a.kb) * kBlockBytes;
  if (!bnn::encode_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq, pitch, static_cast<uint64_t>(a.groups * a.n),
                           pitch, kBlockBytes, kTm, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bnn::encode_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xq, pitch, static_cast<uint64_t>(a.rows), pitch,
                           kBlockBytes, BN, CU_TENSOR_MAP_SWIZZLE_128B))
    return BNN_ERR_UNSUPPORTED;
  unsigned int* errors = bnn::device_error_counter();
  if (!errors) return bnn::cuda_fail(cudaGetLastError());
  auto kern = fp8_narrow_kernel<BN, KS, GROUPED>;
  BNN_TRY(bnn::ensure_smem(kern, Cfg<BN>::kSmem));
  const cudaError_t e =
      bnn::launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), Cfg<BN>::kSmem, a.stream, KS, tw, tx,
                      a.xs, a.ws, a.bias, a.offsets, a.groups, a.rows, a.n, a.kb, a.out, a.out_type, errors);
  if (e != cudaSuccess) return bnn::cuda_fail(e);
  return bnn::check_launch();
}

template <int BN>
bnn_status narrow(const Args& a) {
  if (a.offsets) return launch_narrow<BN, 1, true>(a);
  const int64_t tiles = (a.n + kTm - 1) / kTm * ((a.rows + BN - 1) / BN), slots = 2 * bnn::sm_count();
  if (tiles * 8 <= slots && a.kb >= 16) return launch_narrow<BN, 8, false>(a);
  if (tiles * 4 <= slots && a.kb >= 8) return launch_narrow<BN, 4, false>(a);
  if (tiles * 2 <= slots && a.kb >= 4) return launch_narrow<BN, 2, false>(a);
  return launch_narrow<BN, 1, false>(a);
}

// The tile kernel's shape for `rows` rows in `groups` groups: least modelled
// time, waves x (blocks of k x us a block + us a store), of the shapes that a
// sweep over 64 .. 8192 rows x 4096 .. 11008 x 4096 (and 8192^3) left; the model
// is within about 10% of what it chooses between.  Groups: 128-row tiles (a
// pair's 256 rows end inside groups of a few hundred: 522 us against 416 at 64
// groups, 16384 rows x 4096 x 4096) unless the groups are long.
bnn_status gemm_tiles(const Args& a) {
  struct Shape {
    int ctas, tn;
    double block_us, store_us;
  };
  static constexpr Shape kDense[] = {{1, 32, 0.156, 0.5}, {1, 64, 0.18, 1.0}, {1, 128, 0.26, 2.2}, {2, 256, 0.51, 3.0}};
  static constexpr Shape kGrouped[] = {{1, 128, 0.26, 2.2}, {1, 256, 0.51, 3.0}, {2, 256, 0.51, 3.0}};
  const bool grouped = a.offsets != nullptr;
  const Shape* shapes = grouped ? kGrouped : kDense;
  const int count = grouped ? 3 : 4;
  const int64_t sms = bnn::sm_count(), busy = a.rows < a.groups ? a.rows : a.groups;
  const Shape* best = shapes;
  double best_us = 0.0;
  for (int i = 0; i < count; ++i) {
    const Shape& s = shapes[i];
    const int64_t high = 128 * s.ctas, wide = (a.n + s.tn - 1) / s.tn, slots = sms / s.ctas;
    // groups end inside a tile, in the mean half a tile each
    const int64_t rtiles = grouped ? (a.rows + busy * high / 2) / high + 1 : (a.rows + high - 1) / high;
    const int64_t waves = (rtiles * wide + slots - 1) / slots;
    const double us = static_cast<double>(waves) * (a.kb * s.block_us + s.store_us);
    if (i == 0 || us < best_us) {
      best_us = us;
      best = &s;
    }
  }
  return bnn::fp8::gemm_tile(a, best->ctas, best->tn);
}

// Few rows (in the mean of the groups: their sizes are on the device): the
// kernels that stream the weights.  Up to 8 rows and 2^26 bytes of weights the
// register kernel (1 row, in us, against the tensor-memory one: 1024 x 1000 2.0
// and 3.5, 4096 x 4096 5.6 and 6.5, 11008 x 4096 11.5 and 12.2, but 28672 x 8192
// 54.7 and 41.4).  Above 32 rows the tile kernel (64 x 11008 x 4096: 14.3 us
// against 16.7 with the weights on the lanes; but 32 x 4096 x 4096: 9.3 against
// 7.7).
bnn_status dispatch(const Args& a) {
  if (a.kb == 0) return gemm_empty(a);
  const int64_t per = (a.rows + a.groups - 1) / a.groups;
  if (!a.offsets && a.rows <= 8 && a.n * a.kb < (int64_t{1} << 19)) return bnn::fp8::gemm_skinny(a);
  if (per <= 16) return narrow<16>(a);
  if (per <= 32) return narrow<32>(a);
  return gemm_tiles(a);
}

}  // namespace

extern "C" bnn_status bnn_fp8_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                   const float* bias, int64_t m, int64_t n, int64_t k, void* out, int out_type,
                                   cudaStream_t s) {
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > INT32_MAX || k > BNN_MAX_K_FP8 || out_type < BNN_TYPE_F32 ||
      out_type > BNN_TYPE_F16)
    return BNN_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return BNN_OK;
  if (!out || (k > 0 && (!xq || !xs || !wq || !ws))) return BNN_ERR_INVALID_ARG;
  if (!bnn::aligned(xq, 16) || !bnn::aligned(wq, 16) || !bnn::aligned(xs, 4) || !bnn::aligned(ws, 4) ||
      !bnn::aligned(bias, 4) || !bnn::aligned(out, bnn::fp8::type_size(out_type)))
    return BNN_ERR_MISALIGNED;
  return dispatch(Args{xq, xs, wq, ws, bias, nullptr, 1, m, n, static_cast<int>((k + 127) / 128), out, out_type, s});
}

extern "C" bnn_status bnn_fp8_grouped_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                           const int64_t* offsets, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                           void* out, int out_type, cudaStream_t s) {
  if (groups < 0 || groups > BNN_MAX_GROUPS || rows < 0 || n < 0 || k < 0 || rows > INT32_MAX || n > INT32_MAX ||
      groups * n > INT32_MAX || k > BNN_MAX_K_FP8 || out_type < BNN_TYPE_F32 || out_type > BNN_TYPE_F16)
    return BNN_ERR_INVALID_ARG;
  if (groups == 0 || rows == 0 || n == 0) return BNN_OK;
  if (!out || !offsets || (k > 0 && (!xq || !xs || !wq || !ws))) return BNN_ERR_INVALID_ARG;
  if (!bnn::aligned(xq, 16) || !bnn::aligned(wq, 16) || !bnn::aligned(xs, 4) || !bnn::aligned(ws, 4) ||
      !bnn::aligned(offsets, 8) || !bnn::aligned(out, bnn::fp8::type_size(out_type)))
    return BNN_ERR_MISALIGNED;
  return dispatch(Args{xq, xs, wq, ws, nullptr, offsets, static_cast<int>(groups), rows, n,
                       static_cast<int>((k + 127) / 128), out, out_type, s});
}
