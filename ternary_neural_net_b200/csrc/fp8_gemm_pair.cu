// The e4m3 matmul for many rows: persistent CTA pairs on 256 x 256 tiles.
//
// Activation rows lie on the tensor-memory lanes (operand A, 128 rows per CTA
// of the pair), 256 weight rows are the MMA's N (128 in each CTA's shared
// memory).  So in the epilogue a thread holds one activation row and 128
// columns of one weight scale block: the scale of a block of k is one number
// per thread, and the block's sums cost one packed multiply-add per two
// columns.  (With the weights on the lanes, as for few rows, every column has
// a scale of its own: a shared-memory load per four columns, and shared memory
// is what the operands already fill.)  cta_group::2 halves each SM's copies
// and reads of the weight tile.
//
// A block of k (128 bytes a row) is one ring stage and four MMAs of K = 32 into
// one of two 256-column accumulators, started afresh; while the epilogue reads
// one, scales it and adds it to its 128 float32 registers a thread, the tensor
// cores fill the other.  At the dense rate a block takes 512 clocks; the
// epilogue's multiply-adds take 256 of each SM sub-partition's.
//
// Roles per CTA: warps 0-7 epilogue (lane quarter w % 4, column half w / 4),
// warp 8 TMA, warp 9 MMA (CTA 0's issues for the pair).  Both CTAs' copies
// complete on CTA 0's barrier.  Every wait is bounded; one that runs out stops
// the CTA's roles and leaves the outputs unspecified.
#include <cooperative_groups.h>

#include <mutex>

#include "fp8_common.cuh"

namespace {

using bnn::fp8::Args;
using bnn::tc::mbar_expect_tx;
using bnn::tc::smem_u32;
using bnn::tc::sw128_desc;
using bnn::tc::tmem_ld16;
using bnn::tc::tmem_wait_ld;

constexpr int kTm = 128;                       // rows of each operand per CTA
constexpr int kTile = 2 * kTm;                 // tile: 256 x 256 per pair
constexpr int kBlockBytes = 128;               // bytes of a row's block of k
constexpr uint32_t kOperand = kTm * kBlockBytes;
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kBufs = 2;                       // 256-column accumulators
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 8, kTmaWarp = kEpiWarps, kMmaWarp = kTmaWarp + 1;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kCols = 128;                     // columns of an epilogue thread
constexpr int kAhead = 4;                      // blocks whose scales are in flight
constexpr size_t kSmem = kStages * kStageBytes + 1024;

// One box into this CTA's shared memory, its bytes completing on CTA 0's mbarrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* map, int x, int y, uint32_t bar0) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar0)
      : "memory");
}

// Arrives on the mbarrier in both CTAs once the MMAs issued before have completed.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;\n" : "+l"(acc) : "l"(a), "l"(s));
}

template <bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                const float* __restrict__ xs, const float* __restrict__ ws, const float* __restrict__ bias,
                const int64_t* __restrict__ offsets, int groups, int64_t rows, int64_t n, int kb,
                void* __restrict__ out, int out_type, int wide, unsigned int* errors) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];   // CTA 0's: both CTAs' copies
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t part_full[kBufs];
  __shared__ __align__(8) uint64_t part_empty[kBufs];   // CTA 0's: one arrival per epilogue warp of both CTAs
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int abort_flag;
  __shared__ bnn::fp8::Groups<GROUPED ? BNN_MAX_GROUPS : 1> map;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster.block_rank();
  const uint32_t ring = smem_u32(smem);
  const int wtiles = static_cast<int>((n + kTile - 1) / kTile);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bnn::tc::mbar_init(smem_u32(&full_bar[i]), 1);
      bnn::tc::mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      bnn::tc::mbar_init(smem_u32(&part_full[i]), 1);
      bnn::tc::mbar_init(smem_u32(&part_empty[i]), 2 * kEpiWarps);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid == kTmaWarp * 32) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
  }
  if (warp == kMmaWarp) {  // the same warp of both CTAs allocates the pair's tensor memory
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_holder)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::);
  }
  bnn::pdl_wait();  // activations and offsets may come from the preceding kernel
  if (GROUPED) {
    if (warp == 0) bnn::fp8::build_groups<kTile>(map, offsets, groups, rows, lane);
  } else if (tid == 0) {
    map.start[0] = 0;
    map.start[1] = static_cast<int>(rows);
    map.first[0] = 0;
    map.first[1] = static_cast<int>((rows + kTile - 1) / kTile);
  }
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  cluster.sync();  // both CTAs' barriers exist before any copy or arrival
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
  const uint32_t tmem = tmem_holder;
  bnn::pdl_trigger();
  const int64_t tiles = static_cast<int64_t>(map.first[groups]) * wtiles;
  const int64_t step = gridDim.x >> 1, tile0 = blockIdx.x >> 1;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA copies
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t tile = tile0; tile < tiles && ok; tile += step) {
        const bnn::fp8::Tile t = bnn::fp8::tile_at<kTile>(tile, groups, map.start, map.first, wtiles);
        const int xrow = t.row + kTm * static_cast<int>(rank);
        const int wrow = t.group * static_cast<int>(n) + t.wtile * kTile + kTm * static_cast<int>(rank);
        for (int b = 0; b < kb; ++b, ++it) {
          const int st = static_cast<int>(it % kStages);
          if (it >= static_cast<uint32_t>(kStages) &&
              !bnn::tc::mbar_wait(smem_u32(&empty_bar[st]), (it / kStages + 1) & 1u, &abort_flag, errors)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + st * kStageBytes;
          uint32_t bar0;
          asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(bar0) : "r"(smem_u32(&full_bar[st])));
          if (rank == 0) mbar_expect_tx(smem_u32(&full_bar[st]), 2 * kStageBytes);
          tma_load_pair(dst, &tmap_x, b * kBlockBytes, xrow, bar0);
          tma_load_pair(dst + kOperand, &tmap_w, b * kBlockBytes, wrow, bar0);
        }
      }
      // the pair must not retire with copies in flight (CTA 0's barriers see both CTAs' copies)
      if (rank == 0)
        for (uint32_t c = it >= static_cast<uint32_t>(kStages) ? it - kStages : 0; c < it; ++c)
          bnn::tc::mbar_drain(smem_u32(&full_bar[c % kStages]), (c / kStages) & 1u, errors);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue (CTA 0)
    if (rank == 0 && lane == 0) {
      constexpr uint32_t word = bnn::fp8::mma_word(kTile, kTile);
      uint32_t it = 0;
      bool ok = true;
      for (int64_t tile = tile0; tile < tiles && ok; tile += step) {
        for (int b = 0; b < kb; ++b, ++it) {
          const int st = static_cast<int>(it % kStages), pb = static_cast<int>(it % kBufs);
          ok = (it < static_cast<uint32_t>(kBufs) ||
                bnn::tc::mbar_wait_cluster(smem_u32(&part_empty[pb]), (it / kBufs + 1) & 1u, &abort_flag, errors)) &&
               bnn::tc::mbar_wait_cluster(smem_u32(&full_bar[st]), (it / kStages) & 1u, &abort_flag, errors);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
          const uint64_t ad = sw128_desc(ring + st * kStageBytes);
          const uint64_t bd = sw128_desc(ring + st * kStageBytes + kOperand);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            asm volatile(
                "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem + pb * kTile),
                "l"(ad + static_cast<uint64_t>(2 * kk)), "l"(bd + static_cast<uint64_t>(2 * kk)), "r"(word),
                "r"(kk > 0 ? 1u : 0u));
          commit_both(smem_u32(&empty_bar[st]));
          commit_both(smem_u32(&part_full[pb]));
        }
      }
      // every MMA issued has completed before the pair's memory is given back
      for (uint32_t c = it >= static_cast<uint32_t>(kStages) ? it - kStages : 0; c < it; ++c)
        bnn::tc::mbar_drain(smem_u32(&empty_bar[c % kStages]), (c / kStages) & 1u, errors);
    }
  } else {
    // ------------------------------------------------------------ scale and add
    const int q = warp & 3, half = warp >> 2;
    const uint32_t lanes = (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(half * kCols);
    const int64_t nb = (n + 127) / 128;
    uint32_t it = 0;
    bool ok = true;
    for (int64_t tile = tile0; tile < tiles; tile += step) {
      const bnn::fp8::Tile t = bnn::fp8::tile_at<kTile>(tile, groups, map.start, map.first, wtiles);
      const int64_t row = t.row + kTm * static_cast<int>(rank) + 32 * q + lane;
      const int64_t j0 = static_cast<int64_t>(t.wtile) * kTile + half * kCols;
      const bool rlive = row < t.end, clive = j0 < n;
      const float* wsp = ws + (t.group * nb + j0 / 128) * kb;
      const float* xsp = xs + row;
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) acc[c] = 0;
      float pre[kAhead];
      auto load = [&](int b) -> float {
        return b < kb && rlive && clive ? __ldg(xsp + b * rows) * __ldg(wsp + b) : 0.0f;
      };
#pragma unroll
      for (int a = 0; a < kAhead; ++a) pre[a] = load(a);
      for (int b = 0; b < kb && ok; b += kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (b + a < kb && ok) {
            const uint64_t s = pack2(pre[a], pre[a]);
            pre[a] = load(b + a + kAhead);
            const int pb = static_cast<int>(it % kBufs);
            ok = bnn::tc::mbar_wait(smem_u32(&part_full[pb]), (it / kBufs) & 1u, &abort_flag, errors);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
              const uint32_t src = tmem + lanes + pb * kTile;
              uint32_t r[2][16];
              tmem_ld16(src, r[0]);
#pragma unroll
              for (int c0 = 0; c0 < kCols; c0 += 16) {
                const int u = (c0 / 16) & 1;
                tmem_wait_ld();
                if (c0 + 16 < kCols) tmem_ld16(src + c0 + 16, r[u ^ 1]);
#pragma unroll
                for (int c = 0; c < 16; c += 2)
                  fma2(acc[(c0 + c) / 2], pack2(__uint_as_float(r[u][c]), __uint_as_float(r[u][c + 1])), s);
              }
              asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
              __syncwarp();
              if (lane == 0) bnn::tc::mbar_arrive_rank(smem_u32(&part_empty[pb]), 0u);
            }
            ++it;
          }
        }
      }
      if (!ok) break;
      if (rlive && clive) {
        const int64_t at = row * n + j0;
        const bool whole = wide && j0 + kCols <= n;
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; i += 2) unpack2(acc[(c + i) / 2], y[i], y[i + 1]);
          if (bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += j0 + c + i < n ? __ldg(bias + j0 + c + i) : 0.0f;
          }
          if (whole) {
            if (out_type == BNN_TYPE_F32) {
              float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at + c);
              p[0] = make_float4(y[0], y[1], y[2], y[3]);
              p[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (out_type == BNN_TYPE_BF16) {
                  const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                  v[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                  const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
                  v[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
              }
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at + c) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (j0 + c + i < n) bnn::fp8::store_one(out, out_type, at + c + i, y[i]);
          }
        }
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  cluster.sync();  // neither CTA leaves while the pair's tensor memory or barriers are in use
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols));
}

template <bool GROUPED>
bnn_status launch_pair(const Args& a) {
  const int64_t wtiles = (a.n + kTile - 1) / kTile;
  const int64_t rtiles =
      GROUPED ? a.rows / kTile + (a.rows < a.groups ? a.rows : a.groups) : (a.rows + kTile - 1) / kTile;
  const int64_t tiles = rtiles * wtiles, slots = bnn::sm_count() / 2;
  const int64_t pairs = tiles < slots ? tiles : slots;
  if ((tiles + slots - 1) / slots * a.kb >= (int64_t{1} << 31)) return BNN_ERR_INVALID_ARG;  // stages count in 32 bits
  CUtensorMap tw, tx;
  const uint64_t pitch = static_cast<uint64_t>(a.kb) * kBlockBytes;
  if (!bnn::encode_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq, pitch, static_cast<uint64_t>(a.groups * a.n),
                           pitch, kBlockBytes, kTm, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bnn::encode_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xq, pitch, static_cast<uint64_t>(a.rows), pitch,
                           kBlockBytes, kTm, CU_TENSOR_MAP_SWIZZLE_128B))
    return BNN_ERR_UNSUPPORTED;
  unsigned int* errors = bnn::device_error_counter();
  if (!errors) return bnn::cuda_fail(cudaGetLastError());
  // 16-byte stores need every row's start aligned
  const int wide = bnn::aligned(a.out, 16) && a.n * static_cast<int64_t>(bnn::fp8::type_size(a.out_type)) % 16 == 0;
  auto kern = fp8_pair_kernel<GROUPED>;
  BNN_TRY(bnn::ensure_smem(kern, kSmem));
  const cudaError_t e =
      bnn::launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), kSmem, a.stream, 2u, tw, tx, a.xs,
                      a.ws, a.bias, a.offsets, a.groups, a.rows, a.n, a.kb, a.out, a.out_type, wide, errors);
  if (e != cudaSuccess) return bnn::cuda_fail(e);
  return bnn::check_launch();
}

}  // namespace

namespace bnn {
namespace fp8 {

bnn_status gemm_pair(const Args& a) { return a.offsets ? launch_pair<true>(a) : launch_pair<false>(a); }

}  // namespace fp8
}  // namespace bnn
