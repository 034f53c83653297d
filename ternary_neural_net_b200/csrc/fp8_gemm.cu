// bnn_fp8_gemm / bnn_fp8_grouped_gemm: matrix products of e4m3 operands with a
// float32 scale for each block of 128 (include/bnn.h has the format).
//
//   y[i,j] = sum_b xs[b,i] ws[j/128,b] sum_{e in block b} xq[i,e] wq[j,e] (+ bias[j])
//
// Three kernels: up to 8 rows from registers with mma.sync (fp8_gemm_skinny.cu),
// up to 32 rows with the weights on the tensor-memory lanes (this file), more in
// tiles (fp8_gemm_tile.cu).  The last two run the inner sums on tcgen05.mma
// kind::f8f6f4 (K = 32, four per block of 128).  All start a fresh accumulator
// for every block of k; the block's sum is added, times its scales, to float32
// accumulators in registers.  The scales are arbitrary float32 numbers, so the
// tensor cores' own block scaling (powers of two) cannot apply them.
#include <cooperative_groups.h>

#include "fp8_common.cuh"

namespace {

using bnn::fp8::Args;
using bnn::tc::smem_u32;
using bnn::tc::sw128_desc;
using bnn::tc::tmem_ld16;
using bnn::tc::tmem_wait_ld;

// ---------------------------------------------------------------------------
// Up to 32 rows (of a group): weights on the tensor-memory lanes.
//
// Tile: 128 weight rows (one scale block: the weight scale of a block of k is
// one number for the CTA) x BN activation rows as the MMA's N, so a handful of
// rows costs a handful of columns and the weights stream once at whatever rate
// HBM gives.  A ring stage holds U blocks of k (one 3-D TMA box per operand);
// each block has an accumulator of its own, two sets of U in tensor memory.
// When the tiles leave SMs idle, a cluster of KS CTAs splits the blocks of k and
// adds its partial sums in rank order through distributed shared memory: the
// order is fixed, so results are reproducible.  Two CTAs share an SM.
//
// Roles: four epilogue warps, each 32 weight rows (they read the accumulators,
// scale and add); a TMA warp; an MMA warp; a scale warp, which writes the
// products of the rows' scales and the weight block's to shared memory, ahead,
// from where every lane reads all BN.
//
// Launched with programmatic dependent launch: the weights' first stages are
// fetched before the wait for the kernel ahead (not for groups, whose tiles
// depend on the offsets).
//
// Bound by the weights' bytes: 16 x 28672 x 8192 in 39.8 us = 90% of the measured
// HBM copy (one row 38.5 us = 93%), 512 rows in 64 groups x 2048 x 4096 in 85 us
// = 97%; small weights by latency (32 x 4096 x 4096 in 7.4 us = 2.3 TB/s).  Two
// CTAs an SM leave a thread 128 registers, which 32 rows exceed: ptxas reports 68
// bytes of spill stores with a split of 4, 120 with 8 and 16 for groups; where
// they fall has not been looked into.
// ---------------------------------------------------------------------------
constexpr int kTm = 128;                    // weight rows of a tile
constexpr int kBlockBytes = 128;            // bytes of a row's block of k
constexpr int kEpi = 128;                   // epilogue threads
constexpr int kTmaWarp = kEpi / 32, kMmaWarp = kTmaWarp + 1, kScaleWarp = kTmaWarp + 2;
constexpr int kThreads = kEpi + 3 * 32;
constexpr int U = 2;                        // blocks of k per iteration
constexpr int kBufs = 2;                    // accumulator sets
constexpr int kScaleSlots = 2 * kBufs;      // iterations whose scales are in shared memory
constexpr int kScaleAhead = 2;              // iterations whose scales are in flight

template <int BN>
struct Cfg {
  static constexpr uint32_t kWBlock = kTm * kBlockBytes, kXBlock = BN * kBlockBytes;
  static constexpr uint32_t kStageBytes = U * (kWBlock + kXBlock);
  static constexpr int kStages = 110592 / kStageBytes;               // two CTAs an SM
  static constexpr uint32_t kTmemCols = kBufs * U * BN;              // 64 or 128
  static constexpr size_t kSmem = kStages * kStageBytes + 1024;
  static_assert(kXBlock % 1024 == 0, "swizzle atoms stay aligned");
  static_assert(kStages >= kBufs && BN * kEpi * 4 <= kStages * kStageBytes, "the split's exchange fits the ring");
};

template <int BN, int KS, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 2)
fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                  const float* __restrict__ xs, const float* __restrict__ ws, const float* __restrict__ bias,
                  const int64_t* __restrict__ offsets, int groups, int64_t rows, int64_t n, int kb,
                  void* __restrict__ out, int out_type, uint32_t polls, unsigned int* errors) {
  static_assert(KS == 1 || !GROUPED, "a split cluster takes one tile");
  namespace cg = cooperative_groups;
  using C = Cfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S], done_bar[S], scale_bar[kScaleSlots], free_bar[kBufs];
  __shared__ uint32_t tmem_holder;
  __shared__ int any_bad;
  __shared__ __align__(16) float scales[kScaleSlots][U][BN];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // (behind the ring, as long as this call's groups: two CTAs share an SM's memory)
  int* const group_map = reinterpret_cast<int*>(smem + S * C::kStageBytes);
  const bnn::fp8::Groups map{group_map, group_map + groups + 1};
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem);
  const int rank = KS > 1 ? static_cast<int>(blockIdx.x % KS) : 0;
  const int wtiles = static_cast<int>((n + kTm - 1) / kTm);
  const int its = (kb + U - 1) / U;
  const int i0 = static_cast<int>(static_cast<int64_t>(its) * rank / KS);
  const int i1 = static_cast<int>(static_cast<int64_t>(its) * (rank + 1) / KS);

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bnn::tc::mbar_init(smem_u32(&full_bar[i]), 1);
      bnn::tc::mbar_init(smem_u32(&done_bar[i]), 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) bnn::tc::mbar_init(smem_u32(&scale_bar[i]), 1);
    for (int i = 0; i < kBufs; ++i) bnn::tc::mbar_init(smem_u32(&free_bar[i]), kEpi / 32);
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
  const int tiles = map.first[groups] * wtiles;  // (the launch keeps it within 32 bits)
  const int step = gridDim.x / KS, tile0 = blockIdx.x / KS;
  const uint32_t full = smem_u32(full_bar), done = smem_u32(done_bar), ready = smem_u32(scale_bar),
                 freed = smem_u32(free_bar), leader = bnn::fp8::elected();

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA copies
    bnn::fp8::Ring<S> st;
    bool ok = true, waited = GROUPED;
    for (int tile = tile0; tile < tiles && ok; tile += step) {
      const bnn::fp8::Tile t = bnn::fp8::tile_at<BN>(tile, groups, map, wtiles);
      const int wrow = t.group * static_cast<int>(n) + t.wtile * kTm;
      int ahead = i0;  // the iteration up to which the weights are already on their way
      if (!waited) {
        ahead += min(S, i1 - i0);
        for (int i = i0; i < ahead; ++i) {
          bnn::fp8::expect_if(leader, full + 8 * (i - i0), C::kStageBytes);
          bnn::fp8::load_box<1>(leader, ring + (i - i0) * C::kStageBytes, &tmap_w, wrow, i * U, full + 8 * (i - i0));
        }
        bnn::pdl_wait();
        waited = true;
      }
      for (int i = i0; i < i1; ++i, st.next()) {
        // (the round before a barrier's first counts as done)
        ok = bnn::fp8::wait(done + 8 * st.at, st.round ^ 1u, polls, errors);
        if (!ok) break;
        const uint32_t dst = ring + st.at * C::kStageBytes, bar = full + 8 * st.at;
        if (i >= ahead) {
          bnn::fp8::expect_if(leader, bar, C::kStageBytes);
          bnn::fp8::load_box<1>(leader, dst, &tmap_w, wrow, i * U, bar);
        }
        bnn::fp8::load_box<1>(leader, dst + U * C::kWBlock, &tmap_x, t.row, i * U, bar);
      }
    }
    if (!waited) bnn::pdl_wait();
    bnn::fp8::drain(full, st, errors);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    if (!GROUPED) bnn::pdl_wait();  // before the first bounded wait (for copies that start after it)
    constexpr uint32_t word = bnn::fp8::mma_word(kTm, BN);
    const uint64_t desc = sw128_desc(ring);
    bnn::fp8::Ring<S> st;
    bnn::fp8::Ring<kBufs> acc;
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += step) {
      for (int i = i0; i < i1; ++i, st.next(), acc.next()) {
        ok = bnn::fp8::wait2(freed + 8 * acc.at, acc.round ^ 1u, full + 8 * st.at, st.round, polls, errors);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
        const uint64_t ad = desc + st.at * (C::kStageBytes >> 4), bd = ad + (U * C::kWBlock >> 4);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            bnn::fp8::issue_mma<1>(leader, tmem + acc.at * (U * BN) + u * BN, ad + (u * (C::kWBlock >> 4) + 2 * kk),
                                   bd + (u * (C::kXBlock >> 4) + 2 * kk), word, kk > 0 ? 1u : 0u);
        bnn::fp8::commit<1>(leader, done + 8 * st.at);
      }
    }
    bnn::fp8::drain(done, st, errors);
  } else if (warp == kScaleWarp) {
    // ------------------------------------------------------------ scales
    if (!GROUPED) bnn::pdl_wait();  // the activation scales may come from the preceding kernel
    bnn::fp8::Ring<kScaleSlots> sl;
    bnn::fp8::Ring<kBufs> old;
    bool ok = true;
    int lead = kBufs;
    for (int tile = tile0; tile < tiles && ok; tile += step) {
      const bnn::fp8::Tile t = bnn::fp8::tile_at<BN>(tile, groups, map, wtiles);
      const bool live = lane < BN && lane < t.end - t.row;
      const float* wsp = ws + (static_cast<int64_t>(t.group) * wtiles + t.wtile) * kb;
      const float* xsp = xs + t.row + lane;
      float x[kScaleAhead][U], w[kScaleAhead][U];
      auto load = [&](int i, int a) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int b = i * U + u;
          x[a][u] = b < kb && i < i1 && live ? __ldg(xsp + b * rows) : 0.0f;
          w[a][u] = b < kb && i < i1 ? __ldg(wsp + b) : 0.0f;
        }
      };
#pragma unroll
      for (int a = 0; a < kScaleAhead; ++a) load(i0 + a, a);
      for (int i = i0; i < i1 && ok; i += kScaleAhead) {
#pragma unroll
        for (int a = 0; a < kScaleAhead; ++a) {
          if (i + a < i1 && ok) {
            // Before an iteration's scales are written, those of kScaleSlots before must have been read: it waits
            // until the accumulators of kBufs before have been.  That barrier's next phase is this iteration's,
            // which needs these scales, so the phase cannot be missed.
            if (lead > 0) {
              --lead;
            } else {
              ok = bnn::fp8::wait(freed + 8 * old.at, old.round, polls, errors);
              old.next();
            }
            if (ok) {
#pragma unroll
              for (int u = 0; u < U; ++u)
                if (lane < BN) scales[sl.at][u][lane] = x[a][u] * w[a][u];
              load(i + a + kScaleAhead, a);
              __syncwarp();
              bnn::fp8::arrive_if(leader, ready + 8 * sl.at);
              sl.next();
            }
          }
        }
      }
    }
  }
  if (warp >= kEpi / 32) {
    if (KS > 1) {
      __syncwarp();
      cluster.sync();
      cluster.sync();
    }
  } else {
    // ------------------------------------------------------------ scale and add
    if (!GROUPED) bnn::pdl_wait();
    const uint32_t src0 = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    bnn::fp8::Ring<S> st;
    bnn::fp8::Ring<kScaleSlots> sl;
    uint32_t buf = 0;
    bool ok = true;
    for (int tile = tile0; tile < tiles; tile += step) {
      const bnn::fp8::Tile t = bnn::fp8::tile_at<BN>(tile, groups, map, wtiles);
      const int live = min(BN, t.end - t.row);
      float acc[BN];
#pragma unroll
      for (int c = 0; c < BN; ++c) acc[c] = 0.0f;
      for (int i = i0; i < i1; ++i, st.next(), sl.next(), buf ^= 1u) {
        ok = bnn::fp8::wait2(done + 8 * st.at, st.round, ready + 8 * sl.at, sl.round, polls, errors);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
        uint32_t r[U * BN / 16][16];
#pragma unroll
        for (int c = 0; c < U * BN / 16; ++c) tmem_ld16(src0 + buf * (U * BN) + 16 * c, r[c]);
        tmem_wait_ld();
        asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
        float4 s[U * BN / 4];
#pragma unroll
        for (int c = 0; c < U * BN / 4; ++c) s[c] = reinterpret_cast<const float4*>(&scales[sl.at][0][0])[c];
        bnn::fp8::arrive_if(leader, freed + 8 * buf);  // accumulators and scales are in this warp's registers
#pragma unroll
        for (int c = 0; c < U * BN; c += 4) {
          const float4 v = s[c / 4];
          float* a = acc + c % BN;
          a[0] = fmaf(__uint_as_float(r[c / 16][c % 16]), v.x, a[0]);
          a[1] = fmaf(__uint_as_float(r[c / 16][c % 16 + 1]), v.y, a[1]);
          a[2] = fmaf(__uint_as_float(r[c / 16][c % 16 + 2]), v.z, a[2]);
          a[3] = fmaf(__uint_as_float(r[c / 16][c % 16 + 3]), v.w, a[3]);
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
  if (ctas > INT32_MAX || tiles > INT32_MAX - slots) return BNN_ERR_INVALID_ARG;
  CUtensorMap tw, tx;
  const uint64_t kb = static_cast<uint64_t>(a.kb);
  if (!bnn::encode_tmap_blocks(&tw, a.wq, static_cast<uint64_t>(a.groups * a.n), kb, kTm, U) ||
      !bnn::encode_tmap_blocks(&tx, a.xq, static_cast<uint64_t>(a.rows), kb, BN, U))
    return BNN_ERR_UNSUPPORTED;
  unsigned int* errors = bnn::device_error_counter();
  if (!errors) return bnn::cuda_fail(cudaGetLastError());
  auto kern = fp8_narrow_kernel<BN, KS, GROUPED>;
  const size_t smem = Cfg<BN>::kSmem + 2 * sizeof(int) * (a.groups + 1);
  BNN_TRY(bnn::ensure_smem(kern, Cfg<BN>::kSmem + 2 * sizeof(int) * (BNN_MAX_GROUPS + 1)));
  const cudaError_t e =
      bnn::launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, a.stream, KS, tw, tx,
                      a.xs, a.ws, a.bias, a.offsets, a.groups, a.rows, a.n, a.kb, a.out, a.out_type,
                      bnn::fp8::main_polls(), errors);
  if (e != cudaSuccess) return bnn::cuda_fail(e);
  return bnn::check_launch();
}

template <int BN>
bnn_status narrow(const Args& a, int split) {
  if (a.offsets) return launch_narrow<BN, 1, true>(a);
  if (split == 8) return launch_narrow<BN, 8, false>(a);
  if (split == 4) return launch_narrow<BN, 4, false>(a);
  if (split == 2) return launch_narrow<BN, 2, false>(a);
  return launch_narrow<BN, 1, false>(a);
}

using bnn::fp8::Plan;

// The tile kernel's shape for `rows` rows in `groups` groups: least modelled
// time, waves x (blocks of k x us a block + us a store), of the shapes that a
// sweep over 64 .. 8192 rows x 4096 .. 11008 x 4096 (and 8192^3) left.  The model
// orders the shapes and does not tell times: it leaves out what a launch costs
// (some 4 us), the memory's rate and the power cap, and what is measured is 1-81%
// above it.  Of 15 sizes measured with every shape it took the fastest in 11, and
// one 2-9% slower in 4 (2048 x 4096 x 4096: the pair in 45 us, 128 x 128 in 41).
// Groups: 128-row tiles, 128 or 256 columns wide (x 4096 x 4096, in us: 8192 rows
// in 2 groups 150 and 149, 16384 in 64 410 and 396; but 8192 in 64 262 and 286,
// 2048 in 16 66 and 72, where the model takes the wider all the same).  A pair's
// 256 rows end inside the groups (423 us for 16384 rows in 64, and 100 against 84
// at 4096 rows in 8); in groups of 2048 rows they would save 2%, which is not
// worth a kernel.
Plan plan_tiles(int64_t rows, int64_t n, int kb, int64_t groups, bool grouped, int sms) {
  struct Shape {
    int ctas, tn;
    double block_us, store_us;
  };
  static constexpr Shape kDense[] = {{1, 32, 0.156, 0.4}, {1, 64, 0.19, 0.8}, {1, 128, 0.28, 1.2}, {2, 256, 0.51, 3.0}};
  static constexpr Shape kGrouped[] = {{1, 128, 0.28, 1.2}, {1, 256, 0.51, 3.0}};
  const Shape* shapes = grouped ? kGrouped : kDense;
  const int count = grouped ? 2 : 4;
  const int64_t busy = rows < groups ? rows : groups;
  const Shape* best = shapes;
  double best_us = 0.0;
  for (int i = 0; i < count; ++i) {
    const Shape& s = shapes[i];
    const int64_t high = 128 * s.ctas, wide = (n + s.tn - 1) / s.tn, slots = sms / s.ctas;
    // groups end inside a tile, in the mean half a tile each
    const int64_t rtiles = grouped ? (rows + busy * high / 2) / high + 1 : (rows + high - 1) / high;
    const int64_t waves = (rtiles * wide + slots - 1) / slots;
    const double us = static_cast<double>(waves) * (kb * s.block_us + s.store_us);
    if (i == 0 || us < best_us) {
      best_us = us;
      best = &s;
    }
  }
  return {bnn::fp8::kTiles, 128 * best->ctas, best->tn, 1};
}

bnn_status dispatch(const Args& a) {
  const Plan p = bnn::fp8::plan(a.rows, a.n, a.kb, a.groups, a.offsets != nullptr, bnn::sm_count());
  switch (p.kernel) {
    case bnn::fp8::kEmpty: return gemm_empty(a);
    case bnn::fp8::kRegisters: return bnn::fp8::gemm_skinny(a);
    case bnn::fp8::kLanes: return p.rows == 16 ? narrow<16>(a, p.split) : narrow<32>(a, p.split);
    default: return bnn::fp8::gemm_tile(a, p.rows / 128, p.cols);
  }
}

}  // namespace

namespace bnn {
namespace fp8 {

// Few rows (in the mean of the groups: their sizes are on the device): the
// kernels that stream the weights.  Up to 8 rows and 2^25 bytes of weights the
// register kernel (in us, against the tensor-memory one with 9 rows: 1024 x 1000
// 2.0 and 3.4, 4096 x 4096 5.6 and 5.9, but 11008 x 4096 11.5 and 11.5, and 28672
// x 8192 54.7 and 36.4).  Above 32 rows the tile kernel (64 x 11008 x 4096: 14
// us; but 32 x 4096 x 4096 9.3 against 7.4).  It does not split k, which a long k
// with few tiles pays for: 32 x 512 x 16384 takes 9-10 us, 33 rows 26, 64 x 1024 x
// 16384 27.  The mean is of the whole buffer's rows: 64 rows in 64 groups x 2048 x
// 4096 take 84 us, and 106 (128 x 128 tiles) in a buffer of 4096; 512 rows take 85
// evenly spread, and 24-27 in one group, in 32 tiles of 16 rows.
Plan plan(int64_t rows, int64_t n, int kb, int64_t groups, bool grouped, int sms) {
  if (kb == 0) return {kEmpty, 0, 0, 1};
  const int64_t per = (rows + groups - 1) / groups;
  if (!grouped && rows <= 8 && n * kb <= (int64_t{1} << 18)) return {kRegisters, 8, 16, 1};
  if (per > 32) return plan_tiles(rows, n, kb, groups, grouped, sms);
  const int bn = per <= 16 ? 16 : 32;
  int split = 1;
  if (!grouped) {
    const int64_t tiles = (n + kTm - 1) / kTm * ((rows + bn - 1) / bn), slots = 2 * sms;
    split = tiles * 8 <= slots && kb >= 16 ? 8 : tiles * 4 <= slots && kb >= 8 ? 4 : tiles * 2 <= slots && kb >= 4 ? 2 : 1;
  }
  return {kLanes, bn, kTm, split};
}

}  // namespace fp8
}  // namespace bnn

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
