// The e4m3 matmul for more than a few rows: persistent CTAs, or CTA pairs, on
// tiles of 128 or 256 rows x TN columns.
//
// Activation rows lie on the tensor-memory lanes (operand A, 128 rows per CTA),
// TN weight rows are the MMA's N (a pair's halves in either CTA's shared
// memory).  So in the epilogue a thread holds one activation row and TN / 2
// columns of one weight scale block: the scale of a block of k is one number
// per thread, and the block's sums cost one packed multiply-add per two
// columns.  (With the weights on the lanes, as for few rows, every column has
// a scale of its own: a shared-memory load per four columns, and shared memory
// is what the operands already fill.)
//
// A ring stage holds U blocks of k (128 bytes a row each, one 3-D TMA box per
// operand); each block's four MMAs of K = 32 start an accumulator of their own,
// U x TN = 256 columns (128 at TN = 32), two such sets in tensor memory.  While
// the epilogue reads one set, scales it and adds it to its float32 registers,
// the tensor cores fill the other.  What an iteration of a role costs is mostly
// the latency of its hundred-odd dependent instructions (some 600 clocks
// measured for the MMA warp and the copies alone), so narrow tiles take several
// blocks per iteration (256 x 4096 x 4096 with TN = 64: 15.6 us with one, 10.8
// with four).
//
// What bounds it.  A set is 512 clocks of MMAs.  TN = 128 moves 64 KiB per
// iteration into the SM, 1024 clocks at the 64 bytes a clock that an SM reads
// from L2, and takes 950-1000; a pair's 256 x 256 moves 32 KiB, and its epilogue
// (128 columns a thread, two warps in each sub-partition: loads of tensor memory
// and multiply-adds that wait for them) takes about 930: neither the multiply-adds
// (256 clocks of them) nor the tensor cores are full, and which wait it is that
// adds up has not been measured.  8192^3 takes 0.57-0.58 ms = 1900 TFLOP/s with
// normally distributed values, under the power cap (1480-1790 MHz sampled of
// 1965); short bursts of uniform positive codes, which draw less, 0.48-0.51 ms.
// Tried in such bursts (0.48 ms): sixteen epilogue warps (0.55 ms), 32-column
// loads or the next iteration's loads ahead of this one's end (0.51-0.58 ms:
// registers spill), scalar multiply-adds (0.49 ms), 256 x 192 tiles (0.53-0.59 ms,
// the same with four loads in flight and with six: the epilogue takes some 2.9
// clocks a column and 220 a block whatever is in flight).
//
// Roles per CTA: warps 0-7 epilogue (lane quarter w % 4, column half w / 4),
// warp 8 TMA, warp 9 MMA (CTA 0's issues for a pair), warps 10 and 11 the
// scales: they multiply the rows' with the weight blocks' into shared memory,
// ahead.  A pair's copies complete on CTA 0's barriers.  Every wait is bounded;
// a role whose wait runs out stops (and with it, by their own bounds, those
// that wait for it), and the outputs are unspecified.  Whatever the waits came
// to, no CTA leaves before its copies and MMAs have completed.
#include <cooperative_groups.h>

#include "fp8_common.cuh"

namespace {

using bnn::fp8::Args;
using bnn::tc::smem_u32;
using bnn::tc::sw128_desc;
using bnn::tc::tmem_wait_ld;

constexpr int kTm = 128;                       // activation rows per CTA
constexpr int kBlockBytes = 128;               // bytes of a row's block of k
constexpr int kScaleWarps = 2, kScaleAhead = 4;  // warps, and blocks whose scales are in flight
constexpr int kScaleSlots = 4;                 // iterations whose scales are in shared memory
constexpr int kBufs = 2;                       // accumulator sets
constexpr int kEpiWarps = 8, kTmaWarp = kEpiWarps, kMmaWarp = kTmaWarp + 1, kScaleWarp = kTmaWarp + 2;
constexpr int kThreads = 32 * (kEpiWarps + 4);
constexpr int kStoreCols = 16;                 // columns per step of an unaligned store
constexpr int kStagePitch = 20;                // words per row of a warp's store staging (16-byte accesses without bank conflicts)
// Registers a thread: 168 at launch (three warps in each SM sub-partition's 16384), of
// which the control warpgroup keeps 72 and each epilogue warpgroup takes 216.
constexpr int kControlRegs = 72, kEpiRegs = 216;
static_assert(128 * kControlRegs + 256 * kEpiRegs <= kThreads * 168, "register shares within the launch's");

template <int CTAS, int TN>
struct Cfg {
  static constexpr int U = TN >= 64 ? 256 / TN : 4;                 // blocks of k per iteration
  static constexpr int kWRows = TN / CTAS;                          // weight rows in a CTA's shared memory
  static constexpr uint32_t kXBlock = kTm * kBlockBytes, kWBlock = kWRows * kBlockBytes;
  static constexpr uint32_t kXBytes = U * kXBlock, kStageBytes = kXBytes + U * kWBlock;
  static constexpr int kStages = 196608 / kStageBytes;              // 192 KiB of stages
  static constexpr uint32_t kTmemCols = kBufs * U * TN;             // 512
  static constexpr int kCols = TN / 2;                              // columns of an epilogue thread
  static constexpr int kHold = kCols > 64 ? 3 : 4;                  // 16-column loads in flight per thread
  static constexpr int kHalves = TN > 128 ? 2 : 1;                  // weight scale blocks of a tile
  static constexpr size_t kSmem = kStages * kStageBytes + 1024;
  static_assert(kWBlock % 1024 == 0, "swizzle atoms stay aligned");
  static_assert(kScaleAhead % U == 0 && kStages >= 2, "");
};

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

// Two outputs as words of the output type.
__device__ __forceinline__ void put2(uint32_t* w, float a, float b, float) {
  w[0] = __float_as_uint(a);
  w[1] = __float_as_uint(b);
}
__device__ __forceinline__ void put2(uint32_t* w, float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  w[0] = *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void put2(uint32_t* w, float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  w[0] = *reinterpret_cast<const uint32_t*>(&h);
}

// A warp's 32 rows (lane = row, CW columns each) to `out` (pitch n, 16-byte
// aligned rows), the first `live` of them, in pieces of up to 64 bytes a row.
template <int CW, typename T>
__device__ __forceinline__ void store_rows(const uint64_t (&acc)[CW / 2], float* stage, T* out, const float* bias,
                                           int64_t n, int live, int lane) {
  constexpr int kCols = CW * sizeof(T) < 64 ? CW : 64 / static_cast<int>(sizeof(T));  // columns of a piece
  constexpr int kWords = kCols * sizeof(T) / 4, kLanes = kWords / 4;                  // a lane stores 16 bytes
#pragma unroll
  for (int c = 0; c < CW; c += kCols) {
    constexpr int kQuad = 16 / sizeof(T);  // columns of 16 bytes
    __syncwarp();                          // the last piece has been read
#pragma unroll
    for (int i = 0; i < kCols; i += kQuad) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < kQuad; e += 2) {
        float a, b;
        unpack2(acc[(c + i + e) / 2], a, b);
        if (bias) {
          a += __ldg(bias + c + i + e);
          b += __ldg(bias + c + i + e + 1);
        }
        put2(w + e * sizeof(T) / 4, a, b, T{});
      }
      *reinterpret_cast<uint4*>(stage + lane * kStagePitch + i * sizeof(T) / 4) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; r += 32 / kLanes) {
      const int row = r + lane / kLanes, word = 4 * (lane % kLanes);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + row * kStagePitch + word);
      if (row < live) *reinterpret_cast<uint4*>(out + row * n + c + word * 4 / sizeof(T)) = v;
    }
  }
}

template <int CTAS, int TN, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1)
fp8_tile_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                const float* __restrict__ xs, const float* __restrict__ ws, const float* __restrict__ bias,
                const int64_t* __restrict__ offsets, int groups, int64_t rows, int64_t n, int kb,
                void* __restrict__ out, int out_type, int wide, uint32_t polls, unsigned int* errors) {
  namespace cg = cooperative_groups;
  using C = Cfg<CTAS, TN>;
  constexpr int S = C::kStages, U = C::U, CW = C::kCols, H = C::kHold, kRows = CTAS * kTm;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S];   // a pair: CTA 0's, for both CTAs' copies
  __shared__ __align__(8) uint64_t done_bar[S];   // the stage's MMAs: frees the stage, fills the accumulator
  __shared__ __align__(8) uint64_t scale_bar[kScaleSlots];  // the iteration's scales are in `scales`
  __shared__ __align__(8) uint64_t free_bar[kBufs];         // a pair: CTA 0's; one arrival per epilogue warp
  __shared__ float scales[kScaleSlots][U][C::kHalves][kTm];
  __shared__ __align__(16) float stage_out[kEpiWarps][32 * kStagePitch];
  __shared__ uint32_t tmem_holder;
  __shared__ uint32_t issued[2];            // a pair's CTA 0: how many stages' copies either CTA issued
  __shared__ uint32_t tail_at, tail_round;  // and the ring's position behind them; CTA 1: behind the MMAs issued
  __shared__ int group_map[2][GROUPED ? BNN_MAX_GROUPS + 1 : 2];
  const bnn::fp8::Groups map{group_map[0], group_map[1]};
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CTAS == 2 ? cg::this_cluster().block_rank() : 0;
  const uint32_t ring = smem_u32(smem);
  const int wtiles = static_cast<int>((n + TN - 1) / TN), its = (kb + U - 1) / U;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bnn::tc::mbar_init(smem_u32(&full_bar[i]), 1);
      bnn::tc::mbar_init(smem_u32(&done_bar[i]), 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) bnn::tc::mbar_init(smem_u32(&scale_bar[i]), kScaleWarps);
    for (int i = 0; i < kBufs; ++i) bnn::tc::mbar_init(smem_u32(&free_bar[i]), CTAS * kEpiWarps);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid == kTmaWarp * 32) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
  }
  if (warp == kMmaWarp) {  // (the same warp of both CTAs of a pair)
    if constexpr (CTAS == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_holder)),
                   "r"(C::kTmemCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::);
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_holder)),
                   "r"(C::kTmemCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
    }
  }
  if (GROUPED) {
    bnn::pdl_wait();  // the offsets may come from the preceding kernel
    if (warp == 0) bnn::fp8::build_groups<kRows>(map, offsets, groups, rows, lane);
  } else if (tid == 0) {
    map.start[0] = 0;
    map.start[1] = static_cast<int>(rows);
    map.first[0] = 0;
    map.first[1] = static_cast<int>((rows + kRows - 1) / kRows);
  }
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  if constexpr (CTAS == 2) cg::this_cluster().sync();  // both CTAs' barriers exist before any copy or arrival
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
  const uint32_t tmem = tmem_holder;
  bnn::pdl_trigger();
  const int tiles = map.first[groups] * wtiles;  // (the launch keeps it within 32 bits)
  const int step = gridDim.x / CTAS, tile0 = blockIdx.x / CTAS;

  if (warp >= kEpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kControlRegs));
    const uint32_t full = smem_u32(full_bar), done = smem_u32(done_bar), leader = bnn::fp8::elected();
    if (warp == kTmaWarp) {
      // ---------------------------------------------------------- TMA copies
      uint32_t full0 = full;  // a pair's: CTA 0's
      if constexpr (CTAS == 2) asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(full0) : "r"(full));
      bnn::fp8::Ring<S> st;
      uint32_t count = 0;  // stages whose copies this CTA issued
      bool ok = true, waited = GROUPED;
      for (int tile = tile0; tile < tiles && ok; tile += step) {
        const bnn::fp8::Tile t = bnn::fp8::tile_at<kRows>(tile, groups, map, wtiles);
        const int xrow = t.row + kTm * static_cast<int>(rank);
        const int wrow = t.group * static_cast<int>(n) + t.wtile * TN + C::kWRows * static_cast<int>(rank);
        int ahead = 0;  // stages whose weights are already on their way
        if (!waited) {
          ahead = min(S, its);
          for (int i = 0; i < ahead; ++i) {
            if (rank == 0) bnn::fp8::expect_if(leader, full + 8 * i, CTAS * C::kStageBytes);
            bnn::fp8::load_box<CTAS>(leader, ring + i * C::kStageBytes + C::kXBytes, &tmap_w, wrow, i * U, full0 + 8 * i);
          }
          bnn::pdl_wait();
          waited = true;
        }
        for (int b = 0; b < its; ++b, ++count, st.next()) {
          // (the round before a barrier's first counts as done)
          ok = bnn::fp8::wait(done + 8 * st.at, st.round ^ 1u, polls, errors);
          if (!ok) break;
          const uint32_t dst = ring + st.at * C::kStageBytes, bar = full0 + 8 * st.at;
          if (b >= ahead) {
            if (rank == 0) bnn::fp8::expect_if(leader, full + 8 * st.at, CTAS * C::kStageBytes);
            bnn::fp8::load_box<CTAS>(leader, dst + C::kXBytes, &tmap_w, wrow, b * U, bar);
          }
          bnn::fp8::load_box<CTAS>(leader, dst, &tmap_x, xrow, b * U, bar);
        }
      }
      if (!waited) bnn::pdl_wait();
      if constexpr (CTAS == 1) {
        bnn::fp8::drain(full, st, errors);
      } else if (leader) {  // CTA 0 waits for both CTAs' copies, below
        *cg::this_cluster().map_shared_rank(&issued[rank], 0) = count;
        if (rank == 0) tail_at = st.at, tail_round = st.round;
      }
    } else if (warp == kMmaWarp && rank == 0) {
      // ---------------------------------------------------------- MMA issue
      if (!GROUPED) bnn::pdl_wait();  // before the first bounded wait (for copies that start after it)
      constexpr uint32_t word = bnn::fp8::mma_word(kRows, TN);
      const uint32_t freed = smem_u32(free_bar);
      const uint64_t desc = sw128_desc(ring);
      bnn::fp8::Ring<S> st;
      bnn::fp8::Ring<kBufs> acc;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += step) {
        for (int b = 0; b < its; ++b, st.next(), acc.next()) {
          ok = bnn::fp8::wait2(freed + 8 * acc.at, acc.round ^ 1u, full + 8 * st.at, st.round, polls, errors);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
          const uint64_t ad = desc + st.at * (C::kStageBytes >> 4), bd = ad + (C::kXBytes >> 4);
          const uint32_t d = tmem + acc.at * (U * TN);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              bnn::fp8::issue_mma<CTAS>(leader, d + u * TN, ad + (u * (C::kXBlock >> 4) + 2 * kk),
                              bd + (u * (C::kWBlock >> 4) + 2 * kk), word, kk > 0 ? 1u : 0u);
          bnn::fp8::commit<CTAS>(leader, done + 8 * st.at);
        }
      }
      bnn::fp8::drain(done, st, errors);
      if constexpr (CTAS == 2) {
        if (leader) {
          *cg::this_cluster().map_shared_rank(&tail_at, 1) = st.at;
          *cg::this_cluster().map_shared_rank(&tail_round, 1) = st.round;
        }
      }
    } else if (warp >= kScaleWarp) {
      // ---------------------------------------------------------- scales
      // Per block of k: xs of 64 of this CTA's rows (two a lane) times ws of the tile's weight blocks.
      if (!GROUPED) bnn::pdl_wait();
      const uint32_t ready = smem_u32(scale_bar);
      const int r0 = 64 * (warp - kScaleWarp) + lane, nb = static_cast<int>((n + 127) / 128);
      // Before iteration i's scales are written, iteration i - kScaleSlots's must have been read.  A CTA on its own
      // waits until iteration i - kBufs has been read: the next phase of that barrier is iteration i's, which needs
      // these scales, so it cannot be missed.  In a pair, whose barrier for that is CTA 0's, it waits for the MMAs of
      // i - kBufs, which follow the reading of i - 2 kBufs; their barrier's next phase is S iterations on.
      static_assert(CTAS == 1 || S >= 2 * kBufs, "the next phase needs iteration i's scales");
      static_assert(kScaleSlots == 2 * kBufs, "");
      bnn::fp8::Ring<kScaleSlots> st;
      bnn::fp8::Ring<CTAS == 1 ? kBufs : S> old;
      const uint32_t read = CTAS == 1 ? smem_u32(free_bar) : done;
      bool ok = true;
      int lead = kBufs;
      for (int tile = tile0; tile < tiles && ok; tile += step) {
        const bnn::fp8::Tile t = bnn::fp8::tile_at<kRows>(tile, groups, map, wtiles);
        const int row = t.row + kTm * static_cast<int>(rank) + r0;
        const int live = t.end - row, wb = t.wtile * TN / 128;
        const bool two = C::kHalves == 2 && wb + 1 < nb;
        const float* wsp = ws + (static_cast<int64_t>(t.group) * nb + wb) * kb;
        const float* xsp = xs + row;
        float x[kScaleAhead][2], w[kScaleAhead][2];
        int next = 0;  // block the pointers stand at
        auto load = [&](int a) {
          const bool more = next < kb;
          x[a][0] = more && live > 0 ? __ldg(xsp) : 0.0f;
          x[a][1] = more && live > 32 ? __ldg(xsp + 32) : 0.0f;
          w[a][0] = more ? __ldg(wsp) : 0.0f;
          if (C::kHalves == 2) w[a][1] = more && two ? __ldg(wsp + kb) : 0.0f;
          xsp += rows;
          ++wsp;
          ++next;
        };
#pragma unroll
        for (int a = 0; a < kScaleAhead; ++a) load(a);
        for (int b = 0; b < its && ok; b += kScaleAhead / U) {
#pragma unroll
          for (int a = 0; a < kScaleAhead; a += U) {
            if (b + a / U < its && ok) {
              if (lead > 0) {
                --lead;
              } else {
                ok = bnn::fp8::wait(read + 8 * old.at, old.round, polls, errors);
                old.next();
              }
              if (ok) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                  for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                      scales[st.at][u][h][r0 + 32 * i] = x[a + u][i] * w[a + u][h];
                  load(a + u);
                }
                __syncwarp();
                bnn::fp8::arrive_if(leader, ready + 8 * st.at);
                st.next();
              }
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kEpiRegs));
    // ------------------------------------------------------------ scale and add
    if (!GROUPED) bnn::pdl_wait();
    const int q = warp & 3, part = warp >> 2;
    const uint32_t src0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(part * CW);
    const uint32_t done = smem_u32(done_bar), ready = smem_u32(scale_bar);
    uint32_t freed0 = smem_u32(free_bar);  // a pair's: CTA 0's
    if constexpr (CTAS == 2) asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(freed0) : "r"(smem_u32(free_bar)));
    const uint32_t leader = bnn::fp8::elected();
    auto release = [&](uint32_t buf) {  // this warp has the accumulators in registers (its loads are warp-wide)
      asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
      if constexpr (CTAS == 2)
        bnn::fp8::arrive_cluster_if(leader, freed0 + 8 * buf);
      else
        bnn::fp8::arrive_if(leader, freed0 + 8 * buf);
    };
    bnn::fp8::Ring<S> st;
    bnn::fp8::Ring<kScaleSlots> sl;
    uint32_t buf = 0;
    bool ok = true;
    for (int tile = tile0; tile < tiles; tile += step) {
      uint64_t acc[CW / 2];
#pragma unroll
      for (int c = 0; c < CW / 2; ++c) acc[c] = 0;
      for (int b = 0; b < its; ++b, st.next(), sl.next(), buf ^= 1u) {
        ok = bnn::fp8::wait2(done + 8 * st.at, st.round, ready + 8 * sl.at, sl.round, polls, errors);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
        const uint32_t src = src0 + buf * (U * TN);
        const float* sc = &scales[sl.at][0][C::kHalves == 2 ? part : 0][32 * q + lane];
        uint64_t s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = pack2(sc[u * C::kHalves * kTm], sc[u * C::kHalves * kTm]);
        // 16 columns a load, H loads in flight: a wait is for all of them, so each batch is followed by the loads
        // of the next, issued as its registers fall free.
        constexpr int kLoads = U * CW / 16;
        uint32_t r[H][16];
        auto fetch = [&](int c) { bnn::tc::tmem_ld16(src + c * 16 / CW * TN + c * 16 % CW, r[c % H]); };
#pragma unroll
        for (int c = 0; c < (H < kLoads ? H : kLoads); ++c) fetch(c);
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          if (c % H == 0) {
            tmem_wait_ld();
            if (c + H >= kLoads) release(buf);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            fma2(acc[(c * 16 % CW + j) / 2], pack2(__uint_as_float(r[c % H][j]), __uint_as_float(r[c % H][j + 1])),
                 s[c * 16 / CW]);
          if (c + H < kLoads) fetch(c + H);
        }
      }
      if (!ok) break;
      // ---------------------------------------------------------- store
      const bnn::fp8::Tile t = bnn::fp8::tile_at<kRows>(tile, groups, map, wtiles);
      const int64_t row0 = t.row + kTm * static_cast<int>(rank) + 32 * q;  // this warp's first row
      const int64_t j0 = static_cast<int64_t>(t.wtile) * TN + part * CW;
      const int live = static_cast<int>(min(int64_t{32}, t.end - row0));
      if (live <= 0 || j0 >= n) continue;
      float* const stage = stage_out[warp];
      const float* const bj = bias ? bias + j0 : nullptr;
      if (wide && j0 + CW <= n) {
        if constexpr (CW <= 64) {
          // Pieces of 64 bytes a row through shared memory, so that a store instruction covers whole sectors of a
          // few rows instead of 16 bytes of each of 32 (1024 x 11008 x 4096: 55.9 to 51.5 us).
          if (out_type == BNN_TYPE_F32)
            store_rows<CW, float>(acc, stage, static_cast<float*>(out) + row0 * n + j0, bj, n, live, lane);
          else if (out_type == BNN_TYPE_BF16)
            store_rows<CW, __nv_bfloat16>(acc, stage, static_cast<__nv_bfloat16*>(out) + row0 * n + j0, bj, n, live,
                                          lane);
          else
            store_rows<CW, __half>(acc, stage, static_cast<__half*>(out) + row0 * n + j0, bj, n, live, lane);
        } else {
          // (128 accumulators a thread leave that path's registers no room: it spills inside the loop above, 541 us
          // at 8192^3 against 481 with the rows stored directly.  16-byte units exchanged between the lanes of a quad
          // instead of shared memory spill less and take 590.)
          const int64_t at = (row0 + lane) * n + j0;
#pragma unroll
          for (int c = 0; c < CW; c += 8) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) unpack2(acc[(c + i) / 2], y[i], y[i + 1]);
            if (bias) {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] += __ldg(bj + c + i);
            }
            if (lane < live) bnn::fp8::store_eight(out, out_type, at + c, y);
          }
        }
      } else {
        // Rows whose starts are not aligned, or a tile that ends inside: 16 columns at a time through shared memory,
        // two rows' pieces an instruction.
#pragma unroll
        for (int c = 0; c < CW; c += kStoreCols) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kStoreCols; i += 2)
            unpack2(acc[(c + i) / 2], stage[lane * (kStoreCols + 1) + i], stage[lane * (kStoreCols + 1) + i + 1]);
          __syncwarp();
          const int64_t j = j0 + c + lane % kStoreCols;
          const float y0 = bias && j < n ? __ldg(bias + j) : 0.0f;
          if (j < n)
            for (int r = lane / kStoreCols; r < live; r += 32 / kStoreCols)
              bnn::fp8::store_one(out, out_type, (row0 + r) * n + j,
                                  stage[r * (kStoreCols + 1) + lane % kStoreCols] + y0);
        }
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  if constexpr (CTAS == 2) {
    cg::this_cluster().sync();  // the roles of both CTAs have ended
    // What is in flight is waited for where it completes: both CTAs' copies in CTA 0, and the commits' arrivals in
    // CTA 1 (CTA 0's MMA warp has seen its own).  A stage's barrier expects both CTAs' bytes.  Where a wait ran out,
    // one CTA may have issued up to S stages more than the other: CTA 0's account of those is set right first.
    bnn::fp8::Ring<S> st;
    st.at = tail_at, st.round = tail_round;
    if (warp == kTmaWarp && rank == 0) {
      const uint32_t full = smem_u32(full_bar), leader = bnn::fp8::elected();
      const int more = static_cast<int>(issued[1] - issued[0]);  // CTA 1's stages that CTA 0 did not come to
#pragma unroll 1
      for (int i = 0; i < S; ++i, st.next()) {
        const uint32_t bar = full + 8 * st.at;
        if (i < more) bnn::fp8::expect_if(leader, bar, C::kStageBytes);
        if (i >= S + more) bnn::fp8::complete_if(leader, bar, C::kStageBytes);
        bnn::fp8::wait(bar, i < more ? st.round : st.round ^ 1u, bnn::fp8::kPolls, errors);
      }
    }
    if (warp == kMmaWarp && rank == 1) bnn::fp8::drain(smem_u32(done_bar), st, errors);
    __syncwarp();
    cg::this_cluster().sync();  // neither CTA leaves while the pair's tensor memory or barriers are in use
    if (warp == kMmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::kTmemCols));
  } else {
    if (warp == kMmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::kTmemCols));
  }
}

template <int CTAS, int TN, bool GROUPED>
bnn_status launch(const Args& a) {
  using C = Cfg<CTAS, TN>;
  constexpr int kRows = CTAS * kTm;
  const int64_t wtiles = (a.n + TN - 1) / TN;
  // groups: at most one ragged tile each beside the full ones
  const int64_t rtiles =
      GROUPED ? a.rows / kRows + (a.rows < a.groups ? a.rows : a.groups) : (a.rows + kRows - 1) / kRows;
  const int64_t tiles = rtiles * wtiles, slots = bnn::sm_count() / CTAS;
  const int64_t units = tiles < slots ? tiles : slots;
  if (tiles > INT32_MAX - slots) return BNN_ERR_INVALID_ARG;
  CUtensorMap tw, tx;
  const uint64_t kb = static_cast<uint64_t>(a.kb);
  if (!bnn::encode_tmap_blocks(&tw, a.wq, static_cast<uint64_t>(a.groups * a.n), kb, C::kWRows, C::U) ||
      !bnn::encode_tmap_blocks(&tx, a.xq, static_cast<uint64_t>(a.rows), kb, kTm, C::U))
    return BNN_ERR_UNSUPPORTED;
  unsigned int* errors = bnn::device_error_counter();
  if (!errors) return bnn::cuda_fail(cudaGetLastError());
  // 16-byte stores need every row's start aligned
  const int wide = bnn::aligned(a.out, 16) && a.n * static_cast<int64_t>(bnn::fp8::type_size(a.out_type)) % 16 == 0;
  auto kern = fp8_tile_kernel<CTAS, TN, GROUPED>;
  BNN_TRY(bnn::ensure_smem(kern, C::kSmem));
  const cudaError_t e = bnn::launch_pdl(kern, dim3(static_cast<unsigned>(CTAS * units)), dim3(kThreads), C::kSmem,
                                        a.stream, CTAS, tw, tx, a.xs, a.ws, a.bias, a.offsets, a.groups, a.rows, a.n,
                                        a.kb, a.out, a.out_type, wide, bnn::fp8::main_polls(), errors);
  if (e != cudaSuccess) return bnn::cuda_fail(e);
  return bnn::check_launch();
}

}  // namespace

namespace bnn {
namespace fp8 {

bnn_status gemm_tile(const Args& a, int ctas, int tn) {
  if (a.offsets) return tn == 256 ? launch<1, 256, true>(a) : launch<1, 128, true>(a);
  if (ctas == 2) return launch<2, 256, false>(a);
  return tn == 128 ? launch<1, 128, false>(a) : tn == 64 ? launch<1, 64, false>(a) : launch<1, 32, false>(a);
}

}  // namespace fp8
}  // namespace bnn
