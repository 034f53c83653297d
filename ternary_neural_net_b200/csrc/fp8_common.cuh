// Shared by the e4m3 matmul kernels (not part of the ABI): the map from tiles
// to groups of rows, output stores and the tensor-core instruction words.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bnn_internal.cuh"
#include "tc_common.cuh"

namespace bnn {
namespace fp8 {

// Operands of one call; offsets == nullptr: one group of all rows.
struct Args {
  const uint8_t* xq;
  const float* xs;
  const uint8_t* wq;
  const float* ws;
  const float* bias;
  const int64_t* offsets;
  int groups;
  int64_t rows, n;
  int kb;
  void* out;
  int out_type;
  cudaStream_t stream;
};

// The kernel of a call: the product's rows and columns of a tile, and the CTAs
// that split k.  Host only; sms: the device's SM count.
enum Kernel { kEmpty, kRegisters, kLanes, kTiles };
struct Plan {
  Kernel kernel;
  int rows, cols, split;
};
Plan plan(int64_t rows, int64_t n, int kb, int64_t groups, bool grouped, int sms);

// Up to 8 rows, one group.
bnn_status gemm_skinny(const Args& a);
// Tiles of 128 rows (ctas = 1) x 32, 64 or 128 columns, or of 256 rows (a CTA
// pair) x 256; for groups of 128 rows x 128 or 256.
bnn_status gemm_tile(const Args& a, int ctas, int tn);

// Bounded wait of a whole converged warp for an mbarrier phase: up to `polls`
// polls, each with a vote, so that the branch is uniform.  (A wait on
// a completed phase takes some 70 clocks like this and about 130 as a loop that
// each lane leaves by itself; bnn::tc::mbar_wait, which bounds by the wall
// clock, takes longer still, and polls with a time hint wake hundreds of clocks
// late.  These kernels wait twice per block of k and role.)  Every thread has
// waited for the kernel ahead before its first call, so only copies and MMAs of
// this kernel are waited for: microseconds, against 30 ms for kPolls polls at the
// least.  The roles' waits take the launch's bound (kPolls, or less for a test:
// bnn_probe_wait_limit), the drains always kPolls.
// False, for the whole warp, when it ran out: counted in *errors by each thread.
constexpr uint32_t kPolls = 1u << 20;

// The bound of a launch's waits.
inline uint32_t main_polls() {
  const uint32_t limit = wait_limit();
  return limit && limit < kPolls ? limit : kPolls;
}

// One poll: try_wait, which suspends the warp for a while, or under a test's
// bound test_wait, which returns at once.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, uint32_t polls) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.eq.u32 q, %3, %4;\n"
      "@q mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "@!q mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(polls), "n"(kPolls)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t polls, unsigned int* errors) {
#pragma unroll 1
  for (uint32_t i = polls; i != 0; --i)
    if (__all_sync(0xffffffffu, poll(bar, parity, polls))) return true;
  atomicAdd(errors, 1u);
  return false;
}

// The same for two barriers at once: the polls' latencies overlap.
__device__ __forceinline__ bool wait2(uint32_t bar_a, uint32_t parity_a, uint32_t bar_b, uint32_t parity_b,
                                      uint32_t polls, unsigned int* errors) {
#pragma unroll 1
  for (uint32_t i = polls; i != 0; --i) {
    const bool a = poll(bar_a, parity_a, polls), b = poll(bar_b, parity_b, polls);
    if (__all_sync(0xffffffffu, a && b)) return true;
  }
  atomicAdd(errors, 1u);
  return false;
}

// Position in a ring of N slots and the parity of its current round.
template <int N>
struct Ring {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      round ^= 1u;
    }
  }
};

// Waits for the newest phase of every slot of a ring whose next position is `st`
// (a slot not used yet counts as done).  A CTA must not retire with copies or
// MMAs in flight, whatever its roles' waits came to: so the copies are waited for
// on their own barriers (MMAs that were never issued complete no others), and the
// MMAs on the barriers of their commits.
template <int N>
__device__ __forceinline__ void drain(uint32_t bars, Ring<N> st, unsigned int* errors) {
#pragma unroll 1
  for (int i = 0; i < N; ++i, st.next()) wait(bars + 8 * st.at, st.round ^ 1u, kPolls, errors);
}

// 1 in one thread of a converged warp, 0 in the others.  The copy and MMA warps
// run their loops as whole warps and predicate what one thread issues with it:
// a branch around each issue, or a loop that one lane runs by itself, takes
// longer, since these instructions take warp-uniform operands.
__device__ __forceinline__ uint32_t elected() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}

__device__ __forceinline__ void arrive_if(uint32_t leader, uint32_t bar) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %1, 0;\n@p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar),
               "r"(leader)
               : "memory");
}

__device__ __forceinline__ void expect_if(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(
          bar),
      "r"(bytes), "r"(leader)
      : "memory");
}

// `bytes` that no copy will bring count as landed.
__device__ __forceinline__ void complete_if(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n@p mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n}\n" ::
          "r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}

// Arrival on an mbarrier of the cluster (a shared::cluster address) without
// memory ordering: what it orders is tensor memory, which the tcgen05 fences
// around it and around the wait cover.  (With release at cluster scope it would
// first wait for every load in flight: the scales fetched ahead.)
__device__ __forceinline__ void arrive_cluster_if(uint32_t leader, uint32_t remote) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %1, 0;\n@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n}\n" ::
          "r"(remote),
      "r"(leader)
      : "memory");
}

// Instruction word of tcgen05.mma kind::f8f6f4: float32 accumulator, both
// operands e4m3 and K-major, an m x n tile.
constexpr uint32_t mma_word(uint32_t m, uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24); }

// Blocks [z, z + U) of rows [y, ..) into this CTA's shared memory (out-of-range
// ones read as zero), the bytes completing on an mbarrier of the cluster (a
// pair's CTA 0).
template <int CTAS>
__device__ __forceinline__ void load_box(uint32_t leader, uint32_t dst, const void* map, int y, int z, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
        "@p cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
        "@p cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar), "r"(leader)
        : "memory");
}

// The MMA of one K = 32 step; `add` = 0 starts the accumulator afresh.
template <int CTAS>
__device__ __forceinline__ void issue_mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                          uint32_t add) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"(add), "r"(leader));
  else
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"(add), "r"(leader));
}

// Arrives on the mbarrier (in both CTAs of a pair) once the MMAs issued before have completed.
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n"
        "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::
            "r"(bar),
        "h"(static_cast<uint16_t>(3)), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %1, 0;\n"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(leader)
        : "memory");
}

// The rows' tiles.  Group g's rows are cut into tiles of TM rows; `start` and
// `first` hold each group's first row and first row tile (the last entries:
// the end of the rows and the number of row tiles).
struct Groups {
  int* start;  // [groups + 1] each, in shared memory
  int* first;
};

// Fills `t` from the offsets (one warp), clamped to [0, rows] and to the
// largest before them.
template <int TM>
__device__ __forceinline__ void build_groups(const Groups& t, const int64_t* offsets, int groups, int64_t rows,
                                             int lane) {
  auto clamped = [&](int i) -> int {
    const int64_t o = i <= groups ? offsets[i] : 0;
    return static_cast<int>(o < 0 ? 0 : (o > rows ? rows : o));
  };
  int top = 0, tiles = 0;  // running maximum and tile count before this chunk
  for (int c = 0; c <= groups; c += 32) {
    const int i = c + lane;
    int o = max(top, clamped(i));
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, o, d);
      if (lane >= d) o = max(o, v);
    }
    // tiles of group i - 1, which ends at o
    int before = __shfl_up_sync(0xffffffffu, o, 1);
    if (lane == 0) before = top;
    int sum = i == 0 ? 0 : (o - before + TM - 1) / TM;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    sum += tiles;
    if (i <= groups) {
      t.start[i] = o;
      t.first[i] = sum;
    }
    top = __shfl_sync(0xffffffffu, o, 31);
    tiles = __shfl_sync(0xffffffffu, sum, 31);
  }
}

// Row tile and weight tile of tile index `tile`: the group's tiles run over up
// to kBand row tiles before the next weight tile, so that the tiles at work at
// one time share both their rows and their weights in L2 (8192^3: 250 MB read
// from DRAM with bands of 16, 355 MB with bands of 8; 2048 x 8192 x 8192 in 140.0
// and 141.7 us).
struct Tile {
  int group, row, end, wtile;  // first row, end of the group's rows, weight tile
};
constexpr int kBand = 16;

template <int TM>
__device__ __forceinline__ Tile tile_at(int tile, int groups, const Groups& map, int wtiles) {
  const int* const start = map.start;
  const int* const first = map.first;
  const int slot = tile / wtiles;
  int lo = 0, hi = groups;  // first[lo] <= slot < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= slot) lo = mid; else hi = mid;
  }
  const int mt = first[lo + 1] - first[lo];
  const int local = tile - first[lo] * wtiles, band = local / (kBand * wtiles);
  const int r = local - band * kBand * wtiles;
  const int height = min(kBand, mt - band * kBand);
  Tile t;
  t.group = lo;
  t.wtile = r / height;
  t.row = start[lo] + (band * kBand + r % height) * TM;
  t.end = start[lo + 1];
  return t;
}

__device__ __forceinline__ void store_one(void* out, int type, int64_t at, float y) {
  if (type == BNN_TYPE_F32)
    static_cast<float*>(out)[at] = y;
  else if (type == BNN_TYPE_BF16)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
  else
    static_cast<__half*>(out)[at] = __float2half_rn(y);
}

// Eight consecutive outputs at a 16-byte aligned place.
__device__ __forceinline__ void store_eight(void* out, int type, int64_t at, const float (&y)[8]) {
  if (type == BNN_TYPE_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
    return;
  }
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == BNN_TYPE_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(v[0], v[1], v[2], v[3]);
}

inline size_t type_size(int type) { return type == BNN_TYPE_F32 ? 4 : 2; }

}  // namespace fp8
}  // namespace bnn
