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

bnn_status gemm_narrow(const Args& a);
bnn_status gemm_pair(const Args& a);

// Instruction word of tcgen05.mma kind::f8f6f4: float32 accumulator, both
// operands e4m3 and K-major, an m x n tile.
constexpr uint32_t mma_word(uint32_t m, uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24); }

// The rows' tiles.  Group g's rows are cut into tiles of TM rows; `start` and
// `first` hold each group's first row and first row tile (the last entries:
// the end of the rows and the number of row tiles).
template <int G>
struct Groups {
  int start[G + 1];
  int first[G + 1];
};

// Fills `t` from the offsets (one warp), clamped to [0, rows] and to the
// largest before them.
template <int TM, int G>
__device__ __forceinline__ void build_groups(Groups<G>& t, const int64_t* offsets, int groups, int64_t rows,
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
// one time share both their rows and their weights in L2.
struct Tile {
  int group, row, end, wtile;  // first row, end of the group's rows, weight tile
};
constexpr int kBand = 8;

template <int TM>
__device__ __forceinline__ Tile tile_at(int64_t tile, int groups, const int* start, const int* first, int wtiles) {
  const int slot = static_cast<int>(tile / wtiles);
  int lo = 0, hi = groups;  // first[lo] <= slot < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= slot) lo = mid; else hi = mid;
  }
  const int mt = first[lo + 1] - first[lo];
  const int64_t local = tile - static_cast<int64_t>(first[lo]) * wtiles;
  const int band = static_cast<int>(local / (static_cast<int64_t>(kBand) * wtiles));
  const int r = static_cast<int>(local - static_cast<int64_t>(band) * kBand * wtiles);
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

inline size_t type_size(int type) { return type == BNN_TYPE_F32 ? 4 : 2; }

}  // namespace fp8
}  // namespace bnn
