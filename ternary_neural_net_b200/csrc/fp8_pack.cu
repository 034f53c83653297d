// bnn_fp8_pack_rows / bnn_fp8_pack_weight: float rows and weights -> e4m3 bytes
// with a float32 scale for each block of 128 (include/bnn.h has the format).
//
// Per block, with a = max(max |x|, 2^-100): scale = fl32(a / 448), r =
// fl32(448 / a), q = e4m3(fl32(x r)).  448 is the largest e4m3 value, so the
// block's largest element lands on it and no other one saturates.  The floor
// 2^-100 keeps both quotients normal numbers, so a block of zeros needs no case
// of its own.  The maximum is taken over the absolute bit patterns as unsigned
// integers: they order like the values, with infinities and NaN above every
// number, so one comparison finds a block that holds either.  The product
// x * r is rounded to float32 before the rounding to e4m3; a division would
// cost about ten instructions an element and round as often.
//
// Both kernels are bound by HBM (2 or 4 bytes read and 1 written per element):
// every element is read once, kept in registers over the maximum, and written
// once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bnn_internal.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kTop = 448.0f;
constexpr uint32_t kInfBits = 0x7f800000u;

// E elements of a lane: 16 bytes' worth of the input type.
template <typename T>
struct Lane {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int kLanes = 128 / E;        // lanes of one block of 128
  static constexpr int kBlocks = 32 / kLanes;   // blocks of one row that a warp takes at once
};

__device__ __forceinline__ void to_f32(const float (&v)[4], float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = v[i];
}
__device__ __forceinline__ void to_f32(const __nv_bfloat16 (&v)[8], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(v[i]);
}
__device__ __forceinline__ void to_f32(const __half (&v)[8], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __half2float(v[i]);
}

// V-element vector loads of the lane's E elements starting at element e of a
// row of k elements (k % V == 0 and the row V-aligned); 0 past k.
template <typename T, int V>
__device__ __forceinline__ void load_lane(const T* row, int64_t e, int64_t k, T (&v)[Lane<T>::E]) {
  struct alignas(V * sizeof(T)) Vec {
    T x[V];
  };
#pragma unroll
  for (int i = 0; i < Lane<T>::E; i += V) {
    Vec t;
    if (e + i < k) {
      t = *reinterpret_cast<const Vec*>(row + e + i);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) t.x[j] = static_cast<T>(0.0f);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) v[i + j] = t.x[j];
  }
}

template <int E>
__device__ __forceinline__ uint32_t top_bits(const float (&f)[E]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
  return a;
}

struct Scale {
  float scale, factor;
  bool fine;
};

__device__ __forceinline__ Scale scale_of(uint32_t bits) {
  Scale s;
  s.fine = bits < kInfBits;
  const float a = s.fine ? fmaxf(__uint_as_float(bits), 0x1p-100f) : 1.0f;
  s.scale = s.fine ? __fdiv_rn(a, kTop) : __int_as_float(0x7fffffff);
  s.factor = __fdiv_rn(kTop, a);
  return s;
}

// Four floats times the factor as four e4m3 bytes, lowest address first.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float r) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(__fmul_rn(b, r)), "f"(__fmul_rn(a, r)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(__fmul_rn(d, r)), "f"(__fmul_rn(c, r)));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ void store_lane(uint8_t* dst, const float (&f)[4], const Scale& s) {
  *reinterpret_cast<uint32_t*>(dst) = s.fine ? e4m3x4(f[0], f[1], f[2], f[3], s.factor) : 0u;
}
__device__ __forceinline__ void store_lane(uint8_t* dst, const float (&f)[8], const Scale& s) {
  uint2 v = make_uint2(0u, 0u);
  if (s.fine) v = make_uint2(e4m3x4(f[0], f[1], f[2], f[3], s.factor), e4m3x4(f[4], f[5], f[6], f[7], s.factor));
  *reinterpret_cast<uint2*>(dst) = v;
}

// Rows.  A CTA takes 32 rows x kBlocks blocks, a warp four of the rows: the four
// rows' 16-byte loads are in flight together, and the CTA's scales (32 rows of a
// block) leave as one 128-byte line of the block-major scale matrix.
constexpr int kRowsPerWarp = 4;
constexpr int kTileRows = kWarps * kRowsPerWarp;

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
fp8_pack_rows_kernel(const T* __restrict__ x, int64_t x_rows, const int32_t* __restrict__ index, int64_t rows,
                     int64_t k, int64_t kb, int64_t col_tiles, uint8_t* __restrict__ q, float* __restrict__ scale) {
  using L = Lane<T>;
  __shared__ float sc[L::kBlocks][kTileRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile_row = (blockIdx.x / col_tiles) * kTileRows;
  const int64_t b = (blockIdx.x % col_tiles) * L::kBlocks + lane / L::kLanes;  // this lane's block
  const int64_t e = b * 128 + (lane % L::kLanes) * L::E;
  bnn::pdl_trigger();  // a matmul launched after this kernel may start on its weights now
  T v[kRowsPerWarp][L::E];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = tile_row + warp * kRowsPerWarp + i;
    int64_t src = row;
    if (index) src = row < rows ? static_cast<int64_t>(__ldg(index + row)) : -1;
    const bool live = row < rows && src >= 0 && src < x_rows;
    load_lane<T, V>(x + (live ? src : 0) * k, live ? e : k, k, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int r = warp * kRowsPerWarp + i;
    float f[L::E];
    to_f32(v[i], f);
    uint32_t a = top_bits(f);
#pragma unroll
    for (int off = L::kLanes / 2; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
    const Scale s = scale_of(a);
    if (tile_row + r < rows && b < kb) store_lane(q + (tile_row + r) * kb * 128 + e, f, s);
    if (lane % L::kLanes == 0) sc[lane / L::kLanes][r] = s.scale;
  }
  __syncthreads();
  if (warp < L::kBlocks) {
    const int64_t sb = (blockIdx.x % col_tiles) * L::kBlocks + warp;
    if (sb < kb && tile_row + lane < rows) scale[sb * rows + tile_row + lane] = sc[warp][lane];
  }
}

// Weights.  A CTA takes one 128 x 128 block whole in registers (16 bytes a lane
// and load, 8 or 16 loads), a warp 16 of its rows.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
fp8_pack_weight_kernel(const T* __restrict__ w, int64_t n, int64_t k, int64_t kb, int64_t nb, uint8_t* __restrict__ q,
                       float* __restrict__ scale) {
  using L = Lane<T>;
  constexpr int kRows = 128 / kWarps;          // rows of a warp
  constexpr int kLoads = kRows / L::kBlocks;   // a load covers kBlocks rows
  __shared__ uint32_t tops[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = blockIdx.x % kb, t = blockIdx.x / kb, j0 = (t % nb) * 128, g = t / nb;
  const int64_t e = b * 128 + (lane % L::kLanes) * L::E;
  const int64_t row0 = j0 + warp * kRows + lane / L::kLanes;
  const T* base = w + g * n * k;
  T v[kLoads][L::E];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t row = row0 + i * L::kBlocks;
    const bool live = row < n;
    load_lane<T, V>(base + (live ? row : 0) * k, live ? e : k, k, v[i]);
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    float f[L::E];
    to_f32(v[i], f);
    a = max(a, top_bits(f));
  }
  a = __reduce_max_sync(0xffffffffu, a);
  if (lane == 0) tops[warp] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) a = max(a, tops[i]);
  const Scale s = scale_of(a);
  uint8_t* dst = q + g * n * kb * 128;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t row = row0 + i * L::kBlocks;
    float f[L::E];
    to_f32(v[i], f);
    if (row < n) store_lane(dst + row * kb * 128 + e, f, s);
  }
  if (threadIdx.x == 0) scale[(g * nb + j0 / 128) * kb + b] = s.scale;
}

// Launched after the weight pack: see bnn_fp8_pack_weight.
__global__ void fp8_settle_kernel() {}

// The widest vector that the row pitch and the base allow, in elements.
template <typename T>
int vec_of(const void* p, int64_t k) {
  int v = Lane<T>::E;
  while (v > 1 && (k % v != 0 || !bnn::aligned(p, v * sizeof(T)))) v /= 2;
  return v;
}

template <typename T, int V>
bnn_status launch_rows(const T* x, int64_t x_rows, const int32_t* index, int64_t rows, int64_t k, uint8_t* q,
                       float* scale, cudaStream_t s) {
  const int64_t kb = (k + 127) / 128, col_tiles = (kb + Lane<T>::kBlocks - 1) / Lane<T>::kBlocks;
  const int64_t grid = (rows + kTileRows - 1) / kTileRows * col_tiles;
  if (grid > INT32_MAX) return BNN_ERR_INVALID_ARG;
  fp8_pack_rows_kernel<T, V><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(x, x_rows, index, rows, k, kb, col_tiles,
                                                                             q, scale);
  return bnn::check_launch();
}

template <typename T>
bnn_status pack_rows(const void* xv, int64_t x_rows, const int32_t* index, int64_t rows, int64_t k, uint8_t* q,
                     float* scale, cudaStream_t s) {
  if (!bnn::aligned(xv, sizeof(T))) return BNN_ERR_MISALIGNED;
  const T* x = static_cast<const T*>(xv);
  const int v = vec_of<T>(xv, k);
  if constexpr (Lane<T>::E == 8)
    if (v == 8) return launch_rows<T, 8>(x, x_rows, index, rows, k, q, scale, s);
  if (v == 4) return launch_rows<T, 4>(x, x_rows, index, rows, k, q, scale, s);
  if (v == 2) return launch_rows<T, 2>(x, x_rows, index, rows, k, q, scale, s);
  return launch_rows<T, 1>(x, x_rows, index, rows, k, q, scale, s);
}

template <typename T, int V>
bnn_status launch_weight(const T* w, int64_t groups, int64_t n, int64_t k, uint8_t* q, float* scale, cudaStream_t s) {
  const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128, grid = groups * nb * kb;
  if (grid > INT32_MAX) return BNN_ERR_INVALID_ARG;
  fp8_pack_weight_kernel<T, V><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(w, n, k, kb, nb, q, scale);
  fp8_settle_kernel<<<1, 1, 0, s>>>();
  return bnn::check_launch();
}

template <typename T>
bnn_status pack_weight(const void* wv, int64_t groups, int64_t n, int64_t k, uint8_t* q, float* scale,
                       cudaStream_t s) {
  if (!bnn::aligned(wv, sizeof(T))) return BNN_ERR_MISALIGNED;
  const T* w = static_cast<const T*>(wv);
  const int v = vec_of<T>(wv, k);
  if constexpr (Lane<T>::E == 8)
    if (v == 8) return launch_weight<T, 8>(w, groups, n, k, q, scale, s);
  if (v == 4) return launch_weight<T, 4>(w, groups, n, k, q, scale, s);
  if (v == 2) return launch_weight<T, 2>(w, groups, n, k, q, scale, s);
  return launch_weight<T, 1>(w, groups, n, k, q, scale, s);
}

}  // namespace

extern "C" bnn_status bnn_fp8_pack_rows(const void* x, int x_type, int64_t x_rows, const int32_t* index, int64_t rows,
                                        int64_t k, uint8_t* q, float* scale, cudaStream_t s) {
  if (x_type < BNN_TYPE_F32 || x_type > BNN_TYPE_F16 || x_rows < 0 || rows < 0 || k < 0 || x_rows > INT32_MAX ||
      rows > INT32_MAX || k > BNN_MAX_K_FP8 || (!index && x_rows < rows))
    return BNN_ERR_INVALID_ARG;
  if (rows == 0 || k == 0) return BNN_OK;
  if ((!x && x_rows > 0) || !q || !scale) return BNN_ERR_INVALID_ARG;
  if (!bnn::aligned(q, 16) || !bnn::aligned(scale, 4) || !bnn::aligned(index, 4)) return BNN_ERR_MISALIGNED;
  switch (x_type) {
    case BNN_TYPE_F32: return pack_rows<float>(x, x_rows, index, rows, k, q, scale, s);
    case BNN_TYPE_BF16: return pack_rows<__nv_bfloat16>(x, x_rows, index, rows, k, q, scale, s);
    default: return pack_rows<__half>(x, x_rows, index, rows, k, q, scale, s);
  }
}

// The empty kernel behind the pack is an ordinary launch: it starts when the
// pack is complete and visible, and a matmul launched with programmatic
// dependent launch cannot start before it.  So weights packed here may be read
// by the next matmul on the stream with nothing in between.
extern "C" bnn_status bnn_fp8_pack_weight(const void* w, int w_type, int64_t groups, int64_t n, int64_t k, uint8_t* q,
                                          float* scale, cudaStream_t s) {
  if (w_type < BNN_TYPE_F32 || w_type > BNN_TYPE_F16 || groups < 0 || n < 0 || k < 0 || groups > BNN_MAX_GROUPS ||
      n > INT32_MAX || groups * n > INT32_MAX || k > BNN_MAX_K_FP8)
    return BNN_ERR_INVALID_ARG;
  if (groups == 0 || n == 0 || k == 0) return BNN_OK;
  if (!w || !q || !scale) return BNN_ERR_INVALID_ARG;
  if (!bnn::aligned(q, 16) || !bnn::aligned(scale, 4)) return BNN_ERR_MISALIGNED;
  switch (w_type) {
    case BNN_TYPE_F32: return pack_weight<float>(w, groups, n, k, q, scale, s);
    case BNN_TYPE_BF16: return pack_weight<__nv_bfloat16>(w, groups, n, k, q, scale, s);
    default: return pack_weight<__half>(w, groups, n, k, q, scale, s);
  }
}
