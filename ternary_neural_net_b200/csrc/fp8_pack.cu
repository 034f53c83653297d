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
// once.  Rows of 8192 x 8192: bfloat16 33 us (94% of the measured copy; 36 held
// under the power cap), float32 53.7 us (95%).  Weights: 11008 x 4096 float32
// 35-38 us (91-98%), 16384 x 8192 bfloat16 63.5 us (97%), 8 x 2050 x 4100 bfloat16
// (rows of 8-byte alignment, 2050 = 16 x 128 + 2) 44 us (71%).
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

// A lane's 16 bytes of input as four words.
struct Words {
  uint32_t w[4];
};

// Word i as one float32 or two 16-bit elements.
__device__ __forceinline__ void to_f32(const Words& v, float (&f)[4], float) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v.w[i]);
}
__device__ __forceinline__ void to_f32(const Words& v, float (&f)[8], __nv_bfloat16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v.w[i] << 16);
    f[2 * i + 1] = __uint_as_float(v.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void to_f32(const Words& v, float (&f)[8], __half) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __half2float(__ushort_as_half(static_cast<unsigned short>(v.w[i] & 0xffffu)));
    f[2 * i + 1] = __half2float(__ushort_as_half(static_cast<unsigned short>(v.w[i] >> 16)));
  }
}

// The lane's elements from element e of a row of k on, in loads of V elements
// (k % V == 0 and the row V-aligned); 0 past k.  Narrow loads cost issue slots: rows
// of 4096 bfloat16 x k = 4096, 4100, 4098, 4099 (16-, 8-, 4- and 2-byte loads) take
// 9.5, 11.4, 12.8 and 18.3 us.  (Aligned 16-byte loads whose lanes exchange and
// shift their neighbours' words took 19.3 us for any odd k: more instructions than
// the narrow loads.)
template <typename T, int V>
__device__ __forceinline__ Words load_lane(const T* row, int64_t e, int64_t k) {
  Words v;
  const T* p = row + e;
  if constexpr (V * sizeof(T) == 16) {
    const uint4 x = e < k ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
    v.w[0] = x.x, v.w[1] = x.y, v.w[2] = x.z, v.w[3] = x.w;
  } else if constexpr (V * sizeof(T) == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint2 x = e + i * V < k ? *reinterpret_cast<const uint2*>(p + i * V) : make_uint2(0, 0);
      v.w[2 * i] = x.x, v.w[2 * i + 1] = x.y;
    }
  } else if constexpr (V * sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = e + i * V < k ? *reinterpret_cast<const uint32_t*>(p + i * V) : 0u;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = e + 2 * i < k ? h[2 * i] : 0u, hi = e + 2 * i + 1 < k ? h[2 * i + 1] : 0u;
      v.w[i] = lo | (hi << 16);
    }
  }
  return v;
}

// Largest absolute value among a lane's elements so far, `a`, and those of `v`,
// as bit patterns without the sign: float32, or two 16-bit elements compared at
// a time.  bits_of then gives the float32 bits.
__device__ __forceinline__ uint32_t top(uint32_t a, const Words& v, float) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a = max(a, v.w[i] & 0x7fffffffu);
  return a;
}
template <typename T>
__device__ __forceinline__ uint32_t top(uint32_t a, const Words& v, T) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a = __vmaxu2(a, v.w[i] & 0x7fff7fffu);
  return a;
}
__device__ __forceinline__ uint32_t bits_of(uint32_t a, float) { return a; }
__device__ __forceinline__ uint32_t bits_of(uint32_t a, __nv_bfloat16) { return max(a & 0xffffu, a >> 16) << 16; }
__device__ __forceinline__ uint32_t bits_of(uint32_t a, __half) {
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(max(a & 0xffffu, a >> 16)))));
}

struct Scale {
  float scale, factor;  // factor 0: the block holds an infinity or a NaN
};

__device__ __forceinline__ Scale scale_of(uint32_t bits) {
  Scale s;
  const bool fine = bits < kInfBits;
  const float a = fine ? fmaxf(__uint_as_float(bits), 0x1p-100f) : 1.0f;
  s.scale = fine ? __fdiv_rn(a, kTop) : __int_as_float(0x7fffffff);
  s.factor = fine ? __fdiv_rn(kTop, a) : 0.0f;
  return s;
}

// Four floats times the factor as four e4m3 bytes, lowest address first.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float r) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(__fmul_rn(b, r)), "f"(__fmul_rn(a, r)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(__fmul_rn(d, r)), "f"(__fmul_rn(c, r)));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ void store_lane(uint8_t* dst, const float (&f)[4], float r) {
  *reinterpret_cast<uint32_t*>(dst) = r != 0.0f ? e4m3x4(f[0], f[1], f[2], f[3], r) : 0u;
}
__device__ __forceinline__ void store_lane(uint8_t* dst, const float (&f)[8], float r) {
  uint2 v = make_uint2(0u, 0u);
  if (r != 0.0f) v = make_uint2(e4m3x4(f[0], f[1], f[2], f[3], r), e4m3x4(f[4], f[5], f[6], f[7], r));
  *reinterpret_cast<uint2*>(dst) = v;
}

// Rows.  A warp takes one row x kSteps consecutive steps of kBlocks blocks: its
// 16-byte loads are in flight together and read the row contiguously.  A CTA's
// eight rows' scales leave as 32-byte pieces of the block-major scale matrix.
constexpr int kSteps = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
fp8_pack_rows_kernel(const T* __restrict__ x, int64_t x_rows, const int32_t* __restrict__ index, int64_t rows,
                     int64_t k, int64_t kb, int64_t col_tiles, uint8_t* __restrict__ q, float* __restrict__ scale) {
  using L = Lane<T>;
  constexpr int kTileBlocks = kSteps * L::kBlocks;
  __shared__ float sc[kTileBlocks][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile_row = (blockIdx.x / col_tiles) * kWarps, row = tile_row + warp;
  const int64_t b0 = (blockIdx.x % col_tiles) * kTileBlocks;
  const int64_t e0 = b0 * 128 + lane * L::E;
  bnn::pdl_trigger();  // a matmul launched after this kernel may start on its weights now
  int64_t src = row;
  if (index) src = row < rows ? static_cast<int64_t>(__ldg(index + row)) : -1;
  const bool live = row < rows && src >= 0 && src < x_rows;
  Words v[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) v[i] = load_lane<T, V>(x + (live ? src : 0) * k, live ? e0 + i * 32 * L::E : k, k);
  // The steps' maxima, then both divisions once for all of the warp's blocks: lane i of each block's lanes takes
  // step i.
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    uint32_t a = bits_of(top(0u, v[i], T{}), T{});
#pragma unroll
    for (int off = L::kLanes / 2; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (lane % L::kLanes == i) mine = a;
  }
  const Scale s = scale_of(mine);
  if (lane % L::kLanes < kSteps) sc[lane % L::kLanes * L::kBlocks + lane / L::kLanes][warp] = s.scale;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const float r = __shfl_sync(0xffffffffu, s.factor, i, L::kLanes);
    float f[L::E];
    to_f32(v[i], f, T{});
    if (row < rows && b0 + i * L::kBlocks + lane / L::kLanes < kb)
      store_lane(q + row * kb * 128 + e0 + i * 32 * L::E, f, r);
  }
  __syncthreads();
  const int b = threadIdx.x / kWarps, r = threadIdx.x % kWarps;
  if (b < kTileBlocks && b0 + b < kb && tile_row + r < rows) scale[(b0 + b) * rows + tile_row + r] = sc[b][r];
}

// Weights.  A CTA takes 128 rows x kBlocks blocks (512 bytes of a row) whole in
// registers, a warp 16 of the rows, one 16-byte load a lane for each.  (2-byte
// loads spill 68 bytes a thread at two CTAs an SM, the wide ones 16 at three.)
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, V * sizeof(T) >= 8 ? 3 : 2)
fp8_pack_weight_kernel(const T* __restrict__ w, int64_t n, int64_t k, int64_t kb, int64_t nb, int64_t col_tiles,
                       uint8_t* __restrict__ q, float* __restrict__ scale) {
  using L = Lane<T>;
  constexpr int kRows = 128 / kWarps;  // rows of a warp
  __shared__ uint32_t tops[kWarps][L::kBlocks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blk = lane / L::kLanes;
  const int64_t t = blockIdx.x / col_tiles, j0 = (t % nb) * 128, g = t / nb;
  const int64_t b0 = (blockIdx.x % col_tiles) * L::kBlocks, e = b0 * 128 + lane * L::E;
  const int64_t row0 = j0 + warp * kRows;
  bnn::pdl_trigger();  // (for the settle kernel, which waits for this one's end)
  const T* base = w + g * n * k;
  Words v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const bool live = row0 + i < n;
    v[i] = load_lane<T, V>(base + (live ? row0 + i : 0) * k, live ? e : k, k);
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) a = top(a, v[i], T{});
  a = bits_of(a, T{});
#pragma unroll
  for (int off = L::kLanes / 2; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
  if (lane % L::kLanes == 0) tops[warp][blk] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) a = max(a, tops[i][blk]);
  const Scale s = scale_of(a);
  uint8_t* dst = q + g * n * kb * 128;
  if (b0 + blk < kb) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float f[L::E];
      to_f32(v[i], f, T{});
      if (row0 + i < n) store_lane(dst + (row0 + i) * kb * 128 + e, f, s.factor);
    }
    if (warp == 0 && lane % L::kLanes == 0) scale[(g * nb + j0 / 128) * kb + b0 + blk] = s.scale;
  }
}

// Launched after the weight pack: see bnn_fp8_pack_weight.
__global__ void fp8_settle_kernel() { bnn::pdl_wait(); }

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
  constexpr int kTileBlocks = kSteps * Lane<T>::kBlocks;
  const int64_t kb = (k + 127) / 128, col_tiles = (kb + kTileBlocks - 1) / kTileBlocks;
  const int64_t grid = (rows + kWarps - 1) / kWarps * col_tiles;
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
  const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128, col_tiles = (kb + Lane<T>::kBlocks - 1) / Lane<T>::kBlocks;
  const int64_t grid = groups * nb * col_tiles;
  if (grid > INT32_MAX) return BNN_ERR_INVALID_ARG;
  fp8_pack_weight_kernel<T, V><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(w, n, k, kb, nb, col_tiles, q, scale);
  const bnn_status st = bnn::check_launch();
  if (st != BNN_OK) return st;
  const cudaError_t e = bnn::launch_pdl(fp8_settle_kernel, dim3(1), dim3(1), 0, s, 1u);
  if (e != cudaSuccess) return bnn::cuda_fail(e);
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

// The kernel behind the pack waits until the pack is complete and visible and
// then ends, without letting its successor start earlier.  A matmul launched
// with programmatic dependent launch starts after that end at the earliest, so
// weights packed here may be read by the next matmul on the stream with nothing
// in between.
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
