// bnn_fp8_gemm / bnn_fp8_grouped_gemm: matrix products of e4m3 operands with a
// float32 scale for each block of 128 (include/bnn.h has the format).
//
//   y[i,j] = sum_b xs[b,i] ws[j/128,b] sum_{e in block b} xq[i,e] wq[j,e] (+ bias[j])
//
// First form: one thread per output, 16 x 16 outputs a CTA, both operands' tiles
// of one block of k converted to float32 in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "bnn_internal.cuh"

namespace {

constexpr int kTile = 16;

__device__ __forceinline__ float e4m3_value(uint8_t v) {
  __nv_fp8_e4m3 t;
  t.__x = v;
  return static_cast<float>(t);
}

__device__ __forceinline__ void store_out(void* out, int type, int64_t at, float y) {
  if (type == BNN_TYPE_F32)
    static_cast<float*>(out)[at] = y;
  else if (type == BNN_TYPE_BF16)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
  else
    static_cast<__half*>(out)[at] = __float2half_rn(y);
}

// offsets == nullptr: one group of all rows.
__global__ void __launch_bounds__(kTile* kTile)
fp8_gemm_simple_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
                       const float* __restrict__ ws, const float* __restrict__ bias,
                       const int64_t* __restrict__ offsets, int groups, int64_t rows, int64_t n, int64_t kb,
                       void* __restrict__ out, int out_type) {
  __shared__ float xt[kTile][129], wt[kTile][129];
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  const int64_t nb = (n + 127) / 128;
  for (int64_t tile = blockIdx.y; tile * kTile < rows + static_cast<int64_t>(groups) * kTile; tile += gridDim.y) {
    // the tile's group: groups are cut into tiles of kTile rows one after another
    int64_t i0 = tile * kTile, end = rows, g = 0;
    if (offsets) {
      int64_t left = tile, lo = 0;
      bool found = false;
      int64_t prev = max(int64_t{0}, min(rows, offsets[0]));
      for (g = 0; g < groups; ++g) {
        const int64_t next = max(prev, min(rows, offsets[g + 1]));
        const int64_t tiles = (next - prev + kTile - 1) / kTile;
        if (left < tiles) {
          lo = prev + left * kTile;
          end = next;
          found = true;
          break;
        }
        left -= tiles;
        prev = next;
      }
      if (!found) return;
      i0 = lo;
    }
    if (i0 >= end) return;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int64_t i = i0 + ty, j = j0 + tx;
    float acc = 0.0f;
    for (int64_t b = 0; b < kb; ++b) {
      __syncthreads();
      for (int t = threadIdx.x; t < kTile * 128; t += kTile * kTile) {
        const int r = t / 128, e = t % 128;
        xt[r][e] = i0 + r < end ? e4m3_value(xq[(i0 + r) * kb * 128 + b * 128 + e]) : 0.0f;
        wt[r][e] = j0 + r < n ? e4m3_value(wq[(g * n + j0 + r) * kb * 128 + b * 128 + e]) : 0.0f;
      }
      __syncthreads();
      float part = 0.0f;
      for (int e = 0; e < 128; ++e) part = fmaf(xt[ty][e], wt[tx][e], part);
      if (i < end && j < n) acc = fmaf(part, xs[b * rows + i] * ws[(g * nb + j / 128) * kb + b], acc);
    }
    if (i < end && j < n) store_out(out, out_type, i * n + j, bias ? acc + bias[j] : acc);
  }
}

bnn_status launch_simple(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const float* bias,
                         const int64_t* offsets, int64_t groups, int64_t rows, int64_t n, int64_t kb, void* out,
                         int out_type, cudaStream_t s) {
  const int64_t gx = (n + kTile - 1) / kTile, gy = (rows + kTile - 1) / kTile + groups;
  if (gx > INT32_MAX) return BNN_ERR_INVALID_ARG;
  fp8_gemm_simple_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy < 65535 ? gy : 65535)),
                           kTile * kTile, 0, s>>>(xq, xs, wq, ws, bias, offsets, static_cast<int>(groups), rows, n, kb,
                                                  out, out_type);
  return bnn::check_launch();
}

size_t type_size(int type) { return type == BNN_TYPE_F32 ? 4 : 2; }

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
      !bnn::aligned(bias, 4) || !bnn::aligned(out, type_size(out_type)))
    return BNN_ERR_MISALIGNED;
  return launch_simple(xq, xs, wq, ws, bias, nullptr, 1, m, n, (k + 127) / 128, out, out_type, s);
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
      !bnn::aligned(offsets, 8) || !bnn::aligned(out, type_size(out_type)))
    return BNN_ERR_MISALIGNED;
  return launch_simple(xq, xs, wq, ws, nullptr, offsets, groups, rows, n, (k + 127) / 128, out, out_type, s);
}
