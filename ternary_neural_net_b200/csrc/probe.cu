// Measurement helpers (see bnn_probe.h): the integer-pipe rate probe and a
// read-only HBM stream.
#include "bnn_internal.cuh"
#include "bnn_probe.h"
#include "fp8_common.cuh"

namespace {

constexpr int kChains = 8;

__global__ void __launch_bounds__(256) probe_popc_kernel(int mode, int64_t iters, int32_t* __restrict__ sink) {
  const uint32_t tid = blockIdx.x * blockDim.x + threadIdx.x;
  uint32_t a[kChains], b[kChains];
#pragma unroll
  for (int c = 0; c < kChains; ++c) {
    a[c] = tid * 2654435761u + c * 40503u;
    b[c] = tid ^ (c * 0x9E3779B9u);
  }
  if (mode == 0) {
    for (int64_t i = 0; i < iters; ++i) {
#pragma unroll
      for (int c = 0; c < kChains; ++c) a[c] = __popc(a[c]) + b[c] + a[c];
    }
  } else {
    for (int64_t i = 0; i < iters; ++i) {
#pragma unroll
      for (int c = 0; c < kChains; ++c) {
        // one 64-bit word pair: XOR both halves, popcount both, accumulate
        const uint32_t lo = a[c] ^ b[c];
        const uint32_t hi = a[c] ^ (b[c] + 0x5bd1e995u);
        a[c] = a[c] + __popc(lo) + __popc(hi);
      }
    }
  }
  uint32_t r = 0;
#pragma unroll
  for (int c = 0; c < kChains; ++c) r ^= a[c];
  sink[tid] = static_cast<int32_t>(r);
}

// Read-only stream: each warp reads one contiguous 2 KiB block per step (four
// 16-byte streaming loads per lane, 512 consecutive bytes per load
// instruction), blocks strided by the number of warps in the grid.  The loads
// are folded into one register, which is written only when it equals a value
// no input of the bench produces, so the kernel's DRAM traffic is the
// buffer's bytes read once.
__global__ void __launch_bounds__(512) probe_read_kernel(const uint4* __restrict__ p, int64_t n16,
                                                         uint32_t key, uint32_t* __restrict__ sink) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  uint32_t acc = 0;
  for (int64_t b = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; 128 * b < n16; b += warps) {
    const int64_t i = 128 * b + lane;
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i + 32 * u < n16 ? __ldcs(p + i + 32 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u) acc ^= v[u].x + v[u].y + v[u].z + v[u].w;
  }
  if (acc == key) sink[0] = acc;
}

}  // namespace

extern "C" bnn_status bnn_probe_stream_read(const void* buf, int64_t bytes, int64_t blocks, uint32_t* sink,
                                            cudaStream_t s) {
  if (!buf || !sink || bytes < 0 || bytes % 16 != 0 || blocks <= 0 || blocks > (1 << 22)) return BNN_ERR_INVALID_ARG;
  if (!bnn::aligned(buf, 16) || !bnn::aligned(sink, 4)) return BNN_ERR_MISALIGNED;
  if (bytes == 0) return BNN_OK;
  probe_read_kernel<<<static_cast<unsigned>(blocks), 512, 0, s>>>(static_cast<const uint4*>(buf), bytes / 16,
                                                                   0x9E3779B9u, sink);
  return bnn::check_launch();
}

extern "C" bnn_status bnn_probe_popc(int mode, int64_t blocks, int64_t iters, int32_t* sink, double* ops,
                                     cudaStream_t s) {
  if ((mode != 0 && mode != 1) || blocks <= 0 || blocks > (1 << 22) || iters < 0 || !sink || !ops)
    return BNN_ERR_INVALID_ARG;
  if (!bnn::aligned(sink, 4)) return BNN_ERR_MISALIGNED;
  *ops = static_cast<double>(blocks) * 256.0 * static_cast<double>(iters) * kChains;
  probe_popc_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(mode, iters, sink);
  return bnn::check_launch();
}

extern "C" bnn_status bnn_probe_ternary_plan(int64_t n, int64_t k, const int* active, int* rows, int* ks) {
  if (n < 1 || k < 1 || !active || !rows || !ks) return BNN_ERR_INVALID_ARG;
  bnn::ternary_tmem_plan(n, k, active, rows, ks);
  return BNN_OK;
}

extern "C" bnn_status bnn_probe_fp8_plan(int64_t rows, int64_t n, int64_t k, int64_t groups, int sms, int* kernel,
                                         int* tile_rows, int* tile_cols, int* split) {
  if (rows < 1 || n < 1 || k < 0 || groups < 0 || sms < 2 || rows > INT32_MAX || n > INT32_MAX || k > BNN_MAX_K_FP8 ||
      groups > BNN_MAX_GROUPS || !kernel || !tile_rows || !tile_cols || !split)
    return BNN_ERR_INVALID_ARG;
  const bnn::fp8::Plan p =
      bnn::fp8::plan(rows, n, static_cast<int>((k + 127) / 128), groups > 0 ? groups : 1, groups > 0, sms);
  *kernel = p.kernel;
  *tile_rows = p.rows;
  *tile_cols = p.cols;
  *split = p.split;
  return BNN_OK;
}
