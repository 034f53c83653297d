// The e4m3 matmul for up to 8 rows: bound by the weights' bytes, and for small
// weights by latency.  Weights go from global memory straight to registers and
// into mma.sync (m16n8k32, e4m3): no shared memory, barrier or tensor memory
// stands between the launch and the first load, and all of a small layer's
// bytes are in flight at once.  (The tensor cores are nearly idle: a few
// hundred clocks of work per SM.)
//
// A CTA takes 16 weight rows (the MMA's M) times all rows of x (its N);
// its eight warps take every eighth block of k, four in flight each, and
// add their sums through shared memory in warp order.  Small CTAs in waves keep
// the SMs evenly loaded.  Within a block of 128 bytes a lane loads the 16-byte
// pieces t and 4 + t (t = lane mod 4) of its rows, for weights and x alike: that
// permutes k in both operands the same way, so the sums are unchanged, and every
// load instruction of a warp reads whole 64-byte pieces of eight rows.
//
// The weights' first blocks are fetched before the wait for the kernel ahead
// (programmatic dependent launch).
//
// 1024 x 1000 in 2.1 us back to back, weights in cache; 4096 x 4096 in 5.6-6.2 us;
// 11008 x 4096 in 11.5 us (15.9 us cold: 45.1 MB at 2.8 TB/s, the ramp of so
// short a launch).  At 28672 x 8192 it runs at 65% of what HBM gives (54.7 us),
// with 128 registers a thread limiting the bytes in flight, so larger weights go
// to the tensor-memory kernel.
#include "fp8_common.cuh"

namespace {

using bnn::fp8::Args;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 16, kCols = 8;  // weight rows of a CTA, rows of x (the MMA's M and N)
constexpr int D = 4;                  // blocks of k in flight per warp

__device__ __forceinline__ uint4 load_weights(const uint8_t* p) {  // read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kThreads, 2)
fp8_skinny_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
                  const float* __restrict__ ws, const float* __restrict__ bias, int m, int64_t n, int kb,
                  void* __restrict__ out, int out_type) {
  __shared__ float red[kWarps][kCols][kRows + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kRows, pitch = static_cast<int64_t>(kb) * 128;
  const uint8_t* wrow[2];  // this lane's weight rows (past n: the last one, not stored)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t j = j0 + 8 * i + g;
    wrow[i] = wq + (j < n ? j : n - 1) * pitch + 16 * t;
  }
  const float* wsp = ws + j0 / 128 * kb;
  uint4 w[D][2][2], x[2][2];
  float sw[D], sx[2][2];
  auto fetch_w = [&](int b, int d) {
    if (b < kb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[d][i][0] = load_weights(wrow[i] + static_cast<int64_t>(b) * 128);
        w[d][i][1] = load_weights(wrow[i] + static_cast<int64_t>(b) * 128 + 64);
      }
      sw[d] = __ldg(wsp + b);
    }
  };
  auto fetch_x = [&](int b, int d) {
    const int c = 2 * t;
    x[d][0] = x[d][1] = make_uint4(0, 0, 0, 0);
    sx[d][0] = sx[d][1] = 0.0f;
    if (b < kb) {
      if (g < m) {
        const uint4* p = reinterpret_cast<const uint4*>(xq + g * pitch + static_cast<int64_t>(b) * 128 + 16 * t);
        x[d][0] = __ldg(p);
        x[d][1] = __ldg(p + 4);
      }
      if (c < m) sx[d][0] = __ldg(xs + static_cast<int64_t>(b) * m + c);
      if (c + 1 < m) sx[d][1] = __ldg(xs + static_cast<int64_t>(b) * m + c + 1);
    }
  };
  bnn::pdl_trigger();
#pragma unroll
  for (int d = 0; d < D; ++d) fetch_w(warp + kWarps * d, d);
  bnn::pdl_wait();  // the activations may come from the preceding kernel
  fetch_x(warp, 0);
  float acc[4] = {};
  for (int b = warp; b < kb; b += kWarps * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int bd = b + kWarps * d, u = d & 1;
      if (bd < kb) {
        fetch_x(bd + kWarps, u ^ 1);
        float c[4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 lo = w[d][0][h], hi = w[d][1][h], v = x[u][h];
          mma(c, lo.x, hi.x, lo.y, hi.y, v.x, v.y);
          mma(c, lo.z, hi.z, lo.w, hi.w, v.z, v.w);
        }
        const float s0 = sx[u][0] * sw[d], s1 = sx[u][1] * sw[d];
        acc[0] = fmaf(c[0], s0, acc[0]);
        acc[1] = fmaf(c[1], s1, acc[1]);
        acc[2] = fmaf(c[2], s0, acc[2]);
        acc[3] = fmaf(c[3], s1, acc[3]);
        fetch_w(bd + kWarps * D, d);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[warp][2 * t + (e & 1)][g + 8 * (e >> 1)] = acc[e];
  __syncthreads();
  for (int o = tid; o < kRows * kCols; o += kThreads) {
    const int c = o / kRows, r = o % kRows;
    const int64_t j = j0 + r;
    if (c < m && j < n) {
      float y = 0.0f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) y += red[v][c][r];
      bnn::fp8::store_one(out, out_type, c * n + j, bias ? y + __ldg(bias + j) : y);
    }
  }
}

bnn_status launch(const Args& a) {
  const int64_t grid = (a.n + kRows - 1) / kRows;
  const cudaError_t e = bnn::launch_pdl(fp8_skinny_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                                        0, a.stream, 1u, a.xq, a.xs, a.wq, a.ws, a.bias, static_cast<int>(a.rows), a.n,
                                        a.kb, a.out, a.out_type);
  if (e != cudaSuccess) return bnn::cuda_fail(e);
  return bnn::check_launch();
}

}  // namespace

namespace bnn {
namespace fp8 {

bnn_status gemm_skinny(const Args& a) { return launch(a); }

}  // namespace fp8
}  // namespace bnn
