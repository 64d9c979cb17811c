// Column sums: out[n] = sum over rows of in[., n], in fp32, for the partial
// weight gradients of the norm and the bias gradients of the feed-forward
// block.  The order of the additions depends on the sizes alone (no atomics),
// so the same inputs give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr int kGroups = 16;   // row groups per block: one warp each, 32 columns wide

__global__ void __launch_bounds__(32 * kGroups) column_sum_kernel(const float* __restrict__ in, int rows, int N,
                                                                  float* __restrict__ out) {
  __shared__ float part[kGroups][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 4
    for (int r = g; r < rows; r += kGroups) s += in[static_cast<int64_t>(r) * N + n];
  }
  part[g][lane] = s;
  __syncthreads();
  if (g == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) s += part[i][lane];
    out[n] = s;
  }
}

// bf16 rows [rows, N] -> one row of partial sums per blockIdx.y; a thread owns
// two adjacent columns (N is even).
__global__ void __launch_bounds__(128) column_sum_bf16_kernel(const uint32_t* __restrict__ in, int rows, int N,
                                                              int rows_per_block, float* __restrict__ partial) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (2 * c >= N) return;
  const int r0 = blockIdx.y * rows_per_block;
  const int r1 = min(rows, r0 + rows_per_block);
  float lo = 0.0f, hi = 0.0f;
#pragma unroll 8
  for (int r = r0; r < r1; ++r) {
    const uint32_t v = in[static_cast<int64_t>(r) * (N >> 1) + c];
    lo += __uint_as_float(v << 16);
    hi += __uint_as_float(v & 0xFFFF0000u);
  }
  reinterpret_cast<float2*>(partial + static_cast<int64_t>(blockIdx.y) * N)[c] = make_float2(lo, hi);
}

}  // namespace

cudaError_t launch_column_sum(const float* in, int rows, int N, float* out, cudaStream_t s) {
  return launch_pdl(column_sum_kernel, dim3((N + 31) / 32), dim3(32 * kGroups), 0, s, in, rows, N, out);
}

int column_sum_bf16_blocks(int rows) {
  const int b = (rows + 63) / 64;
  return b < 1 ? 1 : (b > 128 ? 128 : b);
}

cudaError_t launch_column_sum_bf16(const uint16_t* in, int rows, int N, float* partial, float* out, cudaStream_t s) {
  const int blocks = column_sum_bf16_blocks(rows);
  const int per = (rows + blocks - 1) / blocks;
  const cudaError_t e = launch_pdl(column_sum_bf16_kernel, dim3((N / 2 + 127) / 128, blocks), dim3(128), 0, s,
                                   reinterpret_cast<const uint32_t*>(in), rows, N, per, partial);
  return e != cudaSuccess ? e : launch_column_sum(partial, blocks, N, out, s);
}

}  // namespace e4b
