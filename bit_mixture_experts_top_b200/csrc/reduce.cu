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

constexpr int kGroups = 32;   // row groups per block: one warp each, so that a few hundred rows are one round of loads

// 32 columns of fp32 rows [rows, N].
__device__ __forceinline__ void sum_f32(const float* __restrict__ in, int rows, int N, float* __restrict__ out,
                                        int block, float2 (*part)[32]) {
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int n = block * 32 + lane;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 4
    for (int r = g; r < rows; r += kGroups) s += in[static_cast<int64_t>(r) * N + n];
  }
  part[g][lane].x = s;
  __syncthreads();
  if (g == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) s += part[i][lane].x;
    out[n] = s;
  }
}

// 64 columns of the bf16 rows [r0, r1) of [., N]; a lane owns two adjacent columns (N is even).
__device__ __forceinline__ void sum_bf16(const uint32_t* __restrict__ in, int r0, int r1, int N,
                                         float* __restrict__ out, int block, float2 (*part)[32]) {
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = block * 32 + lane;
  float2 s = make_float2(0.0f, 0.0f);
  if (2 * c < N) {
#pragma unroll 16
    for (int r = r0 + g; r < r1; r += kGroups) {
      const uint32_t v = in[static_cast<int64_t>(r) * (N >> 1) + c];
      s.x += __uint_as_float(v << 16);
      s.y += __uint_as_float(v & 0xFFFF0000u);
    }
  }
  part[g][lane] = s;
  __syncthreads();
  if (g == 0 && 2 * c < N) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
      s.x += part[i][lane].x;
      s.y += part[i][lane].y;
    }
    out[2 * c] = s.x;
    out[2 * c + 1] = s.y;
  }
}

__global__ void __launch_bounds__(32 * kGroups) column_sum_kernel(const float* __restrict__ in, int rows, int N,
                                                                  float* __restrict__ out) {
  __shared__ float2 part[kGroups][32];
  pdl_wait();
  pdl_launch_dependents();
  sum_f32(in, rows, N, out, blockIdx.x, part);
}

// Blocks 0..blocks_a-1 sum the fp32 rows, the others a share of the bf16 rows each: `splits` shares of `per` rows,
// into one row of partial sums per share (straight into the result where there is one share).
__global__ void __launch_bounds__(32 * kGroups)
    column_sums_kernel(const float* __restrict__ a, int rows_a, int Na, float* __restrict__ out_a, int blocks_a,
                       const uint32_t* __restrict__ b, int rows_b, int Nb, int per, int blocks_b,
                       float* __restrict__ out_b) {
  __shared__ float2 part[kGroups][32];
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x;
  if (i < blocks_a) {
    sum_f32(a, rows_a, Na, out_a, i, part);
  } else {
    const int split = (i - blocks_a) / blocks_b;
    sum_bf16(b, split * per, min(rows_b, (split + 1) * per), Nb, out_b + static_cast<int64_t>(split) * Nb,
             (i - blocks_a) % blocks_b, part);
  }
}

}  // namespace

cudaError_t launch_column_sum(const float* in, int rows, int N, float* out, cudaStream_t s) {
  return launch_pdl(column_sum_kernel, dim3((N + 31) / 32), dim3(32 * kGroups), 0, s, in, rows, N, out);
}

// One share up to 1024 rows (32 per warp), then as many as keep that.
int column_sum_splits(int rows) {
  const int b = (rows + 1023) / 1024;
  return b < 1 ? 1 : (b > 128 ? 128 : b);
}

cudaError_t launch_column_sums(const ColumnSums& c, cudaStream_t s) {
  const int splits = column_sum_splits(c.rows_b), per = (c.rows_b + splits - 1) / splits;
  const int blocks_a = c.out_a ? (c.Na + 31) / 32 : 0, blocks_b = (c.Nb + 63) / 64;
  const int grid = blocks_a + (c.out_b ? blocks_b * splits : 0);
  if (grid == 0) return cudaSuccess;
  const cudaError_t e = launch_pdl(column_sums_kernel, dim3(grid), dim3(32 * kGroups), 0, s, c.a, c.rows_a, c.Na,
                                   c.out_a, blocks_a, reinterpret_cast<const uint32_t*>(c.b), c.rows_b, c.Nb, per,
                                   blocks_b, splits > 1 ? c.partial : c.out_b);
  if (e != cudaSuccess || !c.out_b || splits == 1) return e;
  return launch_column_sum(c.partial, splits, c.Nb, c.out_b, s);
}

}  // namespace e4b
