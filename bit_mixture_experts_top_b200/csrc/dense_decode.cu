// The gated feed-forward block for a few tokens: the products are bound by the
// weight stream, so every weight is read once, straight from global memory
// into the registers of a warp-level MMA, with no shared-memory stage.
//
//   gate_up : h = act(x W_gate^T + b, x W_up^T + b)      8 features per block
//   down    : out = h W_dn^T (+ b) (+ add)               16 rows per block
//
// The weights are the 16-row operand of mma.m16n8k16 and the tokens its eight
// columns (NB tiles of eight).  The order of K inside a product is free as long
// as both operands agree, so a lane takes the eight consecutive values of K
// that one 16-byte load brings as its elements of two MMAs.  In gate_up the
// upper eight rows of the tile are the up features of the lower eight's gate
// features, so a lane ends with gate and up of the same (feature, token).
// The block's eight warps split K and add their partial tiles through shared
// memory in a fixed order.
//
// The down kernel loads its first weights before it waits for the gate_up
// kernel (they do not depend on it).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr int WARPS = 8;
constexpr int UNROLL = 4;                   // chunks of 32 K in flight per warp

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int NB, bool GATE_UP>
__global__ void __launch_bounds__(32 * WARPS) dense_decode_kernel(const DenseDecodeLaunch p) {
  __shared__ float part[WARPS][NB][16][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int chunks = (p.K + 31) / 32;
  // weight rows of this lane: MMA rows g and g + 8
  const int n0 = blockIdx.x * (GATE_UP ? 8 : 16);
  const int row_lo = n0 + g, row_hi = GATE_UP ? p.N + n0 + g : n0 + 8 + g;
  const bool lo_in = row_lo < p.N, hi_in = GATE_UP || row_hi < p.N;
  const uint16_t* w_lo = p.w + static_cast<int64_t>(lo_in ? row_lo : 0) * p.K + 8 * t;
  const uint16_t* w_hi = p.w + static_cast<int64_t>(hi_in ? row_hi : 0) * p.K + 8 * t;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 lo[UNROLL], hi[UNROLL];
  auto load_w = [&](int c0) {
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int k = 32 * (c0 + i * WARPS);
      const bool in = k + 8 * t < p.K;          // K is a multiple of 8
      lo[i] = in && lo_in ? load_stream(w_lo + k) : zero;
      hi[i] = in && hi_in ? load_stream(w_hi + k) : zero;
    }
  };
  // Everything up to the launch before the previous one has completed when this
  // grid may start (that one waits before it releases its dependents), so of the
  // down kernel's inputs only h, which the previous launch writes, has to wait.
  if (GATE_UP) {
    pdl_wait();
    pdl_launch_dependents();
    load_w(warp);
    if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  } else {
    load_w(warp);
    pdl_wait();
    pdl_launch_dependents();
  }
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
  for (int c0 = warp; c0 < chunks; c0 += UNROLL * WARPS) {
    uint4 x[UNROLL][NB];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int k = 32 * (c0 + i * WARPS) + 8 * t;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int tok = 8 * b + g;
        x[i][b] = tok < p.T && k < p.K ? *reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(tok) * p.K + k) : zero;
      }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mma16816(acc[b], lo[i].x, hi[i].x, lo[i].y, hi[i].y, x[i][b].x, x[i][b].y);
        mma16816(acc[b], lo[i].z, hi[i].z, lo[i].w, hi[i].w, x[i][b].z, x[i][b].w);
      }
    if (c0 + UNROLL * WARPS < chunks) load_w(c0 + UNROLL * WARPS);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    *reinterpret_cast<float2*>(&part[warp][b][g][2 * t]) = make_float2(acc[b][0], acc[b][1]);
    *reinterpret_cast<float2*>(&part[warp][b][g + 8][2 * t]) = make_float2(acc[b][2], acc[b][3]);
  }
  __syncthreads();
  // one output per thread: consecutive threads take consecutive rows of one token
  constexpr int ROWS = GATE_UP ? 8 : 16;
  for (int i = threadIdx.x; i < ROWS * 8 * NB; i += 32 * WARPS) {
    const int r = i % ROWS, tok = i / ROWS, n = n0 + r;
    if (tok >= p.T || n >= p.N) continue;
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      a += part[w][tok >> 3][r][tok & 7];
      if (GATE_UP) b += part[w][tok >> 3][r + 8][tok & 7];
    }
    const int64_t at = static_cast<int64_t>(tok) * p.N + n;
    if (GATE_UP) {
      if (p.bias) {
        a += __ldg(p.bias + n);
        b += __ldg(p.bias + p.N + n);
      }
      if (p.g_out) {
        p.g_out[2 * static_cast<int64_t>(tok) * p.N + n] = a;
        p.g_out[2 * static_cast<int64_t>(tok) * p.N + p.N + n] = b;
      }
      a = expert_act(p.ep, a, b);
    } else {
      if (p.bias) a += __ldg(p.bias + n);
      if (p.add) a += __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.add)[at]);
    }
    reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(a);
  }
}

}  // namespace

cudaError_t launch_dense_decode(const DenseDecodeLaunch& p, bool gate_up, cudaStream_t s) {
  const int per = gate_up ? 8 : 16;
  const dim3 grid((p.N + per - 1) / per), block(32 * WARPS);
  if (p.T <= 8)
    return gate_up ? launch_pdl(dense_decode_kernel<1, true>, grid, block, 0, s, p)
                   : launch_pdl(dense_decode_kernel<1, false>, grid, block, 0, s, p);
  return gate_up ? launch_pdl(dense_decode_kernel<2, true>, grid, block, 0, s, p)
                 : launch_pdl(dense_decode_kernel<2, false>, grid, block, 0, s, p);
}

}  // namespace e4b
