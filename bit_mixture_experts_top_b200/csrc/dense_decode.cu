// The gated feed-forward block for a few tokens: the products are bound by the
// weight stream, so every weight is read once, by asynchronous copies into
// shared memory that its own warp feeds to warp-level MMAs.
//
//   gate_up : h = act(x W_gate^T + b, x W_up^T + b)      8 features per block
//   down    : out = h W_dn^T (+ b) (+ add)               16 rows per block
//
// The weights are the 16-row operand of mma.m16n8k16 and the tokens its eight
// columns (NB tiles of eight).  In gate_up the upper eight rows of the tile are
// the up features of the lower eight's gate features, so a lane ends with gate
// and up of the same (feature, token).  The block's eight warps split K in
// blocks of 64 and add their partial tiles through shared memory in a fixed
// order.
//
// Every warp feeds itself: cp.async brings whole 128-byte pieces of its weight
// and token rows into a private ring of STAGES blocks (swizzled, so that the
// fragment reads are free of bank conflicts), which keeps STAGES x 24 KB and
// more in flight per block without registers or block barriers.  The order of K
// inside a product is free as long as both operands agree, so a lane takes the
// eight consecutive values of a 16-byte word as its elements of two MMAs.
//
// The down kernel's first weights are on their way before it waits for the
// gate_up kernel (they do not depend on it).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr int WARPS = 8;
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes, or zeros where `in` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t smem, const uint16_t* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

template <int NB>
constexpr int stage_bytes() { return 2048 + NB * 1024; }       // 16 weight rows and 8 NB token rows of 128 bytes

template <int NB, int STAGES>
constexpr int smem_bytes() { return WARPS * STAGES * stage_bytes<NB>(); }

template <int NB, int STAGES, bool GATE_UP>
__global__ void __launch_bounds__(32 * WARPS) dense_decode_kernel(const DenseDecodeLaunch p) {
  extern __shared__ __align__(1024) uint8_t ring[];
  static_assert(WARPS * NB * 16 * 8 * 4 <= smem_bytes<NB, STAGES>(), "the partial tiles reuse the rings");
  float (*part)[NB][16][8] = reinterpret_cast<float (*)[NB][16][8]>(ring);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int blocks = (p.K + 63) / 64;
  const int n0 = blockIdx.x * (GATE_UP ? 8 : 16);
  // copies: a lane moves the 16-byte word lane & 7 of rows lane / 8 + {0, 4, 8, 12}
  const int cr = lane >> 3, cw = lane & 7;
  const uint32_t mine = smem_u32(ring) + warp * STAGES * stage_bytes<NB>();
  const uint16_t* wsrc[4];
  const uint16_t* xsrc[2 * NB];
  bool win[4], xin[2 * NB];
  uint32_t dst[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = cr + 4 * i;
    const int row = GATE_UP && r >= 8 ? p.N + n0 + r - 8 : n0 + r;
    win[i] = GATE_UP || row < p.N;
    wsrc[i] = p.w + static_cast<int64_t>(win[i] ? row : 0) * p.K;
    dst[i] = r * 128 + ((cw ^ (r & 7)) << 4);
  }
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i) {
    const int tok = cr + 4 * i;
    xin[i] = tok < p.T;
    xsrc[i] = p.x + static_cast<int64_t>(xin[i] ? tok : 0) * p.K;
  }
  auto copy_w = [&](int kb, int stage) {
    const int k = kb * 64 + cw * 8;              // K is a multiple of 8
    const bool in = k < p.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) copy16(mine + stage * stage_bytes<NB>() + dst[i], wsrc[i] + (in ? k : 0), in && win[i]);
  };
  auto copy_x = [&](int kb, int stage) {
    const int k = kb * 64 + cw * 8;
    const bool in = k < p.K;
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i)             // (token rows are swizzled like weight rows: rows 8b + r by r)
      copy16(mine + stage * stage_bytes<NB>() + 2048 + (i >> 1) * 1024 + dst[i & 1], xsrc[i] + (in ? k : 0), in && xin[i]);
  };
  // Everything up to the launch before the previous one has completed when this
  // grid may start (that one waits before it releases its dependents), so of the
  // down kernel's inputs only h, which the previous launch writes, has to wait.
  if (GATE_UP) {
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  }
#pragma unroll
  for (int s = 0; s < STAGES; ++s)
    if (warp + s * WARPS < blocks) copy_w(warp + s * WARPS, s);
  if (!GATE_UP) {
    pdl_wait();
    pdl_launch_dependents();
  }
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    if (warp + s * WARPS < blocks) copy_x(warp + s * WARPS, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
  int stage = 0;
  for (int kb = warp; kb < blocks; kb += WARPS) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    __syncwarp();
    const uint32_t at = mine + stage * stage_bytes<NB>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {                // words t and t + 4 of this lane's rows: 32 of K each
      const uint32_t o = g * 128 + (((t + 4 * h) ^ g) << 4);
      const uint4 lo = lds16(at + o), hi = lds16(at + 1024 + o);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 x = lds16(at + 2048 + b * 1024 + o);
        mma16816(acc[b], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        mma16816(acc[b], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
      }
    }
    __syncwarp();                                // every lane has read the slot
    const int next = kb + STAGES * WARPS;
    if (next < blocks) {
      copy_w(next, stage);
      copy_x(next, stage);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();                               // the partial tiles go where the rings were
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
      a = dense_act(p.ep, a, b);
    } else {
      if (p.bias) a += __ldg(p.bias + n);
      if (p.add) a += __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.add)[at]);
    }
    reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(a);
  }
}

template <int NB, int STAGES, bool GATE_UP>
cudaError_t launch_typed(const DenseDecodeLaunch& p, int grid, cudaStream_t s) {
  auto kern = dense_decode_kernel<NB, STAGES, GATE_UP>;
  constexpr int smem = smem_bytes<NB, STAGES>();
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(32 * WARPS), smem, s, p);
}

// Blocks of 64 K in flight per warp.  Up to eight tokens four (two blocks per
// SM: 5.8 TB/s on 4096 x 12288), but two where that leaves room for the whole
// grid at once and four does not.  One token, us with two / with four: I of 2400
// to 4704 over H = 1024 6.7 / 8.1, 7.6 / 8.7 (2880), 10.6 / 12.2 (4096), 11.5 / 13.4;
// H of 4800 to 9400 over I = 1024 9.4 / 10.2, 14.4 / 15.7 (7168), 17.5 / 19.4.  Beside
// that range two cost as much or more (I = 1600 6.1 / 5.5).  More tokens need more
// shared memory per stage and keep two blocks per SM.
template <bool GATE_UP>
cudaError_t launch_tokens(const DenseDecodeLaunch& p, cudaStream_t s) {
  const int per = GATE_UP ? 8 : 16, grid = (p.N + per - 1) / per, sms = device_sm_count();
  if (p.T <= 8)
    return grid > 2 * sms && grid <= 4 * sms ? launch_typed<1, 2, GATE_UP>(p, grid, s)
                                             : launch_typed<1, 4, GATE_UP>(p, grid, s);
  if (p.T <= 16) return launch_typed<2, 3, GATE_UP>(p, grid, s);
  return launch_typed<4, 2, GATE_UP>(p, grid, s);
}

}  // namespace

// Measured against the tcgen05 kernels: at 17 to 32 tokens 7.3 us against 9.4 for 2048 x 768 and 12.4 against 11.8 for
// 1536 x 2048, 22.5 against 17.7 for 2880 x 2880 (each weight byte then meets four token tiles); up to 8 tokens it wins
// at every size (4096 x 12288: 51 against 68), from 9 to 16 at most (10.2 against 13.1 for 2048 x 2048, 60 against 57
// to 70 for 4096 x 12288).
bool dense_decode_takes(int32_t T, int32_t H, int32_t I) {
  return T <= 16 || (T <= 32 && static_cast<int64_t>(H) * I <= (int64_t(1) << 21));
}

cudaError_t launch_dense_decode(const DenseDecodeLaunch& p, bool gate_up, cudaStream_t s) {
  return gate_up ? launch_tokens<true>(p, s) : launch_tokens<false>(p, s);
}

}  // namespace e4b
