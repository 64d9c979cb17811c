// Root-mean-square norm of the hidden stream around the routed layer, with the
// residual's addition in the same pass, a bf16 or an 8-bit output, and its
// backward.
//
// Forward, per row of H values:
//   r    = bf16(x + residual)          (r = x without a residual)
//   rstd = fl32(1 / sqrt(mean(r^2) + eps))      mean, root and quotient in fp64
//   y    = fl32(fl32(r * rstd) * w)    -> bf16, or e4m3 with scales
// What is normed is the rounded r: it is the stream that the next block and
// the backward see.  The statistics are held in fp64 (the squares of bf16
// values are exact in fp32, so only the sum rounds): rstd is then the same
// fp32 value for every summation order, and an 8-bit code next to a rounding
// border does not depend on how the row was split over threads.
//
// 8-bit forms.  MX: 32 values share one E8M0 byte, as in the library's MXFP4
// stacks; the exponent is the smallest e with max|y| <= 448 * 2^e, so nothing
// saturates.  Row: one fp32 scale = max|y| / 448 per row.
//
// Backward, with xh = r * rstd and c = mean(dy * w * xh):
//   dx = rstd * (dy * w - xh * c) (+ dr),   dw = sum over rows of dy * xh.
//
// Both passes only stream rows: they are bound by HBM.  A row stays in
// registers between the reduction and the output, so every input is read once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kMaxWarps = 32;

__device__ __forceinline__ float bf16_f32(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ uint16_t f32_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  return static_cast<uint16_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

// Sums over the block, the same value in every thread; the order is fixed by
// the thread layout.  `red` holds one slot per warp and may be reused after
// the next barrier that every thread passes.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = red[0];
  for (int w = 1; w < nw; ++w) t += red[w];
  return t;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(kFull, v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t t = red[0];
  for (int w = 1; w < nw; ++w) t = max(t, red[w]);
  return t;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

constexpr uint32_t kInfBits = 0x7F800000u;   // abs_bits at or above: infinity or NaN

// Row scale of an 8-bit row from the largest |y| (as bits, so that a NaN or an
// infinity wins the maximum).  Bounded below so that a row of tiny values
// still divides to finite codes; NaN marks a row that is not finite.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  if (amax_bits >= kInfBits) return __uint_as_float(0x7FC00000u);
  return fmaxf(__fdiv_rn(__uint_as_float(amax_bits), 448.0f), 0x1p-126f);
}

// E8M0 byte of a block: the smallest e with amax <= 448 * 2^e, 448 = 1.75 * 2^8,
// biased by 127 and not below 0; 255 (NaN) for a block that is not finite.
__device__ __forceinline__ uint32_t mx_byte(uint32_t amax_bits) {
  if (amax_bits >= kInfBits) return 255u;
  if (amax_bits == 0u) return 0u;
  const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));   // (a subnormal amax has exponent field 0 and ends at byte 0)
}

// 2^(127 - byte) as fp32, exact (a finite block's byte is at most 247).
__device__ __forceinline__ float mx_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ float rstd_of(double sum, double inv_h, double eps) {
  return static_cast<float>(1.0 / sqrt(sum * inv_h + eps));
}

// ---------------------------------------------------------------------- forward

// One block per row, VPT vectors of eight values per thread.
template <int VPT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormLaunch p) {
  __shared__ double red_d[kMaxWarps];
  __shared__ uint32_t red_u[kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const int nvec = p.H >> 3;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.H);
  const uint4* res = reinterpret_cast<const uint4*>(p.residual + row * p.H);
  uint4 raw[VPT], add[VPT], wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    const bool in = v < nvec;
    raw[i] = in ? x[v] : make_uint4(0, 0, 0, 0);
    add[i] = in && p.residual ? res[v] : make_uint4(0, 0, 0, 0);
    wv[i] = in ? __ldg(reinterpret_cast<const uint4*>(p.weight) + v) : make_uint4(0, 0, 0, 0);
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[8];
    unpack8(raw[i], f);
    if (p.residual) {
      float a[8];
      unpack8(add[i], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += a[j];
      raw[i] = pack8(f);
      const int v = i * blockDim.x + threadIdx.x;
      if (p.r_out && v < nvec) reinterpret_cast<uint4*>(p.r_out + row * p.H)[v] = raw[i];
      unpack8(raw[i], f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += static_cast<double>(f[j] * f[j]);
  }
  const float rstd = rstd_of(block_sum(sum, red_d), p.inv_h, p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    float f[8], w[8];
    unpack8(raw[i], f);
    unpack8(wv[i], w);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = f[j] * rstd * w[j];
      if (v < nvec) m = max(m, abs_bits(f[j]));   // outside the row 0 * rstd may be NaN
    }
    if (p.y && v < nvec) reinterpret_cast<uint4*>(p.y + row * p.H)[v] = pack8(f);
    if (p.q_format == E4B_Q8_MX) {   // the four lanes of one 32-value block
      m = max(m, __shfl_xor_sync(kFull, m, 1));
      m = max(m, __shfl_xor_sync(kFull, m, 2));
      const uint32_t byte = mx_byte(m);
      const float s = mx_inverse(byte);
      uint2 q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      if (byte != 255u)
        q = make_uint2(e4m3x2(f[0] * s, f[1] * s) | (static_cast<uint32_t>(e4m3x2(f[2] * s, f[3] * s)) << 16),
                       e4m3x2(f[4] * s, f[5] * s) | (static_cast<uint32_t>(e4m3x2(f[6] * s, f[7] * s)) << 16));
      if (v < nvec) {
        reinterpret_cast<uint2*>(p.q + row * p.H)[v] = q;
        if ((v & 3) == 0) static_cast<uint8_t*>(p.q_scales)[row * (p.H >> 5) + (v >> 2)] = static_cast<uint8_t>(byte);
      }
    }
    amax = max(amax, m);
  }
  if (p.q_format == E4B_Q8_ROW) {
    amax = block_max(amax, red_u);
    const float s = row_scale(amax);
    if (threadIdx.x == 0) static_cast<float*>(p.q_scales)[row] = s;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v >= nvec) continue;
      float f[8], w[8];
      unpack8(raw[i], f);
      unpack8(wv[i], w);
      uint2 q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      if (amax < kInfBits) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j] * rstd * w[j], s);
        q = make_uint2(e4m3x2(f[0], f[1]) | (static_cast<uint32_t>(e4m3x2(f[2], f[3])) << 16),
                       e4m3x2(f[4], f[5]) | (static_cast<uint32_t>(e4m3x2(f[6], f[7])) << 16));
      }
      reinterpret_cast<uint2*>(p.q + row * p.H)[v] = q;
    }
  }
}

// Any H, any alignment: one block per row, single values, the row read again
// after the reduction (from L1 or L2).  A thread touches the same columns in
// every pass, so an output may be the same buffer as an input.
__global__ void __launch_bounds__(256) norm_any_kernel(const NormLaunch p) {
  __shared__ double red_d[kMaxWarps];
  __shared__ uint32_t red_u[kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * p.H;
  auto stream_value = [&](int h) -> float {
    if (!p.residual) return bf16_f32(p.x[at + h]);
    return bf16_f32(f32_bf16(bf16_f32(p.x[at + h]) + bf16_f32(p.residual[at + h])));
  };
  double sum = 0.0;
  for (int h = threadIdx.x; h < p.H; h += blockDim.x) {
    const float r = stream_value(h);
    if (p.residual && p.r_out) p.r_out[at + h] = static_cast<uint16_t>(__float_as_uint(r) >> 16);
    sum += static_cast<double>(r * r);
  }
  const float rstd = rstd_of(block_sum(sum, red_d), p.inv_h, p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[blockIdx.x] = rstd;
  // after the first pass the stream is in r_out where there is one: x or residual may be the same buffer
  const bool kept = p.residual && p.r_out;
  auto y_of = [&](int h) -> float {
    const float r = kept ? bf16_f32(p.r_out[at + h]) : stream_value(h);
    return r * rstd * bf16_f32(__ldg(p.weight + h));
  };
  if (p.q_format == E4B_Q8_MX) {
    for (int h0 = (threadIdx.x >> 5) * 32; h0 < p.H; h0 += blockDim.x) {   // one warp per 32-value block
      const int h = h0 + (threadIdx.x & 31);
      const float y = y_of(h);
      const uint32_t byte = mx_byte(__reduce_max_sync(kFull, abs_bits(y)));
      p.q[at + h] = byte == 255u ? 0x7Fu : static_cast<uint8_t>(e4m3x2(y * mx_inverse(byte), 0.0f) & 0xFFu);
      if ((threadIdx.x & 31) == 0)
        static_cast<uint8_t*>(p.q_scales)[(at + h) >> 5] = static_cast<uint8_t>(byte);
    }
  } else if (p.q_format == E4B_Q8_ROW) {
    uint32_t amax = 0;
    for (int h = threadIdx.x; h < p.H; h += blockDim.x) amax = max(amax, abs_bits(y_of(h)));
    amax = block_max(amax, red_u);
    const float s = row_scale(amax);
    if (threadIdx.x == 0) static_cast<float*>(p.q_scales)[blockIdx.x] = s;
    for (int h = threadIdx.x; h < p.H; h += blockDim.x)
      p.q[at + h] = amax >= kInfBits ? 0x7Fu : static_cast<uint8_t>(e4m3x2(__fdiv_rn(y_of(h), s), 0.0f) & 0xFFu);
  }
  if (p.y)
    for (int h = threadIdx.x; h < p.H; h += blockDim.x) p.y[at + h] = f32_bf16(y_of(h));
}

// ---------------------------------------------------------------------- backward

template <typename DY>
__device__ __forceinline__ void load_dy8(const void* dy, int64_t vec, float (&f)[8]) {
  if constexpr (sizeof(DY) == 4) {
    const float4* p = static_cast<const float4*>(dy) + 2 * vec;
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(static_cast<const uint4*>(dy)[vec], f);
  }
}

// Blocks walk groups of ROWS rows; a thread owns VPT vectors of eight columns
// and keeps their weight gradient in registers over all its rows, so dw costs
// one row of partial sums per block.  ROWS rows are loaded together and share
// one reduction: that many times the bytes in flight per barrier.
template <typename DY, int VPT, int ROWS>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackwardLaunch p) {
  __shared__ float red[2][ROWS][16];
  pdl_wait();
  pdl_launch_dependents();
  const int nvec = p.H >> 3, nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float dw[VPT][8];
  uint4 wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    wv[i] = v < nvec ? __ldg(reinterpret_cast<const uint4*>(p.weight) + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  const float inv_h = static_cast<float>(p.inv_h);
  int buf = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * ROWS; r0 < p.T; r0 += static_cast<int64_t>(gridDim.x) * ROWS) {
    float dy[ROWS][VPT][8];
    uint4 rr[ROWS][VPT], dr[ROWS][VPT];
    float rs[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const bool row_in = r0 + k < p.T;
      rs[k] = row_in ? __ldg(p.rstd + r0 + k) : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        const int64_t vec = (r0 + k) * nvec + v;
        rr[k][i] = dr[k][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dy[k][i][j] = 0.0f;
        if (row_in && v < nvec) {
          load_dy8<DY>(p.dy, vec, dy[k][i]);
          rr[k][i] = reinterpret_cast<const uint4*>(p.r)[vec];
          if (p.dr) dr[k][i] = reinterpret_cast<const uint4*>(p.dr)[vec];
        }
      }
    }
    float c[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      c[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float r[8], w[8];
        unpack8(rr[k][i], r);
        unpack8(wv[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = r[j] * rs[k];
          dw[i][j] = fmaf(dy[k][i][j], xh, dw[i][j]);
          c[k] = fmaf(dy[k][i][j] * w[j], xh, c[k]);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) c[k] += __shfl_xor_sync(kFull, c[k], off);
      if (lane == 0) red[buf][k][warp] = c[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      float s = red[buf][k][0];
      for (int w = 1; w < nw; ++w) s += red[buf][k][w];
      s *= inv_h;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (r0 + k >= p.T || v >= nvec) continue;
        float r[8], w[8], d[8];
        unpack8(rr[k][i], r);
        unpack8(wv[i], w);
        unpack8(dr[k][i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += rs[k] * (dy[k][i][j] * w[j] - r[j] * rs[k] * s);
        reinterpret_cast<uint4*>(p.dx)[(r0 + k) * nvec + v] = pack8(d);
      }
    }
    buf ^= 1;   // a warp may be one group ahead of the slowest reader, never two
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v >= nvec) continue;
    float4* o = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(blockIdx.x) * p.H) + 2 * v;
    o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
  }
}

template <typename DY>
__device__ __forceinline__ float load_dy(const void* dy, int64_t i) {
  if constexpr (sizeof(DY) == 4) return static_cast<const float*>(dy)[i];
  else return bf16_f32(static_cast<const uint16_t*>(dy)[i]);
}

// Any H, any alignment.  The weight gradient comes first: dx may be the buffer
// that dy or r is read from.
template <typename DY>
__global__ void __launch_bounds__(128) norm_dw_any_kernel(const NormBackwardLaunch p) {
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= p.H) return;
  float dw = 0.0f;
  for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y)
    dw = fmaf(load_dy<DY>(p.dy, t * p.H + h), bf16_f32(p.r[t * p.H + h]) * __ldg(p.rstd + t), dw);
  p.partial[static_cast<int64_t>(blockIdx.y) * p.H + h] = dw;
}

template <typename DY>
__global__ void __launch_bounds__(256) norm_dx_any_kernel(const NormBackwardLaunch p) {
  __shared__ float red[kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * p.H;
  const float rs = __ldg(p.rstd + blockIdx.x);
  float c = 0.0f;
  for (int h = threadIdx.x; h < p.H; h += blockDim.x)
    c = fmaf(load_dy<DY>(p.dy, at + h) * bf16_f32(__ldg(p.weight + h)), bf16_f32(p.r[at + h]) * rs, c);
  c = block_sum(c, red) * static_cast<float>(p.inv_h);
  for (int h = threadIdx.x; h < p.H; h += blockDim.x) {
    float d = rs * (load_dy<DY>(p.dy, at + h) * bf16_f32(__ldg(p.weight + h)) - bf16_f32(p.r[at + h]) * rs * c);
    if (p.dr) d += bf16_f32(p.dr[at + h]);
    p.dx[at + h] = f32_bf16(d);
  }
}

// Smallest block of whole warps whose threads hold the row in VPT vectors each.
int threads_for(int H, int vpt) {
  const int nvec = (H + 7) / 8;
  return ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
}

template <typename DY>
cudaError_t launch_backward_typed(NormBackwardLaunch p, bool vec, cudaStream_t s) {
  const int blocks = norm_backward_blocks(p.T);
  cudaError_t e;
  if (vec && p.H <= 16384) {
    if (p.H <= 4096)
      e = launch_pdl(norm_backward_kernel<DY, 1, 4>, dim3(blocks), dim3(threads_for(p.H, 1)), 0, s, p);
    else if (p.H <= 8192)
      e = launch_pdl(norm_backward_kernel<DY, 2, 2>, dim3(blocks), dim3(threads_for(p.H, 2)), 0, s, p);
    else
      e = launch_pdl(norm_backward_kernel<DY, 4, 1>, dim3(blocks), dim3(threads_for(p.H, 4)), 0, s, p);
  } else {
    e = launch_pdl(norm_dw_any_kernel<DY>, dim3((p.H + 127) / 128, blocks), dim3(128), 0, s, p);
    if (e == cudaSuccess) e = launch_pdl(norm_dx_any_kernel<DY>, dim3(p.T), dim3(256), 0, s, p);
  }
  if (e != cudaSuccess) return e;
  return launch_column_sum(p.partial, blocks, p.H, p.dweight, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormLaunch& p, cudaStream_t s) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.residual) |
                      reinterpret_cast<uintptr_t>(p.weight) | reinterpret_cast<uintptr_t>(p.r_out) |
                      reinterpret_cast<uintptr_t>(p.y) | (2 * reinterpret_cast<uintptr_t>(p.q));
  if (p.H % 8 != 0 || a % 16 != 0 || p.H > 32768)
    return launch_pdl(norm_any_kernel, dim3(p.T), dim3(256), 0, s, p);
  if (p.H <= 2048) return launch_pdl(norm_kernel<1>, dim3(p.T), dim3(threads_for(p.H, 1)), 0, s, p);
  if (p.H <= 8192) return launch_pdl(norm_kernel<2>, dim3(p.T), dim3(threads_for(p.H, 2)), 0, s, p);
  return launch_pdl(norm_kernel<4>, dim3(p.T), dim3(threads_for(p.H, 4)), 0, s, p);
}

// One row of partial weight gradients per block: one block per SM, fewer for few rows.
int norm_backward_blocks(int32_t T) {
  const int rows = (T + 3) / 4, sms = device_sm_count();
  return rows < sms ? (rows > 0 ? rows : 1) : sms;
}

cudaError_t launch_rmsnorm_backward(const NormBackwardLaunch& p, cudaStream_t s) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p.dy) | reinterpret_cast<uintptr_t>(p.r) |
                reinterpret_cast<uintptr_t>(p.dr) | reinterpret_cast<uintptr_t>(p.weight) |
                reinterpret_cast<uintptr_t>(p.dx);
  const bool vec = p.H % 8 == 0 && a % 16 == 0;
  return p.dy_f32 ? launch_backward_typed<float>(p, vec, s) : launch_backward_typed<uint16_t>(p, vec, s);
}

}  // namespace e4b
