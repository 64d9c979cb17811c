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
// values are exact there, so only the sum rounds, by less than H 2^-53 of it):
// whatever the order of the sum, rstd is the same fp32 value unless an fp32
// rounding border, 2^-24 apart, falls into that gap, and no more often does an
// 8-bit code next to a border hang on how the row was split over threads.
//
// 8-bit forms.  MX: 32 values share one E8M0 byte, as in the library's MXFP4
// stacks; the exponent is the smallest e with max|y| <= 448 * 2^e, so nothing
// saturates.  Row: one fp32 scale = max|y| / 448 per row.
//
// Backward, with xh = r * rstd and c = mean(dy * w * xh):
//   dx = rstd * (dy * w - xh * c) (+ dr),   dw = sum over rows of dy * xh.
// Its sums are held in fp32: c over the H products of a row, dw over a block's
// rows and then over the blocks, in a fixed order.
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
constexpr int kBackThreads = 512, kBackGroups = 15;   // backward: a block's threads, and its groups (one named barrier each)
constexpr int kSlotBytes = 208 * 1024;                // and the shared memory of its row slots
// From so many rows per SM on, fewer threads take a row of up to 2048 values, one warp up to 1024.  MX output in us, with
// fewer threads / as for few rows: 1200 x 512 2.6 / 2.5, 2400 x 512 3.1 / 3.9, 2400 x 1024 5.6 / 4.9, 8192 x 1024 11.4 / 12.1,
// 1200 x 2048 5.5 / 5.1, 2400 x 2048 7.4 / 8.4, 16384 x 2048 37.6 / 44.9.  Wider rows gain nothing (2400 x 2880 10.1 / 9.9,
// 16384 x 4096 74.3 / 74.0).
constexpr int kManyRowsPerSm = 16;

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

// Two products in one instruction, each rounded as a single one.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 c, a, b;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The larger of m and both magnitudes; a NaN wins (as 0x7FFFFFFF, above infinity when read as an integer).
__device__ __forceinline__ float max_abs2(float m, float2 v) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v.x)));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v.y)));
  return m;
}

// x + residual, each element one exact sum rounded once to bf16.
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&y[i]));
    r[i] = *reinterpret_cast<const uint32_t*>(&s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Adds the eight squares in fp64 (each exact there, whatever its size).
__device__ __forceinline__ double squares8(const uint4& v, double sum) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = pair_of(w[i]);
    sum = fma(static_cast<double>(f.x), static_cast<double>(f.x), sum);
    sum = fma(static_cast<double>(f.y), static_cast<double>(f.y), sum);
  }
  return sum;
}

// y = fl32(fl32(r * rstd) * w) of eight values, and the largest magnitude with m.
__device__ __forceinline__ void normed8(const uint4& r, const uint4& w, float rstd, float2 (&y)[4], float& m) {
  const uint32_t a[4] = {r.x, r.y, r.z, r.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = mul2(mul2(pair_of(a[i]), make_float2(rstd, rstd)), pair_of(b[i]));
    m = max_abs2(m, y[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y));
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

__device__ __forceinline__ uint2 codes8(const float2 (&f)[4]) {
  return make_uint2(e4m3x2(f[0].x, f[0].y) | (static_cast<uint32_t>(e4m3x2(f[1].x, f[1].y)) << 16),
                    e4m3x2(f[2].x, f[2].y) | (static_cast<uint32_t>(e4m3x2(f[3].x, f[3].y)) << 16));
}

// Byte of the 32-value block that four adjacent lanes hold, from each lane's own maximum.
__device__ __forceinline__ uint32_t block_byte(uint32_t m) {
  m = max(m, __shfl_xor_sync(kFull, m, 1));
  m = max(m, __shfl_xor_sync(kFull, m, 2));
  return mx_byte(m);
}

__device__ __forceinline__ uint2 mx_codes(const float2 (&f)[4], uint32_t byte) {
  if (byte == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float s = mx_inverse(byte);
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = mul2(f[j], make_float2(s, s));
  return codes8(v);
}

__device__ __forceinline__ uint2 row_codes(const float2 (&f)[4], float s, uint32_t amax_bits) {
  if (amax_bits >= kInfBits) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  // fl32(f / s) by Markstein's correction of f * RN(1/s), as in the NF4 quantiser; a tiny scale is lifted
  // with its values by 2^96 so that the residual stays normal (quotients that underflow have code 0 anyway)
  const float up = s < 0x1p-60f ? 0x1p96f : 1.0f;
  const float a = s * up, r = __frcp_rn(a);
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = mul2(f[j], make_float2(up, up)), q = mul2(x, make_float2(r, r));
    // (the correction would turn -0 into 0)
    v[j].x = copysignf(fmaf(fmaf(-a, q.x, x.x), r, q.x), x.x);
    v[j].y = copysignf(fmaf(fmaf(-a, q.y, x.y), r, q.y), x.y);
  }
  return codes8(v);
}

// fl32(1 / sqrt(v)): an fp32 estimate refined by two Newton steps in fp64,
// y <- y (1.5 - 0.5 v y^2), which leave a few units of 2^-53; far cheaper per
// thread than the fp64 root and quotient.  Zero, infinite, NaN and very small or
// large v take those.
__device__ __forceinline__ float rstd_of(double sum, double inv_h, double eps) {
  const double v = sum * inv_h + eps;
  if (!(v > 1e-30 && v < 1e30)) return static_cast<float>(1.0 / sqrt(v));
  double y = static_cast<double>(rsqrtf(static_cast<float>(v)));
  const double half = 0.5 * v;
  y = y * fma(-half * y, y, 1.5);
  y = y * fma(-half * y, y, 1.5);
  return static_cast<float>(y);
}

// ---------------------------------------------------------------------- forward

// One block per row, VPT vectors of eight values per thread.
template <int VPT, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_kernel(const NormLaunch p) {
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
    if (p.residual) {
      raw[i] = add8(raw[i], add[i]);
      const int v = i * blockDim.x + threadIdx.x;
      if (p.r_out && v < nvec) reinterpret_cast<uint4*>(p.r_out + row * p.H)[v] = raw[i];
    }
    sum = squares8(raw[i], sum);
  }
  const float rstd = rstd_of(block_sum(sum, red_d), p.inv_h, p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    float2 y[4];
    float big = 0.0f;
    normed8(raw[i], wv[i], rstd, y, big);
    const uint32_t m = v < nvec ? __float_as_uint(big) : 0u;      // outside the row 0 * rstd may be NaN
    if (p.y && v < nvec) reinterpret_cast<uint4*>(p.y + row * p.H)[v] = pack8(y);
    if (p.q_format == E4B_Q8_MX) {
      const uint32_t byte = block_byte(m);
      if (v < nvec) {
        reinterpret_cast<uint2*>(p.q + row * p.H)[v] = mx_codes(y, byte);
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
      float2 y[4];
      float big = 0.0f;
      normed8(raw[i], wv[i], rstd, y, big);
      reinterpret_cast<uint2*>(p.q + row * p.H)[v] = row_codes(y, s, amax);
    }
  }
}

// One warp per row, VPT vectors of eight values per lane: for many rows the
// reduction is five shuffles and no barrier, and the statistics are formed once
// per 8 VPT values of a lane.  The weights come from L1 when they are used.
template <int VPT>
__global__ void __launch_bounds__(128) norm_warp_kernel(const NormLaunch p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= p.T) return;
  const int nvec = p.H >> 3;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.H);
  uint4 raw[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) raw[i] = 32 * i + lane < nvec ? x[32 * i + lane] : make_uint4(0, 0, 0, 0);
  double sum = 0.0;
  if (p.residual) {
    const uint4* res = reinterpret_cast<const uint4*>(p.residual + row * p.H);
    uint4 add[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) add[i] = 32 * i + lane < nvec ? res[32 * i + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      raw[i] = add8(raw[i], add[i]);
      if (p.r_out && 32 * i + lane < nvec) reinterpret_cast<uint4*>(p.r_out + row * p.H)[32 * i + lane] = raw[i];
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) sum = squares8(raw[i], sum);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  const float rstd = rstd_of(sum, p.inv_h, p.eps);
  if (p.rstd && lane == 0) p.rstd[row] = rstd;
  const uint4* weight = reinterpret_cast<const uint4*>(p.weight);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = 32 * i + lane;
    const bool in = v < nvec;
    float2 y[4];
    float big = 0.0f;
    normed8(raw[i], in ? __ldg(weight + v) : make_uint4(0, 0, 0, 0), rstd, y, big);
    const uint32_t m = in ? __float_as_uint(big) : 0u;            // outside the row 0 * rstd may be NaN
    if (p.y && in) reinterpret_cast<uint4*>(p.y + row * p.H)[v] = pack8(y);
    if (p.q_format == E4B_Q8_MX) {
      const uint32_t byte = block_byte(m);
      if (in) {
        reinterpret_cast<uint2*>(p.q + row * p.H)[v] = mx_codes(y, byte);
        if ((v & 3) == 0) static_cast<uint8_t*>(p.q_scales)[row * (p.H >> 5) + (v >> 2)] = static_cast<uint8_t>(byte);
      }
    }
    amax = max(amax, m);
  }
  if (p.q_format == E4B_Q8_ROW) {
    amax = __reduce_max_sync(kFull, amax);
    const float s = row_scale(amax);
    if (lane == 0) static_cast<float*>(p.q_scales)[row] = s;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = 32 * i + lane;
      if (v >= nvec) continue;
      float2 y[4];
      float big = 0.0f;
      normed8(raw[i], __ldg(weight + v), rstd, y, big);
      reinterpret_cast<uint2*>(p.q + row * p.H)[v] = row_codes(y, s, amax);
    }
  }
}

// Any H up to kOddValues per thread of the largest block, any alignment: single
// values, held in registers between the reduction and the output, every load in
// flight before the first use: 5000 rows of 2883 take 25 us, with the loops of
// norm_any_kernel 44.  Two blocks of the largest size per SM: with one, 3451
// rows of 7417 take 75 us instead of 54.
constexpr int kOddValues = 8;
__host__ __device__ constexpr int odd_threads(int H) { return ((H + kOddValues - 1) / kOddValues + 31) / 32 * 32; }

__global__ void __launch_bounds__(1024, 2) norm_odd_kernel(const NormLaunch p) {
  __shared__ double red_d[kMaxWarps];
  __shared__ uint32_t red_u[kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * p.H;
  float r[kOddValues];
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) {
    const int h = threadIdx.x + i * blockDim.x;
    r[i] = h < p.H ? bf16_f32(p.x[at + h]) : 0.0f;
  }
  if (p.residual) {
    float o[kOddValues];
#pragma unroll
    for (int i = 0; i < kOddValues; ++i) {
      const int h = threadIdx.x + i * blockDim.x;
      o[i] = h < p.H ? bf16_f32(p.residual[at + h]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kOddValues; ++i) {
      const int h = threadIdx.x + i * blockDim.x;
      const uint16_t sum = f32_bf16(r[i] + o[i]);
      r[i] = bf16_f32(sum);
      if (p.r_out && h < p.H) p.r_out[at + h] = sum;
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) sum = fma(static_cast<double>(r[i]), static_cast<double>(r[i]), sum);
  const float rstd = rstd_of(block_sum(sum, red_d), p.inv_h, p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[blockIdx.x] = rstd;
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) {
    const int h = threadIdx.x + i * blockDim.x;
    r[i] = h < p.H ? r[i] * rstd * bf16_f32(__ldg(p.weight + h)) : 0.0f;
  }
  if (p.q_format == E4B_Q8_MX) {                         // (H % 32 == 0: a warp's values are one block, or past the row)
#pragma unroll
    for (int i = 0; i < kOddValues; ++i) {
      const int h = threadIdx.x + i * blockDim.x;
      if (h >= p.H) break;
      const uint32_t byte = mx_byte(__reduce_max_sync(kFull, abs_bits(r[i])));
      p.q[at + h] = byte == 255u ? 0x7Fu : static_cast<uint8_t>(e4m3x2(r[i] * mx_inverse(byte), 0.0f) & 0xFFu);
      if ((threadIdx.x & 31) == 0)
        static_cast<uint8_t*>(p.q_scales)[(at + h) >> 5] = static_cast<uint8_t>(byte);
    }
  } else if (p.q_format == E4B_Q8_ROW) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kOddValues; ++i)
      if (threadIdx.x + i * blockDim.x < p.H) amax = max(amax, abs_bits(r[i]));
    amax = block_max(amax, red_u);
    const float scale = row_scale(amax);
    if (threadIdx.x == 0) static_cast<float*>(p.q_scales)[blockIdx.x] = scale;
#pragma unroll
    for (int i = 0; i < kOddValues; ++i) {
      const int h = threadIdx.x + i * blockDim.x;
      if (h < p.H)
        p.q[at + h] = amax >= kInfBits ? 0x7Fu : static_cast<uint8_t>(e4m3x2(__fdiv_rn(r[i], scale), 0.0f) & 0xFFu);
    }
  }
  if (p.y) {
#pragma unroll
    for (int i = 0; i < kOddValues; ++i) {
      const int h = threadIdx.x + i * blockDim.x;
      if (h < p.H) p.y[at + h] = f32_bf16(r[i]);
    }
  }
}

// Wider rows of any alignment: one block per row, single values, the row read
// again after the reduction (from L1 or L2).  A thread touches the same columns
// in every pass, so an output may be the same buffer as an input.
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
    sum = fma(static_cast<double>(r), static_cast<double>(r), sum);
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

// Rows are dealt to groups of `tx` threads, several per block; a thread owns
// VPT vectors of eight columns and keeps their weight gradient in registers over
// all its rows, so dw costs one row of partial sums per block.  One thread of a
// group brings its next STAGES rows into shared memory by bulk copies (whole
// rows are contiguous), which keeps HBM busy whatever the group computes; what a
// row costs beside its values (the waits, the row sum over the group) is paid
// once per 8 VPT values of a thread.
template <typename DY, int VPT, int STAGES>
__global__ void __launch_bounds__(kBackThreads, 1) norm_backward_kernel(const NormBackwardLaunch p, int tx) {
  constexpr int DYV = sizeof(DY) / 2;                   // 16-byte words of dy per vector
  extern __shared__ uint4 slots[];                      // [group][stage][dy row | r row | dr row], then the weights
  __shared__ float red[2][kBackGroups][16];
  __shared__ uint64_t full[kBackGroups][STAGES];
  __shared__ int32_t abort_flag;
  const int nvec = p.H >> 3, g = threadIdx.x / tx, t = threadIdx.x - g * tx, groups = blockDim.x / tx;
  const int nw = tx >> 5, warp = t >> 5, lane = threadIdx.x & 31;
  const int row_words = (DYV + (p.dr ? 2 : 1)) * nvec;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  uint4* mine = slots + static_cast<int64_t>(g) * STAGES * row_words;
  uint4* wsm = slots + static_cast<int64_t>(groups) * STAGES * row_words;
  if (threadIdx.x == 0) {
    for (int i = 0; i < groups; ++i)
      for (int s = 0; s < STAGES; ++s) mbar_init(&full[i][s], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;   // (a wait can only run out seconds later)
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) wsm[v] = __ldg(reinterpret_cast<const uint4*>(p.weight) + v);
  __syncthreads();
  const WaitCtx wctx{&abort_flag, p.status, kWaitLimitNs};
  const uint4* dyp = static_cast<const uint4*>(p.dy);
  const uint4* rp = reinterpret_cast<const uint4*>(p.r);
  const uint4* drp = reinterpret_cast<const uint4*>(p.dr);
  auto fetch = [&](int64_t row, int stage) {            // by the group's first thread
    if (row >= p.T) return;
    uint4* d = mine + stage * row_words;
    mbar_arrive_expect_tx(&full[g][stage], 16u * row_words);
    bulk_load(d, dyp + row * DYV * nvec, 16u * DYV * nvec, &full[g][stage]);
    bulk_load(d + DYV * nvec, rp + row * nvec, 16u * nvec, &full[g][stage]);
    if (drp) bulk_load(d + (DYV + 1) * nvec, drp + row * nvec, 16u * nvec, &full[g][stage]);
  };
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  const float inv_h = static_cast<float>(p.inv_h);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + g;
  if (t == 0)
#pragma unroll
    for (int s = 0; s < STAGES; ++s) fetch(first + s * step, s);
  int buf = 0, stage = 0;
  uint32_t phase = 0;
  bool ok = true;               // after a wait that ran out the thread keeps the group's barriers company, no more
  for (int64_t row = first; row < p.T; row += step) {
    const float rs = __ldg(p.rstd + row);
    ok = ok && mbar_wait(&full[g][stage], phase, wctx, 2101);
    float a[VPT][8], c = 0.0f;
    uint4 rr[VPT];
    const uint4* d = mine + stage * row_words;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tx + t;
      rr[i] = make_uint4(0, 0, 0, 0);
      if (v >= nvec || !ok) break;
      if constexpr (DYV == 2) {
        const uint4 lo = d[2 * v], hi = d[2 * v + 1];
        a[i][0] = __uint_as_float(lo.x); a[i][1] = __uint_as_float(lo.y);
        a[i][2] = __uint_as_float(lo.z); a[i][3] = __uint_as_float(lo.w);
        a[i][4] = __uint_as_float(hi.x); a[i][5] = __uint_as_float(hi.y);
        a[i][6] = __uint_as_float(hi.z); a[i][7] = __uint_as_float(hi.w);
      } else {
        unpack8(d[v], a[i]);
      }
      rr[i] = d[DYV * nvec + v];
      float r[8], w[8];
      unpack8(rr[i], r);
      unpack8(wsm[v], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = r[j] * rs;
        dw[i][j] = fmaf(a[i][j], xh, dw[i][j]);
        a[i][j] *= w[j];
        c = fmaf(a[i][j], xh, c);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(kFull, c, off);
    if (nw > 1) {                                       // the group's warps, through shared memory
      if (lane == 0) red[buf][g][warp] = c;
      asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(tx) : "memory");
      c = red[buf][g][0];
      for (int w = 1; w < nw; ++w) c += red[buf][g][w];
      buf ^= 1;   // a warp may be one row ahead of the slowest reader, never two
    } else {
      __syncwarp();
    }
    // every thread of the group is past the row before: its slot takes the row STAGES after it
    if (STAGES > 1 && t == 0 && ok && row != first)
      fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    const float k = c * inv_h * rs;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tx + t;
      if (v >= nvec || !ok) break;
      float r[8], o[8];
      unpack8(rr[i], r);
      if (drp) {
        unpack8(d[(DYV + 1) * nvec + v], o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(rs, fmaf(-r[j], k, a[i][j]), o[j]);
      reinterpret_cast<uint4*>(p.dx)[row * nvec + v] = pack8(o);
    }
    if constexpr (STAGES == 1) {                        // the only slot: wait for the row's last reader
      asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(tx) : "memory");
      if (t == 0 && ok) fetch(row + step, 0);
    }
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (!ok && t == 0)            // let copies in flight land before the shared memory is used or released
    for (int s = 0; s < STAGES; ++s) mbar_drain(&full[g][s], phase ^ (s < stage ? 1u : 0u), 50000000ull);
  __syncthreads();
  // the groups' weight gradients, added in order
  float4* sum = reinterpret_cast<float4*>(slots);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * tx + t;
    if (v >= nvec) break;
    sum[static_cast<int64_t>(2 * g) * nvec + v] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    sum[static_cast<int64_t>(2 * g + 1) * nvec + v] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
  }
  __syncthreads();
  float4* out = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(blockIdx.x) * p.H);
  for (int v = threadIdx.x; v < 2 * nvec; v += blockDim.x) {
    const int half = v & 1, at = v >> 1;
    float4 s = sum[static_cast<int64_t>(half) * nvec + at];
    for (int h = 1; h < groups; ++h) {
      const float4 o = sum[static_cast<int64_t>(2 * h + half) * nvec + at];
      s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
    }
    out[v] = s;
  }
}

template <typename DY>
__device__ __forceinline__ float load_dy(const void* dy, int64_t i) {
  if constexpr (sizeof(DY) == 4) return static_cast<const float*>(dy)[i];
  else return bf16_f32(static_cast<const uint16_t*>(dy)[i]);
}

// Any H, any alignment.  The weight gradient comes first: dx may be the buffer
// that dy or r is read from.  So dy and r are read twice, by the second launch
// from L2 where they fit, and single values go at half the rate: 5000 x 2883 in fp32 73 us, 5000 x 2880 31.
template <typename DY>
__global__ void __launch_bounds__(128) norm_dw_any_kernel(const NormBackwardLaunch p) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= p.H) return;
  float dw = 0.0f;
  for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y)
    dw = fmaf(load_dy<DY>(p.dy, t * p.H + h), bf16_f32(p.r[t * p.H + h]) * __ldg(p.rstd + t), dw);
  p.partial[static_cast<int64_t>(blockIdx.y) * p.H + h] = dw;
}

template <typename DY>
__global__ void __launch_bounds__(1024, 2) norm_dx_odd_kernel(const NormBackwardLaunch p) {
  __shared__ float red[kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * p.H;
  const float rs = __ldg(p.rstd + blockIdx.x);
  float g[kOddValues], x[kOddValues];
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) {
    const int h = threadIdx.x + i * blockDim.x;
    g[i] = h < p.H ? load_dy<DY>(p.dy, at + h) * bf16_f32(__ldg(p.weight + h)) : 0.0f;
    x[i] = h < p.H ? bf16_f32(p.r[at + h]) * rs : 0.0f;
  }
  float c = 0.0f;
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) c = fmaf(g[i], x[i], c);
  c = block_sum(c, red) * static_cast<float>(p.inv_h);
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) {
    const int h = threadIdx.x + i * blockDim.x;
    if (h < p.H) g[i] = rs * (g[i] - x[i] * c) + (p.dr ? bf16_f32(p.dr[at + h]) : 0.0f);
  }
#pragma unroll
  for (int i = 0; i < kOddValues; ++i) {
    const int h = threadIdx.x + i * blockDim.x;
    if (h < p.H) p.dx[at + h] = f32_bf16(g[i]);
  }
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

// A block per row.  The block counts that go with the kernels keep their registers at what full residency allows.
template <int VPT, int THREADS, int BLOCKS>
cudaError_t launch_rows(const NormLaunch& p, cudaStream_t s) {
  return launch_pdl(norm_kernel<VPT, THREADS, BLOCKS>, dim3(p.T), dim3(threads_for(p.H, VPT)), 0, s, p);
}

template <typename DY, int VPT, int STAGES>
cudaError_t launch_backward_vec(const NormBackwardLaunch& p, int blocks, cudaStream_t s) {
  auto kern = norm_backward_kernel<DY, VPT, STAGES>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, kSlotBytes, allowed);
  if (e != cudaSuccess) return e;
  // as many groups as threads, barriers and shared memory allow; their weight gradients (4 H bytes each) reuse
  // the slots, which are never smaller
  const int tx = threads_for(p.H, VPT), group = STAGES * (static_cast<int>(sizeof(DY)) + (p.dr ? 4 : 2)) * p.H;
  int groups = kBackThreads / tx;
  if (groups > (kSlotBytes - 2 * p.H) / group) groups = (kSlotBytes - 2 * p.H) / group;
  if (groups > kBackGroups) groups = kBackGroups;
  return launch_pdl(kern, dim3(blocks), dim3(groups * tx), groups * group + 2 * p.H, s, p, tx);
}

// Two rows ahead where two rows of one group fit in shared memory, one for the
// widest; narrow rows (one or two vectors per thread) four.
template <typename DY>
cudaError_t launch_backward_typed(const NormBackwardLaunch& p, bool vec, cudaStream_t s) {
  const int blocks = norm_backward_blocks(p.T);
  const int64_t row = static_cast<int64_t>(static_cast<int>(sizeof(DY)) + (p.dr ? 4 : 2)) * p.H;
  cudaError_t e;
  if (vec && p.H <= 16384) {
    if (p.H <= 256) e = launch_backward_vec<DY, 1, 4>(p, blocks, s);
    else if (p.H <= 512) e = launch_backward_vec<DY, 2, 4>(p, blocks, s);
    else if (2 * row + 2 * p.H <= kSlotBytes) e = launch_backward_vec<DY, 4, 2>(p, blocks, s);
    else e = launch_backward_vec<DY, 4, 1>(p, blocks, s);
  } else {
    e = launch_pdl(norm_dw_any_kernel<DY>, dim3((p.H + 127) / 128, blocks), dim3(128), 0, s, p);
    if (e == cudaSuccess)
      e = odd_threads(p.H) <= 1024 ? launch_pdl(norm_dx_odd_kernel<DY>, dim3(p.T), dim3(odd_threads(p.H)), 0, s, p)
                                   : launch_pdl(norm_dx_any_kernel<DY>, dim3(p.T), dim3(256), 0, s, p);
  }
  if (e != cudaSuccess) return e;
  return launch_column_sum(p.partial, blocks, p.H, p.dweight, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormLaunch& p, cudaStream_t s) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.residual) |
                      reinterpret_cast<uintptr_t>(p.weight) | reinterpret_cast<uintptr_t>(p.r_out) |
                      reinterpret_cast<uintptr_t>(p.y) | (2 * reinterpret_cast<uintptr_t>(p.q));
  if (p.H % 8 != 0 || a % 16 != 0 || p.H > 32768) {
    if (odd_threads(p.H) <= 1024) return launch_pdl(norm_odd_kernel, dim3(p.T), dim3(odd_threads(p.H)), 0, s, p);
    return launch_pdl(norm_any_kernel, dim3(p.T), dim3(256), 0, s, p);
  }
  if (p.T >= kManyRowsPerSm * device_sm_count() && p.H <= 2048) {
    if (p.H <= 1024) {
      const dim3 grid((p.T + 3) / 4), block(128);
      if (p.H <= 256) return launch_pdl(norm_warp_kernel<1>, grid, block, 0, s, p);
      if (p.H <= 512) return launch_pdl(norm_warp_kernel<2>, grid, block, 0, s, p);
      return launch_pdl(norm_warp_kernel<4>, grid, block, 0, s, p);
    }
    return launch_rows<2, 128, 12>(p, s);
  }
  if (p.H <= 2048) return launch_rows<1, 256, 8>(p, s);
  if (p.H <= 8192) return launch_rows<2, 512, 3>(p, s);
  return launch_rows<4, 1024, 1>(p, s);
}

// One row of partial weight gradients per block: one block per SM, fewer for few rows.
int norm_backward_blocks(int32_t T) {
  const int most = device_sm_count();
  return T < most ? (T > 0 ? T : 1) : most;
}

cudaError_t launch_rmsnorm_backward(const NormBackwardLaunch& p, cudaStream_t s) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p.dy) | reinterpret_cast<uintptr_t>(p.r) |
                reinterpret_cast<uintptr_t>(p.dr) | reinterpret_cast<uintptr_t>(p.weight) |
                reinterpret_cast<uintptr_t>(p.dx);
  const bool vec = p.H % 8 == 0 && a % 16 == 0;
  return p.dy_f32 ? launch_backward_typed<float>(p, vec, s) : launch_backward_typed<uint16_t>(p, vec, s);
}

}  // namespace e4b
