// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over all tensors of sum g^2),
//   c    = min(1, max_norm / (norm + 1e-6)),   out = g * c.
//
// Two launches for any number of tensors up to kMaxTable (their table travels
// as a kernel argument, so nothing is copied to the device and a captured
// graph holds it): the first leaves one fp64 partial sum per block, the second
// adds those in every block, in the same order, and scales.  No atomics and no
// counters: the norm has the same bits for the same tensors, and the workspace
// needs no clearing.  Squares are formed and summed in fp64, so values whose
// square leaves the fp32 range still count (a gradient of 1e25, or of 1e-30).
//
// (A list of more than kMaxTable tensors takes several launches of each kind and
// one that sums the partials once for all the scaling blocks.)
//
// Both passes are bound by HBM; the second starts where the first ended, so that
// what was read last is still in L2.  In long lists a chunk is 32 KB, eight
// 16-byte loads per thread, and the scaling pass gives each a block of its own:
// 96 tensors, 705 MB, in 317 us (with eight blocks per SM that walk their chunks
// 343: the blocks drift apart, and what is in L2 is gone before its turn).  In
// short lists a chunk is 16 KB for the norm and 8 KB for scaling, whose blocks
// need fewer registers with it: 401 ragged tensors, 92 MB, in 47 us (51 with 16 KB).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kSmall = 64, kMedium = 384, kMaxTable = 960;   // 2, 12 and 30 KB of kernel arguments
constexpr int kBlocksPerSm = 8;
constexpr int kNormWords = 4, kScaleWords = 2, kLongWords = 8;   // 16-byte words per thread and chunk
constexpr size_t kLongBytes = size_t(160) << 20;   // a launch's tensors from which on chunks are long and strided

// One tensor of the table.  Its 16-byte words start at the boundary at or
// below the first element; `skip` elements of the first word are not its own.
struct ClipEntry {
  const void* in;
  void* out;
  int64_t n;
  int32_t chunk0;       // first chunk of this tensor among the launch's chunks
  int16_t type;
  int8_t skip;
  int8_t words;         // 1: `in` and `out` have the same offset from a 16-byte boundary
};

template <int N>
struct ClipTable {
  int32_t tensors, chunks;
  ClipEntry e[N];
};

template <int TYPE>
__host__ __device__ constexpr int size_of() { return TYPE == E4B_F32 ? 4 : 2; }

// The last tensor whose first chunk is at or before this one: by bisection in the
// argument bank, where a block's threads agree on every step.  (A copy of the
// table's chunks in shared memory cost each block more than its searches: 900
// tensors of 1 MB took 460 us against 423.)
template <int N>
__device__ __forceinline__ int tensor_of(const ClipTable<N>& t, int chunk) {
  int lo = 0, hi = t.tensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].chunk0 <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// Walks a block's chunks, calling body(entry, chunk).  LONG lists: strided over
// the whole list, so that the blocks move through memory together, the tensor
// found anew for each chunk.  Short lists, mostly of small tensors: one
// contiguous run, whose next chunk lies in the same tensor or the one beside it.
// REVERSED: from the last block's last chunk to the first's first.
template <int N, bool LONG, bool REVERSED, typename Body>
__device__ __forceinline__ void walk_chunks(const ClipTable<N>& t, const Body& body) {
  const int n = gridDim.x, b = REVERSED ? n - 1 - static_cast<int>(blockIdx.x) : blockIdx.x;
  if constexpr (LONG) {
    const int count = b < t.chunks ? (t.chunks - 1 - b) / n + 1 : 0;
    for (int i = 0; i < count; ++i) {
      const int c = b + (REVERSED ? count - 1 - i : i) * n;
      body(t.e[tensor_of(t, c)], c);
    }
  } else {
    const int c0 = static_cast<int>(static_cast<int64_t>(t.chunks) * b / n);
    const int c1 = static_cast<int>(static_cast<int64_t>(t.chunks) * (b + 1) / n);
    if (c0 == c1) return;
    int ti = tensor_of(t, REVERSED ? c1 - 1 : c0);
    for (int i = 0; i < c1 - c0; ++i) {
      const int c = REVERSED ? c1 - 1 - i : c0 + i;
      if constexpr (REVERSED) {
        while (t.e[ti].chunk0 > c) --ti;
      } else {
        while (ti + 1 < t.tensors && t.e[ti + 1].chunk0 <= c) ++ti;
      }
      body(t.e[ti], c);
    }
  }
}

// The elements of one 16-byte word as fp32.
template <int TYPE>
__device__ __forceinline__ void word_values(const uint4& v, float (&f)[16 / size_of<TYPE>()]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == E4B_F32) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (TYPE == E4B_BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ uint32_t two_halves(float lo, float hi) {
  if constexpr (TYPE == E4B_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <int TYPE>
__device__ __forceinline__ uint4 scaled_word(const uint4& v, float c) {
  float f[16 / size_of<TYPE>()];
  word_values<TYPE>(v, f);
  if constexpr (TYPE == E4B_F32)
    return make_uint4(__float_as_uint(f[0] * c), __float_as_uint(f[1] * c), __float_as_uint(f[2] * c),
                      __float_as_uint(f[3] * c));
  else
    return make_uint4(two_halves<TYPE>(f[0] * c, f[1] * c), two_halves<TYPE>(f[2] * c, f[3] * c),
                      two_halves<TYPE>(f[4] * c, f[5] * c), two_halves<TYPE>(f[6] * c, f[7] * c));
}

template <int TYPE>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (TYPE == E4B_F32) return static_cast<const float*>(p)[i];
  else if constexpr (TYPE == E4B_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return __half2float(static_cast<const __half*>(p)[i]);
}

template <int TYPE>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (TYPE == E4B_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (TYPE == E4B_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Calls word(i) for this thread's words of the chunk that lie wholly inside the
// tensor and one(k) for the single elements of its first and last word, each
// by another thread.  A chunk in the tensor's middle is only whole words and
// takes no tests.
template <int TYPE, int V, typename Word, typename One>
__device__ __forceinline__ void for_chunk(const ClipEntry& e, int64_t w0, const Word& word, const One& one) {
  constexpr int PER = 16 / size_of<TYPE>();
  const int64_t last = e.n + e.skip;                      // elements counted from the first word's start
  const int64_t c0 = w0 - threadIdx.x;
  const uint4* in = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(e.in) - e.skip * size_of<TYPE>()) + w0;
  if (c0 * PER >= e.skip && (c0 + V * kThreads) * PER <= last) {
    uint4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = in[i * kThreads];
#pragma unroll
    for (int i = 0; i < V; ++i) word(w0 + i * kThreads, v[i]);
    return;
  }
  const int64_t begin = (e.skip + PER - 1) / PER, end = last / PER;   // the whole words
  const int64_t head = begin * PER - e.skip;              // elements before them
  if (c0 == 0 && threadIdx.x < head && threadIdx.x < e.n) one(threadIdx.x);
  if (end >= begin && c0 <= end && end < c0 + V * kThreads) {
    const int64_t k = end * PER - e.skip + static_cast<int>(kThreads - 1 - threadIdx.x);
    if (k < e.n) one(k);
  }
  const int64_t stop = end < c0 + V * kThreads ? end : c0 + V * kThreads;
#pragma unroll 2
  for (int64_t w = w0 < begin ? w0 + kThreads : w0; w < stop; w += kThreads) word(w, in[w - w0]);
}

template <int TYPE, int V>
__device__ __forceinline__ double chunk_squares(const ClipEntry& e, int64_t w0) {
  double sum = 0.0;
  for_chunk<TYPE, V>(
      e, w0,
      [&](int64_t, const uint4& v) {
        float f[16 / size_of<TYPE>()];
        word_values<TYPE>(v, f);
#pragma unroll
        for (int j = 0; j < 16 / size_of<TYPE>(); ++j)
          sum = fma(static_cast<double>(f[j]), static_cast<double>(f[j]), sum);
      },
      [&](int64_t k) {
        const double g = load_one<TYPE>(e.in, k);
        sum = fma(g, g, sum);
      });
  return sum;
}

template <int TYPE, int V>
__device__ __forceinline__ void chunk_scale(const ClipEntry& e, int64_t w0, float c) {
  constexpr int PER = 16 / size_of<TYPE>();
  uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(e.out) - e.skip * size_of<TYPE>());
  for_chunk<TYPE, V>(
      e, w0,
      [&](int64_t w, const uint4& v) {
        if (e.words) {
          __stcs(out + w, scaled_word<TYPE>(v, c));
        } else {
          float f[PER];
          word_values<TYPE>(v, f);
#pragma unroll
          for (int j = 0; j < PER; ++j) store_one<TYPE>(e.out, w * PER + j - e.skip, f[j] * c);
        }
      },
      [&](int64_t k) { store_one<TYPE>(e.out, k, load_one<TYPE>(e.in, k) * c); });
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) t += red[w];
  return t;
}

template <int N, bool LONG>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ ClipTable<N> t,
                                                             double* __restrict__ partial) {
  __shared__ double red[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int V = LONG ? kLongWords : kNormWords;
  double sum = 0.0;
  walk_chunks<N, LONG, false>(t, [&](const ClipEntry& e, int c) {
    const int64_t w0 = static_cast<int64_t>(c - e.chunk0) * (V * kThreads) + threadIdx.x;
    if (e.type == E4B_F32) sum += chunk_squares<E4B_F32, V>(e, w0);
    else if (e.type == E4B_BF16) sum += chunk_squares<E4B_BF16, V>(e, w0);
    else sum += chunk_squares<E4B_F16, V>(e, w0);
  });
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// max_norm is +infinity where only the norm is wanted.
template <int N, bool LONG>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ ClipTable<N> t,
                                                              const double* __restrict__ partial, int partials,
                                                              double max_norm, float* __restrict__ total_norm) {
  __shared__ double red[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int V = LONG ? kLongWords : kScaleWords;
  double sum = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  const double norm = sqrt(block_sum(sum, red));
  if (total_norm && blockIdx.x == 0 && threadIdx.x == 0) *total_norm = static_cast<float>(norm);
  const double ratio = max_norm / (norm + 1e-6);
  const float coef = isinf(max_norm) || ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);   // a NaN norm gives NaN
  walk_chunks<N, LONG, true>(t, [&](const ClipEntry& e, int c) {
    if (e.in == e.out && coef == 1.0f) return;            // in place and unclipped: already there
    const int64_t w0 = static_cast<int64_t>(c - e.chunk0) * (V * kThreads) + threadIdx.x;
    if (e.type == E4B_F32) chunk_scale<E4B_F32, V>(e, w0, coef);
    else if (e.type == E4B_BF16) chunk_scale<E4B_BF16, V>(e, w0, coef);
    else chunk_scale<E4B_F16, V>(e, w0, coef);
  });
}

// One sum of many partials, for the blocks of several scale launches.
__global__ void __launch_bounds__(kThreads) grad_sum_kernel(double* __restrict__ partial, int partials) {
  __shared__ double red[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) partial[0] = sum;
}

template <int N>
void fill_table(ClipTable<N>& t, const e4b_grad* g, int count, int words) {
  const int64_t chunk_bytes = 16 * kThreads * words;
  t.tensors = count;
  int64_t chunk = 0;
  for (int i = 0; i < count; ++i) {
    ClipEntry& e = t.e[i];
    const int size = g[i].dtype == E4B_F32 ? 4 : 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].grad);
    e.in = g[i].grad;
    e.out = g[i].out;
    e.n = g[i].n;
    e.type = static_cast<int16_t>(g[i].dtype);
    e.skip = static_cast<int8_t>((a % 16) / size);
    e.words = reinterpret_cast<uintptr_t>(g[i].out) % 16 == a % 16;
    e.chunk0 = static_cast<int32_t>(chunk);
    if (e.n > 0) chunk += ((e.n + e.skip) * size + chunk_bytes - 1) / chunk_bytes;
  }
  t.chunks = static_cast<int32_t>(chunk);
}

int at_least_one(int64_t chunks, int64_t cap) { return static_cast<int>(chunks < cap ? (chunks > 0 ? chunks : 1) : cap); }

// One partial sum per block, so a bounded number of them.
int norm_blocks(int chunks) { return at_least_one(chunks, int64_t(device_sm_count()) * kBlocksPerSm); }

// In short lists a block sums the partials once for several chunks: 16 blocks per
// SM where each still has four (47 us for the 401 tensors, 49 with 8), else 8
// (9.5 us for 15 MB, 9.8 with 16).
int scale_blocks(int chunks, bool is_long) {
  const int64_t sms = device_sm_count();
  return is_long ? at_least_one(chunks, chunks) : at_least_one(chunks, chunks >= 64 * sms ? 16 * sms : 8 * sms);
}

// Both kernels for `count` tensors; partial and the count of what is in it move on with the norm pass.
struct ClipRun {
  const e4b_grad* g;
  int count;
  bool is_long;
  cudaStream_t s;

  template <int N, bool LONG>
  cudaError_t norm(double* partial, int* blocks) const {
    ClipTable<N> t;
    fill_table(t, g, count, LONG ? kLongWords : kNormWords);
    *blocks = norm_blocks(t.chunks);
    void* args[] = {&t, &partial};
    return launch_pdl_args(reinterpret_cast<const void*>(grad_norm_kernel<N, LONG>), dim3(*blocks), dim3(kThreads), s, args);
  }
  template <int N, bool LONG>
  cudaError_t scale(const double* partial, int partials, double max_norm, float* total_norm) const {
    ClipTable<N> t;
    fill_table(t, g, count, LONG ? kLongWords : kScaleWords);
    void* args[] = {&t, &partial, &partials, &max_norm, &total_norm};
    return launch_pdl_args(reinterpret_cast<const void*>(grad_scale_kernel<N, LONG>), dim3(scale_blocks(t.chunks, LONG)),
                           dim3(kThreads), s, args);
  }
  cudaError_t norm(double* partial, int* blocks) const {
    if (count <= kSmall) return is_long ? norm<kSmall, true>(partial, blocks) : norm<kSmall, false>(partial, blocks);
    if (count <= kMedium) return is_long ? norm<kMedium, true>(partial, blocks) : norm<kMedium, false>(partial, blocks);
    return is_long ? norm<kMaxTable, true>(partial, blocks) : norm<kMaxTable, false>(partial, blocks);
  }
  cudaError_t scale(const double* p, int n, double max_norm, float* out) const {
    if (count <= kSmall) return is_long ? scale<kSmall, true>(p, n, max_norm, out) : scale<kSmall, false>(p, n, max_norm, out);
    if (count <= kMedium)
      return is_long ? scale<kMedium, true>(p, n, max_norm, out) : scale<kMedium, false>(p, n, max_norm, out);
    return is_long ? scale<kMaxTable, true>(p, n, max_norm, out) : scale<kMaxTable, false>(p, n, max_norm, out);
  }
};

}  // namespace

size_t grad_norm_partials(int32_t tensors) {
  const size_t launches = tensors > 0 ? (static_cast<size_t>(tensors) + kMaxTable - 1) / kMaxTable : 1;
  return launches * device_sm_count() * kBlocksPerSm;
}

cudaError_t launch_clip_grads(const e4b_grad* g, int32_t tensors, double max_norm, float* total_norm, double* partial,
                              cudaStream_t s) {
  bool in_place = true;
  auto run_at = [&](int32_t i) {
    ClipRun r{g + i, tensors - i < kMaxTable ? tensors - i : kMaxTable, false, s};
    size_t bytes = 0;
    for (int k = 0; k < r.count; ++k) bytes += static_cast<size_t>(r.g[k].n) * (r.g[k].dtype == E4B_F32 ? 4 : 2);
    r.is_long = bytes >= kLongBytes;
    return r;
  };
  int partials = 0;
  for (int32_t i = 0; i == 0 || i < tensors; i += kMaxTable) {
    int blocks = 0;
    const cudaError_t e = run_at(i).norm(partial + partials, &blocks);
    if (e != cudaSuccess) return e;
    partials += blocks;
  }
  if (tensors > kMaxTable) {
    const cudaError_t e = launch_pdl(grad_sum_kernel, dim3(1), dim3(kThreads), 0, s, partial, partials);
    if (e != cudaSuccess) return e;
    partials = 1;
  }
  for (int32_t k = 0; k < tensors; ++k) in_place = in_place && (g[k].n == 0 || g[k].grad == g[k].out);
  // only the norm is wanted and nothing moves: one block writes it
  if (std::isinf(max_norm) && in_place) return ClipRun{g, 0, false, s}.scale(partial, partials, max_norm, total_norm);
  for (int32_t i = 0; i == 0 || i < tensors; i += kMaxTable) {
    const cudaError_t e = run_at(i).scale(partial, partials, max_norm, i == 0 ? total_norm : nullptr);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace e4b
