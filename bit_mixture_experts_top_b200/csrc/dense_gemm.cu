// Dense bf16 matrix products of the gated feed-forward block on sm_100a tensor
// cores (tcgen05 / TMEM), each with its own epilogue:
//
//   gate_up : h = act(x W_gate^T + b, x W_up^T + b)      both projections and the activation in one kernel
//   linear  : out = A B^T (+ bias) (+ add)               the down product, dx and the weight gradients
//   dact    : dG = act'(G) applied to dout W_dn          (and its column sums, the bias gradient)
//
// D[M, N] = sum over k of A[m, k] B[n, k].  Either operand may be stored
// K-contiguous or M/N-contiguous: the backward reads the same weights and
// activations along their other dimension (dh = dout W_dn contracts the rows of
// W_dn, dW = dG^T x contracts the tokens), so no transposed copy exists.  TMA
// brings 128-byte-swizzled boxes either way; only the matrix descriptors differ.
//
// Large products run on CTA pairs (CG = 2): one MMA spans both SMs, 256 rows by
// 256 columns, and each CTA loads its 128 rows of A and half of B, 32 KB per 64
// of K where a single CTA with the same width loads 48 KB.  No multicast.
//
// One persistent CTA per SM.  Warp 0 issues the TMA loads, warp 1 owns tensor
// memory and issues the MMAs (M = 128 rows per CTA, two accumulators), warps
// 4-19 run the epilogue of one tile while the next is multiplied (sixteen, so
// that the last tile's, which nothing hides, is short).  Every wait is bounded
// (E4B_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int BM = 128;                  // rows of D per CTA
constexpr int BK = 64;                   // K per stage: one 128-byte swizzle row of bf16
constexpr int WARP_TMA = 0, WARP_MMA = 1, WARP_EPI0 = 4, EPI_WARPS = 16;
constexpr int THREADS = 32 * (WARP_EPI0 + EPI_WARPS);
constexpr uint64_t kDrainNs = 50000000ull;
// The tensor cores truncate each step's fp32 sum, so a long accumulation of
// values that do not add up exactly ends short of its sum: by 0.75e-9 to 1.1e-9
// of it per product, measured over K of 256 to 12288 on zero-mean and on positive
// data.  Nothing is put back: a factor would be wrong for every sum that was
// exact (a gate exactly on the clamp would fall outside).  The split kernel, whose
// tensor memory has room, lets two shorter chains meet in a rounded addition
// where an fp32 result leaves the kernel; the tiled kernels, whose two accumulators
// fill the tensor memory, keep one chain (bias gradients 2.8e-6 off at 1500 tokens,
// 4.3e-6 at 4096 with K = 2048, 6.1e-6 at 3000 with K = 2880).
constexpr int kGroupM = 16;              // row tiles that share a sweep over the columns (L2 reuse of both operands)

template <int BN, int CG>
struct Cfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = BN / CG;                      // this CTA's share of B
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 196608 / STAGE_BYTES;         // 4 (one CTA of 256 columns) or 6
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 5) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;     // + slack to align the base
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Params {
  int32_t M, N, K;          // D is M x N; gate_up: N = I features (2I rows of B)
  int32_t width;            // columns of D per tile, a multiple of 32, at most BN
  int32_t m_tiles, n_tiles;
  int32_t act;
  float alpha, limit, beta;
  const float* bias;        // gate_up: [2I]; linear: [N]; or null
  int32_t bias_words;       // bias is 16-byte aligned
  const uint16_t* add;      // linear: [M, N] bf16 or null
  int32_t wide;             // rows of out are whole 32-byte words
  uint16_t* out;            // bf16: h [M, I], D [M, N] or dG [M, 2I]
  float* g_out;             // gate_up: G [M, 2I] fp32 or null
  const float* g_in;        // dact: G [M, 2I]
  float* colsum;            // dact: partial column sums of dG, [rows, 2I] (one per 32 rows, or per split CTA), or null
  int32_t* status;
  int32_t clear_status;     // this launch is the first of its call: block 0 clears the status words
  int32_t b_early;          // split: the launch before this one does not write B
  uint64_t wait_limit_ns;
};

// Matrix descriptor of an operand stored M/N-contiguous: TMA boxes of 64 M/N x
// 64 K, i.e. 64 rows (K) of 128 bytes, swizzled; 8 K rows are one 1024-byte
// atom, the next 64 of M/N start a box (8192 bytes) further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;           // leading byte offset: next 64 of M/N
  d |= static_cast<uint64_t>(1024 >> 4) << 32;           // stride byte offset: next 8 of K
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Row tiles in groups of kGroupM; within a group columns advance slowest-first.
__device__ __forceinline__ void tile_at(const Params& p, int tile, int& mt, int& nt) {
  const int per_group = kGroupM * p.n_tiles;
  const int g = tile / per_group, in = tile - g * per_group;
  const int rows = min(kGroupM, p.m_tiles - g * kGroupM);
  nt = in / rows;
  mt = g * kGroupM + in - nt * rows;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// 32-byte accesses: in the row-per-lane layout of a tensor-memory load every lane touches its own row, and a whole
// sector per lane halves the requests.
__device__ __forceinline__ void store32(void* o, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p)
               : "memory");
}

// Sixteen adjacent bf16 columns of one row, or the first eight of them (the last of a ragged row).
__device__ __forceinline__ void store16(uint16_t* o, const uint4 (&v)[2], bool both, bool wide) {
  if (both && wide) {
    store32(o, v[0], v[1]);
  } else {
    *reinterpret_cast<uint4*>(o) = v[0];
    if (both) *reinterpret_cast<uint4*>(o + 8) = v[1];
  }
}

// d(act)/d(gate) and d(act)/d(up); the clamps pass the gradient inside their range, ends included.
__device__ __forceinline__ void act_grads(const Params& p, float gate, float up, float& dg, float& du) {
  if (p.act == E4B_ACT_CLAMPED_GLU) {
    const float g = clamp_up(gate, p.limit);
    const float u = -clamp_up(-clamp_up(up, p.limit), p.limit);
    const float s = __fdividef(1.0f, 1.0f + __expf(-p.alpha * g));
    const float df = s * (1.0f + p.alpha * g * (1.0f - s));
    dg = gate > p.limit ? 0.0f : df * (u + p.beta);
    du = (up < -p.limit || up > p.limit) ? 0.0f : g * s;
    return;
  }
  const float s = __fdividef(1.0f, 1.0f + __expf(-gate));
  dg = up * s * (1.0f + gate * (1.0f - s));
  du = gate * s;
}

// Sums 8 values per lane over the warp by halving: in three steps a lane keeps
// half of its columns and hands over the rest, then two plain steps; 9 shuffles.
// Lanes 4j hold the sum of one column each, `col`.
__device__ __forceinline__ float warp_column_sum8(const float (&in)[8], int lane, int& col) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = in[i];
  col = 0;
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1) {
    const bool upper = lane & (4 * h);
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = upper ? v[i + h] : v[i];
      const float give = upper ? v[i] : v[i + h];
      v[i] = keep + __shfl_xor_sync(kFull, give, 4 * h);
    }
    col += upper ? h : 0;
  }
  const float s = v[0] + __shfl_xor_sync(kFull, v[0], 2);
  return s + __shfl_xor_sync(kFull, s, 1);
}

__device__ __forceinline__ void add_bias8(const Params& p, int at, float (&f)[8]) {
  if (!p.bias) return;
  if (p.bias_words) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.bias + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + at) + 1);
    f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
    f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += __ldg(p.bias + at + i);
  }
}

// Eight fp32 values of G (its rows are whole 32-byte words: 2I is a multiple of 16).
__device__ __forceinline__ void store8f(float* o, const float (&f)[8]) {
  uint4 a, b;
  a.x = __float_as_uint(f[0]); a.y = __float_as_uint(f[1]); a.z = __float_as_uint(f[2]); a.w = __float_as_uint(f[3]);
  b.x = __float_as_uint(f[4]); b.y = __float_as_uint(f[5]); b.z = __float_as_uint(f[6]); b.w = __float_as_uint(f[7]);
  store32(o, a, b);
}

__device__ __forceinline__ void load8f(const float* p, float (&f)[8]) {
  uint4 a, b;
  load32(p, a, b);
  f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
  f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}

// The epilogues, eight adjacent columns of one row at a time (fp32 sums in, `col` a multiple of 8, below N), packed
// to bf16.  Rows past M hold zeros and are not read or written.
__device__ __forceinline__ uint4 finish_gate_up(const Params& p, int row, bool row_in, int col, float (&g)[8],
                                                float (&u)[8]) {
  add_bias8(p, col, g);
  add_bias8(p, p.N + col, u);
  if (p.g_out && row_in) {
    float* o = p.g_out + static_cast<int64_t>(row) * 2 * p.N + col;
    store8f(o, g);
    store8f(o + p.N, u);
  }
  const Epilogue ep{nullptr, p.act, p.alpha, p.limit, p.beta};
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = dense_act(ep, g[i], u[i]);
  return pack8(g);
}

__device__ __forceinline__ uint4 finish_linear(const Params& p, int row, bool row_in, int col, float (&f)[8]) {
  add_bias8(p, col, f);
  if (p.add && row_in) {
    const uint4 a = *reinterpret_cast<const uint4*>(p.add + static_cast<int64_t>(row) * p.N + col);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] += __uint_as_float(w[i] << 16);
      f[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  return pack8(f);
}

// G of eight columns, loaded ahead of its use.
struct SavedG {
  float g[8], u[8];

  __device__ __forceinline__ void load(const Params& p, int row, bool in, int col) {
    if (!in) return;
    const float* gp = p.g_in + static_cast<int64_t>(row) * 2 * p.N + col;
    load8f(gp, g);
    load8f(gp + p.N, u);
  }
};

// All lanes of the warp call it with rows row0 + lane (row0 a multiple of 32).
__device__ __forceinline__ void finish_dact(const Params& p, int row, bool row_in, int col, int lane, const SavedG& G,
                                            const float (&dh)[8], uint4& og, uint4& ou) {
  float dg[8], du[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dg[i] = du[i] = 0.0f;
  if (row_in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      act_grads(p, G.g[i], G.u[i], dg[i], du[i]);
      dg[i] *= dh[i];
      du[i] *= dh[i];
    }
  }
  og = pack8(dg);
  ou = pack8(du);
  if (p.colsum) {                         // from the fp32 values, before their rounding to bf16
    const int row0 = row - lane;
    int c;
    const float sg = warp_column_sum8(dg, lane, c);
    const float su = warp_column_sum8(du, lane, c);
    if ((lane & 3) == 0 && row0 < p.M) {
      float* o = p.colsum + static_cast<int64_t>(row0 / 32) * 2 * p.N + col + c;
      o[0] = sg;
      o[p.N] = su;
    }
  }
}

__device__ __forceinline__ void take8(const uint32_t (&r)[16], int j, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[j + i]);
}

template <int BN, int CG, bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    dense_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const Params p) {
  using C = Cfg<BN, CG>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* s_never = acc_empty + 2;        // a barrier that nothing arrives on
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int32_t* s_abort = reinterpret_cast<int32_t*>(smem + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;          // rank 0 issues the pair's MMAs

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CG * EPI_WARPS);
    }
    mbar_init(s_never, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  pdl_wait();
  pdl_launch_dependents();
  // a wait can only run out seconds after this, so the clearing needs no ordering among the blocks
  if (p.clear_status && blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  if (warp == WARP_MMA) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(s_tmem, C::TMEM_COLS);
    } else {
      tmem_alloc(s_tmem, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();         // the other CTA's barriers and tensor memory are ready too
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  const WaitCtx wctx{s_abort, p.status, p.wait_limit_ns};
  const int total = p.m_tiles * p.n_tiles;
  const int ksteps = (p.K + BK - 1) / BK;
  const int NT = EPI == kEpiGateUp ? p.width / 2 : p.width;     // output columns (features) per tile
  const int b_rows = p.width / CG;                              // this CTA's rows of B per stage
  const int b_boxes = (b_rows + 63) / 64;                       // B row-contiguous: whole boxes of 64
  const uint32_t stage_tx = C::A_BYTES + (B_MN ? b_boxes * 8192 : b_rows * BK * 2);
  const int first = blockIdx.x / CG, step = gridDim.x / CG;

  if (warp == WARP_TMA) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, par = 0;
    bool ok = true;
    for (int tile = first; ok && tile < total; tile += step) {
      int mt, nt;
      tile_at(p, tile, mt, nt);
      const int m0 = (mt * CG + rank) * BM, n0 = nt * NT;
      for (int ks = 0; ks < ksteps; ++ks) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, wctx, 1101)) { ok = false; break; }
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * stage_tx);
          const uint32_t bar = CG == 2 ? cluster_addr(&full[stage], 0) : 0;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
            if constexpr (CG == 2) tma_load_2d_pair(dst, map, bar, x, y);
            else tma_load_2d(dst, map, &full[stage], x, y);
          };
          uint8_t* a = smem + stage * C::STAGE_BYTES;
          uint8_t* b = a + C::A_BYTES;
          const int k0 = ks * BK;
          if constexpr (A_MN) {
#pragma unroll
            for (int i = 0; i < BM / 64; ++i) load(a + i * 8192, &tm_a, m0 + 64 * i, k0);
          } else {
            load(a, &tm_a, k0, m0);
          }
          const int nb = n0 + static_cast<int>(rank) * b_rows;
          if constexpr (EPI == kEpiGateUp && CG == 2) {  // gate rows in one CTA, the matching up rows in the other
            load(b, &tm_b, k0, rank == 0 ? n0 : p.N + n0);
          } else if constexpr (EPI == kEpiGateUp) {      // gate rows, then the matching up rows
            load(b, &tm_b, k0, n0);
            load(b + NT * BK * 2, &tm_b, k0, p.N + n0);
          } else if constexpr (B_MN) {
            for (int i = 0; i < b_boxes; ++i) load(b + i * 8192, &tm_b, nb + 64 * i, k0);
          } else {
            load(b, &tm_b, k0, nb);
          }
        }
        __syncwarp();
        armed |= 1u << stage;
        par = (par & ~(1u << stage)) | (phase << stage);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) {   // let every issued copy land before the CTA's shared memory is released
      for (int s = 0; s < C::STAGES; ++s)        // (rank 1 has no barrier of its own to watch: it waits the limit out)
        if (armed & (1u << s)) mbar_drain(rank == 0 ? &full[s] : s_never, rank == 0 ? (par >> s) & 1u : 0u, kDrainNs);
    }
  } else if (warp == WARP_MMA) {
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(CG * BM, p.width) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
      // descriptors differ only in their start address (16-byte units): 16 of K are 32 bytes along a row, or two
      // 8-row atoms where K is the row
      const uint32_t base = smem_u32(smem);
      const uint64_t da0 = A_MN ? smem_desc_mn_sw128(base) : smem_desc_sw128(base);
      const uint64_t db0 = B_MN ? smem_desc_mn_sw128(base + C::A_BYTES) : smem_desc_sw128(base + C::A_BYTES);
      constexpr uint32_t a_step = (A_MN ? 2048 : 32) >> 4, b_step = (B_MN ? 2048 : 32) >> 4;
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      uint64_t* last_bar = nullptr;
      uint32_t last_par = 0;
      for (int tile = first; ok && tile < total; tile += step, ++it) {
        const int buf = it & 1;
        const uint32_t aphase = (it >> 1) & 1;
        if (!mbar_wait_warp(&acc_empty[buf], aphase ^ 1u, wctx, 1201)) { ok = false; break; }
        tc_fence_after_sync();
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
        for (int ks = 0; ks < ksteps; ++ks) {
          if (!mbar_wait_warp(&full[stage], phase, wctx, 1202)) { ok = false; break; }
          const uint64_t da = da0 + static_cast<uint32_t>(stage * (C::STAGE_BYTES >> 4));
          const uint64_t db = db0 + static_cast<uint32_t>(stage * (C::STAGE_BYTES >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              if constexpr (CG == 2) umma_bf16_ss_pair(d, da + kk * a_step, db + kk * b_step, idesc, (ks > 0 || kk > 0) ? 1u : 0u);
              else umma_bf16_ss(d, da + kk * a_step, db + kk * b_step, idesc, (ks > 0 || kk > 0) ? 1u : 0u);
            }
            if constexpr (CG == 2) umma_commit_pair(&empty[stage]);
            else umma_commit(&empty[stage]);
            if (ks == ksteps - 1) {
              if constexpr (CG == 2) umma_commit_pair(&acc_full[buf]);
              else umma_commit(&acc_full[buf]);
            }
          }
          __syncwarp();
          issued = true;
          last_bar = &empty[stage];
          last_par = phase;
          if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && issued && lane == 0) mbar_drain(last_bar, last_par, kDrainNs);   // MMAs in flight finish first
    }
  } else if (warp >= WARP_EPI0) {
    const int q = warp & 3;                        // TMEM lanes 32q..32q+31: D row = lane
    const int part = (warp - WARP_EPI0) >> 2;      // the warps of a row quarter take chunks of 16 columns in turn
    int it = 0;
    for (int tile = first; tile < total; tile += step, ++it) {
      int mt, nt;
      tile_at(p, tile, mt, nt);
      const int buf = it & 1;
      const uint32_t aphase = (it >> 1) & 1;
      if (!__all_sync(kFull, mbar_wait_sleep(&acc_full[buf], aphase, wctx, 1401, 64))) break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * BN);
      const int row0 = (mt * CG + static_cast<int>(rank)) * BM + 32 * q;
      const int row = row0 + lane;
      const bool row_in = row < p.M;
#pragma unroll 1
      for (int c0 = 16 * part; c0 < NT; c0 += 16 * (EPI_WARPS / 4)) {
        const int col = nt * NT + c0;
        if (col >= p.N) break;
        const bool both = col + 8 < p.N;               // (a tile's width is a multiple of 16)
        uint32_t r[16], u[16];
        SavedG G[2];
        tmem_ld_32x32b_x16(taddr + c0, r);
        if constexpr (EPI == kEpiGateUp) tmem_ld_32x32b_x16(taddr + NT + c0, u);
        if constexpr (EPI == kEpiDact) {
          G[0].load(p, row, row_in, col);
          G[1].load(p, row, row_in && both, col + 8);
        }
        tmem_ld_wait();
        uint4 v[2], w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (j == 1 && !both) break;
          float f[8];
          take8(r, 8 * j, f);
          if constexpr (EPI == kEpiGateUp) {
            float fu[8];
            take8(u, 8 * j, fu);
            v[j] = finish_gate_up(p, row, row_in, col + 8 * j, f, fu);
          } else if constexpr (EPI == kEpiLinear) {
            v[j] = finish_linear(p, row, row_in, col + 8 * j, f);
          } else {
            finish_dact(p, row, row_in, col + 8 * j, lane, G[j], f, v[j], w[j]);
          }
        }
        if (row_in) {
          uint16_t* o = p.out + static_cast<int64_t>(row) * (EPI == kEpiDact ? 2 * p.N : p.N) + col;
          store16(o, v, both, p.wide);
          if constexpr (EPI == kEpiDact) store16(o + p.N, w, both, p.wide);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
        else mbar_arrive(&acc_empty[buf]);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();         // neither CTA leaves while the other may still signal it
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------- split along K

// A product too small to give every SM a tile: a cluster of S CTAs shares one
// 128 x 128 tile, each multiplies its part of K, and the partial tiles meet
// through distributed shared memory: every CTA adds the S parts, from its own
// rank on, of its share of the rows (whole rows, a warp each: contiguous 512-byte
// reads from every rank and contiguous stores; a lane-per-row layout took five
// times as long) and runs the epilogue on them.  Stages hold 128 of K: with tiles this
// narrow the per-stage wait, not the MMA, is what costs.
//
// B (weights) may be loaded before the previous launch has completed when that
// launch does not write it (b_early): the first stages then hide its tail.
struct SplitCfg {
  static constexpr int BN = 128, SK = 128;
  static constexpr int ATOM = BM * BK * 2;                    // 128 rows of 64 K
  static constexpr int RING_BYTES = 196608;                   // three stages of two atoms of A and two of B, or four
  static constexpr int MAX_STAGES = 4;                        // with half atoms of A
  static constexpr int PITCH = BN + 4;                        // floats per row of the partial tile (conflict-free)
  static constexpr int OFF_SUMS = BM * PITCH * 4;             // dact: column sums per warp, behind the partial tile
  static constexpr int OFF_BAR = RING_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + (2 * MAX_STAGES + 1) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int EPI = 8, THREADS = 32 * (WARP_EPI0 + EPI);
  // G and dh, whose fp32 values are kept or summed up, are accumulated in two chains of half of the CTA's K, added in
  // fp32 with rounding: the gate and up bias gradients of 509 x 2048 x 768 are 7.5e-7 off instead of 1.5e-6 (relative
  // 2-norm) for 0.1 us a launch; four chains bring 3.8e-7 for 0.4.  What leaves as bf16 alone does not see it.
  template <int E>
  static constexpr int chains() { return E == kEpiLinear ? 1 : 2; }
  static_assert(OFF_SUMS + EPI * 2 * BN * 4 <= RING_BYTES, "both reuse the stages");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float4 bias4(const Params& p, int at) {
  if (p.bias_words) return __ldg(reinterpret_cast<const float4*>(p.bias + at));
  return make_float4(__ldg(p.bias + at), __ldg(p.bias + at + 1), __ldg(p.bias + at + 2), __ldg(p.bias + at + 3));
}

__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}

__device__ __forceinline__ uint2 pack4(const float4& v) { return make_uint2(pack2(v.x, v.y), pack2(v.z, v.w)); }

template <bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(SplitCfg::THREADS, 1)
    dense_split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                       const Params p, int S) {
  using C = SplitCfg;
  constexpr int CHAINS = C::chains<EPI>();
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::MAX_STAGES;
  uint64_t* acc_full = empty + C::MAX_STAGES;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int32_t* s_abort = reinterpret_cast<int32_t*>(smem + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  // Up to 64 rows A is loaded in half atoms: what the MMA reads behind them (the next atom) only reaches rows of D
  // that nobody reads, and the ring holds four stages.
  const bool half_a = !A_MN && p.M <= BM / 2;
  const int a_atom = half_a ? C::ATOM / 2 : C::ATOM, stages = half_a ? 4 : 3;
  const int stage_bytes = 2 * (a_atom + C::ATOM);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == WARP_MMA) {      // (no other tensor-memory kernel of the library leaves room for this one on its SM)
    tmem_alloc(s_tmem, CHAINS * C::BN);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  const WaitCtx wctx{s_abort, p.status, p.wait_limit_ns};
  constexpr int NT = EPI == kEpiGateUp ? C::BN / 2 : C::BN;
  int mt, nt;
  tile_at(p, blockIdx.x / S, mt, nt);
  const int m0 = mt * BM, n0 = nt * NT;
  const int steps = (p.K + C::SK - 1) / C::SK;
  const int first = static_cast<int>(static_cast<int64_t>(steps) * rank / S);
  const int last = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / S);      // S <= steps: never empty
  const int per_chain = (last - first + CHAINS - 1) / CHAINS;
  auto atoms_of = [&](int ks) { return min(2, (p.K - ks * C::SK + BK - 1) / BK); };

  if (warp == WARP_TMA) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, par = 0;
    bool ok = true;
    auto load_a = [&](int ks, int stage) {
      uint8_t* a = smem + stage * stage_bytes;
      for (int i = 0; i < atoms_of(ks); ++i, a += a_atom) {
        const int k0 = ks * C::SK + i * BK;
        if constexpr (A_MN) {
          tma_load_2d(a, &tm_a, &full[stage], m0, k0);
          tma_load_2d(a + 8192, &tm_a, &full[stage], m0 + 64, k0);
        } else {
          tma_load_2d(a, &tm_a, &full[stage], k0, m0);
        }
      }
    };
    auto load_b = [&](int ks, int stage) {
      uint8_t* b = smem + stage * stage_bytes + 2 * a_atom;
      mbar_arrive_expect_tx(&full[stage], atoms_of(ks) * (a_atom + C::ATOM));
      for (int i = 0; i < atoms_of(ks); ++i, b += C::ATOM) {
        const int k0 = ks * C::SK + i * BK;
        if constexpr (EPI == kEpiGateUp) {
          tma_load_2d(b, &tm_b, &full[stage], k0, n0);
          tma_load_2d(b + 8192, &tm_b, &full[stage], k0, p.N + n0);
        } else if constexpr (B_MN) {
          tma_load_2d(b, &tm_b, &full[stage], n0, k0);
          tma_load_2d(b + 8192, &tm_b, &full[stage], n0 + 64, k0);
        } else {
          tma_load_2d(b, &tm_b, &full[stage], k0, n0);
        }
      }
    };
    const int early = p.b_early ? min(stages, last - first) : 0;
    if (elect_one())
      for (int i = 0; i < early; ++i) load_b(first + i, i);
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    for (int ks = first; ks < last; ++ks) {
      if (!mbar_wait_warp(&empty[stage], phase ^ 1u, wctx, 1501)) { ok = false; break; }
      if (elect_one()) {
        if (ks - first >= early) load_b(ks, stage);
        load_a(ks, stage);
      }
      __syncwarp();
      armed |= 1u << stage;
      par = (par & ~(1u << stage)) | (phase << stage);
      if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
    if (!ok && lane == 0) {
      for (int s = 0; s < stages; ++s)
        if (armed & (1u << s)) mbar_drain(&full[s], (par >> s) & 1u, kDrainNs);
    }
  } else if (warp == WARP_MMA) {
    constexpr uint32_t idesc = idesc_bf16_f32(BM, C::BN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
    const uint32_t base = smem_u32(smem);
    const uint64_t da0 = A_MN ? smem_desc_mn_sw128(base) : smem_desc_sw128(base);
    const uint64_t db0 = B_MN ? smem_desc_mn_sw128(base + 2 * a_atom) : smem_desc_sw128(base + 2 * a_atom);
    constexpr uint32_t a_step = (A_MN ? 2048 : 32) >> 4, b_step = (B_MN ? 2048 : 32) >> 4;
    int stage = 0, in_chain = 0;
    uint32_t phase = 0, d = tmem_base;
    bool ok = true, issued = false;
    pdl_wait();
    if (p.clear_status && blockIdx.x == 0 && lane < 2) p.status[lane] = 0;
    for (int ks = first; ks < last; ++ks) {
      if (!mbar_wait_warp(&full[stage], phase, wctx, 1502)) { ok = false; break; }
      const int atoms = atoms_of(ks);
      const uint64_t da = da0 + static_cast<uint32_t>(stage * (stage_bytes >> 4));
      const uint64_t db = db0 + static_cast<uint32_t>(stage * (stage_bytes >> 4));
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < C::SK / 16; ++kk) {
          if (kk >= 4 * atoms) break;
          umma_bf16_ss(d, da + static_cast<uint32_t>((kk >> 2) * (a_atom >> 4) + (kk & 3) * a_step),
                       db + (kk >> 2) * (C::ATOM >> 4) + (kk & 3) * b_step, idesc,
                       (in_chain > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(&empty[stage]);
        if (ks == last - 1) umma_commit(acc_full);
      }
      __syncwarp();
      issued = true;
      if (++in_chain == per_chain) { in_chain = 0; d += C::BN; }
      if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
    if (!ok && issued && lane == 0)
      mbar_drain(&empty[stage == 0 ? stages - 1 : stage - 1], stage == 0 ? phase ^ 1u : phase, kDrainNs);
  } else if (warp >= WARP_EPI0) {
    // this CTA's partial tile into its shared memory (every stage has been consumed by then)
    const int q = warp & 3, half = (warp - WARP_EPI0) >> 2;
    pdl_wait();
    if (__all_sync(kFull, mbar_wait_sleep(acc_full, 0, wctx, 1503, 64))) {
      tc_fence_after_sync();
      float* row = reinterpret_cast<float*>(smem) + (32 * q + lane) * C::PITCH;
      if (m0 + 32 * q < p.M) {
#pragma unroll
        for (int c0 = half * (C::BN / 2); c0 < (half + 1) * (C::BN / 2); c0 += 32) {
          const uint32_t at = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c0;
          uint32_t r[16], u[16];
          tmem_ld_32x32b_x16(at, r);
          tmem_ld_32x32b_x16(at + 16, u);
          tmem_ld_wait();
          if constexpr (CHAINS > 1) {
            for (int c = 1; c * per_chain < last - first; ++c) {
              uint32_t v[16], w[16];
              tmem_ld_32x32b_x16(at + c * C::BN, v);
              tmem_ld_32x32b_x16(at + c * C::BN + 16, w);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(v[j]));
                u[j] = __float_as_uint(__uint_as_float(u[j]) + __uint_as_float(w[j]));
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            *reinterpret_cast<uint4*>(row + c0 + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
            *reinterpret_cast<uint4*>(row + c0 + 16 + j) = make_uint4(u[j], u[j + 1], u[j + 2], u[j + 3]);
          }
        }
      }
      tc_fence_before_sync();
    }
  }
  __syncwarp();
  cluster_sync();
  if (warp >= WARP_EPI0) {
    const int ew = warp - WARP_EPI0;
    const int rows = min(BM, p.M - m0);
    const uint32_t mine = smem_u32(smem) + 16 * lane;
    // rows go round the ranks, then round the warps; a lane holds four adjacent columns of the tile
    const int tile_col = 4 * lane;
    const int col = n0 + (EPI == kEpiGateUp ? tile_col & (NT - 1) : tile_col);
    const bool col_in = col < p.N;
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (EPI != kEpiDact && p.bias && col_in) bias = bias4(p, EPI == kEpiGateUp && lane >= 16 ? p.N + col : col);
    float4 sg = make_float4(0.f, 0.f, 0.f, 0.f), su = sg;      // dact: column sums over this warp's rows
    constexpr int GROUP = 2;                       // rows whose parts are on their way together
    for (int r0 = rank + S * ew; r0 < rows; r0 += GROUP * S * C::EPI) {
      float4 sum[GROUP];
#pragma unroll
      for (int i = 0; i < GROUP; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int s = 0; s < S; ++s) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(rank + s < S ? rank + s : rank + s - S));
        float4 part[GROUP];
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          const int r = r0 + i * S * C::EPI;
          part[i] = r < rows ? load_cluster(at + r * C::PITCH * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) add4(sum[i], part[i]);
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        const int r = r0 + i * S * C::EPI;
        if (r >= rows) break;
        const int64_t row = m0 + r;
        float4 f = sum[i];
        if constexpr (EPI != kEpiDact) add4(f, bias);
        if constexpr (EPI == kEpiGateUp) {             // lanes 0..15 hold gate, 16..31 the matching up features
          if (p.g_out && col_in)
            *reinterpret_cast<float4*>(p.g_out + row * 2 * p.N + (lane >= 16 ? p.N : 0) + col) = f;
          float4 u;
          u.x = __shfl_down_sync(kFull, f.x, 16);
          u.y = __shfl_down_sync(kFull, f.y, 16);
          u.z = __shfl_down_sync(kFull, f.z, 16);
          u.w = __shfl_down_sync(kFull, f.w, 16);
          if (lane < 16 && col_in) {
            const Epilogue ep{nullptr, p.act, p.alpha, p.limit, p.beta};
            f.x = dense_act(ep, f.x, u.x);
            f.y = dense_act(ep, f.y, u.y);
            f.z = dense_act(ep, f.z, u.z);
            f.w = dense_act(ep, f.w, u.w);
            *reinterpret_cast<uint2*>(p.out + row * p.N + col) = pack4(f);
          }
        } else if constexpr (EPI == kEpiLinear) {
          if (col_in) {
            if (p.add) {
              const uint2 a = *reinterpret_cast<const uint2*>(p.add + row * p.N + col);
              add4(f, make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u),
                                  __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u)));
            }
            *reinterpret_cast<uint2*>(p.out + row * p.N + col) = pack4(f);
          }
        } else if (col_in) {
          const float* gp = p.g_in + row * 2 * p.N + col;
          const float4 g = *reinterpret_cast<const float4*>(gp), u = *reinterpret_cast<const float4*>(gp + p.N);
          float4 dg, du;
          act_grads(p, g.x, u.x, dg.x, du.x);
          act_grads(p, g.y, u.y, dg.y, du.y);
          act_grads(p, g.z, u.z, dg.z, du.z);
          act_grads(p, g.w, u.w, dg.w, du.w);
          dg = make_float4(dg.x * f.x, dg.y * f.y, dg.z * f.z, dg.w * f.w);
          du = make_float4(du.x * f.x, du.y * f.y, du.z * f.z, du.w * f.w);
          *reinterpret_cast<uint2*>(p.out + row * 2 * p.N + col) = pack4(dg);
          *reinterpret_cast<uint2*>(p.out + row * 2 * p.N + p.N + col) = pack4(du);
          add4(sg, dg);
          add4(su, du);
        }
      }
    }
    if constexpr (EPI == kEpiDact) {
      if (p.colsum) {                                  // the warps' sums, one row of partial sums per CTA
        float4* sums = reinterpret_cast<float4*>(smem + C::OFF_SUMS);
        sums[ew * 64 + lane] = sg;
        sums[ew * 64 + 32 + lane] = su;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * C::EPI) : "memory");
        const int i = threadIdx.x - 32 * WARP_EPI0;
        if (i < 64) {
          float4 t = sums[i];
          for (int w = 1; w < C::EPI; ++w) add4(t, sums[w * 64 + i]);
          const int c = n0 + 4 * (i & 31);
          if (c < p.N)
            *reinterpret_cast<float4*>(p.colsum + (static_cast<int64_t>(mt) * S + rank) * 2 * p.N + (i >> 5) * p.N + c) = t;
        }
      }
    }
  }
  __syncwarp();
  cluster_sync();                                 // the partial tile stays until every rank has read it
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, CHAINS * C::BN);
  }
}

// ---------------------------------------------------------------------- several products in one launch

// The backward's last three products (dx and both weight gradients) depend on
// dG alone.  Where each is too small to fill the device, one launch runs them
// together: the tiles of all products, in order, are dealt by their cost (K
// steps and a fixed part) so that every CTA or pair gets an equal share of the
// whole.  Pairs with tiles of 256 x 256 read each operand half as often as CTAs
// with 128 x 128, which L2 bounds; small tiles deal better where there are few.  A is K- or row-contiguous per
// product, B row-contiguous in all; the epilogue is the plain bf16 store.  Two
// warps that have no other work form the bias gradients' column sums meanwhile
// (5 us as a launch of their own).
// Backward of 509 tokens at 2048 x 768: 31 us with pairs, 35 with small tiles, 38
// one by one; at 2880 x 2880 71, 87 and 93.
constexpr int kMultiMax = 3;
constexpr int kTileFixed = 3;            // a tile's cost beside its K steps, in steps

struct MultiProblem {
  int32_t M, N, K, n_tiles, tiles, a_mn, wide;
  uint16_t* out;
};

struct MultiParams {
  int32_t count;
  int32_t* status;
  uint64_t wait_limit_ns;
  MultiProblem p[kMultiMax];
  ColumnSums sums;
};

struct alignas(64) MultiMaps {
  CUtensorMap a[kMultiMax], b[kMultiMax];
};

// Calls body(problem index, tile) for the tiles of share `share` of `shares`, in order, while it returns true.
template <typename Body>
__device__ __forceinline__ void walk_tiles(const MultiParams& mp, int share, int shares, const Body& body) {
  int64_t total = 0;
  auto cost = [&](int i) { return static_cast<int64_t>((mp.p[i].K + BK - 1) / BK + kTileFixed); };
  for (int i = 0; i < mp.count; ++i) total += mp.p[i].tiles * cost(i);
  const int64_t lo = total * share / shares, hi = total * (share + 1) / shares;
  int64_t at = 0;                          // cost of the products before
  for (int i = 0; i < mp.count; ++i) {
    const int64_t c = cost(i);
    // tiles whose middle lies in [lo, hi)
    auto first = [&](int64_t x) {
      const int64_t d = x - at - c / 2;
      const int64_t t = d <= 0 ? 0 : (d + c - 1) / c;
      return static_cast<int>(t < mp.p[i].tiles ? t : mp.p[i].tiles);
    };
    const int t1 = first(hi);
    for (int t = first(lo); t < t1; ++t)
      if (!body(i, t)) return;
    at += mp.p[i].tiles * c;
  }
}

// Column sums, a warp per strip of eight columns: a lane takes every 32nd row, then the lanes meet.
__device__ __forceinline__ void sum_strips(const ColumnSums& c, int first, int step, int lane) {
  const int strips_b = c.out_b ? c.Nb / 8 : 0, strips = strips_b + (c.out_a ? c.Na / 8 : 0);
  for (int i = first; i < strips; i += step) {
    float v[8] = {};
    const bool is_b = i < strips_b;
    const int at = 8 * (is_b ? i : i - strips_b);
    if (is_b) {
#pragma unroll 8
      for (int r = lane; r < c.rows_b; r += 32) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(c.b + static_cast<int64_t>(r) * c.Nb + at));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] += __uint_as_float(u[j] << 16);
          v[2 * j + 1] += __uint_as_float(u[j] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll 2
      for (int r = lane; r < c.rows_a; r += 32) {
        float f[8];
        load8f(c.a + static_cast<int64_t>(r) * c.Na + at, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
      }
    }
    int col;
    const float sum = warp_column_sum8(v, lane, col);
    if ((lane & 3) == 0) (is_b ? c.out_b : c.out_a)[at + col] = sum;
  }
}

template <int CG>
__global__ void __launch_bounds__(THREADS, 1)
    dense_multi_kernel(const __grid_constant__ MultiMaps maps, const __grid_constant__ MultiParams mp) {
  constexpr int BN = 128 * CG;
  using C = Cfg<BN, CG>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* s_never = acc_empty + 2;        // a barrier that nothing arrives on
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int32_t* s_abort = reinterpret_cast<int32_t*>(smem + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;          // rank 0 issues the pair's MMAs
  const int share = blockIdx.x / CG, shares = gridDim.x / CG;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CG * EPI_WARPS);
    }
    mbar_init(s_never, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == WARP_MMA) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(s_tmem, C::TMEM_COLS);
    } else {
      tmem_alloc(s_tmem, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();         // the other CTA's barriers and tensor memory are ready too
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  const WaitCtx wctx{s_abort, mp.status, mp.wait_limit_ns};

  if (warp == WARP_TMA) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, par = 0;
    bool ok = true;
    walk_tiles(mp, share, shares, [&](int i, int tile) {
      const MultiProblem& q = mp.p[i];
      const int m0 = (tile / q.n_tiles * CG + rank) * BM, n0 = tile % q.n_tiles * BN + rank * C::B_ROWS;
      const int ksteps = (q.K + BK - 1) / BK;
      for (int ks = 0; ks < ksteps; ++ks) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, wctx, 1601)) { ok = false; break; }
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * C::STAGE_BYTES);
          const uint32_t bar = CG == 2 ? cluster_addr(&full[stage], 0) : 0;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
            if constexpr (CG == 2) tma_load_2d_pair(dst, map, bar, x, y);
            else tma_load_2d(dst, map, &full[stage], x, y);
          };
          uint8_t* a = smem + stage * C::STAGE_BYTES;
          const int k0 = ks * BK;
          if (q.a_mn) {
            load(a, &maps.a[i], m0, k0);
            load(a + 8192, &maps.a[i], m0 + 64, k0);
          } else {
            load(a, &maps.a[i], k0, m0);
          }
#pragma unroll
          for (int j = 0; j < C::B_ROWS / 64; ++j) load(a + C::A_BYTES + j * 8192, &maps.b[i], n0 + 64 * j, k0);
        }
        __syncwarp();
        armed |= 1u << stage;
        par = (par & ~(1u << stage)) | (phase << stage);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
      return ok;
    });
    if (!ok && lane == 0) {   // let every issued copy land before the CTA's shared memory is released
      for (int s = 0; s < C::STAGES; ++s)        // (rank 1 has no barrier of its own to watch: it waits the limit out)
        if (armed & (1u << s)) mbar_drain(rank == 0 ? &full[s] : s_never, rank == 0 ? (par >> s) & 1u : 0u, kDrainNs);
    }
  } else if (warp == WARP_MMA && rank == 0) {
    const uint32_t base = smem_u32(smem);
    const uint64_t db0 = smem_desc_mn_sw128(base + C::A_BYTES);
    constexpr uint32_t b_step = 2048 >> 4;
    int stage = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true, issued = false;
    uint64_t* last_bar = nullptr;
    uint32_t last_par = 0;
    walk_tiles(mp, share, shares, [&](int i, int) {
      const MultiProblem& q = mp.p[i];
      const uint32_t idesc = idesc_bf16_f32(CG * BM, BN) | (q.a_mn ? 1u << 15 : 0u) | 1u << 16;
      const uint64_t da0 = q.a_mn ? smem_desc_mn_sw128(base) : smem_desc_sw128(base);
      const uint32_t a_step = (q.a_mn ? 2048 : 32) >> 4;
      const int ksteps = (q.K + BK - 1) / BK, buf = it & 1;
      if (!mbar_wait_warp(&acc_empty[buf], ((it >> 1) & 1) ^ 1u, wctx, 1602)) ok = false;
      tc_fence_after_sync();
      const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
      for (int ks = 0; ok && ks < ksteps; ++ks) {
        if (!mbar_wait_warp(&full[stage], phase, wctx, 1603)) { ok = false; break; }
        const uint64_t da = da0 + static_cast<uint32_t>(stage * (C::STAGE_BYTES >> 4));
        const uint64_t db = db0 + static_cast<uint32_t>(stage * (C::STAGE_BYTES >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            if constexpr (CG == 2) umma_bf16_ss_pair(d, da + kk * a_step, db + kk * b_step, idesc, (ks > 0 || kk > 0) ? 1u : 0u);
            else umma_bf16_ss(d, da + kk * a_step, db + kk * b_step, idesc, (ks > 0 || kk > 0) ? 1u : 0u);
          }
          if constexpr (CG == 2) umma_commit_pair(&empty[stage]);
          else umma_commit(&empty[stage]);
          if (ks == ksteps - 1) {
            if constexpr (CG == 2) umma_commit_pair(&acc_full[buf]);
            else umma_commit(&acc_full[buf]);
          }
        }
        __syncwarp();
        issued = true;
        last_bar = &empty[stage];
        last_par = phase;
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
      ++it;
      return ok;
    });
    if (!ok && issued && lane == 0) mbar_drain(last_bar, last_par, kDrainNs);   // MMAs in flight finish first
  } else if (warp > WARP_MMA && warp < WARP_EPI0) {
    constexpr int kWarps = WARP_EPI0 - WARP_MMA - 1;
    sum_strips(mp.sums, blockIdx.x * kWarps + warp - WARP_MMA - 1, gridDim.x * kWarps, lane);
  } else if (warp >= WARP_EPI0) {
    const int q4 = warp & 3, part = (warp - WARP_EPI0) >> 2;
    int it = 0;
    walk_tiles(mp, share, shares, [&](int i, int tile) {
      const MultiProblem& q = mp.p[i];
      const int n0 = tile % q.n_tiles * BN, buf = it & 1;
      if (!__all_sync(kFull, mbar_wait_sleep(&acc_full[buf], (it >> 1) & 1, wctx, 1604, 64))) return false;
      tc_fence_after_sync();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q4 * 32) << 16) + static_cast<uint32_t>(buf * BN);
      const int row = (tile / q.n_tiles * CG + rank) * BM + 32 * q4 + lane;
#pragma unroll 1
      for (int c0 = 16 * part; c0 < BN; c0 += 16 * (EPI_WARPS / 4)) {
        const int col = n0 + c0;
        if (col >= q.N) break;
        uint32_t r[16];
        tmem_ld_32x32b_x16(taddr + c0, r);
        tmem_ld_wait();
        if (row < q.M) {
          const bool both = col + 8 < q.N;
          float f[8], g[8];
          take8(r, 0, f);
          take8(r, 8, g);
          const uint4 v[2] = {pack8(f), pack8(g)};
          store16(q.out + static_cast<int64_t>(row) * q.N + col, v, both, q.wide);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
        else mbar_arrive(&acc_empty[buf]);
      }
      ++it;
      return true;
    });
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();         // neither CTA leaves while the other may still signal it
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------- host side

// Tensor maps of both operands.  K-contiguous: [rows, K], boxes of 64 K x tile rows; M/N-contiguous:
// [K, rows], boxes of 64 rows x 64 K.
template <bool A_MN, bool B_MN, int EPI>
bool encode_operands(const DenseGemmLaunch& g, int b_box, CUtensorMap* ta, CUtensorMap* tb, int a_box = BM) {
  const uint64_t b_rows = EPI == kEpiGateUp ? 2 * static_cast<uint64_t>(g.N) : g.N;
  auto enc = [](CUtensorMap* m, const uint16_t* p, uint64_t rows, uint64_t K, bool mn, int box) {
    return mn ? encode_tma_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, rows, K, rows * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B)
              : encode_tma_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, K, rows, K * 2, BK, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  return enc(ta, g.a, g.M, g.K, A_MN, a_box) && enc(tb, g.b, b_rows, g.K, B_MN, b_box);
}

Params make_params(const DenseGemmLaunch& g, int tile_rows, int width, int tile_cols) {
  Params p;
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.width = width;
  p.m_tiles = (g.M + tile_rows - 1) / tile_rows;
  p.n_tiles = (g.N + tile_cols - 1) / tile_cols;
  p.act = g.act;
  p.alpha = g.alpha;
  p.limit = g.limit;
  p.beta = g.beta;
  p.bias = g.bias;
  p.bias_words = aligned(g.bias, 16) ? 1 : 0;
  p.add = g.add;
  p.out = g.out;
  p.wide = g.N % 16 == 0 && aligned(g.out, 32) ? 1 : 0;
  p.g_out = g.g_out;
  p.g_in = g.g_in;
  p.colsum = g.colsum;
  p.status = g.status;
  p.clear_status = g.clear_status;
  p.b_early = g.b_early;
  p.wait_limit_ns = kWaitLimitNs;
  return p;
}

template <int BN, int CG, bool A_MN, bool B_MN, int EPI>
e4b_status launch_typed(const DenseGemmLaunch& g, int width, cudaStream_t s) {
  using C = Cfg<BN, CG>;
  auto kern = dense_gemm_kernel<BN, CG, A_MN, B_MN, EPI>;
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem(kern, C::SMEM_BYTES, allowed) != cudaSuccess) return E4B_ERR_CUDA;
  const int NT = EPI == kEpiGateUp ? width / 2 : width;
  CUtensorMap ta, tb;
  if (!encode_operands<A_MN, B_MN, EPI>(g, EPI == kEpiGateUp ? NT : width / CG, &ta, &tb)) return E4B_ERR_CUDA;
  const Params p = make_params(g, CG * BM, width, NT);
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int64_t slots = device_sm_count() / CG;
  const dim3 grid(static_cast<unsigned>(CG * (tiles < slots ? tiles : slots)));
  const cudaError_t e = CG == 2 ? launch_pdl_cluster(2, kern, grid, dim3(THREADS), C::SMEM_BYTES, s, ta, tb, p)
                                : launch_pdl(kern, grid, dim3(THREADS), C::SMEM_BYTES, s, ta, tb, p);
  return e == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

// Clusters of S split CTAs that fit the device at once (a GPC's SMs are not a multiple of every S); 0: refused.
template <bool A_MN, bool B_MN, int EPI>
int split_slots(int S) {
  using C = SplitCfg;
  auto kern = dense_split_kernel<A_MN, B_MN, EPI>;
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem(kern, C::SMEM_BYTES, allowed) != cudaSuccess) return 0;
  static std::atomic<int> cache[16][9];                 // + 1, so that 0 is "not asked yet"
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return 0;
  int n = cache[dev][S].load();
  if (n > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(S));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(S);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 0) n = 0;
  cache[dev][S].store(n + 1);
  return n;
}

template <bool A_MN, bool B_MN, int EPI>
e4b_status launch_split(const DenseGemmLaunch& g, int S, cudaStream_t s) {
  constexpr int NT = EPI == kEpiGateUp ? SplitCfg::BN / 2 : SplitCfg::BN;
  CUtensorMap ta, tb;
  if (!encode_operands<A_MN, B_MN, EPI>(g, NT, &ta, &tb, g.M <= BM / 2 ? BM / 2 : BM)) return E4B_ERR_CUDA;
  const Params p = make_params(g, BM, SplitCfg::BN, NT);
  if (g.colsum_rows) *g.colsum_rows = p.m_tiles * S;
  const dim3 grid(static_cast<unsigned>(p.m_tiles * p.n_tiles * S));
  return launch_pdl_cluster(static_cast<unsigned>(S), dense_split_kernel<A_MN, B_MN, EPI>, grid, dim3(SplitCfg::THREADS),
                            SplitCfg::SMEM_BYTES, s, ta, tb, p, S) == cudaSuccess
             ? E4B_OK
             : E4B_ERR_CUDA;
}

// Which kernel: estimated time in units of one 64-K step of a 256 x 256 pair
// tile (0.28 us on a B200).  A narrower pair tile costs nearly its share, so a
// width that fills the last wave of pairs may win over 256.  A step of a tile of
// one CTA, 128 rows high, costs 0.8 up to 128 columns (issue-bound) and grows to
// 1.4 at 256 (its loads): tiles of 160 to 256 columns stream a large B past few
// rows (gate and up of 4096 x 12288, 33 tokens: 192 columns 59.2 us with the
// down product, 128 columns, whose second wave is a third full, 68.6).  A 128-K
// step of the split kernel costs 1.7 (it waits for its loads), its exchange 2
// and 1 for each CTA of a cluster.  Behind another launch of the library it
// overlaps with that one's end only where clusters find room among its CTAs:
// large ones that fill the device do not (23 of 5 took 1.8 us more than 23 of 4).
enum Kind { kPair, kSingle, kSplit };
struct Choice {
  Kind kind;
  int value;        // columns per tile, or the cluster size of the split kernel
  double time;
};

template <bool A_MN, bool B_MN, int EPI>
Choice choose(const DenseGemmLaunch& g) {
  const int64_t sms = device_sm_count();
  auto tiles = [&](int rows, int cols) {
    const int nt = EPI == kEpiGateUp ? cols / 2 : cols;
    return (static_cast<int64_t>(g.M) + rows - 1) / rows * ((g.N + nt - 1) / nt);
  };
  auto waves = [](int64_t n, int64_t slots) { return static_cast<double>((n + slots - 1) / slots); };
  const int64_t k64 = (g.K + BK - 1) / BK, k128 = (g.K + 127) / 128, t128 = tiles(128, 128);
  Choice c{kPair, 256, waves(tiles(256, 256), sms / 2) * k64 + 4.0};
  for (int w = 224; w >= 160; w -= 32) {
    const double t = waves(tiles(256, w), sms / 2) * k64 * (0.1 + 0.9 * w / 256.0) + 4.0;
    if (t < 0.97 * c.time) c = Choice{kPair, w, t};
  }
  for (int w = 128; w <= 256; w += 32) {
    const double t = waves(tiles(128, w), sms) * k64 * (0.8 + 0.6 * (w - 128) / 128.0);
    if (w == 128 ? t <= c.time : t < 0.97 * c.time) c = Choice{kSingle, w, t};
  }
  for (int n = 2; n <= 8 && n <= k128 && t128 * n <= sms; ++n) {
    double t = static_cast<double>((k128 + n - 1) / n) * 1.7 + 2.0 + n;
    if (t >= c.time) continue;
    const int slots = split_slots<A_MN, B_MN, EPI>(n);
    if (g.b_early && n > 4 && t128 > 0.85 * slots) t += 3.0;
    if (t < c.time && t128 <= slots) c = Choice{kSplit, n, t};
  }
  return c;
}

template <bool A_MN, bool B_MN, int EPI>
e4b_status launch_width(const DenseGemmLaunch& g, cudaStream_t s) {
  const Choice c = choose<A_MN, B_MN, EPI>(g);
  if (c.kind == kSplit) return launch_split<A_MN, B_MN, EPI>(g, c.value, s);
  if (g.colsum_rows) *g.colsum_rows = (g.M + 31) / 32;
  if (c.kind == kPair) return launch_typed<256, 2, A_MN, B_MN, EPI>(g, c.value, s);
  return c.value == 128 ? launch_typed<128, 1, A_MN, B_MN, EPI>(g, 128, s)
                        : launch_typed<256, 1, A_MN, B_MN, EPI>(g, c.value, s);
}

}  // namespace

e4b_status launch_dense_gemm(const DenseGemmLaunch& g, cudaStream_t s) {
  switch (g.epi) {
    case kEpiGateUp: return launch_width<false, false, kEpiGateUp>(g, s);
    case kEpiDact: return launch_width<false, true, kEpiDact>(g, s);
    case kEpiLinear:
      if (g.a_mn && g.b_mn) return launch_width<true, true, kEpiLinear>(g, s);
      if (!g.a_mn && g.b_mn) return launch_width<false, true, kEpiLinear>(g, s);
      if (!g.a_mn && !g.b_mn) return launch_width<false, false, kEpiLinear>(g, s);
  }
  return E4B_ERR_UNSUPPORTED;
}

namespace {

// The tiles of every product on CTAs (CG 1) or pairs, and the launch's time in the units of choose(): the longest
// share that walk_tiles deals out.
template <int CG>
double plan_multi(const DenseGemmLaunch* g, int count, MultiParams& mp) {
  mp.count = count;
  mp.status = g[0].status;
  mp.wait_limit_ns = kWaitLimitNs;
  double total = 0.0, tiles = 0.0, cost[kMultiMax], before[kMultiMax];
  for (int i = 0; i < count; ++i) {
    MultiProblem& q = mp.p[i];
    q.M = g[i].M;
    q.N = g[i].N;
    q.K = g[i].K;
    q.n_tiles = (g[i].N + CG * 128 - 1) / (CG * 128);
    q.tiles = static_cast<int32_t>((static_cast<int64_t>(g[i].M) + CG * BM - 1) / (CG * BM) * q.n_tiles);
    q.a_mn = g[i].a_mn;
    q.out = g[i].out;
    q.wide = g[i].N % 16 == 0 && aligned(g[i].out, 32) ? 1 : 0;
    cost[i] = (g[i].K + BK - 1) / BK + kTileFixed;
    before[i] = total;
    total += cost[i] * q.tiles;
    tiles += q.tiles;
  }
  const int slots = device_sm_count() / CG, shares = tiles < slots ? static_cast<int>(tiles) : slots;
  double worst = 0.0, done[kMultiMax] = {};
  for (int s = 1; s <= shares; ++s) {
    double load = 0.0;
    for (int i = 0; i < count; ++i) {
      const double t = std::ceil((total * s / shares - before[i]) / cost[i] - 0.5);
      const double upto = t < 0.0 ? 0.0 : (t < mp.p[i].tiles ? t : mp.p[i].tiles);
      load += (upto - done[i]) * cost[i];
      done[i] = upto;
    }
    if (load > worst) worst = load;
  }
  return worst * (CG == 2 ? 1.0 : 0.8);
}

template <int CG>
e4b_status launch_multi(const DenseGemmLaunch* g, const MultiParams& mp, cudaStream_t s) {
  using C = Cfg<128 * CG, CG>;
  MultiMaps maps;
  int64_t tiles = 0;
  for (int i = 0; i < mp.count; ++i) {
    if (!(g[i].a_mn ? encode_operands<true, true, kEpiLinear>(g[i], 0, &maps.a[i], &maps.b[i])
                    : encode_operands<false, true, kEpiLinear>(g[i], 0, &maps.a[i], &maps.b[i])))
      return E4B_ERR_CUDA;
    tiles += mp.p[i].tiles;
  }
  for (int i = mp.count; i < kMultiMax; ++i) {
    maps.a[i] = maps.a[0];
    maps.b[i] = maps.b[0];
  }
  auto kern = dense_multi_kernel<CG>;
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem(kern, C::SMEM_BYTES, allowed) != cudaSuccess) return E4B_ERR_CUDA;
  const int64_t slots = device_sm_count() / CG;
  const dim3 grid(static_cast<unsigned>(CG * (tiles < slots ? tiles : slots)));
  const cudaError_t e = CG == 2 ? launch_pdl_cluster(2, kern, grid, dim3(THREADS), C::SMEM_BYTES, s, maps, mp)
                                : launch_pdl(kern, grid, dim3(THREADS), C::SMEM_BYTES, s, maps, mp);
  return e == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

}  // namespace

// Plain linear products (no bias, no addition, B row-contiguous) that depend on earlier launches only: in one launch,
// on CTAs or pairs, or one by one (which costs about 8 units for each launch), whichever should take least.  Against
// the best of the three the rule lost 0.5% in the mean over 42 sizes from 40 x 1024 x 512 to 3000 x 5120 x 1536.
e4b_status launch_dense_group(const DenseGemmLaunch* g, int count, const ColumnSums& sums, cudaStream_t s) {
  if (count > 1 && count <= kMultiMax) {
    double apart = 0.0;
    for (int i = 0; i < count; ++i)
      apart += 8.0 + (g[i].a_mn ? choose<true, true, kEpiLinear>(g[i]) : choose<false, true, kEpiLinear>(g[i])).time;
    if (sums.out_a || sums.out_b) apart += 8.0;
    MultiParams small = {}, pairs = {};
    small.sums = pairs.sums = sums;
    const double t1 = plan_multi<1>(g, count, small), t2 = plan_multi<2>(g, count, pairs);
    if (t1 < t2 && t1 < apart) return launch_multi<1>(g, small, s);
    if (t2 < apart) return launch_multi<2>(g, pairs, s);
  }
  for (int i = 0; i < count; ++i) {
    const e4b_status st = launch_dense_gemm(g[i], s);
    if (st != E4B_OK) return st;
  }
  return launch_column_sums(sums, s) == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

}  // namespace e4b
