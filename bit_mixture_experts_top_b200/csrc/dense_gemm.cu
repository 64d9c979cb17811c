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
// memory and issues the MMAs (M = 128 rows, N = BN columns, two accumulators),
// warps 4-11 run the epilogue of one tile while the next is multiplied.  Every
// wait is bounded (E4B_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int BM = 128;                  // rows of D per CTA
constexpr int BK = 64;                   // K per stage: one 128-byte swizzle row of bf16
constexpr int WARP_TMA = 0, WARP_MMA = 1, WARP_EPI0 = 4, EPI_WARPS = 8;
constexpr int THREADS = 32 * (WARP_EPI0 + EPI_WARPS);
constexpr uint64_t kDrainNs = 50000000ull;
constexpr int kGroupM = 16;              // row tiles that share a sweep over the columns (L2 reuse of both operands)

template <int BN, int CG>
struct Cfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = BN / CG;                      // this CTA's share of B
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 196608 / STAGE_BYTES;         // 4, 6 or 8 (pairs: 6)
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 5) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;     // + slack to align the base
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Params {
  int32_t M, N, K;          // D is M x N; gate_up: N = I features (2I rows of B)
  int32_t m_tiles, n_tiles;
  int32_t act;
  float alpha, limit, beta;
  const float* bias;        // gate_up: [2I]; linear: [N]; or null
  const uint16_t* add;      // linear: [M, N] bf16 or null
  uint16_t* out;            // bf16: h [M, I], D [M, N] or dG [M, 2I]
  float* g_out;             // gate_up: G [M, 2I] fp32 or null
  const float* g_in;        // dact: G [M, 2I]
  float* colsum;            // dact: [ceil(M / 32), 2I] column sums of dG per 32 rows, or null
  int32_t* status;
  int32_t clear_status;     // this launch is the first of its call: block 0 clears the status words
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

__device__ __forceinline__ void store8(uint16_t* o, const float* f) {
  *reinterpret_cast<uint4*>(o) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// d(act)/d(gate) and d(act)/d(up); the clamps pass the gradient inside their range, ends included.
__device__ __forceinline__ void act_grads(const Params& p, float gate, float up, float& dg, float& du) {
  if (p.act == E4B_ACT_CLAMPED_GLU) {
    const float g = fminf(gate, p.limit);
    const float u = fminf(fmaxf(up, -p.limit), p.limit);
    const float s = __fdividef(1.0f, 1.0f + __expf(-p.alpha * g));
    const float df = s * (1.0f + p.alpha * g * (1.0f - s));
    dg = gate <= p.limit ? df * (u + p.beta) : 0.0f;
    du = (up >= -p.limit && up <= p.limit) ? g * s : 0.0f;
    return;
  }
  const float s = __fdividef(1.0f, 1.0f + __expf(-gate));
  dg = up * s * (1.0f + gate * (1.0f - s));
  du = gate * s;
}

// Sums 16 values per lane over the warp by halving: each step a lane keeps half
// of its columns and hands over the rest, 16 shuffles in all.  Lane l ends with
// the sum of column (l >> 1) with its bits reversed in the order kept below.
__device__ __forceinline__ float warp_column_sum16(float (&v)[16], int lane, int& col) {
  col = 0;
#pragma unroll
  for (int h = 8; h >= 1; h >>= 1) {
    const bool upper = lane & (2 * h);
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = upper ? v[i + h] : v[i];
      const float give = upper ? v[i] : v[i + h];
      v[i] = keep + __shfl_xor_sync(kFull, give, 2 * h);
    }
    col += upper ? h : 0;
  }
  return v[0] + __shfl_xor_sync(kFull, v[0], 1);
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
  constexpr int NT = EPI == kEpiGateUp ? BN / 2 : BN;   // output columns (features) per tile
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
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * C::STAGE_BYTES);
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
          const int nb = n0 + static_cast<int>(rank) * C::B_ROWS;
          if constexpr (EPI == kEpiGateUp && CG == 2) {  // gate rows in one CTA, the matching up rows in the other
            load(b, &tm_b, k0, rank == 0 ? n0 : p.N + n0);
          } else if constexpr (EPI == kEpiGateUp) {      // gate rows, then the matching up rows
            load(b, &tm_b, k0, n0);
            load(b + NT * BK * 2, &tm_b, k0, p.N + n0);
          } else if constexpr (B_MN) {
#pragma unroll
            for (int i = 0; i < C::B_ROWS / 64; ++i) load(b + i * 8192, &tm_b, nb + 64 * i, k0);
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
      constexpr uint32_t idesc = idesc_bf16_f32(CG * BM, BN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
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
    const int half = (warp - WARP_EPI0) >> 2;      // this warp's half of the columns
    int it = 0;
    for (int tile = first; tile < total; tile += step, ++it) {
      int mt, nt;
      tile_at(p, tile, mt, nt);
      const int buf = it & 1;
      const uint32_t aphase = (it >> 1) & 1;
      if (!mbar_wait_sleep(&acc_full[buf], aphase, wctx, 1401, 64)) break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * BN);
      const int row0 = (mt * CG + static_cast<int>(rank)) * BM + 32 * q;
      const int row = row0 + lane;
      const bool row_in = row < p.M;
#pragma unroll 1
      for (int c0 = half * (NT / 2); c0 < (half + 1) * (NT / 2); c0 += 16) {
        const int col = nt * NT + c0;
        if (col >= p.N) break;
        if constexpr (EPI == kEpiGateUp) {
          uint32_t g[16], u[16];
          tmem_ld_32x32b_x16(taddr + c0, g);
          tmem_ld_32x32b_x16(taddr + NT + c0, u);
          tmem_ld_wait();
          const Epilogue ep{nullptr, p.act, p.alpha, p.limit, p.beta};
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            if (col + j >= p.N) break;
            float fg[8], fu[8], h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              fg[i] = __uint_as_float(g[j + i]) + (p.bias ? __ldg(p.bias + col + j + i) : 0.0f);
              fu[i] = __uint_as_float(u[j + i]) + (p.bias ? __ldg(p.bias + p.N + col + j + i) : 0.0f);
              h[i] = expert_act(ep, fg[i], fu[i]);
            }
            if (row_in) {
              store8(p.out + static_cast<int64_t>(row) * p.N + col + j, h);
              if (p.g_out) {
                float4* go = reinterpret_cast<float4*>(p.g_out + static_cast<int64_t>(row) * 2 * p.N + col + j);
                go[0] = make_float4(fg[0], fg[1], fg[2], fg[3]);
                go[1] = make_float4(fg[4], fg[5], fg[6], fg[7]);
                go = reinterpret_cast<float4*>(p.g_out + static_cast<int64_t>(row) * 2 * p.N + p.N + col + j);
                go[0] = make_float4(fu[0], fu[1], fu[2], fu[3]);
                go[1] = make_float4(fu[4], fu[5], fu[6], fu[7]);
              }
            }
          }
        } else if constexpr (EPI == kEpiLinear) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            if (col + j >= p.N) break;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              f[i] = __uint_as_float(r[j + i]) + (p.bias ? __ldg(p.bias + col + j + i) : 0.0f);
            if (row_in) {
              const int64_t at = static_cast<int64_t>(row) * p.N + col + j;
              if (p.add) {
                const uint4 a = *reinterpret_cast<const uint4*>(p.add + at);
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  f[2 * i] += __uint_as_float(w[i] << 16);
                  f[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
                }
              }
              store8(p.out + at, f);
            }
          }
        } else {
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + c0, r);
          tmem_ld_wait();
          float dg[16], du[16];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            float4 fg = make_float4(0.f, 0.f, 0.f, 0.f), fu = fg;
            if (row_in && col + j < p.N) {
              const float* gp = p.g_in + static_cast<int64_t>(row) * 2 * p.N + col + j;
              fg = *reinterpret_cast<const float4*>(gp);
              fu = *reinterpret_cast<const float4*>(gp + p.N);
            }
            const float gv[4] = {fg.x, fg.y, fg.z, fg.w}, uv[4] = {fu.x, fu.y, fu.z, fu.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              act_grads(p, gv[i], uv[i], dg[j + i], du[j + i]);
              const float dh = __uint_as_float(r[j + i]);          // 0 in rows past M
              dg[j + i] = row_in ? dg[j + i] * dh : 0.0f;
              du[j + i] = row_in ? du[j + i] * dh : 0.0f;
            }
          }
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            if (row_in && col + j < p.N) {
              uint16_t* o = p.out + static_cast<int64_t>(row) * 2 * p.N + col + j;
              store8(o, dg + j);
              store8(o + p.N, du + j);
            }
          }
          if (p.colsum) {                         // from the fp32 values, before their rounding to bf16
            float* o = p.colsum + static_cast<int64_t>(row0 / 32) * 2 * p.N;
            int c;
            const float sg = warp_column_sum16(dg, lane, c);
            const float su = warp_column_sum16(du, lane, c);
            if ((lane & 1) == 0 && col + c < p.N && row0 < p.M) {
              o[col + c] = sg;
              o[p.N + col + c] = su;
            }
          }
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

// ---------------------------------------------------------------------- host side

template <int BN, int CG, bool A_MN, bool B_MN, int EPI>
e4b_status launch_typed(const DenseGemmLaunch& g, cudaStream_t s) {
  using C = Cfg<BN, CG>;
  auto kern = dense_gemm_kernel<BN, CG, A_MN, B_MN, EPI>;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [&] {
    attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  });
  if (attr_err != cudaSuccess) return E4B_ERR_CUDA;
  constexpr int NT = EPI == kEpiGateUp ? BN / 2 : BN;
  const uint64_t b_rows = EPI == kEpiGateUp ? 2 * static_cast<uint64_t>(g.N) : g.N;
  CUtensorMap ta, tb;
  // K-contiguous: [rows, K], boxes of 64 K x tile rows; M/N-contiguous: [K, rows], boxes of 64 rows x 64 K
  const bool ok_a = A_MN ? encode_tma_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.a, g.M, g.K,
                                         static_cast<uint64_t>(g.M) * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B)
                         : encode_tma_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.a, g.K, g.M,
                                         static_cast<uint64_t>(g.K) * 2, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B);
  const bool ok_b = B_MN ? encode_tma_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.b, b_rows, g.K, b_rows * 2, 64, BK,
                                         CU_TENSOR_MAP_SWIZZLE_128B)
                         : encode_tma_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.b, g.K, b_rows,
                                         static_cast<uint64_t>(g.K) * 2, BK, EPI == kEpiGateUp ? NT : C::B_ROWS,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok_a || !ok_b) return E4B_ERR_CUDA;
  Params p;
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.m_tiles = (g.M + CG * BM - 1) / (CG * BM);
  p.n_tiles = (g.N + NT - 1) / NT;
  p.act = g.act;
  p.alpha = g.alpha;
  p.limit = g.limit;
  p.beta = g.beta;
  p.bias = g.bias;
  p.add = g.add;
  p.out = g.out;
  p.g_out = g.g_out;
  p.g_in = g.g_in;
  p.colsum = g.colsum;
  p.status = g.status;
  p.clear_status = g.clear_status;
  p.wait_limit_ns = kWaitLimitNs;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int64_t slots = device_sm_count() / CG;
  const dim3 grid(static_cast<unsigned>(CG * (tiles < slots ? tiles : slots)));
  const cudaError_t e = CG == 2 ? launch_pdl_cluster(2, kern, grid, dim3(THREADS), C::SMEM_BYTES, s, ta, tb, p)
                                : launch_pdl(kern, grid, dim3(THREADS), C::SMEM_BYTES, s, ta, tb, p);
  return e == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

// Pairs where every pair of SMs gets a 256 x 256 tile; else the widest single-CTA tile that
// still gives every SM one: narrower ones spread a small product.
template <bool A_MN, bool B_MN, int EPI>
e4b_status launch_width(const DenseGemmLaunch& g, cudaStream_t s) {
  const int64_t mt = (g.M + BM - 1) / BM, sms = device_sm_count();
  auto tiles = [&](int bn) {
    const int nt = EPI == kEpiGateUp ? bn / 2 : bn;
    return mt * ((g.N + nt - 1) / nt);
  };
  if ((mt + 1) / 2 * (tiles(256) / mt) >= sms / 2) return launch_typed<256, 2, A_MN, B_MN, EPI>(g, s);
  if (tiles(128) >= sms) return launch_typed<128, 1, A_MN, B_MN, EPI>(g, s);
  return launch_typed<64, 1, A_MN, B_MN, EPI>(g, s);
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

}  // namespace e4b
