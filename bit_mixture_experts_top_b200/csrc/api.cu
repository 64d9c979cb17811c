// C ABI of the library: argument validation, workspace layout and the launch
// sequence of the layer forward (route -> gather -> gate_up -> down -> combine).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "e4b.h"
#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {

int device_sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev < 64) cache[dev] = n;
  return n;
}

// (function-local, so that it is there for whichever source file registers first)
struct WaitFlags {
  cudaError_t (*address[32])(void**);
  int count;
};

static WaitFlags& wait_flags() {
  static WaitFlags f = {};
  return f;
}

bool register_wait_flag(cudaError_t (*address)(void**)) {
  WaitFlags& f = wait_flags();
  if (f.count == 32) return false;
  f.address[f.count++] = address;
  return true;
}

namespace {

__global__ void wait_timeout_probe_kernel(int32_t* status, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int32_t abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtx w{&abort_flag, status, limit_ns};
  if (threadIdx.x == 0) (void)mbar_wait(&bar, 0, w, 9001);   // nothing ever arrives
  __syncthreads();
}

struct ForwardLayout {
  size_t status, topk_ids, topk_w, offsets, chunk_off, block_counts, sorted_slot, slot_pos, x_sorted, xa, h, y;
  size_t gu_absmax, dn_absmax;   // expanded double-quantised absmax (E4B_NF4_DQ only)
  size_t total;
};

// Absmax values of one stack [E, N, K] (one per 64 weights).
size_t absmax_count(const e4b_moe_desc& d, bool gate_up) {
  return static_cast<size_t>(d.E) * (gate_up ? 2 * static_cast<size_t>(d.I) : d.H) *
         (gate_up ? d.H : d.I) / 64;
}

// The format the GEMM kernels see: a double-quantised stack runs as NF4 on its expanded absmax.
int32_t gemm_format(int32_t format) { return format == E4B_NF4_DQ ? E4B_NF4 : format; }

// A nested-form absmax description: every array present, the fp32 ones 4-byte aligned.
bool valid_dq(const e4b_nf4_dq* q) {
  return q && q->codes && q->absmax2 && q->offset && q->table && aligned(q->absmax2, 4) && aligned(q->offset, 4) &&
         aligned(q->table, 4);
}

ForwardLayout forward_layout(const e4b_moe_desc& d, int32_t T) {
  const size_t R = static_cast<size_t>(T) * d.k;
  const size_t nblk = static_cast<size_t>(route_blocks(T) > 0 ? route_blocks(T) : 1);
  ForwardLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.status = take(kStatusBytes);
  L.topk_ids = take(R * 4);
  L.topk_w = take(R * 4);
  L.offsets = take((d.E + 1) * 4);
  L.chunk_off = take((d.E + 1) * 4);
  L.block_counts = take(nblk * d.E * 4);
  L.sorted_slot = take(R * 4);
  L.slot_pos = take(R * 4);
  L.x_sorted = take(R * d.H * 2);
  L.xa = take(d.lora_rank > 0 ? R * 128 : 0);
  L.h = take(R * d.I * 2);
  L.y = take(R * d.H * 4);
  const bool dq = d.format == E4B_NF4_DQ;
  L.gu_absmax = take(dq ? absmax_count(d, true) * 4 : 0);
  L.dn_absmax = take(dq ? absmax_count(d, false) * 4 : 0);
  L.total = o;
  return L;
}

// The training workspace: the forward's layout, then what the backward needs
// besides it (the saved pre-activation G) and its own scratch.
struct TrainLayout {
  ForwardLayout fwd;
  size_t g, dY, dG, dxa, dX, total;
};

TrainLayout train_layout(const e4b_moe_desc& d, int32_t T) {
  TrainLayout L;
  L.fwd = forward_layout(d, T);
  const size_t R = static_cast<size_t>(T) * d.k;
  size_t o = L.fwd.total;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.g = take(R * 2 * d.I * 4);
  L.dY = take(R * d.H * 2);
  L.dG = take(R * 2 * d.I * 2);
  L.dxa = take(d.lora_rank > 0 ? R * 16 * 4 : 0);
  L.dX = take(R * d.H * 4);
  L.total = o;
  return L;
}

struct RouteLayout {
  size_t status, block_counts, slot_pos, total;
};

RouteLayout route_layout(int32_t T, int32_t E, int32_t k) {
  const size_t nblk = static_cast<size_t>(route_blocks(T) > 0 ? route_blocks(T) : 1);
  RouteLayout L;
  size_t o = 0;
  L.status = o;
  o += align_up(kStatusBytes);
  L.block_counts = o;
  o += align_up(nblk * E * 4);
  L.slot_pos = o;
  o += align_up(static_cast<size_t>(T) * k * 4);
  L.total = o;
  return L;
}

e4b_status validate_desc(const e4b_moe_desc* d, int32_t T) {
  if (!d || T < 0) return E4B_ERR_INVALID_ARG;
  if (d->E < 1 || d->E > kMaxExperts || d->k < 1 || d->k > d->E || d->k > kMaxTopK) return E4B_ERR_UNSUPPORTED;
  if (d->H < 64 || d->H % 64 != 0 || d->I < 64 || d->I % 64 != 0) return E4B_ERR_UNSUPPORTED;
  if (d->format != E4B_NF4 && d->format != E4B_MXFP4 && d->format != E4B_NF4_DQ) return E4B_ERR_UNSUPPORTED;
  if (d->act != E4B_ACT_SWIGLU && d->act != E4B_ACT_CLAMPED_GLU) return E4B_ERR_UNSUPPORTED;
  if (d->act == E4B_ACT_CLAMPED_GLU &&
      (!std::isfinite(d->glu_alpha) || !std::isfinite(d->glu_beta) || !(d->glu_limit > 0.0f)))
    return E4B_ERR_INVALID_ARG;
  if (d->lora_rank < 0 || d->lora_rank > kMaxLoraRank) return E4B_ERR_UNSUPPORTED;
  if (d->gating != E4B_GATE_SOFTMAX_TOPK && d->gating != E4B_GATE_SOFTMAX_ALL) return E4B_ERR_INVALID_ARG;
  const int tpt = d->tokens_per_tile;
  const int32_t gf = gemm_format(d->format);
  if (tpt == 8 && !(skinny_gemm_supported(d->H, gf) && skinny_gemm_supported(d->I, gf)))
    return E4B_ERR_UNSUPPORTED;
  if (tpt != 0 && tpt != 8 && tpt != 32 && tpt != 64 && tpt != 128 && tpt != 192 && tpt != 256) return E4B_ERR_UNSUPPORTED;
  const int64_t R = static_cast<int64_t>(T) * d->k;
  if (R > (int64_t(1) << 30)) return E4B_ERR_UNSUPPORTED;
  // TMA row coordinates are 32-bit: E * 2I rows of codes must fit.
  if (static_cast<int64_t>(d->E) * 2 * d->I >= (int64_t(1) << 31)) return E4B_ERR_UNSUPPORTED;
  return E4B_OK;
}

struct KernelChoice {
  bool decode;        // skinny_gemm (decode kernel) or grouped_gemm (tcgen05 tiles)
  int32_t tokens;     // decode: tokens per chunk; tcgen05: tile width
};

// Mean routed rows per active expert decides: a handful per expert -> the decode
// kernel (weight-stream bound), with chunks of 8, 16 or 32 tokens so that one
// decoded weight fragment serves up to 32 tokens; more -> the smallest tcgen05
// tile that holds most experts' rows in one chunk, 256 for prefill (each
// dequantised weight stage then feeds the most tokens).
KernelChoice pick_kernel(const e4b_moe_desc& d, int32_t T) {
  const int64_t R = static_cast<int64_t>(T) * d.k;
  const int64_t active = R < d.E ? R : d.E;
  const int64_t avg = active > 0 ? (R + active - 1) / active : 1;
  const int32_t gf = gemm_format(d.format);
  const bool decode_ok = skinny_gemm_supported(d.H, gf) && skinny_gemm_supported(d.I, gf);
  const int32_t chunk = avg <= 8 ? 8 : (avg <= 16 ? 16 : 32);
  if (d.tokens_per_tile == 8) return {true, chunk};
  if (d.tokens_per_tile) return {false, d.tokens_per_tile};
  if (avg <= kDecodeMaxRows && decode_ok) return {true, chunk};
  if (avg <= 16) return {false, 32};
  if (avg <= 48) return {false, 64};
  if (avg <= 96) return {false, 128};
  return {false, 256};
}

// A byte range of device memory, for the overlap checks of calls that allow some buffers to coincide.
struct Range {
  uintptr_t lo, hi;
};

Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, p ? a + bytes : a};
}

bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

bool same_or_apart(const Range& a, const Range& b) { return !overlap(a, b) || (a.lo == b.lo && a.hi == b.hi); }

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + off);
}

}  // namespace
}  // namespace e4b

using namespace e4b;

extern "C" {

int32_t e4b_abi_version(void) { return E4B_ABI_VERSION; }

const char* e4b_status_string(int32_t status) {
  switch (status) {
    case E4B_OK: return "E4B_OK";
    case E4B_ERR_INVALID_ARG: return "E4B_ERR_INVALID_ARG: bad pointer, size, alignment or workspace";
    case E4B_ERR_UNSUPPORTED: return "E4B_ERR_UNSUPPORTED: shape or option outside what the kernels implement";
    case E4B_ERR_CUDA: return "E4B_ERR_CUDA: a CUDA call or kernel launch failed";
    case E4B_ERR_TIMEOUT: return "E4B_ERR_TIMEOUT: a bounded device-side wait ran out";
    default: return "E4B_ERR_UNKNOWN";
  }
}

void e4b_nf4_codebook(float* out) {
  if (!out) return;
  std::memcpy(out, nf4_table().level, sizeof(float) * 16);
}

e4b_status e4b_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t n, uint16_t* out,
                             e4b_stream stream) {
  if (n < 0 || n % 32 != 0) return E4B_ERR_INVALID_ARG;
  if (n == 0) return E4B_OK;
  if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(out, 16)) return E4B_ERR_INVALID_ARG;
  return launch_dequant_mxfp4(codes, scales, n, out, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? E4B_OK
             : E4B_ERR_CUDA;
}

e4b_status e4b_expand_absmax_dq(const e4b_nf4_dq* dq, int64_t n, float* out, e4b_stream stream) {
  if (n < 0) return E4B_ERR_INVALID_ARG;
  if (n == 0) return E4B_OK;
  if (!valid_dq(dq) || !out || !aligned(out, 4)) return E4B_ERR_INVALID_ARG;
  return launch_expand_absmax_dq(dq->codes, dq->absmax2, dq->offset, dq->table, n, n, nullptr, out,
                                 reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? E4B_OK
             : E4B_ERR_CUDA;
}

e4b_status e4b_deinterleave_rows(const void* in, void* out, int32_t E, int32_t I, int64_t row_bytes,
                                 e4b_stream stream) {
  if (E < 0 || I < 0 || row_bytes < 0) return E4B_ERR_INVALID_ARG;
  const int64_t bytes = static_cast<int64_t>(E) * 2 * I * row_bytes;
  if (bytes == 0) return E4B_OK;
  if (!in || !out) return E4B_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  if (a < b + static_cast<uintptr_t>(bytes) && b < a + static_cast<uintptr_t>(bytes)) return E4B_ERR_INVALID_ARG;
  return launch_deinterleave_rows(in, out, E, I, row_bytes, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? E4B_OK
             : E4B_ERR_CUDA;
}

e4b_status e4b_quantize_nf4(const float* x, int64_t n, uint8_t* codes, float* absmax, e4b_stream stream) {
  if (n < 0 || n % 64 != 0) return E4B_ERR_INVALID_ARG;
  if (n == 0) return E4B_OK;
  if (!x || !codes || !absmax || !aligned(x, 16) || !aligned(codes, 4) || !aligned(absmax, 4))
    return E4B_ERR_INVALID_ARG;
  return launch_quantize_nf4(x, n, codes, absmax, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? E4B_OK
             : E4B_ERR_CUDA;
}

size_t e4b_route_workspace_bytes(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > E || k > kMaxTopK) return 0;
  return route_layout(T, E, k).total;
}

e4b_status e4b_route(const uint16_t* logits, int32_t T, int32_t E, int32_t k, int32_t gating, int32_t* topk_ids,
                     float* topk_w,
                     int32_t* expert_offsets, int32_t* sorted_slot, void* ws, size_t ws_bytes,
                     e4b_stream stream) {
  if (T < 0 || E < 1 || k < 1 || k > E) return E4B_ERR_INVALID_ARG;
  if (gating != E4B_GATE_SOFTMAX_TOPK && gating != E4B_GATE_SOFTMAX_ALL) return E4B_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > kMaxTopK) return E4B_ERR_UNSUPPORTED;
  if (!expert_offsets || !ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !topk_w || !sorted_slot)) return E4B_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * k > (int64_t(1) << 30)) return E4B_ERR_UNSUPPORTED;
  const RouteLayout L = route_layout(T, E, k);
  if (ws_bytes < L.total) return E4B_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  RouteBuffers b;
  b.status = at<int32_t>(ws, L.status);
  b.done_counter = reinterpret_cast<uint32_t*>(b.status + 2);
  b.topk_ids = topk_ids;
  b.topk_w = topk_w;
  b.expert_offsets = expert_offsets;
  b.chunk_off = nullptr;
  b.block_counts = at<int32_t>(ws, L.block_counts);
  b.sorted_slot = sorted_slot;
  b.slot_pos = at<int32_t>(ws, L.slot_pos);
  // the status words are zeroed by the launch sequence (in-kernel for one routing block)
  return launch_route(logits, T, E, k, gating, 0, b, b.status, s) == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

size_t e4b_moe_workspace_bytes(const e4b_moe_desc* d, int32_t T) {
  if (validate_desc(d, T) != E4B_OK) return 0;
  return forward_layout(*d, T).total;
}

e4b_status e4b_moe_workspace_region(const e4b_moe_desc* d, int32_t T, int32_t region, size_t* offset,
                                    size_t* bytes) {
  const e4b_status v = validate_desc(d, T);
  if (v != E4B_OK) return v;
  if (!offset || !bytes) return E4B_ERR_INVALID_ARG;
  const ForwardLayout L = forward_layout(*d, T);
  const size_t R = static_cast<size_t>(T) * d->k;
  switch (region) {
    case E4B_WS_TOPK_IDS: *offset = L.topk_ids; *bytes = R * 4; break;
    case E4B_WS_TOPK_W: *offset = L.topk_w; *bytes = R * 4; break;
    case E4B_WS_EXPERT_OFFSETS: *offset = L.offsets; *bytes = (d->E + 1) * 4; break;
    case E4B_WS_SORTED_SLOT: *offset = L.sorted_slot; *bytes = R * 4; break;
    case E4B_WS_X_SORTED: *offset = L.x_sorted; *bytes = R * d->H * 2; break;
    case E4B_WS_H: *offset = L.h; *bytes = R * d->I * 2; break;
    case E4B_WS_Y: *offset = L.y; *bytes = R * d->H * 4; break;
    case E4B_WS_GU_ABSMAX:
      *offset = L.gu_absmax;
      *bytes = d->format == E4B_NF4_DQ ? absmax_count(*d, true) * 4 : 0;
      break;
    case E4B_WS_DN_ABSMAX:
      *offset = L.dn_absmax;
      *bytes = d->format == E4B_NF4_DQ ? absmax_count(*d, false) * 4 : 0;
      break;
    default: return E4B_ERR_INVALID_ARG;
  }
  return E4B_OK;
}

static e4b_status run_stages(int32_t first, int32_t last, const e4b_moe_desc* d, int32_t T, const uint16_t* x,
                             const uint16_t* logits, const uint8_t* gu_codes, const void* gu_scales,
                             const uint8_t* dn_codes, const void* dn_scales, const uint16_t* lora_A,
                             const uint16_t* lora_B, const float* gu_bias, const float* dn_bias, uint16_t* out,
                             void* ws, size_t ws_bytes, e4b_stream stream, bool train = false) {
  const e4b_status v = validate_desc(d, T);
  if (v != E4B_OK) return v;
  if (first < E4B_STAGE_ROUTE || last > E4B_STAGE_COMBINE || first > last) return E4B_ERR_INVALID_ARG;
  const bool lora = d->lora_rank > 0;
  if ((lora_A != nullptr) != lora || (lora_B != nullptr) != lora) return E4B_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  const ForwardLayout L = forward_layout(*d, T);
  if (ws_bytes < (train ? train_layout(*d, T).total : L.total)) return E4B_ERR_INVALID_ARG;
  const bool dq = d->format == E4B_NF4_DQ;
  if (T > 0) {
    if (!x || !logits || !gu_codes || !gu_scales || !dn_codes || !dn_scales || !out) return E4B_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(gu_codes, 16) || !aligned(dn_codes, 16))
      return E4B_ERR_INVALID_ARG;
    if (dq ? !(valid_dq(static_cast<const e4b_nf4_dq*>(gu_scales)) && valid_dq(static_cast<const e4b_nf4_dq*>(dn_scales)))
           : !(aligned(gu_scales, 16) && aligned(dn_scales, 16)))
      return E4B_ERR_INVALID_ARG;
    if (lora && (!aligned(lora_A, 2) || !aligned(lora_B, 2))) return E4B_ERR_INVALID_ARG;
    if ((gu_bias && !aligned(gu_bias, 4)) || (dn_bias && !aligned(dn_bias, 4))) return E4B_ERR_INVALID_ARG;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const KernelChoice kc = pick_kernel(*d, T);
  const int32_t tpt = kc.tokens;
  const int32_t R = T * d->k;

  RouteBuffers b;
  b.status = at<int32_t>(ws, L.status);
  b.done_counter = reinterpret_cast<uint32_t*>(b.status + 2);
  b.topk_ids = at<int32_t>(ws, L.topk_ids);
  b.topk_w = at<float>(ws, L.topk_w);
  b.expert_offsets = at<int32_t>(ws, L.offsets);
  b.chunk_off = at<int32_t>(ws, L.chunk_off);
  b.block_counts = at<int32_t>(ws, L.block_counts);
  b.sorted_slot = at<int32_t>(ws, L.sorted_slot);
  b.slot_pos = at<int32_t>(ws, L.slot_pos);
  uint16_t* x_sorted = at<uint16_t>(ws, L.x_sorted);
  uint16_t* xa = lora ? at<uint16_t>(ws, L.xa) : nullptr;
  uint16_t* h = at<uint16_t>(ws, L.h);
  float* y = at<float>(ws, L.y);
  float* gu_absmax = at<float>(ws, L.gu_absmax);
  float* dn_absmax = at<float>(ws, L.dn_absmax);

  GroupedGemmLaunch g;
  g.fmt = gemm_format(d->format);
  g.E = d->E;
  g.I = d->I;
  g.R = R;
  g.tokens_per_tile = tpt;
  g.decode = kc.decode ? 1 : 0;
  g.expert_offsets = b.expert_offsets;
  g.chunk_off = b.chunk_off;
  g.status = b.status;
  g.wait_limit_ns = kWaitLimitNs;
  g.glu = d->act;
  g.glu_alpha = d->glu_alpha;
  g.glu_limit = d->glu_limit;
  g.glu_beta = d->glu_beta;
  g.g_out = nullptr;
  float* g_keep = train ? at<float>(ws, train_layout(*d, T).g) : nullptr;

  for (int32_t stage = first; stage <= last; ++stage) {
    switch (stage) {
      case E4B_STAGE_ROUTE:
        // zeroes the status words first (in the routing kernel when one block routes)
        if (launch_route(logits, T, d->E, d->k, d->gating, tpt, b, b.status, s) != cudaSuccess) return E4B_ERR_CUDA;
        break;
      case E4B_STAGE_GATHER:
        if (launch_gather(x, d->H, d->k, R, b.sorted_slot, b.topk_ids, d->E, x_sorted, lora_A, d->lora_rank,
                          d->lora_scale, xa, s) != cudaSuccess)
          return E4B_ERR_CUDA;
        if (dq && T > 0) {   // the touched experts' absmax, expanded to fp32 for this forward
          const e4b_nf4_dq* gq = static_cast<const e4b_nf4_dq*>(gu_scales);
          const e4b_nf4_dq* dqs = static_cast<const e4b_nf4_dq*>(dn_scales);
          const size_t ng = absmax_count(*d, true), nd = absmax_count(*d, false);
          if (launch_expand_absmax_dq(gq->codes, gq->absmax2, gq->offset, gq->table, ng, ng / d->E,
                                      b.expert_offsets, gu_absmax, s) != cudaSuccess ||
              launch_expand_absmax_dq(dqs->codes, dqs->absmax2, dqs->offset, dqs->table, nd, nd / d->E,
                                      b.expert_offsets, dn_absmax, s) != cudaSuccess)
            return E4B_ERR_CUDA;
        }
        break;
      case E4B_STAGE_GATE_UP: {
        g.mode = 0;
        g.N = 2 * d->I;
        g.K = d->H;
        g.codes = gu_codes;
        g.scales = dq ? static_cast<const void*>(gu_absmax) : gu_scales;
        g.act = x_sorted;
        g.xa = xa;
        g.lora_B = lora_B;
        g.lora_rank = d->lora_rank;
        g.bias = gu_bias;
        g.out = h;
        g.g_out = g_keep;
        const e4b_status st = kc.decode ? launch_skinny_gemm(g, s) : launch_grouped_gemm(g, s);
        if (st != E4B_OK) return st;
        break;
      }
      case E4B_STAGE_DOWN: {
        g.mode = 1;
        g.N = d->H;
        g.K = d->I;
        g.codes = dn_codes;
        g.scales = dq ? static_cast<const void*>(dn_absmax) : dn_scales;
        g.act = h;
        g.xa = nullptr;
        g.lora_B = nullptr;
        g.lora_rank = 0;
        g.bias = dn_bias;
        g.out = y;
        g.g_out = nullptr;
        const e4b_status st = kc.decode ? launch_skinny_gemm(g, s) : launch_grouped_gemm(g, s);
        if (st != E4B_OK) return st;
        break;
      }
      case E4B_STAGE_COMBINE:
        if (launch_combine(y, b.topk_w, b.slot_pos, T, d->k, d->H, out, s) != cudaSuccess) return E4B_ERR_CUDA;
        break;
    }
  }
  return E4B_OK;
}

e4b_status e4b_moe_forward(const e4b_moe_desc* d, int32_t T, const uint16_t* x, const uint16_t* logits,
                           const uint8_t* gu_codes, const void* gu_scales, const uint8_t* dn_codes,
                           const void* dn_scales, const uint16_t* lora_A, const uint16_t* lora_B,
                           const float* gu_bias, const float* dn_bias, uint16_t* out, void* ws, size_t ws_bytes,
                           e4b_stream stream) {
  return run_stages(E4B_STAGE_ROUTE, E4B_STAGE_COMBINE, d, T, x, logits, gu_codes, gu_scales, dn_codes, dn_scales,
                    lora_A, lora_B, gu_bias, dn_bias, out, ws, ws_bytes, stream);
}

e4b_status e4b_moe_forward_stage(int32_t stage, const e4b_moe_desc* d, int32_t T, const uint16_t* x,
                                 const uint16_t* logits, const uint8_t* gu_codes, const void* gu_scales,
                                 const uint8_t* dn_codes, const void* dn_scales, const uint16_t* lora_A,
                                 const uint16_t* lora_B, const float* gu_bias, const float* dn_bias, uint16_t* out,
                                 void* ws, size_t ws_bytes, e4b_stream stream) {
  return run_stages(stage, stage, d, T, x, logits, gu_codes, gu_scales, dn_codes, dn_scales, lora_A, lora_B, gu_bias,
                    dn_bias, out, ws, ws_bytes, stream);
}

size_t e4b_moe_train_workspace_bytes(const e4b_moe_desc* d, int32_t T) {
  if (validate_desc(d, T) != E4B_OK) return 0;
  return train_layout(*d, T).total;
}

e4b_status e4b_moe_forward_train(const e4b_moe_desc* d, int32_t T, const uint16_t* x, const uint16_t* logits,
                                 const uint8_t* gu_codes, const void* gu_scales, const uint8_t* dn_codes,
                                 const void* dn_scales, const uint16_t* lora_A, const uint16_t* lora_B,
                                 const float* gu_bias, const float* dn_bias, uint16_t* out, void* ws,
                                 size_t ws_bytes, e4b_stream stream) {
  return run_stages(E4B_STAGE_ROUTE, E4B_STAGE_COMBINE, d, T, x, logits, gu_codes, gu_scales, dn_codes, dn_scales,
                    lora_A, lora_B, gu_bias, dn_bias, out, ws, ws_bytes, stream, true);
}

e4b_status e4b_moe_backward(const e4b_moe_desc* d, int32_t T, const uint16_t* logits, const uint16_t* dout,
                            const uint8_t* gu_codes, const void* gu_scales, const uint8_t* dn_codes,
                            const void* dn_scales, const uint16_t* lora_A, const uint16_t* lora_B, float* dx,
                            float* dlogits, float* dA, float* dB, void* ws, size_t ws_bytes, e4b_stream stream) {
  const e4b_status v = validate_desc(d, T);
  if (v != E4B_OK) return v;
  const bool lora = d->lora_rank > 0;
  if ((lora_A != nullptr) != lora || (lora_B != nullptr) != lora || (dA != nullptr) != lora ||
      (dB != nullptr) != lora)
    return E4B_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  const TrainLayout L = train_layout(*d, T);
  if (ws_bytes < L.total) return E4B_ERR_INVALID_ARG;
  const bool dq = d->format == E4B_NF4_DQ;
  if (T > 0) {
    if (!logits || !dout || !gu_codes || !gu_scales || !dn_codes || !dn_scales || !dx || !dlogits)
      return E4B_ERR_INVALID_ARG;
    if (!aligned(dout, 8) || !aligned(dx, 16) || !aligned(dlogits, 4) || !aligned(gu_codes, 16) ||
        !aligned(dn_codes, 16))
      return E4B_ERR_INVALID_ARG;
    if (dq ? !(valid_dq(static_cast<const e4b_nf4_dq*>(gu_scales)) && valid_dq(static_cast<const e4b_nf4_dq*>(dn_scales)))
           : !(aligned(gu_scales, 16) && aligned(dn_scales, 16)))
      return E4B_ERR_INVALID_ARG;
    if (lora && (!aligned(lora_A, 2) || !aligned(lora_B, 16) || !aligned(dA, 4) || !aligned(dB, 4)))
      return E4B_ERR_INVALID_ARG;
  }
  BackwardLaunch b;
  b.T = T;
  b.k = d->k;
  b.E = d->E;
  b.H = d->H;
  b.I = d->I;
  b.fmt = gemm_format(d->format);
  b.gating = d->gating;
  b.lora_rank = d->lora_rank;
  b.lora_scale = d->lora_scale;
  b.ep = Epilogue{nullptr, d->act, d->glu_alpha, d->glu_limit, d->glu_beta};
  b.logits = logits;
  b.dout = dout;
  b.y = at<float>(ws, L.fwd.y);
  b.topk_w = at<float>(ws, L.fwd.topk_w);
  b.topk_ids = at<int32_t>(ws, L.fwd.topk_ids);
  b.slot_pos = at<int32_t>(ws, L.fwd.slot_pos);
  b.sorted_slot = at<int32_t>(ws, L.fwd.sorted_slot);
  b.expert_offsets = at<int32_t>(ws, L.fwd.offsets);
  b.x_sorted = at<uint16_t>(ws, L.fwd.x_sorted);
  b.xa = lora ? at<uint16_t>(ws, L.fwd.xa) : nullptr;
  b.G = at<float>(ws, L.g);
  b.dY = at<uint16_t>(ws, L.dY);
  b.dG = at<uint16_t>(ws, L.dG);
  b.dxa = lora ? at<float>(ws, L.dxa) : nullptr;
  b.dX = at<float>(ws, L.dX);
  b.dx = dx;
  b.dlogits = dlogits;
  b.dA = dA;
  b.dB = dB;
  b.gu_codes = gu_codes;
  b.dn_codes = dn_codes;
  // the nested-form absmax was expanded into the workspace by the training forward
  b.gu_scales = dq ? static_cast<const void*>(at<float>(ws, L.fwd.gu_absmax)) : gu_scales;
  b.dn_scales = dq ? static_cast<const void*>(at<float>(ws, L.fwd.dn_absmax)) : dn_scales;
  b.lora_A = lora_A;
  b.lora_B = lora_B;
  return launch_moe_backward(b, reinterpret_cast<cudaStream_t>(stream));
}

// The norm's kernels index a row, and step past its end by a block, in 32 bits.
static const int32_t kMaxNormSize = 1 << 30;

e4b_status e4b_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int32_t T, int32_t H,
                       double eps, int32_t q_format, uint16_t* r_out, uint16_t* y, uint8_t* q, void* q_scales,
                       float* rstd, e4b_stream stream) {
  if (T < 0 || H < 1 || !(eps >= 0.0) || !std::isfinite(eps)) return E4B_ERR_INVALID_ARG;
  if (q_format != E4B_Q8_NONE && q_format != E4B_Q8_ROW && q_format != E4B_Q8_MX) return E4B_ERR_INVALID_ARG;
  if (T > kMaxNormSize || H > kMaxNormSize || (q_format == E4B_Q8_MX && H % 32 != 0)) return E4B_ERR_UNSUPPORTED;
  if (T == 0) return E4B_OK;
  const bool quant = q_format != E4B_Q8_NONE;
  if (!x || !weight || (q != nullptr) != quant || (q_scales != nullptr) != quant || (!y && !q) || (r_out && !residual))
    return E4B_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(r_out, 2) || !aligned(y, 2) ||
      !aligned(rstd, 4) || (q_format == E4B_Q8_ROW && !aligned(q_scales, 4)))
    return E4B_ERR_INVALID_ARG;
  const size_t n = static_cast<size_t>(T) * H;
  const Range in[3] = {range_of(x, 2 * n), range_of(residual, 2 * n), range_of(weight, 2 * static_cast<size_t>(H))};
  const Range out[5] = {range_of(r_out, 2 * n), range_of(y, 2 * n), range_of(q, n),
                        range_of(q_scales, q_format == E4B_Q8_ROW ? 4 * static_cast<size_t>(T) : n / 32),
                        range_of(rstd, 4 * static_cast<size_t>(T))};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j)
      if (i < 2 && j < 2 ? !same_or_apart(out[i], in[j]) : overlap(out[i], in[j])) return E4B_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return E4B_ERR_INVALID_ARG;
  }
  const NormLaunch p{x, residual, weight, T, H, 1.0 / H, eps, q_format, r_out, y, q, q_scales, rstd};
  return launch_rmsnorm(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

size_t e4b_rmsnorm_backward_workspace_bytes(int32_t T, int32_t H) {
  if (T < 0 || H < 1 || T > kMaxNormSize || H > kMaxNormSize) return 0;
  return kStatusBytes + align_up(static_cast<size_t>(norm_backward_blocks(T)) * H * 4);
}

e4b_status e4b_rmsnorm_backward(const void* dy, int32_t dy_type, const uint16_t* dr, const uint16_t* r,
                                const uint16_t* weight, const float* rstd, int32_t T, int32_t H, uint16_t* dx,
                                float* dweight, void* ws, size_t ws_bytes, e4b_stream stream) {
  if (T < 0 || H < 1 || (dy_type != E4B_F32 && dy_type != E4B_BF16)) return E4B_ERR_INVALID_ARG;
  if (T > kMaxNormSize || H > kMaxNormSize) return E4B_ERR_UNSUPPORTED;
  if (!dweight || !aligned(dweight, 4)) return E4B_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {                                      // (a workspace may be left out; one that is there gets its status)
    const bool has_ws = ws && aligned(ws, kAlign) && ws_bytes >= kStatusBytes;
    if (has_ws && overlap(range_of(ws, kStatusBytes), range_of(dweight, 4 * static_cast<size_t>(H))))
      return E4B_ERR_INVALID_ARG;
    const bool ok = cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * 4, s) == cudaSuccess &&
                    (!has_ws || cudaMemsetAsync(ws, 0, kStatusBytes, s) == cudaSuccess);
    return ok ? E4B_OK : E4B_ERR_CUDA;
  }
  if (!dy || !r || !weight || !rstd || !dx || !ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  if (!aligned(dy, dy_type == E4B_F32 ? 4 : 2) || !aligned(dr, 2) || !aligned(r, 2) || !aligned(weight, 2) ||
      !aligned(rstd, 4) || !aligned(dx, 2))
    return E4B_ERR_INVALID_ARG;
  const size_t need = e4b_rmsnorm_backward_workspace_bytes(T, H);
  if (ws_bytes < need) return E4B_ERR_INVALID_ARG;
  const size_t n = static_cast<size_t>(T) * H;
  const Range in[5] = {range_of(dy, n * (dy_type == E4B_F32 ? 4 : 2)), range_of(dr, 2 * n), range_of(r, 2 * n),
                       range_of(weight, 2 * static_cast<size_t>(H)), range_of(rstd, 4 * static_cast<size_t>(T))};
  const Range odx = range_of(dx, 2 * n), odw = range_of(dweight, 4 * static_cast<size_t>(H)), w = range_of(ws, need);
  for (int j = 0; j < 5; ++j)
    if ((j < 3 ? !same_or_apart(odx, in[j]) : overlap(odx, in[j])) || overlap(odw, in[j]) || overlap(w, in[j]))
      return E4B_ERR_INVALID_ARG;
  if (overlap(odx, odw) || overlap(odx, w) || overlap(odw, w)) return E4B_ERR_INVALID_ARG;
  const NormBackwardLaunch p{dy, dy_type == E4B_F32 ? 1 : 0, dr, r, weight, rstd, T, H, 1.0 / H, dx, dweight,
                             at<float>(ws, kStatusBytes), static_cast<int32_t*>(ws)};
  return launch_rmsnorm_backward(p, s) == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

// ---------------------------------------------------------------------- gated feed-forward block

static e4b_status validate_ffn(const e4b_ffn_desc* d, int32_t T) {
  if (!d || T < 0) return E4B_ERR_INVALID_ARG;
  if (d->H < 8 || d->H % 8 != 0 || d->I < 8 || d->I % 8 != 0) return E4B_ERR_UNSUPPORTED;
  if (d->I >= (1 << 29) || d->H >= (1 << 29) || T >= (1 << 30)) return E4B_ERR_UNSUPPORTED;
  if (d->act != E4B_ACT_SWIGLU && d->act != E4B_ACT_CLAMPED_GLU) return E4B_ERR_UNSUPPORTED;
  if (d->act == E4B_ACT_CLAMPED_GLU &&
      (!std::isfinite(d->glu_alpha) || !std::isfinite(d->glu_beta) || !(d->glu_limit > 0.0f)))
    return E4B_ERR_INVALID_ARG;
  return E4B_OK;
}

struct FfnLayout {
  size_t status, h, forward_total;                 // e4b_ffn_forward
  size_t g, dG, gu_sums, dn_sums, total;           // and the training pair
};

static FfnLayout ffn_layout(const e4b_ffn_desc& d, int32_t T) {
  const size_t t = static_cast<size_t>(T), I = static_cast<size_t>(d.I);
  FfnLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.status = take(kStatusBytes);
  L.h = take(t * I * 2);
  L.forward_total = o;
  L.g = take(t * 2 * I * 4);
  L.dG = take(t * 2 * I * 2);
  L.gu_sums = take(dense_colsum_rows(T) * 2 * I * 4);
  L.dn_sums = take(static_cast<size_t>(column_sum_splits(T)) * d.H * 4);
  L.total = o;
  return L;
}

size_t e4b_ffn_workspace_bytes(const e4b_ffn_desc* d, int32_t T) {
  return validate_ffn(d, T) == E4B_OK ? ffn_layout(*d, T).forward_total : 0;
}

size_t e4b_ffn_train_workspace_bytes(const e4b_ffn_desc* d, int32_t T) {
  return validate_ffn(d, T) == E4B_OK ? ffn_layout(*d, T).total : 0;
}

static e4b_status run_ffn(const e4b_ffn_desc* d, int32_t T, const uint16_t* x, const uint16_t* w_gu,
                          const uint16_t* w_dn, const float* gu_bias, const float* dn_bias, const uint16_t* add,
                          uint16_t* out, void* ws, size_t ws_bytes, e4b_stream stream, bool train) {
  const e4b_status v = validate_ffn(d, T);
  if (v != E4B_OK) return v;
  if (!ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  const FfnLayout L = ffn_layout(*d, T);
  const size_t need = train ? L.total : L.forward_total;
  if (ws_bytes < need) return E4B_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return cudaMemsetAsync(ws, 0, kStatusBytes, s) == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
  if (!x || !w_gu || !w_dn || !out) return E4B_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w_gu, 16) || !aligned(w_dn, 16) || !aligned(add, 16) || !aligned(out, 16) ||
      !aligned(gu_bias, 4) || !aligned(dn_bias, 4))
    return E4B_ERR_INVALID_ARG;
  const size_t H = d->H, I = d->I, rows = static_cast<size_t>(T) * H * 2;
  const Range o = range_of(out, rows), w = range_of(ws, need);
  const Range in[5] = {range_of(x, rows), range_of(w_gu, 4 * I * H), range_of(w_dn, 2 * I * H),
                       range_of(gu_bias, 8 * I), range_of(dn_bias, 4 * H)};
  for (const Range& r : in)
    if (overlap(o, r) || overlap(w, r)) return E4B_ERR_INVALID_ARG;
  if (!same_or_apart(o, range_of(add, rows)) || overlap(w, range_of(add, rows)) || overlap(o, w))
    return E4B_ERR_INVALID_ARG;
  uint16_t* h = at<uint16_t>(ws, L.h);
  float* g = train ? at<float>(ws, L.g) : nullptr;
  int32_t* status = at<int32_t>(ws, L.status);
  if (dense_decode_takes(T, d->H, d->I)) {
    const Epilogue ep{nullptr, d->act, d->glu_alpha, d->glu_limit, d->glu_beta};
    const DenseDecodeLaunch gu{T, d->I, d->H, x, w_gu, gu_bias, nullptr, h, g, ep, status};
    const DenseDecodeLaunch dn{T, d->H, d->I, h, w_dn, dn_bias, add, out, nullptr, ep, status};
    if (launch_dense_decode(gu, true, s) != cudaSuccess || launch_dense_decode(dn, false, s) != cudaSuccess)
      return E4B_ERR_CUDA;
    return E4B_OK;
  }
  DenseGemmLaunch gu = {};
  gu.epi = kEpiGateUp;
  gu.M = T;
  gu.N = d->I;
  gu.K = d->H;
  gu.a = x;
  gu.b = w_gu;
  gu.act = d->act;
  gu.alpha = d->glu_alpha;
  gu.limit = d->glu_limit;
  gu.beta = d->glu_beta;
  gu.bias = gu_bias;
  gu.out = h;
  gu.g_out = g;
  gu.status = status;
  gu.clear_status = 1;
  const e4b_status st = launch_dense_gemm(gu, s);
  if (st != E4B_OK) return st;
  DenseGemmLaunch dn = {};
  dn.epi = kEpiLinear;
  dn.M = T;
  dn.N = d->H;
  dn.K = d->I;
  dn.a = h;
  dn.b = w_dn;
  dn.bias = dn_bias;
  dn.add = add;
  dn.out = out;
  dn.status = status;
  dn.b_early = 1;
  return launch_dense_gemm(dn, s);
}

e4b_status e4b_ffn_forward(const e4b_ffn_desc* d, int32_t T, const uint16_t* x, const uint16_t* w_gu,
                           const uint16_t* w_dn, const float* gu_bias, const float* dn_bias, const uint16_t* add,
                           uint16_t* out, void* ws, size_t ws_bytes, e4b_stream stream) {
  return run_ffn(d, T, x, w_gu, w_dn, gu_bias, dn_bias, add, out, ws, ws_bytes, stream, false);
}

e4b_status e4b_ffn_forward_train(const e4b_ffn_desc* d, int32_t T, const uint16_t* x, const uint16_t* w_gu,
                                 const uint16_t* w_dn, const float* gu_bias, const float* dn_bias,
                                 const uint16_t* add, uint16_t* out, void* ws, size_t ws_bytes, e4b_stream stream) {
  return run_ffn(d, T, x, w_gu, w_dn, gu_bias, dn_bias, add, out, ws, ws_bytes, stream, true);
}

e4b_status e4b_ffn_backward(const e4b_ffn_desc* d, int32_t T, const uint16_t* x, const uint16_t* dout,
                            const uint16_t* w_gu, const uint16_t* w_dn, uint16_t* dx, uint16_t* dw_gu,
                            uint16_t* dw_dn, float* dgu_bias, float* ddn_bias, void* ws, size_t ws_bytes,
                            e4b_stream stream) {
  const e4b_status v = validate_ffn(d, T);
  if (v != E4B_OK) return v;
  if (!ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  const FfnLayout L = ffn_layout(*d, T);
  if (ws_bytes < L.total) return E4B_ERR_INVALID_ARG;
  if (!aligned(dx, 16) || !aligned(dw_gu, 16) || !aligned(dw_dn, 16) || !aligned(dgu_bias, 4) || !aligned(ddn_bias, 4))
    return E4B_ERR_INVALID_ARG;
  const size_t H = d->H, I = d->I, rows = static_cast<size_t>(T) * H * 2;
  const Range outs[5] = {range_of(dx, rows), range_of(dw_gu, 4 * I * H), range_of(dw_dn, 2 * I * H),
                         range_of(dgu_bias, 8 * I), range_of(ddn_bias, 4 * H)};
  const Range ins[5] = {range_of(ws, L.total), range_of(x, rows), range_of(dout, rows), range_of(w_gu, 4 * I * H),
                        range_of(w_dn, 2 * I * H)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 5; ++j)
      if (overlap(outs[i], ins[j])) return E4B_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return E4B_ERR_INVALID_ARG;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    const bool ok = (!dw_gu || cudaMemsetAsync(dw_gu, 0, 4 * I * H, s) == cudaSuccess) &&
                    (!dw_dn || cudaMemsetAsync(dw_dn, 0, 2 * I * H, s) == cudaSuccess) &&
                    (!dgu_bias || cudaMemsetAsync(dgu_bias, 0, 8 * I, s) == cudaSuccess) &&
                    (!ddn_bias || cudaMemsetAsync(ddn_bias, 0, 4 * H, s) == cudaSuccess);
    return ok ? E4B_OK : E4B_ERR_CUDA;
  }
  if (!x || !dout || !w_gu || !w_dn || !aligned(x, 16) || !aligned(dout, 16) || !aligned(w_gu, 16) ||
      !aligned(w_dn, 16))
    return E4B_ERR_INVALID_ARG;
  uint16_t* dG = at<uint16_t>(ws, L.dG);
  DenseGemmLaunch base = {};
  base.act = d->act;
  base.alpha = d->glu_alpha;
  base.limit = d->glu_limit;
  base.beta = d->glu_beta;
  base.status = at<int32_t>(ws, L.status);
  e4b_status st = E4B_OK;
  int32_t sum_rows = 0;
  if (dx || dw_gu || dgu_bias) {                     // dG = act'(G) applied to dout W_dn
    DenseGemmLaunch g = base;
    g.epi = kEpiDact;
    g.M = T;
    g.N = d->I;
    g.K = d->H;
    g.a = dout;
    g.b = w_dn;
    g.b_mn = true;
    g.out = dG;
    g.g_in = at<float>(ws, L.g);
    g.colsum = dgu_bias ? at<float>(ws, L.gu_sums) : nullptr;
    g.colsum_rows = &sum_rows;
    st = launch_dense_gemm(g, s);
    if (st != E4B_OK) return st;
  }
  DenseGemmLaunch rest[3];                           // the products that follow do not depend on one another
  int n = 0;
  base.epi = kEpiLinear;
  base.b_mn = true;
  if (dx) {                                          // dG W_gu
    DenseGemmLaunch& g = rest[n++] = base;
    g.M = T;
    g.N = d->H;
    g.K = 2 * d->I;
    g.a = dG;
    g.b = w_gu;
    g.out = dx;
    g.b_early = 1;                                   // (dx comes right after dG)
  }
  base.a_mn = true;                                  // both weight gradients contract the tokens
  base.K = T;
  if (dw_gu) {                                       // dG^T x
    DenseGemmLaunch& g = rest[n++] = base;
    g.M = 2 * d->I;
    g.N = d->H;
    g.a = dG;
    g.b = x;
    g.out = dw_gu;
  }
  if (dw_dn) {                                       // dout^T h
    DenseGemmLaunch& g = rest[n++] = base;
    g.M = d->H;
    g.N = d->I;
    g.a = dout;
    g.b = at<uint16_t>(ws, L.h);
    g.out = dw_dn;
  }
  const ColumnSums sums{at<float>(ws, L.gu_sums), sum_rows, 2 * d->I, dgu_bias, dout, T, d->H,
                        at<float>(ws, L.dn_sums), ddn_bias};
  return launch_dense_group(rest, n, sums, s);
}

static const int32_t kMaxGradTensors = 65536;

size_t e4b_clip_grad_norm_workspace_bytes(int32_t tensors) {
  if (tensors < 0 || tensors > kMaxGradTensors) return 0;
  return align_up(grad_norm_partials(tensors) * sizeof(double));
}

// Whether every out lies apart from every other out and from every grad but its own.
static e4b_status check_grads(const e4b_grad* g, int32_t tensors, const Range& norm, const Range& ws) {
  struct Span {
    Range r;
    int32_t owner;
  };
  Span* outs = new (std::nothrow) Span[tensors > 0 ? tensors : 1];
  if (!outs) return E4B_ERR_INVALID_ARG;
  e4b_status st = E4B_OK;
  int32_t n = 0;
  auto bytes = [&](int32_t i) { return static_cast<size_t>(g[i].n) * (g[i].dtype == E4B_F32 ? 4 : 2); };
  for (int32_t i = 0; i < tensors; ++i)
    if (g[i].n > 0) outs[n++] = {range_of(g[i].out, bytes(i)), i};
  auto before = [](const Span& a, const Span& b) { return a.r.lo < b.r.lo; };
  if (!std::is_sorted(outs, outs + n, before)) std::sort(outs, outs + n, before);
  for (int32_t i = 1; i < n; ++i)
    if (outs[i].r.lo < outs[i - 1].r.hi) st = E4B_ERR_INVALID_ARG;
  // the outs are now in order and apart: a grad can only overlap those around it, and none of them where the grads
  // are the outs or lie apart from all of them
  auto clash = [&](const Range& r, int32_t own) {
    const Span key{r, 0};
    const Span* it = std::upper_bound(outs, outs + n, key, before);
    for (const Span* s = it == outs ? it : it - 1; s < outs + n && s->r.lo < r.hi; ++s)
      if (overlap(s->r, r) && !(s->owner == own && s->r.lo == r.lo)) return true;
    return false;
  };
  Range all{~uintptr_t(0), 0};
  bool in_place = true;
  for (int32_t i = 0; i < tensors && st == E4B_OK; ++i)
    if (g[i].n > 0) {
      const Range r = range_of(g[i].grad, bytes(i));
      if (r.lo < all.lo) all.lo = r.lo;
      if (r.hi > all.hi) all.hi = r.hi;
      in_place = in_place && g[i].grad == g[i].out;
      if (overlap(r, norm) || overlap(r, ws)) st = E4B_ERR_INVALID_ARG;
    }
  if (st == E4B_OK && n > 0 && !in_place && overlap(all, Range{outs[0].r.lo, outs[n - 1].r.hi}))
    for (int32_t i = 0; i < tensors && st == E4B_OK; ++i)
      if (g[i].n > 0 && clash(range_of(g[i].grad, bytes(i)), i)) st = E4B_ERR_INVALID_ARG;
  if (st == E4B_OK && (clash(norm, -1) || clash(ws, -1) || overlap(norm, ws))) st = E4B_ERR_INVALID_ARG;
  delete[] outs;
  return st;
}

e4b_status e4b_clip_grad_norm(const e4b_grad* grads, int32_t tensors, double max_norm, float* total_norm, void* ws,
                              size_t ws_bytes, e4b_stream stream) {
  if (tensors < 0 || tensors > kMaxGradTensors || (tensors > 0 && !grads) || !(max_norm >= 0.0))
    return E4B_ERR_INVALID_ARG;
  if (!total_norm || !aligned(total_norm, 4) || !ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  const size_t need = e4b_clip_grad_norm_workspace_bytes(tensors);
  if (ws_bytes < need) return E4B_ERR_INVALID_ARG;
  for (int32_t i = 0; i < tensors; ++i) {
    const e4b_grad& g = grads[i];
    if (g.dtype != E4B_F32 && g.dtype != E4B_BF16 && g.dtype != E4B_F16) return E4B_ERR_UNSUPPORTED;
    const size_t size = g.dtype == E4B_F32 ? 4 : 2;
    if (g.n < 0 || g.n > (int64_t(1) << 40)) return E4B_ERR_INVALID_ARG;
    if (g.n > 0 && (!g.grad || !g.out || !aligned(g.grad, size) || !aligned(g.out, size))) return E4B_ERR_INVALID_ARG;
  }
  const e4b_status v = check_grads(grads, tensors, range_of(total_norm, 4), range_of(ws, need));
  if (v != E4B_OK) return v;
  return launch_clip_grads(grads, tensors, max_norm, total_norm, static_cast<double*>(ws),
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? E4B_OK
             : E4B_ERR_CUDA;
}

e4b_status e4b_device_status(void* ws, e4b_stream stream) {
  if (!ws || !aligned(ws, kAlign)) return E4B_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return E4B_ERR_CUDA;
  int32_t h[2] = {0, 0};
  if (cudaMemcpy(h, ws, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return E4B_ERR_CUDA;
  if (h[0] != 0 && cudaMemset(ws, 0, sizeof(h)) != cudaSuccess) return E4B_ERR_CUDA;
  return static_cast<e4b_status>(h[0]);
}

e4b_status e4b_wait_status(e4b_stream stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return E4B_ERR_CUDA;
  e4b_status st = E4B_OK;
  const WaitFlags& f = wait_flags();
  for (int i = 0; i < f.count; ++i) {
    void* p = nullptr;
    int32_t v = 0;
    if (f.address[i](&p) != cudaSuccess || cudaMemcpy(&v, p, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
      return E4B_ERR_CUDA;
    if (v == 0) continue;
    if (cudaMemset(p, 0, sizeof(v)) != cudaSuccess) return E4B_ERR_CUDA;
    st = static_cast<e4b_status>(v);
  }
  return st;
}

e4b_status e4b_debug_wait_timeout(uint32_t limit_ns, void* ws, size_t ws_bytes, e4b_stream stream) {
  if (!ws || !aligned(ws, kAlign) || ws_bytes < kStatusBytes || limit_ns > 1000000000u) return E4B_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, kStatusBytes, s) != cudaSuccess) return E4B_ERR_CUDA;
  wait_timeout_probe_kernel<<<1, 32, 0, s>>>(static_cast<int32_t*>(ws), limit_ns);
  return cudaGetLastError() == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

}  // extern "C"
