// The gated delta rule over whole prompts (moe_gdn_prefill), sm_100a.
//
// Per sequence and value head, with the state S (d_v x d_k, fp32) and the notation of gdn.cu:
//
//     S_t = e^{g_t} S_{t-1} + beta_t (v_t - e^{g_t} S_{t-1} k^_t) k^_t^T,   o_t = S_t q^_t
//
// k_gdn_plan checks the sequences' row ranges.  k_gdn_recur takes the tokens one after another:
// a warp owns rows of S in registers, as in the decode step.
#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.cuh"
#include "seqs.cuh"
#include "sync.cuh"

namespace moe {

struct GdnSeq {
  int row0, n;  // first row and tokens; n < 0: left out
};

struct GdnPrefillArgs {
  int n_seqs, T, Hk, Hv, dk, dv;
  const int32_t* offsets;
  const float* S_in;     // [n_seqs, Hv, dv, dk] or null (zeros)
  float* S_out;          // [n_seqs, Hv, dv, dk]
  const uint16_t* q;     // bf16 [T, Hk, dk]
  const uint16_t* k;     // bf16 [T, Hk, dk]
  const uint16_t* v;     // bf16 [T, Hv, dv]
  const float* g;        // [T, Hv]
  const float* beta;     // [T, Hv]
  uint16_t* out;         // bf16 [T, Hv, dv]
  Ctrl* ctrl;
  GdnSeq* seqs;          // [n_seqs]
};

namespace {

__global__ void __launch_bounds__(kPlanThreads) k_gdn_plan(const GdnPrefillArgs a) {
  __shared__ int sh[32];
  int seen = 0;
  for (int base = 0; base < a.n_seqs; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const bool in = i < a.n_seqs;
    const int r0 = in ? a.offsets[i] : 0, r1 = in ? a.offsets[i + 1] : 0;
    const int before = block_excl_max(r0, seen, sh);
    if (!in) continue;
    const bool ok = rows_ok(r0, r1, before, a.T);
    a.seqs[i] = GdnSeq{r0, ok ? r1 - r0 : -1};
    if (!ok) atomicOr(&a.ctrl->err, kErrBadRange);
  }
}

constexpr int kRecurWarps = 8, kRecurRpw = 4, kRecurRows = kRecurWarps * kRecurRpw;

__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int DK>
__global__ void __launch_bounds__(kRecurWarps * 32) k_gdn_recur(const GdnPrefillArgs a) {
  constexpr int EPL = DK / 32;
  const int blocks = (a.dv + kRecurRows - 1) / kRecurRows;
  const int bh = blockIdx.x / blocks, rb = blockIdx.x - bh * blocks;
  const int s = bh / a.Hv, h = bh - s * a.Hv, kh = h / (a.Hv / a.Hk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const GdnSeq seq = a.seqs[s];
  if (seq.n < 0) return;
  const int i0 = rb * kRecurRows + warp * kRecurRpw;
  float row[kRecurRpw][EPL];
#pragma unroll
  for (int r = 0; r < kRecurRpw; ++r)
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      row[r][e] = a.S_in && i0 + r < a.dv ? a.S_in[((size_t)bh * a.dv + i0 + r) * DK + lane * EPL + e] : 0.f;
  for (int t = seq.row0; t < seq.row0 + seq.n; ++t) {
    float kn[EPL], qn[EPL], kk = 0.f, qq = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      kn[e] = bf1(a.k[((size_t)t * a.Hk + kh) * DK + lane * EPL + e]);
      qn[e] = bf1(a.q[((size_t)t * a.Hk + kh) * DK + lane * EPL + e]);
      kk = fmaf(kn[e], kn[e], kk);
      qq = fmaf(qn[e], qn[e], qq);
    }
    const float ki = 1.0f / fmaxf(sqrtf(lanes_sum(kk)), 1e-6f);
    const float qi = 1.0f / fmaxf(sqrtf(lanes_sum(qq)), 1e-6f) * rsqrtf((float)DK);
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      kn[e] *= ki;
      qn[e] *= qi;
    }
    const float alpha = expf(a.g[(size_t)t * a.Hv + h]), beta = a.beta[(size_t)t * a.Hv + h];
#pragma unroll
    for (int r = 0; r < kRecurRpw; ++r) {
      if (i0 + r >= a.dv) continue;  // the whole warp takes the same branch
      const size_t at = ((size_t)t * a.Hv + h) * a.dv + i0 + r;
      float u = 0.f, o = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) u = fmaf(row[r][e], kn[e], u);
      u = lanes_sum(u);
      const float c = beta * (bf1(a.v[at]) - alpha * u);
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        row[r][e] = fmaf(alpha, row[r][e], c * kn[e]);
        o = fmaf(row[r][e], qn[e], o);
      }
      o = lanes_sum(o);
      if (lane == 0) a.out[at] = f2bf(o);
    }
  }
#pragma unroll
  for (int r = 0; r < kRecurRpw; ++r)
    if (i0 + r < a.dv)
#pragma unroll
      for (int e = 0; e < EPL; ++e) a.S_out[((size_t)bh * a.dv + i0 + r) * DK + lane * EPL + e] = row[r][e];
}

}  // namespace

cudaError_t launch_gdn_prefill(const GdnPrefillArgs& a, cudaStream_t s) {
  k_gdn_plan<<<1, kPlanThreads, 0, s>>>(a);
  const int blocks = a.n_seqs * a.Hv * ((a.dv + kRecurRows - 1) / kRecurRows);
  switch (a.dk) {
    case 64: k_gdn_recur<64><<<blocks, kRecurWarps * 32, 0, s>>>(a); break;
    case 128: k_gdn_recur<128><<<blocks, kRecurWarps * 32, 0, s>>>(a); break;
    default: k_gdn_recur<256><<<blocks, kRecurWarps * 32, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

moe_status set_error(moe_status s, const char* fmt, ...);
moe_status cuda_fail(cudaError_t e, const char* what);

static moe_status check_gdn_prefill(const moe_gdn_shape* shape, int32_t n_seqs, int32_t T) {
  if (!shape) return set_error(MOE_ERR_INVALID, "shape is NULL");
  const int Hk = shape->n_k_heads, Hv = shape->n_v_heads, dk = shape->d_k, dv = shape->d_v;
  if (Hk < 1 || Hv < 1 || Hv % Hk) return set_error(MOE_ERR_INVALID, "n_v_heads must be a positive multiple of n_k_heads");
  if (dv < 1) return set_error(MOE_ERR_INVALID, "d_v must be >= 1");
  if (dk != 64 && dk != 128 && dk != 256) return set_error(MOE_ERR_UNSUPPORTED, "d_k must be 64, 128 or 256 (got %d)", dk);
  if (n_seqs < 1 || n_seqs > kMaxSeqs) return set_error(MOE_ERR_INVALID, "n_seqs must be 1..%d (got %d)", kMaxSeqs, n_seqs);
  if (T < 0) return set_error(MOE_ERR_INVALID, "T must be >= 0 (got %d)", T);
  const long long blocks = (long long)n_seqs * Hv * ((dv + 15) / 16);
  if (blocks > 0x7fffffffLL) return set_error(MOE_ERR_INVALID, "n_seqs * n_v_heads * d_v too large");
  return MOE_OK;
}

struct GdnPrefillLayout {
  size_t ctrl, seqs, total;
};
static GdnPrefillLayout gdn_prefill_layout(const moe_gdn_shape* shape, int n_seqs, int T) {
  GdnPrefillLayout W{};
  size_t pos = 0;
  auto take = [&](size_t bytes) {
    const size_t at = (size_t)round_up((int64_t)pos, kAlign);
    pos = at + bytes;
    return at;
  };
  W.ctrl = take(sizeof(Ctrl));
  W.seqs = take(sizeof(GdnSeq) * (size_t)n_seqs);
  W.total = (size_t)round_up((int64_t)pos, kAlign);
  return W;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_gdn_prefill_workspace_size(const moe_gdn_shape* shape, int32_t n_seqs, int32_t T, size_t* bytes) {
  const moe_status st = check_gdn_prefill(shape, n_seqs, T);
  if (st != MOE_OK) return st;
  if (!bytes) return set_error(MOE_ERR_INVALID, "bytes is NULL");
  *bytes = gdn_prefill_layout(shape, n_seqs, T).total;
  return MOE_OK;
}

extern "C" moe_status moe_gdn_prefill(const moe_gdn_shape* shape, int32_t n_seqs, int32_t T, const int32_t* offsets,
                                      const float* state_in, float* state_out, const void* q, const void* k,
                                      const void* v, const float* g, const float* beta, void* out, void* ws,
                                      size_t ws_bytes, void* stream) {
  const moe_status st = check_gdn_prefill(shape, n_seqs, T);
  if (st != MOE_OK) return st;
  if (!offsets || !state_out) return set_error(MOE_ERR_INVALID, "offsets and state_out must be non-NULL");
  if (T > 0 && (!q || !k || !v || !g || !beta || !out))
    return set_error(MOE_ERR_INVALID, "q, k, v, g, beta and out must be non-NULL");
  if (!ws) return set_error(MOE_ERR_INVALID, "ws is NULL");
  const uintptr_t all = (uintptr_t)offsets | (uintptr_t)state_in | (uintptr_t)state_out | (uintptr_t)q | (uintptr_t)k |
                        (uintptr_t)v | (uintptr_t)g | (uintptr_t)beta | (uintptr_t)out | (uintptr_t)ws;
  if (all & 15) return set_error(MOE_ERR_INVALID, "every pointer must be 16-byte aligned");
  const size_t state = (size_t)n_seqs * shape->n_v_heads * shape->d_v * shape->d_k * sizeof(float);
  if (state_in && state_in != state_out) {
    const uintptr_t x = (uintptr_t)state_in, y = (uintptr_t)state_out;
    if (x < y + state && y < x + state) return set_error(MOE_ERR_INVALID, "state_in overlaps state_out without being it");
  }
  const GdnPrefillLayout W = gdn_prefill_layout(shape, n_seqs, T);
  if (ws_bytes < W.total) return set_error(MOE_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, W.total);
  uint8_t* w = static_cast<uint8_t*>(ws);
  GdnPrefillArgs a{n_seqs, T, shape->n_k_heads, shape->n_v_heads, shape->d_k, shape->d_v, offsets, state_in, state_out,
                   static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), g,
                   beta, static_cast<uint16_t*>(out), reinterpret_cast<Ctrl*>(w + W.ctrl),
                   reinterpret_cast<GdnSeq*>(w + W.seqs)};
  const cudaError_t e = launch_gdn_prefill(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gated delta prompt launch");
  return MOE_OK;
}
