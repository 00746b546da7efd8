// Causal softmax attention with grouped heads over packed sequences (moe_attn_forward), sm_100a.
//
//     out_i = sum_j p_ij v_j,  p_ij = e^{x_ij - m_i} / sum_j e^{x_ij - m_i},  x_ij = scale q_i.k_j
//
// over the keys j <= len - n + i of the query's sequence, in one pass over the keys with the
// running maximum m_i and sum (a new maximum rescales what was summed before).
#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.cuh"
#include "seqs.cuh"
#include "sync.cuh"

#include <cmath>

namespace moe {

struct AttnSeq {
  int row0, n;    // first query row and queries; n < 0: left out
  int kv0, len;   // first key row and keys
};

struct AttnArgs {
  int n_seqs, T, Hq, Hkv, d, max_kv, kv_rows;
  float scale;
  const int32_t *offsets, *kv_begin, *kv_len;
  const uint16_t *q, *k, *v;
  uint16_t* out;
  Ctrl* ctrl;
  AttnSeq* seqs;  // [n_seqs]
};

namespace {

__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const AttnArgs a) {
  __shared__ int sh[32];
  int seen = 0;
  for (int base = 0; base < a.n_seqs; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const bool in = i < a.n_seqs;
    const int r0 = in ? a.offsets[i] : 0, r1 = in ? a.offsets[i + 1] : 0;
    const int before = block_excl_max(r0, seen, sh);
    if (!in) continue;
    const int kv0 = a.kv_begin ? a.kv_begin[i] : r0, len = a.kv_begin ? a.kv_len[i] : r1 - r0;
    const bool ok = rows_ok(r0, r1, before, a.T) && kv0 >= 0 && len >= 0 && len <= a.max_kv && kv0 <= a.kv_rows &&
                    len <= a.kv_rows - kv0;
    a.seqs[i] = AttnSeq{r0, ok ? r1 - r0 : -1, kv0, len};
    if (!ok) atomicOr(&a.ctrl->err, kErrBadRange);
  }
}

// One warp per query row and head, a lane per d / 32 elements.
template <int D>
__global__ void __launch_bounds__(256) k_attn_rows(const AttnArgs a) {
  constexpr int EPL = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(w / a.Hq), h = (int)(w - (long long)t * a.Hq), kh = h / (a.Hq / a.Hkv);
  if (t >= a.T) return;
  AttnSeq seq{};
  bool found = false;
  for (int base = 0; base < a.n_seqs && !found; base += 32) {
    AttnSeq c{0, -1, 0, 0};
    if (base + lane < a.n_seqs) c = a.seqs[base + lane];
    const unsigned hit = __ballot_sync(0xffffffffu, c.n > 0 && t >= c.row0 && t < c.row0 + c.n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      seq = AttnSeq{__shfl_sync(0xffffffffu, c.row0, src), __shfl_sync(0xffffffffu, c.n, src),
                    __shfl_sync(0xffffffffu, c.kv0, src), __shfl_sync(0xffffffffu, c.len, src)};
      found = true;
    }
  }
  if (!found) return;
  const int seen = seq.len - seq.n + (t - seq.row0) + 1;
  float q[EPL], o[EPL], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < EPL; ++e) {
    q[e] = bf1(a.q[((size_t)t * a.Hq + h) * D + lane * EPL + e]) * a.scale;
    o[e] = 0.f;
  }
  for (int j = 0; j < seen; ++j) {
    const size_t at = ((size_t)(seq.kv0 + j) * a.Hkv + kh) * D + lane * EPL;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) x = fmaf(q[e], bf1(a.k[at + e]), x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    const float mn = fmaxf(m, x), f = m == mn ? 1.f : expf(m - mn), p = x == mn ? 1.f : expf(x - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = fmaf(o[e], f, p * bf1(a.v[at + e]));
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < EPL; ++e) a.out[((size_t)t * a.Hq + h) * D + lane * EPL + e] = f2bf(seen > 0 ? o[e] / l : 0.f);
}

}  // namespace

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
  k_attn_plan<<<1, kPlanThreads, 0, s>>>(a);
  const int blocks = (int)(((long long)a.T * a.Hq + 7) / 8);
  if (a.d == 64) k_attn_rows<64><<<blocks, 256, 0, s>>>(a);
  else k_attn_rows<128><<<blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

moe_status set_error(moe_status s, const char* fmt, ...);
moe_status cuda_fail(cudaError_t e, const char* what);

constexpr int kMaxAttnGroup = 64;  // query heads of one key head

static moe_status check_attn(const moe_attn_shape* shape, int32_t n_seqs, int32_t T, int32_t max_kv) {
  if (!shape) return set_error(MOE_ERR_INVALID, "shape is NULL");
  const int Hq = shape->n_q_heads, Hkv = shape->n_kv_heads, d = shape->d;
  if (Hq < 1 || Hkv < 1 || Hq % Hkv) return set_error(MOE_ERR_INVALID, "n_q_heads must be a positive multiple of n_kv_heads");
  if (d < 1) return set_error(MOE_ERR_INVALID, "d must be >= 1");
  if (d != 64 && d != 128) return set_error(MOE_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", d);
  if (Hq / Hkv > kMaxAttnGroup)
    return set_error(MOE_ERR_UNSUPPORTED, "at most %d query heads per key head (got %d)", kMaxAttnGroup, Hq / Hkv);
  if (Hq > 65536) return set_error(MOE_ERR_INVALID, "n_q_heads must be at most 65536 (got %d)", Hq);
  if (n_seqs < 1 || n_seqs > kMaxSeqs) return set_error(MOE_ERR_INVALID, "n_seqs must be 1..%d (got %d)", kMaxSeqs, n_seqs);
  if (T < 0) return set_error(MOE_ERR_INVALID, "T must be >= 0 (got %d)", T);
  if (max_kv < 0) return set_error(MOE_ERR_INVALID, "max_kv must be >= 0 (got %d)", max_kv);
  if (((long long)T * Hq + 7) / 8 > 0x7fffffffLL) return set_error(MOE_ERR_INVALID, "T * n_q_heads too large");
  return MOE_OK;
}

struct AttnLayout {
  size_t ctrl, seqs, total;
};
static AttnLayout attn_layout(const moe_attn_shape* shape, int n_seqs, int T, int max_kv) {
  AttnLayout W{};
  size_t pos = 0;
  auto take = [&](size_t bytes) {
    const size_t at = (size_t)round_up((int64_t)pos, kAlign);
    pos = at + bytes;
    return at;
  };
  W.ctrl = take(sizeof(Ctrl));
  W.seqs = take(sizeof(AttnSeq) * (size_t)n_seqs);
  W.total = (size_t)round_up((int64_t)pos, kAlign);
  return W;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_attn_workspace_size(const moe_attn_shape* shape, int32_t n_seqs, int32_t T, int32_t max_kv,
                                              size_t* bytes) {
  const moe_status st = check_attn(shape, n_seqs, T, max_kv);
  if (st != MOE_OK) return st;
  if (!bytes) return set_error(MOE_ERR_INVALID, "bytes is NULL");
  *bytes = attn_layout(shape, n_seqs, T, max_kv).total;
  return MOE_OK;
}

extern "C" moe_status moe_attn_forward(const moe_attn_shape* shape, int32_t n_seqs, int32_t T, const int32_t* q_offsets,
                                       const int32_t* kv_begin, const int32_t* kv_len, int32_t max_kv, const void* q,
                                       const void* k, const void* v, int32_t kv_rows, float scale, void* out, void* ws,
                                       size_t ws_bytes, void* stream) {
  const moe_status st = check_attn(shape, n_seqs, T, max_kv);
  if (st != MOE_OK) return st;
  if (!q_offsets) return set_error(MOE_ERR_INVALID, "q_offsets is NULL");
  if (!kv_begin != !kv_len) return set_error(MOE_ERR_INVALID, "kv_begin and kv_len must both be given or both be NULL");
  if (kv_rows < 0) return set_error(MOE_ERR_INVALID, "kv_rows must be >= 0 (got %d)", kv_rows);
  if (!kv_begin && kv_rows < T) return set_error(MOE_ERR_INVALID, "kv_rows must be >= T without kv_begin (got %d < %d)", kv_rows, T);
  if (T > 0 && (!q || !out)) return set_error(MOE_ERR_INVALID, "q and out must be non-NULL");
  if (T > 0 && kv_rows > 0 && (!k || !v)) return set_error(MOE_ERR_INVALID, "k and v must be non-NULL");
  if (!std::isfinite(scale)) return set_error(MOE_ERR_INVALID, "scale must be finite");
  if (!ws) return set_error(MOE_ERR_INVALID, "ws is NULL");
  const uintptr_t all = (uintptr_t)q_offsets | (uintptr_t)kv_begin | (uintptr_t)kv_len | (uintptr_t)q | (uintptr_t)k |
                        (uintptr_t)v | (uintptr_t)out | (uintptr_t)ws;
  if (all & 15) return set_error(MOE_ERR_INVALID, "every pointer must be 16-byte aligned");
  const AttnLayout W = attn_layout(shape, n_seqs, T, max_kv);
  if (ws_bytes < W.total) return set_error(MOE_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, W.total);
  if (T == 0) return MOE_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnArgs a{n_seqs, T, shape->n_q_heads, shape->n_kv_heads, shape->d, max_kv, kv_rows, scale, q_offsets, kv_begin,
             kv_len, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
             static_cast<uint16_t*>(out), reinterpret_cast<Ctrl*>(w + W.ctrl), reinterpret_cast<AttnSeq*>(w + W.seqs)};
  const cudaError_t e = launch_attn(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return MOE_OK;
}
