// The gated delta rule over whole prompts (moe_gdn_prefill), sm_100a.
//
// Per sequence and value head, with the state S (d_v x d_k, fp32) and the notation of gdn.cu:
//
//     S_t = e^{g_t} S_{t-1} + w_t k^_t^T,  w_t = beta_t (v_t - e^{g_t} S_{t-1} k^_t),  o_t = S_t q^_t
//
// Taken 64 tokens at a time (the chunk's tokens i, j; S the state before it; G_i = g_1 + .. + g_i
// inside it; D_ij = e^{G_i - G_j}), the writes solve a unit lower triangular system:
//
//     (I + L) W = diag(beta) R,  L_ij = beta_i D_ij k^_i.k^_j (j < i),  R = V - diag(e^G) K^ S^T
//     O  = diag(e^G) Q^ S^T + (D o Q^ K^^T)_{j <= i} W
//     S' = e^{G_64} S + (diag(e^{G_64 - G}) W)^T K^
//
// L needs no state, so everything but the products with S is done for all chunks at once:
//
//   k_gdn_plan   one CTA: checks the row ranges, lists the chunks, orders the sequences longest
//                first (they are the critical path); small calls of few sequences do without it
//   k_gdn_chunk  a CTA per chunk and key head: norms, K K^T and Q K^T on the tensor cores, the
//                decays, T' = (I + L)^-1 diag(beta) by block inversion and P = D o Q^ K^^T;
//                leaves K, Q, T' and P in the operand layout of the next kernel
//   k_gdn_scan   the sequential part, W = T' R.  A slab of 16 state rows (of one sequence and value
//                head) belongs to d_k / 64 warps, 64 columns each, and stays in their registers as
//                MMA accumulators from the first chunk to the last; rows never mix, so nothing else
//                is shared but the sums S k over the columns (through shared memory, one exchange
//                a chunk).  Everything is held transposed (S [d_v, d_k], R^T, W^T [d_v, token]): an
//                accumulator is then the next product's A operand without moving a value.
//
// Precision.  The state is fp32 and has to stay so, but the tensor cores take 16-bit operands.
// K is exact: its rows, scaled by powers of two to a norm of 2^10 .. 2^11, fit fp16 (bf16 has
// fewer bits), and the norm's factor is applied in fp32.  S, R and W are split x = hi + lo into two
// fp16 values after scaling each row by a power of two to its largest element: 22 bits of the row's
// size; T' likewise by its largest element.  S K^T and W K take two products (hi, lo), T' R three (lo lo
// is below 2^-22).  What only the bf16 output sees (Q S, P W) takes hi alone, 2^-12 of each weight.
// The scale is a row's over the chunk, and fp16 ends at 2^-24: an element below 2^-18 of its row's
// largest in the 64 tokens keeps 2^-39 of that largest, not 22 bits of its own.  Sums of 64 of them are
// good to 2^-30 of it, which can only show where a decay inside the chunk (or the order of the tokens)
// parts writes that are more than 2^16 apart.  A scale of each token's own would have to be undone in T',
// whose entries are shared by all rows.
// mma.sync carries this, not tcgen05: the slab's products are 16 rows high, 8 to 64 wide and
// dependent on each other, and a chunk's chain of six of them through TMEM (a round trip of
// registers, TMEM, MMA and back for each) costs more than the products themselves.
#include "../../include/moe.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels.cuh"
#include "seqs.cuh"
#include "sync.cuh"
#include "tc.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace moe {

constexpr int kGdnChunk = 64;     // tokens of a chunk
constexpr int kGdnSlab = 16;      // state rows of a slab
constexpr int kGdnSlice = 64;     // state columns of a warp

struct GdnSeq {
  int row0, n;   // first row and tokens; n < 0: left out
  int chunk0;    // its first chunk
};
struct GdnChunk {
  int row0, n;
};
struct GdnHdr {
  int n_chunks;
  int chain;  // the longest sequence is the critical path of the scan
};

// What k_gdn_chunk leaves for one chunk and value head.  T' and P as B operands of
// mma.m16n8k16 (n = token i in tiles of 8, k = token j in steps of 16): the 20 (tile, step)
// blocks of the lower triangle, a lane's registers together.
struct GdnTP {
  static constexpr int kBlocks = 20;
  uint4 t[kBlocks][32];              // T': hi (2 registers), lo (2 registers)
  uint2 p[kBlocks][32];              // P
  float xa[kGdnChunk];               // -e^{G_i} / |k_i|: what the state recalls, in R
  float oa[kGdnChunk];               // e^{G_i} / (|q_i| sqrt(d_k))
  float wd[kGdnChunk];               // e^{G_64 - G_i} / |k_i|, over `wd_scale`
  float keep;                        // e^{G_64}
  float t_scale, p_scale, wd_scale;  // what t, p and wd are to be multiplied by (powers of two but p's)
  int plain;                         // the chunk is to be done token by token (see gdn_scan)
  float pad[59];
};
static_assert(sizeof(GdnTP) % 256 == 0, "bulk copies; V behind it starts on a period of its swizzle");
// Block of token tile t (8 tokens) and step k (16 tokens), k <= t / 2
__host__ __device__ constexpr int gdn_block(int t, int k) { return (t / 2) * (t / 2 + 1) + (t & 1) * (t / 2 + 1) + k; }
static_assert(gdn_block(7, 3) == GdnTP::kBlocks - 1, "lower triangle");

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
  int slabs;             // slabs of a scan CTA
  int n_sm;
  int warp_plan;         // no plan kernel (see gdn_warp_plan)
  Ctrl* ctrl;
  GdnHdr* hdr;
  GdnSeq* seqs;          // [n_seqs]
  int32_t* order;        // [n_seqs] sequences, longest first
  GdnChunk* chunks;
  uint8_t* img;          // [chunk][Hk]: fp16 K then Q, 64 x dk each, rows' 16-byte pieces XORed with row & 7
  GdnTP* tp;             // [chunk][Hv]
  alignas(64) CUtensorMap map_v;  // v: boxes of a slab's 16 values x 64 tokens (d_v % 8 == 0)
};

namespace {

// Calls of up to 32 sequences and 16 chunk CTAs an SM need no plan kernel: every warp of the other two
// works the plan out for itself, a lane a sequence (17 tokens: 19.4 -> 16.9 us; but 16 x 1024 tokens,
// 29 chunk CTAs an SM: 564 -> 574).
constexpr int kWarpSeqs = 32;
struct GdnWarpPlan {
  GdnSeq seq;            // this lane's sequence (n < 0: left out, or none)
  int nc, n_chunks;      // its chunks, the call's
  bool bad;
};
__device__ __forceinline__ GdnWarpPlan gdn_warp_plan(const GdnPrefillArgs& a, int lane) {
  const bool in = lane < a.n_seqs;
  const int r0 = in ? a.offsets[lane] : 0, r1 = in ? a.offsets[lane + 1] : 0;
  const int seen = warp_excl_max(r0, lane);
  GdnWarpPlan p;
  const bool ok = in && rows_ok(r0, r1, seen, a.T);
  p.bad = in && !ok;
  p.nc = ok ? (r1 - r0 + kGdnChunk - 1) / kGdnChunk : 0;
  const int sum = warp_incl_sum(p.nc, lane);
  p.n_chunks = __shfl_sync(0xffffffffu, sum, 31);
  p.seq = GdnSeq{r0, ok ? r1 - r0 : -1, sum - p.nc};
  return p;
}
// Two slices a warp take less work, one a shorter time per chunk (6.5 against 4.5 us with all of an
// SM's warps at work): one where the longest sequence's chunks would take longer than all chunks
// spread over the SMs (lengths 1 to 1,531, ten sequences: 209 -> 180 us; four of 1,024: 191 against
// 159, so two there).
__device__ __forceinline__ bool gdn_chain(const GdnPrefillArgs& a, int longest, int n_chunks) {
  return (float)longest * a.n_sm > 1.2f * n_chunks * a.Hv * ((a.dv + 127) / 128);
}

__global__ void __launch_bounds__(kPlanThreads) k_gdn_plan(const GdnPrefillArgs a) {
  __shared__ int sh[32];
  __shared__ int s_longest;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) s_longest = 0;
  int seen = 0, chunks = 0;
  for (int base = 0; base < a.n_seqs; base += kPlanThreads) {
    const int i = base + tid;
    const bool in = i < a.n_seqs;
    const int r0 = in ? a.offsets[i] : 0, r1 = in ? a.offsets[i + 1] : 0;
    const int before = block_excl_max(r0, seen, sh);
    const bool ok = in && rows_ok(r0, r1, before, a.T);
    const int nc = ok ? (r1 - r0 + kGdnChunk - 1) / kGdnChunk : 0;
    const int c0 = block_excl_sum(nc, chunks, sh);
    if (!in) continue;
    a.seqs[i] = GdnSeq{r0, ok ? r1 - r0 : -1, c0};
    if (ok) atomicMax(&s_longest, nc);
    if (!ok) atomicOr(&a.ctrl->err, kErrBadRange);
  }
  __syncthreads();
  if (tid == 0) {
    a.hdr->n_chunks = chunks;
    a.hdr->chain = gdn_chain(a, s_longest, chunks);
  }
  for (int s = warp; s < a.n_seqs; s += kPlanThreads / 32) {
    const GdnSeq q = a.seqs[s];
    for (int c = lane; c * kGdnChunk < q.n; c += 32)
      a.chunks[q.chunk0 + c] = GdnChunk{q.row0 + c * kGdnChunk, min(kGdnChunk, q.n - c * kGdnChunk)};
  }
  // Sequences by length, longest first, in kPlanThreads classes; inside a class by number, so that the
  // order (which may decide a sequence's slices, and with them its bits) is the call's and not the
  // warps': a warp takes consecutive sequences, and its places in a class follow the earlier warps'.
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int s_bins[kWarps][kPlanThreads];
  for (int w = 0; w < kWarps; ++w) s_bins[w][tid] = 0;
  __syncthreads();
  const int per = a.T / (kPlanThreads - 1) + 1, share = (a.n_seqs + kPlanThreads - 1) / kPlanThreads * 32;
  const int end = min(a.n_seqs, (warp + 1) * share);
  for (int pass = 0; pass < 2; ++pass) {
    for (int base = warp * share; base < end; base += 32) {
      const int i = base + lane;
      const int bin = i < end ? kPlanThreads - 1 - max(0, a.seqs[i].n) / per : kPlanThreads;
      const unsigned same = __match_any_sync(0xffffffffu, bin);
      const int at = i < end ? s_bins[warp][bin] + __popc(same & ((1u << lane) - 1)) : 0;
      __syncwarp();  // every lane has read its class's count
      if (i < end) {
        if (pass) a.order[at] = i;
        if (lane == __ffs(same) - 1) s_bins[warp][bin] += __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
    if (!pass) {
      int count = 0, total = 0;
      for (int w = 0; w < kWarps; ++w) count += s_bins[w][tid];
      int first = block_excl_sum(count, total, sh);
      for (int w = 0; w < kWarps; ++w) {
        const int n = s_bins[w][tid];
        s_bins[w][tid] = first;
        first += n;
      }
      __syncthreads();
    }
  }
}

// d (16 x 8, fp32) += a (16 x 16, fp16) b (16 x 8, fp16); mma16z: d = a b.  With g = lane / 4,
// u = 2 (lane % 4): d[0] = row g, columns u, u + 1, d[1] = row g + 8; a0 = (g, u..), a1 = (g + 8, u..),
// a2 = (g, u + 8..), a3 = (g + 8, u + 8..); b0 = (k u.., n g), b1 = (k u + 8.., n g).
__device__ __forceinline__ void mma16(float2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16z(float2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0].x), "=f"(d[0].y), "=f"(d[1].x), "=f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_h2(float2 v) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The power of two that brings a largest element m to [2^TOP, 2^{TOP + 1}) (exact; 0 and values
// below 2^{TOP - 126} by 2^126), and its inverse.
template <int TOP>
__device__ __forceinline__ void pow2_scale(float m, float& up, float& down) {
  const int e = max((int)(__float_as_uint(m) >> 23) - 127 - TOP, -126);
  up = __uint_as_float((uint32_t)(127 - e) << 23);
  down = __uint_as_float((uint32_t)(127 + e) << 23);
}

// (NaN if one is)
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Accumulators of N tiles of 8 columns (rows g and g + 8 of a slab) -> the largest element of
// each of the two rows over the warp's columns; NaN if one is.
template <int N>
__device__ __forceinline__ void row_max(const float2 (&v)[N][2], float (&m)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float x[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < N; ++t) x[t & 1] = max_nan3(x[t & 1], fabsf(v[t][e].x), fabsf(v[t][e].y));
    m[e] = max_nan(x[0], x[1]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m[0] = max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    m[1] = max_nan(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
  }
}
// x = hi + lo in fp16, as A operands: a step of 16 columns takes the registers of two tiles
__device__ __forceinline__ void split(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_h2(x);
  const float2 h = unpack_h2(hi);
  lo = pack_h2(ffma2(h, both(-1.f), x));
}

// ---------------------------------------------------------------------------------------
// k_gdn_chunk
// ---------------------------------------------------------------------------------------
constexpr int kChunkThreads = 256;  // four warps per value head, two value heads at a time
constexpr int kHeadThreads = 128;
// log2 of how far a state may grow in a chunk (g > 0).  P is held relative to the largest factor, in fp16
// times 2^10, and a row's W relative to its largest token: what comes before a growth of 2^16 is still
// rounded by 2^-19 and 2^-22 of its own size, and loses a bit with every doubling.  Beyond it the tokens
// go one by one.
constexpr float kMaxGrowth = 16.f;
constexpr int kMatLd = 68;          // row stride (floats) of the 64 x 64 matrices: 16-byte rows

template <int DK>
struct GdnChunkSmem {
  static constexpr int kImg = kGdnChunk * DK * 2;
  static constexpr int kMat = kGdnChunk * kMatLd * 4;
  // K and Q, later in their place L (then its inverse) of two heads; K K^T, Q K^T.  (Three CTAs an SM.)
  static constexpr int kFirst = 2 * kImg > 2 * kMat ? 2 * kImg : 2 * kMat;
  static constexpr int kBytes = kFirst + 2 * kMat;
};

// 2^(a - b) of sums held as two floats: the difference of the heads is exact or as good as its size
__device__ __forceinline__ float decay(float2 a, float2 b) { return ex2((a.x - b.x) + (a.y - b.y)); }

__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kHeadThreads) : "memory");
}

// d (16 x 8, fp32) += a (16 x 8) b (8 x 8), both fp32 in shared memory with rows of kMatLd, as the
// products of their tf32 heads and rests.  A head is cut off after 10 bits, so a rest is below 2^-10 of its
// element, and the tensor core takes 10 bits of it: rest times rest, and the rests' ends, are below 2^-20 of
// a product.
__device__ __forceinline__ void tf32_parts(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;  // 10 mantissa bits: exact in tf32
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One step of the block inversion: C <- -D (C A) for the block C of B x B below the diagonal, with
// the inverses A above and D right of it in place.  A warp makes 16 rows and B / 2 columns (B = 16: two warps
// a block, B = 32: four).
template <int B>
__device__ __forceinline__ void join_blocks(float* C, const float* A, const float* D, int part, int lane, int team) {
  constexpr int NT = B / 16;
  const int g = lane >> 2, t = lane & 3, r = (part >> 1) * 16 + g, c = (part & 1) * (B / 2) + g;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float* x = half ? D : C;
    const float* y = half ? C : A;
    float s[NT][4] = {};
#pragma unroll
    for (int k = 0; k < B; k += 8) {
      uint32_t ah[4], al[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) tf32_parts(x[(r + 8 * (e & 1)) * kMatLd + k + t + 4 * (e >> 1)], ah[e], al[e]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t bh[2], bl[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) tf32_parts(y[(k + t + 4 * e) * kMatLd + c + n * 8], bh[e], bl[e]);
        mma_tf32(s[n], ah, bh[0], bh[1]);
        mma_tf32(s[n], ah, bl[0], bl[1]);
        mma_tf32(s[n], al, bh[0], bh[1]);
      }
    }
    team_sync(team);  // every thread has read C
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = half ? -1.f : 1.f;
        *reinterpret_cast<float2*>(C + (r + 8 * e) * kMatLd + (c - g) + n * 8 + 2 * t) = make_float2(f * s[n][2 * e], f * s[n][2 * e + 1]);
      }
    team_sync(team);
  }
}

// (I + L)^-1 in place of the strictly lower triangular L (zeros elsewhere), by a team of 128
// threads: the four 16 x 16 diagonal blocks by forward substitution, a thread a column, then
// joined to blocks of 32 and of 64 on the tensor cores (on the FMA units the joins were bound by
// shared-memory reads: 17 us more for the 16,384 tokens and 32 heads of a batch).
__device__ __forceinline__ void invert(float* L, int t, int team) {
  if (t < kGdnChunk) {
    const int b = t / 16, j = t % 16;
    float* D = L + b * 16 * kMatLd + b * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[2] = {i == j ? 1.f : 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < i; ++m) s[m & 1] = fmaf(-D[i * kMatLd + m], x[m], s[m & 1]);
      x[i] = s[0] + s[1];
    }
    __syncwarp();  // the block's columns are all in this warp: they have all read it
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i * kMatLd + j] = x[i];
  }
  team_sync(team);
  {
    float* D = L + (t / 64) * 32 * (kMatLd + 1);
    join_blocks<16>(D + 16 * kMatLd, D, D + 16 * (kMatLd + 1), (t >> 5) & 1, t & 31, team);
  }
  join_blocks<32>(L + 32 * kMatLd, L, L + 32 * (kMatLd + 1), t >> 5, t & 31, team);
}

template <int DK>
__global__ void __launch_bounds__(kChunkThreads, DK == 256 ? 1 : 3) k_gdn_chunk(const GdnPrefillArgs a) {
  using M = GdnChunkSmem<DK>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_up[2 * kGdnChunk], s_ck[kGdnChunk], s_cq[kGdnChunk], s_beta[2][kGdnChunk];
  __shared__ float2 s_G[2][kGdnChunk];  // log2(e) G_i, as two floats
  __shared__ float s_pm[2];             // the largest G_i - G_j, j <= i (0 where nothing grows)
  __shared__ float s_red[2][6];
  __shared__ int s_plain[3];            // a head's decays or writes, or the keys, ask for single tokens
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_plain[2] = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int chunk = blockIdx.x / a.Hk, kh = blockIdx.x - chunk * a.Hk;
  GdnChunk C;
  if (a.warp_plan) {
    const GdnWarpPlan p = gdn_warp_plan(a, lane);
    if (chunk >= p.n_chunks) return;
    const int at = chunk - p.seq.chunk0, src = __ffs(__ballot_sync(0xffffffffu, at >= 0 && at < p.nc)) - 1;
    C.row0 = __shfl_sync(0xffffffffu, p.seq.row0 + at * kGdnChunk, src);
    C.n = __shfl_sync(0xffffffffu, min(kGdnChunk, p.seq.n - at * kGdnChunk), src);
  } else {
    const int n_chunks = a.hdr->n_chunks;
    C = a.chunks[chunk];  // the grid is the table's size; behind n_chunks it holds anything
    if (chunk >= n_chunks) return;
  }
  uint8_t* img[2] = {smem, smem + M::kImg};
  float* kk = reinterpret_cast<float*>(smem + M::kFirst);
  float* qk = kk + kGdnChunk * kMatLd;
  float* Lh = reinterpret_cast<float*>(smem);  // once the products have read K and Q
  const int rep = a.Hv / a.Hk, team = tid / kHeadThreads, tt = tid % kHeadThreads, tw = warp & 3;
  float* L = Lh + team * kGdnChunk * kMatLd;

  // K and Q: rows scaled to a norm in [2^10, 2^11), as fp16.  A row is DK / 8 pieces of 16 bytes, a
  // lane each; all of a thread's pieces are loaded before the first is used.
  constexpr int LPR = DK / 8, N = 2 * kGdnChunk * LPR / kChunkThreads;  // lanes per row, pieces per thread
  {
    uint4 piece[N];
    uint4* dst = reinterpret_cast<uint4*>(a.img + ((size_t)chunk * a.Hk + kh) * 2 * M::kImg);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = i * (kChunkThreads / LPR) + tid / LPR, row = r & 63;  // K, then Q
      piece[i] = make_uint4(0, 0, 0, 0);
      if (row < C.n)
        piece[i] = *reinterpret_cast<const uint4*>((i >= N / 2 ? a.q : a.k) + ((size_t)(C.row0 + row) * a.Hk + kh) * DK + tid % LPR * 8);
    }
    // the rows' sums of squares side by side, then their scales, then the values
    float ss[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ss[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = word_of(piece[i], e);
        ss[i] = fmaf(bf_lo(w), bf_lo(w), fmaf(bf_hi(w), bf_hi(w), ss[i]));
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
    const int col = tid % LPR;
    if (col == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s_up[i * (kChunkThreads / LPR) + tid / LPR] = ss[i];
    __syncthreads();
    if (tid < 2 * kGdnChunk) {  // a thread a row
      const float norm = sqrtf(s_up[tid]);
      // 2^e2 brings the norm to [2^10, 2^11).  A row of a norm below 2^-100 (it vanishes next to
      // 1e-6), and one whose sum of squares overflows (1 / inf), is 0; infinities and NaN give NaN.
      const int ne = (int)(__float_as_uint(norm) >> 23) - 127;
      const bool zero = ne <= -100 || ne == 128;
      const float down = zero ? 0.f : __uint_as_float((uint32_t)(117 + ne) << 23);
      const float c = zero ? 0.f : down / fmaxf(norm, 1e-6f);  // the normalised row is c times the stored one
      s_up[tid] = zero ? 0.f : __uint_as_float((uint32_t)(137 - ne) << 23);
      if (tid < kGdnChunk) s_ck[tid] = c;
      else s_cq[tid - kGdnChunk] = c * rsqrtf((float)DK);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = i * (kChunkThreads / LPR) + tid / LPR, row = r & 63;
      const float up = s_up[r];
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = word_of(piece[i], e);
        h[e] = pack_h2(mul2(make_float2(bf_lo(w), bf_hi(w)), both(up)));
        if (up == 0.f && i < N / 2 && bf16x2_nonfinite(w)) s_plain[2] = 1;  // (rows of a finite norm have none)
      }
      const int at = r * LPR + (col ^ (row & 7));
      const uint4 hv = make_uint4(h[0], h[1], h[2], h[3]);
      reinterpret_cast<uint4*>(smem)[at] = hv;
      dst[at] = hv;
    }
  }
  // Decays: sums in 64 bits (their differences have to be good to 24; a forgotten state's g is
  // clamped, e^-1e4 = 0), kept as two floats, in units of log 2; one warp per head
  auto decays = [&](int h) {
    double x[2];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * lane + e;
      const float gt = t < C.n ? a.g[(size_t)(C.row0 + t) * a.Hv + h] : 0.f;
      const float bt = t < C.n ? a.beta[(size_t)(C.row0 + t) * a.Hv + h] : 0.f;
      x[e] = (gt < -1e4f ? -1e4 : (double)gt) * 1.4426950408889634;
      s_beta[team][t] = bt;
      bad |= !(gt < INFINITY) || !(fabsf(bt) < INFINITY);
    }
    double sum = x[0] + x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    const double g1 = sum, g0 = sum - x[1];
    double low = fmin(g0, g1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_up_sync(0xffffffffu, low, o);
      if (lane >= o) low = fmin(low, u);
    }
    const double before = __shfl_up_sync(0xffffffffu, low, 1);
    const auto two = [](double v) { return make_float2((float)v, (float)(v - (double)(float)v)); };
    s_G[team][2 * lane] = two(g0);
    s_G[team][2 * lane + 1] = two(g1);
    float up = (float)fmax(lane ? g0 - fmin(before, g0) : 0.0, g1 - low);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
    bad = __any_sync(0xffffffffu, bad) || up > kMaxGrowth;
    if (lane == 0) {
      s_pm[team] = up;
      s_plain[team] = bad;
    }
  };
  if (tw == 0 && team < rep) decays(kh * rep + team);
  __syncthreads();
  // K K^T and Q K^T, lower triangle: rows in tiles of 16 (A), columns in pairs of tiles of 8 (B)
  for (int w = warp; w < 20; w += kChunkThreads / 32) {
    const int z = w / 10, u = w % 10;  // u: (row tile i, column pair j <= i)
    const int i = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, j = u - i * (i + 1) / 2;
    const uint32_t sa = smem_u32(img[z]), sb = smem_u32(img[0]);
    const int ra = i * 16 + (lane & 15), rb = j * 16 + (lane & 7) + ((lane >> 4) << 3);
    float2 d[2][2] = {};
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      uint32_t A[4], B[4];
      ldsm4(sa + ra * DK * 2 + (((2 * k + (lane >> 4)) ^ (ra & 7)) << 4), A);
      ldsm4(sb + rb * DK * 2 + (((2 * k + ((lane >> 3) & 1)) ^ (rb & 7)) << 4), B);
      mma16(d[0], A[0], A[1], A[2], A[3], B[0], B[1]);
      mma16(d[1], A[0], A[1], A[2], A[3], B[2], B[3]);
    }
    float* dst = z ? qk : kk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r = i * 16 + (lane >> 2), c = j * 16 + t * 8 + 2 * (lane & 3);
      *reinterpret_cast<float2*>(dst + r * kMatLd + c) = d[t][0];
      *reinterpret_cast<float2*>(dst + (r + 8) * kMatLd + c) = d[t][1];
    }
  }
  __syncthreads();
  for (int h0 = 0; h0 < rep; h0 += 2) {
    const bool on = h0 + team < rep;
    const int h = kh * rep + h0 + team;
    if (h0 > 0) {
      if (on && tw == 0) decays(h);
      __syncthreads();
    }
    GdnTP* tp = a.tp + (size_t)chunk * a.Hv + h;
    if (on) {
      // L by rows: a warp a row, a lane the columns lane and lane + 32
      float2 Gj[2];
      float cj[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        Gj[c] = s_G[team][c * 32 + lane];
        cj[c] = s_ck[c * 32 + lane];
      }
#pragma unroll 4
      for (int i = tw; i < kGdnChunk; i += 4) {
        const float2 Gi = s_G[team][i];
        const float f = s_beta[team][i] * s_ck[i];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int j = c * 32 + lane;
          float l = 0.f;
          if (c * 32 < i) l = j < i ? f * decay(Gi, Gj[c]) * cj[c] * kk[i * kMatLd + j] : 0.f;
          L[i * kMatLd + j] = l;
        }
      }
      team_sync(team);
      invert(L, tt, team);
      // P: block x of 20 is (token tile, step).  Held relative to the largest decay factor (1
      // unless a state grows, see kMaxGrowth) and times 2^10 (fp16's range)
      const float pm = s_pm[team];
      for (int x = tw; x < GdnTP::kBlocks; x += 4) {
        const int half = x < 2 ? 0 : x < 6 ? 1 : x < 12 ? 2 : 3;
        const int rest = x - half * (half + 1), tile = 2 * half + rest / (half + 1), ks = rest % (half + 1);
        const int i = tile * 8 + (lane >> 2), c0 = ks * 16 + 2 * (lane & 3);
        float2 Gi = s_G[team][i];
        Gi.y -= pm;
        const float cq = s_cq[i] * 1024.f;
        uint32_t o[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = c0 + e * 8;
          const float4 Gc = *reinterpret_cast<const float4*>(&s_G[team][c]);
          const float2 ck = *reinterpret_cast<const float2*>(&s_ck[c]), x2 = *reinterpret_cast<const float2*>(qk + i * kMatLd + c);
          const float p0 = decay(Gi, make_float2(Gc.x, Gc.y)) * (cq * ck.x) * x2.x;
          const float p1 = decay(Gi, make_float2(Gc.z, Gc.w)) * (cq * ck.y) * x2.y;
          o[e] = pack_h2(make_float2(c <= i ? p0 : 0.f, c + 1 <= i ? p1 : 0.f));
        }
        tp->p[x][lane] = make_uint2(o[0], o[1]);
      }
      // T' by token tiles (a warp takes tiles tw and 7 - tw: five blocks), scaled to its largest
      // element, and the factors of token tt
      float v[2][4][4], m = 0.f, wd = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int tile = y ? 7 - tw : tw, i = tile * 8 + (lane >> 2);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int c = k * 16 + 2 * (lane & 3) + e * 4;
            float2 x = make_float2(0.f, 0.f);
            if (k <= tile / 2) {
              x = *reinterpret_cast<const float2*>(L + i * kMatLd + c);
              const float2 b = *reinterpret_cast<const float2*>(&s_beta[team][c]);
              x = make_float2(c <= i ? x.x * b.x : 0.f, c + 1 <= i ? x.y * b.y : 0.f);
            }
            v[y][k][e] = x.x;
            v[y][k][e + 1] = x.y;
            m = max_nan3(m, fabsf(x.x), fabsf(x.y));
          }
      }
      if (tt < kGdnChunk) {
        const float2 G = s_G[team][tt];
        const float eg = decay(G, make_float2(0.f, 0.f));
        wd = decay(s_G[team][kGdnChunk - 1], G) * s_ck[tt];
        tp->xa[tt] = -eg * s_ck[tt];
        tp->oa[tt] = eg * s_cq[tt];
      }
      float mw = wd;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
      }
      if (lane == 0) {
        s_red[team][tw] = m;
        if (tw < 2) s_red[team][4 + tw] = mw;
      }
      team_sync(team);
      float up, down, upw, downw;
      const float t_max = max_nan(max_nan(s_red[team][0], s_red[team][1]), max_nan(s_red[team][2], s_red[team][3]));
      pow2_scale<14>(t_max, up, down);
      pow2_scale<0>(fmaxf(s_red[team][4], s_red[team][5]), upw, downw);
      if (tt < kGdnChunk) tp->wd[tt] = wd * upw;
      if (tt == 0) {
        tp->keep = decay(s_G[team][kGdnChunk - 1], make_float2(0.f, 0.f));
        tp->t_scale = down;
        tp->p_scale = ex2(pm) * 0x1p-10f;
        tp->wd_scale = downw;
        // (the rule contracts for 0 <= beta <= 2: |T'| <= 4.  Far above it the writes grow as a state may.)
        tp->plain = s_plain[team] | s_plain[2] | !(t_max < 0x1p10f);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int tile = y ? 7 - tw : tw;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k > tile / 2) continue;
          uint4 o;
          split(make_float2(v[y][k][0] * up, v[y][k][1] * up), o.x, o.z);
          split(make_float2(v[y][k][2] * up, v[y][k][3] * up), o.y, o.w);
          tp->t[gdn_block(tile, k)][lane] = o;
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
// k_gdn_scan
// ---------------------------------------------------------------------------------------
// NS: slices of 64 state columns of a warp
template <int DK, int NS>
struct GdnScanSmem {
  static constexpr int kWarps = DK / (kGdnSlice * NS);      // warps of a slab
  static constexpr int kImg = kGdnChunk * DK * 2;
  static constexpr int kTp = 2 * kImg;                      // stage: K, Q, T' and P, V
  static constexpr int kV = kTp + (int)sizeof(GdnTP);
  static constexpr int kVSlab = kGdnChunk * kGdnSlab * 2;   // 32-byte rows, 16-byte pieces XORed with bit 2 of the row
  static constexpr int stage(int slabs) { return kV + slabs * kVSlab; }
  // exchange: per slab and warp, 8 tiles of S k and 8 of S q
  static constexpr int kXch = kWarps > 1 ? kWarps * 16 * 512 : 0;
  static constexpr int bytes(int slabs) { return 2 * stage(slabs) + slabs * kXch + 256; }
};

__device__ __forceinline__ void slab_sync(int slab, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(slab + 1), "r"(threads) : "memory");
}
__device__ __forceinline__ float4 cat(const float2 (&d)[2]) { return make_float4(d[0].x, d[0].y, d[1].x, d[1].y); }

// Chunk c of a slab, its tokens one by one in fp32, as the decode step does them (k_gdn_step): for chunks
// with infinities or NaN, which then reach the tokens behind them alone, and chunks that grow too far
// (kMaxGrowth).  All of the slab's warps call it;
// xch: its exchange area.  (1.6 us a token, where the chunk takes 3 us in one go; that every chunk can come
// here costs the others 1 to 2 %: 16 x 1024 tokens 549 -> 562 us, 1 x 8192 437 -> 441.)
template <int DK, int NS>
__device__ __forceinline__ void gdn_tokens(const GdnPrefillArgs& a, const GdnSeq seq, int c, int h, int vr, int slab, int w,
                                           float2 (&S)[NS * 8][2], float* xch) {
  constexpr int NW = DK / (kGdnSlice * NS);
  const int lane = threadIdx.x & 31, g = lane >> 2, u = 2 * (lane & 3), kh = h / (a.Hv / a.Hk);
  const auto slab_sum = [&](float (&x)[2], float* at) {  // over the columns of rows g and g + 8
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
      x[1] += __shfl_xor_sync(0xffffffffu, x[1], o);
    }
    if constexpr (NW > 1) {
      if ((lane & 3) == 0) {
        at[w * kGdnSlab + g] = x[0];
        at[w * kGdnSlab + g + 8] = x[1];
      }
      slab_sync(slab, NW * 32);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[e] = at[g + 8 * e];
#pragma unroll
        for (int v = 1; v < NW; ++v) x[e] += at[v * kGdnSlab + g + 8 * e];
      }
    }
  };
  for (int i = 0; i < min(kGdnChunk, seq.n - c * kGdnChunk); ++i) {
    const size_t row = (size_t)seq.row0 + c * kGdnChunk + i;
    float2 x[2][NS * 8];  // k^, q^: this lane's columns
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint16_t* src = (z ? a.q : a.k) + (row * a.Hk + kh) * DK;
      float ss = 0.f;
      for (int j = 2 * lane; j < DK; j += 64) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(src + j);
        ss = fmaf(bf_lo(v), bf_lo(v), fmaf(bf_hi(v), bf_hi(v), ss));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = 1.0f / fmaxf(sqrtf(ss), 1e-6f) * (z ? rsqrtf((float)DK) : 1.f);
#pragma unroll
      for (int t = 0; t < NS * 8; ++t) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(src + w * NS * kGdnSlice + t * 8 + u);
        x[z][t] = make_float2(bf_lo(v) * inv, bf_hi(v) * inv);
      }
    }
    const float alpha = expf(a.g[row * a.Hv + h]), beta = a.beta[row * a.Hv + h];
    float r[2] = {0.f, 0.f}, o[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NS * 8; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) r[e] = fmaf(S[t][e].x, x[0][t].x, fmaf(S[t][e].y, x[0][t].y, r[e]));
    slab_sum(r, xch);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = vr + 8 * e < a.dv ? bf1(a.v[(row * a.Hv + h) * a.dv + vr + 8 * e]) : 0.f;
      const float f = beta * (v - alpha * r[e]);
#pragma unroll
      for (int t = 0; t < NS * 8; ++t) {
        S[t][e].x = fmaf(alpha, S[t][e].x, f * x[0][t].x);
        S[t][e].y = fmaf(alpha, S[t][e].y, f * x[0][t].y);
        o[e] = fmaf(S[t][e].x, x[1][t].x, fmaf(S[t][e].y, x[1][t].y, o[e]));
      }
    }
    slab_sum(o, xch + NW * kGdnSlab);
    if (w == 0 && (lane & 3) == 0)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (vr + 8 * e < a.dv) a.out[(row * a.Hv + h) * a.dv + vr + 8 * e] = f2bf(o[e]);
  }
  if constexpr (NW > 1) slab_sync(slab, NW * 32);  // the area is the next chunk's again
}

// One CTA's slabs of one sequence and value head: state rows rb * slabs * 16 and on.
template <int DK, int NS>
__device__ __forceinline__ void gdn_scan(const GdnPrefillArgs& a, const int slabs, const GdnSeq seq, int s, int h, int rb,
                                         uint8_t* smem, uint64_t* full) {
  using M = GdnScanSmem<DK, NS>;
  constexpr int NW = M::kWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slab = warp / NW, w = warp - slab * NW;
  const int g = lane >> 2, u = 2 * (lane & 3);
  const int stage_bytes = M::stage(slabs);
  const int kh = h / (a.Hv / a.Hk);
  const int n_ch = (seq.n + kGdnChunk - 1) / kGdnChunk;
  const int v0 = rb * slabs * kGdnSlab;       // first state row of the CTA
  const int vr = v0 + slab * kGdnSlab + g;      // this lane's rows: vr and vr + 8
  const size_t state = (size_t)s * a.Hv + h;
  const size_t s_at = (state * a.dv + vr) * DK + w * NS * kGdnSlice + u;  // this lane's first element

  float2 S[NS * 8][2];  // tiles of 8 columns
#pragma unroll
  for (int t = 0; t < NS * 8; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      S[t][e] = make_float2(0.f, 0.f);
      if (a.S_in && vr + 8 * e < a.dv) S[t][e] = *reinterpret_cast<const float2*>(a.S_in + s_at + 8 * e * DK + t * 8);
    }

  const bool v_tma = a.dv % 8 == 0;  // a copy's strides are multiples of 16 bytes
  auto load = [&](int c) {  // chunk c into its stage
    uint8_t* st = smem + (c & 1) * stage_bytes;
    const size_t ch = (size_t)seq.chunk0 + c;
    const int row0 = seq.row0 + c * kGdnChunk;
    if (tid == 0) {
      mbar_expect_tx(&full[c & 1], M::kV + (v_tma ? slabs * M::kVSlab : 0));
      bulk_g2s(st, a.img + (ch * a.Hk + kh) * 2 * M::kImg, 2 * M::kImg, &full[c & 1]);
      bulk_g2s(st + M::kTp, a.tp + ch * a.Hv + h, sizeof(GdnTP), &full[c & 1]);
      if (v_tma)  // values behind d_v and rows behind T are zeros, rows of the next sequence are cleared below
        for (int x = 0; x < slabs; ++x)
          tma_3d(smem_u32(st + M::kV + x * M::kVSlab), &a.map_v, v0 + x * kGdnSlab, h, row0, &full[c & 1]);
    }
    if (!v_tma) {
      const int n = min(kGdnChunk, seq.n - c * kGdnChunk);
      for (int i = tid; i < slabs * kGdnChunk * 2; i += blockDim.x) {  // per slab, token and half (8 values)
        const int half = i % (2 * slabs), r = i / (2 * slabs), col = v0 + half * 8;
        uint8_t* dst = st + M::kV + (half >> 1) * M::kVSlab + r * 32 + (((half & 1) ^ ((r >> 2) & 1)) << 4);
        const uint16_t* src = a.v + ((size_t)(row0 + r) * a.Hv + h) * a.dv + col;
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t l0 = r < n && col + 2 * e < a.dv ? src[2 * e] : 0, l1 = r < n && col + 2 * e + 1 < a.dv ? src[2 * e + 1] : 0;
          x[e] = l0 | (l1 << 16);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  };

  // byte offsets of this lane's operand rows (the pieces' XOR depends on the lane alone)
  uint32_t off_n[NS][2], off_t[NS][4];
#pragma unroll
  for (int sl = 0; sl < NS; ++sl) {
    const int p0 = (w * NS + sl) * 8;  // first 16-byte piece of the slice
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) off_n[sl][k2] = (lane & 7) * DK * 2 + (((p0 + k2 * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
#pragma unroll
    for (int t2 = 0; t2 < 4; ++t2) off_t[sl][t2] = (lane & 15) * DK * 2 + (((p0 + 2 * t2 + (lane >> 4)) ^ (lane & 7)) << 4);
  }

  bool ok = true;
  bool plain = false;  // this slab has left the chunk before undone (every warp of a slab says the same)
  int issued = 0;
  if (n_ch > 0) load(issued++);
  for (int c = 0;; ++c) {
    // everyone is done with the other stage and with the exchange area (and the plain stores of
    // this chunk's V are visible)
    if (__syncthreads_or(!ok || plain)) {
      ok = !__syncthreads_or(!ok);
      if (!ok) break;
      if (plain) gdn_tokens<DK, NS>(a, seq, c - 1, h, vr, slab, w, S, reinterpret_cast<float*>(smem + 2 * stage_bytes + slab * M::kXch));
      plain = false;
    }
    if (c == n_ch) break;
    if (c + 1 < n_ch) load(issued++);
    ok = mbar_wait(&full[c & 1], (c >> 1) & 1);
    const uint32_t st = smem_u32(smem) + (c & 1) * stage_bytes;
    const GdnTP* tp = reinterpret_cast<const GdnTP*>(smem + (c & 1) * stage_bytes + M::kTp);

    // ---- X^T = S K^T (hi, lo) and Y^T = S Q^T (hi), over this warp's columns ----
    float2 X[8][2], Y[8][2];
    {
      float m[2], up[2], dn[2];
      row_max(S, m);
      pow2_scale<14>(m[0], up[0], dn[0]);
      pow2_scale<14>(m[1], up[1], dn[1]);
#pragma unroll
      for (int sl = 0; sl < NS; ++sl) {
        uint32_t hi[8][2], lo[8][2];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) split(mul2(S[sl * 8 + t][e], both(up[e])), hi[t][e], lo[t][e]);
#pragma unroll
        for (int tg = 0; tg < 8; tg += 4) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // K, then Q
            uint32_t B[4][2][4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int k2 = 0; k2 < 2; ++k2) ldsm4(st + z * M::kImg + (tg + t) * 8 * DK * 2 + off_n[sl][k2], B[t][k2]);
            float2 (&D)[8][2] = z ? Y : X;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a0 = hi[2 * k][0], a1 = hi[2 * k][1], a2 = hi[2 * k + 1][0], a3 = hi[2 * k + 1][1];
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint32_t b0 = B[t][k >> 1][2 * (k & 1)], b1 = B[t][k >> 1][2 * (k & 1) + 1];
                if (sl == 0 && k == 0) mma16z(D[tg + t], a0, a1, a2, a3, b0, b1);
                else mma16(D[tg + t], a0, a1, a2, a3, b0, b1);
              }
              if (!z) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                  mma16(D[tg + t], lo[2 * k][0], lo[2 * k][1], lo[2 * k + 1][0], lo[2 * k + 1][1],
                        B[t][k >> 1][2 * (k & 1)], B[t][k >> 1][2 * (k & 1) + 1]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          X[t][e] = mul2(X[t][e], both(dn[e]));
          Y[t][e] = mul2(Y[t][e], both(dn[e]));
        }
    }
    // ---- sums over the slab's warps, each the same in the same order: of X here, of Y at the output,
    // where a warp finishes the tiles t % NW == w ----
    float4* xch = reinterpret_cast<float4*>(smem + 2 * stage_bytes + slab * M::kXch);
    if constexpr (NW > 1) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        xch[(w * 16 + t) * 32 + lane] = cat(X[t]);
        xch[(w * 16 + 8 + t) * 32 + lane] = cat(Y[t]);
      }
      slab_sync(slab, NW * 32);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if constexpr (NW == 2) {  // the sum of two is the same either way
          const float4 x = xch[((1 - w) * 16 + t) * 32 + lane];
          X[t][0] = add2(X[t][0], make_float2(x.x, x.y));
          X[t][1] = add2(X[t][1], make_float2(x.z, x.w));
        } else {
#pragma unroll
          for (int v = 0; v < NW; ++v) {
            const float4 x = xch[(v * 16 + t) * 32 + lane];
            X[t][0] = v ? add2(X[t][0], make_float2(x.x, x.y)) : make_float2(x.x, x.y);
            X[t][1] = v ? add2(X[t][1], make_float2(x.z, x.w)) : make_float2(x.z, x.w);
          }
        }
      }
    }
    // ---- R^T = V^T - e^G S k ----
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
      uint32_t r[4];  // (tile t, rows g), (t, g + 8), (t + 1, g), (t + 1, g + 8)
      const int row = (t + (lane >> 4)) * 8 + (lane & 7), half = (lane >> 3) & 1;
      ldsm4_t(st + M::kV + slab * M::kVSlab + row * 32 + ((half ^ ((row >> 2) & 1)) << 4), r);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float2 xa = *reinterpret_cast<const float2*>(&tp->xa[(t + y) * 8 + u]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          X[t + y][e] = ffma2(xa, X[t + y][e], make_float2(bf_lo(r[2 * y + e]), bf_hi(r[2 * y + e])));
      }
    }
    if (v_tma && seq.n - c * kGdnChunk < kGdnChunk) {  // tokens behind the sequence: V's rows are another's
      const int n = seq.n - c * kGdnChunk;
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (t * 8 + u >= n) X[t][e].x = 0.f;
          if (t * 8 + u + 1 >= n) X[t][e].y = 0.f;
        }
    }
    // ---- W^T = R^T T'^T, left as W 2^k (W = fw * what is held) ----
    float2 W[8][2];
    float fw[2];
    {
      float m[2], up[2], dn[2];
      row_max(X, m);
      // An infinity or NaN in one token's R would reach the tokens before it (as 0 times it, and through
      // the row's scale): the slab then does the chunk's tokens one by one, behind the next barrier.  Not
      // where the row's first R is one already (a state that holds one): all of the row becomes NaN.
      if (__any_sync(0xffffffffu, tp->plain || !(max_nan(m[0], m[1]) < INFINITY))) {
        bool need = tp->plain;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float first = __shfl_sync(0xffffffffu, X[0][e].x, lane & 28);  // (every lane takes part)
          need |= !(m[e] < INFINITY) && fabsf(first) < INFINITY;
        }
        plain = __any_sync(0xffffffffu, need);
        if (plain) continue;
      }
      pow2_scale<14>(m[0], up[0], dn[0]);
      pow2_scale<14>(m[1], up[1], dn[1]);
      uint32_t hi[8][2], lo[8][2];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) split(mul2(X[t][e], both(up[e])), hi[t][e], lo[t][e]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t h0 = hi[2 * k][0], h1 = hi[2 * k][1], h2 = hi[2 * k + 1][0], h3 = hi[2 * k + 1][1];
        uint4 b[8];
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) b[t] = tp->t[gdn_block(t, k)][lane];
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) {
          if (k == 0) mma16z(W[t], h0, h1, h2, h3, b[t].x, b[t].y);
          else mma16(W[t], h0, h1, h2, h3, b[t].x, b[t].y);
        }
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) mma16(W[t], h0, h1, h2, h3, b[t].z, b[t].w);
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) mma16(W[t], lo[2 * k][0], lo[2 * k][1], lo[2 * k + 1][0], lo[2 * k + 1][1], b[t].x, b[t].y);
      }
      row_max(W, m);
      const float ts = tp->t_scale;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float ua, da;
        pow2_scale<13>(m[e], ua, da);
        fw[e] = dn[e] * (da * ts);
#pragma unroll
        for (int t = 0; t < 8; ++t) W[t][e] = mul2(W[t][e], both(ua));
      }
    }
    // ---- O^T = e^G S q + W^T P^T, for this warp's token tiles ----
    {
      uint32_t hi[8][2];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        hi[t][0] = pack_h2(W[t][0]);
        hi[t][1] = pack_h2(W[t][1]);
      }
      const int n = min(kGdnChunk, seq.n - c * kGdnChunk);
      const float ps = tp->p_scale, f0 = fw[0] * ps, f1 = fw[1] * ps;
      uint16_t* out = a.out + ((size_t)(seq.row0 + c * kGdnChunk) * a.Hv + h) * a.dv;
      const size_t tok_stride = (size_t)a.Hv * a.dv;
      // tiles t = i NW + w, their products side by side
      constexpr int NO = 8 / NW;
      float2 o[NO][2];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          // steps k <= t / 2; with NW = 4 that is 2 i + w / 2, and the step 2 i + 1 of the first two
          // warps reads another block and is not added
          if (k > (i * NW + NW - 1) / 2) continue;
          const int t = i * NW + w;
          const bool in = NW < 4 || k <= t / 2;
          uint2 b = tp->p[in ? gdn_block(t, k) : 0][lane];
          if (!in) b = make_uint2(0, 0);
          if (k == 0) mma16z(o[i], hi[0][0], hi[0][1], hi[1][0], hi[1][1], b.x, b.y);
          else mma16(o[i], hi[2 * k][0], hi[2 * k][1], hi[2 * k + 1][0], hi[2 * k + 1][1], b.x, b.y);
        }
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const int t = i * NW + w;
        const float2 oa = *reinterpret_cast<const float2*>(&tp->oa[t * 8 + u]);
        float2 y[2];
        if constexpr (NW == 1) {
          y[0] = Y[i][0];
          y[1] = Y[i][1];
        } else {
#pragma unroll
          for (int v = 0; v < NW; ++v) {
            const float4 x = xch[(v * 16 + 8 + t) * 32 + lane];
            y[0] = v ? add2(y[0], make_float2(x.x, x.y)) : make_float2(x.x, x.y);
            y[1] = v ? add2(y[1], make_float2(x.z, x.w)) : make_float2(x.z, x.w);
          }
        }
        o[i][0] = ffma2(oa, y[0], mul2(o[i][0], both(f0)));
        o[i][1] = ffma2(oa, y[1], mul2(o[i][1], both(f1)));
        if (a.dv % 2 == 0) {
          // pairs of columns: lanes of even g take the token u of rows g, g + 1, odd ones u + 1
          const int odd = g & 1, tok = t * 8 + u + odd, col = vr - odd;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? o[i][e].x : o[i][e].y, 4);
            const uint32_t v = odd ? pack_bf16(got, o[i][e].y) : pack_bf16(o[i][e].x, got);
            if (tok < n && col + 8 * e < a.dv) *reinterpret_cast<uint32_t*>(out + tok * tok_stride + col + 8 * e) = v;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = t * 8 + u + (e & 1), col = vr + 8 * (e >> 1);
            if (tok < n && col < a.dv) out[tok * tok_stride + col] = f2bf(e & 1 ? o[i][e >> 1].y : o[i][e >> 1].x);
          }
        }
      }
    }
    // ---- S' = e^{G_64} S + (e^{G_64 - G} W)^T K ----
    {
      uint32_t hi[8][2], lo[8][2];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float2 wd = *reinterpret_cast<const float2*>(&tp->wd[t * 8 + u]);
#pragma unroll
        for (int e = 0; e < 2; ++e) split(mul2(W[t][e], wd), hi[t][e], lo[t][e]);
      }
      const float keep = tp->keep, ws = tp->wd_scale, f[2] = {fw[0] * ws, fw[1] * ws};
#pragma unroll
      for (int sl = 0; sl < NS; ++sl) {
        float2 D[8][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t B[4][4];
#pragma unroll
          for (int t2 = 0; t2 < 4; ++t2) ldsm4_t(st + k * 16 * DK * 2 + off_t[sl][t2], B[t2]);
          const uint32_t h0 = hi[2 * k][0], h1 = hi[2 * k][1], h2 = hi[2 * k + 1][0], h3 = hi[2 * k + 1][1];
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            if (k == 0) mma16z(D[t], h0, h1, h2, h3, B[t >> 1][2 * (t & 1)], B[t >> 1][2 * (t & 1) + 1]);
            else mma16(D[t], h0, h1, h2, h3, B[t >> 1][2 * (t & 1)], B[t >> 1][2 * (t & 1) + 1]);
          }
#pragma unroll
          for (int t = 0; t < 8; ++t)
            mma16(D[t], lo[2 * k][0], lo[2 * k][1], lo[2 * k + 1][0], lo[2 * k + 1][1], B[t >> 1][2 * (t & 1)],
                  B[t >> 1][2 * (t & 1) + 1]);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) S[sl * 8 + t][e] = ffma2(D[t][e], both(f[e]), mul2(S[sl * 8 + t][e], both(keep)));
      }
    }
  }
  if (!ok) {  // a copy never landed: no state is written, and the copies in flight are waited for
    if (tid == 0) atomicOr(&a.ctrl->err, kErrTimeout);
    for (int c = max(0, issued - 2); c < issued; ++c) mbar_wait(&full[c & 1], (c >> 1) & 1);
    return;
  }
#pragma unroll
  for (int t = 0; t < NS * 8; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (vr + 8 * e < a.dv) *reinterpret_cast<float2*>(a.S_out + s_at + 8 * e * DK + t * 8) = S[t][e];
}

// The units of two slices come one an SM and round; where those of the last, partial round fill at most
// half of the SMs they are cut into units of one slice, which are done sooner.
__device__ __forceinline__ bool last_round_split(const GdnPrefillArgs& a, int unit, int units) {
  const int full = units / a.n_sm * a.n_sm;
  return unit >= full && 2 * (units - full) <= a.n_sm;
}
// NS = 0: one slice a warp and 64 rows a CTA, or two slices and 128 rows, as the plan says; the grid
// is the former's, so that every other CTA of the latter leaves.
template <int DK, int NS>
__global__ void __launch_bounds__(256) k_gdn_scan(const __grid_constant__ GdnPrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[2];
  uint8_t* smem = smem_raw + ((256u - (smem_u32(smem_raw) & 255u)) & 255u);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int blocks = (a.dv + kGdnSlab * a.slabs - 1) / (kGdnSlab * a.slabs), per = a.Hv * blocks;
  const int place = blockIdx.x / per, rest = blockIdx.x % per, h = rest / blocks, rb = rest - h * blocks;
  int s;
  GdnSeq seq;
  bool chain;
  if (a.warp_plan) {
    const int lane = threadIdx.x & 31;
    const GdnWarpPlan p = gdn_warp_plan(a, lane);
    if (blockIdx.x == 0 && threadIdx.x < 32 && p.bad) atomicOr(&a.ctrl->err, kErrBadRange);
    int longest = p.nc, rank = lane < a.n_seqs ? 0 : -1;  // longest first
    for (int i = 0; i < a.n_seqs; ++i) {
      const int nc = __shfl_sync(0xffffffffu, p.nc, i);
      longest = max(longest, nc);
      if (lane < a.n_seqs && (nc > p.nc || (nc == p.nc && i < lane))) ++rank;
    }
    s = __ffs(__ballot_sync(0xffffffffu, rank == place)) - 1;
    seq = GdnSeq{__shfl_sync(0xffffffffu, p.seq.row0, s), __shfl_sync(0xffffffffu, p.seq.n, s), __shfl_sync(0xffffffffu, p.seq.chunk0, s)};
    chain = gdn_chain(a, longest, p.n_chunks);
  } else {
    s = a.order[place];
    seq = a.seqs[s];
    chain = a.hdr->chain;
  }
  if (seq.n < 0) return;
  if constexpr (NS > 0) {
    gdn_scan<DK, NS>(a, a.slabs, seq, s, h, rb, smem, full);
  } else if (chain || last_round_split(a, (place * a.Hv + h) * ((blocks + 1) / 2) + rb / 2, a.n_seqs * a.Hv * ((blocks + 1) / 2))) {
    gdn_scan<DK, 1>(a, a.slabs, seq, s, h, rb, smem, full);
  } else if (rb % 2 == 0) {
    gdn_scan<DK, 2>(a, 2 * a.slabs, seq, s, h, rb / 2, smem, full);
  }
}

}  // namespace

// Slabs of a scan CTA: as many as shared memory holds (they share a chunk's K, Q, T' and P), but
// no more than leave every SM a CTA.  NS = 0: 64 rows, and 128 for the sequences of two slices.
template <int DK, int NS>
static cudaError_t launch_gdn_scan(GdnPrefillArgs& a, int n_sm, cudaStream_t s) {
  using M = GdnScanSmem<DK, NS ? NS : 1>;
  const long long heads = (long long)a.n_seqs * a.Hv;
  int bytes, threads;
  if constexpr (NS > 0) {
    const int most = DK == 256 ? NS : DK == 128 ? 4 : 8;
    a.slabs = 1;
    while (a.slabs < most && heads * ((a.dv + 2 * kGdnSlab * a.slabs - 1) / (2 * kGdnSlab * a.slabs)) * 2 > n_sm &&
           a.slabs * kGdnSlab < a.dv)
      a.slabs *= 2;
    bytes = M::bytes(a.slabs);
    threads = a.slabs * M::kWarps * 32;
  } else {
    a.slabs = 4;
    bytes = std::max(M::bytes(4), GdnScanSmem<DK, 2>::bytes(8));
    threads = 256;
  }
  const int rows = kGdnSlab * a.slabs;
  const cudaError_t e = cudaFuncSetAttribute(k_gdn_scan<DK, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_gdn_scan<DK, NS>, dim3((unsigned)(heads * ((a.dv + rows - 1) / rows))), dim3((unsigned)threads),
                    (size_t)bytes, s, a);
}

template <int DK>
static cudaError_t launch_gdn_prefill_dk(GdnPrefillArgs& a, int n_sm, cudaStream_t s) {
  const long long chunks = (long long)a.T / kGdnChunk + std::min(a.n_seqs, a.T);
  a.warp_plan = a.n_seqs <= kWarpSeqs && chunks * a.Hk <= 16LL * n_sm;
  cudaError_t e = cudaSuccess;
  if (!a.warp_plan) e = launch_pdl(k_gdn_plan, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  if (a.T > 0 && a.dv % 8 == 0) {
    const cuuint64_t dims[3] = {(cuuint64_t)a.dv, (cuuint64_t)a.Hv, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)a.dv * 2, (cuuint64_t)a.Hv * a.dv * 2};
    const cuuint32_t box[3] = {kGdnSlab, 1, kGdnChunk};
    e = encode_map(&a.map_v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B);
    if (e != cudaSuccess) return e;
  }
  if (chunks > 0) {
    // A grid of up to two CTAs an SM asks for as much shared memory as keeps a third from joining
    // them on some SMs while others idle (1,000 tokens, 272 CTAs: 69 against 65 us).
    const long long grid = chunks * a.Hk;
    const int bytes = grid <= 2 * n_sm ? std::max(GdnChunkSmem<DK>::kBytes, 80 * 1024) : GdnChunkSmem<DK>::kBytes;
    e = cudaFuncSetAttribute(k_gdn_chunk<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = launch_pdl(k_gdn_chunk<DK>, dim3((unsigned)grid), dim3(kChunkThreads), (size_t)bytes, s, a);
    if (e != cudaSuccess) return e;
  }
  if constexpr (DK > kGdnSlice) {
    const long long slabs = (long long)a.n_seqs * a.Hv * ((a.dv + kGdnSlab - 1) / kGdnSlab);
    if (slabs >= 4LL * n_sm) return launch_gdn_scan<DK, DK == 128 ? 0 : 2>(a, n_sm, s);
  }
  return launch_gdn_scan<DK, 1>(a, n_sm, s);
}

cudaError_t launch_gdn_prefill(GdnPrefillArgs& a, cudaStream_t s) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  a.n_sm = n_sm;
  switch (a.dk) {
    case 64: return launch_gdn_prefill_dk<64>(a, n_sm, s);
    case 128: return launch_gdn_prefill_dk<128>(a, n_sm, s);
    default: return launch_gdn_prefill_dk<256>(a, n_sm, s);
  }
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
  if (((long long)T / kGdnChunk + n_seqs) * Hk > 0x7fffffffLL) return set_error(MOE_ERR_INVALID, "T * n_k_heads too large");
  return MOE_OK;
}

struct GdnPrefillLayout {
  size_t ctrl, hdr, seqs, order, chunks, img, tp, total;
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
  // the chunks of disjoint sequences of T rows: full ones, and one ragged one per sequence
  const size_t chunks = (size_t)T / kGdnChunk + std::min(n_seqs, T);
  W.hdr = take(sizeof(GdnHdr));
  W.seqs = take(sizeof(GdnSeq) * (size_t)n_seqs);
  W.order = take(sizeof(int32_t) * (size_t)n_seqs);
  W.chunks = take(sizeof(GdnChunk) * chunks);
  W.img = take(chunks * shape->n_k_heads * 2 * kGdnChunk * shape->d_k * 2);
  W.tp = take(chunks * shape->n_v_heads * sizeof(GdnTP));
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
                   beta, static_cast<uint16_t*>(out), 1, 1, 0, reinterpret_cast<Ctrl*>(w + W.ctrl),
                   reinterpret_cast<GdnHdr*>(w + W.hdr), reinterpret_cast<GdnSeq*>(w + W.seqs),
                   reinterpret_cast<int32_t*>(w + W.order), reinterpret_cast<GdnChunk*>(w + W.chunks), w + W.img,
                   reinterpret_cast<GdnTP*>(w + W.tp), {}};
  const cudaError_t e = launch_gdn_prefill(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gated delta prompt launch");
  return MOE_OK;
}
