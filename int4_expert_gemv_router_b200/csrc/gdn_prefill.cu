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
//                first (they are the critical path)
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
// size; T' likewise by its rows.  S K^T and W K take two products (hi, lo), T' R three (lo lo is
// below 2^-22).  What only the bf16 output sees (Q S, P W) takes hi alone, 2^-12 of each weight.
// mma.sync carries this, not tcgen05: the slab's products are 16 rows high, 8 to 64 wide and
// dependent on each other, and a chunk's chain of six of them through TMEM (a round trip of
// registers, TMEM, MMA and back for each) costs more than the products themselves.
#include "../../include/moe.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels.cuh"
#include "seqs.cuh"
#include "sync.cuh"

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
  float wd[kGdnChunk];               // e^{G_64 - G_i} / |k_i|
  float ts[kGdnChunk], ps[kGdnChunk];  // scales of the rows of T' and P
  float keep[32];                    // [0]: e^{G_64}
};
static_assert(sizeof(GdnTP) % 128 == 0, "bulk copies and alignment");
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
  Ctrl* ctrl;
  GdnHdr* hdr;
  GdnSeq* seqs;          // [n_seqs]
  int32_t* order;        // [n_seqs] sequences, longest first
  GdnChunk* chunks;
  uint8_t* img;          // [chunk][Hk]: fp16 K then Q, 64 x dk each, rows' 16-byte pieces XORed with row & 7
  GdnTP* tp;             // [chunk][Hv]
};

namespace {

__global__ void __launch_bounds__(kPlanThreads) k_gdn_plan(const GdnPrefillArgs a) {
  __shared__ int sh[32];
  __shared__ int bins[kPlanThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  bins[tid] = 0;
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
    if (!ok) atomicOr(&a.ctrl->err, kErrBadRange);
  }
  if (tid == 0) a.hdr->n_chunks = chunks;
  __syncthreads();
  for (int s = warp; s < a.n_seqs; s += kPlanThreads / 32) {
    const GdnSeq q = a.seqs[s];
    for (int c = lane; c * kGdnChunk < q.n; c += 32)
      a.chunks[q.chunk0 + c] = GdnChunk{q.row0 + c * kGdnChunk, min(kGdnChunk, q.n - c * kGdnChunk)};
  }
  // sequences by length, longest first, in kPlanThreads classes
  const int per = a.T / (kPlanThreads - 1) + 1;
  for (int pass = 0; pass < 2; ++pass) {
    for (int s = tid; s < a.n_seqs; s += kPlanThreads) {
      const int bin = kPlanThreads - 1 - max(0, a.seqs[s].n) / per;
      const int at = atomicAdd(&bins[bin], 1);
      if (pass) a.order[at] = s;
    }
    __syncthreads();
    if (!pass) {
      int total = 0;
      const int first = block_excl_sum(bins[tid], total, sh);
      bins[tid] = first;
      __syncthreads();
    }
  }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d (16 x 8, fp32) += a (16 x 16, fp16) b (16 x 8, fp16).  With g = lane / 4, u = 2 (lane % 4):
// d0,d1 = (g, u..u+1), d2,d3 = (g + 8, u..); a0 = (g, u..), a1 = (g + 8, u..), a2 = (g, u + 8..),
// a3 = (g + 8, u + 8..); b0 = (k u.., n g), b1 = (k u + 8.., n g).
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// The power of two that brings a row whose largest element is m to [2^14, 2^15) (exact; rows of
// zeros and of values below 2^-112 by 2^126), and its inverse.
__device__ __forceinline__ void row_scale(float m, float& up, float& down) {
  const int e = max((int)(__float_as_uint(m) >> 23) - 127 - 14, -126);
  up = __uint_as_float((uint32_t)(127 - e) << 23);
  down = __uint_as_float((uint32_t)(127 + e) << 23);
}

// Accumulators of N tiles of 8 columns (rows g and g + 8 of a slab) -> the largest element of
// each of the two rows over the warp's columns.
template <int N>
__device__ __forceinline__ void row_max(const float (&v)[N][4], float& m0, float& m1) {
  m0 = m1 = 0.f;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    m0 = fmaxf(m0, fmaxf(fabsf(v[t][0]), fabsf(v[t][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(v[t][2]), fabsf(v[t][3])));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
}
// hi + lo of the scaled rows, as A operands: registers (2t, 2t + 1) of the two tiles of a step of 16
template <int N>
__device__ __forceinline__ void split(const float (&v)[N][4], float up0, float up1, uint32_t (&hi)[N][2], uint32_t (&lo)[N][2]) {
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const float x0 = v[t][0] * up0, x1 = v[t][1] * up0, x2 = v[t][2] * up1, x3 = v[t][3] * up1;
    hi[t][0] = pack_h2(x0, x1);
    hi[t][1] = pack_h2(x2, x3);
    const float2 h0 = unpack_h2(hi[t][0]), h1 = unpack_h2(hi[t][1]);
    lo[t][0] = pack_h2(x0 - h0.x, x1 - h0.y);
    lo[t][1] = pack_h2(x2 - h1.x, x3 - h1.y);
  }
}

// ---------------------------------------------------------------------------------------
// k_gdn_chunk
// ---------------------------------------------------------------------------------------
constexpr int kChunkThreads = 256;  // four warps per value head, two value heads at a time
constexpr int kHeadThreads = 128;
constexpr int kMatLd = 68;          // row stride (floats) of the 64 x 64 matrices: 16-byte rows

template <int DK>
struct GdnChunkSmem {
  static constexpr int kImg = kGdnChunk * DK * 2;
  static constexpr int kMat = kGdnChunk * kMatLd * 4;
  static constexpr int kBytes = 2 * kImg + 4 * kMat;  // K, Q; K K^T, Q K^T; L (then T') of two heads
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(a - b) of sums held as two floats: the difference of the heads is exact or as good as its size
__device__ __forceinline__ float decay(float2 a, float2 b) { return ex2f((a.x - b.x) + (a.y - b.y)); }

__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kHeadThreads) : "memory");
}

// One step of the block inversion, for a block row of B rows below a block of B columns, both with
// their inverses in place: C <- -D (C A), A and D the inverses above and below the diagonal block
// C.  A thread has B / 4 columns of a row.
template <int B>
__device__ __forceinline__ void join_blocks(float* C, const float* A, const float* D, int t, int team) {
  constexpr int NC = B / 4;
  const int r = t / 4, c = (t % 4) * NC;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float* x = half ? D + r * kMatLd : C + r * kMatLd;
    const float* y = (half ? C : A) + c;
    float s[NC] = {};
#pragma unroll 8
    for (int k = 0; k < B; ++k) {
      const float f = x[k];
#pragma unroll
      for (int e = 0; e < NC; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(y + k * kMatLd + e);
        s[e] = fmaf(f, v.x, s[e]);
        s[e + 1] = fmaf(f, v.y, s[e + 1]);
        s[e + 2] = fmaf(f, v.z, s[e + 2]);
        s[e + 3] = fmaf(f, v.w, s[e + 3]);
      }
    }
    team_sync(team);  // every thread has read C
#pragma unroll
    for (int e = 0; e < NC; e += 4)
      *reinterpret_cast<float4*>(C + r * kMatLd + c + e) =
          half ? make_float4(-s[e], -s[e + 1], -s[e + 2], -s[e + 3]) : make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
    team_sync(team);
  }
}

// (I + L)^-1 in place of the strictly lower triangular L (zeros elsewhere), by a team of 128
// threads: the four 16 x 16 diagonal blocks by forward substitution, a thread a column, then
// joined to blocks of 32 and of 64.
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
    join_blocks<16>(D + 16 * kMatLd, D, D + 16 * (kMatLd + 1), t % 64, team);
  }
  join_blocks<32>(L + 32 * kMatLd, L, L + 32 * (kMatLd + 1), t, team);
}

template <int DK>
__global__ void __launch_bounds__(kChunkThreads) k_gdn_chunk(const GdnPrefillArgs a) {
  using M = GdnChunkSmem<DK>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_ck[kGdnChunk], s_cq[kGdnChunk], s_beta[2][kGdnChunk];
  __shared__ float2 s_G[2][kGdnChunk], s_low[2][kGdnChunk];  // log2(e) G_i and the least of them up to i, as two floats
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int chunk = blockIdx.x / a.Hk, kh = blockIdx.x - chunk * a.Hk;
  if (chunk >= a.hdr->n_chunks) return;
  const GdnChunk C = a.chunks[chunk];
  uint8_t* img[2] = {smem, smem + M::kImg};
  float* kk = reinterpret_cast<float*>(smem + 2 * M::kImg);
  float* qk = kk + kGdnChunk * kMatLd;
  float* Lh = qk + kGdnChunk * kMatLd;
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
      const int x = i * kChunkThreads + tid, r = x / LPR, col = x % LPR, z = r >> 6, row = r & 63;
      piece[i] = make_uint4(0, 0, 0, 0);
      if (row < C.n)
        piece[i] = *reinterpret_cast<const uint4*>((z ? a.q : a.k) + ((size_t)(C.row0 + row) * a.Hk + kh) * DK + col * 8);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = i * kChunkThreads + tid, r = x / LPR, col = x % LPR, z = r >> 6, row = r & 63;
      float v[8], ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = word_of(piece[i], e);
        v[2 * e] = bf_lo(w);
        v[2 * e + 1] = bf_hi(w);
        ss = fmaf(v[2 * e], v[2 * e], fmaf(v[2 * e + 1], v[2 * e + 1], ss));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float norm = sqrtf(ss);
      // 2^e2 brings the norm to [2^10, 2^11).  A row of a norm below 2^-100 (it vanishes next to
      // 1e-6), and one whose sum of squares overflows (1 / inf), is 0; infinities and NaN give NaN.
      const int ne = (int)(__float_as_uint(norm) >> 23) - 127;
      const bool zero = ne <= -100 || ne == 128;
      const float up = zero ? 0.f : __uint_as_float((uint32_t)(137 - ne) << 23);
      const float down = zero ? 0.f : __uint_as_float((uint32_t)(117 + ne) << 23);
      if (col == 0) {
        const float c = zero ? 0.f : down / fmaxf(norm, 1e-6f);  // the normalised row is c times the stored one
        if (z) s_cq[row] = c * rsqrtf((float)DK);
        else s_ck[row] = c;
      }
      const uint4 h = make_uint4(pack_h2(v[0] * up, v[1] * up), pack_h2(v[2] * up, v[3] * up), pack_h2(v[4] * up, v[5] * up),
                                 pack_h2(v[6] * up, v[7] * up));
      const int at = r * LPR + (col ^ (row & 7));
      reinterpret_cast<uint4*>(smem)[at] = h;
      dst[at] = h;
    }
  }
  // Decays: sums in 64 bits (their differences have to be good to 24; a forgotten state's g is
  // clamped, e^-1e4 = 0), kept as two floats, in units of log 2; one warp per head
  auto decays = [&](int h) {
    double x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * lane + e;
      const float gt = t < C.n ? a.g[(size_t)(C.row0 + t) * a.Hv + h] : 0.f;
      x[e] = (gt < -1e4f ? -1e4 : (double)gt) * 1.4426950408889634;
      s_beta[team][t] = t < C.n ? a.beta[(size_t)(C.row0 + t) * a.Hv + h] : 0.f;
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
    s_low[team][2 * lane] = two(lane ? fmin(before, g0) : g0);
    s_low[team][2 * lane + 1] = two(low);
  };
  if (tw == 0 && team < rep) decays(kh * rep + team);
  __syncthreads();
  // K K^T and Q K^T, lower triangle: rows in tiles of 16 (A), columns in pairs of tiles of 8 (B)
  for (int w = warp; w < 20; w += kChunkThreads / 32) {
    const int z = w / 10, u = w % 10;  // u: (row tile i, column pair j <= i)
    const int i = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, j = u - i * (i + 1) / 2;
    const uint32_t sa = smem_u32(img[z]), sb = smem_u32(img[0]);
    const int ra = i * 16 + (lane & 15), rb = j * 16 + (lane & 7) + ((lane >> 4) << 3);
    float d[2][4] = {};
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
      *reinterpret_cast<float2*>(dst + r * kMatLd + c) = make_float2(d[t][0], d[t][1]);
      *reinterpret_cast<float2*>(dst + (r + 8) * kMatLd + c) = make_float2(d[t][2], d[t][3]);
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
#pragma unroll 4
      for (int i = tw; i < kGdnChunk; i += 4) {
        const float2 Gi = s_G[team][i];
        const float f = s_beta[team][i] * s_ck[i];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int j = c * 32 + lane;
          L[i * kMatLd + j] = j < i ? f * decay(Gi, s_G[team][j]) * s_ck[j] * kk[i * kMatLd + j] : 0.f;
        }
      }
      team_sync(team);
      invert(L, tt, team);
      // P: block x of 20 is (token tile, step)
      for (int x = tw; x < GdnTP::kBlocks; x += 4) {
        const int half = x < 2 ? 0 : x < 6 ? 1 : x < 12 ? 2 : 3;
        const int rest = x - half * (half + 1), tile = 2 * half + rest / (half + 1), ks = rest % (half + 1);
        const int i = tile * 8 + (lane >> 2), c0 = ks * 16 + 2 * (lane & 3);
        const float2 low = s_low[team][i];
        const float cq = s_cq[i] * 1024.f;
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = c0 + (e & 1) + (e >> 1) * 8;
          pv[e] = c <= i ? decay(low, s_G[team][c]) * (cq * s_ck[c]) * qk[i * kMatLd + c] : 0.f;
        }
        tp->p[x][lane] = make_uint2(pack_h2(pv[0], pv[1]), pack_h2(pv[2], pv[3]));
      }
      if (tt < kGdnChunk) {  // factors of token tt
        const float2 G = s_G[team][tt], last = s_G[team][kGdnChunk - 1], zero = make_float2(0.f, 0.f);
        const float eg = decay(G, zero);
        // P is held relative to its row's least decayed entry and times 2^10 (fp16's range)
        tp->ps[tt] = decay(G, s_low[team][tt]) * 0x1p-10f;
        tp->xa[tt] = -eg * s_ck[tt];
        tp->oa[tt] = eg * s_cq[tt];
        tp->wd[tt] = decay(last, G) * s_ck[tt];
        if (tt < 32) tp->keep[tt] = decay(last, zero);
      }
    }
    if (on) {
      // T' by token tiles (a warp takes tiles tw and 7 - tw: five blocks), each row scaled to its
      // largest element
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int tile = y ? 7 - tw : tw, i = tile * 8 + (lane >> 2), c0 = 2 * (lane & 3);
        float v[4][4], m = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = k * 16 + c0 + (e & 1) + (e >> 1) * 8;
            v[k][e] = c <= i ? L[i * kMatLd + c] * s_beta[team][c] : 0.f;
            m = fmaxf(m, fabsf(v[k][e]));
          }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float up, down;
        row_scale(m, up, down);
        if ((lane & 3) == 0) tp->ts[i] = down;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k > tile / 2) continue;
          uint4 o;
          o.x = pack_h2(v[k][0] * up, v[k][1] * up);
          o.y = pack_h2(v[k][2] * up, v[k][3] * up);
          const float2 f0 = unpack_h2(o.x), f1 = unpack_h2(o.y);
          o.z = pack_h2(v[k][0] * up - f0.x, v[k][1] * up - f0.y);
          o.w = pack_h2(v[k][2] * up - f1.x, v[k][3] * up - f1.y);
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
template <int DK>
struct GdnScanSmem {
  static constexpr int kWarps = DK / kGdnSlice;             // warps of a slab
  static constexpr int kImg = kGdnChunk * DK * 2;
  static constexpr int kTp = 2 * kImg;                      // stage: K, Q, T' and P, V
  static constexpr int kV = kTp + (int)sizeof(GdnTP);
  static constexpr int kVSlab = kGdnChunk * kGdnSlab * 2;   // 32-byte rows, 16-byte pieces XORed with bit 2 of the row
  static constexpr int stage(int slabs) { return kV + slabs * kVSlab; }
  // exchange: per slab and warp, 8 tiles of S k and 8 of S q
  static constexpr int kXch = kWarps > 1 ? kWarps * 16 * 512 : 0;
  static constexpr int bytes(int slabs) { return 2 * stage(slabs) + slabs * kXch; }
};

__device__ __forceinline__ void slab_sync(int slab, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(slab + 1), "r"(threads) : "memory");
}

template <int DK>
__global__ void __launch_bounds__(256) k_gdn_scan(const GdnPrefillArgs a) {
  using M = GdnScanSmem<DK>;
  constexpr int NW = M::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slab = warp / NW, w = warp - slab * NW;
  const int g = lane >> 2, u = 2 * (lane & 3);
  const int stage_bytes = M::stage(a.slabs);
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) mbar_init(&full[s], 1 + blockDim.x);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  const int blocks = (a.dv + kGdnSlab * a.slabs - 1) / (kGdnSlab * a.slabs);
  const int per = a.Hv * blocks;
  const int s = a.order[blockIdx.x / per], rest = blockIdx.x % per, h = rest / blocks, rb = rest - h * blocks;
  const int kh = h / (a.Hv / a.Hk);
  const GdnSeq seq = a.seqs[s];
  if (seq.n < 0) return;
  const int n_ch = (seq.n + kGdnChunk - 1) / kGdnChunk;
  const int v0 = rb * a.slabs * kGdnSlab;       // first state row of the CTA
  const int vr = v0 + slab * kGdnSlab + g;      // this lane's rows: vr and vr + 8
  const size_t state = (size_t)s * a.Hv + h;
  float* So = a.S_out + state * a.dv * DK;

  float S[8][4];  // tiles of 8 columns of this warp's 64
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 x = make_float2(0.f, 0.f);
      if (a.S_in && vr + 8 * e < a.dv)
        x = *reinterpret_cast<const float2*>(a.S_in + (state * a.dv + vr + 8 * e) * DK + w * kGdnSlice + t * 8 + u);
      S[t][2 * e] = x.x;
      S[t][2 * e + 1] = x.y;
    }

  const bool v_wide = a.dv % 8 == 0;
  auto load = [&](int c) {  // chunk c into its stage; every thread arrives on the stage's barrier
    uint8_t* st = smem + (c & 1) * stage_bytes;
    const size_t ch = (size_t)seq.chunk0 + c;
    if (tid == 0) {
      mbar_expect_tx(&full[c & 1], M::kV);
      bulk_g2s(st, a.img + (ch * a.Hk + kh) * 2 * M::kImg, 2 * M::kImg, &full[c & 1]);
      bulk_g2s(st + M::kTp, a.tp + ch * a.Hv + h, sizeof(GdnTP), &full[c & 1]);
    }
    const int row0 = seq.row0 + c * kGdnChunk, n = min(kGdnChunk, seq.n - c * kGdnChunk);
    // V: per slab, token and half (8 values)
    for (int i = tid; i < a.slabs * kGdnChunk * 2; i += blockDim.x) {
      const int half = i % (2 * a.slabs), r = i / (2 * a.slabs), col = v0 + half * 8;
      uint8_t* dst = st + M::kV + (half >> 1) * M::kVSlab + r * 32 + (((half & 1) ^ ((r >> 2) & 1)) << 4);
      const uint16_t* src = a.v + ((size_t)(row0 + r) * a.Hv + h) * a.dv + col;
      if (v_wide && r < n && col < a.dv) {
        cp_async16(dst, src);
      } else {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t l0 = r < n && col + 2 * e < a.dv ? src[2 * e] : 0, l1 = r < n && col + 2 * e + 1 < a.dv ? src[2 * e + 1] : 0;
          x[e] = l0 | (l1 << 16);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
    cp_async_arrive(&full[c & 1]);
  };

  bool ok = true;
  int issued = 0;
  if (n_ch > 0) load(issued++);
  for (int c = 0; c < n_ch; ++c) {
    // everyone is done with the other stage and with the exchange area (and the plain stores of
    // this chunk's V are visible)
    ok = __syncthreads_and(ok);
    if (!ok) break;
    if (c + 1 < n_ch) load(issued++);
    ok = mbar_wait(&full[c & 1], (c >> 1) & 1);
    const uint32_t st = smem_u32(smem) + (c & 1) * stage_bytes;
    const uint32_t sK = st, sQ = st + M::kImg;
    const GdnTP* tp = reinterpret_cast<const GdnTP*>(smem + (c & 1) * stage_bytes + M::kTp);

    // ---- X^T = S K^T (hi, lo) and Y^T = S Q^T (hi), over this warp's columns ----
    float X[8][4], Y[8][4];
    {
      float m0, m1, up0, up1, dn0, dn1;
      row_max(S, m0, m1);
      row_scale(m0, up0, dn0);
      row_scale(m1, up1, dn1);
      uint32_t hi[8][2], lo[8][2];
      split(S, up0, up1, hi, lo);
#pragma unroll
      for (int tg = 0; tg < 8; tg += 4) {
        uint32_t B[4][8];
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // K, then Q
          float (&D)[8][4] = z ? Y : X;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int row = (tg + t) * 8 + (lane & 7);
            const uint32_t base = (z ? sQ : sK) + row * DK * 2;
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              uint32_t r[4];
              ldsm4(base + (((w * 8 + k2 * 4 + (lane >> 3)) ^ (row & 7)) << 4), r);
#pragma unroll
              for (int e = 0; e < 4; ++e) B[t][k2 * 4 + e] = r[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) D[tg + t][e] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              mma16(D[tg + t], hi[2 * k][0], hi[2 * k][1], hi[2 * k + 1][0], hi[2 * k + 1][1], B[t][2 * k], B[t][2 * k + 1]);
            if (!z) {
#pragma unroll
              for (int t = 0; t < 4; ++t)
                mma16(D[tg + t], lo[2 * k][0], lo[2 * k][1], lo[2 * k + 1][0], lo[2 * k + 1][1], B[t][2 * k], B[t][2 * k + 1]);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        X[t][0] *= dn0;
        X[t][1] *= dn0;
        X[t][2] *= dn1;
        X[t][3] *= dn1;
        Y[t][0] *= dn0;
        Y[t][1] *= dn0;
        Y[t][2] *= dn1;
        Y[t][3] *= dn1;
      }
    }
    // ---- sums over the slab's warps (each the same, in the same order); of Y only the tiles
    // t % NW == w that this warp finishes ----
    if constexpr (NW > 1) {
      float4* xch = reinterpret_cast<float4*>(smem + 2 * stage_bytes + slab * M::kXch);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        xch[(w * 16 + t) * 32 + lane] = make_float4(X[t][0], X[t][1], X[t][2], X[t][3]);
        if (t % NW != w) xch[(w * 16 + 8 + t) * 32 + lane] = make_float4(Y[t][0], Y[t][1], Y[t][2], Y[t][3]);
      }
      slab_sync(slab, NW * 32);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float4 sx = make_float4(0.f, 0.f, 0.f, 0.f), sy = sx;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
          const float4 x = v == w ? make_float4(X[t][0], X[t][1], X[t][2], X[t][3]) : xch[(v * 16 + t) * 32 + lane];
          sx = make_float4(sx.x + x.x, sx.y + x.y, sx.z + x.z, sx.w + x.w);
          if (t % NW == w) {
            const float4 y = v == w ? make_float4(Y[t][0], Y[t][1], Y[t][2], Y[t][3]) : xch[(v * 16 + 8 + t) * 32 + lane];
            sy = make_float4(sy.x + y.x, sy.y + y.y, sy.z + y.z, sy.w + y.w);
          }
        }
        X[t][0] = sx.x;
        X[t][1] = sx.y;
        X[t][2] = sx.z;
        X[t][3] = sx.w;
        if (t % NW == w) {
          Y[t][0] = sy.x;
          Y[t][1] = sy.y;
          Y[t][2] = sy.z;
          Y[t][3] = sy.w;
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
      for (int e = 0; e < 2; ++e) {
        const float2 xa = *reinterpret_cast<const float2*>(&tp->xa[(t + e) * 8 + u]);
        X[t + e][0] = fmaf(xa.x, X[t + e][0], bf_lo(r[2 * e]));
        X[t + e][1] = fmaf(xa.y, X[t + e][1], bf_hi(r[2 * e]));
        X[t + e][2] = fmaf(xa.x, X[t + e][2], bf_lo(r[2 * e + 1]));
        X[t + e][3] = fmaf(xa.y, X[t + e][3], bf_hi(r[2 * e + 1]));
      }
    }
    // ---- W^T = R^T T'^T ----
    float W[8][4];
    {
      float m0, m1, up0, up1, dn0, dn1;
      row_max(X, m0, m1);
      row_scale(m0, up0, dn0);
      row_scale(m1, up1, dn1);
      uint32_t hi[8][2], lo[8][2];
      split(X, up0, up1, hi, lo);
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) W[t][e] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 b[8];
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) b[t] = tp->t[gdn_block(t, k)][lane];
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) mma16(W[t], hi[2 * k][0], hi[2 * k][1], hi[2 * k + 1][0], hi[2 * k + 1][1], b[t].x, b[t].y);
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) mma16(W[t], hi[2 * k][0], hi[2 * k][1], hi[2 * k + 1][0], hi[2 * k + 1][1], b[t].z, b[t].w);
#pragma unroll
        for (int t = 2 * k; t < 8; ++t) mma16(W[t], lo[2 * k][0], lo[2 * k][1], lo[2 * k + 1][0], lo[2 * k + 1][1], b[t].x, b[t].y);
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float2 ts = *reinterpret_cast<const float2*>(&tp->ts[t * 8 + u]);
        W[t][0] *= dn0 * ts.x;
        W[t][1] *= dn0 * ts.y;
        W[t][2] *= dn1 * ts.x;
        W[t][3] *= dn1 * ts.y;
      }
    }
    // ---- O^T = e^G S q + W^T P^T, for this warp's token tiles ----
    {
      float m0, m1, up0, up1, dn0, dn1;
      row_max(W, m0, m1);
      row_scale(m0, up0, dn0);
      row_scale(m1, up1, dn1);
      uint32_t hi[8][2];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        hi[t][0] = pack_h2(W[t][0] * up0, W[t][1] * up0);
        hi[t][1] = pack_h2(W[t][2] * up1, W[t][3] * up1);
      }
      const int row0 = seq.row0 + c * kGdnChunk, n = min(kGdnChunk, seq.n - c * kGdnChunk);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (t % NW != w) continue;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k <= t / 2; ++k) {
          const uint2 b = tp->p[gdn_block(t, k)][lane];
          mma16(o, hi[2 * k][0], hi[2 * k][1], hi[2 * k + 1][0], hi[2 * k + 1][1], b.x, b.y);
        }
        const float2 ps = *reinterpret_cast<const float2*>(&tp->ps[t * 8 + u]);
        const float2 oa = *reinterpret_cast<const float2*>(&tp->oa[t * 8 + u]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = fmaf(e & 1 ? oa.y : oa.x, Y[t][e], o[e] * ((e < 2 ? dn0 : dn1) * (e & 1 ? ps.y : ps.x)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = t * 8 + u + (e & 1), col = vr + 8 * (e >> 1);
          if (tok < n && col < a.dv) a.out[((size_t)(row0 + tok) * a.Hv + h) * a.dv + col] = f2bf(o[e]);
        }
      }
    }
    // ---- S' = e^{G_64} S + (e^{G_64 - G} W)^T K ----
    {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float2 wd = *reinterpret_cast<const float2*>(&tp->wd[t * 8 + u]);
        W[t][0] *= wd.x;
        W[t][1] *= wd.y;
        W[t][2] *= wd.x;
        W[t][3] *= wd.y;
      }
      float m0, m1, up0, up1, dn0, dn1;
      row_max(W, m0, m1);
      row_scale(m0, up0, dn0);
      row_scale(m1, up1, dn1);
      uint32_t hi[8][2], lo[8][2];
      split(W, up0, up1, hi, lo);
      float D[8][4];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) D[t][e] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t B[4][4];
        const int row = k * 16 + (lane & 15);
#pragma unroll
        for (int t2 = 0; t2 < 4; ++t2)
          ldsm4_t(sK + row * DK * 2 + (((w * 8 + 2 * t2 + (lane >> 4)) ^ (row & 7)) << 4), B[t2]);
#pragma unroll
        for (int t = 0; t < 8; ++t)
          mma16(D[t], hi[2 * k][0], hi[2 * k][1], hi[2 * k + 1][0], hi[2 * k + 1][1], B[t >> 1][2 * (t & 1)], B[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 0; t < 8; ++t)
          mma16(D[t], lo[2 * k][0], lo[2 * k][1], lo[2 * k + 1][0], lo[2 * k + 1][1], B[t >> 1][2 * (t & 1)], B[t >> 1][2 * (t & 1) + 1]);
      }
      const float keep = tp->keep[0];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        S[t][0] = fmaf(keep, S[t][0], D[t][0] * dn0);
        S[t][1] = fmaf(keep, S[t][1], D[t][1] * dn0);
        S[t][2] = fmaf(keep, S[t][2], D[t][2] * dn1);
        S[t][3] = fmaf(keep, S[t][3], D[t][3] * dn1);
      }
    }
  }
  ok = __syncthreads_and(ok);
  if (!ok) {  // a copy never landed: no state is written, and the copies in flight are waited for
    if (tid == 0) atomicOr(&a.ctrl->err, kErrTimeout);
    for (int c = max(0, issued - 2); c < issued; ++c) mbar_wait(&full[c & 1], (c >> 1) & 1);
    return;
  }
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (vr + 8 * e < a.dv)
        *reinterpret_cast<float2*>(So + (size_t)(vr + 8 * e) * DK + w * kGdnSlice + t * 8 + u) =
            make_float2(S[t][2 * e], S[t][2 * e + 1]);
}

}  // namespace

// Slabs of a scan CTA: as many as shared memory holds (they share a chunk's K, Q, T' and P), but
// no more than leave every SM a CTA.
template <int DK>
static int gdn_slabs(const GdnPrefillArgs& a, int n_sm) {
  const int most = DK == 64 ? 8 : DK == 128 ? 4 : 1;
  int slabs = 1;
  const long long heads = (long long)a.n_seqs * a.Hv;
  while (slabs < most && heads * ((a.dv + 2 * kGdnSlab * slabs - 1) / (2 * kGdnSlab * slabs)) * 2 > n_sm &&
         slabs * kGdnSlab < a.dv)
    slabs *= 2;
  return slabs;
}

template <int DK>
static cudaError_t launch_gdn_prefill_dk(GdnPrefillArgs& a, int n_sm, cudaStream_t s) {
  using M = GdnScanSmem<DK>;
  cudaError_t e = launch_pdl(k_gdn_plan, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const long long chunks = (long long)a.T / kGdnChunk + std::min(a.n_seqs, a.T);
  if (chunks > 0) {
    e = cudaFuncSetAttribute(k_gdn_chunk<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, GdnChunkSmem<DK>::kBytes);
    if (e == cudaSuccess)
      e = launch_pdl(k_gdn_chunk<DK>, dim3((unsigned)(chunks * a.Hk)), dim3(kChunkThreads), GdnChunkSmem<DK>::kBytes, s, a);
    if (e != cudaSuccess) return e;
  }
  a.slabs = gdn_slabs<DK>(a, n_sm);
  const int rows = kGdnSlab * a.slabs;
  e = cudaFuncSetAttribute(k_gdn_scan<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::bytes(a.slabs));
  if (e != cudaSuccess) return e;
  return launch_pdl(k_gdn_scan<DK>, dim3((unsigned)((long long)a.n_seqs * a.Hv * ((a.dv + rows - 1) / rows))),
                    dim3(a.slabs * M::kWarps * 32), M::bytes(a.slabs), s, a);
}

cudaError_t launch_gdn_prefill(GdnPrefillArgs& a, cudaStream_t s) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
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
                   beta, static_cast<uint16_t*>(out), 1, reinterpret_cast<Ctrl*>(w + W.ctrl),
                   reinterpret_cast<GdnHdr*>(w + W.hdr), reinterpret_cast<GdnSeq*>(w + W.seqs),
                   reinterpret_cast<int32_t*>(w + W.order), reinterpret_cast<GdnChunk*>(w + W.chunks), w + W.img,
                   reinterpret_cast<GdnTP*>(w + W.tp)};
  const cudaError_t e = launch_gdn_prefill(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gated delta prompt launch");
  return MOE_OK;
}
