// Causal softmax attention with grouped heads over packed sequences (moe_attn_forward), sm_100a.
//
//     out_i = sum_j p_ij v_j,  p_ij = 2^{x_ij - m_i} / sum_j 2^{x_ij - m_i},  x_ij = scale log2(e) q_i.k_j
//
// over the keys j <= len - n + i of the query's sequence, in one pass over the keys with the
// running maximum m_i and sum.
//
// A work unit is one key head and a block of up to 2 * PT query positions, PT = 128 / G with G
// the query heads of a key head: the rows of a tile are (position, head of the group) pairs, so
// a tile of 128 rows holds every query that shares the key head's keys at PT positions.  (One
// head and 128 positions a tile would fill only G-th part of the rows for single tokens, and
// mask more of the diagonal.)  The block's two tiles A and B share every key and value tile of
// 128 rows:
//
//   k_attn_plan     one CTA: checks the sequences, cuts them into blocks, long blocks into
//                   pieces of keys when the call has fewer blocks than would fill the GPU, and
//                   orders the units by their number of key tiles, longest first
//   k_attn<D>       persistent, one CTA per SM:
//     warps 0-3, 4-7  softmax of tile A, B: a thread owns a row.  S from TMEM, running maximum and
//                     sum, P as bf16 back into TMEM over S, O rescaled when a maximum rises by
//                     more than 2^8, the end of the unit (O / sum, or the piece's O, m, sum)
//     warps 8, 9      issue the MMAs of tile A, B: S = Q K^T (operands in shared memory), O += P V
//                     (P in TMEM).  One tile's softmax overlaps the other's products; a warp each,
//                     because an issuing warp's waits and commits (about 100 cycles each) are
//                     not hidden behind its own products
//     warp 10         Q, K and V tiles by TMA (128-byte swizzle), K and V through one ring
//     warp 11         value tiles with keys that some row does not see: infinities and NaN are taken out
//   k_attn_few<D>   takes the place of k_attn where a call has few rows per sequence (single
//                   tokens): units of 16 rows on mma.sync, see there
//   k_attn_join     joins the pieces of blocks that k_attn had cut
//
// What is rounded: P to bf16 (the tensor core's operand; one half step, 2^-8, of each weight; with
// few rows, where the tensor core has time, to two bf16 values, 2^-16), and the result.  S, O, m and
// the sums are fp32.  A maximum may lag the true one by up to 2^8: P keeps its relative precision and
// the fp32 sums their range.
#include "../../include/moe.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels.cuh"
#include "seqs.cuh"
#include "sync.cuh"
#include "tc.cuh"

#include <algorithm>
#include <cmath>

namespace moe {

struct AttnSeq {
  int row0, n;    // first query row and queries; n < 0: left out
  int kv0, len;   // first key row and keys
};

// A block of query positions of one sequence and a range of its key tiles (every key head is a
// unit of its own).
struct alignas(16) AttnUnit {
  int row, npos;  // first query row, positions
  int kv0, len;   // the sequence's keys
  int seen;       // keys that the block's first position sees (0 or less: none); the next sees one more
  int kt0, kt1;   // key tiles
  int slot;       // -1, or the piece's place among the partial results
  int slot0, pieces;  // the cut block's first piece and its pieces
};
struct alignas(16) AttnRec {  // a block cut into pieces
  int row, npos, seen, slot, pieces;
};
struct AttnHdr {
  int n_units, n_recs;
  int ticket;  // units given out beyond each CTA's first
};

constexpr int kAttnTile = 128;     // rows of a query tile and of a key tile
constexpr int kAttnFill = 222;     // pieces that keys are cut for (tile kernel; pieces after histories: 148 71.2 us, 222 66.8, 296 68.9)
constexpr int kAttnFillFew = 296;  // and for few rows
constexpr int kAttnMinPiece = 4;   // key tiles of a piece at least
constexpr int kAttnMaxSlots = 2 * kAttnFillFew;
constexpr int kPlanSeqs = 1024;
constexpr int kFewRows = 16;       // rows (positions x heads of a group) of a unit of the few-rows kernel

struct AttnArgs {
  int n_seqs, T, Hq, Hkv, G, d, max_kv, kv_rows, rows_slot;
  int PT, BP;        // positions of a query tile and of a unit
  int fill;          // pieces that keys are cut for; 0: nothing is cut
  int sort;          // units in order, longest first
  int few;           // the few-rows kernel's call
  int n_sm;
  int self_plan;     // no plan kernel: every CTA finds its one unit for itself
  float scale_log2;  // scale * log2(e)
  const int32_t *offsets, *kv_begin, *kv_len;
  const uint16_t* v;
  uint16_t* out;
  Ctrl* ctrl;
  AttnSeq* seqs;     // [n_seqs]
  AttnHdr* hdr;
  AttnUnit* units;
  AttnRec* recs;
  int* done;         // [2][slot * Hkv + head], few rows: pieces finished of a group, groups of a block
  float* part_o;     // [slot * Hkv + head], then k_attn: [d / 4][rows_slot][4], k_attn_few: [rows_slot][d]
  float2* part_ml;   // [slot * Hkv + head][rows_slot]: maximum (log2 units) and sum
  alignas(64) CUtensorMap map_q;
  alignas(64) CUtensorMap map_k;
  alignas(64) CUtensorMap map_v;
};

namespace {

// Key tiles that a block of np positions sees, the first of them `seen` keys.
__device__ __forceinline__ int tiles_of(int seen, int np) {
  const int last = seen + np - 1;
  return last > 0 ? (last + kAttnTile - 1) / kAttnTile : 0;
}

__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const __grid_constant__ AttnArgs a) {
  __shared__ int sh[32];
  __shared__ int bins[kPlanThreads];
  __shared__ AttnSeq s_seqs[kPlanSeqs];  // calls of more sequences go through global memory
  __shared__ unsigned long long s_work;
  __shared__ int s_slots, s_recs, s_blocks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, BP = a.BP;
  AttnSeq* seqs = a.n_seqs <= kPlanSeqs ? s_seqs : a.seqs;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) {
    s_work = 0;
    s_slots = s_recs = s_blocks = 0;
  }
  bins[tid] = 0;
  int seen_off = 0;
  for (int base = 0; base < a.n_seqs; base += kPlanThreads) {
    const int i = base + tid;
    const bool in = i < a.n_seqs;
    const int r0 = in ? a.offsets[i] : 0, r1 = in ? a.offsets[i + 1] : 0;
    const int kv0 = !in ? 0 : a.kv_begin ? a.kv_begin[i] : r0, len = !in ? 0 : a.kv_begin ? a.kv_len[i] : r1 - r0;
    const int before = block_excl_max(r0, seen_off, sh);
    if (!in) continue;
    const bool ok = rows_ok(r0, r1, before, a.T) && kv0 >= 0 && len >= 0 && len <= a.max_kv && kv0 <= a.kv_rows &&
                    len <= a.kv_rows - kv0;
    seqs[i] = AttnSeq{r0, ok ? r1 - r0 : -1, kv0, len};
    if (!ok) atomicOr(&a.ctrl->err, kErrBadRange);
  }
  __syncthreads();
  // Pieces of at most P tiles: with P >= the call's key tiles (over blocks and key heads) / fill the
  // pieces of cut blocks number at most 2 fill <= kAttnMaxSlots (a block of t > longest >= P tiles makes
  // ceil(t / P) < 2 t / P).
  int P = 1 << 24, longest = 1 << 24;  // a block of up to `longest` key tiles stays whole
  if (a.fill) {
    unsigned long long work = 0;
    int blocks = 0;
    for (int s = warp; s < a.n_seqs; s += kPlanThreads / 32) {
      const AttnSeq q = seqs[s];
      for (int b = lane; b * BP < q.n; b += 32) {
        work += tiles_of(q.len - q.n + b * BP + 1, min(BP, q.n - b * BP));
        ++blocks;
      }
    }
    // (per warp first: 64-bit shared atomics of 32 lanes take thousands of cycles)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      work += __shfl_xor_sync(0xffffffffu, work, o);
      blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
    }
    if (lane == 0 && blocks) {
      atomicAdd(&s_work, work);
      atomicAdd(&s_blocks, blocks);
    }
    __syncthreads();
    // Few blocks (U of them over the key heads): at most W / P + U <= n_sm pieces, one round of the SMs
    // (one token over 60,001 keys 37 -> 29 us, against 296).
    const float U = (float)s_blocks * (float)a.Hkv, work_all = (float)s_work * (float)a.Hkv;
    const bool round = 2.f * U <= a.n_sm;
    const auto tiles = [](float per) {  // rounded up, and never below the quotient
      return per < 1e7f ? max(kAttnMinPiece, (int)(per * 1.0001f + 0.9999f)) : 1 << 24;
    };
    P = tiles(work_all / (round ? a.n_sm - U : a.fill));
    // A block of no more key tiles than an SM's share is not in the way of the others: cut all the same,
    // its partial results only cost (ragged prompts 101.6 us, whole 90.2).
    longest = round || a.few ? P : tiles(work_all / min(a.n_sm, a.fill));
  }
  // Place the units; longest first (a counting sort, two rounds) where a CTA has several.
  const float to_bin = (float)(kPlanThreads - 1) / (float)(a.fill ? longest : max(1, (a.max_kv + kAttnTile - 1) / kAttnTile));
  for (int pass = a.sort ? 0 : 1; pass < 2; ++pass) {
    for (int s = warp; s < a.n_seqs; s += kPlanThreads / 32) {
      const AttnSeq q = seqs[s];
      for (int b0 = 0; b0 * BP < q.n; b0 += 32) {
        const int b = b0 + lane;
        const bool in = b * BP < q.n;
        const int np = min(BP, q.n - b * BP), seen = q.len - q.n + b * BP + 1, t = in ? tiles_of(seen, np) : 0;
        int len = t, pieces = in ? 1 : 0;
        if (t > longest) {  // equal pieces
          pieces = (t + P - 1) / P;
          len = (t + pieces - 1) / pieces;
          pieces = (t + len - 1) / len;
        }
        const int bin = a.sort ? kPlanThreads - 1 - min(kPlanThreads - 1, (int)(len * to_bin)) : 0;
        const int at = in ? atomicAdd(&bins[bin], pieces) : 0;
        if (pass == 0) continue;
        if (pieces == 1) a.units[at] = AttnUnit{q.row0 + b * BP, np, q.kv0, q.len, seen, 0, t, -1, 0, 1};
        // the pieces of a cut block by the whole warp
        for (unsigned cut = __ballot_sync(0xffffffffu, pieces > 1); cut; cut &= cut - 1) {
          const int src = __ffs(cut) - 1;
          int slot = 0;
          if (lane == src) {
            slot = atomicAdd(&s_slots, pieces);
            if (!a.few) a.recs[atomicAdd(&s_recs, 1)] = AttnRec{q.row0 + b * BP, np, seen, slot, pieces};
          }
          slot = __shfl_sync(0xffffffffu, slot, src);
          const int n = __shfl_sync(0xffffffffu, pieces, src), sz = __shfl_sync(0xffffffffu, len, src);
          const int to = __shfl_sync(0xffffffffu, at, src), tt = __shfl_sync(0xffffffffu, t, src);
          const int bnp = __shfl_sync(0xffffffffu, np, src), bseen = __shfl_sync(0xffffffffu, seen, src);
          for (int i = lane; i < n; i += 32)
            a.units[to + i] = AttnUnit{q.row0 + (b0 + src) * BP, bnp, q.kv0, q.len, bseen, i * sz, min(tt, (i + 1) * sz), slot + i, slot, n};
          if (a.few)
            for (int i = lane; i < n * a.Hkv; i += 32)
              a.done[slot * a.Hkv + i] = a.done[(kAttnMaxSlots + slot) * a.Hkv + i] = 0;
        }
      }
    }
    __syncthreads();
    if (pass == 0) {
      int total = 0;
      const int first = block_excl_sum(bins[tid], total, sh);
      bins[tid] = first;
      __syncthreads();
    }
  }
  // every bin ends where the next begins: the last one's end is the number of units
  if (tid == 0) {
    a.hdr->n_units = bins[a.sort ? kPlanThreads - 1 : 0] * a.Hkv;
    a.hdr->n_recs = s_recs;
    a.hdr->ticket = 0;
  }
}

// Calls of up to 32 sequences whose keys are not cut and whose units (a bound of them) are no more than
// the SMs need no plan kernel: each CTA finds its one unit for itself (37 tokens: 13.7 -> 11.7 us).  (Cut
// keys need the joins' counters cleared beforehand; one warp in the place of the plan's CTA there was no
// faster: one token over 60,001 keys 25.0 -> 25.3, 32 tokens 38.9 -> 39.3.)
constexpr int kWarpSeqs = 32;
struct AttnWarpPlan {
  AttnSeq seq;        // this lane's sequence (n < 0: left out, or none)
  bool bad;
  int blocks, first;  // its blocks, and those of the sequences before
};
__device__ __forceinline__ AttnWarpPlan attn_warp_plan(const AttnArgs& a, int lane) {
  const bool in = lane < a.n_seqs;
  const int r0 = in ? a.offsets[lane] : 0, r1 = in ? a.offsets[lane + 1] : 0;
  const int kv0 = !in ? 0 : a.kv_begin ? a.kv_begin[lane] : r0, len = !in ? 0 : a.kv_begin ? a.kv_len[lane] : r1 - r0;
  const int seen = warp_excl_max(r0, lane);
  const bool ok = in && rows_ok(r0, r1, seen, a.T) && kv0 >= 0 && len >= 0 && len <= a.max_kv && kv0 <= a.kv_rows &&
                  len <= a.kv_rows - kv0;
  AttnWarpPlan p;
  p.seq = AttnSeq{r0, ok ? r1 - r0 : -1, kv0, len};
  p.bad = in && !ok;
  p.blocks = ok ? (r1 - r0 + a.BP - 1) / a.BP : 0;
  p.first = warp_incl_sum(p.blocks, lane) - p.blocks;
  return p;
}
// Without a plan kernel: block e of a call whose blocks are not cut, found by a warp (a CTA takes one
// unit).  Returns the call's blocks.
__device__ __forceinline__ int attn_self_plan(const AttnArgs& a, int e, int lane, AttnUnit& u) {
  const AttnWarpPlan p = attn_warp_plan(a, lane);
  if (blockIdx.x == 0 && p.bad) atomicOr(&a.ctrl->err, kErrBadRange);
  const unsigned has = __ballot_sync(0xffffffffu, e >= p.first && e < p.first + p.blocks);
  const int src = has ? __ffs(has) - 1 : 0;
  const auto from = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
  const AttnSeq q{from(p.seq.row0), from(p.seq.n), from(p.seq.kv0), from(p.seq.len)};
  const int b = e - from(p.first), np = min(a.BP, q.n - b * a.BP), seen = q.len - q.n + b * a.BP + 1;
  u = AttnUnit{q.row0 + b * a.BP, np, q.kv0, q.len, seen, 0, tiles_of(seen, np), -1, 0, 1};
  return __shfl_sync(0xffffffffu, p.first + p.blocks, 31);
}

// ---------------------------------------------------------------------------------------
// Many rows: two query tiles of 128 rows against shared key tiles, on tcgen05
// ---------------------------------------------------------------------------------------
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 10, kCleanWarp = 11;
constexpr int kAttnThreads = 12 * 32;  // three warpgroups
// Registers: launched with 168 a thread (384 x 168 = 64,512), redistributed to 216 for the two
// softmax warpgroups (a row's 128 scores stay in registers) and 72 for the third:
// 256 x 216 + 128 x 72 = 64,512.
constexpr int kSoftRegs = 216, kRestRegs = 72;
constexpr int kHalf = 64;             // keys of an S buffer: two per tile, so that one fills while the other is read
constexpr float kRescale = 8.0f;  // log2 of how far a maximum may rise before O is rescaled

template <int D>
struct AttnSmem {
  static constexpr int kTile = kAttnTile * D * 2;          // bytes of a Q, K or V tile
  static constexpr int kBox = kAttnTile * 64 * 2;          // 64 columns of it: one TMA box, 128-byte rows
  static constexpr int kStages = D == 128 ? 5 : 8;         // K and V tiles in the ring
  static constexpr int kBytes = (2 + kStages) * kTile + 1024;
};

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

#define MOE_R32(r) \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), \
      "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), \
      "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), \
      "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
#define MOE_RW32(r) \
  "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), \
      "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), \
      "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), \
      "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
#define MOE_IN32(r) \
  "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), \
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), \
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), \
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])

// 32 columns of this warp's 32 TMEM lanes (thread = lane).  The registers hold the values only
// after tmem_ld_done on them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : MOE_R32(r)
      : "r"(taddr)
      : "memory");
}
// Waits for every load of this thread; the register operands keep uses of r behind it.
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : MOE_RW32(r)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      MOE_IN32(r)
      : "memory");
}
__device__ __forceinline__ void tmem_st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The MMAs, issued by the lane whose `lead` is set.  The whole warp runs the issuing code with the
// same values, so that descriptors live in uniform registers: issued from a one-lane branch, each
// MMA waits for its operands to be moved there (120 instead of 64 cycles an MMA).  A descriptor's
// high half is a constant; a k-step moves the low one.
// D (TMEM) += A (shared memory) * B (shared memory)
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                        bool acc, bool lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 q, %7, 0;\n"
      " mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((int)acc), "r"((int)lead)
      : "memory");
}
// D (TMEM) += A (TMEM, bf16 pairs: 8 columns per 16 of K) * B (shared memory)
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool acc,
                                        bool lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 db, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((int)acc), "r"((int)lead)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint64_t* bar, bool lead) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"((int)lead)
      : "memory");
}
// V as the B operand: N (the head's columns) runs along the 128-byte rows, K along the rows.
// 128-byte swizzle; the next 64 columns are one box further (LBO), the next 8 rows 1024 bytes
// (SBO); a k-step of 16 rows advances the start by 2048 bytes.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t saddr, uint32_t box) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((box >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((1024u >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// kind::f16, D fp32, A and B bf16, M = 128; b_mn: B is N-major
__device__ __forceinline__ uint32_t attn_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Unit number of this CTA's it-th round, where units are dealt out beforehand (few rows: a ticket costs
// more than it evens out): rounds alternate direction, so that the CTA with the longest unit of one
// round gets the shortest of the next.
__device__ __forceinline__ int unit_index(int it) {
  return it * (int)gridDim.x + ((it & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
}

// Many rows: units are given out one by one, longest first: a CTA's first is its own number, later ones come from
// the ticket counter.  (Dealt out in rounds beforehand, the longest CTA of the ragged prompts had 30
// key tiles, the mean 25.)  The loading warp draws them and hands them to the CTA's other warps.
struct UnitQueue {
  uint64_t full[2], empty[2];
  int unit[2];  // -1: no more
};
__device__ __forceinline__ void queue_init(UnitQueue& q, int readers) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&q.full[i], 1);
    mbar_init(&q.empty[i], readers);
  }
}
// The next unit, by the loading warp (it: units so far); -1 at the end.  False: a wait ran out.
__device__ __forceinline__ bool queue_draw(UnitQueue& q, const AttnArgs& a, int it, int n_units, int lane, int& unit) {
  if (!__all_sync(0xffffffffu, mbar_wait(&q.empty[it & 1], ((it >> 1) & 1) ^ 1) ? 1 : 0)) {
    if (lane == 0) atomicOr(&a.ctrl->err, kErrTimeout);
    return false;
  }
  int u = 0;
  if (lane == 0) {
    u = !it ? (int)blockIdx.x : a.self_plan ? n_units : (int)gridDim.x + atomicAdd(&a.hdr->ticket, 1);
    if (u >= n_units) u = -1;
    q.unit[it & 1] = u;
    mbar_arrive(&q.full[it & 1]);
  }
  unit = __shfl_sync(0xffffffffu, u, 0);
  return true;
}
// ... and by the others, a warp each.
__device__ __forceinline__ bool queue_take(UnitQueue& q, const AttnArgs& a, int it, int lane, int& unit) {
  if (!__all_sync(0xffffffffu, mbar_wait(&q.full[it & 1], (it >> 1) & 1) ? 1 : 0)) {
    if (lane == 0) atomicOr(&a.ctrl->err, kErrTimeout);
    return false;
  }
  unit = *reinterpret_cast<volatile int*>(&q.unit[it & 1]);
  __syncwarp();
  if (lane == 0) mbar_arrive(&q.empty[it & 1]);
  return true;
}

// What every role derives from a unit: per tile (A: 0, B: 1) its positions and key tiles.
struct AttnWork {
  AttnUnit u;
  int np[2], nk[2], n;  // positions, key tiles of the piece; the larger of nk
};
__device__ __forceinline__ AttnWork attn_work(const AttnArgs& a, int idx, const AttnUnit& self, int& head) {
  AttnWork w;
  const int e = idx / a.Hkv;
  head = idx - e * a.Hkv;
  w.u = a.self_plan ? self : a.units[e];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    w.np[x] = max(0, min(a.PT, w.u.npos - x * a.PT));
    const int t = w.np[x] > 0 ? tiles_of(w.u.seen + x * a.PT, w.np[x]) : 0;
    w.nk[x] = max(0, min(w.u.kt1, t) - w.u.kt0);
  }
  w.n = max(w.nk[0], w.nk[1]);
  return w;
}

// Infinities and NaN in values.  A hidden key's weight is 0, and 0 times an infinity or NaN is NaN, so
// a key that only some of a unit's rows see must not meet the others with such a value: it is taken
// out of the tile in shared memory (0 in its place), and added to the rows that do see it afterwards.
// Rows behind the sequence's last key, which hold anything, are cleared.  Tiles whose keys every row
// sees need none of it.  (Looking through those tiles beside their softmax: ragged prompts 89.6 -> 91.9 us,
// pieces 77.1 -> 78.5, the 16,384-token prompt and single tokens unchanged.)
// Rows first .. n - 1 of a value tile in shared memory (64-column boxes of 128-byte rows): rows from `len`
// on cleared, non-finite elements of the others replaced by 0 where `scan`.  A whole warp; true in a
// lane that replaced one.
template <int D>
__device__ __forceinline__ bool clean_rows(uint32_t tile, int first, int n, int len, bool scan, int lane) {
  constexpr int kBox = kAttnTile * 128;
  bool found = false;
  for (int c = 0; c < D / 64; ++c) {
    const uint32_t box = tile + c * kBox;
    if (scan) {
#pragma unroll 4
      for (int o = first * 128 + lane * 16; o < min(len, n) * 128; o += 512) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(box + o) : "memory");
        uint32_t bad = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= bf16x2_nonfinite(w[e]);
        if (bad) {
          found = true;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] &= ~((bf16x2_nonfinite(w[e]) >> 15) * 0xffffu);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + o), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        }
      }
    }
    for (int o = max(first, len) * 128 + lane * 16; o < n * 128; o += 512)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(box + o), "r"(0) : "memory");
  }
  return found;
}
// What clean_rows replaced, added to N columns of one row that sees the keys k0 .. k1 - 1 (v: key k0's
// value at the first of them; a weight above 0 leaves an infinity or NaN as it is).
template <int N>
__device__ __forceinline__ void add_nonfinite(uint32_t (&o)[N], const uint16_t* v, size_t stride, int k0, int k1) {
  for (; k0 < k1; ++k0, v += stride) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(v + i), bad = bf16x2_nonfinite(w);
      if (bad & 0x8000u) o[i] = __float_as_uint(__uint_as_float(o[i]) + bf_lo(w));
      if (bad >> 31) o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) + bf_hi(w));
    }
  }
}
__device__ __forceinline__ const uint16_t* attn_value(const AttnArgs& a, int row, int head) {
  return a.v + ((size_t)row * a.Hkv + head) * a.d;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ bool soft_wait(uint64_t* bar, uint32_t parity, Ctrl* c, int lane) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity) ? 1 : 0);
  if (!ok && lane == 0) atomicOr(&c->err, kErrTimeout);
  return ok;
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1) k_attn(const __grid_constant__ AttnArgs a) {
  using L = AttnSmem<D>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[NS], kv_empty[NS], q_full[2], q_free, s_full[2][2], p_full[2][2],
      o_prev[2], o_done[2], o_free[2], v_raw[NS], drain[2];
  __shared__ UnitQueue queue;
  __shared__ AttnUnit s_unit;
  __shared__ int s_blocks;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_bad[4];  // unit it & 3: elements of its values were taken out (units go at most two ahead of a reader)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;  // 128-byte swizzle atoms: 1024-byte tiles
  const uint32_t ring = smem + 2 * L::kTile;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);  // both tiles are done with it
      mbar_init(&v_raw[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[x][h], 1);
        mbar_init(&p_full[x][h], 4);  // one arrival per softmax warp
      }
      mbar_init(&o_prev[x], 1);
      mbar_init(&drain[x], 1);
      mbar_init(&o_done[x], 1);
      mbar_init(&o_free[x], 4);
    }
    mbar_init(&q_free, 2);
    queue_init(queue, kSoftWarps + 3);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kLoadWarp && lane < (a.kv_rows > 0 ? 3 : 1))
    prefetch_map(lane == 0 ? &a.map_q : lane == 1 ? &a.map_k : &a.map_v);
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;  // columns: S of A 0.., S of B 128.., O of A 256.., O of B 384..
  pdl_wait();                    // the units are the plan kernel's, every input earlier work's
  pdl_launch_dependents();
  if (a.self_plan) {
    if (warp == 0) {
      AttnUnit u;
      const int blocks = attn_self_plan(a, (int)blockIdx.x / a.Hkv, lane, u);
      if (lane == 0) {
        s_unit = u;
        s_blocks = blocks;
      }
    }
    __syncthreads();
  }
  const int n_units = a.self_plan ? s_blocks * a.Hkv : a.hdr->n_units;

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------ softmax and results ------------------------------
    const int x = warp >> 2;                       // tile
    const int r = (warp & 3) * 32 + lane;          // row = TMEM lane
    const int pos = r / a.G, sub = r - pos * a.G;  // position and head of the group
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_s = tmem + x * 128 + lanes, t_o = tmem + 256 + x * 128 + lanes;
    const bool neg = a.scale_log2 < 0.f;  // then the largest x is the smallest product: work on -S
    const float sl = fabsf(a.scale_log2);
    int n_s = 0, n_u = 0;  // key tiles and units (with key tiles) so far
    bool alive = true;
    for (int it = 0; alive && !warp_aborted(&s_abort); ++it) {
      int head, unit;
      if (!queue_take(queue, a, it, lane, unit)) {
        alive = false;
        break;
      }
      if (unit < 0) break;
      const AttnWork w = attn_work(a, unit, s_unit, head);
      const int np = x ? w.np[1] : w.np[0], nk = x ? w.nk[1] : w.nk[0];
      if (np == 0) continue;
      const int seen_r = pos < np ? w.u.seen + x * a.PT + pos : 0;  // keys this row sees (a row in use or 0)
      const int seen_0 = w.u.seen + x * a.PT;                            // the tile's first position
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nk && alive; ++j, ++n_s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 64 keys each
          if (!soft_wait(&s_full[x][h], n_s & 1, a.ctrl, lane)) {
            alive = false;
            break;
          }
          tc_fence_after();
          uint32_t s[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld32_async(t_s + h * kHalf + c * 32, s[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld_done(s[c]);
          const int key0 = (w.u.kt0 + j) * kAttnTile + h * kHalf;
          if (neg) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c][i] ^= 0x80000000u;
          }
          if (key0 + kHalf > seen_0) {  // a key of the half is hidden from some row
            const int lim = seen_r - key0;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i >= lim) s[c][i] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t* v = &s[c >> 1][(c & 1) * 16];
            mx[c] = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
            for (int i = 2; i < 16; i += 2) mx[c] = fmax3(mx[c], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          }
          const float m_new = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmaxf(mx[3], m));
          if (j == 0 && h == 0) {
            m = m_new;
          } else {
            const bool up = (m_new - m) * sl > kRescale;
            if (__any_sync(0xffffffffu, up)) {
              // O holds the sums over the keys before: wait for the last of their products.  It was
              // issued before the next half's S, or before o_prev where there is none.
              const bool last = h == 1 && j + 1 == nk;
              if (!soft_wait(last ? &o_prev[x] : &s_full[x][h ^ 1], (last ? n_u : n_s + h) & 1, a.ctrl, lane)) {
                alive = false;
                break;
              }
              tc_fence_after();
              const float f = up ? ex2((m - m_new) * sl) : 1.f;
              if (up) m = m_new;
              l *= f;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32_async(t_o + c * 32, o);
                tmem_ld_done(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(t_o + c * 32, o);
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : -m * sl;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t* sv = &s[i >> 4][(i & 15) * 2];
            const float2 e = ffma2(make_float2(__uint_as_float(sv[0]), __uint_as_float(sv[1])), make_float2(sl, sl),
                                   make_float2(ms, ms));
            const float2 pv = make_float2(ex2(e.x), ex2(e.y));
            sum[i & 1] = add2(sum[i & 1], pv);
            p[i] = pack_bf16(pv.x, pv.y);
          }
          tmem_st32(t_s + h * kHalf, p);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_done();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x][h]);
        }
      }
      if (!alive) break;
      // the end of the unit: this row's O
      if (nk > 0) {
        if (!soft_wait(&o_done[x], n_u & 1, a.ctrl, lane)) {
          alive = false;
          break;
        }
        ++n_u;
        tc_fence_after();
      }
      const bool mine = pos < np;
      const size_t brow = (size_t)(x * a.PT + pos) * a.G + sub;  // row within the block
      const size_t prow = ((size_t)max(w.u.slot, 0) * a.Hkv + head) * a.rows_slot + brow;
      const float inv = seen_r > 0 ? 1.0f / l : 0.f;
      const bool bad = nk > 0 && *reinterpret_cast<volatile int*>(&s_bad[it & 3]);
      uint16_t* const obase = a.out + ((size_t)(w.u.row + x * a.PT) * a.Hq + (size_t)head * a.G) * D;
      const int orow = mine ? pos * a.Hq + sub : -1;  // row of D columns from obase on
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (nk > 0) {
          tmem_ld32_async(t_o + c * 32, o);
          tmem_ld_done(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (bad) {
          const int k0 = max(w.u.kt0, max(w.u.seen, 0) / kAttnTile) * kAttnTile;
          add_nonfinite(o, attn_value(a, w.u.kv0 + k0, head) + c * 32, (size_t)a.Hkv * D, k0, min(seen_r, w.u.kt1 * kAttnTile));
        }
        if (mine && w.u.slot >= 0) {
          // a row's four columns next to the next row's: whole lines a store
          float4* dst = reinterpret_cast<float4*>(a.part_o) +
                        (((size_t)w.u.slot * a.Hkv + head) * (D / 4) + c * 8) * a.rows_slot + brow;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(size_t)i * a.rows_slot] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                 __uint_as_float(o[4 * i + 3]));
        }
        if (w.u.slot < 0) {
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[i][e] = seen_r > 0 ? pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv)
                                   : 0u;
          if constexpr (D == 128) {
            // a row's 64 bytes by four lanes: piece i of this lane's row <-> piece lane % 4 of row i of the
            // four (a store of 32 rows' 16 bytes takes the LSU 32 turns; ragged prompts 90 -> 87.4 us, 16,384
            // tokens 1,091 -> 1,075.  Two chunks a row do not repay it: pieces with d = 64 66.4 -> 68.3)
#pragma unroll
            for (int b = 1; b < 4; b <<= 1)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i & b) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & b ? v[i][e] : v[i | b][e], b);
                  if (lane & b) v[i][e] = got;
                  else v[i | b][e] = got;
                }
              }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = D == 128 ? __shfl_sync(0xffffffffu, orow, (lane & 28) + i) : orow;
            if (at >= 0)
              *reinterpret_cast<uint4*>(obase + (size_t)at * D + c * 32 + (D == 128 ? lane & 3 : i) * 8) =
                  make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
          }
        }
        __syncwarp();
      }
      if (mine && w.u.slot >= 0) a.part_ml[prow] = make_float2(m == -INFINITY ? m : m * sl, l);
      if (nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[x]);
      }
    }
    if (!alive) s_abort = 1;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
  }
  if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ------------------------------ MMA issuer of tile x (the whole warp; lane 0 issues) ------------------------------
    const int x = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);
    const bool lead = lane == 0;
    const uint32_t id_s = attn_idesc(kHalf, false), id_o = attn_idesc(D, true);
    const uint64_t dq = umma_desc_sw128(smem + x * L::kTile), dk = umma_desc_sw128(ring), dv = umma_desc_mn(ring, L::kBox);
    const uint32_t q_hi = (uint32_t)(dq >> 32), k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
    const uint32_t q_lo = __shfl_sync(0xffffffffu, (uint32_t)dq, 0), k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
    constexpr uint32_t kTileStep = L::kTile >> 4, kHalfStep = (kHalf * 128) >> 4;  // 128-byte rows
    const uint32_t t_s = __shfl_sync(0xffffffffu, tmem + x * 128, 0), t_o = t_s + 256;
    int n_q = 0, n_p = 0, n_o = 0;  // phases used of q_full, p_full, o_free
    int kv = 0;                     // tiles taken from the ring
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait(bar, parity) ? 1 : 0)) {
        ok = false;
        if (lead) atomicOr(&a.ctrl->err, kErrTimeout);
      }
      return ok;
    };
    // Done with a tile of the ring (or with Q): once this warp's products so far are complete, or at
    // once if it made none of it.
    auto release = [&](uint64_t* bar, bool used) {
      if (used) umma_commit_if(bar, lead);
      else if (lead) mbar_arrive(bar);
    };
    auto issue_s = [&](int slot, int h) {  // S = Q K^T of 64 keys
      const uint32_t db = __shfl_sync(0xffffffffu, k_lo + slot * kTileStep, 0) + h * kHalfStep;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t step = (uint32_t)((k / 4) * (L::kBox >> 4) + (k % 4) * 2);
        umma_ss(t_s + h * kHalf, q_lo + step, q_hi, db + step, k_hi, id_s, k > 0, lead);
      }
      umma_commit_if(&s_full[x][h], lead);
    };
    for (int it = 0; ok && !warp_aborted(&s_abort); ++it) {
      int head, unit;
      if (!queue_take(queue, a, it, lane, unit)) {
        ok = false;
        break;
      }
      if (unit < 0) break;
      const AttnWork w = attn_work(a, unit, s_unit, head);
      if (w.n == 0) continue;
      const int nk = x ? w.nk[1] : w.nk[0];
      if (!wait(&kv_full[kv % NS], (kv / NS) & 1)) break;
      if (nk > 0) {
        if (!wait(&q_full[x], n_q++ & 1)) break;
        issue_s(kv % NS, 0);
        issue_s(kv % NS, 1);
      }
      release(&kv_empty[kv % NS], nk > 0);
      if (w.n == 1) release(&q_free, nk > 0);
      for (int j = 0; j < w.n; ++j) {
        const int cv = kv + 2 * j + 1, ck = cv + 1;
        if (!wait(&kv_full[cv % NS], (cv / NS) & 1)) break;
        if (j + 1 < w.n && j >= nk && !wait(&kv_full[ck % NS], (ck / NS) & 1)) break;
        if (j < nk) {
          const uint32_t db = __shfl_sync(0xffffffffu, v_lo + (cv % NS) * kTileStep, 0);
          if (j == 0 && !wait(&o_free[x], (n_o++ & 1) ^ 1)) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(&p_full[x][h], n_p & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kHalf / 16; ++k)
              umma_ts(t_o, t_s + h * kHalf + k * 8, db + h * kHalfStep + k * (2048 >> 4), v_hi, id_o, j > 0 || h > 0 || k > 0, lead);
            if (j + 1 == nk) umma_commit_if(h ? &o_done[x] : &o_prev[x], lead);
            if (j + 1 < w.n) {
              if (h == 0 && !wait(&kv_full[ck % NS], (ck / NS) & 1)) break;
              // in issue order behind the product that reads P where this S goes
              if (j + 1 < nk) issue_s(ck % NS, h);
            }
          }
          if (!ok) break;
          ++n_p;
        }
        release(&kv_empty[cv % NS], j < nk);
        if (j + 1 < w.n) release(&kv_empty[ck % NS], j + 1 < nk);
        if (j + 2 == w.n) release(&q_free, nk > 0);
      }
      kv += 2 * w.n;
    }
    if (!ok) s_abort = 1;
    umma_commit_if(&drain[x], lead);  // every MMA of this warp has completed once it arrives
    if (!mbar_wait(&drain[x], 0)) atomicOr(&a.ctrl->err, kErrTimeout);
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------ TMA loads ------------------------------
    int kv = 0, n_q[2] = {0, 0}, n_act = 0;
    uint32_t raw_used = 0, raw_par = 0;  // a bit a stage: used through v_raw; how often, mod 2
    bool ok = true;
    const uint32_t q_bytes = (uint32_t)a.PT * a.G * D * 2;
    for (int it = 0; ok && !warp_aborted(&s_abort); ++it) {
      int head, unit;
      if (!queue_draw(queue, a, it, n_units, lane, unit)) {
        ok = false;
        break;
      }
      if (unit < 0) break;
      const AttnWork w = attn_work(a, unit, s_unit, head);
      if (w.n == 0) continue;
      if (!soft_wait(&q_free, (n_act++ & 1) ^ 1, a.ctrl, lane)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (w.nk[x] > 0) {
          if (lane == 0) {
            mbar_expect_tx(&q_full[x], q_bytes);
            for (int c = 0; c < D / 64; ++c)
              tma_3d(smem + x * L::kTile + c * L::kBox, &a.map_q, c * 64, head * a.G, w.u.row + x * a.PT, &q_full[x]);
          }
          ++n_q[x];
        }
      for (int j = 0; j < w.n && ok; ++j) {
        const int row = (w.u.kt0 + j) * kAttnTile;
        for (int v = 0; v < 2; ++v, ++kv) {
          const int s = kv % NS;
          if (!soft_wait(&kv_empty[s], ((kv / NS) & 1) ^ 1, a.ctrl, lane) || warp_aborted(&s_abort)) {
            ok = false;
            break;
          }
          const CUtensorMap* map = v ? &a.map_v : &a.map_k;
          const uint32_t dst = ring + s * L::kTile;
          // (the sequence's last tiles go through the cleaning warp)
          const bool fix = v && row + kAttnTile > w.u.seen;
          uint64_t* bar = fix ? &v_raw[s] : &kv_full[s];
          if (fix) {
            raw_used |= 1u << s;
            raw_par ^= 1u << s;
          }
          if (lane == 0) {
            mbar_expect_tx(bar, L::kTile);
            for (int c = 0; c < D / 64; ++c) tma_3d(dst + c * L::kBox, map, c * 64, head, w.u.kv0 + row, bar);
          }
        }
      }
    }
    if (!ok) s_abort = 1;
    // no copy may still be landing when the CTA leaves
    if (lane == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (n_q[x] && !mbar_wait(&q_full[x], (n_q[x] - 1) & 1)) atomicOr(&a.ctrl->err, kErrTimeout);
      for (int s = 0; s < NS; ++s)
        if (((raw_used >> s) & 1) && !mbar_wait(&v_raw[s], ((raw_par >> s) & 1) ^ 1)) atomicOr(&a.ctrl->err, kErrTimeout);
      drain_ring(kv_full, NS, kv, a.ctrl);
    }
    __syncwarp();
  } else if (warp == kCleanWarp) {
    // ------------------------------ infinities and NaN in hidden values ------------------------------
    // (while the tile's scores and softmax are computed: its values are not needed before)
    int kv = 0;
    uint32_t raw_par = 0;
    bool ok = true;
    for (int it = 0; ok && !warp_aborted(&s_abort); ++it) {
      int head, unit;
      if (!queue_take(queue, a, it, lane, unit)) {
        ok = false;
        break;
      }
      if (unit < 0) break;
      const AttnWork w = attn_work(a, unit, s_unit, head);
      if (lane == 0) s_bad[it & 3] = 0;
      __syncwarp();
      for (int j = max(0, max(w.u.seen, 0) / kAttnTile - w.u.kt0); j < w.n; ++j) {
        const int s = (kv + 2 * j + 1) % NS;
        if (!soft_wait(&v_raw[s], (raw_par >> s) & 1, a.ctrl, lane)) {
          ok = false;
          break;
        }
        raw_par ^= 1u << s;
        if (clean_rows<D>(ring + s * L::kTile, 0, kAttnTile, w.u.len - (w.u.kt0 + j) * kAttnTile, true, lane)) s_bad[it & 3] = 1;
        proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[s]);
      }
      kv += 2 * w.n;
    }
    if (!ok) s_abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ---------------------------------------------------------------------------------------
// Few rows (single tokens): 16 rows against all keys, bound by reading the keys
// ---------------------------------------------------------------------------------------
// A unit has at most 16 rows, the height of mma.sync's tile, so the 128-row tiles of tcgen05 would
// be filled to an eighth at most and their chain of products, softmax and TMEM round trips (about
// 3.3 us per 128 keys) would be longer than the keys' way from memory (1.5 us at this SM's share).
// Here eight warps take 16 keys each of a tile of 128, on their own: scores, softmax and the sums
// of P V stay in the warp's registers, with a running maximum of its own; the eight are joined
// once, at the end of the unit.  A ninth warp loads the tiles by TMA.
constexpr int kFewWarps = 8, kFewThreads = (kFewWarps + 1) * 32;

template <int D>
struct FewSmem {
  static constexpr int kTile = kAttnTile * D * 2;        // a K or V tile
  static constexpr int kBox = kAttnTile * 64 * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;       // K and V tile pairs
  static constexpr int kLd = D + 8;                      // row stride (floats) of the joined sums
  static constexpr int kSum = kFewRows * kLd * 4;
  static constexpr int kBytes = kStages * 2 * kTile + 2 * kSum + 1024;
};

// d (16 x 8, fp32) += a (16 x 16, bf16) b (16 x 8, bf16); fragments as in the PTX manual
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void few_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory"); }

// SELF: without a plan kernel (a template: the branches cost the cut calls' kernel registers, 0.4 us of 25 and 39)
template <int D, bool SELF>
__global__ void __launch_bounds__(kFewThreads, 1) k_attn_few(const __grid_constant__ AttnArgs a, const uint16_t* q) {
  using L = FewSmem<D>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS];
  __shared__ int s_last;
  __shared__ AttnUnit s_unit;
  __shared__ int s_blocks;
  __shared__ float2 s_ml2[2][kFewWarps][kFewRows];  // by turns: a warp may still read one unit's while another is at the next's end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* sums = reinterpret_cast<float*>(smem_raw + (smem - smem_u32(smem_raw)) + NS * 2 * L::kTile);
  if (warp == kFewWarps && lane < 2 && a.kv_rows > 0) prefetch_map(lane ? &a.map_v : &a.map_k);
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kFewWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (SELF) {
    if (warp == kFewWarps) {
      AttnUnit u;
      const int blocks = attn_self_plan(a, (int)blockIdx.x / a.Hkv, lane, u);
      if (lane == 0) {
        s_unit = u;
        s_blocks = blocks;
      }
    }
    __syncthreads();
  }
  const int n_units = SELF ? s_blocks * a.Hkv : a.hdr->n_units;

  if (warp == kFewWarps) {
    // ------------------------------ TMA loads ------------------------------
    int kv = 0;
    bool ok = true;
    for (int it = 0; ok && unit_index(it) < n_units; ++it) {
      const int unit = unit_index(it);
      const int e = unit / a.Hkv, head = unit - e * a.Hkv;
      const AttnUnit u = SELF ? s_unit : a.units[e];
      for (int kt = u.kt0; kt < u.kt1; ++kt, ++kv) {
        const int s = kv % NS;
        if (!soft_wait(&empty[s], ((kv / NS) & 1) ^ 1, a.ctrl, lane)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_expect_tx(&full[s], 2 * L::kTile);
          for (int z = 0; z < 2; ++z)
            for (int c = 0; c < D / 64; ++c)
              tma_3d(smem + (2 * s + z) * L::kTile + c * L::kBox, z ? &a.map_v : &a.map_k, c * 64, head, u.kv0 + kt * kAttnTile,
                     &full[s]);
        }
      }
    }
    if (lane == 0) drain_ring(full, NS, kv, a.ctrl);
    return;
  }

  // ------------------------------ the eight warps ------------------------------
  const int g = lane >> 2, u2 = 2 * (lane & 3);
  int kv = 0;
  bool ok = true;  // after a wait that ran out the warp only keeps its place in the barriers
  for (int it = 0; unit_index(it) < n_units; ++it) {
    const int unit = unit_index(it);
    const int e = unit / a.Hkv, head = unit - e * a.Hkv;
    const AttnUnit u = SELF ? s_unit : a.units[e];
    const int rows = u.npos * a.G;
    // row i of the unit is (position i / G, head i % G of the group)
    uint32_t qa[D / 16][4];
    int seen[2];  // keys that this lane's rows g and g + 8 see
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r, pos = row / a.G, sub = row - pos * a.G;
      seen[r] = row < rows ? u.seen + pos : 0;
      const uint16_t* src = q + ((size_t)(u.row + pos) * a.Hq + (size_t)head * a.G + sub) * D + u2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          qa[k][r + 2 * c] = row < rows ? *reinterpret_cast<const uint32_t*>(src + k * 16 + c * 8) : 0u;
    }
    float O[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) O[n][x] = 0.f;

    for (int kt = u.kt0; kt < u.kt1; ++kt, ++kv) {
      const int st = kv % NS;
      if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (kv / NS) & 1) ? 1 : 0);
        if (!ok && lane == 0) atomicOr(&a.ctrl->err, kErrTimeout);
      }
      if (!ok) continue;
      const uint32_t tk = smem + 2 * st * L::kTile, tv = tk + L::kTile;
      const int key0 = kt * kAttnTile + warp * 16;  // this warp's first key
      float x[2][4] = {};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int row = warp * 16 + n * 8 + (lane & 7);
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t b[4];
          ldsm4(tk + (k2 >> 1) * L::kBox + row * 128 + ((((k2 & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4), b);
          mma_bf16(x[n], qa[2 * k2], b[0], b[1]);
          mma_bf16(x[n], qa[2 * k2 + 1], b[2], b[3]);
        }
      }
      float mn[2] = {m[0], m[1]};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[n][i] = key0 + n * 8 + u2 + (i & 1) < seen[i >> 1] ? x[n][i] * a.scale_log2 : -INFINITY;
          mn[i >> 1] = fmaxf(mn[i >> 1], x[n][i]);
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mn[0] = fmaxf(mn[0], __shfl_xor_sync(0xffffffffu, mn[0], o));
        mn[1] = fmaxf(mn[1], __shfl_xor_sync(0xffffffffu, mn[1], o));
      }
      // (-inf) - (-inf) is no rise
      const bool up = mn[0] - m[0] > kRescale || mn[1] - m[1] > kRescale;
      if (__any_sync(0xffffffffu, up)) {
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bool mine = mn[r] - m[r] > kRescale;
          f[r] = mine ? ex2(m[r] - mn[r]) : 1.f;
          if (mine) m[r] = mn[r];
          l[r] *= f[r];
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[n][i] *= f[i >> 1];
      }
      const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
      uint32_t p[4], pl[4];  // the weights and what their rounding to bf16 leaves
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = ex2(x[n][0] - b0), p1 = ex2(x[n][1] - b0), p2 = ex2(x[n][2] - b1), p3 = ex2(x[n][3] - b1);
        l[0] += p0 + p1;
        l[1] += p2 + p3;
        p[2 * n] = pack_bf16(p0, p1);
        p[2 * n + 1] = pack_bf16(p2, p3);
        pl[2 * n] = pack_bf16(p0 - bf_lo(p[2 * n]), p1 - bf_hi(p[2 * n]));
        pl[2 * n + 1] = pack_bf16(p2 - bf_lo(p[2 * n + 1]), p3 - bf_hi(p[2 * n + 1]));
      }
      // keys that not every row sees: this warp cleans its own.  With one position a unit no row sees
      // the keys from u.seen on (the sequence's last ones, if the position is not), so they are all cleared.
      bool bad = false;
      if (key0 + 16 > u.seen) {
        const int end = u.npos > 1 ? u.len : max(u.seen, 0);
        bad = __any_sync(0xffffffffu, clean_rows<D>(tv, warp * 16, warp * 16 + 16, end - kt * kAttnTile, u.npos > 1, lane));
        proxy_fence();  // before the next copy into the tile
        __syncwarp();
      }
      const int vrow = warp * 16 + (lane & 15);
#pragma unroll
      for (int n2 = 0; n2 < D / 16; ++n2) {
        uint32_t b[4];
        ldsm4_t(tv + (n2 >> 2) * L::kBox + vrow * 128 + ((((n2 & 3) * 2 + (lane >> 4)) ^ (vrow & 7)) << 4), b);
        mma_bf16(O[2 * n2], p, b[0], b[1]);
        mma_bf16(O[2 * n2 + 1], p, b[2], b[3]);
        mma_bf16(O[2 * n2], pl, b[0], b[1]);
        mma_bf16(O[2 * n2 + 1], pl, b[2], b[3]);
      }
      if (bad) {
        const uint16_t* src = attn_value(a, u.kv0 + key0, head) + u2;
        for (int j = 0; j < 16 && key0 + j < u.len; ++j, src += (size_t)a.Hkv * D)
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(src + n * 8), nf = bf16x2_nonfinite(w);
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (key0 + j < seen[r]) {
                if (nf & 0x8000u) O[n][2 * r] += bf_lo(w);
                if (nf >> 31) O[n][2 * r + 1] += bf_hi(w);
              }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // ---- join the eight warps ----
    float2 (*s_ml)[kFewRows] = s_ml2[it & 1];
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    if ((lane & 3) == 0) {
      s_ml[warp][g] = make_float2(m[0], l[0]);
      s_ml[warp][g + 8] = make_float2(m[1], l[1]);
    }
    few_sync();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, s_ml[w][g + 8 * r].x);
      const float f = ex2(m[r] - (top == -INFINITY ? 0.f : top));
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        O[n][2 * r] *= f;
        O[n][2 * r + 1] *= f;
      }
    }
    float* mine = sums + (warp & 1) * (L::kSum / 4);
#pragma unroll
    for (int turn = 0; turn < 4; ++turn) {
      if (warp >> 1 == turn) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float2* at = reinterpret_cast<float2*>(mine + (g + 8 * r) * L::kLd + n * 8 + u2);
            float2 v = make_float2(O[n][2 * r], O[n][2 * r + 1]);
            if (turn) v = add2(v, *at);
            *at = v;
          }
      }
      few_sync();
    }
    constexpr int kPer = kFewRows * D / (kFewWarps * 32);  // columns of a thread: 4 or 8
    const int row = tid / (D / kPer), col = (tid % (D / kPer)) * kPer;
    if (row < rows) {
      const int pos = row / a.G, sub = row - pos * a.G;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float2 ml = s_ml[w][row];
        sum += ml.y == 0.f ? 0.f : ml.y * ex2(ml.x - (top == -INFINITY ? 0.f : top));
      }
      float v[kPer];
#pragma unroll
      for (int c = 0; c < kPer; c += 4) {
        const float4 x = *reinterpret_cast<const float4*>(sums + row * L::kLd + col + c);
        const float4 y = *reinterpret_cast<const float4*>(sums + L::kSum / 4 + row * L::kLd + col + c);
        v[c] = x.x + y.x;
        v[c + 1] = x.y + y.y;
        v[c + 2] = x.z + y.z;
        v[c + 3] = x.w + y.w;
      }
      if (!SELF && u.slot >= 0) {
        const size_t prow = ((size_t)u.slot * a.Hkv + head) * a.rows_slot + row;
#pragma unroll
        for (int c = 0; c < kPer; c += 4)
          *reinterpret_cast<float4*>(a.part_o + prow * D + col + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        if (col == 0) a.part_ml[prow] = make_float2(top, sum);
        __threadfence();
      } else {
        const float inv = 1.0f / sum;
        uint32_t o[kPer / 2];
#pragma unroll
        for (int c = 0; c < kPer; c += 2) o[c / 2] = u.seen + pos > 0 ? pack_bf16(v[c] * inv, v[c + 1] * inv) : 0u;
        uint16_t* dst = a.out + ((size_t)(u.row + pos) * a.Hq + (size_t)head * a.G + sub) * D + col;
        if constexpr (kPer == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
      }
    }
    if (SELF || u.slot < 0) continue;
    // ---- join the pieces: the CTA that finishes the last of a group joins the group in the place of
    // its first, the one that finishes the last group joins the groups.  Up to 16 pieces are one
    // group; more make groups of eight (one CTA alone would read a long cache's 70 pieces in 9 us,
    // the two steps take 5) ----
    const int size = u.pieces > 16 ? 8 : u.pieces, group = (u.slot - u.slot0) / size, groups = (u.pieces + size - 1) / size;
    for (int level = 0; level < 2; ++level) {
      const int count = level ? groups : min(size, u.pieces - group * size);
      const int first = level ? u.slot0 : u.slot0 + group * size, step = level ? size : 1;
      few_sync();  // every part of this piece (or group) is written and fenced
      if (tid == 0) s_last = atomicAdd(&a.done[(level * kAttnMaxSlots + first) * a.Hkv + head], 1) == count - 1;
      few_sync();
      if (s_last == 0) break;
      __threadfence();
      constexpr int kLanes = D / 4;  // four columns a thread, 8 (D = 128) or 16 rows at a time
      const bool final = level || groups == 1;
      const size_t next = (size_t)step * a.Hkv * a.rows_slot;
      for (int r = tid / kLanes; r < rows; r += kFewWarps * 32 / kLanes) {
        const size_t at0 = ((size_t)first * a.Hkv + head) * a.rows_slot + r;
        const int c4 = (tid % kLanes) * 4, pos = r / a.G, sub = r - pos * a.G;
        float m = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < count; p += 8) {
          float2 ml[8];
          float4 v[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const size_t at = at0 + min(p + x, count - 1) * next;
            ml[x] = __ldcg(&a.part_ml[at]);
            v[x] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + c4));
          }
          float mn = m;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (ml[x].y != 0.f) mn = fmaxf(mn, ml[x].x);
          const float base = mn == -INFINITY ? 0.f : mn, back = ex2(m - base);
          m = mn;
          sum *= back;
          o = make_float4(o.x * back, o.y * back, o.z * back, o.w * back);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            // a sum of 0: the row sees none of the piece's keys, and what it holds does not count
            if (p + x >= count || ml[x].y == 0.f) continue;
            const float f = ex2(ml[x].x - base);
            sum = fmaf(ml[x].y, f, sum);
            o = make_float4(fmaf(v[x].x, f, o.x), fmaf(v[x].y, f, o.y), fmaf(v[x].z, f, o.z), fmaf(v[x].w, f, o.w));
          }
        }
        if (final) {
          const float inv = 1.0f / sum;
          uint16_t* dst = a.out + ((size_t)(u.row + pos) * a.Hq + (size_t)head * a.G + sub) * D + c4;
          *reinterpret_cast<uint2*>(dst) =
              u.seen + pos > 0 ? make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv)) : make_uint2(0u, 0u);
        } else {
          // A row's lanes, all or half of a warp, have all read the place that is overwritten.  (The other
          // half may be done: an odd number of rows.)
          __syncwarp((kLanes == 32 ? 0xffffffffu : 0xffffu) << (lane & (32 - kLanes)));
          __stcg(reinterpret_cast<float4*>(a.part_o + at0 * D + c4), o);
          if (c4 == 0) __stcg(&a.part_ml[at0], make_float2(m, sum));
          __threadfence();
        }
      }
      if (final) break;
    }
  }
}

// Joins the pieces of the cut blocks of k_attn (k_attn_few joins its own): a thread has eight columns of
// a row, a CTA those of 128 rows; a row's pieces are added in order, four loaded at a time.
constexpr int kJoinRows = 128, kJoinCols = 8;
template <int D>
__global__ void __launch_bounds__(kJoinRows) k_attn_join(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int n_recs = a.hdr->n_recs, row_parts = (a.rows_slot + kJoinRows - 1) / kJoinRows;
  const int per = row_parts * (D / kJoinCols) * a.Hkv;  // of a block
  for (int item = blockIdx.x; item < n_recs * per; item += gridDim.x) {
    const AttnRec rec = a.recs[item / per];
    const int rest = item % per, head = rest % a.Hkv, part = rest / a.Hkv;
    const int c4 = part % (D / kJoinCols) * 2, row = part / (D / kJoinCols) * kJoinRows + threadIdx.x;
    if (row >= rec.npos * a.G) continue;
    const size_t base = (size_t)rec.slot * a.Hkv + head;
    const float2* pml = a.part_ml + base * a.rows_slot + row;
    const float4* po = reinterpret_cast<const float4*>(a.part_o) + (base * (D / 4) + c4) * a.rows_slot + row;
    const size_t ml_step = (size_t)a.Hkv * a.rows_slot, o_step = ml_step * (D / 4);
    float m = -INFINITY, sum = 0.f, o[kJoinCols] = {};
    for (int p = 0; p < rec.pieces; p += 4) {
      float2 ml[4];
      float4 v[4][2];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int q = min(p + x, rec.pieces - 1);
        ml[x] = __ldcg(pml + q * ml_step);
        v[x][0] = __ldcg(po + q * o_step);
        v[x][1] = __ldcg(po + q * o_step + a.rows_slot);
      }
      float mn = m;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (ml[x].y != 0.f) mn = fmaxf(mn, ml[x].x);
      const float base_m = mn == -INFINITY ? 0.f : mn, back = ex2(m - base_m);
      m = mn;
      sum *= back;
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) o[e] *= back;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // a sum of 0: the row sees none of the piece's keys, and what it holds does not count
        if (p + x >= rec.pieces || ml[x].y == 0.f) continue;
        const float f = ex2(ml[x].x - base_m);
        sum = fmaf(ml[x].y, f, sum);
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) o[e] = fmaf(reinterpret_cast<const float*>(v[x])[e], f, o[e]);
      }
    }
    const int pos = row / a.G, sub = row - pos * a.G;
    const float inv = 1.0f / sum;
    uint32_t r[kJoinCols / 2];
#pragma unroll
    for (int e = 0; e < kJoinCols; e += 2) r[e / 2] = rec.seen + pos > 0 ? pack_bf16(o[e] * inv, o[e + 1] * inv) : 0u;
    *reinterpret_cast<uint4*>(a.out + ((size_t)(rec.row + pos) * a.Hq + (size_t)head * a.G + sub) * D + c4 * 4) =
        make_uint4(r[0], r[1], r[2], r[3]);
  }
}

}  // namespace

// The most blocks (units before cutting) that a call can have.
static long long attn_max_blocks(int n_seqs, int T, int BP) { return (long long)T / BP + std::min(n_seqs, T); }
static bool attn_may_cut(int max_kv) { return max_kv > kAttnMinPiece * kAttnTile; }
// Few rows: at most 16 per sequence on average (single tokens, or so few that 16-row units do).
static bool attn_few(const moe_attn_shape* s, int n_seqs, int T) {
  const int G = s->n_q_heads / s->n_kv_heads;
  return G <= kFewRows && (long long)T * G <= (long long)kFewRows * n_seqs;
}

template <int D>
static cudaError_t launch_attn_d(AttnArgs& a, const uint16_t* q, bool few, int n_sm, cudaStream_t s) {
  const long long blocks = attn_max_blocks(a.n_seqs, a.T, a.BP);
  const bool cut = attn_may_cut(a.max_kv);
  const long long units = (blocks + (cut ? kAttnMaxSlots : 0)) * a.Hkv;
  a.fill = !cut ? 0 : few ? kAttnFillFew : kAttnFill;
  // longest first where a CTA has several units (100 tokens over caches of 1 to 3,000: 110 against 120
  // us), but not where few-rows units are mostly equal pieces (32 tokens over caches of 0.2 to 8
  // thousand: 38.5 against 36.3)
  a.sort = units > n_sm && !(few && blocks * a.Hkv <= 2 * n_sm);
  a.few = few;
  a.n_sm = std::min(n_sm, kAttnMaxSlots);  // (pieces of one round have a slot each)
  a.self_plan = a.n_seqs <= kWarpSeqs && !cut && units <= n_sm;
  cudaError_t e = a.self_plan ? cudaSuccess : launch_pdl(k_attn_plan, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)std::min<long long>(n_sm, units));
  if (few) {
    const auto fn = a.self_plan ? k_attn_few<D, true> : k_attn_few<D, false>;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<D>::kBytes);
    if (e == cudaSuccess) e = launch_pdl(fn, grid, dim3(kFewThreads), FewSmem<D>::kBytes, s, a, q);
  } else {
    e = cudaFuncSetAttribute(k_attn<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, AttnSmem<D>::kBytes);
    if (e == cudaSuccess) e = launch_pdl(k_attn<D>, grid, dim3(kAttnThreads), AttnSmem<D>::kBytes, s, a);
  }
  if (e != cudaSuccess || few || !cut) return e;
  const long long parts = std::min<long long>(blocks, kAttnMaxSlots / 2) * a.Hkv * (D / kJoinCols) *
                          ((a.rows_slot + kJoinRows - 1) / kJoinRows);
  return launch_pdl(k_attn_join<D>, dim3((unsigned)std::min<long long>(parts, 8 * n_sm)), dim3(kJoinRows), 0, s, a);
}

cudaError_t launch_attn(AttnArgs& a, bool few, const void* q, const void* k, const void* v, cudaStream_t s) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // [row, head, column]: boxes of 64 columns x the group's heads x PT positions, or one head x 128 keys
  const auto map = [&](CUtensorMap* m, const void* base, int rows, int heads, int box_heads, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)heads * a.d * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!few && (e = map(&a.map_q, q, a.T, a.Hq, a.G, a.PT)) != cudaSuccess) return e;
  // without keys no unit has a key tile and the maps are not used
  if (a.kv_rows > 0) {
    if ((e = map(&a.map_k, k, a.kv_rows, a.Hkv, 1, kAttnTile)) != cudaSuccess) return e;
    if ((e = map(&a.map_v, v, a.kv_rows, a.Hkv, 1, kAttnTile)) != cudaSuccess) return e;
  }
  const uint16_t* qp = static_cast<const uint16_t*>(q);
  return a.d == 64 ? launch_attn_d<64>(a, qp, few, n_sm, s) : launch_attn_d<128>(a, qp, few, n_sm, s);
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
  if (attn_max_blocks(n_seqs, T, 1) * Hkv > 1LL << 30)
    return set_error(MOE_ERR_INVALID, "T * n_q_heads too large");
  return MOE_OK;
}

struct AttnLayout {
  size_t ctrl, seqs, hdr, units, recs, done, part_o, part_ml, total;
  int PT, BP, rows_slot;
  bool few;
};
static AttnLayout attn_layout(const moe_attn_shape* shape, int n_seqs, int T, int max_kv, bool few) {
  AttnLayout W{};
  const int G = shape->n_q_heads / shape->n_kv_heads;
  W.few = few;
  W.PT = W.few ? kFewRows / G : kAttnTile / G;
  W.BP = W.few ? W.PT : 2 * W.PT;
  W.rows_slot = std::min(W.BP, std::max(T, 1)) * G;
  size_t pos = 0;
  auto take = [&](size_t bytes) {
    const size_t at = (size_t)round_up((int64_t)pos, kAlign);
    pos = at + bytes;
    return at;
  };
  W.ctrl = take(sizeof(Ctrl));
  W.seqs = take(sizeof(AttnSeq) * (size_t)n_seqs);
  W.hdr = take(sizeof(AttnHdr));
  const size_t blocks = (size_t)attn_max_blocks(n_seqs, T, W.BP);
  // The pieces of cut blocks number at most kAttnMaxSlots over all key heads; a call whose keys
  // fit one piece cuts nothing.
  const size_t slots = attn_may_cut(max_kv) ? kAttnMaxSlots : 0;
  W.units = take(sizeof(AttnUnit) * (blocks + slots));
  W.recs = take(sizeof(AttnRec) * std::min(blocks, slots / 2));
  W.done = take(W.few ? sizeof(int) * 2 * slots * shape->n_kv_heads : 0);
  W.part_o = take(sizeof(float) * slots * W.rows_slot * shape->d);
  W.part_ml = take(sizeof(float2) * slots * W.rows_slot);
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
  // Each kernel's layout grows with n_seqs, T and max_kv, but which kernel takes a call does not: fewer
  // sequences of as many rows may need the larger layout.  The larger of both serves every smaller call.
  *bytes = attn_layout(shape, n_seqs, T, max_kv, false).total;
  if (shape->n_q_heads / shape->n_kv_heads <= kFewRows)
    *bytes = std::max(*bytes, attn_layout(shape, n_seqs, T, max_kv, true).total);
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
  if (!std::isfinite(scale * 1.44269504088896340736f)) return set_error(MOE_ERR_INVALID, "scale must be finite");
  if (!ws) return set_error(MOE_ERR_INVALID, "ws is NULL");
  const uintptr_t all = (uintptr_t)q_offsets | (uintptr_t)kv_begin | (uintptr_t)kv_len | (uintptr_t)q | (uintptr_t)k |
                        (uintptr_t)v | (uintptr_t)out | (uintptr_t)ws;
  if (all & 15) return set_error(MOE_ERR_INVALID, "every pointer must be 16-byte aligned");
  const AttnLayout W = attn_layout(shape, n_seqs, T, max_kv, attn_few(shape, n_seqs, T));
  if (ws_bytes < W.total) return set_error(MOE_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, W.total);
  if (T == 0) return MOE_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnArgs a{};
  a.n_seqs = n_seqs;
  a.T = T;
  a.Hq = shape->n_q_heads;
  a.Hkv = shape->n_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.d = shape->d;
  a.PT = W.PT;
  a.BP = W.BP;
  a.max_kv = max_kv;
  a.kv_rows = kv_rows;
  a.rows_slot = W.rows_slot;
  // A scale of 0 (every key seen counts the same) as one whose scores vanish next to each other:
  // 0 times the mask's infinity would be NaN.
  a.scale_log2 = scale == 0.f ? 1e-30f : scale * 1.44269504088896340736f;
  a.offsets = q_offsets;
  a.kv_begin = kv_begin;
  a.kv_len = kv_len;
  a.v = static_cast<const uint16_t*>(v);
  a.out = static_cast<uint16_t*>(out);
  a.ctrl = reinterpret_cast<Ctrl*>(w + W.ctrl);
  a.seqs = reinterpret_cast<AttnSeq*>(w + W.seqs);
  a.hdr = reinterpret_cast<AttnHdr*>(w + W.hdr);
  a.units = reinterpret_cast<AttnUnit*>(w + W.units);
  a.recs = reinterpret_cast<AttnRec*>(w + W.recs);
  a.done = reinterpret_cast<int*>(w + W.done);
  a.part_o = reinterpret_cast<float*>(w + W.part_o);
  a.part_ml = reinterpret_cast<float2*>(w + W.part_ml);
  const cudaError_t e = launch_attn(a, W.few, q, k, v, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return MOE_OK;
}
