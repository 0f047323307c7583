// Span attention of prompts on the tensor cores (bf16 caches in device
// memory): Q K^T and P V with tcgen05.mma, accumulators and probabilities in
// tensor memory, K and V blocks by TMA.
//
// The query rows of KV head g of a sequence are its tokens' G heads: a row tile
// is 128 / G whole tokens, row r token r / G, head r % G, so the G heads of a
// token share the K and V blocks they read. One work item is two row tiles, A
// and B, of one (b, g) over the blocks of 128 slots that any of its rows sees.
// The CTAs (one per SM) walk the items, the longest first.
//
// Roles in a CTA (the softmax warps take registers from the others):
//  - warps 0-15: the softmax, two threads per row: warps 0-3 columns 0-63 of
//    tile A's S, 4-7 columns 64-127, 8-15 tile B. S from tensor memory, mask,
//    maximum (the two threads exchange theirs through shared memory), running
//    sum, P as bf16 into the tensor memory of S; at the end of an item half of
//    its output row each, and the next item's queries where they are rotated
//    here. With one thread per row the softmax of a tile (about 1400 cycles)
//    and its products (about 1100, half of them latency) made a chain that
//    kept the tensor core idle for more than a third of the time;
//  - warp 16: issues the products. Per block: O_A += P_A V, S_A' = Q_A K',
//    O_B += P_B V, S_B' = Q_B K' (K' the next block): while one tile's
//    softmax runs, the tensor core works for the other;
//  - warp 17: K and V blocks into a ring of 32 KB stages, and rotated queries.
// Everything one thread issues to the tensor core runs in issue order, so S_A'
// may overwrite P_A without a wait, and S_A' done implies O_A is complete.
//
// The softmax keeps a reference m per row: P = 2^(z - m), and O and the sum l
// are relative to the same m. m follows the running maximum only when that
// has grown by more than 2^8: until then P stays below 2^8, which costs no
// precision in floating point, and O, which lives in tensor memory, need not
// be rescaled. P is rounded to bf16 for the product (relative error 2^-8; the
// sum l adds the unrounded values); rotated queries (given as they are) are
// exact bf16, queries rotated here are kept to 16 bits as two bf16 terms, two
// products into the same accumulator.
//
// Slots of a block that none of the item's rows sees are never loaded (whole
// boxes: an out-of-range TMA coordinate reads zeros) or zeroed in shared
// memory before P V, since 0 * NaN would reach every row.
#pragma once

#include <cuda.h>

#include "attend_tc.cuh"
#include "span.cuh"

namespace fasa {

constexpr int kPrRows = 256;             // query rows per item (two tiles)
constexpr int kPrThreads = 640;          // five warpgroups; registers 4 * 104 + 64 = 5 * 96
// Tokens of a row tile.
__host__ __device__ constexpr int pr_tokens(int group) { return 128 / group; }
constexpr int kPrBlock = 128;            // slots per block
constexpr uint32_t kPrTile = 32768;      // bytes of a 128 x 128 bf16 tile pair
constexpr int kPrMaxSplits = 32;

struct PromptParams {
  CUtensorMap map_k, map_v;  // [rows][128] bf16, boxes of box_rows x 64, 128-byte swizzle
  CUtensorMap map_q;         // [B n_q][Hq][128], boxes of a tile's tokens x G x 64
  SpanParams s;
  int32_t n_items;           // tiles_max * B * Hkv * splits
  int32_t tiles_max;         // items of a (b, g) row at n_q queries
  int32_t splits;            // parts that an item's blocks are cut into
  int32_t box_rows;          // rows of a TMA box
  int32_t n_rows;            // rows of the K (and V) tensor
  float* part;               // [B * Hkv * tiles_max * splits][256][2 + 128]: m, l planes, then o
};

// Floats of a split's partial: m[256], l[256], o[256][128].
constexpr int64_t kPrPart = kPrRows * (2 + kD);

template <int TERMS>
struct PrSmem {
  static constexpr int kStages = TERMS == 1 ? 5 : 3;
  static constexpr uint32_t kQ = 2 * TERMS * kPrTile;  // tile A's terms, tile B's terms
  static constexpr uint32_t kBars = kQ + kStages * kPrTile;
  static constexpr uint32_t kPair = kBars + 256;          // [2 tiles][2 halves][128 rows] f32
  static constexpr uint32_t kTurns = kPair + 2048;
  static constexpr uint32_t kBytes = kTurns + (TERMS == 2 ? kNFC * 8 : 0);  // no static shared memory: the base is
                                                                            // 1024-byte aligned (checked)
};

// One item as every role sees it.
struct PrItem {
  bool valid;
  int b, g, j0, n_tok, L, tile, split;  // tokens j0 .. j0 + n_tok - 1
  int64_t pos0;      // position of the sequence's first query
  Span all;          // slots that some row of the item sees
  SpanUnits u;
  int i0, i1;        // this split's blocks
};

// P of a half's 64 columns takes the place of the upper 32 of them.
constexpr uint32_t kPrP = 32;

// What a role remembers of the sequence it read last: consecutive items are
// mostly of one sequence, and its lengths are two dependent loads.
struct PrSeq {
  int b, L, nq;
  int64_t pos0;
};

__device__ __forceinline__ PrItem pr_item(const PromptParams& p, int it, PrSeq& sq) {
  PrItem w;
  w.valid = false;
  const unsigned grid = gridDim.x, c = blockIdx.x;
  const unsigned n = (unsigned)it * grid + ((it & 1) ? grid - 1 - c : c);  // n_items + grid < 2^31
  if (n >= (unsigned)p.n_items) {
    w.b = -1;  // past the end: n grows with `it`
    return w;
  }
  const unsigned rows = p.s.batch * p.s.n_kv_heads;
  const int G = p.s.group;
  unsigned rk = n;
  w.split = 0;
  if (p.splits > 1) {
    rk = n / (unsigned)p.splits;
    w.split = (int)(n - rk * p.splits);
  }
  const int k = (int)(rk / rows);
  const unsigned r = rk - k * rows;
  w.b = (int)(r / (unsigned)p.s.n_kv_heads);
  w.g = (int)(r - w.b * p.s.n_kv_heads);
  if (w.b != sq.b) {
    sq.b = w.b;
    sq.L = span_len(p.s, w.b);
    sq.nq = span_qlen(p.s, w.b);
    sq.pos0 = span_pos0(p.s, w.b, sq.L, sq.nq);
  }
  w.L = sq.L;
  w.pos0 = sq.pos0;
  const int per = 2 * pr_tokens(G), tiles = (sq.nq + per - 1) / per;
  if (k >= tiles) return w;
  w.valid = true;
  w.tile = tiles - 1 - k;
  w.j0 = w.tile * per;
  w.n_tok = min(per, sq.nq - w.j0);
  const int64_t pa = w.pos0 + w.j0, pb = pa + w.n_tok - 1;
  // the union over positions pa .. pb: the last position's end, the first
  // one's window; its sinks are slots below lo, the rest is inside anyway
  const Span first = span_of(w.L, max(pa, (int64_t)0), p.s.window, p.s.n_sink);
  const Span last = span_of(w.L, pb, p.s.window, p.s.n_sink);
  w.all.hi = last.hi;
  w.all.lo = min(first.lo, last.hi);
  w.all.s = min(last.s, w.all.lo);
  w.u = span_units(w.all, kPrBlock);
  w.i0 = 0;
  w.i1 = w.u.n;
  if (p.splits > 1) {  // u.n * splits < 2^30 / 128 * 32
    w.i0 = (int)((unsigned)(w.u.n * w.split) / (unsigned)p.splits);
    w.i1 = (int)((unsigned)(w.u.n * (w.split + 1)) / (unsigned)p.splits);
  }
  return w;
}

// The 32-column chunks [ca, cb) of the block at slot t0 that hold slots which
// the item sees; the products and the softmax take these alone.
__device__ __forceinline__ void pr_chunks(const Span& all, int t0, int& ca, int& cb) {
  const int w0 = max(all.lo, t0), w1 = min(all.hi, t0 + kPrBlock);  // the window's part
  const int first = t0 < all.s || w1 <= w0 ? t0 : w0;
  const int last = w1 > w0 ? w1 : min(all.s, t0 + kPrBlock);
  ca = min((first - t0) / 32, 3);
  cb = min(max((last - t0 + 31) / 32, ca + 1), 4);  // every listed block holds some
}

// Instruction descriptor of S = Q K^T over n columns (see tc_idesc).
__device__ __forceinline__ uint32_t pr_idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// The products, accumulating or not. One thread issues 32 of them a block, so
// what it does per product counts: operands reach the tensor core through the
// warp's uniform registers, so all that a batch starts from is made uniform
// once (pr_uni) and each product adds constants to it; the accumulate
// predicate is a constant.
__device__ __forceinline__ uint32_t pr_uni(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
__device__ __forceinline__ bool pr_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
template <bool ACC>
__device__ __forceinline__ void pr_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
template <bool ACC>
__device__ __forceinline__ void pr_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// A descriptor (tc_desc) from its low word: start address and leading offset
// of 16-byte units; 1024-byte stride, version, 128-byte swizzle.
__device__ __forceinline__ uint64_t pr_desc(uint32_t lo) {
  return ((uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32) | lo;
}
// S = Q K^T, TERMS terms of Q: q, k low words of the tiles' first K-step.
template <int TERMS>
__device__ __forceinline__ void pr_issue_s(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
#pragma unroll
  for (int t = 0; t < TERMS; ++t)
#pragma unroll
    for (int k8 = 0; k8 < 8; ++k8) {
      const uint32_t o = ((k8 >> 2) * 16384 + (k8 & 3) * 32) >> 4;
      if (t + k8 == 0)
        pr_mma_ss<false>(d, pr_desc(q + o), pr_desc(k + o), idesc);
      else
        pr_mma_ss<true>(d, pr_desc(q + t * (kPrTile >> 4) + o), pr_desc(k + o), idesc);
    }
}
// Column of P for K-step k8 (16 slots), behind the tile's P base.
__host__ __device__ constexpr uint32_t pr_pcol(int k8) { return (k8 >> 2) * 64 + (k8 & 3) * 8; }
// O (+)= P V over the block's eight K-steps, or over [2 ca, 2 cb).
template <bool ACC>
__device__ __forceinline__ void pr_issue_o(uint32_t d, uint32_t pa, uint32_t v) {
  pr_mma_ts<ACC>(d, pa, pr_desc(v), tc_idesc(1));
#pragma unroll
  for (int k8 = 1; k8 < 8; ++k8) pr_mma_ts<true>(d, pa + pr_pcol(k8), pr_desc(v + k8 * (2048 >> 4)), tc_idesc(1));
}
__device__ __forceinline__ void pr_issue_part(uint32_t d, uint32_t pa, uint32_t v, int ca, int cb, bool acc) {
  for (int k8 = 2 * ca; k8 < 2 * cb; ++k8) {
    if (acc || k8 > 2 * ca)
      pr_mma_ts<true>(d, pa + pr_pcol(k8), pr_desc(v + k8 * (2048 >> 4)), tc_idesc(1));
    else
      pr_mma_ts<false>(d, pa + pr_pcol(k8), pr_desc(v + k8 * (2048 >> 4)), tc_idesc(1));
  }
}
__device__ __forceinline__ void pr_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tensor-memory loads; the registers pass through it,
// so that no use of them moves ahead of the wait.
__device__ __forceinline__ void pr_ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// 16 columns, waited for.
__device__ __forceinline__ void pr_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pr_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void pr_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void pr_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The larger, NaN if either is.
__device__ __forceinline__ float pr_max(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float pr_max3(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pr_two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 pr_both(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t pr_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pr_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// One arrival for the warp, behind its tensor-memory stores.
__device__ __forceinline__ void pr_stored(uint64_t* bar, int lane) {
  pr_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) pr_arrive(bar);
}
__device__ __forceinline__ float pr_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void pr_tma3(const CUtensorMap* map, void* dst, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// Tile of box_rows x 64 elements at (column x, row y) into shared memory.
__device__ __forceinline__ void pr_tma(const CUtensorMap* map, void* dst, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// Bounded wait of a whole warp: every lane learns whether all got through.
__device__ __forceinline__ bool pr_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
}

// Word w (columns 32 w .. 32 w + 31) of the columns a row sees in a block
// that starts at slot t0.
__device__ __forceinline__ uint32_t pr_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t pr_mask(const Span& v, int t0, int w) {
  const int t = t0 + 32 * w;
  return pr_below(v.hi - t) & (~pr_below(v.lo - t) | pr_below(v.s - t));
}

// Register k of the four lanes of a group, transposed: lane k ends up with the
// k-th 16 bytes of each of the four lanes.
__device__ __forceinline__ void pr_transpose4(uint32_t (&u)[16], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t &lo = u[4 * i + d], &hi = u[4 * i + 4 + d];
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, b0 ? lo : hi, 1);
      if (b0) lo = got; else hi = got;
    }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t &lo = u[4 * i + d], &hi = u[4 * i + 8 + d];
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, b1 ? lo : hi, 2);
      if (b1) lo = got; else hi = got;
    }
}

// A row's state between blocks.
struct PrRow {
  float m_ref, l;
  Span v;       // the slots it sees
};

// The reference follows the block's maximum m_blk where that has outgrown it;
// O and l with it.
__device__ __forceinline__ void pr_follow(PrRow& row, float m_blk, uint32_t t_o, bool first) {
  if (m_blk != m_blk) row.l = m_blk;  // a NaN logit
  const bool grow = m_blk > row.m_ref + 8.0f || (row.m_ref == -INFINITY && m_blk > -INFINITY);
  if (!__any_sync(0xFFFFFFFFu, grow)) return;
  const float m_new = grow ? m_blk : row.m_ref;
  const float f = row.m_ref == -INFINITY ? 0.0f : pr_ex2(row.m_ref - m_new);
  if (!first && __any_sync(0xFFFFFFFFu, grow && row.m_ref > -INFINITY)) {
    const float fo = grow ? f : 1.0f;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {  // this thread's half of the O row
      uint32_t o[16];
      pr_ld16(t_o + q * 16, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
      pr_st16(t_o + q * 16, o);
    }
  }
  if (grow) {
    row.l *= f;
    row.m_ref = m_new;
  }
}
// 32 columns' P (as 16 words) and its part of the sum; x2 = s c2 + off2.
__device__ __forceinline__ void pr_probs(const uint32_t* s, uint32_t* pk, uint64_t c2, uint64_t off2, uint64_t (&ls)[2]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint64_t x = pr_fma2(pr_two(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, off2);
    float2 y = pr_both(x);
    y = make_float2(pr_ex2(y.x), pr_ex2(y.y));
    ls[e & 1] = pr_add2(ls[e & 1], pr_two(y.x, y.y));
    pk[e] = tc_pack(y.x, y.y);
  }
}
__device__ __forceinline__ float pr_top(const uint32_t* s, int n) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < n; e += 2)
    mx[(e >> 1) & 3] = pr_max3(mx[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
  return pr_max(pr_max(mx[0], mx[1]), pr_max(mx[2], mx[3]));
}
constexpr float kPrScale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)

// The two warps of a row quadrant meet at a named barrier. A warp whose wait
// for the tensor core gave up still comes, and both leave together: the barrier
// itself tells both whether either gave up. (Read from a word in shared memory
// behind the barrier, the answers could differ, and the warp that stayed would
// wait at the barrier for good.)
struct PrPair {
  int id;                 // barrier 1 .. 8
  volatile float* mine;   // this thread's slot, the other thread's
  volatile float* other;
};
// Clears ok of both warps if either comes without it.
__device__ __forceinline__ void pr_meet(const PrPair& pr, bool& ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n barrier.cta.red.and.pred p, %1, 64, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(all)
      : "r"(pr.id), "r"((uint32_t)ok)
      : "memory");
  ok = all != 0;
}
// The larger of the two threads' values. The slots are free again once both
// warps have handed over P, before the next S.
__device__ __forceinline__ float pr_join(float x, const PrPair& pr, bool& ok) {
  *pr.mine = x;
  pr_meet(pr, ok);
  return pr_max(x, *pr.other);
}

// 64 columns of a block that every row sees whole: S out of tensor memory, P
// into it, m_ref, l and this half of O brought along. The lower 32 columns are
// read a second time for the exponentials: keeping all 64 over the exchange of
// the maxima costs the 104 registers some spills (492 against 463 us for a
// causal prompt of 8192 tokens).
__device__ __forceinline__ void pr_softmax_whole(PrRow& row, uint32_t t_s, uint32_t t_o, bool first, const PrPair& pr,
                                                 bool& ok) {
  uint32_t a[32], b[32], pk[16];
  pr_ld32(t_s, b);
  pr_ld32(t_s + 32, a);
  pr_ld_wait(b);
  pr_ld_wait(a);
  const float top = pr_join(pr_max(pr_top(b, 32), pr_top(a, 32)), pr, ok);
  if (!ok) return;
  pr_follow(row, top * kPrScale, t_o, first);
  const float off = row.m_ref == -INFINITY ? 0.0f : -row.m_ref;
  const uint64_t c2 = pr_two(kPrScale, kPrScale), off2 = pr_two(off, off);
  uint64_t ls[2] = {0, 0};
  pr_probs(a, pk, c2, off2, ls);
  pr_ld32(t_s, a);
  pr_st16(t_s + kPrP + 16, pk);
  pr_ld_wait(a);
  pr_probs(a, pk, c2, off2, ls);
  pr_st16(t_s + kPrP, pk);
  const float2 y = pr_both(pr_add2(ls[0], ls[1]));
  row.l += y.x + y.y;
}

// The same under the rows' masks, for those of the half's two 32-column
// chunks (c0, c0 + 1) that lie in [ca, cb). bad: the block's pages outside the
// pool.
__device__ __forceinline__ void pr_softmax_part(PrRow& row, uint32_t t_s, uint32_t t_o, int t0, int c0, int ca, int cb,
                                                bool first, unsigned bad, int log2bs, const PrPair& pr, bool& ok) {
  uint32_t s[32], ms[2];
  float mx = -INFINITY;
  auto hide = [&](int q) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((ms[q] >> e) & 1u)) s[e] = 0xFF800000u;  // -inf
  };
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int ch = c0 + q;
    if (ch < ca || ch >= cb) continue;
    ms[q] = pr_mask(row.v, t0, ch);
    if (bad)
      for (int e = 0; e < 32; ++e)
        if ((bad >> min((ch * 32 + e) >> log2bs, 31)) & 1u) ms[q] &= ~(1u << e);
    pr_ld32(t_s + q * 32, s);
    pr_ld_wait(s);
    hide(q);
    mx = pr_max(mx, pr_top(s, 32));
  }
  const float top = pr_join(mx, pr, ok);
  if (!ok) return;
  pr_follow(row, top * kPrScale, t_o, first);
  const float off = row.m_ref == -INFINITY ? 0.0f : -row.m_ref;
  const uint64_t c2 = pr_two(kPrScale, kPrScale), off2 = pr_two(off, off);
  uint64_t ls[2] = {0, 0};
#pragma unroll
  for (int q = 1; q >= 0; --q) {  // the upper chunk first: P takes its place
    const int ch = c0 + q;
    if (ch < ca || ch >= cb) continue;
    uint32_t pk[16];
    pr_ld32(t_s + q * 32, s);
    pr_ld_wait(s);
    hide(q);
    pr_probs(s, pk, c2, off2, ls);
    pr_st16(t_s + kPrP + q * 16, pk);
  }
  const float2 y = pr_both(pr_add2(ls[0], ls[1]));
  row.l += y.x + y.y;
}

template <int TERMS>
__global__ void __launch_bounds__(kPrThreads, 1) span_prompt_kernel(const __grid_constant__ PromptParams p) {
  using SM = PrSmem<TERMS>;
  constexpr int kStages = SM::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ring = smem + SM::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);  // [kStages]
  uint64_t* empty = full + kStages;                                // [kStages]
  uint64_t* bar_s = empty + kStages;  // [2] S of a tile is ready
  uint64_t* bar_p = bar_s + 2;        // [2] P is in tensor memory
  uint64_t* bar_o = bar_p + 2;        // [2] an item's O is complete
  uint64_t* bar_q = bar_o + 2;        // [2] an item's Q is staged
  uint64_t* bar_f = bar_q + 2;        // [2] an item's Q is no longer read
  uint32_t* tbase_s = reinterpret_cast<uint32_t*>(bar_f + 2);
  double* turns = reinterpret_cast<double*>(smem + SM::kTurns);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.s.group, hq = p.s.n_kv_heads * G, tt = pr_tokens(G);
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles would not be where TMA puts them
    if (tid == 0) flag_status(FASA_ERR_CUDA);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, 8);
      mbar_init(bar_o + i, 1);
      mbar_init(bar_q + i, TERMS == 1 ? 1 : 8);
      mbar_init(bar_f + i, 1);
    }
    fence_mbar_init();
  }
  if (warp == 16) tc_alloc(tbase_s, 512);
  if (tid == 544) {  // the loader
    prefetch_tensor_map(&p.map_k);
    prefetch_tensor_map(&p.map_v);
    if (TERMS == 1) prefetch_tensor_map(&p.map_q);
  }
  if (TERMS == 2) span_stage_turns<kPrThreads>(p.s, turns);
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tbase_s;
  // tensor memory columns: S_A (and P_A) 0, S_B 128, O_A 256, O_B 384

  if (warp < 16) {
    // ----------------------------------- softmax: half of a tile's columns
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int sub = warp >> 3, half = (warp >> 2) & 1, r = tid & 127;  // row of the tile = TMEM lane
    const int rt = r / G, rh = r - rt * G;                             // its token and head
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tbase + sub * 128 + half * 64 + lanes, t_o = tbase + 256 + sub * 128 + half * 64 + lanes;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.s.out);
    float* pair = reinterpret_cast<float*>(smem + SM::kPair) + sub * 256;
    const PrPair pr{1 + sub * 4 + (warp & 3), pair + half * 128 + r, pair + (half ^ 1) * 128 + r};
    bool ok = true;  // of this warp; one whose bounded wait gave up goes on to the next meeting
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = pr_wait(bar, parity); };
    auto part_of = [&](const PrItem& w) {
      return p.part + (((int64_t)(w.b * p.s.n_kv_heads + w.g) * p.tiles_max + w.tile) * p.splits + w.split) * kPrPart;
    };
    auto has_row = [&](const PrItem& w) { return rt < tt && sub * tt + rt < w.n_tok; };
    auto out_row = [&](const PrItem& w) {  // row of out [B n_q Hq][128]
      return ((int64_t)w.b * p.s.n_q + w.j0 + sub * tt + rt) * hq + w.g * G + rh;
    };
    PrSeq sq;
    sq.b = -1;
    // the next item with blocks, from `it` on; items without get their zeros
    // on the way
    auto next = [&](int& it, PrItem& w) -> bool {
      for (;; ++it) {
        w = pr_item(p, it, sq);
        if (w.b < 0) return false;
        if (!w.valid) continue;
        if (w.i0 < w.i1) return true;
        if (!has_row(w)) continue;
        if (p.splits > 1) {
          float* pp = part_of(w);
          pp[sub * 128 + r] = -INFINITY;
          pp[kPrRows + sub * 128 + r] = 0.0f;
        } else {
          uint4* o = reinterpret_cast<uint4*>(out + out_row(w) * kD) + half * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
        }
      }
    };
    // An item's Q rows of this tile, rotated, as two bf16 terms: 8 lanes take a
    // token, each the chunks ch and ch + 8 (dims i and i + 64 of 8 FCs), so
    // that an angle serves the G heads. Rows past the item's are left: what S
    // holds there is masked.
    auto stage_q = [&](const PrItem& w) {
      unsigned char* qs = smem + sub * TERMS * kPrTile;
      const int ch = lane & 7, n_t = min(tt, w.n_tok - sub * tt);
      const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.s.q) +
                                  (((int64_t)w.b * p.s.n_q + w.j0 + sub * tt) * hq + w.g * G) * kD;
      for (int jt = (warp & 7) * 4 + (lane >> 3); jt < n_t; jt += 32) {
        float cs[8], sn[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) span_angle(turns[ch * 8 + e], w.pos0 + w.j0 + sub * tt + jt, cs + e, sn + e);
        const uint4* src = reinterpret_cast<const uint4*>(base + (int64_t)jt * hq * kD);
#pragma unroll 2
        for (int h = 0; h < G; ++h) {
          const int rr = jt * G + h;
          float x[8], y[8], t8[8];
          unpack16(__ldg(src + h * 16 + ch), x, __nv_bfloat16());
          unpack16(__ldg(src + h * 16 + ch + 8), y, __nv_bfloat16());
          uint4 hi, lo;
#pragma unroll
          for (int e = 0; e < 8; ++e) t8[e] = x[e] * cs[e] - y[e] * sn[e];
          tc_split8(t8, hi, lo);
          *reinterpret_cast<uint4*>(qs + tc_sw(rr, ch, 128)) = hi;
          *reinterpret_cast<uint4*>(qs + kPrTile + tc_sw(rr, ch, 128)) = lo;
#pragma unroll
          for (int e = 0; e < 8; ++e) t8[e] = y[e] * cs[e] + x[e] * sn[e];
          tc_split8(t8, hi, lo);
          *reinterpret_cast<uint4*>(qs + tc_sw(rr, ch + 8, 128)) = hi;
          *reinterpret_cast<uint4*>(qs + kPrTile + tc_sw(rr, ch + 8, 128)) = lo;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) pr_arrive(bar_q + sub);
    };
    uint32_t n_s = 0, n_o = 0;  // barrier phases used
    int it = 0;
    PrItem w;
    bool more = next(it, w);
    if (TERMS == 2 && more && sub * tt < w.n_tok) stage_q(w);
    const int n_pg = p.s.pm.table ? max(1, kPrBlock >> p.s.pm.log2bs) : 0;
    while (more && ok) {
      const bool mine = has_row(w), active = sub * tt < w.n_tok;
      PrRow row;
      row.m_ref = -INFINITY;
      row.l = 0.0f;
      if (active) {
        row.v = span_of(w.L, mine ? w.pos0 + w.j0 + sub * tt + rt : -1, p.s.window, p.s.n_sink);
        // blocks [f0, f1) are whole to every row of the tile
        const int64_t pa = w.pos0 + w.j0 + sub * tt;
        const Span first = span_of(w.L, pa, p.s.window, p.s.n_sink);
        const Span last = span_of(w.L, pa + min(tt, w.n_tok - sub * tt) - 1, p.s.window, p.s.n_sink);
        const int f0 = w.u.na + max(0, (last.lo + kPrBlock - 1) / kPrBlock - w.u.first);
        const int f1 = w.u.na + first.hi / kPrBlock - w.u.first;
        for (int i = w.i0; i < w.i1; ++i) {
          unsigned bad = 0;  // the block's pages outside the pool
          if (n_pg) {
            const int t = w.u.unit(i) * kPrBlock + (lane << p.s.pm.log2bs);
            bad = __ballot_sync(0xFFFFFFFFu,
                                lane < n_pg && t < w.all.hi &&
                                    (unsigned)__ldg(p.s.pm.table + (int64_t)w.b * p.s.pm.max_blocks +
                                                    (t >> p.s.pm.log2bs)) >= (unsigned)p.s.pm.n_pages);
          }
          wait(bar_s + sub, n_s++ & 1);
          tc_fence_after();
          if (i >= f0 && i < f1 && !bad) {
            pr_softmax_whole(row, t_s, t_o, i == w.i0, pr, ok);
          } else {
            const int t0 = w.u.unit(i) * kPrBlock;
            int ca, cb;
            pr_chunks(w.all, t0, ca, cb);
            pr_softmax_part(row, t_s, t_o, t0, half * 2, ca, cb, i == w.i0, bad, p.s.pm.log2bs, pr, ok);
          }
          if (!ok) break;
          pr_stored(bar_p + sub, lane);
        }
        if (!ok) break;
      }
      const int64_t at = mine ? out_row(w) : -1;
      float* pp = p.splits > 1 ? part_of(w) : nullptr;
      ++it;
      more = next(it, w);
      if (TERMS == 2 && more && sub * tt < w.n_tok) stage_q(w);  // the last S is done with the old ones
      if (!active) continue;
      wait(bar_o + sub, n_o++ & 1);
      tc_fence_after();
      // the row's sum, once both threads are past their last exchange
      *pr.mine = row.l;
      pr_meet(pr, ok);
      const float l = row.l + *pr.other;
      pr_meet(pr, ok);  // the slots are free again
      if (!ok) break;
      if (p.splits == 1) {
        // rows of the lane's group of four: lane k stores the k-th 16 bytes
        // of each 64, so that a group's store covers 64 bytes of a row
        int64_t at4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) at4[k] = __shfl_sync(0xFFFFFFFFu, at, (lane & ~3) + k);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t o[32], z[16];
          pr_ld32(t_o + q * 32, o);
          pr_ld_wait(o);
#pragma unroll
          for (int d = 0; d < 16; ++d) {
            const float x0 = __uint_as_float(o[2 * d]) * inv, x1 = __uint_as_float(o[2 * d + 1]) * inv;
            z[d] = l == 0.0f ? 0u : tc_pack(x0, x1);
          }
          pr_transpose4(z, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (at4[k] >= 0)
              reinterpret_cast<uint4*>(out + at4[k] * kD)[half * 8 + q * 4 + (lane & 3)] =
                  make_uint4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]);
        }
      } else {
        const int rr = sub * 128 + r;
        if (mine && half == 0) {
          pp[rr] = row.m_ref;
          pp[kPrRows + rr] = l;
        }
        uint4* po = reinterpret_cast<uint4*>(pp + 2 * kPrRows + (int64_t)rr * kD) + half * 16;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t o[32];
          pr_ld32(t_o + q * 32, o);
          pr_ld_wait(o);
          if (mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e) po[q * 8 + e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      tc_fence_before();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (warp == 16) {
    // ----------------------------------------------------- the products
    uint32_t kv = 0, n_p[2] = {0, 0}, n_q[2] = {0, 0};
    bool ok = true;
    PrSeq sq;
    sq.b = -1;
    // low descriptor words of Q of tile A, of a block as K (rows of chunk 0),
    // as V (64-dim halves 16 KB apart)
    const uint32_t tb = pr_uni(tbase);
    const uint32_t q_lo = pr_uni((smem_u32(smem) >> 4) | (1u << 16)), k_lo = pr_uni((smem_u32(ring) >> 4) | (1u << 16)),
                   v_lo = pr_uni((smem_u32(ring) >> 4) | ((16384u >> 4) << 16));
    auto wait_full = [&](uint32_t n) { return pr_wait(full + n % kStages, (n / kStages) & 1); };
    // S of tile `sub` = its queries times chunks [ca, cb) of the block in
    // stage `st`; after an item's last one its queries are free
    auto issue_s = [&](int sub, uint32_t st, int ca, int cb, bool last, bool release) {
      const uint32_t d = pr_uni(tb + sub * 128 + ca * 32), q = pr_uni(q_lo + sub * (TERMS * kPrTile >> 4)),
                     k = pr_uni(k_lo + st * (kPrTile >> 4) + ca * (4096 >> 4)), id = pr_uni(pr_idesc(32 * (cb - ca)));
      if (pr_elect()) {
        pr_issue_s<TERMS>(d, q, k, id);
        tc_commit(bar_s + sub);
        if (last) tc_commit(bar_f + sub);
        if (release) tc_commit(empty + st);
      }
      __syncwarp();
    };
    for (int it = 0; ok; ++it) {
      const PrItem w = pr_item(p, it, sq);
      if (w.b < 0) break;
      if (!w.valid || w.i0 >= w.i1) continue;
      const int subs = w.n_tok > tt ? 2 : 1;
      int ca, cb;
      pr_chunks(w.all, w.u.unit(w.i0) * kPrBlock, ca, cb);
      if (!(ok = wait_full(kv))) break;
      for (int sub = 0; sub < subs && ok; ++sub) {
        if (!(ok = pr_wait(bar_q + sub, n_q[sub]++ & 1))) break;
        tc_fence_after();
        issue_s(sub, kv % kStages, ca, cb, w.i1 - w.i0 == 1, sub == subs - 1);
      }
      ++kv;
      for (int i = w.i0; i < w.i1 && ok; ++i) {
        const uint32_t v_n = kv++;
        const bool last = i + 1 == w.i1;
        const uint32_t k_n = kv;
        if (!last) ++kv;
        if (!(ok = wait_full(v_n))) break;
        const uint32_t vs_st = v_n % kStages;
        // rows of the block's chunks that nobody sees: zeros
        const int t0 = w.u.unit(i) * kPrBlock;
        if (t0 + kPrBlock > w.all.hi || (t0 < w.all.lo && t0 + kPrBlock > w.all.s)) {
          unsigned char* vs = ring + vs_st * kPrTile;
          auto zero = [&](int ra, int rb) {  // rows ra .. rb - 1
            for (int e = ra * 8 + lane; e < rb * 8; e += 32) {
              *reinterpret_cast<uint4*>(vs + e * 16) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(vs + 16384 + e * 16) = make_uint4(0, 0, 0, 0);
            }
          };
          zero(max(w.all.s - t0, ca * 32), min(w.all.lo - t0, cb * 32));
          zero(max(w.all.hi - t0, ca * 32), cb * 32);
          fence_proxy_async_smem();
          __syncwarp();
        }
        int na = 0, nb = 1;  // the next block's chunks
        if (!last) pr_chunks(w.all, w.u.unit(i + 1) * kPrBlock, na, nb);
        for (int sub = 0; sub < subs && ok; ++sub) {
          const uint32_t d = pr_uni(tb + 256 + sub * 128), pa = pr_uni(tb + sub * 128 + kPrP),
                         v = pr_uni(v_lo + vs_st * (kPrTile >> 4));
          if (!(ok = pr_wait(bar_p + sub, n_p[sub]++ & 1))) break;
          tc_fence_after();
          if (pr_elect()) {
            if (cb - ca < 4)
              pr_issue_part(d, pa, v, ca, cb, i > w.i0);
            else if (i > w.i0)
              pr_issue_o<true>(d, pa, v);
            else
              pr_issue_o<false>(d, pa, v);
            if (last) tc_commit(bar_o + sub);
            if (sub == subs - 1) tc_commit(empty + vs_st);
          }
          __syncwarp();
          if (!last) {
            if (sub == 0 && !(ok = wait_full(k_n))) break;
            issue_s(sub, k_n % kStages, na, nb, i + 2 == w.i1, sub == subs - 1);
          }
        }
        ca = na;
        cb = nb;
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------------- the loads
    uint32_t n = 0, n_f[2] = {0, 0};
    bool ok = true;
    PrSeq sq;
    sq.b = -1;
    const int boxes = kPrBlock / p.box_rows;
    auto load = [&](const PrItem& w, int i, bool is_v) {
      const uint32_t st = n % kStages;
      if (n >= (uint32_t)kStages && !pr_wait(empty + st, (n / kStages - 1) & 1)) {
        ok = false;
        return;
      }
      if (lane == 0) mbar_arrive_expect_tx(full + st, kPrTile);
      __syncwarp();
      if (lane < 2 * boxes) {
        const int box = lane >> 1, half = lane & 1;
        const int t = w.u.unit(i) * kPrBlock + box * p.box_rows;
        int row = p.n_rows;  // out of range: zeros
        if (t < w.all.hi && (t + p.box_rows > w.all.lo || t < w.all.s)) {
          if (p.s.pm.table) {
            row = paged_row(p.s.pm, w.b, w.g, t);
            if (row < 0) row = p.n_rows;
          } else {
            row = (int)((int64_t)(w.b * p.s.n_kv_heads + w.g) * p.s.max_len + t);
          }
        }
        pr_tma(is_v ? &p.map_v : &p.map_k, ring + st * kPrTile + half * 16384 + box * p.box_rows * 128, full + st,
               half * 64, row);
      }
      ++n;
    };
    for (int it = 0; ok; ++it) {
      const PrItem w = pr_item(p, it, sq);
      if (w.b < 0) break;
      if (!w.valid) continue;
      for (int i = w.i0; i < w.i1 && ok; ++i) {
        load(w, i, false);
        if (ok) load(w, i, true);
        if (TERMS == 1 && i == w.i0) {  // behind the first block, which does not wait for the queries' place
          for (int sub = 0; sub < 2 && ok && sub * tt < w.n_tok; ++sub) {
            if (n_f[sub] > 0 && !pr_wait(bar_f + sub, (n_f[sub] - 1) & 1)) {
              ok = false;
              break;
            }
            ++n_f[sub];
            if (lane == 0) {
              mbar_arrive_expect_tx(bar_q + sub, (uint32_t)(tt * G) * 256u);
              for (int half = 0; half < 2; ++half)
                pr_tma3(&p.map_q, smem + sub * kPrTile + half * 16384, bar_q + sub, half * 64, w.g * G,
                        w.b * p.s.n_q + w.j0 + sub * tt);
            }
            __syncwarp();
          }
        }
      }
    }
    // every copy has landed before the block ends (the products wait for
    // them all unless something went wrong)
    for (uint32_t k = n > (uint32_t)kStages ? n - kStages : 0; k < n; ++k)
      mbar_wait(full + k % kStages, (k / kStages) & 1);
    if (TERMS == 1)
      for (int sub = 0; sub < 2; ++sub)
        if (n_f[sub] > 0) mbar_wait(bar_q + sub, (n_f[sub] - 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) tc_dealloc(tbase, 512);
  grid_dependents_launch();
}

// Joins the splits of every query row: one warp per row.
__global__ void __launch_bounds__(128) span_prompt_merge_kernel(const __grid_constant__ PromptParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int G = p.s.group, hq = p.s.n_kv_heads * G;
  const int64_t m64 = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);  // token * G + head
  const int row = blockIdx.y, b = row / p.s.n_kv_heads, g = row % p.s.n_kv_heads;
  if (m64 >= (int64_t)span_qlen(p.s, b) * G) return;
  const int m = (int)m64, tt = pr_tokens(G), j = m / G;
  const float* base = p.part + ((int64_t)row * p.tiles_max + j / (2 * tt)) * p.splits * kPrPart;
  const int jj = j % (2 * tt), rr = jj / tt * 128 + jj % tt * G + m % G;
  float ms = -INFINITY, ls = 0.0f;
  if (lane < p.splits) {
    ms = __ldcg(base + lane * kPrPart + rr);
    ls = __ldcg(base + lane * kPrPart + kPrRows + rr);
  }
  float M = ms;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  const float f = ms == -INFINITY ? 0.0f : exp2f(ms - M);
  float L = f * ls;
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < p.splits; ++s) {
    const float fs = __shfl_sync(0xFFFFFFFFu, f, s);
    if (fs == 0.0f) continue;  // an empty split has no sums
    const float4 x = __ldcg(reinterpret_cast<const float4*>(base + s * kPrPart + 2 * kPrRows + (int64_t)rr * kD) + lane);
    acc.x = __fmaf_rn(fs, x.x, acc.x);
    acc.y = __fmaf_rn(fs, x.y, acc.y);
    acc.z = __fmaf_rn(fs, x.z, acc.z);
    acc.w = __fmaf_rn(fs, x.w, acc.w);
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.s.out) +
                                        (((int64_t)b * p.s.n_q + m / G) * hq + g * G + m % G) * kD);
  out[lane] = make_uint2(tc_pack(acc.x * inv, acc.y * inv), tc_pack(acc.z * inv, acc.w * inv));
}

}  // namespace fasa
