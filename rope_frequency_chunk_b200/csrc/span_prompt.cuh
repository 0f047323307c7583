// Span attention of prompts on the tensor cores (bf16 caches in device
// memory): Q K^T and P V with tcgen05.mma, accumulators and probabilities in
// tensor memory, K and V blocks by TMA.
//
// The query rows of KV head g of a sequence are its tokens' G heads, packed:
// row m is token m / G, head m % G, so the G heads of a token share the K and
// V blocks they read. One work item is 256 rows (two row tiles of 128, A and
// B) of one (b, g) over the blocks of 128 slots that any of its rows sees.
// The CTAs (one per SM) walk the items, the longest first.
//
// Roles in a CTA of 12 warps (the softmax ones take registers from the rest:
// 216 + 216 + 72 = 3 * 168):
//  - warps 0-3 and 4-7: the softmax of row tile A and B, one row per thread:
//    S row from tensor memory, mask, running maximum and sum, P as bf16 into
//    the tensor memory of S; they also stage Q and write the output;
//  - warp 8: issues the products. Per block: O_A += P_A V, S_A' = Q_A K',
//    O_B += P_B V, S_B' = Q_B K' (K' the next block): while one tile's
//    softmax runs, the tensor core works for the other;
//  - warp 9: K and V blocks into a ring of 32 KB stages (10 and 11: none).
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

constexpr int kPrThreads = 384;  // three warpgroups; 168 registers a thread at launch
constexpr int kPrRows = 256;             // query rows per item
constexpr int kPrBlock = 128;            // slots per block
constexpr uint32_t kPrTile = 32768;      // bytes of a 128 x 128 bf16 tile pair
constexpr int kPrMaxSplits = 32;

struct PromptParams {
  CUtensorMap map_k, map_v;  // [rows][128] bf16, boxes of box_rows x 64, 128-byte swizzle
  SpanParams s;
  int32_t n_items;           // tiles_max * B * Hkv * splits
  int32_t tiles_max;         // items of a (b, g) row at n_q queries
  int32_t splits;            // parts that an item's blocks are cut into
  int32_t box_rows;          // rows of a TMA box
  int32_t n_rows;            // rows of the K (and V) tensor
  float* part;               // [B * Hkv * tiles_max * splits][256][2 + 128]: m, l planes, then o
};

// Bytes of a split's partial: m[256], l[256], o[256][128].
constexpr int64_t kPrPart = kPrRows * (2 + kD);

template <int TERMS>
struct PrSmem {
  static constexpr int kStages = TERMS == 1 ? 5 : 3;
  static constexpr uint32_t kQ = 2 * TERMS * kPrTile;  // tile A's terms, tile B's terms
  static constexpr uint32_t kBars = kQ + kStages * kPrTile;
  static constexpr uint32_t kBytes = kBars + 256 + 1024;  // barriers; alignment to 1024
};

// One item as every role sees it.
struct PrItem {
  bool valid;
  int b, g, row0, n_rows, L, tile, split;
  int64_t pos0;      // position of the sequence's first query
  Span all;          // slots that some row of the item sees
  SpanUnits u;
  int i0, i1;        // this split's blocks
};

__device__ __forceinline__ PrItem pr_item(const PromptParams& p, int it) {
  PrItem w;
  w.valid = false;
  const int grid = gridDim.x, c = blockIdx.x;
  const int64_t n64 = (int64_t)it * grid + ((it & 1) ? grid - 1 - c : c);
  if (n64 >= p.n_items) {
    w.b = -1;  // past the end
    return w;
  }
  const int n = (int)n64;
  const int rows = p.s.batch * p.s.n_kv_heads, G = p.s.group;
  w.split = n % p.splits;
  const int r = (n / p.splits) % rows, k = n / (p.splits * rows);
  w.b = r / p.s.n_kv_heads;
  w.g = r % p.s.n_kv_heads;
  w.L = span_len(p.s, w.b);
  const int nq = span_qlen(p.s, w.b);
  w.pos0 = span_pos0(p.s, w.b, w.L, nq);
  const int m_all = nq * G, tiles = (m_all + kPrRows - 1) / kPrRows;
  if (k >= tiles) return w;
  w.valid = true;
  w.tile = tiles - 1 - k;
  w.row0 = w.tile * kPrRows;
  w.n_rows = min(kPrRows, m_all - w.row0);
  const int64_t pa = w.pos0 + w.row0 / G, pb = w.pos0 + (w.row0 + w.n_rows - 1) / G;
  // the union over positions pa .. pb: the last position's end, the first
  // one's window; its sinks are slots below lo, the rest is inside anyway
  const Span first = span_of(w.L, max(pa, (int64_t)0), p.s.window, p.s.n_sink);
  const Span last = span_of(w.L, pb, p.s.window, p.s.n_sink);
  w.all.hi = last.hi;
  w.all.lo = min(first.lo, last.hi);
  w.all.s = min(last.s, w.all.lo);
  w.u = span_units(w.all, kPrBlock);
  w.i0 = (int)((int64_t)w.u.n * w.split / p.splits);
  w.i1 = (int)((int64_t)w.u.n * (w.split + 1) / p.splits);
  return w;
}

__device__ __forceinline__ void pr_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
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
__device__ __forceinline__ void pr_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void pr_st32(uint32_t taddr, const uint32_t* r) {
  pr_st16(taddr, r);
  pr_st16(taddr + 16, r + 16);
}
__device__ __forceinline__ void pr_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void pr_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float pr_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

template <int TERMS>
__global__ void __launch_bounds__(kPrThreads, 1) span_prompt_kernel(const __grid_constant__ PromptParams p) {
  using SM = PrSmem<TERMS>;
  constexpr int kStages = SM::kStages;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* ring = smem + SM::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);  // [kStages]
  uint64_t* empty = full + kStages;                                // [kStages]
  uint64_t* bar_s = empty + kStages;  // [2] S of a tile is ready
  uint64_t* bar_p = bar_s + 2;        // [2] P is in tensor memory
  uint64_t* bar_o = bar_p + 2;        // [2] an item's O is complete
  uint64_t* bar_q = bar_o + 2;        // [2] an item's Q is staged
  uint32_t* tbase_s = reinterpret_cast<uint32_t*>(bar_q + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.s.group, hq = p.s.n_kv_heads * G;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, 128);
      mbar_init(bar_o + i, 1);
      mbar_init(bar_q + i, 128);
    }
    fence_mbar_init();
  }
  if (warp == 8) tc_alloc(tbase_s, 512);
  __shared__ double turns[kNFC];
  if (TERMS == 2) span_stage_turns<kPrThreads>(p.s, turns);
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tbase_s;
  // tensor memory columns: S_A (and P_A) 0, S_B 128, O_A 256, O_B 384

  if (warp < 8) {
    // ------------------------------------------------ softmax of one tile
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int sub = warp >> 2, r = tid & 127;  // row of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tbase + sub * 128 + lanes, t_o = tbase + 256 + sub * 128 + lanes;
    unsigned char* qs = smem + sub * TERMS * kPrTile;
    const float c = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
    const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(p.s.q);
    // An item's Q rows into shared memory: 8 lanes take a token's G rows, each
    // the chunks ch and ch + 8 (dims i and i + 64 of 8 FCs), so that an angle
    // serves the G heads. Rows past the item's are left: what S holds there is
    // masked.
    auto stage_q = [&](const PrItem& w) {
      const int ch = lane & 7;
      const int m0 = w.row0 + sub * 128, m1 = min(w.row0 + w.n_rows, m0 + 128);
      for (int j = m0 / G + (warp & 3) * 4 + (lane >> 3); j * G < m1; j += 16) {
        float cs[8], sn[8];
        if (TERMS == 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) span_angle(turns[ch * 8 + e], w.pos0 + j, cs + e, sn + e);
        }
        const uint4* src = reinterpret_cast<const uint4*>(qg + (((int64_t)w.b * p.s.n_q + j) * hq + w.g * G) * kD);
        const int h0 = max(m0 - j * G, 0), h1 = min(G, m1 - j * G);
#pragma unroll 4
        for (int h = h0; h < h1; ++h) {
          const int rr = j * G + h - m0;
          uint4 a = __ldg(src + h * 16 + ch), b2 = __ldg(src + h * 16 + ch + 8);
          if (TERMS == 2) {
            float x[8], y[8], xr[8], yr[8];
            unpack16(a, x, __nv_bfloat16());
            unpack16(b2, y, __nv_bfloat16());
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              xr[e] = x[e] * cs[e] - y[e] * sn[e];
              yr[e] = y[e] * cs[e] + x[e] * sn[e];
            }
            uint4 al, bl;
            tc_split8(xr, a, al);
            tc_split8(yr, b2, bl);
            *reinterpret_cast<uint4*>(qs + kPrTile + tc_sw(rr, ch, 128)) = al;
            *reinterpret_cast<uint4*>(qs + kPrTile + tc_sw(rr, ch + 8, 128)) = bl;
          }
          *reinterpret_cast<uint4*>(qs + tc_sw(rr, ch, 128)) = a;
          *reinterpret_cast<uint4*>(qs + tc_sw(rr, ch + 8, 128)) = b2;
        }
      }
      fence_proxy_async_smem();
      pr_arrive(bar_q + sub);
    };
    // the next item with blocks and rows for this tile, from `it` on; items
    // without blocks get their zeros on the way
    uint32_t n_s = 0, n_o = 0;  // barrier phases used
    auto next = [&](int& it, PrItem& w) -> bool {
      for (;; ++it) {
        w = pr_item(p, it);
        if (w.b < 0) return false;
        if (!w.valid) continue;
        const bool mine = sub * 128 + r < w.n_rows;
        if (w.i0 < w.i1) return true;
        if (p.splits > 1) {
          if (mine) {
            float* pp = p.part + (((int64_t)(w.b * p.s.n_kv_heads + w.g) * p.tiles_max + w.tile) * p.splits + w.split) *
                                     kPrPart;
            pp[sub * 128 + r] = -INFINITY;
            pp[kPrRows + sub * 128 + r] = 0.0f;
          }
        } else if (mine) {
          const int m = w.row0 + sub * 128 + r;
          uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.s.out) +
                                              (((int64_t)w.b * p.s.n_q + m / G) * hq + w.g * G + m % G) * kD);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = make_uint4(0, 0, 0, 0);
        }
      }
    };
    int it = 0;
    PrItem w;
    bool more = next(it, w), ok = true;
    // a tile B without rows takes no part in its item
    if (more && sub * 128 < w.n_rows) stage_q(w);
    while (more && ok) {
      const bool active = sub * 128 < w.n_rows;
      float m_ref = -INFINITY, l = 0.0f;
      const int m = w.row0 + sub * 128 + r;
      const bool mine = sub * 128 + r < w.n_rows;
      const Span v = span_of(w.L, mine ? w.pos0 + m / G : -1, p.s.window, p.s.n_sink);
      if (active) {
        // bad pages of the next block: bit i for its i-th page
        const int n_pg = p.s.pm.table ? max(1, kPrBlock >> p.s.pm.log2bs) : 0;
        auto bad_pages = [&](int i) -> unsigned {
          if (n_pg == 0 || i >= w.i1) return 0u;
          const int t = w.u.unit(i) * kPrBlock + (lane << p.s.pm.log2bs);
          bool bad = false;
          if (lane < n_pg && t < w.all.hi)
            bad = (unsigned)__ldg(p.s.pm.table + (int64_t)w.b * p.s.pm.max_blocks + (t >> p.s.pm.log2bs)) >=
                  (unsigned)p.s.pm.n_pages;
          return __ballot_sync(0xFFFFFFFFu, bad);
        };
        for (int i = w.i0; i < w.i1; ++i) {
          const int t0 = w.u.unit(i) * kPrBlock;
          const unsigned bad = bad_pages(i);
          if (!pr_wait(bar_s + sub, n_s & 1)) {
            ok = false;
            break;
          }
          ++n_s;
          tc_fence_after();
          uint32_t s[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) pr_ld32(t_s + q * 32, s + q * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q) pr_ld_wait(s + q * 32);
          const bool whole = t0 + kPrBlock <= v.hi && (t0 >= v.lo || t0 + kPrBlock <= v.s);
          if (__any_sync(0xFFFFFFFFu, !whole) || bad) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t ms = pr_mask(v, t0, q);
              if (bad) {
                for (int e = 0; e < 32; ++e)
                  if ((bad >> min((q * 32 + e) >> p.s.pm.log2bs, 31)) & 1u) ms &= ~(1u << e);
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((ms >> e) & 1u)) s[q * 32 + e] = 0xFF800000u;  // -inf
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
          const float m_blk = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const bool grow = m_blk > m_ref + 8.0f || (m_ref == -INFINITY && m_blk > -INFINITY);
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float m_new = grow ? m_blk : m_ref;
            const float f = m_ref == -INFINITY ? 0.0f : pr_ex2(m_ref - m_new);
            if (i > w.i0 && __any_sync(0xFFFFFFFFu, grow && m_ref > -INFINITY)) {
              const float fo = grow ? f : 1.0f;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                pr_ld32(t_o + q * 32, o);
                pr_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
                pr_st32(t_o + q * 32, o);
              }
            }
            if (grow) {
              l *= f;
              m_ref = m_new;
            }
          }
          const float off = m_ref == -INFINITY ? 0.0f : m_ref;
          float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float a = pr_ex2(__fmaf_rn(__uint_as_float(s[q * 32 + e]), c, -off));
              const float b2 = pr_ex2(__fmaf_rn(__uint_as_float(s[q * 32 + e + 1]), c, -off));
              ls[(e >> 1) & 1] += a;
              ls[2 + ((e >> 1) & 1)] += b2;
              pk[e >> 1] = tc_pack(a, b2);
            }
            pr_st16(t_s + q * 16, pk);
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          pr_st_wait();
          tc_fence_before();
          pr_arrive(bar_p + sub);
        }
      }
      if (!ok) break;
      // the next item's queries go in while this one's last product runs
      const PrItem done = w;
      ++it;
      more = next(it, w);
      if (more && sub * 128 < w.n_rows) stage_q(w);
      if (active) {
        if (!pr_wait(bar_o + sub, n_o & 1)) {
          ok = false;
          break;
        }
        ++n_o;
        tc_fence_after();
        if (p.splits == 1) {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          uint4* og = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.s.out) +
                                               (((int64_t)done.b * p.s.n_q + m / G) * hq + done.g * G + m % G) * kD);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            pr_ld32(t_o + q * 32, o);
            pr_ld_wait(o);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t z[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                  const float x0 = __uint_as_float(o[e * 8 + 2 * d]) * inv, x1 = __uint_as_float(o[e * 8 + 2 * d + 1]) * inv;
                  z[d] = l == 0.0f ? 0u : tc_pack(x0, x1);
                }
                og[q * 4 + e] = make_uint4(z[0], z[1], z[2], z[3]);
              }
            }
          }
        } else {
          float* pp = p.part + (((int64_t)(done.b * p.s.n_kv_heads + done.g) * p.tiles_max + done.tile) * p.splits +
                                done.split) * kPrPart;
          const int rr = sub * 128 + r;
          if (mine) {
            pp[rr] = m_ref;
            pp[kPrRows + rr] = l;
          }
          uint4* po = reinterpret_cast<uint4*>(pp + 2 * kPrRows + (int64_t)rr * kD);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
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
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  }
  if (warp == 8) {
    // ----------------------------------------------------- the products
    uint32_t kv = 0, n_p[2] = {0, 0}, n_q[2] = {0, 0};
    bool ok = true;
    const uint32_t q_addr = smem_u32(smem), r_addr = smem_u32(ring);
    auto wait_full = [&](uint32_t n) { return pr_wait(full + n % kStages, (n / kStages) & 1); };
    // S of tile `sub` = its queries times the block in stage `st`
    auto issue_s = [&](int sub, uint32_t st) {
      const uint32_t ks = r_addr + st * kPrTile, qa = q_addr + sub * TERMS * kPrTile;
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
#pragma unroll
        for (int k8 = 0; k8 < 8; ++k8) {
          const uint32_t o = (k8 >> 2) * 16384 + (k8 & 3) * 32;
          tc_mma(tbase + sub * 128, tc_desc(qa + t * kPrTile + o, 16, 1024), tc_desc(ks + o, 16, 1024), tc_idesc(0),
                 t + k8 > 0);
        }
      tc_commit(bar_s + sub);
    };
    for (int it = 0; ok; ++it) {
      const PrItem w = pr_item(p, it);
      if (w.b < 0) break;
      if (!w.valid || w.i0 >= w.i1) continue;
      const int subs = w.n_rows > 128 ? 2 : 1;
      for (int sub = 0; sub < subs && ok; ++sub) ok = pr_wait(bar_q + sub, n_q[sub]++ & 1);
      if (!ok || !(ok = wait_full(kv))) break;
      tc_fence_after();
      if (lane == 0) {
        for (int sub = 0; sub < subs; ++sub) issue_s(sub, kv % kStages);
        tc_commit(empty + kv % kStages);
      }
      ++kv;
      for (int i = w.i0; i < w.i1 && ok; ++i) {
        const uint32_t v_n = kv++;
        const bool last = i + 1 == w.i1;
        const uint32_t k_n = kv;
        if (!last) ++kv;
        if (!(ok = wait_full(v_n))) break;
        const uint32_t vs_st = v_n % kStages;
        // rows of the block that nobody sees: zeros
        const int t0 = w.u.unit(i) * kPrBlock;
        if (t0 + kPrBlock > w.all.hi || (t0 < w.all.lo && t0 + kPrBlock > w.all.s)) {
          unsigned char* vs = ring + vs_st * kPrTile;
          auto zero = [&](int ra, int rb) {  // rows ra .. rb - 1
            for (int e = max(ra, 0) * 8 + lane; e < min(rb, kPrBlock) * 8; e += 32) {
              *reinterpret_cast<uint4*>(vs + e * 16) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(vs + 16384 + e * 16) = make_uint4(0, 0, 0, 0);
            }
          };
          zero(w.all.s - t0, w.all.lo - t0);
          zero(w.all.hi - t0, kPrBlock);
          fence_proxy_async_smem();
          __syncwarp();
        }
        for (int sub = 0; sub < subs && ok; ++sub) {
          if (!(ok = pr_wait(bar_p + sub, n_p[sub]++ & 1))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t vs = r_addr + vs_st * kPrTile;
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8)
              pr_mma_ts(tbase + 256 + sub * 128, tbase + sub * 128 + k8 * 8, tc_desc(vs + k8 * 2048, 16384, 1024),
                        tc_idesc(1), i > w.i0 || k8 > 0);
            if (last) tc_commit(bar_o + sub);
            if (sub == subs - 1) tc_commit(empty + vs_st);
          }
          if (!last) {
            if (sub == 0 && !(ok = wait_full(k_n))) break;
            if (lane == 0) {
              issue_s(sub, k_n % kStages);
              if (sub == subs - 1) tc_commit(empty + k_n % kStages);
            }
          }
          __syncwarp();
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------- the loads
    uint32_t n = 0;
    bool ok = true;
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
      const PrItem w = pr_item(p, it);
      if (w.b < 0) break;
      if (!w.valid) continue;
      for (int i = w.i0; i < w.i1 && ok; ++i) {
        load(w, i, false);
        if (ok) load(w, i, true);
      }
    }
    // every copy has landed before the block ends (the products wait for
    // them all unless something went wrong)
    for (uint32_t k = n > (uint32_t)kStages ? n - kStages : 0; k < n; ++k)
      mbar_wait(full + k % kStages, (k / kStages) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tc_dealloc(tbase, 512);
  grid_dependents_launch();
}

// Joins the splits of every query row: one warp per row.
__global__ void __launch_bounds__(128) span_prompt_merge_kernel(const __grid_constant__ PromptParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int G = p.s.group, hq = p.s.n_kv_heads * G;
  const int64_t m64 = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);  // row of the (b, g)
  const int row = blockIdx.y, b = row / p.s.n_kv_heads, g = row % p.s.n_kv_heads;
  if (m64 >= (int64_t)span_qlen(p.s, b) * G) return;
  const int m = (int)m64;
  const float* base = p.part + ((int64_t)row * p.tiles_max + m / kPrRows) * p.splits * kPrPart;
  const int rr = m % kPrRows;
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
