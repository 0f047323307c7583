// Eviction from a cache by accumulated attention weight.
//
// Of a row's L slots, min(L, budget) stay: those of the first tokens
// (position < n_sink), those of the n_recent newest (position > cur_pos -
// n_recent), and of the others the ones with the largest weight, equal
// weights to the lower slot. The kept slots end up in 0 .. budget - 1: a kept
// slot below the budget stays where it is, and the i-th kept slot at or
// behind the budget moves into the i-th evicted slot before it (both lists
// ascending). Attention does not depend on the order of a row's slots, so
// closing the holes this way moves only the kept tail instead of shifting
// every row; sources (>= budget) and targets (< budget) never overlap, so the
// moves need no order among each other.
//
// One cluster of CTAs per (b, g) row. Each CTA keeps the order-preserving keys
// of its share of the slots in shared memory; three histogram passes (11 + 11
// + 10 bits, summed over the cluster through distributed shared memory) give
// the exact budget-th largest key; ballots turn the slots into bit words, one
// word per thread from then on; scans number the holes and the moves, and
// warps copy the moved rows, eight at a time with all their loads in flight.
// Bound by memory: 8 bytes a slot and the moved rows; small rows by the chain
// of barriers.
#pragma once

#include <cooperative_groups.h>

#include "fasa_device.cuh"

namespace fasa {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvMaxChunk = 32768;  // keys per CTA

struct EvictParams {
  void* k;
  void* v;
  void* sketch;
  const int32_t* seq_len;
  const int32_t* cur_pos;
  const float* mass;         // [rows][max_len]
  const int32_t* slot_pos;   // [rows][max_len]
  float* mass_out;
  int32_t* slot_pos_out;
  int32_t* len_out;          // [B]
  int32_t* moves;            // [rows][2][max_moves]: sources, targets
  int32_t* n_moves;          // [rows], where the moves are a launch of their own; else null
  int64_t max_len;
  int32_t max_seq_len;
  int32_t budget;
  int32_t n_sink;
  int32_t n_recent;
  int32_t n_kv_heads;
  int32_t max_moves;
  int32_t chunk;             // slots per CTA, a multiple of 32
  int32_t row16;             // 16-byte vectors of a K (and V) row
  int32_t sk16;              // of a sketch row, a power of two
  int32_t clusters;          // CTAs per row
  PageMap pm;
};

constexpr uint32_t kEvHeld = 0xFFFFFFFFu;

// Moves of one warp at a time: their rows are all in flight together.
constexpr int kEvBatch = 8;

// Moves m0 .. m0 + kEvBatch - 1 of a row by one warp.
__device__ __forceinline__ void evict_batch(const EvictParams& p, int row, uint32_t m0, uint32_t n_moves, int lane) {
  const int b = row / p.n_kv_heads, g = row % p.n_kv_heads;
  const int32_t* src = p.moves + (int64_t)row * 2 * p.max_moves;
  const int32_t* dst = src + p.max_moves;
  const float* mass = p.mass + (int64_t)row * p.max_len;
  const int32_t* pos = p.slot_pos + (int64_t)row * p.max_len;
  // lane i < kEvBatch: the rows of move m0 + i. A move from or to a page outside
  // the pool (flagged) is left out whole: its target slot keeps its own row,
  // and with it its own weight and position.
  int mine_s = -1, mine_d = -1;
  if (lane < kEvBatch && m0 + lane < n_moves) {
    const int ts = __ldcg(src + m0 + lane), td = __ldcg(dst + m0 + lane);
    float m = mass[ts];
    int x = pos[ts];
    mine_s = p.pm.table ? paged_row(p.pm, b, g, ts) : (int)(row * p.max_len + ts);
    mine_d = p.pm.table ? paged_row(p.pm, b, g, td) : (int)(row * p.max_len + td);
    if (mine_s < 0 || mine_d < 0) {
      mine_s = -1;
      m = mass[td];
      x = pos[td];
    }
    p.mass_out[(int64_t)row * p.max_len + td] = m;
    p.slot_pos_out[(int64_t)row * p.max_len + td] = x;
  }
  // the sketch rows' vectors, a power of two each: the first 32 of the batch
  // are requested ahead of K and V
  uint4* sk = static_cast<uint4*>(p.sketch);
  const int n_sk = kEvBatch * p.sk16;
  auto sk_at = [&](int e0, int& rs, int& rd) {
    const int i = min((e0 + lane) / p.sk16, kEvBatch - 1);
    rs = __shfl_sync(0xFFFFFFFFu, mine_s, i);
    rd = __shfl_sync(0xFFFFFFFFu, mine_d, i);
    if (e0 + lane >= n_sk) rs = -1;
  };
  int rs0, rd0;
  sk_at(0, rs0, rd0);
  const int c0 = lane % p.sk16;
  uint4 s0 = make_uint4(0, 0, 0, 0);
  if (rs0 >= 0) s0 = __ldcs(sk + (int64_t)rs0 * p.sk16 + c0);
  // K and V: a bf16 row is half a warp's 16-byte vectors, a float32 row a
  // whole warp's
  const bool half = p.row16 == 16;
  for (int r = 0; r < (half ? 1 : 2); ++r) {
    uint4* base = static_cast<uint4*>((half ? lane >= 16 : r == 1) ? p.v : p.k);
    const int c = half ? lane & 15 : lane;
    uint4 x[kEvBatch];
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i) {
      const int rs = __shfl_sync(0xFFFFFFFFu, mine_s, i);
      if (rs >= 0) x[i] = __ldcs(base + (int64_t)rs * p.row16 + c);
    }
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i) {
      const int rs = __shfl_sync(0xFFFFFFFFu, mine_s, i), rd = __shfl_sync(0xFFFFFFFFu, mine_d, i);
      if (rs >= 0) base[(int64_t)rd * p.row16 + c] = x[i];
    }
  }
  if (rs0 >= 0) sk[(int64_t)rd0 * p.sk16 + c0] = s0;
  for (int e0 = 32; e0 < n_sk; e0 += 32) {
    int rs, rd;
    sk_at(e0, rs, rd);
    const int c = (e0 + lane) % p.sk16;
    if (rs >= 0) sk[(int64_t)rd * p.sk16 + c] = __ldcs(sk + (int64_t)rs * p.sk16 + c);
  }
}

// The lowest k set bits of x.
__device__ __forceinline__ uint32_t ev_lowest(uint32_t x, int k) {
  if (k <= 0) return 0u;
  if (k >= __popc(x)) return x;
  uint32_t rest = x;
  for (int i = 0; i < k; ++i) rest &= rest - 1u;
  return x & ~rest;
}
// Sum of x over the block and, in `before`, over the threads ahead.
__device__ __forceinline__ uint32_t ev_scan(uint32_t x, uint32_t* s_warp, uint32_t& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // s_warp is free
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  const uint32_t w = lane < kEvWarps ? s_warp[lane] : 0u;
  uint32_t ahead = lane < warp ? w : 0u, all = w;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, o);
    all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  }
  before = ahead + inc - x;
  return all;
}

// Two CTAs per SM at most: clusters of 16 then fit every GPC.
__global__ void __launch_bounds__(kEvThreads, 2) evict_kernel(const __grid_constant__ EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) unsigned char ev_smem[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(ev_smem);  // [2048] this CTA's counts
  uint32_t* tot = hist + kEvBins;                         // [2048] the cluster's counts
  uint32_t* part = tot + kEvBins;                         // [4][1024], with more than one CTA
  uint32_t* keys = part + (p.clusters > 1 ? 2 * kEvBins : 0);  // [chunk], chunk a multiple of 32
  uint32_t* gt_w = hist;                                  // [chunk / 32] once the counts are done
  uint32_t* eq_w = tot;
  __shared__ uint32_t s_warp[kEvWarps];
  __shared__ uint32_t s_cnt[3];   // this CTA's equal keys, holes, moves
  __shared__ uint32_t s_bin, s_above;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.y, b = row / p.n_kv_heads, g = row % p.n_kv_heads;
  grid_dependency_wait();
  int L = __ldg(p.seq_len + b);
  if (L < 0 || L > p.max_seq_len) {
    if (tid == 0) flag_status(FASA_ERR_BAD_INDEX);
    L = L < 0 ? 0 : p.max_seq_len;
  }
  const int kept = min(L, p.budget);
  if (rank == 0 && g == 0 && tid == 0) p.len_out[b] = kept;
  const float* mass = p.mass + (int64_t)row * p.max_len;
  const int32_t* pos = p.slot_pos + (int64_t)row * p.max_len;
  float* mass_o = p.mass_out + (int64_t)row * p.max_len;
  int32_t* pos_o = p.slot_pos_out + (int64_t)row * p.max_len;
  const bool copy_m = mass_o != mass, copy_p = pos_o != pos;
  if (L <= p.budget) {  // nothing leaves (the whole cluster agrees)
    if (p.n_moves != nullptr && rank == 0 && tid == 0) p.n_moves[row] = 0;
    for (int t = rank * kEvThreads + tid; t < L; t += C * kEvThreads) {
      if (copy_m) mass_o[t] = mass[t];
      if (copy_p) pos_o[t] = pos[t];
    }
    return;
  }
  const int t0 = rank * p.chunk, n = max(0, min(L - t0, p.chunk));
  const int64_t recent = (int64_t)__ldg(p.cur_pos + b) - p.n_recent;
  for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < n; i += kEvThreads) {
    const int x = pos[t0 + i];
    const float m = mass[t0 + i];
    const bool held = x < p.n_sink || x > recent;
    const uint32_t key = held ? kEvHeld : min(score_key(m), kEvHeld - 1);
    keys[i] = key;
    atomicAdd(&hist[key >> 21], 1u);  // the first digit
  }

  // the budget-th largest key, digit by digit from the top: `prefix` holds
  // the digits found, `want` how many keys with that prefix still to keep
  uint32_t prefix = 0, want = (uint32_t)p.budget;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kBits[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int bins = 1 << kBits[pass];
    if (pass > 0) {
      for (int i = tid; i < bins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      const int done = kShift[pass] + kBits[pass];
#pragma unroll 4
      for (int i = tid; i < n; i += kEvThreads) {
        const uint32_t key = keys[i];
        if ((key >> done) == (prefix >> done)) atomicAdd(&hist[(key >> kShift[pass]) & (bins - 1)], 1u);
      }
    }
    const uint32_t* sum = hist;
    if (C > 1) {
      // this CTA adds up its share of the bins for everyone: four threads a
      // bin, each a quarter of the CTAs (consecutive threads read consecutive
      // words of one CTA)
      cl.sync();
      const int per = bins / C, q = tid / (kEvThreads / 4), i0 = tid % (kEvThreads / 4);
      for (int i = i0; i < per; i += kEvThreads / 4) {
        uint32_t x = 0;
#pragma unroll 4
        for (int c = q; c < C; c += 4) x += cl.map_shared_rank(hist, c)[rank * per + i];
        part[q * (kEvBins / 2) + i] = x;
      }
      __syncthreads();
      for (int i = i0; i < per; i += kEvThreads / 4) {
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) x += part[k * (kEvBins / 2) + i];
#pragma unroll 4
        for (int c = q; c < C; c += 4) cl.map_shared_rank(tot, c)[rank * per + i] = x;
      }
      cl.sync();
      sum = tot;
    } else {
      __syncthreads();
    }
    // counts above each bin: thread t holds the `per_t` bins below bins - t * per_t
    constexpr int per_t = (1 << 11) / kEvThreads;  // two in the last pass
    const int n_t = bins / kEvThreads;
    uint32_t h[per_t], mine = 0;
#pragma unroll
    for (int i = 0; i < per_t; ++i) {
      h[i] = i < n_t ? sum[bins - 1 - (tid * n_t + i)] : 0u;
      mine += h[i];
    }
    uint32_t above;
    ev_scan(mine, s_warp, above);
#pragma unroll
    for (int i = 0; i < per_t; ++i) {
      if (i < n_t && above < want && want <= above + h[i]) {
        s_bin = (uint32_t)(bins - 1 - (tid * n_t + i));
        s_above = above;
      }
      above += h[i];
    }
    __syncthreads();
    prefix |= s_bin << kShift[pass];
    want -= s_above;
  }
  const uint32_t thr = prefix;  // keys above thr stay, and the first `want` slots equal to it

  // bit words of 32 slots: keys above and equal to thr
  const int words = (n + 31) / 32;
  if (C > 1) cl.sync(); else __syncthreads();  // nobody reads the counts any more
#pragma unroll 4
  for (int w = warp; w < words; w += kEvWarps) {
    const int i = w * 32 + lane;
    const uint32_t key = i < n ? keys[i] : 0u;
    const uint32_t gw = __ballot_sync(0xFFFFFFFFu, i < n && key > thr);
    const uint32_t ew = __ballot_sync(0xFFFFFFFFu, i < n && key == thr);
    if (lane == 0) {
      gt_w[w] = gw;
      eq_w[w] = ew;
    }
  }
  __syncthreads();
  // from here on thread t holds words 2 t and 2 t + 1 (chunk <= 32768)
  auto others = [&](int k, uint32_t& all) -> uint32_t {  // sum of s_cnt[k] over the ranks ahead, and over all
    uint32_t x = 0;
    if (lane < C) x = *cl.map_shared_rank(&s_cnt[k], lane);
    uint32_t ahead = lane < rank ? x : 0u;
    all = x;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, o);
      all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    }
    return ahead;
  };
  uint32_t keep[2], hole[2], move[2], eq[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int w = 2 * tid + k;
    keep[k] = w < words ? gt_w[w] : 0u;
    eq[k] = w < words ? eq_w[w] : 0u;
  }
  uint32_t e_at;
  const uint32_t e_all = ev_scan(__popc(eq[0]) + __popc(eq[1]), s_warp, e_at);
  if (C > 1) {
    if (tid == 0) s_cnt[0] = e_all;
    cl.sync();
    uint32_t all;
    e_at += others(0, all);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int w = 2 * tid + k;
    keep[k] |= ev_lowest(eq[k], (int)want - (int)e_at);
    e_at += __popc(eq[k]);
    const int t = t0 + w * 32;
    const int in = max(0, min(32, n - w * 32)), low = max(0, min(32, p.budget - t));
    const uint32_t in_m = in == 32 ? 0xFFFFFFFFu : (1u << in) - 1u, low_m = low == 32 ? 0xFFFFFFFFu : (1u << low) - 1u;
    hole[k] = w < words ? ~keep[k] & in_m & low_m : 0u;
    move[k] = keep[k] & ~low_m;
  }
  // both counts are at most 32768 per CTA: one scan for the two
  uint32_t at;
  const uint32_t both = ev_scan((__popc(hole[0]) + __popc(hole[1])) | ((__popc(move[0]) + __popc(move[1])) << 16),
                                s_warp, at);
  uint32_t h_at = at & 0xFFFFu, m_at = at >> 16, n_moves = both >> 16;
  if (C > 1) {
    if (tid == 0) {
      s_cnt[1] = both & 0xFFFFu;
      s_cnt[2] = both >> 16;
    }
    cl.sync();
    uint32_t all;
    h_at += others(1, all);
    m_at += others(2, n_moves);
  }
  // the lists, a warp per word: the words and what is ahead of each go back to
  // shared memory (the keys are done with)
  uint32_t* hole_w = keys;
  uint32_t* move_w = gt_w;
  uint32_t* ahead_w = eq_w;  // holes | moves << 16 of this CTA ahead of the word
  __syncthreads();
  const uint32_t base_h = h_at - (at & 0xFFFFu), base_m = m_at - (at >> 16);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int w = 2 * tid + k;
    if (w < words) {
      hole_w[w] = hole[k];
      move_w[w] = move[k];
      ahead_w[w] = at;
    }
    at += __popc(hole[k]) | (__popc(move[k]) << 16);
  }
  __syncthreads();
  int32_t* src = p.moves + (int64_t)row * 2 * p.max_moves;
  int32_t* dst = src + p.max_moves;
  const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 2
  for (int w = warp; w < words; w += kEvWarps) {
    const uint32_t hw = hole_w[w], mw = move_w[w], ah = ahead_w[w];
    const int t = t0 + w * 32 + lane;
    if ((hw >> lane) & 1u) dst[base_h + (ah & 0xFFFFu) + __popc(hw & lower)] = t;
    if ((mw >> lane) & 1u) src[base_m + (ah >> 16) + __popc(mw & lower)] = t;
  }
  if (C > 1) cl.sync(); else __syncthreads();  // every CTA's part of the lists is written
  // what stays in its place: every CTA of the cluster a part of the budget
  if (copy_m || copy_p) {
    for (int t = rank * kEvThreads + tid; t < p.budget; t += C * kEvThreads) {
      const int c = t / p.chunk, i = t - c * p.chunk;
      const uint32_t hw = C > 1 ? cl.map_shared_rank(hole_w, c)[i >> 5] : hole_w[i >> 5];
      if ((hw >> (i & 31)) & 1u) continue;
      if (copy_m) mass_o[t] = mass[t];
      if (copy_p) pos_o[t] = pos[t];
    }
  }
  if (p.n_moves != nullptr) {
    if (rank == 0 && tid == 0) p.n_moves[row] = (int)n_moves;
  } else {
    for (uint32_t m0 = (rank * kEvWarps + warp) * kEvBatch; m0 < n_moves; m0 += C * kEvWarps * kEvBatch)
      evict_batch(p, row, m0, n_moves, lane);
  }
  if (C > 1) cl.sync();  // nobody reads this CTA's shared memory any more
}

// The moves of many rows, or of long ones, as a launch of their own: more warps
// in flight than the selection's clusters have. Grid (x, rows).
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictParams p) {
  grid_dependency_wait();
  const int row = blockIdx.y;
  const uint32_t n_moves = (uint32_t)__ldcg(p.n_moves + row);
  const int lane = threadIdx.x & 31;
  for (uint32_t m0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kEvBatch; m0 < n_moves; m0 += gridDim.x * 8 * kEvBatch)
    evict_batch(p, row, m0, n_moves, lane);
}

}  // namespace fasa
