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
// One cluster of CTAs per (b, g) row. Each CTA keeps the order-preserving
// keys of its share of the slots in shared memory; three histogram passes
// (11 + 11 + 10 bits, summed over the cluster through distributed shared
// memory) give the exact budget-th largest key, ballots rank the slots, and
// the cluster's warps copy the moved rows. Bound by memory: 8 bytes a slot
// and the moved rows; a small row by the chain of cluster barriers.
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
  int64_t max_len;
  int32_t max_seq_len;
  int32_t budget;
  int32_t n_sink;
  int32_t n_recent;
  int32_t n_kv_heads;
  int32_t max_moves;
  int32_t chunk;             // slots per CTA, a multiple of 32
  int32_t row16;             // 16-byte vectors of a K (and V) row
  int32_t sk16;              // of a sketch row
  PageMap pm;
};

constexpr uint32_t kEvHeld = 0xFFFFFFFFu;

// Moves of one warp at a time: their rows are all in flight together.
constexpr int kEvBatch = 8;

// Copies `n` 16-byte vectors of each of the warp's rows rs[i] -> rd[i] (-1: none).
__device__ __forceinline__ void evict_copy(void* pool, const int (&rs)[kEvBatch], const int (&rd)[kEvBatch],
                                           int n, int lane) {
  uint4* base = static_cast<uint4*>(pool);
  for (int c = lane; c < n; c += 32) {
    uint4 x[kEvBatch];
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i)
      if (rs[i] >= 0) x[i] = __ldcs(base + (int64_t)rs[i] * n + c);
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i)
      if (rs[i] >= 0) base[(int64_t)rd[i] * n + c] = x[i];
  }
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) unsigned char ev_smem[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(ev_smem);  // [2048] this CTA's counts
  uint32_t* tot = hist + kEvBins;                         // [2048] the cluster's counts
  uint32_t* keys = tot + kEvBins;                         // [chunk]
  __shared__ uint32_t s_warp[kEvWarps], s_warp2[kEvWarps];
  __shared__ uint32_t s_cnt[3];   // this CTA's equal keys, holes, moves
  __shared__ uint32_t s_bin, s_above;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.y, b = row / p.n_kv_heads, g = row % p.n_kv_heads;
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
    for (int t = rank * kEvThreads + tid; t < L; t += C * kEvThreads) {
      if (copy_m) mass_o[t] = mass[t];
      if (copy_p) pos_o[t] = pos[t];
    }
    return;
  }
  const int t0 = rank * p.chunk, n = max(0, min(L - t0, p.chunk));
  const int64_t recent = (int64_t)__ldg(p.cur_pos + b) - p.n_recent;
  for (int i = tid; i < n; i += kEvThreads) {
    const int x = pos[t0 + i];
    const bool held = x < p.n_sink || x > recent;
    keys[i] = held ? kEvHeld : min(score_key(mass[t0 + i]), kEvHeld - 1);
  }

  // the budget-th largest key, digit by digit from the top: `prefix` holds
  // the digits found, `want` how many keys with that prefix still to keep
  uint32_t prefix = 0, want = (uint32_t)p.budget;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kBits[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int bins = 1 << kBits[pass];
    for (int i = tid; i < bins; i += kEvThreads) hist[i] = 0;
    __syncthreads();  // (first pass: the keys too)
    const int done = kShift[pass] + kBits[pass];
    for (int i = tid; i < n; i += kEvThreads) {
      const uint32_t key = keys[i];
      if (pass == 0 || (key >> done) == (prefix >> done))
        atomicAdd(&hist[(key >> kShift[pass]) & (bins - 1)], 1u);
    }
    const uint32_t* sum = hist;
    if (C > 1) {
      cl.sync();
      const int per = bins / C;  // this CTA adds up its share of the bins for everyone
      for (int i = tid; i < per; i += kEvThreads) {
        uint32_t s = 0;
#pragma unroll 4
        for (int c = 0; c < C; ++c) s += cl.map_shared_rank(hist, c)[rank * per + i];
#pragma unroll 4
        for (int c = 0; c < C; ++c) cl.map_shared_rank(tot, c)[rank * per + i] = s;
      }
      cl.sync();
      sum = tot;
    } else {
      __syncthreads();
    }
    // counts above each bin: thread t holds the `per_t` bins below bins - t * per_t
    const int per_t = bins / kEvThreads;
    uint32_t mine = 0;
    for (int i = 0; i < per_t; ++i) mine += sum[bins - 1 - (tid * per_t + i)];
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    uint32_t above = inc - mine;
    for (int w = 0; w < warp; ++w) above += s_warp[w];
    for (int i = 0; i < per_t; ++i) {
      const int bin = bins - 1 - (tid * per_t + i);
      const uint32_t h = sum[bin];
      if (above < want && want <= above + h) {
        s_bin = (uint32_t)bin;
        s_above = above;
      }
      above += h;
    }
    __syncthreads();
    prefix |= s_bin << kShift[pass];
    want -= s_above;
  }
  const uint32_t thr = prefix;  // keys above thr stay, and the first `want` slots equal to it

  // warp w of the CTA takes slots [w * span, (w + 1) * span) of its chunk
  const int span = (p.chunk / 32 + kEvWarps - 1) / kEvWarps * 32;
  const int i0 = min(n, warp * span), i1 = min(n, i0 + span);
  uint32_t eq = 0;
  for (int i = i0; i < i1; i += 32) eq += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < i1 && keys[i + lane] == thr));
  if (lane == 0) s_warp[warp] = eq;
  __syncthreads();
  uint32_t eq_before = 0, eq_all = 0;
  for (int w = 0; w < kEvWarps; ++w) {
    if (w < warp) eq_before += s_warp[w];
    eq_all += s_warp[w];
  }
  if (C > 1) {
    if (tid == 0) s_cnt[0] = eq_all;
    cl.sync();
    for (int c = 0; c < rank; ++c) eq_before += *cl.map_shared_rank(&s_cnt[0], c);
  }
  // one pass over the warp's slots in order: f(i, slot, keep) of the 32 lanes' slots
  auto scan_slots = [&](auto f) {
    uint32_t e = eq_before;
    for (int i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      const uint32_t key = in ? keys[i + lane] : 0u;
      const unsigned eqm = __ballot_sync(0xFFFFFFFFu, in && key == thr);
      const bool keep = in && (key > thr || (key == thr && e + __popc(eqm & ((1u << lane) - 1u)) < want));
      f(t0 + i + lane, in, keep);
      e += __popc(eqm);
    }
  };
  uint32_t holes = 0, moves = 0;
  scan_slots([&](int t, bool in, bool keep) {
    holes += __popc(__ballot_sync(0xFFFFFFFFu, in && !keep && t < p.budget));
    moves += __popc(__ballot_sync(0xFFFFFFFFu, keep && t >= p.budget));
  });
  __syncthreads();  // s_warp is free
  if (lane == 0) {
    s_warp[warp] = holes;
    s_warp2[warp] = moves;
  }
  __syncthreads();
  uint32_t h_at = 0, m_at = 0, h_all = 0, m_all = 0;
  for (int w = 0; w < kEvWarps; ++w) {
    if (w < warp) {
      h_at += s_warp[w];
      m_at += s_warp2[w];
    }
    h_all += s_warp[w];
    m_all += s_warp2[w];
  }
  uint32_t n_moves = m_all;
  if (C > 1) {
    if (tid == 0) {
      s_cnt[1] = h_all;
      s_cnt[2] = m_all;
    }
    cl.sync();
    n_moves = 0;
    for (int c = 0; c < C; ++c) {
      const uint32_t m = *cl.map_shared_rank(&s_cnt[2], c);
      if (c < rank) {
        h_at += *cl.map_shared_rank(&s_cnt[1], c);
        m_at += m;
      }
      n_moves += m;
    }
  }
  int32_t* src = p.moves + (int64_t)row * 2 * p.max_moves;
  int32_t* dst = src + p.max_moves;
  scan_slots([&](int t, bool in, bool keep) {
    const bool hole = in && !keep && t < p.budget, move = keep && t >= p.budget;
    const unsigned hm = __ballot_sync(0xFFFFFFFFu, hole), mm = __ballot_sync(0xFFFFFFFFu, move);
    const unsigned lower = (1u << lane) - 1u;
    if (hole) dst[h_at + __popc(hm & lower)] = t;
    if (move) src[m_at + __popc(mm & lower)] = t;
    h_at += __popc(hm);
    m_at += __popc(mm);
    if (keep && t < p.budget) {
      if (copy_m) mass_o[t] = mass[t];
      if (copy_p) pos_o[t] = pos[t];
    }
  });
  if (C > 1) cl.sync(); else __syncthreads();  // every CTA's part of the lists is written
  const int n_warps = C * kEvWarps;
  for (uint32_t m0 = (rank * kEvWarps + warp) * kEvBatch; m0 < n_moves; m0 += n_warps * kEvBatch) {
    int mine_s = -1, mine_d = -1;  // lane i < kEvBatch: the rows of move m0 + i
    if (lane < kEvBatch && m0 + lane < n_moves) {
      const int ts = src[m0 + lane], td = dst[m0 + lane];
      mass_o[td] = mass[ts];
      pos_o[td] = pos[ts];
      mine_s = p.pm.table ? paged_row(p.pm, b, g, ts) : (int)(row * p.max_len + ts);
      mine_d = p.pm.table ? paged_row(p.pm, b, g, td) : (int)(row * p.max_len + td);
      if (mine_d < 0) mine_s = -1;  // a page outside the pool, flagged
    }
    int rs[kEvBatch], rd[kEvBatch];
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i) {
      rs[i] = __shfl_sync(0xFFFFFFFFu, mine_s, i);
      rd[i] = __shfl_sync(0xFFFFFFFFu, mine_d, i);
    }
    evict_copy(p.k, rs, rd, p.row16, lane);
    evict_copy(p.v, rs, rd, p.row16, lane);
    evict_copy(p.sketch, rs, rd, p.sk16, lane);
  }
}

}  // namespace fasa
