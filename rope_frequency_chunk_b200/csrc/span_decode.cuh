// Span attention of one token per sequence over bf16 caches in device memory:
// K and V steps by TMA, warp-level tensor-core products.
//
// With G <= 16 query rows per KV head the work is the read of K and V: 512
// bytes a slot against 4 G flops a byte. Each warp streams steps of 16 slots
// (4 KB of K, 4 KB of V) through a ring of its own, filled by TMA in the
// 128-byte-swizzled layout that ldmatrix reads without bank conflicts; a step
// lies in one page (pages hold 16 slots or more). The ring runs on from one
// row of the batch to the next, so that the join of a finished row's warps
// does not drain it.
//
// Products are mma.sync m16n8k16 and not tcgen05: G rows fill a sixteenth to
// an eighth of a tcgen05 tile, and at one warp step every operand and result
// stays in the registers of the warp. The 16 rows of an A operand hold two
// terms of the same 8 heads (q = hi + lo, P = hi + lo, 16 bits each), so for
// G <= 8 the second terms cost nothing; for 9 to 16 heads each term is a
// product of its own.
#pragma once

#include <cuda.h>

#include "attend_mma.cuh"
#include "span.cuh"
#include "span_prompt.cuh"

namespace fasa {

constexpr int kSdRows = 16;      // slots per warp step
constexpr int kSdStages = 3;     // steps in flight per warp
constexpr int kSdTile = kSdRows * kD * 2;  // bytes of K (and V) of a step

struct SpanDecodeParams {
  CUtensorMap map_k, map_v;  // [2][rows][64] bf16: boxes of 2 x 16 x 64, 128-byte swizzle
  SpanParams s;
};

// Shared memory: the warps' rings; a buffer that holds the scaled queries at
// a row's start and two warps' states at its end; barriers.
template <int GT>
struct SdSmem {
  static constexpr int kRing = kSpanWarps * kSdStages * 2 * kSdTile;
  static constexpr int kBuf = 2 * GT * kD * 4;
  static constexpr int kBytes = kRing + kBuf + 2 * 2 * GT * 4 + 256 + 512 + 1024;
};

// Row r, 16-byte chunk ch (0 .. 15) of a step's K or V: two halves of 64 dims.
__device__ __forceinline__ uint32_t sd_at(int r, int ch) {
  return (uint32_t)((ch >> 3) * (kSdTile / 2) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void sd_tma(const CUtensorMap* map, void* dst, uint64_t* bar, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(smem_u32(bar))
      : "memory");
}

// Where a CTA is in its run: row (b, g), next unit i of the row, costs left in
// the run (a row's setup counts when the run takes the row up).
struct SdCursor {
  int b, g, i;
  int64_t left;
  int64_t pos;
  Span v;
  SpanUnits u;
};
__device__ __forceinline__ void sd_open(const SpanParams& p, SdCursor& c) {
  const int L = span_len(p, c.b);
  c.pos = span_pos0(p, c.b, L, 1);
  c.v = span_of(L, c.pos, p.window, p.n_sink);
  c.u = span_units(c.v, kSpanUnit);
}
// Moves to the run's next row that has units.
__device__ __forceinline__ void sd_next_row(const SpanParams& p, SdCursor& c) {
  do {
    if (++c.g == p.n_kv_heads) {
      c.g = 0;
      ++c.b;
    }
    if (c.g == 0) sd_open(p, c);
  } while (c.u.n == 0);
  c.i = 0;
  c.left -= kSpanSetup;
}

// The running softmax of a warp: for G <= 8, o[t][0..1] + o[t][2..3] are dims
// 8t + 2q, 8t + 2q + 1 of head lane / 4; for G > 8, o[t][2..3] are those of
// head lane / 4 + 8.
template <int GT>
struct SdState {
  static constexpr int kH = GT / 8;
  float o[16][4];
  float m[kH], l[kH];
};
template <int GT>
struct SdQuery {
  static constexpr int kT = GT / 8;  // A operands per k-step
  uint32_t a[kT][8][4];
};

template <int GT>
__device__ __forceinline__ void sd_query_frags(SdQuery<GT>& Q, const float* qs, int lane) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int s = 0; s < 8; ++s)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int k = 0; k < GT / 8; ++k) {
        const float2 x = *reinterpret_cast<const float2*>(qs + (g + 8 * k) * kD + 16 * s + 8 * half + 2 * q);
        const float h0 = __bfloat162float(__float2bfloat16_rn(x.x)), h1 = __bfloat162float(__float2bfloat16_rn(x.y));
        const uint32_t hi = am_pack(h0, h1), lo = am_pack(x.x - h0, x.y - h1);
        if (GT == 8) {  // [hi; lo]
          Q.a[0][s][2 * half] = hi;
          Q.a[0][s][2 * half + 1] = lo;
        } else {        // hi of 16 heads, lo of 16 heads
          Q.a[0][s][2 * half + k] = hi;
          Q.a[GT / 8 - 1][s][2 * half + k] = lo;
        }
      }
}

// One step: `mask` bit r says whether slot t0 + r takes part.
template <int GT>
__device__ __forceinline__ void sd_step(SdState<GT>& st, const SdQuery<GT>& Q, uint32_t ks, uint32_t vs,
                                        unsigned mask, int lane, float* logits, int64_t ld, int G) {
  constexpr int kH = GT / 8;
  const int q = lane & 3, mi = lane >> 3, r8 = lane & 7;
  float s[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t b[4];
      am_ldsm4(b, ks + sd_at(8 * j + r8, 4 * u + mi));
#pragma unroll
      for (int t = 0; t < kH; ++t) {
        am_mma(s[j], Q.a[t][2 * u][0], Q.a[t][2 * u][1], Q.a[t][2 * u][2], Q.a[t][2 * u][3], b[0], b[1]);
        am_mma(s[j], Q.a[t][2 * u + 1][0], Q.a[t][2 * u + 1][1], Q.a[t][2 * u + 1][2], Q.a[t][2 * u + 1][3], b[2],
               b[3]);
      }
    }
  // logits of head lane / 4 (+ 8 k) for slots 8 j + 2 q + e
  float z[kH][2][2], mx[kH];
#pragma unroll
  for (int k = 0; k < kH; ++k) {
    mx[k] = -INFINITY;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) z[k][j][e] = GT == 8 ? __fadd_rn(s[j][e], s[j][e + 2]) : s[j][2 * k + e];
      const int h = (lane >> 2) + 8 * k;
      if (logits != nullptr && h < G)
        *reinterpret_cast<float2*>(logits + h * ld + 8 * j + 2 * q) = make_float2(z[k][j][0], z[k][j][1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (!((mask >> (8 * j + 2 * q + e)) & 1u)) z[k][j][e] = -INFINITY;
        mx[k] = fmaxf(mx[k], z[k][j][e]);
      }
    }
    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xFFFFFFFFu, mx[k], 1));
    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xFFFFFFFFu, mx[k], 2));
  }
  bool up = false;
#pragma unroll
  for (int k = 0; k < kH; ++k) up |= mx[k] > st.m[k];
  if (__any_sync(0xFFFFFFFFu, up)) {
    float sc[kH];
#pragma unroll
    for (int k = 0; k < kH; ++k) {
      const float mn = fmaxf(st.m[k], mx[k]);
      sc[k] = st.m[k] == -INFINITY ? 0.0f : exp2f(st.m[k] - mn);
      st.m[k] = mn;
      st.l[k] *= sc[k];
    }
#pragma unroll
    for (int t = 0; t < 16; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][e] *= sc[GT == 8 ? 0 : e >> 1];
  }
  uint32_t ph[kH][2], pl[kH][2];  // P terms for slots 8 j + 2 q + {0, 1}
#pragma unroll
  for (int k = 0; k < kH; ++k) {
    const float off = st.m[k] == -INFINITY ? 0.0f : st.m[k];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float a[2], b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float pz = exp2f(z[k][j][e] - off);
        st.l[k] += pz;
        a[e] = __bfloat162float(__float2bfloat16_rn(pz));
        b[e] = pz - a[e];
      }
      ph[k][j] = am_pack(a[0], a[1]);
      pl[k][j] = am_pack(b[0], b[1]);
    }
  }
  const int vr = ((mi & 1) << 3) + r8;
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    uint32_t b[4];
    am_ldsm4_t(b, vs + sd_at(vr, 2 * v + (mi >> 1)));
    if (GT == 8) {
      am_mma(st.o[2 * v], ph[0][0], pl[0][0], ph[0][1], pl[0][1], b[0], b[1]);
      am_mma(st.o[2 * v + 1], ph[0][0], pl[0][0], ph[0][1], pl[0][1], b[2], b[3]);
    } else {
      constexpr int k1 = kH - 1;
      am_mma(st.o[2 * v], ph[0][0], ph[k1][0], ph[0][1], ph[k1][1], b[0], b[1]);
      am_mma(st.o[2 * v + 1], ph[0][0], ph[k1][0], ph[0][1], ph[k1][1], b[2], b[3]);
      am_mma(st.o[2 * v], pl[0][0], pl[k1][0], pl[0][1], pl[k1][1], b[0], b[1]);
      am_mma(st.o[2 * v + 1], pl[0][0], pl[k1][0], pl[0][1], pl[k1][1], b[2], b[3]);
    }
  }
}

// Grid: n_cta CTAs over the rows' units, or with n_cta 0 one CTA per row (x).
template <int GT>
__global__ void __launch_bounds__(kSpanThreads, 2) span_decode_kernel(const __grid_constant__ SpanDecodeParams pp) {
  constexpr int kH = GT / 8;
  const SpanParams& p = pp.s;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ SpanIndex index;
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem + warp * kSdStages * 2 * kSdTile;
  float* buf = reinterpret_cast<float*>(smem + SdSmem<GT>::kRing);  // queries; two warps' o
  float* sm_m = buf + 2 * GT * kD;                                  // [2][GT]
  float* sm_l = sm_m + 2 * GT;
  double* turns = reinterpret_cast<double*>(sm_l + 2 * GT);         // [64]
  uint64_t* full = reinterpret_cast<uint64_t*>(turns + kNFC) + warp * kSdStages;
  const int G = p.group;

  if (lane == 0) {
    for (int i = 0; i < kSdStages; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (tid == 0) {
    prefetch_tensor_map(&pp.map_k);
    prefetch_tensor_map(&pp.map_v);
  }
  span_stage_turns<kSpanThreads>(p, turns);
  grid_dependency_wait();

  // the CTA's run
  SdCursor use;
  if (p.n_cta == 0) {
    use.b = blockIdx.x / p.n_kv_heads;
    use.g = blockIdx.x % p.n_kv_heads;
    sd_open(p, use);
    use.i = 0;
    use.left = use.u.n;
    if (use.u.n == 0) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (int64_t)blockIdx.x * G * kD;
      for (int e = tid; e < G * kD; e += kSpanThreads) out[e] = __float2bfloat16_rn(0.0f);
      return;
    }
  } else {
    span_zero_rows<__nv_bfloat16, kSpanThreads>(p);
    const int64_t total = span_index(p, index);
    const int n_cta = span_ctas(total, p.n_cta);
    if ((int)blockIdx.x >= n_cta) return;
    const SpanDeal deal = span_deal(total, n_cta);
    const int64_t u0 = deal.cut(blockIdx.x);
    const SpanWhere where = span_find(p, index, u0);
    use.b = where.b;
    const int64_t at = u0 - where.base;
    use.g = (int)(at / span_cost(where.units));
    const int a0 = (int)(at % span_cost(where.units));
    use.i = max(a0 - kSpanSetup, 0);
    use.left = deal.cut(blockIdx.x + 1) - u0 - max(kSpanSetup - a0, 0);
    sd_open(p, use);
  }
  SdCursor get = use;  // where the loads are
  uint32_t n_get = 0, n_use = 0;
  unsigned live = 0;   // bit: the stage's step has a page
  bool ok = true;
  // requests the warp's next step that has visible slots; false at the end
  auto request = [&]() -> bool {
    for (;;) {
      if (get.left <= 0) return false;
      if (get.i == get.u.n) {
        if (get.left <= kSpanSetup) return false;  // the run ends in the next row's setup
        sd_next_row(p, get);
      }
      const int t0 = get.u.unit(get.i) * kSpanUnit + warp * kSdRows;
      ++get.i;
      --get.left;
      if (t0 >= get.v.hi || (t0 + kSdRows <= get.v.lo && t0 >= get.v.s)) continue;
      const uint32_t st = n_get % kSdStages;
      int64_t row = p.pm.table ? (int64_t)paged_row(p.pm, get.b, get.g, t0)
                               : (int64_t)(get.b * p.n_kv_heads + get.g) * p.max_len + t0;
      live = row >= 0 ? live | (1u << st) : live & ~(1u << st);
      if (row >= 0 && lane == 0) {
        mbar_arrive_expect_tx(full + st, 2 * kSdTile);
        sd_tma(&pp.map_k, ring + st * 2 * kSdTile, full + st, (int)row);
        sd_tma(&pp.map_v, ring + st * 2 * kSdTile + kSdTile, full + st, (int)row);
      }
      // a step without a page completes its phase at once
      if (row < 0 && lane == 0) pr_arrive(full + st);
      ++n_get;
      return true;
    }
  };
  for (int i = 0; i < kSdStages; ++i) request();
  SpanQuery<__nv_bfloat16, kSpanThreads, GT> next_q;  // the next row's queries, on their way
  next_q.load(p, use.b, 0, use.g);
  __syncthreads();  // the rotation table

  for (bool first = true; use.left > 0 && ok; first = false) {
    if (use.i == use.u.n) {
      if (use.left <= kSpanSetup) break;
      sd_next_row(p, use);
    }
    const int64_t row = (int64_t)use.b * p.n_kv_heads + use.g;
    const int i0 = use.i, i1 = (int)min((int64_t)use.u.n, i0 + use.left);
    const bool whole = i0 == 0 && i1 == use.u.n;
    for (int e = tid; e < (GT - G) * kD; e += kSpanThreads) buf[G * kD + e] = 0.0f;
    next_q.rotate(p, turns, use.pos, buf);
    __syncthreads();
    if (use.left - (i1 - i0) > kSpanSetup) {  // the row after this one
      SdCursor nx = use;
      sd_next_row(p, nx);
      next_q.load(p, nx.b, 0, nx.g);
    }
    SdQuery<GT> Q;
    sd_query_frags<GT>(Q, buf, lane);
    SdState<GT> st;
#pragma unroll
    for (int t = 0; t < 16; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < kH; ++k) {
      st.m[k] = -INFINITY;
      st.l[k] = 0.0f;
    }
    for (int i = i0; i < i1; ++i) {
      const int t0 = use.u.unit(i) * kSpanUnit + warp * kSdRows;
      if (t0 >= use.v.hi || (t0 + kSdRows <= use.v.lo && t0 >= use.v.s)) continue;
      const uint32_t sg = n_use % kSdStages;
      if (!pr_wait(full + sg, (n_use / kSdStages) & 1)) {
        ok = false;
        break;
      }
      if ((live >> sg) & 1u) {
        unsigned char* vst = ring + sg * 2 * kSdTile + kSdTile;
        const unsigned mask = pr_mask(use.v, t0, 0) & 0xFFFFu;
        if (mask != 0xFFFFu) {  // what unseen slots hold must not meet 0 * v
          for (int e = lane; e < kSdRows * 16; e += 32) {
            const int r = e >> 4;
            if (!((mask >> r) & 1u)) *reinterpret_cast<uint4*>(vst + sd_at(r, e & 15)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        sd_step<GT>(st, Q, smem_u32(ring + sg * 2 * kSdTile), smem_u32(vst), mask, lane,
                    p.logits ? p.logits + row * G * p.ld_logits + t0 : nullptr, p.ld_logits, G);
      }
      __syncwarp();  // every lane is done with the stage
      ++n_use;
      request();
    }
    // join the four warps: 2 and 3 into 0 and 1, then 1 into 0
    const int g8 = lane >> 2, q = lane & 3;
    float o[kH][16][2];
#pragma unroll
    for (int k = 0; k < kH; ++k) {
      st.l[k] += __shfl_xor_sync(0xFFFFFFFFu, st.l[k], 1);
      st.l[k] += __shfl_xor_sync(0xFFFFFFFFu, st.l[k], 2);
#pragma unroll
      for (int t = 0; t < 16; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[k][t][e] = GT == 8 ? __fadd_rn(st.o[t][e], st.o[t][e + 2]) : st.o[t][2 * k + e];
    }
    auto put = [&](int slot) {
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        const int h = g8 + 8 * k;
#pragma unroll
        for (int t = 0; t < 16; ++t)
          *reinterpret_cast<float2*>(buf + (slot * GT + h) * kD + 8 * t + 2 * q) = make_float2(o[k][t][0], o[k][t][1]);
        if (q == 0) {
          sm_m[slot * GT + h] = st.m[k];
          sm_l[slot * GT + h] = st.l[k];
        }
      }
    };
    auto take = [&](int slot) {
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        const int h = g8 + 8 * k;
        const float m2 = sm_m[slot * GT + h], l2 = sm_l[slot * GT + h];
        const float M = fmaxf(st.m[k], m2);
        const float f1 = st.m[k] == -INFINITY ? 0.0f : exp2f(st.m[k] - M);
        const float f2 = m2 == -INFINITY ? 0.0f : exp2f(m2 - M);
        st.m[k] = M;
        st.l[k] = f1 * st.l[k] + f2 * l2;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const float2 x = *reinterpret_cast<const float2*>(buf + (slot * GT + h) * kD + 8 * t + 2 * q);
          o[k][t][0] = f1 * o[k][t][0] + f2 * x.x;
          o[k][t][1] = f1 * o[k][t][1] + f2 * x.y;
        }
      }
    };
    // every warp has its query fragments: the buffer is free. If a warp's wait
    // gave up, all leave behind this row: none is left at a barrier.
    ok = __syncthreads_and(ok);
    if (warp >= 2) put(warp - 2);
    __syncthreads();
    if (warp < 2) take(warp);
    __syncwarp();
    if (warp == 1) put(1);
    __syncthreads();
    if (warp == 0) {
      take(1);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * G * kD;
      float* part = p.part + (int64_t)(2 * blockIdx.x + (first ? 0 : 1)) * (kSpanHead + G * kD);
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        const int h = g8 + 8 * k;
        if (h < G) {
          const float inv = st.l[k] == 0.0f ? 0.0f : 1.0f / st.l[k];
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            const int d = h * kD + 8 * t + 2 * q;
            if (whole)
              *reinterpret_cast<__nv_bfloat162*>(out + d) =
                  st.l[k] == 0.0f ? __floats2bfloat162_rn(0.0f, 0.0f)
                                  : __floats2bfloat162_rn(o[k][t][0] * inv, o[k][t][1] * inv);
            else
              *reinterpret_cast<float2*>(part + kSpanHead + d) = make_float2(o[k][t][0], o[k][t][1]);
          }
          if (q == 0) {
            if (!whole) {
              part[h] = st.m[k];
              part[16 + h] = st.l[k];
            } else if (p.rstat != nullptr) {
              p.rstat[row * 2 * G + h] = st.m[k];
              p.rstat[row * 2 * G + G + h] = st.l[k];
            }
          }
        }
      }
    }
    __syncthreads();  // the buffer takes the next row's queries
    use.i = i1;
    use.left -= i1 - i0;
  }
  // copies in flight land before the block ends (none unless a wait gave up)
  for (; n_use < n_get; ++n_use) mbar_wait(full + n_use % kSdStages, (n_use / kSdStages) & 1);
  grid_dependents_launch();
}

}  // namespace fasa
