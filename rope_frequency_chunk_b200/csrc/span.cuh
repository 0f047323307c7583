// Attention of new tokens over a span of cached slots: all of a sequence's
// slots, or a sliding window of them plus the first n_sink (sink tokens).
//
// A token at position p of a sequence with L cached slots sees slot t when
//   t < L, t <= p, and (no window, or t > p - window, or t < n_sink):
// the slots [0, s) and [lo, hi) with hi = min(L, p + 1), lo = max(0, p -
// window + 1) (0 without a window) and s = min(n_sink, lo, hi). Its output is
//   out = sum_t w_t v_t,  w_t = exp(z_t - max z) / sum exp(z - max z),
//   z_t = q' . k_t / sqrt(128),
// computed in one pass with a running maximum and sum in float32, base 2.
//
// Here: the span and the work partition shared by the kernels, the CUDA-core
// kernel (float32 caches, and caches in host memory) and the merge of rows
// that several CTAs shared, which also adds the slots' attention weights.
#pragma once

#include "fasa_device.cuh"

namespace fasa {

constexpr int kSpanUnit = 64;      // slots per unit of work
constexpr int kSpanThreads = 128;  // 4 warps
constexpr int kSpanWarps = kSpanThreads / 32;
constexpr int kSpanHead = 32;      // floats ahead of a partial's o: m[16], l[16]
// Slots per warp step of the CUDA-core kernel: eight rows in flight, or four
// where 16 heads' queries and sums fill the registers.
__host__ __device__ constexpr int span_step(int mg) { return mg > 8 ? 4 : 8; }

struct SpanParams {
  const void* k;
  const void* v;
  const void* q;             // [B][n_q][Hq][128]
  void* out;                 // [B][n_q][Hq][128]
  const int32_t* seq_len;    // [B]
  const int32_t* q_pos;      // [B] or null
  const int32_t* q_len;      // [B] or null
  int64_t max_len;           // slots of a (b, g) plane (contiguous caches)
  int32_t max_seq_len;
  int32_t window;            // 0: none
  int32_t n_sink;
  int32_t q_prerot;
  int32_t pos_at_len;        // q_pos null: the query sits at seq_len (decode), not at seq_len - q_len (prompt)
  int32_t n_q;
  int32_t batch;
  int32_t n_kv_heads;
  int32_t group;
  int32_t n_cta;             // CTAs the units are dealt to; 0: one CTA per row, no partials
  PageMap pm;
  float* part;               // [2 * n_cta][kSpanHead + group * 128]: m[16], l[16], o[G][128]
  float* rstat;              // [rows][2 * group]: m, l of a row one CTA finished
  float* logits;             // [rows][group][ld_logits] base-2 logits, or null
  float* mass;               // [rows][mass_ld] accumulated weights, or null
  int64_t ld_logits;
  int64_t mass_ld;
  double turns[kNFC];        // theta_i / (2 pi)
};

// The visible slots of one token: [0, s) and [lo, hi); empty: hi == 0.
struct Span {
  int s, lo, hi;
  __device__ __forceinline__ bool sees(int t) const { return t < hi && (t >= lo || t < s); }
};
__device__ __forceinline__ Span span_of(int L, int64_t p, int window, int n_sink) {
  Span v;
  v.hi = p < 0 ? 0 : (int)min((int64_t)L, p + 1);
  const int64_t lo = window > 0 ? p - window + 1 : 0;
  v.lo = (int)max((int64_t)0, min(lo, (int64_t)v.hi));
  v.s = min(n_sink, v.lo);
  return v;
}
// The units of kSpanUnit slots that a span touches: the first na units, then
// units first .. first + n - na - 1.
struct SpanUnits {
  int na, first, n;
  __device__ __forceinline__ int unit(int i) const { return i < na ? i : first + i - na; }
};
__device__ __forceinline__ SpanUnits span_units(const Span& v, int unit) {
  SpanUnits u;
  u.na = (v.s + unit - 1) / unit;
  u.first = max(v.lo / unit, u.na);
  u.n = u.na + max(0, (v.hi + unit - 1) / unit - u.first);
  return u;
}

// A sequence's length and (decode) its query's position; a length outside
// 0 .. max_seq_len is clamped and flagged.
__device__ __forceinline__ int span_len(const SpanParams& p, int b) {
  int L = __ldg(p.seq_len + b);
  if (L < 0 || L > p.max_seq_len) {
    flag_status(FASA_ERR_BAD_INDEX);
    L = L < 0 ? 0 : p.max_seq_len;
  }
  return L;
}
__device__ __forceinline__ int span_qlen(const SpanParams& p, int b) {
  if (p.q_len == nullptr) return p.n_q;
  int n = __ldg(p.q_len + b);
  if (n < 0 || n > p.n_q) {
    flag_status(FASA_ERR_BAD_INDEX);
    n = n < 0 ? 0 : p.n_q;
  }
  return n;
}
// Position of sequence b's first query.
__device__ __forceinline__ int64_t span_pos0(const SpanParams& p, int b, int L, int nq) {
  if (p.q_pos != nullptr) return __ldg(p.q_pos + b);
  return p.pos_at_len ? L : (int64_t)L - nq;
}

// cos and sin of pos * theta for turns = theta / (2 pi): whole turns drop out
// in float64, so the float32 argument keeps its precision at any position
// (angle error below 3e-7 for positions up to 2^31).
__device__ __forceinline__ void span_angle(double turns, int64_t pos, float* c, float* s) {
  const double t = (double)pos * turns;
  sincospif(2.0f * (float)(t - rint(t)), s, c);
}

// Units of sequence b (one token per sequence), the same for each KV head.
__device__ __forceinline__ int span_seq_units(const SpanParams& p, int b) {
  const int L = span_len(p, b);
  return span_units(span_of(L, span_pos0(p, b, L, 1), p.window, p.n_sink), kSpanUnit).n;
}

// Sum of x over the block, and the exclusive prefix of this thread's x.
template <int NT>
__device__ __forceinline__ int64_t span_scan(int64_t x, int64_t* sm, int64_t& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // sm is free
  if (lane == 31) sm[warp] = v;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += sm[w];
    total += sm[w];
  }
  before = base + v - x;
  return total;
}

// The units of all (b, g) rows, in that order, are dealt to n_cta CTAs in
// equal runs: CTA c owns units [c T / n, (c + 1) T / n) of the T, n =
// min(n_cta, T), so no run is empty. A run may begin and end inside a row;
// such a row's CTAs leave partials.
__device__ __forceinline__ int span_ctas(int64_t total, int n_cta) { return (int)min((int64_t)n_cta, total); }
__device__ __forceinline__ int64_t span_cut(int64_t total, int c, int n_cta) { return total * c / n_cta; }
// The CTA that owns unit u.
__device__ __forceinline__ int span_owner(int64_t total, int64_t u, int n_cta) {
  int c = (int)((u * n_cta) / total);
  while (span_cut(total, c + 1, n_cta) <= u) ++c;
  while (span_cut(total, c, n_cta) > u) --c;
  return c;
}
// Totals over the sequences: the number of units, and for sequence `at` (or,
// with at < 0, the sequence that holds unit `u`) its index and first unit.
struct SpanWhere {
  int64_t total, base;  // base: first unit of sequence b (its KV head 0)
  int b, units;         // units of one row of b
};
template <int NT>
__device__ __forceinline__ int64_t span_total(const SpanParams& p, int64_t* sm) {
  int64_t t = 0;
  for (int b = threadIdx.x; b < p.batch; b += NT) t += span_seq_units(p, b);
  int64_t before;
  return span_scan<NT>(t, sm, before) * p.n_kv_heads;
}
// Block-wide: finds sequence `at`, or the one that holds unit u (at < 0).
// Returns false (b = -1) when no sequence does. `out` is shared memory.
template <int NT>
__device__ __forceinline__ void span_find(const SpanParams& p, int at, int64_t u, int64_t* sm, SpanWhere* out) {
  if (threadIdx.x == 0) out->b = -1;
  int64_t run = 0;
  for (int b0 = 0; b0 < p.batch; b0 += NT) {
    const int b = b0 + threadIdx.x;
    const int n = b < p.batch ? span_seq_units(p, b) : 0;
    int64_t before;
    const int64_t sum = span_scan<NT>((int64_t)n * p.n_kv_heads, sm, before);
    before += run;
    const bool mine = at >= 0 ? b == at : (n > 0 && before <= u && u < before + (int64_t)n * p.n_kv_heads);
    if (mine) {
      out->b = b;
      out->base = before;
      out->units = n;
    }
    run += sum;
  }
  __syncthreads();
}

// --------------------------------------------------- CUDA-core attention

// Sums v[0 .. N-1] over the 32 lanes, each lane keeping its share: after the
// call lane l holds in v[0 .. M-1] the sums of the M = max(1, N / 32) values
// that start at its index (the returned one); with N < 32, 32 / N lanes hold
// the same value.
template <int N>
__device__ __forceinline__ int span_reduce_scatter(float (&v)[N], int lane) {
  int first = 0;
  int n = N;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
      if (up) first += n;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const float give = up ? v[i] : v[i + n];
          const float keep = up ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    }
  }
  return first;
}

template <typename T>
__device__ __forceinline__ float4 span_load4(const T* p);
template <>
__device__ __forceinline__ float4 span_load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
template <>
__device__ __forceinline__ float4 span_load4(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

// Shared memory of the CUDA-core kernel: the group's scaled rotated queries,
// each warp's probabilities of a step and rescaling factors, the warps'
// states.
template <int MG>
struct alignas(16) SpanCcSmem {
  float q[MG][kD];
  float p[kSpanWarps][span_step(MG)][MG];
  float sc[kSpanWarps][MG];
  float m[kSpanWarps][MG], l[kSpanWarps][MG];
  float o[kSpanWarps][MG][kD];
  int64_t scan[kSpanWarps];
  SpanWhere where;
};

// The G query rows of token (b, j), KV head g, rotated at position pos and
// scaled by log2(e) / sqrt(128), into qs [G][128] (barriers around it are the
// caller's).
template <typename T, int NT>
__device__ __forceinline__ void span_queries(const SpanParams& p, int b, int j, int g, int64_t pos, float* qs) {
  constexpr float kScale = 1.4426950408889634f * 0.08838834764831845f;
  const int G = p.group;
  const T* q = static_cast<const T*>(p.q) + (((int64_t)b * p.n_q + j) * p.n_kv_heads + g) * G * kD;
  for (int e = threadIdx.x; e < G * kNFC; e += NT) {
    const int h = e / kNFC, i = e % kNFC;
    const float x = to_float(q[h * kD + i]), y = to_float(q[h * kD + i + kNFC]);
    float c = 1.0f, s = 0.0f;
    if (!p.q_prerot) span_angle(p.turns[i], pos, &c, &s);
    qs[h * kD + i] = (x * c - y * s) * kScale;
    qs[h * kD + i + kNFC] = (y * c + x * s) * kScale;
  }
}

// One CTA's share of a row, units [i0, i1) of the row's n: the output when
// that is the whole row, else partial `slot`.
template <typename T, int MG>
__device__ __forceinline__ void span_cc_segment(const SpanParams& p, SpanCcSmem<MG>& sm, int b, int j, int g,
                                                const Span& v, const SpanUnits& u, int64_t pos, int i0, int i1,
                                                int slot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group;
  const int64_t row = (int64_t)b * p.n_kv_heads + g;
  __syncthreads();  // the previous segment is done with shared memory
  span_queries<T, kSpanThreads>(p, b, j, g, pos, &sm.q[0][0]);
  __syncthreads();
  float q[MG][4], o[MG][4];
#pragma unroll
  for (int h = 0; h < MG; ++h)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      q[h][d] = h < G ? sm.q[h][lane * 4 + d] : 0.0f;
      o[h][d] = 0.0f;
    }
  // after the reduce-scatter a lane holds kMine values (slot, head) with
  // consecutive heads of one slot: index = slot * MG + head
  constexpr int kSpanStep = span_step(MG);
  constexpr int kVals = kSpanStep * MG;
  constexpr int kMine = kVals / 32 > 0 ? kVals / 32 : 1;
  float m_run[MG];  // every lane keeps every head's running maximum
#pragma unroll
  for (int h = 0; h < MG; ++h) m_run[h] = -INFINITY;
  float l_run[kMine];  // this lane's share of the sums
#pragma unroll
  for (int i = 0; i < kMine; ++i) l_run[i] = 0.0f;
  const bool paged = p.pm.table != nullptr;
  const int64_t plane = paged ? 0 : row * p.max_len;
  const T* kb = static_cast<const T*>(p.k);
  const T* vb = static_cast<const T*>(p.v);

  const int n_steps = (i1 - i0) * (kSpanUnit / kSpanStep);
  for (int st = warp; st < n_steps; st += kSpanWarps) {
    const int t0 = u.unit(i0 + st / (kSpanUnit / kSpanStep)) * kSpanUnit + (st % (kSpanUnit / kSpanStep)) * kSpanStep;
    unsigned ok = 0;  // slots of the step that count
    int64_t r0[kSpanStep];
#pragma unroll
    for (int r = 0; r < kSpanStep; ++r) {
      const int t = t0 + r;
      r0[r] = 0;
      if (v.sees(t)) {
        const int64_t at = paged ? (int64_t)paged_row(p.pm, b, g, t) : plane + t;
        if (at >= 0) {
          r0[r] = at;
          ok |= 1u << r;
        }
      }
    }
    if (ok == 0) continue;
    float4 k4[kSpanStep], v4[kSpanStep];
#pragma unroll
    for (int r = 0; r < kSpanStep; ++r) {
      k4[r] = v4[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if ((ok >> r) & 1u) {
        k4[r] = span_load4(kb + r0[r] * kD + lane * 4);
        v4[r] = span_load4(vb + r0[r] * kD + lane * 4);
      }
    }
    float z[kVals];
#pragma unroll
    for (int r = 0; r < kSpanStep; ++r)
#pragma unroll
      for (int h = 0; h < MG; ++h)
        z[r * MG + h] = q[h][0] * k4[r].x + q[h][1] * k4[r].y + q[h][2] * k4[r].z + q[h][3] * k4[r].w;
    const int first = span_reduce_scatter<kVals>(z, lane);
    const int rz = first / MG, hz = first % MG;  // this lane's slot and first head
    const bool seen = (ok >> rz) & 1u;
    if (p.logits != nullptr && seen) {
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (hz + i < G) p.logits[(row * G + hz + i) * p.ld_logits + t0 + rz] = z[i];
    }
    // the step's probabilities: maxima per head over the step's slots
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kMine; ++i) sm.p[warp][rz][hz + i] = seen ? z[i] : -INFINITY;
    __syncwarp();
#pragma unroll
    for (int h = 0; h < MG; ++h) {
      float mx = m_run[h];
#pragma unroll
      for (int r = 0; r < kSpanStep; ++r) mx = fmaxf(mx, sm.p[warp][r][h]);
      const float sc = m_run[h] == -INFINITY ? 0.0f : exp2f(m_run[h] - mx);
      m_run[h] = mx;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[h][d] *= sc;
      if (lane == 0) sm.sc[warp][h] = sc;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      float mh = -INFINITY;
#pragma unroll
      for (int h = 0; h < MG; ++h)
        if (h == hz + i) mh = m_run[h];
      const float pz = (seen && mh != -INFINITY) ? exp2f(z[i] - mh) : 0.0f;
      l_run[i] = l_run[i] * sm.sc[warp][hz + i] + pz;
      sm.p[warp][rz][hz + i] = pz;
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kSpanStep; ++r)
#pragma unroll
      for (int h = 0; h < MG; ++h) {
        const float pr = sm.p[warp][r][h];
        o[h][0] = __fmaf_rn(pr, v4[r].x, o[h][0]);
        o[h][1] = __fmaf_rn(pr, v4[r].y, o[h][1]);
        o[h][2] = __fmaf_rn(pr, v4[r].z, o[h][2]);
        o[h][3] = __fmaf_rn(pr, v4[r].w, o[h][3]);
      }
  }
  // the warp's sums: lanes with the same head and another slot add up
  {
    constexpr int kCopies = kVals < 32 ? 32 / kVals : 1;  // lanes holding the same value
    __syncwarp();
    // (slot, head) sums to shared memory, then one lane per head adds the slots
    int first = 0, n = kVals;
#pragma unroll
    for (int o2 = 16; o2 >= 1; o2 >>= 1)
      if (n > 1) {
        n >>= 1;
        if (lane & o2) first += n;
      }
    if (lane % kCopies == 0) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) sm.p[warp][first / MG][first % MG + i] = l_run[i];
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < MG; ++h) {
      if (lane == h) {
        float l = 0.0f;
#pragma unroll
        for (int r = 0; r < kSpanStep; ++r) l += sm.p[warp][r][h];
        sm.m[warp][h] = m_run[h];
        sm.l[warp][h] = l;
      }
      *reinterpret_cast<float4*>(&sm.o[warp][h][lane * 4]) = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
    }
  }
  __syncthreads();
  const bool whole = i0 == 0 && i1 == u.n;
  T* out = static_cast<T*>(p.out) + (((int64_t)b * p.n_q + j) * p.n_kv_heads + g) * G * kD;
  float* pp = whole ? nullptr : p.part + (int64_t)slot * (kSpanHead + G * kD);
  for (int e = tid; e < G * kD; e += kSpanThreads) {
    const int h = e / kD, d = e % kD;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSpanWarps; ++w) M = fmaxf(M, sm.m[w][h]);
    float L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kSpanWarps; ++w) {
      const float f = sm.m[w][h] == -INFINITY ? 0.0f : exp2f(sm.m[w][h] - M);
      L += f * sm.l[w][h];
      O += f * sm.o[w][h][d];
    }
    if (whole) {
      store_f(out + e, L == 0.0f ? 0.0f : O / L);
      if (d == 0 && p.rstat != nullptr) {
        p.rstat[row * 2 * G + h] = M;
        p.rstat[row * 2 * G + G + h] = L;
      }
    } else {
      pp[kSpanHead + e] = O;
      if (d == 0) {
        pp[h] = M;
        pp[16 + h] = L;
      }
    }
  }
}

// Grid: n_cta CTAs over the rows' units (decode), or with n_cta 0 one CTA per
// (token, row): x = token, y = row (no partials).
template <typename T, int MG>
__global__ void __launch_bounds__(kSpanThreads) span_cc_kernel(const __grid_constant__ SpanParams p) {
  __shared__ SpanCcSmem<MG> sm;
  grid_dependency_wait();
  if (p.n_cta == 0) {
    const int b = blockIdx.y / p.n_kv_heads, g = blockIdx.y % p.n_kv_heads, j = blockIdx.x;
    const int L = span_len(p, b), nq = span_qlen(p, b);
    if (j >= nq) return;
    const int64_t pos = span_pos0(p, b, L, nq) + j;
    const Span v = span_of(L, pos, p.window, p.n_sink);
    const SpanUnits u = span_units(v, kSpanUnit);
    span_cc_segment<T, MG>(p, sm, b, j, g, v, u, pos, 0, u.n, 0);
    return;
  }
  const int64_t total = span_total<kSpanThreads>(p, sm.scan);
  const int n_cta = span_ctas(total, p.n_cta);
  if ((int)blockIdx.x >= n_cta) return;
  int64_t u0 = span_cut(total, blockIdx.x, n_cta);
  const int64_t u1 = span_cut(total, blockIdx.x + 1, n_cta);
  span_find<kSpanThreads>(p, -1, u0, sm.scan, &sm.where);
  int b = sm.where.b;
  if (b < 0) return;
  int64_t at = u0 - sm.where.base;
  int g = (int)(at / sm.where.units), i0 = (int)(at % sm.where.units);
  for (bool first = true; u0 < u1; first = false) {
    const int L = span_len(p, b);
    const int64_t pos = span_pos0(p, b, L, 1);
    const Span v = span_of(L, pos, p.window, p.n_sink);
    const SpanUnits u = span_units(v, kSpanUnit);
    if (u.n == 0) {  // an empty sequence between others
      ++b;
      g = 0;
      continue;
    }
    const int i1 = (int)min((int64_t)u.n, i0 + (u1 - u0));
    span_cc_segment<T, MG>(p, sm, b, 0, g, v, u, pos, i0, i1, 2 * blockIdx.x + (first ? 0 : 1));
    u0 += i1 - i0;
    i0 = 0;
    if (++g == p.n_kv_heads) {
      g = 0;
      ++b;
    }
  }
}

// ------------------------------------------------------------- the merge

// Grid (rows, G + mass blocks): CTA (row, h) joins head h of a row that
// several CTAs shared, and zeroes the outputs of a row that sees nothing; CTA
// (row, G + x) adds the weights of the row's slots x, x + mass blocks, ... of
// kSpanMassSlots each: mass[t] += sum_h 2^(z_ht - M_h) / L_h.
constexpr int kSpanMassSlots = 1024;

template <typename T>
__global__ void __launch_bounds__(kSpanThreads) span_merge_kernel(const __grid_constant__ SpanParams p) {
  __shared__ int64_t scan[kSpanWarps];
  __shared__ SpanWhere where;
  __shared__ float s_m[16], s_l[16];
  __shared__ __align__(16) float s_o[kSpanWarps][kD];
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group, row = blockIdx.x;
  const int b = row / p.n_kv_heads, g = row % p.n_kv_heads;
  const bool for_out = (int)blockIdx.y < G;
  const int64_t total = span_total<kSpanThreads>(p, scan);
  span_find<kSpanThreads>(p, b, 0, scan, &where);
  const int n = where.units;
  T* out = static_cast<T*>(p.out) + (int64_t)row * G * kD;
  if (n == 0) {
    if (for_out && tid < kD) store_f(out + blockIdx.y * kD + tid, 0.0f);
    return;
  }
  const int64_t ua = where.base + (int64_t)g * n, ub = ua + n;
  const int n_cta = span_ctas(total, p.n_cta);
  const int c0 = n_cta ? span_owner(total, ua, n_cta) : 0, c1 = n_cta ? span_owner(total, ub - 1, n_cta) : 0;
  const int stride = kSpanHead + G * kD;
  // partial i of the row: CTA c0's last segment unless the row opens its run,
  // then one per CTA
  auto part = [&](int c) {
    const bool opens = c > c0 || span_cut(total, c, n_cta) == ua;
    return p.part + (int64_t)(2 * c + (opens ? 0 : 1)) * stride;
  };
  if (for_out) {
    if (c0 == c1) return;  // its CTA wrote the output
    const int h = blockIdx.y;
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, __ldcg(part(c) + h));
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    float L = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = c0 + warp; c <= c1; c += kSpanWarps) {
      const float* pp = part(c);
      const float mc = __ldcg(pp + h);
      const float f = mc == -INFINITY ? 0.0f : exp2f(mc - M);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(pp + kSpanHead + h * kD) + lane);
      L = __fmaf_rn(f, __ldcg(pp + 16 + h), L);
      acc.x = __fmaf_rn(f, x.x, acc.x);
      acc.y = __fmaf_rn(f, x.y, acc.y);
      acc.z = __fmaf_rn(f, x.z, acc.z);
      acc.w = __fmaf_rn(f, x.w, acc.w);
    }
    *reinterpret_cast<float4*>(&s_o[warp][lane * 4]) = acc;
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    float O = 0.0f;
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < kSpanWarps; ++w) {
      O += s_o[w][tid];
      L += s_l[w];
    }
    store_f(out + h * kD + tid, L == 0.0f ? 0.0f : O / L);
    return;
  }
  // the weights: every head's maximum and reciprocal sum, then the slots
  if (c0 == c1) {
    if (tid < G) {
      s_m[tid] = __ldcg(p.rstat + (int64_t)row * 2 * G + tid);
      s_l[tid] = __ldcg(p.rstat + (int64_t)row * 2 * G + G + tid);
    }
  } else {
    for (int h = warp; h < G; h += kSpanWarps) {
      float M = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, __ldcg(part(c) + h));
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
      float L = 0.0f;
      for (int c = c0 + lane; c <= c1; c += 32) {
        const float mc = __ldcg(part(c) + h);
        L += mc == -INFINITY ? 0.0f : exp2f(mc - M) * __ldcg(part(c) + 16 + h);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
      if (lane == 0) {
        s_m[h] = M;
        s_l[h] = L;
      }
    }
  }
  __syncthreads();
  const int L = span_len(p, b);
  const Span v = span_of(L, span_pos0(p, b, L, 1), p.window, p.n_sink);
  const int n_blocks = gridDim.y - G;
  for (int t0 = ((int)blockIdx.y - G) * kSpanMassSlots; t0 < v.hi; t0 += n_blocks * kSpanMassSlots) {
    for (int t = t0 + tid; t < min(v.hi, t0 + kSpanMassSlots); t += kSpanThreads) {
      if (!v.sees(t)) continue;
      if (p.pm.table != nullptr &&
          (unsigned)__ldg(p.pm.table + (int64_t)b * p.pm.max_blocks + (t >> p.pm.log2bs)) >= (unsigned)p.pm.n_pages)
        continue;  // a skipped slot has no logit
      float w = 0.0f;
      for (int h = 0; h < G; ++h) {
        const float z = __ldcg(p.logits + ((int64_t)row * G + h) * p.ld_logits + t);
        if (s_l[h] != 0.0f) w += exp2f(z - s_m[h]) / s_l[h];
      }
      p.mass[row * p.mass_ld + t] += w;
    }
  }
}

}  // namespace fasa
