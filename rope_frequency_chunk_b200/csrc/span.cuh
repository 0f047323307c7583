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
// kernel (float32 decode and short prompts, and caches in host memory) and the
// join of rows that several CTAs shared, which also adds the slots' attention
// weights.
#pragma once

#include "fasa_device.cuh"

namespace fasa {

// Hint: bring a tensor map (a kernel parameter) into the descriptor cache.
__device__ __forceinline__ void prefetch_tensor_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

constexpr int kSpanUnit = 64;      // slots per unit of work
constexpr int kSpanSetup = 2;      // cost of taking up a row (queries, join), in units
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
  int32_t tokens;            // prompts: tokens per CTA of the CUDA-core kernel, tokens * group <= MG
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
  u.n = u.na + (v.lo < v.hi ? max(0, (v.hi + unit - 1) / unit - u.first) : 0);
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
// in float64, so the float32 argument keeps its precision. The angle is off by
// at most 1e-7 + pos * 4e-16 rad: half a step of the float32 argument (2^-26
// turns), and theta, 1 / (2 pi), their product and the turns rounded once each
// in float64 (3.5 * 2^-53 of the angle); 9.3e-7 at position 2^31.
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

// The rows (b, g), in that order, cost kSpanSetup plus their units each (rows
// without units nothing); the total T is dealt to n_cta CTAs in equal runs:
// CTA c owns costs [c T / n, (c + 1) T / n), n = min(n_cta, T / (kSpanSetup +
// 1)), so every run holds a unit. Unit i of a row sits at the row's first cost
// + kSpanSetup + i. A run may begin and end inside a row; such a row's CTAs
// leave partials. Without the setup's weight, the CTA that gets a batch's
// short sequences takes up dozens of rows while the others stream one.
__device__ __forceinline__ int span_ctas(int64_t total, int n_cta) {
  return (int)min((int64_t)n_cta, total / (kSpanSetup + 1));
}
// n equal runs of a total: run c is [cut(c), cut(c + 1)). One 64-bit division
// for all cuts: total = q n + r, so total c / n = c q + c r / n (n < 2^16).
struct SpanDeal {
  int64_t q;
  unsigned r, n;
  float inv;  // n / total
  __device__ __forceinline__ int64_t cut(int c) const { return c * q + (unsigned)c * r / n; }
  __device__ __forceinline__ int owner(int64_t u) const {  // the run that holds u
    int c = min((int)((float)u * inv), (int)n - 1);
    while (cut(c + 1) <= u) ++c;
    while (cut(c) > u) --c;
    return c;
  }
};
__device__ __forceinline__ SpanDeal span_deal(int64_t total, int n) {
  SpanDeal d;
  d.n = (unsigned)max(n, 1);
  d.q = total / d.n;
  d.r = (unsigned)(total - d.q * d.n);
  d.inv = (float)d.n / (float)max(total, (int64_t)1);
  return d;
}
// A sequence's place: its index, the first cost of its KV head 0, the units
// of one of its rows.
struct SpanWhere {
  int64_t base;
  int b, units;
};
__device__ __forceinline__ int span_cost(int units) { return units > 0 ? units + kSpanSetup : 0; }

// The sequences' costs, summed up once per block: thread i's are sequences
// [i q, (i + 1) q), q = ceil(B / 128), and cum[i] is the cost ahead of them.
struct SpanIndex {
  int64_t cum[kSpanThreads + 1];
  int units[kSpanThreads];  // of sequence i, where q is 1
  int64_t scan[kSpanWarps];
};
__device__ __forceinline__ int64_t span_index(const SpanParams& p, SpanIndex& x) {  // returns the total
  const int tid = threadIdx.x, q = (p.batch + kSpanThreads - 1) / kSpanThreads;
  int64_t mine = 0;
  for (int b = tid * q; b < min((tid + 1) * q, p.batch); ++b) {
    const int n = span_seq_units(p, b);
    mine += (int64_t)span_cost(n) * p.n_kv_heads;
    if (q == 1) x.units[tid] = n;
  }
  int64_t before;
  const int64_t total = span_scan<kSpanThreads>(mine, x.scan, before);
  x.cum[tid] = before;
  if (tid == 0) x.cum[kSpanThreads] = total;
  __syncthreads();
  return total;
}
__device__ __forceinline__ int span_units_of(const SpanParams& p, const SpanIndex& x, int b) {
  return p.batch <= kSpanThreads ? x.units[b] : span_seq_units(p, b);
}
// Sequence b, and the sequence that holds cost u < total (a whole warp asks).
__device__ __forceinline__ SpanWhere span_at(const SpanParams& p, const SpanIndex& x, int b) {
  const int q = (p.batch + kSpanThreads - 1) / kSpanThreads;
  SpanWhere w;
  w.b = b / q * q;
  w.base = x.cum[b / q];
  for (w.units = span_units_of(p, x, w.b); w.b < b; w.units = span_units_of(p, x, ++w.b))
    w.base += (int64_t)span_cost(w.units) * p.n_kv_heads;
  return w;
}
__device__ __forceinline__ SpanWhere span_find(const SpanParams& p, const SpanIndex& x, int64_t u) {
  const int q = (p.batch + kSpanThreads - 1) / kSpanThreads, lane = threadIdx.x & 31;
  int n = 0;  // groups that begin at or before u: the last of them holds it (empty ones are ahead of it)
#pragma unroll
  for (int k = 0; k < kSpanThreads / 32; ++k) n += __popc(__ballot_sync(0xFFFFFFFFu, x.cum[k * 32 + lane] <= u));
  // groups behind the last sequence begin at the total, beyond u
  SpanWhere w;
  w.b = (n - 1) * q;
  w.base = x.cum[n - 1];
  for (;; ++w.b) {
    w.units = span_units_of(p, x, w.b);
    const int64_t cost = (int64_t)span_cost(w.units) * p.n_kv_heads;
    if (u < w.base + cost || w.b + 1 >= p.batch) return w;
    w.base += cost;
  }
}

// ------------------------------------------------------- rows seen by no one

// The CTAs of a dealt grid write the zeros of sequences without units.
template <typename T, int NT>
__device__ __forceinline__ void span_zero_rows(const SpanParams& p) {
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (span_seq_units(p, b) != 0) continue;
    const int n = p.n_kv_heads * p.group * kD;
    T* out = static_cast<T*>(p.out) + (int64_t)b * n;
    for (int e = threadIdx.x; e < n; e += NT) store_f(out + e, 0.0f);
  }
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
  double turns[kNFC];
  SpanIndex index;
};

// The rotation table into shared memory. Indexed per thread, the kernel
// parameters are read one address at a time; this runs ahead of the launch
// dependency, which the parameters do not have.
template <int NT>
__device__ __forceinline__ void span_stage_turns(const SpanParams& p, double* turns) {
  for (int i = threadIdx.x; i < kNFC; i += NT) turns[i] = p.turns[i];
}

// The G query rows of n_t tokens (b, j ..), KV head g, token by token: a
// thread's pairs (dims i, i + 64) e = tid, tid + NT, ... of the n_t G * 64,
// loaded (any time ahead) and rotated at positions pos .. and scaled by
// log2(e) / sqrt(128) into qs [n_t G][128].
template <typename T, int NT, int MG>
struct SpanQuery {
  static constexpr int kN = (MG * kNFC + NT - 1) / NT;
  T x[kN], y[kN];
  __device__ __forceinline__ void load(const SpanParams& p, int b, int j, int g, int n_t = 1) {
    const int64_t step = (int64_t)p.n_kv_heads * p.group * kD;  // from token to token
    const T* q = static_cast<const T*>(p.q) + ((int64_t)b * p.n_q + j) * step + (int64_t)g * p.group * kD;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int e = threadIdx.x + n * NT, h = e / kNFC, t = n_t > 1 ? h / p.group : 0;
      if (e < n_t * p.group * kNFC) {
        const T* row = q + t * step + (h - t * p.group) * kD + e % kNFC;
        x[n] = row[0];
        y[n] = row[kNFC];
      }
    }
  }
  __device__ __forceinline__ void rotate(const SpanParams& p, const double* turns, int64_t pos, float* qs,
                                         int n_t = 1) const {
    constexpr float kScale = 1.4426950408889634f * 0.08838834764831845f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int e = threadIdx.x + n * NT, h = e / kNFC, i = e % kNFC, t = n_t > 1 ? h / p.group : 0;
      if (e < n_t * p.group * kNFC) {
        const float a = to_float(x[n]), b = to_float(y[n]);
        float c = 1.0f, s = 0.0f;
        if (!p.q_prerot) span_angle(turns[i], pos + t, &c, &s);
        qs[h * kD + i] = (a * c - b * s) * kScale;
        qs[h * kD + i + kNFC] = (b * c + a * s) * kScale;
      }
    }
  }
};

// One CTA's share of a row, units [i0, i1) of the row's n: the output when
// that is the whole row, else partial `slot`. A prompt's CTA takes n_t tokens
// from j on, so that a slot's K and V serve them all; v is then the union of
// what they see, pos the first one's position.
template <typename T, int MG>
__device__ __forceinline__ void span_cc_segment(const SpanParams& p, SpanCcSmem<MG>& sm, int b, int j, int g,
                                                const Span& v, const SpanUnits& u, int64_t pos, int i0, int i1,
                                                int slot, int L, int n_t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group, R = n_t * G;  // query rows
  const int64_t row = (int64_t)b * p.n_kv_heads + g;
  __syncthreads();  // the previous segment is done with shared memory
  SpanQuery<T, kSpanThreads, MG> raw;
  raw.load(p, b, j, g, n_t);
  raw.rotate(p, sm.turns, pos, &sm.q[0][0], n_t);
  __syncthreads();
  float q[MG][4], o[MG][4];
#pragma unroll
  for (int h = 0; h < MG; ++h)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      q[h][d] = h < R ? sm.q[h][lane * 4 + d] : 0.0f;
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
  // what this lane's rows see (with one token, v itself)
  Span vi[kMine];
  {
    int first = 0, n = kVals;
#pragma unroll
    for (int o2 = 16; o2 >= 1; o2 >>= 1)
      if (n > 1) {
        n >>= 1;
        if (lane & o2) first += n;
      }
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      vi[i] = n_t > 1 ? span_of(L, pos + min((first % MG + i) / G, n_t - 1), p.window, p.n_sink) : v;
  }
  const bool paged = p.pm.table != nullptr;
  const int64_t plane = paged ? 0 : row * p.max_len;
  const T* kb = static_cast<const T*>(p.k);
  const T* vb = static_cast<const T*>(p.v);

  const int n_steps = (i1 - i0) * (kSpanUnit / kSpanStep);
  auto slot_of = [&](int st) {
    return u.unit(i0 + st / (kSpanUnit / kSpanStep)) * kSpanUnit + (st % (kSpanUnit / kSpanStep)) * kSpanStep;
  };
  // requests a step's rows; returns which of its slots count
  auto fetch = [&](int st, float4 (&k4)[kSpanStep], float4 (&v4)[kSpanStep]) -> unsigned {
    unsigned ok = 0;
    if (st >= n_steps) return ok;
    const int t0 = slot_of(st);
#pragma unroll
    for (int r = 0; r < kSpanStep; ++r) {
      const int t = t0 + r;
      k4[r] = v4[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (!v.sees(t)) continue;
      const int64_t at = paged ? (int64_t)paged_row(p.pm, b, g, t) : plane + t;
      if (at < 0) continue;
      ok |= 1u << r;
      k4[r] = span_load4(kb + at * kD + lane * 4);
      v4[r] = span_load4(vb + at * kD + lane * 4);
    }
    return ok;
  };
  // the next step's rows are on their way while one is worked on, where the
  // registers allow
  constexpr bool kAhead = MG <= 4;
  float4 k4[kSpanStep], v4[kSpanStep], kn[kAhead ? kSpanStep : 1], vn[kAhead ? kSpanStep : 1];
  unsigned next_ok = 0;
  if constexpr (kAhead) next_ok = fetch(warp, kn, vn);
  for (int st = warp; st < n_steps; st += kSpanWarps) {
    const int t0 = slot_of(st);
    unsigned ok;  // slots of the step that count
    if constexpr (kAhead) {
      ok = next_ok;
#pragma unroll
      for (int r = 0; r < kSpanStep; ++r) {
        k4[r] = kn[r];
        v4[r] = vn[r];
      }
      next_ok = fetch(st + kSpanWarps, kn, vn);
    } else {
      ok = fetch(st, k4, v4);
    }
    if (ok == 0) continue;
    float z[kVals];
#pragma unroll
    for (int r = 0; r < kSpanStep; ++r)
#pragma unroll
      for (int h = 0; h < MG; ++h)
        z[r * MG + h] = q[h][0] * k4[r].x + q[h][1] * k4[r].y + q[h][2] * k4[r].z + q[h][3] * k4[r].w;
    const int first = span_reduce_scatter<kVals>(z, lane);
    const int rz = first / MG, hz = first % MG;  // this lane's slot and first head
    bool seen[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) seen[i] = ((ok >> rz) & 1u) && vi[i].sees(t0 + rz);
    if (p.logits != nullptr && seen[0]) {
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (hz + i < G) p.logits[(row * G + hz + i) * p.ld_logits + t0 + rz] = z[i];
    }
    // the step's probabilities: maxima per head over the step's slots
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kMine; ++i) sm.p[warp][rz][hz + i] = seen[i] ? z[i] : -INFINITY;
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
      // no maximum yet: -inf logits have no weight, a NaN keeps its own
      const float pz = seen[i] ? exp2f(z[i] - (mh == -INFINITY ? 0.0f : mh)) : 0.0f;
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
  for (int e = tid; e < R * kD; e += kSpanThreads) {
    const int h = e / kD, d = e % kD, t = n_t > 1 ? h / G : 0;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSpanWarps; ++w) M = fmaxf(M, sm.m[w][h]);
    float L_sum = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kSpanWarps; ++w) {
      const float f = sm.m[w][h] == -INFINITY ? 0.0f : exp2f(sm.m[w][h] - M);
      L_sum += f * sm.l[w][h];
      O += f * sm.o[w][h][d];
    }
    if (whole) {
      store_f(out + (int64_t)t * (p.n_kv_heads - 1) * G * kD + e, L_sum == 0.0f ? 0.0f : O / L_sum);
      if (d == 0 && p.rstat != nullptr) {
        p.rstat[row * 2 * G + h] = M;
        p.rstat[row * 2 * G + G + h] = L_sum;
      }
    } else {
      pp[kSpanHead + e] = O;
      if (d == 0) {
        pp[h] = M;
        pp[16 + h] = L_sum;
      }
    }
  }
}

// Grid: n_cta CTAs over the rows' units (decode), or with n_cta 0 one CTA per
// (p.tokens tokens, row): x = tokens, y = row (no partials).
template <typename T, int MG>
__global__ void __launch_bounds__(kSpanThreads) span_cc_kernel(const __grid_constant__ SpanParams p) {
  __shared__ SpanCcSmem<MG> sm;
  span_stage_turns<kSpanThreads>(p, sm.turns);
  grid_dependency_wait();
  if (p.n_cta == 0) {
    const int b = blockIdx.y / p.n_kv_heads, g = blockIdx.y % p.n_kv_heads, j = blockIdx.x * p.tokens;
    const int L = span_len(p, b), nq = span_qlen(p, b);
    if (j >= nq) return;
    const int n_t = min(p.tokens, nq - j);
    const int64_t pos = span_pos0(p, b, L, nq) + j;
    // the union over the tokens: the last one's end and sinks, the first one's window
    Span v = span_of(L, pos, p.window, p.n_sink);
    if (n_t > 1) {
      const Span first = span_of(L, max(pos, (int64_t)0), p.window, p.n_sink);
      v = span_of(L, pos + n_t - 1, p.window, p.n_sink);
      v.lo = min(first.lo, v.hi);
      v.s = min(v.s, v.lo);
    }
    const SpanUnits u = span_units(v, kSpanUnit);
    span_cc_segment<T, MG>(p, sm, b, j, g, v, u, pos, 0, u.n, 0, L, n_t);
    return;
  }
  span_zero_rows<T, kSpanThreads>(p);
  const int64_t total = span_index(p, sm.index);
  const int n_cta = span_ctas(total, p.n_cta);
  if ((int)blockIdx.x >= n_cta) return;
  const SpanDeal deal = span_deal(total, n_cta);
  int64_t u0 = deal.cut(blockIdx.x);
  const int64_t u1 = deal.cut(blockIdx.x + 1);
  const SpanWhere where = span_find(p, sm.index, u0);
  int b = where.b;
  const int64_t at = u0 - where.base;
  int g = (int)(at / span_cost(where.units));
  int a0 = (int)(at % span_cost(where.units));  // cost within the row
  for (bool first = true; u0 < u1;) {
    const int L = span_len(p, b);
    const int64_t pos = span_pos0(p, b, L, 1);
    const Span v = span_of(L, pos, p.window, p.n_sink);
    const SpanUnits u = span_units(v, kSpanUnit);
    if (u.n == 0) {  // an empty sequence between others
      ++b;
      g = 0;
      continue;
    }
    const int a1 = (int)min((int64_t)span_cost(u.n), a0 + (u1 - u0));
    const int i0 = max(a0 - kSpanSetup, 0), i1 = a1 - kSpanSetup;
    if (i1 > i0) span_cc_segment<T, MG>(p, sm, b, 0, g, v, u, pos, i0, i1, 2 * blockIdx.x + (first ? 0 : 1), L, 1);
    first = false;
    u0 += a1 - a0;
    a0 = 0;
    if (++g == p.n_kv_heads) {
      g = 0;
      ++b;
    }
  }
}

// ------------------------------------------------------------- the join

// The last kernel of a call. The warps of CTAs 0 .. n_mass - 1 add the
// attention weights of their run of all rows' units (dealt like the
// attention's, a run per warp):
//   mass[t] += sum_h 2^(z_ht - M_h) / L_h,
// each lane four slots, a float4 per head. The others join rows that several
// CTAs shared: where there are fewer rows than CTAs (by_row) a CTA per row and
// head, a row having many partials; else a CTA per cut between the runs, cut c
// joining the row whose first unit belongs to CTA c - 1.
struct SpanJoinParams {
  SpanParams s;
  int32_t n_mass;
  int32_t by_row;
};

// The CTAs c0 .. c1 that hold a row's units and where their partials are.
struct SpanShare {
  int c0, c1;
  bool opens;  // the row is the first of c0's run
  __device__ __forceinline__ const float* part(const SpanParams& p, int c) const {
    return p.part + (int64_t)(2 * c + (c > c0 || opens ? 0 : 1)) * (kSpanHead + p.group * kD);
  }
};
__device__ __forceinline__ SpanShare span_share(const SpanParams& p, const SpanDeal& d, int64_t row_base, int units) {
  SpanShare w;
  if (p.n_cta == 0) {  // one CTA per row
    w.c0 = w.c1 = 0;
    w.opens = true;
    return w;
  }
  w.c0 = d.owner(row_base + kSpanSetup);
  w.c1 = d.owner(row_base + kSpanSetup + units - 1);
  w.opens = d.cut(w.c0) >= row_base;
  return w;
}

// A warp's sum of head h over partials first, first + step, ...: 2^(m_c - M)
// o_c (four dims per lane) and 2^(m_c - M) l_c, M the maximum over all of the
// row's.
__device__ __forceinline__ float4 span_join(const SpanParams& p, const SpanShare& sh, int h, int first, int step,
                                            int lane, float& L) {
  float M = -INFINITY;
  for (int c = sh.c0 + lane; c <= sh.c1; c += 32) M = fmaxf(M, __ldcg(sh.part(p, c) + h));
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int c = first; c <= sh.c1; c += step) {
    const float* pp = sh.part(p, c);
    const float mc = __ldcg(pp + h);
    const float f = mc == -INFINITY ? 0.0f : exp2f(mc - M);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(pp + kSpanHead + h * kD) + lane);
    L = __fmaf_rn(f, __ldcg(pp + 16 + h), L);
    acc.x = __fmaf_rn(f, x.x, acc.x);
    acc.y = __fmaf_rn(f, x.y, acc.y);
    acc.z = __fmaf_rn(f, x.z, acc.z);
    acc.w = __fmaf_rn(f, x.w, acc.w);
  }
  return acc;
}

template <typename T>
__global__ void __launch_bounds__(kSpanThreads) span_join_kernel(const __grid_constant__ SpanJoinParams jp) {
  const SpanParams& p = jp.s;
  __shared__ SpanIndex index;
  __shared__ float s_l[kSpanWarps];
  __shared__ __align__(16) float s_o[kSpanWarps][kD];
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group;
  const int64_t total = span_index(p, index);
  const SpanDeal deal = span_deal(total, span_ctas(total, p.n_cta));  // the attention's runs

  if ((int)blockIdx.x >= jp.n_mass) {
    const int e = blockIdx.x - jp.n_mass;
    if (jp.by_row) {  // head h of row e / G, a quarter of the partials per warp
      const int h = e % G;
      const int64_t row = e / G;
      const SpanWhere where = span_at(p, index, (int)(row / p.n_kv_heads));
      if (where.units == 0) return;
      const SpanShare sh =
          span_share(p, deal, where.base + (row % p.n_kv_heads) * span_cost(where.units), where.units);
      if (sh.c0 == sh.c1) return;  // its CTA wrote the output
      float L;
      const float4 acc = span_join(p, sh, h, sh.c0 + warp, kSpanWarps, lane, L);
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
      store_f(static_cast<T*>(p.out) + (row * G + h) * kD + tid, L == 0.0f ? 0.0f : O / L);
      return;
    }
    // the row that cut e + 1 goes through, a head per warp: few partials each
    const int n_cta = span_ctas(total, p.n_cta), c = e + 1;
    if (c >= n_cta) return;
    const int64_t cut = deal.cut(c);
    const SpanWhere where = span_find(p, index, cut);
    const int64_t g = (cut - where.base) / span_cost(where.units);
    const int64_t row = (int64_t)where.b * p.n_kv_heads + g, row_base = where.base + g * span_cost(where.units);
    if (cut <= row_base + kSpanSetup) return;                       // its units begin behind the cut
    if (deal.owner(row_base + kSpanSetup) != c - 1) return;         // an earlier cut's
    const SpanShare sh = span_share(p, deal, row_base, where.units);
    for (int h = warp; h < G; h += kSpanWarps) {
      float L;
      const float4 acc = span_join(p, sh, h, sh.c0, 1, lane, L);
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      T* out = static_cast<T*>(p.out) + (row * G + h) * kD + lane * 4;
      store_f(out, acc.x * inv);
      store_f(out + 1, acc.y * inv);
      store_f(out + 2, acc.z * inv);
      store_f(out + 3, acc.w * inv);
    }
    return;
  }

  // the weights of this warp's run
  const int n_run = jp.n_mass * kSpanWarps, run = blockIdx.x * kSpanWarps + warp;
  if (total == 0) return;
  const SpanDeal runs = span_deal(total, n_run);
  int64_t u0 = runs.cut(run);
  const int64_t u1 = runs.cut(run + 1);
  if (u0 >= u1) return;
  const SpanWhere where = span_find(p, index, u0);
  int b = where.b;
  const int64_t at = u0 - where.base;
  const int cost0 = span_cost(where.units);
  int g = (int)(at / cost0), a0 = (int)(at % cost0);
  int64_t row_base = u0 - a0;
  const bool vec = p.mass_ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p.mass) & 15) == 0;
  while (u0 < u1) {
    const int L = span_len(p, b);
    const Span v = span_of(L, span_pos0(p, b, L, 1), p.window, p.n_sink);
    const SpanUnits u = span_units(v, kSpanUnit);
    if (u.n == 0) {
      ++b;
      g = 0;
      continue;
    }
    const int cost = span_cost(u.n);
    const int a1 = (int)min((int64_t)cost, a0 + (u1 - u0));
    const int i0 = max(a0 - kSpanSetup, 0), i1 = a1 - kSpanSetup;
    const int64_t row = (int64_t)b * p.n_kv_heads + g;
    if (i1 > i0) {
      // every head's maximum and reciprocal sum: lane h holds head h's
      const SpanShare sh = span_share(p, deal, row_base, u.n);
      float m_h = -INFINITY, r_h = 0.0f;
      if (sh.c0 == sh.c1) {
        if (lane < G) {
          m_h = __ldcg(p.rstat + row * 2 * G + lane);
          r_h = __ldcg(p.rstat + row * 2 * G + G + lane);
        }
      } else {
        // 32 / gp partials of all heads at a time; the lanes of a head join theirs
        const int gp = G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : G <= 8 ? 8 : 16;
        const int h = lane & (gp - 1);
        for (int c = sh.c0 + lane / gp; c <= sh.c1; c += 32 / gp) {
          if (h >= G) break;
          const float* pp = sh.part(p, c);
          const float m2 = __ldcg(pp + h), l2 = __ldcg(pp + 16 + h);
          const float M = fmaxf(m_h, m2);
          if (M == -INFINITY) continue;
          r_h = r_h * exp2f(m_h - M) + l2 * exp2f(m2 - M);
          m_h = M;
        }
        for (int o = gp; o < 32; o <<= 1) {
          const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m_h, o), l2 = __shfl_xor_sync(0xFFFFFFFFu, r_h, o);
          const float M = fmaxf(m_h, m2);
          if (M != -INFINITY) r_h = r_h * exp2f(m_h - M) + l2 * exp2f(m2 - M);
          m_h = M;
        }
      }
      r_h = r_h == 0.0f ? 0.0f : 1.0f / r_h;
      // 16 lanes a unit, four slots each, two units per lane at a time: all
      // loads of a round are in flight together
      for (int i = i0; i < i1; i += 4) {
        int t[2];
        bool on[2], full[2];
        float4 y[2];
        float w[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int k = i + 2 * j + (lane >> 4);
          t[j] = u.unit(min(k, u.n - 1)) * kSpanUnit + (lane & 15) * 4;
          on[j] = k < i1 && t[j] < v.hi && (t[j] + 4 > v.lo || t[j] < v.s);
          full[j] = vec && t[j] + 4 <= v.hi && (t[j] >= v.lo || t[j] + 4 <= v.s);
          if (on[j] && full[j]) y[j] = *reinterpret_cast<const float4*>(p.mass + row * p.mass_ld + t[j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[j][e] = 0.0f;
        }
        bool there[2] = {true, true};  // slots of a lost page have no logits
        if (p.pm.table != nullptr) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (on[j])
              there[j] = (unsigned)__ldg(p.pm.table + (int64_t)b * p.pm.max_blocks + (t[j] >> p.pm.log2bs)) <
                         (unsigned)p.pm.n_pages;
        }
        for (int h0 = 0; h0 < G; h0 += 4) {
          float4 x[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              x[j][h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (on[j] && h0 + h < G)
                x[j][h] = __ldcg(reinterpret_cast<const float4*>(p.logits + (row * G + h0 + h) * p.ld_logits + t[j]));
            }
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float m = __shfl_sync(0xFFFFFFFFu, m_h, h0 + h), r = __shfl_sync(0xFFFFFFFFu, r_h, h0 + h);
            if (h0 + h >= G) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              w[j][0] = __fmaf_rn(exp2f(x[j][h].x - m), r, w[j][0]);
              w[j][1] = __fmaf_rn(exp2f(x[j][h].y - m), r, w[j][1]);
              w[j][2] = __fmaf_rn(exp2f(x[j][h].z - m), r, w[j][2]);
              w[j][3] = __fmaf_rn(exp2f(x[j][h].w - m), r, w[j][3]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!on[j] || !there[j]) continue;
          float* ms = p.mass + row * p.mass_ld + t[j];
          if (full[j]) {
            *reinterpret_cast<float4*>(ms) =
                make_float4(y[j].x + w[j][0], y[j].y + w[j][1], y[j].z + w[j][2], y[j].w + w[j][3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (v.sees(t[j] + e)) ms[e] += w[j][e];
          }
        }
      }
    }
    u0 += a1 - a0;
    if (a1 == cost) row_base += cost;
    a0 = 0;
    if (++g == p.n_kv_heads) {
      g = 0;
      ++b;
    }
  }
}

}  // namespace fasa
