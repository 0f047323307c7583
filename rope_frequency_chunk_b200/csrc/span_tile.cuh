// Span attention of prompts over float32 caches: tiles of 64 query rows by 64
// slots on CUDA cores.
//
// float32 keys have no exact tensor-core product, so S = Q K^T and O += P V run
// on the FMA pipe, 4 * 128 flops per visible (query, slot) pair and head. A
// tile's rows are 64 / G whole tokens' G heads. Each of 256 threads keeps 4 x 4
// values of S (rows 4 y .. 4 y + 3, columns x + 16 j) and 4 x 8 of O; operands
// come from shared memory as float4, 12 wavefronts for 64 FMAs in S and 20 for
// 128 in P V, so the FMA pipe is what bounds the inner loops. The 16 threads of
// a row are half a warp: maxima and sums go by shuffles and P needs no block
// barrier. V is copied in while S is computed and the next K while P V is.
#pragma once

#include "attend_mma.cuh"
#include "span.cuh"

namespace fasa {

constexpr int kTiRows = 64;
constexpr int kTiThreads = 256;
constexpr int kTiStride = kD + 4;            // floats of a Q or K row: float4 reads of 8 rows hit every bank once
constexpr int kTiP = kSpanUnit + 4;

struct TiSmem {
  float q[kTiRows][kTiStride];
  float k[kSpanUnit][kTiStride];
  float v[kSpanUnit][kD];
  float p[kTiRows][kTiP];
  double turns[kNFC];
  int ok[kSpanUnit];  // the block's slots that lie in a page and that some row sees
};

__global__ void __launch_bounds__(kTiThreads, 1) span_tile_kernel(const __grid_constant__ SpanParams p) {
  extern __shared__ __align__(16) unsigned char ti_smem[];
  TiSmem& sm = *reinterpret_cast<TiSmem*>(ti_smem);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = p.group, tt = kTiRows / G;  // tokens of a tile
  span_stage_turns<kTiThreads>(p, sm.turns);
  grid_dependency_wait();
  const int row = blockIdx.y, b = row / p.n_kv_heads, g = row % p.n_kv_heads;
  const int L = span_len(p, b), nq = span_qlen(p, b);
  const int j0 = (int)(gridDim.x - 1 - blockIdx.x) * tt;  // the longest tiles first
  if (j0 >= nq) return;
  const int n_t = min(tt, nq - j0);
  const int64_t pos = span_pos0(p, b, L, nq) + j0;
  // the union of what the tile sees: the last token's end and sinks, the first one's window
  const Span first = span_of(L, max(pos, (int64_t)0), p.window, p.n_sink);
  Span all = span_of(L, pos + n_t - 1, p.window, p.n_sink);
  all.lo = min(first.lo, all.hi);
  all.s = min(all.s, all.lo);
  const SpanUnits u = span_units(all, kSpanUnit);
  const float* kb = static_cast<const float*>(p.k);
  const float* vb = static_cast<const float*>(p.v);
  const bool paged = p.pm.table != nullptr;
  // requests rows of block i: 16-byte copies, four rows' worth per warp step;
  // slots that nobody sees, or without a page, are zeros
  auto request = [&](int i, const float* base, float* dst, int stride, bool mark) {
    const int t0 = u.unit(i) * kSpanUnit;
#pragma unroll
    for (int e = tid; e < kSpanUnit * (kD / 4); e += kTiThreads) {
      const int r = e / (kD / 4), c = e % (kD / 4), t = t0 + r;
      int64_t at = -1;
      if (all.sees(t)) at = paged ? (int64_t)paged_row(p.pm, b, g, t) : (int64_t)row * p.max_len + t;
      am_cp16(smem_u32(dst + r * stride + c * 4), base + (at < 0 ? 0 : at) * kD + c * 4, at < 0 ? 0u : 16u);
      if (mark && c == 0) sm.ok[r] = at >= 0;
    }
    cp_async_commit();
  };
  __syncthreads();  // the rotation table
  if (u.n > 0) request(0, kb, &sm.k[0][0], kTiStride, true);
  {  // the tile's queries, rotated and scaled by log2(e) / sqrt(128)
    constexpr float kScale = 1.4426950408889634f * 0.08838834764831845f;
    const int64_t step = (int64_t)p.n_kv_heads * G * kD;
    const float* q = static_cast<const float*>(p.q) + ((int64_t)b * p.n_q + j0) * step + (int64_t)g * G * kD;
    for (int e = tid; e < kTiRows * kNFC; e += kTiThreads) {
      const int r = e / kNFC, i = e % kNFC, t = r / G;
      float x = 0.0f, y = 0.0f, c = 1.0f, s = 0.0f;
      if (t < n_t) {
        const float* src = q + t * step + (r - t * G) * kD + i;
        x = src[0];
        y = src[kNFC];
        if (!p.q_prerot) span_angle(sm.turns[i], pos + t, &c, &s);
      }
      sm.q[r][i] = (x * c - y * s) * kScale;
      sm.q[r][i + kNFC] = (y * c + x * s) * kScale;
    }
  }
  Span v[4];
  float m[4], l[4], o[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (ty * 4 + i) / G;
    v[i] = span_of(L, t < n_t ? pos + t : -1, p.window, p.n_sink);
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[i][d] = 0.0f;
  }
  for (int blk = 0; blk < u.n; ++blk) {
    const int t0 = u.unit(blk) * kSpanUnit;
    cp_async_wait<0>();
    __syncthreads();  // K is here for everyone, and everyone is done with V
    request(blk, vb, &sm.v[0][0], kD, false);
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < kD; d += 4) {
      float4 a[4], c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&sm.q[ty * 4 + i][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = __fmaf_rn(a[i].x, c[j].x, s[i][j]);
          s[i][j] = __fmaf_rn(a[i].y, c[j].y, s[i][j]);
          s[i][j] = __fmaf_rn(a[i].z, c[j].z, s[i][j]);
          s[i][j] = __fmaf_rn(a[i].w, c[j].w, s[i][j]);
        }
    }
    bool ok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) ok[j] = sm.ok[tx + 16 * j] != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!ok[j] || !v[i].sees(t0 + tx + 16 * j)) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
      const float f = m[i] == -INFINITY ? 0.0f : exp2f(m[i] - mx), off = mx == -INFINITY ? 0.0f : mx;
      m[i] = mx;
      l[i] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - off);
        l[i] += e;
        sm.p[ty * 4 + i][tx + 16 * j] = e;
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) o[i][d] *= f;
    }
    cp_async_wait<0>();
    __syncthreads();  // V is here for everyone, and everyone is done with K; P's rows are the half warp's own
    if (blk + 1 < u.n) request(blk + 1, kb, &sm.k[0][0], kTiStride, true);
#pragma unroll 2
    for (int k = 0; k < kSpanUnit; k += 4) {
      float4 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&sm.p[ty * 4 + i][k]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float4 c0 = *reinterpret_cast<const float4*>(&sm.v[k + kk][tx * 4]);
        const float4 c1 = *reinterpret_cast<const float4*>(&sm.v[k + kk][64 + tx * 4]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
          o[i][0] = __fmaf_rn(w, c0.x, o[i][0]);
          o[i][1] = __fmaf_rn(w, c0.y, o[i][1]);
          o[i][2] = __fmaf_rn(w, c0.z, o[i][2]);
          o[i][3] = __fmaf_rn(w, c0.w, o[i][3]);
          o[i][4] = __fmaf_rn(w, c1.x, o[i][4]);
          o[i][5] = __fmaf_rn(w, c1.y, o[i][5]);
          o[i][6] = __fmaf_rn(w, c1.z, o[i][6]);
          o[i][7] = __fmaf_rn(w, c1.w, o[i][7]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i, t = r / G;
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], k);
    if (t >= n_t) continue;
    const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
    float* out = static_cast<float*>(p.out) + (((int64_t)b * p.n_q + j0 + t) * p.n_kv_heads + g) * G * kD +
                 (r - t * G) * kD;
    *reinterpret_cast<float4*>(out + tx * 4) =
        make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
    *reinterpret_cast<float4*>(out + 64 + tx * 4) =
        make_float4(o[i][4] * inv, o[i][5] * inv, o[i][6] * inv, o[i][7] * inv);
  }
}

}  // namespace fasa
