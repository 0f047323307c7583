// Append kernel: rotate new keys at their absolute positions, store K and V,
// and write the dominant-FC sketch rows.
//
// "FASA: Frequency-aware Sparse Attention" (gist.science technical summary,
// §2 "A Descoberta": RoPE splits a head into 2-D frequency chunks, each with
// its own angular frequency; FAC bullet 3: tokens keep their original
// absolute positions). A key is rotated exactly once, here, at its slot's
// position, so a later gather of the row needs no re-rotation.
//
// Grid: x = blocks of kAppendTok tokens, y = groups of `heads_per_cta`
// consecutive (b, g) rows. cos/sin of a token block are computed once in
// float64 and reused across the CTA's heads (recomputed per sequence when
// every sequence appends at its own position). Slots are addressed through
// a PageMap, so the same kernel fills contiguous and paged caches. After an
// eviction slots are no longer positions: the first slot then comes apart
// from the first position, and the slots' positions and weights are set too.
#pragma once

#include "fasa_device.cuh"

namespace fasa {

constexpr int kAppendTok = 8;
constexpr int kAppendThreads = 256;

struct AppendParams {
  const void* k_new;     // [B*Hkv][n_new][128]
  const void* v_new;
  void* k;               // [B*Hkv][max_len][128]
  void* v;
  void* sketch;          // [B*Hkv][max_len][stride]
  const int32_t* dom_idx;  // [Hkv][n_dom]
  int64_t max_len;
  int32_t n_rows;        // B*Hkv
  int32_t n_kv_heads;
  int32_t n_new;
  int32_t pos0;
  int32_t n_dom;
  int32_t stride;
  int32_t heads_per_cta;
  const int32_t* pos0v;  // [B] each sequence's first new position, or null: pos0 for all
  const int32_t* slot0v; // [B] each sequence's first new slot, or null: slots are positions
  int32_t* slot_pos;     // [B*Hkv][max_len] the new slots' positions, or null
  float* mass;           // [B*Hkv][max_len] zeroed at the new slots, or null
  PageMap pm;            // paged pools, or pm.table null: [B*Hkv][max_len] planes
  double theta[kNFC];    // base^(-2i/128), computed on the host in float64
};

// Two neighbouring elements of a row, one load or store.
template <typename T>
struct alignas(2 * sizeof(T)) Two {
  T v[2];
};

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  __shared__ double s_cos[kAppendTok][kNFC];
  __shared__ double s_sin[kAppendTok][kNFC];
  __shared__ __align__(16) T s_row[kAppendTok][kD];
  __shared__ int s_dom[kNFC];
  __shared__ int64_t s_dst[kAppendTok];  // each token's row in the K / V / sketch planes, or -1
  __shared__ double s_theta[kNFC];

  const int tid = threadIdx.x;
  const int tok0 = blockIdx.x * kAppendTok;
  const int ntok = min(kAppendTok, p.n_new - tok0);
  const int row0 = blockIdx.y * p.heads_per_cta;
  const int row1 = min(p.n_rows, row0 + p.heads_per_cta);

  // a copy in shared memory: indexed per thread, the kernel parameters are
  // read one address at a time
  if (tid < kNFC) s_theta[tid] = p.theta[tid];
  __syncthreads();
  auto angles = [&](int pos) {
    for (int e = tid; e < ntok * kNFC; e += kAppendThreads) {
      const int t = e / kNFC, i = e % kNFC;
      const double ang = (double)(pos + tok0 + t) * s_theta[i];
      double s, c;
      sincos(ang, &s, &c);
      s_cos[t][i] = c;
      s_sin[t][i] = s;
    }
  };
  int cur = p.pos0v ? -1 : p.pos0;  // the position that s_cos is for (-1: none yet)
  if (!p.pos0v) angles(cur);

  for (int row = row0; row < row1; ++row) {
    const int b = row / p.n_kv_heads, g = row % p.n_kv_heads;
    int pos = p.pos0, slot = p.pos0;
    if (p.pos0v) {
      pos = __ldg(p.pos0v + b);
      slot = p.slot0v ? __ldg(p.slot0v + b) : pos;
      // block-uniform: skip the row
      if (pos < 0 || slot < 0 || (int64_t)slot + p.n_new > p.max_len || (int64_t)pos + p.n_new > INT32_MAX) {
        if (tid == 0 && blockIdx.x == 0) flag_status(FASA_ERR_BAD_INDEX);
        continue;
      }
      if (pos != cur) {
        __syncthreads();  // the previous row is done with the angles
        angles(pos);
        cur = pos;
      }
    }
    // this row's inputs are on their way while the block gets ready: a thread
    // takes two FCs of a token's key (dims i, i + 1, i + 64, i + 65) and
    // 16-byte vectors of its values
    const T* kin = static_cast<const T*>(p.k_new) + ((int64_t)row * p.n_new + tok0) * kD;
    const T* vin = static_cast<const T*>(p.v_new) + ((int64_t)row * p.n_new + tok0) * kD;
    constexpr int kVecRow = kD * (int)sizeof(T) / 16;  // 16-byte vectors per row
    static_assert(kAppendTok * kNFC / 2 == kAppendThreads && kAppendTok * kVecRow <= kAppendThreads,
                  "one pair of FCs and at most one vector per thread");
    const int kt = tid / (kNFC / 2), ki = tid % (kNFC / 2) * 2, vt = tid / kVecRow;
    Two<T> lo, hi;
    uint4 val = make_uint4(0, 0, 0, 0);
    if (kt < ntok) {
      lo = *reinterpret_cast<const Two<T>*>(kin + kt * kD + ki);
      hi = *reinterpret_cast<const Two<T>*>(kin + kt * kD + ki + kNFC);
    }
    if (vt < ntok) val = reinterpret_cast<const uint4*>(vin)[tid];
    __syncthreads();  // s_cos ready; previous row done with s_row / s_dom / s_dst
    if (tid < ntok) {
      const int t = slot + tok0 + tid;
      const int64_t at = (int64_t)row * p.max_len + t;
      const int64_t dst = p.pm.table ? (int64_t)paged_row(p.pm, b, g, t) : at;
      s_dst[tid] = dst;
      if (dst >= 0) {
        if (p.slot_pos) p.slot_pos[at] = pos + tok0 + tid;
        if (p.mass) p.mass[at] = 0.0f;
      }
    }
    if (tid < p.n_dom) {
      int d = p.dom_idx[g * p.n_dom + tid];
      if (d < 0 || d >= kNFC) {
        flag_status(FASA_ERR_BAD_INDEX);
        d = -1;
      }
      s_dom[tid] = d;
    }
    T* kc = static_cast<T*>(p.k);
    T* vc = static_cast<T*>(p.v);
    T* sk = static_cast<T*>(p.sketch);
    __syncthreads();  // s_dst ready

    // RoPE of FC i: (x, y) -> (x cos - y sin, y cos + x sin), float64, no
    // contraction, one rounding to the cache dtype.
    if (kt < ntok) {
      Two<T> xo, yo;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const double x = to_float(lo.v[f]), y = to_float(hi.v[f]);
        const double c = s_cos[kt][ki + f], s = s_sin[kt][ki + f];
        round_store(&xo.v[f], __dsub_rn(__dmul_rn(x, c), __dmul_rn(y, s)));
        round_store(&yo.v[f], __dadd_rn(__dmul_rn(y, c), __dmul_rn(x, s)));
      }
      const int64_t dst = s_dst[kt];
      if (dst >= 0) {
        *reinterpret_cast<Two<T>*>(kc + dst * kD + ki) = xo;
        *reinterpret_cast<Two<T>*>(kc + dst * kD + ki + kNFC) = yo;
      }
      *reinterpret_cast<Two<T>*>(&s_row[kt][ki]) = xo;
      *reinterpret_cast<Two<T>*>(&s_row[kt][ki + kNFC]) = yo;
    }
    // values are stored as given
    if (vt < ntok) {
      const int64_t dst = s_dst[vt];
      if (dst >= 0) reinterpret_cast<uint4*>(vc + dst * kD)[tid % kVecRow] = val;
    }
    __syncthreads();
    // sketch row: dims (dom[j], dom[j]+64) at 2j, 2j+1, zero padding
    for (int e = tid; e < ntok * p.stride; e += kAppendThreads) {
      const int t = e / p.stride, c = e % p.stride, j = c >> 1;
      T val = T(0.0f);
      if (j < p.n_dom) {
        const int d = s_dom[j];
        if (d >= 0) val = s_row[t][d + (c & 1) * kNFC];
      }
      const int64_t dst = s_dst[t];
      if (dst >= 0) sk[dst * p.stride + c] = val;
    }
  }
}

}  // namespace fasa
