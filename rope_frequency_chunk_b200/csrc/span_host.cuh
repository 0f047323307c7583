// Host side of the span attention (fasa_attend_decode, fasa_attend_prompt),
// the eviction (fasa_evict) and the append to slots (fasa_append_kv_at):
// argument checks before any launch, launch shapes, workspaces. Included by
// fasa.cu, whose helpers it uses.
#pragma once

namespace {

fasa_status check_span(const fasa_cache* c, const fasa_span* sp) {
  if (sp == nullptr || !aligned(sp->seq_len, 4)) return FASA_ERR_INVALID_ARG;
  if (sp->q_pos != nullptr && !aligned(sp->q_pos, 4)) return FASA_ERR_INVALID_ARG;
  if (sp->q_len != nullptr && !aligned(sp->q_len, 4)) return FASA_ERR_INVALID_ARG;
  if (sp->max_seq_len < 1 || sp->window < 0 || sp->n_sink < 0 || (sp->q_prerotated != 0 && sp->q_prerotated != 1))
    return FASA_ERR_INVALID_ARG;
  if (sp->max_seq_len > c->max_len) return FASA_ERR_CAPACITY;
  return FASA_OK;
}

// Units of kSpanUnit slots that a row can have: its visible slots' units, the
// window's cut at both ends.
int64_t span_max_units(const fasa_span* sp) {
  int64_t n = ceil_div(sp->max_seq_len, kSpanUnit);
  if (sp->window > 0)
    n = std::min<int64_t>(n, ceil_div(sp->n_sink, kSpanUnit) + ceil_div(sp->window, kSpanUnit) + 1);
  return n;
}

// Rows of up to this many units are one CTA's work each: no partials, and no
// second launch to join them. One CTA a row against units dealt to all CTAs, us
// on the GPU over cold caches (32/8 heads): 256 bf16 slots of 1, 8, 64 sequences
// 7.6, 8.2, 21.8 against 10.7, 12.2, 27.3; 256 float32 slots 16.2, 16.9, 40.8
// against 19.9, 21.6, 54.8. For few sequences the two meet at 384 (float32) to
// 512 (bf16) slots and part fast (1024: 18.7 against 12.0, 53 against 21). 64
// equally long ones would gain from one CTA at any length (2048 slots 88
// against 99), but the lengths are the device's and a batch of unequal ones
// would wait for its longest.
constexpr int kSpanWholeUnits = 4;
constexpr int kSpanMaxPerSm = 4;  // resident CTAs per SM, an upper bound

struct SpanWs {
  int64_t max_cta;  // CTAs the units can be dealt to, 0 when every row is one CTA's
  int64_t ld_logits;
  size_t part, rstat, logits, total;
};
SpanWs span_layout(const fasa_cache* c, const fasa_span* sp, bool with_mass) {
  SpanWs w;
  const int64_t rows = (int64_t)c->batch * c->n_kv_heads, units = span_max_units(sp);
  const int64_t G = c->n_q_heads / c->n_kv_heads;
  w.max_cta = units <= kSpanWholeUnits ? 0 : std::min<int64_t>((int64_t)kAssumedMaxSms * kSpanMaxPerSm, rows * units);
  w.ld_logits = ((int64_t)sp->max_seq_len + 31) / 32 * 32;
  w.part = 0;
  w.rstat = al256((size_t)(2 * w.max_cta * (kSpanHead + G * kD)) * 4);
  w.logits = w.rstat + (with_mass ? al256((size_t)(rows * 2 * G) * 4) : 0);
  w.total = w.logits + (with_mass ? al256((size_t)(rows * G * w.ld_logits) * 4) : 0);
  return w;
}

void span_fill(SpanParams& p, const fasa_cache* c, const fasa_paged* pg, const fasa_span* sp, const void* q,
               void* out, int32_t n_q) {
  p.k = c->k;
  p.v = c->v;
  p.q = q;
  p.out = out;
  p.seq_len = sp->seq_len;
  p.q_pos = sp->q_pos;
  p.q_len = sp->q_len;
  p.max_len = c->max_len;
  p.max_seq_len = sp->max_seq_len;
  p.window = sp->window;
  p.n_sink = sp->n_sink;
  p.q_prerot = sp->q_prerotated;
  p.n_q = n_q;
  p.tokens = 1;
  p.batch = c->batch;
  p.n_kv_heads = c->n_kv_heads;
  p.group = c->n_q_heads / c->n_kv_heads;
  p.pm = page_map(c, pg);
  fill_theta(p.turns, c->rope_base);
  for (int i = 0; i < kNFC; ++i) p.turns[i] *= 0.15915494309189535;  // 1 / (2 pi)
}

struct SpanCc {
  const void* fn;
  void (*kern)(const SpanParams);
};
// G: query rows of a CTA.
template <typename T>
SpanCc span_cc_pick(int G) {
  if (G == 1) return {(const void*)span_cc_kernel<T, 1>, span_cc_kernel<T, 1>};
  if (G == 2) return {(const void*)span_cc_kernel<T, 2>, span_cc_kernel<T, 2>};
  if (G <= 4) return {(const void*)span_cc_kernel<T, 4>, span_cc_kernel<T, 4>};
  if (G <= 8) return {(const void*)span_cc_kernel<T, 8>, span_cc_kernel<T, 8>};
  return {(const void*)span_cc_kernel<T, 16>, span_cc_kernel<T, 16>};
}

fasa_status span_cc_launch(SpanParams& p, int dtype, dim3 grid, cudaStream_t st) {
  const int rows = p.group * p.tokens;
  const SpanCc k = dtype == FASA_F32 ? span_cc_pick<float>(rows) : span_cc_pick<__nv_bfloat16>(rows);
  return launch_pdl(k.kern, grid, kSpanThreads, 0, st, p);
}

// Rows of the K (and V) tensor: every (b, g) plane, or every page.
int64_t span_rows(const fasa_cache* c, const fasa_paged* pg) {
  return pg != nullptr ? (int64_t)pg->n_pages * c->n_kv_heads * pg->block_size
                       : (int64_t)c->batch * c->n_kv_heads * c->max_len;
}

// The tensor-core kernels read K and V with TMA: bf16 caches in device
// memory, rows within the 32-bit coordinates. Others take the CUDA-core one.
bool span_tensor_cores(const fasa_cache* c, const fasa_paged* pg) {
  return c->dtype == FASA_BF16 && span_rows(c, pg) < INT32_MAX && !host_resident(c->k) && !host_resident(c->v);
}

// float32 prompts: the tiled kernel, or the CUDA-core one. A tile takes the
// same time however many of its 64 rows hold queries, the CUDA-core kernel's
// time goes with the query rows per SM: the tiles win from 18 rows per SM and
// wave of tiles on. Over 2000 slots (tiles, CUDA cores): 300 tokens 8/8 heads
// (16 rows per SM) 312, 296 us; 100 tokens 28/4 heads (19) 312, 331 us; 96 and
// 128 tokens 32/8 heads (21, 28) 312, 340 us; 64 tokens (14) 312, 173 us; 16 x
// 16 and 16 x 32 tokens 8/8 heads (14, 28) 314, 196 and 317, 360 us.
constexpr int64_t kTiRowsPerSm = 18;
bool span_tiled(const SpanParams& p, const DevInfo& d) {
  const int64_t rows = (int64_t)p.batch * p.n_kv_heads;
  const int64_t waves = ceil_div(ceil_div(p.n_q, kTiRows / p.group) * rows, d.sms);
  return rows * p.group * p.n_q >= kTiRowsPerSm * waves * d.sms;
}
fasa_status launch_tile(const SpanParams& p, cudaStream_t st) {
  int set = 0;
  fasa_status s = cached_int((const void*)span_tile_kernel, 0, &set, [&](int* v) {
    *v = 1;
    return cuda_status(
        cudaFuncSetAttribute(span_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(TiSmem)));
  });
  if (s != FASA_OK) return s;
  const dim3 grid((unsigned)ceil_div(p.n_q, kTiRows / p.group), (unsigned)(p.batch * p.n_kv_heads), 1);
  return launch_pdl(span_tile_kernel, grid, kTiThreads, sizeof(TiSmem), st, p);
}

// A bf16 tensor read in boxes stored for the 128-byte swizzle (64 elements
// wide); rows out of range read as zeros. strides: bytes, of dimensions 1 ..
fasa_status span_encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                        const cuuint32_t* box) {
  static std::atomic<void*> encode{nullptr};
  void* fn = encode.load(std::memory_order_acquire);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found);
    if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || fn == nullptr)
      return cuda_status(e == cudaSuccess ? cudaErrorNotSupported : e);
    encode.store(fn, std::memory_order_release);
  }
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn)(
      m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FASA_OK : cuda_status(cudaErrorInvalidValue);
}
// [n_rows][128] in boxes of box_rows x 64, or (halves) of box_rows rows' two
// 64-column halves one behind the other.
fasa_status span_map(CUtensorMap* m, const void* base, int64_t n_rows, int box_rows, bool halves) {
  const cuuint64_t dims[3] = {(cuuint64_t)(halves ? kD / 2 : kD), (cuuint64_t)n_rows, 2};
  const cuuint64_t strides[2] = {kD * 2, kD};  // a row, half a row
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 2};
  return span_encode(m, base, halves ? 3 : 2, dims, strides, box);
}
// Queries [n_tokens][Hq][128] in boxes of `tokens` x G x 64.
fasa_status span_map_q(CUtensorMap* m, const void* q, int64_t n_tokens, int hq, int group, int tokens) {
  const cuuint64_t dims[3] = {kD, (cuuint64_t)hq, (cuuint64_t)n_tokens};
  const cuuint64_t strides[2] = {kD * 2, (cuuint64_t)hq * kD * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
  return span_encode(m, q, 3, dims, strides, box);
}

// Work items of a prompt call and the parts their blocks are cut into: one
// part while the items fill half the SMs or more; else enough parts to fill
// them, each with four blocks or more, 32 at most (a lane of the join each).
// Uncut and cut, 32/8 heads: 5 queries on 8192 slots 150, 23 us, 64 on 65536
// 1216, 99, 256 on 4096 86, 40. Parts of two, four and eight blocks or more: 1
// query on 1024 slots 13, 18, 24 us; 64 on 8192 33, 32, 39; 2 x 99 on 512 24,
// 19, 19 (uncut: 19).
struct PromptPlan {
  int64_t tiles, items;  // per (b, g) row; of all rows and parts
  int splits;
  size_t bytes;
};
PromptPlan prompt_layout(const fasa_cache* c, const fasa_span* sp, int32_t n_q, int sms) {
  PromptPlan w;
  const int64_t G = c->n_q_heads / c->n_kv_heads, rows = (int64_t)c->batch * c->n_kv_heads;
  w.tiles = ceil_div(n_q, 2 * pr_tokens((int)G));
  int64_t blocks = ceil_div(sp->max_seq_len, kPrBlock);
  if (sp->window > 0)
    blocks = std::min<int64_t>(blocks, ceil_div(sp->n_sink, kPrBlock) +
                                           ceil_div((int64_t)sp->window + ceil_div(kPrRows, G), kPrBlock) + 1);
  const int64_t items = w.tiles * rows;
  w.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(sms / items, blocks / 4), kPrMaxSplits));
  w.items = items * w.splits;
  w.bytes = 256 + (w.splits > 1 ? (size_t)(w.items * kPrPart) * 4 : 0);
  return w;
}

template <int TERMS>
fasa_status launch_prompt_t(const PromptParams& p, int grid, cudaStream_t st) {
  auto kern = span_prompt_kernel<TERMS>;
  constexpr int smem = (int)PrSmem<TERMS>::kBytes;
  int set = 0;
  fasa_status s = cached_int((const void*)kern, 0, &set, [&](int* v) {
    *v = 1;
    return cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  });
  if (s != FASA_OK) return s;
  return launch_pdl(kern, dim3((unsigned)grid, 1, 1), kPrThreads, smem, st, p);
}

fasa_status launch_prompt(const fasa_cache* c, const fasa_paged* pg, const fasa_span* sp, const void* q, int32_t n_q,
                          void* out, void* workspace, const DevInfo& d, cudaStream_t st) {
  PromptParams p{};
  span_fill(p.s, c, pg, sp, q, out, n_q);
  const PromptPlan w = prompt_layout(c, sp, n_q, std::min(d.sms, kAssumedMaxSms));
  if (w.items > INT32_MAX / 2) return FASA_ERR_UNSUPPORTED;
  p.n_items = (int32_t)w.items;
  p.tiles_max = (int32_t)w.tiles;
  p.splits = w.splits;
  p.box_rows = pg != nullptr ? std::min(pg->block_size, kPrBlock) : kPrBlock;
  p.n_rows = (int32_t)span_rows(c, pg);
  p.part = static_cast<float*>(workspace);
  fasa_status s;
  if ((s = span_map(&p.map_k, c->k, p.n_rows, p.box_rows, false)) != FASA_OK) return s;
  if ((s = span_map(&p.map_v, c->v, p.n_rows, p.box_rows, false)) != FASA_OK) return s;
  const int64_t n_tokens = (int64_t)c->batch * n_q;
  if (n_tokens > INT32_MAX) return FASA_ERR_UNSUPPORTED;
  if (p.s.q_prerot &&
      (s = span_map_q(&p.map_q, q, n_tokens, c->n_q_heads, p.s.group, pr_tokens(p.s.group))) != FASA_OK)
    return s;
  const int grid = (int)std::min<int64_t>(w.items, d.sms);
  s = p.s.q_prerot ? launch_prompt_t<1>(p, grid, st) : launch_prompt_t<2>(p, grid, st);
  if (s != FASA_OK || w.splits == 1) return s;
  const dim3 mgrid((unsigned)ceil_div((int64_t)n_q * p.s.group, 4), (unsigned)(c->batch * c->n_kv_heads), 1);
  return launch_pdl(span_prompt_merge_kernel, mgrid, 128, 0, st, p);
}

// One token per sequence: the tensor-core kernel where it can read the cache,
// else the CUDA-core one, over n_cta CTAs (0: one per row).
struct SpanDecodeKernel {
  const void* fn;
  int smem;
};
SpanDecodeKernel span_decode_pick(int dtype, bool tc, int G) {
  if (tc)
    return G <= 8 ? SpanDecodeKernel{(const void*)span_decode_kernel<8>, SdSmem<8>::kBytes}
                  : SpanDecodeKernel{(const void*)span_decode_kernel<16>, SdSmem<16>::kBytes};
  return {dtype == FASA_F32 ? span_cc_pick<float>(G).fn : span_cc_pick<__nv_bfloat16>(G).fn, 0};
}
fasa_status launch_span_decode(const fasa_cache* c, const fasa_paged* pg, SpanParams& p, bool tc, dim3 grid,
                               cudaStream_t st) {
  if (!tc) return span_cc_launch(p, c->dtype, grid, st);
  SpanDecodeParams q{};
  q.s = p;
  const int64_t n_rows = span_rows(c, pg);
  fasa_status s;
  if ((s = span_map(&q.map_k, c->k, n_rows, kSdRows, true)) != FASA_OK) return s;
  if ((s = span_map(&q.map_v, c->v, n_rows, kSdRows, true)) != FASA_OK) return s;
  grid = dim3(grid.x * grid.y, 1, 1);
  return p.group <= 8 ? launch_pdl(span_decode_kernel<8>, grid, kSpanThreads, SdSmem<8>::kBytes, st, q)
                      : launch_pdl(span_decode_kernel<16>, grid, kSpanThreads, SdSmem<16>::kBytes, st, q);
}

fasa_status check_mass(const float* mass) { return aligned(mass, 4) ? FASA_OK : FASA_ERR_INVALID_ARG; }

}  // namespace

extern "C" {

size_t fasa_attend_decode_workspace_bytes(const fasa_cache* c, const fasa_span* sp, int32_t with_mass) {
  if (check_cache(c) != FASA_OK || check_span(c, sp) != FASA_OK) return 0;
  return span_layout(c, sp, with_mass != 0).total + 256;
}

fasa_status fasa_attend_decode(const fasa_cache* c, const fasa_paged* pg, const fasa_span* sp, const void* q,
                               void* out, float* mass, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  fasa_status s = check_cache(c);
  if (s != FASA_OK) return s;
  if (pg != nullptr && (s = check_paged(c, pg)) != FASA_OK) return s;
  if ((s = check_span(c, sp)) != FASA_OK) return s;
  if (!aligned(q, 16) || !aligned(out, 16)) return FASA_ERR_INVALID_ARG;
  if (mass != nullptr && (s = check_mass(mass)) != FASA_OK) return s;
  const SpanWs w = span_layout(c, sp, mass != nullptr);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total + 256) return FASA_ERR_WORKSPACE;
  DevInfo d;
  if ((s = device_info(&d)) != FASA_OK) return s;
  SpanParams p{};
  span_fill(p, c, pg, sp, q, out, 1);
  p.q_len = nullptr;
  p.pos_at_len = 1;
  const int rows = c->batch * c->n_kv_heads;
  char* base = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(base + w.part);
  if (mass != nullptr) {
    p.mass = mass;
    p.mass_ld = c->max_len;
    p.rstat = reinterpret_cast<float*>(base + w.rstat);
    p.logits = reinterpret_cast<float*>(base + w.logits);
    p.ld_logits = w.ld_logits;
  }
  const bool tc = span_tensor_cores(c, pg);
  const SpanDecodeKernel k = span_decode_pick(c->dtype, tc, p.group);
  int per_sm = 0;
  if ((s = cached_int(k.fn, 7, &per_sm, [&](int* v) {
         cudaError_t e = cudaSuccess;
         if (k.smem > 0) e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
         if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, k.fn, kSpanThreads, (size_t)k.smem);
         return cuda_status(e);
       })) != FASA_OK)
    return s;
  per_sm = std::min(std::max(per_sm, 1), kSpanMaxPerSm);
  dim3 grid(1, (unsigned)rows, 1);
  if (w.max_cta > 0) {
    p.n_cta = (int)std::min<int64_t>((int64_t)per_sm * d.sms, w.max_cta);
    grid = dim3((unsigned)p.n_cta, 1, 1);
  }
  if ((s = launch_span_decode(c, pg, p, tc, grid, stream)) != FASA_OK) return s;
  if (p.n_cta == 0 && mass == nullptr) return FASA_OK;
  SpanJoinParams jp{};
  jp.s = p;
  jp.by_row = rows < p.n_cta ? 1 : 0;
  // about four CTAs per SM over the units that the rows can have
  if (mass != nullptr)
    jp.n_mass = (int)std::max<int64_t>(1, std::min<int64_t>(4LL * d.sms, ceil_div(rows * span_max_units(sp), 4)));
  const int64_t joins = p.n_cta == 0 ? 0 : jp.by_row ? (int64_t)rows * p.group : p.n_cta - 1;
  const dim3 jgrid((unsigned)(jp.n_mass + joins), 1, 1);
  if (jgrid.x == 0) return FASA_OK;
  return c->dtype == FASA_F32 ? launch_pdl(span_join_kernel<float>, jgrid, kSpanThreads, 0, stream, jp)
                              : launch_pdl(span_join_kernel<__nv_bfloat16>, jgrid, kSpanThreads, 0, stream, jp);
}

size_t fasa_attend_prompt_workspace_bytes(const fasa_cache* c, const fasa_span* sp, int32_t n_q) {
  if (check_cache(c) != FASA_OK || check_span(c, sp) != FASA_OK || n_q < 1) return 0;
  // the largest over 1 .. n_q queries: fewer of them make fewer items, which
  // are cut into more parts. Sizes go by tiles per row, and parts only exist
  // while the items fill half the SMs or fewer.
  const int per = 2 * pr_tokens(c->n_q_heads / c->n_kv_heads);
  const int64_t rows = (int64_t)c->batch * c->n_kv_heads;
  size_t bytes = prompt_layout(c, sp, n_q, kAssumedMaxSms).bytes;
  for (int64_t t = 1; t * rows * 2 <= kAssumedMaxSms && t * per < n_q; ++t)
    bytes = std::max(bytes, prompt_layout(c, sp, (int32_t)(t * per), kAssumedMaxSms).bytes);
  return bytes;
}

fasa_status fasa_attend_prompt(const fasa_cache* c, const fasa_paged* pg, const fasa_span* sp, const void* q,
                               int32_t n_q, void* out, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  fasa_status s = check_cache(c);
  if (s != FASA_OK) return s;
  if (pg != nullptr && (s = check_paged(c, pg)) != FASA_OK) return s;
  if ((s = check_span(c, sp)) != FASA_OK) return s;
  if (n_q < 1 || !aligned(q, 16) || !aligned(out, 16)) return FASA_ERR_INVALID_ARG;
  if (n_q > FASA_MAX_LEN) return FASA_ERR_UNSUPPORTED;
  // what this call uses, which may be less than the size for up to n_q queries
  const size_t need = prompt_layout(c, sp, n_q, kAssumedMaxSms).bytes;
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need) return FASA_ERR_WORKSPACE;
  DevInfo d;
  if ((s = device_info(&d)) != FASA_OK) return s;
  if (span_tensor_cores(c, pg)) return launch_prompt(c, pg, sp, q, n_q, out, workspace, d, stream);
  SpanParams p{};
  span_fill(p, c, pg, sp, q, out, n_q);
  if (c->dtype == FASA_F32 && span_tiled(p, d)) return launch_tile(p, stream);
  // Tokens share a CTA, up to 8 query rows, while there are more CTAs than run
  // at once (two per SM): a CTA of more rows takes longer (one, two, four, eight
  // rows 44, 50, 64, 81 us over 1000 float32 slots), a second round takes as
  // long again. 8/8 heads, apart and shared: 32 tokens 44, 81 us; 64 tokens 83,
  // 51; 150 tokens 184, 85; one token of 64 sequences over 500 slots 57, 103.
  // Over the host link the reads are what counts: always (8/8 heads, 1000 bf16
  // slots: 2 tokens 392, 350 us; 8 tokens 675, 377; 40 tokens 3300, 470).
  const int64_t rows = (int64_t)c->batch * c->n_kv_heads;
  const bool host = host_resident(c->k) || host_resident(c->v);
  while (2 * p.tokens * p.group <= 8 && p.tokens < n_q && (host || ceil_div(n_q, p.tokens) * rows > 2LL * d.sms))
    p.tokens *= 2;
  const dim3 grid((unsigned)ceil_div(n_q, p.tokens), (unsigned)rows, 1);
  return span_cc_launch(p, c->dtype, grid, stream);
}

fasa_status fasa_append_kv_at(const fasa_cache* c, const fasa_paged* pg, const void* k_new, const void* v_new,
                              int32_t n_new, const int32_t* slot0, const int32_t* pos0, int32_t* slot_pos,
                              float* mass, cudaStream_t stream) {
  fasa_status s = check_cache(c);
  if (s != FASA_OK) return s;
  if (pg != nullptr && (s = check_paged(c, pg)) != FASA_OK) return s;
  if (n_new < 0 || !aligned(slot0, 4) || !aligned(pos0, 4)) return FASA_ERR_INVALID_ARG;
  if (slot_pos != nullptr && !aligned(slot_pos, 4)) return FASA_ERR_INVALID_ARG;
  if (mass != nullptr && !aligned(mass, 4)) return FASA_ERR_INVALID_ARG;
  if (n_new > c->max_len) return FASA_ERR_CAPACITY;
  if (n_new == 0) return FASA_OK;
  if (!aligned(k_new, 16) || !aligned(v_new, 16)) return FASA_ERR_INVALID_ARG;
  DevInfo d;
  if ((s = device_info(&d)) != FASA_OK) return s;
  return launch_append(c, k_new, v_new, n_new, 0, pos0, pg, d, stream, slot0, slot_pos, mass);
}

}  // extern "C"

namespace {

fasa_status check_evict(const fasa_cache* c, const fasa_evict_desc* e) {
  if (e == nullptr || !aligned(e->seq_len, 4) || !aligned(e->cur_pos, 4)) return FASA_ERR_INVALID_ARG;
  if (e->max_seq_len < 1 || e->budget < 1 || e->n_sink < 0 || e->n_recent < 0) return FASA_ERR_INVALID_ARG;
  if ((int64_t)e->n_sink + e->n_recent > e->budget) return FASA_ERR_INVALID_ARG;
  if (e->max_seq_len > c->max_len) return FASA_ERR_CAPACITY;
  if (e->max_seq_len > FASA_MAX_LEN) return FASA_ERR_UNSUPPORTED;
  return FASA_OK;
}

// Whether two arrays share memory without being the same one.
bool entangled(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != y && (x > y ? x - y : y - x) < bytes;
}

// The selection's own warps move the rows while each has one batch at most and
// all rows' CTAs run at once; else the moves are a launch of their own. One
// launch against two, us on the GPU over cold caches: 64 rows of 8 moves 8.3,
// 8.9; of 32 11.7, 10.7; of 128 13.2, 12.2; 8 rows of 256 18.5, 11.3, of 1024
// 42.6, 24.2; 512 rows of 20 24.8, 18.6. The second launch costs the host 2.2
// us: eager calls of up to 128 moves a row take 11.1 to 12.2 us against 13.5.
bool evict_moves_here(int rows, int max_moves, int sms) {
  return max_moves <= kEvWarps * kEvBatch && rows <= 2 * sms;
}

// A kept slot behind the budget fills a hole before it: at most the smaller
// of the two sides.
int32_t evict_max_moves(const fasa_evict_desc* e) {
  return std::max(1, std::min(e->budget, e->max_seq_len - std::min(e->budget, e->max_seq_len)));
}

}  // namespace

extern "C" {

size_t fasa_evict_workspace_bytes(const fasa_cache* c, const fasa_evict_desc* e) {
  if (check_cache(c) != FASA_OK || check_evict(c, e) != FASA_OK) return 0;
  const size_t rows = (size_t)c->batch * c->n_kv_heads;
  return al256(rows * 4) + al256(rows * 2 * evict_max_moves(e) * 4);
}

fasa_status fasa_evict(const fasa_cache* c, const fasa_paged* pg, const fasa_evict_desc* e, const float* mass,
                       const int32_t* slot_pos, float* mass_out, int32_t* slot_pos_out, int32_t* len_out,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fasa_status s = check_cache(c);
  if (s != FASA_OK) return s;
  if (pg != nullptr && (s = check_paged(c, pg)) != FASA_OK) return s;
  if ((s = check_evict(c, e)) != FASA_OK) return s;
  if (span_rows(c, pg) > INT32_MAX) return FASA_ERR_UNSUPPORTED;  // rows are addressed with 32-bit indices
  if (!aligned(mass, 4) || !aligned(slot_pos, 4) || !aligned(mass_out, 4) || !aligned(slot_pos_out, 4) ||
      !aligned(len_out, 4))
    return FASA_ERR_INVALID_ARG;
  // every row of a sequence reads its length and position while one of them
  // writes the new length; shifted outputs would overwrite other rows' inputs
  const size_t per_seq = (size_t)c->batch * 4, per_slot = (size_t)c->batch * c->n_kv_heads * c->max_len * 4;
  if (len_out == e->seq_len || len_out == e->cur_pos || entangled(len_out, e->seq_len, per_seq) ||
      entangled(len_out, e->cur_pos, per_seq) || entangled(mass_out, mass, per_slot) ||
      entangled(slot_pos_out, slot_pos, per_slot))
    return FASA_ERR_INVALID_ARG;
  const size_t need = fasa_evict_workspace_bytes(c, e);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need) return FASA_ERR_WORKSPACE;
  DevInfo d;
  if ((s = device_info(&d)) != FASA_OK) return s;
  EvictParams p{};
  p.k = c->k;
  p.v = c->v;
  p.sketch = c->sketch;
  p.seq_len = e->seq_len;
  p.cur_pos = e->cur_pos;
  p.mass = mass;
  p.slot_pos = slot_pos;
  p.mass_out = mass_out;
  p.slot_pos_out = slot_pos_out;
  p.len_out = len_out;
  const int rows = c->batch * c->n_kv_heads;
  p.moves = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + al256((size_t)rows * 4));
  p.max_len = c->max_len;
  p.max_seq_len = e->max_seq_len;
  p.budget = e->budget;
  p.n_sink = e->n_sink;
  p.n_recent = e->n_recent;
  p.n_kv_heads = c->n_kv_heads;
  p.max_moves = evict_max_moves(e);
  p.row16 = kD * elem_bytes(c->dtype) / 16;
  p.sk16 = c->sketch_stride * elem_bytes(c->dtype) / 16;
  p.pm = page_map(c, pg);
  if (!evict_moves_here(rows, p.max_moves, d.sms)) p.n_moves = static_cast<int32_t*>(workspace);
  // CTAs per row: enough for a CTA's share of the keys to fit, more while the
  // rows leave SMs idle and a CTA's share stays above 2048 slots
  int C = pow2ceil(ceil_div(e->max_seq_len, kEvMaxChunk));
  while (C < kMaxCluster && (int64_t)rows * C * 2 <= d.sms && ceil_div(e->max_seq_len, 2 * C) >= 2048) C *= 2;
  p.chunk = (int)(ceil_div(ceil_div(e->max_seq_len, C), 32) * 32);
  p.clusters = C;
  const size_t smem = (size_t)(2 * kEvBins + (C > 1 ? 2 * kEvBins : 0) + p.chunk) * 4;
  int set = 0;
  if ((s = cached_int((const void*)evict_kernel, 1, &set, [&](int* v) {
         cudaError_t er = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (4 * kEvBins + kEvMaxChunk) * 4);
         if (er == cudaSuccess) er = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
         *v = 1;
         return cuda_status(er);
       })) != FASA_OK)
    return s;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3((unsigned)C, (unsigned)rows, 1);
  cfg.blockDim = dim3(kEvThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((s = cuda_status(cudaLaunchKernelEx(&cfg, evict_kernel, p))) != FASA_OK || p.n_moves == nullptr) return s;
  const int64_t batches = ceil_div(p.max_moves, 8 * kEvBatch);  // CTAs of 8 warps
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(batches, ceil_div(8LL * d.sms, rows))),
                  (unsigned)rows, 1);
  return launch_pdl(evict_move_kernel, grid, 256, 0, stream, p);
}

}  // extern "C"
