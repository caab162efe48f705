// Host entry points of the paged 4-bit cache: argument checks and launches.
// The contract (arguments, layout, errors) is in include/sq.h.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "sq_common.cuh"

#include "kv4_append.cuh"
#include "kv4_decode.cuh"
#include "kv4_prefill.cuh"

namespace sq {

sq_status cuda_ok(cudaError_t e);      // SQ_OK, or SQ_ERR_CUDA with the error's name kept for sq_last_error (api.cu)

namespace kv4 {
namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool page_ok(int t) { return t >= 16 && t <= 1024 && (t & (t - 1)) == 0; }
bool strides_ok(int64_t tok, int64_t head) { return tok >= 0 && head >= 0 && tok % 8 == 0 && head % 8 == 0; }

bool cache_ok(const sq_kv4_cache* c) {
  return c->pages && aligned(c->pages, 16) && c->table && aligned(c->table, 4) && c->n_pages >= 1 &&
         c->n_pages <= 0x7fffffff && c->batch >= 1 && c->pages_per_row >= 1 && c->table_stride >= c->pages_per_row &&
         c->n_kv_heads >= 1 && c->n_kv_heads <= 65535 && page_ok(c->page_tokens) &&
         (int64_t)c->pages_per_row * c->page_tokens <= 0x7fffffff;
}

bool rope_ok(const sq_rope* r, int d) {
  return !r || (r->table && aligned(r->table, 16) && r->n_pos >= 1 && r->rot_dim >= 16 && r->rot_dim % 16 == 0 &&
                r->rot_dim <= d);
}

Pool pool_of(const sq_kv4_cache* c) {
  Pool p;
  p.pages = c->pages;
  p.table = c->table;
  p.n_pages = c->n_pages;
  p.table_stride = c->table_stride;
  p.batch = c->batch;
  p.per_row = c->pages_per_row;
  p.n_kv = c->n_kv_heads;
  p.d = c->d;
  p.page_shift = 0;
  while ((1 << p.page_shift) < c->page_tokens) ++p.page_shift;
  return p;
}

RopeArgs rope_of(const sq_rope* r) {
  if (!r) return RopeArgs{nullptr, 0, 0, 0};
  return RopeArgs{r->table, r->n_pos, r->rot_dim, r->interleaved != 0};
}

// ---------------------------------------------------------------- append, read
sq_status stream_args_ok(const sq_kv4_cache* c, const void* k, const void* v, sq_dtype dtype, const StreamArgs& a) {
  if (!c) return SQ_ERR_ARG;
  if (!head_dim_ok(c->d) || (dtype != SQ_F32 && dtype != SQ_F16 && dtype != SQ_BF16)) return SQ_ERR_UNSUPPORTED;
  if (!cache_ok(c) || a.n_tok < 0 || a.n_tok > 0x7fffffff || !a.start || !aligned(a.start, 4) || !aligned(a.cu, 4) ||
      !aligned(a.flags, 4) || !strides_ok(a.ks_tok, a.ks_head) || !strides_ok(a.vs_tok, a.vs_head))
    return SQ_ERR_ARG;
  if (a.n_tok > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16))) return SQ_ERR_ARG;
  return SQ_OK;
}

// Blocks of a stream: tokens, parts of a token.
template <int D> dim3 stream_grid(const Pool& c, int64_t n_tok, Share* sh) {
  *sh = Share::of(2 * c.n_kv, vecs_of_block<D>(), vecs_of_block<D>() / kVecs);
  return dim3((unsigned)((n_tok + sh->toks - 1) / sh->toks), sh->parts);
}

template <typename T, int D>
void launch_append(const Pool& c, const RopeArgs& r, const void* k, const void* v, const StreamArgs& a, cudaStream_t st) {
  Share sh;
  const dim3 grid = stream_grid<D>(c, a.n_tok, &sh);
  if (!r.table)
    k_append4<T, D, 0><<<grid, kStreamThreads, 0, st>>>(c, r, (const T*)k, (const T*)v, a, sh);
  else if (!r.inter && r.rot == D)
    k_append4<T, D, 1><<<grid, kStreamThreads, 0, st>>>(c, r, (const T*)k, (const T*)v, a, sh);
  else
    k_append4<T, D, 2><<<grid, kStreamThreads, 0, st>>>(c, r, (const T*)k, (const T*)v, a, sh);
}

template <typename T, int D>
void launch_read(const Pool& c, void* k, void* v, const StreamArgs& a, cudaStream_t st) {
  Share sh;
  const dim3 grid = stream_grid<D>(c, a.n_tok, &sh);
  k_read4<T, D><<<grid, kStreamThreads, 0, st>>>(c, (T*)k, (T*)v, a, sh);
}

#define SQ_KV4_D(T, CALL)                \
  switch (c.d) {                         \
    case 64: CALL(T, 64); break;         \
    case 128: CALL(T, 128); break;       \
    default: CALL(T, 256); break;        \
  }
#define SQ_KV4_TD(CALL)                              \
  if (dtype == SQ_F32) { SQ_KV4_D(float, CALL) }     \
  else if (dtype == SQ_F16) { SQ_KV4_D(__half, CALL) } \
  else { SQ_KV4_D(__nv_bfloat16, CALL) }

sq_status run_append(const Pool& c, const RopeArgs& r, const void* k, const void* v, sq_dtype dtype,
                     const StreamArgs& a, cudaStream_t st) {
#define SQ_CALL(T, DD) launch_append<T, DD>(c, r, k, v, a, st)
  SQ_KV4_TD(SQ_CALL)
#undef SQ_CALL
  return cuda_ok(cudaGetLastError());
}

sq_status run_read(const Pool& c, void* k, void* v, sq_dtype dtype, const StreamArgs& a, cudaStream_t st) {
#define SQ_CALL(T, DD) launch_read<T, DD>(c, k, v, a, st)
  SQ_KV4_TD(SQ_CALL)
#undef SQ_CALL
  return cuda_ok(cudaGetLastError());
}

// ---------------------------------------------------------------- attention
sq_status attn_args_ok(const sq_kv4_cache* c, int n_q, const void* q, sq_dtype dtype, int64_t s_tok, int64_t s_head,
                       const sq_rope* rope, int window, const void* out, sq_dtype out_dtype, const float* lse,
                       const void* ws, const uint32_t* flags) {
  if (!c) return SQ_ERR_ARG;
  if (!head_dim_ok(c->d) || (dtype != SQ_F16 && dtype != SQ_BF16) ||
      (out_dtype != SQ_F32 && out_dtype != SQ_F16 && out_dtype != SQ_BF16))
    return SQ_ERR_UNSUPPORTED;
  if (!cache_ok(c) || n_q < 1 || n_q > 65535 || n_q % c->n_kv_heads != 0 || !q || !aligned(q, 16) ||
      !strides_ok(s_tok, s_head) || !rope_ok(rope, c->d) || window < 0 || !out || !aligned(out, 16) ||
      !aligned(lse, 4) || !ws || !aligned(ws, 16) || !aligned(flags, 4))
    return SQ_ERR_ARG;
  return SQ_OK;
}

// ---------------------------------------------------------------- single tokens
int sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n < 1) {
    cudaGetLastError();
    return 148;              // a B200's, for size queries on a host without a GPU
  }
  return n;
}

// More than 48 KB of dynamic shared memory has to be asked for, once a kernel and device.
template <typename K> cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done->load() & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit);
  return e;
}

// Launch that may begin before the kernel before it on the stream has ended, and waits for that itself: once that one's
// blocks have all allowed it or ended. The append allows nothing, so behind it only the launch itself is hidden.
template <typename... KA, typename... A>
cudaError_t launch_overlapped(void (*kernel)(KA...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KA(args)...);
}

int head_passes(int group) { return group <= 4 ? 1 : (group + 7) / 8; }

// Blocks: two an SM, fewer where the bound on the lengths leaves less than a block's eight tiles each.
// *whole: no pair has more than a block's tiles and every pair has a block, so none is cut.
int decode_blocks(int batch, int n_kv, int group, int d, int64_t max_ctx, bool* whole) {
  const int tt = d == 256 ? 16 : 32;
  const int64_t tiles = (max_ctx + tt - 1) / tt + 1;
  const int64_t units = (tiles + dec::W - 1) / dec::W;
  const double all = (double)batch * n_kv * head_passes(group) * (double)units;
  const int most = 2 * sms();
  if (whole) *whole = units == 1 && all <= most;
  return all < most ? (int)all : most;
}

size_t decode_ws(int blocks, int d) {
  return (size_t)2 * blocks * dec::part_floats(d) * 4 + (size_t)blocks * (sizeof(dec::Desc) + sizeof(int));
}

template <typename T, typename TO, int D, bool PAIR, bool JOIN>
cudaError_t launch_decode(const Pool& c, const RopeArgs& r, const void* q, void* out, const AttnArgs& a, void* ws,
                          bool step, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kernel = dec::k_decode4<T, TO, D, PAIR, JOIN>;
  cudaError_t e = allow_smem(kernel, dec::Smem<D>::TOTAL, &done);
  if (e != cudaSuccess) return e;
  bool whole = false;
  const int blocks = decode_blocks(c.batch, c.n_kv, a.group, D, std::min<int64_t>(a.max_ctx, (int64_t)c.per_row << c.page_shift), &whole);
  const int nsub = head_passes(a.group);
  float* parts = (float*)ws;
  dec::Desc* descs = (dec::Desc*)(parts + (size_t)2 * blocks * dec::part_floats(D));
  if (step)                                     // behind its append
    e = launch_overlapped(kernel, blocks, 32 * dec::W, dec::Smem<D>::TOTAL, st, c, r, (const T*)q, (TO*)out, a, nsub, parts, descs);
  else
    kernel<<<blocks, 32 * dec::W, dec::Smem<D>::TOTAL, st>>>(c, r, (const T*)q, (TO*)out, a, nsub, parts, descs);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || whole || JOIN) return e;
  const int hs = PAIR ? 4 : 8;
  return launch_overlapped(dec::k_join4<TO, D>, dim3(blocks, std::min(hs, a.group)), 256, 0, st, parts, descs, (TO*)out, a, nsub, hs);
}

sq_status run_decode(const Pool& c, const RopeArgs& r, const void* q, sq_dtype dtype, void* out, sq_dtype out_dtype,
                     const AttnArgs& a, void* ws, bool step, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
#define SQ_CALL3(T, TO, DD, PAIR)                                                         \
  e = a.done ? launch_decode<T, TO, DD, PAIR, true>(c, r, q, out, a, ws, step, st)        \
             : launch_decode<T, TO, DD, PAIR, false>(c, r, q, out, a, ws, step, st)
#define SQ_CALL2(T, TO, DD)                   \
  if (a.group <= 4) SQ_CALL3(T, TO, DD, true); \
  else SQ_CALL3(T, TO, DD, false)
#define SQ_CALL(T, DD)                                       \
  if (out_dtype == SQ_F32) { SQ_CALL2(T, float, DD); }       \
  else if (out_dtype == SQ_F16) { SQ_CALL2(T, __half, DD); } \
  else { SQ_CALL2(T, __nv_bfloat16, DD); }
  if (dtype == SQ_F16) { SQ_KV4_D(__half, SQ_CALL) }
  else { SQ_KV4_D(__nv_bfloat16, SQ_CALL) }
#undef SQ_CALL
#undef SQ_CALL2
#undef SQ_CALL3
  return cuda_ok(e);
}

// ---------------------------------------------------------------- chunks
pre::Shape prefill_shape(int batch, int n_kv, int group, int d, int64_t n_tok) {
  pre::Shape s;
  s.nsub = (group + pre::M - 1) / pre::M;
  s.gt = (group + s.nsub - 1) / s.nsub;
  s.tpm = pre::M / s.gt;
  s.tpu = s.tpm * (d == 256 ? 1 : 2);
  s.sms = sms();
  // A unit is cut when it is longer than an even share or more of all tiles of all units, so fewer than `sms` are, into
  // fewer than 2 `sms` pieces: sum ceil(len / cut) < sum len / cut + sms <= 2 sms.
  s.cap_slots = 2 * s.sms;
  const int64_t units = (int64_t)n_kv * s.nsub * ((n_tok + s.tpu - 1) / s.tpu + batch) + s.cap_slots;
  s.cap_units = units > 0x7fffffff ? 0 : (int)units;
  s.q_tiles = n_tok / s.tpm + batch;
  return s;
}

constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t prefill_layout(const pre::Shape& s, int n_kv, int d, uint8_t* ws, pre::Plan* p) {
  const size_t units = 256, done = units + up256((size_t)s.cap_units * sizeof(pre::Unit));
  const size_t parts = done + up256((size_t)s.cap_slots * sizeof(int));
  const size_t rows = (size_t)s.cap_slots * pre::part_rows(d == 256 ? 1 : 2);
  const size_t q = parts + up256(rows * (d + 2) * sizeof(float));
  const size_t image = d == 64 ? pre::Cfg<64>::QIMG : d == 128 ? pre::Cfg<128>::QIMG : pre::Cfg<256>::QIMG;
  if (p)
    *p = pre::Plan{(pre::Head*)ws, (pre::Unit*)(ws + units), (int*)(ws + done), (float*)(ws + parts), ws + q, s.q_tiles};
  return q + (size_t)n_kv * s.nsub * s.q_tiles * image;
}

template <typename T, typename TO, int D>
cudaError_t launch_prefill(const Pool& c, const RopeArgs& r, const void* q, void* out, const AttnArgs& a, const pre::Shape& s,
                           const pre::Plan& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kernel = pre::k_prefill4<TO, D>;
  constexpr int smem = pre::Cfg<D>::TOTAL;
  cudaError_t e = allow_smem(kernel, smem, &done);
  if (e != cudaSuccess) return e;
  const int64_t items = a.n_tok * ((a.n_q + pre::kQHeads - 1) / pre::kQHeads), per = pre::kPlanThreads / (D / 16);
  const unsigned blocks = 1 + (unsigned)std::min<int64_t>((items + per - 1) / per, 8 * s.sms);
  constexpr int plan = sizeof(pre::PlanSmem);
  static_assert(plan <= 48 * 1024, "within what needs no asking for");
  if (!r.table)
    pre::k_prepare4<T, D, 0><<<blocks, pre::kPlanThreads, plan, st>>>(c, r, (const T*)q, a, s, p);
  else if (!r.inter && r.rot == D)
    pre::k_prepare4<T, D, 1><<<blocks, pre::kPlanThreads, plan, st>>>(c, r, (const T*)q, a, s, p);
  else
    pre::k_prepare4<T, D, 2><<<blocks, pre::kPlanThreads, plan, st>>>(c, r, (const T*)q, a, s, p);
  e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_overlapped(kernel, s.cap_units, pre::Cfg<D>::THREADS, smem, st, c, r, (TO*)out, a, s, p);
  return e;
}

sq_status run_prefill(const Pool& c, const RopeArgs& r, const void* q, sq_dtype dtype, void* out, sq_dtype out_dtype,
                      const AttnArgs& a, const pre::Shape& s, uint8_t* ws, cudaStream_t st) {
  pre::Plan p;
  prefill_layout(s, c.n_kv, c.d, ws, &p);
  cudaError_t e = cudaSuccess;
#define SQ_CALL(T, DD)                                                                           \
  if (out_dtype == SQ_F32) e = launch_prefill<T, float, DD>(c, r, q, out, a, s, p, st);          \
  else if (out_dtype == SQ_F16) e = launch_prefill<T, __half, DD>(c, r, q, out, a, s, p, st);    \
  else e = launch_prefill<T, __nv_bfloat16, DD>(c, r, q, out, a, s, p, st)
  if (dtype == SQ_F16) { SQ_KV4_D(__half, SQ_CALL) }
  else { SQ_KV4_D(__nv_bfloat16, SQ_CALL) }
#undef SQ_CALL
  return cuda_ok(e);
}

float scale_of(float scale, int d) { return scale > 0.0f ? scale : 1.0f / sqrtf((float)d); }

}  // namespace
}  // namespace kv4
}  // namespace sq

using namespace sq;
using namespace sq::kv4;

extern "C" {

size_t sq_kv4_page_bytes(int n_kv_heads, int d, int page_tokens) {
  if (n_kv_heads < 1 || n_kv_heads > 65535 || !head_dim_ok(d) || !page_ok(page_tokens)) return 0;
  return (size_t)n_kv_heads * (page_tokens / 16) * blk_bytes(d);
}

sq_status sq_kv4_append(const sq_kv4_cache* cache, const void* k, const void* v, sq_dtype dtype, int64_t k_stride_tok,
                        int64_t k_stride_head, int64_t v_stride_tok, int64_t v_stride_head, int64_t n_tok,
                        const int32_t* d_cu, const int32_t* d_start, const sq_rope* rope, uint32_t* d_flags,
                        sq_stream stream) {
  const StreamArgs a{d_cu, d_start, n_tok, k_stride_tok, k_stride_head, v_stride_tok, v_stride_head, d_flags, nullptr, 0};
  sq_status s = stream_args_ok(cache, k, v, dtype, a);
  if (s != SQ_OK) return s;
  if (!rope_ok(rope, cache->d)) return SQ_ERR_ARG;
  if (n_tok == 0) return SQ_OK;
  return run_append(pool_of(cache), rope_of(rope), k, v, dtype, a, (cudaStream_t)stream);
}

sq_status sq_kv4_read(const sq_kv4_cache* cache, void* k_out, void* v_out, sq_dtype dtype, int64_t k_stride_tok,
                      int64_t k_stride_head, int64_t v_stride_tok, int64_t v_stride_head, int64_t n_tok,
                      const int32_t* d_cu, const int32_t* d_start, uint32_t* d_flags, sq_stream stream) {
  const StreamArgs a{d_cu, d_start, n_tok, k_stride_tok, k_stride_head, v_stride_tok, v_stride_head, d_flags, nullptr, 0};
  sq_status s = stream_args_ok(cache, k_out, v_out, dtype, a);
  if (s != SQ_OK) return s;
  if (n_tok == 0) return SQ_OK;
  return run_read(pool_of(cache), k_out, v_out, dtype, a, (cudaStream_t)stream);
}

size_t sq_kv4_attn_workspace(int batch, int n_q_heads, int n_kv_heads, int d, int64_t max_ctx) {
  if (batch < 1 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads != 0 || !head_dim_ok(d) || max_ctx < 1)
    return 0;
  return decode_ws(decode_blocks(batch, n_kv_heads, n_q_heads / n_kv_heads, d, max_ctx, nullptr), d);
}

sq_status sq_kv4_attn_decode(const sq_kv4_cache* cache, const int32_t* d_seq_lens, int n_q_heads, int64_t max_ctx,
                             const void* q, sq_dtype dtype, int64_t q_stride_row, int64_t q_stride_head,
                             const sq_rope* rope, float scale, int window, void* out, sq_dtype out_dtype,
                             float* lse_out, void* ws, size_t ws_bytes, uint32_t* d_flags, sq_stream stream) {
  sq_status s = attn_args_ok(cache, n_q_heads, q, dtype, q_stride_row, q_stride_head, rope, window, out, out_dtype,
                             lse_out, ws, d_flags);
  if (s != SQ_OK) return s;
  if (!d_seq_lens || !aligned(d_seq_lens, 4) || max_ctx < 1) return SQ_ERR_ARG;
  if (ws_bytes < sq_kv4_attn_workspace(cache->batch, n_q_heads, cache->n_kv_heads, cache->d, max_ctx))
    return SQ_ERR_WORKSPACE;
  const AttnArgs a{nullptr, d_seq_lens, -1, cache->batch, max_ctx, q_stride_row, q_stride_head, n_q_heads,
                   n_q_heads / cache->n_kv_heads, window, scale_of(scale, cache->d), lse_out, d_flags, nullptr};
  return run_decode(pool_of(cache), rope_of(rope), q, dtype, out, out_dtype, a, ws, false, (cudaStream_t)stream);
}

sq_status sq_kv4_decode_step(const sq_kv4_cache* cache, const void* k, const void* v, const void* q, sq_dtype dtype,
                             int64_t k_stride_tok, int64_t k_stride_head, int64_t v_stride_tok, int64_t v_stride_head,
                             int64_t q_stride_row, int64_t q_stride_head, const int32_t* d_pos, int n_q_heads,
                             int64_t max_ctx, const sq_rope* rope, float scale, int window, void* out,
                             sq_dtype out_dtype, float* lse_out, void* ws, size_t ws_bytes, uint32_t* d_flags,
                             sq_stream stream) {
  sq_status s = attn_args_ok(cache, n_q_heads, q, dtype, q_stride_row, q_stride_head, rope, window, out, out_dtype,
                             lse_out, ws, d_flags);
  if (s != SQ_OK) return s;
  StreamArgs ap{nullptr, d_pos, cache->batch, k_stride_tok, k_stride_head, v_stride_tok, v_stride_head, d_flags, nullptr, 0};
  s = stream_args_ok(cache, k, v, dtype, ap);
  if (s != SQ_OK) return s;
  if (max_ctx < 1) return SQ_ERR_ARG;
  if (ws_bytes < sq_kv4_attn_workspace(cache->batch, n_q_heads, cache->n_kv_heads, cache->d, max_ctx))
    return SQ_ERR_WORKSPACE;
  const Pool c = pool_of(cache);
  const RopeArgs r = rope_of(rope);
  const int group = n_q_heads / cache->n_kv_heads;
  const int blocks = decode_blocks(c.batch, c.n_kv, group, c.d, max_ctx, nullptr);
  // Where the step leaves most of the GPU idle, a launch is what it can save (one sequence, 2 KV heads, 501 tokens:
  // 25.3 us a call and its read back with a kernel that joins, 23.6 without); a full one ends sooner with the
  // kernel (four sequences, 8 KV heads, 8192 tokens: 30.7 against 32.1 us).
  int* done = nullptr;
  if (blocks < 2 * sms()) {
    done = (int*)((uint8_t*)ws + decode_ws(blocks, c.d)) - blocks;
    ap.zero = done;
    ap.n_zero = blocks;
  }
  s = run_append(c, r, k, v, dtype, ap, (cudaStream_t)stream);
  if (s != SQ_OK) return s;
  const AttnArgs a{nullptr, d_pos, 0, cache->batch, max_ctx, q_stride_row, q_stride_head, n_q_heads,
                   group, window, scale_of(scale, cache->d), lse_out, d_flags, done};
  return run_decode(c, r, q, dtype, out, out_dtype, a, ws, true, (cudaStream_t)stream);
}

size_t sq_kv4_attn_prefill_workspace(int batch, int n_q_heads, int n_kv_heads, int d, int64_t n_tok) {
  if (batch < 1 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads != 0 || !head_dim_ok(d) || n_tok < 1 ||
      n_tok > 0x7fffffff)
    return 0;
  const pre::Shape s = prefill_shape(batch, n_kv_heads, n_q_heads / n_kv_heads, d, n_tok);
  return s.cap_units ? prefill_layout(s, n_kv_heads, d, nullptr, nullptr) : 0;
}

sq_status sq_kv4_attn_prefill(const sq_kv4_cache* cache, const int32_t* d_cu, const int32_t* d_start, int n_q_heads,
                              int64_t n_tok, const void* q, sq_dtype dtype, int64_t q_stride_tok,
                              int64_t q_stride_head, const sq_rope* rope, float scale, int window, void* out,
                              sq_dtype out_dtype, float* lse_out, void* ws, size_t ws_bytes, uint32_t* d_flags,
                              sq_stream stream) {
  if (n_tok == 0 && cache && d_cu && d_start) return SQ_OK;
  sq_status s = attn_args_ok(cache, n_q_heads, q, dtype, q_stride_tok, q_stride_head, rope, window, out, out_dtype,
                             lse_out, ws, d_flags);
  if (s != SQ_OK) return s;
  if (!d_cu || !aligned(d_cu, 4) || !d_start || !aligned(d_start, 4) || n_tok < 1 || n_tok > 0x7fffffff)
    return SQ_ERR_ARG;
  if (ws_bytes < sq_kv4_attn_prefill_workspace(cache->batch, n_q_heads, cache->n_kv_heads, cache->d, n_tok))
    return SQ_ERR_WORKSPACE;
  const AttnArgs a{d_cu, d_start, 0, n_tok, 0x7fffffff, q_stride_tok, q_stride_head, n_q_heads,
                   n_q_heads / cache->n_kv_heads, window, scale_of(scale, cache->d), lse_out, d_flags, nullptr};
  const pre::Shape sh = prefill_shape(cache->batch, cache->n_kv_heads, a.group, cache->d, n_tok);
  if (!sh.cap_units) return SQ_ERR_ARG;
  return run_prefill(pool_of(cache), rope_of(rope), q, dtype, out, out_dtype, a, sh, (uint8_t*)ws, (cudaStream_t)stream);
}

}  // extern "C"
