// C entry points of the serving operators: argument validation and dispatch.
// As in api.hip, every check runs on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <math.h>

#include "lqmm.h"
#include "lqmm_internal.hpp"

namespace {

using lqmm::ElemType;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
// Index arrays (positions, slots, page tables, lengths) and lse may start
// anywhere in a buffer that a server keeps: natural alignment is enough.
bool aligned_to(const void *p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }
bool dim_ok(int64_t v) { return v > 0 && v <= LQMM_MAX_DIM; }
bool head_dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 256; }
bool page_size_ok(int64_t p) { return p >= 8 && p <= 1024 && (p & (p - 1)) == 0; }
constexpr int64_t kMaxHeads = 65536;

int log2_of(int64_t v) {
  int n = 0;
  while (((int64_t)1 << n) < v) ++n;
  return n;
}

bool elem_type(int t, ElemType *e) {
  switch (t) {
    case LQMM_F32: *e = ElemType::F32; return true;
    case LQMM_F16: *e = ElemType::F16; return true;
    case LQMM_BF16: *e = ElemType::BF16; return true;
  }
  return false;
}
int elem_bytes(ElemType e) { return e == ElemType::F32 ? 4 : 2; }

// A row stride of at least `width` elements, a multiple of 16 bytes.
lqmm_status stride_ok(int64_t ld, int64_t width, ElemType e) {
  if (ld < width || ld > LQMM_MAX_DIM) return LQMM_ERR_SHAPE;
  return ld * elem_bytes(e) % 16 == 0 ? LQMM_OK : LQMM_ERR_ALIGN;
}

lqmm_status done(hipError_t e) { return e == hipSuccess ? LQMM_OK : LQMM_ERR_LAUNCH; }

// What an append checks of its pointers, sizes and strides, and its arguments
// (without the caches' element type).
lqmm_status append_args(lqmm::KvAppend &a, ElemType in, const void *q, const void *k, const void *v,
                        int64_t ldq, int64_t ldk, int64_t ldv, const int32_t *positions,
                        const int64_t *slots, const uint64_t *rope_turns, int64_t rotary_dim,
                        int interleaved, void *q_out, void *k_cache, void *v_cache, int64_t tokens,
                        int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, int64_t page_size,
                        int64_t num_pages) {
  if (!dim_ok(tokens) || !dim_ok(num_pages) || !head_dim_ok(head_dim) || !page_size_ok(page_size))
    return LQMM_ERR_SHAPE;
  if (n_q_heads < 0 || n_q_heads > kMaxHeads || n_kv_heads <= 0 || n_kv_heads > kMaxHeads)
    return LQMM_ERR_SHAPE;
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16 != 0) return LQMM_ERR_SHAPE;
  lqmm_status st;
  if (n_q_heads != 0 && (st = stride_ok(ldq, n_q_heads * head_dim, in)) != LQMM_OK) return st;
  if ((st = stride_ok(ldk, n_kv_heads * head_dim, in)) != LQMM_OK) return st;
  if ((st = stride_ok(ldv, n_kv_heads * head_dim, in)) != LQMM_OK) return st;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned_to(slots, 8))
    return LQMM_ERR_ALIGN;
  if (n_q_heads != 0 && (!aligned16(q) || !aligned16(q_out))) return LQMM_ERR_ALIGN;
  if (rotary_dim != 0 && (!aligned_to(positions, 4) || !aligned_to(rope_turns, 8))) return LQMM_ERR_ALIGN;
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.slots = slots;
  a.turns = rope_turns;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.tokens = tokens;
  a.num_pages = num_pages;
  a.n_q_heads = (int)n_q_heads;
  a.n_kv_heads = (int)n_kv_heads;
  a.head_dim = (int)head_dim;
  a.rot_dim = (int)rotary_dim;
  a.interleaved = interleaved != 0;
  a.page_log2 = log2_of(page_size);
  return LQMM_OK;
}

// The sizes of an attention call that its plan depends on.
lqmm_status attn_sizes(lqmm::AttnPrefix &a, int64_t prefix_len, int64_t max_pages, int64_t max_q,
                       int64_t tokens, int64_t batch, int64_t n_q_heads, int64_t n_kv_heads,
                       int64_t head_dim, int64_t page_size) {
  if (!dim_ok(tokens) || !dim_ok(batch) || !dim_ok(max_pages) || !dim_ok(max_q)) return LQMM_ERR_SHAPE;
  if (n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads > kMaxHeads || n_q_heads % n_kv_heads != 0)
    return LQMM_ERR_SHAPE;
  if (!head_dim_ok(head_dim) || !page_size_ok(page_size)) return LQMM_ERR_SHAPE;
  // rows and keys are counted in 31 bits (with a chunk's slack)
  const int64_t most = ((int64_t)1 << 31) - 65536;
  if (prefix_len < 0 || prefix_len > most || max_pages * page_size > most) return LQMM_ERR_SHAPE;
  const int64_t group = n_q_heads / n_kv_heads;
  if (tokens * group > most || max_q * group > most) return LQMM_ERR_SHAPE;
  a.prefix_len = prefix_len;
  a.max_pages = max_pages;
  a.max_q = max_q < tokens ? max_q : tokens;
  a.tokens = tokens;
  a.batch = batch;
  a.n_q_heads = (int)n_q_heads;
  a.n_kv_heads = (int)n_kv_heads;
  a.head_dim = (int)head_dim;
  a.page_log2 = log2_of(page_size);
  return LQMM_OK;
}

// What an attention call checks of its pointers and strides, and its arguments.
lqmm_status attn_args(lqmm::AttnPrefix &a, ElemType *e, const void *q, int64_t ldq, const void *k_cache,
                      const void *v_cache, int type, const int32_t *prefix_pages, int64_t prefix_len,
                      const int32_t *pages, int64_t max_pages, const int32_t *seq_lens,
                      const int32_t *q_start, int64_t max_q, void *out, float *lse, float scale,
                      int64_t tokens, int64_t batch, int64_t n_q_heads, int64_t n_kv_heads,
                      int64_t head_dim, int64_t page_size, int64_t num_pages, const void *workspace) {
  if (!q || !k_cache || !v_cache || !pages || !seq_lens || !out) return LQMM_ERR_NULL;
  if (prefix_len != 0 && !prefix_pages) return LQMM_ERR_NULL;
  if (!elem_type(type, e) || *e == ElemType::F32) return LQMM_ERR_TYPE;
  lqmm_status st = attn_sizes(a, prefix_len, max_pages, max_q, tokens, batch, n_q_heads, n_kv_heads,
                              head_dim, page_size);
  if (st != LQMM_OK) return st;
  if (!dim_ok(num_pages)) return LQMM_ERR_SHAPE;
  if (!q_start && (tokens != batch || max_q != 1)) return LQMM_ERR_SHAPE;
  if (!isfinite(scale)) return LQMM_ERR_SHAPE;
  if ((st = stride_ok(ldq, n_q_heads * head_dim, *e)) != LQMM_OK) return st;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace))
    return LQMM_ERR_ALIGN;
  if (!aligned_to(prefix_pages, 4) || !aligned_to(pages, 4) || !aligned_to(seq_lens, 4) ||
      !aligned_to(q_start, 4) || !aligned_to(lse, 4))
    return LQMM_ERR_ALIGN;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.prefix_pages = prefix_pages;
  a.pages = pages;
  a.lens = seq_lens;
  a.q_start = q_start;
  a.out = out;
  a.lse = lse;
  a.ldq = ldq;
  a.num_pages = num_pages;
  a.scale_log2 = fmaxf(fabsf(scale) * 1.4426950408889634f, 0x1p-126f);
  a.q_sign = scale < 0 ? 0x80008000u : 0u;
  return LQMM_OK;
}

}  // namespace

extern "C" {

lqmm_status lqmm_rope_turns(const double *inv_freq, int64_t n, uint64_t *turns) {
  if (!inv_freq || !turns) return LQMM_ERR_NULL;
  if (!dim_ok(n)) return LQMM_ERR_SHAPE;
  for (int64_t i = 0; i < n; ++i) {
    const double f = inv_freq[i] / (2.0 * 3.14159265358979323846);
    if (!isfinite(f)) return LQMM_ERR_SHAPE;
    const double g = fabs(f), v = nearbyint(ldexp(g - floor(g), 64));  // an exact fraction
    const uint64_t u = v < 0x1p64 ? (uint64_t)v : 0;  // just below a whole turn
    turns[i] = f < 0 ? 0 - u : u;
  }
  return LQMM_OK;
}

lqmm_status lqmm_kv_append(const void *q, const void *k, const void *v, int in_type, int64_t ldq,
                           int64_t ldk, int64_t ldv, const int32_t *positions, const int64_t *slots,
                           const uint64_t *rope_turns, int64_t rotary_dim, int interleaved,
                           void *q_out, void *k_cache, void *v_cache, int cache_type,
                           int64_t tokens, int64_t n_q_heads, int64_t n_kv_heads,
                           int64_t head_dim, int64_t page_size, int64_t num_pages, void *stream) {
  if (!k || !v || !slots || !k_cache || !v_cache) return LQMM_ERR_NULL;
  if (n_q_heads != 0 && (!q || !q_out)) return LQMM_ERR_NULL;
  if (rotary_dim != 0 && (!positions || !rope_turns)) return LQMM_ERR_NULL;
  ElemType in, cache;
  if (!elem_type(in_type, &in) || !elem_type(cache_type, &cache) || cache == ElemType::F32)
    return LQMM_ERR_TYPE;
  lqmm::KvAppend a{};
  const lqmm_status st = append_args(a, in, q, k, v, ldq, ldk, ldv, positions, slots, rope_turns,
                                     rotary_dim, interleaved, q_out, k_cache, v_cache, tokens, n_q_heads,
                                     n_kv_heads, head_dim, page_size, num_pages);
  if (st != LQMM_OK) return st;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  return done(lqmm::kv_append_launch(a, in, cache, (hipStream_t)stream));
}

lqmm_status lqmm_attn_prefix(const void *q, int64_t ldq, const void *k_cache, const void *v_cache,
                             int type, const int32_t *prefix_pages, int64_t prefix_len,
                             const int32_t *pages, int64_t max_pages, const int32_t *seq_lens,
                             const int32_t *q_start, int64_t max_q, void *out, float *lse,
                             float scale, int64_t tokens, int64_t batch, int64_t n_q_heads,
                             int64_t n_kv_heads, int64_t head_dim, int64_t page_size,
                             int64_t num_pages, void *workspace, size_t workspace_bytes,
                             void *stream) {
  lqmm::AttnPrefix a{};
  ElemType e;
  const lqmm_status st = attn_args(a, &e, q, ldq, k_cache, v_cache, type, prefix_pages, prefix_len,
                                   pages, max_pages, seq_lens, q_start, max_q, out, lse, scale, tokens,
                                   batch, n_q_heads, n_kv_heads, head_dim, page_size, num_pages, workspace);
  if (st != LQMM_OK) return st;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  lqmm::attn_prefix_plan(a, max_pages * page_size, num_cus);
  const size_t need = lqmm::attn_prefix_workspace(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LQMM_ERR_WORKSPACE;
  return done(lqmm::attn_prefix_launch(a, workspace, e, (hipStream_t)stream));
}

size_t lqmm_attn_prefix_workspace_bytes(int64_t prefix_len, int64_t max_pages, int64_t max_q,
                                        int64_t tokens, int64_t batch, int64_t n_q_heads,
                                        int64_t n_kv_heads, int64_t head_dim, int64_t page_size) {
  lqmm::AttnPrefix a{};
  int num_cus = 0;
  if (attn_sizes(a, prefix_len, max_pages, max_q, tokens, batch, n_q_heads, n_kv_heads, head_dim,
                 page_size) != LQMM_OK ||
      !lqmm::device_cus(&num_cus))
    return 0;
  lqmm::attn_prefix_plan(a, max_pages * page_size, num_cus);
  return lqmm::attn_prefix_workspace(a);
}

lqmm_status lqmm_kv_append_norm(const void *q, const void *k, const void *v, int in_type, int64_t ldq,
                                int64_t ldk, int64_t ldv, const int32_t *positions,
                                const int64_t *slots, const uint64_t *rope_turns, int64_t rotary_dim,
                                int interleaved, const float *q_norm, const float *k_norm, float eps,
                                void *q_out, void *k_cache, void *v_cache, uint8_t *k_scales,
                                uint8_t *v_scales, int type, int64_t tokens, int64_t n_q_heads,
                                int64_t n_kv_heads, int64_t head_dim, int64_t page_size,
                                int64_t num_pages, void *stream) {
  if (!k || !v || !slots || !k_cache || !v_cache) return LQMM_ERR_NULL;
  if (n_q_heads != 0 && (!q || !q_out)) return LQMM_ERR_NULL;
  if (rotary_dim != 0 && (!positions || !rope_turns)) return LQMM_ERR_NULL;
  if (!k_scales != !v_scales) return LQMM_ERR_NULL;
  ElemType in, e;
  if (!elem_type(in_type, &in) || !elem_type(type, &e) || e == ElemType::F32) return LQMM_ERR_TYPE;
  lqmm::KvAppendNorm a{};
  const lqmm_status st = append_args(a, in, q, k, v, ldq, ldk, ldv, positions, slots, rope_turns,
                                     rotary_dim, interleaved, q_out, k_cache, v_cache, tokens, n_q_heads,
                                     n_kv_heads, head_dim, page_size, num_pages);
  if (st != LQMM_OK) return st;
  if (!isfinite(eps) || eps < 0.f) return LQMM_ERR_SHAPE;
  if (!aligned16(q_norm) || !aligned16(k_norm) || !aligned16(k_scales) || !aligned16(v_scales))
    return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.eps = eps;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  return done(lqmm::kv_append_norm_launch(a, in, e, (hipStream_t)stream));
}

lqmm_status lqmm_kv_read_f8(const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_scales,
                            const uint8_t *v_scales, const int32_t *pages, int64_t max_pages,
                            const int32_t *starts, void *k_out, void *v_out, int type, int64_t tokens,
                            int64_t batch, int64_t n_kv_heads, int64_t head_dim, int64_t page_size,
                            int64_t num_pages, void *stream) {
  if (!k_cache || !v_cache || !k_scales || !v_scales || !pages || !starts || !k_out || !v_out)
    return LQMM_ERR_NULL;
  ElemType e;
  if (!elem_type(type, &e)) return LQMM_ERR_TYPE;
  if (!dim_ok(tokens) || !dim_ok(batch) || !dim_ok(max_pages) || !dim_ok(num_pages) ||
      !head_dim_ok(head_dim) || !page_size_ok(page_size))
    return LQMM_ERR_SHAPE;
  if (n_kv_heads <= 0 || n_kv_heads > kMaxHeads) return LQMM_ERR_SHAPE;
  const int64_t most = ((int64_t)1 << 31) - 65536;
  if (tokens > most || batch > most) return LQMM_ERR_SHAPE;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) || !aligned16(v_scales) ||
      !aligned16(k_out) || !aligned16(v_out) || !aligned_to(pages, 4) || !aligned_to(starts, 4))
    return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  lqmm::KvRead a{};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.pages = pages;
  a.starts = starts;
  a.k_out = k_out;
  a.v_out = v_out;
  a.batch = batch;
  a.max_pages = max_pages;
  a.tokens = tokens;
  a.num_pages = num_pages;
  a.n_kv_heads = (int)n_kv_heads;
  a.head_dim = (int)head_dim;
  a.page_log2 = log2_of(page_size);
  return done(lqmm::kv_read_f8_launch(a, e, (hipStream_t)stream));
}

lqmm_status lqmm_attn_prefix_f8(const void *q, int64_t ldq, const uint8_t *k_cache,
                                const uint8_t *v_cache, const uint8_t *k_scales,
                                const uint8_t *v_scales, int type, const int32_t *prefix_pages,
                                int64_t prefix_len, const int32_t *pages, int64_t max_pages,
                                const int32_t *seq_lens, const int32_t *q_start, int64_t max_q,
                                void *out, float *lse, float scale, int64_t tokens, int64_t batch,
                                int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                                int64_t page_size, int64_t num_pages, void *workspace,
                                size_t workspace_bytes, void *stream) {
  if (!k_scales || !v_scales) return LQMM_ERR_NULL;
  lqmm::AttnPrefixF8 a{};
  ElemType e;
  lqmm_status st = attn_args(a, &e, q, ldq, k_cache, v_cache, type, prefix_pages, prefix_len, pages,
                             max_pages, seq_lens, q_start, max_q, out, lse, scale, tokens, batch,
                             n_q_heads, n_kv_heads, head_dim, page_size, num_pages, workspace);
  if (st != LQMM_OK) return st;
  if (!aligned16(k_scales) || !aligned16(v_scales)) return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  lqmm::attn_f8_plan(a, max_pages * page_size, num_cus);
  const size_t need = lqmm::attn_prefix_workspace(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LQMM_ERR_WORKSPACE;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  return done(lqmm::attn_f8_launch(a, workspace, e, (hipStream_t)stream));
}

size_t lqmm_attn_prefix_f8_workspace_bytes(int64_t prefix_len, int64_t max_pages, int64_t max_q,
                                           int64_t tokens, int64_t batch, int64_t n_q_heads,
                                           int64_t n_kv_heads, int64_t head_dim, int64_t page_size) {
  lqmm::AttnPrefixF8 a{};
  int num_cus = 0;
  if (attn_sizes(a, prefix_len, max_pages, max_q, tokens, batch, n_q_heads, n_kv_heads, head_dim,
                 page_size) != LQMM_OK ||
      !lqmm::device_cus(&num_cus))
    return 0;
  lqmm::attn_f8_plan(a, max_pages * page_size, num_cus);
  return lqmm::attn_prefix_workspace(a);
}

lqmm_status lqmm_quant_mxfp4(const void *X, int x_type, int64_t ldx, uint8_t *Xq, uint8_t *xscale,
                             int64_t M, int64_t K, void *stream) {
  if (!X || !Xq || !xscale) return LQMM_ERR_NULL;
  ElemType e;
  if (!elem_type(x_type, &e)) return LQMM_ERR_TYPE;
  if (!dim_ok(M) || !dim_ok(K) || K % 32 != 0) return LQMM_ERR_SHAPE;
  const lqmm_status st = stride_ok(ldx, K, e);
  if (st != LQMM_OK) return st;
  if (!aligned16(X) || !aligned16(Xq)) return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  return done(lqmm::quant_mxfp4_launch(X, e, ldx, Xq, xscale, M, K, (hipStream_t)stream));
}

lqmm_status lqmm_gemm_mxfp4(const uint8_t *W, const uint8_t *wscale, const uint8_t *Xq,
                            const uint8_t *xscale, void *Y, int y_type, int64_t M, int64_t N,
                            int64_t K, void *stream) {
  if (!W || !wscale || !Xq || !xscale || !Y) return LQMM_ERR_NULL;
  ElemType e;
  if (!elem_type(y_type, &e)) return LQMM_ERR_TYPE;
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || K % 32 != 0) return LQMM_ERR_SHAPE;
  if (K >= LQMM_GEMM_MAX_K) return LQMM_ERR_SHAPE;  // 31-bit load offsets within a tile
  if (!aligned16(W) || !aligned16(Xq) || !aligned16(Y)) return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  return done(lqmm::gemm_mxfp4_launch(W, wscale, Xq, xscale, Y, e, M, N, K, num_cus,
                                      (hipStream_t)stream));
}

lqmm_status lqmm_quant_f8b128(const void *X, int x_type, int64_t ldx, uint8_t *Xq, float *xscale,
                              int64_t M, int64_t K, void *stream) {
  if (!X || !Xq || !xscale) return LQMM_ERR_NULL;
  ElemType e;
  if (!elem_type(x_type, &e)) return LQMM_ERR_TYPE;
  if (!dim_ok(M) || !dim_ok(K) || K % 16 != 0) return LQMM_ERR_SHAPE;
  const lqmm_status st = stride_ok(ldx, K, e);
  if (st != LQMM_OK) return st;
  if (!aligned16(X) || !aligned16(Xq) || !aligned16(xscale)) return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  return done(lqmm::quant_f8b128_launch(X, e, ldx, Xq, xscale, M, K, (hipStream_t)stream));
}

lqmm_status lqmm_gemm_f8b128(const uint8_t *W, const float *wscale, const uint8_t *Xq,
                             const float *xscale, void *Y, int y_type, int64_t M, int64_t N,
                             int64_t K, void *stream) {
  if (!W || !wscale || !Xq || !xscale || !Y) return LQMM_ERR_NULL;
  ElemType e;
  if (!elem_type(y_type, &e)) return LQMM_ERR_TYPE;
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || K % 16 != 0) return LQMM_ERR_SHAPE;
  if (K >= LQMM_GEMM_MAX_K) return LQMM_ERR_SHAPE;  // 31-bit load offsets within a tile
  if (!aligned16(W) || !aligned16(wscale) || !aligned16(Xq) || !aligned16(xscale) || !aligned16(Y))
    return LQMM_ERR_ALIGN;
  int num_cus = 0;
  if (!lqmm::device_cus(&num_cus)) return LQMM_ERR_DEVICE;
  return done(lqmm::gemm_f8b128_launch(W, wscale, Xq, xscale, Y, e, M, N, K, num_cus,
                                       (hipStream_t)stream));
}

}  // extern "C"
