// What the attention kernels over a paged cache share (attn_prefix.hip,
// attn_f8.hip): work items, rows of no sequence, how partial results are weighed
// when they are joined, and the join of attn_prefix.hip. All in an unnamed
// namespace; gfx950 only.
#pragma once

#include "lqmm_internal.hpp"
#include "serve_device.hpp"

namespace lqmm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;          // rows of a work item
constexpr int kStep = 32;          // keys of one step of a wave
constexpr int kMaxIds = kAttnMaxChunk / 8 + 8;

// ln(2^ref l). The exponent of l goes to the reference first: log2(l) by itself
// would be rounded at the size of the weights' scale.
__device__ __forceinline__ float lse_of(float ref, float l) {
  if (l == 0.f) return -INFINITY;
  return (ref + (float)__builtin_amdgcn_frexp_expf(l) + __log2f(__builtin_amdgcn_frexp_mantf(l))) *
         0.6931471805599453f;
}

// The part of a sequence's (or the prefix's) problem that one workgroup does.
struct Item {
  int h;            // key head
  int row0, rows;   // first row of the block, and rows of the problem
  int64_t tok0;     // first token of the problem
  int part;         // which partial result this is
  int c0, c1;       // keys [c0, c1)
  int past;         // keys that the problem's token 0 sees (before `per_token` is added)
  int per_token;    // 1: token i sees i more keys
  const int32_t *pages;
};

__device__ __forceinline__ bool find_item(const AttnPrefix &a, uint32_t idx, int rows_per_block,
                                          Item &it) {
  const int G = a.group;
  if (idx < (uint32_t)a.prefix_items) {
      // row blocks of one chunk and head follow each other
    const int rb = (int)(idx % (uint32_t)a.prefix_row_blocks);
    const uint32_t rest = idx / (uint32_t)a.prefix_row_blocks;
    it.h = (int)(rest % (uint32_t)a.n_kv_heads);
    const int chunk = (int)(rest / (uint32_t)a.n_kv_heads);
    it.part = chunk;
    it.tok0 = 0;
    it.rows = (int)a.tokens * G;
    it.row0 = rb * rows_per_block;
    const int64_t c0 = (int64_t)chunk * a.prefix_chunk;
    it.c0 = (int)c0;
    it.c1 = (int)(c0 + a.prefix_chunk < a.prefix_len ? c0 + a.prefix_chunk : a.prefix_len);
    it.past = (int)a.prefix_len;
    it.per_token = 0;
    it.pages = a.prefix_pages;
    return true;
  }
  idx -= (uint32_t)a.prefix_items;
  const int rb = (int)(idx % (uint32_t)a.suffix_row_blocks);
  idx /= (uint32_t)a.suffix_row_blocks;
  const int chunk = (int)(idx % (uint32_t)a.suffix_parts);
  idx /= (uint32_t)a.suffix_parts;
  it.h = (int)(idx % (uint32_t)a.n_kv_heads);
  const int64_t b = idx / (uint32_t)a.n_kv_heads;
  // Lengths come from the device: bounded here, so that no value of theirs
  // reaches outside the tensors.
  const int64_t cap = a.max_pages << a.page_log2;
  int64_t len = a.lens[b];
  len = len < 0 ? 0 : len < cap ? len : cap;
  int64_t q0 = b, q1 = b + 1;
  if (a.q_start) {
    q0 = a.q_start[b];
    q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0 < a.tokens ? q0 : a.tokens;
    q1 = q1 < q0 ? q0 : q1 < a.tokens ? q1 : a.tokens;
  }
  // (rows past max_q are left out, and still are new tokens of the sequence)
  const int news = (int)(q1 - q0);
  const int n = a.max_q < news ? (int)a.max_q : news;
  it.part = a.prefix_parts + chunk;
  it.tok0 = q0;
  it.rows = n * G;
  it.row0 = rb * rows_per_block;
  if (it.row0 >= it.rows) return false;
  it.past = (int)len - news + 1;
  it.per_token = 1;
  it.pages = a.pages + b * a.max_pages;
  const int64_t c0 = (int64_t)chunk * a.suffix_chunk;
  it.c0 = (int)(c0 < len ? c0 : len);
  // no row of the block sees more keys than its last token
  int last = it.row0 + rows_per_block - 1;
  last = last < it.rows ? last : it.rows - 1;
  int64_t c1 = it.past + last / G;
  c1 = c1 < c0 + a.suffix_chunk ? c1 : c0 + a.suffix_chunk;
  it.c1 = (int)(c1 > it.c0 ? c1 : it.c0);
  return true;
}

// Rows of q that belong to no sequence (before q_start[0], past max_q of a
// sequence's, from q_start[batch] on) see no key: out is 0 and lse -infinity.
// The first workgroup of a sequence and key head does those beside its rows. Where
// results are joined it leaves the sum kNoSequence in the first of the
// sequences' parts, whose other entries for such rows nothing writes.
constexpr float kNoSequence = -1.0f;

template <class T, int D>
__device__ __forceinline__ void rows_of_no_sequence(const AttnPrefix &a, uint32_t idx, int threads) {
  if (!a.q_start || idx < (uint32_t)a.prefix_items) return;
  idx -= (uint32_t)a.prefix_items;
  const uint32_t first = (uint32_t)a.suffix_row_blocks * (uint32_t)a.suffix_parts;
  if (idx % first) return;
  idx /= first;
  const int h = (int)(idx % (uint32_t)a.n_kv_heads), G = a.group;
  const int64_t b = idx / (uint32_t)a.n_kv_heads;
  int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
  q0 = q0 < 0 ? 0 : q0 < a.tokens ? q0 : a.tokens;
  q1 = q1 < q0 ? q0 : q1 < a.tokens ? q1 : a.tokens;
  if (q1 - q0 > a.max_q) q0 += a.max_q;
  else q0 = q1;
  if (b == a.batch - 1) q1 = a.tokens;
  int64_t before = b == 0 ? a.q_start[0] : 0;  // tokens [0, before) and [q0, q1)
  before = before < 0 ? 0 : before < a.tokens ? before : a.tokens;
  const bool direct = a.prefix_parts + a.suffix_parts == 1;
  constexpr int kVecs = D / 8;
  const int per = direct ? G * kVecs : G;  // stores of a token
  for (int64_t i = threadIdx.x; i < (before + q1 - q0) * per; i += threads) {
    const int64_t n = i / per;
    const int64_t t = n < before ? n : q0 + n - before;
    const int in = (int)(i % per), g = direct ? in / kVecs : in;
    const int64_t flat = t * a.n_q_heads + h * G + g;
    if (!direct) {
      a.part_ml[a.prefix_parts * (a.tokens * a.n_q_heads) + flat] = make_float2(-INFINITY, kNoSequence);
      continue;
    }
    reinterpret_cast<u32x4 *>(static_cast<typename T::elem *>(a.out) + flat * D)[in % kVecs] = u32x4{0u, 0u, 0u, 0u};
    if (a.lse && in % kVecs == 0) a.lse[flat] = -INFINITY;
  }
}

// Workgroups are handed to the 8 XCDs in turn, and each has its own L2:
// renumbered so that consecutive items, which share keys, run on one XCD.
__device__ __forceinline__ uint32_t spread(uint32_t block, uint32_t n) {
  const uint32_t x = block % 8, q = n / 8, r = n % 8;
  return x * q + (x < r ? x : r) + block / 8;
}

// Parts are weighed by at most 2^-18, so that the sum of any number of them
// (under 2^19) stays below the largest value, as each does.
constexpr int kJoinShift = 18;
constexpr float kJoinWeight = 1.0f / (1 << kJoinShift);

// Joins the partial results of each row: D / 4 threads a row, four
// dimensions each.
template <class T, int D>
__global__ void __launch_bounds__(kThreads)
attn_join_kernel(AttnPrefix a, uint32_t first) {
  typedef typename T::elem elem;
  constexpr int kPer = D / 4;
  constexpr int kRowsPerBlock = kThreads / kPer;
  const int64_t nrows = a.tokens * a.n_q_heads;
  const int64_t row = (int64_t)(first + blockIdx.x) * kRowsPerBlock + threadIdx.x / kPer;
  const int d = 4 * (threadIdx.x % kPer);
  if (threadIdx.x / kPer >= kRowsPerBlock || row >= nrows) return;
  const int parts = a.prefix_parts + a.suffix_parts;
  float m = -INFINITY;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) m = fmaxf(m, a.part_ml[p * nrows + row].x);
  float l = 0.f;
  float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    // of a part that sees no key nothing counts
    const float2 ml = a.part_ml[p * nrows + row];
    const float4_t x = *reinterpret_cast<const float4_t *>(a.part_o + (p * nrows + row) * D + d);
    const bool seen = ml.y != 0.f;
    const float w = seen ? __builtin_amdgcn_exp2f(ml.x - m) * kJoinWeight : 0.f;
    l += w * (seen ? ml.y : 0.f);
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] += w * (seen ? x[r] : 0.f);
  }
  // of a row of no sequence nothing read above counts
  if (a.q_start && a.part_ml[a.prefix_parts * nrows + row].y == kNoSequence) {
    l = 0.f;
    o = float4_t{0.f, 0.f, 0.f, 0.f};
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  elem *dst = static_cast<elem *>(a.out) + row * D + d;
#pragma unroll
  for (int r = 0; r < 4; ++r) dst[r] = (elem)(o[r] * inv);
  if (a.lse && d == 0)
    a.lse[row] = lse_of(m, l * (1 << kJoinShift));
}

}  // namespace
}  // namespace lqmm
