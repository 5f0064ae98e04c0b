// Attention over the 8-bit paged cache: attn_prefix.hip's problem with keys and
// values held as e4m3 codes and a power of two for each token and head.
//
// Mathematics. With z_j = scale * log2(e) * q.k_j and V's values code_j 2^(e_j),
//   O = sum_j 2^(z_j) 2^(e_j) code_j / sum_j 2^(z_j).
// bf16 has the range for it as it stands: with a reference m near the largest z
// and w_j = 2^(z_j - m), the matrix cores take w_j 2^(e_j), rounded once, and V's
// codes as they are, and the sum takes w_j.
// fp16 has not. Few rows: the exponents go to the logits; with y_j = z_j + e_j, m
// near the largest y and w_j = 2^(y_j - m),
//   O = sum_j w_j code_j / sum_j w_j 2^(-e_j),
// so that the weights lose nothing by scales that differ from token to token. The
// scale of V costs no instruction at the logits (the multiplication with scale *
// log2(e) becomes a multiply-add) and none at the sum (an addition becomes one).
// (A w_j below 2^-126 is 0, also where 2^(-e_j) would make it count: the scales
// have to lie closer together than fp32's exponents reach, as those that fp16
// takes do, 2^67 apart.)
// Many rows: each code is converted once for all rows of a workgroup, V's with its
// scale (the values are exact down to 2^-14, then in steps of 2^-24), and m is
// near the largest z.
// K's scale costs nothing: the conversion of a lane's codes, all of one token, to
// 16 bits applies it. A partial result is (m, sum of weights, weighted sum) at m,
// whichever it is, joined as in attn_prefix.hip.
//
// Bound (128 dimensions unless said): few rows by reading the cache, 24 ragged
// sequences of up to 8209 keys, 8 key heads, 48 us and 5 for the join (floor 38);
// what is left is the end, where the longest chunks run alone. Many rows by the
// vector ALU (54 % of the cycles, 76 % with 64 dimensions) and the matrix cores
// (43 %, 33 %), mostly in turn: 96 x 8 rows a key head behind 32801 keys, bf16,
// 132 us; 6 x 301 new tokens behind 8200 keys, 64 dimensions, fp16 163 us.
//
// Weights are held at 2^14 in fp16, as there; in bf16 at 1 (values are below 2^69,
// so that no sum of a work item's 2^13 keys comes near the largest number).
#include "attn_common.hpp"
#include "f8_cache.hpp"

namespace lqmm {
namespace {

// log2 of what weights are held at, times their value
template <class T>
constexpr float kShift = __is_same(T, TypeF16) ? 14.0f : 0.0f;
constexpr float kAloneShift = 0.0f;  // of rows done by themselves, in fp32

// Scale bytes as they are taken. What fp16 holds ends at 2^7 times a code, and an
// infinity would leave its row by the product with weights of 0 (a row whose mask
// hides the key): larger scales, which only an append of bf16 writes, count as 2^7.
// bf16: a byte of 254 or 255 beside a key that is not seen must be finite as well.
template <class T>
__device__ __forceinline__ uint32_t taken(uint32_t byte) {
  constexpr uint32_t kMost = __is_same(T, TypeF16) ? kMostScaleF16 : 253;
  return byte < kMost ? byte : kMost;
}

// First token vector of the group of eight that holds key j (in vectors of D
// codes, of which each has one scale).
__device__ __forceinline__ int64_t vector_at(const AttnPrefix &a, const Item &it, int j) {
  const int32_t p = it.pages[j >> a.page_log2];
  const int64_t page = (uint32_t)p < (uint32_t)a.num_pages ? p : 0;
  return ((page * a.n_kv_heads + it.h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
}

// The item of a workgroup. Workgroups are handed to the 8 XCDs in turn, and each
// has its own L2: the row blocks of a chunk and head, which read the same keys,
// follow each other on one XCD, and heads go to the XCDs in turn, the prefix's
// and then the sequences', so that each XCD has its share of both and of the long
// sequences (64 rows behind 16000 shared keys: 73 us when each XCD has the next
// eighth of all items, 46 so). All sequences' first chunks come before the second
// ones, of which some hold nothing (24 sequences of 1000 keys under a page table
// of 131072, 64 chunks: 145 us when a sequence's chunks go to the XCDs in turn,
// 37 so).
__device__ __forceinline__ uint32_t dealt(uint32_t block, uint32_t n, uint32_t row_blocks) {
  const uint32_t whole = n / (8 * row_blocks) * (8 * row_blocks), i = block / 8;
  if (block >= whole) return whole + spread(block - whole, n - whole);
  return (i / row_blocks * 8 + block % 8) * row_blocks + i % row_blocks;
}

__device__ __forceinline__ uint32_t item_of(const AttnPrefix &a, uint32_t item0, uint32_t block, uint32_t n) {
  const uint32_t left = item0 < (uint32_t)a.prefix_items ? (uint32_t)a.prefix_items - item0 : 0;
  const uint32_t pre = left < n ? left : n;
  if (block < pre) return item0 + dealt(block, pre, a.prefix_row_blocks);
  const uint32_t i = dealt(block - pre, n - pre, a.suffix_row_blocks);
  if (n - pre != (uint32_t)a.suffix_items) return item0 + pre + i;  // (one of several launches)
  const uint32_t unit = i / a.suffix_row_blocks, heads = (uint32_t)a.suffix_items / (a.suffix_row_blocks * a.suffix_parts);
  const uint32_t chunk = unit / heads, head = unit - chunk * heads;
  return (uint32_t)a.prefix_items + (head * a.suffix_parts + chunk) * a.suffix_row_blocks + i % a.suffix_row_blocks;
}

// An item without keys (page tables are wider than most sequences): the join is
// told so, and reads nothing else of it (24 sequences of 1000 keys under a table of
// 131072: 158 us with such items' sums stored and read as zeros, 145 so).
__device__ __forceinline__ bool empty_item(const AttnPrefix &a, const Item &it, int rows_per_block, int threads) {
  if (it.c0 < it.c1 || a.prefix_parts + a.suffix_parts == 1) return false;
  const int G = a.group, end = it.rows - it.row0 < rows_per_block ? it.rows - it.row0 : rows_per_block;
  for (int i = threadIdx.x; i < end; i += threads) {
    const int row = it.row0 + i;
    const int64_t flat = (it.tok0 + row / G) * a.n_q_heads + it.h * G + row % G;
    a.part_ml[it.part * (a.tokens * a.n_q_heads) + flat] = make_float2(-INFINITY, 0.f);
  }
  return true;
}

// ---- values behind a mask -------------------------------------------------------
// As in attn_prefix.hip: a masked weight is 0, and 0 times a NaN code is NaN. O
// is looked through for NaN behind the keys' loop, and rows of a block with such
// a code among the keys of its mask's edge are done again, by themselves.

// Whether V of the keys [from, it.c1) has a NaN code (one wave).
template <int D>
__device__ __forceinline__ bool edge_has_nan(const AttnPrefixF8 &a, const Item &it, int from) {
  const int lane = threadIdx.x & 63;
  const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache);
  if (from < it.c0) from = it.c0;
  bool found = false;
#pragma unroll 1
  for (int j0 = from & ~7; j0 < it.c1; j0 += 8) {
    const uint8_t *at = vc + vector_at(a, it, j0) * D;
    for (int d = lane; d < D; d += 64) {
      const u32x2 x = *reinterpret_cast<const u32x2 *>(at + 8 * d);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        found = found || (j0 + e >= from && j0 + e < it.c1 && (x[e >> 2] >> 8 * (e & 3) & 0x7fu) == 0x7fu);
    }
  }
  return __any(found);
}

// One row of an item by one wave: a lane a key for the logits, a lane a
// dimension for O, only of keys that the row sees.
template <class T, int D>
__device__ __forceinline__ void row_alone(const AttnPrefixF8 &a, const Item &it, int row) {
  typedef typename T::elem elem;
  constexpr int kO = (D + 63) / 64;
  const int lane = threadIdx.x & 63, G = a.group;
  const int tok = row / G;
  const int64_t flat = (it.tok0 + tok) * a.n_q_heads + it.h * G + row % G;
  const int limit = it.past + it.per_token * tok;
  const int end = limit < it.c1 ? limit : it.c1;
  const elem *q = static_cast<const elem *>(a.q) + (it.tok0 + tok) * a.ldq + (int64_t)(it.h * G + row % G) * D;
  const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache), *vc = static_cast<const uint8_t *>(a.v_cache);
  const float scale = a.q_sign ? -a.scale_log2 : a.scale_log2;
  float m = -INFINITY, l = 0.f, o[kO];
#pragma unroll
  for (int i = 0; i < kO; ++i) o[i] = 0.f;
  for (int j0 = it.c0; j0 < end; j0 += 64) {
    float z = -INFINITY;
    if (j0 + lane < end) {
      const int64_t vec = vector_at(a, it, j0 + lane);
      const float ks = scale_of(taken<T>(a.k_scales[vec]));
      float dot = 0.f;
#pragma unroll 1
      for (int d = 0; d < D; d += 8) {
        float x[8];
        load8<T>(q + d, x);
        const typename T::vec8 y = values8<T>(*reinterpret_cast<const u32x2 *>(kc + vec * D + d), ks);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(x[e], (float)y[e], dot);
      }
      z = dot * scale;
    }
    float mn = fmaxf(m, z);
    for (int s = 32; s > 0; s >>= 1) mn = fmaxf(mn, __shfl_xor(mn, s));
    const float ref = (mn == -INFINITY ? 0.f : mn) - kAloneShift;
    const float c = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - kAloneShift - ref);
    const float e = __builtin_amdgcn_exp2f(z - ref);
    float sum = e;
    for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
    m = mn;
    l = l * c + sum;
#pragma unroll
    for (int i = 0; i < kO; ++i) o[i] *= c;
    const int n = end - j0 < 64 ? end - j0 : 64;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int j = j0 + i;
      const int64_t vec = vector_at(a, it, j);
      const float w = __shfl(e, i) * scale_of(taken<T>(a.v_scales[vec]));
      const uint8_t *v = vc + (vec & ~7) * D + (vec & 7);
#pragma unroll
      for (int u = 0; u < kO; ++u)
        if (lane + 64 * u < D) o[u] += w * __builtin_amdgcn_cvt_f32_fp8((int)v[8 * (lane + 64 * u)], 0);
    }
  }
  const bool direct = a.prefix_parts + a.suffix_parts == 1;
  const int64_t at = it.part * (a.tokens * a.n_q_heads) + flat;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int u = 0; u < kO; ++u) {
    const int d = lane + 64 * u;
    if (d >= D) continue;
    if (direct) static_cast<elem *>(a.out)[flat * D + d] = (elem)(o[u] * inv);
    else a.part_o[at * D + d] = o[u];
  }
  if (lane) return;
  if (!direct) a.part_ml[at] = make_float2(m - kAloneShift, l);
  else if (a.lse) a.lse[flat] = lse_of(m - kAloneShift, l);
}

// ---- few rows -------------------------------------------------------------------
// 16 rows a workgroup; the waves take different keys, 32 a step, straight from
// memory to the operands, and are joined in LDS.
template <int D, int NW>
struct Rows16 {
  static constexpr int kPass = D / 16 < 8 ? D / 16 : 8;  // O tiles joined at a time
  static constexpr int kLd = 16 * kPass + 4;
  int ids[kMaxIds];
  float wave_m[NW][kRows], wave_l[NW][kRows];
  __attribute__((aligned(16))) float join[NW][kRows][kLd];
};

template <class T, int D, int NW>
__device__ __forceinline__ void rows16_body(const AttnPrefixF8 &a, const Item &it, Rows16<D, NW> &sm) {
  typedef typename T::elem elem;
  typedef typename T::vec8 vec8;
  constexpr int kK = D / 64;                       // 64-wide pieces of a key (and half of one, at 96)
  constexpr bool kRest = D % 64 != 0;
  constexpr int kQ = D / 32;                       // 32-wide products of a logit tile
  constexpr int kDT = D / 16;                      // 16-wide tiles of O
  constexpr int kPass = Rows16<D, NW>::kPass;
  constexpr bool kWithExponents = __is_same(T, TypeF16);  // V's exponents are in the logits
  static_assert(kDT % kPass == 0 && kPass % 2 == 0, "whole passes");
  int *ids = sm.ids;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m16 = lane & 15, g = lane >> 4;
  const int G = a.group;
  const int lg = a.page_log2, pmask = (1 << lg) - 1;
  const bool direct = a.prefix_parts + a.suffix_parts == 1;

  // page numbers of the chunk, bounded to the cache
  const int page0 = it.c0 >> lg;
  if (it.c1 > it.c0) {
    const int n = ((it.c1 - 1) >> lg) - page0 + 1;
    for (int i = tid; i < n; i += 64 * NW) {
      const int32_t p = it.pages[page0 + i];
      ids[i] = (uint32_t)p < (uint32_t)a.num_pages ? p : 0;
    }
  }
  // this lane's row
  const int row = it.row0 + m16;
  const bool live = row < it.rows;
  const int tok = live ? row / G : 0;
  const int64_t t = it.tok0 + tok;
  const int hq = it.h * G + (live ? row % G : 0);
  const int limit = it.past + it.per_token * tok;  // keys below it are seen
  // keys that every row of the block sees
  const int all_see = it.past + it.per_token * (it.row0 / G);
  // Which dimensions are one product is free: a lane's 16 bytes of a key are 16
  // dimensions next to each other, two products' worth.
  vec8 q[kQ];
  {
    const elem *src = static_cast<const elem *>(a.q) + t * a.ldq + (int64_t)hq * D;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int d = i < 2 * kK ? 64 * (i / 2) + 16 * g + 8 * (i % 2) : 64 * kK + 8 * g;
      const u32x4 x = *reinterpret_cast<const u32x4 *>(src + d);
      q[i] = __builtin_bit_cast(vec8, x ^ a.q_sign);
    }
  }
  __syncthreads();

  float4_t o[kDT];
#pragma unroll
  for (int i = 0; i < kDT; ++i) o[i] = float4_t{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache);
  const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache);
  // first vector of the eight-token group that holds key j (j % 8 == 0)
  auto group_at = [&](int j) -> int64_t {
    const int64_t page = ids[(j >> lg) - page0];
    return ((page * a.n_kv_heads + it.h) << lg) + (j & pmask);
  };
  const int last_group = (it.c1 - 1) & ~7;
  auto clamp_group = [&](int j) { return j < last_group ? j : last_group; };

  // A step's codes and scales, loaded one step ahead. Row m of logit tile s is
  // key 8 (m / 4) + 4 s + m % 4. A lane's 16 bytes of V are dimensions 32 i + 2
  // m16 and the next of its group's tokens: rows of two tiles of O.
  struct Stage {
    u32x4 k[2][kK > 0 ? kK : 1], v[kDT / 2];
    u32x2 rest[2], vs;
    uint32_t ks[2];
  } st;
  auto load = [&](int j0) {
    const int64_t kg = group_at(clamp_group(j0 + 8 * (m16 >> 2))), vg = group_at(clamp_group(j0 + 8 * g));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t vec = kg + 4 * s + (m16 & 3);
      const uint8_t *src = kc + vec * D;
#pragma unroll
      for (int i = 0; i < kK; ++i) st.k[s][i] = *reinterpret_cast<const u32x4 *>(src + 64 * i + 16 * g);
      if constexpr (kRest) st.rest[s] = *reinterpret_cast<const u32x2 *>(src + 64 * kK + 8 * g);
      st.ks[s] = a.k_scales[vec];
    }
#pragma unroll
    for (int i = 0; i < kDT / 2; ++i)
      st.v[i] = *reinterpret_cast<const u32x4 *>(vc + vg * D + (32 * i + 2 * m16) * 8);
    st.vs = *reinterpret_cast<const u32x2 *>(a.v_scales + vg);
  };

  int j0 = it.c0 + wave * kStep;
  if (j0 < it.c1) load(j0);
  for (; j0 < it.c1; j0 += NW * kStep) {
    float4_t s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = float4_t{0.f, 0.f, 0.f, 0.f};
      const float f = scale_of(taken<T>(st.ks[u]));
#pragma unroll
      for (int i = 0; i < kK; ++i) {
        const u32x4 k = st.k[u][i];
        s[u] = T::mfma16(values8<T>(u32x2{k[0], k[1]}, f), q[2 * i], s[u]);
        s[u] = T::mfma16(values8<T>(u32x2{k[2], k[3]}, f), q[2 * i + 1], s[u]);
      }
      if constexpr (kRest) s[u] = T::mfma16(values8<T>(st.rest[u], f), q[2 * kK], s[u]);
    }
    u32x4 v[kDT / 2];
#pragma unroll
    for (int i = 0; i < kDT / 2; ++i) v[i] = st.v[i];
    const u32x2 vs = st.vs;
    if (j0 + NW * kStep < it.c1) load(j0 + NW * kStep);
    // logits; what a weight is multiplied by for the product with V (bf16), or for
    // the sum beside logits with V's exponents (fp16)
    float y[2][4], times[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // (what lies below 2^-60 is 0 in fp16's outputs, and its inverse too large for a sum)
        int b = (int)taken<T>(vs[u] >> 8 * r & 255u);
        if (kWithExponents && b < kLeastScale) b = kLeastScale;
        y[u][r] = kWithExponents ? fmaf(s[u][r], a.scale_log2, (float)(b - 127)) : s[u][r] * a.scale_log2;
        times[u][r] = kWithExponents ? scale_inverse(b) : scale_of(b);
      }
    const int seen = limit < it.c1 ? limit : it.c1;
    if (j0 + kStep > it.c1 || j0 + kStep > all_see) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j0 + 8 * g + 4 * u + r >= seen) y[u][r] = -INFINITY;
      // what lies behind the last key may be anything, and 0 * NaN is NaN
      if (j0 + kStep > it.c1) {
        const int valid = it.c1 - (j0 + 8 * g);
        const uint32_t lo = valid <= 0 ? 0u : valid >= 4 ? ~0u : ~0u >> (32 - 8 * valid);
        const uint32_t hi = valid <= 4 ? 0u : valid >= 8 ? ~0u : ~0u >> (64 - 8 * valid);
#pragma unroll
        for (int i = 0; i < kDT / 2; ++i) v[i] &= u32x4{lo, hi, lo, hi};
      }
    }
    float top = fmaxf(fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3])),
                      fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
    const float mn = fmaxf(m, max_over_rows(top));
    const float ref = (mn == -INFINITY ? 0.f : mn) - kShift<T>;
    // (between references, as they were rounded)
    const float corr = __builtin_amdgcn_exp2f(m - kShift<T> - ref);
    const float c = m == -INFINITY ? 0.f : corr;
    m = mn;
    vec8 p;
    l *= c;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = __builtin_amdgcn_exp2f(y[u][r] - ref);
        l = kWithExponents ? fmaf(e, times[u][r], l) : l + e;
        p[4 * u + r] = (elem)(kWithExponents ? e : e * times[u][r]);
      }
#pragma unroll
    for (int i = 0; i < kDT; ++i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) o[i][r] *= c;
      const u32x4 x = v[i / 2];
      o[i] = T::mfma16(values8<T>(i % 2 ? u32x2{x[2], x[3]} : u32x2{x[0], x[1]}, 1.0f), p, o[i]);
    }
  }

  if (it.c1 > all_see) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) bad = bad || o[i][r] != o[i][r];
    if (__syncthreads_or(live && bad) && edge_has_nan<D>(a, it, all_see)) {
      const int end = it.row0 + kRows < it.rows ? it.row0 + kRows : it.rows;
      for (int i = it.row0 + wave; i < end; i += NW) row_alone<T, D>(a, it, i);
      return;
    }
  }

  // Join the waves' results.
  l = sum_over_rows(l);
  if (g == 0) {
    sm.wave_m[wave][m16] = m;
    sm.wave_l[wave][m16] = l;
  }
  __syncthreads();
  float mj = -INFINITY;
#pragma unroll
  for (int w = 0; w < NW; ++w) mj = fmaxf(mj, sm.wave_m[w][m16]);
  constexpr int kPer = 32 / NW;  // values of a row that a thread writes per pass
  const float mine = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - kShift<T> - (mj - kShift<T>));
  const int out_row = tid / (4 * NW), out_d = kPer * (tid % (4 * NW));
  // the row that this thread writes
  float lj = 0.f, mo = -INFINITY;
#pragma unroll
  for (int w = 0; w < NW; ++w) mo = fmaxf(mo, sm.wave_m[w][out_row]);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float mw = sm.wave_m[w][out_row], lw = sm.wave_l[w][out_row];
    lj += lw == 0.f ? 0.f : lw * __builtin_amdgcn_exp2f(mw - kShift<T> - (mo - kShift<T>));
  }
  const int orow = it.row0 + out_row;
  const bool owrite = orow < it.rows;
  const int64_t flat = (it.tok0 + orow / G) * a.n_q_heads + it.h * G + orow % G;
  const int64_t nrows = a.tokens * a.n_q_heads;
#pragma unroll
  for (int pass = 0; pass < kDT / kPass; ++pass) {
    if (pass) __syncthreads();
#pragma unroll
    for (int i = 0; i < kPass; i += 2) {  // rows 4 g + r of two tiles are dimensions 8 g + 2 r and the next
      const float4_t x = o[pass * kPass + i], z = o[pass * kPass + i + 1];
      float4_t *dst = reinterpret_cast<float4_t *>(&sm.join[wave][m16][16 * i + 8 * g]);
      dst[0] = float4_t{x[0] * mine, z[0] * mine, x[1] * mine, z[1] * mine};
      dst[1] = float4_t{x[2] * mine, z[2] * mine, x[3] * mine, z[3] * mine};
    }
    __syncthreads();
    if (owrite && out_d < 16 * kPass) {
      float x[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        x[e] = sm.join[0][out_row][out_d + e];
#pragma unroll
        for (int w = 1; w < NW; ++w) x[e] += sm.join[w][out_row][out_d + e];
      }
      const int64_t d0 = pass * 16 * kPass + out_d;
      if (direct) {
        typedef elem out_vec __attribute__((ext_vector_type(kPer)));
        const float inv = lj == 0.f ? 0.f : 1.0f / lj;
        out_vec y;
#pragma unroll
        for (int e = 0; e < kPer; ++e) y[e] = (elem)(x[e] * inv);
        *reinterpret_cast<out_vec *>(static_cast<elem *>(a.out) + flat * D + d0) = y;
      } else {
        float *dst = a.part_o + (it.part * nrows + flat) * D + d0;
#pragma unroll
        for (int e = 0; e < kPer; e += 4)
          *reinterpret_cast<float4_t *>(dst + e) = float4_t{x[e], x[e + 1], x[e + 2], x[e + 3]};
      }
    }
  }
  if (owrite && out_d == 0) {
    if (direct) {
      if (a.lse) a.lse[flat] = lse_of(mo - kShift<T>, lj);
    } else {
      a.part_ml[it.part * nrows + flat] = make_float2(mo - kShift<T>, lj);
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 2 : 1)
attn_f8_rows16_kernel(AttnPrefixF8 a, uint32_t item0) {
  __shared__ Rows16<D, kThreads / 64> sm;
  Item it;
  const uint32_t idx = item_of(a, item0, blockIdx.x, gridDim.x);
  rows_of_no_sequence<T, D>(a, idx, kThreads);
  if (find_item(a, idx, kRows, it) && !empty_item(a, it, kRows, kThreads))
    rows16_body<T, D, kThreads / 64>(a, it, sm);
}

// ---- many rows -----------------------------------------------------------------
// As in attn_prefix.hip: 32 R rows a wave, all waves of a workgroup take the same
// keys from LDS tiles of 16-bit operands. Here the codes come through registers
// and are converted once for all waves on their way into LDS (K with its scales;
// V's go beside it, as the exponents and powers that logits and sums take).
//
// A running maximum that grows by no more than kSlack (log2) is left where it
// is: O is rescaled when a row needs it, not at every step.
constexpr float kSlack = 8.0f;
// Weights are at most 2^(kSlack + kWideShift): 2^kShift.
template <class T>
constexpr float kWideShift = kShift<T> - kSlack;

// Waves of a SIMD that the wide kernel's registers leave room for, keys of a tile,
// and what a CU then holds: two workgroups, which wait at barriers of their own,
// or one of eight waves (128 dimensions, 256 rows). Measured with 128 rows, 60001
// keys, 8 key heads: 128 dimensions 74 us with two workgroups and tiles of 32
// keys, 84 with one and 64; 64 dimensions 44 us with 64 keys, 57 with 32.
constexpr int wide_waves(int d, int nw, int r) {
  return r > 1 ? (d == 64 ? 2 : 1) : d <= 128 ? 2 : 1;
}
constexpr int wide_keys(int d, int nw, int r) {
  return d > 128 || (d > 64 && nw == 4 && r == 1) ? 32 : 64;
}

template <int D, int KEYS>
struct Wide {
  static constexpr int kKeys = KEYS;
  static constexpr int kHalf = kKeys * D * 2;       // bytes of a tile's K (and V)
  // a round is two tiles between barriers: K of it and of the tile after, V of
  // it, and the next round's two tiles of each on their way
  static constexpr int kStagesK = 5, kStagesV = 4;
  static constexpr int kScales = kKeys * 4;         // V's scales beside its codes
  static constexpr int kLds = (kStagesK + kStagesV) * kHalf + kStagesV * kScales;
};

// The rows of a wave again, if its mask's edge asks for it (whether it did). Item
// and arguments are read once more, so that nothing of them is held in registers
// through the keys' loop for this.
template <class T, int D>
__device__ __forceinline__ bool wave_again(uint32_t item0, int rows_per_block, int from, int n) {
  uint64_t args = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  uint32_t block = blockIdx.x;
  asm volatile("" : "+s"(args), "+s"(block));
  const AttnPrefixF8 &a = *reinterpret_cast<const AttnPrefixF8 *>(args);  // the kernel's first argument
  Item it;
  if (!find_item(a, item_of(a, item0, block, gridDim.x), rows_per_block, it)) return false;
  const int row0 = it.row0 + from;
  if (row0 >= it.rows || !edge_has_nan<D>(a, it, it.past + it.per_token * (row0 / a.group))) return false;
  const int end = row0 + n < it.rows ? row0 + n : it.rows;
  for (int i = row0; i < end; ++i) row_alone<T, D>(a, it, i);
  return true;
}

template <class T, int D, int NW, int R>
__device__ __forceinline__ void wide_body(const AttnPrefixF8 &a, const Item &it, uint32_t item0,
                                          uint8_t *smem) {
  typedef typename T::elem elem;
  typedef typename T::vec8 vec8;
  typedef Wide<D, wide_keys(D, NW, R)> C;
  constexpr int KT = C::kKeys;
  constexpr int kQ = D / 16;                     // k-steps of a logit tile
  constexpr int kDT = D / 32;                    // 32-wide tiles of O
  constexpr int kGroups = KT / 8 / NW;           // eight-key groups that a wave brings
  constexpr int kUnits = kGroups * D / 2;        // 16-byte units of their K, and of their V
  constexpr int kLoads = (kUnits + 63) / 64;     // of a lane
  static_assert(KT % (8 * NW) == 0 && kGroups <= 2, "whole groups");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int G = a.group;
  const int lg = a.page_log2, pmask = (1 << lg) - 1;
  const bool direct = a.prefix_parts + a.suffix_parts == 1;

  // This wave's rows, in R tiles of 32.
  const int row0 = it.row0 + 32 * R * wave;
  int limit[R];  // keys below it are seen
  vec8 q[R][kQ];
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const int row = row0 + 32 * w + l32;
    const bool live = row < it.rows;
    const int tok = live ? row / G : 0;
    const int hq = it.h * G + (live ? row % G : 0);
    limit[w] = it.past + it.per_token * tok;
    const elem *src = static_cast<const elem *>(a.q) + (it.tok0 + tok) * a.ldq + (int64_t)hq * D + 8 * h;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4 *>(src + 16 * i);
      q[w][i] = __builtin_bit_cast(vec8, x ^ a.q_sign);
    }
  }
  const int all_see = it.past + it.per_token * (row0 < it.rows ? row0 / G : 0);

  // Loads. A group of eight keys is 8 D bytes in one piece, of K and of V, at
  // the same offset. A wave brings kGroups groups of a tile, whose page numbers
  // are the same in all lanes (scalar loads). Unit u of a group is 16 dimensions
  // of key u / (D / 16), and of V dimensions 2 u and 2 u + 1 of the eight keys. In
  // LDS, row `key` of K has its 16-byte chunks exchanged by `swz(key)`, so that the
  // eight rows of one read phase (keys 0-3 and 8-11, or 4-7 and 12-15) lie in
  // different banks; V is as in memory.
  const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache);
  const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache);
  auto swz = [](int key) {
    return D == 96 ? (key & 3) : (key & 3) + 4 * (key >> 3 & 1);
  };
  const int last_group = (it.c1 - 1) & ~7;
  typedef const __attribute__((address_space(4))) int32_t *constant_ptr;
  const constant_ptr pages = (constant_ptr)(uintptr_t)it.pages;
  // The page numbers of the wave's groups of a tile, one tile before they are
  // needed; the groups' first vectors of the tile whose K goes out, and of the
  // tile before, whose V goes out with it.
  int32_t page_of[kGroups];
  int64_t k_vec[kGroups], v_vec[kGroups];
  auto key_of_group = [&](int tile, int i) {
    const int j = it.c0 + tile * KT + 8 * (kGroups * wave + i);
    return j < last_group ? j : last_group;
  };
  auto look_up = [&](int tile) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) page_of[i] = pages[key_of_group(tile, i) >> lg];
  };
  auto to_tile = [&](int tile) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      v_vec[i] = k_vec[i];
      const int64_t page = (uint32_t)page_of[i] < (uint32_t)a.num_pages ? page_of[i] : 0;
      k_vec[i] = ((page * a.n_kv_heads + it.h) << lg) + (key_of_group(tile, i) & pmask);
    }
    look_up(tile + 1);
  };
  struct Codes {  // of a tile, on their way
    u32x4 c[kLoads];
    uint32_t s[kLoads];
  };
  struct VCodes {
    u32x4 c[kLoads];
    u32x2 s[kLoads];  // fp16: the scales of the unit's eight keys; bf16: in [0], lane i's of key i
  };
  auto unit_of = [&](int i, int &group, int &u) {
    const int v = 64 * i + lane;
    group = kGroups > 1 ? v / (D / 2) : 0;
    u = kGroups > 1 ? v % (D / 2) : v;
    return kUnits % 64 == 0 || v < kUnits;
  };
  auto load_k = [&](Codes &x, int tile) {
    to_tile(tile);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int g, u;
      if (!unit_of(i, g, u)) continue;
      const int64_t at = kGroups > 1 && g ? k_vec[kGroups - 1] : k_vec[0];
      x.c[i] = *reinterpret_cast<const u32x4 *>(kc + at * D + 16 * u);
      x.s[i] = a.k_scales[at + u / (D / 16)];
    }
  };
  constexpr bool kScaled = __is_same(T, TypeF16);  // V's scales are in its LDS tiles
  auto load_v = [&](VCodes &x) {  // of the tile before load_k's
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int g, u;
      if (!unit_of(i, g, u)) continue;
      const int64_t at = kGroups > 1 && g ? v_vec[kGroups - 1] : v_vec[0];
      x.c[i] = *reinterpret_cast<const u32x4 *>(vc + at * D + 16 * u);
      if constexpr (kScaled) x.s[i] = *reinterpret_cast<const u32x2 *>(a.v_scales + at);
    }
    if constexpr (!kScaled) {
      const int64_t at = kGroups > 1 && (lane & 8) ? v_vec[kGroups - 1] : v_vec[0];
      x.s[0][0] = a.v_scales[at + (lane & 7)];
    }
  };
  uint8_t *const vsmem = smem + C::kStagesK * C::kHalf;
  uint8_t *const ssmem = vsmem + C::kStagesV * C::kHalf;
  auto k_stage = [&](int tile) { return smem + tile % C::kStagesK * C::kHalf; };
  auto v_stage = [&](int tile) { return vsmem + tile % C::kStagesV * C::kHalf; };
  auto s_stage = [&](int tile) { return reinterpret_cast<float *>(ssmem + tile % C::kStagesV * C::kScales); };
  auto store_k = [&](const Codes &x, int tile) {
    uint8_t *st = k_stage(tile);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int g, u;
      if (!unit_of(i, g, u)) continue;
      const int key = 8 * (kGroups * wave + g) + u / (D / 16), chunk = 2 * (u % (D / 16));
      const float f = scale_of(taken<T>(x.s[i]));
      uint8_t *to = st + key * (2 * D);
      *reinterpret_cast<vec8 *>(to + 16 * (chunk ^ swz(key))) = values8<T>(u32x2{x.c[i][0], x.c[i][1]}, f);
      *reinterpret_cast<vec8 *>(to + 16 * ((chunk + 1) ^ swz(key))) = values8<T>(u32x2{x.c[i][2], x.c[i][3]}, f);
    }
  };
  auto v_scale = [](uint32_t b) { return scale_of(taken<T>(b)); };
  auto store_v = [&](const VCodes &x, int tile) {
    uint8_t *st = v_stage(tile);
    const int j0 = it.c0 + tile * KT;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int g, u;
      if (!unit_of(i, g, u)) continue;
      // what lies behind the last key may be anything, and 0 * NaN is NaN
      const int group = kGroups * wave + g, valid = it.c1 - (j0 + 8 * group);
      const uint32_t lo = valid >= 4 ? ~0u : valid <= 0 ? 0u : ~0u >> (32 - 8 * valid);
      const uint32_t hi = valid >= 8 ? ~0u : valid <= 4 ? 0u : ~0u >> (64 - 8 * valid);
      const u32x2 c0 = {x.c[i][0] & lo, x.c[i][1] & hi}, c1 = {x.c[i][2] & lo, x.c[i][3] & hi};
      vec8 *to = reinterpret_cast<vec8 *>(st + (group * D + 2 * u) * 16);
      if constexpr (kScaled) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v_scale(x.s[i][e >> 2] >> 8 * (e & 3) & 255u);
        to[0] = values8_each(c0, f);
        to[1] = values8_each(c1, f);
      } else {
        to[0] = values8<T>(c0, 1.0f);
        to[1] = values8<T>(c1, 1.0f);
      }
    }
    if constexpr (!kScaled)
      if (lane < 8 * kGroups) s_stage(tile)[8 * kGroups * wave + lane] = v_scale(x.s[0][0]);
  };

  float16_t o[R][kDT];
  float m[R], l[R], top[R];
  float ref[R];  // m - kWideShift<T>, finite
#pragma unroll
  for (int w = 0; w < R; ++w) {
    m[w] = top[w] = -INFINITY;
    l[w] = ref[w] = 0.f;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[w][i][r] = 0.f;
  }

  // A step is 32 keys. S^T of a step: row m is key 16 (m / 16) + 8 (m / 4 % 2)
  // + 4 (m / 8 % 2) + m % 4, which leaves the weights of the step's 16-key
  // halves as the B operands of O^T = V^T P^T.
  const int key_of_lane = (l32 & 16) + 8 * (l32 >> 2 & 1) + 4 * (l32 >> 3 & 1) + (l32 & 3);
  constexpr int kM = kQ / 2;  // logit products of half a step
  static_assert(kM == kDT, "as many products of V in half a step");
  auto k_operand = [&](const uint8_t *ks, int sub, int i) {
    const int key = 32 * sub + key_of_lane;
    return *reinterpret_cast<const vec8 *>(ks + key * (2 * D) + 16 * ((2 * i + h) ^ swz(key)));
  };
  auto v_operand = [&](const uint8_t *vs, int half, int i) {  // 16 keys `half`, dimensions 32 i ..
    return *reinterpret_cast<const vec8 *>(vs + ((2 * half + h) * D + 32 * i + l32) * 16);
  };
  typedef float16_t Logits[R];
  auto mask = [&](int j0, Logits &s) {
    asm volatile("");  // stays behind its branch: few steps need it
#pragma unroll
    for (int w = 0; w < R; ++w) {
      const int seen = (limit[w] < it.c1 ? limit[w] : it.c1) - j0 - 8 * h;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (16 * (r >> 3) + (r & 7) >= seen) s[w][r] = -INFINITY;
    }
  };
  const int plain_end = it.c1 < all_see ? it.c1 : all_see;  // steps up to here need no mask
  // One step: the weights of s (32 keys, V at vs + `sub`, its scales sv) on the
  // vector ALU beside the logits of the next 32 keys (from jn, K at kn + `nsub`; past
  // the last key: of what is there, masked) on the matrix cores, then the products
  // with V beside the next maximum. Each half reads the next one's operands from
  // LDS, the last one those of K for the step after (K at ka + `asub`; one-step tiles
  // read them at the step's start, behind the barrier).
  // `first` and `second`, work on the tiles to come, go beside the products with V.
  constexpr bool kCarry = KT == 64;
  vec8 k0[kM];
  auto step = [&](const uint8_t *vs, const float *sv, int sub, const Logits &s, const uint8_t *kn,
                  int nsub, int jn, Logits &next, const uint8_t *ka, int asub, auto first,
                  auto second) {
    bool grown = false;
#pragma unroll
    for (int w = 0; w < R; ++w) grown = grown || top[w] > m[w] + kSlack;
    if (__any(grown)) {
#pragma unroll
      for (int w = 0; w < R; ++w) {
        const float mn = fmaxf(m[w], top[w]);
        const float to = (mn == -INFINITY ? 0.f : mn) - kWideShift<T>;
        const float c = m[w] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref[w] - to);
        m[w] = mn;
        ref[w] = to;
        l[w] *= c;
#pragma unroll
        for (int i = 0; i < kDT; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[w][i][r] *= c;
      }
    }
    vec8 p[R][2], k1[kM], vf[2][kDT];
    if constexpr (!kCarry) {
#pragma unroll
      for (int i = 0; i < kM; ++i) k0[i] = k_operand(kn, nsub, i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float4_t vs_lo, vs_hi;  // this lane's eight keys' scales
      if constexpr (!kScaled) {
        const float4_t *f = reinterpret_cast<const float4_t *>(sv + 32 * sub + 16 * c + 8 * h);
        vs_lo = f[0], vs_hi = f[1];
      }
      if (c == 0) {
#pragma unroll
        for (int i = 0; i < kM; ++i) k1[i] = k_operand(kn, nsub, kM + i);
      } else {
#pragma unroll
        for (int i = 0; i < kDT; ++i) vf[0][i] = v_operand(vs, 2 * sub, i);
      }
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int w = 0; w < R; ++w)
          next[w] = T::mfma32(c == 0 ? k0[i] : k1[i], q[w][c * kM + i], c + i == 0 ? float16_t{} : next[w]);
#pragma unroll
      for (int w = 0; w < R; ++w) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __builtin_amdgcn_exp2f(fmaf(s[w][8 * c + e], a.scale_log2, -ref[w]));
          sum += x;
          p[w][c][e] = (elem)(kScaled ? x : x * (e < 4 ? vs_lo[e & 3] : vs_hi[e & 3]));
        }
        l[w] += sum;
        asm volatile("" : "+v"(p[w][c]));  // computed here, not after the mask's branch
      }
      // matrix and vector instructions in turn
      __builtin_amdgcn_sched_group_barrier(0x100, kM + (kScaled ? 0 : 2), 0);
#pragma unroll
      for (int i = 0; i < R * kM; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x402, 28 / kM, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (jn + 32 > plain_end) mask(jn, next);
    float x[R];
#pragma unroll
    for (int w = 0; w < R; ++w) x[w] = -INFINITY;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c == 0) {
#pragma unroll
        for (int i = 0; i < kDT; ++i) vf[1][i] = v_operand(vs, 2 * sub + 1, i);
      } else if constexpr (kCarry) {
#pragma unroll
        for (int i = 0; i < kM; ++i) k0[i] = k_operand(ka, asub, i);
      }
#pragma unroll
      for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int w = 0; w < R; ++w) o[w][i] = T::mfma32(vf[c][i], p[w][c], o[w][i]);
#pragma unroll
      for (int w = 0; w < R; ++w)
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          x[w] = fmaxf(fmaxf(next[w][8 * c + e], next[w][8 * c + e + 1]), x[w]);
      if (c == 0) first();
      else second();
      __builtin_amdgcn_sched_group_barrier(0x100, kDT, 0);
#pragma unroll
      for (int i = 0; i < R * kDT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, 32 / (R * kDT), 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int w = 0; w < R; ++w) top[w] = max_over_halves(x[w]) * a.scale_log2;
  };

  // K is used up to one tile before V.
  const int tiles = (it.c1 - it.c0 + KT - 1) / KT;
  Logits s, s2;
  Codes xk;
  VCodes xv;
  if (tiles > 0) {
    look_up(0);
    load_k(xk, 0);
    store_k(xk, 0);
    load_k(xk, 1);
    load_v(xv);
    store_k(xk, 1);
    store_v(xv, 0);
    load_k(xk, 2);
    load_v(xv);
    store_k(xk, 2);
    store_v(xv, 1);
    load_k(xk, 3);
    load_v(xv);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const vec8 k = k_operand(smem, 0, i);
#pragma unroll
      for (int w = 0; w < R; ++w) s[w] = T::mfma32(k, q[w][i], i == 0 ? float16_t{} : s[w]);
    }
    if (it.c0 + 32 > plain_end) mask(it.c0, s);
#pragma unroll
    for (int w = 0; w < R; ++w) {
      float x = s[w][0];
#pragma unroll
      for (int r = 1; r < 16; ++r) x = fmaxf(x, s[w][r]);
      top[w] = max_over_halves(x) * a.scale_log2;
    }
    if constexpr (kCarry) {
#pragma unroll
      for (int i = 0; i < kM; ++i) k0[i] = k_operand(smem, 1, i);
    }
  }
#pragma unroll 1
  for (int kt = 0; kt < tiles; ++kt) {  // (two tiles between barriers)
    if (kt && (kt & 1) == 0) __syncthreads();
    const int j0 = it.c0 + kt * KT;
    const uint8_t *vs = v_stage(kt), *kn = k_stage(kt + 1);
    const float *sv = s_stage(kt);
    // K of the tile three ahead and V of the one two ahead have come: they go to
    // LDS, and the next ones out. (Past the last tile too: what is written there is
    // not read, and what is loaded is the last group again.)
    auto k_on = [&]() {
      store_k(xk, kt + 3);
      load_k(xk, kt + 4);
    };
    auto v_on = [&]() {
      store_v(xv, kt + 2);
      load_v(xv);
    };
    auto nothing = []() {};
    if constexpr (KT == 64) {
      step(vs, sv, 0, s, k_stage(kt), 1, j0 + 32, s2, kn, 0, nothing, k_on);
      step(vs, sv, 1, s2, kn, 0, j0 + 64, s, kn, 1, v_on, nothing);
    } else {
      step(vs, sv, 0, s, kn, 0, j0 + 32, s2, nullptr, 0, k_on, v_on);
#pragma unroll
      for (int w = 0; w < R; ++w) s[w] = s2[w];
    }
  }

  // this lane's rows again: nothing of them is held through the loop
  int lane_row = l32;
  asm volatile("" : "+v"(lane_row));
  bool live[R];
  int64_t flat[R];  // (token, head)
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const int row = row0 + 32 * w + lane_row;
    live[w] = row < it.rows;
    const int tok = live[w] ? row / G : 0;
    flat[w] = (it.tok0 + tok) * a.n_q_heads + it.h * G + (live[w] ? row % G : 0);
  }
  if (it.c1 > plain_end) {
    bool bad = false;  // (of rows that are there)
#pragma unroll
    for (int w = 0; w < R; ++w)
#pragma unroll
      for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) bad = bad || (live[w] && o[w][i][r] != o[w][i][r]);
    if (__any(bad) && wave_again<T, D>(item0, 32 * R * NW, 32 * R * wave, 32 * R)) return;
  }

  const int64_t nrows = a.tokens * a.n_q_heads;
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const float sum = sum_over_halves(l[w]);
    if (!live[w]) continue;
    if (direct) {
      typedef elem vec4 __attribute__((ext_vector_type(4)));
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      elem *dst = static_cast<elem *>(a.out) + flat[w] * D + 4 * h;
#pragma unroll
      for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<vec4 *>(dst + 32 * i + 2 * r) =
              vec4{(elem)(o[w][i][r] * inv), (elem)(o[w][i][r + 1] * inv),
                   (elem)(o[w][i][r + 2] * inv), (elem)(o[w][i][r + 3] * inv)};
      if (h == 0 && a.lse) a.lse[flat[w]] = lse_of(m[w] - kWideShift<T>, sum);
    } else {
      float *dst = a.part_o + (it.part * nrows + flat[w]) * D + 4 * h;
#pragma unroll
      for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<float4_t *>(dst + 32 * i + 2 * r) =
              float4_t{o[w][i][r], o[w][i][r + 1], o[w][i][r + 2], o[w][i][r + 3]};
      if (h == 0) a.part_ml[it.part * nrows + flat[w]] = make_float2(m[w] - kWideShift<T>, sum);
    }
  }
}

template <class T, int D, int NW, int R>
__global__ void __launch_bounds__(64 * NW, wide_waves(D, NW, R))
attn_f8_wide_kernel(AttnPrefixF8 a, uint32_t item0) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  Item it;
  const uint32_t idx = item_of(a, item0, blockIdx.x, gridDim.x);
  rows_of_no_sequence<T, D>(a, idx, 64 * NW);
  if (find_item(a, idx, 32 * R * NW, it) && !empty_item(a, it, 32 * R * NW, 64 * NW))
    wide_body<T, D, NW, R>(a, it, item0, smem);
}

// Joins the partial results of each row. D / 4 threads take a part, four
// dimensions each, and `slots` such groups share a row's parts, so that a row of
// many parts is a few round trips to memory (one conversation of 30001 keys, 32
// parts of 32 rows: with one group a row the join is half of the call). Groups'
// sums are added in LDS in a fixed order. Weights as in attn_join_kernel.
template <int D>
constexpr int kJoinGroups = D == 64 ? 16 : D <= 128 ? 8 : 4;

template <class T, int D>
__global__ void __launch_bounds__(kThreads)
attn_f8_join_kernel(AttnPrefix a, uint32_t first, int slots) {
  typedef typename T::elem elem;
  constexpr int kPer = D / 4, kGroups = kJoinGroups<D>;
  __shared__ float top[kGroups], sum[kGroups];
  __shared__ __attribute__((aligned(16))) float part[kGroups][D];
  const int group = threadIdx.x / kPer, slot = group % slots;
  const int64_t nrows = a.tokens * a.n_q_heads;
  const int64_t row = (int64_t)(first + blockIdx.x) * (kGroups / slots) + group / slots;
  const int d = 4 * (threadIdx.x % kPer);
  const bool live = group < kGroups && row < nrows;
  const int parts = a.prefix_parts + a.suffix_parts;
  float m = -INFINITY;
  int end = 0;  // behind the last part that sees a key
  if (live) {
#pragma unroll 4
    for (int p = slot; p < parts; p += slots) {
      const float2 ml = a.part_ml[p * nrows + row];
      m = fmaxf(m, ml.x);
      if (ml.y != 0.f) end = p + 1;
    }
  }
  if (slots > 1) {
    if (live && d == 0) top[group] = m;
    __syncthreads();
  }
  float l = 0.f;
  float4_t o = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    if (slots > 1)
      for (int i = group - slot; i < group - slot + slots; ++i) m = fmaxf(m, top[i]);
#pragma unroll 4
    for (int p = slot; p < end; p += slots) {
      // of a part that sees no key nothing counts
      const float2 ml = a.part_ml[p * nrows + row];
      const float4_t x = *reinterpret_cast<const float4_t *>(a.part_o + (p * nrows + row) * D + d);
      const bool seen = ml.y != 0.f;
      const float w = seen ? __builtin_amdgcn_exp2f(ml.x - m) * kJoinWeight : 0.f;
      l += w * (seen ? ml.y : 0.f);
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] += w * (seen ? x[r] : 0.f);
    }
  }
  if (slots > 1) {
    if (live) {
      *reinterpret_cast<float4_t *>(&part[group][d]) = o;
      if (d == 0) sum[group] = l;
    }
    __syncthreads();
  }
  if (!live || slot) return;
  for (int i = 1; i < slots; ++i) {
    l += sum[group + i];
    o += *reinterpret_cast<const float4_t *>(&part[group + i][d]);
  }
  // of a row of no sequence nothing read above counts
  if (a.q_start && a.part_ml[a.prefix_parts * nrows + row].y == kNoSequence) {
    l = 0.f;
    o = float4_t{0.f, 0.f, 0.f, 0.f};
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  typedef elem vec4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<vec4 *>(static_cast<elem *>(a.out) + row * D + d) =
      vec4{(elem)(o[0] * inv), (elem)(o[1] * inv), (elem)(o[2] * inv), (elem)(o[3] * inv)};
  if (a.lse && d == 0) a.lse[row] = lse_of(m, l * (1 << kJoinShift));
}

template <class T, int D, int NW, int R>
hipError_t launch_wide(const AttnPrefixF8 &a, int64_t item0, int64_t items, hipStream_t stream) {
  constexpr auto kern = attn_f8_wide_kernel<T, D, NW, R>;
  constexpr int kLds = Wide<D, wide_keys(D, NW, R)>::kLds;
  const hipError_t e = ensure_max_lds<kern>(kLds);
  if (e != hipSuccess) return e;
  return launch_in_pieces(items, 64 * NW, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL(kern, dim3(n), dim3(64 * NW), kLds, stream, a, (uint32_t)item0 + first);
  });
}

// Workgroups of 256 rows are eight waves of 32, or four of 64, as in
// attn_prefix.hip.
template <class T, int D>
hipError_t launch_items(const AttnPrefixF8 &a, int wide, int64_t item0, int64_t items,
                        hipStream_t stream) {
  if (items == 0) return hipSuccess;
  if (wide == 2) {
    if constexpr (D == 128) return launch_wide<T, D, 8, 1>(a, item0, items, stream);
    if constexpr (D < 128) return launch_wide<T, D, 4, 2>(a, item0, items, stream);
    return hipErrorInvalidValue;
  }
  if (wide == 1) return launch_wide<T, D, 4, 1>(a, item0, items, stream);
  return launch_in_pieces(items, kThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((attn_f8_rows16_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a,
                       (uint32_t)item0 + first);
  });
}

// The prefix's and the suffixes' items are launched together when they are of
// one kind.
template <class T, int D>
hipError_t launch(const AttnPrefixF8 &a, hipStream_t stream) {
  hipError_t e;
  if (a.prefix_wide == a.suffix_wide || a.prefix_items == 0) {
    e = launch_items<T, D>(a, a.suffix_wide, 0, a.prefix_items + a.suffix_items, stream);
  } else {
    e = launch_items<T, D>(a, a.prefix_wide, 0, a.prefix_items, stream);
    if (e != hipSuccess) return e;
    e = launch_items<T, D>(a, a.suffix_wide, a.prefix_items, a.suffix_items, stream);
  }
  if (e != hipSuccess || a.prefix_parts + a.suffix_parts == 1) return e;
  // parts are shared out where a group a row would leave CUs empty (each takes
  // four workgroups)
  const int64_t rows = a.tokens * a.n_q_heads;
  int slots = 1;
  while (slots < kJoinGroups<D> && 2 * slots <= a.prefix_parts + a.suffix_parts &&
         rows * slots < kJoinGroups<D> * 1024ll)
    slots *= 2;
  const int64_t per = kJoinGroups<D> / slots;
  return launch_in_pieces((rows + per - 1) / per, kThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((attn_f8_join_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a, first, slots);
  });
}

template <class T>
hipError_t launch_dim(const AttnPrefixF8 &a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch<T, 64>(a, stream);
    case 96: return launch<T, 96>(a, stream);
    case 128: return launch<T, 128>(a, stream);
    case 256: return launch<T, 256>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// Splits the keys so that the launch fills the chip. A chunk is a multiple of
// 128 keys and at most kAttnMaxChunk.
void attn_f8_plan(AttnPrefixF8 &a, int64_t max_suffix, int num_cus) {
  // Rows of a work item: 16, 128 or 256 (wide 0, 1, 2), the least of an estimate
  // fitted to measured calls: until the first results, which wait for up to 512
  // or 768 keys, and then for each row block, key and head (ps), to which an
  // item's start counts as 100 or 250 keys. 16 rows read the cache again for every
  // 16. Measured, 8 key heads, fp16 (us; 16 / 128 / 256):
  // 128 dimensions, 60001 keys, 64 rows 59 / 70 / 79, 128 rows 99 / 74 / 85,
  // 256 rows 174 / 112 / 94; 16001 keys, 128 rows 30 / 37 / 34, 256 rows
  // 52 / 46 / 41; 4001 keys, 384 rows 29 / 34 / 36; 64 dimensions, 60001 keys,
  // 64 rows 35 / 42 / 56, 128 rows 59 / 44 / 58, 256 rows 102 / 64 / 65; 32 x 64
  // keys, 128 rows each 18 / 13, 256 rows 30 / 17 / 17; 256 rows behind 8000 shared
  // keys 32 / - / 39.
  auto wide_for = [&](int64_t rows, int64_t sequences, int64_t keys) {
    struct Cost {
      int rows16, rows128, rows256;
    };
    const Cost c = a.head_dim == 64   ? Cost{12, 47, 62}
                   : a.head_dim == 96 ? Cost{15, 80, 158}
                   : a.head_dim == 128 ? Cost{20, 85, 130}
                                       : Cost{47, 242, 0};
    if (rows <= kRows) return 0;
    const double heads = (double)sequences * a.n_kv_heads;
    const auto until = [&](int most) { return 27e3 * (keys < most ? keys : most); };
    const double few = 5e6 + until(512) / 2 + c.rows16 * heads * (keys + 250) * ((rows + 15) / 16);
    const double mid = 8e6 + until(768) + c.rows128 * heads * (keys + 100) * ((rows + 127) / 128);
    const double many = 10e6 + until(768) + c.rows256 * heads * (keys + 100) * ((rows + 255) / 256);
    if (c.rows256 && many < mid && many < few) return 2;
    return mid < few ? 1 : 0;
  };
  // Chunk for `keys` keys of `blocks` row blocks. 16-row kernel: as many chunks as
  // give each CU a workgroup. With few blocks more chunks cost more at the join
  // than they gain (1 x 30001 keys, 8 key heads of 128 fp16: 18.6 us with one
  // workgroup a CU, 22 with two, 26 with four), with many one chunk a sequence is
  // near the cache's read (64 x 8001 ragged: 112 us, 126 with two to four). Once
  // a sequence is cut, it is into chunks of at most 2048 keys: lengths differ, and
  // the call ends with the longest chunks (24 x 8209 ragged, 8 key heads: 51 us,
  // 60 with two chunks; 32 key heads 149, 172 with two; 64 x 12001, 8 key heads
  // 150, 160 with two). That stops at 16 workgroups a CU, since a table may be much
  // wider than the sequences (24 x 1000 keys under a table of 131072: 37 us with 64
  // chunks, 19 with 21, 17 with 16; of 1024: 15.6). Wide kernel: whole rounds over what the CUs hold.
  auto chunk_of = [&](int64_t keys, int64_t blocks, int wide) {
    const int64_t most = (keys + 127) / 128;
    int64_t parts = (num_cus + blocks - 1) / blocks;
    if (wide) {
      const int64_t room = (a.head_dim == 64 || (wide == 1 && a.head_dim <= 128) ? 2 : 1) * num_cus;
      int64_t best = -1;
      for (int64_t p = 1; p <= most && p <= 64; ++p) {
        const int64_t chunk = ((keys + p - 1) / p + 127) / 128 * 128;
        // a workgroup's fixed cost is about that of 256 keys, and a part's, whose
        // results are written and read once more, of blocks * head_dim / 96
        const int64_t cost = (blocks * p + room - 1) / room * (chunk + 256) + p * blocks * a.head_dim / 96;
        if (best < 0 || cost < best) {
          best = cost;
          parts = p;
        }
      }
    }
    if (!wide && (parts > 1 || keys > kAttnMaxChunk)) {
      int64_t cut = (keys + 2047) / 2048;
      if (cut > 16ll * num_cus / blocks) cut = 16ll * num_cus / blocks;
      if (parts < cut) parts = cut;
    }
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    int64_t chunk = ((keys + parts - 1) / parts + 127) / 128 * 128;
    if (chunk > kAttnMaxChunk) chunk = kAttnMaxChunk;
    return (int)chunk;
  };
  auto block_rows = [](int wide) { return wide ? 128 * wide : kRows; };
  a.group = a.n_q_heads / a.n_kv_heads;
  const int64_t prefix_rows = a.tokens * a.group, suffix_rows = a.max_q * a.group;
  a.prefix_wide = wide_for(prefix_rows, 1, a.prefix_len);
  a.suffix_wide = wide_for(suffix_rows, a.batch, max_suffix);
  int64_t per = block_rows(a.prefix_wide);
  a.prefix_row_blocks = (int)((prefix_rows + per - 1) / per);
  a.prefix_chunk = a.prefix_parts = 0;
  if (a.prefix_len > 0) {
    a.prefix_chunk = chunk_of(a.prefix_len, (int64_t)a.prefix_row_blocks * a.n_kv_heads, a.prefix_wide);
    a.prefix_parts = (int)((a.prefix_len + a.prefix_chunk - 1) / a.prefix_chunk);
  }
  a.prefix_items = (int64_t)a.prefix_row_blocks * a.n_kv_heads * a.prefix_parts;
  per = block_rows(a.suffix_wide);
  a.suffix_row_blocks = (int)((suffix_rows + per - 1) / per);
  a.suffix_chunk = chunk_of(max_suffix, a.batch * a.n_kv_heads * a.suffix_row_blocks, a.suffix_wide);
  a.suffix_parts = (int)((max_suffix + a.suffix_chunk - 1) / a.suffix_chunk);
  a.suffix_items = a.batch * a.n_kv_heads * a.suffix_row_blocks * a.suffix_parts;
}

hipError_t attn_f8_launch(AttnPrefixF8 &a, void *ws, ElemType type, hipStream_t stream) {
  if (a.prefix_items + a.suffix_items > 0x7fffffff) return hipErrorInvalidValue;
  const int64_t rows = a.tokens * a.n_q_heads;
  a.part_o = static_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(static_cast<float *>(ws) +
                                         (a.prefix_parts + a.suffix_parts) * rows * a.head_dim);
  return type == ElemType::F16 ? launch_dim<TypeF16>(a, stream) : launch_dim<TypeBF16>(a, stream);
}

}  // namespace lqmm
