// Attention over a paged cache for a batch of sequences that share a prefix.
//
// Mathematics. Row (t, h) (a token and a query head) sees the keys 0 ..
// prefix - 1 of the shared pages and then, of its own sequence's pages, the
// keys 0 .. len - new + i (i: the token's number among the sequence's new
// ones). With z_j = scale * log2(e) * q.k_j and any reference m,
//   O = sum_j 2^(z_j - m) v_j / sum_j 2^(z_j - m),
// so any split of the keys gives partial (m, l, O) triples that are joined
// exactly by rescaling to the largest m. The prefix is one such split: its
// keys are the same for every sequence, so all rows of a key head are
// multiplied with each prefix key while it is on the chip, and the prefix is
// read once and not once for each sequence.
//
// Layout on the matrix cores. S^T = K Q^T puts a row's logits in one lane
// column (lane & 15), four keys per register group; V pages keep eight
// tokens of one dimension adjacent, so the A operand of O^T = V^T P^T is one
// 16-byte load per lane. Which key is which row of the S^T tile is free, so
// tile t of a 32-key step takes key 8 g + 4 t + r as row 4 g + r: then the
// exponentials of the two tiles are, in place, the B operand of the second
// product, and no value crosses a lane except the row maximum.
//
// A row or part that sees no key has the sum 0. Its maximum, -infinity, does not
// tell: maxima leave NaN out, so that a row whose every logit is NaN has it too,
// with a sum of NaN, which has to reach the output.
//
// P is rounded to the cache's 16-bit type, as the matrix cores want it, and
// kept at 2^kShift times its value. In fp16 that is up, so that weights down to
// 2^-(24 + kShift) of the largest do not vanish (values of fp16 are far from
// overflowing O); in bf16, whose values may be as large as an fp32, it is down:
// a work item's at most 2^13 weights add up to less than 1, and so does O to
// less than the largest value. Logits, maxima, sums and O are fp32.
//
// Two kernels. Few rows (one new token's heads) are bound by reading the
// cache: 16 rows a workgroup, the waves take different keys, straight from
// memory to the operands. Many rows (a prefix under a batch, a chunk of new
// tokens) are bound by the matrix cores: 32 rows a wave, all waves of a
// workgroup take the same keys from LDS tiles that are filled ahead.
#include "attn_common.hpp"

namespace lqmm {
namespace {

// log2 of what weights are held at, times their value
template <class T>
constexpr float kShift = __is_same(T, TypeF16) ? 14.0f : -14.0f;
constexpr float kAloneShift = -14.0f;  // of rows done by themselves, in fp32

// ---- values behind a mask -------------------------------------------------------
// A masked weight is 0, and 0 times a value that is infinite or NaN is NaN: a
// new token with such a value would reach the new tokens before it, whose mask
// leaves it out, through the matrix products. That leaves NaN in O, which is
// looked for once, behind the keys' loop; rows of a block that has such a
// value among the keys of its mask's edge are done again, by themselves.
// (A test of the values in the loop would be made for every key of the edge.)
template <class T, int D>
__device__ __forceinline__ int64_t element_at(const AttnPrefix &a, const Item &it, int j) {
  const int32_t p = it.pages[j >> a.page_log2];
  const int64_t page = (uint32_t)p < (uint32_t)a.num_pages ? p : 0;
  return ((page * a.n_kv_heads + it.h) * D << a.page_log2) +
         (int64_t)(j & ((1 << a.page_log2) - 1)) * D;
}

// Whether V of the keys [from, it.c1) has a value that is not finite (one wave).
template <class T, int D>
__device__ __forceinline__ bool edge_not_finite(const AttnPrefix &a, const Item &it, int from) {
  typedef typename T::vec8 vec8;
  const int lane = threadIdx.x & 63;
  const typename T::elem *vc = static_cast<const typename T::elem *>(a.v_cache);
  if (from < it.c0) from = it.c0;
  bool found = false;
#pragma unroll 1
  for (int j0 = from & ~7; j0 < it.c1; j0 += 8) {
    const int64_t at = element_at<T, D>(a, it, j0);
    for (int d = lane; d < D; d += 64) {
      const vec8 x = *reinterpret_cast<const vec8 *>(vc + at + 8 * d);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        found = found || (j0 + e >= from && j0 + e < it.c1 && !(fabsf((float)x[e]) < INFINITY));
    }
  }
  return __any(found);
}

// One row of an item by one wave: a lane a key for the logits, a lane a
// dimension for O, only of keys that the row sees.
template <class T, int D>
__device__ __forceinline__ void row_alone(const AttnPrefix &a, const Item &it, int row) {
  typedef typename T::elem elem;
  constexpr int kO = (D + 63) / 64;
  const int lane = threadIdx.x & 63, G = a.group;
  const int tok = row / G;
  const int64_t flat = (it.tok0 + tok) * a.n_q_heads + it.h * G + row % G;
  const int limit = it.past + it.per_token * tok;
  const int end = limit < it.c1 ? limit : it.c1;
  const elem *q = static_cast<const elem *>(a.q) + (it.tok0 + tok) * a.ldq + (int64_t)(it.h * G + row % G) * D;
  const elem *kc = static_cast<const elem *>(a.k_cache), *vc = static_cast<const elem *>(a.v_cache);
  const float scale = a.q_sign ? -a.scale_log2 : a.scale_log2;
  float m = -INFINITY, l = 0.f, o[kO];
#pragma unroll
  for (int i = 0; i < kO; ++i) o[i] = 0.f;
  for (int j0 = it.c0; j0 < end; j0 += 64) {
    float z = -INFINITY;
    if (j0 + lane < end) {
      const elem *k = kc + element_at<T, D>(a, it, j0 + lane);
      float dot = 0.f;
#pragma unroll 1
      for (int d = 0; d < D; d += 8) {
        float x[8], y[8];
        load8<T>(q + d, x);
        load8<T>(k + d, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(x[e], y[e], dot);
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
      const float w = __shfl(e, i);
      const int j = j0 + i;
      const elem *v = vc + element_at<T, D>(a, it, j & ~7) + (j & 7);
#pragma unroll
      for (int u = 0; u < kO; ++u)
        if (lane + 64 * u < D) o[u] += w * (float)v[8 * (lane + 64 * u)];
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
template <int D, int NW>
struct Rows16 {
  static constexpr int kPass = D / 16 < 8 ? D / 16 : 8;  // O tiles joined at a time
  static constexpr int kLd = 16 * kPass + 4;
  int ids[kMaxIds];
  float wave_m[NW][kRows], wave_l[NW][kRows];
  __attribute__((aligned(16))) float join[NW][kRows][kLd];
};

template <class T, int D, int NW>
__device__ __forceinline__ void rows16_body(const AttnPrefix &a, const Item &it, Rows16<D, NW> &sm) {
  typedef typename T::elem elem;
  typedef typename T::vec8 vec8;
  constexpr int kQ = D / 32;                       // k-steps of one logit tile
  constexpr int kDT = D / 16;                      // 16-wide tiles of O
  constexpr int kPass = Rows16<D, NW>::kPass;
  static_assert(kDT % kPass == 0, "whole passes");
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
  vec8 q[kQ];
  {
    const elem *src = static_cast<const elem *>(a.q) + t * a.ldq + (int64_t)hq * D + 8 * g;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4 *>(src + 32 * i);
      q[i] = __builtin_bit_cast(vec8, x ^ a.q_sign);
    }
  }
  __syncthreads();

  float4_t o[kDT];
#pragma unroll
  for (int i = 0; i < kDT; ++i) o[i] = float4_t{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  const elem *kc = static_cast<const elem *>(a.k_cache);
  const elem *vc = static_cast<const elem *>(a.v_cache);
  const int64_t head_elems = (int64_t)D << lg;
  // first element of the eight-token group that holds key j (j % 8 == 0)
  auto group_at = [&](int j) -> int64_t {
    const int64_t page = ids[(j >> lg) - page0];
    return (page * a.n_kv_heads + it.h) * head_elems + (int64_t)(j & pmask) * D;
  };
  const int last_group = (it.c1 - 1) & ~7;
  auto clamp_group = [&](int j) { return j < last_group ? j : last_group; };

  vec8 kf[2][kQ];
  auto load_k = [&](int j0) {
    const int64_t base = group_at(clamp_group(j0 + 8 * (m16 >> 2)));
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < kQ; ++i)
        kf[s][i] = *reinterpret_cast<const vec8 *>(kc + base + (4 * s + (m16 & 3)) * D + 32 * i + 8 * g);
  };

  int j0 = it.c0 + wave * kStep;
  if (j0 < it.c1) load_k(j0);
  for (; j0 < it.c1; j0 += NW * kStep) {
    vec8 vf[kDT];
    {
      const int64_t base = group_at(clamp_group(j0 + 8 * g));
#pragma unroll
      for (int i = 0; i < kDT; ++i)
        vf[i] = *reinterpret_cast<const vec8 *>(vc + base + (16 * i + m16) * 8);
    }
    float4_t s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kQ; ++i) s[u] = T::mfma16(kf[u][i], q[i], s[u]);
    }
    if (j0 + NW * kStep < it.c1) load_k(j0 + NW * kStep);
    float z[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) z[u][r] = s[u][r] * a.scale_log2;
    const int seen = limit < it.c1 ? limit : it.c1;
    if (j0 + kStep > it.c1 || j0 + kStep > all_see) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j0 + 8 * g + 4 * u + r >= seen) z[u][r] = -INFINITY;
      // what lies behind the last key may be anything, and 0 * NaN is NaN
      if (j0 + kStep > it.c1) {
        const int valid = it.c1 - (j0 + 8 * g);
#pragma unroll
        for (int i = 0; i < kDT; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e >= valid) vf[i][e] = (elem)0.f;
      }
    }
    float top = fmaxf(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3])),
                      fmaxf(fmaxf(z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3])));
    const float mn = fmaxf(m, max_over_rows(top));
    const float ref = (mn == -INFINITY ? 0.f : mn) - kShift<T>;
    // (between references, as they were rounded)
    const float corr = __builtin_amdgcn_exp2f(m - kShift<T> - ref);
    const float c = m == -INFINITY ? 0.f : corr;
    m = mn;
    vec8 p;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = __builtin_amdgcn_exp2f(z[u][r] - ref);
        sum += e;
        p[4 * u + r] = (elem)e;
      }
    l = l * c + sum;
#pragma unroll
    for (int i = 0; i < kDT; ++i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) o[i][r] *= c;
      o[i] = T::mfma16(vf[i], p, o[i]);
    }
  }

  if (it.c1 > all_see) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) bad = bad || o[i][r] != o[i][r];
    if (__syncthreads_or(live && bad) && edge_not_finite<T, D>(a, it, all_see)) {
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
    for (int i = 0; i < kPass; ++i) {
      float4_t x = o[pass * kPass + i];
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] *= mine;
      *reinterpret_cast<float4_t *>(&sm.join[wave][m16][16 * i + 4 * g]) = x;
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
__global__ void __launch_bounds__(kThreads)
attn_rows16_kernel(AttnPrefix a, uint32_t item0) {
  __shared__ Rows16<D, kThreads / 64> sm;
  Item it;
  const uint32_t idx = item0 + spread(blockIdx.x, gridDim.x);
  rows_of_no_sequence<T, D>(a, idx, kThreads);
  if (find_item(a, idx, kRows, it))
    rows16_body<T, D, kThreads / 64>(a, it, sm);
}

// ---- many rows -----------------------------------------------------------------
// A running maximum that grows by no more than kSlack (log2) is left where it
// is: O is rescaled when a row needs it, not at every step.
constexpr float kSlack = 8.0f;
// Weights are at most 2^(kSlack + kWideShift): 2^kShift.
template <class T>
constexpr float kWideShift = kShift<T> - kSlack;

// Waves of a SIMD that the wide kernel's registers leave room for: two of 32
// rows, one of 64 rows (two at 64 dimensions) or of 256 dimensions.
constexpr int wide_waves(int d, int nw, int r) {
  return r > 1 ? (d == 64 ? 2 : 1) : d <= 128 && nw == 8 ? 2 : 1;
}

template <int D>
struct Wide {
  static constexpr int kKeys = D <= 128 ? 64 : 32;  // keys of a tile
  static constexpr int kHalf = kKeys * D * 2;       // bytes of a tile's K (and V)
  // a round is two tiles between barriers: K of it and of the tile after, V of
  // it, and the next round's two tiles of each on their way
  static constexpr int kStagesK = 5, kStagesV = 4;
  static constexpr int kLds = (kStagesK + kStagesV) * kHalf;
};

// The rows of a wave again, if its mask's edge asks for it (whether it did). Item
// and arguments are read once more, so that nothing of them is held in registers
// through the keys' loop for this (768 rows x 32801 keys of 128: 159 us with the
// loop's own, 154 so; the 16-row kernel has registers to spare and is slower this
// way, 24 x 4111 keys 154 / 161 us).
template <class T, int D>
__device__ __forceinline__ bool wave_again(uint32_t item0, int rows_per_block, int from, int n) {
  uint64_t args = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  uint32_t block = blockIdx.x;
  asm volatile("" : "+s"(args), "+s"(block));
  const AttnPrefix &a = *reinterpret_cast<const AttnPrefix *>(args);  // the kernel's first argument
  Item it;
  if (!find_item(a, item0 + spread(block, gridDim.x), rows_per_block, it)) return false;
  const int row0 = it.row0 + from;
  if (row0 >= it.rows || !edge_not_finite<T, D>(a, it, it.past + it.per_token * (row0 / a.group)))
    return false;
  const int end = row0 + n < it.rows ? row0 + n : it.rows;
  for (int i = row0; i < end; ++i) row_alone<T, D>(a, it, i);
  return true;
}

template <class T, int D, int NW, int R>
__device__ __forceinline__ void wide_body(const AttnPrefix &a, const Item &it, uint32_t item0,
                                          uint8_t *smem) {
  typedef typename T::elem elem;
  typedef typename T::vec8 vec8;
  typedef Wide<D> C;
  constexpr int KT = C::kKeys;
  constexpr int kQ = D / 16;                    // k-steps of a logit tile
  constexpr int kDT = D / 32;                   // 32-wide tiles of O
  constexpr int kLoads = C::kHalf / 1024 / NW;  // 1 KB loads of a wave for K, and for V
  constexpr int kGroups = KT / 8 / NW;          // eight-key groups that a wave loads
  static_assert(C::kHalf % (1024 * NW) == 0 && KT % (8 * NW) == 0, "whole loads");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int G = a.group;
  const int lg = a.page_log2, pmask = (1 << lg) - 1;
  const bool direct = a.prefix_parts + a.suffix_parts == 1;

  // This wave's rows, in R tiles of 32.
  const int row0 = it.row0 + 32 * R * wave;
  bool live[R];
  int64_t flat[R];  // (token, head) of this lane's rows
  int limit[R];     // keys below it are seen
  vec8 q[R][kQ];
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const int row = row0 + 32 * w + l32;
    live[w] = row < it.rows;
    const int tok = live[w] ? row / G : 0;
    const int hq = it.h * G + (live[w] ? row % G : 0);
    flat[w] = (it.tok0 + tok) * a.n_q_heads + hq;
    limit[w] = it.past + it.per_token * tok;
    const elem *src = static_cast<const elem *>(a.q) + (it.tok0 + tok) * a.ldq + (int64_t)hq * D + 8 * h;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4 *>(src + 16 * i);
      q[w][i] = __builtin_bit_cast(vec8, x ^ a.q_sign);
    }
  }
  const int all_see = it.past + it.per_token * (row0 < it.rows ? row0 / G : 0);

  // Loads. The eight keys of a group are 16 D bytes in one piece, of K and of
  // V, at the same offset. A wave brings kGroups groups of a tile: its page
  // numbers are the same in all lanes (scalar loads and addresses), its lanes'
  // places in a group are fixed. In LDS, row `key` of K has its 16-byte
  // chunks exchanged by `swz(key)`, so that the eight rows of one read phase
  // (keys 0-3 and 8-11, or 4-7 and 12-15) lie in different banks; V is as in
  // memory.
  const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache);
  const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache);
  const int64_t head_bytes = (int64_t)(2 * D) << lg;
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row of K
  auto swz = [](int key) {
    return D == 96 ? (key & 3) : (key & 3) + 4 * (key >> 3 & 1);
  };
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int u = i * 64 + lane;  // 16-byte unit of the wave's groups
    const int key = 8 * kGroups * wave + u / kChunks;
    koff[i] = (uint32_t)((u % D / kChunks) * 2 * D + 16 * ((u % kChunks) ^ swz(key)));
    voff[i] = (uint32_t)(u % D) * 16;
  }
  const int last_group = (it.c1 - 1) & ~7;
  // The page numbers of the wave's groups of a tile, one tile before they are
  // needed (constant memory: scalar loads, which no pending LDS load holds up).
  typedef const __attribute__((address_space(4))) int32_t *constant_ptr;
  const constant_ptr pages = (constant_ptr)(uintptr_t)it.pages;
  struct Pages {
    int32_t n[kGroups];
  };
  auto key_of_group = [&](int j0, int i) {
    const int j = j0 + 8 * (kGroups * wave + i);
    return j < last_group ? j : last_group;
  };
  auto pages_of = [&](int j0) {
    Pages p;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) p.n[i] = pages[key_of_group(j0, i) >> lg];
    return p;
  };
  auto load_half = [&](const uint8_t *cache, const uint32_t (&off)[kLoads], int j0, const Pages &p,
                       uint8_t *dst) {
    const uint8_t *base[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int64_t page = (uint32_t)p.n[i] < (uint32_t)a.num_pages ? p.n[i] : 0;
      const uint64_t at = reinterpret_cast<uint64_t>(cache) +
                          (uint64_t)((page * a.n_kv_heads + it.h) * head_bytes +
                                     (int64_t)(key_of_group(j0, i) & pmask) * (2 * D));
      base[i] = reinterpret_cast<const uint8_t *>(at);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      constexpr int last = kGroups - 1;
      const int g0 = 64 * i / D, g1 = (64 * i + 63) / D;  // groups that the load touches
      uint8_t *to = dst + (wave * kLoads + i) * 1024;
      if (g0 == g1) {  // scalar base, 32-bit lane offsets
        const rsrc_t r = make_rsrc(base[g0 < last ? g0 : last], 16 * D);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, (int)off[i], 0, 0, 0);
      } else {
        load_to_lds<16>(((i * 64 + lane) / D == g0 ? base[g0] : base[g1 < last ? g1 : last]) + off[i], to);
      }
    }
  };
  // K is used up to one tile before V: the loads go out as pairs K of tile
  // p + 1, V of tile p.
  uint8_t *const vsmem = smem + C::kStagesK * C::kHalf;
  auto k_stage = [&](int tile) { return smem + tile % C::kStagesK * C::kHalf; };
  auto v_stage = [&](int tile) { return vsmem + tile % C::kStagesV * C::kHalf; };
  Pages pk, pv;  // of the next pair
  auto next_pages = [&](int p) {
    pv = pages_of(it.c0 + p * KT);
    pk = pages_of(it.c0 + (p + 1) * KT);
  };
  auto load_pair = [&](int p) {
    load_half(kc, koff, it.c0 + (p + 1) * KT, pk, k_stage(p + 1));
    load_half(vc, voff, it.c0 + p * KT, pv, v_stage(p));
    next_pages(p + 1);
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

  // One step: the weights of s (32 keys, V at vs + `sub`) on the vector ALU
  // beside the logits of the next 32 keys (from jn, K at kn + `nsub`; past the
  // last key: of what is there, masked) on the matrix cores, then the products
  // with V beside the next maximum. Each half reads the next one's operands
  // from LDS, the last one those of K for the step after (K at ka + `asub`;
  // one-step tiles read them at the step's start, behind the barrier).
  constexpr bool kCarry = KT == 64;
  vec8 k0[kM];
  auto step = [&](const uint8_t *vs, int sub, const Logits &s, const uint8_t *kn, int nsub, int jn,
                  Logits &next, const uint8_t *ka, int asub) {
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
          p[w][c][e] = (elem)x;
        }
        l[w] += sum;
        asm volatile("" : "+v"(p[w][c]));  // computed here, not after the mask's branch
      }
      // matrix and vector instructions in turn
      __builtin_amdgcn_sched_group_barrier(0x100, kM, 0);
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
      __builtin_amdgcn_sched_group_barrier(0x100, kDT, 0);
#pragma unroll
      for (int i = 0; i < R * kDT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int w = 0; w < R; ++w) top[w] = max_over_halves(x[w]) * a.scale_log2;
  };

  const int tiles = (it.c1 - it.c0 + KT - 1) / KT;
  Logits s, s2;
  if (tiles > 0) {
    next_pages(0);
    load_half(kc, koff, it.c0, pv, smem);
    load_pair(0);
    if (tiles > 1) load_pair(1);
    wait_loads_and_barrier<0>();
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
  for (int round = 0; round < tiles; round += 2) {
    if (round) wait_loads_and_barrier<0>();
    if (round + 2 < tiles) load_pair(round + 2);
    if (round + 3 < tiles) load_pair(round + 3);
    if (it.c0 + (round + 2) * KT > it.c1) {
      // What lies behind the last key may be anything, and 0 * NaN is NaN: V
      // of the round's keys from c1 on is cleared.
      const int first = it.c1 - it.c0;
      const int last = (round + 2 < tiles ? round + 2 : tiles) * KT;
      for (int u = tid; u < (last - first) * D; u += 64 * NW) {
        const int key = first + u / D, d = u % D, in = key % KT;
        reinterpret_cast<elem *>(v_stage(key / KT))[((in >> 3) * D + d) * 8 + (in & 7)] = (elem)0.f;
      }
      __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int kt = round + b, j0 = it.c0 + kt * KT;
      if (kt >= tiles) break;
      const uint8_t *vs = v_stage(kt), *kn = k_stage(kt + 1);
      if constexpr (KT == 64) {
        step(vs, 0, s, k_stage(kt), 1, j0 + 32, s2, kn, 0);
        step(vs, 1, s2, kn, 0, j0 + 64, s, kn, 1);
      } else {
        step(vs, 0, s, kn, 0, j0 + 32, s2, nullptr, 0);
#pragma unroll
        for (int w = 0; w < R; ++w) s[w] = s2[w];
      }
    }
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
attn_wide_kernel(AttnPrefix a, uint32_t item0) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  Item it;
  const uint32_t idx = item0 + spread(blockIdx.x, gridDim.x);
  rows_of_no_sequence<T, D>(a, idx, 64 * NW);
  if (find_item(a, idx, 32 * R * NW, it))
    wide_body<T, D, NW, R>(a, it, item0, smem);
}

template <class T, int D, int NW, int R>
hipError_t launch_wide(const AttnPrefix &a, int64_t item0, int64_t items, hipStream_t stream) {
  constexpr auto kern = attn_wide_kernel<T, D, NW, R>;
  const hipError_t e = ensure_max_lds<kern>(Wide<D>::kLds);
  if (e != hipSuccess) return e;
  return launch_in_pieces(items, 64 * NW, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL(kern, dim3(n), dim3(64 * NW), Wide<D>::kLds, stream, a, (uint32_t)item0 + first);
  });
}

// Workgroups of 256 rows are eight waves of 32, or four of 64 where the
// registers leave room for two such waves a SIMD. Measured (us): 768 rows x
// 32801 keys x 8 heads of 128 bf16 118 / 145; chunks of 11160 rows x 8200
// keys x 4 heads of 64 fp16 210 / 183.
template <class T, int D>
hipError_t launch_items(const AttnPrefix &a, int wide, int64_t item0, int64_t items,
                        hipStream_t stream) {
  if (items == 0) return hipSuccess;
  if (wide == 2) {
    if constexpr (D == 128) return launch_wide<T, D, 8, 1>(a, item0, items, stream);
    if constexpr (D < 128) return launch_wide<T, D, 4, 2>(a, item0, items, stream);
    return hipErrorInvalidValue;
  }
  if (wide == 1) return launch_wide<T, D, 4, 1>(a, item0, items, stream);
  return launch_in_pieces(items, kThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((attn_rows16_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a,
                       (uint32_t)item0 + first);
  });
}

// The prefix's and the suffixes' items are launched together when they are of
// one kind. (16-row items in the wide kernel's launch measured no faster: its
// LDS leaves them one workgroup a CU, and they need several to cover memory.)
template <class T, int D>
hipError_t launch(const AttnPrefix &a, hipStream_t stream) {
  hipError_t e;
  if (a.prefix_wide == a.suffix_wide || a.prefix_items == 0) {
    e = launch_items<T, D>(a, a.suffix_wide, 0, a.prefix_items + a.suffix_items, stream);
  } else {
    e = launch_items<T, D>(a, a.prefix_wide, 0, a.prefix_items, stream);
    if (e != hipSuccess) return e;
    e = launch_items<T, D>(a, a.suffix_wide, a.prefix_items, a.suffix_items, stream);
  }
  if (e != hipSuccess || a.prefix_parts + a.suffix_parts == 1) return e;
  constexpr int kRowsPerBlock = kThreads / (D / 4);
  const int64_t nrows = a.tokens * a.n_q_heads;
  return launch_in_pieces((nrows + kRowsPerBlock - 1) / kRowsPerBlock, kThreads,
                          [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a, first);
  });
}

template <class T>
hipError_t launch_dim(const AttnPrefix &a, hipStream_t stream) {
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
void attn_prefix_plan(AttnPrefix &a, int64_t max_suffix, int num_cus) {
  // Rows of a work item: 16 while reading the cache is the cost, else 128 or
  // 256 (wide 1, 2). Measured, a prefix of 16001 keys, 8 key heads, fp16 (us;
  // 16-row / 128 / 256): 128 dimensions, 32 rows 29.5 / 33.6 / 35.3, 48 rows
  // 37.3 / 34.5 / 36.2, 128 rows 81 / 38.1 / 40.5, 192 rows 148 / 45.7 / 45.2;
  // 64 dimensions, 64 rows 27.3 / 28.7 / 31.8, 128 rows 45.7 / 31.1 / 34.1.
  auto wide_for = [&](int64_t rows) {
    if (rows <= (a.head_dim == 64 ? 64 : 32)) return 0;
    return rows > 128 && a.head_dim <= 128 ? 2 : 1;
  };
  // Chunk for `keys` keys of `blocks` row blocks: as many chunks as give each
  // CU a 16-row workgroup (one workgroup's four waves keep 64 KB of a CU's
  // loads out; more chunks only add joins: 1 x 30001 keys, 8 key heads of 128
  // fp16 34 us with one workgroup a CU, 39 with two, 49 with four; 24 x 4111,
  // 32 heads 158 / 158 / 173); for the wide kernel whole rounds over the CUs.
  auto chunk_of = [&](int64_t keys, int64_t blocks, int wide) {
    const int64_t most = (keys + 127) / 128;
    int64_t parts = (num_cus + blocks - 1) / blocks;
    if (wide) {
      int64_t best = -1;
      for (int64_t p = 1; p <= most && p <= 64; ++p) {
        const int64_t chunk = ((keys + p - 1) / p + 127) / 128 * 128;
        // a workgroup's fixed cost is about that of 256 keys
        const int64_t cost = (blocks * p + num_cus - 1) / num_cus * (chunk + 256);
        if (best < 0 || cost < best) {
          best = cost;
          parts = p;
        }
      }
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
  a.prefix_wide = wide_for(prefix_rows);
  a.suffix_wide = wide_for(suffix_rows);
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

size_t attn_prefix_workspace(const AttnPrefix &a) {
  const int64_t parts = a.prefix_parts + a.suffix_parts;
  if (parts <= 1) return 0;
  const int64_t rows = a.tokens * a.n_q_heads;
  return (size_t)(parts * rows) * ((size_t)a.head_dim * 4 + 8);
}

hipError_t attn_prefix_launch(AttnPrefix &a, void *ws, ElemType type, hipStream_t stream) {
  if (a.prefix_items + a.suffix_items > 0x7fffffff) return hipErrorInvalidValue;
  const int64_t rows = a.tokens * a.n_q_heads;
  a.part_o = static_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(static_cast<float *>(ws) +
                                         (a.prefix_parts + a.suffix_parts) * rows * a.head_dim);
  return type == ElemType::F16 ? launch_dim<TypeF16>(a, stream) : launch_dim<TypeBF16>(a, stream);
}

}  // namespace lqmm
