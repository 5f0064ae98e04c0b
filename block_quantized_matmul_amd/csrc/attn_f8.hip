// Attention over the 8-bit paged cache: attn_prefix.hip's problem with keys and
// values held as e4m3 codes and a power of two for each token and head.
//
// Mathematics. With z_j = scale * log2(e) * q.k_j and V's values code_j 2^(e_j),
//   O = sum_j 2^(z_j) 2^(e_j) code_j / sum_j 2^(z_j).
// The exponents go to the logits: with y_j = z_j + e_j, any reference m and
// w_j = 2^(y_j - m),
//   O = sum_j w_j code_j / sum_j w_j 2^(-e_j).
// m is kept near the largest y: the weights, which the matrix cores take in 16
// bits, then lose nothing by scales that differ from token to token, and V's
// codes are operands as they are. The scale of V costs no instruction at the
// logits (the multiplication with scale * log2(e) becomes a multiply-add) and
// none at the sum (an addition becomes one). K's scale costs none either: the
// conversion of a lane's codes, all of one token, to 16 bits applies it.
// A partial result is (m, sum w 2^-e, sum w code), joined as in attn_prefix.hip.
//
// Weights are held at 2^14 in fp16, as there; in bf16 at 1 (codes are at most
// 448, so that no sum of a work item's 2^13 keys comes near the largest value).
#include "attn_common.hpp"
#include "f8_cache.hpp"

namespace lqmm {
namespace {

// log2 of what weights are held at, times their value
template <class T>
constexpr float kShift = __is_same(T, TypeF16) ? 14.0f : 0.0f;
constexpr float kAloneShift = 0.0f;  // of rows done by themselves, in fp32

// First token vector of the group of eight that holds key j (in vectors of D
// codes, of which each has one scale).
__device__ __forceinline__ int64_t vector_at(const AttnPrefix &a, const Item &it, int j) {
  const int32_t p = it.pages[j >> a.page_log2];
  const int64_t page = (uint32_t)p < (uint32_t)a.num_pages ? p : 0;
  return ((page * a.n_kv_heads + it.h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
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
      const float ks = scale_of(a.k_scales[vec]);
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
      const float w = __shfl(e, i) * scale_of(a.v_scales[vec]);
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
      const float f = scale_of(st.ks[u]);
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
    float y[2][4], back[2][4];  // logits with V's exponents; 2^-exponent
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int b = (int)(vs[u] >> 8 * r & 255u);
        y[u][r] = fmaf(s[u][r], a.scale_log2, (float)(b - 127));
        back[u][r] = scale_inverse(b);
      }
    const int seen = limit < it.c1 ? limit : it.c1;
    if (j0 + kStep > it.c1 || j0 + kStep > all_see) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j0 + 8 * g + 4 * u + r >= seen) {
            y[u][r] = -INFINITY;
            back[u][r] = 0.f;  // (its byte may be anything)
          }
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
        l = fmaf(e, back[u][r], l);
        p[4 * u + r] = (elem)e;
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
__global__ void __launch_bounds__(kThreads)
attn_f8_rows16_kernel(AttnPrefixF8 a, uint32_t item0) {
  __shared__ Rows16<D, kThreads / 64> sm;
  Item it;
  const uint32_t idx = item0 + spread(blockIdx.x, gridDim.x);
  rows_of_no_sequence<T, D>(a, idx, kThreads);
  if (find_item(a, idx, kRows, it))
    rows16_body<T, D, kThreads / 64>(a, it, sm);
}

template <class T, int D>
hipError_t launch(const AttnPrefixF8 &a, hipStream_t stream) {
  hipError_t e = launch_in_pieces(a.prefix_items + a.suffix_items, kThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((attn_f8_rows16_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a, first);
  });
  if (e != hipSuccess || a.prefix_parts + a.suffix_parts == 1) return e;
  constexpr int kRowsPerBlock = kThreads / (D / 4);
  const int64_t nrows = a.tokens * a.n_q_heads;
  return launch_in_pieces((nrows + kRowsPerBlock - 1) / kRowsPerBlock, kThreads,
                          [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a, first);
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
  auto chunk_of = [&](int64_t keys, int64_t blocks) {
    const int64_t most = (keys + 127) / 128;
    int64_t parts = (num_cus + blocks - 1) / blocks;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    int64_t chunk = ((keys + parts - 1) / parts + 127) / 128 * 128;
    if (chunk > kAttnMaxChunk) chunk = kAttnMaxChunk;
    return (int)chunk;
  };
  a.group = a.n_q_heads / a.n_kv_heads;
  const int64_t prefix_rows = a.tokens * a.group, suffix_rows = a.max_q * a.group;
  a.prefix_wide = a.suffix_wide = 0;
  a.prefix_row_blocks = (int)((prefix_rows + kRows - 1) / kRows);
  a.prefix_chunk = a.prefix_parts = 0;
  if (a.prefix_len > 0) {
    a.prefix_chunk = chunk_of(a.prefix_len, (int64_t)a.prefix_row_blocks * a.n_kv_heads);
    a.prefix_parts = (int)((a.prefix_len + a.prefix_chunk - 1) / a.prefix_chunk);
  }
  a.prefix_items = (int64_t)a.prefix_row_blocks * a.n_kv_heads * a.prefix_parts;
  a.suffix_row_blocks = (int)((suffix_rows + kRows - 1) / kRows);
  a.suffix_chunk = chunk_of(max_suffix, a.batch * a.n_kv_heads * a.suffix_row_blocks);
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
