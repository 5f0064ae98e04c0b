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
// P is rounded to the cache's 16-bit type, as the matrix cores want it; in
// fp16 it is kept at 2^kShift times its value, so that weights down to
// 2^-(24 + kShift) of the largest do not vanish. Logits, maxima, sums and O
// are fp32.
//
// Two kernels. Few rows (one new token's heads) are bound by reading the
// cache: 16 rows a workgroup, the waves take different keys, straight from
// memory to the operands. Many rows (a prefix under a batch, a chunk of new
// tokens) are bound by the matrix cores: 32 rows a wave, all waves of a
// workgroup take the same keys from LDS tiles that are filled ahead.
#include "lqmm_internal.hpp"
#include "serve_device.hpp"

namespace lqmm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;          // rows of a work item
constexpr int kStep = 32;          // keys of one step of a wave
constexpr float kShift = 14.0f;    // weights are held as 2^14 times their value
constexpr int kMaxIds = kAttnMaxChunk / 8 + 8;

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
    if (q1 - q0 > a.max_q) q1 = q0 + a.max_q;
  }
  const int n = (int)(q1 - q0);
  it.part = a.prefix_parts + chunk;
  it.tok0 = q0;
  it.rows = n * G;
  it.row0 = rb * rows_per_block;
  if (it.row0 >= it.rows) return false;
  it.past = (int)len - n + 1;
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

// Workgroups are handed to the 8 XCDs in turn, and each has its own L2:
// renumbered so that consecutive items, which share keys, run on one XCD.
__device__ __forceinline__ uint32_t spread(uint32_t block, uint32_t n) {
  const uint32_t x = block % 8, q = n / 8, r = n % 8;
  return x * q + (x < r ? x : r) + block / 8;
}

// ---- few rows -------------------------------------------------------------------
template <class T, int D>
__global__ void __launch_bounds__(kThreads)
attn_rows16_kernel(AttnPrefix a, uint32_t item0) {
  typedef typename T::elem elem;
  typedef typename T::vec8 vec8;
  constexpr int kQ = D / 32;                       // k-steps of one logit tile
  constexpr int kDT = D / 16;                      // 16-wide tiles of O
  constexpr int kPass = kDT < 8 ? kDT : 8;         // O tiles joined at a time
  constexpr int kLd = 16 * kPass + 4;
  static_assert(kDT % kPass == 0, "whole passes");
  __shared__ int ids[kMaxIds];
  __shared__ float wave_m[4][kRows], wave_l[4][kRows];
  __shared__ __attribute__((aligned(16))) float join[4][kRows][kLd];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m16 = lane & 15, g = lane >> 4;
  Item it;
  if (!find_item(a, item0 + spread(blockIdx.x, gridDim.x), kRows, it)) return;
  const int G = a.group;
  const int lg = a.page_log2, pmask = (1 << lg) - 1;
  const bool direct = a.prefix_parts + a.suffix_parts == 1;

  // page numbers of the chunk, bounded to the cache
  const int page0 = it.c0 >> lg;
  if (it.c1 > it.c0) {
    const int n = ((it.c1 - 1) >> lg) - page0 + 1;
    for (int i = tid; i < n; i += kThreads) {
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
  for (; j0 < it.c1; j0 += 4 * kStep) {
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
    if (j0 + 4 * kStep < it.c1) load_k(j0 + 4 * kStep);
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
    const float ref = (mn == -INFINITY ? 0.f : mn) - kShift;
    const float corr = __builtin_amdgcn_exp2f(m - mn);  // NaN only while m = mn = -inf
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

  // Join the four waves' results.
  l = sum_over_rows(l);
  if (g == 0) {
    wave_m[wave][m16] = m;
    wave_l[wave][m16] = l;
  }
  __syncthreads();
  float mj = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) mj = fmaxf(mj, wave_m[w][m16]);
  const float mine = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mj);
  const int out_row = tid >> 4, out_d = 8 * (tid & 15);
  // the row that this thread writes
  float lj = 0.f, mo = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) mo = fmaxf(mo, wave_m[w][out_row]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float mw = wave_m[w][out_row];
    lj += mw == -INFINITY ? 0.f : wave_l[w][out_row] * __builtin_amdgcn_exp2f(mw - mo);
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
      *reinterpret_cast<float4_t *>(&join[wave][m16][16 * i + 4 * g]) = x;
    }
    __syncthreads();
    if (owrite && out_d < 16 * kPass) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = (join[0][out_row][out_d + e] + join[1][out_row][out_d + e]) +
               (join[2][out_row][out_d + e] + join[3][out_row][out_d + e]);
      const int64_t d0 = pass * 16 * kPass + out_d;
      if (direct) {
        const float inv = lj == 0.f ? 0.f : 1.0f / lj;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
        store8<T>(static_cast<elem *>(a.out) + flat * D + d0, x);
      } else {
        float *dst = a.part_o + (it.part * nrows + flat) * D + d0;
        *reinterpret_cast<float4_t *>(dst) = float4_t{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<float4_t *>(dst + 4) = float4_t{x[4], x[5], x[6], x[7]};
      }
    }
  }
  if (owrite && out_d == 0) {
    if (direct) {
      if (a.lse) a.lse[flat] = lj == 0.f ? -INFINITY : (mo - kShift + __log2f(lj)) * 0.6931471805599453f;
    } else {
      a.part_ml[it.part * nrows + flat] = make_float2(mo - kShift, lj);
    }
  }
}

// ---- many rows -----------------------------------------------------------------
// A running maximum that grows by no more than kSlack (log2) is left where it
// is: O is rescaled when a row needs it, not at every step.
constexpr float kSlack = 8.0f;
constexpr float kWideShift = 6.0f;  // weights are at most 2^(kSlack + kWideShift), in fp16's range

template <int D>
struct Wide {
  static constexpr int kKeys = D <= 128 ? 64 : 32;  // keys of a tile
  static constexpr int kHalf = kKeys * D * 2;       // bytes of a tile's K (and V)
  static constexpr int kStages = 3;
  static constexpr int kLds = kStages * 2 * kHalf + kMaxIds * 4;
};

template <class T, int D, int NW>
__global__ void __launch_bounds__(64 * NW, D <= 128 ? 2 : 1)
attn_wide_kernel(AttnPrefix a, uint32_t item0) {
  typedef typename T::elem elem;
  typedef typename T::vec8 vec8;
  typedef Wide<D> C;
  constexpr int KT = C::kKeys;
  constexpr int kQ = D / 16;                 // k-steps of a logit tile
  constexpr int kDT = D / 32;                // 32-wide tiles of O
  constexpr int kSub = KT / 32;
  constexpr int kLoads = C::kHalf / 1024 / NW;  // 1 KB loads of a wave for K, and for V
  static_assert(C::kHalf % (1024 * NW) == 0, "whole loads");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int *ids = reinterpret_cast<int *>(smem + C::kStages * 2 * C::kHalf);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  Item it;
  if (!find_item(a, item0 + spread(blockIdx.x, gridDim.x), 32 * NW, it)) return;
  const int G = a.group;
  const int lg = a.page_log2, pmask = (1 << lg) - 1;
  const bool direct = a.prefix_parts + a.suffix_parts == 1;

  const int page0 = it.c0 >> lg;
  if (it.c1 > it.c0) {
    const int n = ((it.c1 - 1) >> lg) - page0 + 1;
    for (int i = tid; i < n; i += 64 * NW) {
      const int32_t p = it.pages[page0 + i];
      ids[i] = (uint32_t)p < (uint32_t)a.num_pages ? p : 0;
    }
  }
  const int row0 = it.row0 + 32 * wave;  // this wave's rows
  const int row = row0 + l32;
  const bool live = row < it.rows;
  const int tok = live ? row / G : 0;
  const int64_t t = it.tok0 + tok;
  const int hq = it.h * G + (live ? row % G : 0);
  const int limit = it.past + it.per_token * tok;
  const int all_see = it.past + it.per_token * (row0 < it.rows ? row0 / G : 0);
  vec8 q[kQ];
  {
    const elem *src = static_cast<const elem *>(a.q) + t * a.ldq + (int64_t)hq * D + 8 * h;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4 *>(src + 16 * i);
      q[i] = __builtin_bit_cast(vec8, x ^ a.q_sign);
    }
  }
  __syncthreads();

  // Tile rows of K in LDS are in the order of the logit tile's rows (row m of
  // 32: key 16 (m / 16) + 8 (m / 4 % 2) + 4 (m / 8 % 2) + m % 4), with their
  // 16-byte chunks exchanged per row, so that the eight rows of one read
  // phase lie in different banks. V is as in memory.
  const elem *kc = static_cast<const elem *>(a.k_cache);
  const elem *vc = static_cast<const elem *>(a.v_cache);
  const int64_t head_elems = (int64_t)D << lg;
  const int last_group = (it.c1 - 1) & ~7;
  auto group_at = [&](int j) -> int64_t {
    j = j < last_group ? j : last_group;
    const int64_t page = ids[(j >> lg) - page0];
    return (page * a.n_kv_heads + it.h) * head_elems + (int64_t)(j & pmask) * D;
  };
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  constexpr int kSwz = D == 96 ? 3 : 7;
  auto issue = [&](int j0, int stage) {
    uint8_t *ks = smem + stage * 2 * C::kHalf, *vs = ks + C::kHalf;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int u = (wave * kLoads + i) * 64 + lane;  // 16-byte unit of the tile
      const int r = u / kChunks, c = (u % kChunks) ^ (r & kSwz);
      const int key = (r & ~15) + 8 * (r >> 2 & 1) + 4 * (r >> 3 & 1) + (r & 3);
      load_to_lds<16>(kc + group_at(j0 + (key & ~7)) + (key & 7) * D + 8 * c,
                  ks + (wave * kLoads + i) * 1024);
      load_to_lds<16>(vc + group_at(j0 + 8 * (u / D)) + (u % D) * 8, vs + (wave * kLoads + i) * 1024);
    }
  };

  float16_t o[kDT];
#pragma unroll
  for (int i = 0; i < kDT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
  float m = -INFINITY, l = 0.f;
  float ref = 0.f;  // m - kWideShift, finite

  const int tiles = (it.c1 - it.c0 + KT - 1) / KT;
  if (tiles > 0) issue(it.c0, 0);
  if (tiles > 1) issue(it.c0 + KT, 1);
  for (int kt = 0; kt < tiles; ++kt) {
    const int j0 = it.c0 + kt * KT;
    if (kt + 1 < tiles)
      wait_loads_and_barrier<2 * kLoads>();
    else
      wait_loads_and_barrier<0>();
    if (kt + 2 < tiles) issue(j0 + 2 * KT, (kt + 2) % 3);
    uint8_t *ks = smem + (kt % 3) * 2 * C::kHalf, *vs = ks + C::kHalf;
    if (j0 + KT > it.c1) {
      // what lies behind the last key may be anything, and 0 * NaN is NaN
      const int valid = it.c1 - j0;
      elem *ve = reinterpret_cast<elem *>(vs);
      for (int u = tid; u < (KT - valid) * D; u += 64 * NW) {
        const int key = valid + u / D, d = u % D;
        ve[((key >> 3) * D + d) * 8 + (key & 7)] = (elem)0.f;
      }
      __syncthreads();
    }

    float16_t s[kSub];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[u][r] = 0.f;
      const int r = 32 * u + l32;
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const vec8 kf = *reinterpret_cast<const vec8 *>(ks + r * (2 * D) + 16 * ((2 * i + h) ^ (r & kSwz)));
        s[u] = T::mfma32(kf, q[i], s[u]);
      }
    }
    if (j0 + KT > it.c1 || j0 + KT > all_see) {
      const int seen = limit < it.c1 ? limit : it.c1;
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (j0 + 32 * u + 16 * (r >> 3) + 8 * h + (r & 7) >= seen) s[u][r] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
    top = max_over_halves(top) * a.scale_log2;
    if (__any(top > m + kSlack)) {
      const float mn = fmaxf(m, top);
      const float c = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      ref = (mn == -INFINITY ? 0.f : mn) - kWideShift;
      l *= c;
#pragma unroll
      for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= c;
    }
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        vec8 p;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __builtin_amdgcn_exp2f(fmaf(s[u][8 * w + e], a.scale_log2, -ref));
          l += x;
          p[e] = (elem)x;
        }
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
          const vec8 vf = *reinterpret_cast<const vec8 *>(
              vs + ((4 * u + 2 * w + h) * D + 32 * i + l32) * 16);
          o[i] = T::mfma32(vf, p, o[i]);
        }
      }
  }

  l = sum_over_halves(l);
  if (!live) return;
  const int64_t flat = t * a.n_q_heads + hq;
  const int64_t nrows = a.tokens * a.n_q_heads;
  if (direct) {
    typedef elem vec4 __attribute__((ext_vector_type(4)));
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    elem *dst = static_cast<elem *>(a.out) + flat * D + 4 * h;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<vec4 *>(dst + 32 * i + 2 * r) =
            vec4{(elem)(o[i][r] * inv), (elem)(o[i][r + 1] * inv), (elem)(o[i][r + 2] * inv),
                 (elem)(o[i][r + 3] * inv)};
  } else {
    float *dst = a.part_o + (it.part * nrows + flat) * D + 4 * h;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4_t *>(dst + 32 * i + 2 * r) =
            float4_t{o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]};
  }
  if (h == 0) {
    if (direct) {
      if (a.lse) a.lse[flat] = l == 0.f ? -INFINITY : (m - kWideShift + __log2f(l)) * 0.6931471805599453f;
    } else {
      a.part_ml[it.part * nrows + flat] = make_float2(m - kWideShift, l);
    }
  }
}

// Joins the partial results of each row: D / 4 threads a row, four
// dimensions each.
template <class T, int D>
__global__ void __launch_bounds__(kThreads)
attn_join_kernel(AttnPrefix a) {
  typedef typename T::elem elem;
  constexpr int kPer = D / 4;
  constexpr int kRowsPerBlock = kThreads / kPer;
  const int64_t nrows = a.tokens * a.n_q_heads;
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / kPer;
  const int d = 4 * (threadIdx.x % kPer);
  if (threadIdx.x / kPer >= kRowsPerBlock || row >= nrows) return;
  const int parts = a.prefix_parts + a.suffix_parts;
  float m = -INFINITY;
  for (int p = 0; p < parts; ++p) m = fmaxf(m, a.part_ml[p * nrows + row].x);
  float l = 0.f;
  float4_t o = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; ++p) {
    const float2 ml = a.part_ml[p * nrows + row];
    if (ml.x == -INFINITY) continue;  // no key of this part is seen
    const float w = __builtin_amdgcn_exp2f(ml.x - m);
    const float4_t x = *reinterpret_cast<const float4_t *>(a.part_o + (p * nrows + row) * D + d);
    l += w * ml.y;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] += w * x[r];
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  elem *dst = static_cast<elem *>(a.out) + row * D + d;
#pragma unroll
  for (int r = 0; r < 4; ++r) dst[r] = (elem)(o[r] * inv);
  if (a.lse && d == 0)
    a.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

template <class T, int D, int NW>
hipError_t launch_wide(const AttnPrefix &a, int64_t item0, int64_t items, hipStream_t stream) {
  constexpr auto kern = attn_wide_kernel<T, D, NW>;
  const hipError_t e = ensure_max_lds<kern>(Wide<D>::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)items), dim3(64 * NW), Wide<D>::kLds, stream, a, (uint32_t)item0);
  return hipGetLastError();
}

template <class T, int D>
hipError_t launch_items(const AttnPrefix &a, int wide, int64_t item0, int64_t items,
                        hipStream_t stream) {
  if (items == 0) return hipSuccess;
  if (wide == 8) return launch_wide<T, D, D == 64 || D == 128 ? 8 : 4>(a, item0, items, stream);
  if (wide == 4) return launch_wide<T, D, 4>(a, item0, items, stream);
  hipLaunchKernelGGL((attn_rows16_kernel<T, D>), dim3((unsigned)items), dim3(kThreads), 0, stream, a,
                     (uint32_t)item0);
  return hipGetLastError();
}

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
  hipLaunchKernelGGL((attn_join_kernel<T, D>),
                     dim3((unsigned)((nrows + kRowsPerBlock - 1) / kRowsPerBlock)), dim3(kThreads),
                     0, stream, a);
  return hipGetLastError();
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
  // Waves of the wide kernel for `rows` rows, 0 for the 16-row kernel.
  auto wide_for = [&](int64_t rows) {
    if (rows <= 32) return 0;
    return rows > 128 && (a.head_dim == 64 || a.head_dim == 128) ? 8 : 4;
  };
  // Chunk for `keys` keys of `blocks` row blocks. The 16-row kernel runs
  // several workgroups on a CU; the wide one runs one, so its number of
  // chunks is chosen for whole rounds of the CUs.
  auto chunk_of = [&](int64_t keys, int64_t blocks, int wide) {
    const int64_t most = (keys + 127) / 128;
    int64_t parts = (4 * (int64_t)num_cus + blocks - 1) / blocks;
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
  auto block_rows = [](int wide) { return wide ? 32 * wide : kRows; };
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
