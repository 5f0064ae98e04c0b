// The 8-bit paged cache back to dense rows: sequence b's token j becomes row
// starts[b] + j of k_out and v_out, its codes times the power of two of its
// scale, rounded once to the output's type (exact in fp32 and bf16).
//
// Layout. A workgroup takes the eight tokens of one group of a sequence's page
// and some of its heads: a lane brings 16 codes of one token's K, or the eight
// tokens of two dimensions of V (16 bytes each), and writes V with a word per
// token, lanes side by side. How many groups a sequence has is known on the
// device only: the groups of sequence b are numbered from starts[b] / 8 + b on,
// which leaves room for each, and a workgroup finds its sequence by a search over
// starts, 64 at a time.
//
// Bound by memory, mostly by what is written: 24 ragged sequences of up to 8209
// tokens, 8 heads of 128, to bf16 129 us, which is the rate of a large copy (124).
// 611 tokens 3.5 us: launch and three round trips, starts, page and codes.
#include "f8_cache.hpp"
#include "lqmm_internal.hpp"

namespace lqmm {
namespace {

constexpr int kThreads = 256;
constexpr int kClear = 64;  // workgroups for the rows of no sequence

__device__ __forceinline__ int64_t bounded(int64_t v, int64_t most) {
  return v < 0 ? 0 : v < most ? v : most;
}

// The last b of [0, n) whose number of a first group is at most i (0 if none).
__device__ __forceinline__ int64_t find_sequence(const int32_t *starts, int64_t n, int64_t tokens, int64_t i) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, len = n;
  while (len > 1) {
    const int64_t step = (len + 63) / 64, at = lo + lane * step;
    const bool before = lane * step < len && bounded(starts[at < n ? at : n - 1], tokens) / 8 + at <= i;
    const int k = __builtin_popcountll(__ballot(before));
    const int64_t skip = (k > 0 ? k - 1 : 0) * step;
    lo += skip;
    len = len - skip < step ? len - skip : step;
    if (step == 1) break;
  }
  return lo;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads)
kv_read_f8_kernel(KvRead a, uint32_t first, int64_t groups, int head_blocks) {
  typedef typename T::elem elem;
  constexpr int kUnits = D / 2;                 // of 16 bytes, in a group's K, and in its V
  constexpr int kHeads = kThreads / kUnits;     // heads of a workgroup
  const int tid = threadIdx.x;
  const int64_t block = first + (int64_t)blockIdx.x;
  elem *ko = static_cast<elem *>(a.k_out), *vo = static_cast<elem *>(a.v_out);
  const int64_t row = (int64_t)a.n_kv_heads * D;  // elements of an output row
  if (block >= groups * head_blocks) {
    // Rows of no sequence are zeros.
    const int64_t before = bounded(a.starts[0], a.tokens), after = bounded(a.starts[a.batch], a.tokens);
    const int64_t n = (before + a.tokens - (after > before ? after : before)) * row / 8;
    const float zero[8] = {};
    for (int64_t u = (block - groups * head_blocks) * kThreads + tid; u < n; u += kClear * kThreads) {
      int64_t at = 8 * u;
      if (at >= before * row) at += ((after > before ? after : before) - before) * row;
      if constexpr (T::kBytes == 4) {
        *reinterpret_cast<float4_t *>(ko + at) = *reinterpret_cast<float4_t *>(ko + at + 4) = float4_t{};
        *reinterpret_cast<float4_t *>(vo + at) = *reinterpret_cast<float4_t *>(vo + at + 4) = float4_t{};
      } else {
        store8<T>(ko + at, zero);
        store8<T>(vo + at, zero);
      }
    }
    return;
  }
  const int64_t i = block / head_blocks;
  const int64_t b = find_sequence(a.starts, a.batch, a.tokens, i);
  const int64_t r0 = bounded(a.starts[b], a.tokens), r1 = bounded(a.starts[b + 1], a.tokens);
  const int64_t j0 = 8 * (i - (r0 / 8 + b));  // first token of the group
  const int64_t n = r1 - r0;
  if (j0 < 0 || j0 >= n) return;
  const int u = tid % kUnits, h = (int)(block % head_blocks) * kHeads + tid / kUnits;
  if (tid / kUnits >= kHeads || h >= a.n_kv_heads) return;
  // tokens past the page table are zeros, a page outside the cache is page 0
  const bool in_table = (j0 >> a.page_log2) < a.max_pages;
  const int32_t p = in_table ? a.pages[b * a.max_pages + (j0 >> a.page_log2)] : 0;
  const int64_t page = (uint32_t)p < (uint32_t)a.num_pages ? p : 0;
  const int64_t vec = ((page * a.n_kv_heads + h) << a.page_log2) + (j0 & ((1 << a.page_log2) - 1));
  const int count = (int)(n - j0 < 8 ? n - j0 : 8);
  const int64_t out = (r0 + j0) * row + (int64_t)h * D;
  u32x4 kc = {0u, 0u, 0u, 0u}, vc = kc;
  u32x2 vs = {0u, 0u};
  uint32_t ks = 0;
  const int tk = u / (D / 16), ck = u % (D / 16);  // this lane's token and 16 elements of K
  if (in_table) {
    kc = *reinterpret_cast<const u32x4 *>(a.k_cache + vec * D + 16 * u);
    vc = *reinterpret_cast<const u32x4 *>(a.v_cache + vec * D + 16 * u);
    ks = a.k_scales[vec + tk];
    vs = *reinterpret_cast<const u32x2 *>(a.v_scales + vec);
  }
  if (tk < count) {
    float x[8], y[8];
    values8(u32x2{kc[0], kc[1]}, scale_of(ks), x);
    values8(u32x2{kc[2], kc[3]}, scale_of(ks), y);
    elem *dst = ko + out + tk * row + 16 * ck;
    if constexpr (T::kBytes == 4) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4_t *>(dst + e) = float4_t{x[e], x[e + 1], x[e + 2], x[e + 3]};
        *reinterpret_cast<float4_t *>(dst + 8 + e) = float4_t{y[e], y[e + 1], y[e + 2], y[e + 3]};
      }
    } else {
      store8<T>(dst, x);
      store8<T>(dst + 8, y);
    }
  }
  float x[8], y[8];  // dimensions 2 u and 2 u + 1 of the eight tokens
  values8(u32x2{vc[0], vc[1]}, 1.0f, x);
  values8(u32x2{vc[2], vc[3]}, 1.0f, y);
  typedef elem pair __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t >= count) break;
    const float s = scale_of(vs[t >> 2] >> 8 * (t & 3) & 255u);
    *reinterpret_cast<pair *>(vo + out + t * row + 2 * u) = pair{(elem)(x[t] * s), (elem)(y[t] * s)};
  }
}

template <class T, int D>
hipError_t launch(const KvRead &a, hipStream_t stream) {
  constexpr int kHeads = kThreads / (D / 2);
  const int head_blocks = (a.n_kv_heads + kHeads - 1) / kHeads;
  const int64_t groups = a.tokens / 8 + a.batch;
  return launch_in_pieces(groups * head_blocks + kClear, kThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((kv_read_f8_kernel<T, D>), dim3(n), dim3(kThreads), 0, stream, a, first, groups,
                       head_blocks);
  });
}

template <class T>
hipError_t launch_dim(const KvRead &a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch<T, 64>(a, stream);
    case 96: return launch<T, 96>(a, stream);
    case 128: return launch<T, 128>(a, stream);
    case 256: return launch<T, 256>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t kv_read_f8_launch(const KvRead &a, ElemType type, hipStream_t stream) {
  if ((a.tokens / 8 + a.batch) * a.n_kv_heads > 0x7fffffff) return hipErrorInvalidValue;
  if (type == ElemType::F32) return launch_dim<TypeF32>(a, stream);
  if (type == ElemType::F16) return launch_dim<TypeF16>(a, stream);
  return launch_dim<TypeBF16>(a, stream);
}

}  // namespace lqmm
