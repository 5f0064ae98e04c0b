// Appending keys and values to a paged cache, with the position rotation
// applied on the way.
//
// Mathematics. A rotated head vector has R/2 pairs (x0, x1); pair i of a
// token at position p turns by the angle p * inv_freq[i]:
//   x0' = x0 cos - x1 sin,  x1' = x1 cos + x0 sin.
// The table holds inv_freq[i] / 2 pi as a 64-bit fraction of a turn, so
// p * turns[i] mod 2^64 is the angle with its whole turns dropped, exact to
// p * 2^-65 turns: no position is too large for the 32-bit sine that follows
// (p * inv_freq in fp32 is off by 6e-3 at p = 1e5). Products and sums are
// fp32; each output is rounded once, to the cache's type.
//
// Layout. K pages are [heads][page][D]. V pages are [heads][page / 8][D][8]:
// the eight tokens of a group stand next to each other, which is the order a
// matrix-core operand of P V wants, so that the attention kernels load it
// with one 16-byte load per lane and no transposition. A token's V row is
// then D elements 16 bytes apart: single tokens are stored element by
// element, and eight consecutive tokens that fill a group are stored as
// 16-byte vectors.
//
// Both kinds of work run in one launch: workgroups [0, rot_blocks) rotate q
// and K, the others store V.
#include "lqmm_internal.hpp"
#include "serve_device.hpp"

namespace lqmm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // head_dim <= 256

template <class TI, class TC, bool INTER>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(KvAppend a, uint32_t first) {
  typedef typename TI::elem in_t;
  typedef typename TC::elem cache_t;
  const int tid = threadIdx.x;
  const uint32_t block = first + blockIdx.x;
  const int D = a.head_dim;
  const int64_t nslots = a.num_pages << a.page_log2;
  const int64_t head_elems = (int64_t)D << a.page_log2;  // one head of one page

  if ((int)block < a.rot_blocks) {
    // One token and up to heads_per_block of its q and K heads.
    __shared__ float cs[2][kMaxPairs];
    const int64_t t = block / a.head_blocks;
    const int h0 = (int)(block % a.head_blocks) * a.heads_per_block;
    const int pairs = a.rot_dim / 2;
    if (pairs) {
      const uint64_t pos = (uint64_t)(int64_t)a.positions[t];
      for (int i = tid; i < pairs; i += kThreads) {
        const int32_t turn = (int32_t)((pos * a.turns[i]) >> 32);  // of 2^32, signed
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        cs[0][i] = c;
        cs[1][i] = s;
      }
      __syncthreads();
    }
    const int64_t slot = a.slots[t];
    const bool kept = slot >= 0 && slot < nslots;
    // A work item is 16 elements of a head: 8 pairs, or 16 unrotated ones.
    const int items = D / 16, rot_items = a.rot_dim / 16;
    const int nh = a.n_q_heads + a.n_kv_heads;
    const int hn = h0 + a.heads_per_block < nh ? a.heads_per_block : nh - h0;
    for (int w = tid; w < hn * items; w += kThreads) {
      const int h = h0 + w / items, c = w % items;
      const bool is_k = h >= a.n_q_heads;
      if (is_k && !kept) continue;
      const in_t *src;
      cache_t *dst;
      if (is_k) {
        const int hk = h - a.n_q_heads;
        src = static_cast<const in_t *>(a.k) + t * a.ldk + (int64_t)hk * D;
        dst = static_cast<cache_t *>(a.k_cache) +
              ((slot >> a.page_log2) * a.n_kv_heads + hk) * head_elems +
              (slot & ((1 << a.page_log2) - 1)) * D;
      } else {
        src = static_cast<const in_t *>(a.q) + t * a.ldq + (int64_t)h * D;
        dst = static_cast<cache_t *>(a.q_out) + (t * a.n_q_heads + h) * D;
      }
      float x[8], y[8];
      if (c < rot_items) {
        const int p0 = 8 * c;  // first pair
        const int e0 = INTER ? 2 * p0 : p0, e1 = INTER ? e0 + 8 : p0 + pairs;
        load8<TI>(src + e0, x);
        load8<TI>(src + e1, y);
        float u[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // pair i: (x0, x1) and where its two results go
          const float x0 = INTER ? (i < 4 ? x[(2 * i) & 7] : y[(2 * i) & 7]) : x[i];
          const float x1 = INTER ? (i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7]) : y[i];
          const float cc = cs[0][p0 + i], ss = cs[1][p0 + i];
          u[i] = x0 * cc - x1 * ss;
          v[i] = x1 * cc + x0 * ss;
        }
        if constexpr (INTER) {
          const float lo[8] = {u[0], v[0], u[1], v[1], u[2], v[2], u[3], v[3]};
          const float hi[8] = {u[4], v[4], u[5], v[5], u[6], v[6], u[7], v[7]};
          store8<TC>(dst + e0, lo);
          store8<TC>(dst + e1, hi);
        } else {
          store8<TC>(dst + e0, u);
          store8<TC>(dst + e1, v);
        }
      } else {
        load8<TI>(src + 16 * c, x);
        load8<TI>(src + 16 * c + 8, y);
        store8<TC>(dst + 16 * c, x);
        store8<TC>(dst + 16 * c + 8, y);
      }
    }
    return;
  }

  // V of tokens t0 .. t0 + 7 and some of the heads. A token whose slot starts a group, followed by
  // seven tokens with the next seven slots, leads a whole group, which is
  // stored as vectors (it may reach into the next workgroup's tokens); a
  // token inside such a group is skipped; any other is stored by itself.
  __shared__ int64_t slot[24];
  __shared__ int lead[16];
  const int64_t t0 = (int64_t)((block - a.rot_blocks) / a.v_blocks) * 8;
  if (tid < 22) {
    const int64_t t = t0 - 7 + tid;
    int64_t s = -1;
    if (t >= 0 && t < a.tokens) {
      s = a.slots[t];
      if (s >= nslots) s = -1;
    }
    slot[tid] = s;
  }
  __syncthreads();
  if (tid < 15) {
    const int64_t s = slot[tid];
    bool l = s >= 0 && (s & 7) == 0;
    for (int i = 1; i < 8; ++i) l = l && slot[tid + i] == s + i;
    lead[tid] = l;
  }
  __syncthreads();
  // Two elements of one head per thread; the eight tokens' loads go out
  // together (a workgroup of scattered tokens waits for memory once).
  const int half = D / 2;
  const int h = (int)((block - a.rot_blocks) % a.v_blocks) * (kThreads / half) + tid / half;
  const int d = 2 * (tid % half);
  if (tid / half >= kThreads / half || h >= a.n_kv_heads) return;
  const in_t *src = static_cast<const in_t *>(a.v) + t0 * a.ldv + (int64_t)h * D + d;
  cache_t *vc = static_cast<cache_t *>(a.v_cache) + h * head_elems + 8 * d;
  auto group_of = [&](int64_t s) {
    return vc + (s >> a.page_log2) * a.n_kv_heads * head_elems +
           ((s & ((1 << a.page_log2) - 1)) >> 3) * 8 * D;
  };
  float x[8], y[8];
  bool single[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t s = slot[7 + i];
    const int before = (int)(s & 7);
    single[i] = s >= 0 && !lead[7 + i - before];
    if (single[i]) {
      x[i] = (float)src[i * a.ldv];
      y[i] = (float)src[i * a.ldv + 1];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (single[i]) {
      cache_t *dst = group_of(slot[7 + i]) + (slot[7 + i] & 7);
      dst[0] = (cache_t)x[i];
      dst[8] = (cache_t)y[i];
    }
  }
  for (int i = 0; i < 8; ++i) {
    if (!lead[7 + i]) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = (float)src[(i + j) * a.ldv];
      y[j] = (float)src[(i + j) * a.ldv + 1];
    }
    cache_t *dst = group_of(slot[7 + i]);
    store8<TC>(dst, x);
    store8<TC>(dst + 8, y);
  }
}

template <class TI, class TC>
hipError_t launch(const KvAppend &a, int64_t blocks, hipStream_t stream) {
  return launch_in_pieces(blocks, kThreads, [&](uint32_t first, unsigned n) {
    if (a.interleaved)
      hipLaunchKernelGGL((kv_append_kernel<TI, TC, true>), dim3(n), dim3(kThreads), 0, stream, a, first);
    else
      hipLaunchKernelGGL((kv_append_kernel<TI, TC, false>), dim3(n), dim3(kThreads), 0, stream, a, first);
  });
}

}  // namespace

hipError_t kv_append_launch(KvAppend a, ElemType in, ElemType cache, hipStream_t stream) {
  // Heads per workgroup: as many as give every thread one item of 16
  // elements (the sines are computed once per workgroup).
  const int items = a.head_dim / 16, nh = a.n_q_heads + a.n_kv_heads;
  a.heads_per_block = kThreads / items;
  a.head_blocks = (nh + a.heads_per_block - 1) / a.heads_per_block;
  const int v_heads = kThreads / (a.head_dim / 2);
  a.v_blocks = (a.n_kv_heads + v_heads - 1) / v_heads;
  const int64_t rot = a.tokens * a.head_blocks, vb = (a.tokens + 7) / 8 * a.v_blocks;
  if (rot + vb > 0x7fffffff) return hipErrorInvalidValue;
  a.rot_blocks = (int)rot;
  const int64_t blocks = rot + vb;
  if (cache == ElemType::F16) {
    if (in == ElemType::F32) return launch<TypeF32, TypeF16>(a, blocks, stream);
    if (in == ElemType::F16) return launch<TypeF16, TypeF16>(a, blocks, stream);
    return launch<TypeBF16, TypeF16>(a, blocks, stream);
  }
  if (in == ElemType::F32) return launch<TypeF32, TypeBF16>(a, blocks, stream);
  if (in == ElemType::F16) return launch<TypeF16, TypeBF16>(a, blocks, stream);
  return launch<TypeBF16, TypeBF16>(a, blocks, stream);
}

}  // namespace lqmm
