// Norms of the heads of q and k, the position rotation, and the append to a
// paged cache of 16 bits or of e4m3 codes, in one pass over the projections.
//
// Mathematics. A head's vector x becomes y = w x / sqrt(mean(x^2) + eps) (each
// of q and k with a weight of its own, or none), then its first R elements turn
// by the position as in kv_append.hip. Into an 8-bit cache go, for each token
// and head, the codes of y 2^-e and e (f8_cache.hpp); V is quantized the same
// way, without norm and rotation. Sums, products and the largest value are fp32;
// each output is rounded once.
//
// Layout. D / 16 lanes hold a head's vector in registers, 16 elements each (the
// halves of eight pairs, as the rotation wants them), so that the sum of squares
// and the largest value are DPP reductions over neighbouring lanes. Workgroups
// [0, rot_blocks) do one token's heads of q and K; the others V of eight tokens,
// whose codes go through LDS, since a page keeps eight tokens of one dimension
// adjacent and a token's scale is known only behind its whole vector.
//
// Bound by memory from some thousand tokens on: 16381 tokens, 64/8 heads of 128,
// bf16 into 8 bits 130 us (124 at the rate of a large copy; the vector ALU is
// busy 60 % of the time, with norms, turns and codes). 203 tokens, 40/8
// heads, fp32 into 16 bits 7.1 us: half a token's heads are one workgroup's round
// trip, V's lines are written in part. 1 token 3.9 us: launch and two dependent
// round trips.
#include "f8_cache.hpp"
#include "lqmm_internal.hpp"

namespace lqmm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // head_dim <= 256

// Lanes of a head's vector: D / 16, or the next power of two (96: 6 of 8).
constexpr int lanes_of(int d) { return d == 64 ? 4 : d <= 128 ? 8 : 16; }

template <int L>
__device__ __forceinline__ float max_of_lanes(float v) {
  v = fmaxf(v, dpp<0xB1>(v));                       // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp<0x4E>(v));                       // quad_perm [2,3,0,1]
  if constexpr (L > 4) v = fmaxf(v, dpp<0x141>(v)); // row_half_mirror
  if constexpr (L > 8) v = fmaxf(v, dpp<0x140>(v)); // row_mirror
  return v;
}

// 1 / sqrt(mean(x^2) + eps) of the vector that L lanes hold. Where the fp32 sum
// leaves its range (or a value is infinite or NaN) it is done in 64 bits.
template <int L, int D>
__device__ __forceinline__ double inverse_norm_far(const float (&x)[8], const float (&y)[8], float eps) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += (double)x[i] * x[i] + (double)y[i] * y[i];
#pragma unroll
  for (int n = 1; n < L; n *= 2) s += __shfl_xor(s, n);
  return 1.0 / sqrt(s * (1.0 / D) + (double)eps);
}

template <int L, int D>
__device__ __forceinline__ void normalize(float (&x)[8], float (&y)[8], float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], fmaf(y[i], y[i], s));
  s = group_sum(s, L);
  // (a lane's own test would split the vector's lanes: s is the same in all)
  if (s > 0x1p-90f && s < 0x1p100f) {
    const float r = 1.0f / sqrtf(fmaf(s, 1.0f / D, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r, y[i] *= r;
  } else {
    const double r = inverse_norm_far<L, D>(x, y, eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)(x[i] * r), y[i] = (float)(y[i] * r);
  }
}

// Scale byte of the vector that L lanes hold. An infinity has no code: it
// becomes NaN, and the finite values keep a scale of their own. Values past the
// largest scale's codes are held as the largest code.
template <int L>
__device__ __forceinline__ int vector_scale(float (&x)[8], float (&y)[8], int most) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(y[i])));
  top = max_of_lanes<L>(top);
  if (top == INFINITY) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(x[i]) == INFINITY) x[i] = NAN;
      if (fabsf(y[i]) == INFINITY) y[i] = NAN;
      top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(y[i])));
    }
    top = max_of_lanes<L>(top);
  }
  const int b = scale_byte(top, most);
  if (b == most) {
    const float lim = kCodeMax * scale_of(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(x[i]) > lim) x[i] = copysignf(lim, x[i]);
      if (fabsf(y[i]) > lim) y[i] = copysignf(lim, y[i]);
    }
  }
  return b;
}

// Elements [i, i + 8) of a head's weights, which all 16-byte aligned.
__device__ __forceinline__ void weigh(float (&x)[8], const float *w) {
  float f[8];
  load8<TypeF32>(w, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= f[i];
}

template <class TI, class TC, int D, bool INTER, bool F8>
__global__ void __launch_bounds__(kThreads)
kv_append_norm_kernel(KvAppendNorm a, uint32_t first) {
  typedef typename TI::elem in_t;
  typedef typename TC::elem type_t;
  constexpr int L = lanes_of(D), kItems = D / 16;
  constexpr int kHeads = kThreads / L;  // heads of q and K in a workgroup
  const int tid = threadIdx.x;
  const uint32_t block = first + blockIdx.x;
  const int64_t nslots = a.num_pages << a.page_log2;
  const int in_page = (1 << a.page_log2) - 1;
  const int64_t head_elems = (int64_t)D << a.page_log2;  // one head of one page
  const int c = tid % L;                                 // this lane's 16 elements of a vector
  const bool there = c < kItems;

  if ((int)block < a.rot_blocks) {
    // One token and up to kHeads of its q and K heads.
    __shared__ float cs[2][kMaxPairs];
    const int64_t t = block / a.head_blocks;
    const int h = (int)(block % a.head_blocks) * kHeads + tid / L;
    const int pairs = a.rot_dim / 2;
    const bool is_k = h >= a.n_q_heads;
    const int hk = h - a.n_q_heads;
    const bool live = there && h < a.n_q_heads + a.n_kv_heads;
    // A lane's elements: 8 pairs, or 16 unrotated ones.
    const bool turns = c < a.rot_dim / 16;
    const int e0 = turns ? (INTER ? 16 * c : 8 * c) : 16 * c;
    const int e1 = turns && !INTER ? e0 + pairs : e0 + 8;
    float x[8] = {}, y[8] = {};
    if (live) {
      const in_t *src = is_k ? static_cast<const in_t *>(a.k) + t * a.ldk + (int64_t)hk * D
                             : static_cast<const in_t *>(a.q) + t * a.ldq + (int64_t)h * D;
      load8<TI>(src + e0, x);
      load8<TI>(src + e1, y);
    }
    const int64_t slot = a.slots[t];
    if (pairs) {
      const uint64_t pos = (uint64_t)(int64_t)a.positions[t];
      for (int i = tid; i < pairs; i += kThreads) {
        const int32_t turn = (int32_t)((pos * a.turns[i]) >> 32);  // of 2^32, signed
        float s, co;
        sincospif((float)turn * 0x1p-31f, &s, &co);
        cs[0][i] = co;
        cs[1][i] = s;
      }
      __syncthreads();
    }
    if (h >= a.n_q_heads + a.n_kv_heads) return;  // whole vectors
    const float *weight = is_k ? a.k_norm : a.q_norm;
    if (weight) {
      normalize<L, D>(x, y, a.eps);
      if (there) {
        weigh(x, weight + e0);
        weigh(y, weight + e1);
      }
    }
    if (turns) {
      float z[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = x[i], z[8 + i] = y[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int i0 = INTER ? 2 * i : i, i1 = INTER ? i0 + 1 : 8 + i;
        const float co = cs[0][8 * c + i], s = cs[1][8 * c + i];
        const float x0 = z[i0], x1 = z[i1];
        z[i0] = x0 * co - x1 * s;
        z[i1] = x1 * co + x0 * s;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = z[i], y[i] = z[8 + i];
    }
    if (!is_k) {
      if (!live) return;
      type_t *dst = static_cast<type_t *>(a.q_out) + (t * a.n_q_heads + h) * D;
      store8<TC>(dst + e0, x);
      store8<TC>(dst + e1, y);
      return;
    }
    if (slot < 0 || slot >= nslots) return;
    const int64_t vec = (((slot >> a.page_log2) * a.n_kv_heads + hk) << a.page_log2) + (slot & in_page);
    if constexpr (F8) {
      const int b = vector_scale<L>(x, y, a.most_scale);
      const float mul = scale_inverse(b);
      uint8_t *dst = static_cast<uint8_t *>(a.k_cache) + vec * D;
      if (there) {
        *reinterpret_cast<u32x2 *>(dst + e0) = codes8(x, mul);
        *reinterpret_cast<u32x2 *>(dst + e1) = codes8(y, mul);
      }
      if (c == 0) a.k_scales[vec] = (uint8_t)b;
    } else if (there) {
      type_t *dst = static_cast<type_t *>(a.k_cache) + vec * D;
      store8<TC>(dst + e0, x);
      store8<TC>(dst + e1, y);
    }
    return;
  }

  // V of tokens t0 .. t0 + 7 and some of the heads. A token whose slot starts a
  // group of eight, followed by seven tokens with the next seven slots, leads a
  // whole group, which is stored as vectors (it may reach into the next
  // workgroup's tokens; a window of eight tokens has one such leader at most); a
  // token inside such a group is skipped; any other is stored by itself.
  typedef __attribute__((may_alias)) uint32_t word_t;
  constexpr int kVHeads = 32 / L;             // eight tokens of a head at a time
  constexpr int kBytes = F8 ? 1 : 2;          // of a stored element
  constexpr int kWords = D * kBytes / 4;      // of a vector
  __shared__ __attribute__((aligned(16))) uint8_t held[15][kVHeads][D * kBytes];
  __shared__ int64_t slots[24];
  __shared__ int lead[16];
  const int64_t t0 = (int64_t)((block - a.rot_blocks) / a.v_blocks) * 8;
  const int h0 = (int)((block - a.rot_blocks) % a.v_blocks) * kVHeads;
  if (tid < 22) {
    const int64_t t = t0 - 7 + tid;
    int64_t s = -1;
    if (t >= 0 && t < a.tokens) {
      s = a.slots[t];
      if (s >= nslots) s = -1;
    }
    slots[tid] = s;
  }
  __syncthreads();
  if (tid < 15) {
    const int64_t s = slots[tid];
    bool l = s >= 0 && (s & 7) == 0;
    for (int i = 1; i < 8; ++i) l = l && slots[tid + i] == s + i;
    lead[tid] = l;
  }
  __syncthreads();
  int leader = 8;  // place of the leader in the window
  uint32_t single = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t s = slots[7 + i];
    const int before = (int)(s & 7);
    if (lead[7 + i]) leader = i;
    else if (s >= 0 && !lead[7 + i - before]) single |= 1u << i;
  }
  // Tokens that this workgroup stores, by place: singles, and the leader's eight.
  uint32_t stored = single | (leader < 8 ? 0xffu << leader : 0u);
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    const int p = 8 * round + tid / (L * kVHeads), hh = tid / L % kVHeads, h = h0 + hh;
    const bool live = (stored >> p & 1) && h < a.n_kv_heads;  // the same for a vector's lanes
    if (!live) continue;
    float x[8] = {}, y[8] = {};
    if (there) {
      const in_t *src = static_cast<const in_t *>(a.v) + (t0 + p) * a.ldv + (int64_t)h * D + 16 * c;
      load8<TI>(src, x);
      load8<TI>(src + 8, y);
    }
    uint8_t *to = &held[p][hh][16 * kBytes * c];
    if constexpr (F8) {
      const int b = vector_scale<L>(x, y, a.most_scale);
      const float mul = scale_inverse(b);
      const u32x2 lo = codes8(x, mul), hi = codes8(y, mul);
      if (there) *reinterpret_cast<u32x4 *>(to) = u32x4{lo[0], lo[1], hi[0], hi[1]};
      const int64_t s = slots[7 + p];
      if (c == 0)
        a.v_scales[(((s >> a.page_log2) * a.n_kv_heads + h) << a.page_log2) + (s & in_page)] = (uint8_t)b;
    } else if (there) {
      store8<TC>(reinterpret_cast<type_t *>(to), x);
      store8<TC>(reinterpret_cast<type_t *>(to) + 8, y);
    }
  }
  __syncthreads();
  uint8_t *vc = static_cast<uint8_t *>(a.v_cache);
  auto group_of = [&](int64_t s, int h) {  // first byte of the group of eight that holds slot s
    return vc + ((s >> a.page_log2) * a.n_kv_heads + h) * head_elems * kBytes +
           (int64_t)((s & in_page) >> 3) * (8 * D * kBytes);
  };
  if (leader < 8) {
    // a thread transposes one word (4 codes or 2 elements) of the eight tokens
    for (int i = tid; i < kVHeads * kWords; i += kThreads) {
      const int hh = i / kWords, w = i % kWords;
      if (h0 + hh >= a.n_kv_heads) continue;
      uint32_t r[8], o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = reinterpret_cast<const word_t *>(held[leader + j][hh])[w];
      if constexpr (F8) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t sel = 0x0c0c0400u + 0x0101u * d;
            const uint32_t lo = __builtin_amdgcn_perm(r[4 * q + 1], r[4 * q], sel);
            const uint32_t hi = __builtin_amdgcn_perm(r[4 * q + 3], r[4 * q + 2], sel);
            o[2 * d + q] = lo | hi << 16;
          }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[j] = __builtin_amdgcn_perm(r[2 * j + 1], r[2 * j], 0x05040100u);
          o[4 + j] = __builtin_amdgcn_perm(r[2 * j + 1], r[2 * j], 0x07060302u);
        }
      }
      u32x4 *dst = reinterpret_cast<u32x4 *>(group_of(slots[7 + leader], h0 + hh) + 32 * w);
      dst[0] = u32x4{o[0], o[1], o[2], o[3]};
      dst[1] = u32x4{o[4], o[5], o[6], o[7]};
    }
  }
  if (single) {
    for (int i = tid; i < 8 * kVHeads * kWords; i += kThreads) {
      const int w = i % kWords, hh = i / kWords % kVHeads, p = i / kWords / kVHeads;
      if (!(single >> p & 1) || h0 + hh >= a.n_kv_heads) continue;
      const uint32_t r = reinterpret_cast<const word_t *>(held[p][hh])[w];
      const int64_t s = slots[7 + p];
      uint8_t *dst = group_of(s, h0 + hh) + 32 * w + (s & 7) * kBytes;
      if constexpr (F8) {
#pragma unroll
        for (int d = 0; d < 4; ++d) dst[8 * d] = (uint8_t)(r >> 8 * d);
      } else {
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)r;
        *reinterpret_cast<uint16_t *>(dst + 16) = (uint16_t)(r >> 16);
      }
    }
  }
}

template <class TI, class TC, int D>
hipError_t launch(KvAppendNorm a, hipStream_t stream) {
  constexpr int L = lanes_of(D), kHeads = kThreads / L, kVHeads = 32 / L;
  a.heads_per_block = kHeads;
  a.head_blocks = (a.n_q_heads + a.n_kv_heads + kHeads - 1) / kHeads;
  a.v_blocks = (a.n_kv_heads + kVHeads - 1) / kVHeads;
  const int64_t rot = a.tokens * a.head_blocks, vb = (a.tokens + 7) / 8 * a.v_blocks;
  if (rot + vb > 0x7fffffff) return hipErrorInvalidValue;
  a.rot_blocks = (int)rot;
  return launch_in_pieces(rot + vb, kThreads, [&](uint32_t first, unsigned n) {
    const dim3 g(n), b(kThreads);
    if (a.k_scales) {
      if (a.interleaved)
        hipLaunchKernelGGL((kv_append_norm_kernel<TI, TC, D, true, true>), g, b, 0, stream, a, first);
      else
        hipLaunchKernelGGL((kv_append_norm_kernel<TI, TC, D, false, true>), g, b, 0, stream, a, first);
    } else {
      if (a.interleaved)
        hipLaunchKernelGGL((kv_append_norm_kernel<TI, TC, D, true, false>), g, b, 0, stream, a, first);
      else
        hipLaunchKernelGGL((kv_append_norm_kernel<TI, TC, D, false, false>), g, b, 0, stream, a, first);
    }
  });
}

template <class TI, class TC>
hipError_t launch_dim(const KvAppendNorm &a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch<TI, TC, 64>(a, stream);
    case 96: return launch<TI, TC, 96>(a, stream);
    case 128: return launch<TI, TC, 128>(a, stream);
    case 256: return launch<TI, TC, 256>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t kv_append_norm_launch(KvAppendNorm a, ElemType in, ElemType type, hipStream_t stream) {
  a.most_scale = type == ElemType::F16 ? kMostScaleF16 : kMostScaleBF16;
  if (type == ElemType::F16) {
    if (in == ElemType::F32) return launch_dim<TypeF32, TypeF16>(a, stream);
    if (in == ElemType::F16) return launch_dim<TypeF16, TypeF16>(a, stream);
    return launch_dim<TypeBF16, TypeF16>(a, stream);
  }
  if (in == ElemType::F32) return launch_dim<TypeF32, TypeBF16>(a, stream);
  if (in == ElemType::F16) return launch_dim<TypeF16, TypeBF16>(a, stream);
  return launch_dim<TypeBF16, TypeBF16>(a, stream);
}

}  // namespace lqmm
