// Matrix products in 8-bit floating point (e4m3) with an fp32 scale for each
// block of 128, and the quantization of activations to that form.
//
// Mathematics. W is N x K codes with one scale for each 128 x 128 block, X is
// M x K codes with one scale for each row and group of 128 columns:
//   Y[m][n] = sum_b sx[b][m] sw[n / 128][b] sum_{k in block b} X[m][k] W[n][k].
// The inner sum of one scale block for a 16 x 16 tile is four
// v_mfma_f32_16x16x32_f16, started from zero; the outer sum is one fp32
// multiply-add with the product of the two scales.
//
// Which matrix cores. The f8 ones do not sum in fp32: a product is cut off
// 14 bits below the largest of its group (measured: next to 448 * 448 =
// 200704, products below 8 vanish and 9 counts as 8), so that behind two large
// products that cancel a whole sum can be lost, whatever the output's type.
// The codes are turned into fp16 in registers instead (exactly) and multiplied
// there, at half the rate, with fp32 sums. What that costs with bf16 outputs
// (us, f8 / fp16 cores): 1 x 28672 x 8192 36.2 / 35.9, 45 x 4127 x 4112 8.6 /
// 11.8, 512 x 14336 x 4096 40 / 63, 4096 x 14336 x 4096 253 / 433.
//
// Layout. With W as the A operand, a lane holds four outputs of one row m
// (m = lane & 15), so the scale product is one value per lane and 16 rows of X:
// four multiply-adds per four matrix instructions, which run on the vector ALU
// beside them.
#include "lqmm_internal.hpp"
#include "serve_device.hpp"

namespace lqmm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---- activations to e4m3 ----------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr float kF8Max = 448.0f;

// Largest value over aligned groups of 16 lanes, in every lane.
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = fmaxf(v, dpp<0x141>(v));  // row_half_mirror
  v = fmaxf(v, dpp<0x140>(v));  // row_mirror
  return v;
}

// 16 lanes take one group of 128 (8 elements each); a workgroup takes 16
// rows of one group, so that the codes are written in whole 128-byte lines
// and the scales in 64-byte runs.
template <class T>
__global__ void __launch_bounds__(kQuantThreads)
quant_f8b128_kernel(const typename T::elem *__restrict__ X, int64_t ldx, uint8_t *__restrict__ Xq,
                    float *__restrict__ xs, int64_t M, int64_t K, int blocks, uint32_t first) {
  const int l16 = threadIdx.x & 15;
  const uint32_t block = first + blockIdx.x;
  const int b = block % blocks;
  const int64_t m = (int64_t)(block / blocks) * 16 + (threadIdx.x >> 4);
  const int64_t k = (int64_t)b * 128 + 8 * l16;
  if (m >= M) return;  // whole 16-lane groups
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (k < K) load8<T>(X + m * ldx + k, x);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
  // 2^-126: a group of zeros keeps a finite scale
  const float scale = fmaxf(max16(top) / kF8Max, 0x1p-126f);
  if (k < K) {
    // x / scale, correctly rounded (the codes are those of the quotient, ties
    // included): with r the rounded 1 / scale, one step q + (x - q scale) r
    // from q = x r (Markstein's theorem: the remainder is exact). Three
    // instructions a value; the compiler's division took about ten and half
    // of the kernel's time: 4000 x 8192 fp16 25.7 -> 19.2 us.
    // Of a very small group value and scale are taken 2^64 up first: the
    // remainder would fall below fp32's smallest step.
    float s = scale;
    if (scale < 0x1p-64f) {
      s *= 0x1p64f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
    }
    const float inv = 1.0f / s;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[i] * inv;
      y[i] = fmaf(fmaf(-q, s, x[i]), inv, q);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], v, true);
      w[i] = (uint32_t)v;
    }
    *reinterpret_cast<u32x2 *>(Xq + m * K + k) = u32x2{w[0], w[1]};
  }
  if (l16 == 0) xs[(int64_t)b * M + m] = scale;
}

// ---- product ----------------------------------------------------------------
// Four consecutive outputs y[0..3] of one row, of which the first `n` exist.
template <class T>
__device__ __forceinline__ void store4(typename T::elem *p, float4_t v, int n, bool vec) {
  typedef typename T::elem elem;
  typedef elem vec4 __attribute__((ext_vector_type(4)));
  const vec4 o = {(elem)v[0], (elem)v[1], (elem)v[2], (elem)v[3]};
  if (vec && n >= 4) {
    *reinterpret_cast<vec4 *>(p) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = o[i];
  }
}

constexpr int BK = 128;

// 32 codes as four operands of the fp16 matrix cores (exact).
__device__ __forceinline__ void to_f16(i32x8 c, half8_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * i], 1.0f, false);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * i], 1.0f, true);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * i + 1], 1.0f, false);
    const half2_t e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * i + 1], 1.0f, true);
    h[i] = half8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
  }
}

// A 16-row operand of one scale block, and the sum of one block's products.
struct Operand {
  half8_t v[4];
  __device__ __forceinline__ void set(i32x8 c) { to_f16(c, v); }
};
__device__ __forceinline__ float4_t block_sum(const Operand &a, const Operand &b) {
  float4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], p, 0, 0, 0);
  return p;
}

// A BM x BN tile (rows of X by rows of W). WK groups of WM x WN waves share
// it: a step of the K loop is WK scale blocks, each group takes one of them,
// and the groups' sums are added in LDS at the end, in a fixed order. NS LDS
// stages.
template <int BM, int BN, int WM, int WN, int WK, int NS>
struct Tile {
  static constexpr int kWaves = WM * WN * WK;
  static constexpr int kCodes = (BM + BN) * BK;         // bytes of a block's codes
  static constexpr int kPart = kCodes + (BM + 64) * 4;  // with the scales of its rows, and of W
  static constexpr int kStage = WK * kPart;
  static constexpr int kGroup = WM * WN;                // waves that load and use a block
  static constexpr int kLoads = (BM + BN) / 8 / kGroup; // 1 KB loads of a wave per step
  static constexpr int kSums = (WK - 1) * BM * BN * 4;  // bytes of the groups' sums
  static constexpr int kLds = NS * kStage > kSums ? NS * kStage : kSums;
};

template <class T, int BM, int BN, int WM, int WN, int WK, int NS>
__global__ void __launch_bounds__(64 * WM * WN * WK)
gemm_f8b128_kernel(const uint8_t *__restrict__ W, const float *__restrict__ sw,
                   const uint8_t *__restrict__ X, const float *__restrict__ sx,
                   typename T::elem *__restrict__ Y, int64_t M, int64_t N, int64_t K, uint32_t tiles_m,
                   uint32_t tiles_n, uint32_t first) {
  typedef Tile<BM, BN, WM, WN, WK, NS> C;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave
  constexpr int kScaleLoads = (BM + 63) / 64;          // waves of a group that bring scales of X
  static_assert((BM + BN) / 8 % C::kGroup == 0 && BN / WN <= 128 && 128 % (BN / WN) == 0, "tile");
  static_assert(BM % 64 == 0 && kScaleLoads <= C::kGroup, "scale loads");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave / C::kGroup, gw = wave % C::kGroup;  // block of the step, wave of the group
  const int l16 = lane & 15, g = lane >> 4;
  // Workgroups go to the 8 XCDs in turn; consecutive tiles (the M tiles of one
  // W tile) are put on one XCD, whose L2 then holds the W tile once.
  const uint32_t tiles = tiles_m * tiles_n, block = first + blockIdx.x;
  const uint32_t xcd = block % 8, q8 = tiles / 8, r8 = tiles % 8;
  const uint32_t tile = xcd * q8 + (xcd < r8 ? xcd : r8) + block / 8;
  const int64_t m0 = (int64_t)(tile % tiles_m) * BM;
  const int64_t n0 = (int64_t)(tile / tiles_m) * BN;
  const int wm = (gw % WM) * (BM / WM), wn = (gw / WM) * (BN / WN);
  const int blocks = (int)((K + BK - 1) / BK), steps = (blocks + WK - 1) / WK;
  const uint32_t Ku = (uint32_t)K;

  const int64_t xrows = M - m0 < BM ? M - m0 : BM;
  const int64_t wrows = N - n0 < BN ? N - n0 : BN;
  const rsrc_t xr = make_rsrc(X + m0 * K, (uint32_t)(xrows * K));
  const rsrc_t wr = make_rsrc(W + n0 * K, (uint32_t)(wrows * K));

  // Tile rows of 128 bytes; 16-byte chunk c of row r stands in slot
  // c ^ (r & 7), so that the eight rows that one phase of a 16-byte LDS read
  // touches lie in different banks. A load fills 8 rows, lane by lane.
  const int lrow = lane >> 3, lcol = 16 * ((lane & 7) ^ lrow);
  // The block's scales: wave w < BM / 64 of the group brings those of rows
  // 64 w .. of X; the last wave those of the tile's 128-row blocks of W (the
  // others in between the same again; with too few waves, an extra load).
  constexpr bool kExtra = kScaleLoads == C::kGroup;  // the last wave brings both
  const bool x_scales = gw < kScaleLoads;
  const int64_t sm = m0 + 64 * gw + lane;
  const float *sxp = sx + (sm < M ? sm : M - 1);
  const int64_t nb = n0 / 128 + lane % (BN > 128 ? BN / 128 : 1), last_nb = (N - 1) / 128;
  const float *swp = sw + (nb < last_nb ? nb : last_nb) * blocks;
  auto issue = [&](int step) {
    uint8_t *st = smem + (step % NS) * C::kStage + wk * C::kPart;
    const int kt = step * WK + wk;
    // past K the rows of the next line begin: those chunks read as zeros
    // (an offset past the resource)
    const bool in = (uint32_t)(kt * BK + lcol) < Ku;
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const int j = gw * C::kLoads + i;  // 8 rows: X first, then W
      const bool is_x = j < BM / 8;
      const int r = 8 * (is_x ? j : j - BM / 8) + lrow;
      const int off = in ? (int)((uint32_t)r * Ku + lcol) : (int)0x80000000u;
      if (is_x)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, st + j * 1024, 16, off, kt * BK, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, st + j * 1024, 16, off, kt * BK, 0, 0);
    }
    const int b = kt < blocks ? kt : blocks - 1;
    const bool xs_here = x_scales;
    load_to_lds<4>(xs_here ? sxp + (int64_t)b * M : swp + b,
                   st + C::kCodes + (xs_here ? gw * 256 : BM * 4));
    if constexpr (kExtra) load_to_lds<4>(swp + b, st + C::kCodes + BM * 4);
  };
  constexpr int kStepLoads = C::kLoads + (kExtra ? 2 : 1);
  auto frag = [&](const uint8_t *base, int row) {
    const int s = row & 7;
    const i32x4 lo = *reinterpret_cast<const i32x4 *>(base + row * BK + 16 * (g ^ s));
    const i32x4 hi = *reinterpret_cast<const i32x4 *>(base + row * BK + 16 * ((g + 4) ^ s));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  float4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};
  // The block sums of the 16 rows before, and their scale: they are added
  // while the matrix cores work on the next 16.
  float4_t p[TN];
  float s_prev = 0.f;
#pragma unroll
  for (int j = 0; j < TN; ++j) p[j] = float4_t{0.f, 0.f, 0.f, 0.f};
  // Operands of X that are read ahead: all of a step's when they fit in
  // registers beside the sums, else one.
  constexpr int kAhead = TM + TN <= 8 ? TM : 2;

#pragma unroll
  for (int d = 0; d < NS - 1; ++d)
    if (d < steps) issue(d);
  for (int kt = 0; kt < steps; ++kt) {
    // the loads of step kt are done when only those of the later steps are out
    if (kt + NS - 2 < steps)
      wait_loads_and_barrier<(NS - 2) * kStepLoads>();
    else
      wait_loads_and_barrier<0>();
    if (kt + NS - 1 < steps) issue(kt + NS - 1);
    const uint8_t *xst = smem + (kt % NS) * C::kStage + wk * C::kPart, *wst = xst + BM * BK;
    const float *scales = reinterpret_cast<const float *>(xst + C::kCodes);
    const float s_n = scales[BM + wn / 128];
    i32x8 wraw[TN], xraw[kAhead];
#pragma unroll
    for (int j = 0; j < TN; ++j) wraw[j] = frag(wst, wn + 16 * j + l16);
#pragma unroll
    for (int i = 0; i < (kAhead == TM ? TM : 1); ++i) xraw[i] = frag(xst, wm + 16 * i + l16);
    Operand wf[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) wf[j].set(wraw[j]);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (kAhead != TM && i + 1 < TM) xraw[(i + 1) % kAhead] = frag(xst, wm + 16 * (i + 1) + l16);
      const float s = scales[wm + 16 * i + l16] * s_n;
      Operand xf;
      xf.set(xraw[i % kAhead]);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const float4_t q = block_sum(wf[j], xf);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[(i + TM - 1) % TM][j][r] += p[j][r] * s_prev;
        p[j] = q;
      }
      s_prev = s;
    }
  }
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[TM - 1][j][r] += p[j][r] * s_prev;

  if constexpr (WK > 1) {
    // sums of group k > 0, each lane's values together: the same lane of group
    // 0 adds them
    float4_t *sums = reinterpret_cast<float4_t *>(smem);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (wk > 0) sums[(((wk - 1) * C::kGroup + gw) * TM * TN + i * TN + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int k = 1; k < WK; ++k)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] += sums[(((k - 1) * C::kGroup + gw) * TM * TN + i * TN + j) * 64 + lane];
  }

  const bool vec = N % 4 == 0;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + wm + 16 * i + l16;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int64_t n = n0 + wn + 16 * j + 4 * g;
      if (n < N) store4<T>(Y + m * N + n, acc[i][j], (int)(N - n < 4 ? N - n : 4), vec);
    }
  }
}

// Few rows of X (decode): bound by reading W once. A workgroup takes 16 * TN
// rows of W; its waves share K, wave w taking a contiguous run of scale
// blocks, and their sums are added in LDS in a fixed order. W and X go
// straight from memory to the operands, DEPTH blocks ahead, in registers.
constexpr int kRowWaves = 8;

template <class T, int TM, int TN, int DEPTH>
__global__ void __launch_bounds__(64 * kRowWaves)
gemm_f8b128_rows_kernel(const uint8_t *__restrict__ W, const float *__restrict__ sw,
                        const uint8_t *__restrict__ X, const float *__restrict__ sx,
                        typename T::elem *__restrict__ Y, int64_t M, int64_t N, int64_t K,
                        uint32_t tiles_n, uint32_t first) {
  constexpr int kN = 16 * TN, kM = 16 * TM, kLd = kN + 4;
  __shared__ __attribute__((aligned(16))) float part[kRowWaves][kM][kLd];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const uint32_t block = first + blockIdx.x;
  const int64_t n0 = (int64_t)(block % tiles_n) * kN;
  const int64_t m0 = (int64_t)(block / tiles_n) * kM;
  const int blocks = (int)((K + BK - 1) / BK);
  const int per = (blocks + kRowWaves - 1) / kRowWaves;
  const int kb0 = wave * per, kb1 = kb0 + per < blocks ? kb0 + per : blocks;
  const uint32_t Ku = (uint32_t)K;

  const int64_t wrows = N - n0 < kN ? N - n0 : kN;
  const int xrows = (int)(M - m0 < kM ? M - m0 : kM);
  // rows past the ends read zeros
  const rsrc_t wr = make_rsrc(W + n0 * K, (uint32_t)(wrows * K));
  const rsrc_t xr = make_rsrc(X + m0 * K, (uint32_t)(xrows * K));
  const float *swr = sw + (n0 / 128) * blocks;

  struct Stage {
    u32x4 w[TN][2], x[TM][2];
    float sx[TM], sw;
  } st[DEPTH];
  const uint32_t off = (uint32_t)l16 * Ku + 16 * g;
  auto load = [&](Stage &s, int kb) {
    const uint32_t c = (uint32_t)kb * BK;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) s.w[j][u] = buf_load_b128(wr, off + 16 * j * Ku + 64 * u + c);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int u = 0; u < 2; ++u) s.x[i][u] = buf_load_b128(xr, off + 16 * i * Ku + 64 * u + c);
      const int m = 16 * i + l16;
      s.sx[i] = sx[(int64_t)kb * M + m0 + (m < xrows ? m : 0)];
    }
    s.sw = swr[kb];
  };
  auto operand = [&](const u32x4 (&v)[2]) {
    Operand o;
    o.set(__builtin_bit_cast(i32x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7)));
    return o;
  };

  float4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (kb0 + d < kb1) load(st[d], kb0 + d);
  for (int kb = kb0; kb < kb1; kb += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (kb + d >= kb1) break;
      Stage &s = st[d];
      // past K the next row begins
      if (kb + d == blocks - 1 && Ku % BK != 0) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if ((uint32_t)(kb + d) * BK + 16 * g + 64 * u >= Ku) {
#pragma unroll
            for (int j = 0; j < TN; ++j) s.w[j][u] = zero;
#pragma unroll
            for (int i = 0; i < TM; ++i) s.x[i][u] = zero;
          }
      }
      Operand w[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) w[j] = operand(s.w[j]);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const Operand x = operand(s.x[i]);
        const float f = s.sx[i] * s.sw;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const float4_t p = block_sum(w[j], x);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] += p[r] * f;
        }
      }
      if (kb + d + DEPTH < kb1) load(s, kb + d + DEPTH);
    }
  }

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
      *reinterpret_cast<float4_t *>(&part[wave][16 * i + l16][16 * j + 4 * g]) = acc[i][j];
  __syncthreads();
  for (int o = tid; o < kM * kN; o += 64 * kRowWaves) {
    const int m = o / kN, n = o % kN;
    if (m >= xrows || n >= wrows) continue;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) y += part[w][m][n];
    Y[(m0 + m) * N + n0 + n] = (typename T::elem)y;
  }
}

template <class T, int BM, int BN, int WM, int WN, int WK, int NS>
hipError_t launch_tile(const uint8_t *W, const float *sw, const uint8_t *X, const float *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  constexpr int kLds = Tile<BM, BN, WM, WN, WK, NS>::kLds;
  constexpr auto kern = gemm_f8b128_kernel<T, BM, BN, WM, WN, WK, NS>;
  const int64_t tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN;
  const hipError_t e = ensure_max_lds<kern>(kLds);
  if (e != hipSuccess) return e;
  return launch_in_pieces(tm * tn, 64 * WM * WN * WK, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL(kern, dim3(n), dim3(64 * WM * WN * WK), kLds, stream, W, sw, X, sx,
                       static_cast<typename T::elem *>(Y), M, N, K, (uint32_t)tm, (uint32_t)tn, first);
  });
}

template <class T, int TM, int TN, int DEPTH>
hipError_t launch_rows(const uint8_t *W, const float *sw, const uint8_t *X, const float *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t tn = (N + 16 * TN - 1) / (16 * TN), tm = (M + 16 * TM - 1) / (16 * TM);
  return launch_in_pieces(tm * tn, 64 * kRowWaves, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((gemm_f8b128_rows_kernel<T, TM, TN, DEPTH>), dim3(n), dim3(64 * kRowWaves), 0,
                       stream, W, sw, X, sx, static_cast<typename T::elem *>(Y), M, N, K, (uint32_t)tn,
                       first);
  });
}

template <class T>
hipError_t launch_gemm(const uint8_t *W, const float *sw, const uint8_t *X, const float *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, int num_cus, hipStream_t stream) {
  // Up to 16 rows: W is read once, by 16 of its rows a workgroup; by 64 when
  // that still gives most CUs one and X is worth sharing. Measured (K = 4096,
  // us, 16 / 64 rows of W): M = 16, N = 4096 6.3 / 11.4, N = 14336 18.2 / 12.8,
  // N = 28672 and K = 8192 52 / 42; M = 1, N = 28672 and K = 8192 36 / 39.
  if (M <= 16) {
    if (M > 4 && N >= 48 * (int64_t)num_cus)
      return launch_rows<T, 1, 4, 2>(W, sw, X, sx, Y, M, N, K, stream);
    return launch_rows<T, 1, 1, 4>(W, sw, X, sx, Y, M, N, K, stream);
  }
  // Else the kernel and tile whose estimated time is least: rounds over the
  // CUs times what a workgroup takes, a fixed part and one per scale block.
  // The two parts (ns) were fitted to times at M = 24 .. 4096, N = 1001 ..
  // 14336, K = 1040 and 4096; e.g. (us) 24 x 4127 x 4096 9.6 with 32 x 32 rows
  // and 10.9 with 64 x 32 tiles, 200 x 4127 x 1040 11.9 with 64 x 32 rows, 16.2
  // with 64 x 32 and 12.1 with 64 x 64 tiles, 512 x 14336 x 4096 67 with 128 x
  // 256 and 77 with 64 x 64 tiles, 1024 x 4096 x 4096 34 with 128 x 128 and 61
  // with 128 x 256 tiles.
  struct Choice {
    int bm, bn, per_cu, fixed, block;
  };
  constexpr Choice kChoices[] = {
      // W straight to registers, for few rows of X
      {32, 16, 1, 200, 170}, {32, 32, 1, 200, 250}, {48, 32, 1, 200, 350}, {64, 32, 1, 200, 420},
      // LDS tiles
      {64, 32, 1, 2000, 240}, {64, 64, 1, 3000, 280}, {64, 64, 2, 2000, 660},
      {128, 128, 1, 3000, 1100}, {128, 256, 1, 4000, 2050}};
  const int64_t blocks = (K + BK - 1) / BK;
  int best = -1;
  int64_t best_cost = 0;
  for (int c = 0; c < 9; ++c) {
    const Choice &o = kChoices[c];
    const int64_t tiles = ((M + o.bm - 1) / o.bm) * ((N + o.bn - 1) / o.bn);
    const int64_t slots = (int64_t)o.per_cu * num_cus;
    if (tiles > 0xffffffffll) continue;  // (they are numbered in 32 bits)
    const int64_t cost = (tiles + slots - 1) / slots * (o.fixed + o.block * blocks);
    if (best < 0 || cost < best_cost) {
      best = c;
      best_cost = cost;
    }
  }
  switch (best) {
    case 0: return launch_rows<T, 2, 1, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 1: return launch_rows<T, 2, 2, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 2: return launch_rows<T, 3, 2, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 3: return launch_rows<T, 4, 2, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 4: return launch_tile<T, 64, 32, 2, 1, 4, 3>(W, sw, X, sx, Y, M, N, K, stream);
    case 5: return launch_tile<T, 64, 64, 1, 2, 4, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 6: return launch_tile<T, 64, 64, 2, 2, 2, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 7: return launch_tile<T, 128, 128, 2, 2, 2, 2>(W, sw, X, sx, Y, M, N, K, stream);
    case 8: return launch_tile<T, 128, 256, 2, 4, 1, 3>(W, sw, X, sx, Y, M, N, K, stream);
  }
  return hipErrorInvalidValue;
}

template <class T>
hipError_t launch_quant(const void *X, int64_t ldx, uint8_t *Xq, float *xs, int64_t M, int64_t K,
                        hipStream_t stream) {
  const int64_t blocks = (K + 127) / 128, rows = (M + 15) / 16;
  if (blocks * rows > 0x7fffffff) return hipErrorInvalidValue;
  return launch_in_pieces(blocks * rows, kQuantThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL(quant_f8b128_kernel<T>, dim3(n), dim3(kQuantThreads), 0, stream,
                       static_cast<const typename T::elem *>(X), ldx, Xq, xs, M, K, (int)blocks, first);
  });
}

}  // namespace

hipError_t quant_f8b128_launch(const void *X, ElemType type, int64_t ldx, uint8_t *Xq, float *xs,
                               int64_t M, int64_t K, hipStream_t stream) {
  if (type == ElemType::F32) return launch_quant<TypeF32>(X, ldx, Xq, xs, M, K, stream);
  if (type == ElemType::F16) return launch_quant<TypeF16>(X, ldx, Xq, xs, M, K, stream);
  return launch_quant<TypeBF16>(X, ldx, Xq, xs, M, K, stream);
}

hipError_t gemm_f8b128_launch(const uint8_t *W, const float *sw, const uint8_t *X, const float *sx,
                              void *Y, ElemType type, int64_t M, int64_t N, int64_t K, int num_cus,
                              hipStream_t stream) {
  if (type == ElemType::F32) return launch_gemm<TypeF32>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
  if (type == ElemType::F16) return launch_gemm<TypeF16>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
  return launch_gemm<TypeBF16>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
}

}  // namespace lqmm
