// Microscaled 4-bit floating point (OCP Microscaling Formats v1.0, MXFP4): e2m1
// codes with one power of two for each block of 32 along K; quantization and
// the product of two such matrices.
//
// Mathematics. Y[m][n] = sum over blocks b of 2^(xs + ws) sum_{k in b} X[m][k]
// W[n][k]. One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies four blocks of 16
// rows by 16 rows and applies both scales. It adds as fp32 does: measured, beside
// two products that cancel 2^30 above it 0.25 is kept, and a term below a sum's
// last place rounds it to nearest even (the 8-bit formats of this instruction
// are cut off 14 bits below their largest product; these products have 8 bits).
//
// Layout. A lane's operand is one block: 16 bytes of codes and one byte of
// scale. Which blocks are one instruction is free: of 16 blocks in a row (512 of
// K) a lane takes the four from 4 g on (g = lane / 16), one for each of four
// instructions, so that its scales are one word, of which each instruction names
// a byte, and its codes 64 bytes next to each other.
#include "lqmm_internal.hpp"
#include "serve_device.hpp"

namespace lqmm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---- quantization -------------------------------------------------------------
constexpr int kQuantThreads = 256;

// Four lanes take one block, eight values each: reads are 16 (32) bytes a lane
// side by side, codes 4 bytes a lane.
template <class T>
__global__ void __launch_bounds__(kQuantThreads)
quant_mxfp4_kernel(const typename T::elem *__restrict__ X, int64_t ldx, uint8_t *__restrict__ Xq,
                   uint8_t *__restrict__ xs, int64_t M, int64_t K, uint32_t first) {
  const int tid = threadIdx.x;
  const int64_t per_row = K / 8;  // lanes of a row
  const int64_t u0 = ((int64_t)first + blockIdx.x) * kQuantThreads;
  const int64_t m0 = u0 / per_row;
  const uint32_t in_row = (uint32_t)(u0 - m0 * per_row) + tid;  // (below 2^31)
  const uint32_t skip = in_row / (uint32_t)per_row;
  const int64_t m = m0 + skip;
  const uint32_t c = in_row - skip * (uint32_t)per_row;
  if (m >= M) return;  // whole blocks
  float x[8];
  load8<T>(X + m * ldx + 8 * (int64_t)c, x);
  float top = 0.f;
  bool odd = false;  // an infinity or NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    odd = odd || !(a < INFINITY);
    top = fmaxf(top, a);
  }
  if (odd) top = INFINITY;
  top = fmaxf(top, dpp<0xB1>(top));  // quad_perm [1,0,3,2]
  top = fmaxf(top, dpp<0x4E>(top));  // quad_perm [2,3,0,1]
  // floor(log2 top) - 2, at least -127; a block with an infinity or NaN is NaN
  const int b = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 2;
  const uint32_t byte = top == INFINITY ? 255u : b < 0 ? 0u : (uint32_t)b;
  const float mul = __builtin_bit_cast(float, (byte == 255u ? 0u : 254u - byte) << 23);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // to nearest even, saturated at 6
    const float lo = byte == 255u ? 0.f : x[2 * i] * mul, hi = byte == 255u ? 0.f : x[2 * i + 1] * mul;
    w |= (__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, lo, hi, 1.0f, 0) & 255u) << 8 * i;
  }
  *reinterpret_cast<uint32_t *>(Xq + m * (K / 2) + 4 * (int64_t)c) = w;
  if ((c & 3) == 0) xs[m * (K / 32) + (c >> 2)] = (uint8_t)byte;
}

// ---- product ----------------------------------------------------------------
__device__ __forceinline__ i32x8 operand(u32x4 c) {
  return i32x8{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}
// c + A B^T of one instruction; byte I of the scale words.
template <int I>
__device__ __forceinline__ float4_t mfma(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, float4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), c, 4, 4, I, (int)sa,
                                                          I, (int)sb);
}

// Scales of the blocks [b, b + 4) of a row of `blocks`; past its end 0 (2^-127,
// of codes that are read as 0 there). Rows begin at any byte.
__device__ __forceinline__ uint32_t scales4(const uint8_t *row, int64_t b, int64_t blocks, bool whole) {
  uint32_t w = 0;
  if (whole) {
    __builtin_memcpy(&w, row + b, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < blocks) w |= (uint32_t)row[b + i] << 8 * i;
  }
  return w;
}

// Few rows of X (decode): bound by reading W once. A workgroup takes 16 * TN
// rows of W; its waves share K, wave w taking a contiguous run of pieces of 512,
// and their sums are added in LDS in a fixed order. W and X go straight from
// memory to the operands, DEPTH pieces ahead, in registers.
constexpr int kRowWaves = 8;
constexpr int kPiece = 512;

template <class T, int TM, int TN, int DEPTH>
__global__ void __launch_bounds__(64 * kRowWaves)
gemm_mxfp4_rows_kernel(const uint8_t *__restrict__ W, const uint8_t *__restrict__ sw,
                       const uint8_t *__restrict__ X, const uint8_t *__restrict__ sx,
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
  const int pieces = (int)((K + kPiece - 1) / kPiece);
  const int per = (pieces + kRowWaves - 1) / kRowWaves;
  const int p0 = wave * per, p1 = p0 + per < pieces ? p0 + per : pieces;
  const int64_t blocks = K / 32;
  const uint32_t row_bytes = (uint32_t)(K / 2);

  const int wrows = (int)(N - n0 < kN ? N - n0 : kN);
  const int xrows = (int)(M - m0 < kM ? M - m0 : kM);
  // rows past the ends read zeros
  const rsrc_t wr = make_rsrc(W + n0 * row_bytes, (uint32_t)wrows * row_bytes);
  const rsrc_t xr = make_rsrc(X + m0 * row_bytes, (uint32_t)xrows * row_bytes);
  const uint8_t *swr[TN], *sxr[TM];
#pragma unroll
  for (int j = 0; j < TN; ++j) swr[j] = sw + (n0 + (16 * j + l16 < wrows ? 16 * j + l16 : 0)) * blocks;
#pragma unroll
  for (int i = 0; i < TM; ++i) sxr[i] = sx + (m0 + (16 * i + l16 < xrows ? 16 * i + l16 : 0)) * blocks;

  struct Stage {
    u32x4 w[TN][4], x[TM][4];
    uint32_t sw[TN], sx[TM];
  } st[DEPTH];
  auto load = [&](Stage &s, int p) {
    const bool whole = (int64_t)(p + 1) * kPiece <= K;
    const int64_t b = 16 * (int64_t)p + 4 * g;  // this lane's first block
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // past K the next row begins: those blocks read as zeros
      const bool in = whole || b + t < blocks;
      const uint32_t at = (uint32_t)(16 * (b + t));
#pragma unroll
      for (int j = 0; j < TN; ++j)
        s.w[j][t] = buf_load_b128(wr, in ? (uint32_t)(16 * j + l16) * row_bytes + at : 0x80000000u);
#pragma unroll
      for (int i = 0; i < TM; ++i)
        s.x[i][t] = buf_load_b128(xr, in ? (uint32_t)(16 * i + l16) * row_bytes + at : 0x80000000u);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) s.sw[j] = scales4(swr[j], b, blocks, whole);
#pragma unroll
    for (int i = 0; i < TM; ++i) s.sx[i] = scales4(sxr[i], b, blocks, whole);
  };

  float4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (p0 + d < p1) load(st[d], p0 + d);
  for (int p = p0; p < p1; p += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (p + d >= p1) break;
      Stage &s = st[d];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          acc[i][j] = mfma<0>(s.w[j][0], s.sw[j], s.x[i][0], s.sx[i], acc[i][j]);
          acc[i][j] = mfma<1>(s.w[j][1], s.sw[j], s.x[i][1], s.sx[i], acc[i][j]);
          acc[i][j] = mfma<2>(s.w[j][2], s.sw[j], s.x[i][2], s.sx[i], acc[i][j]);
          acc[i][j] = mfma<3>(s.w[j][3], s.sw[j], s.x[i][3], s.sx[i], acc[i][j]);
        }
      if (p + d + DEPTH < p1) load(s, p + d + DEPTH);
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

template <class T, int TM, int TN, int DEPTH>
hipError_t launch_rows(const uint8_t *W, const uint8_t *sw, const uint8_t *X, const uint8_t *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t tn = (N + 16 * TN - 1) / (16 * TN), tm = (M + 16 * TM - 1) / (16 * TM);
  return launch_in_pieces(tm * tn, 64 * kRowWaves, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((gemm_mxfp4_rows_kernel<T, TM, TN, DEPTH>), dim3(n), dim3(64 * kRowWaves), 0,
                       stream, W, sw, X, sx, static_cast<typename T::elem *>(Y), M, N, K, (uint32_t)tn,
                       first);
  });
}

template <class T>
hipError_t launch_gemm(const uint8_t *W, const uint8_t *sw, const uint8_t *X, const uint8_t *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, int num_cus, hipStream_t stream) {
  if (M <= 16) return launch_rows<T, 1, 1, 2>(W, sw, X, sx, Y, M, N, K, stream);
  return launch_rows<T, 4, 2, 1>(W, sw, X, sx, Y, M, N, K, stream);
}

template <class T>
hipError_t launch_quant(const void *X, int64_t ldx, uint8_t *Xq, uint8_t *xs, int64_t M, int64_t K,
                        hipStream_t stream) {
  const int64_t blocks = (M * (K / 8) + kQuantThreads - 1) / kQuantThreads;
  if (blocks > 0xffffffffll) return hipErrorInvalidValue;
  return launch_in_pieces(blocks, kQuantThreads, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL(quant_mxfp4_kernel<T>, dim3(n), dim3(kQuantThreads), 0, stream,
                       static_cast<const typename T::elem *>(X), ldx, Xq, xs, M, K, first);
  });
}

}  // namespace

hipError_t quant_mxfp4_launch(const void *X, ElemType type, int64_t ldx, uint8_t *Xq, uint8_t *xs,
                              int64_t M, int64_t K, hipStream_t stream) {
  if (type == ElemType::F32) return launch_quant<TypeF32>(X, ldx, Xq, xs, M, K, stream);
  if (type == ElemType::F16) return launch_quant<TypeF16>(X, ldx, Xq, xs, M, K, stream);
  return launch_quant<TypeBF16>(X, ldx, Xq, xs, M, K, stream);
}

hipError_t gemm_mxfp4_launch(const uint8_t *W, const uint8_t *sw, const uint8_t *X, const uint8_t *sx,
                             void *Y, ElemType type, int64_t M, int64_t N, int64_t K, int num_cus,
                             hipStream_t stream) {
  if (type == ElemType::F32) return launch_gemm<TypeF32>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
  if (type == ElemType::F16) return launch_gemm<TypeF16>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
  return launch_gemm<TypeBF16>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
}

}  // namespace lqmm
