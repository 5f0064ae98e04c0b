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
// scale. Which blocks are one instruction is free; a lane takes blocks that
// follow each other for the instructions that follow each other, so that its
// scales are one word, of which each instruction names a byte.
//
// Two kernels. Few rows of X are bound by reading W (1 x 28672 x 8192: 5 TB/s):
// memory to operands, K shared by a workgroup's waves. Many rows by the matrix
// cores: LDS tiles and v_mfma_scale_f32_32x32x64_f8f6f4, which alone reach 7.8
// PFLOP/s where the 16 x 16 x 128 form reaches 4.7 (one wave a SIMD) or 6; on
// random codes, whose power draw lowers the clock, 5.3. 4096 x 14336 x 4096 runs
// at 2.9 to 3.2 PFLOP/s (152 to 163 us, by card; the vendor library 3.0 at
// 8192^3). Of that, measured on timing copies, products 88 us, LDS reads 20, loads
// 30, scales 15, outputs 20: one wave's instructions go out in turn, and the barrier
// of a step puts the two waves of a SIMD in step, so that these overlap in part
// only. From 16 to 1000 rows it stands 1.5 to 5 times above its floor: 19 to 39
// bytes of W and X per ns come into a CU, too few are on their way.
#include <type_traits>

#include "lqmm_internal.hpp"
#include "serve_device.hpp"

namespace lqmm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---- quantization -------------------------------------------------------------
constexpr int kQuantThreads = 256;

// Four lanes take one block, eight values each: reads are 16 (32) bytes a lane
// side by side, codes 4 bytes a lane. 4096 x 4096 bf16 10.3 us (8.2 at the rate
// of a large copy), 45 x 4128 fp32 2.2, one row of 8192 4 to 5: a launch.
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
__device__ __forceinline__ float16_t mfma32(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, float16_t c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, I, (int)sa,
                                                         I, (int)sb);
}
template <int I>
__device__ __forceinline__ float4_t mfma16(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, float4_t c) {
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

// Scales of the 16 blocks from b on of a row of `blocks`; past its end 0 (2^-127,
// of codes that are read as 0 there). Rows begin at any byte.
__device__ __forceinline__ u32x4 scales16(const uint8_t *row, int64_t b, int64_t blocks, bool whole) {
  u32x4 w = {0u, 0u, 0u, 0u};
  if (whole) {
    __builtin_memcpy(&w, row + b, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (b + i < blocks) w[i >> 2] |= (uint32_t)row[b + i] << 8 * (i & 3);
  }
  return w;
}

// Few rows of X (decode): bound by reading W once. A workgroup takes 16 * TN
// rows of W; its waves share K, wave w taking a contiguous run of pieces of 512,
// and their sums are added in LDS in a fixed order. W and X go straight from
// memory to the operands, DEPTH pieces ahead, in registers.
constexpr int kPiece = 512;

template <class T, int TM, int TN, int DEPTH, int NW>
__global__ void __launch_bounds__(64 * NW)
gemm_mxfp4_rows_kernel(const uint8_t *__restrict__ W, const uint8_t *__restrict__ sw,
                       const uint8_t *__restrict__ X, const uint8_t *__restrict__ sx,
                       typename T::elem *__restrict__ Y, int64_t M, int64_t N, int64_t K,
                       uint32_t tiles_n, uint32_t first) {
  constexpr int kN = 16 * TN, kM = 16 * TM, kLd = kN + 4;
  __shared__ __attribute__((aligned(16))) float part[NW][kM][kLd];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const uint32_t block = first + blockIdx.x;
  const int64_t n0 = (int64_t)(block % tiles_n) * kN;
  const int64_t m0 = (int64_t)(block / tiles_n) * kM;
  const int pieces = (int)((K + kPiece - 1) / kPiece);
  const int per = (pieces + NW - 1) / NW;
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
          acc[i][j] = mfma16<0>(s.w[j][0], s.sw[j], s.x[i][0], s.sx[i], acc[i][j]);
          acc[i][j] = mfma16<1>(s.w[j][1], s.sw[j], s.x[i][1], s.sx[i], acc[i][j]);
          acc[i][j] = mfma16<2>(s.w[j][2], s.sw[j], s.x[i][2], s.sx[i], acc[i][j]);
          acc[i][j] = mfma16<3>(s.w[j][3], s.sw[j], s.x[i][3], s.sx[i], acc[i][j]);
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
  for (int o = tid; o < kM * kN; o += 64 * NW) {
    const int m = o / kN, n = o % kN;
    if (m >= xrows || n >= wrows) continue;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) y += part[w][m][n];
    Y[(m0 + m) * N + n0 + n] = (typename T::elem)y;
  }
}

// ---- LDS tiles ------------------------------------------------------------------
constexpr int kStepBytes = 64;  // of a row in a step: 128 of K, four blocks

// Eight outputs of a row, n of which exist; `vec`: their address is a multiple of
// their size. (Rows of an odd N begin at any element; stores of words need no
// alignment, and cost more: 1000 x 9001 x 2048 33 us so, 49 by elements, and 4096 x
// 14336 x 4096 200 us so, 170 by 16 bytes.)
template <class T>
__device__ __forceinline__ void store8_of(typename T::elem *p, const float (&v)[8], int n, bool vec) {
  typedef typename T::elem elem;
  if (vec && n >= 8) {
    if constexpr (T::kBytes == 4) {
      *reinterpret_cast<float4_t *>(p) = float4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<float4_t *>(p + 4) = float4_t{v[4], v[5], v[6], v[7]};
    } else {
      store8<T>(p, v);
    }
    return;
  }
  elem o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (elem)v[i];
  if (n >= 8) {
    __builtin_memcpy(p, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = o[i];
  }
}

// LDS of a tile (codes, and two pieces' scales), and workgroups and waves of a
// SIMD that a CU has room for.
constexpr int tile_lds(int bm, int bn, int ns) { return (bm + bn) * (ns * kStepBytes + 32); }
constexpr int workgroups_of_cu(int bm, int bn, int wm, int wn, int ns) {
  return 2 * tile_lds(bm, bn, ns) <= 160 * 1024 && bm / wm * (bn / wn) <= 64 * 64 ? 2 : 1;
}
constexpr int waves_of_simd(int bm, int bn, int wm, int wn, int ns) {
  return workgroups_of_cu(bm, bn, wm, wn, ns) * wm * wn / 4;
}

// A BM x BN tile (rows of X by rows of W), WM x WN waves, NS LDS stages.
template <int BM, int BN, int WM, int WN, int NS>
struct Tile {
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // 32 x 32 tiles of a wave
  static constexpr int kRows = BM + BN;
  static constexpr int kStage = kRows * kStepBytes;
  static constexpr int kLoads = kRows / 16 / kWaves;          // 1 KB loads of a wave per step
  static constexpr int kScaleLoads = (kRows + kThreads - 1) / kThreads;
  static constexpr int kLds = tile_lds(BM, BN, NS);
  static constexpr int kPerCu = workgroups_of_cu(BM, BN, WM, WN, NS);
};

template <class T, int BM, int BN, int WM, int WN, int NS>
__global__ void __launch_bounds__(64 * WM * WN, waves_of_simd(BM, BN, WM, WN, NS))
gemm_mxfp4_kernel(const uint8_t *__restrict__ W, const uint8_t *__restrict__ sw,
                  const uint8_t *__restrict__ X, const uint8_t *__restrict__ sx,
                  typename T::elem *__restrict__ Y, int64_t M, int64_t N, int64_t K, uint32_t tiles_m,
                  uint32_t tiles_n) {
  typedef Tile<BM, BN, WM, WN, NS> C;
  constexpr int TM = C::TM, TN = C::TN, kHalf = C::kLoads / 2;
  static_assert(C::kRows % (16 * C::kWaves) == 0 && BM / 16 % C::kLoads == 0 && NS >= 3, "tile");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
  const uint32_t row_bytes = (uint32_t)(K / 2);
  const int64_t blocks = K / 32;
  const int steps = (int)((K + 255) / 256) * 2;  // (past K of zeros)

  // Workgroups stay, one or two for each CU, and take one tile after the other;
  // the next tile's first stages are on their way while the last one's outputs
  // are written. Workgroups go to the 8 XCDs in turn; an XCD's tiles follow each
  // other in blocks four wide in N, so that what its CUs read at a time, 8 x 4
  // tiles, shares rows of X and of W in its L2.
  const uint32_t tiles = tiles_m * tiles_n, wgs = gridDim.x;
  const uint32_t xcd = blockIdx.x % 8, q8 = tiles / 8, r8 = tiles % 8;
  const uint32_t first = xcd * q8 + (xcd < r8 ? xcd : r8), end = first + q8 + (xcd < r8 ? 1 : 0);
  const uint32_t stride = wgs / 8 + (xcd < wgs % 8 ? 1 : 0);
  struct Place {
    int64_t m0, n0;
  };
  auto place = [&](uint32_t tile) {
    const uint32_t panel = tile / (4 * tiles_m), in = tile - panel * (4 * tiles_m);
    const uint32_t wide = tiles_n - 4 * panel < 4 ? tiles_n - 4 * panel : 4;
    return Place{(int64_t)(in / wide) * BM, (int64_t)(4 * panel + in % wide) * BN};
  };

  // Tile rows of 64 bytes; 16-byte chunk c of row r stands in slot
  // c ^ (r / 2 % 4), so that the eight rows that one phase of a 16-byte LDS read
  // touches lie in different banks. A load fills 16 rows, lane by lane.
  const int lrow = lane >> 2, lcol = 16 * ((lane & 3) ^ (lrow >> 1 & 3));
  // What a wave loads next: kLoads times 16 rows of X or of W, of a step of a
  // tile, into stage `to`; and of the tile after it.
  const bool of_x = wave * C::kLoads < BM / 16;
  const int row0 = 16 * C::kLoads * wave - (of_x ? 0 : BM);
  uint32_t offset[C::kLoads];
#pragma unroll
  for (int i = 0; i < C::kLoads; ++i) offset[i] = (uint32_t)(row0 + 16 * i + lrow) * row_bytes + lcol;
  struct Rows {
    const uint8_t *at;
    uint32_t bytes;
  };
  auto rows_of = [&](uint32_t tile) {
    const Place p = place(tile < end ? tile : first);
    const int64_t m = M - p.m0 < BM ? M - p.m0 : BM, n = N - p.n0 < BN ? N - p.n0 : BN;
    return Rows{of_x ? X + p.m0 * row_bytes : W + p.n0 * row_bytes,
                tile < end ? (uint32_t)(of_x ? m : n) * row_bytes : 0};  // (behind the last tile: zeros)
  };
  struct {
    Rows rows, after;
    uint32_t tile;  // that `after` belongs to
    int kt, to;
  } ahead;
  auto issue = [&](int from, int to) {  // half of a step's loads
    uint8_t *st = smem + ahead.to * C::kStage + wave * (C::kLoads * 1024);
    const int kt = ahead.kt;
    const rsrc_t r = make_rsrc(ahead.rows.at, ahead.rows.bytes);
    // past K the rows of the next line begin: those chunks read as zeros
    // (an offset past the resource)
    const bool in = (uint32_t)(ahead.kt * kStepBytes + lcol) < row_bytes;
#pragma unroll
    for (int i = from; i < to; ++i) {
      const int off = in ? (int)offset[i] : (int)0x80000000u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, st + i * 1024, 16, off, kt * kStepBytes, 0, 0);
    }
  };
  auto advance = [&]() {  // (no branch: it stands between products)
    const bool over = ahead.kt + 1 == steps;
    ahead.kt = over ? 0 : ahead.kt + 1;
    ahead.to = ahead.to + 1 < NS ? ahead.to + 1 : 0;
    ahead.rows.at = over ? ahead.after.at : ahead.rows.at;
    ahead.rows.bytes = over ? ahead.after.bytes : ahead.rows.bytes;
  };
  auto look_ahead = [&]() {
    if (ahead.kt != 0) return;
    ahead.tile += stride;
    ahead.after = rows_of(ahead.tile);
  };
  // Scales: a thread brings a row's 16 bytes of a piece of 512, four steps,
  // through registers (rows of scales begin at any byte, and end inside a
  // piece). The last piece of a tile has two steps or four.
  struct {
    uint32_t tile;
    int piece, to;
    const uint8_t *row[C::kScaleLoads];
    u32x4 reg[C::kScaleLoads];
  } scales;
  auto scales_at_tile = [&](uint32_t tile) {
    scales.tile = tile;
    scales.piece = 0;
    const Place p = place(tile < end ? tile : first);
#pragma unroll
    for (int i = 0; i < C::kScaleLoads; ++i) {
      const int r = tid + i * C::kThreads;
      const int64_t mr = p.m0 + r < M ? p.m0 + r : M - 1, nr = p.n0 + r - BM < N ? p.n0 + r - BM : N - 1;
      scales.row[i] = r < BM ? sx + mr * blocks : sw + nr * blocks;
    }
  };
  auto load_scales = [&]() {
    if (scales.tile >= end || 16 * (int64_t)(scales.piece + 1) > blocks) return;
#pragma unroll
    for (int i = 0; i < C::kScaleLoads; ++i)
      __builtin_memcpy(&scales.reg[i], scales.row[i] + 16 * (int64_t)scales.piece, 16);
  };
  auto store_scales = [&]() {
    const int64_t at = 16 * (int64_t)scales.piece;
    uint8_t *st = smem + NS * C::kStage + scales.to * (C::kRows * 16);
#pragma unroll
    for (int i = 0; i < C::kScaleLoads; ++i) {
      const int r = tid + i * C::kThreads;
      if (C::kRows % C::kThreads != 0 && r >= C::kRows) continue;
      if (at + 16 <= blocks) {
        *reinterpret_cast<u32x4 *>(st + r * 16) = scales.reg[i];
      } else {  // a row's end: byte by byte, not through the registers ahead
        *reinterpret_cast<u32x4 *>(st + r * 16) = scales16(scales.row[i], at, blocks, false);
      }
    }
    scales.to ^= 1;
    if (++scales.piece == (steps + 3) / 4) scales_at_tile(scales.tile + stride);
  };
  // A lane's operand of instruction t of a step is block 2 h + t of its row.
  struct Operands {
    u32x4 x[TM], w[TN];
  } f[2];
  auto read = [&](Operands &o, int stage, int t) {
    const uint8_t *xst = smem + stage * C::kStage, *wst = xst + BM * kStepBytes;
    auto frag = [&](const uint8_t *base, int row) {
      return *reinterpret_cast<const u32x4 *>(base + row * kStepBytes + 16 * ((2 * h + t) ^ (row >> 1 & 3)));
    };
#pragma unroll
    for (int j = 0; j < TN; ++j) o.w[j] = frag(wst, wn + 32 * j + l32);
#pragma unroll
    for (int i = 0; i < TM; ++i) o.x[i] = frag(xst, wm + 32 * i + l32);
  };
  struct Scales {
    uint32_t x[TM], w[TN];
  } now, next;
  auto read_scales = [&](Scales &o, int piece, int step) {
    const uint8_t *st = smem + NS * C::kStage + piece * (C::kRows * 16) + 4 * step + 2 * h;
#pragma unroll
    for (int j = 0; j < TN; ++j) o.w[j] = *reinterpret_cast<const uint16_t *>(st + 16 * (BM + wn + 32 * j + l32));
#pragma unroll
    for (int i = 0; i < TM; ++i) o.x[i] = *reinterpret_cast<const uint16_t *>(st + 16 * (wm + 32 * i + l32));
  };

  float16_t acc[TM][TN];
  // A step is two instructions for each 32 x 32 tile; while the matrix cores
  // work on one, the next one's operands are read and half a step's loads go
  // out. Between the two, every wave has read what it needs of the step's stage,
  // which is filled again, and the next step's stage is complete.
  uint32_t tile = first + blockIdx.x / 8;
  if (tile >= end) return;
  ahead.to = scales.to = 0;
  ahead.kt = 0;
  ahead.rows = rows_of(tile);
  ahead.tile = tile;
  look_ahead();
  scales_at_tile(tile);
  load_scales();
  store_scales();
  load_scales();
#pragma unroll
  for (int d = 0; d < NS; ++d) {
    issue(0, kHalf);
    if (d == NS - 1) break;
    issue(kHalf, C::kLoads);
    advance();
    look_ahead();
  }
  wait_loads_and_barrier<(NS - 2) * C::kLoads + kHalf>();
  read_scales(now, 0, 0);
  read(f[0], 0, 0);
  constexpr int kReads = TM + TN;
  auto products = [&](auto byte, const Operands &o, const Scales &s) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma32<decltype(byte)::value>(o.w[j], s.w[j], o.x[i], s.x[i], acc[i][j]);
  };
  // Products have no effect but their sums, and the compiler moves them down to
  // where these are used, behind barriers and branches: named here they stay.
  auto stay = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" ::"v"(acc[i][j][0]));
  };
  // kR LDS reads and a half step's loads between the products
  auto mixed = [&](auto reads) {
    constexpr int kR = decltype(reads)::value, kM = TM * TN;
#pragma unroll
    for (int i = 0; i < kM; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * ((kR + kM - 1) / kM), 0);
      if (i >= kM / 2) __builtin_amdgcn_sched_group_barrier(0x20, (2 * (C::kLoads - kHalf) + kM - 1) / kM, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int stage = 0, piece = 0;
  const bool vec = N % 8 == 0;
  for (; tile < end; tile += stride) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    for (int kt = 0; kt < steps; ++kt) {
      const int after = kt + 1 < steps ? (kt + 1) & 3 : 0;
      const int stage1 = stage + 1 < NS ? stage + 1 : 0, piece1 = piece ^ (after == 0);
      __builtin_amdgcn_sched_barrier(0);
      read(f[1], stage, 1);
      products(std::integral_constant<int, 0>(), f[0], now);
      issue(kHalf, C::kLoads);
      mixed(std::integral_constant<int, kReads>());
      stay();
      wait_loads_and_barrier<(NS - 2) * C::kLoads>();
      __builtin_amdgcn_sched_barrier(0);
      read_scales(next, piece1, after);
      read(f[0], stage1, 0);
      products(std::integral_constant<int, 1>(), f[1], now);
      advance();
      issue(0, kHalf);
      mixed(std::integral_constant<int, 2 * kReads>());
      stay();
      now = next;
      stage = stage1;
      piece = piece1;
      look_ahead();
      if ((kt & 3) == 0) {
        store_scales();
        load_scales();
      }
    }
    const Place p = place(tile);
    const int64_t rows = M - p.m0 - wm - l32, cols = N - p.n0 - wn;
    typename T::elem *y = Y + (p.m0 + wm + l32) * N + p.n0 + wn;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (32 * i >= rows) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 8) {
          // a lane has columns 2 r + 4 h .. + 3 and 2 r + 8 + 4 h .. + 3 of 32: the halves
          // of the wave exchange four, for eight next to each other
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = acc[i][j][r + e], hi = acc[i][j][r + 4 + e];
            const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, lo),
                                                            __builtin_bit_cast(uint32_t, hi), false, false);
            const uint32_t s0 = s[0], s1 = s[1];
            v[e] = __builtin_bit_cast(float, s0), v[4 + e] = __builtin_bit_cast(float, s1);
          }
          const int n = 32 * j + 2 * r + 8 * h;
          if (n < cols)
            store8_of<T>(y + 32 * i * N + n, v, (int)(cols - n < 8 ? cols - n : 8), vec);
        }
    }
  }
  wait_loads_and_barrier<0>();  // (LDS is not written behind the kernel's end)
}

template <class T, int BM, int BN, int WM, int WN, int NS>
hipError_t launch_tile(const uint8_t *W, const uint8_t *sw, const uint8_t *X, const uint8_t *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, int num_cus, hipStream_t stream) {
  typedef Tile<BM, BN, WM, WN, NS> C;
  constexpr auto kern = gemm_mxfp4_kernel<T, BM, BN, WM, WN, NS>;
  const int64_t tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN, tiles = tm * tn;
  const hipError_t e = ensure_max_lds<kern>(C::kLds);
  if (e != hipSuccess) return e;
  const int64_t most = (int64_t)num_cus * C::kPerCu;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles < most ? tiles : most)), dim3(C::kThreads), C::kLds, stream,
                     W, sw, X, sx, static_cast<typename T::elem *>(Y), M, N, K, (uint32_t)tm, (uint32_t)tn);
  return hipGetLastError();
}

template <class T, int TM, int TN, int DEPTH, int NW>
hipError_t launch_rows(const uint8_t *W, const uint8_t *sw, const uint8_t *X, const uint8_t *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t tn = (N + 16 * TN - 1) / (16 * TN), tm = (M + 16 * TM - 1) / (16 * TM);
  return launch_in_pieces(tm * tn, 64 * NW, [&](uint32_t first, unsigned n) {
    hipLaunchKernelGGL((gemm_mxfp4_rows_kernel<T, TM, TN, DEPTH, NW>), dim3(n), dim3(64 * NW), 0,
                       stream, W, sw, X, sx, static_cast<typename T::elem *>(Y), M, N, K, (uint32_t)tn,
                       first);
  });
}

template <class T>
hipError_t launch_gemm(const uint8_t *W, const uint8_t *sw, const uint8_t *X, const uint8_t *sx, void *Y,
                       int64_t M, int64_t N, int64_t K, int num_cus, hipStream_t stream) {
  if (M <= 16) return launch_rows<T, 1, 1, 1, 8>(W, sw, X, sx, Y, M, N, K, stream);
  // The kernel and tile whose estimated time is least: rounds over the CUs times
  // what a round takes, a fixed part and one for each 512 of K (ns). The parts
  // were fitted to times at M = 1 .. 4096, N = 1024 .. 28672, K = 1056 .. 8192;
  // e.g. (us, 16 x 16 rows / 32 x 32 rows / 48 x 32 rows / 64 x 64 / 128 x 128 /
  // 256 x 256 tiles): 16 x 28672 x 8192 37 / 46 / 48 / 40 / 38 / 55; 45 x 4127 x
  // 4128 8.5 / 10.1 / 7.6 / 15.8 / 21.7 / 35; 64 x 4096 x 4096 11.3 / 7.2 / 8.6 /
  // 13.0 / 17.0 / 30; 128 x 14336 x 4096 65 / 42 / 43 / 19.0 / 19.3 / 31; 512 x
  // 14336 x 4096 245 / 163 / 145 / 57 / 36 / 38; 4096 x 14336 x 4096 - / - / - /
  // 394 / 239 / 167. 64 x 32 rows are for what then fits one round: 64 x 6144 x 4096
  // 10.4 (32 x 32: 12.4), 64 x 14336 x 4096 20 (64 x 64: 14).
  struct Choice {
    int bm, bn, per_cu, fixed, piece;
  };
  constexpr Choice kChoices[] = {
      // straight to registers, K shared by eight waves
      {16, 16, 2, 100, 520}, {32, 32, 1, 1000, 600}, {48, 32, 1, 1400, 700}, {64, 32, 1, 2600, 970},
      // LDS tiles: alone on a CU, or two on it
      {64, 64, 1, 3500, 1100}, {64, 64, 2, 4500, 1500}, {128, 128, 1, 3500, 1800}, {128, 128, 2, 1000, 4300},
      {256, 256, 1, 6000, 4350}};
  int best = -1;
  int64_t best_cost = 0;
  for (int c = 0; c < 9; ++c) {
    const Choice &o = kChoices[c];
    const int64_t tiles = ((M + o.bm - 1) / o.bm) * ((N + o.bn - 1) / o.bn);
    const int64_t slots = (int64_t)o.per_cu * num_cus;
    if (tiles > 0x7fffffffll) continue;  // (they are numbered in 32 bits)
    const int64_t cost = (tiles + slots - 1) / slots * (o.fixed + o.piece * K / kPiece);
    if (best < 0 || cost < best_cost) {
      best = c;
      best_cost = cost;
    }
  }
  switch (best) {
    case 0: return launch_rows<T, 1, 1, 1, 8>(W, sw, X, sx, Y, M, N, K, stream);
    case 1: return launch_rows<T, 2, 2, 1, 8>(W, sw, X, sx, Y, M, N, K, stream);
    case 2: return launch_rows<T, 3, 2, 1, 8>(W, sw, X, sx, Y, M, N, K, stream);
    case 3: return launch_rows<T, 4, 2, 1, 8>(W, sw, X, sx, Y, M, N, K, stream);
    case 4:
    case 5: return launch_tile<T, 64, 64, 2, 2, 4>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
    case 6:
    case 7: return launch_tile<T, 128, 128, 2, 4, 4>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
    case 8: return launch_tile<T, 256, 256, 4, 2, 4>(W, sw, X, sx, Y, M, N, K, num_cus, stream);
  }
  return hipErrorInvalidValue;
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
