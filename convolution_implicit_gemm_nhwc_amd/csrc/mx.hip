// MXFP4 on gfx950 (CDNA4): quantisation, its inverse, the product of two
// quantised matrices, and their C ABI (include/fconv_mx.h).
//
//   y[m, n] = act( sum_k X[m, k] W[n, k] + bias[n] )
//
// X and W are e2m1 codes with one power-of-two scale per 32 values of a row.
// The scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 takes, per
// lane, 32 codes (16 bytes) of one row and the scale byte of that block, so a
// block's scale costs no arithmetic.  A quantised matrix is stored in exactly
// that order (16-row x 128-column tiles of 1 KiB, a lane's 16 bytes at 16 *
// lane; a lane's scale bytes of four consecutive k tiles in one dword, picked
// by the instruction's byte select), so every copy and every fragment read
// below is linear: no swizzle, no LDS bank conflicts, no shuffles.
//
// The matrix core's A operand is W and its B operand X: a lane then ends with
// four consecutive n of one row m, one store.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>
#include <type_traits>

#include "fconv_mx.h"

struct fconv_mx_plan_s {
  fconv_mx_desc d;
  int32_t esize;    // bytes per x / y element
  bool op_bias;
  int32_t act;      // 0 none, 1 ReLU, 2 leaky, 3 clipped, 4 clamp
  int32_t kt;       // 128-column k tiles
  int32_t tile;     // output tile edge of the tiled kernel (256 or 128)
  size_t ws_x;      // bytes of the quantised x in the workspace
  size_t ws_bytes;
  const char* kernel_name;
};

namespace fconv {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kOutOfRange = 0x80000000u;  // buffer offset past every extent: reads 0
constexpr int kBufferDword3 = 0x00020000;      // raw buffer descriptor, gfx9 family
constexpr int kTileBytes = 1024;               // codes of 16 rows x 128 columns
constexpr int kScaleTile = 256;                // scales of 16 rows x 512 columns
// Workgroups of a launch: its threads stay below 2^32.
constexpr int64_t kMaxGroups = (1 << 23) - 8;
constexpr int32_t kMaxK = 1 << 22;             // 256 rows of codes stay below 2^31 bytes

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Codes and scales of one quantised matrix.
struct MxView {
  const char* codes;
  const char* scales;
  int64_t row_tiles;
};

size_t codes_bytes(int64_t rows, int64_t cols) {
  return static_cast<size_t>(ceil_div(rows, 16) * ceil_div(cols, 128)) * kTileBytes;
}
size_t scales_bytes(int64_t rows, int64_t cols) {
  return static_cast<size_t>(ceil_div(rows, 16) * ceil_div(cols, 512)) * kScaleTile;
}
MxView view(const void* mx, int64_t rows, int64_t cols) {
  const char* c = static_cast<const char*>(mx);
  return MxView{c, c + codes_bytes(rows, cols), ceil_div(rows, 16)};
}

__device__ inline __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const uint32_t n = bytes > 0x7fffffff ? 0x7fffffffu : static_cast<uint32_t>(bytes < 0 ? 0 : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(n), kBufferDword3);
}

__device__ inline float bf16_to_f32(uint16_t v) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
}
__device__ inline uint16_t f32_to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));  // round to nearest even
}

// Eight values of a row at column c, zeros past `cols` (n < 8 live ones at
// the tail).  gfx950 reads global memory at any byte alignment.
template <bool BF16>
__device__ inline void load8(const char* p, int n, float v[8]) {
  if constexpr (BF16) {
    if (n >= 8) {
      uint16_t h[8];
      __builtin_memcpy(h, p, 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bf16_to_f32(h[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint16_t h = 0;
        if (i < n) __builtin_memcpy(&h, p + 2 * i, 2);
        v[i] = bf16_to_f32(h);
      }
    }
  } else {
    if (n >= 8) {
      __builtin_memcpy(v, p, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0.0f;
        if (i < n) __builtin_memcpy(&v[i], p + 4 * i, 4);
      }
    }
  }
}

// Scale byte of a block whose largest magnitude has the bits `m`: the
// exponent field less 2 (e2m1's largest exponent), at least 0.  An infinity
// or NaN (exponent field 255) gives 255.
__device__ inline uint32_t scale_byte(uint32_t m) {
  const uint32_t e = m >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// Eight codes: x * 2^-e is exact (a power of two; what underflows is far
// below the smallest code), then the hardware conversion rounds to nearest
// even and saturates at 6.
__device__ inline uint32_t encode8(const float v[8], uint32_t byte) {
  if (byte == 255u) return 0u;
  const float inv = __builtin_bit_cast(float, (254u - byte) << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.0f, 3);
  return c;
}

__device__ inline uint32_t abs_bits(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7fffffffu; }

// Largest of the four lanes of a quad.
__device__ inline uint32_t quad_max(uint32_t m) {
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xB1, 0xf, 0xf, true)));
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4E, 0xf, 0xf, true)));
  return m;
}

// Quantisation.  One workgroup per 16 rows x 512 columns, one wave per k tile
// of 128 columns: 16 lanes read a row's 128 values (8 each), four rows at a
// time, four loads in flight per lane; the four lanes of a block agree on its
// largest magnitude.  The scale bytes of the four k tiles meet in LDS so that
// a lane's four bytes leave as one dword.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const char* x, int64_t ldx_bytes,
                                                          int64_t rows, int cols, int kt_n, int ks_n,
                                                          char* codes, char* scales) {
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ uint8_t sc[kScaleTile];
  const int64_t rt = blockIdx.x / ks_n;
  const int ks = static_cast<int>(blockIdx.x - rt * ks_n);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kt = 4 * ks + wave;
  const int c = kt * 128 + (lane & 15) * 8;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = rt * 16 + 4 * i + (lane >> 4);
    if (r < rows && c < cols) {
      load8<BF16>(x + r * ldx_bytes + static_cast<int64_t>(c) * ES, cols - c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
    const uint32_t byte = scale_byte(quad_max(m));
    const int row = 4 * i + (lane >> 4), blk = (lane & 15) >> 2;
    if (kt < kt_n) {
      const uint32_t code = encode8(v[i], byte);
      *reinterpret_cast<uint32_t*>(codes + (rt * kt_n + kt) * kTileBytes + (blk * 16 + row) * 16 +
                                   (lane & 3) * 4) = code;
    }
    if ((lane & 3) == 0) sc[(blk * 16 + row) * 4 + wave] = static_cast<uint8_t>(byte);
  }
  __syncthreads();
  if (wave == 0)
    reinterpret_cast<uint32_t*>(scales + (rt * ks_n + ks) * kScaleTile)[lane] =
        reinterpret_cast<const uint32_t*>(sc)[lane];
}

// The values that codes and scales stand for: the quantisation's work split
// backwards, a lane writing 8 values.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const char* codes, const char* scales,
                                                            int64_t rows, int cols, int kt_n,
                                                            int ks_n, char* y, int64_t ldy_bytes) {
  constexpr int ES = BF16 ? 2 : 4;
  const int64_t rt = blockIdx.x / ks_n;
  const int ks = static_cast<int>(blockIdx.x - rt * ks_n);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kt = 4 * ks + wave;
  const int c = kt * 128 + (lane & 15) * 8;
  if (kt >= kt_n || c >= cols) return;
  uint32_t code[4], byte[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * i + (lane >> 4), blk = (lane & 15) >> 2;
    code[i] = *reinterpret_cast<const uint32_t*>(codes + (rt * kt_n + kt) * kTileBytes +
                                                 (blk * 16 + row) * 16 + (lane & 3) * 4);
    byte[i] = static_cast<uint8_t>(scales[(rt * ks_n + ks) * kScaleTile + (blk * 16 + row) * 4 + wave]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = rt * 16 + 4 * i + (lane >> 4);
    if (r >= rows) continue;
    const uint32_t b = byte[i];
    const float s = b == 255u ? __builtin_nanf("")
                              : __builtin_bit_cast(float, b ? b << 23 : 0x00400000u);
    float v[8];
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 0);
    const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 2);
    const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 3);
    v[0] = p0.x * s; v[1] = p0.y * s; v[2] = p1.x * s; v[3] = p1.y * s;
    v[4] = p2.x * s; v[5] = p2.y * s; v[6] = p3.x * s; v[7] = p3.y * s;
    char* p = y + r * ldy_bytes + static_cast<int64_t>(c) * ES;
    const int n = cols - c;
    if constexpr (BF16) {
      uint16_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = f32_to_bf16(v[j]);
      if (n >= 8) {
        __builtin_memcpy(p, h, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) __builtin_memcpy(p + 2 * j, &h[j], 2);
      }
    } else {
      if (n >= 8) {
        __builtin_memcpy(p, v, 32);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) __builtin_memcpy(p + 4 * j, &v[j], 4);
      }
    }
  }
}

// Plain row-major codes and scales into the tile order; a lane moves one
// block's four bytes of codes.  Runs once per weight.
__global__ __launch_bounds__(256) void mx_layout_kernel(const char* src, const uint8_t* src_scales,
                                                        int64_t rows, int cols, int kt_n, int ks_n,
                                                        char* codes, char* scales) {
  __shared__ uint8_t sc[kScaleTile];
  const int64_t rt = blockIdx.x / ks_n;
  const int ks = static_cast<int>(blockIdx.x - rt * ks_n);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kt = 4 * ks + wave;
  const int nb = (cols + 31) / 32;
  const int b = kt * 4 + ((lane & 15) >> 2);  // block of the row
  const int c = kt * 128 + (lane & 15) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * i + (lane >> 4), blk = (lane & 15) >> 2;
    const int64_t r = rt * 16 + row;
    uint32_t code = 0;
    uint8_t byte = 0;
    if (r < rows && b < nb) {
      __builtin_memcpy(&code, src + (r * nb + b) * 16 + (lane & 3) * 4, 4);
      byte = src_scales[r * nb + b];
      if (cols - c < 8) code &= cols > c ? (1u << (4 * (cols - c))) - 1u : 0u;
    }
    if (kt < kt_n)
      *reinterpret_cast<uint32_t*>(codes + (rt * kt_n + kt) * kTileBytes + (blk * 16 + row) * 16 +
                                   (lane & 3) * 4) = code;
    if ((lane & 3) == 0) sc[(blk * 16 + row) * 4 + wave] = byte;
  }
  __syncthreads();
  if (wave == 0)
    reinterpret_cast<uint32_t*>(scales + (rt * ks_n + ks) * kScaleTile)[lane] =
        reinterpret_cast<const uint32_t*>(sc)[lane];
}

struct MxArgs {
  MxView w, x;
  const float* bias;
  char* y;
  int64_t ldy_bytes;
  int32_t M, N, kt, ks;  // k tiles of 128, scale tiles of 512
  int32_t tiles_m, tiles_n;
  int32_t act;
  float act_alpha, act_beta;
};

// The float epilogue of the convolution plans; a NaN stays a NaN.
__device__ inline float activate(float t, int act, float alpha, float beta) {
  switch (act) {  // uniform
    case 1: return t < 0.0f ? 0.0f : t;
    case 2: return t > 0.0f ? t : alpha * t;
    case 3: return t < 0.0f ? 0.0f : t > alpha ? alpha : t;
    case 4: return t < alpha ? alpha : t > beta ? beta : t;
  }
  return t;
}

// Four consecutive n of row m.
template <bool BF16>
__device__ inline void store4(const MxArgs& a, int64_t m, int n, f32x4 t) {
  if (m >= a.M || n >= a.N) return;
  char* p = a.y + m * a.ldy_bytes + static_cast<int64_t>(n) * (BF16 ? 2 : 4);
  const int live = a.N - n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a.bias && i < live) t[i] += a.bias[n + i];
    t[i] = activate(t[i], a.act, a.act_alpha, a.act_beta);
  }
  if constexpr (BF16) {
    uint16_t h[4] = {f32_to_bf16(t[0]), f32_to_bf16(t[1]), f32_to_bf16(t[2]), f32_to_bf16(t[3])};
    if (live >= 4) {
      __builtin_memcpy(p, h, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < live) __builtin_memcpy(p + 2 * i, &h[i], 2);
    }
  } else {
    if (live >= 4) {
      __builtin_memcpy(p, &t, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < live) {
          const float v = t[i];
          __builtin_memcpy(p + 4 * i, &v, 4);
        }
    }
  }
}

// acc += A B over one k tile: 16 rows of W, 16 rows of X; SEL picks the
// scale bytes of this k tile.
template <int SEL>
__device__ inline f32x4 mma(i32x4 w, i32x4 x, f32x4 acc, int ws, int xs) {
  const i32x8 w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 x8 = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  // Formats 4: e2m1 on both sides.
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, acc, 4, 4, SEL, ws, SEL, xs);
}

// Tiled product.  A workgroup owns (16 WA TA) n x (16 WB TB) m, a wave TA x TB
// matrix tiles.  A stage is two k tiles (256 columns) of every row tile of the
// workgroup, copied buffer->LDS into one of two buffers while the other is
// consumed; the scales of two stages (four k tiles) are copied together.
template <bool BF16, int WA, int WB, int TA, int TB>
__global__ __launch_bounds__(WA* WB * 64) void mx_tile_kernel(MxArgs a) {
  constexpr int NW = WA * WB;
  constexpr int RA = WA * TA, RB = WB * TB;  // row tiles of W and of X
  constexpr int SB = (RA + RB) * 2 * kTileBytes;
  constexpr int CW = (RA + RB) * 2 / NW;     // copies per wave and stage
  static_assert((RA + RB) == 4 * NW && RA % 4 == 0, "one scale copy per wave, all W or all X");
  __shared__ __attribute__((aligned(1024))) char buf0[SB];
  __shared__ __attribute__((aligned(1024))) char buf1[SB];
  __shared__ __attribute__((aligned(1024))) char sc0[(RA + RB) * kScaleTile];
  __shared__ __attribute__((aligned(1024))) char sc1[(RA + RB) * kScaleTile];

  // Workgroups of one XCD (block ids go round the 8 XCDs) take neighbouring
  // tiles: eight tile rows of m together, so both panels stay in its L2.
  const int tiles = a.tiles_m * a.tiles_n;
  const int nb = gridDim.x;  // a multiple of 8
  const int id = (blockIdx.x % 8) * (nb / 8) + blockIdx.x / 8;
  if (id >= tiles) return;
  const int per = 8 * a.tiles_n;
  const int m_first = id / per * 8;
  const int m_rows = min(8, a.tiles_m - m_first);
  const int in = id % per;
  const int tm = m_first + in % m_rows, tn = in / m_rows;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave % WA, wb = wave / WA;
  const int64_t rtw = static_cast<int64_t>(tn) * RA, rtx = static_cast<int64_t>(tm) * RB;
  const int64_t row_bytes = static_cast<int64_t>(a.kt) * kTileBytes;
  const int64_t srow_bytes = static_cast<int64_t>(a.ks) * kScaleTile;
  const auto wr = make_rsrc(a.w.codes + rtw * row_bytes, (a.w.row_tiles - rtw) * row_bytes);
  const auto xr = make_rsrc(a.x.codes + rtx * row_bytes, (a.x.row_tiles - rtx) * row_bytes);
  const bool swave = 4 * wave < RA;  // this wave copies scales of W, else of X
  const auto sr = swave ? make_rsrc(a.w.scales + rtw * srow_bytes, (a.w.row_tiles - rtw) * srow_bytes)
                        : make_rsrc(a.x.scales + rtx * srow_bytes, (a.x.row_tiles - rtx) * srow_bytes);
  const uint32_t s_off = static_cast<uint32_t>((4 * wave - (swave ? 0 : RA) + (lane >> 4)) * srow_bytes +
                                               (lane & 15) * 16);

  auto copy_codes = [&](int st, char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      const int c = wave + NW * i;
      const int rt = c >> 1, kt = 2 * st + (c & 1);
      uint32_t off = kOutOfRange;
      if (kt < a.kt)
        off = static_cast<uint32_t>(((rt < RA ? rt : rt - RA) * a.kt + kt) * kTileBytes + lane * 16);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rt < RA ? wr : xr, (lds_ptr_t)(buf + c * kTileBytes), 16,
                                               off, 0, 0, 0);
    }
  };
  auto copy_scales = [&](int ks, char* buf) __attribute__((always_inline)) {
    const uint32_t off = ks < a.ks ? s_off + static_cast<uint32_t>(ks) * kScaleTile : kOutOfRange;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (lds_ptr_t)(buf + wave * 1024), 16, off, 0, 0, 0);
  };

  f32x4 acc[TA][TB];
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  int sa[TA], sb[TB];

  auto read_scales = [&](const char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TA; ++i)
      sa[i] = *reinterpret_cast<const int*>(buf + (wa * TA + i) * kScaleTile + lane * 4);
#pragma unroll
    for (int j = 0; j < TB; ++j)
      sb[j] = *reinterpret_cast<const int*>(buf + (RA + wb * TB + j) * kScaleTile + lane * 4);
  };
  auto half = [&](const char* buf, auto sel, int kk) __attribute__((always_inline)) {
    i32x4 fa[TA], fb[TB];
#pragma unroll
    for (int i = 0; i < TA; ++i)
      fa[i] = *reinterpret_cast<const i32x4*>(buf + ((wa * TA + i) * 2 + kk) * kTileBytes + lane * 16);
#pragma unroll
    for (int j = 0; j < TB; ++j)
      fb[j] = *reinterpret_cast<const i32x4*>(buf + ((RA + wb * TB + j) * 2 + kk) * kTileBytes + lane * 16);
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) acc[i][j] = mma<decltype(sel)::value>(fa[i], fb[j], acc[i][j], sa[i], sb[j]);
  };
  // Every copy of the stage has landed, for every wave, and every wave has
  // consumed the other buffer.
  auto meet = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int nst = (a.kt + 1) / 2;  // stages
  auto pair = [&](int st, const char* sc, char* sc_next) __attribute__((always_inline)) {
    meet();
    copy_codes(st + 1, buf1);  // past the last stage: zeros, never read
    copy_scales(st / 2 + 1, sc_next);
    read_scales(sc);
    half(buf0, std::integral_constant<int, 0>{}, 0);
    half(buf0, std::integral_constant<int, 1>{}, 1);
    if (st + 1 < nst) {
      meet();
      copy_codes(st + 2, buf0);
      half(buf1, std::integral_constant<int, 2>{}, 0);
      half(buf1, std::integral_constant<int, 3>{}, 1);
    }
  };
  copy_codes(0, buf0);
  copy_scales(0, sc0);
  for (int st = 0; st < nst; st += 4) {
    pair(st, sc0, sc1);
    if (st + 2 < nst) pair(st + 2, sc1, sc0);
  }
  __builtin_amdgcn_s_waitcnt(0);  // copies past the last stage land before exit

  const int g = lane >> 4, r = lane & 15;
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int64_t m = (rtx + wb * TB + j) * 16 + r;
#pragma unroll
    for (int i = 0; i < TA; ++i)
      store4<BF16>(a, m, static_cast<int>((rtw + wa * TA + i) * 16 + 4 * g), acc[i][j]);
  }
}

template <bool BF16>
hipError_t launch_tiles(const fconv_mx_plan_s* p, MxArgs a, hipStream_t s) {
  a.tiles_m = static_cast<int32_t>(ceil_div(a.M, p->tile));
  a.tiles_n = static_cast<int32_t>(ceil_div(a.N, p->tile));
  const int grid = static_cast<int>(ceil_div(static_cast<int64_t>(a.tiles_m) * a.tiles_n, 8) * 8);
  if (p->tile == 256)
    hipLaunchKernelGGL((mx_tile_kernel<BF16, 2, 4, 8, 4>), dim3(grid), dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((mx_tile_kernel<BF16, 2, 2, 4, 4>), dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}
bool aligned(const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; }

// Bytes from the first to the last element of a strided matrix.
size_t span(int64_t rows, int64_t cols, int64_t ld, int es) {
  return rows <= 0 ? 0 : static_cast<size_t>((rows - 1) * ld + cols) * es;
}

fconv_status check_matrix(const void* x, int64_t ld, int32_t rows, int32_t cols, int32_t dtype) {
  if (rows < 0 || cols < 1 || ld < cols) return FCONV_ERR_INVALID_ARG;
  if (dtype != FCONV_BF16 && dtype != FCONV_FP32) return FCONV_ERR_UNSUPPORTED;
  if (cols > kMaxK || ceil_div(rows, 16) * ceil_div(cols, 512) > kMaxGroups) return FCONV_ERR_UNSUPPORTED;
  if (!x && rows > 0) return FCONV_ERR_INVALID_ARG;
  if (!aligned(x, dtype == FCONV_BF16 ? 2 : 4)) return FCONV_ERR_MISALIGNED;
  return FCONV_OK;
}

hipError_t launch_quantize(const void* x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype,
                           void* mx, hipStream_t s) {
  const int kt = static_cast<int>(ceil_div(cols, 128)), ks = static_cast<int>(ceil_div(cols, 512));
  const unsigned grid = static_cast<unsigned>(ceil_div(rows, 16) * ks);
  char* codes = static_cast<char*>(mx);
  char* scales = codes + codes_bytes(rows, cols);
  const char* src = static_cast<const char*>(x);
  if (dtype == FCONV_BF16)
    hipLaunchKernelGGL(mx_quantize_kernel<true>, dim3(grid), dim3(256), 0, s, src, ldx * 2,
                       static_cast<int64_t>(rows), cols, kt, ks, codes, scales);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<false>, dim3(grid), dim3(256), 0, s, src, ldx * 4,
                       static_cast<int64_t>(rows), cols, kt, ks, codes, scales);
  return hipGetLastError();
}

}  // namespace
}  // namespace fconv

extern "C" {

fconv_status fconv_mx_bytes(int32_t rows, int32_t cols, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 1) return FCONV_ERR_INVALID_ARG;
  if (cols > fconv::kMaxK) return FCONV_ERR_UNSUPPORTED;
  *bytes = fconv::codes_bytes(rows, cols) + fconv::scales_bytes(rows, cols);
  return FCONV_OK;
}

fconv_status fconv_mx_quantize(void* stream, const void* x, int64_t ldx, int32_t rows, int32_t cols,
                               int32_t dtype, void* mx) {
  using namespace fconv;
  const fconv_status st = check_matrix(x, ldx, rows, cols, dtype);
  if (st != FCONV_OK) return st;
  if (rows == 0) return FCONV_OK;
  if (!mx) return FCONV_ERR_INVALID_ARG;
  if (!aligned(mx, 16)) return FCONV_ERR_MISALIGNED;
  if (overlaps(x, span(rows, cols, ldx, dtype == FCONV_BF16 ? 2 : 4), mx,
               codes_bytes(rows, cols) + scales_bytes(rows, cols)))
    return FCONV_ERR_INVALID_ARG;
  return launch_quantize(x, ldx, rows, cols, dtype, mx, static_cast<hipStream_t>(stream)) == hipSuccess
             ? FCONV_OK
             : FCONV_ERR_DEVICE;
}

fconv_status fconv_mx_dequantize(void* stream, const void* mx, int32_t rows, int32_t cols,
                                 int32_t dtype, void* y, int64_t ldy) {
  using namespace fconv;
  const fconv_status st = check_matrix(y, ldy, rows, cols, dtype);
  if (st != FCONV_OK) return st;
  if (rows == 0) return FCONV_OK;
  if (!mx) return FCONV_ERR_INVALID_ARG;
  if (!aligned(mx, 16)) return FCONV_ERR_MISALIGNED;
  if (overlaps(y, span(rows, cols, ldy, dtype == FCONV_BF16 ? 2 : 4), mx,
               codes_bytes(rows, cols) + scales_bytes(rows, cols)))
    return FCONV_ERR_INVALID_ARG;
  const MxView v = view(mx, rows, cols);
  const int kt = static_cast<int>(ceil_div(cols, 128)), ks = static_cast<int>(ceil_div(cols, 512));
  const unsigned grid = static_cast<unsigned>(ceil_div(rows, 16) * ks);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* dst = static_cast<char*>(y);
  if (dtype == FCONV_BF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<true>, dim3(grid), dim3(256), 0, s, v.codes, v.scales,
                       static_cast<int64_t>(rows), cols, kt, ks, dst, ldy * 2);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<false>, dim3(grid), dim3(256), 0, s, v.codes, v.scales,
                       static_cast<int64_t>(rows), cols, kt, ks, dst, ldy * 4);
  return hipGetLastError() == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_mx_layout(void* stream, const void* codes, const void* scales, int32_t rows,
                             int32_t cols, void* mx) {
  using namespace fconv;
  if (rows < 0 || cols < 1) return FCONV_ERR_INVALID_ARG;
  if (cols > kMaxK || ceil_div(rows, 16) * ceil_div(cols, 512) > kMaxGroups) return FCONV_ERR_UNSUPPORTED;
  if (rows == 0) return FCONV_OK;
  if (!codes || !scales || !mx) return FCONV_ERR_INVALID_ARG;
  if (!aligned(codes, 4) || !aligned(mx, 16)) return FCONV_ERR_MISALIGNED;
  const size_t nb = static_cast<size_t>(ceil_div(cols, 32)) * rows;
  const size_t mb = codes_bytes(rows, cols) + scales_bytes(rows, cols);
  if (overlaps(codes, nb * 16, mx, mb) || overlaps(scales, nb, mx, mb)) return FCONV_ERR_INVALID_ARG;
  const int kt = static_cast<int>(ceil_div(cols, 128)), ks = static_cast<int>(ceil_div(cols, 512));
  const unsigned grid = static_cast<unsigned>(ceil_div(rows, 16) * ks);
  char* dst = static_cast<char*>(mx);
  hipLaunchKernelGGL(mx_layout_kernel, dim3(grid), dim3(256), 0, static_cast<hipStream_t>(stream),
                     static_cast<const char*>(codes), static_cast<const uint8_t*>(scales),
                     static_cast<int64_t>(rows), cols, kt, ks, dst, dst + codes_bytes(rows, cols));
  return hipGetLastError() == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_mx_plan_create(const fconv_mx_desc* desc, fconv_mx_plan* out) {
  using namespace fconv;
  if (!desc || !out) return FCONV_ERR_INVALID_ARG;
  *out = nullptr;
  const fconv_mx_desc& d = *desc;
  if (d.dtype != FCONV_BF16 && d.dtype != FCONV_FP32) return FCONV_ERR_UNSUPPORTED;
  if (d.flags) return FCONV_ERR_UNSUPPORTED;
  if (d.M < 0 || d.N < 1 || d.K < 1 || d.n_ops < 0 || d.n_ops > FCONV_MAX_OPS)
    return FCONV_ERR_INVALID_ARG;
  if (d.K > kMaxK || ceil_div(d.M, 16) * ceil_div(d.K, 512) > kMaxGroups ||
      ceil_div(d.M, 128) * ceil_div(d.N, 128) > kMaxGroups)
    return FCONV_ERR_UNSUPPORTED;
  int i = 0;
  auto next_is = [&](int32_t op) { return i < d.n_ops && d.ops[i] == op ? (++i, true) : false; };
  const bool bias = next_is(FCONV_OP_BIAS);
  const int32_t act = next_is(FCONV_OP_RELU)           ? 1
                      : next_is(FCONV_OP_LEAKY_RELU)   ? 2
                      : next_is(FCONV_OP_CLIPPED_RELU) ? 3
                      : next_is(FCONV_OP_CLAMP)        ? 4
                                                       : 0;
  if (i != d.n_ops) return FCONV_ERR_UNSUPPORTED;
  fconv_mx_plan_s* p = new (std::nothrow) fconv_mx_plan_s();
  if (!p) return FCONV_ERR_INVALID_ARG;
  p->d = d;
  p->esize = d.dtype == FCONV_BF16 ? 2 : 4;
  p->op_bias = bias;
  p->act = act;
  p->kt = static_cast<int32_t>(ceil_div(d.K, 128));
  p->tile = ceil_div(d.M, 256) * ceil_div(d.N, 256) >= 256 ? 256 : 128;
  p->ws_x = codes_bytes(d.M, d.K) + scales_bytes(d.M, d.K);
  p->ws_bytes = p->ws_x;
  p->kernel_name = p->tile == 256 ? "mx_tile_256" : "mx_tile_128";
  *out = p;
  return FCONV_OK;
}

fconv_status fconv_mx_plan_workspace_size(fconv_mx_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->ws_bytes;
  return FCONV_OK;
}

fconv_status fconv_mx_plan_run(fconv_mx_plan p, void* stream, const fconv_mx_args* args) {
  using namespace fconv;
  if (!p || !args) return FCONV_ERR_INVALID_ARG;
  const fconv_mx_desc& d = p->d;
  if (p->act >= 2) {
    const float al = args->activ_alpha, be = args->activ_beta;
    if (!(al - al == 0.0f)) return FCONV_ERR_INVALID_ARG;  // NaN or infinite
    if (p->act == 4 && !(be - be == 0.0f && al <= be)) return FCONV_ERR_INVALID_ARG;
  }
  if (d.M == 0) return FCONV_OK;
  if ((args->x != nullptr) == (args->x_mx != nullptr)) return FCONV_ERR_INVALID_ARG;
  if (!args->w_mx || !args->y || (p->op_bias && !args->bias)) return FCONV_ERR_INVALID_ARG;
  if ((args->x && args->ldx < d.K) || args->ldy < d.N) return FCONV_ERR_INVALID_ARG;
  const size_t ws = args->x ? p->ws_bytes : p->ws_bytes - p->ws_x;
  if (ws > 0 && (!args->workspace || args->workspace_bytes < p->ws_bytes)) return FCONV_ERR_WORKSPACE;
  if (!aligned(args->x, p->esize) || !aligned(args->y, p->esize) || !aligned(args->x_mx, 16) ||
      !aligned(args->w_mx, 16) || (p->op_bias && !aligned(args->bias, 4)) ||
      (ws > 0 && !aligned(args->workspace, 16)))
    return FCONV_ERR_MISALIGNED;
  const size_t yb = span(d.M, d.N, args->ldy, p->esize);
  const size_t xb = args->x ? span(d.M, d.K, args->ldx, p->esize) : 0;
  const size_t wb = codes_bytes(d.N, d.K) + scales_bytes(d.N, d.K);
  const size_t wsb = ws > 0 ? p->ws_bytes : 0;
  const void* in[4] = {args->x, args->x_mx, args->w_mx, p->op_bias ? args->bias : nullptr};
  const size_t in_bytes[4] = {xb, p->ws_x, wb, static_cast<size_t>(d.N) * 4};
  for (int i = 0; i < 4; ++i)
    if (overlaps(args->y, yb, in[i], in_bytes[i]) || overlaps(args->workspace, wsb, in[i], in_bytes[i]))
      return FCONV_ERR_INVALID_ARG;
  if (overlaps(args->y, yb, args->workspace, wsb)) return FCONV_ERR_INVALID_ARG;

  hipStream_t s = static_cast<hipStream_t>(stream);
  const void* xmx = args->x_mx;
  if (args->x) {
    if (launch_quantize(args->x, args->ldx, d.M, d.K, d.dtype, args->workspace, s) != hipSuccess)
      return FCONV_ERR_DEVICE;
    xmx = args->workspace;
  }
  MxArgs a;
  a.w = view(args->w_mx, d.N, d.K);
  a.x = view(xmx, d.M, d.K);
  a.bias = p->op_bias ? args->bias : nullptr;
  a.y = static_cast<char*>(args->y);
  a.ldy_bytes = args->ldy * p->esize;
  a.M = d.M;
  a.N = d.N;
  a.kt = p->kt;
  a.ks = static_cast<int32_t>(ceil_div(d.K, 512));
  a.act = p->act;
  a.act_alpha = args->activ_alpha;
  a.act_beta = args->activ_beta;
  const hipError_t e = d.dtype == FCONV_BF16 ? launch_tiles<true>(p, a, s) : launch_tiles<false>(p, a, s);
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

const char* fconv_mx_plan_kernel_name(fconv_mx_plan p) { return p ? p->kernel_name : nullptr; }

fconv_status fconv_mx_plan_destroy(fconv_mx_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
