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
  int32_t kernel;   // fconv::Kernel
  int32_t kernel_mx;  // of a run whose x comes quantised
  int32_t rows_nt;  // of the rows kernel: tiles of 16 n for a wave
  int32_t ranges;   // of k, whose partial sums a second kernel joins
  size_t ws_x;      // bytes of the quantised x in the workspace
  size_t ws_bytes;
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
int64_t min_of(int64_t a, int64_t b) { return a < b ? a : b; }

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

// BYTES (a multiple of 16) from or to any address.  STREAM: they are not asked
// for again soon and leave the caches to others.  What is larger than
// kStreamBytes (the L2s together) goes that way where each access takes whole
// 64-byte lines: 16384 x 4096 bf16 were quantised in 32 us instead of 43 and
// written back in 25 instead of 38.  Smaller ones took up to 1 us more, fp32
// (whose accesses take half lines) 45 us instead of 32.
constexpr int64_t kStreamBytes = 32 << 20;
bool streams(const void* p, int64_t ld, int64_t rows, int es) {
  return es == 2 && rows * ld * es > kStreamBytes && (reinterpret_cast<uintptr_t>(p) & 63) == 0 && ld * es % 64 == 0;
}
template <bool STREAM, int BYTES>
__device__ inline void load_any(const char* p, void* v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
  for (int i = 0; i < BYTES; i += 16) {
    const u32x4* q = reinterpret_cast<const u32x4*>(p + i);
    const u32x4 x = STREAM ? __builtin_nontemporal_load(q) : *q;
    __builtin_memcpy(static_cast<char*>(v) + i, &x, 16);
  }
}
template <bool STREAM, int BYTES>
__device__ inline void store_any(char* p, const void* v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
  for (int i = 0; i < BYTES; i += 16) {
    u32x4 x;
    __builtin_memcpy(&x, static_cast<const char*>(v) + i, 16);
    u32x4* q = reinterpret_cast<u32x4*>(p + i);
    if constexpr (STREAM)
      __builtin_nontemporal_store(x, q);
    else
      *q = x;
  }
}

// Eight values of a row at column c, zeros past `cols` (n < 8 live ones at
// the tail).  gfx950 reads global memory at any byte alignment.
template <bool BF16, bool STREAM = false>
__device__ inline void load8(const char* p, int n, float v[8]) {
  if constexpr (BF16) {
    if (n >= 8) {
      uint16_t h[8];
      load_any<STREAM, 16>(p, h);
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
      load_any<STREAM, 32>(p, v);
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
template <bool BF16, bool STREAM>
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
      load8<BF16, STREAM>(x + r * ldx_bytes + static_cast<int64_t>(c) * ES, cols - c, v[i]);
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
template <bool BF16, bool STREAM>
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
        store_any<STREAM, 16>(p, h);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) __builtin_memcpy(p + 2 * j, &h[j], 2);
      }
    } else {
      if (n >= 8) {
        store_any<STREAM, 32>(p, v);
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
  int32_t ranges;        // of k
  float* part;           // ranges > 1: partial sums [range][M][ldp], instead of y
  int64_t ldp;
  // An x that is not quantised yet (the kernels that do so themselves).
  const char* raw;
  int64_t ldx_bytes;
  int32_t K;
  int32_t act;
  float act_alpha, act_beta;
};

// The float epilogue of the convolution plans; a NaN stays a NaN.  N values;
// the kind is asked once for all of them.
template <int N>
__device__ inline void activate(f32x4 (&t)[N], int act, float alpha, float beta) {
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[i][e] = f(t[i][e]);
  };
  switch (act) {  // uniform
    case 1: each([](float v) { return v < 0.0f ? 0.0f : v; }); break;
    case 2: each([=](float v) { return v > 0.0f ? v : alpha * v; }); break;
    case 3: each([=](float v) { return v < 0.0f ? 0.0f : v > alpha ? alpha : v; }); break;
    case 4: each([=](float v) { return v < alpha ? alpha : v > beta ? beta : v; }); break;
  }
}

template <bool BF16>
__device__ inline void store4(char* p, f32x4 t) {
  if constexpr (BF16) {
    const uint16_t h[4] = {f32_to_bf16(t[0]), f32_to_bf16(t[1]), f32_to_bf16(t[2]), f32_to_bf16(t[3])};
    __builtin_memcpy(p, h, 8);
  } else {
    __builtin_memcpy(p, &t, 16);
  }
}
// Two matrix tiles side by side in bf16: t0 holds this lane's four n of the
// first, t1 of the second.  Rows of 16 lanes exchange halves, so that a lane
// ends with eight consecutive n (those of tile g % 2 from 8 (g / 2) on) and the
// lanes of a row m write 64 bytes at once.
__device__ inline void store_pair(char* p, f32x4 t0, f32x4 t1) {
  uint32_t v[4];
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const uint32_t x = f32_to_bf16(t0[2 * d]) | static_cast<uint32_t>(f32_to_bf16(t0[2 * d + 1])) << 16;
    const uint32_t y = f32_to_bf16(t1[2 * d]) | static_cast<uint32_t>(f32_to_bf16(t1[2 * d + 1])) << 16;
    const auto s = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    v[d] = s[0];
    v[2 + d] = s[1];
  }
  __builtin_memcpy(p, v, 16);
}
template <bool BF16>
__device__ inline void store1(char* p, float t) {
  if constexpr (BF16) {
    const uint16_t h = f32_to_bf16(t);
    __builtin_memcpy(p, &h, 2);
  } else {
    __builtin_memcpy(p, &t, 4);
  }
}

// The bias of this lane's n[i] .. + 3.
template <int NI>
__device__ inline void load_bias(const MxArgs& a, const int (&n)[NI], bool whole, f32x4 (&bias)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    bias[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!a.bias) continue;
    if (whole) {
      __builtin_memcpy(&bias[i], a.bias + n[i], 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n[i] + e < a.N) bias[i][e] = a.bias[n[i] + e];
    }
  }
}

// Bias, activation and store of this lane's part of a tile: n[i] .. + 3 of rows
// m[j] (g = lane / 16; tiles i, i + 1 of even i lie side by side).  Whether the tile ends inside N is asked once (`whole`): element by
// element these questions took longer than the rest of the tile's end.
template <bool BF16, int NI, int NJ>
__device__ inline void finish(const MxArgs& a, f32x4 (&acc)[NJ][NI], const int (&n)[NI], const int64_t (&m)[NJ],
                              const f32x4 (&bias)[NI], int g, bool whole, int range) {
  constexpr int ES = BF16 ? 2 : 4;
  if (a.part) {  // rows of ldp, a multiple of 4
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (m[j] >= a.M) continue;
      float* row = a.part + (static_cast<int64_t>(range) * a.M + m[j]) * a.ldp;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (n[i] < a.ldp) *reinterpret_cast<f32x4*>(row + n[i]) = acc[j][i];
    }
    return;
  }
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[j][i] += bias[i];
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    activate(acc[j], a.act, a.act_alpha, a.act_beta);
    if (m[j] >= a.M) continue;
    char* row = a.y + m[j] * a.ldy_bytes;
    if (whole) {
      if constexpr (BF16 && NI % 2 == 0) {
#pragma unroll
        for (int i = 0; i < NI; i += 2)
          store_pair(row + static_cast<int64_t>(n[i] - 4 * g + (g & 1) * 16 + (g >> 1) * 8) * ES, acc[j][i],
                     acc[j][i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) store4<BF16>(row + static_cast<int64_t>(n[i]) * ES, acc[j][i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        char* p = row + static_cast<int64_t>(n[i]) * ES;
        if (n[i] + 4 <= a.N) {
          store4<BF16>(p, acc[j][i]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n[i] + e < a.N) store1<BF16>(p + e * ES, acc[j][i][e]);
        }
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

// A wave's copy of 1 KiB into LDS, 16 bytes a lane from base + off (this lane's;
// zeros past `bytes`).
__device__ inline void copy_1k(const char* base, int64_t bytes, char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(base, bytes), (lds_ptr_t)lds, 16, off, 0, 0, 0);
}

// Tiled product.  A workgroup owns a (2 H) n x (2 H) m tile in four quadrants;
// NW waves share each quadrant, two along n, NW / 2 along m.  A slab is two k
// tiles (256 columns) of both operands: four half tiles, copied buffer->LDS,
// in one of two sets of buffers.  A slab takes four phases, a quadrant each:
//   phase   reads (LDS)                copies for the slab after next   products
//   0       W0 but two (and scales)    scales of two slabs on           0 0
//   1       X1, two fragments of W1    W0, X0 (their readers are done)  0 1
//   2       the rest of W1             X1                               1 1
//   3       next slab's X0, two of W0  W1                               1 0
// A phase is two steps between barriers: a wave reads fragments and starts
// copies in one, multiplies in the other.  With eight waves the four of the
// second half of n run one step behind the others, so that on every SIMD one
// wave multiplies while the other reads.  A step of products takes 256 cycles;
// six fragments for each of four waves keep LDS (128 bytes a cycle) busy for
// 192, so the reads are spread evenly.  A copy has more than a slab's time to
// arrive; the waits stand one phase before the first reads, in phase 2 for W0
// and X0 of the next slab and in phase 0 for this one's others.  The scales of
// a pair of slabs (four k tiles) are copied together and read once.
template <bool BF16, int H, int NW>
__global__ __launch_bounds__(NW * 64, 2) void mx_tile_kernel(MxArgs a) {
  constexpr int MI = H / 32, MJ = 2 * H / (16 * NW);  // matrix tiles of a wave in a quadrant
  constexpr int RT = H / 16;                          // row tiles of a half tile
  constexpr int HB = RT * 2 * kTileBytes;             // bytes of a half tile
  static_assert(RT == NW, "one row tile per wave and half tile");
  // Arrays of their own, so that the compiler sees which copies a read does not
  // meet.
  __shared__ __attribute__((aligned(1024))) char wx0[2 * HB], x10[HB], w10[HB];
  __shared__ __attribute__((aligned(1024))) char wx1[2 * HB], x11[HB], w11[HB];
  __shared__ __attribute__((aligned(1024))) char scales[2][4 * RT * kScaleTile];

  // Workgroups of one XCD (block ids go round the 8 XCDs) take neighbouring
  // tiles: eight tile rows of m together, so both panels stay in its L2.
  // The workgroup stays for every so manieth tile of its XCD's share.
  const int tiles = a.tiles_m * a.tiles_n;
  const int total = tiles * a.ranges, share = (total + 7) / 8;
  const int first_id = (blockIdx.x % 8) * share, end = min(share, total - first_id);
  int slot = blockIdx.x / 8;
  if (slot >= end) return;
  const int64_t row_bytes = static_cast<int64_t>(a.kt) * kTileBytes;
  const int64_t srow_bytes = static_cast<int64_t>(a.ks) * kScaleTile;
  const int ks_per = (a.ks + a.ranges - 1) / a.ranges;
  struct Place {
    int range, ks0, kt0, kt1;  // this range's k tiles, whole scale tiles of them
    int64_t rtw, rtx;
  };
  auto locate = [&](int id) __attribute__((always_inline)) {
    Place p;
    const int tile = id % tiles;
    const int per = 8 * a.tiles_n;
    const int m_first = tile / per * 8, m_rows = min(8, a.tiles_m - m_first), in = tile % per;
    p.range = id / tiles;
    p.rtw = static_cast<int64_t>(in / m_rows) * 2 * RT;
    p.rtx = static_cast<int64_t>(m_first + in % m_rows) * 2 * RT;
    p.ks0 = p.range * ks_per;
    p.kt0 = min(4 * p.ks0, a.kt);
    p.kt1 = min(p.kt0 + 4 * ks_per, a.kt);
    return p;
  };
  Place at = locate(first_id + slot);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave / (NW / 2), wb = wave % (NW / 2);
  // A wave copies the scales of four row tiles, of W or of X.
  const bool swave = wave < NW / 2;
  const uint32_t s_off =
      static_cast<uint32_t>((4 * (wave % (NW / 2)) + (lane >> 4)) * srow_bytes + (lane & 15) * 16);
  uint32_t first_off[2];  // of this wave's row tile in either half
#pragma unroll
  for (int h = 0; h < 2; ++h) first_off[h] = static_cast<uint32_t>((h * RT + wave) * row_bytes + lane * 16);
  // The next slab to copy: its offset, k tiles, and scale tile counted from the range's first.
  uint32_t off;
  int next_kt, next_ks;

  // Past the last k tile the copies bring zeros.
  auto copy = [&](bool x, int h, char* buf) __attribute__((always_inline)) {
    const MxView& v = x ? a.x : a.w;
    const int64_t rt = x ? at.rtx : at.rtw;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      copy_1k(v.codes + rt * row_bytes, (v.row_tiles - rt) * row_bytes, buf + (wave * 2 + c) * kTileBytes,
              next_kt + c < at.kt1 ? first_off[h] + off + static_cast<uint32_t>(c * kTileBytes) : kOutOfRange);
  };
  auto advance = [&]() __attribute__((always_inline)) {
    next_kt += 2;
    off += 2 * kTileBytes;
  };
  auto copy_scales = [&]() __attribute__((always_inline)) {
    const MxView& v = swave ? a.w : a.x;
    const int64_t rt = swave ? at.rtw : at.rtx;
    copy_1k(v.scales + rt * srow_bytes, (v.row_tiles - rt) * srow_bytes, scales[next_ks & 1] + wave * 1024,
            at.ks0 + next_ks < a.ks ? s_off + static_cast<uint32_t>(at.ks0 + next_ks) * kScaleTile : kOutOfRange);
    ++next_ks;
  };

  // The first two slabs of a tile, and the scales of both.
  auto begin = [&]() __attribute__((always_inline)) {
    next_kt = at.kt0;
    next_ks = 0;
    off = static_cast<uint32_t>(at.kt0) * kTileBytes;
    copy_scales();
    copy(false, 0, wx0);
    copy(true, 0, wx0 + HB);
    copy(true, 1, x10);
    copy(false, 1, w10);
    advance();
    copy(false, 0, wx1);
    copy(true, 0, wx1 + HB);
    copy(true, 1, x11);
    copy(false, 1, w11);
    advance();
  };
  f32x4 acc[2 * MJ][2 * MI];
  int sw[2 * MI], sx[2 * MJ];
  // Fragments [tile][k tile] of a half of W, but for the first EARLY tiles' first
  // k tile of W1, which are read while W0 is in use; and of the halves of X.
  constexpr int EARLY = MI == 4 ? 2 : 0;
  i32x4 fw[MI][2], fe[EARLY + 1], fx[2][MJ][2];

  auto read_scales = [&](const char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i)
      sw[i] = *reinterpret_cast<const int*>(buf + (i / MI * RT + wa * MI + i % MI) * kScaleTile + lane * 4);
#pragma unroll
    for (int j = 0; j < 2 * MJ; ++j)
      sx[j] = *reinterpret_cast<const int*>(buf + ((2 + j / MJ) * RT + wb * MJ + j % MJ) * kScaleTile + lane * 4);
  };
  auto w_at = [&](const char* buf, int i, int kk) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(buf + ((wa * MI + i) * 2 + kk) * kTileBytes + lane * 16);
  };
  auto read_w_rest = [&](const char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = kk == 0 ? EARLY : 0; i < MI; ++i) fw[i][kk] = w_at(buf, i, kk);
  };
  auto read_x = [&](i32x4 (&x)[MJ][2], const char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < MJ; ++j)
        x[j][kk] = *reinterpret_cast<const i32x4*>(buf + ((wb * MJ + j) * 2 + kk) * kTileBytes + lane * 16);
  };
  auto read_step_ends = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's LDS reads are done
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // SEL: the byte of the scale dwords of the slab's first k tile.
  auto multiply = [&](int i2, int j2, const i32x4 (&x)[MJ][2], auto sel) __attribute__((always_inline)) {
    constexpr int SEL = decltype(sel)::value;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        f32x4& c = acc[j2 * MJ + j][i2 * MI + i];
        c = mma<SEL>(i2 == 1 && i < EARLY ? fe[i] : fw[i][0], x[j][0], c, sw[i2 * MI + i], sx[j2 * MJ + j]);
      }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        f32x4& c = acc[j2 * MJ + j][i2 * MI + i];
        c = mma<SEL + 1>(fw[i][1], x[j][1], c, sw[i2 * MI + i], sx[j2 * MJ + j]);
      }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // x0 holds this slab's X0; xb gets X1, then the next slab's X0.
  auto slab = [&](char* wx, char* x1, char* w1, const char* wx_next, i32x4 (&x0)[MJ][2], i32x4 (&xb)[MJ][2],
                  auto sel) __attribute__((always_inline)) {
    constexpr bool FIRST = decltype(sel)::value == 0;  // of a pair
    if (FIRST) read_scales(scales[(next_ks - 1) & 1]);
    read_w_rest(wx);
    if (FIRST) copy_scales();
    __builtin_amdgcn_s_waitcnt(FIRST ? 0x0F79 : 0x0F78);  // vmcnt(9 or 8): this slab is here
    read_step_ends();
    multiply(0, 0, x0, sel);

    read_x(xb, x1);
#pragma unroll
    for (int i = 0; i < EARLY; ++i) fe[i] = w_at(w1, i, 0);
    copy(false, 0, wx);
    copy(true, 0, wx + HB);
    read_step_ends();
    multiply(0, 1, xb, sel);

    read_w_rest(w1);
    copy(true, 1, x1);
    __builtin_amdgcn_s_waitcnt(FIRST ? 0x0F7B : 0x0F7A);  // vmcnt(11 or 10): the next slab's W0 and X0 are here
    read_step_ends();
    multiply(1, 1, xb, sel);

    read_x(xb, wx_next + HB);
#pragma unroll
    for (int i = 0; i < EARLY; ++i) fw[i][0] = w_at(wx_next, i, 0);
    copy(false, 1, w1);
    advance();
    read_step_ends();
    multiply(1, 0, x0, sel);
  };

  begin();
  for (;;) {
#pragma unroll
    for (int j = 0; j < 2 * MJ; ++j)
#pragma unroll
      for (int i = 0; i < 2 * MI; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    __builtin_amdgcn_s_waitcnt(0x0F78);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_x(fx[0], wx0 + HB);
#pragma unroll
    for (int i = 0; i < EARLY; ++i) fw[i][0] = w_at(wx0, i, 0);
    if (NW == 8 && wa == 1) __builtin_amdgcn_s_barrier();
    const int slabs = (at.kt1 - at.kt0 + 1) / 2;
    for (int s = 0; s + 1 < slabs; s += 2) {
      slab(wx0, x10, w10, wx1, fx[0], fx[1], std::integral_constant<int, 0>{});
      slab(wx1, x11, w11, wx0, fx[1], fx[0], std::integral_constant<int, 2>{});
    }
    if (slabs & 1) slab(wx0, x10, w10, wx1, fx[0], fx[1], std::integral_constant<int, 0>{});
    if (NW == 8 && wa == 0) __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_s_waitcnt(0);  // copies past the last slab have landed

    // The next tile's copies are under way while this one is finished; the bias
    // comes before them, since loads return in order.
    int l = lane;
    asm volatile("" : "+v"(l));  // places computed here, not kept in registers through the products
    const int g = l >> 4, r = l & 15;
    const Place done = at;
    int n[2 * MI];
    int64_t m[2 * MJ];
    f32x4 bias[2 * MI];
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i)
      n[i] = static_cast<int>((done.rtw + i / MI * RT + wa * MI + i % MI) * 16 + 4 * g);
#pragma unroll
    for (int j = 0; j < 2 * MJ; ++j) m[j] = (done.rtx + j / MJ * RT + wb * MJ + j % MJ) * 16 + r;
    const bool whole = (done.rtw + 2 * RT) * 16 <= a.N;
    load_bias(a, n, whole, bias);
    slot += gridDim.x / 8;
    const bool more = slot < end;
    if (more) {
      at = locate(first_id + slot);
      begin();
    }
    finish<BF16>(a, acc, n, m, bias, g, whole, done.range);
    if (!more) break;
  }
}

template <bool STREAM = false>
__device__ inline i32x4 load16(const char* p) {
  const i32x4* q = reinterpret_cast<const i32x4*>(p);
  return STREAM ? __builtin_nontemporal_load(q) : *q;
}

// Few rows of x.  The time is W's way out of memory, so W goes straight into
// registers, in the order in which it is stored: no LDS, no barrier before the
// end.  A workgroup owns 16 NT n and one range of k; its NW waves take turns at
// the range's scale tiles (512 columns: 8 KiB of W, all loads in flight, the
// next turn's while this one is multiplied) and add their sums in LDS, in
// order.  Four waves, or eight where K is longer than a turn of those; sixteen
// and 16 n, see few_deep.
// With STREAM W leaves the caches to others (one row of 4096 -> 32768 12.5 us
// instead of 13.7; but 32 rows of 25088 -> 1024, whose 13 MB stay in the caches
// from call to call, took 3 us longer: above kStreamBytes).
// With RAW the workgroup quantises x itself, into LDS, before it starts: for
// the few thousand values of one or two tokens that is quicker than a launch.
// 64 rows by four waves: two waves a SIMD, where the compiler's 268 registers left
// one (64 rows of 1024 -> 32768 12.1 us instead of 14.5, -> 2048 7.2 and 7.0).
template <bool BF16, int MT, int NW, bool RAW, bool STREAM, int NT = 2>
__global__ __launch_bounds__(NW * 64, MT == 4 && NW == 4 ? 2 : 1) void mx_few_kernel(MxArgs a) {
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ f32x4 sums[NW][NT * MT][64];
  extern __shared__ __attribute__((aligned(16))) char raw_codes[];  // RAW: [k tile][block][M] of 16 bytes, then scales
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int groups = (a.N + 16 * NT - 1) / (16 * NT);
  const int range = blockIdx.x / groups;
  const int64_t nt0 = static_cast<int64_t>(blockIdx.x % groups) * NT;
  const int ks_per = (a.ks + a.ranges - 1) / a.ranges;
  const int ks0 = range * ks_per, ks1 = min(ks0 + ks_per, a.ks);

  // A row tile past the last one reads the last one again (it is not stored).
  const char* wc[NT];
  const char* wsc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t rt = nt0 + t < a.w.row_tiles ? nt0 + t : a.w.row_tiles - 1;
    wc[t] = a.w.codes + rt * a.kt * kTileBytes + lane * 16;
    wsc[t] = a.w.scales + rt * a.ks * kScaleTile + lane * 4;
  }
  const char* xc[MT];
  const char* xsc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t rt = t < a.x.row_tiles ? t : a.x.row_tiles - 1;
    xc[t] = a.x.codes + rt * a.kt * kTileBytes + lane * 16;
    xsc[t] = a.x.scales + rt * a.ks * kScaleTile + lane * 4;
  }

  struct Turn {
    i32x4 w[NT][4], x[RAW ? 1 : MT][4];
    int ws[NT], xs[RAW ? 1 : MT];
  };
  // k tiles past the last one read the last one again; `multiply` skips them.
  auto load = [&](Turn& t, int ks) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = static_cast<int64_t>(min(4 * ks + k, a.kt - 1)) * kTileBytes;
#pragma unroll
      for (int i = 0; i < NT; ++i) t.w[i][k] = load16<STREAM>(wc[i] + at);
      if constexpr (!RAW) {
#pragma unroll
        for (int i = 0; i < MT; ++i) t.x[i][k] = load16(xc[i] + at);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) t.ws[i] = *reinterpret_cast<const int*>(wsc[i] + static_cast<int64_t>(ks) * kScaleTile);
    if constexpr (!RAW) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
        t.xs[i] = *reinterpret_cast<const int*>(xsc[i] + static_cast<int64_t>(ks) * kScaleTile);
    }
  };
  Turn now, next;
  int ks = ks0 + wave;
  if (ks < ks1) load(now, ks);

  const int rows = a.M;  // RAW: of x, at most 16
  char* raw_scales = raw_codes + static_cast<int64_t>(ks_per) * 4 * 64 * rows;
  if constexpr (RAW) {
    // Eight values a thread and step; the four lanes of a block agree on its
    // largest magnitude.
    const int per_row = ks_per * 64, total = per_row * rows;
    for (int i = threadIdx.x; i < total; i += NW * 64) {
      const int row = i / per_row, e8 = i - row * per_row;
      const int64_t c = static_cast<int64_t>(ks0) * 512 + e8 * 8;
      float v[8];
      if (c < a.K) {
        load8<BF16>(a.raw + row * a.ldx_bytes + c * ES, static_cast<int>(a.K - c < 8 ? a.K - c : 8), v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      }
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
      const uint32_t byte = scale_byte(quad_max(m));
      const int blk = e8 >> 2;
      *reinterpret_cast<uint32_t*>(raw_codes + (blk * rows + row) * 16 + (e8 & 3) * 4) = encode8(v, byte);
      if ((e8 & 3) == 0) raw_scales[blk * rows + row] = static_cast<char>(byte);
    }
    __syncthreads();
  }

  f32x4 acc[MT][NT] = {};
  auto multiply = [&](Turn& t, int ks) __attribute__((always_inline)) {
    auto step = [&](auto sel) __attribute__((always_inline)) {
      constexpr int K = decltype(sel)::value;
      if (4 * ks + K >= a.kt) return;  // uniform
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        i32x4 x;
        int xs;
        if constexpr (RAW) {
          // Rows past M stand for row 0: they are not stored.
          const int at = (((ks - ks0) * 4 + K) * 4 + g) * rows + (r < rows ? r : 0);
          x = *reinterpret_cast<const i32x4*>(raw_codes + at * 16);
          xs = static_cast<uint8_t>(raw_scales[at]) * 0x01010101;
        } else {
          x = t.x[j][K];
          xs = t.xs[j];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[j][i] = mma<K>(t.w[i][K], x, acc[j][i], t.ws[i], xs);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  for (; ks < ks1; ks += 2 * NW) {
    if (ks + NW < ks1) load(next, ks + NW);
    multiply(now, ks);
    if (ks + NW >= ks1) break;
    if (ks + 2 * NW < ks1) load(now, ks + 2 * NW);
    multiply(next, ks + NW);
  }

#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i) sums[wave][j * NT + i][lane] = acc[j][i];
  __syncthreads();
  if (wave >= MT) return;
  f32x4 out[1][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    out[0][i] = sums[0][wave * NT + i][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) out[0][i] += sums[w][wave * NT + i][lane];
  }
  int n[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) n[i] = static_cast<int>(nt0 + i) * 16 + 4 * g;
  const int64_t m[1] = {wave * 16 + r};
  f32x4 bias[NT];
  const bool whole = (nt0 + NT) * 16 <= a.N;
  load_bias(a, n, whole, bias);
  finish<BF16>(a, out, n, m, bias, g, whole, range);
}

// Small products, and many rows of few n: x is quantised on its way into the
// product and never written, which saves a launch and, where n is few, x's way
// through memory.  A workgroup owns 64 rows and NT tiles of 16 n, a wave 16 of
// the rows.  A lane holds one block of 32 values of a row and step, which is the
// matrix core's own order: the block's largest magnitude and its codes need no
// other lane.  W comes through the caches; the next step's x is loaded meanwhile.
// Three waves a SIMD (two with NT 8) in 145 registers, where the compiler took 180
// by itself: 100352 rows of 256 -> 64 16.1 us instead of 17.9, 200704 of 128 -> 64
// 18.9 and 22.0; four waves spill (28.5 us).
template <bool BF16, int NT>
__global__ __launch_bounds__(256, NT == 4 ? 3 : 2) void mx_rows_kernel(MxArgs a) {
  constexpr int ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int64_t mt = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (mt * 16 >= a.M) return;
  const int64_t nt0 = static_cast<int64_t>(blockIdx.y) * NT;
  const int64_t row = mt * 16 + r;
  const char* xp = a.raw + (row < a.M ? row : a.M - 1) * a.ldx_bytes + g * 32 * ES;
  const char* wc[NT];
  const char* wsc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t rt = nt0 + t < a.w.row_tiles ? nt0 + t : a.w.row_tiles - 1;
    wc[t] = a.w.codes + rt * a.kt * kTileBytes + lane * 16;
    wsc[t] = a.w.scales + rt * a.ks * kScaleTile + lane * 4;
  }
  struct Raw {
    i32x4 q[2 * ES];
  };
  auto load = [&](Raw& x, int kt) __attribute__((always_inline)) {
    const int left = a.K - kt * 128 - g * 32;  // values of this block
    const char* p = xp + static_cast<int64_t>(kt) * 128 * ES;
    if (left >= 32) {
      __builtin_memcpy(&x, p, 32 * ES);
    } else {
      using U = std::conditional_t<BF16, uint16_t, uint32_t>;
      U u[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        u[i] = 0;
        if (i < left) __builtin_memcpy(&u[i], p + i * ES, ES);
      }
      __builtin_memcpy(&x, u, 32 * ES);
    }
  };
  f32x4 acc[1][NT] = {};
  auto use = [&](const Raw& x, int kt) __attribute__((always_inline)) {
    i32x4 w[NT];
    int ws[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[t] = load16(wc[t] + static_cast<int64_t>(kt) * kTileBytes);
      ws[t] = *reinterpret_cast<const int*>(wsc[t] + static_cast<int64_t>(kt >> 2) * kScaleTile) >> (8 * (kt & 3));
    }
    float v[32];
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t u = static_cast<uint32_t>(x.q[i >> 2][i & 3]);
        v[2 * i] = __builtin_bit_cast(float, u << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
      }
    } else {
      __builtin_memcpy(v, &x, 128);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, abs_bits(v[i]));
    const uint32_t byte = scale_byte(m);
    i32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = static_cast<int>(encode8(v + 8 * i, byte));
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[0][t] = mma<0>(w[t], c, acc[0][t], ws[t], static_cast<int>(byte));
  };
  Raw now, next;
  load(now, 0);
  for (int kt = 0; kt < a.kt; kt += 2) {
    if (kt + 1 < a.kt) load(next, kt + 1);
    use(now, kt);
    if (kt + 1 >= a.kt) break;
    if (kt + 2 < a.kt) load(now, kt + 2);
    use(next, kt + 1);
  }
  int n[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) n[t] = static_cast<int>(nt0 + t) * 16 + 4 * g;
  const int64_t m[1] = {row};
  f32x4 bias[NT];
  const bool whole = (nt0 + NT) * 16 <= a.N;
  load_bias(a, n, whole, bias);
  finish<BF16>(a, acc, n, m, bias, g, whole, 0);
}

// y = act(sum of the ranges, in order, + bias); four n of a row per thread.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_join_kernel(MxArgs a) {
  constexpr int ES = BF16 ? 2 : 4;
  const int quads = (a.N + 3) / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = i / quads;
  const int n = static_cast<int>(i - m * quads) * 4;
  if (m >= a.M) return;
  f32x4 t[1] = {};
  const float* p0 = a.part + m * a.ldp + n;
  const int64_t step = static_cast<int64_t>(a.M) * a.ldp;
  // Eight loads in flight (those past the last range read it again): one at a
  // time, 13 ranges took 11 us.
  for (int k = 0; k < a.ranges; k += 8) {
    f32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const f32x4*>(p0 + min(k + i, a.ranges - 1) * step);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < a.ranges) t[0] += v[i];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (a.bias && n + e < a.N) t[0][e] += a.bias[n + e];
  activate(t, a.act, a.act_alpha, a.act_beta);
  char* p = a.y + m * a.ldy_bytes + static_cast<int64_t>(n) * ES;
  if (n + 4 <= a.N) {
    store4<BF16>(p, t[0]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) store1<BF16>(p + e * ES, t[0][e]);
  }
}

enum Kernel : int32_t { kTile256, kTile128, kFew, kFewRaw, kRows };
const char* const kKernelNames[] = {"mx_tile_256", "mx_tile_128", "mx_few", "mx_few_raw", "mx_rows"};

// LDS of the few-rows kernel that quantises: a range's codes and scales.
int few_raw_bytes(const fconv_mx_plan_s* p) {
  const int64_t ks_per = ceil_div(ceil_div(p->d.K, 512), p->ranges);
  return static_cast<int>(ks_per * 4 * (64 + 4) * p->d.M);
}

// Few outputs of a long K leave most CUs idle, and a wave's turns come one after
// another: sixteen waves for 16 n (32 rows of 25088 -> 1024 12.1 us instead of
// 14.5, of 8192 -> 1024 7.8 and 8.9, 16 of 16384 -> 4096 10.7 and 12.3, with the
// quantisation).
bool few_deep(const fconv_mx_plan_s* p) {
  return p->d.M <= 32 && ceil_div(p->d.N, 16) <= 256 && ceil_div(ceil_div(p->d.K, 512), p->ranges) >= 16;
}

// Time (us) of the rows kernel with NT tiles of 16 n for a wave.  A step of 128 k
// takes a wave alone 0.6 (NT 4) or 0.7 us (NT 8); more than a wave for a SIMD add
// up.  128 to 512 rows of 512 -> 512: 5.7 (NT 4) and 7.0, by the 128 tiles 9.7;
// 2048 of 1024 -> 1024: 13.5, 10.5 and 12.7; 8192 of 512 -> 512: 15.4, 13.5, 12.1.
// Rows of fp32, and of bf16 that begin between dwords, take twice as long (896 of
// 2827 -> 256 fp32 31.6, by the 128 tiles 16.4; 892 of 953 -> 2228 bf16 17.0 and
// 12.6).
double rows_us(const fconv_mx_desc& d, int es, int nt) {
  const double M = d.M, N = d.N, K = d.K, kt = static_cast<double>(ceil_div(d.K, 128));
  const double full = static_cast<double>(ceil_div(d.M, 16) * ceil_div(d.N, 16 * nt)) / 1024;  // waves for a SIMD
  const double slow = es == 4 ? 2.1 : d.K % 2 ? 2.0 : 1.0;
  const double step = slow * (nt == 4 ? (full > 1 ? 0.2 + 0.55 * full : 0.58) : 0.73 * (full > 1 ? full : 1));
  const double base = nt == 4 ? 2.2 + (full > 1 ? full : 1) : 3.0 + (2.4 * full > 1 ? 2.4 * full : 1);
  const double memory = 2.0 + (M * K + M * N) * es / 5.2e6;
  return base + step * kt > memory ? base + step * kt : memory;
}

// The product's kernel and ranges of k, by the least time of rough accounts (us).
void choose_kernel(fconv_mx_plan_s* p) {
  const int64_t M = p->d.M, N = p->d.N, ks = ceil_div(p->d.K, 512);
  const double weights = 0.53 * static_cast<double>(N) * static_cast<double>(p->d.K);
  p->ranges = 1;
  p->rows_nt = 4;
  double rows = 1e300;
  for (int nt = 4; nt <= 8; nt += 4) {
    const double us = rows_us(p->d, p->esize, nt);
    // A longer K reads x and W past what the account knows (8924 of 5696 -> 138
    // 84 us, by the tiles 48).
    if (ceil_div(N, 64) > 65535 || p->d.K > 2048 || us >= rows) continue;
    rows = us;
    p->rows_nt = nt;
  }
  // The others quantise x in a launch of its own (2.5 us captured, 3.9 back to back).
  const double quantise = 3.6 + (p->esize + 0.53) * static_cast<double>(M) * static_cast<double>(p->d.K) / 5e6;
  double least = 1e300;
  if (M <= 64 && ceil_div(N, 32) <= kMaxGroups) {
    p->kernel = kFew;
    // Ranges only where K > 32768: 32 rows of 25088 -> 1024 in eight of them gained
    // less than the launch that joins them takes.
    p->ranges = static_cast<int32_t>(min_of(ceil_div(ks, 64), ceil_div(1024, ceil_div(N, 32))));
    p->ranges = static_cast<int32_t>(ceil_div(ks, ceil_div(ks, p->ranges)));
    // At most 20 scale tiles: its four waves take them in turns (one row of 16384 ->
    // 1024 9.9 us, of 9984 7.3).
    if (M <= 16 && M * ceil_div(ks, p->ranges) * 512 <= 16384 && ceil_div(ks, p->ranges) <= 20) {
      p->kernel = kFewRaw;
      return;
    }
    // W at 5.2, 4.2 or 3 TB/s for 16, 32 or 64 rows (32768 x 4096: 13.7, 17.7 and
    // 24.4 us, the 128 tiles 15.9, 16.3 and 16.9).
    // A long K of few outputs is bound by the turns' latency.
    const double turns = 3.0 + (few_deep(p) ? 2.4e-4 : 3.2e-4) * static_cast<double>(p->d.K);
    least = 1.5 + weights / (M <= 16 ? 5.2e6 : M <= 32 ? 4.2e6 : 3.0e6);
    least = quantise + (least > turns ? least : turns);
    if (p->ranges > 1) return;
  }
  // Tiles: workgroups take turns on the device, each as long as its slabs (256
  // columns) and what a tile costs beside them; partial sums are written and read
  // once more.
  struct Kind {
    int32_t kernel;
    int64_t edge, at_once;
    double slab, slab_alone, tile;
  };
  static const Kind kinds[] = {{kTile256, 256, 256, 1.7, 1.4, 10.0}, {kTile128, 128, 512, 1.05, 0.7, 5.0}};
  for (const Kind& k : kinds) {
    const int64_t tiles = ceil_div(M, k.edge) * ceil_div(N, k.edge);
    for (int64_t r = 1; r <= ks && r <= 32; ++r) {
      const int64_t per = ceil_div(ks, r);
      if (ceil_div(ks, per) != r) continue;  // the same ranges as with fewer
      double us = quantise + static_cast<double>(ceil_div(tiles * r, k.at_once)) *
                                 (2.0 * static_cast<double>(per) * (tiles * r > 256 ? k.slab : k.slab_alone) + k.tile);
      if (r > 1) us += 4.0 + 8.0 * static_cast<double>(r * M) * static_cast<double>(N) / 6e6;
      if (us < least) {
        least = us;
        p->kernel = k.kernel;
        p->ranges = static_cast<int32_t>(r);
      }
    }
  }
  // The tiles' account is the better one where both are close (123 of 256 -> 26939
  // 10.7 us by the tiles, 12.6 by the rows).
  if (rows < 0.9 * least) {
    p->kernel = kRows;
    p->ranges = 1;
  }
}

template <bool BF16, bool STREAM>
void launch_few(const fconv_mx_plan_s* p, const MxArgs& a, bool raw, dim3 grid, hipStream_t s) {
  if (raw)
    hipLaunchKernelGGL((mx_few_kernel<BF16, 1, 4, true, STREAM>), grid, dim3(256), few_raw_bytes(p), s, a);
  else if (few_deep(p)) {
    if (a.M <= 16)
      hipLaunchKernelGGL((mx_few_kernel<BF16, 1, 16, false, STREAM, 1>), grid, dim3(1024), 0, s, a);
    else
      hipLaunchKernelGGL((mx_few_kernel<BF16, 2, 16, false, STREAM, 1>), grid, dim3(1024), 0, s, a);
  } else if (ceil_div(a.ks, a.ranges) <= 4) {
    if (a.M <= 16)
      hipLaunchKernelGGL((mx_few_kernel<BF16, 1, 4, false, STREAM>), grid, dim3(256), 0, s, a);
    else if (a.M <= 32)
      hipLaunchKernelGGL((mx_few_kernel<BF16, 2, 4, false, STREAM>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((mx_few_kernel<BF16, 4, 4, false, STREAM>), grid, dim3(256), 0, s, a);
  } else {
    if (a.M <= 16)
      hipLaunchKernelGGL((mx_few_kernel<BF16, 1, 8, false, STREAM>), grid, dim3(512), 0, s, a);
    else if (a.M <= 32)
      hipLaunchKernelGGL((mx_few_kernel<BF16, 2, 8, false, STREAM>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((mx_few_kernel<BF16, 4, 8, false, STREAM>), grid, dim3(512), 0, s, a);
  }
}

template <bool BF16>
hipError_t launch_product(const fconv_mx_plan_s* p, MxArgs a, int kernel, hipStream_t s) {
  const int64_t edge = kernel == kTile256 ? 256 : 128;
  a.tiles_m = static_cast<int32_t>(ceil_div(a.M, edge));
  a.tiles_n = static_cast<int32_t>(ceil_div(a.N, edge));
  // As many workgroups as the device holds at once (one or two a CU, by their LDS), in eighths.
  const int64_t most = kernel == kTile256 ? 256 : 512;
  const int64_t all = ceil_div(static_cast<int64_t>(a.tiles_m) * a.tiles_n * a.ranges, 8) * 8;
  const dim3 grid(static_cast<unsigned>(all < most ? all : most));
  const dim3 few(static_cast<unsigned>(ceil_div(a.N, kernel == kFew && few_deep(p) ? 16 : 32) * a.ranges));
  const dim3 rows(static_cast<unsigned>(ceil_div(a.M, 64)), static_cast<unsigned>(ceil_div(a.N, 16 * p->rows_nt)));
  switch (kernel) {
    case kTile256: hipLaunchKernelGGL((mx_tile_kernel<BF16, 128, 8>), grid, dim3(512), 0, s, a); break;
    case kTile128: hipLaunchKernelGGL((mx_tile_kernel<BF16, 64, 4>), grid, dim3(256), 0, s, a); break;
    case kFewRaw:
    case kFew:
      if (codes_bytes(a.N, a.K) > static_cast<size_t>(kStreamBytes))
        launch_few<BF16, true>(p, a, kernel == kFewRaw, few, s);
      else
        launch_few<BF16, false>(p, a, kernel == kFewRaw, few, s);
      break;
    case kRows:
      if (p->rows_nt == 4)
        hipLaunchKernelGGL((mx_rows_kernel<BF16, 4>), rows, dim3(256), 0, s, a);
      else
        hipLaunchKernelGGL((mx_rows_kernel<BF16, 8>), rows, dim3(256), 0, s, a);
      break;
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.part) {
    const int64_t threads = static_cast<int64_t>(a.M) * ceil_div(a.N, 4);
    hipLaunchKernelGGL(mx_join_kernel<BF16>, dim3(static_cast<unsigned>(ceil_div(threads, 256))), dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  return e;
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

// Rows of `cols` elements fit into the stride, and the strided matrix into the address space.
bool bad_ld(int64_t ld, int64_t rows, int64_t cols) { return ld < cols || ld > INT64_MAX / 8 / (rows < 1 ? 1 : rows); }

fconv_status check_matrix(const void* x, int64_t ld, int32_t rows, int32_t cols, int32_t dtype) {
  if (rows < 0 || cols < 1 || bad_ld(ld, rows, cols)) return FCONV_ERR_INVALID_ARG;
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
  const int es = dtype == FCONV_BF16 ? 2 : 4;
  const auto kernel = es == 4                          ? mx_quantize_kernel<false, false>
                      : streams(x, ldx, rows, es) ? mx_quantize_kernel<true, true>
                                                  : mx_quantize_kernel<true, false>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, s, src, ldx * es, static_cast<int64_t>(rows), cols, kt, ks,
                     codes, scales);
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
  const int es = dtype == FCONV_BF16 ? 2 : 4;
  const auto kernel = es == 4                          ? mx_dequantize_kernel<false, false>
                      : streams(y, ldy, rows, es) ? mx_dequantize_kernel<true, true>
                                                  : mx_dequantize_kernel<true, false>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, s, v.codes, v.scales, static_cast<int64_t>(rows), cols, kt, ks,
                     static_cast<char*>(y), ldy * es);
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
  choose_kernel(p);
  if (p->kernel != kFewRaw && p->kernel != kRows)
    p->ws_x = (codes_bytes(d.M, d.K) + scales_bytes(d.M, d.K) + 255) / 256 * 256;
  p->ws_bytes = p->ws_x;
  if (p->ranges > 1) p->ws_bytes += static_cast<size_t>(p->ranges) * d.M * ceil_div(d.N, 4) * 16;
  // What quantises x itself has no form for one that is quantised.
  p->kernel_mx = p->kernel == kFewRaw ? kFew : p->kernel != kRows ? p->kernel : d.M <= 64 ? kFew : kTile128;
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
  if ((args->x && bad_ld(args->ldx, d.M, d.K)) || bad_ld(args->ldy, d.M, d.N)) return FCONV_ERR_INVALID_ARG;
  // An x that comes quantised needs no place in the workspace.
  const int kernel = args->x ? p->kernel : p->kernel_mx;
  const bool by_itself = args->x && (kernel == kFewRaw || kernel == kRows);
  const size_t ws = args->x ? p->ws_bytes : p->ws_bytes - p->ws_x;
  if (ws > 0 && (!args->workspace || args->workspace_bytes < p->ws_bytes)) return FCONV_ERR_WORKSPACE;
  if (!aligned(args->x, p->esize) || !aligned(args->y, p->esize) || !aligned(args->x_mx, 16) ||
      !aligned(args->w_mx, 16) || (p->op_bias && !aligned(args->bias, 4)) ||
      (ws > 0 && !aligned(args->workspace, 16)))
    return FCONV_ERR_MISALIGNED;
  const size_t yb = span(d.M, d.N, args->ldy, p->esize);
  const size_t xq = codes_bytes(d.M, d.K) + scales_bytes(d.M, d.K);
  const size_t xb = args->x ? span(d.M, d.K, args->ldx, p->esize) : 0;
  const size_t wb = codes_bytes(d.N, d.K) + scales_bytes(d.N, d.K);
  const size_t wsb = ws > 0 ? p->ws_bytes : 0;
  const void* in[4] = {args->x, args->x_mx, args->w_mx, p->op_bias ? args->bias : nullptr};
  const size_t in_bytes[4] = {xb, xq, wb, static_cast<size_t>(d.N) * 4};
  for (int i = 0; i < 4; ++i)
    if (overlaps(args->y, yb, in[i], in_bytes[i]) || overlaps(args->workspace, wsb, in[i], in_bytes[i]))
      return FCONV_ERR_INVALID_ARG;
  if (overlaps(args->y, yb, args->workspace, wsb)) return FCONV_ERR_INVALID_ARG;

  hipStream_t s = static_cast<hipStream_t>(stream);
  const void* xmx = args->x_mx;
  if (args->x && !by_itself) {
    if (launch_quantize(args->x, args->ldx, d.M, d.K, d.dtype, args->workspace, s) != hipSuccess)
      return FCONV_ERR_DEVICE;
    xmx = args->workspace;
  }
  MxArgs a = {};
  a.w = view(args->w_mx, d.N, d.K);
  if (xmx) a.x = view(xmx, d.M, d.K);
  if (by_itself) {
    a.raw = static_cast<const char*>(args->x);
    a.ldx_bytes = args->ldx * p->esize;
  }
  a.K = d.K;
  a.ranges = p->ranges;
  if (p->ranges > 1) {
    a.part = reinterpret_cast<float*>(static_cast<char*>(args->workspace) + p->ws_x);
    a.ldp = ceil_div(d.N, 4) * 4;
  }
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
  const hipError_t e = d.dtype == FCONV_BF16 ? launch_product<true>(p, a, kernel, s)
                                             : launch_product<false>(p, a, kernel, s);
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

const char* fconv_mx_plan_kernel_name(fconv_mx_plan p) { return p ? fconv::kKernelNames[p->kernel] : nullptr; }
const char* fconv_mx_plan_quantized_kernel_name(fconv_mx_plan p) {
  return p ? fconv::kKernelNames[p->kernel_mx] : nullptr;
}

fconv_status fconv_mx_plan_destroy(fconv_mx_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
