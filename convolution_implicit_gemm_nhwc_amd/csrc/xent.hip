// Linear softmax cross entropy on gfx950 (CDNA4), its gradient, and their
// C ABI (include/fconv_xent.h).
//
//   z = h w^T     loss = lse - z[target]     g = dloss (softmax z - onehot)
//   dh = g w      dw = g^T h
//
// The logits never reach memory.  Forward: each tile of z leaves, per token,
// its largest logit and the sum of exponentials below it (and the target's
// logit where the tile holds it); a second kernel joins the tiles.  Backward:
// the vocabulary is taken in pieces; a piece's z is computed again, becomes
// q = softmax z - onehot in the epilogue, and q feeds both products:
//   dh[t] = dloss[t] sum_v q[t, v] w[v]
//   dw[v] = c sum_t q[t, v] (r[t] h[t]),   c = max |dloss|, r = dloss / c
// Tokens whose target is ignored have no gradient: the others are gathered
// first, so no product spends time on them and nothing they hold (NaN,
// infinities) reaches a sum.
//
// Roundings of bf16 inputs' gradients.  q is rounded to bf16 (the matrix
// cores' type), by half a step, 2^-8 of itself, at most.  dloss q, at the same cost,
// would be off by as much and, with the mean's equal dloss, by the same factor
// in every token (measured on 32 tokens of 1000 classes: error of dw 0.0037 against
// 0.0018).  Two bf16 parts of q would take 10 T D V operations instead of 6; the
// gradients' error against 64 bits is 0.0017 of their norm either way, that of
// their own rounding to bf16 (perf/operators.py's cases, with q in fp32 and here).
// r h is rounded to bf16 too, exactly where all dloss are equal.
//
// Every product has the form C[b, a] = sum_k A(a, k) B(b, k) with a contiguous
// in C: the matrix core then ends with four consecutive a per lane.
//   logits  a = v, b = t, k = d: A = w, B = h, both with k contiguous
//   dh      a = d, b = t, k = v: A = w with a contiguous, B = g
//   dw      a = d, b = v, k = t: A = h, B = g, a and b contiguous
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>
#include <type_traits>

#include "fconv_xent.h"

namespace fconv {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
// What the launches' grids and their whole numbers hold.  Tiles of 64 x 64 logits:
// those of 128 are counted in 32 bits.  Elements of dh, and of a piece's w: a thread
// of a join takes four of them, and a launch's threads stay below 2^32.  Tokens:
// tiles of 64 in grid.y.
constexpr int64_t kMaxTiles = 1ll << 28, kMaxSum = 1ll << 33, kMaxGridY = 65535;
constexpr int64_t kMaxLd = 1 << 21;
constexpr int32_t kMaxD = 1 << 20, kMaxTV = 1 << 24;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// Which index of an operand is contiguous in memory: the sum's (element
// (r, k) at r * ld + k) or the row's (at k * ld + r).
enum Order { kSum, kRow };

struct Operand {
  const char* p;
  int64_t ld;     // elements
  int64_t width;  // kRow: readable elements of a row
};

// kEpiStream: kEpiOut past the caches.  kEpiAdd: kEpiPart added to what is there.
enum Epilogue { kEpiLse, kEpiGrad, kEpiOut, kEpiPart, kEpiStream, kEpiAdd };
constexpr bool is_out(Epilogue e) { return e == kEpiOut || e == kEpiStream; }
constexpr bool is_part(Epilogue e) { return e == kEpiPart || e == kEpiAdd; }

struct GemmArgs {
  Operand a, b;
  int32_t na, nb, nk;
  // Number of live tokens (device), replacing nb (kSum order of b) or nk
  // (kRow order of b); NULL if there is none.
  const int32_t* n_live;
  int32_t ranges;   // of k; the partial sums of each go out apart
  // kEpiLse: partial (max, sum) at [tile of a][ld_out + b]; kEpiGrad: g;
  // kEpiOut: C; kEpiPart, kEpiAdd: fp32 C of this range at range * part_stride,
  // whose rows are whole 16 bytes.
  char* out;
  int64_t ld_out;
  int64_t part_stride;        // elements between ranges
  const int32_t* row_map;     // kEpiOut: row of C for b (-1 - row: zeros go there), or NULL
  // kEpiLse / kEpiGrad
  const int64_t* target;      // kEpiLse: [nb]
  float* target_logit;        // kEpiLse: [nb]
  const int32_t* live_target; // kEpiGrad: [nb], -1 where out of range
  const float* lse;           // kEpiGrad: [nb]
  const float* scale;         // kEpiOut: factor of row b, at b * scale_step
  int32_t scale_step;
  int32_t v0;                 // vocabulary index of a = 0
  int32_t na_pad;             // kEpiGrad: columns of g written, zeros past na
};

__device__ inline uint16_t f32_to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));  // round to nearest even
}

// Four consecutive elements (`live` of them exist) at p.
template <typename E>
__device__ inline void store4(char* p, f32x4 t, int live) {
  if constexpr (sizeof(E) == 2) {
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

// The tiles of two matrix tiles side by side in bf16: t0 holds this lane's four
// a of the first, t1 of the second.  Rows of 16 lanes exchange halves, so that
// a lane ends with eight consecutive a and the 16 lanes of each b write 64
// bytes at once: those of tile q % 2 from a = 8 (q / 2) on.  STREAM: past the caches.
template <bool STREAM = false>
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
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  const u32x4 x = {v[0], v[1], v[2], v[3]};
  if constexpr (STREAM)
    __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(p));
  else
    *reinterpret_cast<u32x4*>(p) = x;
}
__device__ inline int pair_at(int q) { return (q & 1) * 16 + (q >> 1) * 8; }

// What exponents are taken relative to: the maximum, or 0 where it is
// infinite (inf - inf would be NaN; exp(inf) = inf and exp(-inf) = 0 are right).
__device__ inline float base_of(float m) { return __builtin_fabsf(m) < __builtin_inff() ? m : 0.0f; }
__device__ inline float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// exp(x - base), given base * log2 e: one operation less of every logit.  The
// rounding of base * log2 e is at most one of base itself, as lse's own.
__device__ inline float exp_from(float x, float base2) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2e, -base2));
}

// A token's factor of dh.  An infinite dloss has NaN gradients: times a sum of
// products of both signs it would be an infinity here and a NaN there.
__device__ inline float dh_factor(float dloss) {
  return __builtin_fabsf(dloss) < __builtin_inff() ? dloss : __builtin_nanf("");
}

// f over the four lanes l, l ^ 16, l ^ 32, l ^ 48, the same in all of them.
template <typename F>
__device__ inline float across(float x, F f) {
  const uint32_t a = __builtin_bit_cast(uint32_t, x);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t b = __builtin_bit_cast(uint32_t, f(__builtin_bit_cast(float, static_cast<uint32_t>(p[0])),
                                                    __builtin_bit_cast(float, static_cast<uint32_t>(p[1]))));
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return f(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
}

// base * log2 e for exp_from.  Past 2^126 the product would leave fp32: there
// the base is taken off the logits first, and what is left counts from 0.
template <int NI, int NJ>
__device__ inline float base2_of(f32x4 (&z)[NI][NJ], int j, float base) {
  if (__builtin_fabsf(base) >= 0x1p126f) {
#pragma unroll
    for (int i = 0; i < NI; ++i) z[i][j] -= base;
    base = 0.0f;
  }
  return base * kLog2e;
}

// (m, s) of two sets of logits joined; s counts from base_of(m).
__device__ inline void join(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2), b = base_of(mm);
  // An empty or all -inf set has s = 0, whose factor must not be NaN or inf.
  const float f1 = exp_of(base_of(m) - b), f2 = exp_of(base_of(m2) - b);
  s = (s == 0.0f ? 0.0f : s * f1) + (s2 == 0.0f ? 0.0f : s2 * f2);
  m = mm;
}


// What a workgroup does with its tile of C: NI x NJ matrix tiles per wave, of
// which this lane holds a = a_of(i) .. + 3 of b = b_of(j); ra x rb of the EDGE^2
// tile exist.  Two waves (wa) share the tile's b.  Nothing is asked element by
// element in a whole tile: with such questions the tile's end took several
// times as long as its instructions.
template <Epilogue EPI, int NJ>
struct PerB {  // what it has to know of each b
  int at[NJ];    // kEpiLse, kEpiGrad: the target's place in the tile, or none; kEpiOut: the row
  float f[NJ];   // kEpiGrad: lse; kEpiOut: factor
};
template <Epilogue EPI, int NJ, typename FB>
__device__ inline PerB<EPI, NJ> load_per_b(const GemmArgs& g, int64_t a0, int64_t b0, int ra, int rb, FB b_of) {
  PerB<EPI, NJ> p;
  int64_t b[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) b[j] = b0 + min(b_of(j), rb - 1);
  if constexpr (EPI == kEpiLse) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t t = g.target[b[j]] - g.v0 - a0;
      p.at[j] = t >= 0 && t < ra ? static_cast<int>(t) : -1;
    }
  } else if constexpr (EPI == kEpiGrad) {
    // All loads at once: asking for lse where the target is one took eight in a row.
    int t[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      t[j] = g.live_target[b[j]];
      p.f[j] = g.lse[b[j]];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      p.at[j] = static_cast<int>(t[j] - g.v0 - a0);
      p.f[j] = t[j] < 0 ? __builtin_nanf("") : p.f[j];
    }
  } else if constexpr (is_out(EPI)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      p.at[j] = static_cast<int>(b[j]);
      p.f[j] = g.scale[b[j] * g.scale_step];
    }
    if (g.row_map) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) p.at[j] = g.row_map[b[j]];
    }
  }
  return p;
}
// The loads are done before what follows.
template <Epilogue EPI, int NJ>
__device__ inline void have_per_b(PerB<EPI, NJ>& p) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if constexpr (!is_part(EPI)) asm volatile("" : "+v"(p.at[j]));
    if constexpr (!is_part(EPI) && EPI != kEpiLse) asm volatile("" : "+v"(p.f[j]));
  }
}

template <typename E, Epilogue EPI, int NI, int NJ, int EDGE, typename FA, typename FB>
__device__ inline void epilogue(const GemmArgs& g, f32x4 (&acc)[NI][NJ], const PerB<EPI, NJ>& per, int64_t a0,
                                int64_t b0, int ra, int rb, int tile_a, int range, int wa, int q, FA a_of,
                                FB b_of, float2* red) {
  constexpr int ES = sizeof(E);
  const bool whole = ra == EDGE;
  if constexpr (EPI == kEpiLse) {
    if (!whole) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (a_of(i) + e >= ra)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j][e] = -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int b = b_of(j);
      const int at = b < rb ? per.at[j] : -1;
      if (at >= 0) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (a_of(i) + e == at) g.target_logit[b0 + b] = acc[i][j][e];
      }
      float m = acc[0][j][0], s = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, acc[i][j][e]);
      // The four lanes of a token agree on the largest first: their sums then add
      // up without another exponential.
      m = across(m, [](float x, float y) { return fmaxf(x, y); });
      const float base2 = base2_of(acc, j, base_of(m));
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s += exp_from(acc[i][j][e], base2);
      s = across(s, [](float x, float y) { return x + y; });
      if (q == 0) red[wa * EDGE + b] = make_float2(m, s);
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(rb)) {
      const float2 p0 = red[threadIdx.x], p1 = red[EDGE + threadIdx.x];
      float m = p0.x, s = p0.y;
      join(m, s, p1.x, p1.y);
      reinterpret_cast<float2*>(g.out)[tile_a * g.ld_out + b0 + threadIdx.x] = make_float2(m, s);
    }
  } else if constexpr (EPI == kEpiGrad) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int b = b_of(j);
      if (b >= rb) continue;
      const int at = per.at[j];
      const float lse2 = base2_of(acc, j, per.f[j]);
      char* row = g.out + ((b0 + b) * g.ld_out + a0) * ES;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = exp_from(acc[i][j][e], lse2);
      if (at >= 0 && at < ra) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (a_of(i) + e == at) acc[i][j][e] -= 1.0f;
      }
      if (whole) {
        if constexpr (ES == 2) {
#pragma unroll
          for (int i = 0; i < NI; i += 2)
            store_pair(row + (a_of(i) - 4 * q + pair_at(q)) * ES, acc[i][j], acc[i + 1][j]);
        } else {
#pragma unroll
          for (int i = 0; i < NI; ++i) store4<E>(row + a_of(i) * ES, acc[i][j], 4);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (a0 + a_of(i) >= g.na_pad) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (a_of(i) + e >= ra) acc[i][j][e] = 0.0f;
          store4<E>(row + a_of(i) * ES, acc[i][j], 4);
        }
      }
    }
  } else {
    using O = std::conditional_t<is_out(EPI), E, float>;
    // kEpiAdd: what is there, the next b's on its way while this one is added to
    // (rows past the last one, and places past a row's end, read others again).
    f32x4 old[EPI == kEpiAdd ? 2 : 1][NI];
    auto load_old = [&](int j) __attribute__((always_inline)) {
      const char* p = g.out + (range * g.part_stride + (b0 + min(b_of(j), rb - 1)) * g.ld_out + a0) * 4;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        old[j & 1][i] = *reinterpret_cast<const f32x4*>(p + (a_of(i) < ra ? a_of(i) : 0) * 4);
    };
    if constexpr (EPI == kEpiAdd) load_old(0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (EPI == kEpiAdd) {
        if (j + 1 < NJ) load_old(j + 1);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i][j] += old[j & 1][i];
      }
      const int b = b_of(j);
      if (b >= rb) continue;
      int64_t row = b0 + b;
      float scale = 1.0f;
      if constexpr (is_out(EPI)) {
        row = per.at[j];
        scale = per.f[j];
        if (row < 0) {
          row = -1 - row;
#pragma unroll
          for (int i = 0; i < NI; ++i) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
      char* out = g.out + ((is_part(EPI) ? range * g.part_stride : 0) + row * g.ld_out + a0) *
                              static_cast<int64_t>(sizeof(O));
      if (whole) {
        if constexpr (sizeof(O) == 2) {
#pragma unroll
          for (int i = 0; i < NI; i += 2)
            store_pair<EPI == kEpiStream>(out + (a_of(i) - 4 * q + pair_at(q)) * sizeof(O), acc[i][j] * scale,
                                          acc[i + 1][j] * scale);
        } else {
#pragma unroll
          for (int i = 0; i < NI; ++i) store4<O>(out + a_of(i) * sizeof(O), acc[i][j] * scale, 4);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int n = ra - a_of(i);
          if (n > 0) store4<O>(out + a_of(i) * sizeof(O), acc[i][j] * scale, n);
        }
      }
    }
  }
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16* lds_v4i16_t;

constexpr uint32_t kOutOfRange = 0x80000000u;  // buffer offset past every extent: reads 0
constexpr int kBufferDword3 = 0x00020000;      // raw buffer descriptor, gfx9 family

__device__ inline __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const uint32_t n = bytes > 0x7fffffff ? 0x7fffffffu : static_cast<uint32_t>(bytes < 0 ? 0 : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(n), kBufferDword3);
}

// Place of 16-byte pieces in a row k of H bf16 in LDS (xor of their number), so
// that the rows that one transposed read touches lie on different banks.
template <int H>
__device__ inline int row_swz(int k) {
  return H == 128 ? ((k & 3) << 1) | (((k >> 3) & 1) << 3) : (((k & 3) << 1) ^ (((k >> 3) & 1) << 1)) & 7;
}

// Eight consecutive k of row a of an operand in kRow order: lane i's element e
// of a 16-lane group is element i % 4 of the 8 bytes addressed by the group's
// lane 4 e + i / 4; `p` is this lane's address, `next` bytes on are four rows.
__device__ inline bf16x8 read_transposed(const char* p, int next) {
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t)p);
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t)(p + next));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ------------------------------------------------------------ general kernel
//
// Any type, alignment and stride: 64 x 64 tiles, four waves of 32 x 32, slabs
// of 128 bytes of k staged through registers into one of two LDS buffers
// (rows of 128 + 16 bytes, so that fragment reads spread over the banks).  A
// fragment is eight consecutive k of a row; for fp32 the eight 16x16x4
// products take one of them each, in both operands alike.  An operand in kRow
// order is transposed on its way out of LDS for bf16 (the tiled kernel's order
// and reads), on its way in for fp32.
template <typename E>
struct Gen {
  static constexpr int ES = sizeof(E);
  static constexpr int SLAB = 128 / ES;
  static constexpr int PITCH = 144;
  static constexpr int BUF = 64 * PITCH;
};

// 32 bytes of an operand's slab for this thread.
template <typename E, Order O>
__device__ inline void gen_load(const Operand& op, int64_t row0, int rows, int64_t k0, int64_t k1,
                                E v[32 / sizeof(E)]) {
  constexpr int N = 32 / sizeof(E);
  const int tid = threadIdx.x;
  const char* p;
  int n;
  if constexpr (O == kSum) {
    const int r = tid >> 2;
    const int64_t k = k0 + (tid & 3) * N;
    n = r < rows ? static_cast<int>(min(k1 - k, static_cast<int64_t>(N))) : 0;
    p = op.p + ((row0 + r) * op.ld + k) * static_cast<int64_t>(sizeof(E));
  } else {
    constexpr int TPK = 64 / N;  // threads per k
    const int64_t k = k0 + tid / TPK;
    const int c = (tid % TPK) * N;
    n = k < k1 ? min(rows - c, N) : 0;
    p = op.p + (k * op.ld + row0 + c) * static_cast<int64_t>(sizeof(E));
  }
  if (n >= N) {
    __builtin_memcpy(v, p, 32);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = static_cast<E>(0.0f);
      if (i < n) __builtin_memcpy(&v[i], p + i * sizeof(E), sizeof(E));
    }
  }
}

template <typename E, Order O>
__device__ inline void gen_write(char* buf, const E v[32 / sizeof(E)]) {
  constexpr int N = 32 / sizeof(E);
  const int tid = threadIdx.x;
  if constexpr (O == kSum) {
    __builtin_memcpy(buf + (tid >> 2) * Gen<E>::PITCH + (tid & 3) * 32, v, 32);
  } else if constexpr (sizeof(E) == 2) {
    const int k = tid >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_memcpy(buf + k * 128 + (((2 * (tid & 3) + i) ^ row_swz<64>(k)) << 4), v + 8 * i, 16);
  } else {
    constexpr int TPK = 64 / N;
    const int k = tid / TPK, c = (tid % TPK) * N;
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<E*>(buf + (c + i) * Gen<E>::PITCH + k * sizeof(E)) = v[i];
  }
}

// Fragment of rows row0 + lane % 16, k from kk + 8 (lane / 16) on.
template <typename E, Order O>
__device__ inline auto gen_read(const char* buf, int row0, int kk) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  if constexpr (O == kRow && sizeof(E) == 2) {
    const int k = kk + 8 * q + (r >> 2);
    return read_transposed(buf + k * 128 + (((row0 / 8 + ((r & 3) >> 1)) ^ row_swz<64>(k)) << 4) + (r & 1) * 8, 512);
  } else {
    std::conditional_t<sizeof(E) == 2, bf16x8, f32x8> f;
    __builtin_memcpy(&f, buf + (row0 + r) * Gen<E>::PITCH + (kk + 8 * q) * sizeof(E), 8 * sizeof(E));
    return f;
  }
}

__device__ inline f32x4 mma8(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x4 mma8(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// LDS of a workgroup: two buffers of both operands, then the epilogue's.
template <typename E>
struct GenLds {
  __attribute__((aligned(16))) char buf[2][2][Gen<E>::BUF];
  float2 red[2 * 64];
};

// Tile (x, y) of range z.
template <typename E, Order OA, Order OB, Epilogue EPI>
__device__ inline void gen_tile(const GemmArgs& g, GenLds<E>& lds, int x, int y, int z) {
  using G = Gen<E>;
  using Frag = std::conditional_t<sizeof(E) == 2, bf16x8, f32x8>;
  auto& buf = lds.buf;
  const int live = g.n_live ? *g.n_live : 0;
  const int nb = g.n_live && OB == kSum ? live : g.nb;
  const int nk = g.n_live && OB == kRow ? live : g.nk;
  const int64_t a0 = static_cast<int64_t>(x) * 64, b0 = static_cast<int64_t>(y) * 64;
  if (b0 >= nb) return;
  const int ra = static_cast<int>(min<int64_t>(g.na - a0, 64)), rb = static_cast<int>(min<int64_t>(nb - b0, 64));
  const int64_t per = round_up(ceil_div(nk, g.ranges), G::SLAB);
  const int64_t k0 = z * per;
  const int64_t k1 = min<int64_t>(nk, k0 + per);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave & 1, wb = wave >> 1, r = lane & 15, q = lane >> 4;

  f32x4 acc[2][2] = {};
  const int slabs = k1 > k0 ? static_cast<int>(ceil_div(k1 - k0, G::SLAB)) : 0;
  // Two slabs are on their way in registers while one is multiplied: with one,
  // a workgroup alone on its CU waited for most of a slab's time.
  E va[2][32 / G::ES], vb[2][32 / G::ES];
  auto load = [&](int s, E(&xa)[32 / G::ES], E(&xb)[32 / G::ES]) __attribute__((always_inline)) {
    if (s >= slabs) return;
    gen_load<E, OA>(g.a, a0, ra, k0 + s * static_cast<int64_t>(G::SLAB), k1, xa);
    gen_load<E, OB>(g.b, b0, rb, k0 + s * static_cast<int64_t>(G::SLAB), k1, xb);
  };
  auto step = [&](int s, char* ba, char* bb, E(&xa)[32 / G::ES], E(&xb)[32 / G::ES]) __attribute__((always_inline)) {
    gen_write<E, OA>(ba, xa);
    gen_write<E, OB>(bb, xb);
    __syncthreads();
    load(s + 2, xa, xb);
#pragma unroll
    for (int kk = 0; kk < G::SLAB; kk += 32) {
      Frag fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = gen_read<E, OA>(ba, wa * 32 + 16 * i, kk);
        fb[i] = gen_read<E, OB>(bb, wb * 32 + 16 * i, kk);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mma8(fa[i], fb[j], acc[i][j]);
    }
  };
  load(0, va[0], vb[0]);
  load(1, va[1], vb[1]);
  for (int s = 0; s < slabs; s += 2) {
    step(s, buf[0][0], buf[0][1], va[0], vb[0]);
    if (s + 1 < slabs) step(s + 1, buf[1][0], buf[1][1], va[1], vb[1]);
  }

  auto b_of = [&](int j) { return wb * 32 + 16 * j + r; };
  const auto per_b = load_per_b<EPI, 2>(g, a0, b0, ra, rb, b_of);
  epilogue<E, EPI, 2, 2, 64>(
      g, acc, per_b, a0, b0, ra, rb, x, z, wa, q, [&](int i) { return wa * 32 + 16 * i + 4 * q; }, b_of, lds.red);
}

template <typename E, Order OA, Order OB, Epilogue EPI>
__global__ __launch_bounds__(256) void xent_gen_kernel(GemmArgs g) {
  __shared__ GenLds<E> lds;
  gen_tile<E, OA, OB, EPI>(g, lds, blockIdx.x, blockIdx.y, blockIdx.z);
}

// Both gradients in one launch: the first workgroups take dh's tiles and
// ranges, the others dw's.
template <typename E, Epilogue EPI_DH>
__global__ __launch_bounds__(256) void xent_gen_grads_kernel(GemmArgs dh, GemmArgs dw) {
  __shared__ GenLds<E> lds;
  const int ta = (dh.na + 63) / 64, n_dh = ta * ((dh.nb + 63) / 64) * dh.ranges;
  int i = blockIdx.x;
  if (i < n_dh) {
    gen_tile<E, kRow, kSum, EPI_DH>(dh, lds, i % ta, i / ta % ((dh.nb + 63) / 64), i / ta / ((dh.nb + 63) / 64));
  } else {
    i -= n_dh;
    gen_tile<E, kRow, kRow, kEpiOut>(dw, lds, i % ta, i / ta, 0);
  }
}

// dh of at most 16 MT tokens over a short vocabulary, sixteen d of all tokens for
// a workgroup, so that no partial sums go out and no launch joins them: its four
// waves take turns at steps of 32 v and add their sums in LDS, in order.  A lane
// picks its eight v of a column out of memory one by one, from any row distance
// and alignment; rows of g are whole 64s, zeros past the vocabulary.
template <typename E, int MT>
__device__ inline void few_dh(const GemmArgs& g, f32x4* sums, int d0) {
  using Frag = std::conditional_t<sizeof(E) == 2, bf16x8, f32x8>;
  constexpr int ES = sizeof(E), STEPS = 2;  // of a turn, whose loads are in flight together
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int steps = (g.nk + 31) / 32;
  const int64_t row = g.a.ld * ES;
  // Columns past the last one read it again; they are not stored.
  const char* wp = g.a.p + static_cast<int64_t>(min(d0 + r, g.na - 1)) * ES;
  const char* gp[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
    gp[j] = g.b.p + (static_cast<int64_t>(min(16 * j + r, g.nb - 1)) * g.b.ld + 8 * q) * ES;
  struct Turn {
    E a[STEPS][8];
    Frag b[STEPS][MT];
  };
  auto load = [&](Turn& x, int first) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int step = first + 4 * s;
      if (step >= steps) break;  // uniform
      const int v = 32 * step + 8 * q;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        __builtin_memcpy(&x.a[s][e], wp + static_cast<int64_t>(min(v + e, g.nk - 1)) * row, ES);
#pragma unroll
      for (int j = 0; j < MT; ++j) __builtin_memcpy(&x.b[s][j], gp[j] + static_cast<int64_t>(step) * 32 * ES, 8 * ES);
    }
  };
  f32x4 acc[MT] = {};
  auto multiply = [&](const Turn& x, int first) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int step = first + 4 * s;
      if (step >= steps) break;
      E v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 32 * step + 8 * q + e < g.nk ? x.a[s][e] : static_cast<E>(0.0f);
      Frag a;
      __builtin_memcpy(&a, v, sizeof(a));
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[j] = mma8(a, x.b[s][j], acc[j]);
    }
  };
  Turn now, next;
  constexpr int NEXT = 4 * STEPS;
  int first = wave;
  if (first < steps) load(now, first);
  for (; first < steps; first += 2 * NEXT) {
    if (first + NEXT < steps) load(next, first + NEXT);
    multiply(now, first);
    if (first + NEXT >= steps) break;
    if (first + 2 * NEXT < steps) load(now, first + 2 * NEXT);
    multiply(next, first + NEXT);
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) sums[(wave * MT + j) * 64 + lane] = acc[j];
  __syncthreads();
  const int t = 16 * wave + r, d = d0 + 4 * q;
  if (wave >= MT || t >= g.nb || d >= g.na) return;
  f32x4 sum = sums[wave * 64 + lane];
#pragma unroll
  for (int x = 1; x < 4; ++x) sum += sums[(x * MT + wave) * 64 + lane];
  sum *= g.scale[t];
  if (g.row_map[t] < 0) sum = f32x4{0.f, 0.f, 0.f, 0.f};
  store4<E>(g.out + (t * g.ld_out + d) * static_cast<int64_t>(ES), sum, g.na - d);
}

// The first workgroups take dh, the others (if dw is wanted) dw's tiles.
template <typename E, int MT>
__global__ __launch_bounds__(256) void xent_few_grads_kernel(GemmArgs dh, GemmArgs dw) {
  __shared__ GenLds<E> lds;
  static_assert(sizeof(lds.buf) >= 4 * MT * 64 * sizeof(f32x4), "the sums fit");
  const int n_dh = (dh.na + 15) / 16, i = static_cast<int>(blockIdx.x) - n_dh;
  if (i < 0) {
    few_dh<E, MT>(dh, reinterpret_cast<f32x4*>(&lds.buf[0][0][0]), static_cast<int>(blockIdx.x) * 16);
  } else {
    const int ta = (dw.na + 63) / 64;
    gen_tile<E, kRow, kRow, kEpiOut>(dw, lds, i % ta, i / ta, 0);
  }
}

// -------------------------------------------------------------- tiled kernel
//
// bf16, rows and their length multiples of 16 bytes.  A workgroup owns a
// (2 H) x (2 H) tile of C in four quadrants; NW waves share each quadrant, two
// along a, NW / 2 along b.  A slab is 64 k of both operands: four half tiles,
// copied buffer->LDS, in one of two sets of buffers.  A slab takes four
// phases, one quadrant each:
//   phase   reads (LDS)                copies for the slab after next   products
//   0       A0 but two                 -                                C00
//   1       B1, two fragments of A1    A0, B0 (their readers are done)  C01
//   2       the rest of A1             B1                               C11
//   3       next slab's B0, two of A0  A1                               C10
// A phase is two steps between barriers: a wave reads fragments and starts
// copies in one, multiplies in the other.  With eight waves the four of a = 1
// run one step behind the others, so that on every SIMD one wave multiplies
// while the other reads.  A step of products takes 256 cycles, and LDS gives
// 128 bytes a cycle: six fragments for each of four waves take 192, so the
// reads are spread evenly, 6 a phase (12, 4, 8, 0 made the steps of phases 0
// and 2 wait for LDS: 2.98 against 2.85 million cycles of 8192 x 4096 x 32768
// logits; the clock falls meanwhile, so less is won in time).  A copy has more
// than a slab's time to arrive; the waits stand one phase before the first
// reads, in phase 2 for A0 and B0 of the next slab and in phase 0 for this
// one's others.
//
// Measured: 8192 x 4096 x 32768 logits 1.60 to 1.68 ms from box to box, 1.31 to
// 1.38 PFLOP/s; the matrix cores are busy 71% of the cycles, at 1.8 GHz: power
// bounds the clock.  Of its gradient's products the logits 66% (q is written), dh
// 66%, dw 71%.
//
// LDS order.  kSum: rows of 64 k (128 bytes), the 16-byte piece c of row r at
// c ^ (r % 8): eight consecutive lanes of a fragment read hit eight places.
// kRow: rows k of H elements; fragments come from the transposed read
// (ds_read_b64_tr_b16: lane i's element e of a 16-lane group is element i % 4
// of the 8 bytes addressed by the group's lane 4 e + i / 4), pieces swizzled
// by swz(k) so that the rows that one read touches lie on different banks.
// One operand of a workgroup: where its half tiles come from, and this lane's
// places in them.
template <Order O, int H, int NW>
struct Feed {
  const char* base;  // of the tile's first element of the next slab to copy
  int64_t left;      // bytes readable from base
  int64_t step;      // bytes from slab to slab
  int krem;          // k left from base (kSum)
  uint32_t off[2][2];  // per half and copy of this wave
  int chunk;           // kSum: first k of this lane's piece

  __device__ void init(const Operand& op, int wave, int lane) {
    if constexpr (O == kSum) {
      step = 128;
      chunk = ((lane & 7) ^ (lane >> 3)) * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          off[h][c] = static_cast<uint32_t>(((h * H + (wave * 2 + c) * 8 + (lane >> 3)) * op.ld + chunk) * 2);
    } else {
      step = op.ld * 128;
      krem = 0;
      chunk = 0;
      constexpr int PPR = H / 8, RPC = 64 / PPR;  // pieces of a row, rows of a copy
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int k = (wave * 2 + c) * RPC + lane / PPR;
          off[h][c] = static_cast<uint32_t>((k * op.ld + h * H + ((lane % PPR) ^ row_swz<H>(k)) * 8) * 2);
        }
    }
  }
  // The tile at (row0, k0): `rows` of its rows and k0 .. k1 of the sum exist.
  __device__ void start(const Operand& op, int64_t row0, int64_t rows, int64_t k0, int64_t k1) {
    if constexpr (O == kSum) {
      base = op.p + (row0 * op.ld + k0) * 2;
      // The last row ends with k1, rounded up to whole pieces (their rest is zeros or masked).
      left = ((rows - 1) * op.ld + ((k1 - k0 + 7) & ~7)) * 2;
      krem = static_cast<int>(k1 - k0);
    } else {
      base = op.p + (k0 * op.ld + row0) * 2;
      left = ((k1 - k0 - 1) * op.ld + ((rows + 7) & ~7)) * 2;
    }
  }
  // Copies half h of the next slab into buf (this wave's 2 KiB of it).
  __device__ void copy(int h, char* buf, int wave) const {
    const auto rsrc = make_rsrc(base, left);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t o = off[h][c];
      if (O == kSum && chunk >= krem) o = kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(buf + (wave * 2 + c) * 1024), 16, o, 0, 0, 0);
    }
  }
  __device__ void next() {
    base += step;
    left -= step;
    krem -= 64;
  }
};

// Where this wave finds its fragments in a half tile: N matrix tiles of 16
// rows from row w * 16 N on, two steps of 32 k.
template <Order O, int H, int N>
struct Frags {
  int at[O == kSum ? 2 : N];

  __device__ void init(int w, int lane) {
    const int r = lane & 15, q = lane >> 4;
    if constexpr (O == kSum) {
      at[0] = (w * 16 * N + r) * 128 + ((q ^ (r & 7)) << 4);
      at[1] = (w * 16 * N + r) * 128 + (((q + 4) ^ (r & 7)) << 4);
    } else {
      const int k = 8 * q + (r >> 2);
#pragma unroll
      for (int i = 0; i < N; ++i)
        at[i] = k * 2 * H + (((2 * (w * N + i) + ((r & 3) >> 1)) ^ row_swz<H>(k)) << 4) + (r & 1) * 8;
    }
  }
  __device__ bf16x8 one(const char* buf, int i, int kk) const {
    if constexpr (O == kSum) {
      return *reinterpret_cast<const bf16x8*>(buf + at[kk] + i * 2048);
    } else {
      return read_transposed(buf + at[i] + kk * 64 * H, 8 * H);
    }
  }
};

template <Order OA, Order OB, Epilogue EPI, int H, int NW>
__global__ __launch_bounds__(NW * 64, 2) void xent_tile_kernel(GemmArgs g) {
  constexpr int MI = H / 32, MJ = 2 * H / (16 * NW);  // matrix tiles of a wave in a quadrant
  constexpr int HB = H * 128;                         // bytes of a half tile
  static_assert(HB == NW * 2048, "two copies per wave and half tile");
  // Arrays of their own, so that the compiler sees which copies a read does not
  // meet; few enough for it to follow them all (A0 and B0 go together).
  __shared__ __attribute__((aligned(1024))) char ab0[2 * HB], b01[HB], a01[HB];
  __shared__ __attribute__((aligned(1024))) char ab1[2 * HB], b11[HB], a11[HB];
  __shared__ float2 red[EPI == kEpiLse ? 4 * H : 1];

  const int live = g.n_live ? *g.n_live : 0;
  const int nb = g.n_live && OB == kSum ? live : g.nb;
  const int nk = g.n_live && OB == kRow ? live : g.nk;
  // Workgroups of one XCD (block ids go round the 8 XCDs) take neighbouring
  // tiles: eight rows of them together, so both operands stay in its L2; the
  // ranges of a sum come one after the other.
  const int tiles_a = (g.na + 2 * H - 1) / (2 * H), tiles_b = (nb + 2 * H - 1) / (2 * H);
  const int tiles = tiles_a * tiles_b;
  const int total = tiles * g.ranges, share = (total + 7) / 8;
  const int first_id = (blockIdx.x % 8) * share, end = min(share, total - first_id);
  int slot = blockIdx.x / 8;
  if (slot >= end) return;
  const int all = (nk + 63) / 64, per = (all + g.ranges - 1) / g.ranges;  // slabs: of all ranges, of one
  struct Place {
    int range, ta, ra, rb, slabs;
    int64_t a0, b0, k0, k1;
  };
  auto locate = [&](int id) __attribute__((always_inline)) {
    Place p;
    const int tile = id % tiles;
    const int first = tile / (8 * tiles_a) * 8, rows8 = min(8, tiles_b - first), in = tile % (8 * tiles_a);
    p.range = id / tiles;
    p.ta = in / rows8;
    p.a0 = static_cast<int64_t>(p.ta) * 2 * H;
    p.b0 = static_cast<int64_t>(first + in % rows8) * 2 * H;
    p.ra = static_cast<int>(min<int64_t>(g.na - p.a0, 2 * H));
    p.rb = static_cast<int>(min<int64_t>(nb - p.b0, 2 * H));
    p.k0 = static_cast<int64_t>(p.range) * per * 64;
    p.slabs = max(0, min(per, all - p.range * per));
    p.k1 = min<int64_t>(nk, p.k0 + static_cast<int64_t>(p.slabs) * 64);
    return p;
  };
  Place at = locate(first_id + slot);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave / (NW / 2), wb = wave % (NW / 2);

  f32x4 acc[2 * MI][2 * MJ];
  Feed<OA, H, NW> fa;
  Feed<OB, H, NW> fb;
  fa.init(g.a, wave, lane);
  fb.init(g.b, wave, lane);
  // Past the last slab the copies bring zeros that nobody uses.
  auto advance = [&]() __attribute__((always_inline)) {
    fa.next();
    fb.next();
  };
  // The first two slabs of a tile.
  auto begin = [&](const Place& p) __attribute__((always_inline)) {
    fa.start(g.a, p.a0, OA == kRow ? g.a.width - p.a0 : p.ra, p.k0, p.k1);
    fb.start(g.b, p.b0, OB == kRow ? g.b.width - p.b0 : p.rb, p.k0, p.k1);
    fa.copy(0, ab0, wave);
    fb.copy(0, ab0 + HB, wave);
    fb.copy(1, b01, wave);
    fa.copy(1, a01, wave);
    advance();
    fa.copy(0, ab1, wave);
    fb.copy(0, ab1 + HB, wave);
    fb.copy(1, b11, wave);
    fa.copy(1, a11, wave);
    advance();
  };
  Frags<OA, H, MI> pa;
  Frags<OB, H, MJ> pb;
  pa.init(wa, lane);
  pb.init(wb, lane);
  // Fragments [tile][step] of a half of A, but for the first EARLY tiles' first
  // step of A1, which are read while A0 is in use; and of the halves of B.
  constexpr int EARLY = MI == 4 ? 2 : 0;
  bf16x8 xa[MI][2], xe[EARLY + 1], xb[2][MJ][2];
  auto read_b = [&](bf16x8 (&x)[MJ][2], const char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < MJ; ++j) x[j][kk] = pb.one(buf, j, kk);
  };
  auto read_a_rest = [&](const char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = kk == 0 ? EARLY : 0; i < MI; ++i) xa[i][kk] = pa.one(buf, i, kk);
  };
  auto read_step_ends = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's LDS reads are done
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int i2, int j2, const bf16x8 (&b)[MJ][2]) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j)
          acc[i2 * MI + i][j2 * MJ + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              i2 == 1 && kk == 0 && i < EARLY ? xe[i] : xa[i][kk], b[j][kk], acc[i2 * MI + i][j2 * MJ + j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // b0 holds this slab's B0 and gets nothing; b1 gets B1, then the next slab's B0.
  auto slab = [&](char* ab, char* b1b, char* a1b, const char* ab_next, bf16x8 (&b0)[MJ][2], bf16x8 (&b1)[MJ][2])
                  __attribute__((always_inline)) {
    read_a_rest(ab);
    __builtin_amdgcn_s_waitcnt(0x0F78);  // vmcnt(8): this slab is here
    read_step_ends();
    multiply(0, 0, b0);

    read_b(b1, b1b);
#pragma unroll
    for (int i = 0; i < EARLY; ++i) xe[i] = pa.one(a1b, i, 0);
    fa.copy(0, ab, wave);
    fb.copy(0, ab + HB, wave);
    read_step_ends();
    multiply(0, 1, b1);

    read_a_rest(a1b);
    fb.copy(1, b1b, wave);
    __builtin_amdgcn_s_waitcnt(0x0F7A);  // vmcnt(10): the next slab's A0 and B0 are here
    read_step_ends();
    multiply(1, 1, b1);

    read_b(b1, ab_next + HB);
#pragma unroll
    for (int i = 0; i < EARLY; ++i) xa[i][0] = pa.one(ab_next, i, 0);
    fa.copy(1, a1b, wave);
    advance();
    read_step_ends();
    multiply(1, 0, b0);
  };

  if (at.slabs > 0) begin(at);
  for (;;) {
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i)
#pragma unroll
      for (int j = 0; j < 2 * MJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (at.slabs > 0) {
      __builtin_amdgcn_s_waitcnt(0x0F78);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      read_b(xb[0], ab0 + HB);
#pragma unroll
      for (int i = 0; i < EARLY; ++i) xa[i][0] = pa.one(ab0, i, 0);
      if (NW == 8 && wa == 1) __builtin_amdgcn_s_barrier();
      for (int s = 0; s + 1 < at.slabs; s += 2) {
        slab(ab0, b01, a01, ab1, xb[0], xb[1]);
        slab(ab1, b11, a11, ab0, xb[1], xb[0]);
      }
      if (at.slabs & 1) slab(ab0, b01, a01, ab1, xb[0], xb[1]);
      if (NW == 8 && wa == 0) __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_s_waitcnt(0);  // copies past the last slab have landed
    }
    // The next tile's copies are under way while this one is finished; what the
    // finish has to load comes before them, since loads return in order.
    int l = lane;
    asm volatile("" : "+v"(l));  // computed here, not kept in registers through the products
    const int r = l & 15, q = l >> 4;
    auto a_of = [&](int i) { return i / MI * H + (wa * MI + i % MI) * 16 + 4 * q; };
    auto b_of = [&](int j) { return j / MJ * H + (wb * MJ + j % MJ) * 16 + r; };
    auto per_b = load_per_b<EPI, 2 * MJ>(g, at.a0, at.b0, at.ra, at.rb, b_of);
    have_per_b<EPI, 2 * MJ>(per_b);
    const Place done = at;
    slot += gridDim.x / 8;
    const bool more = slot < end;
    if (more) {
      at = locate(first_id + slot);
      if (at.slabs > 0) begin(at);
    }
    epilogue<__bf16, EPI, 2 * MI, 2 * MJ, 2 * H>(g, acc, per_b, done.a0, done.b0, done.ra, done.rb, done.ta,
                                                 done.range, wa, q, a_of, b_of, red);
    if (!more) break;
  }
}

// ------------------------------------------------------------- few tokens
//
// At most 64 tokens: the logits' time is w's way out of memory, so fragments
// of both operands go straight into registers, from any address, without LDS
// or barriers.  A workgroup owns 32 v and up to 64 tokens (32 with ODD, whose
// fragments take more registers); its four waves take
// turns at steps of 128 bytes of k, the next turn's loads in flight, and add
// their sums in LDS, in order; wave j then finishes tokens 16 j .. + 15.
//
// Forward: a workgroup keeps (max, sum) of its tokens over several such groups
// of v and leaves them once.  Backward: nothing is gathered (three launches
// less are worth more than the ignored tokens' share); ignored tokens get q = 0
// and r h = 0, and the products' rows a sign: see row_map.
// BYTES of elements from p on, in registers.  Loads of 16 bytes whose address is
// no multiple of 4 took more than twice as long (61 tokens of 2895 x 7168: 52 us,
// of 2894 and 2896: 25), so with ODD (some row of bf16 begins between dwords)
// the dwords around the elements are loaded and shifted when they are used.
// Every dword that is read holds one of the elements.
template <int BYTES, bool ODD>
struct Raw;

template <int BYTES>
struct Raw<BYTES, false> {
  typedef uint32_t Words __attribute__((ext_vector_type(BYTES / 4)));
  Words d;
  static __device__ uint32_t shift_of(const char*) { return 0; }
  __device__ void load(const char* p) { __builtin_memcpy(&d, p, BYTES); }
  template <typename F>
  __device__ F get(uint32_t) const {
    return __builtin_bit_cast(F, d);
  }
};

template <int BYTES>
struct Raw<BYTES, true> {
  static constexpr int N = BYTES / 4;
  uint32_t d[N + 1];
  static __device__ uint32_t shift_of(const char* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 2) * 8;
  }
  __device__ void load(const char* p) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const char* q = reinterpret_cast<const char*>(at & ~static_cast<uintptr_t>(3));
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) __builtin_memcpy(&d[4 * i], __builtin_assume_aligned(q + 16 * i, 4), 16);
    d[N] = reinterpret_cast<const uint32_t*>(q)[at & 2 ? N : 0];
  }
  // The elements, given shift_of their address.
  template <typename F>
  __device__ F get(uint32_t shift) const {
    uint32_t v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_alignbit(d[i + 1], d[i], shift);
    F f;
    __builtin_memcpy(&f, v, BYTES);
    return f;
  }
};

// n (8 or more, or less than none) elements of a row of at least eight from p on,
// zeros past them: the last eight, shifted down.  One by one they cost a load and
// a branch each.
template <typename F, typename R, int ES>
__device__ inline F row_end(const char* p, int n) {
  constexpr int N = 2 * ES, PER = 4 / ES;  // dwords of eight elements, elements of a dword
  const char* at = n >= 8 ? p : p + (n - 8) * ES;
  R x;
  x.load(at);
  const F f = x.template get<F>(R::shift_of(at));
  uint32_t d[N];
  __builtin_memcpy(d, &f, sizeof(d));
  const int s = n >= 8 ? 0 : n > 0 ? 8 - n : 8;
#pragma unroll
  for (int by = 8; by >= PER; by /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t v = i + by / PER < N ? d[i + by / PER] : 0u;
      d[i] = s & by ? v : d[i];
    }
  if constexpr (PER == 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t v = d[i] >> 16 | (i + 1 < N ? d[i + 1] << 16 : 0u);
      d[i] = s & 1 ? v : d[i];
    }
  }
  F r;
  __builtin_memcpy(&r, d, sizeof(r));
  return r;
}
// The same of a shorter row.
template <typename F, typename E>
__device__ inline F row_end_short(const char* p, int n) {
  E v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = static_cast<E>(0.0f);
    if (e < n) __builtin_memcpy(&v[e], p + e * sizeof(E), sizeof(E));
  }
  F r;
  __builtin_memcpy(&r, v, sizeof(r));
  return r;
}

struct FewArgs {
  const char* w;
  int64_t ldw;
  const char* h;
  int64_t ldh;
  const int64_t* target;
  int64_t ignore;
  int32_t T, D, V;
  int32_t v0, nv;  // the piece of the vocabulary: w begins with row v0
  // Forward: partial (max, sum) [workgroup][T], and the targets' logits.
  float2* part;
  float* target_logit;
  // Backward.
  const float* lse;
  const float* dloss;
  char* g;
  int64_t ld_g;
  char* rh;  // or NULL
  int64_t ld_rh;
  int32_t* row_map;
  float* live_dloss;
  float* c;
};

template <typename E, bool ODD, Epilogue EPI, int MT>
__global__ __launch_bounds__(256, 2) void xent_few_kernel(FewArgs f) {
  using Frag = std::conditional_t<sizeof(E) == 2, bf16x8, f32x8>;
  constexpr int ES = sizeof(E), NA = 2, STEP = 128 / ES, KK = STEP / 32;
  __shared__ f32x4 sums[4][MT * NA][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int groups = (f.nv + 31) / 32;
  // Tokens from t0 on; workgroups of the same v and other tokens follow on the same XCD (every eighth).
  const int halves = (f.T + 16 * MT - 1) / (16 * MT);
  const int t0 = static_cast<int>(blockIdx.x / 8 % halves) * 16 * MT;
  const int block = blockIdx.x / (8 * halves) * 8 + blockIdx.x % 8, blocks = gridDim.x / halves;
  const int full = f.D / STEP;  // whole steps

  // Rows past T read the last one again; they are not stored.
  const char* hp[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) hp[j] = f.h + (static_cast<int64_t>(min(t0 + 16 * j + r, f.T - 1)) * f.ldh + 8 * q) * ES;
  // This wave's tokens at the end.
  const int t = t0 + 16 * wave + r;
  const bool mine = wave < MT && t < f.T;
  const int64_t tgt = mine ? f.target[t] : -1;
  const int64_t at_v = tgt - f.v0;  // the target's place in this piece
  float run_m = -__builtin_inff(), run_s = 0.0f;

  if constexpr (EPI == kEpiGrad) {
    // r h, and what the products need of each token.  Every workgroup takes a
    // part of the elements.
    const int tl = lane < f.T ? lane : f.T - 1;
    const bool live = f.target[tl] != f.ignore;
    int m = live ? static_cast<int>(__builtin_bit_cast(uint32_t, f.dloss[tl]) & 0x7fffffffu) : 0;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) m = max(m, __shfl_xor(m, x));
    const float c = __builtin_bit_cast(float, m);
    if (blockIdx.x == 0 && wave == 0) {
      if (lane < f.T) {
        f.row_map[lane] = live ? lane : -1 - lane;
        f.live_dloss[lane] = live ? dh_factor(f.dloss[lane]) : 0.0f;
      }
      if (lane == 0) *f.c = c;
    }
    if (f.rh) {
      constexpr int N = 16 / ES;
      const int pieces = static_cast<int>(f.ld_rh / N), total = pieces * f.T;
      for (int i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
        const int row = i / pieces, col = (i - row * pieces) * N;
        const float dl = f.dloss[row];
        const float ratio = c > 0.0f ? dl / c : dl;
        const bool on = f.target[row] != f.ignore;
        E v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          v[k] = static_cast<E>(0.0f);
          if (on && col + k < f.D) {
            __builtin_memcpy(&v[k], f.h + (row * f.ldh + col + k) * ES, ES);
            v[k] = static_cast<E>(ratio * static_cast<float>(v[k]));
          }
        }
        __builtin_memcpy(f.rh + (row * f.ld_rh + col) * ES, v, 16);
      }
    }
  }

  for (int grp = block; grp < groups; grp += blocks) {
    const char* wp[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i)
      wp[i] = f.w + (static_cast<int64_t>(min(32 * grp + 16 * i + r, f.nv - 1)) * f.ldw + 8 * q) * ES;
    f32x4 acc[MT][NA] = {};
    using R = Raw<8 * ES, ODD>;
    struct Turn {
      R a[NA][KK], b[MT][KK];
    };
    uint32_t sa[NA], sb[MT];  // steps are whole dwords: the same in all of them
#pragma unroll
    for (int i = 0; i < NA; ++i) sa[i] = R::shift_of(wp[i]);
#pragma unroll
    for (int j = 0; j < MT; ++j) sb[j] = R::shift_of(hp[j]);
    auto load = [&](Turn& x, int step) __attribute__((always_inline)) {
      const int64_t at = static_cast<int64_t>(step) * 128;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
#pragma unroll
        for (int i = 0; i < NA; ++i) x.a[i][k].load(wp[i] + at + k * 32 * ES);
#pragma unroll
        for (int j = 0; j < MT; ++j) x.b[j][k].load(hp[j] + at + k * 32 * ES);
      }
    };
    auto multiply = [&](const Turn& x) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        Frag a[NA], b[MT];
#pragma unroll
        for (int i = 0; i < NA; ++i) a[i] = x.a[i][k].template get<Frag>(sa[i]);
#pragma unroll
        for (int j = 0; j < MT; ++j) b[j] = x.b[j][k].template get<Frag>(sb[j]);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < NA; ++i) acc[j][i] = mma8(a[i], b[j], acc[j][i]);
      }
    };
    Turn now, next;
    int step = wave;
    if (step < full) load(now, step);
    for (; step < full; step += 8) {
      if (step + 4 < full) load(next, step + 4);
      multiply(now);
      if (step + 4 >= full) break;
      if (step + 8 < full) load(now, step + 8);
      multiply(next);
    }
    if (full % 4 == wave && full * STEP < f.D) {  // the rest of k
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        const int64_t at = static_cast<int64_t>(full) * STEP + k * 32;
        const int n = static_cast<int>(f.D - at) - 8 * q;  // elements of this lane's eight
        auto part = [&](const char* p) __attribute__((always_inline)) {
          return f.D >= 8 ? row_end<Frag, R, ES>(p + at * ES, n) : row_end_short<Frag, E>(p + at * ES, n);
        };
        Frag a[NA], b[MT];
#pragma unroll
        for (int i = 0; i < NA; ++i) a[i] = part(wp[i]);
#pragma unroll
        for (int j = 0; j < MT; ++j) b[j] = part(hp[j]);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < NA; ++i) acc[j][i] = mma8(a[i], b[j], acc[j][i]);
      }
    }
    __syncthreads();  // the sums of the group before are used
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NA; ++i) sums[wave][j * NA + i][lane] = acc[j][i];
    __syncthreads();
    if (wave >= MT) continue;
    f32x4 z[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      z[i] = sums[0][wave * NA + i][lane];
#pragma unroll
      for (int x = 1; x < 4; ++x) z[i] += sums[x][wave * NA + i][lane];
    }
    if constexpr (EPI == kEpiLse) {
      float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = 32 * grp + 16 * i + 4 * q + e;
          if (v >= f.nv) z[i][e] = -__builtin_inff();
          m = fmaxf(m, z[i][e]);
          if (mine && v < f.nv && v == at_v) f.target_logit[t] = z[i][e];
        }
      const float base = base_of(m);
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s += exp_of(z[i][e] - base);
      join(run_m, run_s, m, s);
    } else if (mine) {
      const bool live = tgt != f.ignore;
      const float lse = tgt >= 0 && tgt < f.V ? f.lse[t] : __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int v = 32 * grp + 16 * i + 4 * q;
        if (v >= f.ld_g) continue;  // rows of whole 64s, zeros past V
        f32x4 p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = exp_of(z[i][e] - lse);
          if (v + e == at_v) p[e] -= 1.0f;
          if (!live || v + e >= f.nv) p[e] = 0.0f;
        }
        store4<E>(f.g + (t * f.ld_g + v) * ES, p, 4);
      }
    }
  }
  if constexpr (EPI == kEpiLse) {
    if (wave >= MT) return;
#pragma unroll
    for (int x = 16; x < 64; x *= 2) {
      const float m2 = __shfl_xor(run_m, x), s2 = __shfl_xor(run_s, x);
      join(run_m, run_s, m2, s2);
    }
    if (q == 0 && mine) f.part[block * static_cast<int64_t>(f.T) + t] = make_float2(run_m, run_s);
  }
}

// ------------------------------------------------------------ small kernels

// Joins the tiles of TOK tokens: 256 / TOK threads per token, each its share of
// the tiles, four loads in flight, met in LDS in order.
template <int TOK>
__global__ __launch_bounds__(256) void xent_join_kernel(const float2* part, int tiles, int64_t ld,
                                                        const float* target_logit,
                                                        const int64_t* target, int64_t ignore,
                                                        int T, int V, float* loss, float* lse) {
  constexpr int PER = 256 / TOK;
  __shared__ float2 red[PER][TOK];
  const int c = threadIdx.x % TOK, k = threadIdx.x / TOK;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TOK + c;
  float m = -__builtin_inff(), s = 0.0f;
  if (t < T)
    for (int i = k; i < tiles; i += 4 * PER) {
      float2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = part[(i + PER * u < tiles ? i + PER * u : i) * ld + t];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + PER * u < tiles) join(m, s, p[u].x, p[u].y);
    }
  red[k][c] = make_float2(m, s);
#pragma unroll
  for (int n = PER / 2; n > 0; n /= 2) {
    __syncthreads();
    if (k < n) {
      join(m, s, red[k + n][c].x, red[k + n][c].y);
      red[k][c] = make_float2(m, s);
    }
  }
  if (k != 0 || t >= T) return;
  const float l = base_of(m) + logf(s);
  lse[t] = l;
  const int64_t tgt = target[t];
  loss[t] = tgt == ignore ? 0.0f : tgt >= 0 && tgt < V ? l - target_logit[t] : __builtin_nanf("");
}

struct GatherArgs {
  const char* h;
  int64_t ldh;
  const int64_t* target;
  const float* lse;
  const float* dloss;
  int64_t ignore;
  int32_t T, D, V;
  const int2* blocks;  // live tokens and the bits of max |dloss| of each 1024, NULL: found here
  // Out: h of the live tokens [.., ld_live], zeros past D, and r h (NULL: not
  // needed); and their scalars.
  char* h_live;
  char* rh_live;
  int64_t ld_live;
  int32_t* index;
  int32_t* live_target;
  float* live_lse;
  float* live_dloss;
  int32_t* n_live;
  float* c;  // max |dloss| of the live tokens
  char* dh;  // zeros for the ignored tokens, or NULL
  int64_t lddh;
};

// Sum of a workgroup's 256 n, and the largest of its m.
__device__ inline int2 block_stats(int n, int m) {
  __shared__ int2 red[4];
#pragma unroll
  for (int x = 1; x < 64; x *= 2) {
    n += __shfl_xor(n, x);
    m = max(m, __shfl_xor(m, x));
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_int2(n, m);
  __syncthreads();
  return make_int2(red[0].x + red[1].x + red[2].x + red[3].x,
                   max(max(red[0].y, red[1].y), max(red[2].y, red[3].y)));
}

// Bits of |x|, in the order of the values; NaN above all.
__device__ inline int abs_bits(float x) { return __builtin_bit_cast(int, x) & 0x7fffffff; }

__global__ __launch_bounds__(256) void xent_count_kernel(const int64_t* target, const float* dloss,
                                                         int64_t ignore, int T, int2* blocks) {
  int n = 0, m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 1024 + 256 * i + threadIdx.x;
    if (t < T && target[t] != ignore) {
      ++n;
      m = max(m, abs_bits(dloss[t]));
    }
  }
  const int2 all = block_stats(n, m);
  if (threadIdx.x == 0) blocks[blockIdx.x] = all;
}

// Gathers the live tokens among ROWS, in order: a workgroup counts the live
// ones before its own and finds the largest |dloss|, then copies the rows.
// Sixteen rows, or four where those would leave CUs idle (1999 x 1000: 13.4 and
// 8.6 us).
template <typename E, int ROWS>
__global__ __launch_bounds__(256) void xent_gather_kernel(GatherArgs g) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * ROWS;
  int n = 0, m = 0;
  if (g.blocks) {
    const int64_t own = t0 / 1024, blocks = (g.T + 1023) / 1024;
    for (int64_t i = threadIdx.x; i < blocks; i += 256) {
      const int2 b = g.blocks[i];
      if (i < own) n += b.x;
      m = max(m, b.y);
    }
    // At most 1023 tokens before its own in the block; all loads at once.
    int64_t tgt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = own * 1024 + 256 * i + threadIdx.x;
      tgt[i] = g.target[t < t0 ? t : t0];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) n += own * 1024 + 256 * i + threadIdx.x < t0 && tgt[i] != g.ignore;
  } else {
    // Eight tokens of a thread in flight (one after the other: 2 us longer for 1999).
    for (int64_t first = threadIdx.x; first < g.T; first += 256 * 8) {
      int64_t tgt[8];
      float dl[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t t = first + 256 * i, at = t < g.T ? t : first;
        tgt[i] = g.target[at];
        dl[i] = g.dloss[at];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t t = first + 256 * i;
        if (t >= g.T || tgt[i] == g.ignore) continue;
        n += t < t0;
        m = max(m, abs_bits(dl[i]));
      }
    }
  }
  const int2 stats = block_stats(n, m);
  const int before = stats.x;
  const float c = __builtin_bit_cast(float, stats.y);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mine = t0 + lane;
  const int64_t tgt = lane < ROWS && mine < g.T ? g.target[mine] : g.ignore;
  __shared__ float ratios[ROWS];
  if (wave == 0 && tgt != g.ignore) ratios[lane] = c > 0.0f ? g.dloss[mine] / c : g.dloss[mine];
  __syncthreads();
  const uint64_t live = __ballot(tgt != g.ignore);
  const int pos = before + __popcll(live & ((1ull << lane) - 1));
  if (wave == 0 && tgt != g.ignore) {
    g.index[pos] = static_cast<int32_t>(mine);
    g.live_target[pos] = tgt >= 0 && tgt < g.V ? static_cast<int32_t>(tgt) : -1;
    g.live_lse[pos] = g.lse[mine];
    g.live_dloss[pos] = dh_factor(g.dloss[mine]);
  }
  if (threadIdx.x == 0 && t0 + ROWS >= g.T) {
    *g.n_live = before + __popcll(live);
    *g.c = c;
  }
  // The rows' pieces of 16 bytes, four of a thread in flight.
  constexpr int N = 16 / sizeof(E), U = 4;
  const int rows = static_cast<int>(g.T - t0 < ROWS ? g.T - t0 : ROWS);
  const int per_row = static_cast<int>(g.ld_live / N), total = rows * per_row;
  for (int first = threadIdx.x; first < total; first += 256 * U) {
    E v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = first + 256 * u, row = i / per_row, col = (i - row * per_row) * N;
      if (i >= total || !(live >> row & 1)) continue;
      const char* src = g.h + ((t0 + row) * g.ldh + col) * static_cast<int64_t>(sizeof(E));
      if (col + N <= g.D) {
        __builtin_memcpy(v[u], src, 16);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          v[u][j] = static_cast<E>(0.0f);
          if (col + j < g.D) __builtin_memcpy(&v[u][j], src + j * sizeof(E), sizeof(E));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = first + 256 * u, row = i / per_row, col = (i - row * per_row) * N;
      if (i >= total) continue;
      if (live >> row & 1) {
        const int64_t to = before + __popcll(live & ((1ull << row) - 1));
        const int64_t at = (to * g.ld_live + col) * static_cast<int64_t>(sizeof(E));
        __builtin_memcpy(g.h_live + at, v[u], 16);
        if (g.rh_live) {
          const float ratio = ratios[row];
#pragma unroll
          for (int j = 0; j < N; ++j) v[u][j] = static_cast<E>(ratio * static_cast<float>(v[u][j]));
          __builtin_memcpy(g.rh_live + at, v[u], 16);
        }
      } else if (g.dh) {
        char* dst = g.dh + ((t0 + row) * g.lddh + col) * static_cast<int64_t>(sizeof(E));
        const E z = static_cast<E>(0.0f);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (col + j < g.D) __builtin_memcpy(dst + j * sizeof(E), &z, sizeof(E));
      }
    }
  }
}

// Rows of bf16 from anywhere into rows of ld (a multiple of 8) from 16-byte
// boundaries, zeros past cols.  Four pieces of 16 bytes per thread in flight.
__global__ __launch_bounds__(256) void xent_pack_kernel(const char* src, int64_t ld_src, int64_t rows, int cols,
                                                        char* dst, int64_t ld) {
  const int per_row = static_cast<int>(ld / 8);
  const int64_t total = rows * per_row, first = static_cast<int64_t>(blockIdx.x) * 1024 + threadIdx.x;
  uint16_t v[4][8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t i = first + 256 * u, row = i / per_row;
    const int c = static_cast<int>(i - row * per_row) * 8;
    if (i >= total) break;
    const char* p = src + (row * ld_src + c) * 2;
    if (c + 8 <= cols) {
      __builtin_memcpy(v[u], p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[u][e] = 0;
        if (c + e < cols) __builtin_memcpy(&v[u][e], p + 2 * e, 2);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t i = first + 256 * u;
    if (i < total) __builtin_memcpy(dst + i * 16, v[u], 16);
  }
}

// C[row, a] = sum of the ranges' partial sums, in order; four a per thread.  Many
// ranges are shared by PARTS threads, whose sums meet in LDS, in order: one after
// another 64 of them took 6 us.
template <typename E, int PARTS>
__global__ __launch_bounds__(256) void xent_sum_kernel(const float* part, int ranges, int64_t stride,
                                                       int64_t ld, int rows, const int32_t* n_live,
                                                       const int32_t* row_map, const float* scale,
                                                       int scale_step, int cols, char* out,
                                                       int64_t ld_out) {
  constexpr int QUADS = 256 / PARTS;
  __shared__ f32x4 sums[PARTS > 1 ? 256 : 1];
  const int quads = (cols + 3) / 4, own = threadIdx.x / QUADS;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * QUADS + threadIdx.x % QUADS;
  const int64_t row = i / quads;
  const int c = static_cast<int>(i - row * quads) * 4;
  const bool live = row < (n_live ? *n_live : rows);
  f32x4 s = {};
  if (live) {
    const int per = (ranges + PARTS - 1) / PARTS, first = own * per, last = min(first + per, ranges);
    const float* p0 = part + row * ld + c;  // rows of ld floats, a multiple of 4
    // Eight loads in flight; those past the last range read it again.
    for (int k = first; k < last; k += 8) {
      f32x4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = *reinterpret_cast<const f32x4*>(p0 + (k + i < last ? k + i : last - 1) * stride);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < last) s += v[i];
    }
  }
  if constexpr (PARTS > 1) {
    sums[threadIdx.x] = s;
    __syncthreads();
    if (own > 0) return;
#pragma unroll
    for (int p = 1; p < PARTS; ++p) s += sums[p * QUADS + threadIdx.x];
  }
  if (!live) return;
  s *= scale[row * scale_step];
  int64_t to = row_map ? row_map[row] : row;
  if (to < 0) {
    to = -1 - to;
    s = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  store4<E>(out + (to * ld_out + c) * static_cast<int64_t>(sizeof(E)), s, cols - c);
}

// Zeros (dw of no tokens), of any number of elements.
template <typename E>
__global__ __launch_bounds__(256) void xent_zero_kernel(char* out, int64_t ld, int64_t rows, int cols) {
  const E z = static_cast<E>(0.0f);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256)
      __builtin_memcpy(out + (row * ld + c) * static_cast<int64_t>(sizeof(E)), &z, sizeof(E));
}

}  // namespace
}  // namespace fconv

namespace fconv {
namespace {
// How a product is divided: the edge of its tiles (64: general kernel) and
// the ranges of its sum.
struct Split {
  int32_t edge, ranges;
  double us;  // by choose()'s account
};
}  // namespace
}  // namespace fconv

struct fconv_xent_plan_s {
  fconv_xent_desc d;
  int32_t es;
  // Forward workspace: partial (max, sum) [tiles of V, at most][T], target logits [T].
  size_t fwd_target, fwd_bytes;
  bool few_fwd, few_bwd;  // at most kFewTokens, by their own kernel
  // bf16 rows that are no multiple of 16 bytes are packed for the tiled kernel
  // where that is quicker than the general one: h, and w piece by piece.
  bool pack_fwd, pack_bwd;
  int32_t fwd_piece;  // rows of w packed at a time
  int64_t ld_pack;
  size_t fwd_h, fwd_w, o_w;
  fconv::Split logits, grad, dh, dw;  // dh and dw: of one piece
  // Backward workspace.
  int64_t ld_live;               // row stride of the gathered h
  int32_t piece, pieces;         // vocabulary columns of a piece
  int64_t ld_g;
  size_t o_g, o_h, o_index, o_target, o_lse, o_dloss, o_n, o_c, o_blocks, o_rh, o_dh, o_dw, bwd_bytes;
};

namespace fconv {
namespace {

// Of q at a time.  Fewer pieces mean that dh's sums are added to less often; it is far from
// the caches' size either way (8192 x 512 x 65536, both passes: 128 MB 2355 us,
// 256 MB 2192, 512 MB 2077, 1 GB 2043).
constexpr int64_t kGBytes = 512ll << 20;

// The division of a product that takes the least time by a rough account (us):
// workgroups take turns on the device, each turn as long as its slabs of 64 k
// and what a tile costs beside them; the ranges' partial sums are written and
// read once more.
// Those fill at most kGBytes, as a piece of q does: what a call needs beside its
// inputs and outputs stays linear in the tokens and in the vocabulary.
Split choose(int64_t na, int64_t nb, int64_t nk, bool tiled, bool split) {
  struct Kind {
    int32_t edge;
    int64_t at_once;  // workgroups on the device
    double slab, slab_alone, tile;
  };
  static const Kind kinds[] = {{256, 256, 1.0, 1.0, 5.0}, {128, 512, 0.7, 0.55, 5.0}, {64, 1024, 1.15, 0.7, 2.5}};
  Split best = {64, 1, 1e300};
  for (const Kind& k : kinds) {
    if (k.edge != 64 && !tiled) continue;
    const int64_t tiles = ceil_div(na, k.edge) * ceil_div(nb, k.edge), slabs = ceil_div(nk, 64);
    for (int32_t r = 1; r <= (split ? 128 : 1) && (r == 1 || (slabs / r >= 2 && r * na * nb * 4 <= kGBytes)); ++r) {
      const int64_t n = tiles * r;
      double us = static_cast<double>(ceil_div(n, k.at_once)) *
                  (static_cast<double>(ceil_div(slabs, r)) * (n > 256 ? k.slab : k.slab_alone) + k.tile);
      if (r > 1) us += 6.0 + 8.0 * r * static_cast<double>(na) * static_cast<double>(nb) / 4e6;
      if (us < best.us) best = Split{k.edge, r, us};
    }
  }
  return best;
}

// Time (us) of the few-token kernel on a piece of the vocabulary: w at 4.1, 3.2
// or 2.5 TB/s for 16, 32 or 64 tokens (4096 x 60000 and x 30000), or what each 32
// v cost a workgroup (fitted over D 72 .. 1024, V 600 .. 33000; `grad`: q is
// written too).
double few_us(int64_t T, int64_t V, int64_t D, bool grad) {
  const int k = T <= 16 ? 0 : T <= 32 ? 1 : 2;
  static const double rate[] = {4.1e6, 3.2e6, 2.5e6}, base[] = {0.0042, 0.0055, 0.0085},
                      per_d[] = {0.8e-5, 1.0e-5, 1.85e-5}, store[] = {0.003, 0.004, 0.006};
  const double memory = 4.0 + 2.0 * static_cast<double>(V) * static_cast<double>(D) / rate[k];
  const double each = base[k] + per_d[k] * static_cast<double>(D) + (grad ? store[k] : 0.0);
  const double work = 2.6 + static_cast<double>(ceil_div(V, 32)) * each + (D % 64 ? 1.0 : 0.0);
  return memory > work ? memory : work;
}
// What choose() leaves out of the tiles' time for few tokens: nothing hides a
// slab's latency where a workgroup is alone on its CU (59 x 1024 x 4544: 13 us
// for 16 slabs).
double few_tiles_us(const Split& s, int64_t D) { return s.edge == 64 ? 0.3 * static_cast<double>(ceil_div(D, 64)) : 0.0; }

// Time (us) of packing a matrix: a launch, one read and one write.
double pack_us(int64_t rows, int64_t cols) { return 4.0 + 4.0 * static_cast<double>(rows) * static_cast<double>(cols) / 4e6; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// The kernel of a product: tiles of 64 (general), 128 or 256.
template <typename E, Order OA, Order OB, Epilogue EPI>
hipError_t launch_gemm(const GemmArgs& g, int edge, hipStream_t s) {
  const int64_t ta = ceil_div(g.na, edge), tb = ceil_div(g.nb, edge);
  if constexpr (sizeof(E) == 2) {
    // As many workgroups as the device holds at once (one or two a CU, by their
    // LDS), in eighths; each takes every so manieth tile of its XCD's share.
    const int64_t most = edge == 256 ? 256 : 512, n = round_up(ta * tb * g.ranges, 8);
    const dim3 grid(static_cast<unsigned>(n < most ? n : most));
    if (edge == 256)
      hipLaunchKernelGGL((xent_tile_kernel<OA, OB, EPI, 128, 8>), grid, dim3(512), 0, s, g);
    else if (edge == 128)
      hipLaunchKernelGGL((xent_tile_kernel<OA, OB, EPI, 64, 4>), grid, dim3(256), 0, s, g);
    if (edge != 64) return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(ta), static_cast<unsigned>(tb), static_cast<unsigned>(g.ranges));
  hipLaunchKernelGGL((xent_gen_kernel<E, OA, OB, EPI == kEpiStream ? kEpiOut : EPI>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

// Rows that the tiled kernel's copies may start at.
bool fits_tiles(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

constexpr int32_t kFewTokens = 64;
// Vocabularies up to this take few_dh: it grows with the vocabulary, the tiles'
// way costs a launch more (both gradients of 16 x 512 x 1000 10.0 instead of 12.6
// us, x 2048 12.0 and 13.7, x 4096 15.9 and 15.7; of 64 tokens 14.2 and 14.6, 18.4
// and 15.8).
int32_t few_dh_v(int32_t T) { return T <= 32 ? 2048 : 1024; }
// Workgroups of the few-token forward kernel.
int64_t few_groups(int32_t V) { return ceil_div(V, 32) < 1024 ? round_up(ceil_div(V, 32), 8) : 1024; }

// Whether rows of bf16 begin between dwords.
bool odd_rows(const Operand& o) { return (reinterpret_cast<uintptr_t>(o.p) & 3) != 0 || o.ld % 2 != 0; }

hipError_t launch_pack(const void* src, int64_t ld_src, int64_t rows, int32_t cols, char* dst, int64_t ld,
                       hipStream_t s) {
  hipLaunchKernelGGL(xent_pack_kernel, dim3(static_cast<unsigned>(ceil_div(rows * (ld / 8), 1024))), dim3(256), 0, s,
                     static_cast<const char*>(src), ld_src, rows, cols, dst, ld);
  return hipGetLastError();
}

FewArgs few_args(const fconv_xent_plan_s* p, const fconv_xent_args* args) {
  FewArgs f = {};
  f.w = static_cast<const char*>(args->w);
  f.ldw = args->ldw;
  f.h = static_cast<const char*>(args->h);
  f.ldh = args->ldh;
  f.target = args->target;
  f.ignore = p->d.ignore_index;
  f.T = p->d.T;
  f.D = p->d.D;
  f.V = f.nv = p->d.V;
  return f;
}

// `groups` workgroups of v (a multiple of 8), for each 32 tokens with ODD.
template <typename E, bool ODD, Epilogue EPI>
hipError_t launch_few_of(const FewArgs& f, int64_t groups, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ODD ? groups * ceil_div(f.T, 32) : groups));
  if (f.T <= 16) {
    hipLaunchKernelGGL((xent_few_kernel<E, ODD, EPI, 1>), grid, dim3(256), 0, s, f);
  } else if (ODD || f.T <= 32) {
    hipLaunchKernelGGL((xent_few_kernel<E, ODD, EPI, 2>), grid, dim3(256), 0, s, f);
  } else {
    if constexpr (!ODD) hipLaunchKernelGGL((xent_few_kernel<E, ODD, EPI, 4>), grid, dim3(256), 0, s, f);
  }
  return hipGetLastError();
}
template <typename E, Epilogue EPI>
hipError_t launch_few(const FewArgs& f, int64_t groups, hipStream_t s) {
  if constexpr (sizeof(E) == 2) {
    if (odd_rows(Operand{f.w, f.ldw}) || odd_rows(Operand{f.h, f.ldh})) return launch_few_of<E, true, EPI>(f, groups, s);
  }
  return launch_few_of<E, false, EPI>(f, groups, s);
}

template <typename E>
hipError_t run_forward(const fconv_xent_plan_s* p, const fconv_xent_args* args, hipStream_t s) {
  const fconv_xent_desc& d = p->d;
  char* ws = static_cast<char*>(args->workspace);
  float2* part = reinterpret_cast<float2*>(ws);
  float* target_logit = reinterpret_cast<float*>(ws + p->fwd_target);
  int tiles;
  hipError_t e;
  const bool fits = fits_tiles(args->w, args->ldw) && fits_tiles(args->h, args->ldh);
  if (p->few_fwd || (d.T <= kFewTokens && !fits && p->logits.edge != 64)) {
    FewArgs f = few_args(p, args);
    f.part = part;
    f.target_logit = target_logit;
    tiles = static_cast<int>(few_groups(d.V));
    e = launch_few<E, kEpiLse>(f, tiles, s);
  } else {
    GemmArgs g = {};
    g.a = Operand{static_cast<const char*>(args->w), args->ldw};
    g.b = Operand{static_cast<const char*>(args->h), args->ldh};
    g.nb = d.T;
    g.nk = d.D;
    g.ranges = 1;
    g.ld_out = d.T;
    g.target = args->target;
    g.target_logit = target_logit;
    int edge = p->logits.edge;
    if (p->pack_fwd) {
      if ((e = launch_pack(args->h, args->ldh, d.T, d.D, ws + p->fwd_h, p->ld_pack, s)) != hipSuccess) return e;
      g.b = Operand{ws + p->fwd_h, p->ld_pack};
    } else if (!fits) {
      edge = 64;
    }
    tiles = static_cast<int>(ceil_div(d.V, edge));
    for (int32_t v0 = 0; v0 < d.V; v0 += p->fwd_piece) {
      g.na = d.V - v0 < p->fwd_piece ? d.V - v0 : p->fwd_piece;
      g.v0 = v0;
      g.out = ws + static_cast<size_t>(v0 / edge) * d.T * 8;
      if (p->pack_fwd) {
        if ((e = launch_pack(g.a.p + v0 * args->ldw * 2, args->ldw, g.na, d.D, ws + p->fwd_w, p->ld_pack, s)) !=
            hipSuccess)
          return e;
        GemmArgs piece = g;
        piece.a = Operand{ws + p->fwd_w, p->ld_pack};
        e = launch_gemm<E, kSum, kSum, kEpiLse>(piece, edge, s);
      } else {
        e = launch_gemm<E, kSum, kSum, kEpiLse>(g, edge, s);
      }
      if (e != hipSuccess) return e;
    }
  }
  if (e != hipSuccess) return e;
  if (d.T <= 256)
    hipLaunchKernelGGL(xent_join_kernel<4>, dim3(static_cast<unsigned>(ceil_div(d.T, 4))), dim3(256), 0, s, part,
                       tiles, static_cast<int64_t>(d.T), target_logit, args->target, d.ignore_index, d.T, d.V,
                       args->loss, args->lse);
  else
    hipLaunchKernelGGL(xent_join_kernel<16>, dim3(static_cast<unsigned>(ceil_div(d.T, 16))), dim3(256), 0, s, part,
                       tiles, static_cast<int64_t>(d.T), target_logit, args->target, d.ignore_index, d.T, d.V,
                       args->loss, args->lse);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sum(const float* part, int ranges, int64_t stride, int64_t ld, int rows,
                      const int32_t* n_live, const int32_t* row_map, const float* scale, int scale_step,
                      int cols, char* out, int64_t ld_out, hipStream_t s) {
  const int64_t quads = static_cast<int64_t>(rows) * ((cols + 3) / 4);
  if (ranges > 8 && quads <= 1 << 16)
    hipLaunchKernelGGL((xent_sum_kernel<E, 8>), dim3(static_cast<unsigned>(ceil_div(quads, 32))), dim3(256), 0, s,
                       part, ranges, stride, ld, rows, n_live, row_map, scale, scale_step, cols, out, ld_out);
  else
    hipLaunchKernelGGL((xent_sum_kernel<E, 1>), dim3(static_cast<unsigned>(ceil_div(quads, 256))), dim3(256), 0, s,
                       part, ranges, stride, ld, rows, n_live, row_map, scale, scale_step, cols, out, ld_out);
  return hipGetLastError();
}

template <typename E>
hipError_t run_backward(const fconv_xent_plan_s* p, const fconv_xent_args* args, hipStream_t s) {
  const fconv_xent_desc& d = p->d;
  char* ws = static_cast<char*>(args->workspace);
  hipError_t e;
  if (d.T == 0) {
    if (!args->dw) return hipSuccess;
    hipLaunchKernelGGL(xent_zero_kernel<E>, dim3(d.V < 4096 ? d.V : 4096), dim3(256), 0, s,
                       static_cast<char*>(args->dw), args->lddw, static_cast<int64_t>(d.V), d.D);
    return hipGetLastError();
  }
  float* live_dloss = reinterpret_cast<float*>(ws + p->o_dloss);
  float* c_max = reinterpret_cast<float*>(ws + p->o_c);
  int32_t* index = reinterpret_cast<int32_t*>(ws + p->o_index);
  int32_t* n_live = reinterpret_cast<int32_t*>(ws + p->o_n);
  const bool few = p->few_bwd || (d.T <= kFewTokens && !p->pack_bwd && p->grad.edge != 64 && !fits_tiles(args->w, args->ldw));
  GatherArgs ga = {};
  if (few) {
    n_live = nullptr;
  } else {
    ga.h = static_cast<const char*>(args->h);
    ga.ldh = args->ldh;
    ga.target = args->target;
    ga.lse = args->lse;
    ga.dloss = args->dloss;
    ga.ignore = d.ignore_index;
    ga.T = d.T;
    ga.D = d.D;
    ga.V = d.V;
    ga.h_live = ws + p->o_h;
    ga.ld_live = p->ld_live;
    ga.index = index;
    ga.live_target = reinterpret_cast<int32_t*>(ws + p->o_target);
    ga.live_lse = reinterpret_cast<float*>(ws + p->o_lse);
    ga.live_dloss = live_dloss;
    ga.n_live = n_live;
    ga.dh = static_cast<char*>(args->dh);
    ga.lddh = args->lddh;
    ga.c = c_max;
    ga.rh_live = args->dw ? ws + p->o_rh : nullptr;
    // Every workgroup looks at all tokens, which is quicker than another launch
    // up to some thousands of them.
    if (d.T > 2048) {
      int2* blocks = reinterpret_cast<int2*>(ws + p->o_blocks);
      hipLaunchKernelGGL(xent_count_kernel, dim3(static_cast<unsigned>(ceil_div(d.T, 1024))), dim3(256), 0, s,
                         args->target, args->dloss, d.ignore_index, d.T, blocks);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      ga.blocks = blocks;
    }
    if (d.T <= 4096)
      hipLaunchKernelGGL((xent_gather_kernel<E, 4>), dim3(static_cast<unsigned>(ceil_div(d.T, 4))), dim3(256), 0, s, ga);
    else
      hipLaunchKernelGGL((xent_gather_kernel<E, 16>), dim3(static_cast<unsigned>(ceil_div(d.T, 16))), dim3(256), 0, s, ga);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }

  for (int i = 0; i < p->pieces; ++i) {
    const int32_t v0 = i * p->piece;
    const int32_t nv = d.V - v0 < p->piece ? d.V - v0 : p->piece;
    const char* w = static_cast<const char*>(args->w) + v0 * args->ldw * p->es;
    int64_t ldw = args->ldw;
    if (p->pack_bwd) {
      if ((e = launch_pack(w, ldw, nv, d.D, ws + p->o_w, p->ld_pack, s)) != hipSuccess) return e;
      w = ws + p->o_w;
      ldw = p->ld_pack;
    }
    const bool w_fits = fits_tiles(w, ldw);
    if (few) {
      FewArgs f = few_args(p, args);
      f.w = w;
      f.v0 = v0;
      f.nv = nv;
      f.lse = args->lse;
      f.dloss = args->dloss;
      f.g = ws + p->o_g;
      f.ld_g = p->ld_g;
      f.rh = args->dw ? ws + p->o_rh : nullptr;
      f.ld_rh = p->ld_live;
      f.row_map = index;
      f.live_dloss = live_dloss;
      f.c = c_max;
      e = launch_few<E, kEpiGrad>(f, round_up(ceil_div(nv, 32), 8), s);
    } else {
      GemmArgs g = {};
      g.a = Operand{w, ldw};
      g.b = Operand{ga.h_live, p->ld_live};
      g.na = nv;
      g.nb = d.T;
      g.nk = d.D;
      g.ranges = 1;
      g.n_live = n_live;
      g.out = ws + p->o_g;
      g.ld_out = p->ld_g;
      g.live_target = ga.live_target;
      g.lse = ga.live_lse;
      g.v0 = v0;
      g.na_pad = static_cast<int32_t>(round_up(nv, 8));
      e = launch_gemm<E, kSum, kSum, kEpiGrad>(g, w_fits ? p->grad.edge : 64, s);
    }
    if (e != hipSuccess) return e;

    // dh of this piece: written at once, or as the ranges' partial sums, to which
    // every further piece adds its own and which are joined after the last one.
    const bool dh_whole = p->pieces * p->dh.ranges == 1;
    const int dh_edge = w_fits ? p->dh.edge : 64;
    GemmArgs h = {};
    h.a = Operand{w, ldw, p->pack_bwd ? ldw : d.D};
    h.b = Operand{ws + p->o_g, p->ld_g};
    h.na = d.D;
    h.nb = d.T;
    h.nk = nv;
    h.n_live = n_live;
    h.ranges = p->dh.ranges;
    if (dh_whole) {
      h.out = static_cast<char*>(args->dh);
      h.ld_out = args->lddh;
      h.row_map = index;
      h.scale = live_dloss;
      h.scale_step = 1;
    } else {
      h.ld_out = round_up(d.D, 4);
      h.part_stride = h.ld_out * d.T;
      h.out = ws + p->o_dh;
    }
    const bool dw_whole = p->dw.ranges == 1;
    // dw goes past the caches where it is larger than the L2s together and
    // written in whole lines (64 x 4096 x 30000: both passes 237 us instead of
    // 264; with rows of 2000 bytes, 1999 x 1000 x 32001, 485 instead of 474).
    const bool past = p->es == 2 && static_cast<int64_t>(d.V) * d.D * 2 > (32 << 20) && d.D % 64 == 0 &&
                      args->lddw % 64 == 0 && (reinterpret_cast<uintptr_t>(args->dw) & 127) == 0;
    char* dw = static_cast<char*>(args->dw) + (args->dw ? v0 * args->lddw * p->es : 0);
    GemmArgs c = {};
    c.a = Operand{ws + p->o_rh, p->ld_live, p->ld_live};
    c.b = Operand{ws + p->o_g, p->ld_g, round_up(nv, 8)};
    c.na = d.D;
    c.nb = nv;
    c.nk = d.T;
    c.n_live = n_live;
    c.ranges = p->dw.ranges;
    if (dw_whole) {
      c.out = dw;
      c.ld_out = args->lddw;
      c.scale = c_max;
    } else {
      c.ld_out = round_up(d.D, 4);
      c.part_stride = c.ld_out * nv;
      c.out = ws + p->o_dw;
    }
    auto launch_dw = [&](const GemmArgs& c) {
      return dw_whole ? past ? launch_gemm<E, kRow, kRow, kEpiStream>(c, p->dw.edge, s)
                             : launch_gemm<E, kRow, kRow, kEpiOut>(c, p->dw.edge, s)
                      : launch_gemm<E, kRow, kRow, kEpiPart>(c, p->dw.edge, s);
    };
    bool dh_done = false;
    const bool one_dw = args->dw && p->dw.edge == 64 && dw_whole;  // in a launch with dh
    if (args->dh && few && d.V <= few_dh_v(d.T)) {
      h.out = static_cast<char*>(args->dh);
      h.ld_out = args->lddh;
      h.row_map = index;
      h.scale = live_dloss;
      const dim3 grid(static_cast<unsigned>(ceil_div(d.D, 16) + (one_dw ? ceil_div(d.D, 64) * ceil_div(nv, 64) : 0)));
      if (d.T <= 16)
        hipLaunchKernelGGL((xent_few_grads_kernel<E, 1>), grid, dim3(256), 0, s, h, c);
      else if (d.T <= 32)
        hipLaunchKernelGGL((xent_few_grads_kernel<E, 2>), grid, dim3(256), 0, s, h, c);
      else
        hipLaunchKernelGGL((xent_few_grads_kernel<E, 4>), grid, dim3(256), 0, s, h, c);
      e = hipGetLastError();
      if (e == hipSuccess && args->dw && !one_dw) e = launch_dw(c);
      dh_done = true;
    } else if (args->dh && one_dw && dh_edge == 64) {
      const int64_t ta = ceil_div(d.D, 64);
      const dim3 grid(static_cast<unsigned>(ta * (ceil_div(d.T, 64) * h.ranges + ceil_div(nv, 64))));
      if (dh_whole)
        hipLaunchKernelGGL((xent_gen_grads_kernel<E, kEpiOut>), grid, dim3(256), 0, s, h, c);
      else if (i > 0)
        hipLaunchKernelGGL((xent_gen_grads_kernel<E, kEpiAdd>), grid, dim3(256), 0, s, h, c);
      else
        hipLaunchKernelGGL((xent_gen_grads_kernel<E, kEpiPart>), grid, dim3(256), 0, s, h, c);
      e = hipGetLastError();
    } else {
      if (args->dh)
        e = dh_whole ? launch_gemm<E, kRow, kSum, kEpiOut>(h, dh_edge, s)
            : i > 0  ? launch_gemm<E, kRow, kSum, kEpiAdd>(h, dh_edge, s)
                     : launch_gemm<E, kRow, kSum, kEpiPart>(h, dh_edge, s);
      if (e == hipSuccess && args->dw) e = launch_dw(c);
    }
    if (e == hipSuccess && args->dh && !dh_done && !dh_whole && i == p->pieces - 1)
      e = launch_sum<E>(reinterpret_cast<const float*>(ws + p->o_dh), h.ranges, h.part_stride,
                        h.ld_out, d.T, n_live, index, live_dloss, 1, d.D, static_cast<char*>(args->dh),
                        args->lddh, s);
    if (e == hipSuccess && args->dw && !dw_whole)
      e = launch_sum<E>(reinterpret_cast<const float*>(ws + p->o_dw), c.ranges, c.part_stride, c.ld_out, nv,
                        nullptr, nullptr, c_max, 0, d.D, dw, args->lddw, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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

struct Range {
  const void* p;
  size_t bytes;
};
// Whether any of the written ranges meets another range.
bool clash(const Range* out, int n_out, const Range* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

bool bad_ld(int64_t ld, int32_t D) { return ld < D || ld > kMaxLd; }

}  // namespace
}  // namespace fconv

extern "C" {

fconv_status fconv_xent_plan_create(const fconv_xent_desc* desc, fconv_xent_plan* out) {
  using namespace fconv;
  if (!desc || !out) return FCONV_ERR_INVALID_ARG;
  *out = nullptr;
  const fconv_xent_desc& d = *desc;
  if (d.dtype != FCONV_BF16 && d.dtype != FCONV_FP32) return FCONV_ERR_UNSUPPORTED;
  if (d.flags) return FCONV_ERR_UNSUPPORTED;
  if (d.T < 0 || d.D < 1 || d.V < 1) return FCONV_ERR_INVALID_ARG;
  if (d.D > kMaxD || d.T > kMaxTV || d.V > kMaxTV) return FCONV_ERR_UNSUPPORTED;
  if (ceil_div(d.T, 64) > kMaxGridY || ceil_div(d.V, 64) * ceil_div(d.T, 64) > kMaxTiles ||
      static_cast<int64_t>(d.T) * d.D > kMaxSum)
    return FCONV_ERR_UNSUPPORTED;
  fconv_xent_plan_s* p = new (std::nothrow) fconv_xent_plan_s();
  if (!p) return FCONV_ERR_INVALID_ARG;
  p->d = d;
  p->es = d.dtype == FCONV_BF16 ? 2 : 4;
  const bool bf16 = d.dtype == FCONV_BF16, tiled = bf16 && d.D % 8 == 0;
  p->ld_pack = round_up(d.D, 8);
  p->logits = choose(d.V, d.T, d.D, tiled, false);
  p->fwd_piece = d.V;
  if (bf16 && !tiled && d.T > kFewTokens) {
    const Split packed = choose(d.V, d.T, d.D, true, false);
    p->pack_fwd = packed.us + pack_us(d.V, d.D) + pack_us(d.T, d.D) < p->logits.us;
    if (p->pack_fwd) {
      p->logits = packed;
      const int64_t piece = round_up((128 << 20) / p->ld_pack, 256);
      if (piece < d.V) p->fwd_piece = static_cast<int32_t>(piece);
    }
  }
  p->few_fwd = d.T <= kFewTokens && few_us(d.T, d.V, d.D, false) < p->logits.us + few_tiles_us(p->logits, d.D);
  // Either kernel may run: which one depends on the pointers too.
  int64_t parts = ceil_div(d.V, 64);
  if (d.T <= kFewTokens && parts < few_groups(d.V)) parts = few_groups(d.V);
  p->fwd_target = static_cast<size_t>(parts) * d.T * 8;
  p->fwd_h = (p->fwd_target + static_cast<size_t>(d.T) * 4 + 255) / 256 * 256;
  p->fwd_w = p->fwd_h;
  p->fwd_bytes = p->fwd_h;
  if (p->pack_fwd) {
    p->fwd_w += (static_cast<size_t>(d.T) * p->ld_pack * 2 + 255) / 256 * 256;
    p->fwd_bytes = p->fwd_w + static_cast<size_t>(p->fwd_piece) * p->ld_pack * 2;
  }

  if (d.T > 0) {
    const int64_t T = d.T;
    p->ld_live = round_up(d.D, 64);
    int64_t piece = kGBytes / (T * p->es) / 256 * 256;
    if (piece < 256) piece = 256;
    if (piece > kMaxGridY * 64) piece = kMaxGridY * 64;  // grid.y of dw
    if (piece > kMaxSum / d.D / 256 * 256) piece = kMaxSum / d.D / 256 * 256;
    if (piece > d.V) piece = d.V;
    p->pieces = static_cast<int32_t>(ceil_div(d.V, piece));
    // Pieces of about the same length.
    piece = round_up(ceil_div(d.V, p->pieces), 256);
    if (piece > d.V) piece = d.V;
    p->piece = static_cast<int32_t>(piece);
    p->pieces = static_cast<int32_t>(ceil_div(d.V, piece));
    p->ld_g = round_up(piece, 64);
    p->grad = choose(piece, T, d.D, tiled, false);
    p->dh = choose(d.D, T, piece, tiled, true);
    if (bf16 && !tiled && T > kFewTokens) {
      const Split grad = choose(piece, T, d.D, true, false), dh = choose(d.D, T, piece, true, true);
      p->pack_bwd = grad.us + dh.us + pack_us(piece, d.D) < p->grad.us + p->dh.us;
      if (p->pack_bwd) {
        p->grad = grad;
        p->dh = dh;
      }
    }
    p->dw = choose(d.D, piece, T, d.dtype == FCONV_BF16, true);
    // Both gradients in general tiles take one launch, in which they overlap.
    const Split dh64 = choose(d.D, T, piece, false, true), dw64 = choose(d.D, piece, T, false, false);
    const double longer = dh64.us > dw64.us ? dh64.us : dw64.us, other = dh64.us + dw64.us - longer;
    if (!p->pack_bwd && longer + 0.5 * other < p->dh.us + p->dw.us + 4.0) {
      p->dh = dh64;
      p->dw = dw64;
    }
    // The gather is a launch and some microseconds more, and its rows are read again.
    p->few_bwd = T <= kFewTokens && few_us(d.T, piece, d.D, true) < p->grad.us + few_tiles_us(p->grad, d.D) + 10.0;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t o = at;
      at += (bytes + 255) / 256 * 256;
      return o;
    };
    const size_t ld4 = static_cast<size_t>(round_up(d.D, 4)) * 4;
    p->o_g = take(static_cast<size_t>(T) * p->ld_g * p->es);
    p->o_h = take(static_cast<size_t>(T) * p->ld_live * p->es);
    p->o_index = take(T * 4);
    p->o_target = take(T * 4);
    p->o_lse = take(T * 4);
    p->o_dloss = take(T * 4);
    p->o_n = take(4);
    p->o_c = take(4);
    p->o_blocks = take(ceil_div(T, 1024) * 8);
    p->o_rh = take(static_cast<size_t>(T) * p->ld_live * p->es);
    p->o_w = take(p->pack_bwd ? static_cast<size_t>(piece) * p->ld_pack * 2 : 0);
    p->o_dh = take(p->pieces > 1 || p->dh.ranges > 1 ? static_cast<size_t>(p->dh.ranges) * T * ld4 : 0);
    p->o_dw = take(p->dw.ranges > 1 ? static_cast<size_t>(p->dw.ranges) * piece * ld4 : 0);
    p->bwd_bytes = at;
  }
  *out = p;
  return FCONV_OK;
}

fconv_status fconv_xent_plan_forward_workspace_size(fconv_xent_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->fwd_bytes;
  return FCONV_OK;
}

fconv_status fconv_xent_plan_backward_workspace_size(fconv_xent_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->bwd_bytes;
  return FCONV_OK;
}

fconv_status fconv_xent_plan_forward(fconv_xent_plan p, void* stream, const fconv_xent_args* a) {
  using namespace fconv;
  if (!p || !a) return FCONV_ERR_INVALID_ARG;
  const fconv_xent_desc& d = p->d;
  if (d.T == 0) return FCONV_OK;
  if (!a->h || !a->w || !a->target || !a->loss || !a->lse) return FCONV_ERR_INVALID_ARG;
  if (bad_ld(a->ldh, d.D) || bad_ld(a->ldw, d.D)) return FCONV_ERR_INVALID_ARG;
  if (!a->workspace || a->workspace_bytes < p->fwd_bytes) return FCONV_ERR_WORKSPACE;
  if (!aligned(a->h, p->es) || !aligned(a->w, p->es) || !aligned(a->target, 8) || !aligned(a->loss, 4) ||
      !aligned(a->lse, 4) || !aligned(a->workspace, 16))
    return FCONV_ERR_MISALIGNED;
  const size_t t4 = static_cast<size_t>(d.T) * 4;
  const Range in[] = {{a->h, span(d.T, d.D, a->ldh, p->es)}, {a->w, span(d.V, d.D, a->ldw, p->es)},
                      {a->target, 2 * t4}};
  const Range wr[] = {{a->loss, t4}, {a->lse, t4}, {a->workspace, p->fwd_bytes}};
  if (clash(wr, 3, in, 3)) return FCONV_ERR_INVALID_ARG;
  const hipError_t e = d.dtype == FCONV_BF16 ? run_forward<__bf16>(p, a, as_stream(stream))
                                             : run_forward<float>(p, a, as_stream(stream));
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_xent_plan_backward(fconv_xent_plan p, void* stream, const fconv_xent_args* a) {
  using namespace fconv;
  if (!p || !a) return FCONV_ERR_INVALID_ARG;
  const fconv_xent_desc& d = p->d;
  if (!a->dh && !a->dw) return FCONV_ERR_INVALID_ARG;
  if ((a->dh && bad_ld(a->lddh, d.D)) || (a->dw && bad_ld(a->lddw, d.D))) return FCONV_ERR_INVALID_ARG;
  if (!aligned(a->dh, p->es) || !aligned(a->dw, p->es)) return FCONV_ERR_MISALIGNED;
  if (d.T > 0) {
    if (!a->h || !a->w || !a->target || !a->lse || !a->dloss) return FCONV_ERR_INVALID_ARG;
    if (bad_ld(a->ldh, d.D) || bad_ld(a->ldw, d.D)) return FCONV_ERR_INVALID_ARG;
    if (!a->workspace || a->workspace_bytes < p->bwd_bytes) return FCONV_ERR_WORKSPACE;
    if (!aligned(a->h, p->es) || !aligned(a->w, p->es) || !aligned(a->target, 8) || !aligned(a->lse, 4) ||
        !aligned(a->dloss, 4) || !aligned(a->workspace, 16))
      return FCONV_ERR_MISALIGNED;
    const size_t t4 = static_cast<size_t>(d.T) * 4;
    const Range in[] = {{a->h, span(d.T, d.D, a->ldh, p->es)}, {a->w, span(d.V, d.D, a->ldw, p->es)},
                        {a->target, 2 * t4}, {a->lse, t4}, {a->dloss, t4}};
    const Range wr[] = {{a->dh, span(d.T, d.D, a->lddh, p->es)}, {a->dw, span(d.V, d.D, a->lddw, p->es)},
                        {a->workspace, p->bwd_bytes}};
    if (clash(wr, 3, in, 5)) return FCONV_ERR_INVALID_ARG;
  }
  const hipError_t e = d.dtype == FCONV_BF16 ? run_backward<__bf16>(p, a, as_stream(stream))
                                             : run_backward<float>(p, a, as_stream(stream));
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

const char* fconv_xent_plan_kernel_name(fconv_xent_plan p, int32_t product) {
  using namespace fconv;
  if (!p || p->d.T == 0 || product < FCONV_XENT_LOGITS || product > FCONV_XENT_DW) return nullptr;
  const Split* const splits[] = {&p->logits, &p->grad, &p->dh, &p->dw};
  const bool packed = product == FCONV_XENT_LOGITS ? p->pack_fwd : product != FCONV_XENT_DW && p->pack_bwd;
  if (product == FCONV_XENT_LOGITS && p->few_fwd) return "xent_few";
  if (product == FCONV_XENT_GRAD && p->few_bwd) return "xent_few";
  if (product == FCONV_XENT_DH && p->few_bwd && p->d.V <= few_dh_v(p->d.T)) return "xent_few_grads";
  const int edge = splits[product]->edge;
  if (edge == 64) return packed ? "xent_gen_64_packed" : "xent_gen_64";
  if (edge == 128) return packed ? "xent_tile_128_packed" : "xent_tile_128";
  return packed ? "xent_tile_256_packed" : "xent_tile_256";
}

fconv_status fconv_xent_plan_division(fconv_xent_plan p, int32_t product, int32_t* pieces, int32_t* ranges) {
  using namespace fconv;
  if (!p || !pieces || !ranges || product < FCONV_XENT_LOGITS || product > FCONV_XENT_DW) return FCONV_ERR_INVALID_ARG;
  const bool logits = product == FCONV_XENT_LOGITS;
  *pieces = p->d.T == 0 ? 0 : logits ? static_cast<int32_t>(ceil_div(p->d.V, p->fwd_piece)) : p->pieces;
  *ranges = p->d.T == 0                  ? 0
            : product == FCONV_XENT_DH ? p->dh.ranges
            : product == FCONV_XENT_DW ? p->dw.ranges
                                       : 1;
  return FCONV_OK;
}

fconv_status fconv_xent_plan_destroy(fconv_xent_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
