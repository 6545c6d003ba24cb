// The matrix products of the dense operators (xent.hip, gated.hip) on gfx950:
// the tiled and the general kernel, what is done with a finished tile, how a
// product is divided, and the joining of its partial sums.
//
// Every product has the form C[b, a] = sum_k A(a, k) B(b, k) with a contiguous
// in C: the matrix core then ends with four consecutive a per lane.  Each
// operand has k or its row index contiguous (Order).
#ifndef FCONV_GEMM_H
#define FCONV_GEMM_H

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "dense.h"

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
constexpr int32_t kMaxD = 1 << 20, kMaxTV = 1 << 24;

// Which index of an operand is contiguous in memory: the sum's (element
// (r, k) at r * ld + k) or the row's (at k * ld + r).
enum Order { kSum, kRow };

struct Operand {
  const char* p;
  int64_t ld;     // elements
  int64_t width;  // kRow: readable elements of a row; kEpiGated's A: rows to its second half
};

// kEpiStream: kEpiOut past the caches.  kEpiAdd: kEpiPart added to what is there.
// kEpiStore: C as it is, kEpiStoreStream: past the caches.  kEpiGated: A has two
// halves of na rows; a tile holds the same rows of both, and what goes out is
// act(C of the first) (C of the second).
enum Epilogue { kEpiLse, kEpiGrad, kEpiOut, kEpiPart, kEpiStream, kEpiAdd, kEpiStore, kEpiStoreStream, kEpiGated };
constexpr bool is_scaled(Epilogue e) { return e == kEpiOut || e == kEpiStream; }
constexpr bool is_out(Epilogue e) { return is_scaled(e) || e == kEpiStore || e == kEpiStoreStream; }
constexpr bool is_stream(Epilogue e) { return e == kEpiStream || e == kEpiStoreStream; }
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
  // kEpiGated
  int32_t act;
  float* kept;                // both halves of C: row b at b * 2 * ld_kept, the second ld_kept on (16-byte rows); or NULL
  int64_t ld_kept;
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


// ------------------------------------------------------- activations of a gate
//
// The logistic function and its complement from one exponential that cannot
// overflow: both keep their relative accuracy in the tails.
enum Act { kSilu, kGelu, kGeluTanh, kActRelu };

struct Logistic {
  float s, c;  // 1 / (1 + exp(-x)) and 1 - that
};
__device__ inline Logistic logistic(float x) {
  const float e = exp_of(-__builtin_fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e), l = e * r;
  return x < 0.0f ? Logistic{l, r} : Logistic{r, l};  // NaN: both are
}
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi): 0.5 (1 + tanh y) is the logistic function of 2 y
constexpr float kGeluK = 0.044715f, kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;

template <int ACT>
__device__ inline float act_of(float g) {
  if constexpr (ACT == kSilu) return g * logistic(g).s;
  if constexpr (ACT == kGelu) return g * (0.5f * erfcf(-kSqrtHalf * g));
  if constexpr (ACT == kGeluTanh) return g * logistic(kGeluC * __builtin_fmaf(kGeluK * g * g, g, g)).s;
  return g <= 0.0f ? 0.0f : g;  // NaN stays
}
// act and its derivative.
template <int ACT>
__device__ inline float2 act_grad(float g) {
  if constexpr (ACT == kSilu) {
    const Logistic p = logistic(g);
    return make_float2(g * p.s, __builtin_fmaf(g * p.s, p.c, p.s));
  }
  if constexpr (ACT == kGelu) {
    const float cdf = 0.5f * erfcf(-kSqrtHalf * g);
    return make_float2(g * cdf, __builtin_fmaf(g * kInvSqrt2Pi, exp_of(-0.5f * g * g), cdf));
  }
  if constexpr (ACT == kGeluTanh) {
    const Logistic p = logistic(kGeluC * __builtin_fmaf(kGeluK * g * g, g, g));
    const float d = p.s * p.c;
    // g g may be infinite where d is 0.
    const float slope = d > 0.0f ? g * d * (kGeluC * __builtin_fmaf(3.0f * kGeluK * g, g, 1.0f)) : 0.0f;
    return make_float2(g * p.s, p.s + slope);
  }
  return g <= 0.0f ? make_float2(0.0f, 0.0f) : make_float2(g, g > 0.0f ? 1.0f : g);
}

// The first half of column j's tiles through the activation.
template <int ACT, int NI, int NJ>
__device__ inline void activate_by(f32x4 (&acc)[NI][NJ], int j) {
#pragma unroll
  for (int i = 0; i < NI / 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = act_of<ACT>(acc[i][j][e]);
}
template <int NI, int NJ>
__device__ inline void activate(f32x4 (&acc)[NI][NJ], int j, int act) {
  switch (act) {
    case kSilu: return activate_by<kSilu>(acc, j);
    case kGelu: return activate_by<kGelu>(acc, j);
    case kGeluTanh: return activate_by<kGeluTanh>(acc, j);
    default: return activate_by<kActRelu>(acc, j);
  }
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
  } else if constexpr (is_scaled(EPI)) {
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
    if constexpr (EPI == kEpiLse || EPI == kEpiGrad || is_scaled(EPI)) asm volatile("" : "+v"(p.at[j]));
    if constexpr (EPI == kEpiGrad || is_scaled(EPI)) asm volatile("" : "+v"(p.f[j]));
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
        // One comparison after another: with the masks of all of them at once, what
        // every tile runs through lacked scalar registers (1728 x 72 x 51605 59.6 us,
        // 55.2 so; 4096 x 2048 x 50021 648 and 640).
        float x = 0.0f;
        int here = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool is = a_of(i) + e == at;
            x = is ? acc[i][j][e] : x;
            here = is ? 1 : here;
            asm volatile("" : "+v"(x), "+v"(here));
          }
        if (here) g.target_logit[b0 + b] = x;
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
  } else if constexpr (EPI == kEpiGated) {
    constexpr int N = NI / 2;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int b = b_of(j);
      if (b >= rb) continue;
      if (g.kept) {
        float* row = g.kept + (b0 + b) * 2 * g.ld_kept + a0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (whole || a_of(i % N) < ra)  // rows are whole fours
            *reinterpret_cast<f32x4*>(row + (i / N) * g.ld_kept + a_of(i % N)) = acc[i][j];
      }
      activate(acc, j, g.act);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i][j] *= acc[N + i][j];
      char* row = g.out + ((b0 + b) * g.ld_out + a0) * ES;
      if (whole && ES == 2 && N > 1) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
          store_pair(row + (a_of(i) - 4 * q + pair_at(q)) * ES, acc[i][j], acc[N > 1 ? i + 1 : i][j]);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int n = ra - a_of(i);
          if (n > 0) store4<E>(row + a_of(i) * ES, acc[i][j], n);
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
      if constexpr (is_scaled(EPI)) {
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
            store_pair<is_stream(EPI)>(out + (a_of(i) - 4 * q + pair_at(q)) * sizeof(O), acc[i][j] * scale,
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

// 32 bytes of an operand's slab for this thread.  In place of rows past the last one
// others are read again, and what comes of them is not stored: with zeros there
// every load waited for the slab before it, since either may be what fills a register.
// In the same way columns past the last one hold what follows them in memory, up to
// the matrix's last row (gradients of 960 x 256 x 119 18 us with zeros, 10 so).
// GATED: 32 rows of each half of A, 16 of the first and the same of the second in turn,
// so that a wave's two tiles are a gate's and what it multiplies.
// FEW (kSum): a wave all of whose sixteen rows are past the last one leaves `v` as it is.
template <typename E, Order O, bool GATED, bool FEW>
__device__ inline void gen_load(const Operand& op, int64_t row0, int rows, int64_t k0, int64_t k1,
                                E v[32 / sizeof(E)]) {
  constexpr int N = 32 / sizeof(E);
  const int tid = threadIdx.x;
  const char* p;
  int n;
  if constexpr (GATED) {
    const int r = tid >> 2, f = min((r >> 5) * 16 + (r & 15), rows - 1);
    const int64_t k = k0 + (tid & 3) * N;
    n = static_cast<int>(min(k1 - k, static_cast<int64_t>(N)));
    p = op.p + ((row0 + f + (r & 16 ? op.width : 0)) * op.ld + k) * static_cast<int64_t>(sizeof(E));
  } else if constexpr (O == kSum) {
    if (FEW && __builtin_amdgcn_readfirstlane(tid >> 6) * 16 >= rows) return;
    const int r = min(tid >> 2, rows - 1);
    const int64_t k = k0 + (tid & 3) * N;
    n = static_cast<int>(min(k1 - k, static_cast<int64_t>(N)));
    p = op.p + ((row0 + r) * op.ld + k) * static_cast<int64_t>(sizeof(E));
  } else {
    constexpr int TPK = 64 / N;  // threads per k
    const int64_t k = k0 + tid / TPK;
    const int c = (tid % TPK) * N < rows ? (tid % TPK) * N : 0;
    // Past a row's end the next row is read, if there is one.
    n = k >= k1 ? 0 : k + 1 < k1 && op.ld >= N ? N : min(rows - c, N);
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

// Tile (x, y) of range z.  FEW: waves load no b where there is none.
template <typename E, Order OA, Order OB, Epilogue EPI, bool FEW = false>
__device__ inline void gen_tile(const GemmArgs& g, GenLds<E>& lds, int x, int y, int z) {
  using G = Gen<E>;
  using Frag = std::conditional_t<sizeof(E) == 2, bf16x8, f32x8>;
  auto& buf = lds.buf;
  const int live = g.n_live ? *g.n_live : 0;
  const int nb = g.n_live && OB == kSum ? live : g.nb;
  const int nk = g.n_live && OB == kRow ? live : g.nk;
  constexpr bool GATED = EPI == kEpiGated;
  constexpr int EA = GATED ? 32 : 64;
  const int64_t a0 = static_cast<int64_t>(x) * EA, b0 = static_cast<int64_t>(y) * 64;
  if (b0 >= nb) return;
  const int ra = static_cast<int>(min<int64_t>(g.na - a0, EA)), rb = static_cast<int>(min<int64_t>(nb - b0, 64));
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
  if constexpr (FEW) {
#pragma unroll
    for (int i = 0; i < 32 / G::ES; ++i) vb[0][i] = vb[1][i] = static_cast<E>(0.0f);
  }
  auto load = [&](int s, E(&xa)[32 / G::ES], E(&xb)[32 / G::ES]) __attribute__((always_inline)) {
    if (s >= slabs) return;
    gen_load<E, OA, GATED, false>(g.a, a0, ra, k0 + s * static_cast<int64_t>(G::SLAB), k1, xa);
    gen_load<E, OB, false, FEW>(g.b, b0, rb, k0 + s * static_cast<int64_t>(G::SLAB), k1, xb);
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
  epilogue<E, EPI, 2, 2, EA>(
      g, acc, per_b, a0, b0, ra, rb, x, z, wa, q, [&](int i) { return (wa * EA / 2) + 16 * i + 4 * q; }, b_of, lds.red);
}

template <typename E, Order OA, Order OB, Epilogue EPI, bool FEW = false>
__global__ __launch_bounds__(256) void gemm_gen_kernel(GemmArgs g) {
  __shared__ GenLds<E> lds;
  gen_tile<E, OA, OB, EPI, FEW>(g, lds, blockIdx.x, blockIdx.y, blockIdx.z);
}

// ------------------------------------------------- few rows, a short sum (kEpiOut, kEpiStore)
//
// C of at most 16 MT b and a sum over few k, A with a contiguous: sixteen a of all b
// for a workgroup, so that no partial sums go out and no launch joins them.  Its four
// waves take turns at steps of 32 k and add their sums in LDS, in order.  A lane
// picks its eight k of a column out of memory one by one, from any row distance
// and alignment; rows of B are whole 64s, zeros past nk.
template <typename E, int MT, Epilogue EPI>
__device__ inline void few_rows(const GemmArgs& g, f32x4* sums, int d0) {
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
  if constexpr (is_scaled(EPI)) {
    sum *= g.scale[t];
    if (g.row_map[t] < 0) sum = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  store4<E>(g.out + (t * g.ld_out + d) * static_cast<int64_t>(ES), sum, g.na - d);
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
// Measured: 8192 x 4096 x 32768 logits 1.54 to 1.68 ms from box to box, 1.31 to
// 1.43 PFLOP/s; the matrix cores are busy 71% of the cycles, at 1.8 GHz: power
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
// GATED: the halves are the same H rows of A's two halves.
template <Order O, int H, int NW, bool GATED = false>
struct Feed {
  const char* base;  // of the tile's first element of the next slab to copy
  int64_t left;      // bytes readable from base
  int64_t step;      // bytes from slab to slab
  int krem;          // k left from base (kSum)
  int64_t second;    // GATED: bytes to the second half
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
          off[h][c] = static_cast<uint32_t>((((GATED ? 0 : h * H) + (wave * 2 + c) * 8 + (lane >> 3)) * op.ld + chunk) * 2);
      if constexpr (GATED) second = op.width * op.ld * 2;
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
    const auto rsrc = make_rsrc(GATED && h == 1 ? base + second : base, left);
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

// Workgroup `block` of `blocks`.
template <Order OA, Order OB, Epilogue EPI, int H, int NW>
__device__ __forceinline__ void tile_work(const GemmArgs& g, char* ab0, char* b01, char* a01, char* ab1, char* b11, char* a11,
                                          float2* red, unsigned block, unsigned blocks) {
  constexpr int MI = H / 32, MJ = 2 * H / (16 * NW);  // matrix tiles of a wave in a quadrant
  constexpr int HB = H * 128;                         // bytes of a half tile
  static_assert(HB == NW * 2048, "two copies per wave and half tile");
  const int live = g.n_live ? *g.n_live : 0;
  const int nb = g.n_live && OB == kSum ? live : g.nb;
  const int nk = g.n_live && OB == kRow ? live : g.nk;
  // Workgroups of one XCD (block ids go round the 8 XCDs) take neighbouring
  // tiles: eight rows of them together, so both operands stay in its L2; the
  // ranges of a sum come one after the other.
  constexpr bool GATED = EPI == kEpiGated;
  constexpr int EA = GATED ? H : 2 * H;
  const int tiles_a = (g.na + EA - 1) / EA, tiles_b = (nb + 2 * H - 1) / (2 * H);
  const int tiles = tiles_a * tiles_b;
  const int total = tiles * g.ranges, share = (total + 7) / 8;
  const int first_id = (block % 8) * share, end = min(share, total - first_id);
  int slot = block / 8;
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
    p.a0 = static_cast<int64_t>(p.ta) * EA;
    p.b0 = static_cast<int64_t>(first + in % rows8) * 2 * H;
    p.ra = static_cast<int>(min<int64_t>(g.na - p.a0, EA));
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
  Feed<OA, H, NW, GATED> fa;
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
    slot += blocks / 8;
    const bool more = slot < end;
    if (more) {
      at = locate(first_id + slot);
      if (at.slabs > 0) begin(at);
    }
    epilogue<__bf16, EPI, 2 * MI, 2 * MJ, EA>(g, acc, per_b, done.a0, done.b0, done.ra, done.rb, done.ta,
                                                 done.range, wa, q, a_of, b_of, red);
    if (!more) break;
  }
}

// Arrays of their own, so that the compiler sees which copies a read does not
// meet; few enough for it to follow them all (A0 and B0 go together).
#define FCONV_TILE_LDS(H)                                                                      \
  __shared__ __attribute__((aligned(1024))) char ab0[2 * H * 128], b01[H * 128], a01[H * 128]; \
  __shared__ __attribute__((aligned(1024))) char ab1[2 * H * 128], b11[H * 128], a11[H * 128]

template <Order OA, Order OB, Epilogue EPI, int H, int NW>
__global__ __launch_bounds__(NW * 64, 2) void gemm_tile_kernel(GemmArgs g) {
  FCONV_TILE_LDS(H);
  __shared__ float2 red[EPI == kEpiLse ? 4 * H : 1];
  tile_work<OA, OB, EPI, H, NW>(g, ab0, b01, a01, ab1, b11, a11, red, blockIdx.x, gridDim.x);
}

// Two products in one launch, C[b, a] of x with B's k contiguous, of y with its rows:
// workgroups of y start as those of x end, so that neither leaves CUs idle at its end.
// The first blocks_x (a multiple of eight) are x's.  dx and dw of a gated layer of 1999
// x 1000 x 2731: 54 us (0.80 PFLOP/s; each alone leaves CUs idle), 70 apart.
template <Epilogue EPI_X, Epilogue EPI_Y, int H, int NW>
__global__ __launch_bounds__(NW * 64, 2) void gemm_tile_pair_kernel(GemmArgs x, GemmArgs y, unsigned blocks_x) {
  FCONV_TILE_LDS(H);
  __shared__ float2 red[1];
  const unsigned block = blockIdx.x;
  if (block < blocks_x)
    tile_work<kRow, kSum, EPI_X, H, NW>(x, ab0, b01, a01, ab1, b11, a11, red, block, blocks_x);
  else
    tile_work<kRow, kRow, EPI_Y, H, NW>(y, ab0, b01, a01, ab1, b11, a11, red, block - blocks_x,
                                        gridDim.x - blocks_x);
}

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

// Rows of bf16 from anywhere into rows of ld (a multiple of 8) from 16-byte
// boundaries, zeros past cols.  Four pieces of 16 bytes per thread in flight.
__global__ __launch_bounds__(256) void gemm_pack_kernel(const char* src, int64_t ld_src, int64_t rows, int cols,
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
__global__ __launch_bounds__(256) void gemm_sum_kernel(const float* part, int ranges, int64_t stride,
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
  if (scale) s *= scale[row * scale_step];
  int64_t to = row_map ? row_map[row] : row;
  if (to < 0) {
    to = -1 - to;
    s = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  store4<E>(out + (to * ld_out + c) * static_cast<int64_t>(sizeof(E)), s, cols - c);
}

// Zeros (dw of no tokens), of any number of elements.
template <typename E>
__global__ __launch_bounds__(256) void gemm_zero_kernel(char* out, int64_t ld, int64_t rows, int cols) {
  const E z = static_cast<E>(0.0f);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256)
      __builtin_memcpy(out + (row * ld + c) * static_cast<int64_t>(sizeof(E)), &z, sizeof(E));
}

// How a product is divided: the edge of its tiles (64: general kernel) and
// the ranges of its sum.
struct Split {
  int32_t edge, ranges;
  double us;  // by choose()'s account
};

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
// slab64, alone64: what a slab takes in the general kernel, busy and alone.
inline Split choose(int64_t na, int64_t nb, int64_t nk, bool tiled, bool split, double slab64 = 1.15,
                    double alone64 = 0.7) {
  struct Kind {
    int32_t edge;
    int64_t at_once;  // workgroups on the device
    double slab, slab_alone, tile;
  };
  const Kind kinds[] = {{256, 256, 1.0, 1.0, 5.0}, {128, 512, 0.7, 0.55, 5.0}, {64, 1024, slab64, alone64, 2.5}};
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

// Time (us) of packing a matrix: a launch, one read and one write.
inline double pack_us(int64_t rows, int64_t cols) { return 4.0 + 4.0 * static_cast<double>(rows) * static_cast<double>(cols) / 4e6; }

// Workgroups of the tiled kernel for n tiles: as many as the device holds at once (one
// or two a CU, by their LDS), in eighths; each takes every so manieth tile of its XCD's share.
inline unsigned tile_blocks(int64_t n, int edge) {
  const int64_t most = edge == 256 ? 256 : 512, blocks = round_up(n, 8);
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

// The kernel of a product: tiles of 64 (general), 128 or 256.
template <typename E, Order OA, Order OB, Epilogue EPI>
hipError_t launch_gemm(const GemmArgs& g, int edge, hipStream_t s) {
  const int64_t ta = ceil_div((EPI == kEpiGated ? 2ll : 1ll) * g.na, edge), tb = ceil_div(g.nb, edge);
  if constexpr (sizeof(E) == 2) {
    const dim3 grid(tile_blocks(ta * tb * g.ranges, edge));
    if (edge == 256)
      hipLaunchKernelGGL((gemm_tile_kernel<OA, OB, EPI, 128, 8>), grid, dim3(512), 0, s, g);
    else if (edge == 128)
      hipLaunchKernelGGL((gemm_tile_kernel<OA, OB, EPI, 64, 4>), grid, dim3(256), 0, s, g);
    if (edge != 64) return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(ta), static_cast<unsigned>(tb), static_cast<unsigned>(g.ranges));
  if constexpr (OB == kSum && (EPI == kEpiLse || EPI == kEpiGrad)) {
    // Some of the last tile's waves have no b: their loads of the last one again took as long as others (loss of 10 x
    // 343 x 41728 16.1 us, 13.3 without them; 130 29.4 and 27.7, 1030 x 343 x 9000 31.0 and 31.1).  Where every wave
    // has some, asking is for nothing (4096 x 1024 x 8192 fp32 557 us, 565 with it).
    if ((g.nb - 1) % 64 < 48) {
      hipLaunchKernelGGL((gemm_gen_kernel<E, OA, OB, EPI, true>), grid, dim3(256), 0, s, g);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((gemm_gen_kernel<E, OA, OB, EPI == kEpiStream ? kEpiOut : EPI == kEpiStoreStream ? kEpiStore : EPI>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

// Rows that the tiled kernel's copies may start at.
inline bool fits_tiles(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

// Whether rows of bf16 begin between dwords.
inline bool odd_rows(const Operand& o) { return (reinterpret_cast<uintptr_t>(o.p) & 3) != 0 || o.ld % 2 != 0; }

inline hipError_t launch_pack(const void* src, int64_t ld_src, int64_t rows, int32_t cols, char* dst, int64_t ld,
                       hipStream_t s) {
  hipLaunchKernelGGL(gemm_pack_kernel, dim3(static_cast<unsigned>(ceil_div(rows * (ld / 8), 1024))), dim3(256), 0, s,
                     static_cast<const char*>(src), ld_src, rows, cols, dst, ld);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sum(const float* part, int ranges, int64_t stride, int64_t ld, int rows,
                      const int32_t* n_live, const int32_t* row_map, const float* scale, int scale_step,
                      int cols, char* out, int64_t ld_out, hipStream_t s) {
  const int64_t quads = static_cast<int64_t>(rows) * ((cols + 3) / 4);
  if (ranges > 8 && quads <= 1 << 16)
    hipLaunchKernelGGL((gemm_sum_kernel<E, 8>), dim3(static_cast<unsigned>(ceil_div(quads, 32))), dim3(256), 0, s,
                       part, ranges, stride, ld, rows, n_live, row_map, scale, scale_step, cols, out, ld_out);
  else
    hipLaunchKernelGGL((gemm_sum_kernel<E, 1>), dim3(static_cast<unsigned>(ceil_div(quads, 256))), dim3(256), 0, s,
                       part, ranges, stride, ld, rows, n_live, row_map, scale, scale_step, cols, out, ld_out);
  return hipGetLastError();
}

}  // namespace
}  // namespace fconv

#endif  // FCONV_GEMM_H
