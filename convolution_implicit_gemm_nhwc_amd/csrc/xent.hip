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
// cores' type): at most 2^-9 of a value below 1, where dloss q, at the same
// cost, would be off by as much as 2^-8 and, with the mean's equal dloss, by
// the same factor in every token (measured on 32 tokens of 1000 classes: error of dw
// 0.0037 against 0.0018).
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
constexpr int64_t kMaxGroups = (1 << 23) - 8;  // a launch's threads stay below 2^32
constexpr int64_t kMaxLd = 1 << 21;
constexpr int32_t kMaxD = 1 << 20, kMaxTV = 1 << 24;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// Which index of an operand is contiguous in memory: the sum's (element
// (r, k) at r * ld + k) or the row's (at k * ld + r).
enum Order { kSum, kRow };

struct Operand {
  const char* p;
  int64_t ld;  // elements
};

enum Epilogue { kEpiLse, kEpiGrad, kEpiOut, kEpiPart };

struct GemmArgs {
  Operand a, b;
  int32_t na, nb, nk;
  // Number of live tokens (device), replacing nb (kSum order of b) or nk
  // (kRow order of b); NULL if there is none.
  const int32_t* n_live;
  int32_t k_split;  // length of one range of k, blockIdx.z ranges
  // kEpiLse: partial (max, sum) at [tile of a][ld_out + b]; kEpiGrad: g;
  // kEpiOut: C; kEpiPart: fp32 C of this range at range * nb_max * ld_out.
  char* out;
  int64_t ld_out;
  int64_t part_stride;        // elements between ranges
  const int32_t* row_map;     // kEpiOut: row of C for b, or NULL
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

// What exponents are taken relative to: the maximum, or 0 where it is
// infinite (inf - inf would be NaN; exp(inf) = inf and exp(-inf) = 0 are right).
__device__ inline float base_of(float m) { return __builtin_fabsf(m) < __builtin_inff() ? m : 0.0f; }
__device__ inline float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// (m, s) of two sets of logits joined; s counts from base_of(m).
__device__ inline void join(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2), b = base_of(mm);
  // An empty or all -inf set has s = 0, whose factor must not be NaN or inf.
  const float f1 = exp_of(base_of(m) - b), f2 = exp_of(base_of(m2) - b);
  s = (s == 0.0f ? 0.0f : s * f1) + (s2 == 0.0f ? 0.0f : s2 * f2);
  m = mm;
}

// q of one logit.
__device__ inline float grad_of(float z, float lse, bool hit) {
  const float p = exp_of(z - lse);
  return hit ? p - 1.0f : p;
}

// ------------------------------------------------------------ general kernel
//
// Any type, alignment and stride: 64 x 64 tiles, four waves of 32 x 32, slabs
// of 128 bytes of k staged through registers into one of two LDS buffers
// (rows of 128 + 16 bytes, so that fragment reads spread over the banks).  A
// fragment is eight consecutive k of a row; for fp32 the eight 16x16x4
// products take one of them each, in both operands alike.
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
  } else {
    constexpr int TPK = 64 / N;
    const int k = tid / TPK, c = (tid % TPK) * N;
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<E*>(buf + (c + i) * Gen<E>::PITCH + k * sizeof(E)) = v[i];
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

template <typename E, Order OA, Order OB, Epilogue EPI>
__global__ __launch_bounds__(256) void xent_gen_kernel(GemmArgs g) {
  using G = Gen<E>;
  using Frag = std::conditional_t<sizeof(E) == 2, bf16x8, f32x8>;
  __shared__ __attribute__((aligned(16))) char buf[2][2][G::BUF];
  const int live = g.n_live ? *g.n_live : 0;
  const int nb = g.n_live && OB == kSum ? live : g.nb;
  const int nk = g.n_live && OB == kRow ? live : g.nk;
  const int64_t a0 = static_cast<int64_t>(blockIdx.x) * 64, b0 = static_cast<int64_t>(blockIdx.y) * 64;
  if (b0 >= nb) return;
  const int ra = static_cast<int>(min<int64_t>(g.na - a0, 64)), rb = static_cast<int>(min<int64_t>(nb - b0, 64));
  const int64_t k0 = static_cast<int64_t>(blockIdx.z) * g.k_split;
  const int64_t k1 = min<int64_t>(nk, k0 + g.k_split);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave & 1, wb = wave >> 1, r = lane & 15, q = lane >> 4;

  f32x4 acc[2][2] = {};
  const int slabs = k1 > k0 ? static_cast<int>(ceil_div(k1 - k0, G::SLAB)) : 0;
  E va[32 / G::ES], vb[32 / G::ES];
  if (slabs > 0) {
    gen_load<E, OA>(g.a, a0, ra, k0, k1, va);
    gen_load<E, OB>(g.b, b0, rb, k0, k1, vb);
  }
  for (int s = 0; s < slabs; ++s) {
    char* ba = buf[s & 1][0];
    char* bb = buf[s & 1][1];
    gen_write<E, OA>(ba, va);
    gen_write<E, OB>(bb, vb);
    __syncthreads();
    if (s + 1 < slabs) {
      gen_load<E, OA>(g.a, a0, ra, k0 + (s + 1) * static_cast<int64_t>(G::SLAB), k1, va);
      gen_load<E, OB>(g.b, b0, rb, k0 + (s + 1) * static_cast<int64_t>(G::SLAB), k1, vb);
    }
#pragma unroll
    for (int kk = 0; kk < G::SLAB; kk += 32) {
      Frag fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        __builtin_memcpy(&fa[i], ba + (wa * 32 + 16 * i + r) * G::PITCH + (kk + 8 * q) * G::ES, 8 * G::ES);
        __builtin_memcpy(&fb[i], bb + (wb * 32 + 16 * i + r) * G::PITCH + (kk + 8 * q) * G::ES, 8 * G::ES);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mma8(fa[i], fb[j], acc[i][j]);
    }
  }

  if constexpr (EPI == kEpiLse) {
    __shared__ float2 red[2][64];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = wb * 32 + 16 * j + r;
      const int64_t tgt = b < rb ? g.target[b0 + b] : -1;
      float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int a = wa * 32 + 16 * i + 4 * q + e;
          if (a < ra) m = fmaxf(m, acc[i][j][e]);
          if (a < ra && b < rb && tgt == a0 + a) g.target_logit[b0 + b] = acc[i][j][e];
        }
      const float base = base_of(m);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (wa * 32 + 16 * i + 4 * q + e < ra) s += exp_of(acc[i][j][e] - base);
#pragma unroll
      for (int x = 16; x < 64; x *= 2) {
        const float m2 = __shfl_xor(m, x), s2 = __shfl_xor(s, x);
        join(m, s, m2, s2);
      }
      if (q == 0) red[wa][b] = make_float2(m, s);
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(rb)) {
      const float2 p0 = red[0][threadIdx.x], p1 = red[1][threadIdx.x];
      float m = p0.x, s = p0.y;
      join(m, s, p1.x, p1.y);
      reinterpret_cast<float2*>(g.out)[blockIdx.x * g.ld_out + b0 + threadIdx.x] = make_float2(m, s);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = wb * 32 + 16 * j + r;
      if (b >= rb) continue;
      if constexpr (EPI == kEpiGrad) {
        const int tgt = g.live_target[b0 + b];
        const float lse = tgt < 0 ? __builtin_nanf("") : g.lse[b0 + b];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t a = a0 + wa * 32 + 16 * i + 4 * q;
          if (a >= g.na_pad) continue;
          f32x4 t;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            t[e] = a + e < g.na ? grad_of(acc[i][j][e], lse, tgt == g.v0 + a + e) : 0.0f;
          store4<E>(g.out + ((b0 + b) * g.ld_out + a) * G::ES, t, 4);
        }
      } else {
        const int64_t row = EPI == kEpiOut && g.row_map ? g.row_map[b0 + b] : b0 + b;
        const float scale = EPI == kEpiOut ? g.scale[(b0 + b) * g.scale_step] : 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t a = a0 + wa * 32 + 16 * i + 4 * q;
          const int n = static_cast<int>(g.na - a);
          if (n <= 0) continue;
          if constexpr (EPI == kEpiOut)
            store4<E>(g.out + (row * g.ld_out + a) * G::ES, acc[i][j] * scale, n);
          else
            store4<float>(g.out + (blockIdx.z * g.part_stride + row * g.ld_out + a) * 4, acc[i][j], n);
        }
      }
    }
  }
}

// ------------------------------------------------------------ small kernels

// Joins the tiles of 64 tokens: four threads per token, each every fourth
// tile, met in LDS.
__global__ __launch_bounds__(256) void xent_join_kernel(const float2* part, int tiles, int64_t ld,
                                                        const float* target_logit,
                                                        const int64_t* target, int64_t ignore,
                                                        int T, int V, float* loss, float* lse) {
  __shared__ float2 red[4][64];
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 64 + c;
  float m = -__builtin_inff(), s = 0.0f;
  if (t < T)
    for (int i = k; i < tiles; i += 4) {
      const float2 p = part[i * ld + t];
      join(m, s, p.x, p.y);
    }
  red[k][c] = make_float2(m, s);
  __syncthreads();
  if (k != 0 || t >= T) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) join(m, s, red[i][c].x, red[i][c].y);
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

// Gathers the live tokens among 16, in order: a workgroup counts the live
// ones before its own and finds the largest |dloss|, then each wave copies the
// rows of four tokens.
template <typename E>
__global__ __launch_bounds__(256) void xent_gather_kernel(GatherArgs g) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 16;
  int n = 0, m = 0;
  if (g.blocks) {
    const int64_t own = t0 / 1024, blocks = (g.T + 1023) / 1024;
    for (int64_t i = threadIdx.x; i < blocks; i += 256) {
      const int2 b = g.blocks[i];
      if (i < own) n += b.x;
      m = max(m, b.y);
    }
    for (int64_t t = own * 1024 + threadIdx.x; t < t0; t += 256) n += g.target[t] != g.ignore;
  } else {
    for (int64_t t = threadIdx.x; t < g.T; t += 256)
      if (g.target[t] != g.ignore) {
        n += t < t0;
        m = max(m, abs_bits(g.dloss[t]));
      }
  }
  const int2 stats = block_stats(n, m);
  const int before = stats.x;
  const float c = __builtin_bit_cast(float, stats.y);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mine = t0 + lane;
  const int64_t tgt = lane < 16 && mine < g.T ? g.target[mine] : g.ignore;
  const uint64_t live = __ballot(tgt != g.ignore);
  const int pos = before + __popcll(live & ((1ull << lane) - 1));
  if (wave == 0 && tgt != g.ignore) {
    g.index[pos] = static_cast<int32_t>(mine);
    g.live_target[pos] = tgt >= 0 && tgt < g.V ? static_cast<int32_t>(tgt) : -1;
    g.live_lse[pos] = g.lse[mine];
    g.live_dloss[pos] = g.dloss[mine];
  }
  if (threadIdx.x == 0 && t0 + 16 >= g.T) {
    *g.n_live = before + __popcll(live);
    *g.c = c;
  }
  constexpr int N = 16 / sizeof(E);
  for (int i = 4 * wave; i < 4 * wave + 4; ++i) {
    if (t0 + i >= g.T) break;
    if (live >> i & 1) {
      const int64_t to = before + __popcll(live & ((1ull << i) - 1));
      const char* src = g.h + (t0 + i) * g.ldh * static_cast<int64_t>(sizeof(E));
      const int64_t at = to * g.ld_live * static_cast<int64_t>(sizeof(E));
      const float ratio = c > 0.0f ? g.dloss[t0 + i] / c : g.dloss[t0 + i];
      for (int col = lane * N; col < g.ld_live; col += 64 * N) {
        E v[N];
        if (col + N <= g.D) {
          __builtin_memcpy(v, src + col * sizeof(E), 16);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            v[j] = static_cast<E>(0.0f);
            if (col + j < g.D) __builtin_memcpy(&v[j], src + (col + j) * sizeof(E), sizeof(E));
          }
        }
        __builtin_memcpy(g.h_live + at + col * sizeof(E), v, 16);
        if (g.rh_live) {
#pragma unroll
          for (int j = 0; j < N; ++j) v[j] = static_cast<E>(ratio * static_cast<float>(v[j]));
          __builtin_memcpy(g.rh_live + at + col * sizeof(E), v, 16);
        }
      }
    } else if (g.dh) {
      char* dst = g.dh + (t0 + i) * g.lddh * static_cast<int64_t>(sizeof(E));
      const E z = static_cast<E>(0.0f);
      for (int c = lane; c < g.D; c += 64) __builtin_memcpy(dst + c * sizeof(E), &z, sizeof(E));
    }
  }
}

// C[row, a] = sum of the ranges' partial sums, in order; four a per thread.
template <typename E>
__global__ __launch_bounds__(256) void xent_sum_kernel(const float* part, int ranges, int64_t stride,
                                                       int64_t ld, int rows, const int32_t* n_live,
                                                       const int32_t* row_map, const float* scale,
                                                       int scale_step, int cols, char* out,
                                                       int64_t ld_out) {
  const int quads = (cols + 3) / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = i / quads;
  const int c = static_cast<int>(i - row * quads) * 4;
  if (row >= (n_live ? *n_live : rows)) return;
  f32x4 s = {};
  for (int k = 0; k < ranges; ++k)  // rows of ld floats, a multiple of 4
    s += *reinterpret_cast<const f32x4*>(part + k * stride + row * ld + c);
  s *= scale[row * scale_step];
  store4<E>(out + ((row_map ? row_map[row] : row) * ld_out + c) * static_cast<int64_t>(sizeof(E)), s,
            cols - c);
}

// Zeros (dw of no tokens).
template <typename E>
__global__ __launch_bounds__(256) void xent_zero_kernel(char* out, int64_t ld, int64_t rows, int cols) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = i / cols;
  if (row >= rows) return;
  const E z = static_cast<E>(0.0f);
  __builtin_memcpy(out + (row * ld + i % cols) * static_cast<int64_t>(sizeof(E)), &z, sizeof(E));
}

}  // namespace
}  // namespace fconv

struct fconv_xent_plan_s {
  fconv_xent_desc d;
  int32_t es;
  // Forward workspace: partial (max, sum) [a_tiles][T], target logits [T].
  int64_t a_tiles;
  size_t fwd_target, fwd_bytes;
  // Backward workspace.
  int64_t ld_live;               // row stride of the gathered h
  int32_t piece, pieces;         // vocabulary columns of a piece
  int64_t ld_g;
  int32_t dh_ranges, dh_split;   // ranges of a piece's k, and their length
  int32_t dw_ranges, dw_split;
  size_t o_g, o_h, o_index, o_target, o_lse, o_dloss, o_n, o_c, o_blocks, o_rh, o_dh, o_dw, bwd_bytes;
};

namespace fconv {
namespace {

constexpr int64_t kGBytes = 256 << 20;  // of g at a time: it stays in the 256 MB last-level cache

// Ranges of a sum of nk terms for `tiles` output tiles: enough workgroups to
// fill the device twice over, none shorter than 256 terms.
int32_t ranges_of(int64_t tiles, int64_t nk) {
  const int64_t want = ceil_div(512, tiles);
  const int64_t most = ceil_div(nk, 256);
  const int64_t n = want < most ? want : most;
  return static_cast<int32_t>(n < 1 ? 1 : n);
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

template <typename E, Order OA, Order OB, Epilogue EPI>
hipError_t launch_gemm(const GemmArgs& g, int ranges, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(g.na, 64)), static_cast<unsigned>(ceil_div(g.nb, 64)),
                  static_cast<unsigned>(ranges));
  hipLaunchKernelGGL((xent_gen_kernel<E, OA, OB, EPI>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

template <typename E>
hipError_t run_forward(const fconv_xent_plan_s* p, const fconv_xent_args* args, hipStream_t s) {
  const fconv_xent_desc& d = p->d;
  char* ws = static_cast<char*>(args->workspace);
  GemmArgs g = {};
  g.a = Operand{static_cast<const char*>(args->w), args->ldw};
  g.b = Operand{static_cast<const char*>(args->h), args->ldh};
  g.na = d.V;
  g.nb = d.T;
  g.nk = g.k_split = d.D;
  g.out = ws;
  g.ld_out = d.T;
  g.target = args->target;
  g.target_logit = reinterpret_cast<float*>(ws + p->fwd_target);
  hipError_t e = launch_gemm<E, kSum, kSum, kEpiLse>(g, 1, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(xent_join_kernel, dim3(static_cast<unsigned>(ceil_div(d.T, 64))), dim3(256), 0, s,
                     reinterpret_cast<const float2*>(ws), static_cast<int>(p->a_tiles),
                     static_cast<int64_t>(d.T), g.target_logit, args->target, d.ignore_index, d.T, d.V,
                     args->loss, args->lse);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sum(const float* part, int ranges, int64_t stride, int64_t ld, int rows,
                      const int32_t* n_live, const int32_t* row_map, const float* scale, int scale_step,
                      int cols, char* out, int64_t ld_out, hipStream_t s) {
  const int64_t threads = static_cast<int64_t>(rows) * ((cols + 3) / 4);
  hipLaunchKernelGGL(xent_sum_kernel<E>, dim3(static_cast<unsigned>(ceil_div(threads, 256))), dim3(256), 0, s,
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
    const int64_t n = static_cast<int64_t>(d.V) * d.D;
    hipLaunchKernelGGL(xent_zero_kernel<E>, dim3(static_cast<unsigned>(ceil_div(n, 256))), dim3(256), 0, s,
                       static_cast<char*>(args->dw), args->lddw, static_cast<int64_t>(d.V), d.D);
    return hipGetLastError();
  }
  GatherArgs ga = {};
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
  ga.index = reinterpret_cast<int32_t*>(ws + p->o_index);
  ga.live_target = reinterpret_cast<int32_t*>(ws + p->o_target);
  ga.live_lse = reinterpret_cast<float*>(ws + p->o_lse);
  ga.live_dloss = reinterpret_cast<float*>(ws + p->o_dloss);
  ga.n_live = reinterpret_cast<int32_t*>(ws + p->o_n);
  ga.dh = static_cast<char*>(args->dh);
  ga.lddh = args->lddh;
  ga.c = reinterpret_cast<float*>(ws + p->o_c);
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
  hipLaunchKernelGGL(xent_gather_kernel<E>, dim3(static_cast<unsigned>(ceil_div(d.T, 16))), dim3(256), 0, s, ga);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  for (int i = 0; i < p->pieces; ++i) {
    const int32_t v0 = i * p->piece;
    const int32_t nv = d.V - v0 < p->piece ? d.V - v0 : p->piece;
    const char* w = static_cast<const char*>(args->w) + v0 * args->ldw * p->es;
    GemmArgs g = {};
    g.a = Operand{w, args->ldw};
    g.b = Operand{ga.h_live, p->ld_live};
    g.na = nv;
    g.nb = d.T;
    g.nk = g.k_split = d.D;
    g.n_live = ga.n_live;
    g.out = ws + p->o_g;
    g.ld_out = p->ld_g;
    g.live_target = ga.live_target;
    g.lse = ga.live_lse;
    g.v0 = v0;
    g.na_pad = static_cast<int32_t>(round_up(nv, 8));
    if ((e = launch_gemm<E, kSum, kSum, kEpiGrad>(g, 1, s)) != hipSuccess) return e;
    if (args->dh) {
      GemmArgs c = {};
      c.a = Operand{w, args->ldw};
      c.b = Operand{ws + p->o_g, p->ld_g};
      c.na = d.D;
      c.nb = d.T;
      c.nk = nv;
      c.n_live = ga.n_live;
      c.k_split = p->dh_split;
      const int ranges = static_cast<int>(ceil_div(nv, p->dh_split));
      if (p->pieces * p->dh_ranges == 1) {
        c.out = static_cast<char*>(args->dh);
        c.ld_out = args->lddh;
        c.row_map = ga.index;
        c.scale = ga.live_dloss;
        c.scale_step = 1;
        e = launch_gemm<E, kRow, kSum, kEpiOut>(c, 1, s);
      } else {
        c.ld_out = round_up(d.D, 4);
        c.part_stride = c.ld_out * d.T;
        c.out = ws + p->o_dh + static_cast<size_t>(c.part_stride) * 4 * i * p->dh_ranges;
        e = launch_gemm<E, kRow, kSum, kEpiPart>(c, ranges, s);
        if (e == hipSuccess && i == p->pieces - 1)
          e = launch_sum<E>(reinterpret_cast<const float*>(ws + p->o_dh), i * p->dh_ranges + ranges,
                            c.part_stride, c.ld_out, d.T, ga.n_live, ga.index, ga.live_dloss, 1, d.D,
                            static_cast<char*>(args->dh), args->lddh, s);
      }
      if (e != hipSuccess) return e;
    }
    if (args->dw) {
      char* dw = static_cast<char*>(args->dw) + v0 * args->lddw * p->es;
      GemmArgs c = {};
      c.a = Operand{ga.rh_live, p->ld_live};
      c.b = Operand{ws + p->o_g, p->ld_g};
      c.na = d.D;
      c.nb = nv;
      c.nk = d.T;
      c.n_live = ga.n_live;
      c.k_split = p->dw_split;
      if (p->dw_ranges == 1) {
        c.out = dw;
        c.ld_out = args->lddw;
        c.scale = ga.c;
        e = launch_gemm<E, kRow, kRow, kEpiOut>(c, 1, s);
      } else {
        c.ld_out = round_up(d.D, 4);
        c.part_stride = c.ld_out * nv;
        c.out = ws + p->o_dw;
        e = launch_gemm<E, kRow, kRow, kEpiPart>(c, p->dw_ranges, s);
        if (e == hipSuccess)
          e = launch_sum<E>(reinterpret_cast<const float*>(ws + p->o_dw), p->dw_ranges, c.part_stride,
                            c.ld_out, nv, nullptr, nullptr, ga.c, 0, d.D, dw, args->lddw, s);
      }
      if (e != hipSuccess) return e;
    }
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
  // Every launch stays below kMaxGroups workgroups (and 65535 in grid.y).
  if (ceil_div(d.T, 64) > 65535 || ceil_div(d.V, 64) * ceil_div(d.T, 64) > kMaxGroups ||
      ceil_div(d.D, 64) * ceil_div(d.T, 64) > kMaxGroups || ceil_div(d.V, 256) * d.D > kMaxGroups ||
      ceil_div(d.T, 256) * d.D > kMaxGroups)
    return FCONV_ERR_UNSUPPORTED;
  fconv_xent_plan_s* p = new (std::nothrow) fconv_xent_plan_s();
  if (!p) return FCONV_ERR_INVALID_ARG;
  p->d = d;
  p->es = d.dtype == FCONV_BF16 ? 2 : 4;
  p->a_tiles = ceil_div(d.V, 64);
  p->fwd_target = static_cast<size_t>(p->a_tiles) * d.T * 8;
  p->fwd_bytes = p->fwd_target + static_cast<size_t>(d.T) * 4;

  if (d.T > 0) {
    const int64_t T = d.T;
    p->ld_live = round_up(d.D, 64);
    int64_t piece = kGBytes / (T * p->es) / 256 * 256;
    if (piece < 256) piece = 256;
    if (piece > 65535 * 64) piece = 65535 * 64;  // grid.y of dw
    if (piece > d.V) piece = d.V;
    p->pieces = static_cast<int32_t>(ceil_div(d.V, piece));
    // Pieces of about the same length.
    piece = round_up(ceil_div(d.V, p->pieces), 256);
    if (piece > d.V) piece = d.V;
    p->piece = static_cast<int32_t>(piece);
    p->pieces = static_cast<int32_t>(ceil_div(d.V, piece));
    p->ld_g = round_up(piece, 64);
    const int64_t td = ceil_div(d.D, 64);
    p->dh_split = static_cast<int32_t>(
        round_up(ceil_div(piece, ranges_of(td * ceil_div(T, 64), piece)), 64));
    p->dh_ranges = static_cast<int32_t>(ceil_div(piece, p->dh_split));
    p->dw_split = static_cast<int32_t>(round_up(ceil_div(T, ranges_of(td * ceil_div(piece, 64), T)), 64));
    p->dw_ranges = static_cast<int32_t>(ceil_div(T, p->dw_split));
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
    const size_t dh_parts = static_cast<size_t>(p->pieces) * p->dh_ranges;
    p->o_dh = take(dh_parts > 1 ? dh_parts * T * ld4 : 0);
    p->o_dw = take(p->dw_ranges > 1 ? static_cast<size_t>(p->dw_ranges) * piece * ld4 : 0);
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

fconv_status fconv_xent_plan_destroy(fconv_xent_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
