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
// The products as gemm.h has them, C[b, a] = sum_k A(a, k) B(b, k):
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
#include "gemm.h"

namespace fconv {
namespace {

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

// The first workgroups take dh, the others (if dw is wanted) dw's tiles.
template <typename E, int MT>
__global__ __launch_bounds__(256) void xent_few_grads_kernel(GemmArgs dh, GemmArgs dw) {
  __shared__ GenLds<E> lds;
  static_assert(sizeof(lds.buf) >= 4 * MT * 64 * sizeof(f32x4), "the sums fit");
  const int n_dh = (dh.na + 15) / 16, i = static_cast<int>(blockIdx.x) - n_dh;
  if (i < 0) {
    few_rows<E, MT, kEpiOut>(dh, reinterpret_cast<f32x4*>(&lds.buf[0][0][0]), static_cast<int>(blockIdx.x) * 16);
  } else {
    const int ta = (dw.na + 63) / 64;
    gen_tile<E, kRow, kRow, kEpiOut>(dw, lds, i % ta, i / ta, 0);
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

constexpr int32_t kFewTokens = 64;
// Vocabularies up to this take few_dh: it grows with the vocabulary, the tiles'
// way costs a launch more (both gradients of 16 x 512 x 1000 10.0 instead of 12.6
// us, x 2048 12.0 and 13.7, x 4096 15.9 and 15.7; of 64 tokens 14.2 and 14.6, 18.4
// and 15.8).
int32_t few_dh_v(int32_t T) { return T <= 32 ? 2048 : 1024; }
// Workgroups of the few-token forward kernel.
int64_t few_groups(int32_t V) { return ceil_div(V, 32) < 1024 ? round_up(ceil_div(V, 32), 8) : 1024; }

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
hipError_t run_backward(const fconv_xent_plan_s* p, const fconv_xent_args* args, hipStream_t s) {
  const fconv_xent_desc& d = p->d;
  char* ws = static_cast<char*>(args->workspace);
  hipError_t e;
  if (d.T == 0) {
    if (!args->dw) return hipSuccess;
    hipLaunchKernelGGL(gemm_zero_kernel<E>, dim3(d.V < 4096 ? d.V : 4096), dim3(256), 0, s,
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
