// Gated feed-forward layer on gfx950 (CDNA4), its gradients, and their C ABI
// (include/fconv_gated.h).
//
//   [g u] = x w^T     y = act(g) u     dg = dy u act'(g)     du = dy act(g)
//   dx = [dg du] w    dw = [dg du]^T x
//
// The products as gemm.h has them, C[b, a] = sum_k A(a, k) B(b, k):
//   forward  a = f, b = t, k = d: A = w, B = x, both with k contiguous; a tile
//            holds the same f of g and of u, so y leaves the registers as a product
//   dx       a = d, b = t, k = g's f, then u's: A = w with a contiguous, B = [dg du]
//   dw       a = d, b = g's f, then u's, k = t: A = x, B = [dg du], a and b contiguous
//
// g and u are kept for the gradients: computing them again would take half as
// much as the gradients' own products (4 T D F operations beside 8), writing and
// reading them 16 T F bytes.  They are kept in fp32: rounded to bf16, with dg and
// du that are rounded too, bf16 gradients were off by 0.0030 of their norm instead
// of 0.0023, of which 0.0017 is their own rounding.
//
// Measured, bf16: forward in tiles 8192 x 4096 x 12288 1.20 to 1.28 ms (1.29 to
// 1.37 PFLOP/s), 8192 x 4096 x 8192 with g and u kept 0.90 to 0.94 ms (0.79 without:
// 537 MB of stores at the tiles' ends); its dx 0.77 to 0.80 ms and dw the same (1.38 to
// 1.43 PFLOP/s): matrix cores at the clock that power allows.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <new>
#include <type_traits>

#include "fconv_gated.h"
#include "gemm.h"

namespace fconv {
namespace {

static_assert(kSilu == FCONV_ACT_SILU && kGelu == FCONV_ACT_GELU && kGeluTanh == FCONV_ACT_GELU_TANH &&
                  kActRelu == FCONV_ACT_RELU,
              "activations as the header counts them");

// ------------------------------------------------------------- few tokens
//
// Few tokens: the time is w's way out of memory, so fragments of both
// operands go straight into registers, from any address, without LDS or
// barriers.  A workgroup owns 16 f of both projections and 16 MT tokens (at most 32
// with ODD, whose fragments take more registers); its NW waves take turns at
// steps of 128 bytes of k, the next turn's loads in flight, and add their sums
// in LDS, in order; wave j then finishes tokens 16 j .. + 15.  One token of 4096 x
// 12288 bf16: 33 us, w at 6.1 TB/s.
//
// More tokens of a layer with few f and a long k have so few tiles that one's slabs,
// one after another, are the time.  Here the waves share k, and tokens are spread
// over workgroups until the device is full: 128 x 8192 x 512 bf16 24 us instead of
// 80, fp32 47 instead of 197; 200 x 4000 x 300 13 and 43, 32 and 98.
struct GatedFew {
  const char* w;
  int64_t ldw;
  const char* x;
  int64_t ldx;
  char* y;
  int64_t ldy;
  float* kept;
  int64_t ld_kept;
  int32_t T, D, F, act;
};

template <typename E, bool ODD, int MT, int NW>
__global__ __launch_bounds__(NW * 64, 2) void gated_few_kernel(GatedFew f) {
  using Frag = std::conditional_t<sizeof(E) == 2, bf16x8, f32x8>;
  using R = Raw<8 * sizeof(E), ODD>;
  constexpr int ES = sizeof(E), STEP = 128 / ES, KK = STEP / 32;
  __shared__ f32x4 sums[NW][MT * 2][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  // Tokens from t0 on; workgroups of the same f and other tokens follow on the same XCD (every eighth).
  const int blocks = (f.T + 16 * MT - 1) / (16 * MT);
  const int t0 = static_cast<int>(blockIdx.x / 8 % blocks) * 16 * MT;
  const int f0 = static_cast<int>(blockIdx.x / (8 * blocks) * 8 + blockIdx.x % 8) * 16;
  if (f0 >= f.F) return;
  const int full = f.D / STEP;  // whole steps

  // Rows past the last one read it again; they are not stored.
  const char *xp[MT], *wp[2];
  uint32_t sa[2], sb[MT];  // steps are whole dwords: the same in all of them
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    xp[j] = f.x + (static_cast<int64_t>(min(t0 + 16 * j + r, f.T - 1)) * f.ldx + 8 * q) * ES;
    sb[j] = R::shift_of(xp[j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    wp[i] = f.w + ((static_cast<int64_t>(i) * f.F + min(f0 + r, f.F - 1)) * f.ldw + 8 * q) * ES;
    sa[i] = R::shift_of(wp[i]);
  }
  f32x4 acc[MT][2] = {};
  struct Turn {
    R a[2][KK], b[MT][KK];
  };
  auto load = [&](Turn& x, int step) __attribute__((always_inline)) {
    const int64_t at = static_cast<int64_t>(step) * 128;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) x.a[i][k].load(wp[i] + at + k * 32 * ES);
#pragma unroll
      for (int j = 0; j < MT; ++j) x.b[j][k].load(xp[j] + at + k * 32 * ES);
    }
  };
  auto multiply = [&](const Turn& x) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      Frag a[2], b[MT];
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] = x.a[i][k].template get<Frag>(sa[i]);
#pragma unroll
      for (int j = 0; j < MT; ++j) b[j] = x.b[j][k].template get<Frag>(sb[j]);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[j][i] = mma8(a[i], b[j], acc[j][i]);
    }
  };
  Turn now, next;
  int step = wave;
  if (step < full) load(now, step);
  for (; step < full; step += 2 * NW) {
    if (step + NW < full) load(next, step + NW);
    multiply(now);
    if (step + NW >= full) break;
    if (step + 2 * NW < full) load(now, step + 2 * NW);
    multiply(next);
  }
  if (full % NW == wave && full * STEP < f.D) {  // the rest of k
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const int64_t at = static_cast<int64_t>(full) * STEP + k * 32;
      const int n = static_cast<int>(f.D - at) - 8 * q;  // elements of this lane's eight
      auto part = [&](const char* p) __attribute__((always_inline)) {
        return f.D >= 8 ? row_end<Frag, R, ES>(p + at * ES, n) : row_end_short<Frag, E>(p + at * ES, n);
      };
      Frag a[2], b[MT];
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] = part(wp[i]);
#pragma unroll
      for (int j = 0; j < MT; ++j) b[j] = part(xp[j]);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[j][i] = mma8(a[i], b[j], acc[j][i]);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) sums[wave][j * 2 + i][lane] = acc[j][i];
  __syncthreads();
  const int t = t0 + 16 * wave + r, at = f0 + 4 * q;
  if (wave >= MT || t >= f.T || at >= f.F) return;
  f32x4 z[2][1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    z[i][0] = sums[0][wave * 2 + i][lane];
#pragma unroll
    for (int x = 1; x < NW; ++x) z[i][0] += sums[x][wave * 2 + i][lane];
  }
  if (f.kept) {
    float* row = f.kept + 2 * t * f.ld_kept + at;  // rows are whole fours
    *reinterpret_cast<f32x4*>(row) = z[0][0];
    *reinterpret_cast<f32x4*>(row + f.ld_kept) = z[1][0];
  }
  activate(z, 0, f.act);
  store4<E>(f.y + (t * f.ldy + at) * ES, z[0][0] * z[1][0], f.F - at);
}

// ----------------------------------------------------------------- dg and du
//
// [dg du] in rows of ld_dz, zeros past 2 F (what reads them takes whole pieces, and
// multiplies the rest by zeros).  A thread takes eight f of a row: 3 T F elements are
// read and 2 T F written (8192 x 8192 bf16, g and u in fp32: 0.94 GB in 190 to 203 us,
// 4.6 to 4.9 TB/s, as a copy).
struct GatedDz {
  const float* kept;
  int64_t ld_kept;
  const char* dy;
  int64_t lddy;
  char* dz;
  int64_t ld_dz;
  int32_t T, F, act;
};

// f(act and act' of a gate) of the activation.
template <typename F>
__device__ inline void with_act(int act, F f) {
  switch (act) {
    case kSilu: return f(act_grad<kSilu>);
    case kGelu: return f(act_grad<kGelu>);
    case kGeluTanh: return f(act_grad<kGeluTanh>);
    default: return f(act_grad<kActRelu>);
  }
}
// The two gradients of one f, rounded as they are multiplied.  In bf16 that is half a
// step of each: dx and dw are off by 0.0023 of their norm, 0.0017 of which is their own
// rounding (0.0026 from what fp32 in between gives).  As two bf16 each they would
// take twice the gradients' products.
template <typename E>
__device__ inline E dg_of(float dy, float u, float2 a) { return static_cast<E>(dy * u * a.y); }
template <typename E>
__device__ inline E du_of(float dy, float2 a) { return static_cast<E>(dy * a.x); }

template <typename E>
__global__ __launch_bounds__(256) void gated_dz_kernel(GatedDz z) {
  constexpr int64_t ES = sizeof(E);
  const uint32_t per_row = static_cast<uint32_t>(z.ld_kept / 8);
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;  // below 2^30: T F is at most 2^32
  const int64_t row = i / per_row;
  if (row >= z.T) return;
  const int c = static_cast<int>(i - static_cast<uint32_t>(row) * per_row) * 8;
  const int n = min(z.F - c, 8);
  float g[8], u[8];
  E dy[8], dg[8], du[8];
  const float* kept = z.kept + 2 * row * z.ld_kept + c;
  __builtin_memcpy(g, __builtin_assume_aligned(kept, 16), sizeof(g));
  __builtin_memcpy(u, __builtin_assume_aligned(kept + z.ld_kept, 16), sizeof(u));
  const char* src = z.dy + (row * z.lddy + c) * ES;
  if (n == 8) {
    __builtin_memcpy(dy, src, sizeof(dy));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dy[e] = static_cast<E>(0.0f);
      if (e < n) __builtin_memcpy(&dy[e], src + e * ES, ES);
    }
  }
  with_act(z.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 a = act(g[e]);
      dg[e] = dg_of<E>(static_cast<float>(dy[e]), u[e], a);
      du[e] = du_of<E>(static_cast<float>(dy[e]), a);
    }
  });
  char* to = z.dz + (row * z.ld_dz + c) * ES;
  if (n == 8) {
    __builtin_memcpy(__builtin_assume_aligned(to, 16), dg, sizeof(dg));
    __builtin_memcpy(to + z.F * ES, du, sizeof(du));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) {
        __builtin_memcpy(to + e * ES, &dg[e], ES);
        __builtin_memcpy(to + (z.F + e) * ES, &du[e], ES);
      }
  }
  if (c + 8 < z.F) return;
  const E zero = static_cast<E>(0.0f);
  for (int64_t e = 2 * z.F; e < z.ld_dz; ++e) __builtin_memcpy(z.dz + (row * z.ld_dz + e) * ES, &zero, ES);
}

// Both gradients in one launch: the first workgroups take dx's tiles and
// ranges, the others dw's (32 x 512 x 1000 fp32: 8.4 us, of which the launch and a
// workgroup's few slabs are nearly all).
template <typename E, Epilogue EPI_DX>
__global__ __launch_bounds__(256) void gated_gen_grads_kernel(GemmArgs dx, GemmArgs dw) {
  __shared__ GenLds<E> lds;
  const int ta = (dx.na + 63) / 64, tb = (dx.nb + 63) / 64, n_dx = ta * tb * dx.ranges;
  int i = blockIdx.x;
  if (i < n_dx) {
    gen_tile<E, kRow, kSum, EPI_DX>(dx, lds, i % ta, i / ta % tb, i / ta / tb);
  } else {
    i -= n_dx;
    gen_tile<E, kRow, kRow, kEpiStore>(dw, lds, i % ta, i / ta, 0);
  }
}

// The same with dx by few_rows, at most 16 MT tokens.
template <typename E, int MT>
__global__ __launch_bounds__(256) void gated_few_grads_kernel(GemmArgs dx, GemmArgs dw) {
  __shared__ GenLds<E> lds;
  static_assert(sizeof(lds.buf) >= 4 * MT * 64 * sizeof(f32x4), "the sums fit");
  const int n_dx = (dx.na + 15) / 16, i = static_cast<int>(blockIdx.x) - n_dx;
  if (i < 0) {
    few_rows<E, MT, kEpiStore>(dx, reinterpret_cast<f32x4*>(&lds.buf[0][0][0]), static_cast<int>(blockIdx.x) * 16);
  } else {
    const int ta = (dw.na + 63) / 64;
    gen_tile<E, kRow, kRow, kEpiStore>(dw, lds, i % ta, i / ta, 0);
  }
}

}  // namespace
}  // namespace fconv

struct fconv_gated_plan_s {
  fconv_gated_desc d;
  int32_t es;
  int64_t ld_kept;  // F in whole eights: kept is fp32 [T, 2, ld_kept]
  size_t kept_bytes;
  bool few;                       // few tokens, by their own kernel
  int32_t few_mt;                 // sixteens of them in a workgroup
  bool few_dx;                    // dx by few_rows, in one launch with dw
  bool pair;                      // both gradients in one launch of tiles
  bool pack_fwd, pack_dx;         // rows of bf16 copied to 16-byte boundaries: x and w; w
  fconv::Split fwd, dx, dw;
  int64_t ld_pack;
  size_t fwd_x, fwd_w, fwd_bytes;
  int64_t ld_dz;
  size_t o_dz, o_x, o_w, o_dx, o_dw, bwd_bytes;
};

namespace fconv {
namespace {

constexpr int32_t kFewTokens = 64;  // that one workgroup can take
// 2 F up to which few_rows takes dx: its time grows with the sum, partial sums cost a launch more (both gradients
// of 32 x 512 x 500 bf16 8.2 instead of 10.9 us, x 1000 10.0 and 10.7, of 64 x 512 x 1000 13.4 and 11.1; fp32, whose
// fragments are twice as large, 11.1 and 13.2, 16.4 and 14.3, 24.6 and 16.1).
int32_t few_dx_sum(int32_t T, int es) {
  static const int32_t most[][3] = {{2048, 2048, 1024}, {2048, 1024, 704}};
  return most[es == 4][T <= 16 ? 0 : T <= 32 ? 1 : 2];
}

// Time (us) of the few-token kernel: w out of memory, at a rate that falls with the
// tokens (16, 32, 64), or the steps of a wave one after another (fitted to D 64 ..
// 8192, F 64 .. 16384).  The steps are bf16's; fp32's take twice as long, so that
// up to 64 tokens of few f and a long k stay in one workgroup where several would be
// quicker (fp32, D 8192, F 512: 32 tokens 59 us, 64 89, 65 and 128 45).
double few_us(int64_t T, int64_t F, int64_t D, int es) {
  const int k = T <= 16 ? 0 : T <= 32 ? 1 : 2;
  static const double rates[][3] = {{5.5e6, 4.6e6, 3.2e6}, {5.0e6, 3.8e6, 2.3e6}}, each[] = {0.0025, 0.0033, 0.005};
  const double memory = 2.0 * es * static_cast<double>(F) * static_cast<double>(D) / rates[es == 4][k];
  const double steps = each[k] * static_cast<double>(D);
  return 3.0 + (memory > steps ? memory : steps);
}
// Tokens of a workgroup of the few-token kernel, in sixteens, and its time.
struct Few {
  int32_t mt;
  double us;
};
// All of them where that is at most 64, or fewer in several workgroups: those take as
// long as a wave's steps for each 256 of them, and past 1024 tiles do better (fitted to T 65 .. 2000, D 200 .. 8192, F
// 64 .. 12288; bf16 rows at odd places take half as long again).
Few few_shape(int64_t T, int64_t F, int64_t D, int es) {
  static const double each[][4] = {{0.0026, 0.0034, 0.0, 0.0051}, {0.0052, 0.0068, 0.0, 0.0143}};
  const bool odd = es == 2 && D % 2;
  Few best = {T <= 16 ? 1 : T <= 32 || odd ? 2 : 4, T <= kFewTokens ? few_us(T, F, D, es) : 1e300};
  for (int32_t mt = 1; mt <= (odd ? 2 : 4); mt *= 2) {
    const int64_t n = round_up(ceil_div(F, 16), 8) * ceil_div(T, 16 * mt);
    const double steps = each[es == 4][mt - 1] * static_cast<double>(D) * (odd ? 1.5 : 1.0);
    const double us = 2.0 + (1.0 + steps) * static_cast<double>(ceil_div(n, 256));
    if (T > 16 * mt && n <= 1024 && us < best.us) best = Few{mt, us};
  }
  return best;
}
// The tiles' time for few tokens: choose() leaves w's way out of memory out (64 x 8192
// x 16384: 132 us).
double few_tiles_us(const Split& s, int64_t F, int64_t D, int es) {
  const double memory = 4.0 + 2.0 * es * static_cast<double>(F) * static_cast<double>(D) / 4.4e6;
  return memory > s.us ? memory : s.us;
}

// What 64 k take in the general kernel (us) of a workgroup alone on its CU and of one
// among four.  Forward both operands' k are contiguous (69 x 2590 x 704: 0.55 alone, 65 x
// 4096 x 4096: 0.45, fp32 1.5), backward a fragment is transposed.  Rows of bf16 that are not aligned take longer
// where the CU is busy (384 x 3754 x 5440: 1.75); fp32 takes 64 k in two slabs (2048 x
// 1024 x 2816: 4.6).
struct Slab {
  double alone, busy;
  double us(int64_t n) const {  // of n workgroups
    return n <= 256 ? alone : n >= 1024 ? busy : alone + (busy - alone) * static_cast<double>(n - 256) / 768.0;
  }
};
Slab slab_us(int64_t D, int es, bool forward) {
  return es == 4 ? Slab{forward ? 1.55 : 2.3, 4.6} : Slab{!forward ? 0.85 : D % 8 ? 0.6 : 0.45, D % 8 ? 1.9 : 1.15};
}
// What r ranges of na x nb values cost beside their slabs: a launch that joins them, and their bytes (dx of 32 x
// 1024 x 2816 in 15 ranges 15.2 us with dw, in 44 17.0).
double ranges_us(int32_t r, int64_t na, int64_t nb) {
  return r == 1 ? 0.0 : 6.0 + 0.06 * r + 8.0 * r * static_cast<double>(na) * static_cast<double>(nb) / 4e6;
}
// The division of a product in general tiles, `beside` other workgroups of
// `beside_slabs` in the same launch.
Split general(int64_t na, int64_t nb, int64_t nk, bool split, const Slab& slab, int64_t beside = 0,
              int64_t beside_slabs = 0) {
  const int64_t tiles = ceil_div(na, 64) * ceil_div(nb, 64), slabs = ceil_div(nk, 64);
  Split best = {64, 1, 1e300};
  for (int32_t r = 1; r <= (split ? 128 : 1) && (r == 1 || (slabs / r >= 2 && r * na * nb * 4 <= kGBytes)); ++r) {
    const int64_t n = tiles * r + beside, own = ceil_div(slabs, r), most = own > beside_slabs ? own : beside_slabs;
    double us = static_cast<double>(most) * slab.us(n) + 2.5;
    // More of them than the device holds: their work.
    const double work = (static_cast<double>(tiles * slabs + beside * beside_slabs) * slab.busy + 2.5 * static_cast<double>(n)) / 1024.0;
    us = (work > us ? work : us) + ranges_us(r, na, nb);
    if (us < best.us) best = Split{64, r, us};
  }
  return best;
}
// In general tiles or, where they can be, in those of 128 or 256.
Split divide(int64_t na, int64_t nb, int64_t nk, bool tiled, bool split, const Slab& slab) {
  const Split g = general(na, nb, nk, split, slab);
  if (!tiled) return g;
  const Split t = choose(na, nb, nk, true, split, 1e9, 1e9);
  return t.edge != 64 && t.us < g.us ? t : g;
}
// dx's ranges where it shares a launch of tiles of one edge with dw (of one range),
// and the time of both: dx's tiles first, dw's as places become free.
Split pair(int64_t T, int64_t D, int64_t F2) {
  struct Kind {
    int32_t edge;
    int64_t at_once;
    double slab;
  };
  Split best = {64, 1, 1e300};
  for (const Kind& k : {Kind{256, 256, 1.0}, Kind{128, 512, 0.7}}) {
    const int64_t tx = ceil_div(D, k.edge) * ceil_div(T, k.edge), tw = ceil_div(D, k.edge) * ceil_div(F2, k.edge);
    const int64_t sx = ceil_div(F2, 64);
    const double each_w = static_cast<double>(ceil_div(T, 64)) * k.slab + 5.0;
    for (int32_t r = 1; r <= 128 && (r == 1 || (sx / r >= 2 && r * D * T * 4 <= kGBytes)); ++r) {
      const int64_t n = tx * r, late = n % k.at_once;  // places that dx leaves a turn later than the others
      const double each_x = static_cast<double>(ceil_div(sx, r)) * k.slab + 5.0;
      const double first = static_cast<double>(n / k.at_once) * each_x, second = first + each_x;
      // The first time by which all of dw's tiles fit, in turns after either.
      double us = 1e300;
      for (int i = 0; i < 2; ++i) {
        const double from = i ? second : first;
        for (int64_t turns = 0; turns <= ceil_div(tw, k.at_once) + 1; ++turns) {
          const double end = from + static_cast<double>(turns) * each_w;
          if (end < (late ? second : first) || end >= us) continue;
          const int64_t a = static_cast<int64_t>((end - first) / each_w + 1e-6), b = static_cast<int64_t>((end - second) / each_w + 1e-6);
          if ((k.at_once - late) * a + late * (b > 0 ? b : 0) >= tw) us = end;
        }
      }
      // A range's sums go out and come back (4 TB/s), and a launch joins them.
      if (r > 1) us += 6.0 + 8.0 * r * static_cast<double>(D) * static_cast<double>(T) / 4e6;
      if (us < best.us) best = Split{k.edge, r, us};
    }
  }
  return best;
}
// Time (us) of copying a matrix to 16-byte boundaries (10880 x 3754: 26).
double copy_us(int64_t rows, int64_t cols) { return 4.0 + 4.0 * static_cast<double>(rows) * static_cast<double>(cols) / 6e6; }

template <typename E, bool ODD>
hipError_t launch_few_of(const GatedFew& f, int mt, hipStream_t s) {
  if (ODD && mt > 2) mt = 2;
  const dim3 grid(static_cast<unsigned>(round_up(ceil_div(f.F, 16), 8) * ceil_div(f.T, 16 * mt)));
  // Of a few tokens the waves' loads are nearly all of w, and more of them read a large one quicker
  // (one token, 4096 x 12288: eight 37.2 us, four 38.8; 8192 x 16384: 107 and 124; 16 tokens: 43.4 and 41.9).
  if (f.T <= 8 && static_cast<int64_t>(f.F) * f.D * 2 * static_cast<int64_t>(sizeof(E)) >= 128 << 20) {
    hipLaunchKernelGGL((gated_few_kernel<E, ODD, 1, 8>), grid, dim3(512), 0, s, f);
  } else if (mt == 1) {
    hipLaunchKernelGGL((gated_few_kernel<E, ODD, 1, 4>), grid, dim3(256), 0, s, f);
  } else if (mt == 2) {
    hipLaunchKernelGGL((gated_few_kernel<E, ODD, 2, 4>), grid, dim3(256), 0, s, f);
  } else {
    if constexpr (!ODD) hipLaunchKernelGGL((gated_few_kernel<E, ODD, 4, 4>), grid, dim3(256), 0, s, f);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t run_forward(const fconv_gated_plan_s* p, const fconv_gated_args* args, hipStream_t s) {
  const fconv_gated_desc& d = p->d;
  char* ws = static_cast<char*>(args->workspace);
  Operand w = {static_cast<const char*>(args->w), args->ldw, d.F};
  Operand x = {static_cast<const char*>(args->x), args->ldx, 0};
  const bool fits = fits_tiles(w.p, w.ld) && fits_tiles(x.p, x.ld);
  if (p->few || (d.T <= kFewTokens && !fits && p->fwd.edge != 64)) {
    const GatedFew f = {w.p, w.ld, x.p, x.ld, static_cast<char*>(args->y), args->ldy, static_cast<float*>(args->kept),
                        p->ld_kept, d.T, d.D, d.F, d.activation};
    if constexpr (sizeof(E) == 2) {
      if (odd_rows(w) || odd_rows(x)) return launch_few_of<E, true>(f, p->few_mt, s);
    }
    return launch_few_of<E, false>(f, p->few_mt, s);
  }
  int edge = p->fwd.edge;
  hipError_t e;
  if (p->pack_fwd) {
    if ((e = launch_pack(x.p, x.ld, d.T, d.D, ws + p->fwd_x, p->ld_pack, s)) != hipSuccess) return e;
    if ((e = launch_pack(w.p, w.ld, 2ll * d.F, d.D, ws + p->fwd_w, p->ld_pack, s)) != hipSuccess) return e;
    x = {ws + p->fwd_x, p->ld_pack, 0};
    w = {ws + p->fwd_w, p->ld_pack, d.F};
  } else if (!fits) {
    // Rows from anywhere: 2048 x 1024 x 2816 57 us instead of the tiles' 27, 8192 x 4096 x 12288 4.1 ms instead of 1.2.
    edge = 64;
  }
  GemmArgs g = {};
  g.a = w;
  g.b = x;
  g.na = d.F;
  g.nb = d.T;
  g.nk = d.D;
  g.ranges = 1;
  g.out = static_cast<char*>(args->y);
  g.ld_out = args->ldy;
  g.act = d.activation;
  g.kept = static_cast<float*>(args->kept);
  g.ld_kept = p->ld_kept;
  return launch_gemm<E, kSum, kSum, kEpiGated>(g, edge, s);
}

// Both gradients in one launch of tiles of an edge.
template <Epilogue EPI_X, Epilogue EPI_Y>
hipError_t launch_pair(const GemmArgs& x, const GemmArgs& y, int edge, hipStream_t s) {
  auto blocks = [&](const GemmArgs& g) { return tile_blocks(ceil_div(g.na, edge) * ceil_div(g.nb, edge) * g.ranges, edge); };
  const unsigned bx = blocks(x);
  const dim3 grid(bx + blocks(y));
  if (edge == 256)
    hipLaunchKernelGGL((gemm_tile_pair_kernel<EPI_X, EPI_Y, 128, 8>), grid, dim3(512), 0, s, x, y, bx);
  else
    hipLaunchKernelGGL((gemm_tile_pair_kernel<EPI_X, EPI_Y, 64, 4>), grid, dim3(256), 0, s, x, y, bx);
  return hipGetLastError();
}

template <typename E>
hipError_t run_backward(const fconv_gated_plan_s* p, const fconv_gated_args* args, hipStream_t s) {
  const fconv_gated_desc& d = p->d;
  char* ws = static_cast<char*>(args->workspace);
  char* dw = static_cast<char*>(args->dw);
  char* dx = static_cast<char*>(args->dx);
  const int32_t F2 = 2 * d.F;
  hipError_t e;
  if (d.T == 0) {
    if (!dw) return hipSuccess;
    hipLaunchKernelGGL(gemm_zero_kernel<E>, dim3(F2 < 4096 ? F2 : 4096), dim3(256), 0, s, dw, args->lddw,
                       static_cast<int64_t>(F2), d.D);
    return hipGetLastError();
  }
  const GatedDz z = {static_cast<const float*>(args->kept), p->ld_kept, static_cast<const char*>(args->dy), args->lddy,
                     ws + p->o_dz, p->ld_dz, d.T, d.F, d.activation};
  hipLaunchKernelGGL(gated_dz_kernel<E>, dim3(static_cast<unsigned>(ceil_div(d.T * (p->ld_kept / 8), 256))), dim3(256), 0,
                     s, z);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  Operand w = {static_cast<const char*>(args->w), args->ldw, d.D};
  Operand x = {static_cast<const char*>(args->x), args->ldx, d.D};
  const int dx_edge = p->pack_dx || fits_tiles(w.p, w.ld) ? p->dx.edge : 64;
  const bool dx_whole = p->dx.ranges == 1, dw_whole = p->dw.ranges == 1;
  if (dx && p->pack_dx) {
    if ((e = launch_pack(w.p, w.ld, F2, d.D, ws + p->o_w, p->ld_pack, s)) != hipSuccess) return e;
    w = {ws + p->o_w, p->ld_pack, p->ld_pack};
  }
  // A last row that is no whole pieces of 16 bytes would be read past its end.
  if (dw && p->dw.edge != 64 && (d.D % 8 != 0 || !fits_tiles(x.p, x.ld))) {
    if ((e = launch_pack(x.p, x.ld, d.T, d.D, ws + p->o_x, p->ld_pack, s)) != hipSuccess) return e;
    x = {ws + p->o_x, p->ld_pack, p->ld_pack};
  }
  GemmArgs gx = {};
  gx.a = w;
  gx.b = Operand{ws + p->o_dz, p->ld_dz, 0};
  gx.na = d.D;
  gx.nb = d.T;
  gx.nk = F2;
  gx.ranges = p->dx.ranges;
  gx.out = dx_whole ? dx : ws + p->o_dx;
  gx.ld_out = dx_whole ? args->lddx : round_up(d.D, 4);
  gx.part_stride = gx.ld_out * d.T;
  GemmArgs gw = {};
  gw.a = x;
  gw.b = Operand{ws + p->o_dz, p->ld_dz, round_up(F2, 8)};
  gw.na = d.D;
  gw.nb = F2;
  gw.nk = d.T;
  gw.ranges = p->dw.ranges;
  gw.out = dw_whole ? dw : ws + p->o_dw;
  gw.ld_out = dw_whole ? args->lddw : round_up(d.D, 4);
  gw.part_stride = gw.ld_out * F2;
  if (dx && p->few_dx) {
    const dim3 grid(static_cast<unsigned>(ceil_div(d.D, 16) + (dw ? ceil_div(d.D, 64) * ceil_div(F2, 64) : 0)));
    if (d.T <= 16)
      hipLaunchKernelGGL((gated_few_grads_kernel<E, 1>), grid, dim3(256), 0, s, gx, gw);
    else if (d.T <= 32)
      hipLaunchKernelGGL((gated_few_grads_kernel<E, 2>), grid, dim3(256), 0, s, gx, gw);
    else
      hipLaunchKernelGGL((gated_few_grads_kernel<E, 4>), grid, dim3(256), 0, s, gx, gw);
    return hipGetLastError();
  }
  // Past the caches where dw is larger than the L2s together and written in whole lines.
  const bool past = p->es == 2 && static_cast<int64_t>(F2) * d.D * 2 > (32 << 20) && d.D % 64 == 0 &&
                    args->lddw % 64 == 0 && (reinterpret_cast<uintptr_t>(dw) & 127) == 0;
  if (dx && dw && dx_edge == 64 && p->dw.edge == 64 && dw_whole) {
    const dim3 grid(static_cast<unsigned>(ceil_div(d.D, 64) * (ceil_div(d.T, 64) * gx.ranges + ceil_div(F2, 64))));
    if (dx_whole)
      hipLaunchKernelGGL((gated_gen_grads_kernel<E, kEpiStore>), grid, dim3(256), 0, s, gx, gw);
    else
      hipLaunchKernelGGL((gated_gen_grads_kernel<E, kEpiPart>), grid, dim3(256), 0, s, gx, gw);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else if (dx && dw && p->pair && dx_edge == p->dw.edge) {
    if constexpr (sizeof(E) == 2)
      e = dx_whole ? past ? launch_pair<kEpiStore, kEpiStoreStream>(gx, gw, dx_edge, s)
                          : launch_pair<kEpiStore, kEpiStore>(gx, gw, dx_edge, s)
          : past ? launch_pair<kEpiPart, kEpiStoreStream>(gx, gw, dx_edge, s)
                 : launch_pair<kEpiPart, kEpiStore>(gx, gw, dx_edge, s);
    if (e != hipSuccess) return e;
  } else {
    if (dx) {
      e = dx_whole ? launch_gemm<E, kRow, kSum, kEpiStore>(gx, dx_edge, s)
                   : launch_gemm<E, kRow, kSum, kEpiPart>(gx, dx_edge, s);
      if (e != hipSuccess) return e;
    }
    if (dw) {
      e = !dw_whole ? launch_gemm<E, kRow, kRow, kEpiPart>(gw, p->dw.edge, s)
          : past    ? launch_gemm<E, kRow, kRow, kEpiStoreStream>(gw, p->dw.edge, s)
                    : launch_gemm<E, kRow, kRow, kEpiStore>(gw, p->dw.edge, s);
      if (e != hipSuccess) return e;
    }
  }
  if (dx && !dx_whole) {
    e = launch_sum<E>(reinterpret_cast<const float*>(ws + p->o_dx), gx.ranges, gx.part_stride, gx.ld_out, d.T, nullptr,
                      nullptr, nullptr, 0, d.D, dx, args->lddx, s);
    if (e != hipSuccess) return e;
  }
  if (dw && !dw_whole)
    return launch_sum<E>(reinterpret_cast<const float*>(ws + p->o_dw), gw.ranges, gw.part_stride, gw.ld_out, F2, nullptr,
                         nullptr, nullptr, 0, d.D, dw, args->lddw, s);
  return hipSuccess;
}

const Split* split_of(const fconv_gated_plan_s* p, int32_t product) {
  switch (product) {
    case FCONV_GATED_FORWARD: return &p->fwd;
    case FCONV_GATED_DX: return &p->dx;
    case FCONV_GATED_DW: return &p->dw;
    default: return nullptr;
  }
}

}  // namespace
}  // namespace fconv

extern "C" {

fconv_status fconv_gated_plan_create(const fconv_gated_desc* desc, fconv_gated_plan* out) {
  using namespace fconv;
  if (!desc || !out) return FCONV_ERR_INVALID_ARG;
  *out = nullptr;
  const fconv_gated_desc& d = *desc;
  if (d.dtype != FCONV_BF16 && d.dtype != FCONV_FP32) return FCONV_ERR_UNSUPPORTED;
  if (d.activation < FCONV_ACT_SILU || d.activation > FCONV_ACT_RELU || d.flags) return FCONV_ERR_UNSUPPORTED;
  if (d.T < 0 || d.D < 1 || d.F < 1) return FCONV_ERR_INVALID_ARG;
  if (d.D > kMaxD || d.F > kMaxD) return FCONV_ERR_UNSUPPORTED;
  const int64_t T = d.T, D = d.D, F2 = 2ll * d.F, tb = ceil_div(T, 64);
  if (tb > kMaxGridY || ceil_div(F2, 64) * tb > kMaxTiles || ceil_div(D, 64) * tb > kMaxTiles || T * D > kMaxSum ||
      T * F2 > kMaxSum || F2 * D > kMaxSum)
    return FCONV_ERR_UNSUPPORTED;
  fconv_gated_plan_s* p = new (std::nothrow) fconv_gated_plan_s();
  if (!p) return FCONV_ERR_INVALID_ARG;
  p->d = d;
  p->es = d.dtype == FCONV_BF16 ? 2 : 4;
  p->ld_kept = round_up(d.F, 8);
  p->kept_bytes = static_cast<size_t>(T) * 2 * p->ld_kept * 4;
  const bool bf16 = d.dtype == FCONV_BF16, tiled = bf16 && D % 8 == 0;
  p->ld_pack = round_up(D, 8);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  if (T > 0) {
    const Slab fwd = slab_us(D, p->es, true), bwd = slab_us(D, p->es, false);
    p->fwd = divide(F2, T, D, tiled, false, fwd);
    if (bf16 && !tiled && T > kFewTokens) {
      const Split packed = divide(F2, T, D, true, false, fwd);
      p->pack_fwd = packed.edge != 64 && packed.us + copy_us(F2, D) + copy_us(T, D) < p->fwd.us;
      if (p->pack_fwd) p->fwd = packed;
    }
    const Few few = few_shape(T, d.F, D, p->es);
    p->few = few.us < (T <= kFewTokens ? few_tiles_us(p->fwd, d.F, D, p->es) : p->fwd.us);
    p->few_mt = few.mt;
    if (p->few) p->pack_fwd = false;
    p->fwd_x = take(p->pack_fwd ? static_cast<size_t>(T) * p->ld_pack * 2 : 0);
    p->fwd_w = take(p->pack_fwd ? static_cast<size_t>(F2) * p->ld_pack * 2 : 0);
    p->fwd_bytes = at;
    at = 0;
    p->ld_dz = round_up(F2, 64);
    p->dx = divide(D, T, F2, tiled, true, bwd);
    double dx_us = p->dx.us;
    if (bf16 && !tiled) {
      const Split packed = divide(D, T, F2, true, true, bwd);
      p->pack_dx = packed.edge != 64 && packed.us + copy_us(F2, D) < p->dx.us;
      if (p->pack_dx) {
        p->dx = packed;
        dx_us = packed.us + copy_us(F2, D);
      }
    }
    p->dw = divide(D, F2, T, bf16, true, bwd);
    const double dw_us = p->dw.us + (bf16 && !tiled && p->dw.edge != 64 ? copy_us(T, D) : 0.0);
    // Both gradients in general tiles take one launch, in which they overlap.
    const Split both = general(D, T, F2, true, bwd, ceil_div(D, 64) * ceil_div(F2, 64), ceil_div(T, 64));
    // Tiles of both products in one launch have to win from two launches by a margin: where each product fills the
    // device by itself, one launch gains nothing (8192 x 4096 x 8192: 1560 us, 771 and 769 apart).
    double us = 0.95 * (dx_us + dw_us + 4.0);
    if (both.us < dx_us + dw_us + 4.0) {
      us = both.us;
      p->pack_dx = false;
      p->dx = both;
      p->dw = Split{64, 1, both.us};
    }
    if (bf16) {
      const Split tiles = pair(T, D, F2);
      if (tiles.us + (tiled ? 0.0 : copy_us(F2, D) + copy_us(T, D)) < us) {
        p->pair = true;
        p->pack_dx = !tiled;
        p->dx = tiles;
        p->dw = Split{tiles.edge, 1, tiles.us};
      }
    }
    p->few_dx = T <= kFewTokens && F2 <= few_dx_sum(d.T, p->es) && !p->pair && p->dw.edge == 64 && p->dw.ranges == 1;
    if (p->few_dx) {
      p->pack_dx = false;
      p->dx.ranges = 1;
    }
    const size_t ld4 = static_cast<size_t>(round_up(D, 4)) * 4;
    p->o_dz = take(static_cast<size_t>(T) * p->ld_dz * p->es);
    p->o_x = take(bf16 && p->dw.edge != 64 ? static_cast<size_t>(T) * p->ld_pack * 2 : 0);
    p->o_w = take(p->pack_dx ? static_cast<size_t>(F2) * p->ld_pack * 2 : 0);
    p->o_dx = take(p->dx.ranges > 1 ? static_cast<size_t>(p->dx.ranges) * T * ld4 : 0);
    p->o_dw = take(p->dw.ranges > 1 ? static_cast<size_t>(p->dw.ranges) * F2 * ld4 : 0);
    p->bwd_bytes = at;
  }
  *out = p;
  return FCONV_OK;
}

fconv_status fconv_gated_plan_kept_size(fconv_gated_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->kept_bytes;
  return FCONV_OK;
}

fconv_status fconv_gated_plan_forward_workspace_size(fconv_gated_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->fwd_bytes;
  return FCONV_OK;
}

fconv_status fconv_gated_plan_backward_workspace_size(fconv_gated_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->bwd_bytes;
  return FCONV_OK;
}

fconv_status fconv_gated_plan_forward(fconv_gated_plan p, void* stream, const fconv_gated_args* a) {
  using namespace fconv;
  if (!p || !a) return FCONV_ERR_INVALID_ARG;
  const fconv_gated_desc& d = p->d;
  if (d.T == 0) return FCONV_OK;
  if (!a->x || !a->w || !a->y) return FCONV_ERR_INVALID_ARG;
  if (bad_ld(a->ldx, d.D) || bad_ld(a->ldw, d.D) || bad_ld(a->ldy, d.F)) return FCONV_ERR_INVALID_ARG;
  if (p->fwd_bytes && (!a->workspace || a->workspace_bytes < p->fwd_bytes)) return FCONV_ERR_WORKSPACE;
  if (!aligned(a->x, p->es) || !aligned(a->w, p->es) || !aligned(a->y, p->es) || !aligned(a->kept, 16) ||
      !aligned(a->workspace, 16))
    return FCONV_ERR_MISALIGNED;
  const Range in[] = {{a->x, span(d.T, d.D, a->ldx, p->es)}, {a->w, span(2ll * d.F, d.D, a->ldw, p->es)}};
  const Range wr[] = {{a->y, span(d.T, d.F, a->ldy, p->es)}, {a->kept, p->kept_bytes}, {a->workspace, p->fwd_bytes}};
  if (clash(wr, 3, in, 2)) return FCONV_ERR_INVALID_ARG;
  const hipError_t e = d.dtype == FCONV_BF16 ? run_forward<__bf16>(p, a, as_stream(stream))
                                             : run_forward<float>(p, a, as_stream(stream));
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_gated_plan_backward(fconv_gated_plan p, void* stream, const fconv_gated_args* a) {
  using namespace fconv;
  if (!p || !a) return FCONV_ERR_INVALID_ARG;
  const fconv_gated_desc& d = p->d;
  if (!a->dx && !a->dw) return FCONV_ERR_INVALID_ARG;
  if ((a->dx && bad_ld(a->lddx, d.D)) || (a->dw && bad_ld(a->lddw, d.D))) return FCONV_ERR_INVALID_ARG;
  if (!aligned(a->dx, p->es) || !aligned(a->dw, p->es)) return FCONV_ERR_MISALIGNED;
  if (d.T > 0) {
    if (!a->x || !a->w || !a->kept || !a->dy) return FCONV_ERR_INVALID_ARG;
    if (bad_ld(a->ldx, d.D) || bad_ld(a->ldw, d.D) || bad_ld(a->lddy, d.F)) return FCONV_ERR_INVALID_ARG;
    if (!a->workspace || a->workspace_bytes < p->bwd_bytes) return FCONV_ERR_WORKSPACE;
    if (!aligned(a->x, p->es) || !aligned(a->w, p->es) || !aligned(a->kept, 16) || !aligned(a->dy, p->es) ||
        !aligned(a->workspace, 16))
      return FCONV_ERR_MISALIGNED;
    const Range in[] = {{a->x, span(d.T, d.D, a->ldx, p->es)}, {a->w, span(2ll * d.F, d.D, a->ldw, p->es)},
                        {a->kept, p->kept_bytes}, {a->dy, span(d.T, d.F, a->lddy, p->es)}};
    const Range wr[] = {{a->dx, span(d.T, d.D, a->lddx, p->es)}, {a->dw, span(2ll * d.F, d.D, a->lddw, p->es)},
                        {a->workspace, p->bwd_bytes}};
    if (clash(wr, 3, in, 4)) return FCONV_ERR_INVALID_ARG;
  }
  const hipError_t e = d.dtype == FCONV_BF16 ? run_backward<__bf16>(p, a, as_stream(stream))
                                             : run_backward<float>(p, a, as_stream(stream));
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

const char* fconv_gated_plan_kernel_name(fconv_gated_plan p, int32_t product) {
  using namespace fconv;
  if (!p || p->d.T == 0) return nullptr;
  const Split* split = split_of(p, product);
  if (!split) return nullptr;
  if (product == FCONV_GATED_FORWARD && p->few) return "gated_few";
  if (product == FCONV_GATED_DX && p->few_dx) return "gated_few_grads";
  const bool packed = product == FCONV_GATED_FORWARD ? p->pack_fwd
                      : product == FCONV_GATED_DX    ? p->pack_dx
                                                     : split->edge != 64 && p->d.D % 8 != 0;
  if (split->edge == 64) return packed ? "gemm_gen_64_packed" : "gemm_gen_64";
  if (split->edge == 128) return packed ? "gemm_tile_128_packed" : "gemm_tile_128";
  return packed ? "gemm_tile_256_packed" : "gemm_tile_256";
}

fconv_status fconv_gated_plan_ranges(fconv_gated_plan p, int32_t product, int32_t* ranges) {
  using namespace fconv;
  if (!p || !ranges) return FCONV_ERR_INVALID_ARG;
  const Split* split = split_of(p, product);
  if (!split) return FCONV_ERR_INVALID_ARG;
  *ranges = p->d.T == 0 ? 0 : split->ranges;
  return FCONV_OK;
}

fconv_status fconv_gated_plan_destroy(fconv_gated_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
