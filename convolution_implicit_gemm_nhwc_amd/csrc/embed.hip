// Embedding lookup on gfx950 (CDNA4), its gradient, and their C ABI
// (include/fconv_embed.h).
//
//   y[t] = scale w[token[t]]        dw[v] = scale sum over token[t] = v of dy[t]
//
// Both are bound by memory: rows are read once and written once, 16 bytes of a
// thread at a time, at any alignment.
//
// The gradient sums each row's tokens in the order of their places, so tokens
// are sorted first, as 64-bit keys of token and place (all different, so the
// order is unique).  Up to kSmall tokens every workgroup sorts them all itself,
// in LDS, and the gradient is one launch.  Above:
//   rank    chunks of up to kChunk tokens, sorted by counting for each key the
//           smaller ones of its chunk: n^2 / 2 operations a token and no passes
//   merge   sixteen sorted runs at a time: a key's place is the sum of its ranks
//           in them, found by binary searches
//   reduce  pieces of `piece` sorted keys: their rows of dy are summed; a token
//           whose keys all lie in the piece is done, the others' sums of the piece
//           go out.  Other workgroups of the launch write the rows of zeros.
//   join    adds the pieces' sums of a token, in order
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <cmath>
#include <new>
#include <type_traits>

#include "dense.h"
#include "fconv_embed.h"

namespace fconv {
namespace {

constexpr int kSmall = 256;   // tokens that a workgroup sorts by itself
constexpr int kChunk = 4096;  // tokens of a chunk that is ranked, at most
constexpr int kWays = 16;     // runs merged at a time
constexpr uint32_t kNoToken = 0xffffffffu;  // sorts behind every token

__device__ inline uint64_t key_of(uint32_t token, uint32_t place) { return static_cast<uint64_t>(token) << 32 | place; }
__device__ inline uint32_t token_of(uint64_t key) { return static_cast<uint32_t>(key >> 32); }
__device__ inline uint32_t usable(int64_t token, int64_t ignore, int32_t V) {
  return token != ignore && token >= 0 && token < V ? static_cast<uint32_t>(token) : kNoToken;
}

// 16 bytes of elements of type E.
template <typename E>
struct Vec {
  static constexpr int N = 16 / sizeof(E);
  E v[N];
  // n of them at p, zeros past those.
  __device__ void load(const char* p, int n) {
    if (n >= N) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[e] = static_cast<E>(0.0f);
        if (e < n) __builtin_memcpy(&v[e], p + e * sizeof(E), sizeof(E));
      }
    }
  }
  __device__ void store(char* p, int n) const {
    if (n >= N) {
      __builtin_memcpy(p, v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < n) __builtin_memcpy(p + e * sizeof(E), &v[e], sizeof(E));
    }
  }
};

// --------------------------------------------------------------------- lookup

struct LookupArgs {
  const int64_t* token;
  int64_t ignore;
  const char* w;
  int64_t ldw;
  char* y;
  int64_t ldy;
  int32_t T, D, V;
  float scale;
};

// Four pieces of 16 bytes of a thread in flight.  Pieces are counted in 32 bits:
// T D is at most 2^33 elements.
template <typename E>
__global__ __launch_bounds__(256) void embed_lookup_kernel(LookupArgs a) {
  constexpr int N = Vec<E>::N, U = 4;
  constexpr int64_t ES = sizeof(E);
  const uint32_t per_row = static_cast<uint32_t>((a.D + N - 1) / N), total = per_row * static_cast<uint32_t>(a.T);
  const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
  Vec<E> v[U];
  int64_t tok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + 256u * u;
    tok[u] = a.token[i < total ? i / per_row : 0];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + 256u * u;
    if (i >= total) break;
    const int c = static_cast<int>(i % per_row) * N;
    if (usable(tok[u], a.ignore, a.V) != kNoToken) v[u].load(a.w + (tok[u] * a.ldw + c) * ES, a.D - c);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + 256u * u;
    if (i >= total) break;
    const int64_t row = i / per_row;
    const int c = static_cast<int>(i - static_cast<uint32_t>(row) * per_row) * N;
    if (usable(tok[u], a.ignore, a.V) == kNoToken) {
      const float f = tok[u] == a.ignore ? 0.0f : __builtin_nanf("");
#pragma unroll
      for (int e = 0; e < N; ++e) v[u].v[e] = static_cast<E>(f);
    } else if (a.scale != 1.0f) {
#pragma unroll
      for (int e = 0; e < N; ++e) v[u].v[e] = static_cast<E>(a.scale * static_cast<float>(v[u].v[e]));
    }
    v[u].store(a.y + (row * a.ldy + c) * ES, a.D - c);
  }
}

// -------------------------------------------------------------------- sorting

// Keys of chunk blockIdx.y, sorted: a workgroup ranks 64 of them, each wave
// against every fourth block of 64.  Of equal tokens the earlier one is smaller:
// in a block before the own one "not larger" counts, in one behind it "smaller".
__global__ __launch_bounds__(256) void embed_rank_kernel(const int64_t* token, int64_t ignore, int32_t T, int32_t V,
                                                         int chunk, uint64_t* keys) {
  __shared__ __attribute__((aligned(16))) uint32_t all[kChunk];
  __shared__ int ranks[4][64];
  const int base = blockIdx.y * chunk, n = min(chunk, T - base), n64 = (n + 63) / 64 * 64;
  const int own = blockIdx.x * 64;
  if (own >= n) return;
  for (int i = threadIdx.x; i < n64; i += 256) all[i] = i < n ? usable(token[base + i], ignore, V) : kNoToken;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t mine = all[own + lane];
  int rank = 0;
  for (int b = wave * 64; b < n64; b += 256) {
    const uint4* p = reinterpret_cast<const uint4*>(all + b);
    if (b < own) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 k = p[i];
        rank += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
      }
    } else if (b > own) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 k = p[i];
        rank += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
      }
    } else {
      for (int i = 0; i < 64; ++i) rank += all[b + i] < mine || (all[b + i] == mine && i < lane);
    }
  }
  ranks[wave][lane] = rank;
  __syncthreads();
  // What fills the last block up ranks behind the chunk's own keys.
  if (wave == 0 && own + lane < n)
    keys[base + ranks[0][lane] + ranks[1][lane] + ranks[2][lane] + ranks[3][lane]] =
        key_of(mine, static_cast<uint32_t>(base + own + lane));
}

// Groups of kWays sorted runs of `run` keys become one each.  Four lanes share a
// key, each with four of the runs, whose searches go on side by side.
__global__ __launch_bounds__(256) void embed_merge_kernel(const uint64_t* in, uint64_t* out, int32_t T, int32_t run) {
  constexpr int M = kWays / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x / 4;
  const int part = threadIdx.x & 3;
  const bool live = i < T;
  const int64_t at = live ? i : T - 1;
  const uint64_t key = in[at];
  const int64_t own = at / run, group = own / kWays * kWays;
  int len[M], lo[M];
  int64_t base[M];
#pragma unroll
  for (int k = 0; k < M; ++k) {
    const int64_t r = group + part * M + k;
    base[k] = r * run;
    const int64_t left = T - base[k];
    len[k] = left <= 0 ? 0 : left < run ? static_cast<int>(left) : run;
    lo[k] = 0;
  }
  // The number of keys of each run that are below this one.
  for (int step = 1 << (31 - __builtin_clz(run)); step > 0; step >>= 1) {
    uint64_t x[M];
#pragma unroll
    for (int k = 0; k < M; ++k) x[k] = lo[k] + step <= len[k] ? in[base[k] + lo[k] + step - 1] : ~0ull;
#pragma unroll
    for (int k = 0; k < M; ++k) lo[k] += x[k] < key ? step : 0;
  }
  int rank = 0;
#pragma unroll
  for (int k = 0; k < M; ++k) rank += lo[k];
  rank += __shfl_xor(rank, 1);
  rank += __shfl_xor(rank, 2);
  if (live && part == 0) out[group * run + rank] = key;
}

// ------------------------------------------------------------------- gradient

struct GradArgs {
  const uint64_t* keys;   // sorted
  const int64_t* token;   // kSmall tokens at most: unsorted
  int64_t ignore;
  const char* dy;
  int64_t lddy;
  char* dw;
  int64_t lddw;
  float* part;            // [piece][2][ld_part]: of a token that began before it, and of its last one
  int64_t ld_part;
  int32_t T, D, V;
  int32_t piece, pieces;  // sorted keys of a piece
  int32_t team;           // threads that share a piece's columns, a power of two
  int32_t col_blocks;     // workgroups that share a piece's columns
  int32_t sum_groups;     // workgroups of the sums, in front of those of the zeros
  int32_t zero_rows;      // rows of dw of a workgroup of the zeros
  float scale;
  bool add;
};

// First index of the sorted keys at or above `key`: 64 probes of a wave at a time.
__device__ inline int lower_bound(const uint64_t* keys, int n, uint64_t key) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = n;  // the answer is one of lo .. hi
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + step * (lane + 1) - 1;  // the last of this lane's part
    lo += step * __popcll(__ballot(at < hi && keys[at] < key));  // the first parts are below
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// scale sum, or that added to what is there.
template <typename E>
__device__ inline void put_row(const GradArgs& g, uint32_t v, int c, const float (&sum)[Vec<E>::N]) {
  constexpr int N = Vec<E>::N;
  const int n = g.D - c;
  char* p = g.dw + (static_cast<int64_t>(v) * g.lddw + c) * static_cast<int64_t>(sizeof(E));
  Vec<E> x;
  if (g.add) {
    x.load(p, n);
#pragma unroll
    for (int e = 0; e < N; ++e) x.v[e] = static_cast<E>(__builtin_fmaf(g.scale, sum[e], static_cast<float>(x.v[e])));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) x.v[e] = static_cast<E>(g.scale * sum[e]);
  }
  x.store(p, n);
}

// The keys of all (at most kSmall) tokens, sorted, in LDS.
__device__ inline void sort_small(const GradArgs& g, uint64_t* sorted) {
  __shared__ uint32_t all[kSmall];
  const int i = threadIdx.x;
  const uint32_t mine = i < g.T ? usable(g.token[i], g.ignore, g.V) : kNoToken;
  all[i] = mine;
  __syncthreads();
  int rank = 0;
  for (int j = 0; j < g.T; ++j) rank += all[j] < mine || (all[j] == mine && j < i);
  if (i < g.T) sorted[rank] = key_of(mine, static_cast<uint32_t>(i));
  __syncthreads();
}

// Sums of dy's rows.  A team's threads each hold 16 bytes of columns; eight rows
// are in flight.  Without SMALL, a piece's first token may have begun before it and
// its last one may go on behind it: their sums go to `part`.  With SMALL a token
// belongs to the piece in which it begins, which then reads on.
template <typename E, bool SMALL>
__device__ inline void sum_rows(const GradArgs& g, const uint64_t* keys) {
  constexpr int N = Vec<E>::N, U = 8;
  constexpr int64_t ES = sizeof(E);
  const int teams = 256 / g.team, block = blockIdx.x % g.col_blocks;
  const int piece = blockIdx.x / g.col_blocks * teams + threadIdx.x / g.team;
  const int c = (block * g.team + threadIdx.x % g.team) * N;
  if (piece >= g.pieces || c >= g.D) return;
  int at = piece * g.piece;
  const int end = min(at + g.piece, g.T);
  // Whether the token at `at` began before this piece; with SMALL it is another piece's.
  bool began = at > 0 && token_of(keys[at - 1]) == token_of(keys[at]);
  if (SMALL && began) {
    while (at < end && token_of(keys[at]) == token_of(keys[at - 1])) ++at;
    began = false;
  }
  const int last = SMALL ? g.T : end;
  float sum[N] = {};
  uint32_t now = at < end ? token_of(keys[at]) : kNoToken;
  auto flush = [&](bool goes_on) __attribute__((always_inline)) {
    if (!SMALL && (began || goes_on)) {
      float* p = g.part + (2ll * piece + (began ? 0 : 1)) * g.ld_part + c;
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 x = {sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
        __builtin_memcpy(p + e, &x, 16);
      }
    } else {
      put_row<E>(g, now, c, sum);
    }
  };
  bool done = now == kNoToken;  // tokens without a gradient come last
  while (!done && at < last) {
    Vec<E> x[U];
    uint32_t tok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t key = keys[min(at + u, last - 1)];
      tok[u] = at + u < last ? token_of(key) : kNoToken;
      // Rows past the end, and of tokens without a gradient, are read for nothing.
      x[u].load(g.dy + (static_cast<int64_t>(static_cast<uint32_t>(key)) * g.lddy + c) * ES, g.D - c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (done || at + u >= last) continue;
      if (tok[u] != now) {
        flush(false);
        began = false;
        now = tok[u];
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] = 0.0f;
        // With SMALL only tokens that begin in the piece are its own.
        done = now == kNoToken || (SMALL && at + u >= end);
        if (done) continue;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) sum[e] += static_cast<float>(x[u].v[e]);
    }
    at += U;
  }
  if (!done) flush(!SMALL && end < g.T && token_of(keys[end]) == now);
}

// Zeros in the rows without a token, of zero_rows rows.
template <typename E, bool SMALL>
__device__ inline void zero_rows(const GradArgs& g, const uint64_t* keys, uint32_t* used) {
  constexpr int N = Vec<E>::N;
  constexpr int64_t ES = sizeof(E);
  const int v0 = (static_cast<int>(blockIdx.x) - g.sum_groups) * g.zero_rows, rows = min(g.zero_rows, g.V - v0);
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += 256) used[i] = 0;
  __syncthreads();
  if (SMALL) {
    if (threadIdx.x < static_cast<unsigned>(g.T)) {
      const uint32_t v = usable(g.token[threadIdx.x], g.ignore, g.V) - static_cast<uint32_t>(v0);
      if (v < static_cast<uint32_t>(rows)) atomicOr(&used[v / 32], 1u << (v % 32));
    }
  } else {
    // 256 keys at a time from the first of these rows on.  Where the next token is
    // the last one again, its end is searched for: a batch may be one token.
    int at = lower_bound(keys, g.T, key_of(v0, 0));
    while (at < g.T) {
      const int i = at + static_cast<int>(threadIdx.x);
      const uint32_t v = i < g.T ? token_of(keys[i]) - static_cast<uint32_t>(v0) : kNoToken;
      if (v < static_cast<uint32_t>(rows)) atomicOr(&used[v / 32], 1u << (v % 32));
      at += 256;
      if (at >= g.T) break;
      const uint32_t before = token_of(keys[at - 1]), next = token_of(keys[at]);
      if (next >= static_cast<uint32_t>(v0 + rows)) break;
      if (next == before) at = lower_bound(keys, g.T, key_of(next + 1, 0));
    }
  }
  __syncthreads();
  const uint32_t per_row = static_cast<uint32_t>((g.D + N - 1) / N), total = per_row * static_cast<uint32_t>(rows);
  Vec<E> z;
#pragma unroll
  for (int e = 0; e < N; ++e) z.v[e] = static_cast<E>(0.0f);
  for (uint32_t i = threadIdx.x; i < total; i += 256) {
    const uint32_t row = i / per_row;
    const int c = static_cast<int>(i - row * per_row) * N;
    if (!(used[row / 32] >> (row % 32) & 1)) z.store(g.dw + ((v0 + static_cast<int64_t>(row)) * g.lddw + c) * ES, g.D - c);
  }
}

constexpr int kZeroRows = 1024;  // of a workgroup, at most

template <typename E, bool SMALL>
__global__ __launch_bounds__(256) void embed_grad_kernel(GradArgs g) {
  __shared__ uint64_t sorted[SMALL ? kSmall : 1];
  __shared__ uint32_t used[kZeroRows / 32];
  if (static_cast<int>(blockIdx.x) >= g.sum_groups) return zero_rows<E, SMALL>(g, g.keys, used);
  if constexpr (SMALL) sort_small(g, sorted);
  sum_rows<E, SMALL>(g, SMALL ? sorted : g.keys);
}

// The sums of a token that goes on from piece to piece: the piece in which it
// begins adds up its own part and the others', in order.  Four waves share the
// pieces; a lane has four columns, eight loads in flight.
template <typename E>
__global__ __launch_bounds__(256) void embed_join_kernel(GradArgs g) {
  constexpr int64_t ES = sizeof(E);
  __shared__ float4 sums[4][64];
  const int piece = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int first = piece * g.piece, end = first + g.piece;  // not the last piece
  const uint32_t v = token_of(g.keys[end]);
  if (v == kNoToken || token_of(g.keys[end - 1]) != v) return;  // nothing goes on
  if (first > 0 && token_of(g.keys[first - 1]) == v) return;    // it began before
  const int stop = lower_bound(g.keys, g.T, key_of(v + 1, 0));
  const int n = (stop - 1) / g.piece - piece;  // pieces behind this one, one at least
  const int per = (n + 3) / 4, from = wave * per, to = min(from + per, n);
  for (int c = (blockIdx.y * 64 + lane) * 4; c - 4 * lane < g.D; c += gridDim.y * 256) {
    const bool live = c < g.D;
    float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](const float4& x) __attribute__((always_inline)) {
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    };
    if (live) {
      const float* p = g.part + 2ll * (piece + 1) * g.ld_part + c;
      if (wave == 0) add(*reinterpret_cast<const float4*>(p - g.ld_part));
      for (int k = from; k < to; k += 8) {
        float4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = *reinterpret_cast<const float4*>(p + 2ll * min(k + u, to - 1) * g.ld_part);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (k + u < to) add(x[u]);
      }
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && live) {
#pragma unroll
      for (int x = 1; x < 4; ++x) add(sums[x][lane]);
      const float v4[4] = {s.x, s.y, s.z, s.w};
      char* to_row = g.dw + (static_cast<int64_t>(v) * g.lddw + c) * ES;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c + e >= g.D) continue;
        E x;
        if (g.add) {
          __builtin_memcpy(&x, to_row + e * ES, ES);
          x = static_cast<E>(__builtin_fmaf(g.scale, v4[e], static_cast<float>(x)));
        } else {
          x = static_cast<E>(g.scale * v4[e]);
        }
        __builtin_memcpy(to_row + e * ES, &x, ES);
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace fconv

struct fconv_embed_plan_s {
  fconv_embed_desc d;
  int32_t es;
  bool small;
  int32_t chunk, merges;          // tokens of a ranked chunk; launches that merge
  int32_t piece, pieces, team, col_blocks, zero_rows;
  int64_t ld_part;
  size_t o_other, o_part, bytes;  // workspace: keys, keys, parts
};

namespace fconv {
namespace {

constexpr int64_t kMaxElements = 1ll << 33, kMaxTokens = 4194240;
constexpr int32_t kMaxWidth = 1 << 20, kMaxRows = 1 << 24;

template <typename E>
hipError_t run_forward(const fconv_embed_plan_s* p, const fconv_embed_args* a, hipStream_t s) {
  const fconv_embed_desc& d = p->d;
  const LookupArgs g = {a->token, d.ignore_index, static_cast<const char*>(a->w), a->ldw, static_cast<char*>(a->y),
                        a->ldy, d.T, d.D, d.V, d.scale};
  const int64_t pieces = d.T * ceil_div(d.D, Vec<E>::N);
  hipLaunchKernelGGL(embed_lookup_kernel<E>, dim3(static_cast<unsigned>(ceil_div(pieces, 1024))), dim3(256), 0, s, g);
  return hipGetLastError();
}

template <typename E>
hipError_t run_backward(const fconv_embed_plan_s* p, const fconv_embed_args* a, hipStream_t s) {
  const fconv_embed_desc& d = p->d;
  const bool add = a->run_flags & FCONV_EMBED_ADD;
  char* ws = static_cast<char*>(a->workspace);
  hipError_t e;
  uint64_t *keys = reinterpret_cast<uint64_t*>(ws), *other = reinterpret_cast<uint64_t*>(ws + p->o_other);
  if (!p->small) {
    const dim3 grid(static_cast<unsigned>(ceil_div(d.T < p->chunk ? d.T : p->chunk, 64)),
                    static_cast<unsigned>(ceil_div(d.T, p->chunk)));
    hipLaunchKernelGGL(embed_rank_kernel, grid, dim3(256), 0, s, a->token, d.ignore_index, d.T, d.V, p->chunk, keys);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    int64_t run = p->chunk;
    for (int i = 0; i < p->merges; ++i, run *= kWays) {
      hipLaunchKernelGGL(embed_merge_kernel, dim3(static_cast<unsigned>(ceil_div(d.T, 64))), dim3(256), 0, s, keys,
                         other, d.T, static_cast<int32_t>(run));
      if ((e = hipGetLastError()) != hipSuccess) return e;
      uint64_t* t = keys;
      keys = other;
      other = t;
    }
  }
  GradArgs g = {};
  g.keys = keys;
  g.token = a->token;
  g.ignore = d.ignore_index;
  g.dy = static_cast<const char*>(a->dy);
  g.lddy = a->lddy;
  g.dw = static_cast<char*>(a->dw);
  g.lddw = a->lddw;
  g.part = reinterpret_cast<float*>(ws + p->o_part);
  g.ld_part = p->ld_part;
  g.T = d.T;
  g.D = d.D;
  g.V = d.V;
  g.piece = p->piece;
  g.pieces = p->pieces;
  g.team = p->team;
  g.col_blocks = p->col_blocks;
  g.sum_groups = static_cast<int32_t>(ceil_div(p->pieces, 256 / p->team) * p->col_blocks);
  g.zero_rows = p->zero_rows;
  g.scale = d.scale;
  g.add = add;
  const int64_t groups = g.sum_groups + (add ? 0 : ceil_div(d.V, p->zero_rows));
  if (groups == 0) return hipSuccess;
  if (p->small)
    hipLaunchKernelGGL((embed_grad_kernel<E, true>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((embed_grad_kernel<E, false>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, s, g);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (p->small || p->pieces < 2) return hipSuccess;
  const int64_t cols = ceil_div(d.D, 256);
  hipLaunchKernelGGL(embed_join_kernel<E>, dim3(static_cast<unsigned>(p->pieces - 1), static_cast<unsigned>(cols < 64 ? cols : 64)),
                     dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace
}  // namespace fconv

extern "C" {

fconv_status fconv_embed_plan_create(const fconv_embed_desc* desc, fconv_embed_plan* out) {
  using namespace fconv;
  if (!desc || !out) return FCONV_ERR_INVALID_ARG;
  *out = nullptr;
  const fconv_embed_desc& d = *desc;
  if (d.dtype != FCONV_BF16 && d.dtype != FCONV_FP32) return FCONV_ERR_UNSUPPORTED;
  if (d.flags) return FCONV_ERR_UNSUPPORTED;
  if (d.T < 0 || d.D < 1 || d.V < 1 || !std::isfinite(d.scale)) return FCONV_ERR_INVALID_ARG;
  if (d.D > kMaxWidth || d.V > kMaxRows || d.T > kMaxTokens || static_cast<int64_t>(d.T) * d.D > kMaxElements ||
      static_cast<int64_t>(d.V) * d.D > kMaxElements)
    return FCONV_ERR_UNSUPPORTED;
  fconv_embed_plan_s* p = new (std::nothrow) fconv_embed_plan_s();
  if (!p) return FCONV_ERR_INVALID_ARG;
  p->d = d;
  p->es = d.dtype == FCONV_BF16 ? 2 : 4;
  const int64_t T = d.T, vecs = ceil_div(d.D, 16 / p->es);
  p->small = T <= kSmall;
  // Up to kChunk tokens one chunk; of more, sixteen chunks if they can be.
  p->chunk = static_cast<int32_t>(T <= kChunk ? round_up(T < 64 ? 64 : T, 64) : round_up(ceil_div(T, kWays), 64));
  if (p->chunk > kChunk) p->chunk = kChunk;
  for (int64_t run = p->chunk; run < T; run *= kWays) ++p->merges;
  p->piece = T <= 4096 ? 16 : T <= 32768 ? 32 : 64;
  p->pieces = static_cast<int32_t>(ceil_div(T, p->piece));
  p->team = 8;
  while (p->team < 256 && p->team < vecs) p->team *= 2;
  p->col_blocks = static_cast<int32_t>(ceil_div(vecs, p->team));
  int64_t rows = (256 << 10) / (static_cast<int64_t>(d.D) * p->es);
  p->zero_rows = static_cast<int32_t>(rows < 4 ? 4 : rows > kZeroRows ? kZeroRows : rows);
  p->ld_part = round_up(d.D, 8);
  if (!p->small) {
    const size_t keys = static_cast<size_t>(round_up(T * 8, 256));
    p->o_other = keys;
    p->o_part = keys + (p->merges ? keys : 0);
    p->bytes = p->o_part + static_cast<size_t>(p->pieces) * 2 * p->ld_part * 4;
  }
  *out = p;
  return FCONV_OK;
}

fconv_status fconv_embed_plan_workspace_size(fconv_embed_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->bytes;
  return FCONV_OK;
}

fconv_status fconv_embed_plan_forward(fconv_embed_plan p, void* stream, const fconv_embed_args* a) {
  using namespace fconv;
  if (!p || !a) return FCONV_ERR_INVALID_ARG;
  const fconv_embed_desc& d = p->d;
  if (a->run_flags) return FCONV_ERR_INVALID_ARG;
  if (d.T == 0) return FCONV_OK;
  if (!a->token || !a->w || !a->y) return FCONV_ERR_INVALID_ARG;
  if (bad_ld(a->ldw, d.D) || bad_ld(a->ldy, d.D)) return FCONV_ERR_INVALID_ARG;
  if (!aligned(a->token, 8) || !aligned(a->w, p->es) || !aligned(a->y, p->es)) return FCONV_ERR_MISALIGNED;
  const Range in[] = {{a->token, static_cast<size_t>(d.T) * 8}, {a->w, span(d.V, d.D, a->ldw, p->es)}};
  const Range wr[] = {{a->y, span(d.T, d.D, a->ldy, p->es)}};
  if (clash(wr, 1, in, 2)) return FCONV_ERR_INVALID_ARG;
  const hipError_t e = d.dtype == FCONV_BF16 ? run_forward<__bf16>(p, a, as_stream(stream))
                                             : run_forward<float>(p, a, as_stream(stream));
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_embed_plan_backward(fconv_embed_plan p, void* stream, const fconv_embed_args* a) {
  using namespace fconv;
  if (!p || !a) return FCONV_ERR_INVALID_ARG;
  const fconv_embed_desc& d = p->d;
  if (a->run_flags & ~static_cast<uint32_t>(FCONV_EMBED_ADD)) return FCONV_ERR_INVALID_ARG;
  if (!a->dw || bad_ld(a->lddw, d.D)) return FCONV_ERR_INVALID_ARG;
  if (!aligned(a->dw, p->es)) return FCONV_ERR_MISALIGNED;
  if (d.T > 0) {
    if (!a->token || !a->dy || bad_ld(a->lddy, d.D)) return FCONV_ERR_INVALID_ARG;
    if (p->bytes && (!a->workspace || a->workspace_bytes < p->bytes)) return FCONV_ERR_WORKSPACE;
    if (!aligned(a->token, 8) || !aligned(a->dy, p->es) || !aligned(a->workspace, 16)) return FCONV_ERR_MISALIGNED;
    const Range in[] = {{a->token, static_cast<size_t>(d.T) * 8}, {a->dy, span(d.T, d.D, a->lddy, p->es)}};
    const Range wr[] = {{a->dw, span(d.V, d.D, a->lddw, p->es)}, {a->workspace, p->bytes}};
    if (clash(wr, 2, in, 2)) return FCONV_ERR_INVALID_ARG;
  }
  const hipError_t e = d.dtype == FCONV_BF16 ? run_backward<__bf16>(p, a, as_stream(stream))
                                             : run_backward<float>(p, a, as_stream(stream));
  return e == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_embed_plan_destroy(fconv_embed_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
