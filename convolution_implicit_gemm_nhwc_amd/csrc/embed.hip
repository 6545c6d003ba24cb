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
//           smaller ones of its chunk: as many comparisons a token as the chunk
//           has tokens, and no passes
//   merge   sixteen sorted runs at a time: a key's place is the sum of its ranks
//           in them, found by binary searches
//   sums    pieces of `piece` sorted keys: their rows of dy are summed; a token
//           whose keys all lie in the piece is done, the others' sums of the piece
//           go out
//   join    adds the pieces' sums of a token, in order
// Rows without a token are written by other workgroups: beside the ranking, whose
// time that hides, as long as each of them can look at all tokens (kScan), and of
// longer batches beside the sums, by searching the sorted keys.
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
constexpr int kScan = 32768;  // tokens that a workgroup looks through for its rows
constexpr int kChunk = 4096;  // tokens of a chunk that is ranked, at most
constexpr int kWays = 16;     // runs merged at a time
constexpr uint32_t kNoToken = 0x7fffffffu;  // sorts behind every token

__device__ inline uint64_t key_of(uint32_t token, uint32_t place) { return static_cast<uint64_t>(token) << 32 | place; }
__device__ inline uint32_t token_of(uint64_t key) { return static_cast<uint32_t>(key >> 32); }
__device__ inline uint32_t usable(int64_t token, int64_t ignore, int32_t V) {
  return token != ignore && token >= 0 && token < V ? static_cast<uint32_t>(token) : kNoToken;
}

// 16 bytes of elements of type E.  A row's last piece, if it is not whole, is moved
// back to end with the row (piece_at), so that every piece of a row of at least N
// elements is whole: a load that may not happen waits for the one before it, since
// either may be what fills a register (sums of 448 tokens of 667 columns: 18 us with
// the last piece's elements one by one).  What two threads then both have is the
// same in both.
template <typename E>
struct Vec {
  static constexpr int N = 16 / sizeof(E);
  E v[N];
  // WHOLE: rows of at least N elements; else n of them at p, zeros past those.
  template <bool WHOLE>
  __device__ void load(const char* p, int n) {
    if (WHOLE || n >= N) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[e] = static_cast<E>(0.0f);
        if (e < n) __builtin_memcpy(&v[e], p + e * sizeof(E), sizeof(E));
      }
    }
  }
  // PAST: past the caches.
  template <bool WHOLE, bool PAST = false>
  __device__ void store(char* p, int n) const {
    if (WHOLE || n >= N) {
      if constexpr (PAST) {
        typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
        Words w;
        __builtin_memcpy(&w, v, 16);
        __builtin_nontemporal_store(w, reinterpret_cast<Words*>(p));
      } else {
        __builtin_memcpy(p, v, 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < n) __builtin_memcpy(p + e * sizeof(E), &v[e], sizeof(E));
    }
  }
};
// First column of a row's piece that begins with c.
template <typename E, bool WHOLE>
__device__ inline int piece_at(int c, int D) {
  return WHOLE ? min(c, D - Vec<E>::N) : c;
}

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
// T D is at most 2^33 elements.  32768 x 2048 bf16: 31 us, 134 MB written at 4.3 TB/s
// while 74 MB of rows are read (tokens repeat, and caches hold their rows).
template <typename E, bool WHOLE>
__device__ inline void lookup(const LookupArgs& a) {
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
    const int c = piece_at<E, WHOLE>(static_cast<int>(i % per_row) * N, a.D);
    if (usable(tok[u], a.ignore, a.V) != kNoToken) v[u].template load<WHOLE>(a.w + (tok[u] * a.ldw + c) * ES, a.D - c);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + 256u * u;
    if (i >= total) break;
    const int64_t row = i / per_row;
    const int c = piece_at<E, WHOLE>(static_cast<int>(i - static_cast<uint32_t>(row) * per_row) * N, a.D);
    if (usable(tok[u], a.ignore, a.V) == kNoToken) {
      const float f = tok[u] == a.ignore ? 0.0f : __builtin_nanf("");
#pragma unroll
      for (int e = 0; e < N; ++e) v[u].v[e] = static_cast<E>(f);
    } else if (a.scale != 1.0f) {
#pragma unroll
      for (int e = 0; e < N; ++e) v[u].v[e] = static_cast<E>(a.scale * static_cast<float>(v[u].v[e]));
    }
    v[u].template store<WHOLE>(a.y + (row * a.ldy + c) * ES, a.D - c);
  }
}

template <typename E>
__global__ __launch_bounds__(256) void embed_lookup_kernel(LookupArgs a) {
  if (a.D >= Vec<E>::N)
    lookup<E, true>(a);
  else
    lookup<E, false>(a);
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
  bool past;              // zeros go past the caches
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

// scale sum, or that added to what is there, from column c on; the first `own` of
// the columns are another thread's.
template <typename E>
__device__ inline void put_row(const GradArgs& g, uint32_t v, int c, int own, const float (&sum)[Vec<E>::N]) {
  constexpr int N = Vec<E>::N;
  constexpr int64_t ES = sizeof(E);
  char* p = g.dw + (static_cast<int64_t>(v) * g.lddw + c) * ES;
  if (own == 0 && g.D - c >= N) {
    Vec<E> x;
    if (g.add) {
      x.template load<true>(p, N);
#pragma unroll
      for (int e = 0; e < N; ++e) x.v[e] = static_cast<E>(__builtin_fmaf(g.scale, sum[e], static_cast<float>(x.v[e])));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x.v[e] = static_cast<E>(g.scale * sum[e]);
    }
    x.template store<true>(p, N);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (e < own || c + e >= g.D) continue;
    E x = static_cast<E>(g.scale * sum[e]);
    if (g.add) {
      __builtin_memcpy(&x, p + e * ES, ES);
      x = static_cast<E>(__builtin_fmaf(g.scale, sum[e], static_cast<float>(x)));
    }
    __builtin_memcpy(p + e * ES, &x, ES);
  }
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

// Sums of dy's rows of a piece of the sorted keys, 16 bytes of columns from c on, of
// which the first `own` are another thread's.  Eight rows are in flight.  Without
// SMALL, a piece's first token may have begun before it and its last one may go on
// behind it: their sums go to `part`.  With SMALL a token belongs to the piece in
// which it begins, which then reads on.  16384 x 4096 bf16: 35 us for 121 MB read and
// 53 written, 5 TB/s; 1999 x 1000 fp32: 8 us, a piece's rows one after another.
template <typename E, bool SMALL, bool WHOLE>
__device__ inline void sum_piece(const GradArgs& g, const uint64_t* keys, int piece, int c, int own) {
  constexpr int N = Vec<E>::N, U = 8;
  constexpr int64_t ES = sizeof(E);
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
      put_row<E>(g, now, c, own, sum);
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
      x[u].template load<WHOLE>(g.dy + (static_cast<int64_t>(static_cast<uint32_t>(key)) * g.lddy + c) * ES, g.D - c);
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

// A team's threads each hold 16 bytes of a piece's columns.
template <typename E, bool SMALL>
__device__ inline void sum_rows(const GradArgs& g, const uint64_t* keys) {
  constexpr int N = Vec<E>::N;
  const int teams = 256 / g.team, block = blockIdx.x % g.col_blocks;
  const int piece = blockIdx.x / g.col_blocks * teams + threadIdx.x / g.team;
  const int c = (block * g.team + threadIdx.x % g.team) * N;
  if (piece >= g.pieces || c >= g.D) return;
  if (g.D >= N) {
    const int at = piece_at<E, true>(c, g.D);
    sum_piece<E, SMALL, true>(g, keys, piece, at, c - at);
  } else {
    sum_piece<E, SMALL, false>(g, keys, piece, c, 0);
  }
}

constexpr int kZeroRows = 1024;  // of a workgroup, at most

// Zeros in the rows without a token, of the `group`th zero_rows rows; THREADS
// threads.  SCAN: which rows have one is seen by looking through all tokens,
// eight of a thread in flight, else by the sorted keys.
template <typename E, bool SCAN, int THREADS>
__device__ inline void zero_rows(const GradArgs& g, int group) {
  __shared__ uint32_t used[kZeroRows / 32];
  constexpr int N = Vec<E>::N, U = 8;
  constexpr int64_t ES = sizeof(E);
  const int v0 = group * g.zero_rows, rows = min(g.zero_rows, g.V - v0), tid = threadIdx.x;
  for (int i = tid; i < (rows + 31) / 32; i += THREADS) used[i] = 0;
  __syncthreads();
  auto mark = [&](uint32_t token) __attribute__((always_inline)) {
    const uint32_t v = token - static_cast<uint32_t>(v0);
    if (v < static_cast<uint32_t>(rows)) atomicOr(&used[v / 32], 1u << (v % 32));
  };
  if (SCAN) {
    for (int i = tid; i < g.T; i += THREADS * U) {
      int64_t tok[U];
#pragma unroll
      for (int u = 0; u < U; ++u) tok[u] = g.token[min(i + u * THREADS, g.T - 1)];
#pragma unroll
      for (int u = 0; u < U; ++u) mark(usable(tok[u], g.ignore, g.V));
    }
  } else {
    // From the first of these rows on.  Where the next token is the last one again,
    // its end is searched for: a batch may be one token.
    int at = lower_bound(g.keys, g.T, key_of(v0, 0));
    while (at < g.T) {
      mark(at + tid < g.T ? token_of(g.keys[at + tid]) : kNoToken);
      at += THREADS;
      if (at >= g.T) break;
      const uint32_t before = token_of(g.keys[at - 1]), next = token_of(g.keys[at]);
      if (next >= static_cast<uint32_t>(v0 + rows)) break;
      if (next == before) at = lower_bound(g.keys, g.T, key_of(next + 1, 0));
    }
  }
  __syncthreads();
  const uint32_t per_row = static_cast<uint32_t>((g.D + N - 1) / N), total = per_row * static_cast<uint32_t>(rows);
  Vec<E> z;
#pragma unroll
  for (int e = 0; e < N; ++e) z.v[e] = static_cast<E>(0.0f);
  for (uint32_t i = tid; i < total; i += THREADS) {
    const uint32_t row = i / per_row;
    const int c0 = static_cast<int>(i - row * per_row) * N, c = g.D >= N ? piece_at<E, true>(c0, g.D) : c0;
    if (used[row / 32] >> (row % 32) & 1) continue;
    char* p = g.dw + ((v0 + static_cast<int64_t>(row)) * g.lddw + c) * ES;
    if (g.past)
      z.template store<false, true>(p, g.D - c);
    else
      z.template store<false>(p, g.D - c);
  }
}

template <typename E, bool SMALL>
__global__ __launch_bounds__(256) void embed_grad_kernel(GradArgs g) {
  if (static_cast<int>(blockIdx.x) >= g.sum_groups)
    return zero_rows<E, SMALL, 256>(g, static_cast<int>(blockIdx.x) - g.sum_groups);
  if constexpr (SMALL) {
    __shared__ uint64_t sorted[kSmall];
    sort_small(g, sorted);
    sum_rows<E, SMALL>(g, sorted);
  } else {
    sum_rows<E, SMALL>(g, g.keys);
  }
}

// -------------------------------------------------------------------- sorting

// Keys of each chunk, sorted: a workgroup ranks 64 of them, each of its sixteen
// waves against every sixteenth block of 64.  Of equal tokens the earlier
// one is smaller: in a block before the own one "not larger" counts, in one behind
// it "smaller".  Workgroups behind those that rank write the rows of zeros: they set
// the time (65536 x 4096 bf16, 16384 tokens: 491 MB in 90 to 94 us, 5.3 TB/s; 32001 x
// 1000 fp32, 1999 tokens: 124 MB in 22 to 23 us).
template <typename E>
__global__ __launch_bounds__(1024) void embed_rank_kernel(GradArgs g, int chunk, int rank_groups, uint64_t* keys) {
  if (static_cast<int>(blockIdx.x) >= rank_groups)
    return zero_rows<E, true, 1024>(g, static_cast<int>(blockIdx.x) - rank_groups);
  __shared__ __attribute__((aligned(16))) uint32_t all[kChunk];
  __shared__ int ranks[16][64];
  const int blocks = chunk / 64, base = blockIdx.x / blocks * chunk, n = min(chunk, g.T - base), n64 = (n + 63) / 64 * 64;
  const int own = blockIdx.x % blocks * 64;
  if (own >= n) return;
  int64_t tok[kChunk / 1024];
#pragma unroll
  for (int u = 0; u < kChunk / 1024; ++u) {
    const int i = u * 1024 + static_cast<int>(threadIdx.x);
    tok[u] = i < n ? g.token[base + i] : -1;
  }
#pragma unroll
  for (int u = 0; u < kChunk / 1024; ++u) {
    const int i = u * 1024 + static_cast<int>(threadIdx.x);
    if (i < n64) all[i] = i < n ? usable(tok[u], g.ignore, g.V) : kNoToken;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t mine = all[own + lane];
  int rank = 0;
  for (int b = wave * 64; b < n64; b += 1024) {
    const uint4* p = reinterpret_cast<const uint4*>(all + b);
    // Smaller than mine, or than the next one where equal ones count too (no overflow: kNoToken is not the largest).
    const uint32_t below = b < own ? mine + 1 : mine;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint4 k = p[i];
      rank += (k.x < below) + (k.y < below) + (k.z < below) + (k.w < below);
      if (b == own) {
        rank += (k.x == mine && 4 * i < lane) + (k.y == mine && 4 * i + 1 < lane) + (k.z == mine && 4 * i + 2 < lane) +
                (k.w == mine && 4 * i + 3 < lane);
      }
    }
  }
  ranks[wave][lane] = rank;
  __syncthreads();
  // What fills the last block up ranks behind the chunk's own keys.
  if (wave != 0 || own + lane >= n) return;
  rank = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) rank += ranks[w][lane];
  keys[base + rank] = key_of(mine, static_cast<uint32_t>(base + own + lane));
}

// Groups of kWays sorted runs of `run` keys become one each.  Four lanes share a
// key, each with four of the runs, whose searches go on side by side.  The last
// keys of 64 parts of each run are brought to LDS first: a step of a search that
// goes to memory takes most of a microsecond (16384 tokens, sixteen runs: 11.7 us
// with all eleven steps there, 7 now).
__global__ __launch_bounds__(512) void embed_merge_kernel(const uint64_t* in, uint64_t* out, int32_t T, int32_t run) {
  constexpr int M = kWays / 4;
  __shared__ uint64_t samples[kWays][64];
  const int per_group = run * kWays, blocks = (per_group + 127) / 128;  // of 128 keys
  const int64_t first = static_cast<int64_t>(blockIdx.x / blocks) * per_group;  // of the group
  const int step = (run + 63) / 64;  // of a part
  const int64_t block = first + static_cast<int64_t>(blockIdx.x % blocks) * 128, at = block + threadIdx.x / 4;
  if (block >= T) return;
#pragma unroll
  for (int i = threadIdx.x; i < kWays * 64; i += 512) {
    const int k = i / 64, p = i % 64;
    const int in_run = (p + 1) * step - 1;
    const int64_t x = first + static_cast<int64_t>(k) * run + in_run;
    samples[k][p] = in_run < run && x < T ? in[x] : ~0ull;
  }
  const bool live = at < T && at < first + per_group;
  const uint64_t key = in[live ? at : first];
  const int part = threadIdx.x & 3;
  __syncthreads();
  int lo[M], hi[M];  // keys below this one: of lo .. hi of the run
  int64_t base[M];
#pragma unroll
  for (int k = 0; k < M; ++k) {
    const int r = part * M + k;
    base[k] = first + static_cast<int64_t>(r) * run;
    const int64_t left = T - base[k];
    const int len = left <= 0 ? 0 : left < run ? static_cast<int>(left) : run;
    int p = 0;  // parts whose last key is below
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) p += samples[r][p + s - 1] < key ? s : 0;
    p += samples[r][p] < key;  // p is at most 63 here
    lo[k] = min(p * step, len);
    hi[k] = min(lo[k] + step - 1, len);
  }
  for (int s = step; s > 1; s = (s + 1) / 2) {  // hi - lo is below s
    uint64_t x[M];
#pragma unroll
    for (int k = 0; k < M; ++k) x[k] = lo[k] < hi[k] ? in[base[k] + (lo[k] + hi[k]) / 2] : 0;
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const int mid = (lo[k] + hi[k]) / 2;
      if (lo[k] < hi[k]) {
        if (x[k] < key)
          lo[k] = mid + 1;
        else
          hi[k] = mid;
      }
    }
  }
  int rank = 0;
#pragma unroll
  for (int k = 0; k < M; ++k) rank += lo[k];
  rank += __shfl_xor(rank, 1);
  rank += __shfl_xor(rank, 2);
  if (live && part == 0) out[first + rank] = key;
}

// The sums of a token that goes on from piece to piece: the piece in which it
// begins adds up its own part and the others', in order.  A workgroup has 1024
// columns: each wave 256 of them, four of a lane, or of a long token (kShared pieces)
// all waves the same 256 at a time, each with a quarter of the pieces.  Eight
// loads of a lane are in flight (16384 x 4096: 6 us, the launch and one round of loads).
constexpr int kShared = 32;

template <typename E>
__global__ __launch_bounds__(256) void embed_join_kernel(GradArgs g) {
  constexpr int64_t ES = sizeof(E);
  __shared__ float4 sums[4][64];
  const int piece = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int first = piece * g.piece, end = first + g.piece;  // not the last piece
  // All at once: the keys about this piece's ends, and those that the next 64 begin with.
  auto begins = [&](int n) __attribute__((always_inline)) {
    return g.keys[min(end + (static_cast<int64_t>(n) + lane) * g.piece, static_cast<int64_t>(g.T) - 1)];
  };
  uint64_t key = begins(0);
  const uint32_t last = token_of(g.keys[end - 1]), before = token_of(g.keys[first > 0 ? first - 1 : 0]);
  const uint32_t v = token_of(__shfl(key, 0));
  if (v == kNoToken || last != v || (first > 0 && before == v)) return;  // nothing goes on, or it began before
  // Pieces behind this one that begin with the token, one at least.
  int n = 0;
  for (;;) {
    const bool there = end + (static_cast<int64_t>(n) + lane) * g.piece < g.T && token_of(key) == v;
    const int more = __popcll(__ballot(there));
    n += more;
    if (more < 64) break;
    key = begins(n);
  }
  auto add = [&](float4& s, const float4& x) __attribute__((always_inline)) {
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  };
  // Parts [from, to) behind this piece's own, which comes first if `own`.
  auto sum = [&](int c, int from, int to, bool own) __attribute__((always_inline)) {
    float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    const float* p = g.part + 2ll * (piece + 1) * g.ld_part + c;
    if (own) s = *reinterpret_cast<const float4*>(p - g.ld_part);
    for (int k = from; k < to; k += 8) {
      float4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = *reinterpret_cast<const float4*>(p + 2ll * min(k + u, to - 1) * g.ld_part);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k + u < to) add(s, x[u]);
    }
    return s;
  };
  auto put = [&](int c, const float4& s) __attribute__((always_inline)) {
    const float f[4] = {s.x, s.y, s.z, s.w};
    char* p = g.dw + (static_cast<int64_t>(v) * g.lddw + c) * ES;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e >= g.D) continue;
      E x;
      if (g.add) {
        __builtin_memcpy(&x, p + e * ES, ES);
        x = static_cast<E>(__builtin_fmaf(g.scale, f[e], static_cast<float>(x)));
      } else {
        x = static_cast<E>(g.scale * f[e]);
      }
      __builtin_memcpy(p + e * ES, &x, ES);
    }
  };
  const int c0 = blockIdx.y * 1024 + lane * 4;
  if (n < kShared) {
    const int c = c0 + wave * 256;
    if (c < g.D) put(c, sum(c, 0, n, true));
    return;
  }
  const int per = (n + 3) / 4, from = wave * per, to = min(from + per, n);
  for (int b = 0; b < 4; ++b) {
    const int c = c0 + b * 256;
    if (c < g.D) sums[wave][lane] = sum(c, from, to, wave == 0);
    __syncthreads();
    if (wave == b && c < g.D) {
      float4 s = sums[0][lane];
#pragma unroll
      for (int x = 1; x < 4; ++x) add(s, sums[x][lane]);
      put(c, s);
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
  GradArgs g = {};
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
  // Where dy and dw are more than the last-level cache holds, zeros past it leave dy there (16384 tokens, 65536 x
  // 4096 bf16: 135 us instead of 160; 65536 tokens, 65536 x 1024: 100 and 110); where dw stays in it, or dy is
  // small, they cost (1999 tokens, 32001 x 1000: 29 and 27; 300 tokens, 65536 x 4096: 105 and 103).
  const int64_t dy_bytes = static_cast<int64_t>(d.T) * d.D * p->es, dw_bytes = static_cast<int64_t>(d.V) * d.D * p->es;
  g.past = dy_bytes + dw_bytes >= 256ll << 20 && dy_bytes >= 32ll << 20;
  int64_t zero_groups = add ? 0 : ceil_div(d.V, p->zero_rows);
  if (!p->small) {
    const int64_t rank_groups = ceil_div(d.T, p->chunk) * (p->chunk / 64), beside = d.T <= kScan ? zero_groups : 0;
    hipLaunchKernelGGL(embed_rank_kernel<E>, dim3(static_cast<unsigned>(rank_groups + beside)), dim3(1024), 0, s, g,
                       p->chunk, static_cast<int>(rank_groups), keys);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    zero_groups -= beside;
    int64_t run = p->chunk;
    for (int i = 0; i < p->merges; ++i, run *= kWays) {
      const int64_t group = run * kWays, blocks = ceil_div(d.T, group) * ceil_div(group, 128);
      hipLaunchKernelGGL(embed_merge_kernel, dim3(static_cast<unsigned>(blocks)), dim3(512), 0, s, keys, other, d.T,
                         static_cast<int32_t>(run));
      if ((e = hipGetLastError()) != hipSuccess) return e;
      uint64_t* t = keys;
      keys = other;
      other = t;
    }
    g.keys = keys;
  }
  const int64_t groups = g.sum_groups + zero_groups;
  if (groups == 0) return hipSuccess;
  if (p->small)
    hipLaunchKernelGGL((embed_grad_kernel<E, true>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((embed_grad_kernel<E, false>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, s, g);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (p->small || p->pieces < 2) return hipSuccess;
  hipLaunchKernelGGL(embed_join_kernel<E>, dim3(static_cast<unsigned>(p->pieces - 1), static_cast<unsigned>(ceil_div(d.D, 1024))),
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
  p->team = 8;
  while (p->team < 256 && p->team < vecs) p->team *= 2;
  p->col_blocks = static_cast<int32_t>(ceil_div(vecs, p->team));
  // Long pieces leave fewer sums to join; four workgroups a CU hide the reads' latency.
  p->piece = 64;
  while (p->piece > 16 && ceil_div(ceil_div(T, p->piece), 256 / p->team) * p->col_blocks < 1024) p->piece /= 2;
  p->pieces = static_cast<int32_t>(ceil_div(T, p->piece));
  // 256 KB of zeros for a workgroup, in four rows at least; less of a small table, for more workgroups, up to 512 and
  // as long as those do not look through more than 32 MB of tokens for it.  What 256 KB each make of a large table has no
  // such bound: the 2048 workgroups of 65536 x 4096 bf16 look through 268 MB for 16384 tokens, out of the caches.
  int64_t rows = (256 << 10) / (static_cast<int64_t>(d.D) * p->es), most = (4ll << 20) / (T > 0 ? T : 1);
  most = most > 512 ? 512 : most < 1 ? 1 : most;
  if (rows > ceil_div(d.V, most)) rows = ceil_div(d.V, most);
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
