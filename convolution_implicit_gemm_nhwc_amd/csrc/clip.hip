// Norm of many gradients together on gfx950 (CDNA4), clipping by it, and their
// C ABI (include/fconv_clip.h).
//
//   norm = sqrt(sum of squares)     out = min(1, max_norm / (norm + eps)) in
//
// Both are bound by memory.  Tensors are taken in chunks of 16 KiB; a launch has
// up to kBatch tensors in its arguments, so nothing about them has to be in device
// memory beforehand, and a captured call holds its own list.  A workgroup owns a
// range of a launch's chunks, one after another: it finds its first tensor once.
//   squares  each workgroup leaves the sum of its elements' squares, in 64 bits
//   norm     adds those up (one workgroup; only where the next kernel does not)
//   scale    every workgroup adds up to kOwnParts sums itself, in the same order,
//            which is quicker than a launch, then scales its chunks, the last one
//            first: the last-level cache still holds what `squares` read last, and
//            results that it could not hold go past it (505 million bf16 gradients:
//            537 us instead of 600)
// Those 505 million: squares 156 to 163 us (6.2 to 6.5 TB/s), scale 381 to 390 (5.2 to
// 5.3 TB/s, read and written); of 185 million fp32 squares 123 to 125 us (5.9 to 6.0).
//
// Squares and sums are in 64 bits: in 32 those of gradients above 2^64 are infinite
// and those below 2^-75 vanish.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "dense.h"
#include "fconv_clip.h"

namespace fconv {
namespace {

constexpr int kBatch = 128;                // tensors of a launch: 3.6 KiB of arguments
constexpr int64_t kChunkBytes = 16 << 10;  // 256 threads, four pieces of 16 bytes each
// Workgroups of a launch, at most: two a CU keep enough loads in flight, and more of
// them only add sums (738 MB in place, below the limit: 512 127.7 us, 1024 133, 2048
// 134; 1 GB clipped: 537, 542, 599).
constexpr int kGroups = 512;
constexpr int kOwnParts = 2048;            // sums that every workgroup adds up by itself

struct Batch {
  const char* in[kBatch];
  char* out[kBatch];
  int64_t numel[kBatch];  // that of fp32 as -1 - numel
  int32_t first[kBatch + 1];  // chunks before each tensor
  int32_t n;
  bool in_place;  // all of them
};

struct ScaleArgs {
  const double* parts;  // n_parts sums; or n_parts = 0:
  const float* norm;    // the norm itself
  int32_t n_parts;
  float* write_norm;    // the norm is written there by the first workgroup, or NULL
  float max_norm, eps;
  bool past;            // results go past the caches
};

struct Chunk {
  const char* in;
  char* out;
  int left;  // bytes
  bool bf16;
};

// A workgroup's chunks, one after another (BACK: from the last one back).
template <bool BACK>
struct Walk {
  const Batch& b;
  int c, end;
  // Of the present tensor: its number, its chunks, its bytes, its places.
  int t, lo, hi;
  int64_t bytes;
  bool bf16;
  const char* in;
  char* out;

  __device__ explicit Walk(const Batch& batch) : b(batch) {
    const int64_t total = b.first[b.n];
    const int from = static_cast<int>(total * blockIdx.x / gridDim.x);
    const int to = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
    c = BACK ? to - 1 : from;
    end = BACK ? from - 1 : to;
    // The last tensor that begins at c or before: a wave looks at all of them at once.
    const int lane = threadIdx.x & 63;
    static_assert(kBatch == 128, "two tensors of a lane");
    const int before = __popcll(__ballot(lane < b.n && b.first[lane] <= c)) +
                       __popcll(__ballot(lane + 64 < b.n && b.first[lane + 64] <= c));
    tensor(__builtin_amdgcn_readfirstlane(before - 1));
  }
  __device__ void tensor(int number) {
    t = number;
    lo = b.first[t];
    hi = b.first[t + 1];
    const int64_t coded = b.numel[t];
    bf16 = coded >= 0;
    bytes = bf16 ? coded * 2 : (-1 - coded) * 4;
    in = b.in[t];
    out = b.out[t];
  }
  __device__ bool more() const { return c != end; }
  __device__ Chunk next() {
    if (BACK ? c < lo : c >= hi) tensor(BACK ? t - 1 : t + 1);
    const int64_t at = (c - lo) * kChunkBytes, left = bytes - at;
    c += BACK ? -1 : 1;
    return Chunk{in + at, out + at, static_cast<int>(left < kChunkBytes ? left : kChunkBytes), bf16};
  }
};

// Four pieces of 16 bytes of a chunk of `left` bytes: those of this thread.  A
// whole chunk asks nothing: a load that may not happen waits for the one before.
struct Pieces {
  uint32_t d[4][4];
  __device__ static int at(int u) { return (u * 256 + static_cast<int>(threadIdx.x)) * 16; }
  __device__ void load(const char* p, int left) {
    if (left == kChunkBytes) {
#pragma unroll
      for (int u = 0; u < 4; ++u) __builtin_memcpy(d[u], p + at(u), 16);
      return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (at(u) + 16 <= left) {
        __builtin_memcpy(d[u], p + at(u), 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t lo = 0, hi = 0;
          if (at(u) + 4 * i < left) __builtin_memcpy(&lo, p + at(u) + 4 * i, 2);
          if (at(u) + 4 * i + 2 < left) __builtin_memcpy(&hi, p + at(u) + 4 * i + 2, 2);
          d[u][i] = lo | static_cast<uint32_t>(hi) << 16;
        }
      }
    }
  }
  __device__ void store(char* p, int left, bool past) const {
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const Words w = {d[u][0], d[u][1], d[u][2], d[u][3]};
      if (at(u) + 16 <= left && past) {
        __builtin_nontemporal_store(w, reinterpret_cast<Words*>(p + at(u)));
      } else if (at(u) + 16 <= left) {
        *reinterpret_cast<Words*>(p + at(u)) = w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t lo = static_cast<uint16_t>(d[u][i]), hi = static_cast<uint16_t>(d[u][i] >> 16);
          if (at(u) + 4 * i < left) __builtin_memcpy(p + at(u) + 4 * i, &lo, 2);
          if (at(u) + 4 * i + 2 < left) __builtin_memcpy(p + at(u) + 4 * i + 2, &hi, 2);
        }
      }
    }
  }
};

__device__ inline float bits_float(uint32_t x) { return __builtin_bit_cast(float, x); }

// Sum over the workgroup's four waves, in all of its threads.
__device__ inline double group_sum(double x) {
  __shared__ double red[4];
#pragma unroll
  for (int n = 1; n < 64; n *= 2) x += __shfl_xor(x, n);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(256) void clip_squares_kernel(Batch b, double* parts) {
  double sum[2] = {};
  Walk<false> w(b);
  while (w.more()) {
    const Chunk c = w.next();
    Pieces x;
    x.load(c.in, c.left);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = x.d[u][i];
        if (c.bf16) {
          const double lo = bits_float(d << 16), hi = bits_float(d & 0xffff0000u);
          sum[0] = __builtin_fma(lo, lo, sum[0]);
          sum[1] = __builtin_fma(hi, hi, sum[1]);
        } else {
          const double f = bits_float(d);
          sum[i & 1] = __builtin_fma(f, f, sum[i & 1]);
        }
      }
  }
  const double all = group_sum(sum[0] + sum[1]);
  if (threadIdx.x == 0) parts[blockIdx.x] = all;
}

// The norm of all parts, the same in every workgroup: each thread's in order, eight loads in flight.
__device__ inline float norm_of(const double* parts, int n) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256 * 8) {
    double x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = parts[min(i + 256 * u, n - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + 256 * u < n) s += x[u];
  }
  return static_cast<float>(sqrt(group_sum(s)));
}

__global__ __launch_bounds__(256) void clip_norm_kernel(const double* parts, int n, float* norm, float* copy) {
  const float all = norm_of(parts, n);
  if (threadIdx.x != 0) return;
  *norm = all;
  *copy = all;
}

__global__ __launch_bounds__(256) void clip_scale_kernel(Batch b, ScaleArgs a) {
  Walk<true> w(b);
  Chunk c = w.next();  // every workgroup has one
  Pieces x;
  // A workgroup's only chunk is on its way while the norm is found; of several, one
  // that stays where it is would be read for nothing.
  const bool early = !w.more();
  if (early) x.load(c.in, c.left);
  const float norm = a.n_parts > 0 ? norm_of(a.parts, a.n_parts) : *a.norm;
  if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *a.write_norm = norm;
  const double share = static_cast<double>(a.max_norm) / (static_cast<double>(norm) + static_cast<double>(a.eps));
  const float by = a.max_norm == __builtin_inff() || share >= 1.0 ? 1.0f : static_cast<float>(share);
  const bool stay = by == 1.0f;
  if (stay && b.in_place) return;
  for (;; c = w.next()) {
    if (!stay || c.in != c.out) {
      if (!early) x.load(c.in, c.left);
      if (!stay) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t& d = x.d[u][i];
            if (c.bf16) {
              const __bf16 lo = static_cast<__bf16>(by * bits_float(d << 16));
              const __bf16 hi = static_cast<__bf16>(by * bits_float(d & 0xffff0000u));
              d = __builtin_bit_cast(uint16_t, lo) | static_cast<uint32_t>(__builtin_bit_cast(uint16_t, hi)) << 16;
            } else {
              d = __builtin_bit_cast(uint32_t, by * bits_float(d));
            }
          }
      }
      x.store(c.out, c.left, a.past);
    }
    if (!w.more()) break;
  }
}

}  // namespace
}  // namespace fconv

struct fconv_clip_plan_s {
  fconv_clip_tensor* tensors = nullptr;
  int32_t n = 0;
  float eps = 0.0f;
  int32_t parts = 0;  // sums of all launches
  size_t bytes = 0;   // of the sums, and the norm behind them
  int64_t total = 0;  // bytes of all tensors
  ~fconv_clip_plan_s() { delete[] tensors; }
};

namespace fconv {
namespace {

constexpr int64_t kMaxNumel = 1ll << 40, kMaxTotal = 1ll << 43;
constexpr int32_t kMaxTensors = 1 << 20;
constexpr int64_t kCacheBytes = 256ll << 20;  // the last-level cache

int elem_size(const fconv_clip_tensor& t) { return t.dtype == FCONV_BF16 ? 2 : 4; }
int64_t chunks_of(const fconv_clip_tensor& t) { return ceil_div(t.numel * elem_size(t), kChunkBytes); }
int32_t groups_of(int64_t chunks) { return static_cast<int32_t>(chunks < kGroups ? chunks : kGroups); }

// f(first tensor, number of tensors, chunks) for each launch, until it returns false.
template <typename F>
void each_batch(const fconv_clip_plan_s* p, F f) {
  for (int32_t i = 0; i < p->n;) {
    const int32_t from = i;
    int32_t live = 0;  // tensors without elements are in no launch
    int64_t chunks = 0;
    for (; i < p->n && live < kBatch; ++i) {
      const int64_t c = chunks_of(p->tensors[i]);
      if (live && chunks + c > INT32_MAX) break;
      live += c > 0;
      chunks += c;
    }
    if (live && !f(from, i - from, chunks)) return;
  }
}

void fill(Batch& b, const fconv_clip_plan_s* p, const void* const* in, void* const* out, int32_t from, int32_t count) {
  b.n = 0;
  b.first[0] = 0;
  b.in_place = true;
  for (int32_t i = from; i < from + count; ++i) {
    const fconv_clip_tensor& t = p->tensors[i];
    if (t.numel == 0) continue;
    b.in[b.n] = static_cast<const char*>(in[i]);
    b.out[b.n] = out ? static_cast<char*>(out[i]) : nullptr;
    b.in_place = b.in_place && b.in[b.n] == b.out[b.n];
    b.numel[b.n] = t.dtype == FCONV_BF16 ? t.numel : -1 - t.numel;
    b.first[b.n + 1] = b.first[b.n] + static_cast<int32_t>(chunks_of(t));
    ++b.n;
  }
}

hipError_t run(const fconv_clip_plan_s* p, const fconv_clip_args* a, bool clip, hipStream_t s) {
  Batch b;
  hipError_t e = hipSuccess;
  double* parts = static_cast<double*>(a->workspace);
  const bool given = clip && a->given_norm;
  int32_t n = 0;
  if (!given)
    each_batch(p, [&](int32_t from, int32_t count, int64_t chunks) {
      fill(b, p, a->in, nullptr, from, count);
      const int32_t groups = groups_of(chunks);
      hipLaunchKernelGGL(clip_squares_kernel, dim3(groups), dim3(256), 0, s, b, parts + n);
      n += groups;
      return (e = hipGetLastError()) == hipSuccess;
    });
  if (e != hipSuccess) return e;
  ScaleArgs c = {};
  c.max_norm = a->max_norm;
  c.eps = p->eps;
  c.past = p->total > kCacheBytes;
  if (given) {
    c.norm = a->given_norm;
  } else if (!clip || n == 0 || n > kOwnParts) {
    float* own = reinterpret_cast<float*>(parts + p->parts);
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(256), 0, s, parts, n, own, a->norm);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    c.norm = own;
  } else {
    c.parts = parts;
    c.n_parts = n;
    c.write_norm = a->norm;
  }
  if (clip)
    each_batch(p, [&](int32_t from, int32_t count, int64_t chunks) {
      fill(b, p, a->in, a->out, from, count);
      hipLaunchKernelGGL(clip_scale_kernel, dim3(groups_of(chunks)), dim3(256), 0, s, b, c);
      c.write_norm = nullptr;
      return (e = hipGetLastError()) == hipSuccess;
    });
  return e;
}

struct Extent {
  uintptr_t from, to;
  bool written;
};

fconv_status check(const fconv_clip_plan_s* p, const fconv_clip_args* a, bool clip) {
  if (!p || !a || (p->n && !a->in)) return FCONV_ERR_INVALID_ARG;
  const bool given = clip && a->given_norm;
  if (!given && !a->norm) return FCONV_ERR_INVALID_ARG;
  if (clip && ((p->n && !a->out) || !(a->max_norm >= 0.0f))) return FCONV_ERR_INVALID_ARG;
  if (!given && (!a->workspace || a->workspace_bytes < p->bytes)) return FCONV_ERR_WORKSPACE;
  for (int32_t i = 0; i < p->n; ++i) {
    const fconv_clip_tensor& t = p->tensors[i];
    if (t.numel && (!a->in[i] || (clip && !a->out[i]))) return FCONV_ERR_INVALID_ARG;
  }
  if (given ? !aligned(a->given_norm, 4) : !aligned(a->norm, 4) || !aligned(a->workspace, 16)) return FCONV_ERR_MISALIGNED;
  for (int32_t i = 0; i < p->n; ++i) {
    const fconv_clip_tensor& t = p->tensors[i];
    if (t.numel && (!aligned(a->in[i], elem_size(t)) || (clip && !aligned(a->out[i], elem_size(t)))))
      return FCONV_ERR_MISALIGNED;
  }
  // In the order of their beginnings, a range meets one before it if it begins before that one's end.
  Extent few[520];
  const int64_t most = 2ll * p->n + 2;
  Extent* x = most <= 520 ? few : new (std::nothrow) Extent[most];
  if (!x) return FCONV_ERR_INVALID_ARG;
  int64_t n = 0;
  auto add = [&](const void* at, size_t bytes, bool written) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(at);
    x[n++] = Extent{from, from + bytes, written};
  };
  for (int32_t i = 0; i < p->n; ++i) {
    const fconv_clip_tensor& t = p->tensors[i];
    if (t.numel == 0) continue;
    const size_t bytes = static_cast<size_t>(t.numel) * elem_size(t);
    const bool in_place = clip && a->in[i] == a->out[i];
    add(a->in[i], bytes, in_place);
    if (clip && !in_place) add(a->out[i], bytes, true);
  }
  if (given) {
    add(a->given_norm, 4, false);
  } else {
    add(a->norm, 4, true);
    add(a->workspace, p->bytes, true);
  }
  std::sort(x, x + n, [](const Extent& l, const Extent& r) { return l.from < r.from; });
  fconv_status st = FCONV_OK;
  uintptr_t any = 0, written = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (x[i].from < (x[i].written ? any : written)) st = FCONV_ERR_INVALID_ARG;
    any = std::max(any, x[i].to);
    if (x[i].written) written = std::max(written, x[i].to);
  }
  if (x != few) delete[] x;
  return st;
}

}  // namespace
}  // namespace fconv

extern "C" {

fconv_status fconv_clip_plan_create(const fconv_clip_tensor* tensors, int32_t n, float eps, fconv_clip_plan* out) {
  using namespace fconv;
  if (!out) return FCONV_ERR_INVALID_ARG;
  *out = nullptr;
  if (n < 0 || (n && !tensors) || !(eps >= 0.0f) || !std::isfinite(eps)) return FCONV_ERR_INVALID_ARG;
  if (n > kMaxTensors) return FCONV_ERR_UNSUPPORTED;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].dtype != FCONV_BF16 && tensors[i].dtype != FCONV_FP32) return FCONV_ERR_UNSUPPORTED;
    if (tensors[i].numel < 0) return FCONV_ERR_INVALID_ARG;
    if (tensors[i].numel > kMaxNumel || (total += tensors[i].numel) > kMaxTotal) return FCONV_ERR_UNSUPPORTED;
  }
  fconv_clip_plan_s* p = new (std::nothrow) fconv_clip_plan_s();
  if (!p) return FCONV_ERR_INVALID_ARG;
  p->tensors = new (std::nothrow) fconv_clip_tensor[n > 0 ? n : 1];
  if (!p->tensors) {
    delete p;
    return FCONV_ERR_INVALID_ARG;
  }
  for (int32_t i = 0; i < n; ++i) p->tensors[i] = tensors[i];
  p->n = n;
  p->eps = eps;
  each_batch(p, [&](int32_t, int32_t, int64_t chunks) {
    p->parts += groups_of(chunks);
    p->total += chunks * kChunkBytes;
    return true;
  });
  p->bytes = static_cast<size_t>(p->parts) * 8 + 16;
  *out = p;
  return FCONV_OK;
}

fconv_status fconv_clip_plan_workspace_size(fconv_clip_plan p, size_t* bytes) {
  if (!p || !bytes) return FCONV_ERR_INVALID_ARG;
  *bytes = p->bytes;
  return FCONV_OK;
}

fconv_status fconv_clip_plan_tensors(fconv_clip_plan p, const fconv_clip_tensor** tensors, int32_t* n) {
  if (!p || !tensors || !n) return FCONV_ERR_INVALID_ARG;
  *tensors = p->tensors;
  *n = p->n;
  return FCONV_OK;
}

fconv_status fconv_clip_plan_norm(fconv_clip_plan p, void* stream, const fconv_clip_args* a) {
  using namespace fconv;
  const fconv_status st = check(p, a, false);
  if (st != FCONV_OK) return st;
  return run(p, a, false, as_stream(stream)) == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_clip_plan_clip(fconv_clip_plan p, void* stream, const fconv_clip_args* a) {
  using namespace fconv;
  const fconv_status st = check(p, a, true);
  if (st != FCONV_OK) return st;
  return run(p, a, true, as_stream(stream)) == hipSuccess ? FCONV_OK : FCONV_ERR_DEVICE;
}

fconv_status fconv_clip_plan_destroy(fconv_clip_plan p) {
  delete p;
  return FCONV_OK;
}

}  // extern "C"
