// Log probabilities of given tokens with entropy and top alternatives, and the
// gradient they send into the logits (HBM-bound).
//
//   lse = log sum_v exp x_v,  logp = x_token - lse,  entropy = lse - sum_v p_v x_v
//   dx_v = dlogp (1[v = token] - p_v) - dentropy p_v (x_v - lse + entropy)
//
// Forward: one pass over a row with a running reference m, the sum of e =
// exp(x - m) and the sum of e (x - m); entropy = log(sum e) - sum e (x - m) /
// sum e, which has no cancellation against large logits.  An element costs a
// difference, a product with log2(e), an exponential and two accumulations,
// all but the exponential in pairs (f32x2).  m moves only when an element
// passes it by 11 (a factor 2^16, far from fp32's range), so that threads
// hardly ever rescale.  A row is taken by one block or, when there are few
// rows, by a cluster of up to 8 blocks whose sums and top lists the first block
// reads through distributed shared memory: one launch and no workspace.
//
// Top alternatives: the pass also keeps each thread's maximum.  The top-th
// largest of a block's thread maxima bounds its top-th largest element from
// below, so the vectors of the few threads that reach that bound are read again
// (from L2) for the elements at or above it, which are sorted.  Where more than kCandidates reach
// it (ties), warps keep sorted lists of 32 keys instead, one per lane.  A key
// holds the value's order and the complemented index, so equal values keep the
// lowest index first, and NaN counts as the largest.
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace muon {
namespace {

// Threads of a block: as few as leave each of them 64 vectors of a row at most
// (several rows on an SM then overlap one's reductions and sorts with another's
// loads), 512 for long rows and for rows cut over a cluster.  Measured, us:
//   10218 rows of 1403 fp32, top 1    512 threads 181, 128 threads 45, 64 threads 34
//   3000 rows of 32003 fp32, top 5    512 threads 111, 128 threads 85
//   6000 rows of 65000 bf16           512 threads 152, 128 threads 127
constexpr int kThreads = 512, kMidThreads = 128, kFewThreads = 64;
constexpr int kMaxSplit = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float *d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 *d, float v) { *d = __float2bfloat16_rn(v); }

// elements of a 16-byte vector
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &x, float (&v)[kVec<T>]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  }
}

// Running softmax sums: s = sum e and w = sum e (x - m) with e = exp(x - m).  m
// starts at the lowest finite value, so that x - m is -inf and not NaN for x =
// -inf.
struct Sums {
  float m, s, w;
};

constexpr float kFar = 1e30f;   // a difference beyond which exp(-kFar) is 0 whatever it is
constexpr float kVeryLow = -0.9f * kFar;   // elements above it are as they were after clamp_vector

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// moves the reference up to m
__device__ __forceinline__ void rebase(Sums &a, float m) {
  const float d = fmaxf(a.m - m, -kFar), e = ex2(d * kLog2e);   // finite: an empty side adds 0 and not 0 * inf
  a.w = e * fmaf(a.s, d, a.w);
  a.s *= e;
  a.m = m;
}

__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m);
  rebase(b, m);
  return {m, a.s + b.s, a.w + b.w};
}

// Any values.  A NaN, or +inf, makes s and w NaN (x - m is NaN); a masked
// -inf adds zero to both.
template <int N>
__device__ void add_any(Sums &a, const float (&x)[N]) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  if (top > a.m) rebase(a, top);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = x[i] - a.m, e = ex2(t * kLog2e);
    a.s += e;
    a.w = fmaf(e, fmaxf(t, -kFar), a.w);
  }
}

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(f32x2 v, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest of a vector's elements (NaN if one is), and the elements raised
// to -kFar (about) at least, so that a masked one's x - m is finite.
template <typename T>
__device__ __forceinline__ float clamp_vector(uint4 &x) {
  if constexpr (sizeof(T) == 2) {
    constexpr uint32_t low = 0xf149f149u;   // -1e30 in bf16, twice
    x.x = max_nan_bf16x2(x.x, low), x.y = max_nan_bf16x2(x.y, low);
    x.z = max_nan_bf16x2(x.z, low), x.w = max_nan_bf16x2(x.w, low);
    const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(x.x, x.y), max_nan_bf16x2(x.z, x.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  } else {
    x.x = __float_as_uint(max_nan(__uint_as_float(x.x), -kFar));
    x.y = __float_as_uint(max_nan(__uint_as_float(x.y), -kFar));
    x.z = __float_as_uint(max_nan(__uint_as_float(x.z), -kFar));
    x.w = __float_as_uint(max_nan(__uint_as_float(x.w), -kFar));
    return max_nan(max_nan(__uint_as_float(x.x), __uint_as_float(x.y)),
                   max_nan(__uint_as_float(x.z), __uint_as_float(x.w)));
  }
}

// A thread's sums over vectors: two halves of s and w, and the reference.
template <typename T>
struct VectorSums {
  float m = kLowest, top = -INFINITY;   // top: the largest element above kVeryLow (NaN left out), -inf if there is none
  f32x2 s = 0, w = 0;

  __device__ Sums total() const {
    float s0, s1, w0, w1;
    split(s, s0, s1);
    split(w, w0, w1);
    return {m, s0 + s1, w0 + w1};
  }
  __device__ void set(const Sums &a) {
    m = a.m;
    s = pair(a.s, 0.f);
    w = pair(a.w, 0.f);
  }

  __device__ __forceinline__ void add(uint4 raw) {
    uint4 x = raw;
    const float most = clamp_vector<T>(x);
    if (most > kVeryLow) top = fmaxf(top, most);   // else all it says is that they lie below
    if (!(most <= m + 11.f) || m < -0.5f * kFar) {
      // a new reference, a NaN or infinity, or nothing but masked elements so far
      Sums a = total();
      if (most > kVeryLow && most < INFINITY) {
        if (most > m) rebase(a, most);
        set(a);
      } else {
        float v[kVec<T>];
        unpack<T>(raw, v);
        add_any(a, v);
        set(a);
        return;
      }
    }
    const f32x2 l = pair(kLog2e, kLog2e), ref = pair(-m, -m);
    float v[kVec<T>];
    unpack<T>(x, v);
#pragma unroll
    for (int i = 0; i < kVec<T>; i += 2) {
      const f32x2 d = add2(pair(v[i], v[i + 1]), ref);
      float t0, t1;
      split(mul2(d, l), t0, t1);
      const f32x2 e = pair(ex2(t0), ex2(t1));
      s = add2(s, e);
      w = fma2(e, d, w);
    }
  }
};

__device__ __forceinline__ uint64_t top_key(float x, uint32_t index) {
  x += 0.f;   // -0 and 0 are equal
  const uint32_t b = __float_as_uint(x);
  const uint32_t order = x != x ? 0xffffffffu : b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((uint64_t)order << 32) | (uint32_t)~index;
}

__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  if (o == 0xffffffffu) return __uint_as_float(0x7fffffffu);
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// a warp's keys, sorted in descending order over the lanes
__device__ __forceinline__ uint64_t sort_keys(uint64_t key, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int o = n >> 1; o; o >>= 1) {
      const uint64_t q = shfl_xor64(key, o);
      const bool larger = ((lane & o) == 0) == ((lane & n) == 0);   // the last level sorts one way: lane & 32 is 0
      key = larger == (key > q) ? key : q;
    }
  return key;
}

// The 32 largest of two sorted lists (lane i holds the i-th key of each):
// element-wise maxima of one against the other reversed are those 32 in
// bitonic order, which five exchanges sort.
__device__ __forceinline__ uint64_t merge_keys(uint64_t key, uint64_t other, int lane) {
  const uint64_t rev = __shfl_sync(0xffffffffu, other, 31 - lane);
  key = key > rev ? key : rev;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t q = shfl_xor64(key, o);
    key = ((lane & o) == 0) == (key > q) ? key : q;
  }
  return key;
}

// A warp's list: lane i holds the i-th largest key, `last` is the key in place
// top - 1.
struct TopList {
  uint64_t key = 0, last = 0;
  int top;

  __device__ void offer(uint64_t k, bool wanted, int lane) {
    wanted = wanted && k > last;
    if (!__any_sync(0xffffffffu, wanted)) return;
    key = merge_keys(key, sort_keys(wanted ? k : 0, lane), lane);
    last = __shfl_sync(0xffffffffu, key, top - 1);
  }
};

// The block's sorted list from its warps' lists, in `lists[0]`.
template <int WARPS>
__device__ __forceinline__ void merge_lists(uint64_t key, uint64_t (*lists)[32], int warp, int lane) {
  lists[warp][lane] = key;
  __syncthreads();
  for (int n = WARPS / 2; n; n >>= 1) {
    if (warp < n) {
      key = merge_keys(key, lists[warp + n][lane], lane);
      lists[warp][lane] = key;
    }
    __syncthreads();
  }
}

struct FwdArgs {
  const void *logits;
  const int64_t *tokens;
  int64_t stride;
  float *logp, *entropy, *lse, *top_logp;
  int64_t *top_ids;
  int vocab, top;
  unsigned *err;
};

template <typename T, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS) token_logprobs_kernel(const __grid_constant__ FwdArgs a, int split) {
  constexpr int kWarps = THREADS / 32, kCandidates = 64 * kWarps;   // two sorts of 32 keys per warp
  __shared__ Sums sums[kWarps];
  __shared__ uint64_t lists[TOP ? kWarps : 1][32];
  __shared__ uint64_t found[TOP ? kCandidates : 1];
  __shared__ int count;
  constexpr int N = kVec<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x / split;
  const int part = blockIdx.x % split;   // the block's rank in its cluster
  const T *x = static_cast<const T *>(a.logits) + row * a.stride;
  // Elements before the first 16-byte boundary, whole vectors, the rest: the
  // first block of a row takes the ragged ends, one element a thread.
  int head = (int)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T));
  if (head > a.vocab) head = a.vocab;
  const int vecs = (a.vocab - head) / N, tail0 = head + vecs * N;
  const int ends = part == 0 ? head + (a.vocab - tail0) : 0;   // fewer than 2 N, one warp's
  const int end_at = (int)threadIdx.x < head ? (int)threadIdx.x : tail0 + (int)threadIdx.x - head;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
  const int v0 = (int)((int64_t)vecs * part / split), v1 = (int)((int64_t)vecs * (part + 1) / split);
  if (TOP && threadIdx.x == 0) count = 0;
  VectorSums<T> mine;
  constexpr int U = 4;   // vectors in flight per thread
  // The next vectors are on their way while these are added.
  auto fetch = [&](int v) { return TOP ? __ldg(xv + v) : __ldcs(xv + v); };
  int v = v0 + threadIdx.x;
  uint4 next[U];
  const bool full = v + (U - 1) * THREADS < v1;
  if (full)
#pragma unroll
    for (int i = 0; i < U; ++i) next[i] = fetch(v + i * THREADS);
  for (; v + (U - 1) * THREADS < v1; v += THREADS * U) {
    uint4 raw[U];
    const bool more = v + (2 * U - 1) * THREADS < v1;
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = next[i];
    if (more)
#pragma unroll
      for (int i = 0; i < U; ++i) next[i] = fetch(v + (U + i) * THREADS);
#pragma unroll
    for (int i = 0; i < U; ++i) mine.add(raw[i]);
  }
  for (; v < v1; v += THREADS) mine.add(fetch(v));
  Sums acc = mine.total();
  if ((int)threadIdx.x < ends) {
    const float f[1] = {to_f(x[end_at])};
    add_any(acc, f);
    // by the vectors' rule: an exact maximum beside theirs, which leave very low elements
    // out, could put the bound below above elements of threads that do not reach it
    if (f[0] > kVeryLow) mine.top = fmaxf(mine.top, f[0]);
  }
  const bool odd = !(acc.s == acc.s);   // this thread met a NaN or +inf
  // the block's sums
#pragma unroll
  for (int o = 16; o; o >>= 1)
    acc = join(acc, Sums{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o),
                         __shfl_xor_sync(0xffffffffu, acc.w, o)});
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (warp == 0) {
    acc = lane < kWarps ? sums[lane] : Sums{kLowest, 0.f, 0.f};
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1)
      acc = join(acc, Sums{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o),
                           __shfl_xor_sync(0xffffffffu, acc.w, o)});
    if (lane == 0) sums[0] = acc;
  }
  uint64_t key = 0;
  if (TOP) {
    // a lower bound of the block's top-th element: the top-th of its threads'
    // maxima, taken before any element of that value (index bits 0)
    const bool any = v0 + (int)threadIdx.x < v1 || (int)threadIdx.x < ends;
    merge_lists<kWarps>(sort_keys(any ? top_key(mine.top, 0xffffffffu) : 0, lane), lists, warp, lane);
    const uint64_t bound = lists[0][a.top - 1];
    const float least = key_value(bound);
    if (bound) {
      // Only a thread whose maximum reaches the bound (or that met a NaN) has
      // candidates.  Its vectors are read again: by itself where they are few,
      // else by its warp, 32 at a time.
      auto candidates = [&](int v) {
        float f[N];
        unpack<T>(__ldg(xv + v), f);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (!(f[j] < least)) {
            const int at = atomicAdd(&count, 1);
            if (at < kCandidates) found[at] = top_key(f[j], (uint32_t)(head + v * N + j));
          }
      };
      const bool reaches = any && (!(mine.top < least) || odd);
      if (v1 - v0 <= 4 * THREADS) {
        if (reaches)
          for (int v = v0 + threadIdx.x; v < v1; v += THREADS) candidates(v);
      } else {
        uint32_t who = __ballot_sync(0xffffffffu, reaches);
        while (who && *reinterpret_cast<volatile int *>(&count) <= kCandidates) {
          const int owner = warp * 32 + __ffs(who) - 1;
          who &= who - 1;
          for (int v = v0 + owner + lane * THREADS; v < v1; v += 32 * THREADS) candidates(v);
        }
      }
      if ((int)threadIdx.x < ends) {
        const float f = to_f(x[end_at]);
        if (!(f < least)) {
          const int at = atomicAdd(&count, 1);
          if (at < kCandidates) found[at] = top_key(f, (uint32_t)end_at);
        }
      }
    }
    __syncthreads();
    const int n = count;
    if (bound && n <= kCandidates) {
      const int at = warp * 64 + lane;
      if (warp * 64 < n) key = sort_keys(at < n ? found[at] : 0, lane);
      if (warp * 64 + 32 < n) key = merge_keys(key, sort_keys(at + 32 < n ? found[at + 32] : 0, lane), lane);
    } else {
      TopList list;
      list.top = a.top;
      for (int v = v0 + warp * 32; v < v1; v += THREADS) {
        const bool in = v + lane < v1;
        float f[N];
        unpack<T>(in ? __ldg(xv + v + lane) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
        for (int j = 0; j < N; ++j) list.offer(top_key(f[j], (uint32_t)(head + (v + lane) * N + j)), in, lane);
      }
      if (warp == 0) {
        const bool in = lane < ends;
        list.offer(top_key(in ? to_f(x[end_at]) : 0.f, (uint32_t)end_at), in, lane);
      }
      key = list.key;
    }
    merge_lists<kWarps>(key, lists, warp, lane);
    if (warp == 0) key = lists[0][lane];
  }
  if (split > 1) {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (part == 0 && warp == 0) {
      for (int r = 1; r < split; ++r) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at)
                     : "r"((uint32_t)__cvta_generic_to_shared(&sums[0])), "r"(r));
        Sums other;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other.m) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other.s) : "r"(at + 4) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other.w) : "r"(at + 8) : "memory");
        acc = join(acc, other);
        if (TOP) {
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(at)
                       : "r"((uint32_t)__cvta_generic_to_shared(&lists[0][lane])), "r"(r));
          uint64_t k;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(at) : "memory");
          key = merge_keys(key, k, lane);
        }
      }
    }
    // no block leaves while the first may still read its shared memory
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
  if (part != 0 || warp != 0) return;
  acc = {__shfl_sync(0xffffffffu, acc.m, 0), __shfl_sync(0xffffffffu, acc.s, 0), __shfl_sync(0xffffffffu, acc.w, 0)};
  // a row whose mask leaves nothing (s = 0): lse = -inf, logp = -inf, entropy = 0
  const bool none = acc.s == 0.f;
  const float ls = logf(acc.s), lse = none ? -INFINITY : acc.m + ls;
  if (lane == 0) {
    const int64_t token = a.tokens ? a.tokens[row] : -1;
    if (a.lse) a.lse[row] = lse;
    if (a.entropy) a.entropy[row] = none ? 0.f : ls - acc.w / acc.s;
    if (a.logp) {
      float lp = 0.f;
      if (token >= a.vocab) {
        atomicOr(a.err, kErrDevice);
        lp = __uint_as_float(0x7fffffffu);
      } else if (token >= 0) {
        lp = none ? -INFINITY : (to_f(x[token]) - acc.m) - ls;
      }
      a.logp[row] = lp;
    }
  }
  if (TOP && lane < a.top) {
    a.top_ids[row * a.top + lane] = (int64_t)(uint32_t)~(uint32_t)key;
    if (a.top_logp) a.top_logp[row * a.top + lane] = none ? -INFINITY : (key_value(key) - acc.m) - ls;
  }
}

struct BwdArgs {
  const void *logits;
  const int64_t *tokens;
  const float *lse, *entropy, *dlogp, *dentropy;
  void *dlogits;
  int64_t stride, out_stride;
  int vocab, chunk;   // elements of a row per block
  unsigned *err;
};

struct Slope {
  float lse, dlogp, dent, ent;
  __device__ float operator()(float x) const {
    const float t = x - lse, p = ex2(t * kLog2e);
    // p (x - lse + entropy) is zero where p is: below t = -88 p is, and a t no lower than -128
    // keeps the other factor finite, whatever dentropy is scaled by
    return -p * fmaf(dent, fmaxf(t, -128.f) + ent, dlogp);
  }
};

template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_backward_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int N = kVec<T>;
  const int threads = blockDim.x;
  const int64_t row = blockIdx.y;
  const T *x = static_cast<const T *>(a.logits) + row * a.stride;
  T *out = static_cast<T *>(a.dlogits) + row * a.out_stride;
  const int64_t token = a.tokens ? a.tokens[row] : -1;
  Slope f;
  f.lse = a.lse[row];
  f.dlogp = a.dlogp && token >= 0 ? a.dlogp[row] : 0.f;
  f.dent = a.dentropy ? a.dentropy[row] : 0.f;
  f.ent = a.dentropy ? a.entropy[row] : 0.f;
  if (token >= a.vocab && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.err, kErrDevice);
  // a row whose mask leaves nothing, and one with nothing to send, get zeros
  const bool none = f.lse == -INFINITY || (f.dlogp == 0.f && f.dent == 0.f);
  const int c0 = blockIdx.x * a.chunk, c1 = min(a.vocab, c0 + a.chunk);
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x + c0), oa = reinterpret_cast<uintptr_t>(out + c0);
  int head = c1 - c0, vecs = 0;   // where the two rows lie differently to 16 bytes: element by element
  if (((xa ^ oa) & 15) == 0) {
    head = min(c1 - c0, (int)(((16 - (xa & 15)) & 15) / sizeof(T)));
    vecs = (c1 - c0 - head) / N;
  }
  const int v0 = c0 + head, tail0 = v0 + vecs * N;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + v0);
  uint4 *ov = reinterpret_cast<uint4 *>(out + v0);
  constexpr int U = 4;
  for (int v = threadIdx.x; v < vecs; v += threads * U) {
    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v + i * threads < vecs) raw[i] = __ldcs(xv + v + i * threads);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = v + i * threads;
      if (k >= vecs) break;
      float e[N];
      unpack<T>(raw[i], e);
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = none ? 0.f : f(e[j]);
      const int64_t hit = token - (v0 + (int64_t)k * N);
      if (hit >= 0 && hit < N && !none)
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (j == (int)hit) e[j] += f.dlogp;
      uint4 o;
      if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          __nv_bfloat162 h = __floats2bfloat162_rn(e[2 * j], e[2 * j + 1]);
          w[j] = *reinterpret_cast<uint32_t *>(&h);
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        o = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
      }
      __stcs(ov + k, o);
    }
  }
  // the elements before the first boundary and after the last vector
  const int rest = head + (c1 - tail0);
  for (int i = threadIdx.x; i < rest; i += threads) {
    const int k = i < head ? c0 + i : tail0 + (i - head);
    const float v = none ? 0.f : f(to_f(x[k])) + (k == token ? f.dlogp : 0.f);
    from_f(out + k, v);
  }
}

template <typename T, bool TOP>
int launch_fwd(const FwdArgs &a, int64_t rows, cudaStream_t s) {
  // Blocks per row: enough to give every SM about two, and at least 8192
  // elements each.
  int split = 1;
  while (split < kMaxSplit && rows * split < 2 * num_sms() && a.vocab >= 2 * split * 8192) split *= 2;
  const int vecs = a.vocab / kVec<T>;
  const int threads = split > 1 ? kThreads : vecs <= 16 * kFewThreads ? kFewThreads
                                         : vecs <= 64 * kMidThreads ? kMidThreads : kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)threads);
  cfg.gridDim = dim3((unsigned)(rows * split));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  trace_before(kTraceLogprobs, s);
  const cudaError_t e =
      threads == kFewThreads   ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOP, kFewThreads>, a, split)
      : threads == kMidThreads ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOP, kMidThreads>, a, split)
                               : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOP, kThreads>, a, split);
  const int st = trace_after(kTraceLogprobs, s);
  return e == cudaSuccess ? st : MUON_ERR_CUDA;
}

bool bad_type(int t) { return t != MUON_BF16 && t != MUON_F32; }
constexpr int64_t kMaxVocab = int64_t(1) << 30, kMaxRows = int64_t(1) << 27;

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_token_logprobs(const void *logits, int64_t stride, const int64_t *tokens, int64_t rows, int64_t vocab,
                        int type, float *logp, float *entropy, float *lse, int top, int64_t *top_ids, float *top_logp,
                        muon_stream_t stream) {
  if (rows < 0 || vocab < 1 || bad_type(type) || top < 0 || stride < vocab) return MUON_ERR_INVALID_ARG;
  if (top > 32 || vocab > kMaxVocab || rows > kMaxRows) return MUON_ERR_UNSUPPORTED;
  if (top > vocab) return MUON_ERR_INVALID_ARG;
  if (rows == 0) return MUON_OK;
  if ((top > 0 && !top_ids) || (top == 0 && (top_ids || top_logp))) return MUON_ERR_INVALID_ARG;
  if (!logits || (logp && !tokens) || (!logp && !entropy && !lse && !top)) return MUON_ERR_INVALID_ARG;
  if (!on_elements({logits}, type == MUON_BF16 ? 2 : 4) || !on_elements({logp, entropy, lse, top_logp}, 4) ||
      !on_elements({tokens, top_ids}, 8))
    return MUON_ERR_UNSUPPORTED;
  FwdArgs a{};
  a.logits = logits;
  a.tokens = tokens;
  a.stride = stride;
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.vocab = (int)vocab;
  a.top = top;
  a.err = device_error_word();
  if (!a.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (type == MUON_BF16)
    return top ? launch_fwd<__nv_bfloat16, true>(a, rows, s) : launch_fwd<__nv_bfloat16, false>(a, rows, s);
  return top ? launch_fwd<float, true>(a, rows, s) : launch_fwd<float, false>(a, rows, s);
}

int muon_token_logprobs_backward(const void *logits, int64_t stride, const int64_t *tokens, const float *lse,
                                 const float *entropy, const float *dlogp, const float *dentropy, int64_t rows,
                                 int64_t vocab, int type, void *dlogits, int64_t dlogits_stride, muon_stream_t stream) {
  if (rows < 0 || vocab < 1 || bad_type(type) || stride < vocab || dlogits_stride < vocab) return MUON_ERR_INVALID_ARG;
  if (vocab > kMaxVocab || rows > kMaxRows) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (!logits || !lse || !dlogits || (!dlogp && !dentropy) || (dlogp && !tokens) || (dentropy && !entropy))
    return MUON_ERR_INVALID_ARG;
  const uintptr_t es = type == MUON_BF16 ? 2 : 4;
  if (!on_elements({logits, dlogits}, es) || !on_elements({lse, entropy, dlogp, dentropy}, 4) ||
      !on_elements({tokens}, 8))
    return MUON_ERR_UNSUPPORTED;
  BwdArgs a{};
  a.logits = logits;
  a.tokens = tokens;
  a.lse = lse;
  a.entropy = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.dlogits = dlogits;
  a.stride = stride;
  a.out_stride = dlogits_stride;
  a.vocab = (int)vocab;
  a.chunk = 16384;
  a.err = device_error_word();
  if (!a.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned chunks = (unsigned)((vocab + a.chunk - 1) / a.chunk);
  // 4 vectors a thread, so that short rows do not leave most of a block idle
  const int64_t vecs = std::min<int64_t>(vocab, a.chunk) * (int64_t)es / 16;
  const unsigned threads = (unsigned)std::clamp<int64_t>((vecs / 4 + 31) / 32 * 32, 64, 256);
  // grid.y holds at most 65535 rows
  for (int64_t r = 0; r < rows; r += 65535) {
    BwdArgs b = a;
    b.logits = static_cast<const uint8_t *>(logits) + r * stride * (int64_t)es;
    b.dlogits = static_cast<uint8_t *>(dlogits) + r * dlogits_stride * (int64_t)es;
    b.tokens = tokens ? tokens + r : nullptr;
    b.lse = lse + r;
    b.entropy = entropy ? entropy + r : nullptr;
    b.dlogp = dlogp ? dlogp + r : nullptr;
    b.dentropy = dentropy ? dentropy + r : nullptr;
    const dim3 grid(chunks, (unsigned)std::min<int64_t>(65535, rows - r));
    trace_before(kTraceLogprobsBwd, s);
    if (type == MUON_BF16) token_logprobs_backward_kernel<__nv_bfloat16><<<grid, threads, 0, s>>>(b);
    else token_logprobs_backward_kernel<float><<<grid, threads, 0, s>>>(b);
    const int st = trace_after(kTraceLogprobsBwd, s);
    if (st != MUON_OK) return st;
  }
  return MUON_OK;
}

}  // extern "C"
