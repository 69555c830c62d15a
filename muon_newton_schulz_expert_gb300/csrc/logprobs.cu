// Log probabilities of given tokens with entropy and top alternatives, and the
// gradient they send into the logits (HBM-bound).
//
//   lse = log sum_v exp x_v,  logp = x_token - lse,  entropy = lse - sum_v p_v x_v
//   dx_v = dlogp (1[v = token] - p_v) - dentropy p_v (x_v - lse + entropy)
//
// Forward: one pass over a row with the running maximum m, sum of e = exp(x - m)
// and sum of e (x - m); the entropy is log(sum e) - sum e (x - m) / sum e, which
// has no cancellation against large logits.  A row is taken by one block or,
// when there are few rows, by a cluster of up to 8 blocks whose sums and top
// lists the first block reads through distributed shared memory: one launch
// and no workspace.  The top list of a warp is a sorted list of 32 keys, one
// per lane; an element costs a compare against the list's last place unless it
// enters.  A key holds the value's order and the complemented index, so equal
// values keep the lowest index first, and NaN counts as the largest.
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace muon {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
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

// Running softmax sums: m the maximum (never below the lowest finite value, so
// that x - m is -inf and not NaN for x = -inf), s = sum e, w = sum e (x - m).
struct Sums {
  float m, s, w;
};

__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = a.m - r.m, db = b.m - r.m, ea = exp2f(da * kLog2e), eb = exp2f(db * kLog2e);
  r.s = a.s * ea + b.s * eb;
  // (x - r.m) = (x - a.m) + da; an empty or vanished part adds nothing
  r.w = (ea > 0.f ? ea * fmaf(a.s, da, a.w) : 0.f * a.w) + (eb > 0.f ? eb * fmaf(b.s, db, b.w) : 0.f * b.w);
  return r;
}

// Adds N values.  A NaN, or +inf, makes s and w NaN (x - m is NaN); a masked
// -inf adds zero to both.
template <int N>
__device__ __forceinline__ float add_values(Sums &a, const float (&x)[N]) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  if (top > a.m) {
    const float d = a.m - top, e = exp2f(d * kLog2e);
    a.w = a.s > 0.f ? e * fmaf(a.s, fmaxf(d, -1e30f), a.w) : a.w;
    a.s *= e;
    a.m = top;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = x[i] - a.m, e = exp2f(t * kLog2e);
    a.s += e;
    a.w = fmaf(e, fmaxf(t, -1e30f), a.w);
  }
  return top;
}

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

// A warp's list: lane i holds the i-th largest key, `last` the key in place
// top - 1 and `bound` its value.
struct TopList {
  uint64_t key = 0, last = 0;
  float bound = -INFINITY;
  int top;

  __device__ void offer(uint64_t k, bool wanted, int lane) {
    uint32_t who = __ballot_sync(0xffffffffu, wanted && k > last);
    while (who) {
      const int src = __ffs(who) - 1;
      const uint64_t k2 = __shfl_sync(0xffffffffu, k, src);
      const int at = __popc(__ballot_sync(0xffffffffu, key > k2));
      const uint64_t up = __shfl_up_sync(0xffffffffu, key, 1);
      if (lane == at) key = k2;
      if (lane > at) key = up;
      last = __shfl_sync(0xffffffffu, key, top - 1);
      who = __ballot_sync(0xffffffffu, wanted && k > last) & (0xfffffffeu << src);
    }
    bound = last ? key_value(last) : -INFINITY;
  }

  // The 32 largest of this list and another sorted one (lane i holds its i-th
  // key): element-wise maxima of one against the other reversed are those 32
  // in bitonic order, which five exchanges sort.
  __device__ void merge(uint64_t other, int lane) {
    const uint64_t rev = __shfl_sync(0xffffffffu, other, 31 - lane);
    key = key > rev ? key : rev;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t q = __shfl_xor_sync(0xffffffffu, key, o);
      key = ((lane & o) == 0) == (key > q) ? key : q;
    }
  }
};

struct FwdArgs {
  const void *logits;
  const int64_t *tokens;
  int64_t stride;
  float *logp, *entropy, *lse, *top_logp;
  int64_t *top_ids;
  int vocab, top;
  unsigned *err;
};

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const __grid_constant__ FwdArgs a, int split) {
  __shared__ Sums sums[kWarps];
  __shared__ uint64_t lists[kWarps][32];
  constexpr int N = kVec<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x / split;
  const int part = blockIdx.x % split;   // the block's rank in its cluster
  const T *x = static_cast<const T *>(a.logits) + row * a.stride;
  // Elements before the first 16-byte boundary, whole vectors, the rest.
  int head = (int)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T));
  if (head > a.vocab) head = a.vocab;
  const int vecs = (a.vocab - head) / N, tail0 = head + vecs * N;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
  const int v0 = (int)((int64_t)vecs * part / split), v1 = (int)((int64_t)vecs * (part + 1) / split);
  Sums acc{kLowest, 0.f, 0.f};
  TopList list;
  if (TOP) list.top = a.top;
  constexpr int U = 4;   // vectors in flight per thread
  for (int v = v0 + warp * 32 * U; v < v1; v += kThreads * U) {
    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = v + i * 32 + lane;
      if (k < v1) raw[i] = __ldcs(xv + k);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = v + i * 32 + lane;
      const bool in = k < v1;
      float f[N];
      unpack<T>(raw[i], f);
      if (!TOP) {
        if (in) add_values<N>(acc, f);
        continue;
      }
      bool some = false;
      if (in) {
        add_values<N>(acc, f);
#pragma unroll
        for (int j = 0; j < N; ++j) some |= !(f[j] < list.bound);
      }
      if (__any_sync(0xffffffffu, some))
#pragma unroll
        for (int j = 0; j < N; ++j)
          list.offer(top_key(f[j], (uint32_t)(head + k * N + j)), in && !(f[j] < list.bound), lane);
    }
  }
  if (warp == 0 && part == 0) {   // fewer than 2 * N elements outside the vectors
    for (int pass = 0; pass < 2; ++pass) {
      const int k = pass ? tail0 + lane : lane, end = pass ? a.vocab : head;
      const bool in = k < end;
      const float f[1] = {in ? to_f(x[k]) : 0.f};
      if (in) add_values<1>(acc, f);
      if (TOP) list.offer(top_key(f[0], (uint32_t)k), in, lane);
    }
  }
  // the block's sums and list
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Sums other{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o),
                     __shfl_xor_sync(0xffffffffu, acc.w, o)};
    acc = join(acc, other);
  }
  if (lane == 0) sums[warp] = acc;
  if (TOP) lists[warp][lane] = list.key;
  __syncthreads();
  if (TOP) {
    for (int n = kWarps / 2; n; n >>= 1) {
      if (warp < n) {
        list.merge(lists[warp + n][lane], lane);
        lists[warp][lane] = list.key;
      }
      __syncthreads();
    }
  }
  if (warp == 0) {
    acc = lane < kWarps ? sums[lane] : Sums{kLowest, 0.f, 0.f};
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) {
      const Sums other{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o),
                       __shfl_xor_sync(0xffffffffu, acc.w, o)};
      acc = join(acc, other);
    }
    if (lane == 0) sums[0] = acc;
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
          list.merge(k, lane);
        }
      }
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
  if (part != 0 || warp != 0) return;
  acc = {__shfl_sync(0xffffffffu, acc.m, 0), __shfl_sync(0xffffffffu, acc.s, 0), __shfl_sync(0xffffffffu, acc.w, 0)};
  // a row whose mask leaves nothing (s = 0): lse = -inf, logp = -inf, entropy = 0
  const float ls = logf(acc.s), lse = acc.s == 0.f ? -INFINITY : acc.m + ls;
  if (lane == 0) {
    const int64_t token = a.tokens ? a.tokens[row] : -1;
    if (a.lse) a.lse[row] = lse;
    if (a.entropy) a.entropy[row] = acc.s == 0.f ? 0.f : ls - acc.w / acc.s;
    if (a.logp) {
      float lp = 0.f;
      if (token >= a.vocab) {
        atomicOr(a.err, kErrDevice);
        lp = __uint_as_float(0x7fffffffu);
      } else if (token >= 0) {
        lp = acc.s == 0.f ? -INFINITY : (to_f(x[token]) - acc.m) - ls;
      }
      a.logp[row] = lp;
    }
  }
  if (TOP && lane < a.top) {
    const float v = key_value(list.key);
    a.top_ids[row * a.top + lane] = (int64_t)(uint32_t)~(uint32_t)list.key;
    if (a.top_logp) a.top_logp[row * a.top + lane] = acc.s == 0.f ? -INFINITY : (v - acc.m) - ls;
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
    const float t = x - lse, p = exp2f(t * kLog2e);
    // p (x - lse + entropy) is zero where p is (x = -inf)
    return -p * fmaf(dent, fmaxf(t, -1e30f) + ent, dlogp);
  }
};

template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_backward_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int N = kVec<T>;
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
  for (int v = threadIdx.x; v < vecs; v += 256 * U) {
    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v + i * 256 < vecs) raw[i] = __ldcs(xv + v + i * 256);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = v + i * 256;
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
  for (int i = threadIdx.x; i < rest; i += 256) {
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
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3((unsigned)(rows * split));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_before(kTraceLogprobs, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOP>, a, split);
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
  if (reinterpret_cast<uintptr_t>(logits) % (type == MUON_BF16 ? 2 : 4)) return MUON_ERR_UNSUPPORTED;
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
  if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(dlogits) % es)
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
    if (type == MUON_BF16) token_logprobs_backward_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(b);
    else token_logprobs_backward_kernel<float><<<grid, 256, 0, s>>>(b);
    const int st = trace_after(kTraceLogprobsBwd, s);
    if (st != MUON_OK) return st;
  }
  return MUON_OK;
}

}  // extern "C"
