// Tokens to rows sorted by expert and back (HBM-bound):
//   dispatch   a stable counting sort of the T k slots by their expert; the row of a slot
//              is a copy of its token's
//   combine    out[t] = sum_j w[t][j] y[place[t][j]]   (without weights: dispatch's gradient)
//   gradient   dy[place[t][j]] = w[t][j] dout[t];  dw[t][j] = <dout[t], y[place[t][j]]>
//
// place[t][j] is the row of slot j of token t; a slot that is not routed (a negative id) has
// -1 - row instead, so that its row, one of the last, can still be given the zeros that the
// products after this read there.
//
// Every kernel goes by token: the token's own row is read once (or written once) and its k
// others meet it in registers.  Sums run over the slots in their order, in fp32.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>
#include <mutex>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace muon {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxTop = 32, kSlots = 8;     // slots of a token, and of those in registers at once
constexpr int64_t kMaxExperts = 1024, kMaxSlots = int64_t(1) << 30, kMaxHidden = int64_t(1) << 20;
// Slots that every token's block sorts for itself, in one launch: its k places need one pass over
// the ids each.
constexpr int64_t kFewSlots = 2048;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float *d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 *d, float v) { *d = __float2bfloat16_rn(v); }

// N elements that are read and written in one access
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};
template <int BYTES>
struct Raw;
template <> struct Raw<16> { typedef uint4 type; };
template <> struct Raw<8> { typedef uint2 type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<2> { typedef uint16_t type; };

template <typename T, int N>
__device__ __forceinline__ void load(float (&f)[N], const T *p) {
  typedef typename Raw<sizeof(T) * N>::type R;
  union {
    R r;
    Vec<T, N> v;
  } u;
  u.r = *reinterpret_cast<const R *>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = to_f(u.v.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store(T *p, const float (&f)[N]) {
  typedef typename Raw<sizeof(T) * N>::type R;
  union {
    R r;
    Vec<T, N> v;
  } u;
#pragma unroll
  for (int i = 0; i < N; ++i) from_f(&u.v.v[i], f[i]);
  *reinterpret_cast<R *>(p) = u.r;
}

// the expert of a slot as the sort takes it: slots that are not routed come last
__device__ __forceinline__ int key_of(int64_t id, int experts, unsigned *err) {
  if (id >= experts) atomicOr(err, kErrDevice);
  return id < 0 || id >= experts ? experts : (int)id;
}

// ---------------------------------------------------------------------------- the sort
struct OrderArgs {
  const int64_t *ids;
  int n, experts;         // slots
  int64_t *offsets, *place;
  unsigned *err;
};

// One cluster of 8 blocks of 32 warps.  Each warp takes a run of consecutive slots: first it counts
// them by expert, then, with the counts of all warps before it added up, gives them their rows in
// order, 32 at a time (lanes of one expert by their number).  Counters are whole numbers and each
// warp's own, so the order is that of the slots.  16384 tokens x 8: see the table of the operators.
constexpr int kOrderBlocks = 8, kOrderThreads = 1024, kOrderWarps = kOrderThreads / 32;

__global__ void __cluster_dims__(kOrderBlocks, 1, 1) __launch_bounds__(kOrderThreads)
    expert_order_kernel(const OrderArgs p) {
  extern __shared__ unsigned order_smem[];
  const int E = p.experts, width = E + 1;
  unsigned *hist = order_smem;                          // [kOrderWarps][width]
  unsigned *total = hist + kOrderWarps * width;         // [width], read by the other blocks
  unsigned *start = total + width;                      // [width]
  __shared__ unsigned warp_sums[kOrderWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  let_next_grid_start();
  for (int i = tid; i < kOrderWarps * width; i += kOrderThreads) hist[i] = 0u;
  __syncthreads();
  const long long runs = (long long)kOrderBlocks * kOrderWarps;
  const long long run = ((long long)p.n + 32 * runs - 1) / (32 * runs) * 32;
  const long long lo = min((long long)p.n, (rank * kOrderWarps + wp) * run), hi = min((long long)p.n, lo + run);
  unsigned *mine = hist + wp * width;
  for (long long b = lo; b < hi; b += 32) {
    const bool in = b + lane < hi;
    const int key = in ? key_of(p.ids[b + lane], E, p.err) : -1;
    const unsigned same = __match_any_sync(kAll, key);
    if (in && (same & ((1u << lane) - 1u)) == 0u) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e < width; e += kOrderThreads) {
    unsigned sum = 0u;
    for (int w = 0; w < kOrderWarps; ++w) {
      const unsigned v = hist[w * width + e];
      hist[w * width + e] = sum;
      sum += v;
    }
    total[e] = sum;
  }
  cluster.sync();
  // this thread's expert (at most kOrderThreads of them): slots of it in all blocks and in those before this one
  unsigned all = 0u, before = 0u;
  if (tid < E)
    for (int r = 0; r < kOrderBlocks; ++r) {
      const unsigned v = cluster.map_shared_rank(total, r)[tid];
      all += v;
      if (r < rank) before += v;
    }
  unsigned upto = all;
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_sums[wp] = upto;
  __syncthreads();
  unsigned first = upto - all, routed = 0u;
  for (int w = 0; w < kOrderWarps; ++w) {
    const unsigned v = warp_sums[w];
    if (w < wp) first += v;
    routed += v;
  }
  if (tid < E) {
    start[tid] = first + before;
    if (rank == 0) p.offsets[tid] = first;
  }
  if (tid == 0) {
    unsigned b = 0u;
    for (int r = 0; r < rank; ++r) b += cluster.map_shared_rank(total, r)[E];
    start[E] = routed + b;
    if (rank == 0) p.offsets[E] = p.n;   // rows of no slot count to the last expert
  }
  __syncthreads();
  for (long long b = lo; b < hi; b += 32) {
    const bool in = b + lane < hi;
    const int key = in ? key_of(p.ids[b + lane], E, p.err) : -1;
    const unsigned same = __match_any_sync(kAll, key), below = same & ((1u << lane) - 1u);
    unsigned at = 0u;
    if (in) at = start[key] + mine[key] + __popc(below);
    __syncwarp();
    if (in && below == 0u) mine[key] += __popc(same);
    __syncwarp();
    if (in) p.place[b + lane] = key < E ? (int64_t)at : -1 - (int64_t)at;
  }
  cluster.sync();   // no block leaves while another reads its totals
}

// ---------------------------------------------------------------------------- rows by token
struct RowArgs {
  const void *x;           // dispatch: the tokens' rows;  gradient: dout
  int64_t ldx;
  void *rows;              // dispatch: rows by expert;  gradient: dy;  [slots][hidden] dense
  const void *y;           // combine, gradient: rows by expert, dense
  void *out;               // combine
  int64_t ldo;
  const int64_t *place;
  const float *weights;
  float *dweights;
  int64_t tokens;
  int top, hidden, vecs;   // vecs: accesses of a row
  int tx;                  // threads of a token, a power of two
  const int64_t *ids;      // few slots: what place is made of
  int experts;
  int64_t *offsets, *place_out;
  unsigned *err;
};

// The row that a place names, or -1; `zero`: of a slot that is not routed.
__device__ __forceinline__ int64_t row_of(int64_t place, int64_t slots, bool *zero, unsigned *err) {
  *zero = place < 0;
  const int64_t r = place < 0 ? -1 - place : place;
  if (r >= slots) {
    atomicOr(err, kErrDevice);
    return -1;
  }
  return r;
}

// Copies of a token's row: one access of it a thread, written k times.
template <int BYTES>
__device__ __forceinline__ void copy_out(const RowArgs &p, int64_t token, int c, const int64_t *place) {
  typedef typename Raw<BYTES>::type R;
  const int64_t slots = p.tokens * p.top;
  const R v = reinterpret_cast<const R *>(p.x)[token * p.ldx + c];
  R *rows = reinterpret_cast<R *>(p.rows);
  for (int j = 0; j < p.top; ++j) {
    bool zero;
    const int64_t r = row_of(place[j], slots, &zero, p.err);
    if (r >= 0) rows[r * p.vecs + c] = zero ? R{} : v;
  }
}

template <int BYTES>
__global__ void __launch_bounds__(kThreads) dispatch_rows_kernel(const RowArgs p) {
  const int64_t token = blockIdx.x * (int64_t)(kThreads / p.tx) + threadIdx.x / p.tx;
  const int c = blockIdx.y * p.tx + threadIdx.x % p.tx;
  wait_for_previous_grid();
  if (token < p.tokens && c < p.vecs) copy_out<BYTES>(p, token, c, p.place + token * p.top);
}

// Few slots: a block per token finds its k places by counting, block `tokens` makes the offsets.
template <int BYTES>
__global__ void __launch_bounds__(kThreads) dispatch_few_kernel(const RowArgs p) {
  __shared__ unsigned count[kMaxExperts];
  __shared__ int64_t place[kMaxTop];
  __shared__ unsigned warp_sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, n = (int)p.tokens * p.top;
  if (blockIdx.x == p.tokens) {
    if (blockIdx.y) return;
    for (int e = tid; e < p.experts; e += kThreads) count[e] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const int key = key_of(p.ids[i], p.experts, p.err);
      if (key < p.experts) atomicAdd(&count[key], 1u);
    }
    __syncthreads();
    unsigned base = 0u;   // slots before these experts
    for (int e0 = 0; e0 < p.experts; e0 += kThreads) {
      const unsigned all = e0 + tid < p.experts ? count[e0 + tid] : 0u;
      unsigned upto = all;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += v;
      }
      if (lane == 31) warp_sums[wp] = upto;
      __syncthreads();
      unsigned first = base + upto - all;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < wp) first += warp_sums[w];
        base += warp_sums[w];
      }
      if (e0 + tid < p.experts) p.offsets[e0 + tid] = first;
      __syncthreads();
    }
    if (tid == 0) p.offsets[p.experts] = n;   // rows of no slot count to the last expert
    return;
  }
  const int token = (int)blockIdx.x;
  if (tid < p.top) count[tid] = 0u;
  __syncthreads();
  for (int j = 0; j < p.top; ++j) {
    const int slot = token * p.top + j, key = key_of(p.ids[slot], p.experts, p.err);
    unsigned before = 0u;
    for (int i = tid; i < n; i += kThreads) {
      const int k = key_of(p.ids[i], p.experts, p.err);
      before += k < key || (k == key && i < slot);
    }
    before = __reduce_add_sync(kAll, before);
    if (lane == 0 && before) atomicAdd(&count[j], before);
  }
  __syncthreads();
  if (tid < p.top) {
    const int64_t at = count[tid];
    const int64_t v = key_of(p.ids[token * p.top + tid], p.experts, p.err) < p.experts ? at : -1 - at;
    place[tid] = v;
    if (blockIdx.y == 0) p.place_out[token * p.top + tid] = v;
  }
  __syncthreads();
  const int c = blockIdx.y * kThreads + tid;
  if (c < p.vecs) copy_out<BYTES>(p, token, c, place);
}

// out[t]: one access of a row a thread, its k rows' loads in flight together
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowArgs p) {
  const int64_t token = blockIdx.x * (int64_t)(kThreads / p.tx) + threadIdx.x / p.tx;
  const int c = (blockIdx.y * p.tx + threadIdx.x % p.tx) * N;
  if (token >= p.tokens || c >= p.hidden) return;
  const T *y = static_cast<const T *>(p.y);
  const int64_t slots = p.tokens * p.top;
  const int64_t *place = p.place + token * p.top;
  const float *weights = p.weights ? p.weights + token * p.top : nullptr;
  float sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.f;
  for (int j0 = 0; j0 < p.top; j0 += kSlots) {
    float v[kSlots][N];
    bool has[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      has[j] = false;
      if (j0 + j < p.top) {
        bool zero;
        const int64_t r = row_of(__ldg(place + j0 + j), slots, &zero, p.err);
        has[j] = r >= 0 && !zero;
        if (has[j]) load<T, N>(v[j], y + r * p.hidden + c);
      }
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (has[j]) {
        const float w = weights ? __ldg(weights + j0 + j) : 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = fmaf(w, v[j][i], sum[i]);
      }
  }
  store<T, N>(static_cast<T *>(p.out) + token * p.ldo + c, sum);
}

// The gradient: a token's threads go over its row once for every kSlots slots, each access of dout
// meeting those of y; the products' sums are joined over the threads in a fixed tree.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const RowArgs p) {
  __shared__ float part[kThreads / 32][kSlots];
  const int tx = p.tx, me = threadIdx.x % tx, lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int64_t token = blockIdx.x * (int64_t)(kThreads / tx) + threadIdx.x / tx;
  const bool in = token < p.tokens;
  const T *y = static_cast<const T *>(p.y), *dout = static_cast<const T *>(p.x) + token * p.ldx;
  T *dy = static_cast<T *>(p.rows);
  const int64_t slots = p.tokens * p.top;
  for (int j0 = 0; j0 < p.top; j0 += kSlots) {
    int64_t at[kSlots];
    bool zero[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      at[j] = -1, zero[j] = true, w[j] = 1.f, dot[j] = 0.f;
      if (in && j0 + j < p.top) {
        at[j] = row_of(__ldg(p.place + token * p.top + j0 + j), slots, &zero[j], p.err);
        if (p.weights) w[j] = __ldg(p.weights + token * p.top + j0 + j);
      }
    }
    if (in)
      for (int c = me * N; c < p.hidden; c += tx * N) {
        float d[N], v[kSlots][N];
        load<T, N>(d, dout + c);
        if (p.dweights)
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (at[j] >= 0 && !zero[j]) load<T, N>(v[j], y + at[j] * p.hidden + c);
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (at[j] >= 0) {
            float o[N];
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = zero[j] ? 0.f : w[j] * d[i];
            if (dy) store<T, N>(dy + at[j] * p.hidden + c, o);
            if (p.dweights && !zero[j])
#pragma unroll
              for (int i = 0; i < N; ++i) dot[j] = fmaf(d[i], v[j][i], dot[j]);
          }
      }
    if (!p.dweights) continue;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      for (int o = min(tx, 32) / 2; o; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
    if (tx > 32) {
      __syncthreads();   // the sums before these have been read
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (lane == j) part[wp][j] = dot[j];
      __syncthreads();
      if (in && me < kSlots && j0 + me < p.top) {
        float s = 0.f;
        for (int k = 0; k < tx / 32; ++k) s += part[wp + k][me];
        p.dweights[token * p.top + j0 + me] = s;
      }
    } else if (in && me == 0) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (j0 + j < p.top) p.dweights[token * p.top + j0 + j] = dot[j];
    }
  }
}

// ---------------------------------------------------------------------------- launches
bool bad_type(int t) { return t != MUON_BF16 && t != MUON_F32; }
int size_of(int type) { return type == MUON_BF16 ? 2 : 4; }

// the widest access, in bytes, that rows of `hidden` elements at these places and strides take
int access_bytes(int size, int64_t hidden, std::initializer_list<const void *> ptrs,
                 std::initializer_list<int64_t> strides) {
  int b = 16;
  auto fits = [&] {
    for (const void *p : ptrs)
      if (reinterpret_cast<uintptr_t>(p) % b) return false;
    for (int64_t s : strides)
      if (s * size % b) return false;
    return hidden * size % b == 0;
  };
  while (b > size && !fits()) b /= 2;
  return b;
}

// threads of a token: a power of two that covers its accesses, 8 to 256
int threads_of(int vecs) {
  int t = 8;
  while (t < kThreads && t < vecs) t *= 2;
  return t;
}

template <typename F>
void with_bytes(int bytes, F &&f) {
  switch (bytes) {
    case 16: f(std::integral_constant<int, 16>()); break;
    case 8: f(std::integral_constant<int, 8>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    default: f(std::integral_constant<int, 2>()); break;
  }
}
// f(element, elements of an access)
template <typename F>
void with_vec(int type, int bytes, F &&f) {
  with_bytes(bytes, [&](auto b) {
    constexpr int B = decltype(b)::value;
    if (type == MUON_BF16) f(__nv_bfloat16(), std::integral_constant<int, B / 2>());
    else if constexpr (B >= 4) f(float(), std::integral_constant<int, B / 4>());
  });
}

int check_sizes(int64_t tokens, int64_t top, int64_t hidden, int type) {
  if (tokens < 0 || top < 1 || hidden < 1 || bad_type(type)) return MUON_ERR_INVALID_ARG;
  if (top > kMaxTop || tokens > kMaxSlots / top || hidden > kMaxHidden) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

int order(const OrderArgs &a, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  auto bytes = [](int64_t experts) { return (size_t)(kOrderWarps + 2) * (experts + 1) * sizeof(unsigned); };
  std::call_once(once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(expert_order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)bytes(kMaxExperts));
  });
  if (attr_err[dev] != cudaSuccess) return MUON_ERR_CUDA;
  trace_before(kTraceExpertOrder, s);
  expert_order_kernel<<<kOrderBlocks, kOrderThreads, bytes(a.experts), s>>>(a);
  return trace_after(kTraceExpertOrder, s);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_dispatch(const void *x, int64_t x_stride, const int64_t *ids, int64_t tokens, int64_t top, int64_t experts,
                  int64_t hidden, int type, void *rows, int64_t *offsets, int64_t *place, muon_stream_t stream) {
  const int st = check_sizes(tokens, top, hidden, type);
  if (st != MUON_OK) return st;
  if (experts < 1) return MUON_ERR_INVALID_ARG;
  if (experts > kMaxExperts) return MUON_ERR_UNSUPPORTED;
  if (!offsets) return MUON_ERR_INVALID_ARG;
  if (!on_elements({offsets}, 8)) return MUON_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) return cudaMemsetAsync(offsets, 0, (experts + 1) * 8, s) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  if (!x || !ids || !rows || !place || x_stride < hidden) return MUON_ERR_INVALID_ARG;
  const int size = size_of(type);
  if (!on_elements({x, rows}, size) || !on_elements({ids, place}, 8)) return MUON_ERR_UNSUPPORTED;
  unsigned *err = device_error_word();
  if (!err) return MUON_ERR_CUDA;
  const int bytes = access_bytes(size, hidden, {x, rows}, {x_stride});
  RowArgs p{};
  p.x = x;
  p.ldx = x_stride * size / bytes;   // in accesses
  p.rows = rows;
  p.place = place;
  p.tokens = tokens;
  p.top = (int)top;
  p.vecs = (int)(hidden * size / bytes);
  p.err = err;
  if (tokens * top <= kFewSlots) {
    p.ids = ids;
    p.experts = (int)experts;
    p.offsets = offsets;
    p.place_out = place;
    const dim3 grid((unsigned)tokens + 1, (unsigned)((p.vecs + kThreads - 1) / kThreads));
    trace_before(kTraceDispatchRows, s);
    with_bytes(bytes, [&](auto b) { dispatch_few_kernel<decltype(b)::value><<<grid, kThreads, 0, s>>>(p); });
    return trace_after(kTraceDispatchRows, s);
  }
  const int so = order({ids, (int)(tokens * top), (int)experts, offsets, place, err}, s);
  if (so != MUON_OK) return so;
  p.tx = threads_of(p.vecs);
  const int per = kThreads / p.tx;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tokens + per - 1) / per), (unsigned)((p.vecs + p.tx - 1) / p.tx));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  trace_before(kTraceDispatchRows, s);
  with_bytes(bytes, [&](auto b) { e = cudaLaunchKernelEx(&cfg, dispatch_rows_kernel<decltype(b)::value>, p); });
  const int sl = trace_after(kTraceDispatchRows, s);
  return e == cudaSuccess ? sl : MUON_ERR_CUDA;
}

int muon_combine(const void *y, const int64_t *place, const float *weights, int64_t tokens, int64_t top,
                 int64_t hidden, int type, void *out, int64_t out_stride, muon_stream_t stream) {
  const int st = check_sizes(tokens, top, hidden, type);
  if (st != MUON_OK) return st;
  if (tokens == 0) return MUON_OK;
  if (!y || !place || !out || out_stride < hidden) return MUON_ERR_INVALID_ARG;
  const int size = size_of(type);
  if (!on_elements({y, out}, size) || !on_elements({place}, 8) || !on_elements({weights}, 4))
    return MUON_ERR_UNSUPPORTED;
  const int bytes = access_bytes(size, hidden, {y, out}, {out_stride});
  RowArgs p{};
  p.y = y;
  p.out = out;
  p.ldo = out_stride;
  p.place = place;
  p.weights = weights;
  p.tokens = tokens;
  p.top = (int)top;
  p.hidden = (int)hidden;
  p.vecs = (int)(hidden * size / bytes);
  p.tx = threads_of(p.vecs);
  p.err = device_error_word();
  if (!p.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int per = kThreads / p.tx;
  const dim3 grid((unsigned)((tokens + per - 1) / per), (unsigned)((p.vecs + p.tx - 1) / p.tx));
  trace_before(kTraceCombine, s);
  with_vec(type, bytes, [&](auto t, auto n) {
    combine_kernel<decltype(t), decltype(n)::value><<<grid, kThreads, 0, s>>>(p);
  });
  return trace_after(kTraceCombine, s);
}

int muon_dispatch_backward(const void *drows, const int64_t *place, int64_t tokens, int64_t top, int64_t hidden,
                           int type, void *dx, int64_t dx_stride, muon_stream_t stream) {
  return muon_combine(drows, place, nullptr, tokens, top, hidden, type, dx, dx_stride, stream);
}

int muon_combine_backward(const void *dout, int64_t dout_stride, const void *y, const int64_t *place,
                          const float *weights, int64_t tokens, int64_t top, int64_t hidden, int type, void *dy,
                          float *dweights, muon_stream_t stream) {
  const int st = check_sizes(tokens, top, hidden, type);
  if (st != MUON_OK) return st;
  if (tokens == 0) return MUON_OK;
  if (!dout || !place || (!dy && !dweights) || (dweights && !y) || dout_stride < hidden) return MUON_ERR_INVALID_ARG;
  const int size = size_of(type);
  if (!on_elements({dout, y, dy}, size) || !on_elements({place}, 8) || !on_elements({weights, dweights}, 4))
    return MUON_ERR_UNSUPPORTED;
  const int bytes = access_bytes(size, hidden, {dout, dweights ? y : nullptr, dy}, {dout_stride});
  RowArgs p{};
  p.x = dout;
  p.ldx = dout_stride;
  p.y = y;
  p.rows = dy;
  p.place = place;
  p.weights = weights;
  p.dweights = dweights;
  p.tokens = tokens;
  p.top = (int)top;
  p.hidden = (int)hidden;
  p.vecs = (int)(hidden * size / bytes);
  p.tx = threads_of(p.vecs);
  p.err = device_error_word();
  if (!p.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int per = kThreads / p.tx;
  const unsigned blocks = (unsigned)((tokens + per - 1) / per);
  trace_before(kTraceCombineBwd, s);
  with_vec(type, bytes, [&](auto t, auto n) {
    combine_backward_kernel<decltype(t), decltype(n)::value><<<blocks, kThreads, 0, s>>>(p);
  });
  return trace_after(kTraceCombineBwd, s);
}

}  // extern "C"
