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
#include <limits.h>


#include <algorithm>
#include <type_traits>
#include <mutex>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace muon {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxTop = 32;     // slots of a token
constexpr int64_t kMaxExperts = 1024, kMaxSlots = int64_t(1) << 30, kMaxHidden = int64_t(1) << 20;
// Slots that every token's block sorts for itself, in one launch: its places need one look at all ids each.  64, 256
// and 512 tokens of 6144 bf16, 4 slots each: 3.5, 5.3 and 8.2 us, against 8.5, 12.6 and 14.3 us with the sort in a launch
// of its own; the looks grow with the square.
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
using Access = typename Raw<sizeof(T) * N>::type;

template <typename T, int N>
__device__ __forceinline__ Access<T, N> load(const T *p) {
  return *reinterpret_cast<const Access<T, N> *>(p);
}
// rows that nothing reads again
template <typename T, int N>
__device__ __forceinline__ Access<T, N> load_once(const T *p) {
  return __ldcs(reinterpret_cast<const Access<T, N> *>(p));
}
template <typename T, int N>
__device__ __forceinline__ void unpack(float (&f)[N], const Access<T, N> &r) {
  union {
    Access<T, N> r;
    Vec<T, N> v;
  } u;
  u.r = r;
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = to_f(u.v.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store(T *p, const float (&f)[N]) {
  union {
    Access<T, N> r;
    Vec<T, N> v;
  } u;
#pragma unroll
  for (int i = 0; i < N; ++i) from_f(&u.v.v[i], f[i]);
  *reinterpret_cast<Access<T, N> *>(p) = u.r;
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

// One cluster of 16 blocks of 32 warps.  Each warp takes a run of consecutive slots: first it counts
// them by expert, then, with the counts of all warps before it added up, gives them their rows in
// order, 32 at a time (lanes of one expert by their number).  Counters are whole numbers and each
// warp's own, so the order is that of the slots.  The ids of kAhead steps are loaded together: a
// warp does little between two loads, and there are few warps.
constexpr int kAhead = 8;

// lanes whose key is this lane's, by a vote on each of its bits
__device__ __forceinline__ unsigned same_key(int key, int bits) {
  unsigned same = kAll;
#pragma unroll
  for (int b = 0; b < 11; ++b) {   // kMaxExperts + 1 has 11
    if (b >= bits) break;
    const bool set = (key >> b) & 1;
    const unsigned v = __ballot_sync(kAll, set);
    same &= set ? v : ~v;
  }
  return same;
}

constexpr int kOrderBlocks = 16, kOrderThreads = 1024, kOrderWarps = kOrderThreads / 32;

__global__ void __launch_bounds__(kOrderThreads) expert_order_kernel(const OrderArgs p) {
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
  for (long long b = lo; b < hi; b += 32 * kAhead) {
    int64_t id[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) id[a] = b + 32 * a + lane < hi ? p.ids[b + 32 * a + lane] : 0;
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (b + 32 * a + lane < hi) atomicAdd(&mine[key_of(id[a], E, p.err)], 1u);
  }
  __syncthreads();
  for (int e = tid; e < width; e += kOrderThreads) {
    unsigned v[kOrderWarps], sum = 0u;
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) v[w] = hist[w * width + e];
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) {
      hist[w * width + e] = sum;
      sum += v[w];
    }
    total[e] = sum;
  }
  cluster.sync();
  // this thread's expert (at most kOrderThreads of them): slots of it in all blocks and in those before this one
  unsigned all = 0u, before = 0u;
  if (tid < E) {
#pragma unroll
    for (int r = 0; r < kOrderBlocks; ++r) {
      const unsigned v = cluster.map_shared_rank(total, r)[tid];
      all += v;
      before += r < rank ? v : 0u;
    }
  }
  // the slots before this block's that are not routed
  if (wp == kOrderWarps - 1) {
    const unsigned v = lane < rank ? cluster.map_shared_rank(total, lane)[E] : 0u;
    const unsigned sum = __reduce_add_sync(kAll, v);
    if (lane == 0) start[E] = sum;
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
    start[E] += routed;
    if (rank == 0) p.offsets[E] = p.n;   // rows of no slot count to the last expert
  }
  __syncthreads();
  const int bits = 32 - __clz(E + 1);   // of a key, and of E + 1, which the lanes behind the run's end have
  for (long long b = lo; b < hi; b += 32 * kAhead) {
    int64_t id[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) id[a] = b + 32 * a + lane < hi ? p.ids[b + 32 * a + lane] : 0;
    unsigned same[kAhead];
    int key[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      key[a] = b + 32 * a + lane < hi ? key_of(id[a], E, p.err) : E + 1;
      same[a] = same_key(key[a], bits);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const bool in = key[a] <= E;
      const unsigned below = same[a] & ((1u << lane) - 1u);
      unsigned at = 0u;
      if (in) at = start[key[a]] + mine[key[a]] + __popc(below);
      __syncwarp();
      if (in && below == 0u) mine[key[a]] += __popc(same[a]);
      __syncwarp();
      if (in) p.place[b + 32 * a + lane] = key[a] < E ? (int64_t)at : -1 - (int64_t)at;
    }
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
  int tx, turns;           // threads of a token, a power of two; tokens one after the other in a block
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

// Copies of one access of a token's row, written k times.
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

// A block's tokens are blockIdx.x * turns * (kThreads / tx) and on, kThreads / tx of them at a time. Their places and
// weights come first, all at once: with each token reading its own, a block spent as long on waiting for the
// places as on the rows (combine, 16384 tokens x 8 of 6144 bf16: 346 us).
// A routed slot's row is >= 0, that of one which is not -1 - row, kNoRow one out of range.
constexpr int kBatchSlots = 1024, kPartSlots = 128, kNoRow = INT_MIN;
struct Batch {
  int row[kBatchSlots];
  float w[kBatchSlots];

  // tokens of this block
  __device__ __forceinline__ int load(const RowArgs &p, int64_t first) {
    const int n = (int)min((int64_t)p.turns * (kThreads / p.tx), p.tokens - first);
    const int64_t slots = p.tokens * p.top, s0 = first * p.top;
    for (int i = threadIdx.x; i < n * p.top; i += kThreads) {
      const int64_t at = p.place[s0 + i];
      const bool in = at < slots && at >= -slots;
      if (!in) atomicOr(p.err, kErrDevice);
      row[i] = in ? (int)at : kNoRow;
      w[i] = p.weights ? p.weights[s0 + i] : 1.f;
    }
    __syncthreads();
    return n;
  }
};

// Accesses of a thread: 16 bytes' worth, so that narrow ones (rows or strides that are no multiple of 16 bytes)
// have as much in flight.
template <int BYTES>
constexpr int kAccesses = 16 / BYTES;

template <int BYTES>
__global__ void __launch_bounds__(kThreads) dispatch_rows_kernel(const RowArgs p) {
  typedef typename Raw<BYTES>::type R;
  constexpr int U = kAccesses<BYTES>;
  __shared__ Batch batch;
  const int per = kThreads / p.tx, sub = threadIdx.x / p.tx, c0 = blockIdx.y * p.tx * U + threadIdx.x % p.tx;
  const int64_t first = blockIdx.x * (int64_t)(p.turns * per);
  wait_for_previous_grid();
  const int n = batch.load(p, first);
  const R *x = reinterpret_cast<const R *>(p.x);
  R *rows = reinterpret_cast<R *>(p.rows);
  for (int t = sub; t < n; t += per) {
    R v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * p.tx < p.vecs) v[u] = __ldcs(x + (first + t) * p.ldx + c0 + u * p.tx);
    for (int j = 0; j < p.top; ++j) {
      const int r = batch.row[t * p.top + j];
      if (r == kNoRow) continue;
      R *dst = rows + (int64_t)(r < 0 ? -1 - r : r) * p.vecs + c0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * p.tx < p.vecs) dst[u * p.tx] = r < 0 ? R{} : v[u];
    }
  }
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
  int key[kFewSlots / kThreads];   // of this thread's slots, all read at once
#pragma unroll
  for (int a = 0; a < kFewSlots / kThreads; ++a)
    key[a] = a * kThreads + tid < n ? key_of(p.ids[a * kThreads + tid], p.experts, p.err) : INT_MAX;
  __syncthreads();
  for (int j = 0; j < p.top; ++j) {
    const int slot = token * p.top + j, mine = key_of(p.ids[slot], p.experts, p.err);
    unsigned before = 0u;
#pragma unroll
    for (int a = 0; a < kFewSlots / kThreads; ++a)
      before += key[a] < mine || (key[a] == mine && a * kThreads + tid < slot);
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
  for (int c = blockIdx.y * kThreads + tid; c < p.vecs; c += gridDim.y * kThreads) copy_out<BYTES>(p, token, c, place);
}

// out[t]: a thread has the same place of the k rows, the loads of kSlots of them in flight together.  kSlots is 2, 4 or 8
// by k: fewer registers leave more blocks on an SM (gradient of 30000 tokens x 1 of 2048: 78 us with 2, 133 us with 8).
template <typename T, int N, int kSlots>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowArgs p) {
  constexpr int U = kAccesses<sizeof(T) * N>;
  __shared__ Batch batch;
  const int per = kThreads / p.tx, sub = threadIdx.x / p.tx, step = p.tx * N;
  const int c0 = (blockIdx.y * p.tx * U + threadIdx.x % p.tx) * N;
  const int64_t first = blockIdx.x * (int64_t)(p.turns * per);
  const int n = batch.load(p, first);
  const T *y = static_cast<const T *>(p.y) + c0;
  T *out = static_cast<T *>(p.out) + c0;
  for (int t = sub; t < n; t += per) {
    float sum[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) sum[u][i] = 0.f;
    for (int j0 = 0; j0 < p.top; j0 += kSlots) {
      Access<T, N> v[kSlots][U];
      const int *row = batch.row + t * p.top + j0;
      const float *w = batch.w + t * p.top + j0;
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (j0 + j < p.top && row[j] >= 0) {
          const T *src = y + (int64_t)row[j] * p.hidden;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + u * step < p.hidden) v[j][u] = load_once<T, N>(src + u * step);
        }
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (j0 + j < p.top && row[j] >= 0) {
          const float wj = w[j];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float f[N];
            unpack<T, N>(f, v[j][u]);
#pragma unroll
            for (int i = 0; i < N; ++i) sum[u][i] = fmaf(wj, f[i], sum[u][i]);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * step < p.hidden) store<T, N>(out + (first + t) * p.ldo + u * step, sum[u]);
  }
}

// The gradient: a token's threads go over its row once for every kSlots slots, each access of dout
// meeting those of y.  The products' sums: a thread's in turn, a tree over the warp, and the warps' in order
// when the block's tokens are done.
template <typename T, int N, int kSlots>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const RowArgs p) {
  constexpr int U = kAccesses<sizeof(T) * N>;
  __shared__ Batch batch;
  __shared__ float part[kThreads / 32][kPartSlots];   // per warp of a token: its slots' sums
  const int tx = p.tx, me = threadIdx.x % tx, lane = threadIdx.x & 31, per = kThreads / tx, sub = threadIdx.x / tx;
  const int warps = tx / 32, wp = me >> 5;                                // of a token; 0: tokens share a warp
  const int64_t first = blockIdx.x * (int64_t)(p.turns * per);
  const int n = batch.load(p, first);
  const T *y = static_cast<const T *>(p.y);
  T *dy = static_cast<T *>(p.rows);
  for (int t0 = 0; t0 < n; t0 += per) {
    const int t = t0 + sub;
    const bool in = t < n;
    const T *dout = static_cast<const T *>(p.x) + (first + t) * p.ldx;
    for (int j0 = 0; j0 < p.top; j0 += kSlots) {
      const int *row = batch.row + t * p.top + j0;
      const float *w = batch.w + t * p.top + j0;
      float dot[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) dot[j] = 0.f;
      if (in)
        for (int c = me * N; c < p.hidden; c += tx * N * U) {
          float d[U][N];
          Access<T, N> v[kSlots][U];
          if (p.dweights)
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
              if (j0 + j < p.top && row[j] >= 0) {
                const T *src = y + (int64_t)row[j] * p.hidden + c;
#pragma unroll
                for (int u = 0; u < U; ++u)
                  if (c + u * tx * N < p.hidden) v[j][u] = load_once<T, N>(src + u * tx * N);
              }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c + u * tx * N < p.hidden) unpack<T, N>(d[u], load<T, N>(dout + c + u * tx * N));
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (j0 + j < p.top && row[j] != kNoRow) {
              const int r = row[j];
              T *dst = dy + (int64_t)(r < 0 ? -1 - r : r) * p.hidden + c;
              const float wj = w[j];
#pragma unroll
              for (int u = 0; u < U; ++u) {
                if (c + u * tx * N >= p.hidden) break;
                float o[N];
                if (dy) {
#pragma unroll
                  for (int i = 0; i < N; ++i) o[i] = r < 0 ? 0.f : wj * d[u][i];
                  store<T, N>(dst + u * tx * N, o);
                }
                if (p.dweights && r >= 0) {
                  unpack<T, N>(o, v[j][u]);
#pragma unroll
                  for (int i = 0; i < N; ++i) dot[j] = fmaf(d[u][i], o[i], dot[j]);
                }
              }
            }
        }
      if (!p.dweights) continue;
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (j0 + j < p.top)   // the same for all
          for (int o = min(tx, 32) / 2; o; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
      if (warps > 1) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (in && lane == j && j0 + j < p.top) part[wp][t * p.top + j0 + j] = dot[j];
      } else if (in && me == 0) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (j0 + j < p.top) p.dweights[(first + t) * p.top + j0 + j] = dot[j];
      }
    }
  }
  if (!p.dweights || warps <= 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < n * p.top; i += kThreads) {
    float s = part[0][i];
    for (int k = 1; k < warps; ++k) s += part[k][i];
    p.dweights[first * p.top + i] = s;
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

// How a kernel by tokens is laid out: threads of a token (a power of two that covers its accesses, 8 to 256), the
// columns' blocks, and how many tokens a block takes in turn: up to 8, as many as leave `each` blocks an SM, and whose
// slots fit `most` (a batch's).  Measured with 16 and 8 blocks an SM: combine's gradient, 4099 tokens x 8 of 2048, 61.6
// and 54.6 us, dispatch's gradient, 4099 x 4 of 1001 fp32, 21.3 and 17.1, but dispatch 34.0 and 35.4; up to 16 tokens in
// turn are slower where there are many (16384 x 8 of 6144: combine 277 and 287).
dim3 layout(RowArgs &p, int accesses, bool columns, int most, int64_t each) {
  const int need = (p.vecs + accesses - 1) / accesses;
  p.tx = 8;
  while (p.tx < kThreads && p.tx < need) p.tx *= 2;
  const int per = kThreads / p.tx;
  const int64_t cols = columns ? (need + p.tx - 1) / p.tx : 1;
  const int64_t turns = std::min<int64_t>(p.tokens * cols / (each * per * num_sms()), 8);
  p.turns = (int)std::clamp<int64_t>(turns, 1, std::max(1, most / (per * p.top)));
  return dim3((unsigned)((p.tokens + per * p.turns - 1) / (per * p.turns)), (unsigned)cols);
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
// f(element, elements of an access, slots in registers at once)
template <typename F>
void with_vec(int type, int bytes, int top, F &&f) {
  with_bytes(bytes, [&](auto b) {
    constexpr int B = decltype(b)::value;
    auto slots = [&](auto element, auto n) {
      // rows of 16-bit elements on 2- or 4-byte boundaries: 16384 tokens x 6 of 2001, 122 us with 4 slots, 140 with 8
      const bool narrow = B <= 4 && sizeof(element) == 2;
      if (top <= 2) f(element, n, std::integral_constant<int, 2>());
      else if (top <= 4 || narrow) f(element, n, std::integral_constant<int, 4>());
      else f(element, n, std::integral_constant<int, 8>());
    };
    if (type == MUON_BF16) slots(__nv_bfloat16(), std::integral_constant<int, B / 2>());
    else if constexpr (B >= 4) slots(float(), std::integral_constant<int, B / 4>());
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
  auto *kernel = expert_order_kernel;
  auto bytes = [](int64_t experts) { return (size_t)(kOrderWarps + 2) * (experts + 1) * sizeof(unsigned); };
  std::call_once(once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(kMaxExperts));
    if (attr_err[dev] == cudaSuccess)
      attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (attr_err[dev] != cudaSuccess) return MUON_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kOrderBlocks);
  cfg.blockDim = dim3(kOrderThreads);
  cfg.dynamicSmemBytes = bytes(a.experts);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kOrderBlocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_before(kTraceExpertOrder, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  const int st = trace_after(kTraceExpertOrder, s);
  return e == cudaSuccess ? st : MUON_ERR_CUDA;
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
    // every block sorts again, so a token's row is shared among blocks only while SMs are left
    const int64_t share = std::min<int64_t>((p.vecs + kThreads - 1) / kThreads, std::max<int64_t>(1, 2 * num_sms() / tokens));
    const dim3 grid((unsigned)tokens + 1, (unsigned)share);
    trace_before(kTraceDispatchRows, s);
    with_bytes(bytes, [&](auto b) { dispatch_few_kernel<decltype(b)::value><<<grid, kThreads, 0, s>>>(p); });
    return trace_after(kTraceDispatchRows, s);
  }
  const OrderArgs oa{ids, (int)(tokens * top), (int)experts, offsets, place, err};
  const int so = order(oa, s);
  if (so != MUON_OK) return so;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = layout(p, 16 / bytes, true, kBatchSlots, 16);
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
  p.err = device_error_word();
  if (!p.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid = layout(p, 16 / bytes, true, kBatchSlots, 8);
  trace_before(kTraceCombine, s);
  with_vec(type, bytes, p.top, [&](auto t, auto n, auto k) {
    combine_kernel<decltype(t), decltype(n)::value, decltype(k)::value><<<grid, kThreads, 0, s>>>(p);
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
  p.err = device_error_word();
  if (!p.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned blocks = layout(p, 16 / bytes, false, kPartSlots, 8).x;
  trace_before(kTraceCombineBwd, s);
  with_vec(type, bytes, p.top, [&](auto t, auto n, auto k) {
    combine_backward_kernel<decltype(t), decltype(n)::value, decltype(k)::value><<<blocks, kThreads, 0, s>>>(p);
  });
  return trace_after(kTraceCombineBwd, s);
}

}  // extern "C"
