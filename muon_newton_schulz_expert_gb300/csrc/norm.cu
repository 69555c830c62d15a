// RMS norms before and after a block, fused with the block's gate and residual
// scale, and their gradients (HBM-bound).
//
//   n  = b * q * w_post,            q = 1/sqrt(mean(b^2) + eps)    (norm after the block)
//   r' = r + scale * gate * n                                      (residual stream)
//   y  = r' * p * w_pre,            p = 1/sqrt(mean(r'^2) + eps)   (norm before the next block)
//
// Backward, with bh = b q and xh = r' p (q, p saved by the forward pass):
//   dr'  = dr_out + p (w_pre dy - xh mean(w_pre dy xh)),     dr = dr'
//   dn   = scale gate dr'
//   db   = q (w_post dn - bh mean(w_post dn bh))
//   dw_pre = sum_rows dy xh,  dw_post = sum_rows dn bh,  dgate = scale dr' bh w_post
//
// One pass over memory.  A group of threads takes one row at a time and walks
// the rows of the array; several groups on an SM overlap one's reductions with
// another's loads.  The weights and a shared gate stay in L1, and so does the
// part of a row that is read a second time after its reduction rather than held
// in registers; where rows have many bytes they come through shared memory, copied
// ahead (Stages), and the weights are in registers.  The weights' gradients
// stay in registers over a group's rows; each block writes its sums and a
// second kernel adds them, in a fixed order (no atomics).  All arithmetic is
// fp32, in pairs (f32x2) where vectors are moved.
#include <algorithm>
#include <type_traits>

#include "tc.cuh"

namespace muon {
namespace {

constexpr int kMaxHidden = 16384;
constexpr int kRowsPerCta = 4;   // rows of one CTA where a warp holds a whole row

// Rows of more than 128 vectors give each thread kPlaces of them.  The largest
// block of an instance and how many of them an SM has to hold fix its
// registers: 56 a thread forward, 80 backward, where two sums per column are
// kept besides.  A backward thread of two places keeps 370 to 520 bytes in local
// memory all the same, one of a wide block, with 64 registers, 460 to 680: these forms
// take 1.6 to 2.5 times what their bytes do (6144 and 9216 columns).  Measured at
// 16384 x 6144: forward in bf16 150 us (79% of the measured copy bandwidth).  Rows
// that need more threads than that take an
// instance with wide blocks.
constexpr int kPlaces = 2;
constexpr int max_threads(int w, int vpt, bool backward) {
  if (w == 1) return vpt == 4 ? 512 : 1024;
  return vpt == 1 ? 128 : 384;
}
constexpr int kWideThreads = 1024;
constexpr int blocks_per_sm(int w, int threads, bool backward) {
  const int all = w == 1 ? 1024 : backward ? 768 : 1152;
  return threads > all / 2 ? 1 : all / (threads < 64 ? 64 : threads);
}

struct Row {
  const void *p;
  int64_t stride;   // elements
};
struct RowOut {
  void *p;
  int64_t stride;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float *d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 *d, float v) { *d = __float2bfloat16_rn(v); }

// ------------------------------------------------------------ one or two floats
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 halves(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(F2 a) {
  const float2 h = halves(a);
  return h.x + h.y;
}
__device__ __forceinline__ float total(float a) { return a; }
template <typename P>
__device__ __forceinline__ P both(float x) {
  if constexpr (std::is_same_v<P, F2>) return pair(x, x);
  else return x;
}

// W consecutive elements of a thread: four pairs (16-byte vectors), or one
// element (widths or strides that are not multiples of 8, unaligned pointers).
template <int W>
using Item = std::conditional_t<W == 8, F2, float>;
template <int W>
constexpr int kItems = W == 8 ? 4 : 1;

// Eight elements of type T from 16-byte vectors `step` vectors apart.
template <typename T>
__device__ __forceinline__ void widen(const uint4 *src, int step, F2 (&v)[4]) {
  const uint4 x = src[0];
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
    const uint4 y = src[step];
    v[0] = pair(__uint_as_float(x.x), __uint_as_float(x.y)), v[1] = pair(__uint_as_float(x.z), __uint_as_float(x.w));
    v[2] = pair(__uint_as_float(y.x), __uint_as_float(y.y)), v[3] = pair(__uint_as_float(y.z), __uint_as_float(y.w));
  }
}

template <typename T>
__device__ __forceinline__ void load(const T *src, F2 (&v)[4]) {
  widen<T>(reinterpret_cast<const uint4 *>(src), 1, v);
}
template <typename T>
__device__ __forceinline__ void load(const T *src, float (&v)[1]) {
  v[0] = to_f(*src);
}

// Rows are written once: evict-first, which leaves L2 to the rows being read.
template <typename T>
__device__ __forceinline__ void store(T *dst, const F2 (&v)[4]) {
  const float2 a = halves(v[0]), b = halves(v[1]), c = halves(v[2]), d = halves(v[3]);
  uint4 *out = reinterpret_cast<uint4 *>(dst);
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 h[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(b.x, b.y),
                           __floats2bfloat162_rn(c.x, c.y), __floats2bfloat162_rn(d.x, d.y)};
    const uint32_t *w = reinterpret_cast<const uint32_t *>(h);
    __stcs(out, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    __stcs(reinterpret_cast<float4 *>(out), make_float4(a.x, a.y, b.x, b.y));
    __stcs(reinterpret_cast<float4 *>(out) + 1, make_float4(c.x, c.y, d.x, d.y));
  }
}
template <typename T>
__device__ __forceinline__ void store(T *dst, const float (&v)[1]) {
  from_f(dst, v[0]);
}

// Plain stores (shared memory).
__device__ __forceinline__ void keep(float *dst, const F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = halves(v[i]);
    dst[2 * i] = h.x, dst[2 * i + 1] = h.y;
  }
}
__device__ __forceinline__ void keep(float *dst, const float (&v)[1]) { dst[0] = v[0]; }

// Sums of N values over the threads of a row (blockDim.x, a multiple of 32);
// with one warp per row no shared memory and no barrier is used.  Successive
// sums alternate between two buffers, so one barrier each is enough: a buffer
// is written again only after a barrier that every reader of its last sums has
// passed.  Every thread adds the warps' sums itself (broadcast reads).
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float4 (*buf)[8]) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (blockDim.x == 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<float *>(buf[i])[warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < warps; w += 4) {   // places past the last warp hold zeros
      const float4 x = buf[i][w >> 2];
      v[i] += (x.x + x.y) + (x.z + x.w);
    }
  }
}
// before the first row_sums
template <int N>
__device__ __forceinline__ void clear_sums(float4 (*buf)[N][8]) {
  for (int i = threadIdx.x + threadIdx.y * blockDim.x; i < 2 * N * 8; i += blockDim.x * blockDim.y)
    (&buf[0][0][0])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
}

// A thread's place in one input or output: its columns of the row at hand, and
// the step to its group's next row.
template <typename T>
struct Walk {
  T *p;
  int64_t step;

  __device__ Walk(const void *base, int64_t stride, int64_t row, int64_t rows, int c)
      : p(base ? const_cast<T *>(static_cast<const T *>(base)) + row * stride + c : nullptr), step(rows * stride) {}
  __device__ void next() { p += step; }
};

// Which parts a call has.  The forms with everything (both norms and their
// weights, the incoming gradient, every output) are compiled with that
// knowledge, which nearly halves their instructions; ANY asks at run time.
enum Form { ANY = 0, FULL, FULL_SHARED_GATE, FULL_ROW_GATE };

// Multiplies by a vector of the weights.
template <typename T, int W>
__device__ __forceinline__ void times(const T *w, Item<W> (&v)[kItems<W>]) {
  Item<W> x[kItems<W>];
  load(w, x);
#pragma unroll
  for (int j = 0; j < kItems<W>; ++j) v[j] = mul(v[j], x[j]);
}

// Rows on their way in: the rows that one token reads (backward: dr_out, r', dy, b
// and a gate of its own; forward: r, b and the gate) are copied to shared memory
// whole, by one thread and the copy engine, up to `stages` tokens ahead.  The threads
// then spend no instructions and hold no registers on loads in flight, so that
// few of them suffice and each has registers for the weights: the kernel was
// bound by the instructions it issued (about 40 an element, 5 of every 8 vector
// loads being of weights).  16384 x 6144 in bf16: 232 us, by now 226 to 229 (78% of the
// measured copy bandwidth), against 301 us with plain loads, 2 blocks of 384 threads; 272 us
// with the weights re-read and 512 threads, 317 us with 768 threads of one place,
// 225 us with 256 threads of three, which takes 165 us where this takes 125 (30000 x
// 2048).  8192 columns, fp32 stream: 334 against 493 us.
// Every wait is bounded; after one that ran out the block goes on without
// waiting, on whatever it has, and the error word says so.
constexpr int kMaxStages = 8;
struct Staging {
  const uint8_t *src[5];     // in the order of their places in a slot
  int64_t pitch[5];          // bytes from row to row
  uint32_t bytes[5];
  int count, stages, slot_bytes;
  unsigned *err;
  unsigned long long timeout_ns;
};

struct Stages {
  const Staging &in;
  const int64_t rows;
  unsigned long long *full;   // shared: a barrier for each slot
  int *abort;
  int slot = 0;
  uint32_t phase = 0, issued = 0, parity = 0;   // thread 0: slots ever filled, and their last fill's parity

  __device__ Stages(const Staging &s, int64_t n, unsigned long long *bars, int *flag)
      : in(s), rows(n), full(bars), abort(flag) {}
  __device__ static uint8_t *rows_in() {
    extern __shared__ __align__(128) uint8_t staged_rows[];
    return staged_rows;
  }
  __device__ void fetch(int64_t row, int to_slot, uint32_t ph) {
    issued |= 1u << to_slot;
    parity = (parity & ~(1u << to_slot)) | (ph << to_slot);
    const uint32_t bar = smem_u32(full + to_slot);
    uint32_t to = smem_u32(rows_in()) + (uint32_t)(to_slot * in.slot_bytes), all = 0;
    for (int i = 0; i < in.count; ++i) all += in.bytes[i];
    mbar_expect_tx(bar, all);
    for (int i = 0; i < in.count; ++i) {
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                   "l"(in.src[i] + row * in.pitch[i]), "r"(in.bytes[i]), "r"(bar)
                   : "memory");
      to += in.bytes[i];
    }
  }
  // before a __syncthreads
  __device__ void start(int64_t first, int64_t step) {
    if (threadIdx.x != 0) return;
    *abort = 0;
    for (int i = 0; i < in.stages; ++i) mbar_init(smem_u32(full + i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < in.stages && first + i * step < rows; ++i) fetch(first + i * step, i, 0);
  }
  // the row at hand, complete
  __device__ const uint8_t *wait() {
    volatile int *flag = abort;
    if (!*flag) wait_bounded(smem_u32(full + slot), phase, Watch{flag, in.err, in.timeout_ns});
    return rows_in() + slot * in.slot_bytes;
  }
  // after a __syncthreads that follows wait(): every thread is done with the
  // row before, whose slot takes the next one due
  __device__ void next(int64_t row, int64_t first, int64_t step) {
    const int64_t due = row + (in.stages - 1) * step;
    if (threadIdx.x == 0 && row != first && due < rows && !*static_cast<volatile int *>(abort))
      fetch(due, slot ? slot - 1 : in.stages - 1, slot ? phase ^ 1u : phase);
    if (++slot == in.stages) slot = 0, phase ^= 1u;
  }
  // after the last row: if a wait ran out, copies may still be landing
  __device__ void finish() {
    if (threadIdx.x != 0 || !*static_cast<volatile int *>(abort)) return;
    const unsigned long long limit = in.timeout_ns < 20000000ull ? in.timeout_ns : 20000000ull;
    for (int i = 0; i < in.stages; ++i)
      if (issued & (1u << i)) drain_wait(smem_u32(full + i), (parity >> i) & 1u, limit);
  }
};

struct FwdArgs {
  Row residual, block, gate;   // gate: a row for each token (a shared gate is a column factor)
  RowOut residual_out, normed;
  const void *w_post, *shared_gate, *w_pre;
  float *rstd_post, *rstd_pre;
  int64_t rows;
  int hidden;
  float scale, eps;
  Staging in;
};

template <typename R, typename B, int W, int VPT, int THREADS, int FORM, bool STAGED = false>
__global__ void __launch_bounds__(THREADS, STAGED ? 1 : blocks_per_sm(W, THREADS, false))
    block_norm_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float4 red[2][1][8];
  using P = Item<W>;
  constexpr int N = kItems<W>;
  const int64_t group = blockIdx.x * (int64_t)blockDim.y + threadIdx.y, groups = gridDim.x * (int64_t)blockDim.y;
  const int c0 = threadIdx.x * W, across = blockDim.x * W;   // this thread's columns: c0, c0 + across, ...
  const float inv_h = 1.f / (float)a.hidden;
  constexpr bool full = FORM != ANY;
  const bool post = full || a.block.p, pre = full || a.normed.p;
  const bool gate_rows = full ? FORM == FULL_ROW_GATE : a.gate.p != nullptr;
  const bool gate_shared = full ? FORM == FULL_SHARED_GATE : a.shared_gate != nullptr;
  __shared__ unsigned long long bars[STAGED ? kMaxStages : 1];
  __shared__ int aborted;
  Stages staged(a.in, a.rows, bars, &aborted);
  if (STAGED) staged.start(group, groups);
  clear_sums<1>(red);
  Walk<R> res(a.residual.p, a.residual.stride, group, groups, c0);
  Walk<B> blk(a.block.p, a.block.stride, group, groups, c0), gate(a.gate.p, a.gate.stride, group, groups, c0);
  Walk<R> out(a.residual_out.p, a.residual_out.stride, group, groups, c0);
  Walk<B> y(a.normed.p, a.normed.stride, group, groups, c0);
  const B *w_post = static_cast<const B *>(a.w_post), *w_pre = static_cast<const B *>(a.w_pre);
  const B *shared_gate = static_cast<const B *>(a.shared_gate);
  // staged: the weights stay in registers: w_pre, and w_post times a shared gate
  P keep_pre[STAGED ? VPT : 1][N], keep_post[STAGED ? VPT : 1][N];
  if constexpr (STAGED) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * across;
#pragma unroll
      for (int j = 0; j < N; ++j) keep_pre[i][j] = keep_post[i][j] = both<P>(0.f);
      if (c < a.hidden) {
        load(w_pre + c, keep_pre[i]);
        load(w_post + c, keep_post[i]);
        if (gate_shared) times<B, W>(shared_gate + c, keep_post[i]);
      }
    }
  }
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += groups) {
    const R *res_at = res.p;   // this thread's columns of the row at hand
    const B *blk_at = blk.p, *gate_at = gate.p;
    if constexpr (STAGED) {
      const uint8_t *at = staged.wait();
      res_at = reinterpret_cast<const R *>(at) + c0;
      blk_at = reinterpret_cast<const B *>(at + sizeof(R) * a.hidden) + c0;
      gate_at = blk_at + a.hidden;
    }
    P r[VPT][N], ss = both<P>(0.f);
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (c0 + i * across < a.hidden) load(res_at + i * across, r[i]);
    if (post) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (c0 + i * across < a.hidden) {
          P b[N];
          load(blk_at + i * across, b);
#pragma unroll
          for (int j = 0; j < N; ++j) ss = fma(b[j], b[j], ss);
        }
      float sum[1] = {total(ss)};
      row_sums(sum, red[turn]);
      if (STAGED) staged.next(row, group, groups);
      turn ^= 1;
      q = rsqrtf(fmaf(sum[0], inv_h, a.eps));
      if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[row] = q;
    }
    ss = both<P>(0.f);
    const P qs = both<P>(a.scale * q);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (c0 + i * across < a.hidden) {
        const int c = c0 + i * across;
        if (post) {
          P b[N];
          load(blk_at + i * across, b);   // again, from L1 or shared memory
          if constexpr (STAGED) {
#pragma unroll
            for (int j = 0; j < N; ++j) b[j] = mul(b[j], keep_post[i][j]);
          } else if (full || w_post) {
            times<B, W>(w_post + c, b);
          }
          if (gate_rows) times<B, W>(gate_at + i * across, b);
          else if (gate_shared && !STAGED) times<B, W>(shared_gate + c, b);
#pragma unroll
          for (int j = 0; j < N; ++j) r[i][j] = fma(b[j], qs, r[i][j]);
          store(out.p + i * across, r[i]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) ss = fma(r[i][j], r[i][j], ss);
      }
    if (pre) {
      // y is formed from r' before its rounding to the stream's type
      float sum[1] = {total(ss)};
      row_sums(sum, red[turn]);
      turn ^= 1;
      const float p = rsqrtf(fmaf(sum[0], inv_h, a.eps));
      if (threadIdx.x == 0 && a.rstd_pre) a.rstd_pre[row] = p;
      const P p2 = both<P>(p);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (c0 + i * across < a.hidden) {
#pragma unroll
          for (int j = 0; j < N; ++j) r[i][j] = mul(r[i][j], p2);
          if constexpr (STAGED) {
#pragma unroll
            for (int j = 0; j < N; ++j) r[i][j] = mul(r[i][j], keep_pre[i][j]);
          } else if (full || w_pre) {
            times<B, W>(w_pre + c0 + i * across, r[i]);
          }
          store(y.p + i * across, r[i]);
        }
    }
    res.next(), blk.next(), gate.next(), out.next(), y.next();
  }
  if (STAGED) staged.finish();
}

struct BwdArgs {
  Row dresidual_out, dnormed, residual, block, gate;   // gate: a row for each token
  RowOut dresidual, dblock, dgate;                     // dgate: a row for each token
  const void *w_post, *shared_gate, *w_pre;
  const float *rstd_post, *rstd_pre;
  float *partial;                    // [blocks][2][hidden]: sums of dy xh, and of (per-row gate) dr bh
  int64_t rows;
  int hidden;
  float scale;
  Staging in;
};

// The two means of a row come from one reduction of three sums over the raw
// rows.  With tp = p w_pre dy, z = dr_out + tp and k = scale gate w_post,
//   dr = z - c1 r',           c1 = p^2 S1 / H,            S1 = sum tp r'
//   db = q k dr - c2 b,       c2 = q^3 (S2 - c1 S3) / H,  S2 = sum k b z,  S3 = sum k b r'
// For a shared gate, sum over rows of dr b q serves dw_post (times scale gate)
// and dgate (times scale w_post) alike.
template <typename R, typename B, int W, int VPT, int THREADS, int FORM, bool STAGED = false>
__global__ void __launch_bounds__(THREADS, STAGED ? 1 : blocks_per_sm(W, THREADS, true))
    block_norm_backward_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float4 red[2][3][8];
  using P = Item<W>;
  constexpr int N = kItems<W>;
  const int64_t group = blockIdx.x * (int64_t)blockDim.y + threadIdx.y, groups = gridDim.x * (int64_t)blockDim.y;
  const int c0 = threadIdx.x * W, across = blockDim.x * W;
  const float inv_h = 1.f / (float)a.hidden;
  constexpr bool full = FORM != ANY;
  let_next_grid_start();   // norm_weight_sum_kernel, which waits for this one's end
  const bool post = full || a.block.p, pre = full || a.dnormed.p;
  const bool from_above = full || a.dresidual_out.p;
  const bool gate_rows = full ? FORM == FULL_ROW_GATE : a.gate.p != nullptr;
  const bool gate_shared = full ? FORM == FULL_SHARED_GATE : a.shared_gate != nullptr;
  // staged: rows come in through shared memory
  __shared__ unsigned long long bars[STAGED ? kMaxStages : 1];
  __shared__ int aborted;
  Stages staged(a.in, a.rows, bars, &aborted);
  if (STAGED) staged.start(group, groups);
  clear_sums<3>(red);
  P dwp[VPT][N], dwq[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dwp[i][j] = dwq[i][j] = both<P>(0.f);
  Walk<R> dres(a.dresidual_out.p, a.dresidual_out.stride, group, groups, c0);
  Walk<R> res(a.residual.p, a.residual.stride, group, groups, c0);
  Walk<B> dnorm(a.dnormed.p, a.dnormed.stride, group, groups, c0);
  Walk<B> blk(a.block.p, a.block.stride, group, groups, c0), gate(a.gate.p, a.gate.stride, group, groups, c0);
  Walk<R> dr(a.dresidual.p, a.dresidual.stride, group, groups, c0);
  Walk<B> db(a.dblock.p, a.dblock.stride, group, groups, c0);
  const B *w_post = static_cast<const B *>(a.w_post), *w_pre = static_cast<const B *>(a.w_pre);
  const B *shared_gate = static_cast<const B *>(a.shared_gate);
  const R *dres_at = nullptr, *res_at = nullptr;   // this thread's columns of the row at hand
  const B *dnorm_at = nullptr, *blk_at = nullptr, *gate_at = nullptr;
  // staged: the weights stay in registers: w_pre, and w_post times a shared gate
  P keep_pre[STAGED ? VPT : 1][N], keep_post[STAGED ? VPT : 1][N];
  if constexpr (STAGED) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * across;
#pragma unroll
      for (int j = 0; j < N; ++j) keep_pre[i][j] = keep_post[i][j] = both<P>(0.f);
      if (c < a.hidden) {
        load(w_pre + c, keep_pre[i]);
        load(w_post + c, keep_post[i]);
        if (gate_shared) times<B, W>(shared_gate + c, keep_post[i]);
      }
    }
  }
  auto times_pre = [&](int i, P (&v)[N]) {
    if constexpr (STAGED) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = mul(v[j], keep_pre[i][j]);
    } else if (full || w_pre) {
      times<B, W>(w_pre + c0 + i * across, v);
    }
  };
  auto times_post = [&](int i, P (&v)[N]) {
    if constexpr (STAGED) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = mul(v[j], keep_post[i][j]);
    } else if (full || w_post) {
      times<B, W>(w_post + c0 + i * across, v);
    }
  };
  // k / scale = gate w_post, in g
  auto factors = [&](int i, P (&g)[N]) {
    const int c = c0 + i * across;
    if (STAGED && !gate_rows) {
#pragma unroll
      for (int j = 0; j < N; ++j) g[j] = keep_post[STAGED ? i : 0][j];
      return;
    }
    if (gate_rows) {
      load(gate_at + i * across, g);
    } else if (gate_shared) {
      load(shared_gate + c, g);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) g[j] = both<P>(1.f);
    }
    times_post(i, g);
  };
  int turn = 0;
  float p_next = 0.f, q_next = 0.f;   // staged: read a row ahead
  if (STAGED) p_next = a.rstd_pre[group], q_next = a.rstd_post[group];
  for (int64_t row = group; row < a.rows; row += groups) {
    const float p = STAGED ? p_next : pre ? a.rstd_pre[row] : 0.f;
    const float q = STAGED ? q_next : post ? a.rstd_post[row] : 0.f;
    if constexpr (STAGED) {
      if (row + groups < a.rows) p_next = a.rstd_pre[row + groups], q_next = a.rstd_post[row + groups];
      const uint8_t *at = staged.wait();
      dres_at = reinterpret_cast<const R *>(at) + c0;
      res_at = dres_at + a.hidden;
      dnorm_at = reinterpret_cast<const B *>(at + 2 * sizeof(R) * a.hidden) + c0;
      blk_at = dnorm_at + a.hidden;
      gate_at = blk_at + a.hidden;
    } else {
      dres_at = dres.p, res_at = res.p, dnorm_at = dnorm.p, blk_at = blk.p, gate_at = gate.p;
    }
    P z[VPT][N];
    P s1 = both<P>(0.f), s2 = s1, s3 = s1;
    const P p2 = both<P>(p);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (c0 + i * across < a.hidden) {
        P r[N];
        if (from_above) {
          load(dres_at + i * across, z[i]);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) z[i][j] = both<P>(0.f);
        }
        if (pre) {
          P t[N];
          load(res_at + i * across, r);
          load(dnorm_at + i * across, t);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            t[j] = mul(t[j], p2);
            dwp[i][j] = fma(t[j], r[j], dwp[i][j]);
          }
          times_pre(i, t);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            s1 = fma(t[j], r[j], s1);
            z[i][j] = add(z[i][j], t[j]);
          }
        }
        if (post) {
          P b[N], g[N];
          load(blk_at + i * across, b);
          factors(i, g);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const P kb = mul(g[j], b[j]);
            s2 = fma(kb, z[i][j], s2);
            if (pre) s3 = fma(kb, r[j], s3);
          }
        }
      }
    float sum[3] = {total(s1), total(s2), total(s3)};
    row_sums(sum, red[turn]);
    if (STAGED) staged.next(row, group, groups);
    turn ^= 1;
    // s2 and s3 lack the factor scale.  They carry one b, so one q goes onto them first: q^3
    // alone leaves fp32's range for blocks (rms 1e-13, 1e13) whose mean square does not.
    const float c1 = p * p * sum[0] * inv_h;
    const float c2 = (q * inv_h * a.scale) * (sum[1] - c1 * sum[2]) * (q * q);
    const P c1n = both<P>(-c1), c2n = both<P>(-c2), q2 = both<P>(q), scale = both<P>(a.scale);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (c0 + i * across < a.hidden) {
        if (pre) {
          P r[N];
          load(res_at + i * across, r);
#pragma unroll
          for (int j = 0; j < N; ++j) z[i][j] = fma(c1n, r[j], z[i][j]);
        }
        if (full || dr.p) store(dr.p + i * across, z[i]);
        if (post) {
          P b[N], g[N];
          load(blk_at + i * across, b);
#pragma unroll
          for (int j = 0; j < N; ++j) z[i][j] = mul(z[i][j], q2);   // dr q
          if (full ? gate_rows : a.dgate.p != nullptr) {
            P v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = mul(mul(z[i][j], b[j]), scale);
            times_post(i, v);
            store(static_cast<B *>(a.dgate.p) + row * a.dgate.stride + c0 + i * across, v);
          }
          if (gate_rows) {
            load(gate_at + i * across, g);
#pragma unroll
            for (int j = 0; j < N; ++j) dwq[i][j] = fma(mul(z[i][j], g[j]), b[j], dwq[i][j]);
          } else {
#pragma unroll
            for (int j = 0; j < N; ++j) dwq[i][j] = fma(z[i][j], b[j], dwq[i][j]);
          }
          factors(i, g);
#pragma unroll
          for (int j = 0; j < N; ++j) z[i][j] = fma(mul(g[j], scale), z[i][j], mul(c2n, b[j]));
          if (full || db.p) store(db.p + i * across, z[i]);
        }
      }
    dres.next(), res.next(), dnorm.next(), blk.next(), gate.next();
    dr.next(), db.next();
  }
  if (STAGED) staged.finish();
  if (!a.partial) return;
  // the block's sums: those of its groups where warps hold rows, through shared memory
  if (blockDim.y > 1) {
    constexpr int MOST = 32 * VPT * W;   // columns of a warp's row
    __shared__ float block_sums[VPT * W <= 8 ? kRowsPerCta : 1][2][VPT * W <= 8 ? MOST : 1];
    if constexpr (VPT * W <= 8) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        keep(&block_sums[threadIdx.y][0][c0 + i * across], dwp[i]);
        keep(&block_sums[threadIdx.y][1][c0 + i * across], dwq[i]);
      }
      __syncthreads();
      const int tid = threadIdx.x + threadIdx.y * 32;
      for (int k = tid; k < 2 * a.hidden; k += 32 * kRowsPerCta) {
        const int which = k >= a.hidden, c = k - which * a.hidden;
        float v = 0.f;
#pragma unroll
        for (int y = 0; y < kRowsPerCta; ++y) v += block_sums[y][which][c];
        a.partial[(int64_t)blockIdx.x * 2 * a.hidden + k] = v;
      }
    }
    return;
  }
  float *out = a.partial + blockIdx.x * (int64_t)2 * a.hidden + c0;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (c0 + i * across < a.hidden) {
      if (pre) store(out + i * across, dwp[i]);
      if (post) store(out + a.hidden + i * across, dwq[i]);
    }
}

// The weights' gradients from the blocks' sums: dw_pre = sum of the first,
// dw_post = scale (shared gate) times the sum of the second, and for a shared
// gate dgate = scale w_post times it.  16 x 4 interleaved partial sums per
// column, added in a fixed order.
template <typename B>
__global__ void __launch_bounds__(512) norm_weight_sum_kernel(const float *partial, int64_t blocks, int hidden,
                                                              float scale, const B *w_post, const B *shared_gate,
                                                              B *dw_pre, B *dw_post, B *dgate) {
  __shared__ float part[16][33];
  const int which = blockIdx.y;
  wait_for_previous_grid();
  if (which == 0 ? !dw_pre : !dw_post && !dgate) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v[4] = {};
  if (c < hidden)
    for (int64_t g = threadIdx.y; g < blocks; g += 64)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (g + 16 * k < blocks) v[k] += partial[((g + 16 * k) * 2 + which) * hidden + c];
  part[threadIdx.y][threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (threadIdx.y != 0 || c >= hidden) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += part[i][threadIdx.x];
  if (which == 0) {
    from_f(dw_pre + c, sum);
    return;
  }
  sum *= scale;
  if (dw_post) from_f(dw_post + c, shared_gate ? sum * to_f(shared_gate[c]) : sum);
  if (dgate) from_f(dgate + c, w_post ? sum * to_f(w_post[c]) : sum);
}

// Threads, and places per thread, of a row.
struct Plan {
  int w, vpt, threads, rows_per_cta;
};

Plan plan_rows(int hidden, bool vec, bool backward) {
  Plan p{};
  p.w = vec ? 8 : 1;
  const int n = (hidden + p.w - 1) / p.w;
  if (vec) {
    p.vpt = n <= 128 ? 1 : kPlaces;   // up to 128 places: one each
  } else {
    p.vpt = n <= 4 * max_threads(1, 4, backward) ? 4 : n <= 8 * max_threads(1, 8, backward) ? 8 : 16;
  }
  p.threads = (n + p.vpt - 1) / p.vpt;
  p.threads = (p.threads + 31) / 32 * 32;
  p.rows_per_cta = p.threads == 32 ? kRowsPerCta : 1;
  return p;
}
static_assert(8 * kPlaces * kWideThreads >= kMaxHidden && 16 * max_threads(1, 16, true) >= kMaxHidden,
              "every width has a plan");

inline bool vec_row(const void *p, int64_t stride, int type) {
  if (!p) return true;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % (type == MUON_BF16 ? 8 : 4) == 0;
}

// Groups of threads, each walking its share of the rows: as many as the
// registers of all SMs hold.
int64_t groups_of(const Plan &p, int64_t rows, bool backward) {
  const int per_sm = blocks_per_sm(p.w, p.threads * p.rows_per_cta, backward);
  return std::min<int64_t>((rows + p.rows_per_cta - 1) / p.rows_per_cta, (int64_t)num_sms() * per_sm) * p.rows_per_cta;
}

template <typename Kernel, typename Args>
int launch_rows(Kernel *kernel, const Args &a, const Plan &p, bool backward, int trace, cudaStream_t s) {
  trace_before(trace, s);
  kernel<<<dim3((unsigned)(groups_of(p, a.rows, backward) / p.rows_per_cta)), dim3(p.threads, p.rows_per_cta), 0, s>>>(
      a);
  return trace_after(trace, s);
}

template <typename R, typename B, int W, int VPT, int THREADS = max_threads(W, VPT, false)>
int launch_fwd_as(const FwdArgs &a, const Plan &p, cudaStream_t s) {
  auto go = [&](auto *kernel) { return launch_rows(kernel, a, p, false, kTraceBlockNorm, s); };
  if (a.block.p && a.normed.p && a.w_post && a.w_pre) {
    if (a.gate.p) return go(block_norm_kernel<R, B, W, VPT, THREADS, FULL_ROW_GATE>);
    if (a.shared_gate) return go(block_norm_kernel<R, B, W, VPT, THREADS, FULL_SHARED_GATE>);
    return go(block_norm_kernel<R, B, W, VPT, THREADS, FULL>);
  }
  return go(block_norm_kernel<R, B, W, VPT, THREADS, ANY>);
}

// Rows of more than 128 vectors with everything present go through shared
// memory, where two rows or more fit.  Few threads with many registers: backward 384
// of 168 an SM with two places each, in as many blocks as that gives, or one block of
// 256 with four places for rows that need it; forward 512 of 128.
constexpr int kStagedBytes = 216 * 1024;
constexpr int staged_threads(int places, bool backward) { return places == 4 ? 256 : backward ? 384 : 512; }

// Forward, which waits for two sums a row, it takes rows of many bytes, or ones that
// need wide blocks otherwise: 16384 x 6144 with an fp32 stream and a gate of its own
// for each row (48 KB) 219 us staged, 237 us not; the shared gate (36 KB) 210 and 202;
// bf16 (24 KB) 173 and 154; 8192 columns of bf16 (32 KB) 192 and 215.  And rows enough
// to fill the slots more than once: 1200 rows of 48 KB take 22 us staged, 19 us not,
// 2400 rows 41 and 44.
constexpr int kStagedRowBytes = 40 * 1024;
constexpr int64_t kStagedRows = 2048;

// Adds the rows of one input to a slot.
void stage_input(Staging &in, const Row &r, int hidden, int each) {
  const int i = in.count++;
  in.src[i] = static_cast<const uint8_t *>(r.p);
  in.pitch[i] = r.stride * each;
  in.bytes[i] = (uint32_t)(hidden * each);
  in.slot_bytes += hidden * each;
}

bool stage_rows(Staging &in, Plan &p, int hidden, int64_t rows, bool backward, int *blocks) {
  const int places = !backward || hidden <= 8 * 2 * staged_threads(2, true) ? 2 : 4;
  const int most = staged_threads(places, backward);
  const int threads = (hidden / 8 + 32 * places - 1) / (32 * places) * 32;
  in.slot_bytes = (in.slot_bytes + 127) / 128 * 128;
  const int per_sm = std::max(1, std::min(most / threads, kStagedBytes / (2 * in.slot_bytes)));
  in.stages = std::min(kMaxStages, kStagedBytes / per_sm / in.slot_bytes);
  if (threads > most || in.stages < 2) return false;
  in.err = device_error_word();
  in.timeout_ns = wait_timeout_ns();
  if (!in.err) return false;
  p.vpt = places, p.threads = threads;
  *blocks = (int)std::min<int64_t>(rows, (int64_t)num_sms() * per_sm);
  return true;
}

template <auto kernel, typename Args>
int launch_staged(const Args &a, const Plan &p, int blocks, int trace, cudaStream_t s) {
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedBytes);
    cudaGetLastError();
  });
  if (attr_err[dev] != cudaSuccess) return MUON_ERR_CUDA;
  trace_before(trace, s);
  kernel<<<blocks, p.threads, a.in.stages * a.in.slot_bytes, s>>>(a);
  return trace_after(trace, s);
}

template <typename R, typename B>
int launch_fwd(FwdArgs &a, bool vec, cudaStream_t s) {
  const Plan p = plan_rows(a.hidden, vec, false);
  if (p.w == 8 && p.vpt == kPlaces && a.block.p && a.normed.p && a.w_post && a.w_pre && a.rows >= kStagedRows) {
    stage_input(a.in, a.residual, a.hidden, sizeof(R));
    stage_input(a.in, a.block, a.hidden, sizeof(B));
    if (a.gate.p) stage_input(a.in, a.gate, a.hidden, sizeof(B));
    Plan q = p;
    int blocks = 0;
    if ((a.in.slot_bytes >= kStagedRowBytes || p.threads > max_threads(8, kPlaces, false)) &&
        stage_rows(a.in, q, a.hidden, a.rows, false, &blocks)) {
      constexpr int T = staged_threads(2, false), trace = kTraceBlockNormStaged;
      if (a.gate.p)
        return launch_staged<block_norm_kernel<R, B, 8, 2, T, FULL_ROW_GATE, true>>(a, q, blocks, trace, s);
      if (a.shared_gate)
        return launch_staged<block_norm_kernel<R, B, 8, 2, T, FULL_SHARED_GATE, true>>(a, q, blocks, trace, s);
      return launch_staged<block_norm_kernel<R, B, 8, 2, T, FULL, true>>(a, q, blocks, trace, s);
    }
  }
  if (p.w == 8 && p.vpt == 1) return launch_fwd_as<R, B, 8, 1>(a, p, s);
  if (p.w == 8)
    return p.threads <= max_threads(8, kPlaces, false) ? launch_fwd_as<R, B, 8, kPlaces>(a, p, s)
                                                          : launch_fwd_as<R, B, 8, kPlaces, kWideThreads>(a, p, s);
  if (p.vpt == 4) return launch_fwd_as<R, B, 1, 4>(a, p, s);
  return p.vpt == 8 ? launch_fwd_as<R, B, 1, 8>(a, p, s) : launch_fwd_as<R, B, 1, 16>(a, p, s);
}

// everything present: the forms other than ANY
bool full_backward(const BwdArgs &a) {
  return a.dresidual_out.p && a.dnormed.p && a.block.p && a.w_post && a.w_pre && a.dresidual.p && a.dblock.p &&
         !a.gate.p == !a.dgate.p;
}

template <typename R, typename B, int W, int VPT, int THREADS = max_threads(W, VPT, true)>
int launch_bwd_as(const BwdArgs &a, const Plan &p, cudaStream_t s) {
  auto go = [&](auto *kernel) { return launch_rows(kernel, a, p, true, kTraceBlockNormBwd, s); };
  // bf16 branches of two places a thread and up to 384 threads are always staged
  constexpr bool all_forms = !(W == 8 && VPT == kPlaces && THREADS == max_threads(W, VPT, true) && sizeof(B) == 2);
  if constexpr (all_forms)
    if (full_backward(a)) {
      if (a.gate.p) return go(block_norm_backward_kernel<R, B, W, VPT, THREADS, FULL_ROW_GATE>);
      if (a.shared_gate) return go(block_norm_backward_kernel<R, B, W, VPT, THREADS, FULL_SHARED_GATE>);
      return go(block_norm_backward_kernel<R, B, W, VPT, THREADS, FULL>);
    }
  return go(block_norm_backward_kernel<R, B, W, VPT, THREADS, ANY>);
}

template <typename R, typename B, int PLACES, int T = staged_threads(PLACES, true)>
int launch_staged_as(const BwdArgs &a, const Plan &p, int blocks, cudaStream_t s) {
  constexpr int trace = kTraceBlockNormBwdStaged;
  if (a.gate.p)
    return launch_staged<block_norm_backward_kernel<R, B, 8, PLACES, T, FULL_ROW_GATE, true>>(a, p, blocks, trace, s);
  if (a.shared_gate)
    return launch_staged<block_norm_backward_kernel<R, B, 8, PLACES, T, FULL_SHARED_GATE, true>>(a, p, blocks, trace, s);
  return launch_staged<block_norm_backward_kernel<R, B, 8, PLACES, T, FULL, true>>(a, p, blocks, trace, s);
}

template <typename R, typename B>
int launch_bwd(BwdArgs &a, bool vec, void *dw_pre, void *dw_post, void *dgate, cudaStream_t s) {
  Plan p = plan_rows(a.hidden, vec, true);
  int st, blocks = (int)(groups_of(p, a.rows, true) / p.rows_per_cta);
  bool staged = p.w == 8 && p.vpt == kPlaces && full_backward(a);
  if (staged) {
    stage_input(a.in, a.dresidual_out, a.hidden, sizeof(R));
    stage_input(a.in, a.residual, a.hidden, sizeof(R));
    stage_input(a.in, a.dnormed, a.hidden, sizeof(B));
    stage_input(a.in, a.block, a.hidden, sizeof(B));
    if (a.gate.p) stage_input(a.in, a.gate, a.hidden, sizeof(B));
    staged = stage_rows(a.in, p, a.hidden, a.rows, true, &blocks);
  }
  if (staged) {
    st = p.vpt == 2 ? launch_staged_as<R, B, 2>(a, p, blocks, s) : launch_staged_as<R, B, 4>(a, p, blocks, s);
  } else if (p.w == 8 && p.vpt == 1) st = launch_bwd_as<R, B, 8, 1>(a, p, s);
  else if (p.w == 8 && p.threads <= max_threads(8, kPlaces, true)) st = launch_bwd_as<R, B, 8, kPlaces>(a, p, s);
  else if (p.w == 8) st = launch_bwd_as<R, B, 8, kPlaces, kWideThreads>(a, p, s);
  else if (p.vpt == 4) st = launch_bwd_as<R, B, 1, 4>(a, p, s);
  else if (p.vpt == 8) st = launch_bwd_as<R, B, 1, 8>(a, p, s);
  else st = launch_bwd_as<R, B, 1, 16>(a, p, s);
  if (st != MUON_OK || !a.partial) return st;
  trace_before(kTraceNormWeightSum, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.hidden + 31) / 32), 2);
  cfg.blockDim = dim3(32, 16);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, norm_weight_sum_kernel<B>, (const float *)a.partial, (int64_t)blocks, a.hidden,
      a.scale, static_cast<const B *>(a.w_post), static_cast<const B *>(a.shared_gate), static_cast<B *>(dw_pre),
      static_cast<B *>(dw_post), static_cast<B *>(dgate));
  if (e != cudaSuccess) {
    trace_after(kTraceNormWeightSum, s);
    return MUON_ERR_CUDA;
  }
  return trace_after(kTraceNormWeightSum, s);
}

bool bad_type(int t) { return t != MUON_BF16 && t != MUON_F32; }
uintptr_t size_of(int t) { return t == MUON_BF16 ? 2 : 4; }

}  // namespace

size_t block_norm_backward_workspace(int64_t rows, int64_t hidden) {
  // the larger of the two plans' groups (vector and element-wise access)
  const int64_t g = std::max(groups_of(plan_rows((int)hidden, true, true), rows, true),
                             groups_of(plan_rows((int)hidden, false, true), rows, true));
  return ((size_t)g * 2 * (size_t)hidden * sizeof(float) + 255) & ~size_t(255);
}

}  // namespace muon

using namespace muon;

extern "C" {

int muon_block_norm(const muon_block_norm_args *a, muon_stream_t stream) {
  if (!a || a->rows < 0 || a->hidden < 1 || bad_type(a->residual_type) || bad_type(a->branch_type))
    return MUON_ERR_INVALID_ARG;
  if (a->hidden > kMaxHidden || a->rows > (int64_t(1) << 31) - 1 ||
      (a->residual_type == MUON_BF16 && a->branch_type == MUON_F32))
    return MUON_ERR_UNSUPPORTED;
  if (!(a->eps >= 0.f) || !isfinite(a->eps) || !isfinite(a->scale)) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0) return MUON_OK;
  if (!a->residual || (!a->block && !a->normed) || (a->block && !a->residual_out)) return MUON_ERR_INVALID_ARG;
  const int64_t h = a->hidden;
  if (a->residual_stride < h || (a->block && (a->block_stride < h || a->residual_out_stride < h)) ||
      (a->normed && a->normed_stride < h) || (a->block && a->gate && a->gate_stride != 0 && a->gate_stride < h))
    return MUON_ERR_INVALID_ARG;
  if (!on_elements({a->residual, a->residual_out}, size_of(a->residual_type)) ||
      !on_elements({a->block, a->w_post, a->gate, a->w_pre, a->normed}, size_of(a->branch_type)) ||
      !on_elements({a->rstd_post, a->rstd_pre}, 4))
    return MUON_ERR_UNSUPPORTED;
  FwdArgs k{};
  k.residual = {a->residual, a->residual_stride};
  k.block = {a->block, a->block_stride};
  const void *gate = a->block ? a->gate : nullptr;
  if (a->gate_stride) k.gate = {gate, a->gate_stride};
  else k.shared_gate = gate;
  k.residual_out = {a->residual_out, a->residual_out_stride};
  k.normed = {a->normed, a->normed_stride};
  k.w_post = a->block ? a->w_post : nullptr;
  k.w_pre = a->w_pre;
  k.rstd_post = a->rstd_post;
  k.rstd_pre = a->rstd_pre;
  k.rows = a->rows;
  k.hidden = (int)h;
  k.scale = a->scale;
  k.eps = a->eps;
  const int rt = a->residual_type, bt = a->branch_type;
  const bool vec = h % 8 == 0 && vec_row(a->residual, a->residual_stride, rt) &&
                   vec_row(k.block.p, a->block_stride, bt) && vec_row(gate, a->gate_stride, bt) &&
                   vec_row(k.block.p ? a->residual_out : nullptr, a->residual_out_stride, rt) &&
                   vec_row(a->normed, a->normed_stride, bt) && vec_row(k.w_post, 0, bt) && vec_row(a->w_pre, 0, bt);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rt == MUON_BF16) return launch_fwd<__nv_bfloat16, __nv_bfloat16>(k, vec, s);
  if (bt == MUON_BF16) return launch_fwd<float, __nv_bfloat16>(k, vec, s);
  return launch_fwd<float, float>(k, vec, s);
}

size_t muon_block_norm_backward_workspace_bytes(int64_t rows, int64_t hidden) {
  if (rows < 1 || hidden < 1 || hidden > kMaxHidden) return 0;
  return block_norm_backward_workspace(rows, hidden);
}

int muon_block_norm_backward(const muon_block_norm_backward_args *a, void *workspace, size_t workspace_bytes,
                             muon_stream_t stream) {
  if (!a || a->rows < 0 || a->hidden < 1 || bad_type(a->residual_type) || bad_type(a->branch_type))
    return MUON_ERR_INVALID_ARG;
  if (a->hidden > kMaxHidden || a->rows > (int64_t(1) << 31) - 1 ||
      (a->residual_type == MUON_BF16 && a->branch_type == MUON_F32))
    return MUON_ERR_UNSUPPORTED;
  if (!isfinite(a->scale) || a->gate_stride < 0) return MUON_ERR_INVALID_ARG;
  const int64_t h = a->hidden;
  const bool pre = a->dnormed != nullptr, post = a->block != nullptr;
  const bool gate = post && a->gate != nullptr, gate_rows = gate && a->gate_stride != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rt = a->residual_type, bt = a->branch_type;
  if (a->rows == 0) {   // sums over no rows
    const size_t bytes = (size_t)h * (bt == MUON_BF16 ? 2 : 4);
    void *const sums[3] = {a->dw_pre, a->dw_post, gate_rows ? nullptr : a->dgate};
    for (void *d : sums)
      if (d && cudaMemsetAsync(d, 0, bytes, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if ((!pre && !a->dresidual_out) || (pre && (!a->residual || !a->rstd_pre)) || (post && !a->rstd_post) ||
      (!pre && a->dw_pre) || (!post && (a->dw_post || a->dblock)) || (!gate && a->dgate) ||
      (!a->dresidual && !a->dblock && !a->dw_pre && !a->dw_post && !a->dgate))
    return MUON_ERR_INVALID_ARG;
  if ((a->dresidual_out && a->dresidual_out_stride < h) ||
      (pre && (a->dnormed_stride < h || a->residual_stride < h)) || (post && a->block_stride < h) ||
      (gate_rows && a->gate_stride < h) || (a->dresidual && a->dresidual_stride < h) ||
      (a->dblock && a->dblock_stride < h) || (gate_rows && a->dgate && a->dgate_stride < h))
    return MUON_ERR_INVALID_ARG;
  if (!on_elements({a->dresidual_out, a->residual, a->dresidual}, size_of(rt)) ||
      !on_elements({a->dnormed, a->block, a->w_post, a->gate, a->w_pre, a->dblock, a->dw_post, a->dgate, a->dw_pre},
                   size_of(bt)) ||
      !on_elements({a->rstd_post, a->rstd_pre}, 4))
    return MUON_ERR_UNSUPPORTED;
  BwdArgs k{};
  k.dresidual_out = {a->dresidual_out, a->dresidual_out_stride};
  k.dnormed = {a->dnormed, a->dnormed_stride};
  if (pre) k.residual = {a->residual, a->residual_stride};
  k.block = {a->block, a->block_stride};
  if (gate_rows) k.gate = {a->gate, a->gate_stride};
  else if (gate) k.shared_gate = a->gate;
  k.dresidual = {a->dresidual, a->dresidual_stride};
  k.dblock = {a->dblock, a->dblock_stride};
  k.dgate = {gate_rows ? a->dgate : nullptr, a->dgate_stride};
  k.w_post = post ? a->w_post : nullptr;
  k.w_pre = pre ? a->w_pre : nullptr;
  k.rstd_post = a->rstd_post;
  k.rstd_pre = a->rstd_pre;
  k.rows = a->rows;
  k.hidden = (int)h;
  k.scale = a->scale;
  void *dg = gate_rows ? nullptr : a->dgate;
  const bool sums = a->dw_pre || a->dw_post || dg;
  const bool vec = h % 8 == 0 && vec_row(a->dresidual_out, a->dresidual_out_stride, rt) &&
                   vec_row(a->dnormed, a->dnormed_stride, bt) &&
                   vec_row(pre ? a->residual : nullptr, a->residual_stride, rt) &&
                   vec_row(a->block, a->block_stride, bt) && vec_row(gate ? a->gate : nullptr, a->gate_stride, bt) &&
                   vec_row(a->dresidual, a->dresidual_stride, rt) && vec_row(a->dblock, a->dblock_stride, bt) &&
                   vec_row(k.dgate.p, a->dgate_stride, bt) && vec_row(k.w_post, 0, bt) && vec_row(k.w_pre, 0, bt);
  const size_t need = block_norm_backward_workspace(a->rows, h);
  void *owned = nullptr;
  if (sums) {
    if (workspace) {
      if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_ERR_INVALID_ARG;
      if (workspace_bytes < need) return MUON_ERR_NO_MEMORY;
      k.partial = static_cast<float *>(workspace);
    } else {
      if (alloc_async(&owned, need, s) != cudaSuccess) {
        cudaGetLastError();
        return MUON_ERR_NO_MEMORY;
      }
      k.partial = static_cast<float *>(owned);
    }
  }
  int st;
  if (rt == MUON_BF16) st = launch_bwd<__nv_bfloat16, __nv_bfloat16>(k, vec, a->dw_pre, a->dw_post, dg, s);
  else if (bt == MUON_BF16) st = launch_bwd<float, __nv_bfloat16>(k, vec, a->dw_pre, a->dw_post, dg, s);
  else st = launch_bwd<float, float>(k, vec, a->dw_pre, a->dw_post, dg, s);
  if (owned && cudaFreeAsync(owned, s) != cudaSuccess && st == MUON_OK) st = MUON_ERR_CUDA;
  return st;
}

}  // extern "C"
