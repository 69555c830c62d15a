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
// One pass over memory: a row lives in the registers of one thread group
// between its two reductions (the second depends on the first through r' or
// dr').  All sums are fp32 and in a fixed order (no atomics): the weight
// gradients accumulate in registers over the rows a group takes, each group
// writes its sums, and a second kernel adds them.
#include <algorithm>

#include "common.cuh"

namespace muon {
namespace {

constexpr int kMaxHidden = 16384;
constexpr int kRowsPerCta = 4;   // rows of one CTA where a warp holds a whole row

// Largest block of an instance.  The backward kernel keeps three sums per
// column in registers, so its blocks are smaller (768 threads leave it 85
// registers, 512 leave 128).
constexpr int max_threads(int w, int vpt, bool backward) {
  if (w == 1) return vpt == 32 ? 512 : backward && vpt == 4 ? 512 : 1024;
  return vpt == 1 ? (backward ? 768 : 256) : 512;
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

// W consecutive elements: W = 8 moves 16-byte vectors, W = 1 single elements
// (widths or strides that are not multiples of 8, unaligned pointers).
template <typename T, int W>
__device__ __forceinline__ void load(const T *src, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = to_f(*src);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 x = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = reinterpret_cast<const float4 *>(src)[i];
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  }
}

template <typename T, int W>
__device__ __forceinline__ void store(T *dst, const float (&v)[W]) {
  if constexpr (W == 1) {
    from_f(dst, v[0]);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<float4 *>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// Sum over the threads of a row (blockDim.x, a multiple of 32); with one warp
// per row no shared memory and no barrier is used.  Successive sums alternate
// between two buffers, so one barrier each is enough: a buffer is written
// again only after a barrier that every reader of its last sum has passed.
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? buf[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct FwdArgs {
  Row residual, block, gate;   // gate stride 0: one gate for all rows
  RowOut residual_out, normed;
  const void *w_post, *w_pre;
  float *rstd_post, *rstd_pre;
  int64_t rows;
  int hidden;
  float scale, eps;
};

template <typename R, typename B, int W, int VPT>
__global__ void __launch_bounds__(max_threads(W, VPT, false)) block_norm_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  if (row >= a.rows) return;   // only where a warp holds a row (no barriers)
  const R *res = static_cast<const R *>(a.residual.p) + row * a.residual.stride;
  float r[VPT][W];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * W;
    if (c < a.hidden) load<R, W>(res + c, r[i]);
  }
  if (a.block.p) {
    const B *blk = static_cast<const B *>(a.block.p) + row * a.block.stride;
    const B *gate = static_cast<const B *>(a.gate.p) + (a.gate.p ? row * a.gate.stride : 0);
    float b[VPT][W], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * W;
      if (c < a.hidden) {
        load<B, W>(blk + c, b[i]);
#pragma unroll
        for (int j = 0; j < W; ++j) ss = fmaf(b[i][j], b[i][j], ss);
      }
    }
    const float q = 1.f / sqrtf(row_sum(ss, red[0]) / (float)a.hidden + a.eps);
    if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[row] = q;
    R *out = static_cast<R *>(a.residual_out.p) + row * a.residual_out.stride;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * W;
      if (c < a.hidden) {
        float w[W], g[W];
        if (a.w_post) load<B, W>(static_cast<const B *>(a.w_post) + c, w);
        if (a.gate.p) load<B, W>(gate + c, g);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          float n = b[i][j] * q;
          if (a.w_post) n *= w[j];
          if (a.gate.p) n *= g[j];
          r[i][j] = fmaf(a.scale, n, r[i][j]);
        }
        store<R, W>(out + c, r[i]);
      }
    }
  }
  if (!a.normed.p) return;
  // y is formed from r' before its rounding to the stream's type
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if ((threadIdx.x + i * blockDim.x) * W < a.hidden)
#pragma unroll
      for (int j = 0; j < W; ++j) ss = fmaf(r[i][j], r[i][j], ss);
  const float p = 1.f / sqrtf(row_sum(ss, red[1]) / (float)a.hidden + a.eps);
  if (threadIdx.x == 0 && a.rstd_pre) a.rstd_pre[row] = p;
  B *y = static_cast<B *>(a.normed.p) + row * a.normed.stride;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * W;
    if (c < a.hidden) {
      float w[W], v[W];
      if (a.w_pre) load<B, W>(static_cast<const B *>(a.w_pre) + c, w);
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = a.w_pre ? r[i][j] * p * w[j] : r[i][j] * p;
      store<B, W>(y + c, v);
    }
  }
}

struct BwdArgs {
  Row dresidual_out, dnormed, residual, block, gate;
  RowOut dresidual, dblock, dgate;   // dgate here: one row per token
  const void *w_post, *w_pre;
  const float *rstd_post, *rstd_pre;
  float *partial;                    // [groups][3][hidden]: dw_pre, dw_post, shared dgate
  int64_t rows;
  int hidden;
  float scale;
  int want_pre, want_post, want_gate;   // which sums over rows are wanted
};

template <typename R, typename B, int W, int VPT>
__global__ void __launch_bounds__(max_threads(W, VPT, true)) block_norm_backward_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float red[2][32];
  const int64_t group = blockIdx.x * (int64_t)blockDim.y + threadIdx.y, groups = gridDim.x * (int64_t)blockDim.y;
  const float inv_h = 1.f / (float)a.hidden;
  int turn = 0;   // which buffer the next sum uses
  float dwp[VPT][W] = {}, dwq[VPT][W] = {}, dgs[VPT][W] = {};
  for (int64_t row = group; row < a.rows; row += groups) {
    float dr[VPT][W];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * W;
#pragma unroll
      for (int j = 0; j < W; ++j) dr[i][j] = 0.f;
      if (c < a.hidden && a.dresidual_out.p)
        load<R, W>(static_cast<const R *>(a.dresidual_out.p) + row * a.dresidual_out.stride + c, dr[i]);
    }
    if (a.dnormed.p) {
      const float p = a.rstd_pre[row];
      float t[VPT][W], xh[VPT][W], sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * W;
        if (c < a.hidden) {
          float dy[W], w[W];
          load<B, W>(static_cast<const B *>(a.dnormed.p) + row * a.dnormed.stride + c, dy);
          load<R, W>(static_cast<const R *>(a.residual.p) + row * a.residual.stride + c, xh[i]);
          if (a.w_pre) load<B, W>(static_cast<const B *>(a.w_pre) + c, w);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            xh[i][j] *= p;
            dwp[i][j] = fmaf(dy[j], xh[i][j], dwp[i][j]);
            t[i][j] = a.w_pre ? dy[j] * w[j] : dy[j];
            sum = fmaf(t[i][j], xh[i][j], sum);
          }
        }
      }
      const float mean = row_sum(sum, red[turn]) * inv_h;
      turn ^= 1;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if ((threadIdx.x + i * blockDim.x) * W < a.hidden)
#pragma unroll
          for (int j = 0; j < W; ++j) dr[i][j] = fmaf(p, fmaf(-xh[i][j], mean, t[i][j]), dr[i][j]);
    }
    if (a.dresidual.p)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * W;
        if (c < a.hidden) store<R, W>(static_cast<R *>(a.dresidual.p) + row * a.dresidual.stride + c, dr[i]);
      }
    if (!a.block.p) continue;
    const float q = a.rstd_post[row];
    float bh[VPT][W], sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * W;
      if (c < a.hidden) {
        float w[W], g[W];
        load<B, W>(static_cast<const B *>(a.block.p) + row * a.block.stride + c, bh[i]);
        if (a.w_post) load<B, W>(static_cast<const B *>(a.w_post) + c, w);
        if (a.gate.p) load<B, W>(static_cast<const B *>(a.gate.p) + row * a.gate.stride + c, g);
        float dg[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          bh[i][j] *= q;
          const float sdr = a.scale * dr[i][j];
          const float wj = a.w_post ? w[j] : 1.f;
          dg[j] = sdr * bh[i][j] * wj;
          dgs[i][j] += dg[j];
          const float dn = a.gate.p ? sdr * g[j] : sdr;
          dwq[i][j] = fmaf(dn, bh[i][j], dwq[i][j]);
          dr[i][j] = dn * wj;
          sum = fmaf(dr[i][j], bh[i][j], sum);
        }
        if (a.dgate.p) store<B, W>(static_cast<B *>(a.dgate.p) + row * a.dgate.stride + c, dg);
      }
    }
    const float mean = row_sum(sum, red[turn]) * inv_h;
    turn ^= 1;
    if (a.dblock.p)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * W;
        if (c < a.hidden) {
          float v[W];
#pragma unroll
          for (int j = 0; j < W; ++j) v[j] = q * fmaf(-bh[i][j], mean, dr[i][j]);
          store<B, W>(static_cast<B *>(a.dblock.p) + row * a.dblock.stride + c, v);
        }
      }
  }
  if (!a.partial) return;
  float *out = a.partial + group * 3 * a.hidden;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * W;
    if (c < a.hidden)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (a.want_pre) out[c + j] = dwp[i][j];
        if (a.want_post) out[a.hidden + c + j] = dwq[i][j];
        if (a.want_gate) out[2 * a.hidden + c + j] = dgs[i][j];
      }
  }
}

// out[s][c] = sum over groups of partial[group][s][c], in 16 interleaved
// partial sums that are then added in a fixed order.
template <typename B>
__global__ void __launch_bounds__(512) norm_weight_sum_kernel(const float *partial, int64_t groups, int hidden, B *d0,
                                                              B *d1, B *d2) {
  __shared__ float part[16][33];
  const int which = blockIdx.y;
  B *dst = which == 0 ? d0 : which == 1 ? d1 : d2;
  if (!dst) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < hidden)
    for (int64_t g = threadIdx.y; g < groups; g += 16) v += partial[(g * 3 + which) * hidden + c];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < hidden) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][threadIdx.x];
    from_f(dst + c, v);
  }
}

// Threads, and elements per thread, of a row.
struct Plan {
  int w, vpt, threads, rows_per_cta;
};

Plan plan_rows(int hidden, bool vec, bool backward) {
  Plan p{};
  p.w = vec ? 8 : 1;
  const int n = (hidden + p.w - 1) / p.w;
  const int small = vec ? 1 : 4, mid = vec ? 2 : 8, large = vec ? 4 : 32;
  p.vpt = n <= small * max_threads(p.w, small, backward) ? small
          : n <= mid * max_threads(p.w, mid, backward)   ? mid
                                                         : large;
  p.threads = (n + p.vpt - 1) / p.vpt;
  p.threads = (p.threads + 31) / 32 * 32;
  p.rows_per_cta = p.threads == 32 ? kRowsPerCta : 1;
  return p;
}
static_assert(8 * 4 * max_threads(8, 4, true) >= kMaxHidden && 32 * max_threads(1, 32, true) >= kMaxHidden,
              "every width has a plan");

inline bool vec_row(const void *p, int64_t stride, int type) {
  if (!p) return true;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % (type == MUON_BF16 ? 8 : 4) == 0;
}

int64_t backward_groups(const Plan &p, int64_t rows) {
  const int per_sm = std::max(1, std::min(2048 / (p.threads * p.rows_per_cta), p.threads >= 512 ? 1 : 8));
  const int64_t ctas = std::min<int64_t>((rows + p.rows_per_cta - 1) / p.rows_per_cta, (int64_t)num_sms() * per_sm);
  return ctas * p.rows_per_cta;
}

template <typename R, typename B>
int launch_fwd(const FwdArgs &a, bool vec, cudaStream_t s) {
  const Plan p = plan_rows(a.hidden, vec, false);
  const dim3 block(p.threads, p.rows_per_cta);
  const dim3 grid((unsigned)((a.rows + p.rows_per_cta - 1) / p.rows_per_cta));
  trace_before(kTraceBlockNorm, s);
  if (p.w == 8 && p.vpt == 1) block_norm_kernel<R, B, 8, 1><<<grid, block, 0, s>>>(a);
  else if (p.w == 8 && p.vpt == 2) block_norm_kernel<R, B, 8, 2><<<grid, block, 0, s>>>(a);
  else if (p.w == 8) block_norm_kernel<R, B, 8, 4><<<grid, block, 0, s>>>(a);
  else if (p.vpt == 4) block_norm_kernel<R, B, 1, 4><<<grid, block, 0, s>>>(a);
  else if (p.vpt == 8) block_norm_kernel<R, B, 1, 8><<<grid, block, 0, s>>>(a);
  else block_norm_kernel<R, B, 1, 32><<<grid, block, 0, s>>>(a);
  return trace_after(kTraceBlockNorm, s);
}

template <typename R, typename B>
int launch_bwd(const BwdArgs &a, bool vec, void *dw_pre, void *dw_post, void *dgate, cudaStream_t s) {
  const Plan p = plan_rows(a.hidden, vec, true);
  const int64_t groups = backward_groups(p, a.rows);
  const dim3 block(p.threads, p.rows_per_cta);
  const dim3 grid((unsigned)(groups / p.rows_per_cta));
  trace_before(kTraceBlockNormBwd, s);
  if (p.w == 8 && p.vpt == 1) block_norm_backward_kernel<R, B, 8, 1><<<grid, block, 0, s>>>(a);
  else if (p.w == 8 && p.vpt == 2) block_norm_backward_kernel<R, B, 8, 2><<<grid, block, 0, s>>>(a);
  else if (p.w == 8) block_norm_backward_kernel<R, B, 8, 4><<<grid, block, 0, s>>>(a);
  else if (p.vpt == 4) block_norm_backward_kernel<R, B, 1, 4><<<grid, block, 0, s>>>(a);
  else if (p.vpt == 8) block_norm_backward_kernel<R, B, 1, 8><<<grid, block, 0, s>>>(a);
  else block_norm_backward_kernel<R, B, 1, 32><<<grid, block, 0, s>>>(a);
  int st = trace_after(kTraceBlockNormBwd, s);
  if (st != MUON_OK || !a.partial) return st;
  trace_before(kTraceNormWeightSum, s);
  norm_weight_sum_kernel<B><<<dim3((unsigned)((a.hidden + 31) / 32), 3), dim3(32, 16), 0, s>>>(
      a.partial, groups, a.hidden, static_cast<B *>(dw_pre), static_cast<B *>(dw_post), static_cast<B *>(dgate));
  return trace_after(kTraceNormWeightSum, s);
}

bool bad_type(int t) { return t != MUON_BF16 && t != MUON_F32; }

}  // namespace

size_t block_norm_backward_workspace(int64_t rows, int64_t hidden) {
  // the larger of the two plans' groups (vector and element-wise access)
  const int64_t g = std::max(backward_groups(plan_rows((int)hidden, true, true), rows),
                             backward_groups(plan_rows((int)hidden, false, true), rows));
  return ((size_t)g * 3 * (size_t)hidden * sizeof(float) + 255) & ~size_t(255);
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
  FwdArgs k{};
  k.residual = {a->residual, a->residual_stride};
  k.block = {a->block, a->block_stride};
  k.gate = {a->block ? a->gate : nullptr, a->gate_stride};
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
                   vec_row(k.block.p, a->block_stride, bt) && vec_row(k.gate.p, a->gate_stride, bt) &&
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
  BwdArgs k{};
  k.dresidual_out = {a->dresidual_out, a->dresidual_out_stride};
  k.dnormed = {a->dnormed, a->dnormed_stride};
  k.residual = {a->residual, a->residual_stride};
  k.block = {a->block, a->block_stride};
  k.gate = {gate ? a->gate : nullptr, a->gate_stride};
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
  k.want_pre = a->dw_pre != nullptr;
  k.want_post = a->dw_post != nullptr;
  k.want_gate = a->dgate && !gate_rows;
  const bool sums = k.want_pre || k.want_post || k.want_gate;
  const bool vec = h % 8 == 0 && vec_row(a->dresidual_out, a->dresidual_out_stride, rt) &&
                   vec_row(a->dnormed, a->dnormed_stride, bt) &&
                   vec_row(pre ? a->residual : nullptr, a->residual_stride, rt) &&
                   vec_row(a->block, a->block_stride, bt) && vec_row(k.gate.p, a->gate_stride, bt) &&
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
  void *dg = k.want_gate ? a->dgate : nullptr;
  int st;
  if (rt == MUON_BF16) st = launch_bwd<__nv_bfloat16, __nv_bfloat16>(k, vec, a->dw_pre, a->dw_post, dg, s);
  else if (bt == MUON_BF16) st = launch_bwd<float, __nv_bfloat16>(k, vec, a->dw_pre, a->dw_post, dg, s);
  else st = launch_bwd<float, float>(k, vec, a->dw_pre, a->dw_post, dg, s);
  if (owned && cudaFreeAsync(owned, s) != cudaSuccess && st == MUON_OK) st = MUON_ERR_CUDA;
  return st;
}

}  // extern "C"
