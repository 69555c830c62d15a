// Softmax cross entropy from hidden states and a head matrix, and its gradients:
// argument checks, workspace, the order of the products (head_tc.cu) and the small
// kernels around them.
#include <math.h>

#include <algorithm>

#include "head_loss.cuh"

namespace muon {
namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxVocab = int64_t(1) << 30, kMaxHidden = int64_t(1) << 20;
// rows of one pass over W in the forward call: the partial statistics of a pass are 8 bytes per row and
// 256 vocabulary entries, 66 MB for a vocabulary of 128000, a copy of x that rows off 128 bytes need is 201 MB at a
// hidden size of 6144, and 16384 rows keep the tensor cores busy for 60 times the time that W's bytes take
constexpr int64_t kPassRows = 16384;

int check_shape(const HeadShape &h) {
  if (h.rows < 0 || h.vocab < 1 || h.hidden < 1) return MUON_ERR_INVALID_ARG;
  if (h.rows > kMaxRows || h.vocab > kMaxVocab || h.hidden > kMaxHidden || h.hidden % 8) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

#define MUON_TRY(expr)              \
  do {                              \
    const int _st = (expr);         \
    if (_st != MUON_OK) return _st; \
  } while (0)

// Joins a row's partial statistics, in a fixed order: 32 rows a block (lane = row, so that reads of a part are
// whole lines), the parts spread over the block's warps.
//   loss = ((c - z_target log2(e)) + log2 s) ln 2;  of far logits (z_largest - z_target) + ln s
// c is a whole number and not the largest logit's exponent, so a likely target's loss is the difference of two numbers of
// up to 1, one of which has the exponentials' errors (2^-22, and a rounding of exponents up to 100): it is within 2^-18
// absolutely, whatever its size, and what would be below 0 by that is 0.
constexpr int kJoinWarps = 32, kJoinAhead = 8;   // kJoinAhead parts of a warp are loaded together
__global__ void __launch_bounds__(32 * kJoinWarps)
    head_join_kernel(const float2 *parts, int64_t num, const float *target_logit, const int64_t *targets, int64_t rows,
                     int64_t vocab, float *loss, float *lse, unsigned *err) {
  __shared__ float2 part[kJoinWarps][32];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x * 32ll + lane;
  wait_for_previous_grid();
  let_next_grid_start();
  float m = -INFINITY, s = 0.f;   // the largest c so far
  if (row < rows) {
    for (int64_t c = wp; c < num; c += kJoinWarps * kJoinAhead) {
      float2 v[kJoinAhead];
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i)
        v[i] = c + i * kJoinWarps < num ? __ldcs(parts + (c + i * kJoinWarps) * rows + row) : make_float2(-INFINITY, 0.f);
      float most = m;
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) most = fmaxf(most, v[i].x);
      // -inf on both sides (a part beyond the vocabulary's end has no sum) leaves the sum as it is
      s *= m == most ? 1.f : exp2f(m - most);
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) s = fmaf(v[i].y, v[i].x == most ? 1.f : exp2f(v[i].x - most), s);
      m = most;
    }
  }
  part[wp][lane] = make_float2(m, s);
  __syncthreads();
  if (wp || row >= rows) return;
  for (int i = 1; i < kJoinWarps; ++i) {
    const float2 v = part[i][lane];
    const float most = fmaxf(m, v.x);
    const float a = m == most ? 1.f : exp2f(m - most), b = v.x == most ? 1.f : exp2f(v.x - most);
    s = s * a + v.y * b;
    m = most;
  }
  const float ls = log2f(s);
  // 1 / kLog2e in two parts, of the very kLog2e that the logits were multiplied by, so that lse is rounded once
  constexpr float kLn2 = (float)(1.0 / kLog2e), kLn2Rest = (float)(1.0 / kLog2e - kLn2);
  const bool far = is_far(m);
  if (lse) lse[row] = far ? fmaf(ls, kLn2, far_logit(m)) : fmaf(m, kLn2, fmaf(m, kLn2Rest, ls * kLn2));
  if (!loss) return;
  const int64_t t = targets[row];
  if (t >= vocab) atomicOr(err, kErrDevice);
  float v = t < 0 ? 0.f : NAN;
  if (t >= 0 && t < vocab) {
    const float zt = target_logit[row];
    v = far ? fmaf(ls, kLn2, far_logit(m) - zt) : (fmaf(-zt, kLog2e, m) + ls) * kLn2;
    if (v < 0.f) v = 0.f;   // a NaN stays
  }
  loss[row] = v;
}

// The rows' factors, and x without the rows that take no part (0 times a NaN would reach dW, and d): dense, `cols`
// wide (hidden rounded up to 64, zeros behind it).  16 bytes a thread and step.
__global__ void __launch_bounds__(256)
    head_rows_kernel(const float *dloss, const float *dlse, const float *lse, const int64_t *targets, int64_t rows,
                     int64_t vocab, const uint4 *x, int64_t ldx, int hidden8, int cols8, HeadRow *out, uint4 *xc,
                     unsigned *err) {
  wait_for_previous_grid();
  let_next_grid_start();
  const int64_t row = blockIdx.x;
  const int64_t t = targets[row];
  const bool part = t >= 0 && t < vocab;
  if (threadIdx.x == 0) {
    if (t >= vocab) atomicOr(err, kErrDevice);
    HeadRow r{0.f, 0.f, 0.f, -1};
    if (part) r = {lse[row], dloss[row] + (dlse ? dlse[row] : 0.f), dloss[row], (int)t};
    out[row] = r;
  }
  for (int c = threadIdx.x; c < cols8; c += 256)
    xc[row * cols8 + c] = part && c < hidden8 ? x[row * ldx + c] : make_uint4(0u, 0u, 0u, 0u);
}

// x in rows that begin on 128 bytes: the tensor core's loads take rows of 128 bytes, and one that lies across two lines
// is two requests, for every vocabulary tile again (4096 rows of 3000 over 30000 entries: 483 us, 391 with the copy).
__global__ void __launch_bounds__(256)
    head_align_kernel(const uint4 *x, int64_t ldx, int hidden8, int cols8, uint4 *xa) {
  wait_for_previous_grid();
  let_next_grid_start();
  const int64_t row = blockIdx.x;
  for (int c = threadIdx.x; c < cols8; c += 256)
    xa[row * cols8 + c] = c < hidden8 ? x[row * ldx + c] : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}

// dx from its parts' sums, added in order; 8 columns a thread and step
__global__ void __launch_bounds__(256)
    head_dx_kernel(const float4 *acc, int splits, int64_t rows, int hidden8, uint4 *dx, int64_t lddx8) {
  wait_for_previous_grid();
  let_next_grid_start();
  const int64_t n = rows * hidden8;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int s = 0; s < splits; ++s) {
      const float4 u = __ldcs(acc + (s * n + i) * 2), v = __ldcs(acc + (s * n + i) * 2 + 1);
      a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
      b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
    }
    const int64_t row = i / hidden8, c = i - row * hidden8;
    dx[row * lddx8 + c] = make_uint4(pack_pair(a.x, a.y), pack_pair(a.z, a.w), pack_pair(b.x, b.y), pack_pair(b.z, b.w));
  }
}

// a launch that may start while the kernel before it ends (each waits for it before it reads or writes)
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), unsigned blocks, unsigned threads, int trace_kind, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_before(trace_kind, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  const int st = trace_after(trace_kind, s);
  return e == cudaSuccess ? st : MUON_ERR_CUDA;
}

// `need` bytes: the caller's workspace, or the library's own (freed by done())
struct Scratch {
  uint8_t *p = nullptr;
  bool owned = false;
  cudaStream_t s;

  explicit Scratch(cudaStream_t stream) : s(stream) {}

  int take(void *workspace, size_t bytes, size_t need) {
    if (workspace) {
      if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_ERR_INVALID_ARG;
      if (bytes < need) return MUON_ERR_NO_MEMORY;
      p = static_cast<uint8_t *>(workspace);
      return MUON_OK;
    }
    void *q = nullptr;
    if (alloc_async(&q, need, s) != cudaSuccess) {
      cudaGetLastError();
      return MUON_ERR_NO_MEMORY;
    }
    p = static_cast<uint8_t *>(q);
    owned = true;
    return MUON_OK;
  }

  int done(int st) {
    if (owned && cudaFreeAsync(p, s) != cudaSuccess && st == MUON_OK) return MUON_ERR_CUDA;
    return st;
  }
};

HeadShape pass_of(const HeadShape &h) { return {std::min(h.rows, kPassRows), h.vocab, h.hidden}; }

size_t parts_bytes(const HeadShape &h) { return align256((size_t)head_parts(h) * h.rows * sizeof(float2)); }

// Is x copied first?  Where its rows do not begin on 128 bytes, and are read often enough: from two row tiles of a CTA
// and two tiles a pair of CTAs on.
bool off_lines(const void *x, int64_t ldx) { return ldx % 64 || (reinterpret_cast<uintptr_t>(x) & 127u); }
bool read_often(const HeadShape &pass) {
  return pass.rows > 128 && cdiv(pass.rows, 256) * cdiv(pass.vocab, 256) >= num_sms();
}

// the forward call's workspace: offsets and the whole.  `off`: x may have to be copied (a pass of fewer rows is read no
// more often than the first, and its rows begin where the first's do).
struct ForwardRegions {
  size_t parts, xa, bytes;

  ForwardRegions(const HeadShape &h, bool off) {
    const HeadShape pass = pass_of(h), last{h.rows % kPassRows, h.vocab, h.hidden};
    // a shorter last pass may cut the vocabulary finer
    const size_t rest = h.rows > kPassRows && last.rows ? parts_bytes(last) : 0;
    parts = align256((size_t)pass.rows * 4);   // behind the targets' logits
    xa = parts + std::max(parts_bytes(pass), rest);
    bytes = xa + (off && read_often(pass) ? align256((size_t)pass.rows * cdiv(h.hidden, 64) * 128) : 0);
  }
};

int forward(const HeadShape &h, const void *x, int64_t ldx, const void *w, const int64_t *targets, float *loss,
            float *lse, uint8_t *scratch, cudaStream_t s) {
  unsigned *err = device_error_word();
  if (!err) return MUON_ERR_CUDA;
  const bool off = off_lines(x, ldx);
  const ForwardRegions g(h, off);
  float *target_logit = reinterpret_cast<float *>(scratch);
  float2 *parts = reinterpret_cast<float2 *>(scratch + g.parts);
  const int64_t cols = cdiv(h.hidden, 64) * 64;
  for (int64_t r = 0; r < h.rows; r += kPassRows) {
    const HeadShape pass{std::min(kPassRows, h.rows - r), h.vocab, h.hidden};
    const void *xr = static_cast<const uint8_t *>(x) + r * ldx * 2;
    int64_t ld = ldx;
    if (off && read_often(pass)) {
      MUON_TRY(launch_after(head_align_kernel, (unsigned)pass.rows, 256, kTraceHeadRows, s,
                            static_cast<const uint4 *>(xr), ldx / 8, (int)(h.hidden / 8), (int)(cols / 8),
                            reinterpret_cast<uint4 *>(scratch + g.xa)));
      xr = scratch + g.xa;
      ld = cols;
    }
    MUON_TRY(head_stats(pass, xr, ld, w, targets + r, parts, target_logit, s));
    MUON_TRY(launch_after(head_join_kernel, (unsigned)cdiv(pass.rows, 32), 32 * kJoinWarps, kTraceHeadJoin, s, parts,
                          head_parts(pass), target_logit, targets + r, pass.rows, h.vocab, loss ? loss + r : nullptr,
                          lse ? lse + r : nullptr, err));
  }
  return MUON_OK;
}

// the backward call's workspace
struct Regions {
  HeadPlan plan;
  int64_t xc_cols;
  size_t row, xc, d, acc, bytes;   // offsets and the whole

  Regions(const HeadShape &h, bool need_dx, bool need_dw) : plan(head_plan(h, need_dx, need_dw)) {
    xc_cols = cdiv(h.hidden, 64) * 64;
    row = 0;
    xc = row + align256((size_t)h.rows * sizeof(HeadRow));
    d = xc + align256((size_t)h.rows * xc_cols * 2);
    acc = d + align256((size_t)h.rows * plan.width() * 2);
    const bool sums = need_dx && (plan.pieces > 1 || plan.splits > 1);
    bytes = acc + (sums ? align256((size_t)plan.splits * h.rows * h.hidden * 4) : 0);
  }
};

int backward(const HeadShape &h, const Regions &g, const float *dloss, const float *dlse, const void *x, int64_t ldx,
             const void *w, const int64_t *targets, const float *lse, void *dx, int64_t lddx, void *dweight,
             uint8_t *scratch, cudaStream_t s) {
  unsigned *err = device_error_word();
  if (!err) return MUON_ERR_CUDA;
  HeadRow *row = reinterpret_cast<HeadRow *>(scratch + g.row);
  uint4 *xc = reinterpret_cast<uint4 *>(scratch + g.xc);
  void *d = scratch + g.d;
  float *acc = reinterpret_cast<float *>(scratch + g.acc);
  const int hidden8 = (int)(h.hidden / 8);
  MUON_TRY(launch_after(head_rows_kernel, (unsigned)h.rows, 256, kTraceHeadRows, s, dloss, dlse, lse, targets, h.rows,
                        h.vocab, static_cast<const uint4 *>(x), ldx / 8, hidden8, (int)(g.xc_cols / 8), row, xc, err));
  for (int64_t v0 = 0; v0 < h.vocab; v0 += g.plan.width()) {
    MUON_TRY(head_dlogits(h, g.plan, v0, xc, g.xc_cols, w, row, d, s));
    MUON_TRY(head_grads(h, g.plan, v0, v0 == 0, d, w, xc, g.xc_cols, dx, lddx, acc, dweight, s));
  }
  if (dx && (g.plan.pieces > 1 || g.plan.splits > 1)) {
    const unsigned blocks = (unsigned)std::min<int64_t>(cdiv(h.rows * hidden8, 256), 8ll * num_sms());
    MUON_TRY(launch_after(head_dx_kernel, blocks, 256, kTraceHeadDx, s, reinterpret_cast<const float4 *>(acc),
                          g.plan.splits, h.rows, hidden8, static_cast<uint4 *>(dx), lddx / 8));
  }
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_head_loss_workspace_bytes(int64_t rows, int64_t vocab, int64_t hidden) {
  const HeadShape h{rows, vocab, hidden};
  if (rows < 1 || check_shape(h) != MUON_OK) return 0;
  return ForwardRegions(h, true).bytes;
}

int muon_head_loss(const void *x, int64_t x_stride, const void *weight, const int64_t *targets, int64_t rows,
                   int64_t vocab, int64_t hidden, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                   muon_stream_t stream) {
  const HeadShape h{rows, vocab, hidden};
  MUON_TRY(check_shape(h));
  if (rows == 0) return MUON_OK;
  if (!x || !weight || !targets || (!loss && !lse) || x_stride < hidden) return MUON_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(weight) || x_stride % 8 || !on_elements({targets}, 8) || !on_elements({loss, lse}, 4))
    return MUON_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Scratch ws(s);
  MUON_TRY(ws.take(workspace, workspace_bytes, ForwardRegions(h, off_lines(x, x_stride)).bytes));
  return ws.done(forward(h, x, x_stride, weight, targets, loss, lse, ws.p, s));
}

size_t muon_head_loss_backward_workspace_bytes(int64_t rows, int64_t vocab, int64_t hidden) {
  const HeadShape h{rows, vocab, hidden};
  if (rows < 1 || check_shape(h) != MUON_OK) return 0;
  // enough whichever of the gradients is wanted
  return std::max({Regions(h, true, true).bytes, Regions(h, true, false).bytes, Regions(h, false, true).bytes});
}

int muon_head_loss_backward(const float *dloss, const float *dlse, const void *x, int64_t x_stride,
                            const void *weight, const int64_t *targets, const float *lse, int64_t rows, int64_t vocab,
                            int64_t hidden, void *dx, int64_t dx_stride, void *dweight, void *workspace,
                            size_t workspace_bytes, muon_stream_t stream) {
  const HeadShape h{rows, vocab, hidden};
  MUON_TRY(check_shape(h));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {   // a sum over no rows
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)vocab * hidden * 2, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if (!dloss || !x || !weight || !targets || !lse || (!dx && !dweight) || x_stride < hidden ||
      (dx && dx_stride < hidden))
    return MUON_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(weight) || !aligned16(dweight) || x_stride % 8 ||
      (dx && (!aligned16(dx) || dx_stride % 8)) || !on_elements({targets}, 8) || !on_elements({dloss, dlse, lse}, 4))
    return MUON_ERR_UNSUPPORTED;
  const Regions g(h, dx != nullptr, dweight != nullptr);
  Scratch ws(s);
  MUON_TRY(ws.take(workspace, workspace_bytes, g.bytes));
  return ws.done(backward(h, g, dloss, dlse, x, x_stride, weight, targets, lse, dx, dx_stride, dweight, ws.p, s));
}

}  // extern "C"
