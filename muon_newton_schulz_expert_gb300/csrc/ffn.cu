// C entry points of the gated feed-forward block: argument checks, workspace
// and the order of the products (ffn_tc.cu).
#include <algorithm>
#include <initializer_list>

#include "common.cuh"

namespace muon {
namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxExperts = 65535, kMaxWidth = int64_t(1) << 20;

int check_shape(const FfnShape &f) {
  if (f.rows < 0 || f.experts < 1 || f.hidden < 1 || f.ffn < 1 || (f.act != MUON_ACT_SILU && f.act != MUON_ACT_GELU) ||
      (!f.offsets && f.experts != 1))
    return MUON_ERR_INVALID_ARG;
  if (f.rows > kMaxRows || f.experts > kMaxExperts || f.hidden > kMaxWidth || f.ffn > kMaxWidth || f.hidden % 8 ||
      f.ffn % 8)
    return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

// every pointer 16-byte aligned, every row stride a multiple of 8 (TMA)
bool takes(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> strides) {
  for (const void *p : ptrs)
    if (!aligned16(p)) return false;
  for (int64_t st : strides)
    if (st % 8) return false;
  return true;
}

// `need` bytes: the caller's workspace, or the library's own (freed by done())
struct Scratch {
  void *p = nullptr;
  bool owned = false;
  cudaStream_t s;

  explicit Scratch(cudaStream_t stream) : s(stream) {}

  int take(void *workspace, size_t bytes, size_t need) {
    if (workspace) {
      if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_ERR_INVALID_ARG;
      if (bytes < need) return MUON_ERR_NO_MEMORY;
      p = workspace;
      return MUON_OK;
    }
    if (alloc_async(&p, need, s) != cudaSuccess) {
      cudaGetLastError();
      return MUON_ERR_NO_MEMORY;
    }
    owned = true;
    return MUON_OK;
  }

  int done(int st) {
    if (owned && cudaFreeAsync(p, s) != cudaSuccess && st == MUON_OK) return MUON_ERR_CUDA;
    return st;
  }
};

// Which kernels take a row product with `cols` output columns (of tiles of
// `tile`): where 256-row tiles leave pairs of CTAs without one, and an expert's
// rows fit two row tiles of ffn_few.cu, its smaller tiles and cut K loop.
// Measured at 6144 x 1792, one expert: 1 row 33 + 17 us against 17 + 15 us.
// With more rows an expert the smaller tiles read the weights again for each:
// 1777 rows, 5 experts, 1000 x 328: 19 + 13 us against 32 + 17 us.
bool few_tiles(const FfnShape &f, int64_t cols, int64_t tile) {
  const int64_t active = std::min(f.experts, f.rows);
  return f.rows <= 128 * active && (f.rows / 256 + active) * ((cols + tile - 1) / tile) < num_sms() / 2;
}
bool few_up(const FfnShape &f) { return few_tiles(f, f.ffn, 128); }

size_t rows_bytes(const FfnShape &f) { return align256((size_t)f.rows * f.ffn * 2); }
size_t fwd_bytes(const FfnShape &f) { return 2 * rows_bytes(f); }   // h, and for few rows what its rounding left
size_t bwd_bytes(const FfnShape &f) {
  return 3 * rows_bytes(f) + align256(ffn_tail_elems(f) * 2) + align256(ffn_parts_elems(f) * 4);
}

#define MUON_TRY(expr)              \
  do {                              \
    const int _st = (expr);         \
    if (_st != MUON_OK) return _st; \
  } while (0)

int backward(const FfnShape &f, const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *gate,
             const void *up, const void *w1, const void *w3, const void *w2, void *dx, int64_t lddx, void *dw1,
             void *dw3, void *dw2, void *scratch, cudaStream_t s) {
  uint8_t *p = static_cast<uint8_t *>(scratch);
  void *dg = p, *du = p + rows_bytes(f), *hid = p + 2 * rows_bytes(f), *tails = p + 3 * rows_bytes(f);
  float *parts = reinterpret_cast<float *>(p + 3 * rows_bytes(f) + align256(ffn_tail_elems(f) * 2));
  MUON_TRY(few_tiles(f, f.ffn, 256) ? ffn_few_dh(f, dy, lddy, w2, gate, up, dg, du, hid, s)
                                    : ffn_dh(f, dy, lddy, w2, gate, up, dg, du, hid, s));
  if (dx)
    MUON_TRY(few_tiles(f, f.hidden, 256) ? ffn_few_dx(f, dg, du, w1, w3, dx, lddx, s)
                                         : ffn_dx(f, dg, du, w1, w3, dx, lddx, s));
  if (dw1) MUON_TRY(ffn_dw(f, x, ldx, dy, lddy, dg, du, hid, tails, parts, dw1, dw3, dw2, s));
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_gated_ffn_workspace_bytes(int64_t rows, int64_t experts, int64_t hidden, int64_t ffn) {
  const FfnShape f{nullptr, rows, 1, hidden, ffn, MUON_ACT_SILU};
  if (rows < 1 || experts < 1 || experts > kMaxExperts || check_shape(f) != MUON_OK) return 0;
  return fwd_bytes(f);
}

int muon_gated_ffn(const void *x, int64_t x_stride, const void *w1, const void *w3, const void *w2,
                   const int64_t *offsets, int64_t rows, int64_t experts, int64_t hidden, int64_t ffn, int act,
                   void *y, int64_t y_stride, void *gate, void *up, void *workspace, size_t workspace_bytes,
                   muon_stream_t stream) {
  const FfnShape f{offsets, rows, experts, hidden, ffn, act};
  MUON_TRY(check_shape(f));
  if (rows == 0) return MUON_OK;
  if (!x || !w1 || !w3 || !w2 || !y || !gate != !up || x_stride < hidden || y_stride < hidden)
    return MUON_ERR_INVALID_ARG;
  if (!on_elements({offsets}, 8) || !takes({x, w1, w3, w2, y, gate, up}, {x_stride, y_stride})) return MUON_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Scratch ws(s);
  MUON_TRY(ws.take(workspace, workspace_bytes, fwd_bytes(f)));
  void *hid = ws.p, *rest = static_cast<uint8_t *>(ws.p) + rows_bytes(f);
  int st;
  if (few_up(f)) {
    st = ffn_few_up(f, x, x_stride, w1, w3, hid, rest, gate, up, s);
    if (st == MUON_OK) st = ffn_few_down(f, hid, rest, w2, y, y_stride, s);
  } else {
    st = ffn_up(f, x, x_stride, w1, w3, hid, gate, up, s);
    if (st == MUON_OK) st = ffn_down(f, hid, w2, y, y_stride, s);
  }
  return ws.done(st);
}

size_t muon_gated_ffn_backward_workspace_bytes(int64_t rows, int64_t experts, int64_t hidden, int64_t ffn) {
  FfnShape f{nullptr, rows, 1, hidden, ffn, MUON_ACT_SILU};
  if (rows < 1 || experts < 1 || experts > kMaxExperts || check_shape(f) != MUON_OK) return 0;
  f.experts = experts;
  return bwd_bytes(f);
}

int muon_gated_ffn_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, const void *gate,
                            const void *up, const void *w1, const void *w3, const void *w2, const int64_t *offsets,
                            int64_t rows, int64_t experts, int64_t hidden, int64_t ffn, int act, void *dx,
                            int64_t dx_stride, void *dw1, void *dw3, void *dw2, void *workspace,
                            size_t workspace_bytes, muon_stream_t stream) {
  const FfnShape f{offsets, rows, experts, hidden, ffn, act};
  MUON_TRY(check_shape(f));
  if (!dw1 != !dw3 || !dw1 != !dw2) return MUON_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {   // sums over no rows
    const size_t bytes = (size_t)experts * hidden * ffn * 2;
    for (void *d : {dw1, dw3, dw2})
      if (d && cudaMemsetAsync(d, 0, bytes, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if (!dy || !gate || !up || !w2 || (!dx && !dw1) || (dx && (!w1 || !w3)) || (dw1 && !x) || dy_stride < hidden ||
      (dw1 && x_stride < hidden) || (dx && dx_stride < hidden))
    return MUON_ERR_INVALID_ARG;
  // what is not read or written may lie anywhere
  const bool aligned = takes({dy, gate, up, w2}, {dy_stride}) && (!dx || takes({w1, w3, dx}, {dx_stride})) &&
                       (!dw1 || takes({x, dw1, dw3, dw2}, {x_stride}));
  if (!aligned || !on_elements({offsets}, 8)) return MUON_ERR_UNSUPPORTED;
  Scratch ws(s);
  MUON_TRY(ws.take(workspace, workspace_bytes, bwd_bytes(f)));
  return ws.done(backward(f, dy, dy_stride, x, x_stride, gate, up, w1, w3, w2, dx, dx_stride, dw1, dw3, dw2, ws.p, s));
}

}  // extern "C"
