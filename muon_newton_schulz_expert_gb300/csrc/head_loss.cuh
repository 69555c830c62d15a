// Internal declarations of the loss over a head matrix: the tensor-core products
// (head_tc.cu) that the entry points (head_loss.cu) put together.
#pragma once

#include "common.cuh"

namespace muon {

// z = x W^T of rows x vocab places is never whole in memory.  Sizes are at least 1,
// hidden a multiple of 8, every array 16-byte aligned, x's row stride a multiple of 8.
struct HeadShape {
  int64_t rows, vocab, hidden;
};

// Softmax statistics (c, s) of a row: s = sum 2^(z log2(e) - c), c a whole number.  Up to 2^23 such a c can be moved by any
// exponent exactly, and up to 2^30 the product z log2(e) is rounded by 2^5 at most, so that c stays next to the largest
// term's exponent.  From there on (logits beyond 7e8, where two are 64 apart or equal, so that the sum counts the
// largest alone) c is twice the largest logit itself: such a c is beyond 2^30, in the logits' order with whole ones too,
// and so far from any other that 2^(c' - c) is 0 as it has to be.  Joins of statistics need not tell the two apart.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWholeReference = 0x1p23f, kFarReference = 0x1p30f;
__device__ __forceinline__ float far_reference(float most) { return 2.f * most; }   // beyond 2^127: infinite
__device__ __forceinline__ bool is_far(float c) { return fabsf(c) >= kFarReference; }
__device__ __forceinline__ float far_logit(float c) { return 0.5f * c; }

// columns of z in a tile of head_stats, chosen so that there are tiles for all SMs
int head_stats_columns(const HeadShape &h);
// Partial softmax statistics of z: parts[i][row] = (c, s) over the i-th part of the vocabulary (head_parts of them), and
// target_logit[row] = z[row][targets[row]] where that target is in the vocabulary.
int64_t head_parts(const HeadShape &h);
int head_stats(const HeadShape &h, const void *x, int64_t ldx, const void *w, const int64_t *targets, float2 *parts,
               float *target_logit, cudaStream_t s);

// What a row sends into z: d_v = g p_v - hit [v = target]; g = hit = 0 and target -1 for a row that takes no part.
struct HeadRow {
  float lse, g, hit;
  int target;
};
// Where the backward pass cuts the vocabulary: pieces of piece_tiles * 256 columns, dx summed in `splits` parts.
struct HeadPlan {
  int64_t piece_tiles, pieces;
  int splits;
  int64_t width() const { return piece_tiles * 256; }
};
HeadPlan head_plan(const HeadShape &h, bool need_dx, bool need_dw);
// d[rows][plan.width()] (bf16) of the piece from vocabulary entry v0 on, zeros past the vocabulary's end.  xc: dense
// rows of x of width xc_cols, a multiple of 64, zeros in rows that take no part.
int head_dlogits(const HeadShape &h, const HeadPlan &plan, int64_t v0, const void *xc, int64_t xc_cols, const void *w,
                 const HeadRow *row, void *d, cudaStream_t s);
// From that piece: its rows of dweight and its part of dx: dx itself where there are neither pieces nor splits, else sums in
// acc[splits][rows][hidden] (`first`: written, else added to).
int head_grads(const HeadShape &h, const HeadPlan &plan, int64_t v0, bool first, const void *d, const void *w,
               const void *xc, int64_t xc_cols, void *dx, int64_t lddx, float *acc, void *dweight, cudaStream_t s);

}  // namespace muon
