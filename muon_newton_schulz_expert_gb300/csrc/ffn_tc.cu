// Tensor-core products of the gated feed-forward block over expert matrices.
//
// Rows (tokens) are sorted by expert; rows offsets[e] .. offsets[e+1] belong
// to expert e, whose weights are W1, W3 (H x F) and W2 (F x H):
//   forward   G = X W1, U = X W3, Hid = act(G) * U            (UP)
//             Y = Hid W2                                       (DOWN)
//   backward  D = dY W2^T, dG = D*U*act'(G), dU = D*act(G), Hid again   (DH)
//             dX = dG W1^T + dU W3^T                           (DX)
//             dW1 = X^T dG, dW3 = X^T dU                       (DW13)
//             dW2 = Hid^T dY                                   (DW2)
// One kernel, instantiated for the six products; all are persistent CTA pairs
// on output tiles of up to 256 x 256 (tcgen05.mma.cta_group::2, M = 256, K = 16,
// bf16 operands, fp32 accumulation in TMEM), fed by TMA through a ring of
// three stages of two k-blocks of 64.
//
// The row products (UP, DOWN, DH, DX) have the weights on M and the rows on N:
//   D[256 weight columns, N rows] = W^T X^T
// since N may be any multiple of 32 up to 256, and groups of rows end anywhere.
// A group's n rows are ceil(n / 32) units, spread evenly over ceil(n / 256)
// tiles, so that 16 rows of a group are computed in vain on average and no tile
// is much shorter than its neighbours.  (With the rows on M every tile counts 256:
// 16384 rows over 32 experts, 6144 x 1792, fill 83% of those.)  Rows past a
// group's end belong to the next expert: computed and not stored, since rows do
// not mix.
//
// UP forms both products of the same places: the M axis of a CTA holds 64
// columns of W1 and the same 64 of W3, so X is read once for both.  G is then in
// TMEM lanes 0..63 and U in lanes 64..127; the two warps that hold the same places
// exchange halves through shared memory.
//
// DX runs one K loop over both products: first W1 dG^T, then W3 dU^T.
//
// DW13 has 128 columns of dG on the even CTA's half of N and of dU on the odd
// one's, so that X is read once for both gradients.
//
// The weight gradients sum over the group's rows, so there the last, partial
// k-block must hold zeros past the group's end in both operands: it is read
// from copies of those rows padded with zeros (`tail` arrays,
// [experts][64][columns]), which keeps a NaN of one expert's rows out of
// another's gradient.  An expert without rows gets zeros.
// Where the gradients have few tiles and many rows, the rows are cut into parts: each
// leaves its sums in fp32, and a second kernel adds them in order.
//
// Rounding: Hid, dG and dU are stored in bf16, the operand type of the product
// that reads them; everything before that rounding is fp32.  Outputs are then within
// 0.0023 (relative) of 64 bits where their own rounding alone leaves 0.0017; carrying
// remainders besides, as ffn_few.cu does for Hid, would double the rows of DOWN and DX and
// the K of the gradients.
//
// Roles per CTA (320 threads): warp 0 TMA producer, warp 1 MMA issuer (even
// CTA) and TMEM owner, warps 2..9 epilogue.  Two accumulators, so that the
// epilogue of one tile overlaps the next tile's products.  Every wait is
// bounded (tc.cuh); an epilogue warp that gave up still meets its partner of UP.
#include <algorithm>

#include "ffn.cuh"

namespace muon {
namespace {

constexpr int CM = 256, BM = 128;   // M of a pair tile, M held by one CTA
constexpr int BN = 256, BNH = 128;  // most N of a pair tile, N loaded by one CTA
constexpr int UNIT = 32;            // rows by which a row product's N grows
constexpr int BK = 64;              // one 128-byte swizzle row of bf16
constexpr int UMMA_K = 16;
constexpr int A_STAGE = BM * BK * 2;
constexpr int B_STAGE = BNH * BK * 2;
constexpr int KB_BYTES = A_STAGE + B_STAGE;
constexpr int STAGES = 3, KSUB = 2;
constexpr int STAGE_BYTES = KSUB * KB_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int BOX_BYTES = 32 * 64 * 2;    // output staging box of an epilogue warp: 32 rows x 64 columns
constexpr int ACC_COLS = BN;
constexpr int TMEM_COLS = 2 * ACC_COLS;
constexpr int NFULL = STAGES * KSUB;
constexpr int NUM_BARS = NFULL + STAGES + 5;
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * BOX_BYTES + NUM_BARS * 8 + 16;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

enum Mode { UP = 0, DOWN, DH, DX, DW13, DW2 };

template <int MODE>
struct Form {
  static constexpr bool dw = MODE == DW13 || MODE == DW2;
  static constexpr bool a_mn = dw || MODE == UP || MODE == DOWN;
  static constexpr bool b_mn = dw;
  // two weight matrices side by side in the accumulator's columns
  static constexpr bool paired = MODE == DW13;
};

struct Args {
  // weights of the row products (UP, DX: a2 = W3), A of the gradients (a2 = tail copy)
  CUtensorMap a, a2;
  union {
    CUtensorMap rows_of[2][BN / UNIT];   // row products: boxes of 16, 32, .. 128 rows; DX: of dG and of dU
    struct {
      CUtensorMap b, b2, bt, bt2;        // gradients: B (DW13: dG, dU) and its tail copies
    };
  };
  CUtensorMap out[2];                // DW: boxes of 32 rows x 64 columns
  void *outp[3];
  long long out_ld[3];               // row strides in elements
  const int64_t *offsets;            // null: one group of all rows
  long long rows;
  int experts;
  int M, N;                          // DW: output rows; all: output columns of one weight matrix
  int kblocks;                       // row products: k-blocks of one K segment
  int tiles_m, tiles_n;              // DW: row tiles; all: column tiles
  int act;
  bool wide;                         // 128-column operands load in one piece
  const __nv_bfloat16 *g, *u;        // DH: saved pre-activations [rows][N]
  int split;                         // DW: parts of a group's rows, summed by ffn_parts_kernel if above 1
  float *parts;                      // [split][matrices][experts][M][N]
  unsigned *err;
  unsigned long long timeout_ns;
};

// A tile: expert, row tile and column tile, rows of the expert; of a row product
// also the tile's first row and the units of 32 rows it spans.
template <int MODE>
struct Tile {
  int e, ti, tj, lo, hi, row0 = 0, units = BN / UNIT;
  int part = 0, kb0 = 0, num_kb;   // of a cut sum; first k-block and their number


  __device__ Tile(const Args &p, const WarpCursor &cur) {
    e = cur.e, lo = cur.lo, hi = cur.hi;
    const int tm = Form<MODE>::dw ? p.tiles_m : (hi - lo + BN - 1) / BN;
    tj = (int)((unsigned)cur.index / (unsigned)tm);   // 2^32 tiles of 256 x 256 fit no memory
    ti = (int)((unsigned)cur.index - (unsigned)tj * (unsigned)tm);
    num_kb = Form<MODE>::dw ? (hi - lo + BK - 1) / BK : MODE == DX ? 2 * p.kblocks : p.kblocks;
    if (Form<MODE>::dw && p.split > 1) {   // parts of the rows, the slowest of the three
      const int all = num_kb;
      part = tj / p.tiles_n;
      tj -= part * p.tiles_n;
      kb0 = (int)((long long)all * part / p.split);
      num_kb = (int)((long long)all * (part + 1) / p.split) - kb0;
    }
    if (!Form<MODE>::dw) {
      const int all = (hi - lo + UNIT - 1) / UNIT, each = all / tm, more = all - each * tm;
      units = each + (ti < more ? 1 : 0);
      row0 = lo + UNIT * (ti * each + min(ti, more));
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
}

// 32 lanes x 64 consecutive fp32 columns -> 64 registers per thread, waited.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&lo)[32], uint32_t (&hi)[32]) {
  tmem_ld32_issue(taddr, lo);
  tmem_ld32_issue(taddr + 32, hi);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // the registers are only valid from here on
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(lo[i]), "+r"(hi[i]));
}

// 128 columns x 64 K-rows into two atoms of 64 columns: one load where the columns
// are whole blocks of 64, two boxes otherwise (16384 rows, 32 experts, 6144 x 1792:
// dW1 and dW3 530 us with one, 555 us with two; dW2 281 and 291; DOWN the same).
__device__ __forceinline__ void load_columns(uint32_t dst, const CUtensorMap *map, uint32_t bar, int col, int row,
                                             int z, bool wide, unsigned *err) {
  if (wide) {
    tma_load_4d_pair(dst, map, bar, 0, row, col / 64, z, err);
  } else {
    tma_load_3d_pair(dst, map, bar, col, row, z, err);
    tma_load_3d_pair(dst + 64 * BK * 2, map, bar, col + 64, row, z, err);
  }
}

// Weight gradients: one epilogue warp's way out, 32 rows x 64 columns of bf16,
// lane = row, through shared memory and TMA, which clips at the array's edge:
// 128-byte rows, since 64-byte ones (32 columns) held the stores to 2.6 TB/s.
struct Writer {
  uint8_t *box;
  uint32_t box_s;

  __device__ void put(const uint32_t (&w)[32], const CUtensorMap *map, int lane, int col0, int row0, int mat,
                      unsigned *err) {
    if (lane == 0) bulk_wait_read_all();  // the box's last store has read it
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(map, box_s, col0, row0, mat, err);
      bulk_commit();
    }
  }
};

// Row products: a lane holds one column's sums for 32 rows of the output.
// Lanes 2i and 2i + 1 exchange halves, so that each has both columns, c[j][0]
// and c[j][1], of the 16 rows 2j + (lane & 1): 4-byte accesses, a warp's 64 bytes
// of two rows, whole 32-byte sectors.
__device__ __forceinline__ void pair_columns(const uint32_t (&v)[32], float (&c)[16][2], int lane) {
  const bool odd = lane & 1;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float mine = __uint_as_float(odd ? v[2 * j + 1] : v[2 * j]);
    const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(odd ? v[2 * j] : v[2 * j + 1]), 1);
    c[j][0] = odd ? other : mine;
    c[j][1] = odd ? mine : other;
  }
}

// rows first + 2 j, j in [0, N), of a lane's two columns.  A pointer that moves on and
// 32-bit comparisons: with 64-bit ones an epilogue of UP took 6.6 us instead of 4.1,
// which a call of one tile per pair waits for.
template <int N>
__device__ __forceinline__ void put_pairs(void *base, long long ld, long long first, long long row_end, int col,
                                          int cols, const uint32_t (&w)[N]) {
  const int left = col < cols ? (int)min(row_end - first, 2ll * N) : 0;
  char *dst = reinterpret_cast<char *>(static_cast<__nv_bfloat16 *>(base) + first * ld + col);
  const long long step = ld * 4;
  if (left >= 2 * N - 1) {
#pragma unroll
    for (int j = 0; j < N; ++j, dst += step) *reinterpret_cast<uint32_t *>(dst) = w[j];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j, dst += step)
      if (2 * j < left) *reinterpret_cast<uint32_t *>(dst) = w[j];
  }
}

template <int MODE>
__global__ void __launch_bounds__(THREADS, 1) ffn_gemm_kernel(const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + STAGES * STAGE_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + EPI_WARPS * BOX_BYTES);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NUM_BARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // 0: issues the MMAs; 1: its peer
  const long long cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  auto full = [&](int s, int j) { return bar0 + 8u * (uint32_t)(s * KSUB + j); };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(NFULL + s); };
  auto accf = [&](int a) { return bar0 + 8u * (uint32_t)(NFULL + STAGES + a); };
  auto acce = [&](int a) { return bar0 + 8u * (uint32_t)(NFULL + STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(NFULL + STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NFULL; ++s) mbar_init(bar0 + 8u * s, 1);   // used in CTA 0: expect_tx for both halves
    for (int s = 0; s < STAGES; ++s) mbar_init(empty(s), 1);       // multicast commit
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf(a), 1);               // multicast commit
      mbar_init(acce(a), 2 * EPI_WARPS);   // used in CTA 0: every epilogue warp of the pair
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.a);
    if (Form<MODE>::dw) tma_prefetch_desc(&p.b);
    if (Form<MODE>::dw) tma_prefetch_desc(&p.out[0]);
  }
  if (warp == 1) {  // one warp in each CTA of the pair allocates the same columns in both
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers are initialised before anyone signals them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watch w{abort_flag, p.err, p.timeout_ns};
  const unsigned long long drain_ns = p.timeout_ns < 20000000ull ? p.timeout_ns : 20000000ull;
  wait_for_previous_grid();
  let_next_grid_start();
  if (warp == 2 && blockIdx.x == 0) report_offsets(p.offsets, p.experts, p.rows, p.err);
  WarpCursor walk(p.offsets, p.rows, p.experts, Form<MODE>::dw ? 0 : BN,
                  (long long)(Form<MODE>::dw ? p.tiles_m * p.split : 1) * p.tiles_n);

  if (warp == 0) {
    // ---------------------------------------------------------------- producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0, issued_parity = 0;  // stages ever filled, and the parity of their last fill
    bool ok = true;
    for (long long t = cid; walk.seek(t); t += ncl) {
      const Tile<MODE> cur(p, walk);
      if (lane == 0 && ok) {
        const int num_kb = cur.num_kb;
        // first of this CTA's places on M and N
        const int mn_a = Form<MODE>::dw ? cur.ti * CM + (int)rank * BM
                         : MODE == UP   ? cur.tj * BM + (int)rank * (BM / 2)
                                        : cur.tj * CM + (int)rank * BM;
        const int n_b = Form<MODE>::paired ? cur.tj * BNH : cur.tj * BN + (int)rank * BNH;
        const int half_rows = cur.units * (UNIT / 2), row_b = cur.row0 + (int)rank * half_rows;
        const uint32_t kb_bytes = Form<MODE>::dw ? KB_BYTES : A_STAGE + half_rows * (BK * 2);
        const CUtensorMap *row_maps = p.rows_of[0] + (cur.units - 1);   // boxes of half_rows rows
        const CUtensorMap *mb = Form<MODE>::paired && rank ? &p.b2 : &p.b;
        for (int kb = 0; kb < num_kb; kb += KSUB) {
          if (!wait_polled(empty(stage), phase ^ 1u, w)) {
            ok = false;
            break;
          }
          const int valid = num_kb - kb < KSUB ? num_kb - kb : KSUB;
          // CTA 0's barrier counts the bytes of both CTAs; a k-block past the
          // end of K still completes its phase, with no bytes
          if (rank == 0)
#pragma unroll
            for (int j = 0; j < KSUB; ++j) mbar_expect_tx(full(stage, j), j < valid ? 2 * kb_bytes : 0);
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
#pragma unroll
          for (int j = 0; j < KSUB; ++j) {
            if (j >= valid) break;
            const int k = cur.kb0 + kb + j;
            const uint32_t sa = sbase + stage * STAGE_BYTES + j * KB_BYTES, sb = sa + A_STAGE;
            const uint32_t bar = map_to_rank(full(stage, j), 0);
            if (Form<MODE>::dw) {
              // boxes of 64 columns x 64 rows; the group's last rows from the padded copies
              const bool tail = cur.hi - cur.lo - k * BK < BK;
              const int kr = tail ? 0 : cur.lo + k * BK, z = tail ? cur.e : 0;
              const CUtensorMap *ma = tail ? &p.a2 : &p.a;
              const CUtensorMap *mbk = !tail ? mb : Form<MODE>::paired && rank ? &p.bt2 : &p.bt;
              load_columns(sa, ma, bar, mn_a, kr, z, p.wide, p.err);
              load_columns(sb, mbk, bar, n_b, kr, z, p.wide, p.err);
            } else {
              const bool second = MODE == DX && k >= p.kblocks;
              const int kc = (second ? k - p.kblocks : k) * BK;
              if (MODE == UP) {         // boxes of 64 weight columns x 64 K-rows
                tma_load_3d_pair(sa, &p.a, bar, mn_a, kc, cur.e, p.err);
                tma_load_3d_pair(sa + 64 * BK * 2, &p.a2, bar, mn_a, kc, cur.e, p.err);
              } else if (MODE == DOWN) {
                load_columns(sa, &p.a, bar, mn_a, kc, cur.e, p.wide, p.err);
              } else {                  // one box of 128 weight rows x 64 K-columns
                tma_load_3d_pair(sa, second ? &p.a2 : &p.a, bar, kc, mn_a, cur.e, p.err);
              }
              tma_load_3d_pair(sb, second ? row_maps + BN / UNIT : row_maps, bar, kc, row_b, 0, p.err);
            }
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      __syncwarp();
    }
    // After an abort, stages may still be filling: let those copies land.
    if (*abort_flag && rank == 0 && lane == 0)
      for (int s2 = 0; s2 < STAGES; ++s2)
        if (issued & (1u << s2))
          for (int j = 0; j < KSUB; ++j) drain_wait(full(s2, j), (issued_parity >> s2) & 1u, drain_ns);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (CTA 0 of the pair)
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (long long t = cid; walk.seek(t); t += ncl) {
        const Tile<MODE> cur(p, walk);
        if (lane == 0 && ok) ok = wait_bounded(acce(acc), acc_phase ^ 1u, w);
        if (lane == 0 && ok) {
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * ACC_COLS);
          const int num_kb = cur.num_kb;
          const uint32_t idesc = make_idesc(CM, UNIT * cur.units, Form<MODE>::a_mn, Form<MODE>::b_mn);
          for (int kb = 0; kb < num_kb; kb += KSUB) {
            const int valid = num_kb - kb < KSUB ? num_kb - kb : KSUB;
#pragma unroll
            for (int j = 0; j < KSUB; ++j) {
              if (j >= valid) break;
              if (!wait_polled(full(stage, j), phase, w)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t sa = sbase + stage * STAGE_BYTES + j * KB_BYTES, sb = sa + A_STAGE;
              // K-major: advance 16 K-elements (32 bytes) inside the swizzle row.
              // MN-major: advance 16 K-rows (two 8-row groups of 1024 bytes);
              // 8192 bytes between 64-wide atoms, 1024 between 8-row groups.
#pragma unroll
              for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                const uint64_t ad = Form<MODE>::a_mn ? smem_desc(sa + kk * (UMMA_K * 128), 64 * BK * 2, 1024)
                                               : smem_desc(sa + kk * (UMMA_K * 2), 16, 1024);
                const uint64_t bd = Form<MODE>::b_mn ? smem_desc(sb + kk * (UMMA_K * 128), 64 * BK * 2, 1024)
                                               : smem_desc(sb + kk * (UMMA_K * 2), 16, 1024);
                tc_mma(d, ad, bd, idesc, ((kb + j) | kk) != 0 ? 1u : 0u);
              }
            }
            if (!ok) break;
            tc_commit_mc(empty(stage), 0x3);  // both CTAs may refill this stage
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit_mc(accf(acc), 0x3);  // both CTAs' accumulators are ready
        }
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (lane == 0) {
        tc_commit_mc(drain_bar, 0x1);  // flips once all MMAs issued by this thread have completed
        volatile int no_abort = 0;
        wait_bounded(drain_bar, 0, Watch{&no_abort, p.err, p.timeout_ns});
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - 2;
    const int q = warp & 3, half = ew >> 2;  // TMEM lanes 32q.., and which half of the columns
    uint8_t *box = epi_smem + ew * BOX_BYTES;
    Writer out{box, smem_u32(box)};
    int acc = 0;
    uint32_t acc_phase = 0, flip = 0;
    bool ok = true;
    for (long long t = cid; walk.seek(t); t += ncl) {
      const Tile<MODE> cur(p, walk);
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(accf(acc), acc_phase, w));   // warp-uniform
      if (!ok && MODE != UP) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * ACC_COLS);
      if (MODE == UP) {
        // lanes of q = 0, 1 hold G of 32 columns each, those of q = 2, 3 U of the same
        const bool has_u = q >= 2;
        const int col = cur.tj * BM + (int)rank * (BM / 2) + (q & 1) * 32 + (lane & ~1);
        float2 *mine = reinterpret_cast<float2 *>(box) + lane;
        const float2 *partner = reinterpret_cast<const float2 *>(epi_smem + (ew ^ 2) * BOX_BYTES) + lane;
        for (int ch = half; ch < cur.units; ch += 2) {
          float c[16][2];
          if (ok) {
            uint32_t v[32];
            tmem_ld32(taddr + (uint32_t)(UNIT * ch), v);
            pair_columns(v, c, lane);
            // each of the two warps finishes 16 of the 32 rows: it hands over its sums of the others
#pragma unroll
            for (int j = 0; j < 8; ++j)
              mine[(flip * 8 + j) * 32] = has_u ? make_float2(c[j][0], c[j][1]) : make_float2(c[8 + j][0], c[8 + j][1]);
          }
          asm volatile("bar.sync %0, 64;" ::"r"(1 + half * 2 + (q & 1)) : "memory");
          if (ok) {
            const long long first = (long long)cur.row0 + UNIT * ch + (lane & 1);
            uint32_t wh[8], w16[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 o = partner[(flip * 8 + j) * 32];
              float h[2], dv;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float ov = i ? o.y : o.x, mv = has_u ? c[8 + j][i] : c[j][i];
                const float g = has_u ? ov : mv, u = has_u ? mv : ov;
                h[i] = g * sigmoid_of(g, p.act, &dv) * u;
              }
              wh[j] = pack_bf16(h[0], h[1]);
            }
            put_pairs<8>(p.outp[0], p.out_ld[0], first + (has_u ? 16 : 0), cur.hi, col, p.N, wh);
            if (p.outp[1]) {
#pragma unroll
              for (int j = 0; j < 16; ++j) w16[j] = pack_bf16(c[j][0], c[j][1]);
              put_pairs<16>(p.outp[has_u ? 2 : 1], p.out_ld[1], first, cur.hi, col, p.N, w16);
            }
          }
          flip ^= 1u;   // the partner may still be reading this half of the box
        }
      } else if (!Form<MODE>::dw) {
        const int col = cur.tj * CM + (int)rank * BM + q * 32 + (lane & ~1);
        for (int ch = half; ch < cur.units; ch += 2) {
          const long long first = (long long)cur.row0 + UNIT * ch + (lane & 1);
          uint32_t wg[16], wu[16], wh[16];
          if (MODE == DH) {
            const int left = col < p.N ? (int)min(cur.hi - first, 32ll) : 0;
            const char *pg = reinterpret_cast<const char *>(p.g + first * p.N + col);
            const char *pu = reinterpret_cast<const char *>(p.u + first * p.N + col);
            const long long step = (long long)p.N * 4;
#pragma unroll
            for (int j = 0; j < 16; ++j, pg += step, pu += step) {
              wg[j] = 2 * j < left ? __ldg(reinterpret_cast<const unsigned *>(pg)) : 0u;
              wu[j] = 2 * j < left ? __ldg(reinterpret_cast<const unsigned *>(pu)) : 0u;
            }
            __syncwarp();
          }
          uint32_t v[32];
          tmem_ld32(taddr + (uint32_t)(UNIT * ch), v);
          float c[16][2];
          pair_columns(v, c, lane);
          if (MODE == DH) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 g2 = unpack_bf16(wg[j]), u2 = unpack_bf16(wu[j]);
              float dg[2], du[2], h[2];
              gated_gradient(c[j][0], g2.x, u2.x, p.act, &dg[0], &du[0], &h[0]);
              gated_gradient(c[j][1], g2.y, u2.y, p.act, &dg[1], &du[1], &h[1]);
              wg[j] = pack_bf16(dg[0], dg[1]);
              wu[j] = pack_bf16(du[0], du[1]);
              wh[j] = pack_bf16(h[0], h[1]);
            }
            put_pairs<16>(p.outp[0], p.out_ld[0], first, cur.hi, col, p.N, wg);
            put_pairs<16>(p.outp[1], p.out_ld[1], first, cur.hi, col, p.N, wu);
            put_pairs<16>(p.outp[2], p.out_ld[2], first, cur.hi, col, p.N, wh);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) wh[j] = pack_bf16(c[j][0], c[j][1]);
            put_pairs<16>(p.outp[0], p.out_ld[0], first, cur.hi, col, p.N, wh);
          }
          __syncwarp();
        }
      } else {
        const int row0 = cur.ti * CM + (int)rank * BM + q * 32;
        if (row0 < p.M) {
          const bool empty_sum = cur.num_kb == 0;            // no MMA ran: the accumulator holds nothing
          const int which = Form<MODE>::paired ? half : 0;   // DW13: dW1 in the low columns, dW3 in the high
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            const int cc = half * 128 + ch * 64;
            const int col0 = Form<MODE>::paired ? cur.tj * BNH + ch * 64 : cur.tj * BN + cc;
            if (col0 >= p.N) break;
            uint32_t lo[32], hi[32], wo[32];
            tmem_ld64(taddr + (uint32_t)cc, lo, hi);
            if (p.split > 1) {
              // this part's sums, in fp32
              const int row = row0 + lane, mats = Form<MODE>::paired ? 2 : 1;
              float *dst = p.parts + ((((long long)cur.part * mats + which) * p.experts + cur.e) * p.M + row) * p.N + col0;
              if (row < p.M)
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                  const uint32_t *v = c < 32 ? lo + c : hi + c - 32;
                  if (col0 + c < p.N)
                    *reinterpret_cast<uint4 *>(dst + c) =
                        empty_sum ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(v[0], v[1], v[2], v[3]);
                }
              __syncwarp();
              continue;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              wo[i] = empty_sum ? 0u : pack_bf16(__uint_as_float(lo[2 * i]), __uint_as_float(lo[2 * i + 1]));
              wo[16 + i] = empty_sum ? 0u : pack_bf16(__uint_as_float(hi[2 * i]), __uint_as_float(hi[2 * i + 1]));
            }
            out.put(wo, &p.out[which], lane, col0, row0, cur.e, p.err);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive_cluster(map_to_rank(acce(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA frees TMEM or exits while its peer may still use them
  if (*abort_flag) {
    // after an abort: a copy that only CTA 1 issued is not covered by the
    // drain above; it lands within microseconds
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 200000ull) __nanosleep(1000);
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// The rows of a group's last, partial k-block, followed by zeros up to 64
// rows, for each of the arrays the weight gradients read.  One block per
// expert and slice of columns; 16 bytes per thread and step.
struct TailArgs {
  const __nv_bfloat16 *src[5];
  __nv_bfloat16 *dst[5];      // [experts][64][cols]
  long long ld[5];
  int cols[5];
  const int64_t *offsets;
  long long rows;
};

__global__ void __launch_bounds__(256) ffn_tail_kernel(const __grid_constant__ TailArgs p) {
  const int e = blockIdx.x, which = blockIdx.z;
  long long lo = 0, hi = p.rows;
  if (p.offsets) {
    const long long a = __ldg(p.offsets + e), b = __ldg(p.offsets + e + 1);
    lo = a < 0 ? 0 : a > p.rows ? p.rows : a;
    hi = b < lo ? lo : b > p.rows ? p.rows : b;
  }
  const int n = (int)((hi - lo) % BK);
  if (n == 0) return;  // never read
  const int vecs = p.cols[which] / 8;
  const uint4 *src = reinterpret_cast<const uint4 *>(p.src[which] + (hi - n) * p.ld[which]);
  uint4 *dst = reinterpret_cast<uint4 *>(p.dst[which]) + (long long)e * BK * vecs;
  const long long src_ld = p.ld[which] / 8;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < BK * vecs; i += gridDim.y * 256) {
    const int r = i / vecs, c = i - r * vecs;
    dst[i] = r < n ? src[r * src_ld + c] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// The parts of a cut sum, added in order; eight elements a thread and step.
__global__ void __launch_bounds__(256) ffn_parts_kernel(const float *parts, int split, long long each, int mats,
                                                        __nv_bfloat16 *out0, __nv_bfloat16 *out1) {
  const long long n = each * mats / 8;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
    for (int s = 0; s < split; ++s) {
      const float4 *src = reinterpret_cast<const float4 *>(parts + s * mats * each) + 2 * i;
      const float4 x = __ldcs(src), y = __ldcs(src + 1);
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
      b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
    }
    const long long at = i * 8;
    __nv_bfloat16 *dst = at < each ? out0 + at : out1 + (at - each);
    *reinterpret_cast<uint4 *>(dst) =
        make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
  }
}

template <int MODE>
int launch(Args &p, int trace_kind, cudaStream_t s) {
  static std::once_flag attr_once[64];
  static int max_pairs[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  auto *kernel = ffn_gemm_kernel<MODE>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS, 1, 1);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // the occupancy query knows clusters only
  cfg.dynamicSmemBytes = SMEM_BYTES;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    int n = 0;
    cfg.gridDim = dim3(2 * (unsigned)std::max(1, num_sms() / 2), 1, 1);
    if (attr_err[dev] == cudaSuccess && cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0)
      max_pairs[dev] = n;
    else
      max_pairs[dev] = std::max(1, num_sms() / 2);
    cudaGetLastError();
  });
  if (attr_err[dev] != cudaSuccess) return MUON_ERR_CUDA;
  p.err = device_error_word();
  p.timeout_ns = wait_timeout_ns();
  if (!p.err) return MUON_ERR_CUDA;
  // at most this many tiles, whatever the groups' sizes are
  const long long row_tiles =
      Form<MODE>::dw ? (long long)p.tiles_m * p.split * p.experts : p.rows / BN + std::min<long long>(p.experts, p.rows);
  const long long pairs = std::min<long long>(row_tiles * p.tiles_n, max_pairs[dev]);
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.numAttrs = 2;
  cfg.stream = s;
  trace_before(trace_kind, s);
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, p);
  if (Form<MODE>::dw && le == cudaSuccess && p.split > 1) {
    const long long each = (long long)p.experts * p.M * p.N;
    const int mats = Form<MODE>::paired ? 2 : 1;
    const int blocks = (int)std::min<long long>((each * mats / 8 + 255) / 256, 8ll * num_sms());
    ffn_parts_kernel<<<blocks, 256, 0, s>>>(p.parts, p.split, each, mats, static_cast<__nv_bfloat16 *>(p.outp[0]),
                                            static_cast<__nv_bfloat16 *>(p.outp[1]));
  }
  const int st = trace_after(trace_kind, s);
  return le == cudaSuccess ? st : MUON_ERR_CUDA;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// operand maps: K-major weights (boxes of 128 rows x 64 columns), MN-major (64 x 64)
int map_k(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols) {
  return make_map(m, base, batch, rows, cols, BM);
}
int map_cols(CUtensorMap *m, const Args &p, const void *base, int64_t batch, int64_t rows, int64_t cols,
             int64_t ld = 0) {
  return p.wide ? make_map_blocks(m, base, batch, rows, cols, BK, 2, ld) : make_map(m, base, batch, rows, cols, BK, ld);
}
int map_mn(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols, int64_t ld = 0) {
  return make_map(m, base, batch, rows, cols, 64, ld);
}
// One box of exactly the rows that a tile's half has: boxes are paid for by the
// piece and by the bytes (16384 rows, 32 experts, forward: 797 us; 816 with boxes of
// 64 rows, 906 with exactly the rows in boxes of 64 and 16).
int map_rows(CUtensorMap (&m)[BN / UNIT], const void *base, const FfnShape &f, int64_t cols, int64_t ld = 0) {
  for (int u = 0; u < BN / UNIT; ++u)
    if (const int st = make_map(&m[u], base, 1, f.rows, cols, (u + 1) * UNIT / 2, ld)) return st;
  return MUON_OK;
}
int map_out(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols, int64_t ld = 0) {
  return make_map(m, base, batch, rows, cols, 32, ld);
}

Args base_args(const FfnShape &f) {
  Args p{};
  p.offsets = f.offsets;
  p.rows = f.rows;
  p.experts = (int)f.experts;
  p.act = f.act;
  p.split = 1;
  p.wide = f.hidden % 64 == 0 && f.ffn % 64 == 0;
  return p;
}

#define FFN_TRY(expr)               \
  do {                              \
    const int _st = (expr);         \
    if (_st != MUON_OK) return _st; \
  } while (0)

// an output of a row product, and of a weight gradient
void set_rows(Args &p, int i, void *base, int64_t ld) { p.outp[i] = base, p.out_ld[i] = ld; }
int set_dw(Args &p, int i, void *base, const FfnShape &f, int64_t rows, int64_t cols) {
  p.outp[i] = base;
  return map_out(&p.out[i], base, f.experts, rows, cols);
}

}  // namespace

int ffn_up(const FfnShape &f, const void *x, int64_t ldx, const void *w1, const void *w3, void *hid, void *gate,
           void *up, cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_rows(p.rows_of[0], x, f, f.hidden, ldx));
  FFN_TRY(map_mn(&p.a, w1, f.experts, f.hidden, f.ffn));
  FFN_TRY(map_mn(&p.a2, w3, f.experts, f.hidden, f.ffn));
  set_rows(p, 0, hid, f.ffn);
  set_rows(p, 1, gate, f.ffn);
  set_rows(p, 2, up, f.ffn);
  p.N = (int)f.ffn;
  p.kblocks = cdiv(f.hidden, BK);
  p.tiles_n = cdiv(f.ffn, BM);
  return launch<UP>(p, kTraceFfnUp, s);
}

int ffn_down(const FfnShape &f, const void *hid, const void *w2, void *y, int64_t ldy, cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_rows(p.rows_of[0], hid, f, f.ffn));
  FFN_TRY(map_cols(&p.a, p, w2, f.experts, f.ffn, f.hidden));
  set_rows(p, 0, y, ldy);
  p.N = (int)f.hidden;
  p.kblocks = cdiv(f.ffn, BK);
  p.tiles_n = cdiv(f.hidden, CM);
  return launch<DOWN>(p, kTraceFfnDown, s);
}

int ffn_dh(const FfnShape &f, const void *dy, int64_t lddy, const void *w2, const void *gate, const void *up, void *dg,
           void *du, void *hid, cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_rows(p.rows_of[0], dy, f, f.hidden, lddy));
  FFN_TRY(map_k(&p.a, w2, f.experts, f.ffn, f.hidden));
  set_rows(p, 0, dg, f.ffn);
  set_rows(p, 1, du, f.ffn);
  set_rows(p, 2, hid, f.ffn);
  p.g = static_cast<const __nv_bfloat16 *>(gate);
  p.u = static_cast<const __nv_bfloat16 *>(up);
  p.N = (int)f.ffn;
  p.kblocks = cdiv(f.hidden, BK);
  p.tiles_n = cdiv(f.ffn, CM);
  return launch<DH>(p, kTraceFfnDh, s);
}

int ffn_dx(const FfnShape &f, const void *dg, const void *du, const void *w1, const void *w3, void *dx, int64_t lddx,
           cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_rows(p.rows_of[0], dg, f, f.ffn));
  FFN_TRY(map_rows(p.rows_of[1], du, f, f.ffn));
  FFN_TRY(map_k(&p.a, w1, f.experts, f.hidden, f.ffn));
  FFN_TRY(map_k(&p.a2, w3, f.experts, f.hidden, f.ffn));
  set_rows(p, 0, dx, lddx);
  p.N = (int)f.hidden;
  p.kblocks = cdiv(f.ffn, BK);
  p.tiles_n = cdiv(f.hidden, CM);
  return launch<DX>(p, kTraceFfnDx, s);
}

namespace {

// A weight gradient of few tiles sums long columns of rows: the rows are cut into
// parts while they fit the SMs' pairs of CTAs (76), each of 8 k-blocks or more by
// the groups' average.  30000 rows of one expert, 512 x 512: dW1 and dW3 43 us against
// 141 uncut, dW2 35 against 142; 28429 rows of 2, 264 x 984: 66 against 105, 44
// against 105.
int dw_split(const FfnShape &f, int64_t tiles) {
  return (int)std::max<int64_t>(1, std::min<int64_t>({16, num_sms() / 2 / std::max<int64_t>(tiles * f.experts, 1),
                                                      f.rows / (f.experts * BK * 8)}));
}
int split13(const FfnShape &f) { return dw_split(f, (int64_t)cdiv(f.hidden, CM) * cdiv(f.ffn, BNH)); }
int split2(const FfnShape &f) { return dw_split(f, (int64_t)cdiv(f.ffn, CM) * cdiv(f.hidden, BN)); }

}  // namespace

size_t ffn_parts_elems(const FfnShape &f) {
  const int a = split13(f), b = split2(f);
  return (size_t)std::max(a > 1 ? 2 * a : 0, b > 1 ? b : 0) * f.experts * f.hidden * f.ffn;
}

size_t ffn_tail_elems(const FfnShape &f) { return (size_t)f.experts * BK * (2 * f.hidden + 3 * f.ffn); }

int ffn_dw(const FfnShape &f, const void *x, int64_t ldx, const void *dy, int64_t lddy, const void *dg, const void *du,
           const void *hid, void *tails, float *parts, void *dw1, void *dw3, void *dw2, cudaStream_t s) {
  // the five arrays' tails: x, dy, dg, du, hid
  TailArgs ta{};
  const void *src[5] = {x, dy, dg, du, hid};
  const int64_t ld[5] = {ldx, lddy, f.ffn, f.ffn, f.ffn};
  __nv_bfloat16 *t = static_cast<__nv_bfloat16 *>(tails);
  for (int i = 0; i < 5; ++i) {
    ta.src[i] = static_cast<const __nv_bfloat16 *>(src[i]);
    ta.ld[i] = ld[i];
    ta.cols[i] = (int)(i < 2 ? f.hidden : f.ffn);
    ta.dst[i] = t;
    t += (size_t)f.experts * BK * ta.cols[i];
  }
  ta.offsets = f.offsets;
  ta.rows = f.rows;
  trace_before(kTraceFfnTail, s);
  ffn_tail_kernel<<<dim3((unsigned)f.experts, 24, 5), 256, 0, s>>>(ta);
  FFN_TRY(trace_after(kTraceFfnTail, s));
  {
    Args p = base_args(f);
    FFN_TRY(map_cols(&p.a, p, x, 1, f.rows, f.hidden, ldx));
    FFN_TRY(map_cols(&p.a2, p, ta.dst[0], f.experts, BK, f.hidden));
    FFN_TRY(map_cols(&p.b, p, dg, 1, f.rows, f.ffn));
    FFN_TRY(map_cols(&p.b2, p, du, 1, f.rows, f.ffn));
    FFN_TRY(map_cols(&p.bt, p, ta.dst[2], f.experts, BK, f.ffn));
    FFN_TRY(map_cols(&p.bt2, p, ta.dst[3], f.experts, BK, f.ffn));
    FFN_TRY(set_dw(p, 0, dw1, f, f.hidden, f.ffn));
    FFN_TRY(set_dw(p, 1, dw3, f, f.hidden, f.ffn));
    p.M = (int)f.hidden;
    p.N = (int)f.ffn;
    p.tiles_m = cdiv(f.hidden, CM);
    p.tiles_n = cdiv(f.ffn, BNH);
    p.split = split13(f);
    p.parts = parts;
    FFN_TRY(launch<DW13>(p, kTraceFfnDw13, s));
  }
  Args p = base_args(f);
  FFN_TRY(map_cols(&p.a, p, hid, 1, f.rows, f.ffn));
  FFN_TRY(map_cols(&p.a2, p, ta.dst[4], f.experts, BK, f.ffn));
  FFN_TRY(map_cols(&p.b, p, dy, 1, f.rows, f.hidden, lddy));
  FFN_TRY(map_cols(&p.bt, p, ta.dst[1], f.experts, BK, f.hidden));
  FFN_TRY(set_dw(p, 0, dw2, f, f.ffn, f.hidden));
  p.M = (int)f.ffn;
  p.N = (int)f.hidden;
  p.tiles_m = cdiv(f.ffn, CM);
  p.tiles_n = cdiv(f.hidden, BN);
  p.split = split2(f);
  p.parts = parts;
  return launch<DW2>(p, kTraceFfnDw2, s);
}

}  // namespace muon
