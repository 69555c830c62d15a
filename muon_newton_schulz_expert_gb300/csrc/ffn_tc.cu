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
// on 256 x 256 output tiles (tcgen05.mma.cta_group::2, M = N = 256, K = 16,
// bf16 operands, fp32 accumulation in TMEM), fed by TMA through a ring of
// three stages of two k-blocks of 64.
//
// The two halves of a pair tile's N axis are loaded by the two CTAs of the
// pair.  UP and DW13 use that: the even CTA loads 128 columns of W1 (dG), the
// odd one the same 128 columns of W3 (dU), so that columns 0..127 of the
// accumulator hold G (dW1) and 128..255 U (dW3) of the same places.  One
// kernel forms both products, reads X once for both, and the activation and
// the product meet in one thread's registers.
//
// DX runs one K loop over both products: first dG W1^T, then dU W3^T.
//
// Rows of a group end anywhere.  The row products (UP, DOWN, DH, DX) compute
// whole tiles: rows past a group's end belong to the next expert and are
// computed but not stored (rows do not mix).  The weight gradients sum over
// the group's rows, so there the last, partial k-block must hold zeros past
// the group's end in both operands: it is read from copies of those rows
// padded with zeros (`tail` arrays, [experts][64][columns]), which keeps a
// NaN of one expert's rows out of another's gradient.  An expert without rows
// gets zeros.
//
// Rounding: Hid, dG and dU are stored in bf16, the operand type of the product
// that reads them; everything before that rounding is fp32.
//
// Roles per CTA (320 threads): warp 0 TMA producer, warp 1 MMA issuer (even
// CTA) and TMEM owner, warps 2..9 epilogue.  Two accumulators, so that the
// epilogue of one tile overlaps the next tile's products.  Every wait is
// bounded (tc.cuh).
#include <algorithm>

#include "ffn.cuh"

namespace muon {
namespace {

constexpr int CM = 256, BM = 128;   // rows of a pair tile, rows held by one CTA
constexpr int BN = 256, BNH = 128;  // columns of a pair tile, columns loaded by one CTA
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
  static constexpr bool a_mn = dw;
  static constexpr bool b_mn = MODE == UP || MODE == DOWN || dw;
  // two weight matrices side by side in the accumulator's columns
  static constexpr bool paired = MODE == UP || MODE == DW13;
};

struct Args {
  // operands: A and its second K segment (DX) or tail copy (DW); B and its
  // partner (UP: W3, DX: W3, DW13: dU) and their tail copies
  CUtensorMap a, a2, b, b2, bt, bt2;
  CUtensorMap out[3];                // boxes of 32 rows x 64 columns
  void *outp[3];
  long long out_ld[3];               // row strides in elements
  const int64_t *offsets;            // null: one group of all rows
  long long rows;
  int experts;
  int M, N;                          // DW: output rows; all: output columns of one weight matrix
  int kblocks;                       // row products: k-blocks of one K segment
  int tiles_m, tiles_n;              // DW: row tiles; all: column tiles
  int act;
  const __nv_bfloat16 *g, *u;        // DH: saved pre-activations [rows][N]
  unsigned *err;
  unsigned long long timeout_ns;
};

// A tile: expert, row tile and column tile, rows of the expert.
template <int MODE>
struct Tile {
  int e, ti, tj, lo, hi;

  __device__ Tile(const Args &p, const WarpCursor &cur) {
    e = cur.e, lo = cur.lo, hi = cur.hi;
    const int tm = Form<MODE>::dw ? p.tiles_m : (hi - lo + CM - 1) / CM;
    tj = (int)(cur.index / tm);
    ti = (int)(cur.index - (long long)tj * tm);
  }
  __device__ int num_kb(const Args &p) const {
    return Form<MODE>::dw ? (hi - lo + BK - 1) / BK : MODE == DX ? 2 * p.kblocks : p.kblocks;
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

// One epilogue warp's way out: 32 rows x 64 columns of bf16, lane = row.  A
// full box leaves through shared memory and TMA (clipped at the array's edge):
// 128-byte rows, since 64-byte ones (32 columns) held the stores of the weight
// gradients to 2.6 TB/s.  A box that a group ends in is written row by row.
struct Writer {
  uint8_t *box;
  uint32_t box_s;

  __device__ void put(const uint32_t (&w)[32], const CUtensorMap *map, void *base, long long ld, int lane, int col0,
                      int cols, long long row0, long long row_end, bool clip_rows, int mat, unsigned *err) {
    if (clip_rows && row0 + 32 > row_end) {
      const long long row = row0 + lane;
      if (row < row_end) {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(base) + row * ld + col0;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (col0 + 8 * c < cols)
            *reinterpret_cast<uint4 *>(dst + 8 * c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      }
      return;
    }
    if (lane == 0) bulk_wait_read_all();  // the box's last store has read it
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(map, box_s, col0, (int)row0, mat, err);
      bulk_commit();
    }
  }
};

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
    tma_prefetch_desc(&p.b);
    tma_prefetch_desc(&p.out[0]);
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
  WarpCursor walk(p.offsets, p.rows, p.experts, Form<MODE>::dw ? 0 : CM,
                  (long long)(Form<MODE>::dw ? p.tiles_m : 1) * p.tiles_n);

  if (warp == 0) {
    // ---------------------------------------------------------------- producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0, issued_parity = 0;  // stages ever filled, and the parity of their last fill
    bool ok = true;
    for (long long t = cid; walk.seek(t); t += ncl) {
      const Tile<MODE> cur(p, walk);
      if (lane == 0 && ok) {
        const int num_kb = cur.num_kb(p);
        const int mn_a = cur.ti * CM + (int)rank * BM;   // DW: first column of A's rows in this CTA
        const int row_a = cur.lo + mn_a;                 // row products: first row
        const int n_b = Form<MODE>::paired ? cur.tj * BNH : cur.tj * BN + (int)rank * BNH;
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
            for (int j = 0; j < KSUB; ++j) mbar_expect_tx(full(stage, j), j < valid ? 2 * KB_BYTES : 0);
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
#pragma unroll
          for (int j = 0; j < KSUB; ++j) {
            if (j >= valid) break;
            const int k = kb + j;
            const uint32_t sa = sbase + stage * STAGE_BYTES + j * KB_BYTES, sb = sa + A_STAGE;
            const uint32_t bar = map_to_rank(full(stage, j), 0);
            if (Form<MODE>::dw) {
              // boxes of 64 columns x 64 rows; the group's last rows from the padded copies
              const bool tail = cur.hi - cur.lo - k * BK < BK;
              const int kr = tail ? 0 : cur.lo + k * BK, z = tail ? cur.e : 0;
              const CUtensorMap *ma = tail ? &p.a2 : &p.a;
              const CUtensorMap *mbk = !tail ? mb : Form<MODE>::paired && rank ? &p.bt2 : &p.bt;
#pragma unroll
              for (int q = 0; q < 2; ++q)
                tma_load_3d_pair(sa + q * (64 * BK * 2), ma, bar, mn_a + q * 64, kr, z, p.err);
#pragma unroll
              for (int q = 0; q < 2; ++q)
                tma_load_3d_pair(sb + q * (64 * BK * 2), mbk, bar, n_b + q * 64, kr, z, p.err);
            } else {
              const bool second = MODE == DX && k >= p.kblocks;
              const int kc = (second ? k - p.kblocks : k) * BK;
              tma_load_3d_pair(sa, second ? &p.a2 : &p.a, bar, kc, row_a, 0, p.err);
              if (Form<MODE>::b_mn) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  tma_load_3d_pair(sb + q * (64 * BK * 2), mb, bar, n_b + q * 64, kc, cur.e, p.err);
              } else {
                tma_load_3d_pair(sb, second ? &p.b2 : &p.b, bar, kc, n_b, cur.e, p.err);
              }
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
      constexpr uint32_t idesc = make_idesc(CM, BN, Form<MODE>::a_mn, Form<MODE>::b_mn);
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
          const int num_kb = cur.num_kb(p);
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
    Writer out{epi_smem + ew * BOX_BYTES, smem_u32(epi_smem) + (uint32_t)(ew * BOX_BYTES)};
    int acc = 0;
    uint32_t acc_phase = 0;
    for (long long t = cid; walk.seek(t); t += ncl) {
      const Tile<MODE> cur(p, walk);
      const bool ok = wait_bounded(accf(acc), acc_phase, w);
      if (!__all_sync(0xffffffffu, ok)) break;  // warp-uniform: the TMEM loads below are .sync.aligned
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * ACC_COLS);
      const int rt = cur.ti * CM + (int)rank * BM + q * 32;
      const long long row0 = Form<MODE>::dw ? rt : (long long)cur.lo + rt;
      const long long row_end = Form<MODE>::dw ? p.M : cur.hi;
      const int mat = Form<MODE>::dw ? cur.e : 0;
      if (row0 < row_end) {
        if (MODE == UP) {
          // this warp's 64 columns of the tile: G from the low half of the accumulator, U from the high one
          const int cc = half * 64, col0 = cur.tj * BNH + cc;
          if (col0 < p.N) {
            uint32_t wg[32], wu[32], wh[32];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t g[32], u[32];
              tmem_ld32(taddr + (uint32_t)(cc + 32 * part), g);
              tmem_ld32(taddr + (uint32_t)(BNH + cc + 32 * part), u);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float h[2], dv;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float gf = __uint_as_float(g[2 * i + j]);
                  h[j] = gf * sigmoid_of(gf, p.act, &dv) * __uint_as_float(u[2 * i + j]);
                }
                wh[16 * part + i] = pack_bf16(h[0], h[1]);
                wg[16 * part + i] = pack_bf16(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
                wu[16 * part + i] = pack_bf16(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
              }
            }
            out.put(wh, &p.out[0], p.outp[0], p.out_ld[0], lane, col0, p.N, row0, row_end, true, 0, p.err);
            if (p.outp[1]) {
              out.put(wg, &p.out[1], p.outp[1], p.out_ld[1], lane, col0, p.N, row0, row_end, true, 0, p.err);
              out.put(wu, &p.out[2], p.outp[2], p.out_ld[2], lane, col0, p.N, row0, row_end, true, 0, p.err);
            }
          }
        } else if (MODE == DH) {
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            const int cc = half * 128 + ch * 64, col0 = cur.tj * BN + cc;
            if (col0 >= p.N) break;
            uint32_t wg[32], wu[32], wh[32];   // g, u and then dg, du in wg and wu
            const bool in_row = row0 + lane < row_end;
            const long long at = (row0 + lane) * p.N + col0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
              if (in_row && col0 + 8 * c < p.N) {
                a = __ldg(reinterpret_cast<const uint4 *>(p.g + at + 8 * c));
                b = __ldg(reinterpret_cast<const uint4 *>(p.u + at + 8 * c));
              }
              wg[4 * c] = a.x, wg[4 * c + 1] = a.y, wg[4 * c + 2] = a.z, wg[4 * c + 3] = a.w;
              wu[4 * c] = b.x, wu[4 * c + 1] = b.y, wu[4 * c + 2] = b.z, wu[4 * c + 3] = b.w;
            }
            __syncwarp();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t r[32];
              tmem_ld32(taddr + (uint32_t)(cc + 32 * part), r);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 g2 = unpack_bf16(wg[16 * part + i]), u2 = unpack_bf16(wu[16 * part + i]);
                float dg[2], du[2], h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  gated_gradient(__uint_as_float(r[2 * i + j]), j ? g2.y : g2.x, j ? u2.y : u2.x, p.act, &dg[j], &du[j],
                                 &h[j]);
                wg[16 * part + i] = pack_bf16(dg[0], dg[1]);
                wu[16 * part + i] = pack_bf16(du[0], du[1]);
                wh[16 * part + i] = pack_bf16(h[0], h[1]);
              }
            }
            out.put(wg, &p.out[0], p.outp[0], p.out_ld[0], lane, col0, p.N, row0, row_end, true, 0, p.err);
            out.put(wu, &p.out[1], p.outp[1], p.out_ld[1], lane, col0, p.N, row0, row_end, true, 0, p.err);
            out.put(wh, &p.out[2], p.outp[2], p.out_ld[2], lane, col0, p.N, row0, row_end, true, 0, p.err);
          }
        } else {
          const bool empty_sum = Form<MODE>::dw && cur.hi == cur.lo;  // no MMA ran: the accumulator holds nothing
          const int which = Form<MODE>::paired ? half : 0;            // DW13: dW1 in the low columns, dW3 in the high
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            const int cc = half * 128 + ch * 64;
            const int col0 = Form<MODE>::paired ? cur.tj * BNH + ch * 64 : cur.tj * BN + cc;
            if (col0 >= p.N) break;
            uint32_t lo[32], hi[32], wo[32];
            tmem_ld64(taddr + (uint32_t)cc, lo, hi);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              wo[i] = empty_sum ? 0u : pack_bf16(__uint_as_float(lo[2 * i]), __uint_as_float(lo[2 * i + 1]));
              wo[16 + i] = empty_sum ? 0u : pack_bf16(__uint_as_float(hi[2 * i]), __uint_as_float(hi[2 * i + 1]));
            }
            out.put(wo, &p.out[which], p.outp[which], p.out_ld[which], lane, col0, p.N, row0, row_end,
                    !Form<MODE>::dw, mat, p.err);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(acce(acc), 0));
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
      Form<MODE>::dw ? (long long)p.tiles_m * p.experts : p.rows / CM + std::min<long long>(p.experts, p.rows);
  const long long pairs = std::min<long long>(row_tiles * p.tiles_n, max_pairs[dev]);
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.numAttrs = 2;
  cfg.stream = s;
  trace_before(trace_kind, s);
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, p);
  const int st = trace_after(trace_kind, s);
  return le == cudaSuccess ? st : MUON_ERR_CUDA;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// operand maps: K-major rows (boxes of 128 rows x 64 columns), MN-major (64 x 64)
int map_k(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols, int64_t ld = 0) {
  return make_map(m, base, batch, rows, cols, 128, ld);
}
int map_mn(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols, int64_t ld = 0) {
  return make_map(m, base, batch, rows, cols, 64, ld);
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
  return p;
}

#define FFN_TRY(expr)               \
  do {                              \
    const int _st = (expr);         \
    if (_st != MUON_OK) return _st; \
  } while (0)

int set_out(Args &p, int i, void *base, int64_t batch, int64_t rows, int64_t cols, int64_t ld) {
  p.outp[i] = base;
  p.out_ld[i] = ld;
  return base ? map_out(&p.out[i], base, batch, rows, cols, ld) : MUON_OK;
}

}  // namespace

int ffn_up(const FfnShape &f, const void *x, int64_t ldx, const void *w1, const void *w3, void *hid, void *gate,
           void *up, cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_k(&p.a, x, 1, f.rows, f.hidden, ldx));
  FFN_TRY(map_mn(&p.b, w1, f.experts, f.hidden, f.ffn));
  FFN_TRY(map_mn(&p.b2, w3, f.experts, f.hidden, f.ffn));
  FFN_TRY(set_out(p, 0, hid, 1, f.rows, f.ffn, f.ffn));
  FFN_TRY(set_out(p, 1, gate, 1, f.rows, f.ffn, f.ffn));
  FFN_TRY(set_out(p, 2, up, 1, f.rows, f.ffn, f.ffn));
  p.N = (int)f.ffn;
  p.kblocks = cdiv(f.hidden, BK);
  p.tiles_n = cdiv(f.ffn, BNH);
  return launch<UP>(p, kTraceFfnUp, s);
}

int ffn_down(const FfnShape &f, const void *hid, const void *w2, void *y, int64_t ldy, cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_k(&p.a, hid, 1, f.rows, f.ffn));
  FFN_TRY(map_mn(&p.b, w2, f.experts, f.ffn, f.hidden));
  FFN_TRY(set_out(p, 0, y, 1, f.rows, f.hidden, ldy));
  p.N = (int)f.hidden;
  p.kblocks = cdiv(f.ffn, BK);
  p.tiles_n = cdiv(f.hidden, BN);
  return launch<DOWN>(p, kTraceFfnDown, s);
}

int ffn_dh(const FfnShape &f, const void *dy, int64_t lddy, const void *w2, const void *gate, const void *up, void *dg,
           void *du, void *hid, cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_k(&p.a, dy, 1, f.rows, f.hidden, lddy));
  FFN_TRY(map_k(&p.b, w2, f.experts, f.ffn, f.hidden));
  FFN_TRY(set_out(p, 0, dg, 1, f.rows, f.ffn, f.ffn));
  FFN_TRY(set_out(p, 1, du, 1, f.rows, f.ffn, f.ffn));
  FFN_TRY(set_out(p, 2, hid, 1, f.rows, f.ffn, f.ffn));
  p.g = static_cast<const __nv_bfloat16 *>(gate);
  p.u = static_cast<const __nv_bfloat16 *>(up);
  p.N = (int)f.ffn;
  p.kblocks = cdiv(f.hidden, BK);
  p.tiles_n = cdiv(f.ffn, BN);
  return launch<DH>(p, kTraceFfnDh, s);
}

int ffn_dx(const FfnShape &f, const void *dg, const void *du, const void *w1, const void *w3, void *dx, int64_t lddx,
           cudaStream_t s) {
  Args p = base_args(f);
  FFN_TRY(map_k(&p.a, dg, 1, f.rows, f.ffn));
  FFN_TRY(map_k(&p.a2, du, 1, f.rows, f.ffn));
  FFN_TRY(map_k(&p.b, w1, f.experts, f.hidden, f.ffn));
  FFN_TRY(map_k(&p.b2, w3, f.experts, f.hidden, f.ffn));
  FFN_TRY(set_out(p, 0, dx, 1, f.rows, f.hidden, lddx));
  p.N = (int)f.hidden;
  p.kblocks = cdiv(f.ffn, BK);
  p.tiles_n = cdiv(f.hidden, BN);
  return launch<DX>(p, kTraceFfnDx, s);
}

size_t ffn_tail_elems(const FfnShape &f) { return (size_t)f.experts * BK * (2 * f.hidden + 3 * f.ffn); }

int ffn_dw(const FfnShape &f, const void *x, int64_t ldx, const void *dy, int64_t lddy, const void *dg, const void *du,
           const void *hid, void *tails, void *dw1, void *dw3, void *dw2, cudaStream_t s) {
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
  ffn_tail_kernel<<<dim3((unsigned)f.experts, 8, 5), 256, 0, s>>>(ta);
  FFN_TRY(trace_after(kTraceFfnTail, s));
  {
    Args p = base_args(f);
    FFN_TRY(map_mn(&p.a, x, 1, f.rows, f.hidden, ldx));
    FFN_TRY(map_mn(&p.a2, ta.dst[0], f.experts, BK, f.hidden));
    FFN_TRY(map_mn(&p.b, dg, 1, f.rows, f.ffn));
    FFN_TRY(map_mn(&p.b2, du, 1, f.rows, f.ffn));
    FFN_TRY(map_mn(&p.bt, ta.dst[2], f.experts, BK, f.ffn));
    FFN_TRY(map_mn(&p.bt2, ta.dst[3], f.experts, BK, f.ffn));
    FFN_TRY(set_out(p, 0, dw1, f.experts, f.hidden, f.ffn, f.ffn));
    FFN_TRY(set_out(p, 1, dw3, f.experts, f.hidden, f.ffn, f.ffn));
    p.M = (int)f.hidden;
    p.N = (int)f.ffn;
    p.tiles_m = cdiv(f.hidden, CM);
    p.tiles_n = cdiv(f.ffn, BNH);
    FFN_TRY(launch<DW13>(p, kTraceFfnDw13, s));
  }
  Args p = base_args(f);
  FFN_TRY(map_mn(&p.a, hid, 1, f.rows, f.ffn));
  FFN_TRY(map_mn(&p.a2, ta.dst[4], f.experts, BK, f.ffn));
  FFN_TRY(map_mn(&p.b, dy, 1, f.rows, f.hidden, lddy));
  FFN_TRY(map_mn(&p.bt, ta.dst[1], f.experts, BK, f.hidden));
  FFN_TRY(set_out(p, 0, dw2, f.experts, f.ffn, f.hidden, f.hidden));
  p.M = (int)f.ffn;
  p.N = (int)f.hidden;
  p.tiles_m = cdiv(f.ffn, CM);
  p.tiles_n = cdiv(f.hidden, BN);
  return launch<DW2>(p, kTraceFfnDw2, s);
}

}  // namespace muon
