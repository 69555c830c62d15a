// Row products of the gated feed-forward block for few rows: decoding, and
// training with so few rows that ffn_tc.cu's 256 x 256 tiles would occupy a
// part of the SMs only.
//
// With few rows a product reads its weights once and little else, so it is
// bound by their bandwidth and needs every SM to stream a share of them.  The
// roles of the operands are exchanged (weights on M, rows on N):
//   D[128 weight columns, TN rows] = W^T X^T
// with tcgen05.mma of one CTA (M = 128, N = TN = 16, 32 or 64), and the K loop
// is cut into S parts (1 to 8) that the CTAs of a cluster take.  Each CTA
// finishes a part of the tile's columns: all send it their parts of its sums
// (fp32, distributed shared memory), and after a cluster barrier it adds them in
// order of rank.  Stores to the others need no answer: reading the parts where
// they were made took 1.2 to 3.3 us a tile, this 1.5 us less (one row, 6144 x 1792,
// from HBM: 23.9 against 22.4 us; 64 rows 32.1 against 27.6 us).  No workspace, no
// atomics, one launch per product.
//   UP    two accumulators (W1, W3) over one load of the rows; h = act(g) * u
//   DOWN  y = h W2; h comes as two bf16 halves (value and remainder), which
//         are 2 TN rows of one N, so h's rounding costs no accuracy and the
//         weights are still read once
//   DH    dh = dy W2^T, then dg, du, h;    DX  dx = dg W1^T + du W3^T
//
// Roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer and TMEM owner,
// warps 2..5 accumulators out of TMEM; all add and finish where K is cut.
// Without a cut (S = 1) the tiles are a stream: producer and MMA run ahead.
// Every wait is bounded (tc.cuh); a role that gave up still takes part in the
// cluster barriers, so none of them is left waiting.
#include <algorithm>

#include "ffn.cuh"

namespace muon {
namespace {

constexpr int BM = 128, BK = 64, UMMA_K = 16;
constexpr int A_BYTES = BM * BK * 2;
constexpr int EPI_THREADS = 128, THREADS = 64 + EPI_THREADS;
constexpr int MAX_STAGES = 12, MAX_TN = 64;
constexpr int NUM_BARS = 2 * MAX_STAGES + 4;

enum Mode { UP = 0, DOWN, DH, DX };

struct Args {
  CUtensorMap a, a2, b, b2;      // weights (UP, DX: W1 and W3), rows (DOWN: both halves of h, DX: dg and du)
  const int64_t *offsets;
  long long rows;
  int experts;
  int M;                         // output columns of one weight matrix
  int kblocks, segments;         // k-blocks of one K segment, and segments (DX: 2)
  int tiles_m, tn, split, stages;
  int act;
  long long ld;                  // row stride of y or dx
  __nv_bfloat16 *out[4];         // UP: h, h's remainder, gate, up; DOWN: y; DH: dg, du, h; DX: dx
  const __nv_bfloat16 *g, *u;    // DH
  unsigned *err;
  unsigned long long timeout_ns;
};

// tiles: expert, 128 weight columns, up to tn rows
struct Tile {
  int e, tm, row0, hi;

  __device__ Tile(const Args &p, const WarpCursor &cur) {
    const int tt = (cur.hi - cur.lo + p.tn - 1) / p.tn;
    e = cur.e;
    tm = (int)((unsigned)cur.index / (unsigned)tt);   // few tiles: 32 bits hold their number
    row0 = cur.lo + ((int)cur.index - tm * tt) * p.tn;
    hi = cur.hi;
  }
};

__device__ __forceinline__ void tc_mma1(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_commit1(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t *>(&h);
}

// four values as bf16; what the rounding left, if asked for
__device__ __forceinline__ void put4(__nv_bfloat16 *dst, __nv_bfloat16 *rest, const float (&v)[4]) {
  const uint2 w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  *reinterpret_cast<uint2 *>(dst) = w;
  if (rest) {
    const float d0 = v[0] - __uint_as_float(w.x << 16), d1 = v[1] - __uint_as_float(w.x & 0xffff0000u);
    const float d2 = v[2] - __uint_as_float(w.y << 16), d3 = v[3] - __uint_as_float(w.y & 0xffff0000u);
    // an infinite or NaN value has no remainder to add
    *reinterpret_cast<uint2 *>(rest) = make_uint2(pack_bf16(isfinite(d0) ? d0 : 0.f, isfinite(d1) ? d1 : 0.f),
                                                  pack_bf16(isfinite(d2) ? d2 : 0.f, isfinite(d3) ? d3 : 0.f));
  }
}

// The columns of a tile that a CTA of its cluster finishes: as many as any other,
// the last CTA possibly fewer, in fours.
__device__ __forceinline__ int cut_width(int split) { return (32 + split - 1) / split * 4; }

// Adds the S parts of this CTA's columns and finishes them: items of 4 columns of
// one row.  `part` holds the parts, [rank][accumulator][row][width].
template <int MODE>
__device__ __forceinline__ void finish(const Args &p, const Tile &cur, const float *part, int rank, int width,
                                       int thread, int threads) {
  const int n = min(cur.hi - cur.row0, p.tn);
  const int quads = min(width, BM - rank * width) / 4;
  const int col_base = cur.tm * BM + rank * width, per_mat = p.tn * width, per_rank = (MODE == UP ? 2 : 1) * per_mat;
  for (int i = thread; i < n * quads; i += threads) {
    const int t = i / quads, c = (i - t * quads) * 4, col = col_base + c;
    if (col >= p.M) continue;   // M is a multiple of 8
    float s0[4] = {}, s1[4] = {};
    const float *from = part + t * width + c;
#pragma unroll 4
    for (int r = 0; r < p.split; ++r, from += per_rank) {
      const float4 x = *reinterpret_cast<const float4 *>(from);
      s0[0] += x.x, s0[1] += x.y, s0[2] += x.z, s0[3] += x.w;
      if (MODE == UP) {
        const float4 y = *reinterpret_cast<const float4 *>(from + per_mat);
        s1[0] += y.x, s1[1] += y.y, s1[2] += y.z, s1[3] += y.w;
      }
    }
    const long long row = (long long)cur.row0 + t;
    if (MODE == UP) {
      const long long at = row * p.M + col;
      float h[4], dv;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = s0[j] * sigmoid_of(s0[j], p.act, &dv) * s1[j];
      put4(p.out[0] + at, p.out[1] + at, h);
      if (p.out[2]) {
        put4(p.out[2] + at, nullptr, s0);
        put4(p.out[3] + at, nullptr, s1);
      }
    } else if (MODE == DH) {
      const long long at = row * p.M + col;
      const uint2 gw = *reinterpret_cast<const uint2 *>(p.g + at), uw = *reinterpret_cast<const uint2 *>(p.u + at);
      const uint32_t g2[2] = {gw.x, gw.y}, u2[2] = {uw.x, uw.y};
      float dg[4], du[4], h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g = __uint_as_float(j & 1 ? g2[j >> 1] & 0xffff0000u : g2[j >> 1] << 16);
        const float u = __uint_as_float(j & 1 ? u2[j >> 1] & 0xffff0000u : u2[j >> 1] << 16);
        gated_gradient(s0[j], g, u, p.act, &dg[j], &du[j], &h[j]);
      }
      put4(p.out[0] + at, nullptr, dg);
      put4(p.out[1] + at, nullptr, du);
      put4(p.out[2] + at, nullptr, h);
    } else {
      put4(p.out[0] + row * p.ld + col, nullptr, s0);
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(THREADS) ffn_few_kernel(const __grid_constant__ Args p) {
  constexpr bool A_MN = MODE == UP || MODE == DOWN;
  constexpr int MATS = MODE == UP ? 2 : 1;        // weight tiles of a stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int n_rows = MODE == DOWN ? 2 * p.tn : p.tn;   // N of one MMA
  // TMEM: two accumulators, UP's and DOWN's of 2 tn columns (64 to 256 in all, a power of two)
  const uint32_t acc_cols = (MODE == UP || MODE == DOWN ? 2u : 1u) * p.tn, tmem_cols = max(64u, 2 * acc_cols);
  const uint32_t b_bytes = (uint32_t)n_rows * (BK * 2), stage_bytes = MATS * A_BYTES + b_bytes;
  const int width = cut_width(p.split);
  float *part = reinterpret_cast<float *>(smem + p.stages * stage_bytes);   // [split][MATS][tn][width]
  uint64_t *bars = reinterpret_cast<uint64_t *>(part + p.split * MATS * p.tn * width);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NUM_BARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool cut = p.split > 1;
  const int rank = cut ? (int)cluster_rank() : 0;
  const long long cid = blockIdx.x / p.split, ncl = gridDim.x / p.split;
  auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(MAX_STAGES + s); };
  auto accf = [&](int a) { return bar0 + 8u * (uint32_t)(2 * MAX_STAGES + a); };
  auto acce = [&](int a) { return bar0 + 8u * (uint32_t)(2 * MAX_STAGES + 2 + a); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf(a), 1);
      mbar_init(acce(a), 4);   // the warps that read the accumulator
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.a);
    tma_prefetch_desc(&p.b);
  }
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (cut) cluster_arrive();   // this CTA runs, and its parts may be written
  // UP and DH read what earlier calls wrote, offsets among it; DOWN and DX run
  // after one of them in the same call, so that only the rows that it makes are
  // waited for, below.
  constexpr bool SECOND = MODE == DOWN || MODE == DX;
  if (!SECOND) {
    wait_for_previous_grid();
    let_next_grid_start();
  }
  if (warp == 2 && blockIdx.x == 0) report_offsets(p.offsets, p.experts, p.rows, p.err);
  const Watch w{abort_flag, p.err, p.timeout_ns};
  const unsigned long long drain_ns = p.timeout_ns < 20000000ull ? p.timeout_ns : 20000000ull;
  // this CTA's share of the K loop
  const int all_kb = p.kblocks * p.segments;
  const int kb0 = all_kb * rank / p.split, kb1 = all_kb * (rank + 1) / p.split;   // all_kb < 2^26

  WarpCursor walk(p.offsets, p.rows, p.experts, p.tn, p.tiles_m);
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;   // of this warp's role
  bool rows_ready = !SECOND;
  long long t = cid;
  bool more = walk.seek(t);
  if (cut && !more) cluster_wait();
  while (more) {
    const Tile cur(p, walk);
    if (warp == 0) {
      if (lane == 0 && ok) {
        auto rows_of = [&](int k, int st) {
          const bool second = MODE == DX && k >= p.kblocks;
          const int kc = (second ? k - p.kblocks : k) * BK;
          const uint32_t sb = sbase + st * stage_bytes + MATS * A_BYTES;
          tma_load_3d(sb, second ? &p.b2 : &p.b, full(st), kc, cur.row0, 0, p.err);
          if (MODE == DOWN) tma_load_3d(sb + p.tn * (BK * 2), &p.b2, full(st), kc, cur.row0, 0, p.err);
        };
        for (int k = kb0; k < kb1; ++k) {
          if (!wait_polled(empty(stage), phase ^ 1u, w)) {
            ok = false;
            break;
          }
          mbar_expect_tx(full(stage), stage_bytes);
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          const bool second = MODE == DX && k >= p.kblocks;
          const int kc = (second ? k - p.kblocks : k) * BK, m0 = cur.tm * BM;
          const uint32_t sa = sbase + stage * stage_bytes, bar = full(stage);
#pragma unroll
          for (int i = 0; i < MATS; ++i) {
            const CUtensorMap *ma = i || second ? &p.a2 : &p.a;
            if (A_MN) {   // boxes of 64 weight columns x 64 K-rows
              tma_load_3d(sa + i * A_BYTES, ma, bar, m0, kc, cur.e, p.err);
              tma_load_3d(sa + i * A_BYTES + A_BYTES / 2, ma, bar, m0 + 64, kc, cur.e, p.err);
            } else {      // one box of 128 weight rows x 64 K-columns
              tma_load_3d(sa, ma, bar, kc, m0, cur.e, p.err);
            }
          }
          if (rows_ready) {
            rows_of(k, stage);
          } else if (k + 1 == kb1 || k + 1 - kb0 == p.stages) {
            // the first stages' weights are on their way; their rows once the
            // kernel that makes them has ended
            wait_for_previous_grid();
            rows_ready = true;
            for (int i = kb0; i <= k; ++i) rows_of(i, i - kb0);
          }
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      if (lane == 0 && ok) {
        const uint32_t idesc = make_idesc(BM, n_rows, A_MN, false);
        ok = wait_bounded(acce(acc), acc_phase ^ 1u, w);
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)acc * acc_cols;
        for (int k = kb0; ok && k < kb1; ++k) {
          if (!wait_polled(full(stage), phase, w)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = sbase + stage * stage_bytes, sb = sa + MATS * A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk) {
            const uint64_t bd = smem_desc(sb + kk * (UMMA_K * 2), 16, 1024);
#pragma unroll
            for (int i = 0; i < MATS; ++i) {
              const uint32_t at = sa + i * A_BYTES;
              const uint64_t ad = A_MN ? smem_desc(at + kk * (UMMA_K * 128), 64 * BK * 2, 1024)
                                       : smem_desc(at + kk * (UMMA_K * 2), 16, 1024);
              tc_mma1(d + (uint32_t)(i * p.tn), ad, bd, idesc, ((k - kb0) | kk) != 0 ? 1u : 0u);
            }
          }
          tc_commit1(empty(stage));
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit1(accf(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
    } else {
      const int q = warp & 3;   // TMEM lanes 32q..
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(accf(acc), acc_phase, w));
      if (cut) cluster_wait();   // the parts of the tile before have been added
      if (ok) {
        tc_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * acc_cols;
        // this lane's column: the CTA that finishes it, and its place there
        const int column = q * 32 + lane, owner = column / width;
        const uint32_t here = smem_u32(part);
        const uint32_t there = (cut ? map_to_rank(here, (uint32_t)owner) : here) +
                               4u * (uint32_t)(rank * MATS * p.tn * width + column - owner * width);
        const int n = min(cur.hi - cur.row0, p.tn);
#pragma unroll
        for (int i = 0; i < MATS; ++i)
          for (int c = 0; c < n; c += 16) {
            uint32_t r[32], r2[32];
            tmem_ld16(taddr + (uint32_t)(i * p.tn + c), r);
            if (MODE == DOWN) tmem_ld16(taddr + (uint32_t)(p.tn + c), r2);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < n)
                st_cluster(there + 4u * (uint32_t)((i * p.tn + c + j) * width),
                           MODE == DOWN ? __uint_as_float(r[j]) + __uint_as_float(r2[j]) : __uint_as_float(r[j]));
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!cut) {
        // the four warps have the whole tile in `part`
        asm volatile("bar.sync 1, %0;" ::"r"(EPI_THREADS) : "memory");
        if (ok) finish<MODE>(p, cur, part, 0, width, (int)threadIdx.x - 64, EPI_THREADS);
        asm volatile("bar.sync 1, %0;" ::"r"(EPI_THREADS) : "memory");
      }
    }
    __syncwarp();
    if (cut) {
      if (warp < 2) cluster_wait();
      cluster_sync_all();   // all parts of this CTA's columns are here
      if (!*abort_flag) finish<MODE>(p, cur, part, rank, width, (int)threadIdx.x, THREADS);
    }
    t += ncl;
    more = walk.seek(t);
    if (cut && more) cluster_arrive();   // and have been added
  }
  // a kernel ends after the one it was started early beside, whatever it had to do
  if (!rows_ready) wait_for_previous_grid();
  // After an abort, stages may still be filling: let those copies land.  MMAs
  // already issued complete by themselves; a full barrier they wait for cannot
  // be outstanding, since they are issued after it.
  if (warp == 0 && lane == 0 && *abort_flag)
    for (int s2 = 0; s2 < p.stages; ++s2)
      if (issued & (1u << s2)) drain_wait(full(s2), (issued_parity >> s2) & 1u, drain_ns);
  if (warp == 1 && lane == 0 && *abort_flag) {
    const unsigned long long t0 = global_ns();   // the last MMAs end within microseconds
    while (global_ns() - t0 < 200000ull) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols) : "memory");
  }
}

// Rows of a tile, by the rows an expert has on average (twice that, since
// routers are uneven), so that few tiles are mostly empty.
int row_tile(const FfnShape &f) {
  const int64_t per = f.experts == 1 ? f.rows : std::min(f.rows, 2 * ((f.rows + f.experts - 1) / f.experts));
  return per <= 16 ? 16 : per <= 32 ? 32 : MAX_TN;
}

template <int MODE>
int launch(Args &p, const FfnShape &f, int trace_kind, cudaStream_t s) {
  constexpr int MATS = MODE == UP ? 2 : 1;
  const int64_t active = std::min(f.experts, f.rows);
  p.tn = row_tile(f);
  // UP takes an SM for itself (34 to 40 KB stages: 4 of 16 rows, 3 of 64), the
  // others share it between two blocks.  K is cut while the blocks still fit
  // the SMs at once and each keeps 6 k-blocks or more (6144 x 1792, one row, in
  // L2: 53 us uncut, 34, 24 and 21 us cut in 2, 4 and 8; from HBM 22.4 us, and
  // 27.4 us if 4 k-blocks are enough, which cuts DOWN in 6 instead of 4 and
  // leaves its clusters waiting for places; 2048 x 1024 takes 19.6 us with 6
  // k-blocks, 18.6 us with 4).  Of the 22.4 us the weights' bytes take 9.8 at the
  // copy bandwidth; each kernel adds about 1.5 us until its first loads leave,
  // 1 us for their latency, 2 to 3 us for sums, exchange and end.
  const int per_sm = MODE == UP ? 1 : 2;
  const int64_t tiles = (int64_t)p.tiles_m * (f.experts == 1 ? (f.rows + p.tn - 1) / p.tn : active);
  const int all_kb = p.kblocks * p.segments;
  p.split = 1;
  while (p.split < 8 && (p.split + 1) * tiles <= (int64_t)num_sms() * per_sm && 6 * (p.split + 1) <= all_kb) ++p.split;
  const size_t stage = MATS * A_BYTES + (size_t)(MODE == DOWN ? 2 : 1) * p.tn * BK * 2;
  const size_t parts = (size_t)p.split * ((32 + p.split - 1) / p.split * 4) * MATS * p.tn * 4;
  const size_t fixed = 1024 + parts + NUM_BARS * 8 + 16;
  const size_t budget = MODE != UP ? 112 * 1024 : p.tn == MAX_TN ? 220 * 1024 : 160 * 1024;
  p.stages = (int)std::min<size_t>({(size_t)MAX_STAGES, (budget - fixed) / stage,
                                    (size_t)std::max(2, (all_kb + p.split - 1) / p.split)});
  if (p.stages < 2) return MUON_ERR_UNSUPPORTED;   // cannot be: DOWN has 2 of 64 rows, every other case more
  const size_t smem = fixed + p.stages * stage;
  p.err = device_error_word();
  p.timeout_ns = wait_timeout_ns();
  if (!p.err) return MUON_ERR_CUDA;
  auto *kernel = ffn_few_kernel<MODE>;
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         MODE == UP ? 220 * 1024 : 112 * 1024);
    cudaGetLastError();
  });
  if (attr_err[dev] != cudaSuccess) return MUON_ERR_CUDA;
  // at most this many tiles, whatever the groups' sizes are
  const int64_t most = ((f.rows + p.tn - 1) / p.tn + active) * p.tiles_m;
  const int64_t clusters = std::min<int64_t>(most, std::max(1, num_sms() * per_sm / p.split));
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS);
  cfg.gridDim = dim3((unsigned)(clusters * p.split));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  trace_before(trace_kind, s);
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, p);
  const int st = trace_after(trace_kind, s);
  return le == cudaSuccess ? st : MUON_ERR_CUDA;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int map_weights(CUtensorMap *m, const void *base, const FfnShape &f, int64_t rows, int64_t cols, bool mn) {
  return make_map(m, base, f.experts, rows, cols, mn ? 64 : 128);
}
int map_rows(CUtensorMap *m, const void *base, const FfnShape &f, int64_t cols, int64_t ld) {
  return make_map(m, base, 1, f.rows, cols, row_tile(f), ld);
}

Args base_args(const FfnShape &f, int64_t M, int64_t K) {
  Args p{};
  p.offsets = f.offsets;
  p.rows = f.rows;
  p.experts = (int)f.experts;
  p.act = f.act;
  p.M = (int)M;
  p.tiles_m = cdiv(M, BM);
  p.kblocks = cdiv(K, BK);
  p.segments = 1;
  return p;
}

__nv_bfloat16 *bf(void *v) { return static_cast<__nv_bfloat16 *>(v); }

#define FFN_TRY(expr)               \
  do {                              \
    const int _st = (expr);         \
    if (_st != MUON_OK) return _st; \
  } while (0)

}  // namespace

int ffn_few_up(const FfnShape &f, const void *x, int64_t ldx, const void *w1, const void *w3, void *hid, void *hid_rest,
               void *gate, void *up, cudaStream_t s) {
  Args p = base_args(f, f.ffn, f.hidden);
  FFN_TRY(map_weights(&p.a, w1, f, f.hidden, f.ffn, true));
  FFN_TRY(map_weights(&p.a2, w3, f, f.hidden, f.ffn, true));
  FFN_TRY(map_rows(&p.b, x, f, f.hidden, ldx));
  p.out[0] = bf(hid), p.out[1] = bf(hid_rest), p.out[2] = bf(gate), p.out[3] = bf(up);
  return launch<UP>(p, f, kTraceFfnUp, s);
}

int ffn_few_down(const FfnShape &f, const void *hid, const void *hid_rest, const void *w2, void *y, int64_t ldy,
                 cudaStream_t s) {
  Args p = base_args(f, f.hidden, f.ffn);
  FFN_TRY(map_weights(&p.a, w2, f, f.ffn, f.hidden, true));
  FFN_TRY(map_rows(&p.b, hid, f, f.ffn, f.ffn));
  FFN_TRY(map_rows(&p.b2, hid_rest, f, f.ffn, f.ffn));
  p.out[0] = bf(y);
  p.ld = ldy;
  return launch<DOWN>(p, f, kTraceFfnDown, s);
}

int ffn_few_dh(const FfnShape &f, const void *dy, int64_t lddy, const void *w2, const void *gate, const void *up,
               void *dg, void *du, void *hid, cudaStream_t s) {
  Args p = base_args(f, f.ffn, f.hidden);
  FFN_TRY(map_weights(&p.a, w2, f, f.ffn, f.hidden, false));
  FFN_TRY(map_rows(&p.b, dy, f, f.hidden, lddy));
  p.out[0] = bf(dg), p.out[1] = bf(du), p.out[2] = bf(hid);
  p.g = static_cast<const __nv_bfloat16 *>(gate);
  p.u = static_cast<const __nv_bfloat16 *>(up);
  return launch<DH>(p, f, kTraceFfnDh, s);
}

int ffn_few_dx(const FfnShape &f, const void *dg, const void *du, const void *w1, const void *w3, void *dx,
               int64_t lddx, cudaStream_t s) {
  Args p = base_args(f, f.hidden, f.ffn);
  p.segments = 2;
  FFN_TRY(map_weights(&p.a, w1, f, f.hidden, f.ffn, false));
  FFN_TRY(map_weights(&p.a2, w3, f, f.hidden, f.ffn, false));
  FFN_TRY(map_rows(&p.b, dg, f, f.ffn, f.ffn));
  FFN_TRY(map_rows(&p.b2, du, f, f.ffn, f.ffn));
  p.out[0] = bf(dx);
  p.ld = lddx;
  return launch<DX>(p, f, kTraceFfnDx, s);
}

}  // namespace muon
