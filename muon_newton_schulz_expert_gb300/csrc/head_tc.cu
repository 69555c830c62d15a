// Tensor-core products of the loss over a head matrix W [V][H] and rows x [T][H]:
//   z = x W^T  (T x V), lse = log sum_v exp z_v, loss = lse - z_target
//   d_v = g p_v - hit [v = target],  dx = d W,  dW = d^T x
// z and d exist as tiles only: STATS reduces a tile of z to a reference and a sum per
// row in its epilogue; the backward pass recomputes z by pieces of the vocabulary,
// DLOGITS stores a piece of d in bf16 and GRADS forms both products that read it.
//
// One kernel, instantiated for the three; persistent CTA pairs on output tiles of
// 256 x up to 256 (tcgen05.mma.cta_group::2, M = 256, K = 16, bf16 operands, fp32
// accumulation in TMEM), fed by TMA through a ring of k-blocks of 64.  Loop bound: a k-block
// of MMAs is 512 cycles (128 and 256 with 64 and 128 columns), and takes 560 to 600 with its operands' way into
// shared memory.
//
// Rows of x are on M, the vocabulary on N: a thread of the epilogue then holds 32
// columns of one row at a time, so the softmax's sum needs no exchange between
// threads but at a tile's end, where one (c, s) per row is left.  Tiles
// walk the vocabulary with the row tiles of a group fastest, a group being as many row
// tiles as keep their x in L2 (kGroupBytes), so that W is read once per group.
// With few tiles N is 128 or 64, so that more pairs of CTAs load and reduce one.
//
// GRADS runs dx's and dW's tiles in one launch: dx has few tiles with long sums (K =
// the piece), dW many with short ones (K = rows), and the short ones fill what the long
// ones leave of the last wave (Schedule).  Where dx's tiles are so few that one is more
// than a pair's share of the work, its K is cut and the parts are added in order.
//
// Rounding: d is stored in bf16, the operand type of the products that read it, once
// (the feed-forward products round h, dg and du the same way); the rest is fp32.  Its two
// halves as two operands would leave dx and dW their own rounding alone, 0.0017 instead of 0.0024 from 64 bits over the
// batch, for four products in place of two: two thirds more of the whole call's.
//
// Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer (even CTA) and TMEM owner, the
// others (16, in GRADS 8) epilogue.  Two accumulators, so that the epilogue of one tile
// overlaps the next tile's products.  Every wait is bounded (tc.cuh).
#include <math.h>

#include <algorithm>

#include "head_loss.cuh"
#include "tiles.cuh"

namespace muon {
namespace {

constexpr int CM = 256, BM = 128;   // M of a pair tile, M held by one CTA
constexpr int BN = 256, BNH = 128;  // most N of a pair tile, N loaded by one CTA
constexpr int UMMA_K = 16;
constexpr int A_STAGE = BM * BK * 2;
constexpr int B_STAGE = BNH * BK * 2;
constexpr int KB_BYTES = A_STAGE + B_STAGE;
constexpr int ACC_COLS = BN;
constexpr int TMEM_COLS = 2 * ACC_COLS;
constexpr int MAX_STAGES = 16;      // of the ring, whose stages are as many as fit (Args)

enum Mode { STATS = 0, DLOGITS, GRADS };

// Shared memory of a mode: the ring of k-blocks (stages of KSUB, each given back by one commit: with one a k-block
// 4096 rows of 6144 over 128000 entries took 3290 us, not 3082), and what the epilogue's warps need.
constexpr int KSUB = 2, RING_BYTES = 6 * KB_BYTES;
template <int MODE>
struct Form {
  // the exponentials take 16 warps, 4 on each scheduler: a warp's work on a tile is a chain of latencies
  static constexpr int EPI_WARPS = MODE == GRADS ? 8 : 16;
  static constexpr int EPI_BYTES = MODE == STATS ? 2 * 4 * BM * (int)sizeof(float2) : MODE == GRADS ? EPI_WARPS * BOX_BYTES : 0;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int NUM_BARS = MAX_STAGES * KSUB + MAX_STAGES + 5;
  static constexpr int SMEM_BYTES = 1024 + RING_BYTES + EPI_BYTES + NUM_BARS * 8 + 16;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

constexpr int64_t kGroupBytes = 48 << 20;   // of x that is used again and again, beside W's stream through 129 MB of L2

// GRADS: dx's tiles (`longs` of them) and then dW's (`shorts`), dealt to the pairs one after the
// other.  Where dx's do not come out even, the pairs without the last one take `extra` of dW's
// meanwhile.
struct Schedule {
  int longs, shorts, extra;

  __host__ __device__ int before(int ncl) const { return longs % ncl ? extra * (ncl - longs % ncl) : 0; }
  // the i-th tile of pair c of ncl: < longs a dx tile, else longs + a dW tile; -1: none
  __device__ int tile(int i, int c, int ncl) const {
    const int full = longs / ncl, rem = longs % ncl;
    const int mine = full + (c < rem ? 1 : 0);
    if (i < mine) return i * ncl + c;
    i -= mine;
    int at;
    if (rem && c >= rem) {
      if (i < extra) at = i * (ncl - rem) + (c - rem);
      else at = before(ncl) + (i - extra) * ncl + c;
    } else {
      at = before(ncl) + i * ncl + c;
    }
    return at < shorts ? longs + at : -1;
  }
};

struct Args {
  CUtensorMap a, b;        // STATS, DLOGITS: x and W, K-major;  GRADS: dx's d (K-major) and W (MN-major)
  CUtensorMap a_last;      // a by boxes of the rows that the last CTA with any has
  CUtensorMap a2, b2;      // GRADS: dW's d and x, MN-major
  CUtensorMap out, out2;   // GRADS: dx or its sums, and dW
  int rows, vocab, v0;     // vocab: entries from v0 on
  int hidden;
  int kblocks, kblocks2;   // of K;  GRADS: of dx's K (the piece) and of dW's (the rows)
  int tiles_m, tiles_n;    // row tiles and vocabulary tiles (of bn);  GRADS: row tiles and tiles of H
  int bn, group;           // columns of a tile, row tiles of a group
  int step_n, step_r;      // STATS, DLOGITS: a step of the number of pairs, in vocabulary tiles and row tiles of a group
  int stages, a_bytes;     // of the ring; of A in a k-block (less than A_STAGE where there are few rows)
  int splits;              // GRADS: parts of dx's K
  Schedule schedule;
  bool wide;               // GRADS: W's 128 columns load in one piece
  int out_kind;            // GRADS: 0 dx in bf16, 1 sums written, 2 sums added to
  const int64_t *targets;  // STATS
  float2 *parts;
  float *target_logit;
  const HeadRow *row;      // DLOGITS
  __nv_bfloat16 *d;
  int width;
  unsigned *err;
  unsigned long long timeout_ns;
};

// A pair's tiles, one after the other: places on M and N in tiles, first k-block and their number.
template <int MODE>
struct Walk {
  int tm, tn, kb0 = 0, num_kb;
  int part = 0;       // GRADS, dx: of a cut sum
  bool dw = false;    // GRADS: a tile of dW (M = the piece's vocabulary entries, N = H)
  int i = 0, group = 0, r = -1, gm = 0;

  // the next tile of this pair, or false.  STATS, DLOGITS: tile tn * gm + r of the group's gm row tiles; moving on by
  // the number of pairs takes no division (with one in each step, and 64-bit places, a STATS epilogue took 4250
  // cycles whatever K was).
  __device__ __forceinline__ bool next(const Args &p) {
    const int c = (int)(blockIdx.x >> 1), ncl = (int)(gridDim.x >> 1);
    if (MODE == GRADS) {
      int t = p.schedule.tile(i++, c, ncl);
      if (t < 0) return false;
      dw = t >= p.schedule.longs;
      kb0 = 0;
      if (dw) {
        t -= p.schedule.longs;
        tm = t / p.tiles_n;
        tn = t - tm * p.tiles_n;
        num_kb = p.kblocks2;
      } else {
        const int per = p.tiles_m * p.tiles_n;
        part = t / per;
        t -= part * per;
        tm = t / p.tiles_n;
        tn = t - tm * p.tiles_n;
        kb0 = (int)((long long)p.kblocks * part / p.splits);
        num_kb = (int)((long long)p.kblocks * (part + 1) / p.splits) - kb0;
      }
      return true;
    }
    int step = ncl;
    if (r < 0) {
      gm = min(p.group, p.tiles_m), tn = 0, r = 0, step = c, num_kb = p.kblocks;
    }
    if (gm == p.group) {   // as the host divided it
      tn += step == ncl ? p.step_n : step / gm;
      r += step == ncl ? p.step_r : step % gm;
    } else {
      tn += step / gm, r += step % gm;
    }
    if (r >= gm) r -= gm, ++tn;
    while (tn >= p.tiles_n) {
      // the rest of the step is in the next group
      const int over = (tn - p.tiles_n) * gm + r;
      group += p.group;
      if (group >= p.tiles_m) return false;
      gm = min(p.group, p.tiles_m - group);
      tn = over / gm;
      r = over - tn * gm;
    }
    tm = group + r;
    return true;
  }
};

// Rows of an operand K-major on M (x, or dx's d) that a CTA loads from its first one on: there is nothing to load
// behind the last row, and rows that are not loaded leave the others' results as they are.  (With whole boxes, of
// zeros behind the end, one row of 6144 over 128000 entries took 418 us, 128 rows 274.)
__device__ __forceinline__ int rows_from(int rows, int first) { return max(0, min(rows - first, BM)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 bytes, a whole sector, at once
__device__ __forceinline__ void store_sector(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Waits for the loads that are under way into v.
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // the registers are only valid from here on
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}

// Running softmax statistics of a row, Reference and sum as in head_loss.cuh: s = sum 2^(z log2(e) - c).  c is a whole
// number, so that z log2(e) - c is one fused operation whose reference has no rounding.
struct Stats {
  float c = -INFINITY, s = 0.f;

  // 32 columns with c as it is: right while no term passes 2^100, so that c need not be the largest logit's, any of
  // the row's will do, and no maximum is looked for.
  __device__ __forceinline__ float terms(const uint32_t (&v)[32]) const {
    const f32x2 scale = pair(kLog2e, kLog2e), ref = pair(-c, -c);
    f32x2 a[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 p = split(fma2(pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), scale, ref));
      const f32x2 e = pair(ex2(p.x), ex2(p.y));
      a[i & 3] = i < 4 ? e : add2(a[i & 3], e);
    }
    const float2 r = split(add2(add2(a[0], a[1]), add2(a[2], a[3])));
    return r.x + r.y;
  }
  // `in`: of a row that there is; the others hold anything
  __device__ __forceinline__ void add(const uint32_t (&v)[32], bool in) {
    if (c == -INFINITY) c = ceilf(__uint_as_float(v[0]) * kLog2e);
    const float more = terms(v);
    if ((more < 0x1p100f && fabsf(c) < kWholeReference) || !in) {
      s += more;
    } else {
      uint32_t copy[32];   // its address is taken, and registers have none
#pragma unroll
      for (int i = 0; i < 32; ++i) copy[i] = v[i];
      *this = add_any(*this, copy);
    }
  }
  // s between 1 and 2, where c can be moved by its exponent exactly; else its terms had the largest logit as reference
  __device__ __forceinline__ void normalise() {
    if (!(s > 0.f && s < INFINITY) || fabsf(c) >= kWholeReference) return;
    const uint32_t b = __float_as_uint(s);
    c += (float)((int)(b >> 23) - 127);
    s = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
  }

  // any values
  static __device__ __noinline__ Stats add_any(Stats a, const uint32_t (&v)[32]) {
    float most = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
#pragma unroll
    for (int i = 3; i + 1 < 32; i += 2) most = max3(most, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    most = fmaxf(most, __uint_as_float(v[31]));
    if (a.s == 0.f) a.c = -INFINITY;   // a guess that no term has met
    if (fabsf(most * kLog2e) < kFarReference) {
      const float up = ceilf(most * kLog2e);
      if (up > a.c) {
        a.s *= ex2(a.c - up);   // c = -inf: s is 0, and so is the factor
        a.c = up;
      }
      a.s += a.terms(v);   // a NaN is one of the sum
    } else {
      // Logits so large are 64 apart or equal: those of the largest count one, the others nothing.
      const float ref = far_reference(most);
      if (ref > a.c) {
        a.s *= ex2(a.c - ref);
        a.c = ref;
      }
      // +inf makes the sum NaN; a whole chunk of -inf adds nothing
      const float one = ref != a.c || ref == -INFINITY ? 0.f : ref < INFINITY ? 1.f : NAN;
#pragma unroll 4
      for (int i = 0; i < 32; ++i) {
        const float z = __uint_as_float(v[i]);
        a.s += z != z ? z : z == most ? one : 0.f;
      }
    }
    return a;
  }
};

__device__ __forceinline__ void tma_add_3d(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2,
                                           unsigned *err) {
  if (!dcheck((c0 & 15) == 0 && c0 >= 0 && c1 >= 0 && c2 >= 0, err)) return;
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// 32 rows x 32 columns of fp32 out of a warp (lane = row), written or added
__device__ __forceinline__ void put_sums(const Writer &out, const uint32_t (&v)[32], const CUtensorMap *map, bool add,
                                         int lane, int col0, int row0, int part, unsigned *err) {
  if (lane == 0) bulk_wait_read_all();  // the box's last store has read it
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4 *>(out.box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add) tma_add_3d(map, out.box_s, col0, row0, part, err);
    else tma_store_3d(map, out.box_s, col0, row0, part, err);
    bulk_commit();
  }
}

template <int MODE>
__global__ void __launch_bounds__(Form<MODE>::THREADS, 1) head_gemm_kernel(const __grid_constant__ Args p) {
  constexpr int EPI_WARPS = Form<MODE>::EPI_WARPS, NFULL = MAX_STAGES * KSUB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + RING_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + Form<MODE>::EPI_BYTES);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Form<MODE>::NUM_BARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // 0: issues the MMAs; 1: its peer
  auto full = [&](int s, int j) { return bar0 + 8u * (uint32_t)(s * KSUB + j); };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(NFULL + s); };
  auto accf = [&](int a) { return bar0 + 8u * (uint32_t)(NFULL + MAX_STAGES + a); };
  auto acce = [&](int a) { return bar0 + 8u * (uint32_t)(NFULL + MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(NFULL + MAX_STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NFULL; ++s) mbar_init(bar0 + 8u * s, 1);   // used in CTA 0: expect_tx for both halves
    for (int s = 0; s < MAX_STAGES; ++s) mbar_init(empty(s), 1);       // multicast commit
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf(a), 1);               // multicast commit
      mbar_init(acce(a), 2 * EPI_WARPS);   // used in CTA 0: every epilogue warp of the pair
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    if (MODE != GRADS || p.schedule.longs) {
      tma_prefetch_desc(&p.a);
      tma_prefetch_desc(&p.b);
    }
    if (MODE == GRADS && p.schedule.shorts) {
      tma_prefetch_desc(&p.a2);
      tma_prefetch_desc(&p.b2);
    }
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
  const uint32_t a_bytes = MODE == GRADS ? A_STAGE : (uint32_t)p.a_bytes;
  const uint32_t kb_smem = MODE == GRADS ? KB_BYTES : a_bytes + (uint32_t)p.bn * (BK * 2) / 2;
  wait_for_previous_grid();
  let_next_grid_start();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;  // stages ever filled, and the parity of their last fill
      bool ok = true;
      for (Walk<MODE> cur; ok && cur.next(p);) {
        const int bnh = MODE == GRADS ? BNH : p.bn / 2;
        const int m_a = cur.tm * CM + (int)rank * BM;                  // first of this CTA's places on M and N
        const int n_b = cur.tn * (2 * bnh) + (int)rank * bnh;
        const bool by_rows = MODE != GRADS || !cur.dw;
        const int mine = by_rows ? rows_from(p.rows, m_a) : BM;
        const CUtensorMap *map_a = mine == BM ? &p.a : &p.a_last;
        // of both CTAs
        const int both = by_rows ? rows_from(p.rows, cur.tm * CM) + rows_from(p.rows, cur.tm * CM + BM) : CM;
        const uint32_t kb_bytes = (uint32_t)((both + 2 * bnh) * (BK * 2));
        for (int kb = 0; kb < cur.num_kb; kb += KSUB) {
          if (!wait_polled(empty(stage), phase ^ 1u, w)) {
            ok = false;
            break;
          }
          const int valid = cur.num_kb - kb < KSUB ? cur.num_kb - kb : KSUB;
          // CTA 0's barrier counts the bytes of both CTAs; a k-block past the
          // end of K still completes its phase, with no bytes
          if (rank == 0)
#pragma unroll
            for (int j = 0; j < KSUB; ++j) mbar_expect_tx(full(stage, j), j < valid ? kb_bytes : 0);
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
#pragma unroll
          for (int j = 0; j < KSUB; ++j) {
            if (j >= valid) break;
            const int k = (cur.kb0 + kb + j) * BK;
            const uint32_t sa = sbase + (uint32_t)(stage * KSUB + j) * kb_smem, sb = sa + a_bytes;
            const uint32_t bar = map_to_rank(full(stage, j), 0);
            if (MODE != GRADS) {
              if (mine) tma_load_3d_pair(sa, map_a, bar, k, m_a, 0, p.err);
              tma_load_3d_pair(sb, &p.b, bar, k, p.v0 + n_b, 0, p.err);
            } else if (!cur.dw) {
              if (mine) tma_load_3d_pair(sa, map_a, bar, k, m_a, 0, p.err);
              load_columns(sb, &p.b, bar, n_b, p.v0 + k, 0, p.wide, p.err);
            } else {
              load_columns(sa, &p.a2, bar, m_a, k, 0, true, p.err);
              load_columns(sb, &p.b2, bar, n_b, k, 0, true, p.err);
            }
          }
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // After an abort, stages may still be filling: let those copies land.
      if (*abort_flag && rank == 0)
        for (int s2 = 0; s2 < p.stages; ++s2)
          if (issued & (1u << s2))
            for (int j = 0; j < KSUB; ++j) drain_wait(full(s2, j), (issued_parity >> s2) & 1u, drain_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (CTA 0 of the pair)
    if (rank == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (Walk<MODE> cur; ok && cur.next(p);) {
        // one thread that polls: with 6 and 8 k-blocks a tile 136 and 166 us, 144 and 173 suspended (8192 rows over
        // 32768 entries); the epilogue's 512 threads are suspended, since their polling slows long sums by 5 to 15%
        ok = wait_polled(acce(acc), acc_phase ^ 1u, w);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * ACC_COLS);
        const bool a_mn = MODE == GRADS && cur.dw;
        constexpr bool b_mn = MODE == GRADS;
        const uint32_t idesc = make_idesc(CM, MODE == GRADS ? BN : p.bn, a_mn, b_mn);
        for (int kb = 0; kb < cur.num_kb; kb += KSUB) {
          const int valid = cur.num_kb - kb < KSUB ? cur.num_kb - kb : KSUB;
#pragma unroll
          for (int j = 0; j < KSUB; ++j) {
            if (j >= valid) break;
            if (!wait_polled(full(stage, j), phase, w)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = sbase + (uint32_t)(stage * KSUB + j) * kb_smem, sb = sa + a_bytes;
            // K-major: advance 16 K-elements (32 bytes) inside the swizzle row.
            // MN-major: advance 16 K-rows (two 8-row groups of 1024 bytes);
            // 8192 bytes between 64-wide atoms, 1024 between 8-row groups.
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk) {
              const uint64_t ad = a_mn ? smem_desc(sa + kk * (UMMA_K * 128), 64 * BK * 2, 1024)
                                       : smem_desc(sa + kk * (UMMA_K * 2), 16, 1024);
              const uint64_t bd = b_mn ? smem_desc(sb + kk * (UMMA_K * 128), 64 * BK * 2, 1024)
                                       : smem_desc(sb + kk * (UMMA_K * 2), 16, 1024);
              tc_mma(d, ad, bd, idesc, ((kb + j) | kk) != 0 ? 1u : 0u);
            }
          }
          if (!ok) break;
          tc_commit_mc(empty(stage), 0x3);  // both CTAs may refill this stage
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit_mc(accf(acc), 0x3);  // both CTAs' accumulators are ready
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit_mc(drain_bar, 0x1);  // flips once all MMAs issued by this thread have completed
      volatile int no_abort = 0;
      wait_bounded(drain_bar, 0, Watch{&no_abort, p.err, p.timeout_ns});
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - 2;
    // TMEM lanes 32q.., and which of the tile's column ranges: halves in GRADS, else quarters (32 columns at least)
    const int q = warp & 3, range = ew >> 2;
    const int each = MODE == GRADS ? BNH : max(p.bn / 4, 32);
    uint8_t *box = epi_smem + (MODE == GRADS ? ew * BOX_BYTES : 0);
    Writer out{box, smem_u32(box)};
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (Walk<MODE> cur; cur.next(p);) {
      const int row0 = cur.tm * CM + (int)rank * BM + q * 32, row = row0 + lane;
      HeadRow hr{0.f, 0.f, 0.f, -1};
      int target = -1;   // counted from v0
      if (MODE == DLOGITS && row < p.rows) {
        hr = p.row[row];
        target = hr.target < 0 ? -1 : hr.target - p.v0;
      }
      if (MODE == STATS && row < p.rows) {
        const int64_t v = __ldg(p.targets + row);
        target = v >= 0 && v < p.vocab ? (int)v : -1;
      }
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(accf(acc), acc_phase, w));   // warp-uniform
      if (!ok && MODE != STATS) break;   // in STATS a warp that gave up still meets the others of its quarter
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * ACC_COLS);
      // This warp's columns, 32 at a time, the next 32 on their way while these are worked on.  The
      // accumulator is free again when the last are in registers.
      const int chunks = each / 32, first = range * each;
      bool busy = row0 < p.rows && (MODE == GRADS || first < p.bn);
      int row_at = row0;
      bool sums = false;
      if (MODE == GRADS) {
        if (cur.dw) row_at += p.v0;
        // a part without k-blocks (of a last piece that is short) has nothing to add
        busy = (cur.dw ? row0 < p.vocab : busy) && cur.num_kb > 0;
        sums = !cur.dw && p.out_kind != 0;
      }
      const CUtensorMap *map = MODE == GRADS && cur.dw ? &p.out2 : &p.out;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(acce(acc), 0));
      };
      if (!ok) busy = false;
      else if (!busy) release();
      Stats stats;
      uint32_t v[2][32], wo[32];
      if (busy) {
        // a target among this warp's columns?  Rarely, and then once.
        const int col_first = cur.tn * (MODE == GRADS ? BN : p.bn) + first;   // of z's piece, or of hidden
        const int hit0 = MODE != GRADS && (unsigned)(target - col_first) < (unsigned)each ? target - col_first : -1;
        const bool any_hit = MODE != GRADS && __any_sync(0xffffffffu, hit0 >= 0);
        tmem_ld32_issue(taddr + (uint32_t)first, v[0]);
#pragma unroll
        for (int ch = 0; ch < (MODE == GRADS ? BNH / 32 : 2); ++ch) {
          if (ch >= chunks) break;
          uint32_t (&z)[32] = v[ch & 1];
          tmem_wait(z);
          if (ch + 1 < chunks) tmem_ld32_issue(taddr + (uint32_t)(first + 32 * (ch + 1)), v[(ch + 1) & 1]);
          else release();
          const int col0 = col_first + 32 * ch;
          if (MODE == STATS) {
            const int left = p.vocab - col0;
            if (left <= 0) continue;
            if (left < 32)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left) z[i] = __float_as_uint(-INFINITY);
            if (any_hit)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (hit0 == 32 * ch + i && i < left) p.target_logit[row] = __uint_as_float(z[i]);
            stats.add(z, row < p.rows);
          } else if (MODE == DLOGITS) {
            // rows that take no part have g = 0 and finite z (x's copy holds zeros there).  The difference first: next
            // to a certain target it is exact, and p has no rounding but lse's own.
            float d[32];
            const f32x2 scale = pair(kLog2e, kLog2e), minus = pair(-hr.lse, -hr.lse);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const f32x2 below = add2(pair(__uint_as_float(z[i]), __uint_as_float(z[i + 1])), minus);
              const float2 e = split(mul2(below, scale));
              d[i] = hr.g * ex2(e.x);
              d[i + 1] = hr.g * ex2(e.y);
            }
            if (any_hit)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (hit0 == 32 * ch + i) d[i] -= hr.hit;
            const int left = p.vocab - col0;
            if (left < 32)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left) d[i] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) wo[i] = pack_bf16(d[2 * i], d[2 * i + 1]);
            if (row < p.rows) {
              __nv_bfloat16 *dst = p.d + (long long)row * p.width + col0;
              store_sector(dst, wo);
              store_sector(dst + 16, wo + 8);
            }
          } else if (sums) {
            if (col0 < p.hidden) put_sums(out, z, map, p.out_kind == 2, lane, col0, row_at, cur.part, p.err);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              wo[(ch & 1) * 16 + i] = pack_bf16(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1]));
            if ((ch & 1) && col0 - 32 < p.hidden) out.put(wo, map, lane, col0 - 32, row_at, 0, p.err);
          }
        }
      }
      if (MODE == STATS) {
        // The four ranges of these rows' columns meet; the next tile writes the other half of the array.  Quarters
        // without rows meet too: the barrier of the tile between is what keeps a tile's reads before the writes to
        // the same half two tiles later, and a pair's tiles may have rows here, none, and rows again.
        const bool rows_here = row0 < p.rows;
        float2 *meet = reinterpret_cast<float2 *>(epi_smem) + acc * (4 * BM) + q * 32 + lane;
        if (rows_here) {
          stats.normalise();
          meet[range * BM] = make_float2(stats.c, stats.s);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
        if (rows_here && range == 0 && row < p.rows) {
          float c = stats.c, s = stats.s;
#pragma unroll
          for (int r = 1; r < 4; ++r) {
            const float2 o = meet[r * BM];
            const float up = fmaxf(c, o.x);
            s = s * (c == up ? 1.f : ex2(c - up)) + o.y * (o.x == up ? 1.f : ex2(o.x - up));
            c = up;
          }
          p.parts[(long long)cur.tn * p.rows + row] = make_float2(c, s);
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (MODE == GRADS && lane == 0) bulk_wait_all();
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

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 3-D map over [parts][rows][cols] of fp32, boxes of 32 x 32
int make_map_sums(CUtensorMap *map, const void *base, int64_t parts, int64_t rows, int64_t cols) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return MUON_ERR_CUDA;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)rows * cols * 4};
  cuuint32_t box[3] = {32u, 32u, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MUON_OK : MUON_ERR_CUDA;
}

template <int MODE>
int launch(Args &p, int64_t tiles, int trace_kind, cudaStream_t s) {
  static std::once_flag attr_once[64];
  static int max_pairs[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  auto *kernel = head_gemm_kernel<MODE>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Form<MODE>::THREADS, 1, 1);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // the occupancy query knows clusters only
  cfg.dynamicSmemBytes = Form<MODE>::SMEM_BYTES;
  std::call_once(attr_once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Form<MODE>::SMEM_BYTES);
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
  // Few rows leave room for more k-blocks on their way (5 rows of 2048 over 120000 entries 86 us, 93 with three stages
  // of whole ones).  The MMAs read 128 rows of A all the same, of what lies behind, inside the ring.
  p.a_bytes = MODE == GRADS ? A_STAGE : (int)((std::min<int64_t>(p.rows, BM) + 7) / 8 * 8 * BK * 2);
  const int kb_smem = p.a_bytes + (MODE == GRADS ? B_STAGE : p.bn * BK);
  p.stages = std::min(MAX_STAGES, (RING_BYTES - (A_STAGE - p.a_bytes)) / (kb_smem * KSUB));
  const int64_t pairs = std::min<int64_t>(tiles, max_pairs[dev]);
  if (MODE != GRADS) p.step_n = (int)pairs / p.group, p.step_r = (int)pairs % p.group;
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.numAttrs = 2;
  cfg.stream = s;
  if (MODE == GRADS && p.schedule.longs % pairs) {
    // dW tiles that take as long as one of dx; an epilogue costs about as much as 4 k-blocks
    const int64_t rest = pairs - p.schedule.longs % pairs, each = p.kblocks / p.splits / (p.kblocks2 + 4);
    p.schedule.extra = (int)std::min<int64_t>(each, p.schedule.shorts / rest);
  }
  trace_before(trace_kind, s);
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, p);
  const int st = trace_after(trace_kind, s);
  return le == cudaSuccess ? st : MUON_ERR_CUDA;
}

#define HEAD_TRY(expr)              \
  do {                              \
    const int _st = (expr);         \
    if (_st != MUON_OK) return _st; \
  } while (0)

// a's maps: whole boxes, and boxes of the rows that the last CTA has
int map_rows(Args &p, const void *base, int64_t rows, int64_t cols, int64_t ld) {
  HEAD_TRY(make_map(&p.a, base, 1, rows, cols, BM, ld));
  return make_map(&p.a_last, base, 1, rows, cols, (int)((rows - 1) % BM + 1), ld);
}

int pairs_of_sms() { return std::max(1, num_sms() / 2); }

// Columns of a tile of z: fewer than 256 only where the tiles still come out as one for each pair of CTAs.  The tensor
// pipe is busy for 128, 256 and 512 cycles a k-block with 64, 128 and 256 columns, but the loop takes about 485 with the
// fewest too: A's 16 KB for each CTA come in whatever N is.  So narrow tiles spread the loads of W and the epilogue and save no
// time on the products: 513 rows of 4320 over 3802 entries, gradient: 62 us with 45 tiles of 256, 79 us with 90 of 128.
int columns(const HeadShape &h, int64_t vocab, int least) {
  int bn = BN;
  while (bn > least && cdiv(h.rows, CM) * cdiv(vocab, bn / 2) <= pairs_of_sms()) bn /= 2;
  return bn;
}

int group_of(const HeadShape &h) { return (int)std::clamp<int64_t>(kGroupBytes / (CM * h.hidden * 2), 4, 1 << 20); }

}  // namespace

int head_stats_columns(const HeadShape &h) { return columns(h, h.vocab, 64); }
int64_t head_parts(const HeadShape &h) { return cdiv(h.vocab, head_stats_columns(h)); }

int head_stats(const HeadShape &h, const void *x, int64_t ldx, const void *w, const int64_t *targets, float2 *parts,
               float *target_logit, cudaStream_t s) {
  Args p{};
  p.bn = head_stats_columns(h);
  HEAD_TRY(map_rows(p, x, h.rows, h.hidden, ldx));
  HEAD_TRY(make_map(&p.b, w, 1, h.vocab, h.hidden, p.bn / 2));
  p.rows = (int)h.rows;
  p.vocab = (int)h.vocab;
  p.hidden = (int)h.hidden;
  p.kblocks = (int)cdiv(h.hidden, BK);
  p.tiles_m = (int)cdiv(h.rows, CM);
  p.tiles_n = (int)cdiv(h.vocab, p.bn);
  p.group = std::min(group_of(h), p.tiles_m);
  p.targets = targets;
  p.parts = parts;
  p.target_logit = target_logit;
  return launch<STATS>(p, (int64_t)p.tiles_m * p.tiles_n, kTraceHeadStats, s);
}

// A piece is at most as wide as makes d 256 MB (16384 columns of many rows: few additions to dx's sums, few last
// waves), and of those widths from three quarters of that on the one that leaves the least of the last wave empty.
// With 64, 128, 256 and 512 MB: 4096 rows of 6144 over 64000 entries 5.39, 5.24, 5.18, 5.10 ms; 16384 of 2048 over
// 40003 4.57, 4.55, 4.58, 4.31 ms; 4096 of 512 over 50003 562, 502, 465, 438 us.
HeadPlan head_plan(const HeadShape &h, bool need_dx, bool need_dw) {
  const int64_t all = cdiv(h.vocab, CM), tm = cdiv(h.rows, CM), pairs = pairs_of_sms();
  const int64_t most = std::min(all, std::max<int64_t>(64, (int64_t(256) << 20) / (h.rows * CM * 2)));
  HeadPlan plan{most, 1, 1};
  if (most < all) {
    double best = 0;
    for (int64_t n = most; n >= std::max<int64_t>(1, most * 3 / 4); --n) {
      const double used = (double)(tm * n) / (double)(cdiv(tm * n, pairs) * pairs);
      if (used > best + 1e-9) best = used, plan.piece_tiles = n;
    }
    plan.pieces = cdiv(all, plan.piece_tiles);
  }
  if (need_dx) {
    // a dx tile no longer than half a pair's share of the whole (4 rows of 6144 over 64000 entries 439 us, 508 with
    // tiles of a whole share; 4096 of 512 over 50003 432 and 465)
    const int64_t th = cdiv(h.hidden, BN), kb = plan.piece_tiles * (CM / BK);
    const int64_t work = tm * th * kb + (need_dw ? plan.piece_tiles * th * (cdiv(h.rows, BK) + 4) : 0);
    plan.splits = (int)std::clamp<int64_t>(2 * kb * pairs / std::max<int64_t>(work, 1), 1,
                                         std::min<int64_t>(16, std::max<int64_t>(1, kb / 8)));
  }
  return plan;
}

int head_dlogits(const HeadShape &h, const HeadPlan &plan, int64_t v0, const void *xc, int64_t xc_cols, const void *w,
                 const HeadRow *row, void *d, cudaStream_t s) {
  Args p{};
  p.bn = columns(h, plan.width(), 128);
  HEAD_TRY(map_rows(p, xc, h.rows, h.hidden, xc_cols));
  HEAD_TRY(make_map(&p.b, w, 1, h.vocab, h.hidden, p.bn / 2));
  p.d = static_cast<__nv_bfloat16 *>(d);
  p.width = (int)plan.width();
  p.rows = (int)h.rows;
  p.vocab = (int)(h.vocab - v0);
  p.hidden = (int)h.hidden;
  p.v0 = (int)v0;
  p.kblocks = (int)cdiv(h.hidden, BK);
  p.tiles_m = (int)cdiv(h.rows, CM);
  // the last piece ends with the vocabulary's last 256 columns
  p.tiles_n = (int)(std::min(plan.piece_tiles, cdiv(h.vocab - v0, CM)) * (CM / p.bn));
  p.group = std::min(group_of(h), p.tiles_m);
  p.row = row;
  return launch<DLOGITS>(p, (int64_t)p.tiles_m * p.tiles_n, kTraceHeadDlogits, s);
}

int head_grads(const HeadShape &h, const HeadPlan &plan, int64_t v0, bool first, const void *d, const void *w,
               const void *xc, int64_t xc_cols, void *dx, int64_t lddx, float *acc, void *dweight, cudaStream_t s) {
  Args p{};
  const int64_t tiles_v = std::min(plan.piece_tiles, cdiv(h.vocab - v0, CM));
  p.wide = h.hidden % 64 == 0;
  p.rows = (int)h.rows;
  p.vocab = (int)(h.vocab - v0);
  p.hidden = (int)h.hidden;
  p.v0 = (int)v0;
  p.tiles_m = (int)cdiv(h.rows, CM);
  p.tiles_n = (int)cdiv(h.hidden, BN);
  p.kblocks = (int)(tiles_v * (CM / BK));
  p.kblocks2 = (int)cdiv(h.rows, BK);
  p.splits = plan.splits;
  if (dx) {
    HEAD_TRY(map_rows(p, d, h.rows, plan.width(), plan.width()));
    HEAD_TRY(p.wide ? make_map_blocks(&p.b, w, 1, h.vocab, h.hidden, BK, 2) : make_map(&p.b, w, 1, h.vocab, h.hidden, BK));
    p.out_kind = plan.pieces == 1 && plan.splits == 1 ? 0 : first ? 1 : 2;
    HEAD_TRY(p.out_kind == 0 ? make_map(&p.out, dx, 1, h.rows, h.hidden, 32, lddx)
                             : make_map_sums(&p.out, acc, plan.splits, h.rows, h.hidden));
    p.schedule.longs = p.tiles_m * p.tiles_n * p.splits;
  }
  if (dweight) {
    HEAD_TRY(make_map_blocks(&p.a2, d, 1, h.rows, plan.width(), BK, 2));
    HEAD_TRY(make_map_blocks(&p.b2, xc, 1, h.rows, xc_cols, BK, 2));
    HEAD_TRY(make_map(&p.out2, dweight, 1, h.vocab, h.hidden, 32));
    p.schedule.shorts = (int)tiles_v * p.tiles_n;
  }
  return launch<GRADS>(p, (int64_t)p.schedule.longs + p.schedule.shorts, kTraceHeadGrads, s);
}

}  // namespace muon
