// What the kernels on 256 x 256 tiles of CTA pairs share: operand boxes, the way
// of a tile's rows out of TMEM and through shared memory.
#pragma once

#include "tc.cuh"

namespace muon {
namespace {

constexpr int BK = 64;              // one 128-byte swizzle row of bf16
constexpr int BOX_BYTES = 32 * 64 * 2;    // output staging box of an epilogue warp: 32 rows x 128 bytes

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t *>(&h);
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

}  // namespace
}  // namespace muon
