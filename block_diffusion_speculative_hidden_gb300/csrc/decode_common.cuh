// What the kernels of the caller's decode steps (append.cu, prefix_*.cu,
// w4_*.cu) share beyond common.cuh, whose text the captures of the GEMMs'
// traffic are taken on.
#pragma once

#include "common.cuh"

namespace dflash {

// Status bits, continued.
enum : int {
  ST_BAD_PAGE = 64,        // a page-table entry outside the pool
  ST_BAD_POS = 128,        // a position outside the rotation table
};

// One thread of a converged warp, the same one every time.  Copies and MMAs
// take their operands from uniform registers: where the whole warp computes
// them alike and one thread is elected to issue, they are there already.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(is));
  return is != 0;
}

// tma_load_2d to a shared-memory address.
__device__ __forceinline__ void tma_load_2d_to(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace dflash
