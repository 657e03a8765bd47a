// What the kernels of the caller's decode steps (append.cu, prefix_*.cu,
// w4_*.cu, fp4_*.cu, verify.cu, pages.cu) share beyond common.cuh, whose text the captures of the GEMMs'
// traffic are taken on.
#pragma once

#include "common.cuh"

namespace dflash {

// Status bits, continued.
enum : int {
  ST_BAD_PAGE = 64,        // a page-table entry outside the pool
  ST_BAD_POS = 128,        // a position outside the rotation table
  ST_BAD_PROB = 256,       // a probability or a random number that cannot be one
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

// The bytes of a caller's array, null for none; whether two of them share none.
struct Span {
  const void* at;
  long long bytes;
};
inline Span ints(const int32_t* a, long long n) { return {a, 4 * n}; }
inline bool apart(const Span& a, const Span& b) {
  const auto lo = [](const Span& s) { return reinterpret_cast<uintptr_t>(s.at); };
  return a.at == nullptr || b.at == nullptr || lo(a) + a.bytes <= lo(b) || lo(b) + b.bytes <= lo(a);
}

// A kernel that may start before its predecessor completes (it waits first), in clusters of `cluster` blocks; as launch_k, but
// the driver picks the L1 cache's share: with all of it given to shared memory, streams through L1 are slower (quantising
// 8192 rows of 12,288 42.8 us against 53.6, taking back 38.7 against 47.9).
template <typename Params>
cudaError_t launch_cached(void (*k)(const Params), unsigned blocks, unsigned threads, size_t smem, cudaStream_t s,
                          unsigned cluster, const Params& p) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(blocks);
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = at;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, k, p);
}

}  // namespace dflash
