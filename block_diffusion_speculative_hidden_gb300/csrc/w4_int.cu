// dflash_gemm_w4 of integer codes with up to 16 activation rows.
#include "w4_resident.cuh"

namespace dflash {

cudaError_t launch_w4_int(const W4Args& a, cudaStream_t s) {
  return a.x_elem == DFLASH_ELEM_BF16 ? launch_w4_x<__nv_bfloat16, false>(a, s) : launch_w4_x<__half, false>(a, s);
}

}  // namespace dflash
