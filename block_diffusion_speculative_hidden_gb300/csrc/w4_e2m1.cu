// dflash_gemm_w4 of E2M1 codes with up to 16 activation rows.
#include "w4_resident.cuh"

namespace dflash {

cudaError_t launch_w4_e2m1(const W4Args& a, cudaStream_t s) {
  return a.x_elem == DFLASH_ELEM_BF16 ? launch_w4_x<__nv_bfloat16, true>(a, s) : launch_w4_x<__half, true>(a, s);
}

}  // namespace dflash
