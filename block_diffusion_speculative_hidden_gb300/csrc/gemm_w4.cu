// dflash_gemm_w4: products of a few activation rows with 4-bit weights under
// group scales,
//     out[m][n] = sum_k X[m][k] scale[n][k/g] (code[n][k] - zero[n][k/g]).
//
// The differences code - zero (and the E2M1 values) are exact in bf16 (there in
// 64ths) and fp16, so a block of 32 k enters the matrix instruction as it is,
// with fp32 sums, and the scale multiplies the block's fp32 sum.  The order of
// k inside a block is free as long as weights and activations agree on it:
// thread t of a quad holds codes 8t .. 8t+7 of the block (one 32-bit word),
// whose halves come out of the word as pairs (k, k+4).
#include "w4_common.cuh"

using namespace dflash;

extern "C" dflash_status dflash_gemm_w4(const void* W, int format, const void* scale, int scale_elem, const void* zero,
                                        int N, int K, int group, const void* X, int x_elem, int M, float* out,
                                        int* status, dflash_stream stream) {
  if (W == nullptr || scale == nullptr || X == nullptr || out == nullptr || N < 1 || K < 1 || M < 1)
    return DFLASH_ERR_INVALID_ARG;
  if (format != DFLASH_W4_INT && (format != DFLASH_W4_E2M1 || zero != nullptr)) return DFLASH_ERR_INVALID_ARG;
  if (x_elem != DFLASH_ELEM_BF16 && x_elem != DFLASH_ELEM_F16) return DFLASH_ERR_INVALID_ARG;
  const int ss = scale_elem == DFLASH_ELEM_F32 ? 4 : 2;
  if (scale_elem != DFLASH_ELEM_F32 && scale_elem != DFLASH_ELEM_BF16 && scale_elem != DFLASH_ELEM_F16)
    return DFLASH_ERR_INVALID_ARG;
  if (M > 32 || K % 32 || (group != 32 && group != 64 && group != 128)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // (row and unit counts, and the bytes of all activations, stay within 32 bits)
  if (N > 1 << 30 || static_cast<long long>(M) * K > 1 << 29) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (reinterpret_cast<uintptr_t>(W) % 16 || reinterpret_cast<uintptr_t>(X) % 16 ||
      reinterpret_cast<uintptr_t>(scale) % ss || reinterpret_cast<uintptr_t>(out) % 4)
    return DFLASH_ERR_INVALID_ARG;
  W4Args a{};
  a.W = W;
  a.scale = static_cast<const uint8_t*>(scale);
  a.zero = static_cast<const uint8_t*>(zero);
  a.x = X;
  a.out = out;
  a.status = status;
  a.N = N;
  a.K = K;
  a.groups = (K + group - 1) / group;
  a.M = M;
  a.group = group;
  a.scale_elem = scale_elem;
  a.scale_size = ss;
  a.x_elem = x_elem;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&a.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = M > kW4ResidentM           ? launch_w4_stream(a, format == DFLASH_W4_E2M1, stream)
        : format == DFLASH_W4_E2M1 ? launch_w4_e2m1(a, stream)
                                   : launch_w4_int(a, stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
