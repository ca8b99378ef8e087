// Product of 8-bit integers with scales for each row of A (token) and of W
// (channel): C[m][n] = a_scale[m] w_scale[n] sum_k A[m][k] W[n][k].
//
// The sums are exact in int32 (at most 8192 products of 127^2 or less).  Each
// is converted to float32 (one rounding), multiplied by the row's scale and
// then by the channel's (one each), which keeps the result within 2^-22 of the
// real value; scales are not multiplied together first, so that a channel of
// large scale meets the sum before an underflow can.
#include "common.h"
#include "kernels.h"

namespace domino {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mma16_i8(i32x4 acc, u32x4 a, u32x4 w) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, w), acc, 0, 0, 0);
}

// One wave per 16 x 16 tile of C; 64 bytes of K a step (the second half of a
// last step of 32 is zero in both operands).
__global__ void __launch_bounds__(256)
    gemm_i8_tile_kernel(const int8_t* __restrict__ A, const float* __restrict__ as, int M, const int8_t* __restrict__ W,
                        const float* __restrict__ ws, int N, int K, float* __restrict__ C) {
  const int lane = threadIdx.x & 63, grp = lane >> 4, col = lane & 15;
  const int n0 = (blockIdx.x * 4 + wave_id()) * 16, m0 = blockIdx.y * 16;
  if (n0 >= N) return;
  const int8_t* ar = A + (size_t)min(m0 + col, M - 1) * K;
  const int8_t* wr = W + (size_t)min(n0 + col, N - 1) * K;
  i32x4 acc = {0, 0, 0, 0};
  for (int k0 = 0; k0 < K; k0 += 64) {
    const int k = k0 + grp * 16;
    u32x4 a = {0, 0, 0, 0}, w = {0, 0, 0, 0};
    if (k < K) {
      a = ld16(ar + k);
      w = ld16(wr + k);
    }
    acc = mma16_i8(acc, a, w);
  }
  const int n = n0 + col;
  if (n >= N) return;
  const float wsn = ws[n];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = m0 + grp * 4 + j;
    if (m < M) C[(size_t)m * N + n] = (float)acc[j] * as[m] * wsn;
  }
}

hipError_t launch_gemm_i8(const int8_t* A, const float* a_scale, int M, const int8_t* W, const float* w_scale, int N,
                          int K, float* C, int num_cu, hipStream_t s) {
  if (M <= 0 || N <= 0) return hipSuccess;
  if (K <= 0 || K % 32) return hipErrorNotSupported;
  (void)num_cu;
  hipLaunchKernelGGL(gemm_i8_tile_kernel, dim3((unsigned)((N + 63) / 64), (unsigned)((M + 15) / 16)), dim3(256), 0, s, A,
                     a_scale, M, W, w_scale, N, K, C);
  return hipGetLastError();
}

}  // namespace domino
