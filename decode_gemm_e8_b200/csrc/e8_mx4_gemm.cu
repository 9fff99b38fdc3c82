// Product of two matrices in the microscaled 4-bit form.
//
// Y[m][n] = bf16(sum_k A[m][k] W[n][k]); a product of two e2m1 values and two
// powers of two is exact in fp32, the sums are fp32.
#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace e8 {
namespace mx4 {

// 64 x 64 outputs a CTA, 4 x 4 a thread, one block of 32 columns at a time.
__global__ void __launch_bounds__(256)
    k_mx4_gemm(const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, int64_t M,
               const uint8_t* __restrict__ W, const uint8_t* __restrict__ Ws, int64_t N, int64_t K,
               uint16_t* __restrict__ Y) {
  __shared__ float sa[32][65], sw[32][65];
  const int64_t cs = code_stride(K), kqs = scale_tiles(K);
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lq = threadIdx.x & 3;   // row, 8-value quarter of the block
  float acc[4][4] = {};
  for (int64_t b = 0; b < (K + 31) / 32; ++b) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int64_t row = (side ? n0 : m0) + lr, rows = side ? N : M;
      uint32_t code = 0, byte = 0;
      if (row < rows) {
        code = *reinterpret_cast<const uint32_t*>((side ? W : A) + row * cs + b * 16 + lq * 4);
        byte = (side ? Ws : As)[scale_at(row, b >> 2, kqs) + (b & 3)];
      }
      const float s = scale_value(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        (side ? sw : sa)[lq * 8 + i][lr] = code_value(code >> (4 * i)) * s;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      float a[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sa[k][ty * 4 + i];
        w[i] = sw[k][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], w[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) Y[m * N + n] = (uint16_t)(pack_bf16x2(acc[i][j], 0.0f) & 0xFFFFu);
    }
}

}  // namespace mx4

cudaError_t launch_mx4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                            const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int64_t K,
                            uint16_t* Y, void* ws, uint32_t* status, int sm_count,
                            cudaStream_t st) {
  (void)ws; (void)status; (void)sm_count;
  const int64_t gy = (M + 63) / 64;
  if (gy > 65535) return cudaErrorInvalidValue;
  mx4::k_mx4_gemm<<<dim3((unsigned)((N + 63) / 64), (unsigned)gy), 256, 0, st>>>(
      a_codes, a_scales, M, w_codes, w_scales, N, K, Y);
  return cudaGetLastError();
}

size_t mx4_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  (void)M; (void)N; (void)K;
  return 0;
}

}  // namespace e8
