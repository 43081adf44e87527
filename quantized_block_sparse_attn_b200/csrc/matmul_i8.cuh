// Product of INT8 codes with a scale for each row of either side:
//   out[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] + bias[n].
// The sum is exact in s32 (K < 2^17 keeps |sum| <= 2^14 K below 2^31); it is then rounded to
// f32 and scaled in f32, by a_scale first, with the second product and the bias in one fused
// multiply-add, and rounded once to the output's type.
#pragma once

#include <cstdint>

#include "norm_quant.cuh"

namespace qbsa {

constexpr int kMatmulMaxK = 131071;  // 2^14 K < 2^31

struct MatmulI8Params {
  const int8_t* a;
  const int8_t* b;
  const float* a_scale;
  const float* b_scale;
  const float* bias;  // or nullptr
  void* out;
  int64_t a_stride, b_stride, o_stride;
  int M, N, K;
};

__device__ __forceinline__ float scale_acc(int32_t acc, float sa, float sb, float bias) {
  return __fmaf_rn(__fmul_rn(__int2float_rn(acc), sa), sb, bias);
}

// 64 x 64 tile, 256 threads of 4 x 4 sums, 64 bytes of K per step, dp4a.
template <typename O>
__global__ void __launch_bounds__(256) matmul_i8_simple_kernel(const __grid_constant__ MatmulI8Params p) {
  __shared__ uint32_t ta[16][65], tb[16][65];
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int32_t acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += 64) {
    const int r = threadIdx.x >> 2, c = threadIdx.x & 3, k = k0 + c * 16;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int row = (side ? n0 : m0) + r, rows = side ? p.N : p.M;
      const int8_t* src = side ? p.b + row * p.b_stride + k : p.a + row * p.a_stride + k;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (row < rows && k < p.K) {
        if (k + 16 <= p.K) {
          const uint4 u = *reinterpret_cast<const uint4*>(src);
          w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
          for (int i = 0; i < p.K - k; ++i) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[i])) << (8 * (i & 3));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) (side ? tb : ta)[c * 4 + i][r] = w[i];
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __dp4a(static_cast<int>(ta[kk][ty * 4 + i]), static_cast<int>(tb[kk][tx + 16 * j]), acc[i][j]);
    __syncthreads();
  }
  O* out = static_cast<O*>(p.out);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m < p.M && n < p.N)
        out[m * p.o_stride + n] =
            from_f32<O>(scale_acc(acc[i][j], p.a_scale[m], p.b_scale[n], p.bias ? p.bias[n] : 0.f));
    }
}

}  // namespace qbsa
