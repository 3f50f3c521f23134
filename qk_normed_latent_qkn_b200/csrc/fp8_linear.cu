// qkn_fp8_linear: out = A W^T for rows and a weight in 8 bits with a scale for each block of 128.
//
// out[i, n] = sum_b sa[b, i] sw[n / 128, b] sum_{k in b} a[i, k] w[n, k].  The products of two e4m3
// values are exact in fp32, a block's 128 of them are summed unscaled, and each block's sum enters
// the fp32 total with its two scales; one rounding at the end.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace qkn {
namespace {

constexpr int kTile = 64;

__device__ __forceinline__ float value_of(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

// A tile of 64 x 64 outputs per CTA, 4 x 4 per thread, on the CUDA cores.
template <typename O>
__global__ void __launch_bounds__(256) fp8_linear_simple_kernel(Fp8LinearArgs p) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sa[32][kTile + 1], sw[32][kTile + 1];
  const int i0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int groups = (p.k + kFp8Group - 1) / kFp8Group;
  float acc[4][4] = {};
  for (int b = 0; b < groups; ++b) {
    float t[4][4] = {};
    for (int k0 = b * kFp8Group; k0 < min(p.k, (b + 1) * kFp8Group); k0 += 32) {
      for (int e = threadIdx.x; e < kTile * 32; e += 256) {
        const int row = e / 32, k = e % 32;
        const bool in = k0 + k < p.k;
        sa[k][row] = in && i0 + row < p.m ? value_of(p.a[(int64_t)(i0 + row) * p.lda + k0 + k]) : 0.f;
        sw[k][row] = in && n0 + row < p.n ? value_of(p.w[(int64_t)(n0 + row) * p.ldw + k0 + k]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) t[i][j] += sa[k][ty * 4 + i] * sw[k][tx * 4 + j];
      __syncthreads();
    }
    const float s = p.w_scale[(int64_t)(n0 / kFp8Group) * groups + b];
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + ty * 4 + i;
      const float u = row < p.m ? p.a_scale[b * p.ld_as + row] * s : 0.f;
      for (int j = 0; j < 4; ++j) acc[i][j] += t[i][j] * u;
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int row = i0 + ty * 4 + i, col = n0 + tx * 4 + j;
      if (row >= p.m || col >= p.n) continue;
      int o = 0;
      while (col >= p.outs[o].end) ++o;
      static_cast<O*>(p.outs[o].out)[row * p.outs[o].ld + col - p.outs[o].begin] = from_f32<O>(acc[i][j]);
    }
}

}  // namespace

cudaError_t launch_fp8_linear(const Fp8LinearArgs& a, bool bf16_out, cudaStream_t st) {
  const dim3 grid((a.n + kTile - 1) / kTile, (a.m + kTile - 1) / kTile);
  return bf16_out ? launch_chained(fp8_linear_simple_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, a)
                  : launch_chained(fp8_linear_simple_kernel<float>, grid, dim3(256), 0, st, a);
}

}  // namespace qkn
