// Quantisation to 8 bits: activations row by row with the residual addition and RMSNorm in front
// (qkn_norm_quant), and weights (qkn_quant_weight).
//
// Mathematics.  h = x + r (rounded to the storage type, which is what the next layer reads back);
// y = h * gamma * (mean(h^2) + eps)^-1/2; for every block of 128 columns s = max(max|y| / 448, 2^-100)
// and code = e4m3(y / s).  All in fp32: the only roundings to fewer bits are the stored h, the optional
// y and the codes.  The codes are formed as y * (1 / s): the reciprocal's rounding moves a value by at
// most 2^-23 of itself, which changes a code only where y / s lies that close to the middle between
// two codes.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace qkn {
namespace {

// Larger of two magnitudes; NaN if either is (fmaxf would drop it and hide a NaN in a block).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float scale_of(float amax) { return max_nan(amax / kFp8Top, kFp8Least); }

__device__ __forceinline__ uint8_t code_of(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum over the CTA's threads (a multiple of 32, at most 1024); every thread gets it.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += part[w];
  return s;
}

constexpr int kAnyThreads = 256;

// Any width, alignment and row stride: one CTA per row, element loads.  The row is read twice (the
// second time from the cache): once for the sum of squares, once for the codes, a warp per block of
// 128 columns.  The second pass reads h back where it was stored, so x and residual may be
// overwritten in place.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) norm_quant_any_kernel(NormQuantArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = blockIdx.x;
  const int d = a.d;
  const T* x = static_cast<const T*>(a.x) + i * a.ld_x;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + i * d : nullptr;
  T* h_out = a.residual ? static_cast<T*>(a.residual_out) + i * d : nullptr;
  float inv = 1.f;
  if (r || a.gamma) {
    float sum = 0.f;
    for (int j = threadIdx.x; j < d; j += kAnyThreads) {
      float h = to_f32(x[j]);
      if (r) {
        const T t = from_f32<T>(h + to_f32(r[j]));
        h_out[j] = t;
        h = to_f32(t);
      }
      sum += h * h;
    }
    sum = block_sum(sum);   // (also orders the stores of h before the second pass of other threads)
    if (a.gamma) inv = 1.f / sqrtf(sum / (float)d + a.eps);
  }
  const T* h_in = r ? h_out : x;
  T* y_out = a.y ? static_cast<T*>(a.y) + i * d : nullptr;
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g * kFp8Group < d; g += kAnyThreads / 32) {
    float v[4], amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = g * kFp8Group + e * 32 + lane;
      v[e] = 0.f;
      if (j < d) {
        v[e] = to_f32(h_in[j]);
        if (a.gamma) v[e] = v[e] * inv * a.gamma[j];
      }
      amax = max_nan(amax, fabsf(v[e]));
    }
    const float s = scale_of(warp_max_nan(amax)), rs = 1.f / s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = g * kFp8Group + e * 32 + lane;
      if (j < d) {
        a.codes[i * a.ld + j] = code_of(v[e] * rs);
        if (y_out) y_out[j] = from_f32<T>(v[e]);
      }
    }
    if (lane == 0) a.scale[g * a.ld_scale + i] = s;
  }
}

constexpr int kWeightThreads = 256;

// One CTA per block of 128 x 128: the largest magnitude, then the codes (the second read is from the cache).
template <typename T>
__global__ void __launch_bounds__(kWeightThreads) quant_weight_kernel(QuantWeightArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float part[kWeightThreads / 32];
  const int kb = blockIdx.x, nb = blockIdx.y;
  const T* w = static_cast<const T*>(a.w);
  const int col = kb * kFp8Group + (threadIdx.x & 127);
  float amax = 0.f;
  for (int r = threadIdx.x >> 7; r < kFp8Group; r += kWeightThreads / 128) {
    const int64_t row = (int64_t)nb * kFp8Group + r;
    if (row < a.n && col < a.k) amax = max_nan(amax, fabsf(to_f32(w[row * a.k + col])));
  }
  amax = warp_max_nan(amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int i = 0; i < kWeightThreads / 32; ++i) amax = max_nan(amax, part[i]);
  const float s = scale_of(amax), rs = 1.f / s;
  for (int r = threadIdx.x >> 7; r < kFp8Group; r += kWeightThreads / 128) {
    const int64_t row = (int64_t)nb * kFp8Group + r;
    if (row < a.n && col < a.k) a.codes[row * a.ld + col] = code_of(to_f32(w[row * a.k + col]) * rs);
  }
  if (threadIdx.x == 0) a.scale[(int64_t)nb * gridDim.x + kb] = s;
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_chained(norm_quant_any_kernel<__nv_bfloat16>, dim3(a.n), dim3(kAnyThreads), 0, st, a)
              : launch_chained(norm_quant_any_kernel<float>, dim3(a.n), dim3(kAnyThreads), 0, st, a);
}

cudaError_t launch_quant_weight(const QuantWeightArgs& a, bool bf16, cudaStream_t st) {
  const dim3 grid((a.k + kFp8Group - 1) / kFp8Group, (a.n + kFp8Group - 1) / kFp8Group);
  return bf16 ? launch_chained(quant_weight_kernel<__nv_bfloat16>, grid, dim3(kWeightThreads), 0, st, a)
              : launch_chained(quant_weight_kernel<float>, grid, dim3(kWeightThreads), 0, st, a);
}

}  // namespace qkn
