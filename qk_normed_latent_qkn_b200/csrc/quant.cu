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

// ---------------------------------------------------------------- rows held in registers
// One CTA per row, and the row read once: every thread keeps its values of h until the sum of squares
// is known.  Two layouts:
//   * pieces of 8 (rows that are 16-byte aligned, d a multiple of 8): thread t holds the pieces t, t + T,
//     ..., of T threads, so 16 neighbouring lanes hold a block of 128 and its maximum takes 4 exchanges;
//   * elements (anything else): a warp holds the blocks w, w + W, ..., lane l the elements l + 32 e, so
//     that every access is a run of 32 elements wherever it starts.
constexpr int kPiece = 8;
constexpr int kMaxThreads = 1024;

template <typename T>
__device__ __forceinline__ void load_piece(const T* p, float (&v)[kPiece]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}

// Rounds the piece to T, stores it and leaves the rounded values in v.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, float (&v)[kPiece]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<uint32_t*>(&t);
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ uint2 codes_of(const float (&v)[kPiece], float rs) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * e] * rs, v[2 * e + 1] * rs), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ float piece_max(const float (&v)[kPiece]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < kPiece; ++e) m = max_nan(m, fabsf(v[e]));
  return m;
}
// Maximum over the 16 lanes that hold a block's pieces.
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

template <typename T, int PIECES, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_quant_pieces_kernel(NormQuantArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = blockIdx.x;
  const int d = a.d, threads = blockDim.x;
  const T* x = static_cast<const T*>(a.x) + i * a.ld_x;
  float h[PIECES][kPiece];
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    const int j = ((int)threadIdx.x + c * threads) * kPiece;
    if (j < d) {
      load_piece(x + j, h[c]);
    } else {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) h[c][e] = 0.f;
    }
  }
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + i * d;
    float t[PIECES][kPiece];
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      const int j = ((int)threadIdx.x + c * threads) * kPiece;
      if (j < d) load_piece(r + j, t[c]);
    }
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      const int j = ((int)threadIdx.x + c * threads) * kPiece;
      if (j < d) {
#pragma unroll
        for (int e = 0; e < kPiece; ++e) h[c][e] += t[c][e];
        store_piece(static_cast<T*>(a.residual_out) + i * d + j, h[c]);
      }
    }
  }
  if (a.gamma) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < PIECES; ++c)
#pragma unroll
      for (int e = 0; e < kPiece; ++e) sum += h[c][e] * h[c][e];
    const float inv = 1.f / sqrtf(block_sum(sum) / (float)d + a.eps);
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      const int j = ((int)threadIdx.x + c * threads) * kPiece;
      if (j < d) {
        float g[kPiece];
        load_piece(a.gamma + j, g);
#pragma unroll
        for (int e = 0; e < kPiece; ++e) h[c][e] = h[c][e] * inv * g[e];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    const int j = ((int)threadIdx.x + c * threads) * kPiece;
    const float s = scale_of(half_warp_max(piece_max(h[c])));
    if (j < d) {
      *reinterpret_cast<uint2*>(a.codes + i * a.ld + j) = codes_of(h[c], 1.f / s);
      if (j % kFp8Group == 0) a.scale[j / kFp8Group * a.ld_scale + i] = s;
      if (a.y) store_piece(static_cast<T*>(a.y) + i * d + j, h[c]);
    }
  }
}

template <typename T, int BLOCKS, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_quant_elements_kernel(NormQuantArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = blockIdx.x;
  const int d = a.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const T* x = static_cast<const T*>(a.x) + i * a.ld_x;
  float h[BLOCKS][4];
#pragma unroll
  for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
      h[c][e] = j < d ? to_f32(x[j]) : 0.f;
    }
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + i * d;
    float t[BLOCKS][4];
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
        t[c][e] = j < d ? to_f32(r[j]) : 0.f;
      }
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
        const T u = from_f32<T>(h[c][e] + t[c][e]);
        h[c][e] = to_f32(u);
        if (j < d) static_cast<T*>(a.residual_out)[i * d + j] = u;
      }
  }
  if (a.gamma) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += h[c][e] * h[c][e];
    const float inv = 1.f / sqrtf(block_sum(sum) / (float)d + a.eps);
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
        if (j < d) h[c][e] = h[c][e] * inv * a.gamma[j];
      }
  }
#pragma unroll
  for (int c = 0; c < BLOCKS; ++c) {
    const int g = warp + c * warps;
    if (g * kFp8Group >= d) break;
    float m = fabsf(h[c][0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) m = max_nan(m, fabsf(h[c][e]));
    const float s = scale_of(warp_max_nan(m)), rs = 1.f / s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = g * kFp8Group + e * 32 + lane;
      if (j < d) {
        a.codes[i * a.ld + j] = code_of(h[c][e] * rs);
        if (a.y) static_cast<T*>(a.y)[i * d + j] = from_f32<T>(h[c][e]);
      }
    }
    if (lane == 0) a.scale[g * a.ld_scale + i] = s;
  }
}

// ---------------------------------------------------------------- rows too long for registers
// The row is read twice (the second time from the cache): once for the sum of squares, once for the
// codes, a warp per block of 128 columns.  The second pass reads h back where it was stored, so x and
// residual may be overwritten in place.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_quant_long_kernel(NormQuantArgs a) {
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
    for (int j = threadIdx.x; j < d; j += kMaxThreads) {
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
  for (int64_t g = threadIdx.x >> 5; g * kFp8Group < d; g += kMaxThreads / 32) {
    float v[4], m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t j = g * kFp8Group + e * 32 + lane;
      v[e] = 0.f;
      if (j < d) {
        v[e] = to_f32(h_in[j]);
        if (a.gamma) v[e] = v[e] * inv * a.gamma[j];
      }
      m = max_nan(m, fabsf(v[e]));
    }
    const float s = scale_of(warp_max_nan(m)), rs = 1.f / s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t j = g * kFp8Group + e * 32 + lane;
      if (j < d) {
        a.codes[i * a.ld + j] = code_of(v[e] * rs);
        if (y_out) y_out[j] = from_f32<T>(v[e]);
      }
    }
    if (lane == 0) a.scale[g * a.ld_scale + i] = s;
  }
}

// ---------------------------------------------------------------- weights
constexpr int kWeightThreads = 256;

// Largest magnitude of the CTA's threads.
__device__ __forceinline__ float block_max(float m) {
  __shared__ float part[kWeightThreads / 32];
  m = warp_max_nan(m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWeightThreads / 32; ++i) m = max_nan(m, part[i]);
  return m;
}

// One CTA per block of 128 x 128, read once into registers.  WIDE: in pieces of 8 (16-byte aligned rows),
// 16 threads along a row; else element by element, 128 threads along a row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kWeightThreads) quant_weight_kernel(QuantWeightArgs a, int k_blocks) {
  pdl_trigger();
  pdl_wait();
  const int kb = blockIdx.x % k_blocks;
  const int64_t row0 = (int64_t)(blockIdx.x / k_blocks) * kFp8Group;
  const T* w = static_cast<const T*>(a.w);
  constexpr int W = WIDE ? kPiece : 1, ACROSS = kFp8Group / W, STEP = kWeightThreads / ACROSS, ROWS = kFp8Group / STEP;
  const int col = kb * kFp8Group + (int)(threadIdx.x % ACROSS) * W;
  const int64_t row = row0 + threadIdx.x / ACROSS;
  float v[ROWS][W], m = 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const bool in = row + r * STEP < a.n && col < a.k;
    if constexpr (WIDE) {
      if (in) {
        load_piece(w + (row + r * STEP) * a.k + col, v[r]);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) v[r][e] = 0.f;
      }
    } else {
      v[r][0] = in ? to_f32(w[(row + r * STEP) * a.k + col]) : 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int e = 0; e < W; ++e) m = max_nan(m, fabsf(v[r][e]));
  const float s = scale_of(block_max(m)), rs = 1.f / s;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (row + r * STEP >= a.n || col >= a.k) continue;
    uint8_t* dst = a.codes + (row + r * STEP) * a.ld + col;
    if constexpr (WIDE) {
      *reinterpret_cast<uint2*>(dst) = codes_of(v[r], rs);
    } else {
      *dst = code_of(v[r][0] * rs);
    }
  }
  if (threadIdx.x == 0) a.scale[blockIdx.x] = s;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

template <typename T>
cudaError_t launch_norm(const NormQuantArgs& a, cudaStream_t st) {
  const dim3 grid(a.n);
  const bool wide = a.d % kPiece == 0 && a.ld_x * sizeof(T) % 16 == 0 && on16(a.x) && on16(a.residual) &&
                    on16(a.residual_out) && on16(a.gamma) && on16(a.y);
  const int pieces = (a.d + kPiece - 1) / kPiece, blocks = (a.d + kFp8Group - 1) / kFp8Group;
  if (wide && pieces <= 4 * kMaxThreads) {
    // few rows: one piece per thread, the shortest chain; many: more loads in flight per thread
    const bool few = a.n <= 512;
    if (pieces <= (few ? kMaxThreads : 128))
      return launch_chained(norm_quant_pieces_kernel<T, 1, kMaxThreads>, grid, dim3(round32(pieces)), 0, st, a);
    if (pieces <= (few ? 2 * kMaxThreads : 1024))
      return launch_chained(norm_quant_pieces_kernel<T, 2, kMaxThreads>, grid, dim3(round32((pieces + 1) / 2)), 0, st,
                            a);
    const dim3 block(round32((pieces + 3) / 4));
    return pieces <= 4 * 512 ? launch_chained(norm_quant_pieces_kernel<T, 4, 512>, grid, block, 0, st, a)
                             : launch_chained(norm_quant_pieces_kernel<T, 4, kMaxThreads>, grid, block, 0, st, a);
  }
  if (blocks <= 2 * 32)
    return launch_chained(norm_quant_elements_kernel<T, 2, kMaxThreads>, grid, dim3((blocks + 1) / 2 * 32), 0, st, a);
  if (blocks <= 8 * 16)
    return launch_chained(norm_quant_elements_kernel<T, 8, 512>, grid, dim3((blocks + 7) / 8 * 32), 0, st, a);
  return launch_chained(norm_quant_long_kernel<T>, grid, dim3(kMaxThreads), 0, st, a);
}

template <typename T>
cudaError_t launch_weight(const QuantWeightArgs& a, cudaStream_t st) {
  const int k_blocks = (int)(((int64_t)a.k + kFp8Group - 1) / kFp8Group);
  const int64_t ctas = (int64_t)k_blocks * (((int64_t)a.n + kFp8Group - 1) / kFp8Group);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas), block(kWeightThreads);
  return a.k % kPiece == 0 && on16(a.w) ? launch_chained(quant_weight_kernel<T, true>, grid, block, 0, st, a, k_blocks)
                                        : launch_chained(quant_weight_kernel<T, false>, grid, block, 0, st, a, k_blocks);
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_norm<__nv_bfloat16>(a, st) : launch_norm<float>(a, st);
}

cudaError_t launch_quant_weight(const QuantWeightArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_weight<__nv_bfloat16>(a, st) : launch_weight<float>(a, st);
}

}  // namespace qkn
