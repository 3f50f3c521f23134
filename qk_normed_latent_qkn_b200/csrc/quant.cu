// Quantisation to 8 bits: activations row by row with the residual addition and RMSNorm in front
// (qkn_norm_quant), and weights (qkn_quant_weight).
//
// Mathematics.  h = x + r (rounded to the storage type, which is what the next layer reads back);
// y = h * gamma * (mean(h^2) + eps)^-1/2; for every block of 128 columns s = max(max|y| / 448, 2^-100)
// and code = e4m3(y / s).  All in fp32: the only roundings to fewer bits are the stored h, the optional
// y and the codes.  A code is the nearest e4m3 to the fp32 quotient y / s, taken without a division per
// value: see Quotient.
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

// (times the rounded reciprocal, within 1.75 * 2^-24 of the quotient: what a tensor divided by a number is in
// torch on a GPU, so that scales and codes agree with weights that were quantised there)
__device__ __forceinline__ float scale_of(float amax) { return max_nan(amax * (1.f / kFp8Top), kFp8Least); }

// v / s for the values of a block from r = 1 / s: q = v r, corrected by its remainder, v - q s, times r
// (Markstein's division).  It gives the code that the correctly rounded quotient gives, for every v and s: before
// its last rounding it is within 2^-22 units of the last place of v / s, so the codes could part only where v / s
// lies that close to a border between the fp32 numbers that round to the middle of two codes and their
// neighbours; a test goes through all significands for which it does.  (Below a scale of 2^-93 a remainder may
// underflow; a code can then differ where v / s is within 2^-16 units of such a border.)  v r alone gives
// another code for 0.05 % of normal bf16 weights.  The correction costs nothing on the norm below (71.5 us either
// way on a B200), 47.7 -> 52 us on the weight and 11.4 -> 12.2 on 1021 x 16384 bf16 without a norm; one value at a
// time it cost 1.5 us more on each.
struct Quotient {
  float s, r;
  // (an infinite scale has r = 0: finite values become 0, infinities NaN, and a remainder would spoil the former)
  __device__ __forceinline__ explicit Quotient(float scale) : s(isinf(scale) ? 0.f : scale), r(1.f / scale) {}
  __device__ __forceinline__ float operator()(float v) const {
    const float q = v * r;
    return fmaf(fmaf(-q, s, v), r, q);
  }
  // Two at once, in packed instructions.
  __device__ __forceinline__ float2 operator()(float a, float b) const {
    float2 o;
    asm("{\n\t.reg .b64 v, s, r, q;\n\t"
        "mov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
        "mul.rn.f32x2 q, v, r;\n\t"
        "fma.rn.f32x2 v, q, s, v;\n\t"
        "fma.rn.f32x2 q, v, r, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=f"(o.x), "=f"(o.y)
        : "f"(a), "f"(b), "f"(-s), "f"(r));
    return o;
  }
};

__device__ __forceinline__ uint8_t code_of(float q) {
  return (uint8_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
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
// One CTA per row (without a norm: per 4096 columns of a row), and the row read once: every thread keeps
// its values of h until the sum of squares is known, as they are stored, so that in bf16 32 registers
// suffice and an SM holds all its 2048 threads.  Bound by memory: 16384 x 4096 bf16 with the residual
// (472 MB) takes 71.5 us on a B200, 6.6 TB/s; 82 to 90 us with h kept in fp32.  Thread t holds the pieces of
// 8 values t, t + T, ..., of T threads, so 16 neighbouring lanes hold a block of 128 and its maximum takes 4
// exchanges.  bf16 rows that are not 16-byte aligned are read in aligned chunks and shifted into place;
// fp32 ones go by elements, a warp per block of 128.
constexpr int kPiece = 8;
constexpr int kMaxThreads = 1024;

// 8 consecutive values of type T as they are stored.
template <typename T>
struct Piece {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int e = 0; e < (int)sizeof(T) / 2; ++e) u[e] = reinterpret_cast<const uint4*>(p)[e];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int e = 0; e < (int)sizeof(T) / 2; ++e) reinterpret_cast<uint4*>(p)[e] = u[e];
  }
  // The first `valid` values from p, which need not be aligned: the 16-byte chunks that hold them, shifted
  // into place, where all of these lie within [lo, hi), the array's bounds; else element by element.
  __device__ __forceinline__ void load_any(const T* p, int valid, const T* lo, const T* hi) {
    constexpr int NW = sizeof(T) * 2, NC = NW / 4 + 1;   // words of a piece, chunks that hold it
    const uintptr_t off = reinterpret_cast<uintptr_t>(p) & 15;
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
    uint32_t w[4 * NC];
    if (valid == kPiece && reinterpret_cast<const char*>(q) >= reinterpret_cast<const char*>(lo) &&
        reinterpret_cast<const char*>(q + NC) <= reinterpret_cast<const char*>(hi)) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint4 c = q[i];
        w[4 * i] = c.x, w[4 * i + 1] = c.y, w[4 * i + 2] = c.z, w[4 * i + 3] = c.w;
      }
      if (off & 8) {
#pragma unroll
        for (int i = 0; i < NW + 2; ++i) w[i] = w[i + 2];
      }
      if (off & 4) {
#pragma unroll
        for (int i = 0; i < NW + 1; ++i) w[i] = w[i + 1];
      }
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < NW; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (uint32_t)(off & 2) * 8);
      }
    } else {
      float f[kPiece];
#pragma unroll
      for (int e = 0; e < kPiece; ++e) f[e] = e < valid ? to_f32(p[e]) : 0.f;
      set(f);   // (exact: the values are T's)
      return;
    }
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  // The first `valid` values to p, in the widest stores that its alignment allows.
  __device__ __forceinline__ void store_any(T* p, int valid) const {
    uint32_t w[sizeof(T) * 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[4 * i] = u[i].x, w[4 * i + 1] = u[i].y, w[4 * i + 2] = u[i].z, w[4 * i + 3] = u[i].w;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    if (valid < kPiece) {
      float f[kPiece];
      values(f);
#pragma unroll
      for (int e = 0; e < kPiece; ++e)
        if (e < valid) p[e] = from_f32<T>(f[e]);
    } else if (off == 0) {
      store(p);
    } else if constexpr (sizeof(T) == 4) {
      if (off == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint4*>(p + 2) = make_uint4(w[2], w[3], w[4], w[5]);
        *reinterpret_cast<uint2*>(p + 6) = make_uint2(w[6], w[7]);
      } else {
        *reinterpret_cast<uint32_t*>(p) = w[0];
#pragma unroll
        for (int i = 1; i < 7; i += 2) *reinterpret_cast<uint2*>(p + i) = make_uint2(w[i], w[i + 1]);
        *reinterpret_cast<uint32_t*>(p + 7) = w[7];
      }
    } else {
      if (off & 2) {
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(p + 1 + 2 * i) = __funnelshift_r(w[i], w[i + 1], 16);
        *reinterpret_cast<uint16_t*>(p + 7) = (uint16_t)(w[3] >> 16);
      } else if (off & 4) {
        *reinterpret_cast<uint32_t*>(p) = w[0];
        *reinterpret_cast<uint2*>(p + 2) = make_uint2(w[1], w[2]);
        *reinterpret_cast<uint32_t*>(p + 6) = w[3];
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < (int)sizeof(T) / 2; ++e) u[e] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&v)[kPiece]) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
      for (int e = 0; e < kPiece; ++e) v[e] = __uint_as_float(w[e]);
    } else {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
  // Rounds to T.
  __device__ __forceinline__ void set(const float (&v)[kPiece]) {
    if constexpr (sizeof(T) == 4) {
      u[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      u[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        w[e] = *reinterpret_cast<uint32_t*>(&t);
      }
      u[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

__device__ __forceinline__ uint2 codes_of(const float (&v)[kPiece], const Quotient& by) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = __nv_cvt_float2_to_fp8x2(by(v[2 * e], v[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// A piece's codes (rows of codes are 16-byte aligned); ANY: only the first `valid` of them.
template <bool ANY>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 c, int valid) {
  if (!ANY || valid >= kPiece) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
    const uint64_t b = (uint64_t)c.y << 32 | c.x;
#pragma unroll
    for (int e = 0; e < kPiece - 1; ++e)
      if (e < valid) p[e] = (uint8_t)(b >> (8 * e));
  }
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

// ANY: rows of any alignment and width; else 16-byte aligned rows of whole pieces.
template <typename T, int PIECES, int THREADS, int CTAS, bool ANY>
__global__ void __launch_bounds__(THREADS, CTAS) norm_quant_pieces_kernel(NormQuantArgs a, int parts) {
  pdl_trigger();
  pdl_wait();
  int64_t i = blockIdx.x;
  const int d = a.d, threads = blockDim.x;
  int j0 = (int)threadIdx.x * kPiece;
  if (parts > 1) {   // (only without a norm)
    i = blockIdx.x / parts;
    j0 += (int)(blockIdx.x % parts) * threads * PIECES * kPiece;
  }
  const int step = threads * kPiece;
  const T* x = static_cast<const T*>(a.x) + i * a.ld_x;
  Piece<T> h[PIECES];   // as stored: h is rounded to T, so nothing is lost
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    const int j = j0 + c * step;
    if (j >= d) {
      h[c].zero();
    } else if constexpr (ANY) {
      const T* x0 = static_cast<const T*>(a.x);
      h[c].load_any(x + j, min(d - j, kPiece), x0, x0 + (a.n - 1) * a.ld_x + d);
    } else {
      h[c].load(x + j);
    }
  }
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + i * d;
    Piece<T> t[PIECES];
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      const int j = j0 + c * step;
      if (j >= d) continue;
      if constexpr (ANY) {
        const T* r0 = static_cast<const T*>(a.residual);
        t[c].load_any(r + j, min(d - j, kPiece), r0, r0 + (int64_t)a.n * d);
      } else {
        t[c].load(r + j);
      }
    }
#pragma unroll
    for (int c = 0; c < PIECES; ++c)
      if (j0 + c * step < d) {
        float f[kPiece], g[kPiece];
        h[c].values(f);
        t[c].values(g);
#pragma unroll
        for (int e = 0; e < kPiece; ++e) f[e] += g[e];
        h[c].set(f);
        T* out = static_cast<T*>(a.residual_out) + i * d + j0 + c * step;
        if constexpr (ANY) h[c].store_any(out, min(d - j0 - c * step, kPiece));
        else h[c].store(out);
      }
  }
  float inv = 1.f;
  if (a.gamma) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      float f[kPiece];
      h[c].values(f);
#pragma unroll
      for (int e = 0; e < kPiece; ++e) sum += f[e] * f[e];
    }
    inv = 1.f / sqrtf(block_sum(sum) / (float)d + a.eps);
  }
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    const int j = j0 + c * step;
    float f[kPiece];
    h[c].values(f);
    if (a.gamma && j < d) {
      Piece<float> g;
      if constexpr (ANY) g.load_any(a.gamma + j, min(d - j, kPiece), a.gamma, a.gamma + d);
      else g.load(a.gamma + j);
      float gf[kPiece];
      g.values(gf);
#pragma unroll
      for (int e = 0; e < kPiece; ++e) f[e] = f[e] * inv * gf[e];
    }
    const float s = scale_of(half_warp_max(piece_max(f)));
    if (j < d) {
      store_codes<ANY>(a.codes + i * a.ld + j, codes_of(f, Quotient(s)), d - j);
      if (j % kFp8Group == 0) a.scale[j / kFp8Group * a.ld_scale + i] = s;
      if (a.y) {
        Piece<T> y;
        y.set(f);
        if constexpr (ANY) y.store_any(static_cast<T*>(a.y) + i * d + j, min(d - j, kPiece));
        else y.store(static_cast<T*>(a.y) + i * d + j);
      }
    }
  }
}

// fp32 rows of any alignment: element loads are whole 128-byte lines, pieces of 8 are not (2048 x 4095: 25 us
// on a B200, 34 in shifted pieces; in bf16 24.4 and 23.9, and 177 and 138 at 16384 rows).
template <int BLOCKS, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_quant_elements_kernel(NormQuantArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = blockIdx.x;
  const int d = a.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const float* x = static_cast<const float*>(a.x) + i * a.ld_x;
  float h[BLOCKS][4];
#pragma unroll
  for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
      h[c][e] = j < d ? x[j] : 0.f;
    }
  if (a.residual) {
    const float* r = static_cast<const float*>(a.residual) + i * d;
    float t[BLOCKS][4];
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
        t[c][e] = j < d ? r[j] : 0.f;
      }
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (warp + c * warps) * kFp8Group + e * 32 + lane;
        h[c][e] += t[c][e];
        if (j < d) static_cast<float*>(a.residual_out)[i * d + j] = h[c][e];
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
    const float s = scale_of(warp_max_nan(m));
    const Quotient by(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = g * kFp8Group + e * 32 + lane;
      if (j < d) {
        a.codes[i * a.ld + j] = code_of(by(h[c][e]));
        if (a.y) static_cast<float*>(a.y)[i * d + j] = h[c][e];
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
    const float s = scale_of(warp_max_nan(m));
    const Quotient by(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t j = g * kFp8Group + e * 32 + lane;
      if (j < d) {
        a.codes[i * a.ld + j] = code_of(by(v[e]));
        if (y_out) y_out[j] = from_f32<T>(v[e]);
      }
    }
    if (lane == 0) a.scale[g * a.ld_scale + i] = s;
  }
}

// ---------------------------------------------------------------- weights
// One CTA per block of 128 x 128, read once in pieces of 8, 16 lanes along a row (ANY: rows of any alignment
// and width; else 16-byte aligned rows of whole pieces).  Every thread keeps what it read, as it was read,
// until the block's maximum is known.  Bound by memory: several CTAs share an SM so that one block's loads run
// beside another's stores, and what a thread keeps decides how many.  bf16, 25152 x 4096 (309 MB) on a B200:
// 52 us, 5.9 TB/s, with three CTAs (which spill 4 bytes a thread); 61 with two, 55 with four (which spill 52).
constexpr int kWeightThreads = 512;

// Largest magnitude of the CTA's threads.
__device__ __forceinline__ float block_max(float m) {
  __shared__ float part[kWeightThreads / 32];
  m = warp_max_nan(m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  m = part[threadIdx.x & (kWeightThreads / 32 - 1)];
#pragma unroll
  for (int o = kWeightThreads / 64; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

template <typename T, bool ANY>
__global__ void __launch_bounds__(kWeightThreads, sizeof(T) == 2 ? 3 : 2)
    quant_weight_kernel(QuantWeightArgs a, int k_blocks) {
  pdl_trigger();
  pdl_wait();
  constexpr int STEP = kWeightThreads / 16, ROWS = kFp8Group / STEP;
  const int col = (int)(blockIdx.x % k_blocks) * kFp8Group + (int)(threadIdx.x & 15) * kPiece;
  const int64_t row = (int64_t)(blockIdx.x / k_blocks) * kFp8Group + (threadIdx.x >> 4);
  const T* w0 = static_cast<const T*>(a.w);
  const T* w = w0 + row * a.k + col;
  Piece<T> v[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (row + r * STEP >= a.n || col >= a.k) v[r].zero();
    else if constexpr (ANY) v[r].load_any(w + (int64_t)r * STEP * a.k, min(a.k - col, kPiece), w0, w0 + (int64_t)a.n * a.k);
    else v[r].load(w + (int64_t)r * STEP * a.k);
  }
  float m = 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float f[kPiece];
    v[r].values(f);
    m = max_nan(m, piece_max(f));
  }
  const float s = scale_of(block_max(m));
  const Quotient by(s);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (row + r * STEP >= a.n || col >= a.k) continue;
    float f[kPiece];
    v[r].values(f);
    store_codes<ANY>(a.codes + (row + r * STEP) * a.ld + col, codes_of(f, by), a.k - col);
  }
  if (threadIdx.x == 0) a.scale[blockIdx.x] = s;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

// CTAs of 256 threads on an SM that the pieces kernel is compiled for: what a thread keeps of a row fits 32
// registers in bf16 (all of an SM's threads), 64 in fp32.
template <typename T>
constexpr int kCtasOf = sizeof(T) == 2 ? 8 : 4;

template <typename T, bool ANY>
cudaError_t launch_norm_pieces(const NormQuantArgs& a, cudaStream_t st) {
  constexpr int kCtas = ANY ? kCtasOf<T> / 2 : kCtasOf<T>;
  const dim3 grid(a.n);
  const int pieces = (a.d + kPiece - 1) / kPiece;
  if (!a.gamma) {   // every block of 128 stands alone: rows in parts of up to 4096 columns
    const int per = (pieces + 1) / 2, threads = per < 256 ? round32(per) : 256;
    const int parts = (pieces + 2 * threads - 1) / (2 * threads);
    if ((int64_t)a.n * parts <= INT32_MAX)
      return launch_chained(norm_quant_pieces_kernel<T, 2, 256, kCtas, ANY>, dim3(a.n * parts), dim3(threads), 0, st, a,
                            parts);
  }
  // few rows: one piece per thread, the shortest chain; many: CTAs of 256 threads with 2 pieces, an SM full of them
  // (us on a B200, this way and the other, bf16 with residual: 1 x 4096 2.0 and 2.4, 256 x 4096 4.6 and 5.8,
  // 512 x 4096 5.4 and 7.0, 512 x 7168 9.0 and 7.9; 1024 x 4096 8.5 and 8.6, 2048 x 4096 13.5 and 14.1,
  // 1024 x 7168 12.9 and 14.9)
  const bool few = a.n <= 512;
  if (pieces <= (few ? kMaxThreads : 256))
    return launch_chained(norm_quant_pieces_kernel<T, 1, kMaxThreads, 1, ANY>, grid, dim3(round32(pieces)), 0, st, a, 1);
  if (!few && pieces <= 2 * 256)
    return launch_chained(norm_quant_pieces_kernel<T, 2, 256, kCtas, ANY>, grid, dim3(round32((pieces + 1) / 2)), 0, st,
                          a, 1);
  if (pieces <= 2 * kMaxThreads)
    return launch_chained(norm_quant_pieces_kernel<T, 2, kMaxThreads, (kCtas >= 4 ? kCtas / 4 : 1), ANY>, grid,
                          dim3(round32((pieces + 1) / 2)), 0, st, a, 1);
  // (in fp32 this instance spills 156 bytes a thread)
  return launch_chained(norm_quant_pieces_kernel<T, 4, kMaxThreads, 1, ANY>, grid, dim3(round32((pieces + 3) / 4)), 0,
                        st, a, 1);
}

template <typename T>
cudaError_t launch_norm(const NormQuantArgs& a, cudaStream_t st) {
  const bool aligned = a.d % kPiece == 0 && a.ld_x * sizeof(T) % 16 == 0 && on16(a.x) && on16(a.residual) &&
                       on16(a.residual_out) && on16(a.gamma) && on16(a.y);
  if (a.d > 4 * kMaxThreads * kPiece)
    return launch_chained(norm_quant_long_kernel<T>, dim3(a.n), dim3(kMaxThreads), 0, st, a);
  if (aligned) return launch_norm_pieces<T, false>(a, st);
  if constexpr (sizeof(T) == 4) {
    const int blocks = (a.d + kFp8Group - 1) / kFp8Group;
    if (blocks <= 2 * 32)
      return launch_chained(norm_quant_elements_kernel<2, kMaxThreads>, dim3(a.n), dim3((blocks + 1) / 2 * 32), 0, st, a);
    if (blocks <= 8 * 16)
      return launch_chained(norm_quant_elements_kernel<8, 512>, dim3(a.n), dim3((blocks + 7) / 8 * 32), 0, st, a);
    return launch_chained(norm_quant_long_kernel<T>, dim3(a.n), dim3(kMaxThreads), 0, st, a);
  } else {
    return launch_norm_pieces<T, true>(a, st);
  }
}

template <typename T>
cudaError_t launch_weight(const QuantWeightArgs& a, cudaStream_t st) {
  const int k_blocks = (int)(((int64_t)a.k + kFp8Group - 1) / kFp8Group);
  const int64_t ctas = (int64_t)k_blocks * (((int64_t)a.n + kFp8Group - 1) / kFp8Group);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas), block(kWeightThreads);
  return a.k % kPiece == 0 && on16(a.w) ? launch_chained(quant_weight_kernel<T, false>, grid, block, 0, st, a, k_blocks)
                                        : launch_chained(quant_weight_kernel<T, true>, grid, block, 0, st, a, k_blocks);
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_norm<__nv_bfloat16>(a, st) : launch_norm<float>(a, st);
}

cudaError_t launch_quant_weight(const QuantWeightArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_weight<__nv_bfloat16>(a, st) : launch_weight<float>(a, st);
}

}  // namespace qkn
