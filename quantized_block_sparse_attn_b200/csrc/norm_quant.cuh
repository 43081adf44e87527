// INT8 codes with one scale per token, from activations: the residual's addition, the
// root-mean-square norm and the quantiser in one pass (rms_norm_quant), or the quantiser
// alone (quantize_token).
//
// For a row x of `width` values: h = x, or x + residual rounded to x's type (the rounded sum
// is what the next layer reads, so it is also what is normalised), g = h * weight in f32,
// a = max|g|, s = max(a / 127, 2^-126) (1 if a = 0), codes = rint_half_even(RN(g / s)) and
// scale = s / sqrt(mean(h^2) + eps) (1 if a = 0).  The norm's factor 1 / sqrt(..) is common to
// a row, so it cancels in the codes: they depend on g alone, not on the order in which the
// mean is summed, and the sum and the maximum come out of one pass and one reduction.
// Without the norm, g = h = x and scale = s, the rule of the Q / K quantiser per row.
// 2^-126 keeps the quotient finite and below 127.5 when a / 127 would be subnormal.
// A row that holds (or whose products reach) a NaN or an infinity has no scale: codes 0,
// scale NaN.
//
// Bound by HBM: x (and the residual) read once, h and the codes written once.  The row
// stays in registers between the reduction and the codes.
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "quantize.cuh"

namespace qbsa {

struct NormQuantParams {
  const void* x;
  const void* residual;  // kRes
  const void* weight;    // kNorm
  void* h_out;           // kRes
  int8_t* codes;
  float* scales;
  int64_t x_stride, r_stride, h_stride, c_stride;  // row strides in elements
  int64_t rows;
  int width;
  int group;  // threads of a row: a power of two up to 32, or all of the CTA
  int weight_f32;
  float eps;
};

constexpr int kNormWideThreads = 1024;
constexpr int kNormScalarValues = 8;  // values of a thread when rows are not 16-byte aligned

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// E values of a row as they are stored.  Loads of a whole piece come before the first use, so
// that every piece of a thread is in flight at once.
template <typename T, int E>
struct alignas(E * sizeof(T)) Piece {
  T v[E];
};

// E consecutive values, or the last n < E of a row.  E > 1: p is 16-byte aligned and E values of
// T are 16 bytes.
template <typename T, int E>
__device__ __forceinline__ Piece<T, E> load_piece(const T* p, int n) {
  Piece<T, E> out;
  if constexpr (E > 1) {
    static_assert(E * sizeof(T) == 16, "a piece is one 16-byte load");
    if (n >= E) {
      uint4 u;
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                   : "l"(p)
                   : "memory");
      memcpy(&out, &u, 16);
      return out;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) out.v[i] = i < n ? p[i] : from_f32<T>(0.f);
  return out;
}

// The norm's weights, read by every row: kept in L1.
template <typename T, int E>
__device__ __forceinline__ void load_weight(const NormQuantParams& p, int at, int n, float (&f)[E]) {
  if (p.weight_f32) {
    const float* w = static_cast<const float*>(p.weight) + at;
    if (E > 1 && n >= E) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(w) + i);
        f[4 * i] = u.x;
        f[4 * i + 1] = u.y;
        f[4 * i + 2] = u.z;
        f[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = i < n ? __ldg(w + i) : 0.f;
    }
  } else {
    const T* w = static_cast<const T*>(p.weight) + at;
    if (E > 1 && n >= E) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(w));
      const T* v = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = to_f32(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = i < n ? to_f32(w[i]) : 0.f;
    }
  }
}

template <typename T, int E>
__device__ __forceinline__ void store_values(T* p, int n, const float (&f)[E]) {
  if constexpr (E > 1) {
    if (n >= E) {
      uint4 u;
      T* v = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = from_f32<T>(f[i]);
      *reinterpret_cast<uint4*>(p) = u;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < n) p[i] = from_f32<T>(f[i]);
}

template <int E>
__device__ __forceinline__ void store_codes(int8_t* p, int n, const uint32_t (&c)[E]) {
  if constexpr (E == 8) {
    if (n >= E) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_low_bytes(c[0], c[1], c[2], c[3]),
                                                pack_low_bytes(c[4], c[5], c[6], c[7]));
      return;
    }
  }
  if constexpr (E == 4) {
    if (n >= E) {
      *reinterpret_cast<uint32_t*>(p) = pack_low_bytes(c[0], c[1], c[2], c[3]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < n) p[i] = static_cast<int8_t>(c[i]);
}

// Sum and maximum over the threads of a row.  `a` is a magnitude's bits: unsigned order is the
// order of the magnitudes, with infinity and then NaN above every number.
__device__ __forceinline__ void row_reduce(int group, float& sum, uint32_t& a) {
  for (int o = min(group, 32) >> 1; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  }
  if (group <= 32) return;
  __shared__ float red_sum[32];
  __shared__ uint32_t red_max[32];
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) {
    red_sum[threadIdx.x >> 5] = sum;
    red_max[threadIdx.x >> 5] = a;
  }
  __syncthreads();
  sum = lane < warps ? red_sum[lane] : 0.f;
  a = lane < warps ? red_max[lane] : 0u;
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  a = __reduce_max_sync(0xffffffffu, a);
}

// Whether a row's values are numbers; their step s and its reciprocal for int8_code_byte.
__device__ __forceinline__ bool row_step(uint32_t a_bits, float& s, float& r) {
  const float a = __uint_as_float(a_bits);
  s = a_bits == 0 ? 1.0f : fmaxf(__fdiv_rn(a, 127.0f), 1.17549435e-38f);
  r = __frcp_rn(s);  // at most 2^126: finite
  return a_bits < 0x7f800000u;
}

// The row's scale.  sum = sum of (h * unit)^2, unit 1 unless the squares overflow.
template <bool kNorm>
__device__ __forceinline__ float row_scale(uint32_t a_bits, bool numbers, float s, float sum, float unit, int width,
                                           float eps) {
  if (!numbers) return __uint_as_float(0x7fc00000u);
  if (!kNorm || a_bits == 0) return s;
  const float mean = __fdiv_rn(sum, static_cast<float>(width));
  return __fdiv_rn(s, __fsqrt_rn(mean + eps * unit * unit)) * unit;
}

// h (stored), its square sum and g of the E values at `at`
template <typename T, bool kNorm, bool kRes, int E>
__device__ __forceinline__ void take_values(const NormQuantParams& p, int64_t row, int at, int n,
                                            const Piece<T, E>& x, const Piece<T, E>& q, float (&g)[E], float& sum,
                                            uint32_t& a) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    g[i] = to_f32(x.v[i]);
    if constexpr (kRes) g[i] = to_f32(from_f32<T>(g[i] + to_f32(q.v[i])));
  }
  if constexpr (kRes) store_values<T, E>(static_cast<T*>(p.h_out) + row * p.h_stride + at, n, g);
  if constexpr (kNorm) {
    float w[E];
    load_weight<T, E>(p, at, n, w);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      sum = __fmaf_rn(g[i], g[i], sum);
      g[i] *= w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) a = max(a, __float_as_uint(g[i]) & 0x7fffffffu);
}

// Squares that overflow in f32 (a finite row above about 1e19): the sum again, of h * 2^-64.
template <typename T, bool kRes>
__device__ __noinline__ float sum_scaled(const NormQuantParams& p, int64_t row, int member, int step) {
  const T* h = kRes ? static_cast<const T*>(p.h_out) + row * p.h_stride
                    : static_cast<const T*>(p.x) + row * p.x_stride;
  float sum = 0.f;
  for (int i = member; i < p.width; i += step) {
    const float v = to_f32(h[i]) * 5.421010862427522e-20f;
    sum = __fmaf_rn(v, v, sum);
  }
  return sum;
}

// A row in registers: kChunks pieces of E values per thread (E = 16 bytes of T, or 1 where
// rows are not 16-byte aligned).  Either a CTA per row, or (group <= 32) several rows per CTA.
template <typename T, bool kNorm, bool kRes, int E, int kChunks>
__global__ void __launch_bounds__(kChunks * E > 16 ? 512 : 1024)
    norm_quant_kernel(const __grid_constant__ NormQuantParams p) {
  const bool shared_cta = p.group <= 32;
  const int member = shared_cta ? threadIdx.x & (p.group - 1) : threadIdx.x;
  const int64_t row = shared_cta ? (int64_t)blockIdx.x * (blockDim.x / p.group) + threadIdx.x / p.group : blockIdx.x;
  const bool live = row < p.rows;
  Piece<T, E> x[kChunks], q[kRes ? kChunks : 1];
  float g[kChunks][E];
  float sum = 0.f;
  uint32_t a = 0u;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * p.group + member) * E, n = live ? p.width - at : 0;
    x[c] = load_piece<T, E>(static_cast<const T*>(p.x) + row * p.x_stride + at, n);
    if constexpr (kRes) q[c] = load_piece<T, E>(static_cast<const T*>(p.residual) + row * p.r_stride + at, n);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * p.group + member) * E;
    if (live && at < p.width) take_values<T, kNorm, kRes, E>(p, row, at, p.width - at, x[c], q[kRes ? c : 0], g[c], sum, a);
  }
  row_reduce(p.group, sum, a);
  float s, r, unit = 1.f;
  const bool numbers = row_step(a, s, r);
  if (kNorm) {
    // the same answer in every thread of a row; a warp of several rows takes it together
    const bool again = numbers && !(sum <= 3.4e38f);
    if (shared_cta ? __any_sync(0xffffffffu, again) : again) {
      // h of the row's other threads is written, and the first reduction read
      if (shared_cta) __syncwarp();
      else __syncthreads();
      float small = again && live ? sum_scaled<T, kRes>(p, row, member, p.group) : 0.f;
      row_reduce(p.group, small, a);
      if (again) {
        sum = small;
        unit = 5.421010862427522e-20f;
      }
    }
  }
  if (!live) return;
  if (member == 0) p.scales[row] = row_scale<kNorm>(a, numbers, s, sum, unit, p.width, p.eps);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * p.group + member) * E;
    if (at >= p.width) continue;
    uint32_t code[E];
#pragma unroll
    for (int i = 0; i < E; ++i) code[i] = numbers ? int8_code_byte(g[c][i], s, r) : 0u;
    store_codes<E>(p.codes + row * p.c_stride + at, p.width - at, code);
  }
}

// Rows wider than a CTA's registers: a CTA per row, the row read again (from L2) for the codes.
template <typename T, bool kNorm, bool kRes, int E>
__global__ void __launch_bounds__(kNormWideThreads) norm_quant_wide_kernel(const __grid_constant__ NormQuantParams p) {
  const int64_t row = blockIdx.x;
  float sum = 0.f;
  uint32_t a = 0u;
  for (int at = threadIdx.x * E; at < p.width; at += kNormWideThreads * E) {
    const int n = p.width - at;
    const Piece<T, E> x = load_piece<T, E>(static_cast<const T*>(p.x) + row * p.x_stride + at, n);
    Piece<T, E> q;
    if constexpr (kRes) q = load_piece<T, E>(static_cast<const T*>(p.residual) + row * p.r_stride + at, n);
    float g[E];
    take_values<T, kNorm, kRes, E>(p, row, at, n, x, q, g, sum, a);
  }
  row_reduce(kNormWideThreads, sum, a);
  float s, r, unit = 1.f;
  const bool numbers = row_step(a, s, r);
  if (kNorm && numbers && !(sum <= 3.4e38f)) {
    __syncthreads();
    sum = sum_scaled<T, kRes>(p, row, threadIdx.x, kNormWideThreads);
    row_reduce(kNormWideThreads, sum, a);
    unit = 5.421010862427522e-20f;
  }
  if (threadIdx.x == 0) p.scales[row] = row_scale<kNorm>(a, numbers, s, sum, unit, p.width, p.eps);
  const T* h = kRes ? static_cast<const T*>(p.h_out) + row * p.h_stride
                    : static_cast<const T*>(p.x) + row * p.x_stride;
  for (int at = threadIdx.x * E; at < p.width; at += kNormWideThreads * E) {
    const Piece<T, E> x = load_piece<T, E>(h + at, p.width - at);
    float g[E];
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = to_f32(x.v[i]);
    if constexpr (kNorm) {
      float w[E];
      load_weight<T, E>(p, at, p.width - at, w);
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] *= w[i];
    }
    uint32_t code[E];
#pragma unroll
    for (int i = 0; i < E; ++i) code[i] = numbers ? int8_code_byte(g[i], s, r) : 0u;
    store_codes<E>(p.codes + row * p.c_stride + at, p.width - at, code);
  }
}

}  // namespace qbsa
