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

#include "ptx_cluster.cuh"
#include "quantize.cuh"
#include "stream_plan.h"

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
  int weight_vec;  // weight on a 16-byte boundary
  int codes_vec;   // rows of codes on boundaries of a piece's codes
  int stages;  // rows in flight per CTA (norm_quant_stream_kernel)
  float eps;
  float square_limit;  // a row's sum of squares is taken again of scaled values above it
};

constexpr int kNormWideThreads = 1024;

// Shared memory of a row in norm_quant_stream_kernel: its 16-byte pieces, and one unit more where
// the row does not start on a unit's boundary.
template <typename T>
__host__ __device__ constexpr uint32_t stream_slot_bytes(int width, bool aligned) {
  return (width * static_cast<uint32_t>(sizeof(T)) + 15u) / 16u * 16u + (aligned ? 0u : 16u);
}

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

// Packed pairs: two lanes of f32 in one instruction, each rounded as the single operation.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// max(m, |a|, |b|), NaN if one of them is
__device__ __forceinline__ float amax2(float m, float2 v) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(v.x)), "f"(fabsf(v.y)));
  return d;
}
// Two neighbouring values of a 32-bit word
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 v) { return pack_bf16x2(v.x, v.y); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 v) {
  const __half2 h = __float22half2_rn(v);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

// E values of a row as they are stored: 16 bytes in words, or one value.
template <typename T, int E>
struct Piece {
  static_assert(E == 1 || E * sizeof(T) == 16, "a piece is one 16-byte load or one value");
  uint32_t w[E == 1 ? 1 : 4];
};

template <typename T>
__device__ __forceinline__ uint32_t bits_of(T v) {
  if constexpr (sizeof(T) == 4) return __float_as_uint(v);
  else {
    uint16_t u;
    memcpy(&u, &v, 2);
    return u;
  }
}
template <typename T>
__device__ __forceinline__ T value_of(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
  else {
    const uint16_t u = static_cast<uint16_t>(bits);
    T v;
    memcpy(&v, &u, 2);
    return v;
  }
}

// 16 bytes from byte `off` < 16 of two neighbouring 16-byte units.  off is the same in every thread
// of a row, so the branch does not diverge.
__device__ __forceinline__ void take_unaligned(const uint4& a, const uint4& b, uint32_t off, uint32_t (&w)[4]) {
  const uint32_t shift = (off & 3u) * 8u;
  auto cut = [&](uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, uint32_t v4) {
    w[0] = __funnelshift_r(v0, v1, shift);
    w[1] = __funnelshift_r(v1, v2, shift);
    w[2] = __funnelshift_r(v2, v3, shift);
    w[3] = __funnelshift_r(v3, v4, shift);
  };
  switch (off >> 2) {
    case 0: cut(a.x, a.y, a.z, a.w, b.x); break;
    case 1: cut(a.y, a.z, a.w, b.x, b.y); break;
    case 2: cut(a.z, a.w, b.x, b.y, b.z); break;
    default: cut(a.w, b.x, b.y, b.z, b.w); break;
  }
}

// E consecutive values, or the last n < E of a row with zeros after them.  E > 1: p is 16-byte
// aligned.  Volatile, so that the loads of a thread's pieces stay ahead of the first store.
template <typename T, int E>
__device__ __forceinline__ Piece<T, E> load_piece(const T* p, int n, bool aligned = true) {
  Piece<T, E> x;
  if constexpr (E == 1) {
    x.w[0] = n > 0 ? bits_of(p[0]) : 0u;
  } else if (aligned && n >= E) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3])
                 : "l"(p)
                 : "memory");
  } else {
    constexpr int kPer = 4 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) x.w[i / kPer] |= bits_of(p[i]) << (16 * (i % kPer));
  }
  return x;
}

// The norm's weights, read by every row: kept in L1.
template <typename T, int E>
__device__ __forceinline__ void load_weight(const NormQuantParams& p, int at, int n, float (&f)[E]) {
  if (E > 1 && n >= E && p.weight_vec) {
    if (sizeof(T) == 4 || p.weight_f32) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.weight) + at) + i);
        f[4 * i] = u.x;
        f[4 * i + 1] = u.y;
        f[4 * i + 2] = u.z;
        f[4 * i + 3] = u.w;
      }
    } else if constexpr (E == 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.weight) + at));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2<T>(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      f[i] = i >= n ? 0.f
             : p.weight_f32 ? __ldg(static_cast<const float*>(p.weight) + at + i)
                            : to_f32(static_cast<const T*>(p.weight)[at + i]);
  }
}

// Values 2i and 2i + 1 of a piece.
template <typename T, int E>
__device__ __forceinline__ float2 pair_of(const Piece<T, E>& x, int i) {
  if constexpr (sizeof(T) == 2) return unpack2<T>(x.w[i]);
  else return make_float2(__uint_as_float(x.w[2 * i]), __uint_as_float(x.w[2 * i + 1]));
}

template <typename T, int E>
__device__ __forceinline__ void store_piece(T* p, int n, const Piece<T, E>& x) {
  if constexpr (E == 1) {
    if (n > 0) p[0] = value_of<T>(x.w[0]);
  } else if (n >= E) {
    *reinterpret_cast<uint4*>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  } else {
    constexpr int kPer = 4 / sizeof(T);
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) p[i] = value_of<T>(x.w[i / kPer] >> (16 * (i % kPer)));
  }
}

template <int E>
__device__ __forceinline__ void store_codes(int8_t* p, int n, const uint32_t (&c)[E], bool vec = true) {
  if constexpr (E == 8) {
    if (vec && n >= E) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_low_bytes(c[0], c[1], c[2], c[3]),
                                                pack_low_bytes(c[4], c[5], c[6], c[7]));
      return;
    }
  }
  if constexpr (E == 4) {
    if (vec && n >= E) {
      *reinterpret_cast<uint32_t*>(p) = pack_low_bytes(c[0], c[1], c[2], c[3]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < n) p[i] = static_cast<int8_t>(c[i]);
}

// Sum (with a norm) and maximum over the threads of a row.  `a` is a magnitude's bits: unsigned order
// is the order of the magnitudes, with infinity and then NaN above every number.
template <bool kNorm>
__device__ __forceinline__ void row_reduce_group(int group, float& sum, uint32_t& a) {
  if (group == 32) {
    a = __reduce_max_sync(0xffffffffu, a);
    if constexpr (kNorm) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    return;
  }
  for (int o = group >> 1; o > 0; o >>= 1) {
    if constexpr (kNorm) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  }
}

// The same over a CTA.  Several calls of a kernel take the two buffers in turn, with one barrier each.
template <bool kNorm>
__device__ __forceinline__ void row_reduce_cta(float& sum, uint32_t& a, int buffer) {
  __shared__ float red_sum[2][32];
  __shared__ uint32_t red_max[2][32];
  row_reduce_group<kNorm>(32, sum, a);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) {
    if constexpr (kNorm) red_sum[buffer][threadIdx.x >> 5] = sum;
    red_max[buffer][threadIdx.x >> 5] = a;
  }
  __syncthreads();
  if constexpr (kNorm) sum = lane < warps ? red_sum[buffer][lane] : 0.f;
  a = lane < warps ? red_max[buffer][lane] : 0u;
  row_reduce_group<kNorm>(32, sum, a);
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
  const float root = __fsqrt_rn(__fdiv_rn(sum, static_cast<float>(width)) + eps * unit * unit);
  return __fdiv_rn(s, root) * unit;
}

// h (stored, or staged at shared-memory address h_stage), its square sum, g and its largest
// magnitude, of the E values at `at`.
template <typename T, bool kNorm, bool kRes, int E>
__device__ __forceinline__ void take_values(const NormQuantParams& p, int64_t row, int at, int n,
                                            const Piece<T, E>& x, const Piece<T, E>& q, float (&g)[E], float2& sum,
                                            float& a, uint32_t h_stage = 0) {
  float w[E];
  if constexpr (kNorm) load_weight<T, E>(p, at, n, w);
  if constexpr (E == 1) {
    g[0] = to_f32(value_of<T>(x.w[0]));
    if constexpr (kRes) {
      const T h = from_f32<T>(g[0] + to_f32(value_of<T>(q.w[0])));
      static_cast<T*>(p.h_out)[row * p.h_stride + at] = h;
      g[0] = to_f32(h);
    }
    if constexpr (kNorm) {
      sum.x = __fmaf_rn(g[0], g[0], sum.x);
      g[0] *= w[0];
    }
    a = amax2(a, make_float2(g[0], 0.f));
  } else {
    Piece<T, E> h;
    float2 f[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      f[i] = pair_of<T, E>(x, i);
      if constexpr (kRes) {
        f[i] = add2(f[i], pair_of<T, E>(q, i));
        if constexpr (sizeof(T) == 2) {
          h.w[i] = pack2<T>(f[i]);
          f[i] = unpack2<T>(h.w[i]);
        } else {
          h.w[2 * i] = __float_as_uint(f[i].x);
          h.w[2 * i + 1] = __float_as_uint(f[i].y);
        }
      }
    }
    if constexpr (kRes) {
      if (h_stage)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(h_stage), "r"(h.w[0]), "r"(h.w[1]), "r"(h.w[2]),
                     "r"(h.w[3])
                     : "memory");
      else
        store_piece<T, E>(static_cast<T*>(p.h_out) + row * p.h_stride + at, n, h);
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if constexpr (kNorm) {
        sum = fma2(f[i], f[i], sum);
        f[i] = mul2(f[i], make_float2(w[2 * i], w[2 * i + 1]));
      }
      a = amax2(a, f[i]);
      g[2 * i] = f[i].x;
      g[2 * i + 1] = f[i].y;
    }
  }
}

// Codes of E values: rint_half_even(RN(g / s)), with r = RN(1 / s).
//
// In general as int8_code_byte: both ends of each quotient's bracket are rounded, and the values
// are taken one by one if any of them differ.  That is rare for products with a weight (unless the
// weight is as short: 87 us for ones, 69 else, at 16384 x 5120), but not for 16-bit values alone
// (kFew): both x and a are short there, so that x / s often is a half-integer up to s's own rounding
// (about one value in a hundred of bf16), which sent most warps into the slow branch (65 us against 49
// at 16384 x 5120, both streamed with two pieces per thread).  Their quotient is taken with
// 1 / s in two parts instead, r and RN(r RN(1 - s r)): FMA(x, r, RN(x r_low)) equals RN(x / s) for
// every significand of x and a that bf16 or fp16 have and every ratio up to 2^8 (tested over all
// of them, on the host and here; beyond that the code is 0).  Powers of two only scale it while r_low
// is normal; above that, up to the limit of 1.2e27 for s, bf16 is tested in the same way.
template <bool kFew, int E>
__device__ __forceinline__ void codes_of(const float (&g)[E], float s, float r, uint32_t (&code)[E]) {
  const float2 magic = make_float2(12582912.0f, 12582912.0f);
  if (kFew && s < 1.2e27f) {
    const float r_low = __fmul_rn(__fmaf_rn(-s, r, 1.0f), r);
    if constexpr (E == 1) {
      code[0] = __float_as_uint(__fadd_rn(__fmaf_rn(g[0], r, __fmul_rn(g[0], r_low)), magic.x));
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 v = make_float2(g[2 * i], g[2 * i + 1]);
        const float2 n = add2(fma2(v, make_float2(r, r), mul2(v, make_float2(r_low, r_low))), magic);
        code[2 * i] = __float_as_uint(n.x);
        code[2 * i + 1] = __float_as_uint(n.y);
      }
    }
  } else if constexpr (E == 1) {
    code[0] = int8_code_byte(g[0], s, r);
  } else {
    const float2 lo = make_float2(kBracketLo, kBracketLo), hi = make_float2(kBracketHi, kBracketHi);
    bool open = false;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 y = mul2(make_float2(g[2 * i], g[2 * i + 1]), make_float2(r, r));
      const float2 l = fma2(y, lo, magic), h = fma2(y, hi, magic);
      open |= l.x != h.x;
      open |= l.y != h.y;
      code[2 * i] = __float_as_uint(l.x);
      code[2 * i + 1] = __float_as_uint(l.y);
    }
    if (open) {
#pragma unroll
      for (int i = 0; i < E; ++i) code[i] = int8_code_byte(g[i], s, r);
    }
  }
}

// Squares that overflow in f32 (a finite row above about 1e19): the sum again, of h * 2^-96.  |h| < 2^128
// and width <= 2^24 keep it at most 2^88.
constexpr float kOverflowUnit = 1.2621774483536189e-29f;  // 2^-96
template <typename T, bool kRes>
__device__ __noinline__ float sum_scaled(const NormQuantParams& p, int64_t row, int member, int step) {
  const T* h = kRes ? static_cast<const T*>(p.h_out) + row * p.h_stride
                    : static_cast<const T*>(p.x) + row * p.x_stride;
  float sum = 0.f;
  for (int i = member; i < p.width; i += step) {
    const float v = to_f32(h[i]) * kOverflowUnit;
    sum = __fmaf_rn(v, v, sum);
  }
  return sum;
}

// The codes of a thread's pieces of a row, piece c at c * step + member.
template <typename T, bool kNorm, int E, int kChunks>
__device__ __forceinline__ void write_codes(const NormQuantParams& p, int64_t row, int member, int step,
                                            const float (&g)[kChunks][E], bool numbers, float s, float r) {
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * step + member) * E;
    if (at < p.width) {
      uint32_t code[E] = {};
      if (numbers) codes_of<!kNorm && sizeof(T) == 2, E>(g[c], s, r, code);
      store_codes<E>(p.codes + row * p.c_stride + at, p.width - at, code, p.codes_vec);
    }
  }
}

// Such a row's (sum, unit) for row_scale: both are raised by the power of two that brings the larger of sum
// and eps to about 2^120.  The root is then between 2^47 and 2^61, so that s / root, with s below 2^122,
// does not overflow, and the unit at most 1, so that it loses no bits that the scale has.  (Choosing in
// row_scale whether s or the quotient takes the unit, or comparing sum + eps with the limit, cost every
// row 1 %: its thread is the one that the others of the CTA wait for.)
__device__ __noinline__ float2 raise_sum(float sum, float eps) {
  const float larger = fmaxf(sum, eps * kOverflowUnit * kOverflowUnit);
  const int exponent = static_cast<int>(__float_as_uint(larger) >> 23) - 127;  // -70 to 88
  const float f = __uint_as_float(static_cast<uint32_t>(127 + (120 - exponent) / 2) << 23);
  return make_float2(sum * f * f, kOverflowUnit * f);
}
__device__ __forceinline__ bool squares_overflow(bool numbers, float sum, float limit) {
  return numbers && !(sum <= limit);
}

// Narrow rows: p.group <= 32 threads per row, several rows per CTA, no barrier.  (A second row per
// group with its loads in flight together cost more registers than it hid latency: 10.5 us against
// 9.6 at 65536 x 128 bf16; one piece per thread in place of two: 11.8.)
template <typename T, bool kNorm, bool kRes, int E, int kChunks>
__global__ void __launch_bounds__(256) norm_quant_rows_kernel(const __grid_constant__ NormQuantParams p) {
  const int member = threadIdx.x & (p.group - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / p.group) + threadIdx.x / p.group;
  const bool live = row < p.rows;
  Piece<T, E> x[kChunks], q[kRes ? kChunks : 1];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * p.group + member) * E, n = live ? p.width - at : 0;
    x[c] = load_piece<T, E>(static_cast<const T*>(p.x) + row * p.x_stride + at, n);
    if constexpr (kRes) q[c] = load_piece<T, E>(static_cast<const T*>(p.residual) + row * p.r_stride + at, n);
  }
  float g[kChunks][E];
  float2 sum2 = make_float2(0.f, 0.f);
  float a_own = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * p.group + member) * E;
    if (live && at < p.width)
      take_values<T, kNorm, kRes, E>(p, row, at, p.width - at, x[c], q[kRes ? c : 0], g[c], sum2, a_own);
  }
  float sum = sum2.x + sum2.y;
  uint32_t a = __float_as_uint(a_own);
  row_reduce_group<kNorm>(p.group, sum, a);
  float s, r, unit = 1.f;
  const bool numbers = row_step(a, s, r);
  if constexpr (kNorm) {
    const bool again = squares_overflow(numbers, sum, p.square_limit);  // the same in a row's threads
    if (__any_sync(0xffffffffu, again)) {
      __syncwarp();  // h of the row's other threads is written
      float small = again && live ? sum_scaled<T, kRes>(p, row, member, p.group) : 0.f;
      row_reduce_group<kNorm>(p.group, small, a);
      const float2 raised = raise_sum(small, p.eps);  // in every lane: behind a second branch 1 % slower
      sum = again ? raised.x : sum;
      unit = again ? raised.y : unit;
    }
  }
  if (!live) return;
  if (member == 0) p.scales[row] = row_scale<kNorm>(a, numbers, s, sum, unit, p.width, p.eps);
  write_codes<T, kNorm, E, kChunks>(p, row, member, p.group, g, numbers, s, r);
}

// A CTA per row, the row in registers: kChunks pieces of E values per thread (E = 16 bytes of T,
// or 1 where rows are not 16-byte aligned).
template <typename T, bool kNorm, bool kRes, int E, int kChunks>
__global__ void __launch_bounds__(kChunks * E > 16 ? 640 : 1024)
    norm_quant_kernel(const __grid_constant__ NormQuantParams p) {
  const int member = threadIdx.x, step = blockDim.x;
  const int64_t row = blockIdx.x;
  Piece<T, E> x[kChunks], q[kRes ? kChunks : 1];
  float g[kChunks][E];
  float2 sum2 = make_float2(0.f, 0.f);
  float a_own = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * step + member) * E, n = p.width - at;
    x[c] = load_piece<T, E>(static_cast<const T*>(p.x) + row * p.x_stride + at, n);
    if constexpr (kRes) q[c] = load_piece<T, E>(static_cast<const T*>(p.residual) + row * p.r_stride + at, n);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int at = (c * step + member) * E;
    if (at < p.width)
      take_values<T, kNorm, kRes, E>(p, row, at, p.width - at, x[c], q[kRes ? c : 0], g[c], sum2, a_own);
  }
  float sum = sum2.x + sum2.y;
  uint32_t a = __float_as_uint(a_own);
  row_reduce_cta<kNorm>(sum, a, 0);
  float s, r, unit = 1.f;
  const bool numbers = row_step(a, s, r);
  if (kNorm && squares_overflow(numbers, sum, p.square_limit)) {  // the same in every thread
    __syncthreads();                               // h of the other threads is written
    sum = sum_scaled<T, kRes>(p, row, member, step);
    row_reduce_cta<kNorm>(sum, a, 1);
    const float2 raised = raise_sum(sum, p.eps);
    sum = raised.x;
    unit = raised.y;
  }
  if (member == 0) p.scales[row] = row_scale<kNorm>(a, numbers, s, sum, unit, p.width, p.eps);
  write_codes<T, kNorm, E, kChunks>(p, row, member, step, g, numbers, s, r);
}

// Many rows: the grid stays resident and each CTA takes every gridDim.x-th row, its next rows on
// their way into a ring in shared memory by bulk copies.  The reduction's barrier also says that
// every thread has read the row, so its stage is refilled right behind it.
// kAligned: rows are whole 16-byte pieces on 16-byte boundaries.  Otherwise a copy takes the 16-byte
// units that hold the row (with neighbouring bytes of the same tensor), pieces are cut out of two
// units each, and h goes out by its own units through shared memory; the tensor's first and last
// rows, whose units may reach beyond it, are read in place.  Rows do not overlap then.  (Value by value, coalesced,
// such rows ran at 20 % of HBM's bandwidth, bound by their instructions.)
// Four pieces per thread: what a row costs its warps beside its values (the reduction, the step) is
// shared by more values (42 us against 49 with two pieces for the quantiser alone at 16384 x 5120
// bf16, 382 against 395 at 65536 x 5120 with a residual; eight: 48 and 432).  Two for unaligned rows
// with a residual (134 against 143 at 16384 x 4097).
template <typename T, bool kNorm, bool kRes, int kChunks, bool kAligned>
__global__ void __launch_bounds__(kChunks == 4 ? 640 : 512, kChunks == 4 ? 1 : 2)
    norm_quant_stream_kernel(const __grid_constant__ NormQuantParams p) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kNormMaxStages];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, step = blockDim.x;
  const uint32_t row_bytes = static_cast<uint32_t>(p.width) * sizeof(T);
  const uint32_t slot = stream_slot_bytes<T>(p.width, kAligned), stage_bytes = slot * (kRes ? 2 : 1);
  const uint32_t base = smem_u32(ring);
  const uint32_t h_base = base + p.stages * stage_bytes;  // two rows of h (kRes, not kAligned)
  const T* const x = static_cast<const T*>(p.x);
  const T* const res = static_cast<const T*>(p.residual);
  auto offset = [](const T* t) { return static_cast<uint32_t>(reinterpret_cast<uint64_t>(t)) & 15u; };
  auto fetch = [&](int64_t row, int s) {  // thread 0
    const uint32_t bar = smem_u32(&full[s]), dst = base + s * stage_bytes;
    const T* const xr = x + row * p.x_stride;
    const T* const rr = kRes ? res + row * p.r_stride : nullptr;
    if constexpr (kAligned) {
      mbar_arrive_expect_tx(bar, stage_bytes);
      bulk_load(dst, xr, row_bytes, bar);
      if constexpr (kRes) bulk_load(dst + slot, rr, row_bytes, bar);
    } else {
      const bool inside = row != 0 && row != p.rows - 1;
      const uint32_t x_off = offset(xr), r_off = kRes ? offset(rr) : 0u;
      const uint32_t x_bytes = (x_off + row_bytes + 15u) & ~15u, r_bytes = kRes ? (r_off + row_bytes + 15u) & ~15u : 0u;
      mbar_arrive_expect_tx(bar, inside ? x_bytes + r_bytes : 0u);
      if (inside) {
        bulk_load(dst, reinterpret_cast<const uint8_t*>(xr) - x_off, x_bytes, bar);
        if constexpr (kRes) bulk_load(dst + slot, reinterpret_cast<const uint8_t*>(rr) - r_off, r_bytes, bar);
      }
    }
  };
  // piece `at` of the row t, whose slot is at `src`
  auto piece = [&](const T* t, bool inside, int at, uint32_t src) -> Piece<T, E> {
    Piece<T, E> v;
    const uint32_t unit = src + at * static_cast<uint32_t>(sizeof(T));
    if constexpr (kAligned) {
      const uint4 u = lds128(unit);
      v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    } else {
      const int n = p.width - at;
      if (!inside) return load_piece<T, E>(t + at, n, false);
      take_unaligned(lds128(unit), lds128(unit + 16), offset(t), v.w);
      if (n < E) {  // the row's last piece: zeros behind it
        constexpr int kPer = 4 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int have = n - i * kPer;
          v.w[i] = have >= kPer ? v.w[i] : have <= 0 ? 0u : v.w[i] & 0xffffu;
        }
      }
    }
    return v;
  };
  int fetched = 0;  // thread 0: rows asked for
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_mbar_init();
    for (; fetched < p.stages && blockIdx.x + (int64_t)fetched * gridDim.x < p.rows; ++fetched)
      fetch(blockIdx.x + (int64_t)fetched * gridDim.x, fetched);
  }
  __syncthreads();
  int it = 0, s = 0, phase = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    // a wait that runs out is reported; the CTA goes on, so that its barriers stay in step
    mbar_wait_hot(smem_u32(&full[s]), phase, &abort_flag);
    float g[kChunks][E];
    float2 sum2 = make_float2(0.f, 0.f);
    float a_own = 0.f;
    const uint32_t src = base + s * stage_bytes, h_row = h_base + (it & 1) * slot;
    const bool inside = row != 0 && row != p.rows - 1;
    const T* const xr = x + row * p.x_stride;
    const T* const rr = kRes ? res + row * p.r_stride : nullptr;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int at = (c * step + tid) * E;
      if (at < p.width) {
        const Piece<T, E> v = piece(xr, inside, at, src);
        Piece<T, E> q;
        if constexpr (kRes) q = piece(rr, inside, at, src + slot);
        take_values<T, kNorm, kRes, E>(p, row, at, p.width - at, v, q, g[c], sum2, a_own,
                                       kRes && !kAligned ? h_row + at * static_cast<uint32_t>(sizeof(T)) : 0u);
      }
    }
    float sum = sum2.x + sum2.y;
    uint32_t a = __float_as_uint(a_own);
    row_reduce_cta<kNorm>(sum, a, it & 1);
    if (tid == 0) {
      const int64_t next = row + (int64_t)p.stages * gridDim.x;
      if (next < p.rows && !*static_cast<volatile int*>(&abort_flag)) {
        fetch(next, s);
        ++fetched;
      }
    }
    if (++s == p.stages) {
      s = 0;
      phase ^= 1;
    }
    if constexpr (kRes && !kAligned) {
      // h by its 16-byte units: unit j holds the row's bytes from 16 j - off on
      T* const h = static_cast<T*>(p.h_out) + row * p.h_stride;
      const uint32_t off = offset(h);
      for (int j = tid; 16u * j < off + row_bytes; j += step) {
        const int first = 16 * j - static_cast<int>(off);  // byte of the row
        if (first >= 0 && first + 16 <= static_cast<int>(row_bytes)) {
          uint32_t w[4];
          if (off == 0) {
            const uint4 u = lds128(h_row + first);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
          } else {
            take_unaligned(lds128(h_row + 16 * (j - 1)), lds128(h_row + 16 * j), 16u - off, w);
          }
          *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(h) + first) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          const T* staged = reinterpret_cast<const T*>(ring + (h_row - base));
          const int from = max(first, 0) / static_cast<int>(sizeof(T));
          const int to = min(first + 16, static_cast<int>(row_bytes)) / static_cast<int>(sizeof(T));
          for (int i = from; i < to; ++i) h[i] = staged[i];
        }
      }
    }
    float width, r, unit = 1.f;
    const bool numbers = row_step(a, width, r);
    if (kNorm && squares_overflow(numbers, sum, p.square_limit)) {  // the same in every thread
      __syncthreads();
      sum = sum_scaled<T, kRes>(p, row, tid, step);
      row_reduce_cta<kNorm>(sum, a, it & 1);
      const float2 raised = raise_sum(sum, p.eps);
      sum = raised.x;
      unit = raised.y;
      __syncthreads();
    }
    if (tid == 0) p.scales[row] = row_scale<kNorm>(a, numbers, width, sum, unit, p.width, p.eps);
    write_codes<T, kNorm, E, kChunks>(p, row, tid, step, g, numbers, width, r);
  }
  // let the copies still in flight land (matters only after a wait that ran out)
  if (tid == 0)
    for (int q = max(0, fetched - p.stages); q < fetched; ++q)
      mbar_wait_drain(smem_u32(&full[q % p.stages]), (q / p.stages) & 1);
}

// Rows wider than a CTA's registers: a CTA per row, the row read again (from L2) for the codes.
template <typename T, bool kNorm, bool kRes, int E>
__global__ void __launch_bounds__(kNormWideThreads) norm_quant_wide_kernel(const __grid_constant__ NormQuantParams p) {
  const int64_t row = blockIdx.x;
  float2 sum2 = make_float2(0.f, 0.f);
  float a_own = 0.f;
  for (int at = threadIdx.x * E; at < p.width; at += kNormWideThreads * E) {
    const int n = p.width - at;
    const Piece<T, E> x = load_piece<T, E>(static_cast<const T*>(p.x) + row * p.x_stride + at, n);
    Piece<T, E> q;
    if constexpr (kRes) q = load_piece<T, E>(static_cast<const T*>(p.residual) + row * p.r_stride + at, n);
    float g[E];
    take_values<T, kNorm, kRes, E>(p, row, at, n, x, q, g, sum2, a_own);
  }
  float sum = sum2.x + sum2.y;
  uint32_t a = __float_as_uint(a_own);
  row_reduce_cta<kNorm>(sum, a, 0);
  float s, r, unit = 1.f;
  const bool numbers = row_step(a, s, r);
  if (kNorm && squares_overflow(numbers, sum, p.square_limit)) {
    __syncthreads();
    sum = sum_scaled<T, kRes>(p, row, threadIdx.x, kNormWideThreads);
    row_reduce_cta<kNorm>(sum, a, 1);
    const float2 raised = raise_sum(sum, p.eps);
    sum = raised.x;
    unit = raised.y;
  }
  if (threadIdx.x == 0) p.scales[row] = row_scale<kNorm>(a, numbers, s, sum, unit, p.width, p.eps);
  const T* h = kRes ? static_cast<const T*>(p.h_out) + row * p.h_stride
                    : static_cast<const T*>(p.x) + row * p.x_stride;
  for (int at = threadIdx.x * E; at < p.width; at += kNormWideThreads * E) {
    const Piece<T, E> x = load_piece<T, E>(h + at, p.width - at);
    float g[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if constexpr (E == 1) g[0] = to_f32(value_of<T>(x.w[0]));
      else g[i] = i & 1 ? pair_of<T, E>(x, i / 2).y : pair_of<T, E>(x, i / 2).x;
    }
    if constexpr (kNorm) {
      float w[E];
      load_weight<T, E>(p, at, p.width - at, w);
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] *= w[i];
    }
    uint32_t code[E] = {};
    if (numbers) codes_of<!kNorm && sizeof(T) == 2, E>(g, s, r, code);
    store_codes<E>(p.codes + row * p.c_stride + at, p.width - at, code, p.codes_vec);
  }
}

}  // namespace qbsa
