// aqfq_layer.cuh -- device-side pieces shared by the layer kernels (layer norm,
// 8-bit activation checkpoints, linear epilogues): element access for BF16 and
// binary32 rows, the activations with their derivatives, and the checkpoint's
// quantizer.  Everything is computed in binary32; a value is rounded to BF16
// once, when it is stored.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "aqfq.h"
#include "aqfq_device.cuh"

namespace aqfq {
namespace layer {

// ---------------------------------------------------------------------------
// rows of BF16 or binary32 elements
// ---------------------------------------------------------------------------
struct bf16 {
  uint16_t b;
};
__device__ __forceinline__ float to_f(bf16 v) { return __uint_as_float(uint32_t(v.b) << 16); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void from_f(float v, bf16& o) { o.b = uint16_t(pack_bf16x2(0.0f, v)); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }

// V consecutive elements at p as binary32.  vec: p is aligned to min(16, the
// V elements' bytes) and all V lie in the row; else the first n of them are
// read one by one and the rest are zero.
template <int V>
__device__ __forceinline__ void load_row(const bf16* p, bool vec, int n, float (&v)[V]) {
  if (vec) {
    if constexpr (V == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      v[0] = bf_lo(w.x), v[1] = bf_hi(w.x), v[2] = bf_lo(w.y), v[3] = bf_hi(w.y);
      v[4] = bf_lo(w.z), v[5] = bf_hi(w.z), v[6] = bf_lo(w.w), v[7] = bf_hi(w.w);
    } else {
      static_assert(V == 4, "4 or 8 elements");
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[0] = bf_lo(w.x), v[1] = bf_hi(w.x), v[2] = bf_lo(w.y), v[3] = bf_hi(w.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? to_f(p[i]) : 0.0f;
  }
}
template <int V>
__device__ __forceinline__ void load_row(const float* p, bool vec, int n, float (&v)[V]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 w = *reinterpret_cast<const float4*>(p + i);
      v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}
template <int V>
__device__ __forceinline__ void store_row(bf16* p, bool vec, int n, const float (&v)[V]) {
  if (vec) {
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[1], v[0]), pack_bf16x2(v[3], v[2]),
                                                pack_bf16x2(v[5], v[4]), pack_bf16x2(v[7], v[6]));
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[1], v[0]), pack_bf16x2(v[3], v[2]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) from_f(v[i], p[i]);
  }
}
template <int V>
__device__ __forceinline__ void store_row(float* p, bool vec, int n, const float (&v)[V]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Whether V-element accesses at multiples of V in rows of `ld` elements are
// aligned (host side; NULL tensors pass).
template <int V>
inline bool rows_aligned(const void* p, int64_t ld, int esize) {
  const uintptr_t a = uintptr_t(V * esize < 16 ? V * esize : 16);
  return !p || ((reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0 && (ld * esize) % int64_t(a) == 0);
}

// ---------------------------------------------------------------------------
// activations.  Exponentials and reciprocals are the hardware approximations
// (relative error about 2^-22), far below the BF16 rounding of what is stored.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.0f + ex2_approx(-kLog2e * x));
}

// Phi(x), the standard normal distribution function, and g = exp(-x^2 / 2):
// erfc(z) = (a1 t + ... + a5 t^5) exp(-z^2), t = 1 / (1 + p z), z >= 0, with
// an absolute error below 1.5e-7 (Abramowitz and Stegun, Handbook of
// Mathematical Functions, formula 7.1.26); z = |x| / sqrt 2, so that its
// exponential is the one the derivative needs.
__device__ __forceinline__ float normal_cdf(float x, float& g) {
  const float a = fabsf(x);
  const float t = rcp_approx(fmaf(0.3275911f * 0.70710678f, a, 1.0f));
  g = ex2_approx(x * x * (-0.5f * kLog2e));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float q = 0.5f * p * t * g;  // upper tail Phi(-|x|)
  return x < 0.0f ? q : 1.0f - q;
}

constexpr float kTanhC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_f(float x) {
  if constexpr (ACT == AQFQ_ACT_RELU) {
    return x < 0.0f ? 0.0f : x;  // a NaN stays
  } else if constexpr (ACT == AQFQ_ACT_GELU) {
    float g;
    return x * normal_cdf(x, g);
  } else if constexpr (ACT == AQFQ_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = sigmoid(2 u)
    return x * sigmoid(2.0f * kTanhC * x * fmaf(kTanhA * x, x, 1.0f));
  } else if constexpr (ACT == AQFQ_ACT_SILU) {
    return x * sigmoid(x);
  } else {
    return x;
  }
}

// value and derivative
template <int ACT>
__device__ __forceinline__ float act_fd(float x, float& d) {
  if constexpr (ACT == AQFQ_ACT_RELU) {
    d = x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);
    return x < 0.0f ? 0.0f : x;
  } else if constexpr (ACT == AQFQ_ACT_GELU) {
    float g;
    const float c = normal_cdf(x, g);
    d = fmaf(x * 0.3989422804f, g, c);  // Phi + x phi
    return x * c;
  } else if constexpr (ACT == AQFQ_ACT_GELU_TANH) {
    const float s = sigmoid(2.0f * kTanhC * x * fmaf(kTanhA * x, x, 1.0f));
    // d/dx [x s(2u)] = s + x s (1 - s) 2 u'; s (1 - s) is 0 beyond |x| = 16, where x is
    // clamped so that u' stays finite
    const float c = fminf(fmaxf(x, -16.0f), 16.0f);
    d = fmaf(c * s * (1.0f - s), 2.0f * kTanhC * fmaf(3.0f * kTanhA * c, c, 1.0f), s);
    return x * s;
  } else if constexpr (ACT == AQFQ_ACT_SILU) {
    const float s = sigmoid(x);
    d = s * fmaf(x, 1.0f - s, 1.0f);
    return x * s;
  } else {
    d = 1.0f;
    return x;
  }
}

// the same for V values, the activation chosen at run time (uniform)
template <int V>
__device__ __forceinline__ void act_apply(int act, float (&v)[V]) {
  switch (act) {
    case AQFQ_ACT_RELU:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_f<AQFQ_ACT_RELU>(v[i]);
      break;
    case AQFQ_ACT_GELU:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_f<AQFQ_ACT_GELU>(v[i]);
      break;
    case AQFQ_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_f<AQFQ_ACT_GELU_TANH>(v[i]);
      break;
    case AQFQ_ACT_SILU:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_f<AQFQ_ACT_SILU>(v[i]);
      break;
    default:
      break;
  }
}
template <int ACT, int V>
__device__ __forceinline__ void slope_one(const float (&p)[V], float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float d;
    act_fd<ACT>(p[i], d);
    v[i] *= d;
  }
}
// v *= act'(p)
template <int V>
__device__ __forceinline__ void slope_apply(int act, const float (&p)[V], float (&v)[V]) {
  switch (act) {
    case AQFQ_ACT_RELU: slope_one<AQFQ_ACT_RELU>(p, v); break;
    case AQFQ_ACT_GELU: slope_one<AQFQ_ACT_GELU>(p, v); break;
    case AQFQ_ACT_GELU_TANH: slope_one<AQFQ_ACT_GELU_TANH>(p, v); break;
    case AQFQ_ACT_SILU: slope_one<AQFQ_ACT_SILU>(p, v); break;
    default: break;
  }
}

// ---------------------------------------------------------------------------
// 8-bit checkpoint.  Per group: amax as the bits of |x| (a NaN or an infinity
// has bits >= 0x7F800000, above every finite value), s = amax / qmax, code =
// grid(x / s) with the IEEE quotient (Markstein's correction on the reciprocal
// where s is in its range, else the division itself).
// ---------------------------------------------------------------------------
struct Ckpt {
  uint8_t* codes;  // [rows, cols]
  float* scale;    // [rows, groups]
  int64_t groups;  // per row
  int fmt;         // AQFQ_INT8 or AQFQ_FP8_E4M3
  int lg;          // log2 of the group
};

__device__ __forceinline__ float ckpt_scale(uint32_t amax_bits, int fmt) {
  if (amax_bits >= 0x7F800000u) return __int_as_float(0x7FC00000);
  return __fdiv_rn(__uint_as_float(amax_bits), fmt == AQFQ_INT8 ? 127.0f : 448.0f);
}

// four codes of x / s, element 0 in the low byte; a scale of zero or NaN gives zeros
__device__ __forceinline__ uint32_t ckpt_codes4(const float* x, const Divisor& d, int fmt) {
  if (!(d.s > 0.0f)) return 0u;
  float v[4];
  if (d.fast) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mdiv(x[i], d);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fdiv_rn(x[i], d.s);
  }
  if (fmt == AQFQ_INT8) {
    const IntRange r{-127.0f, 127.0f};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) int_round(v[i], r, c[i]);
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  }
  return cvt_e4m3x2(v[1], v[0]) | (cvt_e4m3x2(v[3], v[2]) << 16);
}

// four stored values (code * s, rounded to binary32)
__device__ __forceinline__ void ckpt_values4(uint32_t c, float s, int fmt, float* v) {
  if (fmt == AQFQ_INT8) {
    // byte + 128 in the low mantissa bits of 2^23: exact
    const uint32_t u = c ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __fmul_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650 + i)) - 8388736.0f, s);
  } else {
    const float2 a = dec_e4m3x2(c & 0xFFFFu), b = dec_e4m3x2(c >> 16);
    v[0] = __fmul_rn(a.x, s), v[1] = __fmul_rn(a.y, s);
    v[2] = __fmul_rn(b.x, s), v[3] = __fmul_rn(b.y, s);
  }
}

template <int V>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// V code bytes at p (vec: aligned to V bytes and all in the row)
template <int V>
__device__ __forceinline__ void store_bytes(uint8_t* p, bool vec, int n, const uint32_t (&w)[V / 4]) {
  if (vec) {
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
  }
}
template <int V>
__device__ __forceinline__ void load_bytes(const uint8_t* p, bool vec, int n, uint32_t (&w)[V / 4]) {
  if (vec) {
    if constexpr (V == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) w[i >> 2] |= uint32_t(p[i]) << (8 * (i & 3));
  }
}

// ---------------------------------------------------------------------------
// host side: argument checks shared by the entry points
// ---------------------------------------------------------------------------
inline bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int esize(int dtype) { return dtype == AQFQ_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == AQFQ_BF16 || dtype == AQFQ_F32; }

// a [rows, cols] view with rows `ld` elements apart: sizes and addresses
// within 2^62 bytes
inline bool view_ok(int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0 || cols > 0x7FFFFFF0ll || rows > (int64_t(1) << 40)) return false;
  if (rows > 1 && ld < cols) return false;
  return ld >= 0 && (rows == 0 || ld <= (int64_t(1) << 59) / rows);
}

// fills c from the caller's struct; need: the buffers hold elements
inline aqfq_status make_ckpt(const aqfq_ckpt8* in, int64_t rows, int64_t cols, Ckpt& c) {
  if (!in) return AQFQ_ERR_NULL;
  if (in->fmt != AQFQ_INT8 && in->fmt != AQFQ_FP8_E4M3) return AQFQ_ERR_UNSUPPORTED;
  if (in->group != 32 && in->group != 64 && in->group != 128) return AQFQ_ERR_UNSUPPORTED;
  if (rows > 0 && cols > 0 && (!in->codes || !in->scale)) return AQFQ_ERR_NULL;
  if (!al(in->scale, 4)) return AQFQ_ERR_ALIGN;
  c.codes = static_cast<uint8_t*>(in->codes);
  c.scale = in->scale;
  c.fmt = in->fmt;
  c.lg = in->group == 32 ? 5 : in->group == 64 ? 6 : 7;
  c.groups = (cols + in->group - 1) / in->group;
  return AQFQ_OK;
}

inline bool act_ok(int act) { return act >= AQFQ_ACT_NONE && act <= AQFQ_ACT_SILU; }

// Column sums [rows, cols] -> partial sums of at most kMaxParts row slices
// (two per SM), then the sum of the slices in order.
constexpr int kMaxParts = 304;

// out[c] (+)= sum over p < parts of part[p * cols + c], in a fixed order; out2 /
// part2 likewise when out2 is not NULL (ckpt8.cu)
cudaError_t launch_part_sums(const float* part, const float* part2, int parts, int64_t cols,
                             float* out, float* out2, int accumulate, cudaStream_t st);

}  // namespace layer
}  // namespace aqfq
