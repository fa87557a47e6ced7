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

// The pair forms below use the packed f32x2 instructions (aqfq_device.cuh): two
// elements per FMA; only exponential, reciprocal and selection are per element.
__device__ __forceinline__ f2 pair(float c) { return mk2(c, c); }
__device__ __forceinline__ f2 ex2_pair(f2 v) { return mk2(ex2_approx(lo2(v)), ex2_approx(hi2(v))); }
__device__ __forceinline__ f2 rcp_pair(f2 v) { return mk2(rcp_approx(lo2(v)), rcp_approx(hi2(v))); }
// 1 / (1 + 2^z)
__device__ __forceinline__ f2 logistic2(f2 z) { return rcp_pair(add2(ex2_pair(z), pair(1.0f))); }

// Phi(x), the standard normal distribution function, and g = exp(-x^2 / 2):
// erfc(z) = (a1 t + ... + a5 t^5) exp(-z^2), t = 1 / (1 + p z), z >= 0, with
// an absolute error below 1.5e-7 (Abramowitz and Stegun, Handbook of
// Mathematical Functions, formula 7.1.26); z = |x| / sqrt 2, so that its
// exponential is the one the derivative needs.  The coefficients are halved: the
// upper tail is erfc / 2.
__device__ __forceinline__ f2 normal_cdf(f2 x, f2& g) {
  const f2 a = x & 0x7FFFFFFF7FFFFFFFull;
  const f2 t = rcp_pair(fma2(pair(0.3275911f * 0.70710678f), a, pair(1.0f)));
  g = ex2_pair(mul2(mul2(x, x), pair(-0.5f * kLog2e)));
  f2 p = fma2(pair(0.5f * 1.061405429f), t, pair(0.5f * -1.453152027f));
  p = fma2(p, t, pair(0.5f * 1.421413741f));
  p = fma2(p, t, pair(0.5f * -0.284496736f));
  p = fma2(p, t, pair(0.5f * 0.254829592f));
  const f2 q = mul2(mul2(p, t), g);  // Phi(-|x|)
  const f2 c = sub2(pair(1.0f), q);
  return mk2(lo2(x) < 0.0f ? lo2(q) : lo2(c), hi2(x) < 0.0f ? hi2(q) : hi2(c));
}

constexpr float kTanhC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;
// (1 + tanh u) / 2 = sigmoid(2 u), u = sqrt(2/pi) (x + a x^3)
__device__ __forceinline__ f2 tanh_gate(f2 x) {
  const f2 k = fma2(mul2(x, x), pair(-2.0f * kTanhC * kLog2e * kTanhA), pair(-2.0f * kTanhC * kLog2e));
  return logistic2(mul2(x, k));
}

template <int ACT>
__device__ __forceinline__ f2 act2(f2 x) {
  if constexpr (ACT == AQFQ_ACT_RELU) {
    return mk2(lo2(x) < 0.0f ? 0.0f : lo2(x), hi2(x) < 0.0f ? 0.0f : hi2(x));  // a NaN stays
  } else if constexpr (ACT == AQFQ_ACT_GELU) {
    f2 g;
    return mul2(x, normal_cdf(x, g));
  } else if constexpr (ACT == AQFQ_ACT_GELU_TANH) {
    return mul2(x, tanh_gate(x));
  } else if constexpr (ACT == AQFQ_ACT_SILU) {
    return mul2(x, logistic2(mul2(x, pair(-kLog2e))));
  } else {
    return x;
  }
}

__device__ __forceinline__ float relu_slope(float x) { return x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x); }

// value and derivative
template <int ACT>
__device__ __forceinline__ f2 act_fd2(f2 x, f2& d) {
  if constexpr (ACT == AQFQ_ACT_RELU) {
    d = mk2(relu_slope(lo2(x)), relu_slope(hi2(x)));
    return act2<ACT>(x);
  } else if constexpr (ACT == AQFQ_ACT_GELU) {
    f2 g;
    const f2 c = normal_cdf(x, g);
    d = fma2(mul2(x, pair(0.3989422804f)), g, c);  // Phi + x phi
    return mul2(x, c);
  } else if constexpr (ACT == AQFQ_ACT_GELU_TANH) {
    const f2 s = tanh_gate(x);
    // d/dx [x s(2u)] = s + x s (1 - s) 2 u'; s (1 - s) is 0 beyond |x| = 16, where x is
    // clamped so that u' stays finite
    const f2 c = mk2(fminf(fmaxf(lo2(x), -16.0f), 16.0f), fminf(fmaxf(hi2(x), -16.0f), 16.0f));
    const f2 u = fma2(mul2(c, c), pair(6.0f * kTanhC * kTanhA), pair(2.0f * kTanhC));
    d = fma2(mul2(mul2(c, s), sub2(pair(1.0f), s)), u, s);
    return mul2(x, s);
  } else if constexpr (ACT == AQFQ_ACT_SILU) {
    const f2 s = logistic2(mul2(x, pair(-kLog2e)));
    d = mul2(s, fma2(x, sub2(pair(1.0f), s), pair(1.0f)));
    return mul2(x, s);
  } else {
    d = pair(1.0f);
    return x;
  }
}

// the same for V values (even)
template <int ACT, int V>
__device__ __forceinline__ void act_all(float (&v)[V]) {
  if constexpr (ACT != AQFQ_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const f2 y = act2<ACT>(mk2(v[i], v[i + 1]));
      v[i] = lo2(y), v[i + 1] = hi2(y);
    }
  }
}
// v *= act'(p), p = act(p)
template <int ACT, int V>
__device__ __forceinline__ void slope_all(float (&p)[V], float (&v)[V]) {
  if constexpr (ACT != AQFQ_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      f2 d;
      const f2 y = act_fd2<ACT>(mk2(p[i], p[i + 1]), d);
      const f2 w = mul2(mk2(v[i], v[i + 1]), d);
      p[i] = lo2(y), p[i + 1] = hi2(y);
      v[i] = lo2(w), v[i + 1] = hi2(w);
    }
  }
}

// the activation chosen at run time (uniform)
template <int V>
__device__ __forceinline__ void act_apply(int act, float (&v)[V]) {
  switch (act) {
    case AQFQ_ACT_RELU: act_all<AQFQ_ACT_RELU>(v); break;
    case AQFQ_ACT_GELU: act_all<AQFQ_ACT_GELU>(v); break;
    case AQFQ_ACT_GELU_TANH: act_all<AQFQ_ACT_GELU_TANH>(v); break;
    case AQFQ_ACT_SILU: act_all<AQFQ_ACT_SILU>(v); break;
    default: break;
  }
}
// v *= act'(p)
template <int V>
__device__ __forceinline__ void slope_apply(int act, float (&p)[V], float (&v)[V]) {
  switch (act) {
    case AQFQ_ACT_RELU: slope_all<AQFQ_ACT_RELU>(p, v); break;
    case AQFQ_ACT_GELU: slope_all<AQFQ_ACT_GELU>(p, v); break;
    case AQFQ_ACT_GELU_TANH: slope_all<AQFQ_ACT_GELU_TANH>(p, v); break;
    case AQFQ_ACT_SILU: slope_all<AQFQ_ACT_SILU>(p, v); break;
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
  f2 v[2];
  if (d.fast) {
    v[0] = mdiv2(mk2(x[0], x[1]), d), v[1] = mdiv2(mk2(x[2], x[3]), d);
  } else {  // a quotient may leave the grid here (a rounded subnormal scale)
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = __fdiv_rn(x[i], d.s);
      if (fmt == AQFQ_INT8) q[i] = fminf(fmaxf(q[i], -127.0f), 127.0f);
    }
    v[0] = mk2(q[0], q[1]), v[1] = mk2(q[2], q[3]);
  }
  if (fmt == AQFQ_INT8) {
    // |x / s| <= 127 (1 + 2^-23) rounds to at most 127: no clamp.  The sum with 1.5 * 2^23
    // holds the rounded integer in its low bits.
    const f2 a = add2(v[0], pair(12582912.0f)), b = add2(v[1], pair(12582912.0f));
    return __byte_perm(__byte_perm(uint32_t(a), uint32_t(a >> 32), 0x0040),
                       __byte_perm(uint32_t(b), uint32_t(b >> 32), 0x0040), 0x5410);
  }
  return cvt_e4m3x2(hi2(v[0]), lo2(v[0])) | (cvt_e4m3x2(hi2(v[1]), lo2(v[1])) << 16);
}

// four stored values (code * s, rounded to binary32)
__device__ __forceinline__ void ckpt_values4(uint32_t c, float s, int fmt, float* v) {
  f2 a, b;
  if (fmt == AQFQ_INT8) {
    // byte + 128 in the low mantissa bits of 2^23: exact
    const uint32_t u = c ^ 0x80808080u;
    a = mk2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650)),
            __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7651)));
    b = mk2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7652)),
            __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7653)));
    a = sub2(a, pair(8388736.0f)), b = sub2(b, pair(8388736.0f));
  } else {
    const float2 p = dec_e4m3x2(c & 0xFFFFu), q = dec_e4m3x2(c >> 16);
    a = mk2(p.x, p.y), b = mk2(q.x, q.y);
  }
  a = mul2(a, pair(s)), b = mul2(b, pair(s));
  v[0] = lo2(a), v[1] = hi2(a), v[2] = lo2(b), v[3] = hi2(b);
}

// bits of the largest |x|, at or above those of infinity when one is NaN
template <int V>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[V]) {
  static_assert(V % 2 == 0, "pairs");
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[i]), "f"(v[i + 1]));
  return __float_as_uint(m) & 0x7FFFFFFFu;
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

// V consecutive elements as they are in memory (V = 8: rows allow 16-byte accesses;
// V = 1: any row), so that loads can be in flight before anything is converted
template <typename T, int V>
struct Vec {
  static constexpr int W = V == 1 ? 1 : V * int(sizeof(T)) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 2) w[0] = reinterpret_cast<const uint16_t*>(p)[0];
      else w[0] = __float_as_uint(*reinterpret_cast<const float*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) ld_stream_v4(reinterpret_cast<const uint32_t*>(p) + i, w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void get(float* v) const {
    if constexpr (V == 1) {
      v[0] = sizeof(T) == 2 ? __uint_as_float(w[0] << 16) : __uint_as_float(w[0]);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[2 * i] = bf_lo(w[i]), v[2 * i + 1] = bf_hi(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ void put(T* p, const float* v) {
  if constexpr (V == 1) {
    from_f(v[0], *p);
  } else {
    float t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = v[i];
    store_row(p, true, V, t);
  }
}
template <int V>
struct CodeVec {
  uint32_t w[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (V == 8) {
      asm("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
      w[0] = __ldg(p);
    }
  }
  __device__ __forceinline__ void values(float s, int fmt, float* v) const {
    if constexpr (V == 8) {
      ckpt_values4(w[0], s, fmt, v);
      ckpt_values4(w[1], s, fmt, v + 4);
    } else {
      float t[4];
      ckpt_values4(w[0], s, fmt, t);
      v[0] = t[0];
    }
  }
};

// the 8-bit checkpoint of a warp's columns from col0 on; v: the lane's values,
// zero beyond the row.  V = 8: a group is a run of lanes; V = 1: one, two or four
// whole vectors (NV is a multiple of four or a vector a whole group).
template <int V, int NV>
__device__ __forceinline__ void ckpt_row(const Ckpt& c, int64_t r, int64_t cols, int64_t col0,
                                         const float* v) {
  const int lane = threadIdx.x & 31;
  uint8_t* codes = c.codes + r * cols;
  float* scale = c.scale + r * c.groups;
  if constexpr (V == 8) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = col0 + (j * 32 + lane) * 8;
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[j * 8 + i];
      uint32_t m = amax_bits(t);
      for (int o = 1; o < (1 << (c.lg - 3)); o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const Divisor d = make_divisor(ckpt_scale(m, c.fmt));
      if (col < cols) {
        st_64(codes + col, ckpt_codes4(v + j * 8, d, c.fmt), ckpt_codes4(v + j * 8 + 4, d, c.fmt));
        if ((col & ((1 << c.lg) - 1)) == 0) scale[col >> c.lg] = d.s;
      }
    }
  } else {
    static_assert(NV % 4 == 0, "groups of four vectors");
#pragma unroll
    for (int j = 0; j < NV; j += 4) {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m[i] = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j + i]) & 0x7FFFFFFFu);
      if (c.lg > 5) m[0] = m[1] = max(m[0], m[1]), m[2] = m[3] = max(m[2], m[3]);
      if (c.lg > 6) m[0] = m[1] = m[2] = m[3] = max(m[0], m[2]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t col = col0 + (j + i) * 32 + lane;
        const Divisor d = make_divisor(ckpt_scale(m[i], c.fmt));
        if (col < cols) {
          const float one[4] = {v[j + i], 0.0f, 0.0f, 0.0f};
          codes[col] = uint8_t(ckpt_codes4(one, d, c.fmt));
          if ((col & ((1 << c.lg) - 1)) == 0) scale[col >> c.lg] = d.s;
        }
      }
    }
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
