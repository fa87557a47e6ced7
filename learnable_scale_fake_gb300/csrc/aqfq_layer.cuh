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
// (relative error about 2^-22; an exponential's argument is rounded too, 2^-23 of it).
// Down to x = -13, where gelu leaves binary32's normal range, each value and derivative
// keeps a relative error (of the derivative: of its two terms) below 2^-15, against the
// 2^-8 of a stored BF16 value.
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

// Phi(x), the standard normal distribution function, and g = exp(-x^2 / 2).  The upper
// tail: Phi(-z) = g R(t), t = 1 / (1 + c z), z >= 0, R a polynomial without a constant (so that
// it falls like 1 / z).  Its coefficients and c minimise the largest relative error over
// 0 <= z <= 14 (a linear program over 1600 points), as evaluated in binary32:
//   degree 8  4e-7   derivatives, whose column sums are stored in binary32
//   degree 6  4e-6   values that are stored in BF16 (2^-8): 8192 x 8192 recomputed
//                    46 us, with degree 8 51
// A bound on the absolute error would not do: gelu(x) for x < -4 is this tail alone.
// (The exponential adds its argument's rounding, 2^-23 of x^2 / 2.)
template <int DEGREE>
__device__ __forceinline__ f2 normal_cdf(f2 x, f2& g) {
  static_assert(DEGREE == 6 || DEGREE == 8, "fitted degrees");
  const f2 a = x & 0x7FFFFFFF7FFFFFFFull;
  const f2 t = rcp_pair(fma2(pair(DEGREE == 8 ? 0.305f : 0.308f), a, pair(1.0f)));
  g = ex2_pair(mul2(mul2(x, x), pair(-0.5f * kLog2e)));
  f2 p;
  if constexpr (DEGREE == 8) {
    p = fma2(pair(0.036641013f), t, pair(-0.152744919f));
    p = fma2(p, t, pair(0.185308799f));
    p = fma2(p, t, pair(-0.0376242623f));
    p = fma2(p, t, pair(0.12085367f));
    p = fma2(p, t, pair(0.103464633f));
    p = fma2(p, t, pair(0.122461125f));
    p = fma2(p, t, pair(0.121640012f));
  } else {
    p = fma2(pair(-0.0754334107f), t, pair(0.189625621f));
    p = fma2(p, t, pair(0.00726738665f));
    p = fma2(p, t, pair(0.13653487f));
    p = fma2(p, t, pair(0.118881285f));
    p = fma2(p, t, pair(0.12312267f));
  }
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
    return mul2(x, normal_cdf<6>(x, g));
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
    const f2 c = normal_cdf<8>(x, g);
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

// value and derivative where they are stored in binary32: as above, but
//   gelu       within |x| <= 1.5 from Phi = 1/2 + x C(x^2), C of degree 6 (absolute error of Phi
//              7e-10), outside from a tail of degree 6 fitted to |z| >= 1.45 (2.4e-7 of itself)
//   tanh gelu  the gate's complement as 2^z times the gate: 1 - s cancels for large x
// On normal inputs the 2-norm of the error is 4e-8 for gelu and its derivative, as of a
// plain binary32 evaluation with erf; the tail alone, as for BF16, leaves 6.6e-8 in the
// derivative.  Recomputed at 8192 x 8192: 71 us (without an activation 70),
// with that tail 62, with CUDA's normcdff 143.
template <int ACT>
__device__ __forceinline__ f2 act_fd2_f32(f2 x, f2& d) {
  if constexpr (ACT == AQFQ_ACT_GELU) {
    const f2 a = x & 0x7FFFFFFF7FFFFFFFull, s = mul2(x, x);
    const f2 g = ex2_pair(mul2(s, pair(-0.5f * kLog2e)));
    const f2 t = rcp_pair(fma2(pair(0.335f), a, pair(1.0f)));
    f2 p = fma2(pair(-0.0726788342f), t, pair(0.124253586f));
    p = fma2(p, t, pair(0.0547424667f));
    p = fma2(p, t, pair(0.126858488f));
    p = fma2(p, t, pair(0.132618517f));
    p = fma2(p, t, pair(0.133697599f));
    const f2 q = mul2(mul2(p, t), g);  // Phi(-|x|)
    const f2 r = sub2(pair(1.0f), q);
    f2 m = fma2(pair(3.99588544e-07f), s, pair(-8.62985507e-06f));
    m = fma2(m, s, pair(0.000114104412f));
    m = fma2(m, s, pair(-0.00118614291f));
    m = fma2(m, s, pair(0.00997301005f));
    m = fma2(m, s, pair(-0.0664902702f));
    m = fma2(m, s, pair(0.398942262f));
    const bool mid0 = lo2(a) <= 1.5f, mid1 = hi2(a) <= 1.5f;
    const f2 tail = mk2(lo2(x) < 0.0f ? lo2(q) : lo2(r), hi2(x) < 0.0f ? hi2(q) : hi2(r));
    const f2 cm = fma2(m, x, pair(0.5f)), ym = fma2(m, s, mul2(x, pair(0.5f))), yt = mul2(x, tail);
    const f2 c = mk2(mid0 ? lo2(cm) : lo2(tail), mid1 ? hi2(cm) : hi2(tail));
    d = fma2(mul2(x, pair(0.3989422804f)), g, c);
    return mk2(mid0 ? lo2(ym) : lo2(yt), mid1 ? hi2(ym) : hi2(yt));
  } else if constexpr (ACT == AQFQ_ACT_GELU_TANH) {
    const f2 k = fma2(mul2(x, x), pair(-2.0f * kTanhC * kLog2e * kTanhA), pair(-2.0f * kTanhC * kLog2e));
    const f2 z = ex2_pair(mul2(x, k));
    const f2 e = mk2(fminf(lo2(z), 1e38f), fminf(hi2(z), 1e38f));  // (times a gate of zero)
    const f2 s = rcp_pair(add2(z, pair(1.0f)));
    const f2 c = mk2(fminf(fmaxf(lo2(x), -16.0f), 16.0f), fminf(fmaxf(hi2(x), -16.0f), 16.0f));
    const f2 u = fma2(mul2(c, c), pair(6.0f * kTanhC * kTanhA), pair(2.0f * kTanhC));
    d = fma2(mul2(mul2(c, s), mul2(e, s)), u, s);
    return mul2(x, s);
  } else {
    return act_fd2<ACT>(x, d);
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

// the same for pairs; F32: stored in binary32
template <int ACT, bool F32, int P>
__device__ __forceinline__ void act_all(f2 (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (F32) {
      f2 d;
      v[i] = act_fd2_f32<ACT>(v[i], d);
    } else {
      v[i] = act2<ACT>(v[i]);
    }
  }
}
template <int ACT, bool F32, int P>
__device__ __forceinline__ void slope_all(f2 (&p)[P], f2 (&v)[P]) {
  if constexpr (ACT != AQFQ_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      f2 d;
      if constexpr (F32) {
        p[i] = act_fd2_f32<ACT>(p[i], d);
      } else {
        p[i] = act_fd2<ACT>(p[i], d);
      }
      v[i] = mul2(v[i], d);
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

// The group's divisor: s = RN(amax / qmax) and RN(1 / s).  The quotient by the
// constant is Markstein's correction with RN(1 / qmax) (equal to the IEEE quotient
// for every binary32 mantissa; checked for both constants); tiny amax divides.
template <int FMT>
__device__ __forceinline__ Divisor ckpt_divisor(uint32_t amax_bits) {
  constexpr float qm = FMT == AQFQ_INT8 ? 127.0f : 448.0f, rc = 1.0f / qm;
  const float a = __uint_as_float(amax_bits);
  const float q0 = __fmul_rn(a, rc);
  float s = __fmaf_rn(__fmaf_rn(-q0, qm, a), rc, q0);
  if (!(a >= 0x1p-90f && a < 0x1p127f))  // rare: tiny, huge, infinite or NaN
    s = amax_bits >= 0x7F800000u ? __int_as_float(0x7FC00000) : __fdiv_rn(a, qm);
  return make_divisor(s);
}

// four codes of x / s, element 0 in the low byte; a scale of zero or NaN gives zeros
template <int FMT>
__device__ __forceinline__ uint32_t grid_codes4(f2 a, f2 b) {
  if constexpr (FMT == AQFQ_INT8) {
    // |x / s| <= 127 (1 + 2^-23) rounds to at most 127: no clamp.  The sum with 1.5 * 2^23
    // holds the rounded integer in its low bits.
    a = add2(a, pair(12582912.0f)), b = add2(b, pair(12582912.0f));
    return __byte_perm(__byte_perm(uint32_t(a), uint32_t(a >> 32), 0x0040),
                       __byte_perm(uint32_t(b), uint32_t(b >> 32), 0x0040), 0x5410);
  } else {
    return cvt_e4m3x2(hi2(a), lo2(a)) | (cvt_e4m3x2(hi2(b), lo2(b)) << 16);
  }
}
// x: 2 P pairs; w: P words of codes
template <int FMT, int P>
__device__ __forceinline__ void ckpt_codes(const f2* x, const Divisor& d, uint32_t (&w)[P]) {
  if (d.fast) {
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = grid_codes4<FMT>(mdiv2(x[2 * i], d), mdiv2(x[2 * i + 1], d));
  } else {  // zero, NaN, or beyond the fast range (a rounded subnormal scale may leave the grid)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 p = x[2 * i + (j >> 1)];
        q[j] = d.s > 0.0f ? __fdiv_rn(j & 1 ? hi2(p) : lo2(p), d.s) : 0.0f;
        if (FMT == AQFQ_INT8) q[j] = fminf(fmaxf(q[j], -127.0f), 127.0f);
      }
      w[i] = grid_codes4<FMT>(mk2(q[0], q[1]), mk2(q[2], q[3]));
    }
  }
}
// the format chosen at run time (uniform)
__device__ __forceinline__ Divisor ckpt_divisor(uint32_t amax_bits, int fmt) {
  return fmt == AQFQ_INT8 ? ckpt_divisor<AQFQ_INT8>(amax_bits) : ckpt_divisor<AQFQ_FP8_E4M3>(amax_bits);
}
template <int P>
__device__ __forceinline__ void ckpt_codes(const f2* x, const Divisor& d, int fmt, uint32_t (&w)[P]) {
  if (fmt == AQFQ_INT8) ckpt_codes<AQFQ_INT8>(x, d, w);
  else ckpt_codes<AQFQ_FP8_E4M3>(x, d, w);
}

// four stored values (code * s, rounded to binary32) as two pairs
__device__ __forceinline__ void ckpt_values4(uint32_t c, float s, int fmt, f2* v) {
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
  v[0] = mul2(a, pair(s)), v[1] = mul2(b, pair(s));
}
__device__ __forceinline__ void ckpt_values4(uint32_t c, float s, int fmt, float* v) {
  f2 p[2];
  ckpt_values4(c, s, fmt, p);
  v[0] = lo2(p[0]), v[1] = hi2(p[0]), v[2] = lo2(p[1]), v[3] = hi2(p[1]);
}

// bits of the largest |x|, at or above those of infinity when one is NaN
__device__ __forceinline__ void amax_step(float& m, f2 p) {
  asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(lo2(p)), "f"(hi2(p)));
}
template <int V>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[V]) {
  static_assert(V % 2 == 0, "pairs");
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < V; i += 2) amax_step(m, mk2(v[i], v[i + 1]));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}
template <int P>
__device__ __forceinline__ uint32_t amax_bits(const f2 (&v)[P]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i) amax_step(m, v[i]);
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

// ---------------------------------------------------------------------------
// A lane's share of a row: NV vectors of V consecutive elements, kept as they are
// in memory until all loads are under way.  V = 8 where rows allow 16-byte
// accesses (16 BF16 where they allow 32-byte ones); V = 2 (the norms between blocks)
// or 1 (neighbouring lanes on neighbouring columns) where they do not.  In arithmetic
// the E = NV V elements are E / 2 pairs: neighbours within a vector (V > 1), or the
// same lane's elements of vectors 2k and 2k + 1 (V = 1).
// ---------------------------------------------------------------------------
template <typename T, int V, int NV>
struct Row {
  static constexpr int W = V == 1 ? 1 : V * int(sizeof(T)) / 4;
  uint32_t w[NV][W];
  __device__ __forceinline__ void load(int j, const T* p) {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 2) w[j][0] = __ldg(reinterpret_cast<const uint16_t*>(p));
      else w[j][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (V == 2) {
      if constexpr (sizeof(T) == 2) {
        w[j][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        w[j][0] = u.x, w[j][1] = u.y;
      }
    } else if constexpr (V == 16) {
      static_assert(sizeof(T) == 2, "32 bytes");
      ld_stream(p, w[j]);
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        ld_stream_v4(reinterpret_cast<const uint32_t*>(p) + i, w[j][i], w[j][i + 1], w[j][i + 2], w[j][i + 3]);
    }
  }
  __device__ __forceinline__ void zero(int j) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[j][i] = 0;
  }
  __device__ __forceinline__ f2 pair_at(int i) const {  // 0 <= i < E / 2
    if constexpr (V == 1) {
      const uint32_t a = w[2 * i][0], b = w[2 * i + 1][0];
      return sizeof(T) == 2 ? mk2(__uint_as_float(a << 16), __uint_as_float(b << 16))
                            : mk2(__uint_as_float(a), __uint_as_float(b));
    } else if constexpr (sizeof(T) == 2) {
      return bf2(w[i / W][i % W]);
    } else if constexpr (V == 2) {
      return mk2(__uint_as_float(w[i][0]), __uint_as_float(w[i][1]));
    } else {
      return mk2(__uint_as_float(w[i / 4][2 * (i % 4)]), __uint_as_float(w[i / 4][2 * (i % 4) + 1]));
    }
  }
};
// stores vector j of a lane's pairs
template <typename T, int V>
__device__ __forceinline__ void put(T* p, const f2* v, int j) {
  if constexpr (V == 1) {
    from_f(j & 1 ? hi2(v[j / 2]) : lo2(v[j / 2]), *p);
  } else if constexpr (V == 2) {
    if constexpr (sizeof(T) == 2) st_32(p, pack2(v[j]));
    else st_64(p, uint32_t(v[j]), uint32_t(v[j] >> 32));
  } else if constexpr (V == 16) {
    const f2* q = v + 8 * j;
    const uint32_t w[8] = {pack2(q[0]), pack2(q[1]), pack2(q[2]), pack2(q[3]),
                           pack2(q[4]), pack2(q[5]), pack2(q[6]), pack2(q[7])};
    st_256(p, w);
  } else if constexpr (sizeof(T) == 2) {
    const f2* q = v + 4 * j;
    st_128(p, pack2(q[0]), pack2(q[1]), pack2(q[2]), pack2(q[3]));
  } else {
    const f2* q = v + 4 * j;
    const uint32_t w[8] = {uint32_t(q[0]), uint32_t(q[0] >> 32), uint32_t(q[1]), uint32_t(q[1] >> 32),
                           uint32_t(q[2]), uint32_t(q[2] >> 32), uint32_t(q[3]), uint32_t(q[3] >> 32)};
    st_128(p, w[0], w[1], w[2], w[3]);
    st_128(p + 4, w[4], w[5], w[6], w[7]);
  }
}
// the codes of a lane's vectors
template <int V, int NV>
struct CodeRow {
  static constexpr int W = V == 1 ? 1 : V / 4;
  uint32_t w[NV][W];
  float s[NV];
  __device__ __forceinline__ void load(int j, const Ckpt& c, int64_t r, int64_t cols, int64_t col) {
    const uint8_t* p = c.codes + r * cols + col;
    if constexpr (V == 16)
      ld_stream_v4(p, w[j][0], w[j][1], w[j][2], w[j][3]);
    else if constexpr (V == 8)
      asm("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[j][0]), "=r"(w[j][1]) : "l"(p));
    else
      w[j][0] = __ldg(p);
    s[j] = __ldg(c.scale + r * c.groups + (col >> c.lg));
  }
  __device__ __forceinline__ void zero(int j) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[j][i] = 0;
    s[j] = 0.0f;
  }
  __device__ __forceinline__ void values(int fmt, f2 (&v)[NV * V / 2]) const {
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < W; ++i) ckpt_values4(w[j][i], s[j], fmt, v + (j * W + i) * 2);
    } else {
#pragma unroll
      for (int j = 0; j < NV; j += 2) {
        f2 a[2], b[2];
        ckpt_values4(w[j][0], s[j], fmt, a);
        ckpt_values4(w[j + 1][0], s[j + 1], fmt, b);
        v[j / 2] = mk2(lo2(a[0]), lo2(b[0]));
      }
    }
  }
};

// Writes the 8-bit checkpoint of a warp's share of row r.  v: pairs, zero beyond
// the row; col[j] the first column of vector j, in[j] whether it is stored.
// V = 8: a group is a run of lanes; V = 1: one, two or four whole vectors, vector j
// a multiple of four ones starting a multiple of 128 columns.
template <int FMT, int V, int NV>
__device__ __forceinline__ void ckpt_write(const Ckpt& c, int64_t r, int64_t cols,
                                           const int64_t (&col)[NV], const bool (&in)[NV],
                                           const f2 (&v)[NV * V / 2]) {
  uint8_t* codes = c.codes + r * cols;
  float* scale = c.scale + r * c.groups;
  const int mask = (1 << c.lg) - 1;
  if constexpr (V == 8) {
    uint32_t m[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const f2 t[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
      m[j] = amax_bits(t);
    }
    // a group is at least four lanes
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      if (o < 4 || o < (1 << (c.lg - 3))) {
#pragma unroll
        for (int j = 0; j < NV; ++j) m[j] = max(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Divisor d = ckpt_divisor<FMT>(m[j]);
      uint32_t w[2];
      ckpt_codes<FMT>(v + 4 * j, d, w);
      if (in[j]) {
        st_64(codes + col[j], w[0], w[1]);
        if ((int(col[j]) & mask) == 0) scale[col[j] >> c.lg] = d.s;
      }
    }
  } else {
    static_assert(NV % 4 == 0, "groups of four vectors");
#pragma unroll
    for (int j = 0; j < NV; j += 4) {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 p = v[(j + i) / 2];
        m[i] = __reduce_max_sync(0xFFFFFFFFu, uint32_t(i & 1 ? p >> 32 : p) & 0x7FFFFFFFu);
      }
      if (c.lg > 5) m[0] = m[1] = max(m[0], m[1]), m[2] = m[3] = max(m[2], m[3]);
      if (c.lg > 6) m[0] = m[1] = m[2] = m[3] = max(m[0], m[2]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Divisor d = ckpt_divisor<FMT>(m[i]);
        const f2 p = v[(j + i) / 2];
        const f2 one[2] = {mk2(i & 1 ? hi2(p) : lo2(p), 0.0f), 0ull};
        uint32_t w[1];
        ckpt_codes<FMT>(one, d, w);
        if (in[j + i]) {
          codes[col[j + i]] = uint8_t(w[0]);
          if ((int(col[j + i]) & mask) == 0) scale[col[j + i] >> c.lg] = d.s;
        }
      }
    }
  }
}

// The checkpoint of a lane's 16 consecutive columns (in two halves of 8, zero beyond
// the row): a group is 2, 4 or 8 neighbouring lanes.  p: its codes (a16: 16-byte
// aligned), scale: its group's, written by the lane with the group's first column.
template <int FMT>
__device__ __forceinline__ void ckpt_write16(int lg, uint8_t* p, bool a16, float* scale, bool first,
                                             bool in0, bool in1, const f2 (&v)[8]) {
  uint32_t m = amax_bits(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  if (lg > 5) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  if (lg > 6) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
  const Divisor d = ckpt_divisor<FMT>(m);
  uint32_t w[4];
  ckpt_codes<FMT>(v, d, w);
  if (a16 && in1) {
    st_128(p, w[0], w[1], w[2], w[3]);
  } else {
    if (in0) st_64(p, w[0], w[1]);
    if (in1) st_64(p + 8, w[2], w[3]);
  }
  if (first && in0) *scale = d.s;
}

// ---------------------------------------------------------------------------
// Column sums of a few blocks that form one cluster: each block has its sums in
// shared memory (out at [0, cols), out2 at [second, second + cols)), block i finishes
// the i-th share of the columns, adding the blocks' values in order.  Every thread
// of every block calls it.
// ---------------------------------------------------------------------------
struct Join {
  float *out, *out2;  // either may be NULL
  int accumulate;
  bool on;
};
__device__ __forceinline__ void join_columns(const Join& j, const float* sums, int second, int64_t cols) {
  uint32_t rank, n;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  if (n == 1) {  // a single block
    __syncthreads();
    for (int c = int(threadIdx.x); c < int(cols); c += int(blockDim.x)) {
      if (j.out) j.out[c] = j.accumulate ? j.out[c] + sums[c] : sums[c];
      if (j.out2) j.out2[c] = j.accumulate ? j.out2[c] + sums[second + c] : sums[second + c];
    }
    return;
  }
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  const int c0 = int(cols * rank / n), c1 = int(cols * (rank + 1) / n);
  for (int k = 0; k < 2; ++k) {
    float* out = k ? j.out2 : j.out;
    if (!out) continue;
    for (int c = c0 + int(threadIdx.x); c < c1; c += int(blockDim.x)) {
      const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(sums + (k ? second : 0) + c));
      float v[8], t = 0.0f;
#pragma unroll
      for (uint32_t b = 0; b < 8; ++b) {
        v[b] = 0.0f;
        if (b < n)
          asm volatile(
              "{ .reg .b32 a;\n\t"
              "mapa.shared::cluster.u32 a, %1, %2;\n\t"
              "ld.shared::cluster.f32 %0, [a]; }"
              : "=f"(v[b])
              : "r"(at), "r"(b)
              : "memory");
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) t += v[b];
      out[c] = j.accumulate ? out[c] + t : t;
    }
  }
  // the others have read this block's sums
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
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
