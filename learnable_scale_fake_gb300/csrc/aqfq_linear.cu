// aqfq_linear.cu -- the matrix product with bias, activation and residual in
// its epilogue, and the two gradient products.
//
//   forward       y = act(p) (+ res),  p = x W^T + b   (p optionally kept in 8 bits)
//   input grad    dx = (dy W) act'(p') (+ res)         (p' from its 8-bit checkpoint)
//   weight grad   dw = dy^T x (+ dw)
//
// All three are out[r, c] = sum over k of A(r, k) B(c, k) with other strides:
//   forward       r = m, c = n, k = k:  A = x (k contiguous), B = W (k contiguous)
//   input grad    r = m, c = k, k = n:  A = dy (n contiguous), B = W (c contiguous)
//   weight grad   r = n, c = k, k = m:  A = dy (r contiguous), B = x (c contiguous)
#include "aqfq_internal.h"
#include "aqfq_layer.cuh"

namespace aqfq {
namespace layer {
namespace {

enum Pass { P_FWD = AQFQ_LINEAR_FWD, P_DGRAD = AQFQ_LINEAR_DGRAD, P_WGRAD = AQFQ_LINEAR_WGRAD };

// ---------------------------------------------------------------------------
// epilogue: a warp holds 128 columns of one row, a lane 4 of them, so an 8-bit
// group of 32, 64 or 128 columns is 8, 16 or 32 neighbouring lanes
// ---------------------------------------------------------------------------
struct Epi {
  int64_t rows, cols;
  const void* bias;     // forward
  const bf16* res;      // forward, input gradient
  int64_t ldr;
  void* out;
  int64_t ldo;
  int bias_dtype, out_dtype, act, accumulate;
  bool vec_out, vec_res, vec_bias, vec_codes;  // 4-element accesses are aligned
  Ckpt c;               // forward: written; input gradient: read
};

// v: the sums of row r, columns [col, col + 4); every lane of the warp calls it
template <int PASS>
__device__ __forceinline__ void epilogue4(const Epi& e, int64_t r, int64_t col, float (&v)[4]) {
  const int n = e.cols - col > 4 ? 4 : int(e.cols - col);
  const bool in = r < e.rows && n > 0, full = n == 4;
  if constexpr (PASS == P_FWD) {
    if (e.bias && in) {
      float b[4];
      if (e.bias_dtype == AQFQ_BF16)
        load_row(static_cast<const bf16*>(e.bias) + col, e.vec_bias && full, n, b);
      else
        load_row(static_cast<const float*>(e.bias) + col, e.vec_bias && full, n, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += b[i];
    }
    if (e.c.codes) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = i < n ? v[i] : 0.0f;  // beyond the row: no share in amax
      uint32_t m = amax_bits(v);
      for (int o = 1; o < (1 << (e.c.lg - 2)); o <<= 1)
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const Divisor d = make_divisor(ckpt_scale(m, e.c.fmt));
      if (in) {
        const uint32_t w[1] = {ckpt_codes4(v, d, e.c.fmt)};
        store_bytes<4>(e.c.codes + r * e.cols + col, e.vec_codes && full, n, w);
        if ((col & ((1 << e.c.lg) - 1)) == 0) e.c.scale[r * e.c.groups + (col >> e.c.lg)] = d.s;
      }
    }
    act_apply(e.act, v);
  }
  if (!in) return;
  if constexpr (PASS == P_DGRAD) {
    if (e.c.codes) {
      uint32_t w[1];
      load_bytes<4>(e.c.codes + r * e.cols + col, e.vec_codes && full, n, w);
      float p[4];
      ckpt_values4(w[0], e.c.scale[r * e.c.groups + (col >> e.c.lg)], e.c.fmt, p);
      slope_apply(e.act, p, v);
    }
  }
  if constexpr (PASS != P_WGRAD) {
    if (e.res) {
      float b[4];
      load_row(e.res + r * e.ldr + col, e.vec_res && full, n, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += b[i];
    }
    store_row(static_cast<bf16*>(e.out) + r * e.ldo + col, e.vec_out && full, n, v);
  } else if (e.out_dtype == AQFQ_BF16) {
    bf16* o = static_cast<bf16*>(e.out) + r * e.ldo + col;
    if (e.accumulate) {
      float b[4];
      load_row(o, e.vec_out && full, n, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += b[i];
    }
    store_row(o, e.vec_out && full, n, v);
  } else {
    float* o = static_cast<float*>(e.out) + r * e.ldo + col;
    if (e.accumulate) {
      float b[4];
      load_row(o, e.vec_out && full, n, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += b[i];
    }
    store_row(o, e.vec_out && full, n, v);
  }
}

// ---------------------------------------------------------------------------
// product: 64 x 128 outputs per CTA, 16 of k at a time through shared memory;
// a warp computes 8 rows, a lane 4 columns of each
// ---------------------------------------------------------------------------
struct Operands {
  const bf16 *a, *b;
  int64_t ars, aks, brs, bks;  // element strides along r / c and k
  int64_t rows, cols, depth;
};

constexpr int BM = 64, BN = 128, BK = 16;

template <int PASS>
__global__ void __launch_bounds__(256) linear_kernel(const Operands o, const Epi e) {
  __shared__ float sa[BK][BM + 1];
  __shared__ __align__(16) float sb[BK][BN + 4];
  const int64_t r0 = int64_t(blockIdx.y) * BM, c0 = int64_t(blockIdx.x) * BN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[8][4] = {};
  for (int64_t k0 = 0; k0 < o.depth; k0 += BK) {
    for (int i = threadIdx.x; i < BM * BK; i += 256) {
      // consecutive threads along the contiguous axis
      const int k = o.aks == 1 ? i % BK : i / BM, r = o.aks == 1 ? i / BK : i % BM;
      sa[k][r] = (r0 + r < o.rows && k0 + k < o.depth)
                     ? to_f(o.a[(r0 + r) * o.ars + (k0 + k) * o.aks]) : 0.0f;
    }
    for (int i = threadIdx.x; i < BN * BK; i += 256) {
      const int k = o.bks == 1 ? i % BK : i / BN, c = o.bks == 1 ? i / BK : i % BN;
      sb[k][c] = (c0 + c < o.cols && k0 + k < o.depth)
                     ? to_f(o.b[(c0 + c) * o.brs + (k0 + k) * o.bks]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      const float4 b = *reinterpret_cast<const float4*>(&sb[k][lane * 4]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = sa[k][warp * 8 + i];
        acc[i][0] = fmaf(a, b.x, acc[i][0]);
        acc[i][1] = fmaf(a, b.y, acc[i][1]);
        acc[i][2] = fmaf(a, b.z, acc[i][2]);
        acc[i][3] = fmaf(a, b.w, acc[i][3]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) epilogue4<PASS>(e, r0 + warp * 8 + i, c0 + lane * 4, acc[i]);
}

template <int PASS>
cudaError_t launch(const Operands& o, const Epi& e, cudaStream_t st) {
  const int64_t gx = (o.cols + BN - 1) / BN, gy = (o.rows + BM - 1) / BM;
  linear_kernel<PASS><<<dim3(unsigned(gx), unsigned(gy)), 256, 0, st>>>(o, e);
  return cudaGetLastError();
}

// sizes of one product; operands that the tensor memory accelerator can read
// (16-byte base, rows a multiple of 16 bytes apart)
bool size_ok(int64_t v) { return v >= 0 && v <= 0x3FFFFFFF; }
bool operand_ok(const void* p, int64_t ld) { return al(p, 16) && ld % 8 == 0; }

void finish_epi(Epi& e, int es) {
  e.vec_out = rows_aligned<4>(e.out, e.ldo, es);
  e.vec_res = rows_aligned<4>(e.res, e.ldr, 2);
  e.vec_bias = rows_aligned<4>(e.bias, 4, esize(e.bias_dtype));
  e.vec_codes = rows_aligned<4>(e.c.codes, e.cols, 1);
}

}  // namespace
}  // namespace layer
}  // namespace aqfq

using namespace aqfq;
using namespace aqfq::layer;

extern "C" size_t aqfq_linear_workspace_bytes(int pass, int64_t M, int64_t N, int64_t K) {
  (void)pass, (void)M, (void)N, (void)K;
  return 0;
}

extern "C" aqfq_status aqfq_linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                       int64_t M, int64_t N, int64_t K, int bias_dtype,
                                       const void* bias, int act, const void* residual,
                                       int64_t ldr, void* y, int64_t ldy, const aqfq_ckpt8* ckpt,
                                       void* workspace, size_t workspace_bytes,
                                       int32_t* error_flag, void* stream) {
  (void)workspace, (void)workspace_bytes, (void)error_flag;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !view_ok(M, K, ldx) || !view_ok(N, K, ldw) ||
      !view_ok(M, N, ldy) || (residual && !view_ok(M, N, ldr)))
    return AQFQ_ERR_SHAPE;
  if (!act_ok(act) || !dtype_ok(bias_dtype)) return AQFQ_ERR_UNSUPPORTED;
  Epi e = {};
  if (ckpt) {
    const aqfq_status s = make_ckpt(ckpt, M, N, e.c);
    if (s != AQFQ_OK) return s;
  }
  if (M > 0 && N > 0 && (!y || (K > 0 && (!x || !w)))) return AQFQ_ERR_NULL;
  if (!operand_ok(x, ldx) || !operand_ok(w, ldw) || !al(bias, esize(bias_dtype)) ||
      !al(residual, 2) || !al(y, 2) || !al(error_flag, 4))
    return AQFQ_ERR_ALIGN;
  if (M == 0 || N == 0) return AQFQ_OK;
  e.rows = M, e.cols = N;
  e.bias = bias, e.bias_dtype = bias_dtype;
  e.res = static_cast<const bf16*>(residual), e.ldr = ldr;
  e.out = y, e.ldo = ldy, e.out_dtype = AQFQ_BF16, e.act = act;
  finish_epi(e, 2);
  const Operands o = {static_cast<const bf16*>(x), static_cast<const bf16*>(w), ldx, 1, ldw, 1, M, N, K};
  return launch<P_FWD>(o, e, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA;
}

extern "C" aqfq_status aqfq_linear_dgrad(const void* dy, int64_t lddy, const void* w, int64_t ldw,
                                         int64_t M, int64_t N, int64_t K, int act,
                                         const aqfq_ckpt8* ckpt, const void* residual,
                                         int64_t ldr, void* dx, int64_t lddx, void* workspace,
                                         size_t workspace_bytes, int32_t* error_flag,
                                         void* stream) {
  (void)workspace, (void)workspace_bytes, (void)error_flag;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !view_ok(M, N, lddy) || !view_ok(N, K, ldw) ||
      !view_ok(M, K, lddx) || (residual && !view_ok(M, K, ldr)))
    return AQFQ_ERR_SHAPE;
  if (!act_ok(act)) return AQFQ_ERR_UNSUPPORTED;
  Epi e = {};
  if (ckpt) {
    const aqfq_status s = make_ckpt(ckpt, M, K, e.c);
    if (s != AQFQ_OK) return s;
  } else if (act != AQFQ_ACT_NONE) {
    return AQFQ_ERR_NULL;  // an activation's derivative needs its input
  }
  if (M > 0 && K > 0 && (!dx || (N > 0 && (!dy || !w)))) return AQFQ_ERR_NULL;
  if (!operand_ok(dy, lddy) || !operand_ok(w, ldw) || !al(residual, 2) || !al(dx, 2) ||
      !al(error_flag, 4))
    return AQFQ_ERR_ALIGN;
  if (M == 0 || K == 0) return AQFQ_OK;
  e.rows = M, e.cols = K;
  e.res = static_cast<const bf16*>(residual), e.ldr = ldr;
  e.out = dx, e.ldo = lddx, e.out_dtype = AQFQ_BF16, e.act = act;
  finish_epi(e, 2);
  const Operands o = {static_cast<const bf16*>(dy), static_cast<const bf16*>(w), lddy, 1, 1, ldw, M, K, N};
  return launch<P_DGRAD>(o, e, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA;
}

extern "C" aqfq_status aqfq_linear_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                         int64_t M, int64_t N, int64_t K, int dtype, void* dw,
                                         int64_t lddw, int accumulate, void* workspace,
                                         size_t workspace_bytes, int32_t* error_flag,
                                         void* stream) {
  (void)workspace, (void)workspace_bytes, (void)error_flag;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !view_ok(M, N, lddy) || !view_ok(M, K, ldx) ||
      !view_ok(N, K, lddw))
    return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype)) return AQFQ_ERR_UNSUPPORTED;
  if (N > 0 && K > 0 && (!dw || (M > 0 && (!dy || !x)))) return AQFQ_ERR_NULL;
  if (!operand_ok(dy, lddy) || !operand_ok(x, ldx) || !al(dw, esize(dtype)) || !al(error_flag, 4))
    return AQFQ_ERR_ALIGN;
  if (N == 0 || K == 0) return AQFQ_OK;
  Epi e = {};
  e.rows = N, e.cols = K;
  e.out = dw, e.ldo = lddw, e.out_dtype = dtype, e.accumulate = accumulate;
  finish_epi(e, esize(dtype));
  const Operands o = {static_cast<const bf16*>(dy), static_cast<const bf16*>(x), 1, lddy, 1, ldx, N, K, M};
  return launch<P_WGRAD>(o, e, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA;
}
