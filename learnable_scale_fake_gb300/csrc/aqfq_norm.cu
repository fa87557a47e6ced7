// aqfq_norm.cu -- layer norm, forward and backward, over the last axis.
//
// Row of C columns: mu = sum x / C, var = sum (x - mu)^2 / C (two passes, so a
// large mean does not cancel), r = (var + eps)^-1/2, y = (x - mu) r gamma + beta.
// Backward, h = (x - mu) r and u = dy gamma:
//   dx = r (u - mean(u) - h mean(u h)) (+ dres)
//   dgamma = sum over rows of dy h,   dbeta = sum over rows of dy
// with x as it was, or as its 8-bit checkpoint gives it back (then mu and r
// are still those of the exact x).
#include "aqfq_internal.h"
#include "aqfq_layer.cuh"

namespace aqfq {
namespace layer {
namespace {

constexpr int kT = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// sum over the block, the same value in every thread
__device__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();  // red is free
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) t += red[w];
  return t;
}

// gamma / beta: columns [col, col + 8) of a vector of either type; NULL gives `def`
__device__ __forceinline__ void load_param(const void* p, int pdtype, bool vec, int64_t col, int n,
                                           float def, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = def;
  } else if (pdtype == AQFQ_BF16) {
    load_row(static_cast<const bf16*>(p) + col, vec && n == 8, n, v);
  } else {
    load_row(static_cast<const float*>(p) + col, vec && n == 8, n, v);
  }
}

struct FwdArgs {
  int64_t ldx, ldy, rows, cols;
  const void *gamma, *beta;
  float *mean, *rstd;
  float eps;
  int pdtype;
  bool vec, pvec, cvec;
  Ckpt c;
};

template <typename T>
__global__ void __launch_bounds__(kT) norm_fwd_kernel(const T* x, T* y, const FwdArgs a) {
  __shared__ float red[kT / 32];
  const float inv = 1.0f / float(a.cols);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* row = x + r * a.ldx;
    float s = 0.0f;
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kT * 8) {
      const int n = a.cols - col > 8 ? 8 : int(a.cols - col);
      float v[8];
      load_row(row + col, a.vec && n == 8, n, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    const float mu = block_sum(s, red) * inv;
    s = 0.0f;
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kT * 8) {
      const int n = a.cols - col > 8 ? 8 : int(a.cols - col);
      float v[8];
      load_row(row + col, a.vec && n == 8, n, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) s = fmaf(v[i] - mu, v[i] - mu, s);
    }
    const float rs = rsqrtf(block_sum(s, red) * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mu;
      if (a.rstd) a.rstd[r] = rs;
    }
    // whole warps walk together: a checkpoint group is a run of lanes
    for (int64_t c0 = (threadIdx.x & ~31) * 8; c0 < a.cols; c0 += kT * 8) {
      const int64_t col = c0 + (threadIdx.x & 31) * 8;
      const int n = a.cols - col > 8 ? 8 : int(a.cols - col);
      float v[8], g[8], b[8];
      load_row(row + col, a.vec && n == 8, n, v);
      if (a.c.codes) {
        uint32_t m = amax_bits(v);
        for (int o = 1; o < (1 << (a.c.lg - 3)); o <<= 1)
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const Divisor d = make_divisor(ckpt_scale(m, a.c.fmt));
        if (n > 0) {
          const uint32_t w[2] = {ckpt_codes4(v, d, a.c.fmt), ckpt_codes4(v + 4, d, a.c.fmt)};
          store_bytes<8>(a.c.codes + r * a.cols + col, a.cvec && n == 8, n, w);
          if ((col & ((1 << a.c.lg) - 1)) == 0) a.c.scale[r * a.c.groups + (col >> a.c.lg)] = d.s;
        }
      }
      if (n > 0) {
        load_param(a.gamma, a.pdtype, a.pvec, col, n, 1.0f, g);
        load_param(a.beta, a.pdtype, a.pvec, col, n, 0.0f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf((v[i] - mu) * rs, g[i], b[i]);
        store_row(y + r * a.ldy + col, a.vec && n == 8, n, v);
      }
    }
  }
}

struct BwdArgs {
  int64_t lddy, ldx, lddres, lddx, rows, cols;
  const float *mean, *rstd;
  const void* gamma;
  int pdtype;
  bool vec, pvec, cvec;
  Ckpt c;
};

// h of 8 columns: from x, or from its checkpoint
template <typename T>
__device__ __forceinline__ void load_h(const T* x, const BwdArgs& a, int64_t r, int64_t col, int n,
                                       float mu, float rs, float (&h)[8]) {
  if (x) {
    load_row(x + r * a.ldx + col, a.vec && n == 8, n, h);
  } else {
    uint32_t w[2];
    load_bytes<8>(a.c.codes + r * a.cols + col, a.cvec && n == 8, n, w);
    const float s = a.c.scale[r * a.c.groups + (col >> a.c.lg)];
    ckpt_values4(w[0], s, a.c.fmt, h);
    ckpt_values4(w[1], s, a.c.fmt, h + 4);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = i < n ? (h[i] - mu) * rs : 0.0f;
}

template <typename T>
__global__ void __launch_bounds__(kT)
    norm_dx_kernel(const T* dy, const T* x, const T* dres, T* dx, const BwdArgs a) {
  __shared__ float red[kT / 32];
  const float inv = 1.0f / float(a.cols);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float mu = a.mean[r], rs = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kT * 8) {
      const int n = a.cols - col > 8 ? 8 : int(a.cols - col);
      float v[8], g[8], h[8];
      load_row(dy + r * a.lddy + col, a.vec && n == 8, n, v);
      load_param(a.gamma, a.pdtype, a.pvec, col, n, 1.0f, g);
      load_h(x, a, r, col, n, mu, rs, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = v[i] * g[i];
        s1 += u;
        s2 = fmaf(u, h[i], s2);
      }
    }
    const float m1 = block_sum(s1, red) * inv, m2 = block_sum(s2, red) * inv;
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kT * 8) {
      const int n = a.cols - col > 8 ? 8 : int(a.cols - col);
      float v[8], g[8], h[8], e[8] = {};
      load_row(dy + r * a.lddy + col, a.vec && n == 8, n, v);
      load_param(a.gamma, a.pdtype, a.pvec, col, n, 1.0f, g);
      load_h(x, a, r, col, n, mu, rs, h);
      if (dres) load_row(dres + r * a.lddres + col, a.vec && n == 8, n, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(rs, fmaf(-h[i], m2, fmaf(v[i], g[i], -m1)), e[i]);
      store_row(dx + r * a.lddx + col, a.vec && n == 8, n, v);
    }
  }
}

// column sums of a slice of rows: a warp covers 256 columns of one row
template <typename T>
__global__ void __launch_bounds__(kT)
    norm_cols_kernel(const T* dy, const T* x, float* pg, float* pb, const BwdArgs a) {
  __shared__ float red[2][kT / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = int64_t(blockIdx.x) * 256 + lane * 8;
  const int n = a.cols - col > 8 ? 8 : int(a.cols - col);
  float sg[8] = {}, sb[8] = {};
  if (n > 0) {
    for (int64_t r = int64_t(blockIdx.y) * (kT / 32) + warp; r < a.rows;
         r += int64_t(gridDim.y) * (kT / 32)) {
      float v[8], h[8];
      load_row(dy + r * a.lddy + col, a.vec && n == 8, n, v);
      load_h(x, a, r, col, n, a.mean[r], a.rstd[r], h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sg[i] = fmaf(v[i], h[i], sg[i]);
        sb[i] += v[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[0][warp][lane * 8 + i] = sg[i], red[1][warp][lane * 8 + i] = sb[i];
  __syncthreads();
  const int64_t cc = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (cc < a.cols) {
    float g = 0.0f, b = 0.0f;
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) g += red[0][w][threadIdx.x], b += red[1][w][threadIdx.x];
    pg[int64_t(blockIdx.y) * a.cols + cc] = g;
    pb[int64_t(blockIdx.y) * a.cols + cc] = b;
  }
}

int bwd_parts(int64_t rows) {
  const int64_t p = (rows + kT / 32 - 1) / (kT / 32);
  return int(p > kMaxParts ? kMaxParts : p);
}

template <typename T>
cudaError_t launch_fwd(const void* x, void* y, const FwdArgs& a, cudaStream_t st) {
  const unsigned grid = unsigned(a.rows > 0x7FFFFFFF ? 0x7FFFFFFF : a.rows);
  norm_fwd_kernel<T><<<grid, kT, 0, st>>>(static_cast<const T*>(x), static_cast<T*>(y), a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const void* dy, const void* x, const void* dres, void* dx, float* dgamma,
                       float* dbeta, int accumulate, float* ws, const BwdArgs& a, cudaStream_t st) {
  const T *tdy = static_cast<const T*>(dy), *tx = static_cast<const T*>(x);
  if (dx) {
    const unsigned grid = unsigned(a.rows > 0x7FFFFFFF ? 0x7FFFFFFF : a.rows);
    norm_dx_kernel<T><<<grid, kT, 0, st>>>(tdy, tx, static_cast<const T*>(dres),
                                           static_cast<T*>(dx), a);
  }
  if (dgamma || dbeta) {
    const int parts = bwd_parts(a.rows);
    float* pb = ws + size_t(parts) * size_t(a.cols);
    norm_cols_kernel<T><<<dim3(unsigned((a.cols + 255) / 256), parts), kT, 0, st>>>(tdy, tx, ws,
                                                                                   pb, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_part_sums(ws, pb, parts, a.cols, dgamma, dbeta, accumulate, st);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace layer
}  // namespace aqfq

using namespace aqfq;
using namespace aqfq::layer;

extern "C" aqfq_status aqfq_layernorm_fwd(int dtype, const void* x, int64_t ldx, int64_t rows,
                                          int64_t cols, int param_dtype, const void* gamma,
                                          const void* beta, float eps, void* y, int64_t ldy,
                                          float* mean, float* rstd, const aqfq_ckpt8* ckpt,
                                          void* stream) {
  FwdArgs a = {};
  if (!view_ok(rows, cols, ldx) || !view_ok(rows, cols, ldy) || cols == 0) return AQFQ_ERR_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return AQFQ_ERR_UNSUPPORTED;
  if (ckpt) {
    if (!view_ok(rows, cols, cols)) return AQFQ_ERR_SHAPE;
    const aqfq_status s = make_ckpt(ckpt, rows, cols, a.c);
    if (s != AQFQ_OK) return s;
  }
  if (rows > 0 && (!x || !y)) return AQFQ_ERR_NULL;
  const int es = esize(dtype), ps = esize(param_dtype);
  if (!al(x, es) || !al(y, es) || !al(gamma, ps) || !al(beta, ps) || !al(mean, 4) || !al(rstd, 4))
    return AQFQ_ERR_ALIGN;
  if (rows == 0) return AQFQ_OK;
  a.ldx = ldx, a.ldy = ldy, a.rows = rows, a.cols = cols;
  a.gamma = gamma, a.beta = beta, a.mean = mean, a.rstd = rstd, a.eps = eps;
  a.pdtype = param_dtype;
  a.vec = rows_aligned<8>(x, ldx, es) && rows_aligned<8>(y, ldy, es);
  a.pvec = rows_aligned<8>(gamma, 8, ps) && rows_aligned<8>(beta, 8, ps);
  a.cvec = rows_aligned<8>(a.c.codes, cols, 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == AQFQ_BF16 ? launch_fwd<bf16>(x, y, a, st) : launch_fwd<float>(x, y, a, st);
  return e == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA;
}

extern "C" size_t aqfq_layernorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (!view_ok(rows, cols, cols)) return 0;
  return size_t(bwd_parts(rows)) * size_t(cols) * 8;
}

extern "C" aqfq_status aqfq_layernorm_bwd(int dtype, const void* dy, int64_t lddy, const void* x,
                                          int64_t ldx, const aqfq_ckpt8* ckpt, int64_t rows,
                                          int64_t cols, const float* mean, const float* rstd,
                                          int param_dtype, const void* gamma, const void* dres,
                                          int64_t lddres, void* dx, int64_t lddx, float* dgamma,
                                          float* dbeta, int accumulate, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  BwdArgs a = {};
  if (!view_ok(rows, cols, lddy) || cols == 0 || (x && !view_ok(rows, cols, ldx)) ||
      (dres && !view_ok(rows, cols, lddres)) || (dx && !view_ok(rows, cols, lddx)))
    return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return AQFQ_ERR_UNSUPPORTED;
  if (x && ckpt) return AQFQ_ERR_UNSUPPORTED;  // one form of the input
  if (ckpt) {
    if (!view_ok(rows, cols, cols)) return AQFQ_ERR_SHAPE;
    const aqfq_status s = make_ckpt(ckpt, rows, cols, a.c);
    if (s != AQFQ_OK) return s;
  }
  if (rows > 0 && (!dy || (!x && !ckpt) || !mean || !rstd)) return AQFQ_ERR_NULL;
  if (rows > 0 && !dx && !dgamma && !dbeta) return AQFQ_ERR_NULL;
  if (dres && !dx) return AQFQ_ERR_UNSUPPORTED;
  const int es = esize(dtype), ps = esize(param_dtype);
  if (!al(dy, es) || !al(x, es) || !al(dres, es) || !al(dx, es) || !al(gamma, ps) ||
      !al(mean, 4) || !al(rstd, 4) || !al(dgamma, 4) || !al(dbeta, 4))
    return AQFQ_ERR_ALIGN;
  const size_t need = aqfq_layernorm_bwd_workspace_bytes(rows, cols);
  if ((dgamma || dbeta) && need > 0) {
    if (!workspace || workspace_bytes < need) return AQFQ_ERR_WORKSPACE;
    if (!al(workspace, 8)) return AQFQ_ERR_ALIGN;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if ((dgamma || dbeta) && !accumulate &&
        launch_part_sums(nullptr, nullptr, 0, cols, dgamma, dbeta, 0, st) != cudaSuccess)
      return AQFQ_ERR_CUDA;
    return AQFQ_OK;
  }
  a.lddy = lddy, a.ldx = ldx, a.lddres = lddres, a.lddx = lddx, a.rows = rows, a.cols = cols;
  a.mean = mean, a.rstd = rstd, a.gamma = gamma, a.pdtype = param_dtype;
  a.vec = rows_aligned<8>(dy, lddy, es) && rows_aligned<8>(x, ldx, es) &&
          rows_aligned<8>(dres, lddres, es) && rows_aligned<8>(dx, lddx, es);
  a.pvec = rows_aligned<8>(gamma, 8, ps);
  a.cvec = rows_aligned<8>(a.c.codes, cols, 1);
  float* ws = static_cast<float*>(workspace);
  const cudaError_t e =
      dtype == AQFQ_BF16
          ? launch_bwd<bf16>(dy, x, dres, dx, dgamma, dbeta, accumulate, ws, a, st)
          : launch_bwd<float>(dy, x, dres, dx, dgamma, dbeta, accumulate, ws, a, st);
  return e == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA;
}
