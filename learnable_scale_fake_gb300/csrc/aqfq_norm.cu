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
constexpr int kSms = 152;

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

// ---------------------------------------------------------------------------
// Rows held in registers.  A row belongs to G warps; warp w of it holds columns
// [w 32 NV V, ...): NV vectors of V consecutive columns per lane, vector j of the
// lane at ((w NV + j) 32 + lane) V.  V = 8 where the rows allow 16-byte accesses;
// V = 1 where they do not: neighbouring lanes on neighbouring columns.
// ---------------------------------------------------------------------------
// V parameters at column col
template <int V>
__device__ __forceinline__ void params(const void* p, int pdtype, int64_t col, float def, float* v) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = def;
  } else if constexpr (V == 1) {
    v[0] = pdtype == AQFQ_BF16 ? to_f(static_cast<const bf16*>(p)[col]) : static_cast<const float*>(p)[col];
  } else {
    float t[V];
    if (pdtype == AQFQ_BF16) load_row(static_cast<const bf16*>(p) + col, true, V, t);
    else load_row(static_cast<const float*>(p) + col, true, V, t);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = t[i];
  }
}


// sum over the G warps of a row; G > 1: one barrier (named `bar`, of the row's
// warps) through red[G], which the caller alternates between two calls
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red, int bar) {
  v = warp_sum(v);
  if constexpr (G > 1) {
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x >> 5) % G] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(32 * G) : "memory");
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < G; ++w) v += red[w];
  }
  return v;
}

template <typename T, int V, int NV, int G>
__global__ void __launch_bounds__(G == 1 ? 128 : 32 * G)
    norm_fwd_rows(const T* x, T* y, const FwdArgs a) {
  constexpr int RB = G == 1 ? 4 : 1;  // rows per block
  __shared__ float red[2][G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col0 = G == 1 ? 0 : int64_t(warp) * (NV * 32 * V);
  const float inv = 1.0f / float(a.cols);
  for (int64_t r = int64_t(blockIdx.x) * RB + (G == 1 ? warp : 0); r < a.rows;
       r += int64_t(gridDim.x) * RB) {
    const T* row = x + r * a.ldx;
    Vec<T, V> raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = col0 + (j * 32 + lane) * V;
      if (col < a.cols) raw[j].load(row + col);
      else raw[j].zero();
    }
    float v[NV * V], s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j].get(v + j * V);
    if (a.c.codes) ckpt_row<V, NV>(a.c, r, a.cols, col0, v);
#pragma unroll
    for (int i = 0; i < NV * V; ++i) s += v[i];
    const float mu = row_sum<G>(s, red[0], 1) * inv;
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = col0 + (j * 32 + lane) * V < a.cols;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[j * V + i] -= mu;
        if (in) s = fmaf(v[j * V + i], v[j * V + i], s);
      }
    }
    const float rs = rsqrtf(row_sum<G>(s, red[1], 1) * inv + a.eps);
    if (lane == 0 && col0 == 0) {
      if (a.mean) a.mean[r] = mu;
      if (a.rstd) a.rstd[r] = rs;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = col0 + (j * 32 + lane) * V;
      if (col < a.cols) {
        float g[V], b[V];
        params<V>(a.gamma, a.pdtype, col, 1.0f, g);
        params<V>(a.beta, a.pdtype, col, 0.0f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = fmaf(v[j * V + i] * rs, g[i], b[i]);
        put<T, V>(y + r * a.ldy + col, g);
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

// ---------------------------------------------------------------------------
// backward with the row in registers: dx and the column sums in one pass.  A block
// is NG rows' worth of warps (blockDim / 32 G) that walk down the rows; a lane
// keeps its columns' sums for gamma and beta, and the next row's loads are in
// flight while this one is reduced.
// ---------------------------------------------------------------------------
template <typename T, int V, int NV>
struct RowRegs {
  Vec<T, V> dy[NV], x[NV], res[NV];  // x: or, in its first words, the codes
  float s[NV];                       // scale of the codes
  float mu, rs;
  __device__ __forceinline__ void load(const T* pdy, const T* px, const T* pres, const BwdArgs& a,
                                       int64_t r, int64_t col0) {
    const int lane = threadIdx.x & 31;
    if (r >= a.rows) return;
    mu = __ldg(a.mean + r), rs = __ldg(a.rstd + r);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = col0 + (j * 32 + lane) * V;
      s[j] = 0.0f;
      if (col < a.cols) {
        dy[j].load(pdy + r * a.lddy + col);
        if (px) {
          x[j].load(px + r * a.ldx + col);
        } else {
          const uint8_t* c = a.c.codes + r * a.cols + col;
          if constexpr (V == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(c));
            x[j].w[0] = u.x, x[j].w[1] = u.y;
          } else {
            x[j].w[0] = __ldg(c);
          }
          s[j] = __ldg(a.c.scale + r * a.c.groups + (col >> a.c.lg));
        }
        if (pres) res[j].load(pres + r * a.lddres + col);
      } else {
        dy[j].zero(), x[j].zero(), res[j].zero();
      }
    }
  }
  // h of vector j
  __device__ __forceinline__ void hat(const T* px, const BwdArgs& a, int j, float* h) const {
    if (px) {
      x[j].get(h);
    } else if constexpr (V == 8) {
      ckpt_values4(x[j].w[0], s[j], a.c.fmt, h);
      ckpt_values4(x[j].w[1], s[j], a.c.fmt, h + 4);
    } else {
      float t[4];
      ckpt_values4(x[j].w[0], s[j], a.c.fmt, t);
      h[0] = t[0];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = (h[i] - mu) * rs;
  }
};

template <typename T, int V, int NV, int G, bool PF>
__global__ void __launch_bounds__(512, 1)
    norm_bwd_rows(const T* dy, const T* x, const T* dres, T* dx, float* pg, float* pb,
                  const BwdArgs a) {
  constexpr int C = 32 * G * NV * V;  // columns a row may have
  extern __shared__ float sums[];     // [2][C] when several rows share the block
  __shared__ float red[16][2][2];     // [warp][parity][sum]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ng = int(blockDim.x) / (32 * G), grp = warp / G, wr = warp % G;
  const int64_t col0 = int64_t(wr) * (NV * 32 * V);
  const float inv = 1.0f / float(a.cols);
  float ag[NV * V] = {}, ab[NV * V] = {};
  const int64_t step = int64_t(gridDim.x) * ng;
  int64_t r = int64_t(blockIdx.x) * ng + grp;
  RowRegs<T, V, NV> cur;
  cur.load(dy, x, dres, a, r, col0);
  int par = 0;
  for (; r < a.rows; r += step, par ^= 1) {
    RowRegs<T, V, NV> nxt;
    if constexpr (PF) nxt.load(dy, x, dres, a, r + step, col0);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = col0 + (j * 32 + lane) * V;
      if (col < a.cols) {
        float h[V], d[V], g[V];
        cur.hat(x, a, j, h);
        cur.dy[j].get(d);
        params<V>(a.gamma, a.pdtype, col, 1.0f, g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ag[j * V + i] = fmaf(d[i], h[i], ag[j * V + i]);
          ab[j * V + i] += d[i];
          const float u = d[i] * g[i];
          s1 += u;
          s2 = fmaf(u, h[i], s2);
        }
      }
    }
    if (dx) {
      s1 = warp_sum(s1), s2 = warp_sum(s2);
      if constexpr (G > 1) {
        if (lane == 0) red[warp][par][0] = s1, red[warp][par][1] = s2;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * G) : "memory");
        s1 = s2 = 0.0f;
#pragma unroll
        for (int w = 0; w < G; ++w) s1 += red[grp * G + w][par][0], s2 += red[grp * G + w][par][1];
      }
      const float m1 = s1 * inv, m2 = s2 * inv;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t col = col0 + (j * 32 + lane) * V;
        if (col < a.cols) {
          float h[V], d[V], g[V], e[V];
          cur.hat(x, a, j, h);
          cur.dy[j].get(d);
          params<V>(a.gamma, a.pdtype, col, 1.0f, g);
          if (dres) {
            cur.res[j].get(e);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] = fmaf(cur.rs, fmaf(-h[i], m2, fmaf(d[i], g[i], -m1)), e[i]);
          put<T, V>(dx + r * a.lddx + col, d);
        }
      }
    }
    if constexpr (PF) cur = nxt;
    else cur.load(dy, x, dres, a, r + step, col0);
  }
  if (!pg) return;
  // the block's column sums: group after group into shared memory, in order
  if (ng > 1) {
    for (int g = 0; g < ng; ++g) {
      if (g == grp) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int c = int(col0) + (j * 32 + lane) * V + i;
            sums[c] = (g ? sums[c] : 0.0f) + ag[j * V + i];
            sums[C + c] = (g ? sums[C + c] : 0.0f) + ab[j * V + i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      pg[int64_t(blockIdx.x) * a.cols + c] = sums[c];
      pb[int64_t(blockIdx.x) * a.cols + c] = sums[C + c];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = col0 + (j * 32 + lane) * V;
      if (col < a.cols) {
        put<float, V>(pg + int64_t(blockIdx.x) * a.cols + col, ag + j * V);
        put<float, V>(pb + int64_t(blockIdx.x) * a.cols + col, ab + j * V);
      }
    }
  }
}

// row slices of the column sums: at most two per SM, the larger of what the
// kernels below use
int bwd_parts(int64_t rows) {
  const int64_t p = (rows + kT / 32 - 1) / (kT / 32);
  const int64_t q = rows < kSms ? rows : kSms;  // one per block of the register kernel
  const int64_t m = p > q ? p : q;
  return int(m > kMaxParts ? kMaxParts : m);
}

template <typename T, int V, int NV, int G>
cudaError_t run_fwd(const void* x, void* y, const FwdArgs& a, cudaStream_t st) {
  constexpr int RB = G == 1 ? 4 : 1;
  const int64_t blocks = (a.rows + RB - 1) / RB;
  const unsigned grid = unsigned(blocks > 0x7FFFFFFF ? 0x7FFFFFFF : blocks);
  norm_fwd_rows<T, V, NV, G><<<grid, G == 1 ? 128 : 32 * G, 0, st>>>(static_cast<const T*>(x),
                                                                    static_cast<T*>(y), a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_fwd(const void* x, void* y, const FwdArgs& a, cudaStream_t st) {
  const int64_t c = a.cols;
  // wide accesses need whole vectors: columns a multiple of 8 and every row aligned
  if (a.vec && a.pvec && c % 8 == 0 && a.cvec) {
    if (c <= 256) return run_fwd<T, 8, 1, 1>(x, y, a, st);
    if (c <= 512) return run_fwd<T, 8, 2, 1>(x, y, a, st);
    if (c <= 1024) return run_fwd<T, 8, 4, 1>(x, y, a, st);
    if (c <= 2048) return run_fwd<T, 8, 2, 4>(x, y, a, st);
    if (c <= 4096) return run_fwd<T, 8, 2, 8>(x, y, a, st);
    if (c <= 8192) return run_fwd<T, 8, 4, 8>(x, y, a, st);
    if (c <= 16384) return run_fwd<T, 8, 4, 16>(x, y, a, st);
  } else {
    if (c <= 256) return run_fwd<T, 1, 8, 1>(x, y, a, st);
    if (c <= 512) return run_fwd<T, 1, 16, 1>(x, y, a, st);
    if (c <= 1024) return run_fwd<T, 1, 16, 2>(x, y, a, st);
    if (c <= 2048) return run_fwd<T, 1, 16, 4>(x, y, a, st);
    if (c <= 4096) return run_fwd<T, 1, 16, 8>(x, y, a, st);
    if (c <= 8192) return run_fwd<T, 1, 16, 16>(x, y, a, st);
  }
  const unsigned grid = unsigned(a.rows > 0x7FFFFFFF ? 0x7FFFFFFF : a.rows);
  norm_fwd_kernel<T><<<grid, kT, 0, st>>>(static_cast<const T*>(x), static_cast<T*>(y), a);
  return cudaGetLastError();
}

struct BwdOut {
  void* dx;
  float *dgamma, *dbeta, *ws;
  int accumulate;
};

template <typename T, int V, int NV, int G, bool PF>
cudaError_t run_bwd(const void* dy, const void* x, const void* dres, const BwdOut& o, const BwdArgs& a,
                    cudaStream_t st) {
  // rows per block: up to 16 warps, fewer when there are few rows
  int64_t ng = (a.rows + kSms - 1) / kSms;
  if (ng > 16 / G) ng = 16 / G;
  int64_t parts = (a.rows + ng - 1) / ng;
  if (parts > kSms) parts = kSms;
  const bool cols = o.dgamma || o.dbeta;
  float* pb = cols ? o.ws + size_t(parts) * size_t(a.cols) : nullptr;
  const size_t smem = ng > 1 && cols ? size_t(2) * 32 * G * NV * V * 4 : 0;  // 32 KiB at most
  norm_bwd_rows<T, V, NV, G, PF><<<unsigned(parts), unsigned(32 * G * ng), smem, st>>>(
      static_cast<const T*>(dy), static_cast<const T*>(x), static_cast<const T*>(dres),
      static_cast<T*>(o.dx), cols ? o.ws : nullptr, pb, a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !cols) return e;
  return launch_part_sums(o.ws, pb, int(parts), a.cols, o.dgamma, o.dbeta, o.accumulate, st);
}

template <typename T>
cudaError_t launch_bwd(const void* dy, const void* x, const void* dres, const BwdOut& o,
                       const BwdArgs& a, cudaStream_t st) {
  const int64_t c = a.cols;
  if (a.vec && a.pvec && c % 8 == 0 && a.cvec) {
    if (c <= 512) return run_bwd<T, 8, 2, 1, sizeof(T) == 2>(dy, x, dres, o, a, st);
    if (c <= 1024) return run_bwd<T, 8, 2, 2, sizeof(T) == 2>(dy, x, dres, o, a, st);
    if (c <= 2048) return run_bwd<T, 8, 2, 4, sizeof(T) == 2>(dy, x, dres, o, a, st);
    if (c <= 4096) return run_bwd<T, 8, 2, 8, sizeof(T) == 2>(dy, x, dres, o, a, st);
    if (c <= 8192) return run_bwd<T, 8, 2, 16, sizeof(T) == 2>(dy, x, dres, o, a, st);
  } else {
    if (c <= 256) return run_bwd<T, 1, 8, 1, true>(dy, x, dres, o, a, st);
    if (c <= 512) return run_bwd<T, 1, 8, 2, true>(dy, x, dres, o, a, st);
    if (c <= 1024) return run_bwd<T, 1, 8, 4, true>(dy, x, dres, o, a, st);
    if (c <= 2048) return run_bwd<T, 1, 8, 8, true>(dy, x, dres, o, a, st);
    if (c <= 4096) return run_bwd<T, 1, 8, 16, true>(dy, x, dres, o, a, st);
  }
  const T *tdy = static_cast<const T*>(dy), *tx = static_cast<const T*>(x);
  if (o.dx) {
    const unsigned grid = unsigned(a.rows > 0x7FFFFFFF ? 0x7FFFFFFF : a.rows);
    norm_dx_kernel<T><<<grid, kT, 0, st>>>(tdy, tx, static_cast<const T*>(dres),
                                           static_cast<T*>(o.dx), a);
  }
  if (o.dgamma || o.dbeta) {
    const int parts = bwd_parts(a.rows);
    float* pb = o.ws + size_t(parts) * size_t(a.cols);
    norm_cols_kernel<T><<<dim3(unsigned((a.cols + 255) / 256), parts), kT, 0, st>>>(tdy, tx, o.ws,
                                                                                   pb, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_part_sums(o.ws, pb, parts, a.cols, o.dgamma, o.dbeta, o.accumulate, st);
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
  const BwdOut o = {dx, dgamma, dbeta, static_cast<float*>(workspace), accumulate};
  const cudaError_t e = dtype == AQFQ_BF16 ? launch_bwd<bf16>(dy, x, dres, o, a, st)
                                           : launch_bwd<float>(dy, x, dres, o, a, st);
  return e == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA;
}
