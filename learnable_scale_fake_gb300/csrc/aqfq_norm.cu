// aqfq_norm.cu -- layer norm, forward and backward, over the last axis.
//
// Row of C columns: mu = sum x / C, var = sum (x - mu)^2 / C (two passes, so a
// large mean does not cancel), r = (var + eps)^-1/2, y = (x - mu) r gamma + beta.
// Backward, h = (x - mu) r and u = dy gamma:
//   dx = r (u - mean(u) - h mean(u h)) (+ dres)
//   dgamma = sum over rows of dy h,   dbeta = sum over rows of dy
// with x as it was, or as its 8-bit checkpoint gives it back (then mu and r
// are still those of the exact x).
#include <type_traits>

#include "aqfq_internal.h"
#include "aqfq_layer.cuh"
#include "aqfq_sm100_pair.cuh"

namespace aqfq {
namespace layer {
namespace {

constexpr int kT = 256;
constexpr int kSms = 152;  // of a GB300: grids and the workspace's size; the results do not need it

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
        const Divisor d = ckpt_divisor(m, a.c.fmt);
        if (n > 0) {
          const f2 t[4] = {mk2(v[0], v[1]), mk2(v[2], v[3]), mk2(v[4], v[5]), mk2(v[6], v[7])};
          uint32_t w[2];
          ckpt_codes(t, d, a.c.fmt, w);
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
// lane at ((w NV + j) 32 + lane) V.  A block takes R rows at a time (G = 1: each of
// its four warps does): their loads are all under way before the first sum, they
// share the barriers of the two reductions and the conversion of gamma and beta.
// ---------------------------------------------------------------------------
// V parameters as pairs
template <int V, int NV>
__device__ __forceinline__ void params(const void* p, int pdtype, const int64_t (&col)[NV],
                                       const bool (&in)[NV], float def, f2 (&v)[NV * V / 2]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < NV * V / 2; ++i) v[i] = pair(def);
  } else if (pdtype == AQFQ_BF16) {
    Row<bf16, V, NV> w;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j]) w.load(j, static_cast<const bf16*>(p) + col[j]);
      else w.zero(j);
    }
#pragma unroll
    for (int i = 0; i < NV * V / 2; ++i) v[i] = w.pair_at(i);
  } else {
    Row<float, V, NV> w;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j]) w.load(j, static_cast<const float*>(p) + col[j]);
      else w.zero(j);
    }
#pragma unroll
    for (int i = 0; i < NV * V / 2; ++i) v[i] = w.pair_at(i);
  }
}
// whether pair i's elements lie in the row (V = 1: each on its own)
template <int V, int NV>
__device__ __forceinline__ f2 masked(f2 v, int i, const bool (&in)[NV]) {
  if constexpr (V == 8) return in[i / 4] ? v : 0ull;
  else return mk2(in[2 * i] ? lo2(v) : 0.0f, in[2 * i + 1] ? hi2(v) : 0.0f);
}

// a lane's vector j of column sums to scratch, which the caller aligns to 8 bytes only
template <int V>
__device__ __forceinline__ void put_sums(float* p, const f2* v, int j) {
  if constexpr (V == 1) {
    put<float, 1>(p, v, j);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) *reinterpret_cast<f2*>(p + 2 * i) = v[j * (V / 2) + i];
  }
}

template <typename T, int V, int NV, int G, int R>
__global__ void __launch_bounds__(G == 1 ? 128 : 32 * G)
    norm_fwd_rows(const T* x, T* y, const FwdArgs a) {
  constexpr int RB = G == 1 ? 4 : 1, P = NV * V / 2;
  __shared__ float red[2][R][G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv = 1.0f / float(a.cols);
  const int64_t r0 = (int64_t(blockIdx.x) * RB + (G == 1 ? warp : 0)) * R;
  if (G == 1 && r0 >= a.rows) return;
  int64_t col[NV];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    col[j] = ((G == 1 ? 0 : int64_t(warp) * (NV * 32)) + j * 32 + lane) * V;
    in[j] = col[j] < a.cols;
  }
  Row<T, V, NV> raw[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const T* row = x + (r0 + k < a.rows ? r0 + k : a.rows - 1) * a.ldx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j]) raw[k].load(j, row + col[j]);
      else raw[k].zero(j);
    }
  }
  f2 v[R][P];
  float s[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    f2 t = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[k][i] = raw[k].pair_at(i);
      t = add2(t, v[k][i]);
    }
    s[k] = lo2(t) + hi2(t);
  }
  if (a.c.codes) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      bool ink[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) ink[j] = in[j] && r0 + k < a.rows;
      if (a.c.fmt == AQFQ_INT8) ckpt_write<AQFQ_INT8, V, NV>(a.c, r0 + k, a.cols, col, ink, v[k]);
      else ckpt_write<AQFQ_FP8_E4M3, V, NV>(a.c, r0 + k, a.cols, col, ink, v[k]);
    }
  }
  // two passes over the registers: mean, then the sum of squared deviations
  float mu[R], rs[R];
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < R; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
    if constexpr (G > 1) {
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < R; ++k) red[pass][k][warp] = s[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < R; ++k) {
        s[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < G; ++w) s[k] += red[pass][k][w];
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (pass == 0) {
        mu[k] = s[k] * inv;
        f2 t = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          v[k][i] = sub2(v[k][i], pair(mu[k]));
          const f2 d = masked<V, NV>(v[k][i], i, in);
          t = fma2(d, d, t);
        }
        s[k] = lo2(t) + hi2(t);
      } else {
        rs[k] = rsqrtf(fmaf(s[k], inv, a.eps));
      }
    }
  }
  if (lane == 0 && (G == 1 || warp == 0)) {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (r0 + k < a.rows) {
        if (a.mean) a.mean[r0 + k] = mu[k];
        if (a.rstd) a.rstd[r0 + k] = rs[k];
      }
  }
  f2 g[P], b[P];
  params<V, NV>(a.gamma, a.pdtype, col, in, 1.0f, g);
  params<V, NV>(a.beta, a.pdtype, col, in, 0.0f, b);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k >= a.rows) break;
#pragma unroll
    for (int i = 0; i < P; ++i) v[k][i] = fma2(mul2(v[k][i], pair(rs[k])), g[i], b[i]);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in[j]) put<T, V>(y + (r0 + k) * a.ldy + col[j], v[k], j);
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
// flight while this one is reduced (one barrier per row).
// ---------------------------------------------------------------------------
template <typename T, int V, int NV, bool CK>
struct RowRegs {
  Row<T, V, NV> dy, res;
  typename std::conditional<CK, CodeRow<V, NV>, Row<T, V, NV>>::type x;
  float mu, rs;
  // r: a row that exists
  __device__ __forceinline__ void load(const T* pdy, const T* px, const T* pres, const BwdArgs& a,
                                       int64_t r, const int64_t (&col)[NV], const bool (&in)[NV]) {
    mu = __ldg(a.mean + r), rs = __ldg(a.rstd + r);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j]) {
        dy.load(j, pdy + r * a.lddy + col[j]);
        if constexpr (CK) x.load(j, a.c, r, a.cols, col[j]);
        else x.load(j, px + r * a.ldx + col[j]);
        if (pres) res.load(j, pres + r * a.lddres + col[j]);
      } else {
        dy.zero(j), x.zero(j), res.zero(j);
      }
    }
  }
};

// (with 1024 threads, 64 registers each, 30 to 60 of them spilled: 64 x 1024 11 us instead
// of 4.7, 2000 x 4001 from a checkpoint 53 instead of 31.  The kernel of 4097 to 8192 columns
// that allow no wide access still spills: 88 to 144 bytes, from a checkpoint 468 to 592.)
constexpr int kBwdThreads = 512;
template <typename T, int V, int NV, int G, bool CK, bool PF>
__global__ void __launch_bounds__(kBwdThreads, 1)
    norm_bwd_rows(const T* dy, const T* x, const T* dres, T* dx, float* pg, float* pb,
                  const BwdArgs a, const Join jn) {
  constexpr int C = 32 * G * NV * V, P = NV * V / 2;  // columns a row may have
  extern __shared__ float sums[];     // [2][C] when several rows share the block
  __shared__ float2 red[32][2];       // [warp][parity]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ng = int(blockDim.x) / (32 * G), grp = warp / G, wr = warp % G;
  const float inv = 1.0f / float(a.cols);
  int64_t col[NV];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    col[j] = (int64_t(wr) * (NV * 32) + j * 32 + lane) * V;
    in[j] = col[j] < a.cols;
  }
  f2 g[P], ag[P] = {}, ab[P] = {};
  params<V, NV>(a.gamma, a.pdtype, col, in, 1.0f, g);
  const int64_t step = int64_t(gridDim.x) * ng;
  int64_t r = int64_t(blockIdx.x) * ng + grp;
  RowRegs<T, V, NV, CK> cur;
  if (r < a.rows) cur.load(dy, x, dres, a, r, col, in);
  int par = 0;
  for (; r < a.rows; r += step, par ^= 1) {
    RowRegs<T, V, NV, CK> nxt;
    if constexpr (PF) nxt.load(dy, x, dres, a, r + step < a.rows ? r + step : r, col, in);
    f2 h[P], t1 = 0, t2 = 0;
    if constexpr (CK) {
      cur.x.values(a.c.fmt, h);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) h[i] = cur.x.pair_at(i);
    }
    const f2 mu = pair(cur.mu), rs = pair(cur.rs);
    // dy is zero beyond the row, and h has to be finite there: (0 - mu) rstd may overflow where
    // the row's own h do not
    f2 rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) rv[j] = V == 8 && !in[j] ? 0ull : rs;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const f2 d = cur.dy.pair_at(i);
      h[i] = mul2(sub2(h[i], mu), V == 8 ? rv[i / 4] : rs);
      if constexpr (V == 1) h[i] = masked<V, NV>(h[i], i, in);
      ag[i] = fma2(d, h[i], ag[i]);
      ab[i] = add2(ab[i], d);
      const f2 u = mul2(d, g[i]);
      t1 = add2(t1, u);
      t2 = fma2(u, h[i], t2);
    }
    if (dx) {
      float s1 = lo2(t1) + hi2(t1), s2 = lo2(t2) + hi2(t2);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
        s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
      }
      if constexpr (G > 1) {
        if (lane == 0) red[warp][par] = make_float2(s1, s2);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * G) : "memory");
        s1 = s2 = 0.0f;
#pragma unroll
        for (int w = 0; w < G; ++w) {
          const float2 p = red[grp * G + w][par];
          s1 += p.x, s2 += p.y;
        }
      }
      const f2 m1 = pair(-s1 * inv), m2 = pair(-s2 * inv);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const f2 t = fma2(h[i], m2, fma2(cur.dy.pair_at(i), g[i], m1));
        h[i] = dres ? fma2(rs, t, cur.res.pair_at(i)) : mul2(rs, t);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (in[j]) put<T, V>(dx + r * a.lddx + col[j], h, j);
    }
    if constexpr (PF) cur = nxt;
    else if (r + step < a.rows) cur.load(dy, x, dres, a, r + step, col, in);
  }
  if (!pg && !jn.on) return;  // uniform over the grid
  // the block's column sums: group after group into shared memory, in order
  if (ng > 1 || jn.on) {
    for (int k = 0; k < ng; ++k) {
      if (k == grp) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c0 = V == 8 ? int(col[i / 4]) + 2 * (i % 4) : int(col[2 * i % NV]);
          const int c1 = V == 8 ? c0 + 1 : int(col[(2 * i + 1) % NV]);
          sums[c0] = (k ? sums[c0] : 0.0f) + lo2(ag[i]);
          sums[c1] = (k ? sums[c1] : 0.0f) + hi2(ag[i]);
          sums[C + c0] = (k ? sums[C + c0] : 0.0f) + lo2(ab[i]);
          sums[C + c1] = (k ? sums[C + c1] : 0.0f) + hi2(ab[i]);
        }
      }
      __syncthreads();
    }
    if (jn.on) {
      join_columns(jn, sums, C, a.cols);
      return;
    }
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      pg[int64_t(blockIdx.x) * a.cols + c] = sums[c];
      pb[int64_t(blockIdx.x) * a.cols + c] = sums[C + c];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j]) {
        put_sums<V>(pg + int64_t(blockIdx.x) * a.cols + col[j], ag, j);
        put_sums<V>(pb + int64_t(blockIdx.x) * a.cols + col[j], ab, j);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows: persistent blocks whose rows arrive by bulk asynchronous copies.  A
// group of G warps owns a ring of stages in shared memory, one row (x; or dy, the
// kept input and the residual's gradient) per stage; a lane works on NV vectors of 8
// columns.  The copies need no registers, so the bytes in flight per SM (the
// rings, about 200 KB) cover the memory latency whatever the row's arithmetic
// holds.  The barrier of a row's reduction also says that the row before it has been
// read by every warp, so one thread refills that stage right after it.
// A wait gives up after about a second; the rows left are then written as NaN.
// ---------------------------------------------------------------------------
constexpr int kMaxStages = 16;
constexpr int kFwdBlocks = 2;           // blocks per SM of the forward ring
constexpr int kRingBytes = 200 * 1024;  // per SM

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
      : "memory");
}

template <int G>
__device__ __forceinline__ void group_sync(int grp) {
  if constexpr (G == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * G) : "memory");
}
// pairs of V = 8 vectors of a row in shared memory
// (MASK: zeros where the vector lies beyond the row)
template <bool MASK, typename T, int NV>
__device__ __forceinline__ void smem_pairs(const uint8_t* row, const int (&col)[NV], const bool (&in)[NV],
                                           f2 (&v)[NV * 4]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint4* p = reinterpret_cast<const uint4*>(row + col[j] * int(sizeof(T)));
    uint4 a = p[0];
    if (MASK && !in[j]) a = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(T) == 2) {
      v[4 * j] = bf2(a.x), v[4 * j + 1] = bf2(a.y), v[4 * j + 2] = bf2(a.z), v[4 * j + 3] = bf2(a.w);
    } else {
      uint4 b = p[1];
      if (MASK && !in[j]) b = make_uint4(0, 0, 0, 0);
      v[4 * j] = mk2(__uint_as_float(a.x), __uint_as_float(a.y));
      v[4 * j + 1] = mk2(__uint_as_float(a.z), __uint_as_float(a.w));
      v[4 * j + 2] = mk2(__uint_as_float(b.x), __uint_as_float(b.y));
      v[4 * j + 3] = mk2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
  }
}

// Loads on their way when a wait for row r gives up: the rows left, at most one per stage, and
// after the first turn the stage of the row before r has not been refilled yet.
__device__ __forceinline__ int64_t in_flight(int stages, bool first, int64_t r, int64_t step, int64_t rows) {
  const int64_t left = (rows - r + step - 1) / step, most = first ? stages : stages - 1;
  return left < most ? left : most;
}

struct RingArgs {
  int stages, stage_bytes;  // per group
  int row_bytes;            // of a tensor's row; a multiple of 16
};

// sums of two values over a group: half a warp carries each of them, so that five
// exchanges serve both; the totals of every warp through red[2][G]
template <int G>
__device__ __forceinline__ void group_sum2(float (&s)[2], float* red, int grp) {
  const int lane = threadIdx.x & 31;
  const bool up = lane >= 16;
  float t = (up ? s[1] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? s[0] : s[1], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  if constexpr (G == 1) {
    s[0] = __shfl_sync(0xFFFFFFFFu, t, 0);
    s[1] = __shfl_sync(0xFFFFFFFFu, t, 16);
    group_sync<G>(grp);
  } else {
    if ((lane & 15) == 0) red[(up ? G : 0) + (threadIdx.x >> 5) % G] = t;
    group_sync<G>(grp);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f2* p = reinterpret_cast<const f2*>(red + k * G);
      f2 u = p[0];
#pragma unroll
      for (int w = 1; w < G / 2; ++w) u = add2(u, p[w]);
      s[k] = lo2(u) + hi2(u);
    }
  }
}

// NW warps per block, MB blocks per SM.  A lane has 16 consecutive columns; a stage is
// two rows, which share the waits, the barriers and the sums' exchanges.  CK: the
// checkpoint's format, or -1 (a run-time choice kept the two rows' arithmetic apart).
// At 8192 x 4096 in BF16: 25 us (5.4 TB/s), with a checkpoint 35 us (4.8 TB/s): the two
// reductions and the quantizer's chain of divisions leave half the issue slots empty.
template <typename T, int G, int NW, int MB, int CK>
__global__ void __launch_bounds__(32 * NW, MB)
    norm_fwd_ring(const T* x, T* y, const FwdArgs a, const RingArgs q) {
  constexpr int NG = NW / G, P = 8, R = 2;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[NG][kMaxStages];
  __shared__ __align__(8) float red[NG][2][R * G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / G, wr = warp % G;
  uint8_t* mine = ring + size_t(grp) * q.stages * q.stage_bytes;
  if (threadIdx.x == 0) {
    for (int g = 0; g < NG; ++g)
      for (int i = 0; i < q.stages; ++i) sm100::mbar_init(&full[g][i], 1);
    sm100::fence_barrier_init();
  }
  __syncthreads();
  const int64_t step = int64_t(gridDim.x) * NG * R;
  int64_t r = (int64_t(blockIdx.x) * NG + grp) * R;
  const bool loader = wr == 0 && lane == 0;
  auto fetch = [&](int64_t row, int st) {
    if (row < a.rows) {
      uint64_t* bar = &full[grp][st];
      const uint32_t dst = sm100::smem_u32(mine + st * q.stage_bytes), n = uint32_t(q.row_bytes);
      const bool two = row + 1 < a.rows;
      sm100::mbar_arrive_expect_tx(bar, two ? 2 * n : n);
      bulk_load(dst, x + row * a.ldx, n, bar);
      if (two) bulk_load(dst + n, x + (row + 1) * a.ldx, n, bar);
    }
  };
  if (loader)
    for (int i = 0; i < q.stages; ++i) fetch(r + i * step, i);
  const float inv = 1.0f / float(a.cols);
  const int col = (wr * 32 + lane) * 16;
  const bool in[2] = {col < a.cols, col + 8 < a.cols};
  const int cl[2] = {in[0] ? col : 0, in[1] ? col + 8 : 0};
  const int64_t col64[2] = {cl[0], cl[1]};
  f2 g[P], b[P];
  params<8, 2>(a.gamma, a.pdtype, col64, in, 1.0f, g);
  params<8, 2>(a.beta, a.pdtype, col64, in, 0.0f, b);
  T* yrow = y + r * a.ldy + col;
  const int64_t ystep = step * a.ldy;
  // 32-byte stores where the rows allow them
  const bool wide = sizeof(T) == 2 && in[1] &&
                    ((reinterpret_cast<uintptr_t>(yrow) | uintptr_t(a.ldy * sizeof(T))) & 31) == 0;
  // the checkpoint's place, advanced with the rows
  uint8_t* code = CK >= 0 ? a.c.codes + r * a.cols + col : nullptr;
  float* scale = CK >= 0 ? a.c.scale + r * a.c.groups + (col >> a.c.lg) : nullptr;
  const int64_t cstep = step * a.cols, sstep = step * a.c.groups;
  const bool c16 = a.cols % 16 == 0 && (reinterpret_cast<uintptr_t>(a.c.codes) & 15) == 0;
  const bool lead = (col & ((1 << a.c.lg) - 1)) == 0;
  int st = 0, prev = q.stages - 1;
  uint32_t phase = 0;
  bool ok = true;
  for (bool first = true; r < a.rows; r += step, yrow += ystep, first = false) {
    if (ok && !sm100::mbar_test(&full[grp][st], phase)) {
      ok = sm100::mbar_wait_suspend(&full[grp][st], phase);
      if (!ok && loader) sm100::drain_ring(full[grp], q.stages, st, phase, in_flight(q.stages, first, r, step, a.rows));
    }
    const bool two = r + 1 < a.rows;
    f2 v[R][P];
    float s[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      smem_pairs<true, T, 2>(mine + st * q.stage_bytes + k * q.row_bytes, cl, in, v[k]);
      if (!ok) v[k][0] = pair(__int_as_float(0x7FC00000));
      f2 t = v[k][0];
#pragma unroll
      for (int i = 1; i < P; ++i) t = add2(t, v[k][i]);
      s[k] = lo2(t) + hi2(t);
    }
    if constexpr (CK >= 0) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const bool e = k == 0 || two;  // uniform
        ckpt_write16<CK>(a.c.lg, code + (k ? a.cols : 0), c16, scale + (k ? a.c.groups : 0), lead,
                         in[0] && e, in[1] && e, v[k]);
      }
      code += cstep, scale += sstep;
    }
    group_sum2<G>(s, red[grp][0], grp);
    // every warp has read the rows before these
    if (loader && !first && ok) fetch(r + (q.stages - 1) * step, prev);
    float mu[R], rs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mu[k] = s[k] * inv;
      s[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f2 t = 0;
#pragma unroll
        for (int i = 4 * j; i < 4 * j + 4; ++i) {
          v[k][i] = sub2(v[k][i], pair(mu[k]));
          t = fma2(v[k][i], v[k][i], t);
        }
        s[k] += in[j] ? lo2(t) + hi2(t) : 0.0f;
      }
    }
    group_sum2<G>(s, red[grp][1], grp);
#pragma unroll
    for (int k = 0; k < R; ++k) rs[k] = rsqrtf(fmaf(s[k], inv, a.eps));
    if (wr == 0 && lane < R && r + lane < a.rows) {
      if (a.mean) a.mean[r + lane] = lane ? mu[1] : mu[0];
      if (a.rstd) a.rstd[r + lane] = lane ? rs[1] : rs[0];
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (k == 1 && !two) break;
      const f2 f = pair(rs[k]);
#pragma unroll
      for (int i = 0; i < P; ++i) v[k][i] = fma2(mul2(v[k][i], f), g[i], b[i]);
      T* p = yrow + (k ? a.ldy : 0);
      if (wide) {
        const uint32_t w[8] = {pack2(v[k][0]), pack2(v[k][1]), pack2(v[k][2]), pack2(v[k][3]),
                               pack2(v[k][4]), pack2(v[k][5]), pack2(v[k][6]), pack2(v[k][7])};
        st_256(p, w);
      } else {
        if (in[0]) put<T, 8>(p, v[k], 0);
        if (in[1]) put<T, 8>(p + 8, v[k], 1);
      }
    }
    prev = st;
    if (++st == q.stages) st = 0, phase ^= 1;
  }
}

// One row per stage and turn; CK as above.  At 8192 x 4096 in BF16 with the residual's
// gradient: 47 us from x (5.7 TB/s), 47 us from a checkpoint (5.0 TB/s; the format as a
// run-time choice 51 us).  The 128 registers hold the sums for gamma and beta, gamma and one
// row: with two rows per turn, as forward, a few registers spilled or gamma moved to shared
// memory, 54 to 61 us.  Issue slots are 57 % busy, the packed arithmetic and the exchanges
// of the row's two sums bound it.
template <typename T, int NV, int G, int CK>
__global__ void __launch_bounds__(512, 1)
    norm_bwd_ring(const T* dy, const T* x, const T* dres, T* dx, float* pg, float* pb, const BwdArgs a,
                  const RingArgs q) {
  constexpr int NG = 16 / G, P = NV * 4, C = 32 * G * NV * 8;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[NG][kMaxStages];
  __shared__ __align__(8) float red[NG][2][G * 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / G, wr = warp % G;
  uint8_t* mine = ring + size_t(grp) * q.stages * q.stage_bytes;
  if (threadIdx.x == 0) {
    for (int g = 0; g < NG; ++g)
      for (int i = 0; i < q.stages; ++i) sm100::mbar_init(&full[g][i], 1);
    sm100::fence_barrier_init();
  }
  __syncthreads();
  const int64_t step = int64_t(gridDim.x) * NG;
  int64_t r = int64_t(blockIdx.x) * NG + grp;
  const bool loader = wr == 0 && lane == 0;
  const uint32_t xbytes = CK >= 0 ? uint32_t(a.cols) : uint32_t(q.row_bytes);
  // a stage: dy, the residual's gradient, the kept input
  const int off_res = q.row_bytes, off_x = dres ? 2 * q.row_bytes : q.row_bytes;
  auto fetch = [&](int64_t row, int st) {
    if (row < a.rows) {
      uint64_t* bar = &full[grp][st];
      const uint32_t dst = sm100::smem_u32(mine + st * q.stage_bytes);
      sm100::mbar_arrive_expect_tx(bar, uint32_t(off_x) + xbytes);
      bulk_load(dst, dy + row * a.lddy, uint32_t(q.row_bytes), bar);
      if (dres) bulk_load(dst + off_res, dres + row * a.lddres, uint32_t(q.row_bytes), bar);
      if (CK >= 0) bulk_load(dst + off_x, a.c.codes + row * a.cols, xbytes, bar);
      else bulk_load(dst + off_x, x + row * a.ldx, xbytes, bar);
    }
  };
  if (loader)
    for (int i = 0; i < q.stages; ++i) fetch(r + i * step, i);
  const float inv = 1.0f / float(a.cols);
  int col[NV];
  int64_t col64[NV];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    col64[j] = (wr * NV * 32 + j * 32 + lane) * 8;
    in[j] = col64[j] < a.cols;
    col[j] = in[j] ? int(col64[j]) : 0;
  }
  f2 g[P], ag[P] = {}, ab[P] = {};
  params<8, NV>(a.gamma, a.pdtype, col64, in, 1.0f, g);
  // the row's scalars are fetched one row ahead
  float mu_n = 0.0f, rs_n = 0.0f, sc_n[NV];
  auto scalars = [&](int64_t row) {
    if (row < a.rows) {
      mu_n = __ldg(a.mean + row), rs_n = __ldg(a.rstd + row);
      if constexpr (CK >= 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) sc_n[j] = __ldg(a.c.scale + row * a.c.groups + (col[j] >> a.c.lg));
      }
    }
  };
  scalars(r);
  T* dxrow = dx + r * a.lddx;
  const int64_t dxstep = step * a.lddx;
  int st = 0, prev = q.stages - 1, par = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (bool first = true; r < a.rows; r += step, dxrow += dxstep, first = false, par ^= 1) {
    const f2 mu = pair(mu_n), rs = pair(rs_n);
    float sc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) sc[j] = CK >= 0 ? sc_n[j] : 0.0f;
    scalars(r + step);
    if (ok && !sm100::mbar_test(&full[grp][st], phase)) {
      ok = sm100::mbar_wait_suspend(&full[grp][st], phase);
      if (!ok && loader) sm100::drain_ring(full[grp], q.stages, st, phase, in_flight(q.stages, first, r, step, a.rows));
    }
    const uint8_t* stage = mine + st * q.stage_bytes;
    f2 d[P], h[P], t1 = 0, t2 = 0;
    smem_pairs<true, T, NV>(stage, col, in, d);  // zero beyond the row: nothing there counts
    if constexpr (CK >= 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint2 w = *reinterpret_cast<const uint2*>(stage + off_x + col[j]);
        ckpt_values4(w.x, sc[j], CK, h + 4 * j);
        ckpt_values4(w.y, sc[j], CK, h + 4 * j + 2);
      }
    } else {
      smem_pairs<false, T, NV>(stage + off_x, col, in, h);
    }
    if (!ok) h[0] = d[0] = pair(__int_as_float(0x7FC00000));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      h[i] = mul2(sub2(h[i], mu), rs);
      ag[i] = fma2(d[i], h[i], ag[i]);
      ab[i] = add2(ab[i], d[i]);
      d[i] = mul2(d[i], g[i]);
      t1 = add2(t1, d[i]);
      t2 = fma2(d[i], h[i], t2);
    }
    float s[2] = {lo2(t1) + hi2(t1), lo2(t2) + hi2(t2)};
    group_sum2<G>(s, red[grp][par], grp);
    // every warp has read the row before this one
    if (loader && !first && ok) fetch(r + (q.stages - 1) * step, prev);
    if (dx) {
      const f2 m1 = pair(-s[0] * inv), m2 = pair(-s[1] * inv);
      f2 e[P];
      if (dres) smem_pairs<false, T, NV>(stage + off_res, col, in, e);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const f2 t = fma2(h[i], m2, add2(d[i], m1));
        h[i] = dres ? fma2(rs, t, e[i]) : mul2(rs, t);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (in[j]) put<T, 8>(dxrow + col[j], h, j);
    }
    prev = st;
    if (++st == q.stages) st = 0, phase ^= 1;
  }
  if (!pg) return;
  float* sums = reinterpret_cast<float*>(ring);
  if constexpr (NG > 1) {
    // group after group into shared memory (every copy has landed and been read), in order
    __syncthreads();
    for (int k = 0; k < NG; ++k) {
      if (k == grp) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2* p = reinterpret_cast<float2*>(sums + col64[j] + 2 * i);
            float2* p2 = reinterpret_cast<float2*>(sums + C + col64[j] + 2 * i);
            const float2 o = k ? *p : make_float2(0.0f, 0.0f), o2 = k ? *p2 : make_float2(0.0f, 0.0f);
            *p = make_float2(o.x + lo2(ag[4 * j + i]), o.y + hi2(ag[4 * j + i]));
            *p2 = make_float2(o2.x + lo2(ab[4 * j + i]), o2.y + hi2(ab[4 * j + i]));
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
      if (in[j]) {
        put_sums<8>(pg + int64_t(blockIdx.x) * a.cols + col[j], ag, j);
        put_sums<8>(pb + int64_t(blockIdx.x) * a.cols + col[j], ab, j);
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

template <typename T, int V, int NV, int G, int R>
cudaError_t run_fwd(const void* x, void* y, const FwdArgs& a, cudaStream_t st) {
  constexpr int RB = G == 1 ? 4 * R : R;
  norm_fwd_rows<T, V, NV, G, R><<<unsigned((a.rows + RB - 1) / RB), G == 1 ? 128 : 32 * G, 0, st>>>(
      static_cast<const T*>(x), static_cast<T*>(y), a);
  return cudaGetLastError();
}

// the ring's stages for `groups` groups in `bytes` of shared memory; fewer than 3: no ring
inline RingArgs make_ring(int stage_bytes, int row_bytes, int groups, int bytes) {
  RingArgs q;
  q.stage_bytes = (stage_bytes + 127) / 128 * 128;
  q.row_bytes = row_bytes;
  q.stages = bytes / (groups * q.stage_bytes);
  if (q.stages > kMaxStages) q.stages = kMaxStages;
  return q;
}

template <typename K>
cudaError_t ring_smem(DeviceOnce& once, K kernel) {
  return once_per_device(once, [=] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  });
}

template <typename T, int G, int NW, int MB>
cudaError_t run_fwd_ring(const void* x, void* y, const FwdArgs& a, const RingArgs& q, cudaStream_t st) {
  constexpr int NG = NW / G;
  static DeviceOnce once[3];
  const int k = !a.c.codes ? 0 : a.c.fmt == AQFQ_INT8 ? 1 : 2;
  auto kernel = k == 0   ? norm_fwd_ring<T, G, NW, MB, -1>
                : k == 1 ? norm_fwd_ring<T, G, NW, MB, AQFQ_INT8>
                         : norm_fwd_ring<T, G, NW, MB, AQFQ_FP8_E4M3>;
  const cudaError_t attr = ring_smem(once[k], kernel);
  if (attr != cudaSuccess) return attr;
  int64_t blocks = (a.rows + 2 * NG - 1) / (2 * NG);
  if (blocks > MB * kSms) blocks = MB * kSms;
  kernel<<<unsigned(blocks), 32 * NW, size_t(NG) * q.stages * q.stage_bytes, st>>>(
      static_cast<const T*>(x), static_cast<T*>(y), a, q);
  return cudaGetLastError();
}

// Whether a ring serves [rows, cols]: enough rows that every group has several.
// fwd: groups on the GPU; the ring's set-up costs about a microsecond
inline bool ring_rows(int64_t rows, int64_t groups) { return rows >= 4 * groups; }

// Warps per row of the ring that serves the forward pass of aligned tensors; 0: none.
// (1024 columns and fewer: norm_fwd_rows is faster, 16384 x 768 14.9 us against 16.4)
int fwd_ring(int64_t rows, int64_t c, int esize, RingArgs& q) {
  if (c % 8 != 0 || c <= 1024 || c > 8192) return 0;
  // blocks of 8 warps, or of 16 for the widest rows
  const int G = c <= 2048 ? 4 : c <= 4096 ? 8 : 16;
  const int nw = G == 16 ? 16 : 8, mb = G == 16 ? 1 : kFwdBlocks, row = int(c) * esize;
  q = make_ring(2 * row, row, nw / G, kRingBytes / mb);
  return q.stages >= 3 && ring_rows(rows, 2 * kSms * mb * (nw / G)) ? G : 0;
}

// The same of the backward pass.  Bulk copies: every row's bytes and its start a multiple
// of 16 (kept codes: columns); 16 columns per lane.
int bwd_ring(int64_t rows, int64_t c, int esize, bool ckpt, bool dres, RingArgs& q) {
  if (c % (ckpt ? 16 : 8) != 0 || c <= 256 || c > 8192) return 0;
  const int G = c <= 512 ? 1 : c <= 1024 ? 2 : c <= 2048 ? 4 : c <= 4096 ? 8 : 16;
  const int row = int(c) * esize;
  q = make_ring(row * (dres ? 2 : 1) + (ckpt ? int(c) : row), row, 16 / G, kRingBytes);
  return q.stages >= 3 && ring_rows(rows, kSms * (16 / G)) ? G : 0;
}

template <typename T>
cudaError_t launch_fwd(const void* x, void* y, const FwdArgs& a, cudaStream_t st) {
  const int64_t c = a.cols;
  if (a.vec && a.pvec && a.cvec) {
    RingArgs q;
    const int G = fwd_ring(a.rows, c, sizeof(T), q);
    if (G == 4) return run_fwd_ring<T, 4, 8, kFwdBlocks>(x, y, a, q, st);
    if (G == 8) return run_fwd_ring<T, 8, 8, kFwdBlocks>(x, y, a, q, st);
    if (G == 16) return run_fwd_ring<T, 16, 16, 1>(x, y, a, q, st);
  }
  // one block per (few) rows: the grid has to hold them
  const bool regs = a.rows <= 0x7FFFFFFF;
  // wide accesses need whole vectors: columns a multiple of 8 and every row aligned
  if (regs && a.vec && a.pvec && c % 8 == 0 && a.cvec) {
    if (c <= 256) return run_fwd<T, 8, 1, 1, 2>(x, y, a, st);
    if (c <= 512) return run_fwd<T, 8, 2, 1, 1>(x, y, a, st);
    if (c <= 1024) return run_fwd<T, 8, 2, 2, 2>(x, y, a, st);
    if (c <= 2048) return run_fwd<T, 8, 2, 4, 2>(x, y, a, st);
    if (c <= 4096) return run_fwd<T, 8, 2, 8, 2>(x, y, a, st);
    if (c <= 8192) return run_fwd<T, 8, 2, 16, 2>(x, y, a, st);
    if (c <= 16384) return run_fwd<T, 8, 4, 16, 1>(x, y, a, st);
  } else if (regs) {
    if (c <= 256) return run_fwd<T, 1, 8, 1, 2>(x, y, a, st);
    if (c <= 512) return run_fwd<T, 1, 8, 2, 2>(x, y, a, st);
    if (c <= 1024) return run_fwd<T, 1, 8, 4, 2>(x, y, a, st);
    if (c <= 2048) return run_fwd<T, 1, 8, 8, 2>(x, y, a, st);
    if (c <= 4096) return run_fwd<T, 1, 8, 16, 2>(x, y, a, st);
    if (c <= 8192) return run_fwd<T, 1, 16, 16, 1>(x, y, a, st);
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
  // rows per block: up to 32 warps (and 15 named barriers), fewer when there are few rows
  constexpr int most = G == 1 ? 16 : kBwdThreads / 32 / G, C = 32 * G * NV * V;
  const bool cols = o.dgamma || o.dbeta;
  int64_t ng = (a.rows + kSms - 1) / kSms;
  Join jn = {o.dgamma, o.dbeta, o.accumulate, false};
  // at most one row per group of a cluster's eight blocks: one launch, the blocks' column
  // sums meet in the cluster (32 x 1024 6.1 us on the GPU against 4.2 for two launches, the
  // second of which costs the host 3.3 us; at four rows per group 7.9 against 4.6)
  if (cols && C <= 4096 && a.rows <= 8 * most) {
    jn.on = true;
    ng = a.rows < most ? a.rows : most;
  }
  if (ng > most) ng = most;
  int64_t parts = (a.rows + ng - 1) / ng;
  if (parts > kSms) parts = kSms;
  if (jn.on && parts > 8) parts = 8;
  float* pg = cols && !jn.on ? o.ws : nullptr;
  float* pb = pg ? o.ws + size_t(parts) * size_t(a.cols) : nullptr;
  const size_t smem = (ng > 1 && cols) || jn.on ? size_t(2) * C * 4 : 0;  // 32 KiB at most
  auto kernel = x ? norm_bwd_rows<T, V, NV, G, false, PF> : norm_bwd_rows<T, V, NV, G, true, PF>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(parts)), cfg.blockDim = dim3(unsigned(32 * G * ng));
  cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(jn.on ? parts : 1), at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const T*>(dy), static_cast<const T*>(x),
                                           static_cast<const T*>(dres), static_cast<T*>(o.dx), pg, pb, a, jn);
  if (e != cudaSuccess || !pg) return e;
  return launch_part_sums(pg, pb, int(parts), a.cols, o.dgamma, o.dbeta, o.accumulate, st);
}

template <typename T, int NV, int G, int CK>
cudaError_t run_bwd_ring(const void* dy, const void* x, const void* dres, const BwdOut& o,
                         const BwdArgs& a, const RingArgs& q, cudaStream_t st) {
  constexpr int NG = 16 / G;
  static DeviceOnce once;
  const cudaError_t attr = ring_smem(once, norm_bwd_ring<T, NV, G, CK>);
  if (attr != cudaSuccess) return attr;
  const bool cols = o.dgamma || o.dbeta;
  int64_t parts = (a.rows + NG - 1) / NG;
  if (parts > kSms) parts = kSms;
  float* pb = cols ? o.ws + size_t(parts) * size_t(a.cols) : nullptr;
  size_t smem = size_t(NG) * q.stages * q.stage_bytes;
  if (NG > 1 && smem < size_t(2) * 32 * G * NV * 8 * 4) smem = size_t(2) * 32 * G * NV * 8 * 4;
  norm_bwd_ring<T, NV, G, CK><<<unsigned(parts), 512, smem, st>>>(
      static_cast<const T*>(dy), static_cast<const T*>(x), static_cast<const T*>(dres),
      static_cast<T*>(o.dx), cols ? o.ws : nullptr, pb, a, q);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !cols) return e;
  return launch_part_sums(o.ws, pb, int(parts), a.cols, o.dgamma, o.dbeta, o.accumulate, st);
}

template <typename T, int NV, int G>
cudaError_t run_bwd_ring(const void* dy, const void* x, const void* dres, const BwdOut& o,
                         const BwdArgs& a, const RingArgs& q, cudaStream_t st) {
  if (x) return run_bwd_ring<T, NV, G, -1>(dy, x, dres, o, a, q, st);
  return a.c.fmt == AQFQ_INT8 ? run_bwd_ring<T, NV, G, AQFQ_INT8>(dy, x, dres, o, a, q, st)
                              : run_bwd_ring<T, NV, G, AQFQ_FP8_E4M3>(dy, x, dres, o, a, q, st);
}

template <typename T>
cudaError_t launch_bwd(const void* dy, const void* x, const void* dres, const BwdOut& o,
                       const BwdArgs& a, cudaStream_t st) {
  const int64_t c = a.cols;
  if (a.vec && a.pvec && (x || al(a.c.codes, 16))) {
    RingArgs q;
    const int G = bwd_ring(a.rows, c, sizeof(T), !x, dres != nullptr, q);
    if (G == 1) return run_bwd_ring<T, 2, 1>(dy, x, dres, o, a, q, st);
    if (G == 2) return run_bwd_ring<T, 2, 2>(dy, x, dres, o, a, q, st);
    if (G == 4) return run_bwd_ring<T, 2, 4>(dy, x, dres, o, a, q, st);
    if (G == 8) return run_bwd_ring<T, 2, 8>(dy, x, dres, o, a, q, st);
    if (G == 16) return run_bwd_ring<T, 2, 16>(dy, x, dres, o, a, q, st);
  }
  if (a.vec && a.pvec && c % 8 == 0 && a.cvec) {
    if (c <= 256) return run_bwd<T, 8, 1, 1, true>(dy, x, dres, o, a, st);
    if (c <= 512) return run_bwd<T, 8, 1, 2, true>(dy, x, dres, o, a, st);
    if (c <= 1024) return run_bwd<T, 8, 1, 4, true>(dy, x, dres, o, a, st);
    if (c <= 2048) return run_bwd<T, 8, 1, 8, true>(dy, x, dres, o, a, st);
    if (c <= 4096) return run_bwd<T, 8, 1, 16, true>(dy, x, dres, o, a, st);
    if (c <= 8192) return run_bwd<T, 8, 2, 16, sizeof(T) == 2>(dy, x, dres, o, a, st);
  } else {
    if (c <= 128) return run_bwd<T, 1, 4, 1, true>(dy, x, dres, o, a, st);
    if (c <= 512) return run_bwd<T, 1, 4, 4, true>(dy, x, dres, o, a, st);
    if (c <= 1024) return run_bwd<T, 1, 4, 8, true>(dy, x, dres, o, a, st);
    if (c <= 2048) return run_bwd<T, 1, 4, 16, true>(dy, x, dres, o, a, st);
    if (c <= 4096) return run_bwd<T, 1, 8, 16, true>(dy, x, dres, o, a, st);
    if (c <= 8192) return run_bwd<T, 1, 16, 16, false>(dy, x, dres, o, a, st);
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

extern "C" int32_t aqfq_selftest_layernorm_ring(int backward, int dtype, int64_t rows, int64_t cols,
                                                int ckpt, int dres) {
  if (!view_ok(rows, cols, cols) || !dtype_ok(dtype)) return 0;
  RingArgs q;
  return backward ? bwd_ring(rows, cols, esize(dtype), ckpt != 0, dres != 0, q)
                  : fwd_ring(rows, cols, esize(dtype), q);
}

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
