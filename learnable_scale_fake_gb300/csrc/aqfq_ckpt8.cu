// aqfq_ckpt8.cu -- activation checkpoints in 8 bits: pack, unpack (with the
// activation recomputed) and the activation gradient read from a checkpoint.
//
// A row is cut into groups of 32, 64 or 128 columns (the last one may be
// shorter).  One lane holds 8 or 16 consecutive columns, so a group is 2 to 16
// neighbouring lanes and its amax a butterfly over them.  A warp covers 256 or 512
// columns of one row (narrow rows: several rows per warp) and walks down the
// rows of its slice; the bias gradient's column sums stay in its registers.
// Memory is the floor: pack moves 2 + 1 bytes per BF16 element, unpack 1 + 2, the
// gradient 1 + 2 + 2 (+ 2 with the recomputed activation).  At 8192 x 8192 in E4M3, a
// plain copy moving 6.78 TB/s: pack 35 us (5.7 TB/s), unpack 33 us (6.0), the gradient
// with SiLU 59 us (5.7), with GELU 75 us (4.5: two transcendental instructions and about
// fifteen packed ones per pair keep the issue slots 60 % busy), with GELU, the recomputed
// activation and the bias gradient 86 us (5.4).  FP32 from INT8: pack 55 us (6.2), unpack 70
// (4.8), with GELU 71, the gradient with GELU, activation and bias gradient 143 (6.1).
// The gradient through a gate moves 2 + 2 + 4 bytes, 2 more with the product: with SiLU 110-114 us
// (5.9-6.1 TB/s).
#include <type_traits>

#include "aqfq_internal.h"
#include "aqfq_layer.cuh"

namespace aqfq {
namespace layer {
namespace {

constexpr int kWarps = 8;
// rows in flight per lane
constexpr int kU = 2, kUB = 2;

// How a [rows, cols] matrix is covered.  V = 8 (rows allow 16-byte accesses) or 16
// (BF16 rows that allow 32-byte ones): a lane holds V columns, 2^lr lanes share a row
// (narrow rows: several per warp).
// V = 1: a warp holds 128 columns of one row as four vectors of 32.
struct Map {
  int lr;          // log2 of the lanes that share a row
  unsigned gx;     // column segments
  unsigned gy;     // row slices
};

// Enough blocks for eight per SM; the bias gradient's partial sums bound the slices.
inline Map make_map(int64_t rows, int64_t cols, int lg, int v, int64_t max_parts) {
  Map m;
  m.lr = v == 16 ? lg - 4 : v == 8 ? lg - 3 : 5;
  const int least = m.lr;  // a group's lanes
  while (m.lr < 5 && (int64_t(v) << m.lr) < cols) ++m.lr;
  // fewer lanes per row where more than an eighth of them would have no columns
  auto idle = [&] { return (cols + (int64_t(v) << m.lr) - 1) / (int64_t(v) << m.lr) * (int64_t(v) << m.lr) - cols; };
  while (v > 1 && m.lr > least && idle() * 8 > cols) --m.lr;
  const int64_t seg = v > 1 ? int64_t(v) << m.lr : 128;
  m.gx = unsigned((cols + seg - 1) / seg);
  const int64_t per = int64_t(kWarps) << (5 - m.lr);  // rows of one block step
  int64_t gy = (rows + per - 1) / per;
  const int64_t fill = int64_t(sm_count()) * 8 / m.gx;  // (not one block more: it would run alone)
  if (gy > fill) gy = fill;
  if (gy > max_parts) gy = max_parts;
  m.gy = unsigned(gy < 1 ? 1 : gy);
  return m;
}

template <int V>
struct Lane {
  static constexpr int NV = V > 1 ? 1 : 4;
  int64_t row, step;  // first row, rows between two of this lane's rows
  int64_t base;       // first row of the warp (the same trip count in every lane)
  int64_t col0;       // first column of the warp
  int64_t col[NV];    // this lane's vectors, clamped into the row
  bool in[NV];
};
template <int V>
__device__ __forceinline__ Lane<V> lane_of(int lr, int64_t cols) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Lane<V> l;
  const int rpw = 32 >> lr;
  l.base = (int64_t(blockIdx.y) * kWarps + warp) * rpw;
  l.row = l.base + (lane >> lr);
  l.step = int64_t(gridDim.y) * kWarps * rpw;
  l.col0 = V > 1 ? (int64_t(blockIdx.x) << lr) * V : int64_t(blockIdx.x) * 128;
#pragma unroll
  for (int j = 0; j < Lane<V>::NV; ++j) {
    const int64_t c = l.col0 + (V > 1 ? (lane & ((1 << lr) - 1)) * V : j * 32 + lane);
    l.in[j] = c < cols;
    l.col[j] = l.in[j] ? c : 0;
  }
  return l;
}

// Rows in flight per lane: loads of all of them are issued before the first is
// used.  Rows past the end reread the last row and store nothing.
template <typename T, int V, int FMT, int U>
__global__ void __launch_bounds__(kWarps * 32)
    pack_kernel(const T* x, int64_t ldx, int64_t rows, int64_t cols, int lr, const Ckpt c) {
  constexpr int NV = Lane<V>::NV, P = NV * V / 2;
  const Lane<V> l = lane_of<V>(lr, cols);
  for (int64_t b = l.base, r = l.row; b < rows; b += l.step * U, r += l.step * U) {
    Row<T, V, NV> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ru = r + u * l.step < rows ? r + u * l.step : rows - 1;
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[u].load(j, x + ru * ldx + l.col[j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ru = r + u * l.step;
      bool in[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!l.in[j]) raw[u].zero(j);
        in[j] = l.in[j] && ru < rows;
      }
      f2 v[P];
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = raw[u].pair_at(i);
      ckpt_write<FMT, V, NV>(c, ru, cols, l.col, in, v);
    }
  }
}

// Wide rows of BF16: a lane packs 16 consecutive columns (one division and one 16-byte
// store for them), a warp 512; 2^lr lanes share a row.
template <int FMT, int U>
__global__ void __launch_bounds__(kWarps * 32)
    pack16_kernel(const bf16* x, int64_t ldx, int64_t rows, int64_t cols, int lr, bool a32, const Ckpt c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rpw = 32 >> lr;
  const int64_t base = (int64_t(blockIdx.y) * kWarps + warp) * rpw;
  const int64_t step = int64_t(gridDim.y) * kWarps * rpw;
  const int64_t col = ((int64_t(blockIdx.x) << lr) + (lane & ((1 << lr) - 1))) * 16;
  const bool in0 = col < cols, in1 = col + 8 < cols, first = (int(col) & ((1 << c.lg) - 1)) == 0;
  const bool a16 = cols % 16 == 0 && (reinterpret_cast<uintptr_t>(c.codes) & 15) == 0;
  int64_t r = base + (lane >> lr);
  const bf16* from = x + (in0 ? col : 0);
  uint8_t* code = c.codes + r * cols + col;
  float* scale = c.scale + r * c.groups + (col >> c.lg);
  for (int64_t b = base; b < rows; b += step * U, r += step * U) {
    uint32_t w[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bf16* p = from + (r + u * step < rows ? r + u * step : rows - 1) * ldx;
      if (a32 && in1) {
        ld_stream(p, w[u]);
      } else {
        ld_stream_v4(p, w[u][0], w[u][1], w[u][2], w[u][3]);
        ld_stream_v4(in1 ? p + 8 : p, w[u][4], w[u][5], w[u][6], w[u][7]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool e = r + u * step < rows;
      f2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (i < 4 ? in0 : in1) ? bf2(w[u][i]) : 0ull;
      ckpt_write16<FMT>(c.lg, code, a16, scale, first, in0 && e, in1 && e, v);
      code += step * cols, scale += step * c.groups;
    }
  }
}

template <typename T, int V, int ACT, int U>
__global__ void __launch_bounds__(kWarps * 32)
    unpack_kernel(const Ckpt c, int64_t rows, int64_t cols, int lr, T* y, int64_t ldy) {
  constexpr int NV = Lane<V>::NV, P = NV * V / 2;
  const Lane<V> l = lane_of<V>(lr, cols);
  for (int64_t r = l.row; r < rows; r += l.step * U) {
    CodeRow<V, NV> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ru = r + u * l.step < rows ? r + u * l.step : rows - 1;
#pragma unroll
      for (int j = 0; j < NV; ++j) w[u].load(j, c, ru, cols, l.col[j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ru = r + u * l.step;
      f2 v[P];
      w[u].values(c.fmt, v);
      act_all<ACT, sizeof(T) == 4>(v);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (ru < rows && l.in[j]) put<T, V>(y + ru * ldy + l.col[j], v, j);
    }
  }
}

template <typename T, int V, int ACT, int U>
__global__ void __launch_bounds__(kWarps * 32)
    act_bwd_kernel(const Ckpt c, const T* dy, int64_t lddy, int64_t rows, int64_t cols, int lr, T* dx,
                   int64_t lddx, T* y, int64_t ldy, float* part, const Join jn) {
  constexpr int NV = Lane<V>::NV, E = NV * V, P = E / 2;
  const Lane<V> l = lane_of<V>(lr, cols);
  f2 sum2[P] = {};
  for (int64_t r = l.row; r < rows; r += l.step * U) {
    Row<T, V, NV> raw[U];
    CodeRow<V, NV> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ru = r + u * l.step < rows ? r + u * l.step : rows - 1;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        raw[u].load(j, dy + ru * lddy + l.col[j]);
        if (c.codes) w[u].load(j, c, ru, cols, l.col[j]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ru = r + u * l.step;
      if (ru >= rows) break;
      f2 v[P];
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = raw[u].pair_at(i);
      if (c.codes) {
        f2 p[P];
        w[u].values(c.fmt, p);
        slope_all<ACT, sizeof(T) == 4>(p, v);
        if (y) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (l.in[j]) put<T, V>(y + ru * ldy + l.col[j], p, j);
        }
      }
      if (dx) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (l.in[j]) put<T, V>(dx + ru * lddx + l.col[j], v, j);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) sum2[i] = add2(sum2[i], v[i]);
    }
  }
  if (part || jn.on) {
    // the lanes of a column, then the eight warps, in a fixed order
    __shared__ float red[kWarps + 1][32 * E];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float sum[E];
#pragma unroll
    for (int i = 0; i < P; ++i) sum[2 * i] = lo2(sum2[i]), sum[2 * i + 1] = hi2(sum2[i]);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      for (int o = 16; o >= (1 << lr); o >>= 1) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
      if (lane < (1 << lr)) red[warp][V == 8 ? lane * 8 + i : i * 32 + lane] = sum[i];
    }
    __syncthreads();
    const int64_t col = l.col0 + threadIdx.x;
    const int seg = V == 8 ? 8 << lr : 128;
    if (int(threadIdx.x) < seg && col < cols) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += red[w][threadIdx.x];
      if (jn.on) red[kWarps][threadIdx.x] = t;
      else part[int64_t(blockIdx.y) * cols + col] = t;
    }
    if (jn.on) {  // the segment's row slices are one cluster
      const int64_t left = cols - l.col0;
      join_columns(Join{jn.out + l.col0, nullptr, jn.accumulate, true}, red[kWarps], 0, left < seg ? left : seg);
    }
  }
}

// Gate and up kept in 8 bits: dg = dy u act'(g), du = dy act(g), y = act(g) u.
template <typename T, int V, int ACT, int U>
__global__ void __launch_bounds__(kWarps * 32)
    gated_bwd_kernel(const Ckpt cg, const Ckpt cu, const T* dy, int64_t lddy, int64_t rows, int64_t cols, int lr,
                     T* dg, T* du, int64_t lddp, T* y, int64_t ldy) {
  constexpr int NV = Lane<V>::NV, P = NV * V / 2;
  const Lane<V> l = lane_of<V>(lr, cols);
  for (int64_t r = l.row; r < rows; r += l.step * U) {
    Row<T, V, NV> raw[U];
    CodeRow<V, NV> wg[U], wu[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t ru = r + k * l.step < rows ? r + k * l.step : rows - 1;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (dg) raw[k].load(j, dy + ru * lddy + l.col[j]);
        wg[k].load(j, cg, ru, cols, l.col[j]);
        wu[k].load(j, cu, ru, cols, l.col[j]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t ru = r + k * l.step;
      if (ru >= rows) break;
      f2 g[P], u[P], d[P];
      wg[k].values(cg.fmt, g);
      wu[k].values(cu.fmt, u);
#pragma unroll
      for (int i = 0; i < P; ++i) d[i] = dg ? mul2(raw[k].pair_at(i), u[i]) : 0ull;
      slope_all<ACT, sizeof(T) == 4>(g, d);  // g becomes act(g)
      if (dg) {
        f2 e[P];
#pragma unroll
        for (int i = 0; i < P; ++i) e[i] = mul2(raw[k].pair_at(i), g[i]);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (l.in[j]) put<T, V>(dg + ru * lddp + l.col[j], d, j);
          if (l.in[j]) put<T, V>(du + ru * lddp + l.col[j], e, j);
        }
      }
      if (y) {
#pragma unroll
        for (int i = 0; i < P; ++i) u[i] = mul2(u[i], g[i]);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (l.in[j]) put<T, V>(y + ru * ldy + l.col[j], u, j);
      }
    }
  }
}

// 32 columns x 32 slices per block: slice j adds the parts j, j + 32, ... in
// order, then the slices are added pairwise.  At most ten parts per slice, all of
// them under way at once.
__global__ void __launch_bounds__(1024)
    part_sums_kernel(const float* part, const float* part2, int parts, int64_t cols, float* out,
                     float* out2, int accumulate) {
  constexpr int MOST = (kMaxParts + 31) / 32;
  __shared__ float red[32][33];
  const float* src = blockIdx.y ? part2 : part;
  float* dst = blockIdx.y ? out2 : out;
  const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  float v[MOST], t = 0.0f;
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    v[i] = c < cols && j + 32 * i < parts ? src[int64_t(j + 32 * i) * cols + c] : 0.0f;
#pragma unroll
  for (int i = 0; i < MOST; ++i) t += v[i];
  red[j][lane] = t;
  __syncthreads();
  // warp j adds up column j of the 32 x 32 totals
  t = red[lane][j];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  const int64_t cj = int64_t(blockIdx.x) * 32 + j;
  if (lane == 0 && cj < cols) dst[cj] = accumulate ? dst[cj] + t : t;
}

size_t act_bwd_ws(int64_t rows, int64_t cols) {
  int64_t parts = (rows + kWarps - 1) / kWarps;
  if (parts > kMaxParts) parts = kMaxParts;
  return size_t(parts) * size_t(cols) * 4;
}

template <typename T>
struct Type {
  using type = T;
};

// f(tag of the element type, columns per vector)
template <typename F>
void by_type(int dtype, int v, F f) {
  using V8 = std::integral_constant<int, 8>;
  using V1 = std::integral_constant<int, 1>;
  if (dtype == AQFQ_BF16) {
    if (v == 8) f(Type<bf16>(), V8());
    else f(Type<bf16>(), V1());
  } else {
    if (v == 8) f(Type<float>(), V8());
    else f(Type<float>(), V1());
  }
}

// f(tag of the activation)
template <typename F>
void by_act(int act, F f) {
  switch (act) {
    case AQFQ_ACT_RELU: f(std::integral_constant<int, AQFQ_ACT_RELU>()); break;
    case AQFQ_ACT_GELU: f(std::integral_constant<int, AQFQ_ACT_GELU>()); break;
    case AQFQ_ACT_GELU_TANH: f(std::integral_constant<int, AQFQ_ACT_GELU_TANH>()); break;
    case AQFQ_ACT_SILU: f(std::integral_constant<int, AQFQ_ACT_SILU>()); break;
    default: f(std::integral_constant<int, AQFQ_ACT_NONE>()); break;
  }
}

aqfq_status done() { return cudaGetLastError() == cudaSuccess ? AQFQ_OK : AQFQ_ERR_CUDA; }

}  // namespace

cudaError_t launch_part_sums(const float* part, const float* part2, int parts, int64_t cols,
                             float* out, float* out2, int accumulate, cudaStream_t st) {
  if (cols <= 0) return cudaSuccess;
  if (!out) {
    out = out2, part = part2;
    out2 = nullptr;
  }
  part_sums_kernel<<<dim3(unsigned((cols + 31) / 32), out2 ? 2 : 1), 1024, 0, st>>>(
      part, part2, parts, cols, out, out2, accumulate);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace aqfq

using namespace aqfq;
using namespace aqfq::layer;

extern "C" aqfq_status aqfq_ckpt8_pack(const aqfq_ckpt8* ckpt, int dtype, const void* x,
                                       int64_t ldx, int64_t rows, int64_t cols, void* stream) {
  Ckpt c;
  if (!view_ok(rows, cols, ldx) || !view_ok(rows, cols, cols)) return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype)) return AQFQ_ERR_UNSUPPORTED;
  aqfq_status s = make_ckpt(ckpt, rows, cols, c);
  if (s != AQFQ_OK) return s;
  if (rows == 0 || cols == 0) return AQFQ_OK;
  if (!x) return AQFQ_ERR_NULL;
  if (!al(x, esize(dtype))) return AQFQ_ERR_ALIGN;
  if (sm_count() <= 0) return AQFQ_ERR_CUDA;
  const bool wide = cols % 8 == 0 && rows_aligned<8>(x, ldx, esize(dtype)) && al(c.codes, 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (wide && dtype == AQFQ_BF16 && cols > 256) {
    const Map m = make_map(rows, cols, c.lg, 16, 65535);
    const bf16* in = static_cast<const bf16*>(x);
    const bool a32 = al(x, 32) && ldx % 16 == 0;
    const dim3 grid(m.gx, m.gy);
    if (c.fmt == AQFQ_INT8)
      pack16_kernel<AQFQ_INT8, kU><<<grid, kWarps * 32, 0, st>>>(in, ldx, rows, cols, m.lr, a32, c);
    else
      pack16_kernel<AQFQ_FP8_E4M3, kU><<<grid, kWarps * 32, 0, st>>>(in, ldx, rows, cols, m.lr, a32, c);
    return done();
  }
  const Map m = make_map(rows, cols, c.lg, wide ? 8 : 1, 65535);
  by_type(dtype, wide ? 8 : 1, [&](auto t, auto v) {
    using T = typename decltype(t)::type;
    constexpr int V = decltype(v)::value;
    const dim3 grid(m.gx, m.gy);
    const T* in = static_cast<const T*>(x);
    if (c.fmt == AQFQ_INT8)
      pack_kernel<T, V, AQFQ_INT8, kU><<<grid, kWarps * 32, 0, st>>>(in, ldx, rows, cols, m.lr, c);
    else
      pack_kernel<T, V, AQFQ_FP8_E4M3, kU><<<grid, kWarps * 32, 0, st>>>(in, ldx, rows, cols, m.lr, c);
  });
  return done();
}

extern "C" aqfq_status aqfq_ckpt8_unpack(const aqfq_ckpt8* ckpt, int act, int dtype, void* y,
                                         int64_t ldy, int64_t rows, int64_t cols, void* stream) {
  Ckpt c;
  if (!view_ok(rows, cols, ldy) || !view_ok(rows, cols, cols)) return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype) || !act_ok(act)) return AQFQ_ERR_UNSUPPORTED;
  aqfq_status s = make_ckpt(ckpt, rows, cols, c);
  if (s != AQFQ_OK) return s;
  if (rows == 0 || cols == 0) return AQFQ_OK;
  if (!y) return AQFQ_ERR_NULL;
  if (!al(y, esize(dtype))) return AQFQ_ERR_ALIGN;
  if (sm_count() <= 0) return AQFQ_ERR_CUDA;
  const int vec = cols % 8 == 0 && rows_aligned<8>(y, ldy, esize(dtype)) && al(c.codes, 8) ? 8 : 1;
  // 16 columns per lane for many elements (8192 x 8192 with GELU 52 -> 46 us, 8192 x 4096
  // 28 -> 26; 2048 x 2048 would go from 5.1 to 7.0, 16384 x 768 from 13.2 to 12.1)
  const bool v16 = dtype == AQFQ_BF16 && cols > 256 && cols % 16 == 0 && ldy % 16 == 0 && al(y, 32) &&
                   al(c.codes, 16) && rows * cols >= (int64_t(1) << 24);
  const Map m = make_map(rows, cols, c.lg, v16 ? 16 : vec, 65535);
  by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (v16) {
      unpack_kernel<bf16, 16, ACT, kU>
          <<<dim3(m.gx, m.gy), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
              c, rows, cols, m.lr, static_cast<bf16*>(y), ldy);
      return;
    }
    by_type(dtype, vec, [&](auto t, auto v) {
      using T = typename decltype(t)::type;
      constexpr int V = decltype(v)::value;
      unpack_kernel<T, V, ACT, kU>
          <<<dim3(m.gx, m.gy), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
              c, rows, cols, m.lr, static_cast<T*>(y), ldy);
    });
  });
  return done();
}

extern "C" size_t aqfq_ckpt8_act_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (!view_ok(rows, cols, cols)) return 0;
  return act_bwd_ws(rows, cols);
}

extern "C" aqfq_status aqfq_ckpt8_act_bwd(const aqfq_ckpt8* ckpt, int act, int dtype,
                                          const void* dy, int64_t lddy, int64_t rows, int64_t cols,
                                          void* dx, int64_t lddx, void* y, int64_t ldy,
                                          float* dbias, int accumulate, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  Ckpt c = {};
  c.lg = 5;
  if (!view_ok(rows, cols, lddy) || !view_ok(rows, cols, cols) ||
      (dx && !view_ok(rows, cols, lddx)) || (y && !view_ok(rows, cols, ldy)))
    return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype) || !act_ok(act)) return AQFQ_ERR_UNSUPPORTED;
  if (ckpt) {
    const aqfq_status s = make_ckpt(ckpt, rows, cols, c);
    if (s != AQFQ_OK) return s;
  } else if (act != AQFQ_ACT_NONE || y) {
    return AQFQ_ERR_NULL;  // an activation needs its input
  }
  const bool any = rows > 0 && cols > 0;
  if (any && (!dy || (!dx && !y && !dbias))) return AQFQ_ERR_NULL;
  const int es = esize(dtype);
  if (!al(dy, es) || !al(dx, es) || !al(y, es) || !al(dbias, 4)) return AQFQ_ERR_ALIGN;
  if (dbias && any) {
    if (!workspace || workspace_bytes < act_bwd_ws(rows, cols)) return AQFQ_ERR_WORKSPACE;
    if (!al(workspace, 8)) return AQFQ_ERR_ALIGN;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!any) {
    if (dbias && !accumulate && cols > 0)
      return launch_part_sums(nullptr, nullptr, 0, cols, dbias, nullptr, 0, st) == cudaSuccess
                 ? AQFQ_OK
                 : AQFQ_ERR_CUDA;
    return AQFQ_OK;
  }
  if (sm_count() <= 0) return AQFQ_ERR_CUDA;
  const int vec = cols % 8 == 0 && rows_aligned<8>(dy, lddy, es) && rows_aligned<8>(dx, lddx, es) &&
                          rows_aligned<8>(y, ldy, es) && al(c.codes, 8)
                      ? 8
                      : 1;
  Map m = make_map(rows, cols, c.lg, vec, dbias ? kMaxParts : 65535);
  // few rows (eight per warp in eight slices): the slices of a column segment form a
  // cluster and add up their sums there (512 x 1024 6.7 us on the GPU against 4.9 with a
  // second launch, which costs the host 3.3 us; 64 x 4096 3.8 both ways)
  const Join jn = {dbias, nullptr, accumulate, dbias && rows <= (int64_t(8 * 8 * kWarps) << (5 - m.lr))};
  if (jn.on && m.gy > 8) m.gy = 8;
  cudaError_t launched = cudaSuccess;
  float* part = dbias && !jn.on ? static_cast<float*>(workspace) : nullptr;
  by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    by_type(dtype, vec, [&](auto t, auto v) {
      using T = typename decltype(t)::type;
      constexpr int V = decltype(v)::value;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(m.gx, m.gy), cfg.blockDim = dim3(kWarps * 32), cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = at[0].val.clusterDim.z = 1, at[0].val.clusterDim.y = jn.on ? m.gy : 1;
      cfg.attrs = at, cfg.numAttrs = 1;
      launched = cudaLaunchKernelEx(&cfg, act_bwd_kernel<T, V, ACT, kUB>, c, static_cast<const T*>(dy), lddy,
                                    rows, cols, m.lr, static_cast<T*>(dx), lddx, static_cast<T*>(y), ldy,
                                    part, jn);
    });
  });
  if (launched != cudaSuccess) return AQFQ_ERR_CUDA;
  if (part &&
      launch_part_sums(part, nullptr, int(m.gy), cols, dbias, nullptr, accumulate, st) != cudaSuccess)
    return AQFQ_ERR_CUDA;
  return AQFQ_OK;
}

extern "C" aqfq_status aqfq_ckpt8_gated_bwd(const aqfq_ckpt8* gate, const aqfq_ckpt8* up, int act, int dtype,
                                            const void* dy, int64_t lddy, int64_t rows, int64_t cols, void* dp,
                                            int64_t lddp, void* y, int64_t ldy, void* stream) {
  Ckpt cg = {}, cu = {};
  if (!view_ok(rows, cols, cols) || (dy && !view_ok(rows, cols, lddy)) || (y && !view_ok(rows, cols, ldy)) ||
      cols > 0x3FFFFFF8 || (dp && !view_ok(rows, 2 * cols, lddp)))
    return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype) || !act_ok(act)) return AQFQ_ERR_UNSUPPORTED;
  aqfq_status s = make_ckpt(gate, rows, cols, cg);
  if (s == AQFQ_OK) s = make_ckpt(up, rows, cols, cu);
  if (s != AQFQ_OK) return s;
  if (cg.fmt != cu.fmt || cg.lg != cu.lg) return AQFQ_ERR_UNSUPPORTED;
  const bool any = rows > 0 && cols > 0;
  if (any && ((!dp && !y) || (dp && !dy))) return AQFQ_ERR_NULL;
  const int es = esize(dtype);
  if (!al(dy, es) || !al(dp, es) || !al(y, es)) return AQFQ_ERR_ALIGN;
  if (!any) return AQFQ_OK;
  if (sm_count() <= 0) return AQFQ_ERR_CUDA;
  const int vec = cols % 8 == 0 && rows_aligned<8>(dy, lddy, es) && rows_aligned<8>(dp, lddp, es) &&
                          rows_aligned<8>(y, ldy, es) && al(cg.codes, 8) && al(cu.codes, 8)
                      ? 8
                      : 1;
  const Map m = make_map(rows, cols, cg.lg, vec, 65535);
  by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    by_type(dtype, vec, [&](auto t, auto v) {
      using T = typename decltype(t)::type;
      constexpr int V = decltype(v)::value;
      T* out = static_cast<T*>(dp);
      gated_bwd_kernel<T, V, ACT, kUB><<<dim3(m.gx, m.gy), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
          cg, cu, static_cast<const T*>(dy), lddy, rows, cols, m.lr, out, out ? out + cols : nullptr, lddp,
          static_cast<T*>(y), ldy);
    });
  });
  return done();
}
