// aqfq_ckpt8.cu -- activation checkpoints in 8 bits: pack, unpack (with the
// activation recomputed) and the activation gradient read from a checkpoint.
//
// A row is cut into groups of 32, 64 or 128 columns (the last one may be
// shorter).  One lane holds 8 consecutive columns, so a group is 4, 8 or 16
// neighbouring lanes and its amax a butterfly over them.  A warp covers 256
// columns of one row (narrow rows: several rows per warp) and walks down the
// rows of its slice; the bias gradient's column sums stay in its registers.
// All three are bound by memory: pack moves 2 + 1 bytes per BF16 element,
// unpack 1 + 2, the gradient 1 + 2 + 2 (+ 2 with the recomputed activation).
#include <type_traits>

#include "aqfq_internal.h"
#include "aqfq_layer.cuh"

namespace aqfq {
namespace layer {
namespace {

constexpr int kWarps = 8;

// lanes per row: a whole group at least, 32 at most
struct Map {
  int lr;          // log2 of the lanes that share a row
  unsigned gx;     // column segments
  unsigned gy;     // row slices
};

inline Map make_map(int64_t rows, int64_t cols, int lg, int64_t max_parts) {
  Map m;
  m.lr = lg - 3;
  while (m.lr < 5 && (int64_t(8) << m.lr) < cols) ++m.lr;
  m.gx = unsigned((cols + (int64_t(8) << m.lr) - 1) / (int64_t(8) << m.lr));
  const int64_t per = int64_t(kWarps) << (5 - m.lr);  // rows of one block step
  int64_t gy = (rows + per - 1) / per;
  const int64_t fill = (int64_t(sm_count()) * 16 + m.gx - 1) / m.gx;
  if (gy > fill) gy = fill;
  if (gy > max_parts) gy = max_parts;
  m.gy = unsigned(gy < 1 ? 1 : gy);
  return m;
}

struct Lane {
  int64_t row, step;  // first row, rows between two of this lane's rows
  int64_t col;
  int n;              // columns in range (<= 0: none)
};
__device__ __forceinline__ Lane lane_of(int lr, int64_t cols) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Lane l;
  const int sub = lane >> lr, rpw = 32 >> lr;
  l.row = (int64_t(blockIdx.y) * kWarps + warp) * rpw + sub;
  l.step = int64_t(gridDim.y) * kWarps * rpw;
  l.col = ((int64_t(blockIdx.x) << lr) + (lane & ((1 << lr) - 1))) * 8;
  const int64_t left = cols - l.col;
  l.n = left > 8 ? 8 : int(left);
  return l;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    pack_kernel(const T* x, int64_t ldx, int64_t rows, int64_t cols, int lr, bool vec, bool cvec,
                const Ckpt c) {
  const Lane l = lane_of(lr, cols);
  const int64_t last = l.row - (l.row % (32 >> lr));  // warp-uniform trip count
  for (int64_t r0 = last, r = l.row; r0 < rows; r0 += l.step, r += l.step) {
    const bool in = r < rows;
    float v[8];
    load_row(x + r * ldx + l.col, vec && in && l.n == 8, in ? l.n : 0, v);
    uint32_t m = amax_bits(v);
    for (int o = 1; o < (1 << (c.lg - 3)); o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const Divisor d = make_divisor(ckpt_scale(m, c.fmt));
    if (in && l.n > 0) {
      const uint32_t w[2] = {ckpt_codes4(v, d, c.fmt), ckpt_codes4(v + 4, d, c.fmt)};
      store_bytes<8>(c.codes + r * cols + l.col, cvec && l.n == 8, l.n, w);
      if ((l.col & ((1 << c.lg) - 1)) == 0) c.scale[r * c.groups + (l.col >> c.lg)] = d.s;
    }
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kWarps * 32)
    unpack_kernel(const Ckpt c, int64_t rows, int64_t cols, int lr, bool cvec, T* y, int64_t ldy,
                  bool vec) {
  const Lane l = lane_of(lr, cols);
  if (l.n <= 0) return;
  for (int64_t r = l.row; r < rows; r += l.step) {
    uint32_t w[2];
    load_bytes<8>(c.codes + r * cols + l.col, cvec && l.n == 8, l.n, w);
    const float s = c.scale[r * c.groups + (l.col >> c.lg)];
    float v[8];
    ckpt_values4(w[0], s, c.fmt, v);
    ckpt_values4(w[1], s, c.fmt, v + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_f<ACT>(v[i]);
    store_row(y + r * ldy + l.col, vec && l.n == 8, l.n, v);
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kWarps * 32)
    act_bwd_kernel(const Ckpt c, const T* dy, int64_t lddy, int64_t rows, int64_t cols, int lr,
                   bool vec, bool cvec, T* dx, int64_t lddx, T* y, int64_t ldy, float* part) {
  const Lane l = lane_of(lr, cols);
  float sum[8] = {};
  if (l.n > 0) {
    for (int64_t r = l.row; r < rows; r += l.step) {
      float v[8];
      load_row(dy + r * lddy + l.col, vec && l.n == 8, l.n, v);
      if (c.codes) {
        uint32_t w[2];
        load_bytes<8>(c.codes + r * cols + l.col, cvec && l.n == 8, l.n, w);
        const float s = c.scale[r * c.groups + (l.col >> c.lg)];
        float p[8];
        ckpt_values4(w[0], s, c.fmt, p);
        ckpt_values4(w[1], s, c.fmt, p + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float d;
          p[i] = act_fd<ACT>(p[i], d);
          v[i] *= d;
        }
        if (y) store_row(y + r * ldy + l.col, vec && l.n == 8, l.n, p);
      }
      if (dx) store_row(dx + r * lddx + l.col, vec && l.n == 8, l.n, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
  if (part) {
    __shared__ float red[kWarps][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      for (int o = 16; o >= (1 << lr); o >>= 1) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
      if (lane < (1 << lr)) red[warp][lane * 8 + i] = sum[i];
    }
    __syncthreads();
    const int64_t col = (int64_t(blockIdx.x) << lr) * 8 + threadIdx.x;
    if (int(threadIdx.x) < (8 << lr) && col < cols) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += red[w][threadIdx.x];
      part[int64_t(blockIdx.y) * cols + col] = t;
    }
  }
}

// 32 columns x 8 slices per block: slice j adds the parts j, j + 8, ... in
// order, then the eight slices are added in order
__global__ void __launch_bounds__(256)
    part_sums_kernel(const float* part, const float* part2, int parts, int64_t cols, float* out,
                     float* out2, int accumulate) {
  __shared__ float red[8][32];
  const float* src = blockIdx.y ? part2 : part;
  float* dst = blockIdx.y ? out2 : out;
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x % 32;
  const int j = threadIdx.x / 32;
  float t = 0.0f;
  if (c < cols)
    for (int p = j; p < parts; p += 8) t += src[int64_t(p) * cols + c];
  red[j][threadIdx.x % 32] = t;
  __syncthreads();
  if (j == 0 && c < cols) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
    dst[c] = accumulate ? dst[c] + t : t;
  }
}

size_t act_bwd_ws(int64_t rows, int64_t cols) {
  int64_t parts = (rows + kWarps - 1) / kWarps;
  if (parts > kMaxParts) parts = kMaxParts;
  return size_t(parts) * size_t(cols) * 4;
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
  part_sums_kernel<<<dim3(unsigned((cols + 31) / 32), out2 ? 2 : 1), 256, 0, st>>>(
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
  const Map m = make_map(rows, cols, c.lg, 65535);
  const bool vec = rows_aligned<8>(x, ldx, esize(dtype)), cvec = rows_aligned<8>(c.codes, cols, 1);
  const dim3 grid(m.gx, m.gy);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == AQFQ_BF16)
    pack_kernel<<<grid, kWarps * 32, 0, st>>>(static_cast<const bf16*>(x), ldx, rows, cols, m.lr,
                                              vec, cvec, c);
  else
    pack_kernel<<<grid, kWarps * 32, 0, st>>>(static_cast<const float*>(x), ldx, rows, cols, m.lr,
                                              vec, cvec, c);
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
  const Map m = make_map(rows, cols, c.lg, 65535);
  const bool vec = rows_aligned<8>(y, ldy, esize(dtype)), cvec = rows_aligned<8>(c.codes, cols, 1);
  const dim3 grid(m.gx, m.gy);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (dtype == AQFQ_BF16)
      unpack_kernel<bf16, ACT><<<grid, kWarps * 32, 0, st>>>(c, rows, cols, m.lr, cvec,
                                                             static_cast<bf16*>(y), ldy, vec);
    else
      unpack_kernel<float, ACT><<<grid, kWarps * 32, 0, st>>>(c, rows, cols, m.lr, cvec,
                                                              static_cast<float*>(y), ldy, vec);
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
  const Map m = make_map(rows, cols, c.lg, dbias ? kMaxParts : 65535);
  const bool vec = rows_aligned<8>(dy, lddy, es) && rows_aligned<8>(dx, lddx, es) &&
                   rows_aligned<8>(y, ldy, es);
  const bool cvec = rows_aligned<8>(c.codes, cols, 1);
  const dim3 grid(m.gx, m.gy);
  float* part = dbias ? static_cast<float*>(workspace) : nullptr;
  by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (dtype == AQFQ_BF16)
      act_bwd_kernel<bf16, ACT><<<grid, kWarps * 32, 0, st>>>(
          c, static_cast<const bf16*>(dy), lddy, rows, cols, m.lr, vec, cvec,
          static_cast<bf16*>(dx), lddx, static_cast<bf16*>(y), ldy, part);
    else
      act_bwd_kernel<float, ACT><<<grid, kWarps * 32, 0, st>>>(
          c, static_cast<const float*>(dy), lddy, rows, cols, m.lr, vec, cvec,
          static_cast<float*>(dx), lddx, static_cast<float*>(y), ldy, part);
  });
  if (cudaGetLastError() != cudaSuccess) return AQFQ_ERR_CUDA;
  if (dbias &&
      launch_part_sums(part, nullptr, int(m.gy), cols, dbias, nullptr, accumulate, st) != cudaSuccess)
    return AQFQ_ERR_CUDA;
  return AQFQ_OK;
}
