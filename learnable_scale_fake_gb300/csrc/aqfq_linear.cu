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
//
// Products of BF16 are exact in binary32 and their sums are held in it.  Over 3680 terms the
// tensor cores' sums measured 4e-6 off (2-norm, relative), a blocked sum of FMAs 6e-7: far
// below a BF16 output's rounding of 4e-3, but an FP32 weight gradient shows it.
#include <cuda.h>

#include <mutex>

#include "aqfq_internal.h"
#include "aqfq_layer.cuh"
#include "aqfq_sm100_pair.cuh"

namespace aqfq {
namespace layer {
namespace {

enum Pass { P_FWD = AQFQ_LINEAR_FWD, P_DGRAD = AQFQ_LINEAR_DGRAD, P_WGRAD = AQFQ_LINEAR_WGRAD };

// ---------------------------------------------------------------------------
// epilogue of sums in memory: 16 lanes hold 128 columns of a row, a lane 8 of them, a
// warp two rows; an 8-bit group of 32, 64 or 128 columns is 4, 8 or 16 neighbouring
// lanes.  (4 columns per lane and 32 lanes per row: twice the address arithmetic per
// element, 0.9 us instead of 0.55 us per turn of 16 warps with GELU and residual.)
// ---------------------------------------------------------------------------
struct Epi {
  int64_t rows, cols;
  const void* bias;     // forward
  const bf16* res;      // forward, input gradient
  int64_t ldr;
  void* out;
  int64_t ldo;
  int bias_dtype, out_dtype, act, accumulate;
  bool vec_out, vec_res, vec_bias, vec_codes;  // 8-element accesses are aligned
  bool wide;            // 16-element accesses (32 bytes) of out and res, 16 of codes
  Ckpt c;               // forward: written; input gradient: read
};

// columns of [col, col + V) that lie in the row
template <int V>
__device__ __forceinline__ int in_row(const Epi& e, int64_t col) {
  const int64_t left = e.cols - col;
  return left > V ? V : int(left);
}

// the bias of columns [col, col + V)
template <int V>
__device__ __forceinline__ void load_bias(const Epi& e, int64_t col, float (&b)[V]) {
  const int n = in_row<V>(e, col);
  if (e.bias && n > 0) {
    if (e.bias_dtype == AQFQ_BF16)
      load_row(static_cast<const bf16*>(e.bias) + col, e.vec_bias && n == V, n, b);
    else
      load_row(static_cast<const float*>(e.bias) + col, e.vec_bias && n == V, n, b);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
  }
}

// v: the sums of row r, columns [col, col + 8); `in`: the row is this call's.  Every
// lane of the warp calls it.
template <int PASS>
__device__ __forceinline__ void epilogue8(const Epi& e, int64_t r, bool in, int64_t col,
                                          const float (&bias)[8], float (&v)[8]) {
  const int n = in_row<8>(e, col);
  const bool full = n == 8;
  in = in && n > 0;
  const bool adds = PASS == P_WGRAD ? e.accumulate != 0 : e.res != nullptr;
  float add[8];
  if (adds && in) {
    if constexpr (PASS == P_WGRAD) {
      if (e.out_dtype == AQFQ_BF16)
        load_row(static_cast<const bf16*>(e.out) + r * e.ldo + col, e.vec_out && full, n, add);
      else
        load_row(static_cast<const float*>(e.out) + r * e.ldo + col, e.vec_out && full, n, add);
    } else {
      load_row(e.res + r * e.ldr + col, e.vec_res && full, n, add);
    }
  }
  if constexpr (PASS == P_DGRAD) {
    if (e.c.codes && in) {
      uint32_t w[2];
      load_bytes<8>(e.c.codes + r * e.cols + col, e.vec_codes && full, n, w);
      const float s = e.c.scale[r * e.c.groups + (col >> e.c.lg)];
      float p[8];
      ckpt_values4(w[0], s, e.c.fmt, p);
      ckpt_values4(w[1], s, e.c.fmt, p + 4);
      slope_apply(e.act, p, v);
    }
  }
  if constexpr (PASS == P_FWD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += bias[i];
    if (e.c.codes) {
      if (!full) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] : 0.0f;  // no share beyond the row
      }
      uint32_t m = amax_bits(v);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1)
        if (o < 4 || o < (1 << (e.c.lg - 3))) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (in) {
        const Divisor d = ckpt_divisor(m, e.c.fmt);
        const f2 x[4] = {mk2(v[0], v[1]), mk2(v[2], v[3]), mk2(v[4], v[5]), mk2(v[6], v[7])};
        uint32_t w[2];
        ckpt_codes(x, d, e.c.fmt, w);
        store_bytes<8>(e.c.codes + r * e.cols + col, e.vec_codes && full, n, w);
        if ((int(col) & ((1 << e.c.lg) - 1)) == 0) e.c.scale[r * e.c.groups + (col >> e.c.lg)] = d.s;
      }
    }
    act_apply(e.act, v);
  }
  if (!in) return;
  if (adds) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += add[i];
  }
  if (PASS == P_WGRAD && e.out_dtype == AQFQ_F32)
    store_row(static_cast<float*>(e.out) + r * e.ldo + col, e.vec_out && full, n, v);
  else
    store_row(static_cast<bf16*>(e.out) + r * e.ldo + col, e.vec_out && full, n, v);
}

// Partial sums of 128 columns in shared memory: the 16-byte units of 4 columns with an
// even number first, then the odd ones, so that the two units of a lane's 8 columns
// lie at unit `lane` and unit 16 + `lane`: both reads of 16 lanes are contiguous (at a
// stride of 32 bytes the reads from other CTAs took twice as long).
__device__ __forceinline__ int unit_at(int unit) { return ((unit & 1) << 4) + (unit >> 1); }

// The sums of 8 columns at `mine` (this CTA's address) over `slices` CTAs of the cluster,
// `stride` ranks apart from rank `first`; all reads are on their way before the first
// addition, which go in the slices' order.
__device__ __forceinline__ void cluster_sum8(uint32_t mine, int slices, uint32_t first, uint32_t stride,
                                             float (&v)[8]) {
  float4 f[8][2];
#pragma unroll
  for (int sl = 0; sl < 8; ++sl) {
    if (sl < slices) {
      const uint32_t base = sm100::peer_addr(mine, first + stride * uint32_t(sl));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(f[sl][j].x), "=f"(f[sl][j].y), "=f"(f[sl][j].z), "=f"(f[sl][j].w)
                     : "r"(base + uint32_t(256 * j)));
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    v[4 * j] = f[0][j].x, v[4 * j + 1] = f[0][j].y, v[4 * j + 2] = f[0][j].z, v[4 * j + 3] = f[0][j].w;
#pragma unroll
  for (int sl = 1; sl < 8; ++sl) {
    if (sl < slices) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        v[4 * j] += f[sl][j].x, v[4 * j + 1] += f[sl][j].y, v[4 * j + 2] += f[sl][j].z, v[4 * j + 3] += f[sl][j].w;
    }
  }
}

// ---------------------------------------------------------------------------
// epilogue from tensor memory: a lane holds one row, 16 columns at a time, so a
// checkpoint group is a run of one lane's values (no exchange between lanes, one
// division per group) and every access is a whole 32-byte sector.
// ---------------------------------------------------------------------------
// 16 BF16 at p; a16 / a32: p is 16- / 32-byte aligned (all 16 in the row), else n single ones
__device__ __forceinline__ void ld16(const bf16* p, bool a32, bool a16, int n, uint32_t (&w)[8]) {
  if (a32) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else if (a16) {
    const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 8);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = 2 * i < n ? p[2 * i].b : 0u;
      w[i] |= 2 * i + 1 < n ? uint32_t(p[2 * i + 1].b) << 16 : 0u;
    }
  }
}
__device__ __forceinline__ void st16(bf16* p, bool a32, bool a16, int n, const uint32_t (&w)[8]) {
  if (a32) {
    st_256(p, w);
  } else if (a16) {
    st_128(p, w[0], w[1], w[2], w[3]);
    st_128(p + 8, w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (2 * i < n) p[2 * i].b = uint16_t(w[i]);
      if (2 * i + 1 < n) p[2 * i + 1].b = uint16_t(w[i] >> 16);
    }
  }
}

constexpr int kEpiWarps = 16;
constexpr int kBN = 256;                            // columns of a pair's tile
constexpr int kChunks = kBN / (kEpiWarps / 4) / 16;  // 16-column chunks of an epilogue warp

// alignment of a row segment of 16 columns that lies in the row
struct Seg {
  bool a32, a16;
};
__device__ __forceinline__ Seg seg(const void* p, bool whole) {
  const uint32_t a = uint32_t(reinterpret_cast<uintptr_t>(p));
  return {whole && (a & 31) == 0, whole && (a & 15) == 0};
}

// 16 accumulator columns of the lane's row: issued, then waited for
__device__ __forceinline__ void tmem_issue(uint32_t taddr, uint32_t (&r)[16]) {
  __syncwarp();  // the load is a warp-wide instruction
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// (the registers pass through, so that no use moves above the wait)
__device__ __forceinline__ void tmem_take(uint32_t (&r)[16], float (&v)[16]) {
  __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// n <= 16 codes at p: whole, in halves where rows start at odd multiples of 8 (300 x 1000 x
// 576 with a checkpoint: single bytes 15 us instead of 8), or one by one
__device__ __forceinline__ void store_codes16(uint8_t* p, int n, const uint32_t (&w)[4]) {
  const uint32_t a = uint32_t(reinterpret_cast<uintptr_t>(p));
  if (n == 16 && (a & 15) == 0) {
    st_128(p, w[0], w[1], w[2], w[3]);
  } else if ((n & 7) == 0 && (a & 7) == 0) {
    st_64(p, w[0], w[1]);
    if (n > 8) st_64(p + 8, w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
  }
}

// What 16 columns of a row read besides the sums: the residual, or the previous
// output of an accumulation.
template <int PASS>
struct ChunkIn {
  uint32_t w[PASS == P_WGRAD ? 16 : 8];
  __device__ __forceinline__ void load(const Epi& e, int64_t r, int64_t cc) {
    const int64_t left = e.cols - cc;
    const int n = left > 16 ? 16 : int(left);
    if (PASS == P_WGRAD && e.out_dtype == AQFQ_F32) {
      if (e.accumulate) {
        const float* p = static_cast<const float*>(e.out) + r * e.ldo + cc;
        const bool a16 = seg(p, n == 16).a16;
#pragma unroll
        for (int i = 0; i < (PASS == P_WGRAD ? 16 : 0); i += 4) {
          if (a16) {
            const uint4 f = *reinterpret_cast<const uint4*>(p + i);
            w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i + j] = i + j < n ? __float_as_uint(p[i + j]) : 0u;
          }
        }
      }
    } else if (PASS == P_WGRAD ? e.accumulate != 0 : e.res != nullptr) {
      const bf16* p = PASS == P_WGRAD ? static_cast<const bf16*>(e.out) + r * e.ldo + cc
                                      : e.res + r * e.ldr + cc;
      const Seg s = seg(p, n == 16);
      uint32_t t[8];
      ld16(p, s.a32, s.a16, n, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = t[i];
    }
  }
};

// 16 columns of row r from cc on (n of them in the row): adds what `cur` holds and stores
template <int PASS>
__device__ __forceinline__ void finish_chunk(const Epi& e, int64_t r, int64_t cc, int n,
                                             const ChunkIn<PASS>& cur, float (&v)[16]) {
  const bool adds = PASS == P_WGRAD ? e.accumulate != 0 : e.res != nullptr;
  if (PASS == P_WGRAD && e.out_dtype == AQFQ_F32) {
    float* p = static_cast<float*>(e.out) + r * e.ldo + cc;
    const bool a16 = seg(p, n == 16).a16;
    if constexpr (PASS == P_WGRAD) {
      if (adds) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(cur.w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      if (a16) {
        *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < n) p[i + j] = v[i + j];
      }
    }
  } else {
    if (adds) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[2 * i] += bf_lo(cur.w[i]), v[2 * i + 1] += bf_hi(cur.w[i]);
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i + 1], v[2 * i]);
    bf16* p = static_cast<bf16*>(e.out) + r * e.ldo + cc;
    const Seg q = seg(p, n == 16);
    st16(p, q.a32, q.a16, n, w);
  }
}

// The codes of a row's 16 CH columns from col on and their scales (one per 32 columns):
// all of them are fetched before the accumulators are waited for.
template <int CH>
struct RowCodes {
  uint32_t w[CH][4];
  float scale[CH / 2];
  __device__ __forceinline__ void load(const Epi& e, int64_t r, int64_t col) {
    const uint8_t* p = e.c.codes + r * e.cols + col;
    const float* sc = e.c.scale + r * e.c.groups;
    const int64_t left = e.cols - col;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (c * 16 >= left) break;
      if (seg(p + c * 16, left >= c * 16 + 16).a16) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + c * 16);
        w[c][0] = u.x, w[c][1] = u.y, w[c][2] = u.z, w[c][3] = u.w;
      } else if (e.vec_codes) {  // rows start at multiples of 8
        const uint2 u = *reinterpret_cast<const uint2*>(p + c * 16);
        const uint2 z = left > c * 16 + 8 ? *reinterpret_cast<const uint2*>(p + c * 16 + 8) : make_uint2(0, 0);
        w[c][0] = u.x, w[c][1] = u.y, w[c][2] = z.x, w[c][3] = z.y;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[c][i] = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c * 16 + i < left) w[c][i >> 2] |= uint32_t(p[c * 16 + i]) << (8 * (i & 3));
      }
      if (c % 2 == 0) scale[c / 2] = sc[(col + c * 16) >> e.c.lg];
    }
  }
};

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// The row's residual or previous output for w columns on their way to L2: the
// accumulators of this tile are still being summed.
template <int PASS>
__device__ __forceinline__ void prefetch_inputs(const Epi& e, int64_t r, int64_t col, int w) {
  const int n = e.cols - col < w ? int(e.cols - col) : w;
  const uint8_t *p = nullptr, *q = nullptr;
  if (PASS == P_WGRAD) {
    const int es = e.out_dtype == AQFQ_F32 ? 4 : 2;
    if (e.accumulate) p = static_cast<const uint8_t*>(e.out) + (r * e.ldo + col) * es, q = p + n * es;
  } else if (e.res) {
    p = reinterpret_cast<const uint8_t*>(e.res + r * e.ldr + col), q = p + n * 2;
  }
  for (; p < q; p += 128) prefetch_l2(p);
}

// 16 bias values in shared memory (16-byte aligned, the same for every lane)
__device__ __forceinline__ void add_bias16(const float* sb, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(sb + i);
    v[i] += b.x, v[i + 1] += b.y, v[i + 2] += b.z, v[i + 3] += b.w;
  }
}

// lines of what row r's 128 columns from c0 on read, one per lane (of 16)
template <int PASS>
__device__ __forceinline__ void prefetch_row(const Epi& e, int64_t r, int64_t c0, int lane) {
  const int64_t n = e.cols - c0 > 128 ? 128 : e.cols - c0;
  const int64_t at = lane * 128;  // byte
  if (PASS == P_WGRAD) {
    const int es = e.out_dtype == AQFQ_F32 ? 4 : 2;
    if (e.accumulate && at < n * es)
      prefetch_l2(static_cast<const uint8_t*>(e.out) + (r * e.ldo + c0) * es + at);
  } else {
    if (e.res && at < n * 2) prefetch_l2(reinterpret_cast<const uint8_t*>(e.res + r * e.ldr + c0) + at);
    if (PASS == P_DGRAD && e.c.codes && lane == 8) prefetch_l2(e.c.codes + r * e.cols + c0);
  }
}

// Columns [col, col + 16 kChunks) of row r (one row per lane of the warp), sums at
// taddr.  `in`: the row exists.  Every lane of the warp calls it.  sb: the columns'
// bias in shared memory.  A checkpoint group may be larger than the warp's columns:
// its amax is then taken by every warp that has a part of it (the accumulators and
// the bias of the 128 columns around are at hand).  The next chunk's sums are under way
// while one is computed; its other inputs, sent to L2 before, are read when it begins (held
// a chunk ahead, they cost every warp of the kernel 30 spilled registers: 8191 x 4104 x 768
// with GELU and residual 86 us instead of 75).
template <int PASS, int ACT>
__device__ __forceinline__ void epilogue_row(const Epi& e, int64_t r, bool in, int64_t col,
                                             uint32_t taddr, const float* sb,
                                             const RowCodes<kChunks>& codes) {
  constexpr bool CODES_IN = PASS == P_DGRAD && ACT != AQFQ_ACT_NONE;
  const bool codes_out = PASS == P_FWD && e.c.codes;
  const int64_t avail = (e.cols - col + 15) / 16;
  const int nch = avail < kChunks ? int(avail) : kChunks;
  const int gch = codes_out ? 1 << (e.c.lg - 4) : nch;  // chunks per group
  const int lead = codes_out ? int(col >> 4) & (gch - 1) : 0;  // chunks of the group before col
  uint32_t t[16];
  float v[16];
#pragma unroll 1
  for (int g0 = -lead; g0 < nch; g0 += gch) {
    const int g = g0 < 0 ? 0 : g0, end = g0 + gch < nch ? g0 + gch : nch;
    Divisor div = {};
    if (codes_out) {
      uint32_t m = 0;
      const int gend = g0 + gch < avail ? g0 + gch : int(avail);
      tmem_issue(taddr + uint32_t(g0 * 16), t);
#pragma unroll 1
      for (int c = g0; c < gend; ++c) {
        tmem_take(t, v);
        if (c + 1 < gend) tmem_issue(taddr + uint32_t((c + 1) * 16), t);
        const int64_t left = e.cols - (col + c * 16);
        if (e.bias) add_bias16(sb + c * 16, v);
        if (left < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = i < left ? v[i] : 0.0f;
        }
        m = max(m, amax_bits(v));
      }
      div = ckpt_divisor(m, e.c.fmt);
      if (in && g0 >= 0) e.c.scale[r * e.c.groups + ((col + g0 * 16) >> e.c.lg)] = div.s;
    }
    tmem_issue(taddr + uint32_t(g * 16), t);
    // (the codes are in registers: unrolled, so that their indices are constants)
#pragma unroll(CODES_IN ? kChunks : 1)
    for (int i0 = 0; i0 < kChunks; ++i0) {
      const int c = CODES_IN ? i0 : g + i0;
      if (c >= end) break;
      const int64_t cc = col + c * 16;
      const int64_t left = e.cols - cc;
      const int n = left > 16 ? 16 : int(left);
      ChunkIn<PASS> cur;
      if (in) cur.load(e, r, cc);
      tmem_take(t, v);
      if (c + 1 < end) tmem_issue(taddr + uint32_t((c + 1) * 16), t);
      if (PASS == P_FWD) {
        if (e.bias) add_bias16(sb + c * 16, v);
        if (codes_out && in) {
          uint32_t w[4];
          f2 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = mk2(v[2 * i], v[2 * i + 1]);
          ckpt_codes(x, div, e.c.fmt, w);
          store_codes16(e.c.codes + r * e.cols + cc, n, w);
        }
        act_all<ACT>(v);
      }
      if (CODES_IN) {
        float p[16];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ckpt_values4(codes.w[CODES_IN ? i0 : 0][i], codes.scale[CODES_IN ? i0 / 2 : 0], e.c.fmt, p + 4 * i);
        slope_all<ACT>(p, v);
      }
      if (in) finish_chunk<PASS>(e, r, cc, n, cur, v);
    }
  }
}

// Whether epilogue_whole serves a warp's 32 rows and 16 kChunks columns: all of them
// exist and every access is aligned (uniform).
template <int PASS>
__device__ __forceinline__ bool whole_block(const Epi& e, int64_t r0, int64_t col) {
  if (r0 + 32 > e.rows || col + 16 * kChunks > e.cols || !e.wide) return false;
  return PASS != P_WGRAD || !e.accumulate;
}

// epilogue_row for such a block: no bounds, the chunks unrolled, one base address per
// tensor (the general form spends about 240 instructions per chunk without an
// activation, this one a third of that).
template <int PASS, int ACT>
__device__ __forceinline__ void epilogue_whole(const Epi& e, int64_t r, int64_t col, uint32_t taddr,
                                               const float* sb, const RowCodes<kChunks>& codes) {
  constexpr bool CODES_IN = PASS == P_DGRAD && ACT != AQFQ_ACT_NONE;
  const bool codes_out = PASS == P_FWD && e.c.codes;
  const bool adds = PASS != P_WGRAD && e.res;
  uint32_t t[16], add[8];
  float v[16];
  Divisor div[kChunks / 2];  // per 32 columns
  if (codes_out) {
    const int gch = 1 << (e.c.lg - 4), lead = int(col >> 4) & (gch - 1);
#pragma unroll
    for (int h = 0; h < kChunks / 2; ++h) {
      if (h > 0 && gch > 2) {  // the same group
        div[h] = div[0];
        continue;
      }
      const int g0 = 2 * h - (gch > 2 ? lead : 0);
      const int64_t left = (e.cols - (col + g0 * 16) + 15) / 16;
      const int n = left < gch ? int(left) : gch;
      uint32_t m = 0;
      tmem_issue(taddr + uint32_t(g0 * 16), t);
#pragma unroll 1
      for (int c = 0; c < n; ++c) {
        tmem_take(t, v);
        if (c + 1 < n) tmem_issue(taddr + uint32_t((g0 + c + 1) * 16), t);
        if (e.bias) add_bias16(sb + (g0 + c) * 16, v);
        const int64_t in = e.cols - (col + (g0 + c) * 16);
        if (in < 16) {  // (a group that reaches past this block)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = i < in ? v[i] : 0.0f;
        }
        m = max(m, amax_bits(v));
      }
      div[h] = ckpt_divisor(m, e.c.fmt);
      if (g0 >= 0) e.c.scale[r * e.c.groups + ((col + g0 * 16) >> e.c.lg)] = div[h].s;
    }
  }
  const bf16* res = adds ? e.res + r * e.ldr + col : nullptr;
  uint8_t* code = codes_out ? e.c.codes + r * e.cols + col : nullptr;
  const bool f32 = PASS == P_WGRAD && e.out_dtype == AQFQ_F32;
  uint8_t* out = static_cast<uint8_t*>(e.out) + (r * e.ldo + col) * (f32 ? 4 : 2);
  if (adds) ld16(res, true, true, 16, add);
  tmem_issue(taddr, t);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    tmem_take(t, v);
    if (c + 1 < kChunks) tmem_issue(taddr + uint32_t((c + 1) * 16), t);
    if (PASS == P_FWD) {
      if (e.bias) add_bias16(sb + c * 16, v);
      if (codes_out) {
        uint32_t w[4];
        f2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mk2(v[2 * i], v[2 * i + 1]);
        ckpt_codes(x, div[c / 2], e.c.fmt, w);
        st_128(code + c * 16, w[0], w[1], w[2], w[3]);
      }
      act_all<ACT>(v);
    }
    if (CODES_IN) {
      float p[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) ckpt_values4(codes.w[c][i], codes.scale[c / 2], e.c.fmt, p + 4 * i);
      slope_all<ACT>(p, v);
    }
    if (adds) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[2 * i] += bf_lo(add[i]), v[2 * i + 1] += bf_hi(add[i]);
      if (c + 1 < kChunks) ld16(res + (c + 1) * 16, true, true, 16, add);
    }
    uint32_t w[8];
    if (f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
        st_256(out + c * 64 + h * 32, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i + 1], v[2 * i]);
      st_256(out + c * 32, w);
    }
  }
}

// ---------------------------------------------------------------------------
// product on a pair of CTAs: tiles of 256 rows x BN columns, 64 of k per stage.
// Each CTA loads 128 rows of A and BN / 2 of B by TMA; one thread of the leader
// issues the MMAs for both (tcgen05, cta_group::2); the accumulators (128 rows
// x BN columns per CTA) are double-buffered in tensor memory, so the epilogue of
// a tile runs under the next tile's MMAs.  Ragged edges and the tail of k are
// zeros from the TMA's fill.
//   warp 0  TMA producer    warp 1  MMA issuer (leader), tensor memory
//   warps 2-17  epilogue, four per quarter of the rows, a quarter of the columns each
//               (with two per quarter the forward with GELU and checkpoint took 192 us at
//               8192 x 4096 x 4096, with four 167 us).  Five of the eighteen warps share a
//               quarter of the SM, which leaves 96 registers a thread, and spilled ones go to
//               L2 beside 200 KB of shared memory: 8 to 28 bytes in the forward kernels and
//               in the input gradient with GELU or tanh GELU, 248 and 116 in the forward's
//               and the input gradient's split tail, none in the other kernels but 16 in the
//               weight gradient's split tail.
// At 8192 x 4096 x 4096 (plain library products beside: 137-152, 147-156 and 155-168 us):
// forward with GELU 146-153 us, with a checkpoint too 160-167 us, input gradient 142-167 us,
// weight gradient 152-175 us; two runs differ by so much with the clock under the power
// limit.  The MMAs run 81 to 89 % of the time; the rest is the first loads, the last tile's
// epilogue and tiles that do not divide evenly among 76 pairs.
// Every wait is bounded; on a timeout the pair drains, frees its tensor memory,
// raises the caller's flag and returns.
// ---------------------------------------------------------------------------
using namespace sm100;

constexpr int kRows = 256, kHalf = 128, kBK = 64;
constexpr int kThreadsP = 64 + 32 * kEpiWarps;
constexpr uint32_t kABytes = kHalf * kBK * 2;  // 16 KiB per CTA and stage

template <int BN>
struct Cfg {
  static constexpr int STAGES = 6;
  static constexpr uint32_t B_BYTES = BN / 2 * kBK * 2;
  static constexpr uint32_t STAGE = kABytes + B_BYTES;
  static constexpr uint32_t BIAS = kEpiWarps * 128 * 4;  // the 128 columns around a warp's
  static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE + BIAS + 256;
  // a split tile's partial sums (one row per 16-byte odd stride) reuse the stages
  static constexpr int PSTRIDE = BN + 4;
  static_assert(size_t(kHalf) * PSTRIDE * 4 <= size_t(STAGES) * STAGE, "partial sums fit the stages");
};

struct __align__(8) PairShared {
  uint64_t full[6], empty[6];  // TMA bytes of both CTAs (leader) / MMA commit
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem;
  int32_t abort, stop[2];
  int32_t issued;  // steps whose loads were issued
};

struct PairArgs {
  int nr, nc;        // tiles
  int first, count;  // the tiles of this launch
  int splits;        // slices of the inner axis
  int a_rows;        // rows of A per box (tile_kernel: fewer when there are fewer rows)
  int ksteps;        // 64-element steps of the inner axis
  float* part;       // [splits][rows][cols4] partial sums when splits > 1
  int64_t cols4;     // cols rounded up to 4
  int32_t* err;
};

// tile t: groups of 8 tile rows, column by column, so that the tiles in flight share
// their operands in L2
__device__ __forceinline__ void tile_of(const PairArgs& a, int t, int& tr, int& tc) {
  const int width = 8 * a.nc, g = t / width, first = g * 8;
  const int gm = a.nr - first < 8 ? a.nr - first : 8;
  const int in = t - g * width;
  tr = first + in % gm;
  tc = in / gm;
}

// SPLIT: a cluster of S pairs takes one tile, pair i the i-th slice of the inner
// axis; the partial sums meet through distributed shared memory, each CTA finishing
// its share of the rows (one launch, no scratch; the sums in the slices' order).
template <int PASS, int ACT, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreadsP, 1)
    pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const PairArgs a, const Epi e) {
  using C = Cfg<BN>;
  constexpr bool A_MN = PASS == P_WGRAD, B_MN = PASS != P_FWD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sb = smem + C::STAGES * kABytes;
  float* sbias = reinterpret_cast<float*>(sb + C::STAGES * C::B_BYTES);
  PairShared* sh = reinterpret_cast<PairShared*>(reinterpret_cast<uint8_t*>(sbias) + C::BIAS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), rank = crank & 1, lead = crank & ~1u;
  const int tiles = a.count, units = SPLIT ? tiles : tiles * a.splits;
  // one unit per cluster, or a strided share of the units per pair
  const int pair = SPLIT ? blockIdx.x / (2 * a.splits) : blockIdx.x >> 1;
  const int npairs = SPLIT ? units : gridDim.x >> 1;
  const int slice = int(crank >> 1);
  const uint32_t mask = 3u << lead;  // the pair's CTAs

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->tfull[b], 1);
      mbar_init(&sh->tempty[b], 2 * kEpiWarps);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
  }
  if (warp == 1) tmem_alloc_pair(&sh->tmem, 512);
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = sh->tmem;
  volatile int32_t* abort = &sh->abort;

  if (warp == 0) {
    // a warp-uniform loop; one elected lane issues (see elect_one)
    int s = 0, it = 0;
    uint32_t phase = 1;  // the first round finds every stage empty
    bool ok = true;
    const uint32_t full0 = peer_addr(smem_u32(&sh->full[0]), lead);
    const uint32_t da0 = smem_u32(smem), db0 = smem_u32(sb);
    for (int u = pair; u < units && ok; u += npairs) {
      int tr, tc;
      tile_of(a, a.first + u % tiles, tr, tc);
      const int sp = SPLIT ? slice : u / tiles;
      const int k0 = int(int64_t(a.ksteps) * sp / a.splits);
      const int k1 = int(int64_t(a.ksteps) * (sp + 1) / a.splits);
      const int r0 = tr * kRows + int(rank) * kHalf, c0 = tc * BN + int(rank) * (BN / 2);
      for (int k = k0; k < k1; ++k, ++it) {
        if (it >= C::STAGES && !mbar_wait_warp(&sh->empty[s], phase)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t bar = full0 + uint32_t(s * 8);
          if (rank == 0) mbar_arrive_expect_tx(&sh->full[s], 2 * C::STAGE);
          const uint32_t da = da0 + s * kABytes, db = db0 + s * C::B_BYTES;
          if constexpr (A_MN) {
            tma_load_2d_pair(da, &ta, bar, r0, k * kBK);
            tma_load_2d_pair(da + kABytes / 2, &ta, bar, r0 + 64, k * kBK);
          } else {
            tma_load_2d_pair(da, &ta, bar, k * kBK, r0);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_2d_pair(db + j * 8192, &tb, bar, c0 + 64 * j, k * kBK);
          } else {
            tma_load_2d_pair(db, &tb, bar, k * kBK, c0);
          }
        }
        __syncwarp();
        if (++s == C::STAGES) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) *abort = 1;
    if (lane == 0) sh->issued = it;
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kRows, BN) | (A_MN ? kIdescTransA : 0) |
                                 (B_MN ? kIdescTransB : 0);
      const uint64_t da0 = A_MN ? smem_desc_mn_sw128(smem_u32(smem), 8192)
                                : smem_desc_sw128(smem_u32(smem));
      const uint64_t db0 = B_MN ? smem_desc_mn_sw128(smem_u32(sb), 8192)
                                : smem_desc_sw128(smem_u32(sb));
      // 16 of k: 32 bytes along a row, or two atoms of 8
      constexpr uint32_t ka = A_MN ? 2048 >> 4 : 32 >> 4, kb = B_MN ? 2048 >> 4 : 32 >> 4;
      int s = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += npairs, ++n) {
        const int sp = SPLIT ? slice : u / tiles;
        const int k0 = int(int64_t(a.ksteps) * sp / a.splits);
        const int k1 = int(int64_t(a.ksteps) * (sp + 1) / a.splits);
        const int buf = n & 1;
        if (n >= 2 && !mbar_wait_warp(&sh->tempty[buf], ((n >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + uint32_t(buf * 256);
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait_warp(&sh->full[s], phase)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t da = da0 + ((s * kABytes) >> 4), db = db0 + ((s * C::B_BYTES) >> 4);
          if (elect_one()) {
            tc_mma_f16_pair(d, da, db, idesc, k > k0 ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < kBK / 16; ++kk) tc_mma_f16_pair(d, da + kk * ka, db + kk * kb, idesc, 1u);
            tc_commit_pair(&sh->empty[s], mask);
            if (k + 1 == k1) tc_commit_pair(&sh->tfull[buf], mask);
          }
          __syncwarp();
          if (++s == C::STAGES) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {  // a wait timed out: drain the MMAs already issued
        *abort = 1;
        if (elect_one()) tc_commit_pair(&sh->drain, mask);
        __syncwarp();
        mbar_wait_warp(&sh->drain, 0);
      }
    }
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;
    constexpr int W = BN / (kEpiWarps / 4);  // columns of this warp
    float* mybias = sbias + (warp - 2) * 128;
    int n = 0;
    for (int u = pair; u < units; u += npairs, ++n) {
      int tr, tc;
      tile_of(a, a.first + u % tiles, tr, tc);
      const int buf = n & 1;
      const int64_t r0 = int64_t(tr) * kRows + int(rank) * kHalf + q * 32, r = r0 + lane;
      const int64_t col = int64_t(tc) * BN + part * W;
      const bool live = r0 < e.rows && col < e.cols, whole = !SPLIT && a.splits == 1;
      const bool fast = whole_block<PASS>(e, r0, col);
      RowCodes<kChunks> codes;
      if (live && whole) {
        if (PASS == P_FWD && e.bias) {
          float b[4];
          __syncwarp();
          load_bias(e, (col & ~int64_t(127)) + lane * 4, b);
          *reinterpret_cast<float4*>(mybias + lane * 4) = make_float4(b[0], b[1], b[2], b[3]);
          __syncwarp();
        }
        if (r < e.rows) {
          prefetch_inputs<PASS>(e, r, col, W);
          if (PASS == P_DGRAD && ACT != AQFQ_ACT_NONE) codes.load(e, r, col);
        }
      }
      // one thread waits for the tile, the other warps for it at a barrier: sixteen
      // polling warps slowed the MMAs beside them by a tenth
      if (warp == 2 && lane == 0) {
        const bool ok = mbar_wait_long(&sh->tfull[buf], (n >> 1) & 1) && !*abort;
        if (!ok) *abort = 1;
        sh->stop[buf] = ok ? 0 : 1;  // read by every warp after this barrier, before the next one
      }
      __syncwarp();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
      if (*reinterpret_cast<volatile int32_t*>(&sh->stop[buf])) break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + uint32_t(buf * 256 + part * W);
      if (live) {
        if (SPLIT) {
          // into this CTA's shared memory (its stages are all consumed)
          float* dst = reinterpret_cast<float*>(smem) + (q * 32 + lane) * C::PSTRIDE + part * W / 128 * 128;
          uint32_t t[16];
          float v[16];
          tmem_issue(taddr, t);
#pragma unroll 1
          for (int c = 0; c < W / 16; ++c) {
            tmem_take(t, v);
            if (c + 1 < W / 16) tmem_issue(taddr + uint32_t((c + 1) * 16), t);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(dst + unit_at((part * W % 128 + c * 16 + i) / 4) * 4) =
                  make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        } else if (a.splits > 1) {
          float* dst = a.part + (int64_t(u / tiles) * e.rows + r) * a.cols4 + col;
          uint32_t t[16];
          float v[16];
#pragma unroll 1
          for (int c = 0; c < W / 16 && col + c * 16 < e.cols; ++c) {
            tmem_issue(taddr + uint32_t(c * 16), t);
            tmem_take(t, v);
            if (r < e.rows) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                if (col + c * 16 + i < a.cols4)
                  *reinterpret_cast<float4*>(dst + c * 16 + i) =
                      make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        } else {
          if (fast) epilogue_whole<PASS, ACT>(e, r, col, taddr, mybias + int(col & 127), codes);
          else epilogue_row<PASS, ACT>(e, r, r < e.rows, col, taddr, mybias + int(col & 127), codes);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (!SPLIT && lane == 0) mbar_arrive_cluster(peer_addr(smem_u32(&sh->tempty[buf]), lead));
    }
  }
  if constexpr (SPLIT) {
    // this CTA's rows of the tile; a warp takes half the columns of two rows per turn
    constexpr int NW = kThreadsP / 32;
    int tr, tc;
    tile_of(a, a.first + pair, tr, tc);
    const int64_t r0 = int64_t(tr) * kRows + int(rank) * kHalf;
    const int nrows = e.rows - r0 > kHalf ? kHalf : (e.rows > r0 ? int(e.rows - r0) : 0);
    const int half = warp & 1, row0 = nrows * slice / a.splits, rend = nrows * (slice + 1) / a.splits;
    const int64_t c0 = int64_t(tc) * BN + half * (BN / 2), col = c0 + (lane & 15) * 8;
    float bias[8] = {};
    if (PASS == P_FWD) load_bias(e, col, bias);
    if (warp >= 2 && c0 < e.cols)
      for (int row = row0 + (warp >> 1) * 2 + (lane >> 4); row < rend; row += NW)
        prefetch_row<PASS>(e, r0 + row, c0, lane & 15);
    __syncwarp();
    cluster_sync();  // every slice's partial sums are in shared memory
    if (c0 < e.cols) {
#pragma unroll 1
      for (int base = row0 + (warp >> 1) * 2; base < rend; base += NW) {
        const int row = base + (lane >> 4);
        // (a row past rend is another CTA's or the last one again: read, not used)
        float v[8];
        cluster_sum8(smem_u32(smem) + uint32_t((row < kHalf ? row : base) * C::PSTRIDE + half * (BN / 2) +
                                               (lane & 15) * 4) * 4,
                     a.splits, rank, 2, v);
        epilogue8<PASS>(e, r0 + row, row < rend, col, bias, v);
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  // whichever wait gave up: the pair's copies, which all count on the leader's barriers
  if (warp == 0 && rank == 0 && *abort) drain_loads(sh->full, C::STAGES, sh->issued);
  __syncwarp();
  cluster_sync();  // the peer's MMAs and arrivals into this CTA are done
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort && a.err) atomicExch(a.err, 1);
}

// ---------------------------------------------------------------------------
// small products: one CTA per 128 x 128 tile and slice of the inner axis, the S
// slices of a tile in a cluster.  Six stages of 32 KiB; warp 0 issues the loads (the
// first six before the block has set up), warp 1 the MMAs.  A whole sum (one slice) goes
// from tensor memory through the epilogue, a row per lane;
// else all sixteen warps move the accumulators to shared memory (the stages are
// consumed), the cluster meets, and each CTA finishes its share of the rows that exist: a
// warp takes whole rows of 128 columns, reads every slice's value through distributed
// shared memory and adds them in the slices' order.
// Few rows (a token or two): the weight is streamed once by tiles x S CTAs.
// 24 x 2048 x 768 5 us, 1 x 4096 x 4096 8.4-8.7 us (the weight at 3.9 TB/s; up to 10 after
// a hot kernel), 1000 x 1536 x 2048 11.1 us: about 4.5 us are launch, first loads and
// epilogue, a step of 64 takes 0.2 us (a whole SM's MMAs: 0.17).
// ---------------------------------------------------------------------------
constexpr int kTile = 128;
constexpr int kWarpsC = 16;
constexpr int kStagesC = 6;
constexpr int kStrideC = kTile + 4;  // floats per row of partial sums
constexpr size_t kSmemC = 1024 + size_t(kStagesC) * 2 * kABytes + 256;
static_assert(size_t(kTile) * kStrideC * 4 <= size_t(kStagesC) * 2 * kABytes, "partial sums fit the stages");

struct __align__(8) CtaShared {
  uint64_t full[kStagesC], empty[kStagesC];
  uint64_t accum;
  uint32_t tmem;
  int32_t abort;
  int32_t issued;  // steps whose loads were issued
};

template <int PASS>
__global__ void __launch_bounds__(32 * kWarpsC, 1)
    tile_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const PairArgs a, const Epi e) {
  constexpr bool A_MN = PASS == P_WGRAD, B_MN = PASS != P_FWD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  CtaShared* sh = reinterpret_cast<CtaShared*>(smem + kStagesC * 2 * kABytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = int(cluster_rank());
  const int tile = blockIdx.x / a.splits;
  // tiles column by column: neighbours share their columns' operand
  const int tr = tile % a.nr, tc = tile / a.nr;
  const int64_t r0 = int64_t(tr) * kTile, c0 = int64_t(tc) * kTile;
  const int k0 = int(int64_t(a.ksteps) * slice / a.splits);
  const int n = int(int64_t(a.ksteps) * (slice + 1) / a.splits) - k0;

  auto load = [&](int k, int s) {
    if (elect_one()) {
      uint8_t *da = smem + s * 2 * kABytes, *db = da + kABytes;
      const int kk = (k0 + k) * kBK;
      mbar_arrive_expect_tx(&sh->full[s], kABytes + (A_MN ? kABytes : uint32_t(a.a_rows * kBK * 2)));
      if constexpr (A_MN) {
        tma_load_2d(da, &ta, &sh->full[s], int(r0), kk);
        tma_load_2d(da + kABytes / 2, &ta, &sh->full[s], int(r0) + 64, kk);
      } else {
        tma_load_2d(da, &ta, &sh->full[s], kk, int(r0));
      }
      if constexpr (B_MN) {
        tma_load_2d(db, &tb, &sh->full[s], int(c0), kk);
        tma_load_2d(db + kABytes / 2, &tb, &sh->full[s], int(c0) + 64, kk);
      } else {
        tma_load_2d(db, &tb, &sh->full[s], kk, int(c0));
      }
    }
    __syncwarp();
  };
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < kStagesC; ++s) {
        mbar_init(&sh->full[s], 1);
        mbar_init(&sh->empty[s], 1);
      }
      mbar_init(&sh->accum, 1);
      sh->abort = 0;
      fence_barrier_init();
    }
    __syncwarp();
    // the first stages are on their way before the others have set up
    for (int k = 0; k < n && k < kStagesC; ++k) load(k, k);
  } else if (warp == 1) {
    tmem_alloc(&sh->tmem, kTile);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh->tmem;
  volatile int32_t* abort = &sh->abort;

  if (warp == 0) {
    int s = 0;
    uint32_t phase = 0;
    int k = n < kStagesC ? n : kStagesC;
    for (; k < n; ++k) {
      if (!mbar_wait_warp(&sh->empty[s], phase)) {
        *abort = 1;
        break;
      }
      load(k, s);
      if (++s == kStagesC) {
        s = 0;
        phase ^= 1;
      }
    }
    if (lane == 0) sh->issued = k;
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(kTile, kTile) | (A_MN ? kIdescTransA : 0) |
                               (B_MN ? kIdescTransB : 0);
    const uint32_t base = smem_u32(smem);
    const uint64_t da0 = A_MN ? smem_desc_mn_sw128(base, 8192) : smem_desc_sw128(base);
    const uint64_t db0 = B_MN ? smem_desc_mn_sw128(base + kABytes, 8192) : smem_desc_sw128(base + kABytes);
    constexpr uint32_t ka = A_MN ? 2048 >> 4 : 32 >> 4, kb = B_MN ? 2048 >> 4 : 32 >> 4;
    int s = 0;
    uint32_t phase = 0;
    for (int k = 0; k < n; ++k) {
      if (!mbar_wait_warp(&sh->full[s], phase)) {
        *abort = 1;
        break;
      }
      tc_fence_after_sync();
      const uint64_t da = da0 + ((s * 2 * kABytes) >> 4), db = db0 + ((s * 2 * kABytes) >> 4);
      if (elect_one()) {
        tc_mma_f16(tmem, da, db, idesc, k > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 1; kk < kBK / 16; ++kk) tc_mma_f16(tmem, da + kk * ka, db + kk * kb, idesc, 1u);
        tc_commit(&sh->empty[s]);
      }
      __syncwarp();
      if (++s == kStagesC) {
        s = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) tc_commit(&sh->accum);  // also after a timeout: what was issued drains
    __syncwarp();
  }
  __syncwarp();
  const int nrows = e.rows - r0 > kTile ? kTile : int(e.rows - r0);
  if (a.splits == 1) {
    // a whole sum: from tensor memory, a row per lane and 32 columns per warp (through shared
    // memory below, 1000 x 1536 x 2048 took 12.1 us instead of 10.5)
    const int q = warp & 3;
    const int64_t r = r0 + q * 32 + lane, col = c0 + (warp >> 2) * 32;
    const bool live = q * 32 < nrows && col < e.cols, in = live && r < e.rows;  // live: uniform
    ChunkIn<PASS> add[2];
    RowCodes<2> codes;
    float bias[4][8];
    if (in) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (col + c * 16 < e.cols) add[c].load(e, r, col + c * 16);
      if (PASS == P_DGRAD && e.c.codes) codes.load(e, r, col);
      if (PASS == P_FWD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) load_bias(e, col + i * 8, bias[i]);
      }
    }
    __syncwarp();
    if (!mbar_wait_warp(&sh->accum, 0)) *abort = 1;
    __syncwarp();
    tc_fence_after_sync();
    float v[2][16];
    if (live) {
      const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + uint32_t((warp >> 2) * 32);
      uint32_t t[16];
      tmem_issue(taddr, t);
      tmem_take(t, v[0]);
      tmem_issue(taddr + 16, t);
      tmem_take(t, v[1]);
    }
    if (PASS == P_FWD && in) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i / 16][i % 16] += bias[i / 8][i % 8];
    }
    if (PASS == P_FWD && e.c.codes) {  // uniform over the grid
      // a group is this warp's 32 columns, or those of two or four neighbouring warps too
      float* most = reinterpret_cast<float*>(smem);  // [4][128]; the stages are consumed
      uint32_t m = 0;
      if (in) {
        const int64_t left = e.cols - col;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i / 16][i % 16] = i < left ? v[i / 16][i % 16] : 0.0f;
        m = max(amax_bits(v[0]), amax_bits(v[1]));
      }
      const int part = warp >> 2, at = q * 32 + lane;
      most[part * 128 + at] = __uint_as_float(m);
      __syncthreads();
      if (in) {
        const int first = part & ~((1 << (e.c.lg - 5)) - 1);
        for (int i = 0; i < (1 << (e.c.lg - 5)); ++i)
          m = max(m, __float_as_uint(most[(first + i) * 128 + at]));
        const Divisor d = ckpt_divisor(m, e.c.fmt);
        if (part == first) e.c.scale[r * e.c.groups + (col >> e.c.lg)] = d.s;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int64_t left = e.cols - (col + c * 16);
          uint32_t w[4];
          f2 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = mk2(v[c][2 * i], v[c][2 * i + 1]);
          ckpt_codes(x, d, e.c.fmt, w);
          if (left > 0) store_codes16(e.c.codes + r * e.cols + col + c * 16, left > 16 ? 16 : int(left), w);
        }
      }
    }
    if (in) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t left = e.cols - (col + c * 16);
        if (left <= 0) continue;
        if (PASS == P_FWD) act_apply(e.act, v[c]);
        if (PASS == P_DGRAD && e.c.codes) {
          float p[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) ckpt_values4(codes.w[c][i], codes.scale[0], e.c.fmt, p + 4 * i);
          slope_apply(e.act, p, v[c]);
        }
        finish_chunk<PASS>(e, r, col + c * 16, left > 16 ? 16 : int(left), add[c], v[c]);
      }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after_sync();
      tmem_dealloc(tmem, kTile);
    }
    if (warp == 0 && *abort) drain_loads(sh->full, kStagesC, sh->issued);
    if (threadIdx.x == 0 && *abort && a.err) atomicExch(a.err, 1);
    return;
  }
  // this CTA's rows, two per warp and turn; what they read is sent to L2 meanwhile
  const int row0 = nrows * slice / a.splits + warp * 2, rend = nrows * (slice + 1) / a.splits;
  for (int row = row0 + (lane >> 4); row < rend; row += 2 * kWarpsC)
    prefetch_row<PASS>(e, r0 + row, c0, lane & 15);
  const int64_t col = c0 + (lane & 15) * 8;
  float bias[8] = {};
  if (PASS == P_FWD) load_bias(e, col, bias);
  __syncwarp();
  if (!mbar_wait_warp(&sh->accum, 0)) *abort = 1;
  __syncwarp();
  tc_fence_after_sync();
  float* sums = reinterpret_cast<float*>(smem);
  {
    const int q = warp & 3, part = warp >> 2;  // 32 rows x 32 columns
    if (q * 32 < nrows) {
      const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + uint32_t(part * 32);
      float* dst = sums + (q * 32 + lane) * kStrideC;
      uint32_t t[16];
      float v[16];
      tmem_issue(taddr, t);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tmem_take(t, v);
        if (c < 1) tmem_issue(taddr + 16, t);
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(dst + unit_at((part * 32 + c * 16 + i) / 4) * 4) =
              make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
  }
  __syncwarp();
  cluster_sync();
#pragma unroll 1
  for (int base = row0; base < rend; base += 2 * kWarpsC) {
    const int row = base + (lane >> 4);
    // (a row past rend is another CTA's or the last one again: read, not used)
    const float* at = sums + (row < kTile ? row : base) * kStrideC + (lane & 15) * 4;
    float v[8];
    cluster_sum8(smem_u32(at), a.splits, 0, 1, v);
    epilogue8<PASS>(e, r0 + row, row < rend, col, bias, v);
  }
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync();  // the others have read this CTA's sums
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTile);
  }
  if (warp == 0 && *abort) drain_loads(sh->full, kStagesC, sh->issued);
  if (threadIdx.x == 0 && *abort && a.err) atomicExch(a.err, 1);
}

// out = epilogue(sum of the slices' partial sums, in order); also the empty
// product (splits 0): a warp takes 128 columns of two rows
template <int PASS>
__global__ void __launch_bounds__(256)
    finish_kernel(const float* part, int splits, int64_t cols4, const Epi e) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = int64_t(blockIdx.x) * 128 + (lane & 15) * 8;
  float bias[8] = {};
  if (PASS == P_FWD) load_bias(e, col, bias);
  for (int64_t base = int64_t(blockIdx.y) * 16 + warp * 2; base < e.rows; base += int64_t(gridDim.y) * 16) {
    const int64_t r = base + (lane >> 4);
    float v[8] = {};
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      if (r < e.rows && col + j < cols4) {
        const float* p = part + r * cols4 + col + j;
        for (int s = 0; s < splits; ++s) {
          const float4 f = *reinterpret_cast<const float4*>(p + int64_t(s) * e.rows * cols4);
          v[j] += f.x, v[j + 1] += f.y, v[j + 2] += f.z, v[j + 3] += f.w;
        }
      }
    }
    epilogue8<PASS>(e, r, r < e.rows, col, bias, v);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

struct Operand {
  const void* p;
  int64_t inner, outer, ld;  // contiguous axis, the other one, its stride
};

bool encode(CUtensorMap* tm, const Operand& o, unsigned box0, unsigned box1) {
  const cuuint64_t dims[2] = {cuuint64_t(o.inner), cuuint64_t(o.outer)};
  const int64_t ld = o.outer > 1 ? o.ld : (o.inner + 7) / 8 * 8;  // a single row has no stride
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {box0, box1};
  const cuuint32_t estr[2] = {1, 1};
  return encode_fn()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(o.p), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// How a product of rows x cols over `depth` is cut.
struct Plan {
  int nr, nc;     // tiles
  int ksteps;
  int splits;     // slices of the inner axis: of tile_kernel's clusters, or through scratch
  bool small;     // tile_kernel (128 x 128 tiles, one CTA each)
  int a_rows;     // rows of A per box
  int tail, tail_splits;  // last tiles that a second launch splits (0: none)
  int64_t cols4;
  size_t bytes;   // scratch
};

constexpr int kPairs = 76;  // SM pairs
constexpr double kStepPair = 0.336;  // us per 64 of the inner axis, every SM busy
static_assert(kBN / 2 == kHalf && kTile == kHalf, "one box for every operand tile");

// Clusters of 2 S CTAs (one per SM) that run at the same time on this GPU, by S
// (what the occupancy query reports; clusters stay within a GPC)
constexpr int kClusters[9] = {0, 76, 36, 23, 15, 13, 8, 7, 7};
// the same for clusters of S CTAs
constexpr int kClustersC[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};

constexpr int64_t kMostScratch = int64_t(64) << 20;

// The plan by an estimate of its time in us (steps of 64 of the inner axis with every
// SM busy as measured above):
//   - at most one 128 x 128 tile per SM and no long inner axis: tile_kernel, with as
//     many slices as still run together (its steps are short, 0.2 us, and it has one
//     launch; 24 x 2048 x 768 5 us, 515 x 776 x 1032 9 us where pairs took 13 and 15);
//   - else rounds of 256 x 256 tiles on pairs, 76 at once;
//   - the tiles of the last round, where they are few, may be split by a second launch, at
//     about 17 us of its own (start, joining, epilogue);
//   - or every tile's inner axis in slices through scratch, at 6 us for the second
//     kernel and the partial sums' way to memory and back (weight gradients of many
//     tokens: few tiles, a long sum).
// (The same with and without a checkpoint, so that keeping one changes no sum.)
Plan make_plan(int64_t rows, int64_t cols, int64_t depth) {
  Plan p;
  p.nr = int((rows + kRows - 1) / kRows);
  p.nc = int((cols + kBN - 1) / kBN);
  p.ksteps = int((depth + kBK - 1) / kBK);
  p.splits = p.ksteps > 0 ? 1 : 0;
  p.small = false;
  p.a_rows = kHalf, p.tail = p.tail_splits = 0;
  p.cols4 = (cols + 3) / 4 * 4;
  p.bytes = 0;
  if (p.ksteps == 0) return p;
  const int64_t small = ((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
  if (small <= kClustersC[1] && p.ksteps < 512) {
    p.small = true;
    // zero rows that only the fill would write cost as much as loaded ones (1 row, 4096 x
    // 4096: 12.9 us with boxes of 128 rows, 9.4 us with 8); rows past the box stay unread
    if (rows < kHalf) p.a_rows = int((rows + 7) / 8 * 8);
    p.nr = int((rows + kTile - 1) / kTile), p.nc = int((cols + kTile - 1) / kTile);
    int sp = 8;
    while (sp > 1 && (small > kClustersC[sp] || sp > p.ksteps)) --sp;
    // a short sum over whole tiles is not worth the joining (weight gradient 300 x 520 x
    // 1032, five steps: 5.5 us in one slice, 7.3 in five; nine steps 6.9 and 7.8; sixteen
    // steps, 300 x 1000 x 1000, 10.9 and 8.0); few rows are joined quickly
    if (rows > 64 && p.ksteps <= 10) sp = 1;
    p.splits = sp;
    return p;
  }
  const int64_t tiles = int64_t(p.nr) * p.nc;
  const double step = p.ksteps * kStepPair;
  const int64_t rounds = tiles / kPairs;
  const int rem = int(tiles % kPairs);
  double best = step * double(rounds + (rem > 0));
  int cut = 8;
  while (cut > 1 && (rem > kClusters[cut] || cut > p.ksteps / 2)) --cut;
  const double split = step * double(rounds) + step / cut + 17.0;
  if (rounds > 0 && rem > 0 && cut > 1 && split < best) best = split, p.tail = rem, p.tail_splits = cut;
  for (int sp = 2; sp <= 64 && p.ksteps / sp >= 16; ++sp) {
    const int64_t bytes = int64_t(sp) * rows * p.cols4 * 4;
    if (bytes > kMostScratch) break;
    const int64_t all = (tiles * sp + kPairs - 1) / kPairs;
    const double t = double(all) * double((p.ksteps + sp - 1) / sp) * kStepPair + 6.0 + double(bytes) * 2 / 5e6;
    if (t < best) best = t, p.splits = sp, p.tail = p.tail_splits = 0, p.bytes = size_t(bytes);
  }
  return p;
}

template <int PASS, int ACT, bool SPLIT>
cudaError_t launch_pair(const CUtensorMap& ta, const CUtensorMap& tb, const PairArgs& a, const Epi& e,
                        cudaStream_t st) {
  auto kernel = pair_kernel<PASS, ACT, kBN, SPLIT>;
  static DeviceOnce once;
  const cudaError_t attr = once_per_device(once, [&] {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg<kBN>::SMEM));
    if (e != cudaSuccess || !SPLIT) return e;
    // more than 8 CTAs per cluster
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (attr != cudaSuccess) return attr;
  const int64_t tiles = a.count, units = tiles * a.splits;
  cudaLaunchConfig_t cfg = {};
  const int csize = SPLIT ? 2 * a.splits : 2;
  cfg.gridDim = dim3(SPLIT ? unsigned(tiles * csize) : 2 * unsigned(units < kPairs ? units : kPairs));
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = Cfg<kBN>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(csize), at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, a, e);
}

template <int PASS>
cudaError_t launch_act(const CUtensorMap& ta, const CUtensorMap& tb, const PairArgs& a, const Epi& e,
                       cudaStream_t st) {
  if constexpr (PASS == P_WGRAD) {
    return launch_pair<PASS, AQFQ_ACT_NONE, false>(ta, tb, a, e, st);
  } else {
    switch (e.act) {
      case AQFQ_ACT_RELU: return launch_pair<PASS, AQFQ_ACT_RELU, false>(ta, tb, a, e, st);
      case AQFQ_ACT_GELU: return launch_pair<PASS, AQFQ_ACT_GELU, false>(ta, tb, a, e, st);
      case AQFQ_ACT_GELU_TANH: return launch_pair<PASS, AQFQ_ACT_GELU_TANH, false>(ta, tb, a, e, st);
      case AQFQ_ACT_SILU: return launch_pair<PASS, AQFQ_ACT_SILU, false>(ta, tb, a, e, st);
      default: return launch_pair<PASS, AQFQ_ACT_NONE, false>(ta, tb, a, e, st);
    }
  }
}

template <int PASS>
cudaError_t launch_tile(const CUtensorMap& ta, const CUtensorMap& tb, const PairArgs& a, const Epi& e,
                        cudaStream_t st) {
  static DeviceOnce once;
  const cudaError_t attr = once_per_device(once, [] {
    return cudaFuncSetAttribute(tile_kernel<PASS>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemC));
  });
  if (attr != cudaSuccess) return attr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.nr * a.nc * a.splits));
  cfg.blockDim = dim3(32 * kWarpsC);
  cfg.dynamicSmemBytes = kSmemC;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(a.splits), at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tile_kernel<PASS>, ta, tb, a, e);
}

// out[r, c] = epilogue(sum over k of A(r, k) B(c, k)); A, B as stored
template <int PASS>
aqfq_status product(const Operand& A, const Operand& B, int64_t depth, const Epi& e, void* workspace,
                    size_t workspace_bytes, int32_t* err, cudaStream_t st) {
  const Plan p = make_plan(e.rows, e.cols, depth);
  if (p.bytes > 0) {
    if (!workspace || workspace_bytes < p.bytes) return AQFQ_ERR_WORKSPACE;
    if (!al(workspace, 16)) return AQFQ_ERR_ALIGN;
  }
  float* part = static_cast<float*>(workspace);
  if (p.splits > 0) {
    if (!encode_fn()) return AQFQ_ERR_CUDA;
    CUtensorMap ta, tb;
    constexpr bool A_MN = PASS == P_WGRAD, B_MN = PASS != P_FWD;
    if (!encode(&ta, A, kBK, A_MN ? kBK : unsigned(p.a_rows)) ||
        !encode(&tb, B, kBK, B_MN ? kBK : kHalf))
      return AQFQ_ERR_CUDA;
    PairArgs a = {p.nr, p.nc, 0, p.nr * p.nc, p.splits, p.a_rows, p.ksteps, part, p.cols4, err};
    cudaError_t r;
    a.count -= p.tail;
    if (p.small) {
      r = launch_tile<PASS>(ta, tb, a, e, st);
    } else if (p.splits > 1) {  // finish_kernel has the epilogue
      r = launch_pair<PASS, AQFQ_ACT_NONE, false>(ta, tb, a, e, st);
    } else {
      r = launch_act<PASS>(ta, tb, a, e, st);
    }
    if (r != cudaSuccess) return AQFQ_ERR_CUDA;
    if (p.tail > 0) {
      a.first = a.count, a.count = p.tail, a.splits = p.tail_splits;
      if (launch_pair<PASS, AQFQ_ACT_NONE, true>(ta, tb, a, e, st) != cudaSuccess) return AQFQ_ERR_CUDA;
    }
  }
  if (!p.small && p.splits != 1) {
    const int64_t gy = (e.rows + 15) / 16;
    finish_kernel<PASS><<<dim3(unsigned((e.cols + 127) / 128), unsigned(gy > 65535 ? 65535 : gy)), 256,
                          0, st>>>(part, p.splits, p.cols4, e);
    if (cudaGetLastError() != cudaSuccess) return AQFQ_ERR_CUDA;
  }
  return AQFQ_OK;
}

// Sizes of one product.  The inner axis is bounded so that no tile's sum takes
// longer than a bounded wait (2^20 steps of about 0.35 us).
bool size_ok(int64_t v) { return v >= 0 && v <= 0x3FFFFFFF; }
bool inner_ok(int64_t v, int64_t lda, int64_t ldb) {
  return v <= (1 << 26) && lda < (int64_t(1) << 38) && ldb < (int64_t(1) << 38);
}
// operands that the tensor memory accelerator can read: 16-byte base, rows a
// multiple of 16 bytes (and less than 2^40 bytes) apart; an empty one is not read
bool operand_ok(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  return rows == 0 || cols == 0 || (al(p, 16) && ld % 8 == 0);
}

void finish_epi(Epi& e, int es) {
  e.vec_out = rows_aligned<8>(e.out, e.ldo, es);
  e.vec_res = rows_aligned<8>(e.res, e.ldr, 2);
  e.vec_bias = rows_aligned<8>(e.bias, 8, esize(e.bias_dtype));
  e.vec_codes = rows_aligned<8>(e.c.codes, e.cols, 1);
  e.wide = al(e.out, 32) && (e.ldo * es) % 32 == 0 && (!e.res || (al(e.res, 32) && e.ldr % 16 == 0)) &&
           (!e.c.codes || (al(e.c.codes, 16) && e.cols % 16 == 0));
}

}  // namespace
}  // namespace layer
}  // namespace aqfq

using namespace aqfq;
using namespace aqfq::layer;

extern "C" size_t aqfq_linear_workspace_bytes(int pass, int64_t M, int64_t N, int64_t K) {
  if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return 0;
  switch (pass) {
    case AQFQ_LINEAR_FWD: return make_plan(M, N, K).bytes;
    case AQFQ_LINEAR_DGRAD: return make_plan(M, K, N).bytes;
    case AQFQ_LINEAR_WGRAD: return make_plan(N, K, M).bytes;
    default: return 0;
  }
}

extern "C" aqfq_status aqfq_selftest_linear_plan(int pass, int64_t M, int64_t N, int64_t K, int32_t* plan) {
  if (!plan) return AQFQ_ERR_NULL;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return AQFQ_ERR_SHAPE;
  Plan p;
  switch (pass) {
    case AQFQ_LINEAR_FWD: p = make_plan(M, N, K); break;
    case AQFQ_LINEAR_DGRAD: p = make_plan(M, K, N); break;
    case AQFQ_LINEAR_WGRAD: p = make_plan(N, K, M); break;
    default: return AQFQ_ERR_UNSUPPORTED;
  }
  plan[0] = p.ksteps == 0 ? 0 : p.small ? 1 : 2;
  plan[1] = p.splits, plan[2] = p.tail, plan[3] = p.tail_splits;
  return AQFQ_OK;
}

extern "C" aqfq_status aqfq_linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                       int64_t M, int64_t N, int64_t K, int bias_dtype,
                                       const void* bias, int act, const void* residual,
                                       int64_t ldr, void* y, int64_t ldy, const aqfq_ckpt8* ckpt,
                                       void* workspace, size_t workspace_bytes,
                                       int32_t* error_flag, void* stream) {
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !view_ok(M, K, ldx) || !view_ok(N, K, ldw) ||
      !view_ok(M, N, ldy) || (residual && !view_ok(M, N, ldr)) || !inner_ok(K, ldx, ldw))
    return AQFQ_ERR_SHAPE;
  if (!act_ok(act) || !dtype_ok(bias_dtype)) return AQFQ_ERR_UNSUPPORTED;
  Epi e = {};
  if (ckpt) {
    const aqfq_status s = make_ckpt(ckpt, M, N, e.c);
    if (s != AQFQ_OK) return s;
  }
  if (M > 0 && N > 0 && (!y || (K > 0 && (!x || !w)))) return AQFQ_ERR_NULL;
  if (!operand_ok(x, ldx, M, K) || !operand_ok(w, ldw, N, K) || !al(bias, esize(bias_dtype)) ||
      !al(residual, 2) || !al(y, 2) || !al(error_flag, 4))
    return AQFQ_ERR_ALIGN;
  if (M == 0 || N == 0) return AQFQ_OK;
  e.rows = M, e.cols = N;
  e.bias = bias, e.bias_dtype = bias_dtype;
  e.res = static_cast<const bf16*>(residual), e.ldr = ldr;
  e.out = y, e.ldo = ldy, e.out_dtype = AQFQ_BF16, e.act = act;
  finish_epi(e, 2);
  return product<P_FWD>({x, K, M, ldx}, {w, K, N, ldw}, K, e, workspace, workspace_bytes, error_flag,
                        static_cast<cudaStream_t>(stream));
}

extern "C" aqfq_status aqfq_linear_dgrad(const void* dy, int64_t lddy, const void* w, int64_t ldw,
                                         int64_t M, int64_t N, int64_t K, int act,
                                         const aqfq_ckpt8* ckpt, const void* residual,
                                         int64_t ldr, void* dx, int64_t lddx, void* workspace,
                                         size_t workspace_bytes, int32_t* error_flag,
                                         void* stream) {
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !view_ok(M, N, lddy) || !view_ok(N, K, ldw) ||
      !view_ok(M, K, lddx) || (residual && !view_ok(M, K, ldr)) || !inner_ok(N, lddy, ldw))
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
  if (!operand_ok(dy, lddy, M, N) || !operand_ok(w, ldw, N, K) || !al(residual, 2) || !al(dx, 2) ||
      !al(error_flag, 4))
    return AQFQ_ERR_ALIGN;
  if (M == 0 || K == 0) return AQFQ_OK;
  e.rows = M, e.cols = K;
  e.res = static_cast<const bf16*>(residual), e.ldr = ldr;
  e.out = dx, e.ldo = lddx, e.out_dtype = AQFQ_BF16, e.act = act;
  finish_epi(e, 2);
  return product<P_DGRAD>({dy, N, M, lddy}, {w, K, N, ldw}, N, e, workspace, workspace_bytes,
                          error_flag, static_cast<cudaStream_t>(stream));
}

extern "C" aqfq_status aqfq_linear_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                         int64_t M, int64_t N, int64_t K, int dtype, void* dw,
                                         int64_t lddw, int accumulate, void* workspace,
                                         size_t workspace_bytes, int32_t* error_flag,
                                         void* stream) {
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !view_ok(M, N, lddy) || !view_ok(M, K, ldx) ||
      !view_ok(N, K, lddw) || !inner_ok(M, lddy, ldx))
    return AQFQ_ERR_SHAPE;
  if (!dtype_ok(dtype)) return AQFQ_ERR_UNSUPPORTED;
  if (N > 0 && K > 0 && (!dw || (M > 0 && (!dy || !x)))) return AQFQ_ERR_NULL;
  if (!operand_ok(dy, lddy, M, N) || !operand_ok(x, ldx, M, K) || !al(dw, esize(dtype)) || !al(error_flag, 4))
    return AQFQ_ERR_ALIGN;
  if (N == 0 || K == 0) return AQFQ_OK;
  Epi e = {};
  e.rows = N, e.cols = K;
  e.out = dw, e.ldo = lddw, e.out_dtype = dtype, e.accumulate = accumulate;
  finish_epi(e, esize(dtype));
  return product<P_WGRAD>({dy, N, M, lddy}, {x, K, M, ldx}, M, e, workspace, workspace_bytes,
                          error_flag, static_cast<cudaStream_t>(stream));
}
