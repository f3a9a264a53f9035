// The residual stream around the layer: sum = residual + dropout(x) and its
// root-mean-square norm, forward and backward, and dropout with a residual
// alone.  All of it is one pass over [T][d] rows, bound by memory: 6 to 12
// operations a value beside the random numbers.
//
// Rows are held in registers between the row's sum and its use, so every byte
// is read and written once: in the forward up to 16384 columns, in the backward
// up to 8192 (and once more for dw up to 1024 rows).  LPR lanes take a row, CH
// chunks of eight columns each; LPR <= 64 needs no barrier, and 256 / LPR rows
// share a workgroup where LPR < 256.
// Wider rows do not fit the 128 registers a lane of 1024 threads, and part of
// them goes through scratch memory (forward to 32768 columns 9 to 51 registers a
// lane, beyond 174 to 252; backward to 16384 16 to 35); beyond 16384 columns the
// backward reads its rows twice instead.  75 million values, fp32 x or dy, bf16
// rest, dropout: forward 129 us at 2304 columns, 153 at 12288, 145 at 16384, 188
// at 32768, 454 at 65536; backward 180 at 2304, 171 at 8192, 181 at 12288, 179 at
// 16384, 369 at 16392, 350 at 32768, 392 at 65536.
#include "internal.hpp"
#include "row_ops.hpp"

namespace twell {

namespace {

struct mx8_t { static constexpr int size = 1; };   // MXFP8 y

// Sum over the LPR lanes of a row; every lane gets it.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int o = 1; o < (LPR < 64 ? LPR : 64); o <<= 1) v += __shfl_xor(v, o);
  if constexpr (LPR > 64) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    const float* mine = sh + threadIdx.x / LPR * (LPR / 64);
    v = mine[0];
#pragma unroll
    for (int i = 1; i < LPR / 64; ++i) v += mine[i];
    __syncthreads();
  }
  return v;
}

// Eight of the norm's weights as loaded, of either type, with no branch (they are
// loaded with the row, ahead of its sum): two 16-byte loads, of which bf16 needs the
// first.
template <bool SHORT>
struct RawW {
  uint32_t u[8];
};
template <bool SHORT>
__device__ __forceinline__ RawW<SHORT> load_w(const NormArgs& a, int c) {
  RawW<SHORT> r;
  if constexpr (SHORT) {
    if (a.w_dt == DT_F32) {
      const Raw8<f32_t> q = load_raw<f32_t>(a.w, c, a.d - c);
      memcpy(r.u, q.u, 32);
    } else {
      const Raw8<bf16_t> q = load_raw<bf16_t>(a.w, c, a.d - c);
      memcpy(r.u, q.u, 16);
    }
  } else {
    const bool f = a.w_dt == DT_F32;
    const char* p = (const char*)a.w + ((int64_t)min(c, a.d - 8) << (f ? 2 : 1));
    memcpy(r.u, p, 16);
    memcpy(r.u + 4, p + (f ? 16 : 0), 16);
  }
  return r;
}
template <bool SHORT>
__device__ __forceinline__ void w_values(const NormArgs& a, const RawW<SHORT>& r, int c, float w[8]) {
  if (!a.w_given) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (a.w_dt == DT_F32) {
    Raw8<f32_t> q;
    memcpy(q.u, r.u, 32);
    chunk_values<f32_t, SHORT>(q, c, a.d, w);
  } else {
    Raw8<bf16_t> q;
    memcpy(q.u, r.u, 16);
    chunk_values<bf16_t, SHORT>(q, c, a.d, w);
  }
}

template <class E>
__device__ __forceinline__ char* row_of(const RowMat& m, int64_t t) {
  return (char*)m.p + t * m.ld * E::size;
}

// Eight columns as e4m3 codes with the scale of their group of 32 columns,
// which four neighbouring lanes hold (values past the row's end are 0): the
// smallest power of two with |v| <= 448 = 1.75 * 2^8 times it, from the bits of
// the largest |v|.  Every lane of the group has to call it.
__device__ __forceinline__ void mx_encode(const float v[8], uint32_t code[2], uint32_t& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);   // NaN above inf above the rest
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  if (m >= 0x7f800000u) {
    byte = 255;
    code[0] = code[1] = 0x7f7f7f7fu;
    return;
  }
  const int e = (int)(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  byte = (uint32_t)max(e, 0);
  const float inv = __uint_as_float((254u - byte) << 23);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
    code[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, c, true);
  }
}

__device__ __forceinline__ void mx_store(const NormArgs& a, int64_t t, int c, int n, const float v[8]) {
  uint32_t code[2], byte;
  mx_encode(v, code, byte);
  char* p = (char*)a.y.p + t * a.y.ld + c;
  if (n >= 8) {
    memcpy(p, code, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (char)(code[i >> 2] >> (8 * (i & 3)));
  }
  if ((c & 31) == 0 && n > 0) a.y_scale[t * ((a.d + 31) / 32) + (c >> 5)] = (uint8_t)byte;
}

constexpr int threads_of(int lpr) { return lpr < 256 ? 256 : lpr; }

}  // namespace

template <class X, class R, class Y, int LPR, int CH, bool SHORT>
__global__ __launch_bounds__(threads_of(LPR)) void norm_fwd_kernel(NormArgs a) {
  __shared__ float sh[threads_of(LPR) / 64];
  constexpr int RPB = threads_of(LPR) / LPR;
  const int lane = threadIdx.x % LPR;
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  // A row past the end is computed as the last one and not stored (its lanes
  // take part in the shuffles).
  for (int64_t t0 = (int64_t)blockIdx.x * RPB; t0 < a.T; t0 += (int64_t)gridDim.x * RPB) {
    int64_t t = t0 + threadIdx.x / LPR;
    const bool live = t < a.T;
    t = live ? t : a.T - 1;
    const char* xr = row_of<X>(a.x, t);
    const char* rr = row_of<R>(a.res, t);
    char* sr = row_of<R>(a.sum, t);
    Raw8<X> xv[CH];
    Raw8<R> rv[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * LPR + lane) * 8;
      xv[k] = load_chunk<X, SHORT>(xr, c, a.d);
    }
    if (a.res.p) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (k * LPR + lane) * 8;
        rv[k] = load_chunk<R, SHORT>(rr, c, a.d);
      }
    }
    RawW<SHORT> wv[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) wv[k] = load_w<SHORT>(a, (k * LPR + lane) * 8);
    float v[CH][8], sq = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * LPR + lane) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
      if (c < a.d) {
        chunk_values<X, SHORT>(xv[k], c, a.d, v[k]);
        if (a.drop) dropout8(g, t * nb + (c >> 3), a.drop, a.keep_scale, v[k]);
        if (a.res.p) {
          float r[8];
          chunk_values<R, SHORT>(rv[k], c, a.d, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[k][i] += r[i];
        }
        if (a.sum.p) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[k][i] = stored<R>(v[k][i]);
          if (live) store8<R>(sr, c, a.d - c, v[k]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sq += v[k][i] * v[k][i];     // columns past d are 0
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<LPR>(sq, sh) / (float)a.d + a.eps);
    if (live && lane == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * LPR + lane) * 8;
      float w[8];
      if (c < a.d) {
        w_values(a, wv[k], c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * rstd * w[i];
      }
      if constexpr (Y::size == 1) mx_store(a, t, c, live ? a.d - c : 0, v[k]);
      else if (live && c < a.d) store8<Y>(row_of<Y>(a.y, t), c, a.d - c, v[k]);
    }
  }
}

// Some columns of dw by a workgroup of its own, from dy, sum and rstd alone: 8 columns
// a thread, its rows added in order and the threads' sums after them.  As few columns
// as whole 64-byte pieces of both rows allow where a workgroup has only four waves for
// the rows (777 rows of 1001 fp32: 8.8 us, 9.6 with 32 columns).
constexpr int DW_COLS = 32;
constexpr int dw_cols(int y_size, int r_size, int threads) {
  return y_size == 4 && r_size == 4 && threads == 256 ? 16 : DW_COLS;
}
template <class Y, class R, int NTH>
__device__ __forceinline__ void dw_columns(const NormArgs& a, int block, float* sh) {
  constexpr int COLS = dw_cols(Y::size, R::size, NTH), TPR = COLS / 8, ROWS = NTH / TPR, U = 4;
  const int c0 = block * COLS, y = threadIdx.x / TPR, c = c0 + threadIdx.x % TPR * 8, cl = min(c, (a.d - 1) / 8 * 8);
  float s[8] = {};
  for (int64_t t0 = y; t0 < a.T; t0 += ROWS * U) {
    Raw8<Y> yv[U];
    Raw8<R> sv[U];
    float r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = min(t0 + u * ROWS, (int64_t)a.T - 1);
      yv[u] = load_chunk<Y, false>(row_of<Y>(a.y, t), cl, a.d);
      sv[u] = load_chunk<R, false>(row_of<R>(a.sum, t), cl, a.d);
      r[u] = a.rstd_in[t];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + u * ROWS < a.T) {
        float dy[8], v[8];
        chunk_values<Y, false>(yv[u], cl, a.d, dy);
        chunk_values<R, false>(sv[u], cl, a.d, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += dy[i] * (v[i] * r[u]);
      }
  }
  // Threads of a column are added over the lanes of a wave and then over the waves.
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = TPR; o < 64; o <<= 1) s[i] += __shfl_xor(s[i], o);
    if ((threadIdx.x & 63) < TPR) sh[threadIdx.x / 64 * COLS + threadIdx.x % TPR * 8 + i] = s[i];
  }
  __syncthreads();
  if (threadIdx.x < COLS && c0 + (int)threadIdx.x < a.d) {
    float v = sh[threadIdx.x];
    for (int w = 1; w < NTH / 64; ++w) v += sh[w * COLS + threadIdx.x];
    a.dw[c0 + threadIdx.x] = v;
  }
}

// The rows are dealt out to the workgroups past the first a.dw_blocks, of which each
// has some columns of dw; with dw_blocks 0 each leaves its rows' part of dw in its
// row of `part`.
template <class Y, class R, class X, int LPR, int CH, bool SHORT>
__global__ __launch_bounds__(threads_of(LPR)) void norm_bwd_kernel(NormArgs a) {
  constexpr int NTH = threads_of(LPR), RPB = NTH / LPR;
  constexpr int ROW_SH = RPB > 1 ? 8 * NTH : NTH / 64, COL_SH = NTH / 64 * DW_COLS;
  __shared__ float sh[ROW_SH > COL_SH ? ROW_SH : COL_SH];
  if constexpr (!SHORT)
    if ((int)blockIdx.x < a.dw_blocks) return dw_columns<Y, R, NTH>(a, blockIdx.x, sh);
  const int block = blockIdx.x - a.dw_blocks, blocks = gridDim.x - a.dw_blocks;
  const int lane = threadIdx.x % LPR;
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  float dw[CH][8] = {};
  RawW<SHORT> wv[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) wv[k] = load_w<SHORT>(a, (k * LPR + lane) * 8);
  for (int64_t t0 = (int64_t)block * RPB; t0 < a.T; t0 += (int64_t)blocks * RPB) {
    int64_t t = t0 + threadIdx.x / LPR;
    const bool live = t < a.T;
    t = live ? t : a.T - 1;
    const char* yr = row_of<Y>(a.y, t);
    const char* sr = row_of<R>(a.sum, t);
    Raw8<Y> yv[CH];
    Raw8<R> sv[CH], ds[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * LPR + lane) * 8;
      yv[k] = load_chunk<Y, SHORT>(yr, c, a.d);
      sv[k] = load_chunk<R, SHORT>(sr, c, a.d);
    }
    if (a.res.p) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (k * LPR + lane) * 8;
        ds[k] = load_chunk<R, SHORT>(row_of<R>(a.res, t), c, a.d);
      }
    }
    const float rstd = a.rstd_in[t];
    float dot = 0.f;
    float gy[CH][8];                                           // dy * w
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * LPR + lane) * 8;
      if (c < a.d) {
        float v[8], w[8];
        chunk_values<Y, SHORT>(yv[k], c, a.d, gy[k]);
        chunk_values<R, SHORT>(sv[k], c, a.d, v);
        w_values(a, wv[k], c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {                          // columns past d: 0 * 0
          const float xh = v[i] * rstd;
          if (live) dw[k][i] += gy[k][i] * xh;
          gy[k][i] *= w[i];
          dot += gy[k][i] * xh;
        }
      }
    }
    const float cm = row_sum<LPR>(dot, sh) / (float)a.d;
    if (live) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (k * LPR + lane) * 8, n = a.d - c;
        if (n > 0) {
          float v[8], o[8] = {};
          chunk_values<R, SHORT>(sv[k], c, a.d, v);
          if (a.res.p) chunk_values<R, SHORT>(ds[k], c, a.d, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += rstd * (gy[k][i] - v[i] * rstd * cm);
          if (a.dres.p) store8<R>(row_of<R>(a.dres, t), c, n, o);
          if (a.x.p) {
            if (a.drop) dropout8(g, t * nb + (c >> 3), a.drop, a.keep_scale, o);
            store8<X>(row_of<X>(a.x, t), c, n, o);
          }
        }
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)block * a.d;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sh[i * NTH + threadIdx.x] = dw[k][i];
      __syncthreads();
      if (threadIdx.x < LPR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[k][i] = sh[i * NTH + threadIdx.x];
#pragma unroll
          for (int r = 1; r < RPB; ++r) dw[k][i] += sh[i * NTH + r * LPR + threadIdx.x];
        }
      }
    }
    const int c = (k * LPR + lane) * 8;
    if (threadIdx.x < LPR && c < a.d) store8<f32_t>(part, c, a.d - c, dw[k]);
  }
}

// The backward of wide rows (their values, gradients and part of dw do not fit
// the registers): two passes over the row, dw's part kept in memory.
constexpr int WIDE = 1024;
template <class Y, class R, class X>
__global__ __launch_bounds__(WIDE) void norm_bwd_wide_kernel(NormArgs a) {
  __shared__ float sh[WIDE / 64];
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  float* part = a.part ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const char* yr = row_of<Y>(a.y, t);
    const char* sr = row_of<R>(a.sum, t);
    const float rstd = a.rstd_in[t];
    float dot = 0.f;
    for (int c = threadIdx.x * 8; c < a.d; c += WIDE * 8) {
      const int n = min(a.d - c, 8);
      float dy[8], v[8], w[8];
      load8<Y>(yr, c, n, dy);
      load8<R>(sr, c, n, v);
      w_values(a, load_w<false>(a, c), c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) dot += dy[i] * w[i] * (v[i] * rstd);
    }
    const float cm = row_sum<WIDE>(dot, sh) / (float)a.d;
    for (int c = threadIdx.x * 8; c < a.d; c += WIDE * 8) {
      const int n = min(a.d - c, 8);
      float dy[8], v[8], w[8], ds[8] = {}, p[8] = {};
      load8<Y>(yr, c, n, dy);
      load8<R>(sr, c, n, v);
      w_values(a, load_w<false>(a, c), c, w);
      if (a.res.p) load8<R>(row_of<R>(a.res, t), c, n, ds);
      if (part && t != blockIdx.x) load8<f32_t>(part, c, n, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = v[i] * rstd;
        p[i] += dy[i] * xh;
        ds[i] += rstd * (dy[i] * w[i] - xh * cm);
      }
      if (part) store8<f32_t>(part, c, n, p);
      if (a.dres.p) store8<R>(row_of<R>(a.dres, t), c, n, ds);
      if (a.x.p) {
        if (a.drop) dropout8(g, t * nb + (c >> 3), a.drop, a.keep_scale, ds);
        store8<X>(row_of<X>(a.x, t), c, n, ds);
      }
    }
  }
}

// dw = the parts, added in a fixed order: 32 columns a workgroup, 32 threads a
// column.
constexpr int DW_ROWS = 32;
__global__ __launch_bounds__(DW_COLS * DW_ROWS) void norm_dw_kernel(const float* part, int parts, int d, float* dw) {
  __shared__ float sh[DW_ROWS][DW_COLS + 1];
  const int x = threadIdx.x % DW_COLS, y = threadIdx.x / DW_COLS, c = blockIdx.x * DW_COLS + x;
  float s = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int i = y; i < parts; i += DW_ROWS) s += part[(int64_t)i * d + c];
  }
  sh[y][x] = s;
  __syncthreads();
  if (y == 0 && c < d) {
    for (int i = 1; i < DW_ROWS; ++i) s += sh[i][x];
    dw[c] = s;
  }
}

// rpb rows a workgroup where a row has fewer than 256 chunks of eight columns,
// otherwise one.
constexpr int DROP_NTH = 256;
template <class X, class R, class Y, bool SHORT>
__global__ __launch_bounds__(DROP_NTH) void dropout_add_kernel(NormArgs a, int rpb) {
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  const int row = rpb > 1 ? threadIdx.x / nb : 0;
  if (row >= rpb) return;
  for (int64_t t = (int64_t)blockIdx.x * rpb + row; t < a.T; t += (int64_t)gridDim.x * rpb)
    for (int b = rpb > 1 ? threadIdx.x % nb : threadIdx.x; b < nb; b += DROP_NTH) {
      const int c = 8 * b;
      float v[8], r[8];
      const Raw8<X> xv = load_chunk<X, SHORT>(row_of<X>(a.x, t), c, a.d);
      Raw8<R> rv;
      if (a.res.p) rv = load_chunk<R, SHORT>(row_of<R>(a.res, t), c, a.d);
      chunk_values<X, SHORT>(xv, c, a.d, v);
      if (a.drop) dropout8(g, t * nb + b, a.drop, a.keep_scale, v);
      if (a.res.p) {
        chunk_values<R, SHORT>(rv, c, a.d, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      store8<Y>(row_of<Y>(a.y, t), c, a.d - c, v);
    }
}

namespace {

// Calls f(e0, e1, e2) with the element types of three dtypes.
template <class F>
void with_types(int a, int b, int c, F f) {
  auto one = [](int dt, auto g) {
    if (dt == DT_BF16) g(bf16_t{});
    else if (dt == DT_F32) g(f32_t{});
  };
  one(a, [&](auto x) { one(b, [&](auto y) { one(c, [&](auto z) { f(x, y, z); }); }); });
}

constexpr int64_t ROW_GRID = 1 << 20;    // workgroups of a launch; more rows are walked in a loop

// Lanes per row and chunks per lane.
template <int LPR_, int CH_, bool SHORT_ = false>
struct Cfg {
  static constexpr bool SHORT = SHORT_;
  static constexpr int LPR = LPR_, CH = CH_, RPB = threads_of(LPR_) / LPR_;
};

// Few chunks per lane and few idle lanes: two or three chunks in flight per lane
// fill the memory pipe, more cost registers and so waves.  32768 rows of 2304
// (fp32 x, bf16 rest, dropout): <128, 3> 129 us (5.8 TB/s), <256, 2> 144, <64, 5>
// 166, <64, 8> 273; 26810 rows of 2816, <128, 3> 130 and <256, 2> 127 (bf16 x, no
// dropout: 104 and 105).  Up to 1024 rows the time is one row's latency and one chunk
// a lane is fastest: 1 row of 2304 to MXFP8 in a graph, <512, 1> 3.3 us, <128, 3> 4.6;
// fp32 x with dropout, 700 rows of 2048, <256, 1> 5.3, <128, 2> 5.8; 1024 of 2304, 7.6
// and 8.0; 1500 of 4096, 12.4 and 11.9.
template <class F>
void with_fwd_cfg(int T, int d, F f) {
  if (d < 8) return f(Cfg<16, 1, true>{});
  if (T <= 1024 && d > 512) {
    if (d <= 2048) return f(Cfg<256, 1>{});
    if (d <= 4096) return f(Cfg<512, 1>{});
  }
  if (d <= 128) return f(Cfg<16, 1>{});
  if (d <= 256) return f(Cfg<32, 1>{});
  if (d <= 512) return f(Cfg<64, 1>{});
  if (d <= 1024) return f(Cfg<128, 1>{});
  if (d <= 2048) return f(Cfg<128, 2>{});
  if (d <= 2560) return f(Cfg<128, 3>{});
  if (d <= 4096) return f(Cfg<256, 2>{});
  if (d <= 8192) return f(Cfg<512, 2>{});
  if (d <= 16384) return f(Cfg<1024, 2>{});
  if (d <= 32768) return f(Cfg<1024, 4>{});
  return f(Cfg<1024, 8>{});
}

// The backward holds two inputs, the gradient and its part of dw per chunk, and
// its workgroups (the second argument: as many as 256 CUs hold at once) walk
// the rows, so that a part of dw is written once.  32768 rows of 2304: <512, 1>
// 181 us (5.0 TB/s; 187 with twice the workgroups), <128, 3> 226, <256, 2> 288.
constexpr int BWD_MAX_D = 16384;
template <class F>
void with_bwd_cfg(int d, F f) {
  if (d < 8) return f(Cfg<16, 1, true>{}, 1280);
  if (d <= 128) return f(Cfg<16, 1>{}, 1280);
  if (d <= 256) return f(Cfg<32, 1>{}, 1280);
  if (d <= 512) return f(Cfg<64, 1>{}, 1280);
  if (d <= 1024) return f(Cfg<128, 1>{}, 1024);
  if (d <= 2048) return f(Cfg<128, 2>{}, 768);
  if (d <= 4096) return f(Cfg<512, 1>{}, 512);
  if (d <= 8192) return f(Cfg<1024, 1>{}, 256);
  return f(Cfg<1024, 2>{}, 256);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  with_types(a.x.dt, a.res.dt, a.y.dt == DT_MXFP8 ? DT_F32 : a.y.dt, [&](auto x, auto r, auto y) {
    using X = decltype(x); using R = decltype(r); using Y = decltype(y);
    with_fwd_cfg(a.T, a.d, [&](auto c) {
      using C = decltype(c);
      const int64_t blocks = ((int64_t)a.T + C::RPB - 1) / C::RPB;
      const dim3 grid((unsigned)(blocks < ROW_GRID ? blocks : ROW_GRID));
      if (a.y.dt == DT_MXFP8) norm_fwd_kernel<X, R, mx8_t, C::LPR, C::CH, C::SHORT><<<grid, threads_of(C::LPR), 0, s>>>(a);
      else norm_fwd_kernel<X, R, Y, C::LPR, C::CH, C::SHORT><<<grid, threads_of(C::LPR), 0, s>>>(a);
    });
  });
  return hipGetLastError();
}

// Whether dw comes from workgroups of its own: they read dy and sum again, and save the
// second launch and the parts.  fp32 dy, bf16 rest, dropout, 1 row of 2304: 4.0 us, 7.0
// by parts; 500 of 4096: 9.8 and 12.9; 1024 of 2304: 11.7 and 12.7; 777 of 1001, all
// fp32: 8.8 and 10.0; 1000 of 8000: 31.2 and 27.2; 2000 of 512: 11.2 and 9.3.  Not where
// dres or dx is written over dy or sum: other workgroups of the launch would read what
// is new.
bool dw_apart(const NormArgs& a) {
  return a.dw_may_reread && a.d >= 8 && a.d <= BWD_MAX_D && a.T <= 1024 && (int64_t)a.T * a.d <= 4 << 20;
}

int norm_bwd_parts(int T, int d) {
  int64_t blocks = T, most = 512;
  if (d <= BWD_MAX_D)
    with_bwd_cfg(d, [&](auto c, int n) {
      blocks = ((int64_t)T + c.RPB - 1) / c.RPB;
      most = n;
    });
  return (int)(blocks < most ? blocks : most);
}

hipError_t launch_norm_bwd(NormArgs a, hipStream_t s) {
  const int parts = norm_bwd_parts(a.T, a.d);
  const bool apart = a.dw && a.T > 0 && dw_apart(a);
  if (!a.dw || apart) a.part = nullptr;
  if (a.T > 0)
    with_types(a.y.dt, a.res.dt, a.x.dt, [&](auto y, auto r, auto x) {
      using Y = decltype(y); using R = decltype(r); using X = decltype(x);
      if (a.d > BWD_MAX_D) return norm_bwd_wide_kernel<Y, R, X><<<dim3(parts), WIDE, 0, s>>>(a);
      with_bwd_cfg(a.d, [&](auto c, int) {
        using C = decltype(c);
        const int cols = dw_cols(Y::size, R::size, threads_of(C::LPR));
        a.dw_blocks = apart ? (a.d + cols - 1) / cols : 0;
        norm_bwd_kernel<Y, R, X, C::LPR, C::CH, C::SHORT><<<dim3(parts + a.dw_blocks), threads_of(C::LPR), 0, s>>>(a);
      });
    });
  if (a.dw && !apart)
    norm_dw_kernel<<<dim3((a.d + DW_COLS - 1) / DW_COLS), DW_COLS * DW_ROWS, 0, s>>>(a.part, parts, a.d, a.dw);
  return hipGetLastError();
}

hipError_t launch_dropout_add(const NormArgs& a, hipStream_t s) {
  const int nb = (a.d + 7) / 8, rpb = nb < DROP_NTH ? DROP_NTH / nb : 1;
  const int64_t blocks = ((int64_t)a.T + rpb - 1) / rpb;
  const dim3 grid((unsigned)(blocks < ROW_GRID ? blocks : ROW_GRID));
  with_types(a.x.dt, a.res.dt, a.y.dt, [&](auto x, auto r, auto y) {
    using X = decltype(x); using R = decltype(r); using Y = decltype(y);
    if (a.d < 8) dropout_add_kernel<X, R, Y, true><<<grid, DROP_NTH, 0, s>>>(a, rpb);
    else dropout_add_kernel<X, R, Y, false><<<grid, DROP_NTH, 0, s>>>(a, rpb);
  });
  return hipGetLastError();
}

}  // namespace twell
