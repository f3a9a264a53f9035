// The residual stream around the layer: sum = residual + dropout(x) and its
// root-mean-square norm, forward and backward, and dropout with a residual
// alone.  All of it is a pass over [T][d] rows, bound by memory: 6 to 12
// operations a value.
#include "internal.hpp"
#include "row_ops.hpp"

namespace twell {

namespace {

constexpr int NTH = 256;

struct mx8_t { static constexpr int size = 1; };   // MXFP8 y

__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NTH / 64; ++i) s += sh[i];
  __syncthreads();
  return s;
}

__device__ __forceinline__ void load_w(const NormArgs& a, int c, int n, float w[8]) {
  if (!a.w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (a.w_dt == DT_F32) {
    load8<f32_t>(a.w, c, n, w);
  } else {
    load8<bf16_t>(a.w, c, n, w);
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
  if (n == 8) {
    memcpy(p, code, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (char)(code[i >> 2] >> (8 * (i & 3)));
  }
  if ((c & 31) == 0 && n > 0) a.y_scale[t * ((a.d + 31) / 32) + (c >> 5)] = (uint8_t)byte;
}

}  // namespace

// One workgroup a row; the second pass reads the stored sum back.
template <class X, class R, class Y>
__global__ __launch_bounds__(NTH) void norm_fwd_kernel(NormArgs a) {
  __shared__ float sh[NTH / 64];
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const char* xr = row_of<X>(a.x, t);
    const char* rr = a.res.p ? row_of<R>(a.res, t) : nullptr;
    char* sr = a.sum.p ? row_of<R>(a.sum, t) : nullptr;
    float sq = 0.f;
    for (int c = threadIdx.x * 8; c < a.d; c += NTH * 8) {
      const int n = min(a.d - c, 8);
      float v[8], r[8];
      load8<X>(xr, c, n, v);
      if (a.drop) dropout8(g, t * nb + (c >> 3), a.drop, a.keep_scale, v);
      if (rr) {
        load8<R>(rr, c, n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      if (sr) {
        store8<R>(sr, c, n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = stored<R>(v[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) sq += v[i] * v[i];
    }
    const float rstd = 1.f / sqrtf(block_sum(sq, sh) / (float)a.d + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
    for (int c0 = 0; c0 < a.d; c0 += NTH * 8) {
      const int c = c0 + threadIdx.x * 8, n = max(0, min(a.d - c, 8));
      float v[8] = {}, w[8] = {};
      if (n > 0) {
        if (sr) load8<R>(sr, c, n, v);
        else load8<X>(xr, c, n, v);
        load_w(a, c, n, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] * rstd * w[i] : 0.f;
      if constexpr (Y::size == 1) mx_store(a, t, c, n, v);
      else if (n > 0) store8<Y>(row_of<Y>(a.y, t), c, n, v);
    }
  }
}

// The rows are dealt out to gridDim.x workgroups; each leaves its rows' part
// of dw in its row of `part`.
template <class Y, class R, class X>
__global__ __launch_bounds__(NTH) void norm_bwd_kernel(NormArgs a) {
  __shared__ float sh[NTH / 64];
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  float* part = a.dw ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const char* yr = row_of<Y>(a.y, t);
    const char* sr = row_of<R>(a.sum, t);
    const float rstd = a.rstd_in[t];
    float dot = 0.f;
    for (int c = threadIdx.x * 8; c < a.d; c += NTH * 8) {
      const int n = min(a.d - c, 8);
      float dy[8], v[8], w[8];
      load8<Y>(yr, c, n, dy);
      load8<R>(sr, c, n, v);
      load_w(a, c, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) dot += dy[i] * w[i] * (v[i] * rstd);
    }
    const float cm = block_sum(dot, sh) / (float)a.d;
    for (int c = threadIdx.x * 8; c < a.d; c += NTH * 8) {
      const int n = min(a.d - c, 8);
      float dy[8], v[8], w[8], ds[8] = {};
      load8<Y>(yr, c, n, dy);
      load8<R>(sr, c, n, v);
      load_w(a, c, n, w);
      if (a.res.p) load8<R>(row_of<R>(a.res, t), c, n, ds);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = v[i] * rstd;
        if (part && i < n) part[c + i] = (t == blockIdx.x ? 0.f : part[c + i]) + dy[i] * xh;
        ds[i] += rstd * (dy[i] * w[i] - xh * cm);
      }
      if (a.dres.p) store8<R>(row_of<R>(a.dres, t), c, n, ds);
      if (a.x.p) {
        if (a.drop) dropout8(g, t * nb + (c >> 3), a.drop, a.keep_scale, ds);
        store8<X>(row_of<X>(a.x, t), c, n, ds);
      }
    }
  }
}

// dw = the parts, added in a fixed order.
__global__ __launch_bounds__(NTH) void norm_dw_kernel(const float* part, int parts, int d, float* dw) {
  const int c = blockIdx.x * NTH + threadIdx.x;
  if (c >= d) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += part[(int64_t)i * d + c];
  dw[c] = s;
}

template <class X, class R, class Y>
__global__ __launch_bounds__(NTH) void dropout_add_kernel(NormArgs a) {
  Philox g{};
  if (a.drop) g.load(a.rng);
  const int nb = (a.d + 7) / 8;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
    for (int c = threadIdx.x * 8; c < a.d; c += NTH * 8) {
      const int n = min(a.d - c, 8);
      float v[8], r[8];
      load8<X>(row_of<X>(a.x, t), c, n, v);
      if (a.drop) dropout8(g, t * nb + (c >> 3), a.drop, a.keep_scale, v);
      if (a.res.p) {
        load8<R>(row_of<R>(a.res, t), c, n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      store8<Y>(row_of<Y>(a.y, t), c, n, v);
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

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.T < ROW_GRID ? a.T : ROW_GRID));
  with_types(a.x.dt, a.res.dt, a.y.dt == DT_MXFP8 ? DT_F32 : a.y.dt, [&](auto x, auto r, auto y) {
    using X = decltype(x); using R = decltype(r); using Y = decltype(y);
    if (a.y.dt == DT_MXFP8) norm_fwd_kernel<X, R, mx8_t><<<grid, NTH, 0, s>>>(a);
    else norm_fwd_kernel<X, R, Y><<<grid, NTH, 0, s>>>(a);
  });
  return hipGetLastError();
}

int norm_bwd_parts(int T, int d) {
  (void)d;
  return T < 1024 ? T : 1024;
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const int parts = norm_bwd_parts(a.T, a.d);
  if (a.T > 0)
    with_types(a.y.dt, a.res.dt, a.x.dt, [&](auto y, auto r, auto x) {
      norm_bwd_kernel<decltype(y), decltype(r), decltype(x)><<<dim3(parts), NTH, 0, s>>>(a);
    });
  if (a.dw) norm_dw_kernel<<<dim3((a.d + NTH - 1) / NTH), NTH, 0, s>>>(a.part, parts, a.d, a.dw);
  return hipGetLastError();
}

hipError_t launch_dropout_add(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.T < ROW_GRID ? a.T : ROW_GRID));
  with_types(a.x.dt, a.res.dt, a.y.dt, [&](auto x, auto r, auto y) {
    dropout_add_kernel<decltype(x), decltype(r), decltype(y)><<<grid, NTH, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace twell
