// Products with MXFP4 weights for few tokens, and the few-token layer on them.
#include "internal.hpp"
#include "row_ops.hpp"

namespace twell {

namespace {

__device__ __forceinline__ float e8m0(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Value of an e2m1 code.
__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * (float)m : (1.f + 0.5f * (float)(m & 1)) * (float)(1 << ((m >> 1) - 1));
  return c & 8u ? -v : v;
}

// 32 values of block b of a row.
__device__ __forceinline__ void w4_block(const W4View& W, int K, int64_t n, int b, float v[32]) {
  const uint4 q = *(const uint4*)(W.code + n * (K / 2) + b * 16);
  const float s = e8m0(W.scale[n * (K / 32) + b]);
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = e2m1(u[i >> 3] >> (4 * (i & 7))) * s;
}

// 32 values of block b of token t.
__device__ __forceinline__ void x_block(const W4Args& a, int64_t t, int b, float v[32]) {
  if (a.x_scale) {
    const uint8_t* p = (const uint8_t*)a.x + t * a.ldx + b * 32;
    const float s = e8m0(a.x_scale[t * (a.K / 32) + b]);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __builtin_amdgcn_cvt_f32_fp8((int)p[i], 0) * s;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) load8<bf16_t>((const uint16_t*)a.x + t * a.ldx, b * 32 + 8 * i, 8, v + 8 * i);
  }
}

// x_t . W[n] by one wave.
__device__ __forceinline__ float w4_dot(const W4Args& a, const W4View& W, int64_t t, int64_t n) {
  float s = 0.f;
  for (int b = threadIdx.x & 63; b < a.K / 32; b += 64) {
    float x[32], w[32];
    x_block(a, t, b, x);
    w4_block(W, a.K, n, b, w);
#pragma unroll
    for (int i = 0; i < 32; ++i) s += x[i] * w[i];
  }
  return wave_sum(s);
}

}  // namespace

// One wave per (token, neuron).
__global__ __launch_bounds__(256) void w4_matvec_kernel(W4Args a) {
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  const float b = a.bias ? bf16_to_f32(a.bias[n]) : 0.f;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const float v = w4_dot(a, a.W, t, n) + b;
    if ((threadIdx.x & 63) == 0) {
      if (a.y_bf16) ((uint16_t*)a.y)[t * a.ldy + n] = (uint16_t)bf16_round(v);
      else ((float*)a.y)[t * a.ldy + n] = v;
    }
  }
}

// a = ReLU(x . Wg^T + bg) * (x . Wu^T).
__global__ __launch_bounds__(256) void w4_act_kernel(W4Args a) {
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  const float b = a.bias ? bf16_to_f32(a.bias[n]) : 0.f;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const float g = w4_dot(a, a.W, t, n) + b;
    const float v = g > 0.f ? g * w4_dot(a, a.Wu, t, n) : 0.f;
    if ((threadIdx.x & 63) == 0) a.act[t * a.N + n] = v;
  }
}

// y_t = sum over n of a * Wd[n]: one thread per 32 columns of a token.
__global__ __launch_bounds__(64) void w4_down_kernel(W4Args a) {
  const int b = blockIdx.x * 64 + threadIdx.x;
  if (b >= a.K / 32) return;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    float acc[32] = {};
    for (int n = 0; n < a.N; ++n) {
      const float v = a.act[t * a.N + n];
      if (v == 0.f) continue;
      float w[32];
      w4_block(a.Wd, a.K, n, b, w);
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] += v * w[i];
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int64_t e = t * a.ldy + b * 32 + i;
      if (a.y_bf16) ((uint16_t*)a.y)[e] = (uint16_t)bf16_round(acc[i]);
      else ((float*)a.y)[e] = acc[i];
    }
  }
}

hipError_t launch_w4_matvec(const W4Args& a, hipStream_t s) {
  w4_matvec_kernel<<<dim3((a.N + 3) / 4, a.T < 1024 ? a.T : 1024), 256, 0, s>>>(a);
  return hipGetLastError();
}

size_t ffn_w4_ws_bytes(int T, int d, int F) {
  (void)d;
  return (size_t)T * F * 4;
}

hipError_t launch_ffn_w4(W4Args a, void* ws, hipStream_t s) {
  a.act = (float*)ws;
  const int ty = a.T < 1024 ? a.T : 1024;
  w4_act_kernel<<<dim3((a.N + 3) / 4, ty), 256, 0, s>>>(a);
  w4_down_kernel<<<dim3((a.K / 32 + 63) / 64, ty), 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace twell
