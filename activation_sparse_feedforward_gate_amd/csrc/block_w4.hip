// Products with MXFP4 weights for few tokens, and the few-token layer on them.
//
// y = x . W^T reads N K / 2 bytes of codes for 2 T N K operations: at up to 64
// tokens it is bound by the weights' bytes, and by latency where they are few.
// So the weights go from memory straight into the matrix instructions' operand
// registers: a lane's 32 consecutive K of one row are one block, 16 bytes of
// codes and one scale byte.  The tokens are the other operand, read from cache
// in fragments too; no tile goes through LDS.  The waves of a workgroup split K
// between them and add their sums in LDS in a fixed order.
// The codes become bf16, times their scale, eight at a time on the way into the
// 16x16x32 bf16 instruction (both e2m1 and e4m3 are exact in bf16).  The scaled
// 8- and 4-bit instructions take them undecoded, but add the products of a step
// at less than fp32's precision: 2^-16 of the sum of magnitudes was seen at
// K = 128, and fp32 outputs are to keep their 24 bits.
#include "internal.hpp"
#include "row_ops.hpp"

namespace twell {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int CHUNK = 128;       // K of one step: four blocks, one per 16 lanes

// Lane l's part of 16 rows (row l % 16) and one chunk (block l / 16) of W.
struct WFrag {
  uint4 q;
  uint32_t s;
};
// The same part of 16 tokens (token l % 16), as loaded.
template <bool MX>
struct XFrag;
template <>
struct XFrag<true> {
  uint4 q[2];
  uint32_t s;
};
template <>
struct XFrag<false> {
  uint4 q[4];
};

struct WPtr {
  const uint8_t* q;
  const uint8_t* s;
};
struct XPtr {
  const char* q;
  const uint8_t* s;
};

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  memcpy(&v, p, 16);
  return v;
}

__device__ __forceinline__ WPtr w_ptr(const W4View& W, int K, int64_t n) {
  const int b = (threadIdx.x >> 4) & 3;
  return {W.code + n * (K / 2) + b * 16, W.scale + n * (K / 32) + b};
}

template <bool MX>
__device__ __forceinline__ XPtr x_ptr(const W4Args& a, int64_t t) {
  const int b = (threadIdx.x >> 4) & 3;
  if constexpr (MX) return {(const char*)a.x + t * a.ldx + b * 32, a.x_scale + t * (a.K / 32) + b};
  else return {(const char*)a.x + (t * a.ldx + b * 32) * 2, nullptr};
}

__device__ __forceinline__ WFrag load_w(const WPtr& p, int ck) {
  return {*(const uint4*)(p.q + (int64_t)ck * 64), p.s[ck * 4]};
}
template <bool MX>
__device__ __forceinline__ XFrag<MX> load_x(const XPtr& p, int ck) {
  XFrag<MX> f;
  if constexpr (MX) {
    f.q[0] = load16(p.q + (int64_t)ck * 128);
    f.q[1] = load16(p.q + (int64_t)ck * 128 + 16);
    f.s = p.s[ck * 4];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.q[j] = load16(p.q + (int64_t)ck * 256 + j * 16);
  }
  return f;
}

// The last chunk where K is no multiple of 128: blocks at and past `left` of it
// count as zeros (of both operands: an infinity or NaN elsewhere must not meet
// them) and are read from the chunk's first block.
__device__ __forceinline__ WFrag load_w_tail(const WPtr& p, int ck, int left) {
  const int b = (threadIdx.x >> 4) & 3, back = b < left ? 0 : b;
  WFrag f{*(const uint4*)(p.q + (int64_t)ck * 64 - back * 16), p.s[ck * 4 - back]};
  if (back) f = {make_uint4(0, 0, 0, 0), 127};
  return f;
}
template <bool MX>
__device__ __forceinline__ XFrag<MX> load_x_tail(const XPtr& p, int ck, int left) {
  const int b = (threadIdx.x >> 4) & 3, back = b < left ? 0 : b;
  constexpr int BLOCK = MX ? 32 : 64;
  XFrag<MX> f;
#pragma unroll
  for (int j = 0; j < BLOCK / 16; ++j) {
    f.q[j] = load16(p.q + (int64_t)ck * (4 * BLOCK) + j * 16 - back * BLOCK);
    if (back) f.q[j] = make_uint4(0, 0, 0, 0);
  }
  if constexpr (MX) f.s = back ? 127 : p.s[ck * 4];
  return f;
}

// Eight codes as bf16, times 2^(s - 127).
__device__ __forceinline__ bf16x8 w_bf16(uint32_t codes, uint32_t s) {
  const float scale = __uint_as_float(s << 23);      // the conversion takes the exponent bits: 0 is 2^-127, 255 NaN
  const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// Eight tokens' values as bf16, j of the block's four.
template <bool MX>
__device__ __forceinline__ bf16x8 x_bf16(const XFrag<MX>& x, int j) {
  if constexpr (MX) {
    const float scale = __uint_as_float(x.s << 23);
    const uint4 q = x.q[j / 2];
    const uint32_t lo = j & 1 ? q.z : q.x, hi = j & 1 ? q.w : q.y;
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
  } else {
    return __builtin_bit_cast(bf16x8, x.q[j]);
  }
}

// acc[r][t] += rows of w[r] x tokens of x[t] over one chunk; lane l's register
// i is row 4 (l / 16) + i of token l % 16.
template <bool MX, int RT, int TT>
__device__ __forceinline__ void chunk_mma(const WFrag w[RT], const XFrag<MX> x[TT], f32x4 acc[RT][TT]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bf16x8 B[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) B[t] = x_bf16<MX>(x[t], j);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const bf16x8 A = w_bf16(j == 0 ? w[r].q.x : j == 1 ? w[r].q.y : j == 2 ? w[r].q.z : w[r].q.w, w[r].s);
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[t], acc[r][t], 0, 0, 0);
    }
  }
}

// Row tiles, token tiles of a workgroup; its waves, which split K; chunks a wave
// has in flight.
template <bool MX_, int RT_, int TT_, int NW_, int U_>
struct Tile {
  static constexpr bool MX = MX_;
  static constexpr int RT = RT_, TT = TT_, NW = NW_, U = U_, NTH = 64 * NW, E = RT * TT;   // E: 16x16 results
  static constexpr int EPW = (E + NW - 1) / NW;      // of them per wave after the sum
};

// Sums of the workgroup's rows (n[r]: this lane's row of tile r) and tokens over
// K: wave w returns results e = w, w + NW, ... of index r * TT + t.
template <class C>
__device__ __forceinline__ void tile_product(const W4Args& a, const W4View& W, const int64_t n[C::RT], int t0,
                                             f32x4 (*red)[C::E][64], f32x4 out[C::EPW]) {
  constexpr int RT = C::RT, TT = C::TT, NW = C::NW, U = C::U;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  WPtr wp[RT];
  XPtr xp[TT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wp[r] = w_ptr(W, a.K, n[r]);
#pragma unroll
  for (int t = 0; t < TT; ++t) xp[t] = x_ptr<C::MX>(a, min(t0 + 16 * t + (lane & 15), a.T - 1));
  f32x4 acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int full = a.K / CHUNK, left = (a.K % CHUNK) / 32;
  for (int ck = w; ck < full; ck += NW * U) {
    // All loads of U chunks first; one past the end repeats the last (no branch
    // between loads) and is not used.
    WFrag wf[U][RT];
    XFrag<C::MX> xf[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = min(ck + u * NW, full - 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) wf[u][r] = load_w(wp[r], c);
#pragma unroll
      for (int t = 0; t < TT; ++t) xf[u][t] = load_x<C::MX>(xp[t], c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ck + u * NW < full) chunk_mma<C::MX, RT, TT>(wf[u], xf[u], acc);
  }
  if (left && w == full % NW) {
    WFrag wf[RT];
    XFrag<C::MX> xf[TT];
#pragma unroll
    for (int r = 0; r < RT; ++r) wf[r] = load_w_tail(wp[r], full, left);
#pragma unroll
    for (int t = 0; t < TT; ++t) xf[t] = load_x_tail<C::MX>(xp[t], full, left);
    chunk_mma<C::MX, RT, TT>(wf, xf, acc);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) red[w][r * TT + t][lane] = acc[r][t];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < C::EPW; ++k) {
    const int e = w + k * NW;
    if (e < C::E) {
      out[k] = red[0][e][lane];
#pragma unroll
      for (int i = 1; i < NW; ++i) out[k] += red[i][e][lane];
    }
  }
}

__device__ __forceinline__ f32x4 bias4(const W4Args& a, int64_t n) {
  f32x4 b{0.f, 0.f, 0.f, 0.f};
  if (a.bias)
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = bf16_to_f32(a.bias[min(n + i, (int64_t)a.N - 1)]);
  return b;
}

}  // namespace

template <class C>
__global__ __launch_bounds__(C::NTH) void w4_matvec_kernel(W4Args a) {
  __shared__ f32x4 red[C::NW][C::E][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * C::RT);
  for (int t0 = blockIdx.y * (16 * C::TT); t0 < a.T; t0 += gridDim.y * (16 * C::TT)) {
    int64_t n[C::RT];
#pragma unroll
    for (int r = 0; r < C::RT; ++r) n[r] = min(n0 + 16 * r + (lane & 15), (int64_t)a.N - 1);
    f32x4 v[C::EPW];
    tile_product<C>(a, a.W, n, t0, red, v);
#pragma unroll
    for (int k = 0; k < C::EPW; ++k) {
      const int e = w + k * C::NW;
      if (e >= C::E) break;
      const int64_t t = t0 + 16 * (e % C::TT) + (lane & 15), m = n0 + 16 * (e / C::TT) + 4 * (lane >> 4);
      if (t >= a.T || m >= a.N) continue;
      const f32x4 o = v[k] + bias4(a, m);
      const int left = (int)min((int64_t)4, a.N - m);
      if (a.y_bf16) {
        uint16_t* y = (uint16_t*)a.y + t * a.ldy + m;
        if (left == 4) {
          const uint32_t u[2] = {bf16_round(o[0]) | bf16_round(o[1]) << 16, bf16_round(o[2]) | bf16_round(o[3]) << 16};
          memcpy(y, u, 8);
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (i < left) y[i] = (uint16_t)bf16_round(o[i]);
        }
      } else {
        float* y = (float*)a.y + t * a.ldy + m;
        if (left == 4) {
          memcpy(y, &o, 16);
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (i < left) y[i] = o[i];
        }
      }
    }
    __syncthreads();
  }
}

// The layer's gate and up products of 16 RT neurons: g = x . Wg^T + bg; where a
// neuron fires (g > 0) for some token of the workgroup, u = x . Wu^T on the
// neurons that fire, and a = g u is stored for the pairs that do, with a bit for
// each pair.  Rows of Wu that no token fires are not read: their lanes take the
// addresses of one that is.
template <class C>
__global__ __launch_bounds__(C::NTH) void w4_gate_up_kernel(W4Args a) {
  __shared__ f32x4 red[C::NW][C::E][64];
  __shared__ uint32_t fires[C::RT];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n0 = blockIdx.x * (16 * C::RT);
  for (int t0 = blockIdx.y * (16 * C::TT); t0 < a.T; t0 += gridDim.y * (16 * C::TT)) {
    int64_t n[C::RT];
#pragma unroll
    for (int r = 0; r < C::RT; ++r) n[r] = n0 + 16 * r + (lane & 15);
    if (threadIdx.x < C::RT) fires[threadIdx.x] = 0;
    f32x4 h[C::EPW], u[C::EPW];
    tile_product<C>(a, a.W, n, t0, red, h);            // has a barrier after the line above
#pragma unroll
    for (int k = 0; k < C::EPW; ++k) {
      const int e = w + k * C::NW;
      if (e >= C::E) break;
      const int t = t0 + 16 * (e % C::TT) + (lane & 15), q = lane >> 4;
      h[k] += bias4(a, n0 + 16 * (e / C::TT) + 4 * q);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m |= (t < a.T && h[k][i] > 0.f) ? 1u << (4 * q + i) : 0u;
      m |= __shfl_xor((int)m, 16);
      m |= __shfl_xor((int)m, 32);
      if (q == 0 && t < a.T) a.mask[(int64_t)t * (a.N / 16) + n0 / 16 + e / C::TT] = (uint16_t)m;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m |= __shfl_xor((int)m, o);
      if (lane == 0 && m) atomicOr(&fires[e / C::TT], m);
    }
    __syncthreads();
    int first = -1;
#pragma unroll
    for (int r = C::RT - 1; r >= 0; --r)
      if (fires[r]) first = n0 + 16 * r + __builtin_ctz(fires[r]);
    if (first >= 0) {
#pragma unroll
      for (int r = 0; r < C::RT; ++r) n[r] = (fires[r] >> (lane & 15)) & 1 ? n[r] : first;
      tile_product<C>(a, a.Wu, n, t0, red, u);
#pragma unroll
      for (int k = 0; k < C::EPW; ++k) {
        const int e = w + k * C::NW;
        if (e >= C::E) break;
        const int64_t t = t0 + 16 * (e % C::TT) + (lane & 15);
        f32x4 v;
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = h[k][i] > 0.f ? h[k][i] * u[k][i] : 0.f;
          any |= h[k][i] > 0.f;
        }
        if (any && t < a.T) *(f32x4*)(a.act + t * a.N + n0 + 16 * (e / C::TT) + 4 * (lane >> 4)) = v;
      }
    }
    __syncthreads();
  }
}

// y_t = sum over the pairs (t, n) that fire, n ascending within a slot, of
// a * Wd[n].  One workgroup per token and DB blocks of 32 columns: the pairs are
// listed in LDS from their bits, NS slots take every NS-th pair, a thread one
// slot and one block (16 bytes of codes, one scale), and the slots are added in
// order.
constexpr int DB = 8, NS = 32, DLIST = 2048;
__global__ __launch_bounds__(DB * NS) void w4_down_kernel(W4Args a) {
  __shared__ int ln[DLIST];
  __shared__ float la[DLIST];
  __shared__ float part[NS][DB][33];
  __shared__ int wsum[DB * NS / 64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int slot = tid / DB, b = blockIdx.x * DB + tid % DB, nblk = a.K / 32;
  const bool live = b < nblk;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const uint64_t* mask = (const uint64_t*)(a.mask + t * (a.N / 16));
    const float* act = a.act + t * a.N;
    float acc[32] = {};
    for (int w0 = 0; w0 < a.N / 64; w0 += DB * NS) {
      uint64_t m = w0 + tid < a.N / 64 ? mask[w0 + tid] : 0;
      const int cnt = popc64(m);
      int pre = cnt;                                    // inclusive scan over the workgroup
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(pre, o);
        if (lane >= o) pre += v;
      }
      if (lane == 63) wsum[w] = pre;
      __syncthreads();
      int total = 0;
#pragma unroll
      for (int i = 0; i < DB * NS / 64; ++i) {
        if (i < w) pre += wsum[i];
        total += wsum[i];
      }
      int at = pre - cnt;
      for (int e0 = 0; e0 < total; e0 += DLIST) {
        while (m && at < e0 + DLIST) {
          const int k = __builtin_ctzll(m);
          m &= m - 1;
          ln[at - e0] = (w0 + tid) * 64 + k;
          ++at;
        }
        __syncthreads();
        const int cntr = min(DLIST, total - e0);
        for (int i = tid; i < cntr; i += DB * NS) la[i] = act[ln[i]];
        __syncthreads();
        if (live)
          for (int i = slot; i < cntr; i += NS) {
            const int64_t n = ln[i];
            const float v = la[i];
            const uint4 q = *(const uint4*)(a.Wd.code + n * (a.K / 2) + b * 16);
            const float s = __uint_as_float((uint32_t)a.Wd.scale[n * nblk + b] << 23);
            const uint32_t c[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#define TWELL_PAIR(k)                                                          \
    {                                                                            \
      const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], s, k);       \
      acc[8 * j + 2 * k] += v * p[0];                                            \
      acc[8 * j + 2 * k + 1] += v * p[1];                                        \
    }
              TWELL_PAIR(0) TWELL_PAIR(1) TWELL_PAIR(2) TWELL_PAIR(3)
#undef TWELL_PAIR
            }
          }
        __syncthreads();
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) part[slot][tid % DB][i] = acc[i];
    __syncthreads();
    const int c = blockIdx.x * (DB * 32) + tid;
    if (c < a.K) {
      float s = part[0][tid / 32][tid % 32];
      for (int i = 1; i < NS; ++i) s += part[i][tid / 32][tid % 32];
      if (a.y_bf16) ((uint16_t*)a.y)[t * a.ldy + c] = (uint16_t)bf16_round(s);
      else ((float*)a.y)[t * a.ldy + c] = s;
    }
    __syncthreads();
  }
}

namespace {

// Calls f with the tile for T tokens and N rows.
template <bool MX, class F>
void with_tile(int T, int64_t N, F f) {
  if (T <= 16) {
    if (N <= 16384) f(Tile<MX, 1, 1, 8, 2>{});
    else f(Tile<MX, 2, 1, 4, 2>{});
  } else if (T <= 32) {
    f(Tile<MX, 1, 2, 4, 2>{});
  } else {
    f(Tile<MX, 1, 4, 4, 1>{});
  }
}

template <class F>
void with_tile(const W4Args& a, F f) {
  if (a.x_scale) with_tile<true>(a.T, a.N, f);
  else with_tile<false>(a.T, a.N, f);
}

constexpr int TOKEN_GRID = 1024;      // workgroups along the tokens; more tokens are walked in a loop

}  // namespace

hipError_t launch_w4_matvec(const W4Args& a, hipStream_t s) {
  with_tile(a, [&](auto c) {
    using C = decltype(c);
    const int rows = 16 * C::RT, toks = (a.T + 16 * C::TT - 1) / (16 * C::TT);
    w4_matvec_kernel<C><<<dim3((a.N + rows - 1) / rows, toks < TOKEN_GRID ? toks : TOKEN_GRID), C::NTH, 0, s>>>(a);
  });
  return hipGetLastError();
}

size_t ffn_w4_ws_bytes(int T, int d, int F) {
  (void)d;
  return (size_t)T * F * 4 + (size_t)T * (F / 8);      // a, and a bit for each pair that fires
}

hipError_t launch_ffn_w4(W4Args a, void* ws, hipStream_t s) {
  a.act = (float*)ws;
  a.mask = (uint16_t*)((char*)ws + (size_t)a.T * a.N * 4);
  with_tile(a, [&](auto c) {
    using C = decltype(c);
    const int rows = 16 * C::RT, toks = (a.T + 16 * C::TT - 1) / (16 * C::TT);
    w4_gate_up_kernel<C><<<dim3(a.N / rows, toks < TOKEN_GRID ? toks : TOKEN_GRID), C::NTH, 0, s>>>(a);
  });
  w4_down_kernel<<<dim3((a.K + DB * 32 - 1) / (DB * 32), a.T < TOKEN_GRID ? a.T : TOKEN_GRID), DB * NS, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace twell
