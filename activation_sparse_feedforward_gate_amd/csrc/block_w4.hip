// Products with MXFP4 weights for few tokens, and the few-token layer on them.
//
// y = x . W^T reads N K / 2 bytes of codes for 2 T N K operations: at up to 64
// tokens it is bound by the weights' bytes, and by latency where they are few.
// The codes become bf16, times their scale, eight at a time on the way into the
// 16x16x32 bf16 instruction (both e2m1 and e4m3 are exact in bf16).  The scaled
// 8- and 4-bit instructions take them undecoded, but add the products of a step
// at less than fp32's precision: 2^-16 of the sum of magnitudes was seen at
// K = 128, and fp32 outputs are to keep their 24 bits.
//
// The address unit takes four lanes a clock if they share 64 bytes and one if they
// do not, and the instruction wants its 16 rows from 16 neighbouring lanes: loads
// straight into its operands run at a quarter of the rate.  Codes, tokens and scales
// are loaded in whole lines instead and turned round in LDS, each wave in a piece of
// its own with no barrier: the waves of a workgroup split K.
// One and two tokens do not use the matrix instruction: 16 lanes take a row, the
// tokens stay in registers, and the waves split K.
// A vector instruction of a wave takes a SIMD 1.8 ns (the conversions are no slower
// than others), so a few hundred of them are as long as the memory's part of a small
// call: the loops below hold little beside the conversions.
// 16 tokens, 40001 x 2048 (46 MB): 11.4 us, 4.1 TB/s; 30001 x 4096 (66 MB): 14.5 us,
// 4.5 TB/s; one token, 9216 x 2304 (11 MB): 4.6 us, one round of loads and the sums over
// the waves (in a graph the shortest kernel takes 1.6 us a launch).
#include <algorithm>
#include <type_traits>

#include "internal.hpp"
#include "row_ops.hpp"

namespace twell {

namespace {

typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int CHUNK = 128;       // K of one step of the matrix path: four blocks, one per 16 lanes
constexpr int GROUP = 512;       // K a wave of the path without it takes at a time

__device__ __forceinline__ u32x4 load16(const void* p) {
  u32x4 v;
  memcpy(&v, p, 16);
  return v;
}

// Between accesses of a wave's own LDS by different lanes.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A scale byte as fp32 2^(byte - 127); the conversions take the exponent bits as
// they are (0 is 2^-127, 255 NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t dword(u32x4 q, int j) { return q[j]; }

__device__ __forceinline__ uint32_t bits(bf16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// Eight codes of weights as bf16, times scale.
__device__ __forceinline__ bf16x8 w_bf16(uint32_t codes, float scale) {
  const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}
// acc += v times eight codes of weights, times scale.
__device__ __forceinline__ void add8(uint32_t codes, float scale, float v, float acc[8]) {
  const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
  const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
  const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
  const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
  const float w[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] += v * w[i];
}
// Eight codes of tokens as bf16, times scale.
__device__ __forceinline__ u32x4 x_bf16(uint32_t lo, uint32_t hi, float scale) {
  return u32x4{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
                    bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
                    bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
                    bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
}

// ---------------------------------------------------------------- the matrix path

// The waves of a workgroup split K; each has RT tiles of 16 rows times TT tiles of
// 16 tokens, with the loads of D chunks in flight.  Up to WAVES waves, with the
// registers of OCC a SIMD.
template <bool MX_, int RT_, int TT_, int WAVES_, int OCC_, int D_>
struct Tile {
  static constexpr bool MX = MX_;
  static constexpr int RT = RT_, TT = TT_, ROWS = 16 * RT, TOKS = 16 * TT;
  static constexpr int E = RT * TT;                  // 16x16 results
  static constexpr int WAVES = WAVES_, OCC = OCC_, D = D_;
  static constexpr int XB = MX ? 128 : 256;          // bytes of a token's chunk
  static constexpr int XP = XB + 16;                 // and of its row in LDS: 16 tokens' same unit lies in all banks
  static constexpr int XL = XB * 16 / 1024;          // loads of a chunk of 16 tokens
};
constexpr int WP = 64;                               // bytes of a row's codes there
// Where 16 bytes `unit` of a row's codes lie: neighbouring lanes write four units of a
// row, and read one unit of as many rows, from all banks either way.
__device__ __forceinline__ int w_at(int row, int unit) {
  return row * WP + (unit ^ ((row >> 1) & 3) ^ (row >> 3 & 1)) * 16;
}
// A wave's piece of LDS.
template <class C>
struct WaveLds {
  char x[C::TOKS * C::XP];
  char w[C::ROWS * WP];
  uint32_t s[C::RT][16 * 4];                         // a group's scales, a chunk's four a dword
  uint32_t xs[C::MX ? C::TT : 1][16 * 4];
};
// A workgroup's, for its waves: their pieces, and then their sums over them.
template <class C>
int tile_lds(int waves) {
  const size_t a = sizeof(WaveLds<C>), b = sizeof(f32x4) * 64 * C::E;
  return waves * (int)(a > b ? a : b);
}

// Byte hi of a dword of scales at the exponent's place of an fp32 (the conversions
// take no other bits of it).
__device__ __forceinline__ float scale_at(uint32_t s, int hi) {
  return __uint_as_float(__builtin_rotateright32(s, 9 + 8 * hi));
}

// Four scales of a row from block b on, a byte each: loaded as the last four at most
// and shifted into place when they are used, so that nothing waits for the load
// before that.  Blocks past the row's end are not to be used.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p, int b, int blocks) {
  uint32_t v = 0;
  if (blocks >= 4) {
    v = *(const u32_any*)(p + min(b, blocks - 4));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) v |= (uint32_t)p[min(i, blocks - 1)] << (8 * i);
  }
  return v;
}
__device__ __forceinline__ uint32_t scales_at(uint32_t v, int b, int blocks) {
  return v >> (8 * (b - min(b, max(blocks - 4, 0))) & 31);
}

// Sums over K of 16 RT rows (row(i): the row of W behind row i) and the tokens from
// t0: wave w of `waves` gets results e = w, w + waves, ... of index r * TT + t in
// out(e, sum); lane l's register i is row 4 (l / 16) + i of token l % 16.
// Each wave takes a run of K's chunks, in pieces of four (their scales are one load).
template <class C, class Row, class Out>
__device__ __forceinline__ void tile_product(const W4Args& a, const W4View& W, Row row, int t0, char* lds, Out out) {
  constexpr int RT = C::RT, TT = C::TT, XL = C::XL, D = C::D;
  constexpr bool MX = C::MX;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int lo = lane & 15, hi = lane >> 4;
  const int blocks = a.K / 32, chunks = (blocks + 3) / 4;
  const int c0 = chunks * w / waves, c1 = chunks * (w + 1) / waves;      // this wave's
  WaveLds<C>& my = *(WaveLds<C>*)(lds + w * sizeof(WaveLds<C>));
  // This lane's addresses: a block of a chunk and a chunk's scales of row lane / 4,
  // and 16 bytes of a token of each load.
  const uint8_t *wp[RT], *sp[RT], *xsp[TT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t n = row(16 * r + lane / 4);
    wp[r] = W.code + n * (a.K / 2);
    sp[r] = W.scale + n * blocks;
  }
  constexpr int TPL = 16 / XL;                       // tokens of a load
  const char* xp[TT][XL];
  const int xt = lane / (64 / TPL), xu = lane % (64 / TPL) * 16;
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int i = 0; i < XL; ++i)
      xp[t][i] = (const char*)a.x + (int64_t)min(t0 + 16 * t + i * TPL + xt, a.T - 1) * a.ldx * (MX ? 1 : 2);
    xsp[t] = MX ? a.x_scale + (int64_t)min(t0 + 16 * t + lane / 4, a.T - 1) * blocks : nullptr;
  }
  char* const xw = my.x + xt * C::XP + xu;
  char* const ww = my.w + w_at(lane / 4, lane & 3);
  const char* const xr = my.x + lo * C::XP + hi * (C::XB / 4);   // block hi of token lo
  const char* const wr = my.w + w_at(lo, hi);                    // block hi of row lo

  f32x4 acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // One chunk from LDS, with its blocks' scales, a byte each; blocks from `nb` on
  // count as zeros of both operands (an infinity or a NaN of one must not meet what
  // was read for the other).
  auto multiply = [&](const uint32_t (&sc)[RT], const uint32_t (&xsc)[TT], int nb) {
    u32x4 q[RT], x[TT][XL];
    float ws[RT], xs[TT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      q[r] = *(const u32x4*)(wr + 16 * r * WP);
      ws[r] = scale_at(sc[r], hi);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int j = 0; j < XL; ++j) x[t][j] = *(const u32x4*)(xr + 16 * t * C::XP + j * 16);
      xs[t] = MX ? scale_at(xsc[t], hi) : 1.f;
    }
    if (nb < 4) {
      const bool in = hi < nb;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        q[r] = in ? q[r] : u32x4{0, 0, 0, 0};
        ws[r] = in ? ws[r] : 1.f;
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        xs[t] = in ? xs[t] : 1.f;
#pragma unroll
        for (int j = 0; j < XL; ++j) x[t][j] = in ? x[t][j] : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 B[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if constexpr (MX) {
          B[t] = __builtin_bit_cast(bf16x8, x_bf16(dword(x[t][j / 2], 2 * (j & 1)), dword(x[t][j / 2], 2 * (j & 1) + 1), xs[t]));
        } else {
          B[t] = __builtin_bit_cast(bf16x8, x[t][j]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const bf16x8 A = w_bf16(dword(q[r], j), ws[r]);
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[t], acc[r][t], 0, 0, 0);
      }
    }
  };

  if (c0 < c1) {
    u32x4 wf[D][RT], xf[D][TT][XL];
    uint32_t sf[RT], xsf[TT] = {};
    // Chunks past the wave's end: its last one again, and blocks past the row's end:
    // its last one, neither used.
    auto load = [&](int ck, int slot) {
      ck = min(ck, c1 - 1);
      const int wo = min(ck * 64 + (lane & 3) * 16, blocks * 16 - 16), xo = min(ck * C::XB + xu, blocks * (C::XB / 4) - 16);
#pragma unroll
      for (int r = 0; r < RT; ++r) wf[slot][r] = *(const u32x4*)(wp[r] + wo);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < XL; ++i) xf[slot][t][i] = load16(xp[t][i] + xo);
    };
    auto load_piece_scales = [&](int ck) {
#pragma unroll
      for (int r = 0; r < RT; ++r) sf[r] = load_scales(sp[r], (ck + (lane & 3)) * 4, blocks);
      if constexpr (MX) {
#pragma unroll
        for (int t = 0; t < TT; ++t) xsf[t] = load_scales(xsp[t], (ck + (lane & 3)) * 4, blocks);
      }
    };
    load_piece_scales(c0);
#pragma unroll
    for (int c = 0; c < D; ++c) load(c0 + c, c);
    auto piece = [&](int g, auto last) {
#pragma unroll
      for (int r = 0; r < RT; ++r) my.s[r][lane] = scales_at(sf[r], (g + (lane & 3)) * 4, blocks);
      if constexpr (MX) {
#pragma unroll
        for (int t = 0; t < TT; ++t) my.xs[t][lane] = scales_at(xsf[t], (g + (lane & 3)) * 4, blocks);
      }
      if constexpr (!last.value) load_piece_scales(g + 4);
      u32x4 sc[RT], xsc[TT];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (last.value && g + c >= c1) break;
#pragma unroll
        for (int r = 0; r < RT; ++r) *(u32x4*)(ww + 16 * r * WP) = wf[c % D][r];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < XL; ++i) *(u32x4*)(xw + (16 * t + i * TPL) * C::XP) = xf[c % D][t][i];
        wave_lds_fence();
        if (c == 0) {
#pragma unroll
          for (int r = 0; r < RT; ++r) sc[r] = *(const u32x4*)&my.s[r][4 * lo];
          if constexpr (MX) {
#pragma unroll
            for (int t = 0; t < TT; ++t) xsc[t] = *(const u32x4*)&my.xs[t][4 * lo];
          }
        }
        if (!last.value || c + D < 4) load(g + c + D, c % D);
        uint32_t s[RT], xs[TT] = {};
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r] = sc[r][c];
        if constexpr (MX) {
#pragma unroll
          for (int t = 0; t < TT; ++t) xs[t] = xsc[t][c];
        }
        multiply(s, xs, blocks - 4 * (g + c));
        wave_lds_fence();
      }
    };
    int g = c0;
#pragma unroll 1
    for (; g + 4 < c1; g += 4) piece(g, std::false_type{});
    piece(g, std::true_type{});
  }
  __syncthreads();                                   // the sums lie over the waves' pieces
  f32x4 (*sum)[C::E][64] = (f32x4(*)[C::E][64])lds;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) sum[w][r * TT + t][lane] = acc[r][t];
  __syncthreads();
  for (int e = w; e < C::E; e += waves) {
    f32x4 v = sum[0][e][lane];
    for (int i = 1; i < waves; ++i) v += sum[i][e][lane];
    out(e, v);
  }
}

__device__ __forceinline__ f32x4 bias4(const W4Args& a, int64_t n) {
  f32x4 b{0.f, 0.f, 0.f, 0.f};
  if (a.bias)
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = bf16_to_f32(a.bias[min(n + i, (int64_t)a.N - 1)]);
  return b;
}

extern __shared__ __attribute__((aligned(16))) char dyn_lds[];

}  // namespace

template <class C>
__global__ __launch_bounds__(64 * C::WAVES, C::OCC) void w4_matvec_kernel(W4Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t n0 = (int64_t)blockIdx.x * C::ROWS;
  for (int t0 = blockIdx.y * C::TOKS; t0 < a.T; t0 += gridDim.y * C::TOKS) {
    tile_product<C>(a, a.W, [&](int i) { return min(n0 + i, (int64_t)a.N - 1); }, t0, dyn_lds, [&](int e, f32x4 o) {
      const int64_t t = t0 + 16 * (e % C::TT) + (lane & 15), m = n0 + 16 * (e / C::TT) + 4 * (lane >> 4);
      if (t >= a.T || m >= a.N) return;
      o += bias4(a, m);
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
    });
    __syncthreads();
  }
}

// The layer's gate and up products of a workgroup's neurons: g = x . Wg^T + bg;
// where a neuron fires (g > 0) for some token of the workgroup, u = x . Wu^T on the
// neurons that fire, listed, 16 at a time, and a = g u is stored for the pairs that
// do, with a bit for each pair.  Other rows of Wu are not read.  (One pair after the
// other, without the tile: the few neurons that fire for many tokens hold their
// workgroup up; 64 tokens at 2048 x 5632, 21.6 us and 17.9.)  F is a multiple of the
// workgroup's rows.
template <class C>
__global__ __launch_bounds__(64 * C::WAVES, C::OCC) void w4_gate_up_kernel(W4Args a) {
  using U = Tile<C::MX, 1, C::TT, C::WAVES, C::OCC, C::D>;
  __shared__ uint32_t fires[C::RT];                  // of each tile of 16 rows
  __shared__ float hl[C::TOKS][C::ROWS + 1];         // max(g, 0), NaN as 0
  __shared__ int list[C::ROWS];                      // the rows that fire
  const int lane = threadIdx.x & 63, n0 = blockIdx.x * C::ROWS;
  for (int t0 = blockIdx.y * C::TOKS; t0 < a.T; t0 += gridDim.y * C::TOKS) {
    if (threadIdx.x < C::RT) fires[threadIdx.x] = 0;
    tile_product<C>(a, a.W, [&](int i) { return (int64_t)(n0 + i); }, t0, dyn_lds, [&](int e, f32x4 h) {
      const int tl = 16 * (e % C::TT) + (lane & 15), t = t0 + tl, q = lane >> 4, r0 = 16 * (e / C::TT);
      h += bias4(a, n0 + r0 + 4 * q);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool f = t < a.T && h[i] > 0.f;
        m |= f ? 1u << (4 * q + i) : 0u;
        hl[tl][r0 + 4 * q + i] = f ? h[i] : 0.f;
      }
      m |= __shfl_xor((int)m, 16);
      m |= __shfl_xor((int)m, 32);
      if (q == 0 && t < a.T) a.mask[(int64_t)t * (a.N / 16) + (n0 + r0) / 16] = (uint16_t)m;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m |= __shfl_xor((int)m, o);
      if (lane == 0 && m) atomicOr(&fires[e / C::TT], m);
    });
    __syncthreads();
    int count = 0;
#pragma unroll
    for (int r = 0; r < C::RT; ++r) {
      const uint32_t m = fires[r];
      if (threadIdx.x < 16 && ((m >> lane) & 1)) list[count + __builtin_popcount(m & ((1u << lane) - 1))] = 16 * r + lane;
      count += __builtin_popcount(m);
    }
    __syncthreads();
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += 16) {
      tile_product<U>(
          a, a.Wu, [&](int i) { return (int64_t)(n0 + list[min(k0 + i, count - 1)]); }, t0, dyn_lds,
          [&](int e, f32x4 u) {
            const int tl = 16 * (e % U::TT) + (lane & 15);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = k0 + 4 * (lane >> 4) + i;
              if (k < count) {
                const float h = hl[tl][list[k]];
                if (h > 0.f) a.act[(int64_t)(t0 + tl) * a.N + n0 + list[k]] = h * u[i];
              }
            }
          });
      __syncthreads();                             // the next tile lies over its sums
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- one and two tokens

namespace {

constexpr int GEMV_ROWS = 16, GEMV_WAVES = 8, GEMV_T = 2;

// Sum over the 16 lanes of a row, in lane 15 of them.
__device__ __forceinline__ float sum16(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x111, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x112, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x114, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x118, 0xf, 0xf, true));
  return v;
}

// A lane's block of weights of four rows, and its eight values of each token.
template <int T>
struct GemvLoads {
  u32x4 q[GEMV_ROWS / 4];
  uint32_t s[GEMV_ROWS / 4];
  u32x4 x[T];
  uint32_t xs[T];
};
template <int T, class Row>
__device__ __forceinline__ void gemv_load(const W4Args& a, const W4View& W, Row row, int rows, int group,
                                          GemvLoads<T>& f) {
  const int lane = threadIdx.x & 63, blocks = a.K / 32, b = min(group * 16 + (lane & 15), blocks - 1);
#pragma unroll
  for (int i = 0; i < GEMV_ROWS / 4; ++i)
    if (4 * i < rows) {
      const int64_t n = row(min(4 * i + (lane >> 4), rows - 1)) * blocks + b;
      f.q[i] = *(const u32x4*)(W.code + n * 16);
      f.s[i] = W.scale[n];
    }
  const int u = min(group * 64 + lane, 4 * blocks - 1);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t tok = min(t, a.T - 1);
    if (a.x_scale) {
      u32x2 q;
      memcpy(&q, (const char*)a.x + tok * a.ldx + 8 * u, 8);
      f.x[t].x = q.x;
      f.x[t].y = q.y;
      f.xs[t] = a.x_scale[tok * blocks + u / 4];
    } else {
      f.x[t] = load16((const char*)a.x + (tok * a.ldx + 8 * u) * 2);
    }
  }
}

// part[wave][t][i]: the wave's part of row(i) . x_t for i < rows; f holds its first
// group's loads.  16 lanes take a row, a block each, so that a load takes 256 bytes
// of each of four rows; the tokens are loaded in whole lines and go through LDS
// (the wave's own, no barrier) into the order of the blocks.
template <int T, class Row>
__device__ __forceinline__ void gemv(const W4Args& a, const W4View& W, Row row, int rows, GemvLoads<T>& f,
                                     u32x4 (*xl)[T][64], float (*part)[T][GEMV_ROWS]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int blocks = a.K / 32;
  float acc[GEMV_ROWS / 4][T] = {};
  for (int g = wave;;) {
#pragma unroll
    for (int t = 0; t < T; ++t)
      xl[wave][t][lane ^ ((lane >> 4) & 3)] = a.x_scale ? x_bf16(f.x[t].x, f.x[t].y, scale_of(f.xs[t])) : f.x[t];
    wave_lds_fence();
    u32x4 x[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = 4 * (lane & 15) + j;
        x[t][j] = xl[wave][t][u ^ ((u >> 4) & 3)];
      }
    wave_lds_fence();
    if (g * 16 + (lane & 15) < blocks) {
#pragma unroll
      for (int i = 0; i < GEMV_ROWS / 4; ++i)
        if (4 * i < rows) {
          const float s = scale_of(f.s[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 w = w_bf16(dword(f.q[i], j), s);
#pragma unroll
            for (int t = 0; t < T; ++t) {
              const bf16x8 v = __builtin_bit_cast(bf16x8, x[t][j]);
#pragma unroll
              for (int k = 0; k < 8; k += 2)
                acc[i][t] = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{w[k], w[k + 1]}, bf16x2{v[k], v[k + 1]}, acc[i][t], false);
            }
          }
        }
    }
    g += waves;
    if (g * 16 >= blocks) break;
    gemv_load<T>(a, W, row, rows, g, f);
  }
#pragma unroll
  for (int i = 0; i < GEMV_ROWS / 4; ++i)
    if (4 * i < rows) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float v = sum16(acc[i][t]);
        if ((lane & 15) == 15) part[wave][t][4 * i + (lane >> 4)] = v;
      }
    }
}

}  // namespace

template <int T>
__global__ __launch_bounds__(64 * GEMV_WAVES) void w4_gemv_kernel(W4Args a) {
  __shared__ u32x4 xl[GEMV_WAVES][T][64];
  __shared__ float part[GEMV_WAVES][T][GEMV_ROWS];
  const int64_t n0 = (int64_t)blockIdx.x * GEMV_ROWS;
  const int rows = (int)min((int64_t)GEMV_ROWS, a.N - n0);
  auto row = [&](int i) { return n0 + i; };
  GemvLoads<T> f;
  gemv_load<T>(a, a.W, row, rows, threadIdx.x >> 6, f);
  gemv<T>(a, a.W, row, rows, f, xl, part);
  __syncthreads();
  const int i = threadIdx.x % GEMV_ROWS, t = threadIdx.x / GEMV_ROWS;
  if (t >= min(T, a.T) || i >= rows) return;
  float v = part[0][t][i];
  for (int w = 1; w < (int)(blockDim.x >> 6); ++w) v += part[w][t][i];
  if (a.bias) v += bf16_to_f32(a.bias[n0 + i]);
  if (a.y_bf16) ((uint16_t*)a.y)[t * a.ldy + n0 + i] = (uint16_t)bf16_round(v);
  else ((float*)a.y)[t * a.ldy + n0 + i] = v;
}

// The layer's gate and up products of 16 neurons, as w4_gate_up_kernel.
template <int T>
__global__ __launch_bounds__(64 * GEMV_WAVES) void w4_gate_up_gemv_kernel(W4Args a) {
  __shared__ u32x4 xl[GEMV_WAVES][T][64];
  __shared__ float part[GEMV_WAVES][T][GEMV_ROWS];
  const int64_t n0 = (int64_t)blockIdx.x * GEMV_ROWS;
  auto row = [&](int i) { return n0 + i; };
  GemvLoads<T> f;
  gemv_load<T>(a, a.W, row, GEMV_ROWS, threadIdx.x >> 6, f);
  gemv<T>(a, a.W, row, GEMV_ROWS, f, xl, part);
  __syncthreads();
  // every wave adds and packs for itself: lane 16 t + i has token t, row i
  const int lane = threadIdx.x & 63, i = lane & 15, t = lane >> 4, waves = blockDim.x >> 6;
  const bool live = t < T && t < a.T;
  float h = 0.f;
  if (live) {
    for (int w = 0; w < waves; ++w) h += part[w][t][i];
    if (a.bias) h += bf16_to_f32(a.bias[n0 + i]);
  }
  const uint64_t m = ballot(live && h > 0.f);
  const uint32_t any = (uint32_t)(m | m >> 16 | m >> 32 | m >> 48) & 0xffffu;      // neurons that fire for some token
  if (threadIdx.x < 64 && i == 0 && live) a.mask[(int64_t)t * (a.N / 16) + blockIdx.x] = (uint16_t)(m >> (16 * t));
  if (!any) return;
  const int rows = __builtin_popcount(any);
  auto fired = [&](int k) {                            // the k-th of them
    uint32_t r = any;
    for (; k > 0; --k) r &= r - 1;
    return n0 + __builtin_ctz(r);
  };
  gemv_load<T>(a, a.Wu, fired, rows, threadIdx.x >> 6, f);
  __syncthreads();                                     // part is read
  gemv<T>(a, a.Wu, fired, rows, f, xl, part);
  __syncthreads();
  if (threadIdx.x < 64 && h > 0.f) {
    const int k = __builtin_popcount(any & ((1u << i) - 1));
    float u = 0.f;
    for (int w = 0; w < waves; ++w) u += part[w][t][k];
    a.act[(int64_t)t * a.N + n0 + i] = h * u;
  }
}

// ---------------------------------------------------------------- the down product

// y_t = sum over the pairs (t, n) that fire of a * Wd[n].  One workgroup per token
// and DC columns: the pairs are listed in LDS from their bits, in order; DL lanes take
// a row, eight columns each (whole lines), DS slots every DS-th pair with DU of them in
// flight, and the slots are added in order.  Its time is a chain of waits: bits, list,
// rows, sums.
constexpr int DLIST = 2048;
template <int DC_, int DS_, int DU_>
struct Down {
  static constexpr int DC = DC_, DL = DC / 8, DS = DS_, DU = DU_, DTH = DL * DS;
};

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);        // from 1, 2, 4, 8 lanes down in 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);       // lane 15 of the 16 before, to every other 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);       // lane 31, to the upper half
  return v;
}

template <class C>
__global__ __launch_bounds__(C::DTH) void w4_down_kernel(W4Args a) {
  constexpr int DC = C::DC, DL = C::DL, DS = C::DS, DU = C::DU, DTH = C::DTH;
  __shared__ int ln[DLIST];
  __shared__ __attribute__((aligned(16))) float part[DS][DC];
  __shared__ int wsum[DTH / 64];
  const int tid = threadIdx.x, w = tid >> 6;
  const int slot = tid / DL, c = blockIdx.x * DC + tid % DL * 8, nblk = a.K / 32;
  const bool live = c < a.K;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const uint64_t* mask = (const uint64_t*)(a.mask + t * (a.N / 16));
    const float* act = a.act + t * a.N;
    float acc[8] = {};
    for (int w0 = 0; w0 < a.N / 64; w0 += DTH) {
      uint64_t m = w0 + tid < a.N / 64 ? mask[w0 + tid] : 0;
      const int cnt = popc64(m);
      int pre = wave_scan(cnt);
      if ((tid & 63) == 63) wsum[w] = pre;
      __syncthreads();
      int total = 0;
#pragma unroll
      for (int i = 0; i < DTH / 64; ++i) {
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
        if (live)
          for (int i0 = slot; i0 < cntr; i0 += DS * DU) {
            uint32_t q[DU], sc[DU];
            float v[DU];
#pragma unroll
            for (int u = 0; u < DU; ++u) {
              const int64_t n = ln[min(i0 + u * DS, cntr - 1)];
              v[u] = act[n];
              q[u] = *(const uint32_t*)(a.Wd.code + n * (a.K / 2) + c / 2);
              sc[u] = a.Wd.scale[n * nblk + c / 32];
            }
#pragma unroll
            for (int u = 0; u < DU; ++u)
              if (i0 + u * DS < cntr) add8(q[u], scale_of(sc[u]), v[u], acc);
          }
        __syncthreads();
      }
      __syncthreads();
    }
    *(f32x4*)&part[slot][tid % DL * 8] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    *(f32x4*)&part[slot][tid % DL * 8 + 4] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    __syncthreads();
    const int o = blockIdx.x * DC + tid;
    if (tid < DC && o < a.K) {            // DC <= DTH
      float s = part[0][tid];
#pragma unroll
      for (int i = 1; i < DS; ++i) s += part[i][tid];
      if (a.y_bf16) ((uint16_t*)a.y)[t * a.ldy + o] = (uint16_t)bf16_round(s);
      else ((float*)a.y)[t * a.ldy + o] = s;
    }
    __syncthreads();
  }
}

namespace {

// Calls f with the tile for the tokens and rows.  32 rows x 16 tokens, unless there is
// no more than one workgroup of 16 x 16 for each CU, or more than 16 tokens go with
// enough rows of a product for tiles that read them half as often and still are many (the
// borders in rows were measured with 20 to 64 tokens; the layer's list of
// rows that fire grows with its tile).  With the tile of the neighbouring range: 30
// tokens, 700 x 8192, 6.2 us and 9.1 (small); 64 tokens, 2048 x 2048, 4.3 and 5.0
// (narrow); 9216 x 2304, 11.4 and 11.8 (middle); 12000 x 2048, 11.9 and 14.3 (small);
// 20 tokens, 16000 x 4096, 12.0 and 16.8 (small); 64 tokens, 40001 x 2048, 25 and 28
// (middle).  MXFP8 tokens take half the registers and leave room for a second chunk in
// flight (16 tokens, 40001 x 2048: 12.4 us, and 11.4 with it; in bf16, 64 tokens, 9216
// x 2304, 11.1 and 11.8).
template <bool MX>
using Narrow = Tile<MX, 1, 1, 8, 3, MX ? 2 : 1>;
template <bool MX>
using Small = Tile<MX, 2, 1, 8, 3, MX ? 2 : 1>;
template <bool MX>
using Middle = Tile<MX, 2, 2, 4, 2, 1>;
template <bool MX>
using Large = Tile<MX, 4, 2, 4, 2, 1>;
template <bool PRODUCT, class F>
void with_tile(const W4Args& a, F f) {
  auto go = [&](auto mx) {
    if constexpr (PRODUCT) {
      if (a.T > 16 && a.N > 16384) return f(Large<mx.value>{});
      if (a.T > 16 && a.N > 10240) return f(Middle<mx.value>{});
    }
    if ((int64_t)((a.N + 15) / 16) * ((a.T + 15) / 16) <= 256) f(Narrow<mx.value>{});
    else f(Small<mx.value>{});
  };
  if (a.x_scale) go(std::true_type{});
  else go(std::false_type{});
}

// Waves of a workgroup: one per group of K, up to `most`.
int waves_of(const W4Args& a, int most) {
  const int groups = (a.K + GROUP - 1) / GROUP;
  return groups < most ? groups : most;
}

constexpr int TOKEN_GRID = 1024;      // workgroups along the tokens; more tokens are walked in a loop

template <class C>
dim3 tile_grid(const W4Args& a) {
  const int toks = (a.T + C::TOKS - 1) / C::TOKS;
  return dim3((a.N + C::ROWS - 1) / C::ROWS, toks < TOKEN_GRID ? toks : TOKEN_GRID);
}

// The same of the matrix path.  Where workgroups are many, about one per four chunks (the
// waves' sums go through LDS at the end) and no three, which load the SIMDs unevenly;
// otherwise one per chunk, up to four, and to eight where there is no more than a
// workgroup for each CU and K is long.  9 tokens, 3001 x 480: 3.2 us, and 4.0 with one
// per four; 5 tokens, 5000 x 16384: 13.2, and 17.1 with four; 64 tokens, 9216 x 2304:
// 14.6 with eight and 11.5; 41 tokens, 39755 x 1248: 22.7 with four, 25.4 with three; 64
// tokens, 16000 x 1024: 8.0 with two, 10.4 with three; 65536 x 512: 18.7 with two, 15.2
// with one.
template <class C>
int tile_waves(const W4Args& a) {
  const dim3 g = tile_grid<C>(a);
  const int64_t groups = (int64_t)g.x * g.y;
  const int chunks = (a.K + CHUNK - 1) / CHUNK;
  if (C::TT > 1 || groups > 1024) return chunks > 8 ? 4 : chunks > 4 ? 2 : 1;
  const int most = groups <= 256 && (C::RT == 1 || chunks >= 32) ? 8 : 4;
  return chunks < most ? chunks : most;
}

// Calls f with the down product's workgroup: 64 columns and many slots, the shortest
// chain, while there are few of them; 256 columns list the pairs a quarter as often.
// The layer, one token at 2304 x 9216: 9.7 us and 10.3; 48 tokens at 4096 x 6144: 30.3
// and 24.8.
template <class F>
void with_down(const W4Args& a, F f) {
  if ((int64_t)a.T * ((a.K + 63) / 64) <= 512) f(Down<64, 32, 4>{});
  else f(Down<256, 16, 6>{});
}

bool use_gemv(const W4Args& a) { return a.T <= GEMV_T; }

// Calls f with the tokens of the kernel and its workgroup.
template <class F>
void with_gemv(const W4Args& a, F f) {
  const int threads = 64 * waves_of(a, GEMV_WAVES);
  if (a.T == 1) f(std::integral_constant<int, 1>{}, threads);
  else f(std::integral_constant<int, GEMV_T>{}, threads);
}

}  // namespace

// Rows and tokens of one launch.  A grid holds fewer than 2^32 threads along an axis (32
// a row at most: 16 rows to eight waves), and the kernels count tokens in 32 bits, with up
// to TOKEN_GRID tiles added to the last one's.
constexpr int64_t ROW_RUN = 1 << 26, TOKEN_RUN = 1 << 24;

hipError_t launch_w4_matvec(const W4Args& all, hipStream_t s) {
  for (int64_t n = 0; n < all.N; n += ROW_RUN)
    for (int64_t t = 0; t < all.T; t += TOKEN_RUN) {
      W4Args a = all;
      a.N = (int)std::min(ROW_RUN, all.N - n);
      a.T = (int)std::min(TOKEN_RUN, all.T - t);
      a.x = (const char*)all.x + t * all.ldx * (all.x_scale ? 1 : 2);
      if (all.x_scale) a.x_scale = all.x_scale + t * (all.K / 32);
      a.W.code = all.W.code + n * (all.K / 2);
      a.W.scale = all.W.scale + n * (all.K / 32);
      if (all.bias) a.bias = all.bias + n;
      a.y = (char*)all.y + (t * all.ldy + n) * (all.y_bf16 ? 2 : 4);
      if (use_gemv(a)) {
        with_gemv(a, [&](auto t, int threads) {
          w4_gemv_kernel<t.value><<<dim3((a.N + GEMV_ROWS - 1) / GEMV_ROWS), threads, 0, s>>>(a);
        });
      } else {
        with_tile<true>(a, [&](auto c) {
          using C = decltype(c);
          w4_matvec_kernel<C><<<tile_grid<C>(a), 64 * tile_waves<C>(a), tile_lds<C>(tile_waves<C>(a)), s>>>(a);
        });
      }
    }
  return hipGetLastError();
}

size_t ffn_w4_ws_bytes(int T, int d, int F) {
  (void)d;
  return (size_t)T * F * 4 + (size_t)T * (F / 8);      // a, and a bit for each pair that fires
}

hipError_t launch_ffn_w4(W4Args a, void* ws, hipStream_t s) {
  a.act = (float*)ws;
  a.mask = (uint16_t*)((char*)ws + (size_t)a.T * a.N * 4);
  if (use_gemv(a)) {
    with_gemv(a, [&](auto t, int threads) {
      w4_gate_up_gemv_kernel<t.value><<<dim3(a.N / GEMV_ROWS), threads, 0, s>>>(a);
    });
  } else {
    with_tile<false>(a, [&](auto c) {
      using C = decltype(c);
      w4_gate_up_kernel<C><<<tile_grid<C>(a), 64 * tile_waves<C>(a), tile_lds<C>(tile_waves<C>(a)), s>>>(a);
    });
  }
  with_down(a, [&](auto c) {
    using C = decltype(c);
    w4_down_kernel<C><<<dim3((a.K + C::DC - 1) / C::DC, a.T < TOKEN_GRID ? a.T : TOKEN_GRID), C::DTH, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace twell
