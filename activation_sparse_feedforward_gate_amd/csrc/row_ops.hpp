// Device helpers of the row kernels: eight columns of a row at a time, fp32 in
// registers, and the counter-based random numbers of dropout.
#pragma once
#include <string.h>

#include "common.hpp"

namespace twell {

struct f32_t { static constexpr int size = 4; };
struct bf16_t { static constexpr int size = 2; };

// bf16 of v, round to nearest even (any v, NaN included).
__device__ __forceinline__ uint32_t bf16_round(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// n valid (0..8) of the eight columns from element c0 of a row: one or two
// 16-byte loads for a whole chunk, single loads at the row's ragged end.  The
// 16-byte accesses need no more than the elements' alignment (global memory is
// in unaligned access mode), so any row stride takes them.
template <class E>
__device__ __forceinline__ void load8(const void* row, int c0, int n, float v[8]) {
  const char* p = (const char*)row + (int64_t)c0 * E::size;
  if (n == 8) {
    if constexpr (E::size == 4) {
      memcpy(v, __builtin_assume_aligned(p, 4), 32);
    } else {
      uint32_t u[4];
      memcpy(u, __builtin_assume_aligned(p, 2), 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(u[i]);
        v[2 * i + 1] = bf16_hi(u[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (i < n) {
        if constexpr (E::size == 4) v[i] = ((const float*)p)[i];
        else v[i] = bf16_to_f32(((const uint16_t*)p)[i]);
      }
    }
  }
}

template <class E>
__device__ __forceinline__ void store8(void* row, int c0, int n, const float v[8]) {
  char* p = (char*)row + (int64_t)c0 * E::size;
  if (n == 8) {
    if constexpr (E::size == 4) {
      memcpy(__builtin_assume_aligned(p, 4), v, 32);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = bf16_round(v[2 * i]) | (bf16_round(v[2 * i + 1]) << 16);
      memcpy(__builtin_assume_aligned(p, 2), u, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (E::size == 4) ((float*)p)[i] = v[i];
        else ((uint16_t*)p)[i] = (uint16_t)bf16_round(v[i]);
      }
  }
}

// v as it reads back from a matrix of element type E.
template <class E>
__device__ __forceinline__ float stored(float v) {
  if constexpr (E::size == 4) return v;
  else return __uint_as_float(bf16_round(v) << 16);
}

// ---------------------------------------------------------------- dropout
// Philox4x32, ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): key and the counter's upper half are
// wave-uniform, the counter's lower half is the block of eight columns.
struct Philox {
  uint32_t k0, k1, o0, o1;
  __device__ __forceinline__ void load(const uint64_t* rng) {
    const uint64_t k = rng[0], o = rng[1];
    k0 = (uint32_t)k; k1 = (uint32_t)(k >> 32);
    o0 = (uint32_t)o; o1 = (uint32_t)(o >> 32);
  }
  __device__ __forceinline__ void words(uint64_t block, uint32_t w[4]) const {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = o0, c3 = o1, a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
      c0 = (uint32_t)(p1 >> 32) ^ c1 ^ a;
      c2 = (uint32_t)(p0 >> 32) ^ c3 ^ b;
      c1 = (uint32_t)p1;
      c3 = (uint32_t)p0;
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
  }
};

// Drops the values of one block whose 16-bit number is below `drop` and scales
// the others: 16 bits a value, so one block of the generator serves eight
// values (its ten rounds cost more than the chunk's loads and stores; at 32
// bits a value they would be paid twice).
__device__ __forceinline__ void dropout8(const Philox& g, uint64_t block, uint32_t drop, float scale, float v[8]) {
  uint32_t w[4];
  g.words(block, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] & 0xffffu) < drop ? 0.f : v[2 * i] * scale;
    v[2 * i + 1] = (w[i] >> 16) < drop ? 0.f : v[2 * i + 1] * scale;
  }
}

}  // namespace twell
