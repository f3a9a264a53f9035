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

// Eight columns of a row as loaded, and their fp32 values.
template <class E>
struct Raw8;
template <>
struct Raw8<f32_t> {
  uint32_t u[8];
  __device__ __forceinline__ void values(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
  }
};
template <>
struct Raw8<bf16_t> {
  uint32_t u[4];
  __device__ __forceinline__ void values(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(u[i]);
      v[2 * i + 1] = bf16_hi(u[i]);
    }
  }
};

// n valid (0..8, the others 0) of the eight columns from element c0 of a row:
// one or two 16-byte loads for a whole chunk, single loads at the row's ragged
// end.  The 16-byte accesses need no more than the elements' alignment (global
// memory is in unaligned access mode), so any row stride takes them.
template <class E>
__device__ __forceinline__ Raw8<E> load_raw(const void* row, int c0, int n) {
  Raw8<E> r;
  const char* p = (const char*)row + (int64_t)c0 * E::size;
  if (n >= 8) {
    memcpy(r.u, __builtin_assume_aligned(p, E::size), sizeof(r.u));
  } else {
#pragma unroll
    for (uint32_t& u : r.u) u = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) {
        if constexpr (E::size == 4) r.u[i] = ((const uint32_t*)p)[i];
        else r.u[i / 2] |= (uint32_t)((const uint16_t*)p)[i] << (16 * (i & 1));
      }
  }
  return r;
}

template <class E>
__device__ __forceinline__ void load8(const void* row, int c0, int n, float v[8]) {
  load_raw<E>(row, c0, n).values(v);
}

// The same for a kernel that issues the loads of many chunks before it uses
// them: one whole load at min(c, d - 8), with no branch (a branch per chunk ends
// in a wait for its loads), and the ragged last chunk of a row is shifted into
// place when it is used.  Chunks past the row's end load its last columns and
// are not to be used.  SHORT: rows of fewer than eight columns, one chunk in all.
template <class E, bool SHORT>
__device__ __forceinline__ Raw8<E> load_chunk(const void* row, int c, int d) {
  if constexpr (SHORT) return load_raw<E>(row, c, d - c);
  else return load_raw<E>(row, min(c, d - 8), 8);
}
template <class E, bool SHORT>
__device__ __forceinline__ void chunk_values(const Raw8<E>& r, int c, int d, float v[8]) {
  r.values(v);
  if (!SHORT && d % 8) {
    const int miss = c - min(c, d - 8);
#pragma unroll
    for (int k = 4; k; k >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = miss & k ? (i + k < 8 ? v[i + k] : 0.f) : v[i];
  }
}

template <class E>
__device__ __forceinline__ void store8(void* row, int c0, int n, const float v[8]) {
  char* p = (char*)row + (int64_t)c0 * E::size;
  if (n >= 8) {
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
