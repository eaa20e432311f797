// rope.cuh -- rows of a head in registers and their rotation by position, for
// the kernels that rotate (nsa_cache.cu, nsa_cache4.cu, qk_rope.cu).
//
// A thread holds one unit of 16 elements of a row: two runs of eight that are
// loaded and stored 16 (bf16) or 32 (fp32) bytes at a time.
#pragma once

#include "ptx.cuh"

namespace bsa {

constexpr int UNIT = 16;  // elements a thread handles of one row

// f / 2 pi as a fraction of a turn in 2^-64 units, modulo one turn, of a
// finite f >= 0: 24-bit mantissa times 2^64 / 2 pi in 128 bits.
static __device__ uint64_t turns_of(float f) {
  const uint32_t bits = __float_as_uint(fabsf(f));
  const int ex = static_cast<int>(bits >> 23);
  if (ex == 255 || bits == 0u) return 0ull;
  const uint64_t m = ex == 0 ? (bits & 0x7fffffu) : ((bits & 0x7fffffu) | 0x800000u);
  const int sh = (ex == 0 ? 1 : ex) - 150;  // f = m * 2^sh
  constexpr uint64_t C = 2935890503282001226ull;  // 2^64 / 2 pi to the nearest integer
  const uint64_t lo = m * C, hi = __umul64hi(m, C);
  uint64_t u;
  if (sh >= 0) u = sh < 64 ? lo << sh : 0ull;
  else if (sh > -64) u = (lo >> -sh) | (hi << (64 + sh));
  else u = sh > -128 ? hi >> (-sh - 64) : 0ull;
  return f < 0.0f ? 0ull - u : u;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// The 16 elements of unit u of a row: two runs of eight, starting at lo and
// hi, and the first of their eight frequencies (-1: not rotated).  In halves,
// the runs are the two partners of eight pairs; interleaved, and past the
// rotated part, they follow each other.
struct UnitMap {
  int lo, hi, freq;
};
__device__ __forceinline__ UnitMap unit_map(int u, int rotary, bool interleaved) {
  const bool rot = u * UNIT < rotary;
  if (rot && !interleaved) return {8 * u, rotary / 2 + 8 * u, 8 * u};
  return {UNIT * u, UNIT * u + 8, rot ? 8 * u : -1};
}

__device__ __forceinline__ void sincos8(const uint64_t* turns, int freq, int pos, float (&c)[8], float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t t = turns[freq + j] * static_cast<uint64_t>(static_cast<int64_t>(pos));
    // the signed top 32 bits: half-turns in [-1, 1)
    sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, &w[j], &c[j]);
  }
}
__device__ __forceinline__ void rotate16(float (&x)[UNIT], const float (&c)[8], const float (&w)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      x[2 * j] = a * c[j] - b * w[j];
      x[2 * j + 1] = a * w[j] + b * c[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = x[j], b = x[8 + j];
      x[j] = a * c[j] - b * w[j];
      x[8 + j] = a * w[j] + b * c[j];
    }
  }
}

// The same from the pairs' frequencies themselves, times a factor.
__device__ __forceinline__ void sincos8_of(const float* inv_freq, int pos, float factor, float (&c)[8], float (&w)[8]) {
  const float4 f0 = reinterpret_cast<const float4*>(inv_freq)[0], f1 = reinterpret_cast<const float4*>(inv_freq)[1];
  const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t t = turns_of(f[j]) * static_cast<uint64_t>(static_cast<int64_t>(pos));
    sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, &w[j], &c[j]);
    c[j] *= factor;
    w[j] *= factor;
  }
}

// Rows of D elements over a block of ROW_THREADS threads: 2^lanes_log lanes a
// row (the units of a row, rounded up to a power of two: idle lanes hold
// zeros), `tokens` of them at once for each of ROW_THREADS / lanes / tokens
// heads, and `rows` heads a thread one after the other.
constexpr int ROW_THREADS = 256;
struct RowTile {
  int lanes_log, tokens_log;
  int rows;
};

// Fills a block's slots with tokens, then with heads, and gives a thread up to `most` rows once every SM has
// blocks enough (152 x 128 row slots are four blocks a SM of rows of 128).
inline RowTile row_tile(long long tokens, int heads, int D, int most) {
  RowTile t{0, 0, 1};
  while ((UNIT << t.lanes_log) < D) ++t.lanes_log;
  const int slots = ROW_THREADS >> t.lanes_log;
  while ((2 << t.tokens_log) <= slots && (1LL << t.tokens_log) < tokens) ++t.tokens_log;
  const long long share = tokens * heads / (152LL * 4 * slots);
  while (2 * t.rows <= most && 2 * t.rows <= share) t.rows *= 2;
  return t;
}
// Heads of one block.
__host__ __device__ inline int row_heads(const RowTile& t) {
  return (ROW_THREADS >> t.lanes_log >> t.tokens_log) * t.rows;
}

// Sum over a row's lanes.
__device__ __forceinline__ float row_sum(float x, int lanes_log) {
  for (int d = (1 << lanes_log) >> 1; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// A unit as it lies in memory, read ahead of its use.
template <typename T>
struct RawUnit {
  uint4 v[sizeof(T)];
  __device__ __forceinline__ void load(const T* row, const UnitMap& m) {
    const uint4 *lo = reinterpret_cast<const uint4*>(row + m.lo), *hi = reinterpret_cast<const uint4*>(row + m.hi);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      v[i] = lo[i];
      v[sizeof(T) / 2 + i] = hi[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void unpack(float (&x)[UNIT]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
          x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          x[4 * i + j] = __uint_as_float(w[j]);
        }
      }
    }
  }
};

// Sixteen weights of a unit.
__device__ __forceinline__ void load_weights(const void* w, bool f32, const UnitMap& m, float (&x)[UNIT]) {
  float lo[8], hi[8];
  if (f32) {
    load8(static_cast<const float*>(w) + m.lo, lo);
    load8(static_cast<const float*>(w) + m.hi, hi);
  } else {
    load8(static_cast<const __nv_bfloat16*>(w) + m.lo, lo);
    load8(static_cast<const __nv_bfloat16*>(w) + m.hi, hi);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = lo[j];
    x[8 + j] = hi[j];
  }
}

}  // namespace bsa
