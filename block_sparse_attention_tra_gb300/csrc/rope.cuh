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

// Rows of D elements over a block of ROW_THREADS threads: 2^lanes_log lanes a
// row (its units, rounded up to a power of two: idle lanes hold zeros),
// 2^tokens_log tokens side by side, where tokens are fewer than the block's
// rows several heads of each, and then `rows` heads a thread, one after the
// other.  Blocks over the heads of one tile of tokens follow each other.
//
// Tokens side by side, not heads: [B, H, T, D] tensors have their heads
// megabytes apart, often by a power of two, and with four heads of eight tokens
// side by side 2 x 8192 tokens of 32 + 2 heads of 128 took 123 us in place of
// 54, their gradients 188 in place of 90.
constexpr int ROW_THREADS = 256;
template <int SIDES>
struct RowPlan {
  int lanes_log, tokens_log, rows;
  int groups[SIDES], all_groups;  // blocks over each tensor's heads, over all
  uint32_t tiles;
  __host__ __device__ int head_step() const { return ROW_THREADS >> lanes_log >> tokens_log; }
};
// False if there are too many blocks.  A thread gets up to `most` rows (a power of two): as many as leave six blocks a
// SM (4 x 1031 fp32 rows of 16 + 2 heads of 64: 12.8 us; three blocks 15.0, nine 14.6).
template <int SIDES>
bool plan_rows(RowPlan<SIDES>& p, long long tokens, const int (&heads)[SIDES], int D, int most) {
  p.lanes_log = p.tokens_log = 0;
  while ((UNIT << p.lanes_log) < D) ++p.lanes_log;
  const int slots = ROW_THREADS >> p.lanes_log;
  while ((2 << p.tokens_log) <= slots && (1LL << p.tokens_log) < tokens) ++p.tokens_log;
  const long long tiles = (tokens + (1LL << p.tokens_log) - 1) >> p.tokens_log;
  long long steps = 0;
  for (int s = 0; s < SIDES; ++s) steps += tiles * ((heads[s] + p.head_step() - 1) / p.head_step());
  p.rows = 1;
  while (2 * p.rows <= most && steps > 6LL * 152 * p.rows) p.rows *= 2;
  p.all_groups = 0;
  for (int s = 0; s < SIDES; ++s) {
    const int per = p.head_step() * p.rows;
    p.groups[s] = (heads[s] + per - 1) / per;
    p.all_groups += p.groups[s];
  }
  p.tiles = static_cast<uint32_t>(tiles);
  return tiles * p.all_groups <= 0x7fffffffLL;
}

// What a thread holds: tensor and its group of heads, tile, token (and whether it and the unit are there), first head
// and how many heads, `head_step` apart; `most`: the most of the block's threads.
struct RowPlace {
  int side, group;
  uint32_t tile, token;
  int head, rows, most, head_step, unit;
  bool live;
};
template <int SIDES>
__device__ __forceinline__ RowPlace place_of(const RowPlan<SIDES>& p, long long tokens, const int (&heads)[SIDES], int D) {
  RowPlace x;
  x.tile = blockIdx.x / p.all_groups;
  x.group = static_cast<int>(blockIdx.x % p.all_groups);
  x.side = 0;
  int H = heads[0];
#pragma unroll
  for (int s = 1; s < SIDES; ++s)
    if (x.side == s - 1 && x.group >= p.groups[s - 1]) {
      x.group -= p.groups[s - 1];
      x.side = s;
      H = heads[s];
    }
  x.unit = threadIdx.x & ((1 << p.lanes_log) - 1);
  const int slot = static_cast<int>(threadIdx.x) >> p.lanes_log;
  x.head_step = p.head_step();
  const long long token =
      (static_cast<long long>(x.tile) << p.tokens_log) + (slot & ((1 << p.tokens_log) - 1));
  x.live = token < tokens && x.unit * UNIT < D;
  x.token = x.live ? static_cast<uint32_t>(token) : 0u;  // (all tokens together are a 31-bit number)
  const int head0 = x.group * x.head_step * p.rows;
  x.head = head0 + (slot >> p.tokens_log);
  x.most = min(p.rows, (H - head0 - 1) / x.head_step + 1);
  const int left = H - x.head;  // heads from this thread's first on
  x.rows = x.live && left > 0 ? min(p.rows, (left - 1) / x.head_step + 1) : 0;
  return x;
}

// Sum over a row's lanes (those behind its last unit: zero).
__device__ __forceinline__ float row_sum(float x, int lanes_log, bool in_row) {
  if (!in_row) x = 0.0f;
  if (lanes_log > 2) x += __shfl_xor_sync(0xffffffffu, x, 4);
  if (lanes_log > 1) x += __shfl_xor_sync(0xffffffffu, x, 2);
  if (lanes_log > 0) x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x;
}

// A block's frequencies as fractions of a turn (rotary / 2 <= 64 of them); block-wide.
__device__ __forceinline__ void block_turns(uint64_t (&turns)[64], const float* inv_freq, int rotary) {
  if (static_cast<int>(threadIdx.x) < rotary / 2) turns[threadIdx.x] = turns_of(inv_freq[threadIdx.x]);
  __syncthreads();
}
// Cosines and sines of a unit's eight pairs at a position, times a factor.
__device__ __forceinline__ void unit_sincos(const uint64_t (&turns)[64], int freq, int pos, float factor, float (&c)[8],
                                            float (&w)[8]) {
  sincos8(turns, freq, pos, c, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] *= factor;
    w[j] *= factor;
  }
}

// A unit's 16-byte pieces as numbers.
template <typename T>
__device__ __forceinline__ void unpack(const uint4 (&v)[sizeof(T)], float (&x)[UNIT]) {
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

// Rows on their way to a thread: a ring in shared memory that each thread fills and reads for itself, so that it needs
// no barrier and no registers, in batches of BATCH rows, one in work and one on its way.  A batch's rows are asked for
// at once: out of a projection's layout that is a kilobyte a token.  (In registers, two rows ahead one by one, 2 x 8192
// tokens of 32 + 2 heads of 128 took 54 us in place of 47, their gradients 90 in place of 72.)
template <typename T, int TENSORS>
struct RowRing {
  static constexpr int BATCH = 8 / (static_cast<int>(sizeof(T)) * TENSORS);  // bf16: 4; two tensors or fp32: half
  static constexpr int PIECES = static_cast<int>(sizeof(T));                 // 16-byte pieces of a unit
  static constexpr int BYTES = 2 * BATCH * TENSORS * PIECES * ROW_THREADS * 16;
  // Shared memory of a launch whose threads have `rows` rows, and the kernel made to take it (48 KB need no asking).
  template <class Kernel>
  static int bytes_for(Kernel kern, int rows) {
    const int bytes = rows < 2 * BATCH ? BYTES / (2 * BATCH) * rows : BYTES;
    if (bytes > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES) != cudaSuccess)
      return -1;
    return bytes;
  }
  uint32_t mine;
  __device__ __forceinline__ explicit RowRing(const void* smem) : mine(smem_u32(smem) + threadIdx.x * 16) {}
  __device__ __forceinline__ uint32_t at(int slot, int tensor, int piece) const {
    return mine + ((slot * TENSORS + tensor) * PIECES + piece) * (ROW_THREADS * 16);
  }
  // A unit whose first run starts at lo, its second `apart` elements behind it.
  __device__ __forceinline__ void ask(int slot, int tensor, const T* lo, int apart) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const void* from = reinterpret_cast<const uint4*>(i < PIECES / 2 ? lo : lo + apart) + i % (PIECES / 2);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(slot, tensor, i)), "l"(from) : "memory");
    }
  }
  __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Until all but the batch asked for last are there.
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
  __device__ __forceinline__ void take(int slot, int tensor, float (&x)[UNIT]) const {
    uint4 v[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                   : "r"(at(slot, tensor, i))
                   : "memory");
    unpack<T>(v, x);
  }
};

// Norm and rotation of a unit as one linear map times the row's factor: with c, w the pairs' cosines and sines and g the
// weights (1 without), y_a = s (g_a c x_a - g_b w x_b), y_b = s (g_a w x_a + g_b c x_b).
struct UnitMap2 {
  float aa[8], ab[8], ba[8], bb[8];
};
template <bool INTERLEAVED>
__device__ __forceinline__ void make_map(UnitMap2& m, const float (&c)[8], const float (&w)[8], const float (&g)[UNIT]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float ga = g[INTERLEAVED ? 2 * j : j], gb = g[INTERLEAVED ? 2 * j + 1 : 8 + j];
    m.aa[j] = ga * c[j];
    m.ab[j] = -gb * w[j];
    m.ba[j] = ga * w[j];
    m.bb[j] = gb * c[j];
  }
}
template <bool INTERLEAVED>
__device__ __forceinline__ void apply_map(const UnitMap2& m, float s, float (&x)[UNIT]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int ia = INTERLEAVED ? 2 * j : j, ib = INTERLEAVED ? 2 * j + 1 : 8 + j;
    const float a = x[ia], b = x[ib];
    x[ia] = s * fmaf(m.ab[j], b, m.aa[j] * a);
    x[ib] = s * fmaf(m.bb[j], b, m.ba[j] * a);
  }
}

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
