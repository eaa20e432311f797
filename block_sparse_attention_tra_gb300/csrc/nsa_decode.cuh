// nsa_decode.cuh -- what the single-token decodes share: their units of
// softmax, the products and the list of work over whole sequences.  Args: the
// kernels' arguments, with B, Hkv, page, max_pages and lens.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace bsa {

constexpr int STAGE_LOG = 7, STAGE_TOK = 1 << STAGE_LOG;  // tokens of a stage (stream kernel)
constexpr int ROWS = 16;    // heads of a group, padded
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;
constexpr float LSE_EMPTY = -1.0e9f;
// Exponents (log2 domain) are taken against a reference that is set P_SET below the largest score so far when one
// exceeds it by P_MAX: probabilities stay below 2^15 (an f16 ends at 65504).  Sums and accumulators leave a warp in
// units of 2^P_SET.
constexpr float P_SET = 11.0f, P_MAX = 15.0f, P_UNIT = 1.0f / 2048.0f;

// (scores past 2^24, from which 11 cannot be taken without a rounding, are their own reference)
__device__ __forceinline__ float reference_of(float mx) { return fabsf(mx) < 16777216.0f ? mx - P_SET : mx; }

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (not volatile: the compiler interleaves the chains of dependent products)
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// N bytes in 32-bit words, and their copy to shared memory.
template <int N>
struct Words {
  uint32_t w[N / 4];
};
template <int N>
__device__ __forceinline__ Words<N> load_shared(uint32_t p) {
  Words<N> r;
  if constexpr (N == 16)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "r"(p)
                 : "memory");
  else if constexpr (N == 8)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(p) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(p) : "memory");
  return r;
}

// Floats of one partial: (m, l) of each row, then the accumulator rows.
__host__ __device__ constexpr int part_floats(int D) { return ROWS * (D + 2); }

// Tokens that sequence b holds (at most max_pages * page <= 2^31 - 16: what lies behind the last of them is counted in
// unsigned numbers), and the pages and stages of 128 that they make.
template <class Args>
__device__ __forceinline__ int tokens_of(const Args& a, int b) {
  return max(0, min(a.lens[b], a.max_pages * a.page));
}
__host__ __device__ __forceinline__ int pieces_of(int tokens, int size_log) {
  return static_cast<int>((static_cast<uint32_t>(tokens) + (1u << size_log) - 1u) >> size_log);
}
template <class Args>
__device__ __forceinline__ int stages_of(const Args& a, int b) {
  return pieces_of(tokens_of(a, b), STAGE_LOG);
}

// The units (a stage of one kv head) before sequence `upto`; a block-wide call,
// scratch: a long long for each warp.
template <class Args>
__device__ long long units_before(const Args& a, int upto, long long* scratch) {
  long long n = 0;
  for (int b = threadIdx.x; b < upto; b += blockDim.x) n += stages_of(a, b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) n += scratch[w];
  return n * a.Hkv;
}

// The sequence that holds unit u (u < all units), and the units before it; one warp.
template <class Args>
__device__ int sequence_of(const Args& a, long long u, long long* before) {
  const int lane = threadIdx.x & 31;
  long long at = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    long long n = b < a.B ? static_cast<long long>(stages_of(a, b)) * a.Hkv : 0;
    const long long mine = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, u < at + n);
    if (hit != 0u || b0 + 32 >= a.B) {
      const int l = hit != 0u ? __ffs(hit) - 1 : 31;
      *before = at + __shfl_sync(0xffffffffu, n - mine, l);
      return min(b0 + l, a.B - 1);
    }
    at += __shfl_sync(0xffffffffu, n, 31);
  }
}

// Units of the whole list; one warp.
template <class Args>
__device__ long long units_of_warp(const Args& a) {
  long long n = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) n += stages_of(a, b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  return n * a.Hkv;
}

// First unit of range c, floor(units c / ranges), and the range that holds unit u < units.
__device__ __forceinline__ long long range_start(long long units, int c, int ranges) { return units * c / ranges; }
__device__ __forceinline__ int range_of(long long units, long long u, int ranges) {
  return static_cast<int>(((u + 1) * ranges + units - 1) / units - 1);
}

// 1 / sum for a row with tokens, 0 for one without (NaN stays).
__device__ __forceinline__ float inverse_sum(float sum) { return sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum; }
__device__ __forceinline__ float lse_of(float M, float sum) {
  return sum == 0.0f ? LSE_EMPTY : (M + (P_SET + __log2f(sum))) * LN2;
}

}  // namespace bsa
