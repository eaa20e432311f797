// nsa_decode.cuh -- what the single-token decodes share: their units of
// softmax, the products, the list of work over whole sequences and the join of
// the parts that its ranges leave.  Args: the kernels' arguments, with B, Hq,
// Hkv, G, page, max_pages, ranges, lens, ws, out and lse.
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
__device__ __forceinline__ int pieces_of(int tokens, int size_log) {
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

// Joins the parts of a (sequence, kv head) that several ranges cover, and
// answers for a sequence without tokens.  One block for two rows of it, eight
// warps a row: each takes every eighth part, and the eight are joined last (a
// pair of long sequences has tens of parts: with four warps a row four
// sequences of up to 131072 tokens took 44.1 us, with one 48.9, now 43.2).
constexpr int JOIN_ROWS = 2, JOIN_WARPS = 8, JOIN_THREADS = JOIN_ROWS * JOIN_WARPS * 32;
template <int D, class Args>
__global__ void __launch_bounds__(JOIN_THREADS) nsa_decode_join_kernel(const Args a) {
  constexpr int V = D / 32 > 0 ? D / 32 : 1, LANES = D / V;  // dims of a lane, lanes of a row
  __shared__ long long scratch[JOIN_ROWS * JOIN_WARPS];
  __shared__ int ends[2];  // ranges that hold its first and last unit
  __shared__ float2 state[JOIN_ROWS][JOIN_WARPS];
  __shared__ float rows[JOIN_ROWS][JOIN_WARPS][D];
  const int groups = (a.G + JOIN_ROWS - 1) / JOIN_ROWS;
  const int item = blockIdx.x / groups;
  const int b = item / a.Hkv, h = item % a.Hkv;
  const int np = stages_of(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / JOIN_WARPS, w4 = warp % JOIN_WARPS, row = blockIdx.x % groups * JOIN_ROWS + sub;
  float M = -INFINITY, sum = 0.0f, o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = 0.0f;
  if (np > 0) {
    const long long units = units_before(a, a.B, scratch);
    const long long u0 = units_before(a, b, scratch) + static_cast<long long>(h) * np, u1 = u0 + np;
    if (threadIdx.x < 2) ends[threadIdx.x] = range_of(units, threadIdx.x ? u1 - 1 : u0, a.ranges);
    __syncthreads();
    const int c0 = ends[0], c1 = ends[1];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel is complete
    if (c0 == c1) return;  // written by its only range
    if (row < a.G) {
      // the part that range c left (none if the range is empty: a list shorter than the ranges)
      auto part_of = [&](int c) -> const float* {
        const long long start = range_start(units, c, a.ranges);
        if (c > c1 || start == range_start(units, c + 1, a.ranges)) return nullptr;
        return a.ws + (2 * static_cast<size_t>(c) + (start < u0 ? 1 : 0)) * part_floats(D);
      };
      for (int base = c0; base <= c1; base += 32 * JOIN_WARPS) {
        const int c = base + lane * JOIN_WARPS + w4;  // this lane's part
        const float* mine = part_of(c);
        const float2 pml = mine != nullptr ? *reinterpret_cast<const float2*>(mine + 2 * row)
                                           : make_float2(-INFINITY, 0.0f);
        float n = fmaxf(M, pml.x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
        const float nb = n == -INFINITY ? 0.0f : n, s = ex2f(M - nb), w = ex2f(pml.x - nb);
        M = n;
        float part_sum = pml.y * w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) part_sum += __shfl_xor_sync(0xffffffffu, part_sum, d);
        sum = sum * s + part_sum;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= s;
        const int count = min(32, (c1 - base - w4 + JOIN_WARPS) / JOIN_WARPS);  // parts of this warp in this turn
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          const float* from = reinterpret_cast<const float*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), k));
          const float* acc = from + 2 * ROWS + row * D;
          if (from != nullptr && lane < LANES) {
            if constexpr (V == 4) {
              const float4 v = *reinterpret_cast<const float4*>(acc + lane * 4);
              o[0] = fmaf(wk, v.x, o[0]);
              o[1] = fmaf(wk, v.y, o[1]);
              o[2] = fmaf(wk, v.z, o[2]);
              o[3] = fmaf(wk, v.w, o[3]);
            } else {
#pragma unroll
              for (int e = 0; e < V; ++e) o[e] = fmaf(wk, acc[lane * V + e], o[e]);
            }
          }
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (lane == 0) state[sub][w4] = make_float2(M, sum);
  if (lane < LANES)
#pragma unroll
    for (int e = 0; e < V; ++e) rows[sub][w4][lane * V + e] = o[e];
  __syncthreads();
  if (w4 != 0 || row >= a.G) return;
  float top = -INFINITY, total = 0.0f;
#pragma unroll
  for (int k = 0; k < JOIN_WARPS; ++k) top = fmaxf(top, state[sub][k].x);
  const float tb = top == -INFINITY ? 0.0f : top;
  float x[V];
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = 0.0f;
#pragma unroll
  for (int k = 0; k < JOIN_WARPS; ++k) {
    const float w = ex2f(state[sub][k].x - tb);
    total += w * state[sub][k].y;
    if (lane < LANES)
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] += w * rows[sub][k][lane * V + e];
  }
  const float inv = inverse_sum(total);
  const size_t orow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G + row;
  if (lane < LANES)
#pragma unroll
    for (int e = 0; e < V; ++e) a.out[orow * D + lane * V + e] = __float2bfloat16_rn(x[e] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[orow] = lse_of(top, total);
}

// Its launch behind the first kernel: started while that one's last blocks run
// (its blocks wait before they read a part).
template <int D, class Args>
int launch_decode_join(const Args& a, cudaStream_t stream) {
  const long long joins = static_cast<long long>(a.B) * a.Hkv * ((a.G + JOIN_ROWS - 1) / JOIN_ROWS);  // (at most B * Hq)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(joins));
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, nsa_decode_join_kernel<D, Args>, a) == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace bsa
