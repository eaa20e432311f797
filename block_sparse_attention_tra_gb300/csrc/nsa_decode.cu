// nsa_decode.cu -- selection attention of one query token per sequence over a
// paged cache of e4m3 codes with a scale for each page and kv head.
//
// For sequence b of length n (its query is token n - 1), kv head h and the G
// query heads of its group, over the tokens t < n of the selected pages (or of
// every page):
//     s_t = (q . c^K_t) sigma^K_page D^-0.5,   out = sum_t softmax(s)_t sigma^V_page c^V_t,
//     lse = ln sum_t exp(s_t)          (no token: out 0, lse -1e9),
// c the codes' values, exact in f16, so no key or value is rounded on the way.
//
// Bound by the cache's bytes.  A warp takes slices of 16 tokens; its lanes
// load the slice's codes from global memory straight into the places that
// mma.sync.m16n8k16 wants them in, 16 bytes a lane and no shared memory:
//  - scores: D is summed over, so its order is free: lane (g, t) reads the
//    bytes of token row g that lie in its own share of the row, and the query
//    fragments are gathered in that order once.
//  - output: the columns' order is free: lane (g, t) reads, of the four tokens
//    whose probabilities it holds, the D/8 consecutive dims that are its
//    column g of the D/8 column tiles; two byte permutes pair two tokens.
// The next slice's loads are issued before this one's arithmetic.  The query
// rows (heads of the group, 16 with zero rows behind the last) go to f16 under
// a power-of-two factor of their own that brings their largest element near
// 2^14: exact for what is not 2^-28 of it.  Probabilities are rounded to f16
// (2^-12); each slice's product is taken on its own and added in fp32 under
// its page's scale.
//
// The work is the list of (sequence, kv head, page) in that order, cut into
// equal contiguous ranges, one a block, so that ragged lengths cost nothing.
// A block writes the (sequence, kv head) pairs that it covers whole; of the
// one it starts or ends in the middle of, it leaves (max, sum, accumulator) in
// the workspace, and a second kernel joins these in order.
#include <cuda_fp8.h>

#include "kernels.h"
#include "nsa_slots.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int SLICE = 16;   // tokens a warp takes at a time
constexpr int ROWS = 16;    // heads of a group, padded
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;
constexpr float LSE_EMPTY = -1.0e9f;

struct DecodeArgs {
  const __nv_bfloat16* q;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens, *block_idx;  // block_idx null: every page
  __nv_bfloat16* out;
  float* lse;
  float* ws;
  int B, Hq, Hkv, G, page, max_pages, num_pages, S;
  int ranges;  // blocks of the first kernel
  float scale_log2;
};

template <int D>
struct Dec {
  static constexpr int KC = D / 4 < 16 ? D / 4 : 16;  // bytes of one load of a key row
  static constexpr int KN = D / 4 / KC;               // such loads
  static constexpr int VC = D / 8;                    // bytes of one value load
  static constexpr int PART = ROWS * (D + 2);         // floats of one partial: m, l, acc
};

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
// The two e4m3 codes of the low (high) half of w as two f16 values.
__device__ __forceinline__ uint32_t f16_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// N bytes at p (aligned to min(N, 16)) as 32-bit words; N = 2 leaves the upper half zero.
template <int N>
struct Words {
  uint32_t w[(N + 3) / 4];
};
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 16) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
  } else if constexpr (N == 8) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p));
  } else if constexpr (N == 4) {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
  } else {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  return r;
}

// One slice's codes: two 8-token tiles of keys, four tokens of values.
template <int D>
struct Slice {
  Words<Dec<D>::KC> k[2][Dec<D>::KN];
  Words<Dec<D>::VC> v[4];
  float ks, vs;
  int tok0;  // first token; -1: no slice
};

// Where a range of the work list starts: sequence, kv head and page of its first unit.
struct Place {
  int b, h, page;
};

// Pages that sequence b reads.
__device__ __forceinline__ int pages_of(const DecodeArgs& a, int b) {
  if (a.block_idx != nullptr) return a.S;
  const int n = max(a.lens[b], 0);
  return min((n + a.page - 1) / a.page, a.max_pages);
}

// Units of the whole list, and the units before sequence `upto` (a block-wide
// call; scratch: WARPS + 2 long longs).
__device__ long long units_before(const DecodeArgs& a, int upto, long long* scratch) {
  if (a.block_idx != nullptr) return static_cast<long long>(upto) * a.Hkv * a.S;
  long long n = 0;
  for (int b = threadIdx.x; b < upto; b += THREADS) n += pages_of(a, b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < WARPS; ++w) n += scratch[w];
  return n * a.Hkv;
}

// The sequence that holds unit u (u < all units), and the units before it.
__device__ int sequence_of(const DecodeArgs& a, long long u, long long* scratch, long long* before) {
  if (a.block_idx != nullptr) {
    const long long per = static_cast<long long>(a.Hkv) * a.S;
    *before = u / per * per;
    return static_cast<int>(u / per);
  }
  const int per = (a.B + THREADS - 1) / THREADS;  // sequences of one thread
  const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  long long n = 0;
  for (int b = b0; b < b1; ++b) n += pages_of(a, b);
  n *= a.Hkv;
  long long sum = n;  // inclusive scan over the block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += x;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) sum += scratch[w];
  long long at = sum - n;
  if (u >= at && u < sum) {
    for (int b = b0; b < b1; ++b) {
      const long long m = static_cast<long long>(pages_of(a, b)) * a.Hkv;
      if (u < at + m) {
        scratch[WARPS] = at;
        scratch[WARPS + 1] = b;
        break;
      }
      at += m;
    }
  }
  __syncthreads();
  *before = scratch[WARPS];
  return static_cast<int>(scratch[WARPS + 1]);
}

__device__ __forceinline__ long long range_start(long long units, int c, int ranges) {
  return units / ranges * c + units % ranges * c / ranges;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 2) nsa_decode_kernel(const DecodeArgs a) {
  using L = Dec<D>;
  constexpr int NT = D / 8, KS = D / 16;
  constexpr int CST = D + 4;  // row stride of the merge area
  __shared__ float merge[WARPS][ROWS][CST];
  __shared__ float ml[WARPS][ROWS][2];
  __shared__ long long scratch[WARPS + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  const long long units = units_before(a, a.B, scratch);
  const long long u0 = range_start(units, blockIdx.x, a.ranges), u1 = range_start(units, blockIdx.x + 1, a.ranges);
  if (u0 >= u1) return;
  long long before;
  int b = sequence_of(a, u0, scratch, &before);
  int np = pages_of(a, b);
  int h = static_cast<int>((u0 - before) / np);
  int p0 = static_cast<int>((u0 - before) % np);

  for (long long u = u0; u < u1;) {
    const int p1 = static_cast<int>(min(static_cast<long long>(np), p0 + (u1 - u)));
    // ---- pages [p0, p1) of (b, h)
    const int len = min(a.lens[b], a.max_pages * a.page);
    const size_t qrow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G;

    // query fragments, in the order of the keys' bytes; each row under its own power of two
    uint32_t qa[KS][4];
    float f0, f1;  // score factors of rows g and g + 8
    {
      float x[2][D / 4];
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
#pragma unroll
        for (int c = 0; c < L::KN; ++c)
#pragma unroll
          for (int i = 0; i < L::KC; i += 4) {
            uint2 w = make_uint2(0u, 0u);
            if (row < a.G)
              w = *reinterpret_cast<const uint2*>(a.q + (qrow + row) * D + c * 4 * L::KC + t * L::KC + i);
            float* y = &x[r][c * L::KC + i];
            y[0] = __uint_as_float(w.x << 16);
            y[1] = __uint_as_float(w.x & 0xffff0000u);
            y[2] = __uint_as_float(w.y << 16);
            y[3] = __uint_as_float(w.y & 0xffff0000u);
#pragma unroll
            for (int e = 0; e < 4; ++e) m[r] = fmaxf(m[r], fabsf(y[e]));
          }
        m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 1));
        m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 2));
      }
      float up[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // 2^e with the row's maximum in [2^14, 2^15) (1 for zero rows and infinities)
        const int ex = static_cast<int>(__float_as_uint(m[r]) >> 23) - 127;
        const int e = ex >= -100 && ex < 128 ? 14 - ex : 0;
        up[r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        (r ? f1 : f0) = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qa[ks][0] = pack_f16x2(x[0][4 * ks] * up[0], x[0][4 * ks + 1] * up[0]);
        qa[ks][1] = pack_f16x2(x[1][4 * ks] * up[1], x[1][4 * ks + 1] * up[1]);
        qa[ks][2] = pack_f16x2(x[0][4 * ks + 2] * up[0], x[0][4 * ks + 3] * up[0]);
        qa[ks][3] = pack_f16x2(x[1][4 * ks + 2] * up[1], x[1][4 * ks + 3] * up[1]);
      }
    }

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;

    // The pages of up to 32 units at a time, one a lane: first token (or -1), pool page, scales.
    const int spp = a.page / SLICE;
    uint32_t live = 0u;
    SlotRow sel{0u, -1};
    if (a.block_idx != nullptr)
      sel = nsa_live_slots(a.block_idx + (static_cast<size_t>(b) * a.Hkv + h) * a.S, a.S, len - 1,
                           (len + a.page - 1) / a.page, a.page);
    int pb = p0 - 32;  // first unit of the pages held
    int my_tok = -1, my_id = 0;
    float my_ks = 0.0f, my_vs = 0.0f;
    auto hold_pages = [&](int base) {
      pb = base;
      const int y = base + lane;
      int lp = -1;
      if (a.block_idx != nullptr) {
        const int blk = __shfl_sync(0xffffffffu, sel.blk_lane, y & 31);
        if (y < p1 && ((sel.live >> (y & 31)) & 1u)) lp = blk;
      } else if (y < p1) {
        lp = y;
      }
      my_tok = -1;
      if (lp >= 0) {
        my_id = a.table[static_cast<size_t>(b) * a.max_pages + lp];
        if (my_id >= 0 && my_id < a.num_pages) {
          my_tok = lp * a.page;
          my_ks = a.k_scale[static_cast<size_t>(my_id) * a.Hkv + h];
          my_vs = a.v_scale[static_cast<size_t>(my_id) * a.Hkv + h];
        }
      }
      live = __ballot_sync(0xffffffffu, my_tok >= 0);
    };
    // The next slice of this warp at or behind slice x of the range; x moves behind it.
    const int nsl = (p1 - p0) * spp;
    int x = warp;
    auto next = [&](Slice<D>& s) {
      s.tok0 = -1;
      while (x < nsl) {
        const int y = p0 + x / spp, sub = x % spp;
        if (y >= pb + 32) hold_pages(y);
        x += WARPS;
        if (!((live >> (y - pb)) & 1u)) continue;
        const int tok0 = __shfl_sync(0xffffffffu, my_tok, y - pb) + sub * SLICE;
        if (tok0 >= len) continue;
        const int id = __shfl_sync(0xffffffffu, my_id, y - pb);
        s.tok0 = tok0;
        s.ks = __shfl_sync(0xffffffffu, my_ks, y - pb);
        s.vs = __shfl_sync(0xffffffffu, my_vs, y - pb);
        const size_t off = ((static_cast<size_t>(id) * a.Hkv + h) * a.page + sub * SLICE) * D;
        const uint8_t* kp = a.k + off + g * D + t * L::KC;
        const uint8_t* vp = a.v + off + 2 * t * D + g * L::VC;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < L::KN; ++c) s.k[j][c] = load_words<L::KC>(kp + j * 8 * D + c * 4 * L::KC);
#pragma unroll
        for (int j = 0; j < 4; ++j) s.v[j] = load_words<L::VC>(vp + ((j & 1) + (j >> 1) * 8) * D);
        return;
      }
    };

    Slice<D> cur, nxt;
    next(cur);
    while (cur.tok0 >= 0) {
      next(nxt);
      // ---- scores of 16 tokens, two 8-token tiles
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        constexpr int WPC = L::KC / 4;  // words per load
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t w = cur.k[j][ks / WPC].w[ks % WPC];
          mma_f16(sc[j], qa[ks], f16_lo(w), f16_hi(w));
        }
      }
      const float e0 = f0 * cur.ks, e1 = f1 * cur.ks;
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = cur.tok0 + 8 * j + 2 * t + e < len;
          sc[j][e] = in ? sc[j][e] * e0 : -INFINITY;
          sc[j][2 + e] = in ? sc[j][2 + e] * e1 : -INFINITY;
          mx0 = fmaxf(mx0, sc[j][e]);
          mx1 = fmaxf(mx1, sc[j][2 + e]);
        }
      if (cur.tok0 + SLICE > len) {  // codes behind the last token may be anything
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (cur.tok0 + (j & 1) + (j >> 1) * 8 + 2 * t >= len)
#pragma unroll
            for (int i = 0; i < (L::VC + 3) / 4; ++i) cur.v[j].w[i] = 0u;
      }
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      // lazy rescale: the running maximum moves only when a score exceeds it by 8 (a probability by 2^8)
      if (__any_sync(0xffffffffu, mx0 > m0 + 8.0f || mx1 > m1 + 8.0f)) {
        const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
        // (a row of -inf scores so far keeps zero sums: exp2(-inf - -inf) is not taken)
        const float s0 = n0 == -INFINITY ? 1.0f : ex2f(m0 - n0), s1 = n1 == -INFINITY ? 1.0f : ex2f(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= s0;
        l1 *= s1;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][0] *= s0;
          acc[j][1] *= s0;
          acc[j][2] *= s1;
          acc[j][3] *= s1;
        }
      }
      const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
      uint32_t pa[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float y0 = ex2f(sc[j][0] - b0), y1 = ex2f(sc[j][1] - b0);
        const float y2 = ex2f(sc[j][2] - b1), y3 = ex2f(sc[j][3] - b1);
        l0 += y0 + y1;
        l1 += y2 + y3;
        pa[2 * j] = pack_f16x2(y0, y1);
        pa[2 * j + 1] = pack_f16x2(y2, y3);
      }
      // ---- acc += sigma^V (P V)
#pragma unroll
      for (int i = 0; i < NT; i += 2) {  // column tiles i and i + 1: bytes i, i + 1 of each token's run
        const int w = i / 4;
        const uint32_t pick = (i & 2) ? 0x7362u : 0x5140u;
        const uint32_t x01 = __byte_perm(cur.v[0].w[w], cur.v[1].w[w], pick);
        const uint32_t x23 = __byte_perm(cur.v[2].w[w], cur.v[3].w[w], pick);
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(d0, pa, f16_lo(x01), f16_lo(x23));
        mma_f16(d1, pa, f16_hi(x01), f16_hi(x23));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[i][e] = fmaf(cur.vs, d0[e], acc[i][e]);
          acc[i + 1][e] = fmaf(cur.vs, d1[e], acc[i + 1][e]);
        }
      }
      cur = nxt;
    }

    // ---- the warps' states into one
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
    for (int c = 0; c < 2; ++c)  // column 2t + c of every tile: dims (2t + c) D/8 + j
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        merge[warp][g][(2 * t + c) * NT + j] = acc[j][c];
        merge[warp][g + 8][(2 * t + c) * NT + j] = acc[j][2 + c];
      }
    if (t == 0) {
      ml[warp][g][0] = m0;
      ml[warp][g][1] = l0;
      ml[warp][g + 8][0] = m1;
      ml[warp][g + 8][1] = l1;
    }
    __syncthreads();
    {
      const bool whole = p0 == 0 && p1 == np;
      constexpr int PER = D / 8;  // dims of one thread
      const int row = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * PER;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w][row][0]);
      const float mb = M == -INFINITY ? 0.0f : M;
      float sum = 0.0f, wt[WARPS];
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        wt[w] = ex2f(ml[w][row][0] - mb);
        sum += wt[w] * ml[w][row][1];
      }
      if (row < a.G) {
        float* part = a.ws + (2 * static_cast<size_t>(blockIdx.x) + (u != u0 ? 1 : 0)) * L::PART + row * (D + 2);
        const float inv = whole ? (sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum) : 1.0f;
        __nv_bfloat16* o = a.out + (qrow + row) * D + d0;
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
          float y0 = 0.f, y1 = 0.f;
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            y0 += wt[w] * merge[w][row][d0 + e];
            y1 += wt[w] * merge[w][row][d0 + e + 1];
          }
          if (whole) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(y0 * inv, y1 * inv);
          else *reinterpret_cast<float2*>(part + 2 + d0 + e) = make_float2(y0, y1);
        }
        if ((threadIdx.x & 7) == 0) {
          if (!whole) *reinterpret_cast<float2*>(part) = make_float2(M, sum);
          else if (a.lse != nullptr) a.lse[qrow + row] = sum == 0.0f ? LSE_EMPTY : (M + __log2f(sum)) * LN2;
        }
      }
    }
    __syncthreads();
    // ---- on to the next (sequence, head)
    u += p1 - p0;
    p0 = 0;
    if (u < u1 && ++h == a.Hkv) {
      h = 0;
      do np = pages_of(a, ++b);
      while (np == 0);
    }
  }
}

// One block per (sequence, kv head): joins the parts of one that several
// ranges cover, and answers for a sequence without tokens.
template <int D>
__global__ void __launch_bounds__(THREADS) nsa_decode_join_kernel(const DecodeArgs a) {
  using L = Dec<D>;
  __shared__ long long scratch[WARPS + 2];
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int np = pages_of(a, b);
  const int row = threadIdx.x >> 3;
  constexpr int PER = D / 8;
  const int d0 = (threadIdx.x & 7) * PER;
  const size_t qrow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G + row;
  float M = -INFINITY, sum = 0.0f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.0f;
  if (np > 0) {
    const long long units = units_before(a, a.B, scratch);
    const long long u0 = units_before(a, b, scratch) + static_cast<long long>(h) * np, u1 = u0 + np;
    auto range_of = [&](long long u) {  // the range that holds unit u
      int lo = 0, hi = a.ranges - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (range_start(units, mid, a.ranges) <= u) lo = mid;
        else hi = mid - 1;
      }
      return lo;
    };
    const int c0 = range_of(u0), c1 = range_of(u1 - 1);
    if (c0 == c1) return;  // written by its only range
    if (row < a.G) {
      for (int c = c0; c <= c1; ++c) {
        const long long start = range_start(units, c, a.ranges);
        if (start == range_start(units, c + 1, a.ranges)) continue;  // an empty range
        const float* part = a.ws + (2 * static_cast<size_t>(c) + (start < u0 ? 1 : 0)) * L::PART + row * (D + 2);
        const float2 pml = *reinterpret_cast<const float2*>(part);
        const float n = fmaxf(M, pml.x), nb = n == -INFINITY ? 0.0f : n;
        const float s = ex2f(M - nb), w = ex2f(pml.x - nb);
        M = n;
        sum = sum * s + pml.y * w;
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(part + 2 + d0 + e);
          o[e] = o[e] * s + y.x * w;
          o[e + 1] = o[e + 1] * s + y.y * w;
        }
      }
    }
  }
  if (row >= a.G) return;
  const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + qrow * D + d0 + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (a.lse != nullptr && (threadIdx.x & 7) == 0) a.lse[qrow] = sum == 0.0f ? LSE_EMPTY : (M + __log2f(sum)) * LN2;
}

// Ranges of the work list: two blocks on each SM, or one for each page of a short list.
int decode_ranges(int B, int Hkv, int max_pages, int S) {
  const long long units = static_cast<long long>(B) * Hkv * (S > 0 ? S : max_pages);
  long long most = 2LL * sm_count();
  most = most < 1 ? 1 : most > DECODE_MAX_RANGES ? DECODE_MAX_RANGES : most;
  return static_cast<int>(units < most ? units : most);
}

template <int D>
int launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.B) * a.Hkv;
  nsa_decode_kernel<D><<<static_cast<unsigned>(a.ranges), THREADS, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  nsa_decode_join_kernel<D><<<static_cast<unsigned>(items), THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace

// The partials of the most ranges (the size does not depend on the device).
size_t nsa_decode_workspace_bytes(int D) {
  return 2 * static_cast<size_t>(DECODE_MAX_RANGES) * ROWS * (static_cast<size_t>(D) + 2) * sizeof(float);
}

int launch_nsa_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, const int32_t* table, const int32_t* lens, const int32_t* block_idx,
                      void* out, float* lse, int B, int Hq, int Hkv, int D, int page, int max_pages, int num_pages,
                      int S, void* workspace, cudaStream_t stream) {
  DecodeArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const uint8_t*>(k_cache);
  a.v = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.table = table; a.lens = lens; a.block_idx = block_idx;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws = static_cast<float*>(workspace);
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.page = page;
  a.max_pages = max_pages; a.num_pages = num_pages; a.S = block_idx != nullptr ? S : 0;
  a.ranges = decode_ranges(B, Hkv, max_pages, a.S);
  a.scale_log2 = LOG2E / sqrtf(static_cast<float>(D));
  switch (D) {
    case 16: return launch_decode<16>(a, stream);
    case 32: return launch_decode<32>(a, stream);
    case 64: return launch_decode<64>(a, stream);
    case 128: return launch_decode<128>(a, stream);
    default: return ERR_UNSUPPORTED;
  }
}

}  // namespace bsa
