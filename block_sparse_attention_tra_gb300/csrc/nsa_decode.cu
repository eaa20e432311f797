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
// The arithmetic, per warp and 16 or 32 tokens, by mma.sync.m16n8k16 (16 query
// rows fill one M tile; a tcgen05 tile would be 7/8 padding):
//  - scores: D is summed over, so its order is free: lane (g, t) takes the
//    bytes of token row g that lie in its own share of the row, and the query
//    fragments are gathered in that order once.
//  - output: the columns' order is free: lane (g, t) takes, of the tokens
//    whose probabilities it holds, the D/8 consecutive dims that are its
//    column g of the D/8 column tiles; two byte permutes pair two tokens.
// The query rows (heads of the group, 16 with zero rows behind the last) go to
// f16 under a power-of-two factor of their own that brings their largest
// element near 2^14: exact for what is not 2^-28 of it.  Probabilities are
// rounded to f16: their products with the codes then are exact in the tensor
// cores.  They are taken over 2^-11 to 2^-15 of the largest score's
// exponential so far, which puts the largest at the top of the f16 range: a
// token whose probability is 2^-25 of it still has 2^-11 of precision, an
// eighth of the final bf16 rounding, and what is smaller is off by at most
// 2^-36 of it.  (With the largest at 1 that border lay at 2^-14: a first token
// of nearly all the weight and hardly a value, and tens of thousands of others
// that make up the result, lost whole bits of it.)
//
// Two kernels.
//
// Selected pages: one block a (sequence, kv head) pair, or with few pairs a
// cluster of 2, 4 or 8 that shares out its slots and joins the blocks' (max,
// sum, accumulator) through distributed shared memory: one launch.  A warp
// takes chunks of 32 tokens of a page (16 where pages hold 16); its lanes
// bring the chunk's codes by cp.async into their own places of a ring in
// shared memory -- each lane copies what it will read itself, so the ring
// needs no barrier and has no bank conflicts.  One sequence, 16 pages of 64
// tokens, 32 query and 2 kv heads of 128: 6.5 us, the latency of a chain of
// loads (slots, table, codes).  128 sequences of 64 query and 4 kv heads: 134
// MB in 39.5 us (3.4 TB/s); what keeps it from the cache's bytes is that chain
// at the start of each block and the second, two thirds full wave of 512
// blocks.  (Cutting the pairs into equal ranges for the kernel below took 46.6
// us, and up to two and a half times as long on smaller heads, as it joins
// warps and blocks once a pair.)
//
// Every page: persistent blocks, a producer warp that brings stages of 128
// tokens by TMA and eight consumer warps with 16 tokens of a stage each.  The
// list of (sequence, kv head, stage) in that order is cut into equal
// contiguous ranges, one a block, so that ragged lengths cost nothing; a block
// writes the pairs that it covers whole, and of the ones it starts or ends in
// the middle of leaves (max, sum, accumulator) in the workspace, which a
// second kernel joins in order.  Bound by the cache's bytes on paper: four
// sequences of up to 131072 tokens are 155 MB, 42.5 us (3.6 TB/s; the first
// kernel alone 39).  What holds it there is the consumers' latency: a slice
// of 16 tokens is 1450 cycles of load, product, maximum, exponential, product,
// and the registers of eight warps (168 each) leave two a scheduler to hide it
// (issue slots 31% busy).  Slices of 32 tokens on two teams of warps, and score
// sums split over two accumulators, were no faster.
#include <cooperative_groups.h>

#include "kernels.h"
#include "nsa_slots.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int STAGE_LOG = 7, STAGE_TOK = 1 << STAGE_LOG;  // tokens of a stage (stream kernel)
constexpr int ROWS = 16;    // heads of a group, padded
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;
constexpr float LSE_EMPTY = -1.0e9f;
// Exponents (log2 domain) are taken against a reference that is set P_SET below the largest score so far when one
// exceeds it by P_MAX: probabilities stay below 2^15 (an f16 ends at 65504).  Sums and accumulators leave a warp in
// units of 2^P_SET.
constexpr float P_SET = 11.0f, P_MAX = 15.0f, P_UNIT = 1.0f / 2048.0f;

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

template <int D, int C>
struct Dec {
  // Blocks of a SM, and the tokens that a warp's ring holds.  D = 128: the accumulators (64 registers), query fragments
  // (32) and scores leave two blocks, three chunks of 32 tokens a warp; at D = 64 four blocks of two chunks take 27.8
  // us where three of three take 32.2 (256 sequences, 4 kv heads, 16 pages of 64, codes in L2).
  static constexpr int CTAS = D == 128 ? 2 : 4;
  static constexpr int RING = (D == 128 ? 96 : 64) / C;  // chunks of a warp in flight or in use
  static constexpr int KC = D / 4 < 16 ? D / 4 : 16;  // bytes of one piece of a key row
  static constexpr int KN = D / 4 / KC;               // such pieces of a lane
  static constexpr int VB = D / 8;                    // bytes of a lane's run of a value row
  static constexpr int VC = VB < 4 ? 4 : VB;          // copied for it (D = 16: the aligned word around its two)
  static constexpr int KT = 32 * KN * KC;             // ring bytes of an 8-token tile of keys
  static constexpr int SLOT = C / 8 * KT + C / 4 * 32 * VC;  // one chunk of one warp
  static constexpr int CST = D + 8;                   // row stride of the merge area
  // the ring, and over it (a range's chunks are done with then) the merge area
  static constexpr int MERGE = WARPS * ROWS * CST * 4;
  static constexpr int BYTES = WARPS * RING * SLOT > MERGE ? WARPS * RING * SLOT : MERGE;
};

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
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A chunk on its way: first token (-1: none) and slot.
struct Chunk {
  int tok0, slot;
};

// Floats of one partial: (m, l) of each row, then the accumulator rows.
__host__ __device__ constexpr int part_floats(int D) { return ROWS * (D + 2); }

// Tokens that sequence b holds (at most max_pages * page <= 2^31 - 16: what lies behind the last of them is counted in
// unsigned numbers), and the pages and stages of 128 that they make.
__device__ __forceinline__ int tokens_of(const DecodeArgs& a, int b) {
  return max(0, min(a.lens[b], a.max_pages * a.page));
}
__device__ __forceinline__ int pieces_of(int tokens, int size_log) {
  return static_cast<int>((static_cast<uint32_t>(tokens) + (1u << size_log) - 1u) >> size_log);
}
__device__ __forceinline__ int stages_of(const DecodeArgs& a, int b) {
  return pieces_of(tokens_of(a, b), STAGE_LOG);
}

// The units (a stage of one kv head) before sequence `upto`; a block-wide call,
// scratch: a long long for each warp.
__device__ long long units_before(const DecodeArgs& a, int upto, long long* scratch) {
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
__device__ int sequence_of(const DecodeArgs& a, long long u, long long* before) {
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
__device__ long long units_of_warp(const DecodeArgs& a) {
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

// Slots [p0, p1) of (b, h)'s selection: the block's 128 threads leave the range's unnormalised
// accumulator, weighted into one, in y (row threadIdx.x / 8, dims (threadIdx.x
// % 8) D/8 ..), its maximum (log2 domain) in M and its sum of exponentials in sum.
template <int D, int C>
__device__ __forceinline__ void decode_range(const DecodeArgs& a, int b, int h, int p0, int p1, uint8_t* smem,
                                             float (*ml)[ROWS][2], float (&y)[D / 8], float& M, float& sum) {
  using L = Dec<D, C>;
  constexpr int NT = D / 8, KS = D / 16, RING = L::RING, SL = C / 16;  // SL: k-steps of P V
  float(*merge)[ROWS][L::CST] = reinterpret_cast<float(*)[ROWS][L::CST]>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * RING * L::SLOT;
  const int len = tokens_of(a, b);
  const size_t qrow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G;

  // The slots' pages, one a lane: first token (or -1), pool page, scales.
  const int cpp_log = 31 - __clz(a.page / C);  // chunks of a page (a power of two)
  int my_tok = -1, my_id = 0;
  float my_ks = 0.0f, my_vs = 0.0f;
  {
    const SlotRow sel = nsa_live_slots(a.block_idx + (static_cast<size_t>(b) * a.Hkv + h) * a.S, a.S, len - 1,
                                       pieces_of(len, 31 - __clz(a.page)), a.page);
    if (lane >= p0 && lane < p1 && ((sel.live >> lane) & 1u)) {
      my_id = a.table[static_cast<size_t>(b) * a.max_pages + sel.blk_lane];
      if (my_id >= 0 && my_id < a.num_pages) {
        my_tok = sel.blk_lane * a.page;
        my_ks = a.k_scale[static_cast<size_t>(my_id) * a.Hkv + h];
        my_vs = a.v_scale[static_cast<size_t>(my_id) * a.Hkv + h];
      }
    }
  }
  const uint32_t live = __ballot_sync(0xffffffffu, my_tok >= 0);
  // This warp's next chunk of the range into a place of the ring.
  const int n_chunks = (p1 - p0) << cpp_log;
  int x = warp;
  auto fetch = [&](int place) -> Chunk {
    Chunk s{-1, 0};
    while (x < n_chunks) {
      const int u = p0 + (x >> cpp_log), sub = x & ((1 << cpp_log) - 1);
      x += WARPS;
      if (!((live >> u) & 1u)) continue;
      const int tok0 = __shfl_sync(0xffffffffu, my_tok, u) + sub * C;
      if (tok0 >= len) continue;
      const int id = __shfl_sync(0xffffffffu, my_id, u);
      s.tok0 = tok0;
      s.slot = u;
      const size_t off = ((static_cast<size_t>(id) * a.Hkv + h) * a.page + sub * C) * D;
      const uint8_t* kp = a.k + off + g * D + t * L::KC;
      const uint8_t* vp = a.v + off + 2 * t * D + (g * L::VB & ~3);
      uint32_t dst = ring + place * L::SLOT;
#pragma unroll
      for (int j = 0; j < C / 8; ++j)
#pragma unroll
        for (int c = 0; c < L::KN; ++c, dst += 32 * L::KC)
          copy_async<L::KC>(dst + lane * L::KC, kp + j * 8 * D + c * 4 * L::KC);
#pragma unroll
      for (int j = 0; j < C / 4; ++j, dst += 32 * L::VC)  // tokens 8 (j / 2) + 2t + j % 2
        copy_async<L::VC>(dst + lane * L::VC, vp + ((j & 1) + (j >> 1) * 8) * D);
      break;
    }
    copy_commit();
    return s;
  };
  Chunk ahead[RING - 1];  // those on their way, the next first
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) ahead[i] = fetch(i);

  // query fragments, in the order of the keys' bytes; each row under its own power of two
  uint32_t qa[KS][4];
  float f0, f1;  // score factors of rows g and g + 8
  {
    uint2 w[2][KS];
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int i = 4 * ks;  // of this lane's D / 4 elements
        w[r][ks] = make_uint2(0u, 0u);
        if (row < a.G)
          w[r][ks] = *reinterpret_cast<const uint2*>(a.q + (qrow + row) * D + i / L::KC * 4 * L::KC + t * L::KC +
                                                     i % L::KC);
        m[r] = fmaxf(m[r], fmaxf(fmaxf(fabsf(__uint_as_float(w[r][ks].x << 16)),
                                       fabsf(__uint_as_float(w[r][ks].x & 0xffff0000u))),
                                 fmaxf(fabsf(__uint_as_float(w[r][ks].y << 16)),
                                       fabsf(__uint_as_float(w[r][ks].y & 0xffff0000u)))));
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
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        qa[ks][r] = pack_f16x2(__uint_as_float(w[r][ks].x << 16) * up[r],
                               __uint_as_float(w[r][ks].x & 0xffff0000u) * up[r]);
        qa[ks][2 + r] = pack_f16x2(__uint_as_float(w[r][ks].y << 16) * up[r],
                                   __uint_as_float(w[r][ks].y & 0xffff0000u) * up[r]);
      }
  }

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;

  int place = 0;
  while (ahead[0].tok0 >= 0) {
    const Chunk cur = ahead[0];
#pragma unroll
    for (int i = 0; i < RING - 2; ++i) ahead[i] = ahead[i + 1];
    ahead[RING - 2] = fetch(place == 0 ? RING - 1 : place - 1);  // into the place freed last
    copy_wait<RING - 1>();
    const uint32_t src = ring + place * L::SLOT;
    place = place == RING - 1 ? 0 : place + 1;
    // ---- scores, 16 tokens at a time (two 8-token tiles: two chains of products)
    float sc[C / 8][4];
#pragma unroll
    for (int jj = 0; jj < C / 8; jj += 2) {
      constexpr int WPC = L::KC / 4;  // words of a piece
      Words<L::KC> kw[2][L::KN];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int c = 0; c < L::KN; ++c)
          kw[j][c] = load_shared<L::KC>(src + (jj + j) * L::KT + c * 32 * L::KC + lane * L::KC);
        sc[jj + j][0] = sc[jj + j][1] = sc[jj + j][2] = sc[jj + j][3] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t w = kw[j][k / WPC].w[k % WPC];
          mma_f16(sc[jj + j], qa[k], f16_lo(w), f16_hi(w));
        }
    }
    const float ks = __shfl_sync(0xffffffffu, my_ks, cur.slot);
    const float vs = __shfl_sync(0xffffffffu, my_vs, cur.slot) * P_UNIT;
    const float e0 = f0 * ks, e1 = f1 * ks;
    const bool tail = cur.tok0 + C > len;
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < C / 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in = !tail || cur.tok0 + 8 * j + 2 * t + e < len;
        sc[j][e] = in ? sc[j][e] * e0 : -INFINITY;
        sc[j][2 + e] = in ? sc[j][2 + e] * e1 : -INFINITY;
        mx0 = fmaxf(mx0, sc[j][e]);
        mx1 = fmaxf(mx1, sc[j][2 + e]);
      }
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    // lazy rescale: the reference moves only when a probability would exceed 2^15
    if (__any_sync(0xffffffffu, mx0 - m0 > P_MAX || mx1 - m1 > P_MAX)) {
      const float n0 = fmaxf(m0, reference_of(mx0)), n1 = fmaxf(m1, reference_of(mx1));
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
    uint32_t pa[SL][4];
#pragma unroll
    for (int j = 0; j < C / 8; ++j) {
      const float y0 = ex2f(sc[j][0] - b0), y1 = ex2f(sc[j][1] - b0);
      const float y2 = ex2f(sc[j][2] - b1), y3 = ex2f(sc[j][3] - b1);
      l0 += y0 + y1;
      l1 += y2 + y3;
      pa[j >> 1][2 * (j & 1)] = pack_f16x2(y0, y1);
      pa[j >> 1][2 * (j & 1) + 1] = pack_f16x2(y2, y3);
    }
    // ---- acc += sigma^V (P V)
    Words<L::VC> vw[C / 4];
#pragma unroll
    for (int j = 0; j < C / 4; ++j) {
      vw[j] = load_shared<L::VC>(src + C / 8 * L::KT + (j * 32 + lane) * L::VC);
      if constexpr (L::VB < L::VC) vw[j].w[0] >>= (g & 1) * 16;
    }
    if (tail) {  // codes behind the last token may be anything
#pragma unroll
      for (int j = 0; j < C / 4; ++j)
        if (cur.tok0 + (j & 1) + (j >> 1) * 8 + 2 * t >= len)
#pragma unroll
          for (int i = 0; i < L::VC / 4; ++i) vw[j].w[i] = 0u;
    }
#pragma unroll
    for (int i = 0; i < NT; i += 2) {  // column tiles i and i + 1: bytes i, i + 1 of each token's run
      const int w = i / 4;
      const uint32_t pick = (i & 2) ? 0x7362u : 0x5140u;
      float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        const uint32_t x01 = __byte_perm(vw[4 * k].w[w], vw[4 * k + 1].w[w], pick);
        const uint32_t x23 = __byte_perm(vw[4 * k + 2].w[w], vw[4 * k + 3].w[w], pick);
        mma_f16(d0, pa[k], f16_lo(x01), f16_lo(x23));
        mma_f16(d1, pa[k], f16_hi(x01), f16_hi(x23));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[i][e] = fmaf(vs, d0[e], acc[i][e]);
        acc[i + 1][e] = fmaf(vs, d1[e], acc[i + 1][e]);
      }
    }
  }
  copy_wait<0>();

  // ---- the warps' states into one (over the ring: every warp is done with its chunks)
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  __syncthreads();
  // column n = 2t, 2t + 1 of tile j, which is dim n D/8 + j, at place 8 j + n: no bank conflicts here or below
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    *reinterpret_cast<float2*>(&merge[warp][g][8 * j + 2 * t]) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(&merge[warp][g + 8][8 * j + 2 * t]) = make_float2(acc[j][2], acc[j][3]);
  }
  if (t == 0) {
    ml[warp][g][0] = m0;
    ml[warp][g][1] = l0 * P_UNIT;
    ml[warp][g + 8][0] = m1;
    ml[warp][g + 8][1] = l1 * P_UNIT;
  }
  __syncthreads();
  const int row = threadIdx.x >> 3;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w][row][0]);
  const float mb = M == -INFINITY ? 0.0f : M;
  sum = 0.0f;
  float wt[WARPS];
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    wt[w] = ex2f(ml[w][row][0] - mb);
    sum += wt[w] * ml[w][row][1];
  }
#pragma unroll
  for (int e = 0; e < NT; ++e) {
    y[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) y[e] += wt[w] * merge[w][row][8 * e + (threadIdx.x & 7)];
  }
}

// 1 / sum for a row with tokens, 0 for one without (NaN stays).
__device__ __forceinline__ float inverse_sum(float sum) { return sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum; }
__device__ __forceinline__ float lse_of(float M, float sum) {
  return sum == 0.0f ? LSE_EMPTY : (M + (P_SET + __log2f(sum))) * LN2;
}

// ------------------------------------------------------------ stream kernel

constexpr int CONSUMERS = STAGE_TOK / 16;  // consumer warps, one for each slice of 16 tokens
constexpr int STREAM_THREADS = (CONSUMERS + 1) * 32;
enum : int { SEG_FIRST = 1, SEG_LAST = 2, SEG_WHOLE = 4, SEG_END = 8 };

// What the producer says of a stage: its slices of 16 tokens (first token, or
// -1, and scales); and of a segment, a run of stages of one (sequence, kv head).
struct StageHead {
  int4 slice[CONSUMERS];  // tok0, key scale, value scale
  int flags, pad[3];
};
struct SegmentHead {
  int b, h, len, part;
};

template <int D>
struct StreamLayout {
  static constexpr int KV = STAGE_TOK * D;  // bytes of a stage's keys (values)
  static constexpr int NS = D == 128 ? 4 : 6;
  static constexpr int CST = D + 8;
  static constexpr int Q_BYTES = 32 * (D / 16) * 16 + ROWS * 4;  // fragments, then the rows' score factors
  static constexpr int MERGE_OFF = NS * 2 * KV;  // float[CONSUMERS][ROWS][CST]
  static constexpr int ML_OFF = MERGE_OFF + CONSUMERS * ROWS * CST * 4;
  static constexpr int Q_OFF = ML_OFF + CONSUMERS * ROWS * 8;  // two segments' queries
  static constexpr int HEAD_OFF = Q_OFF + 2 * Q_BYTES;
  static constexpr int SEG_OFF = HEAD_OFF + NS * static_cast<int>(sizeof(StageHead));
  static constexpr int WIN_OFF = SEG_OFF + 2 * static_cast<int>(sizeof(SegmentHead));  // int4[32]
  static constexpr int BAR_OFF = WIN_OFF + 32 * 16;
  // full[NS] | empty[NS] | q_empty[2] | merge[2]
  static constexpr int BYTES = BAR_OFF + (2 * NS + 4) * 8 + 1024;
  static_assert(BYTES <= 232448, "shared memory");
};

// Byte `off` of a tile of 128-byte lines that TMA wrote with 128-byte swizzle (1024-byte aligned).
__device__ __forceinline__ uint32_t swz128(uint32_t off) { return off ^ ((off >> 3) & 0x70u); }

// Persistent blocks, each on one contiguous range of the (sequence, kv head, stage) list; stage k holds tokens 128 k ..
// of the sequence.
template <int D>
__global__ void __launch_bounds__(STREAM_THREADS, 1)
    nsa_decode_stream_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const DecodeArgs a) {
  using L = StreamLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t *empty = full + L::NS, *q_empty = empty + L::NS, *merge_bar = q_empty + 2;
  StageHead* heads = reinterpret_cast<StageHead*>(smem + L::HEAD_OFF);
  SegmentHead* segs = reinterpret_cast<SegmentHead*>(smem + L::SEG_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the joining kernel's blocks may take the places that this one's leave (they wait for all of it)
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    for (int x = 0; x < L::NS; ++x) {
      mbar_init(&full[x], 1);
      mbar_init(&empty[x], CONSUMERS);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_empty[x], CONSUMERS);
      mbar_init(&merge_bar[x], CONSUMERS);
    }
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == CONSUMERS) {
    // -------------------------------------------------------------- producer
    // The warp resolves pages 32 at a time into a window in shared memory {pool page or -1, first token, scales};
    // BATCH lanes then put up a stage each, in step (one stage after another, by the whole warp or by one lane, a
    // stage took 1200 cycles, and that held the copies at 4 TB/s).
    constexpr int BATCH = 2;
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    int4* win = reinterpret_cast<int4*>(smem + L::WIN_OFF);
    const int page_log = 31 - __clz(a.page);
    const uint32_t page_bytes = static_cast<uint32_t>(D * a.page);
    int it = 0, seg = 0;
    bool ok = true;
    // stage number `at` of this block's, whose first token is number `pos` of the window's pages, `n` of them in use
    auto put = [&](const SegmentHead& sg, int flags, int at, int pos, int n) {
      const int st = at % L::NS;
      if (!(ok = mbar_wait(&empty[st], ((at / L::NS) & 1) ^ 1))) return;
      StageHead* hd = &heads[st];
      uint8_t* dst = smem + st * 2 * L::KV;
      // the stage's whole pages, and (pages of a stage's size) no others: a page's box where it has a token
      uint32_t bytes = 0u, live = 0u;
#pragma unroll
      for (int k = 0; k < CONSUMERS; ++k) {
        const int e = (pos + 16 * k) >> page_log, in = (pos + 16 * k) & (a.page - 1);
        const int4 w = e < n ? win[e] : make_int4(-1, 0, 0, 0);
        const bool some = w.x >= 0 && w.y + in < sg.len;
        hd->slice[k] = make_int4(some ? w.y + in : -1, w.z, w.w, 0);
        if (some && in == 0) {
          bytes += 2 * page_bytes;
          live |= 1u << k;
        }
      }
      hd->flags = flags;
      if (bytes != 0u) mbar_arrive_expect_tx(&full[st], bytes);
      else mbar_arrive(&full[st]);
      for (; live != 0u; live &= live - 1u) {
        const int k = __ffs(live) - 1, head = win[(pos + 16 * k) >> page_log].x * a.Hkv + sg.h;
        tma_load_3d(dst + 16 * k * D, &tmK, &full[st], 0, 0, head);
        tma_load_3d(dst + L::KV + 16 * k * D, &tmV, &full[st], 0, 0, head);
      }
    };
    // stages [s, end) of a segment that has [s0, s1); stage x begins with token x * STAGE_TOK - origin of the window
    auto put_all = [&](const SegmentHead& sg, int whole, int s0, int s1, int s, int end, int origin, int n) {
      for (; s < end && ok; s += BATCH) {
        const int x = s + lane;
        if (lane < BATCH && x < end)
          put(sg, whole | (x == s0 ? SEG_FIRST : 0) | (x == s1 - 1 ? SEG_LAST : 0), it + lane, x * STAGE_TOK - origin,
              n);
        ok = __all_sync(0xffffffffu, ok);
        it += min(BATCH, end - s);
      }
      if (end == s1) ++seg;
    };
    // The whole warp: a segment's head and its query fragments, for lane (g, t) rows g and g + 8, dims t D/4 + 4k ..
    // of k-step k, each row under its own power of two (rows G .. 15 zero).  The rows are loaded a segment ahead.
    constexpr int KS = D / 16;
    struct QRows {
      uint2 w[2][KS];
    };
    auto load_q = [&](int b, int h) {
      QRows q;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          q.w[r][k] = make_uint2(0u, 0u);
          const int row = (lane >> 2) + 8 * r;
          if (row < a.G)
            q.w[r][k] = *reinterpret_cast<const uint2*>(
                a.q + (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G + row) * D + (lane & 3) * (D / 4) +
                4 * k);
        }
      return q;
    };
    auto open_segment = [&](const SegmentHead& sg, const QRows& q) {
      ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[seg & 1], ((seg >> 1) & 1) ^ 1));
      if (!ok) return;
      uint8_t* dst = smem + L::Q_OFF + (seg & 1) * L::Q_BYTES;
      float up[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
          m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(q.w[r][k].x << 16)),
                                   fabsf(__uint_as_float(q.w[r][k].x & 0xffff0000u))),
                             fmaxf(fabsf(__uint_as_float(q.w[r][k].y << 16)),
                                   fabsf(__uint_as_float(q.w[r][k].y & 0xffff0000u)))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^e with the row's maximum in [2^14, 2^15) (1 for zero rows and infinities)
        const int ex = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        const int e = ex >= -100 && ex < 128 ? 14 - ex : 0;
        up[r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        if ((lane & 3) == 0)
          reinterpret_cast<float*>(dst + 32 * KS * 16)[(lane >> 2) + 8 * r] =
              a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      }
      auto two = [](uint32_t w, float u) {
        return pack_f16x2(__uint_as_float(w << 16) * u, __uint_as_float(w & 0xffff0000u) * u);
      };
#pragma unroll
      for (int k = 0; k < KS; ++k)
        reinterpret_cast<uint4*>(dst)[32 * k + lane] = make_uint4(two(q.w[0][k].x, up[0]), two(q.w[1][k].x, up[1]),
                                                                  two(q.w[0][k].y, up[0]), two(q.w[1][k].y, up[1]));
      if (lane == 0) segs[seg & 1] = sg;
      __syncwarp();
    };
    // the whole warp: lane l's page into the window
    auto open_window = [&](int id, int tok, float ks, float vs) {
      __syncwarp();  // the lanes that put stages up are done with the last one
      win[lane] = make_int4(id, tok, __float_as_int(ks), __float_as_int(vs));
      __syncwarp();
    };
    struct Page {
      int id;
      float ks, vs;
    };
    auto scales_of = [&](int id, int h) -> Page {
      if (id < 0 || id >= a.num_pages) return {-1, 0.0f, 0.0f};
      const size_t at = static_cast<size_t>(id) * a.Hkv + h;
      return {id, a.k_scale[at], a.v_scale[at]};
    };

    const long long units = units_of_warp(a);
    const long long u0 = range_start(units, blockIdx.x, a.ranges), u1 = range_start(units, blockIdx.x + 1, a.ranges);
    if (u0 < u1) {
      long long before;
      int b = sequence_of(a, u0, &before);
      int n_st = stages_of(a, b);
      int h = static_cast<int>((u0 - before) / n_st), s0 = static_cast<int>((u0 - before) % n_st);
      QRows q = load_q(b, h);
      for (long long u = u0; u < u1 && ok;) {
        const int s1 = static_cast<int>(min(static_cast<long long>(n_st), s0 + (u1 - u)));
        const int len = tokens_of(a, b), n_pages = pieces_of(len, page_log);
        const int whole = s0 == 0 && s1 == n_st ? SEG_WHOLE : 0;
        const SegmentHead sg{b, h, len, 2 * static_cast<int>(blockIdx.x) + (u != u0 ? 1 : 0)};
        // The window in use, the next one with its scales, and the pool pages of the one behind that: no stage
        // waits for a chain of loads.
        const int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
        auto pool_page = [&](int w0) { return w0 + lane < n_pages ? row[w0 + lane] : -1; };
        int w0 = s0 * STAGE_TOK >> page_log;  // first page of the window
        Page next = scales_of(pool_page(w0), h);
        int behind = pool_page(w0 + 32);
        open_segment(sg, q);
        for (int s = s0; s < s1 && ok;) {
          open_window(next.id, static_cast<int>(static_cast<uint32_t>(w0 + lane) << page_log), next.ks, next.vs);
          next = scales_of(behind, h);
          behind = pool_page(w0 + 64);
          // stages of this window (its end may be past 2^31 tokens)
          const int end = min(s1, static_cast<int>((static_cast<uint32_t>(w0 + 32) << page_log) >> STAGE_LOG));
          put_all(sg, whole, s0, s1, s, end, w0 << page_log, 32);
          s = end;
          w0 += 32;
        }
        u += s1 - s0;
        s0 = 0;
        if (u < u1 && ++h == a.Hkv) {
          h = 0;
          do n_st = stages_of(a, ++b);
          while (n_st == 0);
        }
        if (u < u1) q = load_q(b, h);
      }
    }
    if (lane == 0) {
      if (ok) put(SegmentHead{0, 0, 0, 0}, SEG_END, it++, 0, 0);
      // never leave a copy landing in a finished block
      for (int k = it > L::NS ? it - L::NS : 0; k < it; ++k) mbar_wait(&full[k % L::NS], (k / L::NS) & 1);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  constexpr int NT = D / 8, KS = D / 16, VB = D / 8, KB = D / 4;  // KB, VB: bytes of a lane's part of a row
  constexpr int KC = KB < 16 ? KB : 16, VC = VB < 4 ? 4 : VB;
  float(*merge)[ROWS][L::CST] = reinterpret_cast<float(*)[ROWS][L::CST]>(smem + L::MERGE_OFF);
  float2(*ml)[ROWS] = reinterpret_cast<float2(*)[ROWS]>(smem + L::ML_OFF);
  const int g = lane >> 2, t = lane & 3, slice = warp;
  uint32_t qa[KS][4];
  float f0 = 0.0f, f1 = 0.0f, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f, vref = 0.0f;
  float acc[NT][4];
  int merges = 0, seg = 0;
  SegmentHead sg{0, 0, 0, 0};
  for (int it = 0;; ++it) {
    const int st = it % L::NS;
    if (!mbar_wait(&full[st], (it / L::NS) & 1)) break;
    const StageHead* hd = &heads[st];
    const int flags = hd->flags;
    if (flags & SEG_END) break;
    if (flags & SEG_FIRST) {
      const uint8_t* qs = smem + L::Q_OFF + (seg & 1) * L::Q_BYTES;
      sg = segs[seg & 1];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint4 w = reinterpret_cast<const uint4*>(qs)[32 * k + lane];
        qa[k][0] = w.x;
        qa[k][1] = w.y;
        qa[k][2] = w.z;
        qa[k][3] = w.w;
      }
      f0 = reinterpret_cast<const float*>(qs + 32 * KS * 16)[g];
      f1 = reinterpret_cast<const float*>(qs + 32 * KS * 16)[g + 8];
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[seg & 1]);
      ++seg;
      m0 = m1 = -INFINITY;
      l0 = l1 = vref = 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    }
    const int4 what = hd->slice[slice];
    const int tok0 = what.x, len = sg.len;
    if (tok0 >= 0) {
      const uint32_t sK = smem_u32(smem + st * 2 * L::KV), sV = sK + L::KV;
      const uint32_t k_off = (slice * 16 + g) * D + t * KB;
      float sc[2][4];
      {
        Words<KC> kw[2][KB / KC];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int c = 0; c < KB / KC; ++c) kw[j][c] = load_shared<KC>(sK + swz128(k_off + j * 8 * D + c * KC));
          sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = kw[j][k / (KC / 4)].w[k % (KC / 4)];
            mma_f16(sc[j], qa[k], f16_lo(w), f16_hi(w));
          }
      }
      Words<VC> vw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t off = (slice * 16 + 2 * t + (j & 1) + (j >> 1) * 8) * D + (g * VB & ~3);
        vw[j] = load_shared<VC>(sV + swz128(off));
        if constexpr (VB < VC) vw[j].w[0] >>= (g & 1) * 16;
      }
      const float ks = __int_as_float(what.y), vs = __int_as_float(what.z);
      const float e0 = f0 * ks, e1 = f1 * ks;
      const bool tail = tok0 + 16 > len;
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = !tail || tok0 + 8 * j + 2 * t + e < len;
          sc[j][e] = in ? sc[j][e] * e0 : -INFINITY;
          sc[j][2 + e] = in ? sc[j][2 + e] * e1 : -INFINITY;
          mx0 = fmaxf(mx0, sc[j][e]);
          mx1 = fmaxf(mx1, sc[j][2 + e]);
        }
      if (tail) {  // codes behind the last token may be anything
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tok0 + (j & 1) + (j >> 1) * 8 + 2 * t >= len)
#pragma unroll
            for (int i = 0; i < VC / 4; ++i) vw[j].w[i] = 0u;
      }
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      // lazy rescale: the reference moves only when a probability would exceed 2^15
      if (__any_sync(0xffffffffu, mx0 - m0 > P_MAX || mx1 - m1 > P_MAX)) {
        const float n0 = fmaxf(m0, reference_of(mx0)), n1 = fmaxf(m1, reference_of(mx1));
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
      // The accumulator is held in units of vref, the largest scale so far.  A page whose scale is at least 2^-3 of it
      // (nearly all are) has the ratio folded into its probabilities, and its product goes straight into the
      // accumulator; another's is taken on its own and added under its scale: an f16 would lose what a smaller ratio
      // leaves of a probability, and what a larger one makes of it.
      if (vref == 0.0f) vref = vs;
      const float ratio = vref != 0.0f ? vs / vref : 0.0f;
      const bool fold = ratio >= 0.125f && ratio <= 1.0f;
      const float fr = fold ? ratio : 1.0f;
      uint32_t pa[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float y0 = ex2f(sc[j][0] - b0), y1 = ex2f(sc[j][1] - b0);
        const float y2 = ex2f(sc[j][2] - b1), y3 = ex2f(sc[j][3] - b1);
        l0 += y0 + y1;
        l1 += y2 + y3;
        pa[2 * j] = pack_f16x2(y0 * fr, y1 * fr);
        pa[2 * j + 1] = pack_f16x2(y2 * fr, y3 * fr);
      }
      // acc += (sigma^V / vref) (P V)
      if (fold) {
#pragma unroll
        for (int i = 0; i < NT; i += 2) {  // column tiles i and i + 1: bytes i, i + 1 of each token's run
          const int w = i / 4;
          const uint32_t pick = (i & 2) ? 0x7362u : 0x5140u;
          const uint32_t x01 = __byte_perm(vw[0].w[w], vw[1].w[w], pick);
          const uint32_t x23 = __byte_perm(vw[2].w[w], vw[3].w[w], pick);
          mma_f16(acc[i], pa, f16_lo(x01), f16_lo(x23));
          mma_f16(acc[i + 1], pa, f16_hi(x01), f16_hi(x23));
        }
      } else {
        const float grow = ratio > 1.0f ? vref / vs : 1.0f, add = ratio > 1.0f ? 1.0f : ratio;
        if (ratio > 1.0f) vref = vs;
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          const int w = i / 4;
          const uint32_t pick = (i & 2) ? 0x7362u : 0x5140u;
          const uint32_t x01 = __byte_perm(vw[0].w[w], vw[1].w[w], pick);
          const uint32_t x23 = __byte_perm(vw[2].w[w], vw[3].w[w], pick);
          float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(d0, pa, f16_lo(x01), f16_lo(x23));
          mma_f16(d1, pa, f16_hi(x01), f16_hi(x23));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[i][e] = fmaf(add, d0[e], acc[i][e] * grow);
            acc[i + 1][e] = fmaf(add, d1[e], acc[i + 1][e] * grow);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (!(flags & SEG_LAST)) continue;

    // ---- the segment's end: the eight warps' states into one (the producer is already at the next segment)
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // every warp has read the last merge (bounded waits, so that a warp that gave up leaves no other behind)
    if (merges > 0 && !mbar_wait(&merge_bar[1], (merges - 1) & 1)) break;
    // column n = 2t, 2t + 1 of tile j, which is dim n D/8 + j, at place 8 j + n: no bank conflicts here or below
    const float unit = vref * P_UNIT;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(&merge[warp][g][8 * j + 2 * t]) = make_float2(acc[j][0] * unit, acc[j][1] * unit);
      *reinterpret_cast<float2*>(&merge[warp][g + 8][8 * j + 2 * t]) = make_float2(acc[j][2] * unit, acc[j][3] * unit);
    }
    if (t == 0) {
      ml[warp][g] = make_float2(m0, l0 * P_UNIT);
      ml[warp][g + 8] = make_float2(m1, l1 * P_UNIT);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&merge_bar[0]);
    if (!mbar_wait(&merge_bar[0], merges & 1)) break;
    {
      // 16 threads a row: two columns n, n + 1 of a quarter of the tiles (D = 16: of half of them, 8 threads)
      constexpr int PER = NT >= 4 ? NT / 4 : 1;
      const int row = threadIdx.x >> 4, n = 2 * (threadIdx.x & 3), j0 = (threadIdx.x >> 2 & 3) * PER;
      float M = -INFINITY, sum = 0.0f, wt[CONSUMERS], y[2][PER];
#pragma unroll
      for (int w = 0; w < CONSUMERS; ++w) M = fmaxf(M, ml[w][row].x);
      const float mb = M == -INFINITY ? 0.0f : M;
#pragma unroll
      for (int w = 0; w < CONSUMERS; ++w) {
        wt[w] = ex2f(ml[w][row].x - mb);
        sum += wt[w] * ml[w][row].y;
      }
      const bool mine = j0 < NT;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        y[0][e] = y[1][e] = 0.0f;
        if (mine)
#pragma unroll
          for (int w = 0; w < CONSUMERS; ++w) {
            const float2 v = *reinterpret_cast<const float2*>(&merge[w][row][8 * (j0 + e) + n]);
            y[0][e] += wt[w] * v.x;
            y[1][e] += wt[w] * v.y;
          }
      }
      if (row < a.G) {
        const size_t orow = static_cast<size_t>(sg.b) * a.Hq + static_cast<size_t>(sg.h) * a.G + row;
        if (flags & SEG_WHOLE) {
          const float inv = inverse_sum(sum);
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // dims (n + c) D/8 + j0 ..
            __nv_bfloat16* o = a.out + orow * D + (n + c) * NT + j0;
            if constexpr (PER == 1) {
              if (mine) o[0] = __float2bfloat16_rn(y[c][0] * inv);
            } else {
#pragma unroll
              for (int e = 0; e < PER; e += 2)
                *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(y[c][e] * inv, y[c][e + 1] * inv);
            }
          }
          if (a.lse != nullptr && (threadIdx.x & 15) == 0) a.lse[orow] = lse_of(M, sum);
        } else {  // partial: [m, l] of every row, then the accumulator rows
          float* part = a.ws + static_cast<size_t>(sg.part) * part_floats(D);
          if ((threadIdx.x & 15) == 0) *reinterpret_cast<float2*>(part + 2 * row) = make_float2(M, sum);
          if (mine)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < PER; ++e) part[2 * ROWS + row * D + (n + c) * NT + j0 + e] = y[c][e];
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&merge_bar[1]);
    ++merges;
  }
}

// Selected pages: a cluster for each (sequence, kv head), its slots shared out over the cluster's blocks.
template <int D, int C>
__global__ void __launch_bounds__(THREADS, (Dec<D, C>::CTAS)) nsa_decode_select_kernel(const DecodeArgs a) {
  using L = Dec<D, C>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float ml[WARPS][ROWS][2];
  __shared__ float part_ml[ROWS][2];
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int cs = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int item = blockIdx.x / cs, b = item / a.Hkv, h = item % a.Hkv;
  const int row = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * (D / 8);
  const size_t qrow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G;
  float y[D / 8], M, sum;
  decode_range<D, C>(a, b, h, a.S * rank / cs, a.S * (rank + 1) / cs, smem, ml, y, M, sum);
  if (cs == 1) {
    if (row < a.G) {
      const float inv = inverse_sum(sum);
#pragma unroll
      for (int e = 0; e < D / 8; e += 2)
        *reinterpret_cast<uint32_t*>(a.out + (qrow + row) * D + d0 + e) = pack_bf16x2(y[e] * inv, y[e + 1] * inv);
      if (a.lse != nullptr && (threadIdx.x & 7) == 0) a.lse[qrow + row] = lse_of(M, sum);
    }
    return;
  }
  // this block's rows, over the merge area of its warps
  float(*part)[L::CST] = reinterpret_cast<float(*)[L::CST]>(smem);
  __syncthreads();
  if ((threadIdx.x & 7) == 0) {
    part_ml[row][0] = M;
    part_ml[row][1] = sum;
  }
#pragma unroll
  for (int e = 0; e < D / 8; e += 2) *reinterpret_cast<float2*>(&part[row][d0 + e]) = make_float2(y[e], y[e + 1]);
  cluster.sync();
  // rank r joins rows r, r + cs, ...
  for (int e = threadIdx.x; e < ROWS / cs * (D / 2); e += THREADS) {
    const int r = e / (D / 2) * cs + rank, d = e % (D / 2) * 2;
    if (r >= a.G) break;
    float top = -INFINITY, total = 0.0f, x0 = 0.0f, x1 = 0.0f;
    for (int k = 0; k < cs; ++k) top = fmaxf(top, cluster.map_shared_rank(&part_ml[r][0], k)[0]);
    const float tb = top == -INFINITY ? 0.0f : top;
    for (int k = 0; k < cs; ++k) {
      const float* pm = cluster.map_shared_rank(&part_ml[r][0], k);
      const float w = ex2f(pm[0] - tb);
      const float2 v = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&part[r][d], k));
      total += w * pm[1];
      x0 += w * v.x;
      x1 += w * v.y;
    }
    const float inv = inverse_sum(total);
    *reinterpret_cast<uint32_t*>(a.out + (qrow + r) * D + d) = pack_bf16x2(x0 * inv, x1 * inv);
    if (a.lse != nullptr && d == 0) a.lse[qrow + r] = lse_of(top, total);
  }
  cluster.sync();  // no block leaves while another reads its rows
}

// Joins the parts of a (sequence, kv head) that several ranges cover, and
// answers for a sequence without tokens.  One block for two rows of it, eight
// warps a row: each takes every eighth part, and the eight are joined last (a
// pair of long sequences has tens of parts: with four warps a row four
// sequences of up to 131072 tokens took 44.1 us, with one 48.9, now 43.2).
constexpr int JOIN_ROWS = 2, JOIN_WARPS = 8, JOIN_THREADS = JOIN_ROWS * JOIN_WARPS * 32;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) nsa_decode_join_kernel(const DecodeArgs a) {
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

template <int D, int C>
int launch_cluster(const DecodeArgs& a, cudaStream_t stream) {
  using L = Dec<D, C>;
  const long long items = static_cast<long long>(a.B) * a.Hkv;
  // Blocks of a cluster: as many, of whole slots, as leave each a SM.  More share the SMs (24 sequences of 4 kv heads
  // and 16 pages of 64 tokens of 128, with cold caches: one block a pair 15.0 us, two 17.7, four 23.7, eight 27.4; of
  // 64 dims 10.6, 11.0, 10.1, 15.7); fewer leave some idle (one sequence of 2 kv heads: 14.1, 13.3, 9.5, 8.1).
  int cs = 1;
  while (cs < 8 && 2 * cs <= a.S && 2 * items * cs <= sm_count()) cs *= 2;
  auto kern = nsa_decode_select_kernel<D, C>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) != cudaSuccess)
    return ERR_LAUNCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * cs));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = L::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? OK : ERR_LAUNCH;
}

template <int D>
int launch_stream(DecodeArgs a, cudaStream_t stream) {
  using L = StreamLayout<D>;
  const int sms = sm_count();
  if (sms < 1) return ERR_DEVICE;
  const long long items = static_cast<long long>(a.B) * a.Hkv;
  // the pool's pages of one head as 128-byte lines
  CUtensorMap mk, mv;
  const uint64_t lines = static_cast<uint64_t>(a.page) * D / 128, heads = static_cast<uint64_t>(a.num_pages) * a.Hkv;
  int st = encode_tmap_3d_u8(&mk, a.k, 128, lines, heads, 128, lines * 128, 128, static_cast<uint32_t>(lines), 1);
  if (st == OK)
    st = encode_tmap_3d_u8(&mv, a.v, 128, lines, heads, 128, lines * 128, 128, static_cast<uint32_t>(lines), 1);
  if (st != OK) return st;
  const long long units = items * ((static_cast<long long>(a.max_pages) * a.page + STAGE_TOK - 1) / STAGE_TOK);
  const long long most = sms < DECODE_MAX_RANGES ? sms : DECODE_MAX_RANGES;
  a.ranges = static_cast<int>(units < most ? units : most);
  if (cudaFuncSetAttribute(nsa_decode_stream_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) !=
      cudaSuccess)
    return ERR_LAUNCH;
  nsa_decode_stream_kernel<D><<<static_cast<unsigned>(a.ranges), STREAM_THREADS, L::BYTES, stream>>>(mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  // started while the first kernel's last blocks run (its blocks wait before they read a part)
  const long long joins = items * ((a.G + JOIN_ROWS - 1) / JOIN_ROWS);  // (no more than B * Hq)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(joins));
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, nsa_decode_join_kernel<D>, a) == cudaSuccess ? OK : ERR_LAUNCH;
}

template <int D>
int launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  if (a.block_idx == nullptr) return launch_stream<D>(a, stream);
  // chunks of 32 tokens (half the work for masks, maxima and scales per token) where a page holds them
  return a.page >= 32 ? launch_cluster<D, 32>(a, stream) : launch_cluster<D, 16>(a, stream);
}

}  // namespace

// The partials of the most ranges (the size does not depend on the device); selected pages leave none.
size_t nsa_decode_workspace_bytes(int D, int S) {
  return S > 0 ? 256 : 2 * static_cast<size_t>(DECODE_MAX_RANGES) * part_floats(D) * sizeof(float);
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
  a.scale_log2 = LOG2E / sqrtf(static_cast<float>(D));
  switch (D) {
    case 16: return launch_decode<16>(a, stream);
    case 32: return launch_decode<32>(a, stream);
    case 64: return launch_decode<64>(a, stream);
    case 128: return launch_decode<128>(a, stream);
    default: return ERR_UNSUPPORTED;
  }
}

unsigned int nsa_decode_device_error() { return read_and_clear_device_error(); }

}  // namespace bsa
