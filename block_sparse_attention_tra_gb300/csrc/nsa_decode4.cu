// nsa_decode4.cu -- selection attention of one query token per sequence over a
// paged cache of e2m1 codes with an e4m3 scale for every 16 elements.
//
// The formulas are nsa_decode.cu's; a key or value element is scale * code
// (times a factor of the kv head, which goes into the scores and the result).
// A code has two significant bits and a scale four, so their product is exact
// in f16, and no key or value is rounded on the way: a lane turns pairs of
// codes into f16x2 by one conversion and multiplies them by their scales
// before the products, mma.sync.m16n8k16 over 16 query rows as there, or over
// 16 tokens (scores) and 16 dims (output) by eight query rows where a kv head
// has no more: half the products, scores and accumulators.
//  - scores: D is summed over, so its order is free: lane (g, t) takes the D/4
//    dims of its own quarter of a token's row.
//  - output: lane (g, t) takes, of four tokens, the D/8 dims that are its
//    column g of the D/8 column tiles; the nibbles of two tokens are laid side
//    by side (a shift and a select for four pairs), and a pair's scales are
//    one f16x2.  The tokens of a slice of 16 are numbered so that the four
//    that a lane has probabilities of follow each other.
// The fragments are the same numbers either way; with eight rows a slice's
// probabilities are transposed (movmatrix) from a lane's row of tokens to its
// column of them.
// Query rows, probabilities (f16 over 2^-11 to 2^-15 of the largest so far),
// sums and joins are those of nsa_decode.cu.
//
// A warp works for itself: chunks of 32 tokens (16 where pages hold 16) of its
// pages come by cp.async into a ring of its own in shared memory, whose places
// it alone fills and empties, so that warps wait for nothing but their copies.
// (By four bulk copies a chunk, codes and scales of keys and values, four
// sequences of up to 131072 tokens took a sixth longer.)
//
// Selected pages: a block of four warps a (sequence, kv head), or with few of
// them a cluster that shares out the slots; and so, by their stages of 128
// tokens, every page of short tables.  Else the list of (sequence, kv head,
// stage) is cut into equal contiguous ranges, one a
// block, or with few pairs each of these by itself; pairs that several ranges
// cover are joined by a second launch.
//
// Long lists of 16 query rows run at 67% of what the measured copy rate takes for their bytes (32 sequences of 131072
// tokens of 32 query and 2 kv heads of 128: 1209 MB in 265 us, 4.6 TB/s), of eight at 78% (16 of 20000 to 60000, 4 kv
// heads: 70 us), at 58% with heads of 64 and at 38% with heads of 32 (46.6 and 35.7 us): a chunk then has a half or a
// quarter of the bytes under the same softmax and page steps.  The copies by themselves, nothing worked out, take the copy rate's time to within 1%, the work by itself
// 93% of the whole: a chunk of 32 tokens is some 700 instructions of a warp, 128 conversions and 128 products with scales
// of two cycles and 64 matrix products (eight rows: 32) of eight among them, and three or four warps a scheduler do not
// fill the gaps of their chains.  (Packed pairs of fp32 for the softmax, 24 instructions fewer, changed nothing.)  The
// rest of a call is the chain at its start (lengths, pages, codes) and the joins: four sequences of 20011 to 131072
// tokens, 87 MB, take 29.3 us with the second launch, some 3 of them in it; 128 on 16 pages each 26.0, one 5.5,
// 17 of up to 5003 in one launch 8.5.
#include <cooperative_groups.h>

#include "codes4.cuh"
#include "kernels.h"
#include "nsa_decode.cuh"
#include "nsa_slots.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int PAIR_STAGES = 16;  // of a block in a cluster over every page, at most

struct Decode4Args {
  const __nv_bfloat16* q;
  const uint8_t *k, *v, *k_scale, *v_scale;
  const float *k_factor, *v_factor;         // per kv head, or null
  const int32_t *table, *lens, *block_idx;  // block_idx null: every page
  __nv_bfloat16* out;
  float* lse;
  float* ws;
  int B, Hq, Hkv, G, page, max_pages, num_pages, S;
  int ranges;     // blocks of the first kernel over every page
  bool pairwise;  // ranges within a (sequence, kv head)
  float scale_log2;
};

template <int D, int C, bool FEW>
struct Dec4 {  // FEW: at most eight query rows a kv head
  // Blocks of a SM at most.  D = 128: 64 of a thread's registers are accumulators.  Of 128 each, sixteen warps fit, which
  // selected pages want for their start (128 sequences of 4 kv heads on 16 pages of 64: 27.5 us, twelve warps of 160
  // registers 28.4); ranges over every page are faster with twelve (four sequences of up to 131072 tokens: 27.8 and 29.6).
  // FEW, 32 accumulators, is no different: twelve 70.3 us, sixteen 72.6 over every page (16 sequences of 4 kv heads), 65.2
  // and 60.5 on selected ones (512 sequences), twenty 62.5.
  static constexpr int SELECT_CTAS = 4, STREAM_CTAS = D == 128 ? 3 : 4;
  static constexpr int PAIR_CTAS(bool select) { return select || FEW ? SELECT_CTAS : STREAM_CTAS; }
  static constexpr int RING = (D == 128 ? 64 : 128) / C;  // chunks of a warp in flight or in use
  static constexpr int RB = D / 2, SB = D / 16;  // bytes of a token's codes, of its scales
  static constexpr int V_OFF = C * RB, KS_OFF = 2 * C * RB, VS_OFF = KS_OFF + C * SB;
  static constexpr int SLOT = VS_OFF + C * SB;  // a chunk of a warp
  static constexpr int CST = D + 8;             // row stride of the merge area
  // the ring, and over it (a range's chunks are done with then) the merge area
  static constexpr int MERGE = WARPS * ROWS * CST * 4;
  static constexpr int Q_OFF = WARPS * RING * SLOT > MERGE ? WARPS * RING * SLOT : MERGE;
  static constexpr int Q_STEP = FEW ? 256 : 512;                 // query fragments of 16 dims: two or four words a lane
  static constexpr int BYTES = Q_OFF + D / 16 * Q_STEP + ROWS * 4;  // and the rows' factors
  static_assert(SLOT % 16 == 0 && (C * SB) % 16 == 0 && C * SB <= 256, "16-byte copies");
};

// Where byte `off` of a chunk's codes lies: 16-byte pieces of a 128-byte line change places so that neither keys (whole
// quarters of rows) nor values (runs of four rows) meet in a bank.
template <int D>
__device__ __forceinline__ uint32_t place_of(uint32_t off) {
  if constexpr (D == 128) return off ^ (off >> 3 & 0x60u);
  else if constexpr (D == 64) return off ^ (off >> 1 & 0x40u) ^ (off >> 3 & 0x20u);
  else return off;
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two e4m3 scales (the low 16 bits) as f16x2.
__device__ __forceinline__ uint32_t f16_of_scales(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A matrix of 8 x 8 f16, two neighbours of row lane / 4 a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// N bytes of shared memory in 32-bit words (fewer than four: the low ones of one).  (Plain loads: the compiler moves them
// ahead of the products between two waits.)
template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t (&w)[(N + 3) / 4]) {
  if constexpr (N == 16) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  } else if constexpr (N == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else if constexpr (N == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    w[0] = N == 2 ? *reinterpret_cast<const uint16_t*>(p) : *p;
  }
}

// N words of device memory, in pieces of up to 16 bytes.
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// A warp's pages in shared memory: SELECT: first token (-1: none) and (pool page, head) of each slot; else the (pool page,
// head) of pages w0 + i (-1: none).
struct PageList {
  int tok[32], id[32];
};

// The chunks of one warp: its share of a range, page by page, and their way into its ring.  (Kept small: with sixteen warps
// a SM, 64 of a thread's 128 registers are accumulators, and as the rings leave little L1, what is spilled goes to the L2.)
template <int D, int C, bool FEW, bool SELECT>
struct Feed {
  using L = Dec4<D, C, FEW>;
  const Decode4Args& a;
  PageList& list;
  int at, end;      // SELECT: next chunk, chunks of the range; else next token, the range's last
  int first, len;   // SELECT: first slot; tokens of the sequence
  int w0, id_next;  // else: the list's first page; a page of the list after it

  __device__ __forceinline__ int page_log() const { return 31 - __clz(a.page); }
  // (pool page, head) of page p, one number of 31 bits, or -1.
  __device__ __forceinline__ int page_id(int p, int b, int h) const {
    if (p >= pieces_of(len, page_log())) return -1;
    const int i = a.table[static_cast<size_t>(b) * a.max_pages + p];
    return i >= 0 && i < a.num_pages ? i * a.Hkv + h : -1;
  }
  // Next chunk into place `place` (a group of copies, empty behind the last): its first token, or -1.
  __device__ __forceinline__ int put(uint32_t ring, int place, const volatile int* bh) {
    const int tok0 = next(ring + place * L::SLOT, bh);
    copy_commit();
    return tok0;
  }
  __device__ __forceinline__ int next(uint32_t dst, const volatile int* bh) {
    const int lane = threadIdx.x & 31;
    while (at < end) {
      int tok0, id;
      if constexpr (SELECT) {
        const int cpp_log = page_log() - (C == 32 ? 5 : 4), u = first + (at >> cpp_log);
        const int sub = at & ((1 << cpp_log) - 1);
        tok0 = list.tok[u];
        id = list.id[u];
        at += WARPS;
        if (tok0 < 0) continue;
        tok0 += sub * C;
        if (tok0 >= len) continue;
      } else {
        tok0 = at;
        at = end - at > WARPS * C ? at + WARPS * C : end;  // (at most 2^31 - 16)
        const int p = tok0 >> page_log();
        if (p >= w0 + 32) {
          int now;
          do {
            w0 += 32;
            now = id_next;
            id_next = page_id(w0 + 32 + lane, bh[0], bh[1]);
          } while (p >= w0 + 32);
          __syncwarp();
          list.id[lane] = now;
          __syncwarp();
        }
        id = list.id[p - w0];
        if (id < 0) continue;
      }
      debug_check(id >= 0 && id < a.num_pages * a.Hkv && tok0 + C <= pieces_of(len, page_log()) << page_log());
      const size_t row = (static_cast<size_t>(id) << page_log()) + (tok0 & (a.page - 1));
      const uint8_t *k = a.k + row * L::RB + lane * 16, *v = a.v + row * L::RB + lane * 16;
#pragma unroll
      for (int i = 0; i < (C * L::RB + 511) / 512; ++i)
        if (C * L::RB >= 512 || lane * 16 < C * L::RB) {
          const uint32_t off = place_of<D>(lane * 16 + i * 512);
          copy16(dst + off, k + i * 512);
          copy16(dst + L::V_OFF + off, v + i * 512);
        }
      // scales of keys by the first half of the warp, of values by the second
      const uint8_t* sc = (lane < 16 ? a.k_scale : a.v_scale) + row * L::SB;
      if ((lane & 15) * 16 < C * L::SB)
        copy16(dst + (lane < 16 ? L::KS_OFF : L::VS_OFF) + (lane & 15) * 16, sc + (lane & 15) * 16);
      return tok0;
    }
    return -1;
  }
};

// Slots [p0, p1) of (b, h)'s selection, or tokens [p0, p1) of the sequence: the block's 128 threads leave the range's
// unnormalised accumulator, weighted into one, in y (row threadIdx.x / 8, dims (threadIdx.x % 8) D/8 ..), its maximum
// (log2 domain) in M and its sum of exponentials in sum.
template <int D, int C, bool FEW, bool SELECT>
__device__ __forceinline__ void decode_range(const Decode4Args& a, int b, int h, int p0, int p1, uint8_t* smem,
                                             PageList* lists, float (*ml)[ROWS][2], float (&y)[D / 8], float& M,
                                             float& sum, const volatile int* bh) {
  using L = Dec4<D, C, FEW>;
  constexpr int NT = D / 8, KS = D / 16, RING = L::RING;
  float(*merge)[ROWS][L::CST] = reinterpret_cast<float(*)[ROWS][L::CST]>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int len = tokens_of(a, b);
  const size_t qrow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G;

  // The query rows, eight threads each, asked for before anything else.
  constexpr int PAIRS = D / 16;  // of a thread
  uint32_t qw[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) qw[i] = 0u;
  if (static_cast<int>(threadIdx.x >> 3) < a.G)
    load_words<PAIRS>(a.q + (qrow + (threadIdx.x >> 3)) * D + (threadIdx.x & 7) * (D / 8), qw);
  const float factor = a.scale_log2 * (a.k_factor != nullptr ? a.k_factor[h] : 1.0f);

  Feed<D, C, FEW, SELECT> feed{a, lists[warp]};
  feed.len = len;
  if constexpr (SELECT) {
    const int32_t* pages = a.table + static_cast<size_t>(b) * a.max_pages;
    const SlotRow sel = nsa_live_slots(a.block_idx + (static_cast<size_t>(b) * a.Hkv + h) * a.S, a.S, len - 1,
                                       pieces_of(len, feed.page_log()), a.page);
    int tok = -1, id = 0;
    if (lane >= p0 && lane < p1 && ((sel.live >> lane) & 1u)) {
      id = pages[sel.blk_lane];
      if (id >= 0 && id < a.num_pages) tok = sel.blk_lane * a.page;
    }
    lists[warp].tok[lane] = tok;
    lists[warp].id[lane] = tok >= 0 ? id * a.Hkv + h : -1;
    feed.first = p0;
    feed.at = warp;
    feed.end = (p1 - p0) << (feed.page_log() - (C == 32 ? 5 : 4));
  } else {
    feed.w0 = p0 >> feed.page_log();
    lists[warp].id[lane] = feed.page_id(feed.w0 + lane, b, h);
    feed.id_next = feed.page_id(feed.w0 + 32 + lane, b, h);
    feed.end = p1;
    feed.at = p1 - p0 > warp * C ? p0 + warp * C : p1;
  }
  __syncwarp();
  // Query fragments, in the order of the keys' codes, each row under its own power of two.  (Loaded behind the first
  // chunks they came 5500 cycles later: after every SM's first copies.)
  uint8_t* q_frag = smem + L::Q_OFF;
  {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i)
      m = fmaxf(m, fmaxf(fabsf(__uint_as_float(qw[i] << 16)), fabsf(__uint_as_float(qw[i] & 0xffff0000u))));
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    // 2^e with the row's maximum in [2^14, 2^15) (1 for zero rows and infinities)
    const int ex = static_cast<int>(__float_as_uint(m) >> 23) - 127;
    const int e = ex >= -100 && ex < 128 ? 14 - ex : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    if ((threadIdx.x & 7) == 0)
      reinterpret_cast<float*>(q_frag + KS * L::Q_STEP)[threadIdx.x >> 3] =
          factor * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      // lane (row % 8, part / 2) of k-step (4 dims of a lane's D/4 each), rows g and g + 8, dims 0, 1 and 2, 3 of the four
      const int qr = threadIdx.x >> 3, part = threadIdx.x & 7, at = (part & 1) * (D / 8) + 2 * i;
      const uint32_t two = pack_f16x2(__uint_as_float(qw[i] << 16) * up, __uint_as_float(qw[i] & 0xffff0000u) * up);
      uint8_t* of_lane = q_frag + at / 4 * L::Q_STEP + (4 * (qr & 7) + (part >> 1)) * (L::Q_STEP / 32);
      if constexpr (FEW) {
        if (qr < 8) *reinterpret_cast<uint32_t*>(of_lane + (at >> 1 & 1) * 4) = two;
      } else {
        *reinterpret_cast<uint32_t*>(of_lane + (at >> 1 & 1) * 8 + (qr >> 3) * 4) = two;
      }
    }
  }
  const uint8_t* ring = smem + warp * RING * L::SLOT;
  const uint32_t ring32 = smem_u32(ring);
  int ahead[RING - 1];  // first tokens of those on their way, the next first
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) ahead[i] = feed.put(ring32, i, bh);

  __syncthreads();
  // A lane's two rows: of eight, 2 t and 2 t + 1 (the columns of its scores), else g and g + 8; their score factors
  const int row0 = FEW ? 2 * t : g, row1 = FEW ? 2 * t + 1 : g + 8;
  const float f0 = reinterpret_cast<const float*>(q_frag + KS * L::Q_STEP)[row0];
  const float f1 = reinterpret_cast<const float*>(q_frag + KS * L::Q_STEP)[row1];
  q_frag += lane * (L::Q_STEP / 32);

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  constexpr int NA = FEW ? NT / 2 : NT;
  float acc[NA][4];
#pragma unroll
  for (int j = 0; j < NA; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;

  int place = 0;
  while (ahead[0] >= 0) {
    const int tok0 = ahead[0];
#pragma unroll
    for (int i = 0; i < RING - 2; ++i) ahead[i] = ahead[i + 1];
    __syncwarp();  // every lane is done with the chunk used last, whose place is filled now
    ahead[RING - 2] = feed.put(ring32, place == 0 ? RING - 1 : place - 1, bh);
    copy_wait<RING - 1>();
    __syncwarp();  // and every lane's copies of this one are there
    const uint8_t* src = ring + place * L::SLOT;
    place = place == RING - 1 ? 0 : place + 1;
    // ---- scores: slices of 16 tokens, two tiles of 8 each; tile j's column n is token 4 (n / 2) + 2 j + n % 2
    constexpr int SC = FEW ? C / 16 : C / 8;
    float sc[SC][4];
#pragma unroll
    for (int j = 0; j < SC; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
    uint32_t kw[C / 8][(D / 8 + 3) / 4], ks2[C / 8][D == 128 ? 2 : 1];
#pragma unroll
    for (int j = 0; j < C / 8; ++j) {
      const int tk = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
      load_bytes<D / 8>(src + place_of<D>(tk * L::RB + t * (D / 8)), kw[j]);
      const uint8_t* sp = src + L::KS_OFF + tk * L::SB + t * (D / 4) / 16;
      if constexpr (D == 128) {
        const uint32_t s = *reinterpret_cast<const uint16_t*>(sp);
        ks2[j][0] = f16_of_scales(__byte_perm(s, 0u, 0x4400));
        ks2[j][1] = f16_of_scales(__byte_perm(s, 0u, 0x4411));
      } else {
        ks2[j][0] = f16_of_scales(*sp * 0x101u);
      }
    }
#pragma unroll
    for (int k = 0; k < (KS + 1) / 2; ++k) {  // a word of the row: two k-steps (D = 16: half a word, one)
      uint32_t q[2][L::Q_STEP / 128];
#pragma unroll
      for (int i = 0; i < 2 && 2 * k + i < KS; ++i) load_bytes<L::Q_STEP / 32>(q_frag + (2 * k + i) * L::Q_STEP, q[i]);
#pragma unroll
      for (int j = 0; j < C / 8; j += 2) {
        uint32_t x[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f16_of_codes(kw[j + e][k], x[e]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[e][i] = mul_f16x2(x[e][i], ks2[j + e][D == 128 ? k / 2 : 0]);
        }
#pragma unroll
        for (int i = 0; i < 2 && 2 * k + i < KS; ++i) {
          if constexpr (FEW) {  // tokens as rows, query rows as columns
            const uint32_t keys[4] = {x[0][2 * i], x[1][2 * i], x[0][2 * i + 1], x[1][2 * i + 1]};
            mma_f16(sc[j / 2], keys, q[i][0], q[i][1]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) mma_f16(sc[j + e], q[i], x[e][2 * i], x[e][2 * i + 1]);
          }
        }
      }
    }
    // The values' codes and scales, asked for before the scores are looked at (behind the probabilities: 17 sequences of
    // up to 5003 tokens of 3 heads of 64 8.7 us in place of 8.45, 16 of up to 60000 of 4 heads 47.7 and 46.7).
    uint32_t vw[C / 16][4][(D / 16 + 3) / 4], vs[C / 16][4];
#pragma unroll
    for (int s = 0; s < C / 16; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = 16 * s + 4 * t + i;
        load_bytes<D / 16>(src + L::V_OFF + place_of<D>(tk * L::RB + g * (D / 16)), vw[s][i]);
        vs[s][i] = src[L::VS_OFF + tk * L::SB + g * (D / 8) / 16];
      }
    }
    const bool tail = tok0 + C > len;
    // score e of sc[j]: of the lane's row `second(e)`, at token `token(j, e)` of the chunk
    const auto second = [](int e) { return FEW ? e & 1 : e >> 1; };
    const auto token = [&](int j, int e) {
      return FEW ? 16 * j + 4 * (g >> 1) + (g & 1) + (e & 2) : 16 * (j >> 1) + 4 * t + 2 * (j & 1) + (e & 1);
    };
    float mx0 = -INFINITY, mx1 = -INFINITY;
    // (rounded before the maximum is taken off: a fused form leaves the rounding of scores past 2^24 in the exponent)
#pragma unroll
    for (int j = 0; j < SC; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] *= second(e) ? f1 : f0;
    if (tail) {
#pragma unroll
      for (int j = 0; j < SC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tok0 + token(j, e) >= len) sc[j][e] = -INFINITY;
#pragma unroll
      for (int s = 0; s < C / 16; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tok0 + 16 * s + 4 * t + i >= len) vs[s][i] = 0u;  // scales behind the last token may be anything
    }
#pragma unroll
    for (int j = 0; j < SC; ++j) {
      mx0 = fmaxf(mx0, fmaxf(sc[j][0], sc[j][FEW ? 2 : 1]));
      mx1 = fmaxf(mx1, fmaxf(sc[j][FEW ? 1 : 2], sc[j][3]));
    }
    // over the lanes that hold scores of the same rows
#pragma unroll
    for (int d = FEW ? 4 : 1; d < (FEW ? 32 : 4); d *= 2) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
    }
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
      for (int j = 0; j < NA; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] *= second(e) ? s1 : s0;
    }
    const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
    for (int s = 0; s < C / 16; ++s) {
      uint32_t pa[4];
      if constexpr (FEW) {
        const float y0 = ex2f(sc[s][0] - b0), y1 = ex2f(sc[s][1] - b1);
        const float y2 = ex2f(sc[s][2] - b0), y3 = ex2f(sc[s][3] - b1);
        l0 += y0 + y2;
        l1 += y1 + y3;
        // from a lane's row of tokens to its column of them
        pa[0] = transpose8(pack_f16x2(y0, y1));
        pa[1] = transpose8(pack_f16x2(y2, y3));
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float y0 = ex2f(sc[2 * s + j][0] - b0), y1 = ex2f(sc[2 * s + j][1] - b0);
          const float y2 = ex2f(sc[2 * s + j][2] - b1), y3 = ex2f(sc[2 * s + j][3] - b1);
          l0 += y0 + y1;
          l1 += y2 + y3;
          pa[2 * j] = pack_f16x2(y0, y1);
          pa[2 * j + 1] = pack_f16x2(y2, y3);
        }
      }
      // ---- acc += P V of tokens 4t .. 4t + 3 of the slice
      const auto& of = vw[s];
      const uint32_t s01 = f16_of_scales(vs[s][0] | vs[s][1] << 8), s23 = f16_of_scales(vs[s][2] | vs[s][3] << 8);
#pragma unroll
      for (int w = 0; w < (D / 16 + 3) / 4; ++w) {
        uint32_t x01[2][4], x23[2][4];
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {  // even and odd nibbles of tokens 0 and 1, 2 and 3 side by side
          constexpr uint32_t LOW = 0x0f0f0f0fu;
          f16_of_codes(odd ? (of[0][w] >> 4 & LOW) | (of[1][w] & ~LOW) : (of[0][w] & LOW) | (of[1][w] << 4 & ~LOW),
                       x01[odd]);
          f16_of_codes(odd ? (of[2][w] >> 4 & LOW) | (of[3][w] & ~LOW) : (of[2][w] & LOW) | (of[3][w] << 4 & ~LOW),
                       x23[odd]);
          if constexpr (!FEW) {
#pragma unroll
            for (int i = 0; i < 4 && 2 * i + odd < NT; ++i)
              mma_f16(acc[8 * w + 2 * i + odd], pa, mul_f16x2(x01[odd][i], s01), mul_f16x2(x23[odd][i], s23));
          }
        }
        if constexpr (FEW) {  // dims as rows, query rows as columns
#pragma unroll
          for (int i = 0; i < 4 && 2 * i < NT; ++i) {
            const uint32_t values[4] = {mul_f16x2(x01[0][i], s01), mul_f16x2(x01[1][i], s01),
                                        mul_f16x2(x23[0][i], s23), mul_f16x2(x23[1][i], s23)};
            mma_f16(acc[4 * w + i], values, pa[0], pa[1]);
          }
        }
      }
    }
  }
  copy_wait<0>();

  // ---- the warps' states into one (over the ring: every warp is done with its chunks)
#pragma unroll
  for (int d = FEW ? 4 : 1; d < (FEW ? 32 : 4); d *= 2) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  __syncthreads();
  // dim n D/8 + j at place 8 j + n: no bank conflicts (few rows: two lanes a bank) here or below
  if constexpr (FEW) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      merge[warp][row0][8 * j + g] = acc[j / 2][2 * (j & 1)];
      merge[warp][row1][8 * j + g] = acc[j / 2][2 * (j & 1) + 1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(&merge[warp][row0][8 * j + 2 * t]) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(&merge[warp][row1][8 * j + 2 * t]) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  if ((FEW ? g : t) == 0) {
    ml[warp][row0][0] = m0;
    ml[warp][row0][1] = l0 * P_UNIT;
    ml[warp][row1][0] = m1;
    ml[warp][row1][1] = l1 * P_UNIT;
  }
  __syncthreads();
  const int row = threadIdx.x >> 3;
  const float unit = P_UNIT * (a.v_factor != nullptr ? a.v_factor[h] : 1.0f);
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
    y[e] *= unit;
  }
}

// A row's result, from y of its eight threads.
template <int D>
__device__ __forceinline__ void store_result(const Decode4Args& a, size_t row, int d0, const float (&y)[D / 8], float M,
                                             float sum) {
  const float inv = inverse_sum(sum);
#pragma unroll
  for (int e = 0; e < D / 8; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + row * D + d0 + e) = pack_bf16x2(y[e] * inv, y[e + 1] * inv);
  if (a.lse != nullptr && d0 == 0) a.lse[row] = lse_of(M, sum);
}

// Selected pages (SELECT), or every page of short sequences: a cluster for each (sequence, kv head), whose blocks share out
// the slots or the stages.
template <int D, int C, bool FEW, bool SELECT>
__global__ void __launch_bounds__(THREADS, (Dec4<D, C, FEW>::PAIR_CTAS(SELECT)))
    nsa_decode4_pair_kernel(const Decode4Args a) {
  using L = Dec4<D, C, FEW>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PageList lists[WARPS];
  __shared__ float ml[WARPS][ROWS][2];
  __shared__ float part_ml[ROWS][2];
  __shared__ int bh[2];
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int cs = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int item = blockIdx.x / cs, b = item / a.Hkv, h = item % a.Hkv;
  const int row = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * (D / 8);
  const size_t qrow = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G;
  float y[D / 8], M, sum;
  int p0 = 0, p1 = 0;
  if constexpr (SELECT) {
    p0 = a.S * rank / cs;
    p1 = a.S * (rank + 1) / cs;
  } else {
    if (threadIdx.x == 0) {
      bh[0] = b;
      bh[1] = h;
    }
    __syncthreads();
    const int n = tokens_of(a, b), n_st = pieces_of(n, STAGE_LOG);  // (at most 8 * PAIR_STAGES)
    p0 = min(n_st * rank / cs << STAGE_LOG, n);
    p1 = min(n_st * (rank + 1) / cs << STAGE_LOG, n);
  }
  decode_range<D, C, FEW, SELECT>(a, b, h, p0, p1, smem, lists, ml, y, M, sum, bh);
  if (cs == 1) {
    if (row < a.G) store_result<D>(a, qrow + row, d0, y, M, sum);
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

// range_start in 32 bits where its product is one.
__device__ __forceinline__ long long range_begin(long long units, int c, int ranges) {
  return units < (1LL << 21) ? static_cast<uint32_t>(units) * static_cast<uint32_t>(c) / static_cast<uint32_t>(ranges)
                             : range_start(units, c, ranges);
}

// range_of likewise.
__device__ __forceinline__ int range_at(long long units, long long u, int ranges) {
  static_assert(DECODE4_MAX_RANGES < 1024, "(u + 1) ranges + units in 32 bits");
  if (units >= (1LL << 21)) return range_of(units, u, ranges);
  const uint32_t n = static_cast<uint32_t>(units);
  return static_cast<int>(((static_cast<uint32_t>(u) + 1) * static_cast<uint32_t>(ranges) + n - 1) / n - 1);
}

// What a block of whole pairs' ranges takes: ranges of its pair, and the first of these ranges.  A pair of n of all stages
// has 1 + n (ranges - pairs) / stages of them, at most n.  One warp, lane i's sequence being i (B <= 32).
struct PairRanges {
  int tokens, n_st, count, before;  // of sequence `lane`: its ranges are Hkv times `count`, after `before` others
};
__device__ __forceinline__ PairRanges pair_ranges(const Decode4Args& a) {
  const int lane = threadIdx.x & 31;
  PairRanges r;
  r.tokens = lane < a.B ? tokens_of(a, lane) : 0;
  r.n_st = pieces_of(r.tokens, STAGE_LOG);
  long long units = r.n_st;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) units += __shfl_xor_sync(0xffffffffu, units, d);
  units *= a.Hkv;
  const int spare = a.ranges - a.B * a.Hkv;
  r.count = 0;
  if (r.n_st > 0)
    r.count = min(r.n_st, 1 + (units < (1LL << 21) ? static_cast<int>(static_cast<uint32_t>(r.n_st) * spare /
                                                                      static_cast<uint32_t>(units))
                                                   : static_cast<int>(static_cast<long long>(r.n_st) * spare / units)));
  int n = r.count * a.Hkv;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, n, d);
    if (lane >= d) n += x;
  }
  r.before = n - r.count * a.Hkv;
  return r;
}

// Every page: a block on one contiguous range of the (sequence, kv head, stage) list, or of a pair's stages; stage k holds
// tokens 128 k .. of the sequence.
template <int D, int C, bool FEW>
__global__ void __launch_bounds__(THREADS, (Dec4<D, C, FEW>::STREAM_CTAS))
    nsa_decode4_stream_kernel(const Decode4Args a) {
  using L = Dec4<D, C, FEW>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PageList lists[WARPS];
  __shared__ float ml[WARPS][ROWS][2];
  // the joining kernel's blocks may take the places that this one's leave (they wait for all of it)
  asm volatile("griddepcontrol.launch_dependents;");
  long long u0, u1;
  int b, h, s0, n_st;
  if (a.pairwise) {
    const PairRanges r = pair_ranges(a);
    const int block = static_cast<int>(blockIdx.x);
    const unsigned hit = __ballot_sync(0xffffffffu, block < r.before + r.count * a.Hkv);
    if (hit == 0u) return;
    b = __ffs(hit) - 1;
    n_st = __shfl_sync(0xffffffffu, r.n_st, b);
    const int count = __shfl_sync(0xffffffffu, r.count, b), k = block - __shfl_sync(0xffffffffu, r.before, b);
    h = k / count;
    s0 = static_cast<int>(range_begin(n_st, k % count, count));
    u0 = 0;
    u1 = range_begin(n_st, k % count + 1, count) - s0;
  } else {
    const long long units = units_of_warp(a);
    u0 = range_begin(units, blockIdx.x, a.ranges), u1 = range_begin(units, blockIdx.x + 1, a.ranges);
    if (u0 >= u1) return;
    long long before;
    b = sequence_of(a, u0, &before);
    n_st = stages_of(a, b);
    // (a sequence's units are fewer than 2^31 heads of 2^24 stages; nearly always a 32-bit number)
    const long long in = u0 - before;
    if (in >> 32 == 0) {
      h = static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(n_st));
      s0 = static_cast<int>(static_cast<uint32_t>(in) % static_cast<uint32_t>(n_st));
    } else {
      h = static_cast<int>(in / n_st);
      s0 = static_cast<int>(in % n_st);
    }
  }
  // What the loop needs behind a range waits in shared memory, not in registers beside the accumulators.
  __shared__ struct {
    long long u, u1;
    int bh[2], n_st, whole, part;
  } at;
  for (long long u = u0, last = u1; u < last;) {
    const int s1 = static_cast<int>(min(static_cast<long long>(n_st), s0 + (last - u)));
    const int end = static_cast<int>(min(static_cast<uint32_t>(s1) << STAGE_LOG, static_cast<uint32_t>(tokens_of(a, b))));
    if (threadIdx.x == 0) {
      at.u = u + (s1 - s0);
      at.u1 = last;
      at.bh[0] = b;
      at.bh[1] = h;
      at.n_st = n_st;
      at.whole = s0 == 0 && s1 == n_st;
      at.part = 2 * static_cast<int>(blockIdx.x) + (u != u0 ? 1 : 0);
    }
    __syncthreads();
    float y[D / 8], M, sum;
    decode_range<D, C, FEW, false>(a, b, h, s0 << STAGE_LOG, end, smem, lists, ml, y, M, sum, at.bh);
    const volatile auto& back = at;
    b = back.bh[0];
    h = back.bh[1];
    const int row = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * (D / 8);
    if (row < a.G) {
      if (back.whole) {
        store_result<D>(a, static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G + row, d0, y, M, sum);
      } else {  // partial: [m, l] of every row, then the accumulator rows
        float* part = a.ws + static_cast<size_t>(back.part) * part_floats(D);
        if ((threadIdx.x & 7) == 0) *reinterpret_cast<float2*>(part + 2 * row) = make_float2(M, sum);
#pragma unroll
        for (int e = 0; e < D / 8; e += 2)
          *reinterpret_cast<float2*>(part + 2 * ROWS + row * D + d0 + e) = make_float2(y[e], y[e + 1]);
      }
    }
    u = back.u;
    last = back.u1;
    n_st = back.n_st;
    s0 = 0;
    if (u < last) {
      if (++h == a.Hkv) {
        h = 0;
        do n_st = stages_of(a, ++b);
        while (n_st == 0);
      }
      __syncthreads();  // the merge area and what was kept are read before the next copies and range over them
    }
  }
}

// Joins the parts of a pair that several ranges cover, and answers for a sequence without tokens.  A block for R rows of
// a pair, WARPS_A_ROW warps each: its first warp works out which parts it joins, beside the first kernel's last blocks, and
// all wait for that kernel before they read one.  Warp w of a row takes the parts c0 + w, c0 + w + WARPS_A_ROW, ...,
// eight on their way at once.
constexpr int JOIN_WARPS = 8, JOIN_AHEAD = 8;
template <int D, int R>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4) nsa_decode4_join_kernel(const Decode4Args a) {
  constexpr int V = D / 32 > 0 ? D / 32 : 1, LANES = D / V;  // dims of a lane, lanes of a row
  constexpr int WARPS_A_ROW = JOIN_WARPS / R;
  __shared__ float2 state[JOIN_WARPS];
  __shared__ float part_o[JOIN_WARPS][D];
  __shared__ struct {
    long long units;
    int c0, c1, first;  // the pair's ranges; 1 if the first begins before it, and so leaves it second
  } in;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.G + R - 1) / R, pair = static_cast<int>(blockIdx.x / groups);
  const int b = pair / a.Hkv, h = pair % a.Hkv, row0 = static_cast<int>(blockIdx.x % groups) * R;
  const int row = row0 + warp / WARPS_A_ROW, w0 = warp % WARPS_A_ROW;
  if (warp == 0 && a.pairwise) {
    const PairRanges r = pair_ranges(a);
    const int count = __shfl_sync(0xffffffffu, r.count, b), before = __shfl_sync(0xffffffffu, r.before, b);
    if (lane == 0) {
      in.units = a.ranges;  // (no range is empty)
      in.c0 = before + h * count;
      in.c1 = before + (h + 1) * count - 1;
      in.first = 0;
    }
  } else if (warp == 0) {
    // units before the sequence and in all
    long long before = 0, units = 0;
    for (int i = lane; i < a.B; i += 32) {
      const int n = stages_of(a, i);
      units += n;
      if (i < b) before += n;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      units += __shfl_xor_sync(0xffffffffu, units, d);
      before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    units *= a.Hkv;
    const int np = stages_of(a, b);
    const long long u0 = before * a.Hkv + static_cast<long long>(h) * np, u1 = u0 + np;
    if (lane == 0) {
      in.units = units;
      in.c0 = np > 0 ? range_at(units, u0, a.ranges) : 0;
      in.c1 = np > 0 ? range_at(units, u1 - 1, a.ranges) : -1;
      in.first = np > 0 && range_begin(units, in.c0, a.ranges) < u0 ? 1 : 0;
    }
  }
  __syncthreads();
  const int c0 = in.c0, c1 = in.c1, first = in.first;
  const long long units = in.units;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel is complete
  if (c0 == c1) return;                                // written by its only range
  float M = -INFINITY, sum = 0.0f, o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = 0.0f;
  if (row < a.G)
    for (int base = c0; base <= c1; base += 32 * WARPS_A_ROW) {
      const int c = base + lane * WARPS_A_ROW + w0;
      const float* mine = a.ws + (2 * static_cast<size_t>(c) + (c == c0 ? first : 0)) * part_floats(D);
      // (in a list shorter than the ranges some are empty, and leave nothing)
      const unsigned live = __ballot_sync(
          0xffffffffu, c <= c1 && (units >= a.ranges || range_begin(units, c, a.ranges) <
                                                             range_begin(units, c + 1, a.ranges)));
      float x[JOIN_AHEAD][V];
      const auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < JOIN_AHEAD; ++k) {
          const float* acc = reinterpret_cast<const float*>(__shfl_sync(
                                 0xffffffffu, reinterpret_cast<unsigned long long>(mine), k0 + k)) +
                             2 * ROWS + row * D + lane * V;
          const bool some = (live >> (k0 + k) & 1u) && lane < LANES;
          if constexpr (V == 4) {
            const float4 v = some ? *reinterpret_cast<const float4*>(acc) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[k][0] = v.x;
            x[k][1] = v.y;
            x[k][2] = v.z;
            x[k][3] = v.w;
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = some ? acc[e] : 0.0f;
          }
        }
      };
      const float2 ml = (live >> lane & 1u) ? *reinterpret_cast<const float2*>(mine + 2 * row)
                                            : make_float2(-INFINITY, 0.0f);
      load(0);
      float n = fmaxf(M, ml.x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
      const float nb = n == -INFINITY ? 0.0f : n, s = ex2f(M - nb), w = ex2f(ml.x - nb);
      M = n;
      float part_sum = ml.y * w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) part_sum += __shfl_xor_sync(0xffffffffu, part_sum, d);
      sum = sum * s + part_sum;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] *= s;
      for (int k0 = 0;;) {
#pragma unroll
        for (int k = 0; k < JOIN_AHEAD; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k0 + k);  // (0 where there is no part)
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = fmaf(wk, x[k][e], o[e]);
        }
        k0 += JOIN_AHEAD;
        if (k0 >= 32 || live >> k0 == 0u) break;
        load(k0);
      }
    }
  if (lane == 0) state[warp] = make_float2(M, sum);
  if (lane < LANES)
#pragma unroll
    for (int e = 0; e < V; ++e) part_o[warp][lane * V + e] = o[e];
  __syncthreads();
  for (int i = threadIdx.x; i < R * D; i += JOIN_WARPS * 32) {
    const int r = i / D, d = i % D;
    if (row0 + r >= a.G) break;
    const float2* st = state + r * WARPS_A_ROW;
    float top = -INFINITY, total = 0.0f, y = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS_A_ROW; ++k) top = fmaxf(top, st[k].x);
    const float tb = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int k = 0; k < WARPS_A_ROW; ++k) {
      const float wt = ex2f(st[k].x - tb);
      total += wt * st[k].y;
      y += wt * part_o[r * WARPS_A_ROW + k][d];
    }
    const size_t q = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G + row0 + r;
    a.out[q * D + d] = __float2bfloat16_rn(y * inverse_sum(total));
    if (a.lse != nullptr && d == 0) a.lse[q] = lse_of(top, total);
  }
}

template <int D, int R>
int launch_join(const Decode4Args& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hkv * ((a.G + R - 1) / R)));
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, nsa_decode4_join_kernel<D, R>, a) == cudaSuccess ? OK : ERR_LAUNCH;
}

template <int D, int C, bool FEW, bool SELECT>
int launch_pairs(const Decode4Args& a, int cs, cudaStream_t stream) {
  using L = Dec4<D, C, FEW>;
  auto kern = nsa_decode4_pair_kernel<D, C, FEW, SELECT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) != cudaSuccess)
    return ERR_LAUNCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hkv * cs));
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

template <int D, int C, bool FEW>
int launch_select(const Decode4Args& a, cudaStream_t stream) {
  // Blocks of a cluster: as many, of whole slots, as leave each a SM.  More do not pay for their start and their join (512
  // pairs: one block a pair 30 us, two 44, four 54).
  int cs = 1;
  while (cs < 8 && 2 * cs <= a.S && 2LL * a.B * a.Hkv * cs <= sm_count()) cs *= 2;
  return launch_pairs<D, C, FEW, true>(a, cs, stream);
}

template <int D, int C, bool FEW>
int launch_stream(Decode4Args a, cudaStream_t stream) {
  using L = Dec4<D, C, FEW>;
  const int sms = sm_count();
  if (sms < 1) return ERR_DEVICE;
  const long long pairs = static_cast<long long>(a.B) * a.Hkv, most_st = pieces_of(a.max_pages * a.page, STAGE_LOG);
  const long long units = pairs * most_st, places = static_cast<long long>(sms) * L::STREAM_CTAS;
  const long long most = places < DECODE4_MAX_RANGES ? places : DECODE4_MAX_RANGES;
  a.ranges = static_cast<int>(units < most ? units : most);
  // Short tables: a cluster a pair, up to eight blocks that all fit at once, in one launch, while its blocks' longest share
  // (at most 2048 tokens: nothing evens out what sequences differ by) is up to four stages longer than half of a range of
  // full sequences.  (Two kv heads of 128: 4 sequences of up to 1000 tokens 5.5 us, by ranges 7.0, of 4000 both 8.0, of
  // 8000 11.5 and 9.1; 512 of 1000 36.6 and 55.9; 100 with 4 kv heads of 64 of up to 500 6.7 and 14.2.)
  int cs = 1;
  while (cs < 8 && cs < most_st && 2 * pairs * cs <= static_cast<long long>(sms) * L::PAIR_CTAS(false)) cs *= 2;
  if (most_st <= PAIR_STAGES * cs && 2LL * a.ranges * (most_st - 4 * cs) <= units * cs)
    return launch_pairs<D, C, FEW, false>(a, cs, stream);
  // Ranges of one pair each where every pair has ten on average: no block then starts twice, and they differ in length by
  // less than it costs to (four sequences of up to 131072 tokens 29.5 us, of equal ranges 30.4; 16 of 1000 to 5000
  // 11.6 and 13.1).  With eight a pair, 28 sequences of up to 90000: 113 and 105.
  a.pairwise = a.B <= 32 && 10LL * a.B * a.Hkv <= a.ranges;
  auto kern = nsa_decode4_stream_kernel<D, C, FEW>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) != cudaSuccess)
    return ERR_LAUNCH;
  kern<<<static_cast<unsigned>(a.ranges), THREADS, L::BYTES, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  // A block a row while all of them fit at once, else four rows a block (four sequences of up to 131072 tokens, 128 rows:
  // 30.6 us, of four rows a block 33.4; 32 of 32768, 1024 rows: 84.1 and 81.3; 512 of 1024, 16384 rows: 103 and 70).
  return static_cast<long long>(a.B) * a.Hq <= 4LL * sms ? launch_join<D, 1>(a, stream) : launch_join<D, 4>(a, stream);
}

template <int D, bool FEW>
int launch_rows(const Decode4Args& a, cudaStream_t stream) {
  // chunks of 32 tokens (half the work for masks and maxima per token) where a page holds them
  if (a.block_idx == nullptr)
    return a.page >= 32 ? launch_stream<D, 32, FEW>(a, stream) : launch_stream<D, 16, FEW>(a, stream);
  return a.page >= 32 ? launch_select<D, 32, FEW>(a, stream) : launch_select<D, 16, FEW>(a, stream);
}
// Eight query rows a kv head or fewer have products of their own (32 query and 4 kv heads of 128, 16 sequences of 20000 to
// 60000 tokens: 70 us, by the form for sixteen 88; 512 on 16 pages each: 60.5 and 76.5; heads of 64: 47.7 and 57.9).
template <int D>
int launch_decode4(const Decode4Args& a, cudaStream_t stream) {
  return a.G <= 8 ? launch_rows<D, true>(a, stream) : launch_rows<D, false>(a, stream);
}

}  // namespace

// The partials of the most ranges (the size does not depend on the device); selected pages leave none.
size_t nsa_decode4_workspace_bytes(int D, int S) {
  return S > 0 ? 256 : 2 * static_cast<size_t>(DECODE4_MAX_RANGES) * part_floats(D) * sizeof(float);
}

int launch_nsa_decode4(const Cache4& c, const void* q, const int32_t* lens, const int32_t* block_idx, void* out,
                       float* lse, int Hq, int S, void* workspace, cudaStream_t stream) {
  Decode4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = c.k; a.v = c.v; a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.k_factor = c.k_factor; a.v_factor = c.v_factor;
  a.table = c.table; a.lens = lens; a.block_idx = block_idx;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws = static_cast<float*>(workspace);
  a.B = c.B; a.Hq = Hq; a.Hkv = c.Hkv; a.G = Hq / c.Hkv; a.page = c.page;
  a.max_pages = c.max_pages; a.num_pages = c.num_pages; a.S = block_idx != nullptr ? S : 0;
  a.scale_log2 = LOG2E / sqrtf(static_cast<float>(c.D));
  switch (c.D) {
    case 16: return launch_decode4<16>(a, stream);
    case 32: return launch_decode4<32>(a, stream);
    case 64: return launch_decode4<64>(a, stream);
    case 128: return launch_decode4<128>(a, stream);
    default: return ERR_UNSUPPORTED;
  }
}

unsigned int nsa_decode4_device_error() { return read_and_clear_device_error(); }

}  // namespace bsa
