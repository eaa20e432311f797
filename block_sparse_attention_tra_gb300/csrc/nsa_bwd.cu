// nsa_bwd.cu -- gradients of the NSA selection attention (bf16 in and out,
// fp32 sums).
//
// With s = D^-0.5, J_i the tokens j <= i of the blocks that row i selects (a
// set), and the forward's out and lse, for query head h of kv head h / G:
//     p_ij  = exp(s q_i . k_j - lse_i)             (recomputed, not stored)
//     dP_ij = dout_i . v_j,    delta_i = dout_i . out_i
//     dS_ij = s p_ij (dP_ij - delta_i)
//     dq_i = sum_{j in J_i} dS_ij k_j
//     dk_j = sum_{i: j in J_i} sum_{h of the group} dS_ij q_i,   dv_j = the same of p_ij dout_i
// A row that selects nothing has no pair: dq 0, nothing for dk and dv.
//
// Launches, all on the caller's stream, scratch in the caller's workspace:
//   1. mark    per 128 query rows: how many of them select each block
//   2. prefix  per block: where each 128 rows' share of its list starts
//   3. scan    where each block's list starts; lists cut into work items
//   4. fill    the lists: for each block the queries that select it, ascending
// then, for 64 and 128 dims (nsa_bwd_tc.cu, on tcgen05),
//   5. pack    Q and dO by query; (lse, delta) of every row
//   6. tc      one work item at a time: a block's keys and values stay, its
//              queries stream past; every slot's row of dq, the items' dk, dv
//   7. dq sum  the slots' rows, in slot order
// and for 16 and 32 dims (mma.sync)
//   5. dq      one query group at a time, gathering its blocks' keys and
//              values; leaves (lse, delta) of its rows for 6
//   6. dkdv    one work item at a time: a block's keys and values stay in
//              registers, the items' query rows stream past
// and last, for blocks cut into several items,
//   8. join    the items' sums, in order
// The order of every sum is fixed (lists are ranked with bit masks, not with
// atomic cursors), so results repeat bit for bit.
//
// dq and dkdv each form the scores: 14 instead of 10 D flops per pair, for no
// atomic additions and no rows of dq in memory.  The tcgen05 pass forms them
// once and writes a row of dq per slot.  The whole call on 4096 tokens, 32
// heads of 128 in groups of 16, with 1024 tokens selected in blocks of 128, 64
// and 32 (512 in blocks of 16): 865, 1040, 1167 and 1260 us by kernels of the
// mma.sync kind, 399, 374, 681 and 668 by the tcgen05 pass.  The pass is built
// for 64 and 128 dims.  The mma.sync kernels, which serve 16 and 32, take 271
// and 324 us there (64-token blocks) where the pass takes 243 for 64 dims:
// rows filled up to 64 columns with zeros would be the faster form of 32 at
// these sizes, and are not built.
//
// Where the sizes are small every step is a few microseconds of latency (256
// tokens of 8 heads of 32: 23 us of kernels in the 45 us that seven launches
// and the call cost).  Mark and fill, four threads a row, take 3 and 5 us for
// 4096 tokens of 16 slots (one a row: 3 and 12).
#include <algorithm>

#include "kernels.h"
#include "mma_sync.cuh"
#include "nsa_bwd.cuh"
#include "nsa_slots.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int QCHUNK = 128;      // query rows of one mark / fill block
constexpr int MASKS = QCHUNK / 32;
constexpr int SLOT_PARTS = 4;    // threads of a row there, each with every fourth slot
constexpr int LIST_THREADS = QCHUNK * SLOT_PARTS;
constexpr int BLK_TILE = 2048;   // blocks whose masks a mark / fill block holds

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes = 16u) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------ inverted lists

// Bit q of mask[blk - blk0] for every row q of this block's 128 that selects
// blk: the live rule of nsa_slots.cuh (a repeated block sets the same bit).
__device__ __forceinline__ void mark_rows(uint32_t (*mask)[MASKS], const int32_t* __restrict__ block_idx, long long bh,
                                          int T, int S, int n_blk, int bs, int blk0, int nb) {
  for (int e = threadIdx.x; e < nb * MASKS; e += LIST_THREADS) mask[e / MASKS][e % MASKS] = 0u;
  __syncthreads();
  const int q = threadIdx.x / SLOT_PARTS, i = blockIdx.x * QCHUNK + q;
  if (i < T) {
    const int32_t* row = block_idx + (bh * T + i) * S;
#pragma unroll 4
    for (int s = threadIdx.x % SLOT_PARTS; s < S; s += SLOT_PARTS) {
      const int blk = row[s];
      if (blk >= blk0 && blk < blk0 + nb && blk < n_blk && blk * bs <= i)
        atomicOr(&mask[blk - blk0][q >> 5], 1u << (q & 31));
    }
  }
  __syncthreads();
}

// grid (chunks of 128 rows, B * Hkv, tiles of blocks).  counts[bh][chunk][blk].
__global__ void __launch_bounds__(LIST_THREADS) bwd_mark_kernel(const int32_t* __restrict__ block_idx,
                                                                int* __restrict__ counts, int T, int S, int n_blk,
                                                                int bs) {
  extern __shared__ uint32_t mask_raw[];
  uint32_t(*mask)[MASKS] = reinterpret_cast<uint32_t(*)[MASKS]>(mask_raw);
  const int blk0 = blockIdx.z * BLK_TILE, nb = min(BLK_TILE, n_blk - blk0);
  const long long bh = blockIdx.y;
  mark_rows(mask, block_idx, bh, T, S, n_blk, bs, blk0, nb);
  int* dst = counts + (bh * gridDim.x + blockIdx.x) * n_blk + blk0;
  for (int e = threadIdx.x; e < nb; e += LIST_THREADS) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < MASKS; ++w) c += __popc(mask[e][w]);
    dst[e] = c;
  }
}

// grid (tiles of 32 blocks, B * Hkv), block (32 blocks, 32 parts of the
// chunks): counts[bh][chunk][blk] becomes the number of earlier queries in
// the block's list, total[bh][blk] its length.
__global__ void __launch_bounds__(1024) bwd_prefix_kernel(int* __restrict__ counts, int* __restrict__ total,
                                                          int chunks, int n_blk) {
  __shared__ int part[32][33];
  const int blk = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  const int per = (chunks + 31) / 32;
  const int c0 = min(chunks, y * per), c1 = min(chunks, c0 + per);
  int* col = counts + static_cast<long long>(blockIdx.y) * chunks * n_blk + blk;
  int n = 0;
  if (blk < n_blk)
    for (int c = c0; c < c1; ++c) n += col[static_cast<long long>(c) * n_blk];
  part[y][threadIdx.x] = n;
  __syncthreads();
  if (y == 0) {
    int sum = 0;
    for (int w = 0; w < 32; ++w) {
      const int x = part[w][threadIdx.x];
      part[w][threadIdx.x] = sum;
      sum += x;
    }
    if (blk < n_blk) total[static_cast<long long>(blockIdx.y) * n_blk + blk] = sum;
  }
  __syncthreads();
  if (blk >= n_blk) return;
  n = part[y][threadIdx.x];
  for (int c = c0; c < c1; ++c) {
    const int x = col[static_cast<long long>(c) * n_blk];
    col[static_cast<long long>(c) * n_blk] = n;
    n += x;
  }
}

// One block: total[NB] -> off[NB] (where each list starts), item_off[NB + 1]
// (first work item of each block) and the items {block, first list entry,
// queries, items of its block}.
constexpr int SCAN_THREADS = 1024;
__global__ void __launch_bounds__(SCAN_THREADS) bwd_scan_kernel(const int* __restrict__ total, int* __restrict__ off,
                                                                int* __restrict__ item_off, int4* __restrict__ items,
                                                                int NB, int item_queries) {
  __shared__ int wp[32], wi[32];
  const int per = (NB + SCAN_THREADS - 1) / SCAN_THREADS;
  const int lo = min(NB, static_cast<int>(threadIdx.x) * per), hi = min(NB, lo + per);
  int np = 0, ni = 0;
  for (int e = lo; e < hi; ++e) {
    np += total[e];
    ni += (total[e] + item_queries - 1) / item_queries;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sp = np, si = ni;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sp, d), b = __shfl_up_sync(0xffffffffu, si, d);
    if (lane >= d) { sp += a; si += b; }
  }
  if (lane == 31) { wp[warp] = sp; wi[warp] = si; }
  __syncthreads();
  if (warp == 0) {
    int a = wp[lane], b = wi[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
      if (lane >= d) { a += x; b += y; }
    }
    wp[lane] = a;
    wi[lane] = b;
  }
  __syncthreads();
  int pb = sp - np + (warp > 0 ? wp[warp - 1] : 0), ib = si - ni + (warp > 0 ? wi[warp - 1] : 0);
  for (int e = lo; e < hi; ++e) {
    const int c = total[e], k = (c + item_queries - 1) / item_queries;
    off[e] = pb;
    item_off[e] = ib;
    // equal shares, so that no item of a block is a short rest
    const int share = k > 0 ? (c + k - 1) / k : 0;
    for (int s = 0; s < k; ++s) items[ib++] = make_int4(e, pb + s * share, min(share, c - s * share), k);
    pb += c;
  }
  if (threadIdx.x == SCAN_THREADS - 1) item_off[NB] = ib;
}

// grid as mark: query i goes to place (start of the block's list) + (queries
// of earlier chunks) + (its rank in the chunk's mask).
__global__ void __launch_bounds__(LIST_THREADS) bwd_fill_kernel(const int32_t* __restrict__ block_idx,
                                                                const int* __restrict__ counts,
                                                                const int* __restrict__ off, int* __restrict__ list,
                                                                int T, int S, int n_blk, int bs) {
  extern __shared__ uint32_t mask_raw[];
  uint32_t(*mask)[MASKS] = reinterpret_cast<uint32_t(*)[MASKS]>(mask_raw);
  const int blk0 = blockIdx.z * BLK_TILE, nb = min(BLK_TILE, n_blk - blk0);
  const long long bh = blockIdx.y;
  mark_rows(mask, block_idx, bh, T, S, n_blk, bs, blk0, nb);
  const int q = threadIdx.x / SLOT_PARTS, i = blockIdx.x * QCHUNK + q;
  if (i >= T) return;
  const int32_t* row = block_idx + (bh * T + i) * S;
  const int* before = counts + (bh * gridDim.x + blockIdx.x) * n_blk;
  const int w = q >> 5;
  const uint32_t below = (1u << (q & 31)) - 1u;
  for (int s = threadIdx.x % SLOT_PARTS; s < S; s += SLOT_PARTS) {
    const int blk = row[s];
    if (blk < blk0 || blk >= blk0 + nb || blk >= n_blk || blk * bs > i) continue;
    bool again = false;  // a repeated block counts in its first slot
    for (int x = 0; x < s; ++x) again |= row[x] == blk;
    if (again) continue;
    const uint32_t* m = mask[blk - blk0];
    int rank = __popc(m[w] & below);
    for (int x = 0; x < w; ++x) rank += __popc(m[x]);
    list[off[bh * n_blk + blk] + before[blk] + rank] = i * 32 + s;
  }
}

// ------------------------------------------------------------------------ dq

// The 16-token chunks of one query's live blocks, in slot order (every lane
// of the warp steps it alike).
struct ChunkIter {
  SlotRow row;
  int i, bs, s, c, nc, tok0;
  bool valid;

  __device__ __forceinline__ void seek_slot() {
    const uint32_t rest = s < 32 ? row.live & ~((1u << s) - 1u) : 0u;
    valid = rest != 0u;
    if (valid) {
      s = __ffs(rest) - 1;
      tok0 = nsa_slot_block(row, s) * bs;
      nc = (min(tok0 + bs - 1, i) - tok0) / 16 + 1;
      c = 0;
    }
  }
  __device__ __forceinline__ void step() {
    if (++c < nc) {
      tok0 += 16;
    } else {
      ++s;
      seek_slot();
    }
  }
};

constexpr int DQ_WARPS = 4;
constexpr int DQ_THREADS = DQ_WARPS * 32;
constexpr int DQ_CTAS = 5;  // blocks of a SM

template <int D>
struct DqLayout {
  static constexpr int RB = (D + 8) * 2;        // padded row, bytes
  static constexpr int Q_BYTES = 16 * RB;       // 16 rows
  static constexpr int STAGE = 2 * 16 * RB;     // K rows, then V rows, of one chunk
  static constexpr int WARP_BYTES = 2 * STAGE;  // the query and dout rows pass through the stages first
  static constexpr int BYTES = DQ_WARPS * WARP_BYTES;
};

// One warp per query group (persistent grid), K and V chunks through its own
// double-buffered shared memory.
template <int D>
__global__ void __launch_bounds__(DQ_THREADS, DQ_CTAS)
    nsa_bwd_dq_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                      const __nv_bfloat16* __restrict__ v, const int32_t* __restrict__ block_idx,
                      const __nv_bfloat16* __restrict__ out, const float* __restrict__ lse,
                      const __nv_bfloat16* __restrict__ dout, __nv_bfloat16* __restrict__ dq,
                      float2* __restrict__ stats, int G, int T, int S, int bs, long long n_queries,
                      float scale) {
  using L = DqLayout<D>;
  constexpr int CPR = D / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3, mat = lane >> 3, mrow = lane & 7;
  const int n_blk = T / bs;
  const uint32_t sKV = smem_u32(smem + warp * L::WARP_BYTES);
  const float scale_log2 = scale * NSA_LOG2E;

  const long long stride = static_cast<long long>(gridDim.x) * DQ_WARPS;
  for (long long qg = static_cast<long long>(blockIdx.x) * DQ_WARPS + warp; qg < n_queries; qg += stride) {
    const int i = static_cast<int>(qg % T);
    const long long bg = qg / T;  // b * Hkv + hkv; its heads are rows bg * G .. of [B * Hq]
    const __nv_bfloat16* kb = k + static_cast<size_t>(bg) * T * D;
    const __nv_bfloat16* vb = v + static_cast<size_t>(bg) * T * D;

    // ---- query and dout rows through shared memory into fragments; delta from dout and out
    uint32_t qa[D / 16][4], da[D / 16][4];
    float delta0 = 0.0f, delta1 = 0.0f, lse0, lse1;
    {
      for (int e = lane; e < 16 * CPR; e += 32) {
        const int r = e / CPR, c = e % CPR;
        const size_t off = ((static_cast<size_t>(bg) * G + min(r, G - 1)) * T + i) * D + c * 8;
        cp_async16(sKV + r * L::RB + c * 16, q + off, r < G ? 16u : 0u);
        cp_async16(sKV + L::Q_BYTES + r * L::RB + c * 16, dout + off, r < G ? 16u : 0u);
        cp_async16(sKV + 2 * L::Q_BYTES + r * L::RB + c * 16, out + off, r < G ? 16u : 0u);
      }
      cp_async_commit();
      const size_t lr = static_cast<size_t>(bg) * G * T + i;
      lse0 = g < G ? lse[lr + static_cast<size_t>(g) * T] : 0.0f;
      lse1 = g + 8 < G ? lse[lr + static_cast<size_t>(g + 8) * T] : 0.0f;
      cp_async_wait<0>();
      __syncwarp();
      const uint32_t a = sKV + (mrow + 8 * (mat & 1)) * L::RB + (8 * (mat >> 1)) * 2;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        ldsm_x4(a + ks * 32, qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3]);
        ldsm_x4(a + L::Q_BYTES + ks * 32, da[ks][0], da[ks][1], da[ks][2], da[ks][3]);
        uint32_t oa[4];
        ldsm_x4(a + 2 * L::Q_BYTES + ks * 32, oa[0], oa[1], oa[2], oa[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __uint_as_float(da[ks][e] << 16) * __uint_as_float(oa[e] << 16) +
                          __uint_as_float(da[ks][e] & 0xffff0000u) * __uint_as_float(oa[e] & 0xffff0000u);
          if (e & 1) delta1 += x;
          else delta0 += x;
        }
      }
      delta0 += __shfl_xor_sync(0xffffffffu, delta0, 1);
      delta0 += __shfl_xor_sync(0xffffffffu, delta0, 2);
      delta1 += __shfl_xor_sync(0xffffffffu, delta1, 1);
      delta1 += __shfl_xor_sync(0xffffffffu, delta1, 2);
      lse0 *= NSA_LOG2E;
      lse1 *= NSA_LOG2E;
      if (t == 0) {
        if (g < G) stats[qg * G + g] = make_float2(lse0, delta0);
        if (g + 8 < G) stats[qg * G + g + 8] = make_float2(lse1, delta1);
      }
      __syncwarp();
    }

    auto load_chunk = [&](int tok0, int buf) {
      const uint32_t dk = sKV + buf * L::STAGE, dv = dk + 16 * L::RB;
      for (int e = lane; e < 16 * CPR; e += 32) {
        const int r = e / CPR, c = e % CPR;
        const size_t off = static_cast<size_t>(debug_index(tok0 + r, 0, T)) * D + c * 8;
        // (dS of the keys that the mask hides is 0; what they hold may not be a number)
        cp_async16(dk + r * L::RB + c * 16, kb + off, tok0 + r <= i ? 16u : 0u);
        cp_async16(dv + r * L::RB + c * 16, vb + off);
      }
    };
    ChunkIter cur{nsa_live_slots(block_idx + qg * S, S, i, n_blk, bs), i, bs, 0, 0, 0, 0, false};
    cur.seek_slot();
    ChunkIter pf = cur;
    if (pf.valid) {
      load_chunk(pf.tok0, 0);
      pf.step();
    }
    cp_async_commit();

    float acc[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;

    for (int it = 0; cur.valid; ++it) {
      if (pf.valid) {
        load_chunk(pf.tok0, (it + 1) & 1);
        pf.step();
      }
      cp_async_commit();
      cp_async_wait<1>();
      __syncwarp();
      const uint32_t sK = sKV + (it & 1) * L::STAGE, sV = sK + 16 * L::RB;
      const int tok0 = cur.tok0;
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float dp[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const uint32_t rowb = (8 * (mat >> 1) + mrow) * L::RB + 8 * (mat & 1) * 2;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t b00, b01, b10, b11;
        ldsm_x4(sK + rowb + ks * 32, b00, b01, b10, b11);
        mma16816(sc[0], qa[ks], b00, b01);
        mma16816(sc[1], qa[ks], b10, b11);
        ldsm_x4(sV + rowb + ks * 32, b00, b01, b10, b11);
        mma16816(dp[0], da[ks], b00, b01);
        mma16816(dp[1], da[ks], b10, b11);
      }
      // dS, rounded to bf16 as the tensor cores' operand
      uint32_t pa[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float ds[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = ex2f(fmaf(sc[j][e], scale_log2, -(e < 2 ? lse0 : lse1)));
          const float x = p * (dp[j][e] - (e < 2 ? delta0 : delta1)) * scale;
          ds[e] = tok0 + 8 * j + 2 * t + (e & 1) <= i ? x : 0.0f;
        }
        pa[2 * j] = pack_bf16x2(ds[0], ds[1]);
        pa[2 * j + 1] = pack_bf16x2(ds[2], ds[3]);
      }
      const uint32_t rowt = (8 * (mat & 1) + mrow) * L::RB + 8 * (mat >> 1) * 2;
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(sK + rowt + jj * 32, b0, b1, b2, b3);
        mma16816(acc[2 * jj], pa, b0, b1);
        mma16816(acc[2 * jj + 1], pa, b2, b3);
      }
      __syncwarp();
      cur.step();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = g + 8 * half;
      if (row < G) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(dq + ((static_cast<size_t>(bg) * G + row) * T + i) * D);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) dst[4 * j + t] = pack_bf16x2(acc[j][2 * half], acc[j][2 * half + 1]);
      }
    }
    __syncwarp();
  }
}

// --------------------------------------------------------------------- dk, dv

template <int D>
struct KvLayout {
  static constexpr int NS = 3;             // stages
  static constexpr int RB = (D + 8) * 2;   // padded row, bytes
  static constexpr int TILE = 16 * RB;     // 16 rows of q or dout
  static constexpr int STAGE = 2 * TILE + 16 * 8 + 16 * 4;  // q, dout, (lse, delta), query index
  static constexpr int BYTES = NS * STAGE;
};

// One block per work item, a warp for every 16 tokens of the key block; the
// item's queries in tiles of 16 rows = 16 / G queries x G heads.
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    nsa_bwd_dkdv_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                        const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ dout,
                        const float2* __restrict__ stats, const int* __restrict__ list,
                        const int4* __restrict__ items, const int* __restrict__ n_items, float* __restrict__ part,
                        __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, int G, int T, int n_blk,
                        float scale) {
  using L = KvLayout<D>;
  constexpr int CPR = D / 8, BS = WARPS * 16, NTH = WARPS * 32;
  if (static_cast<int>(blockIdx.x) >= *n_items) return;  // fewer items than the launch bound
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3, mat = lane >> 3, mrow = lane & 7;
  const int4 item = items[blockIdx.x];
  const int blk = item.x % n_blk;
  const long long bg = item.x / n_blk;
  const int first = item.y, nq = item.z;
  const int qpt = 16 / G, nt = (nq + qpt - 1) / qpt;
  const float scale_log2 = scale * NSA_LOG2E;
  const int tok0 = blk * BS + warp * 16;  // this warp's tokens

  // A fragments of this warp's 16 key and value rows
  uint32_t ka[D / 16][4], va[D / 16][4];
  {
    const size_t r0 = (static_cast<size_t>(bg) * T + tok0 + g) * D + 2 * t, r8 = r0 + 8 * D;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      ka[ks][0] = *reinterpret_cast<const uint32_t*>(k + r0 + 16 * ks);
      ka[ks][1] = *reinterpret_cast<const uint32_t*>(k + r8 + 16 * ks);
      ka[ks][2] = *reinterpret_cast<const uint32_t*>(k + r0 + 16 * ks + 8);
      ka[ks][3] = *reinterpret_cast<const uint32_t*>(k + r8 + 16 * ks + 8);
      va[ks][0] = *reinterpret_cast<const uint32_t*>(v + r0 + 16 * ks);
      va[ks][1] = *reinterpret_cast<const uint32_t*>(v + r8 + 16 * ks);
      va[ks][2] = *reinterpret_cast<const uint32_t*>(v + r0 + 16 * ks + 8);
      va[ks][3] = *reinterpret_cast<const uint32_t*>(v + r8 + 16 * ks + 8);
    }
  }

  auto load_tile = [&](int x) {  // tile x of the item into stage x % NS (nothing past the last)
    if (x < nt) {
      const uint32_t st = sm + (x % L::NS) * L::STAGE;
      for (int e = threadIdx.x; e < 16 * CPR; e += NTH) {
        const int r = e / CPR, c = e % CPR;
        const int slot = x * qpt + r / G;
        const bool in = r < qpt * G && slot < nq;
        const int i = in ? debug_index(list[first + slot] >> 5, 0, T) : 0;
        const size_t off = ((static_cast<size_t>(bg) * G + (in ? r % G : 0)) * T + i) * D + c * 8;
        cp_async16(st + r * L::RB + c * 16, q + off, in ? 16u : 0u);
        cp_async16(st + L::TILE + r * L::RB + c * 16, dout + off, in ? 16u : 0u);
        if (c == 0) {
          cp_async8(st + 2 * L::TILE + r * 8, stats + (bg * T + i) * G + (in ? r % G : 0), in ? 8u : 0u);
          // -1: a row of no query, causally before every token
          *reinterpret_cast<int*>(smem + (x % L::NS) * L::STAGE + 2 * L::TILE + 128 + r * 4) = in ? i : -1;
        }
      }
    }
    cp_async_commit();
  };

  float dka[D / 8][4], dva[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) dka[j][e] = dva[j][e] = 0.0f;

#pragma unroll
  for (int x = 0; x < L::NS - 1; ++x) load_tile(x);
  for (int x = 0; x < nt; ++x) {
    cp_async_wait<L::NS - 2>();
    __syncthreads();  // tile x has landed for everyone; everyone is done with tile x - 1
    load_tile(x + L::NS - 1);
    const uint32_t sQ = sm + (x % L::NS) * L::STAGE, sDO = sQ + L::TILE;
    const uint8_t* meta = smem + (x % L::NS) * L::STAGE + 2 * L::TILE;
    // S^T and dP^T: 16 tokens x 16 rows
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    float dp[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const uint32_t rowb = (8 * (mat >> 1) + mrow) * L::RB + 8 * (mat & 1) * 2;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b00, b01, b10, b11;
      ldsm_x4(sQ + rowb + ks * 32, b00, b01, b10, b11);
      mma16816(sc[0], ka[ks], b00, b01);
      mma16816(sc[1], ka[ks], b10, b11);
      ldsm_x4(sDO + rowb + ks * 32, b00, b01, b10, b11);
      mma16816(dp[0], va[ks], b00, b01);
      mma16816(dp[1], va[ks], b10, b11);
    }
    uint32_t pa[4], sa[4];  // P^T and dS^T, rounded to bf16 as the tensor cores' operands
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float p[4], ds[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // columns (rows of q) 8j + 2t + c
        const int col = 8 * j + 2 * t + c;
        const float2 ld = *reinterpret_cast<const float2*>(meta + col * 8);
        const int i = *reinterpret_cast<const int*>(meta + 128 + col * 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // tokens g and g + 8
          const int e = 2 * h + c;
          const bool in = tok0 + g + 8 * h <= i;
          p[e] = in ? ex2f(fmaf(sc[j][e], scale_log2, -ld.x)) : 0.0f;
          ds[e] = in ? p[e] * (dp[j][e] - ld.y) * scale : 0.0f;
        }
      }
      pa[2 * j] = pack_bf16x2(p[0], p[1]);
      pa[2 * j + 1] = pack_bf16x2(p[2], p[3]);
      sa[2 * j] = pack_bf16x2(ds[0], ds[1]);
      sa[2 * j + 1] = pack_bf16x2(ds[2], ds[3]);
    }
    const uint32_t rowt = (8 * (mat & 1) + mrow) * L::RB + 8 * (mat >> 1) * 2;
#pragma unroll
    for (int jj = 0; jj < D / 16; ++jj) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(sDO + rowt + jj * 32, b0, b1, b2, b3);
      mma16816(dva[2 * jj], pa, b0, b1);
      mma16816(dva[2 * jj + 1], pa, b2, b3);
      ldsm_x4_t(sQ + rowt + jj * 32, b0, b1, b2, b3);
      mma16816(dka[2 * jj], sa, b0, b1);
      mma16816(dka[2 * jj + 1], sa, b2, b3);
    }
  }
  cp_async_wait<0>();

  if (item.w == 1) {  // the block's only item
    const size_t r0 = (static_cast<size_t>(bg) * T + tok0 + g) * D + 2 * t, r8 = r0 + 8 * D;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      *reinterpret_cast<uint32_t*>(dk + r0 + 8 * j) = pack_bf16x2(dka[j][0], dka[j][1]);
      *reinterpret_cast<uint32_t*>(dk + r8 + 8 * j) = pack_bf16x2(dka[j][2], dka[j][3]);
      *reinterpret_cast<uint32_t*>(dv + r0 + 8 * j) = pack_bf16x2(dva[j][0], dva[j][1]);
      *reinterpret_cast<uint32_t*>(dv + r8 + 8 * j) = pack_bf16x2(dva[j][2], dva[j][3]);
    }
  } else {  // part[item][dk, dv][token][D]
    float* p0 = part + static_cast<size_t>(blockIdx.x) * 2 * BS * D + (warp * 16 + g) * D + 2 * t;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      *reinterpret_cast<float2*>(p0 + 8 * j) = make_float2(dka[j][0], dka[j][1]);
      *reinterpret_cast<float2*>(p0 + 8 * D + 8 * j) = make_float2(dka[j][2], dka[j][3]);
      *reinterpret_cast<float2*>(p0 + BS * D + 8 * j) = make_float2(dva[j][0], dva[j][1]);
      *reinterpret_cast<float2*>(p0 + (BS + 8) * D + 8 * j) = make_float2(dva[j][2], dva[j][3]);
    }
  }
}

// grid (blocks, dk / dv, 1024 elements of the block): sums a block's items in
// order; zeros for a block that no query selects.  A block that every query
// selects has up to a hundred items: with one CTA for all of its elements the
// join took 46 us where 4096 tokens share two kv heads.
__global__ void __launch_bounds__(256) bwd_join_kernel(const float* __restrict__ part,
                                                       const int* __restrict__ item_off,
                                                       __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                                                       int n) {
  const int it0 = item_off[blockIdx.x], k = item_off[blockIdx.x + 1] - it0;
  if (k == 1) return;
  // (blocks of all heads follow each other as their tokens do)
  __nv_bfloat16* dst = (blockIdx.y ? dv : dk) + static_cast<size_t>(blockIdx.x) * n;
  const float* src = part + (static_cast<size_t>(it0) * 2 + blockIdx.y) * n;
  const int e = blockIdx.z * 1024 + threadIdx.x * 4;
  if (e < n) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = 0; x < k; ++x) {
      const float4 y = *reinterpret_cast<const float4*>(src + static_cast<size_t>(x) * 2 * n + e);
      s.x += y.x;
      s.y += y.y;
      s.z += y.z;
      s.w += y.w;
    }
    *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// ------------------------------------------------------------ workspace plan

// Head dims that the tcgen05 pass serves.
constexpr bool tc_dim(int D) { return D >= 64; }

struct BwdPlan {
  long long NB, max_items;
  int chunks, n_blk, item_queries;
  size_t stats_off, list_off, count_off, total_off, off_off, ioff_off, item_off, part_off, rows_off, dqp_off, dqs_off,
      total;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

BwdPlan bwd_plan(int B, int Hq, int Hkv, int T, int D, int bs, int S) {
  BwdPlan p{};
  const long long slots = static_cast<long long>(B) * Hkv * T * S;
  p.n_blk = T / bs;
  p.NB = static_cast<long long>(B) * Hkv * p.n_blk;
  p.chunks = (T + QCHUNK - 1) / QCHUNK;
  // Work items: a few for each of 152 SMs, not so short that the start of one
  // (and its partial result) outweighs its tiles, not so long that the last
  // ones run alone.  tcgen05 pass: three a SM, of 8 to 86 tiles of 96 / G
  // queries (4096 tokens of 16 heads of 64 in groups of four: two a SM 146 us,
  // three 140, four 149, six 155); general kernels: eight a SM, of 32 to 512
  // queries.
  const bool tc = tc_dim(D);
  const int halves = tc && bs == 128 ? 2 : 1;  // (each of them a CTA)
  const long long per_tile = tc ? 96 / (Hq / Hkv) : 1, share = halves * slots / (152 * (tc ? 3 : 8));
  p.item_queries = static_cast<int>(std::max((tc ? 8 : 32) * per_tile, std::min((tc ? 86 : 512) * per_tile, share)));
  p.max_items = (slots + p.item_queries - 1) / p.item_queries + p.NB;
  size_t o = 0;
  p.stats_off = o;  o = align256(o + static_cast<size_t>(B) * Hq * T * sizeof(float2));
  p.list_off = o;   o = align256(o + static_cast<size_t>(slots) * sizeof(int));
  p.count_off = o;  o = align256(o + static_cast<size_t>(p.NB) * p.chunks * sizeof(int));
  p.total_off = o;  o = align256(o + static_cast<size_t>(p.NB) * sizeof(int));
  p.off_off = o;    o = align256(o + static_cast<size_t>(p.NB) * sizeof(int));
  p.ioff_off = o;   o = align256(o + static_cast<size_t>(p.NB + 1) * sizeof(int));
  p.item_off = o;   o = align256(o + static_cast<size_t>(p.max_items) * sizeof(int4));
  p.part_off = o;   o = align256(o + static_cast<size_t>(p.max_items) * 2 * bs * D * sizeof(float));
  p.rows_off = p.dqp_off = p.dqs_off = o;
  if (tc) {
    const size_t rows = static_cast<size_t>(slots) * halves * (Hq / Hkv);
    // (one query of zeros behind the last)
    o = align256(o + (static_cast<size_t>(B) * Hq * T + Hq / Hkv) * 2 * D * sizeof(__nv_bfloat16));
    p.dqp_off = o;
    o = align256(o + rows * D * sizeof(__half));
    p.dqs_off = o;  o = align256(o + rows * sizeof(float));
  }
  p.total = o;
  return p;
}

template <int D, int WARPS>
int launch_dkdv(const NsaBwdArgs& a, const NsaBwdScratch& w, cudaStream_t stream) {
  using L = KvLayout<D>;
  auto kern = nsa_bwd_dkdv_kernel<D, WARPS>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) != cudaSuccess)
    return ERR_LAUNCH;
  kern<<<static_cast<unsigned>(w.max_items), WARPS * 32, L::BYTES, stream>>>(
      a.q, a.k, a.v, a.dout, w.stats, w.list, w.items, w.n_items, w.part, a.dk, a.dv, a.Hq / a.Hkv, a.T, a.T / a.bs,
      1.0f / sqrtf(static_cast<float>(D)));
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

// dq, then dk and dv (or their items' sums), by the general kernels.
template <int D>
int launch_general(const NsaBwdArgs& a, const NsaBwdScratch& w, cudaStream_t stream) {
  using L = DqLayout<D>;
  auto kern = nsa_bwd_dq_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) != cudaSuccess)
    return ERR_LAUNCH;
  const int sms = sm_count();
  if (sms <= 0) return ERR_DEVICE;
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, DQ_THREADS, L::BYTES) != cudaSuccess || per_sm < 1)
    return ERR_LAUNCH;
  const long long nq = static_cast<long long>(a.B) * a.Hkv * a.T;
  const long long need = (nq + DQ_WARPS - 1) / DQ_WARPS, cap = static_cast<long long>(sms) * per_sm;
  kern<<<static_cast<unsigned>(std::min(need, cap)), DQ_THREADS, L::BYTES, stream>>>(
      a.q, a.k, a.v, a.idx, a.out, a.lse, a.dout, a.dq, w.stats, a.Hq / a.Hkv, a.T, a.S, a.bs, nq,
      1.0f / sqrtf(static_cast<float>(D)));
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  switch (a.bs) {
    case 16: return launch_dkdv<D, 1>(a, w, stream);
    case 32: return launch_dkdv<D, 2>(a, w, stream);
    case 64: return launch_dkdv<D, 4>(a, w, stream);
    case 128: return launch_dkdv<D, 8>(a, w, stream);
    default: return ERR_UNSUPPORTED;
  }
}

template <int D>
int launch_bwd(const NsaBwdArgs& a, uint8_t* ws, cudaStream_t stream) {
  const BwdPlan p = bwd_plan(a.B, a.Hq, a.Hkv, a.T, D, a.bs, a.S);
  if (p.max_items > 0x3fffffffLL) return ERR_SHAPE;
  int* counts = reinterpret_cast<int*>(ws + p.count_off);
  int* total = reinterpret_cast<int*>(ws + p.total_off);
  int* off = reinterpret_cast<int*>(ws + p.off_off);
  int* ioff = reinterpret_cast<int*>(ws + p.ioff_off);
  NsaBwdScratch w{};
  w.stats = reinterpret_cast<float2*>(ws + p.stats_off);
  w.list = reinterpret_cast<int*>(ws + p.list_off);
  w.items = reinterpret_cast<int4*>(ws + p.item_off);
  w.n_items = ioff + p.NB;
  w.part = reinterpret_cast<float*>(ws + p.part_off);
  w.rows = reinterpret_cast<__nv_bfloat16*>(ws + p.rows_off);
  w.dq_part = reinterpret_cast<__half*>(ws + p.dqp_off);
  w.dq_scale = reinterpret_cast<float*>(ws + p.dqs_off);
  w.max_items = p.max_items;
  const int bh = a.B * a.Hkv;

  const dim3 grid(p.chunks, bh, (p.n_blk + BLK_TILE - 1) / BLK_TILE);
  const size_t mask_bytes = static_cast<size_t>(std::min(p.n_blk, BLK_TILE)) * MASKS * sizeof(uint32_t);
  bwd_mark_kernel<<<grid, LIST_THREADS, mask_bytes, stream>>>(a.idx, counts, a.T, a.S, p.n_blk, a.bs);
  bwd_prefix_kernel<<<dim3((p.n_blk + 31) / 32, bh), dim3(32, 32), 0, stream>>>(counts, total, p.chunks, p.n_blk);
  bwd_scan_kernel<<<1, SCAN_THREADS, 0, stream>>>(total, off, ioff, w.items, static_cast<int>(p.NB), p.item_queries);
  bwd_fill_kernel<<<grid, LIST_THREADS, mask_bytes, stream>>>(a.idx, counts, off, w.list, a.T, a.S, p.n_blk, a.bs);
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;

  int st;
  if constexpr (tc_dim(D)) st = launch_nsa_bwd_tc(a, w, D, stream);
  else st = launch_general<D>(a, w, stream);
  if (st != OK) return st;
  const int elements = a.bs * D;
  bwd_join_kernel<<<dim3(static_cast<unsigned>(p.NB), 2, (elements + 1023) / 1024), 256, 0, stream>>>(
      w.part, ioff, a.dk, a.dv, elements);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace

size_t nsa_bwd_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int block_size, int S) {
  return bwd_plan(B, Hq, Hkv, T, D, block_size, S).total;
}

int launch_nsa_bwd(const void* q, const void* k, const void* v, const int32_t* block_idx, const void* out,
                   const float* lse, const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int T,
                   int D, int block_size, int S, void* workspace, cudaStream_t stream) {
  NsaBwdArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.out = static_cast<const __nv_bfloat16*>(out);
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.idx = block_idx;
  a.lse = lse;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.T = T; a.bs = block_size; a.S = S;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  switch (D) {
    case 16: return launch_bwd<16>(a, ws, stream);
    case 32: return launch_bwd<32>(a, ws, stream);
    case 64: return launch_bwd<64>(a, ws, stream);
    case 128: return launch_bwd<128>(a, ws, stream);
    default: return ERR_UNSUPPORTED;
  }
}

unsigned int nsa_bwd_device_error() { return read_and_clear_device_error(); }

}  // namespace bsa
