// nsa_bwd_tc.cu -- the block-outer pass of the NSA selection attention's
// backward for 64 and 128 dims, on tcgen05.
//
// Formulas as in nsa_bwd.cu.  One CTA per work item (a key block and a share
// of the queries that select it; a block of 128 tokens is two of 64 with the
// same queries); K and V of the block stay in shared memory,
// the queries pass in tiles of 96 rows = 96 / G queries x G heads, gathered by
// bulk copies (G = 8, 16: one of G rows per query and 64-column panel) or by
// cp.async from rows that a first kernel has packed by query.  Per tile, all
// accumulators fp32 in TMEM:
//     S  = Q K^T, dP = dO V^T                [96 rows x 64 keys]
//     P  = exp2(S c log2e - lse2), dS = c P (dP - delta)     (epilogue; to bf16,
//                                   as both operands of an MMA have one type)
//     dV^T += dO^T P, dK^T += Q^T dS         [D x 64 keys]
//     dQ = dS K                              [96 rows x D]
// Every product has 128 rows of A this way (64 keys as M would run the tensor
// cores at half rate): dV and dK are accumulated transposed, the dO and Q
// tiles read MN-major as A, P and dS read MN-major as B and dS once more
// K-major as A of dQ.  At D = 64 dO and Q stand side by side as one 128-row A
// and P and dS as one 128-column B; the two diagonal quarters of the product
// are dV^T and dK^T.
//
// A query's dq is the sum of its blocks' dQ rows.  They leave as f16 under a
// power-of-two factor per row, taken from the bound sum_j |dS_j| max|K| so
// that nothing overflows (an f16 keeps 2^-11 of each element down to 2^-29 of
// the bound): half the bytes of fp32 at an eighth of the final bf16 rounding.
// max|K| is over the keys that a query of the item reads: what lies behind them
// in the block (a padded tail) does not count.  (A bound of every row's own,
// sum_j |dS_j| max|K_j|, took 3 to 10% longer at D = 64 and for blocks of 32
// tokens.)
// A last kernel sums them per query in slot order, so nothing depends on the
// order in which CTAs run.  Adding fp32 rows to dq in L2 instead would move
// twice the bytes through the L2's atomic units and not repeat bit for bit.
//
// The drain threads, one a row, store their rows straight from registers, 32
// bytes (a whole sector) at a time: what a stage for them would take of the
// shared memory is a second buffer of P and dS, without which a tile's
// epilogue could not begin to store before the tile before's products ended.
//
// Tiles have 96 rows, not the 128 an MMA takes: what the stages of Q and dO
// then leave of the shared memory is a third stage, and with two the gathers
// (2 to 4 thousand cycles under load) stood in the way of every tile.  Two
// warps issue MMAs, one the scores' and one the gradients', because issuing
// one costs about what it takes to run.
//
// Bound by shared memory.  With 64 keys on the N side an MMA reads 6 KB of
// operands for 32 cycles of arithmetic (48.5 measured; 65 for N = 128, which
// is both bounds at once).  A tile of D = 128 reads 200 KB, the gather writes
// 48 KB and the epilogue 24 KB: 2140 cycles at 128 bytes a cycle of the 2700
// that it takes.  Two sequences of 8192 tokens, 32 query and 2 kv heads of 128,
// 16 slots: 922 us, 0.68 PFLOP/s at the 10 D flops a (query, key) pair needs,
// besides 102 us to pack (6.6 TB/s) and 345 us to sum dQ (6.6 TB/s).  With one
// buffer of P and dS, and a stage for the dQ rows, the pass took 976 us.
#include <algorithm>

#include "kernels.h"
#include "nsa_bwd.cuh"
#include "nsa_slots.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int BS = 64;     // tokens of a CTA's key tile
constexpr int ROWS = 96;   // rows per tile (queries x heads) of the 128 that an MMA takes
constexpr int GROUP = ROWS / 32;    // warps of one epilogue half, and of the drain
// Warps 0-2 and 4-6 epilogue (left and right 32 keys), 8-10 drain (warp w reads TMEM lanes 32 (w & 3) ..), 7 issues the
// scores' MMAs, 11 or 12 the gradients'; 3 gathers by bulk copies, or 3, the other of 11 and 12, and 13 by cp.async, 32
// rows each.  At D = 64 the gradients' MMAs are issued from the scheduler that has no epilogue warp (2 x 4096 tokens,
// 32 heads in groups of 16: 497 us for the call in place of 511); at D = 128, where an MMA stands longer in the queue
// than it takes to issue, that scheduler is left to the gather and the scores (1416 us in place of 1428).
constexpr int PROD_WARP = 3, MMA_WARP = 7, DRAIN_WARP = 8, PROD3_WARP = 13, WARPS = 14;
template <int D>
constexpr int GRAD_WARP = D == 64 ? 11 : 12;
template <int D>
constexpr int PROD2_WARP = 23 - GRAD_WARP<D>;
template <int D, bool TMA_IN>
constexpr int tc_threads() {
  return (TMA_IN ? GRAD_WARP<D> + 1 : WARPS) * 32;
}
constexpr int PANEL = ROWS * 128;   // 96 rows x 128 bytes
constexpr int KV_PANEL = BS * 128;

template <int D>
struct TcLayout {
  static constexpr int NP = D / 64;
  static constexpr int NS = D == 128 ? 3 : 6;    // stages of dO and Q
  static constexpr int TILE = NP * PANEL;        // 96 rows x D
  static constexpr int KV_TILE = NP * KV_PANEL;
  static constexpr int STAGE = 2 * TILE;         // dO, then Q
  static constexpr int P_OFF = NS * STAGE;       // two buffers of P, then dS: 96 rows x 64 keys bf16
  static constexpr int DS_OFF = P_OFF + PANEL;
  static constexpr int PDS = 2 * PANEL;          // bytes of a buffer
  static constexpr int K_OFF = P_OFF + 2 * PDS, V_OFF = K_OFF + KV_TILE;
  static constexpr int SUM_OFF = V_OFF + KV_TILE;  // float[2 tiles][2 halves][96]: sums of |dS|
  static constexpr int KMAX_OFF = SUM_OFF + 4 * ROWS * 4;  // float[8]
  static constexpr int BAR_OFF = KMAX_OFF + 8 * 4;
  // kv_full | dq_full | dq_empty | acc_full | pds_ready[2] | pds_free[2] | sp_full[2] | sum_full[2] | sum_free[2] |
  // sp_empty[2] | mma_done[2] | q_full[NS] | q_empty[NS] | do_full[NS] | do_empty[NS]
  static constexpr int NBAR = 18 + 4 * NS;
  static constexpr int TPTR_OFF = BAR_OFF + NBAR * 8;
  static constexpr int ALLOC = TPTR_OFF + 16 + 1024;
  static_assert(ALLOC <= 232448, "shared memory");
  // An MMA reads 128 rows of A: the 32 behind a tile's last lie in what follows it, and their results are not read.
  static_assert(128 * 128 - PANEL <= PDS && 128 * 128 - PANEL <= 2 * KV_TILE, "rows behind the last tile");
  // TMEM columns: S[2], dP[2], dV^T, dK^T, dQ
  static constexpr uint32_t TS = 0, TP = 128, TV = 256, TK = 320, TQ = 384;
  static constexpr uint32_t TMEM_COLS = 512;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// 32 bytes of an f16 row.  The lines are the first to leave L2: the rows are
// read once, by a later kernel, while the packed rows are read S times.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The MMA issuer's operands as the low words of 128-byte-swizzle descriptors
// (start address and leading byte offset, both >> 4): the high word (stride
// 1024 bytes, version, swizzle) is the same for all of them, and a step along
// K adds a constant, where building each descriptor anew kept the issuer at
// one MMA per ~110 cycles, twice what the tensor cores take.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return (saddr >> 4) | ((lbo_bytes >> 4) << 16);
}
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
      : "memory");
}

// One of the item's queries: list entry -> query index and slot.
struct Pair {
  int i, s;
  bool valid;
};

// KEYS: tokens of the CTA's key block, 64, 32 or 16.  Below 64 the products are narrower (N = KEYS, and K = KEYS for
// dQ); of the 64-key tiles only that part is read (at D = 64 zeros behind it), and half of the epilogue has only zeros
// to write.  An MMA then reads the same A for less arithmetic: a tile takes about as long, for half or a quarter of
// the keys.
template <int D, int KEYS, bool TMA_IN>
__global__ void __launch_bounds__(tc_threads<D, TMA_IN>(), 1)
    nsa_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __nv_bfloat16* __restrict__ rows, const float2* __restrict__ stats,
                      const int* __restrict__ list, const int4* __restrict__ items,
                      const int* __restrict__ n_items, float* __restrict__ part, __half* __restrict__ dq_part,
                      float* __restrict__ dq_scale, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                      int G, int T, int S, int n_blk, int n_bh, int two, float scale) {
  using L = TcLayout<D>;
  // two = 1: selected blocks of 128 tokens, an item's two halves beside one another
  const int item_no = static_cast<int>(blockIdx.x) >> two, half = static_cast<int>(blockIdx.x) & two;
  if (item_no >= *n_items) return;  // fewer items than the launch bound
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t *kv_full = bars, *dq_full = bars + 1, *dq_empty = bars + 2, *acc_full = bars + 3, *pds_ready = bars + 4,
           *pds_free = bars + 6, *sp_full = bars + 8, *sum_full = bars + 10, *sum_free = bars + 12,
           *sp_empty = bars + 14, *mma_done = bars + 16, *q_full = bars + 18, *q_empty = q_full + L::NS,
           *do_full = q_empty + L::NS, *do_empty = do_full + L::NS;
  uint32_t* tptr = reinterpret_cast<uint32_t*>(smem + L::TPTR_OFF);
  float* sums = reinterpret_cast<float*>(smem + L::SUM_OFF);
  float* km = reinterpret_cast<float*>(smem + L::KMAX_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 item = items[item_no];
  const int bg = item.x / n_blk, key0 = ((item.x % n_blk << two) + half) * KEYS;  // the first key's token
  const int first = item.y, npairs = item.z;
  const int qpt = ROWS / G;                    // queries per tile
  const int nt = (npairs + qpt - 1) / qpt;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int x = 0; x < L::NS; ++x) {
      mbar_init(&q_full[x], TMA_IN ? 1 : 3 * 32);
      mbar_init(&q_empty[x], 1);
      mbar_init(&do_full[x], TMA_IN ? 1 : 3 * 32);
      mbar_init(&do_empty[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sp_full[x], 1);
      mbar_init(&mma_done[x], 1);
      mbar_init(&sum_full[x], 2 * GROUP);
      mbar_init(&sum_free[x], GROUP);
      mbar_init(&sp_empty[x], 2 * GROUP);
      mbar_init(&pds_ready[x], 2 * GROUP);
      mbar_init(&pds_free[x], 1);
    }
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, GROUP);
    mbar_init(acc_full, 1);
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tptr, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tptr;

  // What the issuing warps broadcast (descriptors) the compiler keeps in uniform registers, which MMAs take their
  // operands from: a step along K then is one uniform addition.
  auto uniform = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
  constexpr uint32_t STAGE16 = L::STAGE >> 4, TILE16 = L::TILE >> 4;
  auto pair_of = [&](int slot) -> Pair {
    if (slot >= npairs) return {0, 0, false};
    const int e = list[first + slot];
    return {debug_index(e >> 5, 0, T), e & 31, true};
  };

  if (warp == PROD_WARP || warp == PROD2_WARP<D> || warp == PROD3_WARP) {
    if constexpr (TMA_IN) {
      if (warp == PROD_WARP) {
        // Lane l copies query l of the tile: per panel G rows (G = 8, 16: whole
        // swizzle atoms).  Past the item's last query the zero rows behind the
        // packed ones are copied.
        const uint32_t bytes = static_cast<uint32_t>(G) * 128;
        const long long none = static_cast<long long>(n_bh) * T;
        auto query_of = [&](int slot) -> long long {
          return slot < npairs ? static_cast<long long>(bg) * T + debug_index(list[first + slot] >> 5, 0, T) : none;
        };
        int t = 0;
        bool ok = true;
        long long next = lane < qpt ? query_of(lane) : none;
        for (; t < nt && ok; ++t) {
          const int x = t % L::NS;
          const __nv_bfloat16* src = rows + next * (2 * G * D);
          next = lane < qpt ? query_of((t + 1) * qpt + lane) : none;
          // rows of the tile that takes this stage next: on their way to L2 while the stage is in use
          if (lane < qpt && (t + L::NS) * qpt + lane < npairs)
            bulk_prefetch(rows + query_of((t + L::NS) * qpt + lane) * (2 * G * D), 4 * G * D);
          uint8_t* st = smem + x * L::STAGE + lane * G * 128;
          const uint32_t par = ((t / L::NS) & 1) ^ 1;
          if (lane == 0 && (ok = mbar_wait(&q_empty[x], par))) mbar_arrive_expect_tx(&q_full[x], L::TILE);
          if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
          if (lane < qpt)
#pragma unroll
            for (int p = 0; p < L::NP; ++p)
              bulk_load(st + L::TILE + p * PANEL, src + (L::NP + p) * G * 64, bytes, &q_full[x]);
          if (lane == 0 && (ok = mbar_wait(&do_empty[x], par))) mbar_arrive_expect_tx(&do_full[x], L::TILE);
          if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) {
            if (lane == 0) mbar_wait(&q_full[x], (t / L::NS) & 1);  // what was just issued must land first
            break;
          }
          if (lane < qpt)
#pragma unroll
            for (int p = 0; p < L::NP; ++p) bulk_load(st + p * PANEL, src + p * G * 64, bytes, &do_full[x]);
        }
        // never leave a copy landing in a finished CTA
        if (lane == 0)
          for (int u = t > L::NS ? t - L::NS : 0; u < t; ++u) {
            mbar_wait(&q_full[u % L::NS], (u / L::NS) & 1);
            mbar_wait(&do_full[u % L::NS], (u / L::NS) & 1);
          }
      }
    } else {
      // Lane l resolves row 32 x + l of the tile (x: which gathering warp); rows are copied by 8 consecutive lanes
      // to a panel, so that a warp instruction reads whole runs of 128 bytes.
      const int row0 = warp == PROD_WARP ? 0 : warp == PROD2_WARP<D> ? 32 : 64;
      const int rr = row0 + lane, rq = rr / G < qpt ? rr / G : -1, rg = rr % G;
      const uint32_t panels = 2 * L::NP * G;  // 128-byte runs of a query
      auto run_of = [&](int t) -> uint32_t {  // first run of this lane's row of tile t; all ones: no row
        const Pair p = pair_of(rq >= 0 ? t * qpt + rq : npairs);
        return p.valid ? static_cast<uint32_t>((static_cast<long long>(bg) * T + p.i) * panels) + rg : 0xffffffffu;
      };
      const int c = lane & 7;
      // the packed rows' chunk orders (head & 7) of the eight rows this lane copies from, three bits each
      uint32_t keys = 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) keys |= static_cast<uint32_t>(((row0 + 4 * k + (lane >> 3)) % G) & 7) << (3 * k);
      uint32_t next = run_of(0);
      for (int t = 0; t < nt; ++t) {
        const int x = t % L::NS;
        const uint32_t par = ((t / L::NS) & 1) ^ 1;
        const uint32_t run = next;
        next = run_of(t + 1);  // (its list entry is on its way while this tile is copied)
        const uint32_t st = smem_u32(smem + x * L::STAGE);
        // (bounded waits: on a failure nothing new is issued, and every copy issued has landed)
        if (!mbar_wait(&q_empty[x], par) || !mbar_wait(&do_empty[x], par)) break;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int from = 4 * k + (lane >> 3), r = row0 + from;
          const uint32_t o = __shfl_sync(0xffffffffu, run, from);
          const uint32_t bytes = o != 0xffffffffu ? 16u : 0u;
          const __nv_bfloat16* src =
              rows + static_cast<size_t>(bytes ? o : 0u) * 64 + ((c ^ ((keys >> (3 * k)) & 7u)) << 3);
          const uint32_t dst = st + r * 128 + ((c ^ (r & 7)) << 4);
#pragma unroll
          for (int p = 0; p < L::NP; ++p) {
            cp_async16(dst + p * PANEL, src + p * G * 64, bytes);
            cp_async16(dst + L::TILE + p * PANEL, src + (L::NP + p) * G * 64, bytes);
          }
        }
        cp_async_commit();
        // A tile is announced before the next is issued: behind that it would wait for the next one's stage, and so for
        // the products of a tile before it (one more in flight: 4096 tokens of 16 heads of 64 in groups of four 2%
        // longer, all but two of the stages 8%).
        cp_async_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&q_full[x]);
        mbar_arrive(&do_full[x]);
      }
    }
  } else if (warp == MMA_WARP) {
    const bool leader = lane == 0;
    if (leader) {
      debug_check(key0 >= 0 && key0 + KEYS <= T);
      mbar_arrive_expect_tx(kv_full, 2 * L::NP * KEYS * 128);
#pragma unroll
      for (int p = 0; p < L::NP; ++p) {
        tma_load_3d(smem + L::K_OFF + p * KV_PANEL, &tmK, kv_full, 64 * p, key0, bg);
        tma_load_3d(smem + L::V_OFF + p * KV_PANEL, &tmV, kv_full, 64 * p, key0, bg);
      }
    }
    constexpr uint32_t ID_S = idesc_bf16_f32(128, KEYS, 0, 0);
    const uint32_t tm = uniform(tmem), base = uniform(smem_u32(smem));
    const uint32_t kK = desc_lo(base + L::K_OFF, 16), kV = desc_lo(base + L::V_OFF, 16);
    const uint32_t kDO = desc_lo(base, 16);
    bool ok = mbar_wait(kv_full, 0);
    for (int t = 0; t < nt && ok; ++t) {
      const int x = t % L::NS, b = t & 1;  // stage, TMEM buffer
      const uint32_t par = (t / L::NS) & 1;
      const uint32_t aQ = uniform(kDO + x * STAGE16 + TILE16), aDO = uniform(kDO + x * STAGE16);
      const uint32_t dS = uniform(tm + L::TS + b * BS), dP = uniform(tm + L::TP + b * BS);
      if (t >= 2 && !(ok = mbar_wait(&sp_empty[b], ((t >> 1) - 1) & 1))) break;
      if (!(ok = mbar_wait(&q_full[x], par))) break;
      tc_fence_after();
      __syncwarp();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_lo(dS, aQ + ((kk >> 2) * PANEL + (kk & 3) * 32) / 16, kK + ((kk >> 2) * KV_PANEL + (kk & 3) * 32) / 16,
                 ID_S, kk > 0 ? 1u : 0u);
      }
      if (!(ok = mbar_wait(&do_full[x], par))) break;
      tc_fence_after();
      __syncwarp();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_lo(dP, aDO + ((kk >> 2) * PANEL + (kk & 3) * 32) / 16, kV + ((kk >> 2) * KV_PANEL + (kk & 3) * 32) / 16,
                 ID_S, kk > 0 ? 1u : 0u);
        mma_commit(&sp_full[b]);
      }
      __syncwarp();
    }
    if (leader) {
      mma_commit(&mma_done[0]);
      mbar_wait(&mma_done[0], 0);
    }
  } else if (warp == GRAD_WARP<D>) {
    // (the scores of a tile are complete before its gradients' inputs are: what this warp commits frees the stage)
    const bool leader = lane == 0;
    constexpr uint32_t ID_ACC = idesc_bf16_f32(128, D == 128 ? KEYS : 2 * BS, 1, 1);
    constexpr uint32_t ID_Q = idesc_bf16_f32(128, D, 0, 1);
    const uint32_t tm = uniform(tmem), base = uniform(smem_u32(smem));
    // MN-major operands (a step of 16 rows is 2048 bytes), and dS K-major
    const uint32_t mK = desc_lo(base + L::K_OFF, L::NP > 1 ? KV_PANEL : 1024);
    constexpr uint32_t PDS16 = L::PDS >> 4;
    const uint32_t m0 = desc_lo(base + L::P_OFF, D == 128 ? 1024 : PANEL);
    const uint32_t m1 = desc_lo(base + L::DS_OFF, 1024), k1 = desc_lo(base + L::DS_OFF, 16);
    const uint32_t mDO = desc_lo(base, PANEL);
    bool ok = mbar_wait(kv_full, 0);
    for (int t = 0; t < nt && ok; ++t) {
      const int x = t % L::NS;
      const uint32_t aDO = uniform(mDO + x * STAGE16), aQ = uniform(mDO + x * STAGE16 + TILE16);
      const uint32_t more = uniform(t > 0 ? 1u : 0u);
      const uint32_t buf = (t & 1) * PDS16, mP = uniform(m0 + buf), mDS = uniform(m1 + buf), kDS = uniform(k1 + buf);
      if (!(ok = mbar_wait(&pds_ready[t & 1], (t >> 1) & 1))) break;
      tc_fence_after();
      __syncwarp();
      if (leader) {
        if constexpr (D == 128) {
#pragma unroll
          for (int kk = 0; kk < ROWS / 16; ++kk)
            mma_lo(tm + L::TV, aDO + kk * 128, mP + kk * 128, ID_ACC, kk > 0 ? 1u : more);
          mma_commit(&do_empty[x]);
#pragma unroll
          for (int kk = 0; kk < ROWS / 16; ++kk)
            mma_lo(tm + L::TK, aQ + kk * 128, mDS + kk * 128, ID_ACC, kk > 0 ? 1u : more);
          mma_commit(&q_empty[x]);
        } else {  // [dO | Q]^T [P | dS]
#pragma unroll
          for (int kk = 0; kk < ROWS / 16; ++kk)
            mma_lo(tm + L::TV, aDO + kk * 128, mP + kk * 128, ID_ACC, kk > 0 ? 1u : more);
          mma_commit(&do_empty[x]);
          mma_commit(&q_empty[x]);
        }
      }
      __syncwarp();
      if (t > 0 && !(ok = mbar_wait(dq_empty, (t - 1) & 1))) break;
      tc_fence_after();
      __syncwarp();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < KEYS / 16; ++kk)
          mma_lo(tm + L::TQ, kDS + kk * 2, mK + kk * 128, ID_Q, kk > 0 ? 1u : 0u);
        mma_commit(dq_full);
        mma_commit(&pds_free[t & 1]);
      }
      __syncwarp();
    }
    if (leader) {
      if (ok) mma_commit(acc_full);
      mma_commit(&mma_done[1]);
      mbar_wait(&mma_done[1], 0);
    }
  } else if (warp >= DRAIN_WARP) {  // (8..10)
    // ---- dQ rows: thread = row of the tile
    const int r = threadIdx.x - DRAIN_WARP * 32;
    const uint32_t tQ = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::TQ;
    const int qi = r / G, g = r % G;
    Pair next = pair_of(qi < qpt ? qi : npairs);
    float kmax = 0.0f;
    for (int t = 0; t < nt; ++t) {
      const Pair p = next;
      next = pair_of(qi < qpt ? (t + 1) * qpt + qi : npairs);
      if (!mbar_wait(&sum_full[t & 1], (t >> 1) & 1)) break;
      // the row's power-of-two factor 2^e: bound * 2^e in [2^14, 2^15) (1%: dS rounded to bf16, the sums' own rounding)
      if (t == 0)
#pragma unroll
        for (int j = 0; j < GROUP; ++j) kmax = fmaxf(kmax, fmaxf(km[j], km[4 + j]));
      const float* sm = sums + (t & 1) * 2 * ROWS + r;
      const float bound = (sm[0] + sm[ROWS]) * kmax * 1.01f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sum_free[t & 1]);
      const int ex = static_cast<int>(__float_as_uint(bound) >> 23) - 127;
      const int e = bound > 0.0f && ex < 128 ? min(14 - ex, 126) : 0;
      const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      const size_t to = ((((static_cast<size_t>(bg) * T + p.i) * S + p.s) << two) + half) * G + g;
      if (p.valid) dq_scale[to] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      __half* row = dq_part + to * D;
      if (!mbar_wait(dq_full, t & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tQ + c * 32, v);
        tmem_wait_ld();
        if (c == D / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dq_empty);
        }
        if (p.valid)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = pack_f16x2(__uint_as_float(v[16 * x + 2 * e]) * f, __uint_as_float(v[16 * x + 2 * e + 1]) * f);
            store32(row + 32 * c + 16 * x, w);
          }
      }
    }
  } else {  // warps 0..2, 4..6
    // ---- epilogue half w: keys 32w .. 32w + 31; thread = row of the tile
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const int qi = r / G, g = r % G;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 32 * w;
    const float sl2 = scale * NSA_LOG2E;
    bool ok = mbar_wait(kv_full, 0);
    // max |K| over the keys up to the item's last query, for the drain's bound on a dQ row.  The keys behind it become
    // zeros, as dS of them does: what they hold may not be a number.  (The first scores may be read before that or
    // after: the mask hides them.  dQ's products come behind this warp's first proxy fence and arrival below.)
    {
      const int live = (list[first + npairs - 1] >> 5) - key0;
      uint4* kt = reinterpret_cast<uint4*>(smem + L::K_OFF);
      uint32_t m = 0u;
      for (int e = r + w * ROWS; e < L::NP * KEYS * 8; e += 2 * ROWS) {
        uint4& u = kt[e / (KEYS * 8) * (KV_PANEL / 16) + e % (KEYS * 8)];
        if (e % (KEYS * 8) / 8 > live) u = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max((x[j] & 0x7fffu) << 16, x[j] & 0x7fff0000u));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) km[warp] = __uint_as_float(m);
    }
    auto stats_of = [&](const Pair& p) {
      return p.valid ? stats[(static_cast<size_t>(bg) * T + p.i) * G + g] : make_float2(0.0f, 0.0f);
    };
    Pair p = pair_of(qi < qpt ? qi : npairs), p2 = pair_of(qi < qpt ? qpt + qi : npairs);
    float2 ld = stats_of(p);
    for (int t = 0; t < nt && ok; ++t) {
      const int lim = p.valid ? min(p.i - key0 - 32 * w, KEYS - 1) : -1;  // this half's keys c <= lim are causal
      const bool none = KEYS < 64 && w == 1;                              // a half without keys
      const float lse2 = ld.x, delta = ld.y;
      p = p2;  // the next tile's row: its numbers are on their way before this tile's arithmetic
      ld = stats_of(p);
      p2 = pair_of(qi < qpt ? (t + 2) * qpt + qi : npairs);
      if (!(ok = mbar_wait(&sp_full[t & 1], (t >> 1) & 1))) break;
      tc_fence_after();
      uint32_t sv[32], pv[32];
      if (!none) {
        tmem_ld32(lane_base + L::TS + (t & 1) * BS, sv);
        tmem_ld32(lane_base + L::TP + (t & 1) * BS, pv);
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sp_empty[t & 1]);  // the next but one tile's scores may overwrite these
      uint32_t pk[16], dk2[16];
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (none) {
          pk[c] = dk2[c] = 0u;
          continue;
        }
        float pp[2], dd[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 2 * c + e;
          const float y = ex2f(fmaf(__uint_as_float(sv[col]), sl2, -lse2));
          pp[e] = col <= lim ? y : 0.0f;
          const float z = y * (__uint_as_float(pv[col]) - delta) * scale;
          dd[e] = col <= lim ? z : 0.0f;
          sum += fabsf(dd[e]);
        }
        pk[c] = pack_bf16x2(pp[0], pp[1]);
        dk2[c] = pack_bf16x2(dd[0], dd[1]);
      }
      // the products of the tile before the last have read this buffer, and its drain the sums
      const uint32_t past = ((t >> 1) - 1) & 1;
      if (t >= 2 && !(ok = mbar_wait(&pds_free[t & 1], past) && mbar_wait(&sum_free[t & 1], past))) break;
      uint8_t* pds = smem + L::P_OFF + (t & 1) * L::PDS;
      sums[((t & 1) * 2 + w) * ROWS + r] = sum;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t off = r * 128 + (((4 * w + x) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(pds + off) =
            make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
        *reinterpret_cast<uint4*>(pds + PANEL + off) =
            make_uint4(dk2[4 * x], dk2[4 * x + 1], dk2[4 * x + 2], dk2[4 * x + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&pds_ready[t & 1]);
        mbar_arrive(&sum_full[t & 1]);
      }
    }
  }
  // ---- the block's dV^T and dK^T: lane = dim, column = token; warps 0..3 and 4..7, done with their parts
  if (warp < 8) {
    __syncwarp();
    if (mbar_wait(acc_full, 0)) {
      tc_fence_after();
      // D = 128: warps 0..3 store dV, 4..7 dK.  D = 64: lanes 0..63 hold dV (columns 0..63), 64..127 dK (64..127);
      // warps 0..3 and 4..7 each take half of the tokens.
      const int w = warp >> 2, r = (warp & 3) * 32 + lane;
      const int which = D == 128 ? w : r >> 6;  // 0: dV, 1: dK
      const int d = D == 128 ? r : r & 63;
      const int c0 = D == 128 ? 0 : w * 32;
      const uint32_t tA =
          tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (which ? L::TK : L::TV) + c0;
      __nv_bfloat16* dst = (which ? dk : dv) + (static_cast<size_t>(bg) * T + key0) * D + d;
      float* pd = part + (((static_cast<size_t>(item_no) * 2 + (which ? 0 : 1)) << two) + half) * KEYS * D + d;
#pragma unroll
      for (int h = 0; h < (D == 128 && KEYS == 64 ? 2 : 1); ++h) {
        if (c0 >= KEYS) break;
        uint32_t v[32];
        tmem_ld32(tA + 32 * h, v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < (KEYS < 32 ? KEYS : 32); ++c) {
          const int tok = c0 + 32 * h + c;
          if (item.w == 1) dst[tok * D] = __float2bfloat16_rn(__uint_as_float(v[c]));
          else pd[tok * D] = __uint_as_float(v[c]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Packs the rows that the pass gathers: per query (b, kv head, i) the G heads'
// dO rows, then their Q rows, each as 64-column panels of G rows of 128 bytes
// in the order of the 128-byte swizzle (chunk ^ (g & 7)); and each row's
// (lse log2e, dout . out).  A query's rows then are 4 G D contiguous bytes (as
// the heads lie T D elements apart, gathering them unpacked costs a request
// and an address translation for every 128 bytes).  One more query of zeros is
// written behind the last.  D / 8 lanes a row, the heads of a query beside one
// another.
template <int D>
__global__ void __launch_bounds__(256) nsa_bwd_pack_kernel(const __nv_bfloat16* __restrict__ q,
                                                           const __nv_bfloat16* __restrict__ out,
                                                           const __nv_bfloat16* __restrict__ dout,
                                                           const float* __restrict__ lse,
                                                           __nv_bfloat16* __restrict__ rows,
                                                           float2* __restrict__ stats, uint32_t n_rows, int G, int T) {
  constexpr int LPR = D / 8;
  const uint32_t row = blockIdx.x * (256u / LPR) + threadIdx.x / LPR, heads = G;  // ((b, kv head), i, g)
  const int c = threadIdx.x % LPR;
  const uint32_t g = row % heads, query = row / heads;
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a, o = a;
  const uint32_t bg = query / T, i = query % T;
  const size_t src = (static_cast<size_t>(bg * heads + g) * T + i) * D + c * 8;
  if (row < n_rows) {
    a = *reinterpret_cast<const uint4*>(dout + src);
    b = *reinterpret_cast<const uint4*>(q + src);
    o = *reinterpret_cast<const uint4*>(out + src);
  }
  if (row < n_rows + G) {
    __nv_bfloat16* dst = rows + static_cast<size_t>(query) * (2 * G * D) + ((c >> 3) * G + g) * 64 +
                         (((c & 7) ^ (g & 7)) << 3);
    *reinterpret_cast<uint4*>(dst) = a;
    *reinterpret_cast<uint4*>(dst + G * D) = b;
  }
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {o.x, o.y, o.z, o.w};
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s = fmaf(__uint_as_float(x[j] << 16), __uint_as_float(y[j] << 16), s);
    s = fmaf(__uint_as_float(x[j] & 0xffff0000u), __uint_as_float(y[j] & 0xffff0000u), s);
  }
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (row < n_rows && c == 0) stats[row] = make_float2(lse[static_cast<size_t>(bg * heads + g) * T + i] * NSA_LOG2E, s);
}

// dq of every row: the f16 rows of its query's live slots under their
// factors, in slot order.  D / 8 lanes a row, the heads of a query beside one
// another, so that a slot's G rows are read as one run.
// Four rows ahead in 64 registers (four blocks a SM) read 2.2 GB at 6.6 TB/s
// (345 us); eight ahead in 85 took as long, and either in fewer registers
// spills.  With 64-bit row numbers, and the live slots read once a row where
// the warp's rows are one query's, 134 MB of rows of 64 took 29 us, now 25.
template <int D>
__global__ void __launch_bounds__(256, 4) nsa_bwd_dq_sum_kernel(const int32_t* __restrict__ block_idx,
                                                             const __half* __restrict__ dq_part,
                                                             const float* __restrict__ dq_scale,
                                                             __nv_bfloat16* __restrict__ dq, uint32_t n_rows, int G,
                                                             int T, int S, int n_blk, int bs, int two) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes a row, rows a warp
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const uint32_t row0 = (blockIdx.x * 8u + (threadIdx.x >> 5)) * RPW;  // the warp's first row
  const uint32_t row = row0 + lane / LPR, heads = G;
  const bool in = row < n_rows;
  const uint32_t g = row % heads;
  const size_t query = in ? row / heads : 0;
  const int n = S << two;  // rows of a query: one for each slot, or each half of a slot's 128 tokens
  const __half* src = dq_part + (query * n * G + g) * D + (c << 3);
  const float* sc = dq_scale + query * n * G + g;
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.0f;
  constexpr int AHEAD = 4;  // slots whose loads are in flight
  uint4 u[AHEAD];
  float f[AHEAD];
  // Rows are loaded before it is known which slots are live (those of dead
  // slots hold anything and are not added).
  auto load = [&](int x, int s) {
    if (in && s < n) {
      u[x] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<size_t>(s) * G * D));
      f[x] = sc[s * G];
    }
  };
#pragma unroll
  for (int x = 0; x < AHEAD; ++x) load(x, x);
  // live slots of the warp's queries (the warp steps them together); mostly its rows are one query's
  uint32_t live = 0u;
  const uint32_t y0 = row0 / heads, y1 = (min(row0 + RPW, n_rows) - 1) / heads;
  if (row0 < n_rows)
    for (uint32_t y = y0; y <= y1; ++y) {
      const int i = static_cast<int>(y % T);
      const uint32_t m = nsa_live_slots(block_idx + static_cast<size_t>(y) * S, S, i, n_blk, bs).live;
      if (query == y) live = m;
    }
  for (int s0 = 0; s0 < n; s0 += AHEAD) {
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      if (in && s0 + x < n && ((live >> ((s0 + x) >> two)) & 1u)) {
        const uint32_t w[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
          o[2 * e] = fmaf(f[x], h.x, o[2 * e]);
          o[2 * e + 1] = fmaf(f[x], h.y, o[2 * e + 1]);
        }
      }
      load(x, s0 + x + AHEAD);
    }
  }
  if (!in) return;
  const uint32_t bg = row / heads / T, i = row / heads % T;
  *reinterpret_cast<uint4*>(dq + (static_cast<size_t>(bg * heads + g) * T + i) * D + c * 8) =
      make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
}

template <int D, int KEYS>
int launch_tc(const NsaBwdArgs& a, const NsaBwdScratch& w, cudaStream_t stream) {
  using L = TcLayout<D>;
  const int G = a.Hq / a.Hkv, n_blk = a.T / a.bs, two = a.bs / KEYS - 1;
  const long long bh = static_cast<long long>(a.B) * a.Hkv, rows = bh * G * a.T;
  CUtensorMap mk, mv;
  const uint64_t rs = static_cast<uint64_t>(D) * 2, hs = rs * a.T;
  int st = encode_tmap_3d(&mk, a.k, D, a.T, bh, rs, hs, 64, KEYS, 1);
  if (st == OK) st = encode_tmap_3d(&mv, a.v, D, a.T, bh, rs, hs, 64, KEYS, 1);
  if (st != OK) return st;

  constexpr int BLOCK_ROWS = 256 / (D / 8);  // rows of one block of the two row kernels
  if (rows > 0x7fffffffLL) return ERR_SHAPE;  // (no such sizes reach this; the row kernels count in 32 bits)
  const uint32_t n_rows = static_cast<uint32_t>(rows);
  const long long pack_blocks = (rows + G + BLOCK_ROWS - 1) / BLOCK_ROWS;
  nsa_bwd_pack_kernel<D><<<static_cast<unsigned>(pack_blocks), 256, 0, stream>>>(a.q, a.out, a.dout, a.lse, w.rows,
                                                                                 w.stats, n_rows, G, a.T);
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  const bool bulk = G == 8 || G == 16;
  auto kern = bulk ? nsa_bwd_tc_kernel<D, KEYS, true> : nsa_bwd_tc_kernel<D, KEYS, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC) != cudaSuccess)
    return ERR_LAUNCH;
  kern<<<static_cast<unsigned>(w.max_items << two), bulk ? tc_threads<D, true>() : tc_threads<D, false>(), L::ALLOC,
         stream>>>(
      mk, mv, w.rows, w.stats, w.list, w.items, w.n_items, w.part, w.dq_part, w.dq_scale, a.dk, a.dv, G, a.T, a.S,
      n_blk, static_cast<int>(bh), two, 1.0f / sqrtf(static_cast<float>(D)));
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  const long long sum_blocks = (rows + BLOCK_ROWS - 1) / BLOCK_ROWS;
  nsa_bwd_dq_sum_kernel<D><<<static_cast<unsigned>(sum_blocks), 256, 0, stream>>>(
      a.idx, w.dq_part, w.dq_scale, a.dq, n_rows, G, a.T, a.S, n_blk, a.bs, two);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace

int launch_nsa_bwd_tc(const NsaBwdArgs& a, const NsaBwdScratch& w, int D, cudaStream_t stream) {
  if (a.bs == 16) return D == 128 ? launch_tc<128, 16>(a, w, stream) : launch_tc<64, 16>(a, w, stream);
  if (a.bs == 32) return D == 128 ? launch_tc<128, 32>(a, w, stream) : launch_tc<64, 32>(a, w, stream);
  return D == 128 ? launch_tc<128, 64>(a, w, stream) : launch_tc<64, 64>(a, w, stream);
}

unsigned int nsa_bwd_tc_device_error() { return read_and_clear_device_error(); }

}  // namespace bsa
