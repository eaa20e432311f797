// nsa_cache.cu -- appends the keys and values of new tokens to a paged cache
// of e4m3 codes, keys (and, beside them, queries) rotated by position on the
// way.
//
// A page holds `page` tokens of one sequence -- the selected block of the NSA
// selection -- and per kv head one scale: code = e4m3(x / s), x ~ s * code.
// The scale of a page that begins is the least power of two s = 2^e, e >= -96,
// with max |x| <= 448 s over the tokens written; a page that was begun keeps
// its scale while that is 2^-96 or more and the new tokens fit under 448 s, and
// otherwise takes the larger one, the codes it holds being multiplied by the (power-of-two) ratio
// and rounded to e4m3 again.  NaN and infinities do not count towards the
// maximum; NaN is stored as NaN, an infinity as +-448 s.
//
// Rotation of token position m: the pair (x_a, x_b) becomes
// (x_a c - x_b w, x_a w + x_b c) with c, w = cos, sin(m f_j).  m f_j is needed
// modulo one turn: f_j / 2 pi is taken once per block as a 64-bit fixed-point
// fraction of a turn and multiplied by the 32-bit position in integers, which
// drops the whole turns exactly (the angle of position 2^30 is off by 2^-33
// turns, where an fp32 product would be off by whole turns), and the fraction's
// top 32 bits go through sincospi.  fp64 would need three operations an angle
// on a pipe that runs at 1/64 of the fp32 rate here.
//
// One block per (sequence, page it touches, kv head, K or V): the values of
// its tokens are rotated into registers, their maximum reduced over the block,
// then written as codes: each input is read once, each code written once.
// Further blocks rotate the queries, each thread keeping the sines of its row
// over eight heads: with sixteen a prompt takes 205 us in place of 209, four
// chunks of 1031 fp32 tokens 12.8 in place of 9.5.  A thread holds two units
// of 16 values: with four, at half the warps a SM, the prompt took 276 us.
//
// Bound by memory for long prompts: 32768 tokens of 64 query and 4 kv heads of
// 128 in bf16 are 1174 MB, 209 us (5.6 TB/s); for single tokens by the latency
// of one trip through load, reduction and store (4.4 us; 128 sequences 6.1).
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int E_MIN = -96;        // exponent of the least page scale
constexpr int UNIT = 16;          // elements a thread handles of one row
constexpr int KV_UNITS = 2;       // units of a page per thread
constexpr int Q_HEADS = 8;        // query heads per block
constexpr int MAX_THREADS = 512;  // a page of 128 tokens of 128

struct AppendArgs {
  const void *k, *v, *q;
  void* q_out;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const int32_t *table, *lens, *new_lens;
  const float* inv_freq;
  int B, Hq, Hkv, n, D, page, max_pages, num_pages, rotary, interleaved;
  int seq_pages;           // pages a sequence may touch
  long long kv_blocks;     // blocks of the cache part; the rest rotate queries
  int q_rows, q_chunks, q_groups;  // rows per query block, blocks over a sequence's rows, blocks over its heads
};

// f / 2 pi as a fraction of a turn in 2^-64 units, modulo one turn, of a
// finite f >= 0: 24-bit mantissa times 2^64 / 2 pi in 128 bits.
__device__ uint64_t turns_of(float f) {
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

__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return a | (b << 16);
}
// Four codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float f) {
  float x[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
    x[2 * h] = __half2float(__half(__half_raw{r.x}));
    x[2 * h + 1] = __half2float(__half(__half_raw{r.y}));
  }
  return codes4(x, f);
}

// The least e >= E_MIN with amax <= 448 2^e, amax finite (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, E_MIN);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <typename T>
__device__ void append_kv(const AppendArgs& a, const uint64_t* turns, float* red) {
  const int kv = static_cast<int>(blockIdx.x & 1);
  long long r = blockIdx.x >> 1;
  const int h = static_cast<int>(r % a.Hkv);
  r /= a.Hkv;
  const int pl = static_cast<int>(r % a.seq_pages), b = static_cast<int>(r / a.seq_pages);
  const int held = a.lens[b];
  const int n = a.new_lens != nullptr ? min(a.n, a.new_lens[b]) : a.n;
  if (held < 0 || n <= 0) return;
  const long long lp = held / a.page + static_cast<long long>(pl);  // logical page
  const long long first = lp * a.page - held;                       // new token of the page's first slot
  const int t0 = static_cast<int>(max(0LL, first));
  const int t1 = static_cast<int>(min(static_cast<long long>(n), first + a.page));
  if (t0 >= t1 || lp >= a.max_pages) return;
  const int id = a.table[static_cast<size_t>(b) * a.max_pages + lp];
  if (id < 0 || id >= a.num_pages) return;
  const int r0 = static_cast<int>(t0 - first);  // slot of token t0

  const int upr = a.D / UNIT;
  const int units = (t1 - t0) * upr;
  debug_check(units <= KV_UNITS * static_cast<int>(blockDim.x));
  const T* src = static_cast<const T*>(kv ? a.v : a.k) + ((static_cast<size_t>(b) * a.Hkv + h) * a.n + t0) * a.D;
  float x[KV_UNITS][UNIT];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < KV_UNITS; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      const UnitMap m = unit_map(u % upr, kv ? 0 : a.rotary, a.interleaved != 0);
      const T* row = src + static_cast<size_t>(u / upr) * a.D;
      float lo[8], hi[8];
      load8(row + m.lo, lo);
      load8(row + m.hi, hi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[i][j] = lo[j];
        x[i][8 + j] = hi[j];
      }
      if (m.freq >= 0) {
        float c[8], w[8];
        sincos8(turns, m.freq, held + t0 + u / upr, c, w);
        rotate16(x[i], c, w, a.interleaved != 0);
      }
#pragma unroll
      for (int j = 0; j < UNIT; ++j) {
        const float y = fabsf(x[i][j]);
        amax = fmaxf(amax, y <= 3.402823466e38f ? y : 0.0f);
      }
    }
  }
  float* scale = (kv ? a.v_scale : a.k_scale) + static_cast<size_t>(id) * a.Hkv + h;
  const float old = r0 > 0 ? *scale : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) amax = fmaxf(amax, red[w]);

  uint8_t* dst = (kv ? a.v_cache : a.k_cache) + (static_cast<size_t>(id) * a.Hkv + h) * a.page * a.D;
  float s = old;
  // (a page begun elsewhere may have a scale of zero, which no value can be divided by)
  if (r0 == 0 || !(amax <= 448.0f * old && old >= exp2i(E_MIN))) {
    s = exp2i(scale_exponent(amax));
    if (threadIdx.x == 0) *scale = s;
    const float f = old / s;  // the codes already held move to the larger scale
    uint4* p = reinterpret_cast<uint4*>(dst);
    const int held16 = r0 * (a.D / 16);
    constexpr int AHEAD = 2;  // loads in flight
    for (int e0 = threadIdx.x; e0 < held16; e0 += AHEAD * blockDim.x) {
      uint4 u[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (e0 + i * static_cast<int>(blockDim.x) < held16) u[i] = p[e0 + i * blockDim.x];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (e0 + i * static_cast<int>(blockDim.x) < held16)
          p[e0 + i * blockDim.x] =
              make_uint4(recode4(u[i].x, f), recode4(u[i].y, f), recode4(u[i].z, f), recode4(u[i].w, f));
    }
  }
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < KV_UNITS; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      const UnitMap m = unit_map(u % upr, kv ? 0 : a.rotary, a.interleaved != 0);
      uint8_t* row = dst + static_cast<size_t>(r0 + u / upr) * a.D;
      *reinterpret_cast<uint2*>(row + m.lo) = make_uint2(codes4(x[i], inv), codes4(x[i] + 4, inv));
      *reinterpret_cast<uint2*>(row + m.hi) = make_uint2(codes4(x[i] + 8, inv), codes4(x[i] + 12, inv));
    }
  }
}

template <typename T>
__device__ void rotate_q(const AppendArgs& a, const uint64_t* turns) {
  long long r = blockIdx.x - a.kv_blocks;
  const int hg = static_cast<int>(r % a.q_groups);
  r /= a.q_groups;
  const int chunk = static_cast<int>(r % a.q_chunks), b = static_cast<int>(r / a.q_chunks);
  const int upr = a.D / UNIT;
  const int t = chunk * a.q_rows + static_cast<int>(threadIdx.x) / upr;
  const int n = a.new_lens != nullptr ? min(a.n, a.new_lens[b]) : a.n;
  if (static_cast<int>(threadIdx.x) >= a.q_rows * upr || t >= n) return;
  const bool il = a.interleaved != 0;
  const UnitMap m = unit_map(threadIdx.x % upr, a.rotary, il);
  float c[8], w[8];
  if (m.freq >= 0) sincos8(turns, m.freq, a.lens[b] + t, c, w);
  const int h1 = min(a.Hq, (hg + 1) * Q_HEADS);
#pragma unroll 4
  for (int h = hg * Q_HEADS; h < h1; ++h) {
    const size_t row = ((static_cast<size_t>(b) * a.Hq + h) * a.n + t) * a.D;
    const T* src = static_cast<const T*>(a.q) + row;
    T* dst = static_cast<T*>(a.q_out) + row;
    float lo[8], hi[8], x[UNIT];
    load8(src + m.lo, lo);
    load8(src + m.hi, hi);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = lo[j];
      x[8 + j] = hi[j];
    }
    if (m.freq >= 0) rotate16(x, c, w, il);
    store8(dst + m.lo, x);
    store8(dst + m.hi, x + 8);
  }
}

template <typename T>
__global__ void __launch_bounds__(MAX_THREADS, 2) nsa_cache_append_kernel(const AppendArgs a) {
  __shared__ uint64_t turns[64];
  __shared__ float red[MAX_THREADS / 32];
  for (int j = threadIdx.x; j < a.rotary / 2; j += blockDim.x) turns[j] = turns_of(a.inv_freq[j]);
  __syncthreads();
  if (blockIdx.x < a.kv_blocks) append_kv<T>(a, turns, red);
  else rotate_q<T>(a, turns);
}

}  // namespace

int launch_nsa_cache_append(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, const int32_t* table, const int32_t* lens,
                            const int32_t* new_lens, const float* inv_freq, int B, int Hq, int Hkv, int n, int D,
                            int page, int max_pages, int num_pages, int rotary, bool interleaved, bool f32,
                            cudaStream_t stream) {
  AppendArgs a{};
  a.k = k; a.v = v; a.q = q; a.q_out = q_out;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.table = table; a.lens = lens; a.new_lens = new_lens; a.inv_freq = inv_freq;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.n = n; a.D = D; a.page = page;
  a.max_pages = max_pages; a.num_pages = num_pages;
  a.rotary = rotary; a.interleaved = interleaved ? 1 : 0;
  // n tokens behind any length touch at most ceil((n - 1) / page) + 1 pages
  const long long seq_pages = (static_cast<long long>(n) + page - 2) / page + 1;
  a.seq_pages = static_cast<int>(seq_pages < max_pages ? seq_pages : max_pages);
  a.kv_blocks = 2LL * B * a.seq_pages * Hkv;
  // threads for the tokens that a page takes at most: single tokens need a warp (128 of them 6.2 us, with a thread for
  // every unit of a page 11.9)
  const int upr = D / UNIT, units = (n < page ? n : page) * upr;
  const int threads = ((units + KV_UNITS - 1) / KV_UNITS + 31) / 32 * 32;
  static_assert(128 * (128 / UNIT) <= MAX_THREADS * KV_UNITS, "threads for the largest page");
  a.q_rows = threads / upr < n ? threads / upr : n;
  a.q_chunks = (n + a.q_rows - 1) / a.q_rows;
  a.q_groups = (Hq + Q_HEADS - 1) / Q_HEADS;
  const long long blocks = a.kv_blocks + (q != nullptr ? static_cast<long long>(B) * a.q_chunks * a.q_groups : 0LL);
  if (blocks > 0x7fffffffLL) return ERR_SHAPE;
  if (f32) nsa_cache_append_kernel<float><<<static_cast<unsigned>(blocks), threads, 0, stream>>>(a);
  else nsa_cache_append_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), threads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace bsa
