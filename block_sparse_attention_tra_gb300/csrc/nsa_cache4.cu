// nsa_cache4.cu -- new tokens' keys and values into a paged cache of 4-bit
// codes, keys (and, beside them, queries) normalised and rotated on the way,
// and the values read back.
//
// Every 16 elements of a row share a scale s = e4m3(max |x| / 6), and an
// element is kept as the e2m1 code nearest to x / s (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives), ties to the even code; it stands for s times the code.
// A token's codes are its own: a page that was begun is not read, and no value
// held changes when tokens follow.  The quotient has to be the rounded one,
// since codes change at it: values of few bits lie on the borders often.  With
// y = x (1/s), y + (x - y s) (1/s) is (one step of residual correction, the
// residual exact in an fma; compared with the division in the tests).
//
// Rows, norm and rotation are those of qk_rope.cu: a thread holds 16 elements,
// in halves the two runs of eight that are rotated into each other, so that a
// group of 16 is shared by two runs, of one thread or of two lanes of a row;
// they exchange the runs' maxima by shuffles.  Memory bounds long prompts
// (values that need no rotation: 2 bytes read and 0.56 written an element), the
// latency of one trip through load and store single tokens.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "rope.cuh"

namespace bsa {
namespace {

constexpr int APPEND_ROWS = 8;  // rows a thread walks at most

struct Append4Args {
  Cache4 c;
  const void* x[3];  // q, k, v
  long long stride[3][3];
  void* q_out;
  const void* weight[2];  // q, k
  const int32_t *lens, *new_lens;
  const float* inv_freq;
  int Hq, n, rotary, interleaved, w_f32, page_log;
  long long tokens;
  float factor, eps;
  RowTile tile;
  int groups[3], all_groups;  // blocks over the heads of q, k, v and of all
};

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// The larger magnitude; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// Eight elements under a scale as codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float* x, float s, float inv) {
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float q = x[j + e] * inv;
      y[e] = fmaf(fmaf(-q, s, x[j + e]), inv, q);
    }
    w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(y[0], y[1]), __NV_E2M1, cudaRoundNearest))
         << (4 * j);
  }
  return w;
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS, 3) nsa_cache4_append_kernel(const __grid_constant__ Append4Args a) {
  constexpr int AHEAD = sizeof(T) == 2 ? 2 : 1;  // rows on their way
  int group = static_cast<int>(blockIdx.x % a.all_groups), s = 0;  // s: q, k, v
  while (group >= a.groups[s]) group -= a.groups[s++];
  const int heads = s == 0 ? a.Hq : a.c.Hkv, D = a.c.D;
  const int u = threadIdx.x & ((1 << a.tile.lanes_log) - 1), slot = static_cast<int>(threadIdx.x) >> a.tile.lanes_log;
  const long long token = (static_cast<long long>(blockIdx.x / a.all_groups) << a.tile.tokens_log) +
                          (slot & ((1 << a.tile.tokens_log) - 1));
  const int head_step = ROW_THREADS >> a.tile.lanes_log >> a.tile.tokens_log;
  const int head0 = group * row_heads(a.tile) + (slot >> a.tile.tokens_log);
  bool live = token < a.tokens && u * UNIT < D;
  const int b = live ? static_cast<int>(static_cast<uint32_t>(token) / static_cast<uint32_t>(a.n)) : 0;
  const int t = live ? static_cast<int>(static_cast<uint32_t>(token) % static_cast<uint32_t>(a.n)) : 0;
  const bool il = a.interleaved != 0;
  const UnitMap m = unit_map(u, s < 2 ? a.rotary : 0, il);
  const T* src = static_cast<const T*>(a.x[s]) + b * a.stride[s][0] + t * a.stride[s][2];
  const long long head_stride = a.stride[s][1];
  const int held = live ? a.lens[b] : 0;
  if (live && a.new_lens != nullptr) live = t < a.new_lens[b];
  RawUnit<T> raw[AHEAD];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int h = head0 + (r0 + i) * head_step;
      if (live && r0 + i < a.tile.rows && h < heads) raw[i].load(src + h * head_stride, m);
      else raw[i].clear();
    }
  };
  fetch(0);
  // the token's slot of the cache (where it has one)
  size_t at = 0;
  bool kept = false;
  if (s > 0 && live && held >= 0) {
    const long long pos = static_cast<long long>(held) + t, lp = pos >> a.page_log;
    if (lp < a.c.max_pages) {
      const int id = a.c.table[static_cast<size_t>(b) * a.c.max_pages + lp];
      kept = id >= 0 && id < a.c.num_pages;
      at = (static_cast<size_t>(id) * a.c.Hkv << a.page_log) + static_cast<size_t>(pos & (a.c.page - 1));
    }
  }
  float c[8], w[8], wt[UNIT];
  const bool turn = live && m.freq >= 0;
  if (turn) sincos8_of(a.inv_freq + m.freq, static_cast<int>(static_cast<uint32_t>(held) + t), a.factor, c, w);
  const void* weight = s < 2 ? a.weight[s] : nullptr;
  const bool norm = weight != nullptr;
  if (norm && live) load_weights(weight, a.w_f32 != 0, m, wt);
  const float inv_d = 1.0f / static_cast<float>(D);
  // the runs of eight that share a group with this thread's: run r of a row is half `r_hi` of unit `r_unit`
  const int turned = s < 2 && !il ? a.rotary / 16 : 0;  // units whose runs lie apart
  auto run_at = [&](int r, int& unit, bool& hi) {
    if (r < 2 * turned) {
      hi = r >= turned;
      unit = hi ? r - turned : r;
    } else {
      unit = r >> 1;
      hi = (r & 1) != 0;
    }
  };
  const int run_lo = m.lo >> 3, run_hi = m.hi >> 3, row_lane = threadIdx.x & 31 & ~((1 << a.tile.lanes_log) - 1);
  int mate_lo, mate_hi;
  bool mate_lo_hi, mate_hi_hi;
  run_at(run_lo ^ 1, mate_lo, mate_lo_hi);
  run_at(run_hi ^ 1, mate_hi, mate_hi_hi);

  for (int r0 = 0; r0 < a.tile.rows; r0 += AHEAD) {
    if (r0 > 0) fetch(r0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (r0 + i >= a.tile.rows) break;
      float x[UNIT];
      raw[i].unpack(x);
      if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < UNIT; ++j) ss = fmaf(x[j], x[j], ss);
        const float r = rsqrtf(fmaf(row_sum(ss, a.tile.lanes_log), inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < UNIT; ++j) x[j] = x[j] * r * wt[j];
      }
      if (turn) rotate16(x, c, w, il);
      const int h = head0 + (r0 + i) * head_step;
      if (s == 0) {
        if (!live || h >= heads) continue;
        T* row = static_cast<T*>(a.q_out) + ((static_cast<size_t>(b) * a.Hq + h) * a.n + t) * D;
        store8(row + m.lo, x);
        store8(row + m.hi, x + 8);
        continue;
      }
      const float* factor = s == 1 ? a.c.k_factor : a.c.v_factor;
      if (factor != nullptr && h < heads) {
        const float f = factor[h];
#pragma unroll
        for (int j = 0; j < UNIT; ++j) x[j] = __fdiv_rn(x[j], f);
      }
      float max_lo = 0.0f, max_hi = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        max_lo = max_nan(max_lo, x[j]);
        max_hi = max_nan(max_hi, x[8 + j]);
      }
      // (lanes past the row's last unit name mates past it too: lanes of the same warp)
      const float lo_a = __shfl_sync(0xffffffffu, max_lo, row_lane + mate_lo);
      const float lo_b = __shfl_sync(0xffffffffu, max_hi, row_lane + mate_lo);
      const float hi_a = __shfl_sync(0xffffffffu, max_lo, row_lane + mate_hi);
      const float hi_b = __shfl_sync(0xffffffffu, max_hi, row_lane + mate_hi);
      max_lo = max_nan(max_lo, mate_lo_hi ? lo_b : lo_a);
      max_hi = max_nan(max_hi, mate_hi_hi ? hi_b : hi_a);
      if (!kept || h >= heads) continue;
      const size_t row = at + (static_cast<size_t>(h) << a.page_log);
      uint8_t* codes = (s == 1 ? a.c.k : a.c.v) + row * (D / 2);
      uint8_t* scales = (s == 1 ? a.c.k_scale : a.c.v_scale) + row * (D / 16);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float top = e ? max_hi : max_lo;
        const int start = e ? m.hi : m.lo;
        // NaN and infinities: the group's scale is NaN
        const uint32_t sc = top <= 3.402823466e38f ? __nv_cvt_float_to_fp8(top / 6.0f, __NV_SATFINITE, __NV_E4M3) : 0x7fu;
        const float sv = e4m3_value(sc), inv = sc == 0u ? 0.0f : __fdiv_rn(1.0f, sv);
        *reinterpret_cast<uint32_t*>(codes + start / 2) = sc == 0x7fu ? 0u : codes8(x + 8 * e, sv, inv);
        if ((start & 8) == 0) scales[start / 16] = static_cast<uint8_t>(sc);
      }
    }
  }
}

struct Read4Args {
  Cache4 c;
  const int32_t *starts, *lens;
  void* out[2];
  int n, page_log;
  long long units;  // groups of 16 of one tensor
};

// One thread a group of 16: 8 bytes of codes and a scale.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) nsa_cache4_read_kernel(const __grid_constant__ Read4Args a) {
  const long long x = static_cast<long long>(blockIdx.x >> 1) * ROW_THREADS + threadIdx.x;
  const int s = blockIdx.x & 1;
  if (x >= a.units) return;
  const int upr = a.c.D / UNIT;
  const int u = static_cast<int>(x % upr);
  const long long row = x / upr;  // (b, h, t)
  const int t = static_cast<int>(row % a.n);
  const long long bh = row / a.n;
  const int h = static_cast<int>(bh % a.c.Hkv), b = static_cast<int>(bh / a.c.Hkv);
  const int start = a.starts != nullptr ? a.starts[b] : 0;
  const long long pos = static_cast<long long>(start) + t, lp = pos >> a.page_log;
  int id = -1;
  if (start >= 0 && pos < a.lens[b] && lp < a.c.max_pages) id = a.c.table[static_cast<size_t>(b) * a.c.max_pages + lp];
  float y[UNIT];
  if (id >= 0 && id < a.c.num_pages) {
    const size_t at =
        ((static_cast<size_t>(id) * a.c.Hkv + h) << a.page_log) + static_cast<size_t>(pos & (a.c.page - 1));
    const uint2 w = *reinterpret_cast<const uint2*>((s ? a.c.v : a.c.k) + at * (a.c.D / 2) + 8 * u);
    const uint32_t sc = (s ? a.c.v_scale : a.c.k_scale)[at * upr + u];
    const float* factor = s ? a.c.v_factor : a.c.k_factor;
    const float sv = e4m3_value(sc), f = factor != nullptr ? factor[h] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
      const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
      y[2 * i] = __half2float(__half(__half_raw{r.x})) * sv * f;
      y[2 * i + 1] = __half2float(__half(__half_raw{r.y})) * sv * f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < UNIT; ++i) y[i] = 0.0f;
  }
  T* dst = static_cast<T*>(a.out[s]) + row * a.c.D + u * UNIT;
  store8(dst, y);
  store8(dst + 8, y + 8);
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

}  // namespace

int launch_nsa_cache4_append(const Append4Call& r, cudaStream_t stream) {
  Append4Args a{};
  a.c = r.cache;
  const void* x[3] = {r.q, r.k, r.v};
  for (int s = 0; s < 3; ++s) {
    a.x[s] = x[s];
    for (int i = 0; i < 3; ++i) a.stride[s][i] = r.stride[s][i];
  }
  a.q_out = r.q_out;
  a.weight[0] = r.q_weight; a.weight[1] = r.k_weight;
  a.lens = r.lens; a.new_lens = r.new_lens; a.inv_freq = r.inv_freq;
  a.Hq = r.Hq; a.n = r.n; a.rotary = r.rotary; a.interleaved = r.interleaved ? 1 : 0;
  a.w_f32 = r.weight_f32 ? 1 : 0; a.page_log = log2_of(r.cache.page);
  a.factor = r.factor; a.eps = r.eps;
  a.tokens = static_cast<long long>(r.cache.B) * r.n;
  const int Hq = r.q != nullptr ? r.Hq : 0;
  a.tile = row_tile(a.tokens, Hq + 2 * r.cache.Hkv, r.cache.D, APPEND_ROWS);
  const int heads = row_heads(a.tile);
  a.groups[0] = (Hq + heads - 1) / heads;
  a.groups[1] = a.groups[2] = (r.cache.Hkv + heads - 1) / heads;
  a.all_groups = a.groups[0] + 2 * a.groups[1];
  const long long blocks = ((a.tokens + (1LL << a.tile.tokens_log) - 1) >> a.tile.tokens_log) * a.all_groups;
  if (blocks > 0x7fffffffLL) return ERR_SHAPE;
  if (r.f32) nsa_cache4_append_kernel<float><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  else nsa_cache4_append_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

int launch_nsa_cache4_read(const Cache4& c, const int32_t* starts, const int32_t* lens, void* k_out, void* v_out,
                           int n, bool f32, cudaStream_t stream) {
  Read4Args a{};
  a.c = c;
  a.starts = starts; a.lens = lens;
  a.out[0] = k_out; a.out[1] = v_out;
  a.n = n; a.page_log = log2_of(c.page);
  a.units = static_cast<long long>(c.B) * c.Hkv * n * (c.D / UNIT);
  const long long blocks = 2 * ((a.units + ROW_THREADS - 1) / ROW_THREADS);
  if (blocks > 0x7fffffffLL) return ERR_SHAPE;
  if (f32) nsa_cache4_read_kernel<float><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  else nsa_cache4_read_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace bsa
