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
#include <cuda_fp16.h>

#include "codes4.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace bsa {
namespace {

struct Append4Args {
  Cache4 c;
  const void* x[3];  // q, k, v
  long long stride[3][3];
  void* q_out;
  const void* weight[2];  // q, k
  const int32_t *lens, *new_lens;
  const float* inv_freq;
  int Hq, n, rotary, w_f32, page_log;
  long long tokens;
  float factor, eps;
  RowPlan<2> plan;  // q; keys and values, as 2 Hkv heads
};

// The larger magnitude; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float approximate_inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// x / s from an inverse of s that is off by a few steps: the product's residual, exact in an fma, times the inverse.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, s, x), inv, q);
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(code));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r)));
}

// A group's scale: its e4m3 code, value and inverse (0 of 0).
struct Scale {
  uint32_t code;
  float value, inverse;
};
__device__ __forceinline__ Scale scale_of(float top) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(quotient(top, 6.0f, 1.0f / 6.0f)));
  Scale s;
  s.code = top <= 3.402823466e38f ? r : 0x7fu;  // NaN and infinities: the group's scale is NaN
  s.value = e4m3_value(s.code);
  s.inverse = s.code != 0u ? approximate_inverse(s.value) : 0.0f;
  return s;
}

// Eight elements under a scale as codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float* x, const Scale& s) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = quotient(x[j], s.value, s.inverse);
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(ROW_THREADS, 2) nsa_cache4_append_kernel(const __grid_constant__ Append4Args a) {
  using Ring = RowRing<T, 1>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[64];
  const Ring ring(smem);
  const int D = a.c.D, lanes = 1 << a.plan.lanes_log;
  RowPlace p = place_of(a.plan, a.tokens, {a.Hq, 2 * a.c.Hkv}, D);
  const bool is_q = p.side == 0;
  const uint32_t b = p.token / static_cast<uint32_t>(a.n), t = p.token % static_cast<uint32_t>(a.n);
  const int held = a.lens[b];
  if (a.new_lens != nullptr && static_cast<int>(t) >= a.new_lens[b]) p.rows = 0;
  // values lie as plain rows, keys and queries by their pairs
  const UnitMap m = unit_map(p.unit, a.rotary, INTERLEAVED), plain = unit_map(p.unit, 0, false);
  auto ask = [&](int r0) {
#pragma unroll
    for (int i = 0; i < Ring::BATCH; ++i) {
      const int h = p.head + (r0 + i) * p.head_step;
      const int x = is_q ? 0 : h < a.c.Hkv ? 1 : 2;  // q, k, v
      const T* row = static_cast<const T*>(a.x[x]) + b * a.stride[x][0] + t * a.stride[x][2] +
                     (x == 2 ? h - a.c.Hkv : h) * a.stride[x][1];
      const UnitMap& u = x == 2 ? plain : m;
      if (r0 + i < p.rows) ring.ask((r0 + i) % (2 * Ring::BATCH), 0, row + u.lo, u.hi - u.lo);
    }
    Ring::commit();
  };
  ask(0);
  ask(Ring::BATCH);
  // the token's slot of the cache (where it has one)
  size_t at = 0;
  bool kept = false;
  if (!is_q && p.rows > 0 && held >= 0) {
    const long long pos = static_cast<long long>(held) + t, lp = pos >> a.page_log;
    if (lp < a.c.max_pages) {
      const int id = a.c.table[static_cast<size_t>(b) * a.c.max_pages + lp];
      kept = id >= 0 && id < a.c.num_pages;
      at = (static_cast<size_t>(kept ? id : 0) * a.c.Hkv << a.page_log) + static_cast<size_t>(pos & (a.c.page - 1));
    }
  }
  const void* weight = a.weight[is_q ? 0 : 1];
  // (a block of values alone needs neither norm nor rotation)
  const bool keys = p.group * p.head_step * a.plan.rows < (is_q ? a.Hq : a.c.Hkv);
  const bool norm = weight != nullptr && keys, turn = m.freq >= 0 && keys;
  float c[8], w[8], g[UNIT];
  UnitMap2 map;
  if (norm || a.rotary > 0) {
#pragma unroll
    for (int j = 0; j < UNIT; ++j) g[j] = 1.0f;
    if (norm) load_weights(weight, a.w_f32 != 0, m, g);
    if (a.rotary > 0 && keys) block_turns(turns, a.inv_freq, a.rotary);
    if (turn) {
      unit_sincos(turns, m.freq, static_cast<int>(static_cast<uint32_t>(held) + t), a.factor, c, w);
      make_map<INTERLEAVED>(map, c, w, g);
    }
  }
  const float inv_d = 1.0f / static_cast<float>(D);
  // Where pairs are halves of more than 16 elements, a group of 16 is shared by two runs of eight that lie in two lanes
  // (or in either half of one): the lane and half of the run that shares a group with this lane's.
  const bool split = !is_q && keys && !INTERLEAVED && a.rotary > UNIT;
  auto mate_of = [&](int run, bool& hi) {
    const int half = a.rotary / UNIT, r = run ^ 1;  // runs of either half
    hi = r < 2 * half ? r >= half : (r & 1) != 0;
    return (threadIdx.x & 31 & ~(lanes - 1)) + (r < 2 * half ? (hi ? r - half : r) : r >> 1);
  };
  bool lo_hi = false, hi_hi = false;
  int lo_mate = 0, hi_mate = 0;
  if (split) {
    lo_mate = mate_of(m.lo >> 3, lo_hi);
    hi_mate = mate_of(m.hi >> 3, hi_hi);
  }

  for (int r0 = 0; r0 < p.most; r0 += Ring::BATCH) {
    Ring::wait();
#pragma unroll
    for (int i = 0; i < Ring::BATCH; ++i) {
      if (i > 0 && r0 + i >= p.most) break;
      const bool mine = r0 + i < p.rows;
      const int head = p.head + (r0 + i) * p.head_step;
      const bool value = !is_q && head >= a.c.Hkv;
      float x[UNIT];
      ring.take((r0 + i) % (2 * Ring::BATCH), 0, x);  // (anything where no row was asked for; it stays in its row)
      if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < UNIT; ++j) ss = fmaf(x[j], x[j], ss);
        const float rs = rsqrtf(fmaf(row_sum(ss, a.plan.lanes_log, true), inv_d, a.eps));
        if (!value) {
          if (turn) {
            apply_map<INTERLEAVED>(map, rs, x);
          } else {
#pragma unroll
            for (int j = 0; j < UNIT; ++j) x[j] *= rs * g[j];
          }
        }
      } else if (turn && !value) {
        apply_map<INTERLEAVED>(map, 1.0f, x);
      }
      if (is_q) {
        if (mine) {
          T* row = static_cast<T*>(a.q_out) + ((static_cast<size_t>(b) * a.Hq + head) * a.n + t) * D;
          store8(row + m.lo, x);
          store8(row + m.hi, x + 8);
        }
        continue;
      }
      const float* factors = value ? a.c.v_factor : a.c.k_factor;
      const int h = value ? head - a.c.Hkv : head;
      if (factors != nullptr && mine) {
        const float f = factors[h];
#pragma unroll
        for (int j = 0; j < UNIT; ++j) x[j] = __fdiv_rn(x[j], f);
      }
      float top_lo = 0.0f, top_hi = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top_lo = max_nan(top_lo, x[j]);
        top_hi = max_nan(top_hi, x[8 + j]);
      }
      const size_t row = at + (static_cast<size_t>(h) << a.page_log);
      uint8_t* codes = (value ? a.c.v : a.c.k) + row * (D / 2);
      uint8_t* scales = (value ? a.c.v_scale : a.c.k_scale) + row * (D / 16);
      float mate_of_lo = top_hi, mate_of_hi = top_lo;  // the other run's largest
      if (split) {
        const float lo_a = __shfl_sync(0xffffffffu, top_lo, lo_mate), lo_b = __shfl_sync(0xffffffffu, top_hi, lo_mate);
        const float hi_a = __shfl_sync(0xffffffffu, top_lo, hi_mate), hi_b = __shfl_sync(0xffffffffu, top_hi, hi_mate);
        if (!value) {
          mate_of_lo = lo_hi ? lo_b : lo_a;
          mate_of_hi = hi_hi ? hi_b : hi_a;
        }
      }
      if (!kept || !mine) continue;
      const Scale lo = scale_of(max_nan(top_lo, mate_of_lo));
      if (!split || value) {  // one group
        *reinterpret_cast<uint2*>(codes + p.unit * 8) = make_uint2(codes8(x, lo), codes8(x + 8, lo));
        scales[p.unit] = static_cast<uint8_t>(lo.code);
      } else {
        const Scale hi = scale_of(max_nan(top_hi, mate_of_hi));
        *reinterpret_cast<uint32_t*>(codes + m.lo / 2) = codes8(x, lo);
        *reinterpret_cast<uint32_t*>(codes + m.hi / 2) = codes8(x + 8, hi);
        if ((m.lo & 8) == 0) scales[m.lo / 16] = static_cast<uint8_t>(lo.code);
        if ((m.hi & 8) == 0) scales[m.hi / 16] = static_cast<uint8_t>(hi.code);
      }
    }
    ask(r0 + 2 * Ring::BATCH);
  }
}

// Keys and values that are neither normalised nor rotated, without queries: nothing is shared over the heads of a token,
// so a thread takes a group of 16 of STORE_ROWS tokens, of keys and of values, all on their way at once.  (By the kernel
// above, whose blocks load, work and store in step, a prompt of 32768 tokens of 4 heads of 128 took 36 us, now 19.3.)
template <typename T>
constexpr int STORE_ROWS = sizeof(T) == 2 ? 2 : 1;

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS, 4) nsa_cache4_store_kernel(const __grid_constant__ Append4Args a) {
  const int D = a.c.D, u = threadIdx.x & ((1 << a.plan.lanes_log) - 1), per = ROW_THREADS >> a.plan.lanes_log;
  const uint32_t tile = blockIdx.x % a.plan.tiles, bh = blockIdx.x / a.plan.tiles;
  const int h = static_cast<int>(bh % a.c.Hkv), b = static_cast<int>(bh / a.c.Hkv);
  const int t0 = static_cast<int>(tile) * per * STORE_ROWS<T> + (static_cast<int>(threadIdx.x) >> a.plan.lanes_log);
  const int held = a.lens[b], n = a.new_lens != nullptr ? min(a.n, a.new_lens[b]) : a.n;
  uint4 raw[STORE_ROWS<T>][2][sizeof(T)];
#pragma unroll
  for (int r = 0; r < STORE_ROWS<T>; ++r)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int t = t0 + r * per;
      const T* row = static_cast<const T*>(a.x[1 + s]) + b * a.stride[1 + s][0] + h * a.stride[1 + s][1] +
                     t * a.stride[1 + s][2] + u * UNIT;
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
        if (t < n) raw[r][s][i] = __ldg(reinterpret_cast<const uint4*>(row) + i);
    }
#pragma unroll
  for (int r = 0; r < STORE_ROWS<T>; ++r) {
    const int t = t0 + r * per;
    const long long pos = static_cast<long long>(held) + t, lp = pos >> a.page_log;
    if (t >= n || held < 0 || lp >= a.c.max_pages) continue;
    const int id = a.c.table[static_cast<size_t>(b) * a.c.max_pages + lp];
    if (id < 0 || id >= a.c.num_pages) continue;
    const size_t at =
        ((static_cast<size_t>(id) * a.c.Hkv + h) << a.page_log) + static_cast<size_t>(pos & (a.c.page - 1));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float x[UNIT], top = 0.0f;
      unpack<T>(raw[r][s], x);
      const float* factors = s ? a.c.v_factor : a.c.k_factor;
      if (factors != nullptr) {
        const float f = factors[h];
#pragma unroll
        for (int j = 0; j < UNIT; ++j) x[j] = __fdiv_rn(x[j], f);
      }
#pragma unroll
      for (int j = 0; j < UNIT; ++j) top = max_nan(top, x[j]);
      const Scale sc = scale_of(top);
      *reinterpret_cast<uint2*>((s ? a.c.v : a.c.k) + at * (D / 2) + u * 8) = make_uint2(codes8(x, sc), codes8(x + 8, sc));
      (s ? a.c.v_scale : a.c.k_scale)[at * (D / 16) + u] = static_cast<uint8_t>(sc.code);
    }
  }
}

constexpr int READ_ROWS = 4;  // tokens a thread reads, all on their way at once

struct Read4Args {
  Cache4 c;
  const int32_t *starts, *lens;
  void *k_out, *v_out;
  int n, page_log, lanes_log;
  uint32_t tiles;  // blocks over a sequence's tokens
};

// Eight elements a thread, of keys and of values: a word of codes and a scale each.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) nsa_cache4_read_kernel(const __grid_constant__ Read4Args a) {
  const int D = a.c.D, u = threadIdx.x & ((1 << a.lanes_log) - 1), per = ROW_THREADS >> a.lanes_log;
  const uint32_t tile = blockIdx.x % a.tiles, bh = blockIdx.x / a.tiles;
  const int h = static_cast<int>(bh % a.c.Hkv), b = static_cast<int>(bh / a.c.Hkv);
  const int t0 = static_cast<int>(tile) * per * READ_ROWS + (static_cast<int>(threadIdx.x) >> a.lanes_log);
  const int start = a.starts != nullptr ? a.starts[b] : 0, len = a.lens[b];
  const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.max_pages;
  uint32_t code[READ_ROWS][2], scale[READ_ROWS][2];
  int id[READ_ROWS];
#pragma unroll
  for (int r = 0; r < READ_ROWS; ++r) {
    const int t = t0 + r * per;
    const long long pos = static_cast<long long>(start) + t, lp = pos >> a.page_log;
    id[r] = t < a.n && start >= 0 && pos < len && lp < a.c.max_pages ? table[lp] : -1;
  }
#pragma unroll
  for (int r = 0; r < READ_ROWS; ++r) {
    code[r][0] = code[r][1] = scale[r][0] = scale[r][1] = 0u;
    if (id[r] >= 0 && id[r] < a.c.num_pages) {
      const size_t at = ((static_cast<size_t>(id[r]) * a.c.Hkv + h) << a.page_log) +
                        ((start + t0 + r * per) & (a.c.page - 1));
      code[r][0] = __ldg(reinterpret_cast<const uint32_t*>(a.c.k + at * (D / 2)) + u);
      code[r][1] = __ldg(reinterpret_cast<const uint32_t*>(a.c.v + at * (D / 2)) + u);
      scale[r][0] = __ldg(a.c.k_scale + at * (D / 16) + u / 2);
      scale[r][1] = __ldg(a.c.v_scale + at * (D / 16) + u / 2);
    }
  }
#pragma unroll
  for (int r = 0; r < READ_ROWS; ++r) {
    const int t = t0 + r * per;
    if (t >= a.n) break;
    const size_t at = (static_cast<size_t>(bh) * a.n + t) * D + 8 * u;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t x[4];
      f16_of_codes(code[r][s], x);
      const float* factor = s ? a.c.v_factor : a.c.k_factor;
      const float sv = e4m3_value(scale[r][s]);
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
        y[2 * i] = f.x * sv;
        y[2 * i + 1] = f.y * sv;
      }
      if (factor != nullptr) {
        const float f = factor[h];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= f;
      }
      store8(static_cast<T*>(s ? a.v_out : a.k_out) + at, y);
    }
  }
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

constexpr int APPEND_ROWS = 8;  // rows a thread walks at most

template <typename T>
int launch_append(const Append4Args& a, bool interleaved, cudaStream_t stream) {
  auto kern = interleaved ? nsa_cache4_append_kernel<T, true> : nsa_cache4_append_kernel<T, false>;
  const int smem = RowRing<T, 1>::bytes_for(kern, a.plan.rows);
  if (smem < 0) return ERR_LAUNCH;
  kern<<<a.plan.tiles * a.plan.all_groups, ROW_THREADS, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

template <typename T>
int launch_store(Append4Args& a, cudaStream_t stream) {
  a.plan.lanes_log = log2_of(a.c.D / UNIT);
  const int tokens = (ROW_THREADS >> a.plan.lanes_log) * STORE_ROWS<T>;  // of a block
  a.plan.tiles = (static_cast<uint32_t>(a.n) + tokens - 1) / tokens;
  const long long blocks = static_cast<long long>(a.c.B) * a.c.Hkv * a.plan.tiles;
  if (blocks > 0x7fffffffLL) return ERR_SHAPE;
  nsa_cache4_store_kernel<T><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
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
  a.Hq = r.Hq; a.n = r.n; a.rotary = r.rotary;
  a.w_f32 = r.weight_f32 ? 1 : 0; a.page_log = log2_of(r.cache.page);
  a.factor = r.factor; a.eps = r.eps;
  a.tokens = static_cast<long long>(r.cache.B) * r.n;
  if (r.q == nullptr && r.k_weight == nullptr && r.rotary == 0)
    return r.f32 ? launch_store<float>(a, stream) : launch_store<__nv_bfloat16>(a, stream);
  if (!plan_rows<2>(a.plan, a.tokens, {r.q != nullptr ? r.Hq : 0, 2 * r.cache.Hkv}, r.cache.D, APPEND_ROWS))
    return ERR_SHAPE;
  return r.f32 ? launch_append<float>(a, r.interleaved, stream)
               : launch_append<__nv_bfloat16>(a, r.interleaved, stream);
}

int launch_nsa_cache4_read(const Cache4& c, const int32_t* starts, const int32_t* lens, void* k_out, void* v_out,
                           int n, bool f32, cudaStream_t stream) {
  Read4Args a{};
  a.c = c;
  a.starts = starts; a.lens = lens;
  a.k_out = k_out; a.v_out = v_out;
  a.n = n; a.page_log = log2_of(c.page); a.lanes_log = log2_of(c.D / 8);
  const int tokens = (ROW_THREADS >> a.lanes_log) * READ_ROWS;  // of a block
  a.tiles = (static_cast<uint32_t>(n) + tokens - 1) / tokens;
  const long long blocks = static_cast<long long>(c.B) * c.Hkv * a.tiles;
  if (blocks > 0x7fffffffLL) return ERR_SHAPE;
  if (f32) nsa_cache4_read_kernel<float><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  else nsa_cache4_read_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), ROW_THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace bsa
