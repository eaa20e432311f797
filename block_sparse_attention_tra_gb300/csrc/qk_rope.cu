// qk_rope.cu -- the RMS norm of query and key heads and their rotation by
// position, in one pass over the rows, and its gradients.
//
// For a row x of D elements (one head of one token at position m), with r =
// (mean x^2 + eps)^-1/2, weights w and R the rotation of nsa_cache.cu times a
// factor on the rotated elements:
//     y = R (r x w).
// Backward, with g = R^T dy and h = r x:
//     dw = sum over rows of g h,   dx = r (g w - h mean(g w h)).
// Without weights there is no norm: y = R x, dx = R^T dy.
//
// Memory bounds both: each element is read once and written once (backward: x
// and dy read, dx written), nothing else grows with the rows.  A thread holds
// 16 elements of a row -- in halves, the two runs of eight that are rotated
// into each other -- and keeps its token's sines and cosines and its weights
// over the heads it walks; a row's lanes add up their squares by shuffles.  The
// weights' gradients stay in registers over those heads, are added up over the
// block and left as one row of the workspace per block; a second launch adds
// the rows in a fixed order, so results repeat bit for bit.
#include "kernels.h"
#include "rope.cuh"

namespace bsa {
namespace {

// One of the two tensors, strides in elements.
struct Side {
  const void *x, *dy, *w;
  void *out, *dw;
  long long x_stride[3], dy_stride[3], out_stride[3];  // batch, head, token
  int H;
};
struct RopeArgs {
  Side side[2];
  const int32_t* positions;
  const float* inv_freq;
  float* ws;
  int T, D, rotary, w_f32;
  long long tokens;
  float factor, eps;
  RowPlan<2> plan;
};

// The first run of eight of the thread's unit in its first row.
template <typename T>
__device__ __forceinline__ T* first_row(T* x, const long long (&stride)[3], uint32_t b, int head, uint32_t t, int lo) {
  return x + b * stride[0] + head * stride[1] + t * stride[2] + lo;
}

__device__ __forceinline__ int position_of(const RopeArgs& a, const RowPlace& p, uint32_t t) {
  return a.positions != nullptr ? a.positions[p.token] : static_cast<int>(t);
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(ROW_THREADS, 3) qk_rope_forward_kernel(const __grid_constant__ RopeArgs a) {
  using Ring = RowRing<T, 1>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[64];
  const Ring ring(smem);
  const RowPlace p = place_of(a.plan, a.tokens, {a.side[0].H, a.side[1].H}, a.D);
  const Side& sd = a.side[p.side];
  const bool norm = sd.w != nullptr;
  const UnitMap m = unit_map(p.unit, a.rotary, INTERLEAVED);
  const int apart = m.hi - m.lo;
  const uint32_t b = p.token / static_cast<uint32_t>(a.T), t = p.token % static_cast<uint32_t>(a.T);
  const T* src = first_row(static_cast<const T*>(sd.x), sd.x_stride, b, p.head, t, m.lo);
  T* dst = first_row(static_cast<T*>(sd.out), sd.out_stride, b, p.head, t, m.lo);
  const long long src_step = p.head_step * sd.x_stride[1], dst_step = p.head_step * sd.out_stride[1];
  auto ask = [&](int r0) {
#pragma unroll
    for (int i = 0; i < Ring::BATCH; ++i) {
      if (r0 + i < p.rows) ring.ask((r0 + i) % (2 * Ring::BATCH), 0, src, apart);
      src += src_step;
    }
    Ring::commit();
  };
  ask(0);
  ask(Ring::BATCH);
  float c[8], w[8], g[UNIT];
#pragma unroll
  for (int j = 0; j < UNIT; ++j) g[j] = 1.0f;
  const bool turn = m.freq >= 0, in_row = p.unit * UNIT < a.D;
  if (norm && in_row) load_weights(sd.w, a.w_f32 != 0, m, g);
  UnitMap2 map;
  if (a.rotary > 0) block_turns(turns, a.inv_freq, a.rotary);
  if (turn) {
    unit_sincos(turns, m.freq, position_of(a, p, t), a.factor, c, w);
    make_map<INTERLEAVED>(map, c, w, g);
  } else {  // the weights alone, in the map's place
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      map.aa[j] = g[INTERLEAVED ? 2 * j : j];
      map.bb[j] = g[INTERLEAVED ? 2 * j + 1 : 8 + j];
      map.ab[j] = map.ba[j] = 0.0f;
    }
  }
  const float inv_d = 1.0f / static_cast<float>(a.D);
  for (int r0 = 0; r0 < p.most; r0 += Ring::BATCH) {
    Ring::wait();
#pragma unroll
    for (int i = 0; i < Ring::BATCH; ++i) {
      if (i > 0 && r0 + i >= p.most) break;
      const bool mine = r0 + i < p.rows;
      float x[UNIT];
      ring.take((r0 + i) % (2 * Ring::BATCH), 0, x);  // (anything where no row was asked for; it stays in its row)
      float s = 1.0f;
      if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < UNIT; ++j) ss = fmaf(x[j], x[j], ss);
        s = rsqrtf(fmaf(row_sum(ss, a.plan.lanes_log, in_row), inv_d, a.eps));
      }
      if (mine) {
        if (turn) {
          apply_map<INTERLEAVED>(map, s, x);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[INTERLEAVED ? 2 * j : j] *= s * map.aa[j];
            x[INTERLEAVED ? 2 * j + 1 : 8 + j] *= s * map.bb[j];
          }
        }
        store8(dst, x);
        store8(dst + apart, x + 8);
      }
      dst += dst_step;
    }
    ask(r0 + 2 * Ring::BATCH);
  }
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(ROW_THREADS, 2) qk_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
  using Ring = RowRing<T, 2>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[64];
  // the second launch's blocks may take the places that this one's leave (they wait for all of it)
  asm volatile("griddepcontrol.launch_dependents;");
  const Ring ring(smem);
  const RowPlace p = place_of(a.plan, a.tokens, {a.side[0].H, a.side[1].H}, a.D);
  const Side& sd = a.side[p.side];
  const bool norm = sd.w != nullptr;
  const UnitMap m = unit_map(p.unit, a.rotary, INTERLEAVED);
  const int apart = m.hi - m.lo;
  const uint32_t b = p.token / static_cast<uint32_t>(a.T), t = p.token % static_cast<uint32_t>(a.T);
  const T* src = first_row(static_cast<const T*>(sd.x), sd.x_stride, b, p.head, t, m.lo);
  const T* up = first_row(static_cast<const T*>(sd.dy), sd.dy_stride, b, p.head, t, m.lo);
  T* dst = first_row(static_cast<T*>(sd.out), sd.out_stride, b, p.head, t, m.lo);
  const long long src_step = p.head_step * sd.x_stride[1], up_step = p.head_step * sd.dy_stride[1];
  const long long dst_step = p.head_step * sd.out_stride[1];
  auto ask = [&](int r0) {
#pragma unroll
    for (int i = 0; i < Ring::BATCH; ++i) {
      if (r0 + i < p.rows) {
        ring.ask((r0 + i) % (2 * Ring::BATCH), 0, up, apart);
        if (norm) ring.ask((r0 + i) % (2 * Ring::BATCH), 1, src, apart);
      }
      up += up_step;
      src += src_step;
    }
    Ring::commit();
  };
  ask(0);
  ask(Ring::BATCH);
  float c[8], w[8], wt[UNIT], dw[UNIT];
#pragma unroll
  for (int j = 0; j < UNIT; ++j) wt[j] = dw[j] = 0.0f;
  const bool turn = m.freq >= 0, in_row = p.unit * UNIT < a.D;
  if (norm && in_row) load_weights(sd.w, a.w_f32 != 0, m, wt);
  if (a.rotary > 0) block_turns(turns, a.inv_freq, a.rotary);
  if (turn) {
    unit_sincos(turns, m.freq, position_of(a, p, t), a.factor, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = -w[j];  // the transpose
  }
  const float inv_d = 1.0f / static_cast<float>(a.D);
  for (int r0 = 0; r0 < p.most; r0 += Ring::BATCH) {
    Ring::wait();
#pragma unroll
    for (int i = 0; i < Ring::BATCH; ++i) {
      if (i > 0 && r0 + i >= p.most) break;
      const bool mine = r0 + i < p.rows;
      float g[UNIT], x[UNIT];
      ring.take((r0 + i) % (2 * Ring::BATCH), 0, g);  // (anything where no row was asked for; it stays in its row)
      if (turn) rotate16(g, c, w, INTERLEAVED);
      if (norm) {
        ring.take((r0 + i) % (2 * Ring::BATCH), 1, x);
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < UNIT; ++j) ss = fmaf(x[j], x[j], ss);
        const float rs = rsqrtf(fmaf(row_sum(ss, a.plan.lanes_log, in_row), inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {  // r g, the weights' gradient r g x, then z = r g w
          g[j] *= rs;
          if (mine) dw[j] = fmaf(g[j], x[j], dw[j]);
          g[j] *= wt[j];
          dot = fmaf(g[j], x[j], dot);
        }
        const float k = row_sum(dot, a.plan.lanes_log, in_row) * inv_d * rs * rs;  // dx = z - x r^2 mean(z x)
#pragma unroll
        for (int j = 0; j < UNIT; ++j) g[j] = fmaf(-k, x[j], g[j]);
      }
      if (mine) {
        store8(dst, g);
        store8(dst + apart, g + 8);
      }
      dst += dst_step;
    }
    ask(r0 + 2 * Ring::BATCH);
  }
  if (!norm) return;
  // the block's sums: the lanes of a warp that hold the same unit, then the warps (over the ring)
  float(*part)[128] = reinterpret_cast<float(*)[128]>(smem);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < UNIT; ++j)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      if (d >= 1 << a.plan.lanes_log) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], d);
  if (lane < 1 << a.plan.lanes_log && p.unit * UNIT < a.D) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      part[warp][m.lo + j] = dw[j];
      part[warp][m.hi + j] = dw[8 + j];
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < a.D; j += ROW_THREADS) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < ROW_THREADS / 32; ++k) sum += part[k][j];
    const size_t row = p.side ? static_cast<size_t>(a.plan.tiles) * a.plan.groups[0] : 0;
    a.ws[(row + static_cast<size_t>(p.tile) * a.plan.groups[p.side] + p.group) * a.D + j] = sum;
  }
}

// Adds up the blocks' rows: one block for 16 columns of one tensor's weights, four columns a thread.
// (Roundings that a row's product goes through in all: up to 16 rows of a thread, 5 shuffles and 8 warps above, the 256th
// part of the blocks, 3 shuffles and 32 warps here.)
constexpr int SUM_THREADS = 1024;
__global__ void __launch_bounds__(SUM_THREADS) qk_rope_weights_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float4 part[SUM_THREADS / 32][4];
  const int per = a.D / 16, s = blockIdx.x / per, col = blockIdx.x % per * 16;
  const Side& sd = a.side[s];
  if (sd.dw == nullptr) return;
  const size_t rows = static_cast<size_t>(a.plan.tiles) * a.plan.groups[s];
  const float* from = a.ws + (s ? static_cast<size_t>(a.plan.tiles) * a.plan.groups[0] : 0) * a.D + col +
                      (threadIdx.x & 3) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel is complete
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (size_t r = threadIdx.x >> 2; r < rows; r += SUM_THREADS / 4) {
    const float4 v = *reinterpret_cast<const float4*>(from + r * a.D);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
#pragma unroll
  for (int d = 16; d >= 4; d >>= 1) {
    sum.x += __shfl_xor_sync(0xffffffffu, sum.x, d);
    sum.y += __shfl_xor_sync(0xffffffffu, sum.y, d);
    sum.z += __shfl_xor_sync(0xffffffffu, sum.z, d);
    sum.w += __shfl_xor_sync(0xffffffffu, sum.w, d);
  }
  if ((threadIdx.x & 31) < 4) part[threadIdx.x >> 5][threadIdx.x & 3] = sum;
  __syncthreads();
  if (threadIdx.x >= 16) return;
  float total = 0.0f;
#pragma unroll
  for (int k = 0; k < SUM_THREADS / 32; ++k) total += reinterpret_cast<const float*>(&part[k][0])[threadIdx.x];
  static_cast<float*>(sd.dw)[col + threadIdx.x] = total;
}

// Rows a thread walks at most: sines, weights and the sums' reduction are paid once for them.
constexpr int MOST_ROWS = 16;
bool plan(RopeArgs& a, int B) {
  a.tokens = static_cast<long long>(B) * a.T;
  return plan_rows<2>(a.plan, a.tokens, {a.side[0].H, a.side[1].H}, a.D, MOST_ROWS);
}

RopeArgs args_of(const RopeCall& r) {
  RopeArgs a{};
  const void *x[2] = {r.q, r.k}, *dy[2] = {r.dq_out, r.dk_out}, *w[2] = {r.q_weight, r.k_weight};
  void *out[2] = {r.q_out, r.k_out}, *dw[2] = {r.dq_weight, r.dk_weight};
  for (int s = 0; s < 2; ++s) {
    Side& d = a.side[s];
    d.x = x[s]; d.dy = dy[s]; d.w = w[s]; d.out = out[s]; d.dw = dw[s];
    d.H = s ? r.Hkv : r.Hq;
    for (int i = 0; i < 3; ++i) {
      d.x_stride[i] = r.x_stride[s][i];
      d.dy_stride[i] = r.dy_stride[s][i];
      d.out_stride[i] = r.out_stride[s][i];
    }
  }
  a.positions = r.positions;
  a.inv_freq = r.inv_freq;
  a.T = r.T; a.D = r.D; a.rotary = r.rotary;
  a.w_f32 = r.weight_f32 ? 1 : 0;
  a.factor = r.factor; a.eps = r.eps;
  return a;
}

template <typename T>
int launch_forward(const RopeArgs& a, bool interleaved, cudaStream_t stream) {
  auto kern = interleaved ? qk_rope_forward_kernel<T, true> : qk_rope_forward_kernel<T, false>;
  const int smem = RowRing<T, 1>::bytes_for(kern, a.plan.rows);
  if (smem < 0) return ERR_LAUNCH;
  kern<<<a.plan.tiles * a.plan.all_groups, ROW_THREADS, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}
template <typename T>
int launch_backward(const RopeArgs& a, bool interleaved, cudaStream_t stream) {
  auto kern = interleaved ? qk_rope_backward_kernel<T, true> : qk_rope_backward_kernel<T, false>;
  const int smem = RowRing<T, 2>::bytes_for(kern, a.plan.rows);
  if (smem < 0) return ERR_LAUNCH;
  kern<<<a.plan.tiles * a.plan.all_groups, ROW_THREADS, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace

int launch_qk_rope_forward(const RopeCall& r, cudaStream_t stream) {
  RopeArgs a = args_of(r);
  if (!plan(a, r.B)) return ERR_SHAPE;
  return r.f32 ? launch_forward<float>(a, r.interleaved, stream)
               : launch_forward<__nv_bfloat16>(a, r.interleaved, stream);
}

size_t qk_rope_backward_workspace_bytes(int B, int Hq, int Hkv, int T, int D) {
  RopeArgs a{};
  a.side[0].H = Hq;
  a.side[1].H = Hkv;
  a.T = T; a.D = D;
  if (!plan(a, B)) return 0;
  return (static_cast<size_t>(a.plan.tiles) * a.plan.all_groups * D * sizeof(float) + 255) / 256 * 256;
}

int launch_qk_rope_backward(const RopeCall& r, void* workspace, cudaStream_t stream) {
  RopeArgs a = args_of(r);
  a.ws = static_cast<float*>(workspace);
  if (!plan(a, r.B)) return ERR_SHAPE;
  const int st = r.f32 ? launch_backward<float>(a, r.interleaved, stream)
                       : launch_backward<__nv_bfloat16>(a, r.interleaved, stream);
  if (st != OK || (r.q_weight == nullptr && r.k_weight == nullptr)) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (a.D / 16)));
  cfg.blockDim = dim3(SUM_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_rope_weights_kernel, a) == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace bsa
