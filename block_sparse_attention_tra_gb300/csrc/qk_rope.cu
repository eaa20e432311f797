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
  int T, D, rotary, interleaved, w_f32;
  long long tokens;
  float factor, eps;
  RowTile tile;
  int q_groups, groups;  // blocks over the heads of q, of both
  long long q_blocks, k_blocks;  // blocks in all: rows of the workspace
};

// What a thread holds: its token, its unit of the rows, and its first head.
struct Place {
  int s, group, u, slot, head;
  long long tile, token, b;
  int t;
  bool live;
};
__device__ __forceinline__ Place place_of(const RopeArgs& a) {
  Place p;
  p.group = static_cast<int>(blockIdx.x % a.groups);
  p.tile = blockIdx.x / a.groups;
  p.s = p.group >= a.q_groups ? 1 : 0;
  if (p.s) p.group -= a.q_groups;
  p.u = threadIdx.x & ((1 << a.tile.lanes_log) - 1);
  p.slot = static_cast<int>(threadIdx.x) >> a.tile.lanes_log;
  p.token = (p.tile << a.tile.tokens_log) + (p.slot & ((1 << a.tile.tokens_log) - 1));
  p.head = p.group * row_heads(a.tile) + (p.slot >> a.tile.tokens_log);
  p.live = p.token < a.tokens && p.u * UNIT < a.D;
  // (all tokens together are a 31-bit number)
  p.b = p.live ? static_cast<uint32_t>(p.token) / static_cast<uint32_t>(a.T) : 0;
  p.t = p.live ? static_cast<int>(static_cast<uint32_t>(p.token) % static_cast<uint32_t>(a.T)) : 0;
  return p;
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS, 3) qk_rope_forward_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int AHEAD = sizeof(T) == 2 ? 2 : 1;  // rows on their way
  const Place p = place_of(a);
  const Side& sd = a.side[p.s];
  const bool il = a.interleaved != 0, norm = sd.w != nullptr;
  const int head_step = ROW_THREADS >> a.tile.lanes_log >> a.tile.tokens_log;
  const UnitMap m = unit_map(p.u, a.rotary, il);
  const T* src = static_cast<const T*>(sd.x) + p.b * sd.x_stride[0] + p.t * sd.x_stride[2];
  T* dst = static_cast<T*>(sd.out) + p.b * sd.out_stride[0] + p.t * sd.out_stride[2];
  RawUnit<T> raw[AHEAD];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int h = p.head + (r0 + i) * head_step;
      if (p.live && r0 + i < a.tile.rows && h < sd.H) raw[i].load(src + h * sd.x_stride[1], m);
      else raw[i].clear();
    }
  };
  fetch(0);
  float c[8], w[8], wt[UNIT];
  const bool turn = p.live && m.freq >= 0;
  if (turn)
    sincos8_of(a.inv_freq + m.freq, a.positions != nullptr ? a.positions[p.token] : p.t, a.factor, c, w);
  if (norm && p.live) load_weights(sd.w, a.w_f32 != 0, m, wt);
  const float inv_d = 1.0f / static_cast<float>(a.D);
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
      const int h = p.head + (r0 + i) * head_step;
      if (!p.live || h >= sd.H) continue;
      if (turn) rotate16(x, c, w, il);
      T* row = dst + h * sd.out_stride[1];
      store8(row + m.lo, x);
      store8(row + m.hi, x + 8);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS, 2) qk_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int AHEAD = sizeof(T) == 2 ? 2 : 1;  // rows on their way
  __shared__ float part[ROW_THREADS / 32][128];
  // the second launch's blocks may take the places that this one's leave (they wait for all of it)
  asm volatile("griddepcontrol.launch_dependents;");
  const Place p = place_of(a);
  const Side& sd = a.side[p.s];
  const bool il = a.interleaved != 0, norm = sd.w != nullptr;
  const int head_step = ROW_THREADS >> a.tile.lanes_log >> a.tile.tokens_log;
  const UnitMap m = unit_map(p.u, a.rotary, il);
  const T* src = static_cast<const T*>(sd.x) + p.b * sd.x_stride[0] + p.t * sd.x_stride[2];
  const T* up = static_cast<const T*>(sd.dy) + p.b * sd.dy_stride[0] + p.t * sd.dy_stride[2];
  T* dst = static_cast<T*>(sd.out) + p.b * sd.out_stride[0] + p.t * sd.out_stride[2];
  RawUnit<T> raw_x[AHEAD], raw_g[AHEAD];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int h = p.head + (r0 + i) * head_step;
      const bool in = p.live && r0 + i < a.tile.rows && h < sd.H;
      if (in) raw_g[i].load(up + h * sd.dy_stride[1], m);
      else raw_g[i].clear();
      if (in && norm) raw_x[i].load(src + h * sd.x_stride[1], m);
      else raw_x[i].clear();
    }
  };
  fetch(0);
  float c[8], w[8], wt[UNIT], dw[UNIT];
  const bool turn = p.live && m.freq >= 0;
  if (turn) {
    sincos8_of(a.inv_freq + m.freq, a.positions != nullptr ? a.positions[p.token] : p.t, a.factor, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = -w[j];  // the transpose
  }
#pragma unroll
  for (int j = 0; j < UNIT; ++j) wt[j] = dw[j] = 0.0f;
  if (norm && p.live) load_weights(sd.w, a.w_f32 != 0, m, wt);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  for (int r0 = 0; r0 < a.tile.rows; r0 += AHEAD) {
    if (r0 > 0) fetch(r0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (r0 + i >= a.tile.rows) break;
      float g[UNIT];
      raw_g[i].unpack(g);
      if (turn) rotate16(g, c, w, il);
      if (norm) {
        float x[UNIT], ss = 0.0f, dot = 0.0f;
        raw_x[i].unpack(x);
#pragma unroll
        for (int j = 0; j < UNIT; ++j) ss = fmaf(x[j], x[j], ss);
        const float r = rsqrtf(fmaf(row_sum(ss, a.tile.lanes_log), inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {
          x[j] *= r;
          dw[j] = fmaf(g[j], x[j], dw[j]);
          g[j] *= wt[j];
          dot = fmaf(g[j], x[j], dot);
        }
        dot = row_sum(dot, a.tile.lanes_log) * inv_d;
#pragma unroll
        for (int j = 0; j < UNIT; ++j) g[j] = r * fmaf(-x[j], dot, g[j]);
      }
      const int h = p.head + (r0 + i) * head_step;
      if (!p.live || h >= sd.H) continue;
      T* row = dst + h * sd.out_stride[1];
      store8(row + m.lo, g);
      store8(row + m.hi, g + 8);
    }
  }
  if (!norm) return;
  // the block's rows: lanes of a warp that hold the same unit, then the warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < UNIT; ++j)
    for (int d = 16; d >= 1 << a.tile.lanes_log; d >>= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], d);
  if (lane < 1 << a.tile.lanes_log && p.u * UNIT < a.D) {
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
    const long long row = p.s ? a.q_blocks + p.tile * (a.groups - a.q_groups) + p.group : p.tile * a.q_groups + p.group;
    a.ws[row * a.D + j] = sum;
  }
}

// Adds up the blocks' rows: one block for 16 columns of one tensor's weights.
__global__ void __launch_bounds__(256) qk_rope_weights_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float4 part[64][4];
  const int per = a.D / 16, s = blockIdx.x / per, col = blockIdx.x % per * 16 + (threadIdx.x & 3) * 4;
  const int lane = threadIdx.x >> 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel is complete
  const Side& sd = a.side[s];
  if (sd.dw == nullptr) return;
  const long long rows = s ? a.k_blocks : a.q_blocks;
  const float* from = a.ws + (s ? a.q_blocks : 0) * a.D + col;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (long long r = lane; r < rows; r += 64) {
    const float4 v = *reinterpret_cast<const float4*>(from + r * a.D);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  part[lane][threadIdx.x & 3] = sum;
  __syncthreads();
  if (threadIdx.x >= 16) return;
  float total = 0.0f;
  for (int k = 0; k < 64; ++k) total += reinterpret_cast<const float*>(&part[k][0])[threadIdx.x];
  static_cast<float*>(sd.dw)[blockIdx.x % per * 16 + threadIdx.x] = total;
}

// Rows a thread walks at most: sines, weights and the weights' gradients are paid once for them.
constexpr int FORWARD_ROWS = 8, BACKWARD_ROWS = 8;

// Fills in the blocks; false if there are too many.
bool plan(RopeArgs& a, int B, int most) {
  a.tokens = static_cast<long long>(B) * a.T;
  const int Hq = a.side[0].H, Hk = a.side[1].H;
  a.tile = row_tile(a.tokens, Hq + Hk, a.D, most);
  const int heads = row_heads(a.tile);
  a.q_groups = (Hq + heads - 1) / heads;
  a.groups = a.q_groups + (Hk + heads - 1) / heads;
  const long long tiles = (a.tokens + (1LL << a.tile.tokens_log) - 1) >> a.tile.tokens_log;
  a.q_blocks = tiles * a.q_groups;
  a.k_blocks = tiles * (a.groups - a.q_groups);
  return a.q_blocks + a.k_blocks <= 0x7fffffffLL;
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
  a.T = r.T; a.D = r.D; a.rotary = r.rotary; a.interleaved = r.interleaved ? 1 : 0;
  a.w_f32 = r.weight_f32 ? 1 : 0;
  a.factor = r.factor; a.eps = r.eps;
  return a;
}

}  // namespace

int launch_qk_rope_forward(const RopeCall& r, cudaStream_t stream) {
  RopeArgs a = args_of(r);
  if (!plan(a, r.B, FORWARD_ROWS)) return ERR_SHAPE;
  const unsigned blocks = static_cast<unsigned>(a.q_blocks + a.k_blocks);
  if (r.f32) qk_rope_forward_kernel<float><<<blocks, ROW_THREADS, 0, stream>>>(a);
  else qk_rope_forward_kernel<__nv_bfloat16><<<blocks, ROW_THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OK : ERR_LAUNCH;
}

size_t qk_rope_backward_workspace_bytes(int B, int Hq, int Hkv, int T, int D) {
  RopeArgs a{};
  a.side[0].H = Hq;
  a.side[1].H = Hkv;
  a.T = T; a.D = D;
  if (!plan(a, B, BACKWARD_ROWS)) return 0;
  return (static_cast<size_t>(a.q_blocks + a.k_blocks) * D * sizeof(float) + 255) / 256 * 256;
}

int launch_qk_rope_backward(const RopeCall& r, void* workspace, cudaStream_t stream) {
  RopeArgs a = args_of(r);
  a.ws = static_cast<float*>(workspace);
  if (!plan(a, r.B, BACKWARD_ROWS)) return ERR_SHAPE;
  const unsigned blocks = static_cast<unsigned>(a.q_blocks + a.k_blocks);
  if (r.f32) qk_rope_backward_kernel<float><<<blocks, ROW_THREADS, 0, stream>>>(a);
  else qk_rope_backward_kernel<__nv_bfloat16><<<blocks, ROW_THREADS, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ERR_LAUNCH;
  if (r.q_weight == nullptr && r.k_weight == nullptr) return OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (a.D / 16)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_rope_weights_kernel, a) == cudaSuccess ? OK : ERR_LAUNCH;
}

}  // namespace bsa
