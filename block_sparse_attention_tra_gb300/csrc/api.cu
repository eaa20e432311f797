// api.cu -- the C ABI of libbsa.so (declared in include/bsa.h): argument
// validation, dtype / head-dim dispatch and launch on the caller's stream.
// Validation happens on the host before any CUDA call, so a bad argument
// returns an error without touching the device.
#include <math.h>

#include <atomic>
#include <mutex>

#include "../../include/bsa.h"
#include "kernels.h"
#include "ptx.cuh"

namespace bsa {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The library's own stream-ordered memory pool on `dev`, created on first use.
// Its release threshold keeps freed temporaries mapped, so repeated calls
// recycle the same memory instead of mapping it again each time; the
// caller's default pool is left untouched.
cudaMemPool_t scratch_pool(int dev) {
  constexpr int MAX_DEVICES = 64;
  static std::mutex mu;
  static cudaMemPool_t pools[MAX_DEVICES] = {};
  if (dev < 0 || dev >= MAX_DEVICES) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (pools[dev] == nullptr) {
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaMemPool_t pool = nullptr;
    if (cudaMemPoolCreate(&pool, &props) != cudaSuccess) return nullptr;
    uint64_t keep = 1ull << 30;  // keep up to 1 GiB of freed temporaries mapped
    cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
    pools[dev] = pool;
  }
  return pools[dev];
}

// Sizes and parameters of the NSA selection entry points (pointers aside).
int check_nsa_shape(int B, int Hq, int Hkv, int T, int D, int block_size, int S) {
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || D < 1 || block_size < 1 || S < 1) return BSA_ERR_SHAPE;
  if (Hq % Hkv != 0) return BSA_ERR_SHAPE;
  if (T % block_size != 0) return BSA_ERR_SHAPE;
  if (S > 32) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * Hq * T * D >= (1LL << 40)) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * Hq > 0x7fffffffLL || static_cast<long long>(B) * Hkv * T * S >= (1LL << 40))
    return BSA_ERR_SHAPE;
  if (D != 16 && D != 32 && D != 64 && D != 128) return BSA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return BSA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

// The split-K form is built for 64-token blocks of 64 or 128 dims.
bool fsa_shape_supported(int D, int block_size) { return block_size == 64 && (D == 64 || D == 128); }

int check_nsa_args(const void* q, const void* k, const void* v, const int32_t* block_idx, const void* out,
                   const float* lse, int B, int Hq, int Hkv, int T, int D, int block_size, int S) {
  if (q == nullptr || k == nullptr || v == nullptr || block_idx == nullptr || out == nullptr)
    return BSA_ERR_NULLPTR;
  const int sh = check_nsa_shape(B, Hq, Hkv, T, D, block_size, S);
  if (sh != BSA_OK) return sh;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(block_idx) & 3u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return BSA_ERR_ALIGN;
  return BSA_OK;
}

// Sizes of the paged-cache entry points.
int check_cache_shape(int B, int Hq, int Hkv, int D, int page_size, int max_pages, int num_pages) {
  if (B < 1 || Hq < 1 || Hkv < 1 || D < 1 || page_size < 1 || max_pages < 1 || num_pages < 1) return BSA_ERR_SHAPE;
  if (Hq % Hkv != 0) return BSA_ERR_SHAPE;
  // positions and (sequence, head) pairs are 32-bit numbers
  if (static_cast<long long>(max_pages) * page_size > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * Hq > 0x7fffffffLL || static_cast<long long>(B) * max_pages >= (1LL << 40))
    return BSA_ERR_SHAPE;
  if (static_cast<long long>(num_pages) * Hkv >= (1LL << 40) / (static_cast<long long>(page_size) * D))
    return BSA_ERR_SHAPE;
  // (page, head) pairs of the pool are a tensor map's coordinate
  if (static_cast<long long>(num_pages) * Hkv > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (D != 16 && D != 32 && D != 64 && D != 128) return BSA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return BSA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool finite_value(float x) { return fabsf(x) <= 3.402823466e38f; }

// Norm and rotation of rows: sizes and parameters of qk_norm_rope and nsa_cache4_append.
int check_rows(int D, int rotary_dim, float rotary_scale, float eps) {
  if (D < 16 || D > 128 || D % 16 != 0) return BSA_ERR_UNSUPPORTED;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0) return BSA_ERR_UNSUPPORTED;
  if (!finite_value(rotary_scale) || !(eps > 0.0f) || !finite_value(eps)) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}
// `count` tensors' strides (batch, head, token) from the caller's list, or those of contiguous [., heads[i], T, D].
int take_strides(const int64_t* from, int count, const int* heads, int T, int D, int elsize, int64_t (*to)[3]) {
  for (int i = 0; i < count; ++i) {
    const int64_t own[3] = {static_cast<int64_t>(heads[i]) * T * D, static_cast<int64_t>(T) * D, D};
    for (int j = 0; j < 3; ++j) {
      to[i][j] = from != nullptr ? from[3 * i + j] : own[j];
      if (to[i][j] < 0 || to[i][j] >= (1LL << 40)) return BSA_ERR_SHAPE;
      if (to[i][j] * elsize % 16 != 0) return BSA_ERR_ALIGN;
    }
  }
  return BSA_OK;
}
// A written tensor's rows are all its own.
bool repeats_rows(const int64_t (&to)[3], int B, int H, int T) {
  return (to[0] == 0 && B > 1) || (to[1] == 0 && H > 1) || (to[2] == 0 && T > 1);
}
int check_dtypes(int dtype, int weight_dtype) {
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  if (weight_dtype != BSA_F32 && weight_dtype != BSA_BF16) return BSA_ERR_DTYPE;
  return BSA_OK;
}
int check_rope_shape(int B, int Hq, int Hkv, int T, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || Hq > 65535 || Hkv > 65535) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * T > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * T * (Hq > Hkv ? Hq : Hkv) >= (1LL << 40) / (D > 0 ? D : 1)) return BSA_ERR_SHAPE;
  return BSA_OK;
}
// The 4-bit cache's tensors.
int check_cache4(const Cache4& c, int Hq) {
  if (c.k == nullptr || c.v == nullptr || c.k_scale == nullptr || c.v_scale == nullptr || c.table == nullptr)
    return BSA_ERR_NULLPTR;
  const int sh = check_cache_shape(c.B, Hq, c.Hkv, c.D, c.page, c.max_pages, c.num_pages);
  if (sh != BSA_OK) return sh;
  const void* ptrs[4] = {c.k, c.v, c.k_scale, c.v_scale};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  return aligned4(c.k_factor) && aligned4(c.v_factor) && aligned4(c.table) ? BSA_OK : BSA_ERR_ALIGN;
}
Cache4 cache4_of(const void* k, const void* v, const void* k_scale, const void* v_scale, const float* k_factor,
                 const float* v_factor, const int32_t* table, int B, int Hkv, int D, int page, int max_pages,
                 int num_pages) {
  auto bytes = [](const void* p) { return static_cast<uint8_t*>(const_cast<void*>(p)); };
  return {bytes(k), bytes(v), bytes(k_scale), bytes(v_scale), k_factor, v_factor, table,
          B,        Hkv,      D,              page,           max_pages, num_pages};
}

// The kernels are built for sm_103a only; refuse other devices up front
// instead of failing inside the launch.
// (Asked once for each device.)
int check_device() {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<int> known[MAX_DEVICES];  // 0: not asked, 1: fits, 2: does not
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return ERR_DEVICE;
  if (dev < MAX_DEVICES && known[dev].load(std::memory_order_relaxed) != 0)
    return known[dev].load(std::memory_order_relaxed) == 1 ? OK : ERR_DEVICE;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return ERR_DEVICE;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return ERR_DEVICE;
  const bool fits = major == 10 && minor == 3;
  if (dev < MAX_DEVICES) known[dev].store(fits ? 1 : 2, std::memory_order_relaxed);
  return fits ? OK : ERR_DEVICE;
}

}  // namespace

int encode_tmap_3d(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                   uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return ERR_DEVICE;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
  const cuuint32_t box[3] = {box0, box1, box2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? OK : ERR_SHAPE;
}

int encode_tmap_3d_u8(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                       uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return ERR_DEVICE;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
  const cuuint32_t box[3] = {box0, box1, box2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? OK : ERR_SHAPE;
}

int encode_tmap_2d_f32(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t stride1_bytes,
                      uint32_t box0, uint32_t box1) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return ERR_DEVICE;
  const cuuint64_t dims[2] = {d0, d1};
  const cuuint64_t strides[1] = {stride1_bytes};
  const cuuint32_t box[2] = {box0, box1};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? OK : ERR_SHAPE;
}

int encode_tmap_3d_f32(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                       uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return ERR_DEVICE;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
  const cuuint32_t box[3] = {box0, box1, box2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? OK : ERR_SHAPE;
}

int sm_count() {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<int> counts[MAX_DEVICES] = {};  // 0 = not read yet; callers may race, all store one value
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return 0;
  int n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace bsa

using namespace bsa;

extern "C" {

int tra_forward(const void* q, const void* k, const void* v, void* out, int B, int H, int T, int D, float beta,
                float p, int dtype, cudaStream_t stream) {
  return tra_forward_ex(q, k, v, out, B, H, T, D, beta, p, dtype, 0, stream);
}

int tra_forward_ex(const void* q, const void* k, const void* v, void* out, int B, int H, int T, int D, float beta,
                   float p, int dtype, int flags, cudaStream_t stream) {
  if ((flags & ~BSA_TRA_SQRT_HALF_POWERS) != 0) return BSA_ERR_UNSUPPORTED;
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr) return BSA_ERR_NULLPTR;
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  if (B < 1 || H < 1 || T < 1 || D < 1) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * T * D >= (1LL << 40)) return BSA_ERR_SHAPE;
  if (!tra_head_dim_supported(D)) return BSA_ERR_UNSUPPORTED;
  if (!isfinite(beta) || !isfinite(p) || !(p > 0.0f)) return BSA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return BSA_ERR_ALIGN;
  const int dv = check_device();
  if (dv != OK) return dv;
  if (dtype == BSA_F32)
    return launch_tra_f32(static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v),
                          static_cast<float*>(out), B, H, T, D, beta, p, stream);
  return launch_tra_bf16(q, k, v, out, B, H, T, D, beta, p, (flags & BSA_TRA_SQRT_HALF_POWERS) != 0, stream);
}

size_t tra_forward_host_workspace_size(int B, int H, int T, int D, int dtype) {
  if (dtype != BSA_F32 && dtype != BSA_BF16) return 0;
  if (B < 1 || H < 1 || T < 1 || !tra_head_dim_supported(D)) return 0;
  if (static_cast<long long>(B) * H > 0x7fffffffLL || static_cast<long long>(B) * H * T * D >= (1LL << 40)) return 0;
  return tra_host_workspace_bytes(static_cast<long long>(B) * H, T, D, dtype == BSA_F32 ? 4 : 2);
}

int tra_forward_host(const void* q, const void* k, const void* v, void* out, int B, int H, int T, int D, float beta,
                     float p, int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || workspace == nullptr) return BSA_ERR_NULLPTR;
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  if (B < 1 || H < 1 || T < 1 || D < 1) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * T * D >= (1LL << 40)) return BSA_ERR_SHAPE;
  if (!tra_head_dim_supported(D)) return BSA_ERR_UNSUPPORTED;
  if (!isfinite(beta) || !isfinite(p) || !(p > 0.0f)) return BSA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return BSA_ERR_ALIGN;
  if (workspace_bytes < tra_forward_host_workspace_size(B, H, T, D, dtype)) return BSA_ERR_SCRATCH_LIMIT;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_tra_host(q, k, v, out, B, H, T, D, beta, p, dtype == BSA_F32, workspace, stream);
}

int tra_backward_ex(const void* q, const void* k, const void* v, const void* dout, void* dq, void* dk, void* dv,
                    int B, int H, int T, int D, float beta, float p, int dtype, int flags, cudaStream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || dout == nullptr || dq == nullptr || dk == nullptr ||
      dv == nullptr)
    return BSA_ERR_NULLPTR;
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  if (B < 1 || H < 1 || T < 1 || D < 1) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * T * D >= (1LL << 40)) return BSA_ERR_SHAPE;
  if (!tra_head_dim_supported(D)) return BSA_ERR_UNSUPPORTED;
  if (!isfinite(beta) || !isfinite(p) || !(p > 0.0f)) return BSA_ERR_UNSUPPORTED;
  if ((flags & ~BSA_TRA_BWD_DETERMINISTIC) != 0) return BSA_ERR_UNSUPPORTED;
  const void* ptrs[7] = {q, k, v, dout, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  const int dvs = check_device();
  if (dvs != OK) return dvs;
  if (dtype == BSA_F32)
    return launch_tra_bwd_f32(static_cast<const float*>(q), static_cast<const float*>(k),
                              static_cast<const float*>(v), static_cast<const float*>(dout), static_cast<float*>(dq),
                              static_cast<float*>(dk), static_cast<float*>(dv), B, H, T, D, beta, p, stream);
  if (flags & BSA_TRA_BWD_DETERMINISTIC)
    return launch_tra_bwd_bf16(q, k, v, dout, dq, dk, dv, B, H, T, D, beta, p, stream);
  // fp32 dq accumulator: a stream-ordered temporary, released on the same stream.
  float* acc = nullptr;
  const size_t bytes = static_cast<size_t>(B) * H * T * D * sizeof(float);
  int dev = 0;
  cudaMemPool_t pool = cudaGetDevice(&dev) == cudaSuccess ? scratch_pool(dev) : nullptr;
  if (pool == nullptr) return BSA_ERR_MEMORY;
  if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&acc), bytes, pool, stream) != cudaSuccess)
    return BSA_ERR_MEMORY;
  const int st = launch_tra_bwd_fused_bf16(q, k, v, dout, dq, dk, dv, B, H, T, D, beta, p, acc, stream);
  if (cudaFreeAsync(acc, stream) != cudaSuccess && st == OK) return BSA_ERR_MEMORY;
  return st;
}

int tra_backward(const void* q, const void* k, const void* v, const void* dout, void* dq, void* dk, void* dv, int B,
                 int H, int T, int D, float beta, float p, int dtype, cudaStream_t stream) {
  return tra_backward_ex(q, k, v, dout, dq, dk, dv, B, H, T, D, beta, p, dtype, 0, stream);
}

// Argument checks of tra_diff_forward and tra_diff_forward_noalloc.
static int check_diff_args(const void* q1, const void* q2, const void* k1, const void* k2, const void* v,
                           const void* out, int B, int H, int T, int D, float beta, float lambda, float p,
                           int dtype) {
  if (q1 == nullptr || q2 == nullptr || k1 == nullptr || k2 == nullptr || v == nullptr || out == nullptr)
    return BSA_ERR_NULLPTR;
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  if (B < 1 || H < 1 || T < 1 || D < 1) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 0x7fffffffLL) return BSA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * T * D >= (1LL << 40)) return BSA_ERR_SHAPE;
  if (!tra_head_dim_supported(D)) return BSA_ERR_UNSUPPORTED;
  if (!isfinite(beta) || !isfinite(p) || !(p > 0.0f) || isnan(lambda)) return BSA_ERR_UNSUPPORTED;
  const void* ptrs[6] = {q1, q2, k1, k2, v, out};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  return BSA_OK;
}

int tra_diff_forward(const void* q1, const void* q2, const void* k1, const void* k2, const void* v, void* out, int B,
                     int H, int T, int D, float beta, float lambda, float p, int normalize, int dtype,
                     cudaStream_t stream) {
  const int chk = check_diff_args(q1, q2, k1, k2, v, out, B, H, T, D, beta, lambda, p, dtype);
  if (chk != BSA_OK) return chk;
  const int dvs = check_device();
  if (dvs != OK) return dvs;
  if (dtype == BSA_F32)  // no scratch: the fp32 kernel folds the normalisation into its scores
    return launch_tra_diff_f32(static_cast<const float*>(q1), static_cast<const float*>(q2),
                               static_cast<const float*>(k1), static_cast<const float*>(k2),
                               static_cast<const float*>(v), static_cast<float*>(out), B, H, T, D, beta, lambda, p,
                               normalize != 0, stream);
  if (!normalize)
    return launch_tra_diff_bf16(q1, q2, k1, k2, v, out, B, H, T, D, beta, lambda, p, nullptr, nullptr, stream);
  // Normalised copies of k1 and k2 (the kernel takes the query rows' factors
  // from its resident Q tiles): a stream-ordered temporary, released on the
  // same stream.
  void* kn = nullptr;
  const size_t bytes = 2 * sizeof(uint16_t) * static_cast<size_t>(B) * H * T * D;
  int dev = 0;
  cudaMemPool_t pool = cudaGetDevice(&dev) == cudaSuccess ? scratch_pool(dev) : nullptr;
  if (pool == nullptr) return BSA_ERR_MEMORY;
  if (cudaMallocFromPoolAsync(&kn, bytes, pool, stream) != cudaSuccess) return BSA_ERR_MEMORY;
  const int st = launch_tra_diff_bf16(q1, q2, k1, k2, v, out, B, H, T, D, beta, lambda, p, nullptr, kn, stream);
  if (cudaFreeAsync(kn, stream) != cudaSuccess && st == OK) return BSA_ERR_MEMORY;
  return st;
}

int tra_diff_backward(const void* q1, const void* q2, const void* k1, const void* k2, const void* v,
                      const void* dout, void* dq1, void* dq2, void* dk1, void* dk2, void* dv, float* dlambda, int B,
                      int H, int T, int D, float beta, float lambda, float p, int normalize, int dtype,
                      cudaStream_t stream) {
  const int chk = check_diff_args(q1, q2, k1, k2, v, dq1, B, H, T, D, beta, lambda, p, dtype);
  if (chk != BSA_OK) return chk;
  const void* more[5] = {dout, dq2, dk1, dk2, dv};
  for (const void* ptr : more) {
    if (ptr == nullptr) return BSA_ERR_NULLPTR;
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  }
  if ((reinterpret_cast<uintptr_t>(dlambda) & 3u) != 0) return BSA_ERR_ALIGN;
  const int dvs = check_device();
  if (dvs != OK) return dvs;
  const bool f32 = dtype == BSA_F32;
  const size_t bytes = tra_diff_bwd_scratch_bytes(B, H, T, D, f32, normalize != 0, dlambda != nullptr);
  void* scratch = nullptr;
  int dev = 0;
  cudaMemPool_t pool = cudaGetDevice(&dev) == cudaSuccess ? scratch_pool(dev) : nullptr;
  if (pool == nullptr) return BSA_ERR_MEMORY;
  if (cudaMallocFromPoolAsync(&scratch, bytes, pool, stream) != cudaSuccess) return BSA_ERR_MEMORY;
  const int st = launch_tra_diff_bwd(q1, q2, k1, k2, v, dout, dq1, dq2, dk1, dk2, dv, dlambda, B, H, T, D, beta,
                                     lambda, p, normalize != 0, f32, scratch, stream);
  if (cudaFreeAsync(scratch, stream) != cudaSuccess && st == OK) return BSA_ERR_MEMORY;
  return st;
}

int tra_diff_forward_noalloc(const void* q1, const void* q2, const void* k1, const void* k2, const void* v,
                             void* out, int B, int H, int T, int D, float beta, float lambda, float p, int normalize,
                             int dtype, cudaStream_t stream) {
  const int chk = check_diff_args(q1, q2, k1, k2, v, out, B, H, T, D, beta, lambda, p, dtype);
  if (chk != BSA_OK) return chk;
  if (dtype == BSA_F32) {  // the fp32 kernel uses no scratch at all
    const int dvs = check_device();
    if (dvs != OK) return dvs;
    return launch_tra_diff_f32(static_cast<const float*>(q1), static_cast<const float*>(q2),
                               static_cast<const float*>(k1), static_cast<const float*>(k2),
                               static_cast<const float*>(v), static_cast<float*>(out), B, H, T, D, beta, lambda, p,
                               normalize != 0, stream);
  }
  if (normalize && !tra_diff_noalloc_fits(B, H, T)) return BSA_ERR_SCRATCH_LIMIT;
  const int dvs = check_device();
  if (dvs != OK) return dvs;
  return launch_tra_diff_noalloc_bf16(q1, q2, k1, k2, v, out, B, H, T, D, beta, lambda, p, normalize != 0, stream);
}

int nsa_select_forward(const void* q, const void* k, const void* v, const int32_t* block_idx, void* out, float* lse,
                       int B, int Hq, int Hkv, int T, int D, int block_size, int S, cudaStream_t stream) {
  const int chk = check_nsa_args(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S);
  if (chk != BSA_OK) return chk;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_nsa_select(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S, stream);
}

size_t nsa_select_fsa_workspace_size(int B, int Hq, int Hkv, int T, int D, int block_size, int S) {
  if (check_nsa_shape(B, Hq, Hkv, T, D, block_size, S) != BSA_OK || !fsa_shape_supported(D, block_size)) return 0;
  // The partial rows are indexed with 32-bit integers inside the kernels.
  if (static_cast<long long>(B) * Hq * T * S >= (1LL << 31)) return 0;
  return nsa_fsa_workspace_bytes(B, Hq, Hkv, T, D, S);
}

int nsa_select_forward_fsa(const void* q, const void* k, const void* v, const int32_t* block_idx, void* out,
                           float* lse, int B, int Hq, int Hkv, int T, int D, int block_size, int S, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  const int chk = check_nsa_args(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S);
  if (chk != BSA_OK) return chk;
  if (!fsa_shape_supported(D, block_size)) return BSA_ERR_UNSUPPORTED;
  if (workspace == nullptr) return BSA_ERR_NULLPTR;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return BSA_ERR_ALIGN;
  const size_t need = nsa_select_fsa_workspace_size(B, Hq, Hkv, T, D, block_size, S);
  if (need == 0) return BSA_ERR_SHAPE;
  if (workspace_bytes < need) return BSA_ERR_SCRATCH_LIMIT;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_nsa_fsa(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, S, workspace, stream);
}

size_t nsa_select_backward_workspace_size(int B, int Hq, int Hkv, int T, int D, int block_size, int S) {
  if (check_nsa_shape(B, Hq, Hkv, T, D, block_size, S) != BSA_OK) return 0;
  // list positions and rows are 32-bit numbers, a query and its slot one of them; (batch, kv head) pairs run along a
  // grid's second axis
  if (static_cast<long long>(B) * Hkv * T * S >= (1LL << 31) || T >= (1 << 26) ||
      static_cast<long long>(B) * Hq * T >= (1LL << 31) ||
      static_cast<long long>(B) * Hkv > 65535)
    return 0;
  return nsa_bwd_workspace_bytes(B, Hq, Hkv, T, D, block_size, S);
}

int nsa_select_backward(const void* q, const void* k, const void* v, const int32_t* block_idx, const void* out,
                        const float* lse, const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv,
                        int T, int D, int block_size, int S, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  if (lse == nullptr || dout == nullptr || dq == nullptr || dk == nullptr || dv == nullptr || workspace == nullptr)
    return BSA_ERR_NULLPTR;
  const int chk = check_nsa_args(q, k, v, block_idx, out, lse, B, Hq, Hkv, T, D, block_size, S);
  if (chk != BSA_OK) return chk;
  if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BSA_ERR_ALIGN;
  const size_t need = nsa_select_backward_workspace_size(B, Hq, Hkv, T, D, block_size, S);
  if (need == 0) return BSA_ERR_SHAPE;
  if (workspace_bytes < need) return BSA_ERR_SCRATCH_LIMIT;
  const int dev = check_device();
  if (dev != OK) return dev;
  return launch_nsa_bwd(q, k, v, block_idx, out, lse, dout, dq, dk, dv, B, Hq, Hkv, T, D, block_size, S, workspace,
                        stream);
}

int nsa_cache_append(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                     float* k_scale, float* v_scale, const int32_t* page_table, const int32_t* cache_lens,
                     const int32_t* new_lens, const float* inv_freq, int B, int Hq, int Hkv, int n, int D,
                     int page_size, int max_pages, int num_pages, int rotary_dim, int interleaved, int dtype,
                     cudaStream_t stream) {
  if (k == nullptr || v == nullptr || k_cache == nullptr || v_cache == nullptr || k_scale == nullptr ||
      v_scale == nullptr || page_table == nullptr || cache_lens == nullptr)
    return BSA_ERR_NULLPTR;
  if ((q == nullptr) != (q_out == nullptr) || (rotary_dim != 0 && inv_freq == nullptr)) return BSA_ERR_NULLPTR;
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  const int sh = check_cache_shape(B, Hq, Hkv, D, page_size, max_pages, num_pages);
  if (sh != BSA_OK) return sh;
  if (n < 1 || static_cast<long long>(B) * Hq * n >= (1LL << 40) / D) return BSA_ERR_SHAPE;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0) return BSA_ERR_UNSUPPORTED;
  const void* ptrs[6] = {k, v, q, q_out, k_cache, v_cache};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  const void* words[6] = {k_scale, v_scale, page_table, cache_lens, new_lens, inv_freq};
  for (const void* ptr : words)
    if (!aligned4(ptr)) return BSA_ERR_ALIGN;
  const int dev = check_device();
  if (dev != OK) return dev;
  return launch_nsa_cache_append(k, v, q, q_out, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, new_lens,
                                 inv_freq, B, Hq, Hkv, n, D, page_size, max_pages, num_pages, rotary_dim,
                                 interleaved != 0, dtype == BSA_F32, stream);
}

size_t nsa_select_decode_workspace_size(int B, int Hq, int Hkv, int D, int page_size, int max_pages, int S) {
  if (S < 0 || S > 32 || check_cache_shape(B, Hq, Hkv, D, page_size, max_pages, 1) != BSA_OK) return 0;
  return nsa_decode_workspace_bytes(D, S);
}

int nsa_select_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, const int32_t* page_table, const int32_t* cache_lens,
                      const int32_t* block_idx, void* out, float* lse, int B, int Hq, int Hkv, int D, int page_size,
                      int max_pages, int num_pages, int S, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || k_scale == nullptr || v_scale == nullptr ||
      page_table == nullptr || cache_lens == nullptr || out == nullptr || workspace == nullptr)
    return BSA_ERR_NULLPTR;
  const int sh = check_cache_shape(B, Hq, Hkv, D, page_size, max_pages, num_pages);
  if (sh != BSA_OK) return sh;
  if (block_idx != nullptr ? (S < 1 || S > 32) : S != 0) return BSA_ERR_SHAPE;
  const void* ptrs[5] = {q, k_cache, v_cache, out, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  const void* words[6] = {k_scale, v_scale, page_table, cache_lens, block_idx, lse};
  for (const void* ptr : words)
    if (!aligned4(ptr)) return BSA_ERR_ALIGN;
  if (workspace_bytes < nsa_select_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S))
    return BSA_ERR_SCRATCH_LIMIT;
  const int dev = check_device();
  if (dev != OK) return dev;
  return launch_nsa_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, cache_lens, block_idx, out, lse, B, Hq,
                           Hkv, D, page_size, max_pages, num_pages, S, workspace, stream);
}

int qk_norm_rope_forward(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                         const void* k_weight, const int32_t* positions, const float* inv_freq,
                         const int64_t* strides, int B, int Hq, int Hkv, int T, int D, int rotary_dim, int interleaved,
                         float rotary_scale, float eps, int dtype, int weight_dtype, cudaStream_t stream) {
  if (q == nullptr || k == nullptr || q_out == nullptr || k_out == nullptr || (rotary_dim != 0 && inv_freq == nullptr))
    return BSA_ERR_NULLPTR;
  int st = check_dtypes(dtype, weight_dtype);
  if (st == BSA_OK) st = check_rope_shape(B, Hq, Hkv, T, D);
  if (st == BSA_OK) st = check_rows(D, rotary_dim, rotary_scale, eps);
  if (st != BSA_OK) return st;
  RopeCall r{};
  const int heads[4] = {Hq, Hkv, Hq, Hkv};
  int64_t to[4][3];
  st = take_strides(strides, 4, heads, T, D, dtype == BSA_F32 ? 4 : 2, to);
  if (st != BSA_OK) return st;
  if (repeats_rows(to[2], B, Hq, T) || repeats_rows(to[3], B, Hkv, T)) return BSA_ERR_SHAPE;
  const void* ptrs[7] = {q, k, q_out, k_out, q_weight, k_weight, inv_freq};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  if (!aligned4(positions)) return BSA_ERR_ALIGN;
  for (int s = 0; s < 2; ++s)
    for (int j = 0; j < 3; ++j) {
      r.x_stride[s][j] = to[s][j];
      r.out_stride[s][j] = to[2 + s][j];
    }
  r.q = q; r.k = k; r.q_out = q_out; r.k_out = k_out;
  r.q_weight = q_weight; r.k_weight = k_weight;
  r.positions = positions; r.inv_freq = inv_freq;
  r.B = B; r.Hq = Hq; r.Hkv = Hkv; r.T = T; r.D = D; r.rotary = rotary_dim;
  r.interleaved = interleaved != 0; r.weight_f32 = weight_dtype == BSA_F32; r.f32 = dtype == BSA_F32;
  r.factor = rotary_scale; r.eps = eps;
  const int dev = check_device();
  return dev != OK ? dev : launch_qk_rope_forward(r, stream);
}

size_t qk_norm_rope_backward_workspace_size(int B, int Hq, int Hkv, int T, int D) {
  if (check_rope_shape(B, Hq, Hkv, T, D) != BSA_OK || check_rows(D, 0, 1.0f, 1.0f) != BSA_OK) return 0;
  return qk_rope_backward_workspace_bytes(B, Hq, Hkv, T, D);
}

int qk_norm_rope_backward(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                          float* dq_weight, float* dk_weight, const void* q_weight, const void* k_weight,
                          const int32_t* positions, const float* inv_freq, const int64_t* strides, int B, int Hq,
                          int Hkv, int T, int D, int rotary_dim, int interleaved, float rotary_scale, float eps,
                          int dtype, int weight_dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (q == nullptr || k == nullptr || dq_out == nullptr || dk_out == nullptr || dq == nullptr || dk == nullptr ||
      workspace == nullptr || (rotary_dim != 0 && inv_freq == nullptr) ||
      (q_weight != nullptr && dq_weight == nullptr) || (k_weight != nullptr && dk_weight == nullptr))
    return BSA_ERR_NULLPTR;
  int st = check_dtypes(dtype, weight_dtype);
  if (st == BSA_OK) st = check_rope_shape(B, Hq, Hkv, T, D);
  if (st == BSA_OK) st = check_rows(D, rotary_dim, rotary_scale, eps);
  if (st != BSA_OK) return st;
  RopeCall r{};
  const int heads[6] = {Hq, Hkv, Hq, Hkv, Hq, Hkv};
  int64_t to[6][3];
  st = take_strides(strides, 6, heads, T, D, dtype == BSA_F32 ? 4 : 2, to);
  if (st != BSA_OK) return st;
  if (repeats_rows(to[4], B, Hq, T) || repeats_rows(to[5], B, Hkv, T)) return BSA_ERR_SHAPE;
  const void* ptrs[9] = {q, k, dq_out, dk_out, dq, dk, q_weight, k_weight, inv_freq};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  if (!aligned4(positions) || !aligned4(dq_weight) || !aligned4(dk_weight) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BSA_ERR_ALIGN;
  const size_t need = qk_norm_rope_backward_workspace_size(B, Hq, Hkv, T, D);
  if (need == 0) return BSA_ERR_SHAPE;
  if (workspace_bytes < need) return BSA_ERR_SCRATCH_LIMIT;
  for (int s = 0; s < 2; ++s)
    for (int j = 0; j < 3; ++j) {
      r.x_stride[s][j] = to[s][j];
      r.dy_stride[s][j] = to[2 + s][j];
      r.out_stride[s][j] = to[4 + s][j];
    }
  r.q = q; r.k = k; r.dq_out = dq_out; r.dk_out = dk_out; r.q_out = dq; r.k_out = dk;
  r.q_weight = q_weight; r.k_weight = k_weight;
  r.dq_weight = q_weight != nullptr ? dq_weight : nullptr;
  r.dk_weight = k_weight != nullptr ? dk_weight : nullptr;
  r.positions = positions; r.inv_freq = inv_freq;
  r.B = B; r.Hq = Hq; r.Hkv = Hkv; r.T = T; r.D = D; r.rotary = rotary_dim;
  r.interleaved = interleaved != 0; r.weight_f32 = weight_dtype == BSA_F32; r.f32 = dtype == BSA_F32;
  r.factor = rotary_scale; r.eps = eps;
  const int dev = check_device();
  return dev != OK ? dev : launch_qk_rope_backward(r, workspace, stream);
}

int nsa_cache4_append(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                      void* k_scale, void* v_scale, const float* k_factor, const float* v_factor,
                      const int32_t* page_table, const int32_t* cache_lens, const int32_t* new_lens,
                      const void* q_weight, const void* k_weight, const float* inv_freq, const int64_t* strides, int B,
                      int Hq, int Hkv, int n, int D, int page_size, int max_pages, int num_pages, int rotary_dim,
                      int interleaved, float rotary_scale, float eps, int dtype, int weight_dtype,
                      cudaStream_t stream) {
  if (k == nullptr || v == nullptr || cache_lens == nullptr || (q == nullptr) != (q_out == nullptr) ||
      (rotary_dim != 0 && inv_freq == nullptr))
    return BSA_ERR_NULLPTR;
  Append4Call r{};
  r.cache = cache4_of(k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, B, Hkv, D, page_size,
                      max_pages, num_pages);
  int st = check_dtypes(dtype, weight_dtype);
  if (st == BSA_OK) st = check_cache4(r.cache, Hq);
  if (st != BSA_OK) return st;
  if (n < 1 || n > (1 << 30) || static_cast<long long>(B) * n > 0x7fffffffLL ||
      static_cast<long long>(B) * Hq * n >= (1LL << 40) / D)
    return BSA_ERR_SHAPE;
  st = check_rows(D, rotary_dim, rotary_scale, eps);
  if (st != BSA_OK) return st;
  const int heads[3] = {Hkv, Hkv, Hq};
  int64_t to[3][3];
  st = take_strides(strides, q != nullptr ? 3 : 2, heads, n, D, dtype == BSA_F32 ? 4 : 2, to);
  if (st != BSA_OK) return st;
  const void* ptrs[7] = {k, v, q, q_out, q_weight, k_weight, inv_freq};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  if (!aligned4(cache_lens) || !aligned4(new_lens)) return BSA_ERR_ALIGN;
  for (int j = 0; j < 3; ++j) {
    r.stride[1][j] = to[0][j];
    r.stride[2][j] = to[1][j];
    r.stride[0][j] = q != nullptr ? to[2][j] : 0;
  }
  r.k = k; r.v = v; r.q = q; r.q_out = q_out;
  r.q_weight = q_weight; r.k_weight = k_weight;
  r.lens = cache_lens; r.new_lens = new_lens; r.inv_freq = inv_freq;
  r.Hq = Hq; r.n = n; r.rotary = rotary_dim;
  r.interleaved = interleaved != 0; r.weight_f32 = weight_dtype == BSA_F32; r.f32 = dtype == BSA_F32;
  r.factor = rotary_scale; r.eps = eps;
  const int dev = check_device();
  return dev != OK ? dev : launch_nsa_cache4_append(r, stream);
}

int nsa_cache4_read(const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                    const float* k_factor, const float* v_factor, const int32_t* page_table, const int32_t* starts,
                    const int32_t* cache_lens, void* k_out, void* v_out, int B, int Hkv, int n, int D, int page_size,
                    int max_pages, int num_pages, int dtype, cudaStream_t stream) {
  if (cache_lens == nullptr || k_out == nullptr || v_out == nullptr) return BSA_ERR_NULLPTR;
  if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_DTYPE;
  const Cache4 c = cache4_of(k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, B, Hkv, D, page_size,
                             max_pages, num_pages);
  const int st = check_cache4(c, Hkv);
  if (st != BSA_OK) return st;
  if (n < 1 || n > (1 << 30) || static_cast<long long>(B) * Hkv * n >= (1LL << 40) / D) return BSA_ERR_SHAPE;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(starts) || !aligned4(cache_lens)) return BSA_ERR_ALIGN;
  const int dev = check_device();
  return dev != OK ? dev : launch_nsa_cache4_read(c, starts, cache_lens, k_out, v_out, n, dtype == BSA_F32, stream);
}

size_t nsa_cache4_decode_workspace_size(int B, int Hq, int Hkv, int D, int page_size, int max_pages, int S) {
  if (S < 0 || S > 32 || check_cache_shape(B, Hq, Hkv, D, page_size, max_pages, 1) != BSA_OK) return 0;
  return nsa_decode4_workspace_bytes(D, S);
}

int nsa_cache4_decode(const void* q, const void* k_cache, const void* v_cache, const void* k_scale,
                      const void* v_scale, const float* k_factor, const float* v_factor, const int32_t* page_table,
                      const int32_t* cache_lens, const int32_t* block_idx, void* out, float* lse, int B, int Hq,
                      int Hkv, int D, int page_size, int max_pages, int num_pages, int S, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  if (q == nullptr || cache_lens == nullptr || out == nullptr || (workspace == nullptr && block_idx == nullptr))
    return BSA_ERR_NULLPTR;
  const Cache4 c = cache4_of(k_cache, v_cache, k_scale, v_scale, k_factor, v_factor, page_table, B, Hkv, D, page_size,
                             max_pages, num_pages);
  const int st = check_cache4(c, Hq);
  if (st != BSA_OK) return st;
  if (block_idx != nullptr ? (S < 1 || S > 32) : S != 0) return BSA_ERR_SHAPE;
  const void* ptrs[3] = {q, out, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return BSA_ERR_ALIGN;
  if (!aligned4(cache_lens) || !aligned4(block_idx) || !aligned4(lse)) return BSA_ERR_ALIGN;
  if (workspace != nullptr && workspace_bytes < nsa_cache4_decode_workspace_size(B, Hq, Hkv, D, page_size, max_pages, S))
    return BSA_ERR_SCRATCH_LIMIT;
  const int dev = check_device();
  return dev != OK ? dev : launch_nsa_decode4(c, q, cache_lens, block_idx, out, lse, Hq, S, workspace, stream);
}

const char* bsa_status_string(int status) {
  switch (status) {
    case BSA_OK: return "success";
    case BSA_ERR_NULLPTR: return "a required pointer is NULL";
    case BSA_ERR_SHAPE: return "a size is out of range or inconsistent";
    case BSA_ERR_DTYPE: return "dtype is not a bsa_dtype value";
    case BSA_ERR_UNSUPPORTED: return "unsupported head dim, block size, group size or parameter value";
    case BSA_ERR_LAUNCH: return "CUDA kernel launch failed";
    case BSA_ERR_DEVICE: return "no usable sm_103 device or CUDA driver entry point";
    case BSA_ERR_ALIGN: return "a tensor pointer is not suitably aligned";
    case BSA_ERR_MEMORY: return "scratch memory could not be allocated or released";
    case BSA_ERR_SCRATCH_LIMIT:
      return "the problem needs more scratch than the fixed buffer or the caller's workspace holds";
    default: return "unknown bsa_status";
  }
}

int bsa_version(void) { return 100; }

int bsa_selftest_wait_timeout(long long limit_cycles, int* result, cudaStream_t stream) {
  if (result == nullptr) return BSA_ERR_NULLPTR;
  if (limit_cycles < 1 || limit_cycles > 100000000LL) return BSA_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(result) & 3u) != 0) return BSA_ERR_ALIGN;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_selftest_wait_timeout(limit_cycles, result, stream);
}

int bsa_selftest_log2(const float* x, float* y_fma, float* y_ref, int n, cudaStream_t stream) {
  if (x == nullptr || y_fma == nullptr || y_ref == nullptr) return BSA_ERR_NULLPTR;
  if (n < 1) return BSA_ERR_SHAPE;
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y_fma) |
                         reinterpret_cast<uintptr_t>(y_ref)) & 3u;
  if (mis != 0) return BSA_ERR_ALIGN;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_selftest_log2(x, y_fma, y_ref, n, stream);
}

int bsa_selftest_exp2(const float* y, float* w_fma, float* w_ref, int n, cudaStream_t stream) {
  if (y == nullptr || w_fma == nullptr || w_ref == nullptr) return BSA_ERR_NULLPTR;
  if (n < 1) return BSA_ERR_SHAPE;
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(w_fma) |
                         reinterpret_cast<uintptr_t>(w_ref)) & 3u;
  if (mis != 0) return BSA_ERR_ALIGN;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_selftest_exp2(y, w_fma, w_ref, n, stream);
}

int bsa_read_probe(const void* buf, size_t bytes, int reps, unsigned int* sink, cudaStream_t stream) {
  if (buf == nullptr || sink == nullptr) return BSA_ERR_NULLPTR;
  if (bytes < 16 || bytes % 16 != 0 || bytes > (1ull << 40) || reps < 1 || reps > 100000) return BSA_ERR_SHAPE;
  if (!aligned16(buf) || (reinterpret_cast<uintptr_t>(sink) & 3u) != 0) return BSA_ERR_ALIGN;
  const int dv = check_device();
  if (dv != OK) return dv;
  return launch_read_probe(buf, static_cast<long long>(bytes), reps, sink, stream);
}

int bsa_device_error(void) {
  const unsigned codes[11] = {tra_bf16_device_error(), tra_f32_device_error(), nsa_device_error(),
                              tra_bwd_device_error(), tra_diff_device_error(), nsa_fsa_device_error(),
                              nsa_bwd_device_error(), nsa_bwd_tc_device_error(), nsa_decode_device_error(),
                              nsa_decode4_device_error(), selftest_device_error()};
  unsigned worst = 0;
  for (unsigned c : codes) {
    if (c == 0xffffffffu) return -1;
    if (c > worst) worst = c;
  }
  return static_cast<int>(worst);
}

}  // extern "C"
