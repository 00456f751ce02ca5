// The cache write of any number of tokens by slot (sm_103a): k / v rows copied
// into the pages their slots name, or quantised to e4m3 under the pages' scales.
//
// Bound: HBM, every row read and written once. One thread moves 16 bf16 values
// (two 16-byte loads; two 16-byte stores, or one of e4m3 codes).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_decode.h"
#include "pd_common.cuh"
#include "pd_variants.h"

namespace pd {
namespace {

struct WriteParams {
  const uint16_t* in[2];  // k, v (null: K = V)
  int64_t stride[2];      // elements between tokens
  uint8_t* pool[2];
  const float* scale[2];  // FP8
  const int32_t* slot_map;
  uint32_t* flags;
  int num_tokens, heads, dim, page_size;
  long long num_slots;
};

constexpr int kWriteThreads = 256;

// Two fp32 quotients -> two e4m3 codes (low byte the first), to nearest even, clamped to +-448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool FP8>
__global__ void __launch_bounds__(kWriteThreads) write_slots_kernel(const WriteParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int which = blockIdx.y;
  const int per_row = p.dim / 16, per_token = p.heads * per_row;
  const long long n = (long long)p.num_tokens * per_token;
  for (long long e = blockIdx.x * (long long)kWriteThreads + threadIdx.x; e < n;
       e += (long long)gridDim.x * kWriteThreads) {
    const int t = (int)(e / per_token), c = (int)(e % per_token);
    const int h = c / per_row, d = (c % per_row) * 16;
    const int slot = p.slot_map[t];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1 && c == 0) atomicOr(p.flags, kErrBadPage);
      continue;
    }
    const int page = slot / p.page_size, off = slot - page * p.page_size;
    const uint4* src = reinterpret_cast<const uint4*>(p.in[which] + t * p.stride[which] + h * p.dim + d);
    const uint4 a = src[0], b = src[1];
    const size_t at = (((size_t)page * p.heads + h) * p.page_size + off) * p.dim + d;
    if constexpr (FP8) {
      const float s = p.scale[which][(size_t)page * p.heads + h];
      float x[8], y[8];
      unpack_bf16x8(a, x);
      unpack_bf16x8(b, y);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = e4m3x2(__fdiv_rn(x[4 * i], s), __fdiv_rn(x[4 * i + 1], s)) |
               e4m3x2(__fdiv_rn(x[4 * i + 2], s), __fdiv_rn(x[4 * i + 3], s)) << 16;
        w[2 + i] = e4m3x2(__fdiv_rn(y[4 * i], s), __fdiv_rn(y[4 * i + 1], s)) |
                   e4m3x2(__fdiv_rn(y[4 * i + 2], s), __fdiv_rn(y[4 * i + 3], s)) << 16;
      }
      *reinterpret_cast<uint4*>(p.pool[which] + at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(p.pool[which] + at * 2);
      dst[0] = a;
      dst[1] = b;
    }
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

pd_status write_slots(const pd_layer_desc* layer, bool fp8, int32_t num_tokens, const void* k_in, const void* v_in,
                      int64_t k_stride, int64_t v_stride, const int32_t* slot_map, void* k_pool, void* v_pool,
                      const float* k_scale, const float* v_scale, uint32_t* device_flags, void* stream) {
  if (!layer || num_tokens < 0) return PD_ERR_INVALID_ARG;
  const pd_layer_desc& ly = *layer;
  if (ly.num_kv_heads <= 0 || ly.page_size <= 0 || ly.num_pages <= 0) return PD_ERR_INVALID_ARG;
  if (ly.kv_shared != 0 && ly.kv_shared != 1) return PD_ERR_INVALID_ARG;
  if (ly.kv_dtype != (fp8 ? PD_KV_FP8_E4M3 : PD_KV_BF16)) return PD_ERR_INVALID_ARG;
  if (ly.head_dim != 128 && ly.head_dim != 256 && ly.head_dim != 512) return PD_ERR_UNSUPPORTED;
  const long long slots = (long long)ly.num_pages * ly.page_size;
  if (slots > 0x7fffffffLL || ly.num_kv_heads > (1 << 20)) return PD_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PD_OK;
  const bool kvs = ly.kv_shared != 0;
  const int64_t row = (int64_t)ly.num_kv_heads * ly.head_dim;
  if (!k_in || !slot_map || !k_pool || !device_flags || !aligned(k_in, 16) || !aligned(k_pool, 16) ||
      !aligned(slot_map, 4) || !aligned(device_flags, 4) || k_stride < row || k_stride % 8 != 0 ||
      k_stride > (INT64_MAX >> 33))
    return PD_ERR_INVALID_ARG;
  if (!kvs && (!v_in || !v_pool || v_pool == k_pool || !aligned(v_in, 16) || !aligned(v_pool, 16) ||
               v_stride < row || v_stride % 8 != 0 || v_stride > (INT64_MAX >> 33)))
    return PD_ERR_INVALID_ARG;
  if (kvs && v_pool && v_pool != k_pool) return PD_ERR_INVALID_ARG;
  if (fp8) {
    if (!k_scale || !aligned(k_scale, 4)) return PD_ERR_INVALID_ARG;
    if (!kvs && (!v_scale || !aligned(v_scale, 4))) return PD_ERR_INVALID_ARG;
    if (kvs && v_scale && v_scale != k_scale) return PD_ERR_INVALID_ARG;
  }
  WriteParams p = {};
  p.in[0] = static_cast<const uint16_t*>(k_in);
  p.in[1] = static_cast<const uint16_t*>(v_in);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.pool[0] = static_cast<uint8_t*>(k_pool);
  p.pool[1] = static_cast<uint8_t*>(v_pool);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.slot_map = slot_map;
  p.flags = device_flags;
  p.num_tokens = num_tokens;
  p.heads = ly.num_kv_heads;
  p.dim = ly.head_dim;
  p.page_size = ly.page_size;
  p.num_slots = slots;
  const long long n = (long long)num_tokens * (row / 16);
  const long long want = (n + kWriteThreads - 1) / kWriteThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < (1 << 20) ? want : (1 << 20)), kvs ? 1 : 2);
  cfg.blockDim = dim3(kWriteThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = fp8 ? cudaLaunchKernelEx(&cfg, write_slots_kernel<true>, p)
                            : cudaLaunchKernelEx(&cfg, write_slots_kernel<false>, p);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace
}  // namespace pd

extern "C" {

pd_status paged_decode_write_slots(const pd_layer_desc* layer, int32_t num_tokens, const void* k_in,
                                   const void* v_in, int64_t k_stride, int64_t v_stride, const int32_t* slot_map,
                                   void* k_pool, void* v_pool, uint32_t* device_flags, void* stream) {
  return pd::write_slots(layer, false, num_tokens, k_in, v_in, k_stride, v_stride, slot_map, k_pool, v_pool, nullptr,
                         nullptr, device_flags, stream);
}

pd_status paged_decode_write_slots_fp8(const pd_layer_desc* layer, int32_t num_tokens, const void* k_in,
                                       const void* v_in, int64_t k_stride, int64_t v_stride,
                                       const int32_t* slot_map, void* k_pool, void* v_pool, const float* k_scale,
                                       const float* v_scale, uint32_t* device_flags, void* stream) {
  return pd::write_slots(layer, true, num_tokens, k_in, v_in, k_stride, v_stride, slot_map, k_pool, v_pool, k_scale,
                         v_scale, device_flags, stream);
}

}  // extern "C"
