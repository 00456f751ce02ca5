// The cache write of any number of tokens by slot (sm_103a): k / v rows copied
// into the pages their slots name, or quantised to e4m3 under the pages' scales.
//
// Bound: HBM, every row read and written once. A CTA takes a run of tokens of K
// or of V: their rows' places in the pool are worked out once per token, then
// every thread moves the same 16 bf16 (8 for a bf16 cache) of each token, 128
// bytes of loads in flight.
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
  int num_tokens, heads, dim, page_size, run;
  long long num_slots;
};

constexpr int kWriteThreads = 256;
constexpr int kMaxRun = 16;  // tokens of a CTA

// Two fp32 quotients -> two e4m3 codes (low byte the first), to nearest even, clamped to +-448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// x / s rounded to nearest, for s with its correctly rounded reciprocal r, all
// normal and far from the ends of the range (e4m3x16 sees to that): the quotient
// q = x r corrected by its exact remainder, q + (x - q s) r, is the correctly rounded one (P. W.
// Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, IBM J. Res. Dev. 34, 1990). Three operations, for two elements at
// once; with the general division 74 million elements took 70 us, one element
// at a time 41.2 (38.4 now). It is the negated quotient that is computed, x (-r)
// and so on: where x is a zero the remainder is +0, and added to a quotient of -0
// it would lose its sign; added to the negated one it loses none.
struct Scale2 {
  uint64_t minus_r, s;  // the same in both halves
};
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ Scale2 scale2(float s) {
  const float r = __frcp_rn(s);
  return {f32x2(-r, -r), f32x2(s, s)};
}

// Two bf16 -> their negated quotients' codes.
__device__ __forceinline__ uint32_t minus_e4m3x2(uint32_t w, const Scale2& k) {
  const uint64_t x = f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  uint64_t q, e;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(k.minus_r));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q), "l"(k.s), "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(e), "l"(k.minus_r), "l"(q));
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(q));
  return e4m3x2(lo, hi);
}

__device__ __forceinline__ uint32_t e4m3x4(uint32_t a, uint32_t b, const Scale2& k) {
  return (minus_e4m3x2(a, k) | minus_e4m3x2(b, k) << 16) ^ 0x80808080u;
}

// Any scale and any values: the division itself.
__device__ __noinline__ uint32_t e4m3x4_any(uint32_t a, uint32_t b, float s) {
  return e4m3x2(__fdiv_rn(__uint_as_float(a << 16), s), __fdiv_rn(__uint_as_float(a & 0xffff0000u), s)) |
         e4m3x2(__fdiv_rn(__uint_as_float(b << 16), s), __fdiv_rn(__uint_as_float(b & 0xffff0000u), s)) << 16;
}

// The larger magnitudes of two pairs of bf16, as integers (their order is the magnitudes', infinity and NaN last).
__device__ __forceinline__ uint32_t larger2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

__device__ __forceinline__ uint4 e4m3x16(const uint4& a, const uint4& b, float s) {
  // scales from 2^-60 to 2^60 keep every quotient that matters (2^-11 to 2^9) and its
  // remainder normal, and a smaller quotient rounds to zero; values below 2^67
  // (bf16 0x6100) keep the others below 2^127, which saturate. (A quotient past
  // the fp32 range would have an infinite remainder and end as NaN.) Negative
  // scales, under which zeros would lose their sign, take the division too.
  const uint32_t m = larger2(larger2(larger2(larger2(a.x & 0x7fff7fffu, a.y), larger2(a.z & 0x7fff7fffu, a.w)), b.x),
                             larger2(larger2(b.y & 0x7fff7fffu, b.z), b.w));
  const bool odd = !(s > 0x1p-60f && s < 0x1p60f) || (m & 0xffffu) >= 0x6100u || m >= 0x61000000u;
  if (odd)
    return make_uint4(e4m3x4_any(a.x, a.y, s), e4m3x4_any(a.z, a.w, s), e4m3x4_any(b.x, b.y, s),
                      e4m3x4_any(b.z, b.w, s));
  const Scale2 k = scale2(s);
  return make_uint4(e4m3x4(a.x, a.y, k), e4m3x4(a.z, a.w, k), e4m3x4(b.x, b.y, k), e4m3x4(b.z, b.w, k));
}

// Rows are read once: keep them out of L1.
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <bool FP8>
__global__ void __launch_bounds__(kWriteThreads) write_slots_kernel(const __grid_constant__ WriteParams p) {
  __shared__ long long place[kMaxRun];  // first element of the token's first head in the pool, -1: not written
  __shared__ int page_of[kMaxRun];
  constexpr int ELEMS = FP8 ? 16 : 8;  // of a thread and token
  constexpr int kAhead = FP8 ? 4 : 8;  // tokens a thread has in flight: 128 bytes of loads
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const bool v = blockIdx.y != 0;
  const int first = blockIdx.x * p.run, run = min(p.run, p.num_tokens - first);
  if (tid < run) {
    const int slot = __ldg(p.slot_map + first + tid);
    place[tid] = -1;
    if (slot >= 0 && slot < p.num_slots) {
      const int page = slot / p.page_size;
      page_of[tid] = page;
      place[tid] = ((long long)page * p.heads * p.page_size + (slot - page * p.page_size)) * p.dim;
    } else if (slot != -1) {
      atomicOr(p.flags, kErrBadPage);
    }
  }
  __syncthreads();
  const uint16_t* in = v ? p.in[1] : p.in[0];
  const int64_t stride = v ? p.stride[1] : p.stride[0];
  uint8_t* pool = v ? p.pool[1] : p.pool[0];
  const float* scale = v ? p.scale[1] : p.scale[0];
  // `lanes` threads share a token; narrow rows leave a CTA room for several at a time
  const int per_row = p.dim / ELEMS, per_token = p.heads * per_row;
  const int lanes = min(per_token, kWriteThreads), together = kWriteThreads / lanes;
  const int sub = tid / lanes;
  if (sub >= together) return;
  for (int c = tid - sub * lanes; c < per_token; c += lanes) {
    const int h = c / per_row;
    const uint16_t* src = in + (int64_t)first * stride + c * ELEMS;
    const long long to = (long long)h * (p.page_size - 1) * p.dim + (long long)c * ELEMS;  // h P d + (c mod row) ELEMS
    for (int t0 = sub; t0 < run; t0 += together * kAhead) {
      uint4 a[kAhead], b[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int t = t0 + k * together;
        if (t < run && place[t] >= 0) {
          a[k] = load_once(src + t * stride);
          if constexpr (FP8) b[k] = load_once(src + t * stride + 8);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int t = t0 + k * together;
        if (t >= run || place[t] < 0) continue;
        const long long at = place[t] + to;
        if constexpr (FP8) {
          const float s = __ldg(scale + (size_t)page_of[t] * p.heads + h);
          *reinterpret_cast<uint4*>(pool + at) = e4m3x16(a[k], b[k], s);
        } else {
          *reinterpret_cast<uint4*>(pool + at * 2) = a[k];
        }
      }
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
  // runs of up to 16 tokens, shorter while that leaves SMs without a CTA (a
  // decode step's 64 tokens: a CTA each)
  p.run = kMaxRun;
  while (p.run > 1 && (long long)num_tokens < 304ll * p.run) p.run /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((num_tokens + p.run - 1) / p.run), kvs ? 1 : 2);
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

pd_status paged_decode_write_slots_args(const pd_write_slots_args* a) {
  if (!a) return PD_ERR_INVALID_ARG;
  return pd::write_slots(a->layer, a->fp8 != 0, a->num_tokens, a->k_in, a->v_in, a->k_stride, a->v_stride, a->slot_map,
                         a->k_pool, a->v_pool, a->fp8 ? a->k_scale : nullptr, a->fp8 ? a->v_scale : nullptr,
                         a->device_flags, a->stream);
}

}  // extern "C"
