// Rows of a paged cache by slot (sm_103a): the write of new rows into a 4-bit
// cache, quantised on the way, and the read-back of cached rows as bf16 from a
// 4-bit, an e4m3 or a bf16 cache.
//
// Bound: HBM, every row read and written once. A CTA takes a run of tokens of
// K or of V: their rows' places in the pool are worked out once per token, then
// every thread takes the same 16 elements of each token, so that a warp's loads
// or stores of bf16 rows are 1024 contiguous bytes; several tokens are in flight
// a thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fp4.h"
#include "paged_decode.h"
#include "pd_common.cuh"
#include "pd_variants.h"

namespace pd {
namespace {

struct RowsParams {
  uint16_t* rows[2];        // k, v rows (null: K = V)
  int64_t stride[2];        // elements between tokens
  uint8_t* pool[2];
  void* scale[2];           // 4 bits: e4m3 of every 16 elements; e4m3: fp32 [num_pages, Hkv]
  float up[2];              // 4 bits: 2^exp (read), 2^-exp (write)
  const int32_t* slot_map;
  uint32_t* flags;
  int num_tokens, heads, dim, page_size, run;
  long long num_slots;
};

constexpr int kRowsThreads = 256;
constexpr int kRowsMaxRun = 16;  // tokens of a CTA

// A CTA's tokens: first element of each token's first head in the pool (-1: skipped) and its page.
struct Places {
  long long at[kRowsMaxRun];
  int page[kRowsMaxRun];
};

__device__ __forceinline__ void find_places(const RowsParams& p, Places& s, int first, int run) {
  const int tid = threadIdx.x;
  if (tid < run) {
    const int slot = __ldg(p.slot_map + first + tid);
    s.at[tid] = -1;
    if (slot >= 0 && slot < p.num_slots) {
      const int page = slot / p.page_size;
      s.page[tid] = page;
      s.at[tid] = ((long long)page * p.heads * p.page_size + (slot - page * p.page_size)) * p.dim;
    } else if (slot != -1) {
      atomicOr(p.flags, kErrBadPage);
    }
  }
  __syncthreads();
}

// Rows pass through once: keep them out of L1.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t larger2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

// A block of 16 bf16: 32 bytes of one lane.
struct Block {
  uint32_t w[8];
};
template <bool WIDE>
__device__ __forceinline__ Block load_block(const void* p) {
  Block b;
  if constexpr (WIDE) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(b.w[0]), "=r"(b.w[1]), "=r"(b.w[2]), "=r"(b.w[3]), "=r"(b.w[4]), "=r"(b.w[5]), "=r"(b.w[6]),
                   "=r"(b.w[7])
                 : "l"(p));
  } else {
    const uint4 x = load_once(p), y = load_once(static_cast<const uint8_t*>(p) + 16);
    b.w[0] = x.x, b.w[1] = x.y, b.w[2] = x.z, b.w[3] = x.w;
    b.w[4] = y.x, b.w[5] = y.y, b.w[6] = y.z, b.w[7] = y.w;
  }
  return b;
}

// Its codes, and its scale.
// The quotients have to be right to the last bit only where a value is halfway
// between two codes (a bf16 is 8 bits and a scale 4 wide: any other quotient is
// 2^-9 away from there). x (1 / s) with the reciprocal rounded misses that for
// scales of significand 15/8, so the reciprocal is taken in two parts; over all
// e4m3 scales and all bf16 up to 7 scales the codes are those of the exact quotients.
__device__ __forceinline__ uint2 quantise16(Block v, float down, uint8_t& scale) {
  uint32_t m = 0;  // (as whole numbers: NaN is the largest)
#pragma unroll
  for (int i = 0; i < 8; ++i) m = larger2(m, v.w[i]);
  m = max(m << 16, m & 0xffff0000u);
  const float want = __uint_as_float(m) * ((1.f / 6.f) * down);
  uint16_t s8;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(want));
  scale = (uint8_t)s8;
  uint32_t s16;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"(s8));
  const float s = __half2float(__ushort_as_half((unsigned short)(s16 & 0xffffu)));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = __uint_as_float(__float_as_uint(r) - 16u);  // below 1 / s by some last bits, so that
  const float rest = fmaf(-r, s, 1.f) * r;        // rest > 0 and a zero keeps its sign
  uint64_t r_hi = f32x2(r * down, r * down), r_lo = f32x2(rest * down, rest * down);
  if (__builtin_expect(want > 448.f, 0)) {
    // a clamped scale: quotients may pass the range of fp32, and all past 6 give the largest code
    const float top = 8.f * 448.f / down;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fminf(fmaxf(__uint_as_float(v.w[i] << 16), -top), top);
      const float b = fminf(fmaxf(__uint_as_float(v.w[i] & 0xffff0000u), -top), top);
      v.w[i] = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);  // (cut to a bf16: still above 6)
    }
  }
  if (scale == 0 || scale == 0x7f) r_hi = r_lo = 0;  // zeros, or NaN whatever the codes
  uint32_t codes[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v.w[h * 4 + i];
      uint64_t x = f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), t;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(x), "l"(r_lo));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(x), "l"(r_hi));
      asm("mov.b64 {%0, %1}, %2;" : "=f"(y[2 * i]), "=f"(y[2 * i + 1]) : "l"(t));
    }
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(codes[h])
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  }
  const bool none = scale == 0 || scale == 0x7f;
  return make_uint2(none ? 0u : codes[0], none ? 0u : codes[1]);
}

// WIDE: rows that begin on 32 bytes, a load a block. (16384 tokens of 4 x 512, K
// and V: 30 us, floor 25, waiting for its loads with issue slots at 62%; with their
// read-back 60 us, where 8 elements a lane, two lanes finding the scale that one
// does here, took 74 by their 142 instructions for 8 elements.)
template <bool WIDE>
__global__ void __launch_bounds__(kRowsThreads) write_fp4_kernel(const __grid_constant__ RowsParams p) {
  __shared__ Places places;
  constexpr int kAhead = 4;  // tokens a thread has in flight: 128 bytes of loads
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, v = blockIdx.y;
  const int first = blockIdx.x * p.run, run = min(p.run, p.num_tokens - first);
  find_places(p, places, first, run);
  const uint16_t* in = v ? p.rows[1] : p.rows[0];
  const int64_t stride = v ? p.stride[1] : p.stride[0];
  uint8_t* pool = v ? p.pool[1] : p.pool[0];
  uint8_t* scale = static_cast<uint8_t*>(v ? p.scale[1] : p.scale[0]);
  const float down = v ? p.up[1] : p.up[0];
  const int per_row = p.dim / kFp4Block, per_token = p.heads * per_row;
  const int lanes = min(per_token, kRowsThreads), together = kRowsThreads / lanes;
  const int sub = tid / lanes;
  if (sub >= together) return;
  for (int c = tid - sub * lanes; c < per_token; c += lanes) {
    const int h = c / per_row;
    const uint16_t* src = in + (int64_t)first * stride + c * kFp4Block;
    const long long to = (long long)h * (p.page_size - 1) * per_row + c;  // blocks: h P + (c mod row)
    for (int t0 = sub; t0 < run; t0 += together * kAhead) {
      Block a[kAhead];
      long long at[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int t = t0 + k * together;
        at[k] = t < run ? places.at[t] : -1;
        if (at[k] >= 0) a[k] = load_block<WIDE>(src + t * stride);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (at[k] < 0) continue;
        const long long block = at[k] / kFp4Block + to;
        uint8_t s;
        const uint2 codes = quantise16(a[k], down, s);
        reinterpret_cast<uint2*>(pool)[block] = codes;
        scale[block] = s;
      }
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Eight elements of a row of each type, as bf16.
__device__ __forceinline__ void from_fp4(uint32_t w, float s, uint32_t (&r)[4]) {
  uint32_t o[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
    r[i] = pack2(f.x * s, f.y * s);  // 2 and 4 significant bits: exact
  }
}

__device__ __forceinline__ void from_fp8(uint2 w, float s, uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)((i & 2 ? w.y : w.x) >> (16 * (i & 1)))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    r[i] = pack2(f.x * s, f.y * s);
  }
}

// KV: PD_KV_BF16, PD_KV_FP8_E4M3 or PD_KV_FP4_E2M1. A lane takes 16 elements. WIDE:
// outputs that begin on 32 bytes, one store for them. (30000 tokens of 4 x 512, K and
// V, from 4 bits: 49.1 us; with 8 elements a lane 54.6.)
template <int KV, bool WIDE>
__global__ void __launch_bounds__(kRowsThreads) read_slots_kernel(const __grid_constant__ RowsParams p) {
  __shared__ Places places;
  constexpr int kAhead = KV == PD_KV_BF16 ? 4 : 8, kRaw = KV == PD_KV_BF16 ? 8 : KV == PD_KV_FP8_E4M3 ? 4 : 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, v = blockIdx.y;
  const int first = blockIdx.x * p.run, run = min(p.run, p.num_tokens - first);
  find_places(p, places, first, run);
  uint16_t* out = v ? p.rows[1] : p.rows[0];
  const int64_t stride = v ? p.stride[1] : p.stride[0];
  const uint8_t* pool = v ? p.pool[1] : p.pool[0];
  const void* scale = v ? p.scale[1] : p.scale[0];
  const float up = v ? p.up[1] : p.up[0];
  const int per_row = p.dim / 16, per_token = p.heads * per_row;
  const int lanes = min(per_token, kRowsThreads), together = kRowsThreads / lanes;
  const int sub = tid / lanes;
  if (sub >= together) return;
  for (int c = tid - sub * lanes; c < per_token; c += lanes) {
    const int h = c / per_row;
    uint16_t* dst = out + (int64_t)first * stride + c * 16;
    const long long to = (long long)h * (p.page_size - 1) * per_row + c;  // 16s: h P + (c mod row)
    for (int t0 = sub; t0 < run; t0 += together * kAhead) {
      uint32_t a[kAhead][kRaw];
      float s[kAhead];
      bool here[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int t = t0 + k * together;
        here[k] = t < run && places.at[t] >= 0;
        if (!here[k]) continue;
        const long long block = places.at[t] / 16 + to;
        if constexpr (KV == PD_KV_BF16) {
          const uint4 x = load_once(pool + block * 32), y = load_once(pool + block * 32 + 16);
          a[k][0] = x.x, a[k][1] = x.y, a[k][2] = x.z, a[k][3] = x.w;
          a[k][4] = y.x, a[k][5] = y.y, a[k][6] = y.z, a[k][7] = y.w;
        } else if constexpr (KV == PD_KV_FP8_E4M3) {
          const uint4 x = load_once(pool + block * 16);
          a[k][0] = x.x, a[k][1] = x.y, a[k][2] = x.z, a[k][3] = x.w;
          s[k] = __ldg(static_cast<const float*>(scale) + (size_t)places.page[t] * p.heads + h);
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(pool) + block);
          a[k][0] = x.x, a[k][1] = x.y;
          uint32_t s16;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"((uint16_t)__ldg(static_cast<const uint8_t*>(scale) + block)));
          s[k] = __half2float(__ushort_as_half((unsigned short)(s16 & 0xffffu))) * up;
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!here[k]) continue;
        uint32_t o[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (KV == PD_KV_BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = a[k][i * 4 + j];
          } else if constexpr (KV == PD_KV_FP8_E4M3) {
            from_fp8(make_uint2(a[k][i * 2], a[k][i * 2 + 1]), s[k], o[i]);
          } else {
            from_fp4(a[k][i], s[k], o[i]);
          }
        }
        uint16_t* at = dst + (t0 + k * together) * stride;
        if constexpr (WIDE) {
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(o[0][0]), "r"(o[0][1]),
                       "r"(o[0][2]), "r"(o[0][3]), "r"(o[1][0]), "r"(o[1][1]), "r"(o[1][2]), "r"(o[1][3])
                       : "memory");
        } else {
          reinterpret_cast<uint4*>(at)[0] = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
          reinterpret_cast<uint4*>(at)[1] = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
        }
      }
    }
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks and parameters that the write and the reads share.
pd_status rows_params(const pd_layer_desc* layer, int kv_dtype, int32_t num_tokens, const void* k_rows,
                      const void* v_rows, int64_t k_stride, int64_t v_stride, const int32_t* slot_map,
                      const void* k_pool, const void* v_pool, const void* k_scale, const void* v_scale, int32_t k_exp,
                      int32_t v_exp, uint32_t* device_flags, bool write, RowsParams* out) {
  if (!layer || num_tokens < 0) return PD_ERR_INVALID_ARG;
  const pd_layer_desc& ly = *layer;
  if (ly.num_kv_heads <= 0 || ly.page_size <= 0 || ly.num_pages <= 0) return PD_ERR_INVALID_ARG;
  if (ly.kv_shared != 0 && ly.kv_shared != 1) return PD_ERR_INVALID_ARG;
  if (ly.kv_dtype != kv_dtype) return PD_ERR_INVALID_ARG;
  const bool fp4 = kv_dtype == PD_KV_FP4_E2M1, kvs = ly.kv_shared != 0;
  if (ly.head_dim != 256 && ly.head_dim != 512 && (fp4 || ly.head_dim != 128)) return PD_ERR_UNSUPPORTED;
  const long long slots = (long long)ly.num_pages * ly.page_size;
  if (slots > 0x7fffffffLL || ly.num_kv_heads > (1 << 20)) return PD_ERR_UNSUPPORTED;
  if (fp4 && (k_exp < -64 || k_exp > 64 || v_exp < -64 || v_exp > 64 || (kvs && v_exp != k_exp)))
    return PD_ERR_INVALID_ARG;
  if (num_tokens == 0) return PD_OK;
  const int64_t row = (int64_t)ly.num_kv_heads * ly.head_dim;
  if (!k_rows || !slot_map || !k_pool || !device_flags || !aligned(k_rows, 16) || !aligned(k_pool, 16) ||
      !aligned(slot_map, 4) || !aligned(device_flags, 4) || k_stride < row || k_stride % 8 != 0 ||
      k_stride > (INT64_MAX >> 33))
    return PD_ERR_INVALID_ARG;
  if (!kvs && (!v_rows || !v_pool || v_pool == k_pool || !aligned(v_rows, 16) || !aligned(v_pool, 16) ||
               v_stride < row || v_stride % 8 != 0 || v_stride > (INT64_MAX >> 33)))
    return PD_ERR_INVALID_ARG;
  if (kvs && v_pool && v_pool != k_pool) return PD_ERR_INVALID_ARG;
  if (kv_dtype != PD_KV_BF16) {
    const uintptr_t a = fp4 ? 16 : 4;
    if (!k_scale || !aligned(k_scale, a)) return PD_ERR_INVALID_ARG;
    if (!kvs && (!v_scale || !aligned(v_scale, a) || (fp4 && v_scale == k_scale))) return PD_ERR_INVALID_ARG;
    if (kvs && v_scale && v_scale != k_scale) return PD_ERR_INVALID_ARG;
  }
  RowsParams p = {};
  p.rows[0] = static_cast<uint16_t*>(const_cast<void*>(k_rows));
  p.rows[1] = kvs ? nullptr : static_cast<uint16_t*>(const_cast<void*>(v_rows));
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.pool[0] = static_cast<uint8_t*>(const_cast<void*>(k_pool));
  p.pool[1] = static_cast<uint8_t*>(const_cast<void*>(v_pool));
  p.scale[0] = const_cast<void*>(k_scale);
  p.scale[1] = const_cast<void*>(v_scale);
  p.up[0] = std::ldexp(1.f, write ? -k_exp : k_exp);
  p.up[1] = std::ldexp(1.f, write ? -v_exp : v_exp);
  p.slot_map = slot_map;
  p.flags = device_flags;
  p.num_tokens = num_tokens;
  p.heads = ly.num_kv_heads;
  p.dim = ly.head_dim;
  p.page_size = ly.page_size;
  p.num_slots = slots;
  // runs of up to 16 tokens, shorter while that leaves a GB300's 152 SMs less than two CTAs each (304)
  p.run = kRowsMaxRun;
  while (p.run > 1 && (long long)num_tokens < 304ll * p.run) p.run /= 2;
  *out = p;
  return PD_OK;
}

pd_status launch_rows(const RowsParams& p, bool kvs, void (*kernel)(RowsParams), void* stream) {
  if (p.num_tokens == 0) return PD_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.num_tokens + p.run - 1) / p.run), kvs ? 1 : 2);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

pd_status write_fp4(const pd_layer_desc* layer, int32_t num_tokens, const void* k_in, const void* v_in,
                    int64_t k_stride, int64_t v_stride, const int32_t* slot_map, void* k_pool, void* v_pool,
                    void* k_scale, void* v_scale, int32_t k_exp, int32_t v_exp, uint32_t* device_flags, void* stream) {
  RowsParams p = {};
  const pd_status st = rows_params(layer, PD_KV_FP4_E2M1, num_tokens, k_in, v_in, k_stride, v_stride, slot_map, k_pool,
                                   v_pool, k_scale, v_scale, k_exp, v_exp, device_flags, true, &p);
  if (st != PD_OK) return st;
  const bool kvs = layer->kv_shared != 0;
  const bool wide = aligned(k_in, 32) && k_stride % 16 == 0 && (kvs || (aligned(v_in, 32) && v_stride % 16 == 0));
  return launch_rows(p, kvs, wide ? write_fp4_kernel<true> : write_fp4_kernel<false>, stream);
}

pd_status read_rows(const pd_layer_desc* layer, int kv_dtype, int32_t num_tokens, const int32_t* slot_map,
                    const void* k_pool, const void* v_pool, const void* k_scale, const void* v_scale, int32_t k_exp,
                    int32_t v_exp, void* k_out, void* v_out, int64_t k_stride, int64_t v_stride,
                    uint32_t* device_flags, void* stream) {
  RowsParams p = {};
  const pd_status st = rows_params(layer, kv_dtype, num_tokens, k_out, v_out, k_stride, v_stride, slot_map, k_pool,
                                   v_pool, k_scale, v_scale, k_exp, v_exp, device_flags, false, &p);
  if (st != PD_OK) return st;
  const bool kvs = layer->kv_shared != 0;
  const bool wide = aligned(k_out, 32) && k_stride % 16 == 0 && (kvs || (aligned(v_out, 32) && v_stride % 16 == 0));
  return launch_rows(p, kvs,
                     kv_dtype == PD_KV_FP4_E2M1 ? (wide ? read_slots_kernel<PD_KV_FP4_E2M1, true> : read_slots_kernel<PD_KV_FP4_E2M1, false>)
                     : kv_dtype == PD_KV_FP8_E4M3
                         ? (wide ? read_slots_kernel<PD_KV_FP8_E4M3, true> : read_slots_kernel<PD_KV_FP8_E4M3, false>)
                         : (wide ? read_slots_kernel<PD_KV_BF16, true> : read_slots_kernel<PD_KV_BF16, false>),
                     stream);
}

}  // namespace
}  // namespace pd

extern "C" {

pd_status paged_decode_write_slots_fp4(const pd_layer_desc* layer, int32_t num_tokens, const void* k_in,
                                       const void* v_in, int64_t k_stride, int64_t v_stride,
                                       const int32_t* slot_map, void* k_pool, void* v_pool, void* k_scale,
                                       void* v_scale, int32_t k_exp, int32_t v_exp, uint32_t* device_flags,
                                       void* stream) {
  return pd::write_fp4(layer, num_tokens, k_in, v_in, k_stride, v_stride, slot_map, k_pool, v_pool, k_scale, v_scale,
                       k_exp, v_exp, device_flags, stream);
}

pd_status paged_decode_read_slots(const pd_layer_desc* layer, int32_t num_tokens, const int32_t* slot_map,
                                  const void* k_pool, const void* v_pool, void* k_out, void* v_out, int64_t k_stride,
                                  int64_t v_stride, uint32_t* device_flags, void* stream) {
  return pd::read_rows(layer, PD_KV_BF16, num_tokens, slot_map, k_pool, v_pool, nullptr, nullptr, 0, 0, k_out, v_out,
                       k_stride, v_stride, device_flags, stream);
}

pd_status paged_decode_read_slots_fp8(const pd_layer_desc* layer, int32_t num_tokens, const int32_t* slot_map,
                                      const void* k_pool, const void* v_pool, const float* k_scale,
                                      const float* v_scale, void* k_out, void* v_out, int64_t k_stride,
                                      int64_t v_stride, uint32_t* device_flags, void* stream) {
  return pd::read_rows(layer, PD_KV_FP8_E4M3, num_tokens, slot_map, k_pool, v_pool, k_scale, v_scale, 0, 0, k_out,
                       v_out, k_stride, v_stride, device_flags, stream);
}

pd_status paged_decode_read_slots_fp4(const pd_layer_desc* layer, int32_t num_tokens, const int32_t* slot_map,
                                      const void* k_pool, const void* v_pool, const void* k_scale,
                                      const void* v_scale, int32_t k_exp, int32_t v_exp, void* k_out, void* v_out,
                                      int64_t k_stride, int64_t v_stride, uint32_t* device_flags, void* stream) {
  return pd::read_rows(layer, PD_KV_FP4_E2M1, num_tokens, slot_map, k_pool, v_pool, k_scale, v_scale, k_exp, v_exp,
                       k_out, v_out, k_stride, v_stride, device_flags, stream);
}

pd_status paged_decode_write_slots_fp4_args(const pd_slot_rows_args* a) {
  if (!a) return PD_ERR_INVALID_ARG;
  return pd::write_fp4(a->layer, a->num_tokens, a->k_rows, a->v_rows, a->k_stride, a->v_stride, a->slot_map, a->k_pool,
                       a->v_pool, a->k_scale, a->v_scale, a->k_exp, a->v_exp, a->device_flags, a->stream);
}

pd_status paged_decode_read_slots_args(const pd_slot_rows_args* a) {
  if (!a || !a->layer) return PD_ERR_INVALID_ARG;
  const int kv = a->layer->kv_dtype;
  if (kv != PD_KV_BF16 && kv != PD_KV_FP8_E4M3 && kv != PD_KV_FP4_E2M1) return PD_ERR_INVALID_ARG;
  return pd::read_rows(a->layer, kv, a->num_tokens, a->slot_map, a->k_pool, a->v_pool, a->k_scale, a->v_scale,
                       kv == PD_KV_FP4_E2M1 ? a->k_exp : 0, kv == PD_KV_FP4_E2M1 ? a->v_exp : 0, a->k_rows, a->v_rows,
                       a->k_stride, a->v_stride, a->device_flags, a->stream);
}

}  // extern "C"
