// Stage 1 of paged decode attention over a 4-bit cache (sm_103a): one CTA per
// (KV piece, KV head and column tile, request) streams the piece's codes and
// block scales once and serves up to CC query rows ("columns") of that KV head.
//
// Mathematics: a cached element is e2m1(code) * e4m3(scale of its 16 dims) *
// 2^exp. Scores S = K q^T are a product of two block-scaled 4-bit operands: the
// query row is written as kFp4Terms e2m1 terms, each with its own scale per 16
// dims, the next term taking what the one before left over. A term leaves at
// most 0.177 of its block's largest, so six leave 2^-14.9 of it (the row is
// first brought to [2^10, 2^11) by a power of two, so that the last terms'
// scales still are e4m3 numbers). K then needs no widening at all: the tensor
// core takes codes and scales as they lie in the cache (tcgen05.mma
// kind::mxf4nvf4, 128 tokens x CC * terms columns x 64 dims).
// V's scales lie along the head dims, across the sum over tokens that P V is,
// so V is widened: codes to f16 pairs of two tokens, times the pair of their
// scales (exact: 2 and 4 significant bits), and multiplied by mma.sync.
//
// Roles (one CTA an SM): warp 12 copies tiles of 128 tokens (TMA: codes;
// bulk copies: scales) into the rings; warp 13 issues the score products;
// warps 0-3 write the tile's K scales to tensor memory, read the scores of
// their quarter of the tile (a lane a token), keep its running maximum and sum
// (each quarter its own, joined at the end) and leave P in shared memory as
// f16; warps 4-11 accumulate P V, two warps a quarter (d 512: a half of the
// dims each; d 256: 16 of the 32 tokens each).
// P is held as 2^15 times the probability relative to the running maximum, so
// that f16 keeps tokens down to 2^-39 of the largest.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "fp4.h"
#include "paged_decode.h"
#include "tcgen05.cuh"

namespace pd {
namespace {

constexpr float kPShift = 15.f;

// D[tmem] (+)= A . B over 64 dims, both e2m1 with an e4m3 scale per 16 dims.
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
      : "memory");
}

// Four bytes of two e2m1 codes -> four f16 pairs (low code in the low half), exact.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Four e4m3 bytes -> two f16 pairs, exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The low nibbles of x beside those of y: bytes (x's low code, y's low code).
__device__ __forceinline__ uint32_t pair_codes(uint32_t x, uint32_t y) { return (x & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u); }

// A float's bits in an order of whole numbers.
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// The query rows behind a CTA's columns: column c is pair tile * CC + c of the
// request's T x group (token, head) pairs, token-major.
template <class C>
struct Columns {
  int b, g, first, T, group, Hq;
  __device__ __forceinline__ explicit Columns(const Fp4Params& p) {
    b = blockIdx.z;
    g = blockIdx.y / p.col_tiles;
    first = (blockIdx.y % p.col_tiles) * C::CC;
    T = p.query_tokens;
    group = p.group;
    Hq = p.num_q_heads;
  }
  __device__ __forceinline__ bool valid(int c) const { return first + c < T * group; }
  __device__ __forceinline__ int token(int c) const { return (first + c) / group; }
  __device__ __forceinline__ size_t row(int c) const {
    const int pr = first + c;
    return ((size_t)b * T + pr / group) * Hq + (size_t)g * group + pr % group;
  }
};

// Byte of (row, byte of the row) in a swizzled tile of codes.
template <class C>
__device__ __forceinline__ uint32_t code_offset(int row, int byte) {
  const int sl = byte >> 7, c = (byte >> 4) & 7;
  return (row >> 3) * (C::SL * 1024) + sl * 1024 + (row & 7) * 128 + ((c ^ (row & 7)) << 4) + (byte & 15);
}

// The query rows of the CTA's columns as terms in shared memory, by 8 warps:
// one takes 256 dims of a row, a lane 8 of them, two lanes a block of 16.
template <class C>
__device__ __forceinline__ void write_query_terms(const Fp4Params& p, const Columns<C>& cm, uint8_t* smem, int warp,
                                                  int lane) {
  constexpr int ITEMS = C::CC * C::SL, EACH = (ITEMS + 7) / 8;
  uint4 w[EACH];
  uint32_t big[EACH];
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int item = warp + 8 * k, col = item / C::SL, part = item % C::SL;
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    w[k] = o;
    if (item < ITEMS && cm.valid(col)) {
      const uint4* row = reinterpret_cast<const uint4*>(p.q + cm.row(col) * C::D) + lane;
      w[k] = __ldg(row + part * 32);
      if (C::SL == 2) o = __ldg(row + (part ^ 1) * 32);  // (for the row's largest)
    }
    uint32_t m = 0;
#pragma unroll
    for (uint32_t v : {w[k].x, w[k].y, w[k].z, w[k].w, o.x, o.y, o.z, o.w}) m = __vmaxu2(m, v & 0x7fff7fffu);
    big[k] = max(m << 16, m & 0xffff0000u);
  }
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int item = warp + 8 * k, col = item / C::SL, part = item % C::SL;
    if (item >= ITEMS) break;
    // the row's largest magnitude, as whole numbers (infinity and NaN are the largest)
    const uint32_t top = __reduce_max_sync(kFullMask, big[k]);
    const bool odd = top >= 0x7f800000u;  // a NaN or an infinity: the row's scores are NaN
    // brings the largest to [2^10, 2^11) (a row that is below 2^-116 altogether: as near as a factor of 2^126 does)
    const int shift = min(126, 137 - (int)(top >> 23));
    const float up = __int_as_float((127 + shift) << 23);
    const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = odd ? 0.f : __uint_as_float(v[i] << 16) * up;
      x[2 * i + 1] = odd ? 0.f : __uint_as_float(v[i] & 0xffff0000u) * up;
    }
#pragma unroll
    for (int t = 0; t < kFp4Terms; ++t) {
      float a = fmaxf(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))),
                      fmaxf(fmaxf(fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7]))));
      a = fmaxf(a, __shfl_xor_sync(kFullMask, a, 1));
      uint16_t s8;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(a * (1.f / 6.f)));
      uint32_t s16;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"(s8));
      const float s = __half2float(__ushort_as_half((unsigned short)(s16 & 0xffffu)));
      float r;  // (what a term leaves over, the next one takes: its rounding need not be exact)
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
      r = s > 0.f ? r : 0.f;
      uint32_t codes;
      asm("{\n\t.reg .b8 a, b, c, d;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
          "mov.b32 %0, {a, b, c, d};\n\t}"
          : "=r"(codes)
          : "f"(x[0] * r), "f"(x[1] * r), "f"(x[2] * r), "f"(x[3] * r), "f"(x[4] * r), "f"(x[5] * r), "f"(x[6] * r),
            "f"(x[7] * r));
      if (t + 1 < kFp4Terms) {
        uint32_t f[4];
        e2m1x8_to_f16x8(codes, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
          x[2 * i] = fmaf(-two.x, s, x[2 * i]);
          x[2 * i + 1] = fmaf(-two.y, s, x[2 * i + 1]);
        }
      }
      const int n = t * C::CC + col;
      *reinterpret_cast<uint32_t*>(smem + C::Q_OFFSET + code_offset<C>(n, part * 128 + lane * 4)) = codes;
      if ((lane & 1) == 0)
        smem[C::QSF_OFFSET + n * C::ROW_SF + part * 16 + lane / 2] = odd ? (uint8_t)0x7f : (uint8_t)s8;
    }
    if (part == 0 && lane == 0)
      reinterpret_cast<float*>(smem + C::COL_OFFSET)[col] = p.scale_log2 * __int_as_float((127 - shift) << 23);
  }
  // rows beyond the terms: zeros
  constexpr int USED = C::CC * kFp4Terms;
  for (int i = warp * 32 + lane; i < (C::N - USED) * C::ROW_SF; i += 256) smem[C::QSF_OFFSET + USED * C::ROW_SF + i] = 0;
  for (int i = warp * 32 + lane; i < (C::N - USED) * (C::D / 32); i += 256)
    *reinterpret_cast<uint4*>(smem + C::Q_OFFSET + code_offset<C>(USED + i / (C::D / 32), (i % (C::D / 32)) * 16)) =
        make_uint4(0u, 0u, 0u, 0u);
}

// 16 bytes global -> shared, counted by cp_async_arrive.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// An arrival on `bar` (one that its count holds) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Two e4m3 scales, NaN as zero.
__device__ __forceinline__ uint32_t without_nan(uint32_t s) {
  if ((s & 0x7fu) == 0x7fu) s &= 0xff00u;
  if ((s & 0x7f00u) == 0x7f00u) s &= 0xffu;
  return s;
}

// Sum over tokens of 16 tokens x 256 dims: rows row0 .. row0 + 15 of a tile of V, its slab `sl`.
// b0, b1: P of tokens 2 (lane % 4) + {0, 1} and + {8, 9}, column lane / 4.
// ok: a bit for each of this lane's four tokens (2r, 2r + 1, 2r + 8, 2r + 9) whose row counts; drop: NaN scales are taken
// as zeros.
template <class C>
__device__ __forceinline__ void pv_block(float (&acc)[16][4], const uint8_t* tile, int row0, int sl, uint32_t b0,
                                         uint32_t b1, uint32_t ok, bool drop, int lane) {
  const int qh = lane >> 2, r = lane & 3;
  const uint8_t* g0 = tile + (row0 >> 3) * (C::SL * 1024) + sl * 1024;
  const uint8_t* g1 = g0 + C::SL * 1024;
  const int ra = 2 * r, rb = ra + 1;
  const uint4 xa = *reinterpret_cast<const uint4*>(g0 + ra * 128 + ((qh ^ ra) << 4));
  const uint4 xb = *reinterpret_cast<const uint4*>(g0 + rb * 128 + ((qh ^ rb) << 4));
  const uint4 xc = *reinterpret_cast<const uint4*>(g1 + ra * 128 + ((qh ^ ra) << 4));
  const uint4 xd = *reinterpret_cast<const uint4*>(g1 + rb * 128 + ((qh ^ rb) << 4));
  // scales of blocks 2 qh, 2 qh + 1 of the slab; a row that does not count has scale 0
  const uint8_t* sf = tile + C::CODE_BYTES + (row0 + ra) * C::ROW_SF + sl * 16 + 2 * qh;
  uint32_t sa = *reinterpret_cast<const uint16_t*>(sf), sb = *reinterpret_cast<const uint16_t*>(sf + C::ROW_SF);
  uint32_t sc = *reinterpret_cast<const uint16_t*>(sf + 8 * C::ROW_SF);
  uint32_t sd = *reinterpret_cast<const uint16_t*>(sf + 9 * C::ROW_SF);
  if (ok != 15u) {
    sa = (ok & 1u) ? sa : 0u;
    sb = (ok & 2u) ? sb : 0u;
    sc = (ok & 4u) ? sc : 0u;
    sd = (ok & 8u) ? sd : 0u;
  }
  if (drop) {
    sa = without_nan(sa);
    sb = without_nan(sb);
    sc = without_nan(sc);
    sd = without_nan(sd);
  }
  uint32_t s01[2], s23[2];  // (token, next token) of either block
  e4m3x4_to_f16x4(__byte_perm(sa, sb, 0x5140), s01[0], s01[1]);
  e4m3x4_to_f16x4(__byte_perm(sc, sd, 0x5140), s23[0], s23[1]);
  const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
  const uint32_t wc[4] = {xc.x, xc.y, xc.z, xc.w}, wd[4] = {xd.x, xd.y, xd.z, xd.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    // word w: dims 8 w + 0 .. 7 of the lane's 32; even dims in the low nibbles
    uint32_t e01[4], o01[4], e23[4], o23[4];
    e2m1x8_to_f16x8(pair_codes(wa[w], wb[w] << 4), e01);
    e2m1x8_to_f16x8(pair_codes(wa[w] >> 4, wb[w]), o01);
    e2m1x8_to_f16x8(pair_codes(wc[w], wd[w] << 4), e23);
    e2m1x8_to_f16x8(pair_codes(wc[w] >> 4, wd[w]), o23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mma_f16(acc[w * 4 + i], mul_f16x2(e01[i], s01[w >> 1]), mul_f16x2(o01[i], s01[w >> 1]),
              mul_f16x2(e23[i], s23[w >> 1]), mul_f16x2(o23[i], s23[w >> 1]), b0, b1);
  }
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) stage1_fp4_kernel(const __grid_constant__ Fp4Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFFSET);
  uint64_t* full = bars;                       // [NK + NV]: K's ring, then V's
  uint64_t* empty = full + C::NK + C::NV;      // [NK + NV]
  uint64_t* sf_ready = empty + C::NK + C::NV;  // [2] K scales in tensor memory
  uint64_t* s_full = sf_ready + 2;             // [2] scores computed
  uint64_t* s_empty = s_full + 2;              // [2] scores read
  uint64_t* p_full = s_empty + 2;              // [4][2]
  uint64_t* p_empty = p_full + 8;              // [4][2]
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
  uint32_t* valid = reinterpret_cast<uint32_t*>(smem + C::VALID_OFFSET);
  constexpr int kCopyWarp = 12, kMmaWarp = 13;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool early = p.early_kv != 0 && warp == kCopyWarp;

  if (tid == kCopyWarp * 32) {
    prefetch_tensormap(&p.kmap);
    if (!C::KVS) prefetch_tensormap(&p.vmap);
#pragma unroll 1
    for (int s = 0; s < C::NK + C::NV; ++s) {
      mbar_init(&full[s], 33);  // the codes' byte count, and every copying lane's scales
      // K: the score product's end; V: the 8 PV warps; K = V: both
      mbar_init(&empty[s], C::KVS ? 9 : (s < C::NK ? 1 : 8));
    }
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sf_ready[s], 4);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 4);
    }
#pragma unroll 1
    for (int s = 0; s < 8; ++s) {
      mbar_init(&p_full[s], 1);
      mbar_init(&p_empty[s], 2);
    }
    fence_barrier_init();
  }
  if (warp == kCopyWarp) {
    __syncwarp();
    named_bar_arrive(4, C::THREADS);
  }
  // tensor memory: scores [2] at columns 0 and 64, K scales [2] at 128 and 160, query scales at 192
  if (warp == kMmaWarp) tmem_alloc<1>(tmem_at, 256);
  if (!early) grid_dependency_wait();

  const Columns<C> cm(p);
  const int split = blockIdx.x, b = cm.b, g = cm.g;
  const int cap = p.max_pages * p.page_size;
  const int32_t* table = p.block_tables + (size_t)b * p.max_pages;
  int L = p.seq_lens[b];
  if (L < 0 || L > cap || (cm.T > 1 && L < cm.T)) {
    if (tid == 0) atomicOr(p.err, kErrBadSeqLen);
    L = L < 0 ? 0 : (L > cap ? cap : L);
  }
  // attended range [lo, hi) of the CTA's query rows: the union of their tokens' causal ranges
  int j_last = cm.token(C::CC - 1);
  if (j_last > cm.T - 1) j_last = cm.T - 1;
  const int hi = max(0, L - cm.T + j_last + 1);
  const int first_hi = L - cm.T + cm.token(0) + 1;
  const int lo = (p.window > 0 && first_hi > p.window) ? first_hi - p.window : 0;
  const int base = (lo / 16) * 16;
  const long long piece_lo = (long long)base + (long long)split * p.chunk_tokens;
  const int tlo = (int)min((long long)hi, piece_lo > lo ? piece_lo : lo);
  const long long piece_hi = (split == p.num_splits - 1) ? (long long)hi : piece_lo + p.chunk_tokens;
  const int thi = (int)(piece_hi < hi ? piece_hi : hi);
  const int t_base = (tlo / 16) * 16;
  const int tiles = thi > tlo ? (thi - t_base + kFp4Tile - 1) / kFp4Tile : 0;

  float* my_lse = reinterpret_cast<float*>(smem + C::COEF_OFFSET) + 4 * C::CC;  // [CC]
  float* my_out = reinterpret_cast<float*>(smem + C::OUT_OFFSET);                // [CC][D]
  if (!early) grid_launch_dependents();
  uint32_t tmem = 0;
  if (warp != kCopyWarp) {
    // the barriers and tensor memory are there (the copies do not wait for the other warps)
    named_bar_sync(4, C::THREADS);
    tmem_fence_after();
    tmem = *tmem_at;
  }
  const uint32_t t_s = tmem, t_sfa = tmem + 128, t_sfb = tmem + 192;

  if (tiles > 0 && warp == kCopyWarp) {
    // ---- copies: lane l takes the codes of the 16 tokens l % 8 of a tile (lanes 0-7 K's, 8-15 V's); the scales of
    // each 16 tokens are 16 bytes a lane, by cp.async: as bulk copies they were
    // half of all, and the copy engine's rate (~110 cycles a copy) bound the kernel
    const uint64_t policy = l2_evict_first_policy();
    const int blk = lane & 7, kind = lane >> 3;
    bool waited = !early, stop = false;
    uint32_t err_bits = 0;
    // rows from here on may still be written by the kernel in front
    const int fresh_from = L - p.query_tokens;
    auto page_of = [&](int i) {
      const int t = t_base + i * kFp4Tile + blk * 16;
      return t < thi ? __ldg(table + t / p.page_size) : -1;
    };
    int page = page_of(0);
    int done = 0;  // items whose copies went out
#pragma unroll 1
    for (int i = 0; i < tiles && !stop; ++i) {
      const int next = i + 1 < tiles ? page_of(i + 1) : -1;
      const int t = t_base + i * kFp4Tile + blk * 16;
      const bool there = t < thi, ok = there && (unsigned)page < (unsigned)p.num_pages;
      if (there && !ok) err_bits |= kErrBadPage;
      const uint32_t bits = __ballot_sync(kFullMask, ok) & 0xffu;
      if (!waited && (i >= C::NK || (!C::KVS && i >= C::NV) || t_base + (i + 1) * kFp4Tile > fresh_from)) {
        grid_dependency_wait();
        grid_launch_dependents();
        waited = true;
      }
      const int row0 = ok ? (page * p.num_kv_heads + g) * p.page_size + t % p.page_size : 0;
#pragma unroll
      for (int v = 0; v < (C::KVS ? 1 : 2); ++v) {
        const int n = v ? C::NV : C::NK, st = (v ? C::NK : 0) + i % n, round = i / n;
        if (round > 0) {
          const bool freed = mbar_wait(&empty[st], (round - 1) & 1);
          if (__any_sync(kFullMask, !freed)) {
            err_bits |= kErrTimeout;
            stop = true;
            break;
          }
        }
        if (lane == 0) {
          valid[st] = bits;
          if (bits)
            mbar_arrive_expect_tx(&full[st], __popc(bits) * (16 * C::D / 2) + (v ? 0 : p.stall_bytes));
          else
            mbar_arrive(&full[st]);
        }
        __syncwarp();
        uint8_t* item = smem + st * C::ITEM_BYTES;
        if (ok && kind == v)
          tma_load_4d(item + blk * 16 * (C::D / 2), v ? &p.vmap : &p.kmap, 0, 0, 0, row0 / 8, &full[st], policy);
        constexpr int LANES = C::ROW_SF;  // 16-byte pieces of 16 tokens' scales
        const uint8_t* sf = v ? p.v_sf : p.k_sf;
#pragma unroll
        for (int k = 0; k < 8; k += 32 / LANES) {
          const int at = k + lane / LANES;  // the 16 tokens this lane copies a piece of
          const int row = __shfl_sync(kFullMask, row0, at);
          if ((bits >> at) & 1u)
            cp_async16(item + C::CODE_BYTES + at * 16 * C::ROW_SF + (lane % LANES) * 16,
                       sf + (size_t)row * C::ROW_SF + (lane % LANES) * 16);
        }
        cp_async_arrive(&full[st]);
        done = C::KVS ? i + 1 : 2 * i + v + 1;
      }
      page = next;
    }
    if (!waited) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
    // no copy may still be landing when the shared memory is used for something else
    const unsigned long long deadline = global_timer_ns() + kWaitTimeoutNs;
    const int k_items = C::KVS ? done : (done + 1) / 2, v_items = C::KVS ? 0 : done / 2;
    for (int s = lane; s < C::NK + C::NV; s += 32) {
      const int n = s < C::NK ? C::NK : C::NV, at = s < C::NK ? s : s - C::NK, items = s < C::NK ? k_items : v_items;
      if (at >= items) continue;
      const int last = at + n * ((items - 1 - at) / n);
      if (!mbar_wait_until(&full[s], (last / n) & 1, deadline)) err_bits |= kErrTimeout;
    }
    err_bits = __reduce_or_sync(kFullMask, err_bits);
    if (lane == 0 && err_bits) atomicOr(p.err, err_bits);
  } else if (early) {
    grid_dependency_wait();
    grid_launch_dependents();
  }

  if (tiles > 0 && warp != kCopyWarp) {
    // the query's terms, by the PV warps
    if (warp >= 4 && warp < kCopyWarp) {
      write_query_terms<C>(p, cm, smem, warp - 4, lane);
      fence_proxy_async_smem();
    }
    named_bar_sync(1, (C::WARPS - 1) * 32);
    if (warp < 4) {
      // ---- softmax warps: rows 32 warp .. + 31 of every tile
      const uint32_t quarter = (uint32_t)warp << 21;  // this warp's lanes of tensor memory
      {
        // the query terms' scales: lane l, column 4 k + j: the 4 bytes of row l + 32 j, dims 64 k .. 64 k + 63
#pragma unroll
        for (int k0 = 0; k0 < C::KSTEPS; k0 += 2) {
          uint32_t r8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = lane + 32 * (i & 3);
            r8[i] = row < C::N ? *reinterpret_cast<const uint32_t*>(smem + C::QSF_OFFSET + row * C::ROW_SF +
                                                                    (k0 + (i >> 2)) * 4)
                               : 0u;
          }
          tmem_st(t_sfb + quarter + k0 * 4, r8);
        }
      }
      // K scales of tile i into tensor memory; every quarter of its lanes holds all 128 rows'
      bool good = true;
      uint32_t here_next = 0;  // the 16-token blocks that the tile holds
      auto put_scales = [&](int i) {
        const int st = i % C::NK;
        const bool landed = mbar_wait(&full[st], (i / C::NK) & 1);
        if (__any_sync(kFullMask, !landed)) {
          good = false;
          return;
        }
        const uint8_t* sf = smem + st * C::ITEM_BYTES + C::CODE_BYTES;
#pragma unroll
        for (int k0 = 0; k0 < C::KSTEPS; k0 += 4) {
          uint32_t r16[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(sf + (lane + 32 * j) * C::ROW_SF + k0 * 4);
            r16[j] = w.x;
            r16[4 + j] = w.y;
            r16[8 + j] = w.z;
            r16[12 + j] = w.w;
          }
          tmem_st(t_sfa + (i & 1) * 32 + quarter + k0 * 4, r16);
        }
        here_next = valid[st];
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_ready[i & 1]);
      };
      put_scales(0);
      float col_mul[C::CC];
      int col_hi[C::CC], col_lo[C::CC];
      float m_run[C::CC], l_run[C::CC];
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        col_mul[c] = reinterpret_cast<const float*>(smem + C::COL_OFFSET)[c];
        col_hi[c] = cm.valid(c) ? min(thi, L - cm.T + cm.token(c) + 1) : 0;
        col_lo[c] = max(tlo, (p.window > 0 && cm.valid(c)) ? L - cm.T + cm.token(c) + 1 - p.window : 0);
        m_run[c] = -INFINITY;
        l_run[c] = 0.f;
      }
#pragma unroll 1
      for (int i = 0; i < tiles && good; ++i) {
        const int buf = i & 1;
        const uint32_t here = here_next;
        // the next tile's scales first, if they are there already
        bool ahead = i + 1 < tiles && mbar_test(&full[(i + 1) % C::NK], ((i + 1) / C::NK) & 1);
        ahead = __all_sync(kFullMask, ahead);
        if (ahead) put_scales(i + 1);
        const bool scored = mbar_wait(&s_full[buf], (i >> 1) & 1);
        if (__any_sync(kFullMask, !scored)) {
          good = false;
          break;
        }
        tmem_fence_after();
        float s[C::CC];
        {
          uint32_t w[kFp4Terms * C::CC / 8][8];
#pragma unroll
          for (int k = 0; k < kFp4Terms * C::CC / 8; ++k) tmem_ld(w[k], t_s + buf * 64 + quarter + k * 8);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            float sum = 0.f;
#pragma unroll
            for (int t = kFp4Terms - 1; t >= 0; --t)
              sum += __uint_as_float(w[(t * C::CC + c) / 8][(t * C::CC + c) % 8]);
            s[c] = sum * col_mul[c];
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[buf]);
        const int row = warp * 32 + lane, t = t_base + i * kFp4Tile + row;
        const bool ok = (here >> (row >> 4)) & 1u;
        float pr[C::CC], alpha[C::CC];
#pragma unroll
        for (int c = 0; c < C::CC; ++c) {
          if (!(ok && t >= col_lo[c] && t < col_hi[c])) s[c] = -INFINITY;
          const float mn = fmaxf(m_run[c], unordered(__reduce_max_sync(kFullMask, ordered(s[c]))));
          alpha[c] = mn == -INFINITY ? 1.f : ex2(m_run[c] - mn);
          pr[c] = ex2(s[c] - (mn == -INFINITY ? 0.f : mn) + kPShift);
          l_run[c] = fmaf(l_run[c], alpha[c], pr[c]);
          m_run[c] = mn;
        }
        if (i >= 2) {
          const bool freed = mbar_wait(&p_empty[warp * 2 + buf], ((i >> 1) - 1) & 1);
          if (__any_sync(kFullMask, !freed)) {
            good = false;
            break;
          }
        }
        uint8_t* pb = smem + C::P_OFFSET + (warp * 2 + buf) * C::CC * C::P_ROW + lane * 2;
        float* al = reinterpret_cast<float*>(smem + C::ALPHA_OFFSET) + (warp * 2 + buf) * 8;
#pragma unroll
        for (int c = 0; c < C::CC; ++c) {
          *reinterpret_cast<__half*>(pb + c * C::P_ROW) = __float2half_rn(pr[c]);
          if (lane == c) al[c] = alpha[c];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[warp * 2 + buf]);
        if (!ahead && i + 1 < tiles) put_scales(i + 1);
      }
      if (!good && lane == 0) atomicOr(p.err, kErrTimeout);
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        float l = l_run[c];
#pragma unroll
        for (int m = 16; m; m >>= 1) l += __shfl_xor_sync(kFullMask, l, m);
        if (lane == 0) reinterpret_cast<float2*>(smem + C::ML_OFFSET)[warp * C::CC + c] = make_float2(m_run[c], l);
      }
    } else if (warp == kMmaWarp) {
      // ---- score products
      constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(C::N / 8) << 17) | (8u << 24);  // e2m1 x e2m1, e4m3 scales
      int issued = 0;
      bool good = true;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int st = i % C::NK, buf = i & 1;
        bool ready = mbar_wait(&full[st], (i / C::NK) & 1) && mbar_wait(&sf_ready[buf], (i >> 1) & 1);
        if (ready && i >= 2) ready = mbar_wait(&s_empty[buf], ((i >> 1) - 1) & 1);
        if (__any_sync(kFullMask, !ready)) {
          good = false;
          break;
        }
        tmem_fence_after();
        if (elect_one()) {
          const uint32_t a = smem_u32(smem + st * C::ITEM_BYTES), q = smem_u32(smem + C::Q_OFFSET);
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k) {
            const uint32_t off = (k >> 2) * 1024 + (k & 3) * 32;
            mma_fp4(t_s + buf * 64, smem_desc(a + off, 0, C::SL * 1024), smem_desc(q + off, 0, C::SL * 1024), kIdesc,
                    t_sfa + buf * 32 + k * 4, t_sfb + k * 4, k > 0);
          }
          mma_commit<1>(&s_full[buf]);
          mma_commit<1>(&empty[st]);
        }
        __syncwarp();
        issued = i + 1;
      }
      if (!good) {
        // what was issued ends before its operands and its result are used for something else
        if (issued > 0) mbar_wait(&s_full[(issued - 1) & 1], ((issued - 1) >> 1) & 1);
        if (lane == 0) atomicOr(p.err, kErrTimeout);
      }
    } else {
      // ---- PV warps
      const int qd = (warp - 4) >> 1, part = (warp - 4) & 1;
      const int qh = lane >> 2, r = lane & 3;
      // positions [all_lo, all_hi) are attended by every column
      const int all_hi = cm.T > 1 ? first_hi : hi;
      const int all_lo = p.window > 0 ? L - cm.T + j_last + 1 - p.window : 0;
      float acc[16][4];
#pragma unroll
      for (int m = 0; m < 16; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][k] = 0.f;
      bool good = true;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int n = C::KVS ? C::NK : C::NV, st = (C::KVS ? 0 : C::NK) + i % n, buf = i & 1;
        const bool ready = mbar_wait(&full[st], (i / n) & 1) && mbar_wait(&p_full[qd * 2 + buf], (i >> 1) & 1);
        if (__any_sync(kFullMask, !ready)) {
          good = false;
          break;
        }
        const uint8_t* tile = smem + st * C::ITEM_BYTES;
        const uint32_t here = valid[st];
        const int t0 = t_base + i * kFp4Tile + qd * 32;
        const uint8_t* pb = smem + C::P_OFFSET + (qd * 2 + buf) * C::CC * C::P_ROW + qh * C::P_ROW + r * 4;
        const float* al = reinterpret_cast<const float*>(smem + C::ALPHA_OFFSET) + (qd * 2 + buf) * 8;
        const float a0 = 2 * r < C::CC ? al[2 * r] : 1.f, a1 = 2 * r < C::CC ? al[2 * r + 1] : 1.f;
        if (__any_sync(kFullMask, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
          for (int m = 0; m < 16; ++m) {
            acc[m][0] *= a0;
            acc[m][1] *= a1;
            acc[m][2] *= a0;
            acc[m][3] *= a1;
          }
        }
        constexpr int BLOCKS = C::SL == 2 ? 2 : 1;  // 16-token blocks of this warp
        const int first = C::SL == 2 ? 0 : part, slab = C::SL == 2 ? part : 0;
        const int ta = t0 + first * 16;
        const uint32_t want = BLOCKS == 2 ? 3u : 1u;
        if (((here >> (qd * 2 + first)) & want) == want && ta >= tlo && ta + BLOCKS * 16 <= thi && ta >= all_lo &&
            ta + BLOCKS * 16 <= all_hi) {
          // every token is attended by every column
#pragma unroll
          for (int k = first; k < first + BLOCKS; ++k) {
            uint32_t b0 = 0, b1 = 0;
            if (C::CC == 8 || qh < C::CC) {
              b0 = *reinterpret_cast<const uint32_t*>(pb + k * 32);
              b1 = *reinterpret_cast<const uint32_t*>(pb + k * 32 + 16);
            }
            pv_block<C>(acc, tile, qd * 32 + k * 16, slab, b0, b1, 15u, false, lane);
          }
        } else {
#pragma unroll 1
        for (int k = first; k < first + BLOCKS; ++k) {
          const int tk = t0 + k * 16, row0 = qd * 32 + k * 16;
          if (!((here >> (row0 >> 4)) & 1u) || tk >= thi || tk + 16 <= tlo) continue;
          uint32_t b0 = 0, b1 = 0;
          if (C::CC == 8 || qh < C::CC) {
            b0 = *reinterpret_cast<const uint32_t*>(pb + k * 32);
            b1 = *reinterpret_cast<const uint32_t*>(pb + k * 32 + 16);
          }
          uint32_t ok = 15u;
          if (tk < tlo || tk + 16 > thi) {
            const int tr = tk + 2 * r;
            ok = (uint32_t)(tr >= tlo && tr < thi) | (uint32_t)(tr + 1 >= tlo && tr + 1 < thi) << 1 |
                 (uint32_t)(tr + 8 >= tlo && tr + 8 < thi) << 2 | (uint32_t)(tr + 9 >= tlo && tr + 9 < thi) << 3;
          }
          // Tokens that some columns attend and others do not (several query
          // tokens): a NaN there belongs to the former alone, but 0 * NaN is NaN,
          // so it is taken out of the product and put into their sums.
          const bool mixed = p.query_tokens > 1 && (tk + 16 > all_hi || tk < all_lo);
          if (mixed) {
            const uint8_t* sf = tile + C::CODE_BYTES + row0 * C::ROW_SF + slab * 16 + 2 * qh;
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
              const uint32_t two = *reinterpret_cast<const uint16_t*>(sf + j * C::ROW_SF);
              if (two == without_nan(two)) continue;
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const int c = 2 * r + hh, t = tk + j;
                if (c >= C::CC || !cm.valid(c) || t < tlo || t >= thi) continue;
                const int end = L - cm.T + cm.token(c) + 1;
                if (t >= end || (p.window > 0 && t < end - p.window)) continue;
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                  if ((two >> (m < 8 ? 0 : 8) & 0x7fu) != 0x7fu) continue;
                  acc[m][hh] = NAN;
                  acc[m][2 + hh] = NAN;
                }
              }
            }
          }
          pv_block<C>(acc, tile, row0, slab, b0, b1, ok, mixed, lane);
        }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&p_empty[qd * 2 + buf]);
          mbar_arrive(&empty[st]);
        }
      }
      if (!good && lane == 0) atomicOr(p.err, kErrTimeout);
      // every warp is done with the ring
      named_bar_sync(3, 8 * 32);
      float* comb = reinterpret_cast<float*>(smem) + (warp - 4) * C::CC * C::COMB_ROW + qh * 36;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        if (2 * r + hh >= C::CC) continue;
#pragma unroll
        for (int m = 0; m < 16; ++m)
          *reinterpret_cast<float2*>(comb + (2 * r + hh) * C::COMB_ROW + 2 * m) = make_float2(acc[m][hh], acc[m][2 + hh]);
      }
    }
  }
  __syncthreads();

  // ---- the quarters' sums joined
  float* coef = reinterpret_cast<float*>(smem + C::COEF_OFFSET);  // [4][CC]
  if (tid < C::CC) {
    float M = -INFINITY, sum = 0.f, f[4];
    const float2* ml = reinterpret_cast<const float2*>(smem + C::ML_OFFSET);
    if (tiles > 0) {
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[w * C::CC + tid].x);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = M == -INFINITY ? 0.f : ex2(ml[w * C::CC + tid].x - M);
        sum += f[w] * ml[w * C::CC + tid].y;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) coef[w * C::CC + tid] = sum != 0.f ? f[w] / sum * p.v_mul : 0.f;
    }
    my_lse[tid] = sum != 0.f ? (M + __log2f(sum) - kPShift) * 0.69314718055994530942f : -INFINITY;
  }
  __syncthreads();
  constexpr int D4 = C::D / 4;
  for (int e = tid; e < C::CC * D4; e += C::THREADS) {
    const int c = e / D4, dim = (e % D4) * 4;
    if (!cm.valid(c)) continue;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tiles > 0) {
      const int in = dim % 256 + 4 * ((dim % 256) / 32);
#pragma unroll
      for (int k = 0; k < (C::SL == 2 ? 4 : 8); ++k) {
        const int w = C::SL == 2 ? 2 * k + dim / 256 : k;
        const float f = coef[(w >> 1) * C::CC + c];
        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                          (w * C::CC + c) * C::COMB_ROW + in);
        o.x = fmaf(f, a.x, o.x);
        o.y = fmaf(f, a.y, o.y);
        o.z = fmaf(f, a.z, o.z);
        o.w = fmaf(f, a.w, o.w);
      }
    }
    if (p.direct_out) {
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + cm.row(c) * C::D + dim) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    } else if (p.cluster_merge) {
      *reinterpret_cast<float4*>(my_out + c * C::D + dim) = o;
    } else {
      const size_t row = cm.row(c) * p.num_splits + split;
      *reinterpret_cast<float4*>(p.o_part + row * C::D + dim) = o;
      if (dim == 0) p.lse_part[row] = my_lse[c];
    }
  }
  if (warp == kMmaWarp) tmem_dealloc<1>(tmem, 256);
  if (!p.cluster_merge) return;

  // ---- the pieces' results joined over distributed shared memory: each CTA of
  // the cluster a share of the elements, in piece order
  //   out = sum_s w_s o_s,  w_s = exp(lse_s - M) / sum_s' exp(lse_s' - M)
  cluster_sync_all();
  const int S = p.num_splits, rank = (int)cluster_ctarank();
  const uint32_t out_at = smem_u32(my_out), lse_at = smem_u32(my_lse);
  for (int e = rank * C::THREADS + tid; e < C::CC * D4; e += S * C::THREADS) {
    const int c = e / D4, dim = (e % D4) * 4;
    if (!cm.valid(c)) continue;
    float l[kFp4MaxCluster], M = -INFINITY, sum = 0.f;
    float4 v[kFp4MaxCluster];
#pragma unroll
    for (int s = 0; s < kFp4MaxCluster; ++s) {
      l[s] = s < S ? ld_dsmem_f32(map_smem_rank(lse_at + c * 4, s)) : -INFINITY;
      if (s < S) v[s] = ld_dsmem_f32x4(map_smem_rank(out_at + (c * C::D + dim) * 4, s));
    }
#pragma unroll
    for (int s = 0; s < kFp4MaxCluster; ++s) M = fmaxf(M, l[s]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kFp4MaxCluster; ++s) {
      if (s >= S || l[s] == -INFINITY) continue;
      const float w = ex2((l[s] - M) * 1.4426950408889634f);
      sum += w;
      o.x = fmaf(w, v[s].x, o.x);
      o.y = fmaf(w, v[s].y, o.y);
      o.z = fmaf(w, v[s].z, o.z);
      o.w = fmaf(w, v[s].w, o.w);
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + cm.row(c) * C::D + dim) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
  cluster_sync_all();  // nobody's shared memory goes while another reads it
}

}  // namespace

const void* fp4_kernel_ptr(int variant) {
  switch (variant) {
#define PD_FP4_CASE(ID, D, KVS, CC) \
  case ID:                          \
    return reinterpret_cast<const void*>(&stage1_fp4_kernel<Fp4Cfg<D, KVS, CC>>);
    PD_FOR_EACH_FP4(PD_FP4_CASE)
#undef PD_FP4_CASE
    default:
      return nullptr;
  }
}

bool plan_is_valid(const pd_plan* plan);
pd_status ensure_fp4_smem(int variant, const void* fn, int smem_bytes);
pd_status encode_code_map(CUtensorMap* map, const void* pool, const pd_layer_desc& ly);

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

pd_status decode_fp4(const pd_plan* plan, const void* q, const void* k_pool, const void* v_pool, const void* k_scale,
                     const void* v_scale, int32_t k_exp, int32_t v_exp, const int32_t* block_tables,
                     const int32_t* seq_lens, float scale, void* workspace, size_t workspace_bytes, void* out,
                     void* stream) {
  if (!plan_is_valid(plan) || plan->partial) return PD_ERR_INVALID_ARG;
  const pd_layer_desc& ly = plan->layer;
  if (!std::isfinite(scale) || k_exp < -64 || k_exp > 64 || v_exp < -64 || v_exp > 64) return PD_ERR_INVALID_ARG;
  const float scale_log2 = std::ldexp(scale * 1.4426950408889634f, k_exp);
  if (!std::isfinite(scale_log2)) return PD_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return PD_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes) return PD_ERR_WORKSPACE_TOO_SMALL;
  if (plan->batch == 0) return PD_OK;
  if (!q || !k_pool || !k_scale || !block_tables || !seq_lens || !out) return PD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(k_scale, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4))
    return PD_ERR_INVALID_ARG;
  if (ly.kv_shared) {
    if ((v_pool && v_pool != k_pool) || (v_scale && v_scale != k_scale) || v_exp != k_exp) return PD_ERR_INVALID_ARG;
    v_pool = k_pool;
    v_scale = k_scale;
  } else if (!v_pool || !v_scale || v_pool == k_pool || v_scale == k_scale || !aligned(v_pool, 16) ||
             !aligned(v_scale, 16)) {
    return PD_ERR_INVALID_ARG;
  }
  const void* fn = fp4_kernel_ptr(plan->variant);
  if (!fn) return PD_ERR_INVALID_ARG;
  pd_status st = ensure_fp4_smem(plan->variant - kFp4FirstId, fn, plan->smem_bytes);
  if (st != PD_OK) return st;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Fp4Params p;
  std::memset(&p, 0, sizeof(p));
  st = encode_code_map(&p.kmap, k_pool, ly);
  if (st != PD_OK) return st;
  if (ly.kv_shared)
    p.vmap = p.kmap;
  else if ((st = encode_code_map(&p.vmap, v_pool, ly)) != PD_OK)
    return st;
  p.q = static_cast<const uint16_t*>(q);
  p.k_sf = static_cast<const uint8_t*>(k_scale);
  p.v_sf = static_cast<const uint8_t*>(v_scale);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse_part = reinterpret_cast<float*>(ws + plan->lse_offset);
  p.o_part = reinterpret_cast<float*>(ws + plan->opart_offset);
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.scale_log2 = scale_log2;
  p.v_mul = std::ldexp(1.f, v_exp);
  p.direct_out = plan->num_splits == 1 ? 1 : 0;
  p.cluster_merge = plan->merge_mode == 2 ? 1 : 0;
  p.stall_bytes = plan->test_stall_bytes;
  p.early_kv = plan->early_kv;
  p.window = ly.window;
  p.num_pages = ly.num_pages;
  p.max_pages = ly.max_pages_per_seq;
  p.page_size = ly.page_size;
  p.num_q_heads = ly.num_q_heads;
  p.num_kv_heads = ly.num_kv_heads;
  p.num_splits = plan->num_splits;
  p.chunk_tokens = plan->chunk_tokens;
  p.query_tokens = plan->query_tokens;
  p.group = ly.num_q_heads / ly.num_kv_heads;
  p.col_tiles = plan->grid_y / ly.num_kv_heads;

  void* args[] = {&p};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan->grid_x, plan->grid_y, plan->grid_z);
  cfg.blockDim = dim3(plan->threads_per_cta);
  cfg.dynamicSmemBytes = plan->smem_bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  int na = 0;
  attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  if (p.cluster_merge) {
    // the pieces of one (request, KV head, column tile) are consecutive in x: one cluster
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = plan->num_splits;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
    (void)cudaGetLastError();
    return PD_ERR_CUDA;
  }
  return PD_OK;
}

}  // namespace
}  // namespace pd

extern "C" {

pd_status paged_decode_global_fp4(const pd_plan* plan, const void* q, const void* k_pool, const void* v_pool,
                                  const void* k_scale, const void* v_scale, int32_t k_exp, int32_t v_exp,
                                  const int32_t* block_tables, const int32_t* seq_lens, float scale, void* workspace,
                                  size_t workspace_bytes, void* out, void* stream) {
  if (!plan || plan->layer.window != 0 || plan->layer.kv_dtype != PD_KV_FP4_E2M1) return PD_ERR_INVALID_ARG;
  return pd::decode_fp4(plan, q, k_pool, v_pool, k_scale, v_scale, k_exp, v_exp, block_tables, seq_lens, scale,
                        workspace, workspace_bytes, out, stream);
}

pd_status paged_decode_window_fp4(const pd_plan* plan, const void* q, const void* k_pool, const void* v_pool,
                                  const void* k_scale, const void* v_scale, int32_t k_exp, int32_t v_exp,
                                  const int32_t* block_tables, const int32_t* seq_lens, int32_t window, float scale,
                                  void* workspace, size_t workspace_bytes, void* out, void* stream) {
  if (!plan || window <= 0 || plan->layer.window != window || plan->layer.kv_dtype != PD_KV_FP4_E2M1)
    return PD_ERR_INVALID_ARG;
  return pd::decode_fp4(plan, q, k_pool, v_pool, k_scale, v_scale, k_exp, v_exp, block_tables, seq_lens, scale,
                        workspace, workspace_bytes, out, stream);
}

}  // extern "C"
