// Stage 1 of paged decode attention over a 4-bit cache (sm_103a): one CTA per
// (KV piece, KV head and column tile, request) streams the piece's codes and
// block scales once and serves up to CC query rows ("columns") of that KV head.
//
// Mathematics: a cached element is e2m1(code) * e4m3(scale of its 16 dims) *
// 2^exp. All three products of a tile of 128 tokens run on tcgen05, and no
// cached element passes through the CUDA cores:
//   S = K q^T    kind::mxf4nvf4 on codes and scales as they lie in the cache. The
//                query row is written as kFp4Terms e2m1 terms, each with its own
//                scale per 16 dims, the next taking what the one before left
//                over. A term leaves at most 0.177 of its block's largest, so six
//                leave 2^-14.9 of it (the row is first brought to [2^10, 2^11) by
//                a power of two, so that the last terms' scales still are e4m3
//                numbers); the terms' scores are summed afterwards;
//   V^T = I V^T  the same kind with a unit matrix: V widened, scaled and turned,
//                128 dims at a time, exactly (one term a sum) and as fp32 in
//                tensor memory, where it is a tf32 operand as it is (two and four
//                significant bits make at most six);
//   O^T += V^T P^T  kind::tf32 with V^T out of tensor memory and P from shared
//                memory.
// Widening V for mma.sync instead (codes to f16, times their scales) took 200
// instructions a warp for 16 tokens of 256 dims, 1500 cycles a tile and
// sub-partition at best and 3500 in place; these products take about 1800 a tile
// of 512 dims in all, beside everything else.
//
// Softmax without a running rescale: a column's reference is the maximum of the
// first tile that holds a token it attends, and stays until a score exceeds it
// by 2^60 (tf32 has fp32's exponents), which rescales the sums.
//
// Roles (one CTA an SM): warps 0-3 softmax (a lane a token); 4-7 write the
// tiles' scales to tensor memory; 8, 9 copy codes (TMA), 10 scales (cp.async);
// 11 issues the products. Warps 0-7 read the sums at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "fp4.h"
#include "paged_decode.h"
#include "tcgen05.cuh"

namespace pd {
namespace {

constexpr float kRefRange = 60.f;  // log2 of how far a score may exceed its column's reference
// tensor memory columns: scores [S_BUFS][N], scales of V, of the unit matrix, V^T [2][128], sums [CHUNKS][16],
// scales of K, of the query
constexpr uint32_t kTmemS = 0, kTmemSfv = 64, kTmemSfi = 96, kTmemVt = 128, kTmemO = 384, kTmemSfk = 448,
                   kTmemSfq = 480, kTmemCols = 512;

// D[tmem] (+)= A . B over 64 dims, both e2m1 with an e4m3 scale per 16 dims.
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] . B over 8 tokens, tf32.
__device__ __forceinline__ void mma_tf32(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
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

// Four e4m3 scales: 0x80 in the bytes that are NaN.
__device__ __forceinline__ uint32_t nan_scales(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

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
  constexpr int SB = C::S_BUFS, CH = C::CHUNKS, RINGS = C::NK + C::NV;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFFSET);  // [RINGS]: K's ring, then V's
  uint64_t* empty = full + RINGS;                                      // [RINGS]
  uint64_t* sfk_ready = empty + RINGS;                                 // K's scales in tensor memory
  uint64_t* sfv_ready = sfk_ready + 1;                                 // V's
  uint64_t* s_full = sfv_ready + 1;                                    // [2] scores computed
  uint64_t* s_empty = s_full + 2;                                      // [2] scores read
  uint64_t* vt_full = s_empty + 2;                                     // [2] a chunk of V^T there
  uint64_t* vt_empty = vt_full + 2;                                    // [2] and used
  uint64_t* dq_done = vt_empty + 2;                                    // a tile's V^T all there
  uint64_t* p_full = dq_done + 1;                                      // [2]
  uint64_t* p_empty = p_full + 2;                                      // [2]: the tile is in the sums
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(full + C::NUM_BARS);
  uint32_t* valid = reinterpret_cast<uint32_t*>(smem + C::VALID_OFFSET);
  volatile uint32_t* failed_at = reinterpret_cast<uint32_t*>(smem + C::FAILED_OFFSET);
  uint32_t* poison = reinterpret_cast<uint32_t*>(smem + C::POISON_OFFSET);
  constexpr int kSfWarp = 4, kCodeWarp = 8, kScaleWarp = 10, kMmaWarp = 11;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool copies = warp >= kCodeWarp && warp <= kScaleWarp;
  const bool early = p.early_kv != 0 && copies;

  if (tid == kCodeWarp * 32) {
    prefetch_tensormap(&p.kmap);
    if (!C::KVS) prefetch_tensormap(&p.vmap);
#pragma unroll 1
    for (int s = 0; s < RINGS; ++s) {
      // the codes' byte count (K = V: two warps') and every lane's scales
      mbar_init(&full[s], (C::KVS ? 2 : 1) + 32);
      mbar_init(&empty[s], C::KVS ? 2 : 1);  // the products that read the slot
    }
    mbar_init(sfk_ready, 4);
    mbar_init(sfv_ready, 4);
    mbar_init(dq_done, 1);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 4);
      mbar_init(&vt_full[s], 1);
      mbar_init(&vt_empty[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&p_empty[s], 1);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc<1>(tmem_at, kTmemCols);
  if (copies) {
    named_bar_sync(5, 3 * 32);
    named_bar_arrive(4, C::THREADS);
  }
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
  if (!early) grid_launch_dependents();

  float* red = reinterpret_cast<float*>(smem + C::RED_OFFSET);     // [4][CC]
  float* my_lse = reinterpret_cast<float*>(smem + C::LSE_OFFSET);  // [CC]
  float* coef = reinterpret_cast<float*>(smem + C::COEF_OFFSET);   // [CC]
  float* my_out = reinterpret_cast<float*>(smem);                  // [CC][D], over the ring
  uint32_t tmem = 0;
  if (!copies) {
    // the barriers and tensor memory are there (the copies do not wait for the other warps)
    named_bar_sync(4, C::THREADS);
    tmem_fence_after();
    tmem = *tmem_at;
  }
  const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // this warp's lanes of tensor memory

  if (copies) {
    bool waited = !early;
    uint32_t err_bits = 0;
    if (tiles > 0) {
      // ---- copies. Rows four tiles at a time: lane l the 16 tokens 16 l .. of
      // them, its page id fetched four tiles ahead (one tile ahead, its latency
      // bound the kernel: 4 x 32768 tokens 77 -> 62 us).
      const uint64_t policy = l2_evict_first_policy();
      const int mine = warp - kCodeWarp;  // 0: K's codes, 1: V's (K = V: the lower and the upper half), 2: scales
      const int fresh_from = L - p.query_tokens;  // rows from here on may still be written by the kernel in front
      auto page_of = [&](int i) {
        const int t = t_base + i * kFp4Tile + lane * 16;
        return t < thi ? __ldg(table + t / p.page_size) : -1;
      };
      int page = page_of(0), rows = -1;
      bool stop = false;
      int done = 0;  // tiles whose copies went out
#pragma unroll 1
      for (int i = 0; i < tiles && !stop; ++i) {
        if ((i & 3) == 0) {
          const int t = t_base + i * kFp4Tile + lane * 16;
          const bool here = (unsigned)page < (unsigned)p.num_pages;
          if (t < thi && !here) err_bits |= kErrBadPage;
          rows = t < thi && here ? (page * p.num_kv_heads + g) * p.page_size + t % p.page_size : -1;
          page = page_of(i + 4);
        }
        const int row0 = __shfl_sync(kFullMask, rows, (i & 3) * 8 + (lane & 7));
        const uint32_t bits = __ballot_sync(kFullMask, row0 >= 0) & 0xffu;
        if (!waited && (i >= C::NK || (!C::KVS && i >= C::NV) || t_base + (i + 1) * kFp4Tile > fresh_from)) {
          grid_dependency_wait();
          grid_launch_dependents();
          waited = true;
        }
#pragma unroll
        for (int v = 0; v < (C::KVS ? 1 : 2); ++v) {
          if (!C::KVS && mine != 2 && mine != v) continue;
          const int n = v ? C::NV : C::NK, st = (v ? C::NK : 0) + i % n, round = i / n;
          if (round > 0) {
            const bool freed = mbar_wait(&empty[st], (round - 1) & 1);
            if (__any_sync(kFullMask, !freed)) {
              err_bits |= kErrTimeout;
              stop = true;
              break;
            }
          }
          uint8_t* item = smem + st * C::ITEM_BYTES;
          if (mine < 2) {
            const uint32_t part = C::KVS ? (mine ? bits & 0xf0u : bits & 0x0fu) : bits;
            if (lane == 0) {
              if (!C::KVS || mine == 0) valid[st] = bits;
              if (part)
                mbar_arrive_expect_tx(&full[st], __popc(part) * (16 * C::D / 2) + (mine == 0 ? p.stall_bytes : 0));
              else
                mbar_arrive(&full[st]);
            }
            __syncwarp();
            if (lane < 8 && ((part >> lane) & 1u))
              tma_load_4d(item + lane * 16 * (C::D / 2), v ? &p.vmap : &p.kmap, 0, 0, 0, row0 / 8, &full[st], policy);
          } else {
            // 16 bytes a lane (as bulk copies these would be half of all copies)
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
          }
        }
        if (!stop) done = i + 1;
      }
      // no copy may still be landing when the shared memory is used for something else
      const unsigned long long deadline = global_timer_ns() + kWaitTimeoutNs;
      for (int s = lane; s < RINGS; s += 32) {
        const int n = s < C::NK ? C::NK : C::NV, at = s < C::NK ? s : s - C::NK;
        if (at >= done || (!C::KVS && mine != 2 && (s >= C::NK) != (mine == 1))) continue;
        const int last = at + n * ((done - 1 - at) / n);
        if (!mbar_wait_until(&full[s], (last / n) & 1, deadline)) err_bits |= kErrTimeout;
      }
    }
    if (!waited) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
    err_bits = __reduce_or_sync(kFullMask, err_bits);
    if (lane == 0 && err_bits) atomicOr(p.err, err_bits);
  } else if (tiles > 0) {
    bool good = true;
    if (warp < 8) {
      // the query's terms, the unit matrix and P's unused rows
      write_query_terms<C>(p, cm, smem, warp, lane);
      for (int i = tid; i < C::EYE_BYTES / 16; i += 256) {
        // 16 bytes of row m: dims 32 c ..; its one lies at dim m (e2m1 1.0 is 2)
        const int m = i >> 2, c = (i & 3) ^ ((m >> 1) & 3);
        const uint32_t one = (m >> 5) == c ? 2u << (4 * (m & 7)) : 0u;
        const int word = (m >> 3) & 3;
        *reinterpret_cast<uint4*>(smem + C::EYE_OFFSET + (m >> 3) * 512 + (m & 7) * 64 + (i & 3) * 16) =
            make_uint4(word == 0 ? one : 0u, word == 1 ? one : 0u, word == 2 ? one : 0u, word == 3 ? one : 0u);
      }
      for (int i = tid; i < 2 * C::P_BYTES / 16; i += 256) {
        const int row = ((i >> 6) & 1) * 8 + ((i >> 3) & 7);  // [slab][2 groups][8 rows][128 B]
        if (row >= C::CC) *reinterpret_cast<uint4*>(smem + C::P_OFFSET + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (tid < C::CC) poison[tid] = 0u;
      if (tid == 0) *failed_at = 0u;
      fence_proxy_async_smem();
    }
    named_bar_sync(1, 9 * 32);  // warps 0-7 and the products'

    if (warp < kSfWarp) {
      // ---- softmax: rows 32 warp .. + 31 of every tile
      float col_mul[C::CC], ref[C::CC], sum[C::CC];
      int col_hi[C::CC], col_lo[C::CC];
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        col_mul[c] = reinterpret_cast<const float*>(smem + C::COL_OFFSET)[c];
        col_hi[c] = cm.valid(c) ? min(thi, L - cm.T + cm.token(c) + 1) : 0;
        col_lo[c] = max(tlo, (p.window > 0 && cm.valid(c)) ? L - cm.T + cm.token(c) + 1 - p.window : 0);
        ref[c] = -INFINITY;
        sum[c] = 0.f;
      }
      const uint32_t p_at = smem_u32(smem + C::P_OFFSET) + warp * 2048 + (lane & 3) * 4;
      // whether a tile's 16-token blocks have a page: lane l block l of four tiles, as the copies take them
      auto page_of = [&](int i) {
        const int t = t_base + i * kFp4Tile + lane * 16;
        return t < thi ? __ldg(table + t / p.page_size) : -1;
      };
      int page = page_of(0);
      uint32_t blocks = 0;
      // The four warps leave together: one whose wait ran out says so at the next
      // tile's barrier.
      auto give_up = [&]() {
        good = false;
        if (lane == 0) *failed_at = 1u;
        __syncwarp();
      };
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int sbuf = i % SB, buf = i & 1;
        if ((i & 3) == 0) {
          blocks = __ballot_sync(kFullMask, (unsigned)page < (unsigned)p.num_pages);
          page = page_of(i + 4);
        }
        if (good) {
          const bool scored = mbar_wait(&s_full[sbuf], (i / SB) & 1);
          if (__any_sync(kFullMask, !scored)) give_up();
        }
        tmem_fence_after();
        float s[C::CC];
        {
          uint32_t w[kFp4Terms * C::CC / 8][8];
#pragma unroll
          for (int k = 0; k < kFp4Terms * C::CC / 8; ++k) tmem_ld(w[k], tmem + kTmemS + sbuf * C::N + quarter + k * 8);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            float x = 0.f;
#pragma unroll
            for (int t = kFp4Terms - 1; t >= 0; --t) x += __uint_as_float(w[(t * C::CC + c) / 8][(t * C::CC + c) % 8]);
            s[c] = x * col_mul[c];
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[sbuf]);
        const int row = warp * 32 + lane, t = t_base + i * kFp4Tile + row;
        const bool ok = (blocks >> ((i & 3) * 8 + (row >> 4))) & 1u;
        bool above = !good;
#pragma unroll
        for (int c = 0; c < C::CC; ++c) {
          if (!(ok && t >= col_lo[c] && t < col_hi[c])) s[c] = -INFINITY;
          above = above || s[c] > ref[c] + kRefRange;
        }
        if (named_bar_or(2, 128, above)) {
          if (*failed_at) {
            good = false;
            break;
          }
          // new references: the tile's maximum, where that is out of reach
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            const int top = __reduce_max_sync(kFullMask, ordered(isnan(s[c]) ? -INFINITY : s[c]));
            if (lane == 0) red[warp * C::CC + c] = unordered(top);
          }
          named_bar_sync(2, 128);
          float f[C::CC];
          bool held = false;
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            const float top = fmaxf(fmaxf(red[c], red[C::CC + c]), fmaxf(red[2 * C::CC + c], red[3 * C::CC + c]));
            const bool up = top > ref[c] + kRefRange;
            f[c] = up && ref[c] != -INFINITY ? ex2(ref[c] - top) : 1.f;
            held = held || f[c] != 1.f;
            sum[c] *= f[c];
            if (up) ref[c] = top;
          }
          named_bar_sync(2, 128);  // red may be written again
          if (held) {
            // sums that hold something: rescaled once the tiles before are in them
            const bool summed = mbar_wait(&p_empty[(i - 1) & 1], ((i - 1) >> 1) & 1);
            if (__any_sync(kFullMask, !summed)) give_up();
            tmem_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < CH; ++c0) {
              uint32_t o[8];
              tmem_ld(o, tmem + kTmemO + c0 * 16 + quarter);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < C::CC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
              tmem_st(tmem + kTmemO + c0 * 16 + quarter, o);
            }
            tmem_wait_st();
            tmem_fence_before();
          }
        }
        if (i >= 2) {
          const bool freed = mbar_wait(&p_empty[buf], ((i >> 1) - 1) & 1);
          if (__any_sync(kFullMask, !freed)) give_up();
        }
#pragma unroll
        for (int c = 0; c < C::CC; ++c) {
          // rounded to tf32 here, to nearest (the product would cut it off); the sum takes what the product takes
          uint32_t w;
          const float e = ex2(s[c] - (ref[c] == -INFINITY ? 0.f : ref[c]));
          asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(w) : "f"(e));
          sum[c] += __uint_as_float(w);
          const uint32_t at = p_at + buf * C::P_BYTES + (c >> 3) * 1024 + (c & 7) * 128 + (((lane >> 2) ^ (c & 7)) << 4);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      if (!good && lane == 0) atomicOr(p.err, kErrTimeout);
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        float l = sum[c];
#pragma unroll
        for (int m = 16; m; m >>= 1) l += __shfl_xor_sync(kFullMask, l, m);
        if (lane == 0) red[warp * C::CC + c] = l;
        if (tid == 0) my_lse[c] = ref[c];
      }
    } else if (warp < kCodeWarp) {
      // ---- scales into tensor memory: lane l, column 4 k + j holds the 4 scales of row l + 32 j, dims 64 k ..;
      // every quarter of the lanes all rows'
      {
        uint32_t one[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) one[k] = 0x38383838u;  // e4m3 1.0
        tmem_st(tmem + kTmemSfi + quarter, one);
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
          tmem_st(tmem + kTmemSfq + quarter + k0 * 4, r8);
        }
      }
      auto put = [&](const uint8_t* sf, uint32_t at, bool v, uint32_t here, int t0) {
        uint32_t x[C::KSTEPS * 4];  // [64 dims][row group]
#pragma unroll
        for (int k0 = 0; k0 < C::KSTEPS; k0 += 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(sf + (lane + 32 * j) * C::ROW_SF + k0 * 4);
            x[k0 * 4 + j] = w.x;
            x[k0 * 4 + 4 + j] = w.y;
            x[k0 * 4 + 8 + j] = w.z;
            x[k0 * 4 + 12 + j] = w.w;
          }
        }
        if (v) {
          // V's rows that do not count have scale 0: their probabilities are 0, but 0 * NaN is NaN
          if (!(here == 0xffu && t0 >= tlo && t0 + kFp4Tile <= thi)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = lane + 32 * j, t = t0 + row;
              if (((here >> (row >> 4)) & 1u) && t >= tlo && t < thi) continue;
#pragma unroll
              for (int k = 0; k < C::KSTEPS; ++k) x[k * 4 + j] = 0u;
            }
          }
          // A NaN block would spread over the unit matrix's zeros to other dims
          // (and, of a token that only some of several query tokens attend, to the
          // others): it is taken out and marked for the results it belongs to.
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < C::KSTEPS * 4; ++k) bad |= nan_scales(x[k]);
          if (__any_sync(kFullMask, bad != 0u)) {
#pragma unroll
            for (int k = 0; k < C::KSTEPS * 4; ++k) {
              const uint32_t nan = nan_scales(x[k]);
              if (!nan) continue;
              x[k] &= ~((nan >> 7) * 0xffu);
              if (warp != kSfWarp) continue;
              const int t = t0 + lane + 32 * (k & 3);
              for (int c = 0; c < C::CC && cm.valid(c); ++c) {
                const int end = L - cm.T + cm.token(c) + 1;
                if (t >= end || (p.window > 0 && t < end - p.window)) continue;
                for (int y = 0; y < 4; ++y)
                  if ((nan >> (8 * y + 7)) & 1u) atomicOr(&poison[c], 1u << ((k >> 2) * 4 + y));
              }
            }
          }
        }
#pragma unroll
        for (int k0 = 0; k0 < C::KSTEPS; k0 += 4) {
          uint32_t r16[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) r16[q] = x[k0 * 4 + q];
          tmem_st(at + k0 * 4, r16);
        }
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
      };
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        // K's, once the product before has read the last tile's
        const int st = i % C::NK;
        bool ready = mbar_wait(&full[st], (i / C::NK) & 1);
        if (ready && i > 0) ready = mbar_wait(&s_full[(i - 1) % SB], ((i - 1) / SB) & 1);
        if (__any_sync(kFullMask, !ready)) {
          good = false;
          break;
        }
        tmem_fence_after();
        put(smem + st * C::ITEM_BYTES + C::CODE_BYTES, tmem + kTmemSfk + quarter, false, 0u, 0);
        if (lane == 0) mbar_arrive(sfk_ready);
        // V's likewise
        const int n = C::KVS ? C::NK : C::NV, sv = (C::KVS ? 0 : C::NK) + i % n;
        ready = C::KVS || mbar_wait(&full[sv], (i / n) & 1);
        if (ready && i > 0) ready = mbar_wait(dq_done, (i - 1) & 1);
        if (__any_sync(kFullMask, !ready)) {
          good = false;
          break;
        }
        tmem_fence_after();
        const uint32_t here = valid[sv];
        const int t0 = t_base + i * kFp4Tile;
        put(smem + sv * C::ITEM_BYTES + C::CODE_BYTES, tmem + kTmemSfv + quarter, true, here, t0);
        if (lane == 0) mbar_arrive(sfv_ready);
      }
      if (!good && lane == 0) atomicOr(p.err, kErrTimeout);
    } else {
      // ---- the products, by one warp in an order that keeps the tensor core busy
      // (issued by three warps, a product each, they got in one another's way:
      // a tf32 instruction took 62 cycles instead of 14). Chunks of 128 dims go
      // in pairs, V^T of both and then both sums, so that one waits for its
      // operand while the other runs; the next tile's scores go out between
      // them, as soon as they can.
      constexpr uint32_t kQk = (1u << 7) | (1u << 10) | ((uint32_t)(C::N / 8) << 17) | (8u << 24);  // e2m1, e4m3 scales
      constexpr uint32_t kDq = (1u << 7) | (1u << 10) | ((uint32_t)(kFp4Tile / 8) << 17) | (8u << 24);
      constexpr uint32_t kPv = (1u << 4) | (2u << 7) | (2u << 10) | (2u << 17) | (8u << 24);  // tf32 -> fp32, 128 x 16
      if (elect_one()) {
        // descriptors' bases; a step further is a constant added to the address field
        const uint64_t ring_desc = smem_desc(smem_u32(smem), 0, C::SL * 1024);
        const uint64_t q_desc = smem_desc(smem_u32(smem + C::Q_OFFSET), 0, C::SL * 1024);
        const uint64_t eye_desc = smem_desc(smem_u32(smem + C::EYE_OFFSET), 0, 512, 64);
        const uint64_t p_desc = smem_desc(smem_u32(smem + C::P_OFFSET), 0, 1024);
        constexpr int kItem = C::ITEM_BYTES >> 4;
        int scores = 0, widened = 0, summed = 0;  // tiles, chunks, chunks issued so far
        auto qk = [&](int i) {
          tmem_fence_after();
          const int st = i % C::NK, sbuf = i % SB;
          const uint64_t a = ring_desc + st * kItem;
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k)
            mma_fp4(tmem + kTmemS + sbuf * C::N, a + (k >> 2) * 64 + (k & 3) * 2, q_desc + (k >> 2) * 64 + (k & 3) * 2, kQk,
                    tmem + kTmemSfk + k * 4, tmem + kTmemSfq + k * 4, k > 0);
          mma_commit<1>(&s_full[sbuf]);
          mma_commit<1>(&empty[st]);
          scores = i + 1;
        };
        auto may_qk = [&](int i) {  // without waiting
          return mbar_test(&full[i % C::NK], (i / C::NK) & 1) && mbar_test(sfk_ready, i & 1) &&
                 (i < SB || mbar_test(&s_empty[i % SB], (i / SB - 1) & 1));
        };
#pragma unroll 1
        for (int i = 0; i < tiles && good; ++i) {
          if (scores == i) {
            good = mbar_wait(&full[i % C::NK], (i / C::NK) & 1) && mbar_wait(sfk_ready, i & 1) &&
                   (i < SB || mbar_wait(&s_empty[i % SB], (i / SB - 1) & 1));
            if (!good) break;
            qk(i);
          }
          const int n = C::KVS ? C::NK : C::NV, st = (C::KVS ? 0 : C::NK) + i % n;
          good = mbar_wait(&full[st], (i / n) & 1) && mbar_wait(sfv_ready, i & 1);
          const uint64_t v = ring_desc + st * kItem;
          const uint64_t pd = p_desc + (i & 1) * (C::P_BYTES >> 4);
#pragma unroll 1
          for (int c0 = 0; c0 < CH && good; c0 += 2) {
            const int at = i * CH + c0;  // (even)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (good && at > 0) good = mbar_wait(&vt_empty[c], ((at >> 1) - 1) & 1);
              if (!good) break;
              tmem_fence_after();
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_fp4(tmem + kTmemVt + c * 128, eye_desc + j * 2, v + (c0 >> 1) * 64 + c * 4 + j * 2, kDq, tmem + kTmemSfi,
                        tmem + kTmemSfv + c0 * 8 + (c * 2 + j) * 4, j > 0);
              mma_commit<1>(&vt_full[c]);
              widened = at + c + 1;
            }
            if (!good) break;
            if (c0 + 2 == CH) {
              mma_commit<1>(&empty[st]);
              mma_commit<1>(dq_done);
            }
            if (i + 1 < tiles && scores == i + 1 && may_qk(i + 1)) qk(i + 1);
            if (c0 == 0) good = mbar_wait(&p_full[i & 1], (i >> 1) & 1);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (good) good = mbar_wait(&vt_full[c], (at >> 1) & 1);
              if (!good) break;
              tmem_fence_after();
#pragma unroll
              for (int q = 0; q < kFp4Tile / 8; ++q)
                mma_tf32(tmem + kTmemO + c0 * 16 + c * 16, tmem + kTmemVt + c * 128 + q * 8, pd + (q >> 2) * 128 + (q & 3) * 2,
                         kPv, i > 0 || q > 0);
              mma_commit<1>(&vt_empty[c]);
              summed = at + c + 1;
            }
            if (good && c0 + 2 == CH) mma_commit<1>(&p_empty[i & 1]);
            if (good && i + 1 < tiles && scores == i + 1 && may_qk(i + 1)) qk(i + 1);
          }
        }
        // what was issued ends before its operands and results are used for something else
        if (!good) {
          if (scores > 0) mbar_wait(&s_full[(scores - 1) % SB], ((scores - 1) / SB) & 1);
          if (widened > 0) mbar_wait(&vt_full[(widened - 1) & 1], ((widened - 1) >> 1) & 1);
          atomicOr(p.err, kErrTimeout);
        }
        if (summed > 0) mbar_wait(&vt_empty[(summed - 1) & 1], ((summed - 1) >> 1) & 1);
      }
      __syncwarp();
    }
  }
  __syncthreads();

  // ---- the piece's result
  if (tid < C::CC) {
    const float s = tiles > 0 ? (red[tid] + red[C::CC + tid]) + (red[2 * C::CC + tid] + red[3 * C::CC + tid]) : 0.f;
    coef[tid] = s != 0.f ? p.v_mul / s : 0.f;
    my_lse[tid] = s != 0.f ? (my_lse[tid] + __log2f(s)) * 0.69314718055994530942f : -INFINITY;
  }
  __syncthreads();
  // warps 0-7: lane l of quarter w has dim 32 w + l of a chunk; warps 0-3 the even chunks, 4-7 the odd ones
  if (warp < 8) {
    tmem_fence_after();
#pragma unroll 1
    for (int c0 = warp >> 2; c0 < CH; c0 += 2) {
      uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      if (tiles > 0) {
        tmem_ld(o, tmem + kTmemO + c0 * 16 + quarter);
        tmem_wait_ld();
      }
      const int dim = c0 * 128 + (warp & 3) * 32 + lane;
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        if (!cm.valid(c)) break;
        // (no attended token: coefficient 0, and sums that nothing has written)
        float x = coef[c] != 0.f ? __uint_as_float(o[c]) * coef[c] : 0.f;
        if (tiles > 0 && ((poison[c] >> (dim >> 4)) & 1u)) x = NAN;
        if (p.direct_out)
          reinterpret_cast<__nv_bfloat16*>(p.out)[cm.row(c) * C::D + dim] = __float2bfloat16_rn(x);
        else if (p.cluster_merge)
          my_out[c * C::D + dim] = x;
        else
          p.o_part[(cm.row(c) * p.num_splits + split) * C::D + dim] = x;
      }
    }
    tmem_fence_before();
  }
  if (!p.direct_out && !p.cluster_merge && tid < C::CC && cm.valid(tid))
    p.lse_part[cm.row(tid) * p.num_splits + split] = my_lse[tid];
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    tmem_dealloc<1>(*tmem_at, kTmemCols);
  }
  if (!p.cluster_merge) return;

  // ---- the pieces' results joined over distributed shared memory: each CTA of
  // the cluster a share of the elements, in piece order
  //   out = sum_s w_s o_s,  w_s = exp(lse_s - M) / sum_s' exp(lse_s' - M)
  cluster_sync_all();
  const int S = p.num_splits, rank = (int)cluster_ctarank();
  constexpr int D4 = C::D / 4;
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
