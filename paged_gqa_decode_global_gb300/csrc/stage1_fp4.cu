// Decode attention over a paged 4-bit cache (sm_103a), pieces joined in the same
// launch. A unit of work is a (request, KV head, tile of up to CC query rows,
// "columns"); its tokens come in tiles of 128. One CTA an SM takes an equal share
// of all units' tiles, in order, so that a share may end in the middle of a unit:
// what it holds of one then is a piece, and the last CTA to leave its piece of a
// unit joins them, in the pieces' order. Within a share every role runs on from
// unit to unit without a gap (a CTA's start takes ~4 us; with a CTA a piece, 61
// windows of 1024 tokens took 3.2 waves of them).
//
// Bound and measured (time of a launch in a CUDA graph; floor at the measured copy
// rate): HBM where K and V differ at d 512 (4 x 32768 tokens 54 us, floor 45: a tile
// takes its copies' 3170 cycles, start and end ~8 us); at K = V the chain of V^T's two
// buffers (8 requests of 1K to 128K 65 us, floor 36: ~2600 cycles a tile, its copies
// 1590); at d 256 the softmax warps (61 windows of 1024 38 us, floor 21); latency for
// short lengths (8 x 1024 13.5 us; 10.6 with a CTA a piece, which took 158 us for the
// 8 requests of 1K to 128K when this one took 99).
//
// Mathematics: a cached element is e2m1(code) * e4m3(scale of its 16 dims) *
// 2^exp. All three products of a tile of 128 tokens run on tcgen05, and no
// cached element passes through the CUDA cores:
//   S = K q^T    kind::mxf4nvf4 on codes and scales as they lie in the cache. The
//                query row is written as kFp4Terms e2m1 terms, each with its own
//                scale per 16 dims, the next taking what the one before left
//                over 4 times up; the terms' scores are summed afterwards, each
//                brought down again. A term leaves at most max(0.177 m + 2^-10,
//                6 * 2^-10) of a block whose largest is m (the second parts are
//                half of e4m3's smallest step). With the row's largest in
//                [2^10, 2^11) (by a power of two) and the last term 4^5 up, six
//                leave 2^-14.9 of the block's largest and 2^-27.4 of the row's (all
//                terms at one size left 2^-17.4 of it, for the same time: 61 windows
//                of 1024 37.6 us and 37.5; 4 and 8 times up in turn 38.3);
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
// Roles: warps 0-3 softmax (a lane a token); 4-7 put a tile's scales in tcgen05.cp's
// order; 8-11 write the next unit's query terms, read a unit's sums and join pieces;
// then two that copy codes (TMA), one or two that copy scales (cp.async), and warps of
// which one lane issues the scores, V^T (one or two) and the sums (as many): a look at
// a barrier takes 60 to 150 cycles, and one lane that does all this spends most of
// them looking. (Warps 5 to a quarter of the SM at most, for 96 registers a thread.)
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
// Tensor memory columns: scores [N], scales of V, of the unit matrix, V^T [2][128], sums [CHUNKS][16],
// scales of K, of the query. All of it is allocated, so it begins at column 0.
constexpr uint32_t kTmemS = 0, kTmemSfv = 64, kTmemSfi = 96, kTmemVt = 128, kTmemO = 384, kTmemSfk = 448,
                   kTmemSfq = 480, kTmemCols = 512;

// Descriptors of shared-memory operands as two words, of which only the lower,
// with the address, varies. (row_bytes 0: not swizzled, rows of 16 bytes.)
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, int row_bytes = 128) {
  return (sbo >> 4) | 1u << 14 | (row_bytes ? (uint32_t)swizzle_code(row_bytes) << 29 : 0u);
}

// D[tmem] (+)= A . B over 64 dims, both e2m1 with an e4m3 scale per 16 dims.
template <uint32_t A_HI, uint32_t B_HI, uint32_t IDESC>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t sfa, uint32_t sfb, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %8, [%3], [%4], p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate), "n"(A_HI), "n"(B_HI), "n"(IDESC)
      : "memory");
}

// Scales of 128 rows and 64 dims (512 bytes: row l + 32 j's four at 16 l + 4 j) to
// 4 columns of tensor memory, in every quarter of its lanes. Products issued by the
// same thread afterwards see them.
__device__ __forceinline__ void copy_scales(uint32_t to, uint32_t from) {
  asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\ttcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(to),
               "r"(from), "n"(desc_hi(128, 0))
               : "memory");
}

// D[tmem] (+)= A[tmem] . B over 8 tokens, tf32.
template <uint32_t B_HI, uint32_t IDESC>
__device__ __forceinline__ void mma_tf32(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], b, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"((uint32_t)accumulate), "n"(B_HI), "n"(IDESC)
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

// How far up what a term leaves over is taken for the next one: it never passes what
// the row's largest was (0.177 * 4 of it), so no scale is clamped.
constexpr float kTermStep = 4.f;

// Four e4m3 scales: 0x80 in the bytes that are NaN.
__device__ __forceinline__ uint32_t nan_scales(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// A wait of up to kWaitTimeoutNs. The hardware suspends the thread for up to the
// time asked for, so that a long wait takes no issue slots. One copy for all.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
  unsigned long long start = 0;
#pragma unroll 1
  for (int n = 0;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    if (done) return true;
    const unsigned long long now = global_timer_ns();
    if (n == 0) start = now;
    if (now - start > kWaitTimeoutNs) return false;
  }
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t phase) {
  return __builtin_expect(mbar_test(bar, phase & 1), 1) || wait_long(smem_u32(bar), phase & 1);
}

// What a ring slot's word says of its tile, beside the 16-token blocks that have a page (bits 0-7).
constexpr uint32_t kTileFirst = 0x100u, kTileLast = 0x200u, kTileOdd = 0x400u;  // of its segment; an odd one

// A request's attended range, cut to what its block table holds.
struct Span {
  int L, base, tiles;  // cached tokens; the first one attended, rounded down to 16; tiles from there (at least one)
  bool bad;
  __device__ __forceinline__ Span(const Fp4Params& p, int raw) {
    bad = raw < (p.query_tokens > 1 ? p.query_tokens : 0) || raw > p.cap;
    L = max(0, min(raw, p.cap));
    const int first_hi = L - p.query_tokens + 1;
    base = p.window > 0 && first_hi > p.window ? (first_hi - p.window) & ~15 : 0;
    tiles = max(1, (L - base + kFp4Tile - 1) / kFp4Tile);
  }
};

// The tiles of a share that belong to one unit. Its column c is the c-th
// (token, head) pair from (token, head) on, token-major.
struct alignas(16) Segment {
  int b, g, L, tiles;
  int t_base;    // first token of the first tile
  int tlo, thi;  // tokens of it that some column attends
  int token, head;
  int pieces, piece, first_share;  // of the unit
  int bad;
};
// The (token, head) pair of a column, from one to the next.
struct Pair {
  int j, r;
  __device__ __forceinline__ explicit Pair(const Segment& s) : j(s.token), r(s.head) {}
  __device__ __forceinline__ void next(const Fp4Params& p) {
    if (++r == p.group) {
      r = 0;
      ++j;
    }
  }
  __device__ __forceinline__ bool valid(const Fp4Params& p) const { return j < p.query_tokens; }
  // one past the last position it attends
  __device__ __forceinline__ int end(const Fp4Params& p, const Segment& s) const { return s.L - p.query_tokens + j + 1; }
  __device__ __forceinline__ size_t row(const Fp4Params& p, const Segment& s) const {
    return ((size_t)s.b * p.query_tokens + j) * p.num_q_heads + (size_t)s.g * p.group + r;
  }
};

// One warp's walk over the CTA's share; all lanes take part.
struct Walk {
  int lens, chunk;      // this lane's request's length, of 32
  int b, y, k;          // where the next segment begins
  int unit;             // tiles before unit (b, y) (all of them are fewer than 2^30)
  int left;             // tiles of the share not yet handed out
  int each;             // tiles of a share
  int first_share;      // the share that unit (b, y) begins in
};
__device__ __forceinline__ void walk_load(const Fp4Params& p, Walk& w, int c) {
  if (c == w.chunk) return;
  w.chunk = c;
  const int at = c * 32 + (threadIdx.x & 31);
  w.lens = at < p.batch ? p.seq_lens[at] : 0;
}
__device__ __forceinline__ int walk_count(const Fp4Params& p, const Walk& w) {
  return w.chunk * 32 + (int)(threadIdx.x & 31) < p.batch ? Span(p, w.lens).tiles : 0;
}
__device__ __forceinline__ void walk_start(const Fp4Params& p, Walk& w) {
  const int lane = threadIdx.x & 31, chunks = (p.batch + 31) / 32;
  w.chunk = -1;
  w.b = w.y = w.k = w.unit = w.left = w.first_share = 0;
  int total = 0;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    walk_load(p, w, c);
    total += (int)__reduce_add_sync(kFullMask, walk_count(p, w)) * p.units;
  }
  w.each = (total + gridDim.x - 1) / gridDim.x;
  const int start = blockIdx.x * w.each;  // (below 2^30 + 2^30)
  if (start >= total) return;
  w.left = min(w.each, total - start);
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    walk_load(p, w, c);
    const int n = walk_count(p, w);
    int upto = n;  // tiles of the requests up to this lane's
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(kFullMask, upto, m);
      if (lane >= m) upto += o;
    }
    const uint32_t past = __ballot_sync(kFullMask, w.unit + upto * p.units > start);
    if (past == 0) {
      w.unit += __shfl_sync(kFullMask, upto, 31) * p.units;
      continue;
    }
    const int at = __ffs(past) - 1, tiles = __shfl_sync(kFullMask, n, at);
    w.unit += (__shfl_sync(kFullMask, upto, at) - tiles) * p.units;
    w.b = c * 32 + at;
    w.y = (start - w.unit) / tiles;
    w.unit += w.y * tiles;
    w.k = start - w.unit;
    break;
  }
  w.first_share = w.k ? w.unit / w.each : blockIdx.x;
}
template <int CC>
__device__ __forceinline__ bool walk_next(const Fp4Params& p, Walk& w, Segment& s) {
  if (w.left == 0) return false;
  walk_load(p, w, w.b >> 5);
  const Span sp(p, __shfl_sync(kFullMask, w.lens, w.b & 31));
  s.b = w.b;
  s.g = w.y;
  s.token = s.head = 0;
  int last = p.query_tokens - 1;  // token of the last column
  if (p.col_tiles > 1) {
    s.g = w.y / p.col_tiles;
    const int c0 = (w.y - s.g * p.col_tiles) * CC;
    s.token = c0 / p.group;
    s.head = c0 - s.token * p.group;
    last = min(last, s.token + (s.head + CC - 1) / p.group);
  }
  s.L = sp.L;
  s.bad = sp.bad;
  s.tiles = min(sp.tiles - w.k, w.left);
  s.t_base = sp.base + w.k * kFp4Tile;
  // the union of the columns' tokens' causal ranges
  const int end0 = sp.L - p.query_tokens + 1;
  s.tlo = max(s.t_base, p.window > 0 ? end0 + s.token - p.window : 0);
  s.thi = min(end0 + last, s.t_base + s.tiles * kFp4Tile);
  const bool whole = w.k + s.tiles == sp.tiles;  // the unit ends in this share
  s.first_share = w.first_share;
  s.piece = (int)blockIdx.x - w.first_share;
  s.pieces = s.piece + 1;
  if (!whole) s.pieces = (w.unit + sp.tiles - 1) / w.each - w.first_share + 1;
  w.left -= s.tiles;
  w.k += s.tiles;
  if (whole) {
    w.k = 0;
    w.unit += sp.tiles;
    w.first_share = blockIdx.x;
    if (++w.y == p.units) {
      w.y = 0;
      ++w.b;
    }
  }
  return true;
}

// Byte of (row, byte of the row) in a swizzled tile of codes.
template <class C>
__device__ __forceinline__ uint32_t code_offset(int row, int byte) {
  const int sl = byte >> 7, c = (byte >> 4) & 7;
  return (row >> 3) * (C::SL * 1024) + sl * 1024 + (row & 7) * 128 + ((c ^ (row & 7)) << 4) + (byte & 15);
}

// The query rows of a segment's columns as terms in shared memory (`q`) and their
// scales (`sf`, `mul`), by `warps` warps: one takes 256 dims of a row, a lane 8 of them,
// two lanes a block of 16.
template <class C>
__device__ __forceinline__ void write_query_terms(const Fp4Params& p, const Segment& s, uint8_t* q, uint8_t* sf, float* mul,
                                                  int warp, int warps, int lane) {
#pragma unroll 1
  for (int item = warp; item < C::CC * C::SL; item += warps) {
    const int col = item / C::SL, part = item % C::SL;
    const int pair = s.head + col;
    int j = 0, r = pair;
    if (pair >= p.group) {
      j = pair / p.group;
      r = pair - j * p.group;
    }
    j += s.token;
    uint4 w = make_uint4(0u, 0u, 0u, 0u), o = w;
    if (j < p.query_tokens) {
      const uint4* row = reinterpret_cast<const uint4*>(
          p.q + (((size_t)s.b * p.query_tokens + j) * p.num_q_heads + (size_t)s.g * p.group + r) * C::D) + lane;
      w = __ldg(row + part * 32);
      if (C::SL == 2) o = __ldg(row + (part ^ 1) * 32);  // (for the row's largest)
    }
    // the row's largest magnitude, as whole numbers (infinity and NaN are the largest)
    uint32_t m = 0;
#pragma unroll
    for (uint32_t v : {w.x, w.y, w.z, w.w, o.x, o.y, o.z, o.w}) m = __vmaxu2(m, v & 0x7fff7fffu);
    const uint32_t top = __reduce_max_sync(kFullMask, max(m << 16, m & 0xffff0000u));
    const bool odd = top >= 0x7f800000u;  // a NaN or an infinity: the row's scores are NaN
    // brings the largest to [2^10, 2^11) (a row that is below 2^-116 altogether: as near as a factor of 2^126 does)
    const int shift = min(126, 137 - (int)(top >> 23));
    const float up = __int_as_float((127 + shift) << 23);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = odd ? 0.f : __uint_as_float(v[i] << 16) * up;
      x[2 * i + 1] = odd ? 0.f : __uint_as_float(v[i] & 0xffff0000u) * up;
    }
    if (part == 0 && lane == 0) mul[col] = p.scale_log2 * __int_as_float((127 - shift) << 23);
#pragma unroll 1
    for (int t = 0; t < kFp4Terms; ++t) {
      float a = fmaxf(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))),
                      fmaxf(fmaxf(fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7]))));
      a = fmaxf(a, __shfl_xor_sync(kFullMask, a, 1));
      uint16_t s8;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(a * (1.f / 6.f)));
      uint32_t s16;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"(s8));
      const float sc = __half2float(__ushort_as_half((unsigned short)(s16 & 0xffffu)));
      float rc;  // (what a term leaves over, the next one takes: its rounding need not be exact)
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc) : "f"(sc));
      rc = sc > 0.f ? rc : 0.f;
      uint32_t codes;
      asm("{\n\t.reg .b8 a, b, c, d;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
          "mov.b32 %0, {a, b, c, d};\n\t}"
          : "=r"(codes)
          : "f"(x[0] * rc), "f"(x[1] * rc), "f"(x[2] * rc), "f"(x[3] * rc), "f"(x[4] * rc), "f"(x[5] * rc),
            "f"(x[6] * rc), "f"(x[7] * rc));
      uint32_t f[4];
      e2m1x8_to_f16x8(codes, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        x[2 * i] = fmaf(-two.x, sc * kTermStep, x[2 * i] * kTermStep);
        x[2 * i + 1] = fmaf(-two.y, sc * kTermStep, x[2 * i + 1] * kTermStep);
      }
      const int n = t * C::CC + col;
      *reinterpret_cast<uint32_t*>(q + code_offset<C>(n, part * 128 + lane * 4)) = codes;
      if ((lane & 1) == 0) sf[n * C::ROW_SF + part * 16 + lane / 2] = odd ? (uint8_t)0x7f : (uint8_t)s8;
    }
  }
}

// 16 bytes global -> shared, counted by cp_async_arrive. (With an L2 cache policy the
// instruction is illegal here.)
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// An arrival on `bar` (one that its count holds) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The kernel's loops are kept short: its roles run different code side by side, and
// what does not fit the instruction caches is fetched again every tile (unrolled,
// 350 KB of code, it took three times as long).
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) decode_fp4_kernel(const __grid_constant__ Fp4Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int CH = C::CHUNKS, RINGS = C::NK + C::NV;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFFSET);  // [RINGS]: K's ring, then V's
  uint64_t* empty = full + RINGS;                                      // [RINGS]
  // four arrivals, one a warp: the slot's scales are where tcgen05.cp takes them from
  uint64_t* ready = empty + RINGS;      // [RINGS]
  // one arrival: the products' commits
  uint64_t* vt_empty = ready + RINGS;   // [2] a chunk of V^T used
  uint64_t* qk_done = vt_empty + 2;     // a segment's scores all computed
  // those of every lane that issues the sums
  uint64_t* p_empty = qk_done + 1;      // [2] P used: the tile is in the sums
  // two: a commit, and an arrival of the same lane (which orders what it has seen of others)
  uint64_t* vt_full = p_empty + 2;      // [2] a chunk of V^T there
  uint64_t* s_full = vt_full + 2;       // scores computed
  // both of every such lane
  uint64_t* o_full = s_full + 1;        // a segment's sums complete
  // four warps
  uint64_t* s_empty = o_full + 1;       // scores read
  uint64_t* p_full = s_empty + 1;       // [2]
  uint64_t* q_full = p_full + 2;        // [2] a segment's query terms there
  uint64_t* o_empty = q_full + 2;       // a segment's sums read
  uint64_t* l_full = o_empty + 1;       // [2] a segment's probabilities' sums there
  uint64_t* l_empty = l_full + 2;       // [2] and read
  // one
  uint64_t* seg_full = l_empty + 2;     // [SEGS] a segment told
  static_assert(C::NUM_BARS == 3 * RINGS + 5 + 4 + 10 + C::SEGS, "as listed");
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(full + C::NUM_BARS);
  volatile uint32_t* valid = reinterpret_cast<uint32_t*>(smem + C::VALID_OFFSET);  // [RINGS]
  volatile uint32_t* tile_of = reinterpret_cast<uint32_t*>(smem + C::TILE_OFFSET);      // [2] first, last: by P buffer
  volatile uint32_t* blocks_of = reinterpret_cast<uint32_t*>(smem + C::BLOCKS_OFFSET);  // of the scores' tile
  constexpr int SW = C::SCALE_WARPS;
  constexpr int kSfWarp = 4, kEndWarp = 8, kCodeWarp = 12, kScaleWarp = 14, kScoreWarp = kScaleWarp + C::SCALE_WARPS,
                kWideWarp = kScoreWarp + 1, kSumWarp = kWideWarp + C::LANES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool copies = warp >= kCodeWarp && warp < kScoreWarp;
  const bool early = p.early_kv != 0 && copies;
  uint32_t* poison_of = reinterpret_cast<uint32_t*>(smem + C::POISON_OFFSET);  // [SEGS][CC], by segment

  if (warp == kCodeWarp) {
    if (lane == 0) {
      prefetch_tensormap(&p.kmap);
      if (!C::KVS) prefetch_tensormap(&p.vmap);
    }
    for (int i = lane; i < C::NUM_BARS; i += 32) {
      const int r = i - 3 * RINGS;
      // full: the codes' byte count (K = V: two warps') and every lane's scales; empty: the products that read the slot
      mbar_init(&full[i], i < RINGS       ? (C::KVS ? 2 + 32 * SW : 33)
                          : i < 2 * RINGS ? (C::KVS ? 1 + C::LANES : i - RINGS < C::NK ? 1 : C::LANES)
                          : r < 0         ? 4
                          : r < 3         ? 1
                          : r < 5         ? C::LANES
                          : r < 8         ? 2
                          : r < 9         ? 2 * C::LANES
                          : r < 19        ? 4
                                          : 1);
    }
    fence_barrier_init();
    __syncwarp();
  }
  if (warp == kScoreWarp) tmem_alloc<1>(tmem_at, kTmemCols);
  // what depends on nothing
  if (warp >= kEndWarp && warp < kCodeWarp) {
    const int wt = tid - kEndWarp * 32;
    // the unit matrix in e2m1 (1.0 is 2): 16 bytes of row m hold dims 32 c .., the one lies at dim m
#pragma unroll 1
    for (int i = wt; i < C::EYE_BYTES / 16; i += 128) {
      const int m = i >> 2, c = (i & 3) ^ ((m >> 1) & 3), word = (m >> 3) & 3;
      const uint32_t one = (m >> 5) == c ? 2u << (4 * (m & 7)) : 0u;
      *reinterpret_cast<uint4*>(smem + C::EYE_OFFSET + (m >> 3) * 512 + (m & 7) * 64 + (i & 3) * 16) =
          make_uint4(word == 0 ? one : 0u, word == 1 ? one : 0u, word == 2 ? one : 0u, word == 3 ? one : 0u);
    }
    // the query rows beyond the terms, and the marks
    constexpr int USED = C::CC * kFp4Terms, REST = (C::N - USED) * (C::D / 32);  // 16-byte pieces of a buffer
#pragma unroll 1
    for (int i = wt; i < 2 * REST; i += 128) {
      const int r = i < REST ? i : i - REST;
      *reinterpret_cast<uint4*>(smem + C::Q_OFFSET + (i < REST ? 0 : C::Q_BYTES) +
                                code_offset<C>(USED + r / (C::D / 32), (r % (C::D / 32)) * 16)) = make_uint4(0u, 0u, 0u, 0u);
      if (i < (C::N - USED) * C::ROW_SF / 16)
        *reinterpret_cast<uint4*>(smem + C::QSF_OFFSET + USED * C::ROW_SF + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    for (int i = wt; i < C::SEGS * C::CC; i += 128) poison_of[i] = 0u;
  } else if (warp < kSfWarp && C::CC < 8) {  // P's unused columns
    for (int k = 0; k < 2; ++k)
      for (int i = lane; i < (8 - C::CC) * 8; i += 32)
        *reinterpret_cast<uint4*>(smem + C::P_OFFSET + k * C::P_BYTES + warp * 1024 + C::CC * 128 + i * 16) =
            make_uint4(0u, 0u, 0u, 0u);
  }
  if (!early) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  // One warp finds the share and its segments, and tells all others through shared
  // memory (20 that did it side by side took longer to begin, and the code of it was
  // fetched anew by every role at every segment: ~2000 cycles each).
  Walk walk;
  constexpr int WALK = sizeof(Walk) / 4;
  static_assert(WALK + 1 <= 32, "as laid out");
  int* begin = reinterpret_cast<int*>(smem + C::BEGIN_OFFSET);  // Walk; lengths [32]; tiles at 31
  Segment* seg_of = reinterpret_cast<Segment*>(smem + C::SEG_OFFSET);  // [SEGS]
  auto tell = [&](int sg, const Segment& s) {
    if (lane == 0) {
      seg_of[sg % C::SEGS] = s;
      mbar_arrive(&seg_full[sg % C::SEGS]);
    }
  };
  Segment seg;
  if (warp == kCodeWarp) {
    walk_start(p, walk);
    if (lane == 0) begin[31] = walk.left;
    if (walk_next<C::CC>(p, walk, seg)) tell(0, seg);
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < WALK; ++i) begin[i] = reinterpret_cast<const int*>(&walk)[i];
    }
    begin[32 + lane] = walk.lens;
    __syncwarp();
  }
  // the barriers and tensor memory are there (the copies do not wait for the other warps)
  if (copies) {
    named_bar_sync(5, (2 + SW) * 32);
    named_bar_arrive(4, C::THREADS);
  } else {
    named_bar_sync(4, C::THREADS);
    tmem_fence_after();
  }
  const int share_tiles = begin[31];
  bool any = share_tiles > 0;
  if (any) seg = seg_of[0];
  // the first segment's query terms, by all who have nothing to do yet
  if (warp < kCodeWarp) {
    if (any) {
      write_query_terms<C>(p, seg, smem + C::Q_OFFSET, smem + C::QSF_OFFSET, reinterpret_cast<float*>(smem + C::COL_OFFSET),
                           warp, 12, lane);
      fence_proxy_async_smem();
    }
    if (warp >= kEndWarp)
      named_bar_sync(7, 12 * 32);
    else
      named_bar_arrive(7, 12 * 32);
  }
  const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // this warp's lanes of tensor memory

  // A wait that runs out is reported; its role then goes through what is left of
  // its loops without waiting (the copies and the products stop), so that all
  // threads meet again.
  bool good = true;
  auto await = [&](uint64_t* bar, uint32_t phase) {
    if (good && __any_sync(kFullMask, !wait_for(bar, phase))) {
      good = false;
      if (lane == 0) atomicOr(p.err, kErrTimeout);
    }
  };

  if (copies) {
    // ---- copies, four tiles' page ids ahead (one tile ahead, their latency bound
    // the kernel, then 77 instead of 62 us): lane l has the 16 tokens 16 l .. of
    // four tiles
    const int mine = warp - kCodeWarp;  // 0: K's codes, 1: V's (K = V: the lower and the upper half), 2: scales (or 2: K's, 3: V's)
    const int v0 = C::KVS ? 0 : mine < 2 ? mine : SW == 2 ? mine - 2 : 0, v1 = !C::KVS && SW == 1 && mine == 2 ? 2 : v0 + 1;
    bool waited = !early, stop = false;
    uint32_t err_bits = 0;
    const uint64_t policy = l2_evict_first_policy();
    Segment next = seg;
    if (warp != kCodeWarp) {
#pragma unroll
      for (int i = 0; i < WALK; ++i) reinterpret_cast<int*>(&walk)[i] = begin[i];
      walk.lens = begin[32 + lane];
    }
    int page = -1, in_page = 0, rows = -1;
    auto page_of = [&](const Segment& s, int i) {
      const int t = s.t_base + i * kFp4Tile + lane * 16, at = t / p.page_size;
      in_page = t - at * p.page_size + s.g * p.page_size;
      page = t < s.thi ? __ldg(p.block_tables + (size_t)s.b * p.max_pages + at) : -1;
    };
    if (any) page_of(next, 0);
    int it = 0;  // tiles whose copies went out
#pragma unroll 1
    for (int sg = 0; any && !stop; ++sg) {
      const uint32_t odd = sg & 1 ? kTileOdd : 0u;
      seg = next;
      any = walk_next<C::CC>(p, walk, next);
      if (any && warp == kCodeWarp) tell(sg + 1, next);
#pragma unroll 1
      for (int i = 0; i < seg.tiles; ++i) {
        if ((i & 3) == 0) {
          const int t = seg.t_base + i * kFp4Tile + lane * 16;
          const bool here = (unsigned)page < (unsigned)p.num_pages;
          if (t < seg.thi && !here) err_bits |= kErrBadPage;
          rows = t < seg.thi && here ? page * p.num_kv_heads * p.page_size + in_page : -1;
          const bool on = i + 4 < seg.tiles;
          if (on || any) page_of(on ? seg : next, on ? i + 4 : 0);
        }
        const int row0 = __shfl_sync(kFullMask, rows, (i & 3) * 8 + (lane & 7));
        const uint32_t bits = __ballot_sync(kFullMask, row0 >= 0) & 0xffu;
        const uint32_t word = bits | odd | (i == 0 ? kTileFirst : 0u) | (i + 1 == seg.tiles ? kTileLast : 0u);
        // rows of the newest tokens may still be written by the kernel in front
        if (!waited && (it >= C::NK || (!C::KVS && it >= C::NV) ||
                        seg.t_base + (i + 1) * kFp4Tile > seg.L - p.query_tokens)) {
          grid_dependency_wait();
          grid_launch_dependents();
          waited = true;
        }
#pragma unroll 1
        for (int v = v0; v < v1; ++v) {
          const int n = v ? C::NV : C::NK, round = it / n, st = (v ? C::NK : 0) + it - round * n;
          if (round > 0 && __any_sync(kFullMask, !wait_for(&empty[st], round - 1))) {
            err_bits |= kErrTimeout;
            stop = true;
            break;
          }
          uint8_t* item = smem + st * C::ITEM_BYTES;
          if (mine < 2) {
            const uint32_t part = C::KVS ? bits & (mine ? 0xf0u : 0x0fu) : bits;
            if (lane == 0) {
              if (!C::KVS || mine == 0) valid[st] = word;
              if (part)
                mbar_arrive_expect_tx(&full[st], __popc(part) * (16 * C::D / 2) + (mine == 0 ? p.stall_bytes : 0));
              else
                mbar_arrive(&full[st]);
            }
            __syncwarp();
            // (one lane for all: eight lanes' take turns at ~130 cycles each)
            int at[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) at[k] = __shfl_sync(kFullMask, row0, k);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if ((part >> k) & 1u)
                  tma_load_4d(item + k * 16 * (C::D / 2), v ? &p.vmap : &p.kmap, 0, 0, 0, at[k] / 8, &full[st], policy);
            }
            __syncwarp();
          } else {
            // 16 bytes a lane (as bulk copies these would be half of all copies)
            constexpr int LANES = C::ROW_SF, EACH = C::KVS ? 8 / SW : 8;  // 16-byte pieces of 16 tokens' scales; a warp's 16s
            const int k0 = C::KVS && SW == 2 ? (mine - 2) * EACH : 0;
            const uint8_t* sf = (v ? p.v_sf : p.k_sf) + (lane % LANES) * 16;
            uint8_t* to = item + C::CODE_BYTES + lane * 16 + k0 * 16 * C::ROW_SF;
#pragma unroll
            for (int k = 0; k < EACH; k += 32 / LANES) {
              const int at = k0 + k + lane / LANES;  // the 16 tokens this lane copies a piece of
              const int row = __shfl_sync(kFullMask, row0, at);
              if (row >= 0) cp_async16(to + k * 16 * C::ROW_SF, sf + (size_t)row * C::ROW_SF);
            }
            cp_async_arrive(&full[st]);
          }
        }
        if (stop) break;
        ++it;
      }
    }
    // no copy may still be landing when the CTA ends
    const unsigned long long deadline = global_timer_ns() + kWaitTimeoutNs;
    for (int s = lane; s < RINGS; s += 32) {
      const int n = s < C::NK ? C::NK : C::NV, at = s < C::NK ? s : s - C::NK;
      if (at >= it || (!C::KVS && ((s >= C::NK) < v0 || (s >= C::NK) >= v1))) continue;
      const int last = at + n * ((it - 1 - at) / n);
      if (!mbar_wait_until(&full[s], (last / n) & 1, deadline)) err_bits |= kErrTimeout;
    }
    if (!waited) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
    err_bits = __reduce_or_sync(kFullMask, err_bits);
    if (lane == 0 && err_bits) atomicOr(p.err, err_bits);
  } else if (warp < kSfWarp) {
    // ---- softmax: rows 32 warp .. + 31 of every tile
    const uint32_t p_at = smem_u32(smem + C::P_OFFSET) + warp * 1024 + (lane & 3) * 4;
    float* top_of = reinterpret_cast<float*>(smem + C::TOP_OFFSET);  // [4][CC]
    int it = 0;
#pragma unroll 1
    for (int sg = 0; it < share_tiles; ++sg) {
      await(&q_full[sg & 1], sg >> 1);
      seg = seg_of[sg % C::SEGS];
      if (!good) seg.tiles = share_tiles - it;  // (as many turns as the other warps)
      if (seg.bad && good && tid == 0) atomicOr(p.err, kErrBadSeqLen);
      const float* col_mul = reinterpret_cast<const float*>(smem + C::COL_OFFSET) + (sg & 1) * C::CC;
      const uint32_t reach = p.window > 0 ? p.window : 0x7fffffff;
      float base[C::CC], top[C::CC], sum[C::CC];  // the reference (0 while there is none); what a score may not exceed
      int newest[C::CC];  // position a column attends: it and the reach - 1 before it
      {
        Pair col(seg);
#pragma unroll
        for (int c = 0; c < C::CC; ++c, col.next(p)) {
          newest[c] = col.valid(p) ? col.end(p, seg) - 1 : -1;
          base[c] = 0.f;
          top[c] = -INFINITY;
          sum[c] = 0.f;
        }
      }
      // tokens that all columns attend (of columns without a query row nothing is used: what they hold is finite)
      int whole_lo = 0, whole_hi = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        if (newest[c] < 0) continue;
        whole_hi = min(whole_hi, newest[c] + 1);
        if (p.window > 0) whole_lo = max(whole_lo, newest[c] + 1 - p.window);
      }
#pragma unroll 1
      for (int i = 0; i < seg.tiles; ++i, ++it) {
        const int buf = it & 1;
        await(s_full, it);
        tmem_fence_after();
        float s[C::CC];
        {
          // the terms' columns, smallest terms first, the sum brought down to the next term's size each time; 24 at a
          // time (for the registers), two columns an instruction
          uint64_t x[C::CC / 2];
#pragma unroll
          for (int c = 0; c < C::CC / 2; ++c) x[c] = 0;
#pragma unroll
          for (int k = kFp4Terms * C::CC - 24; k >= 0; k -= 24) {
            uint32_t lo[16], hi[8];
            tmem_ld(lo, kTmemS + quarter + k);
            tmem_ld(hi, kTmemS + quarter + k + 16);
            tmem_wait_ld();
#pragma unroll
            for (int i = 22; i >= 0; i -= 2) {
              const uint32_t a = i < 16 ? lo[i & 15] : hi[i & 7], b = i < 16 ? lo[(i & 15) + 1] : hi[(i & 7) + 1];
              // (volatile: it stays behind the wait for what it takes)
              asm volatile(
                  "{\n\t.reg .b64 f, y;\n\tmov.b64 f, {%3, %3};\n\tmov.b64 y, {%1, %2};\n\tfma.rn.f32x2 %0, %0, f, y;\n\t}"
                  : "+l"(x[i % C::CC / 2])
                  : "r"(a), "r"(b), "f"(1.f / kTermStep));
            }
          }
#pragma unroll
          for (int c = 0; c < C::CC / 2; ++c) {
            float lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x[c]));
            s[2 * c] = lo * col_mul[2 * c];
            s[2 * c + 1] = hi * col_mul[2 * c + 1];
          }
        }
        const int row = warp * 32 + lane, t = seg.t_base + i * kFp4Tile + row;
        const bool ok = (*blocks_of >> (row >> 4)) & 1u;
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        if (!__all_sync(kFullMask, ok && t >= whole_lo && t < whole_hi)) {
#pragma unroll
          for (int c = 0; c < C::CC; ++c)
            if (!ok || (uint32_t)(newest[c] - t) >= reach) s[c] = -INFINITY;
        }
        bool above = false;
#pragma unroll
        for (int c = 0; c < C::CC; ++c) above = above || s[c] > top[c];
        if (__builtin_expect(named_bar_or(2, 128, above), 0)) {
          // new references: the tile's maximum, where that is out of reach
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            const int m = __reduce_max_sync(kFullMask, ordered(isnan(s[c]) ? -INFINITY : s[c]));
            if (lane == 0) top_of[warp * C::CC + c] = unordered(m);
          }
          named_bar_sync(2, 128);
          float f[C::CC];
          bool held = false;
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            const float m = fmaxf(fmaxf(top_of[c], top_of[C::CC + c]), fmaxf(top_of[2 * C::CC + c], top_of[3 * C::CC + c]));
            const bool up = m > top[c];
            f[c] = up && top[c] != -INFINITY ? ex2(base[c] - m) : 1.f;
            held = held || f[c] != 1.f;
            sum[c] *= f[c];
            if (up) {
              base[c] = m;
              top[c] = m + kRefRange;
            }
          }
          named_bar_sync(2, 128);  // the maxima may be written again
          if (held) {
            // sums that hold something: rescaled once the tiles before are in them
            await(&p_empty[(it - 1) & 1], (it - 1) >> 1);
            tmem_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < CH; ++c0) {
              uint32_t o[8];
              tmem_ld(o, kTmemO + c0 * 16 + quarter);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < C::CC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
              tmem_st(kTmemO + c0 * 16 + quarter, o);
            }
            tmem_wait_st();
            tmem_fence_before();
          }
        }
        if (it >= 2) await(&p_empty[buf], (it >> 1) - 1);
        if (i == 0 && sg > 0) await(o_empty, sg - 1);  // (on behalf of the sums' product)
#pragma unroll
        for (int c = 0; c < C::CC; ++c) {
          // rounded to tf32 here, to nearest (the product would cut it off); the sum takes what the product takes
          uint32_t w;
          const float e = ex2(s[c] - base[c]);
          asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(w) : "f"(e));
          sum[c] += __uint_as_float(w);
          const uint32_t at = p_at + buf * C::P_BYTES + c * 128 + (((lane >> 2) ^ c) << 4);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
        }
        if (tid == 0) tile_of[buf] = (i == 0 ? kTileFirst : 0u) | (i + 1 == seg.tiles ? kTileLast : 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      float* sum_of = reinterpret_cast<float*>(smem + C::SUM_OFFSET) + (sg & 1) * 5 * C::CC;  // [4][CC], references
      if (sg >= 2) await(&l_empty[sg & 1], (sg >> 1) - 1);
#pragma unroll
      for (int c = 0; c < C::CC; ++c) {
        float l = sum[c];
#pragma unroll
        for (int m = 16; m; m >>= 1) l += __shfl_xor_sync(kFullMask, l, m);
        if (lane == 0) sum_of[warp * C::CC + c] = l;
        if (tid == 0) sum_of[4 * C::CC + c] = base[c];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&l_full[sg & 1]);
    }
  } else if (warp < kEndWarp) {
    // ---- a tile's scales put where tcgen05.cp takes them from, in place: from a row's
    // behind each other to 64 dims' of all rows behind each other. A lane has a row.
    const int j = warp - kSfWarp, row = j * 32 + lane;
    int it = 0;
#pragma unroll 1
    for (int sg = 0; it < share_tiles; ++sg) {
      await(&seg_full[sg % C::SEGS], sg / C::SEGS);
      seg = seg_of[sg % C::SEGS];
      if (!good) seg.tiles = share_tiles - it;
#pragma unroll 1
      for (int u = 0; u < (C::KVS ? 1 : 2) * seg.tiles; ++u) {
        const bool v = C::KVS || (u & 1) != 0;
        const int n = v && !C::KVS ? C::NV : C::NK, round = it / n, st = (v && !C::KVS ? C::NK : 0) + it - round * n;
        await(&full[st], round);
        uint8_t* sf = smem + st * C::ITEM_BYTES + C::CODE_BYTES;
        uint32_t x[C::KSTEPS];
#pragma unroll
        for (int k = 0; k < C::KSTEPS; k += 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(sf + row * C::ROW_SF + k * 4);
          x[k] = w.x;
          x[k + 1] = w.y;
          x[k + 2] = w.z;
          x[k + 3] = w.w;
        }
        if (v) {
          // rows that do not count have scale 0: their probabilities are 0, but 0 * NaN is NaN
          const int t = seg.t_base + (C::KVS ? u : u >> 1) * kFp4Tile + row;
          const bool counts = ((valid[st] >> (row >> 4)) & 1u) && t >= seg.tlo && t < seg.thi;
          uint32_t bad = 0u;
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k) {
            if (!counts) x[k] = 0u;
            bad |= nan_scales(x[k]);
          }
          if (__builtin_expect(bad != 0u, 0)) {
            // A NaN block would spread over the unit matrix's zeros to other dims (and, of
            // a token that only some of several query tokens attend, to the others): it is
            // taken out and marked for the results it belongs to: its dims' or, as K's
            // too, all.
            uint32_t blocks = 0u;
#pragma unroll
            for (int k = 0; k < C::KSTEPS; ++k) {
              const uint32_t nan = nan_scales(x[k]) >> 7;
              blocks |= ((nan * 0x10204080u) >> 28) << (4 * k);
              x[k] &= ~(nan * 0xffu);
            }
            Pair col(seg);
#pragma unroll 1
            for (int c = 0; c < C::CC && col.valid(p); ++c, col.next(p)) {
              const int end = col.end(p, seg);
              if (t < end && (p.window == 0 || t >= end - p.window))
                atomicOr(&poison_of[(sg % C::SEGS) * C::CC + c], C::KVS ? 0xffffffffu : blocks);
            }
          }
        }
        named_bar_sync(6, 128);  // all are read
#pragma unroll
        for (int k = 0; k < C::KSTEPS; ++k) *reinterpret_cast<uint32_t*>(sf + k * 512 + lane * 16 + j * 4) = x[k];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[st]);
        it += v;
      }
    }
  } else if (warp == kScoreWarp) {
    // ---- S = K q^T, by one lane, a tile after another
    if (share_tiles > 0 && elect_one()) {
      constexpr uint32_t kQk = (1u << 7) | (1u << 10) | ((uint32_t)(C::N / 8) << 17) | (8u << 24);  // e2m1, e4m3 scales
      constexpr uint32_t kRows = desc_hi(C::SL * 1024);
      // descriptors' lower words: 16-byte units, a step further is a constant added
      const uint32_t ring = smem_u32(smem) >> 4, q0 = ring + (C::Q_OFFSET >> 4);
      int i = 0, sk = 0, round = 0, sg = 0;  // the tile, its slot, its segment
      good = *tmem_at == 0;
#pragma unroll 1
      for (; i < share_tiles && good; ++i) {
        if (!(good = wait_for(&ready[sk], round))) break;
        const uint32_t word = valid[sk];
        if (word & kTileFirst) {
          if (!(good = wait_for(&q_full[sg & 1], sg >> 1))) break;
          ++sg;
        }
        // over the scores before once they are read (so their product has read K's scales too)
        if (i > 0 && !(good = wait_for(s_empty, i - 1))) break;
        tmem_fence_after();
        const uint32_t a = ring + sk * (C::ITEM_BYTES >> 4), q = q0 + ((word & kTileOdd) ? C::Q_BYTES >> 4 : 0);
#pragma unroll
        for (int k = 0; k < C::KSTEPS; ++k) copy_scales(kTmemSfk + k * 4, a + (C::CODE_BYTES >> 4) + k * 32);
#pragma unroll
        for (int k = 0; k < C::KSTEPS; ++k)
          mma_fp4<kRows, kRows, kQk>(kTmemS, a + (k >> 2) * 64 + (k & 3) * 2, q + (k >> 2) * 64 + (k & 3) * 2,
                                     kTmemSfk + k * 4, kTmemSfq + k * 4, k > 0);
        *blocks_of = word & 0xffu;
        mma_commit<1>(s_full);
        mma_commit<1>(&empty[sk]);
        if (word & kTileLast) mma_commit<1>(qk_done);
        mbar_arrive(s_full);
        if (++sk == C::NK) {
          sk = 0;
          ++round;
        }
      }
      // what was issued ends before its operands and results are used for something else
      if (i > 0) wait_for(s_full, i - 1);
      if (!good) atomicOr(p.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp >= kWideWarp && warp < kSumWarp) {
    // ---- V^T = I V^T, 128 dims at a time. Two lanes: one has the first buffer's chunks, one the second's.
    if (share_tiles > 0 && elect_one()) {
      constexpr uint32_t kDq = (1u << 7) | (1u << 10) | ((uint32_t)(kFp4Tile / 8) << 17) | (8u << 24);
      constexpr uint32_t kRows = desc_hi(C::SL * 1024), kEye = desc_hi(512, 64);
      const uint32_t me = warp - kWideWarp, ring = smem_u32(smem) >> 4, eye = ring + (C::EYE_OFFSET >> 4);
      int i = 0, sv = C::KVS ? 0 : C::NK, round = 0, use = 0;  // the tile, its slot; uses of a buffer so far
      // The unit matrix and its scales in tensor memory come from the warps that write the query terms, which say so
      // with the first segment's: a tile may be ready before. (That barrier's next phase waits for results of these
      // products, so the first one cannot be missed.)
      good = *tmem_at == 0 && wait_for(&q_full[0], 0);
#pragma unroll 1
      for (; i < share_tiles && good; ++i) {
        if (!(good = wait_for(&ready[sv], round))) break;
        const uint32_t item = ring + sv * (C::ITEM_BYTES >> 4) + me * 4;
        const uint32_t sf = ring + sv * (C::ITEM_BYTES >> 4) + (C::CODE_BYTES >> 4) + me * 64;
#pragma unroll 1
        for (int k = 0; k < CH / C::LANES; ++k) {
          // chunk me + k LANES, in buffer c
          const uint32_t c = C::LANES == 2 ? me : k & 1, sfv = kTmemSfv + me * 8 + k * 8 * C::LANES, to = kTmemVt + c * 128;
          const uint32_t v = item + (C::LANES == 2 ? k * 64 : (k >> 1) * 64 + (k & 1) * 4);
          // Its scales' columns were the chunk's of the tile before, whose product has to be
          // done: with a buffer a lane, the last wait said so of the chunk before last, which
          // that is (K = V at d 512: 66.2 -> 65.2 us); with two, this one will.
          auto scales = [&]() {
            copy_scales(sfv, sf + k * 64 * C::LANES);
            copy_scales(sfv + 4, sf + k * 64 * C::LANES + 32);
          };
          static_assert(C::LANES == 1 ? CH == 2 : CH == 4, "or the columns are another chunk's");
          if (C::LANES == 2) scales();
          if (use > 0 && !(good = good && wait_for(&vt_empty[c], use - 1))) break;
          tmem_fence_after();
          if (C::LANES == 1) scales();
          mma_fp4<kEye, kRows, kDq>(to, eye, v, kTmemSfi, sfv, false);
          mma_fp4<kEye, kRows, kDq>(to, eye + 2, v + 2, kTmemSfi, sfv + 4, true);
          mma_commit<1>(&vt_full[c]);
          mbar_arrive(&vt_full[c]);
          if (C::LANES == 2 || (k & 1)) ++use;
        }
        mma_commit<1>(&empty[sv]);
        if (++sv == RINGS) {
          sv = C::KVS ? 0 : C::NK;
          ++round;
        }
      }
      if (use > 0) wait_for(&vt_full[C::LANES == 2 ? me : 1], use - 1);
      if (!good) atomicOr(p.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp >= kSumWarp) {
    // ---- the sums O^T += V^T P^T, likewise
    if (share_tiles > 0 && elect_one()) {
      constexpr uint32_t kPv = (1u << 4) | (2u << 7) | (2u << 10) | (2u << 17) | (8u << 24);  // tf32 -> fp32, 128 x 16
      constexpr uint32_t kP = desc_hi(0);  // (both 8-column groups of P are the same: the upper columns are not read)
      const uint32_t me = warp - kSumWarp;
      const uint32_t p0 = (smem_u32(smem) + C::P_OFFSET) >> 4;
      int i = 0, use = 0;
#pragma unroll 1
      for (; i < share_tiles && good; ++i) {
        if (!(good = wait_for(&p_full[i & 1], i >> 1))) break;
        const uint32_t word = tile_of[i & 1], pa = p0 + (i & 1) * (C::P_BYTES >> 4);
        const bool more = (word & kTileFirst) == 0;
#pragma unroll 1
        for (int k = 0; k < CH / C::LANES; ++k) {
          const uint32_t c = C::LANES == 2 ? me : k & 1;
          if (!(good = wait_for(&vt_full[c], use))) break;
          tmem_fence_after();
          const uint32_t to = kTmemO + me * 16 + k * 16 * C::LANES, from = kTmemVt + c * 128;
#pragma unroll
          for (int q = 0; q < 16; ++q)
            mma_tf32<kP, kPv>(to, from + q * 8, pa + (q >> 2) * 64 + (q & 3) * 2, more || q > 0);
          mma_commit<1>(&vt_empty[c]);
          if (C::LANES == 2 || (k & 1)) ++use;
        }
        mma_commit<1>(&p_empty[i & 1]);
        if (word & kTileLast) {
          mma_commit<1>(o_full);
          mbar_arrive(o_full);
        }
      }
      if (use > 0) wait_for(&vt_empty[C::LANES == 2 ? me : 1], use - 1);
      if (!good) atomicOr(p.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    // ---- the next segment's query terms, and a segment's results
    const int we = warp - kEndWarp, wt = tid - kEndWarp * 32;
    volatile uint32_t* ticket = reinterpret_cast<uint32_t*>(smem + C::MISC_OFFSET);
    {
      uint32_t one[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) one[k] = 0x38383838u;  // e4m3 1.0
      tmem_st(kTmemSfi + quarter, one);
    }
    int left = share_tiles;  // tiles of the segments to come
    Segment next = seg;
#pragma unroll 1
    for (int sg = -1; sg < 0 ? any : true; ++sg) {
      any = left > 0;
      if (any) {
        await(&seg_full[(sg + 1) % C::SEGS], (sg + 1) / C::SEGS);
        if (named_bar_or(3, 128, !good)) break;  // (all of them or none)
        next = seg_of[(sg + 1) % C::SEGS];
        left -= next.tiles;
        // ---- segment sg + 1's terms (their buffer is free: the scores of segment sg - 1 are computed, as these warps
        // have seen), and their scales once segment sg's scores are computed
        if (sg >= 0) {
          named_bar_sync(3, 128);  // the scales before are in tensor memory
          write_query_terms<C>(p, next, smem + C::Q_OFFSET + ((sg + 1) & 1) * C::Q_BYTES, smem + C::QSF_OFFSET,
                               reinterpret_cast<float*>(smem + C::COL_OFFSET) + ((sg + 1) & 1) * C::CC, we, 4, lane);
          fence_proxy_async_smem();
          named_bar_sync(3, 128);
          await(qk_done, sg);
        }
        tmem_fence_after();
#pragma unroll
        for (int k0 = 0; k0 < C::KSTEPS; k0 += 4) {
          uint32_t x[16] = {};  // [64 dims][row group]
#pragma unroll
          for (int r = 0; r < C::N; r += 32) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (r + 32 <= C::N || r + lane < C::N)
              w = *reinterpret_cast<const uint4*>(smem + C::QSF_OFFSET + (r + lane) * C::ROW_SF + k0 * 4);
            x[r / 32] = w.x;
            x[4 + r / 32] = w.y;
            x[8 + r / 32] = w.z;
            x[12 + r / 32] = w.w;
          }
          tmem_st(kTmemSfq + quarter + k0 * 4, x);
        }
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[(sg + 1) & 1]);
      }
      if (sg >= 0) {
        // ---- segment sg's results
        await(&l_full[sg & 1], sg >> 1);
        const float* sum_of = reinterpret_cast<const float*>(smem + C::SUM_OFFSET) + (sg & 1) * 5 * C::CC;
        uint32_t* poison = poison_of + (sg % C::SEGS) * C::CC;
        const int slot = blockIdx.x * 2 + (seg.piece == 0 ? 1 : 0);
        // 0: no attended token, so zeros, whatever the sums hold. (Times 2^v_exp last: over a sum of 2^80 it would be subnormal.)
        float mul[C::CC];
#pragma unroll
        for (int c = 0; c < C::CC; ++c) {
          const float l = (sum_of[c] + sum_of[C::CC + c]) + (sum_of[2 * C::CC + c] + sum_of[3 * C::CC + c]);
          mul[c] = l != 0.f ? 1.f / l : 0.f;
          if (seg.pieces > 1 && wt == c)
            p.lse_part[slot * C::CC + c] =
                l != 0.f ? (sum_of[4 * C::CC + c] + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
        }
        await(o_full, sg);
        tmem_fence_after();
        // lane l of quarter w has dim 32 w + l of each chunk
        float x[CH][C::CC];
        uint32_t marks = 0u;
        {
          uint32_t o[CH][8];
#pragma unroll
          for (int k = 0; k < CH; ++k) tmem_ld(o[k], kTmemO + k * 16 + quarter);
          tmem_wait_ld();
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty);
#pragma unroll
          for (int c = 0; c < C::CC; ++c) {
            marks |= poison[c];
#pragma unroll
            for (int k = 0; k < CH; ++k) x[k][c] = mul[c] != 0.f ? __uint_as_float(o[k][c]) * mul[c] * p.v_mul : 0.f;
          }
        }
        const int dim = we * 32 + lane;
        if (__builtin_expect(marks != 0u, 0)) {
#pragma unroll
          for (int c = 0; c < C::CC; ++c)
#pragma unroll
            for (int k = 0; k < CH; ++k)
              if ((poison[c] >> ((k * 128 + dim) >> 4)) & 1u) x[k][c] = NAN;
        }
        if (seg.pieces > 1) {
          float* to = p.o_part + (size_t)slot * (C::CC * C::D) + dim;
#pragma unroll
          for (int c = 0; c < C::CC; ++c)
#pragma unroll
            for (int k = 0; k < CH; ++k) to[c * C::D + k * 128] = x[k][c];
        } else {
          Pair col(seg);
#pragma unroll
          for (int c = 0; c < C::CC; ++c, col.next(p)) {
            if (!col.valid(p)) break;
            __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(p.out) + col.row(p, seg) * C::D + dim;
#pragma unroll
            for (int k = 0; k < CH; ++k) to[k * 128] = __float2bfloat16_rn(x[k][c]);
          }
        }
        if (seg.pieces > 1) __threadfence();
        named_bar_sync(3, 128);
        if (lane == 0) mbar_arrive(&l_empty[sg & 1]);
        if (wt < C::CC) poison[wt] = 0u;
        if (seg.pieces > 1) {
          // whoever leaves the last piece joins them all, in their order:
          // out = sum_s w_s o_s,  w_s = exp(lse_s - M) / sum_s' exp(lse_s' - M)
          uint32_t* count = p.counters + seg.first_share / 4;
          const uint32_t byte = seg.first_share % 4 * 8;  // (a unit has at most as many pieces as there are CTAs: no carry)
          if (wt == 0) *ticket = (atomicAdd(count, 1u << byte) >> byte) & 0xffu;
          named_bar_sync(3, 128);
          if (*ticket == (uint32_t)seg.pieces - 1) {
            __threadfence();
            if (wt == 0) atomicAnd(count, ~(0xffu << byte));
            // a warp a column; piece q lies in slot 2 (first_share + q), the first one in the next
            constexpr int V4 = C::D / 128;  // float4s of a lane
            auto slot_of = [&](int q) { return (size_t)((seg.first_share + q) * 2 + (q == 0)) * C::CC; };
#pragma unroll 1
            for (int c = we; c < C::CC; c += 4) {
              const int at = seg.head + c, j = at / p.group + seg.token;
              if (j >= p.query_tokens) break;
              const size_t row = ((size_t)seg.b * p.query_tokens + j) * p.num_q_heads + (size_t)seg.g * p.group + at % p.group;
              float M = -INFINITY;
#pragma unroll 1
              for (int q = lane; q < seg.pieces; q += 32) M = fmaxf(M, __ldcg(p.lse_part + slot_of(q) + c));
#pragma unroll
              for (int m = 16; m; m >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, m));
              float4 acc[V4];
#pragma unroll
              for (int k = 0; k < V4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              float w_sum = 0.f;
#pragma unroll 2
              for (int q = 0; q < seg.pieces; ++q) {
                const float l = __ldcg(p.lse_part + slot_of(q) + c);
                const float4* o = reinterpret_cast<const float4*>(p.o_part + (slot_of(q) + c) * C::D) + lane;
                const float w = l == -INFINITY ? 0.f : ex2((l - M) * 1.4426950408889634f);
                w_sum += w;
#pragma unroll
                for (int k = 0; k < V4; ++k) {
                  const float4 y = __ldcg(o + k * 32);
                  acc[k].x = fmaf(w, y.x, acc[k].x);
                  acc[k].y = fmaf(w, y.y, acc[k].y);
                  acc[k].z = fmaf(w, y.z, acc[k].z);
                  acc[k].w = fmaf(w, y.w, acc[k].w);
                }
              }
              const float inv = w_sum != 0.f ? 1.f / w_sum : 0.f;
              uint2* to = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + row * C::D) + lane;
#pragma unroll
              for (int k = 0; k < V4; ++k)
                to[k * 32] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
            }
          }
        }
      }
      if (!any) break;
      seg = next;
    }
  }
  __syncthreads();
  if (warp == kScoreWarp) {
    tmem_fence_after();
    tmem_dealloc<1>(*tmem_at, kTmemCols);
  }
}

}  // namespace

const void* fp4_kernel_ptr(int variant) {
  switch (variant) {
#define PD_FP4_CASE(ID, D, KVS, CC) \
  case ID:                          \
    return reinterpret_cast<const void*>(&decode_fp4_kernel<Fp4Cfg<D, KVS, CC>>);
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
  p.counters = reinterpret_cast<uint32_t*>(ws + sizeof(uint32_t));
  p.lse_part = reinterpret_cast<float*>(ws + plan->lse_offset);
  p.o_part = reinterpret_cast<float*>(ws + plan->opart_offset);
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.scale_log2 = scale_log2;
  p.v_mul = std::ldexp(1.f, v_exp);
  p.stall_bytes = plan->test_stall_bytes;
  p.early_kv = plan->early_kv;
  p.batch = plan->batch;
  p.window = ly.window;
  p.num_pages = ly.num_pages;
  p.max_pages = ly.max_pages_per_seq;
  p.page_size = ly.page_size;
  p.num_q_heads = ly.num_q_heads;
  p.num_kv_heads = ly.num_kv_heads;
  p.query_tokens = plan->query_tokens;
  p.group = ly.num_q_heads / ly.num_kv_heads;
  p.col_tiles = (p.query_tokens * p.group + kVariants[plan->variant].group - 1) / kVariants[plan->variant].group;
  p.units = ly.num_kv_heads * p.col_tiles;
  p.cap = ly.max_pages_per_seq * ly.page_size;

  void* args[] = {&p};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan->grid_x);
  cfg.blockDim = dim3(plan->threads_per_cta);
  cfg.dynamicSmemBytes = plan->smem_bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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
