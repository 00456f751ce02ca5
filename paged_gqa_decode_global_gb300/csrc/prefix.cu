// The prefix pass of shared-prefix decode (sm_103a): attention of all of a
// group's query rows over its prefix, every prefix byte fetched once per row
// tile.
//
// Mathematics, for one (piece of the prefix, KV head, tile of N query rows),
// 128 tokens at a time, with the query rows on the N side of both products:
//   S^T[128 x N]  = K[128 x d] . q^T          (tokens on the M side)
//   P^T           = 2^(S^T scale log2 e - ref)  ref: each row's reference maximum
//   O^T[d x N]   += V^T[d x 128] . P^T        (head dims on the M side, 128 at a time)
// A query row is a column of both accumulators, so N = 16 rows cost what they
// need and d = 512 leaves room: O^T takes (d / 128) N columns of tensor memory
// (256 at N = 64), S^T two buffers of N. The sum of a row's probabilities is
// kept per token lane in registers and reduced once at the end. The reference
// of a row moves only when a score exceeds it by 2^8 (it then jumps to the true
// maximum and the row's O^T and sum are rescaled): any reference within range
// gives the same quotient, p <= 256 loses nothing in fp32 or bf16, and the
// rescale of O^T, a round trip through registers, becomes rare. Each row's
// references depend on its own scores only.
//
// Roles: warps 0-7 softmax and epilogue (a thread per token lane, two
// warpgroups with half the rows each: with one, its ~1700 instructions a tile
// at one warp per scheduler took 5 us against 1.9 us of products), warp 8 the
// matrix instructions, warps 9-11 the copies (every third stage each: a lone
// warp spends ~60 cycles a copy); FP8: warps 12-15 widen the e4m3 stages to f16 operands. K and V arrive as [8-token group][64-dim slab][8][128 B]
// atoms with the 128-byte swizzle: K-major for the first product, and the same
// layout read M-major for the second, so nothing is transposed; P is written N-major,
// a token's row at a time. A K=V layer fetches the tile again for its second
// use (an L2 hit).
//
// Roundings: P to the operands' type. bf16 cache: bf16, 2^-9 a probability. FP8
// cache: f16, into which e4m3 widens exactly; q rounds to f16 once (as in the
// decode), and P carries the page's V scale over the piece's largest, so that it
// stays below 2^8: 2^-12 a probability, 2^-25 absolute below 2^-14. Sums,
// references and accumulators stay in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "shared.h"
#include "tcgen05.cuh"

namespace pd {
namespace {

constexpr int kTok = kPrefixTile;
constexpr int kStage = kTok * 256;         // an operand stage: 128 dims of 128 tokens of K, or as many bytes of V
constexpr int kRaw = kStage / 2;           // FP8: the same in e4m3
constexpr int kBody = 224 * 1024;          // query rows, probabilities and rings
constexpr int kCopyWarps = 3;              // warps 9..11 (12 or 16 warps keep 168 or 128 registers a thread)
constexpr float kSlack = 8.f;              // log2 of what a probability may exceed 1 by
constexpr float kLow = 3e38f;              // negated reference of a row without a score yet
constexpr int kNoTop = (int)0x807fffff;    // ordered(-inf)

template <int D_, int N_, bool FP8_>
struct PrefixCfg {
  static constexpr int D = D_, N = N_;
  static constexpr bool FP8 = FP8_;
  static constexpr int KS = D / 128;       // stages of a tile's K (and of its V)
  static constexpr int VT = kTok / KS;     // tokens of a V stage
  static constexpr int Q_BYTES = N * D * 2, P_BYTES = N * kTok * 2;
  static constexpr int ROOM = kBody - Q_BYTES - P_BYTES;
  static constexpr int NST = FP8 ? 3 : (ROOM / kStage < 6 ? ROOM / kStage : 6);
  static constexpr int NRAW = FP8 ? ((ROOM - NST * kStage) / kRaw < 6 ? (ROOM - NST * kStage) / kRaw : 6) : 0;
  static constexpr int Q_OFFSET = 0, P_OFFSET = Q_BYTES, RING_OFFSET = P_OFFSET + P_BYTES;
  static constexpr int RAW_OFFSET = RING_OFFSET + NST * kStage;
  static constexpr int REF_OFFSET = RAW_OFFSET + NRAW * kRaw;   // float nref[N]: negated references
  static constexpr int TOP_OFFSET = REF_OFFSET + N * 4;         // int top[N]: a tile's true maxima
  static constexpr int ROW_OFFSET = TOP_OFFSET + N * 4;         // int row[N]: a tile row's row of q and out
  static constexpr int BAR_OFFSET = ROW_OFFSET + N * 4;
  static constexpr int NBAR = 2 * NST + 2 * NRAW + 2 + 2 + 1 + 1 + 1 + 1;
  static constexpr int TMEM_OFFSET = BAR_OFFSET + NBAR * 8;
  static constexpr int SMEM_BYTES = TMEM_OFFSET + 16 + 1024;
  static constexpr int THREADS = 32 * (9 + kCopyWarps + (FP8 ? 4 : 0));
  static constexpr int CW = N / 2;         // rows of a softmax warpgroup
  static constexpr int LD = CW < 32 ? CW : 32;
  // P: [N / 64 blocks][128 tokens][row of up to 64 query rows], swizzled over the row
  static constexpr int P_ROW = N >= 64 ? 128 : N * 2;
  static constexpr int O_COLS = KS * N;
  static constexpr int TMEM_COLS = O_COLS + 2 * N <= 64 ? 64 : O_COLS + 2 * N <= 128 ? 128 :
                                   O_COLS + 2 * N <= 256 ? 256 : 512;
  static_assert(O_COLS + 2 * N <= 512, "tensor memory");
  static_assert(NST >= 3 && (!FP8 || NRAW >= 2), "rings");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(2 * (kTok * (CW + 1) + 128) * 4 <= NST * kStage, "the row sums are reduced in the ring");
};

struct Tile {
  int group, first, rows, start;
};

// Row tile z of the launch: its group, first row and rows (group -1: none).
// Every warp finds it by itself, 32 groups at a time.
__device__ __forceinline__ Tile find_tile(const SharedParams& p, int z) {
  const int lane = threadIdx.x & 31, per_req = p.query_tokens * p.group;
  int at = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
    const int g = g0 + lane;
    int s = 0, rows = 0;
    if (g < p.num_groups) {
      s = max(0, min(__ldg(p.group_starts + g), p.batch));
      rows = (max(s, min(__ldg(p.group_starts + g + 1), p.batch)) - s) * per_req;
    }
    const int n = (rows + p.row_tile - 1) / p.row_tile;
    int end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFullMask, end, o);
      if (lane >= o) end += y;
    }
    end += at;
    const uint32_t in = __ballot_sync(kFullMask, z < end);
    if (in) {
      const int src = __ffs(in) - 1;
      Tile t;
      t.group = g0 + src;
      t.first = (z - __shfl_sync(kFullMask, end - n, src)) * p.row_tile;
      t.rows = min(p.row_tile, __shfl_sync(kFullMask, rows, src) - t.first);
      t.start = __shfl_sync(kFullMask, s, src);
      return t;
    }
    at = __shfl_sync(kFullMask, end, 31);
  }
  return Tile{-1, 0, 0, 0};
}

// Whether the device's group starts cut the batch, in no more row tiles than planned (one warp).
__device__ __forceinline__ bool groups_ok(const SharedParams& p) {
  const int lane = threadIdx.x & 31, per_req = p.query_tokens * p.group;
  bool ok = p.group_starts[0] == 0 && p.group_starts[p.num_groups] == p.batch;
  int tiles = 0;
  for (int g = lane; g < p.num_groups; g += 32) {
    const int s = p.group_starts[g], e = p.group_starts[g + 1];
    ok = ok && s >= 0 && e >= s && e <= p.batch;
    if (ok) tiles += ((e - s) * per_req + p.row_tile - 1) / p.row_tile;
  }
  ok = __all_sync(kFullMask, ok);
  return ok && __reduce_add_sync(kFullMask, tiles) <= p.tiles;
}

// Row r of a tile: its row of q and out, [batch, T, Hq].
__device__ __forceinline__ int row_of(const SharedParams& p, const Tile& t, int r, int g) {
  const int i = t.first + r, per_req = p.query_tokens * p.group;
  return ((t.start + i / per_req) * p.query_tokens + (i / p.group) % p.query_tokens) * p.num_q_heads + g * p.group +
         i % p.group;
}

// Floats as signed integers of the same order, for an integer warp maximum.
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int k) { return __int_as_float(k >= 0 ? k : k ^ 0x7fffffff); }

// Four e4m3 codes -> four f16, exactly (NaN included).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Two fp32 as the operand type, the first in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two bf16 -> two f16.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t w) {
  return pack2<true>(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) prefix_kernel(const __grid_constant__ SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int N = C::N, D = C::D, KS = C::KS, NST = C::NST;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFFSET);
  uint64_t* empty = full + NST;
  uint64_t* raw_full = empty + NST;
  uint64_t* raw_empty = raw_full + C::NRAW;
  uint64_t* s_full = raw_empty + C::NRAW;  // [2]
  uint64_t* s_empty = s_full + 2;          // [2]
  uint64_t* p_full = s_empty + 2;
  uint64_t* p_empty = p_full + 1;
  uint64_t* q_full = p_empty + 1;
  uint64_t* drained = q_full + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::TMEM_OFFSET);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

  if (tid == 288) {
    prefetch_tensormap(&p.kmap);
    prefetch_tensormap(&p.vmap);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], C::FP8 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NRAW; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 256);
    }
    mbar_init(p_full, 256);
    mbar_init(p_empty, 1);
    mbar_init(q_full, 256);
    mbar_init(drained, 1);
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(tmem_at, C::TMEM_COLS);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  // launched behind the own part's stage 1, whose threads let this grid start
  // only after their own wait: all that both read is in place, and nothing here
  // depends on stage 1 itself, so this grid waits for it only as it ends (the
  // join behind it relies on both)
  grid_launch_dependents();

  const int piece = blockIdx.y, g = blockIdx.z;
  if (blockIdx.x == 0 && piece == 0 && g == 0 && warp == 0 && !groups_ok(p) && lane == 0)
    atomicOr(p.err, kErrBadGroup);
  const Tile t = find_tile(p, blockIdx.x);
  int L = 0;
  if (t.group >= 0) {
    L = __ldg(p.prefix_lens + t.group);
    const int cap = p.max_prefix_pages * p.page_size;
    if (L < 0 || L > cap || L % p.page_size != 0) {
      if (tid == 0) atomicOr(p.err, kErrBadSeqLen);
      L = max(0, min(L, cap)) / p.page_size * p.page_size;
    }
  }
  // this piece's tokens [lo, hi); the last piece takes whatever remains
  const long long want = (long long)piece * p.chunk_tokens;
  const int lo = (int)min(want, (long long)L);
  const int hi = piece == p.num_pieces - 1 ? L : (int)min((long long)L, want + p.chunk_tokens);
  const int ntile = (hi - lo + kTok - 1) / kTok;
  const int32_t* table = p.prefix_tables + (size_t)max(t.group, 0) * p.max_prefix_pages;

  if (ntile == 0) {
    // nothing here: weight 0 (the join reads no row of such a piece)
    for (int r = tid; r < t.rows; r += C::THREADS)
      p.lse_part[(size_t)row_of(p, t, r, g) * p.num_pieces + piece] = -INFINITY;
  } else if (warp >= 9 && warp < 9 + kCopyWarps) {
    // ---- copies: stages in the order the products use them, K(0), K(1), V(0), K(2), V(1), ...
    // A K stage is 128 dims of the tile, a V stage all dims of VT tokens; both
    // land as [8-row group][64-dim slab][8 rows][128 B], so that a 16-token page
    // takes one copy of 4 KB (K) or 16 KB (V, d = 512): with a copy per page and
    // slab (2 KB) the copies took 5.5 us a tile. Lane j holds the pool row of
    // the tile's j-th K box and j-th V box.
    const int v_boxes = C::VT / p.v_box;
    const uint64_t policy = p.keep_in_l2 ? l2_evict_normal_policy() : l2_evict_first_policy();
    constexpr int NR = C::FP8 ? C::NRAW : NST;
    constexpr int BYTES = C::FP8 ? kRaw : kStage;
    constexpr int K_SLABS = C::FP8 ? 1 : 2, ROW_BYTES = C::FP8 ? D : 2 * D;
    uint64_t* land = C::FP8 ? raw_full : full;
    uint64_t* freed = C::FP8 ? raw_empty : empty;
    uint8_t* ring = smem + (C::FP8 ? C::RAW_OFFSET : C::RING_OFFSET);
    uint32_t err = 0;
    // the 8-row group of the pool where this lane's box of a tile starts (-1:
    // past the piece); a page outside the pool is fetched past the pool's end,
    // which reads zeros
    auto group_at = [&](int tile, int box) -> int {
      const int tok = lo + tile * kTok + lane * box;
      if (tile >= ntile || tok >= hi || lane >= kTok / box) return -1;
      const int page = __ldg(table + tok / p.page_size);
      if ((unsigned)page >= (unsigned)p.num_pages) {
        err |= kErrBadPage;
        return p.num_pages * p.num_kv_heads * p.page_size / 8;
      }
      return ((page * p.num_kv_heads + g) * p.page_size + tok % p.page_size) / 8;
    };
    int st = 0, uses = 0;  // the next stage, and how many stages were passed
    int turn = warp - 9;   // stages until this warp's next
    uint32_t phase = 1;    // of the stage's release (the first round waits for nothing)
    bool ok = true;
    // this warp's stage, free to be filled? (ok false: the wait ran out)
    auto begin = [&](int boxes, int box_bytes) {
      if (turn != 0) return false;
      ok = __all_sync(kFullMask, uses < NR || mbar_wait(&freed[st], phase));
      if (ok && lane == 0) mbar_arrive_expect_tx(&land[st], boxes * box_bytes + p.stall_bytes);
      __syncwarp();
      return ok;
    };
    auto end = [&] {
      turn = turn == 0 ? kCopyWarps - 1 : turn - 1;
      ++uses;
      if (++st == NR) {
        st = 0;
        phase ^= 1;
      }
    };
    auto load_k = [&](int at) {
      const int bytes = p.k_box * 128 * K_SLABS;
      const int boxes = __popc(__ballot_sync(kFullMask, at >= 0));
#pragma unroll 1
      for (int s = 0; s < KS; ++s) {
        if (begin(boxes, bytes) && at >= 0)
          tma_load_4d(ring + st * BYTES + lane * bytes, &p.kmap, 0, 0, s * K_SLABS, at, &land[st], policy);
        if (!ok) return;
        end();
      }
    };
    auto load_v = [&](int at) {
      const int bytes = p.v_box * ROW_BYTES;
#pragma unroll 1
      for (int s = 0; s < KS; ++s) {
        const bool mine = at >= 0 && lane / v_boxes == s;
        if (begin(__popc(__ballot_sync(kFullMask, mine)), bytes) && mine)
          tma_load_4d(ring + st * BYTES + lane % v_boxes * bytes, &p.vmap, 0, 0, 0, at, &land[st], policy);
        if (!ok) return;
        end();
      }
    };
    int k_next = group_at(0, p.k_box), v_at = group_at(0, p.v_box);
    load_k(k_next);
    k_next = group_at(1, p.k_box);
#pragma unroll 1
    for (int i = 0; i < ntile && ok; ++i) {
      const int k_after = group_at(i + 2, p.k_box), v_next = group_at(i + 1, p.v_box);
      if (i + 1 < ntile) load_k(k_next);
      if (ok) load_v(v_at);
      k_next = k_after;
      v_at = v_next;
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0) {
      const unsigned long long deadline = global_timer_ns() + kWaitTimeoutNs;
      for (int k = max(0, uses - NR); k < uses; ++k)
        if (k % kCopyWarps == warp - 9 && !mbar_wait_until(&land[k % NR], (k / NR) & 1, deadline)) ok = false;
      if (!ok) err |= kErrTimeout;
    }
    err = __reduce_or_sync(kFullMask, err);
    if (lane == 0 && err) atomicOr(p.err, err);
  } else if (warp == 8) {
    // ---- matrix instructions: QK(0), then QK(i + 1) ahead of PV(i). The warp
    // walks the stages together and one elected lane issues: a lone thread
    // computing descriptors took ~180 cycles an instruction.
    constexpr uint32_t kQk = mma_desc_16bit(!C::FP8, 128, N, false, false);
    constexpr uint32_t kPv = mma_desc_16bit(!C::FP8, 128, N, true, true);
    // descriptors' bases; a step further is a constant added to the address field
    const uint32_t base = smem_u32(smem);
    const uint64_t k_desc = smem_desc(base + C::RING_OFFSET, 16, 2048), q_desc = smem_desc(base, 16, 1024);
    const uint64_t v_desc = smem_desc(base + C::RING_OFFSET, 1024, D * 16);
    const uint64_t p_desc = smem_desc(base + C::P_OFFSET, kTok * 128, 8 * C::P_ROW, C::P_ROW);
    int st = 0;
    uint32_t phase = 0;
    bool ok = __all_sync(kFullMask, mbar_wait(q_full, 0));
    auto next_stage = [&] {
      if (++st == NST) {
        st = 0;
        phase ^= 1;
      }
    };
    auto qk = [&](int i) {
      if (ok && i >= 2) ok = __all_sync(kFullMask, mbar_wait(&s_empty[i & 1], ((i >> 1) - 1) & 1));
      const uint32_t d = tmem + C::O_COLS + (i & 1) * N;
#pragma unroll 1
      for (int s = 0; s < KS && ok; ++s) {
        ok = __all_sync(kFullMask, mbar_wait(&full[st], phase));
        if (!ok) return;
        tmem_fence_after();
        if (elect_one()) {
          const uint64_t a = k_desc + st * (kStage >> 4), b = q_desc + s * 2 * (N * 128 >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(d, a + (k >> 2) * (1024 >> 4) + (k & 3) * 2, b + (k >> 2) * (N * 128 >> 4) + (k & 3) * 2, kQk,
                   k != 0 || s != 0);
          mma_commit(&empty[st]);
          if (s == KS - 1) mma_commit(&s_full[i & 1]);
        }
        __syncwarp();
        next_stage();
      }
    };
    qk(0);
#pragma unroll 1
    for (int i = 0; i < ntile && ok; ++i) {
      if (i + 1 < ntile) qk(i + 1);
      if (ok) ok = __all_sync(kFullMask, mbar_wait(p_full, i & 1));
      const int steps = min(kTok, hi - lo - i * kTok) / 16;
#pragma unroll 1
      for (int s = 0; s < KS && ok; ++s) {
        ok = __all_sync(kFullMask, mbar_wait(&full[st], phase));
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) {
          const uint64_t a = v_desc + st * (kStage >> 4), b = p_desc + s * (C::VT * C::P_ROW >> 4);
          // 16 tokens at a time, all head dims
          if ((s + 1) * (C::VT / 16) <= steps) {
#pragma unroll
            for (int k = 0; k < C::VT / 16; ++k)
#pragma unroll
              for (int m = 0; m < KS; ++m)
                mma_ss(tmem + m * N, a + k * (D * 32 >> 4) + m * (2048 >> 4), b + k * (16 * C::P_ROW >> 4), kPv,
                       k != 0 || s != 0 || i != 0);
          } else {
#pragma unroll 1
            for (int k = 0; s * (C::VT / 16) + k < steps; ++k)
#pragma unroll 1
              for (int m = 0; m < KS; ++m)
                mma_ss(tmem + m * N, a + k * (D * 32 >> 4) + m * (2048 >> 4), b + k * (16 * C::P_ROW >> 4), kPv,
                       k != 0 || s != 0 || i != 0);
          }
          mma_commit(&empty[st]);
          if (s == KS - 1) mma_commit(p_empty);
        }
        __syncwarp();
        next_stage();
      }
    }
    if (!ok) {
      // nothing may still be reading shared memory when the CTA exits
      if (elect_one()) {
        mma_commit(drained);
        mbar_wait(drained, 0);
        atomicOr(p.err, kErrTimeout);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ---- softmax: a thread per token lane, warpgroup wg the rows [wg CW, wg CW + CW)
    constexpr int CW = C::CW, LD = C::LD;
    const int wg = warp >> 2, lt = tid & 127, bar = 1 + wg;
    float* nref = reinterpret_cast<float*>(smem + C::REF_OFFSET) + wg * CW;
    int* top = reinterpret_cast<int*>(smem + C::TOP_OFFSET) + wg * CW;
    int* rows = reinterpret_cast<int*>(smem + C::ROW_OFFSET);
    if (tid < N) rows[tid] = tid < t.rows ? row_of(p, t, tid, g) : -1;
    if (lt < CW) {
      nref[lt] = kLow;
      top[lt] = kNoTop;
    }
    __syncwarp();
    named_bar_sync(3, 256);
    // the tile's query rows, swizzled as the K-major operand; all of a round's loads in flight at once
    constexpr int kChunks = N * (D / 8), kRound = kChunks / 256 < 16 ? kChunks / 256 : 16;
#pragma unroll 1
    for (int e0 = tid; e0 < kChunks; e0 += 256 * kRound) {
      uint4 v[kRound];
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        const int e = e0 + u * 256, r = rows[e / (D / 8)];
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= 0) v[u] = __ldg(reinterpret_cast<const uint4*>(p.q + (size_t)r * D) + e % (D / 8));
      }
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        const int e = e0 + u * 256, r = e / (D / 8), c = e % (D / 8);
        if constexpr (C::FP8)
          v[u] = make_uint4(to_f16x2(v[u].x), to_f16x2(v[u].y), to_f16x2(v[u].z), to_f16x2(v[u].w));
        *reinterpret_cast<uint4*>(smem + C::Q_OFFSET + (c >> 3) * N * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
            v[u];
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(q_full);

    float v_top = 1.f, v_inv = 1.f;  // FP8: the piece's largest V scale
    if constexpr (C::FP8) {
      float m = 0.f;
      for (int tok = lo + lt * 16; tok < hi; tok += 128 * 16) {
        const int page = __ldg(table + tok / p.page_size);
        if ((unsigned)page < (unsigned)p.num_pages)
          m = fmaxf(m, fabsf(__ldg(p.v_scale + (size_t)page * p.num_kv_heads + g)));
      }
      const int k = __reduce_max_sync(kFullMask, __float_as_int(m));
      if (lane == 0) atomicMax(top, k);
      __syncwarp();
      named_bar_sync(bar, 128);
      v_top = __int_as_float(top[0]);
      v_inv = v_top > 0.f ? 1.f / v_top : 0.f;
      named_bar_sync(bar, 128);
      if (lt == 0) top[0] = kNoTop;
      __syncwarp();
    }

    const uint32_t quarter = tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t o_at = quarter + wg * CW;
    float l[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) l[c] = 0.f;
    uint32_t err = 0;
    bool ok = true;
    // this lane's token of tile i: whether it is attended, its scales
    auto token = [&](int i, bool& valid, float& ks, float& vs) {
      const int tok = lo + i * kTok + lt;
      valid = false;
      ks = 1.f;
      vs = 1.f;
      if (i < ntile && tok < hi) {
        const int page = __ldg(table + tok / p.page_size);
        valid = (unsigned)page < (unsigned)p.num_pages;
        if constexpr (C::FP8) {
          if (valid) {
            ks = __ldg(p.k_scale + (size_t)page * p.num_kv_heads + g);
            vs = __ldg(p.v_scale + (size_t)page * p.num_kv_heads + g);
          }
        }
      }
    };
    // P: this token's row; its 16-byte chunks swizzled over the row
    constexpr int kChunkMask = C::P_ROW / 16 - 1, kSwShift = N >= 64 ? 0 : N == 32 ? 1 : 2;
    uint8_t* p_row = smem + C::P_OFFSET + lt * C::P_ROW + (N == 128 ? wg * (kTok * 128) : 0);
    const int p_sw = (lt >> kSwShift) & kChunkMask, p_chunk = N == 128 ? 0 : wg * (CW / 8);
    bool valid;
    float ks, vs;
    token(0, valid, ks, vs);
#pragma unroll 1
    for (int i = 0; i < ntile; ++i) {
      bool nvalid;
      float nks, nvs;
      token(i + 1, nvalid, nks, nvs);
      const float sc = p.scale_log2 * ks;
      ok = mbar_wait(&s_full[i & 1], (i >> 1) & 1) && ok;
      __syncwarp();
      tmem_fence_after();
      const uint32_t sa = quarter + C::O_COLS + (i & 1) * N + wg * CW;
      // does any score leave its row's range?
      float over = -INFINITY;
      uint32_t x[LD];
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += LD) {
        tmem_ld(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < LD; ++c) over = fmaxf(over, fmaf(__uint_as_float(x[c]), sc, nref[c0 + c]));
      }
      if (named_bar_or(bar, 128, !ok || (valid && over > kSlack))) {
        // the rows that left theirs take the true maximum; P(i - 1) is spent
        if (i > 0) ok = mbar_wait(p_empty, (i - 1) & 1) && ok;
        __syncwarp();
        if (named_bar_or(bar, 128, !ok)) break;
        tmem_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < CW; c0 += LD) {
          tmem_ld(x, sa + c0);
          tmem_wait_ld();
          int mine = kNoTop;
#pragma unroll
          for (int c = 0; c < LD; ++c) {
            const int m = __reduce_max_sync(kFullMask, ordered(valid ? __uint_as_float(x[c]) * sc : -INFINITY));
            if (lane == c) mine = m;
          }
          if (lane < LD) atomicMax(top + c0 + lane, mine);
        }
        __syncwarp();
        named_bar_sync(bar, 128);
        // a row moves if its maximum left the range: factor of what it holds so far
        auto moves = [&](int c) { return unordered(top[c]) + nref[c] > kSlack; };
        auto factor = [&](int c) { return moves(c) ? ex2(-nref[c] - unordered(top[c])) : 1.f; };
#pragma unroll
        for (int c = 0; c < CW; ++c) l[c] *= factor(c);
        if (i > 0) {
#pragma unroll
          for (int c0 = 0; c0 < CW; c0 += LD) {
            float f[LD];
#pragma unroll
            for (int c = 0; c < LD; ++c) f[c] = factor(c0 + c);
#pragma unroll 1
            for (int s = 0; s < KS; ++s) {
              tmem_ld(x, o_at + s * N + c0);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < LD; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * f[c]);
              tmem_st(o_at + s * N + c0, x);
            }
          }
          tmem_wait_st();
        }
        named_bar_sync(bar, 128);
        if (lt < CW) {
          if (moves(lt)) nref[lt] = -unordered(top[lt]);
          top[lt] = kNoTop;
        }
        __syncwarp();
        named_bar_sync(bar, 128);
      } else if (i > 0) {
        ok = mbar_wait(p_empty, (i - 1) & 1);
        __syncwarp();
      }
      const bool all = __all_sync(kFullMask, valid);
      const float pv = vs * v_inv;
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += LD) {
        tmem_ld(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < LD; c += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float e[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int cc = c + 2 * k + u;
              e[u] = ex2(fmaf(__uint_as_float(x[cc]), sc, nref[c0 + cc]));
              if (!all && !valid) e[u] = 0.f;
              l[c0 + cc] += e[u];
              if constexpr (C::FP8) e[u] = !all && !valid ? 0.f : e[u] * pv;
            }
            w[k] = pack2<C::FP8>(e[0], e[1]);
          }
          *reinterpret_cast<uint4*>(p_row + (((p_chunk + (c0 + c) / 8) ^ p_sw) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      tmem_fence_before();
      mbar_arrive(p_full);
      mbar_arrive(&s_empty[i & 1]);
      if (!valid && lo + i * kTok + lt < hi) err |= kErrBadPage;
      valid = nvalid;
      ks = nks;
      vs = nvs;
    }
    ok = ok && mbar_wait(p_empty, (ntile - 1) & 1);
    __syncwarp();
    // (both warpgroups: the sums go where the other's last products read)
    if (named_bar_or(3, 256, !ok)) {
      err |= kErrTimeout;
    } else {
      tmem_fence_after();
      // the rows' sums over the token lanes, in the ring (every product is done with it)
      float* sum = reinterpret_cast<float*>(smem + C::RING_OFFSET) + wg * (kTok * (CW + 1) + 128);
      float* part = sum + kTok * (CW + 1);
#pragma unroll
      for (int c = 0; c < CW; ++c) sum[lt * (CW + 1) + c] = l[c];
      named_bar_sync(bar, 128);
      const int col = lt % CW, first = lt / CW * CW;
      float a[2] = {0.f, 0.f};
#pragma unroll 4
      for (int k = 0; k < CW; k += 2) {
        a[0] += sum[(first + k) * (CW + 1) + col];
        a[1] += sum[(first + k + 1) * (CW + 1) + col];
      }
      part[lt] = a[0] + a[1];
      named_bar_sync(bar, 128);
      if (lt < CW) {
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < 128 / CW; ++k) total += part[k * CW + lt];
        // no attended token: weight 0 and a zero row; NaN stays NaN
        if (rows[wg * CW + lt] >= 0)
          p.lse_part[(size_t)rows[wg * CW + lt] * p.num_pieces + piece] =
              total == 0.f ? -INFINITY : (log2f(total) - nref[lt]) * 0.69314718055994530942f;
        nref[lt] = total == 0.f ? 0.f : v_top / total;
      }
      __syncwarp();
      named_bar_sync(bar, 128);
      constexpr int OC = CW < 16 ? CW : 16;
#pragma unroll 1
      for (int c0 = 0; c0 < CW; c0 += OC) {
        if (wg * CW + c0 >= t.rows) break;
        uint32_t y[KS][OC];
#pragma unroll
        for (int s = 0; s < KS; ++s) tmem_ld(y[s], o_at + s * N + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < OC; ++c) {
          const int r = rows[wg * CW + c0 + c];
          if (r < 0) break;
          float* dst = p.o_part + ((size_t)r * p.num_pieces + piece) * D + lt;
          const float f = nref[c0 + c];
#pragma unroll
          for (int s = 0; s < KS; ++s) dst[s * 128] = __uint_as_float(y[s][c]) * f;
        }
      }
    }
    err = __reduce_or_sync(kFullMask, err);
    if (lane == 0 && err) atomicOr(p.err, err);
  } else if constexpr (C::FP8) {
    // ---- FP8: e4m3 stages widened to f16 operand stages, a thread per token row
    const int row = tid - 32 * (9 + kCopyWarps), sw = row & 7, total = 2 * KS * ntile;
    bool ok = true;
    for (int it = 0; it < total; ++it) {
      const int st = it % NST, rs = it % C::NRAW;
      ok = mbar_wait(&raw_full[rs], (it / C::NRAW) & 1);
      if (ok && it >= NST) ok = mbar_wait(&empty[st], ((it / NST) - 1) & 1);
      if (__any_sync(kFullMask, !ok)) {
        if (lane == 0) atomicOr(p.err, kErrTimeout);
        break;
      }
      const uint8_t* src = smem + C::RAW_OFFSET + rs * kRaw + row * 128;
      uint8_t* dst = smem + C::RING_OFFSET + st * kStage + (row >> 3) * 2048 + (row & 7) * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
        uint4 a, b;
        widen4(w.x, a.x, a.y);
        widen4(w.y, a.z, a.w);
        widen4(w.z, b.x, b.y);
        widen4(w.w, b.z, b.w);
        uint8_t* to = dst + (c >> 2) * 1024;
        const int cc = (c & 3) * 2;
        *reinterpret_cast<uint4*>(to + ((cc ^ sw) << 4)) = a;
        *reinterpret_cast<uint4*>(to + (((cc + 1) ^ sw) << 4)) = b;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&raw_empty[rs]);
        mbar_arrive(&full[st]);
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, C::TMEM_COLS);
  grid_dependency_wait();
}

#define PD_FOR_EACH_PREFIX(X)                                                                          \
  X(0, 512, 16, false) X(1, 512, 32, false) X(2, 512, 64, false) X(3, 256, 16, false)                  \
  X(4, 256, 32, false) X(5, 256, 64, false) X(6, 256, 128, false) X(7, 128, 16, false)                 \
  X(8, 128, 32, false) X(9, 128, 64, false) X(10, 128, 128, false) X(11, 512, 16, true)                \
  X(12, 512, 32, true) X(13, 512, 64, true) X(14, 256, 16, true) X(15, 256, 32, true)                  \
  X(16, 256, 64, true) X(17, 256, 128, true)

}  // namespace

#define PD_PREFIX_ROW(ID, D, N, F)                                                                     \
  PrefixInstance{ID, D, N, F, PrefixCfg<D, N, F>::THREADS, PrefixCfg<D, N, F>::SMEM_BYTES},
const PrefixInstance kPrefixInstances[] = {PD_FOR_EACH_PREFIX(PD_PREFIX_ROW)};
#undef PD_PREFIX_ROW
const int kNumPrefixInstances = sizeof(kPrefixInstances) / sizeof(kPrefixInstances[0]);

const void* prefix_kernel_ptr(int variant) {
  switch (variant) {
#define PD_PREFIX_CASE(ID, D, N, F) \
  case ID:                          \
    return reinterpret_cast<const void*>(&prefix_kernel<PrefixCfg<D, N, F>>);
    PD_FOR_EACH_PREFIX(PD_PREFIX_CASE)
#undef PD_PREFIX_CASE
    default:
      return nullptr;
  }
}

}  // namespace pd
