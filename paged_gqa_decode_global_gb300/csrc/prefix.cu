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
// Roles: warps 0-3 softmax and epilogue (a thread per token lane), warp 4 the
// matrix instructions (one lane), warp 5 the copies; FP8: warps 6-9 widen the
// e4m3 stages to bf16 operands. K and V arrive as [64-dim slab][128 tokens][128
// B] with the 128-byte swizzle: K-major for the first product, and the same
// layout read M-major for the second, so nothing is transposed. A K=V layer
// fetches the tile again for its second use (an L2 hit).
//
// P is rounded to bf16 (the tensor core's operand): relative error 2^-9 a
// probability; sums, references and accumulators stay in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "shared.h"
#include "tcgen05.cuh"

namespace pd {
namespace {

constexpr int kTok = kPrefixTile;
constexpr int kSlab = kTok * 128;          // bytes of a slab: 64 bf16 dims of 128 tokens
constexpr int kStage = 2 * kSlab;          // an operand stage: 128 dims
constexpr int kRaw = kTok * 128;           // FP8: 128 dims of 128 tokens, e4m3
constexpr int kBody = 224 * 1024;          // query rows, probabilities and rings
constexpr float kSlack = 8.f;              // log2 of what a probability may exceed 1 by

template <int D_, int N_, bool FP8_>
struct PrefixCfg {
  static constexpr int D = D_, N = N_;
  static constexpr bool FP8 = FP8_;
  static constexpr int KS = D / 128;       // stages of a tile's K (and of its V)
  static constexpr int Q_BYTES = N * D * 2, P_BYTES = N * kTok * 2;
  static constexpr int ROOM = kBody - Q_BYTES - P_BYTES;
  static constexpr int NST = FP8 ? 3 : (ROOM / kStage < 6 ? ROOM / kStage : 6);
  static constexpr int NRAW = FP8 ? ((ROOM - NST * kStage) / kRaw < 6 ? (ROOM - NST * kStage) / kRaw : 6) : 0;
  static constexpr int Q_OFFSET = 0, P_OFFSET = Q_BYTES, RING_OFFSET = P_OFFSET + P_BYTES;
  static constexpr int RAW_OFFSET = RING_OFFSET + NST * kStage;
  static constexpr int REF_OFFSET = RAW_OFFSET + NRAW * kRaw;   // float ref[N]
  static constexpr int ROW_OFFSET = REF_OFFSET + N * 4;         // int row[N]: a tile row's row of q and out
  static constexpr int BAR_OFFSET = ROW_OFFSET + N * 4;
  static constexpr int NBAR = 2 * NST + 2 * NRAW + 2 + 2 + 1 + 1 + 1 + 1;
  static constexpr int TMEM_OFFSET = BAR_OFFSET + NBAR * 8;
  static constexpr int SMEM_BYTES = TMEM_OFFSET + 16 + 1024;
  static constexpr int THREADS = FP8 ? 320 : 192;
  static constexpr int O_COLS = KS * N;
  static constexpr int TMEM_COLS = O_COLS + 2 * N <= 64 ? 64 : O_COLS + 2 * N <= 128 ? 128 :
                                   O_COLS + 2 * N <= 256 ? 256 : 512;
  static_assert(O_COLS + 2 * N <= 512, "tensor memory");
  static_assert(NST >= 3 && (!FP8 || NRAW >= 2), "rings");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(kTok * (N + 1) * 4 <= NST * kStage, "the row sums are reduced in the ring");
  static_assert(5 * N * 4 <= P_BYTES, "the references are exchanged in P's buffer");
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

// Four e4m3 codes -> four bf16, exactly. A code's exponent and mantissa bits put
// at bits 4..10 of a bf16 read as the value over 2^120 (subnormal codes as bf16
// subnormals), so one exact multiplication finishes; the NaN codes (0x7f, 0xff)
// would read as 480 and are left to the caller.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = __byte_perm(w, 0u, 0x1404), y = __byte_perm(w, 0u, 0x3424);
  const uint32_t a = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u), b = ((y >> 4) & 0x07f007f0u) | (y & 0x80008000u);
  const uint32_t k = 0x7b807b80u;  // 2^120
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(k));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(k));
}
__device__ __forceinline__ bool has_nan4(uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }
__device__ __forceinline__ uint32_t nan_fix(uint32_t v, uint32_t codes) {
  if ((codes & 0x7fu) == 0x7fu) v |= 0x7fffu;
  if ((codes & 0x7f00u) == 0x7f00u) v |= 0x7fff0000u;
  return v;
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

  if (tid == 160) {
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
      mbar_init(&s_empty[i], 128);
    }
    mbar_init(p_full, 128);
    mbar_init(p_empty, 1);
    mbar_init(q_full, 128);
    mbar_init(drained, 1);
    fence_barrier_init();
  }
  if (warp == 4) tmem_alloc(tmem_at, C::TMEM_COLS);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_dependency_wait();
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
  } else if (warp == 5) {
    // ---- copies: stages in the order the products use them, K(0), K(1), V(0), K(2), V(1), ...
    const int box = p.box_rows, nbox = kTok / box;
    const uint64_t policy = p.keep_in_l2 ? 0 : l2_evict_first_policy();
    const int j = lane % nbox, slab = lane / nbox;
    constexpr int SLABS = C::FP8 ? 1 : 2;
    constexpr int NR = C::FP8 ? C::NRAW : NST;
    constexpr int BYTES = C::FP8 ? kRaw : kStage;
    uint64_t* land = C::FP8 ? raw_full : full;
    uint64_t* freed = C::FP8 ? raw_empty : empty;
    uint8_t* ring = smem + (C::FP8 ? C::RAW_OFFSET : C::RING_OFFSET);
    uint32_t err = 0;
    // the pool row of this lane's box of a tile (-1: past the piece); a page
    // outside the pool is fetched past the pool's end, which reads zeros
    auto row_at = [&](int tile) -> int {
      const int tok = lo + tile * kTok + j * box;
      if (tile >= ntile || tok >= hi || slab >= SLABS) return -1;
      const int page = __ldg(table + tok / p.page_size);
      if ((unsigned)page >= (unsigned)p.num_pages) {
        err |= kErrBadPage;
        return p.num_pages * p.num_kv_heads * p.page_size;
      }
      return (page * p.num_kv_heads + g) * p.page_size + tok % p.page_size;
    };
    int it = 0;
    bool ok = true;
    auto load = [&](int row, const CUtensorMap* map) {
      const int boxes = __popc(__ballot_sync(kFullMask, row >= 0));
      for (int s = 0; s < KS && ok; ++s, ++it) {
        const int st = it % NR;
        if (it >= NR) ok = mbar_wait(&freed[st], ((it / NR) - 1) & 1);
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&land[st], boxes * box * 128 + p.stall_bytes);
        __syncwarp();
        if (row >= 0) {
          uint8_t* dst = ring + st * BYTES + slab * kSlab + j * box * 128;
          const int dim = s * 128 + slab * 64;
          if (p.keep_in_l2)
            tma_load_2d_plain(dst, map, dim, row, &land[st]);
          else
            tma_load_2d(dst, map, dim, row, &land[st], policy);
        }
      }
    };
    int row = row_at(0), next = row_at(1);
    load(row, &p.kmap);
    for (int i = 0; i < ntile && ok; ++i) {
      const int after = row_at(i + 2);
      if (i + 1 < ntile) load(next, &p.kmap);
      if (ok) load(row, &p.vmap);
      row = next;
      next = after;
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0) {
      const unsigned long long deadline = global_timer_ns() + kWaitTimeoutNs;
      for (int k = max(0, it - NR); k < it; ++k)
        if (!mbar_wait_until(&land[k % NR], (k / NR) & 1, deadline)) ok = false;
      if (!ok) err |= kErrTimeout;
    }
    err = __reduce_or_sync(kFullMask, err);
    if (lane == 0 && err) atomicOr(p.err, err);
  } else if (warp == 4) {
    // ---- matrix instructions: QK(0), then QK(i + 1) ahead of PV(i). The warp
    // walks the stages together and one elected lane issues: a lone thread
    // computing descriptors took ~180 cycles an instruction.
    constexpr uint32_t kQk = mma_desc_bf16(128, N, false), kPv = mma_desc_bf16(128, N, true);
    // descriptors' bases; a step further is a constant added to the address field
    const uint32_t base = smem_u32(smem);
    const uint64_t k_desc = smem_desc(base + C::RING_OFFSET, 16, 1024), q_desc = smem_desc(base, 16, 1024);
    const uint64_t v_desc = smem_desc(base + C::RING_OFFSET, kSlab, 1024);
    const uint64_t p_desc = smem_desc(base + C::P_OFFSET, 16, 1024);
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
            mma_ss(d, a + (k >> 2) * (kSlab >> 4) + (k & 3) * 2, b + (k >> 2) * (N * 128 >> 4) + (k & 3) * 2, kQk,
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
      const int steps = (min(kTok, hi - lo - i * kTok)) / 16;
#pragma unroll 1
      for (int s = 0; s < KS && ok; ++s) {
        ok = __all_sync(kFullMask, mbar_wait(&full[st], phase));
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) {
          const uint64_t a = v_desc + st * (kStage >> 4);
          const uint32_t d = tmem + s * N;
          if (steps == 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ss(d, a + k * (2048 >> 4), p_desc + (k >> 2) * (N * 128 >> 4) + (k & 3) * 2, kPv, k != 0 || i != 0);
          } else {
#pragma unroll 1
            for (int k = 0; k < steps; ++k)
              mma_ss(d, a + k * (2048 >> 4), p_desc + (k >> 2) * (N * 128 >> 4) + (k & 3) * 2, kPv, k != 0 || i != 0);
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
  } else if (warp < 4) {
    // ---- softmax: a thread per token lane
    float* ref = reinterpret_cast<float*>(smem + C::REF_OFFSET);
    float* swap = reinterpret_cast<float*>(smem + C::P_OFFSET);  // [4][N] warp maxima, then [N] factors
    int* rows = reinterpret_cast<int*>(smem + C::ROW_OFFSET);
    if (tid < N) {
      ref[tid] = -INFINITY;
      rows[tid] = tid < t.rows ? row_of(p, t, tid, g) : -1;
    }
    named_bar_sync(1, 128);
    // the tile's query rows, swizzled as the K-major operand; all of a round's loads in flight at once
    constexpr int kChunks = N * (D / 8), kRound = kChunks / 128 < 16 ? kChunks / 128 : 16;
#pragma unroll 1
    for (int e0 = tid; e0 < kChunks; e0 += 128 * kRound) {
      uint4 v[kRound];
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        const int e = e0 + u * 128, r = rows[e / (D / 8)];
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= 0) v[u] = __ldg(reinterpret_cast<const uint4*>(p.q + (size_t)r * D) + e % (D / 8));
      }
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        const int e = e0 + u * 128, r = e / (D / 8), c = e % (D / 8);
        *reinterpret_cast<uint4*>(smem + C::Q_OFFSET + (c >> 3) * N * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
            v[u];
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(q_full);
    named_bar_sync(1, 128);

    const uint32_t lanes = tmem + ((uint32_t)warp << 21);
    float l[N];
#pragma unroll
    for (int c = 0; c < N; ++c) l[c] = 0.f;
    uint32_t err = 0;
    bool ok = true;
    // this lane's token of tile i: whether it is attended, its scales
    auto token = [&](int i, bool& valid, float& ks, float& vs) {
      const int tok = lo + i * kTok + tid;
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
      const uint32_t sa = lanes + C::O_COLS + (i & 1) * N;
      // does any score leave its row's range?
      float over = -INFINITY;
#pragma unroll
      for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t x[16];
        tmem_ld16(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 m = *reinterpret_cast<const float4*>(ref + c0 + c);
          over = fmaxf(over, fmaxf(fmaxf(fmaf(__uint_as_float(x[c]), sc, -m.x), fmaf(__uint_as_float(x[c + 1]), sc, -m.y)),
                                   fmaxf(fmaf(__uint_as_float(x[c + 2]), sc, -m.z), fmaf(__uint_as_float(x[c + 3]), sc, -m.w))));
        }
      }
      if (named_bar_or(1, 128, !ok || i == 0 || (valid && over > kSlack))) {
        // the rows that left theirs take the true maximum; P(i - 1) is spent
        if (i > 0) ok = mbar_wait(p_empty, (i - 1) & 1) && ok;
        __syncwarp();
        if (named_bar_or(1, 128, !ok)) break;
        tmem_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < N; c0 += 16) {
          uint32_t x[16];
          tmem_ld16(x, sa + c0);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int m = __reduce_max_sync(kFullMask, ordered(valid ? __uint_as_float(x[c]) * sc : -INFINITY));
            if (lane == c) swap[warp * N + c0 + c] = unordered(m);
          }
        }
        named_bar_sync(1, 128);
        if (tid < N) {
          const float m = fmaxf(fmaxf(swap[tid], swap[N + tid]), fmaxf(swap[2 * N + tid], swap[3 * N + tid]));
          const float was = ref[tid];
          const bool move = m > was + kSlack || was == -INFINITY;
          swap[4 * N + tid] = move && was != -INFINITY ? ex2(was - m) : 1.f;
          if (move) ref[tid] = m;
        }
        __syncwarp();
        named_bar_sync(1, 128);
#pragma unroll
        for (int c = 0; c < N; ++c) l[c] *= swap[4 * N + c];
        if (i > 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < C::O_COLS; c0 += 16) {
            uint32_t x[16];
            tmem_ld16(x, lanes + c0);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * swap[4 * N + (c0 % N) + c]);
            tmem_st16(lanes + c0, x);
          }
          tmem_wait_st();
        }
        named_bar_sync(1, 128);
      } else if (i > 0) {
        ok = mbar_wait(p_empty, (i - 1) & 1);
        __syncwarp();
      }
      // probabilities: [64-token slab][N rows][128 B], swizzled as the K-major operand
      uint8_t* pd = smem + C::P_OFFSET + (tid >> 6) * N * 128 + (tid & 7) * 2;
      const int chunk = (tid & 63) >> 3;
#pragma unroll
      for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t x[16];
        tmem_ld16(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float m = ref[c0 + c];
          // a row without a finite score yet has reference -inf: its probabilities are 2^-inf
          const float e = valid ? ex2(fmaf(__uint_as_float(x[c]), sc, m == -INFINITY ? 0.f : -m)) : 0.f;
          l[c0 + c] += e;
          const __nv_bfloat16 h = __float2bfloat16_rn(C::FP8 && valid ? e * vs : e);
          *reinterpret_cast<__nv_bfloat16*>(pd + (c0 + c) * 128 + ((chunk ^ (c & 7)) << 4)) = h;
        }
      }
      fence_proxy_async_smem();
      tmem_fence_before();
      mbar_arrive(p_full);
      mbar_arrive(&s_empty[i & 1]);
      if (!valid && lo + i * kTok + tid < hi) err |= kErrBadPage;
      valid = nvalid;
      ks = nks;
      vs = nvs;
    }
    ok = ok && mbar_wait(p_empty, (ntile - 1) & 1);
    __syncwarp();
    if (named_bar_or(1, 128, !ok)) {
      err |= kErrTimeout;
    } else {
      tmem_fence_after();
      // the rows' sums over the token lanes, in the ring (every product is done with it)
      float* sum = reinterpret_cast<float*>(smem + C::RING_OFFSET);
#pragma unroll
      for (int c = 0; c < N; ++c) sum[tid * (N + 1) + c] = l[c];
      named_bar_sync(1, 128);
      float* inv = reinterpret_cast<float*>(smem + C::P_OFFSET);
      if (tid < N) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < 128; k += 4)
#pragma unroll
          for (int u = 0; u < 4; ++u) a[u] += sum[(k + u) * (N + 1) + tid];
        const float total = (a[0] + a[1]) + (a[2] + a[3]);
        // no attended token: weight 0 and a zero row; NaN stays NaN
        inv[tid] = total == 0.f ? 0.f : 1.f / total;
        if (tid < t.rows)
          p.lse_part[(size_t)rows[tid] * p.num_pieces + piece] =
              total == 0.f ? -INFINITY : ((ref[tid] == -INFINITY ? 0.f : ref[tid]) + log2f(total)) * 0.69314718055994530942f;
      }
      __syncwarp();
      named_bar_sync(1, 128);
#pragma unroll 1
      for (int c0 = 0; c0 < N; c0 += 16) {
        if (c0 >= t.rows) break;
        uint32_t x[KS][16];
#pragma unroll
        for (int s = 0; s < KS; ++s) tmem_ld16(x[s], lanes + s * N + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (c0 + c >= t.rows) break;
          float* dst = p.o_part + ((size_t)rows[c0 + c] * p.num_pieces + piece) * D + tid;
          const float f = inv[c0 + c];
#pragma unroll
          for (int s = 0; s < KS; ++s) dst[s * 128] = __uint_as_float(x[s][c]) * f;
        }
      }
    }
    err = __reduce_or_sync(kFullMask, err);
    if (lane == 0 && err) atomicOr(p.err, err);
  } else if constexpr (C::FP8) {
    // ---- FP8: e4m3 stages widened to bf16 operand stages, a thread per token row
    const int row = tid - 192, sw = row & 7, total = 2 * KS * ntile;
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
      uint8_t* dst = smem + C::RING_OFFSET + st * kStage + row * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
        uint4 a, b;
        widen4(w.x, a.x, a.y);
        widen4(w.y, a.z, a.w);
        widen4(w.z, b.x, b.y);
        widen4(w.w, b.z, b.w);
        if (has_nan4(w.x) || has_nan4(w.y) || has_nan4(w.z) || has_nan4(w.w)) {
          a.x = nan_fix(a.x, w.x), a.y = nan_fix(a.y, w.x >> 16), a.z = nan_fix(a.z, w.y), a.w = nan_fix(a.w, w.y >> 16);
          b.x = nan_fix(b.x, w.z), b.y = nan_fix(b.y, w.z >> 16), b.z = nan_fix(b.z, w.w), b.w = nan_fix(b.w, w.w >> 16);
        }
        uint8_t* to = dst + (c >> 2) * kSlab;
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
  if (warp == 4) tmem_dealloc(tmem, C::TMEM_COLS);
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
