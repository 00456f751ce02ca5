// The prefix pass of shared-prefix decode (sm_103a): attention of all of a
// group's query rows over its prefix, every prefix byte fetched once per row
// tile.
//
// Mathematics, for one (piece of the prefix, KV head, tile of N query rows),
// a tile of tokens at a time, with the query rows on the N side of both products:
//   S^T[tokens x N] = K[tokens x d] . q^T          (tokens on the M side)
//   P^T             = 2^(S^T scale log2 e - ref)   ref: each row's reference
//   O^T[d x N]     += V^T[d x tokens] . P^T        (head dims on the M side, 128 at a time)
// A query row is a column of both accumulators, so N = 16 rows cost what they
// need and d = 512 leaves room in tensor memory. The sum of a row's
// probabilities is kept per token lane in registers and reduced once at the end.
//
// References: any reference in range gives the same quotient, and fp32 sums and
// bf16 operands lose nothing while scores stay below 2^60 over it (FP8's f16
// operands: 2^12). So a row keeps the maximum of the tile that set its
// reference until a score leaves that range. The tile's P is then not used:
// the rows that left take the tile's true maximum, their sums and O^T are
// rescaled, and P is written again. The matrix warp, which sees every P before
// its product, says which, so the softmax warps need no barrier of their
// own per tile. Each row's references depend on its own scores only.
// FP8: an operand is a probability times its page's V scale (over the piece's
// largest), and that product is what has to stay in f16's range, so references
// and range go by a token's score plus the log2 of its scale: a row whose
// weight lies on pages of small scales keeps f16's precision there. (With the
// scores alone, a peak on a page of 10^-6 of the largest scale sat at f16's
// smallest steps, 3% each, and one of 10^-8 vanished.)
//
// One CTA (CT = 1): tiles of 128 tokens, N <= 64 at d = 512 (O^T takes 4 N
// columns of tensor memory, S^T two buffers of N), 128 below. There the matrix
// instruction is bound by its A operand (M = 128, N = 64: 55 cycles against 64
// at N = 128) and the SM by the bytes it takes in. A pair of CTAs (CT = 2, d =
// 512, 128 rows): tiles of 256 tokens, each CTA the scores of its 128 tokens
// and half of the head dims; every byte of K and V then serves twice the rows
// per SM. The token lanes' probabilities of rows 64 wg .. + 63 go to the CTA of
// rank wg, which holds that half of the B operand.
//
// Roles: warps 0-7 softmax and epilogue (a thread per token lane, two
// warpgroups with half the rows each), warp 8 the matrix instructions, warps
// 9-11 the copies (a third of every stage's each: a lane's copies go out ~70
// cycles apart); FP8: warps 12-15 (up to 32 rows: 12-19) widen the e4m3 stages to f16
// operands. K and V arrive
// as [8-token group][64-dim slab][8][128 B] atoms with the 128-byte swizzle:
// K-major for the first product, and the same layout read M-major for the
// second, so nothing is transposed; P is written N-major, a token's row at a
// time. A K=V layer fetches the tile again for its second use (an L2 hit).
//
// What bounds it, at head_dim 512 (one GB300, the whole call over the tiles of
// its longest CTA): a pair's tile of 256 tokens takes 3.4 us with few pairs and
// 3.9 with 64, 2.15 us of it the products and most of the rest, by elimination,
// the copies' latency over a ring of half a tile's bytes (128 of 224 KB: the query
// rows take 64, P 32; L2's slices deliver 24% of their peak over a launch of 64
// requests and 16384 tokens); one CTA's tile of 128 tokens 2.8 us with 64 rows, 2.3 with 16, and
// 4 with 116 CTAs, which together take 6.1 TB/s; FP8 5.6 us (pair), 3.8 (64
// rows), 3.25 (16): the widening's passes through shared memory. What a refused
// tile costs shows with e4m3's range: 32 requests over 32768 tokens 71 us with
// scores of deviation 1.5 (nats), 130 with 3, 183 with 4, 181 with 12 (16
// requests 52, 65, 87, 93; bf16, 32 requests: 71, 73, 73, 87).
//
// Roundings: P to the operands' type. bf16 cache: bf16, 2^-9 a probability. FP8
// cache: f16, into which e4m3 widens exactly; q rounds to f16 once (as in the
// decode), and P carries the page's V scale over the piece's largest: 2^-12 a
// probability, and below 2^-14 of the row's largest product of probability and
// V scale 2^-25 of that (scales below 2^-32 of the piece's largest count as
// 2^-32 there). Sums, references and accumulators stay in fp32.
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
constexpr int kCopyWarps = 3;              // warps 9..11 (12, 16 or 20 warps leave 168, 128 or 96 registers a thread)
constexpr int kSoftWarps = 8;
constexpr float kLow = 3e38f;              // negated reference of a row without a score yet
constexpr int kNoTop = (int)0x807fffff;    // ordered(-inf)
constexpr float kLeastScale = -32.f;       // log2: a probability may then exceed 1 by 2^44, and sums hold that

template <int D_, int N_, bool FP8_, int CT_>
struct PrefixCfg {
  static constexpr int D = D_, N = N_, CT = CT_;
  static constexpr bool FP8 = FP8_;
  static constexpr float SLACK = FP8 ? 12.f : 60.f;  // log2 of what a probability may exceed 1 by
  static constexpr int TT = kTok * CT;     // tokens of a tile
  static constexpr int KS = D / 128;       // stages of a tile's K (and of its V) in a CTA
  static constexpr int VT = TT / KS;       // tokens of a V stage
  static constexpr int MC = D / 128 / CT;  // 128-dim chunks of O^T in a CTA
  static constexpr int V_ATOMS = D / 64 / CT;  // 64-dim slabs of V in a CTA
  static constexpr int QN = N / CT;        // query rows whose operands a CTA holds
  static constexpr int Q_BYTES = QN * D * 2, P_BYTES = QN * TT * 2;
  static constexpr int ROOM = kBody - Q_BYTES - P_BYTES;
  // FP8: two operand stages (one filled while the other is used), the rest for
  // copies in flight: with three, and so 2 raw stages a pair, copies bound it
  static constexpr int NST = FP8 ? 2 : (ROOM / kStage < 6 ? ROOM / kStage : 6);
  static constexpr int NRAW_FIT = (ROOM - NST * kStage) / kRaw < 8 ? (ROOM - NST * kStage) / kRaw : 8;
  // teams of four widening warps, each with every other stage (of an even
  // ring); the rows of a large tile leave registers for one
  static constexpr int TEAMS = N <= 32 ? 2 : 1;
  static constexpr int NRAW = FP8 ? NRAW_FIT / TEAMS * TEAMS : 0;
  static constexpr int Q_OFFSET = 0, P_OFFSET = Q_BYTES, RING_OFFSET = P_OFFSET + P_BYTES;
  static constexpr int RAW_OFFSET = RING_OFFSET + NST * kStage;
  static constexpr int REF_OFFSET = RAW_OFFSET + NRAW * kRaw;   // float nref[N]: negated references
  static constexpr int TOP_OFFSET = REF_OFFSET + N * 4;         // int top[N]: a tile's true maxima
  static constexpr int ROW_OFFSET = TOP_OFFSET + N * 4;         // int row[N]: a tile row's row of q and out
  static constexpr int BAR_OFFSET = ROW_OFFSET + N * 4;
  static constexpr int NBAR = 2 * NST + 2 * NRAW + 12;
  static constexpr int TMEM_OFFSET = (BAR_OFFSET + NBAR * 8 + 15) / 16 * 16;  // tensor memory address, redo, peer, -, left[8]
  static constexpr int SMEM_BYTES = TMEM_OFFSET + 48 + 1024;
  // pair: what a CTA's P takes from the other CTA a round: 128 tokens' rows, and its warps' flags
  static constexpr int P_TX = kTok * QN * 2 + 16;
  static constexpr int THREADS = 32 * (kSoftWarps + 1 + kCopyWarps + (FP8 ? 4 * TEAMS : 0));
  static constexpr int CW = N / 2;         // rows of a softmax warpgroup
  static constexpr int LD = CW < 32 ? CW : 32;
  // P: [QN / 64 blocks][TT tokens][row of up to 64 query rows], swizzled over the row
  static constexpr int P_ROW = QN >= 64 ? 128 : QN * 2;
  // after the last product, in the ring: the rows' sums (per warpgroup [128][CW + 1], [128]), then a
  // pair's sums of the other CTA's tokens [N]
  static constexpr int SUM_FLOATS = kTok * (CW + 1) + 128;
  static constexpr int TOTAL_OFFSET = RING_OFFSET + 2 * SUM_FLOATS * 4;
  static constexpr int O_COLS = MC * N;
  static constexpr int TMEM_COLS = O_COLS + 2 * N <= 64 ? 64 : O_COLS + 2 * N <= 128 ? 128 :
                                   O_COLS + 2 * N <= 256 ? 256 : 512;
  static_assert(CT == 1 || (D == 512 && N == 128), "a pair serves 128 rows at head_dim 512");
  static_assert(O_COLS + 2 * N <= 512, "tensor memory");
  static_assert(NST >= 2 && (!FP8 || NRAW >= 3), "rings");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(2 * SUM_FLOATS * 4 + N * 4 <= NST * kStage + NRAW * kRaw, "the row sums are reduced in the rings");
  static_assert(N * MC * 128 * 4 <= NST * kStage + NRAW * kRaw, "the partial rows leave through the rings");
};

struct Tile {
  int group, first, rows, start, len;
};

// Row tile z of the launch: its group, first row, rows and prefix length (group
// -1: none). Every warp finds it by itself, 32 groups at a time.
template <int N>
__device__ __forceinline__ Tile find_tile(const SharedParams& p, int z) {
  const int lane = threadIdx.x & 31, per_req = p.query_tokens * p.group;
  int at = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
    const int g = g0 + lane;
    int s = 0, rows = 0, len = 0;
    if (g < p.num_groups) {
      const int a = __ldg(p.group_starts + g), b = __ldg(p.group_starts + g + 1);
      len = __ldg(p.prefix_lens + g);
      s = max(0, min(a, p.batch));
      rows = (max(s, min(b, p.batch)) - s) * per_req;
    }
    const int n = (rows + N - 1) / N;
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
      t.first = (z - __shfl_sync(kFullMask, end - n, src)) * N;
      t.rows = min(N, __shfl_sync(kFullMask, rows, src) - t.first);
      t.start = __shfl_sync(kFullMask, s, src);
      t.len = __shfl_sync(kFullMask, len, src);
      return t;
    }
    at = __shfl_sync(kFullMask, end, 31);
  }
  return Tile{-1, 0, 0, 0, 0};
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

// A lane's tokens, one every TT of the piece: the entry of the page table and
// the place in that page, without a division a tile. left: tokens still to come.
template <int TT>
struct Walk {
  int index, offset, left, step_index, step_offset, page_size;
  // (unsigned: a first token may lie past 2^31, and past `end`)
  __device__ __forceinline__ Walk(const Walk& step, unsigned token, unsigned end)
      : index(token / (unsigned)step.page_size),
        offset(token - index * step.page_size),
        left(token < end ? (end - token + TT - 1) / TT : 0),
        step_index(step.step_index),
        step_offset(step.step_offset),
        page_size(step.page_size) {}
  // the steps alone
  __device__ __forceinline__ explicit Walk(int page) : step_index(TT / page), page_size(page) {
    step_offset = TT - step_index * page;
  }
  __device__ __forceinline__ void next() {
    --left;
    index += step_index;
    offset += step_offset;
    if (offset >= page_size) {
      offset -= page_size;
      ++index;
    }
  }
};

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

// What a role calls the same for one CTA and for a pair.
template <int CT>
struct Sync {
  // an arrival at rank 0's barrier, behind this CTA's own writes
  static __device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    if constexpr (CT == 1) mbar_arrive(bar);
    else mbar_arrive_remote(map_smem_rank(smem_u32(bar), 0));
  }
  // a wait behind which data of the other CTA is read
  static __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if constexpr (CT == 1) return mbar_wait(bar, parity);
    else return mbar_wait_cluster(bar, parity);
  }
  // all threads' barrier, and its two halves
  static __device__ __forceinline__ void arrive() {
    if constexpr (CT == 2) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  }
  static __device__ __forceinline__ void wait_all() {
    if constexpr (CT == 1) __syncthreads();
    else cluster_wait();
  }
  static __device__ __forceinline__ void all_threads() {
    if constexpr (CT == 1) __syncthreads();
    else cluster_sync_all();
  }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) prefix_kernel(const __grid_constant__ SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int N = C::N, D = C::D, KS = C::KS, NST = C::NST, CT = C::CT, TT = C::TT, CW = C::CW, LD = C::LD;
  using S = Sync<CT>;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFFSET);  // (pair: rank 0's, for both CTAs' stages)
  uint64_t* empty = full + NST;
  uint64_t* raw_full = empty + NST;
  uint64_t* raw_empty = raw_full + C::NRAW;
  uint64_t* s_full = raw_empty + C::NRAW;  // [2]
  uint64_t* p_full = s_full + 2;           // (pair: each CTA's, for the P that it holds)
  uint64_t* p_empty = p_full + 1;
  uint64_t* q_full = p_empty + 1;          // (rank 0's)
  uint64_t* drained = q_full + 1;
  uint64_t* looked = drained + 1;          // the matrix warp has looked at the P that arrived
  uint64_t* p_peer = looked + 1;           // pair: rank 1's P is complete
  uint64_t* ref_full = p_peer + 1;         // pair, rank 1: the first references are here
  uint64_t* sums_full = ref_full + 1;      // pair: the other CTA's sums are here
  uint64_t* swapped = sums_full + 1;       // [2], one per softmax warpgroup
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::TMEM_OFFSET);
  volatile uint32_t* redo = tmem_at + 1;  // the round (P arrivals so far) that has to be written again
  volatile uint32_t* peer = tmem_at + 2;     // pair, rank 0: whether a flag of rank 1 is set
  // per softmax warp that writes into this CTA's P: a score left its row's range
  volatile uint32_t* left = tmem_at + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int rank = CT == 1 ? 0 : (int)cluster_ctarank();

  if (tid == 288) {
    prefetch_tensormap(&p.kmap);
    prefetch_tensormap(&p.vmap);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], CT * (C::FP8 ? 4 : kCopyWarps));
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NRAW; ++i) {
      mbar_init(&raw_full[i], kCopyWarps);
      mbar_init(&raw_empty[i], 4);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_full, CT == 1 ? kSoftWarps : 4 + 1);
    mbar_init(p_empty, 1);
    mbar_init(q_full, CT * kSoftWarps);
    mbar_init(drained, 1);
    mbar_init(looked, 1);
    mbar_init(p_peer, 1);
    mbar_init(ref_full, 1);
    mbar_init(sums_full, 1);
    mbar_init(&swapped[0], CT * 4);
    mbar_init(&swapped[1], CT * 4);
    *redo = 0;
    fence_barrier_init();
    if constexpr (CT == 2) {
      // the first round's bytes from the other CTA
      mbar_arrive_expect_tx(p_full, C::P_TX);
      mbar_arrive_expect_tx(sums_full, 4 * N);
      if (rank == 0) {
        mbar_arrive_expect_tx(p_peer, 4);
      } else {
        mbar_arrive_expect_tx(looked, 4);
        mbar_arrive_expect_tx(ref_full, 4 * N);
      }
    }
  }
  if (tid < N) {
    reinterpret_cast<float*>(smem + C::REF_OFFSET)[tid] = kLow;
    reinterpret_cast<int*>(smem + C::TOP_OFFSET)[tid] = kNoTop;
  }
  __syncwarp();
  if (warp == 8) tmem_alloc<CT>(tmem_at, C::TMEM_COLS);
  tmem_fence_before();
  S::arrive();
  const Walk<TT> step(p.page_size);
  // behind whatever wrote what this grid reads; the own part's stage 1 behind
  // this grid may start once every thread here has waited
  grid_dependency_wait();
  grid_launch_dependents();
  const int piece = blockIdx.y, g = blockIdx.z;
  const Tile t = find_tile<N>(p, blockIdx.x / CT);
  S::wait_all();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  if (blockIdx.x == 0 && piece == 0 && g == 0 && warp == 0 && !groups_ok(p) && lane == 0)
    atomicOr(p.err, kErrBadGroup);
  int L = t.len;
  if (t.group >= 0) {
    const int cap = p.max_prefix_pages * p.page_size;
    const int cut = max(0, min(L, cap)) / p.page_size * p.page_size;
    if (L != cut) {
      if (tid == 0) atomicOr(p.err, kErrBadSeqLen);
      L = cut;
    }
  }
  // this piece's tokens [lo, hi); the last piece takes whatever remains
  const long long want = (long long)piece * p.chunk_tokens;
  const int lo = (int)min(want, (long long)L);
  const int hi = piece == p.num_pieces - 1 ? L : (int)min((long long)L, want + p.chunk_tokens);
  const int ntile = (unsigned)(hi - lo + TT - 1) / TT;
  const int32_t* table = p.prefix_tables + (size_t)max(t.group, 0) * p.max_prefix_pages;
  int* rows = reinterpret_cast<int*>(smem + C::ROW_OFFSET);

  if (ntile == 0) {
    // nothing here: weight 0 (the join reads no row of such a piece)
    if (rank == 0)
      for (int r = tid; r < t.rows; r += C::THREADS)
        p.lse_part[(size_t)row_of(p, t, r, g) * p.num_pieces + piece] = -INFINITY;
    S::all_threads();
    if (warp == 8) tmem_dealloc<CT>(tmem, C::TMEM_COLS);
    return;
  }

  const int wg = (warp >> 2) & 1, lt = tid & 127, bar = 1 + wg;
  float* nref = reinterpret_cast<float*>(smem + C::REF_OFFSET) + wg * CW;
  int* top = reinterpret_cast<int*>(smem + C::TOP_OFFSET) + wg * CW;
  const uint32_t quarter = tmem + ((uint32_t)(warp & 3) << 21);
  const uint32_t o_at = quarter + wg * CW;

  if (warp >= 9 && warp < 9 + kCopyWarps) {
    // ---- copies: stages in the order the products use them, K(0), K(1), V(0), K(2), V(1), ...
    // A K stage is 128 dims of this CTA's tokens, a V stage this CTA's dims of
    // VT tokens; a 16-token page takes one copy of 4 KB (K) or 16 KB (V, d =
    // 512): with a copy per page and slab (2 KB) the copies took 5.5 us a tile.
    // Box j of a tile is lane j / 3's of copy warp j mod 3.
    // Filling a stage is on the path of the ring: everything that can be is worked
    // out before the loop or a tile ahead. (Page positions by division,
    // box numbers too, and page ids looked at where they were loaded: ~4000
    // cycles a tile of 7700.)
    const uint64_t policy = p.keep_in_l2 ? l2_evict_normal_policy() : l2_evict_first_policy();
    constexpr int NR = C::FP8 ? C::NRAW : NST;
    const int w = warp - 9, box = lane * kCopyWarps + w;
    constexpr int BYTES = C::FP8 ? kRaw : kStage;
    constexpr int K_SLABS = C::FP8 ? 1 : 2, V_SLABS = C::V_ATOMS / (C::FP8 ? 2 : 1);
    uint64_t* land = C::FP8 ? raw_full : full;
    uint64_t* freed = C::FP8 ? raw_empty : empty;
    uint8_t* ring = smem + (C::FP8 ? C::RAW_OFFSET : C::RING_OFFSET);
    uint32_t err = 0;
    const int k_bytes = p.k_box * 128 * K_SLABS, v_bytes = p.v_box * 128 * V_SLABS;
    const int v_boxes = C::VT / p.v_box;  // of a stage
    const int k_at = box * k_bytes, v_at = box % v_boxes * v_bytes, v_stage = box / v_boxes;
    // this lane's boxes: a tile further every time one is asked for
    Walk<TT> k_walk(step, (unsigned)lo + rank * kTok + box * p.k_box, box < kTok / p.k_box ? hi : 0);
    Walk<TT> v_walk(step, (unsigned)lo + box * p.v_box, box < TT / p.v_box ? hi : 0);
    struct Box {
      int page, offset;  // offset -1: no box
    };
    auto next_box = [&](Walk<TT>& at) -> Box {
      Box b{0, -1};
      if (at.left > 0) b = {__ldg(table + at.index), at.offset};
      at.next();
      return b;
    };
    // the 8-row group of the pool where a box starts (-1: none); a page outside
    // the pool is fetched past the pool's end, which reads zeros
    const int page_groups = p.num_kv_heads * (p.page_size / 8), head_group = g * (p.page_size / 8);
    auto group_of = [&](const Box& b) -> int {
      if (b.offset < 0) return -1;
      if ((unsigned)b.page >= (unsigned)p.num_pages) {
        err |= kErrBadPage;
        return p.num_pages * page_groups;
      }
      return b.page * page_groups + head_group + b.offset / 8;
    };
    // the next stage's number and place, and the phase of its release (the first
    // round waits for nothing)
    int use = 0, st = 0;
    uint32_t phase = 1;
    bool ok = true;
    auto begin = [&](int boxes, int box_bytes) {
      ok = __all_sync(kFullMask, use < NR || mbar_wait(&freed[st], phase));
      if (ok && lane == 0) {
        const uint32_t bytes = boxes * box_bytes + (w == 0 ? p.stall_bytes : 0);
        if (CT == 1 || C::FP8) mbar_arrive_expect_tx(&land[st], bytes);
        else mbar_arrive_expect_tx_remote(map_smem_rank(smem_u32(&land[st]), 0), bytes);
      }
      __syncwarp();
      return ok;
    };
    auto copy = [&](int at_byte, const CUtensorMap* map, int slab, int group) {
      uint8_t* dst = ring + st * BYTES + at_byte;
      if (CT == 1 || C::FP8) tma_load_4d(dst, map, 0, 0, slab, group, &land[st], policy);
      else tma_load_4d_pair(dst, map, 0, 0, slab, group, map_smem_rank(smem_u32(&land[st]), 0), policy);
    };
    auto end = [&] {
      ++use;
      if (++st == NR) {
        st = 0;
        phase ^= 1;
      }
    };
    auto load_k = [&](int at) {
      const int boxes = __popc(__ballot_sync(kFullMask, at >= 0));
#pragma unroll 1
      for (int s = 0; s < KS; ++s) {
        if (!begin(boxes, k_bytes)) return;
        if (at >= 0) copy(k_at, &p.kmap, s * K_SLABS, at);
        end();
      }
    };
    auto load_v = [&](int at) {
#pragma unroll 1
      for (int s = 0; s < KS; ++s) {
        const bool mine = at >= 0 && v_stage == s;
        if (!begin(__popc(__ballot_sync(kFullMask, mine)), v_bytes)) return;
        if (mine) copy(v_at, &p.vmap, rank * V_SLABS, at);
        end();
      }
    };
    const Box k_first = next_box(k_walk);
    Box k_box = next_box(k_walk), v_box = next_box(v_walk);
    load_k(group_of(k_first));
#pragma unroll 1
    for (int i = 0; i < ntile && ok; ++i) {
      const Box k_after = next_box(k_walk), v_after = next_box(v_walk);
      if (i + 1 < ntile) load_k(group_of(k_box));
      if (ok) load_v(group_of(v_box));
      k_box = k_after;
      v_box = v_after;
    }
    // no copy may still be landing when the CTA exits (a pair's land on rank
    // 0's barriers: it waits for both, and the CTAs leave together)
    if (lane == 0) {
      const unsigned long long deadline = global_timer_ns() + kWaitTimeoutNs;
      if (w == 0 && (CT == 1 || C::FP8 || rank == 0))
        for (int n = ok ? 2 * KS * ntile : use, k = max(0, n - NR); k < n; ++k)
          if (!mbar_wait_until(&land[k % NR], (k / NR) & 1, deadline)) ok = false;
      if (!ok) err |= kErrTimeout;
    }
    err = __reduce_or_sync(kFullMask, err);
    if (lane == 0 && err) atomicOr(p.err, err);
  } else if (warp == 8) {
    // ---- matrix instructions (rank 0 for both CTAs of a pair): QK(0), then
    // QK(i + 1) ahead of PV(i). One elected lane walks the stages, two at a time:
    // the tensor core holds little of what is issued ahead, so each look at a
    // barrier leaves it idle (a stage of 8 instructions: 48 cycles each without,
    // 59 with one lane's look, 70 where the warp votes).
    constexpr uint32_t kQk = mma_desc_16bit(!C::FP8, TT, N, false, false);
    constexpr uint32_t kPv = mma_desc_16bit(!C::FP8, TT, N, true, true);
    if (rank == 0 && elect_one()) {
      // descriptors' bases; a step further is a constant added to the address field
      const uint32_t base = smem_u32(smem);
      const uint64_t k_desc = smem_desc(base + C::RING_OFFSET, 16, 2048), q_desc = smem_desc(base, 16, 1024);
      const uint64_t v_desc = smem_desc(base + C::RING_OFFSET, 1024, C::V_ATOMS * 1024);
      const uint64_t p_desc = smem_desc(base + C::P_OFFSET, TT * 128, 8 * C::P_ROW, C::P_ROW);
      int st = 0;
      uint32_t phase = 0, rounds = 0;
      bool ok = mbar_wait_cluster(q_full, 0);
      auto next_stage = [&] {
        if (++st == NST) {
          st = 0;
          phase ^= 1;
        }
      };
      // the next stage is there; a look at its barrier is one at the next's, too
      uint32_t ahead = 0;
      auto landed = [&] {
        if (ahead != 0) {
          ahead = 0;
          return true;
        }
        const int st2 = st + 1 == NST ? 0 : st + 1;
        const uint32_t x = mbar_test(&full[st], phase), y = mbar_test(&full[st2], st2 == 0 ? phase ^ 1 : phase);
        ahead = x & y;
        return x != 0 || mbar_wait(&full[st], phase);
      };
      // the other S buffer is free once P of the tile before last was accepted
      auto qk = [&](int i) {
        const uint32_t d = tmem + C::O_COLS + (i & 1) * N;
#pragma unroll 1
        for (int s = 0; s < KS && ok; ++s) {
          ok = landed();
          if (!ok) return;
          const uint64_t a = k_desc + st * (kStage >> 4), b = q_desc + s * 2 * (C::QN * 128 >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss<CT>(d, a + (k >> 2) * (1024 >> 4) + (k & 3) * 2, b + (k >> 2) * (C::QN * 128 >> 4) + (k & 3) * 2,
                       kQk, k != 0 || s != 0);
          mma_commit<CT>(&empty[st]);
          next_stage();
        }
        mma_commit<CT>(&s_full[i & 1]);
      };
      qk(0);
#pragma unroll 1
      for (int i = 0; i < ntile && ok; ++i) {
        if (i + 1 < ntile) qk(i + 1);
        bool refused = true;
        while (ok && refused) {
          ok = S::wait(p_full, rounds & 1) && (CT == 1 || S::wait(p_peer, rounds & 1));
          ++rounds;
          if (!ok) break;
          const uint4 fa = lds128(tmem_at + 4), fb = lds128(tmem_at + 8);
          refused = (fa.x | fa.y | fa.z | fa.w | fb.x | fb.y | fb.z | fb.w) != 0;
          // a refused P is written again, under references that hold
          if constexpr (CT == 2) {
            refused = refused || *peer != 0;
            fence_proxy_async_smem();  // the rows from the other CTA
            if (refused) *redo = rounds;
            mbar_arrive_expect_tx(p_full, C::P_TX);
            mbar_arrive_expect_tx(p_peer, 4);
            st_async_u32(map_smem_rank(smem_u32(tmem_at + 1), 1), refused ? rounds : 0,
                         map_smem_rank(smem_u32(looked), 1));
          } else {
            if (refused) *redo = rounds;
          }
          mbar_arrive(looked);
        }
        tmem_fence_after();
        const int steps = min(TT, hi - lo - i * TT) / 16;
#pragma unroll 1
        for (int s = 0; s < KS && ok; ++s) {
          ok = landed();
          if (!ok) break;
          // 16 tokens at a time, all of the CTA's head dims
          const uint64_t a = v_desc + st * (kStage >> 4), b = p_desc + s * (C::VT * C::P_ROW >> 4);
          const bool first = i == 0 && s == 0;
          auto step = [&](int k, int m) {
            mma_ss<CT>(tmem + m * N, a + k * (C::V_ATOMS * 2048 >> 4) + m * (2048 >> 4),
                       b + k * (16 * C::P_ROW >> 4), kPv, !first || k != 0);
          };
          if ((s + 1) * (C::VT / 16) <= steps) {
#pragma unroll
            for (int k = 0; k < C::VT / 16; ++k)
#pragma unroll
              for (int m = 0; m < C::MC; ++m) step(k, m);
          } else {
#pragma unroll 1
            for (int k = 0; s * (C::VT / 16) + k < steps; ++k)
#pragma unroll 1
              for (int m = 0; m < C::MC; ++m) step(k, m);
          }
          mma_commit<CT>(&empty[st]);
          next_stage();
        }
        if (ok) mma_commit<CT>(p_empty);
      }
      if (!ok) {
        // nothing may still be reading shared memory when the CTA exits
        mma_commit<CT>(drained);
        mbar_wait(drained, 0);
        atomicOr(p.err, kErrTimeout);
      }
    } else if (rank == 1 && elect_one()) {
      // tells rank 0 of each P that is complete here, and takes its answer
      uint32_t rounds = 0;
      bool ok = true;
      for (int accepted = 0; accepted < ntile;) {
        ok = S::wait(p_full, rounds & 1);
        if (!ok) break;
        const uint4 fa = lds128(tmem_at + 4), fb = lds128(tmem_at + 8);
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(p_full, C::P_TX);
        st_async_u32(map_smem_rank(smem_u32(tmem_at + 2), 0), fa.x | fa.y | fa.z | fa.w | fb.x | fb.y | fb.z | fb.w,
                     map_smem_rank(smem_u32(p_peer), 0));
        ok = S::wait(looked, rounds & 1);
        if (!ok) break;
        ++rounds;
        if (*redo != rounds) ++accepted;
        mbar_arrive_expect_tx(looked, 4);
      }
      if (!ok) atomicOr(p.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ---- softmax: a thread per token lane, warpgroup wg the rows [wg CW, wg CW + CW)
    if (tid < N) rows[tid] = tid < t.rows ? row_of(p, t, tid, g) : -1;
    __syncwarp();
    named_bar_sync(3, 256);
    // this CTA's query rows, swizzled as the K-major operand; all of a round's loads in flight at once
    constexpr int kChunks = C::QN * (D / 8), kRound = kChunks / 256 < 16 ? kChunks / 256 : 16;
#pragma unroll 1
    for (int e0 = tid; e0 < kChunks; e0 += 256 * kRound) {
      uint4 v[kRound];
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        const int e = e0 + u * 256, r = rows[rank * C::QN + e / (D / 8)];
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= 0) v[u] = __ldg(reinterpret_cast<const uint4*>(p.q + (size_t)r * D) + e % (D / 8));
      }
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        const int e = e0 + u * 256, r = e / (D / 8), c = e % (D / 8);
        if constexpr (C::FP8)
          v[u] = make_uint4(to_f16x2(v[u].x), to_f16x2(v[u].y), to_f16x2(v[u].z), to_f16x2(v[u].w));
        *reinterpret_cast<uint4*>(smem + C::Q_OFFSET + (c >> 3) * C::QN * 128 + r * 128 +
                                  (((c & 7) ^ (r & 7)) << 4)) = v[u];
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) S::arrive_leader(q_full);

    float v_inv = 1.f, v_top = 1.f;  // FP8: the piece's largest V scale
    if constexpr (C::FP8) {
      float m = 0.f;
      // (unsigned: the step behind the last token may pass 31 bits)
      for (unsigned tok = (unsigned)lo + lt * 16; tok < (unsigned)hi; tok += 128 * 16) {
        const int page = __ldg(table + tok / (unsigned)p.page_size);
        if ((unsigned)page < (unsigned)p.num_pages)
          m = fmaxf(m, fabsf(__ldg(p.v_scale + (size_t)page * p.num_kv_heads + g)));
      }
      const int k = __reduce_max_sync(kFullMask, __float_as_int(m));
      // (exchanged where the maxima of refused tiles go: the other CTA writes there only after this one's first P)
      if (lane == 0) top[warp & 3] = k;
      __syncwarp();
      named_bar_sync(bar, 128);
      v_top = __int_as_float(max(max(top[0], top[1]), max(top[2], top[3])));
      // (a subnormal one's reciprocal would be infinite: the smallest normal number serves below it, and for zero)
      v_top = fmaxf(v_top, 0x1p-126f);
      v_inv = 1.f / v_top;
      named_bar_sync(bar, 128);
      if (lt < 4) top[lt] = kNoTop;
      __syncwarp();
    }

    float l[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) l[c] = 0.f;
    uint32_t err = 0, round = 0;
    bool ok = true;
    // A lane's token of a tile: whether it is attended, its scales. The page id
    // is loaded a tile before it is looked at, and FP8's scales a tile before use.
    struct Token {
      bool valid;
      float sc, pv;
    };
    Walk<TT> walk(step, (unsigned)lo + rank * kTok + lt, hi);
    const int lane_tiles = walk.left;  // tiles that have a token of this lane
    auto next_page = [&]() -> int {
      const int page = walk.left > 0 ? __ldg(table + walk.index) : 0;
      walk.next();
      return page;
    };
    auto token = [&](int i, int page) -> Token {
      Token k{false, C::FP8 ? 0.f : p.scale_log2, C::FP8 ? 0.f : v_inv};
      if (i < lane_tiles) {
        k.valid = (unsigned)page < (unsigned)p.num_pages;
        if (!k.valid) err |= kErrBadPage;
        if constexpr (C::FP8) {
          if (k.valid) {
            k.sc = __ldg(p.k_scale + (size_t)page * p.num_kv_heads + g);
            k.pv = __ldg(p.v_scale + (size_t)page * p.num_kv_heads + g);
          }
        }
      }
      return k;
    };
    auto scaled = [&](Token k) -> Token {
      if constexpr (C::FP8) {
        k.sc *= p.scale_log2;
        k.pv *= v_inv;
      }
      return k;
    };
    // What a row's reference goes by: the token's score, FP8 with its V scale's log2 (worked out where it is needed:
    // a register the less).
    auto weight = [&](const Token& k) { return C::FP8 ? fminf(fmaxf(__log2f(fabsf(k.pv)), kLeastScale), 0.f) : 0.f; };
    auto level = [&](uint32_t x, const Token& k) -> int {
      const float s = __uint_as_float(x) * k.sc;
      return ordered(!k.valid ? -INFINITY : C::FP8 ? s + weight(k) : s);
    };
    // P: this token's row, in the CTA that holds these query rows; its 16-byte chunks swizzled over the row
    constexpr int kChunkMask = C::P_ROW / 16 - 1, kSwShift = C::QN >= 64 ? 0 : C::QN == 32 ? 1 : 2;
    const int p_tok = rank * kTok + lt;
    const uint32_t p_row = smem_u32(smem + C::P_OFFSET) + p_tok * C::P_ROW +
                           (CT == 1 && N == 128 ? wg * (TT * 128) : 0);
    const bool here = CT == 1 || wg == rank;  // this CTA holds the rows' P
    const uint32_t p_remote = CT == 2 ? map_smem_rank(p_row, wg) : p_row;
    const uint32_t p_bar = CT == 2 ? map_smem_rank(smem_u32(p_full), wg) : 0;
    const int p_sw = (p_tok >> kSwShift) & kChunkMask, p_chunk = CT == 2 || N == 128 ? 0 : wg * (CW / 8);
    // two rows' probabilities of this token, packed; sums kept when `add`
    auto prob = [&](const uint32_t (&x)[LD], int c0, int c, const Token& k, bool all, bool add, float& over) {
      float e[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float y = fmaf(__uint_as_float(x[c + u]), k.sc, nref[c0 + c + u]);
        over = fmaxf(over, y);
        e[u] = ex2(y);
        if (!all && !k.valid) e[u] = 0.f;
        if (add) l[c0 + c + u] += e[u];
        if constexpr (C::FP8) e[u] = !all && !k.valid ? 0.f : e[u] * k.pv;
      }
      return pack2<C::FP8>(e[0], e[1]);
    };
    auto store = [&](uint32_t (&w)[CW / 2]) {
      if constexpr (CT == 2) {
        if (!here) {
          // To the other CTA whole 128-byte rows at a time: eight lanes transpose
          // their eight tokens' eight chunks, lane j then holds chunk j of each
          // token (lone 16-byte pieces took 4300 cycles a tile).
#pragma unroll
          for (int s = 1; s < 8; s <<= 1) {
            const bool up = (lane & s) != 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k & s) continue;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t& a = w[4 * k + q];
                uint32_t& b = w[4 * (k | s) + q];
                const uint32_t got = __shfl_xor_sync(kFullMask, up ? a : b, s);
                if (up) a = got;
                else b = got;
              }
            }
          }
          const int j = lane & 7;
          const uint32_t at = p_remote - j * C::P_ROW;  // the first of the eight tokens' rows
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_async_u32x4(at + k * C::P_ROW + ((j ^ k) << 4),
                           make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]), p_bar);
          return;
        }
      }
#pragma unroll
      for (int c = 0; c < CW / 8; ++c)
        sts128_addr(p_row + (((p_chunk + c) ^ p_sw) << 4),
                    make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
    };
    // P of a tile is complete
    auto publish = [&](bool leaves) {
      leaves = __any_sync(kFullMask, leaves);
      if (here) fence_proxy_async_smem();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (here) {
          left[CT == 1 ? warp : warp & 3] = leaves;
          mbar_arrive(p_full);
        } else {
          st_async_u32(map_smem_rank(smem_u32(tmem_at + 8 + (warp & 3)), wg), leaves, p_bar);
        }
      }
      ++round;
    };
    // Tile i's P was refused: rows that left their range take the tile's true
    // maximum (of scores, FP8 with the V scales) over both CTAs' tokens, what they hold is rescaled, P written again.
    uint32_t swaps = 0;
    auto again = [&](int i, const Token& k) {
      const uint32_t sa = quarter + C::O_COLS + (i & 1) * N + wg * CW;
      uint32_t x[LD];
#pragma unroll 1
      for (int c0 = 0; c0 < CW; c0 += LD) {
        tmem_ld(x, sa + c0);
        tmem_wait_ld();
        int mine = kNoTop;
#pragma unroll
        for (int c = 0; c < LD; ++c) {
          const int m = __reduce_max_sync(kFullMask, level(x[c], k));
          if (lane == c) mine = m;
        }
        if (lane < LD) {
          atomicMax(top + c0 + lane, mine);
          if constexpr (CT == 2) max_dsmem_s32(map_smem_rank(smem_u32(top + c0 + lane), rank ^ 1), mine);
        }
      }
      __syncwarp();
      if constexpr (CT == 2) {
        if (lane < 2) mbar_arrive_cluster(map_smem_rank(smem_u32(&swapped[wg]), lane));
        ok = mbar_wait_cluster(&swapped[wg], swaps & 1) && ok;
        ++swaps;
        __syncwarp();
      }
      named_bar_sync(bar, 128);
      auto moves = [&](int c) { return unordered(top[c]) + nref[c] > C::SLACK; };
      // factor of what a row holds; 1 where it stays
      auto factor = [&](int c) { return moves(c) ? ex2(-nref[c] - unordered(top[c])) : 1.f; };
      // a lane's sum holds this tile's probabilities already, under the old
      // reference; past 2^100 they may be infinite and all before them is
      // negligible: the probability itself, under the new one (a NaN is none of that)
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += LD) {
        tmem_ld(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < LD; ++c) {
          const int cc = c0 + c;
          const float s = __uint_as_float(x[c]) * k.sc;
          const bool far = moves(cc) && k.valid && fmaf(__uint_as_float(x[c]), k.sc, nref[cc]) > 100.f;
          l[cc] = far && !isnan(l[cc]) ? ex2(s - unordered(top[cc])) : l[cc] * factor(cc);
        }
      }
      if (i > 0) {
#pragma unroll
        for (int c0 = 0; c0 < CW; c0 += LD) {
          float f[LD];
#pragma unroll
          for (int c = 0; c < LD; ++c) f[c] = factor(c0 + c);
#pragma unroll 1
          for (int m = 0; m < C::MC; ++m) {
            tmem_ld(x, o_at + m * N + c0);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < LD; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * f[c]);
            tmem_st(o_at + m * N + c0, x);
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
      uint32_t w[CW / 2];
      float over = -INFINITY;
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += LD) {
        tmem_ld(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < LD; c += 2) w[(c0 + c) / 2] = prob(x, c0, c, k, false, false, over);
      }
      store(w);
      publish(false);
    };
    // The first references: the largest of 32 of the first tile's scores (any
    // within range do, and a refused tile costs ~15 us), by rank 0, whose warps
    // take their own tokens' for every fourth block of 8 of their group's rows
    // (the first warp for all, where the tile is short). Kept small: it runs
    // once, out of a cold instruction cache.
    auto first_refs = [&](const Token& k) {
      if (rank == 0) {
        const bool whole = hi - lo >= kTok;
        const int w = warp & 3;
#pragma unroll 1
        for (int c0 = whole ? 8 * w : w == 0 ? 0 : CW; c0 < CW; c0 += whole ? 32 : 8) {
          uint32_t x[8];
          tmem_ld(x, quarter + C::O_COLS + wg * CW + c0);
          tmem_wait_ld();
          int mine = kNoTop;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int m = __reduce_max_sync(kFullMask, level(x[c], k));
            if (lane == c) mine = m;
          }
          if (lane < 8) {
            // (no score among them, or an infinite one: left to the first look)
            const float r = fabsf(unordered(mine)) < kLow ? -unordered(mine) : kLow;
            nref[c0 + lane] = r;
            if constexpr (CT == 2)
              st_async_u32(map_smem_rank(smem_u32(nref + c0 + lane), 1), __float_as_uint(r),
                           map_smem_rank(smem_u32(ref_full), 1));
          }
          __syncwarp();
        }
        named_bar_sync(bar, 128);
      } else {
        ok = mbar_wait_cluster(ref_full, 0) && ok;
        __syncwarp();
      }
    };
    // Until tile i's P was accepted. A wait that ran out shows here, to the
    // whole warpgroup at once: its warps leave together.
    auto settle = [&](int i, const Token& k) {
      while (true) {
        ok = ok && S::wait(looked, (round - 1) & 1);
        __syncwarp();
        ok = !named_bar_or(bar, 128, !ok);
        if (!ok || *redo != round) return;
        tmem_fence_after();
        again(i, k);
      }
    };

    Token now = scaled(token(0, next_page())), before{};
    int page = next_page();
#pragma unroll 1
    for (int i = 0;; ++i) {
      const Token after = token(i + 1, page);
      page = next_page();
      if (i < ntile) ok = mbar_wait(&s_full[i & 1], (i >> 1) & 1) && ok;
      __syncwarp();
      tmem_fence_after();
      if (i > 0) {
        settle(i - 1, before);
        if (!ok || i == ntile) break;
      } else {
        first_refs(now);
      }
      const uint32_t sa = quarter + C::O_COLS + (i & 1) * N + wg * CW;
      const bool all = __all_sync(kFullMask, now.valid);
      uint32_t w[CW / 2];
      float over = -INFINITY;
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += LD) {
        uint32_t x[LD];
        tmem_ld(x, sa + c0);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < LD; c += 2) w[(c0 + c) / 2] = prob(x, c0, c, now, all, true, over);
      }
      if (i > 0) ok = mbar_wait(p_empty, (i - 1) & 1) && ok;
      __syncwarp();
      store(w);
      publish(now.valid && over > C::SLACK - weight(now));
      before = now;
      now = scaled(after);
    }
    ok = ok && mbar_wait(p_empty, (ntile - 1) & 1);
    __syncwarp();
    // ---- epilogue: the last product is done, in both CTAs of a pair
    const bool done = !named_bar_or(bar, 128, !ok);
    if (!done) err |= kErrTimeout;
    // the rows' sums over this CTA's token lanes, in the ring
    float* sum = reinterpret_cast<float*>(smem + C::RING_OFFSET) + wg * C::SUM_FLOATS;
    float* part = sum + kTok * (CW + 1);
    if (done) {
      tmem_fence_after();
#pragma unroll
      for (int c = 0; c < CW; ++c) sum[lt * (CW + 1) + c] = l[c];
    }
    named_bar_sync(bar, 128);
    if (done) {
      const int col = lt % CW, first = lt / CW * CW;
      float a[2] = {0.f, 0.f};
#pragma unroll 4
      for (int k = 0; k < CW; k += 2) {
        a[0] += sum[(first + k) * (CW + 1) + col];
        a[1] += sum[(first + k + 1) * (CW + 1) + col];
      }
      part[lt] = a[0] + a[1];
    }
    named_bar_sync(bar, 128);
    if (done && lt < CW) {
      float total = 0.f;
#pragma unroll
      for (int k = 0; k < 128 / CW; ++k) total += part[k * CW + lt];
      const int c = wg * CW + lt;
      if constexpr (CT == 2) {
        // (a cluster barrier of all threads here took ~1300 cycles)
        const float* other = reinterpret_cast<const float*>(smem + C::TOTAL_OFFSET) + c;
        st_async_u32(map_smem_rank(smem_u32(other), rank ^ 1), __float_as_uint(total),
                     map_smem_rank(smem_u32(sums_full), rank ^ 1));
        if (!mbar_wait_cluster(sums_full, 0)) err |= kErrTimeout;
        total += *other;
      }
      // no attended token: weight 0 and a zero row; NaN stays NaN
      if (rank == 0 && rows[c] >= 0)
        p.lse_part[(size_t)rows[c] * p.num_pieces + piece] =
            total == 0.f ? -INFINITY : (log2f(total) - nref[lt]) * 0.69314718055994530942f;
      nref[lt] = total == 0.f ? 0.f : v_top / total;
    }
    __syncwarp();
    named_bar_sync(3, 256);
    // The partial rows go through shared memory (the rings, idle by now), a row
    // of this CTA's dims contiguous, and out as one bulk copy each, sixteen by one
    // warp while the others go on: stored from the registers, 128 bytes a warp,
    // 128 rows took 4 us.
    constexpr int OC = CW < 16 ? CW : 16, ROW = C::MC * 128;
    float* stage = reinterpret_cast<float*>(smem + C::RING_OFFSET) + wg * CW * ROW;
    const int n = done ? min(CW, t.rows - wg * CW) : 0;
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += OC) {
      uint32_t y[C::MC][OC];
#pragma unroll
      for (int m = 0; m < C::MC; ++m) tmem_ld(y[m], o_at + m * N + c0);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < OC; ++c) {
        const float f = nref[c0 + c];
#pragma unroll
        for (int m = 0; m < C::MC; ++m) stage[(c0 + c) * ROW + m * 128 + lt] = __uint_as_float(y[m][c]) * f;
      }
      fence_proxy_async_smem();
      __syncwarp();
      named_bar_sync(bar, 128);
      const int c = c0 + lane;
      if ((warp & 3) == (c0 / OC & 3) && lane < OC && c < n)
        bulk_s2g(p.o_part + ((size_t)rows[wg * CW + c] * p.num_pieces + piece) * D + rank * ROW, stage + c * ROW, ROW * 4);
    }
    wait_bulk_stores();
    err = __reduce_or_sync(kFullMask, err);
    if (lane == 0 && err) atomicOr(p.err, err);
  } else if constexpr (C::FP8) {
    // ---- FP8: e4m3 stages widened to f16 operand stages, a thread per token row
    const int team = (warp - (kSoftWarps + 1 + kCopyWarps)) / 4;
    const int row = (tid - 32 * (kSoftWarps + 1 + kCopyWarps)) & 127, sw = row & 7, total = 2 * KS * ntile;
    static_assert(NST % C::TEAMS == 0 && C::NRAW % C::TEAMS == 0, "a stage always has the same team");
    bool ok = true;
    for (int it = team; it < total; it += C::TEAMS) {
      const int st = it % NST, rs = it % C::NRAW;
      // One CTA: the stage into registers, and released before the operand stage
      // is waited for (64 rows 4.6 -> 3.8 us a tile, 16 rows 3.5 -> 3.25; a pair
      // 5.4 -> 5.7). Not where its wait ran out (the copies into it are not
      // done), and not before the fence: without it, copies overtook the reads.
      ok = mbar_wait(&raw_full[rs], (it / C::NRAW) & 1);
      if (CT == 2 && ok && it >= NST) ok = mbar_wait(&empty[st], ((it / NST) - 1) & 1);
      if (__any_sync(kFullMask, !ok)) break;
      const uint8_t* src = smem + C::RAW_OFFSET + rs * kRaw + row * 128;
      uint8_t* dst = smem + C::RING_OFFSET + st * kStage + (row >> 3) * 2048 + (row & 7) * 128;
      auto get = [&](int c) { return *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4)); };
      auto put = [&](int c, const uint4& w) {
        uint4 a, b;
        widen4(w.x, a.x, a.y);
        widen4(w.y, a.z, a.w);
        widen4(w.z, b.x, b.y);
        widen4(w.w, b.z, b.w);
        uint8_t* to = dst + (c >> 2) * 1024;
        const int cc = (c & 3) * 2;
        *reinterpret_cast<uint4*>(to + ((cc ^ sw) << 4)) = a;
        *reinterpret_cast<uint4*>(to + (((cc + 1) ^ sw) << 4)) = b;
      };
      if constexpr (CT == 1) {
        uint4 w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = get(c);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
        if (it >= NST) ok = mbar_wait(&empty[st], ((it / NST) - 1) & 1);
        if (__any_sync(kFullMask, !ok)) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) put(c, w[c]);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) put(c, get(c));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (CT == 2) mbar_arrive(&raw_empty[rs]);
        S::arrive_leader(&full[st]);
      }
    }
    if (__any_sync(kFullMask, !ok) && lane == 0) atomicOr(p.err, kErrTimeout);
  }

  __syncwarp();
  tmem_fence_before();
  S::all_threads();
  if (warp == 8) tmem_dealloc<CT>(tmem, C::TMEM_COLS);
}

#define PD_FOR_EACH_PREFIX(X)                                                                          \
  X(0, 512, 16, false, 1) X(1, 512, 32, false, 1) X(2, 512, 64, false, 1) X(3, 256, 16, false, 1)      \
  X(4, 256, 32, false, 1) X(5, 256, 64, false, 1) X(6, 256, 128, false, 1) X(7, 128, 16, false, 1)     \
  X(8, 128, 32, false, 1) X(9, 128, 64, false, 1) X(10, 128, 128, false, 1) X(11, 512, 16, true, 1)    \
  X(12, 512, 32, true, 1) X(13, 512, 64, true, 1) X(14, 256, 16, true, 1) X(15, 256, 32, true, 1)      \
  X(16, 256, 64, true, 1) X(17, 256, 128, true, 1) X(18, 512, 128, false, 2) X(19, 512, 128, true, 2)

}  // namespace

#define PD_PREFIX_ROW(ID, D, N, F, CT) \
  PrefixInstance{ID, D, N, F, CT, PrefixCfg<D, N, F, CT>::THREADS, PrefixCfg<D, N, F, CT>::SMEM_BYTES},
const PrefixInstance kPrefixInstances[] = {PD_FOR_EACH_PREFIX(PD_PREFIX_ROW)};
#undef PD_PREFIX_ROW
const int kNumPrefixInstances = sizeof(kPrefixInstances) / sizeof(kPrefixInstances[0]);

const void* prefix_kernel_ptr(int variant) {
  switch (variant) {
#define PD_PREFIX_CASE(ID, D, N, F, CT) \
  case ID:                              \
    return reinterpret_cast<const void*>(&prefix_kernel<PrefixCfg<D, N, F, CT>>);
    PD_FOR_EACH_PREFIX(PD_PREFIX_CASE)
#undef PD_PREFIX_CASE
    default:
      return nullptr;
  }
}

}  // namespace pd
