// Decode over a 4-bit (e2m1 codes, e4m3 block scales) cache: instances and
// launch geometry, shared by the host planner and the kernel.
#pragma once

#include <cstdint>

#include "pd_kernels.h"

namespace pd {

constexpr int kFp4Block = 16;    // dims under one scale
constexpr int kFp4Tile = 128;    // tokens of a tile: the matrix instruction's rows
constexpr int kFp4Terms = 6;     // e2m1 terms a query element is written as
constexpr int kFp4FirstId = 60;  // variant ids follow stage 1's
// Workspace: [error word][a byte per share: pieces of its last unit that are there][free]
// [fp32 log-sum-exps [shares][2][CC]][fp32 pieces [shares][2][CC][D]]
// The counts have to be zero between launches, whatever plans take the workspace in
// turn: they lie in the 256-byte header, of which other plans write the error word
// alone, and no plan's pieces.
constexpr int kFp4MaxShares = (kWorkspaceHeader - 4) / 4 * 4;  // CTAs of a launch, so the most pieces of a unit
static_assert(kFp4MaxShares <= 255, "a count is a byte");
constexpr uint64_t fp4_parts_offset(int shares) { return kWorkspaceHeader + ((uint64_t)shares * 4 + 255) / 256 * 256; }

// D   head_dim; KVS K=V shared pool; CC columns (query rows) of a CTA
template <int D_, bool KVS_, int CC_>
struct Fp4Cfg {
  static constexpr int D = D_, CC = CC_;
  static constexpr bool KVS = KVS_;
  static constexpr int SL = D / 256;       // 128-byte slabs of a row's codes
  static constexpr int KSTEPS = D / 64;    // 64-dim steps of the matrix instruction
  static constexpr int N = (CC * kFp4Terms + 15) / 16 * 16;  // its columns
  static constexpr int ROW_SF = D / kFp4Block;               // scale bytes of a row
  // one tile of K or V: codes [8-row group][slab][8 rows][128 B, swizzled], then scales [128][D / 16]
  static constexpr int CODE_BYTES = kFp4Tile * D / 2;
  static constexpr int SF_BYTES = kFp4Tile * ROW_SF;
  static constexpr int ITEM_BYTES = CODE_BYTES + SF_BYTES;
  // K != V: a ring for K (a tile is done with once its scores are computed) and
  // one for V, at d 512 a longer one (windows of 1024 at d 256: 4 and 6 43.1 us, 5 and 5 39.3)
  static constexpr int NK = KVS ? (D == 512 ? 5 : 10) : (D == 512 ? 2 : 5);
  static constexpr int NV = KVS ? 0 : (D == 512 ? 3 : 5);
  static constexpr int RING_BYTES = (NK + NV) * ITEM_BYTES;
  // Segments told of at a time. Copies run ahead by a ring's tiles, which may be of as
  // many segments, of one more to come, and of up to 3 whose results are not out yet.
  static constexpr int SEGS = D == 256 ? 32 : 16;
  static constexpr int CHUNKS = D / 128;   // of 128 dims: V is widened and summed a chunk at a time
  static constexpr int Q_BYTES = N * D / 2;                       // a query's terms: codes like a tile's
  static constexpr int Q_OFFSET = RING_BYTES;                     // [2]: of this segment and the next
  static constexpr int P_BYTES = 8 * kFp4Tile * 4;                // P, tf32: [32 tokens][8 columns][128 B, swizzled]
  static constexpr int P_OFFSET = Q_OFFSET + 2 * Q_BYTES;         // [2]
  static constexpr int EYE_OFFSET = P_OFFSET + 2 * P_BYTES;       // the unit matrix in e2m1: 128 rows of 64 B, swizzled
  static constexpr int EYE_BYTES = 128 * 64;
  static constexpr int QSF_OFFSET = EYE_OFFSET + EYE_BYTES;       // query terms' scales [N][D / 16]
  static constexpr int COL_OFFSET = QSF_OFFSET + N * ROW_SF;      // float [2][CC]: score scale of a column
  static constexpr int POISON_OFFSET = COL_OFFSET + 2 * CC * 4;   // u32 [SEGS][CC]: 16-dim blocks that are NaN
  static constexpr int TOP_OFFSET = POISON_OFFSET + SEGS * CC * 4; // float [4][CC]: the softmax warps' maxima
  static constexpr int SUM_OFFSET = TOP_OFFSET + 4 * CC * 4;      // float [2][5][CC]: their sums, and the references
  static constexpr int MISC_OFFSET = SUM_OFFSET + 2 * 5 * CC * 4; // u32: the join's ticket
  static constexpr int BLOCKS_OFFSET = MISC_OFFSET + 4;           // u32: the 16-token blocks that the scores' tile holds
  static constexpr int TILE_OFFSET = BLOCKS_OFFSET + 4;           // u32 [2]: of P's tiles
  static constexpr int BEGIN_OFFSET = TILE_OFFSET + 8;            // int [64]: where the share begins
  static constexpr int SEG_OFFSET = (BEGIN_OFFSET + 256 + 15) / 16 * 16;  // [SEGS] of 64 bytes
  static constexpr int VALID_OFFSET = SEG_OFFSET + SEGS * 64;          // u32 [NK + NV]: what a slot's tile is (kTile...)
  static constexpr int BAR_OFFSET = (VALID_OFFSET + (NK + NV) * 4 + 7) / 8 * 8;
  static constexpr int NUM_BARS = 3 * (NK + NV) + 19 + SEGS;
  static constexpr int SMEM_BYTES = BAR_OFFSET + NUM_BARS * 8 + 16 + 1024;  // (+ 1 KiB to start on a 1024-byte boundary)
  // d 512 has the longer products, d 256 more copies for them
  static constexpr int SCALE_WARPS = D == 256 ? 2 : 1, LANES = D == 256 ? 1 : 2;
  static constexpr int WARPS = 15 + SCALE_WARPS + 2 * LANES;
  static constexpr int THREADS = 32 * WARPS;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(Q_OFFSET % 1024 == 0 && Q_BYTES % 1024 == 0 && P_OFFSET % 1024 == 0 && EYE_OFFSET % 1024 == 0 &&
                    QSF_OFFSET % 16 == 0,
                "alignment");
};

// X(id, head_dim, K=V, columns)
#define PD_FOR_EACH_FP4(X)  \
  X(60, 512, false, 4)      \
  X(61, 512, false, 8)      \
  X(62, 512, true, 4)       \
  X(63, 512, true, 8)       \
  X(64, 256, false, 4)      \
  X(65, 256, false, 8)      \
  X(66, 256, true, 4)       \
  X(67, 256, true, 8)

struct Fp4Params {
  CUtensorMap kmap, vmap;  // codes as {128 B, 8 rows, slabs, 8-row groups}
  const uint16_t* q;       // bf16 [B, T, Hq, D]
  const uint8_t *k_sf, *v_sf;  // e4m3 [num_pages, Hkv, P, D / 16]
  const int32_t *block_tables, *seq_lens;
  void* out;
  uint32_t* counters;  // a byte a share, zero between launches
  float *lse_part, *o_part;
  uint32_t* err;
  float scale_log2;  // softmax scale * log2(e) * 2^k_exp
  float v_mul;       // 2^v_exp
  int32_t stall_bytes, early_kv;
  int32_t batch, window, num_pages, max_pages, page_size, num_q_heads, num_kv_heads;
  int32_t query_tokens, group, col_tiles;
  int32_t units;  // of a request: KV heads x column tiles
  int32_t cap;    // tokens a block table's row holds
};

const void* fp4_kernel_ptr(int variant);

}  // namespace pd
