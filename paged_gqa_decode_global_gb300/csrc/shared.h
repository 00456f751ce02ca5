// Shared-prefix decode: what its planner, entry points and kernels share.
#pragma once

#include <cstdint>

#include "paged_decode.h"
#include "pd_kernels.h"

namespace pd {

constexpr int kPrefixTile = 128;  // prefix tokens of one tile of the prefix pass

struct SharedParams {
  // the pools as {128 bytes, 8 rows, slabs, 8-row groups}, 128-byte swizzle: a
  // box lands as [group][slab][8 rows][128 B]
  CUtensorMap kmap, vmap;
  const uint16_t* q;
  const float* k_scale;  // FP8
  const float* v_scale;
  const int32_t* prefix_tables;
  const int32_t* prefix_lens;
  const int32_t* group_starts;
  float* lse_part;  // [B*T*Hq][num_pieces]
  float* o_part;    // [B*T*Hq][num_pieces][D]
  uint32_t* err;
  float scale_log2;
  int32_t batch, num_groups, query_tokens, num_q_heads, num_kv_heads, group, head_dim;
  int32_t page_size, num_pages, max_prefix_pages;
  int32_t row_tile, tiles, num_pieces, chunk_tokens;
  int32_t k_box, v_box;  // tokens of one copy of K and of V (both divide page_size)
  int32_t keep_in_l2;   // the prefix rows may be read more than once (several row tiles or groups, K=V)
  int32_t stall_bytes;  // tests only: bytes expected per stage beyond what the copies deliver
};

// The prefix pass's kernel instances: head_dim, query rows of a row tile, cache
// type, CTAs that serve a row tile together (a cluster of two, or one).
struct PrefixInstance {
  int id, head_dim, row_tile;
  bool fp8;
  int ctas, threads, smem_bytes;
};
extern const PrefixInstance kPrefixInstances[];
extern const int kNumPrefixInstances;
const void* prefix_kernel_ptr(int variant);

// plan.cu
bool plan_is_valid(const pd_plan* plan);
pd_status plan_own_part(const pd_layer_desc* layer, int32_t batch, int32_t query_tokens,
                        const int32_t* seq_lens_host, int32_t sm_count, pd_plan* plan);
// abi.cu: stage 1 of the own part into the workspace, beside the prefix pass launched in front of it
pd_status launch_own_part(const pd_plan* plan, const void* q, const void* k_pool, const void* v_pool,
                          const float* k_scale, const float* v_scale, const int32_t* block_tables,
                          const int32_t* seq_lens, float scale, void* workspace, size_t workspace_bytes, void* out,
                          void* stream);
// abi.cu: a pool's tensor map with boxes of `rows` rows by `slabs` 128-byte slabs; the shared-memory limit of a
// prefix instance
pd_status encode_group_map(CUtensorMap* map, const void* pool, const pd_layer_desc& ly, int rows, int slabs);
pd_status ensure_prefix_smem(int variant, const void* fn, int smem_bytes);

}  // namespace pd
