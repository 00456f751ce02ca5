// Decode of a batch whose requests share prefixes (sm_103a): planner, prefix
// pass, merge and entry points.
//
// Mathematics: softmax attention over [prefix | own] splits into parts whose
// normalised outputs o_s and log-sum-exps l_s merge exactly,
//   out = sum_s w_s o_s,  w_s = exp(l_s - M) / sum_s' exp(l_s' - M),  M = max_s l_s,
// so the prefix part is computed for all query rows of a group at once (rows =
// requests x query tokens x heads of a KV head's group), the own part by the
// decode's stage 1, and one merge joins the pieces of both.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "pd_common.cuh"
#include "shared.h"

namespace pd {
namespace {

constexpr uint32_t kSharedMagic = 0x50445348u;  // "PDSH"
constexpr int32_t kSharedVersion = 1;

struct JoinParams {
  const float* lse[2];  // own, prefix: [rows][pieces]
  const float* o[2];
  int pieces[2];
  uint16_t* out;
};

constexpr int kJoinThreads = 128;
constexpr int kJoinMaxPieces = 2048;  // both parts' caps
constexpr int kJoinAhead = 8;         // pieces whose rows a thread has in flight

// A CTA per row and COLS float4 columns of it. The weights first (a thread per
// piece), then column `tid % COLS` over the pieces tid / COLS, + 128 / COLS, ...;
// the piece groups of a column are summed in shared memory. The first
// kJoinAhead rows of each thread load together with the log-sum-exps.
template <int D, int COLS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinParams p) {
  constexpr int GROUPS = kJoinThreads / COLS;
  __shared__ float wt[kJoinMaxPieces], red[2][4];
  __shared__ float4 part[GROUPS > 1 ? kJoinThreads : 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, at = tid % COLS, grp = tid / COLS;
  const int col = blockIdx.y * COLS + at;
  const size_t row = blockIdx.x;
  const int s0 = p.pieces[0], total = s0 + p.pieces[1];
  auto rows = [&](int s) {
    return reinterpret_cast<const float4*>(s < s0 ? p.o[0] + (row * s0 + s) * D
                                                  : p.o[1] + (row * p.pieces[1] + (s - s0)) * D) + col;
  };
  float4 ahead[kJoinAhead];
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i) {
    const int s = grp + i * GROUPS;
    ahead[i] = s < total ? __ldg(rows(s)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // NaN log-sum-exps stay NaN all the way
  float M = -INFINITY;
  for (int s = tid; s < total; s += kJoinThreads) {
    const float l = s < s0 ? p.lse[0][row * s0 + s] : p.lse[1][row * p.pieces[1] + (s - s0)];
    wt[s] = l;
    M = (l > M || isnan(l)) ? l : M;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    const float o = __shfl_xor_sync(kFullMask, M, m);
    M = (o > M || isnan(o)) ? o : M;
  }
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) M = (red[0][w] > M || isnan(red[0][w])) ? red[0][w] : M;
  float sum = 0.f;
  for (int s = tid; s < total; s += kJoinThreads) {
    // an empty piece weighs 0 (its row may never have been written)
    const float w = wt[s] == -INFINITY ? 0.f : exp2f((wt[s] - M) * 1.4426950408889634f);
    wt[s] = w;
    sum += w;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int s, const float4& v) {
    const float w = wt[s];
    if (w == 0.f) return;  // selected out, not multiplied
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  };
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i)
    if (grp + i * GROUPS < total) add(grp + i * GROUPS, ahead[i]);
  for (int base = grp + kJoinAhead * GROUPS; base < total; base += kJoinAhead * GROUPS) {
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
      const int s = base + i * GROUPS;
      if (s < total) ahead[i] = __ldg(rows(s));
    }
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i)
      if (base + i * GROUPS < total) add(base + i * GROUPS, ahead[i]);
  }
  if constexpr (GROUPS > 1) {
    part[tid] = acc;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) {
      const float4 v = part[k * COLS + at];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no piece at all: a zero row
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(p.out + row * D)[col] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

uint64_t align_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Query rows a tile of the prefix pass serves: the smallest of 16, 32, 64 and
// 128 that holds the largest group's (128 at head_dim 512: a pair of CTAs).
int row_tile_for(long long rows) {
  const int most = 128;
  int n = 16;
  while (n < most && n < rows) n *= 2;
  return n;
}

const PrefixInstance* find_prefix(int head_dim, int row_tile, bool fp8) {
  for (int i = 0; i < kNumPrefixInstances; ++i) {
    const PrefixInstance& v = kPrefixInstances[i];
    if (v.head_dim == head_dim && v.row_tile == row_tile && v.fp8 == fp8) return &v;
  }
  return nullptr;
}

bool shared_plan_is_valid(const pd_shared_plan* plan) {
  if (!plan || plan->magic != kSharedMagic || plan->version != (uint32_t)kSharedVersion) return false;
  const pd_plan& own = plan->own;
  if (!plan_is_valid(&own) || own.partial != 2) return false;
  if (plan->num_groups < 0 || plan->max_prefix_pages < 1 || plan->tiles < 0 || plan->tiles > 65535) return false;
  // (the own part is ordered behind the prefix pass: without row tiles there would be none to wait for)
  if (own.batch > 0 && (plan->num_groups < 1 || plan->tiles < 1)) return false;
  if (plan->variant < 0 || plan->variant >= kNumPrefixInstances) return false;
  const PrefixInstance& v = kPrefixInstances[plan->variant];
  if (v.head_dim != own.layer.head_dim || v.row_tile != plan->row_tile ||
      v.fp8 != (own.layer.kv_dtype == PD_KV_FP8_E4M3))
    return false;
  if (plan->num_pieces < 1 || plan->num_pieces > 1024) return false;
  if (plan->chunk_tokens < kPrefixTile || plan->chunk_tokens % kPrefixTile != 0) return false;
  if ((long long)plan->max_prefix_pages * own.layer.page_size > 0x7fffffffLL) return false;
  const uint64_t rows = (uint64_t)own.batch * own.query_tokens * own.layer.num_q_heads;
  if (rows > 0x7fffffffull) return false;
  uint64_t lse = 0, o = 0, end = 0;
  if (plan->lse_offset < own.workspace_bytes || plan->lse_offset % 256 != 0 || plan->o_offset % 256 != 0) return false;
  if (__builtin_mul_overflow(rows, (uint64_t)plan->num_pieces * 4ull, &lse) ||
      __builtin_mul_overflow(lse, (uint64_t)own.layer.head_dim, &o) ||
      __builtin_add_overflow(plan->lse_offset, lse, &end) || plan->o_offset < end ||
      __builtin_add_overflow(plan->o_offset, o, &end) || plan->workspace_bytes < end)
    return false;
  return true;
}

// What the cost model takes of the prefix pass, in microseconds on a 152-SM
// GB300: a CTA's start and end, and a tile (128 tokens; a pair's 256), measured
// at head_dim 512 (one figure for 16 to 64 rows, which take 2.3 to 2.8 in bf16
// and 3.25 to 3.8 in e4m3) and taken in proportion to head_dim below, where it
// was not measured; the tiles in flight share the memory's rate, and the pieces'
// partial results are written and read once.
constexpr double kFixedUs = 7.0, kHbmBytesPerUs = 6.8e6, kPartialBytesPerUs = 5.0e6;
constexpr double kOwnFixedUs = 5.0;  // a stage-1 CTA of the own part

double tile_us(const PrefixInstance& v) {
  return (v.ctas == 2 ? (v.fp8 ? 5.5 : 3.6) : (v.fp8 ? 3.8 : 2.9)) * v.head_dim / 512.0;
}

// SM time of the own part in one piece a request, in microseconds (two of its
// CTAs share an SM).
double own_sm_us(const pd_plan& own, const int32_t* lens) {
  const double per_us = 50.0 * 512 / own.layer.head_dim;  // tokens of a lone stage-1 CTA
  double us = 0;
  for (int b = 0; b < own.batch; ++b) us += (kOwnFixedUs + lens[b] / per_us) * own.grid_y;
  return us / 2;
}

// The prefix's pieces: of every count of pieces for the longest prefix, the one
// whose launch is modelled to end first. More pieces fill the SMs and even out
// prefixes of different lengths; each costs a CTA's fixed time and its partials.
void plan_pieces(pd_shared_plan& sp, const int32_t* starts, const int32_t* lens, int per_req, int sm_count,
                 double own_us) {
  const pd_layer_desc& ly = sp.own.layer;
  const int unit = kPrefixTile * kPrefixInstances[sp.variant].ctas;  // tokens of a tile
  const int slots = sm_count / kPrefixInstances[sp.variant].ctas;
  const long long most = ((long long)sp.max_prefix_len + unit - 1) / unit;
  sp.chunk_tokens = unit;
  sp.num_pieces = 1;
  if (most <= 1) return;
  const double cta_us = tile_us(kPrefixInstances[sp.variant]);
  const double tile_bytes = (double)unit * ly.head_dim * (ly.kv_dtype == PD_KV_FP8_E4M3 ? 1 : 2) *
                            (ly.kv_shared ? 1 : 2);
  const double rows = (double)sp.own.batch * sp.own.query_tokens * ly.num_q_heads;
  double best = 1e300;
  for (long long pieces = 1; pieces <= std::min<long long>(most, 1024); ++pieces) {
    const long long c = (most + pieces - 1) / pieces;
    if ((most + c - 1) / c != pieces) continue;  // the same cut as fewer pieces
    double ctas = 0, tiles = 0, distinct = 0;
    for (int n = 0; n < sp.num_groups; ++n) {
      const long long row_tiles = ((long long)(starts[n + 1] - starts[n]) * per_req + sp.row_tile - 1) / sp.row_tile;
      const long long len = (lens[n] + unit - 1) / unit;
      ctas += (double)row_tiles * ly.num_kv_heads * ((len + c - 1) / c);
      tiles += (double)row_tiles * ly.num_kv_heads * len;
      if (row_tiles > 0) distinct += (double)ly.num_kv_heads * len;
    }
    const double one = kFixedUs + c * cta_us;
    // within one wave the longest CTA; beyond, the mean load and part of a last
    // one; and what the own part finds free
    const double load = (ctas * kFixedUs + tiles * cta_us) / slots;
    double us = ctas <= slots ? one : std::max(one, load + 0.4 * one);
    us = std::max(us, load + own_us / sm_count + kOwnFixedUs);
    // (near the memory's rate a tile takes longer: a smooth maximum)
    const double alone = us - kFixedUs, hbm = distinct * tile_bytes / kHbmBytesPerUs;
    us = kFixedUs + std::pow(std::pow(alone, 4) + std::pow(hbm, 4), 0.25) +
         2.0 * rows * pieces * ly.head_dim * 4.0 / kPartialBytesPerUs;
    if (us < best) {
      best = us;
      sp.chunk_tokens = (int32_t)(c * unit);
      sp.num_pieces = (int32_t)pieces;
    }
  }
}

// Alone, the own part is cut to fill the SMs. Where the prefix pass leaves SMs
// free for long enough to take the whole own part beside it, each further piece
// only adds its fixed time: its pieces then grow to what a prefix CTA takes.
void shorten_own(pd_shared_plan& sp, const int32_t* starts, const int32_t* prefix, const int32_t* lens, int per_req,
                 int sm_count, double own_us) {
  pd_plan& own = sp.own;
  const pd_layer_desc& ly = own.layer;
  int longest = 0;
  for (int b = 0; b < own.batch; ++b) longest = std::max(longest, lens[b]);
  if (own.num_splits <= 1 || longest <= 0 || sp.max_prefix_len == 0) return;
  const PrefixInstance& v = kPrefixInstances[sp.variant];
  const double us = kFixedUs + sp.chunk_tokens / (kPrefixTile * v.ctas) * tile_us(v);
  const double per_us = 50.0 * 512 / ly.head_dim;  // tokens of a lone stage-1 CTA
  double prefix_ctas = 0;
  for (int n = 0; n < sp.num_groups; ++n)
    prefix_ctas += (double)(((long long)(starts[n + 1] - starts[n]) * per_req + sp.row_tile - 1) / sp.row_tile) *
                   ((prefix[n] + sp.chunk_tokens - 1) / sp.chunk_tokens) * ly.num_kv_heads * v.ctas;
  if ((sm_count - prefix_ctas) * us < own_us) return;
  const int chunk = std::max(own.chunk_tokens, (int)(us * per_us) / 64 * 64);
  own.chunk_tokens = std::min(chunk, (longest + 63) / 64 * 64);
  own.num_splits = (longest + own.chunk_tokens - 1) / own.chunk_tokens;
  own.grid_x = own.num_splits;
  const uint64_t rows = (uint64_t)own.batch * own.query_tokens * ly.num_q_heads;
  own.opart_offset = align_up(own.lse_offset + rows * own.num_splits * 4ull, 256);
  own.workspace_bytes = own.opart_offset + rows * own.num_splits * (uint64_t)ly.head_dim * 4ull;
}

pd_status plan_shared(const pd_layer_desc* layer, int32_t batch, int32_t query_tokens, const int32_t* seq_lens_host,
                      int32_t num_groups, const int32_t* group_starts_host, const int32_t* prefix_lens_host,
                      int32_t max_prefix_pages, int32_t sm_count, pd_shared_plan* plan) {
  if (!layer || !plan || num_groups < 0 || max_prefix_pages < 1) return PD_ERR_INVALID_ARG;
  if (layer->window != 0) return layer->window < 0 ? PD_ERR_INVALID_ARG : PD_ERR_UNSUPPORTED;
  pd_shared_plan sp;
  std::memset(&sp, 0, sizeof(sp));
  const pd_status st = plan_own_part(layer, batch, query_tokens, seq_lens_host, sm_count, &sp.own);
  if (st != PD_OK) return st;
  const pd_layer_desc& ly = *layer;
  const long long cap = (long long)max_prefix_pages * ly.page_size;
  if (cap > 0x7fffffffLL || num_groups > 65535) return PD_ERR_INVALID_ARG;
  if (batch > 0 && (num_groups < 1 || !group_starts_host || !prefix_lens_host)) return PD_ERR_INVALID_ARG;
  const int per_req = query_tokens * (ly.num_q_heads / ly.num_kv_heads);
  long long most_rows = 0;
  int32_t longest = 0;
  if (batch > 0) {
    if (group_starts_host[0] != 0 || group_starts_host[num_groups] != batch) return PD_ERR_INVALID_ARG;
    for (int n = 0; n < num_groups; ++n) {
      const int32_t s = group_starts_host[n], e = group_starts_host[n + 1], len = prefix_lens_host[n];
      if (e < s || e > batch) return PD_ERR_INVALID_ARG;
      if (len < 0 || len > cap || len % ly.page_size != 0) return PD_ERR_INVALID_ARG;
      most_rows = std::max(most_rows, (long long)(e - s) * per_req);
      if (e > s) longest = std::max(longest, len);
    }
  }
  sp.num_groups = num_groups;
  sp.max_prefix_pages = max_prefix_pages;
  sp.max_prefix_len = longest;
  sp.row_tile = row_tile_for(most_rows);
  const PrefixInstance* v = find_prefix(ly.head_dim, sp.row_tile, ly.kv_dtype == PD_KV_FP8_E4M3);
  if (!v) return PD_ERR_UNSUPPORTED;
  sp.variant = v->id;
  long long tiles = 0;
  for (int n = 0; batch > 0 && n < num_groups; ++n)
    tiles += ((long long)(group_starts_host[n + 1] - group_starts_host[n]) * per_req + sp.row_tile - 1) / sp.row_tile;
  if (tiles > 65535) return PD_ERR_UNSUPPORTED;
  sp.tiles = (int32_t)tiles;
  const double own_us = own_sm_us(sp.own, seq_lens_host);
  plan_pieces(sp, group_starts_host, prefix_lens_host, per_req, sm_count, own_us);
  shorten_own(sp, group_starts_host, prefix_lens_host, seq_lens_host, per_req, sm_count, own_us);
  const uint64_t rows = (uint64_t)batch * query_tokens * ly.num_q_heads;
  if (rows > 0x7fffffffull) return PD_ERR_UNSUPPORTED;
  sp.lse_offset = align_up(sp.own.workspace_bytes, 256);
  sp.o_offset = align_up(sp.lse_offset + rows * sp.num_pieces * 4ull, 256);
  sp.workspace_bytes = sp.o_offset + rows * sp.num_pieces * (uint64_t)ly.head_dim * 4ull;
  sp.magic = kSharedMagic;
  sp.version = kSharedVersion;
  *plan = sp;
  return PD_OK;
}

cudaError_t launch_dependent(const void* kernel, dim3 grid, int threads, int smem_bytes, void* stream, void** args,
                             int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

pd_status decode_shared(const pd_shared_plan* plan, bool fp8, const void* q, const void* k_pool, const void* v_pool,
                        const float* k_scale, const float* v_scale, const int32_t* prefix_tables,
                        const int32_t* prefix_lens, const int32_t* group_starts, const int32_t* block_tables,
                        const int32_t* seq_lens, float scale, void* workspace, size_t workspace_bytes, void* out,
                        void* stream) {
  if (!shared_plan_is_valid(plan)) return PD_ERR_INVALID_ARG;
  const pd_plan& own = plan->own;
  const pd_layer_desc& ly = own.layer;
  if ((ly.kv_dtype == PD_KV_FP8_E4M3) != fp8 || !std::isfinite(scale)) return PD_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return PD_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes) return PD_ERR_WORKSPACE_TOO_SMALL;
  if (own.batch == 0) return PD_OK;
  // everything before anything is queued: what stage 1 refuses too
  if (!q || !k_pool || !block_tables || !seq_lens || !out || !prefix_tables || !prefix_lens || !group_starts)
    return PD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(out, 16) || !aligned(block_tables, 4) ||
      !aligned(seq_lens, 4) || !aligned(prefix_tables, 4) || !aligned(prefix_lens, 4) || !aligned(group_starts, 4))
    return PD_ERR_INVALID_ARG;
  if (ly.kv_shared ? (v_pool && v_pool != k_pool) : (!v_pool || v_pool == k_pool || !aligned(v_pool, 16)))
    return PD_ERR_INVALID_ARG;
  if (fp8) {
    if (!k_scale || !aligned(k_scale, 4)) return PD_ERR_INVALID_ARG;
    if (ly.kv_shared ? (v_scale && v_scale != k_scale) : (!v_scale || !aligned(v_scale, 4))) return PD_ERR_INVALID_ARG;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k_scale = fp8 ? k_scale : nullptr;
  p.v_scale = fp8 ? (ly.kv_shared ? k_scale : v_scale) : nullptr;
  p.prefix_tables = prefix_tables;
  p.prefix_lens = prefix_lens;
  p.group_starts = group_starts;
  p.lse_part = reinterpret_cast<float*>(ws + plan->lse_offset);
  p.o_part = reinterpret_cast<float*>(ws + plan->o_offset);
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.batch = own.batch;
  p.num_groups = plan->num_groups;
  p.query_tokens = own.query_tokens;
  p.num_q_heads = ly.num_q_heads;
  p.num_kv_heads = ly.num_kv_heads;
  p.group = ly.num_q_heads / ly.num_kv_heads;
  p.head_dim = ly.head_dim;
  p.page_size = ly.page_size;
  p.num_pages = ly.num_pages;
  p.max_prefix_pages = plan->max_prefix_pages;
  p.row_tile = plan->row_tile;
  p.tiles = plan->tiles;
  p.num_pieces = plan->num_pieces;
  p.chunk_tokens = plan->chunk_tokens;
  const PrefixInstance& v = kPrefixInstances[plan->variant];
  // a stage of the pass holds 128 tokens x 128 dims of K, or a CTA's dims of v_tokens tokens of V
  const int v_tokens = kPrefixTile * 128 * v.ctas / ly.head_dim;
  p.k_box = 16;
  while (p.k_box < kPrefixTile && ly.page_size % (2 * p.k_box) == 0) p.k_box *= 2;
  p.v_box = std::min<int32_t>(p.k_box, v_tokens);
  p.keep_in_l2 = plan->tiles > 1 || ly.kv_shared;
  p.stall_bytes = own.test_stall_bytes;
  const void* fn = prefix_kernel_ptr(plan->variant);
  pd_status st = ensure_prefix_smem(plan->variant, fn, v.smem_bytes);
  const int slabs = ly.head_dim / (fp8 ? 128 : 64) / v.ctas;
  if (st == PD_OK) st = encode_group_map(&p.kmap, k_pool, ly, p.k_box, fp8 ? 1 : 2);
  if (st == PD_OK) st = encode_group_map(&p.vmap, ly.kv_shared ? k_pool : v_pool, ly, p.v_box, slabs);
  if (st != PD_OK) return st;
  void* args[] = {&p};
  if (launch_dependent(fn, dim3(plan->tiles * v.ctas, plan->num_pieces, ly.num_kv_heads), v.threads, v.smem_bytes,
                       stream, args, v.ctas) != cudaSuccess)
    return PD_ERR_CUDA;
  // the own part's CTAs take the SMs that the prefix pass leaves free
  st = launch_own_part(&own, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, scale, workspace,
                       workspace_bytes, out, stream);
  if (st != PD_OK) return st;
  JoinParams j = {};
  j.lse[0] = reinterpret_cast<const float*>(ws + own.lse_offset);
  j.o[0] = reinterpret_cast<const float*>(ws + own.opart_offset);
  j.pieces[0] = own.num_splits;
  j.lse[1] = p.lse_part;
  j.o[1] = p.o_part;
  j.pieces[1] = plan->num_pieces;
  j.out = static_cast<uint16_t*>(out);
  const unsigned rows = (unsigned)own.batch * own.query_tokens * ly.num_q_heads;
  void* jargs[] = {&j};
  // few rows of many pieces: a CTA per 128 dims, its threads on four pieces at a
  // time (256 rows of 25 pieces: 13.4 -> 6 us); otherwise whole rows a CTA
  const bool wide = rows >= 2048 || j.pieces[0] + j.pieces[1] <= 2 * kJoinAhead;
  const void* join = nullptr;
  if (ly.head_dim == 512)
    join = wide ? reinterpret_cast<const void*>(&join_kernel<512, 128>) : reinterpret_cast<const void*>(&join_kernel<512, 32>);
  else if (ly.head_dim == 256)
    join = wide ? reinterpret_cast<const void*>(&join_kernel<256, 64>) : reinterpret_cast<const void*>(&join_kernel<256, 32>);
  else
    join = reinterpret_cast<const void*>(&join_kernel<128, 32>);
  if (launch_dependent(join, dim3(rows, wide ? 1 : ly.head_dim / 128), kJoinThreads, 0, stream, jargs) != cudaSuccess)
    return PD_ERR_CUDA;
  return PD_OK;
}

}  // namespace
}  // namespace pd

extern "C" {

pd_status paged_decode_plan_shared(const pd_layer_desc* layer, int32_t batch, int32_t query_tokens,
                                   const int32_t* seq_lens_host, int32_t num_groups,
                                   const int32_t* group_starts_host, const int32_t* prefix_lens_host,
                                   int32_t max_prefix_pages, int32_t sm_count, pd_shared_plan* plan) {
  try {
    return pd::plan_shared(layer, batch, query_tokens, seq_lens_host, num_groups, group_starts_host,
                           prefix_lens_host, max_prefix_pages, sm_count, plan);
  } catch (...) {  // the planner's host allocations
    return PD_ERR_UNSUPPORTED;
  }
}

pd_status paged_decode_global_shared(const pd_shared_plan* plan, const void* q, const void* k_pool,
                                     const void* v_pool, const int32_t* prefix_tables, const int32_t* prefix_lens,
                                     const int32_t* group_starts, const int32_t* block_tables,
                                     const int32_t* seq_lens, float scale, void* workspace,
                                     size_t workspace_bytes, void* out, void* stream) {
  return pd::decode_shared(plan, false, q, k_pool, v_pool, nullptr, nullptr, prefix_tables, prefix_lens, group_starts,
                           block_tables, seq_lens, scale, workspace, workspace_bytes, out, stream);
}

pd_status paged_decode_global_shared_fp8(const pd_shared_plan* plan, const void* q, const void* k_pool,
                                         const void* v_pool, const float* k_scale, const float* v_scale,
                                         const int32_t* prefix_tables, const int32_t* prefix_lens,
                                         const int32_t* group_starts, const int32_t* block_tables,
                                         const int32_t* seq_lens, float scale, void* workspace,
                                         size_t workspace_bytes, void* out, void* stream) {
  return pd::decode_shared(plan, true, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens, group_starts,
                           block_tables, seq_lens, scale, workspace, workspace_bytes, out, stream);
}

pd_status paged_decode_global_shared_args(const pd_global_shared_args* a) {
  if (!a) return PD_ERR_INVALID_ARG;
  return pd::decode_shared(a->plan, a->fp8 != 0, a->q, a->k_pool, a->v_pool, a->fp8 ? a->k_scale : nullptr,
                           a->fp8 ? a->v_scale : nullptr, a->prefix_tables, a->prefix_lens, a->group_starts,
                           a->block_tables, a->seq_lens, a->scale, a->workspace, a->workspace_bytes, a->out, a->stream);
}

}  // extern "C"
