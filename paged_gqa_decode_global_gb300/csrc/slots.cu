// Block tables and slot maps of a batch's new tokens, built on the GPU from the
// requests' lengths (sm_103a).
//
// Mathematics: with c_b cached and n_b new tokens, request b needs
//   need_b = ceil((c_b + n_b) / P) - ceil(c_b / P)
// pages; exclusive prefix sums over the requests give its first token
// (sum n) and its first free-list entry (next + sum need); token j of b has
// position c_b + j, page index p = position / P, and its page is the table's
// entry p below ceil(c_b / P), else the free list's at first + p - ceil(c_b / P).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "paged_decode.h"
#include "pd_common.cuh"
#include "pd_variants.h"

namespace pd {
namespace {

struct SlotParams {
  int batch, page_size, num_pages, max_pages, max_tokens, num_free;
  const int32_t* cached_lens;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* free_range;
  int32_t* block_tables;
  int32_t* seq_lens;
  int32_t* token_starts;
  int32_t* slot_map;
  int32_t* positions;  // or null
  int32_t* free_range_out;
  uint32_t* flags;
  uint32_t* ticket;  // workspace: CTAs done reading (0 between calls)
  bool wide;         // slot_map and positions take 16-byte stores
  bool in_place;     // an output is one of the inputs
};

constexpr int kThreads = 1024;

// What a CTA knows of the 1024 requests of one round.
struct Round {
  int start[kThreads];   // first token (clamped to 31 bits)
  int first[kThreads];   // first free-list entry (0 if it needs none), -1 for a request not served
  int cached[kThreads];
};

struct Sums {
  long long tokens, pages;
};

// Inclusive sums over the CTA's threads; `total` of all of them. One barrier:
// every warp scans the 32 warps' sums itself. `scratch` must not be in use.
__device__ __forceinline__ Sums cta_scan(Sums x, Sums* scratch, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(kFullMask, x.tokens, o), b = __shfl_up_sync(kFullMask, x.pages, o);
    if (lane >= o) {
      x.tokens += a;
      x.pages += b;
    }
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  Sums w = scratch[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(kFullMask, w.tokens, o), b = __shfl_up_sync(kFullMask, w.pages, o);
    if (lane >= o) {
      w.tokens += a;
      w.pages += b;
    }
  }
  total.tokens = __shfl_sync(kFullMask, w.tokens, 31);
  total.pages = __shfl_sync(kFullMask, w.pages, 31);
  const long long a = __shfl_sync(kFullMask, w.tokens, (warp + 31) & 31);
  const long long b = __shfl_sync(kFullMask, w.pages, (warp + 31) & 31);
  if (warp > 0) {
    x.tokens += a;
    x.pages += b;
  }
  return x;
}

// The slot and position of token t, which belongs to request b of the batch (entry r of the round).
__device__ __forceinline__ void place(const SlotParams& p, const Round& rd, int r, int b, int t, int& slot, int& pos) {
  slot = pos = -1;
  const int first = rd.first[r];
  if (first < 0) return;
  const int c = rd.cached[r];
  pos = c + t - rd.start[r];
  // (unsigned: a length and a page size of nearly 2^31 each are allowed)
  const int held = ((unsigned)c + (unsigned)p.page_size - 1) / (unsigned)p.page_size, at = pos / p.page_size;
  int32_t* entry = p.block_tables + (size_t)b * p.max_pages + at;
  int page;
  if (at < held) {
    page = *entry;
  } else {
    // every new page begins with a new token, whose thread writes the table's entry
    page = __ldg(p.free_pages + first + at - held);
    if (pos == at * p.page_size) *entry = page;
  }
  if ((unsigned)page < (unsigned)p.num_pages) slot = page * p.page_size + (pos - at * p.page_size);
  else atomicOr(p.flags, kErrBadPage);
}

// A CTA serves TPT * 1024 entries of slot_map, but scans the lengths of every
// request up to its last token (at most a few rounds of 1024): with B requests
// in L2 that costs less than a launch of its own for the sums (12.5 us as two
// launches). Bound: the chain of dependent loads, ~4 us for a decode step of
// 256 requests. The first CTA writes the results per request; where they
// update the inputs in place and other CTAs read those too, the CTA that is
// last to have read them does, in a second walk (~3 us).
template <int TPT>
__global__ void __launch_bounds__(kThreads) slots_kernel(const SlotParams p) {
  __shared__ Round rd;
  __shared__ Sums scratch[2][32];
  __shared__ bool last;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const long long cap = (long long)p.max_pages * p.page_size;
  long long next = p.free_range[0], end = p.free_range[1];
  if (next < 0) next = 0;
  if (end > p.num_free) end = p.num_free;
  if (end < next) end = next;
  const bool only = gridDim.x == 1;
  const long long t0 = (long long)blockIdx.x * (TPT * kThreads);
  const long long t1 = min((long long)p.max_tokens, t0 + TPT * kThreads);

  // all requests in rounds of 1024: fill this CTA's entries, or (write) the results per request
  auto walk = [&](bool fill, bool write) {
    Sums base{0, next}, served{0, 0};
    uint32_t err = 0;
    int turn = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      const int b = b0 + tid;
      long long c = 0, n = 0, need = 0;
      bool ok = false;
      if (b < p.batch) {
        c = p.cached_lens[b];
        n = p.new_tokens[b];
        ok = c >= 0 && n >= 0 && c + n <= cap;
        if (ok)
          need = (unsigned)(c + n + p.page_size - 1) / (unsigned)p.page_size - (unsigned)(c + p.page_size - 1) / (unsigned)p.page_size;
        else if (n < 0 || n > cap)
          n = 0;
      }
      Sums total;
      const Sums in = cta_scan(Sums{n, need}, scratch[turn], total);
      turn ^= 1;
      const long long tok_end = base.tokens + in.tokens, page_end = base.pages + in.pages;
      if (b < p.batch) {
        if (!ok || tok_end > p.max_tokens) {
          ok = false;
          err |= kErrBadSeqLen;
        } else if (need > 0 && page_end > end) {
          ok = false;
          err |= kErrNoPages;
        }
        if (ok && need > 0) served.pages = page_end;  // served requests that take pages come before all that cannot
        if (write) {
          p.seq_lens[b] = (int32_t)(ok ? c + n : c);
          p.token_starts[b] = (int32_t)min(tok_end - n, 0x7fffffffLL);
        }
      }
      if (fill) {
        rd.start[tid] = (int)min(tok_end - n, 0x7fffffffLL);
        // (behind requests that found no page the count may pass 31 bits, where only those without need are served)
        rd.first[tid] = !ok ? -1 : need > 0 ? (int)(page_end - need) : 0;
        rd.cached[tid] = (int)c;
        __syncthreads();
        const int in_round = min(kThreads, p.batch - b0);
        const long long lo = max(t0, base.tokens), hi = min(t1, base.tokens + total.tokens);
        const long long mine = t0 + (long long)tid * TPT;
        if (mine < hi && mine + TPT > lo) {
          // the last request of the round that starts at or before the first of this thread's tokens
          int t = (int)max(mine, lo);
          int a = 0, z = in_round;
          while (z - a > 1) {
            const int mid = (a + z) >> 1;
            if (rd.start[mid] <= t) a = mid;
            else z = mid;
          }
          int slot[TPT], pos[TPT];
#pragma unroll
          for (int k = 0; k < TPT; ++k) {
            const long long tk = mine + k;
            slot[k] = pos[k] = -1;
            if (tk < lo || tk >= hi) continue;
            while (a + 1 < in_round && rd.start[a + 1] <= (int)tk) ++a;
            place(p, rd, a, b0 + a, (int)tk, slot[k], pos[k]);
          }
          if (TPT == 4 && p.wide && mine >= lo && mine + TPT <= hi) {
            *reinterpret_cast<int4*>(p.slot_map + mine) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            if (p.positions) *reinterpret_cast<int4*>(p.positions + mine) = make_int4(pos[0], pos[1], pos[2], pos[3]);
          } else {
#pragma unroll
            for (int k = 0; k < TPT; ++k) {
              if (mine + k < lo || mine + k >= hi) continue;
              p.slot_map[mine + k] = slot[k];
              if (p.positions) p.positions[mine + k] = pos[k];
            }
          }
        }
        __syncthreads();
      }
      base.tokens += total.tokens;
      base.pages += total.pages;
      if (!write && base.tokens >= t1) break;
    }
    if (fill)  // padding behind the last new token
      for (long long t = max(t0, base.tokens) + tid; t < t1; t += kThreads) {
        p.slot_map[t] = -1;
        if (p.positions) p.positions[t] = -1;
      }
    if (write) {
      if (err) atomicOr(p.flags, err);
      // the end of the pages taken: the largest of the threads'
      __syncthreads();
      const Sums mine{0, max(served.pages, next)};
      long long m = mine.pages;
#pragma unroll
      for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
      if ((tid & 31) == 0) scratch[0][tid >> 5].pages = m;
      __syncthreads();
      if (tid < 32) {
        m = scratch[0][tid].pages;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
        if (tid == 0) {
          p.token_starts[p.batch] = (int32_t)min(base.tokens, 0x7fffffffLL);
          p.free_range_out[0] = (int32_t)m;
          p.free_range_out[1] = (int32_t)end;
        }
      }
    }
  };
  if (only || !p.in_place) {
    walk(true, blockIdx.x == 0);
    return;
  }
  walk(true, false);
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    if (last) *p.ticket = 0;
  }
  __syncthreads();
  if (last) walk(false, true);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace pd

extern "C" {

size_t paged_decode_append_slots_workspace(int32_t batch) {
  (void)batch;  // a counter, whatever the batch
  return 256;
}

pd_status paged_decode_append_slots(int32_t batch, int32_t page_size, int32_t num_pages, int32_t max_pages,
                                    int32_t max_tokens, const int32_t* cached_lens, const int32_t* new_tokens,
                                    const int32_t* free_pages, int32_t num_free, const int32_t* free_range,
                                    int32_t* block_tables, int32_t* seq_lens, int32_t* token_starts,
                                    int32_t* slot_map, int32_t* positions, int32_t* free_range_out,
                                    uint32_t* device_flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || page_size <= 0 || num_pages <= 0 || max_pages <= 0 || max_tokens < 0 || num_free < 0)
    return PD_ERR_INVALID_ARG;
  if ((long long)num_pages * page_size > 0x7fffffffLL || (long long)max_pages * page_size > 0x7fffffffLL)
    return PD_ERR_INVALID_ARG;
  if (batch > 0 && (!cached_lens || !new_tokens || !block_tables || !seq_lens)) return PD_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_pages) || (max_tokens > 0 && !slot_map)) return PD_ERR_INVALID_ARG;
  if (!free_range || !free_range_out || !token_starts || !device_flags || !workspace) return PD_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)cached_lens, (const void*)new_tokens, (const void*)free_pages,
                          (const void*)free_range, (const void*)block_tables, (const void*)seq_lens,
                          (const void*)token_starts, (const void*)slot_map, (const void*)positions,
                          (const void*)free_range_out, (const void*)device_flags})
    if (!pd::aligned(ptr, 4)) return PD_ERR_INVALID_ARG;
  if (!pd::aligned(workspace, 256)) return PD_ERR_INVALID_ARG;
  if (workspace_bytes < paged_decode_append_slots_workspace(batch)) return PD_ERR_WORKSPACE_TOO_SMALL;
  pd::SlotParams p;
  p.batch = batch;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.max_tokens = max_tokens;
  p.num_free = num_free;
  p.cached_lens = cached_lens;
  p.new_tokens = new_tokens;
  p.free_pages = free_pages;
  p.free_range = free_range;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.token_starts = token_starts;
  p.slot_map = slot_map;
  p.positions = positions;
  p.free_range_out = free_range_out;
  p.flags = device_flags;
  p.ticket = static_cast<uint32_t*>(workspace);
  p.wide = pd::aligned(slot_map, 16) && pd::aligned(positions, 16);
  p.in_place = seq_lens == cached_lens || free_range_out == free_range;
  // one entry a thread for a decode step (one CTA), four (16-byte stores) above
  const int per_thread = max_tokens > pd::kThreads ? 4 : 1;
  const long long per_cta = (long long)per_thread * pd::kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<long long>(1, (max_tokens + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(pd::kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = per_thread == 4 ? cudaLaunchKernelEx(&cfg, pd::slots_kernel<4>, p)
                                        : cudaLaunchKernelEx(&cfg, pd::slots_kernel<1>, p);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

pd_status paged_decode_append_slots_args(const pd_append_slots_args* a) {
  if (!a) return PD_ERR_INVALID_ARG;
  return paged_decode_append_slots(a->batch, a->page_size, a->num_pages, a->max_pages, a->max_tokens, a->cached_lens,
                                   a->new_tokens, a->free_pages, a->num_free, a->free_range, a->block_tables,
                                   a->seq_lens, a->token_starts, a->slot_map, a->positions, a->free_range_out,
                                   a->device_flags, a->workspace, a->workspace_bytes, a->stream);
}

}  // extern "C"
