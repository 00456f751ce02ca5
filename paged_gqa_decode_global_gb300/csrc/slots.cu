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

#include <cstdint>

#include "paged_decode.h"
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
  int32_t* first_page;  // workspace [batch]: first free-list entry, or -1 for a request not served
  int32_t* cached;      // workspace [batch]: cached_lens (which seq_lens may alias)
};

constexpr int kScanThreads = 1024;

// Inclusive sum over the CTA's threads (warp shuffles, then the warps' sums).
__device__ __forceinline__ long long cta_scan(long long x, long long* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  long long before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  __syncthreads();
  return x + before;
}

__global__ void __launch_bounds__(kScanThreads) slots_scan_kernel(const SlotParams p) {
  __shared__ long long warp_sum[32], total[2];
  const long long cap = (long long)p.max_pages * p.page_size;
  long long next = p.free_range[0], end = p.free_range[1];
  if (next < 0) next = 0;
  if (end > p.num_free) end = p.num_free;
  if (end < next) end = next;
  const long long first_free = next;
  long long tok_base = 0, page_base = next, taken = next;
  uint32_t err = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kScanThreads) {
    const int b = b0 + threadIdx.x;
    long long c = 0, n = 0, need = 0;
    bool ok = false;
    if (b < p.batch) {
      c = p.cached_lens[b];
      n = p.new_tokens[b];
      ok = c >= 0 && n >= 0 && c + n <= cap;
      if (ok) need = (c + n + p.page_size - 1) / p.page_size - (c + p.page_size - 1) / p.page_size;
      else if (n < 0 || n > cap) n = 0;
    }
    const long long tok_end = tok_base + cta_scan(n, warp_sum);
    const long long page_end = page_base + cta_scan(need, warp_sum);
    if (b < p.batch) {
      if (!ok || tok_end > p.max_tokens) {
        ok = false;
        err |= kErrBadSeqLen;
      } else if (need > 0 && page_end > end) {
        ok = false;
        err |= kErrNoPages;
      }
      p.first_page[b] = ok ? (int32_t)(page_end - need) : -1;
      p.cached[b] = (int32_t)c;
      p.seq_lens[b] = (int32_t)(ok ? c + n : c);
      p.token_starts[b] = (int32_t)min(tok_end - n, 0x7fffffffLL);
    }
    const long long got = (b < p.batch && ok && need > 0) ? need : 0;
    const long long sum = cta_scan(got, warp_sum);
    if (threadIdx.x == kScanThreads - 1) {
      total[0] = tok_end;
      total[1] = page_end;
      warp_sum[0] = sum;
    }
    __syncthreads();
    tok_base = total[0];
    page_base = total[1];
    taken += warp_sum[0];
    __syncthreads();
  }
  if (err) atomicOr(p.flags, err);
  if (threadIdx.x == 0) {
    p.token_starts[p.batch] = (int32_t)min(tok_base, 0x7fffffffLL);
    p.free_range_out[0] = (int32_t)(p.batch > 0 ? taken : first_free);
    p.free_range_out[1] = (int32_t)end;
  }
}

// One thread per entry of slot_map; the thread of a new page's first token
// (every new page begins with one) writes the page into the table.
__global__ void __launch_bounds__(256) slots_fill_kernel(const SlotParams p) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= p.max_tokens) return;
  int slot = -1, pos = -1;
  if (p.batch > 0 && t < p.token_starts[p.batch]) {
    int lo = 0, hi = p.batch;  // the last request that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.token_starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int first = p.first_page[lo];
    if (first >= 0) {
      const int c = p.cached[lo];
      pos = c + t - p.token_starts[lo];
      const int held = (c + p.page_size - 1) / p.page_size, at = pos / p.page_size;
      int32_t* entry = p.block_tables + (size_t)lo * p.max_pages + at;
      int page;
      if (at < held) {
        page = *entry;
      } else {
        page = p.free_pages[first + at - held];
        if (pos == at * p.page_size) *entry = page;
      }
      if ((unsigned)page < (unsigned)p.num_pages) slot = page * p.page_size + (pos - at * p.page_size);
      else atomicOr(p.flags, kErrBadPage);
    }
  }
  p.slot_map[t] = slot;
  if (p.positions) p.positions[t] = pos;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace pd

extern "C" {

size_t paged_decode_append_slots_workspace(int32_t batch) {
  const size_t n = batch > 0 ? (size_t)batch : 0;
  return (256 + n * 8 + 255) / 256 * 256;
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
  p.first_page = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
  p.cached = p.first_page + batch;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  pd::slots_scan_kernel<<<1, pd::kScanThreads, 0, s>>>(p);
  if (max_tokens > 0) pd::slots_fill_kernel<<<(max_tokens + 255) / 256, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // extern "C"
