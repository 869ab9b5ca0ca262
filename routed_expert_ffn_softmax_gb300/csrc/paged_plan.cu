// Block tables and slot maps of one serving step, from request lengths (include/paged/moe_paged.h).
//
// With c_b tokens in the cache, n_b new ones and pages of P tokens, sequence b needs
// ceil((c_b + n_b) / P) - ceil(c_b / P) new pages; prefix sums of n_b and of the needs give every packed token
// its sequence and every new page its place in the free list. The work is a few bytes per sequence and 8 bytes
// per token row, so a call is latency: one launch, in which every CTA repeats the two scans over the (at most
// 2048) sequences from L2 rather than waiting for another CTA's, then writes its share of the token rows and
// new table entries. Outputs that may alias inputs (seq_lens, free_left) are written by the CTA that took the
// last ticket: by then every CTA has read them. GB300: 4.6 us for 64 sequences, 5.0 for 1000 with 67 thousand token rows,
// 3 of them the launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_device.cuh"
#include "moe_launch.h"

namespace moe {
namespace plan {

constexpr int kThreads = 512;
constexpr int kPer = kGqaMaxSeqs / kThreads;  // sequences per thread

struct Scan {
  int64_t warp_sum[kThreads / 32];
};

// Inclusive sum of v over the block's threads.
__device__ __forceinline__ int64_t block_scan(int64_t v, Scan& s) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) s.warp_sum[warp] = v;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += s.warp_sum[w];
  __syncthreads();
  return base + v;
}

// The last index i of the ascending a[0..n] with a[i] <= x (a[0] <= x): the non-empty interval that holds x.
__device__ __forceinline__ int interval_of(const int32_t* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PagedPlanArgs p) {
  __shared__ Scan scan;
  __shared__ int32_t cu[kGqaMaxSeqs + 1];     // packed token rows of the sequences before
  __shared__ int32_t base[kGqaMaxSeqs + 1];   // new pages taken by the sequences before
  __shared__ int32_t ctx[kGqaMaxSeqs];        // tokens in the cache c, or -1 - c for a sequence left out
  const int tid = threadIdx.x;
  pdl_wait_predecessor();
  pdl_allow_successor();

  int32_t c[kPer], n[kPer];
  int64_t tokens = 0;
  int status = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * kPer + k;
    c[k] = n[k] = 0;
    if (b < p.B) {
      c[k] = p.ctx_lens[b];
      n[k] = p.new_lens[b];
      if (c[k] < 0 || n[k] < 0) {
        status = kStatusBadSeqLen;
        c[k] = -1 - max(c[k], 0);
        n[k] = max(n[k], 0);
      }
    }
    tokens += n[k];
  }
  int count = *p.free_count;
  if (count < 0 || count > p.n_free) {
    if (tid == 0) status = kStatusPlanNoRoom;
    count = count < 0 ? 0 : p.n_free;
  }
  int64_t run = block_scan(tokens, scan) - tokens;
  int64_t pages = 0;
  int32_t need[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * kPer + k;
    need[k] = 0;
    if (b < p.B) {
      cu[b] = static_cast<int32_t>(min(run, static_cast<int64_t>(p.n_rows)));
      run += n[k];
      if (c[k] >= 0) {
        const int64_t all = (static_cast<int64_t>(c[k]) + n[k] + p.page_size - 1) >> p.page_shift;
        if (all > p.max_pages || run > p.n_rows) {
          status = kStatusPlanNoRoom;
          c[k] = -1 - c[k];
        } else {
          need[k] = static_cast<int32_t>(all - ((static_cast<int64_t>(c[k]) + p.page_size - 1) >> p.page_shift));
        }
      }
      if (b == p.B - 1) cu[p.B] = static_cast<int32_t>(min(run, static_cast<int64_t>(p.n_rows)));
    }
    pages += need[k];
  }
  int64_t used = block_scan(pages, scan) - pages;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * kPer + k;
    if (b < p.B) {
      base[b] = static_cast<int32_t>(min(used, static_cast<int64_t>(count)));
      used += need[k];
      if (need[k] > 0 && used > count) {
        status = kStatusPlanNoRoom;
        c[k] = -1 - c[k];
      }
      ctx[b] = c[k];
      if (b == p.B - 1) base[p.B] = static_cast<int32_t>(min(used, static_cast<int64_t>(count)));
    }
  }
  __shared__ int taken_s;
  if (tid == 0) taken_s = 0;
  __syncthreads();
  // pages handed out: the needs of the sequences that got theirs
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (tid * kPer + k < p.B && c[k] >= 0) mine += need[k];
  if (mine) atomicAdd(&taken_s, mine);
  if (status && blockIdx.x == 0) raise_status(p.status, status);
  __syncthreads();
  const int taken = taken_s;

  // every input that an output may alias has been read
  int ticket = 0;
  if (tid == 0) {
    __threadfence();
    ticket = atomicAdd(p.ticket, 1);
  }

  const int step = gridDim.x * kThreads;
  const int first = blockIdx.x * kThreads + tid;
  auto page_ok = [&](int32_t id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_pages); };
  // new table entries
  for (int k = first; k < taken; k += step) {
    const int b = interval_of(base, p.B, k);
    const int col = ((ctx[b] + p.page_size - 1) >> p.page_shift) + k - base[b];
    p.block_table[static_cast<int64_t>(b) * p.max_pages + col] = p.free_pages[count - 1 - k];
  }
  // token rows (counted in 64 bits: n_rows may lie within a step of 2^31)
  const int rows = cu[p.B];
  for (int64_t t = first; t < p.n_rows; t += step) {
    int32_t pos = 0, slot = -1;
    if (t < rows) {
      const int b = interval_of(cu, p.B, static_cast<int>(t));
      const int cb = ctx[b];
      const int i = static_cast<int>(t) - cu[b];
      pos = static_cast<int32_t>(static_cast<uint32_t>(cb < 0 ? -1 - cb : cb) + static_cast<uint32_t>(i));
      if (cb >= 0) {
        const int idx = pos >> p.page_shift;
        const int owned = (cb + p.page_size - 1) >> p.page_shift;
        const int32_t id = idx < owned ? p.block_table[static_cast<int64_t>(b) * p.max_pages + idx]
                                       : p.free_pages[count - 1 - (base[b] + idx - owned)];
        if (page_ok(id))
          slot = (id << p.page_shift) + (pos & (p.page_size - 1));
        else
          raise_status(p.status, kStatusBadPage);
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }

  __shared__ int last_s;
  if (tid == 0) last_s = ticket == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (last_s) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int b = tid * kPer + k;
      if (b < p.B) {
        p.seq_lens[b] = c[k] < 0 ? 0 : c[k] + n[k];
        p.cu_new[b] = cu[b];
      }
    }
    if (tid == 0) {
      p.cu_new[p.B] = rows;
      *p.free_left = count - taken;
      *p.ticket = 0;
    }
  }
}

}  // namespace plan

cudaError_t launch_paged_plan(const PagedPlanArgs& args, int num_sms, cudaStream_t stream) {
  // one token row per thread until the grid covers the device (each CTA repeats the scans)
  const int64_t want = (static_cast<int64_t>(args.n_rows) + plan::kThreads - 1) / plan::kThreads;
  const int grid = want < 1 ? 1 : (want < num_sms ? static_cast<int>(want) : num_sms);
  return launch_pdl(plan::paged_plan_kernel, dim3(grid), dim3(plan::kThreads), 0, stream, args);
}

}  // namespace moe
