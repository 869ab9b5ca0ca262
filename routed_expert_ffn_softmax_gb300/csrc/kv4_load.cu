// Rows of the 4-bit cache as bf16 rows of another paged cache (include/paged/moe_kv4.h).
//
// 144 bytes are read and 512 written per token and head, so HBM's writes bound it. The work is listed as blocks of 16
// tokens of a head: every CTA repeats the scan over the sequences' block counts (as the plan's kernel does), and each warp
// takes a block at a time, all of its loads before its first store; 4 lanes share a row, 16 bytes of codes and 64 bytes of each
// store instruction. GB300: 262144 tokens of 8 heads in 228 us (6.05 TB/s, 89% of a copy), 9603 in 9.2 (5.5 TB/s; a third of
// it is the launch and the scan). With 16 lanes to a row and loads of 2 bytes between the stores it was 424 and 10.7.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_device.cuh"
#include "step_launch.h"

namespace moe {
namespace kv4 {

constexpr int kLoadThreads = 256;
constexpr int kLoadWarps = kLoadThreads / 32;
constexpr int kPer = kGqaMaxSeqs / kLoadThreads;  // sequences per thread

// Codes n = c + 8 of one 16-bit word, times s, as two packed pairs.
__device__ __forceinline__ uint2 four_values(uint32_t n4, float s) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)  // 2^23 + n is exact in fp32
    v[i] = (__uint_as_float(0x4b000000u | ((n4 >> (4 * i)) & 15u)) - 8388616.0f) * s;
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__global__ void __launch_bounds__(kLoadThreads) kv4_load_kernel(const Kv4LoadArgs p) {
  __shared__ int32_t pre[kGqaMaxSeqs + 1];  // blocks of the sequences before
  __shared__ int32_t warp_sum[kLoadWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_predecessor();
  pdl_allow_successor();

  const int per = (p.B + kLoadThreads - 1) / kLoadThreads;
  const int64_t cap = static_cast<int64_t>(min(p.max_pages, p.dst_max_pages)) << p.page_shift;
  int n[kPer];
  int sum = 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * per + k;
    n[k] = 0;
    if (k < per && b < p.B) {
      const int len = p.seq_lens[b], first = p.first ? p.first[b] : 0;
      if (len < 0 || len > cap || first < 0) bad = true;
      else if (first < len) n[k] = (len + kKv4Tokens - 1) / kKv4Tokens - first / kKv4Tokens;
      sum += n[k];
    }
  }
  if (bad) raise_status(p.status, kStatusBadSeqLen);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += warp_sum[w];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * per + k;
    if (k < per && b < p.B) {
      pre[b] = run;
      run += n[k];
      if (b == p.B - 1) pre[p.B] = run;
    }
  }
  __syncthreads();

  const int q = lane & 3;  // of a row's codes: words 8 q .. 8 q + 7 are dimensions 32 w + 8 q .. + 7 for each w
  const int page_blocks = 1 << (p.page_shift - 4);
  // (up to 2^31 - 1; a turn more still fits 32 bits without a sign)
  const uint32_t total = static_cast<uint32_t>(pre[p.B] * p.h_kv);
  for (uint32_t item = blockIdx.x * kLoadWarps + warp; item < total; item += gridDim.x * kLoadWarps) {
    const int it = static_cast<int>(item);
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {  // the last sequence whose first item is <= it (skips empty ones)
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * p.h_kv <= it) lo = mid; else hi = mid - 1;
    }
    const int count = pre[lo + 1] - pre[lo];
    const int off = it - pre[lo] * p.h_kv;
    const int j = off / count;
    const int first = p.first ? p.first[lo] : 0;
    const int block = first / kKv4Tokens + off - j * count;
    const int r0 = max(0, first - block * kKv4Tokens);
    const int r1 = min(kKv4Tokens, p.seq_lens[lo] - block * kKv4Tokens);
    const int page = block / page_blocks;
    const int src = p.block_table[static_cast<int64_t>(lo) * p.max_pages + page];
    const int dst = p.dst_table[static_cast<int64_t>(lo) * p.dst_max_pages + page];
    const bool from = static_cast<uint32_t>(src) < static_cast<uint32_t>(p.num_pages);
    const bool to = static_cast<uint32_t>(dst) < static_cast<uint32_t>(p.dst_pages);
    if (lane == 0 && !(from && to)) raise_status(p.status, kStatusBadPage);
    if (!to) continue;
    const int in_page = block & (page_blocks - 1);
    const uint8_t* at = p.cache + ((static_cast<int64_t>(from ? src : 0) * p.h_kv + j) * page_blocks + in_page) * kKv4Block;
    const int64_t out = ((static_cast<int64_t>(dst) * p.h_kv + j) * page_blocks + in_page) * (kKv4Tokens * 128) + 8 * q;
    uint4 codes[2][2];
    uint2 scales[2][2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 2) + 8 * i;
        codes[kv][i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        scales[kv][i] = make_uint2(0u, 0u);
        if (from) {
          codes[kv][i] = *reinterpret_cast<const uint4*>(at + kv * kKv4Values + r * kKv4RowBytes + 16 * q);
          scales[kv][i] = *reinterpret_cast<const uint2*>(at + kv * kKv4Values + kKv4Scales + 8 * r);
        }
      }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 2) + 8 * i;
        if (r < r0 || r >= r1) continue;
        uint16_t* row = (kv ? p.v_cache : p.k_cache) + out + r * 128;
        const uint4 c = codes[kv][i];
        const uint2 s2 = scales[kv][i];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int shift = 16 * (w & 1);
          const float f = __uint_as_float(((w < 2 ? s2.x : s2.y) >> shift) << 16);
          const uint2 a = four_values((w < 2 ? c.x : c.y) >> shift, f), b = four_values((w < 2 ? c.z : c.w) >> shift, f);
          *reinterpret_cast<uint4*>(row + 32 * w) = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
  }
}

}  // namespace kv4

cudaError_t launch_kv4_load(const Kv4LoadArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(a.B) * a.h_kv * min(a.max_pages, a.dst_max_pages) << (a.page_shift - 4);
  const int64_t blocks = (most + kv4::kLoadWarps - 1) / kv4::kLoadWarps;
  const int64_t resident = static_cast<int64_t>(num_sms) * 6;
  const int grid = static_cast<int>(blocks < resident ? blocks : resident);
  return launch_pdl(kv4::kv4_load_kernel, dim3(grid), dim3(kv4::kLoadThreads), 0, stream, a);
}

}  // namespace moe
