// Attention of many query rows per key/value head over the paged cache (include/paged/moe_paged.h): prompts and
// chunks (causal, sliding window, sink tokens) and the shared prefix of a decode batch.
//
// First form: one warp per (query token, query head), 4 dimensions per lane, the online softmax over the visible
// keys one at a time. For a shared prefix each warp takes one split of the keys and leaves its (o, m, l).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "moe_device.cuh"
#include "moe_launch.h"

namespace moe {
namespace rows {

constexpr int kThreads = 256;

__device__ __forceinline__ void load4(const uint16_t* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
}

__global__ void __launch_bounds__(kThreads) gqa_rows_kernel(const GqaRowsPlan p) {
  pdl_wait_predecessor();
  pdl_allow_successor();
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const bool prefix = p.prefix_table != nullptr;
  const int splits = prefix ? p.prefix_splits : 1;
  const int64_t row = w / splits;
  const int s = static_cast<int>(w - row * splits);
  const int n = static_cast<int>(row / p.h_q);
  const int hq = static_cast<int>(row - static_cast<int64_t>(n) * p.h_q);
  if (n >= p.N) return;
  const int G = p.h_q / p.h_kv;
  const int j = hq / G;
  const int page = 1 << p.paged.page_shift;
  int beg = 0, end = 0, lo = 0, sk = 0;
  const int32_t* table = p.prefix_table;
  if (prefix) {
    const int tiles = (p.prefix_len + 127) / 128;
    beg = 128 * static_cast<int>(static_cast<int64_t>(s) * tiles / splits);
    end = min(p.prefix_len, 128 * static_cast<int>(static_cast<int64_t>(s + 1) * tiles / splits));
    lo = beg;
  } else {
    int b = -1;
    for (int i = 0; i < p.B; ++i) {
      const int x0 = p.cu_q[i], x1 = p.cu_q[i + 1];
      if (x0 < 0 || x1 < x0 || x1 > p.N) {
        if (lane == 0) atomicExch(p.status, kStatusBadSeqLen);
        continue;
      }
      if (x0 <= n && n < x1) b = i;
    }
    if (b < 0) return;
    int len = p.seq_lens[b];
    if (len < 0 || len > p.paged.max_pages * page) {
      if (lane == 0) atomicExch(p.status, kStatusBadSeqLen);
      len = 0;
    }
    const int pos = len - (p.cu_q[b + 1] - n);
    end = len == 0 ? 0 : max(pos + 1, 0);
    lo = p.paged.window > 0 ? max(0, end - p.paged.window) : 0;
    sk = min(p.paged.n_sink, lo);
    table = p.paged.block_table + static_cast<int64_t>(b) * p.paged.max_pages;
  }
  float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  load4(p.q + (static_cast<int64_t>(n) * p.h_q + hq) * 128 + 4 * lane, q);
  float m = -FLT_MAX, l = 0.0f;
  for (int key = sk > 0 ? 0 : max(beg, lo); key < end; key = key + 1 == sk ? max(sk, lo) : key + 1) {
    const int id = table[key >> p.paged.page_shift];
    const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.paged.num_pages);
    float k[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ok) {
      const int64_t at =
          (((static_cast<int64_t>(id) * p.h_kv + j) << p.paged.page_shift) + (key & (page - 1))) * 128 + 4 * lane;
      load4(p.k_cache + at, k);
      load4(p.v_cache + at, v);
    } else if (lane == 0) {
      atomicExch(p.status, kStatusBadPage);
    }
    float d = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    d *= p.scale_log2;
    const float m_new = fmaxf(m, d);
    const float a = exp2f(m - m_new), e = exp2f(d - m_new);
    l = l * a + e;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = o[x] * a + e * v[x];
    m = m_new;
  }
  if (prefix) {
    const int half = 128 / G;
    const int block = n / (2 * half);
    const int i = n - block * 2 * half;
    const int hf = i >= half ? 1 : 0;
    const int r = hf * 128 + (i - hf * half) * G + hq - j * G;
    const int64_t pieces = static_cast<int64_t>(p.h_kv) * p.prefix_blocks * splits;
    const int64_t at = ((static_cast<int64_t>(j) * p.prefix_blocks + block) * splits + s) * kRowTile + r;
    float* po = p.pieces + at * 128 + 4 * lane;
    for (int x = 0; x < 4; ++x) po[x] = o[x];
    if (lane == 0) {
      p.pieces[pieces * kRowTile * 128 + at] = m;
      p.pieces[pieces * kRowTile * 128 + pieces * kRowTile + at] = l;
    }
  } else {
    uint16_t* out = p.out + (static_cast<int64_t>(n) * p.h_q + hq) * 128 + 4 * lane;
    for (int x = 0; x < 4; ++x) {
      const __nv_bfloat16 b = __float2bfloat16_rn(l > 0.0f ? o[x] / l : 0.0f);
      out[x] = *reinterpret_cast<const uint16_t*>(&b);
    }
  }
}

}  // namespace rows

cudaError_t launch_gqa_rows(const GqaRowsPlan& plan, cudaStream_t stream) {
  const int64_t warps =
      static_cast<int64_t>(plan.N) * plan.h_q * (plan.prefix_table ? plan.prefix_splits : 1);
  const int64_t grid = (warps * 32 + rows::kThreads - 1) / rows::kThreads;
  return launch_pdl(rows::gqa_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(rows::kThreads), 0, stream, plan);
}

}  // namespace moe
