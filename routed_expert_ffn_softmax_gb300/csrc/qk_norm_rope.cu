// Per-head norm of queries and keys, position rotation and the cache store in one pass
// (include/paged/moe_paged.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * inv_freq
//
// Each value is read once and written once (2 B each way), so HBM bounds it. A head's 128 values are 16 lanes of
// 16 bytes, so a warp holds two heads and one load or store instruction moves 512 contiguous bytes; the mean is
// four shuffles. The partner of a rotated pair sits rot / 2 dimensions away in another lane and comes by
// shuffling the packed bf16 inputs (four shuffles for eight values); the partner's norm factor is the same, its
// weight is kept beside the lane's own. Only the result is rounded.
//
// The angle: inv_freq / (2 pi) is kept as a 64-bit fraction of a turn (computed in fp64, rounded once), so
// pos * fraction modulo 2^64 is the angle modulo one turn without any loss for large pos (error below
// pos * 2^-53 turns), and sin and cos are taken of a reduced argument.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_device.cuh"
#include "moe_launch.h"

namespace moe {
namespace qk {

constexpr int kThreads = 256;
constexpr int kD = 128;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The fraction of a turn that one position adds, in units of 2^-64 turns (modulo whole turns).
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  double f = static_cast<double>(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
  f -= floor(f);                                                      // [0, 1)
  return static_cast<uint64_t>(__double2ull_rn(f * 18446744073709551616.0));
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkNormRopeArgs p) {
  __shared__ __align__(16) float cs[2][kD / 2];  // cos, sin of the token's pairs
  const int tid = threadIdx.x;
  const int hw = tid >> 4;       // half-warp: one head
  const int l = tid & 15;        // dimensions 8 l .. 8 l + 7
  const int half = p.rot >> 1;
  pdl_wait_predecessor();
  pdl_allow_successor();

  const uint64_t turn = tid < half ? turn_fraction(p.inv_freq[tid]) : 0;
  // the lane's role in the rotation: first (a) or second (b) of its pairs, or untouched
  const bool rotates = 8 * l < p.rot;
  const bool second = !kInterleaved && 8 * l >= half;
  const int partner = kInterleaved ? l : (second ? l - (half >> 3) : l + (half >> 3));
  const int heads = p.h_q + 2 * p.h_kv;

  for (int n = blockIdx.x; n < p.N; n += gridDim.x) {
    const int pos = p.positions[n];
    const int slot = p.slots[n];
    if (tid < half) {
      const uint64_t a = turn * static_cast<uint64_t>(static_cast<int64_t>(pos));
      // signed fraction of a turn in [-1/2, 1/2), times two for sincospi
      const float f = static_cast<float>(static_cast<double>(static_cast<int64_t>(a)) * (1.0 / 9223372036854775808.0));
      float s, c;
      sincospif(f, &s, &c);
      cs[0][tid] = c;
      cs[1][tid] = s;
    }
    __syncthreads();
    float c8[8], s8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = kInterleaved ? 4 * l + (i >> 1) : (second ? 8 * l - half + i : 8 * l + i);
      c8[i] = rotates ? cs[0][pair] : 1.0f;
      s8[i] = rotates ? cs[1][pair] : 0.0f;
    }
    const bool stored = static_cast<uint32_t>(slot) < (static_cast<uint32_t>(p.num_pages) << p.page_shift);
    const int page = slot >> p.page_shift;
    const int row = slot & ((1 << p.page_shift) - 1);
    const uint16_t* src = p.qkv + static_cast<int64_t>(n) * p.row_stride;
    for (int h0 = 0; h0 < heads; h0 += kThreads / 16) {
      const int h = h0 + hw;
      const bool live = h < heads;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (live) v = *reinterpret_cast<const uint4*>(src + h * kD + 8 * l);
      const bool is_q = h < p.h_q;
      const bool is_v = h >= p.h_q + p.h_kv;
      float x[8], y[8];
      unpack8(v, x);
      const uint16_t* w = is_q ? p.q_weight : p.k_weight;
      float r = 1.0f;
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      uint4 pv = v;
      if (!kInterleaved) {
        pv.x = __shfl_sync(0xffffffffu, v.x, partner, 16);
        pv.y = __shfl_sync(0xffffffffu, v.y, partner, 16);
        pv.z = __shfl_sync(0xffffffffu, v.z, partner, 16);
        pv.w = __shfl_sync(0xffffffffu, v.w, partner, 16);
      }
      if (!live) continue;
      if (!is_v) {
        unpack8(pv, y);
        if (w) {
          r = rsqrtf(ss * (1.0f / kD) + p.eps);
          float wx[8], wy[8];
          unpack8(*reinterpret_cast<const uint4*>(w + 8 * l), wx);
          unpack8(*reinterpret_cast<const uint4*>(w + 8 * (rotates ? partner : l)), wy);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] *= r * wx[i];
            y[i] *= r * wy[i];
          }
        }
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (kInterleaved)
            z[i] = (i & 1) ? fmaf(x[i], c8[i], x[i - 1] * s8[i]) : fmaf(x[i], c8[i], -x[i + 1] * s8[i]);
          else
            z[i] = fmaf(x[i], c8[i], second ? y[i] * s8[i] : -y[i] * s8[i]);
        }
        v = rotates || w ? pack8(rotates ? z : x) : v;
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + (static_cast<int64_t>(n) * p.h_q + h) * kD + 8 * l) = v;
      } else if (stored) {
        const int j = is_v ? h - p.h_q - p.h_kv : h - p.h_q;
        uint16_t* cache = is_v ? p.v_cache : p.k_cache;
        const int64_t at = (((static_cast<int64_t>(page) * p.h_kv + j) << p.page_shift) + row) * kD + 8 * l;
        *reinterpret_cast<uint4*>(cache + at) = v;
      }
    }
    __syncthreads();
  }
}

}  // namespace qk

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& args, int num_sms, cudaStream_t stream) {
  const int grid = args.N < num_sms * 8 ? args.N : num_sms * 8;
  return args.interleaved
             ? launch_pdl(qk::qk_norm_rope_kernel<true>, dim3(grid), dim3(qk::kThreads), 0, stream, args)
             : launch_pdl(qk::qk_norm_rope_kernel<false>, dim3(grid), dim3(qk::kThreads), 0, stream, args);
}

}  // namespace moe
