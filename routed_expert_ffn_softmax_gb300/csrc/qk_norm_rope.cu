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
// A warp takes a token, or a run of its heads when there are few tokens, and needs no other warp: its lanes compute the
// token's 64 sines and cosines and share them through shared memory, and kUnroll pairs of heads are loaded before the
// first is worked on. (A block per token, with two block barriers around the sines, took 115 us for 8191 tokens of
// 64 + 8 heads.) Partial and interleaved rotations take the first kernel below, with the partner shuffled in: 8191 tokens
// of 64 + 8 heads in 59 us interleaved and 69 in halves of 32, where the full rotation in halves takes 56 (44.6 at the copy
// rate).
//
// The angle: inv_freq / (2 pi) is kept as a 64-bit fraction of a turn (computed in fp64, rounded once), so
// pos * fraction modulo 2^64 is the angle modulo one turn without any loss for large pos, and sin and cos are taken of a
// reduced argument. What remains is the fraction's error: 1 / (2 pi) and the product round in fp64 (2^-53 of |inv_freq| /
// (2 pi) each), and so does the step into [0, 1) (2^-54), in all below max(1, |inv_freq|) * 2^-53 turns for each position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_device.cuh"
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

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ldg_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint2 ldg_stream8(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The fraction of a turn that one position adds, in units of 2^-64 turns (modulo whole turns).
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  double f = static_cast<double>(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
  f -= floor(f);                                                      // [0, 1)
  return static_cast<uint64_t>(__double2ull_rn(f * 18446744073709551616.0));
}

constexpr int kUnroll = 4;

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rope_kernel(const QkNormRopeArgs p, int parts, int part_heads) {
  __shared__ __align__(16) float cs[kThreads / 32][2][kD / 2];  // cos, sin of each warp's token
  const int lane = threadIdx.x & 31;
  const int l = lane & 15;       // dimensions 8 l .. 8 l + 7
  const int hw = lane >> 4;      // which of the two heads
  float(*my)[kD / 2] = cs[threadIdx.x >> 5];
  const int half = p.rot >> 1;
  pdl_wait_predecessor();
  pdl_allow_successor();

  uint64_t turn[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) turn[i] = lane + 32 * i < half ? turn_fraction(p.inv_freq[lane + 32 * i]) : 0;
  // the lane's role in the rotation: first (a) or second (b) of its pairs, or untouched
  const bool rotates = 8 * l < p.rot;
  const bool second = !kInterleaved && 8 * l >= half;
  const int partner = kInterleaved || !rotates ? l : (second ? l - (half >> 3) : l + (half >> 3));
  const int pair0 = kInterleaved ? 4 * l : (second ? 8 * l - half : 8 * l);
  const int heads = p.h_q + 2 * p.h_kv;
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  // the weights of the lane's dimensions and of its partner's
  uint4 wq = ones, wqp = ones, wk = ones, wkp = ones;
  if (p.q_weight) {
    wq = *reinterpret_cast<const uint4*>(p.q_weight + 8 * l);
    wqp = *reinterpret_cast<const uint4*>(p.q_weight + 8 * partner);
  }
  if (p.k_weight) {
    wk = *reinterpret_cast<const uint4*>(p.k_weight + 8 * l);
    wkp = *reinterpret_cast<const uint4*>(p.k_weight + 8 * partner);
  }

  const int64_t items = static_cast<int64_t>(p.N) * parts;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int n = static_cast<int>(it / parts);
    const int first = static_cast<int>(it - static_cast<int64_t>(n) * parts) * part_heads;
    const int last = min(heads, first + part_heads);
    const uint16_t* src = p.qkv + static_cast<int64_t>(n) * p.row_stride + 8 * l;
    const int pos = p.positions[n];
    const int slot = p.slots[n];
    uint4 v[kUnroll];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + 2 * u + hw;
        v[u] = h < last ? ldg_stream(src + h * kD) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    load(first);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = lane + 32 * i;
      if (x < half) {
        const uint64_t a = turn[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
        // signed fraction of a turn in [-1/2, 1/2) times two, for sincospi; converted with one rounding
        const float f = static_cast<float>(static_cast<int64_t>(a)) * (1.0f / 9223372036854775808.0f);
        float s, c;
        sincospif(f, &s, &c);
        my[0][x] = c;
        my[1][x] = s;
      }
    }
    __syncwarp();
    float c8[8], s8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = kInterleaved ? pair0 + (i >> 1) : pair0 + i;
      c8[i] = rotates ? my[0][pair] : 0.0f;
      s8[i] = rotates ? (second || (kInterleaved && (i & 1)) ? my[1][pair] : -my[1][pair]) : 0.0f;
    }
    __syncwarp();  // before the next token's overwrite these
    const bool stored = static_cast<uint32_t>(slot) < (static_cast<uint32_t>(p.num_pages) << p.page_shift);
    // this token's row of head 0 in the caches
    const int64_t row = ((static_cast<int64_t>(slot >> p.page_shift) * p.h_kv << p.page_shift) +
                         (slot & ((1 << p.page_shift) - 1))) * kD + 8 * l;
    for (int h0 = first; h0 < last; h0 += 2 * kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) w[u] = v[u];
      if (h0 + 2 * kUnroll < last) load(h0 + 2 * kUnroll);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (h0 + 2 * u >= last) break;
        const int h = h0 + 2 * u + hw;
        const bool is_q = h < p.h_q;
        const bool is_v = h >= p.h_q + p.h_kv;
        uint4 o = w[u];
        float x[8], y[8];
        unpack8(o, x);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (!kInterleaved) {
          uint4 q;
          q.x = __shfl_sync(0xffffffffu, o.x, partner, 16);
          q.y = __shfl_sync(0xffffffffu, o.y, partner, 16);
          q.z = __shfl_sync(0xffffffffu, o.z, partner, 16);
          q.w = __shfl_sync(0xffffffffu, o.w, partner, 16);
          unpack8(q, y);
        }
        if (h >= last) continue;
        if (!is_v) {
          if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
            const float r = rsqrtf(ss * (1.0f / kD) + p.eps);
            float wx[8], wy[8];
            unpack8(is_q ? wq : wk, wx);
            unpack8(is_q ? wqp : wkp, wy);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] *= r * wx[i];
              if (!kInterleaved) y[i] *= r * wy[i];
            }
          }
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = rotates ? fmaf(x[i], c8[i], (kInterleaved ? x[i ^ 1] : y[i]) * s8[i]) : x[i];
          o = pack8(z);
        }
        if (is_q) {
          *reinterpret_cast<uint4*>(p.q_out + (static_cast<int64_t>(n) * p.h_q + h) * kD + 8 * l) = o;
        } else if (stored) {
          const int j = is_v ? h - p.h_q - p.h_kv : h - p.h_q;
          *reinterpret_cast<uint4*>((is_v ? p.v_cache : p.k_cache) + row + (static_cast<int64_t>(j) << p.page_shift) * kD) = o;
        }
      }
    }
  }
}

// The common case, rot = 128 in halves: a lane holds dimensions 4 l .. + 3 and 64 + 4 l .. + 3, so that both values of
// its four pairs are its own: no partner's value is shuffled in or normed twice. Two 8-byte loads and stores per head,
// arithmetic two values an instruction.
constexpr int kUnrollHalves = 4;

__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_halves_kernel(const QkNormRopeArgs p, int parts, int part_heads) {
  __shared__ __align__(16) float cs[kThreads / 32][2][kD / 2];  // cos, sin of each warp's token
  const int lane = threadIdx.x & 31;
  const int l = lane & 15;
  const int hw = lane >> 4;  // which of the two heads
  float(*my)[kD / 2] = cs[threadIdx.x >> 5];
  pdl_wait_predecessor();
  pdl_allow_successor();

  const uint64_t turn[2] = {turn_fraction(p.inv_freq[lane]), turn_fraction(p.inv_freq[lane + 32])};
  const uint2 ones = make_uint2(0x3f803f80u, 0x3f803f80u);
  uint2 w[2][2] = {{ones, ones}, {ones, ones}};  // [q, k][first, second half]
  if (p.q_weight) {
    w[0][0] = *reinterpret_cast<const uint2*>(p.q_weight + 4 * l);
    w[0][1] = *reinterpret_cast<const uint2*>(p.q_weight + 64 + 4 * l);
  }
  if (p.k_weight) {
    w[1][0] = *reinterpret_cast<const uint2*>(p.k_weight + 4 * l);
    w[1][1] = *reinterpret_cast<const uint2*>(p.k_weight + 64 + 4 * l);
  }
  auto pair = [](uint32_t v) { return pack_f32x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); };
  auto round2 = [](uint64_t v) {
    float a, b;
    unpack_f32x2(v, a, b);
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  const int heads = p.h_q + 2 * p.h_kv;
  const int64_t items = static_cast<int64_t>(p.N) * parts;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int n = static_cast<int>(it / parts);
    const int first = static_cast<int>(it - static_cast<int64_t>(n) * parts) * part_heads;
    const int last = min(heads, first + part_heads);
    const uint16_t* src = p.qkv + static_cast<int64_t>(n) * p.row_stride + 4 * l;
    const int pos = p.positions[n];
    const int slot = p.slots[n];
    uint2 v[kUnrollHalves][2];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kUnrollHalves; ++u) {
        const int h = h0 + 2 * u + hw;
        v[u][0] = h < last ? ldg_stream8(src + h * kD) : make_uint2(0u, 0u);
        v[u][1] = h < last ? ldg_stream8(src + h * kD + 64) : make_uint2(0u, 0u);
      }
    };
    load(first);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = turn[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
      // signed fraction of a turn in [-1/2, 1/2) times two, for sincospi; converted with one rounding
      const float f = static_cast<float>(static_cast<int64_t>(a)) * (1.0f / 9223372036854775808.0f);
      sincospif(f, &my[1][lane + 32 * i], &my[0][lane + 32 * i]);
    }
    __syncwarp();
    uint64_t c[2], s[2], ns[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 cc = *reinterpret_cast<const float2*>(&my[0][4 * l + 2 * i]);
      const float2 ss = *reinterpret_cast<const float2*>(&my[1][4 * l + 2 * i]);
      c[i] = pack_f32x2(cc.x, cc.y);
      s[i] = pack_f32x2(ss.x, ss.y);
      ns[i] = pack_f32x2(-ss.x, -ss.y);
    }
    __syncwarp();  // before the next token's overwrite these
    const bool stored = static_cast<uint32_t>(slot) < (static_cast<uint32_t>(p.num_pages) << p.page_shift);
    // this token's row of head 0 in the caches
    const int64_t row = ((static_cast<int64_t>(slot >> p.page_shift) * p.h_kv << p.page_shift) +
                         (slot & ((1 << p.page_shift) - 1))) * kD + 4 * l;
    for (int h0 = first; h0 < last; h0 += 2 * kUnrollHalves) {
      uint2 o[kUnrollHalves][2];
#pragma unroll
      for (int u = 0; u < kUnrollHalves; ++u) {
        o[u][0] = v[u][0];
        o[u][1] = v[u][1];
      }
      if (h0 + 2 * kUnrollHalves < last) load(h0 + 2 * kUnrollHalves);
#pragma unroll
      for (int u = 0; u < kUnrollHalves; ++u) {
        if (h0 + 2 * u >= last) break;
        const int h = h0 + 2 * u + hw;
        const bool is_q = h < p.h_q;
        const bool is_v = h >= p.h_q + p.h_kv;
        uint64_t x[4] = {pair(o[u][0].x), pair(o[u][0].y), pair(o[u][1].x), pair(o[u][1].y)};
        uint64_t sq = mul_f32x2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) sq = fma_f32x2(x[i], x[i], sq);
        float s0, s1;
        unpack_f32x2(sq, s0, s1);
        float sum = s0 + s1;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (h >= last) continue;
        if (!is_v) {
          if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
            const float r = rsqrtf(sum * (1.0f / kD) + p.eps);
            const uint64_t r2 = pack_f32x2(r, r);
            const uint2 wa = is_q ? w[0][0] : w[1][0], wb = is_q ? w[0][1] : w[1][1];
            x[0] = mul_f32x2(x[0], mul_f32x2(r2, pair(wa.x)));
            x[1] = mul_f32x2(x[1], mul_f32x2(r2, pair(wa.y)));
            x[2] = mul_f32x2(x[2], mul_f32x2(r2, pair(wb.x)));
            x[3] = mul_f32x2(x[3], mul_f32x2(r2, pair(wb.y)));
          }
          o[u][0].x = round2(fma_f32x2(x[0], c[0], mul_f32x2(x[2], ns[0])));
          o[u][0].y = round2(fma_f32x2(x[1], c[1], mul_f32x2(x[3], ns[1])));
          o[u][1].x = round2(fma_f32x2(x[2], c[0], mul_f32x2(x[0], s[0])));
          o[u][1].y = round2(fma_f32x2(x[3], c[1], mul_f32x2(x[1], s[1])));
        }
        uint16_t* to = nullptr;
        if (is_q) {
          to = p.q_out + (static_cast<int64_t>(n) * p.h_q + h) * kD + 4 * l;
        } else if (stored) {
          const int j = is_v ? h - p.h_q - p.h_kv : h - p.h_q;
          to = (is_v ? p.v_cache : p.k_cache) + row + (static_cast<int64_t>(j) << p.page_shift) * kD;
        }
        if (to) {
          *reinterpret_cast<uint2*>(to) = o[u][0];
          *reinterpret_cast<uint2*>(to + 64) = o[u][1];
        }
      }
    }
  }
}

}  // namespace qk

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& args, int num_sms, cudaStream_t stream) {
  // A token's heads are cut into equal runs (of pairs of heads), each a warp's work: the runs that make the rounds over
  // the resident warps cheapest, counting a run's start (positions, sines, the first loads) as 4 pairs. 8191 tokens of
  // 72 heads: 61 us uncut (a third of the warps idle in the last round), 56 us (5.4 TB/s) as chosen here.
  const bool halves = args.rot == qk::kD && !args.interleaved;
  const int64_t warps = static_cast<int64_t>(num_sms) * (halves ? 3 : 2) * (qk::kThreads / 32);
  const int pairs = (args.h_q + 2 * args.h_kv + 1) / 2;
  int parts = 1, part_heads = 2 * pairs;
  int64_t least = 0;
  for (int run = pairs; run >= 1; run -= run > 64 ? run / 64 : 1) {
    const int n = (pairs + run - 1) / run;
    const int64_t cost = (args.N * static_cast<int64_t>(n) + warps - 1) / warps * (run + 4);
    if (least == 0 || cost < least) {
      least = cost;
      parts = n;
      part_heads = 2 * run;
    }
  }
  const int64_t blocks = (static_cast<int64_t>(args.N) * parts + qk::kThreads / 32 - 1) / (qk::kThreads / 32);
  const int64_t resident = warps / (qk::kThreads / 32);
  const int grid = static_cast<int>(blocks < resident ? blocks : resident);
  auto kernel = halves ? qk::qk_norm_rope_halves_kernel
                       : (args.interleaved ? qk::qk_norm_rope_kernel<true> : qk::qk_norm_rope_kernel<false>);
  return launch_pdl(kernel, dim3(grid), dim3(qk::kThreads), 0, stream, args, parts, part_heads);
}

}  // namespace moe
