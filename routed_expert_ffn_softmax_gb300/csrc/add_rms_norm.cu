// The residual's addition and the root-mean-square norm of a token's row in one pass, the result in bf16 or in 8 bits
// with a scale for 128 dimensions (include/paged/moe_norm.h).
//
//   r = bf16(x + res),  y = r * rsqrt(mean(r^2) + eps) * w,   or  q = round(127 t / T),  t = r w,  T = max |t| of 128
//
// 4 bytes are read and 3 or 4 written per value, so HBM bounds it. A block holds a row in registers: each thread takes
// vectors of 8 values, one or more, and the sum of squares is a block reduction with one barrier. A block keeps its
// part of the weight from row to row and has the next row's loads under way while it works on one. GB300: 8191 rows of 7168 to
// bf16 in 72.6 us (6.47 TB/s, 96% of a copy), 2048 rows of 6144 to 8 bits in 18.7 (4.7 TB/s), 64 rows of 4096 in 2.8.
// What does not fit the registers: 8 vectors a thread (H above 16384) spill 84 to 428 bytes, the 8-bit form with 2 vectors 36.
//
// The codes: the norm's factor is the same for all of a group, so q does not depend on it, and 127 t is exact in fp32
// (8 + 8 + 7 bits). A multiplication with the rounded 127 / T is off by 127 2^-23 < 2^-16 and decides every code but those
// next to a half; a thread that holds one within 2^-14 (one warp in 30) divides all of its eight, correctly rounded, which makes
// a half of no other quotient: with T = B and t = n 2^-j, whole numbers of 16 bits and t <= T, a quotient Q = 127 t / T that is not
// the half h has |Q - h| >= Q / (254 n) (of Q / (254 n 2^-j) for j < 0), more than 2^-24 Q, and so than half a step of Q in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_device.cuh"
#include "moe_launch.h"
#include "step_launch.h"

namespace moe {
namespace norm {

constexpr int kMaxThreads = 512;

__device__ __forceinline__ uint4 load16(const uint16_t* p) {  // read once
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// round(127 t / T) of eight values, halves to even, as bytes; inv = 127 / T rounded.
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float top, float inv) {
  constexpr float kMagic = 12582912.0f;  // 1.5 2^23: a sum with it has the rounded number in its low bits
  uint32_t c[8];
  bool near_half = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float v = fmaf(t[k], inv, kMagic);
    const float e = fmaf(t[k], inv, -(v - kMagic));
    near_half |= !(fabsf(e) <= 0.5f - 1.0f / 16384);  // (so do an inv of infinity, and NaN)
    c[k] = __float_as_uint(v);
  }
  if (near_half) {
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = static_cast<uint32_t>(__float2int_rn(__fdiv_rn(t[k] * 127.0f, top)));  // (0 for NaN)
  }
  auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  };
  return make_uint2(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]));
}

template <int kVecs, bool kAdd, bool kInt8>
__global__ void __launch_bounds__(kMaxThreads, kVecs <= 2 ? 2 : 1) add_rms_norm_kernel(const AddRmsNormArgs p) {
  __shared__ float sums[2][kMaxThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int warps = blockDim.x >> 5;
  const int vecs = p.H >> 3;
  pdl_wait_predecessor();
  pdl_allow_successor();

  uint4 w[kVecs];
  bool mine[kVecs];
  int at[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = tid + i * static_cast<int>(blockDim.x);
    mine[i] = v < vecs;
    at[i] = 8 * (mine[i] ? v : 0);
    w[i] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    if (p.weight && mine[i]) w[i] = *reinterpret_cast<const uint4*>(p.weight + at[i]);
  }
  uint4 a[kVecs], b[kVecs];
  // (N may be up to 2^31 - 1, and a grid more still fits 32 bits without a sign. Addresses take the sign again: without it the form
  // for H above 16384 is 3 to 5% slower in 8 bits.)
  const uint32_t rows = static_cast<uint32_t>(p.N);
  auto load = [&](uint32_t n) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mine[i] && n < rows) {
        b[i] = load16(p.residual + static_cast<int64_t>(static_cast<int>(n)) * p.H + at[i]);
        if (kAdd) a[i] = load16(p.x + static_cast<int64_t>(static_cast<int>(n)) * p.x_stride + at[i]);
      }
    }
  };
  load(blockIdx.x);
  int turn = 0;
  for (uint32_t n = blockIdx.x; n < rows; n += gridDim.x, turn ^= 1) {
    uint32_t r[kVecs][4];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bv[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        r[i][k] = kAdd ? pack(lo(av[k]) + lo(bv[k]), hi(av[k]) + hi(bv[k])) : bv[k];
        ss = fmaf(lo(r[i][k]), lo(r[i][k]), ss);
        ss = fmaf(hi(r[i][k]), hi(r[i][k]), ss);
      }
      if (p.residual_out && mine[i])
        *reinterpret_cast<uint4*>(p.residual_out + static_cast<int64_t>(static_cast<int>(n)) * p.H + at[i]) =
            make_uint4(r[i][0], r[i][1], r[i][2], r[i][3]);
    }
    load(n + gridDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (warps > 1) {
      // (two sets of sums: a warp that is ahead writes the next row's while others read this one's)
      if (lane == 0) sums[turn][warp] = ss;
      __syncthreads();
      ss = lane < warps ? sums[turn][lane] : 0.0f;
#pragma unroll
      for (int o = kMaxThreads / 64; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      ss = __shfl_sync(0xffffffffu, ss, 0);
    }
    const float factor = rsqrtf(ss / static_cast<float>(p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t wv[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      float t[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        t[2 * k] = lo(r[i][k]) * lo(wv[k]);
        t[2 * k + 1] = hi(r[i][k]) * hi(wv[k]);
      }
      const int64_t to = static_cast<int64_t>(static_cast<int>(n)) * p.H + at[i];
      if (p.y && mine[i])
        *reinterpret_cast<uint4*>(p.y + to) = make_uint4(pack(t[0] * factor, t[1] * factor), pack(t[2] * factor, t[3] * factor),
                                                          pack(t[4] * factor, t[5] * factor), pack(t[6] * factor, t[7] * factor));
      if constexpr (kInt8) {
        // as whole numbers the magnitudes keep their order, and NaN stands above infinity
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(t[k]) & 0x7fffffffu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float big = __uint_as_float(top);
        const float inv = top ? 127.0f / big : 0.0f;
        const uint2 codes = codes8(t, big, inv);
        if (mine[i]) {
          *reinterpret_cast<uint2*>(p.q + to) = codes;
          if ((lane & 15) == 0) p.scales[to >> 7] = top ? big * factor / 127.0f : 1.0f;
        }
      }
    }
  }
}

template <bool kAdd, bool kInt8>
cudaError_t launch(const AddRmsNormArgs& a, int num_sms, cudaStream_t stream) {
  const int vecs = a.H / 8;
  const int per = vecs <= kMaxThreads ? 1 : vecs <= 2 * kMaxThreads ? 2 : vecs <= 4 * kMaxThreads ? 4 : 8;
  const int threads = ((vecs + per - 1) / per + 31) / 32 * 32;
  void (*kernel)(AddRmsNormArgs) = per == 1   ? add_rms_norm_kernel<1, kAdd, kInt8>
                                   : per == 2 ? add_rms_norm_kernel<2, kAdd, kInt8>
                                   : per == 4 ? add_rms_norm_kernel<4, kAdd, kInt8>
                                              : add_rms_norm_kernel<8, kAdd, kInt8>;
  int blocks = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, 0);
  if (e != cudaSuccess) return e;
  const int64_t resident = static_cast<int64_t>(num_sms) * (blocks > 0 ? blocks : 1);
  // every block the same number of rows, as near as it goes
  const int64_t rounds = (a.N + resident - 1) / resident;
  const int grid = static_cast<int>((a.N + rounds - 1) / rounds);
  return launch_pdl(kernel, dim3(grid), dim3(threads), 0, stream, a);
}

}  // namespace norm

cudaError_t launch_add_rms_norm(const AddRmsNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.x) return a.q ? norm::launch<true, true>(a, num_sms, stream) : norm::launch<true, false>(a, num_sms, stream);
  return a.q ? norm::launch<false, true>(a, num_sms, stream) : norm::launch<false, false>(a, num_sms, stream);
}

}  // namespace moe
