// Per-head norm of queries and keys, position rotation and the cache store in one pass
// (include/paged/moe_paged.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * inv_freq
//
// Each value is read once and written once (2 B each way), so HBM bounds it. A head's 128 values are 16 lanes of
// 16 bytes, so a warp holds two heads and one load or store instruction moves 512 contiguous bytes; the mean comes by
// shuffles. The partner of a rotated pair sits rot / 2 dimensions away in another lane and comes by
// shuffling the packed bf16 inputs (four shuffles for eight values); the partner's norm factor is the same, its
// weight is kept beside the lane's own. Only the result is rounded.
//
// A warp takes a token, or a run of its heads when there are few tokens, and needs no other warp: its lanes compute the
// token's 64 sines and cosines and share them through shared memory, and kUnroll pairs of heads are loaded before the
// first is worked on. (A block per token, with two block barriers around the sines, took 115 us for 8191 tokens of
// 64 + 8 heads.) Partial and interleaved rotations take the first kernel below, with the partner shuffled in: 8191 tokens
// of 64 + 8 heads in 53 us interleaved and 60 in halves of 32, where the full rotation in halves takes 53 (44.6 at the copy
// rate; 5.7 TB/s).
//
// Four heads' sums of squares are reduced together (9 shuffles instead of 16, one root instead of four): halves of 32 65 -> 60 us.
// The next heads are loaded after that in the kernel for full rotations, which has no registers for both.
// (With 80 a thread that kernel spills 4 bytes, for several axes or a 4-bit cache 24, for both 40; the first one, with 128, up to 48.)
//
// Positions with several axes (kAxes; include/paged/moe_norm.h): the lanes that compute a pair's sine and cosine look up the
// pair's axis once and load that axis's position per token; nothing else differs (8191 tokens of 64 + 8 heads: 54 us).
//
// A 4-bit cache (kFour; include/paged/moe_kv4.h): keys and values are rounded to bf16 as for the bf16 cache, then the 8 (or
// 4) lanes that hold a group of 32 dimensions share its largest magnitude, taken of the bits as whole numbers (two groups
// in one shuffle; NaN stands above infinity), and lanes that hold parts of the same stored bytes exchange them, so that a
// head's 64 bytes of codes leave in 8- or 16-byte stores. Every code is that of the exact quotient: see codes2. 9603 tokens of
// 32 + 2 8 heads in 48 us (4.3 TB/s; issue slots 60% used; their bf16 store takes 42 for more bytes: the rest is instructions).
//
// The angle: inv_freq / (2 pi) is kept as a 64-bit fraction of a turn (computed in fp64, rounded once), so
// pos * fraction modulo 2^64 is the angle modulo one turn without any loss for large pos, and sin and cos are taken of a
// reduced argument. What remains is the fraction's error: 1 / (2 pi) and the product round in fp64 (2^-53 of |inv_freq| /
// (2 pi) each), and so does the step into [0, 1) (2^-54), in all below max(1, |inv_freq|) * 2^-53 turns for each position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "paged_device.cuh"
#include "moe_launch.h"
#include "step_launch.h"

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

__device__ __forceinline__ uint64_t pair_of(uint32_t v) {  // two packed bf16 values in fp32
  return pack_f32x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// The scales of two groups whose largest magnitudes are packed here: a 7th, in bf16. (The product with the rounded 1/7 is within
// 2^-23 of the 7th, which is representable or 2^-12 or more away from where rounding turns.) Infinity times 0 makes it NaN.
__device__ __forceinline__ uint32_t scales2(uint32_t top) {
  const uint64_t x = pair_of(top);
  const uint64_t seventh = fma_f32x2(x, pack_f32x2(1.0f / 7.0f, 1.0f / 7.0f), mul_f32x2(x, pack_f32x2(0.0f, 0.0f)));
  float a, b;
  unpack_f32x2(seventh, a, b);
  const __nv_bfloat162 s = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&s);
}
// What x is multiplied with for its code: 1 / s, within 2^-23. (Infinity for scales that code4_tiny deals with.)
__device__ __forceinline__ float code_factor(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}
// round(x / s) + 8, halves to even, in the lowest 4 bits, of two values. x and s have 8 bits each, so a quotient (at most 7.04)
// that is not a half is 2^-10 or more away from one, and x times the factor is within 2^-20 of it: rounding that to
// multiples of 2^-11 first makes a half of what is one and no half of what is none. (Infinite and NaN groups get some code.)
__device__ __forceinline__ void codes2(uint64_t x, uint64_t factor, uint32_t& a, uint32_t& b) {
  uint64_t v = fma_f32x2(x, factor, pack_f32x2(6144.0f, 6144.0f));  // 1.5 2^12
  v = add_f32x2(v, pack_f32x2(-6144.0f, -6144.0f));
  v = add_f32x2(v, pack_f32x2(12582920.0f, 12582920.0f));           // 1.5 2^23 + 8
  float fa, fb;
  unpack_f32x2(v, fa, fb);
  a = __float_as_uint(fa);
  b = __float_as_uint(fb);
}
// The same for scales below 2^-100, whose reciprocals may overflow and whose few bits let quotients pass 7.
__device__ __forceinline__ uint32_t code4_tiny(float x, float s) {
  return static_cast<uint32_t>(min(max(s == 0.0f ? 0 : __float2int_rn(__fdiv_rn(x, s)), -7), 7) + 8);
}
constexpr float kTinyScale = 7.8886e-31f;  // 2^-100
// Eight codes, one behind the other in fours: the first four in the lower half. (What codes2 has above a code's 4 bits are
// multiples of 2^16.)
__device__ __forceinline__ uint32_t nibbles8(const uint32_t (&n)[8]) {
  const uint32_t a = n[0] + (n[1] << 4) + (n[2] << 8) + (n[3] << 12), b = n[4] + (n[5] << 4) + (n[6] << 8) + (n[7] << 12);
  return __byte_perm(a, b, 0x5410);
}

// The magnitudes' bits of two packed bf16 values, and the larger of two such in each half.
__device__ __forceinline__ uint32_t magnitudes(uint32_t v) { return v & 0x7fff7fffu; }

// Where a token's rows are in the 4-bit cache: those of head 0, what a head adds, and a row's scales seen from its codes.
struct Kv4Place {
  uint8_t* codes;
  int64_t head;
  int scales;
  __device__ __forceinline__ Kv4Place(const QkNormRopeArgs& p, int slot) {
    const int in_page = slot & ((1 << p.page_shift) - 1);
    head = static_cast<int64_t>(kKv4Block) << (p.page_shift - 4);
    codes = p.kv4 + static_cast<int64_t>(slot >> p.page_shift) * p.h_kv * head + (in_page >> 4) * kKv4Block +
            (in_page & 15) * kKv4RowBytes;
    scales = kKv4Scales - (in_page & 15) * (kKv4RowBytes - 8);
  }
};

// Two heads' 128 values each in 4 bits, from the 16 lanes that hold 8 of them each (all of a warp, lane l dimensions 8 l ..):
// four lanes share a group, and lanes l, l + 4, l + 8, l + 12 hold the four groups' parts of the same 16 bytes.
__device__ __forceinline__ void store4_eight(uint8_t* codes, int scales, const uint4& o, bool stored, int l) {
  const uint32_t v[4] = {o.x, o.y, o.z, o.w};
  uint32_t top = __vmaxu2(__vmaxu2(magnitudes(v[0]), magnitudes(v[1])), __vmaxu2(magnitudes(v[2]), magnitudes(v[3])));
  top = max(top << 16, top & 0xffff0000u);
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  const uint32_t sb = scales2(top);  // (in the upper half)
  const float s = __uint_as_float(sb & 0xffff0000u);
  uint32_t n[8];
  const float factor = code_factor(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) codes2(pair_of(v[i]), pack_f32x2(factor, factor), n[2 * i], n[2 * i + 1]);
  if (s < kTinyScale) {
    float x[8];
    unpack8(o, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = code4_tiny(x[i], s);
  }
  const uint32_t c = nibbles8(n);
  uint32_t cw[4], sw[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    cw[w] = __shfl_sync(0xffffffffu, c, (l & 3) + 4 * w, 16);
    sw[w] = __shfl_sync(0xffffffffu, sb, 4 * w, 16);
  }
  if (!stored || l >= 4) return;
  *reinterpret_cast<uint4*>(codes + 16 * l) =
      make_uint4(__byte_perm(cw[0], cw[1], 0x5410), __byte_perm(cw[2], cw[3], 0x5410), __byte_perm(cw[0], cw[1], 0x7632),
                 __byte_perm(cw[2], cw[3], 0x7632));
  if (l == 0)
    *reinterpret_cast<uint2*>(codes + scales) = make_uint2(__byte_perm(sw[0], sw[1], 0x7632), __byte_perm(sw[2], sw[3], 0x7632));
}

// The same where lane l holds dimensions 4 l .. + 3 (a) and 64 + 4 l .. + 3 (b): eight lanes share two groups, lanes l and
// l + 8 the same 8 bytes.
__device__ __forceinline__ void store4_halves(uint8_t* codes, int scales, const uint2& a, const uint2& b, bool stored, int l) {
  const uint32_t ma = __vmaxu2(magnitudes(a.x), magnitudes(a.y)), mb = __vmaxu2(magnitudes(b.x), magnitudes(b.y));
  uint32_t top = __vmaxu2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));  // group of a, group of b
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, d));
  const uint32_t s = scales2(top);
  const float sa = __uint_as_float(s << 16), sb = __uint_as_float(s & 0xffff0000u);
  const float fa = code_factor(sa), fb = code_factor(sb);
  const uint32_t v[4] = {a.x, a.y, b.x, b.y};
  uint32_t n[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) codes2(pair_of(v[i]), i < 2 ? pack_f32x2(fa, fa) : pack_f32x2(fb, fb), n[2 * i], n[2 * i + 1]);
  if (fminf(sa, sb) < kTinyScale) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      n[i] = code4_tiny(__uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16), i < 4 ? sa : sb);
  }
  const uint32_t c = nibbles8(n);  // lanes below 8: groups 0 and 2, the others 1 and 3
  const uint32_t co = __shfl_xor_sync(0xffffffffu, c, 8);
  const uint32_t so = __shfl_xor_sync(0xffffffffu, s, 8);
  if (!stored || l >= 8) return;
  *reinterpret_cast<uint2*>(codes + 8 * l) = make_uint2(__byte_perm(c, co, 0x5410), __byte_perm(c, co, 0x7632));
  if (l == 0) *reinterpret_cast<uint2*>(codes + scales) = make_uint2(__byte_perm(s, so, 0x5410), __byte_perm(s, so, 0x7632));
}

// The axis of pair x: what it adds to the positions' address, and whether it turns.
struct PairAxis {
  int64_t offset = 0;
  bool turns = true;
  __device__ __forceinline__ PairAxis(const QkNormRopeArgs& p, int x, bool there) {
    if (!there) return;
    const int axis = p.pair_axis[x];
    turns = static_cast<uint32_t>(axis) < static_cast<uint32_t>(p.n_axes);
    offset = turns ? axis * p.axis_stride : 0;
  }
};

// The work of a warp: whole tokens in `rounds` rounds over all warps, and then the next `each` of the list of the remaining
// tokens' units, `token` a token: one for a pair of heads, kKv4Cost for one behind the first `cheap`.
constexpr int kKv4Cost = 2;
struct Shares {
  int rounds, each, token, cheap;
  int first;  // of the remaining tokens
  template <bool kFour>
  __device__ __forceinline__ int pair_at(int units) const {
    return !kFour || units <= cheap ? units : cheap + (units - cheap + kKv4Cost - 1) / kKv4Cost;
  }
};
struct Walk {
  int n, from, to;  // a token, units of it
  int rounds, left;
  __device__ __forceinline__ Walk(const Shares& s) : rounds(s.rounds), left(s.each) {
    const int warp = static_cast<int>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (rounds == 0) rest(s, warp);
    else whole(s, warp);
  }
  __device__ __forceinline__ void whole(const Shares& s, int token) {
    n = token;
    from = 0;
    to = s.token;
  }
  // (The list has fewer than 2^32 units: so many heads do not fit the memory.)
  __device__ __forceinline__ void rest(const Shares& s, int warp) {
    const uint32_t at = static_cast<uint32_t>(warp) * static_cast<uint32_t>(s.each);
    const uint32_t token = at / static_cast<uint32_t>(s.token);
    n = s.first + static_cast<int>(token);
    from = static_cast<int>(at - token * static_cast<uint32_t>(s.token));
    to = min(s.token, from + left);
  }
  __device__ __forceinline__ bool more(int N) const { return n < N; }
  __device__ __forceinline__ void next(const Shares& s, int N) {
    if (rounds > 0) {
      const int step = static_cast<int>(gridDim.x) * (kThreads / 32);
      if (--rounds == 0) rest(s, n + step - s.first);
      else whole(s, n + step);
    } else {
      left -= to - from;
      n = left > 0 ? n + 1 : N;
      from = 0;
      to = min(s.token, left);
    }
  }
};

// The norm factors of four heads from the 16 lanes' parts of their sums of squares (each half-warp its own four): two halving
// steps leave a lane one head's sum, so that a factor is computed once and its root taken once. The order of the additions is
// the same for each.
__device__ __forceinline__ void norm_factors(float eps, int l, float (&part)[4]) {
  const bool hi8 = l & 8, hi4 = l & 4;
  const float a = (hi8 ? part[2] : part[0]) + __shfl_xor_sync(0xffffffffu, hi8 ? part[0] : part[2], 8);
  const float b = (hi8 ? part[3] : part[1]) + __shfl_xor_sync(0xffffffffu, hi8 ? part[1] : part[3], 8);
  float sum = (hi4 ? b : a) + __shfl_xor_sync(0xffffffffu, hi4 ? a : b, 4);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  const float f = rsqrtf(sum * (1.0f / kD) + eps);
#pragma unroll
  for (int u = 0; u < 4; ++u) part[u] = __shfl_sync(0xffffffffu, f, 4 * u, 16);
}

constexpr int kUnroll = 4;

template <bool kInterleaved, bool kAxes, bool kFour>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rope_kernel(const QkNormRopeArgs p, const Shares shares) {
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
  PairAxis axis[2] = {{p, lane, kAxes && lane < half}, {p, lane + 32, kAxes && lane + 32 < half}};
  if constexpr (kAxes) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!axis[i].turns) turn[i] = 0;
  }
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

  for (Walk walk(shares); walk.more(p.N); walk.next(shares, p.N)) {
    const int n = walk.n;
    const int first = 2 * shares.pair_at<kFour>(walk.from), last = min(heads, 2 * shares.pair_at<kFour>(walk.to));
    const uint16_t* src = p.qkv + static_cast<int64_t>(n) * p.row_stride + 8 * l;
    int pos[2];
    pos[0] = p.positions[n + (kAxes ? axis[0].offset : 0)];
    pos[1] = kAxes ? p.positions[n + axis[1].offset] : pos[0];
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
        const uint64_t a = turn[i] * static_cast<uint64_t>(static_cast<int64_t>(pos[i]));
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
    const Kv4Place place(p, stored ? slot : 0);
    for (int h0 = first; h0 < last; h0 += 2 * kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) w[u] = v[u];
      if (h0 + 2 * kUnroll < last) load(h0 + 2 * kUnroll);
      float factor[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float x[8], ss = 0.0f;
        unpack8(w[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        factor[u] = ss;
        asm("" : "+r"(w[u].x), "+r"(w[u].y), "+r"(w[u].z), "+r"(w[u].w));  // (unpacked again, not kept)
      }
      norm_factors(p.eps, l, factor);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int pair = h0 + 2 * u;  // its first head
        if (pair >= last) break;
        const int h = pair + hw;
        const bool is_q = h < p.h_q;
        uint4 o = w[u];
        if (pair < p.h_q + p.h_kv) {  // not both values
          float x[8], y[8];
          unpack8(o, x);
          if (!kInterleaved) {
            uint4 q;
            q.x = __shfl_sync(0xffffffffu, o.x, partner, 16);
            q.y = __shfl_sync(0xffffffffu, o.y, partner, 16);
            q.z = __shfl_sync(0xffffffffu, o.z, partner, 16);
            q.w = __shfl_sync(0xffffffffu, o.w, partner, 16);
            unpack8(q, y);
          }
          if (h < p.h_q + p.h_kv) {
            if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
              const float r = factor[u];
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
        }
        if (pair < p.h_q && is_q && h < last)
          *reinterpret_cast<uint4*>(p.q_out + (static_cast<int64_t>(n) * p.h_q + h) * kD + 8 * l) = o;
        if (pair + 1 >= p.h_q) {
          const bool is_v = h >= p.h_q + p.h_kv;
          const int j = is_v ? h - p.h_q - p.h_kv : h - p.h_q;
          const bool stores = stored && !is_q && h < last;
          if constexpr (kFour)
            store4_eight(place.codes + j * place.head + (is_v ? kKv4Values : 0), place.scales, o, stores, l);
          else if (stores)
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

template <bool kAxes, bool kFour>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_halves_kernel(const QkNormRopeArgs p, const Shares shares) {
  __shared__ __align__(16) float cs[kThreads / 32][2][kD / 2];  // cos, sin of each warp's token
  const int lane = threadIdx.x & 31;
  const int l = lane & 15;
  const int hw = lane >> 4;  // which of the two heads
  float(*my)[kD / 2] = cs[threadIdx.x >> 5];
  pdl_wait_predecessor();
  pdl_allow_successor();

  uint64_t turn[2] = {turn_fraction(p.inv_freq[lane]), turn_fraction(p.inv_freq[lane + 32])};
  const PairAxis axis[2] = {{p, lane, kAxes}, {p, lane + 32, kAxes}};
  if constexpr (kAxes) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!axis[i].turns) turn[i] = 0;
  }
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
  auto round2 = [](uint64_t v) {
    float a, b;
    unpack_f32x2(v, a, b);
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  const int heads = p.h_q + 2 * p.h_kv;
  for (Walk walk(shares); walk.more(p.N); walk.next(shares, p.N)) {
    const int n = walk.n;
    const int first = 2 * shares.pair_at<kFour>(walk.from), last = min(heads, 2 * shares.pair_at<kFour>(walk.to));
    const uint16_t* src = p.qkv + static_cast<int64_t>(n) * p.row_stride + 4 * l;
    int pos[2];
    pos[0] = p.positions[n + (kAxes ? axis[0].offset : 0)];
    pos[1] = kAxes ? p.positions[n + axis[1].offset] : pos[0];
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
      const uint64_t a = turn[i] * static_cast<uint64_t>(static_cast<int64_t>(pos[i]));
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
    const Kv4Place place(p, stored ? slot : 0);
    for (int h0 = first; h0 < last; h0 += 2 * kUnrollHalves) {
      uint2 o[kUnrollHalves][2];
#pragma unroll
      for (int u = 0; u < kUnrollHalves; ++u) {
        o[u][0] = v[u][0];
        o[u][1] = v[u][1];
      }
      float factor[kUnrollHalves];
#pragma unroll
      for (int u = 0; u < kUnrollHalves; ++u) {
        const uint64_t x[4] = {pair_of(o[u][0].x), pair_of(o[u][0].y), pair_of(o[u][1].x), pair_of(o[u][1].y)};
        uint64_t sq = mul_f32x2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) sq = fma_f32x2(x[i], x[i], sq);
        float s0, s1;
        unpack_f32x2(sq, s0, s1);
        factor[u] = s0 + s1;
      }
      norm_factors(p.eps, l, factor);
      if (h0 + 2 * kUnrollHalves < last) load(h0 + 2 * kUnrollHalves);
#pragma unroll
      for (int u = 0; u < kUnrollHalves; ++u) {
        // (unpacked again, not kept)
        asm volatile("" : "+r"(o[u][0].x), "+r"(o[u][0].y), "+r"(o[u][1].x), "+r"(o[u][1].y) : : "memory");
        const int first_h = h0 + 2 * u;
        if (first_h >= last) break;
        const int h = first_h + hw;
        const bool is_q = h < p.h_q;
        if (first_h < p.h_q + p.h_kv) {  // not both values
          uint64_t x[4] = {pair_of(o[u][0].x), pair_of(o[u][0].y), pair_of(o[u][1].x), pair_of(o[u][1].y)};
          if (h < p.h_q + p.h_kv) {
            if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
              const uint64_t r2 = pack_f32x2(factor[u], factor[u]);
              const uint2 wa = is_q ? w[0][0] : w[1][0], wb = is_q ? w[0][1] : w[1][1];
              x[0] = mul_f32x2(x[0], mul_f32x2(r2, pair_of(wa.x)));
              x[1] = mul_f32x2(x[1], mul_f32x2(r2, pair_of(wa.y)));
              x[2] = mul_f32x2(x[2], mul_f32x2(r2, pair_of(wb.x)));
              x[3] = mul_f32x2(x[3], mul_f32x2(r2, pair_of(wb.y)));
            }
            o[u][0].x = round2(fma_f32x2(x[0], c[0], mul_f32x2(x[2], ns[0])));
            o[u][0].y = round2(fma_f32x2(x[1], c[1], mul_f32x2(x[3], ns[1])));
            o[u][1].x = round2(fma_f32x2(x[2], c[0], mul_f32x2(x[0], s[0])));
            o[u][1].y = round2(fma_f32x2(x[3], c[1], mul_f32x2(x[1], s[1])));
          }
        }
        if (first_h < p.h_q && is_q && h < last) {
          uint16_t* to = p.q_out + (static_cast<int64_t>(n) * p.h_q + h) * kD + 4 * l;
          *reinterpret_cast<uint2*>(to) = o[u][0];
          *reinterpret_cast<uint2*>(to + 64) = o[u][1];
        }
        if (first_h + 1 >= p.h_q) {
          const bool is_v = h >= p.h_q + p.h_kv;
          const int j = is_v ? h - p.h_q - p.h_kv : h - p.h_q;
          const bool stores = stored && !is_q && h < last;
          if constexpr (kFour) {
            store4_halves(place.codes + j * place.head + (is_v ? kKv4Values : 0), place.scales, o[u][0], o[u][1], stores, l);
          } else if (stores) {
            uint16_t* to = (is_v ? p.v_cache : p.k_cache) + row + (static_cast<int64_t>(j) << p.page_shift) * kD;
            *reinterpret_cast<uint2*>(to) = o[u][0];
            *reinterpret_cast<uint2*>(to + 64) = o[u][1];
          }
        }
      }
    }
  }
}

}  // namespace qk

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& args, int num_sms, cudaStream_t stream) {
  // Whole tokens in rounds over the warps, as long as there is one for each, in the caches' order; what remains is cut into
  // equal shares, a warp each, of one token where that is hardly more per warp (a start costs as much as some pairs), else
  // across tokens. (Every token cut alike, so that the last round was partly empty: 2000 tokens of 72 heads 17.9 us instead of
  // 16.1, 8191 56.9 instead of 53.2; shares across tokens alone: 16000 105 instead of 99, warps far apart in the caches.)
  // A 4-bit cache has shares across tokens alone, with its heads counted twice: 9603 tokens of 48 heads
  // 49.6 us instead of 52 in rounds.
  // More than a block an SM costs calls that follow one another closely 1 us, so few tokens' warps take two pairs where that
  // avoids it: 64 tokens of 40 heads 3.9 -> 3.2 us (for a 4-bit cache, whose pairs take longer, it does not pay).
  const bool halves = args.rot == qk::kD && !args.interleaved;
  const bool axes = args.pair_axis != nullptr, four = args.kv4 != nullptr;
  constexpr int kPerBlock = qk::kThreads / 32;
  const int64_t sm_warps = static_cast<int64_t>(num_sms) * kPerBlock, warps = sm_warps * (halves ? 3 : 2);
  const int pairs = (args.h_q + 2 * args.h_kv + 1) / 2;
  qk::Shares shares;
  shares.rounds = four ? 0 : static_cast<int>(args.N / warps);
  shares.first = static_cast<int>(shares.rounds * warps);
  const int64_t rest = args.N - shares.first;
  shares.cheap = four ? args.h_q / 2 : pairs;
  shares.token = shares.cheap + (pairs - shares.cheap) * qk::kKv4Cost;
  shares.each = static_cast<int>((rest * shares.token + warps - 1) / warps);
  if (rest > 0 && rest <= warps) {
    const int parts = static_cast<int>(std::min<int64_t>(warps / rest, pairs));
    int cut = (pairs + parts - 1) / parts;
    if (!four && cut == 1 && rest * pairs > sm_warps && rest * ((pairs + 1) / 2) <= sm_warps) cut = 2;
    const int even = static_cast<int>((rest * pairs + warps - 1) / warps);
    if (even <= 2 || cut <= even + (four ? 0 : 1) + 4 * even / pairs) {
      shares.each = cut;
      shares.cheap = shares.token = (pairs + cut - 1) / cut * cut;
    }
  }
  const int64_t used = shares.rounds > 0 ? warps : (rest * shares.token + shares.each - 1) / shares.each;
  const int grid = static_cast<int>((used + kPerBlock - 1) / kPerBlock);
  using Kernel = void (*)(QkNormRopeArgs, qk::Shares);
  static constexpr Kernel kHalves[2][2] = {
      {qk::qk_norm_rope_halves_kernel<false, false>, qk::qk_norm_rope_halves_kernel<false, true>},
      {qk::qk_norm_rope_halves_kernel<true, false>, qk::qk_norm_rope_halves_kernel<true, true>}};
  static constexpr Kernel kGeneral[2][2][2] = {
      {{qk::qk_norm_rope_kernel<false, false, false>, qk::qk_norm_rope_kernel<false, false, true>},
       {qk::qk_norm_rope_kernel<false, true, false>, qk::qk_norm_rope_kernel<false, true, true>}},
      {{qk::qk_norm_rope_kernel<true, false, false>, qk::qk_norm_rope_kernel<true, false, true>},
       {qk::qk_norm_rope_kernel<true, true, false>, qk::qk_norm_rope_kernel<true, true, true>}}};
  const Kernel kernel = halves ? kHalves[axes][four] : kGeneral[args.interleaved][axes][four];
  return launch_pdl(kernel, dim3(grid), dim3(qk::kThreads), 0, stream, args, shares);
}

}  // namespace moe
