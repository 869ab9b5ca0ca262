// Decode attention over a paged cache held in 4 bits (include/paged/moe_kv4.h): one query token per sequence, the G query
// heads of a group against each key/value head, under a sliding window with sink tokens.
//
// What bounds it. A key costs 144 bytes of HBM a key/value head (72 for K, 72 for V), 3.6 times less than in bf16, so an
// SM has 6.2 cycles of memory time per key. Tensor-core operands would have to pass through shared memory as 16-bit tiles:
// 512 bytes written and 512 read per key, 8 cycles of the shared memory's 128 bytes a cycle, more than the memory time. So
// the codes go from shared memory straight into registers as mma.sync operands: the key axis is the M side of both
// products, so a group of up to 8 heads (the N side) wastes nothing.
//     S [16 keys x 8 heads]  = codes(K) [16 x 32] . q [32 x 8]           for each of the 4 groups of 32 dimensions
//     O [16 dims x 8 heads] += codes(V)^T [16 x 16 keys] . (p s) [16 x 8]  s the value scale of the group the dims are in
// K's scales multiply the four group sums in fp32; V's scales go into the probabilities, once per group.
//
// Unpacking. 16 bits of a row hold four codes of a group; two such of the same row (K) or of two keys (V) in one register
// give all four fp16 pairs with four masks and a shift. K's are left as fp16 subnormals n 2^-24 (n 2^-20 for the odd codes,
// whose queries are a 16th): exact products, n = c + 8, and -8 sum(q) is where the accumulator starts. V's are turned into
// exact c by an exponent and a subtraction, as a sum over many keys must not carry an offset.
//
// Range. p s must fit fp16, whatever the scales are: the softmax reference R of a head bounds score + log2(largest scale of
// the key) instead of the score alone, p = 2^(score - R) is held in fp32, and R is raised (outputs and sums rescaled) only
// when a product would pass 2^15. R starts 2^6 below the largest, so products keep fp16's full precision down to 2^-20 of it.
//
// Work split: as in gqa_decode.cu, the key tiles (128 keys) of all segments form one list of which each CTA takes a
// contiguous share; the pieces of a cut segment are joined in CTA order by the last to arrive.
//
// Per CTA: 8 warps, each with 16 keys of a tile and a running (R, sum, O) of its own, joined through shared memory at the
// end of a piece; one warp that brings tiles with bulk copies, a page's 16 tokens of keys and values in one, 2304 bytes.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "gqa_paged.cuh"
#include "paged_device.cuh"
#include "step_launch.h"

namespace moe {
namespace kv4 {

using gqa::DecodeSpan;
using gqa::kFold;
using gqa::kKeys;
using gqa::span_of;

constexpr int kD = 128;
constexpr int kWarps = 8;                  // that compute; the last warp loads
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kWork = 32 * kWarps;
constexpr int kChunk = kKv4Tokens;         // keys of a warp in a tile
constexpr int kChunks = kKeys / kChunk;
constexpr int kStageBytes = kChunks * kKv4Block;
constexpr int kRow = kD + 4;               // floats of a head's outputs in the join buffer (no bank conflicts)
constexpr float kHigh = 15.0f;             // log2 of what p s may reach
constexpr float kStart = 6.0f;             // log2 of the largest p s right after a reference is set
constexpr float kLeastScale = -60.0f;      // log2: smaller value scales count as this when the reference is set
static_assert(kChunks == kWarps && kFold == kChunk, "a warp takes a chunk of each tile");

template <int kNT>
struct Smem {
  static constexpr int kStages = kNT == 1 ? 9 : 7;
  static constexpr int kJoin = kStages * kStageBytes;                    // [kWarps][8 kNT][kRow] floats
  static constexpr int kRef = kJoin + kWarps * 8 * kNT * kRow * 4;       // [2][2][kWarps][16] floats: R, sum
  static constexpr int kBars = kRef + 2 * 2 * kWarps * 16 * 4;           // full, empty
  static constexpr int kBad = kBars + 2 * kStages * 8;                   // [kStages] chunks that read as zeros
  static constexpr int kMisc = (kBad + kStages * 4 + 15) / 16 * 16;      // 16 ints
  static constexpr int kPre = kMisc + 64;
  static constexpr int kLens = kPre + (kGqaMaxSeqs + 4) * 4;
  static constexpr int kBytes = kLens + kGqaMaxSeqs * 4;
  static_assert(kBytes <= 232448, "dynamic shared memory per CTA");
};

struct Params {
  const uint16_t* q;
  const uint8_t* cache;
  const int32_t* seq_lens;
  uint16_t* out;
  float* partials;
  int32_t* counters;
  int32_t* status;
  int B, h_q, h_kv, G, L_cap;
  float scale_log2;
  PagedKv kv;
  int give_up_tile;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements, a row's pair per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// (n + 1024 or n + 64) - (1032 or 72) in both halves.
__device__ __forceinline__ uint32_t sub2(uint32_t v, uint32_t bias) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t code_lo(uint32_t v) { return sub2((v & 0x000f000fu) | 0x64006400u, 0x64086408u); }
__device__ __forceinline__ uint32_t code_hi(uint32_t v) { return sub2((v & 0x00f000f0u) | 0x54005400u, 0x54805480u); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// A warp's queries of up to 8 kNT heads as mma operands, and what goes with them.
template <int kNT>
struct Queries {
  uint32_t b[kNT][4][2][2];  // [heads][group of dims][k16 step][register]
  float start[kNT][4][2];    // -8 sum(q) of the group for heads 2 t, 2 t + 1 (in accumulator units)
  float unit[kNT][2];        // accumulator units to log2 scores

  // q at the group's first head; a lane (g, t) holds head g's dimensions 32 w + 8 t .. + 7.
  __device__ __forceinline__ void load(const uint16_t* q, int G, float scale_log2, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      uint4 v[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[w] = make_uint4(0u, 0u, 0u, 0u);
        if (8 * nt + g < G) v[w] = *reinterpret_cast<const uint4*>(q + (8 * nt + g) * kD + 32 * w + 8 * t);
      }
      uint32_t top = 0;  // the largest magnitude's bits (NaN above infinity)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max((x[i] & 0x7fffu) << 16, x[i] & 0x7fff0000u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest query in [2^13, 2^14)
      const int e = top == 0 ? 0 : min(max(static_cast<int>(top >> 23) - 127, -100), 100);
      const float to = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
      const float back = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 24 - 13 + e) << 23);
      float sum[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf_lo(x[i]) * to;
          f[2 * i + 1] = bf_hi(x[i]) * (to * 0.0625f);
        }
        sum[w] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = __floats2half2_rn(f[i], f[i + 4]);
          b[nt][w][i >> 1][i & 1] = *reinterpret_cast<const uint32_t*>(&h);
          const float2 r = __half22float2(h);
          sum[w] = fmaf(r.x + r.y, (i & 1) ? 16.0f : 1.0f, sum[w]);
        }
        sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 1);
        sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 2);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int from = 4 * (2 * t + h);
#pragma unroll
        for (int w = 0; w < 4; ++w) start[nt][w][h] = __shfl_sync(0xffffffffu, sum[w], from) * -4.76837158203125e-07f;  // -8 2^-24
        unit[nt][h] = __shfl_sync(0xffffffffu, back, from);
      }
    }
  }
};

// A warp's running state: per lane heads 2 t, 2 t + 1 of each 8, and of the outputs dimensions 32 w + 4 g .. + 3.
template <int kNT>
struct State {
  float ref[kNT][2], sum[kNT][2];
  float o[kNT][8][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      ref[nt][0] = ref[nt][1] = -FLT_MAX;
      sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][m][i] = 0.0f;
    }
  }

  // 16 keys at `at` in shared memory; see0, see1: whether the query sees keys g and g + 8; zero: all read as zeros.
  __device__ __forceinline__ void add(const Queries<kNT>& q, const uint8_t* at, bool see0, bool see1, bool zero, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint4 k0 = *reinterpret_cast<const uint4*>(at + g * kKv4RowBytes + 16 * t);
    const uint4 k1 = *reinterpret_cast<const uint4*>(at + (g + 8) * kKv4RowBytes + 16 * t);
    uint2 ks0 = *reinterpret_cast<const uint2*>(at + kKv4Scales + 8 * g);
    uint2 ks1 = *reinterpret_cast<const uint2*>(at + kKv4Scales + 8 * (g + 8));
    const uint8_t* va = at + kKv4Values;
    uint2 vs0 = *reinterpret_cast<const uint2*>(va + kKv4Scales + 8 * g);
    uint2 vs1 = *reinterpret_cast<const uint2*>(va + kKv4Scales + 8 * (g + 8));
    if (zero) ks0 = ks1 = vs0 = vs1 = make_uint2(0u, 0u);
    if (!see0) vs0 = make_uint2(0u, 0u);  // what stands in rows not seen may be NaN
    if (!see1) vs1 = make_uint2(0u, 0u);

    float x[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t sel = (w & 1) ? 0x7632u : 0x5410u;
      const uint32_t r0 = __byte_perm(w < 2 ? k0.x : k0.y, w < 2 ? k0.z : k0.w, sel);
      const uint32_t r1 = __byte_perm(w < 2 ? k1.x : k1.y, w < 2 ? k1.z : k1.w, sel);
      const uint32_t r0h = r0 >> 8, r1h = r1 >> 8;
      const float s0 = (w & 1) ? bf_hi(w < 2 ? ks0.x : ks0.y) : bf_lo(w < 2 ? ks0.x : ks0.y);
      const float s1 = (w & 1) ? bf_hi(w < 2 ? ks1.x : ks1.y) : bf_lo(w < 2 ? ks1.x : ks1.y);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float acc[4] = {q.start[nt][w][0], q.start[nt][w][1], q.start[nt][w][0], q.start[nt][w][1]};
        mma_f16(acc, r0 & 0x000f000fu, r1 & 0x000f000fu, r0 & 0x00f000f0u, r1 & 0x00f000f0u, q.b[nt][w][0][0], q.b[nt][w][0][1]);
        mma_f16(acc, r0h & 0x000f000fu, r1h & 0x000f000fu, r0h & 0x00f000f0u, r1h & 0x00f000f0u, q.b[nt][w][1][0],
                q.b[nt][w][1][1]);
        x[nt][0] = fmaf(acc[0], s0, x[nt][0]);
        x[nt][1] = fmaf(acc[1], s0, x[nt][1]);
        x[nt][2] = fmaf(acc[2], s1, x[nt][2]);
        x[nt][3] = fmaf(acc[3], s1, x[nt][3]);
      }
    }
    // log2 of the largest value scale of the lane's two keys
    auto log_scale = [](const uint2& v) {
      const uint32_t m = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
      return fmaxf(lg2_approx(__uint_as_float(max(m << 16, m & 0xffff0000u))), kLeastScale);
    };
    const float g0 = log_scale(vs0), g1 = log_scale(vs1);
    bool grows = false;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[nt][i] = (i < 2 ? see0 : see1) ? x[nt][i] * q.unit[nt][i & 1] : -INFINITY;
        grows |= x[nt][i] + (i < 2 ? g0 : g1) > ref[nt][i & 1] + kHigh;
      }
    }
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = fmaxf(x[nt][h] + g0, x[nt][h + 2] + g1);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          if (top > ref[nt][h] + kHigh) {
            const float a = ex2_approx(ref[nt][h] - (top - kStart));
            ref[nt][h] = top - kStart;
            sum[nt][h] *= a;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              o[nt][m][h] *= a;
              o[nt][m][h + 2] *= a;
            }
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] = ex2_approx(x[nt][i] - ref[nt][i & 1]);
      sum[nt][0] += x[nt][0] + x[nt][2];
      sum[nt][1] += x[nt][1] + x[nt][3];
    }

    const uint8_t* vr = va + 2 * t * kKv4RowBytes + 8 * g;
    const uint2 v0 = *reinterpret_cast<const uint2*>(vr);
    const uint2 v1 = *reinterpret_cast<const uint2*>(vr + kKv4RowBytes);
    const uint2 v2 = *reinterpret_cast<const uint2*>(vr + 8 * kKv4RowBytes);
    const uint2 v3 = *reinterpret_cast<const uint2*>(vr + 9 * kKv4RowBytes);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t sel = (w & 1) ? 0x7632u : 0x5410u;
      const uint32_t a = __byte_perm(w < 2 ? v0.x : v0.y, w < 2 ? v1.x : v1.y, sel);
      const uint32_t b = __byte_perm(w < 2 ? v2.x : v2.y, w < 2 ? v3.x : v3.y, sel);
      const uint32_t ah = a >> 8, bh = b >> 8;
      const uint32_t c0 = code_lo(a), c1 = code_hi(a), c2 = code_lo(b), c3 = code_hi(b);
      const uint32_t d0 = code_lo(ah), d1 = code_hi(ah), d2 = code_lo(bh), d3 = code_hi(bh);
      const float s0 = (w & 1) ? bf_hi(w < 2 ? vs0.x : vs0.y) : bf_lo(w < 2 ? vs0.x : vs0.y);
      const float s1 = (w & 1) ? bf_hi(w < 2 ? vs1.x : vs1.y) : bf_lo(w < 2 ? vs1.x : vs1.y);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const uint32_t p0 = transpose8(half2_bits(x[nt][0] * s0, x[nt][1] * s0));
        const uint32_t p1 = transpose8(half2_bits(x[nt][2] * s1, x[nt][3] * s1));
        mma_f16(o[nt][2 * w], c0, c1, c2, c3, p0, p1);
        mma_f16(o[nt][2 * w + 1], d0, d1, d2, d3, p0, p1);
      }
    }
  }
};

template <int kNT>
__global__ void __launch_bounds__(kThreads, 1) kv4_decode_kernel(const Params p) {
  using S = Smem<kNT>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + S::kJoin);
  float* refs = reinterpret_cast<float*>(smem + S::kRef);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + kStages;
  uint32_t* bad_chunks = reinterpret_cast<uint32_t*>(smem + S::kBad);
  int* misc = reinterpret_cast<int*>(smem + S::kMisc);
  int* pre = reinterpret_cast<int*>(smem + S::kPre);
  int* lens = reinterpret_cast<int*>(smem + S::kLens);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    fence_mbar_init();
  }
  // ---- tiles of the sequences before, by the working warps, at most 8 sequences a thread
  const int per = (p.B + kWork - 1) / kWork;
  const int i0 = tid * per;
  const int i1 = warp < kWarps ? min(p.B, i0 + per) : 0;
  pdl_wait_predecessor();
  pdl_allow_successor();
  if (warp < kWarps) {
    int sum = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
      const int len = p.seq_lens[i];
      bad |= len < 0 || len > p.L_cap;
      lens[i] = len;
      sum += span_of(len, p.L_cap, p.kv).nt;
    }
    if (bad) raise_status(p.status, kStatusBadSeqLen);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) misc[warp] = incl;
    named_bar_sync(1, kWork);
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += misc[w];
    if (tid == kWork - 1) pre[p.B] = run + sum;
    for (int i = i0; i < i1; ++i) {
      pre[i] = run;
      run += span_of(lens[i], p.L_cap, p.kv).nt;
    }
  }
  __syncthreads();

  // The first min(tiles, CTAs) CTAs share the tiles, each at least one (tile counts fit 32 bits: the host checks).
  const int total = p.h_kv * pre[p.B];
  const int grid = gridDim.x, cta = blockIdx.x;
  const int NC = min(total, grid);
  const int q_tiles = NC > 0 ? total / NC : 0;
  const int rm = NC > 0 ? total - q_tiles * NC : 0;
  auto range_start = [&](int c) { return c * q_tiles + min(c, rm); };
  const int beg = cta < NC ? range_start(cta) : 0;
  const int end = cta < NC ? range_start(cta + 1) : 0;

  // The piece of the range that starts at tile x: sequence b, key/value head j, first tile tl of the segment's nt, n tiles
  // here, the segment's first tile in the list.
  struct Piece {
    int b, j, tl, nt, n, seg0;
  };
  auto locate = [&](int x) -> Piece {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.h_kv * pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    Piece r;
    r.b = lo;
    r.nt = pre[lo + 1] - pre[lo];
    const int off = x - p.h_kv * pre[lo];
    r.j = off / r.nt;
    r.tl = off - r.j * r.nt;
    r.seg0 = x - r.tl;
    r.n = min(end - x, r.nt - r.tl);
    return r;
  };
  auto after = [&](Piece r, int x) -> Piece {
    if (++r.j == p.h_kv) {
      r.j = 0;
      do ++r.b;
      while (pre[r.b + 1] == pre[r.b]);
      r.nt = pre[r.b + 1] - pre[r.b];
    }
    r.tl = 0;
    r.seg0 = x;
    r.n = min(end - x, r.nt);
    return r;
  };

  if (warp == kWarps) {
    // =========================== loads ===========================
    // Lane lp brings the run of chunks lp of a tile: a page's rows, at most a tile's; 16 keys where sink keys are folded in.
    // The next tile's table entry is read while this one's stage is waited for.
    const uint64_t policy = l2_policy_evict_first();
    const int page = 1 << p.kv.page_shift;
    const int rows = min(page, kKeys);
    int it = 0;
    bool ok = true;
    // the run's page in tile t of sequence b: -2 nothing to load, -1 a bad entry (reads as zeros)
    auto entry = [&](const DecodeSpan& sp, int b, int t) {
      const int n = t == 0 && sp.fold > 0 ? kFold : rows;
      const int key = sp.key_of(t, lane * n);
      if (lane * n >= kKeys || !sp.sees_any(key, n)) return -2;
      const int id = p.kv.block_table[static_cast<int64_t>(b) * p.kv.max_pages + (key >> p.kv.page_shift)];
      return static_cast<uint32_t>(id) < static_cast<uint32_t>(p.kv.num_pages) ? id : -1;
    };
    Piece pc{}, np{};
    DecodeSpan sp{}, nsp{};
    int id = -2;
    if (beg < end) {
      np = locate(beg);
      nsp = span_of(lens[np.b], p.L_cap, p.kv);
      id = entry(nsp, np.b, np.tl);
    }
    const int stop = p.give_up_tile < 0 ? end : beg + min(end - beg, p.give_up_tile);
    for (int x = beg; x < stop && ok;) {
      pc = np;
      sp = nsp;
      const bool more = x + pc.n < end;
      if (more) {
        np = after(pc, x + pc.n);
        if (np.b != pc.b) nsp = span_of(lens[np.b], p.L_cap, p.kv);
      }
      for (int t = pc.tl; t < pc.tl + pc.n; ++t, ++it) {
        const int next = t + 1 < pc.tl + pc.n ? entry(sp, pc.b, t + 1) : (more ? entry(nsp, np.b, 0) : -2);
        const int st = it % kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], static_cast<uint32_t>(((it / kStages) & 1) ^ 1)));
        if (!ok) break;
        const int n = t == 0 && sp.fold > 0 ? kFold : rows;
        const int chunks = n / kChunk;
        const uint32_t loads = __popc(__ballot_sync(0xffffffffu, id >= 0));
        const uint32_t bad = __ballot_sync(0xffffffffu, id == -1);
        if (lane == 0) {
          uint32_t mask = 0;
          for (int r = 0; r < kChunks / chunks; ++r)
            if (bad >> r & 1) mask |= ((1u << chunks) - 1) << (r * chunks);
          bad_chunks[st] = mask;
          mbar_arrive_expect_tx(&full[st], loads * static_cast<uint32_t>(chunks * kKv4Block));
        }
        __syncwarp();
        if (id >= 0) {
          const int key = sp.key_of(t, lane * n);
          const int64_t block = ((static_cast<int64_t>(id) * p.h_kv + pc.j) << (p.kv.page_shift - 4)) + ((key & (page - 1)) / kChunk);
          bulk_load(smem + st * kStageBytes + lane * chunks * kKv4Block, p.cache + block * kKv4Block,
                    static_cast<uint32_t>(chunks * kKv4Block), &full[st], policy);
        } else if (id == -1) {
          raise_status(p.status, kStatusBadPage);
        }
        id = next;
      }
      x += pc.n;
    }
    if (lane == 0) {
      if (!ok || stop < end) atomicExch(p.status, kStatusWaitEmptyTimeout);
      // no copy may outlive its CTA
      const int n = min(it, kStages);
      for (int i = it - n; i < it; ++i)
        if (!mbar_wait(&full[i % kStages], static_cast<uint32_t>((i / kStages) & 1))) {
          atomicExch(p.status, kStatusDrainTimeout);
          break;
        }
    }
    __syncwarp();
    return;
  }

  // =========================== work ===========================
  const int g = lane >> 2, t4 = lane & 3;
  Queries<kNT> q;
  State<kNT> s;
  bool ok = true;
  int it = 0, turn = 0;
  Piece pc{};
  for (int x = beg; x < end; turn ^= 1) {
    pc = x == beg ? locate(x) : after(pc, x);
    const DecodeSpan sp = span_of(lens[pc.b], p.L_cap, p.kv);
    q.load(p.q + (static_cast<int64_t>(pc.b) * p.h_q + static_cast<int64_t>(pc.j) * p.G) * kD, p.G, p.scale_log2, lane);
    s.clear();
    for (int t = pc.tl; t < pc.tl + pc.n; ++t, ++it) {
      const int st = it % kStages;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[st], static_cast<uint32_t>((it / kStages) & 1)));
      if (!ok) {
        if (lane == 0) atomicExch(p.status, kStatusWaitFullTimeout);
        break;
      }
      const int key = sp.key_of(t, warp * kChunk);
      if (sp.sees_any(key, kChunk))
        s.add(q, smem + st * kStageBytes + warp * kKv4Block, sp.sees(key + g), sp.sees(key + g + 8), bad_chunks[st] >> warp & 1,
              lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the warps' states joined: references first, then outputs on a common one
    float* my_ref = refs + turn * 2 * kWarps * 16;
    float* my_sum = my_ref + kWarps * 16;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = s.sum[nt][h];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (g == 0) {
          my_ref[warp * 16 + 8 * nt + 2 * t4 + h] = s.ref[nt][h];
          my_sum[warp * 16 + 8 * nt + 2 * t4 + h] = v;
        }
      }
    named_bar_sync(1, kWork);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int head = 8 * nt + 2 * t4 + h;
        float top = my_ref[head];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, my_ref[w * 16 + head]);
        const float a = ex2_approx(s.ref[nt][h] - top);
        float* to = join + (warp * 8 * kNT + head) * kRow + 4 * g;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          *reinterpret_cast<float4*>(to + 32 * w) = make_float4(s.o[nt][2 * w][h] * a, s.o[nt][2 * w][h + 2] * a,
                                                                s.o[nt][2 * w + 1][h] * a, s.o[nt][2 * w + 1][h + 2] * a);
      }
    named_bar_sync(1, kWork);

    // ---- thread: four dimensions of a head (of two, with 16)
    const bool whole = pc.tl == 0 && pc.n == pc.nt;
    const int d4 = 4 * (tid & 31);
    uint16_t* out = p.out + (static_cast<int64_t>(pc.b) * p.h_q + static_cast<int64_t>(pc.j) * p.G) * kD + d4;
    auto store = [&](int head, const float4& o, float l) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(__fdividef(o.x, l), __fdividef(o.y, l));
      const __nv_bfloat162 b = __floats2bfloat162_rn(__fdividef(o.z, l), __fdividef(o.w, l));
      *reinterpret_cast<uint2*>(out + head * kD) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    };
    const int slot = x == beg ? 0 : 1;
    float* mine = p.partials + (static_cast<int64_t>(cta) * 2 + slot) * kGqaSlotFloats;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int head = 8 * nt + warp;
      if (head >= p.G) continue;
      float top = my_ref[head];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, my_ref[w * 16 + head]);
      float l = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        l += my_sum[w * 16 + head] * ex2_approx(my_ref[w * 16 + head] - top);
        const float4 v = *reinterpret_cast<const float4*>(join + (w * 8 * kNT + head) * kRow + d4);
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      if (whole) {
        store(head, o, l);
      } else {
        *reinterpret_cast<float4*>(mine + head * kD + d4) = o;
        if (lane == 0) {
          mine[16 * kD + head] = top;
          mine[16 * kD + 16 + head] = l;
        }
      }
    }
    if (!whole) {
      // a segment cut between CTAs: the last to publish its piece joins them all, in CTA order
      auto cta_of = [&](int i) {
        const int big = rm * (q_tiles + 1);
        return i < big ? i / (q_tiles + 1) : rm + (i - big) / q_tiles;
      };
      const int c_first = cta_of(pc.seg0), c_last = cta_of(pc.seg0 + pc.nt - 1);
      named_bar_sync(1, kWork);
      if (tid == 0) {
        __threadfence();  // publishes what the barrier gathered
        const bool last = atomicAdd(&p.counters[c_first], 1) == c_last - c_first;
        if (last) p.counters[c_first] = 0;
        misc[8] = last;
      }
      named_bar_sync(1, kWork);
      if (misc[8]) {
        __threadfence();
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const int head = 8 * nt + warp;
          if (head >= p.G) continue;
          float top = -FLT_MAX, l = 0.0f;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int c = c_first; c <= c_last; ++c) {
            const float* src = p.partials + (static_cast<int64_t>(c) * 2 + (range_start(c) >= pc.seg0 ? 0 : 1)) * kGqaSlotFloats;
            const float m = __ldcg(src + 16 * kD + head), lc = __ldcg(src + 16 * kD + 16 + head);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + head * kD + d4));
            const float now = fmaxf(top, m);
            const float a = ex2_approx(top - now), b = ex2_approx(m - now);
            o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
            l = l * a + lc * b;
            top = now;
          }
          store(head, o, l);
        }
      }
      named_bar_sync(1, kWork);  // misc[8] is written again by the next cut piece
    }
    x += pc.n;
  }

  // ---- sequences with no keys (or a bad length) attend to nothing: output 0
  for (int b = cta; b < p.B; b += grid) {
    if (pre[b + 1] != pre[b]) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(b) * p.h_q * kD);
    for (int i = tid; i < p.h_q * kD / 8; i += kWork) o[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int kNT>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  constexpr int kMaxDev = 64;  // the shared-memory opt-in is per device: done once on each
  static std::atomic<bool> done[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDev || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv4_decode_kernel<kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<kNT>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev) done[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(kv4_decode_kernel<kNT>, dim3(grid), dim3(kThreads), Smem<kNT>::kBytes, stream, p);
}

}  // namespace kv4

cudaError_t launch_kv4_decode(const Kv4DecodePlan& plan, cudaStream_t stream) {
  kv4::Params p{};
  p.q = plan.q;
  p.cache = plan.cache;
  p.seq_lens = plan.seq_lens;
  p.out = plan.out;
  p.partials = plan.partials;
  p.counters = plan.counters;
  p.status = plan.status;
  p.B = plan.B;
  p.h_q = plan.h_q;
  p.h_kv = plan.h_kv;
  p.G = plan.h_q / plan.h_kv;
  p.L_cap = plan.L_cap;
  p.scale_log2 = plan.scale_log2;
  p.kv = plan.paged;
  p.give_up_tile = plan.give_up_tile;
  return p.G <= 8 ? kv4::launch<1>(p, plan.num_ctas, stream) : kv4::launch<2>(p, plan.num_ctas, stream);
}

}  // namespace moe
