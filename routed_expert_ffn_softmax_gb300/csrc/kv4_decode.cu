// Decode attention over a paged cache held in 4 bits (include/paged/moe_kv4.h): one query token per sequence, the G query
// heads of a group against each key/value head, under a sliding window with sink tokens.
//
// What bounds it. A key costs 144 bytes of HBM a key/value head (72 for K, 72 for V), 3.6 times less than in bf16, so an SM has
// 6.2 cycles of memory time per key. 16-bit operands of tcgen05 would have to pass through shared memory: 512 bytes written and
// 512 read per key, 8 cycles of the shared memory's 128 bytes a cycle, more than the memory time. (In 8 bits the keys would
// pass: the bytes 0 .. 15 are exactly n 2^-9 in e4m3, 128 bytes written and read, 2 cycles. Scores and probabilities would then
// go through TMEM and back; that was not tried.) Here the codes go from shared memory straight into registers as mma.sync
// operands: the key axis is the M side of both products, so a group of up to 8 heads (the N side) wastes nothing.
//     S [16 keys x 8 heads]  = codes(K) [16 x 32] . q [32 x 8]           for each of the 4 groups of 32 dimensions
//     O [16 dims x 8 heads] += codes(V)^T [16 x 16 keys] . (p s) [16 x 8]  s the value scale of the group the dims are in
// K's scales multiply the four group sums in fp32; V's scales go into the probabilities, once per group.
//
// Unpacking is most of the instructions (the integer pipe takes 2 cycles each), but no unit is full over the whole kernel (16
// long sequences: integer pipe 44%, tensor 21%, fma 21%, issue 48%): each of the two working warps of a scheduler goes through
// one chain a unit (score products, 2^x, the vote, fp16, value products) with nothing of the next unit under way, and
// instruction fetch is the largest stall after the waits of idle roles. 16 bits of a row hold four codes of a group; two such
// of the same row (K) or of two keys (V) in one register give all four fp16 pairs with four masks and a shift. K's are left as
// fp16 subnormals n 2^-24 (n 2^-20 for the odd codes, whose queries are a 16th): exact products, n = c + 8, and -8 sum(q) is
// where the accumulator starts. V's are turned into exact c by an exponent and a subtraction, as a sum over many keys must not
// carry an offset (as subnormals too, corrected by a product with -8, a key of large weight and code 0 left 2^-20 of its
// weight; it was no faster). K's codes as e4m3 bytes, two masks for eight, with the queries in two e4m3 parts: the instruction
// is made of conversions and fp16 products, 16 sequences of up to 32K keys took 78 us instead of the 65 of that time.
//
// Range. p s must fit fp16, whatever the scales are: the softmax reference R of a head bounds score + log2(largest scale of
// the key) instead of the score alone, p = 2^(score - R) is held in fp32, and R is raised (outputs and sums rescaled) only
// when a product would pass 2^15. R starts 2^6 below the largest, so products keep fp16's full precision down to 2^-20 of it.
//
// Work split: as in gqa_decode.cu, the key tiles (128 keys) of all segments form one list of which each CTA takes a
// contiguous share, here with some units more for a segment's start, or with few tiles a part of one segment; the pieces of a cut
// segment are joined in CTA order by the last to arrive.
//
// Per CTA, 12 warps, which share out the registers:
//   0, 1   bring tiles with bulk copies, 16 tokens of keys and values or whole runs of a page in one (2304 bytes a chunk);
//   2, 3   prepare the queries as operands, two pieces ahead; join the working warps' parts of a piece, write its output or
//          its partial, and join a cut segment;
//   4..11  work: each takes 32 or 64 keys of a tile, with a running (R, sum, O) of its own, and goes on to the next piece as
//          soon as its part is handed over.
// (One warp that loads, 8 or 11 that work and join through barriers: 255 sequences of up to 4K keys took 125 us, then 85.)
//
// GB300: 16 sequences of up to 32K keys, 4 heads a group, in 60 us (4.8 TB/s, 71% of a copy; 155 us in bf16); 24 with 16 heads
// a group in 74 (3.2 TB/s, 180 TFLOP/s); 64 behind a window of 1024 in 26; 255 of up to 4K in 74 (3.9 TB/s); one sequence of 512
// visible keys in 7.5. With two chunks a warp the working warps were at it 76% of the time in the first of these, the integer pipe
// then 68% busy; the rest is the start (lengths, table, first tile: 3 us), the last pieces' joins, and a hand-over per piece.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

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
constexpr int kChunk = kKv4Tokens;         // keys of one matrix instruction
constexpr int kChunks = kKeys / kChunk;    // of a tile
constexpr int kStageBytes = kChunks * kKv4Block;
constexpr int kRow = kD + 4;               // floats of a head's outputs handed over (no bank conflicts)
constexpr float kMost = 32768.0f;          // what p s may reach
constexpr float kRaise = 14.5f;            // log2 of the p s from which a head's reference is raised when one is too large
constexpr float kStart = 6.0f;             // log2 of the largest p s right after a reference is set
// 2^-80: smaller value scales, 0 among them, count as this where references are concerned. A weight is then below 2^95 (2^kRaise
// over the least), and a sum of 2^31 of them below 2^126, which the last division needs.
constexpr float kLeastScale = 8.2718061e-25f;
static_assert(kFold == kChunk, "sink keys are folded in whole chunks");

// Warps 0..3: two that load, two that prepare queries and finish pieces; the others work.
constexpr int kWarps = 8;                  // that work
constexpr int kThreads = 32 * (4 + kWarps);
// Registers per thread at launch; the warpgroups share out what the launch has.
constexpr int kRegsLaunch = 168;
constexpr int kRegsHelp = 104;
constexpr int kRegsWork = 200;
static_assert(128 * kRegsHelp + 32 * kWarps * kRegsWork <= kThreads * kRegsLaunch, "a larger share would wait forever");

// kNT: eights of heads. (With 12 warps that work and 128 registers at launch, two chunks each: 16 sequences of up to 32K keys
// 62.5 us instead of 65.4, but 255 of up to 4K 92 instead of 85 and one sequence 11.0 instead of 9.3; with 16 heads the same as 8.)
template <int kNT>
struct Split {
  // Chunks a warp takes at once: two, as the code around them costs as much as one (with 16 heads: 24 sequences of up to 32K keys
  // 74.0 us instead of 74.9 with two for these alone, 64 behind a window 26.8 instead of 26.4). Four with up to 8 heads where the
  // sequences' segments have kLong tiles on average: us for two and four with 128 sequences of up to 2K keys 36.1 and 38.9, 64 of
  // up to 4K 33.6 and 32.3, 32 of up to 8K 33.5 and 31.1, 8 of up to 32K 32.6 and 31.0 (4 key/value heads, lengths from half of
  // it). With 16 heads four spill.
  static constexpr int kUnit = 2;
  static constexpr int kLongUnit = kNT == 1 ? 4 : 2;
  static constexpr int kLong = 20;
  // A piece costs a CTA about as much as some tiles (queries, a first tile to wait for, hand-over, join): so many units a segment
  // counts besides its own tiles, where CTAs have kSegmentFrom tiles on average. (With none, CTAs whose share was many short
  // segments came last: 255 sequences of up to 4K keys 85 us instead of 74, with 16 heads 133 instead of 106; 64 of up to 1K with
  // 16 heads 30 instead of 21. 4 units for all: 24 long ones 74.2 instead of 73.7, 16 long ones 60.5 instead of 59.7.)
  static constexpr int kSegment = kNT == 1 ? 2 : 3;
  static constexpr int kSegmentFrom = 2;
  // With few tiles a CTA has tiles of one segment only: all of it where there is a CTA for each segment and none has more than
  // kWhole tiles, as joining pieces takes longer (us without and with: one sequence of 512 visible keys of 5 tiles 9.4 and 7.5, of
  // 8 tiles 8.4 and 9.0; 32 of up to 1K keys 13.5 and 10.1; 4 of up to 512 with 16 heads 15.2 and 9.1); else as many as make the
  // CTAs do, up to kOwn (one of 1300 keys 10.1 and 8.7, 4 of up to 4K 12.1 and 9.6, with 16 heads 16.0 and 12.3).
  static constexpr int kWhole = 8;
  static constexpr int kWholeTiles = 1 << 20;
  static constexpr int kOwn = 6;
  static constexpr int tiles_at_once(bool longs) { return kWarps * (longs ? kLongUnit : kUnit) / kChunks; }
  static constexpr int kStages = kNT == 1 ? 9 : 7;
  // The two loading warps take kTurn tiles in turn, and an mbarrier tells apart only neighbouring phases. So neither loader may
  // get to tile t + 2 kStages of a stage while tile t there is still worked on, nor a working warp to tile t + kStages while t
  // is not loaded. What keeps them: the working warps that are behind with t are so with every kTogether-th tile after it, a
  // turn holds one of those, and a warp needs a tile of every second turn. (tests/test_kv4_schedule_model.py visits every state
  // of these numbers; 5 or 8 stages with 3 tiles together fail.)
  static constexpr int kTurn = 4;
  static constexpr int kTogether = tiles_at_once(kLongUnit != kUnit);
  static_assert(kTurn % kTogether == 0 && kStages > kTurn + kTogether, "phases apart by two");
  // shared memory
  static constexpr int kJoinFloats = kWarps * 8 * kNT * kRow;
  static constexpr int kMost = kJoinFloats * 4 / (128 + 512 * 8 * kNT);  // parts of a cut segment that fit there
  static_assert(kMost >= kWarps && kMost <= 32, "both are joined alike, a lane copies a part");
  static constexpr int kJoin = kStages * kStageBytes;                    // [kWarps][8 kNT][kRow] floats
  static constexpr int kRef = kJoin + kJoinFloats * 4;                   // [2][kWarps][16] floats: reference, sum
  static constexpr int kQ = kRef + 2 * kWarps * 16 * 4;                  // [2] queries as operands
  static constexpr int kQBytes = kNT * (4 * 32 * 16 + 8 * 4 * 4 + 8 * 4);
  static constexpr int kBars = (kQ + 2 * kQBytes + 15) / 16 * 16;
  static constexpr int kBad = kBars + (2 * kStages + 7) * 8;             // [2][kStages] chunks that read as zeros, the last tile there
  static constexpr int kMisc = (kBad + 2 * kStages * 4 + 15) / 16 * 16;      // 32 ints
  static constexpr int kPre = kMisc + 128;
  static constexpr int kLens = kPre + (kGqaMaxSeqs + 4) * 4;
  static constexpr int kPreUnits = kLens + kGqaMaxSeqs * 4;
  static constexpr int kBytes = kPreUnits + (kGqaMaxSeqs + 4) * 4;
  static_assert(kBytes <= 232448, "dynamic shared memory per CTA");
  static_assert(kQ % 16 == 0 && kRef % 16 == 0, "vector loads");
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
  int piece_waits;   // limits of a wait that may last as long as a piece
  int give_up_tile;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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
// (v & mask) | more in one instruction: with both as immediates the compiler takes two.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t more) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "n"(kMask), "r"(more));
  return d;
}

__device__ __forceinline__ void mbar_arrive_many(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
// Orders this thread's plain accesses, to shared and global memory, before copies that are issued after a barrier.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// log2 of the largest of a key's value scales that is not NaN.
__device__ __forceinline__ float log_scale(const uint2& v) {
  return lg2_approx(max3_f32(max3_f32(bf_lo(v.x), bf_hi(v.x), kLeastScale), bf_lo(v.y), bf_hi(v.y)));
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The queries of up to 8 kNT heads as mma operands, and what goes with them, in shared memory: written by one warp per piece,
// read per use (in registers, they took those that keep four chunks, or two with 16 heads, under way: 24 sequences of up to
// 32K keys with 16 heads 81 us instead of 76).
template <int kNT>
struct Queries {
  uint8_t* at;               // per 8 heads and group of dimensions: operands [lane], -8 sum(q) [head]; units [head]
  float unit[kNT][2];        // accumulator units to log2 scores, for heads 2 t, 2 t + 1
  uint32_t exp_low, exp_high;  // fp16 1024 and 64 twice, in registers

  static __device__ __forceinline__ uint4* operands(uint8_t* at) { return reinterpret_cast<uint4*>(at); }
  static __device__ __forceinline__ float* starts(uint8_t* at) { return reinterpret_cast<float*>(at + kNT * 4 * 32 * 16); }
  static __device__ __forceinline__ float* units(uint8_t* at) { return starts(at) + kNT * 32; }

  // q at the group's first head; lane (g, t) takes head g's dimensions 32 w + 8 t .. + 7.
  static __device__ __forceinline__ void prepare(uint8_t* at, const uint16_t* q, int G, float scale_log2, int lane) {
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
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf_lo(x[i]) * to;
          f[2 * i + 1] = bf_hi(x[i]) * (to * 0.0625f);
        }
        uint32_t h[4];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = half2_bits(f[i], f[i + 4]);
          const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
          sum = fmaf(r.x + r.y, (i & 1) ? 16.0f : 1.0f, sum);
        }
        operands(at)[(nt * 4 + w) * 32 + lane] = make_uint4(h[0], h[1], h[2], h[3]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (t == 0) starts(at)[(nt * 4 + w) * 8 + g] = sum * -4.76837158203125e-07f;  // -8 2^-24
      }
      if (t == 0) units(at)[nt * 8 + g] = back;
    }
  }
  // One group's: two registers for each of two k16 steps, and where the accumulators of heads 2 t, 2 t + 1 start.
  __device__ __forceinline__ uint4 operand(int nt, int w, int lane) const { return operands(at)[(nt * 4 + w) * 32 + lane]; }
  __device__ __forceinline__ float2 start(int nt, int w, int lane) const {
    return *reinterpret_cast<const float2*>(starts(at) + (nt * 4 + w) * 8 + 2 * (lane & 3));
  }
  __device__ __forceinline__ void take(uint8_t* from, int lane) {
    at = from;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const float2 u = *reinterpret_cast<const float2*>(units(at) + nt * 8 + 2 * (lane & 3));
      unit[nt][0] = u.x, unit[nt][1] = u.y;
    }
    asm volatile("mov.u32 %0, 0x64006400;" : "=r"(exp_low));
    asm volatile("mov.u32 %0, 0x54005400;" : "=r"(exp_high));
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

  // kCount times 16 keys at `at` in shared memory; bias: 0 for a key (g and g + 8 of each 16) that the query sees, -infinity
  // for others, whose scales are 0.
  template <int kCount>
  __device__ __forceinline__ void add(const Queries<kNT>& q, const uint8_t* at, const float (&bias)[kCount][2], int lane) {
    const int g = lane >> 2, t = lane & 3;
    float x[kCount][kNT][4];
    uint2 vs[kCount][2];
    uint4 k0[kCount], k1[kCount];
    uint2 ks0[kCount], ks1[kCount];
#pragma unroll
    for (int c = 0; c < kCount; ++c) {
      const uint8_t* ka = at + c * kKv4Block;
      k0[c] = *reinterpret_cast<const uint4*>(ka + g * kKv4RowBytes + 16 * t);
      k1[c] = *reinterpret_cast<const uint4*>(ka + (g + 8) * kKv4RowBytes + 16 * t);
      ks0[c] = *reinterpret_cast<const uint2*>(ka + kKv4Scales + 8 * g);
      ks1[c] = *reinterpret_cast<const uint2*>(ka + kKv4Scales + 8 * (g + 8));
      vs[c][0] = *reinterpret_cast<const uint2*>(ka + kKv4Values + kKv4Scales + 8 * g);
      vs[c][1] = *reinterpret_cast<const uint2*>(ka + kKv4Values + kKv4Scales + 8 * (g + 8));
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][nt][i] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint4 qb[kNT];
      float2 st[kNT];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        qb[nt] = q.operand(nt, w, lane);
        st[nt] = q.start(nt, w, lane);
      }
#pragma unroll
      for (int c = 0; c < kCount; ++c) {
        const uint32_t sel = (w & 1) ? 0x7632u : 0x5410u;
        const uint32_t r0 = __byte_perm(w < 2 ? k0[c].x : k0[c].y, w < 2 ? k0[c].z : k0[c].w, sel);
        const uint32_t r1 = __byte_perm(w < 2 ? k1[c].x : k1[c].y, w < 2 ? k1[c].z : k1[c].w, sel);
        const uint32_t r0h = r0 >> 8, r1h = r1 >> 8;
        const float s0 = (w & 1) ? bf_hi(w < 2 ? ks0[c].x : ks0[c].y) : bf_lo(w < 2 ? ks0[c].x : ks0[c].y);
        const float s1 = (w & 1) ? bf_hi(w < 2 ? ks1[c].x : ks1[c].y) : bf_lo(w < 2 ? ks1[c].x : ks1[c].y);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const float from[4] = {st[nt].x, st[nt].y, st[nt].x, st[nt].y};
          float acc[4];
          mma_f16(acc, r0 & 0x000f000fu, r1 & 0x000f000fu, r0 & 0x00f000f0u, r1 & 0x00f000f0u, qb[nt].x, qb[nt].y, from);
          mma_f16(acc, r0h & 0x000f000fu, r1h & 0x000f000fu, r0h & 0x00f000f0u, r1h & 0x00f000f0u, qb[nt].z, qb[nt].w, acc);
          x[c][nt][0] = fmaf(acc[0], s0, x[c][nt][0]);
          x[c][nt][1] = fmaf(acc[1], s0, x[c][nt][1]);
          x[c][nt][2] = fmaf(acc[2], s1, x[c][nt][2]);
          x[c][nt][3] = fmaf(acc[3], s1, x[c][nt][3]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kCount; ++c)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][nt][i] = fmaf(x[c][nt][i], q.unit[nt][i & 1], bias[c][i >> 1]);

    float p[kCount][kNT][4];
    auto weigh = [&]() {
#pragma unroll
      for (int c = 0; c < kCount; ++c)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[c][nt][i] = ex2_approx(x[c][nt][i] - ref[nt][i & 1]);
    };
    weigh();
    // Whether the lane's largest weight times its largest value scale (scales are not negative) is small enough. NaN is not: one
    // among the scales stands above all others here and would hide them.
    auto larger = [](uint32_t a, uint32_t b) { return __vmaxu2(a, b); };
    uint32_t m = larger(larger(vs[0][0].x, vs[0][0].y), larger(vs[0][1].x, vs[0][1].y));
#pragma unroll
    for (int c = 1; c < kCount; ++c) m = larger(m, larger(larger(vs[c][0].x, vs[c][0].y), larger(vs[c][1].x, vs[c][1].y)));
    float top_p = 0.0f;
#pragma unroll
    for (int c = 0; c < kCount; ++c)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) top_p = max3_nan(max3_nan(top_p, p[c][nt][0], p[c][nt][1]), p[c][nt][2], p[c][nt][3]);
    const bool fits = top_p * max3_nan(bf_lo(m), bf_hi(m), kLeastScale) <= kMost;
    if (!__all_sync(0xffffffffu, fits)) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kCount; ++c)
            top = max3_f32(top, x[c][nt][h] + log_scale(vs[c][0]), x[c][nt][h + 2] + log_scale(vs[c][1]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          if (top > ref[nt][h] + kRaise) {
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
      weigh();
    }

#pragma unroll
    for (int c = 0; c < kCount; ++c) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        sum[nt][0] += p[c][nt][0] + p[c][nt][2];
        sum[nt][1] += p[c][nt][1] + p[c][nt][3];
      }
      const uint8_t* vr = at + c * kKv4Block + kKv4Values + 2 * t * kKv4RowBytes + 8 * g;
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
        auto low = [&](uint32_t v) { return sub2(and_or<0x000f000fu>(v, q.exp_low), 0x64086408u); };
        auto high = [&](uint32_t v) { return sub2(and_or<0x00f000f0u>(v, q.exp_high), 0x54805480u); };
        const uint32_t c0 = low(a), c1 = high(a), c2 = low(b), c3 = high(b), d0 = low(ah), d1 = high(ah), d2 = low(bh), d3 = high(bh);
        const float s0 = (w & 1) ? bf_hi(w < 2 ? vs[c][0].x : vs[c][0].y) : bf_lo(w < 2 ? vs[c][0].x : vs[c][0].y);
        const float s1 = (w & 1) ? bf_hi(w < 2 ? vs[c][1].x : vs[c][1].y) : bf_lo(w < 2 ? vs[c][1].x : vs[c][1].y);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const uint32_t p0 = transpose8(half2_bits(p[c][nt][0] * s0, p[c][nt][1] * s0));
          const uint32_t p1 = transpose8(half2_bits(p[c][nt][2] * s1, p[c][nt][3] * s1));
          mma_f16(o[nt][2 * w], c0, c1, c2, c3, p0, p1, o[nt][2 * w]);
          mma_f16(o[nt][2 * w + 1], d0, d1, d2, d3, p0, p1, o[nt][2 * w + 1]);
        }
      }
    }
  }
};

__device__ __forceinline__ int atom_add_acq_rel(int32_t* p, int v) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// What a warp has joined of the parts of four heads, first .. first + 3: lane (x, y), y the lowest two bits, holds the running
// reference and sum of head first + y; each lane four dimensions of all four.
struct Joined {
  float ref, sum;
  float4 o[4];
  __device__ __forceinline__ void clear() {
    ref = -FLT_MAX;
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  // n <= kMost parts: references of the four heads at `refs` (`step` floats from one part to the next; they are overwritten),
  // sums at `sums`, this lane's dimensions of the outputs at `outs` (o_step to the next part's, head_step to the next head's).
  // Every head's factors are found at once, the lanes sharing the parts: one head after the other, with all parts to a lane,
  // joining 8 warps' 16 heads took 10000 cycles. (kUnrolled: the working warps' parts 4 at a time; cut segments' one, as a longer
  // kernel is a slower one: 16 sequences of up to 32K keys 60.2 us, with 2 or 4 at a time there 61.2.)
  template <int kMost, int kUnrolled>
  __device__ __forceinline__ void add(float* refs, const float* sums, int step, int n, const float* outs, int o_step, int head_step,
                                      int lane) {
    constexpr int kPer = (kMost + 7) / 8;
    const int x = lane >> 2, y = lane & 3;
    float m[kPer], l[kPer];
    float top = ref;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool in = x + 8 * i < n;
      m[i] = in ? refs[(x + 8 * i) * step + y] : -INFINITY;
      l[i] = in ? sums[(x + 8 * i) * step + y] : 0.0f;
      top = fmaxf(top, m[i]);
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float more = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float a = ex2_approx(m[i] - top);
      more = fmaf(l[i], a, more);
      if (x + 8 * i < n) refs[(x + 8 * i) * step + y] = a;
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) more += __shfl_xor_sync(0xffffffffu, more, d);
    const float old = ex2_approx(ref - top);
    sum = fmaf(sum, old, more);
    ref = top;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = __shfl_sync(0xffffffffu, old, k);
      o[k] = make_float4(o[k].x * f, o[k].y * f, o[k].z * f, o[k].w * f);
    }
#pragma unroll kUnrolled
    for (int u = 0; u < n; ++u) {
      const float4 a4 = *reinterpret_cast<const float4*>(refs + u * step);
      const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(outs + u * o_step + k * head_step);
        o[k] = make_float4(fmaf(v.x, a[k], o[k].x), fmaf(v.y, a[k], o[k].y), fmaf(v.z, a[k], o[k].z), fmaf(v.w, a[k], o[k].w));
      }
    }
    __syncwarp();
  }
  // out: this lane's dimensions of the group's first head
  __device__ __forceinline__ void store(uint16_t* out, int first, int G) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int head = first + k;
      const float l = __shfl_sync(0xffffffffu, sum, k);
      if (head >= G) continue;
      const __nv_bfloat162 a = __floats2bfloat162_rn(__fdividef(o[k].x, l), __fdividef(o[k].y, l));
      const __nv_bfloat162 b = __floats2bfloat162_rn(__fdividef(o[k].z, l), __fdividef(o[k].w, l));
      *reinterpret_cast<uint2*>(out + head * kD) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
};

template <int kNT>
__global__ void __launch_bounds__(kThreads, 1) kv4_decode_kernel(const Params p) {
  using S = Split<kNT>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + S::kJoin);
  float* refs = reinterpret_cast<float*>(smem + S::kRef);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;  // [2] queries of a piece
  uint64_t* q_empty = q_full + 2;      // [2]
  uint64_t* h_full = q_empty + 2;      // a piece handed over
  uint64_t* h_empty = h_full + 1;
  uint64_t* m_full = h_empty + 1;      // partials of a cut segment
  uint32_t* bad_chunks = reinterpret_cast<uint32_t*>(smem + S::kBad);
  int* last_tile = reinterpret_cast<int*>(bad_chunks + kStages);
  int* misc = reinterpret_cast<int*>(smem + S::kMisc);
  int* pre = reinterpret_cast<int*>(smem + S::kPre);
  int* lens = reinterpret_cast<int*>(smem + S::kLens);
  int* pre_units = reinterpret_cast<int*>(smem + S::kPreUnits);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kChunks);
      last_tile[s] = -1;
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_empty[b], kWarps);
    }
    mbar_init(h_full, kWarps);
    mbar_init(h_empty, 2);
    mbar_init(m_full, 1);
    fence_mbar_init();
  }
  __syncthreads();

  // The first NC CTAs share the tiles: as many as there are with as many tiles as a CTA works on together (tile counts fit 32
  // bits: the host checks, with 8 more a segment). The list that is cut into equal shares has a unit for each tile and `extra`
  // units in front of each segment's tiles; or, with few tiles, a unit for each `own` tiles of a segment, or part of them.
  const int grid = gridDim.x, cta = blockIdx.x;
  int q_units = 0, rm = 0, beg = 0, end = 0, extra = 0;
  int own = 0;  // 0, or tiles of a CTA that has tiles of one segment only
  bool longs = false;  // long segments
  auto range_start = [&](int c) { return c * q_units + min(c, rm); };
  // Where segment j of sequence b begins in units, and the first tile at unit x or behind it.
  auto units_of = [&](int b, int nt) { return own > 0 ? pre_units[b + 1] - pre_units[b] : nt + extra; };
  auto segment_unit = [&](int b, int j, int nt, int seg0) {
    return own == 0 && extra == 0 ? seg0 : p.h_kv * pre_units[b] + j * units_of(b, nt);
  };
  auto tile_at = [&](int x) {
    if (own == 0 && extra == 0) return x;
    if (x >= p.h_kv * pre_units[p.B]) return p.h_kv * pre[p.B];
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.h_kv * pre_units[mid] <= x) lo = mid; else hi = mid - 1;
    }
    const int nt = pre[lo + 1] - pre[lo], off = x - p.h_kv * pre_units[lo];
    const int of = units_of(lo, nt), j = off / of, r = off - j * of;
    return p.h_kv * pre[lo] + j * nt + (own > 0 ? min(nt, r * own) : max(0, r - extra));
  };
  auto find_range = [&]() {
    const int total = p.h_kv * pre[p.B];
    own = misc[17];
    longs = own == 0 && S::kLongUnit != S::kUnit && pre[p.B] >= S::kLong * p.B;
    const int together = S::tiles_at_once(longs);
    const int NC = own > 0 ? p.h_kv * pre_units[p.B] : min((total + together - 1) / together, grid);
    if (NC == 0) return;
    extra = own == 0 && total >= S::kSegmentFrom * grid ? S::kSegment : 0;
    const int units = own > 0 || extra > 0 ? p.h_kv * pre_units[p.B] : total;
    q_units = units / NC;
    rm = units - q_units * NC;
    if (cta >= NC) return;
    const int at = tile_at(range_start(cta + (lane >> 4)));
    beg = __shfl_sync(0xffffffffu, at, 0);
    end = __shfl_sync(0xffffffffu, at, 16);
  };

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
  bool ok = true;  // no wait of this warp has run out (the same for all its lanes); then it waits for nothing more
  auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
    if (!__all_sync(0xffffffffu, ok && mbar_wait(bar, parity))) {
      if (ok && lane == 0) atomicExch(p.status, code);
      ok = false;
    }
  };

  if (warp < 4) {
    reg_dealloc<kRegsHelp>();
    // ---- tiles of the sequences before
    pdl_wait_predecessor();
    pdl_allow_successor();
    const int per = (p.B + 127) / 128;
    const int i0 = tid * per, i1 = min(p.B, i0 + per);
    int64_t sum = 0;  // tiles, and sequences that have some in the upper half
    bool bad_len = false;
    int most = 0;
    auto counts = [](int nt) { return nt + (static_cast<int64_t>(nt > 0) << 32); };
    for (int i = i0; i < i1; ++i) {
      const int len = p.seq_lens[i];
      bad_len |= len < 0 || len > p.L_cap;
      lens[i] = len;
      const int nt = span_of(len, p.L_cap, p.kv).nt;
      sum += counts(nt);
      most = max(most, nt);
    }
    if (bad_len) raise_status(p.status, kStatusBadSeqLen);
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    int64_t* sums = reinterpret_cast<int64_t*>(misc);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) sums[warp] = incl;
    if (lane == 0) misc[8 + warp] = most;
    named_bar_sync(3, 128);
    int64_t run = incl - sum;
    for (int w = 0; w < warp; ++w) run += sums[w];
    const int64_t all = sums[0] + sums[1] + sums[2] + sums[3];
    const int segments = p.h_kv * static_cast<int>(all >> 32);
    int own_tiles = 0;
    if (segments <= grid && max(max(misc[8], misc[9]), max(misc[10], misc[11])) <= S::kWhole) {
      own_tiles = S::kWholeTiles;
    } else if (segments < grid) {  // ceil(nt / t) CTAs for each, nt / t + 1 at most
      const int t = max(S::tiles_at_once(false), (p.h_kv * static_cast<int>(all) + grid - segments - 1) / (grid - segments));
      if (t <= S::kOwn) own_tiles = t;
    }
    if (tid == 0) misc[17] = own_tiles;
    auto note = [&](int i) {
      // (own: at least ceil(nt / t) units further for each sequence)
      const int tiles = static_cast<int>(run), before = static_cast<int>(run >> 32);
      pre[i] = tiles;
      pre_units[i] = own_tiles > 0 ? tiles / own_tiles + before : tiles + S::kSegment * before;
    };
    for (int i = i0; i < i1; ++i) {
      note(i);
      run += counts(span_of(lens[i], p.L_cap, p.kv).nt);
    }
    if (tid == 127) note(p.B);
    named_bar_sync(3, 128);
    named_bar_arrive(4, kThreads);  // the working warps may look at it
    find_range();
    if (warp < 2) {
      // =========================== loads ===========================
      // The two warps take four tiles in turn: lane 8 i + r finds tile i and its run r of chunks (a page's rows, at most a
      // tile's; 16 keys where sink keys are folded in), reads that page's table entry a turn early, and issues the copy when
      // the tile's stage is free. One tile after the other, the chain of searches and loads took a warp 1300 cycles a tile,
      // twice the memory's time.
      const uint64_t policy = l2_policy_evict_first();
      const int page = 1 << p.kv.page_shift;
      struct Run {
        int64_t block;   // the first chunk's place in the cache, without the page's
        int id, chunks;  // the page's table entry; 0 chunks: nothing to load
      };
      auto run_at = [&](int i0) {
        Run r{0, 0, 0};
        const int x = beg + i0 + (lane >> 3);
        if (x >= end) return r;
        const Piece pc = locate(x);
        const DecodeSpan sp = span_of(lens[pc.b], p.L_cap, p.kv);
        const int n = pc.tl == 0 && sp.fold > 0 ? kFold : min(page, kKeys);
        const int row = (lane & 7) * n;
        const int key = sp.key_of(pc.tl, row);
        if (row >= kKeys || !sp.sees_any(key, n)) return r;
        r.id = p.kv.block_table[static_cast<int64_t>(pc.b) * p.kv.max_pages + (key >> p.kv.page_shift)];
        r.block = (static_cast<int64_t>(pc.j) << (p.kv.page_shift - 4)) + ((key & (page - 1)) / kChunk);
        r.chunks = n / kChunk;
        return r;
      };
      const int stop = (p.give_up_tile < 0 ? end : beg + min(end - beg, p.give_up_tile)) - beg;
      Run next = run_at(S::kTurn * warp);
      for (int i0 = S::kTurn * warp; i0 < stop && ok; i0 += 2 * S::kTurn) {
        const Run run = next;
        next = run_at(i0 + 2 * S::kTurn);
        const bool mine = run.chunks > 0;
        const bool there = mine && static_cast<uint32_t>(run.id) < static_cast<uint32_t>(p.kv.num_pages);
        const uint8_t* src = p.cache + ((static_cast<int64_t>(run.id) * p.h_kv << (p.kv.page_shift - 4)) + run.block) * kKv4Block;
        const uint32_t bytes = static_cast<uint32_t>(run.chunks * kKv4Block);
        // the tile's bytes, and its chunks that read as zeros
        uint32_t all = there ? bytes : 0, bad = mine && !there ? ((1u << run.chunks) - 1) << ((lane & 7) * run.chunks) : 0;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
          all += __shfl_xor_sync(0xffffffffu, all, d);
          bad |= __shfl_xor_sync(0xffffffffu, bad, d);
        }
        if (mine && !there && i0 + (lane >> 3) < stop) raise_status(p.status, kStatusBadPage);
        for (int it = i0; it < min(i0 + S::kTurn, stop); ++it) {
          const int st = it % kStages;
          wait(&empty[st], static_cast<uint32_t>(((it / kStages) & 1) ^ 1), kStatusWaitEmptyTimeout);
          if (!ok) break;
          if (lane == 8 * (it - i0)) {
            bad_chunks[st] = bad;
            last_tile[st] = it;
            mbar_arrive_expect_tx(&full[st], all);
          }
          __syncwarp();
          if (lane >> 3 == it - i0 && there)
            bulk_load(smem + st * kStageBytes + (lane & 7) * bytes, src, bytes, &full[st], policy);
        }
      }
      // no copy may outlive its CTA: the last of each stage
      named_bar_sync(2, 64);
      if (tid == 0) {
        if (stop < end - beg) atomicExch(p.status, kStatusWaitEmptyTimeout);
        for (int st = 0; st < kStages; ++st)
          if (last_tile[st] >= 0 && !mbar_wait(&full[st], static_cast<uint32_t>((last_tile[st] / kStages) & 1))) {
            atomicExch(p.status, kStatusDrainTimeout);
            break;
          }
      }
      __syncwarp();
    } else {
      // =========================== queries, pieces finished ===========================
      // Two warps. The first also prepares the queries, two pieces ahead. Of a piece a warp takes four of every eight heads, a
      // lane four dimensions.
      const int half = warp - 2;
      const int d4 = 4 * lane;
      struct Ahead {
        Piece pc;
        int x, pi;
      } ahead{};
      ahead.x = beg;
      auto prepare_next = [&]() {
        if (half != 0 || ahead.x >= end) return;
        ahead.pc = ahead.pi == 0 ? locate(beg) : after(ahead.pc, ahead.x);
        const int slot = ahead.pi & 1;
        wait(&q_empty[slot], ((ahead.pi >> 1) & 1) ^ 1, kStatusWaitEmptyTimeout);
        Queries<kNT>::prepare(smem + S::kQ + slot * S::kQBytes,
                              p.q + (static_cast<int64_t>(ahead.pc.b) * p.h_q + static_cast<int64_t>(ahead.pc.j) * p.G) * kD, p.G,
                              p.scale_log2, lane);
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&q_full[slot]);
        ahead.x += ahead.pc.n;
        ++ahead.pi;
      };
      prepare_next();
      prepare_next();
      int pi = 0;
      uint32_t merges = 0, copied = ~0u;  // batches joined, the last whose copies this warp issued
      Piece pc{};
      for (int x = beg; x < end; x += pc.n, ++pi) {
        pc = x == beg ? locate(x) : after(pc, x);
        // (a piece may take several limits)
        for (int i = 1; ok && i < p.piece_waits && !mbar_wait(h_full, pi & 1);) ++i;
        wait(h_full, pi & 1, kStatusWaitFullTimeout);
        const bool whole = pc.tl == 0 && pc.n == pc.nt;
        uint16_t* out = p.out + (static_cast<int64_t>(pc.b) * p.h_q + static_cast<int64_t>(pc.j) * p.G) * kD + d4;
        float* mine = p.partials + (static_cast<int64_t>(cta) * 2 + (pi == 0 ? 0 : 1)) * kGqaSlotFloats;
        Joined all;
        auto put = [&](float* to, int h) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (h + k < p.G) *reinterpret_cast<float4*>(to + 32 + (h + k) * kD + d4) = all.o[k];
          if (lane < 4) {
            to[h + lane] = all.ref;
            to[16 + h + lane] = all.sum;
          }
        };
        // the warps' parts
        for (int h = 4 * half; h < p.G; h += 8) {
          float* r = refs + h;
          all.clear();
          all.add<kWarps, 4>(r, r + kWarps * 16, 16, kWarps, join + h * kRow + d4, 8 * kNT * kRow, kRow, lane);
          if (whole) {
            all.store(out, h, p.G);
          } else {
            put(mine, h);
          }
        }
        if (!whole) {
          // A segment cut between CTAs: the last to publish its piece joins them all, in CTA order; of more than two batches, the
          // last of each kMost joins those and publishes the result in the first one's place, and the last of these joins those.
          // (All by one CTA: a sequence of 128K keys and one key/value head 41 us instead of 19, one of 10000 with 16 heads 26
          // instead of 16.) Partials (references and sums of 16 heads, then the heads' outputs) come with bulk copies into the
          // hand-over buffer, as many as fit it at once: with loads into registers a warp had a few of them under way, and 20
          // pieces took 8 us.
          auto cta_of = [&](int i) {
            const int big = rm * (q_units + 1);
            return i < big ? i / (q_units + 1) : rm + (i - big) / q_units;
          };
          const int unit0 = segment_unit(pc.b, pc.j, pc.nt, pc.seg0);
          const int c_first = own > 0 ? unit0 : cta_of(unit0 + extra);
          const int c_last = own > 0 ? unit0 + (pc.nt - 1) / own : cta_of(unit0 + extra + pc.nt - 1);
          const int part = 32 + kD * p.G;  // floats
          auto place_of = [&](int c) {
            return p.partials + (static_cast<int64_t>(c) * 2 + (range_start(c) >= unit0 ? 0 : 1)) * kGqaSlotFloats;
          };
          // Whether this CTA is the last of n that count there (both warps ask).
          auto last_of = [&](int counter, int n) {
            fence_proxy_async_all();  // (what was written is read with copies)
            named_bar_sync(1, 64);
            if (tid == 64) {
              // publishes what the barrier gathered (cumulativity), and sees what those before published
              const bool last = n == 1 || atom_add_acq_rel(&p.counters[counter], 1) == n - 1;
              if (last && n > 1) p.counters[counter] = 0;
              misc[16] = last;
            }
            __syncwarp();
            named_bar_sync(1, 64);
            return misc[16] != 0;
          };
          // The partials of n CTAs, `step` apart, to the output or (to) joined into a partial.
          auto join_parts = [&](int first, int step, int parts, float* to) {
            for (int h0 = 0; h0 < p.G; h0 += 8) {  // (both warps take every turn: they meet in it)
              const int h = h0 + 4 * half;
              all.clear();
              for (int i0 = 0; i0 < parts; i0 += S::kMost) {
                const int n = min(S::kMost, parts - i0);
                if (h0 == 0 || parts > S::kMost) {  // (else they are there already)
                  // what was read and written there plainly comes before the copies
                  fence_proxy_async_all();
                  named_bar_sync(1, 64);
                  if (half == 0 && ok) {
                    if (lane == 0) mbar_arrive_expect_tx(m_full, static_cast<uint32_t>(n * part) * 4u);
                    __syncwarp();
                    if (lane < n)
                      bulk_load(join + lane * part, place_of(first + (i0 + lane) * step), static_cast<uint32_t>(part) * 4u, m_full,
                                l2_policy_evict_first());
                    copied = merges;
                  }
                  wait(m_full, merges & 1, kStatusWaitFullTimeout);
                  ++merges;
                }
                if (h < p.G) all.add<S::kMost, 1>(join + h, join + 16 + h, part, n, join + 32 + h * kD + d4, part, kD, lane);
              }
              if (h >= p.G) continue;
              if (to) put(to, h);
              else all.store(out, h, p.G);
            }
          };
          // Counters: a segment's is its first CTA's, a group's too, and that of the second CTA counts groups. CTAs between the first
          // and the last have no other segment; a group of the last CTA alone needs no counter.
          const int parts = c_last - c_first + 1;
          const bool deep = parts > 2 * S::kMost;
          const int lead = deep ? c_first + (cta - c_first) / S::kMost * S::kMost : c_first;
          const int members = deep ? min(S::kMost, c_last + 1 - lead) : parts;
          const int groups = deep ? (parts + S::kMost - 1) / S::kMost : parts;
          bool joins = last_of(lead, members);
          if (deep && joins) {
            if (members > 1) join_parts(lead, 1, members, place_of(lead));
            joins = last_of(c_first + 1, groups);
          }
          if (joins) join_parts(c_first, deep ? S::kMost : 1, groups, nullptr);
          named_bar_sync(1, 64);  // misc[16] is written again by the next cut piece, the buffer by the next piece
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(h_empty);
        prepare_next();
      }
      if (!ok && copied != ~0u && !mbar_wait(m_full, copied & 1) && lane == 0) atomicExch(p.status, kStatusDrainTimeout);
      // ---- sequences with no keys (or a bad length) attend to nothing: output 0
      for (int b = cta; b < p.B; b += grid) {
        if (pre[b + 1] != pre[b]) continue;
        uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(b) * p.h_q * kD);
        for (int i = tid - 64; i < p.h_q * kD / 8; i += 64) o[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  } else {
    // =========================== work ===========================
    // Warp (i, c) takes unit c of tiles i, i + kTiles, ... of the CTA's list, whatever piece they belong to; a piece's part is
    // handed over when the next one begins, and nothing is waited for but the hand-over buffer. After a wait that ran out a
    // warp leaves and hands nothing back: the others' waits then run out with it, once each.
    reg_alloc<kRegsWork>();
    named_bar_sync(4, kThreads);
    find_range();
    auto work = [&](auto chunks) {
      constexpr int kUnit = decltype(chunks)::value, kUnits = kChunks / kUnit, kTiles = kWarps / kUnits;
      const int w = warp - 4;
      const int g = lane >> 2, t4 = lane & 3;
      const int c0 = w % kUnits * kUnit;
      Queries<kNT> q;
      State<kNT> s;
      Piece pc{};
      int it = w / kUnits, pi = 0;
      for (int x = beg; x < end; x += pc.n, ++pi) {
        pc = x == beg ? locate(x) : after(pc, x);
        const int slot = pi & 1;
        const int first = x - beg;  // the piece's first tile in this CTA's count
        wait(&q_full[slot], (pi >> 1) & 1, kStatusWaitFullTimeout);
        if (!ok) break;
        const bool any = it < first + pc.n;
        if (any) q.take(smem + S::kQ + slot * S::kQBytes, lane);
        s.clear();
        if (any) {
          const DecodeSpan sp = span_of(lens[pc.b], p.L_cap, p.kv);
          // the tiles whose keys the query sees all (a folded one is not among them)
          const int from = max(pc.tl, (sp.lo + kKeys - 1) / kKeys - sp.w0 + sp.ns) - pc.tl + first;
          const int to = min(pc.tl + pc.n, sp.len / kKeys - sp.w0 + sp.ns) - pc.tl + first;
          for (; it < first + pc.n; it += kTiles) {
            const int st = it % kStages;
            wait(&full[st], static_cast<uint32_t>((it / kStages) & 1), kStatusWaitFullTimeout);
            if (!ok) break;
            uint8_t* at = smem + st * kStageBytes + c0 * kKv4Block;
            const uint32_t bad = bad_chunks[st];
            float bias[kUnit][2] = {};
            bool none = false;
            if (it < from || it >= to || bad != 0) {
              // some keys are not seen, or read as zeros: their scales become 0 (what stands there may be NaN)
              none = true;
#pragma unroll
              for (int c = 0; c < kUnit; ++c) {
                const int key = sp.key_of(pc.tl + it - first, (c0 + c) * kChunk);
                const bool zero = bad >> (c0 + c) & 1;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const bool see = sp.sees(key + g + 8 * r);
                  bias[c][r] = see ? 0.0f : -INFINITY;
                  none &= !see;
                  if (t4 < 2 && (zero || !see))
                    *reinterpret_cast<uint2*>(at + c * kKv4Block + t4 * kKv4Values + kKv4Scales + 8 * (g + 8 * r)) = make_uint2(0u, 0u);
                }
              }
              none = __all_sync(0xffffffffu, none);
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (!none) s.add(q, at, bias, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive_many(&empty[st], kUnit);
          }
        }
        // ---- hand over
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[slot]);
        wait(h_empty, (pi & 1) ^ 1, kStatusWaitEmptyTimeout);
        if (!ok) break;
        float* ref = refs + w * 16;
        float* l_of = ref + kWarps * 16;
        float* to_o = join + w * 8 * kNT * kRow + 4 * g;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int head = 8 * nt + 2 * t4 + h;
            float v = s.sum[nt][h];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            if (g == 0) {
              ref[head] = s.ref[nt][h];
              l_of[head] = v;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<float4*>(to_o + head * kRow + 32 * k) =
                  make_float4(s.o[nt][2 * k][h], s.o[nt][2 * k][h + 2], s.o[nt][2 * k + 1][h], s.o[nt][2 * k + 1][h + 2]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(h_full);
      }
    };
    if (longs) {
      work(std::integral_constant<int, S::kLongUnit>());
    } else {
      work(std::integral_constant<int, S::kUnit>());
    }
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
    cudaFuncAttributes attr{};
    e = cudaFuncGetAttributes(&attr, kv4_decode_kernel<kNT>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the shares count on it
    e = cudaFuncSetAttribute(kv4_decode_kernel<kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Split<kNT>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev) done[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(kv4_decode_kernel<kNT>, dim3(grid), dim3(kThreads), Split<kNT>::kBytes, stream, p);
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
  // a tile takes at most some 0.9 us (16 heads a group), so 2^20 of them less than half a wait's limit
  p.piece_waits = 1 + (p.L_cap / kv4::kKeys >> 20);
  p.give_up_tile = plan.give_up_tile;
  return p.G <= 8 ? kv4::launch<1>(p, plan.num_ctas, stream) : kv4::launch<2>(p, plan.num_ctas, stream);
}

}  // namespace moe
