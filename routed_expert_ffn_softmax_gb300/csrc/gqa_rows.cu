// Attention of many query rows per key/value head over the paged cache (include/paged/moe_paged.h): prompts, chunks
// and drafted tokens (causal, sliding window, sink tokens), and the prefix a decode batch shares.
//
// A row is one (query token, query head); the G heads of a group read the same keys, so a block of 2 x (128 / G)
// consecutive tokens of one sequence makes 2 x 128 rows (token major) against one key/value head, two halves that
// share every key and value tile. Per tile of 128 keys and half, on tcgen05.mma:
//     S [128 rows x 128 keys] = Q . K^T        (Q and the K tile from shared memory, as TMA lands them)
//     O [128 rows x 128 dims] += P . V         (P from TMEM, the V tile read MN-major: the cache is never rearranged)
// 4 * 128 * 128 * 128 flops per half and tile: long prompts are bound by the tensor pipe, few rows behind long
// contexts by HBM. The halves alternate, so the softmax of one runs under the products of the other.
//
// Softmax: a thread owns a row (TMEM lane): its 128 scores come with one TMEM load and its probabilities leave with one
// store, so the row's maximum and sum need no exchange. (TMEM instructions that meet the running products stall: with
// two threads per row and four times the instructions, 16K prompts took 391 us instead of 357.) The store is in two
// parts, so that most of P . V starts before the last exponentials are done. O stays in TMEM; it is
// rescaled only when a row's maximum has grown by more than 2^8 since the reference in use (probabilities are then at
// most 2^8, exact to the same relative bf16 step, and sums stay far inside fp32), which after the first tiles is rare.
// Probabilities are rounded to bf16, since both factors of a tcgen05 product have one type and V's is bf16; 2^x is the
// hardware's approximation (2^-22 relative); everything else stays in fp32 until the output's one rounding.
//
// Work split: the key tiles of all (sequence, head, block) segments form one list (causal blocks have different
// lengths, windows bound them) and each CTA takes a contiguous range of it, so any mix of prompts balances to within
// a tile. Which range holds what comes from a small table kernel, since lengths are only known on the device. A
// segment cut between CTAs leaves (o, m, l) pieces that a third kernel joins in CTA order, one warp per row (joined in
// this kernel by whoever came last, pairs of pieces at a time, 8 chunks behind contexts took 61 us instead of 55). For a
// shared prefix the host knows the sizes: equal splits per segment, joined the same way; the decode kernel adds the
// result to the sequences' own keys.
//
// Per CTA, 12 warps: 0 TMA producer (Q per piece; K and V tiles alternate in a ring of 4 x 32 KB), 1 and 2 issue the
// MMAs of the two halves in turn, 3 announces the pieces and writes zeros for blocks that see nothing, 4-7 and 8-11 the
// softmax and output of the two halves.
//
// What bounds it: per tile a half's chain of scores, softmax and product, about 2580 cycles (products 1150 with their
// issue, softmax 1180 of which 512 are exponentials, the rest hand-over; the last exponentials under the product). TMEM
// holds two halves, so the tensor pipe is busy 74% of the time. GB300, whole calls: a 16K prompt behind a window of 4096 in
// 329 us (1463 TFLOP/s) and six prompts of up to 4095 tokens in 166 (1127) when replayed for milliseconds, 357 and 175
// (1350, 1068) timed over seconds, under the power cap; a prefix of 32K for 255 sequences 161 of the call's 243 (1700, this
// kernel alone). A call with few rows pays 7 us up to its first scores and 9 to join its pieces.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstdint>
#include <limits>

#include "gqa_paged.cuh"
#include "paged_device.cuh"
#include "moe_launch.h"

namespace moe {
namespace rows {

using namespace gqa;

constexpr int kD = 128;
constexpr int kHalf = 128;                  // rows of a half
constexpr int kStages = 4;
constexpr int kBox = kKeys * 64 * 2;        // queries: 128 rows x 64 dims
constexpr int kTile = 2 * kBox;             // one K or V tile, or the queries of a half: 32 KB
constexpr int kThreads = 384;
constexpr int kSoft = kHalf;                // softmax threads of a half, one per row
constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kTile;
constexpr int kOffBar = kOffRing + kStages * kTile;
constexpr int kItems = 4;                   // pieces announced ahead
constexpr int kNumBars = 2 * kStages + 2 + 2 * 5 + 1 + 2 * kItems;
constexpr int kOffItem = kOffBar + 256;
constexpr int kOutBytes = 4096;                  // per softmax warp 32 rows x 64 dimensions of bf16 output
constexpr int kOffOut = kOffItem + kItems * 64;
constexpr int kSmem = kOffOut + 8 * kOutBytes;
// Registers per thread: at launch, and after the warpgroups have shared them out (128 threads that load and issue,
// 256 softmax threads that hold a row of scores each).
constexpr int kRegsLaunch = 168;
constexpr int kRegsIo = 88;
constexpr int kRegsSoftmax = 208;
static_assert(128 * kRegsIo + 2 * kSoft * kRegsSoftmax <= kThreads * kRegsLaunch, "a larger share would wait forever");
static_assert(kNumBars * 8 + 12 <= 256, "barrier area");
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
static_assert(kRowTile == 2 * kHalf, "partials hold both halves");

// TMEM columns: scores of half h at 128 h (the probabilities, two a column, over their first 64), outputs behind.
constexpr int kTmemCols = 512;
__device__ constexpr uint32_t col_s(int h) { return 128u * h; }
__device__ constexpr uint32_t col_o(int h) { return 256u + 128u * h; }

// What a segment costs beside its tiles (its queries' load, the first scores and the output, which no product
// overlaps), in tiles: the CTAs' shares are cut so that those with many short segments get fewer tiles (ragged and
// 16K prompts take 168 and 340 us at 1, 166 and 329 at 2, 172 and 323 at 3).
constexpr int kSegCost = 2;

constexpr int kReaders = 3 + 2 * kSoft / 32;  // warps that read the announced pieces

constexpr int kTurnBar = 1;  // named barriers 1 and 2: the issuers' turns

// Keys of a tile whose probabilities are handed over first: their part of P . V runs under the exponentials of the rest,
// which take a warp 4 cycles each (16K and ragged prompts take 334 and 169 us with 64 keys first, 329 and 166 with 96; the
// tile as one costs 4% and 2% more than that).
constexpr int kFirst = 96;

constexpr float kGrowth = 8.0f;  // log2 of how far a row's maximum may outgrow its reference

struct Params {
  const int32_t* cu_q;       // [B + 1]
  const int32_t* seq_lens;   // [B]
  PagedKv kv;
  uint16_t* out;
  float* pieces_o;           // see piece_at
  float* pieces_m;           // [pieces][kRowTile]
  float* pieces_l;
  int32_t* status;
  // work is counted in units: a block's tiles and kSegCost more (none for a block that sees nothing)
  int32_t* pre;              // [B + 1] units of the sequences before, for one key/value head
  int32_t* base;             // [B + 1] row blocks of the sequences before
  int32_t* cum;              // [blocks + 1] units of the blocks before
  int4* join;                // [CTAs] the segment that begins in a CTA's share and ends past it: tok0, ntok, head, pieces
  const int32_t* prefix_table;
  int prefix_len, prefix_splits, prefix_blocks;
  int N, B, h_q, h_kv, G, half_tokens, max_blocks, L_cap;
  float scale_log2;
  int piece_waits;   // limits of a wait that may last as long as a piece
  int give_up_tile;  // failure-detection test: the producers stop before this tile (-1: never)
};

// Rows cu_q[b] .. of sequence b, 0 unless they lie within [0, N] in order.
__device__ __forceinline__ int tokens_of(const Params& p, int b, bool* bad) {
  const int x0 = p.cu_q[b], x1 = p.cu_q[b + 1];
  *bad = x0 < 0 || x1 < x0 || x1 > p.N;
  return *bad ? 0 : x1 - x0;
}

// One block of query rows against one key/value head.
struct Block {
  int seq;
  int tok0, ntok;  // packed tokens
  int pos0;        // position of the first
  Span sp;         // keys some row sees
};
__device__ __forceinline__ Block block_of(const Params& p, int b, int r) {
  Block k;
  k.seq = b;
  bool bad;
  const int n = tokens_of(p, b, &bad);
  int len = p.seq_lens[b];
  if (len < 0 || len > p.L_cap) len = 0;
  const int per = 2 * p.half_tokens;
  k.tok0 = p.cu_q[b] + r * per;
  k.ntok = min(per, n - r * per);
  k.pos0 = len - n + r * per;
  // a sequence without keys has queries at negative positions only
  k.sp = span_of_range(max(0, k.pos0 + k.ntok), window_start(k.pos0, p.kv.window), p.kv.n_sink);
  return k;
}

// ---------------------------------------------------------------- tables
constexpr int kTableThreads = 1024;

template <typename T>
__device__ __forceinline__ T scan_block(T v, T* sums) {  // inclusive over the block's threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T n = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += n;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const T out = v + (warp ? sums[warp - 1] : 0);
  __syncthreads();
  return out;
}

__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {  // last i < n with a[i] <= x
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Row blocks and work units before each sequence and each block.
__global__ void __launch_bounds__(kTableThreads) rows_tables_kernel(const Params p) {
  __shared__ int64_t wide_sums[32];
  __shared__ int sums[32];
  __shared__ int base[kGqaMaxSeqs + 1];
  const int tid = threadIdx.x;
  pdl_wait_predecessor();
  pdl_allow_successor();
  const int per = 2 * p.half_tokens;
  int nb[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * tid + k;
    nb[k] = 0;
    if (b < p.B) {
      bool bad;
      nb[k] = (tokens_of(p, b, &bad) + per - 1) / per;
      const int len = p.seq_lens[b];
      if (bad || len < 0 || len > p.L_cap) raise_status(p.status, kStatusBadSeqLen);
    }
  }
  // offsets that run over each other could ask for more blocks than N tokens make, and than 32 bits count: the tables
  // end there
  int64_t run = scan_block(static_cast<int64_t>(nb[0]) + nb[1], wide_sums) - nb[0] - nb[1];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * tid + k;
    if (b < p.B) {
      base[b] = static_cast<int>(min(run, static_cast<int64_t>(p.max_blocks)));
      if (run + nb[k] > p.max_blocks) raise_status(p.status, kStatusBadSeqLen);
    }
    run += nb[k];
    if (b + 1 == p.B) base[p.B] = static_cast<int>(min(run, static_cast<int64_t>(p.max_blocks)));
  }
  __syncthreads();
  const int blocks = base[p.B];
  for (int b = tid; b <= p.B; b += kTableThreads) p.base[b] = base[b];
  int carry = 0;
  for (int i0 = 0; i0 < blocks; i0 += kTableThreads) {
    const int i = i0 + tid;
    int nt = 0, b = 0;
    if (i < blocks) {
      b = last_at_most(base, p.B, i);
      nt = block_of(p, b, i - base[b]).sp.nt;
      if (nt > 0) nt += kSegCost;
    }
    const int t = carry + scan_block(nt, sums);
    if (i < blocks) {
      p.cum[i + 1] = t;
      // the sequences that end with this block's one (empty ones behind it too)
      for (int e = b + 1; e <= p.B && base[e] == i + 1; ++e) p.pre[e] = t;
    }
    if (tid == kTableThreads - 1) sums[0] = t;
    __syncthreads();
    carry = sums[0];
    __syncthreads();
  }
  if (tid == 0) p.cum[0] = 0;
  for (int b = tid; b <= p.B && base[b] == 0; b += kTableThreads) p.pre[b] = 0;
}

// ---------------------------------------------------------------- the list of units, and a CTA's pieces of it
struct Share {  // CTA c's units: the first rm CTAs take q + 1, the others q; CTAs past nc take none
  int total, nc, q, rm;
  __device__ __forceinline__ explicit Share(int t, int ctas) {
    total = t;
    nc = min(t, ctas);
    q = nc > 0 ? t / nc : 0;
    rm = nc > 0 ? t - q * nc : 0;
  }
  __device__ __forceinline__ int start(int c) const { return c < nc ? c * q + min(c, rm) : total; }
  __device__ __forceinline__ int cta_of(int i) const {
    const int big = rm * (q + 1);
    return i < big ? i / (q + 1) : rm + (i - big) / q;
  }
};

struct alignas(64) Piece {
  int j;            // key/value head
  int t0, n;        // tiles t0 .. t0 + n - 1 of the block's; n = 0: no more pieces
  int slot;         // where a partial goes, -1: the piece is the whole segment
  Block k;
};
static_assert(sizeof(Piece) == 64, "a piece's place in shared memory");

// last_at_most by a warp, 32 places at once: a search's loads wait for each other, and the CTA for its first piece.
__device__ __forceinline__ int warp_last_at_most(const int32_t* a, int n, int x) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = (threadIdx.x & 31) * step;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, i == 0 || (i < n && a[lo + i] <= x)));
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// Walks a CTA's pieces in order. A warp constructs it, one lane walks.
class Walk {
 public:
  __device__ __forceinline__ Walk(const Params& p) : p_(p) {
    if (p.prefix_table) {
      x_ = blockIdx.x;
      end_ = p.h_kv * p.prefix_blocks * p.prefix_splits;
      return;
    }
    const Share s(p.h_kv * p.pre[p.B], gridDim.x);
    x_ = s.start(blockIdx.x);
    end_ = s.start(blockIdx.x + 1);
    if (x_ >= end_) return;
    // the last sequence whose first unit is at most x (empty ones before it are skipped by the search)
    b_ = warp_last_at_most(p.pre, p.B, x_ / p.h_kv);
    const int first = p.pre[b_];
    const int tiles = p.pre[b_ + 1] - first;
    const int off = x_ - p.h_kv * first;
    j_ = off / tiles;
    const int rem = off - j_ * tiles;
    const int base = p.base[b_];
    i_ = base + warp_last_at_most(p.cum + base, p.base[b_ + 1] - base, first + rem);
    t_ = first + rem - p.cum[i_];
  }
  __device__ __forceinline__ bool next(Piece& c) {
    if (p_.prefix_table) {
      c.n = 0;
      if (x_ >= end_) return false;
      const int s = x_ % p_.prefix_splits;
      const int seg = x_ / p_.prefix_splits;
      const int per = 2 * p_.half_tokens;
      c.j = seg / p_.prefix_blocks;
      c.k.seq = 0;
      c.k.pos0 = 0;
      c.k.tok0 = (seg - c.j * p_.prefix_blocks) * per;
      c.k.ntok = min(per, p_.B - c.k.tok0);
      c.k.sp = span_of_range(p_.prefix_len, 0, 0);
      c.t0 = static_cast<int>(static_cast<int64_t>(s) * c.k.sp.nt / p_.prefix_splits);
      c.n = static_cast<int>(static_cast<int64_t>(s + 1) * c.k.sp.nt / p_.prefix_splits) - c.t0;
      c.slot = x_;
      x_ += gridDim.x;
      return true;
    }
    while (x_ < end_) {
      c.j = j_;
      c.k = block_of(p_, b_, i_ - p_.base[b_]);
      const int units = min(end_ - x_, c.k.sp.nt + kSegCost - t_);
      c.t0 = max(0, t_ - kSegCost);
      c.n = t_ + units - kSegCost - c.t0;
      // a cut piece that goes on from an earlier CTA's (at most one per CTA), and one that others go on from
      c.slot = c.n == c.k.sp.nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (c.t0 > 0 ? 0 : 1);
      x_ += units;
      t_ = 0;
      if (x_ < end_) {  // the next block with tiles: of this head, of the next head, of the next sequence
        ++i_;
        for (;;) {
          const int stop = p_.base[b_ + 1];
          while (i_ < stop && p_.cum[i_ + 1] == p_.cum[i_]) ++i_;
          if (i_ < stop) break;
          if (++j_ >= p_.h_kv) {
            j_ = 0;
            do ++b_;
            while (p_.pre[b_ + 1] == p_.pre[b_]);
          }
          i_ = p_.base[b_];
        }
      }
      if (c.n > 0) {
        last_ = c;
        return true;
      }
    }
    c.n = 0;
    return false;
  }
  // The segment that the share's last piece begins and later CTAs go on with, pieces = 0 when there is none.
  __device__ __forceinline__ int4 cut() const {
    if (p_.prefix_table || last_.n == 0 || last_.slot != 2 * static_cast<int>(blockIdx.x) + 1) return make_int4(0, 0, 0, 0);
    const Share s(p_.h_kv * p_.pre[p_.B], gridDim.x);
    const int past = last_.k.sp.nt - last_.t0 - last_.n;  // its tiles in later shares
    return make_int4(last_.k.tok0, last_.k.ntok, last_.j, s.cta_of(end_ - 1 + past) - static_cast<int>(blockIdx.x) + 1);
  }

 private:
  const Params& p_;
  int x_ = 0, end_ = 0;           // units done before, and where the CTA's share ends
  int b_ = 0, j_ = 0, i_ = 0;     // sequence, head, row block
  int t_ = 0;                     // unit within the block
  Piece last_{};
};

// ---------------------------------------------------------------- the attention kernel
template <int kN>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* v) {  // kN columns, a multiple of 16
  if constexpr (kN >= 32) {
    tmem_st32(taddr, reinterpret_cast<const uint32_t(&)[32]>(*v));
    tmem_store<kN - 32>(taddr + 32, v + 32);
  } else if constexpr (kN >= 16) {
    tmem_st16(taddr, reinterpret_cast<const uint32_t(&)[16]>(*v));
  }
}

// Bits c of keys cb + c (c = 0 .. 31) that are below `n`.
__device__ __forceinline__ uint32_t bits_below(int n, int cb) {
  const int k = n - cb;
  return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
}

__global__ void __launch_bounds__(kThreads, 1)
    gqa_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;   // [2]
  uint64_t* p_half = s_full + 2;    // [2]
  uint64_t* p_full = p_half + 2;    // [2]
  uint64_t* o_full = p_full + 2;    // [2]
  uint64_t* o_free = o_full + 2;    // [2]
  uint64_t* mma_done = o_free + 2;
  uint64_t* d_full = mma_done + 1;      // [kItems]
  uint64_t* d_empty = d_full + kItems;  // [kItems]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(d_empty + kItems);
  volatile uint32_t* turns_over = tmem_slot + 1;  // [2]: half 1's issuer has left the list; half 0's ends the turns

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // both issuers
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_full[h], 1);
      mbar_init(&p_half[h], kSoft / 32);  // one arrival per warp (likewise below)
      mbar_init(&p_full[h], kSoft / 32);
      mbar_init(&o_full[h], 1);
      mbar_init(&o_free[h], kSoft / 32);
    }
    mbar_init(mma_done, 2);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], kReaders);
    }
    turns_over[0] = turns_over[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
  }
  pdl_wait_predecessor();
  pdl_allow_successor();
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);  // after the wait: a predecessor may still hold columns
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // The pieces come announced in shared memory by warp 3, a few ahead, so that no other role keeps the walk's state in
  // registers or waits for its table look-ups.
  Piece* items = reinterpret_cast<Piece*>(smem + kOffItem);
  int di = 0;
  // A reader that has nothing to do for a piece, and the warp that announces them, wait for others to finish one.
  auto wait_piece = [&](uint64_t* bar, uint32_t parity) {
    bool done = false;
#pragma unroll 1
    for (int i = 0; i < p.piece_waits && !done; ++i) done = mbar_wait_soon(bar, parity);
    return done;
  };
  // The next piece's place, kItems when there is none; its reader copies what it needs and hands the place back.
  auto next_piece = [&]() -> int {
    const int s = di % kItems;
    const bool got = __all_sync(0xffffffffu, wait_piece(&d_full[s], static_cast<uint32_t>((di / kItems) & 1)));
    if (!got && lane == 0) atomicExch(p.status, kStatusWaitFullTimeout);
    ++di;
    return got && items[s].n > 0 ? s : kItems;
  };
  auto hand_back = [&](int s) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&d_empty[s]);
  };

  if (warp < 4) {
  reg_dealloc<kRegsIo>();
  if (warp == 0) {
    // =========================== TMA producer ===========================
    // A tile is 128 / page_size pages (one part of a page from 128 up): a lane of the lower half warp issues a K box, of
    // the upper half warp a V box. Pages no row sees are not loaded.
    const uint64_t policy_q = l2_policy_evict_first();
    const int page = 1 << p.kv.page_shift;
    const int rows = page < kKeys ? page : kKeys;
    const int row0 = (lane & 15) * rows;
    const bool is_v = lane >= 16;
    const bool mine = row0 < kKeys;
    int it = 0, pi = 0;
    int issued = 0;  // K and V tiles whose copies are under way or done
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_soon(bar, parity));
    };
    for (int s; ok && (s = next_piece()) < kItems;) {
      const Span sp = items[s].k.sp;
      const int32_t* table =
          p.prefix_table ? p.prefix_table : p.kv.block_table + static_cast<int64_t>(items[s].k.seq) * p.kv.max_pages;
      const int t0 = items[s].t0, t1 = t0 + items[s].n, j = items[s].j;
      const int tok0 = items[s].k.tok0, ntok = items[s].k.ntok;
      hand_back(s);
      auto entry = [&](int t) {  // this lane's page in tile t: -2 nothing to load, -1 a bad entry (reads as zeros)
        const int key = sp.key_tile(t) * kKeys + row0;
        if (!mine || !sp.sees_any(key, rows)) return -2;
        const int id = table[key >> p.kv.page_shift];
        return static_cast<uint32_t>(id) < static_cast<uint32_t>(p.kv.num_pages) ? id : -1;
      };
      int id = entry(t0);
      for (int t = t0; t < t1; ++t, ++it) {
        const int next = t + 1 < t1 ? entry(t + 1) : -2;
        const int key = sp.key_tile(t) * kKeys + row0;
        const int z = id < 0 ? -1 : id * p.h_kv + j;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id != -2 && !is_v)) * static_cast<uint32_t>(rows) * 256u;
        if (it == p.give_up_tile) ok = false;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int idx = 2 * it + kv;
          const int st = idx % kStages;
          wait_all(&empty[st], static_cast<uint32_t>(((idx / kStages) & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
          __syncwarp();
          issued = idx + 1;
          if (id != -2 && is_v == (kv == 1))
            tma_load_5d(smem + kOffRing + st * kTile + tile_row(row0), kv ? &tmV : &tmK, &full[st], 0, 0, 0,
                        (key & (page - 1)) >> 3, z, policy_q);
          if (kv == 0 && t == t0) {  // the queries go between the first K and V tiles
            wait_all(q_empty, static_cast<uint32_t>((pi & 1) ^ 1));
            if (!ok) break;
            if (lane == 0) {
              const int nh = ntok > p.half_tokens ? 2 : 1;
              mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(nh * p.half_tokens * p.G * 256));
              for (int h = 0; h < nh; ++h)
                for (int d = 0; d < 2; ++d)
                  tma_load_3d(smem + kOffQ + h * kTile + d * kBox, &tmQ, q_full, 64 * d, j * p.G,
                              tok0 + h * p.half_tokens, policy_q);
              ++pi;
            }
            pi = __shfl_sync(0xffffffffu, pi, 0);
          }
        }
        if (!ok) break;
        if (id == -1) raise_status(p.status, kStatusBadPage);
        id = next;
      }
    }
    if (!ok && lane == 0) atomicExch(p.status, kStatusWaitEmptyTimeout);
    // never leave copies in flight: the last stages and queries issued
    if (lane == 0) {
      for (int i = issued < kStages ? 0 : issued - kStages; i < issued; ++i)
        if (!mbar_wait_soon(&full[i % kStages], static_cast<uint32_t>((i / kStages) & 1))) {
          atomicExch(p.status, kStatusDrainTimeout);
          break;
        }
      if (pi > 0 && !mbar_wait_soon(q_full, static_cast<uint32_t>((pi - 1) & 1))) atomicExch(p.status, kStatusDrainTimeout);
    }
    __syncwarp();
  } else if (warp < 3) {
    // =========================== MMA issuer of half h ===========================
    // The tensor pipe holds few MMAs ahead, so whatever their issuer does in between (waits, commits: 300 to 400 cycles
    // in one warp for both halves) leaves it idle. So each half has an issuer, and a pair of named barriers passes the
    // turn: one waits for its operands while the other's MMAs run, and the halves stay half a period apart. (Without
    // turns their MMAs interleave, and both softmaxes wait for both products.) The whole warp runs the loop, so that
    // descriptors are warp-uniform values, as the instruction takes them; one elected lane issues.
    const int h = warp - 1;
    const uint32_t ring = uniform((smem_addr(smem) + kOffRing) >> 4);  // descriptors count 16 bytes
    const uint64_t q = umma_desc_sw128(0) + uniform((smem_addr(smem) + kOffQ + h * kTile) >> 4);
    const uint32_t d_s = uniform(tmem + col_s(h));
    const uint32_t d_o = uniform(tmem + col_o(h));
    const uint32_t idesc_s = umma_idesc_bf16_m128(kKeys);
    const uint32_t idesc_o = umma_idesc_bf16_m128(kD) | kIdescBMajorMN;
    const uint64_t desc_v = umma_desc_sw128_mn_sbo(0, kUpper, kGroupBytes);
    const int my_turn = kTurnBar + h, other_turn = kTurnBar + 1 - h;
    // After a wait that ran out this warp waits for nothing more (only for its turns), issues nothing and hands nothing
    // back: a stage it has not seen full is then never filled again over copies in flight, and the other roles' waits run
    // out in their turn, once each.
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok && !mbar_wait_soon(bar, parity)) ok = false;
    };
    uint32_t pv = 0, seg = 0;    // products P . V issued, pieces begun
    uint32_t st_k = 0, ph = 0;   // ring place and phase of the next K tile; the V tile due is the one before
    if (h == 1) named_bar_arrive(other_turn, 64);
    for (int pi = 0;; ++pi) {
      const uint32_t s = uniform(next_piece());
      if (s >= kItems) break;
      const bool active = uniform(h == 0 || items[s].k.ntok > p.half_tokens) != 0;
      const int n = static_cast<int>(uniform(items[s].n));
      hand_back(s);
      if (active) wait(q_full, static_cast<uint32_t>(pi & 1));
      for (int t = 0; t <= n; ++t) {
        const uint32_t st_v = st_k == 0 ? kStages - 1 : st_k - 1;
        if (t > 0) wait(&full[st_v], st_k == 0 ? ph ^ 1 : ph);
        if (t < n) wait(&full[st_k], ph);
        if (active) {
          if (t == 1) wait(&o_free[h], (seg++ & 1) ^ 1);
          if (t > 0) wait(&p_half[h], pv & 1);
        }
        tc_fence_after_sync();
        named_bar_sync(my_turn, 64);
        const uint64_t v = desc_v + (ring + st_v * (kTile >> 4));
        if (active && t > 0) {
          if (elect_one() && ok) {
            umma_bf16_tmem_a(d_o, d_s, v, idesc_o, t > 1);
#pragma unroll
            for (int x = 1; x < kFirst / 16; ++x)
              umma_bf16_tmem_a(d_o, d_s + 8 * x, v + x * (2 * kGroupBytes >> 4), idesc_o, true);
          }
          __syncwarp();
          wait(&p_full[h], pv++ & 1);
          tc_fence_after_sync();
        }
        if (elect_one() && ok) {
          if (active) {
            if (t > 0) {
#pragma unroll
              for (int x = kFirst / 16; x < kKeys / 16; ++x)
                umma_bf16_tmem_a(d_o, d_s + 8 * x, v + x * (2 * kGroupBytes >> 4), idesc_o, true);
            }
            // the scores overwrite the probabilities of the tile before, whose product was issued just now: MMAs of one
            // thread run in order
            if (t < n) {
              const uint64_t k = umma_desc_sw128_sbo(0, kGroupBytes) + (ring + st_k * (kTile >> 4));
#pragma unroll
              for (int x = 0; x < kD / 16; ++x)
                umma_bf16(d_s, q + (((x >> 2) * kBox + (x & 3) * 32) >> 4), k + (((x >> 2) * kUpper + (x & 3) * 32) >> 4),
                          idesc_s, x > 0);
            }
            // one commit tells of both: the output is read only after the last product or, to rescale it, with scores
            umma_commit(t < n ? &s_full[h] : &o_full[h]);
            if (t > 0) umma_commit(&empty[st_v]);
            if (t < n) umma_commit(&empty[st_k]);
            if (t == n - 1) umma_commit(q_empty);
          } else {
            if (t > 0) mbar_arrive(&empty[st_v]);
            if (t < n) mbar_arrive(&empty[st_k]);
            if (t == n - 1) mbar_arrive(q_empty);
          }
        }
        __syncwarp();
        named_bar_arrive(other_turn, 64);
        if (t < n) {
          st_k += 2;
          if (st_k >= kStages) {
            st_k -= kStages;
            ph ^= 1;
          }
        }
      }
    }
    // The turns have no limit of their own, so they go on until both issuers have left the list (one of them earlier, when
    // its wait for a piece ran out): half 0 ends them after it has seen that half 1 has.
    if (h == 0) {
      for (bool over = false; !over;) {
        named_bar_sync(my_turn, 64);
        over = __any_sync(0xffffffffu, turns_over[0] != 0);
        if (lane == 0) turns_over[1] = over;
        __syncwarp();
        named_bar_arrive(other_turn, 64);
      }
    } else {
      if (lane == 0) turns_over[0] = 1;
      __syncwarp();
      for (;;) {
        named_bar_sync(my_turn, 64);
        if (turns_over[1] != 0) break;
        named_bar_arrive(other_turn, 64);
      }
    }
    if (__any_sync(0xffffffffu, !ok) && lane == 0) atomicExch(p.status, kStatusWaitFullTimeout);
    // every MMA has completed before TMEM is released
    if (elect_one()) umma_commit(mma_done);
    if (!mbar_wait_soon(mma_done, 0) && lane == 0) atomicExch(p.status, kStatusDrainTimeout);
    __syncwarp();
  } else if (warp == 3) {
    // =========================== announces the pieces ===========================
    Walk walk(p);
    if (lane == 0) {
      for (bool more = true; more; ++di) {
        Piece c{};
        more = walk.next(c);
        const int s = di % kItems;
        if (!wait_piece(&d_empty[s], static_cast<uint32_t>(((di / kItems) & 1) ^ 1))) {
          atomicExch(p.status, kStatusWaitEmptyTimeout);
          break;
        }
        items[s] = c;
        mbar_arrive(&d_full[s]);  // releases the write
      }
      if (!p.prefix_table) p.join[blockIdx.x] = walk.cut();
    }
    __syncwarp();
    // =========================== and writes zeros for blocks that see nothing ===========================
    if (!p.prefix_table) {
      const int blocks = p.base[p.B];
      for (int i = blockIdx.x; i < blocks; i += gridDim.x) {
        if (p.cum[i + 1] != p.cum[i]) continue;
        const int b = last_at_most(p.base, p.B, i);
        const Block k = block_of(p, b, i - p.base[b]);
        uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(k.tok0) * p.h_q * kD);
        const int64_t n = static_cast<int64_t>(k.ntok) * p.h_q * (kD / 8);
        for (int64_t e = lane; e < n; e += 32) o[e] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  } else {
    reg_alloc<kRegsSoftmax>();
    // =========================== softmax and output of half h ===========================
    const int h = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the half
    const uint32_t tbase = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int i = r / p.G;                  // token of the half
    const int g = r - i * p.G;
    const bool neg = p.scale_log2 < 0.0f;
    const float scale = fabsf(p.scale_log2);
    bool ok = true;  // the same for the whole warp, which leaves when a wait has run out
    auto settle = [&](bool done) {
      ok = __all_sync(0xffffffffu, done);
      if (!ok) atomicExch(p.status, kStatusWaitFullTimeout);
    };
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) { settle(mbar_wait_soon(bar, parity)); };
    uint32_t cnt = 0;     // tiles of this half so far
    uint32_t pieces = 0;  // and pieces
    int it = 0;           // tiles of the CTA so far
    for (int s; (s = next_piece()) < kItems;) {
      const int t0 = items[s].t0, t1 = t0 + items[s].n;
      if (h == 1 && items[s].k.ntok <= p.half_tokens) {
        hand_back(s);
        it += t1 - t0;
        continue;
      }
      // what only some tiles or the output need stays in shared memory until then
      const Span& sp = items[s].k.sp;
      const int ntok = items[s].k.ntok, pos0 = items[s].k.pos0;
      const int tok = h * p.half_tokens + i;  // within the block
      const bool live = i < p.half_tokens && tok < ntok;
      const int pos = p.prefix_table ? p.prefix_len - 1 : pos0 + tok;
      const int end = live ? min(pos + 1, sp.len) : 0;   // keys below it are seen ...
      const int lo = window_start(pos, p.kv.window);     // ... from here on, or below n_sink
      // a tile needs no mask when the half's first token sees its end and its last token's window begins before it
      const int last = min(ntok, (h + 1) * p.half_tokens) - 1;
      const int end_min = p.prefix_table ? p.prefix_len : pos0 + h * p.half_tokens + 1;
      const int lo_max = p.prefix_table ? 0 : window_start(pos0 + last, p.kv.window);
      float m = -FLT_MAX, l = 0.0f;  // the row's reference and sum
      for (int t = t0; t < t1; ++t, ++it, ++cnt) {
        const int kb = sp.key_tile(t) * kKeys;
        wait_warp(&s_full[h], cnt & 1);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t sc[128];
        tmem_ld128(tbase + col_s(h), sc);
        if (neg) {
#pragma unroll
          for (int x = 0; x < 128; ++x) sc[x] ^= 0x80000000u;
        }
        const bool plain = kb + kKeys <= end_min && (kb >= lo_max || kb + kKeys <= p.kv.n_sink);
        if (!plain) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int cb = kb + 32 * w;
            const uint32_t see = bits_below(end, cb) & (~bits_below(lo, cb) | bits_below(p.kv.n_sink, cb));
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!((see >> x) & 1u)) sc[32 * w + x] = __float_as_uint(-INFINITY);
          }
          bool landed = true;
          if (h == 0 && !sp.sees(kb + r)) {
            // a key no row sees: its cache row is arbitrary (even NaN) and a zero probability times NaN is NaN, so
            // this row of the V tile is cleared (the wait orders the overwrite behind the tile's landing)
            const int idx = 2 * it + 1;
            const int st = idx % kStages;
            landed = mbar_wait_soon(&full[st], static_cast<uint32_t>((idx / kStages) & 1));
            if (landed) {
              uint4* v0 = reinterpret_cast<uint4*>(smem + kOffRing + st * kTile + tile_row(r));
              uint4* v1 = v0 + kUpper / 16;
#pragma unroll
              for (int x = 0; x < 8; ++x)  // neighbours in other banks
                v0[x ^ (r & 7)] = v1[x ^ (r & 7)] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          settle(landed);
          if (!ok) break;
        }
        // four chains, so that their latency overlaps
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 128; x += 2)
          mx[(x >> 1) & 3] = max3_f32(mx[(x >> 1) & 3], __uint_as_float(sc[x]), __uint_as_float(sc[x + 1]));
        const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        // O holds nothing until the row has seen a key
        const bool seen = m > -FLT_MAX;
        const bool grow = live && seen && m_new > m + kGrowth;
        if (__any_sync(0xffffffffu, grow)) {
          const float a = grow ? ex2_approx(m - m_new) : 1.0f;
          // the scores' commit covered the product before them
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            float o[16];
            uint32_t u[16];
            tmem_ld16(tbase + col_o(h) + 16 * x, o);
#pragma unroll
            for (int y = 0; y < 16; ++y) u[y] = __float_as_uint(o[y] * a);
            tmem_st16(tbase + col_o(h) + 16 * x, u);
          }
          l *= a;
          if (grow) m = m_new;
        }
        if (!seen) m = fmaxf(m, m_new);
        const uint64_t minus_m = pack_f32x2(-m, -m);
        const uint64_t scale2 = pack_f32x2(scale, scale);
        uint64_t sum2[4] = {0u, 0u, 0u, 0u};
        uint32_t u[64];
#pragma unroll
        for (int x = 0; x < 64; ++x) {
          if (x == kFirst / 2) {
            tmem_store<kFirst / 2>(tbase + col_s(h), u);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[h]);
          }
          float p0, p1;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(sc[2 * x]), __uint_as_float(sc[2 * x + 1])), scale2, minus_m), p0, p1);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          sum2[x & 3] = add_f32x2(sum2[x & 3], pack_f32x2(p0, p1));
          const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
          u[x] = *reinterpret_cast<const uint32_t*>(&b);
        }
        tmem_store<64 - kFirst / 2>(tbase + col_s(h) + kFirst / 2, u + kFirst / 2);
        float s0, s1;
        unpack_f32x2(add_f32x2(add_f32x2(sum2[0], sum2[1]), add_f32x2(sum2[2], sum2[3])), s0, s1);
        l += s0 + s1;
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[h]);
      }
      // the piece's output, into registers, so that the next products need not wait for its stores
      if (ok) wait_warp(&o_full[h], pieces++ & 1);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t o[128];
      tmem_ld128(tbase + col_o(h), o);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[h]);
      const int row = h * kHalf + r;
      const int j = items[s].j, slot = items[s].slot, tok0 = items[s].k.tok0;
      hand_back(s);
      if (l == 0.0f) {  // (a query of NaN has a sum of NaN, and its output)
#pragma unroll
        for (int x = 0; x < 128; ++x) o[x] = 0u;
      }
      if (slot < 0) {
        // a thread's row is 256 bytes from its neighbour's: through shared memory, so that eight lanes write 128 bytes of
        // a row together (a store instruction then touches 4 lines instead of 32)
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        uint8_t* stage = smem + kOffOut + (warp - 4) * kOutBytes;
        const int64_t mine = live ? static_cast<int64_t>(tok0 + tok) * p.h_q + j * p.G + g : -1;
        int64_t to[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) to[y] = __shfl_sync(0xffffffffu, mine, 4 * y + (lane >> 3));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 64 * x + 8 * y + 2 * e;
              const __nv_bfloat162 ab = __floats2bfloat162_rn(__uint_as_float(o[at]) * inv, __uint_as_float(o[at + 1]) * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&ab);
            }
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((y ^ lane) & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = 4 * y + (lane >> 3);
            const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((lane ^ rr) & 7) * 16);
            if (to[y] >= 0) *reinterpret_cast<uint4*>(p.out + to[y] * kD + 64 * x + 8 * (lane & 7)) = w;
          }
          __syncwarp();
        }
      } else if (live) {
#pragma unroll
        for (int x = 0; x < 16; ++x) st_global_v8(p.pieces_o + piece_at(slot, row, 8 * x), o + 8 * x);
        p.pieces_m[static_cast<int64_t>(slot) * kRowTile + row] = m;
        p.pieces_l[static_cast<int64_t>(slot) * kRowTile + row] = l;
      }
    }
  }

  // ---- teardown: every role has finished; warp 1 releases TMEM
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- joining pieces
constexpr int kMergeThreads = 256;
constexpr int kMergeParts = 16;  // CTAs per cut segment, which mostly has two or three pieces
constexpr int kJoinParts = 32;   // CTAs per segment of a prefix, which may have tens: a row for each warp

// Joins a row's pieces in key order: the first, then n - 1 more from `next` on, `stride` apart. Lane: 4 dimensions.
template <int kChunk>  // pieces whose loads are in flight together
__device__ __forceinline__ void join_row(const Params& p, int row, int64_t first, int64_t next, int stride, int n,
                                         float& M, float& L, float4& O) {
  const int lane = threadIdx.x & 31;
  M = -FLT_MAX;
  L = 0.0f;
  O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s0 = 0; s0 < n; s0 += kChunk) {
    float mc[kChunk], lc[kChunk];
    float4 oc[kChunk];
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      if (s0 + u >= n) continue;
      const int64_t slot = s0 + u == 0 ? first : next + static_cast<int64_t>(s0 + u - 1) * stride;
      mc[u] = p.pieces_m[slot * kRowTile + row];
      lc[u] = p.pieces_l[slot * kRowTile + row];
      oc[u] = *reinterpret_cast<const float4*>(p.pieces_o + piece_at(slot, row, 4 * lane));
    }
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      if (s0 + u >= n) continue;
      const float mn = fmaxf(M, mc[u]);
      const float a = exp2f(M - mn), b = exp2f(mc[u] - mn);
      O.x = O.x * a + oc[u].x * b;
      O.y = O.y * a + oc[u].y * b;
      O.z = O.z * a + oc[u].z * b;
      O.w = O.w * a + oc[u].w * b;
      L = L * a + lc[u] * b;
      M = mn;
    }
  }
}

// CTA (c, part) joins its rows of the segment whose first tile is in CTA c's share and whose last is not.
__global__ void __launch_bounds__(kMergeThreads) rows_merge_kernel(const Params p) {
  pdl_wait_predecessor();
  pdl_allow_successor();
  const int c = blockIdx.x;
  const int4 seg = p.join[c];  // tok0, ntok, head, pieces
  const int row0 = blockIdx.y * (kRowTile / kMergeParts);
  if (seg.w == 0) return;
  for (int row = row0 + (threadIdx.x >> 5); row < row0 + kRowTile / kMergeParts; row += kMergeThreads / 32) {
    const int hf = row / kHalf;
    const int ti = (row - hf * kHalf) / p.G;
    const int tok = hf * p.half_tokens + ti;
    if (ti >= p.half_tokens || tok >= seg.y) continue;
    float M, L;
    float4 O;
    join_row<4>(p, row, 2 * static_cast<int64_t>(c) + 1, 2 * static_cast<int64_t>(c + 1), 2, seg.w, M, L, O);
    const float inv = L != 0.0f ? 1.0f / L : 0.0f;
    const __nv_bfloat162 x0 = __floats2bfloat162_rn(O.x * inv, O.y * inv);
    const __nv_bfloat162 x1 = __floats2bfloat162_rn(O.z * inv, O.w * inv);
    uint16_t* o = p.out + (static_cast<int64_t>(seg.x + tok) * p.h_q + seg.z * p.G + (row - hf * kHalf - ti * p.G)) * kD;
    reinterpret_cast<uint2*>(o)[threadIdx.x & 31] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1));
  }
}

// Joins the splits of each segment of a shared prefix into its first piece.
__global__ void __launch_bounds__(kMergeThreads) prefix_join_kernel(const Params p) {
  pdl_allow_successor();  // the decode kernel's own keys need nothing of the prefix
  pdl_wait_predecessor();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.prefix_splits;
  const int tok0 = (blockIdx.x % p.prefix_blocks) * 2 * p.half_tokens;
  const int row0 = blockIdx.y * (kRowTile / kJoinParts);
  for (int row = row0 + (threadIdx.x >> 5); row < row0 + kRowTile / kJoinParts; row += kMergeThreads / 32) {
    const int hf = row / kHalf;
    const int ti = (row - hf * kHalf) / p.G;
    if (ti >= p.half_tokens || tok0 + hf * p.half_tokens + ti >= p.B) continue;
    float M, L;
    float4 O;
    join_row<10>(p, row, first, first + 1, 1, p.prefix_splits, M, L, O);
    *reinterpret_cast<float4*>(p.pieces_o + piece_at(first, row, 4 * (threadIdx.x & 31))) = O;
    if ((threadIdx.x & 31) == 0) {
      p.pieces_m[first * kRowTile + row] = M;
      p.pieces_l[first * kRowTile + row] = L;
    }
  }
}

// ---------------------------------------------------------------- host
bool encode_q(CUtensorMap* map, const uint16_t* base, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
  const cuuint64_t dims[3] = {kD, d1, d2};
  const cuuint64_t strides[2] = {kD * 2, d1 * kD * 2};
  const cuuint32_t box[3] = {64, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  TensorMapEncodeFn enc = tensor_map_encoder();
  return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace rows

cudaError_t launch_gqa_rows(const GqaRowsPlan& plan, cudaStream_t stream) {
  using namespace rows;
  const int G = plan.h_q / plan.h_kv;
  const int page = 1 << plan.paged.page_shift;
  const int box_rows = page < kKeys ? page : kKeys;
  const bool prefix = plan.prefix_table != nullptr;
  Params p{};
  p.half_tokens = kHalf / G;
  CUtensorMap tk, tv, tq;
  if (!encode_paged(&tk, plan.k_cache, plan.paged.num_pages, plan.h_kv, page, box_rows) ||
      !encode_paged(&tv, plan.v_cache, plan.paged.num_pages, plan.h_kv, page, box_rows) ||
      !encode_q(&tq, plan.q, plan.h_q, plan.N, G, p.half_tokens))
    return cudaErrorInvalidValue;
  const int64_t pieces = prefix ? static_cast<int64_t>(plan.h_kv) * plan.prefix_blocks * plan.prefix_splits
                                : 2 * static_cast<int64_t>(kRowsCtas);
  p.cu_q = plan.cu_q;
  p.seq_lens = plan.seq_lens;
  p.kv = plan.paged;
  p.out = plan.out;
  p.pieces_o = plan.pieces;
  p.pieces_m = plan.pieces + pieces * kRowTile * kD;
  p.pieces_l = p.pieces_m + pieces * kRowTile;
  p.status = plan.status;
  p.join = reinterpret_cast<int4*>(plan.tables);
  p.pre = plan.tables + 4 * kRowsCtas;
  p.base = p.pre + plan.B + 1;
  p.cum = p.base + plan.B + 1;
  p.prefix_table = plan.prefix_table;
  p.prefix_len = plan.prefix_len;
  p.prefix_splits = plan.prefix_splits;
  p.prefix_blocks = plan.prefix_blocks;
  p.N = plan.N;
  p.B = plan.B;
  p.h_q = plan.h_q;
  p.h_kv = plan.h_kv;
  p.G = G;
  p.max_blocks = plan.N / (2 * p.half_tokens) + plan.B;
  p.L_cap = plan.paged.max_pages * page;
  // A scale of 0 makes all scores equal, but the mask's infinities need a factor other than 0: the least there is, which
  // leaves no finite score above 5e-7.
  p.scale_log2 = plan.scale_log2 == 0.0f ? std::numeric_limits<float>::denorm_min() : plan.scale_log2;
  // a tile takes some 1.3 us, so 2^18 of them less than half a wait's limit
  p.piece_waits = 1 + (std::max(p.L_cap, p.prefix_len) / kKeys >> 18);
  p.give_up_tile = plan.give_up_tile;

  constexpr int kMaxDev = 64;  // the shared-memory opt-in is per device: done once on each
  static std::atomic<bool> done[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDev || !done[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, gqa_rows_kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the shares are counted from it
    e = cudaFuncSetAttribute(gqa_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev) done[dev].store(true, std::memory_order_release);
  }
  const int ctas = plan.num_sms;
  if (prefix) {
    p.kv.window = 0;
    p.kv.n_sink = 0;
    const int grid = pieces < ctas ? static_cast<int>(pieces) : ctas;
    e = launch_pdl(gqa_rows_kernel, dim3(grid), dim3(kThreads), kSmem, stream, tk, tv, tq, p);
    if (e != cudaSuccess || plan.prefix_splits == 1) return e;
    return launch_pdl(prefix_join_kernel, dim3(static_cast<unsigned>(pieces / plan.prefix_splits), kJoinParts),
                      dim3(kMergeThreads), 0, stream, p);
  }
  e = launch_pdl(rows_tables_kernel, dim3(1), dim3(kTableThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(gqa_rows_kernel, dim3(ctas), dim3(kThreads), kSmem, stream, tk, tv, tq, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(rows_merge_kernel, dim3(ctas, kMergeParts), dim3(kMergeThreads), 0, stream, p);
}

}  // namespace moe
