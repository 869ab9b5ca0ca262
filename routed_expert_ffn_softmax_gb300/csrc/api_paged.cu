// C ABI of the serving path over a paged key/value cache (include/paged/moe_paged.h): host-side argument
// checks, workspace layout and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "moe_launch.h"
#include "paged/moe_paged.h"
#include "paged/moe_paged_test.h"

namespace {

using namespace moe::api;

// Workspace: the control block (status word; the plan's ticket at byte 8; stream-K counters at byte 256), the
// decode kernel's partials, the row-block kernel's tables, then its partials.
constexpr size_t kTicketOffset = 8;
constexpr size_t kDecodePartialBytes = sizeof(float) * static_cast<size_t>(moe::kPartialCtas) * 2 * moe::kGqaSlotFloats;

// Splits of each of `segs` segments of a shared prefix of `tiles` key tiles over the CTAs: whole waves of pieces, each
// its tiles and about 3 tiles' time of start and output, and for joining about 1/33 of a tile's time per piece (with 1/50
// or 1/25 8 sequences behind 8K keys take 29.7 or 28.2 us instead of 28.3, 255 behind 32K 257 or 265 instead of 257).
constexpr int kMaxPrefixPieces = 4 * moe::kRowsCtas;
int prefix_splits(int64_t segs, int tiles) {
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= tiles && (s == 1 || segs * s <= kMaxPrefixPieces); ++s) {
    const int64_t waves = (segs * s + moe::kRowsCtas - 1) / moe::kRowsCtas;
    const double cost = static_cast<double>(waves) * ((tiles + s - 1) / s + 3) + 0.03 * static_cast<double>(segs * s);
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

struct Layout {
  size_t partials, tables, pieces, total;
  int prefix_blocks, prefix_splits;
};

// Queries per 128-row half of a row block.
int half_tokens(int G) { return 128 / G; }

Layout layout(int64_t N, int64_t B, int h_q, int h_kv, int prefix_len) {
  Layout L{};
  const int per_block = 2 * half_tokens(h_q / h_kv);
  size_t o = kCtrlBytes;
  L.partials = o;
  o = align_up(o + kDecodePartialBytes);
  L.tables = o;
  // per CTA the segment it cuts; per sequence and per row block the work before
  const int64_t blocks = N / per_block + B;
  o = align_up(o + sizeof(int32_t) * static_cast<size_t>(4 * moe::kRowsCtas + 2 * (B + 1) + blocks + 1));
  L.pieces = o;
  int64_t pieces = 2 * moe::kRowsCtas;
  if (prefix_len > 0) {
    L.prefix_blocks = static_cast<int>((B + per_block - 1) / per_block);
    const int64_t segs = static_cast<int64_t>(L.prefix_blocks) * h_kv;
    L.prefix_splits = prefix_splits(segs, (prefix_len + 127) / 128);
    // (the bound does not depend on the split, so that a workspace for larger sizes serves smaller ones)
    pieces = segs > kMaxPrefixPieces ? segs : kMaxPrefixPieces;
  }
  o = align_up(o + sizeof(float) * static_cast<size_t>(pieces) * moe::kRowsPieceFloats);
  L.total = o;
  return L;
}

moe_status_t check_heads(int64_t N, int64_t B, int h_q, int h_kv, int d, int prefix_len) {
  if (N < 0 || B < 0 || h_q < 1 || h_kv < 1 || d < 1 || prefix_len < 0 || h_q % h_kv) return MOE_ERR_INVALID_ARG;
  if (d != 128 || h_q / h_kv > 16 || B > moe::kGqaMaxSeqs) return MOE_ERR_UNSUPPORTED;
  if (N * h_q > INT32_MAX || prefix_len > INT32_MAX - 128) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int page_shift(int page_size) {  // -1 unless a power of two in 16 .. 1024
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

moe_status_t check_pages(int h_kv, int num_pages, int page_size, int max_pages) {
  if (num_pages < 1 || max_pages < 1 || page_shift(page_size) < 0) return MOE_ERR_INVALID_ARG;
  const int64_t p = page_size;
  if (num_pages * p > INT32_MAX || max_pages * p > INT32_MAX - 128 || static_cast<int64_t>(num_pages) * h_kv > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// What the three attention calls check alike.
struct Attention {
  const uint16_t *q, *k_cache, *v_cache;
  const int32_t *block_table, *seq_lens;
  int N, B, h_q, h_kv, d, num_pages, page_size, max_pages;
  float scale;
  int window, n_sink, prefix_len;
  uint16_t* out;
  void* workspace;
  size_t ws_bytes;
};

moe_status_t check_attention(const Attention& a) {
  moe_status_t st = check_heads(a.N, a.B, a.h_q, a.h_kv, a.d, a.prefix_len);
  if (st != MOE_OK) return st;
  st = check_pages(a.h_kv, a.num_pages, a.page_size, a.max_pages);
  if (st != MOE_OK) return st;
  if (!std::isfinite(a.scale) || a.window < 0 || a.n_sink < 0) return MOE_ERR_INVALID_ARG;
  // key tiles are counted in 32 bits, over all key/value heads and row blocks
  const int per_block = 2 * half_tokens(a.h_q / a.h_kv);
  const int64_t tiles = (static_cast<int64_t>(a.max_pages) * a.page_size + 127) / 128 + 8;
  const int64_t blocks = a.N / per_block + a.B;
  if (static_cast<double>(tiles) * a.h_kv * blocks > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (a.B == 0 || a.N == 0) return MOE_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.block_table || !a.seq_lens || !a.out || !a.workspace)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.out, 16) ||
      !aligned(a.block_table, 4) || !aligned(a.seq_lens, 4) || !aligned(a.workspace, kAlign))
    return MOE_ERR_INVALID_ARG;
  if (a.ws_bytes < layout(a.N, a.B, a.h_q, a.h_kv, a.prefix_len).total) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

moe::PagedKv paged_of(const Attention& a) {
  moe::PagedKv kv{};
  kv.block_table = a.block_table;
  kv.num_pages = a.num_pages;
  kv.page_shift = page_shift(a.page_size);
  kv.max_pages = a.max_pages;
  kv.window = a.window;
  kv.n_sink = a.n_sink;
  return kv;
}

float scale_log2(float scale) { return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634); }

// moe_test_paged_give_up
std::atomic<int> g_give_up_tile{-1};

moe::GqaPlan decode_plan(const Attention& a, int sms) {
  char* ws = static_cast<char*>(a.workspace);
  moe::GqaPlan plan{};
  plan.paged = paged_of(a);
  plan.q = a.q;
  plan.k_cache = a.k_cache;
  plan.v_cache = a.v_cache;
  plan.seq_lens = a.seq_lens;
  plan.out = a.out;
  plan.partials = reinterpret_cast<float*>(ws + kCtrlBytes);
  plan.counters = reinterpret_cast<int32_t*>(ws + kCountersOffset);
  plan.status = reinterpret_cast<int32_t*>(ws);
  plan.B = a.B;
  plan.h_q = a.h_q;
  plan.h_kv = a.h_kv;
  plan.L_cap = a.max_pages * a.page_size;
  plan.scale_log2 = scale_log2(a.scale);
  plan.num_ctas = sms < moe::kPartialCtas ? sms : moe::kPartialCtas;
  plan.give_up_tile = g_give_up_tile.load(std::memory_order_relaxed);
  return plan;
}

moe::GqaRowsPlan rows_plan(const Attention& a, const Layout& L, int sms) {
  char* ws = static_cast<char*>(a.workspace);
  moe::GqaRowsPlan plan{};
  plan.q = a.q;
  plan.k_cache = a.k_cache;
  plan.v_cache = a.v_cache;
  plan.seq_lens = a.seq_lens;
  plan.paged = paged_of(a);
  plan.out = a.out;
  plan.status = reinterpret_cast<int32_t*>(ws);
  plan.tables = reinterpret_cast<int32_t*>(ws + L.tables);
  plan.pieces = reinterpret_cast<float*>(ws + L.pieces);
  plan.N = a.N;
  plan.B = a.B;
  plan.h_q = a.h_q;
  plan.h_kv = a.h_kv;
  plan.scale_log2 = scale_log2(a.scale);
  plan.num_sms = sms < moe::kRowsCtas ? sms : moe::kRowsCtas;
  plan.give_up_tile = g_give_up_tile.load(std::memory_order_relaxed);
  return plan;
}

}  // namespace

extern "C" {

size_t moe_paged_workspace_size(int N, int B, int h_q, int h_kv, int d, int prefix_len) {
  if (check_heads(N, B, h_q, h_kv, d, prefix_len) != MOE_OK) return 0;
  return layout(N, B, h_q, h_kv, prefix_len).total;
}

moe_status_t moe_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size, int num_pages,
                            const int32_t* free_pages, int n_free, const int32_t* free_count, int32_t* block_table,
                            int max_pages, int32_t* seq_lens, int32_t* cu_new, int32_t* positions, int32_t* slots,
                            int n_rows, int32_t* free_left, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  if (B < 0 || n_free < 0 || n_rows < 0) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_pages(1, num_pages, page_size, max_pages);
  if (st != MOE_OK) return st;
  if (B > moe::kGqaMaxSeqs || static_cast<int64_t>(B) * max_pages > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!ctx_lens || !new_lens || !free_count || !block_table || !seq_lens || !cu_new || !free_left || !workspace ||
      (n_free > 0 && !free_pages) || (n_rows > 0 && (!positions || !slots)))
    return MOE_ERR_INVALID_ARG;
  const void* words[] = {ctx_lens, new_lens, free_pages, free_count, block_table, seq_lens, cu_new, positions, slots,
                         free_left};
  for (const void* w : words)
    if (!aligned(w, 4)) return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kCtrlBytes) return MOE_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  moe::PagedPlanArgs a{};
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu_new = cu_new;
  a.positions = positions;
  a.slots = slots;
  a.free_left = free_left;
  a.ticket = reinterpret_cast<int32_t*>(ws + kTicketOffset);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.B = B;
  a.n_rows = n_rows;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.page_shift = page_shift(page_size);
  return cuda_status(moe::launch_paged_plan(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_qk_norm_rope(const uint16_t* qkv, int64_t row_stride, int N, int h_q, int h_kv, int d,
                              const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* inv_freq,
                              int rot_dim, int interleaved, const int32_t* positions, const int32_t* slots,
                              uint16_t* q_out, uint16_t* k_cache, uint16_t* v_cache, int num_pages, int page_size,
                              moe_stream_t stream) {
  if (N < 0 || h_q < 1 || h_kv < 1 || d < 1 || rot_dim < 0 || rot_dim > d || rot_dim % 16 || interleaved < 0 ||
      interleaved > 1 || !std::isfinite(eps) || eps < 0.0f)
    return MOE_ERR_INVALID_ARG;
  if (d != 128) return MOE_ERR_UNSUPPORTED;
  const int64_t heads = static_cast<int64_t>(h_q) + 2 * static_cast<int64_t>(h_kv);
  if (heads * d > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (row_stride < heads * d || row_stride % 8) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_pages(h_kv, num_pages, page_size, 1);
  if (st != MOE_OK) return st;
  if (N == 0) return MOE_OK;
  if (!qkv || !positions || !slots || !q_out || !k_cache || !v_cache || (rot_dim > 0 && !inv_freq))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(inv_freq, 4) || !aligned(positions, 4) ||
      !aligned(slots, 4))
    return MOE_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  moe::QkNormRopeArgs a{};
  a.qkv = qkv;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.slots = slots;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.row_stride = row_stride;
  a.eps = eps;
  a.N = N;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  return cuda_status(moe::launch_qk_norm_rope(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_gqa_paged_decode(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache,
                                  const int32_t* block_table, const int32_t* seq_lens, int B, int h_q, int h_kv,
                                  int d, int num_pages, int page_size, int max_pages, float scale, int window,
                                  int n_sink, uint16_t* out, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  const Attention a{q, k_cache, v_cache, block_table, seq_lens, B, B, h_q, h_kv, d, num_pages, page_size, max_pages,
                    scale, window, n_sink, 0, out, workspace, ws_bytes};
  const moe_status_t st = check_attention(a);
  if (st != MOE_OK || B == 0) return st;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  return cuda_status(moe::launch_gqa_decode(decode_plan(a, sms), reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_gqa_paged_prefill(const uint16_t* q, const int32_t* cu_q, const uint16_t* k_cache,
                                   const uint16_t* v_cache, const int32_t* block_table, const int32_t* seq_lens, int N,
                                   int B, int h_q, int h_kv, int d, int num_pages, int page_size, int max_pages,
                                   float scale, int window, int n_sink, uint16_t* out, void* workspace,
                                   size_t ws_bytes, moe_stream_t stream) {
  const Attention a{q, k_cache, v_cache, block_table, seq_lens, N, B, h_q, h_kv, d, num_pages, page_size, max_pages,
                    scale, window, n_sink, 0, out, workspace, ws_bytes};
  const moe_status_t st = check_attention(a);
  if (st != MOE_OK || B == 0 || N == 0) return st;
  if (!cu_q || !aligned(cu_q, 4)) return MOE_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  const Layout L = layout(N, B, h_q, h_kv, 0);
  moe::GqaRowsPlan plan = rows_plan(a, L, sms);
  plan.cu_q = cu_q;
  return cuda_status(moe::launch_gqa_rows(plan, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_gqa_prefix_decode(const uint16_t* q, const int32_t* prefix_table, int prefix_len,
                                   const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* block_table,
                                   const int32_t* seq_lens, int B, int h_q, int h_kv, int d, int num_pages,
                                   int page_size, int max_pages, float scale, uint16_t* out, void* workspace,
                                   size_t ws_bytes, moe_stream_t stream) {
  const Attention a{q, k_cache, v_cache, block_table, seq_lens, B, B, h_q, h_kv, d, num_pages, page_size, max_pages,
                    scale, 0, 0, prefix_len, out, workspace, ws_bytes};
  const moe_status_t st = check_attention(a);
  if (st != MOE_OK || B == 0) return st;
  if (prefix_len > 0 && (!prefix_table || !aligned(prefix_table, 4))) return MOE_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  moe::GqaPlan own = decode_plan(a, sms);
  if (prefix_len > 0) {
    const Layout L = layout(B, B, h_q, h_kv, prefix_len);
    moe::GqaRowsPlan plan = rows_plan(a, L, sms);
    plan.prefix_table = prefix_table;
    plan.prefix_len = prefix_len;
    plan.prefix_blocks = L.prefix_blocks;
    plan.prefix_splits = L.prefix_splits;
    const cudaError_t e = moe::launch_gqa_rows(plan, s);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    const int64_t pieces = static_cast<int64_t>(h_kv) * L.prefix_blocks * L.prefix_splits;
    own.prefix.o = plan.pieces;
    own.prefix.m = plan.pieces + pieces * moe::kRowTile * 128;
    own.prefix.l = own.prefix.m + pieces * moe::kRowTile;
    own.prefix.stride = L.prefix_splits;
    own.prefix.blocks = L.prefix_blocks;
    own.prefix.half_seqs = half_tokens(h_q / h_kv);
  }
  return cuda_status(moe::launch_gqa_decode(own, s));
}

moe_status_t moe_test_paged_give_up(int tile) {
  if (tile < -1) return MOE_ERR_INVALID_ARG;
  g_give_up_tile.store(tile, std::memory_order_relaxed);
  return MOE_OK;
}

}  // extern "C"
