// What a query sees of a paged cache, as key tiles, and the layout of row-block partials: shared by the decode and
// the row-block attention kernels.
#pragma once

#include <cstdint>

#include "moe_launch.h"

namespace moe {
namespace gqa {

constexpr int kKeys = 128;  // keys per tile

// A K or V tile of a paged cache in shared memory: groups of 8 keys, in each the lower 64 dimensions of its keys (a
// 1024-byte swizzle atom of 8 x 128 bytes), then the upper 64. One copy then brings a whole page: a copy costs its warp
// some 70 cycles, and with one for each half a tile of 16-token pages took 32, more than its share of the memory's time.
// Decode over 16 sequences of up to 32K keys, us by layout (halves apart, together): 173, 159 with pages of 16 tokens;
// 159, 157 of 32; 157, 157 of 64; 158, 158 of 128.
constexpr int kGroupBytes = 2048;  // 8 keys
constexpr int kUpper = 1024;       // the upper dimensions within a group
__device__ __forceinline__ uint32_t tile_row(int key) { return (key >> 3) * kGroupBytes + (key & 7) * 128; }
// The cache as {64 dimensions, 8 keys, 2 halves, groups of a page, pages x heads}; a copy moves box_rows keys.
inline bool encode_paged(CUtensorMap* map, const uint16_t* base, int num_pages, int h_kv, int page, int box_rows) {
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(page / 8), static_cast<cuuint64_t>(num_pages) * h_kv};
  const cuuint64_t strides[4] = {256, 128, 2048, static_cast<cuuint64_t>(page) * 256};
  const cuuint32_t box[5] = {64, 8, 2, static_cast<cuuint32_t>(box_rows / 8), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  TensorMapEncodeFn enc = tensor_map_encoder();
  return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint16_t*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The visible keys of a run of queries: the window [lo, len) and the sink keys [0, sk), sk <= lo. Its tiles are
// the sink's (those before the window's first, w0), then the window's.
struct Span {
  int len, lo, sk, w0, ns, nt;
  __device__ __forceinline__ int key_tile(int t) const { return t < ns ? t : w0 + t - ns; }
  __device__ __forceinline__ bool sees(int key) const { return key < len && (key >= lo || key < sk); }
  __device__ __forceinline__ bool sees_any(int key, int n) const { return key < len && (key + n > lo || key < sk); }
};
// Keys below `len` (0: none), from `lo` on or below n_sink.
__device__ __forceinline__ Span span_of_range(int len, int lo, int n_sink) {
  Span s;
  s.len = len;
  s.lo = lo;
  s.sk = min(n_sink, lo);
  s.w0 = lo / kKeys;
  s.ns = min((s.sk + kKeys - 1) / kKeys, s.w0);
  s.nt = len == 0 ? 0 : s.ns + (len + kKeys - 1) / kKeys - s.w0;
  return s;
}
// The first key of the window of a query at position pos.
__device__ __forceinline__ int window_start(int pos, int window) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}
// One query at the end of a sequence of len keys; a length outside [0, L_cap] counts as empty. When the rows of the
// window's first tile that lie before the window have room for the sink keys (in runs of kFold rows), those are
// folded into them and need no tile of their own.
constexpr int kFold = 16;
struct DecodeSpan : Span {
  int fold;  // rows of the first tile that hold keys 0 .. fold - 1 instead
  __device__ __forceinline__ int key_of(int t, int row) const { return t == 0 && row < fold ? row : key_tile(t) * kKeys + row; }
};
__device__ __forceinline__ DecodeSpan span_of(int len, int L_cap, const PagedKv& kv) {
  if (len < 0 || len > L_cap) len = 0;
  DecodeSpan s;
  static_cast<Span&>(s) = span_of_range(len, window_start(len - 1, kv.window), kv.n_sink);
  const int before = s.lo - s.w0 * kKeys;
  s.fold = 0;
  if (s.ns > 0 && s.sk <= kKeys && (s.sk + kFold - 1) / kFold <= before / kFold) {
    s.fold = (s.sk + kFold - 1) / kFold * kFold;
    s.nt -= s.ns;
    s.ns = 0;
  }
  return s;
}

// Row-block partials: per piece the unnormalised output as [16 groups of 8 dimensions][kRowTile rows][8], so that the
// writer (a thread per row) and the readers (a thread per dimension) both move whole 32-byte sectors.
__device__ __forceinline__ int64_t piece_at(int64_t piece, int row, int dim) {
  return ((piece * 16 + (dim >> 3)) * kRowTile + row) * 8 + (dim & 7);
}

}  // namespace gqa
}  // namespace moe
