// Launches of the layer step's operators beside the paged path (include/paged/moe_norm.h, moe_kv4.h).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_launch.h"

namespace moe {

struct AddRmsNormArgs {
  const uint16_t* x;         // [N] rows of H, x_stride apart, or null
  const uint16_t* residual;  // [N, H]
  const uint16_t* weight;    // [H] or null
  uint16_t* residual_out;    // [N, H] or null
  uint16_t* y;               // [N, H] or null
  int8_t* q;                 // [N, H] or null
  float* scales;             // [N, H / 128] or null
  int64_t x_stride;
  float eps;
  int N, H;
};
cudaError_t launch_add_rms_norm(const AddRmsNormArgs& args, int num_sms, cudaStream_t stream);

// The cache held in 4 bits: 16 tokens of a head are a block of keys' codes, keys' scales, values' codes, values' scales.
constexpr int kKv4Tokens = 16;
constexpr int kKv4RowBytes = 64;                                        // a token's codes
constexpr int kKv4Scales = kKv4Tokens * kKv4RowBytes;                   // where its scales begin
constexpr int kKv4Values = kKv4Scales + kKv4Tokens * 8;                 // where the values begin
constexpr int kKv4Block = 2 * kKv4Values;

struct Kv4LoadArgs {
  const uint8_t* cache;
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* dst_table;    // [B, dst_max_pages]
  const int32_t* first;        // [B] or null
  const int32_t* seq_lens;     // [B]
  uint16_t* k_cache;           // [dst_pages, h_kv, page, 128]
  uint16_t* v_cache;
  int32_t* status;
  int B, h_kv, num_pages, dst_pages, max_pages, dst_max_pages, page_shift;
};
cudaError_t launch_kv4_load(const Kv4LoadArgs& args, int num_sms, cudaStream_t stream);

struct Kv4DecodePlan {
  PagedKv paged;
  const uint16_t* q;         // [B, h_q, 128]
  const uint8_t* cache;
  const int32_t* seq_lens;   // [B]
  uint16_t* out;             // [B, h_q, 128]
  float* partials;           // [kPartialCtas][2][kGqaSlotFloats]
  int32_t* counters;         // [kPartialCtas], zero on entry, left zero
  int32_t* status;
  int B, h_q, h_kv, L_cap;
  float scale_log2;
  int num_ctas;
  int give_up_tile;          // failure-detection test: no tile from this one on is loaded (-1: all are)
};
cudaError_t launch_kv4_decode(const Kv4DecodePlan& plan, cudaStream_t stream);

}  // namespace moe
