// A smaller latent cache: parameters and launchers of the decode over 4-bit rows, the keys' attention weights, the
// choice of the rows that stay and their move to the front of their request.
#pragma once
#include "mla_internal.h"

namespace mla {

// a 4-bit cache row: [codes of 512 latent columns | 32 scales | 64 RoPE columns in bf16]
constexpr int kFp4Codes = kLatent / 2;                     // bytes
constexpr int kFp4Scales = kLatent / 16;
constexpr int kFp4Pe = kFp4Codes + kFp4Scales;             // offset of the RoPE columns
constexpr int kFp4Row = kFp4Pe + 2 * kRope;                // 416

// device range codes (below DEV_RANGE_BASE)
enum : uint32_t { Y_PAGE = 0x7A, Y_LEN = 0x7B, Y_SELECT = 0x7C, Y_COMPACT = 0x7D };

// the rows of a request's keys, through its block table
struct PagedRows {
  const uint8_t* cache;          // [num_pages * page_size] rows
  const int32_t* block_table;    // [B, max_pages]
  const int32_t* lens;           // [B] (null where the call has none)
  int64_t num_pages;
  int max_pages, page_size, B;
  int row_bytes;
};

enum CacheFormat : int { kCacheBf16 = 0, kCacheE4m3 = 1, kCacheFp4 = 2 };

struct DecodeFp4Params {
  PagedRows kv;
  const __nv_bfloat16* q;        // [B, s, H, 576]
  const float* sinks;            // [H] or null
  __nv_bfloat16* out;            // [B, s, H, 512]
  float* lse;                    // [B, s, H] or null
  uint32_t* err;
  float scale;                   // scale * kv_scale
  float kv_scale;
  uint32_t spin_limit, debug_stall;
  int s, H;
  int row_tiles;                 // groups of up to 128 query rows a request has
  int part_rows;                 // rows of a partial
  int groups;
  int64_t* before;               // ws: [groups + 1] tiles before each group
  float* part_stat;              // ws: [groups + pairs, part_rows][8]: maximum, four sums
  float* part_o;                 // ws: [groups + pairs, part_rows, 512]
  uint64_t part_stat_bytes, part_o_bytes;
};
struct DecodeFp4Scratch {
  int pairs, row_tiles, part_rows, groups;
  size_t before, part_stat, part_o;     // bytes
};
DecodeFp4Scratch decode_fp4_scratch(int B, int s, int H, int num_splits);
cudaError_t launch_decode_fp4(const DecodeFp4Params& p, int pairs, cudaStream_t stream);

struct KeyWeightsParams {
  PagedRows kv;
  const __nv_bfloat16* q;        // [B, s, H, 576]
  const float* lse;              // [B, s, H]
  float* weights;                // [B, width] rows at stride
  int64_t stride;
  uint32_t* err;
  float scale;                   // scale * kv_scale
  float decay;
  uint32_t spin_limit, debug_stall;
  int format;                    // a CacheFormat
  int s, H, width;
  int32_t* before;               // ws, with more than 128 query rows: [B + 1][2] tiles and ranges before each request
  float* part;                   // ws: sums of ranges of tiles
  uint64_t part_bytes;
};
// bytes of `part`, and of `before`
size_t key_weights_scratch(int B, int64_t rows, int64_t width, size_t* before);
cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream);

struct SelectParams {
  const float* weights;          // [B, width] rows at stride
  const int32_t* lens;           // [B]
  const int32_t* keep;           // [B]
  int32_t* idx;                  // [B, K]
  int32_t* count;                // [B]
  int32_t* dropped;              // [B]
  uint32_t* err;
  int64_t stride;
  int width, first, recent, B, K;
};
cudaError_t launch_select_keys(const SelectParams& p, cudaStream_t stream);

struct CompactParams {
  PagedRows kv;                  // lens null
  const int32_t* idx;            // [B, K]
  const int32_t* count;          // [B]
  float* weights;                // [B, width] rows at stride, or null
  uint32_t* err;
  uint32_t spin_limit, debug_stall;
  int64_t stride;
  int K, width;
};
cudaError_t launch_compact_rows(const CompactParams& p, cudaStream_t stream);

}  // namespace mla
