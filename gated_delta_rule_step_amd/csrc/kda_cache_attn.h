// Attention over the paged 8-bit cache: what its kernels share.
#pragma once

#include "kda_cache.h"

namespace kda {
namespace cache {

struct AttnParams {
  CacheView c;
  int32_t G;            // query heads per key/value head
  const uint16_t* q;
  int64_t q_stride;
  float scale2;         // scale * log2(e)
  uint16_t* out;
  int64_t out_stride;
  float* lse;           // NULL: not wanted
  int64_t lse_stride;
  // the plan
  int32_t row_blocks;   // row blocks of a sequence and key/value head
  int32_t most_rows;    // G * the most tokens of a sequence
  int32_t targets;      // parts that a cache's whole length is cut into, 0: none is cut
  int2* plan;           // [n_seqs]: first slot, parts
  float2* stat;         // [slot][H][row]: reference exponent, sum
  float* part;          // [slot][H][row][128]: sums of p v
};

// Keys are split in units of 128 tokens.
constexpr int kUnit = 128;
constexpr int kMinUnits = 2;  // a part has at least so many
__device__ __forceinline__ int32_t units_of(const CacheView& p, int32_t b) {
  const int32_t len = p.lens[b];
  return len < 0 || len > (int64_t(p.width) << p.page_shift) ? 0 : (len + kUnit - 1) / kUnit;
}

}  // namespace cache
}  // namespace kda
