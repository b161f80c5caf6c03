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
  int32_t few_rows;     // sequences of at most so many rows (G * tokens) have few, the others are
                        // documents
  int32_t most_rows;    // of a sequence of the kernel's kind
  int32_t row_blocks;   // few rows: row blocks of a sequence and key/value head
  int32_t targets;      // parts that all the keys are cut into
  int2* plan;           // [n_seqs]: first slot, parts
  float2* stat;         // [slot][H][row]: reference exponent, sum
  float* part;          // [slot][H][row][128]: sums of p v
};

__device__ __forceinline__ int32_t rows_of(const AttnParams& p, int32_t b) {
  int32_t n = p.c.per_seq;
  if (p.c.cu) n = max(clamp_row(p.c, p.c.cu[b + 1]) - clamp_row(p.c, p.c.cu[b]), 0);
  const int64_t rows = int64_t(n) * p.G;
  return int32_t(min(rows, int64_t(INT32_MAX)));
}
__device__ __forceinline__ bool is_few(const AttnParams& p, int32_t b) {
  const int32_t rows = rows_of(p, b);
  return rows > 0 && rows <= min(p.few_rows, p.most_rows);
}

// Keys are split in units of 128 tokens.
constexpr int kUnit = 128;
constexpr int kMinUnits = 2;  // a part has at least so many
__device__ __forceinline__ int32_t units_of(const CacheView& p, int32_t b) {
  const int32_t len = p.lens[b];
  return len < 0 || len > (int64_t(p.width) << p.page_shift) ? 0 : (len + kUnit - 1) / kUnit;
}

// Rows of a documents' workgroup, and the launch of `grid` of them.
constexpr int kDocRows = 128;
hipError_t launch_documents(const AttnParams& p, bool int8, unsigned grid, hipStream_t stream);

}  // namespace cache
}  // namespace kda
