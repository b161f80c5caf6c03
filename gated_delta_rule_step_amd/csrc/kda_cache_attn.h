// Attention over the paged 8-bit cache: what its kernels share.
//
// Two kernels share the sequences of a call by their rows, G * tokens for each key/value head: few
// rows (one token, or a handful) and documents. Each cuts the keys into parts where its rows alone
// would not fill the chip.
#pragma once

#include <limits.h>

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
  // this kernel's sequences and its plan
  int32_t over, most;   // those with over < rows <= most
  int32_t block_rows;   // rows of a block (of a part's results, too)
  int32_t targets;      // parts that all the blocks' keys are cut into, 0: none is cut
  int32_t min_units;    // units of a part at least
  int4* starts;         // [n_seqs], if listed: first item, cuts before, parts, blocks
  // [0].x: blocks whose keys are cut (y: units of a part, if listed); then their sequence, block,
  // slot, parts
  int4* cuts;
  float2* stat;         // [slot][H][block_rows]: reference exponent, sum of the weights
  float* part;          // [slot][H][block_rows][128]: sums of p v, divided by that sum
};

// Keys are split in units of 128 tokens.
constexpr int kUnit = 128;
__device__ __forceinline__ int32_t units_of(const CacheView& p, int32_t b) {
  const int32_t len = p.lens[b];
  return len < 0 || len > (int64_t(p.width) << p.page_shift) ? 0 : (len + kUnit - 1) / kUnit;
}

__device__ __forceinline__ int32_t rows_of(const AttnParams& p, int32_t b) {
  int32_t n = p.c.per_seq;
  if (p.c.cu) n = max(clamp_row(p.c, p.c.cu[b + 1]) - clamp_row(p.c, p.c.cu[b]), 0);
  // (a call of more rows is refused: only a cu_seqlens that is not the host's copy reaches this)
  return int32_t(min(int64_t(n) * p.G, int64_t(INT_MAX - 255)));
}
// Blocks of a sequence, 0 for another kernel's.
__device__ __forceinline__ int32_t blocks_of(const AttnParams& p, int32_t b) {
  const int32_t rows = rows_of(p, b);
  return rows <= p.over || rows > p.most ? 0 : (rows + p.block_rows - 1) / p.block_rows;
}

// Part `index` of `parts` of the keys of block `rb` of sequence b: tokens from .. to - 1; its
// results go to slot `slot` where there is more than one.
struct Part {
  int32_t b, rb, index, parts, slot, from, to;
  int32_t cut;  // the block among those that are cut, -1: whole
};
struct FindSmem {
  int32_t work[4], items[4];  // a wave's sums
  uint32_t cuts[4];
  int32_t all_cuts;  // blocks that are cut
  Part part;
};
// Up to so many sequences each workgroup finds its work by itself, from kHeld of them a thread;
// more are walked once, by list_sequences, and searched (single tokens, 8 heads, us, walked |
// listed: 300 of 500 keys 68 | 70, 512 of them 111 | 116, 512 of 100 keys 58 | 48, 1024 of 60 keys
// 78 | 56, 4096 of 250 keys 885 | 399, 16384 of 60 keys 11056 | 777).
constexpr int32_t kHeld = 2, kWalked = 512;

// Blocks that are cut << 16 | their slots (both far below 2^16)
__device__ __forceinline__ uint32_t cut_of(int32_t blocks, int32_t parts) {
  return parts > 1 ? uint32_t(blocks) << 16 | uint32_t(blocks * parts) : 0u;
}
// Part of the sequence b, `in` items behind its first one; b = -1 where there is no such part or
// no room for its results: cu_seqlens is not what the host's copy says, so that any of the 32-bit
// sums and counts before this may have wrapped round. What passes is in range, whatever they are.
__device__ __forceinline__ Part part_at(const AttnParams& p, int32_t b, int32_t in, int32_t blocks,
                                        int32_t parts, uint32_t before, int32_t chunk) {
  Part x;
  x.b = in < 0 || in >= int64_t(blocks) * parts ? -1 : b;
  x.parts = parts;
  x.index = parts > 1 ? in / blocks : 0;
  x.rb = blocks - 1 - (in - x.index * blocks);
  const int64_t slot = int64_t(before & 0xffffu) + int64_t(x.rb) * parts + x.index;
  x.slot = int32_t(slot);
  x.from = parts == 1 ? 0 : x.index * chunk * kUnit;
  x.to = x.index + 1 == parts ? INT_MAX : x.from + chunk * kUnit;
  x.cut = parts > 1 ? int32_t(before >> 16) + x.rb : -1;
  if (parts > 1 && (x.cut >= p.targets || slot >= 2 * p.targets)) x.b = -1;
  return x;
}
// Work item `item`: the sequences one after the other, a sequence's parts in turn, the blocks that
// share a part's keys next to each other, the last one (with the most keys to see) first. A
// workgroup of T threads finds it for itself from the lengths on the device, K sequences a thread,
// or (LISTED) from what list_sequences left. SPLIT: the keys may be cut, each sequence's into equal
// parts of a length that is the same for all, however ragged the batch, except for what rounding to
// units leaves. What is cut has less than twice its share of the parts: 2 * targets slots. The blocks
// that are cut are listed for the join, which has workgroups for as many as there may be (with
// workgroups for every row that a sequence may have, 1024 decoded tokens beside a document of 7680
// rows took 1740 us, now 377). (By single waves, 64 sequences at a time, 512 took 10 us to walk.)
template <bool SPLIT, int T, bool LISTED>
__device__ __forceinline__ bool find_part(const AttnParams& p, int32_t item, FindSmem& lds,
                                          Part& out) {
  static_assert(LISTED || kWalked <= kHeld * T, "a thread holds kHeld sequences");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t B = p.c.n_seqs, K = (B + T - 1) / T, b0 = int32_t(threadIdx.x) * K;
  if constexpr (LISTED) {
    int32_t b = 0, span = B;  // the last sequence with a first item <= item is in [b, b + span)
    while (span > 1) {
      const int32_t step = (span + 63) >> 6;
      const bool is = lane * step < span && p.starts[b + lane * step].x <= item;
      b += max(int32_t(__popcll(__ballot(is))) - 1, 0) * step;
      span = min(step, B - b);
    }
    b = __builtin_amdgcn_readfirstlane(b);
    const int4 s = p.starts[b];
    if (s.w == 0) return false;  // behind the last item
    out = part_at(p, b, item - s.x, s.w, s.z, uint32_t(s.y), p.cuts[0].y);
    if (threadIdx.x == 0) {
      lds.part = out;
      lds.all_cuts = p.cuts[0].x;
    }
    out.b = __builtin_amdgcn_readfirstlane(out.b);
    out.rb = __builtin_amdgcn_readfirstlane(out.rb);
    out.index = __builtin_amdgcn_readfirstlane(out.index);
    out.parts = __builtin_amdgcn_readfirstlane(out.parts);
    out.slot = __builtin_amdgcn_readfirstlane(out.slot);
    out.from = __builtin_amdgcn_readfirstlane(out.from);
    out.to = __builtin_amdgcn_readfirstlane(out.to);
    return out.b >= 0;
  }
  const auto sizes = [&](int k, int32_t& blocks, int32_t& units) {
    const bool is = k < K && b0 + k < B;
    blocks = is ? blocks_of(p, b0 + k) : 0;
    units = SPLIT && is ? units_of(p.c, b0 + k) : 0;
  };
  int32_t blocks[kHeld], units[kHeld], chunk = 1 << 28;  // whole sequences
#pragma unroll
  for (int k = 0; k < kHeld; ++k) sizes(k, blocks[k], units[k]);
  if (threadIdx.x == 0) lds.part.b = -1;
  if (SPLIT) {
    int32_t sum = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) sum += blocks[k] * units[k];
    sum = wave_prefix(sum);
    if (lane == 63) lds.work[wave] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) sum += lds.work[w];
    chunk = max(p.min_units, (sum + p.targets - 1) / p.targets);
  }
  const auto parts_of = [&](int32_t u) { return SPLIT ? max((u + chunk - 1) / chunk, 1) : 1; };
  int32_t items = 0;
  uint32_t cuts = 0;
  const auto count = [&](int32_t n, int32_t u) {
    const int32_t parts = parts_of(u);
    items += n * parts;
    cuts += cut_of(n, parts);
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) count(blocks[k], units[k]);
  int32_t first = wave_prefix(items);
  uint32_t before = SPLIT ? uint32_t(wave_prefix(int32_t(cuts))) : 0;
  if (lane == 63) {
    lds.items[wave] = first;
    lds.cuts[wave] = before;
  }
  first -= items;
  before -= cuts;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64 - 1; ++w)
    if (w < wave) {
      first += lds.items[w];
      before += lds.cuts[w];
    }
  if (SPLIT && threadIdx.x == T - 1) lds.all_cuts = int32_t((before + cuts) >> 16);
  if (item >= first && item < first + items) {
    for (int k = 0; k < K; ++k) {
      int32_t n, u;
      sizes(k, n, u);
      const int32_t parts = parts_of(u);
      if (item < first + n * parts) {
        lds.part = part_at(p, b0 + k, item - first, n, parts, before, chunk);
        break;
      }
      first += n * parts;
      before += cut_of(n, parts);
    }
  }
  __syncthreads();
  out.b = __builtin_amdgcn_readfirstlane(lds.part.b);
  if (out.b < 0) return false;
  out.rb = __builtin_amdgcn_readfirstlane(lds.part.rb);
  out.index = __builtin_amdgcn_readfirstlane(lds.part.index);
  out.parts = __builtin_amdgcn_readfirstlane(lds.part.parts);
  out.slot = __builtin_amdgcn_readfirstlane(lds.part.slot);
  out.from = __builtin_amdgcn_readfirstlane(lds.part.from);
  out.to = __builtin_amdgcn_readfirstlane(lds.part.to);
  return true;
}

// Natural logarithm of sum 2^ref; the sum's exponent is added where the reference's is.
__device__ __forceinline__ float log_sum(float ref, float sum) {
  if (sum == 0.0f) return -INFINITY;
  return (ref + float(__builtin_amdgcn_frexp_expf(sum)) +
          __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(sum))) * LN2;
}

// For the join, by the kernel's end (a store in front of its loop has the loop wait for it).
__device__ __forceinline__ void list_cuts(const AttnParams& p, int32_t h, const FindSmem& lds) {
  if (h != 0 || threadIdx.x != 0) return;
  if (blockIdx.x == 0) p.cuts[0].x = min(lds.all_cuts, p.targets);
  const Part& x = lds.part;
  if (x.b >= 0 && x.cut >= 0 && x.index == 0)
    p.cuts[1 + x.cut] = make_int4(x.b, x.rb, x.slot, x.parts);
}

// Documents: workgroups of kDocRows rows.
constexpr int kDocRows = 128;
hipError_t launch_documents(const AttnParams& p, bool int8, unsigned grid, hipStream_t stream);

}  // namespace cache
}  // namespace kda
