// Attention of a few tokens of each sequence over the paged 8-bit cache (gfx950), and the call.
//
// Row r of a sequence and key/value head is query head r mod G of token r / G. With keys
// as the rows of the matrix products (S^T = K Q^T, O^T = V^T P^T), a lane's scores, sums and
// outputs all belong to one query row, so the running maximum and the rescaling need no
// exchange between lanes, and P^T leaves the first product where the second one reads it.
//
// Bound by HBM: every key and value byte passes once. The keys of all sequences are cut into
// parts of about equal length, and a part's four waves walk 32 tokens at a time each.
// The codes are widened to bf16 in registers, exactly; the scales of a page multiply scores
// and weights. The weights p enter the second product as high and low bf16 parts: the
// matrix units idle otherwise, and the output keeps fp32's accuracy.
//
// 128 sequences of 500 to 8190 tokens, 64 query heads on 8: 142 us, 4.6 TB/s of the cache's bytes;
// 512 of 71 to 1500, 12 heads in int8: 158 us, 4.9 TB/s; one of 131070: 60 us, 5 of them the join's.
// 8 tokens of 64 sequences, 64 rows: 79 us, bound by vector instructions (50 % of a SIMD's cycles).

#include <math.h>

#include <algorithm>

#include "kda_cache_attn.h"

namespace kda {
namespace cache {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 32;            // tokens of a wave's step
constexpr int kStride = 4 * kStep;   // and of the workgroup's
constexpr int kRow = D + 4;          // fp32 row in LDS
// Weights stay below 2^kSlack (see `slack`), 2^kLarge times that with the values' scales.
constexpr float kSlack = 8.0f;
// Scales beyond 2^60 bring values whose sums, or products with a weight, may pass fp32's range. From the
// first one on a wave's weights and sums are 2^-64 of what they were, so that sums of 2^28 tokens stay
// below 2^128 whatever the scale; what that flushes to zero is less than 2^-120 of such a value.
constexpr float kLarge = 0x1p60f, kSmaller = 0x1p-64f;

// A wave's 32 tokens are two tiles of 16, each inside one page.
struct Ids {
  int32_t raw[2];  // as the table has them: looked at only where they are used, a step later
};
struct Keys {
  u32x4 w[2][2];  // lane (m, g): token m, channels 64 i + 16 g ..
  float scale[2];
};
struct Values {
  u32x2 w[2][4];  // lane (m, g): token 4 g + r, channels 8 m ..
  float scale[2];
};

__device__ __forceinline__ void load_ids(const AttnParams& p, int32_t b, int32_t at, int32_t end,
                                         Ids& s) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
    s.raw[u] = p.c.table[b * p.c.table_stride +
                         (max(min(at + 16 * u, end - 1), 0) >> p.c.page_shift)];
}
__device__ __forceinline__ int32_t known_page(const AttnParams& p, const Ids& s, int u, int32_t at,
                                              int32_t end) {
  return at + 16 * u < end && uint32_t(s.raw[u]) < uint32_t(p.c.num_pages) ? s.raw[u] : -1;
}
// Page 0's bytes in the place of none's.
__device__ __forceinline__ int64_t tile_at(const CacheView& c, int32_t id, int64_t page, int32_t h,
                                           int32_t tok) {
  return max(id, 0) * page + ((int64_t(h) << c.page_shift) + (tok & ((1 << c.page_shift) - 1))) * D;
}
__device__ __forceinline__ void load_keys(const AttnParams& p, int32_t h, int32_t at, int32_t end,
                                          const Ids& ids, int m, int g, Keys& s) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int32_t id = known_page(p, ids, u, at, end);
    const uint8_t* const k = p.c.k + tile_at(p.c, id, p.c.k_page, h, at + 16 * u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      s.w[u][i] = *reinterpret_cast<const u32x4*>(k + (m * D + i * 64 + g * 16));
    s.scale[u] = p.c.k_scale[int64_t(max(id, 0)) * p.c.H + h];
  }
}
__device__ __forceinline__ void load_values(const AttnParams& p, int32_t h, int32_t at,
                                            int32_t end, const Ids& ids, int m, int g, Values& s) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int32_t id = known_page(p, ids, u, at, end);
    const uint8_t* const v = p.c.v + tile_at(p.c, id, p.c.v_page, h, at + 16 * u);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      s.w[u][r] = *reinterpret_cast<const u32x2*>(v + (4 * g * D + m * 8) + r * D);
    s.scale[u] = p.c.v_scale[int64_t(max(id, 0)) * p.c.H + h];
  }
}

__device__ __forceinline__ float over_groups_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float over_groups_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Values that a row of the block does not see: bytes of tokens that are not there become zeros, and
// so do NaN codes behind `all_see`, which leave the first position that holds one in
// nan_at[channel]: rows that see it become NaN in the end, and the others stay clear of 0 NaN.
template <int KIND>
__device__ __forceinline__ void clear_values(Values& v, const int32_t (&live)[2], int32_t at,
                                             int32_t all_see, int m, int g, int32_t* nan_at) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int in = 4 * g + r;
      if (in >= live[u]) v.w[u][r] = u32x2{0u, 0u};
      if (KIND == kFp8 && at + 16 * u + in > all_see) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t hit = nan_codes(v.w[u][r][j]);
          if (hit) v.w[u][r][j] &= ~note_nans(hit, nan_at + m * 8 + 4 * j, at + 16 * u + in);
        }
      }
    }
}

// One workgroup: (part of a sequence's keys, key/value head) for up to 16 NT rows.
template <int KIND, int NT, bool LISTED>
__global__ __launch_bounds__(kThreads, NT == 1 ? 4 : 3) void attend_kernel(AttnParams p) {
  __shared__ float sums[4][16 * kRow];
  __shared__ float refs[4][16], tots[4][16], units[4];
  __shared__ int32_t nan_at[D];
  __shared__ FindSmem find;
  constexpr bool kInLds = NT > 1;
  __shared__ bf16x8 queries[kInLds ? NT * 4 * 64 : 1];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = blockIdx.x / p.c.H, h = blockIdx.x - item * p.c.H;
  Part part;
  if (!find_part<true, kThreads, LISTED>(p, item, find, part)) return;
  const Seq seq = sequence(p.c, part.b);
  const int rows = rows_of(p, part.b), row0 = part.rb * 16 * NT;
  const int32_t len = p.c.num_pages > 0 ? max(seq.len, 0) : 0;
  const int32_t to = min(part.to, len);
  const int32_t base = len - seq.n;              // position of the first token
  const int32_t all_see = base + row0 / p.G;     // every row sees up to here

  int32_t at = part.from + wave * kStep;
  Ids ids, ids_next;
  Keys k;
  Values v;
  if (at < to) {
    load_ids(p, part.b, at, to, ids);
    load_ids(p, part.b, at + kStride, to, ids_next);
    load_keys(p, h, at, to, ids, m, g, k);
    load_values(p, h, at, to, ids, m, g, v);
  }
  if (threadIdx.x < D) nan_at[threadIdx.x] = INT_MAX;

  // queries: lane (m, g) holds row m's channels of group g, eight per product
  bf16x8 q[4];
  int32_t last[NT];  // the last position that the lane's row sees
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 16 * n + m, t = r / p.G;
    last[n] = base + t;
    if (kInLds && n != wave) continue;
    const uint16_t* const src =
        p.q + (seq.first + t) * p.q_stride + (int64_t(h) * p.G + (r - t * p.G)) * D;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (r < rows)
        w = *reinterpret_cast<const u32x4_u*>(src + (j >> 1) * 64 + g * 16 + (j & 1) * 8);
      q[j] = __builtin_bit_cast(bf16x8, w);
      if (kInLds) queries[(n * 4 + j) * 64 + lane] = q[j];
    }
  }
  __syncthreads();

  f32x4 o[NT][8];
  bool smaller = false;  // see kLarge
  // A row's reference exponent moves when a score passes it by more than `slack`: by anything at
  // first.
  float ref[NT], slack[NT], tot[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    ref[n] = 0.0f;
    slack[n] = -INFINITY;
    tot[n] = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[n][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  for (; at < to; at += kStride) {
    const bool more = at + kStride < to;
    int32_t live[2];  // tokens that exist
#pragma unroll
    for (int u = 0; u < 2; ++u)
      live[u] = known_page(p, ids, u, at, to) < 0 ? 0 : min(16, to - (at + 16 * u));
    const bool masked = live[0] < 16 || live[1] < 16 || at + kStep - 1 > all_see;
    f32x4 acc[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) acc[n][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      whole(k.w[u][0]);
      whole(k.w[u][1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 a = widen8<KIND>(k.w[u][j >> 1][2 * (j & 1)], k.w[u][j >> 1][2 * (j & 1) + 1]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[n][u] = mfma32(a, kInLds ? queries[(n * 4 + j) * 64 + lane] : q[j], acc[n][u]);
      }
    const float f[2] = {p.scale2 * k.scale[0], p.scale2 * k.scale[1]};
    if (more) load_keys(p, h, at + kStride, to, ids_next, m, g, k);
    // (whatever the scale of a page that does not exist is)
    float vs[2] = {live[0] > 0 ? v.scale[0] : 0.0f, live[1] > 0 ? v.scale[1] : 0.0f};
    if (smaller || __any(fmaxf(fabsf(vs[0]), fabsf(vs[1])) > kLarge)) {
      const float down = smaller ? 1.0f : kSmaller;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 8; ++c) o[n][c] *= down;
      vs[0] *= kSmaller;
      vs[1] *= kSmaller;
      smaller = true;
    }
    bf16x8 ph[NT], pl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float s[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[u][r] = fmaf(acc[n][u][r], f[u], -ref[n]);
      if (masked) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int in = 4 * g + r;
            if (in >= live[u] || at + 16 * u + in > last[n]) s[u][r] = -INFINITY;
          }
      }
      const float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                              fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      if (__any(top > slack[n])) {
        const float over = over_groups_max(top);
        if (over > slack[n]) {
          const float down = slack[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(-over);
          ref[n] += over;
          slack[n] = kSlack;
          tot[n] *= down;
#pragma unroll
          for (int c = 0; c < 8; ++c) o[n][c] *= down;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[u][r] -= over;
        }
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[r] = __builtin_amdgcn_exp2f(s[u][r]);
          tot[n] += w[r];
          w[r] *= vs[u];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t x = pack_bf16x2(w[2 * r], w[2 * r + 1]);
          hi[2 * u + r] = x;
          lo[2 * u + r] = pack_bf16x2(w[2 * r] - bf_lo(x), w[2 * r + 1] - bf_hi(x));
        }
      }
      ph[n] = __builtin_bit_cast(bf16x8, u32x4{hi[0], hi[1], hi[2], hi[3]});
      pl[n] = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], lo[2], lo[3]});
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) whole(v.w[u][r]);
    if (masked) clear_values<KIND>(v, live, at, all_see, m, g, nan_at);
#pragma unroll
    for (int c4 = 0; c4 < 2; ++c4) {  // channels 8 m + 4 c4 ..
      uint32_t t0[4], t1[4];
      transpose4(v.w[0][0][c4], v.w[0][1][c4], v.w[0][2][c4], v.w[0][3][c4], t0);
      transpose4(v.w[1][0][c4], v.w[1][1][c4], v.w[1][2][c4], v.w[1][3][c4], t1);
      if constexpr (NT == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bf16x8 a = widen8<KIND>(t0[c], t1[c]);
          o[0][4 * c4 + c] = mfma32(a, ph[0], o[0][4 * c4 + c]);
          o[0][4 * c4 + c] = mfma32(a, pl[0], o[0][4 * c4 + c]);
        }
      } else {  // (a sum's two products apart: 95 -> 92 us; with one row block it costs registers)
        bf16x8 a[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) a[c] = widen8<KIND>(t0[c], t1[c]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[n][4 * c4 + c] = mfma32(a[c], ph[n], o[n][4 * c4 + c]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[n][4 * c4 + c] = mfma32(a[c], pl[n], o[n][4 * c4 + c]);
      }
    }
    if (more) load_values(p, h, at + kStride, to, ids_next, m, g, v);
    ids = ids_next;
    load_ids(p, part.b, at + 2 * kStride, to, ids_next);
  }

  list_cuts(p, h, find);
  if (lane == 0) units[wave] = smaller ? kSmaller : 1.0f;
  // the four waves' sums, 16 rows at a time; thread (row, 8 channels)
  const int row = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float total = over_groups_sum(tot[n]);
    if (n > 0) __syncthreads();
    if (g == 0) {
      refs[wave][m] = slack[n] == -INFINITY ? -INFINITY : ref[n];
      tots[wave][m] = total;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* const to_lds = &sums[wave][m * kRow + (4 * g + r) * 8];
      *reinterpret_cast<f32x4*>(to_lds) = f32x4{o[n][0][r], o[n][1][r], o[n][2][r], o[n][3][r]};
      *reinterpret_cast<f32x4*>(to_lds + 4) = f32x4{o[n][4][r], o[n][5][r], o[n][6][r], o[n][7][r]};
    }
    __syncthreads();
    const int r = row0 + 16 * n + row;
    if (r >= rows || r - row0 >= p.block_rows) continue;
    const int t = r / p.G;
    const float top = fmaxf(fmaxf(refs[0][row], refs[1][row]), fmaxf(refs[2][row], refs[3][row]));
    const float r0 = top == -INFINITY ? 0.0f : top;
    const float unit = fminf(fminf(units[0], units[1]), fminf(units[2], units[3]));
    float sum = 0.0f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float f = __builtin_amdgcn_exp2f(refs[w][row] - r0);
      sum += tots[w][row] * f;
      if (units[w] != unit) f *= unit;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += sums[w][row * kRow + ch + c] * f;
    }
    if (KIND == kFp8) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (nan_at[ch + c] <= base + t) acc[c] = NAN;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = acc[c] * inv;
    if (unit != 1.0f) {
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] *= 1.0f / kSmaller;
    }
    if (part.parts == 1) {
      const int64_t head = int64_t(h) * p.G + (r - t * p.G);
      *reinterpret_cast<u32x4_u*>(p.out + (seq.first + t) * p.out_stride + head * D + ch) =
          u32x4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])};
      if (p.lse && ch == 0) p.lse[(seq.first + t) * p.lse_stride + head] = log_sum(r0, sum);
    } else {
      const int64_t slot = (int64_t(part.slot) * p.c.H + h) * p.block_rows + (r - row0);
      float* const dst = p.part + slot * D + ch;
      *reinterpret_cast<f32x4*>(dst) = f32x4{acc[0], acc[1], acc[2], acc[3]};
      *reinterpret_cast<f32x4*>(dst + 4) = f32x4{acc[4], acc[5], acc[6], acc[7]};
      if (ch == 0) p.stat[slot] = make_float2(top, sum);
    }
  }
}

// Joins the parts of the blocks that are cut, a row by 16 lanes of 8 channels, four parts at a time:
// an average, so that no value is beyond the largest of them.
// WIDE: a workgroup's 16 groups share one row's parts (few rows, many parts), else each has a row
// of its own.
template <bool WIDE>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnParams p) {
  __shared__ float accs[WIDE ? 16 : 1][D];
  __shared__ float2 stats[WIDE ? 16 : 1];
  const int group = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;
  const int pairs = p.block_rows * p.c.H, per = WIDE ? pairs : (pairs + 15) / 16;
  const int n = blockIdx.x / per;
  const int4 cut = p.cuts[1 + n];
  if (n >= p.cuts[0].x) return;
  const int b = cut.x;
  // (an entry that this call did not write: cu_seqlens is not what the host's copy says)
  if (uint32_t(b) >= uint32_t(p.c.n_seqs) || uint32_t(cut.y) >= uint32_t(blocks_of(p, b)) ||
      cut.z < 0 || cut.w < 2 || int64_t(cut.z) + cut.w > 2 * p.targets)
    return;
  const int i = WIDE ? blockIdx.x - n * per : (blockIdx.x - n * per) * 16 + group;
  const int h = i / p.block_rows, in = i - h * p.block_rows, r = cut.y * p.block_rows + in;
  const bool mine = i < pairs && r < rows_of(p, b);
  if (WIDE ? !mine : __ballot(mine) == 0) return;
  const int64_t first = (int64_t(cut.z) * p.c.H + h) * p.block_rows + in;
  const int64_t step = int64_t(p.c.H) * p.block_rows;
  const int parts = mine ? cut.w : 0, stride = WIDE ? 16 : 1;
  float top = -INFINITY, sum = 0.0f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s0 = WIDE ? group : 0; s0 < parts; s0 += 4 * stride) {
    float2 st[4];
    f32x4 x[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = s0 + j * stride;
      st[j] = make_float2(-INFINITY, 0.0f);
      x[j][0] = x[j][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (s < parts) {
        const int64_t at = first + s * step;
        st[j] = p.stat[at];
        x[j][0] = *reinterpret_cast<const f32x4*>(p.part + at * D + ch);
        x[j][1] = *reinterpret_cast<const f32x4*>(p.part + at * D + ch + 4);
      }
    }
    const float now = fmaxf(fmaxf(fmaxf(st[0].x, st[1].x), fmaxf(st[2].x, st[3].x)), top);
    const float r0 = now == -INFINITY ? 0.0f : now;
    float f = sum * __builtin_amdgcn_exp2f(top - r0), all = f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      st[j].y *= __builtin_amdgcn_exp2f(st[j].x - r0);
      all += st[j].y;
    }
    top = now;
    sum = all;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    f *= inv;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f = st[j].y * inv;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += x[j][c >> 2][c & 3] * f;
    }
  }
  if (WIDE) {
#pragma unroll
    for (int c = 0; c < 8; ++c) accs[group][ch + c] = acc[c];
    if (ch == 0) stats[group] = make_float2(top, sum);
    __syncthreads();
    if (group > 0) return;
    top = stats[0].x;
#pragma unroll
    for (int w = 1; w < 16; ++w) top = fmaxf(top, stats[w].x);
    const float r0 = top == -INFINITY ? 0.0f : top;
    sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = 0.0f;
    for (int w = 0; w < 16; ++w) sum += stats[w].y * __builtin_amdgcn_exp2f(stats[w].x - r0);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int w = 0; w < 16; ++w) {
      const float f = stats[w].y * __builtin_amdgcn_exp2f(stats[w].x - r0) * inv;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += accs[w][ch + c] * f;
    }
  }
  if (!mine) return;
  const Seq seq = sequence(p.c, b);
  const int t = r / p.G;
  const int64_t head = int64_t(h) * p.G + (r - t * p.G);
  *reinterpret_cast<u32x4_u*>(p.out + (seq.first + t) * p.out_stride + head * D + ch) =
      u32x4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
            pack_bf16x2(acc[6], acc[7])};
  if (p.lse && ch == 0)
    p.lse[(seq.first + t) * p.lse_stride + head] = log_sum(top == -INFINITY ? 0.0f : top, sum);
}

// What find_part finds by walking all sequences, for its searches: by one workgroup.
constexpr int kListThreads = 1024;
__global__ __launch_bounds__(kListThreads) void list_sequences(AttnParams p) {
  constexpr int T = kListThreads;
  __shared__ int32_t work[T / 64], all_items[T / 64];
  __shared__ uint32_t all_cuts[T / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t K = (p.c.n_seqs + T - 1) / T, b0 = int32_t(threadIdx.x) * K;
  const int32_t b1 = min(b0 + K, p.c.n_seqs);
  int32_t chunk = 1 << 28;  // whole sequences
  if (p.targets > 0) {
    int32_t sum = 0;
    for (int32_t b = b0; b < b1; ++b) sum += blocks_of(p, b) * units_of(p.c, b);
    sum = wave_prefix(sum);
    if (lane == 63) work[wave] = sum;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < T / 64; ++w) sum += work[w];
    chunk = max(p.min_units, (sum + p.targets - 1) / p.targets);
  }
  const auto parts_of = [&](int32_t b) { return max((units_of(p.c, b) + chunk - 1) / chunk, 1); };
  int32_t items = 0;
  uint32_t cuts = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = blocks_of(p, b), parts = parts_of(b);
    items += n * parts;
    cuts += cut_of(n, parts);
  }
  int32_t first = wave_prefix(items);
  uint32_t before = uint32_t(wave_prefix(int32_t(cuts)));
  if (lane == 63) {
    all_items[wave] = first;
    all_cuts[wave] = before;
  }
  first -= items;
  before -= cuts;
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    first += all_items[w];
    before += all_cuts[w];
  }
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = blocks_of(p, b), parts = parts_of(b);
    p.starts[b] = make_int4(first, int32_t(before), parts, n);
    first += n * parts;
    before += cut_of(n, parts);
  }
  if (threadIdx.x == T - 1)
    p.cuts[0] = make_int4(min(int32_t(before >> 16), p.targets), chunk, 0, 0);
}

// Host: the two kernels' shares of a call.
struct Share {
  int32_t over, most;  // its sequences have over < rows <= most
  int32_t block_rows;
  int32_t groups;      // workgroups that the cut aims at
  int32_t min_units;   // of a part
};
constexpr int kFew = 0, kDocuments = 1;
// Up to 128 rows stay with blocks of 32 in registers, whose keys the second to fourth block find in
// the L2 (64 sequences of up to 4000 tokens, 8 heads, as few rows | as documents, us: 72 rows 113 |
// 196, 128 rows 143 | 200; 8 sequences: 128 rows 31 | 35, 160 rows 38 | 39; one of 30000: 54 | 52).
// The cut's sizes matter little: 512 to 4096 workgroups, 4 or 8 units are within 5 %.
constexpr Share kShares[] = {{0, 128, 32, 1024, 8}, {128, INT_MAX, kDocRows, 512, 4}};

struct Plan {
  int32_t block_rows, targets;
  int64_t starts_bytes, cuts_bytes, stat_bytes, bytes, grid;
  int64_t join_blocks;  // blocks that may be cut
};
// `rows`: the most of a sequence; `blocks`: in all.
Plan make_plan(int kind, int32_t n_seqs, int64_t rows, int64_t blocks, int32_t H) {
  const Share& s = kShares[kind];
  Plan r = {};
  r.block_rows = kind == kFew ? int32_t(std::min<int64_t>(rows, s.block_rows)) : s.block_rows;
  const int64_t targets = std::max<int64_t>(1, s.groups / H);
  if (n_seqs > kWalked) {
    r.starts_bytes = (int64_t(n_seqs) * 16 + 255) / 256 * 256;
    r.cuts_bytes = 256;
  }
  // few rows are cut however many sequences there are, since those may differ in length
  if (kind == kFew || blocks < targets) {
    r.targets = int32_t(targets);
    r.join_blocks = std::min(blocks, targets);
    const int64_t vecs = 2 * targets * H * r.block_rows;
    r.cuts_bytes = ((targets + 1) * 16 + 255) / 256 * 256;
    r.stat_bytes = (vecs * 8 + 255) / 256 * 256;
    r.bytes = r.stat_bytes + vecs * D * 4;
  }
  r.bytes += r.starts_bytes + r.cuts_bytes;
  r.grid = (r.targets + blocks) * H;
  return r;
}

template <int KIND, bool LISTED>
hipError_t launch_attend(const AttnParams& p, unsigned grid, hipStream_t stream) {
  if (p.block_rows <= 16)
    hipLaunchKernelGGL((attend_kernel<KIND, 1, LISTED>), dim3(grid), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((attend_kernel<KIND, 2, LISTED>), dim3(grid), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}
hipError_t launch_few(const AttnParams& p, bool int8, unsigned grid, hipStream_t stream) {
  if (p.starts)
    return int8 ? launch_attend<kInt8, true>(p, grid, stream)
                : launch_attend<kFp8, true>(p, grid, stream);
  return int8 ? launch_attend<kInt8, false>(p, grid, stream)
              : launch_attend<kFp8, false>(p, grid, stream);
}

hipError_t launch_join(const AttnParams& p, int64_t blocks, hipStream_t stream) {
  const int64_t pairs = int64_t(p.block_rows) * p.c.H;
  if (blocks * pairs <= 1024)
    hipLaunchKernelGGL(join_kernel<true>, dim3(unsigned(blocks * pairs)), dim3(kThreads), 0, stream,
                       p);
  else
    hipLaunchKernelGGL(join_kernel<false>, dim3(unsigned(blocks * ((pairs + 15) / 16))),
                       dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

bool bad_heads(int32_t H_q, int32_t H_kv) {
  return H_q < 1 || H_kv < 1 || H_q % H_kv != 0;
}

}  // namespace
}  // namespace cache
}  // namespace kda

extern "C" size_t kda_cache_attention_workspace_size(int32_t n_seqs, int64_t total_tokens,
                                                     int32_t H_q, int32_t H_kv) {
  namespace kc = kda::cache;
  if (n_seqs < 1 || total_tokens < 1 || total_tokens > (int64_t(1) << 30) ||
      kc::bad_heads(H_q, H_kv) || H_q / H_kv > 256 || H_kv > kc::kMaxHeads)
    return 0;
  // whatever the sequences' shares of the tokens
  const int64_t rows = total_tokens * (H_q / H_kv);
  int64_t bytes = 0;
  for (int i = 0; i < 2; ++i)
    if (rows > kc::kShares[i].over)
      bytes += kc::make_plan(i, n_seqs, std::min<int64_t>(rows, kc::kShares[i].most), 0, H_kv).bytes;
  return size_t(bytes);
}

extern "C" kda_status kda_cache_attention(
    int32_t n_seqs, int64_t total_tokens, int32_t H_q, int32_t H_kv, int32_t D,
    const int32_t* cu_seqlens_host, const int32_t* cu_seqlens, const void* q, int64_t q_row_stride,
    int32_t cache_dtype, int32_t page_size, int64_t num_pages, const void* k_cache,
    int64_t k_page_stride, const void* v_cache, int64_t v_page_stride, const float* k_scale,
    const float* v_scale, const int32_t* page_table, int32_t table_width, int64_t table_row_stride,
    const int32_t* kv_lens, float scale, void* out, int64_t out_row_stride, float* lse,
    int64_t lse_row_stride, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  namespace kc = kda::cache;
  if (kc::bad_heads(H_q, H_kv)) return KDA_ERR_BAD_SHAPE;
  kc::AttnParams p;
  const kc::CacheArgs a = {n_seqs,  total_tokens, H_kv, D, cu_seqlens, cache_dtype, page_size,
                           num_pages, k_cache, k_page_stride, v_cache, v_page_stride, k_scale,
                           v_scale, page_table, table_width, table_row_stride, kv_lens};
  if (const kda_status st = kc::check(a, &p.c)) return st;
  if (H_q / H_kv > 256 || !isfinite(scale * kda::LOG2E)) return KDA_ERR_UNSUPPORTED;
  const int64_t row = int64_t(H_q) * D;
  if (q_row_stride < 0 || out_row_stride < 0 || (lse && lse_row_stride < 0) ||
      !kc::rows_apart(total_tokens, out_row_stride, row) ||
      (lse && !kc::rows_apart(total_tokens, lse_row_stride, H_q)))
    return KDA_ERR_BAD_STRIDE;
  if (total_tokens == 0) return KDA_OK;
  if (!q || !out) return KDA_ERR_NULL_POINTER;
  if ((cu_seqlens != nullptr) != (cu_seqlens_host != nullptr)) return KDA_ERR_NULL_POINTER;
  p.G = H_q / H_kv;
  int64_t most[2] = {}, blocks[2] = {};
  const auto note = [&](int64_t n, int64_t times) {
    const int64_t rows = n * p.G;
    for (int i = 0; i < 2; ++i)
      if (rows > kc::kShares[i].over && (rows <= kc::kShares[i].most || i == kc::kDocuments)) {
        most[i] = std::max(most[i], rows);
        blocks[i] += (rows + kc::kShares[i].block_rows - 1) / kc::kShares[i].block_rows * times;
      }
  };
  if (cu_seqlens_host) {
    if (cu_seqlens_host[0] != 0 || cu_seqlens_host[n_seqs] > total_tokens)
      return KDA_ERR_BAD_SEQLENS;
    for (int32_t b = 0; b < n_seqs; ++b) {
      const int64_t n = int64_t(cu_seqlens_host[b + 1]) - cu_seqlens_host[b];
      if (n < 0) return KDA_ERR_BAD_SEQLENS;
      note(n, 1);
    }
  } else {
    note(p.c.per_seq, n_seqs);
  }
  kc::Plan plan[2];
  int64_t bytes = 0;
  for (int i = 0; i < 2; ++i) {
    plan[i] = {};
    if (blocks[i] == 0) continue;
    plan[i] = kc::make_plan(i, n_seqs, most[i], blocks[i], H_kv);
    bytes += plan[i].bytes;
    if (most[i] > INT32_MAX - 128 || plan[i].grid > kc::kMaxGrid) return KDA_ERR_UNSUPPORTED;
  }
  if (bytes > 0) {
    if (workspace_bytes < size_t(bytes)) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace) return KDA_ERR_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_UNSUPPORTED;
  }
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_row_stride;
  p.scale2 = scale * kda::LOG2E;
  p.out = static_cast<uint16_t*>(out);
  p.out_stride = out_row_stride;
  p.lse = lse;
  p.lse_stride = lse_row_stride;
  const bool int8 = cache_dtype == KDA_CACHE_INT8;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  for (int i = 0; i < 2; ++i) {
    if (blocks[i] == 0) continue;
    const kc::Share& s = kc::kShares[i];
    p.over = s.over;
    p.most = s.most;
    p.block_rows = plan[i].block_rows;
    p.targets = plan[i].targets;
    p.min_units = s.min_units;
    p.starts = plan[i].starts_bytes > 0 ? reinterpret_cast<int4*>(ws) : nullptr;
    p.cuts = reinterpret_cast<int4*>(ws + plan[i].starts_bytes);
    uint8_t* const results = ws + plan[i].starts_bytes + plan[i].cuts_bytes;
    p.stat = reinterpret_cast<float2*>(results);
    p.part = reinterpret_cast<float*>(results + plan[i].stat_bytes);
    ws += plan[i].bytes;
    const unsigned grid = unsigned(plan[i].grid);
    if (p.starts) {
      hipLaunchKernelGGL(kc::list_sequences, dim3(1), dim3(kc::kListThreads), 0, stream, p);
      if (hipGetLastError() != hipSuccess) return KDA_ERR_LAUNCH;
    }
    if ((i == kc::kDocuments ? kc::launch_documents(p, int8, grid, stream)
                             : kc::launch_few(p, int8, grid, stream)) != hipSuccess)
      return KDA_ERR_LAUNCH;
    // nothing is cut where the table is too short for two parts
    if (plan[i].targets > 0 && int64_t(table_width) * page_size > s.min_units * kc::kUnit &&
        kc::launch_join(p, plan[i].join_blocks, stream) != hipSuccess)
      return KDA_ERR_LAUNCH;
  }
  return KDA_OK;
}
