// Attention of a few tokens of each sequence over the paged 8-bit cache (gfx950).
//
// Row r of a sequence and key/value head is query head r mod G of token r / G. With keys
// as the rows of the matrix products (S^T = K Q^T, O^T = V^T P^T), a lane's scores, sums and
// outputs all belong to one query row, so the running maximum and the rescaling need no
// exchange between lanes, and P^T leaves the first product where the second one reads it.
//
// Bound by HBM: every key and value byte passes once. The keys of all sequences are cut into
// parts of about equal length, however ragged the batch (every wave finds its part from
// kv_lens; no host copy is needed), and a part's four waves walk 32 tokens at a time each.
// The codes are widened to bf16 in registers, exactly; the scales of a page multiply scores
// and weights. The weights p enter the second product as high and low bf16 parts: the
// matrix units idle otherwise, and the output keeps fp32's accuracy.

#include <limits.h>
#include <math.h>

#include <algorithm>

#include "kda_cache_attn.h"

namespace kda {
namespace cache {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 32;     // tokens of a wave's step
constexpr int32_t kWhole = 1 << 28;  // units of a part where nothing is cut
constexpr int kRow = D + 4;   // fp32 row in LDS
// The reference exponent of a row moves only when a score passes it by this much (base 2):
// weights stay below 2^8, far inside bf16 and fp32.
constexpr float kSlack = 8.0f;

struct Part {
  int32_t b, index, parts, slot;
  int32_t from, to;  // tokens
};

// Part `item` of all sequences' parts, by each wave for itself.
__device__ __forceinline__ bool find_part(const AttnParams& p, int32_t item, int lane, Part& out) {
  const int32_t B = p.c.n_seqs;
  int32_t chunk = kWhole;
  if (p.targets > 0) {
    int32_t sum = 0;
    for (int32_t b = lane; b < B; b += 64) sum += is_few(p, b) ? units_of(p.c, b) : 0;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s);
    chunk = max(kMinUnits, (sum + p.targets - 1) / p.targets);
  }
  int32_t items = 0, slots = 0;
  for (int32_t b0 = 0; b0 < B; b0 += 64) {
    const int32_t b = b0 + lane;
    const bool few = b < B && is_few(p, b);
    const int32_t units = few ? units_of(p.c, b) : 0;
    const int32_t n = few ? max((units + chunk - 1) / chunk, 1) : 0;
    const int32_t s = n > 1 ? n : 0;
    int32_t ni = n, si = s;  // inclusive prefix sums
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t x = __shfl_up(ni, d), y = __shfl_up(si, d);
      if (lane >= d) ni += x, si += y;
    }
    const uint64_t hit = __ballot(item < items + ni);
    if (hit) {
      const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      out.b = b0 + at;
      out.parts = __shfl(n, at);
      out.index = item - (items + __shfl(ni - n, at));
      out.slot = slots + __shfl(si - s, at);
      out.from = out.parts == 1 ? 0 : out.index * chunk * kUnit;
      out.to = out.index + 1 == out.parts ? INT_MAX : out.from + chunk * kUnit;
      out.b = __builtin_amdgcn_readfirstlane(out.b);
      out.parts = __builtin_amdgcn_readfirstlane(out.parts);
      out.index = __builtin_amdgcn_readfirstlane(out.index);
      out.slot = __builtin_amdgcn_readfirstlane(out.slot);
      out.from = __builtin_amdgcn_readfirstlane(out.from);
      out.to = __builtin_amdgcn_readfirstlane(out.to);
      return true;
    }
    items += __shfl(ni, 63);
    slots += __shfl(si, 63);
  }
  return false;
}

// 32 tokens of a wave: two tiles of 16, each inside one page.
struct Step {
  u32x4 k[2][2];  // lane (m, g): token m, channels 64 i + 16 g ..
  u32x2 v[2][4];  // lane (m, g): token 4 g + r, channels 8 m ..
  float ks[2], vs[2];
  int32_t live[2];  // tokens that exist
};

__device__ __forceinline__ void load_step(const AttnParams& p, int32_t b, int32_t h, int32_t at,
                                          int32_t end, int lane, Step& s) {
  const int m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int32_t tok = at + 16 * u;
    int32_t id = -1;
    if (tok < end) id = page_of(p.c, b, tok >> p.c.page_shift);
    s.live[u] = id < 0 ? 0 : min(16, end - tok);
    id = max(id, 0);  // page 0's bytes in the place of none's
    const int64_t in_page =
        ((int64_t(h) << p.c.page_shift) + (tok & ((1 << p.c.page_shift) - 1))) * D;
    const uint8_t* const k = p.c.k + id * p.c.k_page + in_page;
    const uint8_t* const v = p.c.v + id * p.c.v_page + in_page;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      s.k[u][i] = *reinterpret_cast<const u32x4*>(k + m * D + i * 64 + g * 16);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      s.v[u][r] = *reinterpret_cast<const u32x2*>(v + (4 * g + r) * D + m * 8);
    const int64_t sc = int64_t(id) * p.c.H + h;
    s.ks[u] = p.c.k_scale[sc];
    s.vs[u] = p.c.v_scale[sc];
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

// O^T += V^T P^T over the step's 32 tokens.
template <int KIND, int NT>
__device__ __forceinline__ void weigh(const Step& s, const bf16x8 (&ph)[NT], const bf16x8 (&pl)[NT],
                                      f32x4 (&o)[NT][8]) {
#pragma unroll
  for (int c4 = 0; c4 < 2; ++c4) {  // channels 8 m + 4 c4 ..
    uint32_t t0[4], t1[4];
    transpose4(s.v[0][0][c4], s.v[0][1][c4], s.v[0][2][c4], s.v[0][3][c4], t0);
    transpose4(s.v[1][0][c4], s.v[1][1][c4], s.v[1][2][c4], s.v[1][3][c4], t1);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bf16x8 v = widen8<KIND>(t0[c], t1[c]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][4 * c4 + c] = mfma32(v, ph[n], o[n][4 * c4 + c]);
        o[n][4 * c4 + c] = mfma32(v, pl[n], o[n][4 * c4 + c]);
      }
    }
  }
}
// Whether a value code of a token behind `all_see` is e4m3's NaN.
__device__ __forceinline__ bool nan_beyond(const Step& s, int32_t at, int32_t all_see, int g) {
  uint32_t any = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (at + 16 * u + 4 * g + r > all_see)
        any |= ((s.v[u][r][0] & 0x7f7f7f7fu) + 0x01010101u) |
               ((s.v[u][r][1] & 0x7f7f7f7fu) + 0x01010101u);
  return __any((any & 0x80808080u) != 0);
}

// One workgroup: (part, key/value head, block of 16 NT rows).
template <int KIND, int NT>
__global__ __launch_bounds__(kThreads) void attend_kernel(AttnParams p) {
  __shared__ float sums[4][16 * kRow];
  __shared__ float refs[4][16], tots[4][16];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = p.c.H * p.row_blocks;
  const int item = blockIdx.x / per, hb = blockIdx.x - item * per;
  const int rb = hb / p.c.H, h = hb - rb * p.c.H;
  Part part;
  if (!find_part(p, item, lane, part)) return;
  const Seq seq = sequence(p.c, part.b);
  if (hb == 0 && part.index == 0 && threadIdx.x == 0)
    p.plan[part.b] = make_int2(part.slot, part.parts);
  const int rows = rows_of(p, part.b), row0 = rb * 16 * NT;
  if (row0 >= rows) return;
  const int32_t len = p.c.num_pages > 0 ? max(seq.len, 0) : 0;
  const int32_t to = min(part.to, len);

  // queries: lane (m, g) holds row m's channels of group g, eight per product
  bf16x8 q[NT][4];
  int32_t last[NT];  // the last position that the lane's row sees
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 16 * n + m, t = r / p.G;
    last[n] = len - seq.n + t;
    const uint16_t* const at =
        p.q + (seq.first + t) * p.q_stride + (int64_t(h) * p.G + (r - t * p.G)) * D;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (r < rows)
        w = *reinterpret_cast<const u32x4_u*>(at + (j >> 1) * 64 + g * 16 + (j & 1) * 8);
      q[n][j] = __builtin_bit_cast(bf16x8, w);
    }
  }
  const int32_t all_see = len - seq.n + row0 / p.G;  // every row of the block sees up to here

  f32x4 o[NT][8];
  float ref[NT], tot[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    ref[n] = -INFINITY;
    tot[n] = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[n][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  Step next;
  int32_t at = part.from + wave * kStep;
  if (at < to) load_step(p, part.b, h, at, to, lane, next);
  for (; at < to; at += 4 * kStep) {
    Step cur = next;
    if (at + 4 * kStep < to) load_step(p, part.b, h, at + 4 * kStep, to, lane, next);
    const bool masked = cur.live[0] < 16 || cur.live[1] < 16 || at + kStep - 1 > all_see;
    if (cur.live[0] < 16 || cur.live[1] < 16) {  // bytes of tokens that are not there
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * g + r >= cur.live[u]) cur.v[u][r] = u32x2{0u, 0u};
    }
    bf16x8 ph[NT], pl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float s[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc = mfma32(widen8<KIND>(cur.k[u][j >> 1][2 * (j & 1)], cur.k[u][j >> 1][2 * (j & 1) + 1]),
                       q[n][j], acc);
        const float f = p.scale2 * cur.ks[u];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[u][r] = acc[r] * f;
          if (masked && (4 * g + r >= cur.live[u] || at + 16 * u + 4 * g + r > last[n]))
            s[u][r] = -INFINITY;
        }
      }
      float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                        fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      if (__any(top > ref[n] + kSlack)) {
        const float to_ref = fmaxf(ref[n], over_groups_max(top));
        const float f = to_ref == ref[n] ? 1.0f : __builtin_amdgcn_exp2f(ref[n] - to_ref);
        ref[n] = to_ref;
        tot[n] *= f;
#pragma unroll
        for (int c = 0; c < 8; ++c) o[n][c] *= f;
      }
      const float r0 = ref[n] == -INFINITY ? 0.0f : ref[n];
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[r] = __builtin_amdgcn_exp2f(s[u][r] - r0);
          tot[n] += w[r];
          w[r] *= cur.vs[u];
          if (masked && 4 * g + r >= cur.live[u]) w[r] = 0.0f;  // whatever that scale was
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
    if (KIND == kFp8 && masked && nan_beyond(cur, at, all_see, g)) {
      // a NaN value that some rows see and others do not: token by token, since 0 NaN = NaN
      for (int32_t t = row0 / p.G; t <= (row0 + 16 * NT - 1) / p.G; ++t) {
        const int32_t end = len - seq.n + t;
        Step seen = cur;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (at + 16 * u + 4 * g + r > end) seen.v[u][r] = u32x2{0u, 0u};
        f32x4 part_o[NT][8];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 8; ++c) part_o[n][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        weigh<KIND, NT>(seen, ph, pl, part_o);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (last[n] == end) {
#pragma unroll
            for (int c = 0; c < 8; ++c) o[n][c] += part_o[n][c];
          }
      }
    } else {
      weigh<KIND, NT>(cur, ph, pl, o);
    }
  }

  // the four waves' sums, 16 rows at a time; thread (row, 8 channels)
  const int row = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float total = over_groups_sum(tot[n]);
    if (n > 0) __syncthreads();
    if (g == 0) {
      refs[wave][m] = ref[n];
      tots[wave][m] = total;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* const to_lds = &sums[wave][m * kRow + (4 * g + r) * 8];
      *reinterpret_cast<f32x4*>(to_lds) = f32x4{o[n][0][r], o[n][1][r], o[n][2][r], o[n][3][r]};
      *reinterpret_cast<f32x4*>(to_lds + 4) = f32x4{o[n][4][r], o[n][5][r], o[n][6][r], o[n][7][r]};
    }
    __syncthreads();
    const float top = fmaxf(fmaxf(refs[0][row], refs[1][row]), fmaxf(refs[2][row], refs[3][row]));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = __builtin_amdgcn_exp2f(refs[w][row] - base);
      sum += tots[w][row] * f;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += sums[w][row * kRow + ch + c] * f;
    }
    const int r = row0 + 16 * n + row;
    if (r >= rows) continue;
    if (part.parts == 1) {
      const int t = r / p.G;
      const int64_t head = int64_t(h) * p.G + (r - t * p.G);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<u32x4_u*>(p.out + (seq.first + t) * p.out_stride + head * D + ch) =
          u32x4{pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv)};
      if (p.lse && ch == 0)
        p.lse[(seq.first + t) * p.lse_stride + head] =
            sum == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(sum)) * LN2;
    } else {
      const int64_t slot = (int64_t(part.slot + part.index) * p.c.H + h) * p.most_rows + r;
      float* const dst = p.part + slot * D + ch;
      *reinterpret_cast<f32x4*>(dst) = f32x4{acc[0], acc[1], acc[2], acc[3]};
      *reinterpret_cast<f32x4*>(dst + 4) = f32x4{acc[4], acc[5], acc[6], acc[7]};
      if (ch == 0) p.stat[slot] = make_float2(top, sum);
    }
  }
}

// Joins the parts of a row: a wave per row, 32 lanes of 4 channels, every other part each.
__global__ __launch_bounds__(kThreads) void join_kernel(AttnParams p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = (p.most_rows * p.c.H + 3) / 4;
  const int b = blockIdx.x / per, i = (blockIdx.x - b * per) * 4 + wave;
  if (i >= p.most_rows * p.c.H || !is_few(p, b)) return;
  const int2 plan = p.plan[b];
  const Seq seq = sequence(p.c, b);
  const int r = i / p.c.H, h = i - r * p.c.H;
  if (plan.y <= 1 || r >= p.G * seq.n) return;
  const int64_t first = (int64_t(plan.x) * p.c.H + h) * p.most_rows + r;
  const int64_t step = int64_t(p.c.H) * p.most_rows;
  float top = -INFINITY;
  for (int s = lane; s < plan.y; s += 64) top = fmaxf(top, p.stat[first + s * step].x);
#pragma unroll
  for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = lane >> 5; s < plan.y; s += 2) {
    const float2 st = p.stat[first + s * step];
    const float f = __builtin_amdgcn_exp2f(st.x - base);
    sum += st.y * f;
    acc += *reinterpret_cast<const f32x4*>(p.part + (first + s * step) * D + (lane & 31) * 4) * f;
  }
  sum += __shfl_xor(sum, 32);
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] += __shfl_xor(acc[c], 32);
  if (lane >= 32) return;
  const int t = r / p.G;
  const int64_t head = int64_t(h) * p.G + (r - t * p.G);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  typedef u32x2 u32x2_u __attribute__((aligned(2)));
  *reinterpret_cast<u32x2_u*>(p.out + (seq.first + t) * p.out_stride + head * D + lane * 4) =
      u32x2{pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv)};
  if (p.lse && lane == 0)
    p.lse[(seq.first + t) * p.lse_stride + head] =
        sum == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(sum)) * LN2;
}

// Host: the plan of a call.
constexpr int64_t kGroups = 1024;  // workgroups that the cut aims at
constexpr int32_t kFewRows = 64;   // sequences with more rows are documents

struct Plan {
  int32_t tiles, row_blocks, targets;
  int64_t plan_bytes, stat_bytes, bytes;
};
// Sequences of at most `rows` <= kFewRows rows for each of H key/value heads.
Plan make_plan(int32_t n_seqs, int32_t rows, int32_t H) {
  Plan r;
  r.tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  r.row_blocks = (rows + 16 * r.tiles - 1) / (16 * r.tiles);
  r.targets = int32_t(std::max<int64_t>(1, kGroups / (int64_t(H) * r.row_blocks)));
  // a cut sequence has less than twice its share of the parts
  const int64_t vecs = 2 * int64_t(r.targets) * H * rows;
  r.plan_bytes = (int64_t(n_seqs) * 8 + 255) / 256 * 256;
  r.stat_bytes = (vecs * 8 + 255) / 256 * 256;
  r.bytes = r.plan_bytes + r.stat_bytes + vecs * D * 4;
  return r;
}

template <int KIND>
hipError_t launch_attend(const AttnParams& p, const Plan& plan, unsigned grid, hipStream_t stream) {
  if (plan.tiles == 1)
    hipLaunchKernelGGL((attend_kernel<KIND, 1>), dim3(grid), dim3(kThreads), 0, stream, p);
  else if (plan.tiles == 2)
    hipLaunchKernelGGL((attend_kernel<KIND, 2>), dim3(grid), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((attend_kernel<KIND, 4>), dim3(grid), dim3(kThreads), 0, stream, p);
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
  if (n_seqs < 1 || total_tokens < 1 || kc::bad_heads(H_q, H_kv) || H_q / H_kv > 256) return 0;
  // the largest that any split of the tokens over the sequences needs
  const int32_t G = H_q / H_kv;
  int64_t most = 0;
  for (int64_t n = 1; n <= total_tokens && n * G <= kc::kFewRows; ++n)
    most = std::max(most, kc::make_plan(n_seqs, int32_t(n * G), H_kv).bytes);
  return size_t(most);
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
  if (H_q / H_kv > 256 || !isfinite(scale)) return KDA_ERR_UNSUPPORTED;
  const int64_t row = int64_t(H_q) * D;
  if (q_row_stride < 0 || out_row_stride < 0 || (lse && lse_row_stride < 0) ||
      !kc::rows_apart(total_tokens, out_row_stride, row) ||
      (lse && !kc::rows_apart(total_tokens, lse_row_stride, H_q)))
    return KDA_ERR_BAD_STRIDE;
  if (total_tokens == 0) return KDA_OK;
  if (!q || !out) return KDA_ERR_NULL_POINTER;
  if ((cu_seqlens != nullptr) != (cu_seqlens_host != nullptr)) return KDA_ERR_NULL_POINTER;
  p.G = H_q / H_kv;
  // the most rows of few-token sequences, of documents, and the documents' blocks
  int64_t few = 0, most = 0, blocks = 0;
  const auto note = [&](int64_t n, int64_t times) {
    const int64_t rows = n * p.G;
    if (rows <= kc::kFewRows) {
      few = std::max(few, rows);
    } else {
      most = std::max(most, rows);
      blocks += (rows + kc::kDocRows - 1) / kc::kDocRows * times;
    }
  };
  if (cu_seqlens_host) {
    if (cu_seqlens_host[0] != 0 || cu_seqlens_host[n_seqs] > total_tokens) return KDA_ERR_BAD_SEQLENS;
    for (int32_t b = 0; b < n_seqs; ++b) {
      const int64_t n = int64_t(cu_seqlens_host[b + 1]) - cu_seqlens_host[b];
      if (n < 0) return KDA_ERR_BAD_SEQLENS;
      note(n, 1);
    }
  } else {
    note(p.c.per_seq, n_seqs);
  }
  kc::Plan plan = {};
  int64_t grid = 0, joins = 0;
  if (few > 0) {
    plan = kc::make_plan(n_seqs, int32_t(few), H_kv);
    grid = (int64_t(plan.targets) + n_seqs) * H_kv * plan.row_blocks;
    joins = (few * H_kv + 3) / 4 * n_seqs;
    if (workspace_bytes < size_t(plan.bytes)) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace) return KDA_ERR_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_UNSUPPORTED;
  }
  if (grid > INT32_MAX || joins > INT32_MAX || most > INT32_MAX - kc::kDocRows ||
      blocks * H_kv > INT32_MAX)
    return KDA_ERR_UNSUPPORTED;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_row_stride;
  p.scale2 = scale * kda::LOG2E;
  p.out = static_cast<uint16_t*>(out);
  p.out_stride = out_row_stride;
  p.lse = lse;
  p.lse_stride = lse_row_stride;
  p.few_rows = kc::kFewRows;
  p.row_blocks = plan.row_blocks;
  p.targets = plan.targets;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<int2*>(ws);
  p.stat = reinterpret_cast<float2*>(ws + plan.plan_bytes);
  p.part = reinterpret_cast<float*>(ws + plan.plan_bytes + plan.stat_bytes);
  const bool int8 = cache_dtype == KDA_CACHE_INT8;
  if (few > 0) {
    p.most_rows = int32_t(few);
    if ((int8 ? kc::launch_attend<kc::kInt8>(p, plan, unsigned(grid), stream)
              : kc::launch_attend<kc::kFp8>(p, plan, unsigned(grid), stream)) != hipSuccess)
      return KDA_ERR_LAUNCH;
    // no part is cut where the table is too short for two
    if (int64_t(table_width) * page_size > kc::kMinUnits * kc::kUnit) {
      hipLaunchKernelGGL(kc::join_kernel, dim3(unsigned(joins)), dim3(kc::kThreads), 0, stream, p);
      if (hipGetLastError() != hipSuccess) return KDA_ERR_LAUNCH;
    }
  }
  if (blocks > 0) {
    p.most_rows = int32_t(most);
    if (kc::launch_documents(p, int8, unsigned(blocks * H_kv), stream) != hipSuccess)
      return KDA_ERR_LAUNCH;
  }
  return KDA_OK;
}
