// Attention of packed documents over the paged 8-bit cache (gfx950).
//
// Bound by the matrix units: 4 * 128 operations for every visible (query row, key) pair. Row r of
// a document and key/value head is query head r mod G of token r / G, so that grouped heads
// share what is loaded. A workgroup takes 32 rows per wave and walks 64 keys at a time: their
// codes are widened once for all its waves, into LDS, exactly (keys to bf16, values to fp16), the
// values transposed on the way. The next tile's codes come in meanwhile, and two workgroups share a
// CU, so that one's exponentials run beside the other's products.
//
// With keys as the rows of the products (S^T = K Q^T, O^T = V^T P^T) all of a lane's scores and
// outputs belong to one query row, and the weights P^T leave the first product in the
// layout that the second one reads. A page's scales go to the scores and to the weights, there as
// log2 before the exponential, so that weight times scale is what the running maximum bounds: it
// fits fp16 whatever the scales, and the codes of the values do, too. fp16 rounds a weight by 2^-11
// at most, independently of others, which adds about 1 % to what rounding the output to bf16 leaves (root
// of the mean square; one bf16 part, at the same rate of products, added 41 % and took 1.37 ms
// instead of 1.40 in the first case below). The sum that divides is not rounded.
//
// Documents of 4096 and 1777 tokens behind 2000 to 12000, 64 query heads on 8: 1.40 to 1.46 ms on
// different cards, 912 to 951 TFLOP/s of the 1605 that a large library product reaches; 14 documents of
// 16384 tokens, 12 heads on 4, int8: 160 to 165 us, 710 to 689. In the first case matrix
// instructions take 44 % of a SIMD's cycles and vector ones 45 %.

#include <math.h>

#include "kda_cache_attn.h"

namespace kda {
namespace cache {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;   // keys
// Weights of the second product lie below 2^kSlack, the largest that a row has seen at 2^(kTop - 1)
// at least: fp16 rounds them by 2^-11 down to 2^-20 of that one, and by 2^-31 of it below.
constexpr float kTop = 7.0f, kSlack = 15.0f;
constexpr float kNoRef = -3.0e38f;
constexpr int32_t kWide = 40, kWideTile = 64;  // see `apart`

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __fp16 f16x8 __attribute__((__vector_size__(8 * sizeof(__fp16))));  // MFMA operand

// What a tile's groups of 16 tokens have in LDS: the keys' scale times the scores', log2 of the
// values' (of its magnitude), the reciprocal of that magnitude, and, as an integer, how many of the
// tokens exist (kWideTile less: see `apart`).
constexpr int kKeyScale = 0, kValueLog = 1, kValueInv = 2, kLive = 3, kGroupKinds = 4;

struct Smem {
  alignas(16) float group[2][kGroupKinds][4];  // of 16 tokens each
  // chunk c < 8 of a key's row: channels 16 c .., c >= 8: channels 16 (c - 8) + 8 ..; at
  // c ^ (key & 15): no bank conflicts
  u32x4 k[2][kTile * 16];
  // a channel's row: tokens of each run of 16 in the order 0-3, 8-11, 4-7, 12-15, chunks of 8 at
  // c ^ swizzle(channel)
  u32x2 v[2][D * kTile / 4];
  // the first position behind what every row sees that holds a NaN value
  int32_t nan_at[D];
  float ref_apart[kDocRows], tot_apart[kDocRows][2];  // see `apart`
  FindSmem find;
};
__device__ __forceinline__ int swizzle(int channel) { return (channel ^ (channel >> 3)) & 7; }

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// A wave brings in 16 tokens of a tile, which lie in one page: their bytes are a scalar base and
// a lane's offset. Page indices and scales come by vector loads all the same, whose counter keeps
// their order, and are looked at only where they are used, a tile later.
__device__ __forceinline__ int32_t load_page(const AttnParams& p, int32_t b, int32_t tok,
                                             int32_t end, int32_t zero) {
  return p.c.table[b * p.c.table_stride + (min(tok, end - 1) >> p.c.page_shift) + zero];
}
struct Share {
  u32x4 k[2];  // codes 16 (lane mod 8) .. of token lane / 8 and of the one 8 further on
  u32x2 v[4];  // four tokens of 8 channels; neighbouring lanes hold quads 0 and 2, or 1 and 3
  float ks, vs;
  int32_t live;  // tokens that exist
};
__device__ __forceinline__ int lane_token(int lane) { return (lane & 1) * 8 + (lane >> 5) * 4; }
__device__ __forceinline__ int lane_channel(int lane) { return ((lane >> 1) & 15) * 8; }

__device__ __forceinline__ void load_share(const AttnParams& p, int32_t raw, int32_t h, int32_t tok,
                                           int32_t end, int lane, int32_t zero, Share& s) {
  const int32_t id = __builtin_amdgcn_readfirstlane(raw);
  const bool is = tok < end && uint32_t(id) < uint32_t(p.c.num_pages);
  const int32_t use = is ? id : 0;  // page 0's bytes in the place of none's
  const int32_t in = ((h << p.c.page_shift) + (tok & ((1 << p.c.page_shift) - 1))) * D;
  const uint8_t* const k = p.c.k + (use * p.c.k_page + in);
  const uint8_t* const v = p.c.v + (use * p.c.v_page + in);
#pragma unroll
  for (int i = 0; i < 2; ++i) s.k[i] = *reinterpret_cast<const u32x4*>(k + lane * 16 + i * 8 * D);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    s.v[r] =
        *reinterpret_cast<const u32x2*>(v + (lane_token(lane) * D + lane_channel(lane)) + r * D);
  const int64_t at = int64_t(use) * p.c.H + h + zero;
  s.ks = p.c.k_scale[at];
  s.vs = p.c.v_scale[at];
  s.live = is ? min(16, end - tok) : 0;
}

// Four codes as two fp16 pairs, exact. int8: 0x6400 | b is 1024 + b.
template <int KIND>
__device__ __forceinline__ u32x2 widen4_f16(uint32_t w) {
  if constexpr (KIND == kFp8) {
    return u32x2{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))};
  } else {
    const f16x2 off = {_Float16(1152), _Float16(1152)};
    w ^= 0x80808080u;
    const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u));
    const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u));
    return u32x2{__builtin_bit_cast(uint32_t, a - off), __builtin_bit_cast(uint32_t, b - off)};
  }
}
// log2 of a scale: a whole number for a power of two, -infinity for zero.
__device__ __forceinline__ float log2_of(float x) {
  return float(__builtin_amdgcn_frexp_expf(x)) +
         __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(x));
}

// To LDS. Tokens that do not exist become zeros. With `diagonal`, so do NaN codes, which leave
// their position in nan_at: rows that see it become NaN in the end, and the others stay clear of
// 0 NaN.
template <int KIND>
__device__ __forceinline__ void store_share(Share& s, int wave, int lane, int32_t tok, bool diagonal,
                                            int slot, float scale2, Smem& lds) {
  const int c0 = (lane & 7) ^ (lane >> 3);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * wave + (lane >> 3) + 8 * i;
    whole(s.k[i]);
    const u32x2 a = widen4<KIND>(s.k[i][0]), b = widen4<KIND>(s.k[i][1]);
    const u32x2 d = widen4<KIND>(s.k[i][2]), e = widen4<KIND>(s.k[i][3]);
    lds.k[slot][row * 16 + (c0 ^ 8 * i)] = u32x4{a[0], a[1], b[0], b[1]};
    lds.k[slot][row * 16 + (c0 ^ 8 * (1 - i))] = u32x4{d[0], d[1], e[0], e[1]};
  }
  const int ch = lane_channel(lane);
#pragma unroll
  for (int r = 0; r < 4; ++r) whole(s.v[r]);
  if (s.live < 16) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (lane_token(lane) + r >= s.live) s.v[r] = u32x2{0u, 0u};
  }
  if (KIND == kFp8 && diagonal) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t hit = nan_codes(s.v[r][j]);
        if (hit)
          s.v[r][j] &= ~note_nans(hit, lds.nan_at + ch + 4 * j, tok + lane_token(lane) + r);
      }
  }
  // the scale's magnitude goes to the weights, its sign to the codes
  const uint32_t all = __builtin_amdgcn_readfirstlane(__float_as_int(s.vs));
  const uint32_t bits = s.live == 0 ? 0x3f800000u : all & 0x7fffffffu;
  const int32_t exponent = int32_t(bits >> 23) - 127;
  float lg = float(exponent), inv = __uint_as_float(0x7f000000u - bits);
  if ((bits & 0x007fffffu) != 0 || bits == 0) {  // no power of two
    asm volatile("");                            // (a branch, not a choice)
    lg = log2_of(__uint_as_float(bits));
    inv = __builtin_amdgcn_rcpf(__uint_as_float(bits));
  }
  bool wide = abs(exponent) > kWide;
  if (wide) {
    uint32_t some = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) some |= s.v[r][0] | s.v[r][1];
    if (KIND == kFp8) some &= 0x7f7f7f7fu;
    if (__ballot(some != 0) == 0) {  // zeros, whatever their scale is
      lg = -float(kWide);
      inv = __uint_as_float(uint32_t(127 + kWide) << 23);
      wide = false;
    }
  }
  if (lane == 0) {
    float* const to = &lds.group[slot][0][wave];
    to[4 * kKeyScale] = scale2 * s.ks;
    to[4 * kValueLog] = lg;
    to[4 * kValueInv] = inv;
    to[4 * kLive] = __int_as_float(wide ? s.live - kWideTile : s.live);
  }
  // quad q of 16 tokens goes to place 0, 2, 1, 3
  const int place = wave * 4 + ((lane >> 5) << 1 | (lane & 1));
  const auto put = [&](auto negative) {
    constexpr uint32_t kSigns = decltype(negative)::value ? 0x80008000u : 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
      transpose4(s.v[0][j], s.v[1][j], s.v[2][j], s.v[3][j], w);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int channel = ch + 4 * j + c;
        lds.v[slot][channel * 16 + ((((place >> 1) ^ swizzle(channel)) << 1) | (place & 1))] =
            widen4_f16<KIND>(w[c]) ^ kSigns;
      }
    }
  };
  if (int32_t(all) < 0 && s.live > 0)
    put(std::true_type());
  else
    put(std::false_type());
}

// Order of 16 products and their 16 operands from LDS: four operands ahead. (The compiler waits for
// each operand in front of its product.)
__device__ __forceinline__ void reads_ahead() {
  constexpr int kRead = 0x100, kProduct = 0x8, kAhead = 4;
  __builtin_amdgcn_sched_group_barrier(kRead, kAhead, 0);
#pragma unroll
  for (int i = 0; i < 16 - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(kProduct, kAhead, 0);
}

// One workgroup: (128 rows of a document, key/value head, part of its keys).
template <int KIND, bool SPLIT, bool LISTED>
__global__ __launch_bounds__(kThreads, 2) void document_kernel(AttnParams p) {
  constexpr int ROWS = kDocRows;
  __shared__ Smem lds;
  const int lane = threadIdx.x & 63, m = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = blockIdx.x / p.c.H, h = blockIdx.x - item * p.c.H;
  Part part;
  if (!find_part<SPLIT, kThreads, LISTED>(p, item, lds.find, part)) return;
  const Seq seq = sequence(p.c, part.b);
  const int32_t rows = rows_of(p, part.b);
  const int32_t row0 = part.rb * ROWS + wave * 32;
  const int32_t len = p.c.num_pages > 0 ? max(seq.len, 0) : 0;
  const int32_t base = len - seq.n;  // position of the first token
  // positions up to here are seen by the workgroup's first and last rows, the wave's first and last
  const int32_t all_see = base + part.rb * ROWS / p.G;
  const int32_t most = base + min(part.rb * ROWS + ROWS - 1, rows - 1) / p.G;
  const int32_t wave_all = base + row0 / p.G;
  const int32_t wave_most = row0 < rows ? base + min(row0 + 31, rows - 1) / p.G : -1;
  const int32_t begin = SPLIT ? part.from : 0;
  const int32_t end = min(SPLIT ? min(part.to, len) : len, most + 1);
  const int32_t tiles = begin < end ? (end - begin + kTile - 1) / kTile : 0;

  for (int i = threadIdx.x; i < D; i += kThreads) lds.nan_at[i] = INT_MAX;

  // queries: lane (m, hi) holds row m's chunk 2 j + hi of the keys' order
  bf16x8 q[8];
  const int32_t r = row0 + m, tok = r / p.G;
  const int64_t head = int64_t(h) * p.G + (r - tok * p.G);
  const int32_t last = r < rows ? base + tok : -1;
  {
    const uint16_t* const at = p.q + (seq.first + tok) * p.q_stride + head * D;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = 2 * j + hi;
      u32x4 w = {0u, 0u, 0u, 0u};
      if (r < rows)
        w = *reinterpret_cast<const u32x4_u*>(at + (c < 8 ? 16 * c : 16 * (c - 8) + 8));
      q[j] = __builtin_bit_cast(bf16x8, w);
    }
  }

  // a lane's operands: row m of 32 keys, chunks 2 j + hi; channel m of 32, chunks 2 g + hi
  const u32x4* keys_at[8];
  const u32x4* values_at[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) keys_at[i] = &lds.k[0][m * 16 + ((2 * i + hi) ^ (m & 15))];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    values_at[i] = reinterpret_cast<const u32x4*>(lds.v[0]) + m * 8 + ((2 * i + hi) ^ swizzle(m));
  }
  // the queries are there before the loop, whose waits are for what it loads itself
#pragma unroll
  for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(q[j]));

  f32x16 o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[c][i] = 0.0f;
  // Weights of the second product are 2^(score + vlog - ref), whatever the pages' scales; `tot`, the
  // weights' sum without the scales, is counted in 2^ref too, by vinv. References are whole numbers
  // that move when a weight passes 2^slack (by anything at first).
  float ref = 0.0f, slack = -INFINITY, tot = 0.0f;
  // Where a scale is zero or beyond 2^+-kWide, and the codes under it are not zeros, the weights with
  // and without the scales may be too far apart for one reference in fp32 (up to there, what is
  // flushed to zero is less than 2^-50 of `tot`): from that tile on, which goes the way of masked ones,
  // the wave counts `tot` in a reference of its own, in LDS. (From the first tile on: 160 -> 217 us
  // for the 14 documents, 1.43 -> 1.98 ms for the two chunks.)
  int32_t apart = 16;  // < 0: so it is
  float& ref_apart = lds.ref_apart[wave * 32 + m];
  float& tot_apart = lds.tot_apart[wave * 32 + m][hi];

  // the wave's tokens of a tile; what is stored next, and the page of what is loaded after it
  const int32_t mine = begin + 16 * wave;
  Share share;
  int32_t page = 0, zero = 0;
  asm volatile("" : "+v"(zero));
  if (tiles > 0) {
    page = load_page(p, part.b, mine, end, zero);
    load_share(p, page, h, mine, end, lane, zero, share);
    page = load_page(p, part.b, mine + kTile, end, zero);
  }
  __syncthreads();  // nan_at
  if (tiles > 0)
    store_share<KIND>(share, wave, lane, mine, begin + kTile - 1 > all_see, 0, p.scale2, lds);
  __syncthreads();
  for (int32_t t = 0; t < tiles; ++t) {
    const int32_t at = begin + t * kTile, tok_next = mine + (t + 1) * kTile;
    const int slot = t & 1;
    // (behind the last tile: bytes of page 0, which nothing reads)
    load_share(p, page, h, tok_next, end, lane, zero, share);
    page = load_page(p, part.b, tok_next + kTile, end, zero);
    if (at <= wave_most) {
      f32x16 s[2];
      f16x8 w[4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x4 k = keys_at[j][slot * (kTile * 16) + u * (32 * 16)];
          s[u] = mfma(__builtin_bit_cast(bf16x8, k), q[j], s[u]);
        }
      reads_ahead();
      float f[4];
      f32x4 c = *reinterpret_cast<const f32x4*>(lds.group[slot][kValueLog]);
      int32_t live = apart;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = lds.group[slot][kKeyScale][i];
        live = min(live, __float_as_int(lds.group[slot][kLive][i]));
      }
      if (live < 16 || at + kTile - 1 > wave_all) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int in = 8 * (i >> 2) + 4 * hi + (i & 3);  // key of 32
            const int group = 2 * u + (i >> 3);
            const bool hidden =
                (in & 15) >= (__float_as_int(lds.group[slot][kLive][group]) & 31) ||
                at + 32 * u + in > last;
            s[u][i] = hidden ? -INFINITY : s[u][i] * f[group];
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = 1.0f;
        if (__builtin_amdgcn_readfirstlane(live) < 0) {
          const float was = apart < 0 ? ref_apart : slack == -INFINITY ? kNoRef : ref;
          float now = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) now = fmaxf(now, s[u][i]);
          now = fmaxf(was, ceilf(fmaxf(now, __shfl_xor(now, 32))) - kTop);
          float sum = apart < 0 ? tot_apart : tot;
          if (now != was) sum *= __builtin_amdgcn_exp2f(was - now);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum += __builtin_amdgcn_exp2f(s[u][i] - now);
          tot_apart = sum;
          ref_apart = now;
          apart = -1;
        }
      }
      const f32x4 by = *reinterpret_cast<const f32x4*>(lds.group[slot][kValueInv]);
      c -= ref;
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[u][i] = fmaf(s[u][i], f[2 * u + (i >> 3)], c[2 * u + (i >> 3)]);
          top = fmaxf(top, s[u][i]);
        }
      if (__any(top > slack)) {
        top = fmaxf(top, __shfl_xor(top, 32));
        const float over = top > slack ? ceilf(top) - kTop : 0.0f;
        const float down = slack == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(-over);
        ref += over;
        if (top > slack) slack = kSlack;
        tot *= down;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= down;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[u][i] -= over;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t pk[4];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at8 = 8 * (g & 1) + 2 * i;
          const float a = __builtin_amdgcn_exp2f(s[g >> 1][at8]);
          const float b = __builtin_amdgcn_exp2f(s[g >> 1][at8 + 1]);
          sum = i == 0 ? a + b : sum + (a + b);
          pk[i] = pack_f16x2(a, b);
        }
        tot = fmaf(sum, by[g], tot);
        w[g] = __builtin_bit_cast(f16x8, u32x4{pk[0], pk[1], pk[2], pk[3]});
      }
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const u32x4 v = values_at[g ^ 2 * (c & 1)][slot * (D * kTile / 8) + c * (32 * kTile / 8)];
          o[c] = mfma(__builtin_bit_cast(f16x8, v), w[g], o[c]);
        }
      reads_ahead();
    }
    if (t + 1 < tiles)
      store_share<KIND>(share, wave, lane, tok_next, at + 2 * kTile - 1 > all_see, slot ^ 1,
                        p.scale2, lds);
    __syncthreads();
  }

  if (SPLIT) list_cuts(p, h, lds.find);
  if (apart < 0) tot = tot_apart;
  tot += __shfl_xor(tot, 32);
  if (r >= rows) return;
  const bool whole = !SPLIT || part.parts == 1;
  float inv = tot == 0.0f ? 0.0f : 1.0f / tot, ref_sum = ref;
  if (apart < 0) {
    ref_sum = ref_apart;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        o[c][i] = __builtin_amdgcn_ldexpf(o[c][i] * inv, int(ref - ref_sum));
    inv = 1.0f;
  }
  uint16_t* const dst = p.out + (seq.first + tok) * p.out_stride + head * D;
  const int64_t slot = (int64_t(part.slot) * p.c.H + h) * ROWS + wave * 32 + m;
  typedef u32x2 u32x2_u __attribute__((aligned(2)));
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = c * 32 + 8 * i + 4 * hi;
      f32x4 y;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = o[c][4 * i + j] * inv;
        if (KIND == kFp8 && lds.nan_at[ch + j] <= last) y[j] = NAN;
      }
      if (whole)
        *reinterpret_cast<u32x2_u*>(dst + ch) =
            u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
      else
        *reinterpret_cast<f32x4*>(p.part + slot * D + ch) = y;
    }
  if (hi != 0) return;
  if (!whole)
    p.stat[slot] = make_float2(tot == 0.0f ? -INFINITY : ref_sum, tot);
  else if (p.lse)
    p.lse[(seq.first + tok) * p.lse_stride + head] =
        log_sum(ref_sum, tot);
}

template <int KIND, bool SPLIT, bool LISTED>
hipError_t launch(const AttnParams& p, unsigned grid, hipStream_t stream) {
  hipLaunchKernelGGL((document_kernel<KIND, SPLIT, LISTED>), dim3(grid), dim3(kThreads), 0, stream,
                     p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_documents(const AttnParams& p, bool int8, unsigned grid, hipStream_t stream) {
  if (p.starts)
    return int8 ? launch<kInt8, true, true>(p, grid, stream)
                : launch<kFp8, true, true>(p, grid, stream);
  if (p.targets > 0)
    return int8 ? launch<kInt8, true, false>(p, grid, stream)
                : launch<kFp8, true, false>(p, grid, stream);
  return int8 ? launch<kInt8, false, false>(p, grid, stream)
              : launch<kFp8, false, false>(p, grid, stream);
}

}  // namespace cache
}  // namespace kda
