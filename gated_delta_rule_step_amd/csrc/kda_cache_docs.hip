// Attention of packed documents over the paged 8-bit cache (gfx950).
//
// Bound by the matrix units: 4 * 128 operations for every visible (query row, key) pair. Row r of
// a document and key/value head is query head r mod G of token r / G, so that grouped heads
// share what is loaded. A workgroup of eight waves takes 32 rows per wave and walks 64 keys at a time: their
// codes are widened to bf16 once for all its waves, into LDS (exact for the values' scales that
// kda_cache_write makes; the keys' scales multiply the scores), the values transposed on the way.
//
// With keys as the rows of the products (S^T = K Q^T, O^T = V^T P^T) all of a lane's scores and
// outputs belong to one query row, and the weights P^T leave the first product in the
// layout that the second one reads. They are rounded to bf16 there (the sum that divides them is
// not): errors of half a step, independent of one another, that leave the output about as far off
// as its own rounding does; a second part would cost a quarter more products.
//
// A wave's products and its exponentials take about as long, and neither hides the other. So the
// waves of a SIMD (one of the first four, one of the last four) take turns: in one phase the
// first multiply (scores of tile t + 1, outputs of tile t) while the last do the arithmetic between, in the next the
// other way round, with a barrier after each phase. The first four waves also bring in the keys, the last the
// values.

#include <math.h>

#include "kda_cache_attn.h"

namespace kda {
namespace cache {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 64;   // keys
constexpr float kSlack = 8.0f;
constexpr float kNoRef = -3.0e38f;

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Smem {
  // chunk c < 8 of a key's row: channels 16 c .., c >= 8: channels 16 (c - 8) + 8 ..; at c ^ (key & 7)
  u32x4 k[2][kTile * 16];
  // a channel's row: tokens of each run of 16 in the order 0-3, 8-11, 4-7, 12-15, chunks of 8 at
  // c ^ swizzle(channel)
  u32x2 v[2][D * kTile / 4];
  float ks[2][4];      // the keys' scales, 16 tokens each
  int32_t live[2][4];  // tokens of each 16 that exist
  // the first position behind what every row sees that holds a NaN value
  int32_t nan_at[D];
  FindSmem find;
};
__device__ __forceinline__ int swizzle(int channel) { return (channel ^ (channel >> 3)) & 7; }

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A wave's share of a tile lies in groups of 16 tokens, each inside one page: its bytes are a
// scalar base and a lane's offset. Page indices and scales come by vector loads all the same, whose
// counter keeps their order, and are looked at only where they are used, a tile later.
__device__ __forceinline__ int32_t load_page(const AttnParams& p, int32_t b, int32_t tok,
                                             int32_t end, int32_t zero) {
  return p.c.table[b * p.c.table_stride + (min(tok, end - 1) >> p.c.page_shift) + zero];
}
__device__ __forceinline__ int32_t known_page(const AttnParams& p, int32_t raw, int32_t tok,
                                              int32_t end) {
  const int32_t id = __builtin_amdgcn_readfirstlane(raw);
  return tok < end && uint32_t(id) < uint64_t(p.c.num_pages) ? id : -1;
}
__device__ __forceinline__ const uint8_t* group_at(const CacheView& c, const uint8_t* cache,
                                                   int64_t page, int32_t id, int32_t h, int32_t tok) {
  const int32_t in = tok & ((1 << c.page_shift) - 1);
  return cache + max(id, 0) * page + ((int64_t(h) << c.page_shift) + in) * D;
}

// Keys of a tile, by the first four waves: 16 codes of rows 8 wave + lane / 8 and 32 further on.
struct KeyShare {
  u32x4 w[2];
  float scale[2];
  int32_t live[2];
};
__device__ __forceinline__ void load_share(const AttnParams& p, int32_t h, int32_t tok, int32_t end,
                                           int wave, int lane, int32_t zero,
                                           const int32_t (&raw)[2], KeyShare& s) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t id = known_page(p, raw[i], tok + 32 * i, end);
    s.w[i] = *reinterpret_cast<const u32x4*>(
        group_at(p.c, p.c.k, p.c.k_page, id, h, tok + 32 * i) + ((wave & 1) * 8 * D + lane * 16));
    s.scale[i] = p.c.k_scale[int64_t(max(id, 0)) * p.c.H + h + zero];
    s.live[i] = id < 0 ? 0 : min(16, end - (tok + 32 * i));
  }
}
template <int KIND>
__device__ __forceinline__ void store_share(const KeyShare& s, int wave, int lane, int slot,
                                            Smem& lds) {
  const int c = (lane & 7) ^ (lane >> 3);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * wave + (lane >> 3) + 32 * i;
    const u32x2 a = widen4<KIND>(s.w[i][0]), b = widen4<KIND>(s.w[i][1]);
    const u32x2 d = widen4<KIND>(s.w[i][2]), e = widen4<KIND>(s.w[i][3]);
    lds.k[slot][row * 16 + c] = u32x4{a[0], a[1], b[0], b[1]};
    lds.k[slot][row * 16 + 8 + c] = u32x4{d[0], d[1], e[0], e[1]};
    if ((wave & 1) == 0 && lane == 0) {
      lds.ks[slot][(wave >> 1) + 2 * i] = s.scale[i];
      lds.live[slot][(wave >> 1) + 2 * i] = s.live[i];
    }
  }
}

// Values of a tile, by the last four waves: 16 tokens a wave, four of 8 channels a lane.
// Neighbouring lanes hold quads 0 and 2, or 1 and 3.
struct ValueShare {
  u32x2 w[4];
  float scale;
  int32_t live;
};
__device__ __forceinline__ int lane_token(int lane) { return (lane & 1) * 8 + (lane >> 5) * 4; }
__device__ __forceinline__ int lane_channel(int lane) { return ((lane >> 1) & 15) * 8; }
__device__ __forceinline__ void load_share(const AttnParams& p, int32_t h, int32_t tok, int32_t end,
                                           int lane, int32_t zero, int32_t raw, ValueShare& s) {
  const int32_t id = known_page(p, raw, tok, end);
  const uint8_t* const v = group_at(p.c, p.c.v, p.c.v_page, id, h, tok);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    s.w[r] = *reinterpret_cast<const u32x2*>(v + (lane_token(lane) * D + lane_channel(lane) + r * D));
  s.scale = p.c.v_scale[int64_t(max(id, 0)) * p.c.H + h + zero];
  s.live = id < 0 ? 0 : min(16, end - tok);
}

// Widened values of four tokens of one channel, times their scale (EXACT: a power of two).
template <int KIND, bool EXACT>
__device__ __forceinline__ u32x2 scaled4(uint32_t w, float scale) {
  if constexpr (EXACT) {
    return u32x2{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))};
  } else {
    float x[4];
    decode4<KIND>(w, x);
    return u32x2{pack_bf16x2(x[0] * scale, x[1] * scale), pack_bf16x2(x[2] * scale, x[3] * scale)};
  }
}

// Tokens that do not exist become zeros. With `diagonal`, so do NaN codes, which leave their
// position in nan_at: rows that see it become NaN in the end, and the others stay clear of 0 NaN.
template <int KIND>
__device__ __forceinline__ void store_share(ValueShare& s, int lane, int32_t tok, bool diagonal,
                                            int slot, int group, Smem& lds) {
  const int ch = lane_channel(lane);
  if (s.live < 16) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (lane_token(lane) + r >= s.live) s.w[r] = u32x2{0u, 0u};
  }
  if (KIND == kFp8 && diagonal) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t hit = nan_codes(s.w[r][j]);
        if (hit)
          s.w[r][j] &= ~note_nans(hit, lds.nan_at + ch + 4 * j, tok + lane_token(lane) + r);
      }
  }
  const float scale = s.live > 0 ? __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(
                                                               __builtin_bit_cast(int, s.scale)))
                               : 1.0f;
  // quad q of 16 tokens goes to place 0, 2, 1, 3
  const int place = group * 4 + ((lane >> 5) << 1 | (lane & 1));
  const auto put = [&](auto exact) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
      transpose4(s.w[0][j], s.w[1][j], s.w[2][j], s.w[3][j], w);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int channel = ch + 4 * j + c;
        lds.v[slot][channel * 16 + ((((place >> 1) ^ swizzle(channel)) << 1) | (place & 1))] =
            scaled4<KIND, decltype(exact)::value>(w[c], scale);
      }
    }
  };
  // the hardware's scale is a power of two
  if (KIND == kFp8 && (__float_as_uint(scale) & 0x007fffffu) == 0 && scale > 0.0f)
    put(std::true_type());
  else
    put(std::false_type());
}

// Order of 16 products and their 16 operands from LDS: six operands ahead.
__device__ __forceinline__ void reads_ahead() {
  constexpr int kRead = 0x100, kProduct = 0x8, kAhead = 6;
  __builtin_amdgcn_sched_group_barrier(kRead, kAhead, 0);
#pragma unroll
  for (int i = 0; i < 16 - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(kProduct, kAhead, 0);
}

// One workgroup: (256 rows of a document, key/value head, part of its keys).
template <int KIND, bool SPLIT>
__global__ __launch_bounds__(kThreads, 2) void document_kernel(AttnParams p) {
  constexpr int ROWS = kDocRows;
  extern __shared__ __align__(16) uint8_t smem[];
  Smem& lds = *reinterpret_cast<Smem*>(smem);
  const int lane = threadIdx.x & 63, m = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool first = wave < 4;  // the half that begins
  const int item = blockIdx.x / p.c.H, h = blockIdx.x - item * p.c.H;
  Part part;
  if (!find_part<SPLIT, kThreads>(p, item, lds.find, part)) return;
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

  // a lane's operands: row m of 32 keys, chunks 2 (j & 3) + hi; channel m of 32, chunks 2 g + hi
  const u32x4* keys_at[4];
  const u32x4* values_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    keys_at[i] = &lds.k[0][m * 16 + ((2 * i + hi) ^ (m & 7))];
    values_at[i] = reinterpret_cast<const u32x4*>(lds.v[0]) + m * 8 + ((2 * i + hi) ^ swizzle(m));
  }
  // the queries are there before the loop, whose waits are for what it loads itself
#pragma unroll
  for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(q[j]));

  f32x16 o[4], s[2];
  bf16x8 w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[c][i] = 0.0f;
  float ref = kNoRef, tot = 0.0f;

  __syncthreads();  // nan_at
  int32_t zero = 0;
  asm volatile("" : "+v"(zero));
  // One half's walk, in code of its own, so that what it loads stays in the registers where it arrives.
  // Keys of tile 0 are there before the first phase, keys of tile 1 and values of tile 0 come
  // during the first two, keys and values of tile t + 2 behind the products of step t.
  const auto walk = [&](auto half) {
    constexpr bool kFirst = decltype(half)::value;
    const int32_t mine = 16 * (kFirst ? wave >> 1 : wave - 4);  // the wave's tokens of a tile
    KeyShare keys;
    ValueShare values;
    int32_t pages[2];
    const auto load_ahead = [&](int32_t t) {
#pragma unroll
      for (int i = 0; i < (kFirst ? 2 : 1); ++i)
        pages[i] = load_page(p, part.b, begin + t * kTile + mine + 32 * i, end, zero);
    };
    // (behind the last tile: bytes of page 0, never stored)
    const auto load = [&](int32_t t) {
      const int32_t tok = begin + t * kTile + mine;
      if constexpr (kFirst)
        load_share(p, h, tok, end, wave, lane, zero, pages, keys);
      else
        load_share(p, h, tok, end, lane, zero, pages[0], values);
      load_ahead(t + 1);
    };
    const auto store = [&](int32_t t) {
      if (t >= tiles) return;
      const int32_t at = begin + t * kTile;
      if constexpr (kFirst)
        store_share<KIND>(keys, wave, lane, t & 1, lds);
      else
        store_share<KIND>(values, lane, at + mine, at + kTile - 1 > all_see, t & 1, wave - 4, lds);
    };
    load_ahead(0);
    load(0);
    if (kFirst) {
      store(0);
      load(1);
    }
    __syncthreads();
    if (!kFirst) {
      store(0);
      load(1);
      __syncthreads();
    }
    for (int32_t t = -1; t < tiles; ++t) {
    const int32_t at = begin + (t + 1) * kTile;
    const bool scores = t + 1 < tiles && at <= wave_most;
    const int slot = (t + 1) & 1;
    __builtin_amdgcn_s_setprio(1);
    if (scores) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x4 k = keys_at[j & 3][slot * (kTile * 16) + u * (32 * 16) + (j & 4) * 2];
          s[u] = mfma(__builtin_bit_cast(bf16x8, k), q[j], s[u]);
        }
      reads_ahead();
    }
    if (t >= 0 && at - kTile <= wave_most) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const u32x4 v =
              values_at[g ^ 2 * (c & 1)][(slot ^ 1) * (D * kTile / 8) + c * (32 * kTile / 8)];
          o[c] = mfma(__builtin_bit_cast(bf16x8, v), w[g], o[c]);
        }
      reads_ahead();
    }
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();
    if (scores) {
      float f[4];
      int32_t live = INT_MAX;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = p.scale2 * lds.ks[slot][i];
        live = min(live, lds.live[slot][i]);
      }
      if (live < 16 || at + kTile - 1 > wave_all) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int in = 8 * (i >> 2) + 4 * hi + (i & 3);  // key of 32
            const int group = 2 * u + (i >> 3);
            const bool hidden = (in & 15) >= lds.live[slot][group] || at + 32 * u + in > last;
            s[u][i] = hidden ? -INFINITY : s[u][i] * f[group];
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = 1.0f;
      }
      float x[2][16], top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[u][i] = fmaf(s[u][i], f[2 * u + (i >> 3)], -ref);
          top = fmaxf(top, x[u][i]);
        }
      if (__any(top > kSlack)) {
        float now = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) now = fmaxf(now, s[u][i] * f[2 * u + (i >> 3)]);
        now = fmaxf(ref, fmaxf(now, __shfl_xor(now, 32)));
        const float down = now == ref ? 1.0f : __builtin_amdgcn_exp2f(ref - now);
        ref = now;
        tot *= down;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] *= down;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) x[u][i] = fmaf(s[u][i], f[2 * u + (i >> 3)], -ref);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at8 = 8 * (g & 1) + 2 * i;
          const float a = __builtin_amdgcn_exp2f(x[g >> 1][at8]);
          const float b = __builtin_amdgcn_exp2f(x[g >> 1][at8 + 1]);
          tot += a + b;
          pk[i] = pack_bf16x2(a, b);
        }
        w[g] = __builtin_bit_cast(bf16x8, u32x4{pk[0], pk[1], pk[2], pk[3]});
      }
    }
      store(t + 2);
      load(t + 3);
      __syncthreads();
    }
    if (kFirst) __syncthreads();
  };
  if (tiles > 0) {
    if (first)
      walk(std::true_type());
    else
      walk(std::false_type());
  }

  if (SPLIT && h == 0 && part.rb == 0 && part.index == 0 && threadIdx.x == 0)
    p.plan[part.b] = make_int2(part.first_slot, part.parts);
  tot += __shfl_xor(tot, 32);
  if (r >= rows) return;
  const bool whole = !SPLIT || part.parts == 1;
  const float inv = !whole ? 1.0f : tot == 0.0f ? 0.0f : 1.0f / tot;
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
    p.stat[slot] = make_float2(tot == 0.0f ? -INFINITY : ref, tot);
  else if (p.lse)
    p.lse[(seq.first + tok) * p.lse_stride + head] =
        tot == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(tot)) * LN2;
}

template <int KIND, bool SPLIT>
hipError_t launch(const AttnParams& p, unsigned grid, hipStream_t stream) {
  constexpr int kSmem = sizeof(Smem);
  static const hipError_t ready = hipFuncSetAttribute(
      reinterpret_cast<const void*>(&document_kernel<KIND, SPLIT>),
      hipFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (ready != hipSuccess) return ready;
  hipLaunchKernelGGL((document_kernel<KIND, SPLIT>), dim3(grid), dim3(kThreads), kSmem, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_documents(const AttnParams& p, bool int8, unsigned grid, hipStream_t stream) {
  if (p.targets > 0)
    return int8 ? launch<kInt8, true>(p, grid, stream) : launch<kFp8, true>(p, grid, stream);
  return int8 ? launch<kInt8, false>(p, grid, stream) : launch<kFp8, false>(p, grid, stream);
}

}  // namespace cache
}  // namespace kda
