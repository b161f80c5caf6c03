// Attention of packed documents over the paged 8-bit cache (gfx950).
//
// Bound by the matrix units: 4 * 128 operations for every visible (query row, key) pair. Row r of
// a document and key/value head is query head r mod G of token r / G, so that grouped heads
// share what is loaded. A workgroup takes 32 rows per wave and walks 64 keys at a time: their
// codes are widened to bf16 once for all its waves, into LDS (exact for the values' scales that
// kda_cache_write makes; the keys' scales multiply the scores), the values transposed on the way. The
// next tile's codes come in meanwhile, and two workgroups share a CU, so that one's exponentials
// run beside the other's products.
//
// With keys as the rows of the products (S^T = K Q^T, O^T = V^T P^T) all of a lane's scores and
// outputs belong to one query row, and the weights P^T leave the first product in the
// layout that the second one reads. They are rounded to bf16 there (the sum that divides them is
// not): errors of half a step, independent of one another, that leave the output about as far off
// as its own rounding does; a second part would cost a quarter more products.

#include <math.h>

#include "kda_cache_attn.h"

namespace kda {
namespace cache {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;  // keys
constexpr float kSlack = 8.0f;
constexpr float kNoRef = -3.0e38f;

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Tile {
  // chunk c < 8 of a key's row: channels 16 c .., c >= 8: channels 16 (c - 8) + 8 ..; at c ^ (key & 7)
  u32x4 k[kTile * 16];
  // a channel's row: tokens of each run of 16 in the order 0-3, 8-11, 4-7, 12-15, chunks of 8 at
  // c ^ swizzle(channel)
  u32x2 v[D * kTile / 4];
  float ks[4];
  int32_t live[4];  // tokens of each 16 that exist
};
__device__ __forceinline__ int swizzle(int channel) { return (channel ^ (channel >> 3)) & 7; }

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A thread's share of a tile's codes. T threads.
template <int T>
struct Share {
  static constexpr int KC = kTile * 8 / T, VC = kTile * 4 / T;
  u32x4 k[KC];
  u32x2 v[VC][4];
  float vs[VC];
  float ks;
  int32_t live;
};
// Keys: chunk i of thread t is 16 codes of row (t + i T) / 8. Values: unit t + i T is four tokens
// of 8 channels; neighbouring units are quads 0 and 2 or 1 and 3 of 16 tokens.
__device__ __forceinline__ int unit_token(int unit) {
  return (unit >> 6) * 16 + (unit & 1) * 8 + ((unit >> 5) & 1) * 4;
}
__device__ __forceinline__ int unit_channel(int unit) { return ((unit >> 1) & 15) * 8; }

template <int T>
struct Pages {
  int32_t k[Share<T>::KC], v[Share<T>::VC], s;
};
template <int T>
__device__ __forceinline__ void load_pages(const AttnParams& p, int32_t b, int32_t at, int32_t end,
                                           Pages<T>& g) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < Share<T>::KC; ++i) {
    const int32_t tok = at + ((t + i * T) >> 3);
    g.k[i] = tok < end ? page_of(p.c, b, tok >> p.c.page_shift) : -1;
  }
#pragma unroll
  for (int i = 0; i < Share<T>::VC; ++i) {
    const int32_t tok = at + unit_token(t + i * T);
    g.v[i] = tok < end ? page_of(p.c, b, tok >> p.c.page_shift) : -1;
  }
  const int32_t tok = at + (t & 3) * 16;
  g.s = tok < end ? page_of(p.c, b, tok >> p.c.page_shift) : -1;
}
template <int T>
__device__ __forceinline__ void load_share(const AttnParams& p, int32_t h, int32_t at, int32_t end,
                                           const Pages<T>& g, Share<T>& s) {
  const int t = threadIdx.x;
  const int32_t in = (1 << p.c.page_shift) - 1;
#pragma unroll
  for (int i = 0; i < Share<T>::KC; ++i) {
    const int u = t + i * T;
    const int32_t tok = at + (u >> 3);
    s.k[i] = *reinterpret_cast<const u32x4*>(
        p.c.k + max(g.k[i], 0) * p.c.k_page +
        ((int64_t(h) << p.c.page_shift) + (tok & in)) * D + (u & 7) * 16);
  }
#pragma unroll
  for (int i = 0; i < Share<T>::VC; ++i) {
    const int u = t + i * T;
    const int32_t tok = at + unit_token(u);
    const uint8_t* const v = p.c.v + max(g.v[i], 0) * p.c.v_page +
                             ((int64_t(h) << p.c.page_shift) + (tok & in)) * D + unit_channel(u);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s.v[i][r] = *reinterpret_cast<const u32x2*>(v + r * D);
      if (g.v[i] < 0 || tok + r >= end) s.v[i][r] = u32x2{0u, 0u};
    }
    s.vs[i] = g.v[i] < 0 ? 1.0f : p.c.v_scale[int64_t(g.v[i]) * p.c.H + h];
  }
  s.ks = p.c.k_scale[int64_t(max(g.s, 0)) * p.c.H + h];
  s.live = g.s < 0 ? 0 : min(16, end - (at + (t & 3) * 16));
}

// Widened values of four tokens of one channel, times their scale.
template <int KIND>
__device__ __forceinline__ u32x2 scaled4(uint32_t w, float scale, bool power) {
  if constexpr (KIND == kFp8) {
    if (power)
      return u32x2{
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))};
    const f32x2 a = f8x2_lo(w), b = f8x2_hi(w);
    return u32x2{pack_bf16x2(a[0] * scale, a[1] * scale), pack_bf16x2(b[0] * scale, b[1] * scale)};
  } else {
    return u32x2{pack_bf16x2(float(int8_t(w)) * scale, float(int8_t(w >> 8)) * scale),
                 pack_bf16x2(float(int8_t(w >> 16)) * scale, float(int8_t(w >> 24)) * scale)};
  }
}

// To LDS. With `diagonal`, NaN codes become zeros and leave the first position that holds one in
// nan_at[channel]: rows that see it become NaN in the end, and the others stay clear of 0 NaN.
template <int KIND, int T>
__device__ __forceinline__ void store_share(Share<T>& s, int32_t at, bool diagonal, Tile& to,
                                            int32_t* nan_at) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < Share<T>::KC; ++i) {
    const int u = t + i * T, row = u >> 3, c = (u & 7) ^ (row & 7);
    const u32x2 a = widen4<KIND>(s.k[i][0]), b = widen4<KIND>(s.k[i][1]);
    const u32x2 d = widen4<KIND>(s.k[i][2]), e = widen4<KIND>(s.k[i][3]);
    to.k[row * 16 + c] = u32x4{a[0], a[1], b[0], b[1]};
    to.k[row * 16 + 8 + c] = u32x4{d[0], d[1], e[0], e[1]};
  }
#pragma unroll
  for (int i = 0; i < Share<T>::VC; ++i) {
    const int u = t + i * T, tok = unit_token(u), ch = unit_channel(u);
    if (KIND == kFp8 && diagonal) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t hit = nan_codes(s.v[i][r][j]);
          if (hit) s.v[i][r][j] &= ~note_nans(hit, nan_at + ch + 4 * j, at + tok + r);
        }
    }
    const bool power = !__any((__float_as_uint(s.vs[i]) & 0x007fffffu) != 0 || s.vs[i] <= 0.0f);
    // quad q of 16 tokens goes to place 0, 2, 1, 3
    const int quad = (tok >> 2) & 3, place = (tok >> 4) * 4 + ((quad & 1) << 1 | quad >> 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
      transpose4(s.v[i][0][j], s.v[i][1][j], s.v[i][2][j], s.v[i][3][j], w);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int channel = ch + 4 * j + c;
        to.v[channel * 16 + ((((place >> 1) ^ swizzle(channel)) << 1) | (place & 1))] =
            scaled4<KIND>(w[c], s.vs[i], power);
      }
    }
  }
  if (t < 4) {
    to.ks[t] = s.ks;
    to.live[t] = s.live;
  }
}

// One workgroup: (128 rows of a document, key/value head, part of its keys).
template <int KIND, bool SPLIT>
__global__ __launch_bounds__(kThreads, 2) void document_kernel(AttnParams p) {
  constexpr int T = kThreads, ROWS = kDocRows;
  extern __shared__ __align__(16) uint8_t smem[];
  Tile* const tiles = reinterpret_cast<Tile*>(smem);
  int32_t* const nan_at = reinterpret_cast<int32_t*>(tiles + 2);
  const int lane = threadIdx.x & 63, m = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = blockIdx.x / p.c.H, h = blockIdx.x - item * p.c.H;
  Part part;
  if (!find_part<SPLIT, T>(p, item, *reinterpret_cast<FindSmem*>(smem), part)) return;
  __syncthreads();
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

  for (int i = threadIdx.x; i < D; i += T) nan_at[i] = INT_MAX;

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

  f32x16 o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[c][i] = 0.0f;
  float ref = kNoRef, tot = 0.0f;

  Share<T> next;
  Pages<T> pages;
  if (begin < end) {
    load_pages<T>(p, part.b, begin, end, pages);
    load_share<T>(p, h, begin, end, pages, next);
    load_pages<T>(p, part.b, begin + kTile, end, pages);
  }
  __syncthreads();
  if (begin < end)
    store_share<KIND, T>(next, begin, begin + kTile - 1 > all_see, tiles[0], nan_at);
  __syncthreads();
  int which = 0;
  for (int32_t at = begin; at < end; at += kTile, which ^= 1) {
    const bool more = at + kTile < end;
    if (more) {
      load_share<T>(p, h, at + kTile, end, pages, next);
      load_pages<T>(p, part.b, at + 2 * kTile, end, pages);
    }
    const Tile& tile = tiles[which];
    if (at <= wave_most) {
      f32x16 s[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
        const int row = u * 32 + m;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = 2 * j + hi;
          const u32x4 k = tile.k[row * 16 + ((c & 8) | ((c ^ row) & 7))];
          s[u] = mfma(__builtin_bit_cast(bf16x8, k), q[j], s[u]);
        }
      }
      float f[4];
      int32_t live = INT_MAX;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = p.scale2 * tile.ks[i];
        live = min(live, tile.live[i]);
      }
      if (live < 16 || at + kTile - 1 > wave_all) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int in = 8 * (i >> 2) + 4 * hi + (i & 3);  // key of 32
            const int group = 2 * u + (i >> 3);
            const bool hidden = (in & 15) >= tile.live[group] || at + 32 * u + in > last;
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
        float t = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) t = fmaxf(t, s[u][i] * f[2 * u + (i >> 3)]);
        t = fmaxf(ref, fmaxf(t, __shfl_xor(t, 32)));
        const float down = t == ref ? 1.0f : __builtin_amdgcn_exp2f(ref - t);
        ref = t;
        tot *= down;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] *= down;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) x[u][i] = fmaf(s[u][i], f[2 * u + (i >> 3)], -ref);
      }
      bf16x8 w[4];
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
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int channel = c * 32 + m;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(
              &tile.v[channel * 16 + (((2 * g + hi) ^ swizzle(channel)) << 1)]);
          o[c] = mfma(__builtin_bit_cast(bf16x8, v), w[g], o[c]);
        }
      }
    }
    if (more)
      store_share<KIND, T>(next, at + kTile, at + 2 * kTile - 1 > all_see, tiles[which ^ 1], nan_at);
    __syncthreads();
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
        if (KIND == kFp8 && nan_at[ch + j] <= last) y[j] = NAN;
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
  constexpr int kSmem = 2 * sizeof(Tile) + D * 4;
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
