// Writing and reading the paged 8-bit key/value cache (gfx950).
//
// Both are bound by HBM (2 bytes per value on one side, 1 on the other) and, for a decode
// step's few tokens, by the latency of the chain sequence -> page -> scale -> bytes.
//
// Write: a page's scale needs the largest magnitude of all its new tokens before any can be
// rounded, so the tokens of one (page, head, side) stay in the registers of one workgroup
// (or one wave, where a page gets at most 16) between the two: read once, written once. 16384
// tokens of 8 heads 20.7 us, 4.9 TB/s; 8 tokens of 512 sequences of 12 heads, int8, 11.0 us; 32
// tokens of 8 heads 3.9 us.

#include <stdint.h>

#include "kda_cache.h"

namespace kda {
namespace cache {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -100;  // smallest exponent of a scale

struct WriteParams {
  CacheView c;
  const uint16_t* src[2];  // k, v
  int64_t src_stride[2];
  uint8_t* dst[2];
  float* scale[2];
  int32_t per_seq_items;  // without cu: pages that a sequence's tokens may touch
};

struct ReadParams {
  CacheView c;
  uint16_t* dst[2];
  int64_t dst_stride[2];
  int32_t per_seq_items, shift;  // units of 1 << shift tokens
};

// Work items are (sequence, unit with tokens of the call): a unit is a page or, for reads, an equal
// share of one. n tokens touch at most (n + U - 2) / U + 1 units of U tokens, so items of sequence b
// start at cu[b] / U + 2 b: no prefix sum. The last b with a start <= item, found by 64 lanes at a
// time.
__device__ __forceinline__ int32_t find_seq(const CacheView& p, int32_t item, int32_t shift,
                                            int32_t lane) {
  int32_t lo = 0, span = p.n_seqs;  // the answer lies in [lo, lo + span)
  while (span > 1) {
    const int32_t step = (span + 63) >> 6;
    const int32_t b = lo + lane * step;
    const bool is = lane * step < span &&
                    (clamp_row(p, p.cu[b]) >> shift) + 2 * int64_t(b) <= item;
    const int32_t hits = __popcll(__ballot(is));
    lo += max(hits - 1, 0) * step;
    span = min(step, p.n_seqs - lo);
  }
  return lo;
}

// The item's page (-1: none), the unit's first slot there, and the slots [a, z) that belong to the
// packed rows from `row` on.
struct Item {
  int32_t b, page, at, a, z;
  int64_t row;
};
__device__ __forceinline__ Item find_item(const CacheView& p, int32_t item, int32_t per_seq_items,
                                          int32_t shift, int32_t lane) {
  Item it;
  int32_t j;
  if (p.cu) {
    it.b = __builtin_amdgcn_readfirstlane(find_seq(p, item, shift, lane));
    j = item - ((clamp_row(p, p.cu[it.b]) >> shift) + 2 * it.b);
  } else {
    it.b = item / per_seq_items;
    j = item - it.b * per_seq_items;
  }
  const Seq s = sequence(p, it.b);
  const int32_t U = 1 << shift;
  it.page = -1;
  it.at = it.a = it.z = 0;
  it.row = s.first;
  if (j < 0 || s.n == 0) return it;
  // an inactive sequence's rows are walked as if it began on a page's border
  const int32_t start = s.len < 0 ? 0 : s.len - s.n;
  const int32_t first = start & (U - 1);
  const int64_t from = (int64_t(j) << shift) - first;  // token in the unit's first slot
  if (from >= s.n) return it;
  const int32_t unit = int32_t(start + from);
  it.at = unit & ((1 << p.page_shift) - 1);
  it.a = it.at + (from < 0 ? first : 0);
  it.z = it.at + int32_t(min(int64_t(U), int64_t(s.n) - from));
  it.row = s.first + (from < 0 ? 0 : from);
  if (s.len >= 0) it.page = page_of(p, it.b, unit >> p.page_shift);
  return it;
}

// Magnitude bits of finite bf16 values, 0 for others.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}
// need = 2^e from the bits of amax: 1.m 2^(E - 127) <= 1.75 2^8 2^e (e4m3),
// <= 1.984375 2^6 2^e (int8).
template <int KIND>
__device__ __forceinline__ float need_scale(uint32_t amax) {
  const int32_t E = int32_t(amax >> 7), m = int32_t(amax & 127u);
  const int32_t e = KIND == kFp8 ? E - 135 + (m > 96) : E - 133 + (m > 126);
  return __uint_as_float(uint32_t(max(e, kMinExp) + 127) << 23);
}

// Four values, already divided by the scale, to codes; whatever they are.
template <int KIND>
__device__ __forceinline__ float saturate(float x) {
  if constexpr (KIND == kFp8)
    return x != x ? x : f8_sat(x);  // a NaN stays one
  else
    return x != x ? 0.0f : __builtin_amdgcn_fmed3f(x, -127.0f, 127.0f);
}
// Values within the codes' range, inv a power of two. int8: the low byte of x + 1.5 2^23, whose last
// place is 1, is x rounded to nearest even. (One fused operation, since a inv is exact; it would
// pass over the rounding of any other product.)
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  if constexpr (KIND == kFp8) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true));
  } else {
    const auto code = [&](float x) { return __float_as_uint(fmaf(x, inv, 12582912.0f)); };
    const uint32_t lo = __builtin_amdgcn_perm(code(b), code(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code(d), code(c), 0x04000c0cu);
    return lo | hi;
  }
}
// Any values and any scale: a inv is rounded to fp32 first.
template <int KIND>
__device__ __forceinline__ uint32_t encode4_any(float a, float b, float c, float d, float inv) {
  return encode4<KIND>(saturate<KIND>(a * inv), saturate<KIND>(b * inv), saturate<KIND>(c * inv),
                       saturate<KIND>(d * inv), 1.0f);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  const auto step = [&](auto ctrl, auto rows) {
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), decltype(ctrl)::value,
                                                    decltype(rows)::value, 0xf, false)));
  };
  step(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());
  step(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());
  step(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());
  step(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());
  step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());
  step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());
  return uint32_t(__builtin_amdgcn_readlane(int(x), 63));
}

// A side's new rows of one (page, head): loaded, their largest magnitude, stored. By WAVES waves,
// 4 WAVES PASSES >= the page's new tokens; a row is 16 lanes of 8 channels.
template <int KIND, int WAVES, int PASSES>
struct Rows {
  u32x4 x[PASSES];
  float old;
  bool any;

  __device__ __forceinline__ void load(const WriteParams& p, int side, const Item& it, int h,
                                       int t) {
    old = it.a > 0 ? p.scale[side][int64_t(it.page) * p.c.H + h] : 0.0f;
    const uint16_t* const src =
        p.src[side] + it.row * p.src_stride[side] + h * D + (t & 15) * 8;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = (t >> 4) + i * 4 * WAVES;
      x[i] = u32x4{0u, 0u, 0u, 0u};
      if (r < it.z - it.a) x[i] = *reinterpret_cast<const u32x4_u*>(src + r * p.src_stride[side]);
    }
  }
  // Magnitude bits of the wave's largest finite value; `any`: it has others, too. (An old scale that
  // stays and is no power of two adds to it, in store.)
  __device__ __forceinline__ uint32_t top() {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[i][j] & 0x7fff7fffu));
    uint32_t all = wave_max(max(uint32_t(m[0]), uint32_t(m[1])));
    any = all >= 0x7f80u;
    if (any) {
      all = 0;
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) all = max(all, finite2(x[i][j]));
      all = wave_max(all);
    }
    return all;
  }
  __device__ __forceinline__ void store(const WriteParams& p, int side, const Item& it, int h, int t,
                                        uint32_t top) {
    const float scale = fmaxf(need_scale<KIND>(top), old);
    const float inv = 1.0f / scale;  // exact for powers of two
    uint8_t* const page = p.dst[side] + it.page * (side ? p.c.v_page : p.c.k_page) +
                          ((int64_t(h) << p.c.page_shift) * D);
    if (old != scale) {  // earlier tokens of a page whose scale grew
      const float ratio = old * inv;
      for (int i = t; i < it.a * (D / 4); i += 64 * WAVES) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(page) + i;
        float y[4];
        decode4<KIND>(*w, y);
        *w = encode4_any<KIND>(y[0], y[1], y[2], y[3], ratio);
      }
    }
    if (t == 0) p.scale[side][int64_t(it.page) * p.c.H + h] = scale;
    any |= (__float_as_uint(scale) & 0x007fffffu) != 0;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = (t >> 4) + i * 4 * WAVES;
      if (r < it.z - it.a) {
        float y[8];
        unpack8_bf16(x[i], y);
        *reinterpret_cast<u32x2*>(page + (it.a + r) * D + (t & 15) * 8) =
            any ? u32x2{encode4_any<KIND>(y[0], y[1], y[2], y[3], inv),
                        encode4_any<KIND>(y[4], y[5], y[6], y[7], inv)}
                : u32x2{encode4<KIND>(y[0], y[1], y[2], y[3], inv),
                        encode4<KIND>(y[4], y[5], y[6], y[7], inv)};
      }
    }
  }
};

// A side of a (page, head) by a workgroup, both sides by a wave.
template <int KIND, int PASSES>
__device__ __forceinline__ void write_page(const WriteParams& p, int side, const Item& it, int h,
                                           uint32_t (&tops)[4]) {
  Rows<KIND, 4, PASSES> rows;
  rows.load(p, side, it, h, threadIdx.x);
  const uint32_t top = rows.top();
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  rows.store(p, side, it, h, threadIdx.x, max(max(tops[0], tops[1]), max(tops[2], tops[3])));
}
template <int KIND, int PASSES>
__device__ __forceinline__ void write_few(const WriteParams& p, const Item& it, int h, int lane) {
  Rows<KIND, 1, PASSES> k, v;
  k.load(p, 0, it, h, lane);
  v.load(p, 1, it, h, lane);
  k.store(p, 0, it, h, lane, k.top());
  v.store(p, 1, it, h, lane, v.top());
}

// A workgroup per (page, head, side).
template <int KIND, int PASSES>
__global__ __launch_bounds__(kThreads) void write_kernel(WriteParams p) {
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x & 63, side = blockIdx.y & 1, h = blockIdx.y >> 1;
  const Item it = find_item(p.c, blockIdx.x, p.per_seq_items, p.c.page_shift, lane);
  if (it.page < 0) return;  // the same for all waves
  write_page<KIND, PASSES>(p, side, it, h, tops);
}
// Few tokens: a wave per (page, head), both sides.
template <int KIND, int PASSES>
__global__ __launch_bounds__(kThreads) void write_few_kernel(WriteParams p) {
  const int lane = threadIdx.x & 63;
  const int h = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (h >= p.c.H) return;
  const Item it = find_item(p.c, blockIdx.x, p.per_seq_items, p.c.page_shift, lane);
  if (it.page < 0) return;
  write_few<KIND, PASSES>(p, it, h, lane);
}
// Single tokens and drafts beside documents: four heads by a workgroup, in either way.
template <int KIND, int PASSES>
__global__ __launch_bounds__(kThreads) void write_mixed_kernel(WriteParams p) {
  __shared__ uint32_t tops[2][4];
  const int lane = threadIdx.x & 63, h0 = blockIdx.y * 4, heads = min(p.c.H - h0, 4);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Item it = find_item(p.c, blockIdx.x, p.per_seq_items, p.c.page_shift, lane);
  if (it.page < 0) return;  // the same for all waves, as is what follows
  if (it.z - it.a <= 16) {
    if (wave < heads) write_few<KIND, 4>(p, it, h0 + wave, lane);
    return;
  }
  for (int i = 0; i < 2 * heads; ++i)
    write_page<KIND, PASSES>(p, i & 1, it, h0 + (i >> 1), tops[i & 1]);
}

// Rows (head, slot) of a unit; a workgroup takes kReadRows of them, a
// row by 16 lanes of 8 codes, so that a wave's loads and stores are whole lines. Non-temporal
// stores of few rows per workgroup: 16384 tokens of 8 heads 17.5 us, 5.8 TB/s (with 8 lanes to a row
// 29.6 us, ordinary stores of 256 rows 27.5, non-temporal ones 21.7, of 128 rows 19.1).
constexpr int kReadRows = 64;
constexpr int kReadPasses = kReadRows / 16;
template <int KIND>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadParams p) {
  const int lane = threadIdx.x & 63, side = blockIdx.z;
  const Item it = find_item(p.c, blockIdx.x, p.per_seq_items, p.shift, lane);
  if (it.z == it.a) return;
  const int most = p.c.H << p.shift;
  const uint8_t* const page = (side ? p.c.v + max(it.page, 0) * p.c.v_page
                                    : p.c.k + max(it.page, 0) * p.c.k_page);
  const float* const scales = (side ? p.c.v_scale : p.c.k_scale) + int64_t(max(it.page, 0)) * p.c.H;
  const int ch = (threadIdx.x & 15) * 8, r0 = blockIdx.y * kReadRows + (threadIdx.x >> 4);
  u32x2 w[kReadPasses];
  float scale[kReadPasses];
#pragma unroll
  for (int i = 0; i < kReadPasses; ++i) {
    const int r = r0 + i * 16, h = r >> p.shift, slot = it.at + (r & ((1 << p.shift) - 1));
    w[i] = u32x2{0u, 0u};
    scale[i] = 0.0f;
    if (it.page >= 0 && r < most && slot >= it.a && slot < it.z) {
      w[i] = *reinterpret_cast<const u32x2*>(
          page + ((int64_t(h) << p.c.page_shift) + slot) * D + ch);
      scale[i] = scales[h];
    }
  }
#pragma unroll
  for (int i = 0; i < kReadPasses; ++i) {
    const int r = r0 + i * 16, h = r >> p.shift, slot = it.at + (r & ((1 << p.shift) - 1));
    if (r >= most || slot < it.a || slot >= it.z) continue;
    float x[4], y[4];
    whole(w[i]);
    decode4<KIND>(w[i][0], x);
    decode4<KIND>(w[i][1], y);
    const float f = scale[i];
    const u32x4_u o = u32x4{pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                            pack_bf16x2(y[0] * f, y[1] * f), pack_bf16x2(y[2] * f, y[3] * f)};
    uint16_t* const dst = p.dst[side] + (it.row + slot - it.a) * p.dst_stride[side] + h * D + ch;
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4_u*>(dst));
  }
}

// Work items (see find_seq) of units of 1 << shift tokens, 0: more than a launch takes.
int64_t count_items(const CacheView& c, int32_t shift, int32_t* per_seq) {
  const int64_t U = int64_t(1) << shift;
  *per_seq = int32_t((c.per_seq + U - 2) / U + 1);
  const int64_t n = c.cu ? c.total / U + 2 * int64_t(c.n_seqs) : int64_t(c.n_seqs) * *per_seq;
  return n <= kMaxGrid ? n : 0;
}

template <int KIND>
hipError_t launch_write(const WriteParams& p, unsigned items, hipStream_t stream) {
  const int P = 1 << p.c.page_shift;
  const int most = p.c.cu ? P : (p.c.per_seq < P ? p.c.per_seq : P);
  const dim3 few(items, (p.c.H + 3) / 4), grid(items, 2 * p.c.H), block(kThreads);
  // Sequences of at most 16 tokens on the average: most pages get a few. A workgroup for each side of
  // these has little to do, but one that walks a long page of four heads takes 12 us (24 of 256
  // tokens), so that there have to be many (kernels alone, pages of 64 | 256, 8 heads, us, a workgroup
  // per side against this: 64 sequences, a document of 960 tokens among them, 6.4 against 11.9 | 8.0
  // against 24.3; 256 of them 13.7 against 12.8 | 21.5 against 24.7; 512: 23.8 against 14.5 | 31.6
  // against 27.8; 1024 sequences, of which one has 16384 tokens and the others none, 36.6 against
  // 23.3 | 36.0 against 37.8).
  if (p.c.cu && most > 16 && p.c.total <= 16 * int64_t(p.c.n_seqs) &&
      int64_t(p.c.n_seqs) * p.c.H >= (P > 128 ? 4096 : 2048)) {
    if (most <= 64)
      hipLaunchKernelGGL((write_mixed_kernel<KIND, 4>), few, block, 0, stream, p);
    else
      hipLaunchKernelGGL((write_mixed_kernel<KIND, 16>), few, block, 0, stream, p);
  } else if (most <= 4)
    hipLaunchKernelGGL((write_few_kernel<KIND, 1>), few, block, 0, stream, p);
  else if (most <= 16)
    hipLaunchKernelGGL((write_few_kernel<KIND, 4>), few, block, 0, stream, p);
  else if (most <= 64)
    hipLaunchKernelGGL((write_kernel<KIND, 4>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((write_kernel<KIND, 16>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

kda_status check(const CacheArgs& a, CacheView* c) {
  if (a.n_seqs < 0 || a.total_tokens < 0 || a.H < 1 || a.num_pages < 0 || a.table_width < 1)
    return KDA_ERR_BAD_SHAPE;
  if (a.D != D || (a.cache_dtype != KDA_CACHE_FP8 && a.cache_dtype != KDA_CACHE_INT8))
    return KDA_ERR_UNSUPPORTED;
  int32_t shift = 4;
  while (shift < 8 && (1 << shift) < a.page_size) ++shift;
  if ((1 << shift) != a.page_size) return KDA_ERR_UNSUPPORTED;
  if (a.total_tokens > (int64_t(1) << 30) || a.H > kMaxHeads || a.num_pages > INT32_MAX ||
      int64_t(a.table_width) * a.page_size > (int64_t(1) << 28) ||
      int64_t(a.n_seqs) * a.table_width > (int64_t(1) << 35) / a.page_size)
    return KDA_ERR_UNSUPPORTED;
  if (a.total_tokens > 0 && a.n_seqs == 0) return KDA_ERR_BAD_SHAPE;
  if (!a.cu_seqlens && a.n_seqs > 0 && a.total_tokens % a.n_seqs != 0) return KDA_ERR_BAD_SHAPE;
  if (a.table_row_stride < 0 || a.k_page_stride < 0 || a.v_page_stride < 0)
    return KDA_ERR_BAD_STRIDE;
  if (a.total_tokens == 0) return KDA_OK;
  if (!a.page_table || !a.kv_lens) return KDA_ERR_NULL_POINTER;
  if (a.num_pages > 0 && (!a.k_cache || !a.v_cache || !a.k_scale || !a.v_scale))
    return KDA_ERR_NULL_POINTER;
  const int64_t page = int64_t(a.H) * a.page_size * D;
  if (!rows_apart(a.num_pages, a.k_page_stride, page) ||
      !rows_apart(a.num_pages, a.v_page_stride, page) ||
      !rows_apart(a.n_seqs, a.table_row_stride, a.table_width))
    return KDA_ERR_BAD_STRIDE;
  if (((reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache) |
        uint64_t(a.k_page_stride) | uint64_t(a.v_page_stride)) & 15u) != 0)
    return KDA_ERR_UNSUPPORTED;
  c->n_seqs = a.n_seqs;
  c->H = a.H;
  c->total = a.total_tokens;
  c->cu = a.cu_seqlens;
  c->per_seq = a.cu_seqlens ? 0 : int32_t(a.total_tokens / a.n_seqs);
  c->page_shift = shift;
  c->num_pages = int32_t(a.num_pages);
  c->k = static_cast<const uint8_t*>(a.k_cache);
  c->v = static_cast<const uint8_t*>(a.v_cache);
  c->k_page = a.k_page_stride;
  c->v_page = a.v_page_stride;
  c->k_scale = a.k_scale;
  c->v_scale = a.v_scale;
  c->table = a.page_table;
  c->width = a.table_width;
  c->table_stride = a.table_row_stride;
  c->lens = a.kv_lens;
  return KDA_OK;
}

}  // namespace cache
}  // namespace kda

extern "C" kda_status kda_cache_write(
    int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t D, const int32_t* cu_seqlens,
    const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, int32_t cache_dtype,
    int32_t page_size, int64_t num_pages, void* k_cache, int64_t k_page_stride, void* v_cache,
    int64_t v_page_stride, float* k_scale, float* v_scale, const int32_t* page_table,
    int32_t table_width, int64_t table_row_stride, const int32_t* kv_lens, hipStream_t stream) {
  namespace kc = kda::cache;
  kc::WriteParams p;
  const kc::CacheArgs a = {n_seqs,  total_tokens, H, D, cu_seqlens, cache_dtype, page_size,
                           num_pages, k_cache, k_page_stride, v_cache, v_page_stride, k_scale,
                           v_scale, page_table, table_width, table_row_stride, kv_lens};
  if (const kda_status st = kc::check(a, &p.c)) return st;
  if (k_row_stride < 0 || v_row_stride < 0) return KDA_ERR_BAD_STRIDE;
  if (total_tokens == 0) return KDA_OK;
  if (!k || !v) return KDA_ERR_NULL_POINTER;
  const int64_t items = kc::count_items(p.c, p.c.page_shift, &p.per_seq_items);
  if (items == 0) return KDA_ERR_UNSUPPORTED;
  if (num_pages == 0) return KDA_OK;  // no page to write to
  p.src[0] = static_cast<const uint16_t*>(k);
  p.src[1] = static_cast<const uint16_t*>(v);
  p.src_stride[0] = k_row_stride;
  p.src_stride[1] = v_row_stride;
  p.dst[0] = static_cast<uint8_t*>(k_cache);
  p.dst[1] = static_cast<uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  const hipError_t e = cache_dtype == KDA_CACHE_FP8
                           ? kc::launch_write<kc::kFp8>(p, unsigned(items), stream)
                           : kc::launch_write<kc::kInt8>(p, unsigned(items), stream);
  return e == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" kda_status kda_cache_read(
    int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t D, const int32_t* cu_seqlens, void* k,
    int64_t k_row_stride, void* v, int64_t v_row_stride, int32_t cache_dtype, int32_t page_size,
    int64_t num_pages, const void* k_cache, int64_t k_page_stride, const void* v_cache,
    int64_t v_page_stride, const float* k_scale, const float* v_scale, const int32_t* page_table,
    int32_t table_width, int64_t table_row_stride, const int32_t* kv_lens, hipStream_t stream) {
  namespace kc = kda::cache;
  kc::ReadParams p;
  const kc::CacheArgs a = {n_seqs,  total_tokens, H, D, cu_seqlens, cache_dtype, page_size,
                           num_pages, k_cache, k_page_stride, v_cache, v_page_stride, k_scale,
                           v_scale, page_table, table_width, table_row_stride, kv_lens};
  if (const kda_status st = kc::check(a, &p.c)) return st;
  const int64_t row = int64_t(H) * D;
  if (k_row_stride < 0 || v_row_stride < 0 || !kc::rows_apart(total_tokens, k_row_stride, row) ||
      !kc::rows_apart(total_tokens, v_row_stride, row))
    return KDA_ERR_BAD_STRIDE;
  if (total_tokens == 0) return KDA_OK;
  if (!k || !v) return KDA_ERR_NULL_POINTER;
  // Units about as long as a sequence's tokens (1024 single tokens, 8 heads, pages of 64 | 256: 14 |
  // 15 us, by whole pages 39 | 134).
  const int64_t mean = (total_tokens + n_seqs - 1) / n_seqs;
  p.shift = 4;
  while (p.shift < p.c.page_shift && (1 << p.shift) < mean) ++p.shift;
  const int64_t items = kc::count_items(p.c, p.shift, &p.per_seq_items);
  if (items == 0) return KDA_ERR_UNSUPPORTED;
  p.dst[0] = static_cast<uint16_t*>(k);
  p.dst[1] = static_cast<uint16_t*>(v);
  p.dst_stride[0] = k_row_stride;
  p.dst_stride[1] = v_row_stride;
  const unsigned rows = unsigned(H) << p.shift;
  const dim3 grid(unsigned(items), (rows + kc::kReadRows - 1) / kc::kReadRows, 2);
  if (cache_dtype == KDA_CACHE_FP8)
    hipLaunchKernelGGL(kc::read_kernel<kc::kFp8>, grid, dim3(kc::kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(kc::read_kernel<kc::kInt8>, grid, dim3(kc::kThreads), 0, stream, p);
  return hipGetLastError() == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}
