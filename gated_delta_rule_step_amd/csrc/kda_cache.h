// The paged 8-bit cache: parameter block and helpers that its calls share.
#pragma once

#include <limits.h>

#include "../../include/kda_cache.h"
#include "kda_common.h"

namespace kda {
namespace cache {

constexpr int kFp8 = KDA_CACHE_FP8;
constexpr int kInt8 = KDA_CACHE_INT8;
constexpr int32_t kMaxHeads = 1 << 13;
// Workgroups along x: a launch has less than 2^32 threads there, at 256 a workgroup.
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

typedef u32x4 u32x4_u __attribute__((aligned(2)));  // bf16 rows need no alignment of their own
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct CacheView {
  int32_t n_seqs, H;    // H: key/value heads
  int64_t total;        // packed tokens
  const int32_t* cu;    // NULL: per_seq tokens of every sequence
  int32_t per_seq;
  int32_t page_shift;   // page size: 1 << page_shift tokens
  int32_t num_pages;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_page, v_page;  // page strides
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int32_t width;
  int64_t table_stride;
  const int32_t* lens;
};

// A sequence's tokens of this call, packed rows first .. first + n - 1, and its length with
// them (-1: inactive).
struct Seq {
  int64_t first;
  int32_t n, len;
};
__device__ __forceinline__ int32_t clamp_row(const CacheView& p, int32_t x) {
  return min(max(x, 0), int32_t(p.total));
}
__device__ __forceinline__ Seq sequence(const CacheView& p, int32_t b) {
  Seq s;
  const int32_t len = p.lens[b];
  if (p.cu) {
    const int32_t c0 = clamp_row(p, p.cu[b]), c1 = clamp_row(p, p.cu[b + 1]);
    s.first = c0;
    s.n = max(c1 - c0, 0);
  } else {
    s.first = int64_t(b) * p.per_seq;
    s.n = p.per_seq;
  }
  s.len = len < s.n || len > (int64_t(p.width) << p.page_shift) ? -1 : len;
  return s;
}
// The page that holds position `at` >> page_shift == i of sequence b; -1: none.
__device__ __forceinline__ int32_t page_of(const CacheView& p, int32_t b, int32_t i) {
  const int32_t id = p.table[b * p.table_stride + i];
  return uint32_t(id) < uint32_t(p.num_pages) ? id : -1;
}

// Loaded words stay whole up to here. (The compiler else may keep a register for each byte.)
template <typename T>
__device__ __forceinline__ void whole(T& words) {
  asm("" : "+v"(words));
}
// Four codes as two bf16 pairs, exact: e4m3 has 4 significant bits, int8 7.
template <int KIND>
__device__ __forceinline__ u32x2 widen4(uint32_t w) {
  if constexpr (KIND == kFp8) {
    return u32x2{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
  } else {
    return u32x2{pack_bf16x2_exact(float(int8_t(w)), float(int8_t(w >> 8))),
                 pack_bf16x2_exact(float(int8_t(w >> 16)), float(int8_t(w >> 24)))};
  }
}
template <int KIND>
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const u32x2 a = widen4<KIND>(lo), b = widen4<KIND>(hi);
  return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// Bytes of four tokens' words to one word of four tokens per channel.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                           uint32_t (&o)[4]) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u);  // a0 b0 a1 b1
  const uint32_t AB = __builtin_amdgcn_perm(b, a, 0x07030602u);  // a2 b2 a3 b3
  const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x05010400u);
  const uint32_t CD = __builtin_amdgcn_perm(d, c, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(CD, AB, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(CD, AB, 0x07060302u);
}

template <int KIND>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
  if constexpr (KIND == kFp8) {
    const f32x2 a = f8x2_lo(w), b = f8x2_hi(w);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
  } else {
    x[0] = float(int8_t(w)), x[1] = float(int8_t(w >> 8));
    x[2] = float(int8_t(w >> 16)), x[3] = float(int8_t(w >> 24));
  }
}

// e4m3's NaN codes among four, as the bytes' top bits.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// Leaves the position of these in first[0 .. 3] where none stands before it; the bytes' mask.
__device__ __forceinline__ uint32_t note_nans(uint32_t codes, int32_t* first, int32_t at) {
#pragma unroll
  for (int c = 0; c < 4; ++c) atomicMin(first + c, codes >> (8 * c + 7) & 1 ? at : INT_MAX);
  return (codes >> 7) * 0xffu;
}

__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Inclusive sums over the wave's lanes: prefixes within rows of 16 lanes, then the rows' last
// lanes added to the rows behind them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t dpp_add(int32_t x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int32_t wave_prefix(int32_t x) {
  x = dpp_add<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);  // row_bcast 15 into rows 1 and 3
  x = dpp_add<0x143, 0xc>(x);  // row_bcast 31 into rows 2 and 3
  return x;
}

// Host: the checks that the calls share, and the view (left alone where there are no tokens).
struct CacheArgs {
  int32_t n_seqs;
  int64_t total_tokens;
  int32_t H, D;
  const int32_t* cu_seqlens;
  int32_t cache_dtype, page_size;
  int64_t num_pages;
  const void* k_cache;
  int64_t k_page_stride;
  const void* v_cache;
  int64_t v_page_stride;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  int32_t table_width;
  int64_t table_row_stride;
  const int32_t* kv_lens;
};
kda_status check(const CacheArgs& a, CacheView* view);
// Rows of `len` elements do not overlap.
inline bool rows_apart(int64_t rows, int64_t stride, int64_t len) {
  return rows <= 1 || stride >= len;
}

}  // namespace cache
}  // namespace kda
