// RMS norms of a KDA layer and their gradients (gfx950): residual addition,
// norm, sigmoid gate, bf16 or fp8 e4m3 output with scales.
//
// Per (row, head) vector of n channels, with z = x + residual:
//   s = 1 / sqrt(sum z^2 / n + eps),  y = z s w [sigmoid(gate)]
// and, for the gradient, with a = dy w [sigmoid(gate)]:
//   dz = s (a - z s^2 (sum a z) / n) [+ d_residual]
//   dw = sum over vectors of dy z s [sigmoid(gate)]
//   dgate = dy z s w sig (1 - sig)
//
// Both are bound by HBM: every tensor passes once, and a few operations per
// element sit far below the vector rate. So a vector is held in registers
// between the reduction and the output (read once), by LPR lanes with NV
// groups of 8 consecutive channels each; the lane count follows the width, so
// that a head's 128 channels take 16 lanes (one DPP row, four vectors per
// wave, no LDS) and a wide row one workgroup. A workgroup walks over several
// vectors and keeps its weights in registers meanwhile.
//
// 16384 rows of 8192 with a residual: 192 us, 5.6 TB/s; 13889 rows of 12 heads of 128 with
// a gate, fp8: 21 us, 5.1 TB/s; one row of 1536: 2.5 us. Gradients: 8208 rows of 8192
// 111 us, 4.9 TB/s; 8208 rows of 64 gated heads of 128 122 us, 5.5 TB/s. (A large copy
// reaches 5.2 TB/s.) The partial rows' sum adds 4 to 5 us.
//
// Rows of odd strides or widths use the same 16-byte accesses: gfx950 takes
// unaligned vector loads and stores from global memory.

#include <float.h>
#include <stdint.h>

#include "../../include/kda_norm.h"
#include "kda_common.h"

namespace kda {
namespace {

typedef u32x4 u32x4_u __attribute__((aligned(1)));
typedef u32x2 u32x2_u __attribute__((aligned(1)));
typedef uint32_t u32_u __attribute__((aligned(1)));
typedef uint16_t u16_u __attribute__((aligned(1)));

constexpr int kOutBf16 = 0;
constexpr int kOutFp8 = 1;       // one scale per vector
constexpr int kOutFp8Group = 2;  // one scale per 128 channels

struct NormParams {
  int64_t vecs;  // rows * heads
  int32_t heads, width;
  const uint16_t* x;
  const uint16_t* res;
  uint16_t* res_out;
  const uint16_t* gate;
  const float* weight;
  float eps;
  void* out;
  float* scales;
  int64_t x_stride, res_stride, res_out_stride, gate_stride, out_stride, scales_stride;
};

struct NormBwdParams {
  int64_t vecs;
  int32_t heads, width;
  const uint16_t* z;
  const uint16_t* dy;
  const uint16_t* gate;
  const uint16_t* dres;
  const float* weight;
  float eps;
  uint16_t* dz;
  uint16_t* dgate;
  float* partial;  // [blocks][width], or NULL
  int64_t z_stride, dy_stride, gate_stride, dres_stride, dz_stride, dgate_stride;
};

// 8 channels from c on, to be put right by `own8` once they are used: no lane waits behind a
// branch, those at the end take the vector's last 8 channels. (Against a partial group read
// channel by channel, us: 16384 rows of 2500 100.6 and 63.2, of 8191 262 and 236, their
// gradient 259 and 179.) In place, another lane may have stored some of them by then: those
// are the ones that are shifted out.
__device__ __forceinline__ u32x4 load_ch8(const uint16_t* row, int c, int width) {
  if (width >= 8) return *reinterpret_cast<const u32x4_u*>(row + min(c, width - 8));
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (c + i < width) w[i >> 1] |= uint32_t(row[c + i]) << (16 * (i & 1));
  return w;
}
// Shifts out the channels of other groups; channels past the width become zeros. CAP: what
// the lanes hold in all.
template <int CAP>
__device__ __forceinline__ u32x4 own8(u32x4 w, int c, int width) {
  if (width == CAP || width < 8) return w;
  uint64_t lo = uint64_t(w[1]) << 32 | w[0], hi = uint64_t(w[3]) << 32 | w[2];
  const int over = -width & 7;  // channels that the last group lacks
  if (over != 0) {
    const bool last = c == (width & ~7);
    const uint64_t l =
        over < 4 ? lo >> (16 * over) | hi << (64 - 16 * over) : hi >> (16 * over - 64);
    const uint64_t h = over < 4 ? hi >> (16 * over) : 0;
    lo = last ? l : lo;
    hi = last ? h : hi;
  }
  if (c >= width) lo = hi = 0;
  return u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
}
// The last, partial group leaves in pieces of 4, 2 and 1.
__device__ __forceinline__ void store_ch8(uint16_t* row, int c, int width, u32x4 w) {
  if (c + 8 <= width) {
    *reinterpret_cast<u32x4_u*>(row + c) = w;
  } else if (c < width) {
    const int four = width & 4, two = width & 2;
    if (four) *reinterpret_cast<u32x2_u*>(row + c) = u32x2{w[0], w[1]};
    const uint32_t a = four ? w[2] : w[0], b = four ? w[3] : w[1];
    if (two) *reinterpret_cast<u32_u*>(row + c + four) = a;
    if (width & 1) row[c + four + two] = uint16_t(two ? b : a);
  }
}
__device__ __forceinline__ void store_ch8(uint8_t* row, int c, int width, u32x2 w) {
  if (c + 8 <= width) {
    *reinterpret_cast<u32x2_u*>(row + c) = w;
  } else if (c < width) {
    const int four = width & 4, two = width & 2;
    if (four) *reinterpret_cast<u32_u*>(row + c) = w[0];
    const uint32_t a = four ? w[1] : w[0];
    if (two) *reinterpret_cast<u16_u*>(row + c + four) = uint16_t(a);
    if (width & 1) row[c + four + two] = uint8_t(two ? a >> 16 : a);
  }
}
// 8 weights from c on, zeros past the width.
__device__ __forceinline__ void load_w8(const float* w, int c, int width, float (&x)[8]) {
  typedef f32x4 f32x4_u __attribute__((aligned(4)));
  if (c + 8 <= width) {
    const f32x4 a = *reinterpret_cast<const f32x4_u*>(w + c);
    const f32x4 b = *reinterpret_cast<const f32x4_u*>(w + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = c + i < width ? w[c + i] : 0.f;
}
__device__ __forceinline__ u32x4 pack8(const float (&y)[8]) {
  return u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
               pack_bf16x2(y[6], y[7])};
}
// Four values scaled so that the largest of their group is 448: within the format up to a
// rounding of fp32, which the conversion rounds away, so nothing needs to be clamped and a
// NaN stays one.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true));
}
// With the hardware reciprocal (1 ulp): the per-head norm is bound by vector instructions
// as much as by HBM, and a division takes ten of them.
__device__ __forceinline__ float sigmoid_rcp(float x) {
  return __builtin_amdgcn_rcpf(1.0f + fexp(-x));
}
// The sigmoid and what it lacks of 1, e^-x times it: 1 - sig would leave nothing of it where
// x is large. (e^-x is kept finite: where it would overflow, the sigmoid is 0.)
__device__ __forceinline__ void sigmoid_both(float x, float& sig, float& rest) {
  const float e = fexp(-x);
  sig = __builtin_amdgcn_rcpf(1.0f + e);
  rest = fminf(e, FLT_MAX) * sig;
}

__device__ __forceinline__ float row16_max(float x) {
  x = fmaxf(x, dpp<0xB1>(x));
  x = fmaxf(x, dpp<0x4E>(x));
  x = fmaxf(x, dpp<0x141>(x));
  return fmaxf(x, dpp<0x140>(x));
}

// Reduction over the LPR lanes of a vector; every one of them gets the result.
// Above one wave it goes through `buf` (one float per wave and buffer) with one
// barrier: the caller alternates `buf` between two arrays, so that a wave still
// reading one of them is a barrier ahead of its next use.
template <int LPR, bool MAX>
__device__ __forceinline__ float reduce(float x, float* buf) {
  x = MAX ? row16_max(x) : row16_sum(x);
  if constexpr (LPR >= 64) {
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {
      const float y = __shfl_xor(x, o);
      x = MAX ? fmaxf(x, y) : x + y;
    }
  }
  if constexpr (LPR > 64) {
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    x = buf[0];
#pragma unroll
    for (int w = 1; w < LPR / 64; ++w) x = MAX ? fmaxf(x, buf[w]) : x + buf[w];
  }
  return x;
}

// Threads of a workgroup: LPR lanes per vector, at least four waves. W: the width where it is
// known, that of a head (13889 x 12 heads, gate, fp8: 22.3 us without, 21.1 with).
template <int LPR>
constexpr int kNormThreads = LPR > 256 ? LPR : 256;

template <int LPR, int NV, int W, bool RES, bool GATE, int OUT>
__global__ __launch_bounds__(kNormThreads<LPR>) void rmsnorm_kernel(NormParams p) {
  constexpr int T = kNormThreads<LPR>;
  constexpr int VPB = T / LPR;  // vectors of a workgroup at a time
  constexpr int CAP = LPR * NV * 8;
  __shared__ float buf[4][T / 64];
  const int lane = threadIdx.x % LPR;
  const int width = W ? W : p.width;
  const float inv_n = 1.0f / float(width);

  float w[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_w8(p.weight, (j * LPR + lane) * 8, width, w[j]);

  int turn = 0;
  for (int64_t v = int64_t(blockIdx.x) * VPB + threadIdx.x / LPR; v < p.vecs;
       v += int64_t(gridDim.x) * VPB, turn ^= 1) {
    const int64_t r = p.heads == 1 ? v : v / p.heads;
    const int64_t h0 = p.heads == 1 ? 0 : (v - r * p.heads) * width;
    u32x4 xw[NV], rw[NV], gw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      xw[j] = load_ch8(p.x + r * p.x_stride + h0, c, width);
      if constexpr (RES) rw[j] = load_ch8(p.res + r * p.res_stride + h0, c, width);
      if constexpr (GATE) gw[j] = load_ch8(p.gate + r * p.gate_stride + h0, c, width);
    }
    float z[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack8_bf16(own8<CAP>(xw[j], (j * LPR + lane) * 8, width), z[j]);
      if constexpr (RES) {
        float t[8];
        unpack8_bf16(own8<CAP>(rw[j], (j * LPR + lane) * 8, width), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] += t[i];
        if (p.res_out)
          store_ch8(p.res_out + r * p.res_out_stride + h0, (j * LPR + lane) * 8, width,
                    pack8(z[j]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(z[j][i], z[j][i], ss);
    }
    ss = reduce<LPR, false>(ss, buf[turn]);
    const float s = __builtin_amdgcn_rsqf(fmaf(ss, inv_n, p.eps));
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float t[8];
      if constexpr (GATE) unpack8_bf16(own8<CAP>(gw[j], (j * LPR + lane) * 8, width), t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float y = z[j][i] * s * w[j][i];
        if constexpr (GATE) y *= sigmoid_rcp(t[i]);
        z[j][i] = y;
        if constexpr (OUT == kOutFp8) top = fmaxf(top, fabsf(y));
      }
    }
    if constexpr (OUT == kOutBf16) {
      uint16_t* out = static_cast<uint16_t*>(p.out) + r * p.out_stride + h0;
#pragma unroll
      for (int j = 0; j < NV; ++j) store_ch8(out, (j * LPR + lane) * 8, width, pack8(z[j]));
    } else {
      uint8_t* out = static_cast<uint8_t*>(p.out) + r * p.out_stride + h0;
      float* sc = p.scales + r * p.scales_stride;
      if constexpr (OUT == kOutFp8) top = reduce<LPR, true>(top, buf[2 + turn]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + lane) * 8;
        if constexpr (OUT == kOutFp8Group) {  // 16 lanes hold a group's 128 channels
          top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(z[j][i]));
          top = row16_max(top);
        }
        const bool some = top >= 1e-30f;
        const float mul = some ? 448.0f / top : 1.0f;
        const float scale = some ? top * (1.0f / 448.0f) : 1.0f;
        if constexpr (OUT == kOutFp8Group) {
          if ((lane & 15) == 0 && c < width) sc[(h0 + c) / 128] = scale;
        } else if (j == 0 && lane == 0) {
          sc[p.heads == 1 ? 0 : v - r * p.heads] = scale;
        }
        store_ch8(out, c, width,
                  u32x2{pack_fp8(z[j][0] * mul, z[j][1] * mul, z[j][2] * mul, z[j][3] * mul),
                        pack_fp8(z[j][4] * mul, z[j][5] * mul, z[j][6] * mul, z[j][7] * mul)});
      }
    }
  }
}

// The gradient. The weights' gradient is summed in registers over the
// vectors a workgroup walks, then over its lane groups in LDS, and leaves as
// one partial row per workgroup; reduce_partials adds those in index order.
template <int LPR, int NV, int W, bool RES, bool GATE>
__global__ __launch_bounds__(kNormThreads<LPR>) void rmsnorm_bwd_kernel(NormBwdParams p) {
  constexpr int T = kNormThreads<LPR>;
  constexpr int VPB = T / LPR;
  constexpr int CAP = LPR * NV * 8;
  __shared__ float buf[4][T / 64];
  __shared__ float fold[VPB > 1 ? VPB * CAP : 1];
  const int lane = threadIdx.x % LPR;
  const int width = W ? W : p.width;
  const float inv_n = 1.0f / float(width);

  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_w8(p.weight, (j * LPR + lane) * 8, width, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }

  int turn = 0;
  for (int64_t v = int64_t(blockIdx.x) * VPB + threadIdx.x / LPR; v < p.vecs;
       v += int64_t(gridDim.x) * VPB, turn ^= 1) {
    const int64_t r = p.heads == 1 ? v : v / p.heads;
    const int64_t h0 = p.heads == 1 ? 0 : (v - r * p.heads) * width;
    u32x4 zw[NV], yw[NV], rw[NV], gw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      zw[j] = load_ch8(p.z + r * p.z_stride + h0, c, width);
      yw[j] = load_ch8(p.dy + r * p.dy_stride + h0, c, width);
      if constexpr (GATE) gw[j] = load_ch8(p.gate + r * p.gate_stride + h0, c, width);
      if constexpr (RES) rw[j] = load_ch8(p.dres + r * p.dres_stride + h0, c, width);
    }
    float ss = 0.f, sa = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float z[8], a[8], g[8];
      const int c = (j * LPR + lane) * 8;
      zw[j] = own8<CAP>(zw[j], c, width);
      yw[j] = own8<CAP>(yw[j], c, width);
      if constexpr (GATE) gw[j] = own8<CAP>(gw[j], c, width);
      if constexpr (RES) rw[j] = own8<CAP>(rw[j], c, width);
      unpack8_bf16(zw[j], z);
      unpack8_bf16(yw[j], a);
      if constexpr (GATE) unpack8_bf16(gw[j], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (GATE) a[i] *= sigmoid_rcp(g[i]);
        ss = fmaf(z[i], z[i], ss);
        sa = fmaf(a[i] * w[j][i], z[i], sa);
      }
    }
    ss = reduce<LPR, false>(ss, buf[turn]);
    sa = reduce<LPR, false>(sa, buf[2 + turn]);
    const float s = __builtin_amdgcn_rsqf(fmaf(ss, inv_n, p.eps));
    const float m = sa * s * s * inv_n;  // mean(a n) s, with n = z s
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      float z[8], y[8], g[8], t[8];
      unpack8_bf16(zw[j], z);
      unpack8_bf16(yw[j], y);
      if constexpr (GATE) unpack8_bf16(gw[j], g);
      if constexpr (RES) unpack8_bf16(rw[j], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = z[i] * s;
        float d = y[i];
        if constexpr (GATE) {
          float sig, rest;
          sigmoid_both(g[i], sig, rest);
          d *= sig;
          g[i] = d * rest * n * w[j][i];
        }
        dw[j][i] = fmaf(d, n, dw[j][i]);
        y[i] = s * fmaf(-m, z[i], d * w[j][i]);
        if constexpr (RES) y[i] += t[i];
      }
      store_ch8(p.dz + r * p.dz_stride + h0, c, width, pack8(y));
      if constexpr (GATE) store_ch8(p.dgate + r * p.dgate_stride + h0, c, width, pack8(g));
    }
  }
  if (!p.partial) return;
  float* part = p.partial + int64_t(blockIdx.x) * width;
  if constexpr (VPB > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        fold[(threadIdx.x / LPR) * CAP + (j * LPR + lane) * 8 + i] = dw[j][i];
    __syncthreads();
    for (int c = threadIdx.x; c < width; c += T) {
      float t = fold[c];
#pragma unroll
      for (int g = 1; g < VPB; ++g) t += fold[g * CAP + c];
      part[c] = t;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * LPR + lane) * 8 + i;
        if (c < width) part[c] = dw[j][i];
      }
  }
}

// dweight[c] = sum over the partial rows: 16 waves take every 16th row of 64
// channels, and their sums meet in LDS in wave order.
__global__ __launch_bounds__(1024) void reduce_partials(const float* partial, int blocks,
                                                        int width, float* dweight) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float t = 0.f;
  if (c < width) {
    int b = wave;
    for (; b + 112 < blocks; b += 128) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = partial[int64_t(b + 16 * i) * width + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) t += x[i];
    }
    for (; b < blocks; b += 16) t += partial[int64_t(b) * width + c];
  }
  sum[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && c < width) {
    t = sum[0][lane];
#pragma unroll
    for (int i = 1; i < 16; ++i) t += sum[i][lane];
    dweight[c] = t;
  }
}

// ---------------------------------------------------------------------------
// host

// The lanes and groups of 8 that hold a vector: the narrowest shape that covers its
// width, or, where there are too few vectors to fill the chip (up to two per CU), the one
// with the most lanes, so that a vector's loads are all in flight at once. One border for the
// norm and its gradient (8192 channels, residual, operands in cache, us, most lanes against fewer:
// 16 rows 3.6 and 3.9, 256 rows 4.7 and 4.9, 512 rows 6.9 and 6.6, 1024 rows 13.2 and 11.9; their
// gradient 9.1 and 9.6, 15.0 and 15.3, 16.5 and 17.6, 21.7 and 22.9; 512 rows of 1000 channels 3.5
// and 3.7, 7.6 and 6.4).
constexpr int64_t kFewVecs = 512;
#define KDA_NORM_SHAPES(F)                        \
  if (width == 128) return F(16, 1, 128);         \
  if (width < 128) return F(16, 1, 0);            \
  if (width <= 512) return F(64, 1, 0);           \
  if (vecs <= kFewVecs) {                         \
    if (width <= 2048) return F(256, 1, 0);       \
    if (width <= 4096) return F(512, 1, 0);       \
    if (width <= 8192) return F(1024, 1, 0);      \
    return F(1024, 2, 0);                         \
  }                                               \
  if (width <= 1024) return F(64, 2, 0);          \
  if (width <= 2048) return F(256, 1, 0);         \
  if (width <= 4096) return F(256, 2, 0);         \
  if (width <= 8192) return F(256, 4, 0);         \
  return F(512, 4, 0)

int vecs_per_block(int64_t vecs, int width) {
#define KDA_NORM_VPB(L, N, W) kNormThreads<L> / L
  KDA_NORM_SHAPES(KDA_NORM_VPB);
#undef KDA_NORM_VPB
}

// Workgroups: every vector at once up to `most`, which fills the chip's
// registers; above it they walk.
unsigned norm_blocks(int64_t vecs, int width, int64_t most) {
  const int64_t vpb = vecs_per_block(vecs, width);
  const int64_t b = (vecs + vpb - 1) / vpb;
  return unsigned(b < most ? b : most);
}
constexpr int64_t kNormBlocks = 2048;
// A workgroup of the gradient leaves a partial row, as much traffic as a vector, so it walks
// at least eight vectors as long as every CU has one (8192 channels with d_residual and the
// weights' sums, us, 512 workgroups against this rule: 512 rows 23.9 and 16.9, 1024 rows 26.3 and
// 23.6, 2048 rows equal; 256 against it: 4096 rows 59.3 and 53.5). Wide rows fill the chip with
// two per CU (8208 rows: 1024 workgroups 122.6, 512 112.0), and so do workgroups of several
// vectors (525,312 gated heads of 128: 133.4 and 124.8). One narrow row per workgroup takes
// four where each still walks 16, up to the width where they meet (without d_residual, two and
// four per CU, 16384 rows | 65536 rows: 1536 channels 41.2 and 33.4 | 183 and 119, 2048 41.3 and
// 38.6 | 187 and 153, 2816 66.3 and 58.2 | 242 and 220, 3000 70.5 and 61.2 | 248 and 238, 3200 69.9
// and 65.7 | 249 and 248, 3328 70.7 and 72.3 | 252 and 259, 4096 76.1 and 88.2 | 281 and 323). With
// 9000 rows, a few more workgroups than two per CU, four take 1 to 5 % more.
int64_t most_bwd_blocks(int width) { return width > 1024 && width <= 3200 ? 1024 : 512; }
unsigned norm_bwd_blocks(int64_t vecs, int width) {
  const int64_t walk = vecs / 16;
  int64_t most = vecs / 8 < 256 ? 256 : vecs / 8 > 512 ? 512 : vecs / 8;
  if (walk > most) most = walk < most_bwd_blocks(width) ? walk : most_bwd_blocks(width);
  return norm_blocks(vecs, width, most);
}

template <int L, int N, int W, bool RES, bool GATE>
hipError_t launch_norm3(const NormParams& p, int out, hipStream_t stream) {
  const dim3 grid(norm_blocks(p.vecs, p.width, kNormBlocks)), block(kNormThreads<L>);
  switch (out) {
    case kOutBf16:
      hipLaunchKernelGGL((rmsnorm_kernel<L, N, W, RES, GATE, kOutBf16>), grid, block, 0, stream, p);
      break;
    case kOutFp8:
      hipLaunchKernelGGL((rmsnorm_kernel<L, N, W, RES, GATE, kOutFp8>), grid, block, 0, stream, p);
      break;
    default:
      hipLaunchKernelGGL((rmsnorm_kernel<L, N, W, RES, GATE, kOutFp8Group>), grid, block, 0, stream,
                         p);
  }
  return hipGetLastError();
}
template <int L, int N, int W>
hipError_t launch_norm2(const NormParams& p, int out, hipStream_t stream) {
  if (p.res)
    return p.gate ? launch_norm3<L, N, W, true, true>(p, out, stream)
                  : launch_norm3<L, N, W, true, false>(p, out, stream);
  return p.gate ? launch_norm3<L, N, W, false, true>(p, out, stream)
                : launch_norm3<L, N, W, false, false>(p, out, stream);
}
hipError_t launch_norm(const NormParams& p, int out, hipStream_t stream) {
  const int width = p.width;
  const int64_t vecs = p.vecs;
#define KDA_NORM_GO(L, N, W) launch_norm2<L, N, W>(p, out, stream)
  KDA_NORM_SHAPES(KDA_NORM_GO);
#undef KDA_NORM_GO
}

template <int L, int N, int W>
hipError_t launch_norm_bwd2(const NormBwdParams& p, hipStream_t stream) {
  const dim3 grid(norm_bwd_blocks(p.vecs, p.width)), block(kNormThreads<L>);
  if (p.dres && p.gate)
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<L, N, W, true, true>), grid, block, 0, stream, p);
  else if (p.dres)
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<L, N, W, true, false>), grid, block, 0, stream, p);
  else if (p.gate)
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<L, N, W, false, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<L, N, W, false, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}
hipError_t launch_norm_bwd(const NormBwdParams& p, hipStream_t stream) {
  const int width = p.width;
  const int64_t vecs = p.vecs;
#define KDA_NORM_GO(L, N, W) launch_norm_bwd2<L, N, W>(p, stream)
  KDA_NORM_SHAPES(KDA_NORM_GO);
#undef KDA_NORM_GO
}

kda_status check_sizes(int64_t rows, int32_t heads, int32_t width, float eps) {
  if (rows < 0 || heads < 1 || width < 1) return KDA_ERR_BAD_SHAPE;
  if (width > KDA_NORM_MAX_WIDTH || int64_t(heads) * width > (int64_t(1) << 30))
    return KDA_ERR_UNSUPPORTED;
  if (rows > (int64_t(1) << 62) / (int64_t(heads) * width)) return KDA_ERR_UNSUPPORTED;
  if (!(eps > 0.0f && eps < INFINITY)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// Rows of `len` elements do not overlap.
bool rows_apart(int64_t rows, int64_t stride, int64_t len) { return rows <= 1 || stride >= len; }

}  // namespace
}  // namespace kda

extern "C" kda_status kda_rmsnorm(int64_t rows, int32_t heads, int32_t width, const void* x,
                                  int64_t x_row_stride, const void* residual,
                                  int64_t residual_row_stride, void* residual_out,
                                  int64_t residual_out_row_stride, const void* gate,
                                  int64_t gate_row_stride, const float* weight, float eps,
                                  int32_t out_dtype, void* out, int64_t out_row_stride,
                                  int32_t scale_group, float* scales, int64_t scales_row_stride,
                                  hipStream_t stream) {
  if (const kda_status st = kda::check_sizes(rows, heads, width, eps)) return st;
  const bool fp8 = out_dtype == KDA_NORM_OUT_FP8;
  if (out_dtype != KDA_NORM_OUT_BF16 && !fp8) return KDA_ERR_UNSUPPORTED;
  const bool whole = scale_group == 0 || scale_group == width;
  if (fp8 && !whole && (scale_group != 128 || width % 128 != 0)) return KDA_ERR_UNSUPPORTED;
  if (residual_out && !residual) return KDA_ERR_UNSUPPORTED;
  if (rows == 0) return KDA_OK;
  if (!x || !weight || !out || (fp8 && !scales)) return KDA_ERR_NULL_POINTER;
  const int64_t W = int64_t(heads) * width;
  if (x_row_stride < 0 || out_row_stride < 0 || (residual && residual_row_stride < 0) ||
      (residual_out && residual_out_row_stride < 0) || (gate && gate_row_stride < 0) ||
      (fp8 && scales_row_stride < 0))
    return KDA_ERR_BAD_STRIDE;
  if (!kda::rows_apart(rows, out_row_stride, W) ||
      (residual_out && !kda::rows_apart(rows, residual_out_row_stride, W)) ||
      (fp8 && !kda::rows_apart(rows, scales_row_stride,
                               int64_t(heads) * (whole ? 1 : width / 128))))
    return KDA_ERR_BAD_STRIDE;

  kda::NormParams p;
  p.vecs = rows * heads;
  p.heads = heads;
  p.width = width;
  p.x = static_cast<const uint16_t*>(x);
  p.res = static_cast<const uint16_t*>(residual);
  p.res_out = static_cast<uint16_t*>(residual_out);
  p.gate = static_cast<const uint16_t*>(gate);
  p.weight = weight;
  p.eps = eps;
  p.out = out;
  p.scales = scales;
  p.x_stride = x_row_stride;
  p.res_stride = residual_row_stride;
  p.res_out_stride = residual_out_row_stride;
  p.gate_stride = gate_row_stride;
  p.out_stride = out_row_stride;
  p.scales_stride = scales_row_stride;
  const int kind = !fp8 ? kda::kOutBf16 : whole ? kda::kOutFp8 : kda::kOutFp8Group;
  return kda::launch_norm(p, kind, stream) == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" size_t kda_rmsnorm_backward_workspace_size(int64_t rows, int32_t heads,
                                                      int32_t width) {
  if (kda::check_sizes(rows, heads, width, 1.0f)) return 0;
  const int64_t vecs = rows * heads;  // (never less for more rows, so that one buffer serves all)
  const int64_t most = kda::most_bwd_blocks(width);
  return size_t(vecs < most ? vecs : most) * size_t(width) * 4;
}

extern "C" kda_status kda_rmsnorm_backward(
    int64_t rows, int32_t heads, int32_t width, const void* z, int64_t z_row_stride,
    const void* dy, int64_t dy_row_stride, const void* gate, int64_t gate_row_stride,
    const void* d_residual, int64_t d_residual_row_stride, const float* weight, float eps,
    void* dz, int64_t dz_row_stride, void* dgate, int64_t dgate_row_stride, float* dweight,
    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (const kda_status st = kda::check_sizes(rows, heads, width, eps)) return st;
  if (rows > 0 && (!z || !dy || !weight || !dz)) return KDA_ERR_NULL_POINTER;
  if ((gate != nullptr) != (dgate != nullptr)) return KDA_ERR_NULL_POINTER;
  const int64_t W = int64_t(heads) * width;
  if (rows > 0) {
    if (z_row_stride < 0 || dy_row_stride < 0 || dz_row_stride < 0 ||
        (gate && (gate_row_stride < 0 || dgate_row_stride < 0)) ||
        (d_residual && d_residual_row_stride < 0))
      return KDA_ERR_BAD_STRIDE;
    if (!kda::rows_apart(rows, dz_row_stride, W) ||
        (gate && !kda::rows_apart(rows, dgate_row_stride, W)))
      return KDA_ERR_BAD_STRIDE;
  }
  const int blocks = int(kda::norm_bwd_blocks(rows * heads, width));
  if (dweight && rows > 0) {
    if (workspace_bytes < size_t(blocks) * size_t(width) * 4) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace) return KDA_ERR_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_UNSUPPORTED;
  }

  kda::NormBwdParams p;
  p.vecs = rows * heads;
  p.heads = heads;
  p.width = width;
  p.z = static_cast<const uint16_t*>(z);
  p.dy = static_cast<const uint16_t*>(dy);
  p.gate = static_cast<const uint16_t*>(gate);
  p.dres = static_cast<const uint16_t*>(d_residual);
  p.weight = weight;
  p.eps = eps;
  p.dz = static_cast<uint16_t*>(dz);
  p.dgate = static_cast<uint16_t*>(dgate);
  p.partial = dweight ? static_cast<float*>(workspace) : nullptr;
  p.z_stride = z_row_stride;
  p.dy_stride = dy_row_stride;
  p.gate_stride = gate_row_stride;
  p.dres_stride = d_residual_row_stride;
  p.dz_stride = dz_row_stride;
  p.dgate_stride = dgate_row_stride;
  if (rows > 0 && kda::launch_norm_bwd(p, stream) != hipSuccess) return KDA_ERR_LAUNCH;
  if (dweight) {
    hipLaunchKernelGGL(kda::reduce_partials, dim3((width + 63) / 64), dim3(1024), 0, stream,
                       p.partial, rows > 0 ? blocks : 0, width, dweight);
    if (hipGetLastError() != hipSuccess) return KDA_ERR_LAUNCH;
  }
  return KDA_OK;
}
