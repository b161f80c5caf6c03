// Prefill gradient, preparation (gfx950): everything of a 64-token chunk that depends
// neither on the state entering it nor on the state gradient leaving it, for all chunks
// and heads at once. The method is described in kda_backward.hip.

#include "kda_bwd.h"

namespace kda {
namespace bwd {
namespace {

// ---------------------------------------------------------------------------
// Preparation: one workgroup per (chunk, head); a wave owns 16 channels.
constexpr int RS = D + 4;  // padded row (fp32) of [token][channel] LDS arrays
constexpr int AS = C + 4;  // padded row of [token][token] LDS arrays

// Pairs of different blocks, I > J.
__host__ __device__ constexpr int pair_index(int I, int J) { return I * (I - 1) / 2 + J; }

struct PrepSmem {
  float km[C * RS];    // readers: up k
  float kb[C * RS];    // writers: beta dn k
  float qm[C * RS];    // up q', then V and dO (bf16)
  float am[C * AS];    // A
  float pm[C * AS];    // P
  float tm[C * AS];    // T
  float pair[NP * D];  // factor of a block pair
  float top[2][8];     // largest magnitudes of W and Z, per wave
  alignas(16) float rq[C], rk[C], beta[C];
};
constexpr int VS = 2 * RS;  // row of V and dO in uint16: V first, dO from RS on

__global__ __launch_bounds__(kThreads) void prep_kernel(BwdParams p) {
  extern __shared__ __align__(16) float smem_raw[];
  PrepSmem& s = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int64_t sigma = blockIdx.x;
  const int h = blockIdx.y;
  const Chunk ch = chunk_of(p, sigma);
  if (ch.c == 0 || !ch.active) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int kc = 16 * w + n16;
  uint8_t* ops = p.ops + (sigma * p.H + h) * int64_t(kOps);
  float* tail = reinterpret_cast<float*>(ops + kOpTail);

  RawLane raw;
  load_lane(p, ch, h, kc, g4, raw);
  token_scalars(p, ch, h, s.rq, s.rk, s.beta);
  u32x4 vw[C / (kThreads / 16)], ow[C / (kThreads / 16)];  // V and dO, written to LDS below
  const Rows vr = rows_of(p.v, ch, p.v_stride, int64_t(h) * D);
  const Rows orow = rows_of(p.dout, ch, p.dout_stride, int64_t(h) * D);
#pragma unroll
  for (int j = 0; j < C / (kThreads / 16); ++j) {
    const int t = min(int(threadIdx.x >> 4) + j * (kThreads / 16), ch.c - 1);
    vw[j] = *reinterpret_cast<const u32x4_u*>(vr.at(t, (threadIdx.x & 15) * 8));
    ow[j] = *reinterpret_cast<const u32x4_u*>(orow.at(t, (threadIdx.x & 15) * 8));
  }
  __syncthreads();
  if (threadIdx.x < C) tail[kTailBeta + threadIdx.x] = s.beta[threadIdx.x];

  // ---- the decayed rows, and what depends on them channel by channel alone
  f32x4 kg[NB], ke[NB];  // e^G k, beta e^(Gl-G) k: 4 tokens of channel kc
  {
    Lane ln;
    make_lane<false>(p, ch, h, kc, g4, raw, s.rq, s.rk, ln, nullptr);
    float from[NB], to[NB];  // from the chunk's start to the block's middle, to its end
    float o = 1.f, e = 1.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      from[b] = o * ln.head[b];
      o *= ln.head[b] * ln.tail[b];
    }
#pragma unroll
    for (int b = NB - 1; b >= 0; --b) {
      to[b] = e * ln.tail[b];
      e *= ln.head[b] * ln.tail[b];
    }
    if (g4 == 0) {
      tail[kc] = o;
#pragma unroll
      for (int I = 1; I < NB; ++I) {
        float mid = ln.head[I];
#pragma unroll
        for (int J = I - 1; J >= 0; --J) {
          s.pair[pair_index(I, J) * D + kc] = mid * ln.tail[J];
          mid *= ln.head[J] * ln.tail[J];
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float ef = from[b], et = to[b];
      f32x4 qg, kee;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * b + 4 * g4 + i;
        const float up = ln.up[b][i], down = inverse(up);
        const float km = ln.k[b][i] * up, qm = ln.q[b][i] * up * p.scale;
        const float kb = ln.k[b][i] * down * s.beta[t];
        s.km[t * RS + kc] = km;
        s.qm[t * RS + kc] = qm;
        s.kb[t * RS + kc] = kb;
        kg[b][i] = km * ef;
        qg[i] = ln.q[b][i] * up * ef;
        kee[i] = ln.k[b][i] * down * et;
        ke[b][i] = kb * et;
      }
      const int at = ((w * 2 + (b >> 1)) * 2 * 64 + lane) * 16 + 8 * (b & 1);
      u32x2 hi, lo;
      split4h(kee * kFixedUp, hi, lo);
      *reinterpret_cast<u32x2*>(ops + kOpKE + at) = hi;
      *reinterpret_cast<u32x2*>(ops + kOpKE + at + 1024) = lo;
      split4h(kg[b] * kFixedUp, hi, lo);
      *reinterpret_cast<u32x2*>(ops + kOpKG + at) = hi;
      *reinterpret_cast<u32x2*>(ops + kOpKG + at + 1024) = lo;
      split4h(qg * kFixedUp, hi, lo);
      *reinterpret_cast<u32x2*>(ops + kOpQG + at) = hi;
      *reinterpret_cast<u32x2*>(ops + kOpQG + at + 1024) = lo;
    }
  }
  __syncthreads();

  // ---- A and P, block by block (10 each on and below the diagonal)
  for (int task = w; task < NB * (NB + 1); task += kThreads / 64) {
    const bool is_p = task >= NB * (NB + 1) / 2;
    int I = 0, J = is_p ? task - NB * (NB + 1) / 2 : task;
    while (J > I) J -= ++I;
    const float* left = (is_p ? s.qm : s.km) + (16 * I + n16) * RS + 4 * g4;
    const float* right = s.kb + (16 * J + n16) * RS + 4 * g4;
    f32x4 acc = zero4();
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
      f32x4 a = lds4(left + 16 * m);
      if (I != J) a *= lds4(s.pair + pair_index(I, J) * D + 16 * m + 4 * g4);
      acc = mfma4(a, lds4(right + 16 * m), acc);
    }
    float* dst = (is_p ? s.pm : s.am) + (16 * I + 4 * g4) * AS + 16 * J + n16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int over = I == J ? n16 - (4 * g4 + i) : -1;  // column beyond the row
      dst[i * AS] = over < 0 || (is_p && over == 0) ? acc[i] : 0.f;
    }
  }
  __syncthreads();

  // ---- T = (1 + A)^-1. Diagonal blocks: N = -A is strictly lower, N^16 = 0, so
  // the inverse is (1 + N)(1 + N^2)(1 + N^4)(1 + N^8). A product X Y takes X^T as
  // its left fragment, so every power is kept with its transpose.
  if (w < NB) {
    const float* a = s.am + 16 * w * AS + 16 * w;
    f32x4 n = -col4(a + 4 * g4 * AS + n16, AS), nt = -lds4(a + n16 * AS + 4 * g4);
    f32x4 r = n, rt = nt;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float one = 4 * g4 + i == n16 ? 1.f : 0.f;
      r[i] += one;
      rt[i] += one;
    }
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      const f32x4 n2 = mfma4(nt, n, zero4()), n2t = mfma4(n, nt, zero4());
      const f32x4 r2 = mfma4(rt, n2, r), r2t = mfma4(n2, rt, rt);
      n = n2, nt = n2t, r = r2, rt = r2t;
    }
    float* dst = s.tm + (16 * w + 4 * g4) * AS + 16 * w + n16;
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i * AS] = r[i];
  }
  // V and dO (bf16) take the place of up q'
  {
    uint16_t* vo = reinterpret_cast<uint16_t*>(s.qm);
    const int c0 = (threadIdx.x & 15) * 8;
#pragma unroll
    for (int j = 0; j < C / (kThreads / 16); ++j) {
      const int t = (threadIdx.x >> 4) + j * (kThreads / 16);
      if (t >= ch.c) vw[j] = ow[j] = u32x4{0u, 0u, 0u, 0u};
      typedef u32x4 u32x4_8 __attribute__((aligned(8)));
      *reinterpret_cast<u32x4_8*>(vo + t * VS + c0) = vw[j];
      *reinterpret_cast<u32x4_8*>(vo + t * VS + RS + c0) = ow[j];
    }
  }
  __syncthreads();
  // T_IJ = -T_II sum_K A_IK T_KJ, one wave per block column
  if (w < NB - 1) {
    f32x4 t[NB];
    t[0] = col4(s.tm + (16 * w + 4 * g4) * AS + 16 * w + n16, AS);
    for (int I = w + 1; I < NB; ++I) {
      f32x4 acc = zero4();
#pragma unroll
      for (int d = 0; d < NB - 1; ++d)
        if (w + d < I) acc = mfma4(lds4(s.am + (16 * I + n16) * AS + 16 * (w + d) + 4 * g4), t[d], acc);
      acc = mfma4(lds4(s.tm + (16 * I + n16) * AS + 16 * I + 4 * g4), -acc, zero4());
#pragma unroll
      for (int d = 1; d < NB; ++d)
        if (w + d == I) t[d] = acc;
      float* dst = s.tm + (16 * I + 4 * g4) * AS + 16 * w + n16;
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i * AS] = acc[i];
    }
  }
  __syncthreads();

  // ---- products with T for the wave's 16 channels
  const uint16_t* vo = reinterpret_cast<const uint16_t*>(s.qm);
  f32x4 vv[NB], oo[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * b + 4 * g4 + i;
      vv[b][i] = bf1(vo[t * VS + kc]);
      oo[b][i] = bf1(vo[t * VS + RS + kc]);
    }
  f32x4 y[NB];  // P^T dO
  f32x4 wt[NB], z[NB];
  float wtop = 0.f, ztop = 0.f;
  float* X = reinterpret_cast<float*>(ops + kOpX0);
  float* DV = reinterpret_cast<float*>(ops + kOpDV0);
#pragma unroll
  for (int r = 0; r < NB; ++r) {
    f32x4 xx = zero4();
    wt[r] = z[r] = y[r] = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b <= r) {
        const f32x4 t = lds4(s.tm + (16 * r + n16) * AS + 16 * b + 4 * g4);
        wt[r] = mfma4(kg[b], t, wt[r]);  // transposed: rows are channels
        xx = mfma4(t, vv[b], xx);
      }
      if (b >= r) {
        const int at = (16 * b + 4 * g4) * AS + 16 * r + n16;
        z[r] = mfma4(ke[b], col4(s.tm + at, AS), z[r]);  // transposed
        y[r] = mfma4(col4(s.pm + at, AS), oo[b], y[r]);
      }
    }
    *reinterpret_cast<f32x4*>(X + ((w * NB + r) * 64 + lane) * 4) = xx;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wtop = fmaxf(wtop, fabsf(wt[r][i]));
      ztop = fmaxf(ztop, fabsf(z[r][i]));
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    wtop = fmaxf(wtop, __shfl_xor(wtop, o));
    ztop = fmaxf(ztop, __shfl_xor(ztop, o));
  }
  if (lane == 0) {
    s.top[0][w] = wtop;
    s.top[1][w] = ztop;
  }
#pragma unroll
  for (int r = 0; r < NB; ++r) {
    f32x4 d = zero4();
#pragma unroll
    for (int b = r; b < NB; ++b)
      d = mfma4(col4(s.tm + (16 * b + 4 * g4) * AS + 16 * r + n16, AS), y[b], d);
    *reinterpret_cast<f32x4*>(DV + ((w * NB + r) * 64 + lane) * 4) = d;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wtop = fmaxf(wtop, s.top[0][i]);
    ztop = fmaxf(ztop, s.top[1][i]);
  }
  const Scale sw = scale_for(wtop), sz = scale_for(ztop);
  if (threadIdx.x == 0) {
    tail[kTailUnW] = sw.un;
    tail[kTailUnZ] = sz.un;
  }
#pragma unroll
  for (int r = 0; r < NB; ++r) {
    const int at = ((r * 4 + (w >> 1)) * 2 * 64 + lane) * 16 + 8 * (w & 1);
    u32x2 hi, lo;
    split4h(wt[r] * sw.up, hi, lo);
    *reinterpret_cast<u32x2*>(ops + kOpW + at) = hi;
    *reinterpret_cast<u32x2*>(ops + kOpW + at + 1024) = lo;
    split4h(z[r] * sz.up, hi, lo);
    *reinterpret_cast<u32x2*>(ops + kOpZ + at) = hi;
    *reinterpret_cast<u32x2*>(ops + kOpZ + at + 1024) = lo;
  }
}

}  // namespace

hipError_t launch_prep(const BwdParams& p, hipStream_t stream) {
  static const hipError_t lds = hipFuncSetAttribute(
      reinterpret_cast<const void*>(prep_kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
      int(sizeof(PrepSmem)));
  if (lds != hipSuccess) return lds;
  hipLaunchKernelGGL(prep_kernel, dim3(unsigned(p.slots), unsigned(p.H)), dim3(kThreads),
                     sizeof(PrepSmem), stream, p);
  return hipGetLastError();
}

}  // namespace bwd
}  // namespace kda
