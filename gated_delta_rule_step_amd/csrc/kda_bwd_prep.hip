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

constexpr int PS = C + 8;  // row (fp16) of T and P as MFMA operands

struct PrepSmem {
  float km[C * RS];    // readers: up k; then T and P as operands
  float kb[C * RS];    // writers: beta dn k
  float qm[C * RS];    // up q', then V and dO (bf16)
  float am[C * AS];    // A
  float pm[C * AS];    // P
  float tm[C * AS];    // T
  float pair[NP * D];  // factor of a block pair
  float top[2][8];     // largest magnitudes of W and Z, per wave
  uint32_t ttop, ptop; // of T and P (as bits)
  alignas(16) float rq[C], rk[C], beta[C];
};
// High and low parts, [row][the other index in the order of a right fragment]; blocks
// that a 32-index contraction takes along and that hold nothing are zeros.
struct TPlanes {
  uint16_t t[2][C * PS];   // T
  uint16_t tt[2][C * PS];  // T^T
  uint16_t pt[2][C * PS];  // P^T
};
static_assert(sizeof(TPlanes) <= sizeof(float) * 2 * C * RS, "they fit over km and kb");
// Position of index t among 32: a fragment holds, for lane group g, 4 g .. 4 g + 3 of a
// block of 16 and of the next one.
__device__ __forceinline__ int perm32(int t) {
  return (t & 32) + 8 * ((t & 15) >> 2) + 4 * ((t >> 4) & 1) + (t & 3);
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}
__device__ __forceinline__ float max4(f32x4 x) {
  return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}

constexpr int VS = 2 * RS;  // row of V and dO in uint16: V first, dO from RS on

// 64 tokens of a bf16 column as right fragments, scaled by the column's largest magnitude.
__device__ __forceinline__ void bf16_fragments(const u32x4 (&w)[2], f16x8 (&f)[2], float& un) {
  float x[2][8], top = 0.f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    unpack8_bf16(w[t], x[t]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[t][i]));
  }
  const Scale sc = scale_for(column_max(top));
  un = sc.un;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    u32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack_f16x2(x[t][2 * i] * sc.up, x[t][2 * i + 1] * sc.up);
    f[t] = __builtin_bit_cast(f16x8, h);
  }
}

// Writers' operands carry beta, which may exceed 1 where it is given: a smaller scale.
constexpr float kBetaUp = 16.0f;

__global__ __launch_bounds__(kThreads) void prep_kernel(BwdParams p) {
  extern __shared__ __align__(16) float smem_raw[];
  PrepSmem& s = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int64_t sigma = blockIdx.x;
  const int h = blockIdx.y;
  const Chunk ch = chunk_of(p, sigma);
  if (ch.c == 0 || !ch.active) return;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  if (threadIdx.x == 0) s.ttop = s.ptop = 0;
  if (threadIdx.x < C) tail[kTailBeta + threadIdx.x] = s.beta[threadIdx.x];

  // ---- the decayed rows, and what depends on them channel by channel alone
  // left fragments of e^G k and beta e^(Gl-G) k: channel kc, pairs of token blocks
  f16x8 kgh[2], kgl[2], keh[2], kel[2];
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
    u32x2 half[4];  // of the even block
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float ef = from[b], et = to[b];
      f32x4 qg, kee, kg, ke;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * b + 4 * g4 + i;
        const float up = ln.up[b][i], down = inverse(up);
        const float km = ln.k[b][i] * up, qm = ln.q[b][i] * up * p.scale;
        const float kb = ln.k[b][i] * down * s.beta[t];
        s.km[t * RS + kc] = km;
        s.qm[t * RS + kc] = qm;
        s.kb[t * RS + kc] = kb;
        kg[i] = km * ef;
        qg[i] = ln.q[b][i] * up * ef;
        kee[i] = ln.k[b][i] * down * et;
        ke[i] = kb * et;
      }
      const int at = ((w * 2 + (b >> 1)) * 2 * 64 + lane) * 16 + 8 * (b & 1);
      u32x2 hi, lo;
      split4h(kee * kFixedUp, hi, lo);
      *reinterpret_cast<u32x2*>(ops + kOpKE + at) = hi;
      *reinterpret_cast<u32x2*>(ops + kOpKE + at + 1024) = lo;
      split4h(kg * kFixedUp, hi, lo);
      *reinterpret_cast<u32x2*>(ops + kOpKG + at) = hi;
      *reinterpret_cast<u32x2*>(ops + kOpKG + at + 1024) = lo;
      u32x2 eh, el;
      split4h(ke * kBetaUp, eh, el);
      if (b & 1) {
        kgh[b >> 1] = join8(half[0], hi), kgl[b >> 1] = join8(half[1], lo);
        keh[b >> 1] = join8(half[2], eh), kel[b >> 1] = join8(half[3], el);
      } else {
        half[0] = hi, half[1] = lo, half[2] = eh, half[3] = el;
      }
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
      if (!(over < 0 || (is_p && over == 0))) acc[i] = 0.f;
      dst[i * AS] = acc[i];
    }
    if (is_p) {
      const float top = wave_max(max4(acc));
      if (lane == 0) atomicMax(&s.ptop, __float_as_uint(top));
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
    const float top = wave_max(max4(r));
    if (lane == 0) atomicMax(&s.ttop, __float_as_uint(top));
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
      const float top = wave_max(max4(acc));
      if (lane == 0) atomicMax(&s.ttop, __float_as_uint(top));
    }
  }
  __syncthreads();

  // ---- T, T^T and P^T as operands, over km and kb
  TPlanes& tp = *reinterpret_cast<TPlanes*>(smem_raw);
  const Scale st = scale_for(__uint_as_float(s.ttop)), sp = scale_for(__uint_as_float(s.ptop));
  for (int task = w; task < 30; task += kThreads / 64) {
    const int kind = task / 10;  // T, T^T, P^T
    int I = 0, J = task % 10;
    while (J > I) J -= ++I;
    const float* src = kind == 2 ? s.pm : s.tm;
    const f32x4 x = kind == 0 ? lds4(src + (16 * I + n16) * AS + 16 * J + 4 * g4)
                              : col4(src + (16 * I + 4 * g4) * AS + 16 * J + n16, AS);
    uint16_t(*dst)[C * PS] = kind == 0 ? tp.t : kind == 1 ? tp.tt : tp.pt;
    const int row = 16 * (kind == 0 ? I : J) + n16;
    const int other = 16 * (kind == 0 ? J : I) + 4 * g4;
    u32x2 hi, lo;
    split4h(x * (kind == 2 ? sp.up : st.up), hi, lo);
    *reinterpret_cast<u32x2*>(dst[0] + row * PS + perm32(other)) = hi;
    *reinterpret_cast<u32x2*>(dst[1] + row * PS + perm32(other)) = lo;
    if (I == J) {  // the pair's other block: right of T's even ones, left of the odd transposed
      const bool empty = kind == 0 ? !(I & 1) : (I & 1);
      if (empty) {
        const int at = row * PS + perm32(other ^ 16);
        *reinterpret_cast<u32x2*>(dst[0] + at) = u32x2{0u, 0u};
        *reinterpret_cast<u32x2*>(dst[1] + at) = u32x2{0u, 0u};
      }
    }
  }
  __syncthreads();

  // ---- products with T for the wave's 16 channels
  const uint16_t* vo = reinterpret_cast<const uint16_t*>(s.qm);
  f16x8 vf[2], of[2];  // V and dO: 8 bits, so their high parts are exact
  float unv, uno;
  {
    u32x4 vb[2], ob[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (32 * t + 16 * (i >> 1) + 4 * g4 + 2 * (i & 1)) * VS + kc;
        vb[t][i] = uint32_t(vo[at]) | uint32_t(vo[at + VS]) << 16;
        ob[t][i] = uint32_t(vo[at + RS]) | uint32_t(vo[at + VS + RS]) << 16;
      }
#pragma unroll
    for (int t = 0; t < 2; ++t)
      *reinterpret_cast<u32x4*>(ops + kOpO + ((w * 2 + t) * 64 + lane) * 16) = ob[t];
    bf16_fragments(vb, vf, unv);
    bf16_fragments(ob, of, uno);
  }
  auto frag = [&](const uint16_t* plane, int r, int t) {
    return *reinterpret_cast<const f16x8*>(plane + (16 * r + n16) * PS + 32 * t + 8 * g4);
  };
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
    for (int t = 0; t < 2; ++t) {
      if (t <= r / 2) {
        const f16x8 h = frag(tp.t[0], r, t), l = frag(tp.t[1], r, t);
        wt[r] = mfma_split(kgh[t], kgl[t], h, l, wt[r]);  // transposed: rows are channels
        xx = mfma32(l, vf[t], xx);
        xx = mfma32(h, vf[t], xx);
      }
      if (t >= r / 2) {
        z[r] = mfma_split(keh[t], kel[t], frag(tp.tt[0], r, t), frag(tp.tt[1], r, t), z[r]);
        y[r] = mfma32(frag(tp.pt[1], r, t), of[t], y[r]);
        y[r] = mfma32(frag(tp.pt[0], r, t), of[t], y[r]);
      }
    }
    *reinterpret_cast<f32x4*>(X + ((w * NB + r) * 64 + lane) * 4) = xx * (unv * st.un);
    wtop = fmaxf(wtop, max4(wt[r]));
    ztop = fmaxf(ztop, max4(z[r]));
  }
  wtop = wave_max(wtop);
  ztop = wave_max(ztop);
  if (lane == 0) {
    s.top[0][w] = wtop;
    s.top[1][w] = ztop;
  }
  {
    float top = 0.f;
#pragma unroll
    for (int r = 0; r < NB; ++r) top = fmaxf(top, max4(y[r]));
    const Scale sy = scale_for(column_max(top));
    f16x8 yh[2], yl[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u32x2 h0, l0, h1, l1;
      split4h(y[2 * t] * sy.up, h0, l0);
      split4h(y[2 * t + 1] * sy.up, h1, l1);
      yh[t] = join8(h0, h1);
      yl[t] = join8(l0, l1);
    }
    const float un = (sp.un * uno) * (st.un * sy.un);
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      f32x4 d = zero4();
#pragma unroll
      for (int t = r / 2; t < 2; ++t)
        d = mfma_split(frag(tp.tt[0], r, t), frag(tp.tt[1], r, t), yh[t], yl[t], d);
      *reinterpret_cast<f32x4*>(DV + ((w * NB + r) * 64 + lane) * 4) = d * un;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wtop = fmaxf(wtop, s.top[0][i]);
    ztop = fmaxf(ztop, s.top[1][i]);
  }
  const Scale sw = scale_for(wtop), sz = scale_for(ztop);
  if (threadIdx.x == 0) {
    tail[kTailUnW] = sw.un * (st.un * kFixedUn);
    tail[kTailUnZ] = sz.un * (st.un / kBetaUp);
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
