// Prefill gradient, gradients (gfx950): those of every input from the states, the state
// gradients, x and dV that the chains left, for all chunks and heads at once. The method
// is described in kda_backward.hip.

#include "kda_bwd.h"

namespace kda {
namespace bwd {
namespace {

// Gradients: one workgroup per (chunk, head); a wave owns 16 key channels of all
// tokens, so that the decays and the sums over tokens stay in its registers.
//
// The products with S and dS and those between blocks of tokens run on fp16 MFMA, both
// sides split into high and low parts (dO's 8 bits fit the high one); a token tile (dO,
// dV, x) has one scale, S and dS one per key. Between blocks the decays factor at a block's
// border into two weights of at most 1. Inside a block they reach e^(+-44), beyond fp16,
// and the four diagonal blocks run on fp32 MFMA.
//
// dg without cancellation: what crosses token t from before its block or to behind it is
// added up from the readers' side (a suffix sum over the block) or the writers' (a prefix
// sum), and what passes the whole block from one of the two. Only pairs inside one
// block are taken as readers less writers.
//
// S and dS rows, decays and sums take 247 registers and the token tiles 152 KB, so one
// workgroup fills a CU and nothing hides its loads: of a workgroup's 65,000 cycles 28 % pass
// before the first product. 64 heads of 8208 tokens: 1199 us, 2.50 GB read and 0.56 GB
// written (2.6 TB/s), the vector units busy for 43 % and the matrix units for 16 % of the
// cycles. One chunk alone: 26 us. (Non-temporal loads of what the chains left made the whole
// call 6 % slower.)
constexpr int HS = D + 8;   // row (fp16) of dO, dV, x: 16-byte rows, 4 banks apart
constexpr int PS = C + 8;   // row (fp16) of DP, DA
constexpr int GS = 20;      // row (fp32) of the diagonal blocks
constexpr int kRows = 48;   // DP, DA: readers 16..63; their transposes: writers 0..47

struct GradSmem {
  uint16_t oh[C * HS], vh[C * HS], vl[C * HS], xh[C * HS], xl[C * HS];  // perm32 order
  // off-diagonal blocks, zero elsewhere, columns in the order of the right fragments:
  // [hi, lo]
  uint16_t pr[2][kRows * PS], ar[2][kRows * PS];  // DP, DA: [reader - 16][writer]
  uint16_t pt[2][kRows * PS], at[2][kRows * PS];  // transposed: [writer][reader]
  float dp[NB][16 * GS], da[NB][16 * GS];         // diagonal blocks, strictly lower
  alignas(16) float diag[C];                      // DP's diagonal
  float top[3][8];
  alignas(16) float beta[C];
  alignas(16) float rq[C], rk[C];
  float slope[C];  // beta's derivative by its input
};
// In the place of dO, dV and x once they are read out: sums over a wave's 16 channels per
// token, and every lane's log-decays and gate slopes.
struct RedSmem {
  float red[4][8][C];
  float keep[2 * 16 * kThreads];
};
static_assert(sizeof(RedSmem) <= sizeof(uint16_t) * C * HS * 5, "the sums fit");

// Position of contraction index t: a fragment holds, for lane group g, 4 g .. 4 g + 3 of
// a run of 16 and of the next one.
__device__ __forceinline__ int perm32(int t) {
  return (t & ~31) + 8 * ((t & 15) >> 2) + 4 * ((t >> 4) & 1) + (t & 3);
}

__device__ __forceinline__ void zero_row(uint16_t* p, int64_t t, int64_t stride, int64_t at,
                                         int n) {
  for (int e = threadIdx.x; e < n; e += kThreads) p[t * stride + at + e] = 0;
}

typedef u32x2 u32x2_u __attribute__((aligned(2)));
__device__ __forceinline__ f32x4 widen4(u32x2 w) {
  return f32x4{bf_lo(w[0]), bf_hi(w[0]), bf_lo(w[1]), bf_hi(w[1])};
}
__device__ __forceinline__ float max4(f32x4 x) {
  return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}
__device__ __forceinline__ f16x8 frag8(const uint16_t* p) {
  return *reinterpret_cast<const f16x8*>(p);
}
// Keeps the compiler from moving work of one stage into another: it would fetch the
// fragments of several stages at once and run out of registers.
__device__ __forceinline__ void stage() { __builtin_amdgcn_sched_barrier(0); }

// Sums of four values over a DPP row: lane n of the row ends with that of value n % 4.
// Two exchanges that halve the values, then two rotations over the lanes of equal n % 4.
__device__ __forceinline__ float row16_sums(const float (&v)[4], int n16) {
  const bool b0 = n16 & 1, b1 = n16 & 2;
  const float x = (b0 ? v[1] : v[0]) + dpp<0xB1>(b0 ? v[0] : v[1]);
  const float y = (b0 ? v[3] : v[2]) + dpp<0xB1>(b0 ? v[2] : v[3]);
  float t = (b1 ? y : x) + dpp<0x4E>(b1 ? x : y);
  t += dpp<0x124>(t);         // row_ror:4
  return t + dpp<0x128>(t);   // row_ror:8
}

template <bool PRE>
__global__ __launch_bounds__(kThreads) void grad_kernel(BwdParams p) {
  extern __shared__ __align__(16) float smem_raw[];
  GradSmem& s = *reinterpret_cast<GradSmem*>(smem_raw);
  RedSmem& sr = *reinterpret_cast<RedSmem*>(smem_raw);
  const int64_t sigma = blockIdx.x;
  const int h = blockIdx.y;
  const Chunk ch = chunk_of(p, sigma);
  float* partial = p.partial + (sigma * p.H + h) * int64_t(2 * D);
  const bool per_head = p.gate_mode & KDA_GATE_PER_HEAD;
  if (ch.c == 0 || !ch.active) {
    if (threadIdx.x < 2 * D) partial[threadIdx.x] = 0.f;
    for (int t = 0; t < ch.c; ++t) {
      zero_row(p.dq, ch.t0 + t, p.dq_stride, int64_t(h) * D, D);
      zero_row(p.dk, ch.t0 + t, p.dk_stride, int64_t(h) * D, D);
      zero_row(p.dv, ch.t0 + t, p.dv_stride, int64_t(h) * D, D);
      zero_row(p.dg, ch.t0 + t, p.dg_stride, per_head ? h : int64_t(h) * D, per_head ? 1 : D);
      zero_row(p.dbeta, ch.t0 + t, p.dbeta_stride, h, 1);
    }
    return;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int kc = 16 * w + n16;
  const uint8_t* ops = p.ops + (sigma * p.H + h) * int64_t(kOps);

  // ---- token tiles: a token's 128 values by 32 lanes
  constexpr int NR = C / (kThreads / 32);
  const int c0 = (threadIdx.x & 31) * 4;
  const Rows orow = rows_of(p.dout, ch, p.dout_stride, int64_t(h) * D);
  const Rows dvr = rows_of(p.dv, ch, p.dv_stride, int64_t(h) * D);
  u32x2 ow[NR];
  f32x4 xv[NR], dv[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int t = (threadIdx.x >> 5) + j * (kThreads / 32);
    ow[j] = *reinterpret_cast<const u32x2_u*>(orow.at(min(t, ch.c - 1), c0));
    xv[j] = lds4(reinterpret_cast<const float*>(ops + kOpX) + t * D + c0);
    dv[j] = lds4(reinterpret_cast<const float*>(ops + kOpDV) + t * D + c0);
  }
  token_scalars<true>(p, ch, h, s.rq, s.rk, s.beta, s.slope);
  // rows of S and dS: a key's values by the four lanes that share it, in perm32 order
  f32x4 Sv[8], dSv[8];
  {
    const float* S = reinterpret_cast<const float*>(ops + kOpS) + kc * D + 4 * g4;
    const float* dS = reinterpret_cast<const float*>(ops + kOpDS) + kc * D + 4 * g4;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      Sv[m] = lds4(S + 16 * m);
      dSv[m] = lds4(dS + 16 * m);
    }
  }
  const float eg = reinterpret_cast<const float*>(ops + kOpTail)[kc];

  float top[3] = {0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int t = (threadIdx.x >> 5) + j * (kThreads / 32);
    if (t >= ch.c) ow[j] = u32x2{0u, 0u};
    else
      *reinterpret_cast<u32x2_u*>(dvr.at(t, c0)) =
          u32x2{pack_bf16x2(dv[j][0], dv[j][1]), pack_bf16x2(dv[j][2], dv[j][3])};
    top[0] = fmaxf(top[0], max4(widen4(ow[j])));
    top[1] = fmaxf(top[1], max4(dv[j]));
    top[2] = fmaxf(top[2], max4(xv[j]));
  }
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    top[a] = wave_max(top[a]);
    if (lane == 0) s.top[a][w] = top[a];
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 3; ++a)
#pragma unroll
    for (int i = 0; i < 8; ++i) top[a] = fmaxf(top[a], uniform(s.top[a][i]));
  const Scale so = scale_for(top[0]), sv = scale_for(top[1]), sx = scale_for(top[2]);
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int at = ((threadIdx.x >> 5) + j * (kThreads / 32)) * HS + perm32(c0);
    const f32x4 o = widen4(ow[j]) * so.up;
    *reinterpret_cast<u32x2*>(s.oh + at) = u32x2{pack_f16x2(o[0], o[1]), pack_f16x2(o[2], o[3])};
    u32x2 hi, lo;
    split4h(dv[j] * sv.up, hi, lo);
    *reinterpret_cast<u32x2*>(s.vh + at) = hi;
    *reinterpret_cast<u32x2*>(s.vl + at) = lo;
    split4h(xv[j] * sx.up, hi, lo);
    *reinterpret_cast<u32x2*>(s.xh + at) = hi;
    *reinterpret_cast<u32x2*>(s.xl + at) = lo;
  }
  // the blocks that a 32-token contraction takes along and that hold nothing
  for (int e = threadIdx.x; e < 2 * kRows * PS / 8; e += kThreads) {
    const u32x4 z = {0u, 0u, 0u, 0u};
    reinterpret_cast<u32x4*>(&s.pr[0][0])[e] = z;
    reinterpret_cast<u32x4*>(&s.ar[0][0])[e] = z;
    reinterpret_cast<u32x4*>(&s.pt[0][0])[e] = z;
    reinterpret_cast<u32x4*>(&s.at[0][0])[e] = z;
  }
  __syncthreads();
  RawLane raw;
  load_lane(p, ch, h, kc, g4, raw);

  // ---- DP = tril(dO x^T, -1) and its diagonal, DA = -tril(dV x^T, -1). Both factors
  // are below 2^15, so 128 terms are below 2^37, and 2^-22 of that fits fp16.
  constexpr float kDown = 1.0f / 4194304.0f, kUp = 4194304.0f;
  constexpr float kW = 16.0f;  // writers' scale: leaves room for a beta beyond 1
  const float uo = so.un * p.scale;  // from here on dO stands for scale dO
  for (int task = w; task < NB * (NB + 1); task += kThreads / 64) {
    const bool is_p = task >= NB * (NB + 1) / 2;
    int I = 0, J = is_p ? task - NB * (NB + 1) / 2 : task;
    while (J > I) J -= ++I;
    const int left = (16 * I + n16) * HS + 8 * g4, right = (16 * J + n16) * HS + 8 * g4;
    f32x4 acc = zero4();
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      const f16x8 bh = frag8(s.xh + right + 32 * kt), bl = frag8(s.xl + right + 32 * kt);
      if (is_p) {
        const f16x8 a = frag8(s.oh + left + 32 * kt);
        acc = mfma32(a, bl, acc);
        acc = mfma32(a, bh, acc);
      } else {
        acc = mfma_split(frag8(s.vh + left + 32 * kt), frag8(s.vl + left + 32 * kt), bh, bl, acc);
      }
    }
    if (!is_p) acc = -acc;
    if (I == J) {
      acc *= (is_p ? uo : sv.un) * sx.un;
      float* dst = is_p ? s.dp[I] : s.da[I];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * g4 + i;
        dst[r * GS + n16] = n16 < r ? acc[i] : 0.f;
        if (is_p && n16 == r) s.diag[16 * I + n16] = acc[i];
      }
    } else {
      u32x2 hi, lo;
      split4h(acc * kDown, hi, lo);
      uint16_t(*row)[kRows * PS] = is_p ? s.pr : s.ar;
      uint16_t(*col)[kRows * PS] = is_p ? s.pt : s.at;
      const int at = perm32(16 * J + n16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        row[0][(16 * (I - 1) + 4 * g4 + i) * PS + at] = uint16_t(hi[i >> 1] >> (16 * (i & 1)));
        row[1][(16 * (I - 1) + 4 * g4 + i) * PS + at] = uint16_t(lo[i >> 1] >> (16 * (i & 1)));
      }
      const int to = (16 * J + n16) * PS + perm32(16 * I + 4 * g4);
      *reinterpret_cast<u32x2*>(col[0] + to) = hi;
      *reinterpret_cast<u32x2*>(col[1] + to) = lo;
    }
  }

  stage();
  // ---- dO S^T, dV S^T, x dS^T for the wave's channels
  f32x4 sq[NB], sk[NB], se[NB];
  float uq, uk, ue;  // their scales
  float flow = 0.f;  // e^Gl sum_v S dS: what passes the whole chunk
  {
    float ts = 0.f, td = 0.f;
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        flow = fmaf(Sv[m][i], dSv[m][i], flow);
        ts = fmaxf(ts, fabsf(Sv[m][i]));
        td = fmaxf(td, fabsf(dSv[m][i]));
      }
    ts = fmaxf(ts, __shfl_xor(ts, 16));
    td = fmaxf(td, __shfl_xor(td, 16));
    const Scale ss = scale_for(fmaxf(ts, __shfl_xor(ts, 32)));
    const Scale sd = scale_for(fmaxf(td, __shfl_xor(td, 32)));
    flow = rows_sum(flow) * eg;
#pragma unroll
    for (int r = 0; r < NB; ++r) sq[r] = sk[r] = se[r] = zero4();
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      stage();
      u32x2 h0, l0, h1, l1;
      split4h(Sv[2 * kt] * ss.up, h0, l0);
      split4h(Sv[2 * kt + 1] * ss.up, h1, l1);
      const f16x8 Sh = join8(h0, h1), Sl = join8(l0, l1);
      split4h(dSv[2 * kt] * sd.up, h0, l0);
      split4h(dSv[2 * kt + 1] * sd.up, h1, l1);
      const f16x8 Dh = join8(h0, h1), Dl = join8(l0, l1);
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        const int at = (16 * r + n16) * HS + 32 * kt + 8 * g4;
        const f16x8 o = frag8(s.oh + at);
        sq[r] = mfma32(o, Sl, sq[r]);
        sq[r] = mfma32(o, Sh, sq[r]);
        sk[r] = mfma_split(frag8(s.vh + at), frag8(s.vl + at), Sh, Sl, sk[r]);
        se[r] = mfma_split(frag8(s.xh + at), frag8(s.xl + at), Dh, Dl, se[r]);
      }
    }
    uq = uo * ss.un;
    uk = sv.un * ss.un;
    ue = sx.un * sd.un;
  }
  stage();
  __syncthreads();
  Lane ln;
  float* keep = sr.keep + threadIdx.x;
  make_lane<PRE, true>(p, ch, h, kc, g4, raw, s.rq, s.rk, ln, keep);
  stage();

  // ---- between blocks: readers from the block's start, writers to its end. A pair two
  // blocks apart also takes the whole blocks between, a factor per channel: on the operand
  // where one product holds pairs of both kinds, else on the result.
  const float uqr = kUp * uo * sx.un / kW, ukr = kUp * sv.un * sx.un / kW;
  const float uboth = fmaxf(fabsf(uo), sv.un);  // writers add up DA^T k and DP^T q
  const float uw = kUp * sx.un * uboth * kFixedUn;
  float T[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) T[b] = ln.head[b] * ln.tail[b];
  auto frags = [](f32x4 a, f32x4 b, f16x8& hi, f16x8& lo) {
    u32x2 h0, l0, h1, l1;
    split4h(a, h0, l0);
    split4h(b, h1, l1);
    hi = join8(h0, h1);
    lo = join8(l0, l1);
  };
  auto row = [&](const uint16_t(*m)[kRows * PS], int blk, int t, f16x8 bh, f16x8 bl, f32x4 c) {
    const int at = (16 * blk + n16) * PS + 32 * t + 8 * g4;
    return mfma_split(frag8(m[0] + at), frag8(m[1] + at), bh, bl, c);
  };
  auto writer = [&](int b) {  // beta k of block b's tokens, to its end
    const f32x4 bt = lds4(s.beta + 16 * b + 4 * g4) * (ln.tail[b] * kW);
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = ln.k[b][i] * (bt[i] * inverse(ln.up[b][i]));
    return x;
  };
  f32x4 c0a, c0b, c1, c2;  // writers of block 0 (for 1; for 2, 3), 1 and 2
  {
    f16x8 bh, bl;
    c0a = c0b = c1 = c2 = zero4();
    // brought to one scale, the larger of the two, so that both stay within fp16
    const float cq = kFixedUp * (uo / uboth), ck = kFixedUp * (sv.un / uboth);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      stage();
      const uint16_t(*m)[kRows * PS] = which ? s.pt : s.at;
      f32x4 x[3];  // readers 1..3
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        const float hd = ln.head[b + 1] * (which ? cq : ck);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[b][i] = (which ? ln.q[b + 1][i] : ln.k[b + 1][i]) * (ln.up[b + 1][i] * hd);
      }
      frags(zero4(), x[0], bh, bl);
      c0a = row(m, 0, 0, bh, bl, c0a);
      frags(x[1], x[2] * T[2], bh, bl);
      c0b = row(m, 0, 1, bh, bl, c0b);
      c1 = row(m, 1, 1, bh, bl, c1);
      frags(zero4(), x[2], bh, bl);
      c2 = row(m, 2, 1, bh, bl, c2);
    }
  }

  // ---- block by block: the diagonal block, the sums, and the tokens' gradients
  float dg[NB][4];                 // first what the block itself adds to dg
  f32x4 gq[NB], gk[NB];            // dq_hat, dk_hat
  float reads[NB], ends[NB];       // block sums: readers of S; writers into dS
  float pass1 = 0.f, pass2 = 0.f;  // pairs across block 1, across block 2
  float F = 1.f;                   // from the chunk's start
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    stage();
    // what the block's readers get from earlier ones; of block 3 apart from 0, 1 and from 2
    f32x4 rq = zero4(), rk = zero4(), rqa = zero4(), rka = zero4();
    if (b > 0) {
      f16x8 bh, bl;
      if (b == 1) frags(writer(0), zero4(), bh, bl);
      if (b >= 2) frags(writer(0) * T[1], writer(1), bh, bl);
      rq = row(s.pr, b - 1, 0, bh, bl, zero4());
      rk = row(s.ar, b - 1, 0, bh, bl, zero4());
      if (b == 3) {
        rqa = rq;
        rka = rk;
        frags(writer(2), zero4(), bh, bl);
        rq = row(s.pr, 2, 1, bh, bl, zero4());
        rk = row(s.ar, 2, 1, bh, bl, zero4());
      }
    }
    stage();
    const f32x4 bt = lds4(s.beta + 16 * b + 4 * g4), self = lds4(s.diag + 16 * b + 4 * g4);
    f32x4 kb, km, qm, dn;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // hidden from the compiler, which would keep what it has formed above of these
      asm volatile("" : "+v"(ln.up[b][i]), "+v"(ln.k[b][i]), "+v"(ln.q[b][i]));
      dn[i] = inverse(ln.up[b][i]);
      kb[i] = ln.k[b][i] * bt[i] * dn[i];
      km[i] = ln.k[b][i] * ln.up[b][i];
      qm[i] = ln.q[b][i] * ln.up[b][i];
    }
    const f32x4 dq = mfma4(lds4(s.dp[b] + n16 * GS + 4 * g4), kb, zero4());
    const f32x4 dk = mfma4(lds4(s.da[b] + n16 * GS + 4 * g4), kb, zero4());
    f32x4 dc = mfma4(col4(s.dp[b] + 4 * g4 * GS + n16, GS), qm, zero4());
    dc = mfma4(col4(s.da[b] + 4 * g4 * GS + n16, GS), km, dc);
    float E = ue;  // to the chunk's end
#pragma unroll
    for (int m = b + 1; m < NB; ++m) E *= T[m];
    const float Fq = F * uq, Fk = F * uk, qT = uqr * T[2], kT = ukr * T[2], cT = uw * T[1];
    float rsum = 0.f, esum = 0.f, across = 0.f;
    float suf[4], pre[4], a0[4], a1[4], a2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float k = ln.k[b][i], q = ln.q[b][i], kbeta = k * bt[i];
      const float rd = ln.up[b][i] * ln.head[b], wr = dn[i] * ln.tail[b];
      const float kwr = kbeta * wr;
      // readers: of the state, then of earlier blocks too
      const float fs = Fq * sq[b][i], fk = Fk * sk[b][i];
      float A = fs, B = -fk;
      if (b > 0) {
        A = fmaf(uqr, rq[i], A);
        B = fmaf(ukr, rk[i], B);
      }
      if (b == 3) {
        const float fq = qT * rqa[i], fr = kT * rka[i];
        A += fq;
        B += fr;
        across = fmaf(fmaf(k, fr, q * fq), rd, across);
      }
      if (b > 0) rsum = fmaf(fmaf(-k, fk, q * fs), rd, rsum);
      // writers: into dS, then for later blocks too
      const float we = E * se[b][i];
      float W = we;
      if (b == 0) {
        const float far = cT * c0b[i];
        W = fmaf(uw, c0a[i], W + far);
        across = fmaf(kwr, far, across);
      }
      if (b == 1) W = fmaf(uw, c1[i], W);
      if (b == 2) W = fmaf(uw, c2[i], W);
      if (b < 3) esum = fmaf(kwr, we, esum);
      // with the block's own pairs, and at last the token's own
      const float in = dn[i] * dc[i];
      const float dqt = fmaf(rd, A, ln.up[b][i] * dq[i]);
      const float dkt = fmaf(rd, B, ln.up[b][i] * dk[i]);
      suf[i] = fmaf(-kbeta, in, fmaf(k, dkt, q * dqt));
      pre[i] = kwr * W;
      const float col = fmaf(self[i], q, fmaf(wr, W, in));
      gq[b][i] = fmaf(self[i], kbeta, dqt);
      gk[b][i] = fmaf(bt[i], col, dkt);
      a0[i] = q * gq[b][i];
      a1[i] = k * gk[b][i];
      a2[i] = k * col;
    }
    // q_hat . dq_hat, k_hat . dk_hat, k_hat . col over the wave's channels
    const float r0 = row16_sums(a0, n16), r1 = row16_sums(a1, n16), r2 = row16_sums(a2, n16);
    if (n16 < 4) {
      const int t = 16 * b + 4 * g4 + n16;
      sr.red[0][w][t] = r0;
      sr.red[1][w][t] = r1;
      sr.red[2][w][t] = r2;
    }
    reads[b] = b > 0 ? rows_sum(rsum) : 0.f;
    ends[b] = b < 3 ? rows_sum(esum) : 0.f;
    if (b == 3) pass2 = rows_sum(across);
    if (b == 0) pass1 = rows_sum(across);
    // suffix sums (from the token on) and prefix sums (before it) over the block
    const float stot = (suf[0] + suf[1]) + (suf[2] + suf[3]);
    const float ptot = (pre[0] + pre[1]) + (pre[2] + pre[3]);
    const float s1 = __shfl_xor(stot, 16), p1 = __shfl_xor(ptot, 16);
    const float s2 = __shfl_xor(stot + s1, 32), p2 = __shfl_xor(ptot + p1, 32);
    float sacc = ((g4 & 1) ? 0.f : s1) + ((g4 & 2) ? 0.f : s2);
    float pacc = ((g4 & 1) ? p1 : 0.f) + ((g4 & 2) ? p2 : 0.f);
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      sacc += suf[i];
      dg[b][i] = sacc;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dg[b][i] += pacc;
      pacc += pre[i];
    }
    F *= T[b];
  }
  stage();
  // what passes each block as a whole
  const float across[NB] = {reads[1] + reads[2] + reads[3], reads[2] + reads[3] + ends[0] + pass1,
                            reads[3] + ends[0] + ends[1] + pass2, ends[0] + ends[1] + ends[2]};
  float sum_b = 0.f, sum_a = 0.f;  // of ddt_bias, dA_log
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = dg[b][i] + (across[b] + flow);
      dg[b][i] = x;
      const float slope = keep[(16 + 4 * b + i) * kThreads];
      sum_b = fmaf(x, slope, sum_b);
      sum_a = fmaf(x, slope != 0.f ? keep[(4 * b + i) * kThreads] : 0.f, sum_a);
      if (per_head) {
        const float a3 = row16_sum(x);
        if (n16 == 0) sr.red[3][w][16 * b + 4 * g4 + i] = a3;
      }
    }
  sum_b = rows_sum(sum_b);
  sum_a = rows_sum(sum_a);
  if (g4 == 0) {
    partial[kc] = sum_b;
    partial[D + kc] = sum_a;
  }
  __syncthreads();
  if (threadIdx.x < C * 4) {  // add the eight waves' sums
    const int which = threadIdx.x / C, t = threadIdx.x % C;
    if (which < 3 || per_head) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x += sr.red[which][i][t];
      sr.red[which][0][t] = x;
      if (which == 2 && t < ch.c)
        p.dbeta[(ch.t0 + t) * p.dbeta_stride + h] = to_bf16(x * s.slope[t]);
    }
  }
  __syncthreads();
  const Rows dqr = rows_of(p.dq, ch, p.dq_stride, int64_t(h) * D);
  const Rows dkr = rows_of(p.dk, ch, p.dk_stride, int64_t(h) * D);
  const Rows dgr = rows_of(p.dg, ch, p.dg_stride, per_head ? h : int64_t(h) * D);
  const uint32_t dq0 = dqr.offset(4 * g4, kc), dk0 = dkr.offset(4 * g4, kc);
  const uint32_t dg0 = dgr.offset(4 * g4, per_head ? 0 : kc);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * b + 4 * g4 + i;
      if (t < ch.c) {
        const float rq = s.rq[t], rk = s.rk[t];
        const float slope = keep[(16 + 4 * b + i) * kThreads];
        const float dq = rq * fmaf(-ln.q[b][i], sr.red[0][0][t], gq[b][i]);
        const float dk = rk * fmaf(-ln.k[b][i], sr.red[1][0][t], gk[b][i]);
        *dqr.from(dq0, 16 * b + i) = to_bf16(dq);
        *dkr.from(dk0, 16 * b + i) = to_bf16(dk);
        if (!per_head)
          *dgr.from(dg0, 16 * b + i) = to_bf16(dg[b][i] * slope);
        else if (w == 0 && n16 == 0)
          *dgr.from(dg0, 16 * b + i) = to_bf16(sr.red[3][0][t] * slope);
      }
    }
}

// dA_log and ddt_bias: the partial sums of a head, added in the order of the chunk
// slots by 8 groups of 128 lanes (a channel each), then group by group.
__global__ __launch_bounds__(1024) void param_kernel(BwdParams p) {
  __shared__ float sum[2][8][D];
  __shared__ float half[4];
  const int h = blockIdx.x;
  const int c = threadIdx.x & (D - 1), grp = threadIdx.x / D;
  float b = 0.f, a = 0.f;
  int64_t n = grp;
  for (; n + 56 < p.slots; n += 64) {  // eight loads in flight, added in the same order
    float xb[8], xa[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* x = p.partial + ((n + 8 * i) * p.H + h) * int64_t(2 * D);
      xb[i] = x[c];
      xa[i] = x[D + c];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b += xb[i];
      a += xa[i];
    }
  }
  for (; n < p.slots; n += 8) {
    const float* x = p.partial + (n * p.H + h) * int64_t(2 * D);
    b += x[c];
    a += x[D + c];
  }
  sum[0][grp][c] = b;
  sum[1][grp][c] = a;
  __syncthreads();
  const bool per_head = p.gate_mode & KDA_GATE_PER_HEAD;
  float t = 0.f;
  if (grp < 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sum[grp][i][c];
    if (grp == 0 && !per_head && p.ddt_bias) p.ddt_bias[h * D + c] = t;
    // a head's one value: the sum over its channels
    t = rows_sum(row16_sum(t));
    if ((threadIdx.x & 63) == 0) half[threadIdx.x >> 6] = t;
  }
  __syncthreads();
  if (grp < 2 && c == 0) {
    t = half[2 * grp] + half[2 * grp + 1];
    if (grp == 1 && p.dA_log) p.dA_log[h] = t;
    if (grp == 0 && per_head && p.ddt_bias) p.ddt_bias[h] = t;
  }
}

}  // namespace

template <bool PRE>
static hipError_t launch_grad(const BwdParams& p, hipStream_t stream) {
  static_assert(sizeof(GradSmem) <= 160 * 1024, "LDS of a CU");
  static std::atomic<bool> allowed[kMaxDevices];
  const void* kernel = reinterpret_cast<const void*>(grad_kernel<PRE>);
  if (const hipError_t e = allow_lds(kernel, sizeof(GradSmem), allowed))
    return e;
  hipLaunchKernelGGL(grad_kernel<PRE>, dim3(unsigned(p.slots), unsigned(p.H)), dim3(kThreads),
                     sizeof(GradSmem), stream, p);
  return hipGetLastError();
}

hipError_t launch_grads(const BwdParams& p, hipStream_t stream) {
  return (p.gate_mode & KDA_GATE_PRECOMPUTED) ? launch_grad<true>(p, stream)
                                              : launch_grad<false>(p, stream);
}

hipError_t launch_params(const BwdParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(param_kernel, dim3(unsigned(p.H)), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

}  // namespace bwd
}  // namespace kda
