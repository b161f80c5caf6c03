// Prefill gradient, chains (gfx950): the states up and the state gradients down every
// (document, head), chunk by chunk, from what the preparation left. The method is described
// in kda_backward.hip.

#include "kda_bwd.h"

namespace kda {
namespace bwd {
namespace {

// ---------------------------------------------------------------------------
// Chains: the states up each (document, head), and the state gradients down.
// Value channels do not mix in either, so a wave owns NT tiles of 16 of them, with
// all 128 key channels in eight accumulator tiles each, and the chain is sequential
// over the chunks alone. What bounds it is the latency of one chunk: two products
// that wait for each other. They run on fp16 MFMA with both sides split into high and
// low parts (three terms, fp32 accuracy at 3/16 of fp32 MFMA's time). The right sides,
// which are the state and x in accumulator layout, are scaled per value channel.
//
// A chunk's operands come in two tiles (W, then KE; or Z, then KG and QG) that all
// waves share through LDS. Loads of a tile are issued two phases before it is read
// and wait in registers in between; the barrier between the phases publishes one
// tile and frees the other.
__device__ __forceinline__ float pool_at(const BwdParams& p, int64_t e) {
  if (p.state_dtype == KDA_STATE_FP8)
    return f8x2_lo(static_cast<const uint8_t*>(p.pool)[e])[0];
  const uint16_t b = static_cast<const uint16_t*>(p.pool)[e];
  return p.state_dtype == KDA_STATE_FP16 ? f16_lo(b) : bf1(b);
}

constexpr int kTileBytes = 32768;
constexpr int kChainLds = 3 * kTileBytes + 2 * 1024;

// N 16-byte units per thread, from global memory to registers, and on to LDS.
template <int N, int T>
struct Stage {
  u32x4 u[N];
  __device__ __forceinline__ void load(const uint8_t* src) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      u[i] = *reinterpret_cast<const u32x4*>(src + (i * T + int(threadIdx.x)) * 16);
  }
  __device__ __forceinline__ void store(uint8_t* dst) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<u32x4*>(dst + (i * T + int(threadIdx.x)) * 16) = u[i];
  }
};

// The largest magnitude of a value channel over the four lanes that share it.
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

// Right-side fragments of N accumulator tiles (rows 16 m + 4 g4 + i): pairs of tiles
// give 32 contraction indices.
template <int N>
struct Right {
  f16x8 hi[N / 2], lo[N / 2];
  float un;
  __device__ __forceinline__ void set(const f32x4 (&x)[N]) {
    float top = 0.f;
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[m][i]));
    const Scale sc = scale_for(column_max(top));
    un = sc.un;
#pragma unroll
    for (int t = 0; t < N / 2; ++t) {
      u32x2 h0, l0, h1, l1;
      split4h(x[2 * t] * sc.up, h0, l0);
      split4h(x[2 * t + 1] * sc.up, h1, l1);
      hi[t] = join8(h0, h1);
      lo[t] = join8(l0, l1);
    }
  }
};

template <int NW, int NT>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(1, 2)))
void chain_kernel(BwdParams p, DocOrder ord) {
  constexpr int T = 64 * NW;
  constexpr int PARTS = 8 / (NW * NT);
  constexpr int NA = kTileBytes / 16 / T;
  extern __shared__ __align__(16) float smem_raw[];
  uint8_t* la = reinterpret_cast<uint8_t*>(smem_raw);
  uint8_t* lb = la + kTileBytes;
  float* tails = reinterpret_cast<float*>(lb + 2 * kTileBytes);  // of even and odd chunks

  // Chain c's parts are blocks (c / 8 * PARTS + part) * 8 + c % 8: blocks go to the
  // eight XCDs in turn, so the parts share one L2 copy of the operands.
  const int64_t bid = blockIdx.x;
  const int64_t id = bid / (8 * PARTS) * 8 + (bid & 7);
  const int part = int((bid >> 3) % PARTS);
  const bool down = id & 1;
  const int64_t chain = id >> 1;
  if (chain >= int64_t(p.n_docs) * p.H) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int vt0 = (part * NW + wave) * NT;  // this wave's first value tile
  const int h = int(chain % p.H);
  const int rank = int(chain / p.H);
  const int doc = ord.n > 0 ? ord.doc[rank] : rank;
  const int64_t t0 = p.cu_seqlens[doc];
  const int64_t len = int64_t(p.cu_seqlens[doc + 1]) - t0;
  const int32_t slot = p.state_indices[doc];
  const bool active = slot >= 0 && int64_t(slot) < p.num_slots;
  const int64_t chunks = (len + C - 1) / C;
  const int64_t state = (int64_t(doc) * p.H + h) * HEAD_ELEMS + (16 * vt0 + n16) * D + 4 * g4;
  const int64_t step = int64_t(p.H) * kOps;
  uint8_t* ops0 = p.ops + (doc_slot0(p.cu_seqlens, doc) * p.H + h) * int64_t(kOps);

  f32x4 s[NT][8];  // [key 16 m + 4 g4 + i][value 16 (vt0 + n) + n16]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < 8; ++m) s[n][m] = zero4();

  const uint8_t* left = la + lane * 16;
  const uint8_t* left2 = lb + lane * 16;
  auto frag = [](const uint8_t* base, int unit) {
    return *reinterpret_cast<const f16x8*>(base + unit * 1024);
  };
  // acc[r] = sum over keys of tile A's row block r times the state
  auto product_a = [&](const Right<8> (&b)[NT], f32x4 (&acc)[NT][NB]) {
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        const f16x8 ah = frag(left, (r * 4 + kt) * 2), al = frag(left, (r * 4 + kt) * 2 + 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (kt == 0) acc[n][r] = zero4();
          acc[n][r] = mfma32(al, b[n].hi[kt], acc[n][r]);
          acc[n][r] = mfma32(ah, b[n].lo[kt], acc[n][r]);
          acc[n][r] = mfma32(ah, b[n].hi[kt], acc[n][r]);
        }
      }
  };
  // s = e^Gl s + sign * (tile B's first half)^T b, or with the second half on o too
  auto update = [&](const Right<NB> (&b)[NT], float sign, const f16x8 (*o)[2],
                    const float* uno, const float* tail) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      f32x4 acc[NT], acc2[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n] = acc2[n] = zero4();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const f16x8 ah = frag(left2, (m * 2 + t) * 2), al = frag(left2, (m * 2 + t) * 2 + 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n] = mfma32(al, b[n].hi[t], acc[n]);
          acc[n] = mfma32(ah, b[n].lo[t], acc[n]);
          acc[n] = mfma32(ah, b[n].hi[t], acc[n]);
        }
        if (o) {
          const f16x8 qh = frag(left2, 32 + (m * 2 + t) * 2), ql = frag(left2, 33 + (m * 2 + t) * 2);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc2[n] = mfma32(ql, o[n][t], acc2[n]);
            acc2[n] = mfma32(qh, o[n][t], acc2[n]);
          }
        }
      }
      const f32x4 eg = lds4(tail + 16 * m + 4 * g4);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float un = b[n].un * (sign * kFixedUn);
        s[n][m] *= eg;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][m][i] = fmaf(acc[n][i], un, s[n][m][i]);
        if (o)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][m][i] = fmaf(acc2[n][i], uno[n], s[n][m][i]);
      }
    }
  };

  if (!down) {
    if (!active || len == 0) return;
    if (p.use_initial) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t e = int64_t(slot) * p.slot_stride + int64_t(h) * HEAD_ELEMS +
                          (16 * (vt0 + n) + n16) * D + 4 * g4;
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][m][i] = pool_at(p, e + 16 * m + i);
      }
    }
    Stage<NA, T> sa, sb;
    u32x4 st = {0u, 0u, 0u, 0u};
    auto load_a = [&](int64_t n) {
      sa.load(ops0 + n * step + kOpW);
      if (threadIdx.x < 64) st = *reinterpret_cast<const u32x4*>(ops0 + n * step + threadIdx.x * 16);
    };
    auto store_a = [&](int64_t n) {
      sa.store(la);
      if (threadIdx.x < 64) *reinterpret_cast<u32x4*>(tails + (n & 1) * 256 + threadIdx.x * 4) = st;
    };
    f32x4 x[NT][NB];  // T V of the next chunk, asked for a phase ahead
    auto load_x = [&](int64_t n) {
      const float* X = reinterpret_cast<const float*>(ops0 + n * step + kOpX0) +
                       (vt0 * NB * 64 + lane) * 4;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < NB; ++r) x[j][r] = lds4(X + (j * NB + r) * 256);
    };
    load_a(0);
    load_x(0);
    store_a(0);
    sb.load(ops0 + kOpKE);
    __syncthreads();
    for (int64_t n = 0; n < chunks; ++n) {
      uint8_t* ops = ops0 + n * step;
      const bool more = n + 1 < chunks;
      const float* tail = tails + (n & 1) * 256;
      float* S = reinterpret_cast<float*>(ops + kOpS) + 4 * g4 * D + 16 * vt0 + n16;
      float* X = reinterpret_cast<float*>(ops + kOpX) + 4 * g4 * D + 16 * vt0 + n16;
      // ---- x = T V - W S
      if (more) load_a(n + 1);
      {
        Right<8> b[NT];
        f32x4 acc[NT][NB];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b[j].set(s[j]);
#pragma unroll
          for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[(16 * m + i) * D + 16 * j] = s[j][m][i];
        }
        product_a(b, acc);
        const float unw = tail[kTailUnW];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < NB; ++r) {
            const float un = -b[j].un * unw;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[j][r][i] = fmaf(acc[j][r][i], un, x[j][r][i]);
              X[(16 * r + i) * D + 16 * j] = x[j][r][i];
            }
          }
      }
      if (!more) return;  // the state after the last chunk is not needed
      sb.store(lb);
      __syncthreads();
      // ---- S = e^Gl S + KE^T (beta x)
      {
        Right<NB> b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int r = 0; r < NB; ++r) x[j][r] *= lds4(tail + kTailBeta + 16 * r + 4 * g4);
          b[j].set(x[j]);
        }
        load_x(n + 1);
        sb.load(ops + step + kOpKE);
        update(b, 1.0f, nullptr, nullptr, tail);
      }
      store_a(n + 1);
      __syncthreads();
    }
    return;
  }

  if (p.d_final && active) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][m][i] = p.d_final[state + n * 16 * D + 16 * m + i];
  }
  if (active && chunks > 0) {
    Stage<NA, T> sa;
    Stage<2 * NA, T> sb;
    u32x4 st = {0u, 0u, 0u, 0u};
    auto load_a = [&](int64_t n) {
      sa.load(ops0 + n * step + kOpZ);
      if (threadIdx.x < 64) st = *reinterpret_cast<const u32x4*>(ops0 + n * step + threadIdx.x * 16);
    };
    auto store_a = [&](int64_t n) {
      sa.store(la);
      if (threadIdx.x < 64) *reinterpret_cast<u32x4*>(tails + (n & 1) * 256 + threadIdx.x * 4) = st;
    };
    f32x4 x[NT][NB];  // T^T P^T dO and dO of the next chunk
    uint16_t ow[NT][NB][4];
    auto load_x = [&](int64_t n) {
      const float* DV = reinterpret_cast<const float*>(ops0 + n * step + kOpDV0) +
                        (vt0 * NB * 64 + lane) * 4;
      const int c = int(min<int64_t>(C, len - n * C));
      const Rows o = rows_of(p.dout, Chunk{doc, t0 + n * C, c, true}, p.dout_stride, int64_t(h) * D);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < NB; ++r) {
          x[j][r] = lds4(DV + (j * NB + r) * 256);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ow[j][r][i] = *o.at(min(16 * r + 4 * g4 + i, c - 1), 16 * (vt0 + j) + n16);
        }
    };
    load_a(chunks - 1);
    load_x(chunks - 1);
    store_a(chunks - 1);
    sb.load(ops0 + (chunks - 1) * step + kOpKG);
    __syncthreads();
    for (int64_t n = chunks - 1; n >= 0; --n) {
      uint8_t* ops = ops0 + n * step;
      const int c = int(min<int64_t>(C, len - n * C));
      const float* tail = tails + (n & 1) * 256;
      float* dS = reinterpret_cast<float*>(ops + kOpDS) + 4 * g4 * D + 16 * vt0 + n16;
      float* DV = reinterpret_cast<float*>(ops + kOpDV) + 4 * g4 * D + 16 * vt0 + n16;
      // ---- dV = T^T P^T dO + Z dS
      if (n > 0) load_a(n - 1);
      {
        Right<8> b[NT];
        f32x4 acc[NT][NB];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b[j].set(s[j]);
#pragma unroll
          for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) dS[(16 * m + i) * D + 16 * j] = s[j][m][i];
        }
        product_a(b, acc);
        const float unz = tail[kTailUnZ];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < NB; ++r) {
            const float un = b[j].un * unz;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[j][r][i] = fmaf(acc[j][r][i], un, x[j][r][i]);
              DV[(16 * r + i) * D + 16 * j] = x[j][r][i];
            }
          }
      }
      if (n == 0 && !p.d_initial) return;
      sb.store(lb);
      __syncthreads();
      // ---- dS = e^Gl dS - KG^T dV + scale QG^T dO
      {
        Right<NB> b[NT];
        f16x8 o[NT][2];
        float uno[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b[j].set(x[j]);
          // dO has 8 bits: its high part alone is exact
          f32x4 y[NB];
          float top = 0.f;
#pragma unroll
          for (int r = 0; r < NB; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[r][i] = 16 * r + 4 * g4 + i < c ? bf1(ow[j][r][i]) : 0.f;
              top = fmaxf(top, fabsf(y[r][i]));
            }
          const Scale sc = scale_for(column_max(top));
          uno[j] = sc.un * (p.scale * kFixedUn);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const f32x4 a = y[2 * t] * sc.up, d = y[2 * t + 1] * sc.up;
            o[j][t] = __builtin_bit_cast(
                f16x8, u32x4{pack_f16x2(a[0], a[1]), pack_f16x2(a[2], a[3]),
                             pack_f16x2(d[0], d[1]), pack_f16x2(d[2], d[3])});
          }
        }
        if (n > 0) {
          load_x(n - 1);
          sb.load(ops - step + kOpKG);
        }
        update(b, -1.0f, o, uno, tail);
      }
      if (n > 0) store_a(n - 1);
      __syncthreads();
    }
  }
  if (p.d_initial) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < 8; ++m)
        *reinterpret_cast<f32x4*>(p.d_initial + state + n * 16 * D + 16 * m) = s[n][m];
  }
}

template <int NW, int NT>
void launch_chain(const BwdParams& p, const DocOrder& ord, hipStream_t stream) {
  constexpr int PARTS = 8 / (NW * NT);
  const int64_t ids = (int64_t(p.n_docs) * p.H * 2 + 7) / 8 * 8;  // both directions
  hipLaunchKernelGGL((chain_kernel<NW, NT>), dim3(unsigned(ids * PARTS)), dim3(64 * NW), kChainLds,
                     stream, p, ord);
}

}  // namespace

hipError_t launch_chains(const BwdParams& p, const DocOrder& ord, hipStream_t stream) {
  static const hipError_t lds = [] {
    const void* all[] = {reinterpret_cast<const void*>(chain_kernel<2, 1>),
                         reinterpret_cast<const void*>(chain_kernel<4, 1>),
                         reinterpret_cast<const void*>(chain_kernel<4, 2>)};
    for (const void* f : all)
      if (const hipError_t e = hipFuncSetAttribute(
              f, hipFuncAttributeMaxDynamicSharedMemorySize, kChainLds))
        return e;
    return hipSuccess;
  }();
  if (lds != hipSuccess) return lds;
  const int64_t chains = int64_t(p.n_docs) * p.H;
  // workgroups per chain and direction: as many as it takes to fill the chip
  if (chains <= 32) launch_chain<2, 1>(p, ord, stream);
  else if (chains <= 128) launch_chain<4, 1>(p, ord, stream);
  else launch_chain<4, 2>(p, ord, stream);
  return hipGetLastError();
}

}  // namespace bwd
}  // namespace kda
