// Prefill gradient, chains (gfx950): the states up and the state gradients down every
// (document, head), chunk by chunk, from what the preparation left. The method is described
// in kda_backward.hip.

#include "kda_bwd.h"

namespace kda {
namespace bwd {
namespace {

// ---------------------------------------------------------------------------
// Chains: the states up each (document, head), and the state gradients down.
// Value channels do not mix in either, so a chain splits into tiles of 16 of them, and
// it is sequential over the chunks alone. What bounds it is the latency of one chunk: two
// products that wait for each other, with a handful of waves per CU to hide it. A tile
// therefore belongs to KS waves that hold 128 / KS key channels each: all form their keys'
// part of the first product, exchange the parts through LDS, and then hold the same x for the
// second. Times of the whole call, us; 12 heads of 8191 tokens | 14 documents, 12 heads | 64
// heads, 8208 tokens in six documents:
//   two waves, four tiles (wide)           951 | 1084 | 2510
//   four waves, two tiles (deep)           832 | 1126 | 2790
//   four waves, one tile, operands by LDS  802 | 1412 | 3588
//   the same, operands to registers (few)  722 | 1199 | 2963
//   two waves, two tiles                   884 | 1162 | 2895
//   two waves, one tile                    844 | 1470 | 3806
// so the first, second and fourth are taken where each is best, see launch_chains. (Since
// then dO is prepared once per chunk and rows leave in 16-byte stores: 687 | 1033 | 2562, of
// which this kernel takes 377, 377 and 873, the last at 4.3 TB/s of operands and states.)
//
// The products run on fp16 MFMA, both sides split into high and low parts (three terms,
// 22 bits a side, at 3/16 of fp32 MFMA's time). The right sides, the state and x in
// accumulator layout, are scaled per value channel.
//
// A chunk's left operands come in two tiles (W, then KE; or Z, then KG and QG). With several
// value tiles all waves share them through LDS: loads of a tile are issued two phases before
// it is read and wait in registers in between; the barrier between the phases publishes one
// tile, frees the other, and publishes the exchanged parts too. With one value tile every
// fragment has a single reader: it goes to that wave's registers a chunk ahead, LDS holds the
// exchanged parts alone, and one barrier a chunk is left.
__device__ __forceinline__ float pool_at(const BwdParams& p, int64_t e) {
  if (p.state_dtype == KDA_STATE_FP8)
    return f8x2_lo(static_cast<const uint8_t*>(p.pool)[e])[0];
  const uint16_t b = static_cast<const uint16_t*>(p.pool)[e];
  return p.state_dtype == KDA_STATE_FP16 ? f16_lo(b) : bf1(b);
}

constexpr int kTileBytes = 32768;

// N 16-byte units per thread, from global memory to registers, and on to LDS.
template <int N, int T>
struct Stage {
  u32x4 u[N];
  __device__ __forceinline__ void load(const uint8_t* src) {
#pragma unroll
    for (int i = 0; i < N; ++i) load_one(src, i);
  }
  // share `part` of `parts`: a CU takes in some 32 bytes a cycle, so a whole tile asked
  // for at once would hold up the wave that asks; in shares it hides between products
  template <int PARTS>
  __device__ __forceinline__ void load_share(const uint8_t* src, int part) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * PARTS / N == part) load_one(src, i);
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ void load_one(const uint8_t* src, int i) {
    u[i] = *reinterpret_cast<const u32x4*>(src + (i * T + int(threadIdx.x)) * 16);
  }
  __device__ __forceinline__ void store(uint8_t* dst) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<u32x4*>(dst + (i * T + int(threadIdx.x)) * 16) = u[i];
  }
};

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

// Lanes 4 q + j hold element i of column j; afterwards lane 4 q + j holds column i's element
// j. With it a row's 16 values leave as four 16-byte stores instead of 16 of 4 bytes.
__device__ __forceinline__ f32x4 quad_transpose(f32x4 a, int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const float r0 = dpp<0xB1>(b0 ? a[0] : a[1]), r2 = dpp<0xB1>(b0 ? a[2] : a[3]);
  const f32x4 c = {b0 ? r0 : a[0], b0 ? a[1] : r0, b0 ? r2 : a[2], b0 ? a[3] : r2};
  const float s0 = dpp<0x4E>(b1 ? c[0] : c[2]), s1 = dpp<0x4E>(b1 ? c[1] : c[3]);
  return f32x4{b1 ? s0 : c[0], b1 ? s1 : c[1], b1 ? c[2] : s0, b1 ? c[3] : s1};
}

// Workgroups of TW value tiles, KS waves each.
template <int KS, int TW>
struct ChainShape {
  static constexpr int NM = 8 / KS;   // state tiles of a wave
  static constexpr int NX = NB / KS;  // token blocks of x whose start and result a wave moves
  static constexpr int kThreads = 64 * KS * TW;
  static constexpr int kParts = 8 / TW;
  // With one value tile, every fragment has one reader, and goes to its registers directly.
  static constexpr bool kOwn = TW == 1;
  static constexpr int kXch = KS * TW * 4096;  // each wave's part of x
  static constexpr int kLds = kOwn ? 3 * 1024 + 2 * kXch : 3 * kTileBytes + 2 * 1024 + kXch;
};

// Part `part` of the chain of (doc, h), up the document or down.
template <int KS, int TW>
__device__ __forceinline__ void chain(const BwdParams& p, int doc, int h, bool down, int part) {
  using Shape = ChainShape<KS, TW>;
  constexpr int T = Shape::kThreads;
  constexpr int NM = Shape::NM;
  constexpr int NX = Shape::NX;
  constexpr int NA = kTileBytes / 16 / T;
  constexpr bool OWN = Shape::kOwn;
  extern __shared__ __align__(16) float smem_raw[];
  uint8_t* la = reinterpret_cast<uint8_t*>(smem_raw);
  uint8_t* lb = la + kTileBytes;
  // Those of even and odd chunks; OWN, whose one barrier a chunk lets a wave run further
  // ahead: of every third, and the parts of x of even and odd chunks.
  float* tails = reinterpret_cast<float*>(OWN ? la : lb + 2 * kTileBytes);
  float* xch0 = tails + (OWN ? 768 : 512);  // [wave][rt][lane][4]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kh = wave % KS;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int v = 16 * (part * TW + wave / KS) + n16;  // this lane's value channel
  // where a lane's values go after quad_transpose, in a tile of 16 rows
  const int at_row = (4 * g4 + (lane & 3)) * D + (v & ~3);
  const int k0 = 16 * NM * kh + 4 * g4;                   // its first key channel
  const int32_t t0 = __builtin_amdgcn_readfirstlane(p.cu_seqlens[doc]);
  const int32_t len = __builtin_amdgcn_readfirstlane(p.cu_seqlens[doc + 1]) - t0;
  const int32_t slot = __builtin_amdgcn_readfirstlane(p.state_indices[doc]);
  const bool active = slot >= 0 && int64_t(slot) < p.num_slots;
  const int chunks = (len + C - 1) / C;
  const int64_t state = (int64_t(doc) * p.H + h) * HEAD_ELEMS + v * D + k0;
  const int64_t step = int64_t(p.H) * kOps;
  uint8_t* ops0 = p.ops + ((int64_t(doc) + t0 / C) * p.H + h) * int64_t(kOps);

  f32x4 s[NM];  // [key k0 + 16 m + i][value v]
#pragma unroll
  for (int m = 0; m < NM; ++m) s[m] = zero4();

  // tile A's fragments of this wave's keys, tile B's of its state tiles
  const int at_a = kh * (NM * 1024) + lane * 16, at_b = kh * (NM * 4096) + lane * 16;
  auto frag = [](const uint8_t* base, int unit) {
    return *reinterpret_cast<const f16x8*>(base + unit * 1024);
  };
  constexpr int OA = OWN ? NB * NM : 1, OB = OWN ? NM * 4 : 1;
  f16x8 own_a[OA], own_b[OB], own_q[OB];
  auto frag_a = [&](int r, int t, int low) {
    if constexpr (OWN) return own_a[r * NM + t * 2 + low];
    else return frag(la + at_a, r * 8 + t * 2 + low);
  };
  auto frag_b = [&](int m, int t, int low) {
    if constexpr (OWN) return own_b[m * 4 + t * 2 + low];
    else return frag(lb + at_b, m * 4 + t * 2 + low);
  };
  auto frag_q = [&](int m, int t, int low) {
    if constexpr (OWN) return own_q[m * 4 + t * 2 + low];
    else return frag(lb + at_b, 32 + m * 4 + t * 2 + low);
  };
  auto load_own_a = [&](const uint8_t* src, int r) {
#pragma unroll
    for (int i = 0; i < NM; ++i)
      if constexpr (OWN) own_a[r * NM + i] = frag(src + at_a, r * 8 + i);
  };
  auto load_own_b = [&](f16x8 (&b)[OB], const uint8_t* src, int m) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (OWN) b[m * 4 + i] = frag(src + at_b, m * 4 + i);
  };
  Stage<NA, T> sa;  // the next tile A, and its chunk's tail
  u32x4 st = {0u, 0u, 0u, 0u};
  auto tail_of = [&](int n) { return tails + (OWN ? n % 3 : n & 1) * 256; };
  auto xch_of = [&](int n) { return xch0 + (OWN ? (n & 1) * (Shape::kXch / 4) : 0); };
  // the first tile A (later ones come in shares, a token block at a time)
  auto load_a = [&](const uint8_t* src) {
    if constexpr (OWN) {
#pragma unroll
      for (int r = 0; r < NB; ++r) load_own_a(src, r);
    } else {
      sa.load(src);
    }
  };
  // this wave's part of x: the sum over its keys of tile A times the state
  auto product = [&](const Right<NM>& b, f32x4 (&acc)[NB], const uint8_t* next) {
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      acc[r] = zero4();
#pragma unroll
      for (int t = 0; t < NM / 2; ++t) {
        const f16x8 ah = frag_a(r, t, 0), al = frag_a(r, t, 1);
        acc[r] = mfma32(al, b.hi[t], acc[r]);
        acc[r] = mfma32(ah, b.lo[t], acc[r]);
        acc[r] = mfma32(ah, b.hi[t], acc[r]);
      }
      if constexpr (OWN) {
        load_own_a(next, r);
        __builtin_amdgcn_sched_barrier(0);
      } else {
        sa.template load_share<NB>(next, r);
      }
    }
  };
  // x = x0 + un * (what `product` left), rows written: the waves of a tile add up their
  // parts (x0 and the rows are shared between them, a part of the blocks each).
  auto exchange_out = [&](f32x4 (&x)[NB], const f32x4 (&acc)[NB], float un, f32x4 unr,
                          const f32x4 (&x0)[NX], float* xch) {
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      x[r] = acc[r] * (un * unr[r]);
      if (r / NX == kh) x[r] += x0[r % NX];
      *reinterpret_cast<f32x4*>(xch + ((wave * NB + r) * 64 + lane) * 4) = x[r];
    }
  };
  auto exchange_in = [&](f32x4 (&x)[NB], float* rows, const float* xch) {
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      x[r] += lds4(xch + (((wave ^ 1) * NB + r) * 64 + lane) * 4);
      if constexpr (KS == 4)  // (pairs first: the same sum in all four)
        x[r] += lds4(xch + (((wave ^ 2) * NB + r) * 64 + lane) * 4) +
                lds4(xch + (((wave ^ 3) * NB + r) * 64 + lane) * 4);
      if (r / NX == kh)
        *reinterpret_cast<f32x4*>(rows + 16 * r * D + at_row) = quad_transpose(x[r], lane);
    }
  };
  auto store_state = [&](float* rows) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
      *reinterpret_cast<f32x4*>(rows + 16 * (NM * kh + m) * D + at_row) =
          quad_transpose(s[m], lane);
  };
  // the start of x of chunk n, this wave's token blocks
  auto load_x0 = [&](f32x4 (&x0)[NX], int n, int op) {
    const float* src = reinterpret_cast<const float*>(ops0 + n * step + op) +
                       ((v >> 4) * NB * 64 + lane) * 4;
#pragma unroll
    for (int r = 0; r < NX; ++r) x0[r] = lds4(src + (NX * kh + r) * 256);
  };
  auto load_tail = [&](int n) {
    if (wave == 0) st = *reinterpret_cast<const u32x4*>(ops0 + n * step + lane * 16);
  };
  auto store_tail = [&](int n) {
    if (wave == 0) *reinterpret_cast<u32x4*>(tail_of(n) + lane * 4) = st;
  };
  auto store_a = [&](int n) {
    sa.store(la);
    store_tail(n);
  };

  if (!down) {
    if (!active || len == 0) return;
    if (p.use_initial) {
      const int64_t e = int64_t(slot) * p.slot_stride + int64_t(h) * HEAD_ELEMS + v * D + k0;
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[m][i] = pool_at(p, e + 16 * m + i);
    }
    Stage<NA, T> sb;
    f32x4 x0[NX];  // of the next chunk, asked for a phase ahead
    load_a(ops0 + kOpW);
    load_tail(0);
    load_x0(x0, 0, kOpX0);
    if constexpr (OWN) {
      store_tail(0);
#pragma unroll
      for (int m = 0; m < NM; ++m) load_own_b(own_b, ops0 + kOpKE, m);
    } else {
      store_a(0);
      sb.load(ops0 + kOpKE);
    }
    __syncthreads();
    for (int n = 0; n < chunks; ++n) {
      uint8_t* ops = ops0 + n * step;
      const bool more = n + 1 < chunks;
      const uint8_t* after = more ? ops + step : ops;  // (the last chunk asks for itself again)
      const float* tail = tail_of(n);
      f32x4 x[NB];
      // ---- x = T V - W S
      load_tail(more ? n + 1 : n);
      {
        Right<NM> b;
        f32x4 acc[NB];
        b.set(s);
        product(b, acc, after + kOpW);
        store_state(reinterpret_cast<float*>(ops + kOpS));
        exchange_out(x, acc, -b.un, lds4(tail + kTailUnW), x0, xch_of(n));
      }
      if constexpr (OWN)
        store_tail(n + 1);
      else if (more)
        sb.store(lb);
      __syncthreads();
      exchange_in(x, reinterpret_cast<float*>(ops + kOpX), xch_of(n));
      if (!more) return;  // the state after the last chunk is not needed
      // ---- S = e^Gl S + KE^T (beta x)
      Right<NB> b;
#pragma unroll
      for (int r = 0; r < NB; ++r)
        x[r] *= lds4(tail + kTailBeta + 16 * r + 4 * g4) * tail[kTailDnKE + r];
      b.set(x);
      load_x0(x0, n + 1, kOpX0);
      const float un = b.un * kFixedUn;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        f32x4 acc = zero4();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const f16x8 ah = frag_b(m, t, 0), al = frag_b(m, t, 1);
          acc = mfma32(al, b.hi[t], acc);
          acc = mfma32(ah, b.lo[t], acc);
          acc = mfma32(ah, b.hi[t], acc);
        }
        if constexpr (OWN) {
          load_own_b(own_b, after + kOpKE, m);
          __builtin_amdgcn_sched_barrier(0);
        } else {
          sb.template load_share<NM>(after + kOpKE, m);
        }
        s[m] *= lds4(tail + k0 + 16 * m);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[m][i] = fmaf(acc[i], un, s[m][i]);
      }
      if constexpr (!OWN) {
        store_a(n + 1);
        __syncthreads();
      }
    }
    return;
  }

  if (p.d_final && active) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[m][i] = p.d_final[state + 16 * m + i];
  }
  if (active && chunks > 0) {
    Stage<2 * NA, T> sb;
    f32x4 x0[NX];
    f16x8 ow[2];  // dO: 64 tokens of this lane's value, a right fragment
    float uow;
    auto load_o = [&](int n) {
      const uint8_t* src = ops0 + n * step + kOpO + ((v >> 4) * 2 * 64 + lane) * 16;
#pragma unroll
      for (int t = 0; t < 2; ++t) ow[t] = frag(src, t);
      uow = reinterpret_cast<const float*>(ops0 + n * step + kOpUnO)[v];
    };
    load_a(ops0 + (chunks - 1) * step + kOpZ);
    load_tail(chunks - 1);
    load_x0(x0, chunks - 1, kOpDV0);
    load_o(chunks - 1);
    if constexpr (OWN) {
      store_tail(chunks - 1);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        load_own_b(own_b, ops0 + (chunks - 1) * step + kOpKG, m);
        load_own_b(own_q, ops0 + (chunks - 1) * step + kOpQG, m);
      }
    } else {
      store_a(chunks - 1);
      sb.load(ops0 + (chunks - 1) * step + kOpKG);
    }
    __syncthreads();
    for (int n = chunks - 1; n >= 0; --n) {
      uint8_t* ops = ops0 + n * step;
      const uint8_t* after = n > 0 ? ops - step : ops;
      const float* tail = tail_of(n);
      f32x4 x[NB];
      // ---- dV = T^T P^T dO + Z dS
      load_tail(n > 0 ? n - 1 : 0);
      {
        Right<NM> b;
        f32x4 acc[NB];
        b.set(s);
        product(b, acc, after + kOpZ);
        store_state(reinterpret_cast<float*>(ops + kOpDS));
        exchange_out(x, acc, b.un, lds4(tail + kTailUnZ), x0, xch_of(n));
      }
      const bool more = n > 0 || p.d_initial;
      if constexpr (OWN) {
        if (n > 0) store_tail(n - 1);
      } else if (more) {
        sb.store(lb);
      }
      __syncthreads();
      exchange_in(x, reinterpret_cast<float*>(ops + kOpDV), xch_of(n));
      if (!more) return;
      // ---- dS = e^Gl dS - KG^T dV + scale QG^T dO. dO has 8 bits: its high part is exact.
      Right<NB> b;
      const f32x4 dn = lds4(tail + kTailDnKG);
#pragma unroll
      for (int r = 0; r < NB; ++r) x[r] *= dn[r];
      b.set(x);
      const f16x8 o[2] = {ow[0], ow[1]};
      const float un = -b.un * kFixedUn, uno = uow * (p.scale * kFixedUn);
      load_x0(x0, n > 0 ? n - 1 : 0, kOpDV0);
      load_o(n > 0 ? n - 1 : 0);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        f32x4 acc = zero4(), acc2 = zero4();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const f16x8 ah = frag_b(m, t, 0), al = frag_b(m, t, 1);
          const f16x8 qh = frag_q(m, t, 0), ql = frag_q(m, t, 1);
          acc = mfma32(al, b.hi[t], acc);
          acc2 = mfma32(ql, o[t], acc2);
          acc = mfma32(ah, b.lo[t], acc);
          acc2 = mfma32(qh, o[t], acc2);
          acc = mfma32(ah, b.hi[t], acc);
        }
        if constexpr (OWN) {
          load_own_b(own_b, after + kOpKG, m);
          load_own_b(own_q, after + kOpQG, m);
          __builtin_amdgcn_sched_barrier(0);
        } else {
          sb.template load_share<NM>(after + kOpKG, m);
        }
        s[m] *= lds4(tail + k0 + 16 * m);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[m][i] = fmaf(acc2[i], uno, fmaf(acc[i], un, s[m][i]));
      }
      if constexpr (!OWN) {
        if (n > 0) store_a(n - 1);
        __syncthreads();
      }
    }
  }
  if (p.d_initial) {
#pragma unroll
    for (int m = 0; m < NM; ++m) *reinterpret_cast<f32x4*>(p.d_initial + state + 16 * m) = s[m];
  }
}

// Of `docs` documents from the order's `first` on, the chain and part of block `bid`. Chain
// c's parts are blocks (c / 8 * PARTS + part) * 8 + c % 8: blocks go to the eight XCDs in
// turn, so the parts share one L2 copy of the operands.
template <int KS, int TW>
__device__ __forceinline__ void chain_of_block(const BwdParams& p, const DocOrder& ord, int64_t bid,
                                               int first, int docs) {
  constexpr int PARTS = ChainShape<KS, TW>::kParts;
  const int64_t id = bid / (8 * PARTS) * 8 + (bid & 7);
  const int64_t c = id >> 1;
  if (c >= int64_t(docs) * p.H) return;
  const int rank = first + int(c / p.H);
  const int doc = ord.n > 0 ? ord.doc[rank] : rank;
  chain<KS, TW>(p, doc, int(c % p.H), id & 1, int((bid >> 3) % PARTS));
}
template <int KS, int TW>
__host__ __device__ int64_t blocks_of(int64_t docs, int H) {
  return (docs * H * 2 + 7) / 8 * 8 * ChainShape<KS, TW>::kParts;
}

using Few = ChainShape<4, 1>;
using Deep = ChainShape<4, 2>;
using Wide = ChainShape<2, 4>;

__global__ __launch_bounds__(Few::kThreads) void chain_few_kernel(BwdParams p, DocOrder ord) {
  chain_of_block<4, 1>(p, ord, blockIdx.x, 0, p.n_docs);
}

static_assert(Deep::kThreads == Wide::kThreads && Deep::kLds == Wide::kLds, "one launch for both");

__global__ __launch_bounds__(Wide::kThreads) void chain_kernel(BwdParams p, DocOrder ord) {
  const int64_t bid = int64_t(blockIdx.x) - blocks_of<4, 2>(ord.deep, p.H);
  if (bid < 0)
    chain_of_block<4, 2>(p, ord, blockIdx.x, 0, ord.deep);
  else
    chain_of_block<2, 4>(p, ord, bid, ord.deep, p.n_docs - ord.deep);
}

}  // namespace

// One tile per workgroup as long as all of them run at once, one per CU (8191 tokens, us:
// 12 heads 722 against 832 with two tiles; 4096 tokens, 24 heads 670 against 618). Beyond that four
// tiles, which read the operands least often; but the longest documents' chains, where one
// of them would outlast its share of all the work, two tiles of four waves
// (14 documents, 12 heads: 1056 against 1086).
hipError_t launch_chains(const BwdParams& p, const DocOrder& ord, hipStream_t stream) {
  if (blocks_of<4, 1>(p.n_docs, p.H) <= kCus) {
    static std::atomic<bool> allowed[kMaxDevices];
    const void* kernel = reinterpret_cast<const void*>(chain_few_kernel);
    if (const hipError_t e = allow_lds(kernel, Few::kLds, allowed))
      return e;
    hipLaunchKernelGGL(chain_few_kernel, dim3(unsigned(blocks_of<4, 1>(p.n_docs, p.H))),
                       dim3(Few::kThreads), Few::kLds, stream, p, ord);
    return hipGetLastError();
  }
  static std::atomic<bool> allowed[kMaxDevices];
  const void* kernel = reinterpret_cast<const void*>(chain_kernel);
  if (const hipError_t e = allow_lds(kernel, Wide::kLds, allowed))
    return e;
  const int64_t blocks = blocks_of<4, 2>(ord.deep, p.H) + blocks_of<2, 4>(p.n_docs - ord.deep, p.H);
  hipLaunchKernelGGL(chain_kernel, dim3(unsigned(blocks)), dim3(Wide::kThreads), Wide::kLds, stream,
                     p, ord);
  return hipGetLastError();
}

// Deep chains' blocks run at once, one per CU (48 heads of 4096 tokens, all of them too long
// for their share: 1194 us with twice as many blocks as fit, 1040 wide).
bool deep_chains(int64_t total_tokens, int H, int rank, int len) {
  return len > total_tokens * H * 2 * Wide::kParts / kCus && blocks_of<4, 2>(rank + 1, H) <= kCus;
}

}  // namespace bwd
}  // namespace kda
