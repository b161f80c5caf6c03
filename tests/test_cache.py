"""kda_cache_write, kda_cache_read and kda_cache_attention: host validation (CPU) and parity
with the definitions in 64 bits (GPU).

Tolerances. Bytes, scales and values read back are exact: scales are powers of two, so every
division and product is, and the one rounding is to the nearest code (even on a tie).

Attention. Products of bf16 and widened codes are exact in fp32; a score sums 128 of them and
takes two more roundings, so it is off by at most d = 131 * 2^-24 * |scale| sum |q k|, and its
weight by that relatively, plus 2^-22 for the exponential. A sum of n weights adds n * 2^-24
at most, and so does each output sum. The weights enter the second product with a relative
error of `weight`: 2^-16 as two bf16 parts (up to 128 rows, tokens times query heads of a
key/value head), half a step of bf16, 2^-8, as one (more rows). So out is off by at most
half a step of bf16, 2^-8 |out|, and (weight + 2 d + 2 n 2^-24 + 2^-20) times the mean of |v|
under the weights; lse by d + n 2^-24 + 2^-21 (1 + |lse|). A weight under 2^-126 of the largest one's
range may be flushed to zero, fp32's smallest normal number (the reference exponent is at most
the largest score's, so the sum that divides it is at least 1), and a part of one bf16 pair under
2^-126 too: n 2^-125 max |v| more.
"""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import gated_delta_rule_step_amd as kda

OK, NULLP, SHAPE, STRIDE, UNSUP, SEQ, WS = range(7)
BF, F8, I8, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.int32
KINDS = [F8, I8]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_step_amd import build
        build.build()
    return kda.lib()


# ---------------------------------------------------------------------------
# refusals: every call returns before anything is launched (made-up pointers)

def _args(**kw):
    a = dict(n=2, T=6, H=3, D=128, cu=0, k=4096, ks=384, v=4096, vs=384, dt=0, P=16, N=5, kc=4096,
             kp=6144, vc=4096, vp=6144, ksc=4096, vsc=4096, tab=4096, w=4, ts=4, lens=4096)
    a.update(kw)
    return a


def _rows_call(lib, fn, **kw):
    a, P = _args(**kw), ctypes.c_void_p
    return getattr(lib, fn)(a["n"], a["T"], a["H"], a["D"], P(a["cu"]), P(a["k"]), a["ks"],
                            P(a["v"]), a["vs"], a["dt"], a["P"], a["N"], P(a["kc"]), a["kp"],
                            P(a["vc"]), a["vp"], P(a["ksc"]), P(a["vsc"]), P(a["tab"]), a["w"],
                            a["ts"], P(a["lens"]), P(0))


COMMON = [
    (SHAPE, dict(n=-1)), (SHAPE, dict(T=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(N=-1)),
    (SHAPE, dict(w=0)), (SHAPE, dict(T=7)), (SHAPE, dict(n=0)), (UNSUP, dict(D=64)),
    (UNSUP, dict(dt=2)), (UNSUP, dict(dt=-1)), (UNSUP, dict(P=8)), (UNSUP, dict(P=24)),
    (UNSUP, dict(P=512)), (UNSUP, dict(P=0)), (UNSUP, dict(H=1 << 15)),
    (UNSUP, dict(N=1 << 31)), (UNSUP, dict(n=1 << 20, T=1 << 20, w=1 << 14, ts=1 << 14)),
    (UNSUP, dict(n=1 << 19, T=1 << 19, w=1 << 13, ts=1 << 13)),
    (UNSUP, dict(n=1 << 24, T=1 << 24, w=1, ts=1)), (UNSUP, dict(H=8193, kp=8193 * 2048, vp=8193 * 2048)),
    (UNSUP, dict(T=(1 << 30) + 2)), (UNSUP, dict(kc=4100)), (UNSUP, dict(vp=6148)),
    (STRIDE, dict(ts=-1)), (STRIDE, dict(ts=3)), (STRIDE, dict(kp=6128)), (STRIDE, dict(vp=-16)),
    (NULLP, dict(tab=0)), (NULLP, dict(lens=0)), (NULLP, dict(kc=0)), (NULLP, dict(vc=0)),
    (NULLP, dict(ksc=0)), (NULLP, dict(vsc=0)),
]


@pytest.mark.parametrize("want,kw", COMMON + [
    (STRIDE, dict(ks=-1)), (STRIDE, dict(vs=-384)), (NULLP, dict(k=0)), (NULLP, dict(v=0)),
    (OK, dict(T=0, k=0, v=0, tab=0, lens=0, kc=0)), (OK, dict(n=0, T=0)),
    (OK, dict(N=0, kc=0, vc=0, ksc=0, vsc=0)),
])
def test_write_refusals(lib, want, kw):
    assert _rows_call(lib, "kda_cache_write", **kw) == want


@pytest.mark.parametrize("want,kw", COMMON + [
    (STRIDE, dict(ks=383)), (STRIDE, dict(vs=100)), (STRIDE, dict(ks=-1)), (NULLP, dict(k=0)),
    (NULLP, dict(v=0)), (OK, dict(T=0, k=0, v=0, tab=0, lens=0)),
])
def test_read_refusals(lib, want, kw):
    assert _rows_call(lib, "kda_cache_read", **kw) == want


def _attend(lib, host=None, **kw):
    a, P = _args(Hq=6, q=4096, qs=768, o=4096, os=768, lse=0, ls=6, sc=0.1, ws=4096, wb=1 << 40,
                 cuh=0), ctypes.c_void_p
    a.update(kw)
    if host is not None:
        host = (ctypes.c_int32 * len(host))(*host)
        a["cuh"], a["cu"] = ctypes.addressof(host), a["cu"] or 4096
    return lib.kda_cache_attention(
        a["n"], a["T"], a["Hq"], a["H"], a["D"], P(a["cuh"]), P(a["cu"]), P(a["q"]), a["qs"],
        a["dt"], a["P"], a["N"], P(a["kc"]), a["kp"], P(a["vc"]), a["vp"], P(a["ksc"]),
        P(a["vsc"]), P(a["tab"]), a["w"], a["ts"], P(a["lens"]), a["sc"], P(a["o"]), a["os"],
        P(a["lse"]), a["ls"], P(a["ws"]), a["wb"], P(0))


@pytest.mark.parametrize("want,kw", [x for x in COMMON if "H" not in x[1]] + [
    (SHAPE, dict(Hq=0)), (SHAPE, dict(Hq=7)), (SHAPE, dict(H=0)), (SHAPE, dict(H=-3)),
    (UNSUP, dict(Hq=771)), (UNSUP, dict(sc=float("nan"))), (UNSUP, dict(sc=float("inf"))),
    (UNSUP, dict(sc=3e38)), (UNSUP, dict(H=8193, Hq=8193)),
    (UNSUP, dict(n=1 << 23, T=1 << 23, w=1, ts=1)), (UNSUP, dict(ws=4100)), (WS, dict(wb=3)), (NULLP, dict(ws=0)), (NULLP, dict(q=0)),
    (NULLP, dict(o=0)), (NULLP, dict(cu=4096)), (STRIDE, dict(qs=-1)), (STRIDE, dict(os=767)),
    (STRIDE, dict(lse=4096, ls=5)), (STRIDE, dict(lse=4096, ls=-6)),
    (SEQ, dict(host=[1, 2, 3])), (SEQ, dict(host=[0, 3, 2])), (SEQ, dict(host=[0, 3, 7])),
    (OK, dict(host=[0, 0, 0])), (OK, dict(T=0, q=0, o=0, ws=0, wb=0)),
])
def test_attention_refusals(lib, want, kw):
    assert _attend(lib, **kw) == want


def test_workspace_size(lib):
    size = kda.kda_cache_attention_workspace_size
    assert size(0, 4, 8, 8) == 0 and size(1, 0, 8, 8) == 0
    assert size(1, 1, 8193, 8193) == 0 < size(1, 1, 8192, 8192)
    assert size(1, 1, 7, 2) == 0 and size(1, 1, 0, 0) == 0 and size(1, 1, 514, 2) == 0
    for heads in ((12, 12), (64, 8), (6, 2), (40, 1)):
        got = [size(n, n, *heads) for n in (1, 2, 63, 512, 5000)]
        assert got == sorted(got) and got[0] > 0
        got = [size(3, n, *heads) for n in (1, 2, 8, 17, 64, 1000, 1 << 20)]
        assert got == sorted(got)  # one buffer serves every smaller call


def test_binding_refuses(lib):
    c = torch.zeros(3, 2, 16, 128, dtype=I8)
    s, tab, lens = torch.ones(3, 2), torch.zeros(1, 3, dtype=I32), torch.ones(1, dtype=I32)
    k = torch.zeros(1, 256, dtype=BF)
    with pytest.raises(ValueError):  # not on a GPU
        kda.kda_cache_write(k, k, c, c, s, s, tab, lens)
    with pytest.raises(TypeError):
        kda.kda_cache_write(k, k, c.float(), c.float(), s, s, tab, lens)
    with pytest.raises(ValueError):
        kda.kda_cache_read(k, k, c[0], c[0], s, s, tab, lens)


# ---------------------------------------------------------------------------
# definitions in 64 bits (CPU)

def _value(codes, kind):
    if kind == I8:
        return codes.double()
    b = codes.view(torch.uint8).long()
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 512)
    x = torch.where((b & 127) == 127, torch.nan, x)
    return torch.where(b >= 128, -x, x)


def _nearest(x, kind):
    if kind == I8:
        return torch.nan_to_num(x.round().clamp(-127, 127), nan=0.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(2.0 ** -6, 512))) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _need(x, kind):
    """The scale for rows x [H, tokens, 128], by trial: no logarithm rounds here."""
    a = torch.where(x.isfinite(), x.abs(), 0.0).amax((1, 2))
    out = []
    for top in a.tolist():
        e = -100
        while top > (448.0 if kind == F8 else 127.0) * 2.0 ** e:
            e += 1
        out.append(2.0 ** e)
    return torch.tensor(out, dtype=torch.float64)


class Pool:
    """A cache with everything that no sequence owns poisoned, and its mirror in 64 bits:
    `code` [2][N, H, P, 128] and `scale` [2][N, H]."""

    def __init__(self, kind, H, P, totals, seed=0, spare=3, pad=0, width=None):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.H, self.P, self.g = kind, H, P, g
        used = [-(-max(x, 0) // P) for x in totals]
        self.N = N = sum(used) + spare
        self.width = width or max(used + [1])
        order = torch.randperm(N, generator=g).tolist()
        self.table = torch.full((len(totals), self.width), 2 ** 31 - 1, dtype=torch.int64)
        for b, n in enumerate(used):
            for j in range(min(n, self.width)):
                self.table[b, j] = order.pop()
        poison = 0x7f if kind == F8 else 77
        size = H * P * 128 + pad
        self.raw = [torch.full((N * size + 16,), poison, dtype=torch.uint8) for _ in range(2)]
        self.shape, self.strides = (N, H, P, 128), (size, P * 128, 128, 1)
        self.scale = [torch.full((N, H), torch.nan) for _ in range(2)]
        self.lens = torch.tensor(totals, dtype=torch.int64)

    def fill(self, tokens=None):
        """Random codes and scales for each sequence's first tokens (all: None)."""
        for side in range(2):
            c = self.codes(self.raw)[side]
            for b, n in enumerate(self.lens.tolist() if tokens is None else tokens):
                for j in range(-(-max(n, 0) // self.P)):
                    page = self.table[b, j].item()
                    if not 0 <= page < self.N:
                        continue
                    z = min(self.P, n - j * self.P)
                    x = torch.randn(self.H, z, 128, generator=self.g) * \
                        (40.0 if self.kind == F8 else 35.0)
                    y = x.clamp(-448, 448).to(F8) if self.kind == F8 else \
                        x.round().clamp(-127, 127).to(I8)
                    c[page, :, :z] = y.view(torch.uint8)
                    self.scale[side][page] = torch.exp2(
                        torch.randint(-7, -4, (self.H,), generator=self.g).float())
        return self

    def codes(self, raw):
        return [r.as_strided(self.shape, self.strides) for r in raw]

    def gpu(self):
        """k_cache, v_cache, k_scale, v_scale, page_table, kv_lens for a call."""
        self.dev = [r.cuda() for r in self.raw]
        caches = [c.view(self.kind) for c in self.codes(self.dev)]
        self.dev_scale = [s.cuda() for s in self.scale]
        return (*caches, *self.dev_scale, self.table.to(I32).cuda(), self.lens.to(I32).cuda())

    def tokens(self, side, b, n):
        """Values of positions 0 .. n - 1 [n, H, 128], and whether they exist."""
        x = torch.zeros(max(n, 0), self.H, 128, dtype=torch.float64)
        real = torch.zeros(max(n, 0), dtype=torch.bool)
        c = self.codes(self.raw)[side]
        for j in range(-(-max(n, 0) // self.P)):
            page, z = self.table[b, j].item(), min(self.P, n - j * self.P)
            if 0 <= page < self.N:
                y = _value(c[page, :, :z].contiguous().view(self.kind), self.kind)
                x[j * self.P:j * self.P + z] = \
                    (y * self.scale[side][page].double()[:, None, None]).transpose(0, 1)
                real[j * self.P:j * self.P + z] = True
        return x, real

    def cap(self):
        return self.width * self.P


def _ref_attention(pool, q, counts, G, scale, weight):
    """out, lse and their tolerances [T, Hq, ..]; q fp64 [T, Hq, 128]."""
    T, Hq = q.shape[:2]
    out, tol = torch.zeros(T, Hq, 128, dtype=torch.float64), torch.zeros(T, Hq, 128).double()
    lse, lt = torch.full((T, Hq), -torch.inf).double(), torch.zeros(T, Hq).double()
    at = 0
    for b, n in enumerate(counts):
        total = pool.lens[b].item()
        active = n > 0 and n <= total <= pool.cap()
        if active:
            keys, there = pool.tokens(0, b, total)
            values, _ = pool.tokens(1, b, total)
        for i in range(n):
            row, see = at + i, total - n + i + 1
            if not active or not there[:see].any():
                continue
            k, v, real = keys[:see], values[:see], there[:see]
            for h in range(Hq):
                kh, vh = k[real][:, h // G], v[real][:, h // G]
                s = scale * (kh @ q[row, h])
                d = 131 * 2.0 ** -24 * abs(scale) * (kh.abs() @ q[row, h].abs()).max()
                lse[row, h] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[row, h])
                out[row, h] = p @ vh
                m = len(s)
                tol[row, h] = 2.0 ** -8 * out[row, h].abs() + \
                    (weight + 2 * d + m * 2.0 ** -23 + 2.0 ** -20) * (p @ vh.nan_to_num(0.0).abs()) + \
                    m * 2.0 ** -125 * vh.abs().nan_to_num(0.0).max()
                lt[row, h] = d + m * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[row, h].abs())
        at += n
    return out, lse, tol, lt


def _close(got, want, tol):
    got, want = got.double().cpu(), want
    fine = (got - want).abs() <= tol
    same = (got == want) | (got.isnan() & want.isnan())  # infinities, NaN
    off = int((~(fine | same)).sum())
    assert off == 0, f"{off} of {got.numel()} off, worst {(got - want).abs().max()}"


def _cu(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=I32)


def _strided(t, pad, offset):
    """The same values on the GPU, rows `pad` elements further apart, from `offset` on."""
    n = t.shape[1]
    buf = torch.full((offset + max(t.shape[0], 1) * (n + pad),), -7.0, dtype=t.dtype,
                     device="cuda")
    view = buf[offset:].as_strided(tuple(t.shape), (n + pad, 1))
    view.copy_(t)
    return view, buf


# ---------------------------------------------------------------------------
# writing and reading

def _ref_write(pool, x, counts):
    """The definition, page by page, into pool.raw and pool.scale. x: [2][T, H, 128] fp64."""
    for side in range(2):
        c, at = pool.codes(pool.raw)[side], 0
        for b, n in enumerate(counts):
            end = pool.lens[b].item()
            first, at = at, at + n
            if end < n or end > pool.cap():
                continue
            pos = end - n
            while pos < end:
                page, a = pool.table[b, pos // pool.P].item(), pos % pool.P
                z = min(pool.P, a + end - pos)
                rows = x[side][first:first + z - a].transpose(0, 1)
                first, pos = first + z - a, pos + z - a
                if not 0 <= page < pool.N:
                    continue
                s = _need(rows, pool.kind)
                if a:
                    old = pool.scale[side][page].double()
                    s = torch.maximum(s, old)
                    y = _value(c[page, :, :a].contiguous().view(pool.kind), pool.kind)
                    y = torch.where((s > old)[:, None, None],
                                    _nearest(y * (old / s)[:, None, None], pool.kind), y)
                    c[page, :, :a] = y.float().to(pool.kind).view(torch.uint8)
                y = _nearest(rows / s[:, None, None], pool.kind).float()
                c[page, :, a:z] = y.to(pool.kind).view(torch.uint8)
                pool.scale[side][page] = s.float()


def _tokens(T, H, g, spread=3):
    """Keys or values whose size changes from token to token and head to head."""
    x = torch.randn(T, H, 128, generator=g)
    return (x * torch.exp2(torch.randint(-spread, spread + 1, (T, H, 1), generator=g).float())).to(BF)


def _check_write(pool, k, v, counts, uniform, pad=0, offset=0):
    H, T = pool.H, k.shape[0]
    cache = pool.gpu()
    kd, _ = _strided(k.reshape(T, -1), pad, offset)
    vd, _ = _strided(v.reshape(T, -1), 2 * pad, offset)
    kda.kda_cache_write(kd, vd, *cache, cu_seqlens=None if uniform else _cu(counts).cuda())
    _ref_write(pool, [k.double(), v.double()], counts)
    for side in range(2):
        got = pool.dev[side].cpu()
        if pool.kind == F8:  # a NaN has two codes
            nan = ((got & 127) == 127) & ((pool.raw[side] & 127) == 127)
            assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, pool.raw[side]))
        else:
            assert torch.equal(got, pool.raw[side])
        assert torch.equal(pool.dev_scale[side].cpu().nan_to_num(-1), pool.scale[side].nan_to_num(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T", [1, 4, 5, 17, 70, 300])
def test_write_uniform(lib, kind, P, T):
    totals = [T, T + 1, T + P - 1, T + P, T + 2 * P + 3]
    pool = Pool(kind, 3, P, totals, seed=T, pad=16).fill([x - T for x in totals])
    g = torch.Generator().manual_seed(P)
    _check_write(pool, _tokens(T * 5, 3, g), _tokens(T * 5, 3, g), [T] * 5, True, pad=6, offset=3)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("H", [1, 5])
def test_write_ragged(lib, kind, P, H):
    counts = [0, 1, 300, 0, 16, 15, 33, 0, 129, 2]
    past = [5, 0, 9, 0, 64, 17, 0, 3, 255, 31]
    totals = [a + b for a, b in zip(counts, past)]
    pool = Pool(kind, H, P, totals, seed=1).fill(past)
    g = torch.Generator().manual_seed(P + H)
    T = sum(counts) + 3  # rows behind the last sequence
    _check_write(pool, _tokens(T, H, g), _tokens(T, H, g), counts, False)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [32, 64, 128, 256])
@pytest.mark.parametrize("H", [1, 5, 8])
def test_mixed_batch_written_and_read(lib, kind, P, H):
    """Single tokens and drafts beside documents, some behind earlier tokens, some inactive."""
    counts = [1] * 40
    past = torch.randint(0, 2 * P, (40,), generator=torch.Generator().manual_seed(P)).tolist()
    for b, n in ((0, 0), (3, 17), (4, 8), (9, 300), (10, 16), (21, 0), (22, 70), (39, 33)):
        counts[b] = n
    pool = Pool(kind, H, P, [a + b for a, b in zip(counts, past)], seed=9).fill(past)
    pool.lens[5], pool.lens[12] = 0, pool.cap() + 1
    g = torch.Generator().manual_seed(H)
    T = sum(counts)
    _check_write(pool, _tokens(T, H, g), _tokens(T, H, g), counts, False, pad=6, offset=3)
    got = [torch.full((T + 2, H * 128), -7.0, dtype=BF, device="cuda") for _ in range(2)]
    kda.kda_cache_read(*got, *pool.gpu(), cu_seqlens=_cu(counts).cuda())
    for side in range(2):
        want, at = torch.zeros(T, H, 128, dtype=torch.float64), 0
        for b, n in enumerate(counts):
            total = pool.lens[b].item()
            if n <= total <= pool.cap():
                want[at:at + n] = pool.tokens(side, b, total)[0][total - n:]
            at += n
        assert torch.equal(got[side][:T].double().cpu().reshape(T, H, 128), want)
        assert (got[side][T:] == -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [63, 64, 65, 130, 4100])
def test_write_many_sequences(lib, n):
    g = torch.Generator().manual_seed(n)
    counts = torch.randint(0, 4, (n,), generator=g).tolist()
    past = torch.randint(0, 40, (n,), generator=g).tolist()
    pool = Pool(F8, 1, 16, [a + b for a, b in zip(counts, past)], seed=2).fill(past)
    T = sum(counts)
    _check_write(pool, _tokens(T, 1, g), _tokens(T, 1, g), counts, False)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_write_bad_values_and_sequences(lib, kind):
    """Infinities, NaN, zeros, the smallest and largest values; inactive sequences; pages
    that do not exist."""
    totals = [40, 0, 7, 5000, -3, 20, 33]
    counts = [33, 2, 8, 4, 1, 20, 3]
    pool = Pool(kind, 2, 16, [40, 0, 16, 48, 0, 20, 33], seed=3, width=3).fill()
    pool.lens = torch.tensor(totals)
    pool.table[0, 1] = -1
    pool.table[5, 0] = pool.N
    g = torch.Generator().manual_seed(4)
    T = sum(counts)
    k, v = _tokens(T, 2, g), _tokens(T, 2, g)
    k[0] = 0.0
    k[5, 0, 3], k[6, 1, 0], v[30, 0, 127] = torch.inf, -torch.inf, torch.nan
    v[31, 1, 0], k[-1], v[-1, 0] = 3.3e38, 1e-40, 2.0 ** -133
    k[-2], v[-2], k[-3], v[-3] = 0.0, 0.0, 0.0, -0.0
    _check_write(pool, k, v, counts, False)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 30])
def test_write_behind_scales_of_other_makers(lib, kind, n):
    """Earlier tokens under zero, negative and odd scales, below what the new tokens need."""
    pool = Pool(kind, 3, 64, [13 + n, 64 + 5 + n], seed=7).fill([13, 69])
    for side in range(2):
        for page in (pool.table[0, 0], pool.table[1, 1]):
            pool.scale[side][page] = torch.tensor([0.0, -2.0 ** -6, 1.5 * 2.0 ** -9])
    g = torch.Generator().manual_seed(8)
    k, v = _tokens(2 * n, 3, g), _tokens(2 * n, 3, g)
    k[0], k[n], v[0], v[n] = 9.0, -5.0, 7.0, 30.0
    _check_write(pool, k, v, [n, n], True)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 128])
def test_write_token_by_token(lib, kind, P):
    """A decode loop: scales grow, earlier codes follow, as the definition says call by call."""
    g = torch.Generator().manual_seed(5)
    pool = Pool(kind, 2, P, [40, 23], seed=6)
    pool.lens = torch.zeros(2, dtype=torch.int64)
    cache = pool.gpu()
    for t in range(23):
        pool.lens = torch.tensor([t + 1, t + 1])
        k, v = _tokens(2, 2, g, spread=6), _tokens(2, 2, g, spread=6)
        kda.kda_cache_write(k.reshape(2, -1).cuda(), v.reshape(2, -1).cuda(), *cache[:5],
                            pool.lens.to(I32).cuda())
        _ref_write(pool, [k.double(), v.double()], [1, 1])
    for side in range(2):
        assert torch.equal(pool.dev[side].cpu(), pool.raw[side])
        assert torch.equal(pool.dev_scale[side].cpu().nan_to_num(-1), pool.scale[side].nan_to_num(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H", [1, 3])
def test_read(lib, kind, P, H):
    """Ragged ranges, inactive sequences, pages that do not exist, odd strides; rows behind the
    last sequence and the space between rows stay as they were."""
    counts = [0, 1, 300, 16, 15, 33, 4, 129, 2]
    totals = [5, 1, 309, 80, 32, 33, 3, 400, 70]
    pool = Pool(kind, H, P, totals, seed=7, pad=32).fill()
    pool.table[2, 0] = -5
    pool.table[7, min(1, pool.width - 1)] = pool.N + 1
    pool.lens[6], pool.lens[8] = 3, 100000  # shorter than its tokens; longer than its table
    T = sum(counts) + 2
    seen, bufs = [], []
    for off in (1, 4):
        t, buf = _strided(torch.full((T, H * 128), -7.0, dtype=BF), 5, off)
        seen.append(t)
        bufs.append(buf)
    kda.kda_cache_read(*seen, *pool.gpu(), cu_seqlens=_cu(counts).cuda())
    for side, off in ((0, 1), (1, 4)):
        want = torch.full((T, H * 128), -7.0).double()
        at = 0
        for b, n in enumerate(counts):
            total = pool.lens[b].item()
            want[at:at + n] = 0.0
            if n <= total <= pool.cap():
                want[at:at + n] = pool.tokens(side, b, total)[0][total - n:].reshape(n, H * 128)
            at += n
        assert torch.equal(seen[side].double().cpu(), want)
        whole = bufs[side][off:].cpu().reshape(T, -1)
        assert (whole[:, H * 128:] == -7).all() and (bufs[side][:off] == -7).all()


@pytest.mark.gpu
def test_write_then_read_returns_the_rounded_tokens(lib):
    """e4m3: within half a step, 2^-4 of the value, or half of the smallest step under the
    page's scale; int8 within half its step."""
    for kind in KINDS:
        pool = Pool(kind, 4, 64, [200, 77], seed=8)
        cache = pool.gpu()
        g = torch.Generator().manual_seed(9)
        k, v = _tokens(277, 4, g, spread=0), _tokens(277, 4, g, spread=0)
        cu = _cu([200, 77]).cuda()
        kda.kda_cache_write(k.reshape(277, -1).cuda(), v.reshape(277, -1).cuda(), *cache,
                            cu_seqlens=cu)
        got = [torch.empty(277, 512, dtype=BF, device="cuda") for _ in range(2)]
        kda.kda_cache_read(*got, *cache, cu_seqlens=cu)
        for x, y in zip((k, v), got):
            x, y = x.double().reshape(277, -1), y.double().cpu()
            top = x.abs().max()
            tol = 2.0 ** -4 * x.abs() + 2.0 ** -10 * top / 224 if kind == F8 else top / 63
            assert ((x - y).abs() <= tol).all()


# ---------------------------------------------------------------------------
# attention

def _check_attention(pool, counts, G, uniform, scale=128 ** -0.5, weight=2.0 ** -16, pad=0,
                     offset=0, seed=0, size=1.0, extra=0, q=None):
    T, Hq = sum(counts) + extra, pool.H * G
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = (torch.randn(T, Hq, 128, generator=g) * size).to(BF)
    qd, _ = _strided(q.reshape(T, -1), pad, offset)
    out, buf = _strided(torch.full((T, Hq * 128), -7.0, dtype=BF), 2 * pad, offset)
    lse, lbuf = _strided(torch.full((T, Hq), -7.0), pad, 0)
    cu = None if uniform else _cu(counts)
    kda.kda_cache_attention(qd, out, *pool.gpu(), cu_seqlens_host=cu,
                            cu_seqlens=None if uniform else cu.cuda(), lse=lse, scale=scale)
    want, wl, tol, lt = _ref_attention(pool, q.double(), counts, G, scale, weight)
    n = T - extra
    _close(out[:n].reshape(n, Hq, 128), want[:n], tol[:n])
    _close(lse[:n], wl[:n], lt[:n])
    assert (out[n:] == -7).all() and (lse[n:] == -7).all()
    assert (buf[:offset] == -7).all()
    assert (buf[offset:].reshape(T, -1)[:, Hq * 128:] == -7).all()
    assert (lbuf.reshape(T, -1)[:, Hq:] == -7).all()
    return out, lse


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,G", [(3, 1), (2, 3), (1, 8), (1, 16)])
def test_attention_one_token(lib, kind, P, H, G):
    pool = Pool(kind, H, P, EDGES, seed=P + G, pad=48).fill()
    _check_attention(pool, [1] * len(EDGES), G, True, pad=3, offset=1)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [2, 3, 5, 8])
@pytest.mark.parametrize("H,G", [(2, 1), (1, 3), (1, 8)])
def test_attention_draft_tokens(lib, kind, T, H, G):
    totals = [T + x for x in (0, 1, 13, 16, 27, 32, 120, 128, 250)]
    for P in (16, 64):
        pool = Pool(kind, H, P, totals, seed=T + G).fill()
        _check_attention(pool, [T] * len(totals), G, True, seed=T,
                         weight=2.0 ** (-16 if T * G <= 128 else -8))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_parts(lib, kind):
    """Long caches are cut into parts: one long sequence, and one beside short and empty ones."""
    for totals, H, G, P in (([5003], 1, 2, 64), ([3000, 1, 40, 0, 900], 2, 1, 16),
                            ([2049], 2, 8, 256)):
        pool = Pool(kind, H, P, totals, seed=11).fill()
        _check_attention(pool, [1] * len(totals), G, True, seed=12, size=2.0)


@pytest.mark.gpu
def test_attention_parts_of_draft_tokens(lib):
    """The last parts are seen by some of the rows only."""
    for total in (1025, 1030, 1281):
        pool = Pool(F8, 1, 64, [total, 600], seed=13).fill()
        _check_attention(pool, [8, 8], 2, True, seed=14)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [63, 64, 65, 200])
def test_attention_many_sequences(lib, n):
    g = torch.Generator().manual_seed(n)
    totals = torch.randint(1, 90, (n,), generator=g).tolist()
    totals[n // 2] = 700
    pool = Pool(I8, 1, 16, totals, seed=15).fill()
    _check_attention(pool, [1] * n, 2, True)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 4])
def test_attention_inactive_and_missing(lib, kind, T):
    """Inactive sequences and tokens without any key give zeros and -infinity; pages that do
    not exist are left out."""
    totals = [40, 0, T - 1, 5000, -3, 20, 48, 33]
    pool = Pool(kind, 2, 16, [40, 0, 16, 48, 0, 20, 48, 33], seed=16, width=3).fill()
    pool.lens = torch.tensor(totals)
    pool.table[0, 1] = -1
    pool.table[5] = pool.N
    pool.table[6, 2] = 1 << 30
    pool.table[7, 0] = -(1 << 31)
    out, lse = _check_attention(pool, [T] * 8, 3, True)
    for b in (1, 2, 3, 4, 5):
        assert (out[b * T:(b + 1) * T] == 0).all()
        assert (lse[b * T:(b + 1) * T] == -torch.inf).all()


@pytest.mark.gpu
def test_attention_of_an_empty_pool(lib):
    pool = Pool(F8, 2, 16, [0, 0], spare=0)
    pool.lens = torch.tensor([5, 16])
    _check_attention(pool, [1, 1], 2, True)
    _check_attention(pool, [3, 40], 2, False)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 8])
def test_attention_nan_of_hidden_tokens(lib, T):
    """A NaN key or value reaches exactly the rows that see it."""
    for total in (9, 40, 300):
        for what in range(2):
            pool = Pool(F8, 1, 64, [total], seed=17).fill()
            at = total - 1 - T // 3
            page, slot = pool.table[0, at // 64].item(), at % 64
            pool.codes(pool.raw)[what][page, 0, slot, 5] = 0xff
            out, _ = _check_attention(pool, [T], 2, True, seed=18)
            sees = torch.arange(total - T, total) >= at
            assert torch.equal(out.isnan().any(1).cpu(), sees)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attention_scales(lib, scale):
    """No weight but equal ones, keys of least product first, and weights that all but vanish."""
    pool = Pool(F8, 2, 32, [70, 333], seed=19).fill()
    _check_attention(pool, [1, 1], 3, True, scale=scale, size=3.0)


@pytest.mark.gpu
def test_attention_scores_that_rise(lib):
    """The reference exponent has to follow: keys that grow along the sequence, and fall."""
    for rise in (1, -1):
        pool = Pool(I8, 1, 16, [600], seed=20).fill()
        order = pool.table[0] if rise > 0 else pool.table[0].flip(0)
        for j, page in enumerate(order.tolist()):
            pool.scale[0][page] = 2.0 ** (j // 3 - 8)
        _check_attention(pool, [1], 8, True, seed=21)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("H,G", [(2, 1), (1, 5), (1, 16)])
def test_attention_documents(lib, kind, P, H, G):
    """Packed documents of odd lengths, from their start and over earlier tokens, beside single
    tokens and empty ones; rows behind the last are left as they were."""
    counts = [1, 130, 0, 33, 64, 5, 200, 1]
    past = [0, 0, 7, 100, 64, 31, 57, 150]
    totals = [a + b for a, b in zip(counts, past)]
    pool = Pool(kind, H, P, totals, seed=22, pad=16).fill()
    _check_attention(pool, counts, G, False, weight=2.0 ** -8, pad=5, offset=3, seed=23, extra=2)


@pytest.mark.gpu
def test_attention_document_inactive_and_missing(lib):
    counts, totals = [70, 90, 40, 65], [69, 5000, 100, 200]
    pool = Pool(F8, 1, 16, [69, 100, 100, 200], seed=24, width=13).fill()
    pool.lens = torch.tensor(totals)
    pool.table[2, 2], pool.table[2, 6], pool.table[3] = -1, pool.N, -7
    out, lse = _check_attention(pool, counts, 2, False, weight=2.0 ** -8)
    assert (out[:160] == 0).all() and (lse[:160] == -torch.inf).all()
    assert (out[200:] == 0).all() and (lse[200:] == -torch.inf).all()


@pytest.mark.gpu
def test_attention_document_nan(lib):
    """A NaN key or value in a document reaches exactly the rows that see it."""
    for n, total in ((150, 150), (100, 237)):
        for what in range(2):
            pool = Pool(F8, 1, 64, [total], seed=25).fill()
            at = total - 40
            page, slot = pool.table[0, at // 64].item(), at % 64
            pool.codes(pool.raw)[what][page, 0, slot, 5] = 0x7f
            out, _ = _check_attention(pool, [n], 3, False, weight=2.0 ** -8, seed=26)
            assert torch.equal(out.isnan().any(1).cpu(), torch.arange(total - n, total) >= at)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [256, 257, 1100, 2100])
def test_attention_more_sequences_than_threads(lib, n):
    """The parts are found by workgroups whose threads take several sequences each."""
    g = torch.Generator().manual_seed(n)
    totals = torch.randint(1, 20, (n,), generator=g).tolist()
    totals[5], totals[n - 1] = 2500, 1030
    pool = Pool(F8, 1, 16, totals, seed=27).fill()
    _check_attention(pool, [1] * n, 1, True)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_document_parts(lib, kind):
    """A few tokens more than a handful over a long cache: documents whose keys are cut, the last
    parts seen by some rows only, beside single tokens and one that is not cut."""
    counts = [140, 1, 3, 130]
    totals = [5003, 2900, 3, 131]
    pool = Pool(kind, 1, 64, totals, seed=28).fill()
    _check_attention(pool, counts, 1, False, weight=2.0 ** -8, seed=29)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [290, 1300])
def test_attention_parts_of_a_mixed_batch(lib, n):
    """Decoded tokens, a few of them with long caches, drafts of several blocks and documents, cut
    and whole: every block that is cut is joined, and no other."""
    g = torch.Generator().manual_seed(45)
    counts = [1] * n
    totals = torch.randint(1, 30, (n,), generator=g).tolist()
    for b, m, total in ((3, 45, 2200), (70, 1, 2600), (71, 150, 1700), (140, 0, 1500),
                        (200, 100, 1300), (255, 260, 2000), (256, 129, 129), (n - 1, 1, 1100)):
        counts[b], totals[b] = m, total
    pool = Pool(F8, 2, 32, totals, seed=46).fill()
    _check_attention(pool, counts, 1, False, weight=2.0 ** -8, seed=47, extra=2)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [512, 513, 1025, 5000])
@pytest.mark.parametrize("H", [2, 128])
def test_attention_few_of_many_sequences(lib, n, H):
    """A few sequences among many without tokens: the bits of the few alone. Documents that are
    cut (2 heads) and whole."""
    at = [7, 400, n - 20, n - 1]
    counts, totals = [1, 3, 200, 330], [300, 40, 1200, 333]
    pool = Pool(F8, H, 32, totals, seed=48).fill()
    T = sum(counts)
    q = torch.randn(T, H * 128, generator=torch.Generator().manual_seed(49)).to(BF).cuda()
    cache = pool.gpu()
    table = torch.full((n, pool.width), -1, dtype=I32, device="cuda")
    lens, many = torch.zeros(n, dtype=I32, device="cuda"), [0] * n
    for i, b in enumerate(at):
        table[b], lens[b], many[b] = cache[4][i], cache[5][i], counts[i]
    got = []
    for c, cu in (((*cache[:4], table, lens), _cu(many)), (cache, _cu(counts))):
        out = torch.full((T, H * 128), -7.0, dtype=BF, device="cuda")
        lse = torch.full((T, H), -7.0, device="cuda")
        kda.kda_cache_attention(q, out, *c, cu_seqlens_host=cu, cu_seqlens=cu.cuda(), lse=lse)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,G", [(9, 8), (16, 8), (40, 3), (17, 8)])
def test_attention_rows_between_the_kernels(lib, T, G):
    """Up to 128 rows and more."""
    pool = Pool(I8, 1, 32, [T + 300, T, 1700], seed=30).fill()
    _check_attention(pool, [T] * 3, G, True, seed=31, weight=2.0 ** (-16 if T * G <= 128 else -8))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 160])
def test_attention_arbitrary_scales(lib, T):
    """Scales that are no powers of two, negative and zero ones. Documents round a value times
    such a scale to bf16: half a step of every value more."""
    pool = Pool(F8, 2, 32, [T + 211], seed=32).fill()
    g = torch.Generator().manual_seed(33)
    for side in range(2):
        pool.scale[side] = torch.where(pool.scale[side].isnan(), pool.scale[side],
                                       torch.randn(pool.scale[side].shape, generator=g) * 0.03)
        pool.scale[side][pool.table[0, 1]] = 0.0
    _check_attention(pool, [T], 1, True, weight=2.0 ** -16 if T == 1 else 2.0 ** -7, seed=34)


@pytest.mark.gpu
def test_attention_is_the_same_every_time_and_fits_its_workspace(lib):
    pool = Pool(F8, 2, 64, [4000, 700, 3, 160], seed=35).fill()
    counts = [1, 5, 3, 150]
    T, cu = sum(counts), _cu(counts)
    q = torch.randn(T, 4 * 128).to(BF).cuda()
    cache, size = pool.gpu(), kda.kda_cache_attention_workspace_size(4, T, 4, 2)
    got = []
    for fill in (0, 0xff, 0x5a):
        buf = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(T, 4, device="cuda")
        kda.kda_cache_attention(q, out, *cache, cu_seqlens_host=cu, cu_seqlens=cu.cuda(), lse=lse,
                                workspace=buf[:size])
        assert (buf[size:] == fill).all()
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    with pytest.raises(kda.KdaError) as e:
        kda.kda_cache_attention(q, out, *cache, cu_seqlens_host=cu, cu_seqlens=cu.cuda(),
                                workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == WS


@pytest.mark.gpu
def test_pages_past_32_bits(lib):
    """A pool of which most lies more than 2^32 bytes into its allocation."""
    H, P, stride = 2, 16, 1 << 29
    totals = [150, 40]
    pool = Pool(F8, H, P, totals, seed=36).fill()
    small, N = pool.gpu(), pool.N
    big = []
    for side in range(2):
        buf = torch.empty((N - 1) * stride + H * P * 128, dtype=torch.uint8, device="cuda")
        view = buf.as_strided(pool.shape, (stride,) + pool.strides[1:])
        view.copy_(small[side].view(torch.uint8))
        big.append(view.view(F8))
    assert (N - 1) * stride > 1 << 32
    rest = small[2:]
    q = torch.randn(2, H * 128).to(BF).cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    kda.kda_cache_attention(q, a, *small)
    kda.kda_cache_attention(q, b, *big, *rest)
    assert torch.equal(a, b)
    cu = _cu(totals).cuda()
    k = [torch.empty(190, H * 128, dtype=BF, device="cuda") for _ in range(4)]
    kda.kda_cache_read(k[0], k[1], *small, cu_seqlens=cu)
    kda.kda_cache_read(k[2], k[3], *big, *rest, cu_seqlens=cu)
    assert torch.equal(k[0], k[2]) and torch.equal(k[1], k[3])
    qd = torch.randn(190, H * 128).to(BF).cuda()
    out = [torch.empty_like(qd) for _ in range(2)]
    for o, cache in zip(out, (small, (*big, *rest))):
        kda.kda_cache_attention(qd, o, *cache, cu_seqlens_host=cu.cpu(), cu_seqlens=cu)
    assert torch.equal(*out)
    new = torch.randn(2, H * 128).to(BF).cuda()
    new[0, 5] = 100.0  # its page's scale grows
    scales = [s.clone() for s in rest[:2]]  # each write has the scales as they were
    kda.kda_cache_write(new, new, *small)
    kda.kda_cache_write(new, new, *big, *scales, *rest[2:])
    for side in range(2):
        assert torch.equal(small[side].view(torch.uint8), big[side].view(torch.uint8))
        assert torch.equal(rest[side].nan_to_num(-1), scales[side].nan_to_num(-1))


@pytest.mark.gpu
def test_two_streams_at_once(lib):
    """Calls that overlap in time, each with a workspace of its own, on streams that are not the
    current one."""
    pools = [Pool(F8, 2, 32, [3000 + 64 * i, 200], seed=37 + i).fill() for i in range(2)]
    caches = [p.gpu() for p in pools]
    q = torch.randn(2, 4 * 128).to(BF).cuda()
    want = [torch.empty_like(q) for _ in range(2)]
    for o, c in zip(want, caches):
        kda.kda_cache_attention(q, o, *c)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.zeros_like(q) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for s, o, c in zip(streams, got, caches):
            kda.kda_cache_attention(q, o[i], *c, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(w, x) for x in o)


@pytest.mark.gpu
def test_captured_steps_share_a_workspace(lib):
    """Decode steps (write, attend) of two batches in two graphs that share one workspace: replayed
    in turn with lengths that grow on the device, against eager calls on a copy."""
    dev, g = "cuda", torch.Generator().manual_seed(39)
    H, G, P = 2, 4, 16

    def batch(totals, T):
        pool = Pool(F8, H, P, [x + 64 for x in totals], seed=sum(totals)).fill()
        for side in range(2):
            pool.scale[side].nan_to_num_(1.0)
        pool.lens = torch.tensor(totals)
        n = len(totals) * T
        return dict(cache=pool.gpu(), T=T, k=torch.zeros(n, H * 128, dtype=BF, device=dev),
                    v=torch.zeros(n, H * 128, dtype=BF, device=dev),
                    q=torch.zeros(n, H * G * 128, dtype=BF, device=dev),
                    out=torch.zeros(n, H * G * 128, dtype=BF, device=dev),
                    lse=torch.zeros(n, H * G, device=dev))

    def step(b, ws):
        b["cache"][5].add_(b["T"])
        kda.kda_cache_write(b["k"], b["v"], *b["cache"])
        kda.kda_cache_attention(b["q"], b["out"], *b["cache"], lse=b["lse"], workspace=ws)

    batches = [batch([2100, 37, 1500], 1), batch([1300, 40], 4)]
    copies = [{k: v.clone() if torch.is_tensor(v) else
               [x.clone() for x in v] if k == "cache" else v for k, v in b.items()} for b in batches]
    size = max(kda.kda_cache_attention_workspace_size(len(b["cache"][5]), b["q"].shape[0], H * G, H)
               for b in batches)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    graphs = []
    for b in batches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(b, ws)
        graphs.append(graph)
    for i in range(6):
        for b, c, graph in zip(batches, copies, graphs):
            for name in ("k", "v", "q"):
                x = torch.randn(b[name].shape, generator=g).to(BF)
                b[name].copy_(x)
                c[name].copy_(x)
            graph.replay()
            step(c, None)
            if i % 2:
                torch.cuda.synchronize()
        for b, c in zip(batches, copies):
            assert torch.equal(b["out"], c["out"]) and torch.equal(b["lse"], c["lse"])
            for x, y in zip(b["cache"], c["cache"]):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_a_layer_served(lib, kind):
    """An attention layer as a server runs it next to the recurrent ones: two documents in chunks, then
    verification of three draft tokens, then single tokens; norm in front, residual norm behind. The
    quantised cache is taken as it is written; the rest is compared in 64 bits."""
    g = torch.Generator().manual_seed(41)
    H, G, P, W = 2, 3, 32, 256
    pool = Pool(kind, H, P, [200, 150], seed=42)
    cache = list(pool.gpu())
    for side in range(2):
        cache[2 + side].nan_to_num_(1.0)
    proj = (torch.randn(W, (G + 2) * H * 128, generator=g) * W ** -0.5).to(BF).cuda()
    back = (torch.randn(G * H * 128, W, generator=g) * (G * H * 128) ** -0.5).to(BF).cuda()
    weight = torch.ones(W).cuda()
    done = [0, 0]
    for counts in ([90, 61], [75, 0], [3, 3], [1, 1], [1, 1]):
        T = sum(counts)
        x = torch.randn(T, W, generator=g).to(BF).cuda()
        y = torch.empty_like(x)
        kda.kda_rmsnorm(x, weight, y)
        qkv = y @ proj
        q, k, v = qkv.split([G * H * 128, H * 128, H * 128], 1)  # rows further apart than wide
        done = [a + b for a, b in zip(done, counts)]
        cache[5] = torch.tensor(done, dtype=I32).cuda()
        ragged = counts[0] != counts[1]
        cu = _cu(counts)
        kda.kda_cache_write(k, v, *cache, cu_seqlens=cu.cuda() if ragged else None)
        out, lse = torch.empty(T, G * H * 128, dtype=BF, device="cuda"), \
            torch.empty(T, G * H, device="cuda")
        kda.kda_cache_attention(q, out, *cache, cu_seqlens_host=cu if ragged else None,
                                cu_seqlens=cu.cuda() if ragged else None, lse=lse)
        z = out @ back
        r, s = torch.empty_like(x), torch.empty_like(x)
        kda.kda_rmsnorm(z, weight, s, residual=x, residual_out=r)
        # what the layer has now, in 64 bits
        pool.lens = torch.tensor(done)
        pool.raw = [t.cpu() for t in pool.dev]
        pool.scale = [t.cpu() for t in cache[2:4]]
        want, wl, tol, lt = _ref_attention(pool, q.double().cpu().reshape(T, G * H, 128), counts, G,
                                           128 ** -0.5, 2.0 ** -8)
        _close(out.reshape(T, G * H, 128), want, tol)
        _close(lse, wl, lt)
        assert torch.equal(r, (z.float() + x.float()).to(BF))
        # and the cache holds this call's tokens within half a step
        got = [torch.empty(T, H * 128, dtype=BF, device="cuda") for _ in range(2)]
        kda.kda_cache_read(*got, *cache, cu_seqlens=cu.cuda())
        for a, b in zip((k, v), got):
            a, b = a.double(), b.double()
            top = a.abs().max()
            step = 2.0 ** -4 * a.abs() + 2.0 ** -10 * top / 224 if kind == F8 else top / 63
            assert ((a - b).abs() <= step).all()


def test_workspace_comes_from_the_stream(lib, monkeypatch):
    """Without one given, the workspace is made in the launch stream's pool (stand-ins for the
    library and the GPU)."""
    import contextlib
    seen, at = [], [0x100]

    class Gpu:
        is_cuda, device = True, torch.device("cuda", 0)

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0

    class Lib:
        def kda_cache_attention_workspace_size(self, *a):
            return 512

        def kda_cache_attention(self, *a):
            seen.append(("call", a[-3], a[-2], a[-1]))
            return 0

    class Stream:
        cuda_stream, device = 0x200, torch.device("cuda", 0)

    @contextlib.contextmanager
    def use(stream):
        at.append(stream.cuda_stream)
        yield
        at.pop()

    empty = torch.empty
    keep = []

    def alloc(n, dtype, device):
        keep.append(Gpu(empty(n, dtype=dtype)))
        seen.append(("made", keep[-1].data_ptr(), n, at[-1]))
        return keep[-1]

    monkeypatch.setattr(kda, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream())
    monkeypatch.setattr(torch, "empty", alloc)
    c = Gpu(torch.zeros(3, 2, 16, 128, dtype=I8))
    s, tab, lens = Gpu(torch.ones(3, 2)), Gpu(torch.zeros(1, 3, dtype=I32)), \
        Gpu(torch.ones(1, dtype=I32))
    q, o = Gpu(torch.zeros(1, 512, dtype=BF)), Gpu(torch.zeros(1, 512, dtype=BF))
    kda.kda_cache_attention(q, o, c, c, s, s, tab, lens, stream=Stream())
    (_, adr, n, stream), (_, ws, size, raw) = seen
    assert stream == 0x200 and raw == 0x200 and ws == adr and size == n == 512
    with pytest.raises(ValueError):  # the host's copy alone
        kda.kda_cache_attention(q, o, c, c, s, s, tab, lens,
                                cu_seqlens_host=torch.zeros(2, dtype=I32))
    with pytest.raises(ValueError):  # heads that do not divide
        kda.kda_cache_attention(Gpu(torch.zeros(1, 384, dtype=BF)),
                                Gpu(torch.zeros(1, 384, dtype=BF)), c, c, s, s, tab, lens)
    with pytest.raises(ValueError):  # scales of another shape
        kda.kda_cache_attention(q, o, c, c, Gpu(torch.ones(3, 1)), s, tab, lens)
    with pytest.raises(TypeError):
        kda.kda_cache_attention(q, o, Gpu(c.t.float()), c, s, s, tab, lens)


# ---------------------------------------------------------------------------
# cu_seqlens on the device that is not what the call was planned for: nothing outside of the
# call's rows, pages and workspace is touched

BAD_CU = [
    [-5, 1, 61, 64, 64, 104], [-(1 << 31)] * 6, [0, 1, 61, 1 << 30, 64, (1 << 31) - 1],
    [0, 90, 13, 64, 2, 104], [104, 64, 64, 61, 1, 0], [104] * 6, [0] * 6, [0, 104, 0, 104, 0, 104],
    [0, 104, 104, 104, 104, 104], [50, 51, 52, 52, 60, 104],
]


def _rows_named(cu, T):
    """The rows that some sequence of a clamped cu_seqlens has."""
    named = torch.zeros(T, dtype=torch.bool)
    for a, b in zip(cu, cu[1:]):
        named[min(max(a, 0), T):max(min(max(b, 0), T), 0)] = True
    return named


@pytest.mark.gpu
@pytest.mark.parametrize("cu", BAD_CU)
@pytest.mark.parametrize("kind", KINDS)
def test_bad_cu_seqlens_written_and_read(lib, cu, kind):
    H, P, T = 3, 32, 104
    pool = Pool(kind, H, P, [130, 200, 111, 104, 333], seed=60, pad=16).fill()
    cache = pool.gpu()
    k, v = (torch.full((T, H * 128), x, dtype=BF, device="cuda") for x in (3.0, -0.5))
    bad = torch.tensor(cu, dtype=I32).cuda()
    kda.kda_cache_write(k, v, *cache, cu_seqlens=bad)
    owned = pool.table[(pool.table >= 0) & (pool.table < pool.N)]
    free = torch.ones(pool.N, dtype=torch.bool)
    free[owned] = False
    for side in range(2):
        got, size = pool.dev[side].cpu(), pool.strides[0]
        assert torch.equal(got[pool.N * size:], pool.raw[side][pool.N * size:])
        got, was = (x[:pool.N * size].reshape(pool.N, size) for x in (got, pool.raw[side]))
        assert torch.equal(got[free], was[free]) and torch.equal(got[:, -16:], was[:, -16:])
        assert pool.dev_scale[side].cpu()[free].isnan().all()
    seen, bufs = [], []
    for off in (16, 32):
        buf = torch.full((T * H * 128 + 2 * off,), -7.0, dtype=BF, device="cuda")
        seen.append(buf[off:-off].reshape(T, H * 128))
        bufs.append((buf, off))
    kda.kda_cache_read(*seen, *cache, cu_seqlens=bad)
    for x, (buf, off) in zip(seen, bufs):
        assert (x[~_rows_named(cu, T).cuda()] == -7).all()
        assert (buf[:off] == -7).all() and (buf[-off:] == -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cu", BAD_CU)
@pytest.mark.parametrize("n", [5, 600])
@pytest.mark.parametrize("kind", KINDS)
def test_bad_cu_seqlens_attention(lib, cu, n, kind):
    """Planned for a single token, a document, a draft and another document; 5 sequences, or these
    among 600."""
    H, G, T, counts = 2, 4, 104, [1, 60, 3, 0, 40]
    pool = Pool(kind, H, 32, [1300, 2000, 111, 104, 1500], seed=61).fill()
    cache = list(pool.gpu())
    host, bad = _cu(counts), torch.tensor(cu, dtype=I32)
    if n > 5:
        more = n - 5
        cache[4] = torch.cat([cache[4], cache[4][:1].expand(more, -1)])
        cache[5] = torch.cat([cache[5], torch.full((more,), 300, dtype=I32, device="cuda")])
        host = torch.cat([host, host[-1:].expand(more)])
        bad = torch.cat([bad, bad[torch.arange(more) % 6]])
    q = torch.randn(T, H * G * 128, generator=torch.Generator().manual_seed(62)).to(BF).cuda()
    size = kda.kda_cache_attention_workspace_size(n, T, H * G, H)
    ws = torch.full((size + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    obuf = torch.full((T + 2, H * G * 128), -7.0, dtype=BF, device="cuda")
    lbuf = torch.full((T + 2, H * G), -7.0, device="cuda")
    for device in (bad, host, bad):  # the bad ones find what a call before them left, too
        obuf.fill_(-7.0)
        lbuf.fill_(-7.0)
        kda.kda_cache_attention(q, obuf[1:-1], *cache, cu_seqlens_host=host,
                                cu_seqlens=device.cuda(), lse=lbuf[1:-1],
                                workspace=ws[4096:-4096])
        named = _rows_named(device.tolist(), T).cuda()
        for x in (obuf, lbuf):
            assert (x[0] == -7).all() and (x[-1] == -7).all()
            assert (x[1:-1][~named] == -7).all()
        assert (ws[:4096] == 0x5a).all() and (ws[-4096:] == 0x5a).all()


@pytest.mark.gpu
def test_bad_cu_seqlens_of_more_parts_than_32_bits_count(lib):
    """Planned for one token, with 262194 of 256 query heads on the device: 2^19 + 100 blocks of 128
    rows, and 32761 units of 128 keys. The blocks' units, added up in 32 bits, are negative, so that
    parts are the shortest ones, 8191 of them, and the last blocks' numbers times the parts pass 2^32:
    there is no room for any of their results."""
    T, units = 262194, 32761
    assert (T * 2 * units + (1 << 31)) % (1 << 32) < 1 << 31  # negative
    assert 0 < T * 2 * 8191 - (1 << 32) < 36 * 8191
    c = torch.zeros(1, 1, 256, 128, dtype=I8, device="cuda")
    s = torch.ones(1, 1, device="cuda")
    table = torch.zeros(1, units // 2 + 1, dtype=I32, device="cuda")
    lens = torch.tensor([units * 128], dtype=I32, device="cuda")
    q = torch.ones(1, 256 * 128, dtype=BF, device="cuda").expand(T, -1)
    out = torch.full((T, 256 * 128), -7.0, dtype=BF, device="cuda")
    size = kda.kda_cache_attention_workspace_size(1, T, 256, 1)
    ws = torch.full((size + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    kda.kda_cache_attention(q, out, c, c, s, s, table, lens,
                            cu_seqlens_host=torch.tensor([0, 1], dtype=I32),
                            cu_seqlens=torch.tensor([0, T], dtype=I32).cuda(),
                            workspace=ws[4096:-4096])
    assert (ws[:4096] == 0x5a).all() and (ws[-4096:] == 0x5a).all()
    assert (out == -7).all()  # no part of these fits


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("n", [1, 3, 13, 40])
@pytest.mark.parametrize("bad", [None, torch.nan, -torch.inf])
def test_write_behind_an_odd_scale_that_stays(lib, kind, P, n, bad):
    """Earlier tokens under a scale that is no power of two and more than the new ones need: codes
    are value * (1 / scale), each step rounded to fp32, then to the nearest code. Odd multiples of
    half the scale are ties in exact arithmetic and in fp32, though not of the unrounded product; an
    infinity or a NaN changes its own code only."""
    odd = torch.tensor([1.5, 0.7, 3.1])
    pool = Pool(kind, 3, P, [5 + n], seed=70, width=5).fill([5])
    for side in range(2):
        pool.scale[side][pool.table[0, 0]] = odd
    g = torch.Generator().manual_seed(71)
    x = [(torch.randint(-30, 30, (n, 3, 128), generator=g) + 0.5).float() * odd[:, None]
         for _ in range(2)]
    x[0][:, :, ::3] = torch.randn(n, 3, 43, generator=g) * 9
    k, v = (t.to(BF) for t in x)
    if bad is not None:
        k[0, 0, 1], v[n - 1, 2, 127] = bad, bad
    cache = pool.gpu()
    kda.kda_cache_write(k.reshape(n, -1).cuda(), v.reshape(n, -1).cuda(), *cache)
    here = min(n, P - 5)  # the new tokens in the earlier ones' page
    for side, t in enumerate((k, v)):
        want = _nearest((t[:here].float() * (1 / odd)[:, None]).double(), kind)
        if kind == F8:
            want = torch.where(t[:here].isnan(), torch.nan, want)
        page = pool.table[0, 0]
        got = pool.codes([r.cpu() for r in pool.dev])[side][page].contiguous().view(kind)
        got = _value(got, kind)[:, 5:5 + here].transpose(0, 1)
        assert torch.equal(got.nan_to_num(1000.0), want.nan_to_num(1000.0))
        assert torch.equal(pool.dev_scale[side][page].cpu(), odd)


# ---------------------------------------------------------------------------
# attention by whole sequences, the tolerance by each sequence's rows
#
# As above, with these weights' relative errors: 2^-16 up to 128 rows, and half a step of fp16,
# 2^-11, beyond. fp16's smallest step is 2^-24 where the largest (weight * |scale|) of a row so far is
# 2^6 at least: half of it for each of n tokens, times a code of up to 448 and over a sum that is at
# least as large, n 2^-31 * 448 max (p |scale|). Few rows flush what is below 2^-126, or below 2^-62
# where a scale passes 2^60: n times that, times 448. bf16's smallest step adds 2^-134. log2 of a
# scale that is no power of two, up to 2^7 and a step of 2^-17, is off by 2^-18 + 2^-23, and its
# reciprocal by 2^-23: 2^-18 covers both in a weight, 2^-18 in lse.

def _ref_sequences(pool, q, counts, G, scale):
    """out, lse, tol, lt, and sum (p v)^2; q fp64 [T, Hq, 128]."""
    T, Hq = q.shape[:2]
    out, tol, sq = (torch.zeros(T, Hq, 128, dtype=torch.float64) for _ in range(3))
    lse, lt = torch.full((T, Hq), -torch.inf).double(), torch.zeros(T, Hq).double()
    at = 0
    for b, n in enumerate(counts):
        total = pool.lens[b].item()
        rows, at = slice(at, at + n), at + n
        if n == 0 or not n <= total <= pool.cap():
            continue
        doc = n * G > 128
        (keys, there), (values, _) = pool.tokens(0, b, total), pool.tokens(1, b, total)
        size = torch.zeros(total, pool.H, dtype=torch.float64)
        for j in range(-(-total // pool.P)):
            if 0 <= pool.table[b, j] < pool.N:
                size[j * pool.P:(j + 1) * pool.P] = \
                    pool.scale[1][pool.table[b, j]].abs().double()
        hidden = ~there | (torch.arange(total) > torch.arange(total - n, total)[:, None])
        for h in range(pool.H):
            x = q[rows, h * G:(h + 1) * G].transpose(0, 1)  # [G, n, 128]
            s = (scale * (x @ keys[:, h].T)).masked_fill(hidden, -torch.inf)
            d = (abs(scale) * 131 * 2.0 ** -24 * (x.abs() @ keys[:, h].abs().T)) \
                .masked_fill(hidden, 0.0).amax(-1)
            l = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(l.isfinite(), l, 0.0)[..., None])
            v, m = values[:, h], (~hidden).sum(-1).double()[:, None]
            o = p @ v
            big = (p * size[:, h]).amax(-1, keepdim=True)
            rel = (2.0 ** -11 + 2.0 ** -18 if doc else 2.0 ** -16) + m * 2.0 ** -23 + 2.0 ** -20 + \
                2 * d[..., None]
            lost = 2.0 ** -31 * big if doc else 2.0 ** (-62 if size.max() > 2.0 ** 60 else -126)
            t = 2.0 ** -8 * o.abs() + rel * (p @ v.abs()) + m * 448 * lost + 2.0 ** -134
            where = (rows, slice(h * G, (h + 1) * G))
            out[where], tol[where] = o.transpose(0, 1), t.transpose(0, 1)
            sq[where] = ((p * p) @ (v * v)).transpose(0, 1)
            lse[where] = l.T
            lt[where] = (d + m[:, 0] * 2.0 ** -24 + (2.0 ** -18 if doc else 0) +
                         2.0 ** -21 * (1 + l.abs())).T
    # what bf16 rounds to infinity
    out = torch.where(out.abs() >= 2.0 ** 128 * (1 - 2.0 ** -9), out.sign() * torch.inf, out)
    return out, lse, tol, lt, sq


def _check_sequences(pool, counts, G, scale=128 ** -0.5, seed=0, size=1.0, q=None):
    T, Hq = sum(counts), pool.H * G
    if q is None:
        q = (torch.randn(T, Hq, 128, generator=torch.Generator().manual_seed(seed)) * size).to(BF)
    out = torch.full((T, Hq * 128), -7.0, dtype=BF, device="cuda")
    lse, cu = torch.full((T, Hq), -7.0, device="cuda"), _cu(counts)
    kda.kda_cache_attention(q.reshape(T, -1).cuda(), out, *pool.gpu(), cu_seqlens_host=cu,
                            cu_seqlens=cu.cuda(), lse=lse, scale=scale)
    want, wl, tol, lt, sq = _ref_sequences(pool, q.double(), counts, G, scale)
    out = out.reshape(T, Hq, 128)
    _close(out, want, tol)
    _close(lse, wl, lt)
    return out, want, sq


def _scale_values(pool, choices, seed):
    """Each page and head's values under one of these scales."""
    g = torch.Generator().manual_seed(seed)
    which = torch.randint(0, len(choices), (pool.N, pool.H), generator=g)
    pool.scale[1] = torch.tensor(choices)[which]
    return pool


def _positive_values(pool):
    c = pool.raw[1]
    pool.raw[1] = c & 127 if pool.kind == F8 else c.view(I8).abs().view(torch.uint8)
    return pool


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("totals", [[90, 700, 6], [3000, 40, 900, 2500]])
def test_attention_of_few_rows_large_values(lib, kind, T, totals):
    """Values up to 2^126, whose sums pass fp32's range though their averages do not, alone and
    beside ordinary ones, whole and in parts."""
    big = 2.0 ** (118 if kind == F8 else 119)
    for i, choices in enumerate(([big], [big, 2.0 ** -7], [big, 2.0 ** 61, 2.0 ** 60, 2.0 ** 59])):
        pool = _positive_values(Pool(kind, 2, 16, totals, seed=80).fill())
        _scale_values(pool, choices, 81 + i)
        _check_sequences(pool, [T] * len(totals), 2, seed=82)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,counts,past", [(2, [150, 260], [37, 900]), (64, [130, 259, 190], [0, 70, 12])])
def test_attention_document_weights_keep_11_bits(lib, kind, H, counts, past):
    """Half a step of fp16 is all that a weight is off, in each output and on the average, cut (2 heads)
    and whole. The mean square of an output's rounding to bf16 is a third of its half step's square; the
    weights' errors, independent of one another, add a third of 2^-22 sum (p v)^2 at most, less than
    3 % where values are independent of one another. (Half a step of bf16, 2^-8, would make it about
    twice as large.) Rows' weights are shared by their 128 channels: a few hundred of them leave the mean
    within 10 %."""
    for P in (16, 64):
        pool = Pool(kind, H, P, [a + b for a, b in zip(counts, past)], seed=83).fill()
        G = 2 if H == 2 else 1
        got, want, sq = _check_sequences(pool, counts, G, seed=84)
        got = got.double().cpu()
        step = torch.exp2(torch.floor(torch.log2(want.abs())) - 8)
        expected = ((step * step + 2.0 ** -22 * sq) / 3).sum()
        assert ((got - want) ** 2).sum() <= 1.1 * expected


WIDE = [0.0, 2.0 ** -100, 2.0 ** -41, 2.0 ** -40, 1.37 * 2.0 ** -3, -2.0 ** -5, 2.0 ** 40, 2.0 ** 41,
        1.9 * 2.0 ** 40, 2.0 ** 60, 2.0 ** 61, 2.0 ** 90, 2.0 ** -140]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("counts,past", [([150, 300], [37, 900]), ([1, 8, 1], [3000, 90, 10]),
                                         ([140], [5000])])
@pytest.mark.parametrize("choices", [WIDE, WIDE[:3], WIDE[4:6], [2.0 ** -100], [2.0 ** 116],
                                     [2.0 ** -100, 2.0 ** -7], [2.0 ** -100, 2.0 ** 100],
                                     [2.0 ** -40, 2.0 ** 40]])
def test_attention_scales_far_apart(lib, kind, P, counts, past, choices):
    """Pages whose values are far larger or smaller than others', for documents, cut and whole, and few
    rows; scores that are even, and scores that pick the keys of a few pages."""
    for i, size in enumerate((1.0, 8.0)):
        pool = Pool(kind, 2, P, [a + b for a, b in zip(counts, past)], seed=85).fill()
        _scale_values(pool, choices, 86 + i)
        _check_sequences(pool, counts, 2, seed=87, size=size)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,counts,past", [(2, [150], [37]), (64, [130, 259, 190], [0, 70, 12]),
                                           (1, [140], [3000])])
def test_attention_documents_large_values(lib, kind, H, counts, past):
    """Values up to 2^126, whose sums pass fp32's range though their averages do not; and the code
    that stands for 2^128, which the largest bf16 values are written as: rows that do not see it are as
    if it were not there."""
    big = 2.0 ** (118 if kind == F8 else 119)
    pool = _positive_values(Pool(kind, H, 16, [a + b for a, b in zip(counts, past)], seed=88).fill())
    _scale_values(pool, [big, 2.0 ** -7], 89)
    _check_sequences(pool, counts, 1, seed=90)
    for b, n in enumerate(counts):
        at = past[b] + n // 2
        page = pool.table[b, at // 16]
        c = pool.codes(pool.raw)[1]
        c[page, :, at % 16, 7] = 0x78 if kind == F8 else 64
        pool.scale[1][page] = 2.0 ** (120 if kind == F8 else 122)
        c[page, :, at % 16 + 1:] = 0
        c[page, :, :at % 16] = 0
    _check_sequences(pool, counts, 1, seed=91)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("down", [18, 24, 28])
@pytest.mark.parametrize("H", [1, 300])
def test_attention_documents_small_weights(lib, kind, down, H):
    """One key of weight 1 whose values are zeros, before 4000 of 2^-down with the largest values: fp16's
    subnormal numbers, whose sum is all there is. Cut (one head) and whole."""
    n, total = (140, 4000) if H == 1 else (129, 700)
    pool = Pool(kind, H, 64, [total], seed=92).fill()
    for side in range(2):
        pool.codes(pool.raw)[side][:] = 0
        pool.scale[side][:] = 2.0 ** -6
    page = pool.table[0, 0]
    pool.codes(pool.raw)[0][page, :, 0, 0] = torch.tensor([64.0]).to(kind).view(torch.uint8)
    pool.codes(pool.raw)[1][:] = 0x7e if kind == F8 else 127
    pool.codes(pool.raw)[1][page, :, 0] = 0
    q = torch.zeros(n, H, 128)
    q[:, :, 0] = down * 0.6931471805599453
    _check_sequences(pool, [n], 1, scale=1.0, q=q.to(BF))


# ---------------------------------------------------------------------------
# reading under any scale

@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_read_behind_odd_scales(lib, kind):
    """The product is rounded to fp32, then to bf16: 15 * 9542042 lies between two fp32 numbers, the
    lower of which is a tie in bf16. Negative, zero, tiny and huge scales; a code that stands for 2^128
    is infinity."""
    choices = [9542042.0, 0.1, -3.7, 0.0, 1e-38, 3e-42, 7.3e36, 2.0 ** 120, -1.0 / 3.0]
    pool = Pool(kind, 3, 16, [150, 33], seed=95).fill()
    g = torch.Generator().manual_seed(96)
    for side in range(2):
        which = torch.randint(0, len(choices), (pool.N, 3), generator=g)
        which[pool.table[0, :3]] = 0
        which[pool.table[0, 3:5]] = 7
        pool.scale[side] = torch.tensor(choices)[which]
        c = pool.codes(pool.raw)[side]
        c[pool.table[0, 0], :, 3, 5] = torch.tensor([15.0]).to(kind).view(torch.uint8)
        c[pool.table[0, 3], :, 3, 5] = 0x78 if kind == F8 else 127
    got = [torch.full((183, 3 * 128), -7.0, dtype=BF, device="cuda") for _ in range(2)]
    kda.kda_cache_read(*got, *pool.gpu(), cu_seqlens=_cu([150, 33]).cuda())
    for side in range(2):
        at, c = 0, pool.codes(pool.raw)[side]
        for b, n in ((0, 150), (1, 33)):
            for i in range(n):
                page = pool.table[b, i // 16]
                code = _value(c[page, :, i % 16].contiguous().view(kind), kind).float()
                want = (code * pool.scale[side][page][:, None]).to(BF).reshape(-1)
                assert torch.equal(got[side][at].cpu(), want)
                at += 1
        if kind == F8:
            assert got[side].float()[3 * 16 + 3, 5] == torch.inf


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [32, 64, 128, 256])
def test_many_single_tokens_beside_documents_written(lib, kind, P):
    """520 sequences of 8 heads: single tokens, drafts, empty ones and documents, behind earlier tokens
    and not; NaN and infinities among them."""
    g = torch.Generator().manual_seed(P)
    n, H = 520, 8
    counts = [1] * n
    past = torch.randint(0, 40, (n,), generator=g).tolist()
    for b, c in ((0, 0), (3, 17), (64, 8), (65, 300), (130, 16), (200, 0), (255, 70), (256, 33),
                 (400, 600), (519, 90)):
        counts[b] = c
    past[65], past[400] = 2 * P - 3, P
    pool = Pool(kind, H, P, [a + b for a, b in zip(counts, past)], seed=97, pad=16).fill(past)
    pool.lens[5], pool.lens[130] = 0, pool.cap() + 1
    T = sum(counts)
    k, v = _tokens(T, H, g), _tokens(T, H, g)
    k[40, 3, 7], v[100, 5, 0], v[300, 1, 1] = torch.nan, torch.inf, -torch.inf
    _check_write(pool, k, v, counts, False, pad=6, offset=3)


# ---------------------------------------------------------------------------
# every instance of the attention kernels, each sequence to its own tolerance

@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [513, 1100])
@pytest.mark.parametrize("H,G,T", [(1, 1, 1), (2, 3, 1), (1, 8, 3)])
def test_attention_of_more_than_512_sequences(lib, kind, n, H, G, T):
    """Single tokens and drafts, one and two blocks of rows, most caches short and a few cut."""
    g = torch.Generator().manual_seed(n + H)
    totals = torch.randint(T, 40, (n,), generator=g).tolist()
    totals[5], totals[n - 1], totals[n // 2] = 2500, 1030, 700
    pool = Pool(kind, H, 16, totals, seed=100).fill()
    _check_sequences(pool, [T] * n, G, seed=101)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [290, 1300])
@pytest.mark.parametrize("H", [2, 96])
def test_attention_of_mixed_batches_by_sequences(lib, kind, n, H):
    """Single tokens, drafts of several blocks and documents, cut (2 heads) and whole."""
    g = torch.Generator().manual_seed(102)
    counts = [1 if H == 2 or b % 20 == 0 else 0 for b in range(n)]
    totals = torch.randint(1, 30, (n,), generator=g).tolist()
    for b, m, total in ((3, 45, 2200), (70, 1, 2600), (71, 150, 1700), (140, 0, 1500),
                        (200, 100, 1300), (255, 260, 1400), (256, 129, 129), (n - 1, 1, 1100)):
        counts[b], totals[b] = m, total if H == 2 else min(total, m + 300)
    pool = Pool(kind, H, 32, totals, seed=103).fill()
    _check_sequences(pool, counts, 1, seed=104)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [17, 32, 33, 64, 128, 129, 256])
@pytest.mark.parametrize("T", [1, 2])
def test_attention_of_large_groups(lib, kind, G, T):
    """Up to 256 query heads of a key/value head: single tokens are several blocks, and documents."""
    totals = [T, 40, 333, 2600, 5]
    pool = Pool(kind, 2, 32, totals, seed=105).fill()
    _check_sequences(pool, [T] * 5, G, seed=106)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [513, 5000])
@pytest.mark.parametrize("H", [2, 128])
def test_attention_few_int8_of_many_sequences(lib, n, H):
    """The bits of a few sequences do not depend on a thousand without tokens beside them."""
    at, counts, totals = [7, 400, n - 20, n - 1], [1, 3, 200, 330], [300, 40, 1200, 333]
    pool = Pool(I8, H, 32, totals, seed=107).fill()
    T = sum(counts)
    q = torch.randn(T, H * 128, generator=torch.Generator().manual_seed(108)).to(BF).cuda()
    cache = pool.gpu()
    table = torch.full((n, pool.width), -1, dtype=I32, device="cuda")
    lens, many = torch.zeros(n, dtype=I32, device="cuda"), [0] * n
    for i, b in enumerate(at):
        table[b], lens[b], many[b] = cache[4][i], cache[5][i], counts[i]
    got = []
    for c, cu in (((*cache[:4], table, lens), _cu(many)), (cache, _cu(counts))):
        out = torch.full((T, H * 128), -7.0, dtype=BF, device="cuda")
        lse = torch.full((T, H), -7.0, device="cuda")
        kda.kda_cache_attention(q, out, *c, cu_seqlens_host=cu, cu_seqlens=cu.cuda(), lse=lse)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,total", [(1, 5000), (8, 3000), (150, 200), (150, 4000)])
@pytest.mark.parametrize("what", [0, 1])
def test_attention_nan_through_parts(lib, T, total, what):
    """A NaN key or value, early, in the middle and among the call's own tokens, in whole and in joined
    blocks: NaN in exactly the rows that see it (and, for a value, its channel)."""
    for at in (3, total // 2, total - 1 - T // 2):
        pool = Pool(F8, 1, 64, [total, 40], seed=109).fill()
        pool.codes(pool.raw)[what][pool.table[0, at // 64], 0, at % 64, 5] = 0xff
        q = torch.randn(T + 1, 256, generator=torch.Generator().manual_seed(110)).to(BF).cuda()
        out, lse = torch.empty_like(q), torch.empty(T + 1, 2, device="cuda")
        cu = _cu([T, 1])
        kda.kda_cache_attention(q, out, *pool.gpu(), cu_seqlens_host=cu, cu_seqlens=cu.cuda(), lse=lse)
        sees = torch.zeros(T + 1, 2, 128, dtype=torch.bool)
        sees[:T][torch.arange(total - T, total) >= at] = True
        if what:
            sees[:, :, :5] = False
            sees[:, :, 6:] = False
        assert torch.equal(out.isnan().cpu().reshape(T + 1, 2, 128), sees)
        assert torch.equal(lse.isnan().cpu(), sees.all(-1) if not what else torch.zeros(T + 1, 2).bool())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,total", [(1, 300), (1, 5000), (8, 3000), (150, 200), (150, 4000)])
@pytest.mark.parametrize("bad", [torch.inf, -torch.inf, torch.nan, 3e38])
def test_attention_of_queries_beyond_range(lib, kind, T, total, bad):
    """A query that is not finite, or whose products are not, spoils its own row and head: NaN there, and
    the bits of all others as they are without it."""
    pool = Pool(kind, 1, 64, [total, 40], seed=111).fill()
    q = torch.randn(T + 1, 256, generator=torch.Generator().manual_seed(112)).to(BF).cuda()
    cu, cache, got = _cu([T, 1]), pool.gpu(), []
    for i in range(2):
        if i:
            q[T // 2, 128:] = bad
        out, lse = torch.empty_like(q), torch.empty(T + 1, 2, device="cuda")
        kda.kda_cache_attention(q, out, *cache, cu_seqlens_host=cu, cu_seqlens=cu.cuda(), lse=lse)
        got.append((out.reshape(T + 1, 2, 128), lse))
    others = torch.ones(T + 1, 2, dtype=torch.bool)
    others[T // 2, 1] = False
    for a, b in zip(*got):
        assert torch.equal(a[others], b[others]) and a.isfinite().all()
        assert b[T // 2, 1].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("H", [1, 300])
def test_attention_document_scales(lib, kind, scale, H):
    """No weight but equal ones, keys of least product first, and weights that all but vanish, cut
    (one head) and whole."""
    pool = Pool(kind, H, 32, [1300 if H == 1 else 333], seed=113).fill()
    _check_sequences(pool, [135], 1, scale=scale, seed=114, size=3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("counts,past", [([150, 300], [37, 900]), ([140], [5000])])
def test_attention_documents_over_zeros(lib, kind, P, counts, past):
    """Pages of zeros, which a write leaves under 2^-100 (some by negative zeros, some under a scale of
    zero), that take most of the weight or none, beside ordinary pages and some beyond 2^40."""
    g = torch.Generator().manual_seed(115)
    for keys in (2.0 ** -9, 2.0 ** -4):
        pool = Pool(kind, 2, P, [a + b for a, b in zip(counts, past)], seed=116).fill()
        pool.scale[0][:] = 2.0 ** -8
        zero = torch.rand(pool.N, 2, generator=g) < 0.3
        c = pool.codes(pool.raw)[1]
        c[zero] = 0
        pool.scale[0][zero] = keys
        pool.scale[1][zero] = torch.where(torch.rand(int(zero.sum()), generator=g) < 0.8,
                                          2.0 ** -100, 0.0)
        if kind == F8:
            minus = zero & (torch.rand(pool.N, 2, generator=g) < 0.3)
            c[minus] = 0x80
        _check_sequences(pool, counts, 2, seed=117)
        pool.scale[1][pool.table[0, 2]] = 2.0 ** 41
        _check_sequences(pool, counts, 2, seed=118)
