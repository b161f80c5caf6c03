"""kda_prefill_varlen_backward: host validation (CPU) and parity with automatic
differentiation of the token recurrence in 64 bits (GPU).

Tolerances. The kernels compute in fp32: every product sums at most 128 terms, and a
decay weight inside a block is a product of at most 16 exponentials of gates within 5.5,
each off by its argument's rounding, a step of its own and the product's, (5.5 + 2 + 1)
2^-24, so its relative error stays under 136 * 2^-24 = 8.1e-6; a gradient passes through
fewer than ten such factors. dq, dk and dg then subtract parts of similar size, so the error is
relative to the largest gradient of the document and head, not to the element:
1e-4 of it. bf16 outputs add half a step, 2^-8 of the element. fp32 outputs:
the state gradient 1e-5 of the largest element; dA_log and ddt_bias 2e-5 of
the sum of their terms' magnitudes.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import gated_delta_rule_step_amd as kda

OK, NULLP, SHAPE, STRIDE, UNSUP, SEQ, WS = range(7)
BF, D = torch.bfloat16, 128
PRE, PRESIG, HEAD = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_step_amd import build
        build.build()
    return kda.lib()


# ---------------------------------------------------------------------------
# refusals: every call returns before anything is launched (made-up pointers)

def _call(lib, **kw):
    a = dict(n=2, T=30, H=3, K=128, V=128, cu=(0, 10, 30), cud=4096, q=4096, k=4096, v=4096,
             g=4096, b=4096, al=4096, dt=4096, lb=-5.0, sc=1.0, gm=0, sd=0, pool=4096, N=4,
             ss=3 * 16384, idx=4096, ui=1, do=4096, df=0, dq=4096, dk=4096, dv=4096, dg=4096,
             db=4096, da=4096, dd=4096, di=4096, ws=4096, wb=1 << 40,
             s=(384,) * 4 + (3,), os=(384,) * 4 + (3,), dos=384)
    a.update(kw)
    P = ctypes.c_void_p
    cu = (ctypes.c_int32 * len(a["cu"]))(*a["cu"]) if a["cu"] else None
    s, o = a["s"], a["os"]
    return lib.kda_prefill_varlen_backward(
        a["n"], a["T"], a["H"], a["K"], a["V"], cu, P(a["cud"]), P(a["q"]), s[0], P(a["k"]), s[1],
        P(a["v"]), s[2], P(a["g"]), s[3], P(a["b"]), s[4], P(a["al"]), P(a["dt"]), a["lb"],
        a["sc"], a["gm"], a["sd"], P(a["pool"]), a["N"], a["ss"], P(a["idx"]), a["ui"], P(a["do"]),
        a["dos"], P(a["df"]), P(a["dq"]), o[0], P(a["dk"]), o[1], P(a["dv"]), o[2], P(a["dg"]),
        o[3], P(a["db"]), o[4], P(a["da"]), P(a["dd"]), P(a["di"]), P(a["ws"]), a["wb"], P(0))


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(n=-1)), (SHAPE, dict(T=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(N=-1)),
    (UNSUP, dict(K=64)), (UNSUP, dict(V=64)), (UNSUP, dict(H=70000)), (UNSUP, dict(lb=-6.0)),
    (UNSUP, dict(lb=float("nan"))), (UNSUP, dict(gm=8)), (UNSUP, dict(gm=PRE)),
    (UNSUP, dict(gm=PRE, da=0, dd=0, lb=1.0)), (UNSUP, dict(sd=3)), (UNSUP, dict(sd=-1)),
    (UNSUP, dict(di=4100)), (UNSUP, dict(ws=4100)), (UNSUP, dict(lb=0.5)),
    (UNSUP, dict(s=(384, 384, (1 << 25) + 1, 384, 3))), (UNSUP, dict(dos=1 << 26)),
    (UNSUP, dict(os=(384, 384, 384, 384, 1 << 26))),
    (NULLP, dict(cu=None)), (NULLP, dict(cud=0)), (NULLP, dict(q=0)), (NULLP, dict(do=0)),
    (NULLP, dict(dbeta=0, db=0)), (NULLP, dict(al=0)), (NULLP, dict(idx=0)),
    (NULLP, dict(pool=0)), (NULLP, dict(ws=0)),
    (SEQ, dict(cu=(1, 10, 30))), (SEQ, dict(cu=(0, 31, 30))), (SEQ, dict(cu=(0, 10, 29))),
    (STRIDE, dict(s=(-1, 384, 384, 384, 3))), (STRIDE, dict(dos=-1)),
    (STRIDE, dict(os=(383, 384, 384, 384, 3))), (STRIDE, dict(os=(384, 384, 384, 384, 2))),
    (STRIDE, dict(os=(384, 384, 384, 100, 3))), (STRIDE, dict(ss=100)),
    (WS, dict(wb=1000)),
    (OK, dict(n=0, T=0, cu=(0,), da=0, dd=0)),
])
def test_refusals(lib, want, kw):
    assert _call(lib, **kw) == want


def test_workspace_size(lib):
    size = kda.kda_prefill_backward_workspace_size
    per = size(1, 0, 1)
    assert per > 0 and size(1, 64, 1) == 2 * per and size(3, 127, 5) == 4 * 5 * per
    assert size(0, 0, 1) == 0 and size(-1, 5, 1) == 0 and size(1, 5, 0) == 0
    assert lib.kda_prefill_backward_workspace_size(1, 64, 1, 64, 128) == 0


# ---------------------------------------------------------------------------
# the recurrence in 64 bits, token by token, and its derivative by autograd

def make(lens, H, gate=0, seed=0, state=None, dfinal=False, scale=0.3, lb=-5.0, idx=None,
         spread=False):
    g = torch.Generator().manual_seed(seed)
    T, W, n = sum(lens), H * D, len(lens)

    def rnd(*shape):
        return torch.randn(*shape, generator=g)

    gw = H if gate & HEAD else W
    c = dict(lens=lens, H=H, gate=gate, scale=scale, lb=lb)
    for name in ("q", "k", "v", "do"):
        c[name] = rnd(T, W).to(BF)
    if gate & PRE:
        x = torch.rand(T, gw, generator=g) * 5.6 - 5.1
        c["g"] = torch.where(torch.rand(T, gw, generator=g) < 0.6, x * 0.03, x).to(BF)
    else:
        c["g"] = (rnd(T, gw) * (4.0 if spread else 1.0)).to(BF)
    c["b"] = (torch.rand(T, H, generator=g) if gate & PRESIG else rnd(T, H)).to(BF)
    c["A"] = torch.rand(H, generator=g) * 2 - 1
    c["dt"] = 0.1 * rnd(gw)
    N = n + 2
    c["pool"] = (0.2 * rnd(N, H, D, D)).to(state or BF)
    c["ui"] = state is not None
    c["idx"] = torch.randperm(N, generator=g)[:n].to(torch.int32) if idx is None \
        else torch.tensor(idx, dtype=torch.int32)
    c["df"] = rnd(n, H, D, D) if dfinal else None
    return c


def forward64(c, q, k, v, g, b, A, dt, S0):
    """Outputs [T, H, 128] and final states, differentiable."""
    H, gate = c["H"], c["gate"]
    T = q.shape[0]
    q, k, v = (x.reshape(T, H, D) for x in (q, k, v))
    q = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + 1e-6)
    k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + 1e-6)
    g = g.reshape(T, H, -1)
    if gate & PRE:
        g = g.clamp(c["lb"], 0.0)
    else:
        x = g + dt.reshape(H, -1)
        g = (-torch.exp(A)[:, None] * torch.where(x > 20, x, torch.log1p(torch.exp(x)))) \
            .clamp(min=c["lb"])
    a = torch.exp(g.expand(T, H, D))
    b = b if gate & PRESIG else torch.sigmoid(b)
    outs, finals, t = [], [], 0
    for d, n in enumerate(c["lens"]):
        S = S0[d]
        for _ in range(n):
            S = S * a[t][:, None]
            u = b[t][:, None] * (v[t] - (S * k[t][:, None]).sum(-1))
            S = S + u[:, :, None] * k[t][:, None]
            outs.append(c["scale"] * (S * q[t][:, None]).sum(-1))
            t += 1
        finals.append(S)
    return (torch.stack(outs) if outs else v.new_zeros(0, H, D)), torch.stack(finals)


def reference(c):
    n, H = len(c["lens"]), c["H"]
    ins = [c[x].double().requires_grad_() for x in ("q", "k", "v", "g", "b", "A", "dt")]
    N = c["pool"].shape[0]
    act = [0 <= int(i) < N for i in c["idx"]]
    S0 = torch.zeros(n, H, D, D, dtype=torch.float64)
    if c["ui"]:
        for d in range(n):
            if act[d]:
                S0[d] = c["pool"][int(c["idx"][d])].double()
    S0.requires_grad_()
    out, fin = forward64(c, *ins, S0)
    w = torch.cat([torch.full((x,), float(a)) for x, a in zip(c["lens"], act)]) \
        if sum(c["lens"]) else torch.zeros(0)
    loss = (out * c["do"].double().reshape(out.shape) * w.reshape(-1, 1, 1)).sum()
    if c["df"] is not None:
        loss = loss + (fin * c["df"].double() * torch.tensor(act).double()
                       .reshape(-1, 1, 1, 1)).sum()
    if loss.requires_grad:
        loss.backward()
    gr = [x.grad if x.grad is not None else torch.zeros_like(x) for x in ins]
    return gr, (S0.grad if S0.grad is not None else torch.zeros_like(S0))


def run(c, pad=0, off=0, stream=None, workspace=None, want_di=True):
    def dev(t, like=False):
        rows, w = t.shape
        buf = torch.full((off + max(rows, 1) * (w + pad),), -7.0, dtype=t.dtype, device="cuda")
        view = buf[off:].as_strided((rows, w), (w + pad, 1))
        if not like:
            view.copy_(t)
        return view

    lens, H = c["lens"], c["H"]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    pre = bool(c["gate"] & PRE)
    o = {n: dev(c[m], like=True) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                             ("db", "b"))}
    o["dA"] = None if pre else torch.empty(H, device="cuda")
    o["ddt"] = None if pre else torch.empty(c["dt"].numel(), device="cuda")
    o["dS"] = torch.empty(len(lens), H, D, D, device="cuda") if want_di else None
    kda.kda_prefill_varlen_backward(
        cu, cu.cuda(), dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), dev(c["b"]),
        None if pre else c["A"].cuda(), None if pre else c["dt"].cuda(), c["pool"].cuda(),
        c["idx"].cuda(), dev(c["do"]), o["dq"], o["dk"], o["dv"], o["dg"], o["db"],
        dA_log=o["dA"], ddt_bias=o["ddt"],
        d_final_state=None if c["df"] is None else c["df"].cuda(), d_initial_state=o["dS"],
        workspace=workspace, use_initial_state=c["ui"], lower_bound=c["lb"], scale=c["scale"],
        gate_mode=c["gate"], stream=stream)
    return o


def close_rows(name, got, ref, lens, H):
    """bf16 rows: 2^-8 of the element plus 1e-4 of the document and head's largest."""
    got, ref = got.double().cpu().reshape(ref.shape[0], H, -1), ref.reshape(ref.shape[0], H, -1)
    t = 0
    for d, n in enumerate(lens):
        g, r = got[t:t + n], ref[t:t + n]
        if n:
            top = r.abs().amax((0, 2), keepdim=True)
            bad = ~((g - r).abs() <= 2.0 ** -8 * r.abs() + 1e-4 * top)
            assert not bad.any(), f"{name}, document {d}: {int(bad.sum())} of {bad.numel()}, " \
                f"first {bad.nonzero()[0].tolist()}, worst {float((g - r).abs().max()):.3e} of " \
                f"{float(top.max()):.3e}"
        t += n


def compare(c, o):
    lens, H = c["lens"], c["H"]
    torch.cuda.synchronize()
    gr, dS = reference(c)
    for name, r in zip(("dq", "dk", "dv", "dg", "db"), gr):
        close_rows(name, o[name], r, lens, H)
    if o["dA"] is not None:
        # terms of dA_log: dg_t g_t; of ddt_bias: the gate logits' gradients
        mag = gr[3].abs().reshape(-1, c["dt"].numel()).sum(0)
        assert ((o["ddt"].double().cpu() - gr[6]).abs() <= 2e-5 * mag + 1e-30).all()
        x = c["g"].double() + c["dt"].double()
        ratio = torch.log1p(torch.exp(x)) / torch.sigmoid(x)
        mag = (gr[3] * ratio).abs().reshape(-1, H, c["dt"].numel() // H).sum((0, 2))
        assert ((o["dA"].double().cpu() - gr[5]).abs() <= 2e-5 * mag + 1e-30).all()
    if o["dS"] is not None:
        top = dS.abs().amax((2, 3), keepdim=True)
        assert ((o["dS"].double().cpu() - dS).abs() <= 1e-5 * top).all()


# lengths around the 16-token blocks and the 64-token chunks
@pytest.mark.gpu
@pytest.mark.parametrize("lens", [(1,), (2,), (15,), (16,), (17,), (63,), (64,), (65,), (128,),
                                  (129, 1), (20, 13), (0, 5, 0, 64, 0), (200, 64, 3)], ids=str)
def test_lengths(lens):
    c = make(lens, H=2, seed=sum(lens))
    compare(c, run(c))


@pytest.mark.gpu
@pytest.mark.parametrize("gate", range(8))
@pytest.mark.parametrize("state,dfinal", [(None, False), (BF, True)])
def test_gates(gate, state, dfinal):
    c = make((70, 9), H=3, gate=gate, seed=gate + 10, state=state, dfinal=dfinal)
    compare(c, run(c))


@pytest.mark.gpu
@pytest.mark.parametrize("state", [BF, torch.float16, torch.float8_e4m3fn], ids=str)
def test_state_types_strides_and_inactive(state):
    # slots: one shared by two documents, one below and one past the pool
    c = make((40, 33, 70, 5), H=2, seed=3, state=state, dfinal=True, idx=(1, -1, 1, 6))
    o = run(c, pad=3, off=1)
    compare(c, o)
    dead = torch.cat([o["dq"][40:73], o["dk"][143:], o["dg"][40:73]])
    assert (dead.view(torch.int16) == 0).all()  # +0.0
    assert (o["dS"][1] == 0).all() and (o["dS"][3] == 0).all()
    for n in ("dq", "dk", "dv", "dg", "db"):  # the padding between rows stays
        v = o[n]
        rows, w = v.shape
        gaps = v.as_strided((rows - 1, 3), (w + 3, 1), v.storage_offset() + w)
        assert (gaps == -7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("lb,spread", [(-5.0, True), (-5.5, True), (0.0, False), (-0.01, False)])
def test_gate_extremes(lb, spread):
    """Gates that hit the clamp for whole runs of tokens, and hardly any decay."""
    c = make((90, 20), H=2, seed=5, lb=lb, spread=spread)
    compare(c, run(c))
    c = make((90, 20), H=2, gate=PRE, seed=6, lb=lb)
    c["g"][10:40] = -20.0   # below the bound: no gradient
    c["g"][50:60] = 0.0     # exactly at the upper border: passes
    c["g"][60:70] = 0.5
    compare(c, run(c))


@pytest.mark.gpu
def test_gates_at_the_bound_for_whole_blocks():
    """Every gate at -5.5: 88 per block, the largest factors."""
    c = make((64, 30), H=1, gate=PRE, seed=7, lb=-5.5, state=BF, dfinal=True)
    c["g"][:] = -5.5
    c["g"][16] = 0.0  # one token that keeps the block before it
    compare(c, run(c))


@pytest.mark.gpu
def test_degenerate_inputs():
    """Zero keys and queries, beta of zero and one, a repeated key."""
    c = make((80,), H=2, gate=PRESIG, seed=8)
    c["q"][3] = 0
    c["k"][5] = 0
    c["b"][7:20] = 0.0
    c["b"][20:30] = 1.0
    c["k"][30:40] = c["k"][30]
    o = run(c)
    torch.cuda.synchronize()
    gr, _ = reference(c)
    # the norm of an all-zero row has the slope 1 / sqrt(1e-6) = 1000, so those rows dwarf
    # the others: they are compared apart
    for name, r, rows in (("dq", gr[0], [3]), ("dk", gr[1], [5])):
        got = o[name].double().cpu()
        keep = [t for t in range(80) if t not in rows]
        for sel in (rows, keep):
            close_rows(name, got[sel], r[sel], (len(sel),), 2)
    for name, r in zip(("dv", "dg", "db"), gr[2:5]):
        close_rows(name, o[name], r, c["lens"], 2)


@pytest.mark.gpu
@pytest.mark.parametrize("do,v,state", [(1e-8, 1.0, 0.2), (1e4, 1e-3, 1e-6), (1e-3, 300.0, 50.0),
                                        (1e20, 1e-20, 1e-20), (0.0, 1.0, 1.0)])
def test_magnitudes(do, v, state):
    """Loss scales and value sizes far from 1: the products' operands are scaled to fp16's
    range, so the errors stay relative to the results. (The state gradient at the end has
    the size of do.)"""
    c = make((150, 20), H=2, seed=30, state=BF, dfinal=True)
    for n, f in (("do", do), ("v", v)):
        c[n] = (c[n].float() * f).to(BF)
    c["pool"] = (c["pool"].float() * (state / 0.2)).to(BF)
    c["df"] = c["df"] * do
    compare(c, run(c))


@pytest.mark.gpu
def test_beta_as_given():
    """Given betas need not lie in (0, 1): zero, negative and beyond 1 (up to 2 the
    recurrence is stable; a few beyond grow it)."""
    c = make((130,), H=2, gate=PRESIG | PRE, seed=31, state=BF, dfinal=True)
    c["b"] = (c["b"].float() * 2.4 - 0.2).to(BF)
    c["b"][40:44] = 3.0
    c["b"][60:63] = -1.5
    compare(c, run(c))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.7, 25.0])
def test_scale(scale):
    c = make((70,), H=2, seed=32, scale=scale, dfinal=True)
    compare(c, run(c))


@pytest.mark.gpu
def test_no_tokens():
    c = make((0, 0), H=2, seed=9, state=BF, dfinal=True)
    o = run(c)
    torch.cuda.synchronize()
    assert torch.equal(o["dS"].cpu(), c["df"])
    assert (o["dA"] == 0).all() and (o["ddt"] == 0).all()


@pytest.mark.gpu
def test_two_calls_at_once():
    """On two streams, with workspaces of their own: each gives what it gives alone."""
    cs = [make((300, 40), H=3, seed=61, state=BF, dfinal=True), make((500,), H=20, seed=62)]
    alone = [run(c) for c in cs]
    ws = [torch.empty(kda.kda_prefill_backward_workspace_size(len(c["lens"]), sum(c["lens"]),
                                                              c["H"]),
                      dtype=torch.uint8, device="cuda") for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = []
        for c, st, w in zip(cs, streams, ws):
            with torch.cuda.stream(st):
                got.append(run(c, workspace=w, stream=st))
        torch.cuda.synchronize()
        for o, one in zip(got, alone):
            for n, t in one.items():
                assert t is None or torch.equal(o[n], t), n


# the chains' forms: four long documents in the one of least latency and the rest in the
# wide one; all in the first; all in the second; a document count that leaves blocks over
@pytest.mark.gpu
@pytest.mark.parametrize("lens,H", [((65, 0, 200, 7, 130, 64, 71, 1), 8), ((200,), 20),
                                    ((129, 70), 40), ((193, 3, 80, 66, 5, 64, 1), 3)], ids=str)
@pytest.mark.parametrize("state,dfinal", [(None, False), (BF, True)])
def test_chain_forms(lens, H, state, dfinal):
    c = make(lens, H=H, seed=50 + H, state=state, dfinal=dfinal)
    compare(c, run(c))


@pytest.mark.gpu
def test_many_documents():
    """More documents than the ordered launch holds."""
    lens = tuple([3, 0, 17, 1] * 70)
    c = make(lens, H=1, seed=10)
    compare(c, run(c))


@pytest.mark.gpu
def test_long_document_against_its_halves():
    """One document of 1500 tokens equals its two parts run apart, the state passed up
    and its gradient passed down, within the fp32 arithmetic: the parts' boundary (700)
    is no multiple of the chunk."""
    H, cut = 4, 700
    c = make((1500,), H=H, seed=11, state=BF, dfinal=True)
    whole = run(c)
    # the state after `cut` tokens, in 64 bits, handed on through an fp16 pool
    a = {k: (v[:cut] if k in ("q", "k", "v", "do", "g", "b") else v) for k, v in c.items()}
    b = {k: (v[cut:] if k in ("q", "k", "v", "do", "g", "b") else v) for k, v in c.items()}
    a["lens"], b["lens"] = (cut,), (1500 - cut,)
    with torch.no_grad():
        S0 = c["pool"][c["idx"].long()].double()
        _, S = forward64(a, *(a[x].double() for x in ("q", "k", "v", "g", "b", "A", "dt")), S0)
    b["pool"], b["idx"] = S.to(torch.float16), torch.zeros(1, dtype=torch.int32)
    second = run(b)
    a["df"] = second["dS"].cpu()
    first = run(a)
    torch.cuda.synchronize()
    # fp16 rounds the state by 2^-11 of each element (random signs): the second
    # part's gradients move by about that much of their size, normwise
    for n in ("dq", "dk", "dv", "dg", "db"):
        w = whole[n].double().cpu()
        both = torch.cat([first[n], second[n]]).double().cpu()
        assert (w - both).norm() <= (2.0 ** -8 + 2.0 ** -10) * w.norm()
    assert (first["dS"] - whole["dS"]).norm() <= 2.0 ** -10 * whole["dS"].norm()


@pytest.mark.gpu
def test_against_differences_of_the_forward_kernel():
    """The gradient along a random direction of v (the output is linear in v up to
    rounding) and of the state, against kda_prefill_varlen itself."""
    H, lens = 2, (75, 30)
    c = make(lens, H=H, seed=12, state=torch.float16)
    o = run(c)
    cu = torch.tensor([0, 75, 105], dtype=torch.int32)

    def out_of(v):
        out = torch.empty(105, H * D, dtype=BF, device="cuda")
        kda.kda_prefill_varlen(cu, cu.cuda(), c["q"].cuda(), c["k"].cuda(), v.cuda(),
                               c["g"].cuda(), c["b"].cuda(), c["A"].cuda(), c["dt"].cuda(),
                               c["pool"].cuda(), c["idx"].cuda(), out, lower_bound=c["lb"],
                               scale=c["scale"])
        return out.double().cpu()

    dv = 4 * torch.randn(c["v"].shape, generator=torch.Generator().manual_seed(1))
    up, down = (c["v"].float() + dv).to(BF), (c["v"].float() - dv).to(BF)
    diff = (out_of(up) - out_of(down)) * c["do"].double()
    slope = (o["dv"].double().cpu() * (up.double() - down.double())).sum()
    # forward outputs are rounded to bf16 with up to 5e-3 of error normwise
    assert abs(diff.sum() - slope) <= 1e-2 * diff.norm() + 1e-2 * abs(slope)


@pytest.mark.gpu
def test_same_bits_workspace_and_stream():
    """Twice the same bits, on a side stream too, whatever the workspace held."""
    c = make((300, 64, 130), H=5, seed=13, state=BF, dfinal=True)
    need = kda.kda_prefill_backward_workspace_size(3, 494, 5)
    a = run(c)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    b = run(c, workspace=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    d = run(c, workspace=ws, stream=s)
    s.synchronize()
    for n, x in a.items():
        assert torch.equal(x, b[n]) and torch.equal(x, d[n]), n
    no = run(c, want_di=False)
    torch.cuda.synchronize()
    assert torch.equal(no["dq"], a["dq"])


@pytest.mark.gpu
def test_captured():
    """Two captured calls with a workspace each, replayed with changed inputs and eager
    calls between."""
    H, T = 3, 150
    cases = [make((100, 50), H=H, seed=20 + i) for i in range(3)]
    cu = torch.tensor([0, 100, 150], dtype=torch.int32)
    ins = {n: cases[0][n].cuda() for n in ("q", "k", "v", "g", "b", "do", "A", "dt", "pool", "idx")}
    cud = cu.cuda()
    need = kda.kda_prefill_backward_workspace_size(2, T, H)

    def call(ws):
        o = [torch.empty_like(ins[n]) for n in ("q", "k", "v", "g", "b", "A", "dt")]
        kda.kda_prefill_varlen_backward(
            cu, cud, ins["q"], ins["k"], ins["v"], ins["g"], ins["b"], ins["A"], ins["dt"],
            ins["pool"], ins["idx"], ins["do"], *o[:5], dA_log=o[5], ddt_bias=o[6], workspace=ws,
            use_initial_state=False, scale=0.3)
        return o

    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(3)]
    call(ws[2])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(ws[i]))
        graphs.append(g)
    for c in cases:
        for n, t in ins.items():
            t.copy_(c[n])
        for g in graphs:
            g.replay()
        eager = call(ws[2])
        torch.cuda.synchronize()
        for o in outs:
            for x, y in zip(o, eager):
                assert torch.equal(x, y)


@pytest.mark.gpu
def test_a_layer_forward_and_backward():
    """The calls of a training step together: residual norm, prefill, gated norm per
    head, and their gradients back to the residual stream; q, k and v are the normed stream
    itself (as if the projections were the identity), so its gradient is the sum of three.
    Each call is held to its formula in 64 bits on what it was given: a bound on the whole
    would have to follow every bf16 value in between through the divisions of the norms.
    A bf16 result is off by 2^-8 of each element and the fp32 arithmetic, so normwise by
    at most 2^-8 + 2e-4."""
    H, lens = 2, (75, 20)
    T, W = sum(lens), H * D
    c = make(lens, H=H, seed=40, scale=D ** -0.5)
    g = torch.Generator().manual_seed(41)
    x, r, og = (torch.randn(T, W, generator=g).to(BF) for _ in range(3))
    dy, dr = (torch.randn(T, W, generator=g).to(BF) for _ in range(2))
    w1, w2 = 1 + 0.1 * torch.randn(W, generator=g), 1 + 0.1 * torch.randn(D, generator=g)
    cu = torch.tensor([0, 75, 95], dtype=torch.int32)
    dev = {n: t.cuda() for n, t in dict(x=x, r=r, og=og, dy=dy, dr=dr, w1=w1, w2=w2, g=c["g"],
                                       b=c["b"], A=c["A"], dt=c["dt"], cu=cu,
                                       idx=c["idx"]).items()}
    new = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    z, u, o, y = new(T, W), new(T, W), new(T, W), new(T, H, D)
    kda.kda_rmsnorm(dev["x"], dev["w1"], u, residual=dev["r"], residual_out=z)
    pool = c["pool"].cuda()
    kda.kda_prefill_varlen(cu, dev["cu"], u, u, u, dev["g"], dev["b"], dev["A"], dev["dt"], pool,
                           dev["idx"], o, use_initial_state=False, scale=c["scale"])
    kda.kda_rmsnorm(o.view(T, H, D), dev["w2"], y, gate=dev["og"].view(T, H, D))
    do, dog, dw2 = new(T, H, D), new(T, H, D), torch.empty(D, device="cuda")
    kda.kda_rmsnorm_backward(o.view(T, H, D), dev["w2"], dev["dy"].view(T, H, D), do, dw2,
                             gate=dev["og"].view(T, H, D), dgate=dog)
    dq, dk, dv, dg, db = new(T, W), new(T, W), new(T, W), new(T, W), new(T, H)
    dA, ddt = torch.empty(H, device="cuda"), torch.empty(W, device="cuda")
    kda.kda_prefill_varlen_backward(cu, dev["cu"], u, u, u, dev["g"], dev["b"], dev["A"],
                                    dev["dt"], pool, dev["idx"], do.view(T, W), dq, dk, dv, dg,
                                    db, dA_log=dA, ddt_bias=ddt, use_initial_state=False,
                                    scale=c["scale"])
    dz, dw1 = new(T, W), torch.empty(W, device="cuda")
    kda.kda_rmsnorm_backward(z, dev["w1"], dq + dk + dv, dz, dw1, d_residual=dev["dr"])
    torch.cuda.synchronize()

    from tests.helpers import OUT_NORM_PREFILL

    def far(got, ref):
        return float((got.double().cpu().reshape(ref.shape) - ref).norm() / ref.norm())

    def norm(z, w, gate=None):
        n = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + 1e-6) * w
        return n if gate is None else n * torch.sigmoid(gate)

    def grads(out, dy, *leaves):
        return torch.autograd.grad((out * dy).sum(), leaves)

    bf = 2.0 ** -8 + 2e-4
    back = {n: t.double().cpu() for n, t in dict(z=z, u=u, o=o, do=do).items()}
    Z = x.double() + r.double()
    assert torch.equal(z.cpu(), Z.to(BF)) and far(u, norm(Z, w1.double())) <= bf
    zeros = torch.zeros(2, H, D, D, dtype=torch.float64)
    O, _ = forward64(c, back["u"], back["u"], back["u"], *(c[n].double() for n in
                                                           ("g", "b", "A", "dt")), zeros)
    assert far(o, O) <= OUT_NORM_PREFILL
    ol, wl, gl = (t.requires_grad_() for t in (back["o"].reshape(T, H, D), w2.double(),
                                               og.double().reshape(T, H, D)))
    Y = norm(ol, wl, gl)
    assert far(y, Y.detach()) <= bf
    for got, ref in zip((do, dw2, dog), grads(Y, dy.double().reshape(T, H, D), ol, wl, gl)):
        assert far(got, ref) <= bf
    step = dict(c, q=u.cpu(), k=u.cpu(), v=u.cpu(), do=do.cpu().view(T, W))
    compare(step, dict(dq=dq, dk=dk, dv=dv, dg=dg, db=db, dA=dA, ddt=ddt, dS=None))
    zl, wl = back["z"].requires_grad_(), w1.double().requires_grad_()
    dZ, dW = grads(norm(zl, wl), (dq + dk + dv).double().cpu(), zl, wl)
    assert far(dz, dZ + dr.double()) <= bf and far(dw1, dW) <= 1e-5


@pytest.mark.gpu
def test_binding_refuses():
    c = make((10,), H=2, seed=1)
    c["b"] = c["b"][:, :1]
    with pytest.raises(ValueError, match="beta_raw"):
        run(c)
    c = make((10,), H=2, seed=1)
    with pytest.raises(kda.KdaError):
        run(c, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


# gate logits plus bias of a trained or freshly initialised layer: decays of 1e-1 to 1e-8
@pytest.mark.gpu
@pytest.mark.parametrize("bias,A", [(-2.0, 2.7), (-4.0, 0.0), (-7.0, 0.0), (-9.0, 2.7), (-12.0, 0.0),
                                    (-15.0, 2.7), (-18.0, 0.0), (-40.0, 0.0)])
@pytest.mark.parametrize("gate,alike", [(0, False), (0, True), (HEAD, False)],
                         ids=["spread", "alike", "per head"])
def test_slow_decay(bias, A, gate, alike):
    """Raw gates whose softplus is small: dA_log is the sum of dg g, so the log-decay itself has
    to be right relative to its size. `alike`: one logit for all tokens, whose rounding errors
    add up.

    Tolerances: those of the other cases, and what 300 tokens add to a decay that is nearly 1:
    each a_t = e^g_t is off by 2^-24 (one step below 1), the product of the decays by half of
    that again, in the same direction where the tokens are alike, so a weight is off by
    300 * 1.5 * 2^-24 = 2.7e-5. The softplus adds nothing to speak of: the exponential's
    argument is rounded twice, 2 * 2^-24 |y| < 5e-6 of it at y = -40."""
    c = make((300, 65), H=2, gate=gate, seed=70, state=BF, dfinal=True)
    c["dt"] += bias
    c["A"] += A
    if alike:
        c["g"][:] = c["g"][0]
    o = run(c)
    torch.cuda.synchronize()
    (*rows, dA, ddt), dS = reference(c)
    far, H = 300 * 1.5 * 2.0 ** -24, c["H"]
    t = 0
    for n in c["lens"]:
        for name, r in zip(("dq", "dk", "dv", "dg", "db"), rows):
            got = o[name][t:t + n].double().cpu().reshape(n, H, -1)
            ref = r[t:t + n].reshape(n, H, -1)
            top = ref.abs().amax((0, 2), keepdim=True)
            assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (1e-4 + far) * top).all(), name
        t += n
    x = c["g"].double() + c["dt"].double()
    terms = rows[3].reshape(-1, H, x.shape[1] // H)
    mag = terms.abs().sum(0).reshape(-1)
    assert ((o["ddt"].double().cpu() - ddt).abs() <= (2e-5 + far) * mag).all()
    ratio = (torch.log1p(torch.exp(x)) / torch.sigmoid(x)).reshape(terms.shape)
    mag = (terms * ratio).abs().sum((0, 2))
    assert ((o["dA"].double().cpu() - dA).abs() <= (2e-5 + far) * mag).all()
    top = dS.abs().amax((2, 3), keepdim=True)
    assert ((o["dS"].double().cpu() - dS).abs() <= (1e-5 + far) * top).all()


@pytest.mark.gpu
def test_saturated_beta():
    """Beta logits of -30 .. 30, dbeta to half a bf16 step of each element and 1e-4 of the
    largest derivative by beta itself times the sigmoid's slope: beta (1 - beta) does not
    cancel, its exponential is off by 2 * 2^-24 * 30 = 4e-6 of it."""
    c = make((61, 61), H=2, seed=71, scale=D ** -0.5)
    c["b"] = (torch.arange(-30.0, 31.0).repeat(2)[:, None] + torch.tensor([0.0, 0.3])).to(BF)
    o = run(c)
    torch.cuda.synchronize()
    got = o["db"].double().cpu()
    # the derivative by beta, with beta as given (to 64 bits), times the slope
    x = c["b"].double()
    p = dict(c, gate=PRESIG, b=torch.sigmoid(x))
    by_beta = reference(p)[0][4].reshape(x.shape)
    slope = torch.sigmoid(x) * torch.sigmoid(-x)
    top = torch.cat([t.abs().amax(0).expand(61, 2) for t in by_beta.split(61)])
    assert ((got - by_beta * slope).abs() <= (2.0 ** -8 * by_beta.abs() + 1e-4 * top) * slope).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 40])
def test_no_documents(H):
    """No documents at all: dA_log and ddt_bias become zeros, whatever else is given."""
    lib = kda.lib()
    dA, ddt = torch.full((H,), 7.0, device="cuda"), torch.full((H * D,), 7.0, device="cuda")
    di = torch.full((4,), 7.0, device="cuda")
    assert di.data_ptr() % 16 == 0
    args = dict(n=0, T=0, H=H, cu=(0,), da=dA.data_ptr(), dd=ddt.data_ptr(), ss=H * 16384,
                s=(H * D,) * 4 + (H,), os=(H * D,) * 4 + (H,), dos=H * D)
    for d_initial in (di.data_ptr(), 0):
        dA.fill_(7.0)
        ddt.fill_(7.0)
        assert _call(lib, di=d_initial, **args) == OK
        torch.cuda.synchronize()
        assert (dA == 0).all() and (ddt == 0).all() and (di == 7.0).all()
    assert _call(lib, **dict(args, da=0, dd=0, di=di.data_ptr())) == OK


@pytest.mark.gpu
def test_state_gradients_in_one_tensor():
    """d_initial_state may be d_final_state itself: documents of no tokens, one, several
    chunks, an inactive one, in each of the chains' forms."""
    for lens, H in (((70, 0, 1, 33), 2), ((130, 66, 1, 0), 20)):
        c = make(lens, H=H, seed=72, state=BF, dfinal=True, idx=(1, 0, 3, -1))
        apart = run(c)["dS"]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        x = {n: c[n].cuda() for n in ("q", "k", "v", "g", "b", "do", "A", "dt", "pool", "idx")}
        o = [torch.empty_like(x[n]) for n in ("q", "k", "v", "g", "b")]
        both = c["df"].cuda()
        kda.kda_prefill_varlen_backward(
            cu, cu.cuda(), x["q"], x["k"], x["v"], x["g"], x["b"], x["A"], x["dt"], x["pool"],
            x["idx"], x["do"], *o, d_final_state=both, d_initial_state=both, scale=c["scale"])
        torch.cuda.synchronize()
        assert torch.equal(both, apart)


@pytest.mark.gpu
def test_long_document_of_slow_decay():
    """20,000 tokens in one document, decays of 1e-4 a token, against the recurrence in 64 bits
    token by token on the GPU (one head, states kept every 100 tokens).

    Tolerances: as in test_slow_decay, with the tokens that a state remembers: a write takes
    beta (2 - beta) of the state along its key, 0.75 / 128 of its square on average, so after
    2000 tokens less than e^-5 is left, and 2000 * 1.5 * 2^-24 = 1.8e-4 covers the decays."""
    T, far = 20000, 2000 * 1.5 * 2.0 ** -24
    c = make((T,), H=1, seed=73, dfinal=True, state=BF, scale=D ** -0.5)
    c["dt"] -= 9.0
    o = run(c)
    f64 = {n: c[n].double().cuda() for n in ("q", "k", "v", "do", "g", "b", "A", "dt")}
    nq, nk = (torch.sqrt(f64[n].pow(2).sum(-1, keepdim=True) + 1e-6) for n in ("q", "k"))
    q, k, v, do = f64["q"] / nq, f64["k"] / nk, f64["v"], f64["do"]
    x = f64["g"] + f64["dt"]
    ea, beta = torch.exp(f64["A"]), torch.sigmoid(f64["b"])
    g = -ea * torch.log1p(torch.exp(x))
    a, sc = torch.exp(g), c["scale"]
    S = c["pool"][int(c["idx"][0])][0].double().cuda()

    def step(S, t):  # decayed state, x, u, state
        Sd = S * a[t]
        r = v[t] - Sd @ k[t]
        return Sd, r, beta[t] * r, torch.addr(Sd, beta[t] * r, k[t])

    kept = []
    for t in range(T):
        if t % 100 == 0:
            kept.append(S)
        S = step(S, t)[3]
    dS = c["df"][0, 0].double().cuda()
    dq, dk, dv, dg = (torch.empty_like(q) for _ in range(4))
    db = torch.empty_like(beta)
    for s in reversed(range(len(kept))):
        S, seg = kept[s], []
        for t in range(100 * s, 100 * s + 100):
            seg.append(step(S, t))
            S = seg[-1][3]
        for t in reversed(range(100 * s, 100 * s + 100)):
            Sd, r, u, S1 = seg[t - 100 * s]
            dq[t] = sc * (do[t] @ S1)
            dS = torch.addr(dS, do[t], sc * q[t])
            du = dS @ k[t]
            db[t, 0] = du @ r
            dv[t] = beta[t] * du
            dk[t] = u @ dS - dv[t] @ Sd
            dS = torch.addr(dS, -dv[t], k[t])
            dg[t] = (dS * Sd).sum(0)
            dS = dS * a[t]
    dq = (dq - q * (q * dq).sum(-1, keepdim=True)) / nq
    dk = (dk - k * (k * dk).sum(-1, keepdim=True)) / nk
    db = db * beta * torch.sigmoid(-f64["b"])
    slope = -ea * torch.sigmoid(x)
    for name, ref in (("dq", dq), ("dk", dk), ("dv", dv), ("dg", dg * slope), ("db", db)):
        err = (o[name].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + (1e-4 + far) * ref.abs().max()).all(), name
    assert ((o["ddt"].double() - (dg * slope).sum(0)).abs() <=
            (2e-5 + far) * (dg * slope).abs().sum(0)).all()
    assert abs(o["dA"].double() - (dg * g).sum()) <= (2e-5 + far) * (dg * g).abs().sum()
    assert ((o["dS"][0, 0].double() - dS).abs() <= (1e-5 + far) * dS.abs().max()).all()


@pytest.mark.gpu
def test_strides_past_32_bits():
    """Tokens 2^21 elements apart: 1100 of them span 2.3e9 elements (4.6 GB). The same bits as
    from packed rows."""
    lens, H, stride = (1000, 0, 100), 1, 1 << 21
    c = make(lens, H=H, seed=74, state=BF, dfinal=True)
    want = run(c)
    T = sum(lens)
    ins = torch.empty(T * stride, dtype=BF, device="cuda")
    outs = torch.empty(T * stride, dtype=BF, device="cuda")

    def at(buf, col, t):
        return buf[col:].as_strided(tuple(t.shape), (stride, 1))

    x = {}
    for i, n in enumerate(("q", "k", "v", "g", "do", "b")):
        x[n] = at(ins, stride - 1000 + 129 * i, c[n])
        x[n].copy_(c[n])
    o = {n: at(outs, 131 * i + 5, c[m])
         for i, (n, m) in enumerate((("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("db", "b")))}
    dA, ddt = torch.empty(H, device="cuda"), torch.empty(H * D, device="cuda")
    dS = torch.empty(3, H, D, D, device="cuda")
    cu = torch.tensor([0, 1000, 1000, 1100], dtype=torch.int32)
    kda.kda_prefill_varlen_backward(
        cu, cu.cuda(), x["q"], x["k"], x["v"], x["g"], x["b"], c["A"].cuda(), c["dt"].cuda(),
        c["pool"].cuda(), c["idx"].cuda(), x["do"], *o.values(), dA_log=dA, ddt_bias=ddt,
        d_final_state=c["df"].cuda(), d_initial_state=dS, scale=c["scale"])
    torch.cuda.synchronize()
    for n, t in o.items():
        assert torch.equal(t, want[n]), n
    assert torch.equal(dA, want["dA"]) and torch.equal(ddt, want["ddt"])
    assert torch.equal(dS, want["dS"])
