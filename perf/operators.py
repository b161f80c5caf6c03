"""Workloads of the recurrence's gradient and of the RMS norm around it.

Three operators, as a trainer or a server of a KDA layer calls them:

  prefill_backward  gradients of one packed-document prefill call
  rmsnorm           residual addition + RMS norm (+ sigmoid gate), output in
                    bf16 or in fp8 e4m3 with scales
  rmsnorm_backward  its gradients

`own` selects the library's calls (True) or the plain form in elementary
torch operations (False). `exact` follows the definitions in 64 bits, the
recurrence token by token where the plain form goes chunk by chunk.
"""
from __future__ import annotations

import math

import torch

own = False

D = 128
EPS = 1e-6
LOWER_BOUND = -5.0
GATE_PRECOMPUTED, BETA_PRESIGMOID, GATE_PER_HEAD = 1, 2, 4
FP8_MAX = 448.0


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # two short documents of a small model: the smallest gradient call
        dict(name="bwd_short", op="bwd", docs="20,13", H=2, gate=0, state="none", dfinal=False),
        # the repository's 14-document mix of 16384 tokens, 12 heads, from zeros
        dict(name="bwd_mix14", op="bwd",
             docs="4096,3000,2048,1500,1200,1024,1000,700,600,500,300,217,128,71", H=12, gate=0,
             state="none", dfinal=False),
        # one long document continued from a stored state, whose later part
        # sends a state gradient back (a sequence trained in segments)
        dict(name="bwd_long1", op="bwd", docs="8191", H=12, gate=3, state="bf16", dfinal=True),
        # a whole training batch: 64 heads, ragged lengths, an empty document
        dict(name="bwd_large", op="bwd", docs="4096,2500,0,1024,517,71", H=64, gate=0,
             state="none", dfinal=False),
        # one decay per head (the scalar gate), half-precision initial states
        dict(name="bwd_perhead", op="bwd", docs="1000,700,333,1,64", H=16, gate=4, state="fp16",
             dfinal=True),
        # one decoded token's residual stream, fp8 for the next projections
        dict(name="norm_token", op="norm", rows=1, heads=1, width=1536, residual=True, gated=False,
             out="fp8", group=0),
        # a decode batch at the width of 64 heads, fp8 with a scale per 128
        dict(name="norm_batch", op="norm", rows=512, heads=1, width=8192, residual=True,
             gated=False, out="fp8", group=128),
        # a prefill's residual stream in bf16 (training keeps bf16)
        dict(name="norm_prefill", op="norm", rows=16384, heads=1, width=8192, residual=True,
             gated=False, out="bf16", group=0),
        # the recurrence's output rows, normalised per head and gated, fp8
        dict(name="norm_heads", op="norm", rows=13889, heads=12, width=128, residual=False,
             gated=True, out="fp8", group=0),
        # gradients of the residual norm over a training batch
        dict(name="norm_bwd_wide", op="norm_bwd", rows=8208, heads=1, width=8192, residual=True,
             gated=False),
        # gradients of the gated per-head norm
        dict(name="norm_bwd_heads", op="norm_bwd", rows=8208, heads=64, width=128, residual=False,
             gated=True),
        # an odd width and few rows
        dict(name="norm_bwd_odd", op="norm_bwd", rows=71, heads=1, width=1001, residual=True,
             gated=False),
    ]


def _loguni(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["bwd", "bwd", "norm", "norm_bwd"])
    if op == "bwd":
        H = _loguni(rng, 1, 64)
        n = rng.randint(1, 12)
        lens = [_loguni(rng, 1, 4000) for _ in range(n)]
        if rng.random() < 0.25:
            lens[rng.randrange(n)] = 0
        while H * sum(lens) > 520000 or H * n * max(lens) > 1500000:
            lens = [x * 2 // 3 for x in lens]
        if sum(lens) == 0:
            lens[0] = 1
        state = rng.choice(["none", "bf16", "fp16", "fp8"])
        return dict(op="bwd", docs=",".join(str(x) for x in lens), H=H,
                    gate=rng.choice([0, 0, 1, 2, 3, 4, 5, 7]), state=state,
                    dfinal=rng.random() < 0.5)
    if rng.random() < 0.5:
        heads, width, gated = _loguni(rng, 1, 64), D, True
    else:
        heads, width, gated = 1, _loguni(rng, 64, 8192), rng.random() < 0.2
        if rng.random() < 0.6:
            width = max(D, width // D * D)
    rows = _loguni(rng, 1, min(16384, 64000000 // (heads * width)))
    case = dict(op=op, rows=rows, heads=heads, width=width, residual=rng.random() < 0.6,
                gated=gated)
    if op == "norm":
        case["out"] = rng.choice(["bf16", "fp8"])
        case["group"] = D if width % D == 0 and rng.random() < 0.5 else 0
    return case


def _docs(case):
    return [int(x) for x in case["docs"].split(",")]


# ---------------------------------------------------------------------------
# inputs

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bf = torch.bfloat16
    if case["op"] != "bwd":
        shape = (case["rows"], case["heads"], case["width"])
        st = dict(case=case, x=_rand(gen, *shape).to(bf), residual=None, gate=None)
        st["weight"] = 1.0 + 0.1 * _rand(gen, case["width"])
        if case["residual"]:
            st["residual"] = (2.0 * _rand(gen, *shape)).to(bf)
        if case["gated"]:
            st["gate"] = _rand(gen, *shape).to(bf)
        if case["op"] == "norm":
            fp8 = case["out"] == "fp8"
            st["out"] = torch.empty(shape, device="cuda",
                                    dtype=torch.float8_e4m3fn if fp8 else bf)
            st["residual_out"] = torch.empty(shape, device="cuda", dtype=bf) \
                if case["residual"] else None
            cols = case["heads"] * (case["width"] // case["group"] if case["group"] else 1)
            st["scales"] = torch.empty(case["rows"], cols, device="cuda") if fp8 else None
        else:
            st["dy"] = _rand(gen, *shape).to(bf)
            st["dz"] = torch.empty(shape, device="cuda", dtype=bf)
            st["dgate"] = torch.empty(shape, device="cuda", dtype=bf) if case["gated"] else None
            st["dweight"] = torch.empty(case["width"], device="cuda")
        return st

    lens, H, gate = _docs(case), case["H"], case["gate"]
    n, T, W = len(lens), sum(lens), case["H"] * D
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st = dict(case=case, cu_host=torch.tensor(cu, dtype=torch.int32))
    st["cu"] = st["cu_host"].cuda()
    for name in ("q", "k", "v", "do"):
        st[name] = _rand(gen, T, W).to(bf)
    gw = H if gate & GATE_PER_HEAD else W
    if gate & GATE_PRECOMPUTED:  # log-decays, some of them outside [lower bound, 0]
        g = torch.rand(T, gw, generator=gen, device="cuda") * 5.6 - 5.1
        g = torch.where(torch.rand(T, gw, generator=gen, device="cuda") < 0.5, g * 0.05, g)
    else:
        g = _rand(gen, T, gw)
    st["g"] = g.to(bf)
    b = torch.rand(T, H, generator=gen, device="cuda") if gate & BETA_PRESIGMOID \
        else _rand(gen, T, H)
    st["beta"] = b.to(bf)
    st["A_log"] = torch.rand(H, generator=gen, device="cuda") * 2 - 1
    st["dt_bias"] = 0.1 * _rand(gen, gw)
    slots = 2 * n
    dtype = dict(none=bf, bf16=bf, fp16=torch.float16, fp8=torch.float8_e4m3fn)[case["state"]]
    st["use_initial"] = case["state"] != "none"
    st["pool"] = (0.05 * _rand(gen, slots, H, D, D)).to(dtype)
    st["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
    st["scale"] = D ** -0.5
    st["dstate"] = 0.1 * _rand(gen, n, H, D, D) if case["dfinal"] else None
    for name, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta")):
        st[name] = torch.empty_like(st[like])
    raw = not gate & GATE_PRECOMPUTED
    st["dA_log"] = torch.empty_like(st["A_log"]) if raw else None
    st["ddt_bias"] = torch.empty_like(st["dt_bias"]) if raw else None
    st["dinit"] = torch.empty(n, H, D, D, device="cuda") if st["use_initial"] else None
    return st


# ---------------------------------------------------------------------------
# one pass

def _workspace(st, size):
    """The workspace that a program keeps beside its plan (made on the first pass)."""
    if st.get("workspace") is None:
        st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _run_own(st):
    import gated_delta_rule_step_amd as kda
    case = st["case"]
    if case["op"] == "norm":
        kda.kda_rmsnorm(st["x"], st["weight"], st["out"], residual=st["residual"],
                        residual_out=st["residual_out"], gate=st["gate"], scales=st["scales"],
                        eps=EPS)
        return [st["out"], st["scales"], st["residual_out"]]
    if case["op"] == "norm_bwd":
        ws = _workspace(st, kda.kda_rmsnorm_backward_workspace_size(case["rows"], case["heads"],
                                                                    case["width"]))
        kda.kda_rmsnorm_backward(st["x"], st["weight"], st["dy"], st["dz"], st["dweight"],
                                 gate=st["gate"], dgate=st["dgate"], d_residual=st["residual"],
                                 eps=EPS, workspace=ws)
        return [st["dz"], st["dweight"], st["dgate"]]
    ws = _workspace(st, kda.kda_prefill_backward_workspace_size(
        st["cu_host"].shape[0] - 1, st["q"].shape[0], case["H"]))
    kda.kda_prefill_varlen_backward(
        st["cu_host"], st["cu"], st["q"], st["k"], st["v"], st["g"], st["beta"], st["A_log"],
        st["dt_bias"], st["pool"], st["slots"], st["do"], st["dq"], st["dk"], st["dv"], st["dg"],
        st["dbeta"], dA_log=st["dA_log"], ddt_bias=st["ddt_bias"], d_final_state=st["dstate"],
        d_initial_state=st["dinit"], workspace=ws, use_initial_state=st["use_initial"],
        lower_bound=LOWER_BOUND, scale=st["scale"], gate_mode=case["gate"])
    return [st["dq"], st["dk"], st["dv"], st["dg"], st["dbeta"], st["dA_log"], st["ddt_bias"],
            st["dinit"]]


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    return _plain_norm(st) if op == "norm" else \
        _plain_norm_backward(st) if op == "norm_bwd" else _plain_backward(st)


# ---------------------------------------------------------------------------
# plain forms

def _plain_norm(st):
    case = st["case"]
    z = st["x"].float()
    if case["residual"]:
        z = z + st["residual"].float()
    y = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * st["weight"]
    if case["gated"]:
        y = y * torch.sigmoid(st["gate"].float())
    zr = z.to(torch.bfloat16) if case["residual"] else None
    if case["out"] == "bf16":
        return [y.to(torch.bfloat16), None, zr]
    yg = y.reshape(case["rows"], -1, case["group"] or case["width"])
    scales = yg.abs().amax(-1) / FP8_MAX
    scales = torch.where(scales > 0, scales, 1.0)
    y8 = (yg / scales[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return [y8.reshape(y.shape), scales, zr]


def _plain_norm_backward(st):
    w, z, dy = st["weight"], st["x"].float(), st["dy"].float()
    rstd = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
    xh = z * rstd
    dgate = None
    if st["gate"] is not None:
        s = torch.sigmoid(st["gate"].float())
        dgate = (dy * xh * w * s * (1.0 - s)).to(torch.bfloat16)
        dy = dy * s
    a = dy * w
    dz = rstd * (a - xh * (a * xh).mean(-1, keepdim=True))
    if st["residual"] is not None:
        dz = dz + st["residual"].float()
    return [dz.to(torch.bfloat16), (dy * xh).sum((0, 1)), dgate]


def _padded(st, wide):
    """Index of each document's tokens, padded to a multiple of 16 (`wide`
    of them), and which of them are tokens."""
    cu = st["cu"].long()
    at = torch.arange(wide, device="cuda")
    ok = at < (cu[1:] - cu[:-1])[:, None]
    idx = torch.where(ok, cu[:-1, None] + at, 0)
    return idx, ok


def _gate(st, f64=True):
    """Log-decay [T, H, 128 or 1], its derivative by the gate input and by
    A_log, in 64 bits (the clamp is a border)."""
    H, gate = st["case"]["H"], st["case"]["gate"]
    g = st["g"].double().reshape(-1, H, st["g"].shape[1] // H)
    if gate & GATE_PRECOMPUTED:
        inside = (g >= LOWER_BOUND) & (g <= 0.0)
        return g.clamp(LOWER_BOUND, 0.0), inside.double(), None
    x = g + st["dt_bias"].double().reshape(H, -1)
    ea = torch.exp(st["A_log"].double())[:, None]
    sp = torch.where(x > 20.0, x, torch.log1p(torch.exp(x)))
    gu = -ea * sp
    inside = gu >= LOWER_BOUND
    return torch.where(inside, gu, LOWER_BOUND), inside * (-ea * torch.sigmoid(x)), inside * gu


def _plain_backward(st):
    """Chunks of 16 tokens: everything inside a chunk for all chunks at once,
    the states and their gradients from chunk to chunk."""
    case, C = st["case"], 16
    H, gate, sc = case["H"], case["gate"], st["scale"]
    lens = _docs(case)
    wide = -(-max(max(lens), 1) // C) * C
    idx, ok = _padded(st, wide)
    n, N = len(lens), wide // C

    def rows(x):  # [T, H, w] -> [chains, N, C, w], padding zeroed
        p = x[idx] * ok[..., None, None]
        return p.permute(0, 2, 1, 3).reshape(n * H, N, C, x.shape[-1])

    def tokens(x, like):  # back to the packed tokens, in the inputs' type
        p = x.reshape(n, H, wide, -1).permute(0, 2, 1, 3)[ok]
        return p.reshape(like.shape).to(like.dtype)

    def heads(x):
        return x.float().reshape(x.shape[0], H, -1)

    q, k = rows(heads(st["q"])), rows(heads(st["k"]))
    v, do = rows(heads(st["v"])), rows(heads(st["do"]))
    rq = torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS)
    rk = torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS)
    qh, kh = q * rq, k * rk
    bl = heads(st["beta"])
    beta = rows(bl if gate & BETA_PRESIGMOID else torch.sigmoid(bl))
    gl, dgx, dga = _gate(st)
    G = rows(gl.expand(-1, H, D)).cumsum(2)
    Gl = G[:, :, -1:]
    kin, kout = kh * torch.exp(G).float(), kh * torch.exp(Gl - G).float()
    qin, eg = qh * torch.exp(G).float(), torch.exp(Gl).float().transpose(2, 3)
    up, down = torch.exp(G - 0.5 * Gl).float(), torch.exp(0.5 * Gl - G).float()
    qp, kp, km = qh * up, kh * up, kh * down
    A = (kp @ km.transpose(2, 3)).tril(-1)
    P = (qp @ km.transpose(2, 3)).tril() * sc
    # (1 + beta A)^-1: A's 16th power is zero
    X = -beta * A
    eye = torch.eye(C, device="cuda")
    X2 = X @ X
    X4 = X2 @ X2
    inv = (eye + X) @ (eye + X2) @ (eye + X4) @ (eye + X4 @ X4)
    Tb = inv * beta.transpose(2, 3)
    Wk, U0 = Tb @ kin, Tb @ v
    TbT = Tb.transpose(2, 3)
    Z, dV0 = TbT @ kout, TbT @ (P.transpose(2, 3) @ do)

    S = torch.zeros(n * H, D, D, device="cuda")
    if st["use_initial"]:  # pool slots hold [value][key]
        S = st["pool"][st["slots"].long()].float().reshape(n * H, D, D).transpose(1, 2)
    Ss = torch.empty(n * H, N, D, D, device="cuda")
    U = torch.empty_like(U0)
    for i in range(N):
        Ss[:, i] = S
        U[:, i] = U0[:, i] - Wk[:, i] @ S
        S = eg[:, i] * S + kout[:, i].transpose(1, 2) @ U[:, i]

    dS = torch.zeros(n * H, D, D, device="cuda")
    if st["dstate"] is not None:
        dS = st["dstate"].reshape(n * H, D, D).transpose(1, 2)
    dSs = torch.empty_like(Ss)
    dV = torch.empty_like(U0)
    for i in reversed(range(N)):
        dSs[:, i] = dS
        dV[:, i] = dV0[:, i] + Z[:, i] @ dS
        dS = eg[:, i] * dS + sc * (qin[:, i].transpose(1, 2) @ do[:, i]) \
            - kin[:, i].transpose(1, 2) @ dV[:, i]

    StT, dStT = Ss.transpose(2, 3), dSs.transpose(2, 3)
    dP = (do @ U.transpose(2, 3)).tril() * sc
    dA = -(dV @ U.transpose(2, 3)).tril(-1)
    dqh = (sc * (do @ StT) * torch.exp(G).float()) + (dP @ km) * up
    drow = -(dV @ StT) * torch.exp(G).float() + (dA @ km) * up
    dcol = (dA.transpose(2, 3) @ kp + dP.transpose(2, 3) @ qp) * down
    dend = (U @ dStT) * torch.exp(Gl - G).float()
    dkh = drow + dcol + dend
    dG = qh * dqh + kh * (drow - dcol - dend)
    last = (eg * (Ss * dSs).sum(3, keepdim=True)).transpose(2, 3) \
        + (kh * dend).sum(2, keepdim=True)
    dg = dG.double().flip(2).cumsum(2).flip(2) + last.double()
    dq = rq * (dqh - qh * (qh * dqh).sum(-1, keepdim=True))
    dk = rk * (dkh - kh * (kh * dkh).sum(-1, keepdim=True))
    # dV = beta dR and U = beta (v - ...): with x = v - (decayed state) k
    x = v - kin @ Ss - A @ U
    dR = inv.transpose(2, 3) @ (P.transpose(2, 3) @ do + kout @ dSs)
    dbeta = (dR * x).sum(-1, keepdim=True)
    if not gate & BETA_PRESIGMOID:
        dbeta = dbeta * beta * (1.0 - beta)
    if gate & GATE_PER_HEAD:
        dg = dg.sum(-1, keepdim=True)
    dgraw = dg * rows(dgx)
    out = [tokens(dq, st["q"]), tokens(dk, st["k"]), tokens(dV, st["v"]),
           tokens(dgraw, st["g"]), tokens(dbeta, st["beta"]), None, None, None]
    if dga is not None:
        out[5] = (dg * rows(dga)).reshape(n, H, -1).sum((0, 2)).float()
        out[6] = dgraw.reshape(n, H, wide, -1).sum((0, 2)).reshape(-1).float()
    if st["use_initial"]:
        out[7] = dS.transpose(1, 2).reshape(n, H, D, D)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    if case["op"] != "bwd":
        n = case["rows"] * case["heads"] * case["width"]
        if case["op"] == "norm":
            per = 2 + (4 if case["residual"] else 0) + (2 if case["gated"] else 0) \
                + (2 if case["out"] == "bf16" else 1)
            sc = 0
            if case["out"] == "fp8":
                sc = 4 * n // (case["group"] or case["width"])
            return dict(bytes=n * per + sc + 4 * case["width"], flops=6 * n)
        per = 6 + (2 if case["residual"] else 0) + (4 if case["gated"] else 0)
        return dict(bytes=n * per + 8 * case["width"], flops=12 * n)
    lens, H = _docs(case), case["H"]
    T = sum(lens)
    gw = 2 if case["gate"] & GATE_PER_HEAD else 2 * D
    state = dict(none=0, bf16=2, fp16=2, fp8=1)[case["state"]]
    per_state = state + (4 if state else 0) + (4 if case["dfinal"] else 0)
    nbytes = T * H * (4 * 2 * D + gw + 2 + 3 * 2 * D + gw + 2) + len(lens) * H * D * D * per_state
    # per token and head: 5 D^2 to step the state, 15 D^2 for its adjoint and
    # the gradients (seven products of a D x D matrix and a vector, one decay)
    return dict(bytes=nbytes, flops=20 * D * D * T * H)


# ---------------------------------------------------------------------------
# definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "bwd":
        return _exact_backward(st)
    x, w = st["x"].double(), st["weight"].double()
    ms = x.pow(2).mean(-1, keepdim=True) if case["op"] == "norm_bwd" else None
    if case["op"] == "norm":
        if case["residual"]:
            x = x + st["residual"].double()
        y = w * x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
        if case["gated"]:
            y = y / (1.0 + torch.exp(-st["gate"].double()))
        zr = x if case["residual"] else None
        if case["out"] == "bf16":
            return [y, None, zr]
        yg = y.reshape(case["rows"], -1, case["group"] or case["width"])
        s = yg.abs().amax(-1) / FP8_MAX
        s = torch.where(s == 0, torch.ones_like(s), s)
        return [(yg / s[..., None]).reshape(y.shape), s, zr]
    r = torch.sqrt(ms + EPS)
    dy, n = st["dy"].double(), case["width"]
    sig = 1.0 / (1.0 + torch.exp(-st["gate"].double())) if case["gated"] else 1.0
    up = dy * sig * w
    dz = up / r - x * (up * x).sum(-1, keepdim=True) / (n * r.pow(3))
    if case["residual"]:
        dz = dz + st["residual"].double()
    dgate = dy * w * (x / r) * sig * (1.0 - sig) if case["gated"] else None
    return [dz, (dy * sig * x / r).reshape(-1, n).sum(0), dgate]


def _exact_backward(st):
    """The recurrence and its adjoint token by token; states are kept every 64
    tokens and recomputed in between."""
    case, K = st["case"], 64
    H, gate, sc = case["H"], case["gate"], st["scale"]
    lens = _docs(case)
    n, Tm = len(lens), max(max(lens), 1)
    cu = st["cu_host"].tolist()
    f64 = torch.float64

    def chains(x):  # [T, H, w] -> [Tm, chains, w]
        p = torch.zeros(Tm, n, H, x.shape[-1], dtype=f64, device="cuda")
        for d in range(n):
            p[:lens[d], d] = x[cu[d]:cu[d + 1]]
        return p.reshape(Tm, n * H, -1)

    def split(name):
        return st[name].double().reshape(-1, H, st[name].shape[1] // H)

    q, k, v, do = (chains(split(s)) for s in ("q", "k", "v", "do"))
    nq = torch.sqrt(q.pow(2).sum(-1, keepdim=True) + EPS)
    nk = torch.sqrt(k.pow(2).sum(-1, keepdim=True) + EPS)
    q, k = q / nq, k / nk
    b = split("beta")
    b = chains(b if gate & BETA_PRESIGMOID else 1.0 / (1.0 + torch.exp(-b)))
    gx = split("g")
    if gate & GATE_PRECOMPUTED:
        g, slope, by_a = gx.clamp(LOWER_BOUND, 0), ((gx >= LOWER_BOUND) & (gx <= 0)).double(), None
    else:
        x = gx + st["dt_bias"].double().reshape(H, -1)
        ea = st["A_log"].double().exp().reshape(H, 1)
        raw = -ea * torch.log1p(torch.exp(x))
        keep = (raw >= LOWER_BOUND).double()
        g, slope, by_a = raw.clamp(min=LOWER_BOUND), -keep * ea / (1 + torch.exp(-x)), keep * raw
    a = torch.exp(chains(g.expand(-1, H, D)))
    pad = torch.arange(Tm, device="cuda")[:, None] >= torch.tensor(lens, device="cuda")
    a[pad.repeat_interleave(H, 1)] = 1.0

    S = torch.zeros(n * H, D, D, dtype=f64, device="cuda")  # [value][key]
    if st["use_initial"]:
        S = st["pool"].double()[st["slots"].long()].reshape(n * H, D, D)

    def step(S, t):
        Sd = S * a[t][:, None]
        x = v[t] - torch.bmm(Sd, k[t][:, :, None])[..., 0]
        u = b[t] * x
        return Sd, x, u, torch.baddbmm(Sd, u[:, :, None], k[t][:, None])

    kept = []
    for t in range(Tm):
        if t % K == 0:
            kept.append(S)
        S = step(S, t)[3]
    dS = torch.zeros_like(S)
    if st["dstate"] is not None:
        dS = st["dstate"].double().reshape(n * H, D, D)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dg, db = torch.empty_like(q), torch.empty_like(b)
    for c in reversed(range(len(kept))):
        S, seg = kept[c], []
        for t in range(c * K, min(Tm, (c + 1) * K)):
            parts = step(S, t)
            seg.append((S, parts[0], parts[1], parts[2], parts[3]))
            S = parts[3]
        for t in reversed(range(c * K, min(Tm, (c + 1) * K))):
            S0, Sd, x, u, S1 = seg[t - c * K]
            dq[t] = sc * torch.bmm(do[t][:, None], S1)[:, 0]
            dS = torch.baddbmm(dS, do[t][:, :, None], sc * q[t][:, None])
            du = torch.bmm(dS, k[t][:, :, None])[..., 0]
            db[t] = (du * x).sum(-1, keepdim=True)
            dx = b[t] * du
            dv[t] = dx
            dk[t] = torch.bmm(u[:, None], dS)[:, 0] - torch.bmm(dx[:, None], Sd)[:, 0]
            dS = torch.baddbmm(dS, dx[:, :, None], -k[t][:, None])
            dg[t] = (dS * Sd).sum(1)
            dS = dS * a[t][:, None]

    def packed(x):
        x = x.reshape(Tm, n, H, -1)
        return torch.cat([x[:lens[d], d] for d in range(n)])

    dq = (dq - q * (q * dq).sum(-1, keepdim=True)) / nq
    dk = (dk - k * (k * dk).sum(-1, keepdim=True)) / nk
    if not gate & BETA_PRESIGMOID:
        db = db * b * (1 - b)
    dg = packed(dg)
    if gate & GATE_PER_HEAD:
        dg = dg.sum(-1, keepdim=True)
    T = dg.shape[0]
    out = [packed(dq).reshape(T, -1), packed(dk).reshape(T, -1), packed(dv).reshape(T, -1),
           (dg * slope).reshape(T, -1), packed(db).reshape(T, -1), None, None, None]
    if by_a is not None:
        out[5] = (dg * by_a).sum((0, 2))
        out[6] = (dg * slope).sum(0).reshape(-1)
    if st["use_initial"]:
        out[7] = dS.reshape(n, H, D, D)
    return out
