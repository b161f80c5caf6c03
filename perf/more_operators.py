"""Workloads of the paged 8-bit key/value cache and the attention that reads it.

Four calls of one cache, as a server calls them in the attention layers that
stand between recurrent ones:

  write   quantises the keys and values of new tokens into their pages, one
          scale per page and head
  read    gives tokens back in bf16
  attend  attention of one or a few new tokens of each sequence
  doc     attention of packed documents, from the start or over earlier tokens

`own` selects the library's calls (True) or the plain form in elementary
torch operations (False). `exact` follows the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128
SCALE = D ** -0.5
MIX14 = "4096,3000,2048,1500,1200,1024,1000,700,600,500,300,217,128,71"
MIN_EXP = -100  # smallest exponent of a scale


# ---------------------------------------------------------------------------
# cases
#
# H: key/value heads; G: query heads of each; page: tokens of a page; kind: the
# cache's 8-bit type. New tokens: "docs" (one count for each sequence), or n
# sequences of T tokens. Earlier tokens: spread from lo to hi over their
# logarithm (lo = hi = 0: none), by the number "mix".

def listed():
    return [
        # a decode step of a small batch writes its token
        dict(name="write_step", op="write", kind="e4m3", H=8, page=64, n=32, T=1, lo=1, hi=4000,
             mix=1),
        # draft tokens of a large batch, small pages, one key/value head per query head
        dict(name="write_draft", op="write", kind="int8", H=12, page=16, n=512, T=8, lo=30,
             hi=1500, mix=2),
        # the repository's 14-document mix of 16384 tokens, as a prefill leaves them
        dict(name="write_mix14", op="write", kind="e4m3", H=8, page=64, docs=MIX14, lo=0, hi=0,
             mix=3),
        # one short sequence handed to another device
        dict(name="read_short", op="read", kind="int8", H=12, page=16, docs="217", lo=0, hi=0,
             mix=4),
        # the 14 documents read back as the prefix of a training or scoring pass
        dict(name="read_mix14", op="read", kind="e4m3", H=8, page=128, docs=MIX14, lo=0, hi=0,
             mix=5),
        # one user's token, a short chat
        dict(name="attend_one", op="attend", kind="e4m3", H=12, G=1, page=16, n=1, T=1, lo=500,
             hi=500, mix=6),
        # a decode batch of ragged chats, 64 query heads on 8
        dict(name="attend_batch", op="attend", kind="e4m3", H=8, G=8, page=64, n=128, T=1, lo=500,
             hi=8190, mix=7),
        # a large batch of short chats, 12 heads of their own keys, int8
        dict(name="attend_heads", op="attend", kind="int8", H=12, G=1, page=16, n=512, T=1, lo=71,
             hi=1500, mix=8),
        # one long document
        dict(name="attend_long", op="attend", kind="e4m3", H=8, G=8, page=256, n=1, T=1,
             lo=131070, hi=131070, mix=9),
        # eight draft tokens of each sequence are verified
        dict(name="attend_draft", op="attend", kind="e4m3", H=8, G=8, page=64, n=64, T=8, lo=300,
             hi=4000, mix=10),
        # the 14 documents from their start, 12 query heads on 4
        dict(name="doc_mix14", op="doc", kind="int8", H=4, G=3, page=64, docs=MIX14, lo=0, hi=0,
             mix=11),
        # one prompt's chunks beside another's first one, over a long cache, 64 heads on 8
        dict(name="doc_chunk", op="doc", kind="e4m3", H=8, G=8, page=64, docs="4096,1777", lo=2000,
             hi=12000, mix=12),
    ]


def _loguni(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "doc", "doc"])
    case = dict(op=op, kind=rng.choice(["e4m3", "int8"]), H=rng.choice([1, 2, 4, 5, 8, 12, 16]),
                page=rng.choice([16, 32, 64, 128, 256]), mix=rng.randrange(1 << 30))
    if op in ("attend", "doc"):
        case["G"] = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
    if op == "attend" or (op == "write" and rng.random() < 0.5):
        case.update(n=_loguni(rng, 1, 512), T=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]))
        top = 8000000 // (case["n"] * case["H"])
        case["hi"] = _loguni(rng, 1, max(1, min(131000, top)))
        case["lo"] = _loguni(rng, 1, case["hi"])
        return case
    n = rng.randint(1, 14)
    lens = [_loguni(rng, 1, 8000) for _ in range(n)]
    if rng.random() < 0.25:
        lens[rng.randrange(n)] = 0
    past = rng.choice([0, _loguni(rng, 1, 12000)])
    case["hi"] = past
    case["lo"] = _loguni(rng, 1, past) if past else 0
    G = case.get("G", 1)
    while sum(lens) * case["H"] > 260000 or \
            (op == "doc" and n * max(lens) * (max(lens) + past) * G * case["H"] > 4000000000):
        lens = [x * 2 // 3 for x in lens]
    if sum(lens) == 0:
        lens[0] = 1
    case["docs"] = ",".join(str(x) for x in lens)
    return case


def _lens(case):
    """New tokens of each sequence, and its length with them."""
    new = [int(x) for x in case["docs"].split(",")] if "docs" in case else [case["T"]] * case["n"]
    r = random.Random(case["mix"])
    past = [_loguni(r, case["lo"], case["hi"]) if case["hi"] else 0 for _ in new]
    return new, [a + b for a, b in zip(new, past)]


# ---------------------------------------------------------------------------
# inputs

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _most(kind):
    return 448.0 if kind == "e4m3" else 127.0


def _pages(gen, case, pages):
    """A cache of `pages` pages as writing ordinary keys or values leaves it: the
    heads differ in size, a page's scale is the power of two that its largest
    value needs."""
    H, P, kind = case["H"], case["page"], case["kind"]
    x = _rand(gen, pages, H, P, D) * (0.5 + torch.rand(1, H, 1, 1, generator=gen, device="cuda"))
    top = x.abs().amax((2, 3))
    scale = torch.exp2(torch.ceil(torch.log2(top / _most(kind))))
    x = x / scale[:, :, None, None]
    if kind == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale
    return x.round().clamp(-127.0, 127.0).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    new, total = _lens(case)
    H, P = case["H"], case["page"]
    n, T = len(new), sum(new)
    width = max(1, -(-max(total) // P))
    used = [-(-x // P) for x in total]
    pages = sum(used) + 2  # the pool holds others too
    st = dict(case=case, width=width)
    st["k_cache"], st["k_scale"] = _pages(gen, case, pages)
    st["v_cache"], st["v_scale"] = _pages(gen, case, pages)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    live = torch.arange(width, device="cuda") < torch.tensor(used, device="cuda")[:, None]
    st["page_table"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    st["page_table"][live] = order[:sum(used)]
    st["kv_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    st["cu_host"] = torch.tensor(cu, dtype=torch.int32) if "docs" in case else None
    st["cu"] = st["cu_host"].cuda() if "docs" in case else None
    bf = torch.bfloat16
    if case["op"] in ("write", "read"):
        for name in ("k", "v"):
            st[name] = (2.0 * _rand(gen, T, H * D)).to(bf)
    else:
        st["q"] = _rand(gen, T, H * case["G"] * D).to(bf)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(T, H * case["G"], device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass

def _run_own(st):
    import gated_delta_rule_step_amd as kda
    case = st["case"]
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["page_table"],
             st["kv_lens"])
    if case["op"] == "write":
        kda.kda_cache_write(st["k"], st["v"], *cache, cu_seqlens=st["cu"])
        return list(cache[:4])
    if case["op"] == "read":
        kda.kda_cache_read(st["k"], st["v"], *cache, cu_seqlens=st["cu"])
        return [st["k"], st["v"]]
    if st.get("workspace") is None:  # kept beside the plan, as a server keeps it
        need = kda.kda_cache_attention_workspace_size(
            st["kv_lens"].shape[0], st["q"].shape[0], case["H"] * case["G"], case["H"])
        st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    kda.kda_cache_attention(st["q"], st["out"], *cache, cu_seqlens_host=st["cu_host"],
                            cu_seqlens=st["cu"], lse=st["lse"], scale=SCALE,
                            workspace=st["workspace"])
    return [st["out"], st["lse"]]


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    return _plain_write(st) if op == "write" else \
        _plain_read(st) if op == "read" else _plain_attention(st)


# ---------------------------------------------------------------------------
# plain forms

def _counts(st):
    """New tokens of each sequence."""
    if st["cu"] is None:
        return torch.full_like(st["kv_lens"], st["case"]["T"]).long()
    return (st["cu"][1:] - st["cu"][:-1]).long()


def _places(st, T):
    """Page, slot and sequence of each packed token."""
    n = _counts(st)
    b = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=T)
    first = n.cumsum(0) - n
    pos = st["kv_lens"].long()[b] - n[b] + torch.arange(T, device="cuda") - first[b]
    P = st["case"]["page"]
    return st["page_table"][b, pos // P].long(), pos % P


def _exponent(top, kind):
    """The smallest e >= MIN_EXP with top <= most * 2^e."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8) if kind == "e4m3" else \
        torch.where(m <= 0.9921875, e - 7, e - 6)
    return torch.where(top > 0, e, MIN_EXP).clamp(min=MIN_EXP)


def _encode(x, kind):
    if kind == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return x.round().clamp(-127.0, 127.0).to(torch.int8)


def _bytes(x):
    """For indexing, which some 8-bit types lack."""
    return x.view(torch.uint8)


def _plain_write(st):
    case = st["case"]
    H, P, kind = case["H"], case["page"], case["kind"]
    T = st["k"].shape[0]
    page, slot = _places(st, T)
    n, table = _counts(st), st["page_table"]
    start = st["kv_lens"].long() - n
    # the page that a sequence's first new token falls into may hold earlier ones
    first = table.gather(1, (start // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    keeps = (start % P > 0) & (n > 0)
    first = torch.where(keeps, first, 0)
    for name in ("k", "v"):
        x = st[name].float().reshape(T, H, D)
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        top = torch.zeros_like(scale).scatter_reduce(
            0, page[:, None].expand(T, H), x.abs().amax(-1), "amax")
        touched = torch.zeros(scale.shape[0], device="cuda").index_fill(0, page, 1.0) > 0
        need = torch.exp2(_exponent(top, kind).float())
        held = torch.zeros(scale.shape[0], device="cuda").index_add(0, first, keeps.float()) > 0
        now = torch.where(held[:, None], torch.maximum(need, scale), need)
        now = torch.where(touched[:, None], now, scale)
        old = _bytes(cache)[first]
        ratio = (scale / now)[first][:, :, None, None]
        again = _bytes(_encode(old.view(cache.dtype).float() * ratio, kind))
        earlier = (torch.arange(P, device="cuda") < (start % P)[:, None]) & keeps[:, None]
        which = earlier.nonzero()
        _bytes(cache)[first[which[:, 0]], :, which[:, 1]] = again[which[:, 0], :, which[:, 1]]
        _bytes(cache)[page, :, slot] = _bytes(_encode(x / now[page][..., None], kind))
        scale.copy_(now)
    return [st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]]


def _plain_read(st):
    T = st["k"].shape[0]
    page, slot = _places(st, T)
    got = []
    for name in ("k", "v"):
        cache = st[name + "_cache"]
        x = _bytes(cache)[page, :, slot].view(cache.dtype).float()
        x = x * st[name + "_scale"][page][..., None]
        got.append(x.reshape(T, -1).to(torch.bfloat16))
    return got


def _plain_attention(st):
    case = st["case"]
    H, G, P, W = case["H"], case["G"], case["page"], st["width"]
    n, lens = _counts(st), st["kv_lens"].long()
    B, T = n.numel(), st["q"].shape[0]
    wide = case["T"] if "T" in case else max(int(x) for x in case["docs"].split(","))
    at = torch.arange(wide, device="cuda")
    real = at < n[:, None]
    idx = torch.where(real, (n.cumsum(0) - n)[:, None] + at, 0)

    def keys(name):  # [B, H, W * P, 128]
        page = st["page_table"].clamp(min=0).long()
        cache = st[name + "_cache"]
        x = _bytes(cache)[page].view(cache.dtype).float()
        x = x * st[name + "_scale"][page][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, W * P, D)

    q = st["q"].float().reshape(T, H, G, D)[idx]  # [B, wide, H, G, 128]
    q = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * wide, D)
    s = (q * SCALE) @ keys("k").transpose(2, 3)
    last = (lens - n)[:, None] + at  # the last key that a token sees
    hidden = torch.arange(W * P, device="cuda") > last[..., None]
    s = s.reshape(B, H, G, wide, W * P).masked_fill_(hidden[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top).exp_()
    total = p.sum(-1, keepdim=True)
    seen = hidden.logical_not()[:, :wide].any(1)[:, None, :, None]  # stale pages may hold anything
    v = torch.where(seen, keys("v"), 0.0)
    o = (p.reshape(B, H, G * wide, W * P) @ v).reshape(B, H, G, wide, D) / total
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4)[real].reshape(T, H * G * D)
    return [o.to(torch.bfloat16), lse.permute(0, 3, 1, 2)[real].reshape(T, H * G)]


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    new, total = _lens(case)
    H, T, P = case["H"], sum(new), case["page"]
    values = 2 * T * H * D
    if case["op"] in ("write", "read"):
        pages = sum(-(-b // P) - (b - a) // P for a, b in zip(new, total) if a)
        # an 8-bit and a 16-bit side, a scale for each page that is touched, and the tables
        return dict(bytes=3 * values + 4 * pages * (2 * H + 1) + 4 * len(new), flops=2 * values)
    heads = H * case["G"]
    pages = sum(-(-b // P) for b in total)
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(new, total))
    return dict(bytes=2 * H * D * sum(total) + 4 * pages * (2 * H + 1) + T * heads * (4 * D + 4),
                flops=4 * D * heads * pairs)


# ---------------------------------------------------------------------------
# definitions in 64 bits

def _value(codes, kind):
    """What 8-bit codes stand for, from their bits."""
    if kind == "int8":
        return codes.double()
    b = codes.view(torch.uint8).to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e > 0, (1.0 + m / 8) * torch.exp2((e - 7).double()), m / 512)
    x = torch.where((e == 15) & (m == 7), math.nan, x)
    return torch.where(b >= 128, -x, x)


def _nearest(x, kind):
    """The 8-bit format's value next to x; ties go to the even code."""
    if kind == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_write(st):
    case, out = st["case"], []
    H, P, kind = case["H"], case["page"], case["kind"]
    new, total = _lens(case)
    table = st["page_table"].tolist()
    scales = []
    for name in ("k", "v"):
        codes = _value(st[name + "_cache"], kind)
        scale = st[name + "_scale"].double()
        x, at = st[name].double().reshape(-1, H, D), 0
        for b, (n, end) in enumerate(zip(new, total)):
            pos = end - n
            while pos < end:
                page, a = table[b][pos // P], pos % P
                z = min(P, a + end - pos)
                rows = x[at:at + z - a].transpose(0, 1)  # [H, tokens, 128]
                need = torch.log2(rows.abs().amax((1, 2)) / _most(kind)).ceil()
                need = torch.exp2(need.clamp(min=MIN_EXP))
                if a:
                    need = torch.maximum(need, scale[page])
                    codes[page, :, :a] = _nearest(
                        codes[page, :, :a] * (scale[page] / need)[:, None, None], kind)
                codes[page, :, a:z] = _nearest(rows / need[:, None, None], kind)
                scale[page] = need
                at, pos = at + z - a, pos + z - a
        out.append(codes if kind == "e4m3" else codes.to(torch.int8))
        scales.append(scale)
    return out + scales


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(st)
    H, P, kind = case["H"], case["page"], case["kind"]
    new, total = _lens(case)

    def tokens(name, b):  # [H, total, 128]
        page = st["page_table"][b, :-(-total[b] // P)].long()
        x = _value(st[name + "_cache"].view(torch.uint8)[page].view(st[name + "_cache"].dtype), kind)
        x = x * st[name + "_scale"].double()[page][..., None, None]
        return x.transpose(0, 1).reshape(H, -1, D)[:, :total[b]]

    if case["op"] == "read":
        got = []
        for name in ("k", "v"):
            parts = [tokens(name, b)[:, total[b] - n:].transpose(0, 1) for b, n in enumerate(new) if n]
            got.append(torch.cat(parts).reshape(-1, H * D))
        return got
    G, out, lses, at = case["G"], [], [], 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        q = st["q"][at:at + n].double().reshape(n, H, G, D)
        at += n
        k, v, o, ls = tokens("k", b), tokens("v", b), [], []
        far = torch.arange(total[b], device="cuda") > \
            torch.arange(total[b] - n, total[b], device="cuda")[:, None]
        for h in range(H):
            for g in range(G):
                s = (SCALE * (q[:, h, g] @ k[h].T)).masked_fill_(far, -math.inf)
                ls.append(torch.logsumexp(s, -1))
                o.append(torch.exp(s - ls[-1][:, None]) @ v[h])
        out.append(torch.stack(o, 1).reshape(n, -1))
        lses.append(torch.stack(ls, 1))
    return [torch.cat(out), torch.cat(lses)]
