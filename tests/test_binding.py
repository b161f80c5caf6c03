"""The Python binding's own work around the C calls: where a workspace comes from, and
which one it takes.

On the CPU the library, the allocator and the streams are stand-ins that note what they
are asked for; the GPU tests run the real ones.
"""
from __future__ import annotations

import contextlib

import pytest
import torch

import gated_delta_rule_step_amd as kda

BF, D = torch.bfloat16, 128


class Gpu:
    """A CPU tensor that says it lives on cuda:0."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return Gpu(self.t[i])

    def get_device(self):
        return 0


class Stream:
    def __init__(self, handle, device=torch.device("cuda", 0)):
        self.cuda_stream, self.device = handle, device


class Calls:
    """Stands for the library: every call succeeds, and is noted as (name, last argument:
    the stream, workspace address)."""

    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size"):
                return 512
            raw = args[-1]
            self.seen.append((name, int(getattr(raw, "value", raw) or 0),
                              int(getattr(args[-3], "value", args[-3]) or 0)))
            return 0
        return call


class Holder:
    """Another library's stream object."""
    cuda_stream = 0x400


CURRENT = 0x100


@pytest.fixture
def fake(monkeypatch):
    """(library, list of (stream handle, address) of every allocation)."""
    lib, at, made, empty = Calls(), [Stream(CURRENT)], [], torch.empty

    @contextlib.contextmanager
    def use(stream):
        at.append(stream)
        yield
        at.pop()

    def alloc(n, dtype, device):
        t = Gpu(empty(n, dtype=dtype))
        made.append((at[-1].cuda_stream, t.data_ptr()))
        keep.append(t)
        return t

    keep = []
    monkeypatch.setattr(kda, "lib", lambda: lib)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: at[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: Stream(handle, device))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: at[-1].cuda_stream,
                        raising=False)
    monkeypatch.setattr(torch, "empty", alloc)
    return lib, made


def inputs(T=20, H=2):
    """Arguments of the three calls that may allocate, by name."""
    W = H * D

    def z(*shape, dtype=BF):
        return torch.zeros(*shape, dtype=dtype)

    f = torch.float32
    seq = dict(cu=torch.tensor([0, 13, T], dtype=torch.int32), q=z(T, W), b=z(T, H),
               A=z(H, dtype=f), dt=z(W, dtype=f), pool=z(2, H, D, D),
               idx=torch.tensor([0, 1], dtype=torch.int32))
    return seq, dict(z=z(5, 300), w=z(300, dtype=f), dw=z(300, dtype=f))


def call(name, on, **kw):
    """One call of `name`, its GPU tensors made by `on`."""
    seq, norm = inputs()
    cu, q, b, A, dt, pool, idx = (seq[n] if n == "cu" else on(seq[n]) for n in
                                  ("cu", "q", "b", "A", "dt", "pool", "idx"))
    if name == "kda_prefill_varlen":
        kda.kda_prefill_varlen(cu, on(cu), q, q, q, q, b, A, dt, pool, idx, on(seq["q"]), **kw)
    elif name == "kda_prefill_varlen_backward":
        out = [on(seq["q"].clone()) for _ in range(4)] + [on(seq["b"].clone())]
        kda.kda_prefill_varlen_backward(cu, on(cu), q, q, q, q, b, A, dt, pool, idx, q, *out, **kw)
    else:
        kda.kda_rmsnorm_backward(on(norm["z"]), on(norm["w"]), on(norm["z"]), on(norm["z"].clone()),
                                 on(norm["dw"]), **kw)


NAMES = ["kda_prefill_varlen", "kda_prefill_varlen_backward", "kda_rmsnorm_backward"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream,want", [(None, CURRENT), (Stream(0x200), 0x200), (0x300, 0x300),
                                         (Stream(CURRENT), CURRENT), (Holder(), 0x400)],
                         ids=["current", "stream", "handle", "same", "holder"])
def test_workspace_belongs_to_the_launch_stream(fake, name, stream, want):
    """A workspace that the binding makes comes from the pool of the stream that the
    kernels run on: from another one it could be handed out again while they use it."""
    lib, made = fake
    call(name, Gpu, stream=stream)
    assert len(made) == 1 and made[0][0] == want
    assert lib.seen == [(name, want, made[0][1])]


@pytest.mark.parametrize("name", NAMES)
def test_workspace_of_another_device_stream(fake, name):
    lib, made = fake
    with pytest.raises(ValueError, match="stream"):
        call(name, Gpu, stream=Stream(0x200, torch.device("cuda", 1)))
    assert not lib.seen and not made


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("bad", [
    Gpu(torch.zeros(1, dtype=torch.uint8).expand(1 << 20)),       # one byte
    Gpu(torch.zeros(1 << 12, dtype=torch.uint8)[::2]),
    torch.zeros(1 << 12, dtype=torch.uint8)], ids=["expanded", "every other byte", "on the CPU"])
def test_workspace_refused(fake, name, bad):
    """Memory that holds fewer bytes than its elements would take, or that the kernels
    cannot reach."""
    lib, _ = fake
    with pytest.raises(ValueError, match="workspace"):
        call(name, Gpu, workspace=bad)
    assert not lib.seen


@pytest.mark.parametrize("name", NAMES)
def test_workspace_of_the_caller(fake, name):
    lib, made = fake
    ws = Gpu(torch.zeros(8, 512, dtype=torch.float32))
    call(name, Gpu, workspace=ws)
    assert lib.seen == [(name, CURRENT, ws.data_ptr())] and not made


# ---------------------------------------------------------------------------
# GPU

def _training_step(stream, T=700, H=4):
    """Prefill, its gradients and a norm's, all without a workspace of the caller's."""
    g = torch.Generator().manual_seed(1)
    W = H * D

    def rnd(*shape, dtype=BF):
        return torch.randn(*shape, generator=g).to(dtype).cuda()

    cu = torch.tensor([0, 300, T], dtype=torch.int32)
    cud, idx = cu.cuda(), torch.tensor([1, 0], dtype=torch.int32).cuda()
    q, k, v, gate, do = (rnd(T, W) for _ in range(5))
    b, A, dt = rnd(T, H), rnd(H, dtype=torch.float32), 0.1 * rnd(W, dtype=torch.float32)
    pool, wt = 0.1 * rnd(2, H, D, D), rnd(W, dtype=torch.float32)
    out = torch.empty_like(q)
    grads = [torch.empty_like(t) for t in (q, k, v, gate, b, A, dt)]
    dz, dw = torch.empty_like(q), torch.empty_like(wt)
    torch.cuda.synchronize()

    def step():
        keep = pool.clone()
        torch.cuda.synchronize()
        kda.kda_prefill_varlen(cu, cud, q, k, v, gate, b, A, dt, keep, idx, out, stream=stream)
        kda.kda_prefill_varlen_backward(cu, cud, q, k, v, gate, b, A, dt, pool, idx, do,
                                        *grads[:5], dA_log=grads[5], ddt_bias=grads[6],
                                        stream=stream)
        kda.kda_rmsnorm_backward(out, wt, do, dz, dw, stream=stream)
        return [out, keep, *grads, dz, dw]
    return step


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["stream", "handle", "holder"])
def test_own_workspace_on_a_side_stream(form):
    """Calls on a side stream next to allocations and fills of the current stream: the bits
    of the calls alone."""
    want = [t.clone() for t in _training_step(None)()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    holder = Holder()
    holder.cuda_stream = side.cuda_stream
    step = _training_step(dict(stream=side, handle=side.cuda_stream, holder=holder)[form])
    need = kda.kda_prefill_backward_workspace_size(2, 700, 4)
    for _ in range(5):
        got = step()
        for n in (need, need // 2, 8192):  # takes and overwrites what is free here
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_own_workspace_on_the_default_stream_handle():
    """Handle 0 is the device's default stream."""
    want = [t.clone() for t in _training_step(None)()]
    got = _training_step(0)()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_own_workspace_in_a_captured_call():
    """The capturing stream given by name: the workspace comes from the graph's memory, and the
    replays give the bits of the calls alone, with other work between them."""
    want = [t.clone() for t in _training_step(None)()]
    g = torch.Generator().manual_seed(1)
    T, H = 700, 4
    W = H * D

    def rnd(*shape, dtype=BF):
        return torch.randn(*shape, generator=g).to(dtype).cuda()

    cu = torch.tensor([0, 300, T], dtype=torch.int32)
    cud, idx = cu.cuda(), torch.tensor([1, 0], dtype=torch.int32).cuda()
    q, k, v, gate, do = (rnd(T, W) for _ in range(5))
    b, A, dt = rnd(T, H), rnd(H, dtype=torch.float32), 0.1 * rnd(W, dtype=torch.float32)
    pool, wt = 0.1 * rnd(2, H, D, D), rnd(W, dtype=torch.float32)
    out, dz, dw = torch.empty_like(q), torch.empty_like(q), torch.empty_like(wt)
    grads = [torch.empty_like(t) for t in (q, k, v, gate, b, A, dt)]
    state = pool.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        kda.kda_prefill_varlen(cu, cud, q, k, v, gate, b, A, dt, state, idx, out, stream=s)
        kda.kda_prefill_varlen_backward(cu, cud, q, k, v, gate, b, A, dt, pool, idx, do,
                                        *grads[:5], dA_log=grads[5], ddt_bias=grads[6],
                                        stream=s.cuda_stream)
        kda.kda_rmsnorm_backward(out, wt, do, dz, dw, stream=s)
    for _ in range(3):
        state.copy_(pool)
        for t in (out, dz, dw, *grads):
            t.fill_(-1.0)
        graph.replay()
        torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        for x, y in zip([out, state, *grads, dz, dw], want):
            assert torch.equal(x, y)
