"""Python binding of the KDA step library (libkda.so, HIP for gfx950).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, checks dtype/device/contiguity of the innermost dimension,
and passes raw pointers, element strides and the current HIP stream to the C
ABI declared in include/kda.h (the recurrence: decode, verify, prefill),
kda_backward.h (the prefill's gradients), kda_norm.h (the layer's RMS norms
and their gradients) and kda_cache.h (the paged 8-bit key/value cache of the
attention layers beside it). All arithmetic runs in the library's kernels;
there is no fallback. If libkda.so is missing the first call raises.

bf16 tensors are torch.bfloat16; A_log and dt_bias are float32; indices and
ring metadata are int32.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkda.so")
HEAD_DIM = 128

_lib = None

_c = ctypes
_P = _c.c_void_p
_I32 = _c.c_int32
_I64 = _c.c_int64
_F = _c.c_float

_SIGS = {
    "kda_status_string": (_c.c_char_p, [_c.c_int]),
    "kda_decode": (_c.c_int, [_I32, _I32, _I32, _I32,
                              _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                              _P, _P, _F, _F, _I32, _I32, _P, _I64, _I64, _P, _P, _I64, _P]),
    "kda_verify_ucache_flush": (_c.c_int, [_I32, _I32, _I32, _I32, _I32,
                                           _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64,
                                           _P, _I64, _I64, _P, _I64, _I64,
                                           _P, _P, _F, _F, _I32, _I32, _P, _I64, _I64, _P,
                                           _P, _P, _P, _I32, _P, _P, _I32, _I32, _I32,
                                           _P, _I64, _I64, _P]),
    "kda_prefill_workspace_size": (_c.c_size_t, [_I32, _I64, _I32, _I32, _I32]),
    "kda_prefill_varlen": (_c.c_int, [_I32, _I64, _I32, _I32, _I32, _P, _P,
                                      _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                      _P, _P, _F, _F, _I32, _I32, _P, _I64, _I64, _P, _I32,
                                      _P, _I64, _P, _I64, _P, _I32, _P, _P, _P, _I32, _P,
                                      _I32, _P, _c.c_size_t, _P]),
    "kda_prefill_varlen_noalloc": (_c.c_int, [_I32, _I64, _I32, _I32, _I32, _P, _P,
                                              _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                              _P, _P, _F, _F, _I32, _I32, _P, _I64, _I64, _P,
                                              _I32, _P, _I64, _P, _I64, _P, _I32, _P, _P, _P,
                                              _I32, _P, _I32, _P]),
    "kda_prefill_backward_workspace_size": (_c.c_size_t, [_I32, _I64, _I32, _I32, _I32]),
    "kda_prefill_varlen_backward": (_c.c_int, [_I32, _I64, _I32, _I32, _I32, _P, _P,
                                               _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                               _P, _P, _F, _F, _I32, _I32, _P, _I64, _I64, _P,
                                               _I32, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64,
                                               _P, _I64, _P, _I64, _P, _P, _P, _P, _c.c_size_t,
                                               _P]),
    "kda_rmsnorm": (_c.c_int, [_I64, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _F,
                               _I32, _P, _I64, _I32, _P, _I64, _P]),
    "kda_rmsnorm_backward_workspace_size": (_c.c_size_t, [_I64, _I32, _I32]),
    "kda_rmsnorm_backward": (_c.c_int, [_I64, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                        _P, _F, _P, _I64, _P, _I64, _P, _P, _c.c_size_t, _P]),
    "kda_cache_write": (_c.c_int, [_I32, _I64, _I32, _I32, _P, _P, _I64, _P, _I64, _I32, _I32,
                                   _I64, _P, _I64, _P, _I64, _P, _P, _P, _I32, _I64, _P, _P]),
    "kda_cache_read": (_c.c_int, [_I32, _I64, _I32, _I32, _P, _P, _I64, _P, _I64, _I32, _I32,
                                  _I64, _P, _I64, _P, _I64, _P, _P, _P, _I32, _I64, _P, _P]),
    "kda_cache_attention_workspace_size": (_c.c_size_t, [_I32, _I64, _I32, _I32]),
    "kda_cache_attention": (_c.c_int, [_I32, _I64, _I32, _I32, _I32, _P, _P, _P, _I64, _I32, _I32,
                                       _I64, _P, _I64, _P, _I64, _P, _P, _P, _I32, _I64, _P, _F,
                                       _P, _I64, _P, _I64, _P, _c.c_size_t, _P]),
}

# Scratch held by the library per device for kda_prefill_varlen_noalloc
# (KDA_NOALLOC_SCRATCH_BYTES in include/kda.h).
NOALLOC_SCRATCH_BYTES = 64 << 20
# Prefill calls with at least this many (document, head) chains run the fused
# 64-token chunk kernel (no workspace); fewer run the two-stage form.
FUSED_MIN_CHAINS = 256


# gate_mode bits (include/kda.h): g_raw holds the log-decay g itself (A_log and
# dt_bias may then be None); beta_raw holds beta itself.
GATE_PRECOMPUTED = 1
BETA_PRESIGMOID = 2
GATE_PER_HEAD = 4  # one gate value (and dt_bias) per head


class KdaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {kda_status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load libkda.so (built in-tree by __graft_entry__.build()); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the HIP library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise KdaError(fn, status)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return _P(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return _P(t.data_ptr()) if t is not None else _P(0)


def _workspace(need, dev, stream):
    """A workspace for one call on `stream` (None: dev's current one), from that
    stream's memory pool: it is ordered behind the stream's earlier work, and whatever
    gets the block after the call behind the call's kernels. A block of the current
    stream's pool could be handed out again while another stream's kernels use it."""
    import torch
    if need == 0:
        return None
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if getattr(stream, "device", dev) != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    if not isinstance(stream, torch.cuda.Stream):  # a handle, or anything that holds one
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=dev)


def _workspace_bytes(t, dev):
    """The size of a workspace (None: 0): contiguous, so that it holds as many bytes as it
    has elements, and where the kernels run."""
    if t is None:
        return 0
    if t.device != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous GPU tensor on {dev}")
    return t.numel() * t.element_size()


def _bf16(name, t, last_contig=True):
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if last_contig and t.stride(-1) != 1:
        raise ValueError(f"{name}: the innermost dimension must be contiguous")


def _f32(name, t, optional=False):
    import torch
    if optional and t is None:
        return
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 GPU tensor")


def _i32(name, t):
    import torch
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 GPU tensor")


def _state_dtype(state_pool) -> int:
    """KDA_STATE_BF16 (0), KDA_STATE_FP16 (1) or KDA_STATE_FP8 (2, torch's
    float8_e4m3fn), from the pool tensor's dtype."""
    import torch
    if state_pool.dtype == torch.float16:
        return 1
    if state_pool.dtype == torch.float8_e4m3fn:
        return 2
    _bf16("state_pool", state_pool)
    return 0


def _pool_geometry(state_pool, H):
    """Pool: bf16, fp16 or fp8 e4m3 tensor whose dim 0 indexes slots; each slot's first
    H*128*128 elements are contiguous. Returns (num_slots, slot_stride)."""
    if not state_pool.is_cuda or state_pool.stride(-1) != 1:
        raise ValueError("state_pool must be a GPU tensor with a contiguous last dimension")
    n = state_pool.shape[0]
    inner = state_pool[0] if n > 0 else None
    if n > 0 and not inner.is_contiguous():
        raise ValueError("state_pool: each slot must be contiguous")
    if n > 0 and inner.numel() < H * HEAD_DIM * HEAD_DIM:
        raise ValueError("state_pool: slot smaller than H*128*128")
    return n, (state_pool.stride(0) if n > 0 else H * HEAD_DIM * HEAD_DIM)


def _ring_rows(k_cache, u_cache, g_cache, N, H) -> int:
    """The three ring tensors must each be [N, H, R, 128] with one R; returns R."""
    shapes = [tuple(t.shape) for t in (k_cache, u_cache, g_cache)]
    R = shapes[0][2] if len(shapes[0]) == 4 else -1
    for name, sh in zip(("k_cache", "u_cache", "g_cache"), shapes):
        if sh != (N, H, R, HEAD_DIM):
            raise ValueError(f"{name} must be [N={N}, H={H}, R, 128] with the same R as "
                             f"k_cache, got {list(sh)}")
    return R


def kda_decode(q, k, v, g_raw, beta_raw, A_log, dt_bias, state_pool, state_indices, out,
               lower_bound: float = -5.0, scale: float = 1.0, gate_mode: int = 0,
               stream=None) -> None:
    """T=1 decode. q, k, v, g_raw, out: bf16 [B, H*128] (row-strided views
    allowed); beta_raw bf16 [B, H]; A_log fp32 [H]; dt_bias fp32 [H*128];
    state_pool bf16 or fp16 [N, ...] (slot-major; its dtype selects the state
    element type); state_indices int32 [B]."""
    B, W = q.shape
    H = W // HEAD_DIM
    for n, t in (("q", q), ("k", k), ("v", v), ("g_raw", g_raw), ("beta_raw", beta_raw),
                 ("out", out)):
        _bf16(n, t)
    pre = bool(gate_mode & GATE_PRECOMPUTED)
    _f32("A_log", A_log, optional=pre)
    _f32("dt_bias", dt_bias, optional=pre)
    _i32("state_indices", state_indices)
    N, slot_stride = _pool_geometry(state_pool, H)
    st = lib().kda_decode(B, H, HEAD_DIM, HEAD_DIM,
                          _ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(v), v.stride(0),
                          _ptr(g_raw), g_raw.stride(0), _ptr(beta_raw), beta_raw.stride(0),
                          _ptr(A_log), _ptr(dt_bias), float(lower_bound), float(scale),
                          int(gate_mode), _state_dtype(state_pool),
                          _ptr(state_pool) if N else _P(0), N, slot_stride,
                          _ptr(state_indices), _ptr(out), out.stride(0), _stream(stream))
    _check("kda_decode", st)


def kda_verify_ucache_flush(q, k, v, g_raw, beta_raw, A_log, dt_bias, state_pool,
                            state_indices, k_cache, u_cache, g_cache, hist_len, cache_base,
                            out, flush_min: int, w_ring: int = 16,
                            restart_hist_on_flush: bool = True, lower_bound: float = -5.0,
                            scale: float = 1.0, gate_mode: int = 0, stream=None) -> None:
    """Verify+fold. q, k, v, g_raw, out: bf16 [B, T, H*128]; beta_raw bf16
    [B, T, H]; k_cache/u_cache bf16 [N, H, R, 128]; g_cache fp32 [N, H, R, 128];
    hist_len, cache_base int32 [B]."""
    B, T, W = q.shape
    H = W // HEAD_DIM
    for n, t in (("q", q), ("k", k), ("v", v), ("g_raw", g_raw), ("beta_raw", beta_raw),
                 ("out", out), ("k_cache", k_cache), ("u_cache", u_cache)):
        _bf16(n, t)
    pre = bool(gate_mode & GATE_PRECOMPUTED)
    _f32("A_log", A_log, optional=pre)
    _f32("dt_bias", dt_bias, optional=pre)
    _f32("g_cache", g_cache)
    for n, t in (("state_indices", state_indices), ("hist_len", hist_len),
                 ("cache_base", cache_base)):
        _i32(n, t)
    if not (k_cache.is_contiguous() and u_cache.is_contiguous()):
        raise ValueError("ring caches must be contiguous")
    N, slot_stride = _pool_geometry(state_pool, H)
    R = _ring_rows(k_cache, u_cache, g_cache, N, H)
    st = lib().kda_verify_ucache_flush(
        B, T, H, HEAD_DIM, HEAD_DIM,
        _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.stride(1),
        _ptr(v), v.stride(0), v.stride(1), _ptr(g_raw), g_raw.stride(0), g_raw.stride(1),
        _ptr(beta_raw), beta_raw.stride(0), beta_raw.stride(1),
        _ptr(A_log), _ptr(dt_bias), float(lower_bound), float(scale), int(gate_mode),
        _state_dtype(state_pool), _ptr(state_pool) if N else _P(0), N, slot_stride,
        _ptr(state_indices), _ptr(k_cache), _ptr(u_cache), _ptr(g_cache), R, _ptr(hist_len), _ptr(cache_base),
        int(flush_min), int(w_ring), 1 if restart_hist_on_flush else 0,
        _ptr(out), out.stride(0), out.stride(1), _stream(stream))
    _check("kda_verify_ucache_flush", st)


def kda_prefill_workspace_size(n_docs: int, total_tokens: int, H: int) -> int:
    return int(lib().kda_prefill_workspace_size(n_docs, total_tokens, H, HEAD_DIM, HEAD_DIM))


def kda_prefill_varlen(cu_seqlens_host, cu_seqlens, q, k, v, g_raw, beta_raw, A_log, dt_bias,
                       state_pool, state_indices, out, workspace=None,
                       use_initial_state: bool = True, lower_bound: float = -5.0,
                       scale: float = 1.0, gate_mode: int = 0, checkpoints=None,
                       checkpoint_cu_starts=None, checkpoint_interval: int = 16,
                       ring=None, cache_base=None, ring_tail: int = 0,
                       stream=None) -> None:
    """Varlen prefill. cu_seqlens_host: CPU int32 [n_docs+1]; cu_seqlens: the
    same on the GPU; q, k, v, g_raw, out: bf16 [Ttot, H*128] (token-strided);
    beta_raw bf16 [Ttot, H]; state_indices int32 [n_docs]; workspace: uint8
    GPU tensor of >= kda_prefill_workspace_size(...) bytes, or None to have
    one allocated here for this call. checkpoints: bf16 [rows, H, 128, 128]
    (contiguous) receiving the state after every checkpoint_interval tokens of
    each document at rows checkpoint_cu_starts[d] + i (int64 GPU tensor
    [n_docs]), or None. ring = (k_cache bf16, u_cache bf16, g_cache fp32, each
    [N, H, R, 128]) with cache_base int32 [n_docs] and ring_tail in 1..16: each
    document hands its last prefill_handoff_hist(...)[d] tokens to the ring at
    rows cache_base[d] onwards, and its slot receives the state before them."""
    args = _prefill_args(cu_seqlens_host, cu_seqlens, q, k, v, g_raw, beta_raw, A_log, dt_bias,
                         state_pool, state_indices, out, use_initial_state, lower_bound, scale,
                         gate_mode, checkpoints, checkpoint_cu_starts, checkpoint_interval, ring,
                         cache_base, ring_tail)
    if workspace is None:
        need = kda_prefill_workspace_size(args[0], args[1], args[2])
        workspace = _workspace(need, q.device, stream)
    ws_bytes = _workspace_bytes(workspace, q.device)
    st = lib().kda_prefill_varlen(*args, _ptr(workspace), ws_bytes, _stream(stream))
    _check("kda_prefill_varlen", st)


def kda_prefill_varlen_noalloc(cu_seqlens_host, cu_seqlens, q, k, v, g_raw, beta_raw, A_log,
                               dt_bias, state_pool, state_indices, out,
                               use_initial_state: bool = True, lower_bound: float = -5.0,
                               scale: float = 1.0, gate_mode: int = 0, checkpoints=None,
                               checkpoint_cu_starts=None, checkpoint_interval: int = 16,
                               ring=None, cache_base=None, ring_tail: int = 0,
                               stream=None) -> None:
    """kda_prefill_varlen without a workspace: allocates nothing (here or in the
    library). Where a workspace is needed the library's per-device scratch of
    NOALLOC_SCRATCH_BYTES serves; a call needing more raises KdaError
    (KDA_ERR_SCRATCH_LIMIT). Calls on one device share that scratch, so calls
    on different streams must be ordered."""
    args = _prefill_args(cu_seqlens_host, cu_seqlens, q, k, v, g_raw, beta_raw, A_log, dt_bias,
                         state_pool, state_indices, out, use_initial_state, lower_bound, scale,
                         gate_mode, checkpoints, checkpoint_cu_starts, checkpoint_interval, ring,
                         cache_base, ring_tail)
    st = lib().kda_prefill_varlen_noalloc(*args, _stream(stream))
    _check("kda_prefill_varlen_noalloc", st)


def _prefill_args(cu_seqlens_host, cu_seqlens, q, k, v, g_raw, beta_raw, A_log, dt_bias,
                  state_pool, state_indices, out, use_initial_state, lower_bound, scale,
                  gate_mode, checkpoints, checkpoint_cu_starts, checkpoint_interval, ring,
                  cache_base, ring_tail):
    """Checks and the C arguments shared by both prefill entry points, up to
    (not including) the workspace and the stream."""
    import torch
    if cu_seqlens_host.dtype != torch.int32 or cu_seqlens_host.is_cuda or \
            not cu_seqlens_host.is_contiguous():
        raise ValueError("cu_seqlens_host must be a contiguous int32 CPU tensor")
    _i32("cu_seqlens", cu_seqlens)
    _i32("state_indices", state_indices)
    n_docs = cu_seqlens_host.shape[0] - 1
    Ttot, W = q.shape
    H = W // HEAD_DIM
    for n, t in (("q", q), ("k", k), ("v", v), ("g_raw", g_raw), ("beta_raw", beta_raw),
                 ("out", out)):
        _bf16(n, t)
    pre = bool(gate_mode & GATE_PRECOMPUTED)
    _f32("A_log", A_log, optional=pre)
    _f32("dt_bias", dt_bias, optional=pre)
    N, slot_stride = _pool_geometry(state_pool, H)
    ck_rows = 0
    if checkpoints is not None:
        if checkpoints.dtype != state_pool.dtype or not checkpoints.is_cuda:
            raise ValueError("checkpoints must be a GPU tensor of the state pool's dtype")
        if not checkpoints.is_contiguous() or \
                checkpoints.numel() != checkpoints.shape[0] * H * HEAD_DIM * HEAD_DIM:
            raise ValueError("checkpoints must be a contiguous bf16 [rows, H, 128, 128] tensor")
        if checkpoint_cu_starts is None or checkpoint_cu_starts.dtype != torch.int64 or \
                not checkpoint_cu_starts.is_cuda or not checkpoint_cu_starts.is_contiguous():
            raise ValueError("checkpoint_cu_starts must be a contiguous int64 GPU tensor")
        ck_rows = checkpoints.shape[0]
    kc = uc = gc = None
    R = 0
    if ring_tail:
        kc, uc, gc = ring
        _bf16("k_cache", kc)
        _bf16("u_cache", uc)
        _f32("g_cache", gc)
        _i32("cache_base", cache_base)
        if not (kc.is_contiguous() and uc.is_contiguous() and gc.is_contiguous()):
            raise ValueError("ring caches must be contiguous")
        R = _ring_rows(kc, uc, gc, N, H)
    cu_h = _P(cu_seqlens_host.data_ptr())
    return (
        n_docs, Ttot, H, HEAD_DIM, HEAD_DIM, cu_h, _ptr(cu_seqlens),
        _ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(v), v.stride(0),
        _ptr(g_raw), g_raw.stride(0), _ptr(beta_raw), beta_raw.stride(0),
        _ptr(A_log), _ptr(dt_bias), float(lower_bound), float(scale), int(gate_mode),
        _state_dtype(state_pool), _ptr(state_pool) if N else _P(0), N, slot_stride,
        _ptr(state_indices), 1 if use_initial_state else 0, _ptr(out), out.stride(0),
        _ptr(checkpoints), ck_rows, _ptr(checkpoint_cu_starts), int(checkpoint_interval),
        _ptr(kc), _ptr(uc), _ptr(gc), R, _ptr(cache_base), int(ring_tail))


def prefill_handoff_hist(cu_seqlens_host, ring_tail: int):
    """Ring history entries each document hands off (the hist_len of its next
    verify call): min(ring_tail, tokens after its last 16-token boundary), 0 for
    an empty document. CPU int32 tensor [n_docs]."""
    import torch
    lens = (cu_seqlens_host[1:] - cu_seqlens_host[:-1]).to(torch.int64)
    last = lens - 16 * torch.div(lens - 1, 16, rounding_mode="floor")
    return torch.where(lens > 0, torch.clamp(last, max=int(ring_tail)),
                       torch.zeros_like(lens)).to(torch.int32)


def _same_device(first, named):
    """Every given tensor is on the first one's GPU; returns that device."""
    dev = first.device
    at = first.get_device()
    for name, t in named:
        if t is not None and t.get_device() != at:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return dev


def _adr(t):
    """A tensor's address for a void* argument (None: NULL)."""
    return None if t is None else t.data_ptr()


def _launch(fn, dev, stream, *args):
    """Call a C entry point with `dev` current, on the given stream or on that
    device's current one (appended as the last argument)."""
    import torch
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
    elif getattr(stream, "device", dev) != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    call = getattr(lib(), fn)
    if torch.cuda.current_device() == dev.index:
        st = call(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = call(*args, raw)
    _check(fn, st)


def kda_prefill_backward_workspace_size(n_docs: int, total_tokens: int, H: int) -> int:
    return int(lib().kda_prefill_backward_workspace_size(n_docs, total_tokens, H, HEAD_DIM,
                                                         HEAD_DIM))


def kda_prefill_varlen_backward(cu_seqlens_host, cu_seqlens, q, k, v, g_raw, beta_raw, A_log,
                                dt_bias, state_pool, state_indices, d_out, dq, dk, dv, dg, dbeta,
                                dA_log=None, ddt_bias=None, d_final_state=None,
                                d_initial_state=None, workspace=None,
                                use_initial_state: bool = True, lower_bound: float = -5.0,
                                scale: float = 1.0, gate_mode: int = 0, stream=None) -> None:
    """Gradients of one kda_prefill_varlen call, from the same inputs. state_pool is
    the pool as it was before that call (only read). d_out, dq, dk, dv: bf16
    [Ttot, H*128] (token-strided); dg like g_raw, dbeta like beta_raw; dA_log fp32 like
    A_log and ddt_bias fp32 like dt_bias, or None; d_final_state and d_initial_state:
    contiguous fp32 [n_docs, H, 128, 128] (value, key), or None. workspace: uint8 GPU
    tensor of >= kda_prefill_backward_workspace_size(...) bytes, or None to have one
    allocated here for this call."""
    import torch
    if cu_seqlens_host.dtype != torch.int32 or cu_seqlens_host.is_cuda or \
            not cu_seqlens_host.is_contiguous() or cu_seqlens_host.dim() != 1 or \
            cu_seqlens_host.shape[0] < 1:
        raise ValueError("cu_seqlens_host must be a contiguous int32 CPU tensor [n_docs + 1]")
    n_docs = cu_seqlens_host.shape[0] - 1
    T, W = q.shape
    H = W // HEAD_DIM
    if W != H * HEAD_DIM or H < 1:
        raise ValueError(f"q must be [Ttot, H*128], got {list(q.shape)}")
    gw = H if gate_mode & GATE_PER_HEAD else W
    pre = bool(gate_mode & GATE_PRECOMPUTED)
    for n, t, w in (("q", q, W), ("k", k, W), ("v", v, W), ("g_raw", g_raw, gw),
                    ("beta_raw", beta_raw, H), ("d_out", d_out, W), ("dq", dq, W), ("dk", dk, W),
                    ("dv", dv, W), ("dg", dg, gw), ("dbeta", dbeta, H)):
        _bf16(n, t, last_contig=w > 1)
        if tuple(t.shape) != (T, w):
            raise ValueError(f"{n} must be [{T}, {w}], got {list(t.shape)}")
    for n, t, w in (("A_log", A_log, H), ("dt_bias", dt_bias, gw), ("dA_log", dA_log, H),
                    ("ddt_bias", ddt_bias, gw)):
        if t is None and (pre or n in ("dA_log", "ddt_bias")):
            continue
        _f32(n, t)
        if t.numel() != w:
            raise ValueError(f"{n} must hold {w} values, got {t.numel()}")
    for n, t, w in (("cu_seqlens", cu_seqlens, n_docs + 1), ("state_indices", state_indices,
                                                             n_docs)):
        _i32(n, t)
        if t.numel() != w:
            raise ValueError(f"{n} must hold {w} values, got {t.numel()}")
    for n, t in (("d_final_state", d_final_state), ("d_initial_state", d_initial_state)):
        _f32(n, t, optional=True)
        if t is not None and tuple(t.shape) != (n_docs, H, HEAD_DIM, HEAD_DIM):
            raise ValueError(f"{n} must be [{n_docs}, {H}, 128, 128], got {list(t.shape)}")
    N, slot_stride = _pool_geometry(state_pool, H)
    dev = _same_device(q, (("cu_seqlens", cu_seqlens), ("k", k), ("v", v), ("g_raw", g_raw),
                           ("beta_raw", beta_raw), ("A_log", A_log), ("dt_bias", dt_bias),
                           ("state_pool", state_pool), ("state_indices", state_indices),
                           ("d_out", d_out), ("dq", dq), ("dk", dk), ("dv", dv), ("dg", dg),
                           ("dbeta", dbeta), ("dA_log", dA_log), ("ddt_bias", ddt_bias),
                           ("d_final_state", d_final_state),
                           ("d_initial_state", d_initial_state), ("workspace", workspace)))
    if workspace is None:
        workspace = _workspace(kda_prefill_backward_workspace_size(n_docs, T, H), dev, stream)
    ws_bytes = _workspace_bytes(workspace, dev)
    _launch("kda_prefill_varlen_backward", dev, stream,
            n_docs, T, H, HEAD_DIM, HEAD_DIM, cu_seqlens_host.data_ptr(), _adr(cu_seqlens),
            _adr(q), q.stride(0), _adr(k), k.stride(0), _adr(v), v.stride(0),
            _adr(g_raw), g_raw.stride(0), _adr(beta_raw), beta_raw.stride(0),
            _adr(A_log), _adr(dt_bias), float(lower_bound), float(scale), int(gate_mode),
            _state_dtype(state_pool), _adr(state_pool) if N else None, N, slot_stride,
            _adr(state_indices), 1 if use_initial_state else 0, _adr(d_out), d_out.stride(0),
            _adr(d_final_state), _adr(dq), dq.stride(0), _adr(dk), dk.stride(0),
            _adr(dv), dv.stride(0), _adr(dg), dg.stride(0), _adr(dbeta), dbeta.stride(0),
            _adr(dA_log), _adr(ddt_bias), _adr(d_initial_state), _adr(workspace), ws_bytes)


def _vectors(name, t, rows, heads, width):
    """bf16 [rows, width] or [rows, heads, width] with contiguous rows: the row
    stride (0 for None)."""
    if t is None:
        return 0
    _bf16(name, t, last_contig=False)
    return _row_stride(name, t, rows, heads, width)


def _row_stride(name, t, rows, heads, width):
    shape, st = tuple(t.shape), t.stride()
    if shape != (rows, heads, width) and (heads != 1 or shape != (rows, width)):
        raise ValueError(f"{name} must be [{rows}, {heads}, {width}], got {list(shape)}")
    if (width > 1 and st[-1] != 1) or (len(st) == 3 and heads > 1 and st[1] != width):
        raise ValueError(f"{name}: a row's heads and channels must be contiguous")
    return st[0]


def _norm_sizes(name, x):
    if x.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows, width] or [rows, heads, width]")
    return (x.shape[0], 1, x.shape[1]) if x.dim() == 2 else tuple(x.shape)


def _norm_weight(name, w, width):
    _f32(name, w)
    if tuple(w.shape) != (width,):
        raise ValueError(f"{name} must be [{width}], got {list(w.shape)}")


def kda_rmsnorm(x, weight, out, residual=None, residual_out=None, gate=None, scales=None,
                eps: float = 1e-6, stream=None) -> None:
    """y = norm(x [+ residual]) * weight [* sigmoid(gate)] per vector of the last
    dimension. x, residual, residual_out, gate: bf16 [rows, width] or [rows,
    heads, width] (row-strided); weight fp32 [width]; out bf16, or
    float8_e4m3fn holding y / scale with scales fp32 [rows, n], contiguous rows:
    n = heads (one scale per vector) or n = heads * width / 128 (one per 128
    channels). residual_out (may be residual) receives x + residual."""
    import torch
    rows, heads, width = _norm_sizes("x", x)
    xs = _vectors("x", x, rows, heads, width)
    rs = _vectors("residual", residual, rows, heads, width)
    ro = _vectors("residual_out", residual_out, rows, heads, width)
    gs = _vectors("gate", gate, rows, heads, width)
    _norm_weight("weight", weight, width)
    fp8 = out.dtype == torch.float8_e4m3fn
    if not fp8:
        _bf16("out", out, last_contig=False)
    elif not out.is_cuda:
        raise ValueError("out must be a GPU tensor")
    os_ = _row_stride("out", out, rows, heads, width)
    group = ss = 0
    if fp8:
        if scales is None or scales.dtype != torch.float32 or not scales.is_cuda or \
                scales.dim() != 2 or scales.shape[0] != rows or \
                (scales.shape[1] > 1 and scales.stride(1) != 1):
            raise ValueError("scales must be a float32 GPU tensor [rows, n] with contiguous rows")
        ss = scales.stride(0)
        if scales.shape[1] != heads:
            if width % 128 != 0 or scales.shape[1] != heads * width // 128:
                raise ValueError(f"scales must have {heads} columns, or one per 128 channels, "
                                 f"got {scales.shape[1]}")
            group = 128
    elif scales is not None:
        raise ValueError("scales belong to an fp8 output")
    dev = _same_device(x, (("weight", weight), ("out", out), ("residual", residual),
                           ("residual_out", residual_out), ("gate", gate), ("scales", scales)))
    _launch("kda_rmsnorm", dev, stream, rows, heads, width, _adr(x), xs, _adr(residual), rs,
            _adr(residual_out), ro, _adr(gate), gs, _adr(weight), float(eps), 1 if fp8 else 0,
            _adr(out), os_, group, _adr(scales), ss)


def kda_rmsnorm_backward_workspace_size(rows: int, heads: int, width: int) -> int:
    return int(lib().kda_rmsnorm_backward_workspace_size(rows, heads, width))


def kda_rmsnorm_backward(z, weight, dy, dz, dweight=None, gate=None, dgate=None, d_residual=None,
                         eps: float = 1e-6, workspace=None, stream=None) -> None:
    """Gradients of kda_rmsnorm at its input z (x, or residual_out). z, dy, dz,
    gate, dgate, d_residual: bf16 [rows, width] or [rows, heads, width]
    (row-strided); weight, dweight fp32 [width]. dz receives the gradient at z plus
    d_residual, the gradient that reaches z past the norm. workspace: uint8 GPU
    tensor of >= kda_rmsnorm_backward_workspace_size(...) bytes, or None to have
    one allocated here for this call."""
    rows, heads, width = _norm_sizes("z", z)
    zs = _vectors("z", z, rows, heads, width)
    ys = _vectors("dy", dy, rows, heads, width)
    gs = _vectors("gate", gate, rows, heads, width)
    rs = _vectors("d_residual", d_residual, rows, heads, width)
    ds = _vectors("dz", dz, rows, heads, width)
    dgs = _vectors("dgate", dgate, rows, heads, width)
    _norm_weight("weight", weight, width)
    if dweight is not None:
        _norm_weight("dweight", dweight, width)
    dev = _same_device(z, (("weight", weight), ("dy", dy), ("dz", dz), ("dweight", dweight),
                           ("gate", gate), ("dgate", dgate), ("d_residual", d_residual),
                           ("workspace", workspace)))
    if workspace is None and dweight is not None and rows > 0:
        workspace = _workspace(kda_rmsnorm_backward_workspace_size(rows, heads, width), dev,
                               stream)
    ws_bytes = _workspace_bytes(workspace, dev)
    _launch("kda_rmsnorm_backward", dev, stream, rows, heads, width, _adr(z), zs, _adr(dy), ys,
            _adr(gate), gs, _adr(d_residual), rs, _adr(weight), float(eps), _adr(dz), ds,
            _adr(dgate), dgs, _adr(dweight), _adr(workspace), ws_bytes)


def _paged(name, t, dtype, shape):
    """A cache tensor of that dtype and shape whose pages are contiguous: its page stride."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    st = t.stride()
    if st[1:] != (shape[2] * HEAD_DIM, HEAD_DIM, 1) and shape[0] > 0 and not t[0].is_contiguous():
        raise ValueError(f"{name}: each page must be contiguous")
    return st[0]


def _cache_args(torch, first, tokens, cache, cu_seqlens):
    """Checks of a paged cache, its tables and cu_seqlens, all on the GPU of `first` (a
    (name, tensor)): the C arguments from the dtype to kv_lens, the sequences, the heads."""
    k_cache, v_cache, k_scale, v_scale, page_table, kv_lens = cache
    dtype, shape = k_cache.dtype, k_cache.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM:
        raise ValueError(f"k_cache must be [pages, H, page_size, 128], got {list(shape)}")
    if dtype is not torch.float8_e4m3fn and dtype is not torch.int8:
        raise TypeError(f"k_cache must be float8_e4m3fn or int8, got {dtype}")
    kp = _paged("k_cache", k_cache, dtype, shape)
    vp = _paged("v_cache", v_cache, dtype, shape)
    pages, H, size, _ = shape
    f32, i32 = torch.float32, torch.int32
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype is not f32 or t.shape != (pages, H) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor [{pages}, {H}], got "
                             f"{t.dtype} {list(t.shape)}")
    at = kv_lens.shape
    if kv_lens.dtype is not i32 or len(at) != 1 or not kv_lens.is_contiguous():
        raise ValueError(f"kv_lens must be a contiguous int32 tensor [sequences], got "
                         f"{kv_lens.dtype} {list(at)}")
    n = at[0]
    at, st = page_table.shape, page_table.stride()
    if page_table.dtype is not i32 or len(at) != 2 or at[0] != n or at[1] < 1 or \
            (st[1] != 1 and at[1] > 1):
        raise ValueError(f"page_table must be an int32 tensor [{n}, pages of a sequence] with "
                         f"contiguous rows, got {page_table.dtype} {list(at)}")
    if cu_seqlens is None:
        if tokens > 0 and (n == 0 or tokens % n != 0):
            raise ValueError(f"{tokens} tokens of {n} sequences need cu_seqlens")
        cu = None
    else:
        if cu_seqlens.dtype is not i32 or cu_seqlens.shape != (n + 1,) or \
                not cu_seqlens.is_contiguous():
            raise ValueError(f"cu_seqlens must be a contiguous int32 tensor [{n + 1}], got "
                             f"{cu_seqlens.dtype} {list(cu_seqlens.shape)}")
        cu = cu_seqlens.data_ptr()
    if not first[1].is_cuda:
        raise ValueError(f"{first[0]} must be a GPU tensor")
    gpu = first[1].get_device()
    for t in cache:
        if t.get_device() != gpu:
            raise ValueError(f"the cache and its tables must be on {first[1].device}, got a "
                             f"tensor on {t.device}")
    if cu is not None and cu_seqlens.get_device() != gpu:
        raise ValueError(f"cu_seqlens must be on {first[1].device}, got {cu_seqlens.device}")
    return (1 if dtype is torch.int8 else 0, size, pages, k_cache.data_ptr(), kp,
            v_cache.data_ptr(), vp, k_scale.data_ptr(), v_scale.data_ptr(),
            page_table.data_ptr(), at[1], st[0] if n > 1 else at[1],
            kv_lens.data_ptr()), n, H, cu


def _token_rows(name, t, bf16, tokens, width):
    """bf16 [tokens, width] with contiguous rows: the row stride."""
    if t.dtype is not bf16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    st = t.stride()
    if t.shape != (tokens, width) or st[1] != 1:
        raise ValueError(f"{name} must be [{tokens}, {width}] with contiguous rows, got "
                         f"{list(t.shape)}")
    return st[0]


def _cache_rows(fn, k, v, cache, cu_seqlens, stream):
    """kda_cache_write and kda_cache_read."""
    import torch
    if k.dim() != 2:
        raise ValueError(f"k must be [T, H*128], got {list(k.shape)}")
    T = k.shape[0]
    args, n, H, cu = _cache_args(torch, ("k", k), T, cache, cu_seqlens)
    W, bf16 = H * HEAD_DIM, torch.bfloat16
    ks, vs = _token_rows("k", k, bf16, T, W), _token_rows("v", v, bf16, T, W)
    dev = _same_device(k, (("v", v),))
    _launch(fn, dev, stream, n, T, H, HEAD_DIM, cu, k.data_ptr(), ks, v.data_ptr(), vs, *args)


def kda_cache_write(k, v, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens,
                    cu_seqlens=None, stream=None) -> None:
    """Quantise new tokens into their sequences' pages. k, v: bf16 [T, H*128]
    (row-strided); k_cache, v_cache: float8_e4m3fn or int8 [pages, H, page_size, 128]
    (page_size 16, 32, 64, 128 or 256; page-strided); k_scale, v_scale: fp32 [pages, H];
    page_table: int32 [n, pages of a sequence] (row-strided); kv_lens: int32 [n], lengths
    with the new tokens, which are the last ones of each sequence. cu_seqlens: int32
    [n + 1], or None where every sequence has T / n new tokens. Caches and scales are
    updated in place."""
    _cache_rows("kda_cache_write", k, v, (k_cache, v_cache, k_scale, v_scale, page_table, kv_lens),
                cu_seqlens, stream)


def kda_cache_read(k, v, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens,
                   cu_seqlens=None, stream=None) -> None:
    """The last tokens of each sequence, code * scale, into k and v (bf16 [T, H*128],
    row-strided). Other arguments as for kda_cache_write: sequence b's rows receive its
    positions kv_lens[b] - n_b .. kv_lens[b] - 1."""
    _cache_rows("kda_cache_read", k, v, (k_cache, v_cache, k_scale, v_scale, page_table, kv_lens),
                cu_seqlens, stream)


def kda_cache_attention_workspace_size(n_seqs: int, total_tokens: int, H_q: int,
                                       H_kv: int) -> int:
    return int(lib().kda_cache_attention_workspace_size(n_seqs, total_tokens, H_q, H_kv))


def kda_cache_attention(q, out, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens,
                        cu_seqlens_host=None, cu_seqlens=None, lse=None,
                        scale: float = HEAD_DIM ** -0.5, workspace=None, stream=None) -> None:
    """Causal softmax attention of each sequence's last tokens over its cache, which
    holds them already. q, out: bf16 [T, H_q*128] (row-strided), H_q a multiple of the
    cache's H; lse: fp32 [T, H_q] (row-strided) or None. cu_seqlens_host (CPU int32
    [n + 1]) and cu_seqlens (the same on the GPU), or None where every sequence has T / n
    new tokens. Cache arguments as for kda_cache_write. workspace: uint8 GPU tensor of >=
    kda_cache_attention_workspace_size(...) bytes, or None to have one allocated here for
    this call."""
    import torch
    if q.dim() != 2:
        raise ValueError(f"q must be [T, H_q*128], got {list(q.shape)}")
    T, W = q.shape
    args, n, H, cu = _cache_args(torch, ("q", q), T, (k_cache, v_cache, k_scale, v_scale,
                                                      page_table, kv_lens), cu_seqlens)
    Hq = W // HEAD_DIM
    if W != Hq * HEAD_DIM or Hq < 1 or H < 1 or Hq % H != 0:
        raise ValueError(f"q must be [T, H_q*128] with H_q a multiple of {H}, got {list(q.shape)}")
    bf16 = torch.bfloat16
    qs, os_ = _token_rows("q", q, bf16, T, W), _token_rows("out", out, bf16, T, W)
    ls = 0
    if lse is not None:
        ls = lse.stride()
        if lse.dtype is not torch.float32 or lse.shape != (T, Hq) or (Hq > 1 and ls[1] != 1):
            raise ValueError(f"lse must be a float32 GPU tensor [{T}, {Hq}] with contiguous rows")
        ls = ls[0]
    if (cu is None) != (cu_seqlens_host is None):
        raise ValueError("cu_seqlens and cu_seqlens_host go together")
    host = None
    if cu is not None:
        if cu_seqlens_host.dtype is not torch.int32 or cu_seqlens_host.is_cuda or \
                not cu_seqlens_host.is_contiguous() or cu_seqlens_host.shape != (n + 1,):
            raise ValueError(f"cu_seqlens_host must be a contiguous int32 CPU tensor [{n + 1}]")
        host = cu_seqlens_host.data_ptr()
    dev = _same_device(q, (("out", out), ("lse", lse), ("workspace", workspace)))
    if workspace is None and T > 0:
        workspace = _workspace(kda_cache_attention_workspace_size(n, T, Hq, H), dev, stream)
    ws_bytes = _workspace_bytes(workspace, dev)
    _launch("kda_cache_attention", dev, stream, n, T, Hq, H, HEAD_DIM, host, cu, q.data_ptr(), qs,
            *args, float(scale), out.data_ptr(), os_, _adr(lse), ls, _adr(workspace), ws_bytes)
