"""Binding of the softmax-attention side of a hybrid stack: query and key
conditioning (a norm per head and the rotary positions) and causal attention.

The same rules as in ``binding``: argument marshalling only, every step runs
in the CUDA library, a non-OK status raises ``KlaError``.  Two differences:
q, k and v may be views whose token rows lie a stride apart (the parts of a
fused projection's output) as long as the heads of a row are dense, and a call
runs on the device of its tensors, whichever is current.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from .binding import _check, _dtype_code, _ptr, _workspace, load

_NORMS = {"none": 0, "rms": 1, "l2": 2}
_STYLES = {"half": 0, "pairs": 1}


def _rows(t, name, like=None, lead=None, heads=None, d=None):
    """Checks a [..., H, d] tensor whose token rows may be a stride apart;
    returns that stride in elements."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() < 3:
        raise ValueError(f"{name} must have shape [..., heads, d], got {tuple(t.shape)}")
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    shape = tuple(t.shape)
    if (lead is not None and shape[:-2] != tuple(lead)) or \
            (heads is not None and shape[-2] != heads) or (d is not None and shape[-1] != d):
        raise ValueError(f"{name} must have shape {tuple(lead or shape[:-2])} + "
                         f"({heads or shape[-2]}, {d or shape[-1]}), got {shape}")
    dense = shape[-2] * shape[-1]
    if t.is_contiguous():
        return dense
    st = t.stride()
    if (shape[-1] > 1 and st[-1] != 1) or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError(f"{name}: the heads of a token row must be dense (strides {st})")
    row, step = None, None               # the leading dimensions walk one row at a time
    for n, s in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if n == 1:
            continue
        if row is None:
            row, step = s, s
        elif s != step:
            raise ValueError(f"{name}: the token rows must be evenly spaced (strides {st})")
        step = s * n
    return dense if row is None else row


def _need(t, name, device, dtype, shape):
    """Checks a dense tensor (or None)."""
    if t is None:
        return
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _call(device, stream, fn, *args):
    """Runs a library call with the tensors' device current and its stream
    last in the arguments; raises on a non-OK status."""
    with _device(device):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        _check(fn(*args, ctypes.c_void_p(s)))


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *a):
        return False


_nothing = _Nothing()


def _device(device):
    return _nothing if torch.cuda.current_device() == device.index else torch.cuda.device(device)


@functools.lru_cache(maxsize=64)
def _sections(sections):
    return (ctypes.c_int * len(sections))(*sections)


def _option(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return table[value]


def _conditioning(q, k, positions, inv_freq, wq, wk, sections, norm_q, norm_k, style):
    """The checks that forward and backward share."""
    dt = _dtype_code(q)
    qs = _rows(q, "q")
    lead, (hq, d) = q.shape[:-2], q.shape[-2:]
    hk, ks = 0, 0
    if k is not None:
        ks = _rows(k, "k", q, lead, None, d)
        hk = k.shape[-2]
    elif wk is not None:
        raise ValueError("wk needs k")
    _need(wq, "wq", q.device, torch.float32, (d,))
    _need(wk, "wk", q.device, torch.float32, (d,))
    pairs = 0 if inv_freq is None else inv_freq.numel()
    tokens = math.prod(lead)
    axes = 1
    if pairs:
        sections = (pairs,) if sections is None else tuple(int(n) for n in sections)
        axes = len(sections)
        _need(inv_freq, "inv_freq", q.device, torch.float32, (pairs,))
        if positions is None:
            raise ValueError("inv_freq needs positions")
        one = axes == 1 and tuple(positions.shape) == tuple(lead)
        _need(positions, "positions", q.device, torch.int32, lead if one else (axes, *lead))
    return (dt, qs, ks, tokens, hq, hk, d, 2 * pairs, _sections(sections) if pairs else None, axes,
            _option(_STYLES, style, "style"), _option(_NORMS, norm_q, "norm_q"),
            _option(_NORMS, norm_k, "norm_k"))


def kla_qk_norm_rope_fwd(q, k, positions, inv_freq, wq=None, wk=None, eps=1e-6, norm_q="rms",
                         norm_k="rms", sections=None, style="half", q_out=None, k_out=None,
                         stream=None):
    """A norm of every head's row of q and k and the rotary positions, in one
    pass.  q: [..., Hq, d], k: [..., Hk, d] or None (q alone), views of a fused
    projection's output among them; positions: int32 [...] or [n_axes, ...];
    inv_freq: [rot/2] fp32 radians per position (None: norm only), the first
    sections[0] pairs on axis 0 and so on; wq, wk: [d] fp32 or None; norm_q,
    norm_k: "rms", "l2" or "none"; style "half" (features i, i + rot/2) or
    "pairs" (2i, 2i + 1).  q_out, k_out may be q and k (in place).  Returns
    (q_out, k_out)."""
    dt, qs, ks, n, hq, hk, d, rot, sec, axes, st, nq, nk = _conditioning(
        q, k, positions, inv_freq, wq, wk, sections, norm_q, norm_k, style)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    qo = _rows(q_out, "q_out", q, q.shape[:-2], hq, d)
    ko = 0
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        ko = _rows(k_out, "k_out", q, k.shape[:-2], hk, d)
    _call(q.device, stream, load().kla_qk_norm_rope_fwd, _ptr(q), qs, _ptr(k), ks, _ptr(wq),
          _ptr(wk), _ptr(positions), _ptr(inv_freq), _ptr(q_out), qo, _ptr(k_out), ko, n, hq, hk,
          d, rot, sec, axes, st, nq, nk, float(eps), dt)
    return q_out, k_out


def kla_qk_norm_rope_bwd_workspace_size(tokens, Hq, Hk, d) -> int:
    return int(load().kla_qk_norm_rope_bwd_workspace_size(tokens, Hq, Hk, d))


def kla_qk_norm_rope_bwd(q, k, positions, inv_freq, dq_out, dk_out, wq=None, wk=None, eps=1e-6,
                         norm_q="rms", norm_k="rms", sections=None, style="half", dq=None,
                         dk=None, workspace=None, stream=None):
    """Backward of kla_qk_norm_rope_fwd on the same inputs: dq_out, dk_out are
    the gradients of its outputs.  Returns (dq, dk, dwq, dwk), None for what is
    not there (k, a weight)."""
    dt, qs, ks, n, hq, hk, d, rot, sec, axes, st, nq, nk = _conditioning(
        q, k, positions, inv_freq, wq, wk, sections, norm_q, norm_k, style)
    gqs = _rows(dq_out, "dq_out", q, q.shape[:-2], hq, d)
    if dq is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dqs = _rows(dq, "dq", q, q.shape[:-2], hq, d)
    gks = dks = 0
    if k is not None:
        gks = _rows(dk_out, "dk_out", q, k.shape[:-2], hk, d)
        if dk is None:
            dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dks = _rows(dk, "dk", q, k.shape[:-2], hk, d)
    else:
        dk_out = dk = None
    dwq = None if wq is None else torch.empty_like(wq)
    dwk = None if wk is None else torch.empty_like(wk)
    need = 0
    if dwq is not None or dwk is not None:
        need = kla_qk_norm_rope_bwd_workspace_size(n, hq, hk, d)
    workspace, wsb = _workspace(need, q.device, workspace)
    _call(q.device, stream, load().kla_qk_norm_rope_bwd, _ptr(q), qs, _ptr(k), ks, _ptr(wq),
          _ptr(wk), _ptr(positions), _ptr(inv_freq), _ptr(dq_out), gqs, _ptr(dk_out), gks,
          _ptr(dq), dqs, _ptr(dk), dks, _ptr(dwq), _ptr(dwk), n, hq, hk, d, rot, sec, axes, st,
          nq, nk, float(eps), dt, _ptr(workspace), wsb)
    return dq, dk, dwq, dwk


def _dense_rows(g, like):
    """A gradient as the library takes it: the type of `like`, rows of dense heads."""
    if g is None:
        return torch.zeros(like.shape, dtype=like.dtype, device=like.device)
    return g.to(like.dtype).contiguous()


class _QkNormRope(torch.autograd.Function):
    """kla_qk_norm_rope_fwd under autograd: its backward is kla_qk_norm_rope_bwd."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, wq, wk, how):
        out = kla_qk_norm_rope_fwd(q, k, positions, inv_freq, wq, wk, **how)
        ctx.save_for_backward(q, k, positions, inv_freq, wq, wk)
        ctx.how = how
        return out if k is not None else out[0]

    @staticmethod
    def backward(ctx, *grads):
        q, k, positions, inv_freq, wq, wk = ctx.saved_tensors
        gk = None if k is None else _dense_rows(grads[1], k)
        dq, dk, dwq, dwk = kla_qk_norm_rope_bwd(q, k, positions, inv_freq,
                                                _dense_rows(grads[0], q), gk, wq, wk, **ctx.how)
        return dq, dk, None, None, dwq, dwk, None


def kla_qk_norm_rope(q, k, positions, inv_freq, wq=None, wk=None, eps=1e-6, norm_q="rms",
                     norm_k="rms", sections=None, style="half"):
    """Differentiable kla_qk_norm_rope_fwd: (q_out, k_out), or q_out alone where
    k is None, with gradients for q, k, wq and wk."""
    how = dict(eps=float(eps), norm_q=norm_q, norm_k=norm_k, sections=sections, style=style)
    return _QkNormRope.apply(q, k, positions, inv_freq, wq, wk, how)


# ------------------------------------------------------------------ attention
def kla_attn_fwd_workspace_size(B, Tq, Tk, Hq, Hk, d, dtype=1) -> int:
    return int(load().kla_attn_fwd_workspace_size(B, Tq, Tk, Hq, Hk, d, dtype))


def kla_attn_fwd_varlen_workspace_size(N, total_q, total_k, Hq, Hk, d, dtype=1) -> int:
    return int(load().kla_attn_fwd_varlen_workspace_size(N, total_q, total_k, Hq, Hk, d, dtype))


def kla_attn_bwd_workspace_size(B, Tq, Tk, Hq, Hk, d, dtype=1) -> int:
    return int(load().kla_attn_bwd_workspace_size(B, Tq, Tk, Hq, Hk, d, dtype))


def kla_attn_bwd_varlen_workspace_size(N, total_q, total_k, Hq, Hk, d, dtype=1) -> int:
    return int(load().kla_attn_bwd_varlen_workspace_size(N, total_q, total_k, Hq, Hk, d, dtype))


def _qkv(q, k, v, dims):
    """Checks q, k, v of `dims` dimensions; returns their row strides, the
    dtype code and (Hq, Hk, d)."""
    if q.dim() != dims:
        raise ValueError(f"q must have {dims} dimensions, got {tuple(q.shape)}")
    dt = _dtype_code(q)
    qs = _rows(q, "q")
    hq, d = q.shape[-2:]
    if k.dim() != dims or (dims == 4 and k.shape[0] != q.shape[0]):
        raise ValueError(f"k must have q's batch, got {tuple(k.shape)}")
    ks = _rows(k, "k", q, None, None, d)
    vs = _rows(v, "v", q, k.shape[:-2], k.shape[-2], d)
    return (_ptr(q), qs, _ptr(k), ks, _ptr(v), vs), dt, (hq, k.shape[-2], d)


def _out(t, name, shape, dtype, device, want=True):
    if t is None and want:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, device, dtype, shape)
    return t


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def kla_attn_fwd(q, k, v, scale=None, k_lens=None, o=None, lse=None, return_lse=True,
                 workspace=None, stream=None):
    """Causal attention with grouped heads.  q: [B,Tq,Hq,d], k, v: [B,Tk,Hk,d];
    query i sees the keys j <= i + Tk - Tq (one token over a cache: Tq = 1);
    k_lens: int32 [B], the keys of each sequence of a padded cache, or None
    (all Tk); scale: 1/sqrt(d) unless given.  Returns (o, lse), o dense, lse
    [B,Tq,Hq] fp32 (None with return_lse=False)."""
    rows, dt, (hq, hk, d) = _qkv(q, k, v, 4)
    B, Tq, Tk = q.shape[0], q.shape[1], k.shape[1]
    _need(k_lens, "k_lens", q.device, torch.int32, (B,))
    o = _out(o, "o", q.shape, q.dtype, q.device)
    lse = _out(lse, "lse", (B, Tq, hq), torch.float32, q.device, return_lse)
    lib = load()
    with _device(q.device):
        need = int(lib.kla_attn_fwd_workspace_size(B, Tq, Tk, hq, hk, d, dt))
    workspace, wsb = _workspace(need, q.device, workspace)
    _call(q.device, stream, lib.kla_attn_fwd, *rows, _ptr(k_lens), _scale(scale, d), _ptr(o),
          _ptr(lse), B, Tq, Tk, hq, hk, d, dt, _ptr(workspace), wsb)
    return o, lse


def _tables(q, cu_q, cu_k):
    if cu_k is None:
        cu_k = cu_q
    _need(cu_q, "cu_seqlens_q", q.device, torch.int32, (cu_q.numel(),))
    _need(cu_k, "cu_seqlens_k", q.device, torch.int32, (cu_q.numel(),))
    if cu_q.numel() < 1:
        raise ValueError("cu_seqlens_q must have N + 1 entries")
    return cu_k, cu_q.numel() - 1


def kla_attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k=None, scale=None, o=None, lse=None,
                        return_lse=True, workspace=None, stream=None, check_status=False):
    """kla_attn_fwd over packed sequences: q [total_q,Hq,d], k, v [total_k,Hk,d],
    cu_seqlens_q, cu_seqlens_k: int32 [N+1] on the device (cu_seqlens_k None:
    the same table).  Returns (o, lse)."""
    rows, dt, (hq, hk, d) = _qkv(q, k, v, 3)
    cu_k, N = _tables(q, cu_seqlens_q, cu_seqlens_k)
    nq, nk = q.shape[0], k.shape[0]
    o = _out(o, "o", q.shape, q.dtype, q.device)
    lse = _out(lse, "lse", (nq, hq), torch.float32, q.device, return_lse)
    lib = load()
    with _device(q.device):
        need = int(lib.kla_attn_fwd_varlen_workspace_size(N, nq, nk, hq, hk, d, dt))
    workspace, wsb = _workspace(need, q.device, workspace)
    _call(q.device, stream, lib.kla_attn_fwd_varlen, *rows, _ptr(cu_seqlens_q), _ptr(cu_k),
          _scale(scale, d), _ptr(o), _ptr(lse), N, nq, nk, hq, hk, d, dt, _ptr(workspace), wsb)
    if check_status:
        _call(q.device, stream, lib.kla_workspace_status, _ptr(workspace), wsb)
    return o, lse


def _grads(q, k, v, o, lse, d_o, dq, dk, dv):
    """Checks what the backward takes and allocates what it writes."""
    gs = _rows(d_o, "d_o", q, q.shape[:-2], *q.shape[-2:])
    _need(o, "o", q.device, q.dtype, q.shape)
    _need(lse, "lse", q.device, torch.float32, q.shape[:-1])
    dq = _out(dq, "dq", q.shape, q.dtype, q.device)
    dk = _out(dk, "dk", k.shape, k.dtype, k.device)
    dv = _out(dv, "dv", v.shape, v.dtype, v.device)
    return gs, dq, dk, dv


def kla_attn_bwd(q, k, v, o, lse, d_o, scale=None, dq=None, dk=None, dv=None, workspace=None,
                 stream=None):
    """Backward of kla_attn_fwd (without k_lens): the gradients of sum <d_o, o>
    from the forward's inputs and its o and lse.  Returns (dq, dk, dv), dense."""
    rows, dt, (hq, hk, d) = _qkv(q, k, v, 4)
    B, Tq, Tk = q.shape[0], q.shape[1], k.shape[1]
    gs, dq, dk, dv = _grads(q, k, v, o, lse, d_o, dq, dk, dv)
    lib = load()
    with _device(q.device):
        need = int(lib.kla_attn_bwd_workspace_size(B, Tq, Tk, hq, hk, d, dt))
    workspace, wsb = _workspace(need, q.device, workspace)
    _call(q.device, stream, lib.kla_attn_bwd, *rows, _ptr(o), _ptr(lse), _ptr(d_o), gs,
          _scale(scale, d), _ptr(dq), _ptr(dk), _ptr(dv), B, Tq, Tk, hq, hk, d, dt,
          _ptr(workspace), wsb)
    return dq, dk, dv


def kla_attn_bwd_varlen(q, k, v, o, lse, d_o, cu_seqlens_q, cu_seqlens_k=None, scale=None,
                        dq=None, dk=None, dv=None, workspace=None, stream=None,
                        check_status=False):
    """Backward of kla_attn_fwd_varlen; otherwise as kla_attn_bwd."""
    rows, dt, (hq, hk, d) = _qkv(q, k, v, 3)
    cu_k, N = _tables(q, cu_seqlens_q, cu_seqlens_k)
    nq, nk = q.shape[0], k.shape[0]
    gs, dq, dk, dv = _grads(q, k, v, o, lse, d_o, dq, dk, dv)
    lib = load()
    with _device(q.device):
        need = int(lib.kla_attn_bwd_varlen_workspace_size(N, nq, nk, hq, hk, d, dt))
    workspace, wsb = _workspace(need, q.device, workspace)
    _call(q.device, stream, lib.kla_attn_bwd_varlen, *rows, _ptr(o), _ptr(lse), _ptr(d_o), gs,
          _ptr(cu_seqlens_q), _ptr(cu_k), _scale(scale, d), _ptr(dq), _ptr(dk), _ptr(dv), N, nq,
          nk, hq, hk, d, dt, _ptr(workspace), wsb)
    if check_status:
        _call(q.device, stream, lib.kla_workspace_status, _ptr(workspace), wsb)
    return dq, dk, dv


class _KlaAttn(torch.autograd.Function):
    """Causal attention under autograd: kla_attn_fwd[_varlen] and its backward."""

    @staticmethod
    def forward(ctx, q, k, v, scale, cu_q, cu_k):
        if cu_q is None:
            o, lse = kla_attn_fwd(q, k, v, scale)
        else:
            o, lse = kla_attn_fwd_varlen(q, k, v, cu_q, cu_k, scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        ctx.scale = scale
        return o

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        d_o = _dense_rows(d_o, o)
        if cu_q is None:
            grads = kla_attn_bwd(q, k, v, o, lse, d_o, ctx.scale)
        else:
            grads = kla_attn_bwd_varlen(q, k, v, o, lse, d_o, cu_q, cu_k, ctx.scale)
        return *grads, None, None, None


def kla_attn(q, k, v, scale=None, cu_seqlens_q=None, cu_seqlens_k=None):
    """Differentiable causal attention: o, with gradients for q, k and v.  A
    batch [B,T,H,d], or packed sequences [total,H,d] with their tables."""
    return _KlaAttn.apply(q, k, v, scale, cu_seqlens_q, cu_seqlens_k)
