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
from torch.autograd.function import once_differentiable

from .binding import KlaError, load

_NORMS = {"none": 0, "rms": 1, "l2": 2}
_STYLES = {"half": 0, "pairs": 1}
_TYPES = {torch.float32: 0, torch.bfloat16: 1}

# A small call takes about as long as its checks do, so these go straight: no
# object is made that the library call does not take.


def _type_code(q):
    code = _TYPES.get(q.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {q.dtype}; use bfloat16 or float32")
    return code


def _refuse(t, name, dtype, device, shape):
    """Says what is wrong with a tensor that is not as it has to be."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name, dtype, device, shape):
    """Checks a [..., H, d] tensor whose token rows may be a stride apart;
    returns that stride in elements."""
    size = t.shape
    if t.dtype != dtype or t.get_device() != device or device < 0 or size != shape:
        _refuse(t, name, dtype, device, shape)
    if t.is_contiguous():
        return size[-2] * size[-1]
    st = t.stride()
    if (size[-1] > 1 and st[-1] != 1) or (size[-2] > 1 and st[-2] != size[-1]):
        raise ValueError(f"{name}: the heads of a token row must be dense (strides {st})")
    if len(size) == 3:
        return st[0] if size[0] > 1 else size[-2] * size[-1]
    row, step = None, None               # the leading dimensions walk one row at a time
    for n, x in zip(reversed(size[:-2]), reversed(st[:-2])):
        if n == 1:
            continue
        if row is None:
            row = x
        elif x != step:
            raise ValueError(f"{name}: the token rows must be evenly spaced (strides {st})")
        step = x * n
    return size[-2] * size[-1] if row is None else row


def _dense(t, name, dtype, device, shape):
    """Checks a dense tensor; returns its address (None: None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != device or t.shape != shape:
        _refuse(t, name, dtype, device, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _given(stream, t):
    """A caller's stream (a torch stream or a handle) made current, so that
    what a call allocates belongs to the stream that uses it."""
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if stream
                  else torch.cuda.default_stream(t.device))
    elif stream.device != t.device:
        raise ValueError(f"stream must be one of {t.device}, got one of {stream.device}")
    return torch.cuda.stream(stream)


def _call(device, fn, *args):
    """Runs a library call with the tensors' device current and its stream
    last in the arguments; raises on a non-OK status."""
    if torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            return _call(device, fn, *args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if status:
        lib = load()
        raise KlaError(status, lib.kla_last_error_message().decode() or
                       lib.kla_status_str(status).decode())


def _workspace(device, size, args, t, workspace):
    """The workspace that the library asks for, on t's device: its address and
    size in bytes."""
    if torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            return _workspace(device, size, args, t, workspace)
    need = size(*args)
    if workspace is None:
        # kept by the caller's variable until the call is enqueued
        return torch.empty(need, dtype=torch.uint8, device=t.device) if need else None, need
    have = workspace.numel() * workspace.element_size()
    if workspace.get_device() != device:
        raise ValueError(f"workspace must be on cuda:{device}, got {workspace.device}")
    if have < need:
        raise ValueError(f"workspace needs {need} bytes")
    return workspace, have


def _at(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=64)
def _sections(sections):
    return (ctypes.c_int * len(sections))(*sections)


def _option(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return table[value]


def _conditioning(q, k, positions, inv_freq, wq, wk, sections, norm_q, norm_k, style):
    """The checks that forward and backward share; returns the arguments up to
    the outputs and those behind them."""
    dt, dev, kind = _type_code(q), q.get_device(), q.dtype
    shape = q.shape
    if len(shape) < 3:
        raise ValueError(f"q must have shape [..., heads, d], got {tuple(shape)}")
    lead, hq, d = shape[:-2], shape[-2], shape[-1]
    qs, hk, ks = _rows(q, "q", kind, dev, shape), 0, 0
    if k is not None:
        hk = k.shape[-2] if k.dim() > 1 else 0
        ks = _rows(k, "k", kind, dev, lead + (hk, d))
    elif wk is not None:
        raise ValueError("wk needs k")
    w = (d,)
    pairs, sec, axes, pos, freq = 0, None, 1, None, None
    if inv_freq is not None and inv_freq.numel():
        pairs = inv_freq.numel()
        sec = (pairs,) if sections is None else tuple(sections)
        axes = len(sec)
        sec = _sections(sec)
        freq = _dense(inv_freq, "inv_freq", torch.float32, dev, (pairs,))
        if positions is None:
            raise ValueError("inv_freq needs positions")
        one = axes == 1 and positions.shape == lead
        pos = _dense(positions, "positions", torch.int32, dev, lead if one else (axes, *lead))
    ins = (q.data_ptr(), qs, _at(k), ks, _dense(wq, "wq", torch.float32, dev, w),
           _dense(wk, "wk", torch.float32, dev, w), pos, freq)
    end = (lead.numel(), hq, hk, d, 2 * pairs, sec, axes, _option(_STYLES, style, "style"),
           _option(_NORMS, norm_q, "norm_q"), _option(_NORMS, norm_k, "norm_k"))
    return dev, dt, ins, end


def _new(shape, dtype, like):
    """A dense tensor on like's device."""
    if like.is_contiguous() and like.dtype == dtype and like.shape == shape:
        return torch.empty_like(like)            # the quicker call
    return torch.empty(shape, dtype=dtype, device=like.device)


def _out_rows(t, name, like):
    """An output of like's shape, made dense where there is none; with its row
    stride."""
    shape = like.shape
    if t is None:
        return _new(shape, like.dtype, like), shape[-2] * shape[-1]
    return t, _rows(t, name, like.dtype, like.get_device(), shape)


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
    if stream is not None:
        with _given(stream, q):
            return kla_qk_norm_rope_fwd(q, k, positions, inv_freq, wq, wk, eps, norm_q, norm_k,
                                        sections, style, q_out, k_out)
    dev, dt, ins, end = _conditioning(q, k, positions, inv_freq, wq, wk, sections, norm_q,
                                      norm_k, style)
    q_out, qo = _out_rows(q_out, "q_out", q)
    ko = 0
    if k is None:
        k_out = None
    else:
        k_out, ko = _out_rows(k_out, "k_out", k)
    _call(dev, load().kla_qk_norm_rope_fwd, *ins, q_out.data_ptr(), qo, _at(k_out), ko,
          *end, eps, dt)
    return q_out, k_out


def kla_qk_norm_rope_bwd_workspace_size(tokens, Hq, Hk, d) -> int:
    return int(load().kla_qk_norm_rope_bwd_workspace_size(tokens, Hq, Hk, d))


def kla_qk_norm_rope_bwd(q, k, positions, inv_freq, dq_out, dk_out, wq=None, wk=None, eps=1e-6,
                         norm_q="rms", norm_k="rms", sections=None, style="half", dq=None,
                         dk=None, workspace=None, stream=None):
    """Backward of kla_qk_norm_rope_fwd on the same inputs: dq_out, dk_out are
    the gradients of its outputs.  Returns (dq, dk, dwq, dwk), None for what is
    not there (k, a weight)."""
    if stream is not None:
        with _given(stream, q):
            return kla_qk_norm_rope_bwd(q, k, positions, inv_freq, dq_out, dk_out, wq, wk, eps,
                                        norm_q, norm_k, sections, style, dq, dk, workspace)
    dev, dt, ins, end = _conditioning(q, k, positions, inv_freq, wq, wk, sections, norm_q,
                                      norm_k, style)
    gqs = _rows(dq_out, "dq_out", q.dtype, dev, q.shape)
    dq, dqs = _out_rows(dq, "dq", q)
    gks = dks = 0
    if k is None:
        dk_out = dk = None
    elif dk_out is None:
        raise ValueError("dk_out must be given with k")
    else:
        gks = _rows(dk_out, "dk_out", q.dtype, dev, k.shape)
        dk, dks = _out_rows(dk, "dk", k)
    dwq = None if wq is None else torch.empty_like(wq)
    dwk = None if wk is None else torch.empty_like(wk)
    lib, wsb = load(), 0
    if dwq is not None or dwk is not None:
        workspace, wsb = _workspace(dev, lib.kla_qk_norm_rope_bwd_workspace_size, end[:4], q,
                                    workspace)
    else:
        workspace = None
    _call(dev, lib.kla_qk_norm_rope_bwd, *ins, dq_out.data_ptr(), gqs, _at(dk_out), gks,
          dq.data_ptr(), dqs, _at(dk), dks, _at(dwq), _at(dwk), *end, eps, dt, _at(workspace),
          wsb)
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
    @once_differentiable
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
    """Checks q, k, v of `dims` dimensions; returns the device, the dtype code,
    their addresses and row strides, and (Hq, Hk, d)."""
    if q.dim() != dims or k.dim() != dims:
        raise ValueError(f"q and k must have {dims} dimensions, got {tuple(q.shape)} and "
                         f"{tuple(k.shape)}")
    dt, dev, kind = _type_code(q), q.get_device(), q.dtype
    qs, hq, d = _rows(q, "q", kind, dev, q.shape), q.shape[-2], q.shape[-1]
    nk, hk = k.shape[-3], k.shape[-2]
    shape = (q.shape[0], nk, hk, d) if dims == 4 else (nk, hk, d)
    ks, vs = _rows(k, "k", kind, dev, shape), _rows(v, "v", kind, dev, shape)
    return dev, dt, (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs), (hq, hk, d)


def _out(t, name, shape, dtype, like):
    """A dense output, made where there is none; and its address."""
    if t is None:
        t = _new(shape, dtype, like)
        return t, t.data_ptr()
    return t, _dense(t, name, dtype, like.get_device(), shape)


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else scale


def kla_attn_fwd(q, k, v, scale=None, k_lens=None, o=None, lse=None, return_lse=True,
                 workspace=None, stream=None, check_status=False):
    """Causal attention with grouped heads.  q: [B,Tq,Hq,d], k, v: [B,Tk,Hk,d];
    query i sees the keys j <= i + Tk - Tq (one token over a cache: Tq = 1);
    k_lens: int32 [B], the keys of each sequence of a padded cache, or None
    (all Tk); scale: 1/sqrt(d) unless given; check_status waits for the call and
    raises what the device reports.  Returns (o, lse), o dense, lse [B,Tq,Hq]
    fp32 (None with return_lse=False)."""
    if stream is not None:
        with _given(stream, q):
            return kla_attn_fwd(q, k, v, scale, k_lens, o, lse, return_lse, workspace,
                                check_status=check_status)
    dev, dt, rows, (hq, hk, d) = _qkv(q, k, v, 4)
    B, Tq, Tk = q.shape[0], q.shape[1], k.shape[1]
    lens = _dense(k_lens, "k_lens", torch.int32, dev, (B,))
    o, at = _out(o, "o", q.shape, q.dtype, q)
    stats = None
    if return_lse or lse is not None:
        lse, stats = _out(lse, "lse", (B, Tq, hq), torch.float32, q)
    lib, sizes = load(), (B, Tq, Tk, hq, hk, d, dt)
    workspace, wsb = _workspace(dev, lib.kla_attn_fwd_workspace_size, sizes, q, workspace)
    _call(dev, lib.kla_attn_fwd, *rows, lens, _scale(scale, d), at, stats, *sizes,
          _at(workspace), wsb)
    if check_status:
        _call(dev, _status, workspace, wsb)
    return o, lse


def _tables(q, dev, cu_q, cu_k):
    n = cu_q.numel()
    if n < 1:
        raise ValueError("cu_seqlens_q must have N + 1 entries")
    at = _dense(cu_q, "cu_seqlens_q", torch.int32, dev, (n,))
    return at, at if cu_k is None else _dense(cu_k, "cu_seqlens_k", torch.int32, dev, (n,)), n - 1


def kla_attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k=None, scale=None, o=None, lse=None,
                        return_lse=True, workspace=None, stream=None, check_status=False):
    """kla_attn_fwd over packed sequences: q [total_q,Hq,d], k, v [total_k,Hk,d],
    cu_seqlens_q, cu_seqlens_k: int32 [N+1] on the device (cu_seqlens_k None:
    the same table).  Returns (o, lse)."""
    if stream is not None:
        with _given(stream, q):
            return kla_attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, scale, o, lse,
                                       return_lse, workspace, check_status=check_status)
    dev, dt, rows, (hq, hk, d) = _qkv(q, k, v, 3)
    cu_q, cu_k, N = _tables(q, dev, cu_seqlens_q, cu_seqlens_k)
    o, at = _out(o, "o", q.shape, q.dtype, q)
    stats = None
    if return_lse or lse is not None:
        lse, stats = _out(lse, "lse", q.shape[:-1], torch.float32, q)
    lib, sizes = load(), (N, q.shape[0], k.shape[0], hq, hk, d, dt)
    workspace, wsb = _workspace(dev, lib.kla_attn_fwd_varlen_workspace_size, sizes, q, workspace)
    _call(dev, lib.kla_attn_fwd_varlen, *rows, cu_q, cu_k, _scale(scale, d), at, stats,
          *sizes, _at(workspace), wsb)
    if check_status:
        _call(dev, _status, workspace, wsb)
    return o, lse


def _status(workspace, wsb, stream):
    return load().kla_workspace_status(_at(workspace), wsb, stream)


def _grads(q, k, v, o, lse, d_o, dev, dq, dk, dv):
    """Checks what the backward takes and makes what it writes: the arguments
    of the forward's results and of the gradients, and those."""
    gs = _rows(d_o, "d_o", q.dtype, dev, q.shape)
    ins = (_dense(o, "o", q.dtype, dev, q.shape),
           _dense(lse, "lse", torch.float32, dev, q.shape[:-1]), d_o.data_ptr(), gs)
    dq, a = _out(dq, "dq", q.shape, q.dtype, q)
    dk, b = _out(dk, "dk", k.shape, q.dtype, k)
    dv, c = _out(dv, "dv", v.shape, q.dtype, v)
    return ins, (a, b, c), (dq, dk, dv)


def kla_attn_bwd(q, k, v, o, lse, d_o, scale=None, dq=None, dk=None, dv=None, workspace=None,
                 stream=None, check_status=False):
    """Backward of kla_attn_fwd (without k_lens): the gradients of sum <d_o, o>
    from the forward's inputs and its o and lse.  Returns (dq, dk, dv), dense."""
    if stream is not None:
        with _given(stream, q):
            return kla_attn_bwd(q, k, v, o, lse, d_o, scale, dq, dk, dv, workspace,
                                check_status=check_status)
    dev, dt, rows, (hq, hk, d) = _qkv(q, k, v, 4)
    ins, at, grads = _grads(q, k, v, o, lse, d_o, dev, dq, dk, dv)
    lib, sizes = load(), (q.shape[0], q.shape[1], k.shape[1], hq, hk, d, dt)
    workspace, wsb = _workspace(dev, lib.kla_attn_bwd_workspace_size, sizes, q, workspace)
    _call(dev, lib.kla_attn_bwd, *rows, *ins, _scale(scale, d), *at, *sizes,
          _at(workspace), wsb)
    if check_status:
        _call(dev, _status, workspace, wsb)
    return grads


def kla_attn_bwd_varlen(q, k, v, o, lse, d_o, cu_seqlens_q, cu_seqlens_k=None, scale=None,
                        dq=None, dk=None, dv=None, workspace=None, stream=None,
                        check_status=False):
    """Backward of kla_attn_fwd_varlen; otherwise as kla_attn_bwd."""
    if stream is not None:
        with _given(stream, q):
            return kla_attn_bwd_varlen(q, k, v, o, lse, d_o, cu_seqlens_q, cu_seqlens_k, scale,
                                       dq, dk, dv, workspace, check_status=check_status)
    dev, dt, rows, (hq, hk, d) = _qkv(q, k, v, 3)
    cu_q, cu_k, N = _tables(q, dev, cu_seqlens_q, cu_seqlens_k)
    ins, at, grads = _grads(q, k, v, o, lse, d_o, dev, dq, dk, dv)
    lib, sizes = load(), (N, q.shape[0], k.shape[0], hq, hk, d, dt)
    workspace, wsb = _workspace(dev, lib.kla_attn_bwd_varlen_workspace_size, sizes, q, workspace)
    _call(dev, lib.kla_attn_bwd_varlen, *rows, *ins, cu_q, cu_k, _scale(scale, d), *at,
          *sizes, _at(workspace), wsb)
    if check_status:
        _call(dev, _status, workspace, wsb)
    return grads


class _KlaAttn(torch.autograd.Function):
    """Causal attention under autograd: kla_attn_fwd[_varlen] and its backward."""

    @staticmethod
    def forward(ctx, q, k, v, scale, cu_q, cu_k, check):
        if cu_q is None:
            o, lse = kla_attn_fwd(q, k, v, scale, check_status=check)
        else:
            o, lse = kla_attn_fwd_varlen(q, k, v, cu_q, cu_k, scale, check_status=check)
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        ctx.scale, ctx.check = scale, check
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        d_o = _dense_rows(d_o, o)
        if cu_q is None:
            grads = kla_attn_bwd(q, k, v, o, lse, d_o, ctx.scale, check_status=ctx.check)
        else:
            grads = kla_attn_bwd_varlen(q, k, v, o, lse, d_o, cu_q, cu_k, ctx.scale,
                                        check_status=ctx.check)
        return *grads, None, None, None, None


def kla_attn(q, k, v, scale=None, cu_seqlens_q=None, cu_seqlens_k=None, check_status=False):
    """Differentiable causal attention: o, with gradients for q, k and v.  A
    batch [B,T,H,d], or packed sequences [total,H,d] with their tables.
    check_status waits for the forward and the backward and raises what the device
    reports; without it tables that the device refuses leave o and the gradients
    unwritten and unreported.  Forward and backward may be captured into a CUDA
    graph (without check_status); as for every torch operation, no eager graph of
    the same leaves may be alive then."""
    if cu_seqlens_q is None and cu_seqlens_k is not None:
        raise ValueError("cu_seqlens_k needs cu_seqlens_q")
    return _KlaAttn.apply(q, k, v, scale, cu_seqlens_q, cu_seqlens_k, check_status)
