"""Causal attention: what the host refuses, before any device work, and the
workspaces it asks for."""
import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="uses fake device pointers; host validation only")
FAKE = 0x10000
INVALID, UNSUPPORTED = binding.KLA_ERR_INVALID_ARG, binding.KLA_ERR_UNSUPPORTED
WORKSPACE = binding.KLA_ERR_WORKSPACE
SIZES = dict(q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, scale=0.1, o=FAKE, lse=FAKE, B=2,
             Tq=10, Tk=20, Hq=4, Hk=2, d=64, dtype=1, ws=FAKE, wsb=1 << 40)


def _end(a):
    return a["Hq"], a["Hk"], a["d"], a["dtype"], a["ws"], a["wsb"], None


def _fwd(**over):
    a = {**SIZES, "lens": None, **over}
    return binding.load().kla_attn_fwd(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["lens"], a["scale"], a["o"],
        a["lse"], a["B"], a["Tq"], a["Tk"], *_end(a))


def _packed(**over):
    a = {**SIZES, "cq": FAKE, "ck": FAKE, **over}
    return binding.load().kla_attn_fwd_varlen(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cq"], a["ck"], a["scale"], a["o"],
        a["lse"], a["B"], a["Tq"], a["Tk"], *_end(a))


def _bwd(**over):
    a = {**SIZES, "go": FAKE, "gs": 256, "dq": FAKE, "dk": FAKE, "dv": FAKE, **over}
    return binding.load().kla_attn_bwd(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["o"], a["lse"], a["go"], a["gs"],
        a["scale"], a["dq"], a["dk"], a["dv"], a["B"], a["Tq"], a["Tk"], *_end(a))


SHARED = [
    (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(B=-1), INVALID),
    (dict(Tq=-1), INVALID), (dict(Tk=-2), INVALID), (dict(dtype=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(ks=120), INVALID),
    (dict(vs=132), INVALID), (dict(o=FAKE + 2), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(d=80), UNSUPPORTED), (dict(Hq=2048), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE), (dict(ws=FAKE + 16), INVALID),
]


@no_gpu_only
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(o=None), INVALID), (dict(lens=FAKE + 1), INVALID),
    (dict(B=1 << 16, Tq=1 << 16), UNSUPPORTED), (dict(B=1 << 16, Tk=1 << 16), UNSUPPORTED)])
def test_forward_refuses(over, status):
    assert _fwd(**over) == status
    assert binding.load().kla_last_error_message().decode() != ""


@no_gpu_only
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(cq=None), INVALID), (dict(ck=None), INVALID), (dict(cq=FAKE + 2), INVALID),
    (dict(B=0), INVALID)])
def test_packed_forward_refuses(over, status):
    assert _packed(**over) == status
    assert binding.load().kla_last_error_message().decode() != ""


@no_gpu_only
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(go=None), INVALID), (dict(gs=252), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dv=FAKE + 8), INVALID)])
def test_backward_refuses(over, status):
    assert _bwd(**over) == status
    assert binding.load().kla_last_error_message().decode() != ""


@no_gpu_only
@pytest.mark.parametrize("call", [_fwd, _packed, _bwd])
def test_what_32_bits_do_not_hold_is_refused(call):
    """Rows are counted in 32 bits, a tile past the last; log2 e times the scale
    is finite."""
    most = dict(B=1, Tq=(1 << 31) // 64 - 2, Tk=64, Hq=64, Hk=64, qs=64 * 64, ks=64 * 64, vs=64 * 64,
                gs=64 * 64)
    assert call(**most) == UNSUPPORTED                       # its rows + 128 = 2^31
    assert call(**{**most, "Tq": most["Tq"] - 1}, wsb=64) == WORKSPACE      # not too large
    assert call(scale=2e38, wsb=64) == WORKSPACE and call(scale=3e38) == INVALID


@no_gpu_only
def test_nothing_to_do_and_the_injected_fault(monkeypatch):
    assert _fwd(B=0) == binding.KLA_OK
    assert _fwd(Tq=0, q=None, o=None) == binding.KLA_OK
    assert _packed(B=0, Tq=0, Tk=0, cq=None, ck=None) == binding.KLA_OK
    monkeypatch.setenv("KLA_FAULT_INJECT", "launch")
    assert _fwd() == _bwd() == _packed() == binding.KLA_ERR_CUDA


def test_workspace_sizes():
    size = kla.kla_attn_fwd_workspace_size
    # a prompt that fills the GPU keeps nothing but the status word
    assert size(4, 2048, 2048, 16, 4, 128) == 256
    # one token over a long cache: partial results of every part of the keys
    assert size(1, 1, 32768, 16, 4, 128) >= 256 + 2 * 16 * 128 * 4
    assert size(1, 1, 1, 3, 2, 64) == 0 and size(1, 1, 1, 2, 2, 80) == 0
    assert size(1, 0, 100, 2, 2, 64) == 0
    assert kla.kla_attn_bwd_workspace_size(2, 100, 100, 4, 2, 64) >= 256 + 2 * 100 * 4 * 4
    packed = kla.kla_attn_fwd_varlen_workspace_size(64, 300000, 300000, 16, 4, 128)
    assert 256 < packed < 1 << 22
    assert kla.kla_attn_bwd_varlen_workspace_size(3, 100, 50, 4, 2, 64) > 256


def test_the_binding_refuses():
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        kla.kla_attn_fwd(q, q, q)                  # not on a GPU
    with pytest.raises(ValueError):
        kla.kla_attn_fwd(q[0], q[0], q[0])         # not a batch
    with pytest.raises(TypeError):
        kla.kla_attn_fwd(q.half(), q.half(), q.half())
