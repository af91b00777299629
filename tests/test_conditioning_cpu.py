"""Query and key conditioning: what the host refuses, before any device work."""
import ctypes

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="uses fake device pointers; host validation only")
FAKE = 0x10000


def _fwd(**over):
    a = dict(q=FAKE, qs=256, k=FAKE, ks=128, wq=None, wk=None, pos=FAKE, freq=FAKE, qo=FAKE,
             qos=256, ko=FAKE, kos=128, tokens=3, Hq=4, Hk=2, d=64, rot=32, sec=(16,), axes=1,
             style=0, nq=1, nk=1, eps=1e-6, dtype=1)
    a.update(over)
    sec = None if a["sec"] is None else (ctypes.c_int * len(a["sec"]))(*a["sec"])
    return binding.load().kla_qk_norm_rope_fwd(
        a["q"], a["qs"], a["k"], a["ks"], a["wq"], a["wk"], a["pos"], a["freq"], a["qo"],
        a["qos"], a["ko"], a["kos"], a["tokens"], a["Hq"], a["Hk"], a["d"], a["rot"], sec,
        a["axes"], a["style"], a["nq"], a["nk"], a["eps"], a["dtype"], None)


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(d=96), binding.KLA_ERR_UNSUPPORTED),
    (dict(rot=24, sec=(12,)), binding.KLA_ERR_UNSUPPORTED),
    (dict(rot=80, sec=(40,)), binding.KLA_ERR_UNSUPPORTED),
    (dict(Hq=2000, qs=128000, qos=128000), binding.KLA_ERR_UNSUPPORTED),
    (dict(tokens=-1), binding.KLA_ERR_INVALID_ARG),
    (dict(Hq=0), binding.KLA_ERR_INVALID_ARG),
    (dict(dtype=2), binding.KLA_ERR_INVALID_ARG),
    (dict(style=2), binding.KLA_ERR_INVALID_ARG),
    (dict(nq=3), binding.KLA_ERR_INVALID_ARG),
    (dict(nk=-1), binding.KLA_ERR_INVALID_ARG),
    (dict(eps=-1.0), binding.KLA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), binding.KLA_ERR_INVALID_ARG),
    (dict(sec=(8, 7), axes=2), binding.KLA_ERR_INVALID_ARG),
    (dict(sec=(17, -1), axes=2), binding.KLA_ERR_INVALID_ARG),
    (dict(sec=(4, 4, 4, 2, 2), axes=5), binding.KLA_ERR_INVALID_ARG),
    (dict(sec=None), binding.KLA_ERR_INVALID_ARG),
    (dict(q=None), binding.KLA_ERR_INVALID_ARG),
    (dict(ko=None), binding.KLA_ERR_INVALID_ARG),
    (dict(pos=None), binding.KLA_ERR_INVALID_ARG),
    (dict(freq=None), binding.KLA_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), binding.KLA_ERR_INVALID_ARG),
    (dict(wq=FAKE + 4), binding.KLA_ERR_INVALID_ARG),
    (dict(pos=FAKE + 2), binding.KLA_ERR_INVALID_ARG),
    (dict(qs=252), binding.KLA_ERR_INVALID_ARG),
    (dict(qs=260), binding.KLA_ERR_INVALID_ARG),
])
def test_forward_refuses(over, status):
    assert _fwd(**over) == status
    assert binding.load().kla_last_error_message().decode() != ""


@no_gpu_only
def test_no_tokens_and_the_injected_fault(monkeypatch):
    assert _fwd(tokens=0, q=None) == binding.KLA_OK
    monkeypatch.setenv("KLA_FAULT_INJECT", "launch")
    assert _fwd() == binding.KLA_ERR_CUDA


@no_gpu_only
def test_backward_refuses():
    lib = binding.load()
    sec = (ctypes.c_int * 1)(16)

    def call(wq=FAKE, wk=FAKE, dwq=FAKE, dwk=FAKE, g=FAKE, dq=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.kla_qk_norm_rope_bwd(FAKE, 256, FAKE, 128, wq, wk, FAKE, FAKE, g, 256, FAKE,
                                        128, dq, 256, FAKE, 128, dwq, dwk, 3, 4, 2, 64, 32, sec,
                                        1, 0, 1, 1, 1e-6, 1, ws, wsb, None)

    assert call(wq=None) == binding.KLA_ERR_INVALID_ARG
    assert call(dwk=FAKE + 2) == binding.KLA_ERR_INVALID_ARG
    assert call(g=None) == binding.KLA_ERR_INVALID_ARG
    assert call(dq=FAKE + 8) == binding.KLA_ERR_INVALID_ARG
    assert call(ws=None) == binding.KLA_ERR_WORKSPACE
    assert call(wsb=255) == binding.KLA_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == binding.KLA_ERR_INVALID_ARG
    assert lib.kla_qk_norm_rope_bwd_workspace_size(3, 4, 2, 64) >= 2 * 64 * 4
    assert lib.kla_qk_norm_rope_bwd_workspace_size(3, 4, 2, 96) == 0


def test_the_binding_refuses_cpu_tensors_and_unknown_options():
    q = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        kla.kla_qk_norm_rope_fwd(q, None, None, None)
    with pytest.raises(TypeError):
        kla.kla_qk_norm_rope_fwd(q.half(), None, None, None)
