"""A workspace that a caller gives: what the bindings refuse before the library sees it."""
import pytest
import torch

from gated_delta_rule_kaczmarz_gb300 import attention, binding, cache


class OnGpu:
    """A tensor that says it is on the first GPU."""

    def __init__(self, t, device=0):
        self.t, self.at = t, device

    def get_device(self):
        return self.at

    @property
    def device(self):
        return torch.device("cuda", self.at) if self.at >= 0 else torch.device("cpu")

    def __getattr__(self, name):
        return getattr(self.t, name)


def _bytes(n):
    return torch.zeros(n, dtype=torch.uint8)


def _calls(monkeypatch, need):
    """Each binding's way to a workspace of `need` bytes: (address, bytes) that the library gets."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    monkeypatch.setattr(cache, "_size", lambda *a: need)

    def of_cache(ws):
        got = []
        cache._run(lambda *a: got.append(a[:2]) or 0, 0, (), "kla_kv4_attn_workspace_size", (), ws, False)
        return got[0]

    def of_attention(ws):
        t, size = attention._workspace(0, lambda *a: need, (), OnGpu(_bytes(1)), ws)
        return t.data_ptr(), size

    def of_binding(ws):
        t, size = binding._workspace(need, torch.device("cuda", 0), ws)
        return t.data_ptr(), size

    return dict(cache=of_cache, attention=of_attention, binding=of_binding)


@pytest.mark.parametrize("need", [512, 0])
@pytest.mark.parametrize("name", ["cache", "attention", "binding"])
def test_workspaces_that_are_not_dense(name, need, monkeypatch):
    """An expanded view has one byte behind all of its elements, every second byte belongs to
    somebody else: neither reaches the library."""
    call = _calls(monkeypatch, need)[name]
    dense = _bytes(1024)
    assert call(OnGpu(dense)) == (dense.data_ptr(), 1024)
    for bad in (_bytes(1).expand(1024), _bytes(2048)[::2], _bytes(32).view(1, 32).expand(32, 32)):
        with pytest.raises(ValueError, match="contiguous"):
            call(OnGpu(bad))


@pytest.mark.parametrize("need", [512, 0])
@pytest.mark.parametrize("name", ["cache", "attention", "binding"])
def test_workspaces_on_another_device(name, need, monkeypatch):
    call = _calls(monkeypatch, need)[name]
    for device in (-1, 1):
        with pytest.raises(ValueError, match="cuda:0"):
            call(OnGpu(_bytes(1024), device))
