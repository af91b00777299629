"""What the attention calls take besides their sizes."""
import inspect
import types

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import attention


def test_packed_calls_without_queries_want_a_status_word():
    """Their tables are checked on the device, and reported there."""
    for size in (kla.kla_attn_fwd_varlen_workspace_size, kla.kla_attn_bwd_varlen_workspace_size):
        assert size(2, 0, 40, 4, 2, 64) == size(2, 0, 0, 4, 2, 128) == 256
        assert size(0, 0, 0, 4, 2, 64) == 0
    for size in (kla.kla_attn_fwd_workspace_size, kla.kla_attn_bwd_workspace_size):
        assert size(2, 0, 40, 4, 2, 64) == size(0, 5, 5, 4, 2, 64) == 0


@pytest.mark.parametrize("name", ["kla_attn", "kla_attn_fwd", "kla_attn_bwd",
                                  "kla_attn_fwd_varlen", "kla_attn_bwd_varlen"])
def test_every_call_can_check_its_status(name):
    assert inspect.signature(getattr(kla, name)).parameters["check_status"].default is False


def test_a_stream_of_another_device_is_refused():
    """It would be replaced by the current stream of the tensors' device."""
    stream = types.SimpleNamespace(cuda_stream=1, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        attention._given(stream, types.SimpleNamespace(device=torch.device("cuda", 0)))


@pytest.mark.parametrize("dims", [3, 4])
def test_a_table_of_the_keys_alone_is_refused(dims):
    """A batch would be taken without it."""
    x = torch.zeros(*([1] * (dims - 3)), 4, 2, 64)
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        kla.kla_attn(x, x, x, cu_seqlens_k=torch.tensor([0, 4]).int())
