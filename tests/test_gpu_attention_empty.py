"""Attention calls without queries: the status word is the call's own, and the
tables of packed sequences are checked as in any other."""
import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _table(*x):
    return torch.tensor(x).int().cuda()


def _sides(keys, d=64):
    q, k = torch.empty(0, 4, d, dtype=BF16, device="cuda"), torch.randn(keys, 2, d, device="cuda").to(BF16)
    return q, k, torch.empty(0, 4, device="cuda")


def _refused():
    """A workspace whose last call was refused."""
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    x = torch.randn(20, 2, 64, device="cuda").to(BF16)
    kla.kla_attn_fwd_varlen(x, x, x, _table(0, 12, 11), workspace=ws)
    with pytest.raises(kla.KlaError):
        kla.kla_workspace_status(ws)
    return ws


@pytest.mark.parametrize("keys", [0, 40])
def test_packed_calls_without_queries_leave_their_own_status(keys):
    q, k, lse = _sides(keys)
    cu_q, cu_k = _table(0, 0, 0), _table(0, keys // 2, keys)
    ws = _refused()
    kla.kla_attn_fwd_varlen(q, k, k, cu_q, cu_k, workspace=ws, check_status=True)
    ws = _refused()
    _, dk, dv = kla.kla_attn_bwd_varlen(q, k, k, q, lse, q, cu_q, cu_k, workspace=ws,
                                        check_status=True)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.parametrize("B,Tq,Tk", [(3, 0, 50), (0, 7, 7), (2, 0, 0)])
def test_batches_without_queries_leave_their_own_status(B, Tq, Tk):
    q = torch.empty(B, Tq, 4, 64, dtype=BF16, device="cuda")
    k = torch.randn(B, Tk, 2, 64, device="cuda").to(BF16)
    ws = _refused()
    o, lse = kla.kla_attn_fwd(q, k, k, workspace=ws)
    assert kla.kla_workspace_status(ws) == binding.KLA_OK
    ws = _refused()
    _, dk, dv = kla.kla_attn_bwd(q, k, k, o, lse, q, workspace=ws)
    assert kla.kla_workspace_status(ws) == binding.KLA_OK
    assert bool((dk == 0).all()) and bool((dv == 0).all())


def test_no_sequences_leave_their_own_status():
    q, k, _ = _sides(0)
    ws = _refused()
    kla.kla_attn_fwd_varlen(q, k, k, _table(0), workspace=ws, check_status=True)


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("keys,cu_q,cu_k", [
    (40, (0, 0, 0), (0, 50, 40)), (40, (0, 0, 0), (1, 20, 40)), (40, (0, 0, 0), (0, 20, 39)),
    (40, (1, 0, 0), (0, 20, 40)), (40, (0, 3, 0), (0, 20, 40)), (0, (0, 0, 0), (0, 1, 0))])
def test_bad_tables_without_queries_are_reported_and_nothing_is_written(keys, cu_q, cu_k, own):
    q, k, lse = _sides(keys)
    cu_q, cu_k = _table(*cu_q), _table(*cu_k)
    ws = torch.zeros(1 << 12, dtype=torch.uint8, device="cuda") if own else None
    with pytest.raises(kla.KlaError) as err:
        kla.kla_attn_fwd_varlen(q, k, k, cu_q, cu_k, workspace=ws, check_status=True)
    assert err.value.status == binding.KLA_ERR_INVALID_ARG
    dk, dv = torch.full_like(k, 3.0), torch.full_like(k, 3.0)
    with pytest.raises(kla.KlaError) as err:
        kla.kla_attn_bwd_varlen(q, k, k, q, lse, q, cu_q, cu_k, dk=dk, dv=dv, workspace=ws,
                                check_status=True)
    assert err.value.status == binding.KLA_ERR_INVALID_ARG
    assert bool((dk == 3).all()) and bool((dv == 3).all())


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("keys", [1, 4097])
def test_key_gradients_of_many_keys_without_queries_are_zero(keys, dtype):
    """Written whole and nothing behind them."""
    q = torch.empty(0, 4, 128, dtype=dtype, device="cuda")
    k = torch.randn(keys, 2, 128, device="cuda").to(dtype)
    hold = [torch.full((k.numel() + 64,), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
    dk, dv = (t[:k.numel()].view(k.shape) for t in hold)
    kla.kla_attn_bwd_varlen(q, k, k, q, torch.empty(0, 4, device="cuda"), q, _table(0, 0),
                            _table(0, keys), dk=dk, dv=dv, check_status=True)
    for t in hold:
        assert bool((t[:k.numel()] == 0).all()) and bool((t[k.numel():] == 3).all())
