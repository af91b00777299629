"""A wait of the tensor-core attention kernels that runs out, without a hang or
a fault: with KLA_TEST_LOST_WAIT set every CTA gives up while its first item is
under way.  The call reports KLA_ERR_TIMEOUT, the CTAs that start after others
wrote the status word leave whole, and the next call on the same workspace is
exact."""
import time

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

pytestmark = pytest.mark.gpu


def _normal(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).bfloat16().cuda()


CASES = [
    # lengths (None: a batch), B, Tq, Tk, Hq, Hk, d
    (None, 1, 1000, 1000, 8, 2, 128),
    (None, 8, 2048, 2048, 8, 4, 64),            # more blocks than SMs
    (None, 2, 3, 5000, 8, 2, 128),              # a split key axis
    ([900, 1, 0, 2100, 77] * 9, 0, 0, 0, 12, 4, 64),
    ([900, 1, 0, 2100, 77] * 9, 0, 0, 0, 6, 2, 128),      # three heads: a tile of 126 rows
]


def _sides(case):
    lens, B, Tq, Tk, hq, hk, d = case
    if lens is None:
        q, go = _normal(B, Tq, hq, d, seed=1), _normal(B, Tq, hq, d, seed=2)
        k, v = _normal(B, Tk, hk, d, seed=3), _normal(B, Tk, hk, d, seed=4)
        sizes = B, Tq, Tk, hq, hk, d
        return (q, k, v, go), (), sizes, (kla.kla_attn_fwd, kla.kla_attn_fwd_workspace_size,
                                          kla.kla_attn_bwd, kla.kla_attn_bwd_workspace_size)
    n = sum(lens)
    q, go = _normal(n, hq, d, seed=1), _normal(n, hq, d, seed=2)
    k, v = _normal(n, hk, d, seed=3), _normal(n, hk, d, seed=4)
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    return (q, k, v, go), (cu,), (len(lens), n, n, hq, hk, d), \
        (kla.kla_attn_fwd_varlen, kla.kla_attn_fwd_varlen_workspace_size,
         kla.kla_attn_bwd_varlen, kla.kla_attn_bwd_varlen_workspace_size)


@pytest.mark.parametrize("case", CASES)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_exact(monkeypatch, case):
    (q, k, v, go), cu, sizes, (fwd, fwd_size, bwd, bwd_size) = _sides(case)
    ws = torch.empty(max(fwd_size(*sizes), bwd_size(*sizes)), dtype=torch.uint8, device="cuda")
    want = fwd(q, k, v, *cu, workspace=ws)
    grads = bwd(q, k, v, *want, go, *cu, workspace=ws)
    torch.cuda.synchronize()
    for call, ref in ((lambda: fwd(q, k, v, *cu, workspace=ws), want),
                      (lambda: bwd(q, k, v, *want, go, *cu, workspace=ws), grads)):
        monkeypatch.setenv("KLA_TEST_LOST_WAIT", "1")
        t0 = time.perf_counter()
        call()
        with pytest.raises(kla.KlaError) as err:
            kla.kla_workspace_status(ws)
        assert err.value.status == binding.KLA_ERR_TIMEOUT
        # no role sat out its own bound of about one second
        assert time.perf_counter() - t0 < 0.5
        monkeypatch.delenv("KLA_TEST_LOST_WAIT")
        got = call()
        assert kla.kla_workspace_status(ws) == binding.KLA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("d", [64, 128])
def test_parts_of_a_call_that_timed_out_are_not_joined(monkeypatch, d):
    """A split key axis: the parts that were not written are no result."""
    q, k, v = _normal(2, 3, 8, d, seed=1), _normal(2, 5000, 2, d, seed=2), _normal(2, 5000, 2, d, seed=3)
    size = kla.kla_attn_fwd_workspace_size(2, 3, 5000, 8, 2, d)
    assert size > 256 + 2 * 2 * 3 * 8 * d * 4               # two parts and more
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")        # parts of NaN
    o, lse = torch.full_like(q, 3.0), torch.full((2, 3, 8), 3.0, device="cuda")
    monkeypatch.setenv("KLA_TEST_LOST_WAIT", "1")
    kla.kla_attn_fwd(q, k, v, o=o, lse=lse, workspace=ws)
    with pytest.raises(kla.KlaError) as err:
        kla.kla_workspace_status(ws)
    assert err.value.status == binding.KLA_ERR_TIMEOUT
    assert bool((o == 3).all()) and bool((lse == 3).all())


def test_a_fixed_length_call_raises_what_timed_out(monkeypatch):
    q, k, go = _normal(1, 300, 4, 64, seed=1), _normal(1, 300, 2, 64, seed=2), _normal(1, 300, 4, 64, seed=3)
    o, lse = kla.kla_attn_fwd(q, k, k, check_status=True)
    kla.kla_attn_bwd(q, k, k, o, lse, go, check_status=True)
    leaves = [x.clone().requires_grad_() for x in (q, k, k)]
    y = kla.kla_attn(*leaves, check_status=True)
    monkeypatch.setenv("KLA_TEST_LOST_WAIT", "1")
    for call in (lambda: kla.kla_attn_fwd(q, k, k, check_status=True),
                 lambda: kla.kla_attn_fwd(q, k, k, check_status=True, stream=torch.cuda.Stream()),
                 lambda: kla.kla_attn_bwd(q, k, k, o, lse, go, check_status=True),
                 lambda: kla.kla_attn(*leaves, check_status=True),
                 lambda: torch.autograd.grad(y, leaves, go)):
        with pytest.raises(kla.KlaError) as err:
            call()
        assert err.value.status == binding.KLA_ERR_TIMEOUT


def test_a_refused_table_is_raised_under_autograd():
    x = _normal(20, 2, 64, seed=1).requires_grad_()
    bad, good = torch.tensor([0, 12, 11]).int().cuda(), torch.tensor([0, 5, 20]).int().cuda()
    with pytest.raises(kla.KlaError) as err:
        kla.kla_attn(x, x, x, cu_seqlens_q=bad, check_status=True)
    assert err.value.status == binding.KLA_ERR_INVALID_ARG
    cu = good.clone()
    y = kla.kla_attn(x, x, x, cu_seqlens_q=cu, check_status=True)
    cu.data.copy_(bad)                      # refused in the backward pass
    with pytest.raises(kla.KlaError) as err:
        torch.autograd.grad(y.float().sum(), x)
    assert err.value.status == binding.KLA_ERR_INVALID_ARG
