"""A wait of the pipelined conditioning kernel that runs out, without a hang or a
fault: with KLA_TEST_LOST_WAIT set every warp takes its first wait for lost.
The call has no status word, so all it writes is NaN; the next one is exact."""
import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,d,dtype", [(5, 2, 128, torch.bfloat16), (3, 0, 64, torch.float32)])
def test_rows_whose_copy_did_not_come_are_not_a_number(monkeypatch, hq, hk, d, dtype):
    n = 9731                                      # every warp has several tokens
    g = torch.Generator().manual_seed(1)

    def normal(heads):
        return torch.randn(n, heads, d, generator=g).to(dtype).cuda() if heads else None

    q, k, gq, gk = normal(hq), normal(hk), normal(hq), normal(hk)
    w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    args = (torch.arange(n).int().cuda(), torch.rand(d // 4, generator=g).cuda())
    weights = dict(wq=w, wk=w if hk else None)

    def call():
        x = kla.kla_qk_norm_rope_fwd(q, k, *args, **weights)
        return [t for t in (*x, *kla.kla_qk_norm_rope_bwd(q, k, *args, gq, gk, **weights))
                if t is not None]

    want = call()
    monkeypatch.setenv("KLA_TEST_LOST_WAIT", "1")
    lost = call()
    torch.cuda.synchronize()
    monkeypatch.delenv("KLA_TEST_LOST_WAIT")
    assert all(bool(t.isnan().all()) for t in lost)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
