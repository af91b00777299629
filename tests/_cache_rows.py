"""A paged 4-bit cache that the append has filled, beside its rows' values."""
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla

BF16, FP32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


class Long:
    """A cache of normal rows, written by the append, and the rows' values."""

    def __init__(self, lens, hk, d, page, dtype, columns=0, units=(1.0, 0.5), size=(1.0, 0.3)):
        columns = max(columns, 1 + -(-max(lens) // page))
        n_pages = sum(-(-n // page) for n in lens) + 1
        table = _cache.book(lens, page, columns, n_pages, 1)
        self.pool = _cache.garbage(n_pages, hk, page // 16, 18 * d, seed=2).cuda()
        self.book = (table.cuda(), ints(lens))
        self.units = dict(k_unit=units[0], v_unit=units[1])
        k, v = (x * normal(sum(lens), hk, d, seed=s, dtype=FP32) for x, s in zip(size, (3, 4)))
        k, v = k.to(dtype), v.to(dtype)
        cu = ints([0] + lens).cumsum(0).int()
        kla.kla_kv4_append(k.cuda(), v.cuda(), self.pool, *self.book, cu_seqlens=cu, **self.units,
                           check_status=True)
        self.rows = list(zip(*(_cache.rounded(x, u).split(lens) for x, u in zip((k, v), units))))

    def attn(self, q, **how):
        return kla.kla_kv4_attn(q, self.pool, *self.book, **self.units, **how)

    def check(self, q, scale, unpacked=False, got=None):
        got = self.attn(q.cuda(), scale=scale, check_status=True) if got is None else got
        for b, rows in enumerate(self.rows):
            for x, (want, tol) in zip(got, _cache.attention(q[b], *rows, scale, unpacked)):
                x, hard = x[b].cpu().double(), ~torch.isfinite(want)
                assert torch.equal(x[hard], want[hard]), b
                off = ((x - want).abs() / tol.clamp_min(1e-300))[~hard]
                assert not off.numel() or float(off.max()) <= 1, (b, float(off.max()))
        return got
