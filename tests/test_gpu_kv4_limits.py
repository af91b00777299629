"""The paged 4-bit cache at its limits: rows behind the table's end."""
import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _put_what_has_a_place(pool, table, lens, new, k, v, page):
    """The definition: row i of sequence b's new[b] to position lens[b] - new[b] + i, where the
    table has it."""
    pages, row = _cache.Pages(pool, k.shape[-1]), 0
    (kc, ks), (vc, vs) = _cache.quantise(k, 1.0), _cache.quantise(v, 1.0)
    for b, n in enumerate(new):
        for pos in range(lens[b] - n, lens[b]):
            if 0 <= pos < table.shape[1] * page:
                for h in range(k.shape[1]):
                    pages.put(int(table[b, pos // page]), h, pos % page, (kc[row, h], ks[row, h]),
                              (vc[row, h], vs[row, h]))
            row += 1


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_behind_the_tables_end_are_left_out(packed, dtype):
    """Nothing that the cache holds is written over by a row that has no place."""
    hk, d, page, columns = 2, 64, 16, 2
    lens = [33, 32, 34, 36, 37, 40, 31, 2 ** 31 - 1, 2 ** 31 - 2, 3, 33, 34]
    new = [5, 5, 5, 5, 5, 5, 5, 5, 5, 5, 5, 5]
    if packed:
        new = [1, 2, 1, 7, 5, 0, 40, 9, 50, 5, 40, 39]
    B = len(lens)
    table = torch.randperm(B * columns, generator=torch.Generator().manual_seed(1)).int().view(B, columns)
    pool = _cache.garbage(B * columns, hk, 1, 18 * d, seed=2)
    k, v = (_normal(sum(new), hk, d, seed=s, dtype=dtype) for s in (3, 4))
    dev, kk, vv, cu = pool.cuda(), k.cuda(), v.cuda(), None
    if packed:
        cu = _ints([0] + new).cumsum(0).int()
    else:
        kk, vv = (x.view(B, 5, hk, d) for x in (kk, vv))
    kla.kla_kv4_append(kk, vv, dev, table.cuda(), _ints(lens), cu_seqlens=cu, check_status=True)
    _put_what_has_a_place(pool, table, lens, new, k, v, page)
    assert torch.equal(dev.cpu(), pool)
