"""The paged 4-bit cache at its limits: rows behind the table's end, units at their ends
where the cache is unpacked, more query heads to a key head than a tile has rows, and
caches that are unpacked a few sequences at a time."""
import random

import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla
from _cache_rows import BF16, FP32, Long, ints, normal
from gated_delta_rule_kaczmarz_gb300 import binding, cache

pytestmark = pytest.mark.gpu


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
    k, v = (normal(sum(new), hk, d, seed=s, dtype=dtype) for s in (3, 4))
    dev, kk, vv, cu = pool.cuda(), k.cuda(), v.cuda(), None
    if packed:
        cu = ints([0] + new).cumsum(0).int()
    else:
        kk, vv = (x.view(B, 5, hk, d) for x in (kk, vv))
    kla.kla_kv4_append(kk, vv, dev, table.cuda(), ints(lens), cu_seqlens=cu, check_status=True)
    _put_what_has_a_place(pool, table, lens, new, k, v, page)
    assert torch.equal(dev.cpu(), pool)


def test_units_where_the_cache_is_unpacked():
    """Keys and queries whose products fp32 does not hold unless the keys' unit goes with the
    scale: scale * k_unit is 2^-93."""
    B, Tq, hq, hk, d, page = 1, 64, 4, 2, 64, 16
    columns = -(-_cache.PAIRS // (B * Tq * hq * page))
    c = Long([300], hk, d, page, BF16, columns, units=(2.0 ** 32, 2.0 ** -32),
             size=(2.0 ** 33, 2.0 ** -32))
    q = (normal(B, Tq, hq, d, seed=5, dtype=FP32) * 2.0 ** 92).to(BF16)
    assert _cache.unpacked(B, Tq, hq, hk, page, columns, BF16)
    c.check(q, 2.0 ** -125, True)


@pytest.mark.parametrize("Tq,hq", [(1, 256), (2, 129)])
def test_many_heads_over_many_keys(Tq, hq):
    """More query heads to a key head than the dense attention's tensor cores take: such a cache
    is not unpacked, however wide its table."""
    page, d, lens = 64, 64, [3000, 70]
    columns = -(-2 * _cache.PAIRS // (Tq * hq * page))
    assert kla.kla_kv4_attn_workspace_size(2, Tq, hq, 1, d, page, columns) < columns * page * d * 4
    c = Long(lens, 1, d, page, BF16, columns)
    c.check(normal(2, Tq, hq, d, seed=6, dtype=BF16), d ** -0.5)


def test_a_cache_is_unpacked_a_few_sequences_at_a_time():
    """256 MiB of unpacked rows a sequence, 1 GiB at once: two turns of three."""
    Tq, hq, lens = 16, 64, [700, 0, 2500, 33, 16, 900]
    c = Long(lens, 8, 128, 64, BF16, 1024)
    size = kla.kla_kv4_attn_workspace_size(len(lens), Tq, hq, 8, 128, 64, 1024)
    assert 3 << 28 < size < 4 << 28
    q = normal(len(lens), Tq, hq, 128, seed=7, dtype=BF16)
    wide = torch.zeros(len(lens), Tq, hq * 128 + 64, dtype=BF16, device="cuda")
    part = wide[..., 64:].unflatten(-1, (hq, 128))
    part.copy_(q)
    got = c.check(q, 0.1, True, c.attn(part, scale=0.1, check_status=True))
    alone, none = c.attn(q.cuda(), scale=0.1, return_lse=False)
    assert none is None and torch.equal(alone, got[0])
    # captured, on a workspace of its own
    ws, q2 = torch.empty(size, dtype=torch.uint8, device="cuda"), q.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.attn(q2, scale=0.1, workspace=ws)
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(out, got))
    # an entry that names no page, in each group
    for b in (0, 2, 5):
        table = c.book[0].clone()
        table[b, 0] = -1
        with pytest.raises(kla.KlaError) as e:
            kla.kla_kv4_attn(q2, c.pool, table, c.book[1], scale=0.1, **c.units, workspace=ws, check_status=True)
        assert e.value.status == binding.KLA_ERR_INVALID_ARG
        o, _ = kla.kla_kv4_attn(q2, c.pool, table, c.book[1], scale=0.1, **c.units)
        others = [s for s in range(len(lens)) if s != b]
        assert torch.equal(o[others], got[0][others])
    c.attn(q2, scale=0.1, workspace=ws, check_status=True)


def test_a_wait_that_runs_out_in_any_group_is_reported(monkeypatch):
    Tq, hq, lens = 16, 64, [700, 0, 2500, 33, 16, 900]
    c = Long(lens, 8, 128, 64, BF16, 1024)
    q = normal(len(lens), Tq, hq, 128, seed=7, dtype=BF16).cuda()
    want = c.attn(q)
    monkeypatch.setenv("KLA_TEST_LOST_WAIT", "1")
    with pytest.raises(kla.KlaError) as e:
        c.attn(q, check_status=True)
    assert e.value.status == binding.KLA_ERR_TIMEOUT
    monkeypatch.delenv("KLA_TEST_LOST_WAIT")
    assert all(torch.equal(x, y) for x, y in zip(c.attn(q, check_status=True), want))


def test_a_last_turn_of_fewer_sequences():
    """Of seven two turns, of four and of three."""
    lens = [5, 300, 0, 64, 1000, 16, 129]
    c = Long(lens, 8, 128, 64, BF16, 1024)
    c.check(normal(len(lens), 16, 64, 128, seed=8, dtype=BF16), 0.1, True)


def test_workspaces_stay_small():
    """Whatever the sizes: 1 GiB of unpacked rows, and the parts of the attention."""
    r, largest = random.Random(1), 0
    for _ in range(3000):
        hk, d, page = r.choice([1, 2, 4, 8, 64]), r.choice([64, 128]), r.choice([16, 64, 128])
        columns, B = 2 ** r.randint(0, 14), 2 ** r.randint(0, 8)
        sizes = B, 2 ** r.randint(0, 10), hk * r.choice([1, 4, 7]), hk, d, page, columns
        got = kla.kla_kv4_attn_workspace_size(*sizes)
        largest = max(largest, got)
        assert got < (1 << 30) + (256 << 20), sizes
    assert largest > 1 << 30


@pytest.mark.parametrize("names", [("_empty",), ("_alloc",), ("_free",), ("_empty", "_alloc", "_free")])
def test_a_torch_without_the_faster_allocations(names, monkeypatch):
    """The same results, on outputs and workspaces that torch.empty makes."""
    c = Long([100, 0, 33], 2, 64, 16, BF16)
    q = normal(3, 2, 4, 64, seed=9, dtype=BF16).cuda()
    call = lambda: (*c.attn(q, check_status=True), *kla.kla_kv4_read(c.pool, *c.book, T=7, check_status=True))
    want = call()
    for name in names:
        monkeypatch.setattr(cache, name, None)
    assert all(torch.equal(x, y) for x, y in zip(call(), want))
