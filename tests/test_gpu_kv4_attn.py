"""Attention over the paged 4-bit cache against its definition in 64 bits,
element by element (tolerances: ``_cache.attention``)."""
import math

import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def _check(got, ref, what):
    want, tol = ref
    got = got.cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    hard = ~torch.isfinite(want)
    assert torch.equal(got[hard], want[hard]), (what, "infinities")
    off = ((got - want).abs() / tol.clamp_min(1e-300))[~hard]
    assert not off.numel() or float(off.max()) <= 1, (what, float(off.max()))


def _q(B, Tq, hq, d, dtype, seed):
    return torch.randn(B, Tq, hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _case(lens, Tq, hq, hk, d, page, dtype, units=(1.0, 0.5), scale=None, extra=2, seed=1,
          columns=0):
    columns = max(columns, max(1, -(-max(lens) // page)) + 1)
    n_pages = sum(-(-n // page) for n in lens) + extra
    pool, table, held = _cache.filled(lens, page, columns, n_pages, hk, d, units, seed)
    q = _q(len(lens), Tq, hq, d, dtype, seed + 1)
    scale = scale or d ** -0.5
    other = _cache.unpacked(len(lens), Tq, hq, hk, page, columns, dtype)
    refs = [_cache.attention(x, *h, scale, other) for x, h in zip(q, held)]
    return q, (pool.cuda(), table.cuda(), torch.tensor(lens).int().cuda()), refs, \
        dict(scale=scale, k_unit=units[0], v_unit=units[1])


SIZES = [
    # lens, Tq, hq, hk, d, page
    ([1], 1, 1, 1, 64, 16),
    ([256], 1, 2, 2, 64, 16),
    ([0, 1, 15, 16, 17, 31, 32, 33, 64, 100], 1, 4, 1, 128, 16),
    ([500, 3, 0, 47], 1, 8, 2, 128, 48),
    ([65, 64], 3, 6, 3, 64, 64),
    ([2, 1, 0, 40], 5, 3, 3, 128, 32),            # rows that see nothing
    ([700], 5, 9, 3, 128, 32),
    ([1500], 1, 4, 4, 64, 128),
    ([333, 20], 2, 16, 2, 128, 16),               # 16 rows to a key head
    ([130], 1, 32, 1, 64, 16),
    ([90, 200], 7, 12, 2, 128, 64),               # 42 rows
    ([75], 75, 4, 2, 64, 16),                     # a whole prompt
    ([0, 0], 2, 4, 2, 128, 16),
    # many rows to a key head: 128 and more go another way in bf16
    ([130, 0, 300, 5], 40, 8, 2, 128, 16),
    ([63, 64], 64, 4, 2, 64, 48),
    ([200], 127, 3, 3, 64, 32),
    ([70, 90], 4, 128, 2, 64, 16),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,Tq,hq,hk,d,page", SIZES)
def test_against_the_definition(lens, Tq, hq, hk, d, page, dtype):
    q, cache, refs, how = _case(lens, Tq, hq, hk, d, page, dtype)
    o, lse = kla.kla_kv4_attn(q.cuda(), *cache, **how, check_status=True)
    for b, ref in enumerate(refs):
        _check(o[b], ref[0], ("o", b))
        _check(lse[b], ref[1], ("lse", b))


def _wide(B, Tq, hq, page):
    """Columns from which on the cache is unpacked where there are rows enough."""
    return -(-_cache.PAIRS // (B * Tq * hq * page))


@pytest.mark.parametrize("lens,Tq,hq,hk,d,page", [x for x in SIZES if x[1] * x[2] // x[3] >= _cache.LONG])
def test_unpacked_against_the_definition(lens, Tq, hq, hk, d, page):
    """Many rows over tables of many columns, most of them empty; one column less is not unpacked."""
    columns = _wide(len(lens), Tq, hq, page)
    sizes = [kla.kla_kv4_attn_workspace_size(len(lens), Tq, hq, hk, d, page, c) for c in (columns - 1, columns)]
    assert sizes[1] > len(lens) * columns * page * hk * d * 4 > sizes[0]
    for n in (columns - 1, columns):
        q, cache, refs, how = _case(lens, Tq, hq, hk, d, page, BF16, columns=n)
        o, lse = kla.kla_kv4_attn(q.cuda(), *cache, **how, check_status=True)
        for b, ref in enumerate(refs):
            _check(o[b], ref[0], ("o", b))
            _check(lse[b], ref[1], ("lse", b))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scale,units", [(1.0, (1.0, 1.0)), (30.0, (0.25, 2.0 ** -8)),
                                         (1e-3, (2.0 ** 10, 2.0 ** 12))])
def test_scales_and_units(scale, units, dtype):
    """Sharp and flat distributions: the maximum moves often, or never."""
    q, cache, refs, how = _case([400, 150], 2, 4, 2, 64, 16, dtype, units, scale)
    o, lse = kla.kla_kv4_attn(q.cuda(), *cache, **how, check_status=True)
    for b, ref in enumerate(refs):
        _check(o[b], ref[0], ("o", b))
        _check(lse[b], ref[1], ("lse", b))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_and_small_queries(dtype):
    """Rows whose size fp16 does not hold, and a row of zeros."""
    q, cache, _, how = _case([90], 4, 2, 2, 128, 16, dtype)
    q *= torch.tensor([1e20, 1e-20, 0.0, 3e30]).view(1, 4, 1, 1)
    how["scale"] = 1e-22
    pool, table, held = _cache.filled([90], 16, 7, 8, 2, 128, (1.0, 0.5), 1)
    ref = _cache.attention(q[0], *held[0], how["scale"])
    finite = ref[0][1].isfinite()
    o, lse = kla.kla_kv4_attn(q.cuda(), *cache, **how)
    assert bool(finite[:3].all())
    _check(o[0, :3], tuple(x[:3] for x in ref[0]), "o")
    _check(lse[0, :3], tuple(x[:3] for x in ref[1]), "lse")


def test_ascending_keys():
    """Every tile's maximum is above the last one's, by more and by less than what moves
    the base."""
    d, n, page = 64, 640, 16
    for step in (0.05, 1.0, 8.0):
        table = _cache.book([n], page, n // page, n // page, 1)
        pool = _cache.garbage(n // page, 1, 1, 18 * d, seed=1)
        k = (torch.arange(n).float() * step / 32)[:, None, None] * torch.ones(1, 1, d) / 8
        v = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(2))
        dev, lens = (pool.cuda(), table.cuda()), torch.tensor([n]).int().cuda()
        kla.kla_kv4_append(k[None].cuda(), v[None].cuda(), *dev, lens)
        q = torch.ones(1, 1, 1, d)
        ref = _cache.attention(q[0], _cache.rounded(k, 1.0), _cache.rounded(v, 1.0), 1.0)
        o, lse = kla.kla_kv4_attn(q.cuda(), *dev, lens, scale=1.0)
        _check(o[0], ref[0], ("o", step))
        _check(lse[0], ref[1], ("lse", step))


def test_long_and_ragged():
    """Items of many CTAs beside short ones: every way a part begins and ends."""
    lens = [9000, 1, 0, 31, 2500, 64, 4095, 3, 5000, 17]
    q, cache, refs, how = _case(lens, 1, 4, 2, 64, 16, BF16)
    o, lse = kla.kla_kv4_attn(q.cuda(), *cache, **how, check_status=True)
    for b, ref in enumerate(refs):
        _check(o[b], ref[0], ("o", b))
        _check(lse[b], ref[1], ("lse", b))
    again = kla.kla_kv4_attn(q.cuda(), *cache, **how)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_many_sequences():
    """More of them than a CTA has threads."""
    lens = [(i * 7) % 50 for i in range(1100)]
    q, cache, refs, how = _case(lens, 1, 1, 1, 64, 16, BF16)
    o, lse = kla.kla_kv4_attn(q.cuda(), *cache, **how, check_status=True)
    for b, ref in enumerate(refs):
        _check(o[b], ref[0], ("o", b))
        _check(lse[b], ref[1], ("lse", b))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strided_queries_and_given_outputs(dtype):
    q, cache, refs, how = _case([77, 50], 3, 4, 2, 64, 16, dtype)
    wide = torch.randn(2, 3, 4 * 64 + 96, device="cuda").to(dtype)
    part = wide[..., 64: 64 + 256].unflatten(-1, (4, 64))
    part.copy_(q)
    o, lse = torch.empty_like(q, device="cuda"), torch.empty(2, 3, 4, device="cuda")
    got = kla.kla_kv4_attn(part, *cache, **how, o=o, lse=lse)
    assert got[0] is o and got[1] is lse
    for b, ref in enumerate(refs):
        _check(o[b], ref[0], ("o", b))
        _check(lse[b], ref[1], ("lse", b))
    alone = kla.kla_kv4_attn(part, *cache, **how, return_lse=False)
    assert alone[1] is None and torch.equal(alone[0], o)


def test_shared_pages():
    """Two sequences that share their pages see the same rows."""
    q, (pool, table, lens), refs, how = _case([60], 1, 4, 2, 128, 16, BF16)
    two = kla.kla_kv4_attn(q.cuda().expand(2, -1, -1, -1).contiguous(), pool,
                           table.expand(2, -1).contiguous(), lens.expand(2).contiguous(), **how)
    assert torch.equal(two[0][0], two[0][1])
    _check(two[0][1], refs[0][0], "o")


def test_bad_entries_are_reported():
    _bad_entries(1)


def test_bad_entries_are_reported_for_many_rows():
    _bad_entries(64)


def test_bad_entries_are_reported_where_the_cache_is_unpacked():
    _bad_entries(64, _wide(2, 64, 4, 16))


def _bad_entries(Tq, columns=0):
    q, (pool, table, lens), refs, how = _case([60, 40], Tq, 4, 2, 128, 16, BF16, columns=columns)
    for bad in (-1, pool.shape[0], 1 << 30):
        t = table.clone()
        t[1, 1] = bad
        with pytest.raises(kla.KlaError) as e:
            kla.kla_kv4_attn(q.cuda(), pool, t, lens, **how, check_status=True)
        assert e.value.status == binding.KLA_ERR_INVALID_ARG
        o, _ = kla.kla_kv4_attn(q.cuda(), pool, t, lens, **how)
        _check(o[0], refs[0][0], "the other sequence")
    kla.kla_kv4_attn(q.cuda(), pool, table, lens, **how, check_status=True)
    clamped = torch.tensor([-3, 40]).int().cuda()
    o, lse = kla.kla_kv4_attn(q.cuda(), pool, table, clamped, **how, check_status=True)
    assert not o[0].any() and bool((lse[0] == -math.inf).all())
    _check(o[1], refs[1][0], "o")


def test_no_pages():
    q = torch.randn(2, 3, 4, 64, device="cuda").bfloat16()
    lens = torch.zeros(2).int().cuda()
    for pool, table in ((torch.empty(0, 2, 1, 18 * 64, dtype=torch.uint8, device="cuda"),
                         torch.zeros(2, 3).int().cuda()),
                        (_cache.garbage(4, 2, 1, 18 * 64).cuda(), torch.zeros(2, 0).int().cuda())):
        o, lse = kla.kla_kv4_attn(q, pool, table, lens, check_status=True)
        assert not o.any() and bool((lse == -math.inf).all())
        some = torch.tensor([0, 1]).int().cuda()
        o, lse = kla.kla_kv4_attn(q, pool, table, some)
        assert not o.any() and bool((lse == -math.inf).all())
        if table.shape[1]:                        # an entry that names no page
            with pytest.raises(kla.KlaError):
                kla.kla_kv4_attn(q, pool, table, some, check_status=True)
        else:                                     # the length is clamped
            kla.kla_kv4_attn(q, pool, table, some, check_status=True)
    none = kla.kla_kv4_attn(q[:0], pool, table[:0], lens[:0], check_status=True)
    assert none[0].shape == (0, 3, 4, 64)
    none = kla.kla_kv4_attn(q[:, :0], pool, table, lens, check_status=True)
    assert none[0].shape == (2, 0, 4, 64)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("hq,Tq", [(2, 1), (6, 3), (40, 7), (40, 13)])
def test_what_lies_behind_a_sequence_changes_no_bit(hq, Tq, dtype):
    """Groups of fewer rows than a tile has, lengths that end inside a block, and other
    bytes behind them."""
    lens, d, page = [5, 70, 131, 300], 64, 32
    q, (pool, table, length), _, how = _case(lens, Tq, hq, 2, d, page, dtype)
    ref = kla.kla_kv4_attn(q.cuda(), pool, table, length, **how)
    for seed in range(3):
        other = _cache.Pages(_cache.garbage(*pool.shape, seed=20 + seed), d)
        old = _cache.Pages(pool.cpu(), d)
        for b, n in enumerate(lens):
            for t in range(n):
                for h in range(2):
                    p = int(table[b, t // page])
                    other.put(p, h, t % page, *old.get(p, h, t % page))
        got = kla.kla_kv4_attn(q.cuda(), torch.from_numpy(other.b).cuda(), table, length, **how)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
