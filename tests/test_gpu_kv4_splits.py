"""Attention over the paged 4-bit cache where a launch has many items and where an item has
many parts, against the definition in 64 bits."""
import functools
import math
import random

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from _cache_rows import BF16, FP32, Long, normal

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=1)
def _long(lens, hk, d, page, dtype):
    return Long(list(lens), hk, d, page, dtype)


def _tiles(lens, hq, hk, Tq, dtype):
    """(tiles of all items, warps of a CTA) of the attention's split."""
    rows = hq // hk * Tq
    two = dtype == BF16 and rows > 8
    groups = -(-rows // (16 if two else 8))
    return sum(-(-n // 64) for n in lens) * hk * groups, 8 if two or dtype == FP32 else 12


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _ragged(n, seed):
    g = torch.Generator().manual_seed(seed)
    some = torch.randint(1, 2400, (n,), generator=g).tolist()
    fixed = [0, 1, 64, 65, 63, 128, 0, 0, 31, 2]
    return [fixed[i % 10] if i % 3 else some[i] for i in range(n)]


@pytest.mark.parametrize("Tq", [1, 5])
@pytest.mark.parametrize("n", [200, 256])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_items_count_a_tile_more(Tq, n, dtype):
    """Tiles enough that every item counts as one more in the split: empty caches, caches of a
    tile, so that parts begin and end on what counts and is none."""
    hq, hk, d, page = 8, 4, 64, 32
    lens = _ragged(n, n)
    tiles, warps = _tiles(lens, hq, hk, Tq, dtype)
    assert tiles >= 2 * warps * _sms() and n <= 32 * warps
    c = _long(tuple(lens), hk, d, page, dtype)
    q = normal(n, Tq, hq, d, seed=8, dtype=dtype)
    got = c.check(q, d ** -0.5)
    assert all(torch.equal(x, y) for x, y in zip(c.attn(q.cuda()), got))


@pytest.mark.parametrize("Tq,hq", [(1, 8), (5, 3), (1, 3)])
@pytest.mark.parametrize("lens", [[40000], [250000, 1, 0, 64, 9]])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_items_over_many_parts(lens, Tq, hq, dtype):
    """An item over more than 32 CTAs, by itself and where items count a tile more: more parts
    of a row than the second kernel's warps have lanes."""
    d, page = 64, 128
    tiles, warps = _tiles(lens, hq, 1, Tq, dtype)
    per_cta = max(warps, -(-tiles // _sms()))
    assert -(-lens[0] // 64) // per_cta > 32
    if len(lens) > 1:
        assert tiles >= 2 * warps * _sms()
    c = _long(tuple(lens), 1, d, page, dtype)
    q = normal(len(lens), Tq, hq, d, seed=9, dtype=dtype)
    got = c.check(q, d ** -0.5)
    assert all(torch.equal(x, y) for x, y in zip(c.attn(q.cuda()), got))
    assert bool(torch.isfinite(got[1][0]).all()) and math.isfinite(float(got[0].double().sum()))


def test_the_same_bits_twice():
    """Random calls, each of them again: no sum depends on the order in which CTAs come."""
    r = random.Random(5)
    for i in range(60):
        hk, g, d, page = r.choice([1, 2, 4]), r.choice([1, 3, 8]), r.choice([64, 128]), r.choice([16, 48, 64])
        most = 2 ** r.randint(0, 13)
        lens = [r.choice([0, 1, most, r.randint(0, most)]) for _ in range(r.choice([1, 3, 17]))]
        dtype, Tq = r.choice([BF16, FP32]), r.choice([1, 2, 5, 40])
        columns, n_pages = 1 + -(-max(lens) // page), 300
        pool = torch.randint(0, 256, (n_pages, hk, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
        pool[..., 16 * d:] &= 0x3f                  # scales below 2
        table = torch.randint(0, n_pages, (len(lens), columns), dtype=torch.int32, device="cuda")
        lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = torch.randn(len(lens), Tq, hk * g, d, device="cuda").to(dtype)
        a, b = (kla.kla_kv4_attn(q, pool, table, lengths, check_status=True) for _ in range(2))
        assert bool(torch.isfinite(a[0]).all()), i
        assert all(torch.equal(x, y) for x, y in zip(a, b)), i
