"""Rows into the paged 4-bit cache and out of it, bit for bit against the
definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def _rows(n, hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 2, hk, d, generator=g) * torch.exp2(
        torch.randint(-14, 14, (n, 2, hk, 1), generator=g).float())
    return x[:, 0].to(dtype), x[:, 1].to(dtype)


def _put(pool, table, lens, new, k, v, page, units):
    """The definition: k, v [total, Hk, d] to the last new[b] positions of sequence b."""
    pages = _cache.Pages(pool, k.shape[-1])
    (kc, ks), (vc, vs) = _cache.quantise(k, units[0]), _cache.quantise(v, units[1])
    row = 0
    for b, n in enumerate(new):
        for i in range(n):
            pos = lens[b] - n + i
            if pos >= 0:
                for h in range(k.shape[1]):
                    pages.put(int(table[b, pos // page]), h, pos % page, (kc[row, h], ks[row, h]),
                              (vc[row, h], vs[row, h]))
            row += 1


@pytest.mark.parametrize("lens,T,page,hk,d,dtype,units", [
    ([1], 1, 16, 1, 64, BF16, (1.0, 1.0)),
    ([0, 7, 32, 33, 5], 1, 16, 2, 128, BF16, (1.0, 0.25)),
    ([40, 3, 16, 0, 90], 6, 48, 3, 64, FP32, (0.5, 4.0)),
    ([77, 130, 128], 77, 32, 2, 128, FP32, (2.0 ** -9, 2.0 ** 5)),
    ([65, 64, 63], 63, 64, 1, 128, BF16, (1.0, 1.0)),
    ([300, 301], 300, 128, 8, 64, BF16, (1.0, 1.0)),
])
def test_append_and_read(lens, T, page, hk, d, dtype, units):
    """Odd places, rows before the first position, neighbours that stay."""
    B, columns = len(lens), max(1, -(-max(lens) // page)) + 1
    n_pages = sum(-(-n // page) for n in lens) + 2
    table = _cache.book(lens, page, columns, n_pages, 3)
    pool = _cache.garbage(n_pages, hk, page // 16, 18 * d, seed=4)
    k, v = _rows(B * T, hk, d, dtype, 5)
    dev, book = pool.cuda(), (table.cuda(), torch.tensor(lens).int().cuda())
    kk, vv = (x.cuda().view(B, T, hk, d) for x in (k, v))
    kla.kla_kv4_append(kk, vv, dev, *book, k_unit=units[0], v_unit=units[1], check_status=True)
    _put(pool, table, lens, [T] * B, k, v, page, units)
    assert torch.equal(dev.cpu(), pool)
    got = kla.kla_kv4_read(dev, *book, T=T, dtype=dtype, k_unit=units[0], v_unit=units[1],
                           check_status=True)
    for x, rows, unit in zip(got, (k, v), units):
        want = _cache.rounded(rows, unit).view(B, T, hk, d)
        for b, n in enumerate(lens):
            want[b, :max(0, T - n)] = 0
        assert x.dtype == dtype and torch.equal(x.cpu().double(), want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("new,before,page", [([5, 0, 1, 18, 2], [0, 9, 31, 3, 16], 16),
                                             ([129, 1], [1, 0], 64), ([0, 0], [3, 0], 32),
                                             ([7], [0], 16)])
def test_packed(new, before, page, dtype):
    hk, d, units = 2, 64, (1.0, 0.5)
    lens = [a + b for a, b in zip(new, before)]
    columns, n_pages = max(1, -(-max(lens) // page)), sum(-(-n // page) for n in lens) + 1
    table = _cache.book(lens, page, columns, n_pages, 7)
    pool = _cache.garbage(n_pages, hk, page // 16, 18 * d, seed=8)
    k, v = _rows(sum(new), hk, d, dtype, 9)
    dev, book = pool.cuda(), (table.cuda(), torch.tensor(lens).int().cuda())
    cu = torch.tensor([0] + new).cumsum(0).int().cuda()
    # strided rows, and rows behind the last that stay as they are
    wide = torch.full((sum(new) + 3, 3 * hk * d), 7.0, dtype=dtype, device="cuda")
    kk, vv = (wide[: sum(new), i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in (0, 2))
    kk.copy_(k)
    vv.copy_(v)
    kla.kla_kv4_append(kk, vv, dev, *book, cu_seqlens=cu, k_unit=units[0], v_unit=units[1],
                       check_status=True)
    _put(pool, table, lens, new, k, v, page, units)
    assert torch.equal(dev.cpu(), pool)
    wide.fill_(7.0)
    kla.kla_kv4_read(dev, *book, total=sum(new), cu_seqlens=cu, dtype=dtype, k_unit=units[0],
                     v_unit=units[1], k_out=kk, v_out=vv, check_status=True)
    assert torch.equal(kk.cpu().double(), _cache.rounded(k, units[0]))
    assert torch.equal(vv.cpu().double(), _cache.rounded(v, units[1]))
    assert bool((wide[sum(new):] == 7).all()) and bool((wide[:, hk * d: 2 * hk * d] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_borders(dtype):
    """Ties of scales and codes, the neighbours of both in the type, saturation, zeros and
    what is not finite: a block of each."""
    f = torch.finfo(dtype)
    rows = []
    scales = [s for s in _cache.SCALES if s > 0]
    for s in scales[::3] + [448.0, 1000.0]:
        x = [s * t for t in (6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5)]
        x = torch.tensor(x, dtype=torch.float64).to(dtype)
        rows += [torch.cat([x, -x]), torch.cat([x[:1], x[1:], torch.nextafter(x, x + 1)]),
                 torch.cat([x[:1], x[1:], torch.nextafter(x, x - 1)])]
    for a, b in zip(scales[::2], scales[1::2]):          # amax on a midpoint of scales, and near
        x = torch.tensor([6 * (a + b) / 2], dtype=torch.float64).to(dtype)
        for y in (x, torch.nextafter(x, x + 1), torch.nextafter(x, x - 1)):
            rows.append(torch.cat([y, torch.linspace(-1, 1, 15).to(dtype) * y]))
    tiny = [0.0, 6 * 2.0 ** -10, 6 * 2.0 ** -10 * (1 + f.eps), f.tiny, f.smallest_normal / 2]
    for t in tiny + [f.max, math.inf, -math.inf, math.nan]:
        rows.append(torch.tensor([t] + [0.5] * 0 + [-t / 3] * 15).to(dtype))
        rows.append(torch.tensor([t] + [1.0] * 15).to(dtype))
    x = torch.stack(rows)
    x = torch.cat([x, x[: -len(x) % 4]])
    k = x.view(-1, 1, 64)
    v = k.flip(0).contiguous()
    n, page = len(k), 16
    table = _cache.book([n], page, -(-n // page), -(-n // page), 1)
    pool = _cache.garbage(-(-n // page), 1, 1, 18 * 64, seed=2)
    dev, book = pool.cuda(), (table.cuda(), torch.tensor([n]).int().cuda())
    kla.kla_kv4_append(k[None].cuda(), v[None].cuda(), dev, *book)
    kk, vv = kla.kla_kv4_read(dev, *book, T=n, dtype=FP32)
    for got, want in ((kk, k), (vv, v)):
        want = _cache.rounded(want, 1.0)
        assert torch.equal(got[0].cpu().double().nan_to_num(nan=1e9), want.nan_to_num(nan=1e9))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("unit", [2.0 ** -32, 2.0 ** 32])
def test_units_at_their_ends(unit, dtype):
    """Values that the unit takes out of fp32's range, and into its smallest numbers."""
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(2, 24, 1, 64, generator=g) * torch.exp2(
        torch.randint(-140, 126, (2, 24, 1, 4), generator=g).float()).repeat_interleave(16, -1))
    k, v = k.to(dtype), v.to(dtype)
    k[3, 0, 5] = torch.finfo(dtype).max
    k[4, 0, 5] = -torch.finfo(dtype).max
    table = torch.tensor([[1, 0]]).int().cuda()
    pool, lens = _cache.garbage(2, 1, 1, 18 * 64).cuda(), torch.tensor([24]).int().cuda()
    kla.kla_kv4_append(k[None].cuda(), v[None].cuda(), pool, table, lens, k_unit=unit, v_unit=unit)
    want = _cache.garbage(2, 1, 1, 18 * 64)
    _put(want, table.cpu(), [24], [24], k, v, 16, (unit, unit))
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_on_boundaries_of_16_bytes(dtype):
    n, hk, d, step = 21, 2, 64, 16 // torch.finfo(dtype).bits * 8
    table, lens = _cache.book([n], 16, 2, 2, 1).cuda(), torch.tensor([n]).int().cuda()
    pool = _cache.garbage(2, hk, 1, 18 * d).cuda()
    k, v = _rows(n, hk, d, dtype, 2)
    flat = torch.zeros(2, n * (hk * d + step) + step, dtype=dtype, device="cuda")
    kk, vv = (x[step:].view(n, hk * d + step)[:, : hk * d].unflatten(1, (hk, d))[None] for x in flat)
    kk.copy_(k[None])
    vv.copy_(v[None])
    kla.kla_kv4_append(kk, vv, pool, table, lens)
    flat.zero_()
    kla.kla_kv4_read(pool, table, lens, T=n, dtype=dtype, k_out=kk, v_out=vv)
    assert torch.equal(kk[0].cpu().double(), _cache.rounded(k, 1.0))
    assert torch.equal(vv[0].cpu().double(), _cache.rounded(v, 1.0))


def test_steps_are_a_chunk():
    """Tokens appended one by one are the bytes of the chunk."""
    lens, hk, d, page = [37, 5], 2, 128, 16
    table = _cache.book(lens, page, 3, 6, 1).cuda()
    k, v = (x.view(2, 5, hk, d).cuda() for x in _rows(10, hk, d, BF16, 2))
    pools = [_cache.garbage(6, hk, 1, 18 * d, seed=3).cuda() for _ in range(2)]
    at = torch.tensor(lens).int().cuda()
    kla.kla_kv4_append(k, v, pools[0], table, at)
    for t in range(5):
        kla.kla_kv4_append(k[:, t:t + 1], v[:, t:t + 1], pools[1], table, at - 4 + t)
    assert torch.equal(*pools)


def test_what_the_device_refuses():
    """A page outside the pool and a table that does not hold are reported; nothing else is
    touched."""
    hk, d, page = 1, 64, 16
    pool = _cache.garbage(3, hk, 1, 18 * d, seed=1).cuda()
    before = pool.clone()
    k = torch.randn(1, 4, hk, d, device="cuda")
    lens = torch.tensor([20]).int().cuda()
    for bad in (-1, 3, 1 << 30):
        table = torch.tensor([[0, bad]]).int().cuda()
        with pytest.raises(kla.KlaError) as e:
            kla.kla_kv4_append(k, k, pool, table, lens, check_status=True)
        assert e.value.status == binding.KLA_ERR_INVALID_ARG
        with pytest.raises(kla.KlaError):
            kla.kla_kv4_read(pool, table, lens, T=4, check_status=True)
    assert torch.equal(pool, before)
    table = torch.tensor([[0, 1], [2, 0]]).int().cuda()
    lens = torch.tensor([4, 4]).int().cuda()
    for cu in ([0, 5, 4], [1, 2, 4], [0, 2, 3], [0, -1, 4]):
        with pytest.raises(kla.KlaError) as e:
            kla.kla_kv4_append(k[0], k[0], pool, table, lens, check_status=True,
                               cu_seqlens=torch.tensor(cu).int().cuda())
        assert e.value.status == binding.KLA_ERR_INVALID_ARG
    # sizes of another kind of whole number, and sizes that are none
    for n in (np.int64(2), torch.tensor(2)):
        assert kla.kla_kv4_read(pool, table, lens, T=n)[0].shape[1] == 2
    with pytest.raises(TypeError):
        kla.kla_kv4_read(pool, table, lens, T=2.0)
    with pytest.raises(ValueError, match="negative"):
        kla.kla_kv4_read(pool, table, lens, T=-1)
    # a pool without pages: no row has a place, and rows are read as zeros
    none = pool[:0]
    with pytest.raises(kla.KlaError):
        kla.kla_kv4_append(k, k, none, table[:1], lens[:1], check_status=True)
    with pytest.raises(kla.KlaError):
        kla.kla_kv4_read(none, table[:1], lens[:1], T=4, check_status=True)
    assert not any(x.any() for x in kla.kla_kv4_read(none, table[:1], lens[:1], T=4))
    assert not any(x.any() for x in kla.kla_kv4_read(none, table[:1, :0], lens[:1], T=4, check_status=True))
    # lengths that no row of the table holds are clamped
    kla.kla_kv4_append(k, k, pool, table[:1], torch.tensor([1 << 30]).int().cuda(), check_status=True)
    kla.kla_kv4_append(k, k, pool, table[:1], torch.tensor([-5]).int().cuda(), check_status=True)


def test_tensors_that_lie_elsewhere():
    """Each argument on the host, of another type, shape or order, in turn, is refused."""
    base = _cache.arguments(lambda t: t.cuda())
    before = [x.clone() for x in base["kept"]]
    for name, args, key, bad in _cache.wrong_arguments(base, lambda t: t.cpu()):
        with pytest.raises((ValueError, TypeError)):
            getattr(kla, name)(**{**args, key: bad})
    assert all(torch.equal(x, y) for x, y in zip(base["kept"], before))
