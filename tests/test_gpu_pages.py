"""The pages' operators against plain loops over lists: table, lengths, counts and
contents, equal to the last bit."""
import random

import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _random_book(S, columns, page, n_pages, seed, share=0.3):
    """Sequences, some of which share a prefix with another."""
    r = random.Random(seed)
    free = list(range(n_pages))
    r.shuffle(free)
    table, lens = [[-1] * columns for _ in range(S)], [0] * S
    for s in range(S):
        n = r.choice([0, r.randint(0, columns * page), r.randint(0, columns * page // 2), page])
        held = -(-n // page)
        if s and r.random() < share:
            o = r.randrange(s)
            lens[s] = lens[o]
            table[s] = list(table[o])
        elif held <= len(free) // 2:
            lens[s] = n
            table[s][:held] = [free.pop() for _ in range(held)]
    return table, lens, _cache.counted(table, lens, page, n_pages)


def _same(dev, want):
    for x, y in zip(dev, want):
        assert x.tolist() == y


SIZES = [(1, 1, 1, 1), (3, 4, 16, 9), (40, 7, 5, 300), (300, 20, 64, 5000), (9, 2, 16, 20001),
         (2000, 3, 16, 9000), (5, 700, 16, 4000), (50, 257, 16, 12000)]


@pytest.mark.parametrize("S,columns,page,n_pages", SIZES)
def test_fork_and_free(S, columns, page, n_pages):
    r = random.Random(S)
    table, lens, refs = _random_book(S, columns, page, n_pages, S + 1)
    dev = _ints(table).view(S, columns), _ints(lens), _ints(refs)
    for _ in range(4):
        dst = r.sample(range(S), r.randint(0, S))
        src = [r.randint(-1, S - 1) for _ in dst]        # permutations and repeats among them
        kla.kla_pages_fork(*dev, _ints(src), _ints(dst), page, check_status=True)
        table, lens = _cache.fork(table, lens, src, dst, page)
        refs = _cache.counted(table, lens, page, n_pages)
        _same(dev, (table, lens, refs))
    dst = r.sample(range(S), S // 2 + 1)
    kla.kla_pages_free(*dev, _ints(dst), page, check_status=True)
    table, lens = _cache.fork(table, lens, [-1] * len(dst), dst, page)
    _same(dev, (table, lens, _cache.counted(table, lens, page, n_pages)))


@pytest.mark.parametrize("layers,size", [(1, 16), (3, 4096 * 5 + 48)])
@pytest.mark.parametrize("S,columns,page,n_pages", SIZES)
def test_grow(S, columns, page, n_pages, layers, size):
    if n_pages > 6000 and size > 16:
        size = 144
    r = random.Random(S)
    table, lens, refs = _random_book(S, columns, page, n_pages, S + 2, share=0.5)
    dev = _ints(table).view(S, columns), _ints(lens), _ints(refs)
    pool = torch.randint(0, 256, (layers, n_pages, size), dtype=torch.uint8,
                         generator=torch.Generator().manual_seed(1))
    data = pool.cuda()
    for _ in range(3):
        more = [r.choice([0, 1, 1, 2, page, 2 * page + 1]) for _ in range(S)]
        more = [min(m, columns * page - n) for m, n in zip(more, lens)]
        want = _cache.grow(table, lens, refs, more, page)
        if want is None:
            before = [x.clone() for x in (*dev, data)]
            with pytest.raises(kla.KlaError) as e:
                kla.kla_pages_grow(data, *dev, _ints(more), page, check_status=True)
            assert e.value.status == binding.KLA_ERR_PAGES
            assert all(torch.equal(x, y) for x, y in zip((*dev, data), before))
            continue
        kla.kla_pages_grow(data, *dev, _ints(more), page, check_status=True)
        table, lens, refs, copies = want
        for a, b in copies:
            pool[:, b] = pool[:, a]
        _same(dev, (table, lens, refs))
        assert torch.equal(data.cpu(), pool)


@pytest.mark.parametrize("S,columns,page,n_pages", SIZES)
def test_trim(S, columns, page, n_pages):
    r = random.Random(S)
    table, lens, refs = _random_book(S, columns, page, n_pages, S + 4, share=0.5)
    dev = _ints(table).view(S, columns), _ints(lens), _ints(refs)
    for _ in range(3):
        cut = [r.choice([0, min(1, n), n, n // 2, r.randint(0, n)]) for n in lens]
        kla.kla_pages_trim(*dev, _ints(cut), page, check_status=True)
        table, lens = _cache.trim(table, lens, cut, page)
        refs = _cache.counted(table, lens, page, n_pages)
        _same(dev, (table, lens, refs))


@pytest.mark.parametrize("S,columns,page,n_pages", SIZES)
def test_compact(S, columns, page, n_pages):
    table, lens, refs = _random_book(S, columns, page, n_pages, S + 3)
    # a page that no sequence of the book holds
    extra = max(range(n_pages), key=lambda p: (refs[p] == 0, p))
    refs[extra] += 1
    dev = _ints(table).view(S, columns), _ints(lens), _ints(refs)
    pool = torch.randint(0, 1 << 20, (2, n_pages, 12), dtype=torch.int32,
                         generator=torch.Generator().manual_seed(1))
    data = pool.cuda()
    where, n_used = kla.kla_pages_compact(data, *dev, page, check_status=True)
    want, after, moved, moves = _cache.compact(table, lens, refs, page)
    for a, b in moves:
        pool[:, b] = pool[:, a]
    _same(dev, (want, lens, after))
    assert where.tolist() == moved and n_used.tolist() == [sum(n > 0 for n in refs)]
    n = n_used.item()
    assert torch.equal(data.cpu()[:, :n], pool[:, :n])
    again, _ = kla.kla_pages_compact(data, *dev, page, check_status=True)
    assert again.tolist() == [p if p < n else -1 for p in range(n_pages)]


@pytest.mark.parametrize("layers,n_pages,size,dtype", [(1, 1, 16, torch.uint8), (3, 50, 5000, torch.float32),
                                                       (2, 9, 1 << 20, torch.bfloat16)])
def test_copy(layers, n_pages, size, dtype):
    r = random.Random(n_pages)
    places = r.sample(range(n_pages), n_pages)
    dst, rest = places[: n_pages // 2], places[n_pages // 2:]
    src = [r.choice(rest) for _ in dst]
    pool = torch.randn(layers, n_pages, size, generator=torch.Generator().manual_seed(2)).to(dtype)
    data = pool.cuda()
    kla.kla_pages_copy(data, _ints(src), _ints(dst), check_status=True)
    pool[:, dst] = pool[:, src]
    assert torch.equal(data.cpu(), pool)
    # a page to itself changes nothing
    kla.kla_pages_copy(data, _ints(rest[:1]), _ints(rest[:1]), check_status=True)
    assert torch.equal(data.cpu(), pool)


def test_states_are_pages():
    """KLA's states follow a fork."""
    S = torch.randn(6, 3, 64, 64, device="cuda")
    want = S.clone()
    kla.kla_pages_copy(S[None], _ints([0, 0, 2]), _ints([1, 3, 5]), check_status=True)
    want[[1, 3, 5]] = want[[0, 0, 2]]
    assert torch.equal(S, want)


def test_what_the_device_refuses():
    table, lens, refs = _ints([[0, 1], [2, -1], [-1, -1]]), _ints([20, 3, 0]), _ints([1, 1, 1, 0, 0])
    pool = torch.randn(1, 5, 4, device="cuda")
    before = [x.clone() for x in (table, lens, refs, pool)]

    def refused(call, status=binding.KLA_ERR_INVALID_ARG):
        with pytest.raises(kla.KlaError) as e:
            call()
        assert e.value.status == status
        assert all(torch.equal(x, y) for x, y in zip((table, lens, refs, pool), before))

    for src, dst in (([0, 1], [2, 2]), ([0], [3]), ([0], [-1]), ([3], [2]), ([-2], [2])):
        refused(lambda: kla.kla_pages_fork(table, lens, refs, _ints(src), _ints(dst), 16,
                                           check_status=True))
    for more in ([0, -1, 0], [13, 0, 0], [0, 0, 33], [0, 1 << 30, 0], [0, 2147483647, 0]):
        refused(lambda: kla.kla_pages_grow(pool, table, lens, refs, _ints(more), 16,
                                           check_status=True))
    for cut in ([21, 0, 0], [0, -1, 0], [1, 0, 1], [-2147483648, 0, 0], [0, 2147483647, 0]):
        refused(lambda: kla.kla_pages_trim(table, lens, refs, _ints(cut), 16, check_status=True))
    refused(lambda: kla.kla_pages_grow(pool, table, lens, refs, _ints([0, 20, 20]), 16,
                                       check_status=True), binding.KLA_ERR_PAGES)
    for src, dst in (([0, 1], [3, 3]), ([0], [5]), ([-1], [3]), ([0, 3], [3, 4]), ([1, 0], [0, 1])):
        refused(lambda: kla.kla_pages_copy(pool, _ints(src), _ints(dst), check_status=True))


def test_bad_entries_are_left_and_reported():
    table, lens, refs = _ints([[9, 1], [-3, -1], [0, -1]]), _ints([20, 3, 5]), _ints([1, 1, 0])
    pool = torch.randn(1, 3, 4, device="cuda")
    with pytest.raises(kla.KlaError):
        kla.kla_pages_compact(pool, table, lens, refs, 16, check_status=True)
    assert table.tolist() == [[9, 1], [-3, -1], [0, -1]] and refs.tolist() == [1, 1, 0]
    with pytest.raises(kla.KlaError):
        kla.kla_pages_grow(pool, table, lens, refs, _ints([0, 1, 0]), 16, check_status=True)
    with pytest.raises(kla.KlaError):
        kla.kla_pages_fork(table, lens, refs, _ints([0]), _ints([1]), 16, check_status=True)
    assert table[1].tolist() == [9, 1] and refs.tolist() == [1, 2, 0]
    with pytest.raises(kla.KlaError):
        kla.kla_pages_trim(table, lens, refs, _ints([20, 0, 0]), 16, check_status=True)
    assert table[0].tolist() == [-1, -1] and lens[0].item() == 0 and refs.tolist() == [1, 1, 0]


def test_nothing_to_do():
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = empty.view(0, 4)
    pool = torch.zeros(2, 0, 16, device="cuda")
    kla.kla_pages_fork(table, empty, empty, empty, empty, 16, check_status=True)
    kla.kla_pages_grow(pool, table, empty, empty, empty, 16, check_status=True)
    where, n = kla.kla_pages_compact(pool, table, empty, empty, 16, check_status=True)
    assert where.numel() == 0 and n.tolist() == [0]
    kla.kla_pages_copy(pool, empty, empty, check_status=True)
    kla.kla_pages_trim(table, empty, empty, empty, 16, check_status=True)
    # no layers: the book alone
    table, lens, refs = _ints([[1, -1]]), _ints([3]), _ints([0, 1])
    kla.kla_pages_grow(torch.zeros(0, 2, 16, device="cuda"), table, lens, refs, _ints([20]), 16,
                       check_status=True)
    assert table.tolist() == [[1, 0]] and lens.tolist() == [23] and refs.tolist() == [1, 1]
