"""The paged 4-bit cache: what the host refuses, before any device work, the
workspaces, and the split of attention's tiles over CTAs and warps."""
import random

import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding, cache

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="uses fake device pointers; host validation only")
FAKE = 0x10000
INVALID, UNSUPPORTED = binding.KLA_ERR_INVALID_ARG, binding.KLA_ERR_UNSUPPORTED
WORKSPACE = binding.KLA_ERR_WORKSPACE
KV = dict(pool=FAKE, table=FAKE, lens=FAKE, k_unit=1.0, v_unit=0.5, B=2, Hk=2, d=64, page=32,
          n_pages=9, columns=4, dtype=1, ws=FAKE, wsb=1 << 40)


def _rows(name, **over):
    a = {**KV, "k": FAKE, "ks": 128, "v": FAKE, "vs": 128, "cu": None, "T": 3, **over}
    return getattr(binding.load(), name)(
        a["k"], a["ks"], a["v"], a["vs"], a["pool"], a["table"], a["lens"], a["cu"], a["k_unit"],
        a["v_unit"], a["B"], a["T"], a["Hk"], a["d"], a["page"], a["n_pages"], a["columns"],
        a["dtype"], a["ws"], a["wsb"], None)


def _attn(**over):
    a = {**KV, "q": FAKE, "qs": 256, "scale": 0.1, "o": FAKE, "lse": FAKE, "Tq": 1, "Hq": 4, **over}
    return binding.load().kla_kv4_attn(
        a["q"], a["qs"], a["pool"], a["table"], a["lens"], a["scale"], a["k_unit"], a["v_unit"],
        a["o"], a["lse"], a["B"], a["Tq"], a["Hq"], a["Hk"], a["d"], a["page"], a["n_pages"],
        a["columns"], a["dtype"], a["ws"], a["wsb"], None)


SHARED = [
    (dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(table=None, n_pages=0), INVALID),
    (dict(pool=FAKE + 8), INVALID), (dict(table=FAKE + 2), INVALID), (dict(lens=FAKE + 1), INVALID),
    (dict(k_unit=0.3), INVALID), (dict(v_unit=0.0), INVALID), (dict(k_unit=-1.0), INVALID),
    (dict(v_unit=float("nan")), INVALID), (dict(k_unit=2.0 ** 33), INVALID),
    (dict(v_unit=2.0 ** -33), INVALID), (dict(B=-1), INVALID), (dict(Hk=0), INVALID),
    (dict(page=0), INVALID), (dict(n_pages=-1), INVALID), (dict(columns=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(d=96), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(columns=1 << 30), UNSUPPORTED), (dict(n_pages=2 ** 31 - 1), UNSUPPORTED),
    (dict(columns=(1 << 26) - 1), UNSUPPORTED),
    (dict(ws=FAKE + 16), INVALID), (dict(wsb=64), WORKSPACE),
]


@no_gpu_only
@pytest.mark.parametrize("name", ["kla_kv4_append", "kla_kv4_read"])
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID),
    (dict(ks=120), INVALID), (dict(vs=132), INVALID), (dict(T=-1), INVALID),
    (dict(cu=FAKE + 2), INVALID), (dict(cu=FAKE, B=0, lens=None), INVALID),
    (dict(Hk=2048, ks=1 << 20, vs=1 << 20), UNSUPPORTED),
    (dict(B=1 << 16, T=1 << 16), UNSUPPORTED)])
def test_rows_refuse(name, over, status):
    assert _rows(name, **over) == status
    assert binding.load().kla_last_error_message().decode() != ""


@no_gpu_only
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(o=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(qs=250), INVALID),
    (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Tq=-1), INVALID),
    (dict(Hq=2048), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=1e-36, k_unit=2.0 ** -20), INVALID),
    (dict(ws=None), WORKSPACE), (dict(B=1 << 20, Tq=1 << 10, columns=1), UNSUPPORTED)])
def test_attention_refuses(over, status):
    assert _attn(**over) == status
    assert binding.load().kla_last_error_message().decode() != ""


def _pages(name, **over):
    a = dict(pool=FAKE, layers=2, bytes=64, table=FAKE, lens=FAKE, refs=FAKE, src=FAKE, dst=FAKE,
             more=FAKE, where=FAKE, used=FAKE, S=3, columns=4, page=16, n_pages=10, n=2, ws=FAKE,
             wsb=1 << 40)
    a.update(over)
    pool, book = [a["pool"], a["layers"], a["bytes"]], [a["table"], a["lens"], a["refs"]]
    sizes, end = [a["S"], a["columns"], a["page"], a["n_pages"]], [a["ws"], a["wsb"], None]
    args = {"fork": [*book, a["src"], a["dst"], *sizes, a["n"]],
            "grow": [*pool, *book, a["more"], *sizes],
            "trim": [*book, a["more"], *sizes],
            "compact": [*pool, *book, a["where"], a["used"], *sizes],
            "copy": [*pool, a["src"], a["dst"], a["n_pages"], a["n"]]}
    return getattr(binding.load(), "kla_pages_" + name)(*args[name], *end)


BOOK = [(dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(refs=None), INVALID),
        (dict(table=FAKE + 2), INVALID), (dict(S=-1), INVALID), (dict(page=0), INVALID),
        (dict(columns=1 << 30), UNSUPPORTED)]
POOL = [(dict(pool=None), INVALID), (dict(pool=FAKE + 4), INVALID), (dict(layers=-1), INVALID),
        (dict(bytes=-16), INVALID), (dict(bytes=40), UNSUPPORTED), (dict(bytes=1 << 41), UNSUPPORTED)]
ENDS = [(dict(ws=None), WORKSPACE), (dict(wsb=256), WORKSPACE), (dict(ws=FAKE + 16), INVALID),
        (dict(n_pages=-1), INVALID)]


@no_gpu_only
@pytest.mark.parametrize("name,over,status", [
    *[("fork", *x) for x in BOOK + ENDS], *[("grow", *x) for x in BOOK + POOL + ENDS],
    *[("trim", *x) for x in BOOK + ENDS],
    *[("compact", *x) for x in BOOK + POOL + ENDS], *[("copy", *x) for x in POOL + ENDS],
    ("fork", dict(dst=None), INVALID), ("fork", dict(n=-1), INVALID),
    ("fork", dict(n=1 << 30), UNSUPPORTED), ("fork", dict(src=FAKE + 1), INVALID),
    ("grow", dict(more=None), INVALID), ("trim", dict(more=None), INVALID),
    ("trim", dict(more=FAKE + 2), INVALID), ("compact", dict(where=None), INVALID),
    ("compact", dict(used=None), INVALID), ("copy", dict(src=None), INVALID),
    ("copy", dict(n=-1), INVALID),
    # numbers that a thread's next one would pass in 32 bits
    *[(name, dict(n_pages=2 ** 31 - 2 ** 16), UNSUPPORTED) for name in ("fork", "grow", "trim", "compact",
                                                                         "copy")],
    ("grow", dict(S=2 ** 31 - 2 ** 16, columns=1), UNSUPPORTED),
    ("compact", dict(S=2 ** 31 - 2 ** 16, columns=1), UNSUPPORTED),
    ("trim", dict(S=2 ** 31 - 2 ** 16, columns=1), UNSUPPORTED),
    ("copy", dict(n=2 ** 31 - 2 ** 16), UNSUPPORTED),
    ("fork", dict(n=2 ** 31 - 2 ** 16, columns=0), UNSUPPORTED)])
def test_pages_refuse(name, over, status):
    assert _pages(name, **over) == status
    assert binding.load().kla_last_error_message().decode() != ""


@no_gpu_only
def test_injected_launch_fault(monkeypatch):
    monkeypatch.setenv("KLA_FAULT_INJECT", "launch")
    calls = [lambda: _rows("kla_kv4_append"), lambda: _rows("kla_kv4_read"), _attn]
    calls += [lambda n=n: _pages(n) for n in ("fork", "grow", "trim", "compact", "copy")]
    for call in calls:
        assert call() == binding.KLA_ERR_CUDA
        assert "injected" in binding.load().kla_last_error_message().decode()


def test_sizes():
    assert kla.kla_kv4_page_bytes(64, 4, 128) == 64 * 4 * 144
    for page, hk, d in ((24, 1, 64), (0, 1, 64), (16, 0, 64), (16, 1, 80)):
        assert kla.kla_kv4_page_bytes(page, hk, d) == 0
        with pytest.raises(ValueError):
            kla.kla_kv4_pool(3, page, hk, d, device="cpu")
    assert kla.kla_kv4_pool(3, 32, 2, 64, device="cpu").shape == (3, 2, 2, 18 * 64)
    assert kla.kla_kv4_pool(3, 32, 2, 64, layers=5, device="cpu").shape == (5, 3, 2, 2, 18 * 64)
    assert kla.kla_kv4_attn_workspace_size(2, 1, 4, 2, 64, 32, 4) > 256
    assert kla.kla_kv4_attn_workspace_size(2, 0, 4, 2, 64, 32, 4) == 0
    assert kla.kla_kv4_attn_workspace_size(2, 1, 3, 2, 64, 32, 4) == 0
    for sizes in ((2 ** 31 - 2 ** 16, 1, 1, 0), (1, 1, 2 ** 31 - 2 ** 16, 0), (0, 0, 1, 2 ** 31 - 2 ** 16)):
        assert kla.kla_pages_workspace_size(*sizes) == 0
    assert kla.kla_pages_workspace_size(3, 4, 100, 2) >= 256 + 4 * 100 * 4
    assert binding.load().kla_status_str(binding.KLA_ERR_PAGES) == b"not enough free pages"


def test_the_binding_refuses():
    pool, table = kla.kla_kv4_pool(3, 16, 2, 64, device="cpu"), torch.zeros(2, 4).int()
    lens, q = torch.zeros(2).int(), torch.zeros(2, 1, 4, 64)
    with pytest.raises(ValueError):
        kla.kla_kv4_attn(q, pool, table, lens)                       # not on a GPU
    with pytest.raises(ValueError, match="4|dim|shape"):
        kla.kla_kv4_attn(q[0], pool, table, lens)
    with pytest.raises(ValueError, match="total"):
        kla.kla_kv4_read(pool, table, lens)
    with pytest.raises(ValueError, match="total"):
        kla.kla_kv4_read(pool, table, lens, T=1, cu_seqlens=lens)
    with pytest.raises(ValueError, match="shape"):
        kla.kla_kv4_append(q[0], q[0], pool, table, lens)
    refs, some = torch.zeros(3).int(), torch.zeros(1).int()
    for call in (lambda: kla.kla_pages_fork(table, lens, refs, some, some, 16),
                 lambda: kla.kla_pages_free(table, lens, refs, some, 16),
                 lambda: kla.kla_pages_grow(pool[None], table, lens, refs, lens, 16),
                 lambda: kla.kla_pages_trim(table, lens, refs, lens, 16),
                 lambda: kla.kla_pages_compact(pool[None], table, lens, refs, 16),
                 lambda: kla.kla_pages_copy(pool[None], some, some),
                 lambda: kla.kla_kv4_append(q[:, :, :2], q[:, :, :2], pool, table, lens),
                 lambda: kla.kla_kv4_read(pool, table, lens, T=1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        kla.kla_kv4_append(q.half(), q.half(), pool, table, lens)


def _split(tiles, items, ctas, warps):
    """The kernel's split: tile ranges of every CTA's warps."""
    total = sum(tiles) * items
    ctas = max(1, min(ctas, -(-total // warps)))

    def cta(c):
        return total * c // ctas

    return [[cta(c) + (cta(c + 1) - cta(c)) * w // warps for w in range(warps + 1)]
            for c in range(ctas)]


def _walk(tiles, items, u, end, extra):
    """A warp's way from place u to place end as the kernel goes it: the tiles (counted without
    the extra ones) that it takes, and where its first item's first tile is."""
    y = seq = 0
    x = u // items
    while y + (tiles[seq] + extra if tiles[seq] else 0) <= x:
        y += tiles[seq] + extra if tiles[seq] else 0
        seq += 1
    item, tile = divmod(u - y * items, tiles[seq] + extra)

    def following(seq, item):
        if item + 1 < items:
            return seq, item + 1
        seq += 1
        while not tiles[seq]:
            seq += 1
        return seq, 0

    left, n, at = end - u, end - u, (seq, item)
    if extra:
        n = 0
        skip = tiles[seq] + extra - tile
        if skip <= extra:
            u, left = u + skip, left - skip
            if left > 0:
                at, tile = following(*at), 0
        p, t, rest = at, tile, left
        while rest > 0:
            some = min(rest, tiles[p[0]] - t)
            n, rest = n + some, rest - some - extra
            if rest > 0:
                p, t = following(*p), 0
    got, start = [], u - tile
    for _ in range(n):
        if tile == tiles[at[0]]:
            at, tile = following(*at), 0
        got.append((*at, tile))
        tile += 1
    return got, start


@pytest.mark.parametrize("seed", range(40))
def test_warps_take_every_tile_once(seed):
    """With extra tiles for each item and without, and a CTA's first item begins where the
    warp that has the CTA's first place says."""
    r = random.Random(seed)
    warps, ctas, extra = r.choice([8, 12]), r.choice([1, 3, 20]), seed % 4
    tiles = [r.choice([0, 1, 1, 2, r.randint(0, 9), r.randint(0, 40)]) for _ in range(r.randint(1, 30))]
    items = r.randint(1, 6)
    counted = [n + extra if n else 0 for n in tiles]
    begins, at = {}, 0
    for s, n in enumerate(tiles):
        for i in range(items):
            begins[s, i] = at
            at += counted[s]
    want = [(s, i, t) for s, n in enumerate(tiles) for i in range(items) for t in range(n)]
    got, ranges = [], _split(counted, items, ctas, warps)
    for edges in ranges:
        cta = []
        for w in range(warps):
            if edges[w] < edges[w + 1]:
                some, start = _walk(tiles, items, edges[w], edges[w + 1], extra)
                if edges[w] == edges[0] and some:
                    assert start == begins[some[0][:2]]
                cta += some
        assert cta or not any(tiles)      # an item from an earlier CTA has a part in each between
        got += cta
    assert got == want


@pytest.mark.parametrize("seed", range(24))
def test_parts_that_are_left_are_the_parts_that_are_joined(seed):
    """The model of attention's split: every tile of an item is in one part, and the CTA that
    has an item's end finds all of them."""
    r = random.Random(seed)
    warps, ctas = r.choice([8, 12, 16]), r.choice([3, 20, 152])
    tiles = [r.choice([0, 1, 2, r.randint(0, 40), r.randint(0, 900)]) for _ in range(r.randint(1, 30))]
    items = r.randint(1, 6)
    ranges = _split(tiles, items, ctas, warps)
    starts, at = [], 0
    for n in tiles:
        for _ in range(items):
            if n:
                starts.append((at, at + n))
            at += n
    done, slots, owners = {}, {}, []
    for c, edges in enumerate(ranges):
        parts = []                                   # in the order of 2 w, 2 w + 1
        for w in range(warps):
            s, e = edges[w], edges[w + 1]
            if s == e:
                continue
            for x, y in starts:
                a, b = max(s, x), min(e, y)
                if a >= b:
                    continue
                if (a, b) == (x, y):
                    assert done.setdefault((x, y), "warp") == "warp"
                else:
                    parts.append((2 * w + (b == e), (x, y), a, b))
        assert [p[0] for p in parts] == sorted({p[0] for p in parts})
        groups = []
        for p in parts:
            if groups and groups[-1][0] == p[1]:
                assert groups[-1][2] == p[2]
                groups[-1][2] = p[3]
            else:
                groups.append([p[1], p[2], p[3]])
        for (x, y), a, b in groups:
            if (a, b) == (x, y):
                assert (x, y) not in done
                done[x, y] = "cta"
                continue
            slot = (c, int(a == x))
            assert slot not in slots
            slots[slot] = ((x, y), a, b)
            if a != x and b == y:
                first = next(z for z in range(len(ranges)) if ranges[z][0] <= x < ranges[z][-1])
                owners.append(((x, y), first, c))
    for item, first, last in owners:
        assert item not in done
        done[item] = "join"
        found = [slots.pop((c, int(c == first))) for c in range(first, last + 1)]
        assert all(f[0] == item for f in found)
        assert [f[1] for f in found[1:]] == [f[2] for f in found[:-1]]
        assert (found[0][1], found[-1][2]) == item
    assert not slots and set(done) == set(starts)
    assert len({c for _, _, c in owners}) == len(owners)


class Elsewhere:
    """A tensor that says it is on a device."""

    def __init__(self, t, device=0):
        self.t, self.at = t, device

    def get_device(self):
        return self.at

    @property
    def is_cuda(self):
        return self.at >= 0

    @property
    def device(self):
        return torch.device("cuda", self.at) if self.at >= 0 else torch.device("cpu")

    def __getattr__(self, name):
        x = getattr(self.t, name)
        if name in ("double", "repeat", "expand", "transpose"):
            return lambda *a: Elsewhere(x(*a), self.at)
        return x

    def __getitem__(self, key):
        return Elsewhere(self.t[key], self.at)


def test_the_binding_refuses_wrong_tensors(monkeypatch):
    """Right arguments reach the library with their sizes; wrong ones are refused before it."""
    reached = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 0
            return lambda *a: reached.append(name) or 0

    monkeypatch.setattr(cache, "load", Library)
    monkeypatch.setattr(cache, "_size", lambda *a: 0)
    monkeypatch.setattr(cache, "_empty", lambda size, steps, dtype: Elsewhere(torch.empty(size, dtype=dtype)))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    base = _cache.arguments(Elsewhere)
    for name, args in base["calls"].items():
        getattr(kla, name)(**args)
    assert reached == list(base["calls"])
    for name, args, key, bad in _cache.wrong_arguments(base, lambda t: Elsewhere(t.t, -1)):
        with pytest.raises((ValueError, TypeError)):
            getattr(kla, name)(**{**args, key: bad})
            raise AssertionError((name, key, bad.shape, bad.dtype, bad.at))
