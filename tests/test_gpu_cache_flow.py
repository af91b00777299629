"""The paged 4-bit cache as a program uses it: prompts and decode steps beside the
dense attention, beams that fork with KLA's states, compaction under way, captured
steps, other streams, workspaces shared by captured graphs, pools beyond 32 bits."""
import math
import time

import pytest
import torch

import _cache
import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding
from gated_delta_rule_kaczmarz_gb300.workloads import decode_inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


class Cache:
    """One layer's cache for S sequences, and the same rows as dense tensors of the
    rounded values."""

    def __init__(self, S, columns, page, n_pages, hk, d, units=(1.0, 0.5)):
        self.pool = kla.kla_kv4_pool(n_pages, page, hk, d, layers=1)
        self.pool.copy_(_cache.garbage(*self.pool.shape))
        self.book = (torch.full((S, columns), -1, dtype=torch.int32, device="cuda"),
                     torch.zeros(S, dtype=torch.int32, device="cuda"),
                     torch.zeros(n_pages, dtype=torch.int32, device="cuda"))
        self.page, self.units = page, dict(k_unit=units[0], v_unit=units[1])
        self.rows = [[torch.zeros(0, hk, d, dtype=torch.float64)] * 2 for _ in range(S)]

    def grow(self, more):
        kla.kla_pages_grow(self.pool, *self.book, _ints(more), self.page, check_status=True)

    def keep(self, s, k, v):
        """Rows that were appended to sequence s."""
        self.rows[s] = [torch.cat([old, _cache.rounded(x.cpu(), u)])
                        for old, x, u in zip(self.rows[s], (k, v), self.units.values())]

    def check(self, q, o, lse, scale):
        (B, Tq, hq, _), hk, columns = q.shape, self.pool.shape[2], self.book[0].shape[1]
        other = _cache.unpacked(B, Tq, hq, hk, self.page, columns, q.dtype)
        for s in range(len(q)):
            k, v = self.rows[s]
            for got, (want, tol) in zip((o[s], lse[s]), _cache.attention(q[s].cpu(), k, v, scale, other)):
                hard = ~torch.isfinite(want)
                got = got.cpu().double()
                assert torch.equal(got[hard], want[hard])
                assert bool(((got - want).abs() <= tol)[~hard].all()), s


def test_prompts_then_steps_then_beams():
    S, columns, page, hq, hk, d = 6, 9, 16, 4, 2, 64
    c = Cache(S, columns, page, 40, hk, d)
    table, lens, refs = c.book
    scale = 0.2
    # prompts of the first two sequences, packed; their attention is the dense one
    new = [37, 0, 16, 0, 0, 0]
    c.grow(new)
    cu = _ints([0] + new).cumsum(0).int()
    k, v = _normal(53, hk, d, seed=1), _normal(53, hk, d, seed=2)
    kla.kla_kv4_append(k, v, c.pool[0], table, lens, cu_seqlens=cu, **c.units, check_status=True)
    c.keep(0, k[:37], v[:37])
    c.keep(2, k[37:], v[37:])
    states = torch.randn(S, 2, 64, 64, device="cuda")
    held = states.clone()
    for step in range(12):
        if step == 3:       # sequence 0 forks to 1 and 3, 2 to 4; KLA's states go with them
            src, dst = _ints([0, 0, 2]), _ints([1, 3, 4])
            kla.kla_pages_fork(*c.book, src, dst, page, check_status=True)
            kla.kla_pages_copy(states[None], src, dst, check_status=True)
            held[[1, 3, 4]] = held[[0, 0, 2]]
            for a, b in ((0, 1), (0, 3), (2, 4)):
                c.rows[b] = list(c.rows[a])
        if step == 6:       # beams take their parents: a permutation with a repeat; 2 ends
            src, dst = _ints([3, 0, 3, -1]), _ints([0, 1, 3, 2])
            kla.kla_pages_fork(*c.book, src, dst, page, check_status=True)
            old = [list(r) for r in c.rows]
            for a, b in ((3, 0), (0, 1), (3, 3)):
                c.rows[b] = list(old[a])
            c.rows[2] = [x[:0] for x in c.rows[2]]
        if step == 8:
            kla.kla_pages_compact(c.pool, *c.book, page, check_status=True)
        more = [int(len(r[0]) > 0) for r in c.rows]
        c.grow(more)
        k, v, q = (_normal(S, 1, h, d, seed=10 * step + i) for i, h in ((3, hk), (4, hk), (5, hq)))
        cu = _ints([0] + more).cumsum(0).int()
        on = torch.tensor(more).bool().cuda()
        kla.kla_kv4_append(k[on][:, 0], v[on][:, 0], c.pool[0], table, lens, cu_seqlens=cu,
                           **c.units, check_status=True)
        for s, n in enumerate(more):
            if n:
                c.keep(s, k[s], v[s])
        assert lens.tolist() == [len(r[0]) for r in c.rows]
        want = _cache.counted(table.tolist(), lens.tolist(), page, refs.numel())
        assert refs.tolist() == want
        o, lse = kla.kla_kv4_attn(q, c.pool[0], table, lens, scale=scale, **c.units, check_status=True)
        c.check(q, o, lse, scale)
    assert torch.equal(states, held)
    kla.kla_pages_free(*c.book, _ints(list(range(S))), page, check_status=True)
    assert not refs.any() and not lens.any() and bool((table == -1).all())


def test_drafted_tokens():
    """Rows of drafted tokens go in, attention goes over all of them, and those that were not
    taken are given up: across pages' ends, with a prefix that another sequence holds too."""
    S, page, hq, hk, d, draft = 4, 16, 4, 2, 64, 5
    c = Cache(S, 12, page, 30, hk, d)
    table, lens, refs = c.book
    c.grow([30, 0, 16, 7])
    k, v = _normal(53, hk, d, seed=1), _normal(53, hk, d, seed=2)
    cu = _ints([0, 30, 30, 46, 53])
    kla.kla_kv4_append(k, v, c.pool[0], table, lens, cu_seqlens=cu, **c.units, check_status=True)
    for s, (a, b) in enumerate(((0, 30), (30, 30), (30, 46), (46, 53))):
        c.keep(s, k[a:b], v[a:b])
    kla.kla_pages_fork(*c.book, _ints([0]), _ints([1]), page, check_status=True)
    c.rows[1] = list(c.rows[0])
    for step, taken in enumerate(([1, 5, 2, 3], [0, 1, 4, 0], [5, 5, 0, 2], [2, 0, 3, 1])):
        c.grow([draft] * S)
        k, v, q = (_normal(S, draft, h, d, seed=10 * step + i) for i, h in ((3, hk), (4, hk), (5, hq)))
        kla.kla_kv4_append(k, v, c.pool[0], table, lens, **c.units, check_status=True)
        before = [list(r) for r in c.rows]
        for s in range(S):
            c.keep(s, k[s], v[s])
        o, lse = kla.kla_kv4_attn(q, c.pool[0], table, lens, scale=0.2, **c.units, check_status=True)
        c.check(q, o, lse, 0.2)
        kla.kla_pages_trim(*c.book, _ints([draft - n for n in taken]), page, check_status=True)
        c.rows = before
        for s, n in enumerate(taken):
            c.keep(s, k[s, :n], v[s, :n])
        assert lens.tolist() == [len(r[0]) for r in c.rows]
        assert refs.tolist() == _cache.counted(table.tolist(), lens.tolist(), page, refs.numel())
        q = _normal(S, 1, hq, d, seed=10 * step + 6)
        o, lse = kla.kla_kv4_attn(q, c.pool[0], table, lens, scale=0.2, **c.units, check_status=True)
        c.check(q, o, lse, 0.2)


def test_beside_the_dense_attention():
    """A cache's rows read back and given to kla_attn_fwd: the same within both tolerances."""
    B, n, hq, hk, d, page = 3, 400, 8, 2, 128, 64
    c = Cache(B, 90, page, 25, hk, d)             # (100 tokens: unpacked)
    c.grow([n] * B)
    k, v, q = (_normal(B, n, h, d, seed=i) for i, h in ((1, hk), (2, hk), (3, hq)))
    kla.kla_kv4_append(k, v, c.pool[0], *c.book[:2], **c.units)
    kk, vv = kla.kla_kv4_read(c.pool[0], *c.book[:2], T=n, **c.units)
    for Tq in (1, 5, 100):
        want, _ = kla.kla_attn_fwd(q[:, :Tq].contiguous(), kk, vv)
        got, _ = kla.kla_kv4_attn(q[:, :Tq].contiguous(), c.pool[0], *c.book[:2], **c.units)
        # each within 2^-8 of P|V| and half a step of its size (2^-8 |o|)
        p_v = vv.double().abs().amax(1).repeat_interleave(hq // hk, 1)[:, None]
        assert bool(((got.double() - want.double()).abs() <= 2.0 ** -6 * p_v).all())


def test_conditioned_decode_beside_a_kla_mixer():
    """One token: conditioning, the attention over the cache and KLA's decode step, on views of
    one projection."""
    B, hq, hk, d, page = 4, 4, 2, 128, 16
    c = Cache(B, 4, page, 17, hk, d)
    dec = decode_inputs(B, 2, d, d, steps=3, dtype="bf16", seed=3)
    S = dec["S"].cuda()
    w, freq = torch.ones(d, device="cuda"), 100.0 ** (-torch.arange(d // 2, device="cuda") / d)
    for t in range(3):
        x = _normal(B, (hq + 2 * hk) * d, seed=t)
        q, k, v = (x[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in
                   ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
        q, k = kla.kla_qk_norm_rope_fwd(q, k, _ints([t] * B), freq, w, w)
        c.grow([1] * B)
        kla.kla_kv4_append(k[:, None], v[:, None], c.pool[0], *c.book[:2], **c.units, check_status=True)
        for s in range(B):
            c.keep(s, k[s:s + 1], v[s:s + 1])
        o, lse = kla.kla_kv4_attn(q[:, None], c.pool[0], *c.book[:2], **c.units)
        c.check(q[:, None], o, lse, d ** -0.5)
        kla.kla_decode_step(dec["q"][t].cuda(), dec["k"][t].cuda(), dec["v"][t].cuda(),
                            dec["alpha"][t].cuda(), dec["eta"][t].cuda(), dec["eps"], S)
    assert bool(torch.isfinite(S).all())


def _step(c, k, v, q, more, workspace=None):
    kla.kla_pages_grow(c.pool, *c.book, more, c.page)
    kla.kla_kv4_append(k, v, c.pool[0], *c.book[:2], **c.units)
    return kla.kla_kv4_attn(q, c.pool[0], *c.book[:2], **c.units, workspace=workspace)


@pytest.mark.parametrize("Tq,columns", [(1, 12), (40, 12), (40, 900)])       # (900: unpacked)
def test_captured_steps(Tq, columns):
    """A decode step captured once and replayed as the cache grows; two graphs on one workspace,
    one after the other."""
    B, hq, hk, d, page = 3, 8, 2, 64, 16
    caches = [Cache(B, columns, page, 40, hk, d) for _ in range(2)]
    k, v, q = (_normal(B, Tq, h, d, seed=i) for i, h in ((1, hk), (2, hk), (3, hq)))
    ks, vs, qs = (torch.empty_like(x) for x in (k, v, q))
    more = _ints([Tq] * B)
    size = kla.kla_kv4_attn_workspace_size(B, Tq, hq, hk, d, page, columns)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for c in caches:                     # warm up, then empty again
        _step(c, k, v, q, more, ws)
        kla.kla_pages_free(*c.book, _ints(list(range(B))), page)
    torch.cuda.synchronize()
    graphs = []
    for c in caches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(c, ks, vs, qs, more, ws)
        graphs.append((g, out))
    for t in range(3):
        for i, (c, (g, out)) in enumerate(zip(caches, graphs)):
            new = [_normal(B, Tq, h, d, seed=100 + 10 * t + 3 * i + j) for j, h in ((0, hk), (1, hk), (2, hq))]
            for x, y in zip((ks, vs, qs), new):
                x.copy_(y)
            g.replay()
            for s in range(B):
                c.keep(s, new[0][s], new[1][s])
            c.check(new[2], *out, d ** -0.5)


def test_streams():
    """Every call on a stream that is not the current one, with inputs that only it has ready;
    two of them at once, each with its own workspaces."""
    B, hq, hk, d, page = 5, 4, 2, 128, 16
    sides = []
    for i in range(2):
        c = Cache(B, 40, page, 210, hk, d)
        st = torch.cuda.Stream()
        sides.append((c, st, [_normal(B, 600, h, d, seed=10 * i + j) for j, h in ((0, hk), (1, hk), (2, hq))]))
    everyone, more = _ints(list(range(B))), _ints([600, 0, 30, 600, 1])
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs = []
        for c, st, (k, v, q) in sides:
            with torch.cuda.stream(st):
                torch.cuda._sleep(2000000)
                kk, vv, qq = (x + 0 for x in (k, v, q))
            kla.kla_pages_free(*c.book, everyone, page, stream=st)
            kla.kla_pages_grow(c.pool, *c.book, more, page, stream=st)
            kla.kla_kv4_append(kk, vv, c.pool[0], *c.book[:2], **c.units, stream=st)
            o, lse = kla.kla_kv4_attn(qq[:, -1:], c.pool[0], *c.book[:2], **c.units, stream=st)
            r = kla.kla_kv4_read(c.pool[0], *c.book[:2], T=600, **c.units, stream=st)
            outs.append((o, lse, r))
    torch.cuda.synchronize()
    for (c, _, (k, v, q)), (o, lse, r) in zip(sides, outs):
        for s, n in enumerate([600, 0, 30, 600, 1]):
            c.keep(s, k[s, 600 - n:], v[s, 600 - n:])
            assert torch.equal(r[0][s, 600 - n:].cpu().double(), c.rows[s][0])
        c.check(q[:, -1:], o, lse, d ** -0.5)


def test_pool_beyond_32_bits():
    """Pages whose bytes lie 4 and more GB into the pool."""
    page, hk, d = 128, 4, 128
    n_pages = (5 << 30) // kla.kla_kv4_page_bytes(page, hk, d)
    pool = torch.empty(n_pages, hk, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    n = 300
    table = _ints([[n_pages - 1, 3, n_pages - 2], [n_pages // 2, n_pages - 7, 0]])
    lens = _ints([n, n])
    k, v, q = (_normal(2, t, h, d, seed=i) for i, (t, h) in enumerate(((n, hk), (n, hk), (1, 8))))
    kla.kla_kv4_append(k, v, pool, table, lens, check_status=True)
    kk, vv = kla.kla_kv4_read(pool, table, lens, T=n, check_status=True)
    o, _ = kla.kla_kv4_attn(q, pool, table, lens, check_status=True)
    for s in range(2):
        rows = [_cache.rounded(x[s].cpu(), 1.0) for x in (k, v)]
        assert torch.equal(kk[s].cpu().double(), rows[0]) and torch.equal(vv[s].cpu().double(), rows[1])
        want, tol = _cache.attention(q[s].cpu(), *rows, d ** -0.5)[0]
        assert bool(((o[s].cpu().double() - want).abs() <= tol).all())
    kla.kla_pages_copy(pool[None], table[0, :1], _ints([n_pages - 3]), check_status=True)
    assert torch.equal(pool[n_pages - 3], pool[n_pages - 1])


@pytest.mark.parametrize("Tq,hq,dtype,columns", [(1, 4, BF16, 63), (1, 4, torch.float32, 63), (6, 4, BF16, 63),
                                                 (70, 4, BF16, 63), (70, 4, BF16, 320)])      # (320: unpacked)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_exact(monkeypatch, Tq, hq, dtype, columns):
    """No hang and no fault: with KLA_TEST_LOST_WAIT set every warp gives up its first wait."""
    B, hk, d, page = 9, 2, 128, 16
    c = Cache(B, columns, page, 600, hk, d)
    c.grow([1000, 3, 0, 640, 700, 1, 90, 900, 16])
    k, v = _normal(B, 1000, hk, d, seed=1), _normal(B, 1000, hk, d, seed=2)
    kla.kla_kv4_append(k, v, c.pool[0], *c.book[:2], **c.units)
    q = _normal(B, Tq, hq, d, seed=3).to(dtype)
    size = kla.kla_kv4_attn_workspace_size(B, Tq, hq, hk, d, page, columns, 1 if dtype == BF16 else 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    call = lambda: kla.kla_kv4_attn(q, c.pool[0], *c.book[:2], **c.units, workspace=ws, check_status=True)
    want = call()
    monkeypatch.setenv("KLA_TEST_LOST_WAIT", "1")
    t0 = time.perf_counter()
    with pytest.raises(kla.KlaError) as e:
        call()
    assert e.value.status == binding.KLA_ERR_TIMEOUT and time.perf_counter() - t0 < 5
    monkeypatch.delenv("KLA_TEST_LOST_WAIT")
    for x, y in zip(call(), want):
        assert torch.equal(x, y)


def test_many_heads():
    """1024 query heads to a key head, and 1024 key heads."""
    for hq, hk, dtype in ((1024, 1, torch.float32), (1024, 1, BF16), (1024, 1024, BF16)):
        n, d, page = 20, 64, 16
        table, lens = _ints([[1, 0]]), _ints([n])
        pool = _cache.garbage(2, hk, 1, 18 * d).cuda()
        k, v, q = (_normal(1, t, h, d, seed=i).to(dtype) for i, (t, h) in enumerate(((n, hk), (n, hk), (1, hq))))
        kla.kla_kv4_append(k, v, pool, table, lens, check_status=True)
        o, lse = kla.kla_kv4_attn(q, pool, table, lens, check_status=True)
        rows = [_cache.rounded(x[0].cpu(), 1.0) for x in (k, v)]
        for got, (want, tol) in zip((o, lse), _cache.attention(q[0].cpu(), *rows, d ** -0.5)):
            assert bool(((got[0].cpu().double() - want).abs() <= tol).all())


def test_infinities_and_nan_in_the_cache():
    """A row that is not finite reaches the queries that see it, as in the dense attention, and
    no other sequence."""
    n, hk, d, page = 40, 1, 64, 16
    table, lens = _ints([[0, 1, 2], [3, 4, 5]]), _ints([n, n])
    pool = _cache.garbage(6, hk, 1, 18 * d).cuda()
    k, v, q = (_normal(2, t, h, d, seed=i) for i, (t, h) in enumerate(((n, hk), (n, hk), (4, 2))))
    k[0, n - 2, 0, 3] = math.inf
    v[0, n - 1, 0, 5] = math.nan
    kla.kla_kv4_append(k, v, pool, table, lens)
    o, lse = kla.kla_kv4_attn(q, pool, table, lens)
    assert bool(torch.isnan(lse[0, 2:]).all()) and bool(torch.isfinite(lse[0, :2]).all())
    assert bool(torch.isfinite(o[1]).all())
