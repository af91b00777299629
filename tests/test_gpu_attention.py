"""Causal attention against its definition in 64 bits, element by element.

Tolerances, with u = 2^-24, h = half a step of the inputs' type (bf16 2^-8,
fp32 u): a score is a chain of d fp32 products, off by at most
e = (d + 8) u max_ij sum_c |q_ic k_jc| scale; p is off by 2 e relative and, as
an operand of the next product, rounded once (h); a sum of n terms adds n u.
    o   : (h + 2 e + n u) P |V| + h |o|
    lse : 2 e + 1e-6 (exponential and logarithm) + 4 u |lse|
    dS  : scale P ((h + 2 e) |dP - delta| + d u max sum |dO V| + (h + d u) sum |dO o|)
          (delta is taken from the rounded o)
    dq  : that times |K| + n u |dS| |K| + h |dq|, dk alike
    dv  : (h + 2 e + n u) P^T |dO| + h |dv|
The join of a split key axis adds nothing of that size (its parts are fp32)."""
import math

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla
from gated_delta_rule_kaczmarz_gb300 import binding

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def _half(t):
    return 2.0 ** -8 if t == BF16 else U


def _inputs(nq, nk, hq, hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(dtype)

    return normal(nq, hq, d), normal(nk, hk, d), normal(nk, hk, d), normal(nq, hq, d)


def _ref(q, k, v, go, scale):
    """One sequence, 64 bits: values and tolerances of o, lse, dq, dk, dv."""
    dtype, (nq, hq, d), (nk, hk, _) = q.dtype, q.shape, k.shape
    h, G = _half(dtype), hq // hk
    q, go = (x.double().unflatten(1, (hk, G)).permute(1, 2, 0, 3) for x in (q, go))
    k, v = (x.double().transpose(0, 1)[:, None] for x in (k, v))
    seen = torch.arange(nk) <= torch.arange(nq)[:, None] + nk - nq
    s = (q @ k.mT * scale).masked_fill(~seen, -math.inf)
    lse = s.logsumexp(-1, keepdim=True) if nk else torch.full((hk, G, nq, 1), -math.inf).double()
    p = torch.where(seen, (s - lse.clamp_min(-1e300)).exp(), 0.0)
    o = p @ v
    e = (d + 8) * U * float((q.abs() @ k.abs().mT).max() if nk and nq else 0) * scale
    n = nk * U
    out = {"o": (o, (h + 2 * e + n) * (p @ v.abs()) + h * o.abs()),
           "lse": (lse[..., 0], torch.full_like(lse[..., 0], 2 * e + 1e-6)
                   + 4 * U * lse[..., 0].abs().nan_to_num(posinf=0))}
    dp = go @ v.mT
    delta = (go * o).sum(-1, keepdim=True)
    ds = p * (dp - delta) * scale
    # the forward's o as the backward gets it is within its tolerance of o
    dsum = (go.abs() * (out["o"][1] + (h + d * U) * o.abs())).sum(-1, keepdim=True)
    dots = d * U * float((go.abs() @ v.abs().mT).max() if nk and nq else 0)
    ts = scale * p * ((h + 2 * e) * (dp - delta).abs() + dots + dsum) + n * ds.abs()
    m = nq * G * U
    dq, tq = ds @ k, ts @ k.abs()
    dk = (ds.mT @ q).sum(1)
    tk = ((ts + m * ds.abs()).mT @ q.abs()).sum(1)
    dv = (p.mT @ go).sum(1)
    tv = ((h + 2 * e + m) * p.mT @ go.abs()).sum(1)
    out |= {"dq": (dq, tq + h * dq.abs()), "dk": (dk, tk + h * dk.abs()),
            "dv": (dv, tv + h * dv.abs())}
    rows = {"o": 0, "lse": 0, "dq": 0}
    return {x: tuple((t.permute(2, 0, 1, *range(3, t.dim())).flatten(1, 2) if x in rows
                      else t.transpose(0, 1)) for t in pair) for x, pair in out.items()}


def _check(got, ref, what):
    want, tol = ref
    got = got.cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    hard = ~torch.isfinite(want)
    assert torch.equal(got[hard], want[hard]), what
    off = ((got - want).abs() - tol)[~hard]
    assert off.numel() == 0 or float(off.max()) <= 0, (what, float(off.max()))


CASES = [
    # B, Tq, Tk, Hq, Hk, d
    (1, 1, 1, 1, 1, 64),
    (2, 1, 300, 8, 2, 128),       # single tokens over a cache
    (3, 1, 2000, 16, 4, 64),      # the same, split over the keys
    (1, 2, 5000, 4, 1, 128),
    (2, 64, 64, 2, 2, 64),
    (1, 129, 129, 4, 4, 128),
    (2, 257, 257, 6, 2, 64),      # three heads a group
    (1, 100, 37, 4, 2, 128),      # queries that see nothing
    (2, 37, 100, 7, 1, 128),      # seven heads a group, a chunk of a prompt
    (1, 300, 300, 16, 1, 64),
    (1, 640, 640, 2, 2, 128),
    (1, 1100, 1100, 8, 2, 128),
    (3, 5, 700, 5, 5, 64),
    (1, 3, 200, 160, 1, 64),      # a group larger than a tensor-core tile
    (40, 130, 130, 8, 4, 64),     # more tiles than SMs
    (1, 70, 0, 2, 1, 64),         # no keys
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", CASES)
def test_batches(case, dtype):
    B, Tq, Tk, hq, hk, d = case
    data = [_inputs(Tq, Tk, hq, hk, d, dtype, seed=B * Tq + Tk + b) for b in range(B)]
    q, k, v, go = (torch.stack(x).cuda() for x in zip(*data))
    o, lse = kla.kla_attn_fwd(q, k, v)
    grads = kla.kla_attn_bwd(q, k, v, o, lse, go)
    torch.cuda.synchronize()
    for b in {0, B // 2, B - 1}:
        ref = _ref(*data[b], 1 / math.sqrt(d))
        for what, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            _check(got[b], ref[what], what)


PACKED = [
    # lengths of queries, lengths of keys (None: the same), Hq, Hk, d
    ([1], None, 2, 1, 64),
    ([5, 0, 129, 1, 64, 300], None, 8, 2, 128),
    ([0, 0, 7], None, 3, 3, 64),
    ([1, 1, 1, 1], [500, 3, 0, 1290], 8, 1, 128),
    ([20, 0, 90, 3], [10, 50, 400, 3], 6, 2, 64),
    ([200] * 30, None, 4, 4, 64),
    ([700, 128, 127, 129, 256], None, 12, 4, 128),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", PACKED)
def test_packed(case, dtype):
    lq, lk, hq, hk, d = case
    lk = lq if lk is None else lk
    data = [_inputs(a, b, hq, hk, d, dtype, seed=a + 7 * b + i)
            for i, (a, b) in enumerate(zip(lq, lk))]
    q, k, v, go = (torch.cat(x).cuda() for x in zip(*data))
    cu_q = torch.tensor([0] + lq).cumsum(0).int().cuda()
    cu_k = None if lk is lq else torch.tensor([0] + lk).cumsum(0).int().cuda()
    scale = 0.11
    o, lse = kla.kla_attn_fwd_varlen(q, k, v, cu_q, cu_k, scale, check_status=True)
    grads = kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu_q, cu_k, scale, check_status=True)
    aq = ak = 0
    for part, a, b in zip(data, lq, lk):
        ref = _ref(*part, scale) if a or b else {}
        for what, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            if ref:
                got = got[ak:ak + b] if what in ("dk", "dv") else got[aq:aq + a]
                _check(got, ref[what], what)
        aq, ak = aq + a, ak + b


@pytest.mark.parametrize("d", [64, 128])
def test_many_short_sequences(d):
    """Items of one key tile one after another, every one with a neighbour's
    rows in its last tile: the loads run several items ahead of the products."""
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(1, 41, (1500,), generator=g).tolist()
    hq, hk = 8, 4
    data = [_inputs(n, n, hq, hk, d, BF16, seed=i) for i, n in enumerate(lens)]
    q, k, v, go = (torch.cat(x).cuda() for x in zip(*data))
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    for _ in range(3):
        o, lse = kla.kla_attn_fwd_varlen(q, k, v, cu, check_status=True)
        grads = kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu, check_status=True)
    at = 0
    for i, n in enumerate(lens):
        if i % 37 == 0:
            ref = _ref(*data[i], 1 / math.sqrt(d))
            for what, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
                _check(got[at:at + n], ref[what], what)
        at += n


@pytest.mark.parametrize("d", [64, 128])
def test_many_calls_end_and_give_the_same_bits(d):
    """Every wait of the backward pass's roles, a few million times: one that
    missed its phase would run out and set the status word."""
    lens = [1500, 37, 900, 1, 260, 1100, 640, 5]
    data = [_inputs(n, n, 12, 4, d, BF16, seed=80 + i) for i, n in enumerate(lens)]
    q, k, v, go = (torch.cat(x).cuda() for x in zip(*data))
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    o, lse = kla.kla_attn_fwd_varlen(q, k, v, cu, check_status=True)
    first = kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu, check_status=True)
    for _ in range(400):
        o2, lse2 = kla.kla_attn_fwd_varlen(q, k, v, cu, check_status=True)
        grads = kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu, check_status=True)
    for x, y in zip((o, lse, *first), (o2, lse2, *grads)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("hq, hk, d", [(8, 4, 64), (2, 2, 128), (160, 1, 64)])
def test_rows_with_one_key_have_no_score_gradient(hq, hk, d):
    """p is 1, so dS = p (dp - p dp) is zero but for fp32: both dp are off by
    d u sum |dO V|, both p by 2 e, and nothing that was rounded to bf16 is in it."""
    lens = [1, 130, 1, 0, 1, 1, 40, 1]
    data = [_inputs(n, n, hq, hk, d, BF16, seed=50 + i) for i, n in enumerate(lens)]
    q, k, v, go = (torch.cat(x).cuda() for x in zip(*data))
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    o, lse = kla.kla_attn_fwd_varlen(q, k, v, cu, check_status=True)
    dq, dk, _ = kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu, check_status=True)
    scale, at = 1 / math.sqrt(d), 0
    for i, n in enumerate(lens):
        qq, kk, vv, gg = (x.double() for x in data[i])
        if n:
            qq, gg = (x[0].reshape(hk, hq // hk, d) for x in (qq, gg))     # the first row
            kk, vv = kk[0][:, None], vv[0][:, None]
            e = (d + 8) * U * (qq.abs() * kk.abs()).sum(-1, keepdim=True) * scale + 1e-6
            dots = (gg.abs() * vv.abs()).sum(-1, keepdim=True)
            ds = scale * (2 * d * U + 4 * e) * dots * (1 + 2.0 ** -6)
            got = dq[at].cpu().double().reshape(hk, hq // hk, d)
            assert (got.abs() <= ds * kk.abs()).all(), i
            if n == 1:
                assert (dk[at].cpu().double().abs() <= (ds * qq.abs()).sum(1)).all(), i
        at += n


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tq", [1, 3, 150])
def test_padded_cache_with_anything_behind_its_lengths(dtype, tq):
    B, Tk, hq, hk, d = 5, 600, 8, 2, 128
    lens = [600, 1, 0, 333, 128]
    data = [_inputs(tq, Tk, hq, hk, d, dtype, seed=b) for b in range(B)]
    q, k, v, _ = (torch.stack(x).cuda() for x in zip(*data))
    for b, n in enumerate(lens):
        k[b, n:] = math.nan
        v[b, n:] = math.inf
    o, lse = kla.kla_attn_fwd(q, k, v, k_lens=torch.tensor(lens).int().cuda())
    for b, n in enumerate(lens):
        qq, kk, vv, gg = data[b]
        ref = _ref(qq, kk[:n], vv[:n], gg, 1 / math.sqrt(d))
        _check(o[b], ref["o"], "o")
        _check(lse[b], ref["lse"], "lse")
    wild = torch.tensor([700, 1, -5, 333, 128]).int().cuda()    # clamped to 0..Tk
    o2, _ = kla.kla_attn_fwd(q, k, v, k_lens=wild)
    assert torch.equal(o2, o)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_neighbour_that_is_not_finite_does_not_leak(dtype):
    lens, hq, hk, d = [70, 61, 130], 4, 2, 64
    data = [_inputs(n, n, hq, hk, d, dtype, seed=n) for n in lens]
    q, k, v, go = (torch.cat(x).cuda() for x in zip(*data))
    for x in (q, k, v, go):
        x[70:131] = math.nan
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    o, lse = kla.kla_attn_fwd_varlen(q, k, v, cu)
    grads = kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu)
    for part, at in ((0, slice(0, 70)), (2, slice(131, 261))):
        ref = _ref(*data[part], 1 / math.sqrt(d))
        for what, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            _check(got[at], ref[what], what)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_parts_of_a_projection_are_read_where_they_lie(dtype):
    B, T, hq, hk, d = 2, 190, 6, 2, 128
    x = torch.randn(B, T, (hq + 2 * hk) * d + 64, device="cuda").to(dtype)
    q = x[..., :hq * d].unflatten(-1, (hq, d))
    k = x[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    v = x[..., (hq + hk) * d:(hq + 2 * hk) * d].unflatten(-1, (hk, d))
    go = torch.randn(B, T, 2, hq, d, device="cuda").to(dtype)[:, :, 1]
    dense = [t.contiguous() for t in (q, k, v, go)]
    want = kla.kla_attn_fwd(*dense[:3])
    got = kla.kla_attn_fwd(q, k, v)
    grads = kla.kla_attn_bwd(q, k, v, *got, go)
    ref = kla.kla_attn_bwd(*dense[:3], *want, dense[3])
    assert all(torch.equal(a, b) for a, b in zip((*got, *grads), (*want, *ref)))


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_that_are_only_16_byte_aligned(d):
    q, k, v, go = (x[None].cuda() for x in _inputs(200, 200, 4, 2, d, BF16, seed=12))
    want = kla.kla_attn_fwd(q, k, v)
    grads = kla.kla_attn_bwd(q, k, v, *want, go)

    def odd(t):
        return torch.full((t.numel() + 16,), 7.0, dtype=BF16, device="cuda")

    def inside(t, like):
        return t[8:8 + like.numel()].view(like.shape)          # 16 bytes behind a 512-byte block's start

    hold = [odd(x) for x in (want[0], *grads)]
    o, dq, dk, dv = (inside(t, x) for t, x in zip(hold, (want[0], *grads)))
    kla.kla_attn_fwd(q, k, v, o=o)
    kla.kla_attn_bwd(q, k, v, *want, go, dq=dq, dk=dk, dv=dv)
    for t, x, y in zip(hold, (want[0], *grads), (o, dq, dk, dv)):
        assert torch.equal(x, y)
        assert bool((t[:8] == 7).all()) and bool((t[-8:] == 7).all())


def test_offsets_past_32_bits():
    """Key rows 2^15 elements apart, 70000 of them in two sequences."""
    B, Tk, hk, d = 2, 35000, 2, 64
    far = torch.empty(B * Tk, 1 << 15, dtype=BF16, device="cuda")
    k = far[:, 64:64 + hk * d].unflatten(-1, (hk, d)).unflatten(0, (B, Tk))
    v = far[:, 4096:4096 + hk * d].unflatten(-1, (hk, d)).unflatten(0, (B, Tk))
    k.copy_(torch.randn(B, Tk, hk, d, device="cuda"))
    v.copy_(torch.randn(B, Tk, hk, d, device="cuda"))
    q = torch.randn(B, 2, 4, d, device="cuda").to(BF16)
    got = kla.kla_attn_fwd(q, k, v)
    want = kla.kla_attn_fwd(q, k.contiguous(), v.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_large_scores_and_equal_scores():
    """Scores up to hundreds (the running maximum carries them) and a row of
    equal ones (o is the mean of the values)."""
    q, k, v, go = _inputs(200, 200, 2, 2, 64, BF16, seed=1)
    q, k = (16 * q.float()).to(BF16), (4 * k.float()).to(BF16)
    o, lse = kla.kla_attn_fwd(*(x[None].cuda() for x in (q, k, v)))
    ref = _ref(q, k, v, go, 1 / 8)
    _check(o[0], ref["o"], "o")
    _check(lse[0], ref["lse"], "lse")
    zero = torch.zeros(1, 200, 2, 64, dtype=BF16, device="cuda")
    o, lse = kla.kla_attn_fwd(zero, zero, v[None].cuda())
    mean = v.double().cumsum(0) / torch.arange(1, 201)[:, None, None]
    far = (o[0].cpu().double() - mean).abs()
    absmean = v.double().abs().cumsum(0) / torch.arange(1, 201)[:, None, None]
    assert bool((far <= 2.0 ** -8 * (mean.abs() + absmean)).all())
    assert torch.allclose(lse[0, :, 0].cpu(), torch.arange(1, 201).float().log(), atol=1e-6)


@pytest.mark.parametrize("bad", [[1, 10, 20], [0, 12, 11], [0, 10, 19], [0, -3, 20],
                                 [0, 1 << 30, 20]])
def test_bad_tables_are_reported_and_nothing_is_written(bad):
    q, k, v, go = (x.cuda() for x in _inputs(20, 20, 2, 2, 64, BF16, seed=2))
    cu = torch.tensor(bad).int().cuda()
    o = torch.full_like(q, 3.0)
    lse = torch.full((20, 2), 3.0, device="cuda")
    with pytest.raises(kla.KlaError) as err:
        kla.kla_attn_fwd_varlen(q, k, v, cu, o=o, lse=lse, check_status=True)
    assert err.value.status == binding.KLA_ERR_INVALID_ARG
    assert bool((o == 3).all()) and bool((lse == 3).all())
    grads = [torch.full_like(q, 3.0) for _ in range(3)]
    with pytest.raises(kla.KlaError):
        kla.kla_attn_bwd_varlen(q, k, v, o, lse, go, cu, dq=grads[0], dk=grads[1], dv=grads[2],
                                check_status=True)
    assert all(bool((x == 3).all()) for x in grads)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_the_same_inputs_give_the_same_bits(dtype):
    q, k, v, go = (x[None].cuda() for x in _inputs(500, 500, 8, 2, 128, dtype, seed=3))
    runs = []
    for _ in range(2):
        o, lse = kla.kla_attn_fwd(q, k, v)
        runs.append((o, lse, *kla.kla_attn_bwd(q, k, v, o, lse, go)))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_another_stream_and_a_captured_graph():
    q, k, v, go = (x[None].cuda() for x in _inputs(300, 300, 4, 2, 128, BF16, seed=4))
    o, lse = kla.kla_attn_fwd(q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = torch.empty_like(o)
    kla.kla_attn_fwd(q, k, v, o=o2, stream=side)
    side.synchronize()
    assert torch.equal(o, o2)
    cu = torch.tensor([0, 100, 300]).int().cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kla.kla_attn_fwd(q, k, v)
        grads = kla.kla_attn_bwd(q, k, v, *got, go)
        packed = kla.kla_attn_fwd_varlen(q[0], k[0], v[0], cu)
    q.neg_()
    cu.copy_(torch.tensor([0, 220, 300]))
    graph.replay()
    torch.cuda.synchronize()
    want = kla.kla_attn_fwd(q, k, v)
    ref = kla.kla_attn_bwd(q, k, v, *want, go)
    again = kla.kla_attn_fwd_varlen(q[0], k[0], v[0], cu)
    assert all(torch.equal(a, b) for a, b in zip((*got, *grads, *packed), (*want, *ref, *again)))


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_a_call_on_a_given_stream_belongs_to_it(handle):
    """What the call allocates must not be a block that the current stream still
    reads: here one of the output's size, freed while its reader waits."""
    q, k, v, _ = (x[None].cuda() for x in _inputs(2048, 2048, 4, 4, 128, BF16, seed=6))
    want, _ = kla.kla_attn_fwd(q, k, v)
    side = torch.cuda.Stream()
    ones = torch.ones_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                 # about 10 ms
    twos = ones + 1
    del ones
    got, _ = kla.kla_attn_fwd(q, k, v, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert bool((twos == 2).all()) and torch.equal(got, want)


def test_calls_at_once_on_two_streams():
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    data = [tuple(x[None].cuda() for x in _inputs(n, n, 4, 2, 64, BF16, seed=n)) for n in (900, 333)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for side, (q, k, v, go), g in zip(sides, data, got):
            with torch.cuda.stream(side):
                o, lse = kla.kla_attn_fwd(q, k, v)
                g.append((o, lse, *kla.kla_attn_bwd(q, k, v, o, lse, go)))
    torch.cuda.synchronize()
    for (q, k, v, go), g in zip(data, got):
        o, lse = kla.kla_attn_fwd(q, k, v)
        want = (o, lse, *kla.kla_attn_bwd(q, k, v, o, lse, go))
        assert all(torch.equal(x, y) for run in g for x, y in zip(run, want))


@pytest.mark.parametrize("case", [(2, 5, 300, 128, 1, 64), (1, 3, 150, 100, 1, 128),
                                  (1, 140, 140, 130, 2, 64)])
def test_groups_that_fill_a_tile(case):
    test_batches(case, BF16)


def test_a_second_derivative_is_refused():
    q, k, v, _ = (x.cuda().requires_grad_() for x in _inputs(20, 20, 2, 1, 64, FP32, seed=9))
    cu = torch.tensor([0, 20]).int().cuda()
    dq, = torch.autograd.grad(kla.kla_attn(q, k, v, cu_seqlens_q=cu).square().sum(), q,
                              create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dq.sum(), k)


def test_a_captured_training_step_follows_its_inputs():
    q, k, v, go = (x[None].cuda() for x in _inputs(150, 150, 4, 2, 64, BF16, seed=14))
    w = torch.ones(64, device="cuda")
    pos, freq = torch.arange(150).int().cuda()[None], torch.rand(32).cuda()
    leaves = [x.requires_grad_() for x in (q, k, v, w)]

    def step():
        o = kla.kla_attn(*kla.kla_qk_norm_rope(q, k, pos, freq, w, w), v)
        return (o.detach(), *torch.autograd.grad(o, leaves, go))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        q.mul_(0.5)
        go.neg_()
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(got, step()))


def test_prompt_then_single_tokens_equal_the_whole_prompt():
    """The cache as it is used: a prompt, then tokens one at a time over the
    growing cache, against the whole sequence at once."""
    T, hq, hk, d = 140, 8, 2, 128
    q, k, v, go = (x[None].cuda() for x in _inputs(T, T, hq, hk, d, BF16, seed=5))
    ref = _ref(*(x[0].cpu() for x in (q, k, v, go)), 1 / math.sqrt(d))
    cache_k, cache_v = torch.zeros(1, 512, hk, d, device="cuda").to(BF16), None
    cache_v = torch.full_like(cache_k, math.nan)
    cache_k[:, :130], cache_v[:, :130] = k[:, :130], v[:, :130]
    lens = torch.tensor([130]).int().cuda()
    o, _ = kla.kla_attn_fwd(q[:, :130], cache_k, cache_v, k_lens=lens)
    rows = [o[0]]
    for t in range(130, T):
        cache_k[:, t], cache_v[:, t] = k[:, t], v[:, t]
        lens += 1
        rows.append(kla.kla_attn_fwd(q[:, t:t + 1], cache_k, cache_v, k_lens=lens)[0][0])
    _check(torch.cat(rows), ref["o"], "o")


def test_conditioning_and_attention_together_under_autograd():
    """A hybrid stack's attention layer as it is trained: projection, norms and
    rotation, attention; the projection's gradient against 64 bits."""
    B, T, hq, hk, d = 2, 96, 4, 2, 64
    g = torch.Generator().manual_seed(6)
    x = torch.randn(B, T, (hq + 2 * hk) * d, generator=g)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g) for _ in range(2))
    go = torch.randn(B, T, hq, d, generator=g)
    pos = torch.arange(T).int().expand(B, T).contiguous()
    freq = (100.0 ** (-torch.arange(32) / 32.0)).float()

    def parts(y):
        return (y[..., :hq * d].unflatten(-1, (hq, d)),
                y[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d)),
                y[..., (hq + hk) * d:].unflatten(-1, (hk, d)))

    leaves = [t.cuda().requires_grad_() for t in (x, wq, wk)]
    q, k, v = parts(leaves[0])
    q, k = kla.kla_qk_norm_rope(q, k, pos.cuda(), freq.cuda(), leaves[1], leaves[2])
    o = kla.kla_attn(q, k, v)
    grads = torch.autograd.grad((o * go.cuda()).sum(), leaves)
    ref = [t.double().requires_grad_() for t in (x, wq, wk)]
    q, k, v = parts(ref[0])
    ang = (pos.double()[..., None] * freq.double())[..., None, :]

    def condition(y, w):
        y = y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = y[..., :32], y[..., 32:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    q, k = condition(q, ref[1]), condition(k, ref[2])
    k, v = (t.repeat_interleave(hq // hk, 2) for t in (k, v))
    s = torch.einsum("bihd,bjhd->bhij", q, k) / 8
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -math.inf)
    y = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v)
    want = torch.autograd.grad((y * go.double()).sum(), ref)
    assert float((o.detach().cpu() - y.detach()).abs().max()) <= 1e-4
    for a, b in zip(grads, want):
        # sums of at most B T hq products in fp32: 1e-4 of the largest value
        assert float((a.cpu().double() - b).abs().max()) <= 1e-4 * float(b.abs().max())


def test_gradients_against_differences():
    lens = [9, 0, 30]
    data = [_inputs(n, n, 4, 2, 64, FP32, seed=50 + n) for n in lens]
    q, k, v, go = (torch.cat(x).cuda() for x in zip(*data))
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]

    def loss(*x):
        return (kla.kla_attn(*x, cu_seqlens_q=cu).double() * go).sum()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    g = torch.Generator().manual_seed(2)
    for i in range(3):
        way = torch.randn(leaves[i].shape, generator=g).cuda()
        h, ends = 1e-2, []
        for sign in (h, -h):
            moved = [x.detach() for x in leaves]
            moved[i] = moved[i] + sign * way
            ends.append(float(loss(*moved)))
        want = (ends[0] - ends[1]) / (2 * h)
        got = float((grads[i].double() * way).sum())
        # third-order terms of h^2 = 1e-4, fp32 rounding of the outputs over 2 h
        assert abs(got - want) <= 5e-3 * (abs(want) + 10)


def test_no_queries_zeroes_the_key_gradients():
    _, k, v, _ = (x.cuda() for x in _inputs(1, 40, 2, 2, 64, BF16, seed=7))
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    cu_q, cu_k = torch.zeros(2).int().cuda(), torch.tensor([0, 40]).int().cuda()
    o, lse = kla.kla_attn_fwd_varlen(q, k, v, cu_q, cu_k)
    dq, dk, dv = kla.kla_attn_bwd_varlen(q, k, v, o, lse, q, cu_q, cu_k)
    assert o.numel() == dq.numel() == 0
    assert bool((dk == 0).all()) and bool((dv == 0).all())
