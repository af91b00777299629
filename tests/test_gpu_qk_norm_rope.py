"""Query and key conditioning against its formulas in 64 bits.

Tolerances, fp32 arithmetic with u = 2^-24: a row's sum of squares is 16
products and log2 additions deep, so 1 / norm is off by at most
(16 + 4) u / 2 + 2 u = 12 u relative, the weight and the products add 2 u,
cosine and sine 2 u each and the rotation 2 u: 20 u = 1.2e-6 of the pair's
magnitude, taken as 2e-6 of the row's largest value times sqrt 2.  A bf16
output adds half a step, 2^-8 of its value.  The gradient's row sum is as deep
and its terms cancel: 40 u of r |u|_2 + the output rounding.  A weight's
gradient of n terms: (n + 32) u of the sum of their magnitudes."""
import math

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _sections(pairs, axes):
    base = [pairs // axes] * axes
    base[-1] += pairs - sum(base)
    return base


def _inputs(tokens, hq, hk, d, dtype, rot, axes, seed, far=4096, lead=None):
    g = torch.Generator().manual_seed(seed)
    lead = (tokens,) if lead is None else lead
    pairs = rot // 2
    return dict(
        q=torch.randn(*lead, hq, d, generator=g).to(dtype),
        k=torch.randn(*lead, hk, d, generator=g).to(dtype) if hk else None,
        pos=torch.randint(-far, far, (axes, *lead), generator=g).int(),
        freq=(10000.0 ** (-torch.arange(pairs) / max(1, pairs))).float() if pairs else None,
        wq=1 + 0.2 * torch.randn(d, generator=g), wk=1 + 0.2 * torch.randn(d, generator=g),
        gq=torch.randn(*lead, hq, d, generator=g).to(dtype),
        gk=torch.randn(*lead, hk, d, generator=g).to(dtype) if hk else None)


def _ref(x, w, mode, eps, pos, freq, sections, style):
    """The definition, in 64 bits and differentiable."""
    y = x
    if mode != "none":
        n = x.square().sum(-1, keepdim=True)
        n = (n / x.shape[-1] if mode == "rms" else n) + eps
        y = x * torch.where(n == 0, 0.0, n.clamp_min(1e-300).rsqrt())
    y = y if w is None else y * w
    if freq is None:
        return y
    p = freq.numel()
    axis = torch.arange(len(sections)).repeat_interleave(torch.tensor(sections))
    ang = (pos.double()[axis].movedim(0, -1) * freq.double())[..., None, :]
    c, s = ang.cos(), ang.sin()
    if style == "half":
        a, b = y[..., :p], y[..., p:2 * p]
        turned = [a * c - b * s, b * c + a * s]
    else:
        a, b = y[..., 0:2 * p:2], y[..., 1:2 * p:2]
        turned = [torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)]
    return torch.cat([*turned, y[..., 2 * p:]], -1)


def _half_step(t):
    return torch.finfo(t).eps / 2 if t == torch.bfloat16 else 0.0


def _check(got, ref, dtype, scale, rel):
    got = got.cpu().double()
    tol = rel * scale + _half_step(dtype) * ref.abs()
    assert got.shape == ref.shape
    assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() - tol).max())


def _cuda(d):
    return {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in d.items()}


CASES = [
    # tokens, Hq, Hk, d, rot, axes, style, norm_q, norm_k, weights
    (1, 1, 1, 64, 64, 1, "half", "rms", "rms", True),
    (1, 16, 4, 128, 128, 1, "half", "rms", "none", True),
    (257, 16, 4, 128, 128, 1, "half", "rms", "rms", True),
    (300, 5, 3, 128, 64, 3, "half", "l2", "l2", True),
    (300, 5, 3, 128, 48, 4, "pairs", "rms", "l2", False),
    (77, 9, 2, 64, 32, 2, "pairs", "none", "rms", True),
    (77, 3, 0, 64, 64, 1, "pairs", "rms", "none", True),
    (65, 17, 33, 64, 0, 1, "half", "rms", "l2", True),
    (5001, 2, 1, 128, 128, 1, "half", "none", "none", False),
    (5001, 3, 7, 64, 16, 1, "half", "rms", "rms", True),
    # enough tokens for the pipelined kernel: a warp's ring turns over
    (9001, 2, 1, 128, 128, 1, "half", "rms", "rms", True),
    (9730, 5, 3, 64, 32, 3, "pairs", "l2", "none", True),
    (7297, 3, 0, 128, 64, 2, "half", "rms", "none", True),
    (9728, 1, 16, 64, 0, 1, "half", "none", "rms", False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, dtype):
    tokens, hq, hk, d, rot, axes, style, nq, nk, weights = case
    inp = _inputs(tokens, hq, hk, d, dtype, rot, axes, seed=tokens + hq)
    sections = _sections(rot // 2, axes) if rot else None
    dev = _cuda(inp)
    wq = dev["wq"] if weights else None
    wk = dev["wk"] if weights and hk else None
    how = dict(wq=wq, wk=wk, eps=1e-6, norm_q=nq, norm_k=nk, sections=sections, style=style)
    out = kla.kla_qk_norm_rope_fwd(dev["q"], dev["k"], dev["pos"], dev["freq"], **how)
    grads = kla.kla_qk_norm_rope_bwd(dev["q"], dev["k"], dev["pos"], dev["freq"], dev["gq"],
                                     dev["gk"], **how)
    torch.cuda.synchronize()
    for i, (x, w, g, mode) in enumerate((("q", "wq", "gq", nq), ("k", "wk", "gk", nk))):
        if inp[x] is None:
            assert out[i] is None and grads[i] is None and grads[2 + i] is None
            continue
        leaf = inp[x].double().requires_grad_()
        wl = inp[w].double().requires_grad_() if weights else None
        ref = _ref(leaf, wl, mode, 1e-6, inp["pos"], inp["freq"], sections, style)
        scale = ref.detach().abs().amax(-1, keepdim=True)
        _check(out[i], ref.detach(), dtype, scale, 2e-6 * math.sqrt(2))
        gx = torch.autograd.grad(ref, [leaf] + ([wl] if weights else []), inp[g].double())
        n2 = leaf.detach().square().sum(-1, keepdim=True)
        r = {"none": torch.ones_like(n2), "rms": (n2 / d + 1e-6).rsqrt(),
             "l2": (n2 + 1e-6).rsqrt()}[mode]
        top = inp[w].abs().max() if weights else 1.0
        norm = inp[g].double().norm(dim=-1, keepdim=True) * r * top
        _check(grads[i], gx[0], dtype, norm, 40 * U)
        if weights:
            # |g x r| of every term, the rotation keeping |g| of a pair
            terms = (inp[g].double().norm(dim=-1, keepdim=True)
                     * leaf.detach().abs() * r).flatten(0, -2).sum(0)
            n = tokens * leaf.shape[-2]
            _check(grads[2 + i], gx[1], torch.float32, terms, (n + 32) * U)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_far_positions_lose_nothing(dtype):
    """Positions up to the ends of int32: angles of 2e9 radians."""
    inp = _inputs(64, 2, 1, 128, dtype, 128, 1, seed=3, far=2 ** 31 - 1)
    inp["pos"][0, :3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0])
    dev = _cuda(inp)
    out = kla.kla_qk_norm_rope_fwd(dev["q"], dev["k"], dev["pos"], dev["freq"], norm_q="none",
                                   norm_k="none")
    for x, got in zip("qk", out):
        ref = _ref(inp[x].double(), None, "none", 0, inp["pos"], inp["freq"], [64], "half")
        scale = ref.abs().amax(-1, keepdim=True)
        # 2^-47 turns a position: 2 pi 2^31 / 2^47 = 1e-4 radians at the far end
        _check(got, ref, dtype, scale, 1e-4)
    near = torch.clamp(inp["pos"], -2 ** 20, 2 ** 20)
    out = kla.kla_qk_norm_rope_fwd(dev["q"], dev["k"], near.cuda(), dev["freq"], norm_q="none",
                                   norm_k="none")
    ref = _ref(inp["q"].double(), None, "none", 0, near, inp["freq"], [64], "half")
    _check(out[0], ref, dtype, ref.abs().amax(-1, keepdim=True), 2e-6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_of_a_projection_in_place_and_into_a_cache(dtype):
    B, T, hq, hk, d = 2, 37, 4, 2, 64
    inp = _inputs(B * T, hq, hk, d, dtype, 64, 1, seed=8, lead=(B, T))
    dense = _cuda(inp)
    want = kla.kla_qk_norm_rope_fwd(dense["q"], dense["k"], dense["pos"], dense["freq"],
                                    dense["wq"], dense["wk"])
    x = torch.full((B, T, (hq + 2 * hk) * d), 7.0, dtype=dtype, device="cuda")
    q = x[..., :hq * d].unflatten(-1, (hq, d))
    k = x[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    q.copy_(dense["q"])
    k.copy_(dense["k"])
    cache = torch.full((T * B, 3, hk, d), 5.0, dtype=dtype, device="cuda")
    slot = cache[:, 1].unflatten(0, (B, T))
    got = kla.kla_qk_norm_rope_fwd(q, k, dense["pos"], dense["freq"], dense["wq"], dense["wk"],
                                   k_out=slot)
    assert torch.equal(got[0], want[0]) and torch.equal(slot, want[1])
    assert bool((cache[:, 0] == 5).all()) and bool((cache[:, 2] == 5).all())
    # the gradients through the views equal those of dense rows
    args = (dense["pos"], dense["freq"], dense["gq"], dense["gk"], dense["wq"], dense["wk"])
    for a, b in zip(kla.kla_qk_norm_rope_bwd(q, k, *args),
                    kla.kla_qk_norm_rope_bwd(dense["q"], dense["k"], *args)):
        assert torch.equal(a, b)
    kla.kla_qk_norm_rope_fwd(q, k, dense["pos"], dense["freq"], dense["wq"], dense["wk"],
                             q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert bool((x[..., (hq + hk) * d:] == 7).all())     # the values stayed


def test_many_tokens_of_a_projection_in_place():
    """The pipelined kernel on strided rows: the rows of the values between
    them stay, in place equals out of place, gradients equal those of dense
    rows."""
    T, hq, hk, d = 10000, 4, 2, 128
    dt = torch.bfloat16
    inp = _cuda(_inputs(T, hq, hk, d, dt, 128, 1, seed=12))
    x = torch.full((T, (hq + 2 * hk) * d), 7.0, dtype=dt, device="cuda")
    q, k = x[:, :hq * d].unflatten(-1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    q.copy_(inp["q"])
    k.copy_(inp["k"])
    args = (inp["pos"], inp["freq"])
    want = kla.kla_qk_norm_rope_fwd(inp["q"], inp["k"], *args, inp["wq"], inp["wk"])
    grads = kla.kla_qk_norm_rope_bwd(inp["q"], inp["k"], *args, inp["gq"], inp["gk"], inp["wq"],
                                     inp["wk"])
    again = kla.kla_qk_norm_rope_bwd(q, k, *args, inp["gq"], inp["gk"], inp["wq"], inp["wk"])
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    kla.kla_qk_norm_rope_fwd(q, k, *args, inp["wq"], inp["wk"], q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert bool((x[:, (hq + hk) * d:] == 7).all())


def test_zero_rows_with_eps_zero_and_no_tokens():
    q = torch.zeros(3, 2, 64, device="cuda")
    q[1] = 1.0
    f = torch.ones(16, device="cuda")
    p = torch.arange(3, device="cuda").int()
    for mode in ("rms", "l2"):
        out, _ = kla.kla_qk_norm_rope_fwd(q, None, p, f, eps=0.0, norm_q=mode)
        assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
        assert bool(torch.isfinite(out).all())
        dq = kla.kla_qk_norm_rope_bwd(q, None, p, f, torch.ones_like(q), None, eps=0.0,
                                      norm_q=mode)[0]
        assert bool(torch.isfinite(dq).all())
    w = torch.ones(64, device="cuda")
    none = torch.empty(0, 2, 64, device="cuda")
    out, _ = kla.kla_qk_norm_rope_fwd(none, None, p[:0], f, w)
    assert out.shape == none.shape
    grads = kla.kla_qk_norm_rope_bwd(none, None, p[:0], f, none, None, w)
    assert bool((grads[2] == 0).all())


def test_rotation_keeps_the_key_norm_that_the_write_coefficient_reads():
    """norm_k none: |k| is kept, so beta = eta / (|k|^2 + eps) is what it was."""
    inp = _cuda(_inputs(100, 2, 2, 128, torch.float32, 128, 1, seed=4, far=100000))
    _, k = kla.kla_qk_norm_rope_fwd(inp["q"], inp["k"], inp["pos"], inp["freq"], norm_k="none")
    a, b = k.double().norm(dim=-1), inp["k"].double().norm(dim=-1)
    assert float(((a - b) / b).abs().max()) <= 20 * U


def test_autograd_against_differences():
    inp = _inputs(6, 2, 1, 64, torch.float32, 32, 2, seed=9)
    dev = _cuda(inp)
    leaves = [dev[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk")]
    how = dict(sections=[6, 10], style="pairs", norm_k="l2")

    def loss(q, k, wq, wk):
        a, b = kla.kla_qk_norm_rope(q, k, dev["pos"], dev["freq"], wq, wk, **how)
        return (a.double() * dev["gq"]).sum() + (b.double() * dev["gk"]).sum()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    g = torch.Generator().manual_seed(1)
    for i, leaf in enumerate(leaves):
        way = torch.randn(leaf.shape, generator=g).cuda()
        h = 1e-2
        ends = []
        for s in (h, -h):
            moved = [x.detach() for x in leaves]
            moved[i] = moved[i] + s * way
            ends.append(float(loss(*moved)))
        want = (ends[0] - ends[1]) / (2 * h)
        got = float((grads[i].double() * way).sum())
        # third-order terms of h^2 = 1e-4 and fp32 rounding of the loss over 2 h
        assert abs(got - want) <= 2e-3 * (abs(want) + 10)


def test_another_stream_and_a_captured_graph():
    inp = _cuda(_inputs(513, 4, 2, 128, torch.bfloat16, 128, 1, seed=5))
    args = (inp["q"], inp["k"], inp["pos"], inp["freq"], inp["wq"], inp["wk"])
    want = kla.kla_qk_norm_rope_fwd(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(x) for x in want]
    kla.kla_qk_norm_rope_fwd(*args, q_out=outs[0], k_out=outs[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kla.kla_qk_norm_rope_fwd(*args)
        back = kla.kla_qk_norm_rope_bwd(*args[:4], inp["gq"], inp["gk"], *args[4:])
    inp["q"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    want = kla.kla_qk_norm_rope_fwd(*args)
    ref = kla.kla_qk_norm_rope_bwd(*args[:4], inp["gq"], inp["gk"], *args[4:])
    assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*want, *ref)))


def test_conditioned_queries_and_keys_feed_the_mixer():
    """The layer as it is used: conditioned q and k into kla_chunk, all
    differentiable, against the same steps with the conditioning in 64 bits."""
    B, T, H, d = 1, 128, 2, 128
    inp = _inputs(B * T, H, H, d, torch.bfloat16, d, 1, seed=6, lead=(B, T))
    dev = _cuda(inp)
    v = torch.randn(B, T, H, d, device="cuda").bfloat16()
    gate = torch.full((B, T, H), 0.5, device="cuda")
    q, k = dev["q"].clone().requires_grad_(), dev["k"].clone().requires_grad_()
    a, b = kla.kla_qk_norm_rope(q, k, dev["pos"], dev["freq"], norm_k="l2")
    o, _ = kla.kla_chunk(a, b, v, gate, gate, 1e-6)
    o.float().sum().backward()
    ar, br = a.detach().requires_grad_(), b.detach().requires_grad_()
    o2, _ = kla.kla_chunk(ar, br, v, gate, gate, 1e-6)
    o2.float().sum().backward()
    for leaf, x, g, mode in ((q, "q", ar.grad, "rms"), (k, "k", br.grad, "l2")):
        r = inp[x].double().requires_grad_()
        y = _ref(r, None, mode, 1e-6, inp["pos"], inp["freq"], [64], "half")
        want, = torch.autograd.grad(y, r, g.cpu().double())
        n2 = r.detach().square().sum(-1, keepdim=True)
        rr = (n2 / d + 1e-6).rsqrt() if mode == "rms" else (n2 + 1e-6).rsqrt()
        _check(leaf.grad, want, torch.bfloat16, g.cpu().double().norm(dim=-1, keepdim=True) * rr,
               40 * U)
