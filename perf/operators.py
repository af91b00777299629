"""Cases, plain forms and calls of the operators around the token mixer of a
hybrid stack: query and key conditioning (a norm per head and the rotary
positions, on one or several position axes) and causal softmax attention with
grouped heads over whole prompts, packed sequences and caches.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU
from a seed, ``run`` computes one pass: in elementary torch operations in 32
bits where ``own`` is false, through the framework's entry points where it is
true.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
#: the plain attention keeps at most this many scores at a time
SCORES = 1 << 30


def listed():
    return [
        # One decode token for each of 256 sequences: q and k leave the fused projection, are
        # normed and rotated at far positions, and go to the cache.  Latency counts.
        dict(name="qk_step", op="qk", train=False, dtype="bf16", rows=256, hq=16, hk=4, d=128,
             rot=128, axes=1, style="half", norm_q="rms", norm_k="rms", far=131072),
        # The prompt of a 32K-token context, one layer.
        dict(name="qk_long", op="qk", train=False, dtype="bf16", rows=32768, hq=16, hk=4, d=128,
             rot=128, axes=1, style="half", norm_q="rms", norm_k="rms", far=0),
        # A training step of a layer on B 4, T 2048: forward and backward.
        dict(name="qk_layer_train", op="qk", train=True, dtype="bf16", rows=8192, hq=16, hk=8,
             d=128, rot=128, axes=1, style="half", norm_q="rms", norm_k="rms", far=0),
        # Video frames in a prompt: time, height and width positions, an odd number of rows.
        dict(name="qk_axes", op="qk", train=False, dtype="bf16", rows=30011, hq=16, hk=16, d=128,
             rot=128, axes=3, style="half", norm_q="rms", norm_k="none", far=0),
        # A small model in fp32 with neighbouring pairs, a part of each head rotated, on two axes
        # (an image), trained; unit-norm keys as a given write strength wants them.
        dict(name="qk_axes_fp32_train", op="qk", train=True, dtype="fp32", rows=777, hq=3, hk=3,
             d=64, rot=32, axes=2, style="pairs", norm_q="rms", norm_k="l2", far=0),
        # The smallest model: B 1, H 2, T 256, d 64 in fp32, trained.
        dict(name="attn_fp32_train", op="attn", train=True, dtype="fp32", b=1, tq=256, tk=256,
             hq=2, hk=2, d=64, lens="full"),
        # The prompt of a layer, B 4, T 2048, grouped heads.
        dict(name="attn_layer", op="attn", train=False, dtype="bf16", b=4, tq=2048, tk=2048,
             hq=16, hk=4, d=128, lens="full"),
        # The whole prompt of a 32K-token context.
        dict(name="attn_long", op="attn", train=False, dtype="bf16", b=1, tq=32768, tk=32768,
             hq=16, hk=4, d=128, lens="full"),
        # 64 packed sequences of 128 to 8192 tokens.
        dict(name="attn_packed", op="packed", train=False, dtype="bf16", n=64, lo=128, hi=8192,
             hq=16, hk=4, d=128, draw=4),
        # One token each over a padded cache of long contexts, between half full and full.
        dict(name="attn_step", op="attn", train=False, dtype="bf16", b=16, tq=1, tk=32768,
             hq=16, hk=4, d=128, lens="ragged"),
        # A training step of the layer's attention: forward and backward.
        dict(name="attn_layer_train", op="attn", train=True, dtype="bf16", b=4, tq=2048, tk=2048,
             hq=16, hk=4, d=128, lens="full"),
        # Packed training at head size 64, short and odd lengths, three query heads to a group.
        dict(name="attn_packed_train", op="packed", train=True, dtype="bf16", n=37, lo=1, hi=1500,
             hq=12, hk=4, d=64, draw=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["qk", "qk_train", "attn", "step", "chunk", "train", "packed",
                       "packed_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    hq = hk * rng.choice([1, 1, 2, 3, 4, 7, 8])
    while hq > 32:
        hq -= hk
    if kind.startswith("qk"):
        rot = rng.choice([d, d, d // 2])
        return dict(op="qk", train=kind == "qk_train", dtype=dtype, rows=_log(rng, 1, 32768),
                    hq=hq, hk=hk, d=d, rot=rot, axes=rng.choice([1, 1, 2, 3]),
                    style=rng.choice(["half", "pairs"]),
                    norm_q=rng.choice(["rms", "l2", "none"]),
                    norm_k=rng.choice(["rms", "l2", "none"]),
                    far=rng.choice([0, 0, 131072, 1000003]))
    if kind.startswith("packed"):
        train = kind == "packed_train"
        top = 1 << (8 if dtype == "fp32" else 11)
        return dict(op="packed", train=train, dtype=dtype, n=rng.randint(1, 24),
                    lo=rng.randint(0, 64), hi=_log(rng, 65, top), hq=hq, hk=hk, d=d,
                    draw=rng.randrange(1 << 20))
    if kind == "step":
        return dict(op="attn", train=False, dtype=dtype, b=rng.randint(1, 64), tq=1,
                    tk=_log(rng, 1, 8192), hq=hq, hk=hk, d=d,
                    lens=rng.choice(["full", "ragged"]))
    top = 512 if dtype == "fp32" else 4096
    tq = _log(rng, 1, top)
    tk = tq if kind != "chunk" else max(1, tq + rng.randint(-tq // 4, 2 * top))
    return dict(op="attn", train=kind == "train", dtype=dtype, b=rng.randint(1, 4), tq=tq, tk=tk,
                hq=hq, hk=hk, d=d, lens="full")


def _type(case):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]


def _lengths(case):
    """Lengths of a packed case's sequences: the case's own, whatever the inputs' seed."""
    g = torch.Generator().manual_seed(case["draw"])
    x = torch.randint(case["lo"], case["hi"] + 1, (case["n"],), generator=g).tolist()
    return x if sum(x) else [1] + x[1:]


def _sections(pairs, axes):
    """Frequency pairs of each position axis: a quarter of them the first of three, the rest
    halved."""
    if axes == 1:
        return [pairs]
    if axes == 2:
        return [pairs // 2, pairs - pairs // 2]
    h = (pairs - pairs // 4) // 2
    return [pairs // 4, h, pairs - pairs // 4 - h]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, hq, hk = _type(case), case["d"], case["hq"], case["hk"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] == "qk":
        n = case["rows"]
        x = normal(n, (hq + 2 * hk) * d).to(dt)          # the fused projection's output
        s["q"] = x[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = x[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d))
        s["wq"] = 1 + 0.1 * normal(d) if case["norm_q"] != "none" else None
        s["wk"] = 1 + 0.1 * normal(d) if case["norm_k"] == "rms" else None
        pairs = case["rot"] // 2
        s["freq"] = 10000.0 ** (-torch.arange(pairs, device="cuda").float() / pairs)
        s["sections"] = _sections(pairs, case["axes"])
        if case["far"]:
            pos = torch.randint(0, case["far"], (case["axes"], n), generator=g, device="cuda")
        else:
            i = torch.arange(n, device="cuda")
            pos = torch.stack([i, i // 32 % 32, i % 32][: case["axes"]])
        s["pos"] = pos.int().contiguous()
        if case["train"]:
            s["gq"], s["gk"] = normal(n, hq, d).to(dt), normal(n, hk, d).to(dt)
        return s
    if case["op"] == "packed":
        lens = _lengths(case)
        rows = (sum(lens),)
        s["lengths"] = lens
        s["cu"] = torch.tensor([0] + lens).cumsum(0).int().cuda()
        s["q"] = normal(*rows, hq, d).to(dt)
        s["k"] = normal(*rows, hk, d).to(dt)
    else:
        b, tq, tk = case["b"], case["tq"], case["tk"]
        rows = (b, tq)
        s["q"] = normal(b, tq, hq, d).to(dt)
        s["k"] = normal(b, tk, hk, d).to(dt)
        s["k_lens"] = None
        if case["lens"] == "ragged":
            s["k_lens"] = torch.randint(tk - tk // 2, tk + 1, (b,), generator=g,
                                        device="cuda").int()
    # the values lie in the fused projection's output, the keys went through their conditioning
    x = normal(*s["k"].shape[:-2], 2 * hk * d).to(dt)
    s["v"] = x[..., hk * d:].unflatten(-1, (hk, d))
    if case["train"]:
        s["go"] = normal(*rows, hq, d).to(dt)
    return s


# ----------------------------------------------------------------- plain forms
def _norm(x, w, mode):
    """The normed rows and what the gradient takes of them: (y, x, 1 / norm)."""
    x = x.float()
    if mode == "none":
        r = torch.ones_like(x[..., :1])
    else:
        n = (x * x).sum(-1, keepdim=True)
        r = 1 / torch.sqrt((n / x.shape[-1] if mode == "rms" else n) + EPS)
    return (x * r if w is None else x * r * w), x, r


def _norm_grad(g, x, r, w, mode):
    gw = None if w is None else (g * x * r).sum((0, 1))
    g = g if w is None else g * w
    if mode == "none":
        return g, gw
    dot = (g * x).sum(-1, keepdim=True)
    dot = dot / x.shape[-1] if mode == "rms" else dot
    return r * (g - x * r * r * dot), gw


def _angles(s):
    axis = torch.arange(len(s["sections"]), device="cuda").repeat_interleave(
        torch.tensor(s["sections"], device="cuda"))
    a = s["pos"].double()[axis].T * s["freq"].double()      # far positions: 64 bits
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin, style):
    rot = 2 * cos.shape[-1]
    part, rest = x[..., :rot], x[..., rot:]
    if style == "half":
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([part, rest], -1)


def _plain_qk(s):
    dt = s["q"].dtype
    cos, sin = _angles(s)
    out, grads = [], []
    for x, w, mode, g in (("q", "wq", "norm_q", "gq"), ("k", "wk", "norm_k", "gk")):
        y, xf, r = _norm(s[x], s[w], s[mode])
        out.append(_rotate(y, cos, sin, s["style"]).to(dt))
        if s["train"]:
            back = _rotate(s[g].float(), cos, -sin, s["style"])
            gx, gw = _norm_grad(back, xf, r, s[w], s[mode])
            grads += [gx.to(dt)] + ([] if gw is None else [gw])
    return out + grads


def _plain_attend(q, k, v, k_lens, scale, go=None):
    """q [B, Tq, Hq, d], k and v [B, Tk, Hk, d]: o, lse, and with go the gradients.  Query i of
    Tq sees the keys j <= i + (keys - Tq)."""
    B, Tq, Hq, d = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    qf = q.float().unflatten(2, (Hk, Hq // Hk)).permute(0, 2, 3, 1, 4)       # B Hk G Tq d
    kf, vf = k.float().transpose(1, 2), v.float().transpose(1, 2)            # B Hk Tk d
    G = Hq // Hk
    o, lse = torch.zeros_like(qf), torch.empty_like(qf[..., 0])
    if go is not None:
        gf = go.float().unflatten(2, (Hk, G)).permute(0, 2, 3, 1, 4)
        dq, dk, dv = torch.zeros_like(qf), torch.zeros_like(kf), torch.zeros_like(vf)
    keys = (torch.full((B,), Tk, device=q.device) if k_lens is None else k_lens)[:, None, None]
    step = max(1, SCORES // max(1, B * Hq * Tk))
    for a in range(0, Tq, step):
        e = min(Tq, a + step)
        hi = Tk if k_lens is not None else max(0, min(Tk, e + Tk - Tq))      # the last key seen
        kk, vv = kf[:, :, :hi], vf[:, :, :hi]
        i = torch.arange(a, e, device=q.device)[None, :, None]
        j = torch.arange(hi, device=q.device)
        seen = (j <= i + keys - Tq)[:, None, None]
        qq = qf[:, :, :, a:e].flatten(2, 3)
        x = (qq @ kk.transpose(-1, -2)).mul_(scale).unflatten(2, (G, e - a))
        x.masked_fill_(~seen, -math.inf)
        m = x.amax(-1, keepdim=True) if hi else x.new_full((*x.shape[:-1], 1), -math.inf)
        p = x.sub_(m.clamp_min(-3e38)).exp_()
        n = p.sum(-1, keepdim=True)
        lse[:, :, :, a:e] = (m + n.log())[..., 0]
        p.div_(n.clamp_min(1e-30))
        p = p.flatten(2, 3)
        oo = p @ vv
        o[:, :, :, a:e] = oo.unflatten(2, (G, e - a))
        if go is not None:
            gg = gf[:, :, :, a:e].flatten(2, 3)
            dv[:, :, :hi] += p.transpose(-1, -2) @ gg
            dp = gg @ vv.transpose(-1, -2)
            ds = dp.sub_((gg * oo).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            dq[:, :, :, a:e] = (ds @ kk).unflatten(2, (G, e - a))
            dk[:, :, :hi] += ds.transpose(-1, -2) @ qq

    def heads(x):
        return x.permute(0, 3, 1, 2, 4).flatten(2, 3).to(q.dtype)

    out = [heads(o), lse.permute(0, 3, 1, 2).flatten(2, 3)]
    if go is not None:
        out += [heads(dq), dk.transpose(1, 2).to(q.dtype), dv.transpose(1, 2).to(q.dtype)]
    return out


def _plain_attn(s):
    scale = 1 / math.sqrt(s["d"])
    go = s.get("go")
    if s["op"] == "attn":
        return _plain_attend(s["q"], s["k"], s["v"], s["k_lens"], scale, go)
    # packed: one sequence after another, none of its rows computed for another's keys
    ins = [s[x].split(s["lengths"]) for x in ("q", "k", "v")]
    gos = [None] * len(s["lengths"]) if go is None else go.split(s["lengths"])
    outs = [_plain_attend(q[None], k[None], v[None], None, scale, None if g is None else g[None])
            for q, k, v, g in zip(*ins, gos) if len(q)]
    return [torch.cat([x[0] for x in part]) for part in zip(*outs)]


# ----------------------------------------------------------------- the framework's calls
def _own_qk(s):
    import gated_delta_rule_kaczmarz_gb300 as kla
    how = dict(wq=s["wq"], wk=s["wk"], eps=EPS, norm_q=s["norm_q"], norm_k=s["norm_k"],
               sections=s["sections"], style=s["style"])
    out = kla.kla_qk_norm_rope_fwd(s["q"], s["k"], s["pos"], s["freq"], **how)
    if not s["train"]:
        return list(out)
    gq, gk, gwq, gwk = kla.kla_qk_norm_rope_bwd(s["q"], s["k"], s["pos"], s["freq"], s["gq"],
                                                s["gk"], **how)
    return list(out) + [x for x in (gq, gwq, gk, gwk) if x is not None]


def _own_attn(s):
    import gated_delta_rule_kaczmarz_gb300 as kla
    q, k, v = s["q"], s["k"], s["v"]
    if s["op"] == "attn":
        o, lse = kla.kla_attn_fwd(q, k, v, k_lens=s["k_lens"])
        if not s["train"]:
            return [o, lse]
        return [o, lse, *kla.kla_attn_bwd(q, k, v, o, lse, s["go"])]
    o, lse = kla.kla_attn_fwd_varlen(q, k, v, s["cu"])
    if not s["train"]:
        return [o, lse]
    return [o, lse, *kla.kla_attn_bwd_varlen(q, k, v, o, lse, s["go"], s["cu"])]


def run(state):
    if state["op"] == "qk":
        return _own_qk(state) if own else _plain_qk(state)
    return _own_attn(state) if own else _plain_attn(state)


# ----------------------------------------------------------------- what a pass cannot do without
def _pairs(tq, tk):
    """(query, key) pairs of one head that the mask leaves."""
    first = max(0, tq - tk)                       # rows that see nothing
    n, low = tq - first, max(1, tk - tq + 1)
    return n * low + n * (n - 1) // 2


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    d, hq, hk = case["d"], case["hq"], case["hk"]
    if case["op"] == "qk":
        x = case["rows"] * (hq + hk) * d
        return {"bytes": x * es * (4 if case["train"] else 2) + 4 * case["rows"] * case["axes"],
                "flops": x * (24 if case["train"] else 8)}
    if case["op"] == "packed":
        lens = _lengths(case)
        nq = nk = sum(lens)
        pairs = sum(_pairs(x, x) for x in lens)
    else:
        nq, nk = case["b"] * case["tq"], case["b"] * case["tk"]
        if case["lens"] == "ragged":              # three quarters full on average
            nk = nk * 3 // 4
            pairs = case["tq"] * nk
        else:
            pairs = case["b"] * _pairs(case["tq"], case["tk"])
    many = 2 if case["train"] else 1              # q, k, v, o and their gradients
    return {"bytes": many * es * d * (2 * nq * hq + 2 * nk * hk) + 4 * nq * hq,
            "flops": (14 if case["train"] else 4) * pairs * hq * d}


# ----------------------------------------------------------------- 64 bits
def _exact_qk(s):
    out, grads = [], []
    i = 0
    turn = []
    for axis, n in enumerate(s["sections"]):
        turn.append(s["pos"][axis, :, None].double() * s["freq"][i: i + n].double())
        i += n
    turn = torch.cat(turn, 1)
    turn = torch.polar(torch.ones_like(turn), turn)
    for x, w, mode, g in (("q", "wq", "norm_q", "gq"), ("k", "wk", "norm_k", "gk")):
        leaf = s[x].double().requires_grad_()
        wl = None if s[w] is None else s[w].double().requires_grad_()
        y = leaf
        if s[mode] == "rms":
            y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt()
        elif s[mode] == "l2":
            y = y * (y.square().sum(-1, keepdim=True) + EPS).rsqrt()
        y = y if wl is None else y * wl
        p = s["rot"] // 2
        if s["style"] == "half":
            z = torch.complex(y[..., :p], y[..., p: 2 * p]) * turn[:, None]
            y = torch.cat([z.real, z.imag, y[..., 2 * p:]], -1)
        else:
            z = torch.view_as_complex(y[..., : 2 * p].unflatten(-1, (p, 2)).contiguous())
            z = torch.view_as_real(z * turn[:, None]).flatten(-2)
            y = torch.cat([z, y[..., 2 * p:]], -1)
        out.append(y.detach())
        if s["train"]:
            leaves = [leaf] + ([] if wl is None else [wl])
            grads += torch.autograd.grad(y, leaves, s[g].double())
    return out + grads


def _exact_attn(s):
    scale = s["d"] ** -0.5
    if s["op"] == "packed":
        cut = [0]
        for n in s["lengths"]:
            cut.append(cut[-1] + n)
        parts = [(slice(a, b), slice(a, b)) for a, b in zip(cut, cut[1:])]
    else:
        lens = [s["tk"]] * s["b"] if s["k_lens"] is None else s["k_lens"].tolist()
        parts = [((i, slice(None)), (i, slice(0, n))) for i, n in enumerate(lens)]
    group = s["hq"] // s["hk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    grads = [torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"]
    for at_q, at_k in parts:
        for h in range(s["hk"]):
            heads = slice(h * group, (h + 1) * group)
            q, k, v = s["q"][at_q][:, heads].double(), s["k"][at_k][:, h].double(), \
                s["v"][at_k][:, h].double()
            tq, tk = len(q), len(k)
            first = max(0, tq - tk)
            if tq == first:
                continue
            leaves = [t.requires_grad_(s["train"]) for t in (q, k, v)]
            x = torch.einsum("igd,jd->gij", q[first:], k) * scale
            hide = torch.ones(tq - first, tk, dtype=torch.bool, device="cuda").triu(
                tk - (tq - first) + 1)
            x = x.masked_fill(hide, -math.inf)
            y = torch.einsum("gij,jd->igd", x.softmax(-1), v)
            o[at_q][first:, heads] = y.detach()
            lse[at_q][first:, heads] = x.detach().logsumexp(-1).T
            if s["train"]:
                got = torch.autograd.grad(y, leaves, s["go"][at_q][first:, heads].double())
                grads[0][at_q][:, heads] = got[0]
                grads[1][at_k][:, h] = got[1]
                grads[2][at_k][:, h] = got[2]
    return [o, lse] + (grads if s["train"] else [])


def exact(case, seed):
    if case["op"] != "qk":
        # products in 64 bits run at about a trillion operations a second
        if work(case)["flops"] * 2 > 8e12:
            return None
    s = prepare(case, seed)
    return _exact_qk(s) if case["op"] == "qk" else _exact_attn(s)
