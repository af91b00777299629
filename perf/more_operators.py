"""Cases, plain forms and calls of the paged key/value cache in 4 bits: rows
written to its pages and read back, attention over it, and the pages' own
operators (fork, growth with copies of shared pages, compaction).

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU
from a seed, ``run`` computes one pass: in elementary torch operations in 32
bits where ``own`` is false, through the framework's entry points where it is
true.  ``exact`` gives the same outputs in 64 bits.

The cache.  A page holds `page` tokens (a multiple of 16) of all key heads:
uint8 [Hk, page / 16, 18 d].  The 18 d bytes of a block are 16 tokens of one
head: keys' codes [16][d / 2] (byte i: features 2i, 2i + 1, the first in the
low four bits), values' codes [8][d] (byte i of a pair of tokens: feature i,
the even token in the low four bits), keys' scales [16][d / 16], values'
scales [d / 16][16].  A code is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
(e2m1); a scale is e4m3, one for 16 features: a value is code * scale * unit
with a power of two for all keys and one for all values.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # One decode token of 256 sequences written to caches of up to 2048 tokens, and read back:
        # latency counts.
        dict(name="rows_step", op="rows", dtype="bf16", b=256, t=1, packed=False, before=2047,
             hk=4, d=128, page=64, draw=1),
        # The prompts of 64 packed sequences of 128 to 8192 tokens, behind up to 100 cached ones.
        dict(name="rows_prompt", op="rows", dtype="bf16", b=64, t=8192, packed=True, before=100,
             hk=4, d=128, page=64, draw=4),
        # A chunk of three sequences in fp32 at head size 64, pages of 48 tokens, odd places.
        dict(name="rows_chunk_fp32", op="rows", dtype="fp32", b=3, t=333, packed=False, before=501,
             hk=3, d=64, page=48, draw=2),
        # The smallest model: one token over 256 keys, 2 heads of 64, fp32.
        dict(name="attn_small_fp32", op="attn", dtype="fp32", b=1, tq=1, lo=256, hi=256, hq=2,
             hk=2, d=64, page=16, draw=1),
        # One token each over 16 long contexts, between half full and full.
        dict(name="attn_step", op="attn", dtype="bf16", b=16, tq=1, lo=16384, hi=32768, hq=16,
             hk=4, d=128, page=64, draw=2),
        # A large decode batch over contexts of any length up to 4096.
        dict(name="attn_batch", op="attn", dtype="bf16", b=256, tq=1, lo=1, hi=4096, hq=16,
             hk=4, d=128, page=64, draw=3),
        # Five drafted tokens checked at once, three query heads to a key head, odd sizes.
        dict(name="attn_draft", op="attn", dtype="bf16", b=23, tq=5, lo=3, hi=9001, hq=9,
             hk=3, d=128, page=32, draw=5),
        # A chunk of 512 tokens of a prompt over 32768 keys.
        dict(name="attn_chunk", op="attn", dtype="bf16", b=1, tq=512, lo=32768, hi=32768, hq=16,
             hk=4, d=128, page=64, draw=1),
        # 64 prompts forked to 4 beams each, and a token of room for each beam: its last page,
        # shared until then, is copied in all of 8 layers.
        dict(name="fork_prompts", op="fork", layers=8, n_pages=3200, prompts=64, lo=100, hi=2048,
             beams=4, new=1, hk=4, d=128, page=64, draw=1),
        # A beam step of one request: 5 beams take their parents and a token of room.
        dict(name="fork_small", op="fork", layers=1, n_pages=64, prompts=1, lo=333, hi=333,
             beams=5, new=1, hk=2, d=64, page=16, draw=1),
        # A pool of 8192 pages, half of them free and scattered, compacted in 4 layers.
        dict(name="compact", op="compact", layers=4, n_pages=8192, seqs=128, lo=1000, hi=3000,
             hk=4, d=128, page=64, draw=1),
        # A small pool of small pages.
        dict(name="compact_small", op="compact", layers=2, n_pages=200, seqs=9, lo=1, hi=300,
             hk=3, d=64, page=16, draw=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "chunk", "packed", "attn1", "attn1", "attn_few", "attn_chunk",
                       "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    seed = rng.randrange(1 << 20)
    if kind in ("step", "chunk", "packed"):
        b = _log(rng, 1, 256 if kind == "step" else 32)
        t = 1 if kind == "step" else _log(rng, 2, 2048)
        return dict(op="rows", dtype=dtype, b=b, t=t, packed=kind == "packed",
                    before=_log(rng, 1, 2048), hk=hk, d=d, page=page, draw=seed)
    if kind.startswith("attn"):
        g = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
        if kind == "attn1":
            b, tq, hi = _log(rng, 1, 128), 1, _log(rng, 1, 8192)
        elif kind == "attn_few":
            b, tq, hi = _log(rng, 1, 32), rng.randint(2, 12), _log(rng, 1, 8192)
        else:
            b, tq, hi = rng.randint(1, 3), _log(rng, 13, 512), _log(rng, 13, 8192)
        if kind == "attn_chunk" and dtype == "fp32":
            tq = min(tq, 64)
        while b > 1 and (b * hi * hk > 1 << 21 or b * tq * hi * hk * g > 1 << 28):
            b //= 2
        return dict(op="attn", dtype=dtype, b=b, tq=tq, lo=rng.choice([0, hi // 2, hi]), hi=hi,
                    hq=hk * g, hk=hk, d=d, page=page, draw=seed)
    hi = _log(rng, 16, 1024)
    pages = -(-hi // page)
    layers = rng.randint(1, 4)
    if kind == "fork":
        prompts, beams = rng.randint(1, 16), rng.randint(1, 6)
        new = rng.choice([1, 1, 2, 17, 100])
        n = prompts * pages + prompts * beams * (2 + -(-new // page)) + rng.randint(0, 99)
        return dict(op="fork", layers=layers, n_pages=n, prompts=prompts, lo=rng.randint(0, hi),
                    hi=hi, beams=beams, new=new, hk=hk, d=d, page=page, draw=seed)
    seqs = rng.randint(1, 32)
    return dict(op="compact", layers=layers, n_pages=seqs * pages + rng.randint(0, 500),
                seqs=seqs, lo=rng.randint(0, hi), hi=hi, hk=hk, d=d, page=page, draw=seed)


def _type(case):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]


def _between(case, lo, hi, n, salt=0):
    """n whole numbers of lo..hi: the case's own, whatever the inputs' seed."""
    r = random.Random(case["draw"] * 8 + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _rows_lengths(case):
    """Tokens that each sequence had, and those that it gets."""
    t = case["t"]
    new = _between(case, min(128, t), t, case["b"], 1) if case["packed"] else [t] * case["b"]
    return _between(case, 0, case["before"], case["b"]), new


#: keys' and values' units: keys went through a norm, values lie in a projection's output
K_UNIT, V_UNIT = 1.0, 0.25


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def ints(t):
        return torch.tensor(t, dtype=torch.int32, device="cuda")

    def scattered(n_pages, lens, columns):
        """A table of pages that lie anywhere in the pool; -1 behind a sequence's own."""
        places = torch.randperm(n_pages, generator=g, device="cuda").int()
        held = (ints(lens) + page - 1) // page
        first = held.cumsum(0) - held
        at = torch.arange(columns, device="cuda")
        take = (first[:, None] + at).clamp_max(n_pages - 1)
        return torch.where(at < held[:, None], places[take], -1).int()

    def garbage(*shape):
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device="cuda")

    s, page, hk, d = dict(case), case["page"], case["hk"], case["d"]
    block = (hk, page // 16, 18 * d)
    if case["op"] == "rows":
        before, new = _rows_lengths(case)
        lens = [a + b for a, b in zip(before, new)]
        s["lens"], columns = ints(lens), -(-max(lens) // page)
        s["table"] = scattered(case["b"] * columns + 5, lens, columns)
        s["pool"] = garbage(case["b"] * columns + 5, *block)
        rows = (sum(new),) if case["packed"] else (case["b"], case["t"])
        s["new"] = ints(new)
        s["cu"] = ints([0] + new).cumsum(0).int() if case["packed"] else None
        x = normal(*rows, 2 * hk * d)           # the values lie in the fused projection's output
        s["k"] = (x[..., : hk * d].unflatten(-1, (hk, d)) * (1 + 3 * (torch.arange(
            d, device="cuda") % 37 == 5))).to(_type(case))       # a few large features
        s["v"] = x.mul(0.3).to(_type(case))[..., hk * d:].unflatten(-1, (hk, d))
        return s
    if case["op"] == "attn":
        b, lens = case["b"], _between(case, case["lo"], case["hi"], case["b"])
        columns = max(1, -(-case["hi"] // page))
        s["lens"] = ints(lens)
        n_pages = sum(-(-n // page) for n in lens) + 7
        s["table"] = scattered(n_pages, lens, columns)
        s["pool"] = garbage(n_pages, *block)    # what lies behind a last page's rows is anything
        s["q"] = normal(b, case["tq"], case["hq"], d).to(_type(case))
        k = normal(max(1, sum(lens)), hk, d)
        v = normal(max(1, sum(lens)), hk, d).mul_(0.3)
        if sum(lens):
            _write(s["pool"], k, v, *_places(s["table"], s["lens"], s["lens"], page))
        return s
    n_pages, beams = case["n_pages"], case.get("beams", 0)
    n = case["prompts"] if case["op"] == "fork" else case["seqs"]
    lens = _between(case, case["lo"], case["hi"], n)
    columns = -(-(case["hi"] + case.get("new", 0)) // page)
    lens += [0] * (n * beams)
    s["table"], s["lens"] = scattered(n_pages, lens, columns), ints(lens)
    held = s["table"][s["table"] >= 0].long()
    s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    s["refs"][held] = 1
    s["pool"] = garbage(case["layers"], n_pages, *block)
    if case["op"] == "fork":
        s["src"] = torch.arange(n, device="cuda").repeat_interleave(beams).int()
        s["dst"] = torch.arange(n, n + n * beams, device="cuda").int()
        s["more"] = ints([0] * n + [case["new"]] * (n * beams))
    else:
        s["table_0"], s["refs_0"] = s["table"].clone(), s["refs"].clone()
    return s


# ----------------------------------------------------------------- plain forms
def _places(table, lens, new, page):
    """Of the last new[i] tokens of every sequence, in order: page, place in it."""
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new.long())
    first = (new.long().cumsum(0) - new)[seq]
    pos = torch.arange(len(seq), device="cuda") - first + (lens - new)[seq]
    return table[seq, (pos // page).clamp_min(0)].long(), (pos % page)


def _codes(x):
    """Codes 0..15 [..., d] and scales (e4m3) [..., d / 16] of x, in 32 bits: borders are compared
    as products, which are exact."""
    x = x.unflatten(-1, (-1, 16))
    top = x.abs().amax(-1)
    scale = (top / 6).clamp_max(448).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    a = x.abs()
    code = ((a > 0.25 * s).to(torch.uint8) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s)
            + (a > 2.5 * s) + (a >= 3.5 * s) + (a > 5 * s)) * (s > 0)
    code = code + 8 * torch.signbit(x)
    return code.flatten(-2).to(torch.uint8), scale.view(torch.uint8)


def _write(pool, k, v, at, place):
    """Rows k, v [rows, Hk, d] (in units) to their pages `at` and places in them."""
    d = k.shape[-1]
    n_pages, hk, blocks, _ = pool.shape
    kc, ks = _codes(k)
    vc, vs = _codes(v)
    b, t = place // 16, place % 16
    part = pool.split([8 * d, 8 * d, d, d], -1)
    heads = torch.arange(hk, device="cuda")
    where = (at[:, None], heads, b[:, None])
    part[0].unflatten(-1, (16, d // 2))[(*where, t[:, None])] = kc[..., 0::2] | kc[..., 1::2] << 4
    part[2].unflatten(-1, (16, d // 16))[(*where, t[:, None])] = ks
    # a byte of values belongs to two tokens: the even ones, then the odd ones
    two = part[1].unflatten(-1, (8, d))
    for odd in (0, 1):
        mine = t % 2 == odd
        to = (at[mine][:, None], heads, b[mine][:, None], t[mine][:, None] // 2)
        two[to] = two[to] & (15 if odd else 240) | vc[mine] << 4 * odd
    part[3].unflatten(-1, (d // 16, 16)).transpose(-1, -2)[(*where, t[:, None])] = vs


def _read(pool, at, place, d):
    """Keys and values [rows, Hk, d] of these places, in units."""
    level = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device="cuda")
    t = (place % 16)[:, None]
    where = (at[:, None], torch.arange(pool.shape[1], device="cuda"), place[:, None] // 16)
    kc, vc, ks, vs = pool.split([8 * d, 8 * d, d, d], -1)
    k = kc.unflatten(-1, (16, d // 2))[(*where, t)]
    k = torch.stack([k & 15, k >> 4], -1).flatten(-2)
    v = vc.unflatten(-1, (8, d))[(*where, t // 2)] >> 4 * (t % 2).to(torch.uint8)[..., None] & 15
    ks = ks.unflatten(-1, (16, d // 16))[(*where, t)]
    vs = vs.unflatten(-1, (d // 16, 16)).transpose(-1, -2)[(*where, t)]
    return [(level[c.int()].unflatten(-1, (-1, 16)) * x.view(torch.float8_e4m3fn).float()[..., None])
            .flatten(-2) for c, x in ((k, ks), (v, vs))]


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(pages, d):
    """Keys and values [..., Hk, page, d] that pages [..., Hk, page / 16, 18 d] hold, in units."""
    level = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device="cuda")
    kc, vc, ks, vs = pages.split([8 * d, 8 * d, d, d], -1)
    k = torch.stack([kc & 15, kc >> 4], -1).flatten(-2).unflatten(-1, (16, d // 16, 16))
    k = level[k.int()] * ks.view(torch.float8_e4m3fn).float().unflatten(-1, (16, d // 16, 1))
    vc = vc.unflatten(-1, (8, d))
    v = torch.stack([vc & 15, vc >> 4], -2).flatten(-3, -2).unflatten(-1, (d // 16, 16))
    vs = vs.view(torch.float8_e4m3fn).float().unflatten(-1, (d // 16, 16)).transpose(-1, -2)
    return k.flatten(-2).flatten(-3, -2), (level[v.int()] * vs[..., None]).flatten(-2).flatten(-3, -2)


def _plain_rows(s):
    at, place = _places(s["table"], s["lens"], s["new"], s["page"])
    k, v = (s[x] if s["packed"] else s[x].flatten(0, 1) for x in "kv")
    _write(s["pool"], k.float() / K_UNIT, v.float() / V_UNIT, at, place)
    kk, vv = _read(s["pool"], at, place, s["d"])
    return [(x * unit).to(_type(s)).view(s["k"].shape) for x, unit in ((kk, K_UNIT), (vv, V_UNIT))]


def _plain_attn(s):
    d, hk, tq = s["d"], s["hk"], s["tq"]
    held = s["pool"][s["table"].clamp_min(0).long()]               # B columns Hk page/16 18d
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in _values(held, d))     # B Hk keys d
    j = torch.arange(k.shape[2], device="cuda")
    there = (j < s["lens"][:, None])[:, None, :, None]
    k, v = k.masked_fill(~there, 0.0), v.masked_fill(~there, 0.0)
    q = s["q"].float().unflatten(2, (hk, s["hq"] // hk)).permute(0, 2, 3, 1, 4)    # B Hk G Tq d
    i = torch.arange(tq, device="cuda")[:, None]
    seen = (j <= i + (s["lens"] - tq)[:, None, None])[:, None, None]
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).mul_(K_UNIT / math.sqrt(d)).unflatten(2, q.shape[2:4])
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp_min(-3e38)).exp_()
    n = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, q.shape[2:4]) * V_UNIT / n.clamp_min(1e-30)
    lse = (m + n.log())[..., 0]
    return [o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype),
            lse.permute(0, 3, 1, 2).flatten(2, 3)]


def _counts(table, lens, page, n_pages):
    """How many times each page is held."""
    at = torch.arange(table.shape[1], device="cuda")
    own = at < ((lens + page - 1) // page)[:, None]
    n = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    return n.scatter_add_(0, table.clamp_min(0).long().flatten(), own.int().flatten())


def _plain_fork(s):
    table, lens, refs, page, n_pages = s["table"], s["lens"], s["refs"], s["page"], s["n_pages"]
    src, dst, at = s["src"].long(), s["dst"].long(), torch.arange(s["table"].shape[1], device="cuda")
    refs -= _counts(table[dst], lens[dst], page, n_pages)
    rows, n = table[src], lens[src]
    rows = torch.where(at < ((n + page - 1) // page)[:, None], rows, -1)
    refs += _counts(rows, n, page, n_pages)
    table[dst], lens[dst] = rows, n
    # room: a shared last page that will be written is replaced by a copy, new pages follow
    more = s["more"]
    last = table.gather(1, (lens // page).clamp_max(table.shape[1] - 1).long()[:, None])[:, 0]
    part = (more > 0) & (lens % page > 0)
    copied = part & (refs[last.clamp_min(0).long()] > 1)
    a = torch.where(copied, lens // page, (lens + page - 1) // page)
    b = (lens + more + page - 1) // page
    need = (b - a) * (more > 0)
    free = torch.nonzero(refs == 0)[:, 0].int()
    rank = (need.cumsum(0) - need)[:, None] + at - a[:, None]
    fresh = (at >= a[:, None]) & (at < (a + need)[:, None])
    table.copy_(torch.where(fresh, free[rank.clamp(0, len(free) - 1)], table))
    refs.index_add_(0, last[copied].long(), torch.full_like(last[copied], -1))
    refs.index_add_(0, table[fresh].long(), torch.ones_like(table[fresh]))
    to = table.gather(1, a.clamp_max(table.shape[1] - 1).long()[:, None])[:, 0][copied]
    s["pool"][:, to.long()] = s["pool"][:, last[copied].long()]
    lens += more
    return [table, lens, refs, s["pool"].view(torch.int32)]


def _plain_compact(s):
    table, refs, page = s["table"], s["refs"], s["page"]
    table.copy_(s["table_0"])
    refs.copy_(s["refs_0"])
    used = refs > 0
    n_used = used.sum()
    place = torch.arange(len(refs), device="cuda")
    moved = torch.nonzero(used & (place >= n_used))[:, 0]
    holes = torch.nonzero(~used & (place < n_used))[:, 0]
    to = torch.where(used, place, -1)
    to[moved] = holes
    refs[holes], refs[moved] = refs[moved], torch.zeros_like(refs[moved])
    s["pool"][:, holes] = s["pool"][:, moved]
    at = torch.arange(table.shape[1], device="cuda")
    own = at < ((s["lens"] + page - 1) // page)[:, None]
    table.copy_(torch.where(own, to[table.clamp_min(0).long()].int(), table))
    return [table, refs, to.int(), n_used.int().view(1), s["pool"].view(torch.int32)]


# ----------------------------------------------------------------- the framework's calls
def _own_rows(s):
    import gated_delta_rule_kaczmarz_gb300 as kla
    kla.kla_kv4_append(s["k"], s["v"], s["pool"], s["table"], s["lens"], cu_seqlens=s["cu"],
                       k_unit=K_UNIT, v_unit=V_UNIT)
    rows = {"total": len(s["k"])} if s["packed"] else {"T": s["t"]}
    return list(kla.kla_kv4_read(s["pool"], s["table"], s["lens"], cu_seqlens=s["cu"],
                                 dtype=_type(s), k_unit=K_UNIT, v_unit=V_UNIT, **rows))


def _own_attn(s):
    import gated_delta_rule_kaczmarz_gb300 as kla
    return list(kla.kla_kv4_attn(s["q"], s["pool"], s["table"], s["lens"], k_unit=K_UNIT,
                                 v_unit=V_UNIT))


def _own_fork(s):
    import gated_delta_rule_kaczmarz_gb300 as kla
    kla.kla_pages_fork(s["table"], s["lens"], s["refs"], s["src"], s["dst"], s["page"])
    kla.kla_pages_grow(s["pool"], s["table"], s["lens"], s["refs"], s["more"], s["page"])
    return [s["table"], s["lens"], s["refs"], s["pool"].view(torch.int32)]


def _own_compact(s):
    import gated_delta_rule_kaczmarz_gb300 as kla
    s["table"].copy_(s["table_0"])
    s["refs"].copy_(s["refs_0"])
    page_map, n_used = kla.kla_pages_compact(s["pool"], s["table"], s["lens"], s["refs"], s["page"])
    return [s["table"], s["refs"], page_map, n_used, s["pool"].view(torch.int32)]


def run(state):
    op = state["op"]
    if op == "rows":
        return _own_rows(state) if own else _plain_rows(state)
    if op == "attn":
        return _own_attn(state) if own else _plain_attn(state)
    if op == "fork":
        return _own_fork(state) if own else _plain_fork(state)
    return _own_compact(state) if own else _plain_compact(state)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    d, hk, page = case["d"], case["hk"], case["page"]
    if case["op"] in ("fork", "compact"):
        n = case["prompts"] if case["op"] == "fork" else case["seqs"]
        lens = _between(case, case["lo"], case["hi"], n)
        held = sum(-(-x // page) for x in lens)
        if case["op"] == "fork":
            copies = case["beams"] * sum(x % page > 0 for x in lens)
            words = held * (1 + 2 * case["beams"]) + 2 * case["n_pages"]
        else:       # a page in use lies behind the last of the used ones with their own odds
            copies = held * (case["n_pages"] - held) // case["n_pages"]
            words = 2 * held + 3 * case["n_pages"]
        return {"bytes": 2 * copies * case["layers"] * hk * page * 9 * d // 8 + 4 * words,
                "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rows":
        x = sum(_rows_lengths(case)[1]) * hk * d * 2
        # rows in, codes and scales out; codes and scales in, rows out
        return {"bytes": 2 * x * es + 2 * x * 9 / 16, "flops": 8 * x}
    lens, tq = _between(case, case["lo"], case["hi"], case["b"]), case["tq"]
    pairs = sum(max(0, n - tq + 1 + i) for n in lens for i in range(tq))
    rows = case["b"] * tq * case["hq"]
    return {"bytes": sum(lens) * hk * d * 9 / 8 + rows * (2 * es * d + 4),
            "flops": max(1, 4 * pairs * case["hq"] * d)}


# ----------------------------------------------------------------- 64 bits
def _e4m3(code):
    """The value of e4m3 codes."""
    e, m = (code >> 3 & 15).double(), (code & 7).double()
    x = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    x = torch.where((code & 127) == 127, math.nan, x)
    return torch.where(code >= 128, -x, x)


def _e2m1(code):
    e, m = (code >> 1 & 3).double(), (code & 1).double()
    x = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    return torch.where(code >= 8, -x, x)


def _rounded(x):
    """What the cache holds of x [rows, Hk, d]: the nearest scale, then the nearest of 8 levels
    a sign, ties to the even code."""
    y = x.unflatten(-1, (-1, 16))
    scales = _e4m3(torch.arange(127, device="cuda"))
    want = (y.abs().amax(-1) / 6).clamp_max(448.0)
    i = torch.searchsorted(scales, want).clamp(1, 126)
    up = (scales[i] - want < want - scales[i - 1]) | ((scales[i] - want == want - scales[i - 1]) & (i % 2 == 0))
    s = torch.where(up, scales[i], scales[i - 1])[..., None]
    a = torch.where(s > 0, y.abs() / s.clamp_min(2.0 ** -9), 0.0).clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step * s * torch.sign(y)).flatten(-2)


def _exact_rows(s):
    return [_rounded(s[x].double() / unit).mul(unit) for x, unit in (("k", K_UNIT), ("v", V_UNIT))]


def _exact_attn(s):
    d, hk, tq, page, group = s["d"], s["hk"], s["tq"], s["page"], s["hq"] // s["hk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    table, lens = s["table"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        raw = s["pool"][table[b][: -(-n // page)]].transpose(0, 1).flatten(1, 2).long()
        kc, vc = raw[..., : 8 * d], raw[..., 8 * d: 16 * d]
        ks, vs = raw[..., 16 * d: 17 * d], raw[..., 17 * d:]
        k = torch.empty(*raw.shape[:2], 16, d, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
        kc, vc = kc.unflatten(-1, (16, d // 2)), vc.unflatten(-1, (8, d))
        k[..., 0::2], k[..., 1::2] = _e2m1(kc % 16), _e2m1(kc // 16)
        v[:, :, 0::2], v[:, :, 1::2] = _e2m1(vc % 16), _e2m1(vc // 16)
        k *= _e4m3(ks).unflatten(-1, (16, d // 16)).repeat_interleave(16, -1)
        v *= _e4m3(vs).unflatten(-1, (d // 16, 16)).transpose(-1, -2).repeat_interleave(16, -1)
        k, v = (x.flatten(1, 2)[:, :n] for x in (k, v))
        first = max(0, tq - n)
        if first == tq:
            continue
        q = s["q"][b, first:].double().unflatten(1, (hk, group))
        x = torch.einsum("ihgd,hjd->hgij", q, k) * (K_UNIT * d ** -0.5)
        hide = torch.ones(tq - first, n, dtype=torch.bool, device="cuda").triu(n - (tq - first) + 1)
        x = x.masked_fill(hide, -math.inf)
        o[b, first:] = torch.einsum("hgij,hjd->ihgd", x.softmax(-1), v).flatten(1, 2) * V_UNIT
        lse[b, first:] = x.logsumexp(-1).permute(2, 0, 1).flatten(1)
    return [o, lse]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                 # whole numbers
    # products in 64 bits run at about a trillion operations a second
    if case["op"] == "attn" and work(case)["flops"] * 2 > 8e12:
        return None
    s = prepare(case, seed)
    return _exact_rows(s) if case["op"] == "rows" else _exact_attn(s)
