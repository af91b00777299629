"""The paged 4-bit cache by its definition, on the CPU in 64 bits: its values,
its bytes, attention over it, and its book in plain loops."""
import math

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values():
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m / 8 * 2.0 ** -6)


SCALES = _e4m3_values()


def _nearest(x, values):
    """Index of the value nearest to x >= 0, ties to the even index; the last at most."""
    i = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    up, down = values[i] - x, x - values[i - 1]
    return np.where((up < down) | ((up == down) & (i % 2 == 0)), i, i - 1)


def quantise(x, unit):
    """Codes 0..15 [..., d] and scale codes [..., d / 16] of x (a float tensor)."""
    x = x.double().numpy() / unit
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    with np.errstate(invalid="ignore"):
        top = np.abs(y).max(-1)
    fine = np.isfinite(y).all(-1)
    with np.errstate(over="ignore"):          # a product of two fp32 is exact in 64 bits
        sixth = (np.where(fine, top, 0.0) * np.float64(np.float32(1 / 6))).astype(np.float32)
    s = np.where(fine, _nearest(np.minimum(sixth.astype(np.float64), 448.0), SCALES), 127)
    value = np.where(fine, SCALES[np.minimum(s, 126)], 0.0)[..., None]
    a = np.divide(np.abs(y), value, out=np.zeros_like(y), where=(value > 0) & fine[..., None])
    code = _nearest(a, LEVELS) + 8 * (np.signbit(y) & (value > 0) & fine[..., None])
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def values(code, scale, unit):
    """The values of codes and scale codes, in 64 bits."""
    level = np.concatenate([LEVELS, -LEVELS])[code]
    s = np.append(SCALES, np.nan)[scale & 127] * np.where(scale > 127, -1.0, 1.0)
    return torch.from_numpy(level * np.repeat(s, 16, -1) * unit)


def rounded(x, unit):
    return values(*quantise(x, unit), unit)


class Pages:
    """A pool [n_pages, Hk, page / 16, 18 d] of bytes, on the CPU."""

    def __init__(self, pool, d):
        self.b, self.d = pool.numpy(), d

    def put(self, page, head, place, k, v):
        """(codes, scale codes) of a token's key and value to a place of a page."""
        d, t = self.d, place % 16
        b = self.b[page, head, place // 16]
        b[t * d // 2:(t + 1) * d // 2] = k[0][0::2] | k[0][1::2] << 4
        two = b[8 * d + t // 2 * d: 8 * d + (t // 2 + 1) * d]
        two[:] = (two & 0x0f | v[0] << 4) if t % 2 else (two & 0xf0 | v[0])
        b[16 * d + t * d // 16: 16 * d + (t + 1) * d // 16] = k[1]
        b[17 * d + t::16][: d // 16] = v[1]

    def get(self, page, head, place):
        d, t = self.d, place % 16
        b = self.b[page, head, place // 16]
        kc = b[t * d // 2:(t + 1) * d // 2]
        kc = np.stack([kc & 15, kc >> 4], -1).reshape(d)
        vc = b[8 * d + t // 2 * d: 8 * d + (t // 2 + 1) * d] >> (4 * (t % 2)) & 15
        return (kc, b[16 * d + t * d // 16: 16 * d + (t + 1) * d // 16]), \
            (vc, b[17 * d + t::16][: d // 16])


def book(lens, page, columns, n_pages, seed):
    """A table of pages anywhere in a pool; entries behind a sequence's are out of range."""
    g = np.random.default_rng(seed)
    free = list(g.permutation(n_pages))
    table = np.full((len(lens), columns), 1 << 30, np.int32)
    for b, n in enumerate(lens):
        for c in range(-(-n // page)):
            table[b, c] = free.pop()
    return torch.from_numpy(table)


def garbage(*shape, seed=0):
    """Bytes of any kind: scales that are NaN and codes of every value among them."""
    return torch.randint(0, 256, shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(seed))


def filled(lens, page, columns, n_pages, hk, d, units, seed):
    """A pool and table with normal rows in it, and the rows' values [n, Hk, d] of each
    sequence."""
    g = torch.Generator().manual_seed(seed)
    table = book(lens, page, columns, n_pages, seed)
    pool = garbage(n_pages, hk, page // 16, 18 * d, seed=seed)
    pages, held = Pages(pool, d), []
    for b, n in enumerate(lens):
        k, v = torch.randn(n, hk, d, generator=g), 0.3 * torch.randn(n, hk, d, generator=g)
        (kc, ks), (vc, vs) = quantise(k, units[0]), quantise(v, units[1])
        for t in range(n):
            for h in range(hk):
                pages.put(int(table[b, t // page]), h, t % page, (kc[t, h], ks[t, h]),
                          (vc[t, h], vs[t, h]))
        held.append((values(kc, ks, units[0]), values(vc, vs, units[1])))
    return pool, table, held


U = 2.0 ** -24
#: query rows to a key head, and pairs of a query row and a key that the tables have room for,
#: from which a bf16 cache is unpacked for kla_attn's kernels
LONG, PAIRS = 128, 12 << 20


def unpacked(B, Tq, hq, hk, page, columns, dtype):
    return dtype == torch.bfloat16 and Tq * hq // hk >= LONG and B * columns * page * Tq * hq >= PAIRS


def attention(q, k, v, scale, unpacked=False):
    """One sequence, 64 bits: values and tolerances of o [Tq, Hq, d] and lse [Tq, Hq].

    q times k: products of fp16 parts are exact, their sums on the tensor cores are
    taken to be off by 2 u = 2^-23 an addition, and the parts of an fp32 q by 2^-22:
    e = (d + 8) 2 u max_ij sum_c |q_ic k_jc| scale.  p is off by 2 e, 2^-22 (the
    exponential) and the rounding r of an operand (bf16 calls: fp16, 2^-11, and where
    the cache is unpacked bf16, 2^-8, as in kla_attn; fp32: 2^-22); as an operand
    it has an absolute error too, 2^-25 (fp16's smallest step is 2^-24), and the largest
    p of a row is 2^7 or more: 2^-32 |v| for each key that is seen, which is all that is
    left of a row's o where the keys that matter have v = 0.  n products are summed with
    2 u each; o is rounded once by h."""
    nq, hq, d = q.shape
    n, hk, _ = k.shape
    h, r = (2.0 ** -8, 2.0 ** -11) if q.dtype == torch.bfloat16 else (U, 2.0 ** -22)
    if unpacked:
        r = 2.0 ** -8
    q = q.double().unflatten(1, (hk, hq // hk)).permute(1, 2, 0, 3)
    k, v = (x.transpose(0, 1)[:, None] for x in (k, v))
    seen = torch.arange(n) <= torch.arange(nq)[:, None] + n - nq
    s = (q @ k.mT * scale).masked_fill(~seen, -math.inf)
    lse = s.logsumexp(-1, keepdim=True) if n else torch.full((*q.shape[:3], 1), -math.inf).double()
    p = torch.where(seen, (s - lse.clamp_min(-1e300)).exp(), 0.0)
    o = p @ v
    e = (d + 8) * 2 * U * float((q.abs() @ k.abs().mT).max() if n and nq else 0) * scale
    tol = (r + 2 * e + 2.0 ** -21 + 2 * n * U) * (p @ v.abs()) + h * o.abs() \
        + 2.0 ** -32 * (seen.double() @ v.abs())
    lse = lse[..., 0]
    tols = 2 * e + 1e-6 + 4 * U * lse.abs().nan_to_num(posinf=0)
    return tuple(tuple(t.permute(2, 0, 1, *range(3, t.dim())).flatten(1, 2) for t in pair)
                 for pair in ((o, tol), (lse, tols)))


# ------------------------------------------------------------------ the book
def counted(table, lens, page, n_pages):
    refs = [0] * n_pages
    for row, n in zip(table, lens):
        for c in range(-(-n // page)):
            refs[row[c]] += 1
    return refs


def fork(table, lens, src, dst, page):
    """Lists in, lists out."""
    old, had = [list(r) for r in table], list(lens)
    table, lens = [list(r) for r in table], list(lens)
    for s, d in zip(src, dst):
        lens[d] = 0 if s < 0 else had[s]
        held = -(-lens[d] // page)
        table[d] = [old[s][c] if c < held else -1 for c in range(len(table[d]))]
    return table, lens


def grow(table, lens, refs, more, page):
    """(table, lens, refs, copies) or None where the pages do not suffice."""
    table, lens, after = [list(r) for r in table], list(lens), list(refs)
    free = [p for p, n in enumerate(refs) if n == 0]
    copies = []
    for s, n in enumerate(more):
        if n == 0:
            continue
        at = lens[s] // page
        if lens[s] % page and refs[table[s][at]] > 1:
            if not free:
                return None
            p = free.pop(0)
            copies.append((table[s][at], p))
            after[table[s][at]] -= 1
            table[s][at] = p
            after[p] = 1
        for c in range(-(-lens[s] // page), -(-(lens[s] + n) // page)):
            if not free:
                return None
            table[s][c] = free.pop(0)
            after[table[s][c]] = 1
        lens[s] += n
    return table, lens, after, copies


def trim(table, lens, cut, page):
    table = [[-1 if -(-(n - x) // page) <= c < -(-n // page) else p for c, p in enumerate(row)]
             for row, n, x in zip(table, lens, cut)]
    return table, [n - x for n, x in zip(lens, cut)]


def compact(table, lens, refs, page):
    """(table, refs, page_map, moves)."""
    n_used = sum(n > 0 for n in refs)
    holes = [p for p in range(n_used) if refs[p] == 0]
    moves = [(p, holes.pop(0)) for p in range(n_used, len(refs)) if refs[p] > 0]
    where = [p if n > 0 else -1 for p, n in enumerate(refs)]
    after = list(refs)
    for a, b in moves:
        where[a], after[b], after[a] = b, refs[a], 0
    table = [[where[x] if c < -(-n // page) else x for c, x in enumerate(row)]
             for row, n in zip(table, lens)]
    return table, after, where, moves


# ------------------------------------------------------------------ arguments
def arguments(put):
    """Right arguments of every call on a cache, their tensors where `put` takes them."""
    hk, d, page = 2, 64, 16
    pool = put(garbage(5, hk, 1, 18 * d, seed=1))
    table, lens = put(torch.arange(4).int().view(2, 2)), put(torch.tensor([20, 7]).int())
    refs, one, none = put(torch.ones(5).int()), put(torch.ones(2).int()), put(torch.tensor([0, -1]).int())
    order, q = put(torch.arange(2).int()), put(torch.zeros(2, 1, hk, d))
    k, v, layer = put(torch.zeros(2, 1, hk, d)), put(torch.zeros(2, 1, hk, d)), pool[None]
    book = dict(table=table, lens=lens, refs=refs)
    return dict(kept=(pool, table, lens, refs), calls=dict(
        kla_kv4_append=dict(k=k, v=v, pool=pool, table=table, lens=lens),
        kla_kv4_read=dict(pool=pool, table=table, lens=lens, T=1, k_out=k, v_out=v, dtype=torch.float32),
        kla_kv4_attn=dict(q=q, pool=pool, table=table, lens=lens),
        kla_pages_fork=dict(**book, src=none, dst=order, page=page),
        kla_pages_grow=dict(pool=layer, **book, n_new=one, page=page),
        kla_pages_trim=dict(**book, n_cut=one, page=page),
        kla_pages_compact=dict(pool=layer, **book, page=page),
        kla_pages_copy=dict(pool=layer, src=one, dst=order)))


def wrong_arguments(base, host):
    """(call, its right arguments, the one to replace, by what): on the host, of another type,
    shape or order."""
    for name, args in base["calls"].items():
        for key, t in args.items():
            if not hasattr(t, "get_device"):
                continue
            wrong = [host(t)]
            layers = key == "pool" and name.startswith("kla_pages")
            if not layers:
                wrong.append(t.double())
            if t.dim() == 1:
                wrong.append(t.repeat(2)[::2])
                if key in ("lens", "n_new", "n_cut", "src"):
                    wrong.append(t.repeat(2))
            if key == "table":
                wrong += [t.repeat(1, 2)[:, ::2], t[0]]
                if not name.startswith("kla_pages"):
                    wrong.append(t[:1])
            if key == "pool" and not layers:
                wrong += [t[..., : 17 * 64], t[:, :1].expand(-1, 2, -1, -1), t[0]]
            if layers:
                wrong += [t[:, ::2], t[0, 0, 0, 0]]
            if key in ("q", "k", "v", "k_out", "v_out"):
                wrong += [t[..., :32], t[0], t.transpose(0, 2), t.expand(2, 1, 2, 64)[..., ::2]]
            for bad in wrong:
                yield name, args, key, bad
