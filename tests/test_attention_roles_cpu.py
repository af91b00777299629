"""The barriers of the tensor-core attention kernels, as a model.

A kernel's warps are roles (loads, products, cleaning, softmax) that meet at
barriers which only show the parity of their phase.  Here every role is the
sequence of its waits and arrivals, each with the phase that it means, run under
random schedules with copies and products that complete late.  A model run fails
where a wait passes before its phase is complete, where a barrier is two phases
on before a waiter looks (it would wait for a third), where an arrival counts
for another phase than its own, and where nothing can go on.  Planted mistakes
(``wrong``) show that the model finds what it is for."""
import random
from collections import deque

import pytest

WARPS = 3                    # softmax warps of a tile; the kernels have 8 (forward: 4)


class Bar:
    def __init__(self, count):
        self.count, self.phase, self.got = count, 0, 0

    def arrive(self, phase):
        assert phase == self.phase, "an arrival counts for another phase"
        self.got += 1
        if self.got == self.count:
            self.phase, self.got = self.phase + 1, 0

    def passes(self, phase):
        seen = (self.phase ^ phase) & 1 == 1
        assert not seen or self.phase > phase, "a wait passes early"
        assert seen or self.phase <= phase, "two phases on before the waiter looked"
        return seen


def run(roles, bars, rng):
    """roles: name -> generator of (what, barrier, phase).  A commit arrives
    after the role's earlier ones, a load whenever it lands."""
    live = {n: [g, next(g)] for n, g in roles.items()}
    commits, loads = {n: deque() for n in roles}, []
    weight, late = {n: rng.choice([1, 1, 3, 20]) for n in roles}, rng.choice([1, 3, 20])
    while live or loads or any(commits.values()):
        can = [(weight[n], "role", n) for n, (_, op) in live.items()
               if op[0] != "wait" or bars[op[1]].passes(op[2])]
        can += [(late, "commit", n) for n, q in commits.items() if q] + [(late, "load", None)] * bool(loads)
        assert can, "nothing can go on"
        _, what, n = rng.choices(can, [c[0] for c in can])[0]
        if what == "commit":
            b, phase = commits[n].popleft()
            bars[b].arrive(phase)
        elif what == "load":
            b, phase = loads.pop(rng.randrange(len(loads)))
            bars[b].arrive(phase)
        else:
            g, (kind, b, phase) = live[n]
            if kind == "arrive":
                bars[b].arrive(phase)
            elif kind == "commit":
                commits[n].append((b, phase))
            elif kind == "load":
                loads.append((b, phase))
            op = next(g, None)
            if op is None:
                del live[n]
            else:
                live[n][1] = op
            if rng.random() < 0.02:
                weight[n] = rng.choice([1, 1, 3, 20])


def take(items):
    """An item as every reader takes it: published, read, handed back."""
    for m in range(len(items) + 1):
        yield m, ("wait", f"work{m & 1}", m // 2), ("arrive", f"work_read{m & 1}", m // 2), \
            items[m] if m < len(items) else None


# ------------------------------------------------------------------- backward
def backward(items, two_scores, wrong=None):
    """items: (key tile, steps, a last tile that has to be cleaned)."""
    bars = {f"full{i}": Bar(1) for i in range(5)} | {f"empty{i}": Bar(2 if i > 2 else 1) for i in range(5)}
    for n, c in dict(s=1, dp=1, p=WARPS, ds=WARPS, st=1, read=WARPS, raw=1, work=1,
                     work_read=3 + WARPS).items():
        bars |= {n + "0": Bar(c), n + "1": Bar(c)}
    bars |= dict(fix=Bar(1), fix_read=Bar(2), s_read=Bar(WARPS), zeroed=Bar(1), fin=Bar(2),
                 drained=Bar(WARPS))
    at, g, key, row, with_steps, raw_x, raw_y = [], 0, 0, 0, 0, 0, 0
    for is_key, n, ragged in items:
        at.append((g, key, row, with_steps, raw_x, raw_y))
        g, key, row = g + n, key + n * is_key, row + n * (not is_key)
        with_steps, raw_x, raw_y = with_steps + (n > 0), raw_x + ragged, raw_y + (ragged and is_key)

    def slot(y, g):
        return (3 + (g & 1), g // 2) if y else (g % 3, g // 3)

    def full(y, g):
        return "wait", f"full{slot(y, g)[0]}", slot(y, g)[1]

    def empty(y, g):
        return "commit", f"empty{slot(y, g)[0]}", slot(y, g)[1]

    def pair(what, name, g):
        return what, f"{name}{g & 1}", g >> 1

    def p_bar(what, gk):
        return (what, "p0", gk) if wrong == "one barrier for P" else pair(what, "p", gk)

    def loads():
        for m in range(len(items) + 1):
            if m > 1:
                yield "wait", f"work_read{m & 1}", m // 2 - 1
            yield "arrive", f"work{m & 1}", m // 2
            if m == len(items):
                return
            (is_key, n, ragged), (g0, _, _, item, rx, ry) = items[m], at[m]

            def tile(y, i):
                s, use = slot(y, g0 + i)
                if use:
                    yield "wait", f"empty{s}", use - 1
                raw = ragged and i == n - 1 and (is_key or not y)
                if raw and not y and rx:
                    yield "wait", "zeroed", rx - 1
                yield ("load", f"raw{int(y)}", ry if y else rx) if raw else ("load", f"full{s}", use)
            for i in range(n):
                if i == 0:
                    yield from tile(False, 0)
                yield from tile(True, i)
                if i == 0:
                    if item:
                        yield "wait", "fix_read", item - 1
                    yield "load", "fix", item
                if i + 1 < n:
                    yield from tile(False, i + 1)

    def products(second):
        for m, wait, back, it in take(items):
            yield wait
            yield back
            if it is None:
                return
            (is_key, n, _), (g0, k0, r0, item, _, _) = it, at[m]
            if n == 0:
                continue
            drained = [("wait", "drained", item - 1)] * (item > 0)

            def scores(i):
                yield full(False, g0 + i)
                yield pair("commit", "s", g0 + i)
                if i + 1 == n:
                    yield "commit", "fix_read", item
            if is_key and not second:
                yield "wait", "fix", item
                yield from scores(0)
                yield from drained
                for i in range(n):
                    if two_scores and i + 1 < n:
                        yield from scores(i + 1)
                    yield full(True, g0 + i)
                    yield p_bar("wait", k0 + i)
                    yield empty(True, g0 + i)
                    if not two_scores and i + 1 < n:
                        yield from scores(i + 1)
                yield "commit", "fin", item
            elif is_key:
                yield "wait", "fix", item
                for i in range(n):
                    yield full(True, g0 + i)
                    if i == 0:
                        yield from drained
                    yield pair("commit", "dp", g0 + i)
                    yield empty(True, g0 + i)
                    if i + 1 == n:
                        yield "commit", "fix_read", item
                    yield pair("wait", "ds", g0 + i)
                    yield empty(False, g0 + i)
                yield "commit", "fin", item
            elif not second:
                yield "wait", "fix", item
                for i in range(n + 1):
                    g = g0 + i
                    if i < n:
                        yield full(False, g)
                        if i:
                            yield "wait", "s_read", r0 + i - 1
                        yield pair("commit", "s", g)
                        yield full(True, g)
                        if i == 0:
                            yield from drained
                        yield pair("commit", "dp", g)
                        yield from [empty(True, g)] * 2
                        if i + 1 == n:
                            yield from [("commit", "fix_read", item)] * 2
                    if i:
                        yield pair("wait", "ds", g - 1)
                        yield empty(False, g - 1)
                yield "commit", "fin", item
                yield "wait", "s_read", r0 + n - 1
            else:
                if item and wrong != "an arrival ahead":
                    yield "wait", "fin", item - 1
                yield "arrive", "fin", item
                yield "wait", "fin", item

    def statistics():
        for m, wait, back, it in take(items):
            yield wait
            yield back
            if it is None:
                return
            (is_key, n, ragged), (g0, k0, _, _, rx, ry) = it, at[m]
            for gk in range(k0, k0 + n if is_key else k0):
                if gk > 1:
                    yield pair("wait", "read", gk - 2)
                yield pair("arrive", "st", gk)
            if ragged:
                for y in (False, True)[:1 + is_key]:
                    yield "wait", f"raw{int(y)}", ry if y else rx
                    s, use = slot(y, g0 + n - 1)
                    yield "arrive", f"full{s}", use
                yield "arrive", "zeroed", rx

    def softmax():
        for m, wait, back, it in take(items):
            yield wait
            yield back
            if it is None:
                return
            (is_key, n, _), (g0, k0, r0, item, _, _) = it, at[m]
            for i in range(n):
                if is_key:
                    yield pair("wait", "st", k0 + i)
                yield pair("wait", "s", g0 + i)
                yield p_bar("arrive", k0 + i) if is_key else ("arrive", "s_read", r0 + i)
                yield pair("wait", "dp", g0 + i)
                yield pair("arrive", "ds", g0 + i)
                if is_key:
                    yield pair("arrive", "read", k0 + i)
            if n:
                yield "wait", "fin", item
                yield "arrive", "drained", item

    roles = dict(loads=loads(), v=products(False), k=products(True), statistics=statistics())
    return roles | {f"softmax{i}": softmax() for i in range(WARPS)}, bars


def backward_items(rng):
    n = rng.randint(1, 8)
    kinds = [True] * rng.randint(0, n)
    kinds += [False] * (n - len(kinds))
    if rng.random() < 0.3:
        rng.shuffle(kinds)
    steps = [rng.choice([0, 1, 1, 1, 2, 2, 3, 4, 7]) for _ in kinds]
    return [(k, s, s > 0 and rng.random() < 0.5) for k, s in zip(kinds, steps)]


# -------------------------------------------------------------------- forward
def forward(items, slots, wrong=None):
    """items: (key tiles, those of each row tile, a last V tile to be cleaned)."""
    bars = {f"full{i}": Bar(1) for i in range(slots)} | {f"empty{i}": Bar(2) for i in range(slots)}
    for n, c in dict(q=1, q_read=1, s=1, p=WARPS, o=1, work=1, work_read=3 + 2 * WARPS, turn=1).items():
        bars |= {n + "0": Bar(c), n + "1": Bar(c)}
    bars |= dict(raw=Bar(1), zeroed=Bar(1))

    def slot(what, name, j):
        return what, f"{name}{j % slots}", j // slots

    def loads():
        j, raws, used = 0, 0, [0, 0]
        for m in range(len(items) + 1):
            if m > 1:
                yield "wait", f"work_read{m & 1}", m // 2 - 1
            yield "arrive", f"work{m & 1}", m // 2
            if m == len(items):
                return
            nb, mine, ragged = items[m]
            for i in range(2 * nb + 1):
                for t in (0, 1) if i == 2 else ():
                    if mine[t]:
                        if used[t]:
                            yield "wait", f"q_read{t}", used[t] - 1
                        yield "load", f"q{t}", used[t]
                        used[t] += 1
                if i == 2 * nb:
                    break
                if j >= slots:
                    yield slot("wait", "empty", j - slots)
                if ragged and i == 2 * nb - 1:
                    if raws and wrong != "a second tile to clean":
                        yield "wait", "zeroed", raws - 1
                    yield "load", "raw", raws
                    raws += 1
                else:
                    yield slot("load", "full", j)
                j += 1

    def cleaning():
        j = raws = 0
        for m, wait, back, it in take(items):
            yield wait
            yield back
            if it is None:
                return
            j += 2 * it[0]
            if it[2]:
                yield "wait", "raw", raws
                yield slot("arrive", "full", j - 1)
                yield "arrive", "zeroed", raws
                raws += 1

    def products(t):
        j = used = step = turns = 0
        for m, wait, back, it in take(items):
            yield wait
            yield back
            if it is None:
                return
            nb, (mine, other) = it[0], it[1] if t == 0 else it[1][::-1]
            if nb == 0:
                continue
            yield slot("wait", "full", j)
            if mine:
                yield "wait", f"q{t}", used
                used += 1
                yield "commit", f"s{t}", step
                if mine == 1:
                    yield "commit", f"q_read{t}", used - 1
            yield slot("commit" if mine else "arrive", "empty", j)
            for n in range(nb):
                v, k, last = j + 2 * n + 1, j + 2 * n + 2, n + 1 == nb
                yield slot("wait", "full", v)
                if not last:
                    yield slot("wait", "full", k)
                if n >= mine:
                    yield slot("arrive", "empty", v)
                    if not last:
                        yield slot("arrive", "empty", k)
                    continue
                both = n < other
                if both and (t == 1 or turns):
                    yield "wait", f"turn{t}", turns if t == 1 else turns - 1
                turns += both
                yield "wait", f"p{t}", step
                yield "commit", f"o{t}", step
                yield slot("commit", "empty", v)
                step += 1
                if both:
                    yield "arrive", f"turn{1 - t}", turns - 1
                if n + 1 < mine:
                    yield "commit", f"s{t}", step
                    if n + 2 == mine:
                        yield "commit", f"q_read{t}", used - 1
                    yield slot("commit", "empty", k)
                elif not last:
                    yield slot("arrive", "empty", k)
            j += 2 * nb

    def softmax(t, rng):
        step = 0
        for m, wait, back, it in take(items):
            yield wait
            yield back
            if it is None:
                return
            for n in range(it[1][t]):
                yield "wait", f"s{t}", step
                if n and rng.random() < 0.3:        # a row's maximum grew
                    yield "wait", f"o{t}", step - 1
                yield "arrive", f"p{t}", step
                step += 1
            if it[1][t]:
                yield "wait", f"o{t}", step - 1

    roles = dict(loads=loads(), cleaning=cleaning(), p0=products(0), p1=products(1))
    return roles | {f"softmax{t}{i}": softmax(t, random.Random(i)) for t in (0, 1)
                    for i in range(WARPS)}, bars


def forward_items(rng):
    out = []
    for _ in range(rng.randint(1, 8)):
        nb = rng.choice([0, 1, 1, 1, 2, 2, 3, 5, 9])
        mine = [nb, nb]
        if rng.random() < 0.4:
            mine[rng.randrange(2)] = rng.randint(0, nb)
        out.append((nb, tuple(mine), nb > 0 and rng.random() < 0.5))
    return out


def schedules(model, items, variants, n, wrong=None):
    for seed in range(n):
        rng = random.Random(seed)
        run(*model(items(rng), rng.choice(variants), wrong), rng)


def test_backward_roles():
    schedules(backward, backward_items, (False, True), 400)


def test_forward_roles():
    schedules(forward, forward_items, (4, 6), 400)


@pytest.mark.parametrize("model, items, variants, wrong", [
    (backward, backward_items, (True,), "one barrier for P"),
    (backward, backward_items, (False, True), "an arrival ahead"),
    (forward, forward_items, (4, 6), "a second tile to clean"),
])
def test_planted_mistakes_are_found(model, items, variants, wrong):
    with pytest.raises(AssertionError):
        schedules(model, items, variants, 2000, wrong)
