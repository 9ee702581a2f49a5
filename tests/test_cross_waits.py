"""The waits of the tensor-core cross-attention kernels, on the CPU.

Every warp role of cross_fwd_tc.cu and of both passes of cross_bwd_tc.cu is a
generator that yields the barriers it waits for, in the kernel's order; loads and
MMAs finish at any later time, MMAs of a warp in order.  A barrier is waited for by
parity, as mbarrier.test_wait does, so a wait passes also where the round before
the one that is meant is not over, or the one after it is: random orders of the
roles, some of them slow, look for either, for slots read before or after their
time, and for waits that never end."""

import random

import pytest


class Barrier:
    def __init__(self, name, count=1):
        self.name, self.count, self.left, self.done = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, parity):  # the phase in progress has the other parity
        return (self.done & 1) != parity


def barriers(name, n, count=1):
    return [Barrier(f"{name}[{i}]", count) for i in range(n)]


class Ring:
    def __init__(self, n):
        self.n, self.i, self.round = n, 0, 0

    def next(self, by=1):
        self.i += by
        if self.i >= self.n:
            self.i, self.round = self.i - self.n, self.round + 1

    def copy(self):
        r = Ring(self.n)
        r.i, r.round = self.i, self.round
        return r


class World:
    """Roles, loads that may land now, and the MMAs of each issuing warp."""

    def __init__(self, rng):
        self.rng, self.loads, self.mmas, self.pace = rng, [], {}, {}

    def pick(self, choices):
        for name, _ in choices:
            if name not in self.pace:
                self.pace[name] = self.rng.choice([1, 1, 0.02, 0.0005])
        return self.rng.choices(choices, [self.pace[name] for name, _ in choices])[0][1]

    def run(self, roles):
        at = {name: next(role, None) for name, role in roles.items()}  # the wait that each is at

        def go(name):
            barrier, meant = at[name]
            assert barrier.done > meant, f"{name} passes {barrier.name} before round {meant} is over"
            assert meant < 0 or barrier.done == meant + 1, f"{name} comes to {barrier.name} a round late"
            at[name] = next(roles[name], None)

        while True:
            ready = [(n, lambda n=n: go(n)) for n, w in at.items() if w is not None and w[0].passes(w[1] & 1)]
            ready += [("loads", lambda i=i: self.loads.pop(i)()) for i in range(len(self.loads))]
            ready += [("mmas " + n, lambda q=q: q.pop(0)()) for n, q in self.mmas.items() if q]
            if not ready:
                stuck = {n: w[0].name for n, w in at.items() if w is not None}
                assert not stuck, f"waits that never end: {stuck}"
                return
            self.pick(ready)()


# ----------------------------------------------------------------- forward
def forward_items(rng, D):
    """The items of a CTA: key tiles, query tiles that have rows, whether its
    keys are loaded for it and free after it."""
    tiles, slots = (4, 12) if D == 64 else (2, 4)
    nt, rows = rng.randint(1, 3), rng.randint(1, tiles)  # items of a head, query tiles of its last
    draw = (lambda: rng.choice([0, 1, 2, 3, 6, 7, rng.randint(0, 8)]))
    t, nkt, run, new, total, out = rng.randint(0, nt - 1), draw(), 0, True, rng.randint(2, 9), []
    for i in range(total):
        stays = 2 * nkt <= slots
        out.append(dict(nkt=nkt, nact=rows if t == nt - 1 else tiles, keys=run if stays else (run, i),
                        loads=not stays or new, free=not stays or t == nt - 1 or i == total - 1))
        t, new = t + 1, False
        if t == nt:
            t, run, new, nkt = 0, run + 1, True, draw()
    return out


def forward(rng, D, items, clean, every_step=True, ring_per_warp=True):
    tiles, per, qslots, slots = (4, 2, 8, 12) if D == 64 else (2, 2, 3, 4)
    warps = tiles // per
    rings = warps if ring_per_warp else 1
    span = tiles // rings  # query tiles of a ring
    w = World(rng)
    q_full = [barriers(f"q_full{r}", qslots // rings) for r in range(rings)]
    q_empty = [barriers(f"q_empty{r}", qslots // rings) for r in range(rings)]
    kv_full, kv_empty, kv_clean = barriers("kv_full", slots), barriers("kv_empty", slots, warps), barriers("kv_clean", slots)
    s_full, p_full, o_full, staged = (barriers(n, tiles) for n in ("s_full", "p_full", "o_full", "o_staged"))
    w.mmas = {str(u): [] for u in range(warps)}
    kv, q, bits = {}, {}, {}  # what the slots hold
    live = [it for it in items if it["nkt"] > 0]

    def ring():
        return Ring(qslots // rings)

    def own(it, r):  # query tiles of ring r that have rows
        return min(max(it["nact"] - span * r, 0), span)

    def land(barrier, holds, slot, what):
        def now():
            holds[slot] = what
            barrier.arrive()
        w.loads.append(now)

    def load():
        rq, rk = [ring() for _ in range(rings)], Ring(slots)

        def load_q(n, t):
            r = t // span
            yield q_empty[r][rq[r].i], rq[r].round - 1
            land(q_full[r][rq[r].i], q, (r, rq[r].i), (n, t))
            rq[r].next()

        def load_kv(what):
            yield kv_empty[rk.i], rk.round - 1
            land(kv_full[rk.i], kv, rk.i, what)
            rk.next()

        for n, it in enumerate(live):
            keys = it["nkt"] if it["loads"] else 0
            yield from load_q(n, 0)
            if keys:
                yield from load_kv((it["keys"], "K", 0))
            for t in range(1, it["nact"]):
                yield from load_q(n, t)
            if keys:
                yield from load_kv((it["keys"], "V", 0))
            for j in range(1, keys):
                yield from load_kv((it["keys"], "K", j))
                yield from load_kv((it["keys"], "V", j))

    def mma(u0):
        issue, t0 = w.mmas[str(u0)].append, per * u0
        r, first = t0 // span, t0 % span
        rq, run, at, pv = ring(), Ring(slots), Ring(slots), Ring(slots)
        turn, pend = [0] * per, [False] * per
        state = dict(held=False)

        def reads(holds, slot, what):
            def now():
                assert holds.get(slot) == what, f"{holds.get(slot)} read for {what}"
            issue(now)

        def products(u):
            v = (kv_clean if clean else kv_full)[pv.i], pv.round
            if every_step and u == 0 and state["held"]:
                state["held"] = False
                yield v
            if not pend[u]:
                return
            pend[u] = False
            if not every_step:
                yield v
            yield p_full[t0 + u], turn[u]
            turn[u] += 1
            reads(kv, pv.i, state["v"])
            if state["last"]:
                issue(o_full[t0 + u].arrive)

        for n, it in enumerate(live):
            if it["loads"]:
                run = at.copy()
            else:
                at = run.copy()
            for j in range(it["nkt"]):
                yield kv_full[at.i], at.round
                for u in range(per):
                    yield from products(u)
                    if t0 + u >= it["nact"]:
                        continue
                    mine = rq.copy()
                    mine.next(first + u)
                    if j == 0:
                        yield q_full[r][mine.i], mine.round
                    reads(kv, at.i, (it["keys"], "K", j))
                    reads(q, (r, mine.i), (n, t0 + u))
                    issue(s_full[t0 + u].arrive)
                    pend[u] = True
                if state.get("free"):
                    issue(kv_empty[pv.i].arrive)
                if it["free"]:
                    issue(kv_empty[at.i].arrive)
                pv = at.copy()
                pv.next()
                state.update(held=True, v=(it["keys"], "V", j), last=j == it["nkt"] - 1, free=it["free"])
                at.next(2)
            rq.next(own(it, r))
        for u in range(per):
            yield from products(u)

    def cleaner():
        at = Ring(slots)
        at.next()
        for it in live if clean else ():
            for j in range(it["nkt"] if it["loads"] else 0):
                yield kv_full[at.i], at.round
                bits[at.i] = (it["keys"], j)
                kv_clean[at.i].arrive()
                at.next(2)

    def store():
        rq, turn = [ring() for _ in range(rings)], [0] * tiles
        for it in live:
            for t in range(it["nact"]):
                yield staged[t], turn[t]
                turn[t] += 1
                q_empty[t // span][rq[t // span].i].arrive()
                rq[t // span].next()

    def softmax(t):
        r, first = t // span, t % span
        rq, run, at, last, s_turn, o_turn = ring(), Ring(slots), Ring(slots), None, 0, 0
        at.next()
        for it in live:
            if it["loads"]:
                run = at.copy()
            else:
                at = run.copy()
            mine = rq.copy()
            mine.next(first)
            rq.next(own(it, r))
            for j in range(it["nkt"]):
                if t < it["nact"]:
                    yield s_full[t], s_turn
                    s_turn += 1
                    if clean:
                        yield kv_clean[at.i], at.round
                        assert bits[at.i] == (it["keys"], j)
                    p_full[t].arrive()
                at.next(2)
            if t >= it["nact"]:
                continue
            yield o_full[t], o_turn
            o_turn += 1
            if last is not None:
                yield q_empty[r][last.i], last.round
            last = mine
            staged[t].arrive()

    roles = {"load": load(), "clean": cleaner(), "store": store()}
    roles.update({f"mma {u}": mma(u) for u in range(warps)}, **{f"softmax {t}": softmax(t) for t in range(tiles)})
    w.run(roles)


# ------------------------------------------------------ backward, first pass
def backward(rng, D, items, clean):
    """items: the key tiles of each."""
    groups, slots, sums, sets = (3, 6, 2, 1) if D == 64 else (2, 3, 1, 2)
    aux_warps = 3
    w = World(rng)
    a_full, a_empty = barriers("a_full", 2), barriers("a_empty", 2)
    n_full, n_empty, n_aux = (barriers(n, slots) for n in ("n_full", "n_empty", "n_aux"))
    s_full, p_full = barriers("s_full", groups), barriers("p_full", groups)
    acc_full, acc_free = Barrier("acc_full"), Barrier("acc_free")
    c_full, c_read = barriers("c_full", 2), barriers("c_read", 2, groups + 1)
    x_full, x_read = barriers("x_full", sums, groups), barriers("x_read", sums)
    w.mmas = {"scores": [], "products": []}
    a, n_at, bits, c, x = {}, {}, {}, {}, {}  # what the slots hold
    live = [(n, k) for n, k in enumerate(items) if k > 0]

    def land(barrier, holds, slot, what):
        def now():
            holds[slot] = what
            barrier.arrive()
        w.loads.append(now)

    def reads(queue, *pairs):
        def now():
            for holds, slot, what in pairs:
                assert holds.get(slot) == what, f"{holds.get(slot)} read for {what}"
        w.mmas[queue].append(now)

    def load():
        ra, rn = Ring(2), Ring(slots)
        for n, k in live:
            yield a_empty[ra.i], ra.round - 1
            land(a_full[ra.i], a, ra.i, n)
            ra.next()
            for j in range(k):
                yield n_empty[rn.i], rn.round - 1
                land(n_full[rn.i], n_at, rn.i, (n, j))
                rn.next()

    def scores():
        ra, rn, before, stage, fresh = Ring(2), Ring(slots), Ring(slots), Ring(groups), groups
        for n, k in live:
            yield a_full[ra.i], ra.round
            for j in range(k):
                yield n_full[rn.i], rn.round
                if fresh == 0:
                    yield n_empty[before.i], before.round
                    before.next()
                else:
                    fresh -= 1
                reads("scores", (n_at, rn.i, (n, j)), (a, ra.i, n))
                w.mmas["scores"].append(s_full[stage.i].arrive)
                rn.next()
                stage.next()
            ra.next()

    def products():
        rn, stage, free = Ring(slots), Ring(groups), -1
        for n, k in live:
            for j in range(k):
                if clean:
                    yield n_aux[rn.i], rn.round
                if j == 0:
                    yield acc_free, free
                    free += 1
                yield p_full[stage.i], stage.round
                reads("products", (n_at, rn.i, (n, j)))
                w.mmas["products"].append(n_empty[rn.i].arrive)
                rn.next()
                stage.next()
            w.mmas["products"].append(acc_full.arrive)

    def aux(i):
        rn, j = Ring(slots), i
        rn.next(i)
        for n, k in live if clean else ():
            while j < k:
                yield n_full[rn.i], rn.round
                bits[rn.i] = (n, j)
                n_aux[rn.i].arrive()
                rn.next(aux_warps)
                j += aux_warps
            j -= k

    def dot(i):
        rc = Ring(2)
        rc.next(i)
        for n, _ in live[i::sets]:
            yield c_read[rc.i], rc.round - 1
            c[rc.i] = n
            c_full[rc.i].arrive()
            rc.next(sets)

    def take_c(rc, n):
        yield c_full[rc.i], rc.round
        assert c[rc.i] == n
        c_read[rc.i].arrive()
        rc.next()

    def group(g):
        rn, rc, rx, turn, j = Ring(slots), Ring(2), Ring(sums), 0, g
        rn.next(g)
        for n, k in live:
            have = False
            while j < k:
                yield s_full[g], turn
                turn += 1
                if not have:
                    yield from take_c(rc, n)
                    have = True
                if clean:
                    yield n_aux[rn.i], rn.round
                    assert bits[rn.i] == (n, j)
                p_full[g].arrive()
                rn.next(groups)
                j += groups
            if not have:
                yield from take_c(rc, n)
            j -= k
            yield x_read[rx.i], rx.round - 1
            x[rx.i, g] = n
            x_full[rx.i].arrive()
            rx.next()

    def epilogue():
        ra, rc, rx = Ring(2), Ring(2), Ring(sums)
        for turn, (n, _) in enumerate(live):
            yield from take_c(rc, n)
            yield x_full[rx.i], rx.round
            assert all(x[rx.i, g] == n for g in range(groups))
            x_read[rx.i].arrive()
            rx.next()
            yield acc_full, turn
            acc_free.arrive()
            assert a[ra.i] == n  # dQ is staged over it
            a_empty[ra.i].arrive()
            ra.next()

    roles = {"load": load(), "scores": scores(), "products": products(), "epilogue": epilogue()}
    roles.update({f"aux {i}": aux(i) for i in range(aux_warps)}, **{f"group {g}": group(g) for g in range(groups)})
    roles.update({f"dot {i}": dot(i) for i in range(sets)})
    w.run(roles)


# ----------------------------------------------------- backward, second pass
def backward_second(rng, D, items):
    """items: the query tiles of each."""
    groups, slots, bufs = (3, 6, 2) if D == 64 else (2, 3, 1)
    aux_warps = 3
    w = World(rng)
    a_full, a_empty = barriers("a_full", bufs), barriers("a_empty", bufs)
    n_full, n_empty, n_aux = (barriers(n, slots) for n in ("n_full", "n_empty", "n_aux"))
    s_full, p_full = barriers("s_full", groups), barriers("p_full", groups)
    acc_full, acc_free = Barrier("acc_full"), Barrier("acc_free")
    w.mmas = {"scores": [], "products": []}
    a, n_at, terms = {}, {}, {}  # what the slots hold
    live = [(n, k) for n, k in enumerate(items) if k > 0]

    def land(barrier, holds, slot, what):
        def now():
            holds[slot] = what
            barrier.arrive()
        w.loads.append(now)

    def reads(queue, *pairs):
        def now():
            for holds, slot, what in pairs:
                assert holds.get(slot) == what, f"{holds.get(slot)} read for {what}"
        w.mmas[queue].append(now)

    def load():
        ra, rn = Ring(bufs), Ring(slots)
        for n, k in live:
            yield a_empty[ra.i], ra.round - 1
            land(a_full[ra.i], a, ra.i, n)
            ra.next()
            for j in range(k):
                yield n_empty[rn.i], rn.round - 1
                land(n_full[rn.i], n_at, rn.i, (n, j))
                rn.next()

    def scores():
        ra, rn, before, stage, fresh = Ring(bufs), Ring(slots), Ring(slots), Ring(groups), groups
        for n, k in live:
            yield a_full[ra.i], ra.round
            for j in range(k):
                yield n_full[rn.i], rn.round
                yield n_aux[rn.i], rn.round
                if fresh == 0:
                    yield n_empty[before.i], before.round
                    before.next()
                else:
                    fresh -= 1
                reads("scores", (n_at, rn.i, (n, j)), (terms, rn.i, (n, j)), (a, ra.i, n))
                w.mmas["scores"].append(s_full[stage.i].arrive)
                rn.next()
                stage.next()
            w.mmas["scores"].append(a_empty[ra.i].arrive)
            ra.next()

    def products():
        rn, stage = Ring(slots), Ring(groups)
        for turn, (n, k) in enumerate(live):
            for j in range(k):
                if j == 0:
                    yield acc_free, turn - 1
                yield p_full[stage.i], stage.round
                reads("products", (n_at, rn.i, (n, j)))
                w.mmas["products"].append(n_empty[rn.i].arrive)
                rn.next()
                stage.next()
            w.mmas["products"].append(acc_full.arrive)

    def aux(i):
        rn, j = Ring(slots), i
        rn.next(i)
        for n, k in live:
            while j < k:
                yield n_empty[rn.i], rn.round - 1
                terms[rn.i] = (n, j)
                n_aux[rn.i].arrive()
                rn.next(aux_warps)
                j += aux_warps
            j -= k

    def group(g):
        turn, j = 0, g
        for n, k in live:
            while j < k:
                yield s_full[g], turn
                turn += 1
                p_full[g].arrive()
                j += groups
            j -= k

    def epilogue():
        for turn in range(len(live)):
            yield acc_full, turn
            acc_free.arrive()

    roles = {"load": load(), "scores": scores(), "products": products(), "epilogue": epilogue()}
    roles.update({f"aux {i}": aux(i) for i in range(aux_warps)}, **{f"group {g}": group(g) for g in range(groups)})
    w.run(roles)


@pytest.mark.parametrize("D", [64, 128])
def test_forward_waits(D):
    for seed in range(600):
        rng = random.Random(seed)
        forward(rng, D, forward_items(rng, D), rng.random() < 0.6)


@pytest.mark.parametrize("D", [64, 128])
def test_backward_waits(D):
    for seed in range(400):
        rng = random.Random(seed)
        items = [rng.choice([0, 1, 1, 2, 2, 3, 4, 7]) for _ in range(rng.randint(1, 9))]
        backward(rng, D, items, rng.random() < 0.6)
        backward_second(rng, D, items)


# what the model finds where a rule of the kernel is left out: at D = 64, items
# of six key tiles (all of the ring) after one without rows for tiles 2 and 3
SIX = [dict(nkt=6, nact=n, keys=i, loads=True, free=True) for i, n in enumerate((1, 4, 1, 4))]
ONE = [dict(nkt=1, nact=n, keys=i, loads=True, free=True) for i, n in enumerate((4, 3, 4, 4, 3, 4, 4))]


@pytest.mark.parametrize("items,rule", [(SIX, "every_step"), (ONE, "ring_per_warp")])
def test_the_model_finds_a_wait_for_the_wrong_round(items, rule):
    found = None
    for seed in range(4000):
        try:
            forward(random.Random(seed), 64, items, True, **{rule: False})
        except AssertionError as e:
            found = str(e)
            break
    assert found is not None
    for seed in range(300):
        forward(random.Random(seed), 64, items, True)
