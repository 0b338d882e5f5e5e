"""A model of the barriers of the attention's tiles (tiles_kernel), without a GPU.

The kernel's roles run as coroutines in random order; copies and products end late, in any order and in
order.  It fails on an arrival past a barrier's count, on a wait that an earlier or a later phase answers, on a
tile read before it is there, before it is clean or after it was overwritten, on results overwritten before
they were read, on roles that wait for ever, and on a block that leaves with copies or products on their way.
With a stop (another block's wait ran out) every wait may give up from some moment on.

A warp arrives once here where its 32 threads arrive in the kernel."""
import random

import pytest

LOADERS, SOFTMAX = 4, 4                              # warps, of the softmax for each half
RING, RING_K = 5, 4                                  # bf16 keys and values, e4m3 keys


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.bytes, self.phase = name, count, count, 0, 0

    def _turn(self):
        if not self.pending and not self.bytes:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, expect=0):
        assert self.pending, f"arrival past the count of {self.name}"
        self.bytes += expect
        self.pending -= 1
        self._turn()

    def land(self, n=1):
        self.bytes -= n
        self._turn()

    def done(self, n):
        """Whether a wait for the n-th phase (from 0) by its parity goes on."""
        ok = self.phase & 1 != n & 1
        assert not ok or self.phase == n + 1, f"a wait for phase {n} of {self.name} answered by phase {self.phase - 1}"
        return ok


class Wait:
    def __init__(self, bar, n, drain=False):
        self.bar, self.n, self.drain = bar, n, drain


class Block:
    """One thread block over a list of items: dicts of id, count (blocks of keys), edge (first block that not
    every row attends whole) and two (whether the second half has rows)."""

    def __init__(self, items, fp8, rng, together, cleaning):
        self.items, self.fp8, self.rng, self.together, self.cleaning = items, fp8, rng, together, 2 if fp8 else cleaning
        b = {}
        for name, n, count in (("QF", 2, 1), ("TF", RING, 1), ("TE", RING, 1), ("VF", 2, LOADERS), ("VE", 2, 1), ("SF", 2, 1),
                               ("OF", 2, 1), ("MF", 2, 1), ("ME", 2, 3 + 2 * SOFTMAX + LOADERS), ("GF", 3, 1),
                               ("GE", 3, LOADERS), ("DR", 1, 1)):
            for i in range(n):
                b[name, i] = Barrier(f"{name}{i}", count)
        b["PF", 0], b["PF", 1] = Barrier("PF0", SOFTMAX + 1), Barrier("PF1", SOFTMAX)
        self.bars, self.stopped = b, False
        self.products, self.copies, self.slots = [], [], [None, None]
        self.q, self.k, self.v, self.staged = [None, None], {}, {}, {}
        self.o, self.read, self.written, self.cleaned = [None, None], {}, [], {}
        self.queries, self.armed = [0, 0], {"TF": [], "GF": []}      # copies of each half; (barrier, phase) of the others

    def wait(self, name, i, n):
        return Wait(self.bars[name, i], n)

    def commit(self, name, i):
        self.products.append(self.bars[name, i].arrive)

    def item(self, k):
        """The k-th item, once it is there."""
        got = yield self.wait("MF", k & 1, k >> 1)
        return self.slots[k & 1] if got else None

    # -- roles: each generator yields waits, and is sent whether they went on or gave up
    def walk(self):
        for k, item in enumerate(self.items + [None]):
            if k >= 2 and not (yield self.wait("ME", k & 1, (k >> 1) - 1)):
                return
            self.slots[k & 1] = item
            self.bars["MF", k & 1].arrive()
            yield

    def key_tile(self, n):
        return (n % RING_K, n // RING_K) if self.fp8 else (2 * n % RING, 2 * n // RING)

    def issuer(self):
        yield from self._issue()
        if not self.together and self.stopped:
            yield from self.drain_products()
            yield from self.drain_queries()

    def drain_products(self):
        self.commit("DR", 0)
        yield Wait(self.bars["DR", 0], 0, drain=True)

    def drain_queries(self):
        for t in range(2):
            if self.queries[t]:
                yield Wait(self.bars["QF", t], self.queries[t] - 1, drain=True)

    def _issue(self):
        phases, items, it, k = [0, 0], self.queries, 0, 0
        while True:
            item = yield from self.item(k)
            if item is None:
                return
            me, n, halves = self.bars["ME", k & 1], item["count"], range(2 if item["two"] else 1)
            k += 1
            if n:
                for t in halves:
                    self.q[t] = None
                    self.bars["QF", t].arrive(expect=1)

                    def landed(t=t, item=item):
                        self.q[t] = item["id"]
                        self.bars["QF", t].land()
                    self.copies.append(landed)
            me.arrive()
            if not n:
                continue
            for t in halves:
                items[t] += 1
            for t in halves:
                if not (yield self.wait("QF", t, items[t] - 1)):
                    return
            if not (yield self.wait("TF", *self.key_tile(it))):
                return
            for j in range(n + 1):
                ks = self.key_tile(it)[0]
                vs = (it - 1) & 1 if self.fp8 else (2 * it - 1) % RING
                for t in range(2):
                    if j > 0 and t in halves:
                        if not (yield self.wait("PF", t, phases[t])):
                            return
                        phases[t] += 1
                        self.products.append(lambda t=t, vs=vs, j=j, item=item: self.weigh(t, vs, item["id"], j - 1))
                        if j == n:
                            self.commit("OF", t)
                    if t == 1 and j > 0:
                        self.commit("VE" if self.fp8 else "TE", vs)
                    if j < n and t in halves:
                        self.products.append(lambda t=t, ks=ks, j=j, item=item: self.score(t, ks, item["id"], j))
                        self.commit("SF", t)
                if j < n:
                    self.commit("TE", ks)
                    it += 1
                yield

    def score(self, t, slot, item, j):
        assert self.k.get(slot) == (item, j) and self.q[t] == item, ("S", self.k.get(slot), self.q[t], item, j)

    def weigh(self, t, slot, item, j):
        assert self.v.get(slot) == (item, j, "clean"), ("V", self.v.get(slot), item, j)
        if self.o[t] not in (None, item):
            assert self.read[self.o[t], t] == SOFTMAX, ("results overwritten", t, self.o[t], item)
        self.o[t] = item

    def follower(self):
        it = edges = k = 0
        while True:
            item = yield from self.item(k)
            if item is None:
                return
            n = item["count"]
            for j in range(n):
                if not self.fp8 and j >= item["edge"]:
                    good = yield self.wait("GE", edges % self.cleaning, edges // self.cleaning)
                    edges += 1
                elif self.fp8:
                    good = yield self.wait("VF", it & 1, it >> 1)
                else:
                    good = yield self.wait("TF", (2 * it + 1) % RING, (2 * it + 1) // RING)
                if good and j + 1 < n:
                    good = yield self.wait("TF", *self.key_tile(it + 1))
                if good and it:
                    good = yield self.wait("PF", 0, it - 1)
                if not good:
                    return
                self.bars["PF", 0].arrive()
                it += 1
                yield
            self.bars["ME", k & 1].arrive()
            k += 1

    def copier(self):
        yield from self._copy(self.armed)
        if not self.together and self.stopped:
            yield from self.drain_copier()

    def drain_copier(self):
        for name, last in (("TF", RING_K if self.fp8 else RING), ("GF", self.cleaning)):
            for i, n in self.armed[name][-last:]:
                yield Wait(self.bars[name, i], n, drain=True)

    def leave(self):
        """One thread, when all roles have left."""
        if self.together:
            yield from self.drain_products()
        if self.together and self.stopped:
            yield from self.drain_queries()
            yield from self.drain_copier()

    def _copy(self, armed):
        nt = nk = nx = edges = k = 0
        while True:
            item = yield from self.item(k)
            if item is None:
                return
            n = item["count"]

            def start(name, i, phase, into, slot, value):
                armed[name].append((i, phase))
                self.bars[name, i].arrive(expect=1)
                into.pop(slot, None)

                def landed():
                    into[slot] = value
                    self.bars[name, i].land()
                self.copies.append(landed)
            if not self.fp8:
                for x in range(2 * n):
                    slot, j = nt % RING, x // 2
                    if nt >= RING and not (yield self.wait("TE", slot, nt // RING - 1)):
                        return
                    self.k.pop(slot, None), self.v.pop(slot, None)
                    if x & 1 and j >= item["edge"]:
                        armed["TF"].append((slot, nt // RING))
                        self.bars["TF", slot].arrive()               # the follower waits for the cleaners instead
                        start("GF", edges % self.cleaning, edges // self.cleaning, self.v, slot, (item["id"], j, "raw"))
                        edges += 1
                    elif x & 1:
                        start("TF", slot, nt // RING, self.v, slot, (item["id"], j, "clean"))
                    else:
                        start("TF", slot, nt // RING, self.k, slot, (item["id"], j))
                    nt += 1
                    yield
            else:
                for j in range(n + 2):
                    if j < n:
                        slot = nk % RING_K
                        if nk >= RING_K and not (yield self.wait("TE", slot, nk // RING_K - 1)):
                            return
                        start("TF", slot, nk // RING_K, self.k, slot, (item["id"], j))
                        nk += 1
                        yield
                    if j >= 2:
                        slot = nx & 1
                        if nx >= 2 and not (yield self.wait("GE", slot, (nx >> 1) - 1)):
                            return
                        start("GF", slot, nx >> 1, self.staged, slot, (item["id"], j - 2))
                        nx += 1
                        yield
            self.bars["ME", k & 1].arrive()
            k += 1

    def loader(self):
        nv = edges = k = 0
        while True:
            item = yield from self.item(k)
            if item is None:
                return
            n = item["count"]
            for j in range(0 if self.fp8 else item["edge"], n):
                key = item["id"], j
                if not self.fp8:
                    slot = (2 * (nv + j) + 1) % RING
                    if not (yield self.wait("GF", edges % self.cleaning, edges // self.cleaning)):
                        return
                    assert self.v.get(slot) == (*key, "raw"), ("cleaned", self.v.get(slot), key)
                    yield
                    self.cleaned[key] = self.cleaned.get(key, 0) + 1
                    if self.cleaned[key] == LOADERS:
                        self.v[slot] = (*key, "clean")
                    self.bars["GE", edges % self.cleaning].arrive()
                    edges += 1
                else:
                    slot = nv & 1
                    if nv >= 2 and not (yield self.wait("VE", slot, (nv >> 1) - 1)):
                        return
                    if not (yield self.wait("GF", slot, nv >> 1)):
                        return
                    assert self.staged.get(slot) == key, ("converted", self.staged.get(slot), key)
                    self.cleaned[key] = self.cleaned.get(key, 0) + 1
                    self.v[slot] = (*key, "clean" if self.cleaned[key] == LOADERS else "raw")
                    yield
                    assert self.staged.get(slot) == key
                    self.bars["VF", slot].arrive()
                    self.bars["GE", slot].arrive()
                    nv += 1
                yield
            if not self.fp8:
                nv += n
            self.bars["ME", k & 1].arrive()
            k += 1
            yield

    def softmax(self, t):
        phase = items = k = 0
        while True:
            item = yield from self.item(k)
            if item is None:
                return
            if t == 0 or item["two"]:
                for _ in range(item["count"]):
                    if not (yield self.wait("SF", t, phase)):
                        return
                    phase += 1
                    yield
                    self.bars["PF", t].arrive()
                if item["count"]:
                    if not (yield self.wait("OF", t, items)):
                        return
                    items += 1
                    assert self.o[t] == item["id"]
                yield
                key = item["id"], t
                self.read[key] = self.read.get(key, 0) + 1
                if self.read[key] == SOFTMAX:
                    self.written.append(key)
            self.bars["ME", k & 1].arrive()
            k += 1

    # -- the run
    def run(self, stop=lambda block, live, steps: False):
        rng = self.rng
        roles = [self.walk(), self.issuer(), self.follower(), self.copier()]
        last = len(roles) + LOADERS + 2 * SOFTMAX                    # leaves behind the others
        roles += [self.loader() for _ in range(LOADERS)] + [self.softmax(t) for t in range(2) for _ in range(SOFTMAX)] + [self.leave()]
        waits, live, idle, steps = [None] * len(roles), set(range(len(roles))), 0, 0
        speed = [rng.random() ** 2 + 0.02 for _ in roles]
        slow_copies, slow_products = rng.random() ** 3 + 0.02, rng.random() + 0.05
        while live:
            moved = False
            steps += 1
            self.stopped = self.stopped or stop(self, live, steps)
            if self.products and rng.random() < slow_products:
                self.products.pop(0)()
                moved = True
            if self.copies and rng.random() < slow_copies:
                self.copies.pop(rng.randrange(min(len(self.copies), 4)))()
                moved = True
            for i in rng.sample(sorted(live), len(live)):
                if rng.random() > speed[i] or (i == last and len(live) > 1):
                    continue
                w, went = waits[i], None
                if w is not None:
                    went = w.bar.done(w.n)
                    if not went and (w.drain or not self.stopped):
                        continue
                try:
                    waits[i] = roles[i].send(went)
                except StopIteration:
                    live.discard(i)
                moved = True
            idle = 0 if moved else idle + 1
            assert idle < 5000, f"roles {sorted(live)} wait for ever"
        assert not self.copies and not self.products, "copies or products on their way when the block leaves"
        if not self.stopped:
            want = [(i["id"], t) for i in self.items for t in range(2 if i["two"] else 1)]
            assert sorted(self.written) == sorted(want)
        return steps


def block(seed, fp8, together=True, cleaning=3):
    rng = random.Random(2 * seed + fp8)
    items = []
    for i in range(rng.randint(1, 9)):
        n = rng.choice([0, 1, 1, 1, 2, 2, 3, 4, 6])
        items.append(dict(id=i, count=n, edge=max(0, rng.choice([0, 0, n - 1, n - 2, n, n + 3])), two=rng.random() < 0.5))
    return Block(items, fp8, rng, together, cleaning)


@pytest.mark.parametrize("fp8", [False, True])
def test_all_items_are_computed(fp8):
    for seed in range(150):
        block(seed, fp8).run()


COPIER = 3                                           # of the roles


def at_a_random_moment(seed, fp8):
    moment = random.Random(seed).randint(1, block(seed, fp8).run())
    return lambda block, live, steps: steps >= moment


def when_a_role_has_left(seed, fp8):
    """With copies, or else products, still on their way."""
    return lambda block, live, steps: COPIER not in live and bool(block.copies or block.products)


@pytest.mark.parametrize("moment", [at_a_random_moment, when_a_role_has_left])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_stop_leaves_nothing_on_its_way(fp8, moment):
    for seed in range(100):
        block(seed, fp8).run(moment(seed, fp8))


@pytest.mark.parametrize("fp8", [False, True])
def test_the_model_finds_a_role_that_leaves_before_its_copies_land(fp8):
    """Where a role waits for what it has on its way only if it sees the stop itself, a later stop finds some."""
    with pytest.raises(AssertionError, match="on their way"):
        for seed in range(100):
            block(seed, fp8, together=False).run(when_a_role_has_left(seed, fp8))


def test_the_model_finds_three_tiles_in_cleaning_on_two_barriers():
    with pytest.raises(AssertionError):
        for seed in range(100):
            block(seed, False, cleaning=2).run()
