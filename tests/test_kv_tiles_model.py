"""Host model of the barriers of the tiled attention kernels (csrc/mq_kv_prefill.cu).

Every warp of kv_tiles_f32_kernel and kv_tiles_kernel is a generator of the waits and arrivals that the kernel makes, in its
order, with the tiles that it reads and writes in shared memory and TMEM; the tensor core is one more actor that takes its
work and its commits in order.  Schedules run the actors at random and with each actor, or each kind, as late as the barriers allow.
Checked on each: every actor ends; no barrier completes a phase while a warp still has to look for the one before it (a wait
sees a parity only); whatever is read is the tile that was meant; and what warps read of one another's shared memory, or
overwrite in it, is ordered by barriers that they arrived at and waited for (a tensor core's arrival orders none of that).
"""
import random

import pytest

INFO = 4                                       # tiles that the lookup runs ahead


class Bar:
    def __init__(self, count):
        self.count, self.left, self.done, self.clock, self.next = count, count, 0, {}, {}


def join(a, b):
    for k, v in b.items():
        a[k] = max(a.get(k, 0), v)


class Run:
    """Actors, barriers, and memory places with who wrote and read them when."""

    def __init__(self, bars):
        self.bars = {k: Bar(n) for k, n in bars.items()}
        self.mem, self.clock, self.actors, self.queue = {}, {}, {}, []

    def arrive(self, name, who=None):
        b = self.bars[name]
        if who is not None:
            join(b.next, self.clock[who])
        b.left -= 1
        assert b.left >= 0
        if b.left == 0:
            b.done, b.left = b.done + 1, b.count
            join(b.clock, b.next)

    def write(self, who, place, value):
        if place in self.mem:
            for actor, at in self.mem[place][1]:
                assert actor == who or self.clock[who].get(actor, 0) >= at, f"{who} overwrites {place} under {actor}"
        self.clock[who][who] = self.clock[who].get(who, 0) + 1
        self.mem[place] = (value, [(who, self.clock[who][who])])

    def read(self, who, place, value):
        have, events = self.mem[place]
        assert have == value, f"{who} reads {place}: {have}, not {value}"
        writer, at = events[0]
        assert writer == who or self.clock[who].get(writer, 0) >= at, f"{who} reads {place} of {writer} unordered"
        self.clock[who][who] = self.clock[who].get(who, 0) + 1
        events.append((who, self.clock[who][who]))

    def run(self, actors, pick):
        self.actors = {name: g for name, g in actors.items()}
        self.clock = {name: {name: 1} for name in actors}
        ops = {name: next(g, None) for name, g in self.actors.items()}
        while True:
            ready = []
            for name, op in ops.items():
                if op is None or (op[0] == "idle" and not self.queue):
                    continue
                if op[0] == "wait":                            # ("wait", barrier, phase)
                    b = self.bars[op[1]]
                    assert b.done <= op[2] + 1, f"{name}: {op[1]} is past phase {op[2]}"
                    if b.done & 1 == op[2] & 1:
                        continue
                ready.append(name)
            live = [n for n, op in ops.items() if op is not None and op[0] != "idle"]
            if not ready:
                assert not live, f"stuck: {[(n, ops[n]) for n in live]}"
                return
            name = pick(ready)
            op = ops[name]
            if op[0] == "wait":
                join(self.clock[name], self.bars[op[1]].clock)
            elif op[0] == "arrive":
                self.arrive(op[1], name)
            ops[name] = next(self.actors[name], None)


def order(j, half, nj):
    return (2 * nj - 1 if j == nj - 1 else 2 * j + 2) if half else (0 if j == 0 else 2 * j - 1)


def tensor_core(r):
    """what the MMA warp has issued, in order"""
    while True:
        yield ("idle",)
        if r.queue:
            r.queue.pop(0)()


def lookup(r, me, nj):
    for j in range(nj):
        if j >= INFO:
            yield ("wait", f"info_empty{j % INFO}", j // INFO - 1)
        r.write(me, f"info{j % INFO}", j)
        yield ("arrive", f"info_full{j % INFO}")


def widen(r, me, wi, nj, slots):
    half = wi >> 1
    for j in range(nj):
        yield ("wait", f"info_full{j % INFO}", j // INFO)
        r.read(me, f"info{j % INFO}", j)
        yield ("arrive", f"info_empty{j % INFO}")
        n = order(j, half, nj)
        if n >= slots:
            yield ("wait", f"op_empty{n % slots}", n // slots - 1)
        yield ("arrive", f"op_full{n % slots}")


def check_pages(r, me):
    r.write(me, "lost", 0)
    yield ("arrive", "pages")


class Issue:
    def __init__(self, r, slots):
        self.r, self.slots, self.n = r, slots, 0

    def commit(self, name):
        self.r.queue.append(lambda: self.r.arrive(name))

    def scores(self, buf, j):
        self.r.queue.append(lambda: self.r.mem.__setitem__(f"S{buf}", {"S": j}))

    def output(self, buf, p, j, add):
        def go():
            s = self.r.mem[f"S{p}"]
            assert s["S"] == j and all(s.get(w) == j for w in range(4)), f"weights of tile {j}: {s}"
            assert not add or self.r.mem[f"O{buf}"] == j - 1
            self.r.mem[f"O{buf}"] = j
        self.r.queue.append(go)


def f32_mma(r, nj, slots):
    i, n = Issue(r, slots), 0
    if nj:
        yield ("wait", "q_full", 0)
        yield ("wait", "op_full0", 0)
        i.scores(0, 0), i.commit("s_full0"), i.commit("op_empty0")
        n = 1
    for j in range(nj):
        at = j & 1
        if j + 1 < nj:
            yield ("wait", f"op_full{n % slots}", n // slots)
            i.scores(at ^ 1, j + 1), i.commit(f"s_full{at ^ 1}"), i.commit(f"op_empty{n % slots}")
            n += 1
        yield ("wait", f"op_full{n % slots}", n // slots)
        if j >= 2:
            yield ("wait", f"o_free{at}", (j >> 1) - 1)
        yield ("wait", f"p_full{at}", j >> 1)
        i.output(at, at, j, False), i.commit(f"o_done{at}"), i.commit(f"op_empty{n % slots}")
        n += 1
    i.commit("drain")
    yield ("wait", "drain", 0)


def f32_softmax(r, me, w, nj, sums_wait):
    a2, row = w >> 2, w & 3
    yield ("arrive", "q_full")
    for j in range(nj + 2):
        at = j & 1
        if j >= 2:
            for bar in sums_wait(j, nj, at, a2):
                yield ("wait", f"{bar}{at}", (j >> 1) - 1)
            r.read(me, f"f{(j - 2) & 3},{row}", j - 2)
            assert r.mem[f"O{at}"] == j - 2
            yield ("arrive", f"o_free{at}")
        if j >= nj or at != a2:
            continue
        yield ("wait", f"info_full{j % INFO}", j // INFO)
        yield ("wait", f"s_full{at}", j >> 1)
        r.read(me, f"info{j % INFO}", j)
        assert r.mem[f"S{at}"]["S"] == j
        if j > 0:
            yield ("wait", f"m_full{at ^ 1}", (j - 1) >> 1)
            r.read(me, f"m{(j - 1) & 3},{row}", j - 1)
        r.write(me, f"m{j & 3},{row}", j)
        r.write(me, f"f{j & 3},{row}", j)
        yield ("arrive", f"m_full{at}")
        yield ("arrive", f"info_empty{j % INFO}")
        r.mem[f"S{at}"][row] = j
        yield ("arrive", f"p_full{at}")
    r.write(me, f"l{a2},{row}", f"sum{a2}")
    yield ("arrive", "l_full")
    yield ("wait", "l_full", 0)
    yield ("wait", "pages", 0)
    r.read(me, "lost", 0)
    for g in range(2):
        r.read(me, f"l{g},{row}", f"sum{g}")
    if nj:
        r.read(me, f"m{(nj - 1) & 3},{row}", nj - 1)


def f32_actors(r, nj, sums_wait):
    slots = 4
    a = {"lookup": lookup(r, "lookup", nj), "mma": f32_mma(r, nj, slots), "tc": tensor_core(r), "check": check_pages(r, "check")}
    a.update({f"widen{i}": widen(r, f"widen{i}", i, nj, slots) for i in range(4)})
    a.update({f"soft{w}": f32_softmax(r, f"soft{w}", w, nj, sums_wait) for w in range(8)})
    return a


def f32_bars():
    b = {"q_full": 8, "drain": 1, "l_full": 8, "pages": 1}
    b.update({f"op_full{i}": 2 for i in range(4)}, **{f"op_empty{i}": 1 for i in range(4)})
    b.update({f"info_full{i}": 1 for i in range(INFO)}, **{f"info_empty{i}": 8 for i in range(INFO)})
    for i in range(2):
        b.update({f"s_full{i}": 1, f"p_full{i}": 4, f"o_done{i}": 1, f"o_free{i}": 8, f"m_full{i}": 4})
    return b


def half_mma(r, nj, nt, slots):
    i, n = Issue(r, slots), 0
    if nj:
        yield ("wait", "q_full", 0)
        yield ("wait", "op_full0", 0)
        for t in range(nt):
            i.scores(t, 0), i.commit(f"s_full{t}")
        i.commit("op_empty0")
        n = 1
    for j in range(nj):
        more, k = j + 1 < nj, n
        n += more
        v = n
        n += 1
        if more:
            yield ("wait", f"op_full{k % slots}", k // slots)
        yield ("wait", f"op_full{v % slots}", v // slots)
        for t in range(nt):
            yield ("wait", f"p_full{t}", j)
            i.output(t, t, j, j > 0), i.commit(f"o_done{t}")
            if t == nt - 1:
                i.commit(f"op_empty{v % slots}")
            if more:
                i.scores(t, j + 1), i.commit(f"s_full{t}")
        if more:
            i.commit(f"op_empty{k % slots}")
    i.commit("drain")
    yield ("wait", "drain", 0)


def half_softmax(r, me, w, nj, nt, rescale):
    t, row = w >> 2, w & 3
    yield ("arrive", "q_full")
    if t >= nt:
        return
    for j in range(nj):
        yield ("wait", f"info_full{j % INFO}", j // INFO)
        r.read(me, f"info{j % INFO}", j)
        yield ("arrive", f"info_empty{j % INFO}")
        yield ("wait", f"s_full{t}", j)
        assert r.mem[f"S{t}"]["S"] == j
        if j > 0 and rescale():
            yield ("wait", f"o_done{t}", j - 1)
            assert r.mem[f"O{t}"] == j - 1
        r.mem[f"S{t}"][row] = j
        yield ("arrive", f"p_full{t}")
    if nj:
        yield ("wait", f"o_done{t}", nj - 1)
        assert r.mem[f"O{t}"] == nj - 1
    yield ("wait", "pages", 0)
    r.read(me, "lost", 0)


def half_actors(r, nj, nt, rescale):
    slots = 5
    a = {"lookup": lookup(r, "lookup", nj), "mma": half_mma(r, nj, nt, slots), "tc": tensor_core(r), "check": check_pages(r, "check")}
    a.update({f"widen{i}": widen(r, f"widen{i}", i, nj, slots) for i in range(4)})
    a.update({f"soft{w}": half_softmax(r, f"soft{w}", w, nj, nt, rescale) for w in range(8)})
    return a


def half_bars(nt):
    b = {"q_full": 8, "drain": 1, "pages": 1}
    b.update({f"op_full{i}": 2 for i in range(5)}, **{f"op_empty{i}": 1 for i in range(5)})
    b.update({f"info_full{i}": 1 for i in range(INFO)}, **{f"info_empty{i}": 4 * nt + 4 for i in range(INFO)})
    for i in range(2):
        b.update({f"s_full{i}": 1, f"p_full{i}": 4, f"o_done{i}": 1})
    return b


NAMES = ["lookup", "mma", "tc", "check"] + [f"widen{i}" for i in range(4)] + [f"soft{w}" for w in range(8)]


def schedules(seed):
    """ways to pick the next actor: at random, at random by weights of many sizes, one actor or some of them as late as possible"""
    rng = random.Random(seed)
    for _ in range(4):
        yield rng.choice
    for _ in range(8):
        weight = {n: 10.0 ** rng.uniform(-3, 0) for n in NAMES}
        yield lambda ready, weight=weight: rng.choices(ready, [weight[n] for n in ready])[0]
    late = [{n} for n in NAMES] + [{f"soft{w}" for w in range(4)}, {f"soft{w}" for w in range(4, 8)}] + [set(rng.sample(NAMES, 4)) for _ in range(8)]
    for some in late:
        yield lambda ready, some=some: rng.choice([n for n in ready if n not in some] or ready)


def kernel_wait(j, nj, at, a2):
    return ["o_done"] + (["m_full"] if j == nj + 1 and at != a2 else [])


@pytest.mark.parametrize("nj", [0, 1, 2, 3, 4, 5, 9, 14])
def test_f32_tiles(nj):
    for pick in schedules(nj):
        r = Run(f32_bars())
        r.run(f32_actors(r, nj, kernel_wait), pick)


@pytest.mark.parametrize("nj", [0, 1, 2, 3, 5, 6, 13])
@pytest.mark.parametrize("nt", [1, 2])
def test_16_bit_tiles(nj, nt):
    rng = random.Random(nj)
    for pick in schedules(nj + nt):
        r = Run(half_bars(nt))
        r.run(half_actors(r, nj, nt, lambda: rng.random() < 0.4), pick)


def test_the_model_sees_a_wait_that_can_miss_its_phase():
    # the sums of f32 rows waiting for p_full too: its owner may arrive for the next tile but one before a late warp has looked
    def found(pick):
        r = Run(f32_bars())
        try:
            r.run(f32_actors(r, 9, lambda j, nj, at, a2: ["p_full", "o_done"]), pick)
        except AssertionError as e:
            return "p_full" in str(e)
        return False
    assert any(found(pick) for pick in schedules(1))


def test_the_model_sees_an_unordered_read():
    # ... and after the last tile the other warpgroup's factors come with its m_full, not with the products
    r = Run(f32_bars())
    with pytest.raises(AssertionError, match="unordered"):
        for pick in schedules(2):
            r = Run(f32_bars())
            r.run(f32_actors(r, 5, lambda j, nj, at, a2: ["o_done"]), pick)
