"""CPU model of the hand-offs inside the delta rule's chain kernel
(bayesian_filtering_linear_gb300/csrc/kla_delta_chunk.cu).

A block has warps that keep the state, warps that bring K and W, and one that
issues the products and the copies of M (β V) and the gates. They meet by two
named barriers and by mbarriers whose arrivals also come from copies and from
finished products, at any later time. This file restates each role's waits,
arrivals and accesses in the kernel's order and checks, over random
interleavings, that every role finishes, that nothing is overwritten while a
product or a warp still reads it, that nothing is read before it is there, and
that the block does not end with an arrival or a copy on its way to its shared
memory. Planted mistakes must be caught."""
import random

import pytest


class Barrier:
    """Phases of `count` arrivals; a wait goes by the phase's parity alone."""

    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def run(N, stages, ahead, seed, mistake="", warps=2):
    """A block's walk over N chunks; `warps` warps stand for each group."""
    rng = random.Random(seed)
    m = {f"full{b}": Barrier(warps + 1) for b in range(stages)}  # the feeding warps and the copy
    m.update({f"empty{b}": Barrier(1) for b in range(stages)})
    m.update({f"loaded{b}": Barrier(1) for b in range(ahead)})
    m.update({"done0": Barrier(1), "done1": Barrier(1)})
    named = {1: Barrier(warps + 1), 2: Barrier(warps + 1)}
    held, parts = {}, {}   # what a place holds, and which warps have written their part of it
    reading = []           # places that warps are reading
    products = []          # issued, not done: (places read, accumulator, its readers, arrivals)
    flying = []            # arrivals and copies under way
    unread = {}            # accumulator -> warps that are still to read it

    def write(place, what, warp=None):
        assert all(place not in [p for p, _ in reads] for reads, *_ in products), f"{place} is still an operand"
        assert place not in reading, f"{place} is still being read"
        parts.setdefault((place, what), set()).add(warp)
        if warp is None or len(parts[(place, what)]) == warps:
            held[place] = what

    def issue(reads, acc, arrivals):
        for place, what in reads:
            assert held.get(place) == what, f"a product takes {place} with {held.get(place)} for {what}"
        assert not unread.get(acc), f"{acc} is still to be read"
        unread[acc] = set(range(warps))
        products.append((reads, acc, arrivals))

    def copy(place, what, barrier):
        flying.append(("copy", place, what, barrier))

    def land():  # a product is done, or an arrival or a copy comes in
        if products and (not flying or rng.random() < 0.5):
            _, acc, arrivals = products.pop(0)
            flying.extend(("arrive", b) for b in arrivals)
            ready.add(acc)
        elif flying:
            f = flying.pop(rng.randrange(len(flying)))
            if f[0] == "copy":
                write(f[1], f[2])
                m[f[3]].arrive()
            else:
                m[f[1]].arrive()

    ready = set()

    def wait(name, parity):
        while not m[name].passed(parity):
            yield

    def sync(i, phase):
        named[i].arrive()
        while named[i].phase <= phase:
            yield

    def issuing():
        def bring(i):
            if i < N:
                copy(f"B{i % ahead}", i, f"loaded{i % ahead}")

        for i in range(ahead):
            bring(i)
        for i in range(N):
            b = i % stages
            yield from wait(f"full{b}", i // stages & 1)
            yield from sync(1, i)
            ready.discard("P")
            issue([(f"W{b}", i), ("X", i)], "P", ["done0"])
            yield from sync(2, i)
            ready.discard("P")
            issue([(f"K{b}", i), ("U", i)], "P", ["done1", f"empty{b}"])
            bring(i + ahead)
        for i in range(max(N - stages, 0), N):
            yield from wait(f"full{i % stages}", i // stages & 1)
            if mistake != "the last places are not waited for":
                yield from wait(f"empty{i % stages}", i // stages & 1)
        for i in range(max(N - ahead, 0), N):
            yield from wait(f"loaded{i % ahead}", i // ahead & 1)

    def feeding(me):
        for i in range(N):
            b = i % stages
            if i >= stages and mistake != "a place is taken early":
                yield from wait(f"empty{b}", (i // stages - 1) & 1)
            if me == 0:
                copy(f"W{b}", i, f"full{b}")
            write(f"K{b}", i, me)
            m[f"full{b}"].arrive()
            yield

    def state(me):
        for i in range(N):
            write("X", i, me)
            named[1].arrive()
            if mistake != "the copies of M V are not waited for":
                yield from wait(f"loaded{i % ahead}", i // ahead & 1)
            assert held.get(f"B{i % ahead}") == i, "M V is not there"
            reading.append(f"B{i % ahead}")
            yield
            reading.remove(f"B{i % ahead}")
            yield from wait("done0", i & 1)
            assert "P" in ready and me in unread["P"], "the first product is not there"
            unread["P"].discard(me)
            write("U", i, me)
            named[2].arrive()
            yield
            if mistake != "the second product is not waited for":
                yield from wait("done1", i & 1)
            assert "P" in ready and me in unread["P"], "the second product is not there"
            unread["P"].discard(me)

    tasks = {"issue": issuing()}
    for w in range(warps):
        tasks.update({f"feed{w}": feeding(w), f"state{w}": state(w)})
    idle, eager = 0, rng.choice([0.05, 0.3, 0.8])
    while tasks:
        if (products or flying) and rng.random() < eager:
            land()
            idle = 0
            continue
        n = rng.choice(list(tasks))
        try:
            next(tasks[n])
        except StopIteration:
            del tasks[n]
        idle += 1
        assert idle < 20000, f"stuck: {sorted(tasks)}"
    assert not products and not flying, f"the block ends with {flying or products} under way"


@pytest.mark.parametrize("stages,ahead", [(2, 2), (2, 1), (1, 2), (1, 1)])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 7])
def test_chain_finishes_without_races_and_leaves_nothing_under_way(N, stages, ahead):
    for seed in range(100):
        run(N, stages, ahead, seed)


@pytest.mark.parametrize("mistake", ["the last places are not waited for", "a place is taken early",
                                     "the copies of M V are not waited for", "the second product is not waited for"])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(100):
        try:
            run(5, 2, 2, seed, mistake)
        except AssertionError:
            caught += 1
    assert caught
