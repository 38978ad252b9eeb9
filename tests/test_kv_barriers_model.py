"""The barriers of the cache attention kernels, checked on the CPU against a
restatement of their roles as coroutines under random schedules.

Prompt kernel (``csrc/kv_prompt.cu``): the unpacking warps announce a tile's
exponents in a ring of four (``info_full``) before its key operand; the
softmax warps of an M tile read them for each tile of the items the M tile
takes part in.  An M tile that sits out an item does not wait for that item's
tiles, so when it comes back the parity of ``info_full`` may pass for a round
that is not there yet, and then it has not acquired what the unpacking warps
wrote.  Waiting for the tile's S first makes the second wait exact.

Both kernels: a warp fills stages by bulk copies that consumer warps wait for.
Every wait is bounded; a consumer whose wait ran out sets a flag and goes on
without waiting, so it frees stages whose copies may not have landed.  The
copying warp looks at the flag before it fills a stage, and waits for its last
copies before it ends.
"""

from __future__ import annotations

import random

import pytest


class Barrier:
    """An mbarrier: phases complete after `count` arrivals and all expected bytes."""

    def __init__(self, count):
        self.count, self.left, self.tx, self.phase = count, count, 0, 0

    def arrive(self):
        assert self.left > 0, "an arrival too many in one phase"
        self.left -= 1
        self._turn()

    def land(self, n):
        self.tx -= n
        self._turn()

    def _turn(self):
        if self.left == 0 and self.tx == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passes(self, parity):
        """A wait for the phase of this parity."""
        return (self.phase & 1) != parity


def run(roles, rng):
    """Steps the roles (generators that yield a condition to wait for) in random order, some much slower than others."""
    waiting = {name: next(r, None) for name, r in roles.items()}
    weight = {name: rng.choice([1, 1, 10, 100]) for name in roles}
    while any(w is not None for w in waiting.values()):
        ready = [n for n, w in waiting.items() if w is not None and w()]
        assert ready, "no role can go on"
        name = rng.choices(ready, [weight[n] for n in ready])[0]
        waiting[name] = next(roles[name], None)


class PassedEarly(Exception):
    pass


INFO, K_STAGES = 4, 2


def prompt(items, v_stages, s_first, rng):
    """items: (tiles, M tiles that take part).  Raises PassedEarly when a softmax warp's wait for a tile's exponents
    passed on another round of the ring."""
    info_full = [Barrier(1) for _ in range(INFO)]
    k_full, k_empty = ([Barrier(1) for _ in range(K_STAGES)] for _ in range(2))
    v_full, v_empty = ([Barrier(1) for _ in range(v_stages)] for _ in range(2))
    q_full, s_full, p_full, o_full = ([Barrier(1) for _ in range(2)] for _ in range(4))
    infos = [None] * INFO

    def wait(bar, parity):
        return lambda: bar.passes(parity & 1)

    def unpack():
        kt = 0
        for n, _ in items:
            for _ in range(n):
                infos[kt % INFO] = kt
                info_full[kt % INFO].arrive()
                yield wait(k_empty[kt % K_STAGES], (kt // K_STAGES & 1) ^ 1)
                k_full[kt % K_STAGES].arrive()
                yield wait(v_empty[kt % v_stages], (kt // v_stages & 1) ^ 1)
                v_full[kt % v_stages].arrive()
                kt += 1

    def mma():
        kt, taken, steps = 0, [0, 0], [0, 0]
        for n, m_tiles in items:
            for m in range(m_tiles):
                yield wait(q_full[m], taken[m])
                taken[m] += 1
                if m == 0:
                    yield wait(k_full[kt % K_STAGES], kt // K_STAGES)
                s_full[m].arrive()
            k_empty[kt % K_STAGES].arrive()
            for i in range(n):
                yield wait(v_full[kt % v_stages], kt // v_stages)
                if i + 1 < n:
                    yield wait(k_full[(kt + 1) % K_STAGES], (kt + 1) // K_STAGES)
                for m in range(m_tiles):
                    yield wait(p_full[m], steps[m])
                    steps[m] += 1
                    (s_full if i + 1 < n else o_full)[m].arrive()
                v_empty[kt % v_stages].arrive()
                if i + 1 < n:
                    k_empty[(kt + 1) % K_STAGES].arrive()
                kt += 1

    def softmax(m):
        kt = steps = taken = 0
        if items[0][1] > m:
            q_full[m].arrive()
        for at, (n, m_tiles) in enumerate(items):
            if m_tiles > m:
                for k in range(kt, kt + n):
                    if s_first:
                        yield wait(s_full[m], steps)
                    yield wait(info_full[k % INFO], k // INFO)
                    if info_full[k % INFO].phase != k // INFO + 1:
                        raise PassedEarly(f"tile {k} in round {info_full[k % INFO].phase}")
                    if not s_first:
                        yield wait(s_full[m], steps)
                    assert infos[k % INFO] == k
                    steps += 1
                    p_full[m].arrive()
            kt += n
            if at + 1 < len(items) and items[at + 1][1] > m:
                q_full[m].arrive()
            if m_tiles > m:
                yield wait(o_full[m], taken)
                taken += 1

    run({"unpack": unpack(), "mma": mma(), "softmax 0": softmax(0), "softmax 1": softmax(1)}, rng)


def items_of(rng):
    return [(rng.randint(1, 14), rng.randint(1, 2)) for _ in range(rng.randint(1, 12))]


@pytest.mark.parametrize("v_stages", [1, 2])
def test_prompt_exponents_are_the_tiles_own(v_stages):
    for seed in range(600):
        rng = random.Random(seed)
        prompt(items_of(rng), v_stages, True, rng)


def test_the_other_order_passes_early():
    with pytest.raises(PassedEarly):
        for seed in range(600):
            rng = random.Random(seed)
            prompt(items_of(rng), 2, False, rng)


# ------------------------------------------------------------ rings of bulk copies

class InFlight(Exception):
    pass


def ring(tiles, stages, consumers, looks, drains, rng):
    """One ring of stages that a producer fills by copies and consumer warps empty, any of which may give up any wait
    that does not pass at once (a bounded wait that ran out), and then goes on without waiting.  `looks`: the producer
    reads the flag of a warp that gave up before it fills a stage; `drains`: at its end it waits for its last copies.
    Raises InFlight when a stage is filled again, or the block ends, while copies into it are on their way."""
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(consumers) for _ in range(stages)]
    flying = [0] * stages  # copies on their way, by stage
    state = {"abort": False, "done": 0}
    patience = rng.choice([0.0, 0.02, 0.3])

    def wait(bar, parity, result):
        def ready():
            result["ok"] = bar.passes(parity & 1)
            if not result["ok"] and (state["abort"] or rng.random() < patience):
                state["abort"] = True
                return True
            return result["ok"]
        return ready

    def producer():
        r, issued = {}, 0
        for k in range(tiles):
            s = k % stages
            yield wait(empty[s], (k // stages & 1) ^ 1, r)
            if not r["ok"] or (looks and state["abort"]):
                break
            if full[s].left != 1 or flying[s]:
                raise InFlight(f"stage {s} filled again")
            full[s].tx += 1
            flying[s] += 1
            full[s].arrive()
            issued += 1
            yield lambda: True
        if drains:
            for k in range(max(issued - stages, 0), issued):
                yield lambda k=k: full[k % stages].passes(k // stages & 1)
        state["done"] += 1

    def consumer():
        r = {}
        for k in range(tiles):
            s = k % stages
            yield wait(full[s], k // stages, r)
            yield lambda: True
            empty[s].arrive()
        state["done"] += 1

    def memory():
        while state["done"] < consumers + 1 or any(flying):
            if state["done"] == consumers + 1:
                raise InFlight("the block ended")
            s = rng.randrange(stages)
            if flying[s]:
                flying[s] -= 1
                full[s].land(1)
            yield lambda: True

    run({"producer": producer(), "memory": memory(), **{f"consumer {i}": consumer() for i in range(consumers)}}, rng)


@pytest.mark.parametrize("stages,consumers", [(1, 4), (2, 4), (3, 4)])
def test_copies_land_in_the_block_that_waits_for_them(stages, consumers):
    for seed in range(400):
        rng = random.Random(seed)
        ring(rng.randint(0, 9), stages, consumers, True, True, rng)


@pytest.mark.parametrize("looks,drains", [(False, True), (True, False)])
def test_either_omission_shows(looks, drains):
    with pytest.raises(InFlight):
        for seed in range(400):
            rng = random.Random(seed)
            ring(rng.randint(0, 9), 3, 4, looks, drains, rng)
