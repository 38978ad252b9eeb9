"""The barriers of the cache attention kernels, checked on the CPU against a
restatement of their roles as coroutines under random schedules.

Prompt kernel (``csrc/kv_prompt.cu``): the unpacking warps announce a tile's
exponents in a ring of four (``info_full``) before its key operand; the
softmax warps of an M tile read them for each tile of the items the M tile
takes part in.  An M tile that sits out an item does not wait for that item's
tiles, so when it comes back the parity of ``info_full`` may pass for a round
that is not there yet, and then it has not acquired what the unpacking warps
wrote.  Waiting for the tile's S first makes the second wait exact.
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
