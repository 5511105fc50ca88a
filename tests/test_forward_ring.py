"""The forward kernel's K/V ring as a model: one producer and two MMA issuers (query tiles A and B)
that share stages through barriers of which a wait sees only a phase's parity, and copies that land
in any order. Random schedules look for a wait that is granted by another phase than its own (the
products would then read what the stage held before) and for a schedule in which nobody can move.
Protocols (attn_fwd_sm103.cu): "pass", the windowed kernel's, in which each issuer waits for and
releases the tiles that it does not use as well; and "skip", the causal kernel's, in which it does
not (their user releases them twice). With three query tiles and two Q buffers (hd 32 and 64) the
model finds a stale grant in "skip": those lengths take the windowed kernel."""
import random

import pytest


class Barrier:
    def __init__(self, count=1):
        self.count, self.left, self.done = count, count, 0     # done: completed phases

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def granted(self, phase):                                  # a wait for the parity of `phase`
        return (self.done - 1 - phase) % 2 == 0


def units_of(num_m, heads):
    """(key tiles, has a query tile B) of one CTA's units: `heads` of each pair, longest first."""
    out = []
    for jp in reversed(range((num_m + 1) // 2)):
        has_b = 2 * jp + 1 < num_m
        out += [((2 * jp + 1 if has_b else 2 * jp) + 1, has_b)] * heads
    return out


def run(units, stages, qbufs, protocol, seed):
    """None, or what went wrong under the schedule of this seed."""
    rng = random.Random(seed)
    full, empty = [Barrier() for _ in range(stages)], [Barrier(2) for _ in range(stages)]
    q_full, final = [Barrier() for _ in range(qbufs)], [Barrier(2) for _ in range(qbufs)]
    flying, passes = [], protocol == "pass"

    def wait(bar, phase):
        return bar, phase

    def producer():
        R = 0
        for u, (count, _) in enumerate(units):
            yield wait(final[u % qbufs], u // qbufs - 1)
            flying.append(q_full[u % qbufs])
            for _ in range(count):
                yield wait(empty[R % stages], R // stages - 1)
                flying.append(full[R % stages])
                R += 1

    def issuer(x):
        R = 0
        for u, (count, has_b) in enumerate(units):
            yield wait(q_full[u % qbufs], u // qbufs)
            uses = range(R, R + (0 if x == 1 and not has_b else count - 1 if x == 0 and has_b else count))
            if len(uses):
                yield wait(full[R % stages], R // stages)
            for r in uses:
                if qbufs == 2 and r + 1 in uses:               # the next scores before this P V
                    yield wait(full[(r + 1) % stages], (r + 1) // stages)
                shared = passes or (has_b if x == 0 else r < R + count - 1)
                for _ in range(1 if shared else 2):
                    empty[r % stages].arrive()
                if qbufs == 1 and r + 1 in uses:               # or, at hd 128, behind it
                    yield wait(full[(r + 1) % stages], (r + 1) // stages)
            for r in range(R + len(uses), R + count):
                if passes:
                    yield wait(full[r % stages], r // stages)
                    empty[r % stages].arrive()
            final[u % qbufs].arrive()
            R += count

    actors = [producer(), issuer(0), issuer(1)]
    waiting = [next(a) for a in actors]
    while any(w is not None for w in waiting):
        ready = [i for i, w in enumerate(waiting) if w is not None and w[0].granted(w[1])]
        moves = ready + ["land"] * min(len(flying), 1)
        if not moves:
            return "nobody can move"
        move = rng.choice(moves)
        if move == "land":
            flying.pop(rng.randrange(len(flying))).arrive()
            continue
        bar, phase = waiting[move]
        if bar.done != phase + 1:
            return f"a wait for phase {phase} granted by phase {bar.done - 1}"
        waiting[move] = next(actors[move], None)
    return None


# (query tiles, stages, Q buffers): hd 32 and 64 have three or four stages and two buffers, hd 128
# two stages and one buffer
CONFIGS = [(m, *ring) for m in (1, 2, 3, 4, 5, 6, 7, 9) for ring in ((3, 2), (4, 2), (2, 1))]


def stale(num_m, stages, qbufs):
    return num_m == 3 and qbufs == 2


@pytest.mark.parametrize("num_m,stages,qbufs", CONFIGS)
@pytest.mark.parametrize("protocol", ["pass", "skip"])
def test_every_wait_is_granted_by_its_own_phase(num_m, stages, qbufs, protocol):
    if protocol == "skip" and stale(num_m, stages, qbufs):
        protocol = "pass"                                      # what those lengths run
    for heads in (1, 2, 3):
        units = units_of(num_m, heads)
        for seed in range(150):
            assert run(units, stages, qbufs, protocol, seed) is None, (heads, seed)


@pytest.mark.parametrize("num_m,stages,qbufs", [c for c in CONFIGS if stale(*c)])
def test_the_model_finds_the_fault_of_an_issuer_that_skips_tiles(num_m, stages, qbufs):
    found = [run(units_of(num_m, 3), stages, qbufs, "skip", seed) for seed in range(3000)]
    assert any(f and "granted" in f for f in found)
