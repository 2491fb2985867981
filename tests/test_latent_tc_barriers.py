"""The waits and arrivals of the absorbed attention kernel's roles (csrc/pa_latent_tc.cu), a tile at a time, under
schedules that hold one role back as long as any other can go on.  A parity wait sees a barrier's last phase alone, so
a barrier that completes twice before a role has looked leaves that role waiting for ever."""
import itertools
import os
import random
import re

import pytest

import paged_kv_attention_04_gb300 as P

SOURCE = os.path.join(os.path.dirname(P.__file__), "csrc", "pa_latent_tc.cu")


def from_source(name, bufs):
    """Value of a constant of the kernel's Cfg, which may be kBufs itself."""
    with open(SOURCE) as f:
        m = re.search(rf"static constexpr int {name} = (\w+);", f.read())
    if not m:
        return 2  # (P's barriers alternate)
    return bufs if m.group(1) == "kBufs" else int(m.group(1))


class Barriers:
    def __init__(self, counts):
        self.count = counts
        self.pending = {b: n for b, n in counts.items()}
        self.phase = dict.fromkeys(counts, 0)

    def arrive(self, b):
        self.pending[b] -= 1
        if self.pending[b] == 0:
            self.pending[b] = self.count[b]
            self.phase[b] += 1

    def complete(self, b, parity):
        return (self.phase[b] & 1) != parity


def roles(units, bufs, p_bars, moves):
    """Every role as its sequence of ("wait", barrier, parity), ("arrive", barrier) and ("then", what to note).
    units: tiles of each; moves: tiles whose references move."""
    tiles = sum(units)
    first = set(itertools.accumulate(units)) | {0}  # tiles that begin a unit (and the end)

    def copy(h):
        for g in range(tiles):
            if g >= bufs:
                yield "wait", ("empty", h, g % bufs), (g // bufs - 1) & 1
            yield "then", ("copied", h, g)
            yield "arrive", ("full", h, g % bufs)

    def s():
        for g in range(tiles):
            before = g - 2
            yield "wait", ("full", 0, g % bufs), (g // bufs) & 1
            yield "wait", ("p", before % p_bars), (before // p_bars) & 1
            yield "wait", ("full", 1, g % bufs), (g // bufs) & 1
            yield "then", ("S", g)
            yield "arrive", ("s", g & 1)

    def o():
        for g in range(tiles):
            yield "wait", ("p", g % p_bars), (g // p_bars) & 1
            yield "then", ("O", g)
            yield "arrive", ("empty", 0, g % bufs)
            yield "arrive", ("empty", 1, g % bufs)

    def softmax(half, warp):
        trades = 0

        def meet():
            nonlocal trades
            trades += 1
            return [("arrive", ("trade", half)), ("wait", ("trade", half), (trades - 1) & 1)]

        for g in range(tiles):
            yield "wait", ("s", g & 1), (g >> 1) & 1
            yield from meet()
            if g in moves and g not in first:
                yield from meet()
                yield "wait", ("empty", 1, (g - 1) % bufs), ((g - 1) // bufs) & 1
            yield "then", ("P", g, half, warp)
            yield "arrive", ("p", g % p_bars)
            if g + 1 in first:
                for _ in range(3):
                    yield from meet()
                yield "wait", ("empty", 1, g % bufs), (g // bufs) & 1
                yield from meet()

    out = {"copy0": copy(0), "copy1": copy(1), "S": s(), "O": o()}
    out.update({f"softmax{h}{w}": softmax(h, w) for h in range(2) for w in range(4)})
    return out


def run(units, bufs, p_bars, moves, held, seed):
    """Whether every role ends; `held` steps only when no other role can."""
    bars = Barriers({**{(n, h, b): 1 for n in ("full", "empty") for h in range(2) for b in range(bufs)},
                     **{("s", i): 1 for i in range(2)}, **{("p", i): 8 for i in range(p_bars)},
                     **{("trade", i): 4 for i in range(2)}})
    rng = random.Random(seed)
    todo = {n: (it, next(it)) for n, it in roles(units, bufs, p_bars, moves).items()}
    seen = set()

    def step(n):
        it, (kind, *a) = todo[n]
        if kind == "wait" and not bars.complete(*a):
            return False
        if kind == "arrive":
            bars.arrive(*a)
        if kind == "then":
            what = a[0]
            # what each product and copy needs to be in place
            if what[0] == "S":
                assert all(("copied", h, what[1]) in seen for h in range(2))
                assert what[1] < 2 or all(("P", what[1] - 2, h, w) in seen for h in range(2) for w in range(4))
            if what[0] == "O":
                assert all(("P", what[1], h, w) in seen for h in range(2) for w in range(4))
            if what[0] == "P":
                assert ("S", what[1]) in seen
            if what[0] == "copied":
                assert what[2] < bufs or ("O", what[2] - bufs) in seen
            seen.add(what)
        nxt = next(it, None)
        if nxt is None:
            del todo[n]
        else:
            todo[n] = (it, nxt)
        return True

    while todo:
        names = [n for n in todo if n not in held]
        rng.shuffle(names)
        if not any(step(n) for n in names) and not any(step(n) for n in held if n in todo):
            return False
    return True


@pytest.mark.parametrize("latent,bufs", [(256, 4), (512, 2)])
def test_no_barrier_laps_a_role(latent, bufs):
    p_bars = from_source("kPBars", bufs)
    every = ["copy0", "copy1", "S", "O"] + [f"softmax{h}{w}" for h in range(2) for w in range(4)]
    for units in ([24], [1, 1, 1, 1, 9, 2], [5, 7, 3]):
        for moves in (set(), set(range(24)), {3, 4, 9}):
            for held in [[n] for n in every] + [[], ["softmax00", "softmax12"], ["S", "O"]]:
                for seed in range(3):
                    assert run(units, bufs, p_bars, moves, held, seed), (units, moves, held)
