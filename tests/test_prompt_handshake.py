"""How far the softmax warps of one tile may run ahead of the other's in prompt_kernel, from its barriers: entry
unit % N of the flag "values were put to 0" must not be written for a later unit while a warp of the other tile has
still to read it.  Checked on the CPU, with a model of the kernel's waits; N comes from the source."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_continuous_pa_gb300", "csrc",
                      "pa_prompt.cu")


class Frozen(Exception):
    pass


def run_ahead(units, stages, slow_unit):
    """The last unit whose flag tile A's warps may write while one warp of tile B has yet to read that of `slow_unit`.

    units: (key blocks of tile A, of tile B) in turn.  Each party is a generator that yields a condition until it
    holds; every party runs as far as it can, so that what is reached is reached in some schedule.  Tile B has
    a leading warp, which releases the ring's slots, and the slow one, which stops in front of its read."""
    flag = set()          # events that have happened
    wrote = [-1]
    items = [0]           # tiles of K and V before a unit
    for a, b in units:
        items.append(items[-1] + 2 * max(a, b))

    def has(*event):
        return lambda: event in flag

    def loader():
        item, queries = 0, [0, 0]
        for k, (na, nb) in enumerate(units):
            if k >= 4:  # the entry that names unit k was read by every warp (UE)
                for who in ("A", "B", "slow", "mma0", "mma1"):
                    yield has("knows", who, k - 4)
            flag.add(("unit", k))
            for j in range(max(na, nb)):
                for side in ("K", "V"):
                    if item >= stages:
                        yield has("empty", 0, item - stages)
                        yield has("empty", 1, item - stages)
                    flag.add(("full", item))
                    item += 1
                    if side == "K" and j == 0:
                        for t, n in ((0, na), (1, nb)):
                            if n:
                                if queries[t]:
                                    yield has("queries done", t, queries[t])
                                queries[t] += 1
                                flag.add(("queries", t, queries[t]))

    def mma(t):
        done = 0
        for k, (na, nb) in enumerate(units):
            n = (na, nb)[t]
            yield has("unit", k)
            flag.add(("knows", f"mma{t}", k))
            first = items[k]
            yield has("full", first)
            if n:
                done += 1
                yield has("queries", t, done)
                flag.add(("scores", t, k, 0))
            else:
                flag.add(("empty", t, first))
            for j in range(max(na, nb)):
                yield has("full", first + 2 * j + 1)
                if j >= na - 1:
                    yield has("looked", k, j)
                if j >= n:
                    flag.add(("empty", t, first + 2 * j + 1))
                    if j + 1 < max(na, nb):
                        yield has("full", first + 2 * j + 2)
                        flag.add(("empty", t, first + 2 * j + 2))
                    continue
                for who in (("A",) if t == 0 else ("B", "slow")):
                    yield has("weights", who, k, j)
                if j + 1 < max(na, nb):
                    yield has("full", first + 2 * j + 2)
                    flag.add(("scores", t, k, j + 1) if j + 1 < n else ("empty", t, first + 2 * j + 2))
                if j + 1 == n:
                    flag.add(("product", t, k))
            if n:
                flag.add(("queries done", t, done))

    def softmax(t, who):
        for k, (na, nb) in enumerate(units):
            n, first = (na, nb)[t], items[k]
            yield has("unit", k)
            flag.add(("knows", who, k))
            for j in range(n):
                # each tile looks over the values of its own diagonal where the two differ, else tile A's warps do
                if j == n - 1 and (t == 0 or nb > na):
                    yield has("full", first + 2 * j + 1)
                    if t == 0:
                        wrote[0] = max(wrote[0], k)
                    if who != "slow":
                        flag.add(("looked", k, j))
                yield has("scores", t, k, j)
                flag.add(("weights", who, k, j))
                if who != "slow":
                    flag.add(("empty", t, first + 2 * j))
                    if j:
                        flag.add(("empty", t, first + 2 * j - 1))
            if n == 0:
                continue
            yield has("product", t, k)
            if who != "slow":
                flag.add(("empty", t, first + 2 * n - 1))
            elif k == slow_unit:
                raise Frozen

    parties = [loader(), mma(0), mma(1), softmax(0, "A"), softmax(1, "B"), softmax(1, "slow")]
    waits = [None] * len(parties)
    live = set(range(len(parties)))
    moved = True
    while moved:
        moved = False
        for i in list(live):
            while i in live and (waits[i] is None or waits[i]()):
                moved = True
                try:
                    waits[i] = next(parties[i])
                except (StopIteration, Frozen):
                    live.discard(i)
    return wrote[0], live


PATTERNS = [[(1, 2)] + [(1, 0)] * 12, [(1, 1)] * 12, [(1, 2)] * 12, [(3, 4)] + [(1, 0)] * 12, [(1, 2), (1, 0)] * 6,
            [(5, 5)] + [(1, 1)] * 12, [(2, 2)] * 12]


def test_the_model_runs_to_its_end():
    for units in PATTERNS:
        for stages in (5, 8):
            last, live = run_ahead(units, stages, slow_unit=len(units))
            assert last == len(units) - 1 and not live


def test_flags_outlive_the_run_ahead():
    text = open(SOURCE).read()
    (place,) = set(re.findall(r"odd_values\[k & (\d+|\(FLAGS - 1\))\]", text))  # every place takes the same entry of a unit
    entries = int(place) + 1 if place.isdigit() else int(re.search(r"FLAGS = (\d+);", text).group(1))
    assert entries & (entries - 1) == 0
    ahead = max(run_ahead(units, stages, slow)[0] - slow
                for units in PATTERNS for stages in (5, 8) for slow in range(3) if units[slow][1])
    assert ahead == 4  # every warp knows unit k - 4 before unit k is announced
    assert ahead < entries, f"unit k + {ahead} takes the entry of a unit that a warp has yet to read"
