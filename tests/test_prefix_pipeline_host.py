"""The barriers between the warps of the shared-prefix kernel, on the CPU: every order in which
the loaders, the copies, the converters (pools of codes), the tensor core and the softmax may
come is tried, and none may leave them waiting for one another."""
import os
import re

import pytest

from paged_kv_attention_06_gb300 import build

SOURCE = os.path.join(build.CSRC, "pa_prefix.cu")


def first_wait_of_values():
    """The barrier that the values' loader waits for before its first tile."""
    with open(SOURCE) as f:
        return re.search(r"if \(is_v && g == 0\)\s*mbar_wait_warp\(&bar\[(\w+)\], 0,", f.read()).group(1)


def programs(tiles, pair, gate):
    """Each warp's steps over bf16 pools, one piece of `tiles` tiles: (wait, barrier,
    parity), (arrive, barrier), (load, barrier). A barrier's phase completes with one
    arrival."""
    keys, values = [], []
    first = [("wait", ("kKFull", 0), 0), ("arrive", ("kFirstKeys", 0))]
    for g in range(tiles):
        st, turn = g & 1, (g >> 1) & 1
        if g == 2:
            keys += first
        keys += [("wait", ("kKEmpty", st), turn ^ 1), ("load", ("kKFull", st))]
        if g == 0:
            values += [("wait", (gate, 0), 0)]
        values += [("wait", ("kVEmpty", st), turn ^ 1), ("load", ("kVFull", st))]
    if tiles <= 2:
        keys += first
    for g in range(max(0, tiles - 2), tiles):
        keys += [("wait", ("kKFull", g & 1), (g >> 1) & 1)]
        values += [("wait", ("kVFull", g & 1), (g >> 1) & 1)]
    return [keys, values, *products_and_softmax(tiles, pair, 2)]


def programs_of_codes(tiles, pair, ring=3):
    """The same over pools of codes: one loader of codes into a ring, one converter, one stage
    of values."""
    order = [("K", 0)]
    for g in range(tiles):
        order += ([("K", g + 1)] if g + 1 < tiles else []) + [("V", g)]
    codes, converter = [], []
    for u, (what, g) in enumerate(order):
        slot, turn = u % ring, u // ring & 1
        st, use = (g & 1, g >> 1) if what == "K" else (0, g)
        codes += [("wait", ("kCodeEmpty", slot), turn ^ 1), ("load", ("kCodeFull", slot))]
        converter += [("wait", ("kCodeFull", slot), turn), ("wait", (f"k{what}Empty", st), use & 1 ^ 1),
                      ("arrive", (f"k{what}Full", st)), ("arrive", ("kCodeEmpty", slot))]
    u = len(order)                                           # the end
    codes += [("wait", ("kCodeEmpty", u % ring), u // ring & 1 ^ 1), ("arrive", ("kCodeFull", u % ring))]
    codes += [("wait", ("kCodeEmpty", x % ring), x // ring & 1 ^ 1) for x in range(u + 1, u + ring)]
    converter += [("wait", ("kCodeFull", u % ring), u // ring & 1)]
    return [codes, converter, *products_and_softmax(tiles, pair, 1)]


def products_and_softmax(tiles, pair, value_stages):
    steps = [(g, sub) for g in range(tiles) for sub in range(2 if pair else 1)]
    closes = [not pair or sub == 1 for _, sub in steps]
    products = []

    def scores(j):
        g = steps[j][0]
        out = [("wait", ("kKFull", g & 1), (g >> 1) & 1), ("arrive", ("kSFull", j & 1))]
        return out + ([("arrive", ("kKEmpty", g & 1))] if closes[j] else [])

    for j in range(min(2, len(steps))):
        products += scores(j)
    for j, (g, _) in enumerate(steps):
        phase = (j >> 1) & 1
        st, use = (0, g) if value_stages == 1 else (g & 1, g >> 1)
        products += [("wait", ("kPFull", j & 1), phase), ("wait", ("kVFull", st), use & 1),
                     ("arrive", ("kPVDone", j & 1))]
        if closes[j]:
            products += [("arrive", ("kVEmpty", st))]
        products += [("wait", ("kPVDone", j & 1), phase)]
        if j + 2 < len(steps):
            products += scores(j + 2)
    halves = [[x for j in range(h, len(steps), 2)
               for x in (("wait", ("kSFull", h), (j >> 1) & 1), ("arrive", ("kPFull", h)))] for h in range(2)]
    return [products, *halves]


def stalls(warps):
    """Whether some order of events ends with a warp that waits for ever."""
    bars = sorted({op[1] for w in warps for op in w})
    at = {b: i for i, b in enumerate(bars)}
    start = ((0,) * len(warps), (0,) * len(bars), (0,) * len(bars))   # places, phases done, copies on their way
    seen, todo = {start}, [start]
    while todo:
        places, done, flying = todo.pop()
        nexts = []
        for w, ops in enumerate(warps):
            if places[w] == len(ops):
                continue
            kind, bar, *parity = ops[places[w]]
            i = at[bar]
            if kind == "wait" and (done[i] & 1) == parity[0]:        # that phase has not completed
                continue
            moved = places[:w] + (places[w] + 1,) + places[w + 1:]
            if kind == "arrive":
                nexts.append((moved, done[:i] + (done[i] + 1,) + done[i + 1:], flying))
            elif kind == "load":
                nexts.append((moved, done, flying[:i] + (flying[i] + 1,) + flying[i + 1:]))
            else:
                nexts.append((moved, done, flying))
        for i, n in enumerate(flying):
            if n:
                nexts.append((places, done[:i] + (done[i] + 1,) + done[i + 1:], flying[:i] + (n - 1,) + flying[i + 1:]))
        if not nexts and any(p < len(ops) for p, ops in zip(places, warps)):
            return True
        for x in nexts:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return False


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6])
def test_no_order_of_events_stalls(tiles, pair):
    assert not stalls(programs(tiles, pair, first_wait_of_values()))


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6])
def test_no_order_of_events_stalls_over_codes(tiles, pair):
    assert not stalls(programs_of_codes(tiles, pair))


def test_a_wait_by_parity_from_outside_a_ring_is_found():
    """The values' loader on the keys' own stage: two tiles later the parity is the same."""
    assert not stalls(programs(2, False, "kKFull"))
    assert stalls(programs(3, False, "kKFull")) and stalls(programs(4, True, "kKFull"))
