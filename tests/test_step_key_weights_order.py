"""The gathering pass of the tensor-core key weights hands its columns' statistics from warp to warp through three
buffers of shared memory.  The order of its writes, waits and reads is taken from the source and played through for
every way in which two warps of a group and the products can overtake one another; no GPU is needed."""
from __future__ import annotations

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUFFERS = 3
# what a warp does with a tile, as the source spells it
SPELLED = {
    "show_next": r"show\(b \+ 2,",                # the next tile's statistics, to the next buffer
    "wait_shown": r"wait_warp\(&st_full\[",       # this tile's statistics of all warps
    "wait_product": r"wait_warp\(&s_full\[",      # this tile's scores
    "free_product": r"mbar_arrive\(&s_empty\[",   # the last scores are in registers
    "read": r"int low = sm_chunks\[",            # statistics, for each chunk of columns the last one too
}


def steps():
    text = open(os.path.join(ROOT, "paged_kv_gqa_02_gb300", "csrc", "pa_key_weights_tc.cu")).read()
    loop = text[text.index("for (int b = p.b0 + first; b < p.b1; b += 2, ++seen)"):]
    loop = loop[:loop.index("if (++buf == 3)")]
    at = {}
    for name, spelled in SPELLED.items():
        found = [m.start() for m in re.finditer(spelled, loop)]
        assert len(found) == 1, name
        at[name] = found[0]
    return tuple(sorted(at, key=at.get))


def play(order, parts, warps=2):
    """Plays parts (their tiles) through in every order; returns what went wrong, or None."""
    program = []  # of a warp: (step, tile)
    tile = 0
    for n in parts:
        program.append(("show", tile))
        for i in range(n):
            for step in order:
                if step != "show_next":
                    program.append((step, tile))
                elif i + 1 < n:
                    program.append(("show", tile + 1))
            tile += 1
    total, last = tile, {t: max(i for i, x in enumerate(program) if x == ("read", t)) for t in range(tile)}

    def done(at, what, where=lambda t: True):
        return [sum(1 for step, t in program[:i] if step == what and where(t)) for i in at]

    start = ((0,) * warps, 0)  # places in the program, products made
    seen, todo = {start}, [start]
    while todo:
        at, products = todo.pop()
        went = []
        # a product needs its accumulator free of the one before
        if products < total and min(done(at, "free_product")) >= products:
            went.append((at, products + 1))
        for w in range(warps):
            if at[w] == len(program):
                continue
            step, t = program[at[w]]
            if step == "wait_shown":  # a phase of the buffer's barrier has ended, by its parity
                phases = min(done(at, "show", lambda x: x % BUFFERS == t % BUFFERS))
                if phases & 1 == (t // BUFFERS) & 1:
                    continue
            elif step == "wait_product" and products & 1 == t & 1:
                continue
            elif step == "show":
                for v in range(warps):
                    if t >= BUFFERS and at[v] <= last[t - BUFFERS]:
                        return f"warp {w} writes tile {t}'s statistics over tile {t - BUFFERS}'s, which warp {v} still reads"
            elif step == "read" and min(done(at, "show", lambda x: x == t)) < 1:
                return f"warp {w} reads tile {t}'s statistics before all are written"
            went.append((at[:w] + (at[w] + 1,) + at[w + 1:], products))
        if not went and (products < total or any(i < len(program) for i in at)):
            return f"nobody goes on at {[program[i] if i < len(program) else None for i in at]}"
        for x in went:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None


@pytest.mark.parametrize("parts", [(1,), (9,), (4, 5), (1, 1, 1, 1, 1, 1), (2, 3, 1, 4), (3, 1, 1, 4), (7, 2)])
def test_no_warp_overwrites_what_another_reads(parts):
    assert play(steps(), parts) is None


def test_the_play_tells_orders_apart():
    """Statistics written before this tile's are waited for can land under a reader of two tiles ago."""
    good = ("wait_shown", "show_next", "wait_product", "free_product", "read")
    assert play(good, (9,)) is None
    assert "still reads" in play(("show_next", "wait_shown", "wait_product", "free_product", "read"), (9,))
    assert "before all are written" in play(("show_next", "wait_product", "read", "free_product", "wait_shown"), (9,))
    assert "nobody" in play(("wait_shown", "show_next", "wait_product", "read"), (9,))
