"""The hand-off of chunk states in the one-launch prefill, walked exhaustively in a small model of its steps.

A state warp, for every chunk g: issue the store of its part of the state, wait until its store of chunk g - 1 has
landed and count that, wait for the product of chunk g (which starts when every warp has read accumulator g - NU), read
it, and let the next product start.  Behind the last chunk it waits for all its stores and counts them.  Stores land in
any order that the waits allow.  The publisher releases chunk 0, 1, .. as the counts permit.

And the roles of the launch's CTAs, under every order in which they may start on a device with room for some of them."""
import itertools

import pytest

CHUNKS, WARPS = 4, 2
STORE, COUNT, READ, FREE, DONE = range(5)


def _after(st, nu, ready):
    """Every state that one step leads to.  st: per warp (chunk, step, landed bits, counted), and the chunks published."""
    warps, published = st
    for w, (g, step, landed, counted) in enumerate(warps):
        def to(*x):
            return warps[:w] + (x,) + warps[w + 1:], published

        issued = g + 1 if step in (COUNT, READ, FREE) else g
        for c in range(issued):
            if not landed >> c & 1:
                yield to(g, step, landed | 1 << c, counted)
        if step == STORE:
            if g == CHUNKS:
                if landed == (1 << CHUNKS) - 1:
                    yield to(g, DONE, landed, g)
            else:
                yield to(g, COUNT, landed, counted)
        elif step == COUNT:
            if landed & (1 << g) - 1 == (1 << g) - 1:
                yield to(g, READ, landed, g)
        elif step == READ:
            # the product of chunk g needs its accumulator, which every warp has read for chunk g - nu
            if all(x[0] > g - nu for x in warps):
                yield to(g, FREE, landed, counted)
        elif step == FREE:
            yield to(g + 1, STORE, landed, counted)
    if published < CHUNKS and ready([x[3] for x in warps], published):
        yield warps, published + 1


def _walk(nu, ready):
    """(a chunk was published before all of it had landed, some order ends before everything is published)"""
    first = (((0, STORE, 0, 0),) * WARPS, 0)
    seen, todo = {first}, [first]
    early = stuck = False
    while todo:
        st = todo.pop()
        warps, published = st
        if any(not x[2] >> c & 1 for c in range(published) for x in warps):
            early = True
        nxt = list(_after(st, nu, ready))
        if not nxt and published < CHUNKS:
            stuck = True
        for x in nxt:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return early, stuck


@pytest.mark.parametrize("nu", [1, 2])
def test_least_count_publishes_only_what_is_stored(nu):
    assert _walk(nu, lambda counts, p: min(counts) >= p + 1) == (False, False)


@pytest.mark.parametrize("nu", [1, 2])
def test_sum_of_counts_would_publish_early(nu):
    """Why each warp has a count of its own."""
    early, _ = _walk(nu, lambda counts, p: sum(counts) >= (p + 1) * WARPS)
    assert early


def _all_published(items, at_end, ring=4):
    """Whether one CTA's walk ends: items (their chunks) pass from the producer to a state warp and to the publisher through
    a ring of entries that both have to read.  A chunk is counted when the next one is stored, the last of an item at its
    end (`at_end`) or, otherwise, behind all items.  No step here disables another, so one order shows all."""
    made, counted, read = [0], [0], [0, 0]

    def producer():
        for k in range(len(items) + 1):                       # the last entry says that there are no more
            while k >= ring and min(read) <= k - ring:
                yield
            made[0] = k + 1

    def state_warp():
        g = 0
        for k in range(len(items) + 1):
            while made[0] <= k:
                yield
            read[0] = k + 1
            for _ in range(items[k] if k < len(items) else 0):
                counted[0] = g                                # those before this one
                g += 1
                yield
            if at_end:
                counted[0] = g
        counted[0] = g

    def publisher():
        g = 0
        for k in range(len(items) + 1):
            while made[0] <= k:
                yield
            read[1] = k + 1
            for _ in range(items[k] if k < len(items) else 0):
                g += 1
                while counted[0] < g:
                    yield

    roles = [producer(), state_warp(), publisher()]
    for _ in range(50 * (len(items) + sum(items) + 1)):
        roles = [r for r in roles if next(r, "done") != "done"]
        if not roles:
            return True
    return False


@pytest.mark.parametrize("empty", range(12))
def test_a_walk_over_empty_items_ends(empty):
    for items in ([2] + [0] * empty, [0] * empty + [1], [1] + [0] * empty + [3], [3, 1] + [0] * empty):
        assert _all_published(items, at_end=True), items
    if empty >= 4:      # where the last chunk waits for the next one's store
        assert not _all_published([2] + [0] * empty, at_end=False)


def _finishes(order, room, makers, units, look):
    """Whether the launch ends: CTAs start in this order while there is room.  A maker claims and walks every unit left and
    waits for nobody; a consumer takes the chunks (one a unit) in turn and waits for each.  With `look` a CTA makes states
    too if no unit has been claimed when it starts."""
    todo, waiting = list(order), []          # waiting: the chunks that the resident CTAs wait for
    walked = taken = 0
    while True:
        waiting = [c for c in waiting if c >= walked]
        while taken < walked:                # whoever is not waiting takes what is there
            taken += 1
        if taken >= units and not waiting:
            return True
        if not todo or len(waiting) >= room:
            return False
        cta = todo.pop(0)
        if cta < makers or (look and walked == 0):
            walked = units
        else:
            waiting.append(taken)
            taken += 1


@pytest.mark.parametrize("room", [1, 2, 3])
@pytest.mark.parametrize("makers", [1, 2])
def test_every_start_order_finishes(room, makers):
    orders = list(itertools.permutations(range(5)))
    assert all(_finishes(o, room, makers, 6, look=True) for o in orders)
    # by index alone, a device full of consumers would wait until they give up
    assert not all(_finishes(o, room, makers, 6, look=False) for o in orders)
