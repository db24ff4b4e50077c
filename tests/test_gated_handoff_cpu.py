"""The hand-off of chunk states in the one-launch prefill, walked exhaustively in a small model of its steps.

A state warp, for every chunk g: issue the store of its part of the state, wait until its store of chunk g - 1 has
landed and count that, wait for the product of chunk g (which starts when every warp has read accumulator g - NU), read
it, and let the next product start.  Behind the last chunk it waits for all its stores and counts them.  Stores land in
any order that the waits allow.  The publisher releases chunk 0, 1, .. as the counts permit."""
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
