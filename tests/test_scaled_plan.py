"""How mla_cache_append_scaled hands out its units (a unit: one block of one sequence that new rows fall
into), restated on the host: every such block is found by one unit and by no other, and no unit reads
outside cu_rows, x or the page table."""
import random

import pytest

BLOCKS = [1, 2, 4, 8, 16, 32, 64]


def first_unit(row, b, G):
    return row if G == 1 else row // G + 2 * b


def find(cu, B, unit, G):
    """The last sequence whose units begin at or before `unit`, as a warp of 32 lanes looks for it."""
    lo, n = 0, B
    while True:
        step = (n + 31) // 32
        hits = 0
        for lane in range(32):
            b = lo + lane * step
            if b < lo + n:
                assert 0 <= b < B
                hits += first_unit(cu[b], b, G) <= unit
        if hits == 0:
            return None
        lo += (hits - 1) * step
        n = min(step, n - (hits - 1) * step)
        if step == 1:
            return lo


def blocks_of_unit(cu, lens, n, unit, G):
    B = len(lens)
    b = find(cu, B, unit, G)
    if b is None:
        return None
    m, L = cu[b + 1] - cu[b], lens[b]
    if m <= 0 or L - m < 0 or cu[b] < 0 or cu[b + 1] > n:
        return None
    nth = unit - first_unit(cu[b], b, G)
    begin = ((L - m) // G + nth) * G
    if nth < 0 or begin >= L:
        return None
    assert begin >= 0
    first, end = max(L - m - begin, 0), min(L - begin, G)
    for place in range(first, end):
        assert cu[b] <= cu[b] + begin + place - (L - m) < cu[b + 1] <= n
    return b, begin // G


@pytest.mark.parametrize("G", BLOCKS)
@pytest.mark.parametrize("seed", range(12))
def test_every_block_once(G, seed):
    r = random.Random(1000 * G + seed)
    B = r.choice([1, 2, 31, 32, 33, 100, 1025])
    most = r.choice([1, 2, 5, 70, 300 if B < 200 else 9])
    new = [r.randint(0, most) for _ in range(B)]
    lens = [m + r.choice([0, 0, 1, G - 1, G, r.randint(0, 500)]) for m in new]
    lead, tail = r.choice([0, 0, 3]), r.choice([0, 0, 5])
    cu = [lead]
    for m in new:
        cu.append(cu[-1] + m)
    n = cu[-1] + tail
    got = [u for u in (blocks_of_unit(cu, lens, n, unit, G) for unit in range(first_unit(n, B, G))) if u]
    want = [(b, k) for b, (m, L) in enumerate(zip(new, lens)) if m for k in range((L - m) // G, (L - 1) // G + 1)]
    assert sorted(got) == want


def test_rows_outside_x_and_lengths_too_short():
    assert blocks_of_unit([0, 4, 8], [10, 10], 6, 4, 1) is None  # sequence 1 reaches past x
    assert blocks_of_unit([0, 4], [3], 4, 0, 16) is None         # more rows than positions


@pytest.mark.parametrize("G", BLOCKS)
def test_decreasing_rows_stay_inside(G):
    """cu_rows that decreases leads the search to a sequence whose units begin later: such a unit does nothing."""
    r = random.Random(G)
    astray = 0
    for _ in range(300):
        B, n = r.choice([2, 3, 5, 33, 70]), 60
        cu, lens = [r.randint(-3, n) for _ in range(B + 1)], [r.randint(0, 100) for _ in range(B)]
        for unit in range(first_unit(n, B, G)):
            blocks_of_unit(cu, lens, n, unit, G)  # (its assertions)
            b = find(cu, B, unit, G)
            astray += b is not None and first_unit(cu[b], b, G) > unit and cu[b + 1] > cu[b]
    assert astray or G > 8
    assert blocks_of_unit([7, 9, 0, 20], [2, 2, 30], 20, 3, 1) is None
