"""The work split of a tree's verify, restated on the host (no GPU): nodes in groups, groups over
teams of CTAs in passes, the cost axis cut into one range a team (tree_plan and the plan's tree
branches in mla_attention_tc.cu and mla_merge.cu). Checked: every node of every sequence in exactly
one group, every group over every key exactly once, partial slots that belong to one piece, and
the merge reading exactly the pieces' slots."""
import random

import pytest

from tests.test_plan import KEY_BLOCK, blocks_of, check_decode, decode_units, merge_pieces


def tree_plan(n, H, sms, B, blocks):
    most = 48 // H
    for rows in (32, 16):
        if rows >= H and B * blocks * -(-n // (rows // H)) <= sms:
            most = rows // H
    groups = -(-n // most)
    nodes = -(-n // groups)
    groups = -(-n // nodes)
    team = groups if groups <= sms else 1
    for t in range(4, groups):
        if groups % t == 0 and sms // t * t > sms // team * team:
            team = t
    return nodes, team, groups // team


@pytest.mark.parametrize("seed", range(4))
def test_groups_teams_and_slots(seed):
    rng = random.Random(seed)
    for _ in range(150):
        n, H = rng.randint(1, 64), rng.randint(1, 16)
        B = rng.choice([1, 2, 3, 8, 40])
        lens = [rng.choice([0, n, rng.randint(0, 300), rng.randint(0, 20000)]) for _ in range(B)]
        sms = rng.choice([76, 148, 152])
        width = rng.choice([max(lens) // KEY_BLOCK + 1, 2000])
        nodes, team, passes = tree_plan(n, H, sms, B, width)
        groups = team * passes
        assert nodes * H <= 48 and (groups - 1) * nodes < n <= groups * nodes
        teams = sms // team
        assert teams >= 1
        # the plan's sequences: pass p of sequence b; every member of a team walks the same units
        virtual = [L for L in lens for _ in range(passes)]
        check_decode(virtual, teams)
        units, spans, total = decode_units(virtual, teams)
        slots = {}
        for c, mine in enumerate(units):
            for m in range(team):
                for v, lo, hi, final, slot in mine:
                    group = (v // passes, v % passes * team + m)
                    at = 2 * (c * team + m) + slot - 2 * c
                    if not final:
                        assert at < 2 * teams * team and at not in slots
                        slots[at] = (group, lo, hi)
        for v, first, nb in spans:
            for m in range(team):
                pieces = merge_pieces(first, nb, total, teams)
                if len(pieces) == 1:
                    continue
                group = (v // passes, v % passes * team + m)
                mine = [slots[2 * (s // 2 * team + m) + s % 2] for s in pieces]
                assert all(g == group for g, _, _ in mine)
                assert mine[0][1] == 0 and mine[-1][2] == virtual[v] and blocks_of(virtual[v]) == nb
                assert all(a[2] == b[1] for a, b in zip(mine, mine[1:]))


def tree_ranges(total, teams):
    return (2 * teams + 2) // 3 if total < 5 * teams else teams


@pytest.mark.parametrize("seed", range(4))
def test_fewer_ranges_than_teams(seed):
    """Little work in all: the axis cut into a range for two teams in three. The ranges, units and
    merged pieces of that many; the teams from there on hold nothing."""
    rng = random.Random(100 + seed)
    few = 0
    for _ in range(150):
        B = rng.choice([1, 2, 3, 8, 40])
        lens = [rng.choice([0, rng.randint(1, 300), rng.randint(1, 6000)]) for _ in range(B)]
        teams = rng.choice([1, 2, 3, 4, 11, 19, 38, 50, 76, 152])
        total = sum(blocks_of(L) + 5 for L in lens if L)
        n = tree_ranges(total, teams)
        assert 1 <= n <= teams and (n == teams or total < 5 * teams)
        few += n < teams
        check_decode(lens, n)
        inv = (2 ** 64 - 1) // n + 1 if n > 1 else 0
        for c in range(teams):
            lo, hi = c * total * inv >> 64, ((c + 1) * total * inv >> 64) if inv else total
            if c < n:
                assert (lo, hi) == (c * total // n, (c + 1) * total // n)
            else:
                assert c * total < 2 ** 64  # (and the kernel replaces the range by an empty one)
    assert 30 < few < 120


def test_quotients_by_the_reciprocal():
    """floor(c * total / teams) as the high half of a 64-bit product with ceil(2^64 / teams)."""
    rng = random.Random(1)
    for _ in range(20000):
        teams = rng.randint(2, 304)
        inv = (2 ** 64 - 1) // teams + 1
        total = rng.choice([rng.randint(0, 5000), rng.randint(0, 2 ** 40), 2 ** 40])
        c = rng.randint(0, teams)
        assert c * total * inv >> 64 == c * total // teams


@pytest.mark.parametrize("n,H,want", [(8, 12, (4, 2, 1)), (16, 12, (4, 4, 1)), (32, 12, (4, 8, 1)), (64, 12, (4, 4, 4)),
                                      (64, 16, (3, 11, 2)), (64, 1, (32, 2, 1)), (1, 16, (1, 1, 1))])
def test_wide_tables(n, H, want):
    assert tree_plan(n, H, 152, 4, 2000) == want


def test_narrow_tables_take_smaller_groups():
    assert tree_plan(8, 12, 152, 1, 8) == (1, 8, 1)     # one node of 12 rows a group: 64 blocks in all
    assert tree_plan(8, 12, 152, 1, 30) == (2, 4, 1)    # groups of 16 rows would make 240
    assert tree_plan(8, 12, 152, 1, 80) == (4, 2, 1)
