"""CPU models of the paged cache's index arithmetic: the runs that the attention
of few rows cuts its work into and the pieces it joins, and the page lists."""
import random

import pytest


def runs_model(real, grid, head):
    """real: units of keys per item; head: units that stand for an item's own cost.  Returns
    per item the unit ranges written in full, and the slots joined, as paged_attn.cu lays
    them out."""
    units = [head + x for x in real]
    W = sum(units)
    starts = [sum(units[:i]) for i in range(len(units))]
    runs = min(W, grid)
    pieces, entries, whole = {}, {}, {}
    for c in range(runs):
        u, end = c * W // runs, (c + 1) * W // runs
        assert u < end
        while u < end:
            i = max(k for k in range(len(units)) if starts[k] <= u)
            to = min(units[i], end - starts[i])
            off = max(0, u - starts[i] - head)
            cnt = max(0, to - head) - off
            u = starts[i] + to
            if cnt == 0:
                assert u == end  # a part without keys is a run's last, or all of it
                continue
            begins, ends = off == 0, off + cnt == real[i]
            if begins and ends:
                whole[i] = (0, real[i])
            else:
                slot = grid + c if begins else c
                assert slot not in pieces and slot < 2 * grid
                pieces[slot] = (i, off, cnt)
                if begins:
                    last = ((starts[i] + units[i]) * runs + W - 1) // W - 1
                    assert c not in entries
                    entries[c] = (i, grid + c, c + 1, last - c)
    return whole, pieces, entries


@pytest.mark.parametrize("head", [0, 1, 2, 5])
@pytest.mark.parametrize("seed", range(40))
def test_runs_cover_every_item_once(seed, head):
    r = random.Random(seed)
    units = [r.choice([1, 1, 2, 3, r.randint(1, 60)]) for _ in range(r.randint(1, 40))]
    grid = r.choice([1, 2, 3, 7, 24, 100])
    whole, pieces, entries = runs_model(units, grid, head)
    joined = {}
    for i, head, nxt, count in entries.values():
        assert i not in joined and i not in whole and count >= 1
        got = [pieces[s] for s in [head] + list(range(nxt, nxt + count))]
        at = 0
        for j, off, cnt in got:
            assert j == i and off == at
            at += cnt
        assert at == units[i]
        joined[i] = len(got)
    assert sorted(list(whole) + list(joined)) == list(range(len(units)))
    assert sum(joined.values()) == len(pieces)


def compact_model(ref):
    """The pairs (hole, page) as compact_rank_kernel ranks them, block by block."""
    n = sum(x != 0 for x in ref)
    below = sum(x != 0 for x in ref[:n])
    holes, moves, lp = {}, {}, 0
    for q, x in enumerate(ref):
        if q < n and x == 0:
            holes[q - lp] = q
        if q >= n and x != 0:
            moves[lp - below] = q
        lp += x != 0
    return n, n - below, holes, moves


@pytest.mark.parametrize("seed", range(30))
def test_compaction_pairs_holes_with_moves(seed):
    r = random.Random(seed)
    ref = [r.choice([0, 0, 1, 2]) if r.random() < 0.9 else 0 for _ in range(r.choice([1, 2, 9, 100, 1000]))]
    n, count, holes, moves = compact_model(ref)
    assert sorted(holes) == sorted(moves) == list(range(count))
    assert [holes[i] for i in range(count)] == [q for q in range(n) if ref[q] == 0]
    assert [moves[i] for i in range(count)] == [q for q in range(n, len(ref)) if ref[q] != 0]
    assert 2 * count <= len(ref)


@pytest.mark.parametrize("num_pages", [1, 127, 128, 129, 5000, 262144])
def test_grant_steps_cover_every_page(num_pages):
    steps, warps = (num_pages + 127) // 128, 8 * 32
    seen = []
    for w in range(warps):
        seen += range(steps * w // warps, steps * (w + 1) // warps)
    assert seen == list(range(steps))
