"""Which states reorder_beams takes together, on a host without a GPU: overlaps by byte sets against what the
C ABI says. Every call has one more state that is too large, so that none of them launches anything."""
import random

import pytest

import fp32_gemm_f32_amd as g

LD, ALIAS, LARGE = -2, -4, -7
BASE, ROWS = 1 << 20, 4
TOO_LARGE = (1 << 50, 1 << 52, 1 << 41, 1 << 41, 1 << 20, 1 << 20, 1 << 20, 1 << 12, 16, 16, 16)


def status(states):
    try:
        g.reorder_beams_raw(2, 2, 1 << 40, 8, [tuple(s) for s in states] + [TOO_LARGE])
    except g.SgemmError as e:
        return e.status
    raise AssertionError("launched")


def state(src, dst, rows, d1, d2, run):
    """(src, dst, ...) of equal strides on both sides; d1 and d2 are (count, step)."""
    return BASE + src, BASE + dst, rows, rows, d1[0], d1[1], d1[1], d2[0], d2[1], d2[1], run


def bytes_of(at, row, n1, s1, n2, s2, run):
    """(bytes, whether some are taken twice)"""
    all_of = [at + r * row + i * s1 + j * s2 + k for r in range(ROWS) for i in range(n1) for j in range(n2)
              for k in range(run)]
    return set(all_of), len(set(all_of)) < len(all_of)


def overlap(states):
    """Whether what is written meets anything else."""
    regions = []
    for src, dst, src_row, dst_row, n1, ss1, ds1, n2, ss2, ds2, run in states:
        regions.append((bytes_of(dst, dst_row, n1, ds1, n2, ds2, run)[0], True))
        if src != dst:
            regions.append((bytes_of(src, src_row, n1, ss1, n2, ss2, run)[0], False))
    return any(a & b and (wa or wb) for i, (a, wa) in enumerate(regions) for b, wb in regions[:i])


def test_slices_of_common_strides_are_taken():
    rows, length, heads, dim, e = 1 << 16, 7, 3, 20, 2
    part = heads * dim * e
    # (rows, length, 2, heads, dim) in place: keys and values side by side in each position
    kv = [state(at, at, rows, (1, 0), (length, 2 * part), part) for at in (0, part)]
    assert status(kv) == LARGE and status(kv[::-1]) == LARGE
    # (rows, 2, length, heads, dim), (rows, length, heads, 2, dim), and three of (rows, length, 3, heads, dim)
    assert status([state(at, at, rows, (1, 0), (1, 0), length * part) for at in (0, length * part)]) == LARGE
    assert status([state(at, at, rows, (length, 2 * part), (heads, 2 * dim * e), dim * e) for at in (0, dim * e)]) == LARGE
    assert status([state(at, at, rows, (1, 0), (length, 3 * part), part) for at in (0, part, 2 * part)]) == LARGE
    # (length, rows, 2, heads, dim): positions outermost
    assert status([state(at, at, 2 * part, (1, 0), (length, ROWS * 2 * part), part) for at in (0, part)]) == LARGE
    # one byte too long, one too early
    assert status([state(0, 0, rows, (1, 0), (length, 2 * part), part + 1), kv[1]]) == ALIAS
    assert status([kv[0], state(part - 1, part - 1, rows, (1, 0), (length, 2 * part), part)]) == ALIAS
    # a part that reaches into the next position
    assert status([kv[0], state(part, part, rows, (1, 0), (length, 2 * part), part + 1)]) == ALIAS
    # other strides
    assert status([kv[0], state(part, part, rows, (1, 0), (length, 4 * part), part)]) == ALIAS
    # from one's places to the other's: read where the other writes
    assert status([state(0, part, rows, (1, 0), (length, 2 * part), part), kv[1]]) == ALIAS
    # pieces between each other's without being in place: refused, whether they meet or not
    assert status([state(0, part, rows, (1, 0), (length, 2 * part), part)]) == ALIAS
    # slices of common rows, in place or not
    half = length * part
    assert status([state(0, half, rows, (1, 0), (1, 0), half)]) == LARGE


@pytest.mark.parametrize("seed", range(6))
def test_no_overlap_is_taken(seed):
    """Small random states, most of them of one grid of strides: what is accepted shares no byte; a dst whose
    own pieces meet is refused."""
    rng = random.Random(seed)
    taken = refused = 0
    for _ in range(3000):
        outer, inner, run = rng.choice([24, 32, 40, 48]), rng.choice([4, 6, 8, 12]), rng.randint(1, 6)
        states = []
        for _ in range(rng.randint(1, 3)):
            n1, n2 = rng.randint(1, 3), rng.randint(1, 4)
            steps = [rng.choice([outer * 4, outer * 3, outer]), rng.choice([outer, inner, inner * 2]), rng.choice([inner, run, 2])]
            if rng.random() < 0.5:
                steps = [outer * 4, outer, inner]
            if rng.random() < 0.3:
                rng.shuffle(steps)
            if rng.random() < 0.7:
                src = dst = BASE + rng.randint(0, 60)
            else:
                src, dst = BASE + rng.randint(0, 900), BASE + rng.randint(0, 900)
            if src != dst and rng.random() < 0.3:
                own = [rng.choice([0, steps[0]]), steps[1], rng.choice([0, 1, steps[2]])]
            else:
                own = steps
            states.append((src, dst, own[0], steps[0], n1, own[1], steps[1], n2, own[2], steps[2], rng.randint(1, run)))
        got = status(states)
        assert got in (LD, ALIAS, LARGE)
        twice = any(bytes_of(s[1], s[3], s[4], s[6], s[7], s[9], s[10])[1] for s in states)
        if got == LARGE:
            assert not twice and not overlap(states), states
            taken += 1
        else:
            refused += 1
        if twice:
            assert got == LD, states
    assert taken > 300 and refused > 300
