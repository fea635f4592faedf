"""The oracles of rotary positions and of a cache's pages, and the rotation's plan, on the CPU."""
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import paged, pages, rope


def _plan(*args, **kw):
    turns, axis = fa.rope_table(*args, device="cpu", **kw)
    return [int(t) % 2 ** 64 for t in turns], axis.tolist()


def test_plan_is_the_frequencies_in_turns():
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    turns, axis = _plan(64, 10000.0)
    assert axis == [0] * 32
    for i, t in enumerate(turns):
        w = Decimal(10000) ** (Decimal(-2 * i) / 64)
        exact = w / (2 * pi) * 2 ** 64
        # a power, a quotient by 2 pi (itself rounded) and the floor: four roundings of 2^-53
        assert abs(Decimal(t) - exact) <= exact * 4 / 2 ** 53 + 1


def test_plan_of_sections_and_of_given_frequencies():
    _, axis = _plan(128, sections=[16, 24, 24])
    assert axis == [0] * 16 + [1] * 24 + [2] * 24
    turns, _ = _plan(16, frequencies=[0.0, 2 * np.pi, np.pi, -np.pi / 2, 7 * np.pi, 1e-9, 3.0, 1.0])
    assert turns[0] == 0 and turns[1] == 0 and turns[2] == 2 ** 63 and turns[3] == 3 * 2 ** 62
    assert turns[4] == 2 ** 63


def test_plan_keeps_every_bit_of_its_frequencies_of_either_sign():
    # the turns of the fp64 quotient by 2 pi, off by half a unit at most; the other way round the same
    f = [0.3, 1.0, 1e-6, 1e-9, 7.1, 6.2, 2.0 ** -58, 1000.25]
    turns, _ = _plan(16, frequencies=f)
    back, _ = _plan(16, frequencies=[-x for x in f])
    for x, t, b in zip(f, turns, back):
        exact = Fraction(x / (2 * np.pi)) * 2 ** 64
        assert abs((t - exact + 2 ** 63) % 2 ** 64 - 2 ** 63) <= Fraction(1, 2), x
        assert (t + b) % 2 ** 64 == 0, x


@pytest.mark.parametrize("kw", [dict(sections=[3, 4]), dict(frequencies=[1.0]), dict(sections=[-1, 9]),
                                dict(frequencies=[float("inf")] * 8)])
def test_plan_refuses(kw):
    with pytest.raises(ValueError):
        fa.rope_table(16, device="cpu", **kw)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_against_a_written_out_matrix(interleaved):
    rng = np.random.default_rng(0)
    turns, axis = _plan(16, sections=[3, 5])
    x, pos = rng.standard_normal((4, 20)), rng.integers(-50, 50, (2, 4))
    y, size = rope.rotate(x, pos, turns, axis, interleaved)
    for n in range(4):
        R = np.eye(20)
        for i in range(8):
            a = pos[axis[i], n] * 10000.0 ** (-i / 8)
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
            R[p, p], R[p, q], R[q, p], R[q, q] = np.cos(a), -np.sin(a), np.sin(a), np.cos(a)
        assert np.allclose(y[n], R @ x[n], atol=1e-12)
    assert np.all(size[:, 16:] == 0) and np.all(size[:, :16] > 0)


def test_rotation_keeps_what_scores_depend_on_and_turns_back():
    rng = np.random.default_rng(1)
    turns, axis = _plan(32)
    q, k = rng.standard_normal((2, 1, 32))

    def score(n, m):
        a, b = (rope.rotate(t, np.array([[p]]), turns, axis)[0][0] for t, p in ((q, n), (k, m)))
        return a @ b

    assert abs(score(7, 3) - score(1000004, 1000000)) < 1e-12
    pos = np.array([[123456789]])
    y, _ = rope.rotate(q, pos, turns, axis)
    assert np.allclose(rope.rotate(y, pos, turns, axis, inverse=True)[0], q, atol=1e-14)


def test_rotation_gradient_against_differences():
    rng = np.random.default_rng(2)
    turns, axis = _plan(16, sections=[4, 4])
    x, dy, pos = rng.standard_normal((3, 24)), rng.standard_normal((3, 24)), rng.integers(0, 99, (2, 3))
    dx, _ = rope.rotate(dy, pos, turns, axis, inverse=True)
    for _ in range(5):
        e = rng.standard_normal(x.shape)
        d = [np.sum(dy * rope.rotate(x + s * e, pos, turns, axis)[0]) for s in (0.5, -0.5)]
        assert abs((d[0] - d[1]) - np.sum(dx * e)) < 1e-12      # linear: the difference is exact


def _cache(seed, B=6, M=9, page=16, P=60):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, M * page + 1, B)
    table = np.full((B, M), -1)
    ids = rng.permutation(P)
    at = 0
    for b in range(B):
        n = -(-lens[b] // page)
        table[b, :n] = ids[at:at + n]
        at += n
    return rng, lens, table, ids[at:], rng.standard_normal((P, 2, page, 8))


def _tokens(pool, table, lens, b):
    p, r = paged.visible(table[b], lens[b], pool.shape[-2], pool.shape[0], 10 ** 9)
    return pool[p, :, r]


@pytest.mark.parametrize("seed", range(4))
def test_a_fork_reads_as_its_source_and_takes_its_own_rows(seed):
    rng, lens, table, free, pool = _cache(seed)
    lens[4] = lens[5] = 0
    lens[0] = 37
    before = _tokens(pool, table, lens, 0)
    l2, t2, copies, taken = pages.fork(lens, table, free, [0, 0, 9, 0, 4], [4, 5, 1, 4, 3], 16, 60)
    pool = pages.copy(pool, *([c[i] for c in copies] for i in range(3)))
    assert taken == 2 and [c[2] for c in copies] == [5, 5, 0, 0, 0]
    for b in (4, 5):
        assert l2[b] == 37 and np.array_equal(_tokens(pool, t2, l2, b), before)
        assert t2[b, 2] != t2[0, 2] and np.array_equal(t2[b, :2], t2[0, :2])
    # each appends to its own page
    pool = paged.append(pool, rng.standard_normal((1, 2, 8)), [t2[4, 2] * 16 + 5])
    assert np.array_equal(_tokens(pool, t2, l2, 0), before)


@pytest.mark.parametrize("seed", range(4))
def test_free_then_compact_keeps_every_request_and_fills_the_front(seed):
    rng, lens, table, _, pool = _cache(seed)
    table[1, :2] = table[0, :2]
    held = [_tokens(pool, table, lens, b) for b in range(6)]
    lens, table, refs, free = pages.free(lens, table, [2, 2, 77], 16, 60)
    t2, moved, copies, U = pages.compact(lens, table, 16, 60)
    pool = pages.copy(pool, *zip(*copies)) if copies else pool
    for b in range(6):
        if b == 2:
            assert lens[b] == 0 and np.all(table[b] == -1)
        else:
            assert np.array_equal(_tokens(pool, t2, lens, b), held[b])
    named = {p for _, _, p in pages.live(t2, lens, 16, 60)}
    assert named == set(range(U)) and U == 60 - len(free)
    assert refs.sum() == sum(-(-n // 16) for n in lens)
    assert not {a for a, _ in copies} & {b for _, b in copies}
    assert sorted(moved[moved >= 0]) == list(range(U))


def test_decode_over_forked_tables_is_that_of_the_copies():
    rng, lens, table, free, pool = _cache(9)
    lens[0], lens[4], lens[5] = 70, 0, 0
    lens, table, copies, _ = pages.fork(lens, table, free, [0, 0], [4, 5], 16, 60)
    pool = pages.copy(pool, *([c[i] for c in copies] for i in range(3)))
    q = np.repeat(rng.standard_normal((1, 4, 8)), 3, 0)
    o, lse, _ = paged.decode(q, pool, pool, table[[0, 4, 5]], lens[[0, 4, 5]], 0.3)
    assert np.allclose(o[0], o[1]) and np.allclose(o[0], o[2]) and np.allclose(lse[0], lse[1])
