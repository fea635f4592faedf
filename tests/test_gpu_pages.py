"""Forking, freeing, compacting and copying the pages of a paged cache, on the GPU, against the
oracle: all of it whole numbers and moved rows, so equal or wrong."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import pages

from test_gpu_paged import _gen, _i32, _np, _ok

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


def _cache(seed, B, M, page, P, shared=True):
    """Lengths and a table with holes and pages that several rows name; the pages left over."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, M * page + 1, B)
    lens[rng.random(B) < 0.2] //= page
    used = -(-lens // page)
    table = np.full((B, M), -1)
    ids = rng.permutation(P)
    at = 0
    for b in range(B):
        n = min(used[b], max(0, P - at))
        table[b, :n] = ids[at:at + n]
        at += n
    if shared:
        for _ in range(B // 2):
            a, b = rng.integers(0, B, 2)
            n = min(used[a], used[b]) // 2
            table[b, :n] = table[a, :n]
        holes = rng.random((B, M)) < 0.05
        table[holes] = rng.choice([-1, P, 2 ** 31 - 1, -2 ** 31], holes.sum())
    return rng, lens, table, ids[at:]


# ------------------------------------------------------------------ fork

def _run_fork(lens, table, free, src, dst, page, P):
    l, t = _i32(lens), _i32(table)
    frm, to, rows, taken = fa.paged_fork(l, t, _i32(free), _i32(src), _i32(dst), page, P)
    _ok()
    rl, rt, copies, rtaken = pages.fork(lens, table, free, src, dst, page, P)
    assert np.array_equal(l.cpu().numpy(), rl)
    assert np.array_equal(t.cpu().numpy(), rt)
    assert list(zip(frm.tolist(), to.tolist(), rows.tolist())) == copies
    assert taken.item() == rtaken
    return l, t, frm, to, rows


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("B,M,n", [(2, 1, 1), (9, 5, 4), (300, 3, 290), (70, 700, 60)])
def test_fork(page, B, M, n):
    P = B * M // 2 + n + 3
    rng, lens, table, free = _cache(B + page, B, M, page, P)
    src = rng.integers(0, max(1, B - n), n)
    dst = B - n + rng.permutation(n) if n < B else rng.permutation(B)
    _run_fork(lens, table, free, src, dst, page, P)
    _run_fork(lens, table, free[:n // 3], src, dst, page, P)          # a list too short
    # pairs of every kind that is skipped: padding, out of range, named before, sources as targets
    src, dst = rng.integers(-2, B + 2, n), rng.integers(-2, B + 2, n)
    _run_fork(lens, table, free, src, dst, page, P)


def test_fork_of_odd_tables():
    # lengths below 0 and past the row; a source whose last page is a hole; none; a bad free page
    table = np.array([[3, 4], [5, 99], [-1, 6], [7, 7], [7, 7], [7, 7], [7, 7]])
    _run_fork([20, 25, 9, 1000, -4, 0, 1], table, [1, 200, 0], [0, 1, 2, 0, 0], [6, 5, 4, 3, 9], 16, 8)
    _run_fork([20, 25, 9, 1000, -4, 0, 32], table, [1, 0], [3, 4, 6, 2], [0, 1, 5, 2], 16, 8)
    _run_fork([16, 0], table[:2], [1], [], [], 16, 8)
    _run_fork([17, 0], table[:2], [], [0], [1], 16, 8)


def test_fork_of_the_largest_batch():
    B = 8192
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 33, B)
    table = np.arange(2 * B).reshape(B, 2)
    rows = rng.permutation(B)
    _run_fork(lens, table, 2 * B + rng.permutation(B), np.concatenate([rows[:4096]] * 2),
              np.concatenate([rows[4096:], np.full(4096, -1)]), 16, 3 * B)


def _in_a_new_process(script):
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")])
    done = subprocess.run([sys.executable, "-c", script], env={**os.environ, "PYTHONPATH": path},
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_fork_of_any_size_in_a_new_process():
    # around 48 KB of shared memory, in ascending order: a larger call before would have raised what
    # the device grants to all that follow
    _in_a_new_process("""
import numpy as np
import test_gpu_pages as t
B = 8192
rng = np.random.default_rng(0)
for n in (4080, 4081, 4088, 4089, 4096, 4097, 8192):
    rows = rng.permutation(B)
    src, dst = np.full(n, -1), np.full(n, -1)
    m = min(n, B // 2)
    src[:m], dst[:m] = rows[:m], rows[m:2 * m]
    t._run_fork(rng.integers(0, 33, B), np.arange(2 * B).reshape(B, 2), 2 * B + rng.permutation(B),
                src, dst, 16, 3 * B)
""")


def test_tables_of_any_size_in_a_new_process():
    # as above, 8 B + 72 bytes
    _in_a_new_process("""
import numpy as np
import test_gpu_paged as t
rng = np.random.default_rng(0)
for B in (6134, 6135, 6136, 6140, 6143, 6144, 8192):
    old, new = rng.integers(0, 20, B), rng.integers(0, 3, B)
    t._run_tables(old, new, 2 * B + rng.permutation(B), np.arange(2 * B).reshape(B, 2), 16, 4 * B,
                  int(new.sum()) + 3)
""")


def test_fork_leaves_what_lies_beside_a_view():
    wide = torch.full((3, 8), 42, dtype=I32, device="cuda")
    wide[0, 1:4] = _i32([5, 6, 7])
    lens = _i32([40, 0, 0])
    fa.paged_fork(lens, wide[:, 1:6], _i32([1, 2]), _i32([0, 0]), _i32([2, 1]), 16, 8)
    _ok()
    assert wide.cpu().tolist() == [[42, 5, 6, 7, 42, 42, 42, 42], [42, 5, 6, 2, 42, 42, 42, 42],
                                   [42, 5, 6, 1, 42, 42, 42, 42]]
    assert lens.tolist() == [40, 40, 40]


# ------------------------------------------------------------------ free and compact

def _run_free(lens, table, rows, page, P):
    l, t = _i32(lens), _i32(table)
    refs, free, n = fa.paged_free(l, t, _i32(rows), page, P)
    _ok()
    rl, rt, rrefs, rfree = pages.free(lens, table, rows, page, P)
    assert np.array_equal(l.cpu().numpy(), rl)
    assert np.array_equal(t.cpu().numpy(), rt)
    assert np.array_equal(refs.cpu().numpy(), rrefs)
    assert n.item() == len(rfree)
    assert free.tolist() == rfree + [-1] * (P - len(rfree))
    return rl, rt


def _run_compact(lens, table, page, P):
    l, t = _i32(lens), _i32(table)
    moved, frm, to, used = fa.paged_compact(l, t, page, P)
    _ok()
    rt, rmoved, copies, U = pages.compact(lens, table, page, P)
    assert np.array_equal(l.cpu().numpy(), lens)
    assert np.array_equal(t.cpu().numpy(), rt)
    assert np.array_equal(moved.cpu().numpy(), rmoved)
    assert used.item() == U
    pad = [-1] * (frm.numel() - len(copies))
    assert frm.tolist() == [a for a, _ in copies] + pad
    assert to.tolist() == [b for _, b in copies] + pad
    return frm, to


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("B,M,P", [(1, 1, 1), (1, 3, 2), (5, 4, 40), (40, 30, 1300), (300, 20, 5000),
                                   (3, 900, 2701), (64, 128, 70001)])
def test_free_and_compact(page, B, M, P):
    rng, lens, table, _ = _cache(B + page + P, B, M, page, P)
    rows = rng.integers(-1, B + 1, B // 3 + 1)
    _run_free(lens, table, [], page, P)
    lens, table = _run_free(lens, table, np.concatenate([rows, rows]), page, P)
    _run_compact(lens, table, page, P)


def test_free_and_compact_of_full_and_empty_pools():
    table = np.arange(64).reshape(4, 16)
    full = [256, 256, 250, 241]
    _run_free(full, table, [], 16, 64)
    _run_compact(full, table, 16, 64)                                 # nothing to move
    _run_compact(full, table[::-1].copy() + 3, 16, 67)                # by three pages
    _run_free(full, table, [0, 1, 2, 3], 16, 64)
    _run_compact([0, 0, 0, 0], table, 16, 64)
    _run_compact([-5, 1000, 0, 0], table, 16, 64)                     # lengths are clamped
    # every page named by every row
    _run_free([4096] * 100, np.tile(np.arange(256), (100, 1)), [7], 16, 300)
    _run_compact([4096] * 100, np.tile(300 - 1 - np.arange(256), (100, 1)), 16, 300)


def test_free_and_compact_of_the_largest_batch():
    B = 8192
    rng = np.random.default_rng(5)
    lens, table = rng.integers(0, 33, B), rng.permutation(3 * B)[:2 * B].reshape(B, 2)
    lens, table = _run_free(lens, table, rng.permutation(B)[:3000], 16, 3 * B)
    _run_compact(lens, table, 16, 3 * B)


def test_free_and_compact_captured_and_replayed():
    # what the tables, the lengths and the ended rows hold is read at every replay
    B, M, page, P = 40, 30, 16, 1300
    l, t = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, M, dtype=I32, device="cuda")
    done, pool = torch.zeros(12, dtype=I32, device="cuda"), torch.zeros(P, 1, page, 64, device="cuda")
    pool = pool.bfloat16()

    def step():
        ended = fa.paged_free(l, t, done, page, P)
        moves = fa.paged_compact(l, t, page, P)
        fa.paged_copy(pool, None, *moves[1:3])
        return ended + moves

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        refs, free, n, moved, frm, to, used = step()
    for seed in range(3):
        rng, lens, table, _ = _cache(seed, B, M, page, P)
        rows = rng.integers(-1, B + 1, done.numel())
        before = torch.randn(pool.shape, generator=_gen(seed)).bfloat16()
        for x, y in ((l, lens), (t, table), (done, rows)):
            x.copy_(_i32(y))
        pool.copy_(before)
        gr.replay()
        _ok()
        rl, rt, rrefs, rfree = pages.free(lens, table, rows, page, P)
        rt, rmoved, copies, U = pages.compact(rl, rt, page, P)
        assert np.array_equal(l.cpu().numpy(), rl) and np.array_equal(t.cpu().numpy(), rt)
        assert np.array_equal(refs.cpu().numpy(), rrefs) and n.item() == len(rfree)
        assert free.tolist() == rfree + [-1] * (P - len(rfree))
        assert np.array_equal(moved.cpu().numpy(), rmoved) and used.item() == U
        m = len(copies)
        assert list(zip(frm.tolist(), to.tolist()))[:m] == copies and (frm[m:] == -1).all()
        assert np.array_equal(_np(pool), pages.copy(_np(before), frm.tolist(), to.tolist()))


# ------------------------------------------------------------------ copies

@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hkv,d", [(1, 64), (3, 128), (8, 128), (2, 64)])
@pytest.mark.parametrize("rows", [False, True])
def test_copy(page, Hkv, d, rows):
    g = _gen(page + d)
    P, n = 37, 15
    k, v = (torch.randn(P, Hkv, page, d, generator=g).bfloat16() for _ in range(2))
    ids = torch.randperm(P, generator=g).int()
    src, dst = ids[:n].clone(), ids[n:2 * n].clone()
    src[1], dst[2], src[3], dst[4], src[5] = -1, -1, P, 2 ** 31 - 1, dst[5]
    count = torch.randint(0, page + 1, (n,), generator=g).int()
    count[6], count[7], count[8] = 0, page + 9, -3
    count = count if rows else None
    kg, vg = k.cuda(), v.cuda()
    args = src.cuda(), dst.cuda(), None if count is None else count.cuda()
    fa.paged_copy(kg, vg, *args)
    _ok()
    want = [pages.copy(_np(x), src.tolist(), dst.tolist(), None if count is None else count.tolist())
            for x in (k, v)]
    assert np.array_equal(_np(kg), want[0]) and np.array_equal(_np(vg), want[1])
    one = k.cuda()
    fa.paged_copy(one, None, *args)
    _ok()
    assert torch.equal(one, kg)


@pytest.mark.parametrize("page", [16, 128])
def test_copy_of_latent_and_strided_pools(page):
    g = _gen(3)
    both = torch.randn(9, 2, page, 576, generator=g).bfloat16().cuda()
    keep = _np(both)
    src, dst, rows = [1, 0, 7], [8, 3, 5], [page, 7, 1]
    fa.paged_copy(both[:, 1], None, _i32(src), _i32(dst), _i32(rows))
    _ok()
    assert np.array_equal(_np(both[:, 0]), keep[:, 0])
    assert np.array_equal(_np(both[:, 1]), pages.copy(keep[:, 1], src, dst, rows))
    kv = torch.randn(9, 2, 2, page, 64, generator=g).bfloat16().cuda()
    keep = _np(kv)
    fa.paged_copy(kv[:, 0], kv[:, 1], _i32(src), _i32(dst))
    _ok()
    for i in range(2):
        assert np.array_equal(_np(kv[:, i]), pages.copy(keep[:, i], src, dst))


def test_copy_of_a_long_list_and_of_none():
    g = _gen(4)
    P = 20000
    k = torch.randn(P, 1, 16, 64, generator=g).bfloat16().cuda()
    src, dst = torch.randperm(P, generator=g).int().cuda().chunk(2)
    want = k.clone()
    want[dst.long()] = k[src.long()]
    fa.paged_copy(k, None, src, dst)
    fa.paged_copy(k, None, src[:0], dst[:0])
    _ok()
    assert torch.equal(k, want)


def test_copy_past_32_bit_offsets():
    # 2.2 G elements a pool, the copied pages at its end
    P, Hkv, page, d = 16800, 8, 128, 128
    k = torch.zeros(P, Hkv, page, d, dtype=BF, device="cuda")
    k[P - 2] = torch.randn(Hkv, page, d, generator=_gen(5)).bfloat16().cuda()
    fa.paged_copy(k, None, _i32([P - 2, P - 2]), _i32([P - 1, 3]), _i32([page, 50]))
    _ok()
    assert torch.equal(k[P - 1], k[P - 2]) and torch.equal(k[3, :, :50], k[P - 2, :, :50])
    assert not k[3, :, 50:].any() and not k[4].any()


def test_pages_on_a_named_stream():
    s = torch.cuda.Stream()
    rng, lens, table, free = _cache(3, 8, 6, 16, 60, shared=False)
    l, t, f = _i32(lens), _i32(table), _i32(free)
    done = _i32([2])
    s.wait_stream(torch.cuda.current_stream())
    refs, free_pages, n = fa.paged_free(l, t, done, 16, 60, stream=s)
    moved, frm, to, used = fa.paged_compact(l, t, 16, 60, stream=s)
    s.synchronize()
    _ok()
    rl, rt, rrefs, rfree = pages.free(lens, table, [2], 16, 60)
    rt, rmoved, copies, U = pages.compact(rl, rt, 16, 60)
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(moved.cpu().numpy(), rmoved)
    assert np.array_equal(refs.cpu().numpy(), rrefs) and used.item() == U and n.item() == len(rfree)
