"""Block tables and slot maps, cache appends and decode over a paged cache, on the GPU, against
the oracle."""
import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import paged

from _latent_bound import check_lse, check_o

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _np(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def _ok():
    torch.cuda.synchronize()
    assert fa.fa_device_error() == fa.FA_OK


# ------------------------------------------------------------------ tables

def _run_tables(old, new, free, table, page, P, T):
    t = _i32(table)
    total, start, slots, taken = fa.paged_tables(_i32(old), _i32(new), _i32(free), t, page, P, T)
    _ok()
    rt, rtotal, rstart, rslots, rtaken = paged.tables(old, new, free, table, page, P, T)
    assert np.array_equal(t.cpu().numpy(), rt)
    assert np.array_equal(total.cpu().numpy(), rtotal)
    assert np.array_equal(start.cpu().numpy(), rstart)
    assert np.array_equal(slots.cpu().numpy(), rslots)
    assert taken.item() == rtaken


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("B,max_old,max_new", [(1, 0, 1), (1, 500, 700), (3, 40, 1), (257, 300, 40),
                                               (1000, 70, 9)])
def test_tables(page, B, max_old, max_new):
    rng = np.random.default_rng(B + page)
    old, new = rng.integers(0, max_old + 1, B), rng.integers(0, max_new + 1, B)
    M = -(-(max_old + max_new) // page)
    P = B * M + 10
    ids = rng.permutation(P)
    have = -(-old // page)
    table = np.full((B, M), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    need = int((-(-(old + new) // page) - have).sum())
    T = int(new.sum())
    _run_tables(old, new, ids[at:at + need + 2], table, page, P, T + 5)    # rows behind the last
    _run_tables(old, new, ids[at:at + need // 2], table, page, P, T)       # a list too short
    _run_tables(old, new, ids[at:at + need], table, page, P, T // 2)       # fewer slots than tokens


def test_tables_clamp_lengths_and_leave_the_rest():
    # lengths below 0 and past the row, entries outside the pool, an empty free list
    _run_tables([-5, 70, 10, 64], [3, 9, 100, 5], [], np.full((4, 4), 99), 16, 8, 200)
    _run_tables([0, 0, 0], [0, 0, 0], [1, 2], np.full((3, 2), 7), 16, 8, 4)
    _run_tables([16], [1], [5], np.array([[-3, 6]]), 16, 8, 3)
    _run_tables([15], [2], [11], np.array([[-3, 6]]), 16, 8, 3)            # 11 is no page of 8
    # a view of wider rows keeps what lies beside it
    wide = torch.full((3, 8), 42, dtype=I32, device="cuda")
    fa.paged_tables(_i32([0, 5, 40]), _i32([17, 1, 30]), _i32([3, 1, 0, 2, 4, 5]), wide[:, 1:6],
                    16, 6, 50)
    _ok()
    assert wide.cpu().tolist() == [[42, 3, 1, 42, 42, 42, 42, 42], [42] * 8,
                                   [42, 42, 42, 42, 0, 2, 42, 42]]


def test_tables_of_the_largest_batch():
    B = 8192
    rng = np.random.default_rng(0)
    old, new = rng.integers(0, 20, B), rng.integers(0, 3, B)
    table = np.full((B, 2), -1)
    table[old > 0, 0] = rng.permutation(B)[:(old > 0).sum()]
    table[old > 16, 1] = B + np.arange((old > 16).sum())
    free = 2 * B + np.arange(B)
    _run_tables(old, new, free, table, 16, 4 * B, int(new.sum()) + 3)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("T,Hkv,d", [(1, 1, 64), (7, 3, 128), (300, 8, 128), (33, 2, 64)])
def test_append(T, Hkv, d, page):
    g = _gen(T + d)
    P = -(-T // page) + 3
    k, v = (torch.randn(T, Hkv, d, generator=g).bfloat16() for _ in range(2))
    kc, vc = (torch.randn(P, Hkv, page, d, generator=g).bfloat16() for _ in range(2))
    slots = torch.randperm(P * page, generator=g)[:T].int()
    if T > 3:
        slots[1], slots[2], slots[3] = -1, P * page, 2 ** 31 - 1      # no slots of the pool
    kg, vg = kc.cuda(), vc.cuda()
    fa.paged_append(k.cuda(), v.cuda(), kg, vg, slots.cuda())
    _ok()
    s = slots.tolist()
    assert np.array_equal(_np(kg), paged.append(_np(kc), _np(k), s))
    assert np.array_equal(_np(vg), paged.append(_np(vc), _np(v), s))


def test_append_takes_strided_rows_and_pages():
    # rows as slices of one fused projection; keys and values side by side in one allocation
    T, Hkv, d, page, P = 50, 2, 64, 32, 6
    g = _gen(3)
    fused = torch.randn(T, 3 * Hkv, d, generator=g).bfloat16().cuda()
    pool = torch.zeros(P, 2, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(P * page, generator=g)[:T].int()
    fa.paged_append(fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:], pool[:, 0], pool[:, 1], slots.cuda())
    _ok()
    for i in range(2):
        rows = _np(fused[:, (1 + i) * Hkv:(2 + i) * Hkv])
        assert np.array_equal(_np(pool[:, i]),
                              paged.append(np.zeros((P, Hkv, page, d)), rows, slots.tolist()))


def test_append_of_nothing():
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.ones(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    fa.paged_append(z, z, pool, pool.clone(), _i32([]))
    _ok()
    assert (pool == 1).all()


# ------------------------------------------------------------------ decode

def _case(lens, Hq, Hkv, d, page, seed, M=None, holes=0, nan=True):
    """Queries, pools whose every row outside the sequences is NaN, a table with random pages."""
    g = _gen(seed)
    B = len(lens)
    used = [-(-max(n, 0) // page) for n in lens]
    M = max(1, max(used)) if M is None else M
    P = sum(used) + 2
    order = torch.randperm(P, generator=g)
    table = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, M), generator=g).int()   # unused: anything
    q = torch.randn(B, Hq, d, generator=g).bfloat16()
    k = torch.randn(P, Hkv, page, d, generator=g).bfloat16()
    v = torch.randn(P, Hkv, page, d, generator=g).bfloat16()
    inside = torch.zeros(P, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        pages = order[at:at + used[b]]
        table[b, :used[b]] = pages.int()
        for i, p in enumerate(pages.tolist()):
            inside[p, :max(0, min(page, n - i * page))] = True
        at += used[b]
    for i in range(holes):      # entries of sequence i % B that name no page
        b = i % B
        if used[b]:
            e = int(torch.randint(0, used[b], (1,), generator=g))
            if 0 <= table[b, e] < P:
                inside[table[b, e]] = False
            table[b, e] = [-1, P, 2 ** 31 - 1][i % 3]
    if nan:
        k.masked_fill_(~inside[:, None, :, None], float("nan"))
        v.masked_fill_(~inside[:, None, :, None], float("inf"))
    return q.cuda(), k.cuda(), v.cuda(), table.cuda(), _i32(lens)


def _check(x, scale=None, run=None):
    q, k, v, table, lens = x
    o, lse = fa.decode_paged(q, k, v, table, lens, scale) if run is None else run
    _ok()
    ro, rlse, spread = paged.decode(_np(q), _np(k), _np(v), table.cpu().numpy(), lens.tolist(),
                                    1 / q.shape[-1] ** 0.5 if scale is None else scale)
    assert torch.isfinite(o.float()).all()
    check_o(_np(o), ro, spread)
    check_lse(_np(lse), rlse)
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_lengths_around_tiles_and_pages(d, page):
    lens = [1, 0, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 0, 640]
    _check(_case(lens, 8, 2, d, page, seed=page + d))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_groups_of_heads(G, d):
    _check(_case([200, 1, 333], 3 * G, 3, d, 16, seed=G))


@pytest.mark.parametrize("B", [1, 5])
def test_decode_one_token_and_none(B):
    _check(_case([1] * B, 4, 4, 64, 16, seed=1))
    x = _case([0] * B, 4, 4, 64, 16, seed=2)
    o, lse = _check(x)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_decode_many_short_sequences():
    rng = np.random.default_rng(4)
    _check(_case(rng.integers(0, 90, 700).tolist(), 2, 1, 64, 32, seed=4))


def test_decode_one_long_sequence():
    _check(_case([20011], 8, 1, 128, 64, seed=5))


@pytest.mark.parametrize("page", [16, 128])
def test_decode_holes_hide_their_keys(page):
    _check(_case([700, 130, 5, 900], 4, 2, 64, page, seed=6, holes=9))
    # a sequence whose every page is a hole sees nothing
    x = _case([300, 200], 4, 2, 128, page, seed=7)
    x[3][1] = -1
    o, lse = _check(x)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_decode_clamps_lengths():
    x = _case([64, 64], 4, 2, 64, 32, seed=8, M=2)
    x[4][0], x[4][1] = 1000, -7
    _check(x)


def test_decode_growing_scores():
    # scores that rise along the cache by far more than the rescale threshold, and a huge first
    # one; scores as large as these make one key's weight all of a row's
    q, k, v, table, lens = _case([2000, 700], 8, 2, 128, 16, seed=9)
    ramp = torch.linspace(0.1, 30, k.shape[0], device="cuda").bfloat16()
    _check((q, (k.float() * ramp[:, None, None, None].float()).bfloat16(), v, table, lens))
    _check((q, k, v, table, lens), scale=3.0)
    _check((q, k, v, table, lens), scale=1e-6)


def test_decode_strided_pages_tables_and_a_shared_prefix():
    q, k, v, table, lens = _case([300, 333, 40], 4, 2, 64, 32, seed=10)
    both = torch.full((k.shape[0], 2) + k.shape[1:], float("nan"), device="cuda").bfloat16()
    both[:, 0], both[:, 1] = k, v
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=I32, device="cuda")
    wide[:, 2:-3] = table
    wide[1, 2:6] = wide[0, 2:6]                       # four pages of sequence 0 serve 1 as well
    x = q, both[:, 0], both[:, 1], wide[:, 2:-3], lens
    _check(x)


def test_decode_workspace_may_hold_anything_and_repeats_bits():
    x = _case([1000, 3, 4000, 777], 16, 4, 128, 16, seed=11)
    ws = fa.alloc_decode_paged_workspace(4, 16, 4, 128)
    ws.fill_(0xff)
    a = fa.decode_paged(*x, workspace=ws)
    b = fa.decode_paged(*x, workspace=ws)
    _check(x, run=a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_nan_queries_stay_in_their_heads():
    x = _case([300, 200], 8, 2, 64, 16, seed=12)
    x[0][0, 3] = float("nan")
    o, lse = fa.decode_paged(*x)
    _ok()
    assert torch.isnan(o[0, 3].float()).all() and torch.isnan(lse[0, 3])
    x[0][0, 3] = 0
    ro, rl = _check(x)
    keep = torch.ones(2, 8, dtype=torch.bool)
    keep[0, 3] = False
    assert torch.equal(o[keep], ro[keep]) and torch.equal(lse[keep], rl[keep])


def test_a_long_cache_passes_32_bit_offsets():
    # 2.2 G elements a pool: the last pages lie past 2^31 elements and 2^32 bytes
    P, Hkv, page, d = 16800, 8, 128, 128
    k = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = _gen(13)
    T = 300
    rows = [torch.randn(T, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2)]
    table = _i32([[P - 1, 5, P - 2]])
    x = torch.arange(T)
    slots = (table[0].cpu()[x // page] * page + x % page).int().cuda()
    fa.paged_append(*rows, k, v, slots)
    q = torch.randn(1, 2 * Hkv, d, generator=g).bfloat16().cuda()
    o, lse = fa.decode_paged(q, k, v, table, _i32([T]))
    _ok()
    kk, vv = (r.cpu().transpose(0, 1)[None] for r in rows)      # [1, Hkv, T, d]: one page of T
    ro, rlse, spread = paged.decode(_np(q), _np(kk), _np(vv), np.array([[0]]), [T], d ** -0.5)
    check_o(_np(o), ro, spread)
    check_lse(_np(lse), rlse)


@pytest.mark.parametrize("layout", ["behind", "before", "beside", "beside_before", "one_page",
                                    "gaps"])
def test_append_takes_pools_in_one_allocation(layout):
    # keys' and values' pages next to one another in either order, in one block of memory
    T, Hkv, d, page = 9, 2, 64, 16
    P = 1 if layout == "one_page" else 4
    g = _gen(14)
    k, v = (torch.randn(T, Hkv, d, generator=g).bfloat16() for _ in range(2))
    slots = torch.randperm(P * page, generator=g)[:T].int()
    beside = layout in ("beside", "beside_before", "gaps")
    both = torch.zeros(*((P, 3 if layout == "gaps" else 2) if beside else (2, P)), Hkv, page, d,
                       dtype=torch.bfloat16, device="cuda")
    pools = both.unbind(1 if beside else 0)
    kc, vc = (pools[0], pools[-1]) if "before" not in layout else (pools[1], pools[0])
    fa.paged_append(k.cuda(), v.cuda(), kc, vc, slots.cuda())
    _ok()
    zero = np.zeros((P, Hkv, page, d))
    for c, x in ((kc, k), (vc, v)):
        assert np.array_equal(_np(c), paged.append(zero, _np(x), slots.tolist()))
    if layout == "gaps":
        assert (pools[1] == 0).all()


def test_append_of_the_same_rows_to_one_pool():
    # keys that are the values as well: one pool, the same bytes from both
    g = _gen(15)
    x = torch.randn(9, 2, 64, generator=g).bfloat16()
    slots = torch.randperm(64, generator=g)[:9].int()
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    rows = x.cuda()
    fa.paged_append(rows, rows, pool, pool, slots.cuda())
    _ok()
    assert np.array_equal(_np(pool), paged.append(np.zeros((4, 2, 16, 64)), _np(x), slots.tolist()))
    with pytest.raises(fa.FaError):
        fa.paged_append(rows, rows.clone(), pool, pool, slots.cuda())
