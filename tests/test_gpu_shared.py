"""Decode attention for groups of sequences with a prefix in common, on the GPU, against the oracle
of the paged decode (the definition does not know of groups): lengths around tiles, pages and pieces,
groups of any size, sequences that are shorter than what their group shares, holes and bad values in
hidden places; then the operators of a cache's pages with it, step after step."""
import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import paged, pages, rope

from _latent_bound import check_lse, check_o
from test_gpu_paged import _gen, _i32, _np, _ok

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


def _columns(B, Hkv, page):
    """Columns of a table with so much room that the groups' tokens are read together at any lengths."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return (44 * sms // (B * Hkv) + 2) * 128 // page


def _case(groups, Hq, Hkv, d, page, seed, M=None, nan=True, spare=3):
    """groups: [(shared tokens, [lengths])].  Sequences of a group that reach its shared tokens name the
    same pages for them; rows outside the lengths hold NaN and infinity.  The table is a wide one."""
    g = _gen(seed)
    lens = [n for _, l in groups for n in l]
    B = len(lens)
    M = M or max(1, max(-(-n // page) for n in lens + [s for s, _ in groups])) + 1
    P = B * M + spare
    ids = torch.randperm(P, generator=g).int()
    table = torch.full((B, M), -1, dtype=I32)
    at = b = 0
    start = [0]
    for shared, ls in groups:
        first = None
        for n in ls:
            used = -(-min(n, M * page) // page)
            table[b, :used] = ids[at:at + used]
            at += used
            full = -(-min(shared, M * page) // page)
            if n >= shared and shared > 0:
                if first is None:
                    first = b
                table[b, :full] = table[first, :full]
            b += 1
        start.append(b)
    k, v = (torch.randn(P, Hkv, page, d, generator=g).bfloat16() for _ in range(2))
    if nan:
        inside = torch.zeros(P, page, dtype=torch.bool)
        for i, n in enumerate(lens):
            x = torch.arange(min(n, M * page))
            inside[table[i].long()[x // page], x % page] = True
        k.masked_fill_(~inside[:, None, :, None], float("nan"))
        v.masked_fill_(~inside[:, None, :, None], float("inf"))
    q = torch.randn(B, Hq, d, generator=g).bfloat16()
    table = torch.cat([table, table.new_full((B, _columns(B, Hkv, page)), -1)], 1)
    return [q.cuda(), k.cuda(), v.cuda(), table.cuda(), _i32(lens), _i32(start),
            _i32([s for s, _ in groups])]


def _narrow(x):
    """The same batch with the table's columns behind the last page left out."""
    used = (x[3] != -1).any(0).nonzero()
    return x[:3] + [x[3][:, :int(used.max()) + 1 if used.numel() else 1].contiguous()] + x[4:]


def _check(x, scale=None, run=None):
    """Without `run` also of the narrow table, with which a small batch is decoded apart."""
    runs = [run]
    if run is None:
        runs = [fa.decode_shared(*y, scale) for y in (x, _narrow(x))]
    _ok()
    q, k, v, table, lens = x[:5]
    ro, rlse, spread = paged.decode(_np(q), _np(k), _np(v), table.cpu().numpy(), lens.tolist(),
                                    1 / q.shape[-1] ** 0.5 if scale is None else scale)
    for o, lse in runs:
        assert torch.isfinite(o.float()).all()
        check_o(_np(o), ro, spread)
        check_lse(_np(lse), rlse)
    return runs[0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("shared", [1, 16, 127, 128, 129, 256, 300, 512, 640])
def test_shared_lengths_around_tiles_and_pages(d, page, shared):
    lens = [shared, shared + 1, shared + 15, shared + 16, shared + 128, shared + 300]
    _check(_case([(shared, lens)], 8, 2, d, page, seed=page + d + shared))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [2, 8, 9, 33, 70])
def test_shared_groups_of_heads_and_pieces_of_a_batch(G, d, B):
    # 128 / G sequences a tile, twice as many a piece: one tile, two, several pieces, a rest
    rng = np.random.default_rng(G * B)
    _check(_case([(200, (200 + rng.integers(0, 90, B)).tolist())], 2 * G, 2, d, 16, seed=G + B))


@pytest.mark.parametrize("seed", range(6))
def test_shared_many_groups(seed):
    rng = np.random.default_rng(seed)
    groups = []
    for _ in range(rng.integers(1, 14)):
        shared = int(rng.integers(0, 900))
        n = int(rng.integers(0, 12))
        ls = [int(shared + rng.integers(0, 400)) for _ in range(n)]
        for i in range(n):      # shorter than the prefix, empty
            if rng.random() < 0.2:
                ls[i] = int(rng.integers(0, shared + 1)) if rng.random() < 0.6 else 0
        groups.append((shared, ls))
    groups.append((17, [17]))
    page = [16, 32, 64, 128, 256, 16][seed]
    _check(_case(groups[-14:], 6, 2 if seed % 2 else 3, 64 if seed < 3 else 128, page, seed))


def test_shared_that_nobody_or_everybody_has():
    # nothing shared; a prefix that no sequence reaches; sequences that are the prefix
    _check(_case([(0, [5, 300, 0])], 4, 2, 64, 16, seed=1))
    _check(_case([(500, [100, 0, 499, 33])], 4, 2, 64, 16, seed=2))
    _check(_case([(512, [512] * 9)], 4, 2, 128, 64, seed=3))
    o, lse = _check(_case([(64, [0, 0, 0])], 4, 2, 64, 16, seed=4))
    assert (o == 0).all() and torch.isneginf(lse).all()
    _check(_case([(256, [300])], 4, 2, 64, 16, seed=5))


def test_shared_sequences_in_no_group():
    x = _case([(0, [70, 200]), (320, [400, 320, 500]), (0, [33, 129])], 4, 2, 64, 32, seed=6)
    x[5], x[6] = _i32([2, 5]), _i32([320])
    _check(x)


def test_shared_lengths_are_clamped():
    x = _case([(64, [64, 64]), (64, [64, 80])], 4, 2, 64, 32, seed=7, M=3)
    x[4][0], x[4][1] = 1000, -7
    x[3][0, :3] = torch.arange(3)
    x[1][:3], x[2][:3] = 1.0, 2.0
    x[6] = _i32([-3, 100000])
    _check(x)


@pytest.mark.parametrize("d", [64, 128])
def test_shared_lengths_past_a_wide_row_are_clamped(d):
    # The row is wide enough for the kernels that share, and full; lengths and shared lengths lie past
    # it.  Behind it the buffer goes on with pages whose values would show.
    B, Hq, Hkv, page = 16, 8, 4, 16
    M = _columns(B, Hkv, page)
    cap, far, P = M * page, 2 ** 31 - 1, 4 * M + 12
    lens = [cap + 1000, far, cap, cap - 5, -7, 80, far, 40, 0, cap + 1] + [9, 0, 33, cap + 16, 5, -1]
    start, shared = [0, 4, 6, 9, 10], [cap + 300, -3, far, 5]
    g = _gen(24 + d)
    ids = torch.randperm(P - 2, generator=g).int()
    wide = torch.full((B, M + 6), -1, dtype=I32)
    for b, at in ((0, 0), (6, M), (9, 2 * M), (13, 3 * M)):
        wide[b, :M] = ids[at:at + M]
    wide[1:4] = wide[0]
    for i, b in enumerate((5, 7, 10, 12, 14)):
        wide[b, :5] = ids[4 * M + 2 * i % 5:][:5]
    wide[:, M:] = torch.tensor([P - 2, P - 1, P - 2, P - 1, P - 2, P - 1])
    q = torch.randn(B, Hq, d, generator=g).bfloat16()
    k, v = (torch.randn(P, Hkv, page, d, generator=g).bfloat16() for _ in range(2))
    v[P - 2:] = 1000.0
    table = wide.cuda()[:, :M]
    runs = fa.decode_shared(q.cuda(), k.cuda(), v.cuda(), table, _i32(lens), _i32(start), _i32(shared))
    _ok()
    args = [_np(t) for t in (q, k, v)]
    ro, rlse, spread = paged.decode(*args, wide[:, :M].numpy(), lens, d ** -0.5)
    check_o(_np(runs[0]), ro, spread)
    check_lse(_np(runs[1]), rlse)
    # one token more of the full rows is far outside the bounds
    long = [i for i, n in enumerate(lens) if n > cap]
    po, _, _ = paged.decode(args[0][long], *args[1:], wide[long].numpy(), [cap + 1] * len(long), d ** -0.5)
    for i, b in enumerate(long):
        with pytest.raises(AssertionError):
            check_o(po[i], ro[b], spread[b])


@pytest.mark.parametrize("page", [16, 128])
def test_shared_holes_hide_their_keys(page):
    x = _case([(640, [640, 700, 900, 641]), (256, [256, 300])], 4, 2, 64, page, seed=8)
    P = x[1].shape[0]
    for c, e in ((0, -1), (2, P), (4, 2 ** 31 - 1)):
        if c * page < 640:
            x[3][:4, c] = e
    x[3][4:, 0] = -1
    _check(x)
    # a prefix that is nothing but holes, and one sequence that is
    x = _case([(256, [256, 300, 256])], 4, 2, 128, page, seed=9)
    x[3][:, :256 // page] = -1
    o, lse = _check(x)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_shared_growing_scores():
    x = _case([(2000, [2000, 2300, 2048])], 8, 2, 128, 16, seed=10, nan=False)
    order = x[3][1].clamp(min=0).long()
    ramp = torch.ones(x[1].shape[0], device="cuda")
    ramp[order] = torch.linspace(0.1, 30, order.numel(), device="cuda")
    y = list(x)
    y[1] = (x[1].float() * ramp.bfloat16().float()[:, None, None, None]).bfloat16()
    _check(y)
    _check(x, scale=3.0)
    _check(x, scale=1e-6)


def test_shared_long_prefix_and_large_batch():
    rng = np.random.default_rng(11)
    _check(_case([(9000, (9000 + rng.integers(0, 40, 40)).tolist())], 8, 2, 128, 64, seed=11))
    _check(_case([(130, (130 + rng.integers(0, 20, 300)).tolist())], 4, 1, 64, 32, seed=12))
    # one long prefix among groups of nobody's
    _check(_case([(0, [3])] * 20 + [(4000, [4000, 4100])] + [(100, [100, 150])] * 20, 2, 1, 64, 16,
                 seed=13))


@pytest.mark.parametrize("B, G", [(60, 16), (180, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_many_rows_to_join(B, G, d):
    # more rows than the combine has warps for four each, or for two
    rng = np.random.default_rng(B)
    _check(_case([(160, (160 + rng.integers(0, 40, B)).tolist())], 2 * G, 2, d, 32, seed=B + d))


def test_shared_strided_pages_and_tables():
    x = _case([(96, [96, 200, 130])], 4, 2, 64, 32, seed=14)
    both = torch.full((x[1].shape[0], 2) + x[1].shape[1:], float("nan"), device="cuda").bfloat16()
    both[:, 0], both[:, 1] = x[1], x[2]
    wide = torch.full((3, x[3].shape[1] + 5), -1, dtype=I32, device="cuda")
    wide[:, 2:-3] = x[3]
    x[1], x[2], x[3] = both[:, 0], both[:, 1], wide[:, 2:-3]
    _check(x)


def test_shared_workspace_may_hold_anything_and_repeats_bits():
    x = _case([(1000, [1000, 1500, 1100]), (64, [100, 4000])], 16, 4, 128, 16, seed=15)
    ws = fa.alloc_decode_shared_workspace(5, 16, 4, 128)
    ws.fill_(0xff)
    a = fa.decode_shared(*x, workspace=ws)
    b = fa.decode_shared(*x, workspace=ws)
    _check(x, run=a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_shared_nan_queries_stay_in_their_heads():
    x = _case([(300, [300, 400, 350])], 8, 2, 64, 16, seed=16)
    x[0][1, 3] = float("nan")
    o, lse = fa.decode_shared(*x)
    _ok()
    assert torch.isnan(o[1, 3].float()).all() and torch.isnan(lse[1, 3])
    x[0][1, 3] = 0
    ro, rl = _check(x)
    keep = torch.ones(3, 8, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(o[keep], ro[keep]) and torch.equal(lse[keep], rl[keep])


def test_shared_bad_values_in_the_prefix_do_not_reach_shorter_sequences():
    # a sequence that ends inside its group's tokens does not see those behind its end
    x = _case([(400, [400, 500, 250, 0])], 4, 2, 64, 16, seed=17, nan=False)
    x[3][2, :16] = x[3][0, :16]
    page = int(x[3][0, 20])
    x[2][page] = float("nan")
    o, lse = fa.decode_shared(*x)
    _ok()
    assert torch.isnan(o[:2].float()).all()
    ro, rlse, spread = paged.decode(*(_np(t) for t in x[:3]), x[3].cpu().numpy(), [0, 0, 250, 0],
                                    1 / 8)
    check_o(_np(o[2:]), ro[2:], spread[2:])
    check_lse(_np(lse[2:]), rlse[2:])


def test_shared_starts_that_are_not_ascending_touch_nothing_else():
    # the result is not defined; the call ends, and what lies beside the outputs stays
    x = _case([(200, [200, 300, 250]), (100, [100, 160]), (64, [64, 90, 70])], 4, 2, 64, 16, seed=18,
              nan=False)
    B, Hq, d = x[0].shape
    n = fa.fa_decode_shared_workspace_bytes(B, Hq, 2, d)
    for start in ([0, 5, 2, 8], [3, -9, 100, 2 ** 31 - 1], [8, 0, 8, 0], [0, 8, 0, 8]):
        buf = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        o = torch.zeros(B + 1, Hq, d, dtype=BF, device="cuda")
        lse = torch.zeros(B + 1, Hq, device="cuda")
        x[5] = _i32(start)
        fa.fa_decode_shared(*x, o[:B], lse[:B], buf[:n])
        _ok()
        assert (buf[n:] == 0x5a).all() and not o[B].any() and not lse[B].any()


def test_shared_past_32_bit_offsets():
    P, Hkv, page, d = 16800, 8, 128, 128
    k = torch.zeros(P, Hkv, page, d, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    at = [P - 1, 5, P - 2, P - 3]
    g = _gen(19)
    for p in at:
        k[p], v[p] = (torch.randn(Hkv, page, d, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(2, 2 * Hkv, d, generator=g).bfloat16().cuda()
    table, lens = torch.full((2, _columns(2, Hkv, page)), -1, dtype=I32, device="cuda"), _i32([300, 290])
    table[:, :3] = _i32([[P - 1, 5, P - 2], [P - 1, 5, P - 3]])
    o, lse = fa.decode_shared(q, k, v, table, lens, _i32([0, 2]), _i32([256]))
    _ok()
    small = np.array([[0, 1, 2], [0, 1, 3]])
    ro, rlse, spread = paged.decode(_np(q), _np(k[at]), _np(v[at]), small, [300, 290], d ** -0.5)
    check_o(_np(o), ro, spread)
    check_lse(_np(lse), rlse)


def test_shared_small_batches_are_decoded_apart():
    # a table with room for few tiles: the kernels of the paged decode, so its bits
    x = _narrow(_case([(500, [500, 640, 700, 64]), (0, [0])], 8, 2, 64, 16, seed=23))
    ws = fa.alloc_decode_shared_workspace(5, 8, 2, 64)
    ws.fill_(0xff)
    (o, lse), (po, plse) = fa.decode_shared(*x, workspace=ws), fa.decode_paged(*x[:5])
    _check(x, run=(o, lse))
    assert torch.equal(o, po) and torch.equal(lse, plse)


def test_shared_equals_the_paged_decode_of_the_same_tables():
    # other sums of the same terms: two fp32 roundings of o before its own, and half steps of bf16
    x = _case([(512, [512, 700, 530]), (128, [200, 129])], 8, 2, 128, 64, seed=20)
    a, b = fa.decode_shared(*x), fa.decode_paged(*x[:5])
    _check(x, run=a)
    _check(x, run=b)


def test_shared_captured_and_replayed_on_two_streams():
    xs = [_case([(300, [300, 420, 333, 0])], 8, 2, 64, 16, seed=s, nan=False) for s in (21, 22)]
    xs[0][3][3] = xs[0][3][0]      # the empty sequence's row names the shared pages, for the last replay
    ws = [fa.alloc_decode_shared_workspace(4, 8, 2, 64) for _ in xs]
    want = [fa.decode_shared(*x) for x in xs]
    graphs, outs = [], []
    for x, w in zip(xs, ws):
        o, lse = torch.empty_like(x[0]), torch.empty(4, 8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fa.fa_decode_shared(*x, o, lse, w)
        graphs.append(gr)
        outs.append((o, lse))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    _ok()
    for (o, lse), (ro, rl) in zip(outs, want):
        assert torch.equal(o, ro) and torch.equal(lse, rl)
    # the replay reads what is in the tensors then
    xs[0][4].copy_(_i32([300, 305, 0, 310]))
    graphs[0].replay()
    _check(xs[0], run=outs[0])


# ------------------------------------------------------------------ together

def test_samples_of_prompts_forked_grown_freed_and_compacted():
    """Two prompts are written with their positions, each is forked, the samples grow token by token in
    pages of their own, some end, the pool is compacted, the rest grows on; every step's outputs are
    those of the definition over the whole history."""
    B, page, P, Hq, Hkv, d = 7, 16, 90, 4, 2, 64
    M = _columns(B, Hkv, page)
    g = _gen(30)
    table, lens = torch.full((B, M), -1, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    kc, vc = (torch.full((P, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    free = torch.randperm(P, generator=g).int().cuda()
    plan = fa.rope_table(d, sections=[8, 12, 12])
    turns, axis = [int(t) % 2 ** 64 for t in plan[0]], plan[1].tolist()
    held = [([], []) for _ in range(B)]
    ws = fa.alloc_decode_shared_workspace(B, Hq, Hkv, d)
    groups = [_i32([0, 4, 7]), _i32([0, 0])]

    def step(new):
        nonlocal free
        T = sum(new) + 1                                       # a row of padding
        q, k, v = (torch.randn(T, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
        total, start, slots, taken = fa.paged_tables(lens, _i32(new), free, table, page, P, T)
        begin = start.tolist()
        pos = torch.zeros(3, T, dtype=I32)
        for b in range(B):
            x = torch.arange(begin[b + 1] - begin[b]) + len(held[b][0])
            pos[:, begin[b]:begin[b + 1]] = torch.stack([x, x // 3, x % 3])
        qr = fa.rope_append(q, k, v, pos.cuda(), plan, kc, vc, slots)
        lens.copy_(total)
        last = (start[1:] - 1).clamp(min=0).long()
        o, lse = fa.decode_shared(qr[last], kc, vc, table, lens, *groups, workspace=ws)
        _ok()
        free = free[taken.item():].contiguous()
        kr, _ = rope.rotate(_np(k), pos.numpy()[:, :, None], turns, axis)
        kr = torch.from_numpy(kr).bfloat16()
        for b in range(B):
            for t in range(begin[b], begin[b + 1]):
                held[b][0].append(kr[t])
                held[b][1].append(v[t].cpu())
        # the history, in a pool of one page a sequence; a key off by half a step of bf16 where the
        # fp64 rotation rounds the other way moves a score by 2^-8 of one product: taken from the cache
        n = max(1, max(len(h[0]) for h in held))
        hk, hv = torch.zeros(B, Hkv, n, d), torch.zeros(B, Hkv, n, d)
        for b in range(B):
            p, r = paged.visible(table[b].cpu().numpy(), int(lens[b]), page, P, M * page)
            got = kc[torch.from_numpy(p).long().cuda(), :, torch.from_numpy(r).long().cuda()].cpu()
            for t, (x, y) in enumerate(zip(*held[b])):
                assert torch.allclose(got[t].float(), x.float(), rtol=2.0 ** -7, atol=1e-5)
                hk[b, :, t], hv[b, :, t] = got[t].float(), y.float()
            assert len(p) == len(held[b][0])
        ro, rl, spread = paged.decode(_np(qr[last]), hk.numpy(), hv.numpy(), np.arange(B)[:, None],
                                      [len(h[0]) for h in held], d ** -0.5)
        check_o(_np(o), ro, spread)
        check_lse(_np(lse), rl)

    step([37, 0, 0, 0, 50, 0, 0])
    src, dst = _i32([0, 0, 0, 4, 4, -1]), _i32([1, 2, 3, 5, 6, -1])
    frm, to, rows, taken = fa.paged_fork(lens, table, free, src, dst, page, P)
    fa.paged_copy(kc, vc, frm, to, rows)
    assert taken.item() == 5
    free = free[5:].contiguous()
    for a, b in ((0, 1), (0, 2), (0, 3), (4, 5), (4, 6)):
        held[b] = (list(held[a][0]), list(held[a][1]))
    groups[1] = _i32([37 // page * page, 50])                 # the second one's last page is not shared
    groups[1][1] = 50 // page * page
    for new in ([1] * 7, [1, 0, 20, 1, 1, 3, 1], [1] * 7):
        step(new)
    done = _i32([2, 0, 5])
    refs, pages_free, n_free = fa.paged_free(lens, table, done, page, P)
    for b in (2, 0, 5):
        held[b] = ([], [])
    step([0, 1, 0, 1, 1, 0, 1])
    fa.paged_free(lens, table, _i32([]), page, P)
    moved, frm, to, used = fa.paged_compact(lens, table, page, P)
    fa.paged_copy(kc, vc, frm, to)
    U = used.item()
    free = torch.arange(U, P, dtype=I32, device="cuda")
    assert U == len({p for _, _, p in pages.live(table.cpu().numpy(), lens.tolist(), page, P)})
    for new in ([0, 1, 0, 1, 1, 0, 1], [5, 1, 0, 1, 17, 0, 1]):
        step(new)


def test_a_serving_step_captured_and_replayed():
    """rope_append and decode_shared, with a fork and its copies before, in one graph."""
    B, page, P, Hq, Hkv, d = 4, 16, 40, 4, 2, 128
    x = _case([(48, [48, 60, 49, 77])], Hq, Hkv, d, page, seed=31, nan=False, M=8)
    q0, kc, vc, table, lens, start, shared = x
    P = kc.shape[0]
    g = _gen(32)
    plan = fa.rope_table(d)
    new = [torch.randn(B, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
    pos = torch.zeros(1, B, dtype=I32, device="cuda")
    free = _i32(sorted(set(range(P)) - set(table.flatten().tolist())))
    ones, src, dst = _i32([1] * B), _i32([0]), _i32([3])
    ws = fa.alloc_decode_shared_workspace(B, Hq, Hkv, d)

    def step():
        frm, to, rows, taken = fa.paged_fork(lens, table, free, src, dst, page, P)
        fa.paged_copy(kc, vc, frm, to, rows)
        total, _, slots, _ = fa.paged_tables(lens, ones, free[4:], table, page, P, B)
        qr = fa.rope_append(*new, pos, plan, kc, vc, slots)
        return qr, total, fa.decode_shared(qr, kc, vc, table, total, start, shared, workspace=ws)

    keep = [t.clone() for t in (lens, table, kc, vc)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        qr, total, out = step()
    for n in range(3):
        for t, k in zip((lens, table, kc, vc), keep):
            t.copy_(k)
        pos.fill_(10 * n)
        for t in new:
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())
        gr.replay()
        _ok()
        assert lens.tolist()[3] == lens.tolist()[0]
        _check([qr, kc, vc, table, total], run=out)
