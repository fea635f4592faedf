"""Latent attention on the GPU against the oracle: expanded forward and backward (bf16 and fp32),
absorbed decode over a paged latent cache, and the append that fills it."""
import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import latent, paged

from _latent_bound import G, U, check_grads, check_lse, check_o
from test_gpu_paged import _gen, _i32, _np, _ok

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _inputs(B, H, N, dtype, seed, kv_len=None, mult=1.0):
    g = _gen(seed)
    dt = DT[dtype]
    q = (torch.randn(B, H, N, 192, generator=g) * mult).to(dt)
    kn = torch.randn(B, H, N, 128, generator=g).to(dt)
    kr = torch.randn(B, N, 64, generator=g).to(dt)
    v = torch.randn(B, H, N, 128, generator=g).to(dt)
    do = torch.randn(B, H, N, 128, generator=g).to(dt)
    if kv_len is not None:        # rows past the length may hold anything
        for b, n in enumerate(kv_len):
            kn[b, :, max(n, 0):], kr[b, max(n, 0):] = float("nan"), float("inf")
            v[b, :, max(n, 0):] = float("nan")
    return [t.cuda() for t in (q, kn, kr, v, do)]


def _check(B, H, N, dtype, causal, kv_len=None, seed=0, mult=1.0, grad=True, scale=None):
    q, kn, kr, v, do = _inputs(B, H, N, dtype, seed, kv_len, mult)
    kl = None if kv_len is None else _i32(kv_len)
    o, lse, o_acc = fa.latent_forward(q, kn, kr, v, causal, kl, scale, need_grad=True)
    sc = SCALE if scale is None else scale
    host = [_np(t) for t in (q, kn, kr, v)]
    _ok()
    ro, rlse, spread = latent.forward(*host, sc, causal, kv_len)
    check_o(_np(o), ro, spread, dtype)
    check_lse(_np(lse), rlse, dtype)
    assert o_acc.dtype == torch.float32 and torch.equal(o_acc.to(o.dtype), o)
    o2, lse2 = fa.latent_forward(q, kn, kr, v, causal, kl, scale)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if not grad:
        return
    got = fa.latent_backward(q, kn, kr, v, o_acc, lse, do, causal, kl, scale)
    _ok()
    u = U[dtype] if dtype == "bf16" else 0.0
    ref, err = latent.backward(*host, _np(do), sc, causal, kv_len, u, G[dtype])
    check_grads([_np(t) for t in got], ref, err, dtype)
    if kv_len is not None:
        for b, n in enumerate(kv_len):
            for t in (got[1][b, :, max(n, 0):], got[2][b, max(n, 0):], got[3][b, :, max(n, 0):]):
                assert (t == 0).all()
    again = fa.latent_backward(q, kn, kr, v, o_acc, lse, do, causal, kl, scale)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 200, 256, 257, 333])
def test_lengths(N, causal, dtype):
    _check(1, 2, N, dtype, causal, seed=N)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [False, True])
def test_padded_batches_with_empty_sequences(causal, dtype):
    _check(6, 2, 300, dtype, causal, [300, 1, 0, 129, 64, 255], seed=1)
    _check(3, 1, 130, dtype, causal, [128, 0, 127], seed=2)


@pytest.mark.parametrize("H", [1, 5, 16])
def test_heads(H):
    _check(2, H, 150, "bf16", True, seed=H)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_sequences(dtype):
    _check(1, 1, 1100, dtype, True, seed=3)
    _check(1, 2, 900, dtype, False, [801], seed=4)


@pytest.mark.parametrize("causal", [False, True])
def test_more_units_than_multiprocessors(causal):
    # CTAs take further units as they finish: 480 of them, empty and one-key sequences among them
    lens = [300, 0, 257, 1, 128, 300, 129, 0, 255, 256, 2, 300, 0, 0, 127]
    _check(15, 16, 300, "bf16", causal, lens, seed=8, grad=False)
    _check(13, 4, 700, "bf16", causal, None, seed=9, grad=False)


def test_two_streams_at_once():
    # each grid hands its units to its own CTAs only
    x = [_inputs(B, H, N, "bf16", 10 + N) for B, H, N in ((20, 16, 260), (9, 16, 515))]
    want = [fa.latent_forward(*t[:4], True, need_grad=True) for t in x]
    _ok()
    streams = [torch.cuda.Stream() for _ in x]
    got = [[], []]
    for _ in range(6):
        for i, (t, s) in enumerate(zip(x, streams)):
            got[i].append(fa.latent_forward(*t[:4], True, need_grad=True, stream=s))
    _ok()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


def test_peaked_scores():
    # rows whose weight is almost all on one key: D, dP and dS nearly cancel
    _check(1, 2, 260, "bf16", True, seed=5, mult=6.0)
    _check(1, 2, 260, "bf16", False, seed=6, scale=1e-4)


@pytest.mark.parametrize("causal,N,rows", [(True, 2, 2), (False, 2, 2), (True, 3, 3), (True, 8, 8),
                                           (False, 5, 5), (True, 200, 128)])
def test_gradients_of_few_keys_carry_one_rounding(N, rows, causal):
    # Where a query sees few keys a rounding of dS to bf16 does not average out.  The first query
    # block's dS is exact to 2^-16, so dq there and (N <= 128) dk carry the rounding of the result
    # alone: off by at most h = 2^-8 of a value, evenly, so h / sqrt(3) of it in the mean square at
    # the lowest mantissa.  n values move that by 1 / sqrt(5 n) of it (the fourth moment of an even
    # distribution), below 0.011 for the 1536 values here at the least; four times that is allowed.
    worst = {}
    for seed in range(8):
        q, kn, kr, v, do = _inputs(4, 2, N, "bf16", 100 * N + seed)
        o, lse, o_acc = fa.latent_forward(q, kn, kr, v, causal, need_grad=True)
        got = fa.latent_backward(q, kn, kr, v, o_acc, lse, do, causal)
        _ok()
        ref, _ = latent.backward(*[_np(t) for t in (q, kn, kr, v, do)], SCALE, causal)
        for name, x, r in zip(("dq", "dk_nope", "dk_rope"), got, ref):
            if name != "dq" and N > 128:
                continue
            x = _np(x)
            if name == "dq":
                x, r = x[:, :, :rows], r[:, :, :rows]
            off = np.linalg.norm(x - r) / np.linalg.norm(r)
            worst[name] = max(worst.get(name, 0.0), off)
    limit = 2.0 ** -8 / np.sqrt(3) * 1.05
    assert all(e <= limit for e in worst.values()), (worst, limit)


def test_lengths_past_the_range_are_clamped():
    q, kn, kr, v, do = _inputs(2, 2, 100, "bf16", 7)
    a = fa.latent_forward(q, kn, kr, v, True, _i32([500, -3]))
    b = fa.latent_forward(q, kn, kr, v, True, _i32([100, 0]))
    _ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ absorbed decode

def _decode_case(lens, H, page, seed, holes=0, extra=0):
    g = _gen(seed)
    B = len(lens)
    used = [-(-max(n, 0) // page) for n in lens]
    P, M = sum(used) + 2, max(1, max(used)) + extra
    order = torch.randperm(P, generator=g)
    table = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, M), generator=g).int()
    q = torch.randn(B, H, 576, generator=g).bfloat16()
    cache = torch.randn(P, page, 576, generator=g).bfloat16()
    inside = torch.zeros(P, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        pages = order[at:at + used[b]]
        table[b, :used[b]] = pages.int()
        for i, p in enumerate(pages.tolist()):
            inside[p, :max(0, min(page, n - i * page))] = True
        at += used[b]
    for i in range(holes):
        b = i % B
        if used[b]:
            e = int(torch.randint(0, used[b], (1,), generator=g))
            if 0 <= table[b, e] < P:
                inside[table[b, e]] = False
            table[b, e] = [-1, P, 2 ** 31 - 1][i % 3]
    cache.masked_fill_(~inside[..., None], float("nan"))
    return q.cuda(), cache.cuda(), table.cuda(), _i32(lens)


def _check_decode(x, scale=None, run=None):
    q, cache, table, lens = x
    o, lse = fa.latent_decode(q, cache, table, lens, scale) if run is None else run
    _ok()
    ro, rlse, spread = latent.decode(_np(q), _np(cache), table.cpu().numpy(), lens.tolist(),
                                     SCALE if scale is None else scale, 512)
    assert torch.isfinite(o.float()).all()
    check_o(_np(o), ro, spread)
    check_lse(_np(lse), rlse)
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H", [1, 16, 128])
def test_decode_lengths_around_tiles_and_pages(H, page):
    _check_decode(_decode_case([1, 0, 15, 16, 63, 64, 65, 127, 128, 129, 300, 0, 515], H, page,
                               seed=page + H))


@pytest.mark.parametrize("H", [2, 7, 20, 33, 64, 96, 100, 127])
def test_decode_heads(H):
    _check_decode(_decode_case([130, 1, 70], H, 32, seed=H))


def test_decode_one_long_and_many_short_sequences():
    _check_decode(_decode_case([12001], 16, 64, seed=20))
    rng = np.random.default_rng(21)
    _check_decode(_decode_case(rng.integers(0, 70, 500).tolist(), 4, 16, seed=21))


def test_decode_holes_clamps_and_empties():
    _check_decode(_decode_case([700, 130, 5, 400], 8, 16, seed=22, holes=9))
    x = _decode_case([300, 200], 8, 64, seed=23)
    x[2][1] = -1
    o, lse = _check_decode(x)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    x = _decode_case([128, 128], 8, 64, seed=24)
    x[3][0], x[3][1] = 4000, -1
    _check_decode(x)


def test_decode_growing_scores():
    q, cache, table, lens = _decode_case([1500, 300], 16, 16, seed=25)
    # a rotated part that rises along the pool: maxima that grow tile by tile
    ramp = torch.linspace(0.1, 40, cache.shape[0], device="cuda")
    c = cache.float()
    c[..., 512:] *= ramp[:, None, None]
    _check_decode((q, c.bfloat16(), table, lens))
    _check_decode((q, cache, table, lens), scale=2.0)


def test_decode_strides_and_workspace():
    q, cache, table, lens = _decode_case([500, 90, 700], 24, 32, seed=26)
    wide = torch.full((cache.shape[0], 2) + cache.shape[1:], float("nan"), device="cuda").bfloat16()
    wide[:, 1] = cache
    tw = torch.full((3, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    tw[:, 1:-2] = table
    x = q, wide[:, 1], tw[:, 1:-2], lens
    ws = fa.alloc_latent_decode_workspace(3, 24)
    ws.fill_(0xff)
    a = fa.latent_decode(*x, workspace=ws)
    b = fa.latent_decode(*x, workspace=ws)
    _check_decode(x, run=a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 9, 400])
def test_append(T):
    g = _gen(T)
    page, P = 32, -(-T // 32) + 2
    c, r = torch.randn(T, 512, generator=g).bfloat16(), torch.randn(T, 64, generator=g).bfloat16()
    cache = torch.randn(P, page, 576, generator=g).bfloat16()
    slots = torch.randperm(P * page, generator=g)[:T].int()
    if T > 2:
        slots[0], slots[2] = -1, P * page
    fused = torch.cat([torch.zeros(T, 8), c.float(), r.float()], 1).bfloat16().cuda()
    out = cache.cuda()
    fa.latent_append(fused[:, 8:520], fused[:, 520:], out, slots.cuda())
    _ok()
    rows = np.concatenate([_np(c), _np(r)], 1)
    assert np.array_equal(_np(out), paged.append(_np(cache), rows, slots.tolist()))
