"""Rotary positions on the GPU against the oracle: layouts, strides, axes, far positions, gradients,
and the rows of new tokens turned into a paged cache.

Bound, element by element.  The angle is exact until its upper 32 bits become fp32, of half turns in
[-1, 1]: off by 2^-25 half turns, pi 2^-25, and by 2^-32 turns for the bits that are dropped.  Sine and
cosine are off by at most two steps of 2^-24 more, and each of the two products and the sum rounds
once: in all at most (|x_1| + |x_2|) e with e = pi 2^-25 + 2 pi 2^-32 + 2 2^-24 + 3 2^-24 < 2^-21.2,
taken as 2^-21.  The result is rounded to its type, half a step: 2^-8 of a bf16 value.
"""
import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import paged, rope

from test_gpu_paged import _gen, _np, _ok

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16
E = 2.0 ** -21
HALF = {BF: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _ints(table):
    return [int(t) % 2 ** 64 for t in table[0]], table[1].tolist()


def _close(y, ref, size, dtype):
    bound = (size * E) * (1 + HALF[dtype]) + HALF[dtype] * np.abs(ref)
    assert np.all(np.isfinite(y))
    bad = np.abs(y - ref) > bound
    assert not bad.any(), f"off by {np.max(np.abs(y - ref) / (bound + 1e-30)):.2f} of its bound"


def _check(x, y, pos, table, interleaved=False, inverse=False):
    """x, y [B, H, N, d]; pos [axes, B, N]."""
    turns, axis = _ints(table)
    ref, size = rope.rotate(_np(x), pos.cpu().numpy()[:, :, None], turns, axis, interleaved, inverse)
    _close(_np(y), ref, size, x.dtype)


def _pos(g, axes, B, N, far):
    return torch.randint(-far // 8, far, (axes, B, N), generator=g, dtype=I32).cuda()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,d,rot,axes", [
    (1, 1, 1, 64, 64, 1), (2, 3, 33, 128, 128, 3), (3, 5, 1, 128, 64, 2), (1, 2, 257, 64, 48, 2),
    (2, 1, 17, 24, 16, 1), (1, 9, 40, 192, 112, 3), (1, 33, 7, 16, 16, 1), (1, 1, 5, 1024, 1024, 4),
])
def test_rope_and_its_gradient(B, H, N, d, rot, axes, interleaved, dtype):
    g = _gen(N + d + axes)
    x = torch.randn(B, H, N, d, generator=g).to(dtype).cuda()
    dy = torch.randn(B, H, N, d, generator=g).to(dtype).cuda()
    pairs = rot // 2
    sections = [pairs // axes] * (axes - 1) + [pairs - pairs // axes * (axes - 1)]
    table, pos = fa.rope_table(rot, 10000.0, sections), _pos(g, axes, B, N, 5000)
    keep = x.clone()
    y = fa.rope(x, pos, table, interleaved)
    dx = fa.rope_backward(dy, pos, table, interleaved)
    _ok()
    assert torch.equal(x, keep) and y.is_contiguous()
    _check(x, y, pos, table, interleaved)
    _check(dy, dx, pos, table, interleaved, True)
    if rot < d:
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_gradient_against_differences():
    # linear in x, so a difference of any width is the derivative: <dx, e> = <dy, f(x + e) - f(x)>;
    # both sides are sums of n products, each off by e of the test's bound, in fp32
    g = _gen(1)
    x, e, dy = (torch.randn(1, 2, 50, 64, generator=g).cuda() for _ in range(3))
    table, pos = fa.rope_table(64, 500.0, [10, 22]), _pos(g, 2, 1, 50, 300)
    dx = fa.rope_backward(dy, pos, table)
    left = (dx.double() * e.double()).sum()
    diff = fa.rope(x + e, pos, table).double() - fa.rope(x, pos, table).double()
    right = (dy.double() * diff).sum()
    # every product's factors are off by at most E (|x_1| + |x_2|) + 2^-24, of values below some 10
    room = 6400 * (E + 2.0 ** -24) * 10 * 3
    assert abs(left - right) <= room and abs(left) > 10 * room


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 27, 2 ** 31 - 1])
def test_rope_of_far_positions(far):
    g = _gen(2)
    x = torch.randn(1, 2, 64, 64, generator=g).cuda()
    pos = torch.randint(far - far // 4, far, (1, 1, 64), generator=g, dtype=torch.int64)
    pos[0, 0, 0], pos[0, 0, 1] = far, -far
    pos = pos.to(I32).cuda()
    table = fa.rope_table(64)
    _check(x, fa.rope(x, pos, table), pos, table)


def test_rope_of_given_frequencies():
    # no turn, half and whole turns, backwards, more than a turn a position
    f = [0.0, np.pi, 2 * np.pi, -0.3, 12.345, 1e-7, 1.0, -50.0]
    table = fa.rope_table(16, frequencies=f)
    g = _gen(3)
    x = torch.randn(1, 1, 99, 16, generator=g).cuda()
    pos = torch.arange(99, dtype=I32, device="cuda")[None, None]
    y = fa.rope(x, pos, table)
    _check(x, y, pos, table)
    assert torch.equal(y[..., 0], x[..., 0])
    direct = torch.cos(torch.arange(99).double() * 12.345) * x[0, 0, :, 4].double().cpu() \
        - torch.sin(torch.arange(99).double() * 12.345) * x[0, 0, :, 12].double().cpu()
    assert torch.allclose(y[0, 0, :, 4].double().cpu(), direct, atol=2e-6)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_strides_and_in_place(dtype, interleaved):
    g = _gen(4)
    B, H, N, d = 2, 3, 40, 64
    table, pos = fa.rope_table(48, sections=[8, 16]), _pos(g, 2, B, N, 900)
    # heads behind tokens, as a projection leaves them, with other rows between
    wide = torch.randn(B, N, 2 * H + 1, d + 16, generator=g).to(dtype).cuda()
    x = wide[:, :, 1:1 + H, :d].transpose(1, 2)
    keep = wide.clone()
    out = torch.zeros(B, N, H, d, dtype=dtype, device="cuda").transpose(1, 2)
    y = fa.rope(x, pos, table, interleaved, out=out)
    _ok()
    assert y is out and torch.equal(wide, keep)
    _check(x, y, pos, table, interleaved)
    first = x.clone()
    assert fa.rope(x, pos, table, interleaved, out=x) is x
    _ok()
    assert torch.equal(x, y)
    _check(first, x, pos, table, interleaved)
    keep[:, :, 1:1 + H, :d] = wide[:, :, 1:1 + H, :d]
    assert torch.equal(wide, keep)                       # nothing beside the rows was touched
    # positions that all batches share, and one row for all heads
    same = pos[:, :1].expand(2, B, N)
    one = first[:, :1].expand(B, H, N, d)
    _check(one, fa.rope(one, same, table, interleaved), same, table, interleaved)


def test_rope_of_latent_queries_and_keys():
    # the last 64 of a head's 192 columns, in place, and the keys' part that all heads share
    g = _gen(5)
    q = torch.randn(2, 4, 30, 192, generator=g).bfloat16().cuda()
    k_rope = torch.randn(2, 30, 64, generator=g).bfloat16().cuda()
    table, pos = fa.rope_table(64), torch.arange(30, dtype=I32, device="cuda").expand(1, 2, 30)
    keep, part = q.clone(), q[..., 128:]
    fa.rope(part, pos, table, out=part)
    kr = fa.rope(k_rope[:, None], pos, table)
    _ok()
    assert torch.equal(q[..., :128], keep[..., :128])
    _check(keep[..., 128:], part, pos, table)
    _check(k_rope[:, None], kr, pos, table)


def test_rope_carries_infinities_and_nan_in_their_pairs():
    x = torch.ones(1, 1, 3, 32, device="cuda")
    x[0, 0, 1, 3], x[0, 0, 2, 20] = float("nan"), float("inf")
    pos = torch.tensor([[[1, 2, 5]]], dtype=I32, device="cuda")
    y = fa.rope(x, pos, fa.rope_table(32))
    _ok()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, 1, 3] = want[0, 0, 1, 19] = want[0, 0, 2, 4] = want[0, 0, 2, 20] = True
    assert torch.equal(bad, want)


def test_rope_past_32_bit_offsets():
    # 2.2 G elements; a few rows at either end are looked at
    H, N, d = 4200, 4096, 128
    x = torch.ones(1, H, N, d, dtype=BF, device="cuda")
    x[0, -1, -3:] = torch.arange(d, device="cuda").bfloat16() / 64
    pos = torch.arange(N, dtype=I32, device="cuda")[None, None]
    table = fa.rope_table(d)
    rows = x[:, -1:, -4:].clone()
    fa.rope(x, pos, table, out=x)
    _ok()
    _check(rows, x[:, -1:, -4:], pos[..., -4:], table)
    _check(torch.ones(1, 1, 4, d, dtype=BF, device="cuda"), x[:, 4100:4101, :4], pos[..., :4], table)


def test_rope_on_a_named_stream():
    g = _gen(6)
    s = torch.cuda.Stream()
    pos = torch.arange(500, dtype=I32, device="cuda")[None, None]
    x = torch.randn(1, 8, 500, 128, generator=g).bfloat16().cuda()
    table = fa.rope_table(128)
    want = fa.rope(x, pos, table)
    s.wait_stream(torch.cuda.current_stream())
    y = fa.rope(x, pos, table, stream=s)
    back = fa.rope_backward(y, pos, table, stream=s.cuda_stream)
    s.synchronize()
    _ok()
    assert torch.equal(y, want)
    _check(y, back, pos, table, inverse=True)


# ------------------------------------------------------------------ into the cache

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,axes,page", [
    (1, 1, 1, 64, 64, 1, 16), (7, 6, 2, 128, 128, 3, 32), (300, 8, 8, 64, 48, 2, 16),
    (65, 12, 3, 128, 64, 1, 256), (33, 5, 5, 128, 112, 1, 64),
])
def test_rope_append(T, Hq, Hkv, d, rot, axes, page, interleaved):
    g = _gen(T + d)
    P = -(-T // page) + 3
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv.split((Hq, Hkv, Hkv), 1)
    kc, vc = (torch.randn(P, Hkv, page, d, generator=g).bfloat16().cuda() for _ in range(2))
    k0, v0, keep = _np(kc), _np(vc), qkv.clone()
    slots = torch.randperm(P * page, generator=g)[:T].int()
    if T > 3:
        slots[1], slots[2], slots[3] = -1, P * page, 2 ** 31 - 1
    pairs = rot // 2
    table = fa.rope_table(rot, sections=[pairs // axes] * (axes - 1) + [pairs - pairs // axes * (axes - 1)])
    pos = torch.randint(0, 100000, (axes, T), generator=g, dtype=I32).cuda()
    out = fa.rope_append(q, k, v, pos, table, kc, vc, slots.cuda(), interleaved)
    _ok()
    assert torch.equal(qkv, keep)
    turns, axis = _ints(table)
    at = pos.cpu().numpy()[:, :, None]
    ref, size = rope.rotate(_np(q), at, turns, axis, interleaved)
    _close(_np(out), ref, size, BF)
    ref, size = rope.rotate(_np(k), at, turns, axis, interleaved)
    s = slots.tolist()
    ref, size = paged.append(k0, ref, s), paged.append(np.zeros_like(k0), size, s)
    touched = paged.append(np.zeros_like(k0), np.ones_like(_np(k)), s)
    assert np.array_equal(_np(kc)[touched == 0], k0[touched == 0])
    _close(_np(kc), ref, size, BF)
    assert np.array_equal(_np(vc), paged.append(v0, _np(v), s))
    # in place of the queries, and as rope and append one after the other
    k1, v1 = torch.from_numpy(k0).bfloat16().cuda(), torch.from_numpy(v0).bfloat16().cuda()
    alone = fa.rope(k.transpose(0, 1)[None], pos[:, None], table, interleaved)[0].transpose(0, 1)
    fa.paged_append(alone.contiguous(), v, k1, v1, slots.cuda())
    assert fa.rope_append(q, k, v, pos, table, kc, vc, slots.cuda(), interleaved, out=q) is q
    _ok()
    assert torch.equal(q, out) and torch.equal(kc, k1) and torch.equal(vc, v1)
    keep[:, :Hq] = qkv[:, :Hq]
    assert torch.equal(qkv, keep)


def test_rope_append_of_nothing_and_strided_pages():
    g = _gen(8)
    table = fa.rope_table(64)
    both = torch.zeros(4, 2, 2, 16, 64, dtype=BF, device="cuda")
    none = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    slots = torch.empty(0, dtype=I32, device="cuda")
    out = fa.rope_append(none, none[:, :2], none[:, :2], torch.empty(1, 0, dtype=I32, device="cuda"),
                         table, both[:, 0], both[:, 1], slots)
    assert out.shape == (0, 4, 64)
    q, k, v = (torch.randn(5, h, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    slots = torch.tensor([63, 0, 17, 40, 5], dtype=I32, device="cuda")
    pos = torch.zeros(1, 5, dtype=I32, device="cuda")             # no turn: the rows as they are
    out = fa.rope_append(q, k, v, pos, table, both[:, 0], both[:, 1], slots)
    _ok()
    zero = np.zeros((4, 2, 16, 64))
    assert torch.equal(out, q)
    assert np.array_equal(_np(both[:, 0]), paged.append(zero, _np(k), slots.tolist()))
    assert np.array_equal(_np(both[:, 1]), paged.append(zero, _np(v), slots.tolist()))
