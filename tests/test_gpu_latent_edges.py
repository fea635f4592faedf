"""Latent attention on the GPU where its other tests do not reach: few visible keys anywhere in a
sequence, several groups of heads, tensors and pools past 2^31 elements, NaN in a query."""
import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import latent

from _latent_bound import G, TINY, U, check_grads, check_lse, check_o
from test_gpu_latent import DT, SCALE, _check_decode, _decode_case, _inputs
from test_gpu_paged import _gen, _i32, _np, _ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n", [1, 2, 8, 100, 128])
def test_queries_of_few_keys_carry_one_rounding_wherever_they_are(n, causal):
    # A query that sees at most 128 keys has its dS in two bf16 terms, be it the mask or the length
    # that leaves so few, so a row of its dq (192 values) carries the result's rounding alone: off by
    # h / sqrt(3) of its norm in the mean, h = 2^-8, and 192 values move that by 1 / sqrt(5 192) of
    # it; five times that is allowed.  (With one rounding of dS one row in thirteen over two keys is
    # off by more than 0.85 h.)  On top what the steps before leave: 2^-16 of dS for the second
    # term's rounding, 2^-13 for P (its score is a sum of 192 products, with 2^-24 each), and 192
    # 2^-24 < 2^-16 of the terms of dP and D.  D is that of the o_acc which the backward is given:
    # the forward's P is bf16, so D is off by up to h sum_j p_j |dP_j|, which where dP hardly differs
    # from key to key is many times h of dP - D.
    B, H, N = 2, 4, 300
    q, kn, kr, v, do = _inputs(B, H, N, "bf16", 40 + n, [n, n])
    kl = _i32([n, n])
    o, lse, o_acc = fa.latent_forward(q, kn, kr, v, causal, kl, need_grad=True)
    dq = _np(fa.latent_backward(q, kn, kr, v, o_acc, lse, do, causal, kl)[0])
    _ok()
    q, kn, kr, v, do, o_acc = (_np(t) for t in (q, kn, kr, v, do, o_acc))
    hidden = np.arange(n)[None] > np.arange(N)[:, None] if causal else np.zeros((N, n), bool)
    for b in range(B):
        for h in range(H):
            k, vv, d, oa = np.concatenate([kn[b, h], kr[b]], 1)[:n], v[b, h, :n], do[b, h], o_acc[b, h]
            s = np.where(hidden, -np.inf, q[b, h] @ k.T * SCALE)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            ds = p * (d @ vv.T - (d * oa).sum(1, keepdims=True))
            e_ds = (2.0 ** -16 + 2.0 ** -13) * np.abs(ds) + 2.0 ** -16 * p * (
                np.abs(d) @ np.abs(vv).T + (np.abs(d) * np.abs(oa)).sum(1, keepdims=True))
            ref, left = SCALE * ds @ k, SCALE * e_ds @ np.abs(k)
            off, size, left = (np.linalg.norm(x, axis=1) for x in (dq[b, h] - ref, ref, left))
            limit = 2.0 ** -8 / np.sqrt(3) * (1 + 5 / np.sqrt(5 * 192)) * size + left + TINY
            assert (off <= limit).all(), (off / limit).max()


def _step(x, causal):
    o, lse, o_acc = fa.latent_forward(*x[:4], causal, need_grad=True)
    grads = fa.latent_backward(*x[:4], o_acc, lse, x[4], causal)
    _ok()
    return (o, lse, o_acc) + grads


def _against_oracle(x, out, causal, dtype):
    host = [_np(t) for t in x]
    ro, rlse, spread = latent.forward(*host[:4], SCALE, causal)
    check_o(_np(out[0]), ro, spread, dtype)
    check_lse(_np(out[1]), rlse, dtype)
    u = U[dtype] if dtype == "bf16" else 0.0
    ref, err = latent.backward(*host, SCALE, causal, None, u, G[dtype])
    check_grads([_np(t) for t in out[3:]], ref, err, dtype)


@pytest.mark.parametrize("causal", [False, True])
def test_groups_of_heads_of_unequal_size(causal):
    # 645 heads of 257 rows: 323 and 322 of them in the forward's grid order, 408 and 237 in the
    # backward's.  Sequence by sequence they give the same bits, in one group each.
    x = _inputs(5, 129, 257, "bf16", 60)
    out = _step(x, causal)
    for b in range(5):
        alone = [t[b:b + 1] for t in x]
        for a, w in zip(_step(alone, causal), out):
            assert torch.equal(a, w[b:b + 1])
        if b in (2, 3):          # the groups end in these
            _against_oracle(alone, [t[b:b + 1] for t in out], causal, "bf16")


@pytest.mark.parametrize("dtype,B,H,N", [("bf16", 1000, 65, 260), ("fp32", 960, 62, 190)])
def test_tensors_past_32_bit_offsets(dtype, B, H, N):
    # q has 3.2 and 2.2 G elements.  All rows are 0 but those of the first and the last sequence.
    dt = DT[dtype]
    shapes = (B, H, N, 192), (B, H, N, 128), (B, N, 64), (B, H, N, 128), (B, H, N, 128)
    x = [torch.zeros(s, dtype=dt, device="cuda") for s in shapes]
    for i, b in enumerate((0, B - 1)):
        for t, w in zip(x, _inputs(1, H, N, dtype, 61 + i)):
            t[b] = w[0]
    out = _step(x, True)
    for b in (0, B - 1):
        _against_oracle([t[b:b + 1] for t in x], [t[b:b + 1] for t in out], True, dtype)
    for i in (0, 3, 4, 5, 6):
        assert not out[i][1:-1].any()
    seen = torch.arange(1, N + 1, device="cuda").log()
    assert (out[1][1:-1] - seen).abs().max() <= G[dtype] * (1 + seen[-1].item())


# ------------------------------------------------------------------ absorbed decode

@pytest.mark.parametrize("H", [16, 40])
def test_a_long_latent_cache_passes_32_bit_offsets(H):
    # 2.2 G elements: the last pages lie past 2^31 elements and 2^32 bytes
    P, page, T = 14700, 256, 700
    cache = torch.zeros(P, page, 576, dtype=torch.bfloat16, device="cuda")
    g = _gen(70)
    rows = torch.randn(T, 576, generator=g).bfloat16()
    table = _i32([[P - 1, 5, P - 2]])
    at = torch.arange(T)
    slots = (table[0].cpu()[at // page] * page + at % page).int()
    fa.latent_append(rows[:, :512].contiguous().cuda(), rows[:, 512:].contiguous().cuda(), cache,
                     slots.cuda())
    q = torch.randn(1, H, 576, generator=g).bfloat16().cuda()
    o, lse = fa.latent_decode(q, cache, table, _i32([T]))
    _ok()
    small = torch.zeros(3, page, 576, dtype=torch.bfloat16)
    small.view(-1, 576)[:T] = rows
    ro, rlse, spread = latent.decode(_np(q), _np(small), np.array([[0, 1, 2]]), [T], SCALE, 512)
    check_o(_np(o), ro, spread)
    check_lse(_np(lse), rlse)
    assert torch.equal(cache[table[0].long()].cpu(), small)
    assert cache.view(-1, 576)[::page].any(1).sum() == 3      # the rest is as it was


@pytest.mark.parametrize("H", [7, 16, 40, 128])
@pytest.mark.parametrize("lens", [[300, 200], [9000, 64]])
def test_decode_nan_queries_stay_in_their_heads(lens, H):
    x = _decode_case(lens, H, 16, seed=71)
    x[0][0, 3] = float("nan")
    o, lse = fa.latent_decode(*x)
    _ok()
    assert torch.isnan(o[0, 3].float()).all() and torch.isnan(lse[0, 3])
    x[0][0, 3] = 0
    ro, rl = _check_decode(x)
    keep = torch.ones(2, H, dtype=torch.bool)
    keep[0, 3] = False
    assert torch.equal(o[keep], ro[keep]) and torch.equal(lse[keep], rl[keep])
