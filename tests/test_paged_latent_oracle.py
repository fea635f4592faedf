"""Pins of the paged and latent oracles (CPU): each reaches the result by another route."""
import numpy as np
import pytest

import oracle
from oracle import latent, paged

RNG = np.random.default_rng(11)


def _rand(*shape):
    return RNG.standard_normal(shape)


def _pool(x, page, spare, rng):
    """A contiguous cache [B, Hkv, L, d] scattered into pages; returns (pool, table)."""
    B, Hkv, L, d = x.shape
    M = -(-L // page)
    ids = rng.permutation(B * M + spare)[:B * M].reshape(B, M)
    pool = np.full((B * M + spare, Hkv, page, d), np.nan)
    for b in range(B):
        for i in range(M):
            rows = x[b, :, i * page:(i + 1) * page]
            pool[ids[b, i], :, :rows.shape[1]] = rows
    return pool, ids


@pytest.mark.parametrize("page", [2, 3, 16])
def test_paged_decode_is_the_contiguous_decode(page):
    B, Hq, Hkv, L, d = 3, 6, 2, 17, 4
    q, k, v = _rand(B, Hq, d), _rand(B, Hkv, L, d), _rand(B, Hkv, L, d)
    lens = np.array([17, 5, 0])
    rng = np.random.default_rng(page)
    kp, table = _pool(k, page, 2, rng)
    rng = np.random.default_rng(page)
    vp, _ = _pool(v, page, 2, rng)
    o, lse, _ = paged.decode(q, kp, vp, table, lens, 0.4)
    ro, rlse = oracle.decode(q, k, v, 0.4, lens)
    np.testing.assert_allclose(o, ro, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, rlse, rtol=1e-12)


def test_holes_hide_their_keys():
    q, k, v = _rand(1, 1, 4), _rand(3, 1, 2, 4), _rand(3, 1, 2, 4)
    o, lse, _ = paged.decode(q, k, v, np.array([[2, -1, 0, 9]]), np.array([7]), 0.5)
    ro, rlse = oracle.decode(q, k[[2, 0]].transpose(1, 0, 2, 3).reshape(1, 1, 4, 4),
                             v[[2, 0]].transpose(1, 0, 2, 3).reshape(1, 1, 4, 4), 0.5)
    np.testing.assert_allclose(o, ro, rtol=1e-12)
    np.testing.assert_allclose(lse, rlse, rtol=1e-12)


def test_tables_by_hand():
    table = np.array([[7, -1, -1], [3, 4, -1], [-1, -1, -1]])
    t, total, start, slots, taken = paged.tables([3, 8, 0], [2, 0, 5], [9, 1, 2], table, 4, 12, 9)
    assert t.tolist() == [[7, 9, -1], [3, 4, -1], [1, 2, -1]] and taken == 3
    assert total.tolist() == [5, 8, 5] and start.tolist() == [0, 2, 2, 7]
    assert slots.tolist() == [31, 36, 4, 5, 6, 7, 8, -1, -1]
    # a list that runs out leaves holes; a full row takes no more
    t, total, start, slots, taken = paged.tables([4, 11], [9, 9], [5], table[:2], 4, 12, 9)
    assert t.tolist() == [[7, 5, -1], [3, 4, -1]] and taken == 2
    assert total.tolist() == [12, 12] and slots.tolist() == [20, 21, 22, 23, -1, -1, -1, -1, -1]


def test_append_then_decode_sees_the_rows():
    cache = np.zeros((3, 2, 4, 5))
    rows = _rand(3, 2, 5)
    out = paged.append(cache, rows, [9, -1, 0])
    np.testing.assert_array_equal(out[2, :, 1], rows[0])
    np.testing.assert_array_equal(out[0, :, 0], rows[2])
    assert np.count_nonzero(out) == 2 * 2 * 5


def test_expanded_is_attention_with_the_shared_key_repeated():
    B, H, N = 2, 3, 7
    q, kn, kr, v = _rand(B, H, N, 6), _rand(B, H, N, 4), _rand(B, N, 2), _rand(B, H, N, 5)
    k = np.concatenate([kn, np.repeat(kr[:, None], H, 1)], -1)
    for causal, kv in ((False, None), (True, [7, 3])):
        o, lse, _ = latent.forward(q, kn, kr, v, 0.3, causal, kv)
        ro, rlse = oracle.forward(q, k, v, 0.3, causal, None, kv)
        np.testing.assert_allclose(o, ro, rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(lse, rlse, rtol=1e-12)


def test_gradients_by_central_differences():
    B, H, N = 1, 2, 5
    x = [_rand(B, H, N, 6), _rand(B, H, N, 4), _rand(B, N, 2), _rand(B, H, N, 3)]
    do = _rand(B, H, N, 3)
    kv = [4]
    grads, _ = latent.backward(*x, do, 0.7, True, kv)
    eps = 1e-6
    for i in range(4):
        for at in np.ndindex(x[i].shape):
            lo, hi = [a.copy() for a in x], [a.copy() for a in x]
            lo[i][at] -= eps
            hi[i][at] += eps
            f = [float((latent.forward(*y, 0.7, True, kv)[0] * do).sum()) for y in (lo, hi)]
            assert abs((f[1] - f[0]) / (2 * eps) - grads[i][at]) < 1e-7


def test_absorbed_is_the_expanded_forms_last_row():
    # k_nope_h = c W_k,h and v_h = c W_v,h: the absorbed query is q_nope W_k,h^T, and the output
    # before the value projection gives the head's output after it.
    H, N, R, nope, rope, dv, page = 3, 9, 8, 4, 2, 5, 4
    c, r = _rand(N, R), _rand(N, rope)
    wk, wv = _rand(H, R, nope), _rand(H, R, dv)
    q = _rand(1, H, N, nope + rope)
    kn, v = np.einsum("nr,hrd->hnd", c, wk)[None], np.einsum("nr,hrd->hnd", c, wv)[None]
    o, lse, _ = latent.forward(q, kn, r[None], v, 0.6, True)
    qa = np.concatenate([np.einsum("hd,hrd->hr", q[0, :, -1, :nope], wk), q[0, :, -1, nope:]], -1)
    pool, table = _pool(np.concatenate([c, r], -1)[None, None], page, 1, np.random.default_rng(0))
    ol, lsel, _ = latent.decode(qa[None], pool[:, 0], table, np.array([N]), 0.6, R)
    np.testing.assert_allclose(np.einsum("hr,hrd->hd", ol[0], wv), o[0, :, -1], rtol=1e-10)
    np.testing.assert_allclose(lsel[0], lse[0, :, -1], rtol=1e-10)
