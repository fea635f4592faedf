"""Latent attention on the GPU where its other tests do not reach: few visible keys anywhere in a
sequence."""
import numpy as np
import pytest

from exact_io_aware_28_gb300 import fa

from _latent_bound import TINY
from test_gpu_latent import SCALE, _inputs
from test_gpu_paged import _i32, _np, _ok

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
