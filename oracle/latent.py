"""CPU fp64 oracle for latent attention, in the expanded and the absorbed form.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or execute this
module.  It shares no code with the CUDA path and imports nothing from the package.

Expanded: head h has keys (k_nope_h, k_rope), k_rope shared by the heads, and is otherwise the
plain attention of ``attention.py`` with 192 key columns and 128 value columns; the gradient of
the shared part is the sum over the heads.  Absorbed: a cached row is (c, r); the scores are
q . (c, r) and the values are c.

Besides the results the functions return what their rounding errors are measured against: the
sums of the absolute terms (see ``tests/_latent_bound.py``).
"""
from __future__ import annotations

import numpy as np

from .attention import backward_head, forward_head, keep_mask
from .paged import decode as paged_decode


def _keys(k_nope, k_rope, b, h):
    return np.concatenate([np.asarray(k_nope[b, h], np.float64),
                           np.asarray(k_rope[b], np.float64)], axis=1)


def _masked(x, n):
    """x with the rows from n on set to 0: what they hold belongs to no result."""
    x = np.array(x, np.float64)
    x[n:] = 0.0
    return x


def forward(q, k_nope, k_rope, v, scale: float, causal=False, kv_len=None):
    """Returns (o, lse, spread), spread = sum_j p_j |v_j|."""
    B, H, N, _ = q.shape
    o, lse = np.zeros(v.shape), np.zeros((B, H, N))
    spread = np.zeros(v.shape)
    for b in range(B):
        n = N if kv_len is None else max(0, min(int(kv_len[b]), N))
        keep = keep_mask(N, causal, None, n)
        for h in range(H):
            k, vv = _masked(_keys(k_nope, k_rope, b, h), n), _masked(v[b, h], n)
            o[b, h], lse[b, h], p = forward_head(q[b, h], k, vv, scale, keep)
            spread[b, h] = p @ np.abs(vv)
    return o, lse, spread


def backward(q, k_nope, k_rope, v, do, scale: float, causal=False, kv_len=None, u=0.0, g=0.0):
    """Returns ((dq, dk_nope, dk_rope, dv), errors): errors has the same shapes and bounds what a
    relative error u of each P and dS operand and g of the fp32 steps before them can move."""
    B, H, N, _ = q.shape
    nope = k_nope.shape[-1]
    out = [np.zeros(x.shape) for x in (q, k_nope, k_rope, v)]
    err = [np.zeros(x.shape) for x in (q, k_nope, k_rope, v)]
    for b in range(B):
        n = N if kv_len is None else max(0, min(int(kv_len[b]), N))
        keep = keep_mask(N, causal, None, n)
        for h in range(H):
            k, vv = _masked(_keys(k_nope, k_rope, b, h), n), _masked(v[b, h], n)
            qq, dd = np.asarray(q[b, h], np.float64), np.asarray(do[b, h], np.float64)
            dq, dk, dv, _ = backward_head(qq, k, vv, dd, scale, keep)
            out[0][b, h], out[1][b, h], out[3][b, h] = dq, dk[:, :nope], dv
            out[2][b] += dk[:, nope:]
            o, _, p = forward_head(qq, k, vv, scale, keep)
            dp, D = dd @ vv.T, (dd * o).sum(1, keepdims=True)
            e_ds = u * p * np.abs(dp - D) + g * p * (np.abs(dd) @ np.abs(vv).T +
                                                     (np.abs(dd) * np.abs(o)).sum(1, keepdims=True))
            e_dk = scale * e_ds.T @ np.abs(qq)
            err[0][b, h] = scale * e_ds @ np.abs(k)
            err[1][b, h] = e_dk[:, :nope]
            err[2][b] += e_dk[:, nope:]
            err[3][b, h] = (u + g) * p.T @ np.abs(dd)
    return out, err


def decode(q, cache, table, cache_len, scale: float, rank: int):
    """q [B, H, row] over a pool cache [P, page, row].  Returns (o, lse, spread)."""
    c = np.asarray(cache)[:, None]                     # one key/value head for all queries
    return paged_decode(q, c, c[..., :rank], table, cache_len, scale)
