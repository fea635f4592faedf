"""Error bounds of the paged and latent kernels, element by element.

A weight p_j enters P V as one rounding of its fp32 value (relative error U[dtype], half a step),
o is rounded once more, and the fp32 steps before (scores, exponentials, sums, the rescaling)
are off by a relative G of each term:
    |o - o_ref|   <= (u + g) sum_j p_j |v_j| + u |o_ref| + tiny
    |dX - dX_ref| <= err + u |dX_ref| + tiny,  err from oracle.latent.backward (u on P and dS, g on
                     dP, D and P), for the shared k_rope summed over the heads
    |lse - ref|   <= g (1 + |lse_ref|)
G: a score is a sum of at most 576 fp32 products, so it is off by at most 576 * 2^-24 of the sum
of their absolute values (below 64 for the standard normal inputs used here, after the scale).
That would be 0.0022 with every error at its largest and of one sign; being of either sign they
add up to some sqrt(576) 2^-24 of the sum, 0.0001.  G = 2^-10 is ten times that, which leaves
room for the exponent (2^-22), the sums over up to 1000 keys (1000 * 2^-24) and lse's own
rounding.  For fp32 the operands are not rounded: u = 2^-24 for the result, g = 2^-13.
"""
import numpy as np

U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
G = {"bf16": 2.0 ** -10, "fp32": 2.0 ** -13}
TINY = 1e-6


def check_o(o, ref, spread, dtype="bf16"):
    u, g = U[dtype], G[dtype]
    bound = (u + g) * spread + u * np.abs(ref) + TINY
    worst = np.max(np.abs(o - ref) / bound)
    assert worst <= 1.0, f"o is off by {worst:.2f} of its bound"


def check_lse(lse, ref, dtype="bf16"):
    dead = np.isneginf(ref)
    assert np.array_equal(np.isneginf(lse), dead), "rows without a visible key differ"
    assert np.all(np.isfinite(lse[~dead]))
    if (~dead).any():
        bound = G[dtype] * (1 + np.abs(ref[~dead]))
        worst = np.max(np.abs(lse[~dead] - ref[~dead]) / bound)
        assert worst <= 1.0, f"lse is off by {worst:.2f} of its bound"


def check_grads(got, ref, err, dtype="bf16"):
    for name, x, r, e in zip(("dq", "dk_nope", "dk_rope", "dv"), got, ref, err):
        assert np.all(np.isfinite(x)), name
        worst = np.max(np.abs(x - r) / (e + U[dtype] * np.abs(r) + TINY))
        assert worst <= 1.0, f"{name} is off by {worst:.2f} of its bound"
