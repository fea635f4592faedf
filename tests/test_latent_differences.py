"""Gradients of latent attention against differences of its forward: the oracle's in fp64 (CPU), which
shows that the check fails for wrong gradients, and the fp32 kernels' (GPU)."""
import numpy as np
import pytest
import torch

from oracle import latent

SCALE = 192 ** -0.5
NAMES = ("dq", "dk_nope", "dk_rope", "dv")
B, H, N, LEN = 2, 2, 70, [70, 41]
E = 0.25
# A unit step along the gradient (its terms, weighted by positive numbers, are all of one sign, so that
# the derivative is as large as the sum of their absolute values).  What the quotient of differences
# is off by, for the sizes here: e^2 / 6 of the third derivative, 5e-5 of the derivative (measured in
# fp64), and the two losses' errors over 2 e: an fp32 loss sum_i do_i o_i with o off by 1e-6 of its
# norm is off by at most 1e-6 |do| |o| < 1e-6 190 70 = 0.014, two over 2 e by 0.054, which is 0.003
# of the smallest derivative, 18.
TOL = 2.0 ** -8


def _inputs():
    rng = np.random.default_rng(9)
    x = [rng.standard_normal(s).astype(np.float32).astype(np.float64) for s in (
        (B, H, N, 192), (B, H, N, 128), (B, N, 64), (B, H, N, 128), (B, H, N, 128))]
    return x[:4], x[4]


def _directions(causal):
    """(input, unit step) pairs along the oracle's gradients, and those gradients."""
    x, do = _inputs()
    ref, _ = latent.backward(*x, do, SCALE, causal, LEN)
    rng = np.random.default_rng(10)
    steps = []
    for i, r in enumerate(ref):
        for w in (1.0, rng.uniform(0, 2, r.shape), rng.uniform(0, 2, r.shape)):
            t = r * w
            steps.append((i, t / np.linalg.norm(t)))
    return x, do, steps, ref


def _quotient(loss, x, i, t):
    lo, hi = list(x), list(x)
    lo[i], hi[i] = x[i] - E * t, x[i] + E * t
    return (loss(hi) - loss(lo)) / (2 * E)


def _agrees(grad, t, quotient):
    return abs(np.sum(grad * t) - quotient) <= TOL * abs(quotient)


@pytest.mark.parametrize("causal", [False, True])
def test_wrong_gradients_fail_the_check(causal):
    x, do, steps, ref = _directions(causal)

    def loss(y):
        return (latent.forward(*y, SCALE, causal, LEN)[0] * do).sum()
    quotients = [_quotient(loss, x, i, t) for i, t in steps]
    assert min(quotients) >= 18

    def passes(n, grad):
        return all(_agrees(grad, t, f) for (i, t), f in zip(steps, quotients) if i == n)

    def without(g, *at):
        g = g.copy()
        g[at] = 0
        return g
    rest = slice(None)
    for n, g in enumerate(ref):
        assert passes(n, g), NAMES[n]
        wrong = [-g, 2 * g, g / 2, 1.01 * g, without(g, 0), without(g, rest, slice(1, None)),
                 without(g, ..., slice(0, 64)), without(g, ..., slice(-64, None)), np.roll(g, 1, -1),
                 without(g, rest, rest, slice(32, 64)) if g.ndim == 4 else np.roll(g, 1, 1)]
        for k, bad in enumerate(wrong):
            assert not passes(n, bad), (NAMES[n], k)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_fp32_gradients_against_differences_along_them(causal):
    from exact_io_aware_28_gb300 import fa
    x, do, steps, _ = _directions(causal)
    dev = [torch.from_numpy(a).float().cuda() for a in x]
    kl = torch.tensor(LEN, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(do).float().cuda()

    def loss(y):
        y = [torch.from_numpy(a).float().cuda() for a in y]
        return (fa.latent_forward(*y, causal, kl)[0].double() * g.double()).sum().item()
    o, lse, acc = fa.latent_forward(*dev, causal, kl, need_grad=True)
    grads = [t.double().cpu().numpy() for t in fa.latent_backward(*dev, acc, lse, g, causal, kl)]
    for i, t in steps:
        f = _quotient(loss, x, i, t)
        assert _agrees(grads[i], t, f), (NAMES[i], np.sum(grads[i] * t), f)
    torch.cuda.synchronize()
    assert fa.fa_device_error() == fa.FA_OK
