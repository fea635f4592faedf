"""CPU oracle for rotary positions.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or execute this module.
It shares no code with the CUDA path and imports nothing from the package.

A pair of channels is a complex number, which a position turns: z e^{2 pi i n t}, with t turns a
position given in units of 2^-64.  The angle is formed in whole numbers, modulo a turn, so that it
has no error of its own wherever the position is; sine and cosine of it are taken in fp64.
"""
from __future__ import annotations

import numpy as np


def angles(pos, turns, axis):
    """pos [axes, ...] integers, turns [pairs] integers, axis [pairs].  Returns [..., pairs]."""
    pos = np.asarray(pos)
    out = np.empty(pos.shape[1:] + (len(turns),))
    for i, (t, a) in enumerate(zip(turns, axis)):
        n = pos[min(max(int(a), 0), pos.shape[0] - 1)]
        flat = [((int(x) * int(t) + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 for x in n.flat]
        out[..., i] = 2.0 * np.pi * np.array(flat).reshape(n.shape)
    return out


def rotate(x, pos, turns, axis, interleaved=False, inverse=False):
    """x [..., d]; pos [axes, ...] over the same leading dimensions (or ones that broadcast).
    Returns (y, size): size is |x_1| + |x_2| of each pair, what an error of the angle is measured
    against; 0 for the channels that are not turned."""
    x = np.asarray(x, np.float64)
    pairs = len(turns)
    rot = 2 * pairs
    i = np.arange(pairs)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    w = np.exp((-1j if inverse else 1j) * angles(pos, turns, axis))
    z = (x[..., one] + 1j * x[..., two]) * w
    y, size = np.array(x), np.zeros_like(x)
    y[..., one], y[..., two] = z.real, z.imag
    size[..., one] = size[..., two] = np.abs(x[..., one]) + np.abs(x[..., two])
    assert rot <= x.shape[-1]
    return y, size
