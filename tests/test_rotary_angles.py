"""Sines and cosines of rotary positions in binary32: their error is relative to
themselves, for every position and frequency, also next to their zeros."""
import math

import numpy as np
import pytest
import torch

from kv_ref import ints

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TABLES = [dict(), dict(base=1e6, scaling="yarn", factor=8.0, original=4096), dict(scaling="linear", factor=300.0),
          dict(frequencies=[math.pi * (1 + (i - 32) * 2.0 ** -33) for i in range(64)]),
          dict(frequencies=[math.pi / 2 * (1 + i * 2.0 ** -40) for i in range(64)]),
          dict(frequencies=[(-1) ** i * 2.0 ** -i for i in range(64)]), dict(frequencies=[0.0, -1.0, 1e-9, 2.0 ** -63] * 16)]


def positions():
    rng = np.random.default_rng(0)
    return [0, 1, 2, 3, 5, 1000, 65537, 2 ** 20, 2 ** 31 - 1, *rng.integers(0, 2 ** 31, 500).tolist(), *rng.integers(0, 100000, 500).tolist()]


def sines(at, table):
    """(cosines, sines) in 64 bits: position * turns modulo 2^64 in whole numbers, less
    its nearest quarters, of which the sine is taken."""
    c, n = (np.empty((len(at), len(table.frequencies))) for _ in range(2))
    turns = [t % 2 ** 64 for t in table.turns.tolist()]
    for r, p in enumerate(at):
        for i, t in enumerate(turns):
            angle = p * t % 2 ** 64
            quarter = (angle + 2 ** 61) // 2 ** 62
            x = (angle - quarter * 2 ** 62) * (2 * math.pi * 2.0 ** -64)
            u, v = math.cos(x), math.sin(x)
            c[r, i], n[r, i] = ((u, v), (-v, u), (-u, -v), (v, -u))[quarter % 4]
    return torch.from_numpy(c).cuda()[:, None], torch.from_numpy(n).cuda()[:, None]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim", [128, 130])
@pytest.mark.parametrize("which", range(len(TABLES)))
def test_angles(libgemm, which, dim, layout):
    """Of a head of 130 elements, whose rows no 16 bytes divide, one element a thread."""
    from accelerator_gb300 import sequences
    table, at = sequences.Rotary(128, layout=layout, **TABLES[which]), positions()
    where, m = ints(at), table.magnitude
    c, n = sines(at, table)

    def pairs(x):
        return (x[..., :64], x[..., 64:128]) if layout == "half" else (x[..., 0:128:2], x[..., 1:128:2])

    # (1, 0) becomes (cosine, sine) as they are, times the magnitude.  What is left of the
    # angle is off by E of itself, and a sine or cosine of up to an eighth of a turn by
    # that of itself or less, then by 2 units of its last place (2 E each).
    Q = torch.zeros(len(at), 2, dim, device="cuda")
    pairs(Q)[0].fill_(1.0)
    for inverse in (False, True):
        got = pairs(sequences.rotary(Q, None, where, table, inverse=inverse)[0])
        for x, want in zip(got, (c * m, (-n if inverse else n) * m)):
            limit = 5 * E + (E if m != 1.0 else 0.0)
            assert ((x.double() - want).abs() <= limit * want.abs() * (1 + 2.0 ** -20) + 2.0 ** -126).all()
    # any pair: a product and a sum more
    Q = torch.randn(len(at), 2, dim, device="cuda")
    a, b = (x.double() for x in pairs(Q))
    for x, u, v in zip(pairs(sequences.rotary(Q, None, where, table)[0]), (a * c, b * c), (-b * n, a * n)):
        want = (u + v) * m
        limit = 7 * E * (u.abs() + v.abs()) * m + E * want.abs()
        assert ((x.double() - want).abs() <= limit * (1 + 2.0 ** -20) + 2.0 ** -126).all()
    assert libgemm.debug_status() == libgemm.OK
