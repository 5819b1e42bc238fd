"""Pins of oracle/expert_training.py: hand-made values, closed forms, brute force and differences."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import expert_training as T
from oracle.formats import E2M1_TABLE

RNG = np.random.default_rng(7)


def test_wgrad_by_loops():
    dy, x = RNG.standard_normal((7, 3)), RNG.standard_normal((7, 4))
    off = [0, 2, 2, 6]                                    # the last row belongs to nobody
    dw, mag = T.wgrad(dy, x, off)
    for e in range(3):
        for n in range(3):
            for k in range(4):
                terms = [Fraction(dy[r, n]) * Fraction(x[r, k]) for r in range(off[e], off[e + 1])]
                assert abs(dw[e, n, k] - float(sum(terms))) < 1e-14
                assert abs(mag[e, n, k] - float(sum(map(abs, terms)))) < 1e-14
    assert (dw[1] == 0).all()
    again, _ = T.wgrad(dy, x, off, dw)
    assert np.allclose(again, 2 * dw, atol=1e-15)


def test_wgrad_is_the_gradient():
    x, w, g = RNG.standard_normal((5, 4)), RNG.standard_normal((2, 3, 4)), RNG.standard_normal((5, 3))
    off = [0, 3, 5]

    def loss(w):
        return sum((x[off[e]:off[e + 1]] @ w[e].T * g[off[e]:off[e + 1]]).sum() for e in range(2))

    dw, _ = T.wgrad(g, x, off)
    for at in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[at] = 1e-3
        assert abs((loss(w + d) - loss(w - d)) / 2e-3 - dw[at]) < 1e-9


@pytest.mark.parametrize("off", [[0, 5, 3], [-1, 2, 3], [0, 2, 9]])
def test_wgrad_bad_offsets_have_no_rows(off):
    dw, _ = T.wgrad(np.ones((5, 2)), np.ones((5, 2)), off)
    assert ((dw == 0).all(axis=(1, 2)) == [not (0 <= a <= b <= 5) or a == b
                                           for a, b in zip(off, off[1:])]).all()


def test_weight_exponent_borders():
    for e in range(-126, 120, 7):
        assert T.weight_exponent(6.0 * 2.0 ** e) == e
        assert T.weight_exponent(np.nextafter(6.0 * 2.0 ** e, np.inf)) == e + 1
        assert T.weight_exponent(3.0 * 2.0 ** e) == e - 1
    assert T.weight_exponent(0.0) == 0 and T.weight_exponent(1e-45) == -127


def test_e2m1_ties_and_neighbours():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for mid, code in ties.items():
        assert T.e2m1_rne(np.array([mid, -mid])).tolist() == [code, code | 8]
        lo, hi = np.nextafter(mid, 0), np.nextafter(mid, 9)
        a, b = T.e2m1_rne(np.array([lo, hi]))
        assert b == a + 1 and E2M1_TABLE[a] < mid < E2M1_TABLE[b]
    assert T.e2m1_rne(E2M1_TABLE[:8]).tolist() == list(range(8))


def test_quantize_weights_against_the_generator():
    from synth import quantize_weights
    import torch
    w = RNG.standard_normal((2, 6, 96)).astype(np.float32)
    w[0, 0, :32] = 0
    q, s = T.quantize_weights(w)
    p, t = quantize_weights(torch.from_numpy(w))
    assert (q == p.numpy()).all() and (s == t.numpy()).all()


def test_quantize_weights_not_finite_and_back():
    w = np.ones((1, 64))
    w[0, 3] = np.inf
    q, s = T.quantize_weights(w)
    assert s.tolist() == [[255, 125]] and (q[0, :16] == 0).all()       # 1 = 4 * 2^-2
    back = T.dequantize_weights(q, s)
    assert np.isnan(back[0, :32]).all() and (back[0, 32:] == 1).all()


def test_rmsnorm_closed_forms():
    s, r, v = T.rmsnorm(np.array([[3.0, -4.0]]), None, np.array([1.0, 2.0]), 0.5)
    assert r[0] == 1 / np.sqrt(13.0) and np.allclose(v, [[3 * r[0], -8 * r[0]]], rtol=1e-15)
    s, r, v = T.rmsnorm(np.array([[1.0, 256.0]]), np.array([[2.0 ** -9, 1.0]]), np.ones(2), 0.0)
    assert s.tolist() == [[1.0, 256.0]]                    # 257 is between 256 and 258, a tie
    assert T.rmsnorm(np.zeros((1, 8)), None, np.ones(8), 1e-6)[2].tolist() == [[0.0] * 8]


def test_rmsnorm_bwd_by_differences():
    x, g, dy = RNG.standard_normal((2, 6)), RNG.standard_normal(6), RNG.standard_normal((2, 6))
    dsum = RNG.standard_normal((2, 6))

    def loss(x, g):
        s, _, v = T.rmsnorm(x, None, g, 0.1)
        return (v * dy).sum() + (s * dsum).sum()

    s, r, _ = T.rmsnorm(x, None, g, 0.1)
    dx, dg, _, _ = T.rmsnorm_bwd(dy, s, g, r, dsum)
    for at in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[at] = 1e-4
        assert abs((loss(x + d, g) - loss(x - d, g)) / 2e-4 - dx[at]) < 1e-6
    for i in range(6):
        d = np.zeros(6)
        d[i] = 1e-4
        assert abs((loss(x, g + d) - loss(x, g - d)) / 2e-4 - dg[i]) < 1e-8


def test_dispatch_acts():
    a = np.arange(256, dtype=np.uint8).reshape(2, 128)
    rows, sc = T.dispatch_acts(a, np.array([[7], [9]]), np.array([[2, -1], [0, 4]]),
                               np.full((4, 128), 5, np.uint8), np.full((4, 1), 1, np.uint8))
    assert (rows[2] == a[0]).all() and (rows[0] == a[1]).all()
    assert sc.ravel().tolist() == [9, 1, 7, 1] and (rows[[1, 3]] == 5).all()
