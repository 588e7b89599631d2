"""Pins of the 64-bit implementations of the training operators (CPU): facts
they do not share code with -- published generator outputs, closed forms, and
central differences of the forward passes."""

import numpy as np
import pytest

import synth
from oracle import training as tr


@pytest.mark.parametrize("counter,key,want", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator_known_answers(counter, key, want):
    """The generator's published known-answer vectors."""
    assert tr.philox4x32_10(counter, key) == want


def test_dropout_rate_and_mean():
    """16-bit uniforms: the kept share of 40,000 elements is within five standard
    deviations of 1 - p, and p = 0 / p = 1 keep and drop everything."""
    n = 200 * 200
    for p in (0.05, 0.5, 0.9):
        keep = tr.dropout_keep(200, 200, p, 12345678901234567, 99)
        assert abs(keep.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)
    x = np.ones((3, 11))
    assert (tr.dropout(x, 0.0, 1, 2) == 1).all() and (tr.dropout(x, 1.0, 1, 2) == 0).all()


def test_get_rows_gradient_is_the_adjoint():
    """<get_rows(W), dy> == <W, get_rows_back(dy)> for any W and dy."""
    rng = np.random.default_rng(3)
    W, dy = rng.standard_normal((13, 6)), rng.standard_normal((40, 6))
    ids = rng.integers(0, 13, 40)
    d, mag, count = tr.get_rows_back(dy, ids, 13, 2.5)
    assert np.isclose((tr.get_rows(W, ids, 2.5) * dy).sum(), (W * d).sum(), rtol=1e-12)
    assert count.sum() == 40 and (mag >= np.abs(d) - 1e-12).all()


def test_table_values_match_the_quantiser():
    w = synth.normal(5, 7 * 256, std=0.02).reshape(7, 256)
    for kind in (synth.TYPE_Q8_0, synth.TYPE_Q4_K):
        v = tr.table_values(synth.quantize(kind, w).reshape(7, -1), kind, 256)
        assert np.abs(v - w).max() < 0.02


def _central(f, x, h):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_layer_norm_gradient_by_differences():
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((3, 7)) * 2 + 5, rng.standard_normal((3, 7))
    w, b, eps = rng.standard_normal(7), rng.standard_normal(7), 1e-3
    y, mean, rstd = tr.layer_norm(x, w, b, eps)
    dx, dw, db = tr.layer_norm_back(dy, x, mean, rstd, w)
    # central differences, step 1e-5: error O(h^2) ~ 1e-10 and 1e-16 / h ~ 1e-11
    assert np.allclose(dx, _central(lambda v: (tr.layer_norm(v, w, b, eps)[0] * dy).sum(), x, 1e-5), atol=1e-7)
    assert np.allclose(dw, _central(lambda v: (tr.layer_norm(x, v, b, eps)[0] * dy).sum(), w, 1e-5), atol=1e-7)
    assert np.allclose(db, _central(lambda v: (tr.layer_norm(x, w, v, eps)[0] * dy).sum(), b, 1e-5), atol=1e-7)


def test_layer_norm_of_a_constant_row():
    y, mean, rstd = tr.layer_norm(np.full((1, 5), 3.0), None, None, 0.25)
    assert (y == 0).all() and mean[0] == 3.0 and rstd[0] == 2.0


@pytest.mark.parametrize("e", [0.0, 0.1])
def test_preference_gradient_by_differences(e):
    rng = np.random.default_rng(5)
    x, ref = rng.standard_normal((9, 6)) * 2, rng.standard_normal(9)
    labels = np.array([-1, 2, 5, 0, -1, 1, 3, 3, 4])
    seq = np.array([0, 3, 5, 5, 8])            # two pairs; the third sequence is empty, row 8 in none
    loss, losses, ratios, logps, lse = tr.preference_loss(x, labels, seq, ref, 0.7, e)
    d, coef = tr.preference_loss_back(x, labels, seq, lse, ratios, 0.7, e, dloss=1.5)
    want = _central(lambda v: 1.5 * tr.preference_loss(v, labels, seq, ref, 0.7, e)[0], x, 1e-5)
    assert np.allclose(d, want, atol=1e-8)
    assert (d[[0, 4, 8]] == 0).all() and ratios[2] == 0.0
    assert np.allclose(d.sum(1), 0.0, atol=1e-15)      # a softmax row's gradient sums to zero


def test_preference_loss_closed_forms():
    """Equal ratios: log 2 whatever the smoothing; V = 1: every logp is 0."""
    x = np.zeros((2, 4))
    loss = tr.preference_loss(x, np.array([1, 2]), np.array([0, 1, 2]), None, 0.3, 0.2)[0]
    assert np.isclose(loss, np.log(2.0), rtol=1e-14)
    assert (tr.preference_loss(np.ones((2, 1)), np.zeros(2, int), np.array([0, 1, 2]), None, 1.0, 0.0)[3] == 0).all()
