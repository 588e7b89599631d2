"""What pins the 64-bit implementations of the layer operators (CPU): closed
forms, central differences, and facts outside the formulas."""

import numpy as np
import pytest

from oracle import layer


def _differences(f, x, step=1e-6):
    """Central differences of a scalar function of an array."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n_rot", [0, 4, 6])
def test_norm_rope_gradients(interleaved, n_rot):
    rng = np.random.default_rng(n_rot)
    x, dy, w = rng.standard_normal((3, 2, 6)), rng.standard_normal((3, 2, 6)), rng.standard_normal(6)
    pos, freqs = np.array([0, 7, -3]), np.array([1.0, 0.3, 0.01])[:n_rot // 2]

    def loss(x, w):
        return float((layer.norm_rope(x, w, pos, freqs, 1e-3, interleaved) * dy).sum())

    dx, dw = layer.norm_rope_back(dy, x, w, pos, freqs, 1e-3, interleaved)
    assert np.allclose(dx, _differences(lambda v: loss(v, w), x), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: loss(x, v), w), atol=1e-7)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_distance_alone(interleaved):
    """The product of a rotated query and key is a function of the difference of their positions."""
    rng = np.random.default_rng(1)
    q, k, freqs = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), np.array([1.0, 0.5, 0.2, 0.01])

    def score(a, b):
        return float((layer.turned(q, [a], freqs, interleaved) * layer.turned(k, [b], freqs, interleaved)).sum())

    assert abs(score(5, 2) - score(1005, 1002)) < 1e-9 and abs(score(5, 2) - score(2, 5)) > 1e-3
    # a quarter turn of one pair: (a, b) becomes (-b, a)
    y = layer.turned(q, [1], np.array([np.pi / 2, 0, 0, 0]), interleaved)
    a, b = (0, 1) if interleaved else (0, 4)
    assert np.allclose([y[0, 0, a], y[0, 0, b]], [-q[0, 0, b], q[0, 0, a]])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((2, 3, 16)) * 7
    y = layer.norm_rope(x, None, [4, 9], np.array([0.1, 0.2]), 0.0, False)
    assert np.allclose((y * y).mean(-1), 1.0)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh", "gelu_erf", "relu"])
def test_activations(kind):
    v = np.array([-30.0, -5.0, -1.3, -0.2, 0.4, 1.0, 6.0, 40.0])
    d = np.array([(layer.act(v + 1e-6, kind) - layer.act(v - 1e-6, kind)) / 2e-6])[0]
    assert np.allclose(layer.act_slope(v, kind), d, atol=1e-6)
    assert np.allclose(layer.act(v[-1:], kind), 40.0) and abs(layer.act(v[:1], kind)[0]) < 1e-8
    known = {"silu": 0.7310585786300049, "gelu_erf": 0.8413447460685429, "gelu_tanh": 0.8411919906082768, "relu": 1.0}
    assert abs(layer.act(np.array([1.0]), kind)[0] - known[kind]) < 1e-12


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_ffn_gradients(kind):
    rng = np.random.default_rng(3)
    x, wg, wu, dh = (rng.standard_normal(s) for s in ((3, 4), (5, 4), (5, 4), (3, 5)))

    def loss(x, wg, wu):
        return float((layer.gated_ffn(x, wg, wu, kind)[0] * dh).sum())

    _, gate, up = layer.gated_ffn(x, wg, wu, kind)
    dx, dwg, dwu, _, _ = layer.gated_ffn_back(dh, x, wg, wu, gate, up, kind)
    assert np.allclose(dx, _differences(lambda v: loss(v, wg, wu), x), atol=1e-6)
    assert np.allclose(dwg, _differences(lambda v: loss(x, v, wu), wg), atol=1e-6)
    assert np.allclose(dwu, _differences(lambda v: loss(x, wg, v), wu), atol=1e-6)


@pytest.mark.parametrize("shape", [(3, 5), (5, 3), (4, 4), (1, 7)])
def test_orthogonalise_acts_on_singular_values(shape):
    """The steps are an odd polynomial of the singular values and leave the singular vectors."""
    x = np.random.default_rng(4).standard_normal(shape)
    coefs = [(3.4445, -4.7750, 2.0315)] * 5
    u, s, vt = np.linalg.svd(x, full_matrices=False)
    s = s / np.sqrt((s * s).sum())
    for a, b, c in coefs:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(layer.orthogonalise(x, 5, coefs, 0.0, 2.0), 2.0 * (u * s) @ vt)
    # with the coefficients that converge it gives the nearest orthogonal matrix
    near = layer.orthogonalise(x, 30, [(1.875, -1.25, 0.375)] * 30, 0.0)
    assert np.allclose(near, u @ vt, atol=1e-9)
