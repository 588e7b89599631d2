"""GPU tests of the layer operators at the ends of their range and at the borders of their rules: values that
their intermediate steps could lose, coefficients and scales beyond the usual ones, one row, outliers.  Tolerances are
those of test_gpu_layer, or derived where they stand; all are written before any run."""

import numpy as np
import pytest

from oracle import layer
from test_gpu_layer import ACTS, FLOOR, PROD, TINY, U, UOUT, USUAL, _close, _dt, _np, _rand, _status, _y_tol, op  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# orthogonalised updates
# ---------------------------------------------------------------------------

def _growth(x, coefs, eps=1e-7):
    """How far an error of 1 of each X_s relative to its norm (at least 1) reaches in the result, summed over the steps.
    A step maps every singular value t to p(t) = t (a + b t^2 + c t^4); to first order the part of an error between two
    singular vectors grows by a difference quotient of p at their values, (p(t) -+ p(u)) / (t -+ u)."""
    t = np.linalg.svd(x, compute_uv=False)
    t = t / (np.sqrt((t * t).sum()) + eps)
    norms, factors = [np.sqrt((t * t).sum())], []
    for a, b, c in coefs:
        u, v = t[:, None], np.append(t, 0.0)[None, :]               # 0: what the longer side has beyond them
        s = t * t
        # the quotients as polynomials, without the division
        minus = a + b * (u * u + u * v + v * v) + c * (u ** 4 + u ** 3 * v + u * u * v * v + u * v ** 3 + v ** 4)
        plus = a + b * (u * u - u * v + v * v) + c * (u ** 4 - u ** 3 * v + u * u * v * v - u * v ** 3 + v ** 4)
        factors.append(np.maximum(np.abs(minus), np.abs(plus)))
        t = t * (a + b * s + c * s * s)
        norms.append(np.sqrt((t * t).sum()))
    total, reach = max(1.0, norms[-1]), np.ones_like(u * v)
    for n, f in zip(norms[-2::-1], factors[::-1]):
        reach = reach * f
        total += max(1.0, n) * reach.max()
    return total


def _steps_tol(x, coefs, want, kind, scale=1.0):
    """Every stage is off by a few 2^-22 of its matrix."""
    return 8 * 2.0 ** -22 * abs(scale) * _growth(x, coefs) + UOUT[kind] * np.linalg.norm(want)


def _spectrum(seed, M, N, rank, noise):
    """A matrix of low rank with noise: f32 tensor and its values."""
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, rank)) @ rng.standard_normal((rank, N)) + noise * rng.standard_normal((M, N))).float()
    return x.cuda(), x.double().numpy()


@pytest.mark.parametrize("M,N", [(100, 12000), (300, 9000), (1600, 4800), (4800, 1600)])
@pytest.mark.parametrize("rank,noise", [(1, 1e-5), (6, 1e-3), (40, 1e-2), (0, 1.0)])
def test_orthogonalise_spectra_on_the_smaller_side(op, M, N, rank, noise):  # noqa: F811
    """16-bit results of updates of low rank by the usual steps, which run on A alone where one side is much the smaller."""
    x, xv = _spectrum(rank, min(M, N), max(M, N), rank, noise)
    if M > N:
        x = x.t().contiguous()
    want = layer.orthogonalise(xv, 5, [USUAL] * 5, 1e-7)
    y = op.orthogonalise(x, out_dtype=_dt("bf16"))
    # a rounding of A that reaches the last step: below 2^-9 of the result
    got = _np(y) if M <= N else _np(y).T
    assert np.linalg.norm(got - want) <= _steps_tol(xv, [USUAL] * 5, want, "bf16") + 2.0 ** -9 * np.linalg.norm(want)


@pytest.mark.parametrize("M,N", [(100, 12000), (300, 9000), (9000, 300)])
def test_orthogonalise_spectra_of_a_batch(op, M, N):  # noqa: F811
    """The same for matrices of different ranks in one call."""
    import torch
    made = [_spectrum(rank, min(M, N), max(M, N), rank, noise) for rank, noise in ((1, 1e-5), (0, 1.0), (6, 1e-3))]
    x = torch.stack([t for t, _ in made])
    y = op.orthogonalise(x if M <= N else x.transpose(1, 2).contiguous(), out_dtype=_dt("bf16"))
    y = y if M <= N else y.transpose(1, 2)
    for got, (_, xv) in zip(y, made):
        want = layer.orthogonalise(xv, 5, [USUAL] * 5, 1e-7)
        assert np.linalg.norm(_np(got) - want) <= _steps_tol(xv, [USUAL] * 5, want, "bf16") + 2.0 ** -9 * np.linalg.norm(want)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(100, 12000), (9000, 130)])
def test_orthogonalise_beyond_the_usual_range(op, M, N, out):  # noqa: F811
    """Steps that stay within what the header allows (|X| < 8, |X X'| < 64, |Q| < 256) but take singular values past
    those that the usual coefficients reach, and many steps whose last one has no linear term."""
    import torch
    x, xv = _rand(1, (M, N), "f32", 1e-4)
    x[7, 5], xv[7, 5] = 1e3, 1e3                                    # one singular value, in one place
    for xs, xsv, coefs in ((x, xv, [(2.8, 0.0, 0.0), (0.2, 0.0, 0.04)]),
                           (*_spectrum(2, M, N, 6, 1e-3), [(1.5, 0.0, -0.5)] * 25)):
        coefs32 = np.float32(coefs).astype(np.float64).tolist()
        want = layer.orthogonalise(xsv, len(coefs), coefs32, 1e-7) if M <= N else layer.orthogonalise(xsv.T, len(coefs), coefs32, 1e-7).T
        y = op.orthogonalise(xs, steps=len(coefs), coefs=coefs, out_dtype=_dt(out))
        assert torch.isfinite(y).all()
        tol = _steps_tol(xsv if M <= N else xsv.T, coefs32, want, out)
        assert tol < 0.1 * np.linalg.norm(want)
        assert np.linalg.norm(_np(y) - want) <= tol


# ---------------------------------------------------------------------------
# how much the orthogonalised updates keep
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("steps", [1, 3, 5, 9])
@pytest.mark.parametrize("M,N", [(12, 40), (40, 12), (100, 260), (200, 136), (300, 700)])
def test_orthogonalise_keeps_22_bits(op, steps, M, N):  # noqa: F811
    """Tolerances from the coefficients of the case: half of the bits missing anywhere would show."""
    x, xv = _rand(steps, (M, N), "f32")
    for coefs in ([(1.875 - 0.02 * i, -1.25, 0.375 + 0.01 * i) for i in range(steps)], [(1.5, -0.5, 0.0)] * steps, [USUAL] * steps):
        coefs32 = np.float32(coefs).astype(np.float64).tolist()
        want = layer.orthogonalise(xv, steps, coefs32, 1e-7)
        y = op.orthogonalise(x, steps=steps, coefs=coefs)
        assert np.linalg.norm(_np(y) - want) <= _steps_tol(xv, coefs32, want, "f32")


@pytest.mark.parametrize("M,N", [(64, 64), (70, 300)])
def test_orthogonalise_coefficients_of_one_sign(op, M, N):  # noqa: F811
    """X X' of 62 and a polynomial whose square has its centre on the other side: nothing leaves the range on the way."""
    import torch
    x = torch.zeros(M, N, device="cuda")
    x[3, 5] = 2.0
    coefs = [(7.9, 0.0, 0.0), (0.1, 0.0008, 0.0002)]
    coefs32 = np.float32(coefs).astype(np.float64).tolist()
    want = layer.orthogonalise(_np(x), 2, coefs32, 1e-7)
    assert 7 < np.abs(want).max() < 8
    y = op.orthogonalise(x, steps=2, coefs=coefs)
    assert np.linalg.norm(_np(y) - want) <= _steps_tol(_np(x), coefs32, want, "f32")


@pytest.mark.parametrize("M,N", [(12, 40), (96, 200)])
@pytest.mark.parametrize("scale", [2e-38, -1e-33, 3e30])
def test_orthogonalise_of_any_scale(op, M, N, scale):  # noqa: F811
    """The factor of the result from the smallest to large ones."""
    x, xv = _rand(3, (M, N), "f32")
    scale = float(np.float32(scale))
    for out in ("f32", "bf16"):
        want = layer.orthogonalise(xv, 5, [USUAL] * 5, 1e-7, scale)
        y = op.orthogonalise(x, scale=scale, out_dtype=_dt(out))
        assert np.linalg.norm(_np(y) - want) <= _steps_tol(xv, [USUAL] * 5, want, out, scale) + M * N * FLOOR[out]


# ---------------------------------------------------------------------------
# activations of large projections
# ---------------------------------------------------------------------------

SIZES_OF_GATES = [1e2, 1e4, 1e10, 1e11, 1e12, 1e15, 1e18, 2.5e19, 1e30, 1e33, 1e35, 3e38]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_large_gates(op, act, T, kind):  # noqa: F811
    """Values and slopes from 1e2 to the largest, of both signs: what lies below zero goes to 0 however large the factors
    beside it.  x is a unit matrix, so every sum has one term: gates within 2^-21, activations and slopes within 16 u of
    themselves, and the result's rounding."""
    import torch
    g = torch.tensor([s * v for v in SIZES_OF_GATES for s in (-1.0, 1.0)], dtype=torch.float64).to(_dt(kind)).cuda()
    F = len(g)
    x = torch.eye(T, dtype=_dt(kind), device="cuda")
    wg = g[:, None].expand(F, T).contiguous()
    one = torch.ones_like(wg)
    v = np.broadcast_to(_np(g), (T, F))
    want, slope = layer.act(v, act), layer.act_slope(v, act)
    r = op.gated_ffn(x, wg, one, act=act, keep=True)
    near = 2.0 ** -20 + UOUT[kind]
    _close(r.gate, v, near * np.abs(v), "gate")
    _close(r.h, want, near * np.abs(want) + TINY, "h")
    gate, up = g.expand(T, F).contiguous(), torch.ones(T, F, dtype=_dt(kind), device="cuda")
    dx, dwg, dwu = op.gated_ffn_back(torch.ones_like(up), x, one, torch.zeros_like(one), gate, up, act=act)
    _close(dwg, slope.T, near * np.abs(slope.T) + TINY, "slope")
    _close(dwu, want.T, near * np.abs(want.T) + TINY, "activation")
    total = slope.sum(1)[:, None] * np.ones((1, T))
    _close(dx, total, 2 * near * np.abs(slope).sum(1)[:, None] + TINY, "dx")


# ---------------------------------------------------------------------------
# one row of weights
# ---------------------------------------------------------------------------

def test_gated_ffn_of_one_feature(op):  # noqa: F811
    """F = 1: a row's place does not matter, but its elements have to be contiguous in either weight."""
    import torch
    x, _ = _rand(1, (20, 16), "f32")
    wg, _ = _rand(2, (1, 16), "f32")
    wu, _ = _rand(3, (1, 16), "f32")
    r = op.gated_ffn(x, wg, wu, keep=True)
    apart = torch.cat([wu, wg], 1)[:, :16]                          # a row of a wider matrix
    assert torch.equal(op.gated_ffn(x, wg, apart).h, r.h) and torch.equal(op.gated_ffn(x, apart, wg).h, op.gated_ffn(x, wu, wg).h)
    d = torch.ones_like(r.h)
    for a, b in zip(op.gated_ffn_back(d, x, wg, apart, r.gate, r.up), op.gated_ffn_back(d, x, wg, wu, r.gate, r.up)):
        assert torch.equal(a, b)
    spread = wu.repeat_interleave(2, 1)[:, ::2]
    assert torch.equal(spread, wu) and spread.stride(1) == 2
    for a, b in ((wg, spread), (spread, wu)):
        with pytest.raises(ValueError):
            op.gated_ffn(x, a, b)
        with pytest.raises(ValueError):
            op.gated_ffn_back(d, x, a, b, r.gate, r.up)
    with pytest.raises(ValueError):
        op.gated_ffn(x, wg, wu.cpu())


# ---------------------------------------------------------------------------
# head norms of very large and very small heads
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D,rot", [(64, 64), (128, 96), (33, 32), (7, 4), (1024, 512), (1021, 64)])
@pytest.mark.parametrize("kind,d_kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_qk_norm_rope_of_heads_of_all_scales(op, D, rot, kind, d_kind, eps):  # noqa: F811
    """Heads from 2^-115 to 2^120 side by side: sums of their squares leave fp32's range."""
    import torch
    scales = 2.0 ** np.array([0, 120, -115, 63, -52, 64, -63, 100, -100, 0, 70, -75])
    T, H = 3, len(scales)
    x, _ = _rand(D, (T, H, D), kind)
    x = (x.double() * torch.from_numpy(scales).cuda()[None, :, None]).to(x.dtype)
    xv = _np(x)
    w, wv = _rand(2, (D,), "f32", 0.3, 1.0)
    d, dv = _rand(3, (T, H, D), d_kind)
    pos = np.array([0, 17, 90001], dtype=np.int32)
    freqs = (1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    tp, tf = torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda()
    eps_v = float(np.float32(eps))
    y, yk = op.qk_norm_rope(x, x[:, :5], tp, tf, w, w, eps=eps)
    want = layer.norm_rope(xv, wv, pos, freqs, eps_v, False)
    n = layer.norm_rope(xv, wv, pos, freqs[:0], eps_v, False)
    _close(y, want, _y_tol(n, rot, False, kind, want), "y")
    assert torch.equal(yk, y[:, :5])
    gx, _, gw, _ = op.qk_norm_rope_back(d, None, x, None, tp, tf, w, eps=eps)
    dx, dw = layer.norm_rope_back(dv, xv, wv, pos, freqs, eps_v, False)
    # as in test_qk_norm_rope_back; |dn| is bounded by its pair's elements
    a, b = layer.pairs(D, rot, False)
    dn = np.abs(dv)
    dn[..., a], dn[..., b] = dn[..., a] + np.abs(dv[..., b]), dn[..., b] + np.abs(dv[..., a])
    r = 1 / np.sqrt((xv * xv).mean(-1, keepdims=True) + eps_v)
    xr, wd = np.abs(xv) * r, np.abs(wv) * dn
    tol = r * (50 * U * wd + xr * (wd * xr).mean(-1, keepdims=True) * 130 * U) + UOUT[d_kind] * np.abs(dx) + FLOOR[d_kind]
    _close(gx, dx, tol, "dx")
    _close(gw, dw, (45 + T * H + 400) * U * (dn * xr).sum((0, 1)) + TINY, "dw")


def test_qk_norm_rope_of_heads_that_are_not_finite(op):  # noqa: F811
    """A NaN makes its head NaN, an Inf its own element, as the formula has it; zeros stay zeros; the heads beside them are
    untouched."""
    import torch
    x, _ = _rand(1, (2, 6, 64), "f32")
    want = op.qk_norm_rope(x, None, None, None)[0]
    x[0, 1, 5], x[1, 2, 7], x[0, 3] = float("nan"), float("inf"), 0.0
    y = op.qk_norm_rope(x, None, None, None)[0]
    assert torch.isnan(y[0, 1]).all() and torch.isnan(y[1, 2, 7]) and (y[1, 2, :7] == 0).all() and (y[0, 3] == 0).all()
    for t, h in ((0, 0), (0, 2), (0, 4), (0, 5), (1, 0), (1, 1), (1, 3), (1, 4), (1, 5)):
        assert torch.equal(y[t, h], want[t, h])


# ---------------------------------------------------------------------------
# outliers
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T", [8, 9, 130])
def test_gated_ffn_outlier_that_no_weight_meets(op, T):  # noqa: F811
    """f32: an element of 2^28 under a column of zeros.  Up to eight tokens keep fp32; more of them lose up to 2^-38 of
    their row's largest element in each of the others, whatever weight that one meets."""
    K, F = 256, 40
    x, xv = _rand(T, (T, K), "f32")
    wg, wgv = _rand(2, (F, K), "f32", K ** -0.5)
    wu, wuv = _rand(3, (F, K), "f32", K ** -0.5)
    x[2, 9], xv[2, 9] = 2.0 ** 28, 2.0 ** 28
    wg[:, 9], wgv[:, 9], wu[:, 9], wuv[:, 9] = 0.0, 0.0, 0.0, 0.0
    r = op.gated_ffn(x, wg, wu, keep=True)
    for got, wv in ((r.gate, wgv), (r.up, wuv)):
        ax, aw = np.abs(xv), np.abs(wv)
        tol = PROD(K, "f32") * (ax @ aw.T)
        if T > 8:
            tol = tol + 2.0 ** -38 * (ax.max(1)[:, None] * aw.sum(1) + ax.sum(1)[:, None] * aw.max(1))
        _close(got, xv @ wv.T, tol, "outlier")


# ---------------------------------------------------------------------------
# how much dgate and dup keep between the products
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,K,F", [(1, 96, 130), (16, 264, 24), (40, 72, 48), (256, 136, 72), (257, 2048, 4080), (257, 2048, 4088)])
def test_gated_ffn_back_keeps_16_bits_in_small_calls(op, T, K, F):  # noqa: F811
    """bf16: two bfloat16 terms of dgate and dup, 2^-16, where T is at most 256 or K * F * T at most 2^31; 2^-8 beyond.
    Results that cancel show it: a result's own rounding is 2^-8 of itself, that of the terms of their magnitudes.
    Exact products, sums of two (or one) terms for each of N elements: 2 N / 16 + 4 tensor-core additions."""
    small = T <= 256 or K * F * T <= 2 ** 31
    assert small == ((T, K, F) != (257, 2048, 4088))
    x, xv = _rand(1, (T, K), "bf16")
    wg, wgv = _rand(2, (F, K), "bf16", K ** -0.5)
    wu, wuv = _rand(3, (F, K), "bf16", K ** -0.5)
    gate, gv = _rand(4, (T, F), "bf16")
    up, uv = _rand(5, (T, F), "bf16")
    d, dv = _rand(6, (T, F), "bf16")
    dx, dwg, dwu = op.gated_ffn_back(d, x, wg, wu, gate, up)
    tokens, features = slice(0, min(T, 24)), slice(F - min(F, 72), F)
    held = 2.0 ** -16 if small else 2.0 ** -8

    def terms(rows, cols):
        g, u, e = gv[rows, cols], uv[rows, cols], dv[rows, cols]
        dg, du = e * u * layer.act_slope(g, "silu"), e * layer.act(g, "silu")
        eg, eu = 20 * U * np.abs(e * u) * (1 + np.abs(g)) + held * np.abs(dg), 20 * U * np.abs(e) * (1 + np.abs(g)) + held * np.abs(du)
        return dg, du, eg, eu

    def check(got, want, errors, magnitudes, n, what):
        tol = errors + (2 * n / 16 + 4) * 2.0 ** -23 * magnitudes + UOUT["bf16"] * np.abs(want) * 1.01 + FLOOR["bf16"]
        _close(got, want, tol, what)

    dg, du, eg, eu = terms(tokens, slice(None))
    check(dx[tokens], dg @ wgv + du @ wuv, eg @ np.abs(wgv) + eu @ np.abs(wuv), np.abs(dg) @ np.abs(wgv) + np.abs(du) @ np.abs(wuv), 2 * F, "dx")
    dg, du, eg, eu = terms(slice(None), features)
    check(dwg[features], dg.T @ xv, eg.T @ np.abs(xv), np.abs(dg).T @ np.abs(xv), T, "dw_gate")
    check(dwu[features], du.T @ xv, eu.T @ np.abs(xv), np.abs(du).T @ np.abs(xv), T, "dw_up")
