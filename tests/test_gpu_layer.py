"""GPU parity of the layer operators against plain 64-bit implementations
(oracle/layer.py), at the sizes, strides and values where they can go wrong.

Tolerances follow from the arithmetic and are written before any run.  u = 2^-24 is a
rounding to fp32 and UOUT one to the output's type.  A product's sum of K terms is
off by at most PROD(K, kind) of the sum of the terms' magnitudes:

  f32     operands as three bfloat16 terms each, or two scaled binary16 ones: what is dropped is
          below 2^-22 of a product; at most 24 tensor-core additions into one partial sum, each off by
          at most 2^-23 of the magnitudes, then one rounding for each of K / 64 partial sums: together
          below 50 * 2^-23 + K / 128 * 2^-24 + 2^-25
  16 bit  exact products; K / 16 + 1 tensor-core additions
  mixed   operands as two terms each: three quantities below 2^-18 of a product, and
          three times the additions of the 16-bit form
"""

import math

import numpy as np
import pytest

import synth
from oracle import layer
from oracle import training as tr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UOUT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}
TINY = 1e-30                # far below every value here: what under- and overflow of exp may leave


def PROD(K, kind):
    if kind == "f32":
        return 2.0 ** -25 + 50 * 2.0 ** -23 + (K / 128 + 2) * U
    if kind == "16":
        return (K / 16 + 2) * 2.0 ** -23
    return 3 * 2.0 ** -18 + (3 * K / 16 + 4) * 2.0 ** -23


@pytest.fixture(scope="module")
def op():
    import torch
    import ggml_out_prod_gb300 as g
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    g.build()
    g.lib()
    g.device_status(clear=True)
    return g


@pytest.fixture(autouse=True)
def _status(op):
    yield
    assert op.device_status(clear=True) == op.OK


def _dt(kind):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]


def _rand(seed, shape, kind, std=1.0, mean=0.0):
    """(CUDA tensor of the type, its values in float64)."""
    import torch
    rng = np.random.default_rng(seed)
    t = torch.from_numpy(rng.standard_normal(shape) * std + mean).to(_dt(kind))
    return t.cuda(), t.double().numpy()


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol, what):
    """Every element within its tolerance."""
    got = _np(got)
    assert got.shape == np.shape(want), f"{what}: shape {got.shape}"
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if np.any(bad):
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(tol, 1e-300), 0)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {i} got {got[i]!r} "
                             f"want {np.asarray(want)[i]!r} tol {np.broadcast_to(tol, err.shape)[i]!r}")


def _framed(t, extra=3, at=1):
    """The same values as a view into a larger tensor of NaN: rows (last axis) apart by `extra`
    more elements, starting `at` elements in."""
    import torch
    big = torch.full(tuple(t.shape[:-1]) + (t.shape[-1] + extra,), float("nan"), dtype=t.dtype, device=t.device)
    view = big[..., at:at + t.shape[-1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------
# head norms with rotation
# ---------------------------------------------------------------------------

def _partner(v, n_rot, interleaved):
    """|v| of the other element of each pair, 0 where there is none."""
    y = np.zeros_like(v)
    a, b = layer.pairs(v.shape[-1], n_rot, interleaved)
    y[..., a], y[..., b] = np.abs(v[..., b]), np.abs(v[..., a])
    return y


def _norm_case(seed, T, Hq, Hk, D, rot, kind, w_kind):
    import torch
    q, qv = _rand(seed, (T, Hq, D), kind, 1.3)
    k, kv = _rand(seed + 1, (T, Hk, D), kind, 0.8)
    wq, wqv = _rand(seed + 2, (D,), w_kind, 0.3, 1.0)
    wk, wkv = _rand(seed + 3, (D,), w_kind, 0.3, 1.0)
    pos = np.random.default_rng(seed).integers(0, 200000, T).astype(np.int32)
    freqs = (1e4 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    return (q, qv, wq, wqv), (k, kv, wk, wkv), torch.from_numpy(pos).cuda(), pos, torch.from_numpy(freqs).cuda(), freqs


# r: a sum of squares by chains of at most 40 additions (rel. 40 u, halved by the root), the root, the
# quotient and two products; sin and cos within 4 u.  y = a cos - b sin: 32 u of |a| and of |b| in all.
def _y_tol(n, rot, interleaved, kind, y):
    return 40 * U * (np.abs(n) + _partner(n, rot, interleaved)) + UOUT[kind] * np.abs(y) + FLOOR[kind]


NORM_SIZES = [(1, 1, 1, 1, 0), (1, 1, 1, 2, 2), (5, 3, 1, 7, 4), (3, 2, 2, 64, 64), (17, 4, 1, 128, 128), (9, 5, 5, 80, 40),
              (2, 8, 2, 96, 96), (33, 2, 1, 256, 64), (3, 3, 2, 512, 512), (2, 2, 1, 1024, 1024), (2, 1, 1, 1021, 512),
              (700, 9, 3, 96, 48), (1500, 1, 2, 33, 32)]


@pytest.mark.parametrize("T,Hq,Hk,D,rot", NORM_SIZES)
@pytest.mark.parametrize("kind,w_kind", [("f32", "f32"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_norm_rope(op, T, Hq, Hk, D, rot, kind, w_kind, interleaved):
    a, b, pos, posv, freqs, freqsv = _norm_case(D + T, T, Hq, Hk, D, rot, kind, w_kind)
    yq, yk = op.qk_norm_rope(a[0], b[0], pos, freqs, a[2], b[2], eps=1e-6, interleaved=interleaved)
    for y, (_, x, _, w) in ((yq, a), (yk, b)):
        want = layer.norm_rope(x, w, posv, freqsv, 1e-6, interleaved)
        n = layer.norm_rope(x, w, posv, freqsv[:0], 1e-6, interleaved)
        _close(y, want, _y_tol(n, rot, interleaved, kind, want), "qk_norm_rope")


@pytest.mark.parametrize("T,Hq,Hk,D,rot", NORM_SIZES)
@pytest.mark.parametrize("kind,d_kind,w_kind", [("f32", "f32", "f32"), ("bf16", "bf16", "f32"), ("f16", "bf16", "bf16"),
                                                ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_norm_rope_back(op, T, Hq, Hk, D, rot, kind, d_kind, w_kind, interleaved):
    a, b, pos, posv, freqs, freqsv = _norm_case(D + T, T, Hq, Hk, D, rot, kind, w_kind)
    dq, dqv = _rand(T + 9, (T, Hq, D), d_kind, 2.0)
    dk, dkv = _rand(T + 10, (T, Hk, D), d_kind, 2.0)
    gq, gk, gwq, gwk = op.qk_norm_rope_back(dq, dk, a[0], b[0], pos, freqs, a[2], b[2], eps=1e-6, interleaved=interleaved)
    for g, gw, dv, (_, x, _, w) in ((gq, gwq, dqv, a), (gk, gwk, dkv, b)):
        dx, dw = layer.norm_rope_back(dv, x, w, posv, freqsv, 1e-6, interleaved)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        dn = np.abs(dv) + _partner(dv, rot, interleaved)         # bounds |dn|; dn is off by 10 u of it
        xr, wd = np.abs(x) * r, np.abs(w) * dn
        mean = (wd * xr).mean(-1, keepdims=True)
        # g 12 u, x r 30 u, their mean a chain of 40 more: 90 u of mean |g x r|
        tol = r * (50 * U * wd + xr * mean * 130 * U) + UOUT[d_kind] * np.abs(dx) + FLOOR[d_kind]
        _close(g, dx, tol, "dx")
        n = x.shape[0] * x.shape[1]
        chain = 45 + n / 8 + 400                                  # terms 45 u each; any order of the sum
        _close(gw, dw, chain * U * (dn * xr).sum((0, 1)) + 1e-30, "dw")


@pytest.mark.parametrize("how", ["fused", "heads_first", "unaligned", "in_place"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_qk_norm_rope_layouts(op, how, kind):
    """Slices of one buffer, heads in the outer place, rows off any alignment, in place."""
    import torch
    T, Hq, Hk, D = 37, 6, 2, 64
    a, b, pos, posv, freqs, freqsv = _norm_case(3, T, Hq, Hk, D, D, kind, "f32")
    q, k = a[0], b[0]
    dq, dqv = _rand(5, (T, Hq, D), kind)
    dk, dkv = _rand(6, (T, Hk, D), kind)
    dense = op.qk_norm_rope(q, k, pos, freqs, a[2], b[2])
    dense_back = op.qk_norm_rope_back(dq, dk, q, k, pos, freqs, a[2], b[2])
    outs = {}
    if how == "fused":
        buf = torch.cat([q.reshape(T, -1), k.reshape(T, -1), torch.full((T, Hk * D), float("nan"), device="cuda", dtype=q.dtype)], 1)
        q, k = buf[:, :Hq * D].view(T, Hq, D), buf[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    elif how == "heads_first":
        q, k = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k))
        outs = {"out_q": torch.empty_like(q), "out_k": torch.empty_like(k)}
    elif how == "unaligned":
        q, k, dq, dk = (_framed(t) for t in (q, k, dq, dk))
        outs = {"out_q": _framed(a[0]), "out_k": _framed(b[0])}
    if how == "in_place":
        dx = op.qk_norm_rope_back(dq, dk, q, k, pos, freqs, a[2], b[2], out_q=dq, out_k=dk)
        assert dx[0] is dq and all(torch.equal(x, y) for x, y in zip(dx, dense_back))
        y = op.qk_norm_rope(q, k, pos, freqs, a[2], b[2], out_q=q, out_k=k)
        assert y[0] is q and torch.equal(y[0], dense[0]) and torch.equal(y[1], dense[1])
        return
    y = op.qk_norm_rope(q, k, pos, freqs, a[2], b[2], **outs)
    tol = 0 if how != "unaligned" else 2 * UOUT[kind] + 80 * U      # the one-element form sums in another order
    for got, want in zip(y, dense):
        _close(got, _np(want), tol * np.abs(_np(want)) + tol, how)
    dx = op.qk_norm_rope_back(dq, dk, q, k, pos, freqs, a[2], b[2])
    for got, want in zip(dx, dense_back):
        _close(got, _np(want), (tol * 40) * (1 + np.abs(_np(want))), how)


def test_qk_norm_rope_far_positions_and_edges(op):
    """Positions at both ends of int32, frequencies above one turn and of nothing, no k, no weights, no rotation,
    zero tokens, zero rows."""
    import torch
    D = 64
    pos = np.array([2 ** 31 - 1, -2 ** 31, 1000003, -1, 0, 123456789], dtype=np.int32)
    T = len(pos)
    freqs = np.array([1.0, 6.5, 0.0, 1e-9, -0.37, 100.25, 3.1415927, 2.0 ** -30] * 4, dtype=np.float32)
    q, qv = _rand(1, (T, 3, D), "f32")
    tp, tf = torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda()
    y, none = op.qk_norm_rope(q, None, tp, tf, eps=0.0)
    assert none is None
    # the reference's angle reduced in exact integer arithmetic: pos * freq as a rational number of turns
    from fractions import Fraction
    import decimal
    decimal.getcontext().prec = 60
    two_pi = Fraction(decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194989"))
    turns = np.array([[float((Fraction(int(p)) * Fraction(float(f)) / two_pi) % 1) for f in freqs] for p in pos])
    n = layer.norm_rope(qv, None, pos, freqs[:0], 0.0, False)
    c, s = np.cos(2 * np.pi * turns)[:, None, :], np.sin(2 * np.pi * turns)[:, None, :]
    want = np.concatenate([n[..., :32] * c - n[..., 32:] * s, n[..., :32] * s + n[..., 32:] * c], -1)
    _close(y, want, _y_tol(n, D, False, "f32", want) + 2.0 ** -31 * 8, "far positions")
    y, _ = op.qk_norm_rope(q, None, None, None, eps=1e-6)
    want = layer.norm_rope(qv, None, pos, freqs[:0], 1e-6, False)
    _close(y, want, 40 * U * np.abs(want), "norm alone")
    e = op.qk_norm_rope(q[:0], q[:0], tp[:0], tf)
    assert e[0].shape == (0, 3, D)
    g = op.qk_norm_rope_back(q[:0], q[:0], q[:0], q[:0], tp[:0], tf)
    assert g[0].shape == (0, 3, D) and (g[2] == 0).all() and (g[3] == 0).all()
    z = torch.zeros_like(q)
    y, _ = op.qk_norm_rope(z, None, tp, tf, eps=1e-6)
    assert (y == 0).all()
    bad = tf.clone()
    bad[3] = float("inf")
    y, _ = op.qk_norm_rope(q, None, tp, bad)
    assert torch.isnan(y[..., [3, 35]]).all() and torch.isfinite(y[..., [2, 4, 34, 36]]).all()


def test_qk_norm_rope_gradient_of_its_own_forward(op):
    """Differences of the forward kernel along random directions."""
    import torch
    T, H, D = 5, 3, 32
    q, qv = _rand(1, (T, H, D), "f32")
    w, wv = _rand(2, (D,), "f32", 0.2, 1.0)
    dy, dyv = _rand(3, (T, H, D), "f32")
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 11
    freqs = torch.linspace(1.0, 0.01, D // 2).cuda()
    dx, _, dw, _ = op.qk_norm_rope_back(dy, None, q, None, pos, freqs, w)
    step = 1e-2                                                   # error of the difference ~ step^2 and 1e-7 / step
    for i in range(4):
        e, ev = _rand(10 + i, (T, H, D), "f32")
        up, down = (_np(op.qk_norm_rope(q + s * step * e, None, pos, freqs, w)[0]) for s in (1, -1))
        slope = ((up - down) * dyv).sum() / (2 * step)
        assert abs(slope - (_np(dx) * ev).sum()) < 2e-2 * np.sqrt(T * H * D)
        f, fv = _rand(20 + i, (D,), "f32")
        up, down = (_np(op.qk_norm_rope(q, None, pos, freqs, w + s * step * f)[0]) for s in (1, -1))
        slope = ((up - down) * dyv).sum() / (2 * step)
        assert abs(slope - (_np(dw) * fv).sum()) < 1e-3 * np.sqrt(T * H * D)


# ---------------------------------------------------------------------------
# the gated feed-forward block
# ---------------------------------------------------------------------------

ACTS = ["silu", "gelu_tanh", "gelu_erf", "relu"]
SIZES = [(1, 1, 1), (1, 64, 128), (3, 40, 17), (7, 33, 65), (16, 256, 128), (70, 200, 130), (129, 64, 257), (300, 520, 264),
         (257, 1000, 300), (1, 2560, 640), (9, 1024, 96)]


def _prod_kind(x_kind, w_kind):
    return "f32" if x_kind == "f32" else "16" if x_kind == w_kind else "mixed"


def _h_tol(x, wg, wu, gate, up, act, prod, kind):
    """(tolerance of h, of gate, of up): the slopes of all four activations are below 1.2 in magnitude, and an
    activation is computed within 16 u of |v|."""
    p = PROD(x.shape[1], prod)
    tg, tu = p * (np.abs(x) @ np.abs(wg).T), p * (np.abs(x) @ np.abs(wu).T)
    a = layer.act(gate, act)
    th = (1.2 * tg + 16 * U * np.abs(gate)) * (np.abs(up) + tu) + np.abs(a) * tu
    return [t + UOUT[kind] * np.abs(v) * 1.01 + FLOOR[kind] + TINY for t, v in ((th, a * up), (tg, gate), (tu, up))]


@pytest.mark.parametrize("T,K,F", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_gated_ffn(op, T, K, F, kind):
    act = ACTS[(T + K) % 4]
    x, xv = _rand(T, (T, K), kind)
    wg, wgv = _rand(K, (F, K), kind, K ** -0.5)
    wu, wuv = _rand(F, (F, K), kind, K ** -0.5)
    h, gate, up = layer.gated_ffn(xv, wgv, wuv, act)
    r = op.gated_ffn(x, wg, wu, act=act, keep=True)
    tol = _h_tol(xv, wgv, wuv, gate, up, act, _prod_kind(kind, kind), kind)
    for got, want, t, what in zip(r, (h, gate, up), tol, ("h", "gate", "up")):
        _close(got, want, t, what)
    alone = op.gated_ffn(x, wg, wu, act=act)
    assert alone.gate is None and alone.up is None and (alone.h == r.h).all()


@pytest.mark.parametrize("x_kind,w_kind", [("bf16", "f32"), ("f16", "bf16"), ("bf16", "f16"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("T,K,F", [(5, 72, 40), (140, 264, 200)])
def test_gated_ffn_mixed_types(op, x_kind, w_kind, T, K, F):
    x, xv = _rand(T, (T, K), x_kind)
    wg, wgv = _rand(K, (F, K), w_kind, K ** -0.5)
    wu, wuv = _rand(F, (F, K), w_kind, K ** -0.5)
    h, gate, up = layer.gated_ffn(xv, wgv, wuv, "silu")
    tol = _h_tol(xv, wgv, wuv, gate, up, "silu", _prod_kind(x_kind, w_kind), x_kind)
    for got, want, t in zip(op.gated_ffn(x, wg, wu, keep=True), (h, gate, up), tol):
        _close(got, want, t, "gated_ffn")
    d, dv = _rand(9, (T, F), "f32" if x_kind == "f32" else "bf16")
    _check_back(op, x, xv, wg, wgv, wu, wuv, d, dv, "silu", x_kind, w_kind)


@pytest.mark.parametrize("kind", [synth.TYPE_Q8_0, synth.TYPE_Q4_0, synth.TYPE_Q5_1, synth.TYPE_Q4_K, synth.TYPE_Q6_K])
@pytest.mark.parametrize("x_kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 33])
def test_gated_ffn_quantised(op, kind, x_kind, T):
    import torch
    F = 72
    K = synth.BLOCK[kind][0] * 3
    x, xv = _rand(T, (T, K), x_kind)
    raw = [synth.quantize(kind, synth.normal(s, F * K, std=K ** -0.5).reshape(F, K)).reshape(F, -1) for s in (1, 2)]
    wgv, wuv = (tr.table_values(r, kind, K) for r in raw)
    wg, wu = (torch.from_numpy(r).cuda() for r in raw)
    h, gate, up = layer.gated_ffn(xv, wgv, wuv, "silu")
    tol = _h_tol(xv, wgv, wuv, gate, up, "silu", "f32" if x_kind == "f32" else "mixed", x_kind)
    # a decoded value is rounded once to fp32: 2 u of the block's largest
    extra = 2 * U * np.abs(xv).sum(1)[:, None] * max(np.abs(wgv).max(), np.abs(wuv).max()) * (1.2 * (1 + np.abs(up) + np.abs(gate)))
    for got, want, t in zip(op.gated_ffn(x, wg, wu, keep=True, w_type=kind), (h, gate, up), tol):
        _close(got, want, t + extra, "quantised")
    d, dv = _rand(9, (T, F), x_kind)
    _check_back(op, x, xv, wg, wgv, wu, wuv, d, dv, "silu", x_kind, "q", w_type=kind)


def _check_back(op, x, xv, wg, wgv, wu, wuv, d, dv, act, x_kind, w_kind, w_type=None, gu=None):
    import torch
    d_kind = {torch.float32: "f32", torch.bfloat16: "bf16"}[d.dtype]
    _, gate, up = layer.gated_ffn(xv, wgv, wuv, act)
    if gu is None:
        gu = [torch.from_numpy(v).to(x.dtype).cuda() for v in (gate, up)]
    gate, up = (_np(t) for t in gu)
    dx, dwg, dwu = op.gated_ffn_back(d, x, wg, wu, *gu, act=act, w_type=w_type)
    want = layer.gated_ffn_back(dv, xv, wgv, wuv, gate, up, act)
    dg, du = np.abs(want[3]), np.abs(want[4])
    T, F = dg.shape
    K = xv.shape[1]
    # dgate, dup: the activation and slope within 16 u (1 + |gate|), three products; rounded to dh's type
    held = 2.0 ** -8 if d_kind == "bf16" else 0.0
    eg = 20 * U * np.abs(dv * up) * (1 + np.abs(gate)) + held * dg
    eu = 20 * U * np.abs(dv) * (1 + np.abs(gate)) + held * du
    pw = PROD(2 * F, "f32" if d_kind == "f32" else "16" if w_kind == "bf16" else "mixed")
    px = PROD(T, "f32" if d_kind == "f32" else "16" if x_kind == "bf16" else "mixed")
    axv, ag, au = np.abs(xv), np.abs(wgv), np.abs(wuv)
    tol = (((dg * pw + eg) @ ag + (du * pw + eu) @ au), (dg * px + eg).T @ axv, (du * px + eu).T @ axv)
    if w_type is not None:
        tol = (tol[0] + 2 * U * (dg + du).sum(1)[:, None] * max(ag.max(), au.max()),) + tol[1:]
    for got, v, t, what in zip((dx, dwg, dwu), want, tol, ("dx", "dwg", "dwu")):
        _close(got, v, t + UOUT[d_kind] * np.abs(v) * 1.01 + FLOOR[d_kind] + TINY, what)
        if d_kind == "bf16" and v.size > 64:
            # independent roundings by at most half a step, of the terms and of the result
            assert np.linalg.norm(_np(got) - v) <= 2.0 ** -8 * np.linalg.norm(v) * math.sqrt(2), what
    return dx, dwg, dwu


@pytest.mark.parametrize("T,K,F", SIZES)
@pytest.mark.parametrize("x_kind,d_kind", [("f32", "f32"), ("bf16", "bf16"), ("f16", "bf16"), ("bf16", "f32")])
def test_gated_ffn_back(op, T, K, F, x_kind, d_kind):
    act = ACTS[(T + F) % 4]
    x, xv = _rand(T, (T, K), x_kind)
    wg, wgv = _rand(K, (F, K), x_kind, K ** -0.5)
    wu, wuv = _rand(F, (F, K), x_kind, K ** -0.5)
    d, dv = _rand(T + 7, (T, F), d_kind)
    _check_back(op, x, xv, wg, wgv, wu, wuv, d, dv, act, x_kind, x_kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("extra,at", [(3, 1), (8, 0), (64, 8)])
def test_gated_ffn_strides(op, kind, extra, at):
    """Rows apart and off alignment; what lies between them (NaN) is neither used nor written."""
    import torch
    T, K, F = 150, 136, 200
    x, xv = _rand(1, (T, K), kind)
    wg, wgv = _rand(2, (F, K), kind, K ** -0.5)
    wu, wuv = _rand(3, (F, K), kind, K ** -0.5)
    dense = op.gated_ffn(x, wg, wu, keep=True)
    out = _framed(dense.h, extra, at)
    out.zero_()
    r = op.gated_ffn(_framed(x, extra, at), _framed(wg, extra, at), _framed(wu, extra, at), keep=True, out=out)
    for a, b in zip(r, dense):
        assert torch.equal(a, b)
    frame = out._base
    assert torch.isnan(frame[:, :at]).all() and torch.isnan(frame[:, at + F:]).all()
    d_kind = "f32" if kind == "f32" else "bf16"
    d, dv = _rand(4, (T, F), d_kind)
    want = op.gated_ffn_back(d, x, wg, wu, dense.gate, dense.up)
    dx = torch.full((T, K + extra), float("nan"), dtype=d.dtype, device="cuda")
    got = op.gated_ffn_back(_framed(d, extra, at), _framed(x, extra, at), _framed(wg, extra, at), _framed(wu, extra, at),
                            _framed(dense.gate, extra, at), _framed(dense.up, extra, at), out=dx[:, at:at + K])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.isnan(dx[:, :at]).all() and torch.isnan(dx[:, at + K:]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_gated_ffn_repeated_and_overlapping_rows(op, kind):
    """A stride of 0 (one row for all tokens) and rows that share elements."""
    import torch
    T, K, F = 40, 64, 72
    line, lv = _rand(1, (K + 8 * T,), kind)
    wg, wgv = _rand(2, (F, K), kind, K ** -0.5)
    for step in (0, 8):
        x = torch.as_strided(line, (T, K), (step, 1))
        xd = x.contiguous()
        a, b = op.gated_ffn(x, wg, wg, keep=True), op.gated_ffn(xd, wg, wg, keep=True)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        w = torch.as_strided(line, (F - 40, K), (step, 1))
        assert torch.equal(op.gated_ffn(xd, w, w).h, op.gated_ffn(xd, w.contiguous(), w.contiguous()).h)
        d = torch.ones((T, F), dtype=torch.float32 if kind == "f32" else torch.bfloat16, device="cuda")
        for u, v in zip(op.gated_ffn_back(d, x, wg, wg, a.gate, a.up), op.gated_ffn_back(d, xd, wg, wg, a.gate, a.up)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K,F", [(8, 16), (1000, 37), (6000, 40)])
def test_gated_ffn_of_few_tokens(op, T, kind, K, F):
    """Around the number of tokens where the form changes, and where their values no longer fit shared memory."""
    x, xv = _rand(T, (T, K), kind)
    wg, wgv = _rand(K, (F, K), kind, K ** -0.5)
    wu, wuv = _rand(F, (F, K), kind, K ** -0.5)
    h, gate, up = layer.gated_ffn(xv, wgv, wuv, "silu")
    tol = _h_tol(xv, wgv, wuv, gate, up, "silu", _prod_kind(kind, kind), kind)
    for w in ((wg, wu), (_framed(wg), _framed(wu))):
        for got, want, t in zip(op.gated_ffn(x, *w, keep=True), (h, gate, up), tol):
            _close(got, want, t, "few tokens")


@pytest.mark.parametrize("T,K,F", [(300, 200, 3000), (64, 136, 2048), (256, 96, 520), (2100, 72, 80), (520, 1032, 4100)])
@pytest.mark.parametrize("x_kind,d_kind", [("f32", "f32"), ("bf16", "bf16"), ("f16", "bf16")])
def test_gated_ffn_back_in_parts(op, T, K, F, x_kind, d_kind):
    """Long sums over few tiles, which are taken in parts, and a call so large that dgate has dh's bits."""
    x, xv = _rand(T, (T, K), x_kind)
    wg, wgv = _rand(K, (F, K), x_kind, K ** -0.5)
    wu, wuv = _rand(F, (F, K), x_kind, K ** -0.5)
    d, dv = _rand(T + 7, (T, F), d_kind)
    _check_back(op, x, xv, wg, wgv, wu, wuv, d, dv, "silu", x_kind, x_kind)


def test_gated_ffn_rows_of_all_scales(op):
    """f32 rows from the smallest normal numbers to the largest, of zeros, and with one element far above the rest:
    what an element loses is 2^-24 of itself and 2^-39 of its row's largest."""
    import torch
    T, K, F = 64, 100, 48
    x, xv = _rand(1, (T, K), "f32")
    wg, wgv = _rand(2, (F, K), "f32", 0.1)
    wu, wuv = _rand(3, (F, K), "f32", 0.1)
    scale = 2.0 ** np.linspace(-120, 120, T).round()
    scale[5] = 0.0
    x, xv = x * torch.from_numpy(scale).float().cuda()[:, None], xv * scale[:, None]
    x[9, 3], xv[9, 3] = 2.0 ** 60, 2.0 ** 60
    ws = 2.0 ** np.linspace(-20, 3, F).round()
    wg, wgv = wg * torch.from_numpy(ws).float().cuda()[:, None], wgv * ws[:, None]
    for rows in (slice(0, T), slice(4, 10)):                       # on the tensor cores, and few of them
        _, gate, up = layer.gated_ffn(xv[rows], wgv, wuv, "relu")
        r = op.gated_ffn(x[rows], wg, wu, act="relu", keep=True)
        for got, want, wv in ((r.gate, gate, wgv), (r.up, up, wuv)):
            ax, aw = np.abs(xv[rows]), np.abs(wv)
            tol = PROD(K, "f32") * (ax @ aw.T) + 2.0 ** -39 * (ax.max(1)[:, None] * aw.sum(1) + ax.sum(1)[:, None] * aw.max(1))
            _close(got, want, tol + 2.0 ** -126, "all scales")


def test_gated_ffn_empty(op):
    import torch
    for T, K, F in ((0, 8, 16), (4, 8, 0), (4, 0, 16), (0, 0, 0)):
        x, w = torch.ones(T, K, device="cuda"), torch.ones(F, K, device="cuda")
        r = op.gated_ffn(x, w, w, keep=True)
        assert all(t.shape == (T, F) and (t == 0).all() for t in r)
        dx, dwg, dwu = op.gated_ffn_back(torch.ones(T, F, device="cuda"), x, w, w, r.gate, r.up)
        assert dx.shape == (T, K) and (dx == 0).all() and dwg.shape == (F, K) and (dwg == 0).all() and (dwu == 0).all()


def test_gated_ffn_large_gradients_and_outliers(op):
    """Gradients beyond binary16's range, and weights and activations next to them, as f32."""
    T, K, F = 96, 160, 136
    x, xv = _rand(1, (T, K), "f32")
    wg, wgv = _rand(2, (F, K), "f32", K ** -0.5)
    wu, wuv = _rand(3, (F, K), "f32", K ** -0.5)
    d, dv = _rand(4, (T, F), "f32", 1e4)
    d[3, 5], d[90, 100] = 1.5e5, -1.31e30
    dv[3, 5], dv[90, 100] = 1.5e5, float(d[90, 100])
    _check_back(op, x, xv, wg, wgv, wu, wuv, d, dv, "silu", "f32", "f32")


def test_gated_ffn_non_finite(op):
    """A NaN or Inf operand reaches the results that use it and no others; large projections do not overflow the
    activations."""
    import torch
    T, K, F = 140, 72, 136
    for kind in ("f32", "bf16"):
        x, _ = _rand(1, (T, K), kind)
        wg, _ = _rand(2, (F, K), kind, K ** -0.5)
        wu, _ = _rand(3, (F, K), kind, K ** -0.5)
        x[2, 3], x[130, 0] = float("nan"), float("inf")
        h = op.gated_ffn(x, wg, wu, keep=True)
        rows = torch.tensor([2, 130], device="cuda")
        assert (~torch.isfinite(h.gate[rows])).all() and (~torch.isfinite(h.up[rows])).all()
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert torch.isfinite(h.h[rest]).all()
        gate = torch.tensor([-3e4, -200.0, -90.0, 90.0, 3e4, -0.0], device="cuda").to(x.dtype).repeat(T, F // 6 + 1)[:, :F].contiguous()
        for act in ACTS:
            up, d = torch.ones_like(gate), torch.ones_like(gate)
            dx, dwg, dwu = op.gated_ffn_back(d, torch.ones(T, K, device="cuda", dtype=x.dtype), wg, wu, gate, up, act=act)
            assert torch.isfinite(dx).all() and torch.isfinite(dwg).all() and torch.isfinite(dwu).all()


def test_gated_ffn_gradients_against_differences(op):
    """The backward kernels against differences of the forward one along random directions (f32)."""
    T, K, F, step = 12, 24, 20, 2e-3
    x, xv = _rand(1, (T, K), "f32")
    wg, wgv = _rand(2, (F, K), "f32", 0.2)
    wu, wuv = _rand(3, (F, K), "f32", 0.2)
    d, dv = _rand(4, (T, F), "f32")
    for act in ACTS[:3]:
        r = op.gated_ffn(x, wg, wu, act=act, keep=True)
        dx, dwg, dwu = op.gated_ffn_back(d, x, wg, wu, r.gate, r.up, act=act)
        for g, i in ((dx, 0), (dwg, 1), (dwu, 2)):
            e, ev = _rand(30 + i, tuple(g.shape), "f32")
            ends = []
            for s in (1, -1):
                p = [x, wg, wu]
                p[i] = p[i] + s * step * e
                ends.append((_np(op.gated_ffn(*p, act=act).h) * dv).sum())
            # third derivatives times step^2, and roundings of 1e-7 over the step
            assert abs((ends[0] - ends[1]) / (2 * step) - (_np(g) * ev).sum()) < 5e-3 * math.sqrt(T * F * K)


# ---------------------------------------------------------------------------
# orthogonalised updates
# ---------------------------------------------------------------------------

USUAL = (3.4445, -4.7750, 2.0315)


def _orth_tol(want, steps, kind, scale=1.0):
    """In the 2-norm: every stage is off by a few 2^-22 of its matrix (norms up to 1.5 sqrt(n)), and a step's
    polynomial amplifies by at most 3.4445."""
    n = min(want.shape)
    return 8 * 2.0 ** -22 * 3.4445 ** steps * scale * (1 + 0.02 * math.sqrt(n)) + UOUT[kind] * np.linalg.norm(want)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 9), (4, 4), (8, 2560), (2560, 8), (17, 33), (64, 64), (100, 260), (260, 100), (257, 513),
                                 (384, 384), (33, 1000), (30, 20000)])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_orthogonalise(op, M, N, kind, out):
    x, xv = _rand(M + N, (M, N), kind, 0.02)
    y = op.orthogonalise(x, out_dtype=_dt(out))
    want = layer.orthogonalise(xv, 5, [USUAL] * 5, 1e-7)
    assert y.dtype == _dt(out)
    assert np.linalg.norm(_np(y) - want) <= _orth_tol(want, 5, out)


@pytest.mark.parametrize("steps", [0, 1, 2, 9])
@pytest.mark.parametrize("M,N", [(12, 40), (200, 136)])
def test_orthogonalise_steps_and_coefficients(op, steps, M, N):
    x, xv = _rand(steps, (M, N), "f32")
    coefs = [(1.875 - 0.02 * i, -1.25, 0.375 + 0.01 * i) for i in range(steps)]
    y = op.orthogonalise(x, steps=steps, coefs=coefs, eps=1e-3, scale=-2.5)
    want = layer.orthogonalise(xv, steps, np.float32(coefs).astype(np.float64).tolist(), float(np.float32(1e-3)), -2.5)
    assert np.linalg.norm(_np(y) - want) <= _orth_tol(want, steps, "f32", 2.5)
    if steps:
        same = op.orthogonalise(x, steps=steps, coefs=(1.5, -0.5, 0.0))
        assert np.linalg.norm(_np(same) - layer.orthogonalise(xv, steps, [(1.5, -0.5, 0.0)] * steps, 1e-7)) <= _orth_tol(xv, steps, "f32")


@pytest.mark.parametrize("B,M,N", [(3, 20, 12), (5, 70, 300), (33, 8, 64), (2, 300, 140)])
def test_orthogonalise_batches_and_strides(op, B, M, N):
    """A batch is its matrices one by one, bit for bit; strided ones and in place too; what lies between stays."""
    import torch
    x, xv = _rand(B, (B, M, N), "f32")
    y = op.orthogonalise(x)
    for i in (0, B - 1):
        want = layer.orthogonalise(xv[i], 5, [USUAL] * 5, 1e-7)
        assert np.linalg.norm(_np(y[i]) - want) <= _orth_tol(want, 5, "f32")
        assert torch.equal(op.orthogonalise(x[i].clone()), y[i])
    out = torch.full((B, M + 2, N + 5), float("nan"), device="cuda")
    view = out[:, :M, 3:3 + N]
    op.orthogonalise(_framed(x), out=view)
    assert torch.equal(view, y) and torch.isnan(out[:, M:]).all() and torch.isnan(out[:, :, :3]).all()
    op.orthogonalise(x, out=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("M,N", [(16, 48), (200, 300)])
def test_orthogonalise_scale_of_the_input(op, M, N):
    """The result does not depend on the input's scale (eps = 0), from tiny to huge values; zeros, NaN and Inf."""
    import torch
    x, xv = _rand(7, (M, N), "f32")
    want = layer.orthogonalise(xv, 5, [USUAL] * 5, 0.0)
    for s in (1.0, 2.0 ** -120, 2.0 ** 120, 2.0 ** -60, 2.0 ** 45):
        y = op.orthogonalise(x * s, eps=0.0)
        assert np.linalg.norm(_np(y) - want) <= _orth_tol(want, 5, "f32"), s
    assert (op.orthogonalise(torch.zeros_like(x)) == 0).all()
    for v in (float("nan"), float("inf")):
        bad = torch.stack([x, x])
        bad[1, M // 2, N // 3] = v
        y = op.orthogonalise(bad)
        assert torch.isnan(y[1]).all() and torch.equal(y[0], op.orthogonalise(x))


@pytest.mark.parametrize("M,N,out", [(200, 3000, "f32"), (3000, 200, "bf16"), (40, 5000, "f32"), (1600, 4800, "bf16"),
                                     (4200, 1300, "bf16")])
def test_orthogonalise_in_parts_and_on_the_smaller_side(op, M, N, out):
    """Few tiles of a long sum, and 16-bit results whose steps run on A alone."""
    x, xv = _rand(M, (M, N), "f32", 1e-3)
    y = op.orthogonalise(x, out_dtype=_dt(out))
    want = layer.orthogonalise(xv, 5, [USUAL] * 5, 1e-7)
    # on A alone: the rounding of A that reaches the last step, below 2^-9 of it
    extra = 2.0 ** -9 * np.linalg.norm(want) if out == "bf16" else 0.0
    assert np.linalg.norm(_np(y) - want) <= _orth_tol(want, 5, out) + extra


def test_orthogonalise_low_rank(op):
    """A gradient of low rank with a little noise: the leading singular values come near one, the rest grows by at
    most 3.4445^5."""
    import torch
    rng = np.random.default_rng(5)
    xv = rng.standard_normal((160, 6)) @ rng.standard_normal((6, 420)) + 1e-3 * rng.standard_normal((160, 420))
    x = torch.from_numpy(xv).float().cuda()
    xv = _np(x)
    want = layer.orthogonalise(xv, 5, [USUAL] * 5, 1e-7)
    assert np.linalg.norm(_np(op.orthogonalise(x)) - want) <= _orth_tol(want, 5, "f32")


# ---------------------------------------------------------------------------
# streams, graphs, repeated calls, large offsets
# ---------------------------------------------------------------------------

def _all_calls(op):
    """Each operator on inputs of its own: a list of (function, its results on the current stream)."""
    import torch
    q, _ = _rand(1, (50, 6, 64), "bf16")
    k, _ = _rand(2, (50, 2, 64), "bf16")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    freqs = torch.linspace(1, 0.001, 32).cuda()
    wq, _ = _rand(3, (64,), "f32", 0.1, 1.0)
    x, _ = _rand(4, (200, 128), "bf16")
    wg, _ = _rand(5, (264, 128), "bf16", 0.1)
    wu, _ = _rand(6, (264, 128), "bf16", 0.1)
    xf, wgf, wuf = x.float(), wg.float(), wu.float()
    d, _ = _rand(7, (200, 264), "bf16")
    r = op.gated_ffn(x, wg, wu, keep=True)
    rf = op.gated_ffn(xf, wgf, wuf, keep=True)
    one = x[:1].clone()
    m, _ = _rand(8, (3, 136, 200), "f32")
    a, _ = _rand(9, (8, 640), "f32")
    return [lambda **s: op.qk_norm_rope(q, k, pos, freqs, wq, wq, **s),
            lambda **s: op.qk_norm_rope_back(q, k, q, k, pos, freqs, wq, wq, **s),
            lambda **s: tuple(op.gated_ffn(x, wg, wu, keep=True, **s)),
            lambda **s: tuple(op.gated_ffn(xf, wgf, wuf, keep=True, **s)),
            lambda **s: (op.gated_ffn(one, wg, wu, **s).h,),
            lambda **s: op.gated_ffn_back(d, x, wg, wu, r.gate, r.up, **s),
            lambda **s: op.gated_ffn_back(d.float(), xf, wgf, wuf, rf.gate, rf.up, **s),
            lambda **s: (op.orthogonalise(m, **s),),
            lambda **s: (op.orthogonalise(a, **s),)]


def test_equal_calls_give_equal_bits_on_any_stream(op):
    import torch
    calls = _all_calls(op)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for c, w in zip(calls, want):
        with torch.cuda.stream(side):
            got = c()
        side.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, w))
        got = c(stream=side)
        side.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, w))


def test_calls_on_two_streams_at_once(op):
    import torch
    calls = _all_calls(op)
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = {}
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [c() for c in calls]
    torch.cuda.synchronize()
    for i in got:
        for r, w in zip(got[i], want):
            assert all(torch.equal(g, v) for g, v in zip(r, w))


def test_captured_and_replayed(op):
    import torch
    calls = _all_calls(op)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in calls]
    for _ in range(3):
        for r in got:
            for t in r:
                t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for r, w in zip(got, want):
            assert all(torch.equal(g, v) for g, v in zip(r, w))


def test_captured_over_two_streams(op):
    """A capture that forks to another stream and joins it: the results of one stream's calls feed the other's."""
    import torch
    x, _ = _rand(1, (300, 128), "bf16")
    wg, _ = _rand(2, (264, 128), "bf16", 0.1)
    wu, _ = _rand(3, (264, 128), "bf16", 0.1)
    m, _ = _rand(4, (96, 300), "f32")
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        a = op.orthogonalise(m)                                        # the longer one, on the first stream
        b0 = op.gated_ffn(x, wg, wu, keep=True)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = op.gated_ffn_back(b0.h, x, wg, wu, b0.gate, b0.up)
            c = op.gated_ffn(b[0], wg, wu)
        d = op.orthogonalise(a)
        main.wait_stream(side)
        e = op.gated_ffn(c.h[:, :128].contiguous(), wg, wu)            # first in its call, after both
        return [a, *b, c.h, d, e.h, op.orthogonalise(b[1].float())]

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_two_graphs_that_share_a_workspace(op):
    """Captured with one workspace of the caller's and replayed in turn."""
    import torch
    x, _ = _rand(1, (300, 128), "f32")
    w, _ = _rand(2, (264, 128), "f32", 0.1)
    m, _ = _rand(3, (2, 200, 264), "f32")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    calls = [lambda: op.gated_ffn(x, w, w, workspace=ws).h, lambda: op.orthogonalise(m, workspace=ws)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = c()
        graphs.append((g, r))
    for _ in range(3):
        for g, r in graphs:
            r.fill_(float("nan"))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r, v) for (_, r), v in zip(graphs, want))


def test_calls_from_two_threads(op):
    """Host threads, each with a stream of its own."""
    import threading
    import torch
    calls = _all_calls(op)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                for c, w in zip(calls, want):
                    got = c()
                    s.synchronize()
                    if not all(torch.equal(g, v) for g, v in zip(got, w)):
                        wrong.append(c)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_offsets_beyond_32_bits(op):
    """Rows more than 2^32 bytes apart from the first."""
    import torch
    T, D = 3, 64
    step = (1 << 31) + 64                                          # elements of 2 bytes between tokens
    big = torch.empty(2 * step + 4 * D, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(big, (T, 2, D), (step, D, 1))
    dense, _ = _rand(1, (T, 2, D), "bf16")
    q.copy_(dense)
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), torch.linspace(1, 0.1, D // 2).cuda()
    want = op.qk_norm_rope(dense, None, pos, freqs)[0]
    assert torch.equal(op.qk_norm_rope(q, None, pos, freqs, out_q=q)[0], want)
    x = torch.as_strided(big, (T, 2 * D), (step, 1))
    x.copy_(dense.view(T, 2 * D))
    w, _ = _rand(2, (40, 2 * D), "bf16", 0.1)
    assert torch.equal(op.gated_ffn(x, w, w).h, op.gated_ffn(dense.view(T, 2 * D), w, w).h)
    m = torch.as_strided(big, (T, 2, D), (step, D, 1))
    m.copy_(dense)
    want = op.orthogonalise(dense)
    assert torch.equal(op.orthogonalise(m), want)
    op.orthogonalise(dense, out=m)
    assert torch.equal(m, want)


def test_more_than_32_bits_of_bytes(op):
    """Results and inputs of more than 2^32 bytes: their last rows are those of a small call."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    T, H, D = 430000, 40, 128
    q = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), torch.linspace(1, 0.001, D // 2).cuda()
    want = op.qk_norm_rope(q[-3:].clone(), None, pos[-3:].clone(), freqs)[0]
    back = op.qk_norm_rope_back(q[-3:].clone(), None, q[-3:].clone(), None, pos[-3:].clone(), freqs, want_dw=False)[0]
    dx = op.qk_norm_rope_back(q, None, q, None, pos, freqs, want_dw=False)[0]
    assert torch.equal(dx[-3:], back)
    del dx
    assert torch.equal(op.qk_norm_rope(q, None, pos, freqs, out_q=q)[0][-3:], want)
    del q
    T, K, F = 36000, 64, 61000
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.empty((2, F, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    r = op.gated_ffn(x, w[0], w[1], keep=True)
    small = op.gated_ffn(x[-300:].clone(), w[0, -500:].clone(), w[1, -500:].clone(), keep=True)
    assert all(torch.equal(a[-300:, -500:], b) for a, b in zip(r, small))
    dx, dwg, dwu = op.gated_ffn_back(r.h, x, w[0], w[1], r.gate, r.up)
    assert torch.isfinite(dx).all() and torch.isfinite(dwg).all() and torch.isfinite(dwu).all()
    part = op.gated_ffn_back(r.h[:, -256:].clone(), x, w[0, -256:].clone(), w[1, -256:].clone(), r.gate[:, -256:].clone(),
                             r.up[:, -256:].clone(), want_dx=False)
    for a, b in ((dwg, part[1]), (dwu, part[2])):
        a, b = a[-256:].double(), b.double()
        assert float((a - b).norm()) <= 2.0 ** -8 * float(b.norm())
    del r, dx, x, w
    m = torch.empty((4200, 512, 512), device="cuda").normal_(generator=g)
    y = op.orthogonalise(m)
    assert torch.equal(y[-2:], op.orthogonalise(m[-2:].clone())) and torch.equal(y[:2], op.orthogonalise(m[:2].clone()))


def test_callers_workspace(op):
    """A workspace given by the caller, with garbage in it, and one too small."""
    import torch
    x, _ = _rand(4, (200, 128), "f32")
    w, _ = _rand(5, (264, 128), "f32", 0.1)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    r = op.gated_ffn(x, w, w, keep=True)
    assert torch.equal(op.gated_ffn(x, w, w, workspace=ws).h, r.h)
    d = torch.ones_like(r.h)
    for g, v in zip(op.gated_ffn_back(d, x, w, w, r.gate, r.up, workspace=ws), op.gated_ffn_back(d, x, w, w, r.gate, r.up)):
        assert torch.equal(g, v)
    assert torch.equal(op.orthogonalise(x, workspace=ws), op.orthogonalise(x))
    for call in (lambda: op.gated_ffn(x, w, w, workspace=ws[:256]), lambda: op.orthogonalise(x, workspace=ws[:256]),
                 lambda: op.gated_ffn_back(d, x, w, w, r.gate, r.up, workspace=ws[:256])):
        with pytest.raises(op.OopError):
            call()


def test_refused_by_the_binding(op):
    """Shapes, types and layouts that do not go together raise before anything is enqueued."""
    import torch
    q, k = torch.zeros(5, 4, 32, device="cuda"), torch.zeros(5, 2, 32, device="cuda")
    pos, freqs = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(16, device="cuda")
    x, w = torch.zeros(6, 16, device="cuda"), torch.zeros(24, 16, device="cuda")
    h = torch.zeros(6, 24, device="cuda")
    wide = torch.zeros(24, 20, device="cuda")[:, :16]
    for call in (lambda: op.qk_norm_rope(q, k[:4], pos, freqs), lambda: op.qk_norm_rope(q, k.half(), pos, freqs),
                 lambda: op.qk_norm_rope(q, k, pos[:4], freqs), lambda: op.qk_norm_rope(q, k, pos.long(), freqs),
                 lambda: op.qk_norm_rope(q, k, None, freqs), lambda: op.qk_norm_rope(q, k, pos, freqs, freqs),
                 lambda: op.qk_norm_rope(q[:, :, ::2], None, None, None), lambda: op.qk_norm_rope(q, k, pos, freqs, out_q=q[:4]),
                 lambda: op.qk_norm_rope(q.double(), None, None, None),
                 lambda: op.qk_norm_rope_back(q, None, q, k, pos, freqs), lambda: op.qk_norm_rope_back(q[:4], k, q, k, pos, freqs),
                 lambda: op.gated_ffn(x, w, w[:, :8]), lambda: op.gated_ffn(x, w, wide), lambda: op.gated_ffn(x, w, w, act="tanh"),
                 lambda: op.gated_ffn(x[:, :8], w, w), lambda: op.gated_ffn(x, w.double(), w.double()),
                 lambda: op.gated_ffn(x, w, w, out=h.half()), lambda: op.gated_ffn(x, w, w, w_type=op.TYPE_Q8_0),
                 lambda: op.gated_ffn_back(h[:5], x, w, w, h, h), lambda: op.gated_ffn_back(h, x, w, w, h.half(), h),
                 lambda: op.gated_ffn_back(h, x, w, w, h, torch.zeros(6, 30, device="cuda")[:, :24]),
                 lambda: op.orthogonalise(x, coefs=(1.0, 2.0)), lambda: op.orthogonalise(x, steps=2, coefs=[(1, 2, 3)] * 3),
                 lambda: op.orthogonalise(x.t()), lambda: op.orthogonalise(x, out=x[:5]), lambda: op.orthogonalise(x[0])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: op.qk_norm_rope_back(q.half(), None, q, None, pos, freqs), lambda: op.orthogonalise(x.half()),
                 lambda: op.gated_ffn_back(h.half(), x, w, w, h, h), lambda: op.qk_norm_rope(q, k, pos, freqs, eps=-1.0),
                 lambda: op.qk_norm_rope(q[..., :16], None, pos, freqs), lambda: op.orthogonalise(x, steps=65)):
        with pytest.raises(op.OopError):
            call()
