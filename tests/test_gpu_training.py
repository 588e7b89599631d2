"""GPU parity of the training operators against plain 64-bit implementations
(oracle/training.py), at the sizes, strides and masks where they can go wrong.

Tolerances follow from the arithmetic and are written before any run: u = 2^-24
is a rounding to fp32, UOUT one to the output's type, and a sum of n terms by
any chain of at most c additions is off by at most c * u * sum|terms|.  No sum
here has a chain longer than CHAIN(n) = n / 32 + 64 additions (a warp per row is
the least parallel form).
"""

import numpy as np
import pytest

import synth
from oracle import training as tr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UOUT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = 2.0 ** -126           # below this fp32 (and bf16) spacing is absolute; f16's is 2^-24
FLOOR = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def chain(n):
    return n / 32 + 64


@pytest.fixture(scope="module")
def op():
    import torch
    import ggml_out_prod_gb300 as g
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    g.build()
    g.lib()
    assert g.device_status(clear=True) in (g.OK, g.ERR_BAD_ID)
    return g


def _dt(kind):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]


def _rand(seed, shape, kind, std=1.0, mean=0.0):
    """(CUDA tensor of the type, its values in float64)."""
    import torch
    rng = np.random.default_rng(seed)
    t = torch.from_numpy(rng.standard_normal(shape) * std + mean).to(_dt(kind))
    return t.cuda(), t.double().numpy()


def _strided(t, how):
    """The same values at another layout: `pad` (rows apart by 3 more elements),
    `offset` (rows that start one element off any alignment), `wide` (rows apart
    by a multiple of 16 bytes)."""
    import torch
    T, M = t.shape
    if how == "dense":
        return t
    extra, at = {"pad": (3, 0), "offset": (5, 1), "wide": (64, 16)}[how]
    big = torch.full((T, M + extra), float("nan"), dtype=t.dtype, device=t.device)
    view = big[:, at:at + M]
    view.copy_(t)
    return view


def _close(got, want, tol, what):
    """Every element within its tolerance."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == np.shape(want), f"{what}: shape {got.shape}"
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if np.any(bad):
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(tol, 1e-300), 0)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {i} got {got[i]!r} "
                             f"want {np.asarray(want)[i]!r} tol {np.broadcast_to(tol, err.shape)[i]!r}")


# ---------------------------------------------------------------------------
# get_rows
# ---------------------------------------------------------------------------

TABLES = ["f32", "f16", "bf16"]
QUANTS = list(synth.QUANT_TYPES)


@pytest.mark.parametrize("kind", TABLES)
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,V,T", [(1, 1, 1), (7, 5, 9), (64, 100, 1), (129, 33, 70), (2560, 40, 17),
                                   (4104, 9, 3)])
def test_get_rows_plain(op, kind, out, M, V, T):
    import torch
    table, values = _rand(M + V, (V, M), kind)
    ids = np.random.default_rng(T).integers(0, V, T).astype(np.int32)
    y = op.get_rows(table, torch.from_numpy(ids).cuda(), scale=1.75, out_dtype=_dt(out))
    want = tr.get_rows(values, ids, 1.75)
    _close(y, want, (U + UOUT[out]) * np.abs(want) + FLOOR[out], "get_rows")


@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M", [7, 96, 1026, 2304])
def test_get_rows_of_many_tokens(op, kind, out, M):
    """Several tokens per CTA, the last of them fewer; ids outside among them."""
    import torch
    T, V = 2051, 301
    table, values = _rand(M, (V, M), kind)
    ids = np.random.default_rng(T).integers(-1, V + 1, T).astype(np.int32)
    y = op.get_rows(table, torch.from_numpy(ids).cuda(), scale=0.75, out_dtype=_dt(out))
    assert op.device_status(clear=True) == op.ERR_BAD_ID
    want = tr.get_rows(values, ids, 0.75)
    _close(y, want, (U + UOUT[out]) * np.abs(want) + FLOOR[out], "get_rows")


@pytest.mark.parametrize("kind", QUANTS)
@pytest.mark.parametrize("blocks", [1, 3, 10])
def test_get_rows_quantised(op, kind, blocks):
    import torch
    qk = synth.BLOCK[kind][0]
    M, V = qk * blocks, 37
    raw = synth.quantize(kind, synth.normal(kind + 40, V * M, std=0.3).reshape(V, M)).reshape(V, -1)
    values = tr.table_values(raw, kind, M)
    ids = np.array([0, 36, 5, 5, 17, -1, 37, 2 ** 31 - 1, -2 ** 31, 1], dtype=np.int32)
    for out in ("f32", "bf16"):
        y = op.get_rows(torch.from_numpy(raw).cuda(), torch.from_numpy(ids).cuda(), scale=0.5,
                        table_type=kind, out_dtype=_dt(out))
        assert op.device_status(clear=True) == op.ERR_BAD_ID
        want = tr.get_rows(values, ids, 0.5)
        # decoding: two products and one fused sum of up to 24 bits each
        _close(y, want, (4 * U + UOUT[out]) * np.abs(want) + 2 * U * 0.5 * np.abs(values).max() / 16,
               f"get_rows {kind}")
        assert (y[5:9] == 0).all()


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -2.0])
@pytest.mark.parametrize("T", [5, 2051])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                      (synth.TYPE_Q8_0, "f32"), (synth.TYPE_Q4_K, "bf16")])
def test_get_rows_ids_outside_are_zero_at_any_scale(op, kind, out, T, scale):
    import torch
    V, M = 9, 256
    type_id = None
    if kind in QUANTS:
        table = torch.zeros((V, M // synth.BLOCK[kind][0] * synth.BLOCK[kind][1]), dtype=torch.uint8, device="cuda")
        type_id = kind
    else:
        table, _ = _rand(3, (V, M), kind)
    ids = (torch.arange(T, dtype=torch.int32, device="cuda") % (V + 2)) - 1          # -1 .. V
    y = op.get_rows(table, ids, scale=scale, table_type=type_id, out_dtype=_dt(out))
    assert op.device_status(clear=True) == op.ERR_BAD_ID
    outside = y[(ids < 0) | (ids >= V)]
    assert (outside == 0).all() and not torch.signbit(outside).any()


@pytest.mark.parametrize("how", ["pad", "offset", "wide"])
@pytest.mark.parametrize("kind", TABLES)
def test_get_rows_strides(op, how, kind):
    """Rows of the table and of dst at other strides and alignments; what lies
    between dst's rows is not written."""
    import torch
    table, values = _rand(8, (50, 264), kind)
    ids = np.random.default_rng(9).integers(0, 50, (3, 11)).astype(np.int32)
    big = torch.full((33, 264 + 9), 7.0, dtype=_dt(kind), device="cuda")
    y = big[:, 1:265]
    op.get_rows(_strided(table, how), torch.from_numpy(ids.reshape(-1)).cuda(), out=y)
    _close(y, values[ids.reshape(-1)], 0.0, "copied rows")
    assert (big[:, 0] == 7).all() and (big[:, 265:] == 7).all()
    z = op.get_rows(table, torch.from_numpy(ids).cuda())
    assert z.shape == (3, 11, 264)


# ---------------------------------------------------------------------------
# get_rows_back
# ---------------------------------------------------------------------------

def _ids(seed, how, T, V):
    rng = np.random.default_rng(seed)
    if how == "uniform":
        return rng.integers(0, V, T).astype(np.int32)
    if how == "words":                       # frequencies fall as 1 / rank
        return np.clip(np.exp(rng.random(T) * np.log(V + 1.0)).astype(np.int64) - 1, 0, V - 1).astype(np.int32)
    if how == "one":
        return np.full(T, V // 2, dtype=np.int32)
    if how == "last":
        return np.full(T, V - 1, dtype=np.int32)
    if how == "falling":
        return (V - 1 - np.arange(T) % V).astype(np.int32)
    ids = rng.integers(-3, V + 3, T)         # some outside
    return np.where(ids % 5 == 0, rng.choice([-2 ** 31, 2 ** 31 - 1, V, -1], T), ids).astype(np.int32)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("how,T,V,M", [
    ("uniform", 1, 1, 1), ("uniform", 1, 1000, 8), ("words", 100, 50, 7), ("one", 1000, 3, 64),
    ("one", 2500, 700, 129), ("last", 33, 513, 132), ("words", 4097, 5000, 260), ("falling", 3000, 1024, 36),
    ("uniform", 9000, 300, 20), ("words", 20000, 70000, 12), ("outside", 700, 90, 65),
    ("one", 9001, 262145, 4), ("uniform", 40000, 17, 8)])
def test_get_rows_back(op, kind, how, T, V, M):
    import torch
    dy, dv = _rand(T, (T, M), kind)
    ids = _ids(M, how, T, V)
    d = op.get_rows_back(dy, torch.from_numpy(ids).cuda(), V, scale=1.5)
    bad = bool(((ids < 0) | (ids >= V)).any())
    assert op.device_status(clear=True) == (op.ERR_BAD_ID if bad else op.OK)
    want, mag, count = tr.get_rows_back(dv, ids, V, 1.5)
    _close(d, want, (np.minimum(count[:, None], 200) + count[:, None] / 16 + 8) * U * mag, "get_rows_back")
    again = op.get_rows_back(dy, torch.from_numpy(ids).cuda(), V, scale=1.5)
    assert op.device_status(clear=True) == (op.ERR_BAD_ID if bad else op.OK)
    assert torch.equal(d, again), "equal calls give equal bits"


def test_get_rows_back_accumulates(op):
    """With accumulate, rows that no id names keep their bits and the others
    take the sum."""
    import torch
    T, V, M = 600, 400, 33
    dy, dv = _rand(1, (T, M), "f32")
    ids = _ids(2, "words", T, V)
    start, sv = _rand(3, (V, M), "f32")
    d = start.clone()
    op.get_rows_back(dy, torch.from_numpy(ids).cuda(), V, scale=-0.5, out=d, accumulate=True)
    want, mag, count = tr.get_rows_back(dv, ids, V, -0.5)
    _close(d, want + sv, (count[:, None] + 9) * U * (mag + np.abs(sv)), "accumulated")
    untouched = torch.from_numpy(count == 0).cuda()
    assert torch.equal(d[untouched], start[untouched])


@pytest.mark.parametrize("how", ["pad", "offset", "wide"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_get_rows_back_strides(op, how, kind):
    import torch
    dy, dv = _rand(21, (300, 72), kind)
    ids = _ids(4, "words", 300, 40)
    d = op.get_rows_back(_strided(dy, how), torch.from_numpy(ids).cuda(), 40)
    want, mag, count = tr.get_rows_back(dv, ids, 40, 1.0)
    _close(d, want, (count[:, None] + 8) * U * mag, "strided dy")
    # one row of dy for every token: the gradient of a broadcast output
    one = dy[:1].expand(300, 72)
    d = op.get_rows_back(one, torch.from_numpy(ids).cuda(), 40)
    want, mag, count = tr.get_rows_back(np.repeat(dv[:1], 300, 0), ids, 40, 1.0)
    _close(d, want, (count[:, None] + 8) * U * mag, "broadcast dy")


def test_get_rows_back_empty(op):
    import torch
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    d = op.get_rows_back(torch.empty((0, 24), device="cuda"), none, 5)
    assert d.shape == (5, 24) and (d == 0).all()
    keep = torch.ones((5, 24), device="cuda")
    op.get_rows_back(torch.empty((0, 24), device="cuda"), none, 5, out=keep, accumulate=True)
    assert (keep == 1).all()
    assert op.get_rows(torch.ones((5, 24), device="cuda"), none).shape == (0, 24)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def _norm_tolerance(x, w, b, eps, mean, rstd, y, out):
    """Element tolerances of (y, mean, rstd)."""
    M = x.shape[1]
    c = chain(M)
    d_mean = (c + 1) * U * np.abs(x).mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    # (x - mean) is off by d_mean and one rounding; squares and their sum add 2u + c u
    d_var = (c + 4) * U * var + d_mean ** 2 + 2 * U * np.abs(mean) * np.sqrt(var)
    rel = 0.5 * d_var / (var + eps) + 4 * U
    xh = np.abs(x - mean[:, None]) * rstd[:, None]
    ww = 1.0 if w is None else np.abs(w)
    d_y = ww * (xh * (rel[:, None] + 4 * U) + (d_mean * rstd)[:, None])
    d_y = d_y + U * np.abs(y) + (0 if b is None else 2 * U * np.abs(b)) + UOUT[out] * (np.abs(y) + d_y)
    return d_y + FLOOR[out], d_mean, rel * rstd


WIDTHS = [1, 2, 7, 8, 33, 64, 127, 256, 513, 1000, 2560, 2561, 4096, 5120, 8200, 9728, 16384, 17408]


@pytest.mark.parametrize("T,M", [(1300, 333), (1300, 1001), (2500, 2560), (1217, 4100), (1250, 9000), (1216, 17409),
                                 (1300, 64)])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16")])
def test_layer_norm_of_many_rows(op, T, M, kind, out):
    """More rows than the SMs have warps for: the forms that go from row to row,
    aligned and not."""
    x, xv = _rand(M, (T, M), kind, 1.5, 0.4)
    w, wv = _rand(1, (M,), "f32", 0.3, 1.0)
    b, bv = _rand(2, (M,), "f32", 0.2)
    y, mean, rstd = op.layer_norm(x, w, b, eps=1e-5, out_dtype=_dt(out))
    want, m, r = tr.layer_norm(xv, wv, bv, 1e-5)
    tol = _norm_tolerance(xv, wv, bv, 1e-5, m, r, want, out)
    for got, w_, t_, what in zip((y, mean, rstd), (want, m, r), tol, ("y", "mean", "rstd")):
        _close(got, w_, t_, f"layer_norm {what} M={M} T={T}")


@pytest.mark.parametrize("how", ["pad", "offset", "wide"])
def test_layer_norm_of_many_strided_rows_in_place(op, how):
    """The same at other strides, written over the input: what lies between the
    rows (NaN) is neither used nor written."""
    import torch
    x, xv = _rand(5, (1500, 520), "bf16")
    want, m, r = tr.layer_norm(xv, None, None, 1e-5)
    tol = _norm_tolerance(xv, None, None, 1e-5, m, r, want, "bf16")[0]
    xs = _strided(x, how)
    y = op.layer_norm(xs)[0]
    _close(y, want, tol, "strided")
    assert torch.equal(op.layer_norm(xs, out=xs)[0], y)
    if xs._base is not None:
        assert int(torch.isnan(xs._base).sum()) == xs._base.numel() - x.numel()


@pytest.mark.parametrize("M", WIDTHS)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_layer_norm(op, M, kind):
    for T in (1, 5, 67):
        x, xv = _rand(M + T, (T, M), kind, 1.5, 0.4)
        w, wv = _rand(1, (M,), "f32", 0.3, 1.0)
        b, bv = _rand(2, (M,), "f32", 0.2)
        y, mean, rstd = op.layer_norm(x, w, b, eps=1e-5)
        want, m, r = tr.layer_norm(xv, wv, bv, 1e-5)
        tol = _norm_tolerance(xv, wv, bv, 1e-5, m, r, want, kind)
        for got, w_, t_, what in zip((y, mean, rstd), (want, m, r), tol, ("y", "mean", "rstd")):
            _close(got, w_, t_, f"layer_norm {what} M={M} T={T}")


@pytest.mark.parametrize("M", [31, 64000, 70001])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_layer_norm_types(op, M, out):
    """x and y of different types, weights of every type, either one missing."""
    for kind in ("f32", "f16", "bf16"):
        x, xv = _rand(M, (3, M), kind)
        for wk, has_w, has_b in (("bf16", 1, 1), ("f16", 1, 0), ("f32", 0, 1), ("f32", 0, 0)):
            w, wv = _rand(1, (M,), wk, 0.3, 1.0) if has_w else (None, None)
            b, bv = _rand(2, (M,), wk, 0.2) if has_b else (None, None)
            y, mean, rstd = op.layer_norm(x, w, b, eps=1e-3, out_dtype=_dt(out))
            want, m, r = tr.layer_norm(xv, wv, bv, 1e-3)
            tol = _norm_tolerance(xv, wv, bv, 1e-3, m, r, want, out)
            _close(y, want, tol[0], "y")
            _close(rstd, r, tol[2], "rstd")


@pytest.mark.parametrize("how", ["pad", "offset", "wide"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_norm_strides_and_in_place(op, how, kind):
    import torch
    x, xv = _rand(5, (9, 520), kind)
    want, m, r = tr.layer_norm(xv, None, None, 1e-5)
    tol = _norm_tolerance(xv, None, None, 1e-5, m, r, want, kind)[0]
    xs = _strided(x, how)
    y, _, _ = op.layer_norm(xs)
    _close(y, want, tol, "strided")
    z, _, _ = op.layer_norm(xs, out=xs)          # written over x
    assert z.data_ptr() == xs.data_ptr() and torch.equal(z, y)
    one = x[:1].expand(9, 520)                   # one row for all
    y, _, _ = op.layer_norm(one)
    _close(y, np.repeat(want[:1], 9, 0), tol[:1], "broadcast row")


@pytest.mark.parametrize("wk", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("at", [1, 4, 8])
@pytest.mark.parametrize("T", [3, 1300])
def test_layer_norm_weights_inside_a_larger_vector(op, T, at, kind, wk):
    """Rows on 16 bytes, w and b where a packed vector of parameters puts them:
    one, four and eight elements in."""
    M = 520
    x, xv = _rand(7, (T, M), kind, 1.5, 0.4)
    dy, dv = _rand(8, (T, M), kind, 2.0)
    flat, fv = _rand(9, (2 * M + at,), wk, 0.3, 1.0)
    w, b, wv, bv = flat[at:at + M], flat[at + M:], fv[at:at + M], fv[at + M:]
    y, mean, rstd = op.layer_norm(x, w, b, eps=1e-2)
    want, m, r = tr.layer_norm(xv, wv, bv, 1e-2)
    tol = _norm_tolerance(xv, wv, bv, 1e-2, m, r, want, kind)
    for got, w_, t_, what in zip((y, mean, rstd), (want, m, r), tol, ("y", "mean", "rstd")):
        _close(got, w_, t_, f"layer_norm {what} at={at}")
    mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    want = tr.layer_norm_back(dv, xv, mv, rv, wv)
    tol = _back_tolerance(dv, xv, mv, rv, wv, want[0], kind)
    for got, w_, t_, what in zip(op.layer_norm_back(dy, x, mean, rstd, w), want, tol, ("dx", "dw", "db")):
        _close(got, w_, t_, f"layer_norm_back {what} at={at}")


@pytest.mark.parametrize("T,M,kind", [(1300, 16384, "f16"), (1217, 13312, "bf16"), (1300, 9728, "f32"),
                                      (1300, 5128, "bf16")])
def test_layer_norm_of_many_wide_rows(op, T, M, kind):
    """Rows of which shared memory holds only a few at a time."""
    x, xv = _rand(M, (T, M), kind, 1.5, 0.4)
    w, wv = _rand(1, (M,), "f32", 0.3, 1.0)
    b, bv = _rand(2, (M,), "bf16", 0.2)
    y, mean, rstd = op.layer_norm(x, w, b.float(), eps=1e-5)
    want, m, r = tr.layer_norm(xv, wv, bv, 1e-5)
    tol = _norm_tolerance(xv, wv, bv, 1e-5, m, r, want, kind)
    for got, w_, t_, what in zip((y, mean, rstd), (want, m, r), tol, ("y", "mean", "rstd")):
        _close(got, w_, t_, f"layer_norm {what} M={M} T={T}")


def test_layer_norm_rows_far_from_zero(op):
    """A mean a thousand times the spread: the difference of squares would lose
    every digit."""
    x, xv = _rand(6, (4, 2560), "f32", 1.0, 1000.0)
    y, mean, rstd = op.layer_norm(x, eps=0.0)
    want, m, r = tr.layer_norm(xv, None, None, 0.0)
    tol = _norm_tolerance(xv, None, None, 0.0, m, r, want, "f32")
    _close(y, want, tol[0], "y")
    _close(rstd, r, tol[2], "rstd")


def test_layer_norm_nan_stays_in_its_row(op):
    import torch
    x = torch.randn((5, 300), device="cuda")
    x[2, 7] = float("nan")
    y, mean, rstd = op.layer_norm(x)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4]]).all()


def _back_tolerance(dy, x, mean, rstd, w, dx, out):
    M, T = x.shape[1], x.shape[0]
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    c = chain(M)
    mg, mgx = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    d = rstd[:, None] * (4 * U * np.abs(g) + (c + 6) * U * np.abs(g).mean(1, keepdims=True)
                         + np.abs(xh) * (c + 10) * U * np.abs(g * xh).mean(1, keepdims=True)
                         + 6 * U * (np.abs(mg) + np.abs(xh * mgx)))
    d = d + UOUT[out] * (np.abs(dx) + d) + FLOOR[out]
    c = T + 160
    return d, (c + 6) * U * np.abs(dy * xh).sum(0), c * U * np.abs(dy).sum(0)


@pytest.mark.parametrize("M", WIDTHS + [4099, 8195, 12289, 13001, 15361, 20001, 40000])
@pytest.mark.parametrize("kind,grad", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16"),
                                       ("bf16", "f32")])
def test_layer_norm_back(op, M, kind, grad):
    import torch
    for T in (1, 37, 403):
        if T * M > 4_000_000:
            continue
        x, xv = _rand(M + T, (T, M), kind, 1.5, 0.4)
        dy, dv = _rand(M + T + 1, (T, M), grad, 2.0)
        w, wv = _rand(1, (M,), "f32", 0.3, 1.0)
        _, mean, rstd = op.layer_norm(x, eps=1e-2)
        mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
        dx, dw, db = op.layer_norm_back(dy, x, mean, rstd, w)
        want = tr.layer_norm_back(dv, xv, mv, rv, wv)
        tol = _back_tolerance(dv, xv, mv, rv, wv, want[0], grad)
        for got, w_, t_, what in zip((dx, dw, db), want, tol, ("dx", "dw", "db")):
            _close(got, w_, t_, f"layer_norm_back {what} M={M} T={T}")
        again = op.layer_norm_back(dy, x, mean, rstd, w)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again)), "equal bits"


@pytest.mark.parametrize("how", ["pad", "offset", "wide"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_norm_back_strides(op, how, kind):
    import torch
    x, xv = _rand(31, (41, 264), kind)
    dy, dv = _rand(32, (41, 264), kind)
    _, mean, rstd = op.layer_norm(x)
    mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    want = tr.layer_norm_back(dv, xv, mv, rv, None)
    tol = _back_tolerance(dv, xv, mv, rv, None, want[0], kind)
    ds = _strided(dy, how)
    dx, dw, db = op.layer_norm_back(ds, _strided(x, how), mean, rstd)
    _close(dx, want[0], tol[0], "dx")
    _close(dw, want[1], tol[1], "dw")
    _close(db, want[2], tol[2], "db")
    only, none_w, b2 = op.layer_norm_back(ds, x, mean, rstd, want_dw=False)
    assert none_w is None and torch.equal(b2, db) and torch.equal(only, dx)
    none = op.layer_norm_back(ds, x, mean, rstd, want_dw=False, want_db=False)
    assert none[1] is None and none[2] is None and torch.equal(none[0], dx)
    over = op.layer_norm_back(ds, x, mean, rstd, out=ds)[0]      # written over dy
    assert over.data_ptr() == ds.data_ptr() and torch.equal(over, dx)


@pytest.mark.parametrize("T,M,kind,grad", [(4001, 333, "bf16", "bf16"), (3000, 1024, "bf16", "bf16"),
                                           (2000, 1025, "f32", "f32"), (1500, 4099, "f16", "f32"), (1000, 5120, "f32", "bf16"),
                                           (900, 9000, "bf16", "bf16"), (5000, 17, "f32", "f32")])
def test_layer_norm_back_rows_in_turn(op, T, M, kind, grad):
    """Every thread group takes several rows; written over dy as well."""
    import torch
    x, xv = _rand(M + T, (T, M), kind, 1.5, 0.4)
    dy, dv = _rand(M + T + 1, (T, M), grad, 2.0)
    w, wv = _rand(1, (M,), "bf16", 0.3, 1.0)
    _, mean, rstd = op.layer_norm(x, eps=1e-2)
    mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    got = op.layer_norm_back(dy, x, mean, rstd, w)
    want = tr.layer_norm_back(dv, xv, mv, rv, wv)
    tol = _back_tolerance(dv, xv, mv, rv, wv, want[0], grad)
    for g, w_, t_, what in zip(got, want, tol, ("dx", "dw", "db")):
        _close(g, w_, t_, f"layer_norm_back {what} M={M} T={T}")
    over = op.layer_norm_back(dy, x, mean, rstd, w, out=dy)
    assert all(torch.equal(p, q) for p, q in zip(got, over))


@pytest.mark.parametrize("M,kind,grad", [(11501, "f32", "f32"), (12001, "f32", "f32"), (12289, "bf16", "bf16"),
                                          (20001, "bf16", "bf16"), (12305, "f16", "f32"), (16392, "f32", "f32"),
                                          (16392, "bf16", "bf16"), (20480, "f32", "bf16"), (16384, "bf16", "bf16")])
def test_layer_norm_back_of_wide_rows_over_dy(op, M, kind, grad):
    """dx written over dy changes neither dw nor db, on both sides of the widths
    that one pass holds."""
    import torch
    x, xv = _rand(M, (37, M), kind, 1.5, 0.4)
    dy, dv = _rand(M + 1, (37, M), grad, 2.0)
    w, wv = _rand(1, (M,), "f32", 0.3, 1.0)
    _, mean, rstd = op.layer_norm(x, eps=1e-2)
    mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    apart = op.layer_norm_back(dy, x, mean, rstd, w)
    over = op.layer_norm_back(dy, x, mean, rstd, w, out=dy)
    assert over[0].data_ptr() == dy.data_ptr()
    want = tr.layer_norm_back(dv, xv, mv, rv, wv)
    tol = _back_tolerance(dv, xv, mv, rv, wv, want[0], grad)
    for a, o, w_, t_, what in zip(apart, over, want, tol, ("dx", "dw", "db")):
        _close(o, w_, t_, f"layer_norm_back over dy: {what} M={M}")
        assert torch.equal(a, o), what


@pytest.mark.parametrize("M", [264, 12377])
@pytest.mark.parametrize("how", ["dense", "pad", "offset", "wide"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_norm_back_over_strided_dy(op, kind, how, M):
    import torch
    x, _ = _rand(33, (41, M), kind)
    dy, _ = _rand(34, (41, M), kind)
    _, mean, rstd = op.layer_norm(x)
    ds = _strided(dy, how)
    apart = op.layer_norm_back(ds, x, mean, rstd)
    over = op.layer_norm_back(ds, x, mean, rstd, out=ds)
    assert over[0].data_ptr() == ds.data_ptr()
    assert all(torch.equal(a, o) for a, o in zip(apart, over))


def test_layer_norm_back_many_rows(op):
    """More rows than any launch has CTAs, few columns; and no rows at all."""
    import torch
    x, xv = _rand(33, (30011, 48), "bf16")
    dy, dv = _rand(34, (30011, 48), "f32")
    _, mean, rstd = op.layer_norm(x)
    mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    dx, dw, db = op.layer_norm_back(dy, x, mean, rstd)
    want = tr.layer_norm_back(dv, xv, mv, rv, None)
    tol = _back_tolerance(dv, xv, mv, rv, None, want[0], "f32")
    _close(dx, want[0], tol[0], "dx")
    _close(dw, want[1], tol[1], "dw")
    _close(db, want[2], tol[2], "db")
    e = torch.empty((0, 48), device="cuda")
    s = torch.empty(0, device="cuda")
    dx, dw, db = op.layer_norm_back(e, e, s, s)
    assert dx.shape == (0, 48) and (dw == 0).all() and (db == 0).all()
    assert op.layer_norm(e)[0].shape == (0, 48)


@pytest.mark.parametrize("spread", [1e-20, 1e-25, 1e19])
@pytest.mark.parametrize("M", [264, 333, 5120, 12377])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_layer_norm_back_of_tiny_and_huge_spread(op, spread, M, grad):
    """Rows whose rstd is a float but whose rstd squared is none, or has lost its
    digits: every product of the formula's own order stays in range."""
    import torch
    x, xv = _rand(M, (5, M), "f32", spread, 0.3 * spread)
    dy, dv = _rand(M + 1, (5, M), grad, 1e-3)
    _, m, r = tr.layer_norm(xv, None, None, 0.0)
    mean, rstd = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (m, r))
    mv, rv = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    got = op.layer_norm_back(dy, x, mean, rstd)
    want = tr.layer_norm_back(dv, xv, mv, rv, None)
    tol = _back_tolerance(dv, xv, mv, rv, None, want[0], grad)
    for g, w_, t_, what in zip(got, want, tol, ("dx", "dw", "db")):
        _close(g, w_, t_, f"layer_norm_back {what} M={M} spread={spread}")


def test_layer_norm_gradient_by_differences(op):
    """The GPU's own forward pass, differenced: along a direction v,
    (L(x + h v) - L(x - h v)) / 2h for L = <y, dy> is <dx, v> to O(h^2) and the
    forward's rounding over h."""
    x, xv = _rand(41, (6, 200), "f32")
    dy, dv = _rand(42, (6, 200), "f32")
    v, vv = _rand(43, (6, 200), "f32")
    w, wv = _rand(44, (200,), "f32", 0.2, 1.0)
    h = 2.0 ** -6
    ya = op.layer_norm(x + h * v, w)[0].double().cpu().numpy()
    yb = op.layer_norm(x - h * v, w)[0].double().cpu().numpy()
    _, mean, rstd = op.layer_norm(x, w)
    dx = op.layer_norm_back(dy, x, mean, rstd, w)[0].double().cpu().numpy()
    got, want = (dx * vv).sum(), ((ya - yb) * dv).sum() / (2 * h)
    # third derivatives of a unit-scale norm along a unit-scale direction are below ~10 per element;
    # the forward is off by ~70 u per element of size ~1 (chain of 200 / 32 + 64)
    tol = h * h / 6 * 10 * np.abs(dv).sum() / 10 + 70 * U * np.linalg.norm(dv) / h
    assert abs(got - want) <= tol, (got, want, tol)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,M", [(1, 1), (3, 7), (2, 8), (5, 64), (17, 129), (4, 1000), (9, 264), (2, 2561), (3, 1002), (40, 30),
                                 (1, 258)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(op, kind, T, M, p):
    seed, offset = 0xFEDCBA9876543210, 0x8000000000000005
    x, xv = _rand(T * M, (T, M), kind)
    y = op.dropout(x, p, seed, offset)
    want = tr.dropout(xv, p, seed, offset)
    _close(y, want, (2 * U + UOUT[kind]) * np.abs(want) + (FLOOR[kind] if p < 1 else 0) * (want != 0), "dropout")


@pytest.mark.parametrize("how", ["dense", "pad", "offset", "wide"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_dropout_layouts_share_one_mask(op, how, kind):
    """The mask depends on the position alone: other strides, another type, a
    slice of the rows and the backward pass all drop the same elements."""
    import torch
    x, xv = _rand(3, (11, 520), kind, 0.1, 3.0)
    keep = tr.dropout_keep(11, 520, 0.3, 77, 5)
    y = op.dropout(_strided(x, how), 0.3, 77, 5)
    assert ((y != 0).cpu().numpy() == keep).all()
    dy = op.dropout_back(_strided(x, how), 0.3, 77, 5)
    assert torch.equal(dy, y)
    part = op.dropout(_strided(x, how)[:4, :263], 0.3, 77, 5)
    assert torch.equal(part, y[:4, :263])
    z = _strided(x, how)
    assert torch.equal(op.dropout(z, 0.3, 77, 5, out=z), y)      # in place
    other = op.dropout(x, 0.3, 77, 6)
    assert not torch.equal(other, y)


def test_dropout_counts_from_the_first_row_and_column_of_the_call(op):
    """A part that starts elsewhere is masked as if it started at 0, forward and
    backward; with an offset of its own it has a mask of its own."""
    import torch
    x = torch.ones((11, 520), device="cuda")
    keep = torch.from_numpy(tr.dropout_keep(11, 520, 0.3, 77, 5)).cuda()
    for part in (x[5:], x[:, 16:], x[2:9, 3:]):
        rows, cols = part.shape
        y = op.dropout(part, 0.3, 77, 5)
        assert ((y != 0) == keep[:rows, :cols]).all()
        assert torch.equal(op.dropout_back(part, 0.3, 77, 5), y)
        assert not torch.equal(op.dropout(part, 0.3, 77, 6), y)


def test_dropout_of_infinities(op):
    """A dropped element is zero whatever it held; a kept one stays."""
    import torch
    x = torch.full((3, 4000), float("nan"), device="cuda")
    y = op.dropout(x, 0.5, 1)
    keep = torch.from_numpy(tr.dropout_keep(3, 4000, 0.5, 1, 0)).cuda()
    assert (y[~keep] == 0).all() and torch.isnan(y[keep]).all()


def test_dropout_three_dimensions(op):
    import torch
    x = torch.ones((4, 6, 40), device="cuda")
    y = op.dropout(x, 0.25, 9, 1)
    keep = torch.from_numpy(tr.dropout_keep(24, 40, 0.25, 9, 1)).cuda().view(4, 6, 40)
    assert ((y != 0) == keep).all()
    assert op.dropout(x[:0], 0.25, 9, 1).shape == (0, 6, 40)


# ---------------------------------------------------------------------------
# preference loss
# ---------------------------------------------------------------------------

def _lse_tolerance(x):
    """Of log sum exp: each term's argument is off by two roundings of |x - top| * log2(e)
    and its exponential by 2^-22; the sum's chain is at most 512 additions or joins of
    relative error 4u each."""
    with np.errstate(invalid="ignore"):
        d = np.where(np.isinf(x), 0.0, x.max(1, keepdims=True) - x)
        p = np.exp(-d) * ~np.isinf(x)
    p = p / p.sum(1, keepdims=True)
    return 2.0 ** -22 + (p * d).sum(1) * 4 * U + 512 * 4 * U


def _pairs(seed, lengths, V, kind, std=2.0, scored=0.75):
    import torch
    rng = np.random.default_rng(seed)
    T = sum(lengths)
    x, xv = _rand(seed, (T, V), kind, std)
    labels = rng.integers(0, V, T).astype(np.int32)
    labels[rng.random(T) >= scored] = -1
    seq = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    ref = (-np.log(V) + rng.standard_normal(T)).astype(np.float32)
    cuda = [torch.from_numpy(v).cuda() for v in (labels, seq, ref)]
    return x, xv, labels, seq, ref, cuda


def _check_forward(op, r, xv, labels, seq, ref, beta, e):
    loss, losses, ratios, logps, lse = tr.preference_loss(xv, labels, seq, None if ref is None else ref.astype(np.float64), beta, e)
    use = (labels >= 0) & (labels < xv.shape[1])
    t_lse = np.where(use, _lse_tolerance(xv) + 2 * U * np.abs(lse), 0.0)
    _close(r.lse, lse, t_lse, "lse")
    t_logp = np.where(use, t_lse + 2 * U * np.abs(logps), 0.0)
    _close(r.logps, logps, t_logp, "logps")
    P = len(losses)
    t_ratio = np.array([t_logp[a:b].sum() for a, b in zip(seq[:-1], seq[1:])]) + 2 * U * np.abs(ratios) + 1e-12
    _close(r.ratios, ratios, t_ratio, "ratios")
    t_loss = abs(beta) * (t_ratio[:P] + t_ratio[P:]) + 4 * U * losses + 1e-7
    _close(r.losses, losses, t_loss, "losses")
    _close(r.loss, loss, t_loss.mean() + 4 * U * loss, "loss")


def _check_backward(op, d, xv, labels, seq, lse, ratios, beta, e, out, dloss=1.0):
    lse, ratios = lse.double().cpu().numpy(), ratios.double().cpu().numpy()
    want, coef = tr.preference_loss_back(xv, labels, seq, lse, ratios, beta, e, dloss)
    with np.errstate(invalid="ignore", over="ignore"):
        t = np.where(np.isinf(xv), 0.0, np.abs(xv - lse[:, None]))
        p = np.where(np.isinf(xv), 0.0, np.exp(np.minimum(xv - lse[:, None], 50)))
        tol = np.abs(coef[:, None]) * (p * (2.0 ** -22 + 4 * U * t + 4 * U) + 4 * U * np.abs(1.0 * (want != 0)))
    tol = np.where(coef[:, None] == 0, 0.0, tol + UOUT[out] * (np.abs(want) + tol) + FLOOR[out])
    _close(d, want, tol, "dlogits")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 32, 255, 1000, 4099, 8192, 16384, 16385, 33001])
def test_preference_loss(op, kind, V):
    import torch
    for lengths in ([1, 1], [3, 1, 5, 2], [9, 0, 4, 6, 2, 11]):
        x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(V + len(lengths), lengths, V, kind)
        for rf, trf, e in ((ref, tr_, 0.0), (None, None, 0.2)):
            r = op.preference_loss(x, tl, ts, trf, beta=0.3, label_smoothing=e)
            assert op.device_status(clear=True) == op.OK
            _check_forward(op, r, xv, labels, seq, rf, 0.3, e)
            for out in ("f32", "bf16"):
                d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.3, label_smoothing=e,
                                            out_dtype=_dt(out))
                _check_backward(op, d, xv, labels, seq, r.lse, r.ratios, 0.3, e, out)
        again = op.preference_loss(x, tl, ts, trf, beta=0.3, label_smoothing=e)
        assert all(torch.equal(a, b) for a, b in zip(r, again)), "equal bits"


@pytest.mark.parametrize("how", ["pad", "offset", "wide"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_preference_strides_and_in_place(op, how, kind):
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(50, [4, 7, 3, 5], 1003, kind)
    xs = _strided(x, how)
    r = op.preference_loss(xs, tl, ts, tr_, beta=0.2)
    _check_forward(op, r, xv, labels, seq, ref, 0.2, 0.0)
    d = op.preference_loss_back(xs, tl, ts, r.lse, r.ratios, beta=0.2)
    _check_backward(op, d, xv, labels, seq, r.lse, r.ratios, 0.2, 0.0, kind)
    other = torch.full((19, 1003 + 6), 7.0, dtype=_dt(kind), device="cuda")
    op.preference_loss_back(xs, tl, ts, r.lse, r.ratios, beta=0.2, out=other[:, 2:1005])
    assert torch.equal(other[:, 2:1005], d) and (other[:, :2] == 7).all() and (other[:, 1005:] == 7).all()
    op.preference_loss_back(xs, tl, ts, r.lse, r.ratios, beta=0.2, out=xs)   # over the logits
    assert torch.equal(xs, d)


def test_preference_masked_rows_are_not_read(op):
    """NaN and infinities in rows that are not scored change nothing; a pair with
    nothing scored has loss log 2 and no gradient."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(51, [5, 4, 6, 3], 300, "f32")
    labels[5:9] = -1                 # the second chosen sequence, and its rejected one
    labels[15:] = -7
    labels[0] = 4
    tl = torch.from_numpy(labels).cuda()
    for bad in (float("nan"), float("inf"), -float("inf")):
        x[tl < 0] = bad
        tr_[tl < 0] = float("nan")
        r = op.preference_loss(x, tl, ts, tr_, beta=0.5)
        _check_forward(op, r, xv, labels, seq, ref, 0.5, 0.0)
        assert abs(float(r.losses[1]) - np.log(2)) < 1e-6 and float(r.ratios[1]) == 0.0
        d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.5)
        assert (d[tl < 0] == 0).all() and torch.isfinite(d).all()


@pytest.mark.parametrize("low", ["inf", "lowest"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_preference_masked_vocabulary(op, low, kind):
    """Logits at -Inf or at the type's lowest value: probability 0, gradient 0;
    and whole spans of a row masked, so that some threads see nothing else."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(52, [4, 5], 40000, kind, scored=1.0)
    value = -float("inf") if low == "inf" else torch.finfo(_dt(kind)).min
    x[:, 100:30000] = value
    x[2, 1:] = value
    x[3, :-1] = value
    labels = np.where(np.arange(9) % 2 == 0, 0, 39999).astype(np.int32)
    labels[2], labels[3] = 0, 39999
    tl = torch.from_numpy(labels).cuda()
    xv = x.double().cpu().numpy()
    r = op.preference_loss(x, tl, ts, tr_, beta=0.5)
    _check_forward(op, r, xv, labels, seq, ref, 0.5, 0.0)
    d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.5)
    assert torch.isfinite(d).all() and (d[:, 100:30000] == 0).all()
    _check_backward(op, d, xv, labels, seq, r.lse, r.ratios, 0.5, 0.0, "f32" if kind == "f16" else kind)


def test_preference_rows_of_one_value(op):
    """A row whose every logit is the type's lowest value is uniform; one of -Inf
    alone has no distribution (lse -Inf)."""
    import torch
    lowest = torch.finfo(torch.float32).min
    x = torch.full((2, 5000), lowest, device="cuda")
    x[1] = -float("inf")
    labels = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    logps, lse = op.token_logps(x, labels)
    assert abs(float(logps[0]) + np.log(5000)) < 1e-5 and float(lse[0]) == lowest
    assert float(lse[1]) == -float("inf") and bool(torch.isnan(logps[1]))


def test_preference_large_logits(op):
    """Logits of 1e4 and a label far below the top: no overflow, finite loss."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(53, [3, 3], 2000, "f32", std=3e3, scored=1.0)
    r = op.preference_loss(x, tl, ts, tr_, beta=0.01)
    _check_forward(op, r, xv, labels, seq, ref, 0.01, 0.0)
    d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.01)
    assert torch.isfinite(d).all()


def test_preference_nan_in_a_scored_row(op):
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(54, [3, 3], 500, "f32", scored=1.0)
    x[1, 77] = float("nan")
    r = op.preference_loss(x, tl, ts, tr_)
    assert torch.isnan(r.lse[1]) and torch.isnan(r.ratios[0]) and torch.isnan(r.loss)
    assert torch.isfinite(r.ratios[1])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("how", ["dense", "pad", "offset"])
@pytest.mark.parametrize("V", [5, 37, 300])
def test_preference_infinite_logit_anywhere(op, V, how, kind):
    """A logit of +Inf in a scored row makes the row NaN wherever in the row it
    lies, and with it the pair's loss, chosen or rejected."""
    import torch
    x, _ = _rand(V, (V + 1, V), kind)
    x[torch.arange(V), torch.arange(V)] = float("inf")       # row v has it at v; the last row has none
    x = _strided(x, how)
    labels = torch.full((V + 1,), V // 2, dtype=torch.int32, device="cuda")
    logps, lse = op.token_logps(x, labels)
    assert torch.isnan(lse[:V]).all() and torch.isnan(logps[:V]).all()
    assert torch.isfinite(lse[V]) and torch.isfinite(logps[V])
    for row in (0, V - 1):
        two = x[[row, V]]
        for seq in ([0, 1, 2], [0, 2, 2]):
            ts = torch.tensor(seq, dtype=torch.int32, device="cuda")
            for pair in (two, two.flip(0)):
                r = op.preference_loss(pair, labels[:2], ts)
                assert torch.isnan(r.losses[0]) and torch.isnan(r.loss), (row, seq)


def test_preference_bad_labels_and_offsets(op):
    """A label beyond the vocabulary is not scored; offsets out of order or
    beyond the rows are clamped; both set the device status."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(55, [3, 4], 50, "f32", scored=1.0)
    labels[1] = 50
    r = op.preference_loss(x, torch.from_numpy(labels).cuda(), ts, tr_, beta=0.4)
    assert op.device_status(clear=True) == op.ERR_BAD_ID
    _check_forward(op, r, xv, labels, seq, ref, 0.4, 0.0)
    d = op.preference_loss_back(x, torch.from_numpy(labels).cuda(), ts, r.lse, r.ratios, beta=0.4)
    assert op.device_status(clear=True) == op.ERR_BAD_ID and (d[1] == 0).all()
    for bad in ([0, 3, 900], [-5, 3, 7], [3, 1, 7], [2 ** 31 - 1, 0, -2 ** 31]):
        r = op.preference_loss(x, tl, torch.tensor(bad, dtype=torch.int32, device="cuda"), tr_)
        assert op.device_status(clear=True) == op.ERR_BAD_ID
        op.preference_loss_back(x, tl, torch.tensor(bad, dtype=torch.int32, device="cuda"), r.lse, r.ratios)
        torch.cuda.synchronize()


def test_preference_rows_outside_every_sequence(op):
    """Rows before the first sequence and after the last have logps but no part
    in a ratio and no gradient."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(56, [2, 3, 4, 2], 60, "f32", scored=1.0)
    seq = np.array([2, 5, 9], dtype=np.int32)
    ts = torch.from_numpy(seq).cuda()
    r = op.preference_loss(x, tl, ts, tr_, beta=0.4)
    _check_forward(op, r, xv, labels, seq, ref, 0.4, 0.0)
    d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.4)
    _check_backward(op, d, xv, labels, seq, r.lse, r.ratios, 0.4, 0.0, "f32")
    assert (d[:2] == 0).all() and (d[9:] == 0).all() and (r.lse != 0).all()


@pytest.mark.parametrize("kind,V", [("bf16", 20001), ("f32", 9000)])
def test_preference_many_rows(op, kind, V):
    """Enough rows that a CTA takes several steps of one."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(63, [400, 333, 420, 411], V, kind, scored=0.6)
    r = op.preference_loss(x, tl, ts, tr_, beta=0.05)
    _check_forward(op, r, xv, labels, seq, ref, 0.05, 0.0)
    d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.05)
    _check_backward(op, d, xv, labels, seq, r.lse, r.ratios, 0.05, 0.0, kind)
    assert torch.equal(op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.05, out=x), d)


def test_preference_many_pairs(op):
    """More pairs than threads of a CTA, short sequences."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(57, [1 + i % 3 for i in range(2 * 700)], 40, "f32")
    g = torch.tensor(2.5, device="cuda")
    r = op.preference_loss(x, tl, ts, tr_, beta=0.1, label_smoothing=0.05)
    _check_forward(op, r, xv, labels, seq, ref, 0.1, 0.05)
    d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.1, label_smoothing=0.05, dloss=g)
    _check_backward(op, d, xv, labels, seq, r.lse, r.ratios, 0.1, 0.05, "f32", dloss=2.5)


def test_preference_ratio_is_summed_in_more_than_32_bits(op):
    """Differences of 1e4 that cancel: with one logit a row's log probability is
    0, so the ratio is minus the sum of ref_logps.  A sum in 32 bits loses about
    0.03 here.  What the kernel may lose: the logarithm of a half to one ulp, 2^-24,
    for each row; of the low parts (2^-24 of at most 2^17 each, 16 in all), 22
    roundings; and the rounding of the result."""
    import torch
    n = 4096
    rng = np.random.default_rng(70)
    half = (rng.standard_normal(n // 2) * 1e4).astype(np.float32)
    ref = np.concatenate([half, -half + rng.standard_normal(n // 2).astype(np.float32), [0.0]]).astype(np.float32)
    x, _ = _rand(71, (n + 1, 1), "f32")
    labels = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
    r = op.preference_loss(x, labels, seq, torch.from_numpy(ref).cuda())
    want = -ref[:n].astype(np.float64).sum()
    tol = n * 2.0 ** -24 + 22 * U * 16 + U * abs(want)
    assert abs(float(r.ratios[0]) - want) <= tol, (float(r.ratios[0]), want, tol)


def test_preference_logps_are_not_biased(op):
    """Over many rows the errors of the log probabilities average out: the
    fast exponential's mean error (5e-8 of each term) is taken back, and so is what
    log2 e in one term would cost (1.3e-8 times the distance to the top, 6
    here).  The bound is half of the smaller of the two.  ref_logps are the exact
    values rounded, so the ratio is the sum of the errors."""
    import torch
    n, V = 1536, 8191
    rng = np.random.default_rng(72)
    xv = rng.standard_normal((n + 1, V)).astype(np.float32)
    labels = rng.integers(0, V - 1, n + 1).astype(np.int32)
    xv[:, V - 1] = rng.uniform(6.5, 7.5, n + 1)
    x64 = xv.astype(np.float64)
    top = x64.max(1, keepdims=True)
    logps = x64[np.arange(n + 1), labels] - top[:, 0] - np.log(np.exp(x64 - top).sum(1))
    ref = logps.astype(np.float32)
    seq = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
    r = op.preference_loss(torch.from_numpy(xv).cuda(), torch.from_numpy(labels).cuda(), seq, torch.from_numpy(ref).cuda())
    mean = (float(r.ratios[0]) - (logps[:n] - ref[:n]).sum()) / n
    assert abs(mean) <= 2.5e-8, mean


def test_preference_without_pairs_or_rows(op):
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(58, [300, 301], 130, "bf16")
    logps, lse = op.token_logps(x, tl)
    r = op.preference_loss(x, tl, ts, tr_)
    assert torch.equal(logps, r.logps) and torch.equal(lse, r.lse)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = op.preference_loss(x, tl, none)
    assert float(e.loss) == 0 and e.losses.numel() == 0 and torch.equal(e.logps, logps)
    assert (op.preference_loss_back(x, tl, none, lse, e.ratios) == 0).all()
    no_rows = torch.empty((0, 130), device="cuda")
    no_ids = torch.empty(0, dtype=torch.int32, device="cuda")
    r = op.preference_loss(no_rows, no_ids, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert abs(float(r.loss) - np.log(2)) < 1e-6 and (r.ratios == 0).all()


def test_preference_gradient_by_differences(op):
    """The GPU's own loss differenced along a direction."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(59, [4, 5], 64, "f32", scored=1.0)
    v, vv = _rand(60, (9, 64), "f32")
    h = 2.0 ** -5
    la = op.preference_loss(x + h * v, tl, ts, tr_, beta=0.5)
    lb = op.preference_loss(x - h * v, tl, ts, tr_, beta=0.5)
    r = op.preference_loss(x, tl, ts, tr_, beta=0.5)
    d = op.preference_loss_back(x, tl, ts, r.lse, r.ratios, beta=0.5).double().cpu().numpy()
    got, want = (d * vv).sum(), (float(la.loss) - float(lb.loss)) / (2 * h)
    # third derivative along v: at most beta * rows * |v|^3-type moments, ~0.5 * 9 * 30;
    # the losses are off by ~1e-6 each
    tol = h * h / 6 * 0.5 * 9 * 30 + 2e-6 / h
    assert abs(got - want) <= tol, (got, want, tol)


# ---------------------------------------------------------------------------
# streams, refusals
# ---------------------------------------------------------------------------

def test_calls_on_another_stream(op):
    """Every call on a stream of its own gives the bits of the default stream."""
    import torch
    x, xv, labels, seq, ref, (tl, ts, tr_) = _pairs(61, [40, 41], 3000, "bf16")
    w = torch.ones(3000, device="cuda")
    ids = torch.arange(81, dtype=torch.int32, device="cuda") % 50
    st = torch.cuda.Stream()

    def everything(stream):
        out = []
        y, mean, rstd = op.layer_norm(x, w, eps=1e-5, stream=stream)
        out += [y, mean, rstd]
        out += list(op.layer_norm_back(x, x, mean, rstd, w, stream=stream))
        out += [op.dropout(x, 0.5, 3, stream=stream), op.dropout_back(x, 0.5, 3, stream=stream)]
        out += [op.get_rows(x, ids, stream=stream), op.get_rows_back(x, ids, 50, stream=stream)]
        r = op.preference_loss(x, tl, ts, tr_, stream=stream)
        out += list(r) + [op.preference_loss_back(x, tl, ts, r.lse, r.ratios, stream=stream)]
        return out

    here = everything(None)
    torch.cuda.synchronize()
    there = everything(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(here, there))


def test_calls_in_a_graph(op):
    """Captured once, replayed on new inputs."""
    import torch
    x, _, labels, _, _, (tl, ts, tr_) = _pairs(62, [20, 21], 2000, "f32")
    ids = torch.arange(41, dtype=torch.int32, device="cuda") % 7

    def step():
        y, mean, rstd = op.layer_norm(x)
        back = op.layer_norm_back(y, x, mean, rstd)
        r = op.preference_loss(y, tl, ts, tr_)
        d = op.preference_loss_back(y, tl, ts, r.lse, r.ratios)
        return [y, *back, op.dropout(d, 0.5, 1), op.get_rows_back(d, ids, 9), r.loss]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    x.copy_(torch.randn_like(x))
    g.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals_reach_the_caller(op):
    import torch
    h = torch.ones((4, 16), dtype=torch.float16, device="cuda")
    f = torch.ones((4, 16), device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    s = torch.zeros(4, device="cuda")
    for call in (lambda: op.dropout_back(h, 0.1, 1), lambda: op.get_rows_back(h, i, 3),
                 lambda: op.layer_norm_back(h, f, s, s),
                 lambda: op.preference_loss_back(f, i, i[:3], s, s[:2], out_dtype=torch.float16)):
        with pytest.raises(op.OopError) as e:
            call()
        assert e.value.status == op.ERR_TYPE           # no gradient is ever binary16
    for call in (lambda: op.dropout(f, 1.5, 1), lambda: op.dropout(f, float("nan"), 1),
                 lambda: op.layer_norm(f, eps=-1.0), lambda: op.layer_norm(f, eps=float("nan")),
                 lambda: op.preference_loss(f, i, i[:3], beta=float("inf")),
                 lambda: op.preference_loss(f, i, i[:3], label_smoothing=1.5)):
        with pytest.raises(op.OopError) as e:
            call()
        assert e.value.status == op.ERR_VALUE
    for call in (lambda: op.layer_norm(f.cpu()), lambda: op.layer_norm(f.t()),
                 lambda: op.layer_norm(f.double()), lambda: op.layer_norm(f, f[0, :3]),
                 lambda: op.get_rows(f, i.long()), lambda: op.get_rows_back(f, i[:2], 3),
                 lambda: op.get_rows_back(f, i, 3, accumulate=True),
                 lambda: op.layer_norm_back(f, f, s[:2], s), lambda: op.dropout(f, 0.1, 1, out=h),
                 lambda: op.preference_loss(f, i, i[:2]), lambda: op.preference_loss(f, i[:3], i[:3]),
                 lambda: op.layer_norm(torch.empty((3, 5, 8), device="cuda")[:, 1:4][:, ::2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(op.OopError) as e:              # rows of an output may not overlap
        op.dropout(f, 0.1, 1, out=f[:1].expand(4, 16))
    assert e.value.status == op.ERR_SHAPE
    with pytest.raises(op.OopError) as e:              # a workspace that is too small
        op.layer_norm_back(f, f, s, s, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == op.ERR_WORKSPACE


def test_many_rows_past_32_bits(op):
    """Byte offsets beyond 2^32: rows of a 6 GB matrix, the last of them checked."""
    import torch
    T, M = 400_000, 4096
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    x = torch.empty((T, M), device="cuda").normal_()
    y = op.dropout(x, 0.5, 3)
    keep = torch.from_numpy(np.stack([_keep_row(t, 16, 0.5, 3) for t in range(T - 3, T)])).cuda()
    assert torch.equal(y[-3:, :16], torch.where(keep, x[-3:, :16] * 2, 0))
    n, mean, rstd = op.layer_norm(x, out=y)
    assert torch.allclose(mean[-5:], x[-5:].mean(1), atol=1e-5)
    ids = torch.tensor([T - 1, 0, T - 2], dtype=torch.int32, device="cuda")
    assert torch.equal(op.get_rows(x, ids), x[ids.long()])
    dx, dw, db = op.layer_norm_back(x, x, mean, rstd, out=y)
    xh = (x[-2:].double() - mean[-2:, None]) * rstd[-2:, None]
    g = x[-2:].double()
    want = rstd[-2:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    assert torch.allclose(dx[-2:].double(), want, atol=1e-5)
    assert torch.allclose(db.double(), x.sum(0, dtype=torch.float64), atol=0.2)


def test_dropout_of_more_groups_than_a_launch(op):
    """2^31 + 3 rows of one group each: two launches, one mask."""
    import torch
    T = 2 ** 31 + 3
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("needs 50 GB of device memory")
    x = torch.ones((T, 8), dtype=torch.bfloat16, device="cuda")
    op.dropout(x, 0.5, 3, out=x)
    assert op.last_launch_count() == 2
    for t in (0, 1, 2 ** 31 - 1, 2 ** 31, T - 1):
        assert ((x[t] != 0).cpu().numpy() == _keep_row(t, 8, 0.5, 3)).all()


def _keep_row(t, M, p, seed):
    """One row of dropout_keep."""
    drop = int(np.rint(p * 65536))
    bits = []
    for g in range((M + 7) // 8):
        for word in tr.philox4x32_10([g, t, 0, 0], [seed, 0]):
            bits += [word & 0xFFFF, word >> 16]
    return np.array(bits[:M]) >= drop
