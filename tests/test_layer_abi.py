"""Refusals of the layer operators, on the CPU: every argument is checked before
the device is looked at, so bad calls return their status without a GPU (no
compute call is made here), and the size queries need none."""

import ctypes
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

F32, F16, BF16, Q8_0, Q4_K = 0, 1, 30, 8, 12
NULL, TYPE, SHAPE, ALIGN, WORKSPACE, VALUE = -1, -2, -3, -5, -6, -13
P, ODD, BIG = 0x10000, 0x10001, 2 ** 62      # pointers are never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def L():
    import ggml_out_prod_gb300 as g
    g.build()
    return g.lib()


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _heads(x=P, nb_x=(256, 1024), y=P, nb_y=(256, 1024), w=P, n=4):
    import ggml_out_prod_gb300 as g
    return g.OopHeads(x, *nb_x, y, *nb_y, w, n)


def norm(L, q={}, k={}, t=F32, wt=F32, pos=P, freqs=P, D=64, rot=64, T=3, eps=1e-6):
    a = ctypes.byref(_heads(**q)) if q is not None else None
    b = ctypes.byref(_heads(**k)) if k is not None else None
    return L.oop_qk_norm_rope(a, b, t, wt, pos, freqs, D, rot, T, 0, eps, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(q=dict(x=None)), NULL), (dict(q=dict(y=None)), NULL), (dict(k=dict(x=None)), NULL),
    (dict(pos=None), NULL), (dict(freqs=None), NULL), (dict(t=Q8_0), TYPE), (dict(wt=Q8_0), TYPE), (dict(t=5), TYPE),
    (dict(D=0), SHAPE), (dict(D=1025), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE), (dict(rot=-2), SHAPE),
    (dict(T=-1), SHAPE), (dict(T=2 ** 31), SHAPE), (dict(q=dict(n=-1)), SHAPE), (dict(k=dict(n=2 ** 21)), SHAPE),
    (dict(q=dict(nb_x=(-4, 1024))), SHAPE), (dict(q=dict(nb_x=(6, 1024))), SHAPE), (dict(q=dict(nb_x=(256, BIG))), SHAPE),
    (dict(q=dict(nb_y=(0, 1024))), SHAPE), (dict(q=dict(nb_y=(252, 1024))), SHAPE),
    (dict(q=dict(nb_y=(256, 512))), SHAPE),                  # the second token's heads over the first's
    (dict(q=dict(nb_y=(512, 256))), SHAPE),                  # the second head's tokens over the first's
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE),
    (dict(q=dict(x=ODD)), ALIGN), (dict(k=dict(y=ODD)), ALIGN), (dict(q=dict(w=ODD)), ALIGN),
    (dict(pos=ODD), ALIGN), (dict(freqs=ODD), ALIGN),
    (dict(T=0, pos=None, freqs=None), 0), (dict(q=dict(n=0), k=None), 0),
])
def test_qk_norm_rope_refusals(L, kw, want):
    assert norm(L, **kw) == want


def _grads(dy=P, nb_dy=(256, 1024), x=P, nb_x=(256, 1024), w=P, dx=P, nb_dx=(256, 1024), dw=P, n=4):
    import ggml_out_prod_gb300 as g
    return g.OopHeadsGrad(dy, *nb_dy, x, *nb_x, w, dx, *nb_dx, dw, n)


def norm_back(L, q={}, k={}, dt=F32, t=F32, wt=F32, pos=P, freqs=P, D=64, rot=64, T=3, eps=1e-6, ws=P, nws=1 << 30):
    a = ctypes.byref(_grads(**q)) if q is not None else None
    b = ctypes.byref(_grads(**k)) if k is not None else None
    return L.oop_qk_norm_rope_back(a, b, dt, t, wt, pos, freqs, D, rot, T, 0, eps, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(q=dict(dy=None)), NULL), (dict(q=dict(x=None)), NULL), (dict(k=dict(dx=None)), NULL),
    (dict(pos=None), NULL), (dict(freqs=None), NULL), (dict(dt=F16), TYPE), (dict(t=Q8_0), TYPE), (dict(wt=7), TYPE),
    (dict(D=0), SHAPE), (dict(rot=65), SHAPE), (dict(T=-1), SHAPE), (dict(q=dict(n=-1)), SHAPE),
    (dict(q=dict(nb_dx=(256, 256))), SHAPE), (dict(q=dict(nb_dy=(255, 1024))), SHAPE), (dict(k=dict(nb_x=(-256, 0))), SHAPE),
    (dict(eps=-1e-9), VALUE), (dict(q=dict(dx=ODD)), ALIGN), (dict(q=dict(dw=ODD)), ALIGN), (dict(k=dict(dy=ODD)), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(nws=64), WORKSPACE), (dict(ws=0x10010), WORKSPACE),
    (dict(ws=None, q=dict(dw=None)), WORKSPACE), (dict(q=dict(n=0, dw=None), k=None), 0), (dict(q=dict(dw=None), k=None, T=0), 0),
])
def test_qk_norm_rope_back_refusals(L, kw, want):
    assert norm_back(L, **kw) == want


def test_qk_norm_rope_back_workspace(L):
    size = L.oop_qk_norm_rope_back_workspace_size
    assert size(0, 4, 1, 1) == 0 and size(64, -1, 1, 1) == 0 and size(64, 4, -1, 0) == 0 and size(64, 4, 1, 2 ** 21) == 0
    assert size(64, 1, 1, 0) >= 64 * 4 and size(128, 2 ** 31 - 1, 2 ** 20, 2 ** 20) < 1 << 30


def ffn(L, x=P, t=F32, nbx=256, wg=P, wu=P, wt=F32, nbw=256, h=P, nbh=128, gate=P, up=P, nbg=128, ne=(64, 32, 5), act=0,
        ws=P, nws=1 << 40):
    return L.oop_gated_ffn(x, t, nbx, wg, wu, wt, nbw, h, nbh, gate, up, nbg, _i64(*ne) if ne else None, act, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(x=None), NULL), (dict(wg=None), NULL), (dict(wu=None), NULL), (dict(h=None), NULL),
    (dict(gate=None), NULL), (dict(up=None), NULL), (dict(t=Q8_0), TYPE), (dict(wt=9), TYPE),
    (dict(wt=Q8_0, ne=(48, 32, 5)), SHAPE), (dict(wt=Q4_K, ne=(128, 32, 5), nbx=512), SHAPE), (dict(ne=(-64, 32, 5)), SHAPE),
    (dict(ne=(64, -1, 5)), SHAPE), (dict(ne=(64, 32, -5)), SHAPE), (dict(ne=(64, 2 ** 31, 5)), SHAPE), (dict(nbx=-4), SHAPE),
    (dict(nbx=258), SHAPE), (dict(nbw=-256), SHAPE), (dict(nbh=64), SHAPE), (dict(nbg=0), SHAPE), (dict(act=4), VALUE),
    (dict(act=-1), VALUE), (dict(x=ODD), ALIGN), (dict(wg=ODD), ALIGN), (dict(wu=ODD), ALIGN), (dict(h=ODD), ALIGN),
    (dict(gate=ODD), ALIGN), (dict(up=ODD), ALIGN), (dict(ws=0x10010, ne=(64, 32, 400)), WORKSPACE),
    (dict(ws=None, ne=(64, 32, 400)), WORKSPACE), (dict(nws=16, ne=(64, 32, 400)), WORKSPACE), (dict(ne=(64, 32, 0)), 0),
    (dict(ne=(64, 0, 5), nbh=0, nbg=0), 0),
])
def test_gated_ffn_refusals(L, kw, want):
    assert ffn(L, **kw) == want


def ffn_back(L, dh=P, dt=F32, nbd=128, x=P, t=F32, nbx=256, wg=P, wu=P, wt=F32, nbw=256, gate=P, up=P, nbg=128, dx=P,
             nbdx=256, dwg=P, dwu=P, nbdw=256, ne=(64, 32, 5), act=0, ws=P, nws=1 << 40):
    return L.oop_gated_ffn_back(dh, dt, nbd, x, t, nbx, wg, wu, wt, nbw, gate, up, nbg, dx, nbdx, dwg, dwu, nbdw,
                                _i64(*ne) if ne else None, act, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(dh=None), NULL), (dict(x=None), NULL), (dict(wg=None), NULL), (dict(wu=None), NULL),
    (dict(gate=None), NULL), (dict(up=None), NULL), (dict(dwg=None), NULL), (dict(dwu=None), NULL), (dict(dt=F16), TYPE),
    (dict(t=Q8_0), TYPE), (dict(wt=4), TYPE), (dict(ne=(64, 32, -1)), SHAPE), (dict(nbd=64 + 1), SHAPE), (dict(nbx=-256), SHAPE),
    (dict(nbdx=128), SHAPE), (dict(nbdw=128), SHAPE), (dict(nbg=2), SHAPE), (dict(act=7), VALUE), (dict(dh=ODD), ALIGN),
    (dict(x=ODD), ALIGN), (dict(dx=ODD), ALIGN), (dict(dwg=ODD), ALIGN), (dict(dwu=ODD), ALIGN), (dict(gate=ODD), ALIGN),
    (dict(up=ODD), ALIGN), (dict(wu=ODD), ALIGN), (dict(ws=None), WORKSPACE), (dict(nws=16), WORKSPACE),
    (dict(ws=0x10010), WORKSPACE), (dict(dx=None, dwg=None, dwu=None), 0), (dict(dwg=None, dwu=None, ne=(64, 32, 0)), 0),
    (dict(ne=(0, 32, 5), nbx=0, nbw=0, nbdx=0, nbdw=0), 0),
])
def test_gated_ffn_back_refusals(L, kw, want):
    assert ffn_back(L, **kw) == want


def test_gated_ffn_workspaces(L):
    for fn, types in ((L.oop_gated_ffn_workspace_size, (F32, F32)), (L.oop_gated_ffn_back_workspace_size, (F32, F32, F32))):
        assert fn(*types, _i64(-1, 4, 4), 1) == 0 and fn(*types, None, 1) == 0
        assert fn(*types, _i64(64, 128, 300), 0) >= fn(*types, _i64(64, 128, 300), 1)
    assert L.oop_gated_ffn_workspace_size(Q8_0, F32, _i64(64, 4, 4), 0) == 0
    assert L.oop_gated_ffn_back_workspace_size(F16, F16, F16, _i64(64, 4, 4), 0) == 0


def orth(L, x=P, xt=F32, nbx=(256, 4096), y=P, yt=F32, nby=(256, 4096), ne=(64, 16, 2), steps=5, coefs=None, eps=1e-7,
         scale=1.0, ws=P, nws=1 << 40):
    c = (ctypes.c_float * len(coefs))(*coefs) if coefs else None
    pair = lambda v: _i64(*v) if v else None  # noqa: E731
    return L.oop_orthogonalise(x, xt, pair(nbx), y, yt, pair(nby), pair(ne), steps, c, eps, scale, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(nbx=None), NULL), (dict(nby=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL),
    (dict(xt=F16), TYPE), (dict(yt=F16), TYPE), (dict(xt=Q8_0), TYPE), (dict(ne=(-1, 16, 2)), SHAPE),
    (dict(ne=(64, -1, 2)), SHAPE), (dict(ne=(64, 16, -2)), SHAPE), (dict(ne=(64, 16, 65536)), SHAPE),
    (dict(ne=(2 ** 24, 2, 1)), SHAPE), (dict(nbx=(258, 4096)), SHAPE), (dict(nby=(128, 4096)), SHAPE),
    (dict(nby=(256, 256)), SHAPE), (dict(nbx=(-256, 4096)), SHAPE), (dict(steps=-1), VALUE), (dict(steps=65), VALUE),
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(scale=float("inf")), VALUE),
    (dict(steps=1, coefs=[1.0, float("nan"), 0.0]), VALUE), (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN),
    (dict(ws=None, ne=(96, 80, 2), nbx=(384, 30720), nby=(384, 30720)), WORKSPACE),
    (dict(nws=64, ne=(96, 80, 2), nbx=(384, 30720), nby=(384, 30720)), WORKSPACE),
    (dict(ws=0x10010, ne=(96, 80, 2), nbx=(384, 30720), nby=(384, 30720)), WORKSPACE), (dict(ne=(64, 16, 0)), 0),
    (dict(ne=(64, 0, 2)), 0), (dict(ne=(0, 16, 2)), 0),
])
def test_orthogonalise_refusals(L, kw, want):
    assert orth(L, **kw) == want


def test_orthogonalise_workspace(L):
    assert L.oop_orthogonalise_workspace_size(_i64(-1, 4, 4)) == 0 and L.oop_orthogonalise_workspace_size(None) == 0
    assert L.oop_orthogonalise_workspace_size(_i64(96, 80, 2)) > 0


def test_python_refusals():
    """What the binding refuses before it calls the library."""
    import torch
    import ggml_out_prod_gb300 as g
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        g.gated_ffn(x, x, x)                                 # not on a GPU
    with pytest.raises(ValueError):
        g.orthogonalise(x)
    with pytest.raises(ValueError):
        g.qk_norm_rope(x, None, None, None)


def _runtime(name):
    return subprocess.run(["gcc", f"-print-file-name={name}"], capture_output=True, text=True).stdout.strip()


@pytest.mark.skipif(os.environ.get("GGML_OUT_PROD_GB300_LIBRARY") is not None, reason="already under the sanitizers")
def test_refusals_under_the_sanitizers():
    """The same refusals and size queries with the host code under
    AddressSanitizer and UndefinedBehaviorSanitizer."""
    from ggml_out_prod_gb300 import _build
    _build.build()
    san = _build.build(sanitize=True)
    env = dict(os.environ, GGML_OUT_PROD_GB300_LIBRARY=san,
               LD_PRELOAD=" ".join([_runtime("libasan.so"), _runtime("libubsan.so")]),
               ASAN_OPTIONS="detect_leaks=0:protect_shadow_gap=0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-k", "(refusals or workspace) and not python",
                        os.path.abspath(__file__)], capture_output=True, text=True, timeout=600, env=env, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-3000:]
