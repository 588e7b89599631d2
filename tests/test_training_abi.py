"""Refusals of the training operators, on the CPU: every argument is checked
before the device is looked at, so bad calls return their status without a GPU
(no compute call is made here), and the size queries need none."""

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
P = ctypes.c_void_p(0x10000)          # never dereferenced: every call below is refused
ODD = ctypes.c_void_p(0x10001)
BIG = 2 ** 62


@pytest.fixture(scope="module")
def L():
    import ggml_out_prod_gb300 as g
    g.build()
    return g.lib()


def _ne(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rows(L, table=P, tt=F32, nbt=256, ids=P, dst=P, dt=F32, nbd=256, ne=(64, 10), n=4):
    return L.oop_get_rows(table, tt, nbt, ids, dst, dt, nbd, _ne(*ne) if ne else None, n, 1.0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(table=None), NULL), (dict(ids=None), NULL), (dict(dst=None), NULL),
    (dict(tt=9), TYPE), (dict(dt=Q8_0), TYPE), (dict(tt=Q8_0, ne=(48, 10)), SHAPE),
    (dict(tt=Q4_K, ne=(128, 10)), SHAPE), (dict(ne=(-1, 10)), SHAPE), (dict(ne=(64, -1)), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=2 ** 31), SHAPE), (dict(nbt=-4), SHAPE), (dict(nbt=258), SHAPE),
    (dict(nbd=128), SHAPE), (dict(nbd=0), SHAPE), (dict(nbt=BIG), SHAPE), (dict(ne=(BIG, 10)), SHAPE),
    (dict(table=ODD), ALIGN), (dict(ids=ODD), ALIGN), (dict(dst=ODD), ALIGN),
    (dict(n=0), 0), (dict(ne=(0, 10), nbt=0, nbd=0), 0),
])
def test_get_rows_refusals(L, kw, want):
    assert rows(L, **kw) == want


def rows_back(L, dy=P, dt=F32, nb=256, ids=P, d=P, ne=(64, 10), n=4, ws=P, nws=1 << 30):
    return L.oop_get_rows_back(dy, dt, nb, ids, d, _ne(*ne) if ne else None, n, 1.0, 0, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(dy=None), NULL), (dict(ids=None), NULL), (dict(d=None), NULL),
    (dict(dt=F16, nb=128), TYPE), (dict(dt=Q8_0), TYPE), (dict(ne=(64, -2)), SHAPE), (dict(n=-1), SHAPE),
    (dict(nb=3), SHAPE), (dict(nb=-256), SHAPE), (dict(ne=(64, 2 ** 31)), SHAPE),
    (dict(dy=ODD), ALIGN), (dict(ids=ODD), ALIGN), (dict(d=ODD), ALIGN), (dict(ne=(0, 10)), 0),
    (dict(ne=(64, 0)), 0),
])
def test_get_rows_back_refusals(L, kw, want):
    assert rows_back(L, **kw) == want


def test_get_rows_back_workspace(L):
    ne = _ne(64, 1000)
    need = L.oop_get_rows_back_workspace_size(ne, 5000)
    assert L.oop_get_rows_back_workspace_size(_ne(-1, 3), 5) == 0
    if need:
        assert rows_back(L, ne=(64, 1000), n=5000, ws=None) == WORKSPACE
        assert rows_back(L, ne=(64, 1000), n=5000, nws=need - 1) == WORKSPACE
        assert rows_back(L, ne=(64, 1000), n=5000, ws=ctypes.c_void_p(0x10010)) == WORKSPACE


def norm(L, x=P, xt=F32, nbx=256, w=P, b=P, wt=F32, y=P, yt=F32, nby=256, mean=P, rstd=P, ne=(64, 4), eps=1e-5):
    return L.oop_layer_norm(x, xt, nbx, w, b, wt, y, yt, nby, mean, rstd, _ne(*ne) if ne else None, eps, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(xt=Q8_0), TYPE), (dict(yt=7), TYPE),
    (dict(wt=Q8_0), TYPE), (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE),
    (dict(ne=(0, 4)), SHAPE), (dict(ne=(64, -4)), SHAPE), (dict(nbx=2), SHAPE), (dict(nby=64), SHAPE),
    (dict(ne=(2 ** 31, 1)), SHAPE), (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(b=ODD), ALIGN), (dict(mean=ODD), ALIGN), (dict(rstd=ODD), ALIGN), (dict(ne=(64, 0)), 0),
])
def test_layer_norm_refusals(L, kw, want):
    assert norm(L, **kw) == want


def norm_back(L, dy=P, dt=F32, nbd=256, x=P, xt=F32, nbx=256, mean=P, rstd=P, w=P, wt=F32, dx=P, nbdx=256, dw=P,
              db=P, ne=(64, 4), ws=P, nws=1 << 30):
    return L.oop_layer_norm_back(dy, dt, nbd, x, xt, nbx, mean, rstd, w, wt, dx, nbdx, dw, db,
                                 _ne(*ne) if ne else None, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(dy=None), NULL), (dict(x=None), NULL), (dict(dx=None), NULL),
    (dict(mean=None), NULL), (dict(rstd=None), NULL), (dict(dt=F16), TYPE), (dict(xt=Q8_0), TYPE), (dict(wt=5), TYPE),
    (dict(ne=(0, 4)), SHAPE), (dict(nbd=-4), SHAPE), (dict(nbx=2), SHAPE), (dict(nbdx=0), SHAPE),
    (dict(dy=ODD), ALIGN), (dict(x=ODD), ALIGN), (dict(dx=ODD), ALIGN), (dict(dw=ODD), ALIGN), (dict(db=ODD), ALIGN),
    (dict(mean=ODD), ALIGN), (dict(rstd=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(nws=64), WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE),
    (dict(ws=None, db=None), WORKSPACE), (dict(ne=(0, 0)), 0),
])
def test_layer_norm_back_refusals(L, kw, want):
    assert norm_back(L, **kw) == want


def drop(L, x=P, t=F32, nbx=256, y=P, nby=256, ne=(64, 4), p=0.5, back=False):
    fn = L.oop_dropout_back if back else L.oop_dropout
    return fn(x, t, nbx, y, nby, _ne(*ne) if ne else None, p, 1, 2, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(t=Q8_0), TYPE),
    (dict(t=F16, back=True), TYPE), (dict(p=-0.1), VALUE), (dict(p=1.01), VALUE), (dict(p=float("nan")), VALUE),
    (dict(ne=(-64, 4)), SHAPE), (dict(ne=(2 ** 36, 1)), SHAPE), (dict(ne=(1, 2 ** 33)), SHAPE), (dict(nbx=2), SHAPE),
    (dict(nby=128), SHAPE), (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(ne=(0, 4)), 0), (dict(ne=(64, 0)), 0),
])
def test_dropout_refusals(L, kw, want):
    assert drop(L, **kw) == want


def loss(L, x=P, t=F32, nb=256, labels=P, seq=P, ref=P, loss=P, losses=P, ratios=P, logps=P, lse=P, ne=(64, 4),
         pairs=1, beta=0.1, e=0.0, ws=P, nws=1 << 30):
    return L.oop_preference_loss(x, t, nb, labels, seq, ref, loss, losses, ratios, logps, lse,
                                 _ne(*ne) if ne else None, pairs, beta, e, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(x=None), NULL), (dict(labels=None), NULL), (dict(seq=None), NULL),
    (dict(loss=None), NULL), (dict(losses=None), NULL), (dict(ratios=None), NULL), (dict(logps=None), NULL),
    (dict(lse=None), NULL), (dict(t=Q8_0), TYPE), (dict(beta=float("nan")), VALUE), (dict(beta=float("inf")), VALUE),
    (dict(e=-0.1), VALUE), (dict(e=1.1), VALUE), (dict(e=float("nan")), VALUE), (dict(pairs=-1), SHAPE),
    (dict(ne=(-1, 4)), SHAPE), (dict(ne=(2 ** 31, 4)), SHAPE), (dict(ne=(2 ** 30, 2 ** 30)), SHAPE),
    (dict(nb=6), SHAPE), (dict(x=ODD), ALIGN), (dict(labels=ODD), ALIGN), (dict(seq=ODD), ALIGN),
    (dict(ref=ODD), ALIGN), (dict(lse=ODD), ALIGN), (dict(loss=ODD), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(nws=100), WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE), (dict(ne=(64, 0), pairs=0), 0),
])
def test_preference_loss_refusals(L, kw, want):
    assert loss(L, **kw) == want


def loss_back(L, x=P, t=F32, nb=256, labels=P, seq=P, lse=P, ratios=P, dloss=None, d=P, dt=F32, nbd=256, ne=(64, 4),
              pairs=1, beta=0.1, e=0.0):
    return L.oop_preference_loss_back(x, t, nb, labels, seq, lse, ratios, dloss, d, dt, nbd,
                                      _ne(*ne) if ne else None, pairs, beta, e, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ne=None), NULL), (dict(x=None), NULL), (dict(labels=None), NULL), (dict(seq=None), NULL),
    (dict(lse=None), NULL), (dict(ratios=None), NULL), (dict(d=None), NULL), (dict(t=Q8_0), TYPE),
    (dict(dt=F16, nbd=128), TYPE), (dict(beta=float("inf")), VALUE), (dict(e=2.0), VALUE), (dict(pairs=-1), SHAPE),
    (dict(nbd=0), SHAPE), (dict(nb=-256), SHAPE), (dict(d=ODD), ALIGN), (dict(dloss=ODD), ALIGN), (dict(lse=ODD), ALIGN),
    (dict(ne=(64, 0)), 0), (dict(ne=(0, 4), nb=0, nbd=0), 0),
])
def test_preference_loss_back_refusals(L, kw, want):
    assert loss_back(L, **kw) == want


def test_size_queries_reject_bad_shapes(L):
    assert L.oop_layer_norm_back_workspace_size(_ne(-1, 4)) == 0
    assert L.oop_layer_norm_back_workspace_size(_ne(64, 4)) > 0
    assert L.oop_preference_loss_workspace_size(_ne(64, -4), 1) == 0
    assert L.oop_preference_loss_workspace_size(_ne(64, 4), -1) == 0
    # the partial sums grow with the rows; past every size they stay in 64 bits
    a = L.oop_preference_loss_workspace_size(_ne(128000, 100), 2)
    assert 0 < a < L.oop_preference_loss_workspace_size(_ne(128000, 20000), 2)


def test_last_status_has_a_description(L):
    import ggml_out_prod_gb300 as g
    assert g.status_string(g.ERR_VALUE) != "unknown status"


def test_python_checks_need_no_device():
    """CPU tensors are refused by name before the library is asked."""
    import torch
    import ggml_out_prod_gb300 as g
    x, i = torch.ones((4, 8)), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: g.layer_norm(x), lambda: g.dropout(x, 0.1, 1), lambda: g.get_rows_back(x, i, 3),
                 lambda: g.get_rows(x, i), lambda: g.preference_loss(x, i, i[:3]), lambda: g.token_logps(x, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def _runtime(name):
    p = subprocess.run(["gcc", f"-print-file-name={name}"], capture_output=True, text=True)
    return p.stdout.strip() if os.path.isabs(p.stdout.strip()) else None


@pytest.mark.skipif(shutil.which("gcc") is None or _runtime("libasan.so") is None or
                    "GGML_OUT_PROD_GB300_LIBRARY" in os.environ, reason="gcc's sanitizer runtimes are needed")
def test_refusals_under_sanitizers():
    """This file's calls against the library built with sanitized host code."""
    from ggml_out_prod_gb300 import _build
    _build.build()
    san = _build.build(sanitize=True)
    env = dict(os.environ, GGML_OUT_PROD_GB300_LIBRARY=san,
               LD_PRELOAD=" ".join([_runtime("libasan.so"), _runtime("libubsan.so")]),
               ASAN_OPTIONS="detect_leaks=0:protect_shadow_gap=0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-k", "refusals or workspace or size",
                        os.path.abspath(__file__)], capture_output=True, text=True, timeout=600, env=env, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-3000:]


def test_callers_scratch_lies_on_the_device_of_the_call():
    """A caller's workspace on another GPU, or with gaps, is refused before its
    pointer is taken."""
    import torch
    import ggml_out_prod_gb300 as g

    class Workspace:
        is_cuda, device = True, torch.device("cuda", 1)
        contiguous = True

        def is_contiguous(self):
            return self.contiguous

        def data_ptr(self):
            return 0x10000

        def numel(self):
            return 1 << 20

        def element_size(self):
            return 1

    w = Workspace()
    assert g._scratch(64, torch.device("cuda", 1), w) == (w, 0x10000, 1 << 20)
    with pytest.raises(ValueError):
        g._scratch(64, torch.device("cuda", 0), w)
    w.contiguous = False
    with pytest.raises(ValueError):
        g._scratch(64, torch.device("cuda", 1), w)
    assert g._scratch(0, torch.device("cuda", 0), w) == (None, None, 0)
