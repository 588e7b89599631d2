"""The bounded waits of the layer operators' product kernel, without a GPU fault: the hook oop_debug_inject_timeout
makes the first stage of the next launch expect more than its copies bring, so the products wait for data that never
comes.  The kernel has to give up, record OOP_ERR_DEVICE_TIMEOUT, release its tensor memory in both CTAs and return, and
the next calls have to be right."""

import time

import pytest

from test_gpu_layer import _rand, op  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(op):  # noqa: F811
    x, _ = _rand(1, (300, 200), "bf16")
    w, _ = _rand(2, (136, 200), "bf16", 0.1)
    m, _ = _rand(3, (96, 300), "f32")
    xf, wf = x.float(), w.float()
    return {"gate": lambda: op.gated_ffn(x, w, w).h, "gate folded": lambda: op.gated_ffn(xf, wf, wf).h, "planes": lambda: op.orthogonalise(m)}


@pytest.mark.parametrize("which", ["gate", "gate folded", "planes"])
def test_bounded_wait_of_the_layer_products(op, which):  # noqa: F811
    import torch
    call = _calls(op)[which]
    want = call()
    assert op.device_status(clear=True) == op.OK
    assert op.lib().oop_debug_inject_timeout(1) == op.OK
    t0 = time.time()
    call()
    st = op.device_status(clear=True)
    assert st == op.ERR_DEVICE_TIMEOUT, op.status_string(st)
    assert time.time() - t0 < 30.0
    assert op.device_status() == op.OK                             # cleared
    for _ in range(3):                                             # one launch takes the hook; all that follows is whole
        assert torch.equal(call(), want)
    assert op.device_status() == op.OK
