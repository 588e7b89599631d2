"""The example that runs the layer operators together: its gradients against
torch's automatic ones in 64 bits, and that it runs."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    import ggml_out_prod_gb300 as g
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    g.build()
    spec = importlib.util.spec_from_file_location("decoder_step", os.path.join(ROOT, "examples", "decoder_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(example, p, ids, labels):
    """The loss of the same model in the parameters' type, by torch alone."""
    import torch
    import torch.nn.functional as F
    T = len(ids)

    def heads(x, w):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        pos, freqs = example.rotation(T)
        angle = pos.double()[:, None] * freqs.double()[None, :]
        c, s = angle.cos()[:, None, :], angle.sin()[:, None, :]
        n = example.ROTATED // 2
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., 2 * n:]], -1)

    x = p["E"][ids.long()]
    n1 = F.layer_norm(x, x.shape[1:], p["w1"], p["b1"], example.EPS)
    qkv = (n1 @ p["qkv"].t()).view(T, -1, example.HEAD)
    a, b = example.HEADS, example.HEADS + example.KV_HEADS
    h = x + example.attention(heads(qkv[:, :a], p["wq"]), heads(qkv[:, a:b], p["wk"]), qkv[:, b:]).reshape(T, -1) @ p["o"].t()
    n2 = F.layer_norm(h, h.shape[1:], p["w2"], p["b2"], example.EPS)
    y = h + (F.silu(n2 @ p["gate"].t()) * (n2 @ p["up"].t())) @ p["down"].t()
    return F.cross_entropy(y @ p["U"].t(), labels.long())


def test_gradients_of_one_step(example):
    """Every tensor's gradient against automatic differentiation in float64.  The step's own products run in
    fp32, chains of up to 300 terms (1e-6 of their operands' norms), and nothing in it amplifies by more than
    about 10: 1e-4 of each gradient's norm is a safe bound."""
    import torch
    p = example.make_model()
    ids, labels = example.make_batch()
    logits, kept = example.forward(p, ids)
    logits = logits.detach().requires_grad_()
    loss = torch.nn.functional.cross_entropy(logits, labels.long())
    grads = example.backward(p, ids, torch.autograd.grad(loss, logits)[0], kept)
    exact = {k: v.double().requires_grad_() for k, v in p.items()}
    want = _reference(example, exact, ids, labels)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) < 1e-5
    assert set(grads) == set(p)
    for name, g in grads.items():
        w = exact[name].grad
        assert float((g.double() - w).norm()) <= 1e-4 * float(w.norm()), name


def test_example_runs(example):
    losses = example.main(5)
    assert len(losses) == 5 and all(math.isfinite(v) for v in losses)
