"""The example that runs the training operators together: its gradients against
torch's automatic ones in 64 bits, and its loss going down."""

import importlib.util
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
    spec = importlib.util.spec_from_file_location("preference_step", os.path.join(ROOT, "examples", "preference_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_of_one_step(example):
    """Every learnt tensor's gradient against automatic differentiation of the
    same model in float64, the dropout mask given by what the step kept.  The
    step's forward products run in fp32 (chains of up to 1000 terms, relative
    error ~1e-6 of their operands' norms) and nothing in it amplifies by more
    than ~10: 1e-4 of each gradient's norm is a safe bound."""
    import torch
    import torch.nn.functional as F
    learnt, frozen = example.make_model()
    ids, labels, first = example.make_batch()
    logits, kept = example.forward(learnt, frozen, ids, step=3)
    ref, _ = example.oop.token_logps(logits * 0.97, labels)
    r = example.oop.preference_loss(logits, labels, first, ref, beta=0.5, label_smoothing=0.1)
    d = example.oop.preference_loss_back(logits, labels, first, r.lse, r.ratios, beta=0.5, label_smoothing=0.1)
    grads = example.backward(learnt, frozen, ids, d, kept, step=3)

    p = {k: v.double().requires_grad_() for k, v in learnt.items()}
    h = p["E"][ids.long()] * p["E"].shape[1] ** 0.5
    n = F.layer_norm(h, h.shape[1:], p["w"], p["b"], example.EPS)
    drop = round(0.1 * 65536)
    mask = (kept["d"] != 0).double() * 65536 / (65536 - drop)
    y = n @ frozen["W"].double().t() + 2.0 * ((n * mask) @ p["A"].t()) @ p["B"].t()
    lp = torch.log_softmax(y @ frozen["U"].double().t(), 1)
    use = labels >= 0
    diff = torch.where(use, lp.gather(1, labels.long().clamp(min=0)[:, None])[:, 0] - ref.double(), 0.0)
    ratios = torch.stack([diff[a:b].sum() for a, b in zip(first[:-1].tolist(), first[1:].tolist())])
    P = len(ratios) // 2
    m = 0.5 * (ratios[:P] - ratios[P:])
    loss = (0.9 * F.softplus(-m) + 0.1 * F.softplus(m)).mean()
    loss.backward()
    assert abs(float(r.loss) - float(loss.detach())) < 1e-5
    for name, g in grads.items():
        want = p[name].grad
        assert float((g.double() - want).norm()) <= 1e-4 * float(want.norm()), name


def test_loss_goes_down(example):
    losses = example.main(40)
    assert losses[-1] < 0.5 * losses[0], losses
