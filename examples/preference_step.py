"""Adapter tuning on preference pairs, one training step at a time.

A small language model: token embeddings, a layer norm, a frozen projection
with a LoRA adapter behind dropout, and a frozen output matrix.  The
embeddings, the norm and the adapter learn to prefer the chosen answer of each
pair.  The forward products are torch's; everything else of the step is this
package's: the embedding lookup and its gradient, the norm, the dropout whose
mask is never stored, the loss over pairs and its gradient with respect to the
logits, and the backward products (MUL_MAT's, from a q8_0 weight, and both
adapter gradients of the projection).

    python examples/preference_step.py [steps]
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ggml_out_prod_gb300 as oop  # noqa: E402

EPS = 1e-5


def make_model(vocab=1000, width=256, out_width=320, rank=8, seed=0):
    """Random weights; `frozen` holds the projection twice: values for the
    forward product, q8_0 blocks for the backward one."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g) * std).cuda()

    blocks, values = quantise_q8_0(torch.randn((out_width, width), generator=g) / math.sqrt(width))
    frozen = {"W": values.cuda(), "W_q8_0": blocks.cuda(), "U": normal(vocab, out_width, std=out_width ** -0.5)}
    learnt = {"E": normal(vocab, width, std=1 / math.sqrt(width)), "w": torch.ones(width).cuda(),
              "b": torch.zeros(width).cuda(), "A": normal(rank, width, std=width ** -0.5),
              "B": normal(out_width, rank, std=0.02)}
    return learnt, frozen


def quantise_q8_0(w):
    """(uint8 rows of q8_0 blocks, the values they stand for)."""
    x = w.reshape(len(w), -1, 32)
    d = (x.abs().amax(2, keepdim=True) / 127).half()
    q = torch.round(x / d.float().clamp(min=1e-12)).clamp(-127, 127)
    blocks = torch.cat([d.view(torch.uint8), q.to(torch.int8).view(torch.uint8)], 2)
    return blocks.reshape(len(w), -1).contiguous(), (q * d.float()).reshape(w.shape)


def make_batch(pairs=4, prompt=6, answer=10, vocab=1000, seed=1):
    """Packed sequences, the chosen answers first: tokens, labels (-1 over the
    prompt and at each sequence's end) and first rows."""
    g = torch.Generator().manual_seed(seed)
    ids, labels, first = [], [], [0]
    prompts = torch.randint(0, vocab, (pairs, prompt), generator=g)
    for s in range(2 * pairs):
        n = answer - s % 3
        tokens = torch.cat([prompts[s % pairs], torch.randint(0, vocab, (n,), generator=g)])
        next_token = torch.cat([tokens[1:], torch.tensor([-1])])
        next_token[:prompt - 1] = -1
        ids.append(tokens)
        labels.append(next_token)
        first.append(first[-1] + len(tokens))
    return (torch.cat(ids).int().cuda(), torch.cat(labels).int().cuda(),
            torch.tensor(first, dtype=torch.int32).cuda())


def forward(learnt, frozen, ids, step, p=0.1, seed=1234, adapter=2.0):
    """The logits, and what the backward pass needs."""
    scale = math.sqrt(learnt["E"].shape[1])
    h = oop.get_rows(learnt["E"], ids, scale=scale)
    n, mean, rstd = oop.layer_norm(h, learnt["w"], learnt["b"], eps=EPS)
    d = oop.dropout(n, p, seed, offset=step)
    a = d @ learnt["A"].t()
    y = n @ frozen["W"].t() + adapter * (a @ learnt["B"].t())
    return y @ frozen["U"].t(), {"h": h, "n": n, "mean": mean, "rstd": rstd, "d": d, "a": a, "y": y}


def backward(learnt, frozen, ids, dlogits, kept, step, p=0.1, seed=1234, adapter=2.0):
    """The gradient of every learnt tensor from that of the logits."""
    k = kept
    _, dy = oop.mul_mat_back(frozen["U"], k["y"], dlogits, want_dW=False)
    dz = adapter * dy
    da = dz @ learnt["B"]
    grads = {}
    grads["A"], grads["B"] = oop.lora_backward(k["d"], k["a"], dz, da)
    _, dn = oop.mul_mat_back(frozen["W_q8_0"], k["n"], dy, w_type=oop.TYPE_Q8_0, want_dW=False)
    dn += oop.dropout_back(da @ learnt["A"], p, seed, offset=step)
    dh, grads["w"], grads["b"] = oop.layer_norm_back(dn, k["h"], k["mean"], k["rstd"], learnt["w"], out=dn)
    scale = math.sqrt(learnt["E"].shape[1])
    grads["E"] = oop.get_rows_back(dh, ids, len(learnt["E"]), scale=scale)
    return grads


def train_step(learnt, frozen, batch, ref_logps, step, rate=0.005, beta=0.5, label_smoothing=0.0):
    """One step of gradient descent; the loss before it (a CUDA scalar)."""
    ids, labels, first = batch
    logits, kept = forward(learnt, frozen, ids, step)
    r = oop.preference_loss(logits, labels, first, ref_logps, beta=beta, label_smoothing=label_smoothing)
    dlogits = oop.preference_loss_back(logits, labels, first, r.lse, r.ratios, beta=beta,
                                       label_smoothing=label_smoothing, out=logits)
    for name, g in backward(learnt, frozen, ids, dlogits, kept, step).items():
        learnt[name] -= rate * g
    return r.loss


def main(steps=40):
    learnt, frozen = make_model()
    batch = make_batch()
    logits, _ = forward(learnt, frozen, batch[0], step=0, p=0.0)       # the reference model: no dropout
    ref_logps, _ = oop.token_logps(logits, batch[1])
    losses = [train_step(learnt, frozen, batch, ref_logps, step) for step in range(1, steps + 1)]
    if oop.device_status() != oop.OK:
        raise RuntimeError("a device-side error was recorded")
    losses = [float(v) for v in losses]
    for i in range(0, steps, max(1, steps // 8)):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}")
    print(f"step {steps:4d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
