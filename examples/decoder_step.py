"""Training a one-layer decoder with orthogonalised updates, one step at a time.

Token embeddings, a layer norm, queries and keys normalised and rotated head by head, causal attention, another layer
norm, a gated feed-forward block, and an output matrix.  The attention itself and the forward products of plain
projections are torch's; the rest of the step is this package's: the embedding lookup and its gradient, the norms, the
head norms with rotation, the feed-forward block, every projection's backward product, and the update of each matrix, its
momentum made nearly orthogonal (the Muon optimiser's step).

    python examples/decoder_step.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ggml_out_prod_gb300 as oop  # noqa: E402

EPS = 1e-5
HEADS, KV_HEADS, HEAD = 4, 2, 32
ROTATED = 24                                             # of each head's elements


def make_model(vocab=300, width=96, hidden=256, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=None):
        return (torch.randn(shape, generator=g) * (shape[-1] ** -0.5 if std is None else std)).cuda()

    one, zero = lambda n: torch.ones(n).cuda(), lambda n: torch.zeros(n).cuda()  # noqa: E731
    return {"E": normal(vocab, width, std=1.0), "w1": one(width), "b1": zero(width), "w2": one(width), "b2": zero(width),
            "qkv": normal((HEADS + 2 * KV_HEADS) * HEAD, width), "wq": one(HEAD), "wk": one(HEAD),
            "o": normal(width, HEADS * HEAD), "gate": normal(hidden, width), "up": normal(hidden, width),
            "down": normal(width, hidden), "U": normal(vocab, width)}


def make_batch(vocab=300, length=40, seed=1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (length + 1,), generator=g).int().cuda()
    return ids[:-1].contiguous(), ids[1:].contiguous()


def rotation(length):
    freqs = (1e4 ** (-torch.arange(ROTATED // 2, dtype=torch.float64) / (ROTATED // 2))).float().cuda()
    return torch.arange(length, dtype=torch.int32, device="cuda"), freqs


def attention(q, k, v):
    """Causal attention, each key head shared by neighbouring query heads: (T, heads, size)."""
    k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1) for t in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) * HEAD ** -0.5
    hidden = torch.ones(s.shape[1:], dtype=torch.bool, device=s.device).triu(1)
    return torch.einsum("hqk,khd->qhd", s.masked_fill(hidden, float("-inf")).softmax(-1), v)


def forward(p, ids):
    """The logits, and what the backward pass needs."""
    T = len(ids)
    pos, freqs = rotation(T)
    x = oop.get_rows(p["E"], ids)
    n1, mean1, rstd1 = oop.layer_norm(x, p["w1"], p["b1"], eps=EPS)
    qkv = (n1 @ p["qkv"].t()).view(T, -1, HEAD)
    q0, k0, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
    q, k = oop.qk_norm_rope(q0, k0, pos, freqs, p["wq"], p["wk"])
    a = attention(q, k, v).reshape(T, -1)
    h = x + a @ p["o"].t()
    n2, mean2, rstd2 = oop.layer_norm(h, p["w2"], p["b2"], eps=EPS)
    ffn = oop.gated_ffn(n2, p["gate"], p["up"], keep=True)
    y = h + ffn.h @ p["down"].t()
    kept = dict(x=x, n1=n1, mean1=mean1, rstd1=rstd1, q0=q0, k0=k0, q=q, k=k, v=v, a=a, h=h, n2=n2, mean2=mean2, rstd2=rstd2,
                ffn=ffn, y=y, pos=pos, freqs=freqs)
    return y @ p["U"].t(), kept


def backward(p, ids, dlogits, c):
    """The gradient of every tensor from that of the logits."""
    T, g = len(ids), {}
    g["U"], dy = oop.mul_mat_back(p["U"], c["y"], dlogits)
    g["down"], dffn = oop.mul_mat_back(p["down"], c["ffn"].h, dy)
    dn2, g["gate"], g["up"] = oop.gated_ffn_back(dffn.view(T, -1), c["n2"], p["gate"], p["up"], c["ffn"].gate, c["ffn"].up)
    dh, g["w2"], g["b2"] = oop.layer_norm_back(dn2, c["h"], c["mean2"], c["rstd2"], p["w2"])
    dh = dh + dy.view(T, -1)
    g["o"], da = oop.mul_mat_back(p["o"], c["a"], dh)
    q, k, v = (c[n].detach().requires_grad_() for n in ("q", "k", "v"))
    dq, dk, dv = torch.autograd.grad(attention(q, k, v), (q, k, v), da.view(T, HEADS, HEAD))
    dqkv = torch.empty((T, HEADS + 2 * KV_HEADS, HEAD), device="cuda")       # the gradients go where the slices are
    _, _, g["wq"], g["wk"] = oop.qk_norm_rope_back(dq.contiguous(), dk.contiguous(), c["q0"], c["k0"], c["pos"], c["freqs"], p["wq"],
                                                   p["wk"], out_q=dqkv[:, :HEADS], out_k=dqkv[:, HEADS:HEADS + KV_HEADS])
    dqkv[:, HEADS + KV_HEADS:] = dv
    g["qkv"], dn1 = oop.mul_mat_back(p["qkv"], c["n1"], dqkv.view(T, -1))
    dx, g["w1"], g["b1"] = oop.layer_norm_back(dn1.view(T, -1), c["x"], c["mean1"], c["rstd1"], p["w1"])
    g["E"] = oop.get_rows_back(dx + dh, ids, len(p["E"]))
    return {name: v.reshape(p[name].shape) for name, v in g.items()}


MATRICES = ("qkv", "o", "gate", "up", "down", "U")


def train_step(p, momentum, batch, rate=0.02, keep=0.9):
    """One step; the loss before it (a CUDA scalar)."""
    ids, labels = batch
    logits, kept = forward(p, ids)
    logits = logits.detach().requires_grad_()
    loss = torch.nn.functional.cross_entropy(logits, labels.long())
    for name, g in backward(p, ids, torch.autograd.grad(loss, logits)[0], kept).items():
        m = momentum.setdefault(name, torch.zeros_like(g))
        m.mul_(keep).add_(g)
        if name in MATRICES:
            p[name] -= oop.orthogonalise(g + keep * m, scale=rate * max(1.0, g.shape[0] / g.shape[1]) ** 0.5)
        else:
            p[name] -= 0.1 * rate * m
    return loss.detach()


def main(steps=20):
    p, momentum, batch = make_model(), {}, make_batch()
    losses = [train_step(p, momentum, batch) for _ in range(steps)]
    if oop.device_status() != oop.OK:
        raise RuntimeError("a device-side error was recorded")
    losses = [float(v) for v in losses]
    for i in range(0, steps, max(1, steps // 8)):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}")
    print(f"step {steps:4d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
