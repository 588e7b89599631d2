"""The operators of a decoder layer's training step, as cases that can be timed and compared.

Around its attention and in its feed-forward block, and for the update of the weights whose gradients the products of
this library are:

  qk_norm_rope        RMS norm of every query and key head and the rotation by the token's position, in one pass
  qk_norm_rope_back   dq and dk, and the gradients of the norms' weights over all tokens and heads
  gated_ffn           h = act(x Wg') * (x Wu'): both projections, the activation and the product
  gated_ffn_back      dx, dWg and dWu from dh and the kept projections
  orthogonalise       Newton-Schulz steps on a weight's update: X <- a X + (b A + c A A) X with A = X X'

``run`` computes a case in elementary torch operations in 32 bits (``own`` false) or through this package's public
calls (``own`` true); ``exact`` computes it from the definitions in 64 bits.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
COEF = (3.4445, -4.7750, 2.0315)                        # the usual quintic of five steps
STEPS = 5
NORM_EPS = 1e-7


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token behind a long context: only latency counts
        {"name": "qk_norm_rope bf16 1 token", "op": "qk_norm_rope", "x": "bf16", "w": "f32", "T": 1, "Hq": 32, "Hk": 8,
         "D": 128, "rot": 128, "halves": True},
        # the packed sequences of a training batch, queries and keys as slices of one projection's output
        {"name": "qk_norm_rope bf16 16k tokens", "op": "qk_norm_rope", "x": "bf16", "w": "f32", "T": 16384, "Hq": 32,
         "Hk": 8, "D": 128, "rot": 128, "halves": True},
        # a narrow odd head of which a part is rotated, neighbours as pairs, an odd number of tokens
        {"name": "qk_norm_rope_back f32 odd", "op": "qk_norm_rope_back", "x": "f32", "dy": "f32", "w": "f32", "T": 777,
         "Hq": 9, "Hk": 3, "D": 80, "rot": 40, "halves": False},
        # the backward pass of the same batch
        {"name": "qk_norm_rope_back bf16 16k tokens", "op": "qk_norm_rope_back", "x": "bf16", "dy": "bf16", "w": "f32",
         "T": 16384, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "halves": True},
        # one token: the weights' bytes are all there is
        {"name": "gated_ffn bf16 1 token", "op": "gated_ffn", "x": "bf16", "act": "silu", "T": 1, "K": 2560, "F": 9728,
         "keep": False},
        # the 512 tokens of the adapter workload, everything in 32 bits as its products take it
        {"name": "gated_ffn f32 512 tokens", "op": "gated_ffn", "x": "f32", "act": "silu", "T": 512, "K": 2560,
         "F": 9728, "keep": True},
        # a training batch at the widest layer of the dense workload
        {"name": "gated_ffn bf16 8k tokens", "op": "gated_ffn", "x": "bf16", "act": "silu", "T": 8192, "K": 5120,
         "F": 17408, "keep": True},
        # odd sizes in 32 bits
        {"name": "gated_ffn_back f32 odd", "op": "gated_ffn_back", "x": "f32", "dh": "f32", "act": "gelu_tanh", "T": 333,
         "K": 1001, "F": 1537},
        # the backward pass of a training batch at the adapter workload's widths
        {"name": "gated_ffn_back bf16 8k tokens", "op": "gated_ffn_back", "x": "bf16", "dh": "bf16", "act": "silu",
         "T": 8192, "K": 2560, "F": 9728},
        # the update of one adapter matrix
        {"name": "orthogonalise f32 8x2560", "op": "orthogonalise", "x": "f32", "y": "f32", "M": 8, "N": 2560, "B": 1},
        # the update of one feed-forward weight
        {"name": "orthogonalise f32 9728x2560", "op": "orthogonalise", "x": "f32", "y": "bf16", "M": 9728, "N": 2560,
         "B": 1},
        # the updates of 32 experts' weights, their gradients one tensor
        {"name": "orthogonalise f32 32 experts", "op": "orthogonalise", "x": "f32", "y": "f32", "M": 768, "N": 2048,
         "B": 32},
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of lo..hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "qk_norm_rope_back", "gated_ffn", "gated_ffn_back", "orthogonalise"])
    if op in ("qk_norm_rope", "qk_norm_rope_back"):
        D = rng.choice([64, 80, 96, 128, 192, 256, _between(rng, 8, 256)])
        Hk = _between(rng, 1, 16)
        case = {"op": op, "x": rng.choice(["f32", "f16", "bf16"]), "w": rng.choice(["f32", "bf16"]),
                "T": _between(rng, 1, 16384), "Hq": Hk * rng.choice([1, 2, 4, 5, 8]), "Hk": Hk, "D": D,
                "rot": 2 * (rng.choice([D, D, D // 2, D // 4]) // 2), "halves": rng.random() < 0.6}
        while case["T"] * (case["Hq"] + case["Hk"]) * D > 16384 * 40 * 128 // 2:
            case["T"] = (case["T"] + 1) // 2
        if op == "qk_norm_rope_back":
            case["dy"] = rng.choice(["f32", "bf16"])
        return case
    if op in ("gated_ffn", "gated_ffn_back"):
        case = {"op": op, "x": rng.choice(["f32", "f16", "bf16", "bf16"]),
                "act": rng.choice(["silu", "silu", "gelu_tanh", "gelu_erf", "relu"]),
                "T": _between(rng, 1, 8192), "K": _between(rng, 64, 5120), "F": _between(rng, 64, 17408)}
        if rng.random() < 0.5:                           # most models' widths are multiples of 64
            case["K"], case["F"] = max(64, case["K"] // 64 * 64), max(64, case["F"] // 64 * 64)
        while case["T"] * case["K"] * case["F"] > 8192 * 2560 * 9728 // 2:
            case["T"] = (case["T"] + 1) // 2
        if op == "gated_ffn":
            case["keep"] = rng.random() < 0.5
        else:
            case["dh"] = "f32" if case["x"] == "f32" else "bf16"
        return case
    M, N, B = _between(rng, 4, 4096), _between(rng, 4, 4096), _between(rng, 1, 16)
    while B > 1 and B * M * N > 1 << 24:
        B = (B + 1) // 2
    return {"op": op, "x": rng.choice(["f32", "f32", "bf16"]), "y": rng.choice(["f32", "bf16"]), "M": M, "N": N, "B": B}


def work(case):
    op = case["op"]
    if op == "qk_norm_rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * n * _SIZE[case["x"]] + 4 * case["T"] + 2 * case["D"] * _SIZE[case["w"]], "flops": 8 * n}
    if op == "qk_norm_rope_back":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": n * (_SIZE[case["x"]] + 2 * _SIZE[case["dy"]]) + 4 * case["T"] + 2 * case["D"] * (_SIZE[case["w"]] + 4),
                "flops": 16 * n}
    if op == "gated_ffn":
        T, K, F, e = case["T"], case["K"], case["F"], _SIZE[case["x"]]
        return {"bytes": e * (T * K + 2 * F * K + T * F * (3 if case["keep"] else 1)), "flops": 4 * T * K * F}
    if op == "gated_ffn_back":
        T, K, F, e, d = case["T"], case["K"], case["F"], _SIZE[case["x"]], _SIZE[case["dh"]]
        return {"bytes": e * (T * K + 2 * F * K + 2 * T * F) + d * (T * F + T * K + 2 * F * K), "flops": 8 * T * K * F}
    n, m = sorted((case["M"], case["N"]))
    # products of symmetric results count half; the steps on X itself, or all of them on A and one product with X
    on_x, on_a = STEPS * (3 * n * n * m + n * n * n), 3 * n * n * m + (4 * STEPS - 3) * n * n * n
    return {"bytes": case["B"] * n * m * (_SIZE[case["x"]] + _SIZE[case["y"]]), "flops": case["B"] * min(on_x, on_a)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, kind, std=1.0, mean=0.0):
    x = torch.empty(shape, dtype=_DT[kind], device="cuda")
    return x.normal_(mean, std, generator=g)


def prepare(case, seed):
    op, g = case["op"], _generator(seed)
    if op in ("qk_norm_rope", "qk_norm_rope_back"):
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        qkv = _normal(g, (T, (Hq + 2 * Hk) * D), case["x"], 1.3)
        # packed sequences of up to 4096 tokens, each continuing at a place of its own in a long context
        at = torch.arange(T, device="cuda", dtype=torch.int32)
        starts = torch.randint(0, 131072, (T // 4096 + 1,), device="cuda", generator=g, dtype=torch.int32)
        half = case["rot"] // 2
        freqs = (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()
        s = {"case": case, "q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D),
             "pos": starts[(at // 4096).long()] + at % 4096, "freqs": freqs,
             "wq": _normal(g, (D,), case["w"], 0.2, 1.0), "wk": _normal(g, (D,), case["w"], 0.2, 1.0)}
        if op == "qk_norm_rope_back":
            s["dq"], s["dk"] = _normal(g, (T, Hq, D), case["dy"]), _normal(g, (T, Hk, D), case["dy"])
        return s
    if op in ("gated_ffn", "gated_ffn_back"):
        T, K, F = case["T"], case["K"], case["F"]
        s = {"case": case, "x": _normal(g, (T, K), case["x"]), "wg": _normal(g, (F, K), case["x"], K ** -0.5),
             "wu": _normal(g, (F, K), case["x"], K ** -0.5)}
        if op == "gated_ffn_back":
            s["gate"], s["up"] = s["x"] @ s["wg"].T, s["x"] @ s["wu"].T
            s["dh"] = _normal(g, (T, F), case["dh"])
        return s
    # a batch's gradient: a part of low rank above noise
    M, N, B = case["M"], case["N"], case["B"]
    r = max(1, min(M, N) // 8)
    x = torch.bmm(_normal(g, (B, M, r), "f32", r ** -0.5), _normal(g, (B, r, N), "f32")) + _normal(g, (B, M, N), "f32", 0.3)
    return {"case": case, "x": (x * 1e-3).to(_DT[case["x"]])}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _own_run(state) if own else _plain_run(state)


def _own_run(s):
    import ggml_out_prod_gb300 as oop

    c = s["case"]
    op = c["op"]
    if op == "qk_norm_rope":
        q, k = oop.qk_norm_rope(s["q"], s["k"], s["pos"], s["freqs"], s["wq"], s["wk"], eps=EPS,
                                interleaved=not c["halves"])
        return {"q": q, "k": k}
    if op == "qk_norm_rope_back":
        dq, dk, dwq, dwk = oop.qk_norm_rope_back(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freqs"], s["wq"], s["wk"],
                                                 eps=EPS, interleaved=not c["halves"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "gated_ffn":
        h, gate, up = oop.gated_ffn(s["x"], s["wg"], s["wu"], act=c["act"], keep=c["keep"])
        return {"h": h, "gate": gate, "up": up} if c["keep"] else h
    if op == "gated_ffn_back":
        dx, dwg, dwu = oop.gated_ffn_back(s["dh"], s["x"], s["wg"], s["wu"], s["gate"], s["up"], act=c["act"])
        return {"dx": dx, "dwg": dwg, "dwu": dwu}
    return oop.orthogonalise(s["x"], steps=STEPS, coefs=COEF, eps=NORM_EPS, out_dtype=_DT[c["y"]])


def _plain_run(s):
    c = s["case"]
    op = c["op"]
    if op == "qk_norm_rope":
        cos, sin = _turn(s)
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x = s[name].float()
            n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
            out[name] = _rotated(n, cos, sin, c).to(_DT[c["x"]])
        return out
    if op == "qk_norm_rope_back":
        cos, sin = _turn(s)
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x, dn = s[name].float(), _rotated(s["d" + name].float(), cos, -sin, c)
            r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            g = dn * w.float()
            out["d" + name] = (r * (g - x * (r * r) * (g * x).mean(-1, keepdim=True))).to(_DT[c["dy"]])
            out["dw" + name] = (dn * (x * r)).sum((0, 1))
        return out
    if op == "gated_ffn":
        x = s["x"].float()
        gate, up = x @ s["wg"].float().T, x @ s["wu"].float().T
        h = (_act(gate, c["act"])[0] * up).to(_DT[c["x"]])
        return {"h": h, "gate": gate.to(_DT[c["x"]]), "up": up.to(_DT[c["x"]])} if c["keep"] else h
    if op == "gated_ffn_back":
        x, dh, up = s["x"].float(), s["dh"].float(), s["up"].float()
        a, da = _act(s["gate"].float(), c["act"])
        dg, du = dh * up * da, dh * a
        t = _DT[c["dh"]]
        return {"dx": (dg @ s["wg"].float() + du @ s["wu"].float()).to(t), "dwg": (dg.T @ x).to(t), "dwu": (du.T @ x).to(t)}
    x = s["x"].float()
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NORM_EPS)
    tall = c["M"] > c["N"]
    x = x.transpose(1, 2) if tall else x
    for _ in range(STEPS):
        a = x @ x.transpose(1, 2)
        x = COEF[0] * x + (COEF[1] * a + COEF[2] * (a @ a)) @ x
    return (x.transpose(1, 2) if tall else x).contiguous().to(_DT[c["y"]])


def _turn(s):
    """cos and sin of position times frequency, the angle in 64 bits: far positions lose it in 32."""
    angle = s["pos"].double()[:, None] * s["freqs"].double()[None, :]
    return torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]


def _rotated(n, cos, sin, c):
    """The first `rot` of each head's values turned as pairs, the others as they are."""
    half = c["rot"] // 2
    if c["halves"]:
        a, b = n[..., :half], n[..., half:2 * half]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, n[..., 2 * half:]], -1)
    a, b = n[..., 0:2 * half:2], n[..., 1:2 * half:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), n[..., 2 * half:]], -1)


def _act(v, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return v * s, s * (1.0 + v * (1.0 - s))
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (v + 0.044715 * v * v * v))
        return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * v * v)
    if kind == "gelu_erf":
        e = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
        return v * e, e + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return v.clamp(min=0), (v > 0).to(v.dtype)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    with torch.no_grad():
        if op == "qk_norm_rope":
            return {n: _exact_heads(s, s[n], s["w" + n]) for n in ("q", "k")}
        if op == "qk_norm_rope_back":
            out = {}
            for n in ("q", "k"):
                out["d" + n], out["dw" + n] = _exact_heads_back(s, s["d" + n], s[n], s["w" + n])
            return out
        if op == "gated_ffn":
            gate, up = (torch.einsum("tk,fk->tf", s["x"].double(), s[w].double()) for w in ("wg", "wu"))
            h = _exact_act(gate, case["act"]) * up
            return {"h": h, "gate": gate, "up": up} if case["keep"] else h
        if op == "gated_ffn_back":
            return _exact_ffn_back(s)
        return _exact_orthogonal(s)


def _turns(s):
    """The pairs of a head as complex numbers' indices, and exp(i * position * frequency) for each token."""
    half = s["case"]["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (i, i + half) if s["case"]["halves"] else (2 * i, 2 * i + 1)
    return first, second, torch.exp(1j * torch.outer(s["pos"].double(), s["freqs"].double()))[:, None, :]


def _exact_heads(s, x, w):
    first, second, turn = _turns(s)
    x = x.double()
    y = x * w.double() / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) ** 0.5
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_heads_back(s, dy, x, w):
    """dx by the norm's Jacobian r (I - x x' r^2 / D) applied to w * dn, dn the gradient turned back."""
    first, second, turn = _turns(s)
    x, dn, D = x.double(), dy.double(), x.shape[-1]
    z = torch.complex(dn[..., first], dn[..., second]) * turn.conj()
    dn[..., first], dn[..., second] = z.real, z.imag
    ms = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + EPS
    g = dn * w.double()
    dx = (g - x * (torch.einsum("thd,thd->th", g, x)[..., None] / (D * ms))) / ms ** 0.5
    return dx, torch.einsum("thd,thd->d", dn, x / ms ** 0.5)


def _exact_act(v, kind):
    if kind == "silu":
        return v * torch.sigmoid(v)
    if kind == "gelu_tanh":                              # (1 + tanh z) / 2 is the logistic function of 2 z
        return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))
    if kind == "gelu_erf":
        return v * torch.special.ndtr(v)
    return torch.where(v > 0, v, torch.zeros_like(v))


def _exact_slope(v, kind):
    if kind == "silu":
        s = torch.sigmoid(v)
        return s + v * s * torch.sigmoid(-v)
    if kind == "gelu_tanh":
        k = math.sqrt(8.0 / math.pi)
        z = k * (v + 0.044715 * v ** 3)
        return torch.sigmoid(z) + v * torch.sigmoid(z) * torch.sigmoid(-z) * (k + 3 * k * 0.044715 * v ** 2)
    if kind == "gelu_erf":
        return torch.special.ndtr(v) + v * torch.exp(-v ** 2 / 2) * (2 * math.pi) ** -0.5
    return torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))


def _exact_ffn_back(s):
    kind, gate, dh = s["case"]["act"], s["gate"].double(), s["dh"].double()
    du = dh * _exact_act(gate, kind)
    dg = dh * s["up"].double() * _exact_slope(gate, kind)
    x = s["x"].double()
    dx = torch.einsum("tf,fk->tk", dg, s["wg"].double())
    dx += torch.einsum("tf,fk->tk", du, s["wu"].double())
    return {"dx": dx, "dwg": torch.einsum("tf,tk->fk", dg, x), "dwu": torch.einsum("tf,tk->fk", du, x)}


def _exact_orthogonal(s):
    """The steps from the other side: X (a + b G + c G G) with G = X' X, or the plain side where that is the smaller one,
    the polynomial by Horner's rule."""
    x = s["x"].double()
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + NORM_EPS)
    a, b, c = COEF
    right = x.shape[1] > x.shape[2]
    eye = torch.eye(min(x.shape[1], x.shape[2]), dtype=torch.float64, device="cuda")
    for _ in range(STEPS):
        g = torch.einsum("bmi,bmj->bij", x, x) if right else torch.einsum("bin,bjn->bij", x, x)
        p = a * eye + torch.bmm(g, b * eye + c * g)
        x = torch.bmm(x, p) if right else torch.bmm(p, x)
    return x
