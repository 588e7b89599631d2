"""The training operators around the matmul backward, as cases that can be timed and compared.

A step of adapter tuning on preference pairs runs, next to the matrix products of this library:

  get_rows               token embeddings from a plain or block-quantised table, scaled
  get_rows_back          the table's gradient, tokens that occur often summed once
  layer_norm             y = (x - mean) * rstd * w + b over each row, with the statistics kept
  layer_norm_back        dx, and the weight's and the bias's gradients over all rows
  dropout                the adapter's input dropout, its mask regenerated from a counter and never stored
  preference_loss        token log probabilities from logits, paired log ratios, the loss of each pair
  preference_loss_back   the gradient of the mean loss with respect to the logits

``run`` computes a case in elementary torch operations in 32 bits (``own`` false) or through this package's public
calls (``own`` true); ``exact`` computes it from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_BLOCK = {"q8_0": (32, 34), "q4_0": (32, 18)}          # elements, bytes
EPS = 1e-5
BETA, SMOOTHING = 0.1, 0.02
SEED, OFFSET = 0x5EED0123456789AB, 0x0000000700000003  # dropout's key and stream


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of a generation: the embedding of a quantised model, where only latency counts
        {"name": "get_rows q8_0 1 token", "op": "get_rows", "table": "q8_0", "out": "f32", "V": 32000, "M": 2560, "T": 1},
        # the prompt tokens of a whole batch from a 16-bit table, scaled by the root of the width
        {"name": "get_rows bf16 16k tokens", "op": "get_rows", "table": "bf16", "out": "bf16", "V": 128000, "M": 4096, "T": 16384},
        # the dense gradient of a trained embedding over one batch, word frequencies as in text
        {"name": "get_rows_back f32 8k tokens", "op": "get_rows_back", "dy": "f32", "V": 50257, "M": 2560, "T": 8192},
        # a few tokens of one sequence at the adapter workload's width
        {"name": "layer_norm f32 5 rows", "op": "layer_norm", "x": "f32", "w": "f32", "M": 2560, "T": 5},
        # the activations of a large training batch
        {"name": "layer_norm bf16 16k rows", "op": "layer_norm", "x": "bf16", "w": "f32", "M": 5120, "T": 16384},
        # an odd width and an odd number of tokens
        {"name": "layer_norm_back f32 odd", "op": "layer_norm_back", "x": "f32", "dy": "f32", "w": "f32", "M": 2561, "T": 777},
        # the backward pass of the same large batch
        {"name": "layer_norm_back bf16 16k rows", "op": "layer_norm_back", "x": "bf16", "dy": "bf16", "w": "f32", "M": 5120, "T": 16384},
        # the input of one adapter: the rank-r workload's 512 tokens of width 2560
        {"name": "dropout f32 512 rows", "op": "dropout", "x": "f32", "M": 2560, "T": 512, "p": 0.05},
        # the widest adapter input of a layer over a large batch
        {"name": "dropout bf16 16k rows", "op": "dropout", "x": "bf16", "M": 9728, "T": 16384, "p": 0.1},
        # one pair of short answers
        {"name": "preference f32 1 pair", "op": "preference_loss", "x": "f32", "V": 32000, "P": 1, "L": 24},
        # eight pairs of long answers over a large vocabulary: the largest single read of such a step
        {"name": "preference bf16 8 pairs", "op": "preference_loss", "x": "bf16", "V": 128000, "P": 8, "L": 1024},
        # the gradient of four pairs over a vocabulary whose rows are not aligned
        {"name": "preference_back bf16 4 pairs", "op": "preference_loss_back", "x": "bf16", "d": "bf16", "V": 50257, "P": 4, "L": 1024},
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of lo..hi."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n != 3072 else 3073


def draw(rng):
    op = rng.choice(["get_rows", "get_rows_back", "layer_norm", "layer_norm_back", "dropout", "preference_loss",
                     "preference_loss_back"])
    if op == "get_rows":
        table = rng.choice(["f32", "f16", "bf16", "q8_0", "q4_0"])
        M = 32 * _between(rng, 4, 160) if table in _BLOCK else _between(rng, 64, 5120)
        return {"op": op, "table": table, "out": rng.choice(["f32", "bf16"]), "V": _between(rng, 1000, 128000),
                "M": M if M != 3072 else 3104, "T": _between(rng, 1, 16384)}
    if op == "get_rows_back":
        return {"op": op, "dy": rng.choice(["f32", "bf16"]), "V": _between(rng, 500, 50257),
                "M": _between(rng, 64, 2560), "T": _between(rng, 1, 16384)}
    if op == "layer_norm":
        return {"op": op, "x": rng.choice(["f32", "f16", "bf16"]), "w": rng.choice(["f32", "bf16"]),
                "M": _between(rng, 64, 17408), "T": _between(rng, 1, 4096)}
    if op == "layer_norm_back":
        return {"op": op, "x": rng.choice(["f32", "f16", "bf16"]), "dy": rng.choice(["f32", "bf16"]),
                "w": rng.choice(["f32", "bf16"]), "M": _between(rng, 64, 12000), "T": _between(rng, 1, 6144)}
    if op == "dropout":
        return {"op": op, "x": rng.choice(["f32", "f16", "bf16"]), "M": _between(rng, 64, 17408),
                "T": _between(rng, 1, 8192), "p": rng.choice([0.0, 0.05, 0.1, 0.5])}
    if op == "preference_loss":
        return {"op": op, "x": rng.choice(["f32", "f16", "bf16"]), "V": _between(rng, 500, 128000),
                "P": _between(rng, 1, 8), "L": _between(rng, 1, 512)}
    return {"op": op, "x": rng.choice(["f32", "bf16"]), "d": rng.choice(["f32", "bf16"]), "V": _between(rng, 500, 100000),
            "P": _between(rng, 1, 4), "L": _between(rng, 1, 768)}


def _sequences(case):
    """The packed sequences of P pairs, all the chosen ones first: (first rows, [(rows, prompt rows)])."""
    L, lens = case["L"], []
    for s in range(2 * case["P"]):
        n = max(1, L - (s * 37 + s * s * 11) % (L // 3 + 1))
        lens.append((n, n // 4))
    first = [0]
    for n, _ in lens:
        first.append(first[-1] + n)
    return first, lens


def work(case):
    op = case["op"]
    if op == "get_rows":
        t, m = case["T"], case["M"]
        row = m // _BLOCK[case["table"]][0] * _BLOCK[case["table"]][1] if case["table"] in _BLOCK else m * _SIZE[case["table"]]
        # rows that occur again are counted once for each time: which ones do is the data's
        return {"bytes": t * (row + 4 + m * _SIZE[case["out"]]), "flops": 2 * t * m}
    if op == "get_rows_back":
        t, m = case["T"], case["M"]
        return {"bytes": t * (4 + m * _SIZE[case["dy"]]) + 4 * case["V"] * m, "flops": 2 * t * m}
    if op == "layer_norm":
        t, m = case["T"], case["M"]
        return {"bytes": 2 * t * m * _SIZE[case["x"]] + 2 * m * _SIZE[case["w"]] + 8 * t, "flops": 8 * t * m}
    if op == "layer_norm_back":
        t, m = case["T"], case["M"]
        return {"bytes": t * m * (_SIZE[case["x"]] + 2 * _SIZE[case["dy"]]) + m * _SIZE[case["w"]] + 8 * m + 8 * t,
                "flops": 14 * t * m}
    if op == "dropout":
        return {"bytes": 2 * case["T"] * case["M"] * _SIZE[case["x"]], "flops": 2 * case["T"] * case["M"]}
    first, lens = _sequences(case)
    rows, scored = first[-1], sum(n - k for n, k in lens)
    if op == "preference_loss":
        return {"bytes": scored * case["V"] * _SIZE[case["x"]] + 16 * rows, "flops": 4 * scored * case["V"]}
    return {"bytes": case["V"] * (scored * _SIZE[case["x"]] + rows * _SIZE[case["d"]]) + 8 * rows,
            "flops": 4 * scored * case["V"]}


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


def _tokens(g, n, vocab):
    """Token ids whose frequencies fall as 1/rank, as those of words do."""
    u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1).int()


def _quantised(g, V, M, kind):
    """Rows of blocks: a binary16 scale of a weight around 0.02, then random codes."""
    elems, size = _BLOCK[kind]
    blocks = torch.randint(0, 256, (V, M // elems, size), device="cuda", generator=g, dtype=torch.uint8)
    d = (torch.rand((V, M // elems, 1), device="cuda", generator=g) * 0.5 + 0.75) * (0.06 / (127 if kind == "q8_0" else 8))
    blocks[:, :, :2] = d.half().view(torch.uint8)
    return blocks.reshape(V, -1)


def _token_logps(logits, labels):
    """(log normaliser, log probability of the label) of each row, a block of rows at a time; 0 where the label is negative."""
    lse, lp = torch.zeros(len(labels), device="cuda"), torch.zeros(len(labels), device="cuda")
    for a in range(0, len(labels), 512):
        x, lab = logits[a:a + 512].float(), labels[a:a + 512].long()
        z = torch.logsumexp(x, 1)
        lse[a:a + 512] = torch.where(lab >= 0, z, torch.zeros_like(z))
        picked = x.gather(1, lab.clamp(min=0)[:, None])[:, 0]
        lp[a:a + 512] = torch.where(lab >= 0, picked - z, torch.zeros_like(z))
    return lse, lp


def prepare(case, seed):
    op, g = case["op"], _generator(seed)
    if op == "get_rows":
        V, M = case["V"], case["M"]
        table = _quantised(g, V, M, case["table"]) if case["table"] in _BLOCK else _normal(g, (V, M), case["table"], 0.02)
        return {"case": case, "table": table, "ids": _tokens(g, case["T"], V), "scale": math.sqrt(M)}
    if op == "get_rows_back":
        return {"case": case, "dy": _normal(g, (case["T"], case["M"]), case["dy"]), "ids": _tokens(g, case["T"], case["V"]),
                "scale": math.sqrt(case["M"])}
    if op in ("layer_norm", "layer_norm_back"):
        T, M = case["T"], case["M"]
        x = _normal(g, (T, M), case["x"], 1.5, 0.3)
        s = {"case": case, "x": x, "w": _normal(g, (M,), case["w"], 0.2, 1.0), "b": _normal(g, (M,), case["w"], 0.1)}
        if op == "layer_norm_back":
            s["dy"] = _normal(g, (T, M), case["dy"])
            s["mean"] = x.float().mean(1)
            s["rstd"] = torch.rsqrt(x.float().var(1, unbiased=False) + EPS)
        return s
    if op == "dropout":
        return {"case": case, "x": _normal(g, (case["T"], case["M"]), case["x"])}
    first, lens = _sequences(case)
    T, V = first[-1], case["V"]
    logits = _normal(g, (T, V), case["x"], 2.5)
    labels = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    rows = torch.arange(T, device="cuda")
    logits[rows, labels.long()] += 8.0                     # a model that mostly knows the next token
    for (n, prompt), a in zip(lens, first):
        labels[a:a + prompt] = -1                          # the prompt is not scored
    seq = torch.tensor(first, dtype=torch.int32, device="cuda")
    lse, logps = _token_logps(logits, labels)
    ref = logps + 0.15 * torch.randn(T, device="cuda", generator=g)
    s = {"case": case, "logits": logits, "labels": labels, "seq": seq, "ref": ref}
    if op == "preference_loss_back":
        diff = torch.where(labels >= 0, logps - ref, torch.zeros_like(ref))
        s["lse"], s["ratios"] = lse, _segment_sums(diff, seq)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _own_run(state) if own else _plain_run(state)


def _own_run(s):
    import ggml_out_prod_gb300 as oop

    c = s["case"]
    op = c["op"]
    if op == "get_rows":
        kind = {"q8_0": oop.TYPE_Q8_0, "q4_0": oop.TYPE_Q4_0}.get(c["table"])
        return oop.get_rows(s["table"], s["ids"], scale=s["scale"], table_type=kind, out_dtype=_DT[c["out"]])
    if op == "get_rows_back":
        return oop.get_rows_back(s["dy"], s["ids"], c["V"], scale=s["scale"])
    if op == "layer_norm":
        y, mean, rstd = oop.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "layer_norm_back":
        dx, dw, db = oop.layer_norm_back(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "dropout":
        return oop.dropout(s["x"], c["p"], SEED, OFFSET)
    if op == "preference_loss":
        r = oop.preference_loss(s["logits"], s["labels"], s["seq"], ref_logps=s["ref"], beta=BETA, label_smoothing=SMOOTHING)
        return {"loss": r.loss, "losses": r.losses, "ratios": r.ratios, "logps": r.logps, "lse": r.lse}
    return oop.preference_loss_back(s["logits"], s["labels"], s["seq"], s["lse"], s["ratios"], beta=BETA,
                                    label_smoothing=SMOOTHING, out_dtype=_DT[c["d"]])


def _plain_run(s):
    c = s["case"]
    op = c["op"]
    if op == "get_rows":
        rows = s["table"][s["ids"].long()]
        return (_plain_values(rows, c["table"]) * s["scale"]).to(_DT[c["out"]])
    if op == "get_rows_back":
        d = torch.zeros((c["V"], c["M"]), device="cuda")
        return d.index_add_(0, s["ids"].long(), s["dy"].float() * s["scale"])
    if op == "layer_norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
        y = xc * rstd * s["w"].float() + s["b"].float()
        return {"y": y.to(_DT[c["x"]]), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "layer_norm_back":
        dy, xh = s["dy"].float(), (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["w"].float()
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return {"dx": dx.to(_DT[c["dy"]]), "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    if op == "dropout":
        drop = min(65536, int(round(c["p"] * 65536)))
        keep = _plain_uniform16(c["T"], c["M"]) >= drop
        return torch.where(keep, s["x"].float() * (65536.0 / (65536 - drop)), 0.0).to(_DT[c["x"]])
    if op == "preference_loss":
        at = torch.nonzero(s["labels"] >= 0)[:, 0]
        x, lab = s["logits"][at].float(), s["labels"][at].long()
        top = x.max(1, keepdim=True).values
        z = top[:, 0] + torch.log(torch.exp(x - top).sum(1))
        lse = torch.zeros(len(s["labels"]), device="cuda")
        logps = torch.zeros_like(lse)
        lse[at] = z
        logps[at] = x.gather(1, lab[:, None])[:, 0] - z
        diff = torch.where(s["labels"] >= 0, logps - s["ref"], torch.zeros_like(lse))
        ratios = _segment_sums(diff, s["seq"])
        m = BETA * (ratios[:c["P"]] - ratios[c["P"]:])
        losses = (1 - SMOOTHING) * _softplus(-m) + SMOOTHING * _softplus(m)
        return {"loss": losses.mean(), "losses": losses, "ratios": ratios, "logps": logps, "lse": lse}
    m = BETA * (s["ratios"][:c["P"]] - s["ratios"][c["P"]:])
    slope = (BETA / c["P"]) * (SMOOTHING / (1 + torch.exp(-m)) - (1 - SMOOTHING) / (1 + torch.exp(m)))
    of_seq = torch.cat([slope, -slope])
    n = len(s["labels"])
    which = (torch.arange(n, device="cuda")[:, None] >= s["seq"][None, 1:]).sum(1)
    coef = torch.where(s["labels"] >= 0, of_seq[which], torch.zeros(n, device="cuda"))
    p = torch.exp(s["logits"].float() - s["lse"][:, None])
    d = torch.where(coef[:, None] != 0, p * -coef[:, None], 0.0)
    rows = torch.arange(n, device="cuda")
    d[rows, s["labels"].long().clamp(min=0)] += coef
    return d.to(_DT[c["d"]])


def _softplus(x):
    """log(1 + exp(x)) without overflow."""
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _segment_sums(v, first):
    """The sum of v over each of the packed sequences."""
    t = torch.arange(len(v), device=v.device)
    inside = (t[None, :] >= first[:-1, None]) & (t[None, :] < first[1:, None])
    return torch.where(inside, v[None, :], torch.zeros_like(v)[None, :]).sum(1)


def _plain_values(rows, kind):
    """The values of rows of a table: float32."""
    if kind not in _BLOCK:
        return rows.float()
    blocks = rows.reshape(len(rows), -1, _BLOCK[kind][1])
    d = blocks[:, :, :2].contiguous().view(torch.float16).float()
    codes = blocks[:, :, 2:]
    if kind == "q8_0":
        q = codes.contiguous().view(torch.int8).float()
    else:
        q = torch.cat([codes & 15, codes >> 4], 2).float() - 8.0
    return (d * q).reshape(len(rows), -1)


def _plain_uniform16(T, M):
    """16 random bits for each element: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
    as 1, 2, 3", SC 2011) with the counter (column group of 8, row, offset low, offset high) and the key (seed low,
    high). A call gives four 32-bit words, the low half of each first: one half for each column of the group."""
    groups = (M + 7) // 8
    low = 0xFFFFFFFF
    c0 = torch.arange(groups, device="cuda")[None, :].expand(T, groups)
    c1 = torch.arange(T, device="cuda")[:, None].expand(T, groups)
    c2 = torch.full((T, groups), OFFSET & low, device="cuda")
    c3 = torch.full((T, groups), OFFSET >> 32, device="cuda")
    k0, k1 = SEED & low, SEED >> 32
    for _ in range(10):
        h0, l0 = _wide(c0, 0xD2511F53)
        h1, l1 = _wide(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    halves = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 2)
    return halves.reshape(T, groups * 8)[:, :M]


def _wide(a, m):
    """The two 32-bit halves of a * m, both below 2^32, in 64-bit signed arithmetic."""
    return ((a >> 16) * m + ((a & 0xFFFF) * m >> 16)) >> 16, (a * m) & 0xFFFFFFFF


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    with torch.no_grad():
        if op == "get_rows":
            return _exact_rows(s)
        if op == "get_rows_back":
            out = torch.zeros((case["V"], case["M"]), dtype=torch.float64, device="cuda")
            order = torch.argsort(s["ids"].long(), stable=True)
            out.index_put_((s["ids"].long()[order],), s["dy"].double()[order] * s["scale"], accumulate=True)
            return out
        if op == "layer_norm":
            x = s["x"].double()
            mean, var = x.mean(1), x.var(1, unbiased=False)
            rstd = (var + EPS) ** -0.5
            y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double())
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "layer_norm_back":
            return _exact_norm_back(s)
        if op == "dropout":
            return _exact_dropout(s)
        if op == "preference_loss":
            return _exact_preference(s)
        return _exact_preference_back(s)


def _exact_rows(s):
    kind, ids = s["case"]["table"], s["ids"].long().cpu().numpy()
    if kind not in _BLOCK:
        return s["table"].index_select(0, s["ids"].long()).double() * s["scale"]
    elems, size = _BLOCK[kind]
    raw = s["table"].index_select(0, s["ids"].long()).cpu().numpy().reshape(len(ids), -1, size)
    d = np.ascontiguousarray(raw[:, :, :2]).view(np.float16).astype(np.float64)
    v = np.empty(raw.shape[:2] + (elems,))
    if kind == "q8_0":
        v[...] = np.ascontiguousarray(raw[:, :, 2:]).view(np.int8)
    else:
        v[:, :, :16] = (raw[:, :, 2:] % 16).astype(np.float64) - 8
        v[:, :, 16:] = (raw[:, :, 2:] // 16).astype(np.float64) - 8
    return (d * v).reshape(len(ids), -1) * s["scale"]


def _exact_norm_back(s):
    """dx as the product of the row's Jacobian (rstd / M) (M I - 1 1' - xhat xhat') with w * dy. The statistics are
    inputs, rounded to 32 bits by the forward pass."""
    M = s["x"].shape[1]
    xh = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
    dy = s["dy"].double()
    g = dy * s["w"].double()
    dx = (s["rstd"].double()[:, None] / M) * (M * g - g.sum(1, keepdim=True) - xh * torch.einsum("tm,tm->t", g, xh)[:, None])
    return {"dx": dx, "dw": torch.einsum("tm,tm->m", dy, xh), "db": dy.sum(0)}


def _exact_dropout(s):
    T, M, p = s["case"]["T"], s["case"]["M"], s["case"]["p"]
    x = s["x"].double().cpu().numpy()
    drop = min(65536, int(round(p * 65536)))
    out = np.zeros((T, M))
    groups = -(-M // 8)
    for a in range(0, T, 1024):                            # a block of rows at a time
        rows = np.arange(a, min(T, a + 1024), dtype=np.uint64)
        c = np.zeros((len(rows), groups, 4), dtype=np.uint64)
        c[:, :, 0] = np.arange(groups, dtype=np.uint64)
        c[:, :, 1] = rows[:, None]
        c[:, :, 2], c[:, :, 3] = OFFSET % 2 ** 32, OFFSET // 2 ** 32
        key = [SEED % 2 ** 32, SEED // 2 ** 32]
        for _ in range(10):
            first, second = c[:, :, 0] * np.uint64(0xD2511F53), c[:, :, 2] * np.uint64(0xCD9E8D57)
            c[:, :, 0] = (second >> np.uint64(32)) ^ c[:, :, 1] ^ np.uint64(key[0])
            c[:, :, 2] = (first >> np.uint64(32)) ^ c[:, :, 3] ^ np.uint64(key[1])
            c[:, :, 1], c[:, :, 3] = second & np.uint64(0xFFFFFFFF), first & np.uint64(0xFFFFFFFF)
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        bits = c.astype("<u4").view("<u2").reshape(len(rows), groups * 8)[:, :M]
        part = x[a:a + len(rows)]
        if drop < 65536:
            out[a:a + len(rows)] = np.where(bits >= drop, part * (65536.0 / (65536 - drop)), 0.0)
    return out


def _exact_preference(s):
    P, T = s["case"]["P"], len(s["labels"])
    lse, logps = np.zeros(T), np.zeros(T)
    labels = s["labels"].cpu().numpy()
    for a in range(0, T, 512):
        x = s["logits"][a:a + 512].double()
        z = torch.logsumexp(x, 1).cpu().numpy()
        lab = torch.from_numpy(np.maximum(labels[a:a + 512], 0)).long().cuda()
        picked = torch.take_along_dim(x, lab[:, None], 1)[:, 0].cpu().numpy()
        use = labels[a:a + 512] >= 0
        lse[a:a + 512], logps[a:a + 512] = np.where(use, z, 0.0), np.where(use, picked - z, 0.0)
    ref, first = s["ref"].double().cpu().numpy(), s["seq"].cpu().numpy()
    diff = np.where(labels >= 0, logps - ref, 0.0)
    ratios = np.array([math.fsum(diff[a:b]) for a, b in zip(first[:-1], first[1:])])
    m = BETA * (ratios[:P] - ratios[P:])
    losses = (1 - SMOOTHING) * np.logaddexp(0.0, -m) + SMOOTHING * np.logaddexp(0.0, m)
    return {"loss": float(losses.mean()), "losses": losses, "ratios": ratios, "logps": logps, "lse": lse}


def _exact_preference_back(s):
    P, T = s["case"]["P"], len(s["labels"])
    ratios, first = s["ratios"].double().cpu().numpy(), s["seq"].cpu().numpy()
    labels, lse = s["labels"].cpu().numpy(), s["lse"].double()
    coef = np.zeros(T)
    for i in range(P):
        m = BETA * (ratios[i] - ratios[P + i])
        sigma = 1.0 / (1.0 + math.exp(-m))
        slope = BETA / P * (SMOOTHING * sigma - (1.0 - SMOOTHING) * (1.0 - sigma))
        coef[first[i]:first[i + 1]] = slope
        coef[first[P + i]:first[P + i + 1]] = -slope
    coef[labels < 0] = 0.0
    c = torch.from_numpy(coef).cuda()
    out = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, T, 512):
        part = out[a:a + 512]
        part.copy_(torch.exp(s["logits"][a:a + 512].double() - lse[a:a + 512, None]) * -c[a:a + 512, None])
        part[torch.as_tensor(coef[a:a + 512] == 0.0, device="cuda")] = 0.0
        rows = torch.arange(len(part), device="cuda")
        lab = torch.from_numpy(np.maximum(labels[a:a + 512], 0)).long().cuda()
        part[rows, lab] += c[a:a + 512]
    return out
