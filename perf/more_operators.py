"""Measured cases of the operators between the embedding's lookup and the flat
gradient: a layer's matrix product with bias, activation and residual in its
epilogue, its gradients, the exact top logits of a teacher's rows, and the
distillation loss from them with its gradient.

A case is one call.  run() computes it with elementary torch operations in 32
bits (own = False), or through gradient_compression_dnn_amd.binding (own =
True); exact() gives the same outputs from the definitions in 64 bits.

Layer: W is a segment of the flat model read as rows x cols, b another of rows
elements.  Forward z = x W^T + b, y = act(z) + r; "dz" dz = dy act'(z); "input"
g = dz W + a, dx = g and dzx = g act'(z) with the z of the layer that made x;
"weight" G[W] (+)= dz^T x, G[b] (+)= sum of dz over the tokens.
Top logits: the k entries of a row first in the order (value descending, index
ascending), without -Inf; -1 and -Inf behind the last one; lse = log sum exp(z / T).
Distillation, per row: q = softmax(t / T) over the teacher's entries, or
exp(t / T - lse) with the rest of the mass, q_r = max(0, 1 - sum q), on the rest
of the row; KL = sum q (log q - log p), p = softmax(z / T), with one more term
for the rest; L = weight (kd T^2 KL + ce (log sum exp(z) - z[label])), and its
gradient times grad_scale.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


# --------------------------------------------------------------------- cases
def listed():
    layer = dict(op="forward", n=700, cols=1500, rows=10000, type="bf16", bias=True, act="none", extra=False, keep=False, lead=0, pitch=0)
    top = dict(op="top", n=4096, vocab=131071, k=64, type="bf16", temp=1.0, masked=0.0, pitch=0)
    kd = dict(op="distill", n=700, vocab=10000, k=32, type="f32", temp=2.0, ce=0.5, tail=False, empty=0.0, masked=0.0, pitch=0)
    return [
        # one token through the first matrix of a feed-forward block
        dict(layer, name="forward one token", n=1, cols=4096, rows=16384, act="gelu"),
        # the output layer of the LSTM language model over its batch of 20 sequences of 35 tokens
        dict(layer, name="forward lstm output", type="f32"),
        # a feed-forward block's first matrix in training, the argument of its activation kept for the way back
        dict(layer, name="forward large", n=8192, cols=4096, rows=16384, act="gelu_tanh", keep=True),
        # odd sizes at an odd offset of the flat buffer, half precision, with a residual
        dict(layer, name="forward odd residual", n=1023, cols=4099, rows=1501, type="f16", act="silu", extra=True, lead=3),
        # from the gradient of the logits back into the LSTM
        dict(layer, name="input lstm output", op="input", bias=False),
        # back through the large matrix's partner into its activation, with the gradient of a skip connection
        dict(layer, name="input large", op="input", n=8192, cols=16384, rows=4096, bias=False, act="gelu_tanh", extra=True),
        # the output layer's own gradient, added to that of an earlier micro batch
        dict(layer, name="weight lstm add", op="weight", type="f16", extra=True),
        # the large matrix's gradient, written over its segment
        dict(layer, name="weight large", op="weight", n=8192, cols=4096, rows=16384),
        # a step of 20 sequences of the LSTM as the teacher
        dict(top, name="top step", n=20, vocab=10000, k=8, type="f32", temp=2.0),
        # a teacher's long batch over a large vocabulary
        dict(top, name="top large"),
        # the LSTM as the student, half of the loss from labels
        dict(kd, name="distill lstm"),
        # a long batch over the large vocabulary, the rest of the teacher's mass held too, some rows without a teacher
        dict(kd, name="distill large", n=4096, vocab=131071, k=64, type="bf16", temp=1.0, ce=0.0, tail=True, empty=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("forward", "forward", "input", "weight", "dz", "top", "distill", "distill"))
    kind = rng.choice(("f32", "bf16", "f16"))
    if op in ("top", "distill"):
        n, vocab = _log_int(rng, 1, 4096), _log_int(rng, 500, 131071)
        while kind == "f32" and n * vocab > 2048 * 131071:
            n //= 2
        case = dict(op=op, n=n, vocab=vocab, k=min(_log_int(rng, 1, 256), vocab // 4), type=kind, temp=rng.choice((1.0, 2.0, 4.0)),
                    masked=rng.choice((0.0, 0.0, 0.02)), pitch=rng.choice((0, 0, 8, 5)))
        if op == "distill":
            case.update(ce=rng.choice((0.0, 0.5)), tail=rng.random() < 0.5, empty=rng.choice((0.0, 0.1)))
        return case
    # single tokens and short batches as often as long ones
    n, rows, cols = _log_int(rng, 1, 8192), _log_int(rng, 48, 16384), _log_int(rng, 48, 16384)
    while n * rows * cols > 8192.0 * 4096 * 16384 / (8 if kind == "f32" else 1):
        n //= 2
    if op == "dz":
        rows = cols
    bias = op == "forward" and rng.random() < 0.5 or op == "weight" and rng.random() < 0.5
    return dict(op=op, n=n, cols=cols, rows=rows, type=kind, bias=bias,
                act="none" if op == "weight" else rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                extra=op != "dz" and rng.random() < 0.5, keep=op == "forward" and rng.random() < 0.5, lead=rng.choice((0, 0, 8, 3)),
                pitch=rng.choice((0, 0, 8, 5)))


# --------------------------------------------------------------------- inputs
def _rows(n, cols, pitch, type, g, scale=1.0):
    """n rows of cols normal values, `pitch` elements between them."""
    t = torch.zeros(n, cols + pitch, dtype=TYPES[type], device="cuda")[:, :cols]
    return t.copy_(torch.randn(n, cols, generator=g, device="cuda") * scale)


def _logits(case, g):
    """Logits as a trained model's: frequent tokens above rare ones, and noise."""
    n, v = case["n"], case["vocab"]
    z = torch.zeros(n, v + case["pitch"], dtype=TYPES[case["type"]], device="cuda")[:, :v]
    prior = -torch.log(1.0 + torch.randperm(v, generator=g, device="cuda").float())
    for at in range(0, n, 512):  # a part at a time: float32 noise of all rows would be the largest array here
        m = min(512, n - at)
        z[at:at + m].copy_(0.6 * prior + 2.5 * torch.randn(m, v, generator=g, device="cuda"))
    if case["masked"]:
        z[:, v - max(1, int(case["masked"] * v)):] = -INF  # columns that only fill up the vocabulary
    return z


def _grad_scale(case):
    """The mean over the rows; in half precision times a loss scale."""
    return (1024.0 if case["type"] == "f16" else 1.0) / case["n"]


def _binding():
    from gradient_compression_dnn_amd import binding as B
    return B


def _plan(s, lengths):
    """The flat model's plan: a segment for the elements in front, then those of `lengths`."""
    import numpy as np
    B = _binding()
    at = np.cumsum([0] + lengths)
    keep = [i for i, n in enumerate(lengths) if n]
    s["plan"] = B.Plan(np.array([(int(at[i]), lengths[i], 64, max(1, lengths[i] // 1000)) for i in keep], dtype=np.int64), int(at[-1]))
    return [keep.index(i) if i in keep else -1 for i in range(len(lengths))]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    n, pitch = case["n"], case["pitch"]
    if case["op"] == "top":
        s["z"] = _logits(case, g)
        s["idx"] = torch.zeros(n, case["k"], dtype=torch.int32, device="cuda")
        s["val"] = torch.zeros(n, case["k"], device="cuda")
        s["lse"] = torch.zeros(n, device="cuda")
        return s
    if case["op"] == "distill":
        v, k, temp = case["vocab"], case["k"], case["temp"]
        s["z"] = _logits(case, g)
        s["idx"] = torch.zeros(n, k, dtype=torch.int32, device="cuda")
        s["val"] = torch.zeros(n, k, device="cuda")
        s["tlse"] = torch.zeros(n, device="cuda")
        for at in range(0, n, 512):  # the teacher's logits are the student's and a difference
            t = s["z"][at:at + 512].float()
            t = t + 1.5 * torch.randn(t.shape, generator=g, device="cuda")
            top = torch.topk(t, k)
            s["val"][at:at + 512], s["idx"][at:at + 512] = top.values, top.indices.int()
            s["tlse"][at:at + 512] = torch.logsumexp(t / temp, 1)
        s["idx"][n - int(case["empty"] * n):] = -1
        s["labels"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.9, s["idx"][:, 0], -1)
        s["weights"] = torch.rand(n, generator=g, device="cuda") + 0.5
        s["loss"] = torch.zeros(n, device="cuda")
        s["dz"] = torch.zeros(n, v + pitch, dtype=TYPES[case["type"]], device="cuda")[:, :v]
        if own:
            B = _binding()
            s["opt"] = B.distill_options(temperature=temp, kd_weight=1.0, ce_weight=case["ce"], grad_scale=_grad_scale(case), tail=case["tail"])
        return s
    rows, cols, lead, kind = case["rows"], case["cols"], case["lead"], case["type"]
    lengths = [lead, rows * cols, rows if case["bias"] else 0]
    total = sum(lengths)
    if case["op"] in ("forward", "input"):
        s["w"] = (torch.randn(total, generator=g, device="cuda") / math.sqrt(cols if case["op"] == "forward" else rows)).to(TYPES[kind])
    if case["op"] == "forward":
        s["x"] = _rows(n, cols, pitch, kind, g)
        s["r"] = _rows(n, rows, pitch, kind, g) if case["extra"] else None
        s["z"] = _rows(n, rows, pitch, kind, g) if case["keep"] else None
        s["y"] = _rows(n, rows, pitch, kind, g)
    elif case["op"] == "input":
        s["dz"] = _rows(n, rows, pitch, kind, g, 1e-2)
        s["a"] = _rows(n, cols, pitch, kind, g, 1e-2) if case["extra"] else None
        s["z"] = _rows(n, cols, pitch, kind, g) if case["act"] != "none" else None
        s["dx"] = _rows(n, cols, pitch, kind, g)
        s["dzx"] = _rows(n, cols, pitch, kind, g) if case["act"] != "none" else None
    elif case["op"] == "dz":
        s["dy"], s["z"], s["dz"] = (_rows(n, rows, pitch, kind, g) for _ in range(3))
    else:
        s["dz"] = _rows(n, rows, pitch, kind, g, 1e-2)
        s["x"] = _rows(n, cols, pitch, kind, g)
        s["g"] = torch.randn(total, generator=g, device="cuda") * 1e-2
    if own:
        B = _binding()
        _, seg, bias = _plan(s, lengths)
        s["layer"] = B.linear_layer(seg, rows, TYPES[kind], bias)
        s["act"] = {"none": B.GC_ACT_NONE, "relu": B.GC_ACT_RELU, "gelu": B.GC_ACT_GELU, "gelu_tanh": B.GC_ACT_GELU_TANH, "silu": B.GC_ACT_SILU}[case["act"]]
        s["ws"] = torch.empty(B.gc_linear_workspace_bytes(s["plan"], s["layer"], n), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain form
def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0.0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _weights(s, case):
    """W and b of the flat model, in 32 bits."""
    rows, cols, lead = case["rows"], case["cols"], case["lead"]
    w = s["w"][lead:lead + rows * cols].view(rows, cols).float()
    return w, s["w"][lead + rows * cols:].float() if case["bias"] else None


def _plain_layer(s, case):
    if case["op"] == "forward":
        w, b = _weights(s, case)
        z = s["x"].float() @ w.T
        z = z + b if b is not None else z
        if case["keep"]:
            s["z"].copy_(z)
        y = _act(z, case["act"])
        s["y"].copy_(y + s["r"].float() if case["extra"] else y)
        return {"y": s["y"], "z": s["z"]} if case["keep"] else s["y"]
    if case["op"] == "input":
        d = s["dz"].float() @ _weights(s, case)[0]
        d = d + s["a"].float() if case["extra"] else d
        s["dx"].copy_(d)
        if case["act"] == "none":
            return s["dx"]
        s["dzx"].copy_(d * _slope(s["z"].float(), case["act"]))
        return {"dx": s["dx"], "dzx": s["dzx"]}
    if case["op"] == "dz":
        s["dz"].copy_(s["dy"].float() * _slope(s["z"].float(), case["act"]))
        return s["dz"]
    rows, cols, lead = case["rows"], case["cols"], case["lead"]
    dz, x = s["dz"].float(), s["x"].float()
    w, b = s["g"][lead:lead + rows * cols].view(rows, cols), s["g"][lead + rows * cols:]
    if case["extra"]:
        w.add_(dz.T @ x)
        b.add_(dz.sum(0)) if case["bias"] else None
    else:
        w.copy_(dz.T @ x)
        b.copy_(dz.sum(0)) if case["bias"] else None
    return s["g"]


def _plain_top(s, case):
    v, k = case["vocab"], case["k"]
    z = s["z"].float()
    # keys that no two entries share: the value's order above, the index's below
    bits = (z + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    key = torch.where(z > -INF, key + (v - 1 - torch.arange(v, device=z.device)), torch.iinfo(torch.int64).min)
    best = torch.topk(key, k, dim=1)
    there = best.values > torch.iinfo(torch.int64).min
    s["idx"].copy_(torch.where(there, best.indices, -1))
    s["val"].copy_(torch.where(there, torch.gather(z, 1, best.indices), -INF))
    m = z.amax(1, keepdim=True)
    s["lse"].copy_((m / case["temp"]).squeeze(1) + torch.log(torch.exp((z - m) / case["temp"]).sum(1)))
    return {"idx": s["idx"], "val": s["val"], "lse": s["lse"]}


def _plain_distill(s, case):
    temp, ce = case["temp"], case["ce"]
    z = s["z"].float()
    idx = s["idx"].long()
    there = idx >= 0
    at = torch.where(there, idx, 0)
    some = there.any(1, keepdim=True)
    t = torch.where(there, s["val"] / temp, -INF)
    if case["tail"]:
        q = torch.exp(t - s["tlse"][:, None])
    else:
        e = torch.exp(t - torch.where(some, t.amax(1, keepdim=True), 0.0))
        q = e / torch.where(some, e.sum(1, keepdim=True), 1.0)
    m = z.amax(1, keepdim=True)
    zt = (z - m) / temp
    e = torch.exp(zt)
    lse = torch.log(e.sum(1, keepdim=True))
    logp = torch.gather(zt, 1, at) - lse
    kl = torch.where(q > 0.0, q * (torch.log(torch.where(q > 0.0, q, 1.0)) - logp), 0.0).sum(1)
    if case["tail"]:
        # the rest of the row: every column that no entry names
        rest = torch.ones_like(z, dtype=torch.bool)
        rest.scatter_(1, at, ~there)
        held = torch.where(some, torch.clamp(1.0 - q.sum(1, keepdim=True), min=0.0), 0.0)
        zr = torch.where(rest, zt, -INF)
        mr = zr.amax(1, keepdim=True)
        er = torch.exp(zr - mr)
        lr = torch.log(er.sum(1, keepdim=True))
        kl = kl + torch.where(held > 0.0, held * (torch.log(torch.where(held > 0.0, held, 1.0)) - (mr + lr - lse)), 0.0).squeeze(1)
        mass = q.sum(1, keepdim=True) + held
        dz = mass * e / torch.exp(lse) - held * er / torch.exp(lr)
    else:
        dz = q.sum(1, keepdim=True) * (e / torch.exp(lse))
    dz.scatter_add_(1, at, -q)
    dz, loss = temp * dz, temp * temp * kl
    if ce:
        e1 = torch.exp(z - m)
        sum1 = e1.sum(1, keepdim=True)
        label = s["labels"].long()[:, None]
        good = label >= 0
        label = torch.where(good, label, 0)
        loss = loss + torch.where(good, ce * (torch.log(sum1) - torch.gather(z - m, 1, label)), 0.0).squeeze(1)
        dz = dz + torch.where(good, ce, 0.0) * (e1 / sum1)
        dz.scatter_add_(1, label, torch.where(good, -ce, 0.0))
    s["loss"].copy_(s["weights"] * loss)
    s["dz"].copy_(dz * (s["weights"] * _grad_scale(case))[:, None])
    return {"loss": s["loss"], "dz": s["dz"]}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"top": _plain_top, "distill": _plain_distill}.get(op, _plain_layer)(s, case)
    B = _binding()
    if op == "top":
        B.gc_top_logits(s["z"], s["idx"], s["val"], lse=s["lse"], temperature=case["temp"])
        return {"idx": s["idx"], "val": s["val"], "lse": s["lse"]}
    if op == "distill":
        B.gc_distill_loss(s["z"], s["idx"], s["val"], s["opt"], s["loss"], s["dz"], t_lse=s["tlse"] if case["tail"] else None,
                          labels=s["labels"] if case["ce"] else None, weights=s["weights"])
        return {"loss": s["loss"], "dz": s["dz"]}
    if op == "forward":
        B.gc_linear_forward(s["plan"], s["layer"], s["w"], s["x"], s["y"], s["ws"], act=s["act"], r=s["r"], z=s["z"])
        return {"y": s["y"], "z": s["z"]} if case["keep"] else s["y"]
    if op == "input":
        B.gc_linear_grad_input(s["plan"], s["layer"], s["w"], s["dz"], s["dx"], s["ws"], a=s["a"], act=s["act"], z=s["z"], dzx=s["dzx"])
        return s["dx"] if case["act"] == "none" else {"dx": s["dx"], "dzx": s["dzx"]}
    if op == "dz":
        B.gc_act_grad(s["dy"], s["z"], s["act"], s["dz"])
        return s["dz"]
    B.gc_linear_grad_weight(s["plan"], s["layer"], s["dz"], s["x"], s["g"], case["extra"], s["ws"])
    return s["g"]


# ------------------------------------------------------------------------ work
def work(case):
    n, size = case["n"], TYPES[case["type"]].itemsize
    if case["op"] == "top":
        return {"bytes": float(n * case["vocab"] * size + n * case["k"] * 8 + 4 * n), "flops": 3.0 * n * case["vocab"]}
    if case["op"] == "distill":
        return {"bytes": float(2 * n * case["vocab"] * size + n * case["k"] * 8 + 16 * n), "flops": 6.0 * n * case["vocab"]}
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "dz":
        return {"bytes": 3.0 * n * rows * size, "flops": 10.0 * n * rows}
    if case["op"] == "forward":
        move = n * cols + rows * cols + n * rows * (1 + case["extra"] + case["keep"]) + rows * case["bias"]
    elif case["op"] == "input":
        move = n * rows + rows * cols + n * cols * (1 + case["extra"] + 2 * (case["act"] != "none"))
    else:
        move = n * (rows + cols)
    wrote = (8.0 if case["extra"] else 4.0) * rows * (cols + case["bias"]) if case["op"] == "weight" else 0.0
    return {"bytes": float(move * size) + wrote, "flops": 2.0 * n * rows * cols}


# ----------------------------------------------------------------------- exact
def _exact_act(z, act):
    """act(z) and act'(z) in 64 bits."""
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":  # 1 + tanh(u) = 2 sigmoid(2 u)
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * c * (1 + 0.134145 * z ** 2)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    return z, torch.ones_like(z)


def _exact_layer(s, case):
    rows, cols, lead = case["rows"], case["cols"], case["lead"]
    end = lead + rows * cols
    if case["op"] == "dz":
        return s["dy"].double() * _exact_act(s["z"].double(), case["act"])[1]
    if case["op"] == "weight":
        out = s["g"].double()
        if not case["extra"]:
            out[lead:] = 0.0
        out[lead:end] += torch.matmul(s["dz"].double().T, s["x"].double()).reshape(-1)
        if case["bias"]:
            out[end:] += s["dz"].double().sum(0)
        return out
    w = s["w"][lead:end].double().view(rows, cols)
    if case["op"] == "forward":
        z = torch.matmul(s["x"].double(), w.T)
        if case["bias"]:
            z += s["w"][end:].double()
        y = _exact_act(z, case["act"])[0]
        if case["extra"]:
            y = y + s["r"].double()
        return {"y": y, "z": z} if case["keep"] else y
    d = torch.matmul(s["dz"].double(), w)
    if case["extra"]:
        d += s["a"].double()
    return d if case["act"] == "none" else {"dx": d, "dzx": d * _exact_act(s["z"].double(), case["act"])[1]}


def _exact_top(s, case):
    n, k = case["n"], case["k"]
    idx, val = torch.zeros_like(s["idx"]), torch.zeros(n, k, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, dtype=torch.float64, device="cuda")
    for at in range(0, n, 256):
        z = s["z"][at:at + 256].double()
        v, i = torch.sort(z, dim=1, descending=True, stable=True)
        val[at:at + 256], idx[at:at + 256] = v[:, :k], torch.where(v[:, :k] > -INF, i[:, :k], -1).int()
        lse[at:at + 256] = torch.logsumexp(z / case["temp"], 1)
    return {"idx": idx, "val": val, "lse": lse}


def _exact_distill(s, case):
    n, v, temp = case["n"], case["vocab"], case["temp"]
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    dz = torch.zeros(n, v, dtype=torch.float64, device="cuda")
    for at in range(0, n, 256):
        part = slice(at, at + 256)
        z, idx = s["z"][part].double(), s["idx"][part].long()
        m = z.shape[0]
        # the teacher's distribution over the whole row, and its mass on the rest
        t = torch.full((m, v + 1), -INF, dtype=torch.float64, device="cuda")
        t.scatter_(1, torch.where(idx >= 0, idx, v), s["val"][part].double() / temp)
        t = t[:, :v]
        named = t > -INF
        some = named.any(1)
        if case["tail"]:
            q = torch.exp(t - s["tlse"][part].double()[:, None])
            held = torch.where(some, torch.clamp(1 - q.sum(1), min=0), 0.0)
        else:
            q = torch.where(some[:, None], torch.softmax(t, 1), 0.0)
            held = torch.zeros(m, dtype=torch.float64, device="cuda")
        logp = torch.log_softmax(z / temp, 1)
        p = logp.exp()
        L = temp * temp * (torch.special.xlogy(q, q).sum(1) - torch.where(q > 0, q * logp, 0.0).sum(1))
        d = temp * ((q.sum(1) + held)[:, None] * p - q)
        if case["tail"]:
            rest = torch.where(named, -INF, logp)
            L += temp * temp * (torch.special.xlogy(held, held) - torch.where(held > 0, held * torch.logsumexp(rest, 1), 0.0))
            d -= temp * held[:, None] * torch.softmax(rest, 1)
        if case["ce"]:
            label = s["labels"][part].long()
            good = label >= 0
            one = torch.nn.functional.one_hot(torch.where(good, label, 0), v).double()
            log1 = torch.log_softmax(z, 1)
            L += torch.where(good, -case["ce"] * torch.where(one > 0, log1, 0.0).sum(1), 0.0)
            d += torch.where(good, case["ce"], 0.0)[:, None] * (log1.exp() - one)
        w = s["weights"][part].double()
        loss[part], dz[part] = w * L, (w * _grad_scale(case))[:, None] * d
    return {"loss": loss, "dz": dz}


def exact(case, seed):
    s = prepare(case, seed)
    return {"top": _exact_top, "distill": _exact_distill}.get(case["op"], _exact_layer)(s, case)
