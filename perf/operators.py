"""Measured cases of the training operators that stand around the compression
path: the scaled embedding lookup, its gradient by sorted tokens (dense, added,
or as a sparse message for the exchange), and the orthogonalised momentum
update of weight matrices by Newton-Schulz products.

A case is one call.  run() computes it with elementary torch operations in 32
bits (own = False), or through gradient_compression_dnn_amd.binding (own =
True); exact() gives the same outputs from the definitions in 64 bits.

Embedding: y_i = scale * w[t_i], and g[r] = scale * sum over the positions i
with t_i = r, of dy_i.  A token outside [0, rows) is padding: its row of y is
zero and its row of dy counts for nothing.
Update of a matrix: U <- m U + G, D = m U + G (Nesterov) or U, X_0 = D /
(||D||_F + eps), `steps` times X <- a X + (b A + c A^2) X with A = X X^T on
the matrix or its transpose, whichever has fewer rows, and
W <- (1 - lr wd) W - lr s O, O = X, s = sqrt(max(1, rows / cols)).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i32": torch.int32, "i64": torch.int64}
COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
MOMENTUM, LR, DECAY = 0.95, 0.02, 0.01


# --------------------------------------------------------------------- cases
def _resnet50():
    """Every convolution and the classifier of ResNet-50 as rows x cols, equal
    shapes next to each other."""
    count = {"64x147": 1, "1000x2048": 1}
    inp = 64
    for w, blocks in ((64, 3), (128, 4), (256, 6), (512, 3)):
        for b in range(blocks):
            shapes = [(w, inp), (w, 9 * w), (4 * w, w)] + ([(4 * w, inp)] if b == 0 else [])
            for r, c in shapes:
                count["%dx%d" % (r, c)] = count.get("%dx%d" % (r, c), 0) + 1
            inp = 4 * w
    return ",".join("%s*%d" % kv for kv in count.items())


def listed():
    lookup = dict(op="lookup", rows=10000, cols=1500, tokens=700, type="f32", ids="i64", scale=1.0, pad=0.0, lead=0)
    grad = dict(lookup, op="grad", out="dense")
    update = dict(op="muon", shapes="", steps=5, nesterov=True)
    return [
        # one step of a batch of 20 sequences in the LSTM language model
        dict(lookup, name="lookup step", tokens=20),
        # its training batch: 20 sequences of 35 tokens, rows scaled by sqrt(cols)
        dict(lookup, name="lookup lstm batch", ids="i32", scale=math.sqrt(1500.0)),
        # a long padded batch over a large vocabulary, half precision activations
        dict(lookup, name="lookup large", rows=131071, cols=4096, tokens=32768, type="bf16", scale=64.0, pad=0.1),
        # the gradient of 20 tokens, sent as a message
        dict(grad, name="grad step message", tokens=20, out="message"),
        # the LSTM batch's gradient, written over the embedding's whole segment
        dict(grad, name="grad lstm dense", scale=math.sqrt(1500.0)),
        # many sequences in one micro batch, added to the gradient of the earlier ones
        dict(grad, name="grad long add", tokens=32000, type="f16", ids="i32", out="add", pad=0.05),
        # odd sizes, an odd offset in the flat buffer, half precision, as a message
        dict(grad, name="grad odd message", rows=65537, cols=1023, tokens=16383, type="bf16", out="message", lead=3, pad=0.1),
        # the smallest weight matrix of the speech model
        dict(update, op="orth", name="orth speech fc", shapes="29x1600*1", nesterov=False),
        # every matrix of ResNet-50 in one step
        dict(update, name="update resnet50", shapes=_resnet50()),
        # the four recurrent matrices of the LSTM language model
        dict(update, name="update lstm", shapes="6000x1500*4"),
        # the GRU matrices of the speech model, plain momentum
        dict(update, name="update speech gru", shapes="2400x8640*2,2400x1600*12,2400x800*14", nesterov=False),
        # one large square matrix
        dict(update, op="orth", name="orth square", shapes="4096x4096*1", nesterov=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _shapes(case):
    """[(rows, cols, count)] of a case's matrices."""
    return [(int(r), int(c), int(n)) for r, c, n in (s.replace("*", "x").split("x") for s in case["shapes"].split(","))]


def draw(rng):
    op = rng.choice(("lookup", "grad", "grad", "orth", "muon"))
    if op in ("lookup", "grad"):
        rows, cols = _log_int(rng, 500, 131072), _log_int(rng, 48, 4096)
        tokens = _log_int(rng, 1, 32768)
        case = dict(op=op, rows=rows, cols=cols, tokens=tokens, type=rng.choice(("f32", "bf16", "f16")),
                    ids=rng.choice(("i32", "i64")), scale=rng.choice((1.0, math.sqrt(cols))),
                    pad=rng.choice((0.0, 0.0, 0.1, 0.5)), lead=rng.choice((0, 0, 1, 4)))
        if op == "grad":
            case["out"] = rng.choice(("dense", "add", "message"))
        return case
    groups, flops = [], 0.0
    for _ in range(rng.randint(1, 3)):
        r, c, n = _log_int(rng, 16, 6000), _log_int(rng, 16, 6000), rng.randint(1, 8)
        m, k = min(r, c), max(r, c)
        while n > 1 and flops + n * (3.0 * m * m * k + m ** 3) > 3e11:
            n -= 1
        if groups and flops + n * (3.0 * m * m * k + m ** 3) > 4e11:
            break
        flops += n * (3.0 * m * m * k + m ** 3)
        groups.append("%dx%d*%d" % (r, c, n))
    return dict(op=op, shapes=",".join(groups), steps=rng.choice((3, 5, 5, 6)) if flops < 3e11 else 5, nesterov=op == "muon" and rng.random() < 0.5)


# --------------------------------------------------------------------- inputs
def _table(lengths):
    """Rows (offset, length, bin_len, k) of a segment table without gaps."""
    at = np.cumsum([0] + lengths)
    return np.array([(int(o), n, 64, max(1, n // 1000)) for o, n in zip(at, lengths)], dtype=np.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f32 = dict(dtype=torch.float32, device="cuda")
    s = {"case": case}
    if case["op"] in ("lookup", "grad"):
        rows, cols, n, lead = case["rows"], case["cols"], case["tokens"], case["lead"]
        # ids in order of frequency, the k-th about as likely as 1 / k
        u = torch.rand(n, generator=g, dtype=torch.float64, device="cuda")
        ids = torch.clamp(torch.exp(u * math.log(rows + 1.0)).long() - 1, 0, rows - 1)
        ids[n - int(case["pad"] * n):] = -1
        s["tokens"] = ids.to(TYPES[case["ids"]])
        total = lead + rows * cols
        if case["op"] == "lookup":
            s["w"] = torch.randn(total, generator=g, **f32) / math.sqrt(cols)
            s["y"] = torch.zeros(n, cols, dtype=TYPES[case["type"]], device="cuda")
        else:
            s["dy"] = (torch.randn(n, cols, generator=g, **f32) * 1e-2).to(TYPES[case["type"]])
            if case["out"] == "message":
                cap = min(n, rows) * cols
                s["idx"] = torch.zeros(cap, dtype=torch.int32, device="cuda")
                s["val"] = torch.zeros(cap, **f32)
                s["seg_off"] = torch.zeros((2 if lead else 1) + 1, dtype=torch.int32, device="cuda")
            else:
                s["g"] = torch.randn(total, generator=g, **f32) * 1e-2
        if own:
            from gradient_compression_dnn_amd import binding as B
            s["seg"] = 1 if lead else 0
            s["plan"] = B.Plan(_table([lead, rows * cols] if lead else [rows * cols]), total)
            if case["op"] == "grad":
                s["ws"] = torch.empty(B.gc_embed_workspace_bytes(s["plan"], s["seg"], rows, n), dtype=torch.uint8, device="cuda")
                if case["out"] == "message":
                    s["out"] = B.Sparse(s["idx"], s["val"], s["seg_off"], torch.zeros(2, **f32), s["idx"].numel())
        return s
    # gradients of trained layers: a few strong directions over noise
    shapes = _shapes(case)
    total = sum(r * c * n for r, c, n in shapes)
    s["G"] = torch.randn(total, generator=g, **f32) * 1e-3
    at = 0
    for r, c, n in shapes:
        k = min(r, c, 16)
        left = torch.randn(n, r, k, generator=g, **f32) * torch.exp(-0.3 * torch.arange(k, **f32))
        s["G"][at:at + n * r * c].view(n, r, c).add_(torch.bmm(left, torch.randn(n, k, c, generator=g, **f32)), alpha=2e-3)
        at += n * r * c
    if case["op"] == "orth":
        s["O"] = torch.zeros(total, **f32)
    else:
        s["U"] = torch.randn(total, generator=g, **f32) * 2e-3
        s["W"] = torch.randn(total, generator=g, **f32) * 2e-2
    if own:
        from gradient_compression_dnn_amd import binding as B
        each = [(r, c) for r, c, n in shapes for _ in range(n)]
        s["plan"] = B.Plan(_table([r * c for r, c in each]), total)
        s["mplan"] = B.MatrixPlan(s["plan"], [r for r, _ in each])
        s["ws"] = s["mplan"].workspace("cuda")
        orth = dict(steps=case["steps"], coef=COEF, eps=EPS)
        s["opt"] = (B.orth_options(**orth) if case["op"] == "orth" else
                    B.muon_options(MOMENTUM, LR, weight_decay=DECAY, nesterov=case["nesterov"], scale=B.GC_MUON_SCALE_SHAPE, **orth))
    return s


# ------------------------------------------------------------------ plain form
def _plain_lookup(s, case):
    rows, cols = case["rows"], case["cols"]
    t = s["tokens"].long()
    ok = (t >= 0) & (t < rows)
    w = s["w"][case["lead"]:].view(rows, cols)
    s["y"].copy_(w[torch.where(ok, t, 0)] * case["scale"] * ok[:, None])
    return s["y"]


def _plain_grad(s, case):
    rows, cols, lead, n = case["rows"], case["cols"], case["lead"], case["tokens"]
    t = s["tokens"].long()
    ok = (t >= 0) & (t < rows)
    dy = s["dy"].float() * (case["scale"] * ok[:, None])
    if case["out"] != "message":
        g = s["g"][lead:].view(rows, cols)
        if case["out"] == "dense":
            g.zero_().index_add_(0, torch.where(ok, t, 0), dy)
        else:
            g.add_(torch.zeros_like(g).index_add_(0, torch.where(ok, t, 0), dy))
        return s["g"]
    # the distinct rows in ascending order: rank of each position's token among them
    held = torch.zeros(rows + 1, dtype=torch.int64, device=t.device).index_fill_(0, torch.where(ok, t, rows), 1)
    held[rows] = 0
    rank = torch.cumsum(held, 0) - held
    most = min(n, rows)
    vals = torch.zeros(most, cols, device=t.device).index_add_(0, torch.where(ok, rank[torch.where(ok, t, 0)], 0), dy)
    row_of = torch.zeros(rows + 1, dtype=torch.int64, device=t.device)
    row_of.scatter_(0, torch.where(held > 0, rank, rows), torch.arange(rows + 1, device=t.device))
    count = held.sum()
    there = (torch.arange(most, device=t.device) < count)[:, None]
    idx = lead + row_of[:most, None] * cols + torch.arange(cols, device=t.device)
    s["idx"].copy_((idx * there).reshape(-1))
    s["val"].copy_(vals.reshape(-1))
    s["seg_off"][-1] = count * cols
    return {"idx": s["idx"], "val": s["val"], "seg_off": s["seg_off"]}


def _plain_orth(D, shapes, steps):
    """The orthogonalised matrices of a flat buffer, equal shapes in one batch."""
    a, b, c = COEF
    O, at = torch.empty_like(D), 0
    for r, k, n in shapes:
        X = D[at:at + n * r * k].view(n, r, k)
        X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + EPS)
        X = X.transpose(1, 2).contiguous() if r > k else X
        for _ in range(steps):
            A = torch.bmm(X, X.transpose(1, 2))
            X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
        O[at:at + n * r * k].view(n, r, k).copy_(X.transpose(1, 2) if r > k else X)
        at += n * r * k
    return O


def _plain_update(s, case):
    shapes = _shapes(case)
    if case["op"] == "orth":
        s["O"].copy_(_plain_orth(s["G"], shapes, case["steps"]))
        return s["O"]
    s["U"].mul_(MOMENTUM).add_(s["G"])
    O = _plain_orth(MOMENTUM * s["U"] + s["G"] if case["nesterov"] else s["U"], shapes, case["steps"])
    s["W"].mul_(1.0 - LR * DECAY)
    at = 0
    for r, k, n in shapes:
        s["W"][at:at + n * r * k].sub_(O[at:at + n * r * k], alpha=LR * math.sqrt(max(1.0, r / k)))
        at += n * r * k
    return {"W": s["W"], "U": s["U"]}


def run(s):
    case = s["case"]
    if not own:
        return {"lookup": _plain_lookup, "grad": _plain_grad, "orth": _plain_update, "muon": _plain_update}[case["op"]](s, case)
    from gradient_compression_dnn_amd import binding as B
    if case["op"] == "lookup":
        B.gc_embed_lookup(s["plan"], s["seg"], case["rows"], s["w"], s["tokens"], case["scale"], s["y"])
        return s["y"]
    if case["op"] == "grad":
        if case["out"] == "message":
            B.gc_embed_message(s["plan"], s["seg"], case["rows"], s["dy"], s["tokens"], case["scale"], s["out"], s["ws"])
            return {"idx": s["idx"], "val": s["val"], "seg_off": s["seg_off"]}
        B.gc_embed_grad(s["plan"], s["seg"], case["rows"], s["dy"], s["tokens"], case["scale"], s["g"], case["out"] == "add", s["ws"])
        return s["g"]
    if case["op"] == "orth":
        B.gc_orthogonalize(s["mplan"], s["G"], s["O"], s["opt"], s["ws"])
        return s["O"]
    B.gc_muon_step(s["mplan"], s["G"], s["U"], s["W"], s["opt"], s["ws"])
    return {"W": s["W"], "U": s["U"]}


# ------------------------------------------------------------------------ work
def work(case):
    if case["op"] in ("lookup", "grad"):
        rows, cols, n = case["rows"], case["cols"], case["tokens"]
        live = n - int(case["pad"] * n)
        # rows that a batch is expected to hold, under prepare()'s law of the ids
        k = np.arange(1, rows + 1, dtype=np.float64)
        distinct = float(np.sum(-np.expm1(live * np.log1p(-np.log1p(1.0 / k) / math.log(rows + 1.0)))))
        size, ids = TYPES[case["type"]].itemsize, TYPES[case["ids"]].itemsize * n
        if case["op"] == "lookup":
            return {"bytes": ids + 4.0 * distinct * cols + size * n * cols, "flops": float(live * cols)}
        wrote = {"dense": 4.0 * rows, "add": 8.0 * distinct, "message": 8.0 * distinct}[case["out"]]
        return {"bytes": ids + size * live * cols + wrote * cols, "flops": 2.0 * live * cols}
    total = flops = 0.0
    for r, c, n in _shapes(case):
        m, k = min(r, c), max(r, c)
        total += n * r * c
        # A and A^2 are symmetric: half of each is enough
        flops += n * case["steps"] * (3.0 * m * m * k + m ** 3)
    return {"bytes": total * (8.0 if case["op"] == "orth" else 20.0), "flops": flops}


# ----------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    f64 = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "lookup":
        y = torch.zeros(case["tokens"], case["cols"], **f64)
        at = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["rows"])).reshape(-1)
        w = s["w"][case["lead"]:].view(case["rows"], case["cols"])
        for part in at.split(8192):
            y[part] = w.index_select(0, s["tokens"][part].long()).double() * case["scale"]
        return y
    if case["op"] == "grad":
        rows, cols, lead = case["rows"], case["cols"], case["lead"]
        live = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < rows)).reshape(-1)
        t, order = torch.sort(s["tokens"][live].long(), stable=True)
        ids, counts = torch.unique_consecutive(t, return_counts=True)
        # sums of the runs as differences of running sums, a block of columns at a time
        sums = torch.empty(ids.numel(), cols, **f64)
        ends = torch.cumsum(counts, 0) - 1
        for c in range(0, cols, 256):
            run_to = torch.cumsum(s["dy"][live[order], c:c + 256].double(), 0)[ends]
            sums[:, c:c + 256] = torch.cat([run_to[:1], run_to[1:] - run_to[:-1]]) * case["scale"]
        if case["out"] == "message":
            idx, val, off = torch.zeros_like(s["idx"]), torch.zeros(s["val"].numel(), **f64), torch.zeros_like(s["seg_off"])
            n = ids.numel() * cols
            idx[:n] = (lead + ids[:, None] * cols + torch.arange(cols, device="cuda")).reshape(-1).int()
            val[:n] = sums.reshape(-1)
            off[-1] = n
            return {"idx": idx, "val": val, "seg_off": off}
        g = s["g"].double()
        if case["out"] == "dense":
            g[lead:] = 0.0
        g[lead:].view(rows, cols)[ids] += sums
        return g
    G = s["G"].double()
    if case["op"] == "muon":
        U = s["U"].double() * MOMENTUM + G
        G, W = (U * MOMENTUM + G if case["nesterov"] else U), s["W"].double() * (1.0 - LR * DECAY)
    O, at = torch.empty_like(G), 0
    a, b, c = COEF
    for r, k, n in _shapes(case):
        for _ in range(n):
            # O = q(A) X with A = X X^T: q from the steps taken on A alone,
            # A <- p(A) A p(A) with p(A) = a + b A + c A^2
            X = G[at:at + r * k].view(r, k)
            X = (X if r <= k else X.T) / (torch.linalg.vector_norm(X) + EPS)
            A = X @ X.T
            I, q = torch.eye(min(r, k), **f64), None
            for _ in range(case["steps"]):
                p = a * I + A @ (b * I + c * A)
                A, q = p @ A @ p, p if q is None else p @ q
            O[at:at + r * k].view(r, k).copy_(q @ X if r <= k else (q @ X).T)
            if case["op"] == "muon":
                W[at:at + r * k] -= LR * math.sqrt(max(1.0, r / k)) * O[at:at + r * k]
            at += r * k
    return O if case["op"] == "orth" else {"W": W, "U": U}
