"""The embedding's lookup and gradient on the GPU: bit for bit against the
order of operations that the header states (NumPy, fp32), and within a bound
from the number of roundings against sums in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from gradient_compression_dnn_amd import binding as B
from gradient_compression_dnn_amd import workloads as W
from tests.gpu_util import dev, same_bits, say, ulp_report

pytestmark = pytest.mark.gpu

BLOCK, WAVES = 16, 16  # sorted positions a block, partial sums of a join
U32 = 2.0 ** -24


def ordered_sums(keys, dy, rows):
    """{row: fp32 sum} in the stated order; keys outside [0, rows) dropped."""
    live = np.nonzero((keys >= 0) & (keys < rows))[0]
    order = live[np.argsort(keys[live], kind="stable")]
    k = keys[order]
    out, q = {}, 0
    while q < len(k):
        e = q
        while e < len(k) and k[e] == k[q]:
            e += 1
        parts = []
        for b in range(q // BLOCK, (e - 1) // BLOCK + 1):
            acc = np.zeros(dy.shape[1], np.float32)
            for i in order[max(q, b * BLOCK):min(e, (b + 1) * BLOCK)]:
                acc = acc + dy[i]
            parts.append(acc)
        if len(parts) == 1:
            out[int(k[q])] = parts[0]
        else:
            zs = []
            for w in range(min(WAVES, len(parts))):
                z = np.zeros(dy.shape[1], np.float32)
                for p in parts[w::WAVES]:
                    z = z + p
                zs.append(z)
            tot = zs[0]
            for z in zs[1:]:
                tot = tot + z
            out[int(k[q])] = tot
        q = e
    return out


def f32(a):
    return a.detach().float().cpu().numpy()


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Batch:
    """An embedding of rows x cols behind `lead` elements (and in front of 5),
    and a batch of tokens."""

    def __init__(self, rows, cols, n, dtype, ids=torch.int64, lead=3, kind="mixed", seed=0):
        rng = np.random.default_rng(seed + rows * 31 + cols * 7 + n)
        self.rows, self.cols, self.n, self.lead = rows, cols, n, lead
        lens = ([lead] if lead else []) + [rows * cols, 5]
        self.plan = B.Plan(W.make_table(lens, [1] * len(lens)))
        self.seg = 1 if lead else 0
        if kind == "one":
            k = np.full(n, rows // 2)
        elif kind == "pad":
            k = np.full(n, -1)
        elif kind == "distinct":
            k = rng.permutation(rows)[:n] if n <= rows else rng.integers(0, rows, n)
        else:  # frequent small ids, and padding of every kind
            k = np.minimum((np.exp(rng.random(n) * np.log(rows + 1)) - 1).astype(np.int64), rows - 1)
            bad = [-1, rows, rows + 7, -(1 << 31), (1 << 31) - 1]
            if ids == torch.int64:
                bad += [1 << 32, -(1 << 62)]  # ids whose low word is a valid row
            at = rng.random(n) < 0.1
            k[at] = rng.choice(bad, at.sum())
        self.keys = k.astype(np.int64)
        self.tokens = torch.from_numpy(self.keys).to(dev()).to(ids)
        self.dy = torch.from_numpy(rng.normal(0, 1e-2, (n, cols)).astype(np.float32)).to(dev()).to(DTYPES[dtype])
        # what stands in the rows of padding must not be read
        self.dy[(self.tokens < 0) | (self.tokens >= rows)] = float("nan")
        self.w = torch.from_numpy(rng.normal(0, 1, self.plan.n_total).astype(np.float32)).to(dev())

    def ws(self):
        need = B.gc_embed_workspace_bytes(self.plan, self.seg, self.rows, self.n)
        return torch.full((need,), 0xA5, dtype=torch.uint8, device=dev())

    def message(self):
        return B.Sparse.empty(self.plan, B.gc_embed_message_cap(self.plan, self.seg, self.rows, self.n), dev())


SIZES = [(1, 1, 1), (1, 1, 70), (7, 3, 1), (10, 4, 33), (50, 5, 64), (100, 255, 65), (100, 256, 31), (300, 257, 1000),
         (33, 1500, 100), (5000, 36, 4095), (5000, 31, 4096), (5000, 8, 4097), (70, 12, 9000),
         (60, 40, 255), (3000, 7, 256), (60, 513, 256), (60, 40, 257), (4000, 3, 2049),
         (900, 5, 6144), (900, 5, 6145)]


@pytest.mark.parametrize("rows,cols,n", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_lookup_bits(rows, cols, n, dtype):
    for lead, ids, scale in ((0, torch.int64, 1.0), (3, torch.int32, 0.37)):
        b = Batch(rows, cols, n, dtype, ids, lead)
        say(f"lookup {rows}x{cols} n={n} {dtype} lead={lead}")
        y = torch.full((n, cols), 7.0, dtype=DTYPES[dtype], device=dev())
        B.gc_embed_lookup(b.plan, b.seg, rows, b.w, b.tokens, scale, y)
        table = b.w[lead:lead + rows * cols].view(rows, cols).cpu()
        ok = (b.keys >= 0) & (b.keys < rows)
        want = torch.zeros(n, cols)
        want[ok] = table[b.keys[ok]] * torch.tensor(scale, dtype=torch.float32)
        assert torch.equal(y.cpu(), want.to(DTYPES[dtype]))


@pytest.mark.parametrize("rows,cols,n", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradient_bits_and_bound(rows, cols, n, dtype):
    for kind, ids, lead, scale in (("mixed", torch.int64, 0, 1.0), ("one", torch.int32, 3, 0.37),
                                   ("distinct", torch.int32, 0, 3.0), ("pad", torch.int64, 3, 1.0)):
        b = Batch(rows, cols, n, dtype, ids, lead, kind)
        dy = f32(b.dy)
        sums = ordered_sums(b.keys, dy, rows)
        s32 = np.float32(scale)
        held = sorted(sums)
        base = f32(b.w)
        lo, hi = lead, lead + rows * cols
        for acc in (False, True):
            say(f"grad {rows}x{cols} n={n} {dtype} {kind} add={acc}")
            g = b.w.clone()
            B.gc_embed_grad(b.plan, b.seg, rows, b.dy, b.tokens, scale, g, acc, b.ws())
            want = base.copy()
            seg = want[lo:hi].reshape(rows, cols)
            if not acc:
                seg[:] = 0.0
            for r in held:
                v = s32 * sums[r]
                seg[r] = seg[r] + v if acc else v
            got = f32(g)
            assert same_bits(got, want), ulp_report(got, want)
        # against 64 bits: at most m + 16 additions of a row, a product and,
        # above, one sum, each off by U32 of what it adds up
        d64 = dy.astype(np.float64)
        for r in held[:50]:
            rows_of = d64[b.keys == r]
            tol = (len(rows_of) + 18) * U32 * float(s32) * np.abs(rows_of).sum(0)
            assert (np.abs(float(s32) * rows_of.sum(0) - (s32 * sums[r]).astype(np.float64)) <= tol).all()
        say(f"message {rows}x{cols} n={n} {dtype} {kind}")
        msg = b.message()
        msg.idx.fill_(-3)
        msg.val.fill_(-3.0)
        msg.seg_off.fill_(-3)
        B.gc_embed_message(b.plan, b.seg, rows, b.dy, b.tokens, scale, msg, b.ws())
        idx, val, off, _ = msg.host()
        assert list(off) == [0] * (b.seg + 1) + [len(held) * cols] * (b.plan.nseg - b.seg)
        widx = np.concatenate([lo + r * cols + np.arange(cols) for r in held]) if held else np.zeros(0)
        wval = np.concatenate([s32 * sums[r] for r in held]) if held else np.zeros(0, np.float32)
        assert np.array_equal(idx, widx.astype(np.uint32)) and same_bits(val, wval), ulp_report(val, wval)
        assert bool((msg.idx[len(widx):] == -3).all()) and bool((msg.val[len(widx):] == -3.0).all())


@pytest.mark.parametrize("n", [4096 * 8 + 1, 70_001])
def test_gradient_of_long_batches(n):
    # more than 8 ranked tiles: two rounds of merging; integers, so that every
    # order of the sums gives the same bits
    rows, cols = 300, 5
    b = Batch(rows, cols, n, "f32", torch.int32, 0)
    b.dy = torch.randint(-8, 9, (n, cols), device=dev()).float()
    ok = (b.keys >= 0) & (b.keys < rows)
    want = np.zeros((rows, cols))
    np.add.at(want, b.keys[ok], f32(b.dy)[ok])
    say(f"grad long n={n}")
    g = b.w.clone()
    B.gc_embed_grad(b.plan, b.seg, rows, b.dy, b.tokens, 1.0, g, False, b.ws())
    assert np.array_equal(f32(g)[:rows * cols].reshape(rows, cols), want)
    msg = b.message()
    B.gc_embed_message(b.plan, b.seg, rows, b.dy, b.tokens, 1.0, msg, b.ws())
    idx, val, off, _ = msg.host()
    held = np.unique(b.keys[ok])
    assert off[-1] == len(held) * cols and np.array_equal(val.reshape(-1, cols), want[held])
    assert np.array_equal(idx.reshape(-1, cols)[:, 0], held * cols)


def test_gradient_is_the_lookups():
    """<dy, lookup(w + h) - lookup(w)> = <g, h>, exactly: whole numbers."""
    rows, cols, n = 40, 37, 300
    b = Batch(rows, cols, n, "f32")
    ok = (b.tokens >= 0) & (b.tokens < rows)
    gen = torch.Generator(device=dev()).manual_seed(5)
    w, h = (torch.randint(-4, 5, (b.plan.n_total,), generator=gen, device=dev()).float() for _ in range(2))
    dy = torch.randint(-4, 5, (n, cols), generator=gen, device=dev()).float()
    y0, y1 = torch.empty(n, cols, device=dev()), torch.empty(n, cols, device=dev())
    B.gc_embed_lookup(b.plan, b.seg, rows, w, b.tokens, 2.0, y0)
    B.gc_embed_lookup(b.plan, b.seg, rows, w + h, b.tokens, 2.0, y1)
    assert not y0[~ok].any()
    g = torch.zeros_like(w)
    B.gc_embed_grad(b.plan, b.seg, rows, dy, b.tokens, 2.0, g, False, b.ws())
    assert (dy.double() * (y1 - y0).double()).sum().item() == (g.double() * h.double()).sum().item()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strided_rows_and_token_shapes(dtype):
    rows, cols = 60, 21
    b = Batch(rows, cols, 24, dtype, torch.int32)
    tokens = b.tokens.view(4, 6)
    wide = torch.full((4, 6, cols + 10), 9.0, dtype=DTYPES[dtype], device=dev())
    y = wide[..., 3:3 + cols]
    say("strided lookup")
    B.gc_embed_lookup(b.plan, b.seg, rows, b.w, tokens, 1.0, y)
    flat = torch.empty(24, cols, dtype=DTYPES[dtype], device=dev())
    B.gc_embed_lookup(b.plan, b.seg, rows, b.w, b.tokens, 1.0, flat)
    assert torch.equal(y.reshape(24, cols), flat)
    assert bool((wide[..., :3] == 9).all()) and bool((wide[..., 3 + cols:] == 9).all())
    y.copy_(b.dy.view(4, 6, cols))
    g, h = b.w.clone(), b.w.clone()
    B.gc_embed_grad(b.plan, b.seg, rows, y, tokens, 1.5, g, True, b.ws())
    B.gc_embed_grad(b.plan, b.seg, rows, b.dy, b.tokens, 1.5, h, True, b.ws())
    assert torch.equal(g, h)
    for bad in (wide[..., :cols].transpose(0, 1), wide[:, :5, :cols], y.double(), y.expand(2, 4, 6, cols),
                torch.zeros(1, 1, cols, dtype=y.dtype, device=dev()).expand(4, 6, cols), wide[..., 0:2 * cols:2]):
        with pytest.raises(ValueError):
            B.gc_embed_grad(b.plan, b.seg, rows, bad, tokens, 1.0, g, True, b.ws())
    assert torch.equal(g, h)


def test_special_values():
    rows, cols, n = 9, 6, 40
    b = Batch(rows, cols, n, "f32", kind="distinct")
    b.dy[:] = 1.0
    inf = float("inf")
    b.dy[0, 0], b.dy[1, 1], b.dy[2, 2] = inf, -inf, float("nan")
    g = b.w.clone()
    B.gc_embed_grad(b.plan, b.seg, rows, b.dy, b.tokens, 1.0, g, False, b.ws())
    got = f32(g)[b.lead:b.lead + rows * cols].reshape(rows, cols)
    sums = ordered_sums(b.keys, f32(b.dy), rows)
    want = np.zeros((rows, cols), np.float32)
    for r, s in sums.items():
        want[r] = s
    assert np.array_equal(got, want, equal_nan=True)
    # values past fp16's range become Inf, as torch's own cast makes them
    w = torch.full_like(b.w, 70000.0)
    y = torch.empty(n, cols, dtype=torch.float16, device=dev())
    B.gc_embed_lookup(b.plan, b.seg, rows, w, b.tokens, 1.0, y)
    ok = (b.keys >= 0) & (b.keys < rows)
    assert bool((y[torch.from_numpy(ok).to(dev())] == inf).all())


def test_empty_batch():
    b = Batch(11, 5, 1, "f32")
    none = torch.zeros(0, dtype=torch.int64, device=dev())
    empty = torch.zeros(0, 5, device=dev())
    ws = torch.zeros(1, dtype=torch.uint8, device=dev())
    B.gc_embed_lookup(b.plan, b.seg, 11, b.w, none, 1.0, empty)
    g = b.w.clone()
    B.gc_embed_grad(b.plan, b.seg, 11, empty, none, 1.0, g, True, ws)
    assert torch.equal(g, b.w)
    B.gc_embed_grad(b.plan, b.seg, 11, empty, none, 1.0, g, False, ws)
    assert not g[3:58].any() and torch.equal(g[:3], b.w[:3]) and torch.equal(g[58:], b.w[58:])
    msg = B.Sparse.empty(b.plan, 0, dev())
    msg.seg_off.fill_(9)
    B.gc_embed_message(b.plan, b.seg, 11, empty, none, 1.0, msg, ws)
    assert not msg.seg_off.any()


def test_messages_of_four_learners_travel():
    """The embedding messages of four learners packed, unpacked and averaged
    equal the decode of the oracle on the same entries."""
    rows, cols = 500, 31
    table = W.make_table([9, rows * cols, 100], [1, 1, 1], [9, rows * cols, 100])
    msgs, host = [], []
    plan = None
    for j in range(4):
        b = Batch(rows, cols, 150 + 40 * j, "bf16", seed=j)
        plan = B.Plan(table)
        msg = B.Sparse.empty(plan, B.gc_embed_message_cap(plan, 1, rows, b.n), dev())
        ws = torch.empty(B.gc_embed_workspace_bytes(plan, 1, rows, b.n), dtype=torch.uint8, device=dev())
        B.gc_embed_message(plan, 1, rows, b.dy, b.tokens, 2.0, msg, ws)
        opt = B.dgc_options(0.0, density=(1, 1))
        buf = torch.zeros(B.gc_dgc_pack_bound(plan, opt), dtype=torch.uint8, device=dev())
        size = torch.zeros(1, dtype=torch.int64, device=dev())
        B.gc_pack(plan, B.GC_KIND_DGC, msg, buf, size, plan.workspace(B.GC_OP_PACK, dev()))
        back, status = B.Sparse.empty(plan, msg.cap, dev()), torch.full((1,), 7, dtype=torch.int32, device=dev())
        B.gc_unpack(plan, B.GC_KIND_DGC, buf, int(size.item()), back, status, plan.workspace(B.GC_OP_UNPACK, dev()))
        assert int(status.item()) == 0
        a, c = msg.host(), back.host()
        assert np.array_equal(a[0], c[0]) and same_bits(a[1], c[1]) and np.array_equal(a[2], c[2])
        msgs.append(back)
        host.append((a[0], a[1]))
    dense = torch.ones(plan.n_total, device=dev())
    B.gc_decompress_accumulate(plan, msgs, dense, B.GC_AVG, False, plan.workspace(B.GC_OP_DECODE, dev()))
    want = oracle.decode(table, plan.n_total, host, mode=B.GC_AVG)
    assert same_bits(f32(dense), want), ulp_report(f32(dense), want)


def test_graph_replays_with_new_tokens():
    rows, cols, n = 300, 20, 5000
    bs = [Batch(rows, cols, n, "f16", torch.int32, 3, k, seed=s) for s, k in enumerate(("mixed", "one", "pad", "mixed"))]
    b = bs[0]
    tok, dy = b.tokens.clone(), b.dy.clone()
    g, add, msg = torch.zeros_like(b.w), torch.zeros_like(b.w), b.message()
    y = torch.zeros(n, cols, device=dev())
    ws = b.ws()

    def call(tokens, grads, y, g, add, msg, ws):
        B.gc_embed_lookup(b.plan, b.seg, rows, b.w, tokens, 0.5, y)
        B.gc_embed_grad(b.plan, b.seg, rows, grads, tokens, 0.5, g, False, ws)
        B.gc_embed_grad(b.plan, b.seg, rows, grads, tokens, 0.5, add, True, ws)
        B.gc_embed_message(b.plan, b.seg, rows, grads, tokens, 0.5, msg, ws)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    say("embed graph capture")
    with torch.cuda.graph(graph):
        call(tok, dy, y, g, add, msg, ws)
    add2 = torch.zeros_like(b.w)
    add.zero_()
    for x in bs:
        say("embed graph replay")
        tok.copy_(x.tokens)
        dy.copy_(x.dy)
        graph.replay()
        torch.cuda.synchronize()
        y2, g2, msg2 = torch.zeros_like(y), torch.zeros_like(g), b.message()
        call(x.tokens, x.dy, y2, g2, add2, msg2, b.ws())
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(g, g2) and torch.equal(add, add2)
        for p, q in zip(msg.host()[:3], msg2.host()[:3]):
            assert np.array_equal(p, q)


def test_two_streams():
    bs = [Batch(200, 64, 3000, "f32", seed=s) for s in (1, 2)]
    alone = []
    for b in bs:
        g = torch.zeros_like(b.w)
        B.gc_embed_grad(b.plan, b.seg, 200, b.dy, b.tokens, 1.0, g, False, b.ws())
        alone.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    outs, spaces = [torch.zeros_like(b.w) for b in bs], [b.ws() for b in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s, g, ws in zip(bs, streams, outs, spaces):
            with torch.cuda.stream(s):
                B.gc_embed_grad(b.plan, b.seg, 200, b.dy, b.tokens, 1.0, g, False, ws)
    torch.cuda.synchronize()
    for a, g in zip(alone, outs):
        assert torch.equal(a, g)


def test_a_table_past_two_gigabytes():
    # byte offsets past 2^31 and element offsets past 2^29 in both directions
    rows, cols = 140_000, 4100
    plan = B.Plan(W.make_table([rows * cols], [4096], [1]))
    w = torch.empty(plan.n_total, device=dev())
    v = w.view(rows, cols)
    v.copy_(torch.arange(rows, device=dev())[:, None].expand(rows, cols))
    tokens = torch.tensor([rows - 1, 0, 131_072, rows - 1, -1, 130_944], device=dev())
    y = torch.empty(6, cols, device=dev())
    say("lookup in a large table")
    B.gc_embed_lookup(plan, 0, rows, w, tokens, 1.0, y)
    want = torch.where((tokens >= 0) & (tokens < rows), tokens, 0).float()
    assert bool((y == want[:, None]).all())
    ws = torch.empty(B.gc_embed_workspace_bytes(plan, 0, rows, 6), dtype=torch.uint8, device=dev())
    say("gradient of a large table")
    B.gc_embed_grad(plan, 0, rows, torch.ones_like(y), tokens, 1.0, w, False, ws)
    assert bool((v.sum(1)[[0, 131_072, 130_944, rows - 1]] == torch.tensor([1, 1, 1, 2], device=dev()) * cols).all())
    assert v.sum(dtype=torch.float64).item() == 5 * cols


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [-1.0, -0.37, -0.0, 0.0, 0.37])
def test_lookup_bits_of_padding(dtype, scale):
    """Padding's row is +0 whatever the scale's sign, and a row of zeros has
    the sign of the product: compared bit by bit."""
    bits = {torch.float32: torch.int32, torch.bfloat16: torch.int16, torch.float16: torch.int16}[DTYPES[dtype]]
    for rows, cols, n in ((1, 1, 3), (40, 33, 70), (90, 512, 300)):
        b = Batch(rows, cols, n, dtype)
        b.w[b.lead] = 0.0
        b.tokens[0], b.tokens[n - 1] = 0, rows
        ok = (b.tokens >= 0) & (b.tokens < rows)
        y = torch.full((n, cols), 7.0, dtype=DTYPES[dtype], device=dev())
        say(f"lookup {rows}x{cols} n={n} {dtype} scale={scale}")
        B.gc_embed_lookup(b.plan, b.seg, rows, b.w, b.tokens, scale, y)
        table = b.w[b.lead:b.lead + rows * cols].view(rows, cols).cpu()
        want = torch.zeros(n, cols)
        want[ok.cpu()] = table[b.tokens[ok].cpu()] * torch.tensor(scale, dtype=torch.float32)
        assert torch.equal(y.cpu().view(bits), want.to(DTYPES[dtype]).view(bits))
        assert not y[~ok].view(bits).any()


def banded_tokens(rows, n, rng):
    """Tiles of 2,048 tokens that are alternately spread over all rows and
    packed into a narrow band, so that between two neighbours of a spread run
    stand hundreds of a packed one's tokens, and a twentieth padding."""
    tile = np.arange(n) // 2048
    spread = rng.integers(0, rows, n)
    band = (tile * 37) % rows + rng.integers(0, max(1, rows // 64), n)
    keys = np.where(tile % 2 == 0, spread, band % rows)
    keys[rng.random(n) < 0.05] = -1
    return keys


# two rounds of merging: at one token more than a round's 16 tiles, at odd
# lengths, and with all 16 runs of the second round; then three rounds
@pytest.mark.parametrize("n", [32_768, 32_769, 70_001, 16 * 32_768, 16 * 32_768 + 4_097])
@pytest.mark.parametrize("rows", [64, 5000])
def test_gradient_order_of_long_batches(rows, n):
    """The order of every sum after more than one round of merging, by the bits
    of sums whose order matters."""
    cols = 3
    rng = np.random.default_rng(n + rows)
    keys = banded_tokens(rows, n, rng)
    plan = B.Plan(W.make_table([rows * cols], [1]))
    dy = (rng.normal(size=(n, cols)) * np.exp(2 * rng.normal(size=(n, 1)))).astype(np.float32)
    sums = ordered_sums(keys, dy, rows)
    backwards = ordered_sums(keys[::-1], dy[::-1], rows)
    assert any((sums[r] != backwards[r]).any() for r in sums)  # the order shows in the bits
    want = np.zeros((rows, cols), np.float32)
    for r, v in sums.items():
        want[r] = np.float32(0.5) * v
    tokens, d = torch.from_numpy(keys).to(dev()), torch.from_numpy(dy).to(dev())
    ws = torch.full((B.gc_embed_workspace_bytes(plan, 0, rows, n),), 0xA5, dtype=torch.uint8, device=dev())
    say(f"order of {n} tokens in {rows} rows")
    g = torch.full((rows * cols,), 7.0, device=dev())
    B.gc_embed_grad(plan, 0, rows, d, tokens, 0.5, g, False, ws)
    got = f32(g)
    assert same_bits(got, want.reshape(-1)), ulp_report(got, want.reshape(-1))
    msg = B.Sparse.empty(plan, B.gc_embed_message_cap(plan, 0, rows, n), dev())
    B.gc_embed_message(plan, 0, rows, d, tokens, 0.5, msg, ws)
    idx, val, off, _ = msg.host()
    held = sorted(sums)
    assert off[1] == len(held) * cols and np.array_equal(idx.reshape(-1, cols)[:, 0], np.array(held) * cols)
    assert same_bits(val, want[held].reshape(-1)), ulp_report(val, want[held].reshape(-1))
