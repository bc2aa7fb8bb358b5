"""The operators that verify a drafted tree, against float64 references: page tables and
slots, tree attention over the paged cache, filtered sampling, and a run of them together."""

import numpy as np
import pytest
import torch

from speculative_decoding_block_context_gb300 import _lib as F

from . import verify_ref as ref

pytestmark = pytest.mark.gpu

BITS = F.DEVERR


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_block_context_gb300 import build

    build.build()
    F.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ pages


def run_pages(req, lens, new, held, P, table, free, head, num_pages, cap, extras=True):
    bs = len(req)
    d = dict(table=i32(table), head=i32([-9]), held=i32([-9] * bs), cu=i32([-9] * (bs + 1)),
             slots=torch.full((cap,), -9, dtype=torch.int64, device="cuda"), pos=i32([-9] * cap), own=i32([-9] * cap),
             err=i32([0]))
    F.flashmap_extend_pages(i32(req), i32(lens), i32(new), None if held is None else i32(held), P, d["table"],
                            i32(free), i32([head]), d["head"], d["held"] if extras else None, num_pages, d["cu"],
                            d["slots"], d["pos"] if extras else None, d["own"] if extras else None, d["err"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}


def check_pages(req, lens, new, held, P, table, free, head, num_pages, cap):
    table = np.asarray(table, dtype=np.int32)
    got = run_pages(req, lens, new, held, P, table, free, head, num_pages, cap)
    t, h, ho, cu, slots, pos, own, served = ref.extend_pages(req, lens, new, held, P, table, free, head, num_pages, cap)
    np.testing.assert_array_equal(got["table"], t)
    np.testing.assert_array_equal(got["cu"], cu)
    np.testing.assert_array_equal(got["held"], ho)
    assert got["head"][0] == h
    n = min(cap, cu[-1])
    for key, want in (("slots", slots), ("pos", pos), ("own", own)):
        np.testing.assert_array_equal(got[key][:n], want[:n])
        assert (got[key][n:] == -9).all()  # rows behind the last token
    return got["err"][0], served


@pytest.mark.parametrize("bs,P,longest,most,seed", [
    (1, 16, 2048, 16, 0), (1, 16, 1, 1, 1), (3, 48, 100, 40, 2), (128, 16, 3000, 17, 3), (17, 7, 50, 300, 4),
    (513, 16, 200, 5, 5), (1500, 32, 90, 9, 6), (5, 64, 0, 2000, 7), (4, 1, 9, 9, 8)])
def test_pages_match(bs, P, longest, most, seed):
    g = np.random.default_rng(seed)
    lens, new = g.integers(0, longest + 1, bs), g.integers(0, most + 1, bs)
    held = -(-lens // P) + g.integers(0, 3, bs)
    rows, stride = bs + 3, -(-(longest + most) // P) + 3
    table = g.permutation(rows * stride).reshape(rows, stride)
    req = g.permutation(rows)[:bs]
    free = g.permutation(rows * stride + 5000)[: int(np.maximum(0, -(-(lens + new) // P) - held).sum()) + 3]
    err, served = check_pages(req.tolist(), lens.tolist(), new.tolist(), held.tolist(), P, table, free.tolist(), 2,
                              rows * stride + 5000, max(1, int(new.sum()) + 3))
    assert err == 0 and all(served)
    err, served = check_pages(req.tolist(), lens.tolist(), new.tolist(), None, P, table, free.tolist(), 0,
                              rows * stride + 5000, max(1, int(new.sum())))


@pytest.mark.parametrize("what,bit", [
    ("out of pages", "CAPACITY"), ("out of rows", "CAPACITY"), ("bad head", "CAPACITY"), ("same row twice", "REQUEST"),
    ("row out of range", "REQUEST"), ("held too few", "REQUEST"), ("negative length", "POSITION"),
    ("negative tokens", "POSITION"), ("past the row", "POSITION"), ("bad free page", "PAGE"), ("bad old page", "PAGE")])
def test_pages_refuse_on_the_device(what, bit):
    P, table = 16, np.arange(40).reshape(5, 8)
    req, lens, new, held = [0, 3, 1, 4], [20, 5, 33, 16], [30, 12, 0, 7], [2, 1, 3, 1]
    free, head, cap = list(range(50, 60)), 1, 60
    if what == "out of pages":
        free = free[:4]
    elif what == "out of rows":
        cap = 35
    elif what == "bad head":
        head = 11
    elif what == "same row twice":
        req[2] = req[0]
    elif what == "row out of range":
        req[1] = 5
    elif what == "held too few":
        held[0] = 1
    elif what == "negative length":
        lens[1] = -1
    elif what == "negative tokens":
        new[1] = -4
    elif what == "past the row":
        lens[0], held[0] = 100, 7
    elif what == "bad free page":
        free[2] = 70
    else:
        table[3, 0] = -1
    if what == "bad head":
        got = run_pages(req, lens, new, held, P, table, free, head, 64, cap)
        assert got["head"][0] == 11 and got["err"][0] == BITS[bit]
        assert (got["slots"][:30] == -1).all() and (got["slots"][42:49] == -1).all()
        np.testing.assert_array_equal(got["table"], table)
        return
    err, served = check_pages(req, lens, new, held, P, table, free, head, 64, cap)
    assert err == BITS[bit]


# ------------------------------------------------------------------ attention


class Case:
    def __init__(self, bs, width, heads, kv, hd, P, ctx, nodes=None, ids=False, dtype="bf16", seed=0, spread=1.5):
        g = torch.Generator().manual_seed(seed)
        self.bs, self.width, self.heads, self.P, self.hd = bs, width, heads, P, hd
        self.ctx = [int(c) for c in (ctx if isinstance(ctx, (list, tuple)) else [ctx] * bs)]
        self.nodes = nodes
        need = [-(-(c + width) // P) for c in self.ctx]
        self.stride, pages, rows = max(need), sum(need) + 3, bs + 2
        perm = torch.randperm(pages, generator=g).int()
        self.req = torch.randperm(rows, generator=g)[:bs].int()
        self.table = torch.full((rows, self.stride), -1, dtype=torch.int32)
        at = 0
        for b in range(bs):
            self.table[self.req[b], : need[b]] = perm[at:at + need[b]]
            at += need[b]
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.keys = torch.randn((pages, kv, P, hd), generator=g).to(dt)
        self.values = torch.randn((pages, kv, P, hd), generator=g).to(dt)
        self.q = (spread * torch.randn((bs * width, heads, hd), generator=g)).to(dt)
        self.scale = hd ** -0.5
        self.ids = None
        if ids and width > 1:
            i = torch.arange(1, width)
            back = torch.randint(0, 6, (bs, width - 1), generator=g)
            parent = torch.cummax((i - 1 - back).clamp(min=0), dim=1).values
            self.ids = parent * width + i
        for b in range(bs):  # what lies behind a request's last node is not read into results
            n = self.nodes[b] if self.nodes else width
            for pos in range(self.ctx[b] + max(n, 0), need[b] * P):
                page = self.table[self.req[b], pos // P]
                self.keys[page, :, pos % P] = float("nan")
                self.values[page, :, pos % P] = float("nan") if pos % 2 else float("inf")

    def run(self, fill=7.0, stride=None, stream=None):
        q = self.q.cuda()
        if stride:
            wide = torch.full((q.shape[0], stride), float("nan"), dtype=q.dtype, device="cuda")
            wide[:, : self.heads * self.hd] = q.view(q.shape[0], -1)
            q = wide[:, : self.heads * self.hd].view(-1, self.heads, self.hd)
        cache = F.make_cache_layer(self.keys.cuda(), self.values.cuda())
        ws = torch.full((F.flashmap_tree_attention_workspace(cache, self.bs, self.width, self.heads),), 255,
                        dtype=torch.uint8, device="cuda")
        out = torch.full(self.q.shape, fill, dtype=self.q.dtype, device="cuda")
        err = i32([0])
        F.flashmap_tree_attention(cache, q, self.width, i32(self.ctx), i32(self.nodes) if self.nodes else None,
                                  self.ids.cuda() if self.ids is not None else None, self.req.cuda(),
                                  self.table.cuda(), self.scale, out, ws, err, stream)
        torch.cuda.synchronize()
        return out.cpu(), int(err)

    def check(self, out, fill=7.0, requests=None):
        eps = 2.0 ** -8 if self.q.dtype == torch.bfloat16 else 0.0
        keys, values = self.keys.double().numpy(), self.values.double().numpy()
        for b in requests if requests is not None else range(self.bs):
            n = max(0, min(self.width, self.nodes[b] if self.nodes else self.width))
            got = out[b * self.width:(b + 1) * self.width].double().numpy()
            assert (got[n:] == fill).all()
            if n == 0:
                continue
            parent = ref.parents_of(self.ids[b].tolist() if self.ids is not None else None, self.width)
            q = self.q[b * self.width:b * self.width + n].double().numpy()
            want, mag, big = ref.tree_attention(q, keys, values, self.table[self.req[b]].tolist(), self.ctx[b], n,
                                                parent, self.scale)
            # bf16: each probability is rounded (eps of sum p |v|) and so is the result (eps |o|).
            # Both types: a score is a float32 sum of hd products (hd + 8 roundings of at most
            # sum |q k| scale, doubled by the maximum's), a weight's relative error is its score's,
            # and the two sums over the keys add one rounding per key and a few for joined parts.
            f32 = 2.0 ** -24 * (2 * (self.hd + 8) * big + 2 * (self.ctx[b] + n) + 64)
            tol = eps * (mag + np.abs(want)) + f32 * (1 + eps) * mag * 2 + 1e-30
            worst = float((np.abs(got[:n] - want) / tol).max())
            assert worst <= 1.0, (b, worst)


SHAPES = [
    # bs, width, heads, kv, hd, P, ctx, nodes, ids
    (1, 1, 1, 1, 64, 16, 0, None, False),        # the smallest: one token, no context
    (1, 1, 8, 8, 128, 16, 1, None, False),
    (1, 16, 32, 8, 128, 16, 2048, None, True),
    (3, 16, 10, 5, 64, 16, [37, 300, 129], [16, 3, 1], True),
    (4, 17, 10, 5, 64, 32, [0, 1, 127, 128], [17, 0, 5, 17], False),
    (5, 9, 12, 4, 128, 48, [111, 112, 113, 500, 7], None, True),
    (2, 64, 32, 8, 128, 16, [700, 1300], None, True),     # 256 query rows a head
    (2, 65, 8, 2, 128, 64, [64, 63], [65, 33], True),     # one row more than the tiles hold
    (2, 130, 7, 1, 64, 128, [5, 260], None, False),       # many row tiles, a group of 7
    (1, 300, 2, 1, 128, 16, [40], None, True),            # a tree wider than a position tile
    (1, 4, 4, 1, 128, 16, [9000], None, True),            # one row tile over many CTAs
    (3, 64, 32, 8, 128, 16, [5000, 9000, 300], [64, 64, 20], True),  # two row tiles over many positions
    (3, 50, 24, 4, 64, 32, [6000, 4001, 9000], [50, 3, 27], False),
    (40, 2, 4, 2, 64, 16, [3 * i for i in range(40)], None, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{s[0]}x{s[1]}h{s[2]}k{s[3]}d{s[4]}p{s[5]}" for s in SHAPES])
def test_tree_attention_matches(shape, dtype):
    bs, width, heads, kv, hd, P, ctx, nodes, ids = shape
    c = Case(bs, width, heads, kv, hd, P, ctx, nodes, ids, dtype, seed=bs + width)
    out, err = c.run()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_heads_of_32(dtype):
    c = Case(3, 13, 8, 4, 32, 16, [64, 1000, 333], [13, 5, 12], True, dtype, seed=9)
    out, err = c.run()
    assert err == 0
    c.check(out)


def test_tree_attention_widest_tree():
    c = Case(1, 1025, 2, 1, 64, 16, [33], None, True, "bf16", seed=4)
    out, err = c.run()
    assert err == 0
    c.check(out)


def test_tree_attention_many_requests():
    """More requests than a block has threads."""
    g = np.random.default_rng(3)
    ctx = [int(x) for x in g.integers(0, 90, 700)]
    nodes = [int(x) for x in g.integers(0, 4, 700)]
    for dtype in ("bf16", "f32"):
        c = Case(700, 3, 2, 1, 64, 16, ctx, nodes, True, dtype, seed=3)
        out, err = c.run()
        assert err == 0
        c.check(out, requests=list(range(0, 700, 13)) + [699])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_scores_far_apart(dtype):
    """Long queries: the running maximum moves by hundreds between tiles."""
    c = Case(2, 5, 4, 2, 64, 16, [700, 45], None, True, dtype, seed=6, spread=60.0)
    out, err = c.run()
    assert err == 0
    c.check(out)


def test_tree_attention_reads_strided_queries_the_same():
    c = Case(3, 16, 8, 2, 128, 16, [37, 300, 129], None, True, "bf16", seed=2)
    a, _ = c.run()
    b, _ = c.run(stride=8 * 128 + 512)
    assert torch.equal(a, b)


def test_tree_attention_repeats_bit_for_bit_and_replays():
    for dtype in ("bf16", "f32"):
        c = Case(6, 16, 8, 2, 128, 16, [37, 3000, 129, 5000, 1, 64], None, True, dtype, seed=8)
        a, _ = c.run()
        for _ in range(3):
            assert torch.equal(a, c.run()[0])
        # captured once, replayed with other inputs in the same buffers, on another stream
        s = torch.cuda.Stream()
        cache = F.make_cache_layer(c.keys.cuda(), c.values.cuda())
        ws = torch.empty(F.flashmap_tree_attention_workspace(cache, 6, 16, 8), dtype=torch.uint8, device="cuda")
        q, out, ctx = torch.zeros_like(c.q).cuda(), torch.zeros_like(c.q).cuda(), i32([16] * 6)
        ids, req, table, err = c.ids.cuda(), c.req.cuda(), c.table.cuda(), i32([0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            F.flashmap_tree_attention(cache, q, 16, ctx, None, ids, req, table, c.scale, out, ws, err)
        q.copy_(c.q)
        ctx.copy_(i32(c.ctx))
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.cpu(), a)
        assert int(err) == 0


@pytest.mark.parametrize("what,bit", [("page", "PAGE"), ("negative page", "PAGE"), ("row", "REQUEST"),
                                      ("context", "POSITION"), ("stride", "POSITION"), ("parent", "TREE"),
                                      ("nodes", "TREE"), ("every page", "PAGE")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_refuses_on_the_device(what, bit, dtype):
    c = Case(3, 8, 4, 2, 64, 16, [100, 57, 30], None, True, dtype, seed=5)
    left = [0, 2]
    if what == "page":
        c.table[c.req[1], 2] = c.keys.shape[0]
        left = [0, 1, 2]
    elif what == "negative page":
        c.table[c.req[1], 0] = -5
        left = [0, 1, 2]
    elif what == "every page":
        c.table[c.req[1]] = 1 << 30
        left = [0, 1, 2]
    elif what == "row":
        c.req[1] = 17
    elif what == "context":
        c.ctx[1] = -3
    elif what == "stride":
        c.table = c.table[:, :6].contiguous()  # request 0's last page is past the row
        left = [0, 1, 2]
    elif what == "parent":
        c.ids[1, 3] = 6 * 8 + 4
        c.ids[1, 5] = -1
        left = [0, 1, 2]
    elif what == "nodes":
        c.nodes = [8, 9, 8]
        left = [0, 1, 2]
    out, err = c.run()
    assert err == BITS[bit]
    c.check(out, requests=left)
    if 1 not in left:
        assert (out[8:16] == 7.0).all()  # a request that is skipped leaves its rows


# ------------------------------------------------------------------ sampling


def run_sampling(logits, per, temp, k, p, mp, u, ids=None, probs=True):
    rows = logits.shape[0]
    f = lambda x: None if x is None else torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    tokens = torch.full((rows,), -9, dtype=torch.int64, device="cuda")
    pr = torch.full((rows,), -9.0, device="cuda") if probs else None
    F.flashmap_sample_filtered(logits, per, f(temp), None if k is None else i32(k), f(p), f(mp), f(u), ids, tokens, pr)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), None if pr is None else pr.cpu().numpy()


def check_sampling(logits, per, temp, k, p, mp, u):
    tokens, probs = run_sampling(logits, per, temp, k, p, mp, u)
    host = logits.float().cpu().numpy()
    f = np.float32
    near = 0
    for r in range(host.shape[0]):
        b = r // per
        j, prob, margin = ref.sample_filtered(host[r], f(temp[b]), 0 if k is None else k[b],
                                              1.0 if p is None else float(f(p[b])),
                                              0.0 if mp is None else float(f(mp[b])), float(f(u[r])))
        # weights are good to 2e-9 of their own and 2^-45 of the largest (below 2^-6 of the largest,
        # where not listed: to 2^-22 of their own, either sign, thousands to a sum): a
        # border further than 2^-26 of the mass is not expected on the other side
        if margin < 2.0 ** -26:
            near += 1
            continue
        assert tokens[r] == j, (r, tokens[r], j, margin)
        assert abs(probs[r] - prob) <= 2.0 ** -23 * prob + 2.0 ** -44, (r, probs[r], prob)
    assert near <= host.shape[0] // 8


GRID = [(0, 1.0, 0.0), (1, 1.0, 0.0), (5, 1.0, 0.0), (0, 0.9, 0.0), (0, 0.0, 0.0), (0, 1.0, 0.05), (50, 0.8, 0.02),
        (1000, 0.999, 0.0), (0, 0.5, 1.0), (1 << 30, 1.0, 0.0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,seed,scale", [(1, 0, 1.0), (2, 1, 1.0), (33, 2, 3.0), (1234, 3, 2.0), (5000, 4, 0.1),
                                          (32768, 5, 2.5), (50257, 6, 2.5), (151936, 7, 4.0)])
def test_sampling_matches(V, seed, scale, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bs, per = len(GRID) + 1, 3
    logits = scale * torch.randn((bs * per, V + 3), generator=g, device="cuda")
    logits = logits.to(torch.float32 if dtype == "f32" else torch.bfloat16)[:, :V]
    k, p, mp = [x[0] for x in GRID] + [7], [x[1] for x in GRID] + [0.7], [x[2] for x in GRID] + [0.1]
    temp = [0.5 + 0.1 * i for i in range(len(GRID))] + [0.0]
    u = torch.rand(bs * per, generator=g, device="cuda").tolist()
    u[0], u[4], u[8] = 0.0, 0.99999994, 0.5
    check_sampling(logits, per, temp, k, p, mp, u)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad", [(300, 1), (8192, 0), (9001, 2), (60000, 5)])
def test_sampling_many_rows_as_few(V, pad, dtype):
    """A batch that gives each row a CTA of its own draws what a small one does; rows at odd offsets."""
    g = torch.Generator(device="cuda").manual_seed(V)
    bs = len(GRID) + 1
    buf = 2.5 * torch.randn((3 * bs, V + pad), generator=g, device="cuda")
    buf[:, :9] += 8.0
    few = buf.to(torch.float32 if dtype == "f32" else torch.bfloat16)[:, :V]
    k, p, mp = [x[0] for x in GRID] + [7], [x[1] for x in GRID] + [0.7], [x[2] for x in GRID] + [0.1]
    temp = [0.5 + 0.1 * i for i in range(len(GRID))] + [0.0]
    u = torch.rand(3 * bs, generator=g, device="cuda").tolist()
    check_sampling(few, 3, temp, k, p, mp, u)
    tokens, probs = run_sampling(few, 3, temp, k, p, mp, u)
    times = 10  # 330 rows
    many = buf.to(few.dtype).repeat(times, 1)[:, :V]
    t2, p2 = run_sampling(many, 3, temp * times, k * times, p * times, mp * times, u * times)
    np.testing.assert_array_equal(t2.reshape(times, -1), np.tile(tokens, (times, 1)))
    np.testing.assert_allclose(p2.reshape(times, -1), np.tile(probs, (times, 1)), rtol=2.0 ** -22, atol=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 40000])
def test_sampling_ties_and_odd_values(V, dtype):
    """Rows of equal logits, ties at a border, signed zeros, infinities, NaN, nothing finite."""
    inf, nan = float("inf"), float("nan")
    rows = torch.zeros((10, V))
    rows[1, ::2] = -0.0
    rows[2] = -inf
    rows[2, V // 3] = -5.0
    rows[3] = nan
    rows[3, 5::7] = 1.0
    rows[4] = -inf
    rows[5] = nan
    rows[6, 3::5] = 2.0                     # a tie of V / 5 above a tie of the rest
    rows[7, V - 1] = inf
    rows[7, V // 2] = inf
    rows[8] = torch.linspace(-1, 1, V).round(decimals=1)
    rows[9] = -3e38
    rows[9, 11] = 3e38
    logits = rows.to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    u = [0.37123, 0.9017, 0.5003, 0.1009, 0.2011, 0.3019, 0.7713, 0.6007, 0.4523, 0.9991]
    for k, p, mp in [(0, 1.0, 0.0), (13, 1.0, 0.0), (0, 0.3021, 0.0), (V // 4, 0.7733, 0.0), (0, 1.0, 1.0),
                     (0, 0.9137, 0.3)]:
        check_sampling(logits, 1, [1.0] * 10, [k] * 10, [p] * 10, [mp] * 10, u)
        # as many rows as fill the GPU with a CTA each
        few = run_sampling(logits, 1, [1.0] * 10, [k] * 10, [p] * 10, [mp] * 10, u)
        many = run_sampling(logits.repeat(32, 1), 1, [1.0] * 320, [k] * 320, [p] * 320, [mp] * 320, u * 32)
        for a, b in zip(few, many):
            np.testing.assert_array_equal(np.tile(a, 32), b)
    tokens, probs = run_sampling(logits, 1, [0.0] * 10, None, None, None, u)
    assert tokens.tolist() == [0, 0, V // 3, 5, 0, 0, 3, V // 2, int(logits[8].float().argmax()), 11]
    assert probs[4] == probs[5] == 0 and (probs[[0, 1, 2, 3, 6, 7, 8, 9]] == 1).all()


def test_sampling_odd_parameters():
    V, nan, inf = 300, float("nan"), float("inf")
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn((8, V), generator=g, device="cuda")
    check_sampling(logits, 1, [nan, -1.0, 1e-30, 1e30, inf, 1.0, 1.0, 1.0], [-3] * 8, [1.0, 1, 1, 1, 1, 2.0, -1.0, 1],
                   [0.0, 0, 0, 0, 0, -1.0, 0, 5.0], [0.5, 0.5, 0.5, 0.5, 0.25, -1.0, 2.0, 0.5])
    a = run_sampling(logits, 1, [1.0] * 8, None, [nan] * 8, [nan] * 8, [nan] * 8)[0]
    b = run_sampling(logits, 1, [1.0] * 8, None, None, None, [0.0] * 8)[0]
    assert (a == b).all()


def test_sampling_maps_ids_and_shares_requests():
    V, rows, per = 5000, 50, 16  # the last request has two rows
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = 3 * torch.randn((rows, V), generator=g, device="cuda")
    ids = torch.randperm(151936, generator=g, device="cuda")[:V]
    temp, u = [0.7, 0.0, 1.1, 0.9], torch.rand(rows, generator=g, device="cuda").tolist()
    plain, _ = run_sampling(logits, per, temp, [40] * 4, [0.95] * 4, [0.01] * 4, u)
    named, _ = run_sampling(logits, per, temp, [40] * 4, [0.95] * 4, [0.01] * 4, u, ids, probs=False)
    np.testing.assert_array_equal(ids.cpu().numpy()[plain], named)
    check_sampling(logits, per, temp, [40] * 4, [0.95] * 4, [0.01] * 4, u)


def test_sampling_follows_the_distribution():
    """Evenly spaced uniforms draw every kept entry in proportion: with n uniforms (i + 1/2) / n an
    entry of probability p is drawn within one of n p times."""
    V, n = 40, 4000
    g = torch.Generator(device="cuda").manual_seed(5)
    row = torch.randn((1, V), generator=g, device="cuda")
    u = [(i + 0.5) / n for i in range(n)]
    tokens, _ = run_sampling(row.repeat(n, 1), n, [0.8], [20], [0.9], None, u)
    l = row[0].double().cpu().numpy() / np.float64(np.float32(0.8))
    order = np.argsort(-l)[:20]
    w = np.exp(l[order] - l.max())
    keep = np.cumsum(w) - w < np.float64(np.float32(0.9)) * w.sum()
    p = np.zeros(V)
    p[order[keep]] = w[keep] / w[keep].sum()
    assert np.abs(np.bincount(tokens, minlength=V) - n * p).max() <= 1.01


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_a_drafted_tree(dtype):
    """Candidates -> tree -> pages and slots -> the nodes' keys and values written to their slots ->
    tree attention -> logits -> tokens: each step fed by the one before, as a serving loop does."""
    g = torch.Generator(device="cuda").manual_seed(12)
    bs, width, kv, heads, hd, P, V = 5, 12, 2, 8, 64, 16, 3000
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cand = torch.randint(0, 3, (bs, 4, 6), generator=g, device="cuda")
    toks, ids = (torch.empty((bs, width - 1), dtype=torch.int64, device="cuda") for _ in range(2))
    stats = torch.empty((bs, 2), dtype=torch.int64, device="cuda")
    F.flashmap_build_tree(cand, width, toks, ids, stats)
    lens, held = [30, 0, 77, 16, 5], [3, 0, 5, 1, 1]
    pages, stride = 64, 9
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((bs, stride), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(bs):
        table[b, : held[b]] = order[at:at + held[b]]
        at += held[b]
    keys, values = (torch.randn((pages, kv, P, hd), generator=g, device="cuda").to(dt) for _ in range(2))
    cu, head, held_out = i32([0] * (bs + 1)), i32([0]), i32([0] * bs)
    slots = torch.full((bs * width,), -9, dtype=torch.int64, device="cuda")
    err = i32([0])
    req = i32(list(range(bs)))
    F.flashmap_extend_pages(req, i32(lens), i32([width] * bs), i32(held), P, table, order, i32([at]), head, held_out,
                            pages, cu, slots, None, None, err)
    assert (slots >= 0).all() and len(set(slots.tolist())) == bs * width
    new_k, new_v = (torch.randn((bs * width, kv, hd), generator=g, device="cuda").to(dt) for _ in range(2))
    keys[slots // P, :, slots % P] = new_k
    values[slots // P, :, slots % P] = new_v
    q = torch.randn((bs * width, heads, hd), generator=g, device="cuda").to(dt)
    out = torch.empty_like(q)
    cache = F.make_cache_layer(keys, values)
    ws = torch.empty(F.flashmap_tree_attention_workspace(cache, bs, width, heads), dtype=torch.uint8, device="cuda")
    F.flashmap_tree_attention(cache, q, width, i32(lens), None, ids, req, table, hd ** -0.5, out, ws, err)
    lm = torch.randn((V, heads * hd), generator=g, device="cuda").to(dt)
    logits = out.view(bs * width, -1) @ lm.T
    u = torch.rand(bs * width, generator=g, device="cuda")
    drawn = torch.empty(bs * width, dtype=torch.int64, device="cuda")
    params = dict(temp=[0.9, 0.0, 1.2, 0.5, 1.0], k=[50, 0, 0, 1, 900], p=[0.9, 1.0, 0.95, 1.0, 1.0],
                  mp=[0.0, 0.0, 0.01, 0.0, 0.1])
    f = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
    F.flashmap_sample_filtered(logits, width, f(params["temp"]), i32(params["k"]), f(params["p"]), f(params["mp"]), u,
                               None, drawn, None)
    torch.cuda.synchronize()
    assert int(err) == 0
    c = Case(bs, width, heads, kv, hd, P, lens, None, False, dtype)
    c.keys, c.values, c.q, c.req, c.table = keys.cpu(), values.cpu(), q.cpu(), req.cpu(), table.cpu()
    c.ids = ids.cpu()
    c.check(out.cpu())
    check_sampling(logits, width, params["temp"], params["k"], params["p"], params["mp"], u.tolist())
    assert held_out.tolist() == [3, 1, 6, 2, 2] and int(head) == at + 4


# ------------------------------------------------------------------ how they are called


def cuda_case(c):
    """A case's tensors on the GPU, as the call takes them (the workspace aside)."""
    cache = F.make_cache_layer(c.keys.cuda(), c.values.cuda())
    return dict(cache=cache, q=c.q.cuda(), width=c.width, ctx=i32(c.ctx), nodes=i32(c.nodes) if c.nodes else None,
                ids=c.ids.cuda() if c.ids is not None else None, req=c.req.cuda(), table=c.table.cuda(), scale=c.scale)


def attend(d, out, ws, err=None, stream=None):
    F.flashmap_tree_attention(d["cache"], d["q"], d["width"], d["ctx"], d["nodes"], d["ids"], d["req"], d["table"],
                              d["scale"], out, ws, err, stream)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [
    (17, 17, 10, 5, 64, 32, [37 * i * i % 2999 for i in range(17)], [1 + i for i in range(17)], False),  # shares end inside items
    (16, 3, 8, 4, 64, 16, [2900 + i for i in range(16)], None, True),
    (2, 9, 8, 2, 128, 16, [1500, 40], None, True),       # each item cut apart
    (3, 5, 4, 2, 64, 16, [0, 900, 64], [0, 5, 0], True),  # two of three requests without nodes
    (4, 33, 8, 2, 64, 16, [10, 0, 511, 700], [33, 1, 32, 17], True),  # one or two row tiles
], ids=["even", "even long", "cut", "cut, empty", "cut, ragged"])
def test_tree_attention_shares(shape, dtype):
    bs, width, heads, kv, hd, P, ctx, nodes, ids = shape
    c = Case(bs, width, heads, kv, hd, P, ctx, nodes, ids, dtype, seed=bs)
    out, err = c.run()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_a_hidden_key_does_not_matter(dtype):
    """NaN and infinite keys in nodes: the rows that do not see them are as they were."""
    c = Case(2, 10, 8, 2, 64, 16, [70, 20], None, True, dtype, seed=11)
    a, _ = c.run()
    hit = {0: 7, 1: 4}
    for b, i in hit.items():
        pos = c.ctx[b] + i
        c.keys[c.table[c.req[b], pos // 16], :, pos % 16] = float("nan") if b else float("inf")
    z, err = c.run()
    assert err == 0
    for b, i in hit.items():
        parent = ref.parents_of(c.ids[b].tolist(), 10)
        for node in range(10):
            x, seen = node, False
            while x >= 0:
                seen |= x == i
                x = parent[x]
            if not seen:
                assert torch.equal(a[b * 10 + node], z[b * 10 + node]), (b, node)


@pytest.mark.parametrize("dtype,hd", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("scale", [-0.11, 0.0])
def test_tree_attention_other_scales(scale, dtype, hd):
    c = Case(2, 40, 8, 2, hd, 16, [300, 41], [40, 17], True, dtype, seed=5)  # one item of two row tiles, one of one
    c.scale = scale
    out, err = c.run()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype,hd", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_tree_attention_16_byte_alignment(dtype, hd):
    """Queries and outputs 16 bytes past a boundary, query rows 16 bytes more than dense."""
    c = Case(2, 12, 8, 2, hd, 16, [300, 41], None, True, dtype, seed=6)
    a, _ = c.run()
    d = cuda_case(c)
    rows, step = c.q.shape[0], 8 * hd
    off = 16 // c.q.element_size()
    q = torch.zeros(off + rows * (step + off), dtype=c.q.dtype, device="cuda")[off:].view(rows, step + off)[:, :step]
    q.copy_(d["q"].view(rows, step))
    d["q"] = q.unflatten(1, (8, hd))
    out = torch.zeros(off + rows * step, dtype=c.q.dtype, device="cuda")[off:].view(rows, 8, hd)
    assert d["q"].data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    ws = torch.zeros(F.flashmap_tree_attention_workspace(d["cache"], 2, 12, 8), dtype=torch.uint8, device="cuda")
    attend(d, out, ws)
    assert torch.equal(out.cpu(), a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_refuses_workspaces(dtype):
    c = Case(1, 4, 4, 2, 64, 16, [100], None, True, dtype)
    d = cuda_case(c)
    n = F.flashmap_tree_attention_workspace(d["cache"], 1, 4, 4)
    out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    for bad in (ws[: n - 1], ws[16:], ws[:0]):
        with pytest.raises((F.FlashmapError, ValueError)):
            attend(d, out, bad)
    with pytest.raises((F.FlashmapError, ValueError, TypeError)):
        attend(d, out, torch.zeros(n, dtype=torch.uint8))
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    attend(d, out, ws[:n])
    c.check(out.cpu())


def test_tree_attention_graphs_share_a_workspace():
    """Two captured calls of different shapes over one workspace, replayed in turn."""
    cases = [Case(3, 16, 8, 2, 128, 16, [900, 5, 4000], None, True, "bf16", seed=1),
             Case(2, 40, 8, 2, 128, 16, [3000, 77], [40, 9], True, "bf16", seed=2)]
    ds = [cuda_case(c) for c in cases]
    ws = torch.full((max(F.flashmap_tree_attention_workspace(d["cache"], c.bs, c.width, 8) for c, d in zip(cases, ds)),),
                    255, dtype=torch.uint8, device="cuda")
    outs = [torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda") for c in cases]
    graphs, s = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for d, out in zip(ds, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            attend(d, out, ws)
        graphs.append(graph)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            c.check(out.cpu())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_on_two_streams(dtype):
    """Calls at once, each with a workspace and outputs of its own."""
    c = Case(8, 8, 8, 2, 64, 16, [300 * i for i in range(8)], None, True, dtype, seed=3)
    d = cuda_case(c)
    alone, _ = c.run()
    V = 50257
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = 2.5 * torch.randn((8, V), generator=g, device="cuda")
    f = lambda x: torch.full((8,), x, device="cuda")  # noqa: E731
    u = torch.rand(8, generator=g, device="cuda")
    args = (f(0.9), i32([0, 40] * 4), f(0.9), f(0.0), u, None)
    want = torch.empty(8, dtype=torch.int64, device="cuda")
    F.flashmap_sample_filtered(logits, 1, *args, want, None)
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = F.flashmap_tree_attention_workspace(d["cache"], 8, 8, 8)
    sets = [(torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda"),
             torch.empty(8, dtype=torch.int64, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (ws, out, tokens) in zip(streams, sets):
            with torch.cuda.stream(s):
                attend(d, out, ws)
                F.flashmap_sample_filtered(logits, 1, *args, tokens, None)
    torch.cuda.synchronize()
    for _, out, tokens in sets:
        assert torch.equal(out.cpu(), alone) and torch.equal(tokens, want)


def test_pages_and_sampling_replay():
    """Captured once, replayed with other inputs in the same buffers."""
    P, bs = 16, 3
    req, lens, new, held = i32([2, 0, 1]), i32([0, 0, 0]), i32([1, 1, 1]), i32([0, 0, 0])
    start = torch.arange(40, dtype=torch.int32, device="cuda").reshape(5, 8)
    table, free, head, out_head = start.clone(), i32(list(range(50, 70))), i32([0]), i32([-1])
    cu, slots, err = i32([0] * 4), torch.zeros(64, dtype=torch.int64, device="cuda"), i32([0])
    V = 9000
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = torch.zeros((bs, V), device="cuda")
    temp, k, p, u = torch.ones(bs, device="cuda"), i32([0] * bs), torch.ones(bs, device="cuda"), torch.zeros(bs, device="cuda")
    tokens, probs = torch.zeros(bs, dtype=torch.int64, device="cuda"), torch.zeros(bs, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.flashmap_extend_pages(req, lens, new, held, P, table, free, head, out_head, None, 70, cu, slots, None, None, err)
        F.flashmap_sample_filtered(logits, 1, temp, k, p, None, u, None, tokens, probs)
    for seed in range(2):
        r = np.random.default_rng(seed)
        a, n = [int(x) for x in r.integers(0, 60, bs)], [int(x) for x in r.integers(0, 20, bs)]
        h = [-(-x // P) for x in a]
        for x, y in ((lens, a), (new, n), (held, h)):
            x.copy_(i32(y))
        table.copy_(start)
        slots.fill_(-9)
        logits.copy_(2.5 * torch.randn((bs, V), generator=g, device="cuda"))
        k.copy_(i32([0, 30, 700]))
        p.fill_(0.9)
        u.copy_(torch.rand(bs, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        t, hd, _, c, want, *_ = ref.extend_pages([2, 0, 1], a, n, h, P, start.cpu().numpy(), list(range(50, 70)), 0, 70, 64)
        np.testing.assert_array_equal(table.cpu().numpy(), t)
        assert int(err) == 0 and int(out_head) == hd
        np.testing.assert_array_equal(slots.cpu().numpy()[: c[-1]], want[: c[-1]])
        again = run_sampling(logits, 1, [1.0] * 3, [0, 30, 700], [0.9] * 3, None, u.tolist())
        np.testing.assert_array_equal(tokens.cpu().numpy(), again[0])
        np.testing.assert_array_equal(probs.cpu().numpy(), again[1])
        check_sampling(logits, 1, [1.0] * 3, [0, 30, 700], [0.9] * 3, None, u.tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 35, 129, 1431, 2048])
def test_sampling_many_small_rows(V, dtype):
    """More rows of few entries than the GPU holds at once, every filter, some rows full of ties."""
    g = torch.Generator(device="cuda").manual_seed(V)
    times = 20
    bs = len(GRID) * times
    logits = 2.5 * torch.randn((bs * 4, V), generator=g, device="cuda")
    logits[3::8] = logits[3::8].round()
    logits = logits.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    k, p, mp = [x[0] for x in GRID] * times, [x[1] for x in GRID] * times, [x[2] for x in GRID] * times
    temp = [0.4 + 0.01 * (i % 90) for i in range(bs)]
    u = torch.rand(bs * 4, generator=g, device="cuda").tolist()
    check_sampling(logits, 4, temp, k, p, mp, u)


# ------------------------------------------------------------------ far offsets


def test_pages_far_ids():
    """Slots past 2^31."""
    free = [(1 << 30) - 7, 1 << 29, (1 << 30) - 1]
    err, served = check_pages([0, 1], [0, 16], [20, 1], [0, 1], 16, [[-1] * 4, [(1 << 30) - 2] + [-1] * 3], free, 0,
                              1 << 30, 64)
    assert err == 0 and all(served)


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_tree_attention_far_pages(dtype, hd):
    """Pages whose entries lie past 2^31 elements give what the same pages give near the start."""
    kv, P = 8, 16
    c = Case(2, 6, 16, kv, hd, P, [200, 33], None, True, dtype, seed=4)
    near, _ = c.run()
    few = c.keys.shape[0]
    pages = (1 << 31) // (kv * P * hd) + few + 5
    dt = c.q.dtype
    keys, values = (torch.empty((pages, kv, P, hd), dtype=dt, device="cuda") for _ in range(2))
    keys[pages - few:] = c.keys.cuda()
    values[pages - few:] = c.values.cuda()
    d = cuda_case(c)
    d["cache"] = F.make_cache_layer(keys, values)
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - few), d["table"])
    out = torch.full(c.q.shape, 7.0, dtype=dt, device="cuda")
    ws = torch.zeros(F.flashmap_tree_attention_workspace(d["cache"], 2, 6, 16), dtype=torch.uint8, device="cuda")
    attend(d, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), near)


def test_sampling_far_and_many_rows():
    V, rows, ld = 1000, 9, 1 << 28
    g = torch.Generator(device="cuda").manual_seed(6)
    few = (2.5 * torch.randn((rows, V), generator=g, device="cuda")).bfloat16()
    u = torch.rand(rows, generator=g, device="cuda").tolist()
    want = run_sampling(few, 3, [0.9] * 3, [0, 20, 0], [0.9, 1.0, 1.0], None, u)
    far = torch.empty(((rows - 1) * ld + V,), dtype=torch.bfloat16, device="cuda").as_strided((rows, V), (ld, 1))
    far.copy_(few)
    got = run_sampling(far, 3, [0.9] * 3, [0, 20, 0], [0.9, 1.0, 1.0], None, u)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    del far
    times = 8000
    got = run_sampling(few.repeat(times, 1), 3, [0.9] * 3 * times, [0, 20, 0] * times, [0.9, 1.0, 1.0] * times, None,
                       u * times)
    np.testing.assert_array_equal(got[0].reshape(times, rows), np.tile(want[0], (times, 1)))
