"""The operators that verify a drafted tree on the target's side, as measured work:

- ``pages``: page tables and slot maps extended on the GPU from request lengths;
- ``attention``: a tree of drafted tokens attending to a paged cache and to its own
  ancestors (a chain when the tree is a single block, single tokens when it is one node);
- ``sampling``: tokens drawn from logits under temperature, top-k, top-p and min-p, from
  one given uniform number per row.

Each case is listed with what it stands for. ``run`` computes a case in plain torch
operations, or with ``own`` set through the library's entry points.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a single request growing by a tree of 16 nodes: pure latency
        dict(name="pages, one request", op="pages", bs=1, rows=4, page=16, lo=2048, hi=2048, new_lo=16, new_hi=16),
        # a verify step of a ragged batch: a block and its anchor for each request
        dict(name="pages, batch 128", op="pages", bs=128, rows=131, page=16, lo=16, hi=32768, new_lo=0, new_hi=17),
        # prompts of a batch entering the cache at once
        dict(name="pages, prompts", op="pages", bs=64, rows=67, page=16, lo=0, hi=40, new_lo=1024, new_hi=16384),
        # one request, a tree of 16 nodes over a short context: latency
        dict(name="tree, one request", op="attention", bs=1, width=16, heads=32, kv_heads=8, hd=128, page=16,
             lo=2048, hi=2048, ids=True, ragged=False, dtype="bf16"),
        # a serving batch with small trees: bound by the cache's bytes
        dict(name="tree, batch 32", op="attention", bs=32, width=16, heads=32, kv_heads=8, hd=128, page=16,
             lo=512, hi=8192, ids=True, ragged=False, dtype="bf16"),
        # a large batch with wide ragged trees: products and bytes weigh alike
        dict(name="tree, batch 128, 64 nodes", op="attention", bs=128, width=64, heads=32, kv_heads=8, hd=128,
             page=16, lo=512, hi=8192, ids=True, ragged=True, dtype="bf16"),
        # single drafted blocks (a chain), odd head counts and lengths
        dict(name="chain of 17, 10 heads of 64", op="attention", bs=17, width=17, heads=10, kv_heads=5, hd=64,
             page=32, lo=37, hi=3000, ids=False, ragged=True, dtype="bf16"),
        # plain decoding of single tokens over long caches
        dict(name="single tokens, long cache", op="attention", bs=4, width=1, heads=32, kv_heads=8, hd=128, page=64,
             lo=100000, hi=131072, ids=False, ragged=False, dtype="bf16"),
        # the float32 model's shape, a batch of trees
        dict(name="tree, float32", op="attention", bs=5, width=13, heads=8, kv_heads=4, hd=32, page=16, lo=64,
             hi=1000, ids=True, ragged=True, dtype="f32"),
        # the 16 nodes of one request over the full vocabulary: latency
        dict(name="sampling, one request", op="sampling", bs=1, per=16, vocab=151936, pad=0, dtype="f32"),
        # drafted blocks of a batch over the draft vocabulary
        dict(name="sampling, draft vocabulary", op="sampling", bs=32, per=16, vocab=32768, pad=0, dtype="f32"),
        # the nodes of a batch of trees over the full vocabulary
        dict(name="sampling, 1024 rows", op="sampling", bs=64, per=16, vocab=151936, pad=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "attention", "attention", "sampling"])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "pages":
        bs = _log(rng, 1, 1500)
        lo = _log(rng, 1, 4000)
        new = _log(rng, 1, max(2, min(16384, 500000 // bs)))
        return dict(op="pages", bs=bs, rows=bs + rng.randint(0, 9), page=page, lo=lo - 1, hi=lo + _log(rng, 1, 4000),
                    new_lo=rng.randint(0, new), new_hi=new)
    if op == "sampling":
        dtype = rng.choice(["f32", "bf16"])
        vocab = _log(rng, 2, 200000)
        per = _log(rng, 1, 64)
        bs = _log(rng, 1, max(2, min(4096, 60_000_000 // (vocab * per))))
        return dict(op="sampling", bs=bs, per=per, vocab=vocab, pad=rng.choice([0, 0, 1, 8]), dtype=dtype)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    kv = _log(rng, 1, 16)
    heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    hd = rng.choice([32, 64, 128]) if dtype == "f32" else rng.choice([64, 128, 128])
    width = _log(rng, 1, 200)
    hi = _log(rng, 1, 4000) if dtype == "f32" else _log(rng, 1, 30000)
    most = 40_000_000_000 if dtype == "f32" else 250_000_000_000
    bs = _log(rng, 1, max(1.5, min(200.0, most / (4.0 * width * heads * hd * (hi + width)),
                                   4e9 / (4.0 * kv * hd * (hi + width)), 2e9 / (4.0 * width * heads * (hi + width)))))
    return dict(op="attention", bs=bs, width=width, heads=heads, kv_heads=kv, hd=hd, page=page,
                lo=rng.randint(0, hi), hi=hi, ids=width > 1 and rng.random() < 0.7, ragged=rng.random() < 0.6,
                dtype=dtype)


# ------------------------------------------------------------------ inputs


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int32)


def _prepare_pages(c, seed):
    g = torch.Generator().manual_seed(seed)
    P, bs = c["page"], c["bs"]
    lens, new = _ints(g, c["lo"], c["hi"], bs), _ints(g, c["new_lo"], c["new_hi"], bs)
    # every third request still holds a page or two reserved for rejected tokens
    held = (lens + P - 1) // P + (torch.rand(bs, generator=g) < 0.34).int() * _ints(g, 0, 2, bs)
    stride = (c["hi"] + c["new_hi"] + P - 1) // P + 3
    pages = c["rows"] * stride + 7
    perm = torch.randperm(pages, generator=g).int()
    table = perm[: c["rows"] * stride].view(c["rows"], stride)
    after = torch.maximum(held, (lens + new + P - 1) // P)
    req = torch.randperm(c["rows"], generator=g)[:bs].int()
    # the free list: the table's unheld pages, in a shuffled order, some already handed out
    cols = torch.arange(stride)
    used = torch.zeros(c["rows"], dtype=torch.int32)
    used[req.long()] = held
    free = table[cols >= used[:, None]]
    free = free[torch.randperm(free.numel(), generator=g)]
    head = int(torch.randint(0, max(1, free.numel() - int((after - held).sum()) + 1), (1,), generator=g))
    table = torch.where(cols < used[:, None], table, -1).contiguous()
    cap = bs * c["new_hi"] + 5  # a step's buffers fit its largest case
    d = dict(req=req, lens=lens, new=new, held=held, table=table, free=free.contiguous(),
             head=torch.tensor([head], dtype=torch.int32))
    d = {k: v.int().cuda() for k, v in d.items()}
    d["pages"], d["page"] = pages, P
    d["head_out"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    d["held_out"] = torch.zeros(bs, dtype=torch.int32, device="cuda")
    d["cu"] = torch.zeros(bs + 1, dtype=torch.int32, device="cuda")
    d["slots"] = torch.full((cap,), -7, dtype=torch.int64, device="cuda")
    d["positions"] = torch.full((cap,), -7, dtype=torch.int32, device="cuda")
    d["owner"] = torch.full((cap,), -7, dtype=torch.int32, device="cuda")
    return d


def _parents(c, g):
    """Parents of nodes 1.. of every request, listed by depth (they never decrease): about four branches."""
    q = torch.arange(1, c["width"])
    back = torch.randint(0, 6, (c["bs"], c["width"] - 1), generator=g)
    return torch.cummax((q - 1 - back).clamp(min=0), dim=1).values


def _prepare_attention(c, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    bs, width, P = c["bs"], c["width"], c["page"]
    ctx = _ints(g, c["lo"], c["hi"], bs)
    nodes = _ints(g, 1, width, bs) if c["ragged"] else torch.full((bs,), width, dtype=torch.int32)
    need = (ctx + width + P - 1) // P
    stride = int(need.max())
    pages = int(need.sum()) + 7
    perm = torch.randperm(pages, generator=g).int()
    rows = bs + 3
    req = torch.randperm(rows, generator=g)[:bs].int()
    table = torch.zeros(rows, stride, dtype=torch.int32)
    first = torch.cumsum(need, 0) - need
    cols = torch.arange(stride)
    at = (first[:, None] + cols).clamp(max=pages - 1).long()
    table[req.long()] = torch.where(cols < need[:, None], perm[at], 0)
    dt = DTYPES[c["dtype"]]
    shape = (pages, c["kv_heads"], P, c["hd"])
    keys = torch.randn(shape, generator=gd, device="cuda", dtype=dt)
    values = torch.randn(shape, generator=gd, device="cuda", dtype=dt)
    # scores spread by about 1.5: queries a little longer than the keys
    q = (1.5 * torch.randn((bs * width, c["heads"], c["hd"]), generator=gd, device="cuda")).to(dt)
    ids = None
    if c["ids"]:
        ids = (_parents(c, g) * width + torch.arange(1, width)).cuda()
    return dict(q=q, keys=keys, values=values, ctx=ctx.cuda(), nodes=nodes.cuda() if c["ragged"] else None, ids=ids,
                req=req.cuda(), table=table.cuda(), longest=int((ctx + width).max()), scale=c["hd"] ** -0.5,
                out=torch.zeros_like(q), width=width, err=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_sampling(c, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    rows, V = c["bs"] * c["per"], c["vocab"]
    buf = torch.randn((rows, V + c["pad"]), generator=gd, device="cuda").mul_(2.5)
    # a few likely tokens in each row
    some = torch.randint(0, V, (rows, 12), generator=gd, device="cuda")
    buf.scatter_add_(1, some, 9.0 * torch.rand((rows, 12), generator=gd, device="cuda"))
    logits = buf.to(DTYPES[c["dtype"]])[:, :V]
    bs = c["bs"]
    pick = lambda vals: torch.tensor(vals)[torch.randint(0, len(vals), (bs,), generator=g)].cuda()  # noqa: E731
    greedy = (torch.rand(bs, generator=g) < 0.15) & (torch.arange(bs) > 0)
    temps = torch.where(greedy, 0.0, 0.5 + 0.7 * torch.rand(bs, generator=g)).cuda()
    return dict(logits=logits, temps=temps.float(), top_k=pick([0, 0, 1, 20, 50, 1000]).int(),
                top_p=pick([1.0, 0.8, 0.9, 0.95]).float(), min_p=pick([0.0, 0.0, 0.02, 0.1]).float(),
                u=torch.rand(rows, generator=gd, device="cuda"), per=c["per"],
                tokens=torch.zeros(rows, dtype=torch.int64, device="cuda"),
                probs=torch.zeros(rows, dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    make = {"pages": _prepare_pages, "attention": _prepare_attention, "sampling": _prepare_sampling}[case["op"]]
    return dict(make(case, seed), op=case["op"])


# ------------------------------------------------------------------ one pass


def _plain_pages(s):
    P, req = s["page"], s["req"].long()
    lens, new, held = s["lens"].long(), s["new"].long(), s["held"].long()
    need = ((lens + new + P - 1) // P - held).clamp(min=0)
    first = s["head"].long() + torch.cumsum(need, 0) - need
    cols = torch.arange(s["table"].shape[1], device="cuda")
    k = cols - held[:, None]
    fresh = s["free"][(first[:, None] + k).clamp(0, s["free"].numel() - 1)]
    mine = torch.where((k >= 0) & (k < need[:, None]), fresh, s["table"][req])
    s["table"][req] = mine
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(new, 0)])
    t = torch.arange(s["slots"].numel(), device="cuda")
    live = t < cu[-1]
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=len(req) - 1)
    pos = torch.where(live, lens[b] + t - cu[b], 0)
    slot = mine[b, pos // P].long() * P + pos % P
    s["slots"].copy_(torch.where(live, slot, s["slots"]))
    s["positions"].copy_(torch.where(live, pos, s["positions"]))
    s["owner"].copy_(torch.where(live, b, s["owner"]))
    s["cu"].copy_(cu)
    s["held_out"].copy_(held + need)
    s["head_out"].copy_(s["head"] + need.sum())


def _run_pages(s):
    if own:
        from speculative_decoding_block_context_gb300 import _lib as F

        F.flashmap_extend_pages(s["req"], s["lens"], s["new"], s["held"], s["page"], s["table"], s["free"], s["head"],
                                s["head_out"], s["held_out"], s["pages"], s["cu"], s["slots"], s["positions"],
                                s["owner"])
    else:
        _plain_pages(s)
    return [s[k] for k in ("table", "head_out", "held_out", "cu", "slots", "positions", "owner")]


def _plain_attention(s):
    bs, width, hd = s["ctx"].numel(), s["width"], s["q"].shape[2]
    kv, P = s["keys"].shape[1:3]
    group = s["q"].shape[1] // kv
    at = torch.arange(s["longest"], device="cuda")
    page = s["table"][s["req"].long()][:, at // P].long()  # [bs][longest]
    k = s["keys"][page, :, at % P].float()  # [bs][longest][kv][hd]
    v = s["values"][page, :, at % P].float()
    q = s["q"].float().view(bs, width, kv, group, hd)
    q = q.permute(0, 2, 1, 3, 4).reshape(bs, kv, width * group, hd)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    # sees[b][i][j]: node j is node i or one of its ancestors (powers of the parent relation, doubled)
    i = torch.arange(width, device="cuda")
    if s["ids"] is None:
        sees = (i[None, :] <= i[:, None]).expand(bs, width, width)
    else:
        up = torch.eye(width, device="cuda").repeat(bs, 1, 1)
        up[:, 1:].scatter_(2, (s["ids"] // width)[:, :, None], 1.0)
        for _ in range(max(1, math.ceil(math.log2(width)))):
            up = (torch.matmul(up, up) > 0).float()
        sees = up > 0
    nodes = s["nodes"] if s["nodes"] is not None else torch.full_like(s["ctx"], width)
    j = at[None, :] - s["ctx"][:, None]  # position as a node's index, negative in the context
    tree = torch.gather(sees, 2, j.clamp(0, width - 1)[:, None, :].expand(bs, width, at.numel()))
    mask = (j < 0)[:, None, :] | (tree & (j < nodes[:, None])[:, None, :])
    mask = mask[:, None, :, None, :].expand(bs, kv, width, group, at.numel()).reshape(score.shape)
    score = torch.where(mask, score, -torch.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    live = (j < nodes[:, None])[:, :, None, None]
    o = torch.matmul(p, torch.where(live, v, 0.0).permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    o = o.view(bs, kv, width, group, hd).permute(0, 2, 1, 3, 4).reshape(bs, width, kv * group, hd)
    there = (i[None, :] < nodes[:, None])[:, :, None, None]
    s["out"].copy_(torch.where(there, o.to(s["out"].dtype), s["out"].view(o.shape)).reshape(s["out"].shape))


def _run_attention(s):
    if own:
        from speculative_decoding_block_context_gb300 import _lib as F

        if "cache" not in s:
            s["cache"] = F.make_cache_layer(s["keys"], s["values"])
            n = F.flashmap_tree_attention_workspace(s["cache"], s["ctx"].numel(), s["width"], s["q"].shape[1])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        F.flashmap_tree_attention(s["cache"], s["q"], s["width"], s["ctx"], s["nodes"], s["ids"], s["req"], s["table"],
                                  s["scale"], s["out"], s["workspace"], s["err"])
    else:
        _plain_attention(s)
    return s["out"]


def _plain_sampling(s):
    l, V, per = s["logits"].float(), s["logits"].shape[1], s["per"]
    each = lambda x: x.repeat_interleave(per)[:, None]  # noqa: E731
    temp, top_k = each(s["temps"]).double(), each(s["top_k"]).long()
    top_p, min_p = each(s["top_p"]).double(), each(s["min_p"]).double()
    order, index = torch.sort(l, dim=1, descending=True, stable=True)  # ties: the lowest index first
    greedy = temp <= 0
    # weights and their sums in 64 bits: a cut or a draw may fall next to a border
    w = torch.exp((order.double() - order[:, :1].double()) / torch.where(greedy, 1.0, temp))
    mass = torch.cumsum(w, 1)
    k = torch.where((top_k <= 0) | (top_k > V), V, top_k)
    total = torch.gather(mass, 1, k - 1)
    rank = torch.arange(V, device="cuda")
    keep = (rank < k) & (w >= min_p) & ((top_p >= 1) | (mass - w < top_p * total))
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, index, w * keep)
    run_sum = torch.cumsum(kept, 1)
    j = (run_sum > s["u"][:, None].double() * run_sum[:, -1:]).int().argmax(1, keepdim=True)
    prob = torch.gather(kept, 1, j) / run_sum[:, -1:]
    s["tokens"].copy_(torch.where(greedy, index[:, :1], j)[:, 0])
    s["probs"].copy_(torch.where(greedy, 1.0, prob)[:, 0])


def _run_sampling(s):
    if own:
        from speculative_decoding_block_context_gb300 import _lib as F

        F.flashmap_sample_filtered(s["logits"], s["per"], s["temps"], s["top_k"], s["top_p"], s["min_p"], s["u"],
                                   None, s["tokens"], s["probs"])
    else:
        _plain_sampling(s)
    return [s["tokens"], s["probs"]]


def run(state):
    return {"pages": _run_pages, "attention": _run_attention, "sampling": _run_sampling}[state["op"]](state)


# ------------------------------------------------------------------ what a pass needs


def work(c):
    bs = c["bs"]
    if c["op"] == "pages":
        new, P = bs * (c["new_lo"] + c["new_hi"]) / 2, c["page"]
        fresh = new / P
        # 4 integers in and 2 out per request; a page id read and entered per new page; 16 bytes per token
        return {"bytes": 24.0 * bs + 8.0 * fresh + 16.0 * new + 8, "flops": 0.0}
    el = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "sampling":
        n = float(bs * c["per"]) * c["vocab"]
        return {"bytes": n * el + bs * (16.0 + c["per"] * 16.0), "flops": 3.0 * n}
    ctx, nodes = (c["lo"] + c["hi"]) / 2, (c["width"] + 1) / 2 if c["ragged"] else c["width"]
    cache = bs * (ctx + nodes) * c["kv_heads"] * c["hd"] * 2.0 * el
    queries = bs * nodes * c["heads"] * c["hd"]
    return {"bytes": cache + 2.0 * queries * el, "flops": 4.0 * queries * (ctx + nodes / 2)}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_attention(c, seed):
    s = _prepare_attention(c, seed)
    width, P, kv = c["width"], c["page"], c["kv_heads"]
    group = c["heads"] // kv
    out = torch.zeros(c["bs"], width, c["heads"], c["hd"], dtype=torch.float64, device="cuda")
    ctx = s["ctx"].tolist()
    nodes = s["nodes"].tolist() if s["nodes"] is not None else [width] * c["bs"]
    parent = (s["ids"] // width).cpu().numpy() if s["ids"] is not None else None
    for b in range(c["bs"]):
        n, m = ctx[b] + nodes[b], nodes[b]
        see = np.zeros((m, m), dtype=bool)
        for i in range(m):
            if i:
                see[i] = see[i - 1 if parent is None else parent[b, i - 1]]
            see[i, i] = True
        hidden = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        hidden[:, ctx[b]:] = torch.from_numpy(np.where(see, 0.0, -np.inf)).cuda()
        pages = s["table"][int(s["req"][b]), : (n + P - 1) // P].long()
        q = s["q"].view(c["bs"], width, c["heads"], c["hd"])[b, :m].double()
        for h in range(kv):
            k = s["keys"][pages, h].reshape(-1, c["hd"])[:n].double()
            v = s["values"][pages, h].reshape(-1, c["hd"])[:n].double()
            qh = q[:, h * group:(h + 1) * group].permute(1, 0, 2)
            a = torch.softmax(qh @ k.T / math.sqrt(c["hd"]) + hidden, dim=-1) @ v
            out[b, :m, h * group:(h + 1) * group] = a.permute(1, 0, 2)
    return out.view(s["out"].shape)


def _exact_sampling(c, seed):
    s = _prepare_sampling(c, seed)
    rows, per, V = c["bs"] * c["per"], c["per"], c["vocab"]
    prob = torch.ones(rows, dtype=torch.float64, device="cuda")
    temps, ks, ps, ms = (s[k].tolist() for k in ("temps", "top_k", "top_p", "min_p"))
    us = s["u"].tolist()
    for r in range(rows):
        b = r // per
        if temps[b] <= 0:
            continue
        x = s["logits"][r].double() / temps[b]
        x, place = torch.sort(x, descending=True, stable=True)
        share = torch.softmax(x, 0)
        n = ks[b] if 0 < ks[b] < V else V
        x, place, share = x[:n], place[:n], share[:n]
        if ps[b] < 1:
            before = torch.cumsum(share, 0) - share
            few = int((before < ps[b] * share.sum()).sum())
            x, place, share = x[: max(1, few)], place[: max(1, few)], share[: max(1, few)]
        if ms[b] > 0:
            few = max(1, int((x - x[0] >= math.log(ms[b])).sum()))
            place, share = place[:few], share[:few]
        place, by = torch.sort(place)
        share = share[by] / share.sum()
        j = int((torch.cumsum(share, 0) <= us[r]).sum())
        prob[r] = share[min(j, share.numel() - 1)]
    return [None, prob]


def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, seed)
    if case["op"] == "sampling":
        if case["bs"] * case["per"] > 4096:
            return None
        return _exact_sampling(case, seed)
    return None
