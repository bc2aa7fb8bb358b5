"""Plain float64 references of the verifying operators (page extension, tree attention,
filtered sampling), written from their definitions with Python loops and NumPy."""

import numpy as np


def extend_pages(req, lens, new, held, P, table, free, head, num_pages, max_tokens):
    """(table, head, held_out, cu, slots, positions, owner, served) as Python walks the requests."""
    table = table.copy()
    rows, stride = table.shape
    cu, slots, positions, owner, held_out, served = [0], [], [], [], [], []
    want, first_of = 0, {}
    taken = 0
    for b in range(len(req)):
        h = int(held[b]) if held is not None else -(-int(lens[b]) // P)
        add = max(0, int(new[b]))
        cu.append(cu[-1] + add)
        end = -(-(int(lens[b]) + add) // P)
        ok = new[b] >= 0 and lens[b] >= 0 and 0 <= req[b] < rows and h * P >= lens[b]
        ok = ok and first_of.setdefault(int(req[b]), b) == b
        ok = ok and max(end, h) <= stride and not (add > 0 and cu[-1] > max_tokens)
        need = max(0, end - h) if ok else 0
        first, want = want, want + need
        if need and head + want > len(free):
            ok = False
        if ok and need:
            taken = want
            for i in range(need):
                page = int(free[head + first + i])
                if 0 <= page < num_pages:
                    table[req[b], h + i] = page
        held_out.append(h + (need if ok else 0))
        served.append(ok)
        for t in range(add):
            pos = int(lens[b]) + t
            slot = -1
            if ok:
                c = pos // P
                page = int(free[head + first + c - h]) if c >= h else int(table[req[b], c])
                slot = page * P + pos % P if 0 <= page < num_pages else -1
            slots.append(slot)
            positions.append(pos)
            owner.append(b)
    return table, head + taken, held_out, cu, slots, positions, owner, served


def parents_of(ids, width):
    """Parent of each node 0.., -1 for the root and for ids that name no earlier node."""
    if ids is None:
        return [-1] + list(range(width - 1))
    out = [-1]
    for i, x in enumerate(ids, 1):
        p = int(x) // width
        out.append(p if x >= 0 and p < i and int(x) % width == i else -1)
    return out


def tree_attention(q, keys, values, pages, ctx, n, parent, scale):
    """One request: q (n, heads, hd), keys/values (pages, kv, P, hd) float64, `pages` the table
    row. Returns (out, A) with A = sum_j p_j |v_j|, and the largest scale * sum |q_d k_d|."""
    heads, hd = q.shape[1:]
    kv, P = keys.shape[1:3]
    group = heads // kv
    total = ctx + n
    k = np.zeros((kv, total, hd))
    v = np.zeros((kv, total, hd))
    there = np.zeros(total, dtype=bool)
    for c in range(-(-total // P)):
        p1 = min(total, (c + 1) * P)
        if c < len(pages) and 0 <= pages[c] < keys.shape[0]:
            k[:, c * P:p1] = keys[pages[c], :, : p1 - c * P]
            v[:, c * P:p1] = values[pages[c], :, : p1 - c * P]
            there[c * P:p1] = True
    see = np.zeros((n, total), dtype=bool)
    for i in range(n):
        see[i, :ctx] = True
        j = i
        while j >= 0:
            see[i, ctx + j] = True
            j = parent[j]
    see &= there
    out, mag, big = np.zeros_like(q), np.zeros_like(q), 0.0
    for h in range(heads):
        s = scale * q[:, h] @ k[h // group].T
        big = max(big, float((abs(scale) * np.abs(q[:, h]) @ np.abs(k[h // group]).T)[see].max(initial=0.0)))
        s = np.where(see, s, -np.inf)
        m = s.max(axis=1, keepdims=True)
        e = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
        l = e.sum(axis=1, keepdims=True)
        p = e / np.where(l > 0, l, 1.0)
        out[:, h] = p @ v[h // group]
        mag[:, h] = p @ np.abs(v[h // group])
    return out, mag, big


def sample_filtered(logits, temp, k, top_p, min_p, u):
    """One row: (index, probability, margin): margin is how near, relative to the mass, the
    nearest border came that decided which entries are kept or drawn."""
    l = np.asarray(logits, dtype=np.float64) + 0.0
    V = len(l)
    good = l > -np.inf
    if not good.any():
        return 0, 0.0, 1.0
    order = np.lexsort((np.arange(V), -np.where(good, l, -np.inf)))[: int(good.sum())]
    if not temp > 0:
        return int(order[0]), 1.0, 1.0
    top = l[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(l[order] == top, 1.0, np.exp((l[order] - top) / np.float64(temp)))
    w = np.where(w < 2.0 ** -45, 0.0, w)  # weights are multiples of 2^-44: less than half of one is nothing
    margin, even = 1.0, bool((w == 1.0).all())
    if 0 < k < V:
        order, w = order[:k], w[:k]
    if top_p < 1:
        before = np.cumsum(w) - w
        want = max(top_p, 0.0) * w.sum()
        if top_p > 0:
            margin = min(margin, float(np.abs(before - want)[1:].min(initial=np.inf) / w.sum()))
        n = max(1, int((before < want).sum()))
        order, w = order[:n], w[:n]
    if min_p > 0:
        margin = min(margin, float(np.abs(w - min(min_p, 1.0))[1:].min(initial=np.inf))) if min_p < 1 else margin
        keep = w >= min(min_p, 1.0)
        order, w = order[keep], w[keep]
    by = np.argsort(order)
    order, w = order[by], w[by]
    mass = np.cumsum(w)
    at = min(max(u, 0.0), np.float64(np.float32(1) - np.float32(2) ** -24)) if u == u else 0.0
    if at > 0:
        margin = min(margin, float(np.abs(mass - at * mass[-1])[w > 0].min() / mass[-1]))
    j = int((mass <= at * mass[-1]).sum())
    # equal logits: every weight is exactly 1 on both sides, so no border is uncertain
    return int(order[j]), float(w[j] / mass[-1]), 1.0 if even else margin
