"""The verifying operators on the host: refused arguments (before any device work) and the
references' own pins."""

import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_block_context_gb300 import _lib as F

from . import verify_ref as ref


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_block_context_gb300 import build

    build.build()
    return F.lib()


A = 4096  # a pointer that is never followed: these calls are refused


def pages_args(**change):
    d = dict(bs=2, req=A, lens=A, new=A, held=A, P=16, table=A, rows=3, stride=4, free=A, num_free=5, head=A,
             head_out=A + 64, held_out=A + 128, pages=9, most=20, cu=A, slots=A, pos=None, own=None, err=None, stream=None)
    d.update(change)
    return list(d.values())


@pytest.mark.parametrize("change,status", [
    (dict(req=None), 1), (dict(lens=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(head=None), 1),
    (dict(head_out=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(free=None), 1), (dict(bs=0), 1),
    (dict(P=0), 1), (dict(rows=-1), 1), (dict(stride=0), 1), (dict(pages=0), 1), (dict(most=-1), 1),
    (dict(num_free=-1), 1), (dict(bs=8193), 2), (dict(rows=32769), 2), (dict(head_out=A), 1), (dict(held_out=A), 1)])
def test_extend_pages_refuses(lib, change, status):
    assert lib.flashmap_extend_pages(*pages_args(**change)) == status
    assert F.flashmap_last_error()


def layer(**change):
    d = dict(keys=A, values=A, num_pages=8, num_kv_heads=2, page_size=16, head_dim=64, dtype=F.BF16)
    d.update(change)
    return F.flashmap_cache_layer(**d)


def attention_args(layer_, **change):
    d = dict(cache=ctypes.byref(layer_), q=A, q_stride=8 * 64, bs=1, width=4, heads=8, ctx=A, nodes=None, ids=A, req=A,
             table=A, rows=1, stride=4, scale=0.1, out=A, ws=A, ws_bytes=1 << 40, err=None, stream=None)
    d.update(change)
    return list(d.values())


@pytest.mark.parametrize("change,status", [
    (dict(num_pages=0), 1), (dict(num_kv_heads=0), 1), (dict(num_kv_heads=3), 1), (dict(page_size=24), 2),
    (dict(page_size=0), 1), (dict(head_dim=48), 2), (dict(head_dim=256), 2), (dict(dtype=F.E4M3), 2), (dict(dtype=7), 1),
    (dict(keys=None), 1), (dict(values=None), 1), (dict(keys=A + 8), 1), (dict(values=A + 2), 1),
    (dict(num_pages=1 << 27), 2)])
def test_tree_attention_refuses_caches(lib, change, status):
    assert lib.flashmap_tree_attention(*attention_args(layer(**change))) == status
    assert F.flashmap_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(cache=None), 1), (dict(q=None), 1), (dict(ctx=None), 1), (dict(req=None), 1), (dict(table=None), 1),
    (dict(out=None), 1), (dict(bs=0), 1), (dict(width=0), 1), (dict(width=1026), 2), (dict(heads=0), 1),
    (dict(heads=7), 1), (dict(q=A + 2), 1), (dict(out=A + 8), 1), (dict(q_stride=8 * 64 - 8), 1),
    (dict(q_stride=8 * 64 + 4), 1), (dict(rows=0), 1), (dict(stride=0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(bs=1 << 21), 2)])
def test_tree_attention_refuses(lib, change, status):
    assert lib.flashmap_tree_attention(*attention_args(layer(), **change)) == status
    assert F.flashmap_last_error()


def test_tree_attention_workspace_refuses(lib):
    n = ctypes.c_size_t()
    assert lib.flashmap_tree_attention_workspace(None, 1, 1, 1, ctypes.byref(n)) == 1
    assert lib.flashmap_tree_attention_workspace(ctypes.byref(layer()), 1, 1, 8, None) == 1
    assert lib.flashmap_tree_attention_workspace(ctypes.byref(layer(head_dim=16)), 1, 1, 8, ctypes.byref(n)) == 2


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(temp=None), 1), (dict(u=None), 1), (dict(tokens=None), 1), (dict(dtype=F.E4M3), 1),
    (dict(rows=0), 1), (dict(vocab=0), 1), (dict(per=0), 1), (dict(ld=9), 1), (dict(vocab=393217, ld=393217), 2), (dict(rows=(1 << 27) + 1), 2),
    (dict(logits=A + 1), 1)])
def test_sample_filtered_refuses(lib, change, status):
    d = dict(logits=A, dtype=F.F32, rows=2, vocab=10, ld=10, per=1, temp=A, k=None, p=None, mp=None, u=A, ids=None,
             tokens=A, probs=None, stream=None)
    d.update(change)
    assert lib.flashmap_sample_filtered(*d.values()) == status
    assert F.flashmap_last_error()


def test_binding_refuses_other_tensors(lib):
    """Wrong types, strides and places are refused by the binding before the library sees a pointer."""
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        F.flashmap_extend_pages(x, x, x, x, 16, x.view(2, 2), x, x, x, x, 4, x, x.long())
    with pytest.raises(ValueError):
        F.make_cache_layer(torch.zeros(1, 1, 16, 64, dtype=torch.float16), torch.zeros(1, 1, 16, 64))
    with pytest.raises(ValueError):
        F.flashmap_sample_filtered(torch.zeros(2, 8), 1, x, None, None, None, x, None, x)


# ------------------------------------------------------------------ the references


def test_reference_attention_is_softmax_over_the_ancestors():
    g = np.random.default_rng(0)
    ctx, n, hd, P = 5, 4, 8, 4
    keys, values = g.normal(size=(3, 1, P, hd)), g.normal(size=(3, 1, P, hd))
    q = g.normal(size=(n, 2, hd))
    pages = [2, 0, 1]
    k = np.concatenate([keys[p, 0] for p in pages])
    v = np.concatenate([values[p, 0] for p in pages])
    parent = ref.parents_of([0 * 4 + 1, 0 * 4 + 2, 1 * 4 + 3], 4)
    assert parent == [-1, 0, 0, 1]
    sees = [[0], [0, 1], [0, 2], [0, 1, 3]]
    out, _, _ = ref.tree_attention(q, keys, values, pages, ctx, n, parent, 0.3)
    for i in range(n):
        at = list(range(ctx)) + [ctx + j for j in sees[i]]
        for h in range(2):
            e = [np.exp(0.3 * sum(q[i, h] * k[x])) for x in at]
            want = sum(a * v[x] for a, x in zip(e, at)) / sum(e)
            np.testing.assert_allclose(out[i, h], want, rtol=1e-12)


def test_reference_sampling_by_hand():
    """Weights 4, 2, 1, 1 at indices 1, 3, 0, 2 (logits log w, temperature 1)."""
    l = np.log([1.0, 4.0, 1.0, 2.0])
    draw = lambda k=0, p=1.0, mp=0.0, u=0.0: ref.sample_filtered(l, 1.0, k, p, mp, u)[:2]  # noqa: E731
    assert draw(u=0.1) == (0, 0.125) and draw(u=0.2) == (1, 0.5) and draw(u=0.7)[0] == 2 and draw(u=0.8)[0] == 3
    assert draw(k=3, u=0.1)[0] == 0 and draw(k=3, u=0.99)[0] == 3     # of the tied pair the lower index stays
    assert draw(k=2, u=0.5) == (1, 4 / 6) and draw(k=2, u=0.7)[0] == 3
    assert draw(p=0.49, u=0.99) == (1, 1.0) and draw(p=0.51, u=0.7)[0] == 3
    assert draw(k=2, p=0.6, u=0.99)[0] == 1                            # 4 of 6 already holds 0.6
    assert draw(mp=0.3, u=0.99)[0] == 3 and draw(mp=0.6, u=0.99)[0] == 1
    assert ref.sample_filtered(l, 0.0, 0, 1.0, 0.0, 0.9)[:2] == (1, 1.0)


def test_reference_pages_by_hand():
    table = np.array([[7, -1, -1], [3, 4, -1]])
    t, head, held, cu, slots, pos, own, ok = ref.extend_pages([1, 0], [5, 4], [2, 3], [2, 1], 4, table, [9, 8, 6], 1, 10, 9)
    assert t.tolist() == [[7, 8, -1], [3, 4, -1]] and head == 2 and held == [2, 2] and cu == [0, 2, 5]
    assert slots == [17, 18, 32, 33, 34] and pos == [5, 6, 4, 5, 6] and own == [0, 0, 1, 1, 1] and all(ok)
