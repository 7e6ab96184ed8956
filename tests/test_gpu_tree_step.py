"""examples/tree_step.py: trees, rotation, the cache of 8-bit values and reading
back, together with the MoE and output layers, eager and as a replayed graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from cache8_util import by_slot, check_attention8, dequantise
from tree_util import attention

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tree():
    from moe_decode_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("tree_step", os.path.join(ROOT, "examples", "tree_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_graph_and_eager_steps_give_the_same_tokens(tree):
    a, dec = tree.generate(30, seed=5)
    b, _ = tree.generate(30, seed=5, graph=False)
    assert a == b
    assert dec.ctx.tolist() == [len(t) - 1 for t in a]
    assert all(31 <= len(t) <= 31 + 3 * 30 and max(t) < tree.VOCAB for t in a)
    # with 24 tokens and two guesses some are right, and some are not
    assert any(len(t) > 31 for t in a) and any(len(t) < 31 + 3 * 30 for t in a)


def test_a_step_piece_by_piece(tree):
    """The last layer's attention against the formula on what the cache holds,
    the choice against a walk down the tree, and the kept path in its places."""
    _, dec = tree.generate(6, seed=6, graph=False)
    api, N = tree.api, tree.NODES
    dec.draft()
    dec.verify()
    cache = dec.caches[-1]
    k, v = (torch.from_numpy(dequantise(*x)).cuda().view(cache.k.shape) for x in by_slot(cache))
    s = dict(q=dec.q, k=k, v=v, table=dec.tables, lens=[(n, N) for n in dec.seq.tolist()], window=0)
    masks = dec.masks.tolist()
    check_attention8(dec.attended, None, attention(s, masks), int(dec.seq.max()))
    # depth of each node, from the fixed tree
    depth = []
    for i, p in enumerate(tree.PARENTS):
        depth.append(0 if p < 0 else depth[p] + 1)
    assert dec.positions.tolist() == [c + d for c in dec.ctx.tolist() for d in depth]
    # make a path right by hand: what the logits say becomes the drafted token
    dec.tokens[0, 2] = dec.next[0]
    dec.tokens[0, 6] = dec.next[2]
    dec.tokens[0, 5] = dec.next[2] + 1
    dec.tokens[0, 1] = dec.next[0] + 1
    ctx, slots = dec.ctx.clone(), dec.slots.tolist()
    before = [by_slot(c) for c in dec.caches]
    dec.choose()
    assert dec.accepted[0] == 3 and dec.root[0] == dec.next[6]
    assert dec.path_slots[:N].tolist() == [slots[0], slots[2], slots[6]] + [-1] * 5
    dec.keep()
    for c, was in zip(dec.caches, before):
        for (codes, byte), (codes0, byte0) in zip(by_slot(c), was):
            got = dequantise(codes[slots[:3]], byte[slots[:3]])
            want = dequantise(codes0[[slots[0], slots[2], slots[6]]], byte0[[slots[0], slots[2], slots[6]]])
            assert np.array_equal(got, want)
    assert dec.ctx[0] == ctx[0] + 3
    dec.check()
