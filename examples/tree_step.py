"""Speculative decoding with trees of drafted tokens over a paged cache of 8-bit
values, through the library's own operators: each step plans the trees (masks and
positions), rotates queries and keys and writes keys and values as e4m3 codes,
attends under the masks, runs the MoE and output layers, takes the largest logits
of every node, and keeps the longest path on which each drafted token is what its
parent's logits say: its keys and values are read back and written to the
consecutive places.

    python examples/tree_step.py [--steps N]

The model is the random one of decode_step.py with a small vocabulary, the drafter
a fixed table of two guesses for each token. A step is captured once in a CUDA
graph and replayed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import decode_step as base  # noqa: E402
from moe_decode_gb300 import api, synth  # noqa: E402

HEADS, KV_HEADS, HEAD_DIM, PAGE, HIDDEN = base.HEADS, base.KV_HEADS, base.HEAD_DIM, base.PAGE, base.SHAPE.hidden
VOCAB, REQUESTS = 24, 2
# The tree of each request: the last accepted token, two guesses of the next one,
# two of what follows each, and one more level.
PARENTS = [-1, 0, 0, 1, 1, 2, 2, 3]
NODES = len(PARENTS)
T = REQUESTS * NODES


class TreeDecoder:
    def __init__(self, max_context: int):
        width = -(-(max_context + NODES) // PAGE)
        self.layers = [base.Layer(i, 1) for i in range(base.LAYERS)]
        self.caches = [api.KvCache8.empty(REQUESTS * width, PAGE, KV_HEADS, HEAD_DIM) for _ in self.layers]
        self.angles = api.Rope(HEAD_DIM, base=10000.0)

        def ints(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        self.embed = synth.normal_bf16(78, 1, 0, VOCAB * HIDDEN, 1.0, "cuda").view(VOCAB, HIDDEN)
        self.head = synth.normal_bf16(78, 2, 0, VOCAB * HIDDEN, 0.1, "cuda").view(VOCAB, HIDDEN)
        self.guesses = torch.randint(0, VOCAB, (VOCAB, 2), device="cuda")
        # every request holds its pages from the start
        self.tables = torch.randperm(REQUESTS * width, device="cuda").int().view(REQUESTS, width)
        self.parents = torch.tensor(PARENTS * REQUESTS, dtype=torch.int32, device="cuda")
        self.up = self.parents.view(REQUESTS, NODES).long().clamp_min(0)
        self.q_start = torch.arange(0, T + 1, NODES, device="cuda").int()
        self.ctx, self.seq = ints(REQUESTS), ints(REQUESTS)
        self.root = torch.arange(REQUESTS, device="cuda")  # the last accepted tokens
        self.tokens, self.next, self.positions = ints(REQUESTS, NODES, dtype=torch.int64), ints(T), ints(T)
        self.masks = ints(T, dtype=torch.int64)
        self.slots, self.path_slots, self.kept_slots = ints(T), ints(T), ints(T)
        self.accepted = ints(REQUESTS)
        self.x = torch.empty((T, HIDDEN), dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty_like(self.x)
        self.q, self.attended = (torch.empty((T, HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.moved = torch.empty((2, T, KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        self.logits, self.u, self.greedy = (torch.zeros(s, device="cuda") for s in ((T, VOCAB), T, T))
        self.ws = api.paged_workspace(HEADS, self.caches[0])
        self.ws_moe = api.workspace(self.layers[0].shape, T)
        self.ws_head = torch.zeros(api.LM_HEAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def draft(self):
        """The tree's tokens: a node's children are the guesses for it."""
        self.tokens[:, 0] = self.root
        for i in range(1, NODES):
            first = PARENTS.index(PARENTS[i])
            self.tokens[:, i] = self.guesses[self.tokens[:, PARENTS[i]], i - first]

    def verify(self):
        """One forward pass of all nodes: self.next is what each node's logits say."""
        self.seq.copy_(self.ctx + NODES)
        place = self.ctx[:, None] + torch.arange(NODES, device="cuda")
        self.slots.copy_((self.tables.gather(1, (place // PAGE).long()) * PAGE + place % PAGE).view(-1))
        api.tree_plan(self.parents, self.q_start, self.seq, self.masks, self.positions, self.ws)
        self.x.copy_(self.embed[self.tokens.view(-1)])
        for layer, cache in zip(self.layers, self.caches):
            qkv = (base.rms_norm(self.x, layer.gain) @ layer.qkv.T).view(T, -1, HEAD_DIM)
            q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
            api.paged_rope_append(q, k, v, self.positions, self.slots, self.angles, cache, self.ws, q_out=self.q)
            api.paged_attention(self.q, cache, self.tables, self.q_start, self.seq, self.attended, self.ws, tree_masks=self.masks)
            self.x += self.attended.view(T, -1) @ layer.o.T
            api.decode_layer(self.x, layer.router, layer.experts, layer.shape, self.y, self.ws_moe)
            self.x.copy_(self.y)
        api.lm_head(base.rms_norm(self.x, self.layers[0].gain), self.head, VOCAB, HIDDEN, self.logits, self.ws_head)
        api.sample(self.logits, self.u, self.next, temperature=self.greedy)

    def choose(self):
        """The deepest node all of whose path was drafted rightly, and the slots of that path."""
        node = torch.arange(NODES, device="cuda")
        right = (self.tokens == self.next.view(REQUESTS, NODES).long().gather(1, self.up)) | (node == 0)
        masks = self.masks.view(REQUESTS, NODES)
        bits = (masks[:, :, None] >> node) & 1  # [request, node, node on its path]
        good = ((bits == 0) | right[:, None, :]).all(-1)
        depth = torch.where(good, bits.sum(-1), 0)
        best = depth.argmax(1, keepdim=True)
        path = bits.gather(1, best[:, :, None].expand(-1, -1, NODES))[:, 0]
        count = path.sum(1, keepdim=True)
        order = torch.where(path == 1, node, NODES + node).argsort(1)  # the path's nodes first, in order
        slots = self.slots.view(REQUESTS, NODES)
        held = node < count
        self.path_slots.copy_(torch.where(held, slots.gather(1, order), -1).view(-1))
        self.kept_slots.copy_(torch.where(held, slots, -1).view(-1))
        self.accepted.copy_(count[:, 0])
        self.root.copy_(self.next.view(REQUESTS, NODES).gather(1, best)[:, 0])

    def keep(self):
        """The path's keys and values to the consecutive places (all are read before any is written)."""
        for cache in self.caches:
            api.paged_read(cache, self.path_slots, self.moved[0], self.moved[1], self.ws)
            api.paged_append(self.moved[0], self.moved[1], self.kept_slots, cache, self.ws)
        self.ctx += self.accepted

    def step(self):
        self.draft()
        self.verify()
        self.choose()
        self.keep()

    def check(self):
        for ws in (self.ws, self.ws_moe, self.ws_head):
            status = api.read_status(ws)
            if status != 0:
                raise RuntimeError(f"device status {status}: {api.status_str(status)}")


def generate(steps: int, seed: int = 0, graph: bool = True):
    """Accepted tokens of each request (the last of each step is what the deepest node says), and the decoder."""
    torch.manual_seed(seed)
    dec = TreeDecoder(steps * NODES)
    dec.step()  # (what libraries set up at their first call is not captured)
    dec.ctx.zero_()
    dec.root.copy_(torch.arange(REQUESTS))
    captured = None
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            dec.step()
    out = [[int(t)] for t in dec.root]
    for _ in range(steps):
        captured.replay() if graph else dec.step()
        counts, places, slots, tokens, root = (x.tolist() for x in (dec.accepted, dec.path_slots.view(REQUESTS, NODES),
                                                                    dec.slots.view(REQUESTS, NODES), dec.tokens, dec.root))
        for b in range(REQUESTS):
            out[b] += [tokens[b][slots[b].index(places[b][i])] for i in range(1, counts[b])] + [root[b]]
    dec.check()
    return out, dec


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args()
    tokens, dec = generate(args.steps)
    for b in range(REQUESTS):
        print(f"request {b}: {len(tokens[b]) - 1} tokens in {args.steps} steps:", *tokens[b])
    print("context lengths", dec.ctx.tolist())


if __name__ == "__main__":
    main()
