"""Prompts and decoding of a few requests through the library's own operators:
each step plans its places in the paged KV cache, writes the new keys and
values, attends over the cache, runs the MoE layer, and samples the next tokens
from the output layer's logits.

    python examples/decode_step.py [--steps N]

The model is random and tiny (hidden 256, 2 layers, 16 experts); only the four
projections around the attention are torch products. A decode step is captured
once in a CUDA graph and replayed: the lengths, block tables and tokens that it
reads and writes are device buffers, so nothing of it waits for the host.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_decode_gb300 import api, synth  # noqa: E402

SHAPE = synth.TINY
HEADS, KV_HEADS, HEAD_DIM, PAGE = 4, 2, 64, 16
VOCAB, LAYERS, MAX_TOKENS = 2000, 2, 16  # the MoE layer takes up to 16 tokens a call


def rms_norm(x, gain, eps=1e-6):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps) * gain.float()).to(x.dtype)


class Layer:
    def __init__(self, i: int, n_blocks: int):
        H, bf16 = SHAPE.hidden, torch.bfloat16

        def weight(tid, rows, cols):
            return synth.normal_bf16(500 + i, tid, 0, rows * cols, 1 / math.sqrt(cols), "cuda").view(rows, cols)

        self.qkv = weight(1, (HEADS + 2 * KV_HEADS) * HEAD_DIM, H)
        self.o = weight(2, H, HEADS * HEAD_DIM)
        self.gain = torch.ones(H, dtype=bf16, device="cuda")
        w = synth.device_layer(SHAPE, i)
        self.router = w["Wg"]
        self.experts = api.ExpertWeights(*(w[n] for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2")))
        # the layer normalises its input and adds it to its output
        self.shape = api.make_shape(H, SHAPE.n_experts, SHAPE.top_k, SHAPE.inter, SHAPE.shared_inter,
                                    norm_weight=self.gain, residual=True)
        self.cache = api.KvCache(*(torch.zeros((n_blocks, PAGE, KV_HEADS, HEAD_DIM), dtype=bf16, device="cuda")
                                   for _ in range(2)))


class Decoder:
    """Up to `requests` requests side by side; a step takes up to 16 tokens."""

    def __init__(self, requests: int, max_context: int):
        width = -(-max_context // PAGE)
        self.n_blocks = requests * width
        self.layers = [Layer(i, self.n_blocks) for i in range(LAYERS)]
        self.embed = synth.normal_bf16(77, 1, 0, VOCAB * SHAPE.hidden, 1.0, "cuda").view(VOCAB, SHAPE.hidden)
        self.head = synth.normal_bf16(77, 2, 0, VOCAB * SHAPE.hidden, 0.1, "cuda").view(VOCAB, SHAPE.hidden)

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device="cuda")

        # what outlives a step, on the device
        self.ctx, self.tables = ints(requests), ints(requests, width, fill=-1)
        self.free, self.free_head = torch.randperm(self.n_blocks, device="cuda").int(), ints(1)
        # a step's buffers
        self.new, self.q_start, self.seq, self.taken = ints(requests), ints(requests + 1), ints(requests), ints(1)
        self.tokens, self.slots = ints(MAX_TOKENS), ints(MAX_TOKENS)
        self.x = torch.empty((MAX_TOKENS, SHAPE.hidden), dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty_like(self.x)
        self.attended = torch.empty((MAX_TOKENS, HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        self.last = torch.zeros((requests, SHAPE.hidden), dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty((requests, VOCAB), device="cuda")
        self.next, self.probs = ints(requests), torch.empty(requests, device="cuda")
        self.u = torch.empty(requests, device="cuda")
        self.sampling = dict(temperature=torch.full((requests,), 0.8, device="cuda"), top_k=ints(requests, fill=50),
                             top_p=torch.full((requests,), 0.95, device="cuda"))
        self.ws_plan = api.paged_workspace()
        self.ws_attn = api.paged_workspace(HEADS, self.layers[0].cache)
        self.ws_moe = api.workspace(self.layers[0].shape, MAX_TOKENS)
        self.ws_head = torch.zeros(api.LM_HEAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def forward(self):
        """One step on the buffers: the new tokens of all requests, packed."""
        api.paged_plan(self.ctx, self.new, self.free, self.tables, PAGE, self.q_start, self.seq, self.slots, self.taken,
                       self.ws_plan, free_head=self.free_head)
        self.x.copy_(self.embed[self.tokens.long()])
        for layer in self.layers:
            qkv = (rms_norm(self.x, layer.gain) @ layer.qkv.T).view(MAX_TOKENS, -1, HEAD_DIM)
            q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
            api.paged_append(k, v, self.slots, layer.cache, self.ws_plan)
            api.paged_attention(q, layer.cache, self.tables, self.q_start, self.seq, self.attended, self.ws_attn)
            self.x += self.attended.view(MAX_TOKENS, -1) @ layer.o.T
            api.decode_layer(self.x, layer.router, layer.experts, layer.shape, self.y, self.ws_moe)
            self.x.copy_(self.y)
        # the last token of each request gives its next one
        self.last.copy_(rms_norm(self.x, self.layers[0].gain)[(self.q_start[1:].long() - 1).clamp_min(0)])
        api.lm_head(self.last, self.head, VOCAB, SHAPE.hidden, self.logits, self.ws_head)
        api.sample(self.logits, self.u, self.next, probs=self.probs, **self.sampling)
        # the state of the next step
        self.ctx.copy_(self.seq)
        self.free_head += self.taken

    def decode_inputs(self):
        """Each request's next token is the next step's only one of it."""
        self.tokens.zero_()
        self.tokens[: self.next.numel()].copy_(self.next)
        self.new.fill_(1)

    def prompts(self, prompts):
        """Takes the prompts in steps of up to 16 tokens, request by request."""
        for b, prompt in enumerate(prompts):
            for i in range(0, len(prompt), MAX_TOKENS):
                part = prompt[i:i + MAX_TOKENS]
                self.tokens.zero_()
                self.tokens[: len(part)] = torch.tensor(part, dtype=torch.int32)
                self.new.zero_()
                self.new[b] = len(part)
                keep = self.next.clone()
                self.u.uniform_()
                self.forward()
                if b:  # the requests before keep their tokens
                    self.next[:b] = keep[:b]

    def capture(self) -> torch.cuda.CUDAGraph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.decode_inputs()
            self.forward()
        return graph

    def check(self):
        for ws in (self.ws_plan, self.ws_attn, self.ws_moe, self.ws_head):
            status = api.read_status(ws)
            if status != 0:
                raise RuntimeError(f"device status {status}: {api.status_str(status)}")


def generate(prompts, steps: int, seed: int = 0, graph: bool = True):
    """The sampled tokens [steps, requests], and the decoder."""
    torch.manual_seed(seed)
    dec = Decoder(len(prompts), max(map(len, prompts)) + steps + 1)
    dec.prompts(prompts)
    captured = dec.capture() if graph else None
    out = []
    for _ in range(steps):
        out.append(dec.next.clone())
        dec.u.uniform_()
        if captured is not None:
            captured.replay()
        else:
            dec.decode_inputs()
            dec.forward()
    dec.check()
    return torch.stack(out).cpu(), dec


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args()
    prompts = [[(7 * i + 3 * b) % VOCAB for i in range(n)] for b, n in enumerate((37, 5, 16, 90))]
    tokens, dec = generate(prompts, args.steps)
    for b in range(len(prompts)):
        print(f"request {b}: {len(prompts[b])} prompt tokens, then", *tokens[:, b].tolist())
    print("context lengths", dec.ctx.tolist(), "blocks taken", dec.free_head.item(), "of", dec.n_blocks)


if __name__ == "__main__":
    main()
