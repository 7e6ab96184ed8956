"""examples/decode_step.py: the paged step's operators next to the MoE layer
and the output layer, eager and as a replayed graph."""
import importlib.util
import os

import pytest
import torch

from paged_util import attention, check_attention

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROMPTS = [[(11 * i + b) % 2000 for i in range(n)] for b, n in enumerate((20, 3, 33))]


@pytest.fixture(scope="module")
def step():
    from moe_decode_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_graph_and_eager_steps_give_the_same_tokens(step):
    a, dec = step.generate(PROMPTS, 25, seed=3)
    b, _ = step.generate(PROMPTS, 25, seed=3, graph=False)
    assert torch.equal(a, b)
    assert ((a >= 0) & (a < step.VOCAB)).all()
    lengths = [len(p) + 25 for p in PROMPTS]
    assert dec.ctx.tolist() == lengths
    assert dec.free_head.item() == sum(-(-n // step.PAGE) for n in lengths)


def test_the_last_layer_attends_over_what_the_steps_wrote(step):
    """The last decode step's attention against the formula on the cache, and
    the cache's blocks all different."""
    _, dec = step.generate(PROMPTS, 9, seed=4, graph=False)
    layer = dec.layers[-1]
    used = dec.tables[dec.tables >= 0]
    assert used.unique().numel() == used.numel() == dec.free_head.item()
    q = torch.randn((len(PROMPTS), step.HEADS, step.HEAD_DIM), device="cuda").bfloat16()
    out = torch.empty_like(q)
    starts = torch.arange(len(PROMPTS) + 1, device="cuda").int()
    step.api.paged_attention(q, layer.cache, dec.tables, starts, dec.ctx, out, dec.ws_attn)
    s = dict(q=q, k=layer.cache.k, v=layer.cache.v, table=dec.tables, lens=[(n, 1) for n in dec.ctx.tolist()], window=0)
    check_attention(out, None, attention(s))
