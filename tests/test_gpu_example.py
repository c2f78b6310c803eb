"""The layers of examples/decode_layers.py against the same layers in plain float32
torch: a ragged prompt in two chunks, then a decode step."""
import os
import sys

import pytest
import torch

import packed_qmatmul_gb300 as qm

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain_layer(layer, x, past, rope, table):
    """One sequence through a layer in float32, with the roundings to bfloat16 that the calls make
    between them; past: the keys and values so far."""
    from decode_layers import DIM, EPS, HEADS, KV_HEADS, rms_norm

    def rounded(t):
        return t.to(torch.bfloat16).float()

    def product(w, t):
        return rounded(t.float() @ qm.dequant(w, torch.float32).T)

    def heads(t, n, w, at):
        t = t.view(-1, n, DIM)
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w.float()
        c, s = table[at, None, : DIM // 2], table[at, None, DIM // 2:]
        a, b = t[..., : DIM // 2], t[..., DIM // 2:]
        return rounded(torch.cat([a * c - b * s, b * c + a * s], -1))

    h = rms_norm(x.to(torch.bfloat16), layer.norm1)
    at = torch.arange(past[0].shape[0], past[0].shape[0] + x.shape[0], device="cuda")
    q, k = heads(product(layer.q, h), HEADS, layer.q_norm, at), heads(product(layer.k, h), KV_HEADS, layer.k_norm, at)
    k, v = torch.cat([past[0], k]), torch.cat([past[1], product(layer.v, h).view(-1, KV_HEADS, DIM)])
    group = HEADS // KV_HEADS
    s = torch.einsum("thd,nhd->htn", q, k.repeat_interleave(group, 1)) * DIM ** -0.5
    s = s.masked_fill(torch.arange(k.shape[0], device="cuda")[None, None] > at[None, :, None], -torch.inf)
    o = rounded(torch.einsum("htn,nhd->thd", torch.softmax(s, -1), v.repeat_interleave(group, 1)).flatten(1))
    x = rounded(x + product(layer.o, o))
    h = rms_norm(x.to(torch.bfloat16), layer.norm2)
    inner = rounded(rounded(torch.nn.functional.silu(product(layer.gate, h))) * product(layer.up, h))
    return rounded(x + product(layer.down, inner)), (k, v)


@pytest.mark.parametrize("codes", [False, True])
def test_layers_with_a_paged_cache(codes):
    from decode_layers import HIDDEN, KV_HEADS, DIM, Stack
    from packed_qmatmul_gb300 import build

    build.build()
    torch.cuda.set_device(0)
    news = ([70, 3], [33, 1], [1, 1])  # two chunks of each prompt, then a decode step
    stack = Stack(2, 2, 128, page=16, codes=codes)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = [[torch.randn(n, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16) for n in step] for step in news]
    lens, got = [0, 0], []
    for step, rows in zip(news, x):
        lens = [n + new for n, new in zip(lens, step)]
        got.append(stack.chunk(torch.cat(rows), step, lens).float().split(step))
    qm.qm_device_status()
    for i in range(2):
        empty = torch.zeros(0, KV_HEADS, DIM, device="cuda")
        past = [(empty, empty) for _ in stack.layers]
        for step in range(3):
            want = x[step][i].float()
            for j, layer in enumerate(stack.layers):
                want, past[j] = plain_layer(layer, want, past[j], stack.rope, stack.rope.table)
            # every rounding to bfloat16 in between (a relative 2^-9 each, some ten of them a layer, adding
            # up as their root) and, with codes, the cache's own 1/254 of each head's largest element
            off = (got[step][i] - want).norm() / want.norm()
            assert off < (0.02 if codes else 0.01), (i, step, float(off))
