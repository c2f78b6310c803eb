"""Transformer layers on packed weights: a chunk of a prompt, then decode steps.

Each layer's products (q/k/v, o, gate/up, down) run on MLX affine 4-bit weights of
Qwen3-0.6B's layer shapes (synthetic, seeded); between q/k/v and o the layer norms and rotates the
query heads (head_norm_rope), stores keys and values in a paged cache
(cache_append, keys normed and rotated on the way) and attends over it
(cache_attend). Sequences of different lengths share the calls: their prompts as
ragged chunks, then one new token of each per step, the step replayed as a CUDA
graph. What a sequence's last prompt token gave is computed again as a decode step
over the same cache and compared.

    python examples/decode_layers.py [--layers 4] [--prompts 300,57,1024] [--steps 32] [--codes]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import packed_qmatmul_gb300 as qm  # noqa: E402
from packed_qmatmul_gb300 import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, INNER = 1024, 16, 8, 128, 3072
EPS, THETA = 1e-6, 1e6


def weight(g, n, k):
    w = qm.QWeight.from_arrays(synth.affine_weight(g, n, k, bits=4, group_size=64, scale_sigma=0.005), flags=qm.QM_WEIGHT_STATIC)
    return w


def rms_norm(x, w):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()).to(x.dtype)


class Layer:
    def __init__(self, g, pages, page, codes):
        self.q, self.k, self.v = weight(g, HEADS * DIM, HIDDEN), weight(g, KV_HEADS * DIM, HIDDEN), weight(g, KV_HEADS * DIM, HIDDEN)
        self.o = weight(g, HIDDEN, HEADS * DIM)
        self.gate, self.up, self.down = weight(g, INNER, HIDDEN), weight(g, INNER, HIDDEN), weight(g, HIDDEN, INNER)
        ones = dict(dtype=torch.bfloat16, device="cuda")
        self.norm1, self.norm2 = torch.ones(HIDDEN, **ones), torch.ones(HIDDEN, **ones)
        self.q_norm, self.k_norm = torch.ones(DIM, **ones), torch.ones(DIM, **ones)
        shape = (pages, KV_HEADS, page, DIM)
        if codes:
            k, v = (torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2))
            self.cache = qm.Cache(k, v, *(torch.zeros(shape[:3], device="cuda") for _ in range(2)))
        else:
            self.cache = qm.Cache(*(torch.zeros(shape, **ones) for _ in range(2)))

    def attend(self, q, k, v, batch, positions, rope):
        """q, k, v as the products leave them -> the attention's rows, ready for the o product."""
        T = q.shape[0]
        (q,) = qm.head_norm_rope([q.view(T, HEADS, DIM)], positions, rope, weights=[self.q_norm], eps=EPS)
        qm.cache_append(self.cache, batch, k.view(T, KV_HEADS, DIM), v.view(T, KV_HEADS, DIM), rope, k_weight=self.k_norm, eps=EPS)
        return qm.cache_attend(self.cache, batch, q).view(T, HEADS * DIM)

    def forward(self, x, batch, positions, rope):
        q, k, v = qm.apply_many([self.q, self.k, self.v], rms_norm(x, self.norm1))
        x = x + qm.apply(self.o, self.attend(q, k, v, batch, positions, rope))
        gate, up = qm.apply_many([self.gate, self.up], rms_norm(x, self.norm2))
        return x + qm.apply(self.down, torch.nn.functional.silu(gate) * up)


def rope_table(rows):
    half = DIM // 2
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return qm.Rope(torch.cat([angle.cos(), angle.sin()], 1).float())


class Stack:
    """Layers, their caches and the page table of a set of sequences with room for `room` tokens each."""

    def __init__(self, layers, seqs, room, page=64, codes=False, seed=0):
        g = synth.rng(seed)
        self.seqs, self.page = seqs, page
        width = -(-room // page)
        gen = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(seqs * width, generator=gen).view(seqs, width).to(torch.int32).cuda()
        self.layers = [Layer(g, seqs * width, page, codes) for _ in range(layers)]
        self.rope = rope_table(room)

    def chunk(self, x, news, lens):
        """Hidden rows x of news[i] new tokens of each sequence, which then has lens[i] tokens."""
        offsets, positions = [0], []
        for new, n in zip(news, lens):
            offsets.append(offsets[-1] + new)
            positions += range(n - new, n)
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = qm.Batch(torch.tensor(lens, **i32), self.table, torch.tensor(offsets, **i32), tokens=offsets[-1], max_new=max(news))
        return self.run(x, batch, torch.tensor(positions, **i32))

    def run(self, x, batch, positions):
        for layer in self.layers:
            x = layer.forward(x, batch, positions, self.rope)
        return x


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompts", default="300,57,1024")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--codes", action="store_true", help="8-bit codes in the cache")
    a = ap.parse_args()
    lens = [int(n) for n in a.prompts.split(",")]
    seqs = len(lens)
    stack = Stack(a.layers, seqs, max(lens) + a.steps + 1, codes=a.codes)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(lens), HIDDEN, generator=gen, device="cuda").to(torch.bfloat16)
    out = stack.chunk(x, lens, lens)
    ends = torch.tensor(lens, device="cuda").cumsum(0) - 1
    again = stack.chunk(x[ends], [1] * seqs, lens)  # the last prompt tokens once more, one each
    diff = (again.float() - out[ends].float()).norm() / out[ends].float().norm()
    print(f"prompts of {lens}: the last tokens again as a decode step differ by {diff:.2e} of their norm")

    # decode steps: the tensors a step reads are updated in place, so that it can be replayed
    i32 = dict(dtype=torch.int32, device="cuda")
    held = torch.tensor(lens, **i32)
    positions = held.clone()
    batch = qm.Batch(held, stack.table, max_new=1)
    row = out[ends].clone()

    def step():
        positions.copy_(held)
        held.add_(1)
        row.copy_(stack.run(row, batch, positions))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps - 1):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    qm.qm_device_status()
    ms = start.elapsed_time(end) / max(a.steps - 1, 1)
    print(f"{a.steps - 1} decode steps of {seqs} sequences through {a.layers} layers: {ms * 1e3:.1f} us a step, lengths now {held.tolist()}, "
          f"finite: {bool(torch.isfinite(row).all())}")


if __name__ == "__main__":
    main()
