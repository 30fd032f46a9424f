"""One decoder layer that checks trees of drafted tokens: rotary positions, attention over the whole context, paged beams.

A prompt is prefilled once, its row of the page table is forked to three beams that share its pages, and every beam then
takes some steps.  A step is one CUDA graph: pages for the drafts, the layer over all nodes of all trees at once, the accepted
path moved together behind the context, and the other drafts' pages back (resize -> rotate -> append -> attend -> MoE ->
compact -> resize).  Weights, tokens and which path is accepted are random: the program shows the calls in their order and
what the caller keeps.

    python examples/draft_tree.py [--prompt 200] [--steps 6]
"""
import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from bit_routed_expert_gb300 import (StepGraph, api, kv_append, kv_attend_tree, kv_compact, kv_fork, kv_resize,  # noqa: E402
                                     kv_rotate, moe_residual_norm, rope_turns, synth)
from sparse_layer import SparseLayer  # noqa: E402

PARENT = [-1, 0, 0, 1, 1, 2, 4, 6]   # a tree's nodes, each behind the node it continues


def path_to(node):
    """A node's ancestors and itself, from the root on."""
    return (path_to(PARENT[node]) if PARENT[node] >= 0 else []) + [node]


class TreeLayer(SparseLayer):
    """SparseLayer's weights with rotary positions and attention over the whole context.  Pages are given out as sequences
    grow: refs counts the entries of the table that name each page."""

    def __init__(self, dev, T_max: int, B: int, max_len: int):
        super().__init__(dev, T_max, B, max_len)
        self.table.fill_(-1)
        self.refs = torch.zeros(self.table.numel(), dtype=torch.int32, device=dev)
        self.turns, self.gain = rope_turns(self.DIM, device=dev)
        H, K, D = self.HEADS, self.KV_HEADS, self.DIM
        self.ws = torch.empty(api.kv_attend_tree_workspace(T_max, H, K, D), dtype=torch.uint8, device=dev)
        self.resize_ws = torch.empty(api.kv_resize_workspace(self.refs.numel(), *self.table.shape), dtype=torch.uint8, device=dev)

    def resize(self, start, end):
        kv_resize(self.cache, self.refs, self.table, start, end, ws=self.resize_ws, dev_err=self.err)

    def forward(self, x, seq, slot, at, start=None, mask=None):
        """x [T, d] BF16; seq, slot int32 [T]: where the tokens' keys and values go; at: their positions in the text."""
        T, (H, K, D) = x.shape[0], (self.HEADS, self.KV_HEADS, self.DIM)
        x, u = moe_residual_norm(x, torch.zeros_like(x), 0.0)
        qkv = (u @ self.w_qkv).view(T, H + 2 * K, D)
        q, k = kv_rotate(qkv[:, :H], qkv[:, H:H + K], at, self.turns, self.gain)
        kv_append(self.cache, k, qkv[:, H + K:], seq, slot, self.table, dev_err=self.err)
        att, _ = kv_attend_tree(q, self.cache, seq, slot, self.table, start, mask, ws=self.ws, dev_err=self.err)
        x, u = moe_residual_norm(x, att.reshape(T, H * D) @ self.w_o, 1.0)
        out, _ = self.moe.forward(u)
        return moe_residual_norm(x, out, 2.0 ** -0.5, want_norm=False)[0]


def run(prompt: int = 200, steps: int = 6, beams: int = 3, dev="cuda:0"):
    """(outputs of the accepted tokens, outputs of one prefill over every beam's whole text at the same places, tokens that took
    the same experts in both, pages in use of either)"""
    dev, n = torch.device(dev), len(PARENT)
    i32 = dict(dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(11)
    pick = random.Random(5)

    def tokens(count):
        return torch.randn(count, synth.TINY.d, generator=g, device=dev).to(torch.bfloat16)

    text = tokens(prompt)
    longest = prompt + n * (steps + 1)
    layer = TreeLayer(dev, max(prompt, beams * n), beams, longest)

    # the prompt, once, in row 0; then every row shares its pages
    pos = torch.arange(prompt, **i32)
    lens = torch.zeros(beams, **i32)
    layer.resize(lens, torch.tensor([prompt] + [0] * (beams - 1), **i32))
    layer.forward(text, torch.zeros(prompt, **i32), pos, pos)
    lens.fill_(prompt)
    kv_fork(layer.cache, layer.refs, layer.table, torch.zeros(beams, **i32), lens, dev_err=layer.err)

    # what a step is told: the drafts, and the path that was accepted (here: made up)
    depth = torch.tensor([len(path_to(i)) - 1 for i in range(n)], **i32).repeat(beams)
    node, seq = torch.arange(n, **i32).repeat(beams), torch.arange(beams, **i32).repeat_interleave(n)
    mask = torch.tensor([sum(1 << j for j in path_to(i)) for i in range(n)], dtype=torch.int64, device=dev).repeat(beams).view(-1, 1)
    x, path, count = tokens(beams * n), torch.zeros(beams, n, **i32), torch.zeros(beams, **i32)
    out, after = torch.empty_like(x), torch.empty_like(lens)

    def step():
        first = lens.repeat_interleave(n)
        layer.resize(lens, lens + n)
        out.copy_(layer.forward(x, seq, first + node, first + depth, lens, mask))
        kv_compact(layer.cache, layer.table, lens, path, count, length=after, dev_err=layer.err)
        layer.resize(after, after)
        lens.copy_(after)

    graph = StepGraph(step)   # (its runs before the capture accept nothing)
    texts, outs, experts = [[text] for _ in range(beams)], [[] for _ in range(beams)], [[] for _ in range(beams)]
    for _ in range(steps):
        x.copy_(tokens(beams * n))
        kept = [path_to(pick.randrange(n)) for _ in range(beams)]
        for b, p in enumerate(kept):
            path[b, :len(p)] = torch.tensor(p, **i32)
            count[b] = len(p)
        graph.replay()
        for b, p in enumerate(kept):
            texts[b].append(x.view(beams, n, -1)[b, p])
            outs[b].append(out.view(beams, n, -1)[b, p])
            experts[b].append(layer.moe.ids[:beams * n].view(beams, n, -1)[b, p])
    torch.cuda.synchronize()
    if int(layer.err):
        raise RuntimeError(f"device error {int(layer.err)}")

    # every beam's text in one go, each with pages of its own
    texts = [torch.cat(t) for t in texts]
    ends = [len(t) for t in texts]
    if lens.tolist() != ends:
        raise RuntimeError(f"lengths {lens.tolist()}, not {ends}")
    again = TreeLayer(dev, sum(ends), beams, longest)
    again.resize(torch.zeros(beams, **i32), torch.tensor(ends, **i32))
    seq = torch.cat([torch.full((e,), b, **i32) for b, e in enumerate(ends)])
    pos = torch.cat([torch.arange(e, **i32) for e in ends])
    full = again.forward(torch.cat(texts), seq, pos, pos).split(ends)
    torch.cuda.synchronize()
    if int(again.err):
        raise RuntimeError(f"device error {int(again.err)}")
    used = [int((r.refs > 0).sum()) for r in (layer, again)]
    ids = [torch.cat([torch.cat(e) for e in experts]), torch.cat([e[prompt:] for e in again.moe.ids[:sum(ends)].split(ends)])]
    same = (ids[0].sort(1)[0] == ids[1].sort(1)[0]).all(1)
    return torch.cat([torch.cat(o) for o in outs]), torch.cat([f[prompt:] for f in full]), same, used


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--steps", type=int, default=6)
    a = ap.parse_args()
    tree, full, same, used = run(a.prompt, a.steps)
    off = (tree.float() - full.float())[same].norm() / full.float()[same].norm()
    print(f"{len(tree)} drafted tokens accepted in {a.steps} steps of three beams behind {a.prompt} shared tokens ({used[0]} pages, "
          f"{used[1]} without sharing): difference from prefilling them all: {float(off):.2e} of the norm ({int((~same).sum())} with other experts left out)")


if __name__ == "__main__":
    main()
