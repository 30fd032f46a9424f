"""One decoder layer over a quantised paged cache: block-sparse attention, then the MoE layer.

Two sequences are prefilled in one ragged chunk and then decoded token by token, the decode step being
one CUDA graph (append -> select -> attend -> MoE).  Weights are random (synth.TINY for the MoE half;
projections from a seed): the program shows the calls in their order and what the caller keeps.

    python examples/sparse_layer.py [--prefill 700] [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_routed_expert_gb300 import (BRE_FMT_Q8_0, FfnWeights, KvCache, MoeLayer, StepGraph, kv_append, kv_attend,  # noqa: E402
                                     kv_select, moe_residual_norm)
from bit_routed_expert_gb300 import api, synth  # noqa: E402


class SparseLayer:
    """x -> x + attention(norm(x)) -> x + moe(norm(x)), for up to T_max tokens a call."""

    HEADS, KV_HEADS, DIM, TOP = 8, 2, 64, 6

    def __init__(self, dev, T_max: int, B: int, max_len: int, seed: int = 1):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        s, lw = synth.TINY, synth.layer_weights(seed, 0, synth.TINY, device=dev)
        self.moe = MoeLayer(lw.w_r.to(dev), lw.bias.to(dev), api.routed_weights(lw.gate, lw.up, lw.down, s.d, s.F),
                            FfnWeights(lw.sh_gate, lw.sh_up, lw.sh_down, BRE_FMT_Q8_0, s.d, s.F_shared), s.k, T_max)
        self.d = s.d
        H, K, D = self.HEADS, self.KV_HEADS, self.DIM
        self.w_qkv = (torch.randn(s.d, (H + 2 * K) * D, generator=g, device=dev) * s.d ** -0.5).to(torch.bfloat16)
        self.w_o = (torch.randn(H * D, s.d, generator=g, device=dev) * (H * D) ** -0.5).to(torch.bfloat16)
        # the cache, and which page holds which block of which sequence
        N = -(-max_len // api.KV_BLOCK)
        self.cache = KvCache.empty(B * N, K, D, dev)
        self.table = torch.randperm(B * N, generator=g, device=dev).to(torch.int32).view(B, N).contiguous()
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)

    def forward(self, x, seq, pos):
        """x [T, d] BF16, seq and pos int32 [T]: the next tokens of their sequences."""
        T, (H, K, D) = x.shape[0], (self.HEADS, self.KV_HEADS, self.DIM)
        x, u = moe_residual_norm(x, torch.zeros_like(x), 0.0)
        qkv = (u @ self.w_qkv).view(T, H + 2 * K, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]   # slices: the calls take row strides
        kv_append(self.cache, k, v, seq, pos, self.table, dev_err=self.err)
        ids, _ = kv_select(q, self.cache, seq, pos, self.table, self.TOP, dev_err=self.err)
        att, _ = kv_attend(q, self.cache, seq, pos, self.table, ids, dev_err=self.err)
        x, u = moe_residual_norm(x, att.reshape(T, H * D) @ self.w_o, 1.0)
        out, _ = self.moe.forward(u)
        return moe_residual_norm(x, out, 2.0 ** -0.5, want_norm=False)[0]


def run(prefill: int = 700, steps: int = 8, dev="cuda:0"):
    """(outputs of the decode steps, outputs of one prefill over everything at the same positions)"""
    dev = torch.device(dev)
    lens = [prefill, prefill // 3 + 1]
    total = [n + steps for n in lens]
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    x = [torch.randn(n, synth.TINY.d, generator=g, device=dev).to(torch.bfloat16) for n in total]

    def tokens(spans):
        seq = torch.cat([torch.full((b - a,), i, dtype=torch.int32) for i, (a, b) in enumerate(spans)]).to(dev)
        pos = torch.cat([torch.arange(a, b, dtype=torch.int32) for a, b in spans]).to(dev)
        return torch.cat([x[i][a:b] for i, (a, b) in enumerate(spans)]), seq, pos

    layer = SparseLayer(dev, sum(total), len(lens), max(total))
    layer.forward(*tokens([(0, n) for n in lens]))
    # decode: one graph, its inputs copied in
    xin, seq, pos = tokens([(n, n + 1) for n in lens])
    out = torch.empty_like(xin)
    first = pos.clone()
    graph = StepGraph(lambda: out.copy_(layer.forward(xin, seq, pos)))
    decoded = []
    for i in range(steps):
        xin.copy_(torch.stack([x[b][n + i] for b, n in enumerate(lens)]))
        pos.copy_(first + i)
        graph.replay()
        decoded.append(out.clone())
    torch.cuda.synchronize()
    if int(layer.err):
        raise RuntimeError(f"device error {int(layer.err)}")
    again = SparseLayer(dev, sum(total), len(lens), max(total))
    full = again.forward(*tokens([(0, n) for n in total]))
    at = [torch.arange(n, n + steps, device=dev) + o for n, o in zip(lens, (0, total[0]))]
    return torch.stack(decoded, 1), torch.stack([full[i] for i in at])


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prefill", type=int, default=700)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    step, full = run(a.prefill, a.steps)
    off = (step.float() - full.float()).norm() / full.float().norm()
    print(f"decoded {a.steps} tokens of 2 sequences after {a.prefill} and {a.prefill // 3 + 1}: "
          f"difference from prefilling them all: {float(off):.2e} of the norm")


if __name__ == "__main__":
    main()
