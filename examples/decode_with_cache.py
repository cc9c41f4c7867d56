"""A small decoder on one GPU: attention over the paged 8-bit cache and the activation-sparse FFN, layer by layer.

Random weights of a ReLU-gated model's shape (projections by plain matrix products). Three prompts of different lengths
go in as one ragged batch, one sequence is forked into two continuations, all are decoded for some steps (optionally
under a sliding window with first tokens kept), finished sequences are freed and the pool is made dense.

    python examples/decode_with_cache.py [--steps 32] [--window 0] [--sinks 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_decode_pi_gb300 as P  # noqa: E402
from workload import WORKLOADS, make_layer, scaled  # noqa: E402


def rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Decoder:
    """Pre-norm layers x += attention(rms(x)); x += FFN(rms(x)) in fp32, bf16 FFN weights, an e4m3 cache."""

    def __init__(self, *, d=1024, f=2752, layers=2, heads=8, kv_heads=2, page=16, n_pages=256, max_seqs=8,
                 max_tokens=1024, max_batch=256, window=0, sinks=0, seed=0):
        w = scaled(WORKLOADS["relullama7b_d4096_f11008_bf16_L32"], d=d, f=f, r=128, n_layers=layers)
        self.d, self.heads, self.kv_heads, self.dim = d, heads, kv_heads, d // heads
        self.window, self.sinks, self.max_batch = window, sinks, max_batch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda") / s[0] ** 0.5  # noqa: E731
        self.qkv = [rand(d, (heads + 2 * kv_heads) * self.dim) for _ in range(layers)]
        self.o = [rand(heads * self.dim, d) for _ in range(layers)]
        self.ffn = P.SparseFFN.from_workload(w, [P.apply_hot_first(make_layer(w, i, seed, device="cuda"))[0]
                                                 for i in range(layers)], max_batch=max_batch)
        self.cache = P.KVCache.empty(layers, heads, kv_heads, self.dim, page, n_pages, max_seqs, max_tokens)

    def forward(self, seqs, tok_start, x):
        """One step for the ragged batch: x [tokens, d], the new tokens of `seqs`. Returns the last layer's output."""
        self.cache.reserve(seqs, tok_start)
        for i in range(len(self.qkv)):
            h = (rms(x) @ self.qkv[i]).unflatten(1, (-1, self.dim))   # queries, keys and values side by side
            a, b = self.heads, self.heads + self.kv_heads
            self.cache.append(i, seqs, tok_start, h[:, a:b], h[:, b:])
            att = self.cache.attend(i, seqs, tok_start, h[:, :a], window=self.window, sinks=self.sinks)
            x = x + att.flatten(1) @ self.o[i]
            u = rms(x).contiguous()
            y = torch.empty_like(u)
            for c in range(0, u.shape[0], self.max_batch):            # the FFN takes up to max_batch rows
                part = u[c:c + self.max_batch]
                idx, count = self.ffn.predict(i, part)
                self.ffn.sparse_ffn(i, part, idx, count, y[c:c + self.max_batch])
            x = x + y
        if self.window > 0:
            self.cache.trim(seqs, self.window, self.sinks)
        return x

    def step(self, seqs, x):
        """One token for each of `seqs` (int32 CUDA tensor): x [sequences, d]."""
        return self.forward(seqs, torch.arange(len(seqs) + 1, dtype=torch.int32, device="cuda"), x)

    def check(self):
        for name, status in (("cache", self.cache.status()), ("ffn", self.ffn.status())):
            if status:
                raise RuntimeError(f"{name}: {P.pi_status_string(status)}")

    def close(self):
        self.cache.close()
        self.ffn.close()


def ids(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=4)
    args = ap.parse_args()
    m = Decoder(window=args.window, sinks=args.sinks)
    lens = [70, 5, 130]
    x = torch.randn(sum(lens), m.d, device="cuda")
    y = m.forward(ids(0, 1, 2), ids(0, 70, 75, 205), x)                  # the prompts, as one ragged batch
    m.cache.fork(ids(0), ids(3))                                         # two continuations of the first
    live = ids(0, 1, 2, 3)
    h = torch.stack([y[69], y[74], y[204], y[69] + 0.1 * torch.randn(m.d, device="cuda")])
    for _ in range(args.steps):
        h = m.step(live, rms(h))
    used = int((m.cache.ref > 0).sum())
    m.cache.free(ids(0, 1))
    dense = int(m.cache.compact())
    h = m.step(ids(2, 3), rms(h[2:]))
    m.check()
    print(f"{args.steps} steps of 4 sequences: {used} pages in use, {dense} after freeing two and compacting; "
          f"lengths {m.cache.length.tolist()}, output rms {h.square().mean().sqrt().item():.3f}")
    m.close()


if __name__ == "__main__":
    main()
