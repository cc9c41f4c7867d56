"""A small decoder on one GPU: attention over the paged 8-bit cache and the activation-sparse FFN, layer by layer.

Random weights of a ReLU-gated model's shape (projections by plain matrix products). Three prompts of different lengths
go in as one ragged batch, one sequence is forked into two continuations, all are decoded for some steps (optionally
under a sliding window with first tokens kept), finished sequences are freed and the pool is made dense.

--rope turns queries and keys by their positions, after a norm of each head, in the pass that writes the cache. --int4
takes 4-bit projections. --samples N decodes N continuations of one long prompt that share its pages: their attention
reads what they share once.

    python examples/decode_with_cache.py [--steps 32] [--window 0] [--sinks 4] [--rope] [--int4] [--samples 0]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_decode_pi_gb300 as P  # noqa: E402
from workload import WORKLOADS, make_layer, scaled  # noqa: E402
from workload.gen import quantize_int4_g128  # noqa: E402


def rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Decoder:
    """Pre-norm layers x += attention(rms(x)); x += FFN(rms(x)) in fp32, bf16 FFN weights, an e4m3 cache."""

    def __init__(self, *, d=1024, f=2752, layers=2, heads=8, kv_heads=2, page=16, n_pages=256, max_seqs=8,
                 max_tokens=1024, max_batch=256, window=0, sinks=0, seed=0, rope=False, int4=False):
        w = scaled(WORKLOADS["relullama7b_d4096_f11008_bf16_L32"], d=d, f=f, r=128, n_layers=layers)
        self.d, self.heads, self.kv_heads, self.dim = d, heads, kv_heads, d // heads
        self.window, self.sinks, self.max_batch = window, sinks, max_batch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda") / s[0] ** 0.5  # noqa: E731
        self.qkv = [rand(d, (heads + 2 * kv_heads) * self.dim) for _ in range(layers)]
        self.o = [rand(heads * self.dim, d) for _ in range(layers)]
        self.ffn = P.SparseFFN.from_workload(w, [P.apply_hot_first(make_layer(w, i, seed, device="cuda"))[0]
                                                 for i in range(layers)], max_batch=max_batch)
        if int4:
            def linear(w):
                return P.Int4Linear(*quantize_int4_g128(w.T.contiguous()))

            self.qkv, self.o = [linear(w) for w in self.qkv], [linear(w) for w in self.o]
        self.int4, self.rotary = int4, None
        if rope:
            self.rotary = P.Rotary(P.rotary_frequencies(self.dim), self.dim, norm=True)
        self.cache = P.KVCache.empty(layers, heads, kv_heads, self.dim, page, n_pages, max_seqs, max_tokens)

    def project(self, w, x, add=None):
        """x w (+ add), in 4 bits for up to max_batch rows at a time."""
        if not self.int4:
            return x @ w if add is None else add + x @ w
        y = x.new_empty(x.shape[0], w.n)
        for c in range(0, x.shape[0], self.max_batch):
            part = slice(c, c + self.max_batch)
            w(x[part], out=y[part], add=None if add is None else add[part])
        return y

    def attention(self, i, seqs, tok_start, x, plan=None):
        """x + attention of layer i (room has been reserved); plan: what the sequences share."""
        h = self.project(self.qkv[i], rms(x)).unflatten(1, (-1, self.dim))   # queries, keys and values side by side
        a, b = self.heads, self.heads + self.kv_heads
        q, k, v = h[:, :a], h[:, a:b], h[:, b:]
        if self.rotary is None:
            self.cache.append(i, seqs, tok_start, k, v)
        else:
            q = self.cache.append_rotated(i, seqs, tok_start, self.rotary, q, k, v, q_out=q)
        if plan is None:
            att = self.cache.attend(i, seqs, tok_start, q, window=self.window, sinks=self.sinks)
        else:
            att = self.cache.attend_shared(i, seqs, tok_start, plan, q)
        return self.project(self.o[i], att.flatten(1), add=x)

    def forward(self, seqs, tok_start, x, plan=None):
        """One step for the ragged batch: x [tokens, d], the new tokens of `seqs`. Returns the last layer's output."""
        self.cache.reserve(seqs, tok_start)
        for i in range(len(self.qkv)):
            x = self.attention(i, seqs, tok_start, x, plan)
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

    def step(self, seqs, x, plan=None):
        """One token for each of `seqs` (int32 CUDA tensor): x [sequences, d]."""
        return self.forward(seqs, torch.arange(len(seqs) + 1, dtype=torch.int32, device="cuda"), x, plan)

    def share(self, seqs):
        """The plan for steps of one token for each of `seqs`, all of one group (before the first of them)."""
        return self.cache.share(seqs, torch.arange(len(seqs) + 1, dtype=torch.int32, device="cuda"), ids(0, len(seqs)))

    def check(self):
        for name, status in (("cache", self.cache.status()), ("ffn", self.ffn.status())):
            if status:
                raise RuntimeError(f"{name}: {P.pi_status_string(status)}")

    def close(self):
        self.cache.close()
        self.ffn.close()


def ids(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def samples(m, n, steps, prompt=700):
    """n continuations of one prompt, decoded for some steps with the prompt's attention read once for all of them."""
    y = m.forward(ids(0), ids(0, prompt), torch.randn(prompt, m.d, device="cuda"))
    seqs = torch.arange(n, dtype=torch.int32, device="cuda")
    m.cache.fork(torch.zeros(n - 1, dtype=torch.int32, device="cuda"), seqs[1:])
    plan = m.share(seqs)                  # once: it serves every layer, and every step while the sequences only grow
    h = y[-1:] + 0.1 * torch.randn(n, m.d, device="cuda")
    for _ in range(steps):
        h = m.step(seqs, rms(h), plan)
    m.check()
    print(f"{steps} steps of {n} continuations of a prompt of {prompt}: lengths {m.cache.length[:n].tolist()}, output rms "
          f"{h.square().mean().sqrt().item():.3f}")


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=4)
    ap.add_argument("--rope", action="store_true")
    ap.add_argument("--int4", action="store_true")
    ap.add_argument("--samples", type=int, default=0)
    args = ap.parse_args()
    if args.samples > 1:                  # (shared prefixes are read without a window)
        m = Decoder(rope=args.rope, int4=args.int4, max_seqs=args.samples, n_pages=64 + 8 * args.samples)
        samples(m, args.samples, args.steps)
        return m.close()
    m = Decoder(window=args.window, sinks=args.sinks, rope=args.rope, int4=args.int4)
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
