"""A layer's attention served from the paged MX cache, as a serving loop would
run it: a prompt in chunks, single-token steps of a ragged batch, and the
verification of a tree of drafted tokens.

    python examples/cached_attention.py [--fmt e4m3|e2m1]

Projections are random; every output is compared with attention over the same
keys and values in full precision, so the printed difference is what the
cache's 8 or 4 bits cost.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_quantize_dequantize_amd as mx  # noqa: E402

HEADS, GROUP, DIM, PAGE = 4, 4, 128, 64


class Layer:
    """Rotary attention over the cache; pages are handed out in the order they are asked for."""

    def __init__(self, fmt: int, sequences: int, pages: int, longest: int):
        self.cache = mx.MXCache.allocate(fmt, pages, HEADS, PAGE, DIM)
        self.inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM)
        self.table = torch.zeros((sequences, -(-longest // PAGE)), dtype=torch.int32, device="cuda")
        self.lens = [0] * sequences
        self.free = list(range(pages))
        self.keys = [[] for _ in range(sequences)]  # full precision, for the comparison
        self.values = [[] for _ in range(sequences)]

    def slots(self, b: int, new: int) -> list[int]:
        """Slots of a sequence's next tokens; takes pages as they are needed."""
        out = []
        for t in range(self.lens[b], self.lens[b] + new):
            if t % PAGE == 0:
                self.table[b, t // PAGE] = self.free.pop()
            out.append(int(self.table[b, t // PAGE]) * PAGE + t % PAGE)
        self.lens[b] += new
        return out

    def attend(self, sequences, qkv, positions, tree=None):
        """New tokens of some sequences: sequences is [(index, count), ...], qkv [tokens, heads, dim] of all of
        them, queries first."""
        slots = torch.tensor([s for b, n in sequences for s in self.slots(b, n)], device="cuda")
        q, k, v = qkv[:, :HEADS * GROUP], qkv[:, HEADS * GROUP:HEADS * (GROUP + 1)], qkv[:, HEADS * (GROUP + 1):]
        q = mx.mx_rope(q, positions, self.inv_freq)
        mx.mx_cache_write(self.cache, k, v, slots, positions=positions, inv_freq=self.inv_freq)
        starts = [0]
        for _, n in sequences:
            starts.append(starts[-1] + n)
        rows = [b for b, _ in sequences]
        out = mx.mx_cache_attention(
            self.cache, q, torch.tensor(starts, dtype=torch.int32, device="cuda"),
            torch.tensor([self.lens[b] for b in rows], dtype=torch.int32, device="cuda"), self.table[rows],
            max_q=max(n for _, n in sequences), max_kv=max(self.lens[b] for b in rows), tree=tree)
        return out, self.exact(sequences, starts, q, mx.mx_rope(k, positions, self.inv_freq), v, tree)

    def exact(self, sequences, starts, q, k, v, tree):
        outs = []
        for (b, n), at in zip(sequences, starts):
            self.keys[b].append(k[at:at + n].float())
            self.values[b].append(v[at:at + n].float())
            kk, vv = torch.cat(self.keys[b]), torch.cat(self.values[b])
            s = torch.matmul(q[at:at + n].float().view(n, HEADS, GROUP, DIM).permute(1, 2, 0, 3).reshape(HEADS, -1, DIM),
                             kk.permute(1, 2, 0).contiguous()) / math.sqrt(DIM)
            s = s.view(HEADS, GROUP, n, -1)
            if tree is None:
                see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
            else:
                j = torch.arange(n, device="cuda")
                see = (tree[at:at + n, 0, None] >> j) & 1 == 1
            s[..., -n:].masked_fill_(~see, float("-inf"))
            o = torch.matmul(s.softmax(-1).view(HEADS, GROUP * n, -1), vv.transpose(0, 1).contiguous())
            outs.append(o.view(HEADS, GROUP, n, DIM).permute(2, 0, 1, 3).reshape(n, HEADS * GROUP, DIM))
        return torch.cat(outs)


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--fmt", choices=("e4m3", "e2m1"), default="e4m3")
    args = ap.parse_args()
    torch.manual_seed(0)
    prompts, steps = (700, 130, 391), 5
    layer = Layer(mx.E4M3 if args.fmt == "e4m3" else mx.E2M1, len(prompts), 64, 1024)

    def project(n):
        return torch.randn((n, HEADS * (GROUP + 2), DIM), device="cuda").bfloat16()

    def report(what, out, exact):
        err = float((out.float() - exact).norm() / exact.norm())
        print(f"{what:28s} {tuple(out.shape)}  relative difference {err:.4f}", flush=True)
        # half a step of a 3-bit mantissa is 2^-4, of a 1-bit one 2^-2; keys and values both carry it
        assert err < (0.1 if args.fmt == "e4m3" else 0.4)

    for b, n in enumerate(prompts):  # prompts, in chunks of 256
        for at in range(0, n, 256):
            m = min(256, n - at)
            out, exact = layer.attend([(b, m)], project(m), torch.arange(at, at + m, device="cuda"))
        report(f"prompt of {n}, last chunk", out, exact)
    everyone = [(b, 1) for b in range(len(prompts))]
    for _ in range(steps):  # one token of every sequence
        pos = torch.tensor(layer.lens, device="cuda")
        out, exact = layer.attend(everyone, project(len(prompts)), pos)
    report("single-token step", out, exact)
    # a drafted tree for each sequence: token 0, two children, and two of the first child's
    parents = (None, 0, 0, 1, 1)
    seen, depth = [], []
    for i, p in enumerate(parents):
        seen.append((1 << i) | (seen[p] if p is not None else 0))
        depth.append(depth[p] + 1 if p is not None else 0)
    tree = torch.tensor(seen * len(prompts), device="cuda")[:, None]
    pos = torch.tensor([n + d for n in layer.lens for d in depth], device="cuda")
    out, exact = layer.attend([(b, len(parents)) for b in range(len(prompts))], project(len(parents) * len(prompts)),
                              pos, tree=tree)
    report("drafted trees", out, exact)
    k, v = mx.mx_cache_read(layer.cache, torch.tensor([int(layer.table[0, 0]) * PAGE], device="cuda"))
    err = float((v[0].float() - layer.values[0][0][0]).norm() / v[0].float().norm())
    print(f"first token read back: values differ by {err:.4f}")


if __name__ == "__main__":
    main()
