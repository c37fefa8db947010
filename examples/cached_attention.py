"""A layer's attention served from the paged MX cache, as a serving loop would
run it: a prompt in chunks, single-token steps of a ragged batch, a tree of
drafted tokens, its verification and what is kept of it, a sequence that goes on
in two ways, and queries of another sequence over a prompt.

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
    """Rotary attention over the cache; pages are taken and given back as the sequences' lengths ask for it."""

    def __init__(self, fmt: int, sequences: int, pages: int, longest: int):
        self.cache = mx.MXCache.allocate(fmt, pages, HEADS, PAGE, DIM)
        self.inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM)
        self.table = torch.full((sequences, -(-longest // PAGE)), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")  # rows of the table that hold each page
        self.lens = [0] * sequences
        self.keys = [[] for _ in range(sequences)]  # full precision, for the comparison
        self.values = [[] for _ in range(sequences)]

    def slots(self, b: int, new: int) -> list[int]:
        """Slots of a sequence's next tokens; takes pages as they are needed."""
        self.lens[b] += new
        self.resize()
        row = self.table[b].tolist()
        return [row[t // PAGE] * PAGE + t % PAGE for t in range(self.lens[b] - new, self.lens[b])]

    def resize(self):
        missing = mx.mx_cache_resize(self.cache, self.refs, self.table,
                                     torch.tensor(self.lens, dtype=torch.int32, device="cuda"))
        assert not bool(missing.any()), "no page is free"

    def fork(self, b: int):
        """The last row goes on from sequence b: full pages are shared, the last one is copied."""
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        parent = torch.tensor([b], dtype=torch.int32, device="cuda")
        row, missing = mx.mx_cache_fork(self.cache, self.refs, self.table, lens, parent)
        assert not bool(missing.any()), "no page is free"
        self.table[-1:] = row
        self.lens[-1] = self.lens[b]
        self.keys[-1], self.values[-1] = list(self.keys[b]), list(self.values[b])

    def settle(self, sequences, starts, tokens, target, draft, parents, uniforms):
        """Verifies the drafted trees that attend() has just written and keeps the tokens of the accepted paths."""
        i32 = {"dtype": torch.int32, "device": "cuda"}
        counts, path, out = mx.mx_verify(target, tokens, uniforms, torch.tensor(starts, **i32),
                                         max_q=max(n for _, n in sequences), draft=draft, parents=parents)
        rows = [b for b, _ in sequences]
        first = torch.tensor([self.lens[b] - n for b, n in sequences], **i32)
        lens = mx.mx_cache_compact(self.cache, first, path, counts, self.table[rows])
        for (b, _), n, kept in zip(sequences, lens.tolist(), path.tolist()):
            self.lens[b] = n
            kept = [i for i in kept if i >= 0]
            self.keys[b][-1], self.values[b][-1] = self.keys[b][-1][kept], self.values[b][-1][kept]
        self.resize()
        return counts.tolist(), out

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
    layer = Layer(mx.E4M3 if args.fmt == "e4m3" else mx.E2M1, len(prompts) + 1, 64, 1024)  # and a row for a branch

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
        pos = torch.tensor(layer.lens[:-1], device="cuda")
        out, exact = layer.attend(everyone, project(len(prompts)), pos)
    report("single-token step", out, exact)
    # a drafted tree for each sequence: token 0, two children, and two of the first child's
    parents = (None, 0, 0, 1, 1)
    seen, depth = [], []
    for i, p in enumerate(parents):
        seen.append((1 << i) | (seen[p] if p is not None else 0))
        depth.append(depth[p] + 1 if p is not None else 0)
    tree = torch.tensor(seen * len(prompts), device="cuda")[:, None]
    pos = torch.tensor([n + d for n in layer.lens[:-1] for d in depth], device="cuda")
    trees = [(b, len(parents)) for b in range(len(prompts))]
    nodes = len(parents) * len(prompts)
    out, exact = layer.attend(trees, project(nodes), pos, tree=tree)
    report("drafted trees", out, exact)
    # a model's and its draft's probabilities after each node, and tokens drawn from the latter
    logits = 2.0 * torch.randn((nodes, 1000), device="cuda")
    target, draft = torch.softmax(logits, 1), torch.softmax(logits + 0.3 * torch.randn_like(logits), 1)
    up = torch.tensor([-1] + list(parents[1:]), device="cuda").repeat(len(prompts))
    root = torch.arange(nodes, device="cuda") // len(parents) * len(parents)
    tokens = torch.multinomial(draft[root + up.clamp(min=0)], 1)[:, 0]
    counts, _ = layer.settle(trees, list(range(0, nodes + 1, len(parents))), tokens, target, draft, up.int(),
                             torch.rand(nodes, dtype=torch.float64, device="cuda"))
    print(f"kept of {len(parents)} nodes each: {counts}")
    out, exact = layer.attend(everyone, project(len(prompts)), torch.tensor(layer.lens[:-1], device="cuda"))
    report("step behind the kept paths", out, exact)
    layer.fork(0)  # and both go on
    out, exact = layer.attend([(0, 1), (len(prompts), 1)], project(2), torch.tensor([layer.lens[0]] * 2, device="cuda"))
    report("a sequence and its branch", out, exact)
    q = project(9)[:, :HEADS * GROUP]  # of another sequence
    i32 = {"dtype": torch.int32, "device": "cuda"}
    out = mx.mx_cache_cross_attention(layer.cache, q, torch.tensor([0, 9], **i32), torch.tensor([prompts[1]], **i32),
                                      layer.table[1:2], max_q=9, max_kv=prompts[1])
    k, v = (torch.cat(t[1])[:prompts[1]].transpose(0, 1).repeat_interleave(GROUP, 0) for t in (layer.keys, layer.values))
    s = torch.matmul(q.float().transpose(0, 1), k.transpose(1, 2).contiguous()) / math.sqrt(DIM)
    report("another sequence's queries", out, torch.matmul(s.softmax(-1), v).transpose(0, 1))
    k, v = mx.mx_cache_read(layer.cache, torch.tensor([int(layer.table[0, 0]) * PAGE], device="cuda"))
    err = float((v[0].float() - layer.values[0][0][0]).norm() / v[0].float().norm())
    print(f"first token read back: values differ by {err:.4f}")


if __name__ == "__main__":
    main()
