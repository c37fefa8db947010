"""Verification of drafted tokens in exact rational arithmetic on the CPU, one sequence and one entry at a time: the
plain reference of mx_verify.  Nothing here uses the library."""
from fractions import Fraction

import torch


def row_of(t, r):
    """Entries of a row as exact numbers; negative ones and NaN count as zero, infinity as fp32's largest number."""
    top = torch.finfo(torch.float32).max
    return [Fraction(min(x, top)) if x > 0 else Fraction(0) for x in t[r].double().tolist()]


def sequence(target, draft, tokens, uniforms, parents, first, n):
    """Places that stay and the tokens put out of the nodes first .. first + n."""
    vocab = target.shape[1]
    c, path, out = 0, [0], []
    w, total = row_of(target, first), Fraction(1)
    for i in range(1, n):
        x = tokens[first + i]
        parent = i - 1 if parents is None else parents[first + i]
        if parent != c or not 0 <= x < vocab:
            continue
        q = row_of(draft, first + c) if draft is not None else [Fraction(int(y == x)) for y in range(vocab)]
        if Fraction(uniforms[first + i]) * total * q[x] < w[x]:
            c = i
            path.append(i)
            out.append(x)
            w, total = row_of(target, first + c), Fraction(1)
            continue
        if draft is not None:
            rest = [max(a - total * b, Fraction(0)) for a, b in zip(w, q)]
        else:
            rest = [Fraction(0) if y == x else a for y, a in enumerate(w)]
        if sum(rest) > 0:
            w, total = rest, sum(rest)
    goal, cum, chosen = Fraction(uniforms[first]) * sum(w), Fraction(0), -1
    for y, a in enumerate(w):
        cum += a
        if a > 0:
            chosen = y
            if cum > goal:
                break
    return path, out + [chosen]


def verify(target, tokens, uniforms, q_starts, max_q, draft=None, parents=None):
    target = target.cpu()
    draft = None if draft is None else draft.cpu()
    tokens, uniforms, starts = tokens.tolist(), uniforms.tolist(), q_starts.tolist()
    parents = None if parents is None else parents.tolist()
    batch = len(starts) - 1
    counts = torch.zeros(batch, dtype=torch.int32)
    path = torch.full((batch, max_q), -1, dtype=torch.int32)
    out = torch.full((batch, max_q), -1, dtype=torch.int64)
    for b in range(batch):
        n = min(starts[b + 1] - starts[b], max_q)
        if n < 1:
            continue
        p, o = sequence(target, draft, tokens, uniforms, parents, starts[b], n)
        counts[b] = len(p)
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        out[b, :len(o)] = torch.tensor(o)
    return counts, path, out
