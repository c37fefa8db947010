"""Attention over the paged MX cache in 64 bits, whole sequences at a time: the plain reference for calls with bounds
below the sequences' sizes and for values that are not finite.  Nothing here uses the library."""
import torch

import _cacheref as R


def reference(c, max_q=None, max_kv=None, device="cpu"):
    """Result, weights and sizes as _cacheref.attention gives them, of a case's sequences.  Queries of a sequence beyond
    max_q give zeros, tokens beyond max_kv are not seen.  A value above fp32's range is infinite, and a row that sees
    one (or NaN) has it added to that dimension: its weight is above zero."""
    tok = R.Tokens(c.cache)
    q = c.q.double().cpu().to(device)
    total, q_heads, dim = q.shape
    heads = c.cache.heads
    group = q_heads // heads
    out, weight = torch.zeros_like(q), torch.zeros_like(q)
    size = torch.zeros((total, q_heads, 1), dtype=torch.float64, device=device)
    tree = None if c.tree is None else c.tree.cpu().to(device)
    for b, (n, new, at) in enumerate(zip(c.kv_lens.tolist(), c.nq, c.q_starts.tolist())):
        m = new if max_q is None else min(new, max_q)
        t = n if max_kv is None else min(n, max_kv)
        if m == 0 or t == 0:
            continue
        (k, ok), (v, _) = (tok.take(which, c.table[b].tolist(), t) for which in "kv")
        k, v, ok = k.to(device), v.float().double().to(device), ok.to(device)
        place = torch.arange(t, device=device) - (n - new)
        if tree is None:
            see = place[None] <= torch.arange(m, device=device)[:, None]
        else:
            bits = 64 * tree.shape[1]
            word = place.clamp(min=0, max=bits - 1)
            see = ((tree[at:at + m][:, word // 64] >> (word % 64)) & 1 == 1) & (place < bits) | (place < 0)
        see = see & ok
        kt = k.permute(1, 2, 0).contiguous()
        rows = q[at:at + m].view(m, heads, group, dim).permute(1, 2, 0, 3).reshape(heads, group * m, dim)
        seen = see.repeat(group, 1)
        s = torch.matmul(rows, kt) * dim ** -0.5
        s = torch.where(seen, s, float("-inf"))
        top = s.amax(-1, keepdim=True)
        p = torch.where(seen, torch.exp(s - torch.where(top == float("-inf"), 0.0, top)), 0.0)
        total_p = p.sum(-1, keepdim=True)
        p = p / torch.where(total_p == 0, 1.0, total_p)
        finite = torch.where(torch.isfinite(v), v, 0.0).transpose(0, 1).contiguous()
        o = torch.matmul(p, finite)
        for j, h, d in (~torch.isfinite(v)).nonzero().tolist():
            o[h, :, d] += torch.where(seen[:, j], v[j, h, d], 0.0)
        w = torch.matmul(p, finite.abs())
        z = torch.where(seen, torch.matmul(rows.abs(), kt.abs()), 0.0).amax(-1, keepdim=True) * dim ** -0.5
        for dst, src in ((out, o), (weight, w), (size, z)):
            dst[at:at + m] = src.view(heads, group, m, -1).permute(2, 0, 1, 3).reshape(m, q_heads, -1)
    return out, weight, size


def check(c, got, **kw):
    """The kernel's result against the reference: NaN and infinities where they belong, the rest within the bound."""
    ref, weight, size = reference(c, **kw)
    got = got.double().to(ref.device)
    assert got.shape == ref.shape
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaN elsewhere"
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], ref[inf]), "infinities elsewhere"
    # weights that are off by e_i of themselves, in the products and in their sum, move the result by
    # sum w_i e_i (v_i - out): up to the largest e_i times (sum w |v| + |out|)
    bound = R.attention_bound(ref, weight + ref.abs(), size, ref.shape[2], max(c.kv))
    over = torch.where(torch.isfinite(ref), (got - ref).abs() - bound, -1.0)
    assert float(over.max()) <= 0, float(over.max())
