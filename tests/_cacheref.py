"""Plain 64-bit references of the serving operators on the CPU: rotary
positions, the paged MX cache and attention over it.  Nothing here uses the
library; codes and scales come from the scalar C oracle."""
import numpy as np
import torch

import oracle

GRID = {
    0: np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]),
    1: np.array([m / 512.0 for m in range(8)] +
                [(1.0 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1] + [np.nan]),
}


def bf16_bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def rotate(x, positions, inv_freq, scale, layout, inverse):
    """float64 rotation of x [tokens, heads, dim]; also sum |a c| + |b s| of each element."""
    x = x.double().cpu()
    angle = positions.double().cpu()[:, None] * inv_freq.double().cpu()[None]
    c, s = (scale * angle.cos())[:, None], (scale * angle.sin())[:, None]
    if inverse:
        s = -s
    h = inv_freq.numel()
    out, mag = x.clone(), x.abs()
    ia, ib = (slice(0, h), slice(h, 2 * h)) if layout == 0 else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, mag


def quantise(fmt, x):
    """Codes [..., dim or dim/2] and scales [..., dim/32] of bf16 x, by the oracle."""
    dim = x.shape[-1]
    rows = bf16_bits(x).reshape(-1, dim)
    codes, scales = oracle.quantize(fmt, rows)
    return (torch.from_numpy(codes.reshape(*x.shape[:-1], -1).copy()),
            torch.from_numpy(scales.reshape(*x.shape[:-1], -1).copy()))


def values(fmt, codes, scales):
    """float64 values of codes [..., dim or dim/2] with scales [..., dim/32] (CPU tensors)."""
    c = codes.numpy()
    if fmt == 0:
        c = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)
        sign, mag = c >> 3, c & 7
    else:
        sign, mag = c >> 7, c & 127
    v = np.where(sign == 1, -GRID[fmt][mag], GRID[fmt][mag])
    s = scales.numpy().astype(np.float64)
    unit = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return torch.from_numpy((v.reshape(*v.shape[:-1], -1, 32) * unit[..., None]).reshape(v.shape))


class Tokens:
    """The cache's tensors on the CPU, and sequences' tokens taken out of them."""

    def __init__(self, cache):
        self.fmt, self.page, self.pages = cache.fmt, cache.page, cache.pages
        self.k = (cache.k_codes.cpu(), cache.k_scales.cpu())
        self.v = (cache.v_codes.cpu(), cache.v_scales.cpu())

    def take(self, which, table, n):
        """float64 [n, heads, dim] of a sequence's first n tokens, and whether each is in the cache."""
        codes, scales = getattr(self, which)
        t = torch.arange(n)
        page = torch.as_tensor(table, dtype=torch.long)[t // self.page]
        ok = (page >= 0) & (page < self.pages)
        page = torch.where(ok, page, 0)
        row = t % self.page
        return values(self.fmt, codes[page, :, row], scales[page, :, :, row]), ok


def attention(cache, q, q_starts, kv_lens, table, tree=None, scale=None):
    """float64 result [total_q, q_heads, dim], and for the tolerance: sum p |v| / sum p of every element, and the
    largest sum |q k| scale of every row."""
    tok = Tokens(cache)
    q = q.double().cpu()
    total, qh, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    heads = cache.heads
    group = qh // heads
    out, weight, size = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(total, qh, 1, dtype=torch.float64)
    starts, lens = q_starts.tolist(), kv_lens.tolist()
    for b, n in enumerate(lens):
        nq = starts[b + 1] - starts[b]
        if nq == 0 or n == 0:
            continue
        k, ok = tok.take("k", table[b].tolist(), n)
        v, _ = tok.take("v", table[b].tolist(), n)
        for i in range(nq):
            r = starts[b] + i
            j = torch.arange(n) - (n - nq)  # place among the new tokens
            if tree is None:
                see = j <= i
            else:
                words = tree[r].tolist()
                see = torch.tensor([x < 0 or (words[x // 64] >> (x % 64)) & 1 == 1 for x in j.tolist()])
            see = see & ok
            if not bool(see.any()):
                continue
            for h in range(qh):
                kk, vv = k[see, h // group], v[see, h // group]
                s = (kk @ q[r, h]) * scale
                p = torch.exp(s - s.max())
                out[r, h] = (p[:, None] * vv).sum(0) / p.sum()
                weight[r, h] = (p[:, None] * vv.abs()).sum(0) / p.sum()
                size[r, h] = (kk.abs() @ q[r, h].abs()).max() * scale
    return out, weight, size


def attention_bound(out, weight, size, dim, n):
    """Elementwise tolerance of the kernel against `attention`: the output's rounding to bf16; each weight's rounding
    to bf16; weights whose fp32 scores are off by at most (dim + 2) roundings of 2^-23 of the sum of magnitudes, in
    numerator and denominator; fp32 sums over n tokens, the exponent's argument (below 2^7 in magnitude where the
    weight matters) and the exponential itself."""
    delta = (dim + 2) * 2.0 ** -23 * size
    rel = 2.0 ** -8 + 2 * delta + (n + 64) * 2.0 ** -23 + 2.0 ** -15
    return 2.0 ** -8 * out.abs() + rel * weight * (1 + 2.0 ** -8) + 1e-30
