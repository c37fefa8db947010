"""The measured cases of the operators around drafting, branching and images:
rotary positions with several axes, attention to an encoder's states,
verification of drafted tokens, and the cache's pages.

Four operators, each in a plain form (elementary torch operations) and as a
user's program calls it:

  axes    rotary positions where each pair of dimensions turns with one of
          several positions of its token (time, height, width), and the
          gradient.
  cross   queries attend to all tokens of another sequence (an encoder's
          states, an image's tokens) held in the paged MX cache; neither
          length depends on the other.
  verify  drafted tokens, in a chain or a tree, are kept or refused against
          the target's probabilities with given random numbers, so that what
          is kept and the one token that is sampled after it are distributed
          as the target's own; see _plain_verify for the rule.
  pages   the cache's pages: whole pages copied, sequences forked (full pages
          shared, the last one copied into a free page) and freed, tokens of
          a sequence compacted to those that are kept.

The cache's layout, for `pages` pages of `page` tokens, H key/value heads of
D dimensions, kept apart for keys and values:
  codes   [pages, H, page, D] bytes (MXFP8), [pages, H, page, D/2] (MXFP4,
          the even dimension in the low nibble)
  scales  [pages, H, D/32, page] E8M0 bytes, one for each 32 dimensions.
Token t of a sequence is in page block_table[t // page], row t % page.  A page
is free where its count of holders, refs[page], is zero.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -------------------------------------------------------------------

def _axes(name, tokens, heads, dim, sections, order, layout, dtype, direction, fused):
    """sections: pairs of each axis, as a text; order: axes one after another ("parts") or in turn ("turns")."""
    return {"name": name, "op": "axes", "tokens": tokens, "heads": heads, "dim": dim, "sections": sections,
            "order": order, "layout": layout, "dtype": dtype, "direction": direction, "fused": fused}


def _cross(name, fmt, batch, heads, group, dim, page, kv, q, ragged):
    return {"name": name, "op": "cross", "fmt": fmt, "batch": batch, "heads": heads, "group": group, "dim": dim,
            "page": page, "kv": kv, "q": q, "ragged": ragged}


def _verify(name, batch, nodes, vocab, dtype, draft, tree, ragged):
    return {"name": name, "op": "verify", "batch": batch, "nodes": nodes, "vocab": vocab, "dtype": dtype,
            "draft": draft, "tree": tree, "ragged": ragged}


def _pages(name, what, fmt, heads, dim, page, sequences, tokens, part):
    """part: children of each sequence (fork), or the share of the tokens that is kept (compact)."""
    return {"name": name, "op": "pages", "what": what, "fmt": fmt, "heads": heads, "dim": dim, "page": page,
            "sequences": sequences, "tokens": tokens, "part": part}


def listed():
    return [
        # the queries of one decoding step behind a video; latency counts
        _axes("axes_step", 8, 32, 128, "16,24,24", "parts", "half", "bf16", "forward", True),
        # the queries of a prompt of text and frames, a slice of the fused projection's output
        _axes("axes_video", 8192, 28, 128, "24,20,20", "turns", "half", "bf16", "forward", True),
        # an image encoder's training step in fp32: two axes, neighbouring pairs, odd sizes, output and gradient
        _axes("axes_training", 4111, 16, 96, "24,24", "parts", "interleaved", "fp32", "training", False),
        # one decoding step over the states of 32 recordings
        _cross("cross_step", "e4m3", 32, 16, 1, 64, 64, 1500, 1, False),
        # transcripts' prompts over ragged recordings in 4 bits
        _cross("cross_prompt", "e2m1", 8, 20, 1, 64, 32, 1500, 224, True),
        # text over the tokens of images in high resolution, grouped heads
        _cross("cross_image", "e4m3", 4, 8, 4, 128, 64, 6404, 700, True),
        # five drafted tokens of one user; latency counts
        _verify("verify_one", 1, 6, 32000, "fp32", True, False, False),
        # a batch of chains over a large vocabulary
        _verify("verify_batch", 64, 6, 128001, "fp32", True, False, True),
        # drafted trees in bf16, an odd vocabulary
        _verify("verify_tree", 16, 40, 50001, "bf16", True, True, True),
        # beams: every sequence goes on as eight, those of the step before are freed
        _pages("pages_fork", "fork", "e4m3", 8, 128, 64, 8, 4000, 8.0),
        # a prompt's pages into pages of their own
        _pages("pages_copy", "copy", "e4m3", 8, 128, 64, 4, 16384, 1.0),
        # a copied context of which the tokens that matter are kept
        _pages("pages_compact", "compact", "e2m1", 4, 96, 32, 6, 20001, 0.4),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["axes", "cross", "verify", "pages"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    fmt = rng.choice(["e2m1", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    if op == "axes":
        heads = rng.randint(1, 32)
        tokens = _log(rng, 1, (8192 * 28 * 128) // (heads * dim))
        left, sections = dim // 2, []
        for _ in range(rng.randint(2, 4)):
            sections.append(rng.randint(0, left))
            left -= sections[-1]
        if rng.random() < 0.7:  # the whole head
            sections[-1] += left
        if sum(sections) == 0:
            sections[0] = 1
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "sections": ",".join(map(str, sections)),
                "order": rng.choice(["parts", "turns"]), "layout": rng.choice(["half", "interleaved"]),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "direction": rng.choice(["forward", "training"]),
                "fused": rng.random() < 0.5}
    if op == "cross":
        heads, group = rng.randint(1, 12), rng.randint(1, 6)
        q = rng.choice([1, 1, _log(rng, 2, 700)])
        batch = _log(rng, 1, 32 if q < 64 else 4)
        room = (4 * 8 * 6404 * 128 * 8) // (batch * heads * dim)
        room = min(room, (4 * 8 * 4 * 128 * 6404 * 700) // (batch * heads * group * dim * q))
        return {"op": op, "fmt": fmt, "batch": batch, "heads": heads, "group": group, "dim": dim, "page": page,
                "kv": _log(rng, 1, max(1, min(room, 65536))), "q": q, "ragged": rng.random() < 0.5}
    if op == "verify":
        tree = rng.random() < 0.5
        batch = _log(rng, 1, 32)
        nodes = rng.randint(1, 40) if tree else rng.randint(1, 9)
        vocab = _log(rng, 100, min(200000, (64 * 6 * 128001) // (batch * nodes)))
        return {"op": op, "batch": batch, "nodes": nodes, "vocab": vocab, "dtype": rng.choice(["bf16", "fp32"]),
                "draft": rng.random() < 0.7, "tree": tree, "ragged": rng.random() < 0.5}
    heads, sequences = rng.randint(1, 8), rng.randint(1, 12)
    what = rng.choice(["fork", "copy", "compact"])
    tokens = _log(rng, 1, (4 * 16384 * 8 * 128) // (sequences * heads * dim) // (4 if what == "compact" else 1))
    part = float(rng.randint(1, 8)) if what == "fork" else round(rng.uniform(0.0, 1.0), 3)
    return {"op": op, "what": what, "fmt": fmt, "heads": heads, "dim": dim, "page": page, "sequences": sequences,
            "tokens": tokens, "part": part}


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def _ragged(n, count, ragged):
    """Sizes of `count` sequences, of which the first is the longest."""
    part = [1.0 if b == 0 or not ragged else (b * 0.6180339887498949) % 1.0 for b in range(count)]
    return [max(1, int(n * p)) for p in part]


def work(case):
    if case["op"] == "axes":
        size = 2 if case["dtype"] == "bf16" else 4
        n, passes = case["tokens"] * case["heads"], 2 if case["direction"] == "training" else 1
        pairs, axes = sum(_sections(case)), len(_sections(case))
        return {"bytes": passes * 2 * n * case["dim"] * size + 8 * axes * case["tokens"] + 12 * pairs,
                "flops": passes * 6 * n * pairs}
    if case["op"] == "verify":
        # the sampled position's rows; of the others the drafted tokens' entries alone
        size = 2 if case["dtype"] == "bf16" else 4
        rows = case["batch"] * (2 if case["draft"] else 1)
        return {"bytes": rows * case["vocab"] * size + 32 * case["batch"] * case["nodes"],
                "flops": rows * case["vocab"]}
    code = case["dim"] // (2 if case["fmt"] == "e2m1" else 1) + case["dim"] // 32  # bytes of a token's head
    if case["op"] == "cross":
        kv, q = _ragged(case["kv"], case["batch"], case["ragged"]), _ragged(case["q"], case["batch"], case["ragged"])
        rows = sum(q) * case["heads"] * case["group"]
        pairs = sum(n * m for n, m in zip(kv, q)) * case["heads"] * case["group"]
        return {"bytes": 2 * sum(kv) * case["heads"] * code + 4 * rows * case["dim"], "flops": 4 * pairs * case["dim"]}
    lens = _ragged(case["tokens"], case["sequences"], True)
    token = 2 * case["heads"] * code
    whole = sum(-(-n // case["page"]) for n in lens)  # pages
    if case["what"] == "copy":
        moved = whole * case["page"]
    elif case["what"] == "compact":
        moved = whole * case["page"] + sum(int(n * case["part"]) for n in lens)
    else:
        moved = int(case["part"]) * sum(n % case["page"] for n in lens)
        return {"bytes": 2 * token * moved + 4 * int(case["part"]) * 3 * whole, "flops": 0}
    return {"bytes": 2 * token * moved, "flops": 0}


# ---- inputs ------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _heads(g, tokens, heads, dim, dtype, fused):
    """[tokens, heads, dim] of a projection with some strong channels, alone or as a slice of a wider row."""
    strong = torch.exp(0.7 * torch.randn(dim, generator=g, device="cuda"))
    wide = heads + (2 if fused else 0)
    x = torch.randn((tokens, wide, dim), generator=g, device="cuda", dtype=torch.float32).mul_(strong).to(dtype)
    return x[:, :heads] if fused else x


def _codes(g, fmt, pages, heads, page, dim):
    """Codes and scales of pages full of tokens: normal values with some strong channels, scaled by blocks of 32."""
    codes = torch.empty((pages, heads, page, dim // (2 if fmt == "e2m1" else 1)), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, heads, dim // 32, page), dtype=torch.uint8, device="cuda")
    strong = torch.exp(0.7 * torch.randn(dim, generator=g, device="cuda"))
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // (heads * page * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, heads, page, dim // 32, 32), generator=g, device="cuda")
        x = (x.view(n, heads, page, dim) * strong).view_as(x)
        e = torch.floor(torch.log2(x.abs().amax(-1))) - (2 if fmt == "e2m1" else 8)
        y = (x * torch.exp2(-e)[..., None]).flatten(-2)
        if fmt == "e2m1":
            c = torch.bucketize(y.abs(), border).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
            codes[p:p + n] = c[..., 0::2] + (c[..., 1::2] << 4)
        else:
            codes[p:p + n] = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + n] = (e + 127.0).to(torch.uint8).transpose(2, 3)
    return codes, scales


def _table(order, need):
    """Page numbers [sequences, the longest's pages], taken from `order` one after another, -1 behind them; and how many
    were taken."""
    need = torch.tensor(need, device="cuda")
    j = torch.arange(int(need.max()), device="cuda")
    first = need.cumsum(0) - need
    table = torch.where(j < need[:, None], order[(first[:, None] + j).clamp(max=order.numel() - 1)], -1)
    return table.to(torch.int32), int(need.sum())


def _starts(sizes):
    return torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)


def _probabilities(g, case, total):
    """Rows of the target's and the draft's probabilities: logits with a few strong tokens, the draft's a noisy copy
    of the target's; the tail of either is cut, as by a nucleus, in every other row."""
    v, dtype = case["vocab"], DTYPES[case["dtype"]]
    target = torch.empty((total, v), dtype=dtype, device="cuda")
    draft = torch.empty((total, v), dtype=dtype, device="cuda")
    for r in range(0, total, 32):
        n = min(32, total - r)
        x = 3.0 * torch.randn((n, v), generator=g, device="cuda")
        y = x + 0.8 * torch.randn((n, v), generator=g, device="cuda")
        for z, dst in ((x, target), (y, draft)):
            p = torch.softmax(z, 1)
            p[1::2] = torch.where(p[1::2] > 0.2 / v, p[1::2], 0.0)
            dst[r:r + n] = (p / p.sum(1, keepdim=True)).to(dtype)
    return target, draft


def _draw_tokens(g, rows):
    """A token of each row of probabilities, by its cumulative sum."""
    c = rows.float().cumsum(1)
    u = torch.rand((rows.shape[0], 1), generator=g, device="cuda") * c[:, -1:]
    return torch.searchsorted(c, u, right=True)[:, 0].clamp(max=rows.shape[1] - 1)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "axes":
        sections = _sections(case)
        s["x"] = _heads(g, case["tokens"], case["heads"], case["dim"], DTYPES[case["dtype"]], case["fused"])
        far = torch.tensor([4096 >> (2 * a) for a in range(len(sections))], device="cuda")[:, None]
        at = torch.randint(0, 1 << 40, (len(sections), case["tokens"]), generator=g, device="cuda")
        s["positions"] = at % far + torch.arange(case["tokens"], device="cuda") // 64
        pairs = sum(sections)
        s["inv_freq"] = 1000000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
        axes = torch.arange(len(sections), device="cuda").repeat_interleave(torch.tensor(sections, device="cuda"))
        if case["order"] == "turns":  # t h w t h w ... while an axis has pairs left
            turn = torch.cat([torch.arange(n, device="cuda") for n in sections])
            axes = axes[torch.argsort(turn * len(sections) + axes)]
        s["axes"] = axes.to(torch.int32)
        if case["direction"] == "training":
            s["x"] = s["x"].detach().requires_grad_()
            s["grad"] = _heads(g, case["tokens"], case["heads"], case["dim"], DTYPES[case["dtype"]], False)
        return s
    if case["op"] == "verify":
        sizes = _ragged(case["nodes"], case["batch"], case["ragged"])
        total = sum(sizes)
        s["sizes"], s["q_starts"] = sizes, _starts(sizes)
        s["target"], draft = _probabilities(g, case, total)
        node = torch.cat([torch.arange(n, device="cuda") for n in sizes])
        first = torch.arange(total, device="cuda") - node
        back = torch.rand(total, generator=g, device="cuda")
        # a tree's nodes hang on one of the 12 before them
        parent = node - 1
        if case["tree"]:
            parent = node - 1 - (back * node.clamp(max=12)).long()
        s["parents"] = parent.clamp(min=-1).to(torch.int32) if case["tree"] else None
        s["tokens"] = torch.empty(total, dtype=torch.int64, device="cuda")
        for r in range(0, total, 64):
            s["tokens"][r:r + 64] = _draw_tokens(g, draft[(first + parent.clamp(min=0))[r:r + 64]])
        s["draft"] = draft if case["draft"] else None
        s["uniforms"] = torch.rand(total, generator=g, device="cuda", dtype=torch.float64)
        return s
    heads, dim, page, fmt = case["heads"], case["dim"], case["page"], case["fmt"]
    if case["op"] == "cross":
        s["kv"] = _ragged(case["kv"], case["batch"], case["ragged"])
        s["q_sizes"] = _ragged(case["q"], case["batch"], case["ragged"])
        need = [-(-n // page) for n in s["kv"]]
        pages = sum(need) + 2
        s["table"], _ = _table(torch.randperm(pages, generator=g, device="cuda"), need)
        s["kv_lens"] = torch.tensor(s["kv"], dtype=torch.int32, device="cuda")
        s["q_starts"] = _starts(s["q_sizes"])
        s["q"] = _heads(g, sum(s["q_sizes"]), heads * case["group"], dim, torch.bfloat16, True)
    else:
        s["lens"] = _ragged(case["tokens"], case["sequences"], True)
        need = [-(-n // page) for n in s["lens"]]
        children = int(case["part"]) if case["what"] == "fork" else 1
        pages = sum(need) + (len(need) * children if case["what"] == "fork" else sum(need)) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        s["table"], taken = _table(order, need)
        s["kv_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
        if case["what"] == "fork":
            s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
            s["refs"][order[:taken]] = 1
            s["parents"] = torch.arange(len(need), device="cuda", dtype=torch.int32).repeat_interleave(children)
            s["branches"] = torch.full((len(need) * children, s["table"].shape[1]), -1, dtype=torch.int32,
                                       device="cuda")
            s["none"] = torch.zeros(len(need) * children, dtype=torch.int32, device="cuda")
        else:
            s["src"], s["dst"] = order[:taken].to(torch.int32), order[taken:2 * taken].to(torch.int32)
            s["copy_table"], _ = _table(order[taken:], need)
        if case["what"] == "compact":
            counts = [int(n * case["part"]) for n in s["lens"]]
            s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
            s["kv_starts"] = torch.zeros(len(need), dtype=torch.int32, device="cuda")
            s["keep"] = torch.full((len(need), max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
            for b, (n, m) in enumerate(zip(s["lens"], counts)):
                s["keep"][b, :m] = torch.randperm(n, generator=g, device="cuda")[:m].sort().values
    s["k_codes"], s["k_scales"] = _codes(g, fmt, pages, heads, page, dim)
    s["v_codes"], s["v_scales"] = _codes(g, fmt, pages, heads, page, dim)
    return s


# ---- plain form ----------------------------------------------------------------

def _turn(x, angle, layout, backward):
    """x [tokens, heads, dim] turned by angles [tokens, pairs] (64 bits), in 32 bits."""
    c, t = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if backward:
        t = -t
    h = angle.shape[1]
    f = x.float()
    out = f.clone()
    if layout == "half":
        a, b = f[..., :h], f[..., h:2 * h]
        out[..., :h], out[..., h:2 * h] = a * c - b * t, b * c + a * t
    else:
        a, b = f[..., 0:2 * h:2], f[..., 1:2 * h:2]
        out[..., 0:2 * h:2], out[..., 1:2 * h:2] = a * c - b * t, b * c + a * t
    return out.to(x.dtype)


def _plain_axes(s):
    case = s["case"]
    angle = s["positions"][s["axes"].long()].T.double() * s["inv_freq"]
    y = _turn(s["x"].detach(), angle, case["layout"], False)
    if case["direction"] == "forward":
        return y
    return {"y": y, "x_grad": _turn(s["grad"], angle, case["layout"], True)}


def _values(fmt, device):
    """The value of every code."""
    mbits, bias, bits = (1, 1, 4) if fmt == "e2m1" else (3, 7, 8)
    code = torch.arange(1 << bits, device=device)
    mag = code & ((1 << (bits - 1)) - 1)
    e, m = mag >> mbits, mag & ((1 << mbits) - 1)
    value = torch.ldexp(torch.where(e > 0, m + (1 << mbits), m).float(), e.clamp(min=1) - bias - mbits)
    if fmt == "e4m3":
        value[mag == 127] = float("nan")
    return torch.where(code > mag, -value, value)


def _tokens(s, which, pages):
    """fp32 [batch, heads, tokens, dim] of pages [batch, n] of the cache."""
    fmt = s["case"]["fmt"]
    codes = s[which + "_codes"][pages].transpose(1, 2).flatten(2, 3)
    scales = s[which + "_scales"][pages].permute(0, 2, 1, 4, 3).flatten(2, 3)
    if fmt == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    value = _values(fmt, codes.device)[codes.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(value, scales.int()[..., None] - 127).flatten(-2)


def _plain_cross(s):
    """Sequences are padded to the longest on either side; the padding has no weight and no output."""
    case = s["case"]
    heads, group, dim, batch = case["heads"], case["group"], case["dim"], case["batch"]
    pages = s["table"].long().clamp(min=0)
    k, v = _tokens(s, "k", pages), _tokens(s, "v", pages)
    m = max(s["q_sizes"])
    start, size = s["q_starts"][:-1, None].long(), s["q_starts"].diff()[:, None]
    j = torch.arange(m, device="cuda")
    row = (start + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(batch, m, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)
    score = torch.matmul(q, k.transpose(2, 3)).mul_(dim ** -0.5)
    hidden = torch.arange(k.shape[2], device="cuda") >= s["kv_lens"][:, None]
    score.masked_fill_(hidden[:, None, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.matmul(p / p.sum(-1, keepdim=True), v).view(batch, heads, group, m, dim).permute(0, 3, 1, 2, 4)
    return o.reshape(batch, m, heads * group, dim)[j < size].bfloat16()


def _plain_verify(s):
    """Nodes q_starts[b] .. of sequence b: the first is the last token that is settled, the others are drafted, each
    with a parent before it.  From the first node on, at a node c with weights w = target[c] (sum W = 1 to begin with)
    its children are asked in their order: child i with token x is kept if uniforms[i] * W * q(x) < w(x), where q is
    draft[c], or without a draft's probabilities 1 for x and 0 for all others; then c = i.  If not, w becomes
    max(w - W q, 0) and W its sum (without any rest w stays as it was, and so it does for later children).  At the
    node that no child follows, the token is sampled from w: the first whose cumulative sum is above
    uniforms[first node] * sum(w).  Sums are of 64 bits."""
    case, sizes = s["case"], s["sizes"]
    b, m, v = case["batch"], max(s["sizes"]), case["vocab"]
    start, size = s["q_starts"][:-1].long(), s["q_starts"].diff().long()
    j = torch.arange(m, device="cuda")
    row = (start[:, None] + j).clamp(max=sum(sizes) - 1)
    there = j < size[:, None]
    token, u = s["tokens"][row], s["uniforms"][row]
    seq = torch.arange(b, device="cuda")
    path = torch.where(j == 0, 0, torch.full((b, m), -1, device="cuda"))
    out = torch.full((b, m), -1, device="cuda")
    kept = torch.zeros(b, dtype=torch.long, device="cuda")
    if s["parents"] is None:
        at = row[:, :-1]  # the parents' rows
        x = token[:, 1:]
        p = s["target"][at, x].double()
        q = s["draft"][at, x].double() if s["draft"] is not None else torch.ones_like(p)
        keep = (there[:, 1:] & (u[:, 1:] * q < p)).long().cumprod(1)
        kept = keep.sum(1)
        path[:, 1:] = torch.where(keep == 1, j[1:], -1)
        out[:, :-1] = torch.where(keep == 1, x, -1)
        w = s["target"][start + kept].double()
        fails = kept + 1 < size
        x = token[seq, (kept + 1).clamp(max=m - 1)]
        if s["draft"] is not None:
            rest = (w - s["draft"][start + kept].double()).clamp(min=0)
        else:
            rest = w.clone()
            rest[seq, x] = 0.0
        w = torch.where((fails & (rest.sum(1) > 0))[:, None], rest, w)
    else:
        parent = s["parents"][row].long()
        c = torch.zeros(b, dtype=torch.long, device="cuda")
        w, total = s["target"][start].double(), torch.ones(b, dtype=torch.float64, device="cuda")
        for i in range(1, m):
            asked = there[:, i] & (parent[:, i] == c)
            x = token[:, i]
            q = s["draft"][start + c].double() if s["draft"] is not None else None
            qx = q[seq, x] if q is not None else torch.ones_like(total)
            keep = asked & (u[:, i] * total * qx < w[seq, x])
            if q is not None:
                rest = (w - total[:, None] * q).clamp(min=0)
            else:
                rest = w.clone()
                rest[seq, x] = 0.0
            left = rest.sum(1)
            lose = asked & ~keep & (left > 0)
            w = torch.where(keep[:, None], s["target"][row[:, i]].double(), torch.where(lose[:, None], rest, w))
            total = torch.where(keep, 1.0, torch.where(lose, left, total))
            kept = kept + keep
            path[seq, kept] = torch.where(keep, i, path[seq, kept])
            out[seq, (kept - 1).clamp(min=0)] = torch.where(keep, x, out[seq, (kept - 1).clamp(min=0)])
            c = torch.where(keep, i, c)
    cum = w.cumsum(1)
    chosen = torch.searchsorted(cum, u[:, :1] * cum[:, -1:], right=True)[:, 0]
    last = v - 1 - (w.flip(1) > 0).int().argmax(1)
    out[seq, kept] = torch.minimum(chosen, last)
    return {"counts": (kept + 1).to(torch.int32), "path": path.to(torch.int32), "tokens": out}


NAMES = ("k_codes", "k_scales", "v_codes", "v_scales")


def _copy_pages(s, src, dst):
    for n in NAMES:
        s[n][dst.long()] = s[n][src.long()]


def _plain_fork(s):
    page = s["case"]["page"]
    refs, table, pages = s["refs"], s["table"], s["refs"].numel()
    held = s["branches"].flatten().long()
    held = held[held >= 0]
    refs.index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    s["branches"].fill_(-1)
    parent = s["parents"].long()
    n = s["kv_lens"][parent].long()
    full, rows = n // page, n % page
    j = torch.arange(table.shape[1], device="cuda")
    new = torch.where(j < full[:, None], table[parent], -1)
    shared = new.flatten().long()
    shared = shared[shared >= 0]
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    needs = rows > 0
    place = needs.long().cumsum(0) - 1
    free = torch.argsort((refs != 0).int(), stable=True)
    got = needs & (place < (refs == 0).sum())
    taken = free[place.clamp(min=0, max=pages - 1)]
    child = torch.arange(parent.numel(), device="cuda")[got]
    new[child, full[got]] = taken[got].int()
    refs[taken[got]] = 1
    # rows of the last page
    src = table[parent, full.clamp(max=table.shape[1] - 1)][got].long()
    inside = torch.arange(page, device="cuda") < rows[got][:, None]
    at, row = inside.nonzero(as_tuple=True)
    for n in ("k", "v"):
        s[n + "_codes"][taken[got][at], :, row] = s[n + "_codes"][src[at], :, row]
        s[n + "_scales"][taken[got][at], :, :, row] = s[n + "_scales"][src[at], :, :, row]
    s["branches"] = new
    return {"table": new, "missing": (needs & ~got).int(), "refs": refs}


def _plain_compact(s):
    page = s["case"]["page"]
    _copy_pages(s, s["src"], s["dst"])
    table, keep = s["copy_table"].long(), s["keep"].long()
    i = torch.arange(keep.shape[1], device="cuda").expand_as(keep)
    kept = i < s["counts"][:, None]
    b = torch.arange(keep.shape[0], device="cuda")[:, None].expand_as(keep)[kept]
    old, new = (s["kv_starts"][:, None] + keep)[kept], (s["kv_starts"][:, None] + i)[kept]
    p, r, pn, rn = table[b, old // page], old % page, table[b, new // page], new % page
    for n in ("k", "v"):
        codes, scales = s[n + "_codes"], s[n + "_scales"]
        c, e = codes[p, :, r], scales[p, :, :, r]
        codes[pn, :, rn] = c
        scales[pn, :, :, rn] = e
    return {"kv_lens": s["kv_starts"] + s["counts"]}


def _plain_pages(s):
    what = s["case"]["what"]
    if what == "fork":
        out = _plain_fork(s)
    elif what == "compact":
        out = _plain_compact(s)
    else:
        _copy_pages(s, s["src"], s["dst"])
        out = {}
    return {**out, **_bytes(s)}


def _bytes(s):
    """The cache itself.  Its codes are moved and never computed, so they are compared as they are."""
    return {n: s[n] for n in NAMES}


# ---- the framework's calls -------------------------------------------------------

def _own(s):
    import microscaling_quantize_dequantize_amd as mx
    case = s["case"]
    if case["op"] == "axes":
        layout = mx.HALF if case["layout"] == "half" else mx.INTERLEAVED
        y = mx.mx_rope(s["x"], s["positions"], s["inv_freq"], layout=layout, axes=s["axes"])
        if case["direction"] == "forward":
            return y
        return {"y": y.detach(), "x_grad": torch.autograd.grad(y, s["x"], s["grad"])[0]}
    if case["op"] == "verify":
        counts, path, tokens = mx.mx_verify(s["target"], s["tokens"], s["uniforms"], s["q_starts"],
                                            max_q=max(s["sizes"]), draft=s["draft"], parents=s["parents"])
        return {"counts": counts, "path": path, "tokens": tokens}
    if "cache" not in s:
        fmt = mx.E2M1 if case["fmt"] == "e2m1" else mx.E4M3
        s["cache"] = mx.MXCache(fmt, *(s[n] for n in NAMES))
    cache = s["cache"]
    if case["op"] == "cross":
        return mx.mx_cache_cross_attention(cache, s["q"], s["q_starts"], s["kv_lens"], s["table"],
                                           max_q=max(s["q_sizes"]), max_kv=max(s["kv"]))
    if case["what"] == "fork":
        mx.mx_cache_resize(cache, s["refs"], s["branches"], s["none"])
        s["branches"], missing = mx.mx_cache_fork(cache, s["refs"], s["table"], s["kv_lens"], s["parents"])
        out = {"table": s["branches"], "missing": missing, "refs": s["refs"]}
    else:
        mx.mx_cache_copy(cache, s["src"], s["dst"])
        out = {}
        if case["what"] == "compact":
            out["kv_lens"] = mx.mx_cache_compact(cache, s["kv_starts"], s["keep"], s["counts"], s["copy_table"])
    return {**out, **_bytes(s)}


def run(state):
    if own:
        return _own(state)
    return {"axes": _plain_axes, "cross": _plain_cross, "verify": _plain_verify,
            "pages": _plain_pages}[state["case"]["op"]](state)


# ---- exact values ------------------------------------------------------------------

def _exact_turn(x, angle, layout, sign):
    """Pairs as complex numbers times exp(+-i angle), 64 bits each part."""
    h = angle.shape[1]
    x = x.detach().double()
    head = x[..., :2 * h]
    pairs = head.unflatten(-1, (2, h)).transpose(-1, -2) if layout == "half" else head.unflatten(-1, (h, 2))
    turn = torch.polar(torch.ones_like(angle), sign * angle)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    head = z.transpose(-1, -2).flatten(-2) if layout == "half" else z.flatten(-2)
    return torch.cat((head, x[..., 2 * h:]), -1)


def _exact_values(fmt):
    """Every code's value: the non-negative ones in ascending order, then their negatives."""
    if fmt == "e2m1":
        grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        grid = [m / 512.0 for m in range(8)]
        grid += [(1.0 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1] + [math.nan]
    grid = torch.tensor(grid, dtype=torch.float64, device="cuda")
    return torch.cat((grid, -grid))


def _exact_tokens(s, which, b, n):
    """64-bit values [n, heads, dim] of a sequence's tokens."""
    fmt, page = s["case"]["fmt"], s["case"]["page"]
    t = torch.arange(n, device="cuda")
    p, r = s["table"][b].long()[t // page], t % page
    codes = s[which + "_codes"][p, :, r]
    if fmt == "e2m1":
        pair = torch.empty((*codes.shape, 2), dtype=torch.uint8, device="cuda")
        pair[..., 0], pair[..., 1] = codes % 16, codes // 16
        codes = pair.flatten(-2)
    unit = torch.exp2(s[which + "_scales"][p, :, :, r].double() - 127.0)
    return (torch.take(_exact_values(fmt), codes.long()).unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "axes":
        angle = torch.empty((case["tokens"], s["axes"].numel()), dtype=torch.float64, device="cuda")
        for p, (axis, f) in enumerate(zip(s["axes"].tolist(), s["inv_freq"].tolist())):
            angle[:, p] = s["positions"][axis].double() * f
        y = _exact_turn(s["x"], angle, case["layout"], 1.0)
        if case["direction"] == "forward":
            return y
        return {"y": y, "x_grad": _exact_turn(s["grad"], angle, case["layout"], -1.0)}
    if case["op"] != "cross":
        return None  # whole numbers, compared as they are
    heads, group, dim = case["heads"], case["group"], case["dim"]
    out = []
    for b, (n, m) in enumerate(zip(s["kv"], s["q_sizes"])):
        k, v = _exact_tokens(s, "k", b, n), _exact_tokens(s, "v", b, n)
        first = sum(s["q_sizes"][:b])
        mine = torch.empty((m, heads * group, dim), dtype=torch.float64, device="cuda")
        for h in range(heads * group):
            x = s["q"][first:first + m, h].double() @ k[:, h // group].T / math.sqrt(dim)
            mine[:, h] = torch.softmax(x, 1) @ v[:, h // group]
        out.append(mine)
    return torch.cat(out)
