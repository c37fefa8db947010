"""The measured cases of the serving operators: rotary positions, the paged
MX cache (write and read back) and attention over it.

Three operators, each in a plain form (elementary torch operations) and as a
user's program calls it:

  rope       y = R(position) x on some or all of a head's dimensions, and the
             gradient of x, which is the transposed rotation of that of y.
  cache      keys (rotated on the way) and values are quantised to MXFP8 or
             MXFP4 and written into pages; tokens are read back to bf16.
  attention  queries of one new token, of a tree of drafted tokens or of a
             chunk of a prompt attend to a sequence's pages.

The cache's layout, for `pages` pages of `page` tokens, H key/value heads of
D dimensions, kept apart for keys and values:
  codes   [pages, H, page, D] bytes (MXFP8), [pages, H, page, D/2] (MXFP4,
          the even dimension in the low nibble)
  scales  [pages, H, D/32, page] E8M0 bytes, one for each 32 dimensions.
Token t of a sequence is in page block_table[t // page], row t % page; its
slot is page * page_size + row.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# element formats: mantissa bits, lowest normal exponent, highest exponent, bias, largest value
FORMATS = {"e2m1": (1, 0, 2, 1, 6.0), "e4m3": (3, -6, 8, 7, 448.0)}


# ---- cases -------------------------------------------------------------------

def _rope(name, tokens, heads, dim, rot, layout, dtype, direction, far, fused):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot, "layout": layout,
            "dtype": dtype, "direction": direction, "far": far, "fused": fused}


def _cache(name, fmt, new, context, heads, dim, page, rot, layout, far):
    return {"name": name, "op": "cache", "fmt": fmt, "new": new, "context": context, "heads": heads, "dim": dim,
            "page": page, "rot": rot, "layout": layout, "far": far}


def _attention(name, fmt, batch, heads, group, dim, page, kv, nodes, mask, ragged):
    return {"name": name, "op": "attention", "fmt": fmt, "batch": batch, "heads": heads, "group": group, "dim": dim,
            "page": page, "kv": kv, "nodes": nodes, "mask": mask, "ragged": ragged}


def listed():
    return [
        # the queries of one decoding step of a small batch, far into a long context; latency counts
        _rope("rope_step", 8, 32, 128, 128, "half", "bf16", "forward", 131072, True),
        # the queries of a prompt, a slice of the fused projection's output
        _rope("rope_prompt", 8192, 64, 128, 128, "half", "bf16", "forward", 8192, True),
        # a training step's gradient in fp32: neighbouring pairs, half of each head rotated, odd sizes
        _rope("rope_gradient", 4111, 16, 96, 48, "interleaved", "fp32", "backward", 65536, False),
        # one decoding step of a batch: 64 tokens are written and read back
        _cache("cache_step", "e4m3", 64, 0, 8, 128, 64, 128, "half", 131072),
        # a prompt in one go into 4 bits, and back for the attention among its own tokens
        _cache("cache_prompt", "e2m1", 16384, 0, 8, 128, 64, 128, "half", 16384),
        # a chunk behind a cached prefix, all of it read back; 5 heads of 96, neighbouring pairs on 32 of them
        _cache("cache_prefix", "e4m3", 1003, 70001, 5, 96, 16, 32, "interleaved", 1 << 20),
        # one sequence, one token: the smallest step
        _attention("attend_one", "e4m3", 1, 8, 4, 128, 64, 1999, 1, "causal", False),
        # a batch of ragged sequences, one new token each
        _attention("attend_batch", "e4m3", 64, 8, 4, 128, 64, 16384, 1, "causal", True),
        # one long document in 4 bits
        _attention("attend_long", "e2m1", 1, 8, 8, 128, 128, 500001, 1, "causal", False),
        # verification of drafted trees of 64 nodes
        _attention("attend_tree", "e4m3", 8, 8, 8, 128, 64, 8192, 64, "tree", True),
        # small trees on heads of 64 in 4 bits
        _attention("attend_small_tree", "e2m1", 16, 4, 7, 64, 16, 4001, 13, "tree", True),
        # a chunk of a prompt over what is cached before it, heads of 256
        _attention("attend_chunk", "e4m3", 2, 4, 4, 256, 32, 12000, 1000, "causal", True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attention", "attention"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        heads = rng.randint(1, 64)
        tokens = _log(rng, 1, max(1, (8192 * 64 * 128) // (heads * dim)) if heads * dim > 1024 else 65536)
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "rot": rot, "layout": layout,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "direction": rng.choice(["forward", "backward"]),
                "far": _log(rng, 1024, 1 << 20), "fused": rng.random() < 0.5}
    fmt = rng.choice(["e2m1", "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        heads = rng.randint(1, 16)
        room = (16384 * 8 * 128) // (heads * dim)
        new = _log(rng, 1, max(1, room // 2))
        context = rng.choice([0, _log(rng, 1, max(1, room - new))])
        return {"op": op, "fmt": fmt, "new": new, "context": context, "heads": heads, "dim": dim, "page": page,
                "rot": rng.choice([0, dim, dim // 2, 2 * rng.randint(1, dim // 2)]), "layout": layout,
                "far": _log(rng, 1024, 1 << 20)}
    heads, group = rng.randint(1, 8), rng.randint(1, 8)
    mask, nodes = rng.choice([("causal", 1), ("causal", 1), ("tree", rng.randint(2, 100)),
                              ("causal", _log(rng, 2, 1000))])
    batch = _log(rng, 1, 64 if nodes < 128 else 4)
    room = (64 * 8192 * 8 * 128) // (batch * heads * dim)
    if nodes > 1:
        room = min(room, (1000 * 8000 * 2 * 16 * 256) // (nodes * batch * heads * group * dim))
    kv = max(nodes, _log(rng, 1, max(1, min(room, 262144))))
    return {"op": op, "fmt": fmt, "batch": batch, "heads": heads, "group": group, "dim": dim, "page": page, "kv": kv,
            "nodes": nodes, "mask": mask, "ragged": rng.random() < 0.5}


def _lengths(case):
    """Tokens of each sequence and new tokens of each, the new ones included in the first."""
    kv, nodes = [], []
    for b in range(case["batch"]):
        part = 1.0
        if case["ragged"] and b:
            part = (b * 0.6180339887498949) % 1.0
        q = max(1, int(case["nodes"] * (0.5 + 0.5 * part)))
        nodes.append(q)
        kv.append(max(q, int(case["kv"] * part)))
    return kv, nodes


def work(case):
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 8 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    code = case["dim"] // (2 if case["fmt"] == "e2m1" else 1) + case["dim"] // 32  # bytes of a token's head
    if case["op"] == "cache":
        new, both = case["new"] * case["heads"], (case["new"] + case["context"]) * case["heads"]
        return {"bytes": 2 * new * (2 * case["dim"] + code) + 2 * both * (code + 2 * case["dim"]) + 24 * case["new"],
                "flops": 3 * new * case["rot"]}
    kv, nodes = _lengths(case)
    rows = sum(nodes) * case["heads"] * case["group"]
    pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(kv, nodes)) * case["heads"] * case["group"]
    return {"bytes": 2 * sum(kv) * case["heads"] * code + 4 * rows * case["dim"], "flops": 4 * pairs * case["dim"]}


# ---- inputs ------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _frequencies(rot, far):
    """Angles per position of each pair, and the factor on the rotated values.  Contexts beyond 8192 positions are
    scaled by parts: slow pairs are interpolated, fast ones kept, those between mixed."""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    if far <= 8192:
        return inv, 1.0
    factor = far / 8192.0
    turns = 8192.0 * inv / (2.0 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return inv * (keep + (1.0 - keep) / factor), 0.1 * math.log(factor) + 1.0


def _heads(g, tokens, heads, dim, dtype, fused):
    """[tokens, heads, dim] of a projection with some strong channels, alone or as a slice of a wider row."""
    strong = torch.exp(0.7 * torch.randn(dim, generator=g, device="cuda"))
    wide = heads + (2 if fused else 0)
    x = torch.randn((tokens, wide, dim), generator=g, device="cuda", dtype=torch.float32).mul_(strong).to(dtype)
    return x[:, :heads] if fused else x


def _filled_pages(g, fmt, pages, heads, page, dim):
    """Codes and scales of pages full of tokens."""
    codes = torch.empty((pages, heads, page, dim // (2 if fmt == "e2m1" else 1)), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, heads, dim // 32, page), dtype=torch.uint8, device="cuda")
    strong = torch.exp(0.7 * torch.randn(dim, generator=g, device="cuda"))
    step = max(1, (1 << 27) // (heads * page * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, heads, page, dim), generator=g, device="cuda").mul_(strong).bfloat16().float()
        c, s = _quantise(fmt, x)
        codes[p:p + n] = c
        scales[p:p + n] = s.transpose(2, 3)
    return codes, scales


def _tree(g, nodes):
    """Which of its sequence's drafted tokens each sees: itself and its ancestors in a random tree."""
    parents = (torch.rand(nodes, generator=g, device="cuda") * torch.arange(nodes, device="cuda")).long().tolist()
    seen = torch.zeros((nodes, nodes), dtype=torch.bool)
    for i in range(nodes):
        if i:
            seen[i] = seen[parents[i]]
        seen[i, i] = True
    return seen


def _words(seen, width):
    """Truth values [rows, n] as rows of 64-bit words, bit j of word w for column 64 w + j."""
    full = torch.zeros((seen.shape[0], width * 64), dtype=torch.int64)
    full[:, :seen.shape[1]] = seen.long()
    return (full.view(-1, width, 64) << torch.arange(64)).sum(2)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "rope":
        s["x"] = _heads(g, case["tokens"], case["heads"], case["dim"], DTYPES[case["dtype"]], case["fused"])
        s["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device="cuda")
        s["inv_freq"], s["scale"] = _frequencies(case["rot"], case["far"])
        return s
    heads, dim, page, fmt = case["heads"], case["dim"], case["page"], case["fmt"]
    if case["op"] == "cache":
        total = case["new"] + case["context"]
        pages = -(-total // page) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        token = torch.arange(total, device="cuda")
        s["slots"] = order[token // page] * page + token % page
        s["new_slots"] = s["slots"][case["context"]:].clone()
        s["k"] = _heads(g, case["new"], heads, dim, torch.bfloat16, True)
        s["v"] = _heads(g, case["new"], heads, dim, torch.bfloat16, True)
        s["positions"] = torch.randint(0, case["far"], (case["new"],), generator=g, device="cuda")
        s["inv_freq"], s["scale"] = _frequencies(case["rot"], case["far"])
    else:
        kv, nodes = _lengths(case)
        need = [-(-n // page) for n in kv]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((case["batch"], max(need)), dtype=torch.int32, device="cuda")
        first = 0
        for b, n in enumerate(need):
            table[b, :n] = order[first:first + n]
            first += n
        s["q"] = _heads(g, sum(nodes), heads * case["group"], dim, torch.bfloat16, True)
        s["kv"], s["nodes"], s["table"] = kv, nodes, table
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        starts = [0]
        for q in nodes:
            starts.append(starts[-1] + q)
        s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["tree"] = None
        if case["mask"] == "tree":
            width = -(-max(nodes) // 64)
            s["tree"] = torch.cat([_words(_tree(g, q), width) for q in nodes]).cuda()
    s["k_codes"], s["k_scales"] = _filled_pages(g, fmt, pages, heads, page, dim)
    s["v_codes"], s["v_scales"] = _filled_pages(g, fmt, pages, heads, page, dim)
    if own:
        s["cache"] = _handle(s)
    return s


# ---- plain form ----------------------------------------------------------------

def _rotate(x, positions, inv_freq, scale, layout, backward):
    """The rotation of x [tokens, heads, dim] in the type of x; angles in 64 bits."""
    angle = positions.double()[:, None] * inv_freq
    c = (angle.cos() * scale).to(x.dtype)[:, None]
    s = (angle.sin() * scale).to(x.dtype)[:, None]
    if backward:
        s = -s
    h = inv_freq.numel()
    out = x.clone()
    if layout == "half":
        a, b = x[..., :h], x[..., h:2 * h]
        out[..., :h], out[..., h:2 * h] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        out[..., 0:2 * h:2], out[..., 1:2 * h:2] = a * c - b * s, b * c + a * s
    return out


def _quantise(fmt, x):
    """MX codes (packed) and scale bytes of fp32 x [..., dim]: one power of two for each 32 dimensions."""
    mbits, emin, emax, _, top = FORMATS[fmt]
    g = x.reshape(*x.shape[:-1], -1, 32)
    e = (g.abs().amax(-1).view(torch.int32) >> 23) - 127 - emax
    e = e.clamp(min=-127)
    y = torch.ldexp(g, -e[..., None])
    mag = y.abs()
    ey = ((mag.view(torch.int32) >> 23) - 127).clamp(min=emin)
    m = torch.round(torch.ldexp(mag, mbits - ey)).int()  # ties to even
    code = ((ey - emin) << mbits) + m
    largest = (2 << mbits) - 2 if fmt == "e4m3" else 3  # mantissa of 448 and of 6
    code = code.clamp(max=((emax - emin) << mbits) + largest)
    sign = (y.view(torch.int32) < 0).int()
    code = code + (sign << (3 if fmt == "e2m1" else 7))
    code = code.reshape(x.shape)
    if fmt == "e2m1":
        code = code[..., 0::2] + (code[..., 1::2] << 4)
    return code.to(torch.uint8), (e + 127).to(torch.uint8)


def _dequantise(fmt, codes, scales):
    """fp32 values of codes [..., dim or dim/2] with scales [..., dim/32]."""
    if fmt == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    value = _values(fmt, codes.device)[codes.int()]
    value = value.view(*value.shape[:-1], -1, 32)
    return torch.ldexp(value, scales.int()[..., None] - 127).flatten(-2)


def _values(fmt, device):
    """The value of every code."""
    mbits, _, _, bias, _ = FORMATS[fmt]
    bits = 4 if fmt == "e2m1" else 8
    code = torch.arange(1 << bits, device=device)
    mag = code & ((1 << (bits - 1)) - 1)
    e, m = mag >> mbits, mag & ((1 << mbits) - 1)
    full = torch.where(e > 0, m + (1 << mbits), m)
    value = torch.ldexp(full.float(), e.clamp(min=1) - bias - mbits)
    if fmt == "e4m3":
        value[mag == 127] = float("nan")
    return torch.where(code > mag, -value, value)


def _plain_cache(s):
    case = s["case"]
    page, fmt = case["page"], case["fmt"]
    k, v = s["k"], s["v"]
    if case["rot"]:
        # in 64 bits: the rounding to bf16 and on to 8 or 4 bits has borders
        k = _rotate(k.double(), s["positions"], s["inv_freq"], s["scale"], case["layout"], False).bfloat16()
    p, row = s["new_slots"] // page, s["new_slots"] % page
    for x, codes, scales in ((k, s["k_codes"], s["k_scales"]), (v, s["v_codes"], s["v_scales"])):
        c, e = _quantise(fmt, x.float())
        codes[p, :, row] = c
        scales[p, :, :, row] = e
    p, row = s["slots"] // page, s["slots"] % page
    return {n: _dequantise(fmt, s[n + "_codes"][p, :, row], s[n + "_scales"][p, :, :, row]).bfloat16()
            for n in ("k", "v")}


def _tokens(s, b, n, which):
    """fp32 [heads, n, dim]: the first n tokens of sequence b."""
    case = s["case"]
    pages = s["table"][b, :-(-n // case["page"])].long()
    codes = s[which + "_codes"][pages].transpose(0, 1).flatten(1, 2)[:, :n]
    scales = s[which + "_scales"][pages].permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
    return _dequantise(case["fmt"], codes, scales)


def _plain_attention(s):
    case = s["case"]
    heads, group, dim = case["heads"], case["group"], case["dim"]
    out = torch.empty((s["q"].shape[0], heads * group, dim), dtype=torch.bfloat16, device="cuda")
    first = 0
    for b, (n, q) in enumerate(zip(s["kv"], s["nodes"])):
        k, v = _tokens(s, b, n, "k"), _tokens(s, b, n, "v")
        rows = s["q"][first:first + q].float().view(q, heads, group, dim).permute(1, 2, 0, 3).reshape(heads, -1, dim)
        score = torch.matmul(rows, k.transpose(1, 2)).mul_(dim ** -0.5).view(heads, group, q, n)
        if s["tree"] is None:
            seen = torch.ones((q, q), dtype=torch.bool, device="cuda").tril()
        else:
            j = torch.arange(q, device="cuda")
            seen = (s["tree"][first:first + q][:, j // 64] >> (j % 64)) & 1 == 1
        score[..., n - q:].masked_fill_(~seen, float("-inf"))
        p = torch.exp(score - score.amax(-1, keepdim=True))
        p = (p / p.sum(-1, keepdim=True)).view(heads, group * q, n)
        o = torch.matmul(p, v).view(heads, group, q, dim).permute(2, 0, 1, 3)
        out[first:first + q] = o.reshape(q, heads * group, dim).bfloat16()
        first += q
    return out


# ---- the framework's calls -------------------------------------------------------

def _handle(s):
    import microscaling_quantize_dequantize_amd as mx
    fmt = mx.E2M1 if s["case"]["fmt"] == "e2m1" else mx.E4M3
    return mx.MXCache(fmt, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])


def _own(s):
    import microscaling_quantize_dequantize_amd as mx
    case = s["case"]
    if case["op"] == "rope":
        layout = mx.HALF if case["layout"] == "half" else mx.INTERLEAVED
        return mx.mx_rope(s["x"], s["positions"], s["inv_freq"], layout=layout, scale=s["scale"],
                          inverse=case["direction"] == "backward")
    if "cache" not in s:
        s["cache"] = _handle(s)
    if case["op"] == "cache":
        if case["rot"]:
            layout = mx.HALF if case["layout"] == "half" else mx.INTERLEAVED
            mx.mx_cache_write(s["cache"], s["k"], s["v"], s["new_slots"], positions=s["positions"],
                              inv_freq=s["inv_freq"], layout=layout, scale=s["scale"])
        else:
            mx.mx_cache_write(s["cache"], s["k"], s["v"], s["new_slots"])
        k, v = mx.mx_cache_read(s["cache"], s["slots"])
        return {"k": k, "v": v}
    return mx.mx_cache_attention(s["cache"], s["q"], s["q_starts"], s["kv_lens"], s["table"],
                                 max_q=max(s["nodes"]), max_kv=max(s["kv"]), tree=s["tree"])


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "rope":
        y = _rotate(state["x"].float(), state["positions"], state["inv_freq"], state["scale"], case["layout"],
                    case["direction"] == "backward")
        return y.to(state["x"].dtype)
    return _plain_cache(state) if case["op"] == "cache" else _plain_attention(state)


# ---- exact values ------------------------------------------------------------------

def _grid(fmt):
    """The format's non-negative values in ascending order, and for each whether its mantissa is even."""
    if fmt == "e2m1":
        grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        grid = [m / 512.0 for m in range(8)]
        grid += [(1.0 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
    return torch.tensor(grid, dtype=torch.float64, device="cuda")


def _exact_qdq(fmt, x):
    """x (64 bits) [..., dim] on the MX grid: nearest grid value by bisection, ties to the even code."""
    grid = _grid(fmt)
    blocks = x.unflatten(-1, (-1, 32))
    _, e = torch.frexp(blocks.abs().amax(-1, keepdim=True))  # amax in [2^(e-1), 2^e)
    zero = blocks.abs().amax(-1, keepdim=True) == 0
    e = torch.where(zero, -127, (e - 1 - (2 if fmt == "e2m1" else 8)).clamp(min=-127))
    unit = torch.exp2(e.double())
    mag = (blocks.abs() / unit).clamp(max=float(grid[-1]))
    up = torch.searchsorted(grid, mag.contiguous()).clamp(max=grid.numel() - 1)
    down = (up - 1).clamp(min=0)
    over, under = grid[up] - mag, mag - grid[down]
    take_up = (over < under) | ((over == under) & (up % 2 == 0))
    q = torch.where(take_up, grid[up], grid[down])
    return (torch.where(blocks < 0, -q, q) * unit).flatten(-2)


def _exact_rope(x, positions, inv_freq, scale, layout, backward):
    """Pairs as complex numbers times scale exp(+-i angle), 64 bits each part."""
    h = inv_freq.numel()
    x = x.double()
    head = x[..., :2 * h]
    pairs = head.unflatten(-1, (2, h)).transpose(-1, -2) if layout == "half" else head.unflatten(-1, (h, 2))
    turn = torch.polar(torch.full((positions.numel(), h), scale, dtype=torch.float64, device="cuda"),
                       (-1.0 if backward else 1.0) * torch.outer(positions.double(), inv_freq))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    head = z.transpose(-1, -2).flatten(-2) if layout == "half" else z.flatten(-2)
    return torch.cat((head, x[..., 2 * h:]), -1)


def _code_values(fmt):
    """Every code's value, from its sign and its place in the grid."""
    grid = _grid(fmt)
    if fmt == "e4m3":
        grid = torch.cat((grid, grid.new_full((1,), float("nan"))))
    return torch.cat((grid, -grid))


def _exact_tokens(s, which, pages, rows):
    """64-bit values [n, heads, dim] of tokens by page and row."""
    fmt = s["case"]["fmt"]
    codes = s[which + "_codes"][pages, :, rows]
    if fmt == "e2m1":
        pair = torch.empty((*codes.shape, 2), dtype=torch.uint8, device="cuda")
        pair[..., 0], pair[..., 1] = codes % 16, codes // 16
        codes = pair.flatten(-2)
    value = torch.take(_code_values(fmt), codes.long())
    unit = torch.exp2(s[which + "_scales"][pages, :, :, rows].double() - 127.0)
    return (value.unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s["x"], s["positions"], s["inv_freq"], s["scale"], case["layout"],
                           case["direction"] == "backward")
    page = case["page"]
    if case["op"] == "cache":
        out = {}
        for n in ("k", "v"):
            x = s[n].double()
            if n == "k" and case["rot"]:
                # the keys are held in bf16 between the rotation and the quantisation
                x = _exact_rope(x, s["positions"], s["inv_freq"], s["scale"], case["layout"], False).bfloat16().double()
            old = s["slots"][:case["context"]]
            out[n] = torch.cat((_exact_tokens(s, n, old // page, old % page), _exact_qdq(case["fmt"], x)))
        return out
    heads, group, dim = case["heads"], case["group"], case["dim"]
    out = []
    first = 0
    for b, (n, q) in enumerate(zip(s["kv"], s["nodes"])):
        token = torch.arange(n, device="cuda")
        pages, rows = s["table"][b].long()[token // page], token % page
        see = torch.ones((q, n), dtype=torch.bool, device="cuda")
        for i in range(q):
            if s["tree"] is None:
                see[i, n - q + i + 1:] = False
            else:
                words = s["tree"][first + i].tolist()
                see[i, n - q:] = torch.tensor([words[j // 64] >> (j % 64) & 1 == 1 for j in range(q)], device="cuda")
        mine = torch.empty((q, heads * group, dim), dtype=torch.float64, device="cuda")
        k, v = _exact_tokens(s, "k", pages, rows), _exact_tokens(s, "v", pages, rows)
        for h in range(heads * group):
            x = s["q"][first:first + q, h].double() @ k[:, h // group].T / math.sqrt(dim)
            weight = torch.softmax(torch.where(see, x, float("-inf")), 1)
            mine[:, h] = weight @ v[:, h // group]
        out.append(mine)
        first += q
    return torch.cat(out)
