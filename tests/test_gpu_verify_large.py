"""mx_verify where rows are several workgroups' and trees have more nodes to see to than workgroups: special values,
borders and refusals that leave nothing over 40001 entries, batches whose waves have two shares each, and bushy trees of
many sequences."""
import math

import pytest
import torch

import _verifyref as V
from test_gpu_verify import Case, mx  # noqa: F401

pytestmark = pytest.mark.gpu
WIDE = 40001


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_probabilities_that_are_none(mx, dtype, draft, tree):
    """NaN, infinite and negative entries, and rows of nothing."""
    c = Case([4, 3, 3, 2], WIDE, dtype, tree, draft, seed=17)
    bad = torch.tensor([math.nan, math.inf, -math.inf, -0.25], dtype=dtype, device="cuda").repeat(910)
    for t in (c.target, c.draft):
        if t is not None:
            t[:, 3::11] = bad[:t[:, 3::11].shape[1]]
    c.check(c.run(mx))
    c.target[7:10] = math.nan
    c.target[10:] = 0.0
    want = c.check(c.run(mx))
    assert want[2][2:, 0].tolist() == [-1, -1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_borders_of_the_sample(mx, dtype, offset):
    """Few entries with weight, the first and the last among them: goals on each border, below it, and behind the last."""
    at = [0, 1, 1023, 1024, 4096, 20000, 32768, WIDE - 1]
    wide = torch.zeros((1, WIDE + 8), dtype=dtype, device="cuda")
    p = wide[:, offset:offset + WIDE]
    p[0, at] = 0.125
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    token = torch.zeros(1, dtype=torch.int64, device="cuda")
    goals = [(k / 8, at[k]) for k in range(8)] + [((k + 1) / 8 - 2.0 ** -53, at[k]) for k in range(8)]
    for u, want in goals + [(1.0, WIDE - 1), (math.nan, WIDE - 1)]:
        out = mx.mx_verify(p, token, torch.tensor([u], dtype=torch.float64, device="cuda"), starts, 1)[2]
        assert out.tolist() == [[want]], u


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("children", [1, 3])
def test_refusals_that_leave_nothing(mx, dtype, children):
    """The last refusal is taken back where no weight would be left, of chains and of trees, with a draft's row and
    without one (whose only weight's token is refused by a number that is none of [0, 1))."""
    nodes = 1 + children
    p = torch.zeros((nodes, WIDE), dtype=dtype, device="cuda")
    p[:, 7], p[:, 33000] = 0.25, 0.5
    q = p.clone()
    q[:, 7] = 0.5
    c = Case([nodes], 5, tree=True, seed=1)
    c.target, c.draft = p, q
    c.tokens = torch.tensor([0, 7, 7, 33000][:nodes], device="cuda")
    up = torch.tensor([-1, 0, 0, 0][:nodes], dtype=torch.int32, device="cuda")
    for parents in (up, None) if children == 1 else (up,):
        c.parents = parents
        for u in (0.0, 0.3, 0.6, 1.0 - 2.0 ** -53):
            c.uniforms = torch.tensor([u, 0.9, 0.75, 1.5][:nodes], dtype=torch.float64, device="cuda")
            want = c.check(c.run(mx))
            assert want[2][0, 0] == (7 if u * 0.75 < 0.25 else 33000)
    c.draft = None
    c.target = torch.zeros((nodes, WIDE), dtype=dtype, device="cuda")
    c.target[:, 33000] = 1.0
    c.tokens = torch.full((nodes,), 33000, device="cuda")
    for parents in (up, None) if children == 1 else (up,):
        c.parents = parents
        c.uniforms = torch.tensor([0.5, 1.0, 1.0, 2.0][:nodes], dtype=torch.float64, device="cuda")
        assert c.check(c.run(mx))[2][0, 0] == 33000


def plain(c, b, first, n):
    """The walk of one sequence in 64 bits: places, tokens, and how near a goal, a test or a sum came to its border
    (relative to what is compared)."""
    near, node, places, out = 1.0, 0, [0], []
    p = c.target.cpu()
    q = None if c.draft is None else c.draft.cpu()
    tokens, uniforms = c.tokens.tolist(), c.uniforms.tolist()
    parents = list(range(-1, n - 1)) if c.parents is None else c.parents[first:first + n].tolist()
    w, total = p[first].double(), 1.0
    for i in range(1, n):
        if parents[i] != node:
            continue
        x = tokens[first + i]
        qx = 1.0 if q is None else float(q[first + node, x])
        side, weight = uniforms[first + i] * total * qx, float(w[x])
        near = min(near, abs(side - weight) / max(side, weight, 1e-300))
        if side < weight:
            node = i
            places.append(i)
            out.append(x)
            w, total = p[first + i].double(), 1.0
            continue
        if q is None:
            w[x] = 0.0
        else:
            w = (w - total * q[first + node].double()).clamp(min=0)
        total = float(w.sum())
        assert total > 0
    cum = w.cumsum(0)
    goal = uniforms[first] * float(cum[-1])
    near = min(near, float((cum - goal).abs().min()) / float(cum[-1]))
    return places, out + [int((cum > goal).float().argmax())], near


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
def test_batches_over_large_vocabularies(mx, dtype, tree, draft):
    """36 sequences of 128003 entries: two shares for each wave of the sums, which are 1152 workgroups' in 256 CUs.

    64-bit sums in another order, and weights whose subtractions are rounded apart, differ by less than 128003 * 2^-53 =
    1.5e-11 of the sum; every border is further from its goal than that, which is asserted."""
    sizes = [3 + b % 3 for b in range(36)]
    c = Case(sizes, 128003, dtype, tree, draft, seed=31, noise=1.5, width=3)
    counts, path, out = (t.cpu() for t in c.run(mx))
    first = 0
    for b, n in enumerate(sizes):
        places, tokens, near = plain(c, b, first, n)
        assert near > 1.5e-11, (b, near)
        k = len(places)
        assert int(counts[b]) == k and path[b].tolist() == places + [-1] * (c.max_q - k), b
        assert out[b].tolist() == tokens + [-1] * (c.max_q - k), b
        first += n


def nodes_with_sums(c, sizes):
    """How many nodes of each sequence a walk can reach with a child behind a refused first one."""
    found, first = [], 0
    p, tokens, u = c.target.cpu(), c.tokens.tolist(), c.uniforms.tolist()
    q = None if c.draft is None else c.draft.cpu()
    for n in sizes:
        up = c.parents[first:first + n].tolist()
        kids = [[i for i in range(1, n) if up[i] == k] for k in range(n)]

        def kept(i):
            x = tokens[first + i]
            return u[first + i] * (1.0 if q is None else float(q[first + up[i], x])) < float(p[first + up[i], x])

        todo, count = [0], 0
        while todo:
            mine = kids[todo.pop()]
            if mine and kept(mine[0]):
                todo.append(mine[0])
            elif mine:
                count += len(mine) > 1
                todo += mine[1:]
        found.append(count)
        first += n
    return found


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("batch", [130, 520])
def test_bushy_trees_of_many_sequences(mx, draft, batch):
    """A sequence has four workgroups for the nodes that need sums, so each has several, one after another."""
    sizes = [64 - b % 7 for b in range(batch)]
    c = Case(sizes, 24, tree=True, draft=draft, seed=batch, noise=3.0)
    up = torch.tensor([(i - 1) // 4 for i in range(64)], dtype=torch.int32)  # four children a node
    c.parents = torch.cat([up[:n] for n in sizes]).to(c.parents.device)
    if draft:
        c.uniforms = 1.0 - c.uniforms / 8  # more children are refused
    need = nodes_with_sums(c, sizes)
    assert max(need) > 8 and sum(n > 4 for n in need) > batch // 2, need
    want = c.check(c.run(mx))
    assert int(want[0].max()) > 2  # and walks go on behind refused children


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("vocab", [24, WIDE])
def test_starts_that_do_not_ascend(mx, draft, vocab):
    """Sequences that share nodes: what comes out is not defined, but it is a walk through places of the sequence."""
    c = Case([40, 30, 50], vocab, tree=True, draft=draft, seed=5, noise=1.0)
    c.q_starts = torch.tensor([0, 60, 20, 110, 7, 200, -5, 120], dtype=torch.int32, device="cuda")
    counts, path, out = (t.cpu() for t in c.run(mx, max_q=64))
    starts = c.q_starts.tolist()
    for b in range(7):
        first = max(starts[b], 0)
        n = min(max(min(starts[b + 1], 120) - first, 0), 64)
        k = int(counts[b])
        assert (1 if n else 0) <= k <= n
        places = path[b].tolist()
        assert places[k:] == [-1] * (64 - k) and places[:k] == sorted(set(places[:k]))
        if n:
            assert places[0] == 0 and max(places) < n
            assert out[b, :k - 1].tolist() == [int(c.tokens[first + i]) for i in places[1:k]]
            assert -1 <= int(out[b, k - 1]) < vocab
