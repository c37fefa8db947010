"""Bounds of attention over the paged MX cache that differ from what the sequences hold: max_q and max_kv below the
sequences' sizes, queries of no sequence, batches of one long chunk and many single tokens."""
import pytest
import torch

from _attentionref import check
from test_gpu_cache_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from microscaling_quantize_dequantize_amd import binding
    return binding


def attend(mx, c, max_q, max_kv, out=None):
    return mx.mx_cache_attention(c.cache, c.q, c.q_starts, c.kv_lens, c.table, max_q=max_q, max_kv=max_kv, tree=c.tree,
                                 out=out)


@pytest.mark.parametrize("group,nq", [(1, 10), (2, 12), (8, 40), (4, 90)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("cut_q,cut_kv", [(True, False), (False, True), (True, True)])
def test_bounds_below_the_sizes(mx, group, nq, tree, cut_q, cut_kv):
    """What is beyond max_q and max_kv is left out; the rows that are computed see no token that they should not."""
    c = Case(mx, 1, 2, group, 64, 16, [50 + nq, nq, 900], [nq, nq, nq // 2], seed=nq)
    if tree:
        c.random_tree()
    max_q = nq // 2 - 1 if cut_q else nq
    max_kv = 40 + nq // 2 if cut_kv else 900
    out = attend(mx, c, max_q, max_kv, out=torch.zeros_like(c.q, memory_format=torch.contiguous_format))
    check(c, out, max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("group,nq", [(2, 5), (8, 40)])
def test_tokens_behind_the_table_are_not_seen(mx, group, nq):
    c = Case(mx, 1, 2, group, 64, 16, [700, 300], [nq, nq], seed=3)
    c.table = c.table[:, :20].contiguous()
    out = c.run(mx)
    c.table = torch.cat((c.table, c.table.new_full((2, 24), -1)), 1)  # the reference takes no part of them
    check(c, out)


@pytest.mark.parametrize("group,nq,kv", [(1, 1, 30), (4, 1, 9000), (4, 30, 400), (8, 70, 3000)])
@pytest.mark.parametrize("spare", [1, 57])
def test_queries_of_no_sequence_give_zeros(mx, group, nq, kv, spare):
    """A batch padded at its end: rows from q_starts[batch] on are written, and nothing else changes."""
    c = Case(mx, 1, 2, group, 64, 16, [kv, 17], [nq, 1], seed=spare)
    want = c.run(mx)
    c.q = torch.cat((c.q, torch.full((spare, *c.q.shape[1:]), float("nan"), device="cuda").bfloat16()))
    out = torch.full(c.q.shape, float("nan"), device="cuda").bfloat16()
    c.run(mx, out=out)
    assert torch.equal(out[:nq + 1], want)
    assert not bool(out[nq + 1:].any())


@pytest.mark.parametrize("batch", [0, 2])
def test_only_padding(mx, batch):
    c = Case(mx, 1, 2, 2, 64, 16, [40, 9], [0, 0], seed=1)
    q = torch.ones((5, 4, 64), device="cuda").bfloat16()
    out = torch.full(q.shape, float("nan"), device="cuda").bfloat16()
    mx.mx_cache_attention(c.cache, q, c.q_starts[:batch + 1], c.kv_lens[:batch], c.table[:batch], max_q=0, max_kv=40,
                          out=out)
    assert not bool(out.any())


@pytest.mark.parametrize("batch,heads,group,chunk,dim,fmt", [(1024, 8, 8, 1024, 64, 1), (60, 4, 4, 500, 128, 0),
                                                             (300, 2, 3, 40, 256, 1), (900, 2, 2, 1, 64, 1)])
def test_one_chunk_among_single_tokens(mx, batch, heads, group, chunk, dim, fmt):
    """Bounds that give every sequence the long one's blocks: far more items than there are, or than workgroups."""
    kv = [1 + (37 * b) % 60 for b in range(batch)]
    new = [1] * batch
    kv[3], kv[batch - 2] = 1500, 700
    kv[7], new[7] = 1100 + chunk // 8, chunk
    c = Case(mx, fmt, heads, group, dim, 16, kv, new, seed=batch)
    check(c, c.run(mx), device="cuda")
