"""mx_cache_cross_attention: every query sees all tokens of its sequence, so each is checked as a sequence of its own
against softmax in 64 bits, with the bound of the causal calls."""
import pytest
import torch

import _cacheref as R
from test_gpu_cache_attention import Case, mx  # noqa: F401 (mx is a fixture)

pytestmark = pytest.mark.gpu


def run(mx, c, **kw):
    f = dict(max_q=max(c.nq), max_kv=max(c.kv))
    return mx.mx_cache_cross_attention(c.cache, c.q, c.q_starts, c.kv_lens, c.table, **{**f, **kw})


def check(c, out, max_kv=None, scale=None):
    owner = torch.tensor([b for b, n in enumerate(c.nq) for _ in range(n)], device="cuda", dtype=torch.long)
    lens = (c.kv_lens if max_kv is None else c.kv_lens.clamp(max=max_kv))[owner]
    starts = torch.arange(len(owner) + 1, dtype=torch.int32)
    n = len(owner)
    ref, weight, size = R.attention(c.cache, c.q[:n], starts, lens, c.table[owner], None, scale)
    got = out[:n].double().cpu()
    # weights that are off by e_i of themselves, in the products and in their sum, move the result by up to the largest
    # e_i times (sum w |v| + |out|)
    bound = R.attention_bound(ref, weight + ref.abs(), size, ref.shape[2], max(c.kv))
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    over = torch.where(torch.isnan(ref), 0.0, (got - ref).abs() - bound)
    assert float(over.max()) <= 0, float(over.max())
    assert not bool(out[n:].any())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group,nq,kv", [(1, 1, 77), (4, 1, 1), (2, 9, 5), (5, 12, 130), (3, 45, 20), (1, 150, 3)])
def test_heads_and_rows(mx, fmt, dim, group, nq, kv):
    """More queries than tokens, fewer, one of either."""
    c = Case(mx, fmt, 2, group, dim, 16, [kv, kv // 2 + 1], [nq, max(1, nq // 2)], seed=dim + nq)
    check(c, run(mx, c))


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 63, 64, 65, 257, 1000])
@pytest.mark.parametrize("nq", [1, 40])
def test_lengths_and_pages(mx, page, kv, nq):
    c = Case(mx, 1, 1, 2, 64, page, [kv], [nq], seed=kv)
    check(c, run(mx, c))


@pytest.mark.parametrize("fmt,dim,group,nq", [(0, 64, 1, 1), (1, 128, 4, 1), (1, 64, 2, 30), (0, 256, 1, 3)])
def test_splits_and_ragged(mx, fmt, dim, group, nq):
    """Sequences over several workgroups' spans; one without tokens gives zeros, one without queries nothing."""
    c = Case(mx, fmt, 2, group, dim, 32, [5000, 1, 0, 300, 2600], [nq, 2, 3, 0, nq], seed=dim)
    out = run(mx, c)
    check(c, out)
    assert not bool(out[nq + 2:nq + 5].any())


@pytest.mark.parametrize("fmt,dim,group,nq,kv", [(1, 64, 1, 200, 3000), (0, 128, 4, 60, 2000), (1, 96, 1, 300, 4096),
                                                 (1, 64, 2, 1, 4000), (0, 256, 2, 70, 2500)])
def test_few_sequences_of_some_thousand_tokens(mx, fmt, dim, group, nq, kv):
    """Divided calls below the length from which all calls are divided: their blocks, and so their workspace, are not
    those of the causal calls."""
    c = Case(mx, fmt, 2, group, dim, 64, [kv, kv // 3], [nq, nq], seed=kv)
    check(c, run(mx, c))


def test_bounds_scale_and_padding(mx):
    c = Case(mx, 1, 2, 2, 64, 16, [400, 70, 9], [20, 3, 1], seed=2)
    check(c, run(mx, c, scale=0.3), scale=0.3)
    check(c, run(mx, c, max_kv=65), max_kv=65)
    c.q = torch.cat((c.q, c.q[:5]))  # queries of no sequence
    check(c, run(mx, c))


def test_pages_outside_the_cache_are_not_seen(mx):
    for nq in (2, 60):
        c = Case(mx, 1, 1, 2, 64, 16, [100, 40], [nq, 1], seed=9)
        c.table[0, 2], c.table[0, 5], c.table[1, 0] = -1, 1 << 20, c.cache.pages
        check(c, run(mx, c))
        c.table[1] = -1
        out = run(mx, c)
        check(c, out)
        assert not bool(out[nq:].any())


@pytest.mark.parametrize("nq", [1, 60])
def test_nan_behind_the_sequence_stays_there(mx, nq):
    c = Case(mx, 1, 2, 2, 128, 64, [70, 64], [nq, nq], seed=11)
    for b, n in enumerate(c.kv):
        page = int(c.table[b, n // 64]) if n % 64 else -1
        if page >= 0:
            for t in (c.cache.k_codes, c.cache.v_codes):
                t[page, :, n % 64:] = 127
            for t in (c.cache.k_scales, c.cache.v_scales):
                t[page, :, :, n % 64:] = 255
    out = run(mx, c)
    assert bool(torch.isfinite(out).all())
    check(c, out)
    c.cache.v_scales[int(c.table[1, 0]), 0, 0, 5] = 255  # one that every query of the second sequence sees
    out = run(mx, c)
    assert bool(torch.isnan(out[nq:, :2, :32]).all()) and bool(torch.isfinite(out[:nq]).all())
    check(c, out)


def test_one_query_is_the_causal_call(mx):
    """It is the last token then, so both calls have the same value (their work may be divided in other ways)."""
    c = Case(mx, 0, 2, 4, 128, 32, [700, 31, 64], [1, 1, 1], seed=3)
    c.check(run(mx, c))
    check(c, c.run(mx))


def test_streams_and_replays(mx):
    c = Case(mx, 1, 2, 2, 64, 16, [1500, 800], [7, 30], seed=5)
    eager = run(mx, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run(mx, c)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(again, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(mx, c)
    for _ in range(3):
        held.zero_()
        graph.replay()
        run(mx, c)
        torch.cuda.synchronize()
        assert torch.equal(held, eager)
