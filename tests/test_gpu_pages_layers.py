"""Caches of several layers behind one table: forked once, the other layers copy the last pages by the two tables."""
import pytest
import torch

from test_gpu_pages import I32, NAMES, cache_of, check_resize, fork, i32, mx, resize, same, snapshot, token  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,page,dim", [(1, 16, 32), (3, 32, 96)])
def test_layers_behind_one_table(mx, heads, page, dim):
    """Lengths in the middle of a page, at its end, a whole row, one token, none; the pool is too small for the last
    child."""
    layers = [cache_of(mx, 1, 18, heads, page, dim, seed=k) for k in range(3)]
    lens = [2 * page + 5, page, 4 * page, 1, 0, 3 * page + page - 1]
    refs, table = [0] * 18, [[-1] * 4 for _ in lens]
    resize(refs, table, lens, page)
    parents = [0, 1, 2, 3, 4, 5, 0, 5, 3]
    r, t, n, p = i32(refs), i32(table), i32(lens), i32(parents)
    before = [snapshot(c) for c in layers]
    rows, missing = mx.mx_cache_fork(layers[0], r, t, n, p)
    last = (n[p] // page).clamp(max=3).long()[:, None]
    src, dst = (x.gather(1, last)[:, 0] for x in (t[p], rows))
    for c in layers[1:]:
        mx.mx_cache_copy(c, src, dst)
    want, lack = fork(refs, table, lens, parents, page, before[0])
    assert rows.tolist() == want and missing.tolist() == lack and r.tolist() == refs
    assert any(lack) and 0 in lack
    same(layers[0], before[0])
    for c, data in zip(layers[1:], before[1:]):
        whole = {k: data[k].clone() for k in NAMES}
        for child, s in enumerate(parents):
            j = lens[s] // page
            if lens[s] % page and want[child][j] >= 0:
                for name in NAMES:
                    whole[name][want[child][j]] = data[name][table[s][j]]
        same(c, whole)
        # every token of a child that has all of its pages is its parent's
        for child, s in enumerate(parents):
            if lack[child] == 0:
                for i in range(lens[s]):
                    for name in NAMES:
                        assert torch.equal(token(whole[name], name, want[child][i // page], i % page),
                                           token(data[name], name, table[s][i // page], i % page))
