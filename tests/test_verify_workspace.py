"""The workspace of mx_verify follows the nodes that there are, not the most that every sequence could have."""
from test_cache_checks import ESHAPE, b, mx  # noqa: F401


def test_bytes_follow_the_nodes(b):
    space = b.raw().mx_verify_workspace
    for vocab in (1000, 32768, 128001):
        base = space(1000, 0, 1024, vocab)
        # an end of 24 bytes and a sum of 8 for each share of 1024 entries, of which there are 4 to 8 too many at most,
        # or 16 or 32 of a row that is one workgroup's
        shares = max(32, vocab // 1024 + 9)
        assert 0 < base <= 1000 * (24 + 8 * shares)
        for nodes in (1, 6, 5001):
            for max_q in (1, 6, 1024):
                assert base < space(1000, nodes, max_q, vocab) <= base + 28 * nodes + 4
    # a batch of short chains with a generous bound
    assert space(1 << 20, 1 << 22, 1024, 1000) < 1 << 29
    assert space(1 << 22, 0, 0, 1000) == ESHAPE
