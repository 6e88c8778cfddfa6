"""The size of a tree attention workspace (CPU)."""
import itertools

import pytest


@pytest.fixture(scope="module")
def fd():
    from decode_attention_decoding_gb300 import build
    build.build()
    import decode_attention_decoding_gb300 as fd
    return fd


def test_a_tree_workspace_serves_every_smaller_shape(fd):
    """The size grows with the batch, the query rows of a kv head (nodes x group) and the head dim, each alone or together."""
    batches, dims = (1, 33, 4096), (64, 128, 256)
    trees = (1, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256)
    groups = (1, 2, 4, 7, 16)
    shapes = [(b, t * g, d) for b, t, g, d in itertools.product(batches, trees, groups, dims)]
    size = {(b, t * g, d): fd.fd_tree_workspace_size(b, t, 3 * g, 3, d) for b, t, g, d in itertools.product(batches, trees, groups, dims)}
    assert all(size.values())
    for small, large in itertools.product(set(shapes), repeat=2):
        if all(x <= y for x, y in zip(small, large)):
            assert size[small] <= size[large], (small, large)
