"""Limits of the node operators that are decided on the host."""
import pytest

from test_nodes_cpu import ARG, attn, fc  # noqa: F401


@pytest.mark.parametrize("vjp", [False, True])
def test_attention_refuses_structures_that_the_tile_search_cannot_count(fc, vjp):  # noqa: F811
    """The search for a tile's structure looks up to 31 places past n_struct + 1 in 32 bits."""
    for b in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 3, 2 ** 31 - 64):
        assert attn(fc, vjp, b=b) == ARG, b
