"""Router tiles whose hidden size is shared by several workgroups: sizes that no share divides, one token tile
and several, few experts and many.  The bounds are those of the other tests of the layer."""

import pytest

from tests.test_gpu_moe import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T, D, E, k", [(16, 4104, 8, 2), (9, 8200, 7, 3), (64, 2056, 17, 4), (33, 4120, 16, 16), (5, 6152, 130, 8),
                                        (1, 12296, 40, 5), (16, 1032, 300, 8)])
def test_shared_hidden_size(T, D, E, k, dtype):
    c = Case(T, D, 8, E, k, dtype=dtype, renorm=T % 2 == 0)
    layer = c.layer(max_tokens=64)
    ws = layer.new_workspace()
    first = c.run(layer, ws)
    c.check(first)
    again = c.run(layer, ws)                       # the same workspace, the same bits
    assert all((a == b).all() for a, b in zip(first, again))


def test_ties_across_shares_go_to_the_lowest_index():
    """Equal rows of the router give equal logits whatever the shares add up, so the picks are the first ones."""
    c = Case(16, 4096, 8, 12, 4)
    c.router[:] = c.router[:1]
    c.rb[:] = c.rb[:1]
    _, ids, _ = c.run(c.layer(max_tokens=16))
    assert (ids == [0, 1, 2, 3]).all()
