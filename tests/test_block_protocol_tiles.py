"""The barriers of the CTA pairs' products where the tiles' edges matter most: several tiles whose K blocks are 3 mod 4 in
number.  An issuing warp then takes an accumulator slot 7 blocks after its last use, the farthest that occurs, and both
warps take the same stage by turns."""
import pytest

from tests.test_block_protocol import Broken, _constants, simulate


@pytest.mark.parametrize("blocks", [7, 11, 15])
def test_pairs(blocks):
    _, pair = _constants()
    for seed in range(100):
        simulate(seed, pair[128], 4, [blocks] * 4, late=0.5)
        simulate(seed, pair[256], 4, [blocks] * 4, halves=2, late=0.5)


@pytest.mark.parametrize("blocks", [7, 11, 15])
def test_the_model_sees_a_ring_that_is_too_short(blocks):
    """With four stages the slot's wait says nothing about a stage's last fill, and a wait passes on the fill before; one
    tile alone does not show it."""
    with pytest.raises(Broken):
        for seed in range(300):
            simulate(seed, 4, 4, [blocks] * 4, late=0.5)
    for seed in range(100):
        simulate(seed, 4, 4, [57], late=0.5)
